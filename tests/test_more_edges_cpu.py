"""Edges of the adapters' and the token scores' bindings that need no GPU."""

import numpy as np
import pytest
import torch

from wfst_beam_search_amd import score

CPU = torch.device("cpu")


@pytest.mark.parametrize("kind", [np.uint8, np.uint16, np.uint32, np.uint64, np.int8, np.int64])
def test_host_ids_of_every_integer_type(kind):
    lead = torch.Size((3, 5))
    t, per = score._ids(np.array([0, 2, 1], kind), lead, 3, CPU, None)
    assert t.dtype == torch.int32 and t.tolist() == [0, 2, 1] and per == 5
    top = np.iinfo(kind).max                        # (past the slots; of uint64 past 63 bits too)
    for bad in (3, top):
        with pytest.raises(ValueError, match="below 3"):
            score._ids(np.array([0, bad, 1], kind), lead, 3, CPU, None)
    if np.iinfo(kind).min < 0:
        assert score._ids(np.array([np.iinfo(kind).min, 0, -1], kind), lead, 3, CPU, None)[0].tolist() == [-1, 0, -1]


def test_host_ids_in_torch_tensors():
    lead = torch.Size((3, 5))
    t, per = score._ids(torch.tensor([0, 1, 1], dtype=torch.uint8), lead, 3, CPU, None)
    assert t.dtype == torch.int32 and t.tolist() == [0, 1, 1] and per == 5
    t, per = score._ids(torch.tensor(2, dtype=torch.uint8), lead, 3, CPU, None)
    assert t.shape == () and int(t) == 2 and per == 15
