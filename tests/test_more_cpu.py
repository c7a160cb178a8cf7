"""Refusals of the adapters and the token scores that need no GPU, their C structs, and the 64-bit definitions the
GPU tests compare with, on cases worked out by hand."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import more_ref as ref
import wfst_beam_search_amd as wb
from wfst_beam_search_amd import score

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL = -1


@pytest.fixture(scope="module")
def lib():
    return wb.load_library()


@pytest.mark.parametrize("name,cls", [("wfst_adapters_desc", score._AdaptersDesc),
                                      ("wfst_token_scores_out", score._TokenScoresOut)])
def test_structs_match_header(name, cls):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "wfst.h")).read(), flags=re.S)
    body = re.search(r"typedef struct " + name + r"\s*\{(.*?)\}\s*" + name + ";", src, flags=re.S).group(1)
    fields = re.findall(r"([A-Za-z_][A-Za-z0-9_ ]*?[\s*]+)([a-z_]+)\s*;", body)
    assert [f for _, f in fields] == [f for f, _ in cls._fields_]
    for (ctype, fname), (_, ptype) in zip(fields, cls._fields_):
        assert (ctypes.c_void_p if "*" in ctype else ctypes.c_int32) is ptype, fname


@pytest.mark.parametrize("bad,word", [
    (dict(in_features=0), "in_features"), (dict(in_features=(1 << 24) + 1), "in_features"),
    (dict(out_features=-1), "out_features"), (dict(slots=0), "slots"), (dict(slots=(1 << 16) + 1), "slots"),
    (dict(rank=0), "rank"), (dict(rank=129), "rank"), (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype")])
def test_adapters_create_refuses(lib, bad, word):
    d = dict(in_features=64, out_features=8, slots=2, rank=4, dtype=2)
    d.update(bad)
    h = ctypes.c_void_p()
    desc = score._AdaptersDesc(*(d[n] for n, _ in score._AdaptersDesc._fields_))
    assert lib.wfst_adapters_create(ctypes.byref(desc), 0, None, ctypes.byref(h)) == EINVAL
    assert word in lib.wfst_last_error().decode() and not h.value


def test_adapters_refuse_null(lib):
    n = ctypes.c_int64()
    assert lib.wfst_adapters_create(None, 0, None, ctypes.byref(ctypes.c_void_p())) == EINVAL
    assert lib.wfst_adapters_load(None, 0, 1, 4096, 8, 4096, 8, 1.0, None) == EINVAL
    assert lib.wfst_adapters_release(None) == 0
    assert lib.wfst_layer_adapted_workspace(None, None, 0, 1, ctypes.byref(n)) == EINVAL
    assert lib.wfst_layer_adapted_logits(None, None, 4096, 1, 4096, 0, 8, 1, None, 1, 4096, 0, 8, None, 0, None) == EINVAL


@pytest.mark.parametrize("kw,word", [
    (dict(xt=9), "type"), (dict(rows=-1), "rows"), (dict(V=0), "V"), (dict(V=(1 << 24) + 1), "V"),
    (dict(C=-1), "tokens_per_row"), (dict(C=257), "tokens_per_row"), (dict(n=-1), "top_n"), (dict(n=65), "top_n"),
    (dict(T=-0.5), "temperature"), (dict(T=float("nan")), "temperature"), (dict(T=float("inf")), "temperature"),
    (dict(x=None), "null"), (dict(tok=None), "null"), (dict(lp=None), "null"), (dict(rank=None), "null"),
    (dict(tt=None), "null"), (dict(tl=None), "null"), (dict(xs=7), "stride"), (dict(xs=1 << 61), "large")])
def test_token_scores_refuse(lib, kw, word):
    a = dict(x=4096, xt=0, xs=8, rows=2, V=8, tok=8192, C=1, n=2, T=1.0, lp=12288, rank=16384, ent=20480, tt=24576, tl=28672)
    a.update(kw)
    out = score._TokenScoresOut(a["lp"], a["rank"], a["ent"], a["tt"], a["tl"])
    rc = lib.wfst_token_scores(a["x"], a["xt"], a["xs"], a["rows"], a["V"], a["tok"], a["C"], a["n"], a["T"], None, None,
                               1, ctypes.byref(out), None, 0, None)
    assert rc == EINVAL and word in lib.wfst_last_error().decode()


def test_token_scores_without_rows_or_out(lib):
    out = score._TokenScoresOut()
    args = (None, 0, 8, 0, 8, None, 1, 0, 1.0, None, None, 1)
    assert lib.wfst_token_scores(*args, ctypes.byref(out), None, 0, None) == 0
    assert lib.wfst_token_scores(*args, None, None, 0, None) == EINVAL
    n = ctypes.c_int64()
    assert lib.wfst_token_scores_workspace(0, 4, 8, 1, 65, ctypes.byref(n)) == EINVAL
    assert lib.wfst_token_scores_workspace(0, 4, 8, 1, 64, None) == EINVAL
    assert lib.wfst_token_scores_workspace(0, 4, 8, 1, 64, ctypes.byref(n)) == 0 and n.value >= 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(TypeError, match="GPU"):
        wb.token_scores(x, torch.zeros(2, dtype=torch.int32))
    layer = type("Layer", (), dict(in_features=8, out_features=4, device=torch.device("cuda", 0)))
    ad = object.__new__(wb.Adapters)
    ad.handle = None
    with pytest.raises(ValueError, match="released"):
        ad._check_layer(layer)
    with pytest.raises(ValueError, match="dtype"):
        wb.Adapters(layer, 1, 1, dtype="f64")


def test_ids_geometry(monkeypatch):
    cpu = torch.device("cpu")
    lead = torch.Size((3, 5))
    for ids, per in (([0, 1, -1], 5), (np.zeros((3, 5), np.int64), 1), (2, 15)):
        t, p = score._ids(ids, lead, 3, cpu, None)
        assert t.dtype == torch.int32 and p == per
    assert score._ids([2, -2 ** 40, 0], lead, 3, cpu, None)[0].tolist() == [2, -1, 0]
    assert score._ids([], torch.Size((0, 5)), 3, cpu, None)[0].shape == (0,)
    for bad in ([0, 1], [0, 1, 3], [0.5, 0, 0], [0, 1, 2 ** 32], np.zeros((5, 3), np.int32), None):
        with pytest.raises(ValueError):
            score._ids(bad, lead, 3, cpu, None)


def test_reference_scores_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 4.0, 1.0]))          # probabilities 1/12, 4/12, 2/12, 4/12, 1/12
    lp, rank, ent, tt, tl = ref.scores_row(x, np.array([0, 3, 4, 5, -1]), 3)
    assert np.allclose(lp[:3], np.log([1 / 12, 4 / 12, 1 / 12])) and (lp[3:] == -np.inf).all()
    assert rank.tolist() == [3, 1, 4, -1, -1] and tt.tolist() == [1, 3, 2]
    p = np.array([1, 4, 2, 4, 1]) / 12
    assert np.isclose(ent, -(p * np.log(p)).sum()) and np.allclose(tl, np.log(p[[1, 3, 2]]))
    lp, rank, ent, tt, tl = ref.scores_row(x, np.array([1, 3]), 7, T=0.0)
    assert lp.tolist() == [0.0, -np.inf] and ent == 0.0 and tt.tolist() == [1, 3, 2, 0, 4, -1, -1]
    lp = ref.scores_row(x, np.array([2]), 0, T=2.0)[0]       # masses sqrt: 1, 2, sqrt 2, 2, 1
    assert np.isclose(lp[0], np.log(np.sqrt(2) / (6 + np.sqrt(2))))
    lp, rank, ent, tt, tl = ref.scores_row(np.array([-np.inf, np.nan, 1.0, np.inf]), np.array([0, 1, 2]), 3)
    assert np.isnan(lp).all() and rank.tolist() == [2, 3, 1] and tt.tolist() == [3, 2, -1] and tl[2] == -np.inf
    lp, rank, ent, tt, tl = ref.scores_row(np.full(3, -np.inf), np.array([1]), 1)
    assert lp[0] == -np.inf and rank[0] == 1 and ent == 0.0 and tt[0] == -1


def test_reference_adapters_by_hand():
    down, up = np.array([[1.0, 2.0], [0.0, -1.0]]), np.array([[1.0, 0.0], [2.0, 3.0], [0.0, 1.0]])
    y, size = ref.adapters(np.array([[1.0, 1.0], [1.0, 1.0]]), [4, -1], {4: (down, up, 0.5)})
    assert y[0].tolist() == [1.5, 1.5, -0.5] and size[0].tolist() == [1.5, 4.5, 0.5] and not y[1].any()
