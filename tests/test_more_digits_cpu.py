"""The check of h's digits (more_digits.py) sees each part that would be missing."""

import numpy as np
import pytest

import more_digits as digits


def _cut16(v):
    return (np.float32(v).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)


def _parts(h, a):
    """h in binary32 as the parts that meet up, in 64 bits each."""
    h = np.float32(h)
    if a == "f32":
        return [h.astype(np.float64)]
    if a == "bf16":
        one = _cut16(h)
        two = _cut16(h - one)
        return [p.astype(np.float64) for p in (one, two, h - one - two)]
    e = np.frexp(np.abs(h))[1] - 15
    s = np.ldexp(h.astype(np.float64), -e)
    hi = s.astype(np.float16)
    lo = ((s - hi) * 2048).astype(np.float16)
    return [np.ldexp(hi.astype(np.float64), e), np.ldexp(lo.astype(np.float64) / 2048, e)]


@pytest.mark.parametrize("x,a", [("f32", "f32"), ("f32", "f16"), ("f16", "f16"), ("f32", "bf16"), ("bf16", "bf16")])
def test_a_missing_part_is_seen(x, a):
    xs, _, up = digits.inputs(1, 40, 70, 40, 64, x, a)
    h, want = digits.exact(xs, up)
    parts = _parts(h, a)
    w = up.double().numpy().T[np.arange(40)]
    assert not digits.wrong(sum(parts)[:, None] * w, want).any()
    for k in range(1, len(parts)):                  # cut behind k parts: nearly every row is off
        assert digits.wrong(sum(parts[:k])[:, None] * w, want).any(1).mean() > 0.8
        assert digits.wrong((sum(parts) - parts[k])[:, None] * w, want).any(1).mean() > 0.8
