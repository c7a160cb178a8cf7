"""GPU parity of the operators around the search (output layer with 4-bit
weights, log-softmax, draw of tokens) with their 64-bit definitions
(score_ref.py), and of a run of them into the search.

Tolerances, from the arithmetic (h = half a step of the output's type,
e = 2^-23 bounds any single binary32 rounding, also one that truncates):
* layer: every term passes at most 32 additions inside a matrix instruction, one
  more per 32 features and a few for the scale and the bias, and a binary32 x is
  off by 2^-24 of itself or, next to a 2^23 times larger neighbour, less than
  that of the neighbour: |y - exact| <= h |y| + (K / 32 + 40) e S + tiny, S the
  sum of the absolute terms.
* log-softmax: z is rounded twice, its distance from the maximum and the result
  once; an exponential is off by about its argument's rounding, whose mean under
  the row's own distribution is at most ln V: |out - exact| <= h |out| + 4 e
  (max |z| + |out| + ln V + 8 + V / 1024).
* draw: tokens and counts equal; the log-probability is a binary64 number
  rounded once.
"""

import numpy as np
import pytest
import torch

import score_ref as ref
import synth
import wfst_beam_search_amd as wb
from gpu_util import compare_batch, oracle_lanes

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -23


def _say(*a):
    print(*a, flush=True)


def _np(t):
    return t.detach().double().cpu().numpy()


def _half(dtype):
    return torch.finfo(DT[dtype]).eps / 2


# ---------------------------------------------------------------- output layer

def _layer_arrays(seed, K, N, group, scale="f16", zeros=False, bias=False):
    rng = np.random.default_rng(seed)
    w = rng.integers(0, 256, (N, (K + 1) // 2), dtype=np.uint8)
    ng = -(-K // group)
    s = torch.from_numpy(((0.5 + rng.random((N, ng))) / np.sqrt(K)).astype(np.float32)).to(DT[scale])
    z = rng.integers(0, 16, (N, ng), dtype=np.uint8) if zeros else None
    b = rng.normal(size=N).astype(np.float32) if bias else None
    layer = wb.OutputLayer(torch.from_numpy(w).cuda(), s.cuda(), zeros=None if z is None else torch.from_numpy(z).cuda(),
                           bias=None if b is None else torch.from_numpy(b).cuda(), in_features=K, group_size=group)
    return layer, (w, s.double().numpy(), z, b, K, group)


def _layer_check(y, x, arrays, out):
    want, size = ref.layer(_np(x).reshape(-1, arrays[4]), *arrays)
    got = _np(y).reshape(want.shape)
    sub = 2.0 ** -25 if out == "f16" else 1e-38           # half a step of the smallest numbers
    tol = _half(out) * np.abs(want) * 1.001 + (arrays[4] / 32 + 40) * E * size + sub
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("M,K,N,group,x,scale,out,zeros,bias", [
    (1, 32, 1, 32, "f16", "f16", "f32", False, False),
    (1, 1, 3, 32, "f32", "f32", "f32", True, True),
    (3, 127, 17, 64, "bf16", "bf16", "bf16", True, False),
    (16, 128, 64, 128, "f16", "f32", "f16", False, True),
    (17, 513, 65, 32, "f32", "f16", "f32", True, True),
    (33, 640, 130, 256, "bf16", "f16", "f32", False, True),
    (64, 1024, 250, 1024, "f16", "bf16", "f32", True, False),
    (65, 1025, 129, 96, "f32", "bf16", "f16", False, False),
    (130, 300, 40, 160, "bf16", "f32", "f32", True, True),
    (1, 4096, 200, 128, "bf16", "f16", "f32", False, False),
    (2, 8200, 70, 64, "f16", "f16", "f32", True, True),
    (5, 20000, 33, 128, "f32", "f16", "f32", True, False),
    (300, 257, 515, 32, "bf16", "f16", "f16", True, True),
    # enough workgroups of many rows
    (17, 300, 16500, 64, "bf16", "f16", "f32", True, True),
    (32, 130, 16400, 32, "f16", "f32", "f32", False, False),
    (64, 390, 17001, 32, "f32", "f32", "f16", True, True),
    (3, 2050, 16500, 64, "f32", "f16", "f32", True, True),
    (16, 2049, 16490, 128, "bf16", "f32", "bf16", False, True),
    (5, 2100, 16400, 32, "f16", "bf16", "f32", True, False),
    (65, 1, 8200, 128, "f32", "f16", "f32", True, False),
    (1000, 257, 1100, 96, "f16", "bf16", "bf16", True, False),
    (777, 512, 1300, 128, "bf16", "bf16", "f32", False, True),
])
def test_layer(M, K, N, group, x, scale, out, zeros, bias):
    _say("layer", M, K, N, group, x, scale, out)
    layer, arrays = _layer_arrays(M * K + N, K, N, group, scale, zeros, bias)
    h = torch.from_numpy(np.random.default_rng(K).normal(size=(M, K)).astype(np.float32)).to(DT[x]).cuda()
    _layer_check(layer.logits(h, dtype=out), h, arrays, out)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_layer_strides_lengths_and_untouched_rows(x):
    K, N, B, T = 200, 45, 3, 7
    layer, arrays = _layer_arrays(5, K, N, 64, bias=True)
    buf = torch.randn(B, T, K + 13, device="cuda").to(DT[x])
    h = buf[:, :, 3:3 + K]
    wide = torch.full((B, T, N + 9), 77.0, device="cuda")
    L = torch.tensor([7, 0, 4], dtype=torch.int32, device="cuda")
    layer.logits(h, lengths=L, out=wide[:, :, 4:4 + N])
    got = wide.cpu()
    assert (got[:, :, :4] == 77).all() and (got[:, :, 4 + N:] == 77).all()
    for b, n in enumerate([7, 0, 4]):
        assert (got[b, n:] == 77).all()
        if n:
            _layer_check(got[b, :n, 4:4 + N], h[b, :n].contiguous(), arrays, "f32")
    y = layer.logits(h, lengths=[7, 0, 4])                  # host lengths
    assert torch.equal(y[0], wide[0, :, 4:4 + N]) and torch.equal(y[2, :4], wide[2, :4, 4:4 + N])


@pytest.mark.parametrize("x,values", [
    ("f16", [6e-8, -6e-8, 1.2e-7, 6e-5, 65504.0]),
    ("bf16", [1e-38, 1e30, -3e38, 1e-30, 2.0]),
    ("bf16", [1e-38, -2e-38, 3e-36, 1.1e-38, 1e-37]),
    ("f32", [1e-38, 1e30, -3e37, 1.0000001, 16777217.0]),
    ("f32", [1.0, 1.0 + 2.0 ** -23, 2.0 ** -20, -1.0 - 2.0 ** -22, 2.0 ** -30]),
])
def test_layer_extreme_values(x, values):
    """Subnormal and huge hidden states, one block of features holding both."""
    K, N = 256, 20
    layer, arrays = _layer_arrays(9, K, N, 32, "f32")
    h = torch.zeros(4, K)
    rng = np.random.default_rng(2)
    for r in range(4):
        for v in values:
            h[r, int(rng.integers(0, K))] = v
    h = h.to(DT[x])
    y = layer.logits(h.cuda())
    want, size = ref.layer(_np(h), *arrays)
    big = np.abs(_np(h)).max() * 2.0 ** -38 * 16 * K
    big = big if x == "f32" else (big * 2.0 ** -1 if x == "bf16" else 0.0)
    tol = (K / 32 + 40) * E * size + np.abs(want) * 2.0 ** -24 + big * np.abs(arrays[1]).max() + 1e-41
    assert (np.abs(_np(y) - want) <= tol).all()


def test_layer_infinities_and_nan_stay_in_their_rows():
    K, N = 300, 50
    for x, M in (("f32", 5), ("f16", 5), ("bf16", 5), ("f32", 2100), ("bf16", 2100)):
        N = 50 if M == 5 else 600
        layer, arrays = _layer_arrays(11, K, N, 64, zeros=True, bias=True)
        h = torch.randn(M, K).to(DT[x])
        clean = layer.logits(h.cuda())
        h[1, 17], h[3, 299], h[4, 0] = float("inf"), float("nan"), float("-inf")
        y = layer.logits(h.cuda()).cpu()
        assert torch.equal(y[0], clean[0].cpu()) and torch.equal(y[2], clean[2].cpu())
        w = ref.unpack(arrays[0], K) - arrays[2].astype(np.int64)[:, np.arange(K) // 64]
        for r, k, sign in ((1, 17, 1), (4, 0, -1)):
            d = w[:, k]
            assert np.array_equal(np.isnan(_np(y[r])), d == 0)
            assert (_np(y[r])[d != 0] == sign * np.sign(d[d != 0]) * np.inf).all()
        assert torch.isnan(y[3]).all()


def test_layer_many_rows_lengths():
    """A padded batch on the many-row path: rows behind the last frame stay as they were."""
    K, N, B, T = 200, 1030, 9, 130
    for x in ("f32", "bf16"):
        layer, arrays = _layer_arrays(6, K, N, 32, bias=True, zeros=True)
        h = torch.randn(B, T, K + 5, device="cuda").to(DT[x])[:, :, 5:]
        L = torch.tensor([130, 0, 1, 64, 65, 129, 17, 100, 3], dtype=torch.int32, device="cuda")
        out = torch.full((B, T, N), 5.0, device="cuda")
        layer.logits(h, lengths=L, out=out)
        act = torch.arange(T, device="cuda")[None] < L[:, None]
        assert (out[~act] == 5).all()
        _layer_check(out[act], h[act], arrays, "f32")


def test_layer_far_rows():
    """Rows more than 2^31 elements apart, in x and in out."""
    K, N = 130, 33
    layer, arrays = _layer_arrays(13, K, N, 32)
    step = (1 << 31) + 17
    xb = torch.zeros(step + K, dtype=torch.float16, device="cuda")
    ob = torch.zeros(step + N, dtype=torch.float16, device="cuda")
    h = xb.as_strided((2, K), (step, 1))
    h.copy_(torch.randn(2, K))
    y = layer.logits(h, dtype="f16", out=ob.as_strided((2, N), (step, 1)))
    _layer_check(y.contiguous(), h.contiguous(), arrays, "f16")


def test_layer_repeats_bit_for_bit():
    layer, _ = _layer_arrays(15, 700, 333, 64)
    h = torch.randn(20, 700, device="cuda", dtype=torch.bfloat16)
    a = layer.logits(h)
    for _ in range(3):
        assert torch.equal(a, layer.logits(h))
    # within the few-row path a row's result does not depend on the rows beside it
    assert torch.equal(layer.logits(h[7:8]), a[7:8])
    layer, _ = _layer_arrays(16, 300, 17000, 32)
    h = torch.randn(70, 300, device="cuda")
    a = layer.logits(h)
    for _ in range(3):
        assert torch.equal(a, layer.logits(h))


def test_layer_refuses():
    layer, _ = _layer_arrays(17, 64, 10, 32)
    h = torch.randn(4, 64, device="cuda")
    with pytest.raises(ValueError):
        layer.logits(h[:, :63])
    with pytest.raises(ValueError):
        layer.logits(h, dtype="f64")
    with pytest.raises(TypeError):
        layer.logits(h.double())
    with pytest.raises(TypeError):
        layer.logits(h.cpu())
    with pytest.raises(ValueError):
        layer.logits(h, out=torch.empty(4, 11, device="cuda"))
    with pytest.raises(ValueError):
        layer.logits(h, lengths=[1])
    with pytest.raises(ValueError):
        layer.logits(h.view(2, 2, 64), lengths=[1])
    buf = torch.randn(4, 80, device="cuda")
    with pytest.raises(wb.WfstError, match="overlap"):
        layer.logits(buf[:, :64], out=buf[:, 60:70])
    w = torch.zeros(4, 32, dtype=torch.uint8, device="cuda")
    with pytest.raises(wb.WfstError, match="group_size"):
        wb.OutputLayer(w, torch.ones(4, 4, device="cuda"), group_size=16)
    with pytest.raises(ValueError):
        wb.OutputLayer(w, torch.ones(4, 3, device="cuda"), group_size=32)
    with pytest.raises(ValueError):
        wb.OutputLayer(w, torch.ones(4, 2, device="cuda"), group_size=32, in_features=66)
    layer.release()
    with pytest.raises(ValueError, match="released"):
        layer.logits(h)


# ---------------------------------------------------------------- log-softmax

def _norm_check(y, x, out, scale=1.0, bias=None):
    xs = _np(x).reshape(-1, x.shape[-1])
    b = None if bias is None else _np(bias)
    want = ref.log_softmax(xs, scale, b)
    got = _np(y).reshape(want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    z = xs * scale + (0.0 if b is None else b)
    top = np.abs(np.where(np.isfinite(z), z, 0)).max(-1, keepdims=True)
    V = x.shape[-1]
    with np.errstate(invalid="ignore"):
        tol = _half(out) * np.abs(want) * 1.001 + 4 * E * (top + np.abs(want) + np.log(V) + 8 + V / 1024)
        ok = (got == want) | np.isnan(want) | (np.abs(got - want) <= tol)
    if out == "f16":
        ok |= (want < -65519.9) & (got == -np.inf)
    assert ok.all(), (np.argwhere(~ok)[:4], got[~ok][:4], want[~ok][:4])


@pytest.mark.parametrize("V", [1, 2, 3, 63, 64, 65, 500, 1023, 1024, 1025, 5000, 8191, 16384, 16387, 40001, 131071])
@pytest.mark.parametrize("x,out", [("f32", "f32"), ("f32", "f16"), ("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_log_softmax(V, x, out):
    for R in (1, 5, 300 if V < 20000 else 20):
        _say("log-softmax", V, R, x, out)
        t = (torch.randn(R, V, device="cuda") * 4).to(DT[x])
        _norm_check(wb.log_softmax(t, dtype=out), t, out)
        bias = torch.randn(V, device="cuda")
        _norm_check(wb.log_softmax(t, dtype=out, scale=0.7, bias=bias), t, out, float(np.float32(0.7)), bias)


@pytest.mark.parametrize("V", [7, 500, 5000, 40001, 70001])
def test_log_softmax_masks_and_specials(V):
    inf = float("inf")
    t = torch.randn(9, V) * 3
    t[0] = -inf                                   # a row whose mask leaves nothing
    t[1] = -inf
    t[1, V - 1] = -2.5                            # one label left
    t[2, V // 2] = inf
    t[3, 0] = float("nan")
    t[4] = torch.finfo(torch.float32).min         # masks of the type's lowest value
    t[5] = torch.finfo(torch.float32).min
    t[5, 1] = 3.0
    t[6] = 1e30
    t[7, 1:] = -30.0                              # a dominant label: log-probability near 0
    t[7, 0] = 10.0
    t[8, ::2] = -inf
    y = wb.log_softmax(t.cuda())
    _norm_check(y, t, "f32")
    assert (y[0] == -inf).all() and y[1, V - 1] == 0 and torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    # its digits survive (relative, not absolute): e^-40 by way of 2^(-40 log2 e), the constant and the
    # product each rounded by 2^-24 of an exponent of 40: 40 E, and 8 E for the exponential, sums and log1p
    lead = ref.log_softmax(_np(t[7:8]))[0, 0]
    assert abs(float(y[7, 0]) - lead) <= 48 * E * abs(lead)
    bias = torch.zeros(V, device="cuda")
    bias[::2] = -inf                              # labels that may not be emitted
    y = wb.log_softmax(t[6:8].cuda(), bias=bias)
    _norm_check(y, t[6:8], "f32", 1.0, bias)


@pytest.mark.parametrize("V", [6, 77, 500, 5003, 20001, 70001])
@pytest.mark.parametrize("x", ["f32", "f16"])
def test_log_softmax_strides_lengths_in_place(V, x):
    B, T = 4, 6
    L = torch.tensor([6, 0, 1, 5], dtype=torch.int32, device="cuda")
    for off in (0, 1, 3):
        buf = (torch.randn(B, T, V + 11, device="cuda") * 3).to(DT[x])
        t = buf[:, :, off:off + V]
        wide = torch.full((B, T, V + 5), 9.0, device="cuda", dtype=torch.float16)
        wb.log_softmax(t, dtype="f16", lengths=L, out=wide[:, :, 2:2 + V])
        assert (wide[:, :, :2] == 9).all() and (wide[:, :, 2 + V:] == 9).all()
        for b, n in enumerate([6, 0, 1, 5]):
            assert (wide[b, n:] == 9).all()
            if n:
                _norm_check(wide[b, :n, 2:2 + V], t[b, :n], "f16")
        before = buf.clone()
        apart = wb.log_softmax(t, lengths=L)
        assert torch.equal(before, buf)
        wb.log_softmax(t, lengths=L, out=t)                      # in place
        for b, n in enumerate([6, 0, 1, 5]):
            assert torch.equal(t[b, :n], apart[b, :n]) and torch.equal(t[b, n:], before[b, n:, off:off + V])
        assert torch.equal(buf[:, :, :off], before[:, :, :off])
        assert torch.equal(buf[:, :, off + V:], before[:, :, off + V:])


def test_log_softmax_far_rows():
    V, step = 700, (1 << 31) + 5
    xb = torch.zeros(step + V, dtype=torch.float16, device="cuda")
    t = xb.as_strided((2, V), (step, 1))
    t.copy_(torch.randn(2, V))
    want = wb.log_softmax(t.contiguous())
    y = wb.log_softmax(t, out=t)
    assert torch.equal(y, want)


def test_log_softmax_refuses():
    t = torch.randn(4, 10, device="cuda")
    with pytest.raises(TypeError):
        wb.log_softmax(t.double())
    with pytest.raises(ValueError):
        wb.log_softmax(t.t())
    with pytest.raises(ValueError):
        wb.log_softmax(t, bias=torch.zeros(9, device="cuda"))
    with pytest.raises(ValueError):
        wb.log_softmax(t, out=torch.empty(4, 9, device="cuda"))
    buf = torch.randn(4, 20, device="cuda")
    with pytest.raises(wb.WfstError, match="overlap"):
        wb.log_softmax(buf[:, :10], out=buf[:, 5:15])
    with pytest.raises(wb.WfstError, match="scale"):
        wb.log_softmax(t, scale=float("nan"))
    lib = wb.load_library()
    # a tensor that ends past its allocation
    assert lib.wfst_log_softmax(t.data_ptr(), 0, 1 << 40, 4, 10, 1.0, None, None, 1, t.data_ptr(), 0, 1 << 40,
                                None, 0, None) == -1
    assert b"past its allocation" in lib.wfst_last_error()
    assert lib.wfst_log_softmax(np.zeros(40, np.float32).ctypes.data, 0, 10, 4, 10, 1.0, None, None, 1, t.data_ptr(),
                                0, 10, None, 0, None) == -1
    # a row in pieces needs its workspace
    t = torch.randn(2, 90000, device="cuda")
    n = np.zeros(1, np.int64)
    assert lib.wfst_log_softmax_workspace(0, 2, 90000, 0, n.ctypes.data) == 0 and n[0] > 0
    for w, size in ((None, 0), (t.data_ptr(), int(n[0])), (torch.empty(8, device="cuda").data_ptr(), 8)):
        assert lib.wfst_log_softmax(t.data_ptr(), 0, 90000, 2, 90000, 1.0, None, None, 1, t.data_ptr(), 0, 90000, w, size,
                                    None) == -1


# ---------------------------------------------------------------- draw

def _sample_check(res, x, u, **kw):
    x = _np(x).reshape(-1, x.shape[-1])
    kw = {k: (_np(v).reshape(-1) if torch.is_tensor(v) else v) for k, v in kw.items()}
    kw = {{"temperature": "T"}.get(k, k): v for k, v in kw.items()}
    if "top_k" in kw:
        kw["top_k"] = np.asarray(kw["top_k"]).astype(int)
    tok, lp, kept = ref.sample(x, _np(u).reshape(-1), **kw)
    assert np.array_equal(res.kept.cpu().numpy().reshape(-1), kept)
    assert np.array_equal(res.tokens.cpu().numpy().reshape(-1), tok)
    got = _np(res.log_probs).reshape(-1)
    with np.errstate(invalid="ignore"):
        assert ((got == lp) | (np.abs(got - lp) <= 2.0 ** -24 * np.abs(lp) * 1.001 + 1e-9)).all()


SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.7, top_k=1), dict(top_k=5), dict(top_k=50, top_p=0.9),
            dict(top_p=0.95), dict(top_p=0.3, temperature=1.7), dict(min_p=0.1), dict(top_p=0.0), dict(min_p=1.0),
            dict(top_k=50, min_p=0.01), dict(temperature=0.8, top_k=700, top_p=0.97, min_p=0.01), dict(top_p=0.9, min_p=1e-4), dict(temperature=3.0, top_k=100000, top_p=0.999)]


@pytest.mark.parametrize("V", [1, 2, 5, 64, 65, 257, 500, 1025, 5000, 32003, 70003])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_sample(V, x):
    g = torch.Generator(device="cuda").manual_seed(V)
    for sigma in (0.3, 4.0):
        t = (torch.randn(17, V, generator=g, device="cuda") * sigma).to(DT[x])
        u = torch.rand(17, generator=g, device="cuda")
        u[0], u[1] = 0.0, 1.0 - 2.0 ** -24
        for s in SETTINGS:
            _say("sample", V, x, sigma, s)
            _sample_check(wb.sample(t, u, **s), t, u, **s)


@pytest.mark.parametrize("V,R", [(40, 64), (3000, 64), (20011, 64), (70011, 20)])
def test_sample_settings_per_row(V, R):
    g = torch.Generator(device="cuda").manual_seed(V + 1)
    t = torch.randn(R, V, generator=g, device="cuda") * 3
    u = torch.rand(R, generator=g, device="cuda")
    rng = np.random.default_rng(V)
    pick = lambda v, d: torch.from_numpy(rng.choice(np.array(v, d), R)).cuda()       # noqa: E731
    s = dict(temperature=pick([0.0, 0.5, 1.0, 2.0, -1.0], np.float32), top_k=pick([0, 1, 7, 40, 900, -3], np.int32),
             top_p=pick([1.0, 0.2, 0.9, 1.7, -0.5], np.float32), min_p=pick([0.0, 0.05, 0.5, -1.0, 4.0], np.float32))
    _sample_check(wb.sample(t, u, **s), t, u, **s)


def test_sample_ties_go_to_the_lowest_index():
    """Equal scores: masses of 1 add exactly, so every border is hit exactly."""
    V = 4096
    t = torch.zeros(8, V, device="cuda")
    t[4:, ::2] = -1e9
    u = torch.tensor([0.0, 0.25, 0.5, 0.75] * 2, device="cuda")
    for s in (dict(), dict(top_k=64), dict(top_p=0.5), dict(top_k=1024, top_p=0.25), dict(min_p=1.0)):
        _sample_check(wb.sample(t, u, **s), t, u, **s)
    r = wb.sample(t, u, top_k=64)
    assert r.tokens.tolist()[:4] == [0, 16, 32, 48] and r.tokens.tolist()[4:] == [1, 33, 65, 97]
    q = (torch.randn(6, 30011, device="cuda") * 2).round_().bfloat16()      # few distinct values, many of each
    u = torch.rand(6, device="cuda")
    for s in (dict(top_k=1000), dict(top_p=0.613), dict(top_k=20000, top_p=0.377), dict(min_p=0.2)):
        _sample_check(wb.sample(q, u, **s), q, u, **s)


@pytest.mark.parametrize("V", [9, 700, 5001, 9001, 66001])
def test_sample_masks_and_specials(V):
    inf = float("inf")
    t = torch.randn(10, V)
    t[0] = -inf
    t[1] = float("nan")
    t[2] = -inf
    t[2, V - 1] = 1.0
    t[3, 1], t[3, 5] = inf, inf
    t[4, ::3] = float("nan")
    t[5] = torch.finfo(torch.float32).min
    t[6, ::2] = -inf
    t[7] = torch.tensor([0.0, -0.0]).repeat(V)[:V]
    t[8] = -3e38
    t[8, 3] = 3e38
    t[9, 0] = -float("nan")
    t = t.cuda()
    u = torch.linspace(0.0, 0.99, 10).cuda()
    for s in SETTINGS:
        _sample_check(wb.sample(t, u, **s), t, u, **s)
    bad = torch.tensor([-1.0, 1.0, 2.0, inf, -inf, float("nan"), 0.5, 1.0, 1.0, 1.0], device="cuda")
    t = torch.randn(10, V, device="cuda")
    r = wb.sample(t, bad)
    u = torch.tensor([0.0] + [1.0 - 2.0 ** -24] * 3 + [0.0, 0.0, 0.5] + [1.0 - 2.0 ** -24] * 3, device="cuda")
    assert ((r.tokens >= 0) & (r.tokens < V)).all()
    assert torch.equal(r.tokens[[0, 4, 5, 6]], wb.sample(t, u).tokens[[0, 4, 5, 6]])


def test_sample_strides_lengths_and_untouched_rows():
    B, T, V = 3, 5, 901
    buf = torch.randn(B, T, V + 10, device="cuda").half()
    x = buf[:, :, 5:5 + V]
    u = torch.rand(B, T, device="cuda")
    L = torch.tensor([2, 5, 0], dtype=torch.int32, device="cuda")
    out = (torch.full((B, T), -9, dtype=torch.int32, device="cuda"), torch.full((B, T), -9.0, device="cuda"),
           torch.full((B, T), -9, dtype=torch.int32, device="cuda"))
    r = wb.sample(x, u, top_p=0.9, lengths=L, out=out)
    full = wb.sample(x.contiguous(), u, top_p=0.9)
    for b, n in enumerate([2, 5, 0]):
        for o, f in zip(r, full):
            assert torch.equal(o[b, :n], f[b, :n]) and (o[b, n:] == -9).all()
    _sample_check(full, x, u, top_p=0.9)
    nan = x.contiguous()
    nan[0, 2:] = float("nan")                       # frames behind the last are not read
    assert torch.equal(wb.sample(nan, u, top_p=0.9, lengths=L, out=out).tokens, r.tokens)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("R", [3, 140])
def test_sample_orders_that_mislead_the_lists(R, x):
    """Scores in falling order, in rising order, all equal, all masked but a few,
    and a nucleus of most labels: the short lists do not hold the kept labels."""
    V = 30011 if R > 32 else 66011
    t = torch.empty(5, V)
    t[0] = -torch.arange(V) * 1e-3
    t[1] = torch.arange(V) * 1e-3
    t[2] = 1.5
    t[3] = -1e30
    t[3, 20000:20040] = torch.randn(40)
    t[4] = torch.randn(V) * 0.1
    t = t.repeat(-(-R // 5), 1)[:R].to(DT[x]).cuda()
    u = torch.rand(R, generator=torch.Generator(device="cuda").manual_seed(R), device="cuda")
    for s in (dict(), dict(top_k=40), dict(top_k=900), dict(top_k=5000), dict(top_p=0.9), dict(top_p=0.9, top_k=3000),
              dict(min_p=0.5), dict(top_p=0.31, temperature=20.0), dict(temperature=0.0)):
        _say("orders", R, x, s)
        _sample_check(wb.sample(t, u, **s), t, u, **s)


@pytest.mark.parametrize("R", [2, 40])
def test_sample_language_model_rows(R):
    """A power law over a shuffled vocabulary, odd and large."""
    V = 70001
    g = torch.Generator(device="cuda").manual_seed(R)
    rank = torch.randperm(V, generator=g, device="cuda").float() + 1
    t = (torch.randn(R, V, generator=g, device="cuda") - 1.3 * rank.log() + 9).bfloat16()
    u = torch.rand(R, generator=g, device="cuda")
    for s in SETTINGS:
        _say("language model", R, s)
        _sample_check(wb.sample(t, u, **s), t, u, **s)


def test_sample_far_rows():
    V, step = 1200, (1 << 31) + 9
    xb = torch.zeros(step + V, dtype=torch.float16, device="cuda")
    t = xb.as_strided((2, V), (step, 1))
    t.copy_(torch.randn(2, V))
    u = torch.rand(2, device="cuda")
    _sample_check(wb.sample(t, u, top_k=30), t.contiguous(), u, top_k=30)


def test_sample_longest_rows():
    V = (1 << 20) + 3
    g = torch.Generator(device="cuda").manual_seed(9)
    t = torch.randn(3, V, generator=g, device="cuda") * 3
    u = torch.rand(3, generator=g, device="cuda")
    for s in (dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.8), dict(min_p=0.05)):
        _sample_check(wb.sample(t, u, **s), t, u, **s)


@pytest.mark.parametrize("V", [30, 3000])
def test_sample_extreme_temperatures(V):
    """Infinite (in a tensor only), subnormal, huge and NaN."""
    t = torch.randn(7, V, device="cuda")
    t[:, ::3] = -float("inf")
    u = torch.rand(7, device="cuda")
    T = torch.tensor([float("inf"), 1e-45, 1e-30, 3e38, float("nan"), 1e30, 1e-3], device="cuda")
    for s in (dict(), dict(min_p=1.0), dict(min_p=0.5), dict(top_k=7), dict(top_p=0.613), dict(top_p=0.4, min_p=0.9)):
        full = dict(s, temperature=T)
        _sample_check(wb.sample(t, u, **full), t, u, **full)


def test_more_rows_than_workgroups():
    R = (1 << 20) + 5
    t = torch.randn(R, 4, device="cuda")
    u = torch.rand(R, device="cuda")
    y = wb.log_softmax(t)
    assert torch.allclose(y.double(), torch.log_softmax(t.double(), -1), rtol=0, atol=1e-5)
    keep = t >= t.topk(2, -1).values[:, 1:]
    w = torch.where(keep, torch.exp(t.double() - t.amax(-1, keepdim=True).double()), 0.0)
    run = w.cumsum(-1)
    want = (run > (u.double() * run[:, -1])[:, None]).int().argmax(-1)
    assert torch.equal(wb.sample(t, u, top_k=2).tokens.long(), want)
    w = torch.exp(t.double() - t.amax(-1, keepdim=True).double())
    run = w.cumsum(-1)
    want = (run > (u.double() * run[:, -1])[:, None]).int().argmax(-1)
    assert torch.equal(wb.sample(t, u).tokens.long(), want)


def test_sample_many_rows():
    t = (torch.randn(3000, 50, device="cuda") * 2).bfloat16()
    u = torch.rand(3000, device="cuda")
    for s in (dict(), dict(top_k=8, top_p=0.8)):
        _sample_check(wb.sample(t, u, **s), t, u, **s)


def test_sample_frequencies():
    """Draws fall as often as the masses say (within 5 standard deviations)."""
    p = torch.tensor([0.5, 0.25, 0.125, 0.0625, 0.0625], device="cuda")
    n = 200_000
    r = wb.sample(torch.log(p).expand(n, 5).contiguous(), torch.rand(n, device="cuda"))
    got = torch.bincount(r.tokens.long(), minlength=5).double() / n
    assert ((got - p).abs() < 5 * (p * (1 - p) / n).sqrt()).all()


def test_sample_refuses():
    t = torch.randn(4, 10, device="cuda")
    u = torch.rand(4, device="cuda")
    for kw in (dict(temperature=-1.0), dict(top_k=-1), dict(top_p=2.0), dict(min_p=-0.5)):
        with pytest.raises(wb.WfstError):
            wb.sample(t, u, **kw)
    with pytest.raises(ValueError):
        wb.sample(t, u[:3])
    with pytest.raises(ValueError):
        wb.sample(t, u.double())
    with pytest.raises(ValueError):
        wb.sample(t, u, top_k=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        wb.sample(t, u, out=(torch.empty(4, dtype=torch.int32, device="cuda"), None, None))
    tok = torch.empty(4, dtype=torch.int32, device="cuda")
    with pytest.raises(wb.WfstError, match="overlaps"):
        wb.sample(t, u, out=(tok, torch.empty(4, device="cuda"), tok))


# ---------------------------------------------------------------- a run of them

def test_gradients_are_refused():
    layer, _ = _layer_arrays(20, 64, 10, 32)
    h = torch.randn(3, 64, device="cuda", requires_grad=True)
    for f in (lambda: layer.logits(h), lambda: wb.log_softmax(h), lambda: wb.sample(h, torch.rand(3, device="cuda"))):
        with pytest.raises(ValueError, match="gradient"):
            f()
        with torch.no_grad():
            f()


def test_streams_and_empty_calls():
    layer, arrays = _layer_arrays(21, 96, 300, 32, bias=True)
    h = torch.randn(40, 96, device="cuda")
    u = torch.rand(40, device="cuda")
    want = layer.log_probs(h, dtype="f16")
    drawn = wb.sample(want, u, top_p=0.9)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s in side * 3:
        a = layer.log_probs(h, dtype="f16", stream=s)
        b = wb.sample(a, u, top_p=0.9, stream=s.cuda_stream)
        del a
        junk = torch.full((40, 300), 5.0, dtype=torch.float16, device="cuda")      # must not get a's memory early
        s.synchronize()
        assert torch.equal(b.tokens, drawn.tokens) and torch.equal(b.log_probs, drawn.log_probs)
        del junk
    assert layer.logits(h[:0]).shape == (0, 300)
    assert wb.log_softmax(want[:0]).shape == (0, 300)
    assert wb.sample(want[:0], u[:0]).tokens.shape == (0,)


@pytest.mark.parametrize("B,T,V", [(6, 3, 1111), (4, 5, 70003), (30, 1, 20011)])
def test_captured_run_replays(B, T, V):
    """Hidden states to draws captured into one graph: every replay on new inputs
    equals the eager run, with eager work between the replays (at sizes where the
    operators take one launch, and where they take two and three)."""
    K = 160
    layer, _ = _layer_arrays(23, K, V, 32, zeros=True, bias=True)
    h = torch.randn(B, T, K, device="cuda").bfloat16()
    u = torch.rand(B, T, device="cuda")
    L = torch.full((B,), T, dtype=torch.int32, device="cuda")
    k = torch.full((B, T), 50, dtype=torch.int32, device="cuda")

    def step():
        lp = layer.log_probs(h, dtype="f16", lengths=L)
        return lp, wb.sample(lp, u, top_k=k, top_p=0.9, lengths=L)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp, res = step()
    for i in range(4):
        h.copy_(torch.randn(B, T, K))
        u.copy_(torch.rand(B, T))
        L.copy_(torch.randint(0, T + 1, (B,), dtype=torch.int32))
        k.fill_(5 + 40 * i)
        graph.replay()
        torch.cuda.synchronize()
        lp_e, res_e = step()
        act = torch.arange(T, device="cuda")[None] < L[:, None]
        assert torch.equal(lp[act], lp_e[act])
        for a, b in zip(res, res_e):
            assert torch.equal(a[act], b[act])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_hidden_states_to_words(dtype):
    """decode_hidden searches what the layer and the log-softmax make: the oracle's
    path on those rows; the same frames in chunks through advance_hidden end alike."""
    g = synth.random_graph(61, n=80, deg=(1, 6), vocab=37, self_loop=0.3)
    dg = wb.Graph(g)
    K, B, T = 96, 4, 30
    layer, arrays = _layer_arrays(25, K, g.vocab, 32, bias=True)
    rng = np.random.default_rng(1)
    h = torch.from_numpy(rng.normal(size=(B, T, K)).astype(np.float32)).cuda()
    L = np.array([30, 17, 0, 9], np.int32)
    bias = torch.zeros(g.vocab, device="cuda")
    bias[0] = -1.0
    lp = layer.log_probs(h, dtype=dtype, scale=0.8, bias=bias)
    y, size = ref.layer(_np(h).reshape(-1, K), *arrays)
    want = ref.log_softmax(y, float(np.float32(0.8)), _np(bias)).reshape(B, T, -1)
    slack = 2 * (K / 32 + 40) * E * size.max() + 4 * E * (np.abs(y).max() + 2 * np.abs(want).max() + 16)
    assert (np.abs(_np(lp) - want) <= _half(dtype) * np.abs(want) * 1.001 + slack).all()
    dec = wb.Decoder(dg, 8.0, 300, max_lanes=B, max_frames=T, lp_dtype=dtype)
    r = dec.decode_hidden(layer, h, L, scale=0.8, bias=bias)
    o = oracle_lanes(g, lp.cpu().numpy(), L, 8.0, 300)
    compare_batch(r, None, o, check_steps=False)
    ch = dec.create_streams(2)
    for t0 in range(0, 30, 7):
        n = np.clip(L[:2] - t0, 0, 7).astype(np.int32)
        part = torch.zeros(2, 7, K, device="cuda")
        w = min(7, T - t0)
        part[:, :w] = h[:2, t0:t0 + w]
        dec.advance_hidden(ch, layer, part, n, scale=0.8, bias=bias)
    for c, want_lane in zip(ch, (0, 1)):
        s = dec.finalize_stream(c)
        assert np.array_equal(s.arcs[0], r.arcs[want_lane])
        dec.release_stream(c)
    with pytest.raises(ValueError):
        dec.decode_hidden(layer, h[:, :, :0], L)
    with pytest.raises(ValueError):
        dec.decode_hidden(layer, h, [31, 0, 0, 0])
    other, _ = _layer_arrays(26, K, g.vocab + 1, 32)
    with pytest.raises(ValueError, match="vocab"):
        dec.decode_hidden(other, h, L)
    dec.close()
    dg.release()


# ---------------------------------------------------------------- rows cut into chunks, joined by four wavefronts

@pytest.mark.parametrize("V", [150001, 300001, 520011])
def test_sample_chunks_of_every_wavefront_join(V):
    """The best chunk (whose bound is the row's) with each wavefront of the join in turn, the other chunks'
    lists longer or shorter than its own."""
    g = torch.Generator(device="cuda").manual_seed(V)
    span = 2048                                          # labels of a chunk of binary32 scores
    chunks = -(-V // span)
    t = torch.randn(8, V, generator=g, device="cuda")
    for r in range(8):
        c0 = (chunks - 1) * r // 7
        t[r, c0 * span:c0 * span + (span if r % 2 else 40)] += 6.0
    t[5, ::2] = -float("inf")
    t[6, V // 2:] = t[6, V // 2:].round()                # long lists of equal scores behind the best chunk
    u = torch.rand(8, generator=g, device="cuda")
    for s in (dict(temperature=0.0), dict(top_k=1), dict(top_k=50), dict(top_k=50, top_p=0.9), dict(top_k=600),
              dict(top_k=64, min_p=0.01)):
        _say("chunks", V, s)
        want = wb.sample(t, u, **s)
        _sample_check(want, t, u, **s)
        for r in range(0, 8, 3):
            for a, b in zip(wb.sample(t[r:r + 1], u[r:r + 1], **s), want):
                assert torch.equal(a, b[r:r + 1])
    # every kind of row in one call
    s = dict(temperature=torch.tensor([0.0, 1, 1, 0, 1, 1, 1, 0.5], device="cuda"),
             top_k=torch.tensor([0, 50, 0, 9, 200, 3, 700, 50], dtype=torch.int32, device="cuda"),
             top_p=torch.tensor([1.0, 0.9, 0.8, 1, 1, 1, 0.5, 1], device="cuda"))
    _sample_check(wb.sample(t, u, **s), t, u, **s)


def test_integers_past_32_bits():
    """No limit written as the largest integer keeps every label; sizes and lengths past 32 bits are not cut."""
    import sys
    t = torch.randn(6, 900, device="cuda")
    u = torch.rand(6, device="cuda")
    for k in (sys.maxsize, 2 ** 32 + 1, 2 ** 31):
        _sample_check(wb.sample(t, u, top_k=k, top_p=0.9), t, u, top_p=0.9)
    w = torch.zeros(4, 32, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        wb.OutputLayer(w, torch.ones(4, 1, device="cuda"), group_size=2 ** 32 + 32)
    x = t.view(2, 3, 900)
    out = torch.full_like(x, 9.0)
    wb.log_softmax(x, lengths=np.array([2 ** 32 + 1, -2 ** 32 + 2]), out=out)
    assert torch.equal(out[0], wb.log_softmax(x)[0]) and (out[1] == 9).all()


def test_forward_mode_duals_are_refused():
    import torch.autograd.forward_ad as fw
    layer, _ = _layer_arrays(27, 64, 10, 32)
    h, u, b = torch.randn(3, 64, device="cuda"), torch.rand(3, device="cuda"), torch.randn(64, device="cuda")
    with fw.dual_level():
        d, db = fw.make_dual(h, torch.ones_like(h)), fw.make_dual(b, torch.ones_like(b))
        du, out = fw.make_dual(u, torch.ones_like(u)), fw.make_dual(torch.empty_like(h), h)
        for f in (lambda: layer.logits(d), lambda: layer.log_probs(d[1:]), lambda: wb.log_softmax(d),
                  lambda: wb.log_softmax(h, bias=db), lambda: wb.log_softmax(h, out=out), lambda: wb.sample(d, u),
                  lambda: wb.sample(h, du), lambda: wb.sample(h, u, temperature=du)):
            with pytest.raises(ValueError, match="tangent"):
                f()
        assert torch.equal(wb.log_softmax(d.detach()), wb.log_softmax(h))      # the primal alone
        assert torch.equal(layer.logits(d.detach()), layer.logits(h))
        with torch.inference_mode():
            wb.log_softmax(h)
    with pytest.raises(ValueError, match="tangent"):
        torch.func.jvp(lambda t: wb.log_softmax(t), (h,), (torch.ones_like(h),))
    assert torch.equal(wb.log_softmax(h), wb.log_softmax(h.clone()))


# ---------------------------------------------------------------- output layer: small scales, small and mixed hidden states

def _layer_bound(layer, arrays, h, out="f32", held=0.0):
    """|y - exact| <= half a step of the output + (K / 32 + 40) E S + held sum |w| (the module's bound; each
    addition of two subnormal numbers is exact, each product's rounding among them at most 2^-150; held: how far
    a hidden state may be off by its block's largest)."""
    y = layer.logits(h, dtype=out)
    want, size = ref.layer(_np(h), *arrays)
    n = arrays[4] / 32 + 40
    tol = _half(out) * np.abs(want) * 1.001 + n * E * size + n * 2.0 ** -149
    tol = tol + held * ref.layer(np.ones((1, arrays[4])), *arrays)[1]
    err = np.abs(_np(y) - want)
    bad = err > tol
    assert not bad.any(), (np.argwhere(bad)[:4], _np(y)[bad][:4], want[bad][:4], (err / tol).max())


def _scaled_layer(seed, K, N, group, factor, scale):
    """Scales of about `factor`, rounded to their type."""
    rng = np.random.default_rng(seed)
    w = rng.integers(0, 256, (N, (K + 1) // 2), dtype=np.uint8)
    s = torch.from_numpy(((0.5 + rng.random((N, -(-K // group)))) * factor).astype(np.float32)).to(DT[scale])
    layer = wb.OutputLayer(torch.from_numpy(w).cuda(), s.cuda(), in_features=K, group_size=group)
    return layer, (w, s.double().numpy(), None, None, K, group)


@pytest.mark.parametrize("M,K,N,group", [(1, 256, 20, 32), (4, 300, 40, 128), (16, 513, 33, 64),      # few rows, K split
                                         (2, 140, 24600, 32),                                         # few rows, K whole
                                         (20, 260, 16500, 64), (70, 390, 8200, 128)])                 # operands
@pytest.mark.parametrize("x,scale,factor,size", [("f32", "f32", 1e-7, 1e-32), ("f32", "f16", 3e-5, 1e-32),
                                                 ("bf16", "f32", 2e-7, 1e-32), ("bf16", "bf16", 1e-8, 1e-32),
                                                 ("f32", "bf16", 1e5, 1e33), ("bf16", "f32", 3e4, 3e33)])
def test_layer_scale_and_block_factor_do_not_meet_alone(M, K, N, group, x, scale, factor, size):
    """A block's power of two times a group's scale may leave the binary32 range, or its normal part, where the
    result does not: a row's accuracy depends neither on that nor on the number of rows."""
    _say("small scales", M, K, N, group, x, scale, factor, size)
    layer, arrays = _scaled_layer(M + K, K, N, group, factor, scale)
    h = (torch.from_numpy(np.random.default_rng(K).normal(size=(M, K)).astype(np.float32)) * size).to(DT[x])
    if factor > 1:                          # one huge value a row; the columns whose weight there is 0 stay small
        h *= 1e-5
        h[:, K // 2] = 2e38
        q = ref.unpack(arrays[0], K)[:, K // 2] == 8
        assert q.any() or N < 200
        y = _np(layer.logits(h.cuda()))
        assert not np.isnan(y).any() and (not q.any() or np.isfinite(y[:, q]).all())
        return
    _layer_bound(layer, arrays, h.cuda())


@pytest.mark.parametrize("M,K,N,group", [(1, 256, 64, 32), (3, 300, 40, 128), (16, 513, 33, 64), (2, 140, 24600, 32),
                                         (20, 260, 16500, 64), (70, 390, 8200, 128), (33, 512, 16400, 32)])
def test_layer_binary32_beside_large_values(M, K, N, group):
    """Small binary32 values keep their digits beside a large one in their block: the columns whose weight at the
    large one is 0 see them alone (S counts no more than that). Two binary16 parts, the second scaled by 2^11, hold
    a value within 2^-23 of itself or 2^-50 of its block's largest."""
    rng = np.random.default_rng(M * K)
    w = rng.integers(0, 256, (N, (K + 1) // 2), dtype=np.uint8)
    big = np.arange(7, K, 128)
    w[::2, big // 2] = w[::2, big // 2] & 15 | 8 << 4                    # feature 7 of each block (odd: the high half)
    s = torch.from_numpy(((0.5 + rng.random((N, -(-K // group)))) / np.sqrt(K)).astype(np.float32))
    layer = wb.OutputLayer(torch.from_numpy(w).cuda(), s.cuda(), in_features=K, group_size=group)
    h = rng.normal(size=(M, K)).astype(np.float32) * 0.01
    h[:, big] = rng.normal(size=(M, big.size)) * 1e7
    _layer_bound(layer, (w, s.double().numpy(), None, None, K, group), torch.from_numpy(h).cuda(),
                 held=2.0 ** -50 * float(np.abs(h).max()))


@pytest.mark.parametrize("M,K,N", [(1, 128, 40), (5, 300, 40), (40, 300, 16500)])
def test_layer_subnormal_hidden_states(M, K, N):
    """Blocks of subnormal binary32 (and bfloat16) values, large scales: the result is normal."""
    for x in ("f32", "bf16"):
        layer, arrays = _scaled_layer(3, K, N, 64, 1e8, "f32")
        h = (torch.from_numpy(np.random.default_rng(K).normal(size=(M, K)).astype(np.float32)) * 2e-40).to(DT[x])
        h[:, ::3] *= 1e-2
        _layer_bound(layer, arrays, h.cuda())


# ---------------------------------------------------------------- draw: rows with a long, light tail

def _mass_error(V):
    """Bound of a sum's error: V masses rounded to multiples of 2^-unit, unit = min(51, 62 - ceil(log2 V)), as a share
    of the largest; past 2^20 labels V * (labels of one of at least 256 threads) * 2^-63 of the total."""
    bits = max(0, (V - 1).bit_length())
    return V * 2.0 ** -(min(51, 62 - bits) + 1) if V <= 1 << 20 else V * (V / 256 + 32) * 2.0 ** -63


def _tail_check(R, V, tail, x, s, us):
    """Rows of one label of score 0 and V - 1 of score `tail`: index i has the running mass 1 + i w."""
    t = torch.full((R, V), tail, device="cuda", dtype=DT[x])
    t[:, 0] = 0
    u = torch.tensor([us[i % len(us)] for i in range(R)], device="cuda")
    r = wb.sample(t, u, **s)
    w = float(np.exp(np.float64(float(t[0, 1]))))
    C = 1 + (V - 1) * w
    err = _mass_error(V) * C + 2.0 ** -48
    n = V
    if s.get("top_p", 1.0) < 1:
        n = max(1, int(np.ceil((float(np.float32(s["top_p"])) * C - 1) / w)) + 1)
    kept = r.kept.cpu().numpy()
    room = 0 if n == V else 2 * err / w + 1
    assert (np.abs(kept - n) <= room).all(), (kept, n, room)
    for i in range(min(R, 4 * len(us))):
        total = 1 + (int(kept[i]) - 1) * w
        goal = float(u[i].double()) * total
        want = 0 if goal < 1 else int((goal - 1) / w) + 1
        tok = int(r.tokens[i])
        assert abs(tok - want) <= 2 * err / w + 1 or abs(goal - 1) <= 2 * err, (i, tok, want)
        lp = (float(t[i, tok]) if tok else 0.0) - np.log(total)
        # (total is off by err at most; a binary32 result)
        assert abs(float(r.log_probs[i]) - lp) <= err * 1.001 + 2.0 ** -24 * abs(lp), (i, float(r.log_probs[i]), lp)


US = [0.0, 0.25, 0.6, 0.75, 1.0 - 2.0 ** -24, 0.9999]


@pytest.mark.parametrize("V,R,tail,x", [
    (131072, 1, -31.5, "f32"), (131072, 33, -31.5, "f32"), (131072, 2, -20.0, "bf16"), (131072, 40, -12.25, "bf16"),
    (1 << 20, 3, -28.0, "f16"), ((1 << 20) + 3, 2, -28.125, "f32"), ((1 << 20) + 3, 258, -28.125, "f16"),
    ((1 << 21) + 5, 3, -27.75, "bf16"), (1 << 24, 2, -27.296875, "f32"), (1 << 24, 3, -17.0, "f16"),
    ((1 << 24) - 1, 2, -14.0, "bf16")])
def test_sample_light_tails(V, R, tail, x):
    for s in (dict(), dict(min_p=1e-30), dict(top_p=0.9), dict(top_p=1.0 - 2.0 ** -13)):
        _say("tails", V, R, tail, x, s)
        _tail_check(R, V, tail, x, s, US)


@pytest.mark.parametrize("V", [(1 << 20) + 77, (1 << 22) + 1, 1 << 24])
@pytest.mark.parametrize("sigma", [0.01, 3.0])
def test_sample_longest_rows_against_running_sums(V, sigma):
    """The token's running mass brackets u times the total, within the sums' error."""
    g = torch.Generator(device="cuda").manual_seed(V)
    t = torch.randn(3, V, generator=g, device="cuda") * sigma
    t[1, ::2] = -float("inf")
    t[2, V // 3] = 40.0 * sigma
    u = torch.rand(3, generator=g, device="cuda")
    m = torch.exp(t.double() - t.amax(-1, keepdim=True).double())
    run = m.cumsum(-1)
    for s in (dict(), dict(top_k=V // 2), dict(top_p=0.99), dict(temperature=0.0)):
        _say("longest", V, sigma, s)
        r = wb.sample(t, u, **s)
        if "temperature" in s:
            assert torch.equal(r.tokens.long(), t.argmax(-1))
            continue
        for i in range(3):
            mi, total = m[i], run[i, -1]
            if s:
                order = torch.sort(t[i], descending=True, stable=True).indices
                sorted_run = mi[order].cumsum(0)
                n = min(V // 2, int((t[i] > -float("inf")).sum()))
                if "top_p" in s:
                    goal = float(np.float32(0.99)) * total
                    err = (_mass_error(V) + 2.0 ** -45) * total
                    lo, hi = (int((sorted_run < goal + d).sum()) + 1 for d in (-err, err))
                    assert lo <= int(r.kept[i]) <= hi, (lo, int(r.kept[i]), hi)
                    n = int(r.kept[i])
                assert int(r.kept[i]) == n
                mi = torch.zeros_like(mi).scatter_(0, order[:n], mi[order[:n]])
            c = mi.cumsum(0)
            total = float(c[-1])
            goal, tok = float(u[i].double()) * total, int(r.tokens[i])
            err = (_mass_error(V) + 2.0 ** -45) * total * 2
            assert float(mi[tok]) > 0
            assert float(c[tok]) > goal - err and float(c[tok] - mi[tok]) <= goal + err
            lp = np.log(float(mi[tok])) - np.log(total)
            assert abs(float(r.log_probs[i]) - lp) <= err / total + 2.0 ** -24 * abs(lp) + 1e-12


def test_outputs_over_lengths_are_refused():
    """A row's workgroup would read what another one writes."""
    B, V = 6, 64
    L = torch.ones(B, dtype=torch.int32, device="cuda")
    x = torch.randn(B, 1, V, device="cuda")
    u = torch.rand(B, 1, device="cuda")
    ok = lambda d: torch.zeros(B, 1, dtype=d, device="cuda")          # noqa: E731
    over = L.view(B, 1)
    for out in ((over, ok(torch.float32), ok(torch.int32)), (ok(torch.int32), over.view(torch.float32), ok(torch.int32)),
                (ok(torch.int32), ok(torch.float32), over)):
        with pytest.raises(wb.WfstError, match="overlap lengths"):
            wb.sample(x, u, lengths=L, out=out)
    buf = torch.ones(B * V + B, dtype=torch.int32, device="cuda")
    for L in (buf[:B], buf[B * V - 3:B * V - 3 + B]):
        with pytest.raises(wb.WfstError, match="overlap lengths"):
            wb.log_softmax(x, lengths=L, out=buf[:B * V].view(torch.float32).view(B, 1, V))
        layer, _ = _layer_arrays(31, 32, V, 32)
        with pytest.raises(wb.WfstError, match="overlap lengths"):
            layer.logits(x[:, :, :32].contiguous(), lengths=L, out=buf[:B * V].view(torch.float32).view(B, 1, V))
    assert (buf == 1).all()
    wb.log_softmax(x, lengths=buf[B * V:], out=buf[:B * V].view(torch.float32).view(B, 1, V))     # beside it
    # workspaces
    lib = wb.load_library()
    t, out = torch.randn(2, 90000, device="cuda"), torch.empty(2, 90000, device="cuda")
    n = np.zeros(1, np.int64)
    assert lib.wfst_log_softmax_workspace(0, 2, 90000, 0, n.ctypes.data) == 0 and n[0] > 0
    work = torch.ones(int(n[0]) // 4 + 90000, dtype=torch.int32, device="cuda")
    for bias, L, word in ((None, work[4:6], b"lengths"), (work[8:], None, b"bias")):
        assert lib.wfst_log_softmax(t.data_ptr(), 0, 90000, 2, 90000, 1.0, None if bias is None else bias.data_ptr(),
                                    None if L is None else L.data_ptr(), 1, out.data_ptr(), 0, 90000, work.data_ptr(),
                                    int(n[0]), None) == -1
        assert word in lib.wfst_last_error()


# ---------------------------------------------------------------- 64-row products whose operands load straight into LDS

def _many(M, N):
    """Enough workgroups for 64 rows by 128 features each."""
    assert M > 32 and -(-N // 128) * -(-M // 64) >= 128, (M, N)


@pytest.mark.parametrize("M,K,N,group,x,scale,out,zeros,bias", [
    # one block of features (one step, half of it clamped), part of one
    (64, 100, 16400, 128, "f16", "f16", "f32", True, True),
    (65, 128, 8300, 128, "bf16", "f32", "f16", False, True),
    (200, 7, 4200, 128, "f16", "f32", "f32", True, False),
    # odd numbers of blocks, the last one part of a block
    (70, 385, 8200, 128, "f16", "f32", "f32", True, True),
    (65, 301, 8333, 256, "bf16", "bf16", "bf16", True, False),
    (129, 1153, 5600, 384, "f16", "bf16", "f32", False, True),
    (513, 2049, 2000, 128, "bf16", "f16", "f32", True, True),
    (1000, 2049, 1100, 128, "f16", "f16", "f16", True, False),
    # even numbers, whole and not
    (200, 256, 4100, 128, "f16", "f16", "f32", False, False),
    (2000, 500, 500, 128, "bf16", "f32", "f32", True, True),
    (2000, 1024, 500, 1024, "f16", "f32", "bf16", False, True),
    (100, 3840, 8209, 128, "f16", "bf16", "f32", True, True),
])
def test_layer_direct_loads(M, K, N, group, x, scale, out, zeros, bias):
    _say("direct", M, K, N, group, x, scale, out)
    _many(M, N)
    assert group % 128 == 0 and x != "f32"
    layer, arrays = _layer_arrays(M + K + N, K, N, group, scale, zeros, bias)
    h = torch.from_numpy(np.random.default_rng(K).normal(size=(M, K + 3)).astype(np.float32)).to(DT[x]).cuda()[:, 1:K + 1]
    y = layer.logits(h, dtype=out)
    _layer_check(y, h.contiguous(), arrays, out)
    for _ in range(3):
        assert torch.equal(layer.logits(h, dtype=out), y)


@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("K", [100, 385, 1280])
def test_layer_direct_loads_lengths(x, K):
    """A padded batch: rows behind the last frame hold NaN and are not read, their outputs stay."""
    B, T, N = 7, 90, 1700
    layer, arrays = _layer_arrays(K, K, N, 128, zeros=True, bias=True)
    _many(B * T, N)
    h = torch.randn(B, T, K, device="cuda").to(DT[x])
    L = torch.tensor([90, 0, 1, 64, 63, 17, 89], dtype=torch.int32, device="cuda")
    act = torch.arange(T, device="cuda")[None] < L[:, None]
    h[~act] = float("nan")
    out = torch.full((B, T, N), 5.0, device="cuda")
    layer.logits(h, lengths=L, out=out)
    assert (out[~act] == 5).all()
    _layer_check(out[act], h[act], arrays, "f32")


@pytest.mark.parametrize("x", ["f16", "bf16", "f32"])
def test_workspaces_on_side_streams(x):
    """Layer, log-softmax and draw, all with a workspace, on two streams at once and in turn with work on the current one."""
    K, V, R = 200, 70003, 20
    layer, _ = _layer_arrays(33, K, V, 128, zeros=True, bias=True)
    for rows, code in ((R, "layer"), (R, "norm"), (R, "draw")):
        n = np.zeros(1, np.int64)
        lib = wb.load_library()
        dt = {"f32": 0, "f16": 1, "bf16": 2}[x]
        rc = {"layer": lambda: lib.wfst_layer_workspace(layer.handle, dt, rows, n.ctypes.data),
              "norm": lambda: lib.wfst_log_softmax_workspace(0, rows, V, 1, n.ctypes.data),
              "draw": lambda: lib.wfst_sample_workspace(1, rows, V, n.ctypes.data)}[code]()
        assert rc == 0 and n[0] > 0, code
    hs = [torch.randn(R, K, device="cuda").to(DT[x]) for _ in range(2)]
    u = torch.rand(R, device="cuda")

    def step(h, stream=None):
        lp = layer.log_probs(h, dtype="f16", stream=stream)
        return lp, wb.sample(lp, u, top_k=40, top_p=0.9, stream=stream), wb.sample(lp, u, stream=stream)

    want = [step(h) for h in hs]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for turn in range(4):
        got = [step(h, s) for h, s in zip(hs, side)]
        here = step(hs[turn % 2])
        junk = [torch.full((R, V), 3.0, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        del junk
        for a, b in zip(got + [here], want + [want[turn % 2]]):
            assert torch.equal(a[0], b[0])
            for p, q in zip(a[1:], b[1:]):
                assert all(torch.equal(i, j) for i, j in zip(p, q))


def test_overwriting_a_saved_tensor_stops_its_backward():
    layer, _ = _layer_arrays(35, 8, 64, 32)
    h, u = torch.randn(3, 8, device="cuda"), torch.rand(3, device="cuda")
    tok = torch.empty(3, dtype=torch.int32, device="cuda")
    for write in (lambda t: wb.log_softmax(t, out=t), lambda t: layer.logits(h, out=t), lambda t: layer.log_probs(h, out=t)):
        x = torch.randn(3, 64, device="cuda", requires_grad=True)
        y = x.exp()
        write(y.detach())
        with pytest.raises(RuntimeError, match="inplace"):
            y.sum().backward()
    saved = torch.rand(3, device="cuda", requires_grad=True).exp()
    wb.sample(h, u, out=(tok, saved.detach(), tok.clone()))
    with pytest.raises(RuntimeError, match="inplace"):
        saved.sum().backward()


def test_sample_masks_and_specials_of_longest_rows():
    """Past 2^20 labels, where a row's unit comes from its own masses: empty, masked, infinite, NaN and greedy rows."""
    V, inf = (1 << 20) + 9, float("inf")
    g = torch.Generator(device="cuda").manual_seed(3)
    t = torch.randn(9, V, generator=g, device="cuda") * 4
    t[0] = -inf
    t[1] = float("nan")
    t[2] = -inf
    t[2, V - 1] = 1.0
    t[3, 1], t[3, V - 2], t[3, 700000] = inf, inf, inf
    t[4, ::3] = float("nan")
    t[5] = torch.finfo(torch.float32).min
    t[6, 1000:] = -inf
    t[7, 5] = 3e38
    u = torch.rand(9, generator=g, device="cuda")
    T = torch.tensor([1.0, 1, 1, 1, 0.7, inf, 2, 1, 0], device="cuda")
    for s in (dict(), dict(temperature=T), dict(temperature=0.0), dict(min_p=0.3), dict(top_k=30, top_p=0.9),
              dict(top_k=torch.tensor([0, 3, 0, 2, 90, 0, 2000, 0, 7], dtype=torch.int32, device="cuda"), temperature=T,
                   top_p=torch.tensor([1, 0.5, 0.5, 1, 0.8, 1, 0.9, 0.5, 0.1], device="cuda"))):
        _say("longest specials", {k: type(v).__name__ for k, v in s.items()})
        _sample_check(wb.sample(t, u, **s), t, u, **s)
