"""GPU parity of the scores of given tokens with their 64-bit definition (more_ref.py).

Tolerances, from the arithmetic (E = 2^-23 bounds any single binary32 rounding): a scaled distance d from the
maximum is rounded three times (difference, 1 / T, product); an exponential is off by about its argument's rounding,
whose mean under the row's own distribution is at most ln V, and sums of V terms by V / 1024 + 12 additions each:
* log-probabilities: |lp - exact| <= 4 E (|lp| + ln V + 8 + V / 1024).
* entropy, lz plus a mean of |d| <= ln V with weights off by 2 E |d| + (16 + V / 1024) E:
  <= 4 E (ln^2 V + (1 + ln V) (16 + V / 1024)).
Ranks and top tokens are equal.
"""

import numpy as np
import pytest
import torch

import more_ref as ref
import wfst_beam_search_amd as wb

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -23
INF = float("inf")


def _say(*a):
    print(*a, flush=True)


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, tol):
    with np.errstate(invalid="ignore"):
        ok = (got == want) | (np.isnan(got) & np.isnan(want)) | (np.abs(got - want) <= tol)
    ok |= (want < -3.4028e38) & (got == -np.inf)           # past binary32's range
    assert ok.all(), (np.argwhere(~ok)[:4], got[~ok][:4], want[~ok][:4])


def _check(r, x, tokens, n, T=1.0):
    V = x.shape[-1]
    R = x.numel() // V
    tok = np.zeros((R, 0), np.int64) if tokens is None else tokens.cpu().numpy().reshape(R, -1)
    lp, rank, ent, tt, tl = ref.scores(_np(x).reshape(R, V), tok, n, _np(T).reshape(R) if torch.is_tensor(T) else T)
    ln = np.log(V) + 0.0

    def lp_tol(w):
        with np.errstate(invalid="ignore"):
            return 4 * E * (np.abs(w) + ln + 8 + V / 1024)

    if tokens is None:
        assert r.log_probs is None and r.ranks is None
    else:
        assert r.log_probs.shape == tokens.shape and r.ranks.shape == tokens.shape
        assert np.array_equal(r.ranks.cpu().numpy().reshape(R, -1), rank)
        _close(_np(r.log_probs).reshape(R, -1), lp, lp_tol(lp))
    _close(_np(r.entropies).reshape(R), ent, 4 * E * (ln * ln + (1 + ln) * (16 + V / 1024)))
    if n:
        assert np.array_equal(r.top_tokens.cpu().numpy().reshape(R, n), tt)
        _close(_np(r.top_log_probs).reshape(R, n), tl, lp_tol(tl))
    else:
        assert r.top_tokens is None and r.top_log_probs is None


def _tokens(g, x, C):
    V = x.shape[-1]
    t = torch.randint(0, V, (*x.shape[:-1], C), generator=g, device="cuda", dtype=torch.int32)
    t[..., 0] = x.float().argmax(-1).int()
    return t


@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 63, 64, 65, 500, 511, 513, 1025, 2047, 2049, 4097, 5000, 8191, 8193, 16384,
                               16387, 40001, 131071])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_token_scores(V, x):
    g = torch.Generator(device="cuda").manual_seed(V)
    for R in (1, 6, 70 if V < 9000 else 19):
        for sigma in (0.4, 4.0):
            t = (torch.randn(R, V, generator=g, device="cuda") * sigma).to(DT[x])
            for C, n, T in ((1, 0, 1.0), (1, 5, 0.7), (3, 20, 1.0), (17, 64, 2.5), (0, 1, 1.0)):
                _say("token scores", V, x, R, sigma, C, n, T)
                tok = _tokens(g, t, C) if C else None
                _check(wb.token_scores(t, tok, top_n=n, temperature=T), t, tok, n, T)


@pytest.mark.parametrize("V", [9, 500, 5003, 20011, 70003])
def test_masks_and_specials(V):
    t = torch.randn(14, V) * 3
    t[0] = -INF                                     # a row whose mask leaves nothing
    t[1] = -INF
    t[1, V - 1] = -2.5                              # one label left
    t[2, 1], t[2, 5] = INF, INF
    t[3, 0] = float("nan")
    t[4] = torch.finfo(torch.float32).min           # masks of the type's lowest value
    t[5] = torch.finfo(torch.float32).min
    t[5, 1] = 3.0
    t[6] = float("nan")
    t[7, 1:] = -30.0                                # a dominant label
    t[7, 0] = 10.0
    t[8, ::2] = -INF
    t[9] = torch.tensor([0.0, -0.0]).repeat(V)[:V]
    t[10] = 1.5                                     # all equal
    t[11] = 1e30
    t[12] = -3e38
    t[12, 3] = 3e38
    t[13, ::3] = float("nan")
    t = t.cuda()
    tok = torch.tensor([0, V - 1, 1, 5, -1, V, 2 ** 31 - 1, -2 ** 31, 3, V // 2], dtype=torch.int32, device="cuda")
    tok = tok.repeat(14, 1)
    for x in ("f32", "bf16"):
        s = t.to(DT[x])
        for n in (0, 3, 64):
            for T in (1.0, 0.0, 0.3, 5.0):
                _say("specials", V, x, n, T)
                _check(wb.token_scores(s, tok, top_n=n, temperature=T), s, tok, n, T)
    r = wb.token_scores(t, tok, top_n=3)
    # a dominant label's digits survive (relative, not absolute): e^-40 by way of a rounded argument of 40, its
    # constant and the sums
    lead = ref.scores_row(_np(t[7]), np.array([0]), 1)
    assert abs(float(r.log_probs[7, 0]) - lead[0][0]) <= 52 * E * abs(lead[0][0])
    assert abs(float(r.entropies[7]) - lead[2]) <= 52 * E * lead[2]


@pytest.mark.parametrize("V", [30, 3000, 30011])
def test_temperatures_per_row(V):
    T = torch.tensor([1.0, 0.0, -1.0, float("nan"), INF, 1e-45, 1e-30, 3e38, 1e30, 1e-3, 0.5, 20.0], device="cuda")
    t = torch.randn(12, V, device="cuda")
    t[:, ::3] = -INF
    tok = torch.randint(0, V, (12, 4), dtype=torch.int32, device="cuda")
    _check(wb.token_scores(t, tok, top_n=6, temperature=T), t, tok, 6, T)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("V", [200, 1600, 6007, 30011, 66011])
def test_orders_that_crowd_the_alternatives(V, x):
    """Falling and rising scores, all equal, few distinct values, the best labels side by side or far apart."""
    t = torch.empty(8, V)
    t[0] = -torch.arange(V) * 1e-3
    t[1] = torch.arange(V) * 1e-3
    t[2] = 1.5
    t[3] = -1e30
    t[3, V // 2:V // 2 + 40] = torch.randn(40)
    t[4] = (torch.randn(V) * 2).round()
    t[5] = torch.randn(V)
    t[5, :V // 2] += 20.0
    t[6] = torch.randn(V)
    t[6, ::256] += 30.0
    t[7] = torch.randn(V)
    t[7, 8:16] = t[7, 64:72] = 40.0
    t = t.to(DT[x]).cuda()
    tok = torch.tensor([0, V - 1, V // 2, 8, 71], dtype=torch.int32, device="cuda").repeat(8, 1)
    for n in (1, 2, 20, 63, 64):
        _say("orders", V, x, n)
        _check(wb.token_scores(t, tok, top_n=n), t, tok, n)


@pytest.mark.parametrize("V", [6, 77, 500, 5003, 20001, 70001])
@pytest.mark.parametrize("x", ["f32", "f16"])
def test_strides_lengths_and_untouched_rows(V, x):
    B, T, C, n = 4, 6, 2, 3
    L = torch.tensor([6, 0, 1, 5], dtype=torch.int32, device="cuda")
    act = torch.arange(T, device="cuda")[None] < L[:, None]
    for off in (0, 1, 3):
        buf = (torch.randn(B, T, V + 11, device="cuda") * 3).to(DT[x])
        t = buf[:, :, off:off + V]
        t[~act] = float("nan")                       # frames behind the last are not read
        tok = torch.randint(0, V, (B, T, C), dtype=torch.int32, device="cuda")
        out = (torch.full((B, T, C), -9.0, device="cuda"), torch.full((B, T, C), -9, dtype=torch.int32, device="cuda"),
               torch.full((B, T), -9.0, device="cuda"), torch.full((B, T, n), -9, dtype=torch.int32, device="cuda"),
               torch.full((B, T, n), -9.0, device="cuda"))
        r = wb.token_scores(t, tok, top_n=n, lengths=L, out=out)
        for o, mine in zip(r, out):
            assert o is mine and (o[~act] == -9).all()
        _check(wb.TokenScores(*(o[act] for o in r)), t[act], tok[act], n)
        again = wb.token_scores(t, tok, top_n=n, lengths=[6, 0, 1, 5])
        for a, b in zip(r, again):
            assert torch.equal(a[act], b[act])
    one = torch.randn(V, device="cuda")
    r = wb.token_scores(one, torch.tensor(V - 1, dtype=torch.int32, device="cuda"), top_n=2)
    assert r.entropies.shape == () and r.top_tokens.shape == (2,) and r.log_probs.shape == ()
    _check(r, one, torch.tensor([V - 1], dtype=torch.int32).reshape(()), 2)


def test_far_rows():
    V, step = 700, (1 << 31) + 5
    xb = torch.zeros(step + V, dtype=torch.float16, device="cuda")
    t = xb.as_strided((2, V), (step, 1))
    t.copy_(torch.randn(2, V))
    tok = torch.tensor([3, 699], dtype=torch.int32, device="cuda")
    _check(wb.token_scores(t, tok, top_n=4), t.contiguous(), tok, 4)


def test_longest_rows():
    V = (1 << 20) + 3
    g = torch.Generator(device="cuda").manual_seed(9)
    t = torch.randn(3, V, generator=g, device="cuda") * 3
    t[1] = torch.arange(V, device="cuda") * 1e-4
    t[2] = 0.0
    tok = torch.tensor([[0, V - 1], [V - 3, 5], [7, V - 1]], dtype=torch.int32, device="cuda")
    for n in (0, 20, 64):
        _check(wb.token_scores(t, tok, top_n=n), t, tok, n)
    t = torch.randn(1 << 24, generator=g, device="cuda").half()
    tok = torch.tensor([1 << 23], dtype=torch.int32, device="cuda")
    r = wb.token_scores(t, tok, top_n=64)
    order = torch.sort(t, descending=True, stable=True).indices
    assert torch.equal(r.top_tokens.long(), order[:64])
    assert int(r.ranks[0]) == int((order == (1 << 23)).nonzero()[0, 0])
    d = t.double() - t.double().max()
    lz = torch.logsumexp(d, 0)
    assert abs(float(r.log_probs[0]) - float(d[1 << 23] - lz)) <= 4 * E * (40 + 8 + V / 64)


def test_many_rows_and_many_tokens():
    R = (1 << 20) + 5
    t = torch.randn(R, 4, device="cuda")
    tok = torch.randint(0, 4, (R,), dtype=torch.int32, device="cuda")
    r = wb.token_scores(t, tok, top_n=2)
    order = torch.sort(t, descending=True, stable=True, dim=-1).indices
    lp = torch.log_softmax(t.double(), -1)
    assert torch.equal(r.top_tokens.long(), order[:, :2])
    assert torch.equal(r.ranks.long(), (order == tok[:, None].long()).int().argmax(-1))
    assert ((r.log_probs.double() - lp.gather(1, tok[:, None].long())[:, 0]).abs() <= 1e-5).all()
    assert ((r.entropies.double() + (lp.exp() * lp).sum(-1)).abs() <= 1e-5).all()
    for V in (900, 70001):
        t = torch.randn(3, V, device="cuda").bfloat16()
        tok = torch.randint(-2, V + 2, (3, 256), dtype=torch.int32, device="cuda")
        _check(wb.token_scores(t, tok, top_n=1), t, tok, 1)


def test_log_probabilities_of_the_log_softmax_and_the_draw():
    """Scores of the log-softmax's rows are its entries; of drawn tokens without cuts what the draw says."""
    t = torch.randn(40, 900, device="cuda") * 3
    lp = wb.log_softmax(t)
    drawn = wb.sample(t, torch.rand(40, device="cuda"))
    r = wb.token_scores(lp, drawn.tokens, top_n=1)
    want = lp.gather(1, drawn.tokens[:, None].long())[:, 0]
    assert ((r.log_probs - want).abs() <= 16 * E * (want.abs() + 16)).all()
    assert ((r.log_probs - drawn.log_probs).abs() <= 16 * E * (want.abs() + 16)).all()
    greedy = wb.sample(t, torch.rand(40, device="cuda"), temperature=0.0)
    assert torch.equal(greedy.tokens, r.top_tokens[:, 0])


@pytest.mark.parametrize("B,T,V", [(6, 3, 1111), (4, 5, 70003), (30, 1, 20011)])
def test_captured_replays_and_streams(B, T, V):
    x = torch.randn(B, T, V, device="cuda").bfloat16()
    tok = torch.randint(0, V, (B, T), dtype=torch.int32, device="cuda")
    L = torch.full((B,), T, dtype=torch.int32, device="cuda")

    def step(stream=None):
        return wb.token_scores(x, tok, top_n=7, temperature=0.9, lengths=L, stream=stream)

    want = step()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [step(s) for s in side]
        junk = torch.full((B, T, V), 5.0, device="cuda")
        torch.cuda.synchronize()
        del junk
        for r in got:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for i in range(4):
        x.copy_(torch.randn(B, T, V))
        tok.copy_(torch.randint(0, V, (B, T), dtype=torch.int32))
        L.copy_(torch.randint(0, T + 1, (B,), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        act = torch.arange(T, device="cuda")[None] < L[:, None]
        for a, b in zip(res, step()):
            assert torch.equal(a[act], b[act])


def test_refusals():
    t = torch.randn(4, 10, device="cuda")
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad, kw in ((ValueError, dict(top_n=65)), (ValueError, dict(top_n=-1)), (wb.WfstError, dict(temperature=-1.0)),
                    (wb.WfstError, dict(temperature=float("nan"))), (wb.WfstError, dict(temperature=INF)),
                    (ValueError, dict(temperature=torch.ones(3, device="cuda"))), (ValueError, dict(lengths=[1])),
                    (ValueError, dict(out=(torch.empty(4, device="cuda"),))),
                    (ValueError, dict(out=(torch.empty(5, device="cuda"), tok.clone(), torch.empty(4, device="cuda"))))):
        with pytest.raises(bad):
            wb.token_scores(t, tok, **kw)
    with pytest.raises(TypeError):
        wb.token_scores(t, tok.long())
    with pytest.raises(TypeError):
        wb.token_scores(t, tok.cpu())
    with pytest.raises(ValueError):
        wb.token_scores(t, tok[:3])
    with pytest.raises(wb.WfstError, match="tokens_per_row"):
        wb.token_scores(t, torch.zeros(4, 257, dtype=torch.int32, device="cuda"))
    e = torch.empty(4, device="cuda")
    with pytest.raises(wb.WfstError, match="overlaps"):
        wb.token_scores(t, tok, out=(e, tok, torch.empty(4, device="cuda")))
    with pytest.raises(wb.WfstError, match="overlaps"):
        wb.token_scores(t, tok, out=(e, tok.clone(), e))
    with pytest.raises(wb.WfstError, match="overlaps"):
        wb.token_scores(t, tok, out=(t.view(-1)[:4], tok.clone(), e))
    L = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    both = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(wb.WfstError, match="lengths"):
        wb.token_scores(t.view(2, 2, 10), tok.view(2, 2), lengths=both[:2],
                        out=(e.view(2, 2), both[:4].view(2, 2), torch.empty(2, 2, device="cuda")))
    assert wb.token_scores(t.view(2, 2, 10), tok.view(2, 2), lengths=L).ranks.shape == (2, 2)
    h = t.clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        wb.token_scores(h, tok)
    with torch.no_grad():
        wb.token_scores(h, tok)
    r = wb.token_scores(t[:0], tok[:0], top_n=3)
    assert r.log_probs.shape == (0,) and r.top_tokens.shape == (0, 3)
    r = wb.token_scores(t, tok.view(4, 1)[:, :0])
    assert r.log_probs.shape == (4, 0) and r.entropies.shape == (4,)
    saved = torch.rand(4, device="cuda", requires_grad=True).exp()
    wb.token_scores(t, tok, out=(saved.detach(), tok.clone(), e))
    with pytest.raises(RuntimeError, match="inplace"):
        saved.sum().backward()
