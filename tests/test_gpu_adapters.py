"""GPU parity of the adapters beside the output layer with their 64-bit definition (score_ref.py, more_ref.py).

Tolerance: the layer's own (test_gpu_score.py: every term of S, the sum of the absolute terms, passes at most K / 32 +
40 additions of E = 2^-23), and for the adapters' sum of absolute terms A at most K / 4 additions of four in down, the
scale, rank additions in up and a few joins: |y - exact| <= h |y| + (K / 32 + 40) E S + (K / 4 + rank + 60) E A + tiny,
h half a step of the output's type.
"""

import numpy as np
import pytest
import torch

import more_ref
import score_ref as ref
import synth
import wfst_beam_search_amd as wb

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -23
INF = float("inf")


def _say(*a):
    print(*a, flush=True)


def _np(t):
    return t.detach().double().cpu().numpy()


def _layer(seed, K, N, group=64, scale="f16", zeros=True, bias=True):
    rng = np.random.default_rng(seed)
    w = rng.integers(0, 256, (N, (K + 1) // 2), dtype=np.uint8)
    ng = -(-K // group)
    s = torch.from_numpy(((0.5 + rng.random((N, ng))) / np.sqrt(K)).astype(np.float32)).to(DT[scale])
    z = rng.integers(0, 16, (N, ng), dtype=np.uint8) if zeros else None
    b = rng.normal(size=N).astype(np.float32) if bias else None
    layer = wb.OutputLayer(torch.from_numpy(w).cuda(), s.cuda(), zeros=None if z is None else torch.from_numpy(z).cuda(),
                           bias=None if b is None else torch.from_numpy(b).cuda(), in_features=K, group_size=group)
    return layer, (w, s.double().numpy(), z, b, K, group)


def _fill(ad, layer, seed, ranks, dtype):
    """Loads slot s with a random adapter of rank ranks[s] (0: left empty); returns what more_ref takes."""
    rng = np.random.default_rng(seed)
    K, N = layer.in_features, layer.out_features
    held = {}
    for s, r in enumerate(ranks):
        if r:
            down = torch.from_numpy((rng.normal(size=(r, K)) / np.sqrt(K)).astype(np.float32)).to(DT[dtype])
            up = torch.from_numpy(rng.normal(size=(N, r)).astype(np.float32)).to(DT[dtype])
            scale = float(0.5 + s % 3)
            ad.load(s, down.cuda(), up.cuda(), scale=scale)
            held[s] = (_np(down), _np(up), scale)
    return held


def _check(y, x, arrays, ids, held, out="f32", rank=128):
    K = arrays[4]
    xs = _np(x).reshape(-1, K)
    want, size = ref.layer(xs, *arrays)
    asize = 0.0
    if held:
        add, asize = more_ref.adapters(xs, ids, held)
        want = want + add
    got = _np(y).reshape(want.shape)
    sub = 2.0 ** -25 if out == "f16" else 1e-38
    tol = torch.finfo(DT[out]).eps / 2 * np.abs(want) * 1.001 + (K / 32 + 40) * E * size + sub
    tol = tol + (K / 4 + rank + 60) * E * asize
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("M,K,N,group,x,a,out,ranks", [
    (1, 32, 1, 32, "f16", "f16", "f32", [1]),
    (1, 1, 3, 32, "f32", "f32", "f32", [2, 16]),
    (3, 127, 17, 64, "bf16", "bf16", "bf16", [5, 0, 3]),
    (16, 128, 64, 128, "f16", "f32", "f16", [8] * 16),
    (17, 513, 65, 32, "f32", "f16", "f32", [17, 16, 15, 1]),
    (33, 640, 130, 256, "bf16", "f16", "f32", [32, 33]),
    (64, 1025, 129, 96, "f32", "bf16", "f16", [128, 0, 100]),
    (5, 8200, 70, 64, "f16", "bf16", "f32", [64, 7]),
    (100, 300, 40, 160, "bf16", "f32", "f32", [24] * 7),
    # whole tiles to a wavefront
    (1, 96, 24700, 32, "bf16", "bf16", "f32", [16]),
    (2, 130, 24577, 64, "f32", "f32", "bf16", [40, 3]),
    (11, 65, 24580, 32, "f16", "f16", "f16", [4, 0, 20]),
    # enough workgroups of many rows
    (17, 300, 16500, 64, "bf16", "f16", "f32", [12, 30]),
    (32, 130, 16400, 32, "f16", "f32", "f32", [8] * 40),
    (64, 390, 17001, 32, "f32", "f32", "f16", [24, 1, 17]),
    (3, 2050, 16500, 64, "f32", "bf16", "f32", [16, 16, 16]),
    (5, 2100, 16400, 32, "f16", "f16", "f32", [64]),
    (1000, 257, 1100, 96, "f16", "bf16", "bf16", [9, 16, 33]),
    (777, 512, 1300, 128, "bf16", "bf16", "f32", [32, 32, 0, 64, 1]),
])
def test_adapters(M, K, N, group, x, a, out, ranks):
    _say("adapters", M, K, N, group, x, a, out, ranks)
    layer, arrays = _layer(M * K + N, K, N, group)
    ad = wb.Adapters(layer, len(ranks), max(ranks), dtype=a)
    held = _fill(ad, layer, M, ranks, a)
    rng = np.random.default_rng(K)
    h = torch.from_numpy(rng.normal(size=(M, K)).astype(np.float32)).to(DT[x]).cuda()
    ids = rng.integers(-1, len(ranks), M).astype(np.int32)
    ids[0] = 0
    y = layer.logits(h, dtype=out, adapters=ad, ids=torch.from_numpy(ids).cuda())
    _check(y, h, arrays, ids, held, out, max(ranks))
    # rows without an adapter are the layer's, bit for bit
    none = torch.from_numpy(~np.isin(ids, list(held))).cuda()
    assert torch.equal(y[none], layer.logits(h, dtype=out)[none])
    for _ in range(2):
        assert torch.equal(y, layer.logits(h, dtype=out, adapters=ad, ids=ids))


@pytest.mark.parametrize("M,N", [(21, 90), (21, 17000), (600, 600)])
def test_ids_that_are_no_slot(M, N):
    K = 200
    layer, arrays = _layer(3, K, N)
    ad = wb.Adapters(layer, 3, 8, dtype="f16")
    held = _fill(ad, layer, 1, [8, 0, 5], "f16")
    h = torch.randn(M, K, device="cuda")
    some = np.array([-1, 3, 2 ** 31 - 1, -2 ** 31, 1, 0, 2], np.int32)
    ids = np.resize(some, M)
    y = layer.logits(h, adapters=ad, ids=torch.from_numpy(ids).cuda())
    _check(y, h, arrays, ids, held)
    ad.unload(0)
    del held[0]
    _check(layer.logits(h, adapters=ad, ids=torch.from_numpy(ids).cuda()), h, arrays, ids, held)
    for s in range(3):
        ad.unload(s)
    assert torch.equal(layer.logits(h, adapters=ad, ids=torch.from_numpy(ids).cuda()), layer.logits(h))


@pytest.mark.parametrize("M,N", [(16, 90), (16, 24600), (40, 17000), (600, 600)])
@pytest.mark.parametrize("a", ["f32", "f16", "bf16"])
def test_infinities_and_nan_stay_in_their_rows(M, N, a):
    K = 200
    layer, _ = _layer(4, K, N)
    ad = wb.Adapters(layer, 4, 20, dtype=a)
    _fill(ad, layer, 2, [20, 20, 20, 20], a)
    h = torch.randn(M, K, device="cuda")
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % 5 - 1
    clean = layer.logits(h, adapters=ad, ids=ids)
    up, down = torch.randn(N, 20).to(DT[a]).cuda(), torch.randn(20, K).to(DT[a]).cuda()
    up[3, 4], up[5, 0] = INF, float("nan")
    ad.load(2, down, up)
    down = down.clone()
    down[7, 7] = -INF
    ad.load(3, down, torch.ones(N, 20, dtype=DT[a], device="cuda"))
    h2 = h.clone()
    h2[1, 3], h2[6, 9] = INF, float("nan")
    y = layer.logits(h2, adapters=ad, ids=ids)
    keep = (ids < 2).clone()
    keep[1] = keep[6] = False
    assert torch.equal(y[keep], clean[keep])
    bad = ids == 2
    bad[[1, 6]] = False
    assert (y[bad, 3].abs() == INF).all() and torch.isnan(y[bad, 5]).all()
    fine = torch.ones(N, dtype=torch.bool, device="cuda")
    fine[[3, 5]] = False
    assert torch.isfinite(y[bad][:, fine]).all()
    worse = ids == 3
    worse[[1, 6]] = False
    assert (~torch.isfinite(y[worse])).all()
    assert torch.isnan(y[6]).all()


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [45, 1030, 24580])
def test_strides_lengths_and_untouched_rows(x, N):
    K, B, T = 200, 9, 70 if N < 2000 else 5
    layer, arrays = _layer(5, K, N)
    ad = wb.Adapters(layer, 5, 10, dtype="f16")
    held = _fill(ad, layer, 3, [10, 3, 0, 7, 9], "f16")
    buf = torch.randn(B, T, K + 13, device="cuda").to(DT[x])
    h = buf[:, :, 3:3 + K]
    L = torch.tensor([T, 0, 1, T // 2, 2, T, 3, 0, T - 1], dtype=torch.int32, device="cuda")
    act = torch.arange(T, device="cuda")[None] < L[:, None]
    h[~act] = float("nan")
    wide = torch.full((B, T, N + 9), 77.0, device="cuda")
    lane = torch.tensor([0, 1, 2, 3, 4, -1, 0, 7, 1], dtype=torch.int32, device="cuda")
    y = layer.logits(h, lengths=L, out=wide[:, :, 4:4 + N], adapters=ad, ids=lane)
    assert (wide[:, :, :4] == 77).all() and (wide[:, :, 4 + N:] == 77).all() and (wide[~act] == 77).all()
    rows = lane[:, None].expand(B, T).contiguous()
    _check(y[act], h[act], arrays, rows[act].cpu().numpy(), held)
    again = layer.logits(h, lengths=L, adapters=ad, ids=rows)                # one id a row
    assert torch.equal(again[act], y[act])
    rows[~act] = 2 ** 30                                                       # (of rows that hold nothing)
    assert torch.equal(layer.logits(h, lengths=L, adapters=ad, ids=rows)[act], y[act])
    all_of = layer.logits(h, lengths=L, adapters=ad, ids=np.int32(3))           # one for all
    _check(all_of[act], h[act], arrays, np.full(int(act.sum()), 3), held)
    z = layer.logits(h, lengths=L, adapters=ad, ids=[0, 1, 2, 3, 4, -5, 0, -1, 1])   # host values
    assert torch.equal(z[act], y[act])


def test_matrices_of_other_strides_and_reloads():
    K, N = 130, 50
    layer, arrays = _layer(7, K, N)
    ad = wb.Adapters(layer, 2, 24, dtype="bf16")
    db, ub = torch.randn(30, K + 7, device="cuda").bfloat16(), torch.randn(N, 40, device="cuda").bfloat16()
    h = torch.randn(9, K, device="cuda")
    ids = np.array([0, 1] * 4 + [0], np.int32)
    for r, off in ((24, 0), (5, 3), (17, 1), (1, 6)):         # larger ranks before smaller: nothing stays behind
        down, up = db[2:2 + r, off:off + K], ub[:, off:off + r]
        ad.load(1, down, up, scale=-1.5)
        _check(layer.logits(h, adapters=ad, ids=ids), h, arrays, ids, {1: (_np(down), _np(up), -1.5)})
    ad.load(1, db[:2, :K].expand(2, K)[:1].expand(3, K).contiguous(), ub[:, 4:7])
    wide = db.t().contiguous().t()                             # columns adjacent: refused
    with pytest.raises(ValueError, match="adjacent"):
        ad.load(1, wide[:4, :K], ub[:, :4])


def test_far_slots_and_rows():
    """Slots past 2^31 elements; rows of x and out more than 2^31 elements apart."""
    K, N = 64, 131072
    layer, _ = _layer(8, K, N, 32)
    ad = wb.Adapters(layer, 140, 128, dtype="bf16")
    down, up = torch.randn(128, K, device="cuda").bfloat16(), torch.randn(N, 128, device="cuda").bfloat16()
    ad.load(139, down, up)
    h = torch.randn(2, K, device="cuda")
    y = layer.logits(h, adapters=ad, ids=[139, -1])
    want = layer.logits(h[:1]).double() + (h[:1].double() @ down.double().t()) @ up.double().t()
    A = (h[:1].double().abs() @ down.double().abs().t()) @ up.double().abs().t()
    assert ((y[:1].double() - want).abs() <= (K / 4 + 190) * E * A + 2 * E * want.abs()).all()
    K, N = 130, 33
    layer, arrays = _layer(13, K, N, 32)
    ad = wb.Adapters(layer, 1, 4, dtype="f32")
    held = _fill(ad, layer, 4, [4], "f32")
    step = (1 << 31) + 17
    xb = torch.zeros(step + K, dtype=torch.float16, device="cuda")
    ob = torch.zeros(step + N, dtype=torch.float16, device="cuda")
    h = xb.as_strided((2, K), (step, 1))
    h.copy_(torch.randn(2, K))
    y = layer.logits(h, dtype="f16", out=ob.as_strided((2, N), (step, 1)), adapters=ad, ids=[0, 0])
    _check(y.contiguous(), h.contiguous(), arrays, [0, 0], held, "f16")


@pytest.mark.parametrize("a,x,values", [
    ("f32", "f32", [1e-30, 1e30, -3e20, 1.0000001, 16777217.0]),
    ("bf16", "bf16", [1e-30, 1e30, -3e20, 2.0, 1e-10]),
    ("f16", "f16", [6e-8, -6e-8, 6e-5, 1000.0, 1.0]),
    ("f16", "f32", [1e-20, 1e15, -3.0, 1.0, 1e-3]),
])
@pytest.mark.parametrize("M", [4, 700])
def test_extreme_values(a, x, values, M):
    """Hidden states and matrices of very different sizes beside each other."""
    K, N = 256, 20 if M < 10 else 600
    layer, arrays = _layer(9, K, N, 32, "f32")
    rng = np.random.default_rng(2)
    h = torch.zeros(M, K)
    for v in values:
        h[torch.arange(M), torch.from_numpy(rng.integers(0, K, M))] = v
    h = h.to(DT[x])
    down = torch.from_numpy((rng.normal(size=(20, K)) * 10.0 ** rng.integers(-3, 3, (20, 1))).astype(np.float32)).to(DT[a])
    up = torch.from_numpy((rng.normal(size=(N, 20)) * 10.0 ** rng.integers(-3, 2, (1, 20))).astype(np.float32)).to(DT[a])
    ad = wb.Adapters(layer, 1, 20, dtype=a)
    ad.load(0, down.cuda(), up.cuda(), scale=0.25)
    y = layer.logits(h.cuda(), adapters=ad, ids=np.zeros(M, np.int32))
    want, size = ref.layer(_np(h), *arrays)
    add, asize = more_ref.adapters(_np(h), [0] * M, {0: (_np(down), _np(up), 0.25)})
    big = np.abs(_np(h)).max() * 2.0 ** -38 * 16 * K * np.abs(arrays[1]).max()
    big = big if x == "f32" else (big / 2 if x == "bf16" else 0.0)
    tol = (K / 32 + 40) * E * size + (K / 4 + 80) * E * asize + big + 1e-41
    assert (np.abs(_np(y) - (want + add)) <= tol).all()


def test_captured_replays_read_the_slots_anew():
    K, N, B, T = 160, 1111, 6, 3
    layer, _ = _layer(23, K, N, 32)
    ad = wb.Adapters(layer, 3, 16, dtype="bf16")
    _fill(ad, layer, 5, [16, 9, 0], "bf16")
    h = torch.randn(B, T, K, device="cuda").bfloat16()
    ids = torch.zeros(B, dtype=torch.int32, device="cuda")
    L = torch.full((B,), T, dtype=torch.int32, device="cuda")
    tok = torch.zeros(B, T, dtype=torch.int32, device="cuda")

    def step():
        y = layer.logits(h, lengths=L, adapters=ad, ids=ids)
        return (y, *wb.token_scores(y, tok, top_n=4, lengths=L))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for i in range(4):
        h.copy_(torch.randn(B, T, K))
        ids.copy_(torch.randint(-1, 3, (B,), dtype=torch.int32))
        L.copy_(torch.randint(0, T + 1, (B,), dtype=torch.int32))
        tok.copy_(torch.randint(0, N, (B, T), dtype=torch.int32))
        ad.load(i % 3, torch.randn(4 + i, K, device="cuda").bfloat16(), torch.randn(N, 4 + i, device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        act = torch.arange(T, device="cuda")[None] < L[:, None]
        for a, b in zip(res, step()):
            assert torch.equal(a[act], b[act])


@pytest.mark.parametrize("N", [300, 24600, 17000])
def test_rows_do_not_depend_on_the_rows_beside_them(N):
    """Within a path of the layer (here: up to 16 rows, or more than 16 of a large layer)."""
    K = 300
    layer, _ = _layer(31, K, N)
    ad = wb.Adapters(layer, 9, 70, dtype="bf16")
    _fill(ad, layer, 9, [70, 16, 33, 1, 0, 48, 17, 64, 5], "bf16")
    M = 16 if N != 17000 else 80
    h = torch.randn(M, K, device="cuda")
    ids = torch.arange(M, device="cuda", dtype=torch.int32) * 5 % 10 - 1
    y = layer.logits(h, adapters=ad, ids=ids)
    for lo, hi in ((0, 1), (3, 4), (5, 11)) if M == 16 else ((0, 20), (33, 80)):
        assert torch.equal(layer.logits(h[lo:hi], adapters=ad, ids=ids[lo:hi]), y[lo:hi])


def test_most_slots_of_a_group():
    """Each of 64 rows with a slot of eight blocks of its own: lists past 64 entries."""
    K, N = 140, 16500
    layer, arrays = _layer(33, K, N)
    for a in ("f16", "f32"):
        ad = wb.Adapters(layer, 64, 128, dtype=a)
        held = _fill(ad, layer, 11, [128 - s % 7 for s in range(64)], a)
        h = torch.randn(64, K, device="cuda")
        ids = (torch.arange(64, device="cuda", dtype=torch.int32) * 11) % 64
        _check(layer.logits(h, adapters=ad, ids=ids), h, arrays, ids.cpu().numpy(), held)


@pytest.mark.parametrize("M,N", [(20, 300), (70, 17000)])
def test_sets_of_several_types_and_ranks_beside_one_layer(M, N):
    K = 96
    layer, arrays = _layer(35, K, N)
    h = torch.randn(M, K, device="cuda")
    ids = np.resize(np.array([0, 1, -1], np.int32), M)
    sets = []
    for a, rank in (("f32", 16), ("f16", 16), ("bf16", 16), ("f16", 40), ("bf16", 3)):
        ad = wb.Adapters(layer, 2, rank, dtype=a)
        sets.append((ad, _fill(ad, layer, rank, [rank, 1], a)))
    for ad, held in sets + sets[::-1]:
        _check(layer.logits(h, adapters=ad, ids=ids), h, arrays, ids, held)


def test_streams_at_once():
    K, N, R = 300, 17000, 70
    layer, _ = _layer(24, K, N)
    ad = wb.Adapters(layer, 4, 12, dtype="f16")
    _fill(ad, layer, 6, [12, 5, 7, 1], "f16")
    hs = [torch.randn(R, K, device="cuda") for _ in range(2)]
    ids = torch.arange(R, device="cuda", dtype=torch.int32) % 4
    want = [layer.logits(h, adapters=ad, ids=ids) for h in hs]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [layer.logits(h, adapters=ad, ids=ids, stream=s) for h, s in zip(hs, side)]
        host = layer.logits(hs[0], adapters=ad, ids=[r % 4 for r in range(R)], stream=side[1])
        junk = torch.full((R, N), 3.0, device="cuda")
        torch.cuda.synchronize()
        del junk
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(host, want[0])


def test_hidden_states_to_scores_and_words():
    """Hidden states with adapters to log-posteriors, the search's words, and the confidences of given labels."""
    g = synth.random_graph(61, n=80, deg=(1, 6), vocab=37, self_loop=0.3)
    dg = wb.Graph(g)
    K, B, T = 96, 4, 30
    layer, arrays = _layer(25, K, g.vocab, 32)
    ad = wb.Adapters(layer, 3, 8, dtype="f32")
    held = _fill(ad, layer, 7, [8, 4, 0], "f32")
    h = torch.randn(B, T, K, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    L = np.array([30, 17, 0, 9], np.int32)
    ids = [1, 0, 0, -1]
    lp = layer.log_probs(h, adapters=ad, ids=ids)
    rows = np.repeat(ids, T)
    xs = _np(h).reshape(-1, K)
    want, size = ref.layer(xs, *arrays)
    add, asize = more_ref.adapters(xs, rows, held)
    lps = ref.log_softmax(want + add).reshape(B, T, -1)
    slack = 2 * ((K / 32 + 40) * E * size + (K / 4 + 70) * E * asize).max() + 4 * E * (2 * np.abs(lps).max() + 16)
    assert (np.abs(_np(lp) - lps) <= slack).all()
    dec = wb.Decoder(dg, 8.0, 300, max_lanes=B, max_frames=T)
    r = dec.decode_hidden(layer, h, L, adapters=ad, ids=ids)
    w = dec.decode(lp, L)
    assert all(np.array_equal(a, b) for a, b in zip(r.arcs, w.arcs)) and np.array_equal(r.scores, w.scores)
    # streams, whose search does not know its last frames, against streams of the same rows' log-posteriors
    ch, other = dec.create_streams(2), dec.create_streams(2)
    for t0 in range(0, 30, 7):
        n = np.clip(L[:2] - t0, 0, 7).astype(np.int32)
        part = torch.zeros(2, 7, K, device="cuda")
        k = min(7, T - t0)
        part[:, :k] = h[:2, t0:t0 + k]
        dec.advance_hidden(ch, layer, part, n, adapters=ad, ids=ids[:2])
        rows = torch.zeros(2, 7, g.vocab, device="cuda")
        rows[:, :k] = lp[:2, t0:t0 + k]
        dec.advance_chunk(other, rows, n)
    for a, b in zip(ch, other):
        ra, rb = dec.finalize_stream(a), dec.finalize_stream(b)
        assert np.array_equal(ra.arcs[0], rb.arcs[0]) and ra.scores[0] == rb.scores[0]
        dec.release_stream(a)
        dec.release_stream(b)
    tok = lp.argmax(-1).int()
    Lg = torch.from_numpy(L).cuda()
    s = layer.token_scores(h, tok, top_n=3, lengths=Lg, adapters=ad, ids=ids)
    act = torch.arange(T, device="cuda")[None] < Lg[:, None]
    best = lp.gather(-1, tok[..., None].long())[..., 0]
    assert ((s.log_probs - best)[act].abs() <= 16 * E * (best[act].abs() + 16)).all()
    assert (s.ranks[act] == 0).all() and torch.equal(s.top_tokens[..., 0][act], tok[act])
    with pytest.raises(ValueError):
        dec.decode_hidden(layer, h, L, adapters=ad)
    dec.close()
    dg.release()


def test_refusals():
    K, N = 64, 10
    layer, _ = _layer(17, K, N, 32)
    other, _ = _layer(18, K, N + 1, 32)
    ad = wb.Adapters(layer, 3, 8, dtype="f16")
    _fill(ad, layer, 8, [8, 8, 8], "f16")
    h = torch.randn(4, K, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    for kw in (dict(adapters=ad), dict(ids=ids), dict(adapters=ad, ids=ids[:3]), dict(adapters=ad, ids=[0, 1, 2, 3]),
               dict(adapters=ad, ids=[0.0, 1.0, 0.0, 0.0]), dict(adapters=ad, ids=ids.view(2, 2))):
        with pytest.raises(ValueError):
            layer.logits(h, **kw)
    with pytest.raises(TypeError):
        layer.logits(h, adapters=ad, ids=ids.long())
    with pytest.raises(ValueError, match="size"):
        other.logits(h, adapters=ad, ids=ids)
    buf = torch.zeros(44, dtype=torch.int32, device="cuda")
    with pytest.raises(wb.WfstError, match="ids"):
        layer.logits(h, adapters=ad, ids=buf[:4], out=buf.view(torch.float32)[:40].view(4, 10))
    down, up = torch.randn(8, K, device="cuda").half(), torch.randn(N, 8, device="cuda").half()
    for bad, args in ((TypeError, (0, down.float(), up)), (TypeError, (0, down.cpu(), up)),
                      (ValueError, (0, down[:, :-1], up)), (ValueError, (0, down, up[:, :7])),
                      (ValueError, (0, down[:0], up[:, :0])), (wb.WfstError, (3, down, up)),
                      (wb.WfstError, (-1, down, up)), (wb.WfstError, (0, down, up, INF)),
                      (wb.WfstError, (0, torch.zeros(9, K, device="cuda").half(), torch.zeros(N, 9, device="cuda").half()))):
        with pytest.raises(bad):
            ad.load(*args)
    with pytest.raises(ValueError, match="gradient"):
        ad.load(0, down.requires_grad_(), up)
    for kw in (dict(slots=0, rank=8), dict(slots=3, rank=0), dict(slots=3, rank=129), dict(slots=1 << 17, rank=1)):
        with pytest.raises(wb.WfstError):
            wb.Adapters(layer, **kw)
    with pytest.raises(ValueError):
        wb.Adapters(layer, 1, 1, dtype="f64")
    with pytest.raises(wb.WfstError) as e:
        wb.Adapters(wb.OutputLayer(torch.zeros(1 << 20, 16, dtype=torch.uint8, device="cuda"),
                                   torch.ones(1 << 20, 1, device="cuda"), group_size=32), 1 << 16, 128)
    assert e.value.code == -3                                      # more than the card holds
    lib = wb.load_library()
    y = torch.empty(4, N, device="cuda")
    for per, work in ((3, y), (0, y), (1, None)):
        assert lib.wfst_layer_adapted_logits(layer.handle, ad.handle, ids.data_ptr(), per, h.data_ptr(), 0, K, 4, None, 1,
                                             y.data_ptr(), 0, N, None, 0, None) == -1
    assert layer.logits(h[:0], adapters=ad, ids=ids[:0]).shape == (0, N)
    ad.release()
    with pytest.raises(ValueError, match="released"):
        layer.logits(h, adapters=ad, ids=ids)
    with pytest.raises(ValueError, match="released"):
        ad.load(0, down, up)
