"""Edges of the adapters beside the output layer and of the token scores, each against its definition."""

import numpy as np
import pytest
import torch

import more_digits as digits
import wfst_beam_search_amd as wb
import test_gpu_adapters as adapters
from test_gpu_token_scores import _check as check_scores

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -23
INF = float("inf")
# rows and features: few rows with K over the wavefronts, with a wavefront a tile, many rows, past 512 rows (few, many)
PATHS = [(5, 70), (2, 24580), (40, 17000), (600, 600), (600, 17000)]


def _silent_layer(K, N):
    """A layer whose own logits are 0: scales of 0, no bias."""
    q = torch.randint(0, 256, (N, (K + 1) // 2), dtype=torch.uint8, device="cuda")
    return wb.OutputLayer(q, torch.zeros(N, -(-K // 32), device="cuda"), in_features=K, group_size=32)


@pytest.mark.parametrize("M,N", PATHS)
@pytest.mark.parametrize("a,big,small", [
    ("f32", 2.0 ** 30, 2.0 ** -15), ("f32", 1.0, 2.0 ** -149),
    ("bf16", 2.0 ** 30, 2.0 ** -15), ("bf16", 1.0, 2.0 ** -133), ("bf16", 1.0, 2.0 ** -140), ("bf16", 1.0, 2.0 ** -149),
    ("f16", 2.0 ** 30, 2.0 ** -15), ("f16", 2.0 ** 30, 2.0 ** -126), ("f16", 2.0 ** 100, 2.0 ** -149),
    ("f16", 2.0 ** 30, 1.25 * 2.0 ** -10),
])
def test_an_infinite_weight_meets_a_small_h(M, N, a, big, small):
    """h of very different sizes among a row's 16 ranks: the small ones' infinite weights give infinities of their
    sign (not NaN), and their finite weights their product, off by at most 2^-50 of the largest h (binary16) or what
    lies below 2^-126 (bfloat16), and a binary32 rounding or two."""
    K = 32
    layer = _silent_layer(K, N)
    ad = wb.Adapters(layer, 1, 20, dtype=a)
    down, up = torch.eye(20, K), torch.zeros(N, 20)
    up[1::4, 1], up[2::4, 2], up[3::4, 3] = INF, INF, 3.0
    ad.load(0, down.to(DT[a]).cuda(), up.to(DT[a]).cuda())
    h = torch.zeros(M, K)
    h[:, 0], h[:, 1], h[:, 2], h[:, 3] = big, small, -small, small
    y = layer.logits(h.cuda(), adapters=ad, ids=np.zeros(M, np.int32)).double().cpu()
    assert (y[:, 0::4] == 0).all() and (y[:, 1::4] == INF).all() and (y[:, 2::4] == -INF).all()
    lost = {"f32": 0.0, "f16": 2.0 ** -50 * big, "bf16": 2.0 ** -126}[a]
    assert ((y[:, 3::4] - 3 * small).abs() <= 3 * lost + 3 * E * 3 * small + 2.0 ** -149).all()


@pytest.mark.parametrize("M,N", PATHS)
@pytest.mark.parametrize("x,a", [("f32", "f32"), ("f32", "f16"), ("f16", "f16"), ("f32", "bf16"), ("bf16", "bf16"),
                                 ("bf16", "f32"), ("f16", "bf16")])
def test_h_keeps_its_binary32_digits(M, N, x, a):
    K, rank = 70, 40
    layer = _silent_layer(K, N)
    xs, down, up = digits.inputs(M + N, M, K, rank, N, x, a)
    ad = wb.Adapters(layer, 2, rank, dtype=a)
    ad.load(1, down.cuda(), up.cuda(), scale=digits.SCALE)
    y = layer.logits(xs.cuda(), adapters=ad, ids=np.ones(M, np.int32)).double().cpu().numpy()
    want = digits.exact(xs, up)[1]
    bad = digits.wrong(y, want)
    assert not bad.any(), (np.argwhere(bad)[:4], y[bad][:4], want[bad][:4])


@pytest.mark.parametrize("V", [2, 30, 500, 3000, 6007, 30011])
@pytest.mark.parametrize("T", [2.0 ** -149, 3 * 2.0 ** -149, 2.0 ** -140, 2.0 ** -127, 2.0 ** -126, 1.5 * 2.0 ** -126, 2.0 ** -125])
def test_temperatures_of_the_smallest_numbers(V, T):
    """Scores as close to each other as such a temperature tells apart, far ones and large ones beside them."""
    rng = np.random.default_rng(V)
    x = np.zeros((7, V), np.float32)
    for r, steps in enumerate((1.0, 0.3, 4.0)):         # multiples of T, rounded to the numbers there are
        x[r] = -np.abs(rng.normal(size=V)) * steps * T
    x[2, ::3] = -1.0
    x[3] = np.float32(2.0 ** -130) - x[0]
    x[4] = rng.normal(size=V)
    x[5] = rng.choice(np.array([3e38, 2.9e38, 1.0, -3e38], np.float32), V)
    x[6] = rng.choice(np.array([-3e38, -3.1e38, -np.inf], np.float32), V)
    s = torch.from_numpy(x).cuda()
    tok = torch.from_numpy(rng.integers(0, V, (7, 4)).astype(np.int32)).cuda()
    check_scores(wb.token_scores(s, tok, top_n=5, temperature=T), s, tok, 5, T)
    check_scores(wb.token_scores(s, tok, top_n=5, temperature=torch.full((7,), T, device="cuda")), s, tok, 5, T)


def test_emptying_a_slot_ignores_the_matrices():
    """Rank 0 with pointers that are no matrices, as the header allows; with a rank they are refused."""
    lib = wb.load_library()
    layer = _silent_layer(32, 8)
    ad = wb.Adapters(layer, 2, 4, dtype="f32")
    ad.load(1, torch.eye(4, 32, device="cuda"), torch.ones(8, 4, device="cuda"))
    h = torch.ones(3, 32, device="cuda")
    assert (layer.logits(h, adapters=ad, ids=[1, 1, 1]) == 4).all()
    assert lib.wfst_adapters_load(ad.handle, 1, 1, 2, 32, 3, 4, 1.0, None) == -1
    assert lib.wfst_adapters_load(ad.handle, 1, 0, 2, -5, 3, 0, 1.0, None) == 0
    assert (layer.logits(h, adapters=ad, ids=[1, 1, 1]) == 0).all()


@pytest.mark.parametrize("V,x", [(600011, "f32"), ((1 << 20) + 9, "bf16"), (524289, "f16")])
def test_many_tokens_of_rows_whose_pieces_take_several_runs(V, x):
    g = torch.Generator(device="cuda").manual_seed(V)
    t = (torch.randn(3, V, generator=g, device="cuda") * 3).to(DT[x])
    t[1, ::2] = -INF
    for C in (65, 200, 256):
        tok = torch.randint(-1, V + 1, (3, C), generator=g, device="cuda", dtype=torch.int32)
        tok[:, 64] = t.float().argmax(-1).int()
        for n in (0, 40):
            check_scores(wb.token_scores(t, tok, top_n=n), t, tok, n)


@pytest.mark.parametrize("N", [333, 5000, 17000])
@pytest.mark.parametrize("x,a", [("f16", "f16"), ("bf16", "f32"), ("f32", "bf16")])
def test_ids_of_each_frame_past_512_rows(N, x, a):
    """ids [B, T] of a padded batch, other slots beside each other, runs, repeats, none."""
    B, T, K = 6, 151, 260
    layer, arrays = adapters._layer(N, K, N)
    ranks = [40, 3, 0, 16, 17, 1, 33, 48, 8]
    ad = wb.Adapters(layer, len(ranks), 48, dtype=a)
    held = adapters._fill(ad, layer, N, ranks, a)
    rng = np.random.default_rng(N)
    h = torch.from_numpy(rng.normal(size=(B, T, K)).astype(np.float32)).to(DT[x]).cuda()
    ids = rng.integers(-1, len(ranks), (B, T)).astype(np.int32)
    ids[1] = np.arange(T) // 20 % len(ranks)
    ids[2, :40] = 7
    lens = np.array([T, T - 3, 100, T, 7, T], np.int32)
    L = torch.from_numpy(lens).cuda()
    act = torch.arange(T, device="cuda")[None] < L[:, None]
    h[~act] = float("nan")
    y = layer.logits(h, lengths=L, adapters=ad, ids=torch.from_numpy(ids).cuda())
    adapters._check(y[act], h[act], arrays, ids[act.cpu().numpy()], held)
    assert torch.equal(layer.logits(h, lengths=lens, adapters=ad, ids=ids)[act], y[act])
