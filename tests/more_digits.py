"""Rows whose adapter's sum is one product, so that every digit of h shows in the result.

x has one feature a row that is not 0 and down is a part of the identity: h has one rank that is not 0, scale * x, and
y = h * up exactly one term. Roundings on the way, in units of E = 2^-23 of y: scale * x half of one; binary16 up: h in
two parts off by one, their sum half of one; bfloat16 up: three parts (exact) in three sums, one each; binary32 up: one.
All together at most 3.5: |y - exact| <= 4 E |exact|. A part that went missing would be off by 2^-16 (the third of
bfloat16), 2^-12 (the second of binary16).
"""

import numpy as np
import torch

E = 2.0 ** -23
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SCALE = float(np.float32(0.7310586))


def inputs(seed, M, K, rank, N, x, a):
    """(x [M, K], down [rank, K], up [N, rank]) as CPU tensors of their types."""
    rng = np.random.default_rng(seed)
    v = rng.normal(size=M) * (2.0 ** rng.integers(-20, 21, M) if x != "f16" else 1.0)
    v[np.abs(v) < 2.0 ** -24] = 1.0
    xs = np.zeros((M, K), np.float32)
    xs[np.arange(M), np.arange(M) % rank] = v
    up = rng.normal(size=(N, rank))
    up[np.abs(up) < 2.0 ** -10] = 1.0
    return torch.from_numpy(xs).to(DT[x]), torch.eye(rank, K).to(DT[a]), torch.from_numpy(up).to(DT[a])


def exact(x, up):
    """(h [M], y [M, N]) in 64 bits."""
    M, rank = x.shape[0], up.shape[1]
    j = np.arange(M) % rank
    h = SCALE * x.double().numpy()[np.arange(M), j]
    return h, h[:, None] * up.double().numpy().T[j]


def wrong(y, want):
    return ~(np.abs(y - want) <= 4 * E * np.abs(want))
