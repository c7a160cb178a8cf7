"""The operators between a model's last hidden state and its answer, as they are measured.

Three operators: the output layer with 4-bit weights (hidden states to logits), the log-softmax that makes the
search's log-posteriors of them, and the draw of tokens from scores. A case is one of them at one size; ``run``
computes it in plain torch operations, or (``own``) through the package's entry points.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one frame of one stream, the vocabulary of a mid-size graph: the smallest call
        dict(name="layer_frame_500", op="layer", M=1, K=512, N=500, group=64, x="f16", scale="f16", out="f32",
             zeros=False, bias=True, pad=0),
        # one frame of each of 32 streams, a 5000-label model
        dict(name="layer_lanes_5000", op="layer", M=32, K=1024, N=5000, group=128, x="bf16", scale="bf16", out="f32",
             zeros=True, bias=True, pad=0),
        # one new token, a large vocabulary: the weights' bytes
        dict(name="layer_token_131072", op="layer", M=1, K=4096, N=131072, group=128, x="bf16", scale="f16", out="f32",
             zeros=False, bias=False, pad=0),
        # a batch of 64 sequences, no size a multiple of a tile, rows of a wider buffer
        dict(name="layer_batch_odd", op="layer", M=64, K=2050, N=32003, group=32, x="f32", scale="f32", out="f16",
             zeros=True, bias=False, pad=14),
        # one frame of each of 8 streams
        dict(name="norm_frames_500", op="norm", B=8, T=1, V=500, x="f32", out="f32", bias=False, ragged=False),
        # an offline batch of 32 utterances of 300 to 500 frames, a blank penalty, the search's fp16 rows
        dict(name="norm_utterances_5000", op="norm", B=32, T=500, V=5000, x="f32", out="f16", bias=True, ragged=True),
        # the widest batch: many short rows
        dict(name="norm_wide_500", op="norm", B=64, T=1000, V=500, x="bf16", out="f32", bias=False, ragged=False),
        # few rows of a large, odd vocabulary
        dict(name="norm_tokens_131071", op="norm", B=16, T=1, V=131071, x="bf16", out="f32", bias=True, ragged=False),
        # the next token of one sequence: latency
        dict(name="sample_token_131072", op="sample", B=1, T=1, V=131072, x="f32", kind="tokens", params="scalar",
             temperature=0.8, top_k=50, top_p=0.9, min_p=0.0, ragged=False),
        # a serving batch, each sequence with settings of its own (greedy, top-k, top-p, min-p, none)
        dict(name="sample_batch_131072", op="sample", B=256, T=1, V=131072, x="bf16", kind="tokens", params="rows",
             temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, ragged=False),
        # the nucleus alone, an odd vocabulary
        dict(name="sample_nucleus_32003", op="sample", B=48, T=1, V=32003, x="f32", kind="tokens", params="scalar",
             temperature=1.0, top_k=0, top_p=0.95, min_p=0.0, ragged=False),
        # alignments drawn frame by frame from the search's fp16 rows of an offline batch
        dict(name="sample_frames_5000", op="sample", B=32, T=500, V=5000, x="f16", kind="frames", params="scalar",
             temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer", "norm", "sample"])
    if op == "layer":
        K = _log_int(rng, 200, 4096)
        N = _log_int(rng, 100, 131072)
        M = _log_int(rng, 1, 64)
        M = max(1, min(M, int(64 * 32003 * 2050 / (N * K))))
        return dict(op="layer", M=M, K=K, N=N, group=rng.choice([32, 64, 128]), x=rng.choice(["f16", "bf16", "f32"]),
                    scale=rng.choice(["f16", "bf16", "f32"]), out=rng.choice(["f16", "bf16", "f32"]),
                    zeros=rng.random() < 0.5, bias=rng.random() < 0.5, pad=rng.choice([0, 0, 3, 8]))
    V = _log_int(rng, 2, 131072)
    rows = _log_int(rng, 1, min(64000, 32 * 500 * 5000 // V))
    B = rng.randint(1, min(64, rows))
    T = max(1, rows // B)
    if op == "norm":
        return dict(op="norm", B=B, T=T, V=V, x=rng.choice(["f32", "f16", "bf16"]),
                    out=rng.choice(["f32", "f16", "bf16"]), bias=rng.random() < 0.5, ragged=rng.random() < 0.5)
    return dict(op="sample", B=B, T=T, V=V, x=rng.choice(["f32", "f16", "bf16"]),
                kind=rng.choice(["tokens", "frames"]), params=rng.choice(["scalar", "rows"]),
                temperature=rng.choice([0.6, 0.8, 1.0, 1.3]), top_k=rng.choice([0, 0, 5, 50, 700]),
                top_p=rng.choice([1.0, 0.5, 0.9, 0.95]), min_p=rng.choice([0.0, 0.0, 0.02, 0.1]),
                ragged=rng.random() < 0.3)


# ---- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _lengths(case, g):
    """Valid frames of each lane: 60 % to all of T."""
    if not case["ragged"]:
        return None
    T = case["T"]
    lo = (3 * T + 4) // 5
    return torch.randint(lo, T + 1, (case["B"],), generator=g, device="cuda", dtype=torch.int32)


def _layer_inputs(case, seed):
    g = _gen(seed)
    M, K, N = case["M"], case["K"], case["N"]
    ng = -(-K // case["group"])
    x = _normal(g, M, K + case["pad"]).to(_DT[case["x"]])[:, :K]
    kb = (K + 1) // 2
    q = torch.empty((N, kb), dtype=torch.uint8, device="cuda")
    for n0 in range(0, N, 16384):              # normally distributed weights, quantised to 16 steps
        n1 = min(N, n0 + 16384)
        lo = (_normal(g, n1 - n0, kb) * 2.7 + 8.0).round_().clamp_(0, 15).to(torch.uint8)
        hi = (_normal(g, n1 - n0, kb) * 2.7 + 8.0).round_().clamp_(0, 15).to(torch.uint8)
        q[n0:n1] = lo | (hi << 4)
    scales = ((0.5 + torch.rand((N, ng), generator=g, device="cuda")) * (0.37 / math.sqrt(K))).to(_DT[case["scale"]])
    zeros = torch.randint(6, 11, (N, ng), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    bias = _normal(g, N) if case["bias"] else None
    return dict(x=x, q=q, scales=scales, zeros=zeros, bias=bias)


def _norm_inputs(case, seed):
    g = _gen(seed)
    B, T, V = case["B"], case["T"], case["V"]
    x = _normal(g, B, T, V).mul_(4.0)
    x[..., 0] += 5.0                            # the blank's share of a CTC model
    x = x.to(_DT[case["x"]])
    bias = None
    if case["bias"]:
        bias = _normal(g, V).mul_(0.5)
        bias[0] = -2.0                          # the blank's penalty
    return dict(x=x, bias=bias, lengths=_lengths(case, g), scale=1.0 if not case["bias"] else 0.9,
                out=torch.full((B, T, V), -7.0, dtype=_DT[case["out"]], device="cuda"))


def _sample_inputs(case, seed):
    g = _gen(seed)
    B, T, V = case["B"], case["T"], case["V"]
    if case["kind"] == "tokens":                # a language model's logits: a power law over a shuffled vocabulary
        rank = torch.randperm(V, generator=g, device="cuda").float() + 1.0
        x = _normal(g, B, T, V)
        x -= 1.5 * torch.log(rank)
        x += 12.0
    else:                                       # a CTC model's log-posteriors
        x = _normal(g, B, T, V).mul_(4.0)
        x[..., 0] += 5.0
        x -= torch.logsumexp(x, dim=-1, keepdim=True)
    x = x.to(_DT[case["x"]])
    u = torch.rand((B, T), generator=g, device="cuda", dtype=torch.float32)
    if case["params"] == "scalar":
        p = dict(temperature=case["temperature"], top_k=case["top_k"], top_p=case["top_p"], min_p=case["min_p"])
    else:
        def pick(values, dtype):
            i = torch.randint(0, len(values), (B, T), generator=g, device="cuda")
            return torch.tensor(values, dtype=dtype, device="cuda")[i]
        p = dict(temperature=pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.2], torch.float32),
                 top_k=pick([0, 0, 20, 50, 200], torch.int32),
                 top_p=pick([1.0, 0.8, 0.9, 0.95], torch.float32),
                 min_p=pick([0.0, 0.0, 0.05], torch.float32))
    out = (torch.full((B, T), -2, dtype=torch.int32, device="cuda"),
           torch.full((B, T), -7.0, dtype=torch.float32, device="cuda"),
           torch.full((B, T), -2, dtype=torch.int32, device="cuda"))
    return dict(x=x, u=u, params=p, lengths=_lengths(case, g), out=out)


_INPUTS = {"layer": _layer_inputs, "norm": _norm_inputs, "sample": _sample_inputs}


def prepare(case, seed):
    st = _INPUTS[case["op"]](case, seed)
    st["case"] = case
    if own:
        import wfst_beam_search_amd as wb
        st["wb"] = wb
        if case["op"] == "layer":
            st["layer"] = wb.OutputLayer(st["q"], st["scales"], zeros=st["zeros"], bias=st["bias"],
                                         in_features=case["K"], group_size=case["group"])
    return st


# ---- the plain forms

def _active(lengths, B, T):
    t = torch.arange(T, device="cuda")
    return (t[None, :] < lengths[:, None]) if lengths is not None else None


def _layer_plain(st):
    case = st["case"]
    K, N, G = case["K"], case["N"], case["group"]
    x = st["x"].float()
    y = torch.empty((case["M"], N), dtype=torch.float32, device="cuda")
    for n0 in range(0, N, 16384):
        n1 = min(N, n0 + 16384)
        q = st["q"][n0:n1]
        w = torch.stack((q & 15, q >> 4), dim=-1).reshape(n1 - n0, -1)[:, :K].float()
        s = st["scales"][n0:n1].float().repeat_interleave(G, dim=1)[:, :K]
        if st["zeros"] is None:
            w -= 8.0
        else:
            w -= st["zeros"][n0:n1].float().repeat_interleave(G, dim=1)[:, :K]
        w *= s
        y[:, n0:n1] = x @ w.t()
    if st["bias"] is not None:
        y += st["bias"]
    return y.to(_DT[case["out"]])


def _norm_plain(st):
    case = st["case"]
    z = st["x"].float() * st["scale"]
    if st["bias"] is not None:
        z = z + st["bias"]
    z = z - z.amax(dim=-1, keepdim=True)
    z = z - torch.log(torch.exp(z).sum(dim=-1, keepdim=True))
    z = z.to(_DT[case["out"]])
    act = _active(st["lengths"], case["B"], case["T"])
    return z if act is None else torch.where(act[..., None], z, st["out"])


def _rows(v, dtype, R):
    """A setting as one 64-bit value a row (a number is first rounded to the type it is passed in)."""
    if not torch.is_tensor(v):
        v = torch.tensor(v, dtype=dtype, device="cuda").expand(R)
    return v.reshape(R).double()


def _sample_plain(st):
    # in 64 bits: a draw next to a border has to fall on its right side
    case = st["case"]
    R, V = case["B"] * case["T"], case["V"]
    T = _rows(st["params"]["temperature"], torch.float32, R)
    k = _rows(st["params"]["top_k"], torch.int32, R)
    top_p = _rows(st["params"]["top_p"], torch.float32, R)
    min_p = _rows(st["params"]["min_p"], torch.float32, R)
    greedy = T <= 0
    k = torch.where(greedy, torch.ones_like(k), torch.where(k <= 0, torch.full_like(k, V), k))
    T = torch.where(greedy, torch.ones_like(T), T)
    xs, order = torch.sort(st["x"].reshape(R, V).double(), dim=-1, descending=True, stable=True)
    top = xs[:, :1].clone()
    mass = torch.exp((xs - top) / T[:, None])
    del xs
    keep = torch.arange(V, device="cuda")[None, :] < k[:, None]
    run = torch.cumsum(mass * keep, dim=-1)
    keep &= ((run - mass) < top_p[:, None] * run[:, -1:]) | (top_p >= 1.0)[:, None]
    keep[:, 0] = True
    del run
    keep &= mass >= min_p.clamp(max=1.0)[:, None]
    mass *= keep
    kept = keep.sum(dim=-1).int()
    w = torch.zeros_like(mass).scatter_(1, order, mass)      # back in the vocabulary's order
    run = torch.cumsum(w, dim=-1)
    total = run[:, -1].clone()
    want = st["u"].reshape(R).double() * total
    tok = ((run > want[:, None]) & (w > 0)).int().argmax(dim=-1)
    lp = (torch.log(w.gather(1, tok[:, None])[:, 0]) - torch.log(total)).float()
    out = (tok.int(), lp, kept)
    act = _active(st["lengths"], case["B"], case["T"])
    out = tuple(o.reshape(case["B"], case["T"]) for o in out)
    return out if act is None else tuple(torch.where(act, o, old) for o, old in zip(out, st["out"]))


def run(state):
    case = state["case"]
    if not own:
        return {"layer": _layer_plain, "norm": _norm_plain, "sample": _sample_plain}[case["op"]](state)
    wb = state["wb"]
    if case["op"] == "layer":
        return state["layer"].logits(state["x"], dtype=case["out"])
    if case["op"] == "norm":
        return wb.log_softmax(state["x"], dtype=case["out"], scale=state["scale"], bias=state["bias"],
                              lengths=state["lengths"], out=state["out"])
    r = wb.sample(state["x"], state["u"], lengths=state["lengths"], out=state["out"], **state["params"])
    return r.tokens, r.log_probs, r.kept


# ---- what a pass cannot do without

def work(case):
    if case["op"] == "layer":
        M, K, N = case["M"], case["K"], case["N"]
        ng = -(-K // case["group"])
        b = N * ((K + 1) // 2) + N * ng * (_SIZE[case["scale"]] + (1 if case["zeros"] else 0))
        b += (4 * N if case["bias"] else 0) + M * K * _SIZE[case["x"]] + M * N * _SIZE[case["out"]]
        return {"bytes": b, "flops": 2 * M * N * K}
    R, V = case["B"] * case["T"], case["V"]
    if case["ragged"]:
        R = R * 4 / 5                           # lengths from 3/5 T to T
    if case["op"] == "norm":
        return {"bytes": int(R * V * (_SIZE[case["x"]] + _SIZE[case["out"]]) + (4 * V if case["bias"] else 0)),
                "flops": int(5 * R * V)}
    return {"bytes": int(R * (V * _SIZE[case["x"]] + 4 + 12 + (16 if case["params"] == "rows" else 0))),
            "flops": int(4 * R * V)}


# ---- the definitions in 64 bits

def _layer_exact(case, seed):
    st = _layer_inputs(case, seed)
    K, N, G, M = case["K"], case["N"], case["group"], case["M"]
    x = st["x"].double()
    y = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    for g, k0 in enumerate(range(0, K, G)):     # group by group, the scale outside the sum
        k1 = min(K, k0 + G)
        kk = torch.arange(k0, k1, device="cuda")
        b = st["q"][:, k0 // 2:(k1 + 1) // 2].to(torch.int32)
        nib = (b[:, kk // 2 - k0 // 2] >> (4 * (kk % 2)).int()) & 15
        z = 8 if st["zeros"] is None else st["zeros"][:, g:g + 1].to(torch.int32)
        y += ((nib - z).double() @ x[:, k0:k1].t()).t() * st["scales"][:, g].double()
    if st["bias"] is not None:
        y += st["bias"].double()
    return y


def _norm_exact(case, seed):
    st = _norm_inputs(case, seed)
    z = st["x"].double() * st["scale"]
    if st["bias"] is not None:
        z += st["bias"].double()
    z -= torch.logsumexp(z, dim=-1, keepdim=True)
    if st["lengths"] is not None:
        late = torch.arange(case["T"], device="cuda")[None, :] >= st["lengths"][:, None]
        z[late] = -7.0
    return z


def _sample_exact(case, seed):
    st = _sample_inputs(case, seed)
    B, T, V = case["B"], case["T"], case["V"]
    R = B * T
    x = st["x"].reshape(R, V)
    u = st["u"].reshape(R).double()
    f32 = {n: (v.reshape(R).double() if torch.is_tensor(v) else
               torch.full((R,), float(np.float32(v)), dtype=torch.float64, device="cuda"))
           for n, v in st["params"].items()}
    tok = torch.empty(R, dtype=torch.int64, device="cuda")
    lp = torch.empty(R, dtype=torch.float64, device="cuda")
    kept = torch.empty(R, dtype=torch.int64, device="cuda")
    step = max(1, (1 << 24) // V)
    for r0 in range(0, R, step):                # masses in the vocabulary's order; the kept set from value limits
        r = slice(r0, min(R, r0 + step))
        xd = x[r].double()
        n = xd.shape[0]
        temp = f32["temperature"][r][:, None]
        hot = temp > 0
        e = (xd - xd.amax(-1, keepdim=True)) / torch.where(hot, temp, torch.ones_like(temp))
        m = e.exp()
        ms, ix = torch.sort(-xd, dim=-1, stable=True)
        rank = torch.empty_like(ix).scatter_(1, ix, torch.arange(V, device="cuda").expand(n, V))
        del ms
        k = f32["top_k"][r][:, None]
        lim = torch.where(k > 0, k, torch.full_like(k, V))
        lim = torch.where(hot, lim, torch.ones_like(lim))
        ok = rank < lim
        sorted_m = torch.where(ok, m, torch.zeros_like(m)).gather(1, ix)
        p = f32["top_p"][r][:, None]
        before = torch.cat((torch.zeros((n, 1), dtype=torch.float64, device="cuda"),
                            sorted_m.cumsum(-1)[:, :-1]), dim=1)
        need = p * sorted_m.sum(-1, keepdim=True)
        count = torch.where(p >= 1.0, torch.full_like(p, V), (before < need).sum(-1, keepdim=True).clamp(min=1).double())
        ok &= rank < count
        ok &= m >= f32["min_p"][r][:, None].clamp(max=1.0)
        w = torch.where(ok, m, torch.zeros_like(m))
        c = w.cumsum(-1)
        total = c[:, -1]
        t = (c <= (u[r] * total)[:, None]).sum(-1).clamp(max=V - 1)
        tok[r] = t
        kept[r] = ok.sum(-1)
        lp[r] = e.gather(1, t[:, None])[:, 0] - total.log()
    late = None
    if st["lengths"] is not None:
        late = (torch.arange(T, device="cuda")[None, :] >= st["lengths"][:, None]).reshape(R)
        tok[late], kept[late], lp[late] = -2, -2, -7.0
    return tuple(v.reshape(B, T) for v in (tok.int(), lp, kept.int()))


def exact(case, seed):
    return {"layer": _layer_exact, "norm": _norm_exact, "sample": _sample_exact}[case["op"]](case, seed)
