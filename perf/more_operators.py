"""More operators between a model's last hidden state and its answer, as they are measured.

Two operators: the output layer with a low-rank adapter of each request beside its shared 4-bit weights, and the
scores of given tokens (log-probability and rank, the distribution's entropy, the best alternatives). A case is one
of them at one size; ``run`` computes it in plain torch operations, or (``own``) through the package's entry points.
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one frame of one stream with its speaker's adapter, the vocabulary of a mid-size graph: the smallest call
        dict(name="adapt_frame_500", op="adapt", B=1, T=1, K=512, N=500, group=64, x="f16", scale="f16", out="f32",
             zeros=False, bias=True, pad=0, slots=4, rank=8, mixed=False, a="f16", ragged=False),
        # one frame of each of 32 streams, each with an adapter of its own, a 5000-label model
        dict(name="adapt_lanes_5000", op="adapt", B=32, T=1, K=1024, N=5000, group=128, x="bf16", scale="bf16",
             out="f32", zeros=True, bias=True, pad=0, slots=32, rank=16, mixed=False, a="bf16", ragged=False),
        # one new token of one request, a large vocabulary: the shared weights' bytes
        dict(name="adapt_token_131072", op="adapt", B=1, T=1, K=4096, N=131072, group=128, x="bf16", scale="f16",
             out="f32", zeros=False, bias=False, pad=0, slots=8, rank=16, mixed=False, a="bf16", ragged=False),
        # a serving batch of 64 requests over 48 adapters of ranks up to 24, no size a multiple of a tile
        dict(name="adapt_batch_odd", op="adapt", B=64, T=1, K=2050, N=32003, group=32, x="f32", scale="f32", out="f16",
             zeros=True, bias=False, pad=14, slots=48, rank=24, mixed=True, a="f32", ragged=False),
        # an offline batch: 32 utterances of 300 to 500 frames, each with its speaker's adapter or none
        dict(name="adapt_utterances_5000", op="adapt", B=32, T=500, K=1024, N=5000, group=128, x="f16", scale="f16",
             out="f32", zeros=False, bias=True, pad=0, slots=24, rank=32, mixed=False, a="f16", ragged=True),
        # one frame of each of 8 streams: its label's confidence and the 5 best
        dict(name="score_frames_500", op="score", B=8, T=1, V=500, x="f32", kind="frames", C=1, top=5, temp="one",
             masked=False, ragged=False),
        # confidences of the alignments of an offline batch, the search's fp16 rows
        dict(name="score_utterances_5000", op="score", B=32, T=500, V=5000, x="f16", kind="frames", C=1, top=4,
             temp="one", masked=False, ragged=True),
        # the widest batch: many short rows, no alternatives
        dict(name="score_wide_500", op="score", B=64, T=1000, V=500, x="bf16", kind="frames", C=1, top=0, temp="one",
             masked=False, ragged=False),
        # the new token of one sequence with 20 alternatives: latency
        dict(name="score_token_131072", op="score", B=1, T=1, V=131072, x="f32", kind="tokens", C=1, top=20,
             temp="scalar", masked=False, ragged=False),
        # a serving batch over an odd vocabulary, a temperature for each sequence
        dict(name="score_batch_131071", op="score", B=256, T=1, V=131071, x="bf16", kind="tokens", C=1, top=20,
             temp="rows", masked=False, ragged=False),
        # 16 candidate labels of each of 48 sequences, a third of the labels not permitted
        dict(name="score_candidates_32003", op="score", B=48, T=1, V=32003, x="f32", kind="tokens", C=16, top=64,
             temp="one", masked=True, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        K = _log_int(rng, 200, 4096)
        N = _log_int(rng, 100, 131072)
        B = _log_int(rng, 1, 64)
        rank = _log_int(rng, 1, 64)
        frames = rng.random() < 0.4             # offline batches, else one row a request
        a = rng.choice(["f16", "bf16", "f32"])
        work = 32 * 500 * 5000 * 1024 // 4
        B = max(1, min(B, work // (N * K), int(5e8 // (N * rank))))
        T = max(1, min(_log_int(rng, 2, 500), work // (N * K * B))) if frames else 1
        slots = rng.randint(1, max(1, min(64, int(5e8 // ((N + K) * rank)))))
        return dict(op="adapt", B=B, T=T, K=K, N=N, group=rng.choice([32, 64, 128]), x=rng.choice(["f16", "bf16", "f32"]),
                    scale=rng.choice(["f16", "bf16", "f32"]), out=rng.choice(["f16", "bf16", "f32"]),
                    zeros=rng.random() < 0.5, bias=rng.random() < 0.5, pad=rng.choice([0, 0, 3, 8]), slots=slots,
                    rank=rank, mixed=rng.random() < 0.5, a=a, ragged=T > 1 and rng.random() < 0.5)
    V = _log_int(rng, 2, 131072)
    x = rng.choice(["f32", "f16", "bf16"])
    C = min(V, rng.choice([1, 1, 1, 4, 16]))
    top = min(V, rng.choice([0, 1, 5, 20, 64]))
    cap = 32 * 500 * 5000 * 2 // _SIZE[x]
    if C > 1 or top > 5:
        cap //= 8
    rows = _log_int(rng, 1, min(64000, cap // V))
    B = rng.randint(1, min(64, rows))
    T = max(1, rows // B)
    return dict(op="score", B=B, T=T, V=V, x=x, kind=rng.choice(["tokens", "frames"]), C=C, top=top,
                temp=rng.choice(["one", "scalar", "rows"]), masked=V >= 1000 and rng.random() < 0.3,
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


def _ranks(case):
    """The rank of each adapter: the same, or (mixed) another for each."""
    r = case["rank"]
    return [r - (5 * s) % r if case["mixed"] else r for s in range(case["slots"])]


def _adapt_inputs(case, seed):
    g = _gen(seed)
    B, T, K, N, S, R = case["B"], case["T"], case["K"], case["N"], case["slots"], case["rank"]
    ng = -(-K // case["group"])
    x = _normal(g, B, T, K + case["pad"]).to(_DT[case["x"]])[..., :K]
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
    ranks = _ranks(case)
    down = torch.zeros((S, R, K), dtype=_DT[case["a"]], device="cuda")
    up = torch.zeros((S, N, R), dtype=_DT[case["a"]], device="cuda")
    for s, r in enumerate(ranks):              # past an adapter's rank: zeros
        down[s, :r] = (_normal(g, r, K) / math.sqrt(K)).to(down.dtype)
        up[s, :, :r] = (_normal(g, N, r) * (0.3 / math.sqrt(r))).to(up.dtype)
    factor = [0.5 * (1 + s % 4) for s in range(S)]
    order = torch.randperm(B, generator=g, device="cuda")
    # each adapter in turn over the lanes; with more lanes than adapters, some lanes have none (-1)
    ids = ((order + 1) % (S + 1) - 1).to(torch.int32)
    return dict(x=x, q=q, scales=scales, zeros=zeros, bias=bias, down=down, up=up, ranks=ranks, factor=factor, ids=ids,
                lengths=_lengths(case, g), out=torch.full((B, T, N), -7.0, dtype=_DT[case["out"]], device="cuda"))


def _score_inputs(case, seed):
    g = _gen(seed)
    B, T, V, C = case["B"], case["T"], case["V"], case["C"]
    x = _normal(g, B, T, V)
    if case["kind"] == "tokens":                # a language model's logits: a power law over a shuffled vocabulary
        rank = torch.randperm(V, generator=g, device="cuda").float() + 1.0
        x -= 1.5 * torch.log(rank)
        x += 12.0
    else:                                       # a CTC model's log-posteriors
        x *= 4.0
        x[..., 0] += 5.0
        x -= torch.logsumexp(x, dim=-1, keepdim=True)
    if case["masked"]:                          # labels that may not be emitted
        x[..., torch.randperm(V, generator=g, device="cuda")[:V // 3]] = -math.inf
    x = x.to(_DT[case["x"]])
    # the tokens to score: drawn from the distribution, without repetition
    u = torch.rand((B, T, V), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-6).log_().neg_().log_().neg_()
    u += x
    tokens = torch.topk(u, C, dim=-1).indices.to(torch.int32)
    del u
    tokens = tokens[..., 0].contiguous() if C == 1 else tokens.contiguous()
    if case["temp"] == "rows":
        i = torch.randint(0, 5, (B, T), generator=g, device="cuda")
        temp = torch.tensor([0.5, 0.7, 1.0, 1.0, 1.3], dtype=torch.float32, device="cuda")[i]
    else:
        temp = 1.0 if case["temp"] == "one" else 0.7
    n = case["top"]
    out = [torch.full(tokens.shape, -7.0, device="cuda"), torch.full(tokens.shape, -2, dtype=torch.int32, device="cuda"),
           torch.full((B, T), -7.0, device="cuda")]
    if n:
        out += [torch.full((B, T, n), -2, dtype=torch.int32, device="cuda"), torch.full((B, T, n), -7.0, device="cuda")]
    return dict(x=x, tokens=tokens, temp=temp, lengths=_lengths(case, g), out=tuple(out))


_INPUTS = {"adapt": _adapt_inputs, "score": _score_inputs}


def prepare(case, seed):
    st = _INPUTS[case["op"]](case, seed)
    st["case"] = case
    if own:
        import wfst_beam_search_amd as wb
        st["wb"] = wb
        if case["op"] == "adapt":
            st["layer"] = wb.OutputLayer(st["q"], st["scales"], zeros=st["zeros"], bias=st["bias"],
                                         in_features=case["K"], group_size=case["group"])
            st["adapters"] = wb.Adapters(st["layer"], case["slots"], case["rank"], dtype=case["a"])
            for s, r in enumerate(st["ranks"]):
                st["adapters"].load(s, st["down"][s, :r], st["up"][s, :, :r], scale=st["factor"][s])
    return st


# ---- the plain forms

def _active(lengths, B, T):
    t = torch.arange(T, device="cuda")
    return (t[None, :] < lengths[:, None]) if lengths is not None else None


def _adapt_plain(st):
    case = st["case"]
    B, T, K, N, G = case["B"], case["T"], case["K"], case["N"], case["group"]
    x = st["x"].float().contiguous()
    y = torch.empty((B * T, N), dtype=torch.float32, device="cuda")
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
        y[:, n0:n1] = x.reshape(B * T, K) @ w.t()
    if st["bias"] is not None:
        y += st["bias"]
    # a lane's adapter as its own two matrices, a batched product each
    some = st["ids"] >= 0
    slot = st["ids"].clamp(min=0).long()
    factor = torch.tensor(st["factor"], dtype=torch.float32, device="cuda")[slot] * some
    h = torch.bmm(x, st["down"][slot].float().transpose(1, 2).contiguous()) * factor[:, None, None]
    y = y.reshape(B, T, N) + torch.bmm(h, st["up"][slot].float().transpose(1, 2).contiguous())
    y = y.to(_DT[case["out"]])
    act = _active(st["lengths"], B, T)
    return y if act is None else torch.where(act[..., None], y, st["out"])


def _score_plain(st):
    case = st["case"]
    B, T, V, n = case["B"], case["T"], case["V"], case["top"]
    x = st["x"].float()
    tok = st["tokens"].reshape(B, T, -1).long()
    temp = st["temp"][..., None] if torch.is_tensor(st["temp"]) else st["temp"]
    top = x.amax(dim=-1, keepdim=True)
    d = (x - top) / temp
    e = torch.exp(d)
    total = e.sum(dim=-1, keepdim=True)
    lz = torch.log(total)
    ent = (lz - (torch.where(e > 0, d, torch.zeros_like(d)) * e).sum(dim=-1, keepdim=True) / total)[..., 0]
    lp = d.gather(-1, tok) - lz
    xt = x.gather(-1, tok)
    v = torch.arange(V, device="cuda")
    rank = torch.stack([((x > xt[..., c:c + 1]) | ((x == xt[..., c:c + 1]) & (v < tok[..., c:c + 1]))).sum(dim=-1)
                        for c in range(tok.shape[-1])], dim=-1)
    out = [lp.reshape(st["tokens"].shape), rank.int().reshape(st["tokens"].shape), ent]
    if n:
        order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :n]
        out += [order.int(), d.gather(-1, order) - lz]
    act = _active(st["lengths"], B, T)
    if act is None:
        return tuple(out)
    return tuple(torch.where(act if o.dim() == 2 else act[..., None], o, old) for o, old in zip(out, st["out"]))


def run(state):
    case = state["case"]
    if not own:
        return {"adapt": _adapt_plain, "score": _score_plain}[case["op"]](state)
    if case["op"] == "adapt":
        return state["layer"].logits(state["x"], dtype=case["out"], lengths=state["lengths"], out=state["out"],
                                     adapters=state["adapters"], ids=state["ids"])
    r = state["wb"].token_scores(state["x"], state["tokens"], top_n=case["top"], temperature=state["temp"],
                                 lengths=state["lengths"], out=state["out"])
    return tuple(v for v in r if v is not None)


# ---- what a pass cannot do without

def work(case):
    if case["op"] == "adapt":
        B, K, N = case["B"], case["K"], case["N"]
        M = B * case["T"] * (4 / 5 if case["ragged"] else 1)    # lengths from 3/5 T to T
        ng = -(-K // case["group"])
        ranks = _ranks(case)[:min(B, case["slots"])]            # the adapters in use
        b = N * ((K + 1) // 2) + N * ng * (_SIZE[case["scale"]] + (1 if case["zeros"] else 0))
        b += (4 * N if case["bias"] else 0) + M * K * _SIZE[case["x"]] + M * N * _SIZE[case["out"]]
        b += sum(ranks) * (K + N) * _SIZE[case["a"]] + 4 * B
        mean = sum(ranks) / len(ranks)
        return {"bytes": int(b), "flops": int(2 * M * N * K + 2 * M * mean * (K + N))}
    R, V = case["B"] * case["T"], case["V"]
    if case["ragged"]:
        R = R * 4 / 5
    row = V * _SIZE[case["x"]] + 12 * case["C"] + 4 + 8 * case["top"] + (4 if case["temp"] == "rows" else 0)
    return {"bytes": int(R * row), "flops": int((6 + case["C"]) * R * V)}


# ---- the definitions in 64 bits

def _adapt_exact(case, seed):
    st = _adapt_inputs(case, seed)
    B, T, K, N, G = case["B"], case["T"], case["K"], case["N"], case["group"]
    x = st["x"].double()
    flat = x.reshape(B * T, K)
    y = torch.zeros((B * T, N), dtype=torch.float64, device="cuda")
    for g, k0 in enumerate(range(0, K, G)):     # group by group, the scale outside the sum
        kk = torch.arange(k0, min(K, k0 + G), device="cuda")
        b = st["q"][:, k0 // 2:(int(kk[-1]) + 2) // 2].to(torch.int32)
        nib = (b[:, kk // 2 - k0 // 2] >> (4 * (kk % 2)).int()) & 15
        z = 8 if st["zeros"] is None else st["zeros"][:, g:g + 1].to(torch.int32)
        w = ((nib - z).double() * st["scales"][:, g:g + 1].double()).t().contiguous()
        y.addmm_(flat[:, k0:k0 + kk.numel()], w)
    if st["bias"] is not None:
        y += st["bias"].double()
    y = y.reshape(B, T, N)
    for b, s in enumerate(st["ids"].tolist()):  # lane by lane, over the adapter's own rank
        if s >= 0:
            r = st["ranks"][s]
            h = x[b] @ st["down"][s, :r].double().t()
            y[b] += st["factor"][s] * (h @ st["up"][s, :, :r].double().t())
    if st["lengths"] is not None:
        for b, n in enumerate(st["lengths"].tolist()):
            y[b, n:] = -7.0
    return y


def _score_exact(case, seed):
    st = _score_inputs(case, seed)
    B, T, V, n = case["B"], case["T"], case["V"], case["top"]
    R, C = B * T, case["C"]
    x = st["x"].reshape(R, V)
    tok = st["tokens"].reshape(R, C).long()
    temp = st["temp"].reshape(R) if torch.is_tensor(st["temp"]) else torch.full((R,), st["temp"], device="cuda")
    temp = temp.float().double()
    lp = torch.empty((R, C), dtype=torch.float64, device="cuda")
    rank = torch.empty((R, C), dtype=torch.int32, device="cuda")
    ent = torch.empty(R, dtype=torch.float64, device="cuda")
    top = torch.empty((R, n), dtype=torch.int32, device="cuda")
    top_lp = torch.empty((R, n), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 24) // V)
    for r0 in range(0, R, step):
        r = slice(r0, min(R, r0 + step))
        xd = x[r].double()
        m, at = xd.max(dim=-1, keepdim=True)
        z = (xd - m) / temp[r][:, None]
        p = z.exp()
        rest = p.scatter(1, at, 0.0).sum(dim=-1, keepdim=True)      # the largest apart: exactly 1
        lz = torch.log1p(rest)
        ent[r] = (lz + (-z * p).nan_to_num_(nan=0.0).sum(dim=-1, keepdim=True) / (1.0 + rest))[:, 0]
        lp[r] = z.gather(1, tok[r]) - lz
        order = torch.sort(-xd, dim=-1, stable=True).indices
        place = torch.empty_like(order).scatter_(1, order, torch.arange(V, device="cuda").expand(order.shape))
        rank[r] = place.gather(1, tok[r]).int()
        top[r] = order[:, :n].int()
        top_lp[r] = z.gather(1, order[:, :n]) - lz
    out = [lp.reshape(st["tokens"].shape), rank.reshape(st["tokens"].shape), ent.reshape(B, T)]
    if n:
        out += [top.reshape(B, T, n), top_lp.reshape(B, T, n)]
    if st["lengths"] is not None:
        late = torch.arange(T, device="cuda")[None, :] >= st["lengths"][:, None]
        for o in out:
            o[late] = -7.0 if o.is_floating_point() else -2
    return tuple(out)


def exact(case, seed):
    return {"adapt": _adapt_exact, "score": _score_exact}[case["op"]](case, seed)
