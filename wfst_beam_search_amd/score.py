"""Operators around the search: the output layer with 4-bit weights, the
log-softmax that makes ``log_prob`` of its logits, and the draw of tokens from
scores. Thin bindings like the rest of the package: the work runs in the HIP
library (``wfst_layer_*``, ``wfst_log_softmax``, ``wfst_sample`` of
``include/wfst.h``, which states the formulas); PyTorch supplies device memory
and streams. They are inference operators: no gradient passes through them, and a
tensor that needs one (backward, or a forward-mode dual) is refused.

Every call is asynchronous on ``stream`` (a ``torch.cuda.Stream`` or a raw
handle; default: the current stream of the operands' device; new tensors then
belong to that stream) and may be captured into a HIP graph when its ``lengths``
is a device tensor. Tensors may have any
leading dimensions whose rows lie a constant distance apart. ``lengths`` (int32
[B], for tensors [B, T, ...]; a device tensor, or host values that are copied
first) marks the rows t >= lengths[b] as empty: they are not read, and in ``out``
they stay as they were (in a new tensor they are unspecified).
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import numpy as np

from . import _check, load_library

DTYPES = {"f32": 0, "f16": 1, "bf16": 2}


class _LayerDesc(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("weights", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class _SampleConfig(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float),
                ("min_p", ctypes.c_float), ("temperatures", ctypes.c_void_p), ("top_ks", ctypes.c_void_p),
                ("top_ps", ctypes.c_void_p), ("min_ps", ctypes.c_void_p)]


_codes = None          # torch dtype -> element type code
_names = None          # "f32" ... -> torch dtype
_fw = None             # torch.autograd.forward_ad
_bump = None           # torch.autograd.graph.increment_version


def _types():
    global _codes, _names
    if _codes is None:
        import torch
        _names = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
        _codes = {_names[n]: c for n, c in DTYPES.items()}
    return _codes, _names


def _code(t, what):
    c = _types()[0].get(t.dtype)
    if c is None:
        raise TypeError(f"{what} must be a float32, float16 or bfloat16 tensor")
    return c


def _named(dtype):
    names = _types()[1]
    if dtype not in names:
        raise ValueError(f"dtype must be one of {sorted(names)}")
    return names[dtype]


_INT32_MAX = 2 ** 31 - 1


def _int32(v, what):
    """v as an int that the library's 32 bits hold (ctypes would cut off the bits above them)."""
    v = int(v)
    if not -_INT32_MAX <= v <= _INT32_MAX:
        raise ValueError(f"{what} ({v}) does not fit 32 bits")
    return v


def _gpu(t, what, device=None):
    global _fw
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a torch tensor on the GPU")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient, which these operators do not have (detach it, or use no_grad)")
    if _fw is None:
        _fw = torch.autograd.forward_ad
    if _fw._current_level >= 0 and torch._C._is_fwd_grad_enabled() and _fw.unpack_dual(t).tangent is not None:
        raise ValueError(f"{what} carries a forward-mode tangent, which these operators do not have (detach it)")
    if device is not None and t.device != device:
        raise ValueError(f"{what} must be on {device}")
    return t


def _rows(t, what):
    """(rows, distance between rows) of a tensor [..., n]."""
    if t.dim() == 0:
        raise ValueError(f"{what} must have at least one dimension")
    n = t.shape[-1]
    if n == 0:
        raise ValueError(f"{what} must have a last dimension of at least 1")
    rows = t.numel() // n
    if t.is_contiguous():
        return rows, n
    step = None                                 # the row distance, from the innermost dimension that has one
    expect = None
    if n > 1 and t.stride(-1) != 1:
        raise ValueError(f"the elements of a row of {what} must be adjacent")
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if step is None:
            step = stride
        elif stride != expect:
            raise ValueError(f"the rows of {what} must lie a constant distance apart")
        expect = stride * size
    return rows, n if step is None else step


def _stream(stream, device):
    """(raw handle, the stream when it is not the current one)."""
    import torch
    cur = torch._C._cuda_getCurrentRawStream(device.index)     # (current_stream() builds an object: 2 us)
    if stream is None:
        return cur, None
    raw = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if raw == cur:
        return raw, None
    other = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(raw, device=device)
    return raw, other


def _new(shape, dtype, device, other):
    """Memory for work on ``other`` (None: the current stream), from that stream's
    own pool: what it held before may still be in use on the current one."""
    import torch
    if other is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(other):
        return torch.empty(shape, dtype=dtype, device=device)


def _lengths(lengths, shape, device, other):
    """(device int32 tensor or None, T) for a batch of rows of the given leading shape."""
    if lengths is None:
        return None, 1
    import torch
    if len(shape) != 2:
        raise ValueError("lengths need a tensor [B, T, ...]")
    if isinstance(lengths, torch.Tensor) and lengths.is_cuda:
        if lengths.dtype != torch.int32 or not lengths.is_contiguous():
            raise TypeError("lengths on the GPU must be a packed int32 tensor")
        _gpu(lengths, "lengths", device)
    else:
        if isinstance(lengths, torch.Tensor):
            lengths = lengths.numpy()
        host = np.array(lengths).reshape(-1)
        if host.dtype != np.int32:              # (wider numbers to the nearest 32-bit one: none passes T)
            host = np.array([min(max(int(v), -1), _INT32_MAX) for v in host.tolist()], dtype=np.int32)
        lengths = torch.from_numpy(host).to(device)     # (the copy has ended when this returns)
        if other is not None:
            lengths.record_stream(other)
    if lengths.numel() != shape[0]:
        raise ValueError("lengths must have B entries")
    return lengths, _int32(shape[1], "T")


def _written(outs):
    """Tensors that the call overwrites: a backward pass that saved one says so instead of using it."""
    global _bump
    if _bump is None:
        import torch
        _bump = torch.autograd.graph.increment_version
    _bump(outs)


def _checked(out, shape, dtype, device):
    _gpu(out, "out", device)
    if out.dtype != dtype or out.shape != shape:
        raise ValueError(f"out must be a {dtype} tensor of shape {tuple(shape)}")
    return out


def _out(out, shape, dtype, device, other):
    if out is None:
        return _new(shape, dtype, device, other)
    _checked(out, shape, dtype, device)
    _written((out,))
    return out


def _workspace(nbytes, device, other):
    if nbytes <= 0:
        return None
    import torch
    return _new(nbytes, torch.uint8, device, other)


def _p(t):
    return None if t is None else t.data_ptr()


class OutputLayer:
    """A layer with 4-bit weights on one device: hidden states to logits.

    y = bias + sum over groups of scales * ((q - zeros) . x), with ``weights``
    uint8 [N, ceil(K / 2)] (feature 2i in the low half of byte i), ``scales``
    [N, ceil(K / group_size)] in float32, float16 or bfloat16, ``zeros`` uint8 of
    the same shape (None: 8) and ``bias`` float32 [N] (None: 0), all on the GPU.
    They are laid out anew in the layer's own memory (the call waits for that), so
    the arguments may be freed. ``group_size`` is a multiple of 32; ``in_features``
    (K) defaults to 2 * weights.shape[1].
    """

    def __init__(self, weights, scales, zeros=None, bias=None, in_features: int | None = None,
                 group_size: int = 128, stream=None):
        import torch
        self.handle = None
        lib = load_library()
        _gpu(weights, "weights")
        device = weights.device
        _gpu(scales, "scales", device)
        if weights.dtype != torch.uint8 or weights.dim() != 2 or not weights.is_contiguous():
            raise TypeError("weights must be a packed uint8 tensor [N, ceil(K / 2)]")
        N, half = _int32(weights.shape[0], "out_features"), int(weights.shape[1])
        K = _int32(2 * half if in_features is None else in_features, "in_features")
        group_size = _int32(group_size, "group_size")
        if (K + 1) // 2 != half:
            raise ValueError("weights must have ceil(in_features / 2) columns")
        if group_size < 1:
            raise ValueError("group_size must be positive")
        groups = -(-K // group_size)
        code = _code(scales, "scales")
        if tuple(scales.shape) != (N, groups) or not scales.is_contiguous():
            raise ValueError(f"scales must be a packed tensor [{N}, {groups}]")
        if zeros is not None:
            _gpu(zeros, "zeros", device)
            if zeros.dtype != torch.uint8 or tuple(zeros.shape) != (N, groups) or not zeros.is_contiguous():
                raise ValueError(f"zeros must be a packed uint8 tensor [{N}, {groups}]")
        if bias is not None:
            _gpu(bias, "bias", device)
            if bias.dtype != torch.float32 or tuple(bias.shape) != (N,) or not bias.is_contiguous():
                raise ValueError(f"bias must be a packed float32 tensor [{N}]")
        raw, _ = _stream(stream, device)
        desc = _LayerDesc(K, N, group_size, code, _p(weights), _p(scales), _p(zeros), _p(bias))
        h = ctypes.c_void_p()
        _check(lib.wfst_layer_create(ctypes.byref(desc), device.index, raw, ctypes.byref(h)))
        self.handle = h
        self._logits = lib.wfst_layer_logits
        self._bytes = {}                        # (element type, rows) -> workspace bytes
        self.device = device
        self.in_features, self.out_features = K, N

    def logits(self, hidden, dtype: str = "f32", lengths=None, out=None, stream=None):
        """Logits [..., N] of hidden states [..., K], in ``dtype`` ("f32", "f16", "bf16")."""
        if self.handle is None:
            raise ValueError("the layer was released")
        _gpu(hidden, "hidden", self.device)
        code = _code(hidden, "hidden")
        rows, step = _rows(hidden, "hidden")
        rows = _int32(rows, "rows")
        if hidden.shape[-1] != self.in_features:
            raise ValueError(f"hidden must be [..., {self.in_features}]")
        raw, other = _stream(stream, self.device)
        lead = hidden.shape[:-1]
        lengths, T = _lengths(lengths, lead, self.device, other)
        out = _out(out, (*lead, self.out_features), _named(dtype), self.device, other)
        _, ostep = _rows(out, "out")
        need = self._bytes.get((code, rows))
        if need is None:
            n = ctypes.c_int64(0)
            _check(load_library().wfst_layer_workspace(self.handle, code, rows, ctypes.byref(n)))
            if len(self._bytes) > 256:
                self._bytes.clear()
            need = self._bytes[code, rows] = n.value
        work = _workspace(need, self.device, other)
        _check(self._logits(self.handle, hidden.data_ptr(), code, step, rows, _p(lengths), T, out.data_ptr(),
                            DTYPES[dtype], ostep, _p(work), need, raw))
        return out

    def log_probs(self, hidden, dtype: str = "f32", scale: float = 1.0, bias=None, lengths=None, out=None,
                  stream=None):
        """log_softmax(scale * logits + bias) of hidden states, in ``dtype``: the
        search's ``log_prob`` for hidden states [B, T, K]. The logits in between are binary32."""
        _, other = _stream(stream, self.device)
        if lengths is not None:
            lengths, _ = _lengths(lengths, hidden.shape[:-1], self.device, other)
        direct = dtype == "f32"
        logits = self.logits(hidden, "f32", lengths=lengths, out=out if direct else None, stream=stream)
        return log_softmax(logits, dtype=dtype, scale=scale, bias=bias, lengths=lengths,
                           out=logits if direct else out, stream=stream)

    def release(self):
        if self.handle is not None:
            h, self.handle = self.handle, None
            load_library().wfst_layer_release(h)

    def __del__(self):
        try:
            self.release()
        except Exception:
            pass


@functools.lru_cache(maxsize=256)
def _norm_bytes(code, rows, V, ocode):
    need = ctypes.c_int64(0)
    _check(load_library().wfst_log_softmax_workspace(code, rows, V, ocode, ctypes.byref(need)))
    return need.value


def log_softmax(x, dtype: str | None = None, scale: float = 1.0, bias=None, lengths=None, out=None, stream=None):
    """log_softmax(scale * x + bias) over the last dimension of ``x``, in ``dtype``
    ("f32", "f16", "bf16"; default: x's own), ``bias`` float32 [V] or None. ``out``
    may be ``x`` itself. A row of -inf alone stays -inf; NaN or +inf make a row NaN."""
    import torch
    lib = load_library()
    _gpu(x, "x")
    device = x.device
    code = _code(x, "x")
    rows, step = _rows(x, "x")
    V = _int32(x.shape[-1], "V")
    want = x.dtype if dtype is None else _named(dtype)
    if bias is not None:
        _gpu(bias, "bias", device)
        if bias.dtype != torch.float32 or tuple(bias.shape) != (V,) or not bias.is_contiguous():
            raise ValueError(f"bias must be a packed float32 tensor [{V}]")
    raw, other = _stream(stream, device)
    lengths, T = _lengths(lengths, x.shape[:-1], device, other)
    out = _out(out, x.shape, want, device, other)
    _, ostep = _rows(out, "out")
    ocode = _types()[0][want]
    need = _norm_bytes(code, rows, V, ocode)
    work = _workspace(need, device, other)
    _check(lib.wfst_log_softmax(x.data_ptr(), code, step, rows, V, float(scale), _p(bias), _p(lengths), T,
                                out.data_ptr(), ocode, ostep, _p(work), need, raw))
    return out


class SampleResult(NamedTuple):
    tokens: object       # int32 [...]: the drawn label, -1 for an empty row
    log_probs: object    # float32 [...]: its log-probability among the kept labels
    kept: object         # int32 [...]: labels kept


def _setting(v, dtype, shape, device, name):
    """(number, None) or (0, device tensor with one value a row)."""
    import torch
    if not isinstance(v, torch.Tensor):
        return v, None
    _gpu(v, name, device)
    if v.dtype != dtype or tuple(v.shape) != tuple(shape) or not v.is_contiguous():
        raise ValueError(f"{name} must be a packed {dtype} tensor of shape {tuple(shape)}")
    return 0, v


@functools.lru_cache(maxsize=256)
def _sample_bytes(code, rows, V):
    need = ctypes.c_int64(0)
    _check(load_library().wfst_sample_workspace(code, rows, V, ctypes.byref(need)))
    return need.value


def sample(scores, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, lengths=None, out=None,
           stream=None) -> SampleResult:
    """Draw one token of each row of ``scores`` [..., V] (logits or
    log-probabilities) with the uniform random numbers ``u`` (float32 [...], in
    [0, 1)). The rules apply in this order, ties to the lowest index: temperature
    (0: the largest score), top_k largest (0, or V and more: all), the fewest of these whose mass
    reaches top_p of theirs, of these the ones with at least min_p of the largest
    one's mass. Each setting is a number or a tensor [...] on the GPU (float32;
    top_k int32). ``out``: tensors (tokens, log_probs, kept) to write to."""
    import torch
    lib = load_library()
    _gpu(scores, "scores")
    device = scores.device
    code = _code(scores, "scores")
    rows, step = _rows(scores, "scores")
    V = _int32(scores.shape[-1], "V")
    shape = scores.shape[:-1]
    _gpu(u, "u", device)
    if u.dtype != torch.float32 or u.shape != shape or not u.is_contiguous():
        raise ValueError(f"u must be a packed float32 tensor of shape {tuple(shape)}")
    t, ts = _setting(temperature, torch.float32, shape, device, "temperature")
    k, ks = _setting(top_k, torch.int32, shape, device, "top_k")
    p, ps = _setting(top_p, torch.float32, shape, device, "top_p")
    mp, mps = _setting(min_p, torch.float32, shape, device, "min_p")
    raw, other = _stream(stream, device)
    lengths, T = _lengths(lengths, shape, device, other)
    if out is None:
        buf = _new((3, *shape), torch.int32, device, other)
        res = SampleResult(buf[0], buf[1].view(torch.float32), buf[2])
    else:
        res = SampleResult(*out)
        for o, dt in zip(res, (torch.int32, torch.float32, torch.int32)):
            if o is None or not _checked(o, shape, dt, device).is_contiguous():
                raise ValueError("out must be three packed tensors (int32, float32, int32)")
        _written(res)
    k = max(-1, min(int(k), V))                 # (V and more: all)
    cfg = _SampleConfig(float(t), k, float(p), float(mp), _p(ts), _p(ks), _p(ps), _p(mps))
    need = _sample_bytes(code, rows, V)
    work = _workspace(need, device, other)
    _check(lib.wfst_sample(scores.data_ptr(), code, step, rows, V, u.data_ptr(), ctypes.byref(cfg), _p(lengths), T,
                           _p(res.tokens), _p(res.log_probs), _p(res.kept), _p(work), need, raw))
    return res
