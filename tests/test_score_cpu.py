"""Refusals of the operators around the search that need no GPU (arguments are
checked on the host before any device call), their C structs, and the 64-bit
definitions the GPU tests compare with, on cases worked out by hand."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import score_ref as ref
import wfst_beam_search_amd as wb
from wfst_beam_search_amd import score

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL = -1


@pytest.fixture(scope="module")
def lib():
    return wb.load_library()


@pytest.mark.parametrize("name,cls", [("wfst_layer_desc", score._LayerDesc),
                                      ("wfst_sample_config", score._SampleConfig)])
def test_structs_match_header(name, cls):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "wfst.h")).read(), flags=re.S)
    body = re.search(r"typedef struct " + name + r"\s*\{(.*?)\}\s*" + name + ";", src, flags=re.S).group(1)
    fields = re.findall(r"([A-Za-z_][A-Za-z0-9_ ]*?[\s*]+)([a-z_]+)\s*;", body)
    assert [f for _, f in fields] == [f for f, _ in cls._fields_]
    kinds = {"float": ctypes.c_float, "int32_t": ctypes.c_int32}
    for (ctype, fname), (_, ptype) in zip(fields, cls._fields_):
        assert (ctypes.c_void_p if "*" in ctype else kinds[ctype.strip()]) is ptype, fname


def _layer_rc(lib, fake=4096, **kw):
    d = dict(in_features=64, out_features=8, group_size=32, scale_dtype=0, weights=fake, scales=fake, zeros=None,
             bias=None)
    d.update(kw)
    h = ctypes.c_void_p()
    desc = score._LayerDesc(*(d[n] for n, _ in score._LayerDesc._fields_))
    rc = lib.wfst_layer_create(ctypes.byref(desc), kw.get("device", 0), None, ctypes.byref(h))
    return rc, lib.wfst_last_error().decode()


@pytest.mark.parametrize("bad,word", [
    (dict(in_features=0), "in_features"), (dict(in_features=-5), "in_features"),
    (dict(in_features=(1 << 24) + 1), "in_features"), (dict(out_features=0), "out_features"),
    (dict(group_size=0), "group_size"), (dict(group_size=16), "group_size"), (dict(group_size=48), "group_size"),
    (dict(scale_dtype=3), "scale_dtype"), (dict(weights=None), "null"), (dict(scales=None), "null")])
def test_layer_create_refuses(lib, bad, word):
    bad = {k: v for k, v in bad.items()}
    rc, msg = _layer_rc(lib, **bad)
    assert rc == EINVAL and word in msg


def test_layer_calls_refuse_null(lib):
    assert lib.wfst_layer_create(None, 0, None, ctypes.byref(ctypes.c_void_p())) == EINVAL
    assert lib.wfst_layer_logits(None, 4096, 0, 8, 1, None, 1, 4096, 0, 8, None, 0, None) == EINVAL
    assert lib.wfst_layer_workspace(None, 0, 1, ctypes.byref(ctypes.c_int64())) == EINVAL
    assert lib.wfst_layer_release(None) == 0


@pytest.mark.parametrize("kw,word", [
    (dict(xt=3), "type"), (dict(ot=-1), "type"), (dict(rows=-1), "rows"), (dict(V=0), "V"),
    (dict(V=(1 << 24) + 1), "V"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(x=None), "null"), (dict(out=None), "null"), (dict(xs=7), "stride"), (dict(os=7), "stride"),
    (dict(xs=1 << 61), "large")])
def test_log_softmax_refuses(lib, kw, word):
    a = dict(x=4096, xt=0, xs=8, rows=2, V=8, scale=1.0, out=8192, ot=0, os=8)
    a.update(kw)
    rc = lib.wfst_log_softmax(a["x"], a["xt"], a["xs"], a["rows"], a["V"], a["scale"], None, None, 1, a["out"],
                              a["ot"], a["os"], None, 0, None)
    assert rc == EINVAL and word in lib.wfst_last_error().decode()


@pytest.mark.parametrize("kw,word", [
    (dict(xt=9), "type"), (dict(rows=-1), "rows"), (dict(V=0), "V"), (dict(T=-0.5), "temperature"),
    (dict(T=float("nan")), "temperature"), (dict(T=float("inf")), "temperature"), (dict(k=-1), "top_k"),
    (dict(p=1.5), "top_p"), (dict(p=-0.1), "top_p"), (dict(p=float("nan")), "top_p"), (dict(mp=1.01), "min_p"),
    (dict(mp=float("nan")), "min_p"), (dict(x=None), "null"), (dict(u=None), "null"), (dict(tok=None), "null"),
    (dict(xs=7), "stride")])
def test_sample_refuses(lib, kw, word):
    a = dict(x=4096, xt=0, xs=8, rows=2, V=8, u=8192, T=1.0, k=0, p=1.0, mp=0.0, tok=16384)
    a.update(kw)
    cfg = score._SampleConfig(a["T"], a["k"], a["p"], a["mp"], None, None, None, None)
    rc = lib.wfst_sample(a["x"], a["xt"], a["xs"], a["rows"], a["V"], a["u"], ctypes.byref(cfg), None, 1, a["tok"],
                         None, None, None, 0, None)
    assert rc == EINVAL and word in lib.wfst_last_error().decode()


def test_no_rows_is_no_work(lib):
    cfg = score._SampleConfig(1.0, 0, 1.0, 0.0, None, None, None, None)
    assert lib.wfst_sample(None, 0, 8, 0, 8, None, ctypes.byref(cfg), None, 1, None, None, None, None, 0,
                           None) == 0
    assert lib.wfst_log_softmax(None, 0, 8, 0, 8, 1.0, None, None, 1, None, 0, 8, None, 0, None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(TypeError, match="GPU"):
        wb.log_softmax(x)
    with pytest.raises(TypeError, match="GPU"):
        wb.sample(x, torch.zeros(2))
    with pytest.raises(TypeError, match="GPU"):
        wb.OutputLayer(torch.zeros(4, 16, dtype=torch.uint8), torch.ones(4, 1))


def test_row_geometry():
    t = torch.zeros(4, 6, 10)
    assert score._rows(t, "t") == (24, 10)
    assert score._rows(t[:, :, :7], "t") == (24, 10)
    assert score._rows(t[:1, 1:4], "t") == (3, 10)
    assert score._rows(t[2], "t") == (6, 10)
    assert score._rows(t[0, 0], "t") == (1, 10)
    assert score._rows(t[:, :0], "t")[0] == 0
    with pytest.raises(ValueError, match="distance"):
        score._rows(t[:, 1:4], "t")
    with pytest.raises(ValueError, match="adjacent"):
        score._rows(t.transpose(1, 2), "t")
    with pytest.raises(ValueError, match="last dimension"):
        score._rows(t[:, :, :0], "t")


def test_reference_layer_by_hand():
    # K = 3: q = 1, 15, 9; scale 2; zeros 8: weights -14, 14, 2
    w = np.array([[1 | 15 << 4, 9 | 7 << 4]], np.uint8)
    y, size = ref.layer(np.array([[1.0, 2.0, -0.5]]), w, np.array([[2.0]]), None, np.array([0.25]), 3, 32)
    assert y[0, 0] == -14 + 28 - 1 + 0.25 and size[0, 0] == 14 + 28 + 1 + 0.25


def test_reference_sample_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 4.0, 1.0]))          # masses 1/4, 1, 1/2, 1, 1/4: 3 in all
    assert ref.sample_row(x, 0.0)[0] == 0
    assert ref.sample_row(x, 0.25 / 3 + 1e-6)[0] == 1
    assert ref.sample_row(x, 0.999999)[0] == 4
    assert ref.sample_row(x, 0.999999, T=0.0) == (1, 0.0, 1)
    assert ref.sample_row(x, 0.99, top_k=1)[:1] == (1,)      # the tie goes to the lowest index
    assert ref.sample_row(x, 0.99, top_k=3) [0::2] == (3, 3)
    assert ref.sample_row(x, 0.99, top_p=0.5)[0::2] == (3, 2)
    assert ref.sample_row(x, 0.99, min_p=0.4)[0::2] == (3, 3)
    assert ref.sample_row(np.full(3, -np.inf), 0.5) == (-1, -np.inf, 0)
    assert ref.sample_row(np.array([np.nan, 1.0, np.inf, np.inf]), 0.6)[0::2] == (3, 2)


# ---- integers past 32 bits (meta tensors have such shapes without memory)

@pytest.fixture
def no_gpu_checks(monkeypatch):
    """The binding up to the library call, on tensors without memory."""
    monkeypatch.setattr(score, "_gpu", lambda t, what, device=None: t)
    monkeypatch.setattr(score, "_stream", lambda stream, device: (0, None))


def _meta(*shape, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device="meta")


class _Recorder:
    """The library, but for the calls that would reach a device."""

    def __init__(self, lib):
        self.lib = lib
        self.top_k = []

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def wfst_sample(self, *args):
        self.top_k.append(args[6]._obj.top_k)
        return 0


@pytest.mark.parametrize("given,passed", [
    (0, 0), (1, 1), (7, 7), (999, 999), (1000, 1000), (1001, 1000), (2 ** 31, 1000), (2 ** 32 + 1, 1000),
    (2 ** 63 - 1, 1000), (10 ** 30, 1000), (-1, -1), (-2 ** 31, -1), (-2 ** 32 + 5, -1)])
def test_top_k_keeps_its_meaning_past_32_bits(lib, monkeypatch, no_gpu_checks, given, passed):
    fake = _Recorder(lib)
    monkeypatch.setattr(score, "load_library", lambda: fake)
    wb.sample(_meta(2, 1000), _meta(2, dtype=torch.float32), top_k=given)
    assert fake.top_k == [passed]


def test_sizes_past_32_bits_are_refused(lib, no_gpu_checks):
    wide, tall = _meta(1, 2 ** 32 + 5), _meta(2 ** 32 + 2, 1, 8)
    with pytest.raises(ValueError, match="V .* 32 bits"):
        wb.log_softmax(wide)
    with pytest.raises(ValueError, match="V .* 32 bits"):
        wb.sample(wide, _meta(1, dtype=torch.float32))
    with pytest.raises(ValueError, match="T .* 32 bits"):
        wb.log_softmax(_meta(2, 2 ** 32 + 4, 8), lengths=[1, 1])
    w, s = _meta(4, 32, dtype=torch.uint8), _meta(4, 1)
    with pytest.raises(ValueError, match="group_size .* 32 bits"):
        wb.OutputLayer(w, s, group_size=2 ** 32 + 32)
    with pytest.raises(ValueError, match="in_features .* 32 bits"):
        wb.OutputLayer(_meta(4, 2 ** 31 + 32, dtype=torch.uint8), s, group_size=2 ** 32)
    with pytest.raises(ValueError, match="out_features .* 32 bits"):
        wb.OutputLayer(_meta(2 ** 32 + 4, 32, dtype=torch.uint8), _meta(2 ** 32 + 4, 1), group_size=64)
    layer = object.__new__(wb.OutputLayer)
    layer.handle, layer.device, layer.in_features, layer.out_features, layer._bytes = 1, tall.device, 8, 4, {}
    try:
        with pytest.raises(ValueError, match="rows .* 32 bits"):
            layer.logits(tall)
    finally:
        layer.handle = None


@pytest.mark.parametrize("given", [[2 ** 32 + 5, -2 ** 32 + 5, 3], np.array([2 ** 32 + 5, -2 ** 32 + 5, 3]),
                                   torch.tensor([2 ** 32 + 5, -2 ** 32 + 5, 3])])
def test_host_lengths_past_32_bits(given):
    got, T = score._lengths(given, (3, 7), torch.device("cpu"), None)
    assert T == 7 and got.dtype == torch.int32 and got.tolist() == [2 ** 31 - 1, -1, 3]


def test_host_lengths_of_other_types():
    for given in ([3, 0, 7], np.array([3, 0, 7], np.uint8), torch.tensor([3, 0, 7], dtype=torch.int16), (3.0, 0.0, 7.0)):
        assert score._lengths(given, (3, 7), torch.device("cpu"), None)[0].tolist() == [3, 0, 7]
    assert score._lengths([], (0, 7), torch.device("cpu"), None)[0].numel() == 0
    with pytest.raises((ValueError, OverflowError)):
        score._lengths([float("nan"), 1, 2], (3, 7), torch.device("cpu"), None)


def test_hidden_lengths_are_checked_as_given():
    class Layer:
        out_features = 5

    dec = object.__new__(wb.Decoder)
    dec.handle, dec.graph = None, type("G", (), {"vocab": 5})
    for bad in (np.array([2 ** 32 + 1, 0]), [-2 ** 32 + 1, 0], [8, 0]):
        with pytest.raises(ValueError, match="lengths"):
            dec._log_probs(Layer, torch.zeros(2, 7, 3), bad, 1.0, None, None)


def test_build_jobs_from_any_environment(monkeypatch):
    from wfst_beam_search_amd import build as hip_build
    for given, jobs in (("", 4), ("auto", 4), ("0", 1), ("2", 2), ("16", 4), (" 3 ", 3), ("-1", 4)):
        monkeypatch.setenv("MAX_JOBS", given)
        assert hip_build._jobs() == jobs
    monkeypatch.delenv("MAX_JOBS")
    assert hip_build._jobs() == 4


def test_writing_to_out_is_known_to_autograd(no_gpu_checks):
    """out may share its memory with a tensor that a backward pass has saved."""
    x = torch.randn(2, 3, requires_grad=True)
    y = x.exp()                                     # saved for its own gradient
    out = score._out(y.detach(), (2, 3), torch.float32, x.device, None)
    assert out._version == 1
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
    with torch.inference_mode():
        assert score._out(torch.zeros(2, 3), (2, 3), torch.float32, x.device, None).shape == (2, 3)
