"""vq_norm against the 64-bit oracle within derived bounds: types, gates,
row lengths from one value to the largest, and the e4m3 output."""
import itertools

import numpy as np
import pytest

from oracle import block_oracle as O
from tests.helpers import announce
from vq_dequant_matmul_gemv_amd import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # half a unit of fp32, relative


def _dt(name):
    import torch
    return getattr(torch, name)


def _tensors(T, C, key, block="bfloat16", residual="bfloat16", w="bfloat16", post=True, pre=True, gate=None):
    import torch
    g = synth.rng("norm", *key)

    def t(shape, dtype, scale=1.0, mean=0.0):
        return torch.from_numpy(mean + scale * g.normal(size=shape)).to(_dt(dtype))

    out = {"block": t((T, C), block, 0.3) if block else None, "residual": t((T, C), residual) if residual else None,
           "post_weight": t((C,), w, 0.1, 1.0) if post else None, "pre_weight": t((C,), w, 0.1, 1.0) if pre else None,
           "gate": None if gate is None else t({"channel": (C,), "token": (T, 1), "full": (T, C)}[gate], w)}
    if out["block"] is not None:
        out["block"][:, :: 61] *= 20
    return out


def _errors(ref, beta=1.0):
    """Bounds of v and h.  A sum of squares of 32 values a thread and 10 tree
    steps is off by 42 half units, its root's inverse by half of that; with
    the products, the gate's function and alpha the block term stays within 48
    half units, the residual term within 2, their sum within one more.  h adds
    the row's relative error of v's norm and 32 half units."""
    ev = 48 * U * np.abs(ref["u"]) + 2 * U * np.abs(ref["r"]) + U * np.abs(ref["v"])
    n = np.linalg.norm(ref["v"], axis=1, keepdims=True)
    rel = np.linalg.norm(ev, axis=1, keepdims=True) / np.where(n > 0, n, 1.0) + 32 * U
    return ev, np.abs(ref["w"] / ref["rms"]) * ev + rel * np.abs(ref["h"])


def _close(got, ref, err, dtype):
    import torch
    fi = torch.finfo(dtype)
    tol = err + (fi.eps / 2) * (np.abs(ref) + err) + float(fi.smallest_normal) * fi.eps
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4], tol[bad][:4])


def _check(t, h_dtype="bfloat16", in_place=False, **kw):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    first = t["block"] if t["block"] is not None else t["residual"]
    T, C = first.shape
    announce("norm", (T, C), {k: (tuple(v.shape), str(v.dtype)) for k, v in t.items() if v is not None}, h_dtype, kw)
    ref = O.norm(**{k: None if v is None else v.double().numpy() for k, v in t.items()}, **kw)
    ev, eh = _errors(ref)
    dev = {k: None if v is None else v.cuda() for k, v in t.items()}
    hd = _dt(h_dtype)
    vd = (t["residual"] if t["residual"] is not None else t["block"]).dtype
    vbuf = torch.full(((T + 1) * C,), 33.0, dtype=vd, device="cuda")
    hbuf = torch.full(((T + 1) * C,), 33.0, device="cuda").to(hd)
    vout = vbuf[:T * C].view(T, C)
    if in_place:
        vout.copy_(dev["residual"])
        dev["residual"] = vout
    v, h, s = binding.norm(**dev, h_dtype=hd, residual_out=vout, h=hbuf[:T * C].view(T, C), **kw)
    torch.cuda.synchronize()
    _close(v, ref["v"], ev, vd)
    assert torch.all(vbuf[T * C:] == 33.0).item() and torch.all(hbuf[T * C:].float() == 33.0 - (h_dtype == "float8_e4m3fn")
                                                                 ).item()
    if h_dtype != "float8_e4m3fn":
        assert s is None
        _close(h, ref["h"], eh, hd)
        return
    # e4m3: the scale follows the largest magnitude, every value is within half
    # a step (2^-4 relative, 2^-10 of the scale below the normal codes)
    amax = np.stack([np.abs(ref["h"][:, b * 128:(b + 1) * 128]).max(axis=1) for b in range(s.shape[1])], axis=1)
    ea = np.stack([eh[:, b * 128:(b + 1) * 128].max(axis=1) for b in range(s.shape[1])], axis=1)
    gs = s.double().cpu().numpy()
    assert np.all(np.abs(gs - np.where(amax > 0, amax / 448, 1)) <= ea / 448 + 2 * U * gs)
    sc = np.repeat(gs, 128, axis=1)[:, :C]
    val = h.float().double().cpu().numpy() * sc
    tol = eh + np.maximum(2.0 ** -4 * (np.abs(ref["h"]) + eh), 2.0 ** -10 * sc) * (1 + 2.0 ** -20)
    bad = ~(np.abs(val - ref["h"]) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], val[bad][:4], ref["h"][bad][:4])


@pytest.mark.parametrize("T,C", [(1, 1), (3, 7), (5, 8), (2, 64), (9, 120), (4, 511), (4, 512), (1, 513), (7, 520),
                                 (3, 2000), (2, 2048), (1, 2056), (5, 4095), (3, 5120), (2, 8192), (2, 8193),
                                 (1, 8200), (2, 17408), (1, 32768), (1, 32761), (600, 264)])
def test_row_lengths(T, C):
    _check(_tensors(T, C, ("len", T, C)))


@pytest.mark.parametrize("block,residual,w,h", list(itertools.product(
    ["float32", "float16", "bfloat16"], ["float32", "float16", "bfloat16"], ["bfloat16"],
    ["float32", "float16", "bfloat16"])) + [("float32", "float16", "float32", "float16"),
                                            ("bfloat16", "float32", "float16", "bfloat16")])
@pytest.mark.parametrize("C", [392, 333])
def test_types(block, residual, w, h, C):
    _check(_tensors(11, C, ("types", block, residual, C), block, residual, w, gate="channel"), h)


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("act", [None, "sigmoid", "tanh"])
@pytest.mark.parametrize("T,C", [(6, 1000), (6, 1001), (1, 6), (130, 96)])
def test_gates(gate, act, T, C):
    _check(_tensors(T, C, ("gate", gate, T, C), gate=gate), gate_act=act, alpha=0.5, beta=0.75, weight_offset=0.25,
           eps=1e-5)


@pytest.mark.parametrize("post,pre,residual", list(itertools.product([True, False], [True, False],
                                                                     ["float16", None])))
@pytest.mark.parametrize("C", [640, 641])
def test_parts(post, pre, residual, C):
    _check(_tensors(5, C, ("parts", post, pre, C), "float16", residual, "float16", post, pre), "float16", alpha=2.0)


@pytest.mark.parametrize("C", [512, 100])
def test_plain_norm_of_the_residual(C):
    _check(_tensors(9, C, ("plain", C), None, post=False), beta=0.5)


@pytest.mark.parametrize("T,C", [(1, 16), (3, 128), (2, 144), (9, 496), (5, 2000), (40, 5120), (2, 17408), (1, 32752)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_e4m3_output(T, C, dtype):
    _check(_tensors(T, C, ("e4m3", T, C), "float32", dtype, dtype, gate="token"), "float8_e4m3fn",
           gate_act="sigmoid")


def test_e4m3_output_of_zero_rows_and_bad_values():
    """A zero row gives zeros with scales of one; NaN and infinities spoil
    their own row alone."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    x = _tensors(6, 256, ("bad",), None, post=False)["residual"]
    x[1] = 0
    x[2, 5] = float("nan")
    x[4, 200] = float("inf")
    w = torch.ones(256, dtype=torch.bfloat16).cuda()
    v, h, s = binding.norm(None, x.cuda(), pre_weight=w, h_dtype=torch.float8_e4m3fn)
    torch.cuda.synchronize()
    assert torch.all(h[1].float() == 0).item() and torch.all(s[1] == 1.0).item()
    nan = h.float().isnan().any(dim=1).cpu().tolist()
    assert nan == [False, False, True, False, True, False]
    good, _, _ = binding.norm(None, x[[0, 3, 5]].cuda(), pre_weight=w)
    assert torch.equal(v[[0, 3, 5]], good)
    h0 = binding.norm(None, x[[0, 3, 5]].cuda(), pre_weight=w, h_dtype=torch.float8_e4m3fn)[1]
    assert torch.equal(h[[0, 3, 5]].view(torch.uint8), h0.view(torch.uint8))


@pytest.mark.parametrize("C", [1024, 1023])
def test_residual_in_place(C):
    _check(_tensors(33, C, ("place", C), gate="full"), in_place=True, gate_act="tanh")


@pytest.mark.parametrize("T,C", [(4, 5120), (77, 256)])
def test_same_bits_other_stream_and_captured(T, C):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    t = {k: None if v is None else v.cuda() for k, v in _tensors(T, C, ("again", T, C), gate="full").items()}
    ref = binding.norm(**t, gate_act="sigmoid")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = binding.norm(**t, gate_act="sigmoid", stream=st)
    st.synchronize()
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v, h, _ = binding.norm(**t, gate_act="sigmoid")
    for k in range(3):
        t["block"].copy_(_tensors(T, C, ("replay", k))["block"])
        graph.replay()
        torch.cuda.synchronize()
        rv, rh, _ = binding.norm(**t, gate_act="sigmoid")
        assert torch.equal(v, rv) and torch.equal(h, rh)


def test_only_one_output_and_empty_batch():
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    t = {k: None if v is None else v.cuda() for k, v in _tensors(3, 200, ("one",)).items()}
    v, h, _ = binding.norm(**t)
    pre = t.pop("pre_weight")
    assert torch.equal(binding.norm(**t)[0], v) and binding.norm(**t)[1] is None
    only = binding.norm(**t, pre_weight=pre, store_residual=False)
    assert only[0] is None and torch.equal(only[1], h)
    e = binding.norm(torch.zeros(0, 16, device="cuda"), h_dtype=torch.float8_e4m3fn)
    assert e[0].shape == (0, 16) and e[1].shape == (0, 16) and e[2].shape == (0, 1)


def test_e4m3_output_of_the_smallest_values():
    """Rows from fp32's smallest number to its smallest normal ones: the codes
    and scales of the unrounded h (as the fp32 output shows it), a scale of one
    where h / 448 rounds to nothing."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    g = synth.rng("norm", "smallest")
    x = g.normal(size=(96, 144)) * 10.0 ** np.linspace(-45.5, -36, 96)[:, None]
    x = torch.from_numpy(x.astype(np.float32)).cuda()
    x[:, ::5] = 0
    kw = dict(eps=1.0, store_residual=False)       # h = x but for its rounding
    h = binding.norm(None, x, h_dtype=torch.float32, **kw)[1].double().cpu().numpy()
    _, q, s = binding.norm(None, x, h_dtype=torch.float8_e4m3fn, **kw)
    rq, rs = O.fp8_quant(h)
    assert (rs == 1).any() and (rs < 1).any()
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), rq)
