"""Host checks of the 4-bit operators without a GPU (every refused call returns
before anything is enqueued), and pins of their oracle."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def b():
    from vq_dequant_matmul_gemv_amd import binding
    return binding


def _status(b, st):
    return b.STATUS_NAMES[st]


# ---- oracle ---------------------------------------------------------------

def test_oracle_values_and_quantizer_by_hand():
    from oracle import block_oracle as O
    assert O.E2M1.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert O.e2m1_nearest([0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.9, -0.25, -5.0]).tolist() == \
        [0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 8, 14]
    x = np.zeros((1, 96))
    x[0, :3] = [7.9, -1.0, 0.25]          # scale 1
    x[0, 32:34] = [2.0 ** -140, 2.0 ** -128]   # below the smallest scale's steps
    x[0, 64] = np.inf
    q, s = O.mx4_quant(x)
    assert s.tolist() == [[127, 0, 255]]
    v = O.mx4_values(q, s)
    assert v[0, :3].tolist() == [6.0, -1.0, 0.0] and v[0, 32:34].tolist() == [0.0, 2.0 ** -128]
    assert np.isnan(v[0, 64:]).all() and q[0, 32:].tolist() == [0] * 16
    assert O.mx4_quant(np.zeros((1, 32)))[1].tolist() == [[127]]
    assert O.mx4_pack(np.array([[1, 2, 3, 15]])).tolist() == [[0x21, 0xf3]]


def test_oracle_layer_by_hand():
    from oracle import block_oracle as O
    gu = np.array([[[1.0], [2.0]], [[0.0], [1.0]]])             # two experts, inter 1, hidden 1
    dn = np.array([[[3.0]], [[5.0]]])
    y, g, m, h = O.mx4_moe(np.array([[0, -1], [1, 0]]), np.array([[0.5, 9.0], [1.0, 2.0]]), np.array([[2.0], [-1.0]]),
                           gu, dn)
    silu = lambda v: v / (1 + np.exp(-v))  # noqa: E731
    assert np.allclose(y, [[0.5 * 3 * silu(2.0) * 4.0], [2 * 3 * silu(-1.0) * -2.0]])
    assert h[1, 0, 0] == 0 and m[0, 0].tolist() == [2.0, 4.0] and g[1, 1].tolist() == [-1.0, -2.0]


# ---- quantizer and reader -------------------------------------------------

@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), "VQ_ERR_SHAPE"),
    (dict(dt=4), "VQ_ERR_SHAPE"),
    (dict(dt=-1), "VQ_ERR_SHAPE"),
    (dict(cols=0), "VQ_ERR_SHAPE"),
    (dict(cols=48), "VQ_ERR_SHAPE"),
    (dict(cols=(1 << 20) + 32), "VQ_ERR_SHAPE"),
    (dict(T=-1), "VQ_ERR_SHAPE"),
    (dict(T=(1 << 14) + 1, cols=1 << 20), "VQ_ERR_SHAPE"),
    (dict(x=0), "VQ_ERR_NULL"),
    (dict(q=0), "VQ_ERR_NULL"),
    (dict(s=0), "VQ_ERR_NULL"),
    (dict(x=0x10008), "VQ_ERR_ALIGN"),
    (dict(q=0x20008), "VQ_ERR_ALIGN"),
    (dict(T=0, x=0, q=0, s=0), "VQ_OK"),
])
def test_quant_and_dequant_refuse(b, kw, status):
    a = dict(x=0x10000, dt=0, T=3, cols=64, q=0x20000, s=0x30001)
    a.update(kw)
    assert _status(b, b.LIB.vq_mx4_quant(a["x"], a["dt"], a["T"], a["cols"], a["q"], a["s"], None)) == status
    assert _status(b, b.LIB.vq_mx4_dequant(a["q"], a["s"], a["T"], a["cols"], a["dt"], a["x"], None)) == status


# ---- product --------------------------------------------------------------

def _tensor(b, rows=64, cols=256, E=1, **kw):
    t = b.CMX4Tensor(0x100000, 0x200001, rows, cols, E, 0, E * rows * cols // 2, E * rows * cols // 32)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _gemm(b, w=None, io=None, x=0x10000, xs=0x20001, T=4, y=0x30000, ws=0x40000, wsb=1 << 40):
    w = _tensor(b) if w is None else w
    return _status(b, b.LIB.vq_mx4_gemm(ctypes.byref(w), None if io is None else ctypes.byref(io), x, xs, T, y, ws, wsb,
                                        None))


@pytest.mark.parametrize("w,status", [
    (dict(values=None), "VQ_ERR_NULL"),
    (dict(scales=None), "VQ_ERR_NULL"),
    (dict(rows=0), "VQ_ERR_SHAPE"),
    (dict(rows=(1 << 24) + 1), "VQ_ERR_SHAPE"),
    (dict(cols=0), "VQ_ERR_SHAPE"),
    (dict(cols=240), "VQ_ERR_SHAPE"),
    (dict(num_experts=0), "VQ_ERR_SHAPE"),
    (dict(num_experts=2, value_bytes=2 * 64 * 128, scale_bytes=2 * 64 * 8), "VQ_ERR_SHAPE"),   # a stack
    (dict(reserved=1), "VQ_ERR_SHAPE"),
    (dict(value_bytes=64 * 128 - 16), "VQ_ERR_SHAPE"),
    (dict(scale_bytes=64 * 8 + 1), "VQ_ERR_SHAPE"),
    (dict(values=0x100008), "VQ_ERR_ALIGN"),
])
def test_product_refuses_weights(b, w, status):
    assert _gemm(b, w=_tensor(b, **w)) == status, b.LIB.vq_last_error()


@pytest.mark.parametrize("io,kw,status", [
    ((4, 3, 0, 0), {}, "VQ_ERR_SHAPE"),
    ((4, 4, 0, 0), {}, "VQ_ERR_SHAPE"),
    ((0, 0, 0, 0), {}, "VQ_ERR_SHAPE"),
    ((3, 0, 0, 0), {}, "VQ_ERR_SHAPE"),
    ((4, 0, 2, 0), {}, "VQ_ERR_SHAPE"),
    ((4, 0, 0, 1), {}, "VQ_ERR_SHAPE"),
    ((1, 0, 0, 0), {}, "VQ_ERR_SHAPE"),                       # 16-bit x with scales
    (None, dict(xs=0), "VQ_ERR_NULL"),
    (None, dict(x=0), "VQ_ERR_NULL"),
    (None, dict(y=0), "VQ_ERR_NULL"),
    (None, dict(x=0x10008), "VQ_ERR_ALIGN"),
    (None, dict(y=0x30004), "VQ_ERR_ALIGN"),
    (None, dict(T=-1), "VQ_ERR_SHAPE"),
    (None, dict(T=(1 << 24) + 1), "VQ_ERR_SHAPE"),
    (None, dict(T=0, x=0, xs=0, y=0, ws=0), "VQ_OK"),
])
def test_product_refuses_calls(b, io, kw, status):
    assert _gemm(b, io=None if io is None else b.CIo(*io, None), **kw) == status, b.LIB.vq_last_error()


def test_product_refuses_odd_rows_under_swiglu_and_too_many_tiles(b):
    assert _gemm(b, w=_tensor(b, rows=63), io=b.CIo(4, 0, 1, 0, None)) == "VQ_ERR_SHAPE"
    assert _gemm(b, w=_tensor(b, rows=1 << 24, cols=32), T=1 << 24) == "VQ_ERR_SHAPE"
    assert _status(b, b.LIB.vq_mx4_gemm(None, None, 0x10000, 0x20000, 1, 0x30000, None, 0, None)) == "VQ_ERR_NULL"


def test_product_workspace_bytes(b):
    assert b.LIB.vq_mx4_workspace_bytes(64, 48, 4) == 0 and b"cols" in b.LIB.vq_last_error()
    assert b.LIB.vq_mx4_workspace_bytes(0, 64, 4) == 0
    assert b.LIB.vq_mx4_workspace_bytes(64, 64, 0) == 0


@pytest.mark.parametrize("rows,cols,T", [(1, 32, 1), (5120, 17408, 16), (17408, 5120, 2048), (128, 17408, 100),
                                         (1 << 24, 32, 64), (64, 1 << 20, 1 << 10), (16, 1 << 20, 16)])
def test_product_workspace_is_checked(b, rows, cols, T):
    need = b.LIB.vq_mx4_workspace_bytes(rows, cols, T)
    assert 0 <= need <= 1 << 29
    if need:
        w = _tensor(b, rows=rows, cols=cols)
        for io in (b.CIo(4, 0, 0, 0, None), b.CIo(2, 0, 0, 0, None)):
            xs = 0x20000 if io.x_dtype == 4 else None
            assert _gemm(b, w=w, io=io, xs=xs, T=T, ws=0) == "VQ_ERR_WORKSPACE"
            assert _gemm(b, w=w, io=io, xs=xs, T=T, wsb=need - 1) == "VQ_ERR_WORKSPACE"
            assert _gemm(b, w=w, io=io, xs=xs, T=T, ws=0x40008) == "VQ_ERR_ALIGN"


# ---- layer ----------------------------------------------------------------

def _moe(b, router=None, gu=None, dn=None, io=None, logits=0x10000, x=0x20000, T=4, y=0x30000, ids=0x40000,
         weights=0x50000, ws=0x60000, wsb=1 << 40):
    r = dict(num_experts=16, top_k=2, score=0, logits_dtype=0, groups=1, top_groups=1, group_score=0, renormalize=1,
             scale=1.0, reserved=0, bias=None)
    r.update(router or {})
    gu = _tensor(b, 128, 96, 16) if gu is None else gu
    dn = _tensor(b, 96, 64, 16) if dn is None else dn
    return _status(b, b.LIB.vq_mx4_moe(ctypes.byref(b.CRouter(**r)), ctypes.byref(gu), ctypes.byref(dn),
                                       None if io is None else ctypes.byref(io), logits, x, T, y, ids, weights, ws, wsb,
                                       None))


@pytest.mark.parametrize("kw,status", [
    (dict(router=dict(num_experts=15)), "VQ_ERR_SHAPE"),
    (dict(router=dict(top_k=17)), "VQ_ERR_SHAPE"),
    (dict(router=dict(score=7)), "VQ_ERR_SHAPE"),
    (dict(router=dict(bias=0x1002)), "VQ_ERR_ALIGN"),
    (dict(io=(4, 0, 0, 0)), "VQ_ERR_SHAPE"),
    (dict(io=(0, 0, 0, 0)), "VQ_ERR_SHAPE"),
    (dict(io=(1, 3, 0, 0)), "VQ_ERR_SHAPE"),
    (dict(io=(1, 0, 1, 0)), "VQ_ERR_SHAPE"),
    (dict(io=(1, 0, 0, 1)), "VQ_ERR_SHAPE"),
    (dict(T=-1), "VQ_ERR_SHAPE"),
    (dict(T=65), "VQ_ERR_SHAPE"),
    (dict(logits=0), "VQ_ERR_NULL"),
    (dict(x=0), "VQ_ERR_NULL"),
    (dict(y=0), "VQ_ERR_NULL"),
    (dict(ids=0), "VQ_ERR_NULL"),
    (dict(weights=0), "VQ_ERR_NULL"),
    (dict(ws=0), "VQ_ERR_WORKSPACE"),
    (dict(logits=0x10002), "VQ_ERR_ALIGN"),
    (dict(x=0x20008), "VQ_ERR_ALIGN"),
    (dict(y=0x30008), "VQ_ERR_ALIGN"),
    (dict(ids=0x40002), "VQ_ERR_ALIGN"),
    (dict(ws=0x60004), "VQ_ERR_ALIGN"),
    (dict(T=0, logits=0, x=0, y=0, ids=0, weights=0, ws=0), "VQ_OK"),
])
def test_layer_refuses(b, kw, status):
    kw = dict(kw)
    if "io" in kw:
        kw["io"] = b.CIo(*kw["io"], None)
    assert _moe(b, **kw) == status, b.LIB.vq_last_error()


def test_layer_refuses_experts_that_do_not_fit(b):
    assert _moe(b, dn=_tensor(b, 96, 96, 16)) == "VQ_ERR_SHAPE"
    assert _moe(b, dn=_tensor(b, 64, 64, 16)) == "VQ_ERR_SHAPE"
    assert _moe(b, dn=_tensor(b, 96, 64, 8)) == "VQ_ERR_SHAPE"
    assert _moe(b, gu=_tensor(b, 128, 96, 8)) == "VQ_ERR_SHAPE"
    assert _moe(b, gu=_tensor(b, 128, 96, 16, scale_bytes=5)) == "VQ_ERR_SHAPE"
    assert _moe(b, dn=_tensor(b, 96, 64, 16, values=None)) == "VQ_ERR_NULL"
    # 64 tokens x 32 slots are more pairs than a call takes
    many = dict(num_experts=64, top_k=32)
    assert _moe(b, router=many, gu=_tensor(b, 128, 96, 64), dn=_tensor(b, 96, 64, 64), T=64) == "VQ_ERR_SHAPE"
    # more activations than a launch holds
    assert _moe(b, gu=_tensor(b, 1 << 21, 96, 16), dn=_tensor(b, 96, 1 << 20, 16), T=64) == "VQ_ERR_SHAPE"
    need = b.LIB.vq_mx4_moe_workspace_bytes(4, 2, 96, 64)
    assert need >= 4 * 2 * 64 * 6 and _moe(b, wsb=need - 1) == "VQ_ERR_WORKSPACE"
    assert b.LIB.vq_mx4_moe_workspace_bytes(65, 2, 96, 64) == 0 and b.LIB.vq_mx4_moe_workspace_bytes(0, 2, 96, 64) == 0
    assert b.LIB.vq_mx4_moe_workspace_bytes(4, 2, 90, 64) == 0


# ---- binding --------------------------------------------------------------

def test_wrappers_refuse_before_the_library(b):
    import torch
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    w = b.MX4Tensor(u8(64, 64), u8(64, 4))
    with pytest.raises(ValueError, match="GPU"):
        b.mx4_quant(torch.zeros(2, 64))
    with pytest.raises(ValueError, match="multiple of 32"):
        b.mx4_quant(torch.zeros(2, 48))
    with pytest.raises(ValueError, match="dtype"):
        b.mx4_quant(torch.zeros(2, 64, dtype=torch.float64))
    with pytest.raises(ValueError, match="scales must be"):
        b.mx4_dequant(u8(2, 32), u8(2, 4))
    with pytest.raises(ValueError, match="q must be"):
        b.mx4_dequant(torch.zeros(2, 32), u8(2, 2))
    with pytest.raises(ValueError, match="GPU"):
        b.mx4_gemm(w, u8(3, 64), u8(3, 4))
    with pytest.raises(ValueError, match="one byte for each 32"):
        b.mx4_gemm(b.MX4Tensor(u8(64, 64), u8(64, 2)), u8(3, 64), u8(3, 4))
    with pytest.raises(ValueError, match="must be .*uint8"):
        b.mx4_gemm(b.MX4Tensor(torch.zeros(64, 64), u8(64, 4)), u8(3, 64), u8(3, 4))
    many = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="meta")  # noqa: E731
    with pytest.raises(ValueError, match="at most 2"):
        b.mx4_quant(many(1 << 32, 32, dtype=torch.float16))
    with pytest.raises(ValueError, match="at most 2"):
        b.mx4_dequant(many(1 << 32, 16, dtype=torch.uint8), many(1 << 32, 1, dtype=torch.uint8))
    assert b.mx4_quant.__doc__ and b.mx4_moe.__doc__
    assert ctypes.sizeof(b.CMX4Tensor) == len(b._pack_mx4(1, 2, 3, 4, 5, 0, 7, 8))
