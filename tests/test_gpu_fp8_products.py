"""How exact vq_fp8_gemm's and vq_fp8_gemm_fast's products are: large ones that
cancel, whole numbers, and the 2-norm of the error, on every kernel and split.

Kernels 0 to 6 of the product's table multiply exactly, 7 to 11 are the e4m3
tiles that only vq_fp8_gemm_fast takes (0 to 2 serve it too)."""
import numpy as np
import pytest

from oracle import block_oracle as O
from tests.helpers import announce
from tests.test_gpu_fp8 import _eps, _operands, _product_check, _torch_dt

pytestmark = pytest.mark.gpu

EXACT, FAST = range(7), (0, 1, 2, 7, 8, 9, 10, 11)
TYPES = ["float32", "float16", "bfloat16"]


def _run(ops, dtype, epilogue=None, fast=False):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    xc, xs, wc, ws = ops
    T, R = xc.shape[0], wc.shape[0]
    announce("fp8_gemm", T, R, xc.shape[1], dtype, epilogue, "fast" if fast else "")
    w = binding.FP8Tensor(torch.from_numpy(wc).cuda(), torch.from_numpy(ws).cuda())
    y = binding.fp8_gemm(w, torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), y_dtype=_torch_dt(dtype),
                         epilogue=epilogue, fast=fast)
    torch.cuda.synchronize()
    return y.double().cpu().numpy()


def _ones(T, R, C):
    kb = -(-C // 128)
    return np.ones((T, kb), np.float32), np.ones((-(-R // 128), kb), np.float32)


def _cancelling(T, R, C):
    """In every eight columns 448 * 448, -448 * 448 and six products of 20, at
    places that change from eight to eight and with the row: y = 120 * C / 8."""
    x, w = np.full((T, C), 4.0), np.full((R, C), 5.0)
    for j in range(0, C, 8):
        a, b = j + (j // 8) % 8, j + (j // 8 + 3) % 8
        x[:, a] = x[:, b] = 448.0
        w[:, a], w[:, b] = 448.0, -448.0
        w[1::2, [a, b]] = w[1::2, [b, a]]
    xs, ws = _ones(T, R, C)
    return (O.e4m3_nearest(x), xs, O.e4m3_nearest(w), ws), 15.0 * C


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,R,C", [(1, 256, 256), (18, 130, 400), (140, 300, 512), (300, 640, 2048),
                                   (2048, 4096, 512), (991, 29, 1024)])
def test_large_products_that_cancel(T, R, C, dtype):
    """Whatever the batch, an output is the sum of its small products: all sums
    are whole numbers below 2^24 (two large products and 20 * 2048)."""
    ops, want = _cancelling(T, R, C)
    y = _run(ops, dtype)
    exact = _rounded(np.array([want]), dtype)[0]
    assert np.all(y == exact), (np.unique(y)[:5], exact)


def _rounded(v, dtype):
    import torch
    return torch.from_numpy(v).to(_torch_dt(dtype)).double().numpy()


@pytest.mark.parametrize("kernel", EXACT)
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("dtype", TYPES)
def test_cancelling_on_every_exact_kernel(kernel, splits, dtype, monkeypatch):
    monkeypatch.setenv("VQMI_FP8_PLAN", f"{kernel},{splits}")
    for T, R, C in [(1, 17, 1296), (70, 258, 1152)]:
        ops, want = _cancelling(T, R, C)
        assert np.all(_run(ops, dtype) == _rounded(np.array([want]), dtype)[0])


@pytest.mark.parametrize("kernel", sorted(set(EXACT) | set(FAST)))
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("dtype", TYPES)
def test_whole_numbers_on_every_kernel(kernel, splits, dtype, monkeypatch):
    """Values of -3 to 3: products up to 9, far less than 2^13 apart, so every
    kernel's fp32 sum is exact and only the output's type rounds it."""
    monkeypatch.setenv("VQMI_FP8_PLAN", f"{kernel},{splits}")
    g = np.random.default_rng(11)
    for T, R, C in [(5, 33, 1424), (200, 259, 2048)]:
        xi, wi = g.integers(-3, 4, (T, C)), g.integers(-3, 4, (R, C))
        xs, ws = _ones(T, R, C)
        ops = (O.e4m3_nearest(xi), xs, O.e4m3_nearest(wi), ws)
        want = _rounded((xi @ wi.T).astype(np.float64), dtype)
        if kernel in EXACT:
            assert np.array_equal(_run(ops, dtype), want)
        if kernel in FAST and dtype != "float32":
            assert np.array_equal(_run(ops, dtype, fast=True), want)


def _norm_error(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


# A block's 128 products are summed with at most 128 roundings (or cuts) of
# 2^-23 of a partial sum.  On these inputs of mean zero the partial sums of a
# block stay within three times its products' 2-norm, which is the block's part
# of y; blocks add in squares on both sides: 3 * 128 * 2^-23 = 4.6e-5, and kb
# scaled additions of 2^-24.  The cut of the e4m3 instructions, at most 7 * 2^-13
# of an eight's largest product, has any sign: 7 products lose less than 2^-13
# of the largest (at most the eight's 2-norm) each, in squares sqrt(7) * 2^-13.
SUMS = 4.6e-5
CUT = 7 ** 0.5 * 2.0 ** -13


@pytest.mark.parametrize("kernel", sorted(set(EXACT) | set(FAST)))
@pytest.mark.parametrize("splits", [1, 2, 5])
def test_two_norm_of_the_error(kernel, splits, monkeypatch):
    """Eight columns of 2000 left out would be 6e-2 of the norm."""
    monkeypatch.setenv("VQMI_FP8_PLAN", f"{kernel},{splits}")
    for T, R, C, key in [(65, 126, 3200, "a"), (193, 300, 2000, "b"), (18, 40, 128 * 300 + 16, "long")]:
        ops = _operands(T, R, C, ("two-norm", key), 0.2)
        ref, _ = O.fp8_product(*ops)
        tol = SUMS + (ops[1].shape[1] + 4) * 2.0 ** -24
        for dtype in TYPES:
            half = _eps(_torch_dt(dtype))
            if kernel in EXACT:
                e = _norm_error(_run(ops, dtype), ref)
                assert e <= tol + half, (dtype, e)
            if kernel in FAST and dtype != "float32":
                e = _norm_error(_run(ops, dtype, fast=True), ref)
                assert e <= tol + CUT + half, (dtype, "fast", e)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,R,C", [(1, 64, 512), (300, 1000, 2000), (600, 4096, 1024)])
def test_fast_products_stay_within_their_bound(T, R, C, dtype):
    """Products from 2^-18 to 448^2 side by side: the error against the 64-bit
    sum within 7 * 2^-13 of every eight's largest product, the fp32 sums' part
    and the output's rounding."""
    g = np.random.default_rng(5)
    xc = O.e4m3_nearest(np.sign(g.normal(size=(T, C))) * 2.0 ** g.uniform(-9, 8.8, (T, C)))
    wc = O.e4m3_nearest(np.sign(g.normal(size=(R, C))) * 2.0 ** g.uniform(-9, 8.8, (R, C)))
    ops = (xc, _ones(T, R, C)[0], wc, _ones(T, R, C)[1])
    ref, mag = O.fp8_product(*ops)
    y = _run(ops, dtype, fast=True)
    x8, w8 = np.abs(O.E4M3[xc]).reshape(T, -1, 8), np.abs(O.E4M3[wc]).reshape(R, -1, 8)
    cut = np.zeros((T, R))
    for j in range(x8.shape[1]):
        big = np.zeros((T, R))
        for i in range(8):
            np.maximum(big, x8[:, j, i, None] * w8[None, :, j, i], out=big)
        cut += 7 * 2.0 ** -13 * big
    err = cut + mag * (128 * 2.0 ** -23 + (C // 128 + 5) * 2.0 ** -24)
    half = _eps(_torch_dt(dtype))
    over = np.abs(ref) > 65000 if dtype == "float16" else np.zeros_like(ref, bool)   # past the type's largest value
    assert np.all(over | (np.abs(y - ref) <= err + half * (np.abs(ref) + err)))


def test_fast_swiglu_captured_and_on_another_stream(monkeypatch):
    """The fast call's epilogue against the exact one's, the same bits again,
    from another stream and from a graph; an fp32 y is refused."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    T, R, C = 300, 512, 2048
    xc, xs, wc, ws = _operands(T, R, C, ("fast-swiglu",), 0.2)
    w = binding.FP8Tensor(torch.from_numpy(wc).cuda(), torch.from_numpy(ws).cuda())
    x, s = torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda()
    for kernel in FAST[3:]:
        monkeypatch.setenv("VQMI_FP8_PLAN", f"{kernel},1")
        kw = dict(y_dtype=torch.bfloat16, epilogue="swiglu", fast=True)
        y = binding.fp8_gemm(w, x, s, **kw)
        ref = binding.fp8_gemm(w, x, s, epilogue="swiglu")
        # gate and up carry the cut (silu' up to 1.1, silu's norm at least 0.4 of its argument's), y its rounding
        assert _norm_error(y.double().cpu().numpy(), ref.double().cpu().numpy()) <= 2.0 ** -8 + 4 * CUT
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        other = binding.fp8_gemm(w, x, s, stream=st, **kw)
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g = binding.fp8_gemm(w, x, s, **kw)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, g) and torch.equal(y, other) and torch.equal(y, binding.fp8_gemm(w, x, s, **kw))
    with pytest.raises(binding.VQError, match="F16 or BF16"):
        binding.fp8_gemm(w, x, s, fast=True)


# ---- many tokens on the few-token kernels, and the planner's splits ----------

@pytest.mark.parametrize("kernel", range(3))
@pytest.mark.parametrize("splits", [1, 3])
def test_few_token_kernels_on_many_tokens(kernel, splits, monkeypatch):
    """The planner takes them for any number of tokens where rows are few."""
    monkeypatch.setenv("VQMI_FP8_PLAN", f"{kernel},{splits}")
    for T, R, C, dtype, epi in [(257, 34, 1200, "float32", None), (500, 18, 2000, "bfloat16", "swiglu"),
                                (1030, 29, 640, "float16", None)]:
        _product_check(_operands(T, R, C, ("many", T, R, C)), dtype, epi)
        e = _run(_operands(T, R, C, ("many", T, R, C), 0.2), "float32")
        assert _norm_error(e, O.fp8_product(*_operands(T, R, C, ("many", T, R, C), 0.2))[0]) <= SUMS + 2.0 ** -19


@pytest.mark.parametrize("T,R,C", [(991, 29, 4400), (300, 64, 17408), (89, 290, 1280), (1012, 453, 160), (868, 175, 1008)])
@pytest.mark.parametrize("dtype", TYPES)
def test_few_rows_and_many_tokens_as_planned(T, R, C, dtype):
    ops = _operands(T, R, C, ("planned", T, R, C), 0.2)
    _product_check(ops, dtype)
    assert _norm_error(_run(ops, dtype), O.fp8_product(*ops)[0]) <= SUMS + (ops[1].shape[1] + 4) * 2.0 ** -24 + (
        _eps(_torch_dt(dtype)) if dtype != "float32" else 2.0 ** -24)


@pytest.mark.parametrize("T,R,C", [(40, 640, 17408), (16, 5120, 17408), (64, 512, 17408)])
def test_planned_splits_within_the_fp32_bound(T, R, C):
    """Shapes the planner splits, on a poisoned workspace of the stated size:
    elementwise the bound of exact products summed in fp32 (128 roundings of
    2^-23 a block, the blocks, planes and scales 2^-24 each), and the 2-norm."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    need = binding.LIB.vq_fp8_workspace_bytes(R, C, T)
    assert need > 0
    xc, xs, wc, ws = ops = _operands(T, R, C, ("planned-split", T), 0.2)
    w = binding.FP8Tensor(torch.from_numpy(wc).cuda(), torch.from_numpy(ws).cuda())
    buf = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
    y = binding.fp8_gemm(w, torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), workspace=buf[:need])
    torch.cuda.synchronize()
    assert torch.all(buf[need:] == 0xff).item()
    got = y.double().cpu().numpy()
    ref, mag = O.fp8_product(*ops)
    assert np.all(np.abs(got - ref) <= mag * (128 * 2.0 ** -23 + (xs.shape[1] + 24 + 4) * 2.0 ** -24) + 2.0 ** -24 * np.abs(ref))
    assert _norm_error(got, ref) <= SUMS + (xs.shape[1] + 28) * 2.0 ** -24


@pytest.mark.parametrize("kernel", FAST[3:])
@pytest.mark.parametrize("at", [0, 8, 56, 64, 72, 120])
def test_fast_products_are_cut_by_their_own_eight_alone(kernel, at, monkeypatch):
    """448 * 448 alone in one eight, 15 other eights of 20s in its block, -448 *
    448 alone in the next block: the 20s stay whole (15 * 8 * 20 = 2400), where
    a cut by a neighbour would take 4 of each."""
    monkeypatch.setenv("VQMI_FP8_PLAN", f"{kernel},1")
    T, R, C = 40, 130, 256
    x, w = np.zeros((T, C)), np.zeros((R, C))
    x[:, :128], w[:, :128] = 4.0, 5.0
    x[:, at:at + 8] = 0
    x[:, at] = x[:, 128 + at] = 448.0
    w[:, at], w[:, 128 + at] = 448.0, -448.0
    ops = (O.e4m3_nearest(x), _ones(T, R, C)[0], O.e4m3_nearest(w), _ones(T, R, C)[1])
    assert np.all(_run(ops, "float16", fast=True) == 2400)
