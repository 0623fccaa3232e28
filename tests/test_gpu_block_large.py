"""The operators around the products where offsets pass 32 bits, at their size
limits, and on buffers aligned to no more than they have to be; sampled rows
against the 64-bit oracles."""
import numpy as np
import pytest

from oracle import block_oracle as O
from tests.helpers import announce
from vq_dequant_matmul_gemv_amd import synth

pytestmark = pytest.mark.gpu


def _codes(shape, seed):
    """Random e4m3 codes without NaN, made on the GPU."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
    return torch.where((c & 0x7f) == 0x7f, c - 0x30, c)


def _product_rows(xc, xs, wc, ws, rows):
    """y[:, rows] in 64 bits, and the magnitudes' sums."""
    x = O.fp8_values(xc.cpu().numpy(), xs.cpu().numpy())
    w = np.stack([O.fp8_values(wc[r:r + 1].cpu().numpy(), ws[r // 128:r // 128 + 1].cpu().numpy())[0] for r in rows])
    return x @ w.T, np.abs(x) @ np.abs(w).T


@pytest.mark.parametrize("T,R,C", [
    (2, 1100001, 4096),      # 4.5 GB of weights: byte offsets above 2^32
    (3, 40, 1 << 20),        # the longest rows
    (70001, 17, 128),        # many tokens, few rows
    (33000, 65601, 16),      # 2.2e9 outputs
])
def test_large_products(T, R, C):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    announce("fp8_gemm large", T, R, C)
    kb, rb = -(-C // 128), -(-R // 128)
    g = synth.rng("fp8-large", T, R, C)
    wc, xc = _codes((R, C), 1), _codes((T, C), 2)
    ws = torch.from_numpy((0.5 + g.random((rb, kb))).astype(np.float32) * 2.0 ** -12).cuda()
    xs = torch.from_numpy((0.5 + g.random((T, kb))).astype(np.float32) * 2.0 ** -12).cuda()
    w = binding.FP8Tensor(wc, ws)
    tok = sorted({0, 1, T // 2, T - 2, T - 1} & set(range(T)))
    rows = sorted({0, 15, 16, 127, 128, R // 2, R - 17, R - 1} & set(range(R)))
    for dtype in ([torch.bfloat16] if T * R > 1 << 30 else [torch.float32, torch.bfloat16]):
        y = binding.fp8_gemm(w, xc, xs, y_dtype=dtype)
        torch.cuda.synchronize()
        got = y[tok][:, rows].double().cpu().numpy()
        ref, mag = _product_rows(xc[tok], xs[tok], wc, ws, rows)
        half = torch.finfo(dtype).eps / 2
        err = mag * (128 * 2.0 ** -23 + (kb + 28) * 2.0 ** -24)
        assert np.all(np.abs(got - ref) <= err + half * (np.abs(ref) + err)), (dtype, np.abs(got - ref).max())
        del y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,C", [(140001, 16384), ((1 << 23) + 5, 272)])
def test_quantize_more_than_2_31_values(T, C):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    announce("fp8_quant large", T, C)
    x = torch.empty(T, C, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(3))
    q, s = binding.fp8_quant(x)
    torch.cuda.synchronize()
    at = [0, 1, T // 3, (1 << 31) // C, (1 << 31) // C + 1, T - 2, T - 1]
    rq, rs = O.fp8_quant(x[at].double().cpu().numpy())
    assert np.array_equal(q.view(torch.uint8)[at].cpu().numpy(), rq) and np.array_equal(s[at].cpu().numpy(), rs)
    del x, q, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,C", [(140001, 16384), ((1 << 22) + 3, 513), ((1 << 24) + 7, 136)])
def test_norm_of_more_than_2_31_values(T, C):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    announce("norm large", T, C)
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.empty(T, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.rand(C, device="cuda", generator=g).to(torch.bfloat16)
    _, h, _ = binding.norm(None, x, pre_weight=w, store_residual=False)
    torch.cuda.synchronize()
    at = [0, 1, T // 3, (1 << 31) // C, min(T - 1, (1 << 31) // C + 1), T - 2, T - 1]
    ref = O.norm(None, x[at].double().cpu().numpy(), pre_weight=w.double().cpu().numpy())["h"]
    # 42 + 22 half units of fp32 in the norm and the products, half a bf16 unit at the store
    assert np.all(np.abs(h[at].double().cpu().numpy() - ref) <= (2.0 ** -8 + 64 * 2.0 ** -24) * np.abs(ref))
    del x, h
    torch.cuda.empty_cache()


def test_route_the_most_tokens():
    """2^25 tokens, the documented limit, 96 experts a token: 3.2e9 logits."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    T, E = 1 << 25, 96
    announce("route large", T, E)
    x = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    b = 0.05 * torch.randn(E, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    ids, w = binding.moe_route(binding.Router(E, 4, score="sigmoid", bias=b, groups=8, top_groups=4,
                                              group_score="top2"), x)
    torch.cuda.synchronize()
    at = [0, 1, 63, T // 3, (1 << 31) // E, (1 << 31) // E + 1, T - 2, T - 1]
    rid, rw = O.route(x[at].float().cpu().numpy(), 4, score="sigmoid", bias=b.cpu().numpy(), groups=8, top_groups=4,
                      group_score="top2")
    assert np.array_equal(ids[at].cpu().numpy(), rid) and np.allclose(w[at].cpu().numpy(), rw, rtol=2e-6, atol=0)
    del x, ids, w
    torch.cuda.empty_cache()


def _off(t, by):
    """The same values `by` elements behind an aligned address."""
    import torch
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    out = buf[by:].view(t.shape)
    return out.copy_(t)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("E", [96, 160, 256])
def test_route_from_logits_aligned_to_their_element(dtype, E):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    g = torch.Generator().manual_seed(E)
    x = torch.randn(37, E, generator=g).to(getattr(torch, dtype)).cuda()
    b = (0.05 * torch.randn(E, generator=g)).cuda()
    for T in (1, 37):
        ref = binding.moe_route(binding.Router(E, 6, score="sigmoid", bias=b), x[:T])
        for by in (1, 2, 3, 5):
            ids = _off(torch.zeros(T, 6, dtype=torch.int32, device="cuda"), by)
            w = _off(torch.zeros(T, 6, device="cuda"), by)
            binding.moe_route(binding.Router(E, 6, score="sigmoid", bias=_off(b, by)), _off(x[:T], by), ids, w)
            assert torch.equal(ids, ref[0]) and torch.equal(w, ref[1])


@pytest.mark.parametrize("T,R,C", [(1, 300, 1040), (50, 130, 2000), (300, 257, 656)])
def test_scales_and_token_gates_aligned_to_their_element(T, R, C):
    """x_scales, scales and h_scales 4 bytes off, a gate per token 2 bytes off."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    kb, rb = -(-C // 128), -(-R // 128)
    wc, xc = _codes((R, C), 8), _codes((T, C), 9)
    g = torch.Generator("cuda").manual_seed(10)
    ws, xs = torch.rand(rb, kb, device="cuda", generator=g), torch.rand(T, kb, device="cuda", generator=g)
    ref = binding.fp8_gemm(binding.FP8Tensor(wc, ws), xc, xs)
    assert torch.equal(ref, binding.fp8_gemm(binding.FP8Tensor(wc, _off(ws, 1)), xc, _off(xs, 3)))
    x = torch.randn(T, C, device="cuda", generator=g).to(torch.bfloat16)
    q, s = binding.fp8_quant(x)
    q2, s2 = binding.fp8_quant(x, scales=_off(torch.zeros_like(s), 1))
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    gate = torch.randn(T, 1, device="cuda", generator=g).to(torch.bfloat16)
    kw = dict(gate_act="sigmoid", h_dtype=torch.float8_e4m3fn)
    v, h, hs = binding.norm(x, x, gate=gate, **kw)
    v2, h2, hs2 = binding.norm(x, x, gate=_off(gate, 1), h_scales=_off(torch.zeros_like(hs), 1), **kw)
    assert torch.equal(v, v2) and torch.equal(h.view(torch.uint8), h2.view(torch.uint8)) and torch.equal(hs, hs2)
