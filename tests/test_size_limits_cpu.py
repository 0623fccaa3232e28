"""Sizes past 32 bits are refused by the wrappers: the library's arguments have
32, and what ctypes cuts off would leave a call of a small rest."""
import pytest


@pytest.fixture(scope="module")
def b():
    from vq_dequant_matmul_gemv_amd import binding
    return binding


def _meta(*shape, dtype="uint8"):
    import torch
    return torch.empty(*shape, dtype=getattr(torch, dtype), device="meta")


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 128])
def test_columns_and_rows_past_32_bits(b, n):
    with pytest.raises(ValueError, match=f"{n} columns: at most 2"):
        b.mx4_quant(_meta(1, n, dtype="float16"))
    with pytest.raises(ValueError, match=f"{n} columns: at most 2"):
        b.mx4_dequant(_meta(1, n // 2), _meta(1, n // 32))
    with pytest.raises(ValueError, match=f"{n} columns: at most 2"):
        b.fp8_quant(_meta(1, n, dtype="bfloat16"))
    with pytest.raises(ValueError, match=f"{n} rows: at most 2"):
        b.moe_route(b.Router(1, 1), _meta(n, 1, dtype="float16"))
    for shape in ((n, 32), (32, n), (n, 1, 32)):
        w = b.MX4Tensor(_meta(*shape[:-1], shape[-1] // 2), _meta(*shape[:-1], shape[-1] // 32))
        with pytest.raises(ValueError, match="at most 2"):
            b.mx4_gemm(w, _meta(1, shape[-1], dtype="float16"))


def test_largest_sizes_pass_on(b):
    """One less is the library's to judge (here the tensors' place is)."""
    n = (1 << 31) - 128
    with pytest.raises(ValueError, match="GPU"):
        b.mx4_quant(_meta(1, n, dtype="float16"))
    with pytest.raises(ValueError, match="GPU"):
        b.moe_route(b.Router(1, 1), _meta(n, 1, dtype="float16"))
