"""Refusals of the router, the products and the NVFP4 conversions, on the
host: the C ABI's argument checks return before anything touches the context
or a pointer (both are made-up addresses here), and the torch-level calls
refuse tensors before the library is reached."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import rank_sum_residual_gb300 as farn  # noqa: E402

INVALID, ALIAS = farn.FARN_ERR_INVALID_ARG, farn.FARN_ERR_ALIAS
GB = 1 << 30
A, B, C, D, E_, F, G_ = (GB * (i + 1) for i in range(7))


@pytest.fixture(scope="module")
def ctx():
    farn.build_library()
    # never read: every call below is refused by its arguments
    buf = ctypes.create_string_buffer(4096)
    yield ctypes.addressof(buf)


def route(ctx, **kw):
    a = dict(logits=A, logits_dtype=farn.FARN_F32, T=4, E=8, K=2, renormalize=1, experts=B,
             gates=C, index=D, rows=E_, offsets=F)
    a.update(kw)
    return farn.farn_moe_route(ctx, *a.values())


@pytest.mark.parametrize("kw", [
    dict(logits=0), dict(logits_dtype=2), dict(T=-1), dict(E=0), dict(E=1025), dict(K=0),
    dict(K=9), dict(E=64, K=33), dict(experts=0), dict(gates=0), dict(index=0), dict(rows=0),
    dict(offsets=0), dict(T=1 << 31, K=1), dict(T=1 << 30, K=2), dict(logits=A + 2),
    dict(rows=E_ + 1), dict(logits=A + 1, logits_dtype=farn.FARN_BF16),
    dict(T=0, offsets=0),
])
def test_route_invalid(ctx, kw):
    assert route(ctx, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(experts=A), dict(gates=B), dict(index=B + 28), dict(rows=F + 32), dict(offsets=A + 100),
])
def test_route_alias(ctx, kw):
    assert route(ctx, **kw) == ALIAS


def grouped(ctx, **kw):
    a = dict(x=A, n_rows=4, rows=B, n_slots=8, weights=C, E=3, offsets=D, N=32, H=64, out=E_)
    a.update(kw)
    return farn.farn_grouped_matmul(ctx, *a.values())


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(weights=0), dict(offsets=0), dict(out=0), dict(n_rows=-1), dict(n_slots=-1),
    dict(N=0), dict(H=0), dict(E=0), dict(E=1025), dict(rows=0),  # rows NULL: n_rows == n_slots
    dict(x=A + 1), dict(rows=B + 2), dict(offsets=D + 1), dict(out=E_ + 1),
    dict(n_slots=1 << 31), dict(H=1 << 31), dict(N=1 << 31),
    dict(N=(1 << 31) - 1, H=(1 << 31) - 1, E=1024),
])
def test_grouped_invalid(ctx, kw):
    assert grouped(ctx, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(out=A), dict(out=C + 2), dict(out=D + 8), dict(out=B - 8 * 32 * 2 + 4),
])
def test_grouped_alias(ctx, kw):
    assert grouped(ctx, **kw) == ALIAS


def test_grouped_no_slots_launches_nothing(ctx):
    assert grouped(ctx, n_slots=0, x=0, rows=B, out=0) == farn.FARN_OK


def quantize(ctx, **kw):
    a = dict(x=A, T=4, H=64, tensor_scale=1.0, codes=B, block_scale=C)
    a.update(kw)
    return farn.farn_nvfp4_quantize(ctx, *a.values())


def dequantize(ctx, **kw):
    a = dict(codes=B, block_scale=C, T=4, H=64, tensor_scale=1.0, out=A)
    a.update(kw)
    return farn.farn_nvfp4_dequantize(ctx, *a.values())


SHARED = [dict(T=-1), dict(H=0), dict(H=24), dict(tensor_scale=0.0), dict(tensor_scale=-1.0),
          dict(tensor_scale=float("nan")), dict(tensor_scale=float("inf")), dict(codes=0),
          dict(block_scale=0), dict(T=1 << 60, H=64)]


@pytest.mark.parametrize("kw", SHARED)
def test_conversions_invalid(ctx, kw):
    assert quantize(ctx, **kw) == INVALID
    assert dequantize(ctx, **kw) == INVALID


def test_conversions_own_pointers(ctx):
    assert quantize(ctx, x=0) == INVALID and quantize(ctx, x=A + 1) == INVALID
    assert dequantize(ctx, out=0) == INVALID and dequantize(ctx, out=A + 1) == INVALID
    assert quantize(ctx, codes=A) == ALIAS and quantize(ctx, block_scale=B + 127) == ALIAS
    assert dequantize(ctx, out=B) == ALIAS and dequantize(ctx, out=C - 510) == ALIAS
    assert quantize(ctx, T=0, x=0, codes=0, block_scale=0) == farn.FARN_OK
    assert dequantize(ctx, T=0, out=0, codes=0, block_scale=0) == farn.FARN_OK


def product(ctx, **kw):
    a = dict(a_codes=A, a_scale=B, ga=2.0, b_codes=C, b_scale=D, gb=4.0, T=4, N=32, H=64, out=E_)
    a.update(kw)
    return farn.farn_nvfp4_matmul(ctx, *a.values())


@pytest.mark.parametrize("kw", [
    dict(a_codes=0), dict(a_scale=0), dict(b_codes=0), dict(b_scale=0), dict(out=0),
    dict(T=-1), dict(N=0), dict(H=0), dict(H=24), dict(ga=0.0), dict(gb=float("nan")),
    dict(ga=float("inf")), dict(ga=1e-30, gb=1e-30),   # alpha above fp32
    dict(ga=1e30, gb=1e30),                             # alpha below fp32
    dict(out=E_ + 1), dict(T=1 << 31), dict(N=1 << 31), dict(H=1 << 31),
])
def test_product_invalid(ctx, kw):
    assert product(ctx, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(out=A), dict(out=B + 8), dict(out=C + 100), dict(out=D - 8)])
def test_product_alias(ctx, kw):
    assert product(ctx, **kw) == ALIAS


def test_product_no_rows_launches_nothing(ctx):
    assert product(ctx, T=0, a_codes=0, a_scale=0, out=0) == farn.FARN_OK


def test_too_many_tiles(ctx):
    """More tiles than 32-bit numbers hold are refused before the device is
    touched, by the call and by its plan query."""
    n, far = (1 << 21) + 64, 1 << 46        # outputs of over 2^43 bytes
    assert grouped(ctx, n_rows=n, rows=0, n_slots=n, E=1, N=n, H=1, out=far) == \
        farn.FARN_ERR_UNSUPPORTED
    assert product(ctx, T=n, N=n, H=16, out=far) == farn.FARN_ERR_UNSUPPORTED
    with pytest.raises(farn.FarnError) as e:
        farn.farn_plan_grouped_matmul(ctx, A, n, 0, n, C, 1, n, 1, far)
    assert e.value.status == farn.FARN_ERR_UNSUPPORTED
    with pytest.raises(farn.FarnError) as e:
        farn.farn_plan_nvfp4_matmul(ctx, A, B, C, D, n, n, 16, far)
    assert e.value.status == farn.FARN_ERR_UNSUPPORTED


def test_too_many_elements(ctx):
    """The conversions take 2^31 - 1 thread blocks of 2^14 elements."""
    T = ((1 << 45) - (1 << 14)) // 16 + 1
    far = dict(T=T, H=16)
    assert quantize(ctx, x=1 << 50, codes=1 << 48, block_scale=1 << 47, **far) == \
        farn.FARN_ERR_UNSUPPORTED
    assert dequantize(ctx, out=1 << 50, codes=1 << 48, block_scale=1 << 47, **far) == \
        farn.FARN_ERR_UNSUPPORTED


def test_plan_queries_refuse(ctx):
    good = dict(x=A, n_rows=4, rows=B, n_slots=8, weights=C, E=3, N=32, H=64, out=E_)
    for kw in (dict(n_slots=0), dict(N=0), dict(E=1025), dict(weights=0), dict(out=0),
               dict(rows=0)):
        with pytest.raises(farn.FarnError) as e:
            farn.farn_plan_grouped_matmul(ctx, *(good | kw).values())
        assert e.value.status == INVALID
    good = dict(a=A, sa=B, b=C, sb=D, T=4, N=32, H=64, out=E_)
    for kw in (dict(T=0), dict(H=40), dict(a=0), dict(sb=0), dict(out=0)):
        with pytest.raises(farn.FarnError) as e:
            farn.farn_plan_nvfp4_matmul(ctx, *(good | kw).values())
        assert e.value.status == INVALID


def test_null_context():
    farn.build_library()
    assert route(0) == grouped(0) == quantize(0) == dequantize(0) == product(0) == INVALID


def test_torch_level_refusals():
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    x = torch.zeros(4, 64, dtype=bf)
    with pytest.raises(ValueError, match="logits"):
        farn.moe_route(torch.zeros(4, 8), 2)                        # not on a GPU
    with pytest.raises(ValueError, match=r"\[T, E\]"):
        farn.moe_route(torch.zeros(8), 2)
    with pytest.raises(TypeError, match="logits"):
        farn.moe_route(torch.zeros(4, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="must be"):
        farn.grouped_matmul(x, torch.zeros(64, 64, dtype=bf), torch.zeros(2, dtype=i32))
    with pytest.raises(TypeError, match="x must be"):
        farn.grouped_matmul(x.float(), torch.zeros(1, 64, 64, dtype=bf), torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError, match="x must be"):
        farn.nvfp4_quantize(torch.zeros(64, dtype=bf), 1.0)
    with pytest.raises(ValueError, match="H % 16"):
        farn.nvfp4_dequantize(torch.zeros(4, 12, dtype=u8), torch.zeros(4, 1, dtype=u8), 1.0)
    with pytest.raises(ValueError, match="a_codes must be on"):
        farn.nvfp4_matmul(torch.zeros(4, 32, dtype=u8), torch.zeros(4, 4, dtype=u8), 1.0,
                          torch.zeros(4, 32, dtype=u8), torch.zeros(4, 4, dtype=u8), 1.0)
