"""Refusals of the FP8 quantisation and products, of the heads' norms and
rotations and of the cache, on the host: the C ABI's argument checks return
before anything touches the context or a pointer (both are made-up addresses
here), and the torch-level calls refuse tensors before the library is reached."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import rank_sum_residual_gb300 as farn  # noqa: E402

INVALID, ALIAS, OK = farn.FARN_ERR_INVALID_ARG, farn.FARN_ERR_ALIAS, farn.FARN_OK
UNSUPPORTED = farn.FARN_ERR_UNSUPPORTED
GB = 1 << 30
A, B, C, D, E_, F, G_, H_, I_, J_ = (GB * (i + 1) for i in range(10))


@pytest.fixture(scope="module")
def ctx():
    farn.build_library()
    # never read: every call below is refused by its arguments
    buf = ctypes.create_string_buffer(4096)
    yield ctypes.addressof(buf)


def quantize(ctx, **kw):
    a = dict(x=A, E=1, T=4, H=200, block_rows=1, codes=B, scales=C)
    a.update(kw)
    return farn.farn_fp8_quantize(ctx, *a.values())


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(codes=0), dict(scales=0), dict(E=-1), dict(T=-1), dict(H=0), dict(H=-8),
    dict(block_rows=0), dict(block_rows=64), dict(block_rows=-128), dict(x=A + 1),
    dict(scales=C + 2), dict(T=1 << 60), dict(E=1 << 50, T=1 << 20), dict(H=1 << 62),
])
def test_quantize_invalid(ctx, kw):
    assert quantize(ctx, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(codes=A), dict(codes=A + 1599), dict(scales=A + 8),
                                dict(scales=B + 796), dict(codes=C + 31)])
def test_quantize_alias(ctx, kw):
    assert quantize(ctx, **kw) == ALIAS


def test_quantize_nothing_and_too_much(ctx):
    assert quantize(ctx, T=0, x=0, codes=0, scales=0) == OK
    assert quantize(ctx, E=0, x=0, codes=0, scales=0) == OK
    far = dict(x=1 << 50, codes=1 << 48, scales=1 << 47)
    assert quantize(ctx, T=(1 << 37) - 63, H=8, **far) == UNSUPPORTED
    assert quantize(ctx, T=1 << 38, H=8, block_rows=128, **far) == UNSUPPORTED


def product(ctx, **kw):
    a = dict(a=A, sa=B, b=C, sb=D, T=4, N=32, H=64, out=E_)
    a.update(kw)
    return farn.farn_fp8_matmul(ctx, *a.values())


@pytest.mark.parametrize("kw", [
    dict(a=0), dict(sa=0), dict(b=0), dict(sb=0), dict(out=0), dict(T=-1), dict(N=0), dict(H=0),
    dict(out=E_ + 1), dict(sa=B + 1), dict(sb=D + 2), dict(T=1 << 31), dict(N=1 << 31),
    dict(H=1 << 31),
])
def test_product_invalid(ctx, kw):
    assert product(ctx, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(out=A), dict(out=B + 8), dict(out=C + 100), dict(out=D),
                                dict(out=A - 254)])
def test_product_alias(ctx, kw):
    assert product(ctx, **kw) == ALIAS


def test_product_no_rows_launches_nothing(ctx):
    assert product(ctx, T=0, a=0, sa=0, out=0) == OK


def grouped(ctx, **kw):
    a = dict(x=A, sx=B, n_rows=4, rows=C, n_slots=8, w=D, sw=E_, E=3, offsets=F, N=32, H=64,
             out=G_, workspace=0, workspace_bytes=0)
    a.update(kw)
    return farn.farn_fp8_grouped_matmul(ctx, *a.values())


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(sx=0), dict(w=0), dict(sw=0), dict(offsets=0), dict(out=0), dict(n_rows=-1),
    dict(n_slots=-1), dict(N=0), dict(H=0), dict(E=0), dict(E=1025), dict(rows=0), dict(sx=B + 2),
    dict(sw=E_ + 1), dict(rows=C + 2), dict(offsets=F + 1), dict(out=G_ + 1),
    dict(workspace=H_, workspace_bytes=-1), dict(n_slots=1 << 31), dict(H=1 << 31),
    dict(N=(1 << 31) - 1, H=(1 << 31) - 1, E=1024),
])
def test_grouped_invalid(ctx, kw):
    assert grouped(ctx, **kw) == INVALID


ROOM = dict(workspace_bytes=1 << 20)


@pytest.mark.parametrize("kw", [
    dict(out=A), dict(out=B + 4), dict(out=C + 28), dict(out=D + 2), dict(out=E_), dict(out=F + 12),
    dict(workspace=A, **ROOM), dict(workspace=B, **ROOM), dict(workspace=C, **ROOM),
    dict(workspace=D - 16, **ROOM), dict(workspace=E_, **ROOM), dict(workspace=F, **ROOM),
    dict(workspace=G_ + 496, **ROOM),
])
def test_grouped_alias(ctx, kw):
    assert grouped(ctx, **kw) == ALIAS


def test_grouped_no_slots_launches_nothing(ctx):
    for rows in (0, C):
        assert grouped(ctx, n_slots=0, x=0, sx=0, rows=rows, out=0, w=0) == OK


def test_too_many_tiles(ctx):
    n, far = (1 << 21) + 64, 1 << 46        # outputs of over 2^43 bytes
    assert product(ctx, T=n, N=n, H=1, out=far) == UNSUPPORTED
    assert grouped(ctx, n_rows=n, rows=0, n_slots=n, E=1, N=n, H=1, out=far) == UNSUPPORTED
    for call in (lambda: farn.farn_plan_fp8_matmul(ctx, A, C, n, n, 1, far),
                 lambda: farn.farn_plan_fp8_grouped_matmul(ctx, A, n, 0, n, C, 1, n, 1, far)):
        with pytest.raises(farn.FarnError) as e:
            call()
        assert e.value.status == UNSUPPORTED


def test_plan_queries_refuse(ctx):
    good = dict(a=A, b=B, T=4, N=32, H=64, out=C)
    for kw in (dict(T=0), dict(H=0), dict(a=0), dict(b=0), dict(out=0), dict(N=1 << 31)):
        with pytest.raises(farn.FarnError) as e:
            farn.farn_plan_fp8_matmul(ctx, *(good | kw).values())
        assert e.value.status == INVALID
    good = dict(x=A, n_rows=4, rows=B, n_slots=8, w=C, E=3, N=32, H=64, out=E_)
    for kw in (dict(n_slots=0), dict(N=0), dict(E=1025), dict(w=0), dict(out=0), dict(rows=0)):
        with pytest.raises(farn.FarnError) as e:
            farn.farn_plan_fp8_grouped_matmul(ctx, *(good | kw).values())
        assert e.value.status == INVALID
    for args in ((-1, 3, 32, 64), (8, 0, 32, 64), (8, 3, 0, 64), (8, 3, 32, 1 << 31)):
        with pytest.raises(farn.FarnError):
            farn.farn_fp8_grouped_workspace(ctx, *args)


# ---------------------------------------------------------------- heads, cache
def rope(ctx, **kw):
    a = dict(T=4, D=64, q=A, q_heads=2, q_stride=128, k=B, k_heads=1, k_stride=64, q_weight=C,
             k_weight=D, eps=1e-6, positions=E_, axes=2, sections=(20, 12), freqs=F, R=64,
             interleaved=0, q_out=G_, q_out_stride=128, k_out=H_, k_out_stride=64)
    a.update(kw)
    return farn.farn_qk_norm_rope(ctx, *a.values())


ROPE_INVALID = [
    dict(T=-1), dict(T=1 << 31), dict(D=0), dict(D=1025), dict(q=0), dict(k=0), dict(q_heads=-1),
    dict(q_heads=0, k_heads=0), dict(q_stride=127), dict(k_stride=63), dict(k_stride=-64),
    dict(q=A + 1), dict(q_weight=C + 1), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(positions=0), dict(freqs=0), dict(positions=E_ + 2),
    dict(freqs=F + 1), dict(axes=0), dict(axes=5, sections=(8, 8, 8, 4, 4)), dict(sections=None),
    dict(sections=(20, 11)), dict(sections=(20, 13)), dict(sections=(33, -1)), dict(R=-2),
    dict(R=63), dict(R=66), dict(q_heads=1 << 22, q_stride=1 << 40), dict(q_stride=1 << 62),
]


@pytest.mark.parametrize("kw", ROPE_INVALID + [
    dict(q_out=0), dict(k_out=0), dict(q_out=G_ + 1), dict(q_out_stride=100),
    dict(k_out_stride=0)])
def test_rope_invalid(ctx, kw):
    assert rope(ctx, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(q_out=A + 128), dict(q_out=B), dict(q_out=A, q_out_stride=256), dict(k_out=A + 256),
    dict(q_out=C - 1022), dict(k_out=D + 126), dict(q_out=E_ + 30), dict(k_out=F),
    dict(k_out=G_), dict(q_out=H_),
    # packed rows: the keys' place overlaps the queries' last head
    dict(q_stride=192, k_stride=192, k=A + 256, q_out=A, q_out_stride=192, k_out=A + 255 - 63,
         k_out_stride=192),
])
def test_rope_alias(ctx, kw):
    assert rope(ctx, **kw) == ALIAS


def test_rope_nothing(ctx):
    assert rope(ctx, T=0, q=0, k=0, q_out=0, k_out=0, positions=0) == OK
    # the checks that do not need the tensors come first
    assert rope(ctx, T=0, R=63) == INVALID


def store(**kw):
    a = dict(format=farn.FARN_CACHE_FP8, page_size=16, n_pages=8, heads=1, head_dim=64,
             k_codes=H_, v_codes=I_, k_scale=J_, v_scale=J_ + GB, k_tensor_scale=1.0,
             v_tensor_scale=1.0)
    a.update(kw)
    return farn.KvCache(*a.values())


def to_cache(ctx, cache=None, **kw):
    a = dict(T=4, D=64, q=A, q_heads=2, q_stride=128, k=B, k_stride=64, v=B + GB // 2, v_stride=64,
             kv_heads=1, q_weight=C, k_weight=D, eps=1e-6, positions=E_, axes=2,
             sections=(20, 12), freqs=F, R=64, interleaved=0, q_out=G_, q_out_stride=128,
             cache=store() if cache is None else cache, slots=G_ + GB // 2)
    a.update(kw)
    return farn.farn_qk_norm_rope_cache(ctx, *a.values())


@pytest.mark.parametrize("kw", [{k: v for k, v in kw.items()} for kw in ROPE_INVALID
                                if "k_heads" not in kw] + [
    dict(v=0), dict(v=B + 1), dict(v_stride=10), dict(kv_heads=0), dict(kv_heads=2), dict(D=32),
    dict(slots=0), dict(slots=G_ + 2), dict(q_out=0)])
def test_rope_cache_invalid(ctx, kw):
    assert to_cache(ctx, **kw) == INVALID


NVFP4 = dict(format=farn.FARN_CACHE_NVFP4)


@pytest.mark.parametrize("kw", [
    dict(format=0), dict(format=3), dict(page_size=0), dict(n_pages=-1), dict(heads=0),
    dict(head_dim=0), dict(head_dim=1025), dict(k_codes=0), dict(v_codes=0), dict(k_scale=0),
    dict(v_scale=0), dict(k_scale=J_ + 2), dict(n_pages=1 << 31), dict(n_pages=1 << 27, page_size=16),
    dict(k_tensor_scale=0.0, **NVFP4), dict(v_tensor_scale=-1.0, **NVFP4),
    dict(k_tensor_scale=float("nan"), **NVFP4), dict(v_tensor_scale=float("inf"), **NVFP4),
    dict(head_dim=72, **NVFP4)])
def test_cache_invalid(ctx, kw):
    c = store(**kw)
    heads, dim = c.heads, c.head_dim
    assert to_cache(ctx, c, kv_heads=max(heads, 1), D=max(dim, 1), k_stride=2048, v_stride=2048,
                    q_stride=4096, q_out_stride=4096, R=0) == INVALID
    assert write(ctx, cache=c) == INVALID
    assert read(ctx, cache=c) == INVALID


@pytest.mark.parametrize("kw", [dict(k_codes=A), dict(v_codes=B), dict(k_scale=B + GB // 2),
                                dict(v_scale=G_), dict(k_codes=C - 8000), dict(v_codes=E_),
                                dict(k_scale=F + 124), dict(v_scale=G_ + GB // 2 + 12),
                                dict(k_codes=I_ + 8191), dict(k_scale=H_), dict(k_scale=J_ + GB)])
def test_cache_alias(ctx, kw):
    assert to_cache(ctx, store(**kw)) == ALIAS


def test_rope_cache_alias(ctx):
    assert to_cache(ctx, q_out=B) == ALIAS
    assert to_cache(ctx, q_out=B + GB // 2) == ALIAS


def write(ctx, **kw):
    a = dict(T=4, k=A, k_stride=64, v=B, v_stride=64, cache=store(), slots=C)
    a.update(kw)
    return farn.farn_kv_write(ctx, *a.values())


def test_write_refusals(ctx):
    for kw in (dict(T=-1), dict(k=0), dict(v=0), dict(k=A + 1), dict(k_stride=63),
               dict(v_stride=1), dict(slots=0), dict(slots=C + 1), dict(cache=None)):
        assert write(ctx, **kw) == INVALID, kw
    for kw in (dict(k_codes=A - 8191), dict(v_codes=B), dict(k_scale=C), dict(v_scale=A + 508)):
        assert write(ctx, cache=store(**kw)) == ALIAS, kw
    assert write(ctx, T=0, k=0, v=0, slots=0) == OK


def read(ctx, **kw):
    a = dict(cache=store(), table=A, B=2, width=3, offsets=B, n_tokens=40, k_out=C, v_out=D)
    a.update(kw)
    return farn.farn_kv_read(ctx, *a.values())


def test_read_refusals(ctx):
    for kw in (dict(cache=None), dict(table=0), dict(offsets=0), dict(k_out=0), dict(v_out=0),
               dict(B=-1), dict(width=-1), dict(width=1 << 31), dict(n_tokens=-1),
               dict(n_tokens=1 << 31), dict(table=A + 2), dict(offsets=B + 1), dict(k_out=C + 1),
               dict(v_out=D + 1)):
        assert read(ctx, **kw) == INVALID, kw
    for kw in (dict(k_out=A), dict(v_out=B + 8), dict(k_out=D), dict(k_out=H_ + 8190),
               dict(v_out=I_), dict(k_out=J_), dict(v_out=J_ + GB + 508)):
        assert read(ctx, **kw) == ALIAS, kw
    assert read(ctx, n_tokens=0, k_out=0, v_out=0) == OK
    assert read(ctx, B=0, table=0) == OK
    wide = store(heads=1 << 17, head_dim=512, n_pages=1, page_size=1)
    assert read(ctx, cache=wide) == UNSUPPORTED


def test_read_table_sizes(ctx):
    """A table whose bytes do not fit 63 bits."""
    most = (1 << 31) - 1
    assert read(ctx, B=most, width=most) == INVALID
    assert read(ctx, B=most, width=1 << 30, n_tokens=0) == OK
    assert read(ctx, B=most, width=(1 << 30) + 1) == INVALID


def test_null_context():
    farn.build_library()
    assert quantize(0) == product(0) == grouped(0) == rope(0) == to_cache(0) == write(0) == \
        read(0) == INVALID


def test_torch_level_refusals():
    bf, i32, u8, f32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
    z = torch.zeros
    x = z(4, 256, dtype=bf)
    with pytest.raises(ValueError, match="must be on|must be"):
        farn.fp8_quantize(x)                                        # not on a GPU
    with pytest.raises(ValueError, match="block_rows"):
        farn.fp8_quantize(x, 64)
    with pytest.raises(ValueError, match=r"\[T, H\]"):
        farn.fp8_quantize(x[0])
    with pytest.raises(TypeError, match="x must be"):
        farn.fp8_quantize(x.float())
    q, s = z(4, 256, dtype=u8), z(4, 2)
    with pytest.raises(ValueError, match="a_codes must be on"):
        farn.fp8_matmul(q, s, q, z(1, 2))
    with pytest.raises(ValueError, match=r"\[T, H\]"):
        farn.fp8_matmul(q[0], s, q, z(1, 2))
    with pytest.raises(TypeError, match="a_codes"):
        farn.fp8_matmul(x, s, q, z(1, 2))
    with pytest.raises(ValueError, match=r"\[E, N, H\]"):
        farn.fp8_grouped_matmul(q, s, q, s, z(2, dtype=i32))
    with pytest.raises(ValueError, match="x must be on"):
        farn.fp8_grouped_matmul(q, s, z(1, 8, 256, dtype=u8), z(1, 1, 2), z(2, dtype=i32))
    h = z(4, 2, 64, dtype=bf)
    with pytest.raises(ValueError, match=r"\[T, heads, D\]"):
        farn.qk_norm_rope(x, x, None, None, 1e-6)
    with pytest.raises(TypeError, match="q must be"):
        farn.qk_norm_rope(h.float(), h, None, None, 1e-6)
    with pytest.raises(ValueError, match="q must be on"):
        farn.qk_norm_rope(h, h, None, None, 1e-6)
    c = farn.kv_cache(2, 4, 2, 64, "fp8", "cpu")
    assert [t.dtype for t in c] == [u8, u8, f32, f32] and c[0].shape == (2, 4, 2, 64)
    assert farn.kv_cache(2, 4, 2, 64, "nvfp4", "cpu")[3].shape == (2, 4, 2, 4)
    with pytest.raises(ValueError, match="format"):
        farn.kv_cache(2, 4, 2, 64, "int8", "cpu")
    with pytest.raises(ValueError, match="head_dim % 16"):
        farn.kv_cache(2, 4, 2, 72, "nvfp4", "cpu")
    with pytest.raises(ValueError, match="k must be on"):
        farn.kv_write(h, h, c, z(4, dtype=i32))
    with pytest.raises(ValueError, match="k_codes must be on"):
        farn.kv_read(c, z(1, 2, dtype=i32), z(2, dtype=i32), 8)
