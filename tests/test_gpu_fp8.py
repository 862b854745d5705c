"""FP8 block quantisation and the FP8 products, dense and by expert, on the
GPU, against plain 64-bit definitions."""
import time

import pytest

torch = pytest.importorskip("torch")

import rank_sum_residual_gb300 as farn  # noqa: E402
from gpu_util import make_ctx  # noqa: E402

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    farn.build_library()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


@pytest.fixture(scope="module")
def ctxs(dev):
    return {"auto": farn.Context(0), "generic": make_ctx(FARN_VARIANT="generic"),
            "pair": make_ctx(FARN_TC_TILE=256),
            "one": make_ctx(FARN_TC_TILE=64, FARN_TC_SPLIT=1),
            "split2": make_ctx(FARN_TC_TILE=64, FARN_TC_SPLIT=2),
            "split4": make_ctx(FARN_TC_TILE=64, FARN_TC_SPLIT=4)}


ALL = ["auto", "generic", "pair", "one", "split2", "split4"]


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


# ------------------------------------------------------------- quantisation
def quantize_reference(x, br):
    """The definition in fp32 on the host: IEEE divisions and products, the
    conversion to the nearest code."""
    x = x.cpu()
    if x.dim() == 2:
        q, s = quantize_reference(x[None], br)
        return q[0], s[0]
    E, T, H = x.shape
    TB, HB = -(-T // br), -(-H // 128)
    f = torch.zeros(E, TB * br, HB * 128)
    f[:, :T, :H] = x.float()
    f = f.view(E, TB, br, HB, 128)
    amax = torch.nan_to_num(f.abs(), nan=0.0, posinf=float("inf")).amax(dim=(2, 4), keepdim=True)
    top = torch.tensor(448.0)
    scale = torch.where(amax > 0, amax / top, 1.0)
    inv = torch.where(amax > 0, (top / amax).clamp(max=torch.finfo(torch.float32).max), 1.0)
    q = (f * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(E, TB * br, HB * 128)[:, :T, :H], scale.view(E, TB, HB)


def normal(dev, shape, seed):
    g = gen(dev, seed)
    x = torch.randn(shape, device=dev, generator=g)
    x *= torch.where(torch.rand(shape, device=dev, generator=g) < 0.01, 50.0, 1.0)
    return x.to(BF)


def check_quantized(got, x, br):
    q, s = (t.cpu() for t in got)
    want_q, want_s = quantize_reference(x, br)
    assert torch.equal(s, want_s)
    nan = (want_q & 127) == 127           # a NaN's sign is not given
    assert torch.equal((q & 127) == 127, nan)
    assert torch.equal(q[~nan], want_q[~nan])


@pytest.mark.parametrize("which", ["auto", "generic"])
@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("shape", [(1, 1), (1, 8), (3, 128), (5, 130), (127, 136), (129, 1000),
                                   (256, 384), (1, 16384), (2000, 72), (3, 70, 200), (2, 300, 128),
                                   (4, 128, 264)])
def test_quantize(dev, ctxs, which, br, shape):
    x = normal(dev, shape, sum(shape) + br)
    check_quantized(farn.fp8_quantize(x, br, ctx=ctxs[which]), x, br)


@pytest.mark.parametrize("which", ["auto", "generic"])
@pytest.mark.parametrize("br", [1, 128])
def test_quantize_special_values(dev, ctxs, which, br):
    x = normal(dev, (300, 640), 3)
    x[0:128, 0:128] = 0.0                                   # no magnitude: scale 1
    x[140, 128:132] = torch.tensor([float("nan"), -0.0, 2.0, -3.0], dtype=BF)
    x[0:256, 256:384] = 0.0
    x[3, 300] = 1e-38                                       # 448 / amax overflows
    x[200, 260] = 9.2e-41                                   # a subnormal alone
    x[7, 500] = 3.3e38                                      # the largest values
    x[131, 400] = float("inf")                              # its block is NaN
    x[280, 512:640] = float("nan")
    check_quantized(farn.fp8_quantize(x, br, ctx=ctxs[which]), x, br)


def test_quantize_any_alignment_and_nothing_behind(dev):
    T, H = 5, 264
    xf = normal(dev, (T * H + 16,), 4)
    for br in (1, 128):
        for d in (0, 1, 4, 8):
            x = xf[d:d + T * H].view(T, H)
            qb = torch.full((T * H + 32,), 99, dtype=torch.uint8, device=dev)
            sb = torch.full((T * 3 + 8,), 99.0, device=dev)
            n = -(-T // br) * 3
            out = qb[d:d + T * H].view(T, H), sb[d:d + n].view(-1, 3) if d < 8 else \
                sb[:n].view(-1, 3)
            check_quantized(farn.fp8_quantize(x, br, out=out), x, br)
            assert (qb[:d] == 99).all() and (qb[d + T * H:] == 99).all()
            assert (sb[(d if d < 8 else 0) + n:] == 99.0).all()


def test_quantize_empty(dev):
    q, s = farn.fp8_quantize(torch.zeros(0, 200, dtype=BF, device=dev))
    assert q.shape == (0, 200) and s.shape == (0, 2)
    q, s = farn.fp8_quantize(torch.zeros(2, 0, 128, dtype=BF, device=dev), 128)
    assert q.shape == (2, 0, 128) and s.shape == (2, 0, 1)


def test_quantize_beyond_4_gib(dev):
    """Rows whose byte offsets pass 32 bits."""
    T, H = 70001, 32768
    x = torch.zeros(T, H, dtype=BF, device=dev)
    some = [0, 32767, 32768, 65535, 65536, 70000]
    x[some] = normal(dev, (len(some), H), 5)
    q, s = farn.fp8_quantize(x)
    check_quantized((q[some], s[some]), x[some], 1)
    assert int((s != 1.0).sum()) == int((s[some] != 1.0).sum())
    del x, q, s
    torch.cuda.empty_cache()


# ----------------------------------------------------------------- products
def e4m3(codes):
    c = codes.long()
    e, f = (c >> 3) & 15, (c & 7).double() / 8
    v = torch.where(e == 0, f * 2.0 ** -6, (1 + f) * torch.exp2(e.double() - 7))
    v = torch.where((c & 127) == 127, float("nan"), v)
    return torch.where(c >= 128, -v, v)


def values(codes, scales, rows=1):
    s = scales.double().repeat_interleave(128, dim=-1)[..., :codes.shape[-1]]
    if rows > 1:
        s = s.repeat_interleave(rows, dim=-2)[..., :codes.shape[-2], :]
    return e4m3(codes) * s


WHOLE = torch.tensor([0.0, 1.0, 2.0, 3.0, -1.0, -2.0, -3.0])


def whole(dev, shape, seed, rows=1):
    """Codes of whole numbers up to 3, scales 1/2, 1 and 2: products are
    multiples of 1/4 and at most 36, so sums below 2^22 are exact in fp32
    whatever the order (H up to 116,000)."""
    g = gen(dev, seed)
    pick = torch.randint(0, 7, shape, device=dev, generator=g)
    q = WHOLE.to(dev)[pick].to(torch.float8_e4m3fn).view(torch.uint8)
    s = (*shape[:-2], -(-shape[-2] // rows), -(-shape[-1] // 128))
    return q, torch.exp2(torch.randint(-1, 2, s, device=dev, generator=g).float())


def spread(dev, shape, seed, rows=1):
    """Codes over the whole range and scales that no few bits hold."""
    g = gen(dev, seed)
    q = torch.randint(0, 256, shape, device=dev, generator=g, dtype=torch.uint8)
    q[(q & 127) == 127] = 0x38
    s = (*shape[:-2], -(-shape[-2] // rows), -(-shape[-1] // 128))
    return q, torch.exp2(6 * torch.rand(s, device=dev, generator=g) - 3)


def to_bf16(v):
    return v.float().to(BF)


# one token to long calls; tile borders and one to each side; rests of the row
# in blocks of 128
SHAPES = [(1, 1, 16), (1, 128, 128), (2, 130, 144), (15, 127, 256), (16, 129, 272), (17, 256, 512),
          (32, 300, 528), (33, 257, 1024), (63, 255, 640), (64, 384, 1040), (65, 100, 2048),
          (100, 1000, 2064), (127, 256, 80), (128, 512, 4096), (129, 640, 384), (191, 255, 768),
          (193, 511, 896), (225, 513, 1312), (255, 385, 496), (257, 768, 256), (448, 1024, 160),
          (600, 1030, 608), (1000, 300, 1024)]


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("T,N,H", SHAPES)
def test_product_exact(dev, ctxs, which, T, N, H):
    a, b = whole(dev, (T, H), T), whole(dev, (N, H), N + 1, 128)
    got = farn.fp8_matmul(*a, *b, ctx=ctxs[which])
    want = values(*a) @ values(*b, 128).t()
    torch.cuda.synchronize()
    assert farn.farn_device_status(ctxs[which].handle) == 0
    assert torch.equal(got, to_bf16(want))


@pytest.mark.parametrize("which", ["auto", "generic"])
@pytest.mark.parametrize("T,N,H", [(3, 33, 9), (70, 64, 15), (1, 10, 1), (130, 100, 1001),
                                   (65, 129, 127)])
def test_product_any_row_length(dev, ctxs, which, T, N, H):
    a, b = whole(dev, (T, H), T), whole(dev, (N, H), N + 1, 128)
    got = farn.fp8_matmul(*a, *b, ctx=ctxs[which])
    assert torch.equal(got, to_bf16(values(*a) @ values(*b, 128).t()))


def tolerance(want, mag, H):
    """Products of codes are exact in fp32.  Every addition within a block is off
    by at most a step of fp32 (2^-23 of a partial sum, which the magnitudes
    bound; truncation counts a whole step), 128 of them; the factor, its
    product with the block's sum and the addition by half a step each, for
    each block; the rounding to bf16 by 2^-8 of the value."""
    acc = (128 + 2 * (-(-H // 128)) + 2) * 2.0 ** -23 * mag
    return 2.0 ** -8 * (want.abs() + acc) + acc


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("T,N,H", [(1, 512, 8192), (20, 300, 4096), (130, 260, 5120),
                                   (520, 300, 2064)])
def test_product_rounding(dev, ctxs, which, T, N, H):
    a, b = spread(dev, (T, H), 5), spread(dev, (N, H), 6, 128)
    got = farn.fp8_matmul(*a, *b, ctx=ctxs[which])
    va, vb = values(*a), values(*b, 128)
    want = va @ vb.t()
    assert ((got.double() - want).abs() <= tolerance(want, va.abs() @ vb.abs().t(), H)).all()


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("T", [3, 70, 300])
def test_product_special_values_stay_with_their_row(dev, ctxs, which, T):
    N, H = 200, 512
    a, b = whole(dev, (T, H), 7), whole(dev, (N, H), 8, 128)
    want = to_bf16(values(*a) @ values(*b, 128).t())
    a[0][1, 3] = 0x7F                       # a NaN code
    if T > 3:
        a[1][T - 1, 2] = float("inf")       # an infinite scale
        a[1][T - 2, 0] = float("nan")
    got = farn.fp8_matmul(*a, *b, ctx=ctxs[which])
    assert torch.isnan(got[1]).all()
    keep = torch.arange(T, device=dev) != 1
    if T > 3:
        assert torch.isnan(got[T - 2]).all() and not torch.isfinite(got[T - 1]).any()
        keep[T - 2:] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("T", [2, 40, 500])
def test_product_any_alignment_and_nothing_behind(dev, ctxs, T):
    N, H = 70, 512
    for d in (0, 1, 4, 16):
        a0, b = whole(dev, (T, H), 9), whole(dev, (N, H), 10, 128)
        qb = torch.zeros(T * H + 16, dtype=torch.uint8, device=dev)
        sb = torch.zeros(T * 4 + 16, device=dev)
        q, s = qb[d:d + T * H].view(T, H), sb[d:d + T * 4].view(T, 4)
        q.copy_(a0[0]), s.copy_(a0[1])
        buf = torch.full((T * N + 32,), 7.0, dtype=BF, device=dev)
        out = buf[d:d + T * N].view(T, N)
        farn.fp8_matmul(q, s, *b, out=out, ctx=ctxs["auto"])
        assert torch.equal(out, to_bf16(values(*a0) @ values(*b, 128).t()))
        assert (buf[:d] == 7.0).all() and (buf[d + T * N:] == 7.0).all()


@pytest.mark.parametrize("which", ["pair", "one", "split4"])
@pytest.mark.parametrize("N", [64, 68, 71])
def test_product_rows_of_every_store_width(dev, ctxs, which, N):
    """Output rows of whole 16 and 8 bytes, and neither."""
    T, H = 300, 256
    a, b = whole(dev, (T, H), 11), whole(dev, (N, H), 12, 128)
    assert torch.equal(farn.fp8_matmul(*a, *b, ctx=ctxs[which]),
                       to_bf16(values(*a) @ values(*b, 128).t()))


@pytest.mark.parametrize("which", ["pair", "one"])
def test_product_beyond_4_gib(dev, ctxs, which):
    """Output rows whose byte offsets pass 32 bits."""
    T, N, H = 70001, 32776, 64
    a, b = whole(dev, (T, H), 17), whole(dev, (N, H), 18, 128)
    got = farn.fp8_matmul(*a, *b, ctx=ctxs[which])
    some = torch.tensor([0, 65535, 65536, 69999, 70000], device=dev)
    want = values(a[0][some], a[1][some]) @ values(*b, 128).t()
    assert torch.equal(got[some], to_bf16(want))
    del got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("which", ALL)
def test_product_same_bits_twice(dev, ctxs, which):
    a, b = spread(dev, (333, 2064), 13), spread(dev, (700, 2064), 14, 128)
    first = farn.fp8_matmul(*a, *b, ctx=ctxs[which])
    for _ in range(3):
        assert torch.equal(farn.fp8_matmul(*a, *b, ctx=ctxs[which]), first)


def test_product_plans(dev, ctxs):
    a = 1 << 32

    def plan(T, N, H, codes=a, which="auto"):
        return farn.farn_plan_fp8_matmul(ctxs[which].handle, codes, 2 * a, T, N, H, 3 * a)[:2]
    assert plan(1, 8192, 8192) == ("tensor", 2)
    assert plan(1, 10240, 5120) == ("tensor", 1)
    assert plan(100, 8192, 8192) == ("tensor", 1)
    assert plan(128, 10240, 5120) == ("pair", 2)
    assert plan(8192, 8192, 8192) == ("pair", 2)
    assert plan(64, 512, 1000) == ("generic", 1)
    assert plan(64, 512, 1024, codes=a + 8) == ("generic", 1)
    assert plan(64, 512, 1024, which="generic") == ("generic", 1)
    assert plan(64, 512, 1024, which="split2") == ("tensor", 2)

    def grouped(S, E, N, H, rows=0, workspace=0, which="auto"):
        return farn.farn_plan_fp8_grouped_matmul(ctxs[which].handle, a, S, rows, S, 2 * a, E, N, H,
                                                 3 * a, workspace)[:2]
    assert grouped(32768, 64, 4096, 7168) == ("pair", 2)
    assert grouped(32768, 64, 4096, 7168, rows=4 * a, workspace=5 * a) == ("pair", 2)
    assert grouped(32768, 64, 4096, 7168, rows=4 * a) == ("tensor", 1)
    assert grouped(512, 64, 7168, 2048) == ("tensor", 1)
    assert grouped(64, 1024, 512, 1024, rows=4 * a, which="split4") == ("tensor", 4)
    h = ctxs["auto"].handle
    assert farn.farn_fp8_grouped_workspace(h, 32768, 64, 4096, 7168) == 32768 * (7168 + 4 * 56)
    assert farn.farn_fp8_grouped_workspace(h, 512, 64, 7168, 2048) == 0


# --------------------------------------------------------------- by expert
GROUPS = [([5], 128, 128), ([1, 0, 3], 72, 528), ([0, 0, 70], 264, 272), ([64, 65, 1], 130, 1024),
          ([300, 20], 264, 2064), ([128, 0, 256, 257], 513, 400), ([0, 0, 0], 64, 64),
          ([40] * 9, 300, 640), ([700, 3, 90, 0, 255], 384, 1040)]


def group_inputs(dev, counts, N, H, gather, make, seed):
    S = sum(counts)
    offsets = torch.zeros(len(counts) + 1, dtype=torch.int32, device=dev)
    offsets[1:] = torch.tensor(counts, device=dev).cumsum(0)
    n = max(1, S // 2 + 3) if gather else S
    x = make(dev, (n, H), seed)
    w = make(dev, (len(counts), N, H), seed + 1, 128)
    rows = torch.randint(0, n, (S,), device=dev, generator=gen(dev, seed + 2),
                         dtype=torch.int32) if gather else None
    return x, w, offsets, rows, S


def group_reference(x, w, offsets, rows, S):
    vx, off = values(*x), offsets.tolist()
    want = torch.zeros(S, w[0].shape[1], device=vx.device, dtype=torch.float64)
    mag = torch.zeros_like(want)
    n = vx.shape[0]
    at = torch.arange(S, device=vx.device) if rows is None else rows.long()
    live = (at >= 0) & (at < n)
    for e in range(len(off) - 1):
        if off[e + 1] > off[e]:
            part = slice(off[e], off[e + 1])
            we = values(w[0][e], w[1][e], 128)
            xe = vx[at[part].clamp(0, n - 1)]
            want[part], mag[part] = xe @ we.t(), xe.abs() @ we.abs().t()
    want[~live] = 0.0
    mag[~live] = 0.0
    return want, mag


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,N,H", GROUPS)
def test_grouped_exact(dev, ctxs, which, gather, counts, N, H):
    x, w, offsets, rows, S = group_inputs(dev, counts, N, H, gather, whole, sum(counts) + N)
    got = farn.fp8_grouped_matmul(*x, *w, offsets, rows, ctx=ctxs[which])
    want, _ = group_reference(x, w, offsets, rows, S)
    torch.cuda.synchronize()
    assert farn.farn_device_status(ctxs[which].handle) == 0
    assert torch.equal(got, to_bf16(want))


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_rounding(dev, ctxs, which, gather):
    x, w, offsets, rows, S = group_inputs(dev, [300, 0, 45, 7], 264, 2064, gather, spread, 40)
    got = farn.fp8_grouped_matmul(*x, *w, offsets, rows, ctx=ctxs[which])
    want, mag = group_reference(x, w, offsets, rows, S)
    assert ((got.double() - want).abs() <= tolerance(want, mag, 2064)).all()


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("per", [3, 90, 300])
def test_grouped_rows_that_do_not_exist(dev, ctxs, which, per):
    """Their slots are zeros, whatever the weights and scales hold, and the
    slots next to them are not touched."""
    counts, N, H = [per, 0, per + 1], 136, 400
    x, w, offsets, rows, S = group_inputs(dev, counts, N, H, True, whole, 50 + per)
    n = x[0].shape[0]
    rows[0], rows[per - 1], rows[S - 1] = -1, n, -2 ** 31
    rows[1] = 2 ** 31 - 1
    want, _ = group_reference(x, w, offsets, rows, S)
    w[0][0, 5, 7] = 0x7F                    # NaN code and scale of weights
    w[1][0, 1, 2] = float("inf")
    got = farn.fp8_grouped_matmul(*x, *w, offsets, rows, ctx=ctxs[which])
    dead = torch.tensor([s for s in {0, 1, per - 1, S - 1}], device=dev)
    assert (got[dead] == 0).all()
    fine = torch.ones(S, N, dtype=torch.bool, device=dev)
    fine[:per, 5] = False
    fine[:per, 128:] = False
    assert torch.equal(got[fine], to_bf16(want)[fine])


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_slots_without_an_expert_are_left(dev, ctxs, which, gather):
    counts, N, H = [40, 200, 30], 100, 256
    x, w, offsets, rows, S = group_inputs(dev, counts, N, H, gather, whole, 60)
    offsets = torch.tensor([7, 40, 210, 250], dtype=torch.int32, device=dev)
    out = torch.full((S, N), 5.0, dtype=BF, device=dev)
    farn.fp8_grouped_matmul(*x, *w, offsets, rows, out=out, ctx=ctxs[which])
    want, _ = group_reference(x, w, offsets, rows, S)
    assert (out[:7] == 5.0).all() and (out[250:] == 5.0).all()
    assert torch.equal(out[7:250], to_bf16(want)[7:250])


def test_grouped_offsets_out_of_range_stay_inside(dev, ctxs):
    N, H, S = 64, 128, 50
    x, w = whole(dev, (S, H), 61), whole(dev, (4, N, H), 62, 128)
    buf = torch.full((S * N + 128,), 3.0, dtype=BF, device=dev)
    out = buf[64:64 + S * N].view(S, N)
    for off in ([-5, 10, 3, 70, 2 ** 31 - 1], [60, -1, 60, 5, 9], [0, 50, 20, 50, 10]):
        o = torch.tensor(off, dtype=torch.int32, device=dev)
        for which in ALL:
            farn.fp8_grouped_matmul(*x, *w, o, out=out, ctx=ctxs[which])
    torch.cuda.synchronize()
    assert (buf[:64] == 3.0).all() and (buf[64 + S * N:] == 3.0).all()


@pytest.mark.parametrize("which", ["auto", "pair", "one", "split2"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_many_experts(dev, ctxs, which, gather):
    counts = [(e * 7) % 5 for e in range(1024)]
    x, w, offsets, rows, S = group_inputs(dev, counts, 130, 144, gather, whole, 63)
    got = farn.fp8_grouped_matmul(*x, *w, offsets, rows, ctx=ctxs[which])
    want, _ = group_reference(x, w, offsets, rows, S)
    assert torch.equal(got, to_bf16(want))


def test_grouped_workspaces(dev, ctxs):
    """A given workspace, one that is too small or not aligned, and none give
    the same bits; nothing behind it is written."""
    counts, N, H = [300, 500, 90], 256, 400
    x, w, offsets, rows, S = group_inputs(dev, counts, N, H, True, whole, 64)
    c = ctxs["pair"]
    need = farn.farn_fp8_grouped_workspace(c.handle, S, len(counts), N, H)
    assert need == S * H + S * 4 * 4
    want, _ = group_reference(x, w, offsets, rows, S)
    buf = torch.full((need + 64,), 77, dtype=torch.uint8, device=dev)
    for ws in (buf[16:16 + need], buf[16:15 + need], buf[17:17 + need], buf[:0]):
        out = torch.zeros(S, N, dtype=BF, device=dev)
        farn.fp8_grouped_matmul(*x, *w, offsets, rows, out=out, workspace=ws, ctx=c)
        assert torch.equal(out, to_bf16(want))
    assert (buf[:16] == 77).all() and (buf[16 + need:] == 77).all()


def test_workspace_of_a_side_stream(dev, ctxs):
    """A call on another stream takes no memory that the current stream's pending
    work still reads."""
    counts, N, H = [300, 500, 90], 256, 400
    x, w, offsets, rows, S = group_inputs(dev, counts, N, H, True, whole, 66)
    c, side = ctxs["pair"], torch.cuda.Stream()
    need = farn.farn_fp8_grouped_workspace(c.handle, S, len(counts), N, H)
    out = torch.empty(S, N, dtype=BF, device=dev)
    kept = torch.empty(need, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    before = torch.full((need,), 77, dtype=torch.uint8, device=dev)
    torch.cuda._sleep(100_000_000)
    kept.copy_(before)
    del before                                   # its block is free for the current stream
    farn.fp8_grouped_matmul(*x, *w, offsets, rows, out=out, ctx=c, stream=side)
    torch.cuda.synchronize()
    assert (kept == 77).all()
    want, _ = group_reference(x, w, offsets, rows, S)
    assert torch.equal(out, to_bf16(want))


@pytest.mark.parametrize("which", ALL)
def test_grouped_without_rows_of_x(dev, ctxs, which):
    """x without rows: every slot's row is missing."""
    w = whole(dev, (2, 40, 128), 65, 128)
    x = torch.zeros(0, 128, dtype=torch.uint8, device=dev), torch.zeros(0, 1, device=dev)
    offsets = torch.tensor([0, 2, 5], dtype=torch.int32, device=dev)
    rows = torch.tensor([0, 1, -1, 5, 0], dtype=torch.int32, device=dev)
    assert (farn.fp8_grouped_matmul(*x, *w, offsets, rows, ctx=ctxs[which]) == 0).all()
    none = torch.zeros(0, dtype=torch.int32, device=dev)
    assert farn.fp8_grouped_matmul(*x, *w, offsets, none, ctx=ctxs[which]).shape == (0, 40)


def test_empty_product(dev):
    b = whole(dev, (8, 256), 1, 128)
    a = torch.zeros(0, 256, dtype=torch.uint8, device=dev), torch.zeros(0, 2, device=dev)
    assert farn.fp8_matmul(*a, *b).shape == (0, 8)


# ------------------------------------------------------- waits, graphs, streams
@pytest.mark.parametrize("env", [dict(FARN_TC_TILE=256), dict(FARN_TC_TILE=64, FARN_TC_SPLIT=1),
                                 dict(FARN_TC_TILE=64, FARN_TC_SPLIT=4)])
@pytest.mark.parametrize("gather", [False, True])
def test_waits_are_bounded(dev, env, gather):
    """With FARN_FAULT_INJECT=stall the first CTA's weights never come: its
    waits and those of the CTAs that work with it run out (2 s, not several
    times), the call ends and the status word says so.  Others are unharmed."""
    ctx = make_ctx(FARN_FAULT_INJECT="stall", **env)
    x, w, offsets, rows, S = group_inputs(dev, [70, 300], 512, 1024, gather, whole, 70)
    torch.cuda.synchronize()
    t0 = time.monotonic()
    farn.fp8_grouped_matmul(*x, *w, offsets, rows, ctx=ctx)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 3.5
    assert farn.farn_device_status(ctx.handle) & (16 | 32 | 64 | 128)
    assert farn.farn_device_status(ctx.handle) == 0
    ctx.close()
    want, _ = group_reference(x, w, offsets, rows, S)
    assert torch.equal(farn.fp8_grouped_matmul(*x, *w, offsets, rows), to_bf16(want))


def fp8_layer(x, logits, up, down, res, weight, K):
    """An expert layer in 8 bits: both products on quantised rows."""
    _, _, index, rows, offsets = r = farn.moe_route(logits, K)
    xq, xs = farn.fp8_quantize(x)
    h = torch.relu(farn.fp8_grouped_matmul(xq, xs, *up, offsets, rows))
    hq, hs = farn.fp8_quantize(h)
    y = farn.fp8_grouped_matmul(hq, hs, *down, offsets)
    return (xq, xs, h, hq, hs, y, *r, *farn.moe_combine(y, index, r[1], res, weight, 1e-6))


def layer_inputs(dev, T, E, H, F, seed):
    r = lambda *s: torch.randn(*s, device=dev, generator=gen(dev, seed + len(s) + s[-1]))  # noqa: E731
    x, res, w = r(T, H).to(BF), r(T, H).to(BF) * 0.5, (1 + 0.1 * r(H)).to(BF)
    up = farn.fp8_quantize((r(E, F, H) * H ** -0.5).to(BF), 128)
    down = farn.fp8_quantize((r(E, H, F) * F ** -0.5).to(BF), 128)
    return x, 2 * r(T, E), up, down, res, w


@pytest.mark.parametrize("T", [1, 20, 700])
def test_expert_layer(dev, T):
    """Router, quantisation, products and combine in a row: each product
    against the 64-bit product of the codes that it was given."""
    K, E, H, F = 3, 9, 256, 336
    x, logits, up, down, res, w = layer_inputs(dev, T, E, H, F, 80 + T)
    if T > 1:
        logits[T // 2] = float("-inf")
    xq, xs, h, hq, hs, y, experts, gates, index, rows, offsets, red, ro, nrm = fp8_layer(
        x, logits, up, down, res, w, K)
    check_quantized((xq, xs), x, 1)
    n = int(offsets[-1])
    want, mag = group_reference((xq, xs), up, offsets, rows[:n], n)
    assert ((h[:n].double() - want.relu()).abs() <= tolerance(want, mag, H)).all()
    check_quantized((hq[:n], hs[:n]), h[:n], 1)
    want, mag = group_reference((hq, hs), down, offsets, None, n)
    assert ((y[:n].double() - want).abs() <= tolerance(want, mag, F)).all()
    acc = torch.zeros(T, H, device=dev)
    for k in range(K):
        live = index[:, k] >= 0
        acc[live] += gates[live, k, None] * y[index[live, k].long()].float()
    assert torch.equal(red, acc.to(BF)) or \
        ((red.float() - acc).abs() <= 2.0 ** -7 * acc.abs() + 2.0 ** -20).all()
    if T > 1:
        assert torch.equal(ro[T // 2], res[T // 2])


def test_layer_in_graphs_and_on_streams(dev):
    """Captured twice and both graphs replayed at once on new inputs, and run on
    two streams: the same bits as eager calls."""
    x, logits, up, down, res, w = layer_inputs(dev, 400, 8, 512, 384, 90)
    other = layer_inputs(dev, 400, 8, 512, 384, 91)
    ins = [(x, logits, up, down, res, w), (other[0], other[1], up, down, other[4], w)]
    eager = [[t.clone() for t in fp8_layer(*i, 4)] for i in ins]
    assert int(eager[0][10][-1]) == 1600
    graphs, outs = [], []
    for i in (1, 0):                        # captured on the other inputs
        static = [ins[i][0].clone(), ins[i][1].clone(), up, down, ins[i][4].clone(), w]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fp8_layer(*static, 4)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fp8_layer(*static, 4))
        for k in (0, 1, 4):
            static[k].copy_(ins[1 - i][k])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, e in zip(outs, eager):
        assert all(torch.equal(p, q) for p, q in zip(o, e))
    results = []
    for _ in range(3):
        for s, i in zip(streams, ins):
            with torch.cuda.stream(s):
                results.append(fp8_layer(*i, 4))
    torch.cuda.synchronize()
    for n, r in enumerate(results):
        assert all(torch.equal(p, q) for p, q in zip(r, eager[n % 2]))


def test_prepared_calls_reuse_their_buffers(dev):
    T, H, N = 300, 512, 144
    x, w = normal(dev, (T, H), 31), normal(dev, (N, H), 32)
    wq = farn.fp8_quantize(w, 128)
    quantize = farn.prepare_fp8_quantize(x)
    given = torch.empty(T, N, dtype=BF, device=dev)
    product = farn.prepare_fp8_matmul(*quantize.outputs, *wq, out=given)
    offsets = torch.tensor([0, 100, T], dtype=torch.int32, device=dev)
    w2 = farn.fp8_quantize(normal(dev, (2, N, H), 33), 128)
    rows = torch.arange(T, dtype=torch.int32, device=dev).flip(0).contiguous()
    c = make_ctx(FARN_TC_TILE=256)
    grouped = farn.prepare_fp8_grouped_matmul(*quantize.outputs, *w2, offsets, rows, ctx=c)
    for seed in (34, 35):
        x.copy_(normal(dev, (T, H), seed))
        quantize()
        q, s = farn.fp8_quantize(x)
        assert torch.equal(quantize.outputs[0], q) and torch.equal(quantize.outputs[1], s)
        assert product() is given
        assert torch.equal(given, farn.fp8_matmul(q, s, *wq))
        assert torch.equal(grouped(), farn.fp8_grouped_matmul(q, s, *w2, offsets, rows, ctx=c))
    c.close()


@pytest.mark.parametrize("prepared", [False, True])
def test_calls_on_a_given_stream(dev, prepared):
    """The calls run on the stream that they are given, behind what it has to
    do first, while the current stream stays idle."""
    T, H, N = 200, 512, 144
    x = normal(dev, (T, H), 36)
    w = farn.fp8_quantize(normal(dev, (2, N, H), 37), 128)
    offsets = torch.tensor([0, 120, T], dtype=torch.int32, device=dev)
    rows = torch.arange(T, dtype=torch.int32, device=dev).flip(0).contiguous()
    c = make_ctx(FARN_TC_TILE=256)
    q0, s0 = farn.fp8_quantize(x)
    want = farn.fp8_matmul(q0, s0, w[0][0], w[1][0]), \
        farn.fp8_grouped_matmul(q0, s0, *w, offsets, rows, ctx=c)
    late, q, s = torch.zeros_like(x), torch.empty_like(q0), torch.empty_like(s0)
    y = [torch.empty_like(t) for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pick = (lambda name: getattr(farn, "prepare_" + name)) if prepared else \
        (lambda name: lambda *a, **k: lambda: getattr(farn, name)(*a, **k))
    calls = [pick("fp8_quantize")(late, out=(q, s), stream=side),
             pick("fp8_matmul")(q, s, w[0][0], w[1][0], out=y[0], stream=side),
             pick("fp8_grouped_matmul")(q, s, *w, offsets, rows, out=y[1], ctx=c, stream=side)]
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        late.copy_(x)
    for call in calls:
        call()
    assert torch.cuda.current_stream().query() and not side.query()
    side.synchronize()
    assert torch.equal(q, q0) and torch.equal(s, s0)
    assert all(torch.equal(a, b) for a, b in zip(y, want))
    c.close()


def test_two_threads_with_one_context(dev):
    import threading
    ins = [layer_inputs(dev, 40 + 300 * i, 8, 256, 512, 51 + i) for i in range(2)]
    want = [[t.clone() for t in fp8_layer(*i, 2)] for i in ins]
    torch.cuda.synchronize()
    bad = []

    def work(n):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = fp8_layer(*ins[n], 2)
                s.synchronize()
                if not all(torch.equal(g, w) for g, w in zip(got, want[n])):
                    bad.append(n)
    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_contexts_that_cannot_serve(dev):
    """Set-up of the tensor-core kernels that failed: the slower kernel, the same
    exact values.  Launches that fail, and contexts of another device: errors."""
    a, b = whole(dev, (40, 256), 1), whole(dev, (72, 256), 2, 128)
    ctx = make_ctx(FARN_FAULT_INJECT="setup")
    assert farn.farn_plan_fp8_matmul(ctx.handle, 1 << 32, 1 << 33, 40, 72, 256,
                                     1 << 34)[0] == "generic"
    assert farn.farn_fp8_grouped_workspace(ctx.handle, 32768, 64, 4096, 7168) == 0
    assert torch.equal(farn.fp8_matmul(*a, *b, ctx=ctx), farn.fp8_matmul(*a, *b))
    ctx.close()
    bad = make_ctx(FARN_FAULT_INJECT="launch")
    other = farn.Context(0)
    other.device = 1
    x = normal(dev, (4, 64), 1)
    off = torch.tensor([0, 40], dtype=torch.int32, device=dev)
    for call in (lambda c: farn.fp8_quantize(x, ctx=c), lambda c: farn.fp8_matmul(*a, *b, ctx=c),
                 lambda c: farn.fp8_grouped_matmul(*a, b[0][None], b[1][None], off, ctx=c)):
        with pytest.raises(farn.FarnError) as e:
            call(bad)
        assert e.value.status == farn.FARN_ERR_CUDA
        with pytest.raises(ValueError, match="device"):
            call(other)
