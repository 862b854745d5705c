"""Norms and rotations of query and key heads and the quantised paged cache on
the GPU, against plain 64-bit definitions."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import rank_sum_residual_gb300 as farn  # noqa: E402
from gpu_util import make_ctx  # noqa: E402
from parity import u16  # noqa: E402

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32
G = (168.0, 40.0)


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
    return {"auto": farn.Context(0), "generic": make_ctx(FARN_VARIANT="generic")}


BOTH = ["auto", "generic"]


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def normal(dev, shape, seed):
    return torch.randn(shape, device=dev, generator=gen(dev, seed)).to(BF)


def weights(dev, D, seed):
    return (1 + 0.1 * torch.randn(D, device=dev, generator=gen(dev, seed))).to(BF)


def freqs_of(dev, R, base=1e6):
    half = R // 2
    return (base ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)).float()


def heads_reference(x, w, eps, positions, freqs, sections, interleaved):
    """In 64 bits; also what the roundings of fp32 are relative to: the
    magnitudes of what a pair's element is the sum of."""
    y = x.double()
    D = y.shape[2]
    if w is not None:
        y = y / ((y * y).sum(dim=2, keepdim=True) / D + eps).sqrt() * w.double()
    mag = y.abs()
    if freqs is None:
        return y, mag
    half = freqs.shape[0]
    p = positions if positions.dim() == 2 else positions[None]
    axis = [a for a, n in enumerate(sections or [half]) for _ in range(n)]
    angle = torch.stack([p[a].double() * freqs[i].double() for i, a in enumerate(axis)], dim=1)
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    j = torch.arange(half, device=x.device)
    ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    a, b = y[..., ia], y[..., ib]
    y, mag = y.clone(), mag.clone()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


# In fp32: the sum of squares of D <= 1024 values, its mean and root (an
# approximate one of 2 ulp), two products: (D / 32 + 5 + 8) half steps at most
# for the trees used here; sine and cosine: the angle's place in the turn to
# 2^-31 turns (and rounded to fp32, half a step of at most half a turn: pi *
# 2^-25) and the functions themselves 2 ulp: 2^-22; the rotation: two products and
# a sum, half a step each.  Together below 64 * 2^-24 = 2^-18 of the magnitudes.
F32 = 2.0 ** -18


def check_heads(got, want, mag):
    """One rounding to bf16: half a step, 2^-8 of the value."""
    tol = F32 * mag + 2.0 ** -8 * (want.abs() + F32 * mag)
    # below the smallest normal a step is absolute
    assert ((got.double() - want).abs() <= tol + 2.0 ** -134).all()


# T, HQ, HK, D, R, axes, interleaved
CASES = [
    (1, 1, 1, 64, 64, 1, False), (1, 32, 8, 128, 128, 1, False), (5, 7, 1, 128, 64, 1, True),
    (3, 2, 2, 8, 8, 1, False), (4, 3, 1, 16, 2, 1, True), (9, 4, 2, 80, 80, 1, False),
    (70, 6, 3, 80, 64, 3, True), (33, 5, 5, 96, 48, 2, False), (300, 4, 1, 192, 192, 1, False),
    (17, 3, 3, 256, 128, 4, False), (2, 10, 2, 256, 256, 2, True), (513, 2, 0, 72, 24, 1, False),
    (40, 0, 3, 128, 32, 3, False), (6, 2, 1, 128, 0, 1, False),
    # for the kernel of any size
    (7, 3, 2, 10, 10, 1, False), (3, 2, 1, 1, 0, 1, False), (11, 2, 2, 33, 12, 2, True),
    (5, 2, 1, 100, 90, 3, False), (4, 1, 1, 1024, 1024, 1, False), (3, 2, 1, 300, 4, 1, True),
]


def sections_of(R, axes):
    if axes == 1:
        return None
    part = R // 2 // axes
    return [R // 2 - part * (axes - 1)] + [part] * (axes - 1)


def case_inputs(dev, T, HQ, HK, D, R, axes, seed, far=5000):
    q, k = normal(dev, (T, HQ, D), seed), normal(dev, (T, HK, D), seed + 1)
    pos = torch.randint(-far, far, (axes, T), device=dev, generator=gen(dev, seed + 2), dtype=I32)
    return (q, k, weights(dev, D, seed + 3), weights(dev, D, seed + 4),
            pos[0].contiguous() if axes == 1 else pos, freqs_of(dev, R) if R else None,
            sections_of(R, axes))


@pytest.mark.parametrize("which", BOTH)
@pytest.mark.parametrize("T,HQ,HK,D,R,axes,interleaved", CASES)
def test_heads(dev, ctxs, which, T, HQ, HK, D, R, axes, interleaved):
    q, k, wq, wk, pos, fr, sect = case_inputs(dev, T, HQ, HK, D, R, axes, T + D)
    eps = 1e-5
    got = farn.qk_norm_rope(q, k, wq, wk, eps, pos, fr, sect, interleaved, ctx=ctxs[which])
    for x, w, y in zip((q, k), (wq, wk), got):
        check_heads(y, *heads_reference(x, w, eps, pos, fr, sect, interleaved))


def same_bits(a, b):
    """Equal bits, but for NaN, whose payload no conversion keeps."""
    a, b = a.contiguous(), b.contiguous()
    nan = torch.isnan(b)
    return torch.equal(torch.isnan(a), nan) and \
        torch.equal(a.view(torch.int16)[~nan], b.view(torch.int16)[~nan])


@pytest.mark.parametrize("which", BOTH)
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_without_norms(dev, ctxs, which, interleaved):
    """A weight of None leaves that side's values as they are but for the
    rotation; both None and no rotation copy the bits, infinities too."""
    q, k, wq, wk, pos, fr, _ = case_inputs(dev, 50, 4, 2, 128, 64, 1, 7)
    a, b = farn.qk_norm_rope(q, k, None, wk, 1e-6, pos, fr, None, interleaved, ctx=ctxs[which])
    check_heads(a, *heads_reference(q, None, 1e-6, pos, fr, None, interleaved))
    check_heads(b, *heads_reference(k, wk, 1e-6, pos, fr, None, interleaved))
    q[3, 1, 70] = float("inf")
    q[3, 1, 71] = float("nan")
    a, b = farn.qk_norm_rope(q, k, None, None, 0.0, ctx=ctxs[which])
    assert same_bits(a, q) and same_bits(b, k)
    # what lies behind the rotated part is not touched by it
    a, _ = farn.qk_norm_rope(q, k, None, None, 0.0, pos, fr, ctx=ctxs[which])
    assert same_bits(a[..., 64:], q[..., 64:])


@pytest.mark.parametrize("which", BOTH)
def test_far_positions(dev, ctxs, which):
    """Positions up to the ends of 32 bits, frequencies from far below one to
    2^8 radians per position: fp32 angles would be off by whole turns."""
    T, D = 64, 128
    q, k, wq, wk, _, _, _ = case_inputs(dev, T, 2, 1, D, D, 1, 9)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), device=dev, generator=gen(dev, 10), dtype=I32)
    pos[:6] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6], dtype=I32)
    fr = torch.exp2(torch.linspace(-40, 8, 64, device=dev))
    fr[1], fr[2], fr[3] = 0.0, -0.37, 1e-30
    got = farn.qk_norm_rope(q, k, wq, wk, 1e-6, pos, fr, ctx=ctxs[which])
    # pos * freq is exact in 64 bits (31 + 24 bits, two of which may round); the
    # reference's own turn reduction is the library's
    for x, w, y in zip((q, k), (wq, wk), got):
        want, mag = heads_reference(x, w, 1e-6, pos, fr, None, False)
        # 2^8 radians * 2^31 positions: the reference's angle is off by 2^-53 of
        # 2^39, 2^-14; its share of the magnitudes
        angle = (pos.double()[:, None] * fr.double()).abs() * 2.0 ** -53
        slack = torch.cat((angle, angle), dim=1)[:, None] * mag
        tol = F32 * mag + slack + 2.0 ** -8 * (want.abs() + F32 * mag + slack)
        assert ((y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("which", BOTH)
def test_zero_rows_and_special_values_stay_in_their_head(dev, ctxs, which):
    T, H, D = 6, 4, 128
    q, k, wq, wk, pos, fr, _ = case_inputs(dev, T, H, H, D, D, 1, 11)
    q[0, 0] = 0.0                               # 0 with eps
    q[1, 1] = 0.0
    q[1, 1, 5] = 3e38                           # the squares overflow: 0
    q[2, 2, 7] = float("nan")
    q[3, 3, 9] = float("inf")
    a, _ = farn.qk_norm_rope(q, k, wq, wk, 1e-6, pos, fr, ctx=ctxs[which])
    assert (a[0, 0] == 0).all() and (a[1, 1] == 0).all()
    assert torch.isnan(a[2, 2]).all()
    assert torch.isnan(a[3, 3, 9])
    keep = torch.ones(T, H, dtype=torch.bool, device=dev)
    keep[2, 2] = keep[3, 3] = keep[1, 1] = False
    want, mag = heads_reference(q, wq, 1e-6, pos, fr, None, False)
    check_heads(a[keep], want[keep], mag[keep])


@pytest.mark.parametrize("which", BOTH)
@pytest.mark.parametrize("D,pad", [(128, 0), (64, 8), (80, 3), (128, 1)])
def test_packed_projection_in_place(dev, ctxs, which, D, pad):
    """Heads read where a projection of queries, keys and values wrote them, and
    written back there; the values and what lies between stay as they were."""
    T, HQ, HK = 37, 6, 2
    width = (HQ + 2 * HK) * D + pad
    buf = normal(dev, (T * width + 8,), 12)
    for d in (0, 4, 1):
        qkv = buf.clone()[d:d + T * width].view(T, width)
        before = qkv.clone()
        q = qkv[:, :HQ * D].unflatten(1, (HQ, D))
        k = qkv[:, HQ * D:(HQ + HK) * D].unflatten(1, (HK, D))
        _, _, wq, wk, pos, fr, _ = case_inputs(dev, T, HQ, HK, D, D // 2 // 8 * 8, 1, 13)
        want = [heads_reference(x, w, 1e-6, pos, fr, None, False) for x, w in ((q, wq), (k, wk))]
        out = farn.qk_norm_rope(q, k, wq, wk, 1e-6, pos, fr, out=(q, k), ctx=ctxs[which])
        assert out[0] is q and out[1] is k
        for y, w in zip(out, want):
            check_heads(y, *w)
        at = (HQ + HK) * D
        assert torch.equal(qkv[:, at:].contiguous().view(torch.int16),
                           before[:, at:].contiguous().view(torch.int16))


def test_same_as_the_rms_norm(dev):
    """A head of the norm's own: forward of one partial of zeros and a residual
    is the RMSNorm of the residual.  Each side rounds once to bf16."""
    T, D = 50, 256
    x, w = normal(dev, (T, D), 14), weights(dev, D, 15)
    _, _, nrm = farn.forward([torch.zeros_like(x)], x, w, 1e-6)
    y, _ = farn.qk_norm_rope(x[:, None], x[:, None, :].expand(T, 1, D)[:, :0], w, None, 1e-6)
    step = 2.0 ** -7 * nrm.double().abs()
    assert ((y[:, 0].double() - nrm.double()).abs() <= step).all()


# -------------------------------------------------------------------- cache
def empty(dev, fmt, pages, page, H, D):
    """A cache whose every byte shows whether it was written."""
    c = farn.kv_cache(pages, page, H, D, fmt, dev)
    c[0].fill_(0x21), c[1].fill_(0x32)
    c[2].fill_(7.0 if fmt == "fp8" else 0x43), c[3].fill_(9.0 if fmt == "fp8" else 0x44)
    return c


def scales_arg(fmt):
    return None if fmt == "fp8" else G


def row_codes(O, x, fmt, g):
    """Codes and scales of rows [n, D] of fp32 or bf16 values, by the definition."""
    if fmt == "nvfp4":
        q, s = O.quant_nvfp4(u16(x.contiguous()), g)
        return torch.from_numpy(q), torch.from_numpy(s)
    f = x.float().cpu()
    amax = torch.nan_to_num(f.abs(), nan=0.0, posinf=float("inf")).amax(dim=1, keepdim=True)
    top = torch.tensor(448.0)
    s = torch.where(amax > 0, amax / top, 1.0)
    inv = torch.where(amax > 0, (top / amax).clamp(max=torch.finfo(torch.float32).max), 1.0)
    q = (f * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q, s[:, 0]


@pytest.fixture(scope="module")
def O():
    return oracle.Oracle()


@pytest.mark.parametrize("which", BOTH)
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 16, 1), (1, 8, 128, 16), (40, 2, 64, 16),
                                        (100, 3, 80, 7), (33, 4, 96, 64), (5, 1, 256, 16),
                                        (9, 2, 272, 3), (2, 1, 1024, 2)])
def test_write_exact(O, dev, ctxs, which, fmt, T, H, D, page):
    """The bits of what is written, and that nothing else is: slots in any
    order, those outside the cache skipped."""
    pages = -(-(T + 9) // page) + 1
    c = empty(dev, fmt, pages, page, H, D)
    before = [t.clone() for t in c]
    k, v = normal(dev, (T, H, D), 20), normal(dev, (T, H + 2, D), 21)[:, 1:H + 1]
    k[0, 0] = 0.0
    slots = torch.randperm(pages * page, device=dev, generator=gen(dev, 22))[:T].to(I32)
    live = torch.ones(T, dtype=torch.bool, device=dev)
    if T > 4:
        slots[1], slots[2], slots[3] = -1, pages * page, 2 ** 31 - 1
        slots[4] = -2 ** 31
        live[1:5] = False
    assert farn.kv_write(k, v, c, slots, tensor_scales=scales_arg(fmt), ctx=ctxs[which]) is c
    at = slots[live].long()
    for x, codes, scales, b0, b1, g in ((k, c[0], c[2], before[0], before[2], G[0]),
                                        (v, c[1], c[3], before[1], before[3], G[1])):
        q, s = row_codes(O, x[live].reshape(-1, D), fmt, g)
        rows = codes.view(-1, H, codes.shape[-1])
        sc = scales.view(pages * page, H, -1)
        n = int(live.sum())
        assert torch.equal(rows[at].reshape(n * H, -1).cpu(), q.view(n * H, -1))
        assert torch.equal(sc[at].reshape(n * H, -1).cpu(), s.reshape(n * H, -1))
        rest = torch.ones(pages * page, dtype=torch.bool, device=dev)
        rest[at] = False
        assert torch.equal(rows[rest], b0.view_as(rows)[rest])
        assert torch.equal(sc[rest], b1.view_as(sc)[rest])


@pytest.mark.parametrize("which", BOTH)
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_write_special_values(O, dev, ctxs, which, fmt):
    """NaN, infinities and the smallest magnitudes stay with their row or
    block."""
    T, H, D = 8, 2, 64
    k = normal(dev, (T, H, D), 23)
    k[0, 0, 3] = float("nan")
    k[1, 1, 20:22] = torch.tensor([float("inf"), -float("inf")], dtype=BF)
    k[2, 0] = 0.0
    k[2, 0, 5] = 9.2e-41
    k[3, 1, 40] = 3.3e38
    c = empty(dev, fmt, 2, 4, H, D)
    slots = torch.arange(T, device=dev, dtype=I32)
    farn.kv_write(k, k, c, slots, tensor_scales=scales_arg(fmt), ctx=ctxs[which])
    q, s = row_codes(O, k.view(-1, D), fmt, G[0])
    got = c[0].view(T * H, -1).cpu()
    if fmt == "fp8":
        nan = (q & 127) == 127
        assert torch.equal((got & 127) == 127, nan)
        assert torch.equal(got[~nan], q[~nan])
    else:
        assert torch.equal(got, q)
    assert torch.equal(c[2].view(T * H, -1).cpu(), s.reshape(T * H, -1))


def read_values(codes, scales, fmt, g):
    """Rows' values as the definition rounds them, in fp32 then bf16."""
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float() * scales[..., None]
        return v.to(BF)
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                         device=codes.device)
    f = scales.view(torch.float8_e4m3fn).float() / torch.tensor(g, device=codes.device)
    return (table[c.long()] * f.repeat_interleave(16, dim=-1)).to(BF)


def full(dev, fmt, pages, page, H, D, seed):
    """A cache in use: every code, scales over their range."""
    c = farn.kv_cache(pages, page, H, D, fmt, dev)
    g = gen(dev, seed)
    for i in (0, 1):
        c[i].copy_(torch.randint(0, 256, c[i].shape, device=dev, generator=g, dtype=torch.uint8))
        if fmt == "fp8":
            c[i][(c[i] & 127) == 127] = 0
            c[2 + i].copy_(torch.rand(c[2 + i].shape, device=dev, generator=g))
        else:
            c[2 + i].copy_(torch.randint(0, 127, c[2 + i].shape, device=dev, generator=g,
                                         dtype=torch.uint8))
    return c


@pytest.mark.parametrize("which", BOTH)
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("lengths,H,D,page", [
    ([1], 1, 16, 1), ([5], 2, 64, 16), ([0, 7, 0, 33, 16, 0], 1, 32, 16), ([100, 1, 64], 3, 80, 7),
    ([300, 40], 8, 128, 64), ([17] * 40, 2, 96, 5), ([9, 0], 5, 272, 3), ([40], 1, 1024, 16),
    ([2000], 1, 16, 16)])
def test_read(dev, ctxs, which, fmt, lengths, H, D, page):
    """Pages that end within a sequence and behind it, empty sequences, and rows
    before the first sequence and behind the last, which are left."""
    B, width = len(lengths), max(-(-n // page) for n in lengths) + 1
    pages = B * width + 3
    c = full(dev, fmt, pages, page, H, D, 30)
    table = torch.randperm(pages, device=dev, generator=gen(dev, 31))[:B * width].to(I32).view(
        B, width)
    first = 3
    offsets = torch.tensor(np.cumsum([first] + lengths), dtype=I32, device=dev)
    n = int(offsets[-1]) + 2
    out = [torch.full((n, H, D), 5.0, dtype=BF, device=dev) for _ in range(2)]
    farn.kv_read(c, table, offsets, n, tensor_scales=scales_arg(fmt), out=out, ctx=ctxs[which])
    at = torch.cat([table[b].long()[torch.arange(m, device=dev) // page] * page +
                    torch.arange(m, device=dev) % page for b, m in enumerate(lengths)])
    for y, codes, scales, g in ((out[0], c[0], c[2], G[0]), (out[1], c[1], c[3], G[1])):
        want = read_values(codes.flatten(0, 1)[at], scales.flatten(0, 1)[at], fmt, g)
        assert torch.equal(y[first:-2].view(torch.int16), want.view(torch.int16))
        assert (y[:first] == 5.0).all() and (y[-2:] == 5.0).all()


@pytest.mark.parametrize("which", BOTH)
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_read_bad_pages(dev, ctxs, which, fmt):
    """Pages outside the cache and positions behind the table read as zeros;
    offsets that are not ascending lead nowhere outside the tensors."""
    H, D, page = 2, 64, 4
    c = full(dev, fmt, 6, page, H, D, 32)
    table = torch.tensor([[0, -1, 5], [6, 2 ** 31 - 1, 1]], dtype=I32, device=dev)
    offsets = torch.tensor([0, 15, 27], dtype=I32, device=dev)      # 15 > 3 pages of 4
    k, v = farn.kv_read(c, table, offsets, 27, tensor_scales=scales_arg(fmt), ctx=ctxs[which])
    want = read_values(c[0], c[2], fmt, G[0])
    assert torch.equal(k[:4], want[0]) and torch.equal(k[8:12], want[5])
    assert (k[4:8] == 0).all() and (k[12:23] == 0).all() and torch.equal(k[23:27], want[1])
    buf = torch.full((40 * H * D,), 3.0, dtype=BF, device=dev)
    out = buf[5 * H * D:15 * H * D].view(10, H, D), torch.empty(10, H, D, dtype=BF, device=dev)
    for off in ([0, 100, 27], [9, 3, 20], [-7, 4, 2], [2 ** 31 - 1, -5, 8], [20, 30, 40]):
        farn.kv_read(c, table, torch.tensor(off, dtype=I32, device=dev), 10,
                     tensor_scales=scales_arg(fmt), out=out, ctx=ctxs[which])
    torch.cuda.synchronize()
    assert (buf[:5 * H * D] == 3.0).all() and (buf[15 * H * D:] == 3.0).all()
    none = torch.zeros(2, 0, dtype=I32, device=dev)                 # a table without pages
    k, v = farn.kv_read(c, none, offsets, 27, tensor_scales=scales_arg(fmt), ctx=ctxs[which])
    assert (k == 0).all() and (v == 0).all()


def test_empty_calls(dev):
    c = farn.kv_cache(2, 4, 2, 16, "fp8", dev)
    x, none = torch.zeros(0, 2, 16, dtype=BF, device=dev), torch.zeros(0, dtype=I32, device=dev)
    a, b = farn.qk_norm_rope(x, x, None, None, 0.0)
    assert a.shape == b.shape == (0, 2, 16)
    assert farn.qk_norm_rope_cache(x, x, x, None, None, 0.0, None, None, c, none).shape == (0, 2, 16)
    farn.kv_write(x, x, c, none)
    table = torch.zeros(0, 3, dtype=I32, device=dev)
    k, v = farn.kv_read(c, table, torch.zeros(1, dtype=I32, device=dev), 0)
    assert k.shape == v.shape == (0, 2, 16)
    # a cache without pages takes no slot
    e = farn.kv_cache(0, 4, 2, 16, "nvfp4", dev)
    y = torch.ones(3, 2, 16, dtype=BF, device=dev)
    farn.kv_write(y, y, e, torch.arange(3, dtype=I32, device=dev), tensor_scales=G)
    torch.cuda.synchronize()


@pytest.mark.parametrize("which", BOTH)
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_cache_beyond_4_gib(dev, ctxs, which, fmt):
    """Slots whose byte offsets pass 32 bits, written and read back."""
    H, D, page = 64, 1024 if which == "generic" else 256, 16
    rows = (5 << 30) // (H * D if fmt == "fp8" else H * D // 2)
    pages = rows // page
    c = farn.kv_cache(pages, page, H, D, fmt, dev)
    some = [0, pages // 2, pages - 1]
    x = normal(dev, (3, H, D), 33)
    slots = torch.tensor([p * page + 5 for p in some], dtype=I32, device=dev)
    farn.kv_write(x, -x, c, slots, tensor_scales=scales_arg(fmt), ctx=ctxs[which])
    table = torch.tensor([[p] for p in some], dtype=I32, device=dev)
    offsets = torch.tensor([0, 6, 12, 18], dtype=I32, device=dev)
    k, v = farn.kv_read(c, table, offsets, 18, tensor_scales=scales_arg(fmt), ctx=ctxs[which])
    small = farn.kv_cache(3, 1, H, D, fmt, dev)
    farn.kv_write(x, -x, small, torch.arange(3, dtype=I32, device=dev),
                  tensor_scales=scales_arg(fmt))
    assert torch.equal(k[5::6], read_values(small[0], small[2], fmt, G[0])[:, 0])
    assert torch.equal(v[5::6], read_values(small[1], small[3], fmt, G[1])[:, 0])
    assert (k[:5] == 0).all() and (v[12:17] == 0).all()
    del c, k, v
    torch.cuda.empty_cache()


# ------------------------------------------------- heads straight to the cache
@pytest.mark.parametrize("which", BOTH)
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("T,HQ,HK,D,R,axes,interleaved", [
    (1, 32, 8, 128, 128, 1, False), (16, 5, 1, 64, 64, 1, False), (70, 4, 2, 128, 64, 1, False),
    (33, 0, 3, 96, 96, 3, False), (40, 6, 3, 80, 64, 3, True), (300, 2, 2, 256, 256, 2, True),
    (9, 3, 1, 256, 256, 1, False), (7, 2, 1, 272, 32, 1, False), (5, 3, 2, 128, 0, 1, False),
    (11, 1, 2, 48, 48, 1, False)])
def test_heads_to_cache(O, dev, ctxs, which, fmt, T, HQ, HK, D, R, axes, interleaved):
    """Values' bits as kv_write's; keys' codes are those of the 64-bit values or,
    where the roundings of fp32 reach a border between two codes, a neighbour's."""
    q, k, wq, wk, pos, fr, sect = case_inputs(dev, T, HQ, HK, D, R, axes, 40 + T)
    v = normal(dev, (T, HK, D), 41)
    c = empty(dev, fmt, T + 4, 1, HK, D)
    slots = torch.randperm(T + 4, device=dev, generator=gen(dev, 42))[:T].to(I32)
    if T > 8:
        slots[5] = -1
    live = slots >= 0
    got = farn.qk_norm_rope_cache(q, k, v, wq, wk, 1e-5, pos, fr, c, slots, scales_arg(fmt), sect,
                                  interleaved, ctx=ctxs[which])
    check_heads(got, *heads_reference(q, wq, 1e-5, pos, fr, sect, interleaved))
    at = slots[live].long()
    other = empty(dev, fmt, T + 4, 1, HK, D)
    farn.kv_write(k, v, other, slots, tensor_scales=scales_arg(fmt))
    assert torch.equal(c[1], other[1]) and torch.equal(c[3], other[3])
    want, mag = heads_reference(k, wk, 1e-5, pos, fr, sect, interleaved)
    want, mag = want[live], mag[live]
    err = F32 * mag
    codes, scales = c[0][at, 0], c[2][at, 0]
    if fmt == "fp8":
        amax = want.abs().amax(dim=2, keepdim=True)
        off = err.amax(dim=2, keepdim=True)
        # the scale carries the largest value's error and half a step
        assert ((scales.double()[..., None] * 448 - amax).abs() <= off + 2.0 ** -23 * amax).all()
        y = codes.view(torch.float8_e4m3fn).double() * scales.double()[..., None]
        # half a step of E4M3: 2^-4 of the value, or of the smallest normal, of the
        # scaled value, which is off by its own error and the scale's
        size = want.abs() + err + want.abs() * off / amax
        tol = 2.0 ** -4 * torch.maximum(size, scales.double()[..., None] * 2.0 ** -6)
        assert ((y - want).abs() <= tol * (1 + 2.0 ** -20) + err + 2.0 ** -22 * size).all()
    else:
        b = want.unflatten(2, (D // 16, 16))
        amax, off = b.abs().amax(dim=3), err.unflatten(2, (D // 16, 16)).amax(dim=3)
        s = scales.view(torch.float8_e4m3fn).double()
        # E4M3 of amax / 6 * g: half a step, 2^-4, at most 448
        ideal = (amax / 6 * G[0]).clamp(max=448.0)
        tol = 2.0 ** -4 * ideal.clamp(min=2.0 ** -6) + (off / 6 + 2.0 ** -22 * amax / 6) * G[0] * 1.1
        assert ((s - ideal).abs() <= tol).all()
        # given the scale, a code is the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6
        n = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=dev, dtype=torch.float64)
        y = torch.where(n >= 8, -table[n & 7], table[n & 7]).unflatten(2, (D // 16, 16))
        unit = (s / G[0])[..., None]
        x = torch.where(unit > 0, b / unit, 0.0)
        gap = torch.where(x.abs() > 2, torch.where(x.abs() > 4, 1.0, 0.5), 0.25)
        slack = torch.where(unit > 0, err.unflatten(2, (D // 16, 16)) / unit, 0.0) \
            + 2.0 ** -22 * x.abs()
        # beyond 6 it saturates; a value near 2 or 4 may have either gap
        near = torch.where((x.abs() - 2).abs() <= slack, 0.5, torch.where(
            (x.abs() - 4).abs() <= slack, 1.0, gap))
        assert ((y - x.clamp(-6.0, 6.0)).abs() <= near + slack).all()


def attention_step(dev, hidden, qkv_w, o_w, wq, wk, cache, slots, pos, fr, table, offsets, n, HQ,
                   HK, D):
    """A layer's attention half but for the attention itself, which is plain
    torch: projection in 8 bits, norms, rotation and cache, contexts read back,
    projection in 8 bits."""
    T = hidden.shape[0]
    qkv = farn.fp8_matmul(*farn.fp8_quantize(hidden), *qkv_w)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([HQ * D, HK * D, HK * D], dim=1))
    q = farn.qk_norm_rope_cache(q, k, v, wq, wk, 1e-6, pos, fr, cache, slots)
    kk, vv = farn.kv_read(cache, table, offsets, n)
    # every token attends to the whole of the first sequence
    p = torch.einsum("thd,nhd->thn", q.float(), kk.float().repeat_interleave(HQ // HK, dim=1))
    y = torch.einsum("thn,nhd->thd", (p * D ** -0.5).softmax(dim=2),
                     vv.float().repeat_interleave(HQ // HK, dim=1)).to(BF).reshape(T, HQ * D)
    return farn.fp8_matmul(*farn.fp8_quantize(y), *o_w), q, kk, vv


def test_attention_half(dev):
    """The operators in a row behind the norm of a layer, eagerly and in a
    graph that is replayed on new inputs: the same bits, and near the layer in 64
    bits.  Steps on the way: norm_out, q, k, v (bf16, 2^-8 each), 8-bit operands and
    cache (2^-4 of a value each): what the outputs are off by, relative to their
    norm, stays below the sum of the parts' relative errors, 2^-4 for each of
    the three products' operands and the two caches and their follow-ups through
    the softmax; 1/4 bounds the sum."""
    T, H, HQ, HK, D, L = 24, 512, 8, 2, 64, 40
    x, res, w = normal(dev, (T, H), 50), normal(dev, (T, H), 51), weights(dev, H, 52)
    qkv_f = (normal(dev, ((HQ + 2 * HK) * D, H), 53).float() * H ** -0.5).to(BF)
    o_f = (normal(dev, (H, HQ * D), 54).float() * (HQ * D) ** -0.5).to(BF)
    qkv_w, o_w = farn.fp8_quantize(qkv_f, 128), farn.fp8_quantize(o_f, 128)
    wq, wk = weights(dev, D, 55), weights(dev, D, 56)
    cache = farn.kv_cache(8, 16, HK, D, "fp8", dev)
    fr = freqs_of(dev, D)
    table = torch.tensor([[3, 6, 1]], dtype=I32, device=dev)
    slots = (table[0].long()[(L - T + torch.arange(T, device=dev)) // 16] * 16 +
             (L - T + torch.arange(T, device=dev)) % 16).to(I32)
    pos = torch.arange(L - T, L, device=dev, dtype=I32)
    old = normal(dev, (L - T, HK, D), 57), normal(dev, (L - T, HK, D), 58)
    old_slots = (table[0].long()[torch.arange(L - T, device=dev) // 16] * 16 +
                 torch.arange(L - T, device=dev) % 16).to(I32)
    offsets = torch.tensor([0, L], dtype=I32, device=dev)

    def step():
        farn.kv_write(*old, cache, old_slots)
        _, ro, nrm = farn.forward([x, x], res, w, 1e-6)
        y, *rest = attention_step(dev, nrm, qkv_w, o_w, wq, wk, cache, slots, pos, fr, table,
                                  offsets, L, HQ, HK, D)
        return (nrm, *farn.forward([y], ro, w, 1e-6), y, *rest)
    out = [t.clone() for t in step()]
    nrm = out[0].double()
    qkv = nrm @ qkv_f.double().t()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([HQ * D, HK * D, HK * D], dim=1))
    q, _ = heads_reference(q, wq, 1e-6, pos, fr, None, False)
    k, _ = heads_reference(k, wk, 1e-6, pos, fr, None, False)
    k, v = torch.cat((old[0].double(), k)), torch.cat((old[1].double(), v))
    p = torch.einsum("thd,nhd->thn", q, k.repeat_interleave(HQ // HK, dim=1)) * D ** -0.5
    y = torch.einsum("thn,nhd->thd", p.softmax(dim=2), v.repeat_interleave(HQ // HK, dim=1))
    want = y.reshape(T, HQ * D) @ o_f.double().t()
    assert ((out[4].double() - want).norm() / want.norm()).item() < 0.25
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = step()
    x.copy_(normal(dev, (T, H), 59))
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip([t.clone() for t in static], step()):
        assert torch.equal(a, b)


def test_prepared_calls_reuse_their_buffers(dev):
    T, HQ, HK, D = 30, 4, 2, 64
    q, k, wq, wk, pos, fr, _ = case_inputs(dev, T, HQ, HK, D, D, 1, 60)
    v = normal(dev, (T, HK, D), 61)
    c, c2 = (farn.kv_cache(5, 8, HK, D, "nvfp4", dev) for _ in range(2))
    slots = torch.arange(T, device=dev, dtype=I32)
    table = torch.arange(4, device=dev, dtype=I32)[None]
    offsets = torch.tensor([0, T], dtype=I32, device=dev)
    a = farn.prepare_qk_norm_rope(q, k, wq, wk, 1e-6, pos, fr)
    b = farn.prepare_qk_norm_rope_cache(q, k, v, wq, wk, 1e-6, pos, fr, c, slots, tensor_scales=G)
    w = farn.prepare_kv_write(v, k, c, slots, tensor_scales=G)
    r = farn.prepare_kv_read(c, table, offsets, T, tensor_scales=G)
    for seed in (62, 63):
        q.copy_(normal(dev, q.shape, seed)), k.copy_(normal(dev, k.shape, seed + 2))
        pos += 17
        for x, y in zip(a(), farn.qk_norm_rope(q, k, wq, wk, 1e-6, pos, fr)):
            assert torch.equal(x, y)
        assert torch.equal(b(), farn.qk_norm_rope_cache(q, k, v, wq, wk, 1e-6, pos, fr, c2, slots,
                                                        tensor_scales=G))
        for x, y in zip(r(), farn.kv_read(c2, table, offsets, T, tensor_scales=G)):
            assert torch.equal(x, y)
        assert w() is c
        farn.kv_write(v, k, c2, slots, tensor_scales=G)
        assert all(torch.equal(x, y) for x, y in zip(c, c2))


@pytest.mark.parametrize("prepared", [False, True])
def test_calls_on_a_given_stream(dev, prepared):
    T, HQ, HK, D = 50, 4, 2, 128
    q, k, wq, wk, pos, fr, _ = case_inputs(dev, T, HQ, HK, D, D, 1, 70)
    v = normal(dev, (T, HK, D), 71)
    slots = torch.arange(T, device=dev, dtype=I32)
    table = torch.arange(4, device=dev, dtype=I32)[None]
    offsets = torch.tensor([0, T], dtype=I32, device=dev)
    c, c2 = (farn.kv_cache(4, 16, HK, D, "fp8", dev) for _ in range(2))
    want = [*farn.qk_norm_rope(q, k, wq, wk, 1e-6, pos, fr),
            farn.qk_norm_rope_cache(q, k, v, wq, wk, 1e-6, pos, fr, c2, slots),
            *farn.kv_read(c2, table, offsets, T)]
    late = torch.zeros_like(q)
    out = [torch.empty_like(t) for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pick = (lambda name: getattr(farn, "prepare_" + name)) if prepared else \
        (lambda name: lambda *a, **kw: lambda: getattr(farn, name)(*a, **kw))
    calls = [pick("qk_norm_rope")(late, k, wq, wk, 1e-6, pos, fr, out=out[:2], stream=side),
             pick("kv_write")(v, v, c, slots, stream=side),
             pick("qk_norm_rope_cache")(late, k, v, wq, wk, 1e-6, pos, fr, c, slots, out=out[2],
                                        stream=side),
             pick("kv_read")(c, table, offsets, T, out=out[3:], stream=side)]
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        late.copy_(q)
    for call in calls:
        call()
    assert torch.cuda.current_stream().query() and not side.query()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.equal(a, b) for a, b in zip(c, c2))


def test_contexts_that_cannot_serve(dev):
    q, k, wq, wk, pos, fr, _ = case_inputs(dev, 4, 2, 2, 64, 64, 1, 80)
    c = farn.kv_cache(1, 4, 2, 64, "fp8", dev)
    slots = torch.arange(4, device=dev, dtype=I32)
    table, offsets = slots[None, :1].contiguous(), torch.tensor([0, 4], dtype=I32, device=dev)
    bad = make_ctx(FARN_FAULT_INJECT="launch")
    other = farn.Context(0)
    other.device = 1
    for call in (lambda x: farn.qk_norm_rope(q, k, wq, wk, 1e-6, pos, fr, ctx=x),
                 lambda x: farn.qk_norm_rope_cache(q, k, k, wq, wk, 1e-6, pos, fr, c, slots, ctx=x),
                 lambda x: farn.kv_write(k, k, c, slots, ctx=x),
                 lambda x: farn.kv_read(c, table, offsets, 4, ctx=x)):
        with pytest.raises(farn.FarnError) as e:
            call(bad)
        assert e.value.status == farn.FARN_ERR_CUDA
        with pytest.raises(ValueError, match="device"):
            call(other)
