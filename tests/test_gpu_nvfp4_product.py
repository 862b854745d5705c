"""NVFP4 quantisation, the way back and the product of two NVFP4 tensors on
the GPU, against the oracle's codes and plain 64-bit definitions."""
import math
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import rank_sum_residual_gb300 as farn  # noqa: E402
from gpu_util import make_ctx  # noqa: E402
from parity import u16  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    farn.build_library()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


@pytest.fixture(scope="module")
def O():
    return oracle.Oracle()


@pytest.fixture(scope="module")
def ctxs(dev):
    return {"auto": farn.Context(0), "generic": make_ctx(FARN_VARIANT="generic"),
            "pair": make_ctx(FARN_TC_TILE=256),
            "one": make_ctx(FARN_TC_TILE=64, FARN_TC_SPLIT=1),
            "split2": make_ctx(FARN_TC_TILE=64, FARN_TC_SPLIT=2),
            "split4": make_ctx(FARN_TC_TILE=64, FARN_TC_SPLIT=4)}


ALL = ["auto", "generic", "pair", "one", "split2", "split4"]


def values(codes, scales):
    """code * scale in 64 bits."""
    c = torch.stack((codes & 15, codes >> 4), dim=2).flatten(1).cpu().numpy()
    mag = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])[c & 7] * np.where(c & 8, -1.0, 1.0)
    b = scales.cpu().numpy().astype(np.int64)
    e, f = (b >> 3) & 15, b & 7
    s = np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    s = np.where((b & 127) == 127, math.nan, s)
    return torch.from_numpy(mag * np.repeat(s, 16, axis=1)).to(codes.device)


def inputs(dev, T, H, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(T, H, device=dev, generator=g)
    x *= torch.where(torch.rand(T, H, device=dev, generator=g) < 0.01, 50.0, 1.0)
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("which", ["auto", "generic"])
@pytest.mark.parametrize("g", [168.0, 1.0, 0.03125, 3000.0])
@pytest.mark.parametrize("T,H", [(1, 16), (1, 4096), (3, 48), (7, 1040), (129, 5120)])
def test_quantize_and_back(O, dev, ctxs, which, g, T, H):
    x = inputs(dev, T, H, T + H)
    x[0, :16] = 0.0                                             # a block without a scale
    if H > 16:
        x[T // 2, 16:20] = torch.tensor([math.nan, math.inf, -math.inf, 1.0])
        x[T - 1, 32:36] = torch.tensor([math.nan, -0.0, 2.0, -0.1])
    q, s = farn.nvfp4_quantize(x, g, ctx=ctxs[which])
    want_q, want_s = O.quant_nvfp4(u16(x), g)
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)
    back = farn.nvfp4_dequantize(q, s, g, ctx=ctxs[which])
    # scale / g and its product with the code, each rounded to fp32, then to bf16
    c = torch.stack((q & 15, q >> 4), dim=2).flatten(1)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                         device=dev)
    f = s.view(torch.float8_e4m3fn).float() / torch.tensor(g, device=dev)
    want = (table[c.long()] * f.repeat_interleave(16, dim=1)).to(torch.bfloat16)
    assert torch.equal(back, want)


def test_quantize_same_as_the_norms_copy(dev):
    """The codes of norm_out equal farn_forward_nvfp4's own copy of it."""
    g = 100.0
    x, w = inputs(dev, 33, 2048, 1), inputs(dev, 1, 2048, 2)[0]
    _, _, nrm, q, s = farn.forward_nvfp4([x], x, w, 1e-6, g)
    q2, s2 = farn.nvfp4_quantize(nrm, g)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_conversions_any_alignment(O, dev):
    """Tensors that start off a vector, and nothing written next to them."""
    T, H, g = 5, 80, 168.0
    xf = inputs(dev, 1, T * H + 8, 3)[0]
    for d in (0, 1, 8):
        x = xf[d:d + T * H].view(T, H)
        qb = torch.full((T * H // 2 + 16,), 99, dtype=torch.uint8, device=dev)
        sb = torch.full((T * H // 16 + 16,), 99, dtype=torch.uint8, device=dev)
        ob = torch.full((T * H + 16,), 99.0, dtype=torch.bfloat16, device=dev)
        n, m, k = 8 + d, 8 + d, 8 + d
        q, s = qb[n:n + T * H // 2].view(T, H // 2), sb[m:m + T * H // 16].view(T, H // 16)
        farn.nvfp4_quantize(x, g, out=(q, s))
        want_q, want_s = O.quant_nvfp4(u16(x), g)
        assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)
        o = ob[k:k + T * H].view(T, H) if d < 8 else ob[0:T * H].view(T, H)
        farn.nvfp4_dequantize(q, s, g, out=o)
        assert torch.equal(o, farn.nvfp4_dequantize(q.clone(), s.clone(), g))
        assert (qb[:n] == 99).all() and (qb[n + T * H // 2:] == 99).all()
        assert (sb[:m] == 99).all() and (sb[m + T * H // 16:] == 99).all()
        assert (ob[(k if d < 8 else 0) + T * H:] == 99).all()


def test_empty_conversions(dev):
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=dev)
    q, s = farn.nvfp4_quantize(x, 1.0)
    assert q.shape == (0, 32) and s.shape == (0, 4)
    assert farn.nvfp4_dequantize(q, s, 1.0).shape == (0, 64)
    w = torch.zeros(8, 32, dtype=torch.uint8, device=dev), torch.zeros(8, 4, dtype=torch.uint8,
                                                                        device=dev)
    assert farn.nvfp4_matmul(q, s, 1.0, *w, 1.0).shape == (0, 8)


def random_tensor(dev, rows, H, seed, scales):
    g = torch.Generator(device=dev).manual_seed(seed)
    q = torch.randint(0, 256, (rows, H // 2), device=dev, generator=g, dtype=torch.uint8)
    pick = torch.randint(0, len(scales), (rows, H // 16), device=dev, generator=g)
    return q, torch.tensor(scales, dtype=torch.uint8, device=dev)[pick]


# one token to long calls; tile borders and one to each side; rests of the
# row in codes (32), scales (256) and both; H of 16 modulo 32 (no TMA)
SHAPES = [(1, 1, 16), (1, 8, 32), (1, 128, 64), (2, 130, 96), (15, 127, 256), (16, 129, 288),
          (17, 256, 512), (32, 300, 544), (33, 257, 1024), (64, 384, 1056), (65, 100, 2048),
          (100, 1000, 2080), (127, 256, 80), (128, 512, 4096), (129, 640, 272), (191, 255, 768),
          (193, 511, 800), (223, 257, 320), (225, 513, 1312), (300, 768, 256), (448, 1024, 160),
          (449, 1030, 608), (1000, 300, 1024)]


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("T,N,H", SHAPES)
def test_product_exact(dev, ctxs, which, T, N, H):
    """Scales 1, 2, 4 and 0: products are multiples of 1/4 and at most 576,
    so sums below 2^22 are exact in fp32 whatever the order: one value, one
    rounding to bf16."""
    a = random_tensor(dev, T, H, T, [0x38, 0x40, 0x48, 0x00])
    b = random_tensor(dev, N, H, N + 1, [0x38, 0x40, 0x48, 0x00])
    got = farn.nvfp4_matmul(*a, 1.0, *b, 0.5, ctx=ctxs[which])
    want = 2.0 * (values(*a) @ values(*b).t())
    torch.cuda.synchronize()
    assert farn.farn_device_status(ctxs[which].handle) == 0
    assert torch.equal(got, want.float().to(torch.bfloat16))


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("T,N,H", [(1, 512, 8192), (20, 300, 4096), (130, 260, 5120),
                                   (520, 300, 2080)])
def test_product_rounding(dev, ctxs, which, T, N, H):
    """Scales over their whole range.  Every addition is off by at most a step
    of fp32 (2^-23 of a partial sum, which the magnitudes bound; truncation
    counts a whole step), H + 1 of them, alpha by 2^-24, its product by 2^-24
    and the rounding to bf16 by 2^-8 of the value."""
    scales = [0x00, 0x01, 0x07, 0x08, 0x20, 0x33, 0x38, 0x4D, 0x5A, 0x66, 0x77, 0x7E]
    a, b = random_tensor(dev, T, H, 5, scales), random_tensor(dev, N, H, 6, scales)
    ga, gb = 168.0, 37.5
    got = farn.nvfp4_matmul(*a, ga, *b, gb, ctx=ctxs[which])
    va, vb = values(*a), values(*b)
    want, mag = va @ vb.t() / (ga * gb), va.abs() @ vb.abs().t() / (ga * gb)
    acc = (H + 1) * 2.0 ** -23 * mag + 2.0 ** -23 * want.abs()
    tol = 2.0 ** -8 * (want.abs() + acc) + acc
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("T", [3, 300])
def test_product_nan_scale_stays_with_its_row(dev, ctxs, which, T):
    N, H = 200, 512
    a = random_tensor(dev, T, H, 7, [0x38])
    b = random_tensor(dev, N, H, 8, [0x38])
    a[1][1, 3] = 0x7F
    got = farn.nvfp4_matmul(*a, 1.0, *b, 1.0, ctx=ctxs[which])
    assert torch.isnan(got[1]).all()
    want = (values(*a) @ values(*b).t()).float().to(torch.bfloat16)
    keep = torch.arange(T, device=dev) != 1
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("T", [2, 40, 500])
def test_product_any_alignment_and_nothing_behind(dev, ctxs, T):
    N, H = 70, 256
    for d in (0, 1, 8, 16):
        qb = torch.zeros(T * H // 2 + 16, dtype=torch.uint8, device=dev)
        sb = torch.zeros(T * H // 16 + 16, dtype=torch.uint8, device=dev)
        a0 = random_tensor(dev, T, H, 9, [0x38, 0x40])
        q, s = qb[d:d + T * H // 2].view(T, H // 2), sb[d:d + T * H // 16].view(T, H // 16)
        q.copy_(a0[0]), s.copy_(a0[1])
        b = random_tensor(dev, N, H, 10, [0x38, 0x40])
        buf = torch.full((T * N + 32,), 7.0, dtype=torch.bfloat16, device=dev)
        out = buf[d:d + T * N].view(T, N)
        farn.nvfp4_matmul(q, s, 1.0, *b, 1.0, out=out, ctx=ctxs["auto"])
        want = (values(*a0) @ values(*b).t()).float().to(torch.bfloat16)
        assert torch.equal(out, want)
        assert (buf[:d] == 7.0).all() and (buf[d + T * N:] == 7.0).all()


@pytest.mark.parametrize("which", ["pair", "one", "split2"])
@pytest.mark.parametrize("H", [256, 288])
def test_product_scales_at_any_byte(dev, ctxs, which, H):
    """Block scales that start at any byte, in rows of whole 16-byte pieces and
    not; the bytes before and behind them would show as NaN."""
    T, N = 70, 300
    a, b = random_tensor(dev, T, H, 15, [0x38, 0x40]), random_tensor(dev, N, H, 16, [0x38, 0x40])
    want = (values(*a) @ values(*b).t()).float().to(torch.bfloat16)
    for d in (0, 1, 2, 3, 4, 6, 15):
        def moved(t):
            buf = torch.full((t.numel() + 32,), 0x7F, dtype=torch.uint8, device=dev)
            v = buf[d:d + t.numel()].view(t.shape)
            v.copy_(t)
            return v
        got = farn.nvfp4_matmul(a[0], moved(a[1]), 1.0, b[0], moved(b[1]), 1.0, ctx=ctxs[which])
        assert torch.equal(got, want), d


@pytest.mark.parametrize("which", ["pair", "one"])
def test_product_beyond_4_gib(dev, ctxs, which):
    """Output rows whose byte offsets pass 32 bits."""
    T, N, H = 70001, 32776, 64
    a, b = random_tensor(dev, T, H, 17, [0x38]), random_tensor(dev, N, H, 18, [0x38])
    got = farn.nvfp4_matmul(*a, 1.0, *b, 1.0, ctx=ctxs[which])
    some = torch.tensor([0, 65535, 65536, 69999, 70000], device=dev)
    want = (values(a[0][some], a[1][some]) @ values(*b).t()).float().to(torch.bfloat16)
    assert torch.equal(got[some], want)
    del got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("env", [dict(FARN_TC_TILE=256), dict(FARN_TC_TILE=64, FARN_TC_SPLIT=2)])
@pytest.mark.parametrize("H", [2048, 2080])
def test_product_waits_are_bounded(dev, env, H):
    """As for the grouped product, with both ways the block scales come."""
    ctx = make_ctx(FARN_FAULT_INJECT="stall", **env)
    a, b = random_tensor(dev, 300, H, 19, [0x38]), random_tensor(dev, 600, H, 20, [0x38])
    farn.nvfp4_matmul(*a, 1.0, *b, 1.0, ctx=ctx)
    torch.cuda.synchronize()
    assert farn.farn_device_status(ctx.handle) & (16 | 32 | 64 | 128)
    ctx.close()
    got = farn.nvfp4_matmul(*a, 1.0, *b, 1.0)
    want = (values(*a) @ values(*b).t()).float().to(torch.bfloat16)
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [100, 300])
def test_product_gives_up_within_its_limit(dev, T):
    """A CTA that gave up waits for what it asked for and no longer, also where
    a tile has so few slots that a block of their scales is not loaded: the
    call takes one limit of 2 s, not several.  (A block that is not loaded is
    left to wait for only behind a tile that gave up on one that is; no call
    can be made to do that, so this holds the plain cases.)"""
    ctx = make_ctx(FARN_FAULT_INJECT="stall", FARN_TC_TILE=256)
    a, b = random_tensor(dev, T, 2048, 21, [0x38]), random_tensor(dev, 600, 2048, 22, [0x38])
    torch.cuda.synchronize()
    t0 = time.monotonic()
    farn.nvfp4_matmul(*a, 1.0, *b, 1.0, ctx=ctx)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 3.5
    assert farn.farn_device_status(ctx.handle) & (16 | 32 | 64 | 128)
    ctx.close()


def test_product_plans(dev, ctxs):
    a = 1 << 32

    def plan(T, N, H, codes=a, which="auto"):
        return farn.farn_plan_nvfp4_matmul(ctxs[which].handle, codes, 2 * a, 3 * a, 4 * a + 1, T,
                                           N, H, 5 * a)[:2]
    assert plan(1, 8192, 8192) == ("tensor", 2)
    assert plan(64, 2048, 8192) == ("tensor", 4)
    assert plan(8192, 8192, 8192) == ("pair", 2)
    assert plan(300, 8192, 2080) == ("pair", 2)
    assert plan(64, 512, 1008) == ("generic", 1)
    assert plan(64, 512, 1024, codes=a + 8) == ("generic", 1)
    assert plan(64, 512, 1024, which="generic") == ("generic", 1)
    assert plan(64, 512, 1024, which="split2") == ("tensor", 2)


def test_norm_to_product(dev):
    """The norm's NVFP4 copy into a projection of quantised weights, captured
    and replayed."""
    T, H, N, g, gw = 40, 1024, 384, 168.0, 300.0
    x, w = inputs(dev, T, H, 11), inputs(dev, 1, H, 12)[0]
    proj = inputs(dev, N, H, 13)
    wq, ws = farn.nvfp4_quantize(proj, gw)

    def step():
        _, ro, _, q, s = farn.forward_nvfp4([x, x], x, w, 1e-6, g, write_norm=False)
        return q, s, farn.nvfp4_matmul(q, s, g, wq, ws, gw)
    q, s, y = (t.clone() for t in step())
    want = values(q, s) @ values(wq, ws).t() / (g * gw)
    mag = values(q, s).abs() @ values(wq, ws).abs().t() / (g * gw)
    acc = (H + 1) * 2.0 ** -23 * mag + 2.0 ** -23 * want.abs()
    assert ((y.double() - want).abs() <= 2.0 ** -8 * (want.abs() + acc) + acc).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(inputs(dev, T, H, 14))
    graph.replay()
    torch.cuda.synchronize()
    again = step()
    for a, b in zip(out, again):
        assert torch.equal(a, b)


def test_prepared_calls_reuse_their_buffers(dev):
    """Prepared conversions and products, launched again after their input
    changed in place, give the immediate calls' bits."""
    T, H, N = 21, 512, 144
    x, w = inputs(dev, T, H, 31), inputs(dev, N, H, 32)
    wq, ws = farn.nvfp4_quantize(w, 200.0)
    quantize = farn.prepare_nvfp4_quantize(x, 100.0)
    q, s = quantize.outputs
    given = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
    back = farn.prepare_nvfp4_dequantize(q, s, 100.0)
    product = farn.prepare_nvfp4_matmul(q, s, 100.0, wq, ws, 200.0, out=given)
    for seed in (33, 34):
        x.copy_(inputs(dev, T, H, seed))
        quantize()
        q2, s2 = farn.nvfp4_quantize(x, 100.0)
        assert torch.equal(q, q2) and torch.equal(s, s2)
        assert torch.equal(back(), farn.nvfp4_dequantize(q2, s2, 100.0))
        assert product() is given
        assert torch.equal(given, farn.nvfp4_matmul(q2, s2, 100.0, wq, ws, 200.0))


@pytest.mark.parametrize("prepared", [False, True])
def test_calls_on_a_given_stream(dev, prepared):
    """The calls run on the stream that they are given, behind what it has to
    do first, while the current stream stays idle."""
    T, H, N = 40, 512, 144
    x, w = inputs(dev, T, H, 35), inputs(dev, N, H, 36)
    wq, ws = farn.nvfp4_quantize(w, 200.0)
    q0, s0 = farn.nvfp4_quantize(x, 100.0)
    want = farn.nvfp4_dequantize(q0, s0, 100.0), farn.nvfp4_matmul(q0, s0, 100.0, wq, ws, 200.0)
    late, q, s = torch.zeros_like(x), torch.empty_like(q0), torch.empty_like(s0)
    back, y = torch.empty_like(want[0]), torch.empty_like(want[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pick = (lambda name: getattr(farn, "prepare_" + name)) if prepared else \
        (lambda name: lambda *a, **k: lambda: getattr(farn, name)(*a, **k))
    calls = [pick("nvfp4_quantize")(late, 100.0, out=(q, s), stream=side),
             pick("nvfp4_dequantize")(q, s, 100.0, out=back, stream=side),
             pick("nvfp4_matmul")(q, s, 100.0, wq, ws, 200.0, out=y, stream=side)]
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        late.copy_(x)
    for call in calls:
        call()
    assert torch.cuda.current_stream().query() and not side.query()
    side.synchronize()
    assert torch.equal(q, q0) and torch.equal(s, s0)
    assert torch.equal(back, want[0]) and torch.equal(y, want[1])


def test_launch_fault_reaches_the_caller(dev):
    bad = make_ctx(FARN_FAULT_INJECT="launch")
    x = inputs(dev, 4, 64, 1)
    q, s = farn.nvfp4_quantize(x, 1.0)
    for call in (lambda: farn.nvfp4_quantize(x, 1.0, ctx=bad),
                 lambda: farn.nvfp4_dequantize(q, s, 1.0, ctx=bad),
                 lambda: farn.nvfp4_matmul(q, s, 1.0, q, s, 1.0, ctx=bad)):
        with pytest.raises(farn.FarnError) as e:
            call()
        assert e.value.status == farn.FARN_ERR_CUDA
