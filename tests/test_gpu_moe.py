"""The MoE router and the products grouped by expert on the GPU, against
plain 64-bit definitions; and the router, the products and the combine run
together."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import rank_sum_residual_gb300 as farn  # noqa: E402
from gpu_util import make_ctx  # noqa: E402

pytestmark = pytest.mark.gpu
INF = math.inf


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
    """The library's own choice, the kernel for any shape, and every shape of
    tile of the others."""
    return {"auto": farn.Context(0), "generic": make_ctx(FARN_VARIANT="generic"),
            "pair": make_ctx(FARN_TC_TILE=256),
            "one": make_ctx(FARN_TC_TILE=64, FARN_TC_SPLIT=1),
            "split2": make_ctx(FARN_TC_TILE=64, FARN_TC_SPLIT=2),
            "split4": make_ctx(FARN_TC_TILE=64, FARN_TC_SPLIT=4)}


ALL = ["auto", "generic", "pair", "one", "split2", "split4"]


# ---------------------------------------------------------------- router
def route_reference(logits, K, renorm):
    x = logits.double().cpu().numpy()
    T, E = x.shape
    dead = np.isnan(x) | (x == -INF)
    order = np.argsort(np.where(dead, INF, -x), axis=1, kind="stable")
    # the dead ones sort last; +inf logits (-inf here) first
    chosen = order[:, :K]
    live = ~np.take_along_axis(dead, chosen, axis=1)
    m = np.where(dead, -INF, x).max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.where(dead, 0.0, np.where(x == m, 1.0, np.exp(x - m)))
    pc = np.where(live, np.take_along_axis(p, chosen, axis=1), 0.0)
    total = (pc if renorm else p).sum(axis=1, keepdims=True)
    gates = np.divide(pc, total, out=np.zeros_like(pc), where=total > 0)
    experts = np.where(live, chosen, -1)
    flat = experts.ravel()
    pairs = np.flatnonzero(flat >= 0)
    pairs = pairs[np.argsort(flat[pairs], kind="stable")]
    index = np.full(T * K, -1)
    index[pairs] = np.arange(pairs.size)
    rows = np.full(T * K, -1)
    rows[:pairs.size] = pairs // K
    offsets = np.searchsorted(np.sort(flat[flat >= 0]), np.arange(E + 1))
    return experts, gates, index.reshape(T, K), rows, offsets


def check_route(logits, K, renorm, out=None, ctx=None):
    got = farn.moe_route(logits, K, renorm, out=out, ctx=ctx)
    torch.cuda.synchronize()
    want = route_reference(logits, K, renorm)
    for name, g, w in zip(("experts", "gates", "index", "rows", "offsets"), got, want):
        g = g.cpu().numpy()
        if name == "gates":
            # exp: 2 ulp and its argument's rounding, |l - max| 2^-24 of it;
            # a sum of E positive terms: E 2^-24; the quotient 2^-24
            span = 40.0
            tol = (2 * 2.0 ** -23 + span * 2.0 ** -24 + (logits.shape[1] + 2) * 2.0 ** -24) * 2
            assert np.abs(g - w).max(initial=0) <= tol, name
            assert (np.abs(g - w) <= tol * w + 1e-37).all(), name
        else:
            assert np.array_equal(g, w), name
    return got


def normal(dev, T, E, seed, dtype):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (2 * torch.randn(T, E, device=dev, generator=g)).to(dtype)


SIZES = [(0, 8, 2), (1, 1, 1), (1, 128, 8), (3, 7, 7), (16, 64, 8), (33, 65, 3), (64, 1024, 32),
         (100, 40, 32), (129, 256, 8), (511, 130, 5), (512, 1000, 1), (513, 96, 4),
         (600, 1024, 1), (1000, 1024, 1), (1025, 1024, 1), (2047, 33, 2), (4096, 256, 8),
         (5001, 8, 1), (40000, 64, 2)]


@pytest.mark.parametrize("T,E,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(dev, T, E, K, dtype, renorm):
    check_route(normal(dev, T, E, T + E, dtype), K, renorm)


def test_route_many_tokens(dev):
    """Enough tokens for larger blocks (over 512 blocks of 64)."""
    check_route(normal(dev, 70001, 16, 3, torch.bfloat16), 2, True)
    check_route(normal(dev, 600011, 4, 4, torch.bfloat16), 1, True)


@pytest.mark.parametrize("T", [5, 300, 3000])
def test_route_ties_masks_and_specials(dev, T):
    x = normal(dev, T, 48, 9, torch.float32).round()           # many equal logits
    x[:, ::5] = -INF                                            # masked experts
    x[0] = -INF                                                 # a token without experts
    x[1, :] = 0.0
    x[1, 3] = -0.0                                              # ties with +0
    x[2, 7] = math.nan                                          # never chosen
    x[3, 11] = INF
    x[3, 20] = INF                                              # two infinite logits share
    x[4, 1:] = -INF                                             # fewer than K left
    x[4, 0] = -3.0e38
    x[-1] = -INF
    check_route(x, 8, True)
    check_route(x, 8, False)


@pytest.mark.parametrize("T", [40, 2000])
def test_route_all_masked(dev, T):
    x = torch.full((T, 64), -INF, device=dev)
    e, g, i, r, o = check_route(x, 4, True)
    assert int(e.max()) == -1 and float(g.abs().max()) == 0 and int(o.max()) == 0


@pytest.mark.parametrize("T", [77, 1500])
def test_route_one_expert_takes_all(dev, T):
    x = normal(dev, T, 64, 5, torch.float32)
    x[:, 9] = 50.0
    check_route(x, 2, True)


@pytest.mark.parametrize("T", [12, 900])
def test_route_written_whole_and_nothing_behind(dev, T):
    """Every output element is written, and nothing next to the outputs."""
    K, E = 3, 20
    x = normal(dev, T, E, 1, torch.float32)
    x[T // 2:] = -INF
    pad = 64
    bufs = [torch.full((n + 2 * pad,), 77, dtype=torch.int32, device=dev)
            for n in (T * K, T * K, T * K, T * K, E + 1)]
    v = [b[pad:-pad] for b in bufs]
    out = (v[0].view(T, K), v[1].view(torch.float32).view(T, K), v[2].view(T, K), v[3], v[4])
    check_route(x, K, True, out=out)
    for b in bufs:
        assert (b[:pad] == 77).all() and (b[-pad:] == 77).all()


# --------------------------------------------------------- grouped product
def make_groups(counts, lead=0):
    off = np.concatenate([[0], np.cumsum(counts)]) + lead
    return off.astype(np.int32)


def grouped_reference(x, w, offsets, rows, S):
    out = torch.full((S, w.shape[1]), math.nan, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi == lo:
            continue
        if rows is None:
            a = x[lo:hi].double()
        else:
            r = rows[lo:hi].long()
            ok = (r >= 0) & (r < x.shape[0])
            a = torch.where(ok[:, None], x[r.clamp(0, x.shape[0] - 1)].double(), 0.0)
        b = w[e].double()
        out[lo:hi] = a @ b.t()
        mag[lo:hi] = a.abs() @ b.abs().t()
    return out, mag


# counts per expert, N, H: empty experts, one slot, tile borders of every
# tile size and one to each side, rows of one vector, a short and odd rest
GROUPS = [
    ([1], 8, 8), ([1], 1, 64), ([3, 0, 5], 40, 72), ([0, 0, 2], 128, 64), ([16], 129, 128),
    ([17, 15, 1], 130, 136), ([31, 33, 32], 256, 200), ([64, 65, 63], 257, 320),
    ([0, 127, 129, 0, 128], 300, 264), ([255, 257, 0, 256, 1], 384, 512),
    ([300, 5, 0, 700], 512, 1032), ([2050], 264, 128), ([1] * 100, 200, 256),
    ([2, 1, 0, 3] * 16, 640, 2048), ([9, 4], 1, 4096), ([40, 300], 260, 128),
    ([70, 1], 258, 128), ([70, 1], 259, 128),
]


def integer(shape, dev, seed, top=3):
    """Small whole numbers: every product and sum is exact in fp32, so the
    result has one value whatever the order, and one rounding to bf16."""
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randint(-top, top + 1, shape, device=dev, generator=g).to(torch.bfloat16)


def check_exact(got, want, offsets, what):
    lo, hi = int(offsets[0]), int(offsets[-1])
    assert torch.equal(got[lo:hi], want[lo:hi].float().to(torch.bfloat16)), what


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,N,H", GROUPS)
def test_grouped_exact(dev, ctxs, which, gather, counts, N, H):
    offsets = make_groups(counts)
    S, E = int(offsets[-1]), len(counts)
    x = integer((S if not gather else S // 2 + 1, H), dev, 1)
    w = integer((E, N, H), dev, 2)
    rows = None
    if gather:
        g = torch.Generator(device=dev).manual_seed(3)
        rows = torch.randint(0, x.shape[0], (S,), device=dev, generator=g, dtype=torch.int32)
    got = farn.grouped_matmul(x, w, torch.from_numpy(offsets).to(dev), rows, ctx=ctxs[which])
    want, _ = grouped_reference(x, w, offsets, rows, S)
    torch.cuda.synchronize()
    assert farn.farn_device_status(ctxs[which].handle) == 0
    check_exact(got, want, offsets, (counts, N, H))


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("counts,N,H", [([5, 0, 11], 72, 520), ([300, 20], 264, 2056),
                                        ([1, 1], 512, 7168), ([130] * 4, 300, 1000)])
def test_grouped_rounding(dev, ctxs, which, counts, N, H):
    """Normal values: fp32 sums and one rounding.  Every addition is off by
    at most a step of fp32 (2^-23 of a partial sum that the magnitudes bound:
    truncation counts a whole step), H + 1 of them; the rounding to bf16 by
    2^-8 of the value."""
    offsets = make_groups(counts)
    S, E = int(offsets[-1]), len(counts)
    g = torch.Generator(device=dev).manual_seed(4)
    x = torch.randn(S, H, device=dev, generator=g).to(torch.bfloat16)
    w = torch.randn(E, N, H, device=dev, generator=g).to(torch.bfloat16)
    got = farn.grouped_matmul(x, w, torch.from_numpy(offsets).to(dev), ctx=ctxs[which])
    want, mag = grouped_reference(x, w, offsets, None, S)
    acc = (H + 1) * 2.0 ** -23 * mag
    tol = 2.0 ** -8 * (want.abs() + acc) + acc
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("which", ["auto", "generic"])
@pytest.mark.parametrize("N,H", [(33, 9), (64, 15), (10, 1), (100, 1001)])
def test_grouped_any_row_length(dev, ctxs, which, N, H):
    offsets = make_groups([7, 0, 70])
    x, w = integer((77, H), dev, 5), integer((3, N, H), dev, 6)
    got = farn.grouped_matmul(x, w, torch.from_numpy(offsets).to(dev), ctx=ctxs[which])
    want, _ = grouped_reference(x, w, offsets, None, 77)
    check_exact(got, want, offsets, (N, H))


def test_grouped_any_alignment(dev, ctxs):
    """Operands that start two bytes off a vector."""
    offsets = make_groups([30, 40])
    flat = integer((70 * 64 + 1,), dev, 7)
    wflat = integer((2 * 48 * 64 + 1,), dev, 8)
    off = torch.from_numpy(offsets).to(dev)
    for dx in (0, 1):
        for dw in (0, 1):
            x = flat[dx:dx + 70 * 64].view(70, 64)
            w = wflat[dw:dw + 2 * 48 * 64].view(2, 48, 64)
            obuf = torch.zeros(70 * 48 + 1, dtype=torch.bfloat16, device=dev)
            out = obuf[dx:dx + 70 * 48].view(70, 48)
            got = farn.grouped_matmul(x, w, off, out=out, ctx=ctxs["auto"])
            want, _ = grouped_reference(x, w, offsets, None, 70)
            check_exact(got, want, offsets, (dx, dw))


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("per", [2, 40, 300])
def test_grouped_rows_behind_are_left(dev, ctxs, which, per):
    """Slots before the first expert's and behind the last expert's keep what
    they held, and so does memory next to the output."""
    offsets = make_groups([per, 0, per + 1], lead=3)
    S, N, H = int(offsets[-1]) + 5, 72, 128
    x, w = integer((S, H), dev, 9), integer((3, N, H), dev, 10)
    buf = torch.full(((S + 4) * N,), 5.5, dtype=torch.bfloat16, device=dev)
    out = buf[2 * N:-2 * N].view(S, N)
    farn.grouped_matmul(x, w, torch.from_numpy(offsets).to(dev), out=out, ctx=ctxs[which])
    want, _ = grouped_reference(x, w, offsets, None, S)
    check_exact(out, want, offsets, per)
    assert (buf[:5 * N] == 5.5).all() and (buf[-7 * N:] == 5.5).all()


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("per", [3, 200])
def test_grouped_rows_that_do_not_exist(dev, ctxs, which, per):
    """A slot whose row is outside x gets zeros, whatever the weights hold,
    and infinities in x stay with their own slots."""
    offsets = make_groups([per, per])
    S, N, H = 2 * per, 136, 192
    x, w = integer((50, H), dev, 11), integer((2, N, H), dev, 12)
    x[7] = INF
    w[1, 5] = math.nan
    rows = torch.arange(S, device=dev, dtype=torch.int32) % 50
    rows[0], rows[per], rows[S - 1] = -1, 50, 2 ** 31 - 1
    got = farn.grouped_matmul(x, w, torch.from_numpy(offsets).to(dev), rows, ctx=ctxs[which])
    for s in (0, per, S - 1):
        assert (got[s] == 0).all()
    want, _ = grouped_reference(x, w, offsets, rows, S)
    dead = torch.zeros(S, dtype=torch.bool, device=dev)
    dead[[0, per, S - 1]] = True
    same = torch.isfinite(want) & ~dead[:, None]
    assert torch.equal(got[same], want[same].float().to(torch.bfloat16))
    assert not torch.isfinite(got[~torch.isfinite(want) & ~dead[:, None]]).any()


def test_grouped_offsets_out_of_range_stay_inside(dev, ctxs):
    """Offsets that are not ascending or leave the slots are clamped: nothing
    outside the output is written."""
    S, N, H = 40, 64, 64
    x, w = integer((S, H), dev, 13), integer((4, N, H), dev, 14)
    for bad in ([-5, 10, 4, 100, 2 ** 31 - 1], [40, 30, 20, 10, 0], [0, 2 ** 31 - 1, 0, 0, 40],
                [0, 40, 0, 40, 0], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 7]):
        for which in ALL:
            buf = torch.full(((S + 4) * N,), 5.5, dtype=torch.bfloat16, device=dev)
            farn.grouped_matmul(x, w, torch.tensor(bad, dtype=torch.int32, device=dev),
                                out=buf[2 * N:-2 * N].view(S, N), ctx=ctxs[which])
            torch.cuda.synchronize()
            assert (buf[:2 * N] == 5.5).all() and (buf[-2 * N:] == 5.5).all()
            assert farn.farn_device_status(ctxs[which].handle) == 0


def test_grouped_empty_calls(dev):
    w = torch.zeros(3, 16, 64, dtype=torch.bfloat16, device=dev)
    none = torch.zeros(4, dtype=torch.int32, device=dev)
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=dev)
    assert farn.grouped_matmul(x, w, none).shape == (0, 16)
    # slots without rows to read: every slot gets zeros
    rows = torch.zeros(5, dtype=torch.int32, device=dev)
    off = torch.tensor([0, 2, 2, 5], dtype=torch.int32, device=dev)
    assert (farn.grouped_matmul(x, w + 1, off, rows) == 0).all()


def test_grouped_same_bits_twice(dev):
    """The order of the sums is fixed: the same call gives the same bits."""
    offsets = torch.from_numpy(make_groups([3, 50, 0, 300])).to(dev)
    g = torch.Generator(device=dev).manual_seed(15)
    x = torch.randn(353, 4096, device=dev, generator=g).to(torch.bfloat16)
    w = torch.randn(4, 512, 4096, device=dev, generator=g).to(torch.bfloat16)
    a = farn.grouped_matmul(x, w, offsets)
    for _ in range(3):
        assert torch.equal(farn.grouped_matmul(x, w, offsets), a)


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_many_experts(dev, ctxs, which, gather):
    """The most experts, most of them with a slot or none."""
    E, N, H = 1024, 136, 72
    counts = np.random.RandomState(3).choice([0, 0, 1, 2, 5, 130], size=E, p=[.3, .2, .3, .1, .08, .02])
    offsets = make_groups(counts)
    S = int(offsets[-1])
    x = integer((S if not gather else 300, H), dev, 21)
    w = integer((E, N, H), dev, 22)
    rows = None
    if gather:
        g = torch.Generator(device=dev).manual_seed(23)
        rows = torch.randint(0, 300, (S,), device=dev, generator=g, dtype=torch.int32)
    got = farn.grouped_matmul(x, w, torch.from_numpy(offsets).to(dev), rows, ctx=ctxs[which])
    want, _ = grouped_reference(x, w, offsets, rows, S)
    check_exact(got, want, offsets, which)


@pytest.mark.parametrize("which", ["pair", "one"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_beyond_4_gib(dev, ctxs, which, gather):
    """Rows of x and of the output whose byte offsets pass 32 bits."""
    S, N, H = 70001, 32776, 32768
    x = torch.zeros(S, H, dtype=torch.bfloat16, device=dev)
    some = torch.tensor([0, 1, 32767, 65535, 65536, 65537, 69999, 70000], device=dev)
    x[some] = integer((some.numel(), H), dev, 24)
    w = torch.zeros(1, N, H, dtype=torch.bfloat16, device=dev)
    wsome = torch.tensor([0, 5, 127, 128, 32767, 32775], device=dev)
    w[0, wsome] = integer((wsome.numel(), H), dev, 25)
    rows = torch.arange(S, device=dev, dtype=torch.int32).flip(0).contiguous() if gather else None
    off = torch.tensor([0, S], dtype=torch.int32, device=dev)
    got = farn.grouped_matmul(x, w, off, rows, ctx=ctxs[which])
    want = (x[some].double() @ w[0, wsome].double().t()).float().to(torch.bfloat16)
    at = S - 1 - some if gather else some
    assert torch.equal(got[at][:, wsome], want)
    assert int((got != 0).sum()) == int((want != 0).sum())
    del x, w, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("env", [dict(FARN_TC_TILE=256), dict(FARN_TC_TILE=64, FARN_TC_SPLIT=1),
                                 dict(FARN_TC_TILE=64, FARN_TC_SPLIT=4)])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_waits_are_bounded(dev, env, gather):
    """With FARN_FAULT_INJECT=stall the first CTA's weights never come: its
    waits and those of the CTAs that work with it run out (2 s), the call
    ends and the status word says so.  Other calls are unharmed."""
    ctx = make_ctx(FARN_FAULT_INJECT="stall", **env)
    offsets = torch.tensor([0, 70, 200], dtype=torch.int32, device=dev)
    x, w = integer((200, 1024), dev, 26), integer((2, 512, 1024), dev, 27)
    rows = torch.arange(200, device=dev, dtype=torch.int32) if gather else None
    farn.grouped_matmul(x, w, offsets, rows, ctx=ctx)
    torch.cuda.synchronize()
    assert farn.farn_device_status(ctx.handle) & (16 | 32 | 64 | 128)
    assert farn.farn_device_status(ctx.handle) == 0
    ctx.close()
    got = farn.grouped_matmul(x, w, offsets, rows)
    want, _ = grouped_reference(x, w, offsets.cpu().numpy(), rows, 200)
    check_exact(got, want, offsets, "after")


def test_grouped_plans(dev, ctxs):
    """Rows that TMA can read take the tensor cores: few slots one CTA per tile
    with the row split, long calls pairs; others the kernel for any shape."""
    a = 1 << 32

    def plan(S, E, N, H, x=a, gather=False, which="auto"):
        return farn.farn_plan_grouped_matmul(
            ctxs[which].handle, x, S, 3 * a if gather else 0, S, 2 * a, E, N, H, 4 * a)[:2]
    assert plan(8, 64, 2048, 7168, gather=True) == ("tensor", 1)
    assert plan(1, 64, 2048, 7168, gather=True) == ("tensor", 4)
    assert plan(2, 8, 1024, 2048) == ("tensor", 4)
    assert plan(30, 32, 1200, 5000, gather=True) == ("tensor", 4)
    assert plan(32768, 64, 4096, 7168, gather=True) == ("pair", 2)
    assert plan(32768, 1024, 4096, 7168, gather=True) == ("pair", 2)
    assert plan(8192, 1, 8192, 8192) == ("pair", 2)
    assert plan(64, 4, 512, 1001) == ("generic", 1)
    assert plan(64, 4, 512, 1000, x=a + 2) == ("generic", 1)
    assert plan(64, 4, 512, 1000, which="generic") == ("generic", 1)
    assert plan(64, 1024, 512, 1000, which="pair") == ("pair", 2)
    assert plan(64, 1024, 512, 1000, gather=True, which="split4") == ("tensor", 4)


# ------------------------------------------------------------- together
def moe_layer(x, logits, up, down, residual, weight, K, out=None):
    experts, gates, index, rows, offsets = farn.moe_route(logits, K)
    h = torch.relu(farn.grouped_matmul(x, up, offsets, rows))
    y = farn.grouped_matmul(h, down, offsets)
    return farn.moe_combine(y, index, gates, residual, weight, 1e-6, out=out)


def layer_inputs(dev, T, E, H, F, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731
    x, res = r(T, H).to(torch.bfloat16), r(T, H).to(torch.bfloat16)
    up = (r(E, F, H) * H ** -0.5).to(torch.bfloat16)
    down = (r(E, H, F) * F ** -0.5).to(torch.bfloat16)
    weight = (1 + 0.1 * r(H)).to(torch.bfloat16)
    return x, 2 * r(T, E), up, down, res, weight


def layer_reference(x, logits, up, down, res, K):
    e, gates, *_ = route_reference(logits, K, True)
    acc = torch.zeros_like(x, dtype=torch.float64)
    for t in range(x.shape[0]):
        for k in range(K):
            if e[t, k] < 0:
                continue
            h = (up[e[t, k]].double() @ x[t].double()).to(torch.bfloat16).double().relu()
            y = (down[e[t, k]].double() @ h).to(torch.bfloat16).double()
            acc[t] += gates[t, k] * y
    return acc + res.double()


@pytest.mark.parametrize("T", [1, 20, 150])
def test_moe_layer(dev, T):
    """Router, both products and the combine in a row; one token's logits are
    all masked, so it keeps its residual.  Each intermediate bf16 value is
    off by one rounding: half a step (2^-8) of y and of what h's rounding
    carries through |down|, as of reduced and residual_out."""
    K, E, H, F = 3, 9, 256, 320
    x, logits, up, down, res, weight = layer_inputs(dev, T, E, H, F, 20 + T)
    if T > 1:
        logits[T // 2] = -INF
    red, ro, nrm = moe_layer(x, logits, up, down, res, weight, K)
    want = layer_reference(x, logits, up, down, res, K)
    # |y| <= |down| |h|: the rounding of h may differ between the two sides by
    # a step where the sums do, so each term carries 2^-7 of its magnitudes
    e, gates, *_ = route_reference(logits, K, True)
    mag = torch.zeros_like(want)
    for t in range(T):
        for k in range(K):
            if e[t, k] >= 0:
                h = (up[e[t, k]].double() @ x[t].double()).abs()
                mag[t] += gates[t, k] * (down[e[t, k]].double().abs() @ h)
    tol = 2.0 ** -7 * (mag + want.abs() + res.double().abs()) * 2
    assert ((ro.double() - want).abs() <= tol).all()
    if T > 1:
        assert torch.equal(ro[T // 2], res[T // 2])


def test_moe_layer_in_a_graph_and_on_streams(dev):
    """Captured and replayed on new inputs, and run on two streams at once:
    the same bits as eager calls on one stream."""
    K, E, H, F, T = 4, 16, 512, 256, 70
    ins = [layer_inputs(dev, T, E, H, F, s) for s in (31, 32)]
    eager = [[t.clone() for t in moe_layer(*i, K)] for i in ins]
    static = [t.clone() for t in ins[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe_layer(*static, K)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = moe_layer(*static, K)
    for i, want in zip(ins, eager):
        for dst, src in zip(static, i):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    results = []
    for _ in range(5):
        for s, i in zip(streams, ins):
            with torch.cuda.stream(s):
                results.append(moe_layer(*i, K))
    torch.cuda.synchronize()
    for n, r in enumerate(results):
        for a, b in zip(r, eager[n % 2]):
            assert torch.equal(a, b)


def test_prepared_layer_reuses_its_buffers(dev):
    """Prepared calls, launched again after their inputs changed in place, give
    the immediate calls' bits, into their own outputs or into given ones."""
    K, E, H, F, T = 2, 8, 128, 192, 33
    x, logits, up, *_ = layer_inputs(dev, T, E, H, F, 61)
    other = layer_inputs(dev, T, E, H, F, 62)
    route = farn.prepare_moe_route(logits, K, renormalize=False)
    _, _, _, rows, offsets = route.outputs
    given = torch.empty(T * K, F, dtype=torch.bfloat16, device=dev)
    gather = farn.prepare_grouped_matmul(x, up, offsets, rows, out=given)
    back = torch.empty(E, H, F, dtype=torch.bfloat16, device=dev).copy_(up.transpose(1, 2))
    down = farn.prepare_grouped_matmul(given, back, offsets)
    for again in range(3):
        if again:
            x.copy_(other[0]), logits.copy_(other[1].roll(again, 0))
        a, h, y = route(), gather(), down()
        assert h is given
        b = farn.moe_route(logits, K, renormalize=False)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        want = farn.grouped_matmul(x, up, b[4], b[3])
        assert torch.equal(h, want)
        assert torch.equal(y, farn.grouped_matmul(want, back, b[4]))


@pytest.mark.parametrize("prepared", [False, True])
def test_layer_on_a_given_stream(dev, prepared):
    """The calls run on the stream that they are given: behind what it has to
    do first, here the inputs, while the current stream stays idle."""
    K, E, H, F, T = 3, 8, 128, 72, 50
    x, logits, up, *_ = layer_inputs(dev, T, E, H, F, 63)
    want_r = farn.moe_route(logits, K)
    want_h = farn.grouped_matmul(x, up, want_r[4], want_r[3])
    late = [torch.zeros_like(t) for t in (x, logits)]
    side = torch.cuda.Stream()
    out = [torch.empty_like(t) for t in want_r]
    h = torch.empty_like(want_h)
    torch.cuda.synchronize()
    if prepared:
        calls = [farn.prepare_moe_route(late[1], K, out=out, stream=side),
                 farn.prepare_grouped_matmul(late[0], up, out[4], out[3], out=h, stream=side)]
    else:
        calls = [lambda: farn.moe_route(late[1], K, out=out, stream=side),
                 lambda: farn.grouped_matmul(late[0], up, out[4], out[3], out=h, stream=side)]
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        late[0].copy_(x), late[1].copy_(logits)
    for call in calls:
        call()
    assert torch.cuda.current_stream().query() and not side.query()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want_r)) and torch.equal(h, want_h)


def test_context_of_another_device_is_refused(dev):
    x, logits, up, *_ = layer_inputs(dev, 4, 4, 64, 64, 1)
    off = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device=dev)
    other = farn.Context(0)
    other.device = 1
    for call in (lambda: farn.moe_route(logits, 2, ctx=other),
                 lambda: farn.grouped_matmul(x, up, off, ctx=other),
                 lambda: farn.nvfp4_quantize(x, 1.0, ctx=other)):
        with pytest.raises(ValueError, match="device"):
            call()


def test_long_route_in_a_graph(dev):
    """The three kernels of a long routing call, captured and replayed on new
    logits, twice in one graph."""
    T, E, K = 3000, 40, 4
    x = normal(dev, T, E, 41, torch.float32)
    y = normal(dev, T, E, 42, torch.float32)
    farn.moe_route(x, K)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a, b = farn.moe_route(x, K), farn.moe_route(y, K, renormalize=False)
    x.copy_(normal(dev, T, E, 43, torch.float32))
    y[::3] = -INF
    graph.replay()
    torch.cuda.synchronize()
    for got, want in ((a, farn.moe_route(x, K)), (b, farn.moe_route(y, K, renormalize=False))):
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def test_two_threads_with_one_context(dev):
    """Calls of two host threads on streams of their own share a context."""
    import threading
    ins = [layer_inputs(dev, 40 + 90 * i, 8, 256, 512, 51 + i) for i in range(2)]
    want = [[t.clone() for t in moe_layer(*i, 2)] for i in ins]
    torch.cuda.synchronize()
    bad = []

    def work(n):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = moe_layer(*ins[n], 2)
                s.synchronize()
                if not all(torch.equal(g, w) for g, w in zip(got, want[n])):
                    bad.append(n)
    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_context_without_the_tensor_cores(dev):
    """Where the set-up of the router and of the tensor-core kernels fails the
    context serves the rest: the norm's bits are the same, the products take
    their slower kernel, the router says that it is not there."""
    ctx = make_ctx(FARN_FAULT_INJECT="setup")
    x, logits, up, _, res, weight = layer_inputs(dev, 40, 4, 64, 72, 2)
    for a, b in zip(farn.forward([x, x], res, weight, 1e-6, ctx=ctx),
                    farn.forward([x, x], res, weight, 1e-6)):
        assert torch.equal(a, b)
    with pytest.raises(farn.FarnError) as e:
        farn.moe_route(logits, 2, ctx=ctx)
    assert e.value.status == farn.FARN_ERR_CUDA
    offsets = make_groups([10, 0, 25, 5])
    w = integer((4, 72, 64), dev, 28)
    a = 1 << 32
    assert farn.farn_plan_grouped_matmul(ctx.handle, a, 40, 0, 40, 2 * a, 4, 72, 64,
                                         3 * a)[0] == "generic"
    xi = integer((40, 64), dev, 29)
    got = farn.grouped_matmul(xi, w, torch.from_numpy(offsets).to(dev), ctx=ctx)
    want, _ = grouped_reference(xi, w, offsets, None, 40)
    check_exact(got, want, offsets, "no tensor cores")
    # scales of 1: products are multiples of 1/4 and exact
    q = torch.randint(0, 256, (40, 32), device=dev, dtype=torch.uint8,
                      generator=torch.Generator(device=dev).manual_seed(30))
    s = torch.full((40, 4), 0x38, device=dev, dtype=torch.uint8)
    assert torch.equal(farn.nvfp4_matmul(q, s, 1.0, q, s, 1.0, ctx=ctx),
                       farn.nvfp4_matmul(q, s, 1.0, q, s, 1.0))
    for a, b in zip(farn.nvfp4_quantize(x, 100.0, ctx=ctx), farn.nvfp4_quantize(x, 100.0)):
        assert torch.equal(a, b)
    ctx.close()


def test_launch_fault_reaches_the_caller(dev):
    bad = make_ctx(FARN_FAULT_INJECT="launch")
    x, logits, up, *_ = layer_inputs(dev, 4, 4, 64, 64, 1)
    off = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device=dev)
    with pytest.raises(farn.FarnError) as e:
        farn.moe_route(logits, 2, ctx=bad)
    assert e.value.status == farn.FARN_ERR_CUDA
    with pytest.raises(farn.FarnError) as e:
        farn.grouped_matmul(x, up, off, ctx=bad)
    assert e.value.status == farn.FARN_ERR_CUDA
