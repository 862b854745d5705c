"""The grouped FP8 product with few gathered rows on the kernel that lays them
side by side first, against the definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import rank_sum_residual_gb300 as farn  # noqa: E402
from test_gpu_fp8 import (ctxs, dev, group_inputs, group_reference, spread,  # noqa: E402,F401
                          to_bf16, tolerance, whole)

pytestmark = pytest.mark.gpu


def workspace_of(call):
    return call._args[-2]


@pytest.mark.parametrize("counts,N,H", [([1], 64, 16), ([5], 128, 128), ([1, 0, 3], 72, 528),
                                        ([0, 33, 31], 264, 272), ([0, 0, 64], 513, 400)])
def test_few_rows(dev, ctxs, counts, N, H):  # noqa: F811
    c = ctxs["pair"]
    x, w, offsets, rows, S = group_inputs(dev, counts, N, H, True, whole, sum(counts) + N)
    if S > 2:
        rows[S // 2] = -1                               # zeros
        rows[S - 1] = x[0].shape[0]
    need = farn.farn_fp8_grouped_workspace(c.handle, S, len(counts), N, H)
    call = farn.prepare_fp8_grouped_matmul(*x, *w, offsets, rows, ctx=c)
    assert need == workspace_of(call) == S * H + S * -(-H // 128) * 4
    assert farn.farn_plan_fp8_grouped_matmul(c.handle, 1 << 32, x[0].shape[0], 2 << 32, S, 3 << 32,
                                             len(counts), N, H, 4 << 32, 5 << 32)[0] == "pair"
    want, _ = group_reference(x, w, offsets, rows, S)
    got = call()
    torch.cuda.synchronize()
    assert farn.farn_device_status(c.handle) == 0
    assert torch.equal(got, to_bf16(want))


def test_the_plans_own_border(dev, ctxs):  # noqa: F811
    """64 slots of two experts with many weights: pairs without being asked to."""
    counts, N, H = [23, 41], 8192, 1024
    c = ctxs["auto"]
    x, w, offsets, rows, S = group_inputs(dev, counts, N, H, True, whole, 9)
    call = farn.prepare_fp8_grouped_matmul(*x, *w, offsets, rows, ctx=c)
    need = farn.farn_fp8_grouped_workspace(c.handle, S, 2, N, H)
    assert need == workspace_of(call) == S * H + S * 8 * 4
    want, _ = group_reference(x, w, offsets, rows, S)
    assert torch.equal(call(), to_bf16(want))


def test_rounding_with_every_workspace(dev, ctxs):  # noqa: F811
    """Operands whose sums round: both kernels stay within the roundings of the
    definition, and each repeats bit for bit."""
    counts, N, H = [300, 500, 90], 256, 2064
    c = ctxs["pair"]
    x, w, offsets, rows, S = group_inputs(dev, counts, N, H, True, spread, 65)
    need = farn.farn_fp8_grouped_workspace(c.handle, S, len(counts), N, H)
    buf = torch.zeros(need + 32, dtype=torch.uint8, device=dev)
    want, mag = group_reference(x, w, offsets, rows, S)
    most = tolerance(want, mag, H)
    for ws in (None, buf[:need], buf[:need - 1], buf[1:1 + need], buf[:0]):
        out = [farn.fp8_grouped_matmul(*x, *w, offsets, rows, workspace=ws, ctx=c)
               for _ in range(2)]
        assert ((out[0].double() - want).abs() <= most).all()
        assert torch.equal(*out)
