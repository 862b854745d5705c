"""Which calls of the grouped FP8 product take a workspace, without a GPU: the
library's answer, and that the binding goes by it."""
import os
import subprocess
import types

import pytest

torch = pytest.importorskip("torch")

import rank_sum_residual_gb300 as farn  # noqa: E402
from rank_sum_residual_gb300 import _build  # noqa: E402

TENSOR, PAIR = 6, 7


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    lib = farn.build_library()
    exe = str(tmp_path_factory.mktemp("plan") / "probe")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["nvcc", "-std=c++17", "-I", _build.INCLUDE, "-I", _build.CSRC, "-o", exe,
                    os.path.join(here, "product_plan_probe.cu"), lib, "-Xlinker",
                    "-rpath=" + os.path.dirname(lib)], check=True)

    def query(*args):
        out = subprocess.run([exe, *map(str, args)], check=True, capture_output=True, text=True)
        return tuple(map(int, out.stdout.split()))
    return query


@pytest.mark.parametrize("S,E,N,H", [(64, 2, 8192, 1024), (64, 2, 7552, 256), (63, 2, 9700, 256),
                                     (8, 6, 512, 256), (512, 6, 2048, 256)])
def test_workspace_goes_with_the_plan(probe, S, E, N, H):
    status, variant, ctas, need = probe("experts", S, E, N, H)
    assert status == farn.FARN_OK
    if variant == PAIR:
        assert ctas == 2 and need == S * H + S * -(-H // 128) * 4
    else:
        assert variant == TENSOR and need == 0
    assert (variant == PAIR) == (S >= 64)


class Tensor:
    device = "dev"

    def __init__(self, shape, dtype):
        self.shape, self.dtype = shape, dtype

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return self.shape


@pytest.mark.parametrize("S,answer,status", [(1, 4000, 0), (64, 4000, 0), (65, 4000, 0),
                                             (500, 4000, 0), (64, 0, 0), (500, 0, 0),
                                             (7, 0, farn.FARN_ERR_INVALID_ARG)])
def test_the_binding_asks_for_every_call_with_rows(monkeypatch, S, answer, status):
    """Whatever the library answers is taken, for short calls too."""
    asked, made = [], []

    def workspace(handle, *sizes):
        asked.append(sizes[:4])
        sizes[4]._obj.value = answer
        return status

    def empty(shape, dtype, device):
        made.append(shape)
        return Tensor(shape, dtype)
    monkeypatch.setattr(farn, "_lib", types.SimpleNamespace(farn_fp8_grouped_workspace=workspace))
    monkeypatch.setattr(farn, "_torch", types.SimpleNamespace(
        uint8="u8", int32="i32", float32="f32", bfloat16="bf", empty=empty))
    monkeypatch.setattr(farn, "_current_raw_stream", lambda index: 0)
    ctx = types.SimpleNamespace(device=0, handle=1)
    x, xs = Tensor((9, 256), "u8"), Tensor((9, 2), "f32")
    w, ws = Tensor((3, 128, 256), "u8"), Tensor((3, 1, 2), "f32")
    offsets, rows = Tensor((4,), "i32"), Tensor((S,), "i32")
    args, _, _ = farn._fp8_grouped_args(x, xs, w, ws, offsets, rows, None, None, ctx, None)
    assert asked == [(S, 3, 128, 256)]
    assert args[-2] == answer and (args[-3] is not None) == bool(answer)
    assert made == [(S, 128)] + ([answer] if answer else [])
    # rows as they lie need none
    farn._fp8_grouped_args(x, xs, w, ws, offsets, None, None, None, ctx, None)
    assert len(asked) == 1
