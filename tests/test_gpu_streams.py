"""Calls on a given stream that make their own outputs: whose memory those are,
against the current stream's pending work before and after the call."""
import types

import pytest

torch = pytest.importorskip("torch")

import rank_sum_residual_gb300 as farn  # noqa: E402

pytestmark = pytest.mark.gpu

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32
LONG = 100_000_000          # cycles that the current stream is kept busy


@pytest.fixture(scope="module")
def calls():
    """name -> (function, arguments): every call that makes outputs."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    farn.build_library()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    g = torch.Generator(device=dev).manual_seed(1)
    normal = lambda *s: torch.randn(s, device=dev, generator=g).to(BF)  # noqa: E731
    T, H, E, N, K = 300, 512, 4, 256, 2
    x, w, logits = normal(T, H), normal(H), normal(T, E)
    _, gates, index, rows, offsets = farn.moe_route(logits, K)
    up, up8 = normal(E, N, H), farn.fp8_quantize(normal(E, N, H), 128)
    q8, q4 = farn.fp8_quantize(x), farn.nvfp4_quantize(x, 100.0)
    b8, b4 = farn.fp8_quantize(normal(N, H), 128), farn.nvfp4_quantize(normal(N, H), 100.0)
    q, k, v = normal(T, 4, 64), normal(T, 2, 64), normal(T, 2, 64)
    pos = torch.arange(T, device=dev, dtype=I32)
    freqs = torch.linspace(1.0, 0.001, 32, device=dev)
    cache = farn.kv_cache(T // 4, 4, 2, 64, "fp8", dev)
    slots = torch.randperm(T, device=dev, generator=g).to(I32)
    farn.kv_write(k, v, cache, slots)
    table = torch.arange(T // 4, device=dev, dtype=I32).view(1, -1)
    ends = torch.tensor([0, T], device=dev, dtype=I32)
    torch.cuda.synchronize()
    return dict(
        forward=(farn.forward, ([x, x], x, w, 1e-6)),
        forward_quant=(farn.forward_quant, ([x, x], x, w, 1e-6)),
        forward_nvfp4=(farn.forward_nvfp4, ([x, x], x, w, 1e-6, 100.0, False)),
        moe_combine=(farn.moe_combine, (normal(T * K, H), index, gates, x, w, 1e-6)),
        moe_route=(farn.moe_route, (logits, K)),
        grouped_matmul=(farn.grouped_matmul, (x, up, offsets, rows)),
        nvfp4_quantize=(farn.nvfp4_quantize, (x, 100.0)),
        nvfp4_dequantize=(farn.nvfp4_dequantize, (*q4, 100.0)),
        nvfp4_matmul=(farn.nvfp4_matmul, (*q4, 100.0, *b4, 100.0)),
        fp8_quantize=(farn.fp8_quantize, (x,)),
        fp8_matmul=(farn.fp8_matmul, (*q8, *b8)),
        fp8_grouped_matmul=(farn.fp8_grouped_matmul, (*q8, *up8, offsets, rows)),
        qk_norm_rope=(farn.qk_norm_rope, (q, k, w[:64], w[:64], 1e-6, pos, freqs)),
        qk_norm_rope_cache=(farn.qk_norm_rope_cache, (q, k, v, w[:64], w[:64], 1e-6, pos, freqs,
                                                      cache, slots)),
        kv_read=(farn.kv_read, (cache, table, ends, T)))


NAMES = ["forward", "forward_quant", "forward_nvfp4", "moe_combine", "moe_route",
         "grouped_matmul", "nvfp4_quantize", "nvfp4_dequantize", "nvfp4_matmul", "fp8_quantize",
         "fp8_matmul", "fp8_grouped_matmul", "qk_norm_rope", "qk_norm_rope_cache", "kv_read"]


def tensors(out):
    return [t for t in (out if isinstance(out, (tuple, list)) else (out,)) if t is not None]


def stream_of(t):
    """The stream that torch's allocator keeps a tensor's block for."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]


def same(got, want):
    return all(torch.equal(a.view(U8), b.view(U8)) for a, b in zip(tensors(got), tensors(want)))


@pytest.mark.parametrize("duck", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_lie_in_the_calls_streams_memory(calls, name, duck):
    f, args = calls[name]
    want = f(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    given = types.SimpleNamespace(cuda_stream=side.cuda_stream) if duck else side
    got = f(*args, stream=given)
    side.synchronize()
    assert same(got, want)
    assert {stream_of(t) for t in tensors(got)} == {side.cuda_stream}
    assert {stream_of(t) for t in tensors(want)} == {torch.cuda.current_stream().cuda_stream}


@pytest.mark.parametrize("name", NAMES)
def test_pending_work_keeps_its_memory(calls, name):
    """The current stream still has to read blocks of the outputs' sizes that the
    caller has dropped."""
    f, args = calls[name]
    want = tensors(f(*args))
    kept = [torch.empty(t.numel() * t.element_size(), dtype=U8, device=t.device) for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = [torch.full_like(t, 77) for t in kept]
    torch.cuda._sleep(LONG)
    for a, b in zip(kept, before):
        a.copy_(b)
    del before, b
    got = f(*args, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all((t == 77).all() for t in kept) and same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_dropped_outputs_stay_until_they_are_used(calls, name):
    """The caller makes the current stream wait for the call, uses an output there
    and drops it; the next call on the other stream takes other memory."""
    f, args = calls[name]
    want = tensors(f(*args))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = tensors(f(*args, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(LONG)
    copies = [t.clone() for t in got]
    at = {t.data_ptr() for t in got}
    del got
    again = tensors(f(*args, stream=side))
    assert not torch.cuda.current_stream().query()
    assert not at & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert same(copies, want) and same(again, want)


@pytest.mark.parametrize("name", NAMES)
def test_on_a_forked_stream_of_a_graph(calls, name):
    f, args = calls[name]
    want = [t.clone() for t in tensors(f(*args))]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        f(*args, stream=side)                    # dropped at once
        got = tensors(f(*args, stream=side))
        torch.cuda.current_stream().wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(2):
        for t in got + copies:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want) and same(copies, want)
