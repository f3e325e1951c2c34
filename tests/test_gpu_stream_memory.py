"""Calls with a stream of their own, whose outputs and workspaces the wrappers allocate, next to work on the current
stream that still waits for its turn. Memory that was just freed on the current stream, with a kernel ahead that writes
to it, must not become such an output; nor may an output's memory be handed out on the given stream while the
current stream still has to read it."""
import functools

import pytest
import torch

import async_stage_tile_amd as pt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
LONG = 20_000_000       # clock ticks that the current stream is kept busy, about 10 ms


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[stream memory] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


class TooEarly(Exception):
    """The stream that should have been behind was not, so the case shows nothing."""


def several_tries(test):
    """Few hardware queues carry all streams, and which one a stream gets changes with time."""
    @functools.wraps(test)
    def run(name):
        for _ in range(6):
            try:
                return test(name)
            except TooEarly:
                torch.cuda.synchronize()
        pytest.skip("the streams share a queue")
    return run


def independent_stream():
    """A stream whose work does not wait behind the current stream's: few hardware queues carry all streams."""
    held = []
    for _ in range(8):
        held.append(torch.cuda.Stream(device=DEV))
        torch.cuda.synchronize()
        torch.cuda._sleep(LONG)
        with torch.cuda.stream(held[-1]):
            torch.cuda._sleep(1)
        held[-1].synchronize()
        apart = not torch.cuda.current_stream().query()
        torch.cuda.synchronize()
        if apart:
            return held[-1]
    raise TooEarly


def reserve(sizes, count):
    """Memory of these sizes in the current stream's pool: fetching it later would wait for the device."""
    kept = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(count)]
    del kept


def ints(shape, low, high, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(low, high + 1, shape, device=DEV, generator=g).to(torch.float32).to(dtype)


def calls():
    x, w = ints((512, 1024), -4, 4, BF, 1), ints((1024,), -4, 4, BF, 2)
    a8, w8 = ints((128, 8192), -4, 4, E4, 3), ints((256, 8192), -4, 4, E4, 4)
    one = torch.ones(256, device=DEV)
    a4, s4 = ints((40, 4096), -4, 4, BF, 5), torch.ones(256, 32, device=DEV, dtype=BF)
    q4 = ints((256, 2048), 0, 255, torch.uint8, 6)
    half, gb = ints((1024, 1024), -4, 4, torch.float16, 7), ints((1024, 512), -2, 2, BF, 8)
    assert pt.pipe_gemm_fp8_workspace_bytes(128, 256, 8192) > 0 and pt.pipe_gemm_w4_workspace_bytes(40, 256, 4096) > 0
    assert pt.pipe_rmsnorm_backward_workspace_bytes(512, 1024) > 0
    return {
        "rmsnorm": lambda s: pt.pipe_rmsnorm(x, w, residual=x, out_dtype=E4, stream=s),
        "rmsnorm_backward": lambda s: pt.pipe_rmsnorm_backward(x, x, w, dh=x, stream=s),
        "gemm_fp8": lambda s: pt.pipe_gemm_fp8(a8, one[:128], w8.t(), one, stream=s),
        "gemm_w4": lambda s: pt.pipe_gemm_w4(a4, q4, s4, stream=s),
        "tile_copy": lambda s: pt.pipe_tile_copy(half, checksums=True, stream=s),
        "rowsum": lambda s: pt.pipe_rowsum(half, stream=s, split=4),
        "gemm_mainloop": lambda s: pt.pipe_gemm_mainloop(x, gb, stream=s),
    }


def tensors(out):
    return [t.view(torch.uint8).clone() for t in (out if isinstance(out, tuple) else (out,))]


def sizes(want):
    """Every size up to the largest output's, in steps of the allocator: workspaces are among them."""
    top = max(t.numel() for t in want)
    return sorted({n for n in (512, 1024, 2048, 65536, 1 << 20, 1 << 21, 1 << 22)} | {t.numel() for t in want if t.numel()}) + [top]


@pytest.mark.parametrize("name", ["rmsnorm", "rmsnorm_backward", "gemm_fp8", "gemm_w4", "tile_copy", "rowsum", "gemm_mainloop"])
@several_tries
def test_no_output_in_memory_that_the_current_stream_still_writes(name):
    call = calls()[name]
    want = tensors(call(None))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = independent_stream()
    blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes(want) for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    for b in blocks:
        b.fill_(0x55)           # behind the sleep
    blocks.clear()
    del b
    out = call(side)
    side.synchronize()
    early = torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    if early:
        raise TooEarly
    for got, ref in zip(tensors(out), want):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("name", ["rmsnorm", "rmsnorm_backward", "gemm_fp8", "gemm_w4", "tile_copy", "rowsum", "gemm_mainloop"])
@several_tries
def test_no_output_reused_before_the_current_stream_has_read_it(name):
    call = calls()[name]
    want = tensors(call(None))
    torch.cuda.synchronize()
    side = independent_stream()
    out = call(side)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.stream(side):
        reserve(sizes(want), 6)
    tensors(out)
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    got = tensors(out)          # copies, behind the sleep
    del out
    with torch.cuda.stream(side):
        for n in sizes(want):
            for _ in range(4):
                torch.full((n,), 0x55, dtype=torch.uint8, device=DEV)
    side.synchronize()
    early = torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    if early:
        raise TooEarly
    for g, ref in zip(got, want):
        assert torch.equal(g, ref)


@pytest.mark.parametrize("name", ["rmsnorm", "rmsnorm_backward", "gemm_fp8", "gemm_w4", "tile_copy", "rowsum", "gemm_mainloop"])
def test_captured_on_a_stream_that_joins_the_capture(name):
    """The given stream is forked from the captured one: outputs and workspaces come from the graph's own pool, and every
    replay writes them again."""
    call = calls()[name]
    want = tensors(call(None))
    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(device=DEV), torch.cuda.Stream(device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        out = call(side)
        main.wait_stream(side)
    out = out if isinstance(out, tuple) else (out,)
    for _ in range(4):
        for t in out:
            t.view(torch.uint8).fill_(0x55)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        call(None)
        torch.full((1 << 20,), 7.0, device=DEV).add_(1.0)
        torch.cuda.synchronize()
        for got, ref in zip(tensors(out), want):
            assert torch.equal(got, ref)


def inputs_and_calls():
    """As calls(), with the operands apart: (operands, what to do with them)."""
    one = torch.ones(256, device=DEV)
    rows = lambda: ints((512, 1024), -4, 4, BF, 1)
    return {
        "rmsnorm": ((rows(), ints((1024,), -4, 4, BF, 2), ints((512, 1024), -4, 4, BF, 9)),
                    lambda t, s: pt.pipe_rmsnorm(t[0], t[1], residual=t[2], stream=s)),
        "rmsnorm_backward": ((rows(), ints((512, 1024), -4, 4, BF, 9), ints((1024,), -4, 4, BF, 2), ints((512, 1024), -4, 4, BF, 10)),
                             lambda t, s: pt.pipe_rmsnorm_backward(t[0], t[1], t[2], dh=t[3], stream=s)),
        "gemm_fp8": ((ints((128, 8192), -4, 4, E4, 3), one[:128].clone(), ints((256, 8192), -4, 4, E4, 4), one),
                     lambda t, s: pt.pipe_gemm_fp8(t[0], t[1], t[2].t(), t[3], stream=s)),
        "gemm_w4": ((ints((40, 4096), -4, 4, BF, 5), ints((256, 2048), 0, 255, torch.uint8, 6),
                     torch.ones(256, 32, device=DEV, dtype=BF), ints((256, 32), 0, 15, torch.uint8, 7)),
                    lambda t, s: pt.pipe_gemm_w4(t[0], t[1], t[2], zeros=t[3], stream=s)),
        "tile_copy": ((ints((1024, 1024), -4, 4, torch.float16, 7),), lambda t, s: pt.pipe_tile_copy(t[0], stream=s)),
        "rowsum": ((ints((1024, 1024), -4, 4, torch.float16, 7),), lambda t, s: pt.pipe_rowsum(t[0], stream=s, split=4)),
        "gemm_mainloop": ((rows(), ints((1024, 512), -2, 2, BF, 8)),
                          lambda t, s: pt.pipe_gemm_mainloop(t[0], t[1], stream=s)),
    }


@pytest.mark.parametrize("name", ["rmsnorm", "rmsnorm_backward", "gemm_fp8", "gemm_w4", "tile_copy", "rowsum", "gemm_mainloop"])
@several_tries
def test_no_operand_reused_before_the_given_stream_has_read_it(name):
    """Operands that the caller drops right after the call, while the given stream has not begun it."""
    operands, call = inputs_and_calls()[name]
    want = tensors(call(operands, None))
    sizes_in = [t.numel() * t.element_size() for t in operands]
    side = independent_stream()
    call(operands, side)            # first calls of a stream may allocate
    reserve(sizes_in, 32)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    out = call(operands, side)
    del operands
    fills = [torch.full((n,), 0x55, dtype=torch.uint8, device=DEV) for n in sizes_in for _ in range(24)]
    torch.cuda.current_stream().synchronize()
    early = side.query()
    torch.cuda.synchronize()
    if early:
        raise TooEarly
    for got, ref in zip(tensors(out), want):
        assert torch.equal(got, ref)
