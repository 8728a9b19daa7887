"""The delta rule's and the state cache's calls on a stream beside a busy current one."""
import pytest

from tests import delta_ref as ref
from tests.test_delta_gpu import SIMT, TENSOR, on_gpu, run_packed

pytestmark = pytest.mark.gpu

CYCLES = 800_000_000  # of a busy stream: four tenths of a second


def held_back(shapes, cycles=CYCLES):
    """Queues a long wait on the current stream and, behind it, fills of tensors of these shapes, whose memory is
    handed back at once: whatever is allocated on the current stream next may get it before they are filled."""
    import torch
    torch.cuda._sleep(cycles)
    for shape, dtype in shapes:
        torch.empty(shape, dtype=dtype, device="cuda").fill_(77)


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("handle", [False, True])
def test_prefill(cuda_lib, kernel, handle):
    """Outputs and workspace are not memory that work queued on the current stream still writes."""
    import torch
    cfg = ref.config(nheads=8, ngroups=2)
    cu = [0, 100, 100, 290]
    g = on_gpu(ref.inputs(cfg, 290, 3, seed=2))
    y0, h0 = run_packed(cuda_lib, cfg, g, cu, True, kernel)
    n = cuda_lib.delta_varlen_workspace_size(cfg, cu, kernel)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    shapes = [(y0.shape, y0.dtype), (h0.shape, h0.dtype), ((n,), torch.uint8)]
    for cycles in (100, CYCLES):  # once to have the stream's memory and the kernels in place: getting them would wait
        torch.cuda.synchronize()
        held_back(shapes, cycles)
        y, h = run_packed(cuda_lib, cfg, g, cu, True, kernel, stream=side.cuda_stream if handle else side)
    side.synchronize()
    assert not torch.cuda.current_stream().query(), "the current stream was to be busy"
    with torch.cuda.stream(side):
        early = torch.equal(y, y0) and torch.equal(h, h0)
    torch.cuda.synchronize()
    assert early and torch.equal(y, y0) and torch.equal(h, h0)
    assert cuda_lib.get_device_error() == 0


@pytest.mark.parametrize("slots", [None, [2, -1, 0]])
def test_decode(cuda_lib, slots):
    """y, zero where a row is skipped, is not erased by a fill that waits on the current stream."""
    import torch
    cfg = ref.config(nheads=8, ngroups=2)
    g = on_gpu(ref.inputs(cfg, 3, 3, seed=4))
    rows = [g[x] for x in ("q", "k", "v", "dt", "b")]
    at = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    want_state = g["h0"].clone()
    want = cuda_lib.delta_decode_step(cfg, *rows, g["A"], g["dt_bias"], want_state, at)
    side = torch.cuda.Stream()
    for cycles in (100, CYCLES):
        state = g["h0"].clone()
        torch.cuda.synchronize()
        held_back([(want.shape, want.dtype)], cycles)
        y = cuda_lib.delta_decode_step(cfg, *rows, g["A"], g["dt_bias"], state, at, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query(), "the current stream was to be busy"
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(state, want_state)


def test_what_is_handed_back_waits_for_the_current_stream(cuda_lib):
    """Outputs made for a side stream, used on the current one and dropped: the next call's are other memory until
    that use is done."""
    import torch
    cfg = ref.config(nheads=8, ngroups=2)
    g = on_gpu(ref.inputs(cfg, 200, 1, seed=4))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h = run_packed(cuda_lib, cfg, g, [0, 200], True, TENSOR, stream=side)
    side.synchronize()
    want, other = y.clone(), dict(g, v=2 * g["v"])
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    copy = y.clone()  # on the current stream, behind the wait
    del y, h
    run_packed(cuda_lib, cfg, other, [0, 200], True, TENSOR, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


def test_captured_on_a_forked_stream(cuda_lib):
    """In a graph, on a stream that forks from the captured one and joins it again."""
    import torch
    cfg = ref.config(nheads=8, ngroups=2)
    g = on_gpu(ref.inputs(cfg, 200, 1, seed=6))
    want = run_packed(cuda_lib, cfg, g, [0, 200], True, TENSOR)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = run_packed(cuda_lib, cfg, g, [0, 200], True, TENSOR, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
