"""Outputs that the norms' and the 8-bit cache's calls make for an explicit stream: whose memory they
take, and for how long it stays theirs."""
import pytest
import torch

from causal_video_diffusion_b200 import binding
from causal_video_diffusion_b200.binding import Norm
from tests import q8_reference as R
from tests.test_gpu_q8 import draw, shape_of

pytestmark = pytest.mark.gpu

LONG = 20_000_000      # clocks that a stream is kept busy: about 10 ms


def make_calls():
    """Calls that return new tensors of N bf16 elements each."""
    shape = shape_of(1, 4, 64, 16, 16, (24, 20, 20))
    cache = R.make_cache(shape, 2, 4)
    q, k, v = draw(shape, 1)
    cache.rope_kv_append(q, k, v, 0, 1)
    x = q.view(256, 256).clone()
    y = k.view(256, 256).clone()
    x_out = torch.empty_like(x)
    torch.cuda.synchronize()
    return 256 * 256, [
        lambda s: [binding.norm_modulate(x, Norm(), stream=s)],
        lambda s: [binding.gate_residual_norm(x, y, next=Norm(), x_out=x_out, stream=s)[1]],
        lambda s: [cache.window_attn(q, 1, stream=s)],
        lambda s: list(cache.read_frames(0, 1, stream=s)),
    ]


@pytest.mark.parametrize("which", range(4))
def test_new_outputs_leave_the_current_streams_memory(cuda_lib, which):
    """Temporaries freed on the current stream while a kernel there has yet to read them: a call on
    another stream, which does not wait for that kernel, must not be given their memory."""
    n, calls = make_calls()
    call = calls[which]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    temps = [torch.full((n,), float(i), dtype=torch.bfloat16, device="cuda") for i in range(6)]
    torch.cuda.synchronize()
    where = {t.data_ptr() for t in temps}
    torch.cuda._sleep(LONG)
    kept = [t.clone() for t in temps]
    del temps
    got = call(side)
    assert not where & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for i, t in enumerate(kept):
        assert bool((t == float(i)).all())
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("which", range(4))
def test_new_outputs_outlive_the_current_streams_work(cuda_lib, which):
    """Used on the current stream and dropped before that work has run: the memory is not handed out
    on the call's stream meanwhile."""
    n, calls = make_calls()
    call = calls[which]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(LONG)
    kept = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        others = [torch.full((n,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, kept)) and len(others) == 4


def test_explicit_streams_in_a_graph(cuda_lib):
    """Calls on a stream forked inside a capture, their outputs made there and used behind the join."""
    n, calls = make_calls()
    want = [t.clone() for c in calls for t in c(None)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        made = [t for c in calls for t in c(side)]
        torch.cuda.current_stream().wait_stream(side)
        held = [t + 0 for t in made]
        del made
    for _ in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_a_stream_of_another_kind_is_taken(cuda_lib):
    """An external stream (a handle alone) and the default stream, given explicitly."""
    n, calls = make_calls()
    side = torch.cuda.Stream()
    for s in (torch.cuda.ExternalStream(side.cuda_stream), torch.cuda.default_stream()):
        for c in calls:
            want = [t.clone() for t in c(None)]
            torch.cuda.synchronize()
            got = c(s)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(AttributeError):
        calls[0](7)
