"""The native side of the binding beside other threads, and its errors."""
import ctypes
import threading
import time

import pytest
import torch

from causal_video_diffusion_b200 import binding
from causal_video_diffusion_b200.binding import Norm
from tests import q8_reference as R
from tests.test_gpu_q8 import draw, shape_of
from tests.test_host_calls import load

pytestmark = pytest.mark.gpu


def test_other_threads_run_during_a_call(cuda_lib):
    """A launch may wait for the device.  In its place here: poll(), which takes the norm call's first
    three arguments (rows, their type 0 as the number of descriptors, their stride 500 as the wait in
    milliseconds) and returns 0."""
    poll = ctypes.cast(ctypes.CDLL(None).poll, ctypes.c_void_p).value
    m = load(binding.HOST_PATH)
    m.bind(binding.UnstepError, poll, poll, poll, poll, poll)
    x = torch.zeros((1, 500), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    turns, stop = [0], threading.Event()

    def count():
        while not stop.is_set():
            turns[0] += 1
            time.sleep(0.005)

    t = threading.Thread(target=count)
    t.start()
    try:
        before, t0 = turns[0], time.monotonic()
        assert m.norm_modulate(x, Norm(), out, None) is out
        during, took = turns[0] - before, time.monotonic() - t0
    finally:
        stop.set()
        t.join()
    assert took > 0.45 and during >= 20, (took, during)


def test_two_threads_with_caches_of_their_own(cuda_lib):
    """Calls of two threads at once, each on its own stream and tensors: the bits of the same calls
    one after the other."""
    shape = shape_of(1, 2, 64, 4, 6, (24, 20, 20), 1)
    n = Norm("rms", 1e-6)

    def work(seed, stream, got):
        with torch.cuda.stream(stream):
            cache = R.make_cache(shape, 4, 40, stream=stream)
            for c in range(30):
                q, k, v = draw(shape, 100 * seed + c)
                binding.norm_modulate(k.view(24, 128), n, out=k.view(24, 128))
                cache.rope_kv_append(q, k, v, c, 1)
                got.append(cache.window_attn(q, min(4, c + 1)))
                got += cache.read_frames(c, 1)
            stream.synchronize()

    streams = [torch.cuda.Stream() for _ in range(2)]
    alone, together = [[], []], [[], []]
    for i in range(2):
        work(i, streams[i], alone[i])
    threads = [threading.Thread(target=work, args=(i, streams[i], together[i])) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(alone, together):
        assert len(a) == len(b) == 90 and all(torch.equal(x, y) for x, y in zip(a, b))


def test_out_of_memory_is_torchs_exception(cuda_lib):
    """An output that does not fit raises torch.OutOfMemoryError, as torch's own allocations do."""
    x = torch.zeros((1 << 19, 1024), dtype=torch.bfloat16, device="cuda")     # 1 GiB
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    fraction = (torch.cuda.memory_reserved() + (1 << 28)) / total
    torch.cuda.set_per_process_memory_fraction(fraction)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            binding.norm_modulate(x, Norm())
        with pytest.raises(torch.OutOfMemoryError):
            binding.gate_residual_norm(x, x, next=Norm())
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert binding.norm_modulate(x[:4], Norm()).shape == (4, 1024)
