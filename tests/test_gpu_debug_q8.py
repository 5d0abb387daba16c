"""The 8-bit cache's kernels under the debug build's index checks: a wrapping ring, several heads an
item, split units, a shard, and the read-back of every frame, with the release build's bits."""
import pytest
import torch

from causal_video_diffusion_b200 import binding
from tests.test_gpu_debug_build import dbg  # noqa: F401 (a fixture)
from tests.test_gpu_q8 import draw, shape_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dims,shard", [
    ((1, 2, 64, 4, 6, (24, 20, 20), 3), None),
    ((2, 3, 128, 1, 43, (44, 42, 42), 1), None),         # key tiles with one valid key
    ((2, 4, 128, 9, 31, (44, 42, 42), 2), None),
    ((1, 5, 64, 7, 9, (24, 20, 20), 2), (1, 2, 3, 8)),
    ((1, 12, 128, 30, 52, (44, 42, 42), 3), None),       # split units and their merges
])
def test_checks_hold_and_change_nothing(cuda_lib, dbg, dims, shard):  # noqa: F811
    shape = shape_of(*dims)
    F, cap, chunks = shape.chunk_frames, 2 * shape.chunk_frames + 1, 4
    acts = shape if shard is None else shape_of(shard[2], shard[3], *dims[2:])
    caches = [mod.LayerCacheQ8(shape.B, shape.H, shape.D, shape.Hg, shape.Wg, shape.d_t, shape.d_h,
                               shape.d_w, cap_frames=cap, max_pos_t=chunks * F, theta=shape.theta,
                               shard=shard) for mod in (binding, dbg)]
    for c in range(chunks):
        q, k, v = draw(acts, 7 * c)
        window = min(cap, (c + 1) * F)
        first = (c + 1) * F - window
        got = []
        for cache in caches:
            qo = cache.rope_kv_append(q, k, v, c * F, F, q_out=torch.zeros_like(q))
            out = cache.window_attn(qo, window, out=torch.zeros_like(q))
            got.append((qo, out, *cache.read_frames(first, window)))
        torch.cuda.synchronize()
        assert [cache.device_error() for cache in caches] == [0, 0]
        assert all(torch.equal(a, b) for a, b in zip(*got))
    with pytest.raises(dbg.UnstepError):
        caches[1].read_frames(-1, 1)
    with pytest.raises(binding.UnstepError):
        caches[0].read_frames(-1, 1)
