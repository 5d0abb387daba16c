"""How large a chunk the 8-bit append takes: fewer than 2^31 vectors of eight channels, no smaller limit.
The calls overlap q_out with k, which is refused behind the size check, so none is launched."""
import ctypes

import pytest

from causal_video_diffusion_b200 import binding as B
from tests.test_q8_cache import L, cache  # noqa: F401 (L: a fixture)

P = 0x800000


# D, B, H, frames, Hg, Wg: vectors = B * H * frames * Hg * Wg * D / 8
@pytest.mark.parametrize("D,Bn,H,frames,Hg,Wg,taken", [
    (128, 1, 1, 73, 7, 262657, True),          # 2^31 - 16
    (128, 1, 1, 8, 4096, 4096, False),         # 2^31
    (128, 1, 1, 5, 4096, 4096, True),          # above 2^30
    (128, 1, 1, 4, 4096, 4097, False),         # above 2^30, but a frame of more than 2^24 tokens
    (64, 1, 1, 16, 4096, 4096, False),         # 2^31
    (64, 7, 73, 1, 1, 262657 * 2, True),       # 2^31 - 16, in streams and heads
    (128, 1 << 15, 1 << 12, 1, 1, 1, False),   # 2^31, single tokens
    (64, 1 << 15, 1 << 12, 1, 1, 1, True),
    (128, 1 << 15, 1 << 15, 64, 4096, 4096, False),
])
def test_chunk_size(L, D, Bn, H, frames, Hg, Wg, taken):  # noqa: F811
    q = cache(D=D, cap=frames, split=(D, 0, 0))
    c = q.base
    c.B, c.H, c.Hg, c.Wg = Bn, H, Hg, Wg
    c.frames_written = c.last_chunk_start = c.first_frame = c.last_chunk_frames = 0
    assert (Bn * H * frames * Hg * Wg * D // 8 < 2 ** 31 and Hg * Wg <= 2 ** 24) == taken
    rc = L.unstep_q8_rope_kv_append(P, P + 16, P, P, ctypes.byref(q), 0,
                                    B.unstep_grid_t(frames, Hg, Wg), None)
    assert rc == (B.UNSTEP_ERR_ARG if taken else B.UNSTEP_ERR_UNSUPPORTED)
