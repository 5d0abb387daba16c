"""Outputs of the 8-bit cache's calls that lie across an input, the cache or each other, through the C
ABI: refused before a launch (the cache's pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from causal_video_diffusion_b200 import binding as B
from tests.test_q8_cache import L, c_elements, cache  # noqa: F401 (L: a fixture)

P, Q = 0x800000, 0x900000
CHUNK = 2 * c_elements(cache(), 3)                     # bytes of the latest chunk's queries
CODES, SCALES = 2 * 3 * 6 * 24 * 64, 2 * 3 * 6 * 24 * 2
ROWS = [(0x100000, CODES), (0x200000, CODES), (0x600000, SCALES), (0x700000, SCALES)]
ARG = B.UNSTEP_ERR_ARG


def test_attention(L):  # noqa: F811
    def attn(q, out):
        return L.unstep_q8_window_attn(q, ctypes.byref(cache()), 6, out, None)

    for d in (0, 16, -16, CHUNK - 16, 16 - CHUNK):
        assert attn(P, P + d) == ARG, d
    for at, n in ROWS:
        for d in (0, n - 16, 16 - CHUNK):
            assert attn(P, at + d) == ARG, (at, d)


def test_append(L):  # noqa: F811
    g = B.unstep_grid_t(3, 4, 6)
    c = cache()
    for at, n in ROWS:
        for d in (0, n - 16, 16 - CHUNK):
            assert L.unstep_q8_rope_kv_append(P, at + d, Q, Q, ctypes.byref(c), 9, g, None) == ARG
    assert (c.base.frames_written, c.base.last_chunk_start) == (9, 6)


def test_read(L):  # noqa: F811
    n_out = 2 * 2 * 3 * 2 * 24 * 64                     # two frames

    def read(k, v):
        return L.unstep_q8_cache_read(ctypes.byref(cache()), 7, 2, k, v, None)

    for d in (0, 16, -16, n_out - 16, 16 - n_out):
        assert read(P, P + d) == ARG, d
    for at, n in ROWS:
        for d in (0, n - 16, 16 - n_out):
            for k, v in ((at + d, P), (P, at + d), (at + d, None), (None, at + d)):
                assert read(k, v) == ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on made-up addresses")
def test_what_shares_no_byte_is_not_refused(L):  # noqa: F811
    ref = ctypes.byref
    gone = B.UNSTEP_ERR_CUDA
    for d in (CHUNK, -CHUNK):
        assert L.unstep_q8_window_attn(P, ref(cache()), 6, P + d, None) == gone
    for at, n in ROWS:
        for d in (n + -n % 16, -CHUNK):
            assert L.unstep_q8_window_attn(P, ref(cache()), 6, at + d, None) == gone
    for k, v in ((P, Q), (P, None), (None, P)):
        assert L.unstep_q8_cache_read(ref(cache()), 7, 2, k, v, None) == gone
    for q_out in (P, Q, Q + 0x100000, P - CHUNK):        # q itself, k and v, and apart
        assert L.unstep_q8_rope_kv_append(P, q_out, Q, Q, ref(cache()), 9, B.unstep_grid_t(3, 4, 6),
                                          None) == gone
