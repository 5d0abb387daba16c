"""The 8-bit cache's C ABI without a GPU: sizes, and refusals that return before any launch."""
import ctypes
import random

import pytest
import torch

from causal_video_diffusion_b200 import binding as B
from causal_video_diffusion_b200 import workloads as W
from tests import q8_reference as R

MAGIC_BF16, MAGIC_Q8 = 0x55535450, 0x55535138


@pytest.fixture(scope="module")
def L():
    from causal_video_diffusion_b200 import build
    build.build()
    return B.lib()


def cache(D=64, cap=6, magic=MAGIC_Q8, split=(24, 20, 20)):
    """Pointers are never dereferenced: only calls that fail their checks are made with it."""
    q = B.unstep_q8_cache_t()
    c = q.base
    c.B, c.H, c.D, c.Hg, c.Wg = 2, 3, D, 4, 6
    c.d_t, c.d_h, c.d_w, c.theta = *split, 10000.0
    c.cap_frames, c.max_pos_t = cap, 128
    c.k_cache, c.v_cache, c.slot_frame, c.cos_sin, c.dev_error = (
        0x100000, 0x200000, 0x300000, 0x400000, 0x500000)
    q.k_scale, q.v_scale = 0x600000, 0x700000
    c.frames_written, c.first_frame, c.last_chunk_start, c.last_chunk_frames = 9, 0, 6, 3
    c.initialized = magic
    return q


def test_sizes(L):
    q = cache()
    n = 2 * 3 * 6 * 24 * 64
    assert L.unstep_q8_cache_kv_bytes(ctypes.byref(q)) == n
    assert L.unstep_q8_cache_scale_bytes(ctypes.byref(q)) == n // 32
    head = 128 + 32
    assert L.unstep_q8_cache_state_bytes(ctypes.byref(q)) == head + 2 * n + 2 * n // 32
    q.base.D = 96
    for f in (L.unstep_q8_cache_kv_bytes, L.unstep_q8_cache_scale_bytes,
              L.unstep_q8_cache_state_bytes):
        assert f(ctypes.byref(q)) == 0 and f(None) == 0


def test_init_refusals(L):
    for field, value, want in (("k_scale", None, B.UNSTEP_ERR_ARG),
                               ("v_scale", 0x700008, B.UNSTEP_ERR_ALIGN)):
        q = cache()
        setattr(q, field, value)
        assert L.unstep_q8_cache_init(ctypes.byref(q), None) == want
    for field, value, want in (("k_cache", None, B.UNSTEP_ERR_ARG), ("B", 0, B.UNSTEP_ERR_ARG),
                               ("v_cache", 0x200004, B.UNSTEP_ERR_ALIGN),
                               ("d_t", 23, B.UNSTEP_ERR_ARG)):
        q = cache()
        setattr(q.base, field, value)
        assert L.unstep_q8_cache_init(ctypes.byref(q), None) == want
    assert L.unstep_q8_cache_init(None, None) == B.UNSTEP_ERR_ARG
    # a bf16 reset of an 8-bit cache would clear twice its buffers
    assert L.unstep_cache_init(ctypes.byref(cache().base), None) == B.UNSTEP_ERR_ARG


def test_append_refusals(L):
    P = 0x800000
    g = B.unstep_grid_t(3, 4, 6)

    def append(q=P, qo=P, k=P, v=P, c=None, f=9, grid=g):
        return L.unstep_q8_rope_kv_append(q, qo, k, v, ctypes.byref(c or cache()), f, grid, None)

    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None)):
        assert append(**kw) == B.UNSTEP_ERR_ARG
    for kw in (dict(q=P + 8), dict(qo=P + 2), dict(k=P + 4), dict(v=P + 1)):
        assert append(**kw) == B.UNSTEP_ERR_ALIGN
    assert append(c=cache(magic=MAGIC_BF16)) == B.UNSTEP_ERR_ARG
    assert append(c=cache(magic=0)) == B.UNSTEP_ERR_ARG
    assert append(f=3) == B.UNSTEP_ERR_FRAME_ORDER
    assert append(f=10) == B.UNSTEP_ERR_FRAME_ORDER
    assert append(f=127) == B.UNSTEP_ERR_ARG
    assert append(grid=B.unstep_grid_t(3, 4, 5)) == B.UNSTEP_ERR_SHAPE
    assert append(grid=B.unstep_grid_t(7, 4, 6)) == B.UNSTEP_ERR_WINDOW
    assert L.unstep_q8_rope_kv_append(P, P, P, P, None, 9, g, None) == B.UNSTEP_ERR_ARG
    # 2^31 vectors of eight channels in one chunk
    q = cache()
    q.base.Hg, q.base.Wg, q.base.cap_frames, q.base.B, q.base.H = 4096, 4096, 6, 1 << 10, 1
    assert append(c=q, grid=B.unstep_grid_t(3, 4096, 4096)) == B.UNSTEP_ERR_UNSUPPORTED
    q = cache()
    q.k_scale = None
    assert append(c=q) == B.UNSTEP_ERR_ARG
    assert (q.base.frames_written, q.base.last_chunk_start) == (9, 6)
    # q_out across q, k or v: the last thing checked before a launch
    n = 2 * c_elements(cache(), 3)
    far = P + 4 * n
    for kw in (dict(qo=P + 16), dict(qo=far, k=far + n - 16), dict(qo=far, v=far - n + 16),
               dict(q=far + 16, qo=far)):
        assert append(**kw) == B.UNSTEP_ERR_ARG, kw


def c_elements(q, frames):
    c = q.base
    return c.B * frames * c.Hg * c.Wg * c.H * c.D


def test_attention_and_read_refusals(L):
    P = 0x800000
    ref = ctypes.byref
    attn, read = L.unstep_q8_window_attn, L.unstep_q8_cache_read
    assert attn(None, ref(cache()), 3, P, None) == B.UNSTEP_ERR_ARG
    assert attn(P, ref(cache()), 3, None, None) == B.UNSTEP_ERR_ARG
    assert attn(P, None, 3, P, None) == B.UNSTEP_ERR_ARG
    assert attn(P + 8, ref(cache()), 3, P, None) == B.UNSTEP_ERR_ALIGN
    assert attn(P, ref(cache()), 3, P + 8, None) == B.UNSTEP_ERR_ALIGN
    assert attn(P, ref(cache()), 2, P, None) == B.UNSTEP_ERR_WINDOW
    assert attn(P, ref(cache()), 7, P, None) == B.UNSTEP_ERR_WINDOW
    assert attn(P, ref(cache(magic=MAGIC_BF16)), 3, P, None) == B.UNSTEP_ERR_ARG
    q = cache()
    q.base.frames_written = q.base.last_chunk_frames = 0
    assert attn(P, ref(q), 3, P, None) == B.UNSTEP_ERR_WINDOW
    assert read(ref(q), 0, 1, P, P, None) == B.UNSTEP_ERR_WINDOW
    assert read(ref(cache()), 6, 3, None, None, None) == B.UNSTEP_ERR_ARG
    assert read(ref(cache()), 6, 0, P, P, None) == B.UNSTEP_ERR_ARG
    assert read(ref(cache()), 6, 3, P + 8, P, None) == B.UNSTEP_ERR_ALIGN
    assert read(ref(cache(magic=MAGIC_BF16)), 6, 3, P, P, None) == B.UNSTEP_ERR_ARG
    for first, n in ((2, 1), (7, 3), (9, 1), (-1, 1), (2 ** 31 - 1, 2), (3, 2 ** 31 - 1)):
        assert read(ref(cache()), first, n, P, P, None) == B.UNSTEP_ERR_WINDOW


def test_state_refusals(L):
    q = cache()
    n = L.unstep_q8_cache_state_bytes(ctypes.byref(q))
    buf = (ctypes.c_ubyte * n)()
    assert L.unstep_q8_cache_save(ctypes.byref(q), buf, n - 1, None) == B.UNSTEP_ERR_ARG
    assert L.unstep_q8_cache_save(ctypes.byref(q), None, n, None) == B.UNSTEP_ERR_ARG
    assert L.unstep_q8_cache_restore(ctypes.byref(q), buf, n, None) == B.UNSTEP_ERR_ARG  # no magic
    assert L.unstep_q8_cache_restore(ctypes.byref(q), buf, 64, None) == B.UNSTEP_ERR_ARG
    assert L.unstep_q8_cache_restore(ctypes.byref(q), None, n, None) == B.UNSTEP_ERR_ARG


def test_reference_format_against_torch_and_by_search():
    """The test suite's own definition: rounding as torch's e4m3 cast, exponents by search."""
    rng = random.Random(5)
    x = torch.tensor([rng.uniform(-1, 1) * 2.0 ** rng.randint(-14, 8) for _ in range(4096)],
                     dtype=torch.float64)
    x = torch.cat([x, torch.tensor([448.0, 440.0, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, 17.0, 19.0, 21.0]
                                   + [0.0] * 24, dtype=torch.float64)])
    E = torch.zeros(x.numel() // 32, dtype=torch.int32)
    step = R.step_of(x, E)
    want = x.float().to(torch.float8_e4m3fn).double()
    assert torch.equal(torch.round(x / step) * step, want)
    for a in (448.0, 448.0 * (1 + 2.0 ** -40), 449.0, 896.0, 1.0, 1.75, 1.76, 2.0 ** -200, 0.0):
        b = torch.zeros(32, dtype=torch.float64)
        b[7] = -a
        e = R.E_MIN
        while a > 448 * 2.0 ** e:
            e += 1
        assert int(R.exponents(b)) == e
