"""The 8-bit KV cache on the GPU against its definition in 64 bits: append, read back, attention,
checkpoints, streams and graphs."""
import ctypes

import pytest
import torch

from causal_video_diffusion_b200 import binding
from causal_video_diffusion_b200 import workloads as W
from tests import parity as P
from tests import q8_reference as R

pytestmark = pytest.mark.gpu


def shape_of(B, H, D, Hg, Wg, split, frames=1):
    return W.LayerShape(B=B, H=H, D=D, Hg=Hg, Wg=Wg, d_t=split[0], d_h=split[1], d_w=split[2],
                        chunk_frames=frames)


# B, H, D, Hg, Wg, split, frames
SHAPES = [
    (1, 2, 64, 4, 6, (24, 20, 20), 3),
    (1, 1, 64, 1, 1, (64, 0, 0), 1),          # single tokens, one axis only
    (3, 5, 128, 3, 7, (44, 42, 42), 2),
    (2, 3, 128, 1, 43, (0, 62, 66), 3),       # 129 tokens in a chunk, no temporal axis
    (1, 12, 128, 9, 13, (44, 42, 42), 1),
    (2, 1, 64, 5, 5, (2, 60, 2), 4),
]


def draw(shape, seed, strong=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dims = (shape.B, shape.L, shape.H, shape.D)
    q, k, v = (torch.randn(dims, generator=g, device="cuda") for _ in range(3))
    if strong:
        k[..., :: 17] *= 30
        v[..., 1:: 29] *= 1e-3
    return tuple(t.to(torch.bfloat16) for t in (q, k, v))


def check_rows(shape, cache, k, v, first, frames):
    """The chunk's stored rows against the definition."""
    rows = R.ring_rows(shape, cache.c.cap_frames, first, frames, "cuda")
    kx = R.rotate(k, R.angles(shape, first, frames, "cuda")).transpose(1, 2)
    vx = v.double().transpose(1, 2)
    # v has no arithmetic before its rounding: exponents and values exactly
    vs = cache.v_scale.view(torch.uint8)[:, :, rows]
    assert torch.equal(vs.int() - 127, R.exponents(vx).int())
    vv = R.values(cache.v_codes[:, :, rows], cache.v_scale.view(torch.uint8)[:, :, rows])
    assert torch.equal(vv, R.stored(vx))
    # k: fp32 evaluation of the rotation with fp32 coefficients, four half-ulps of |a| + |b|
    E = cache.k_scale.view(torch.uint8)[:, :, rows].int() - 127
    ev = 4 * 2.0 ** -24 * (k.double()[..., 0::2].abs() + k.double()[..., 1::2].abs())
    ev = ev.repeat_interleave(2, -1).transpose(1, 2)
    lo, hi = R.exponents((kx.abs() - ev).clamp(min=0)), R.exponents(kx.abs() + ev)
    assert bool(((E >= lo) & (E <= hi)).all())
    kv = R.values(cache.k_codes[:, :, rows], cache.k_scale.view(torch.uint8)[:, :, rows])
    err = (kv - kx).abs()
    assert bool((err <= 0.5 * R.step_of(kx.abs() + ev, E) + ev).all())


@pytest.mark.parametrize("dims", SHAPES)
def test_append_matches_the_definition(cuda_lib, dims):
    """A ring that wraps: codes, scales, slots and rotated queries; rows of other frames and the
    buffers' surroundings stay as they were."""
    shape = shape_of(*dims)
    F, cap = shape.chunk_frames, shape.chunk_frames + 1
    cache = R.make_cache(shape, cap, 4 * F)
    bf = P.make_cache(shape, cap, 4 * F)
    for c in range(4):
        q, k, v = draw(shape, 10 * c + shape.D)
        before = [t.view(torch.uint8).clone() for t in (cache.k_codes, cache.v_codes, cache.k_scale,
                                                        cache.v_scale)]
        q_out, q0 = torch.full_like(q, 7.0), q.clone()
        assert cache.rope_kv_append(q, k, v, c * F, F, q_out=q_out) is q_out
        qb = q.clone()
        bf.rope_kv_append(qb, k, v, c * F, F)
        torch.cuda.synchronize()
        assert cache.device_error() == 0
        assert torch.equal(q, q0) and torch.equal(q_out, qb)
        check_rows(shape, cache, k, v, c * F, F)
        keep = torch.ones(cap * shape.Tf, dtype=torch.bool, device="cuda")
        keep[R.ring_rows(shape, cap, c * F, F, "cuda")] = False
        for was, t in zip(before, (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)):
            assert torch.equal(was[:, :, keep], t.view(torch.uint8)[:, :, keep])
        assert torch.equal(cache.slot_frame, bf.slot_frame)
        assert cache.last_chunk == bf.last_chunk and cache.frames_written == bf.frames_written
    # onto k itself, re-forwarding the same chunk: k is read before its place is written
    codes = cache.k_codes.view(torch.uint8).clone()
    over = k.clone()
    assert cache.rope_kv_append(q, over, v, 3 * F, F, q_out=over) is over
    assert torch.equal(over, q_out) and torch.equal(cache.k_codes.view(torch.uint8), codes)
    # in place, re-forwarding the same chunk: the same rows
    codes = cache.k_codes.view(torch.uint8).clone()
    assert cache.rope_kv_append(q, k, v, 3 * F, F) is q
    assert torch.equal(q, q_out) and torch.equal(cache.k_codes.view(torch.uint8), codes)


def test_append_keeps_within_its_shard(cuda_lib):
    """Streams 1..2 of 4 and heads 2..3 of 5: the other rows of q_out are untouched, and the shard's
    are an unsharded cache's."""
    full = shape_of(4, 5, 64, 3, 5, (24, 20, 20), 2)
    part = shape_of(2, 2, 64, 3, 5, (24, 20, 20), 2)
    whole, shard = R.make_cache(full, 3, 8), R.make_cache(part, 3, 8, shard=(1, 2, 4, 5))
    q, k, v = draw(full, 3)
    a, b = torch.full_like(q, 5.0), torch.full_like(q, 5.0)
    whole.rope_kv_append(q, k, v, 0, 2, q_out=a)
    shard.rope_kv_append(q, k, v, 0, 2, q_out=b)
    want = torch.full_like(q, 5.0)
    want[1:3, :, 2:4] = a[1:3, :, 2:4]
    assert torch.equal(b, want)
    for n in ("k_codes", "v_codes", "k_scale", "v_scale"):
        assert torch.equal(getattr(shard, n).view(torch.uint8),
                           getattr(whole, n).view(torch.uint8)[1:3, 2:4])
    oa, ob = torch.full_like(q, 5.0), torch.full_like(q, 5.0)
    whole.window_attn(a, 2, out=oa)
    shard.window_attn(b, 2, out=ob)
    want[1:3, :, 2:4] = oa[1:3, :, 2:4]
    torch.cuda.synchronize()
    assert torch.equal(ob[0], want[0]) and torch.equal(ob[3], want[3])
    assert torch.equal(ob[:, :, :2], want[:, :, :2]) and torch.equal(ob[:, :, 4:], want[:, :, 4:])
    assert (ob.double() - want.double()).abs().max() <= 2.0 ** -6


@pytest.mark.parametrize("D,split", [(64, (24, 20, 20)), (128, (44, 42, 42))])
def test_special_values(cuda_lib, D, split):
    """Zeros, tiny, huge and non-finite channels; v is stored without rotation."""
    shape = shape_of(1, 1, D, 2, 8, split)
    cache = R.make_cache(shape, 1, 2)
    v = torch.zeros((1, 16, 1, D), dtype=torch.bfloat16, device="cuda")
    top = torch.finfo(torch.bfloat16).max
    v[0, 1, 0, :] = 2.0 ** -120
    v[0, 2, 0, ::2] = -2.0 ** -126
    v[0, 3, 0, :32] = top
    v[0, 4, 0, 5], v[0, 4, 0, 6] = 448.0, -464.0
    v[0, 5, 0, 33] = float("nan")
    v[0, 6, 0, 2] = float("inf")
    v[0, 7, 0, 34] = -float("inf")
    v[0, 8, 0, :] = -0.0
    v[0, 9, 0, 0], v[0, 9, 0, 1] = 2.0 ** 100, 2.0 ** 92
    v[0, 10, 0, 0], v[0, 10, 0, 1] = 448.0, 2.0 ** -10        # a tie below the smallest code
    v[0, 11, 0, 0], v[0, 11, 0, 1] = 448.0, 3 * 2.0 ** -10    # a tie between two codes
    z = torch.zeros_like(v)
    cache.rope_kv_append(z.clone(), z, v, 0, 1)
    _, got = cache.read_frames(0, 1)
    got = got[0, 0].double()
    x = v[0, :, 0].double()
    blocks = lambda t: t.unflatten(-1, (-1, 32))  # noqa: E731
    bad = ~torch.isfinite(blocks(x)).all(-1, keepdim=True).expand(-1, -1, 32).flatten(-2)
    assert torch.equal(torch.isnan(got), bad)
    ok = ~bad & (x.abs() < 2.0 ** 127)
    want = R.stored(torch.where(bad, torch.zeros_like(x), x))
    assert torch.equal(got[ok], want[ok])
    assert torch.equal(got[3, :32], torch.full((32,), 240 * 2.0 ** 120, device="cuda").double())
    assert got[9, 1] == 2.0 ** 92 and got[10, 1] == 0 and got[11, 1] == 2.0 ** -8
    assert cache.v_scale.view(torch.uint8)[0, 0, 5].tolist()[1] == 255


@pytest.mark.parametrize("D", [64, 128])
def test_read_gives_every_code_its_value(cuda_lib, D):
    """All 254 codes under scale bytes from the smallest to the largest, exactly."""
    shape = shape_of(1, 1, D, 29, 8, (D, 0, 0))           # 232 tokens: bytes 16 .. 247
    cache = R.make_cache(shape, 2, 4)
    z = torch.zeros((1, 232, 1, D), dtype=torch.bfloat16, device="cuda")
    for f in range(2):
        cache.rope_kv_append(z.clone(), z, z, f, 1)
    rows = 464
    byte = (16 + torch.arange(rows, device="cuda") % 232).to(torch.uint8)
    for base in range(0, 256, D):
        code = (base + torch.arange(D, device="cuda")).to(torch.uint8)
        code[(code & 0x7F) == 0x7F] = 0                   # never written
        for c, s in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
            c.view(torch.uint8)[:] = code
            s.view(torch.uint8)[:] = byte[:, None]
        top = byte == 247                                 # codes up to 240 there
        c64 = R.values(cache.k_codes, cache.k_scale.view(torch.uint8))
        ok = ~(top[:, None] & (cache.k_codes.double().abs() > 240)[0, 0])
        for t in cache.read_frames(0, 2):
            assert torch.equal(t.double()[0, 0][ok], c64[0, 0][ok])


@pytest.mark.parametrize("dims", SHAPES)
def test_read_frames_in_time_order(cuda_lib, dims):
    shape = shape_of(*dims)
    F, cap = shape.chunk_frames, 2 * shape.chunk_frames + 1
    cache = R.make_cache(shape, cap, 9 + 4 * F)
    for c in range(4):
        cache.rope_kv_append(*draw(shape, c), 9 + c * F, F)
    end = 9 + 4 * F
    for first, n in ((end - cap, cap), (end - 1, 1), (end - cap + 1, F), (end - F, F)):
        rows = R.ring_rows(shape, cap, first, n, "cuda")
        k, v = cache.read_frames(first, n)
        for got, c, s in ((k, cache.k_codes, cache.k_scale), (v, cache.v_codes, cache.v_scale)):
            want = R.values(c.view(torch.uint8)[:, :, rows].view(torch.float8_e4m3fn),
                            s.view(torch.uint8)[:, :, rows])
            assert torch.equal(got.double(), want)
    # one of the two alone, through the C ABI; the surroundings stay
    n = shape.B * shape.H * F * shape.Tf * shape.D
    buf = torch.full((n + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    k, v = cache.read_frames(end - F, F)
    s = torch.cuda.current_stream().cuda_stream
    for args, want in (((buf.data_ptr(), None), k), ((None, buf.data_ptr()), v)):
        assert binding.lib().unstep_q8_cache_read(ctypes.byref(cache.q8), end - F, F, *args, s) == 0
        assert torch.equal(buf[:n], want.reshape(-1)) and bool((buf[n:] == 3.0).all())
    for first, m in ((end - cap - 1, 1), (end, 1), (end - 1, 2), (8, 1), (end - cap - 1, cap)):
        with pytest.raises(binding.UnstepError) as e:
            cache.read_frames(first, m)
        assert e.value.status == binding.UNSTEP_ERR_WINDOW


def check_attn(shape, cache, q, window, out=None):
    first, frames = cache.last_chunk
    f0 = max(cache.c.first_frame, first + frames - window)
    rows = R.ring_rows(shape, cache.c.cap_frames, f0, first + frames - f0, "cuda")
    k, v = (R.values(c.view(torch.uint8)[:, :, rows].view(torch.float8_e4m3fn),
                     s.view(torch.uint8)[:, :, rows])
            for c, s in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)))
    out = cache.window_attn(q, window) if out is None else out
    torch.cuda.synchronize()
    assert cache.device_error() == 0
    want, bound = R.attention(q, k, v)
    bad = (out.double() - want).abs() > bound
    assert not bool(bad.any()), (int(bad.sum()), ((out.double() - want).abs() / bound).max())


@pytest.mark.parametrize("use_scratch", [True, False])
@pytest.mark.parametrize("dims", SHAPES)
def test_attention_matches_the_definition(cuda_lib, dims, use_scratch):
    """Every window of a wrapping ring; frames outside the window hold NaN."""
    shape = shape_of(*dims)
    F, cap = shape.chunk_frames, 2 * shape.chunk_frames + 1
    cache = R.make_cache(shape, cap, 4 * F, use_scratch=use_scratch)
    for c in range(4):
        q, k, v = draw(shape, 100 + c)
        cache.rope_kv_append(q, k, v, c * F, F)
        for window in range(F, cap + 1):
            check_attn(shape, cache, q, window)
    keep = [t.view(torch.uint8).clone() for t in (cache.k_scale, cache.v_scale)]
    for window in (F, F + 1):
        inside = R.ring_rows(shape, cap, 4 * F - window, window, "cuda")
        for was, s in zip(keep, (cache.k_scale, cache.v_scale)):
            s.view(torch.uint8)[:] = 255
            s.view(torch.uint8)[:, :, inside] = was[:, :, inside]
        check_attn(shape, cache, q, window)


# keys around the 128-row tile, queries around the 128- and 256-row tiles
@pytest.mark.parametrize("D,split", [(64, (24, 20, 20)), (128, (44, 42, 42))])
@pytest.mark.parametrize("Tf,chunks,window", [(1, 5, 3), (127, 2, 2), (128, 3, 3), (129, 3, 2),
                                              (255, 1, 1), (257, 2, 2), (300, 5, 4)])
def test_attention_tile_borders(cuda_lib, D, split, Tf, chunks, window):
    shape = shape_of(2, 2, D, 1, Tf, split)
    cache = R.make_cache(shape, window, chunks)
    for c in range(chunks):
        q, k, v = draw(shape, 7 * c + Tf)
        cache.rope_kv_append(q, k, v, c, 1)
    check_attn(shape, cache, q, window)
    # rows past the tile that holds the last key: a NaN there must not reach the output
    a = cache.window_attn(q, window)
    assert torch.equal(a, cache.window_attn(q, window))


@pytest.mark.parametrize("D,split", [(64, (24, 20, 20)), (128, (44, 42, 42))])
def test_attention_scale_range(cuda_lib, D, split):
    """Keys and values far above and below 1 (scale bytes above 134 need the second factor), one
    query that prefers a single key, and a chunk of one frame over a long ring."""
    shape = shape_of(1, 2, D, 5, 9, split)
    cache = R.make_cache(shape, 6, 8)
    for c in range(8):
        q, k, v = draw(shape, c, strong=False)
        s = 2.0 ** (12 * (c % 3) - 12)
        v = (v.float() * (1e6 if c % 2 else 1e-6)).to(torch.bfloat16)
        q, k = (q.float() / 4096).to(torch.bfloat16), (k.float() * s).to(torch.bfloat16)
        cache.rope_kv_append(q, k, v, c, 1)
        check_attn(shape, cache, q, min(6, 1 + c))
    assert int(cache.v_scale.view(torch.uint8).max()) > 134
    k[0, 3] *= 8192
    cache.rope_kv_append(q, k, v, 7, 1)
    check_attn(shape, cache, q, 6)


@pytest.mark.parametrize("D,split", [(64, (24, 20, 20)), (128, (44, 42, 42))])
def test_attention_mixed_scales(cuda_lib, D, split):
    """Blocks far apart in scale within a row, a tile and a thread's share of it: each 32 channels
    of each value row have a magnitude of their own, on both sides of the split factor."""
    shape = shape_of(1, 2, D, 10, 13, split)
    cache = R.make_cache(shape, 3, 6)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for c in range(4):
        q, k, v = draw(shape, 30 + c, strong=False)
        power = torch.randint(-30, 31, (1, shape.L, 2, D // 32, 1), generator=g, device="cuda")
        v = torch.ldexp(v.float().unflatten(-1, (-1, 32)), power).flatten(-2).to(torch.bfloat16)
        cache.rope_kv_append(q, k, v, c, 1)
        for window in (1, 2, 3):
            check_attn(shape, cache, q, window)
    b = cache.v_scale.view(torch.uint8)
    assert int(b.max()) > 134 > int(b.min())


def test_attention_of_a_nan_key_is_nan(cuda_lib):
    shape = shape_of(1, 2, 64, 4, 6, (24, 20, 20))
    cache = R.make_cache(shape, 2, 4)
    q, k, v = draw(shape, 1)
    k[0, 5, 0, 3] = float("nan")
    v[0, 7, 1, 40] = float("inf")
    cache.rope_kv_append(q, k, v, 0, 1)
    out = cache.window_attn(q, 1).float()
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[:, :, 0]).all())                       # a NaN key: the whole head
    assert bool(torch.isnan(out[:, :, 1, 32:]).all())                  # a NaN value: its block
    assert bool(torch.isfinite(out[:, :, 1, :32]).all())


@pytest.mark.parametrize("use_scratch", [True, False])
def test_attention_wan_shape(cuda_lib, use_scratch):
    """The 12-head layer with nine frames, split units and merges: sampled heads in full."""
    shape = shape_of(1, 12, 128, 30, 52, (44, 42, 42), 3)
    cache = R.make_cache(shape, 10, 18, use_scratch=use_scratch)
    for c in range(6):
        q, k, v = W.gen_qkv(40 + c, shape, device="cuda")
        cache.rope_kv_append(q, k, v, 3 * c, 3)
    out = cache.window_attn(q, 9)
    assert torch.equal(out, cache.window_attn(q, 9))
    kd, vd = cache.read_frames(9, 9)
    for h in (0, 7, 11):
        want, bound = R.attention(q[:, :, h:h + 1], kd[:, h:h + 1].double(), vd[:, h:h + 1].double())
        assert bool(((out[:, :, h:h + 1].double() - want).abs() <= bound).all())
    assert cache.device_error() == 0


def test_many_streams_and_heads(cuda_lib):
    """More (stream, head) pairs than a grid axis holds in the read-back, single-token frames."""
    shape = shape_of(700, 100, 64, 1, 1, (64, 0, 0))
    cache = R.make_cache(shape, 2, 3, use_scratch=False)
    for c in range(3):
        q, k, v = draw(shape, c)
        cache.rope_kv_append(q, k, v, c, 1)
    k1, v1 = cache.read_frames(1, 2)
    assert torch.equal(v1[:, :, 1].double(), R.stored(v[:, 0].double()))
    want, bound = R.attention(q, k1.double(), v1.double())
    assert bool(((cache.window_attn(q, 2).double() - want).abs() <= bound).all())


def test_save_and_restore(cuda_lib):
    shape = shape_of(2, 3, 64, 4, 6, (24, 20, 20), 2)
    a = R.make_cache(shape, 5, 12)
    for c in range(4):
        a.rope_kv_append(*draw(shape, c), 2 * c, 2)
    buf = a.save_state()
    assert buf.numel() == a.state_bytes()
    b = R.make_cache(shape, 5, 12)
    b.restore_state(buf)
    nxt = draw(shape, 50)
    outs = []
    for c in (a, b):
        q = c.rope_kv_append(nxt[0].clone(), nxt[1], nxt[2], 8, 2)
        outs.append((c.window_attn(q, 5), *c.read_frames(5, 5)))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    # a bf16 cache's buffer and a damaged header are refused, and change nothing
    bf = P.make_cache(shape, 5, 12)
    big = torch.zeros(max(buf.numel(), bf.state_bytes()), dtype=torch.uint8)
    big[: buf.numel()] = buf
    with pytest.raises(binding.UnstepError):
        bf.restore_state(big)
    with pytest.raises(binding.UnstepError):
        b.restore_state(bf.save_state())
    for at, value in ((72, 9), (76, 100), (80, -5), (84, 6), (84, 0)):
        bad = buf.clone()
        bad[at: at + 4] = torch.tensor([value], dtype=torch.int32).view(torch.uint8)
        with pytest.raises(binding.UnstepError):
            b.restore_state(bad)
    assert b.last_chunk == (8, 2) and b.frames_written == 10
    # an empty cache's state
    e = R.make_cache(shape, 5, 12)
    b.restore_state(e.save_state())
    assert b.frames_written == 0 and b.last_chunk == (-1, 0)


def test_bf16_calls_refuse_the_8bit_cache(cuda_lib):
    shape = shape_of(1, 2, 64, 4, 6, (24, 20, 20))
    c = R.make_cache(shape, 2, 4)
    q, k, v = draw(shape, 0)
    c.rope_kv_append(q, k, v, 0, 1)
    L, base = binding.lib(), ctypes.byref(c.c)
    s = torch.cuda.current_stream().cuda_stream
    g = binding.unstep_grid_t(1, 4, 6)
    host = torch.empty(1 << 20, dtype=torch.uint8)
    arg = binding.UNSTEP_ERR_ARG
    assert L.unstep_window_attn(q.data_ptr(), base, 1, v.data_ptr(), s) == arg
    assert L.unstep_window_attn_noalloc(q.data_ptr(), base, 1, v.data_ptr(), s) == arg
    assert L.unstep_rope_kv_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), base, 1, g, s) == arg
    assert L.unstep_cache_init(base, s) == arg
    assert L.unstep_cache_save(base, host.data_ptr(), host.numel(), s) == arg
    assert L.unstep_append_plan(base, 1, g, None) == 1
    c.reset()
    assert c.frames_written == 0 and int(c.k_codes.view(torch.uint8).max()) == 0
    with pytest.raises(ValueError):
        c.rope_kv_append(q, k, v, 0, 1, defer_q=True)
    c.rope_kv_append(q, k, v, 0, 1)
    with pytest.raises(ValueError):
        c.window_attn(q, 1, rope_q=True)
    with pytest.raises(ValueError):
        c.rope_kv_append(q.float(), k, v, 1, 1)
    for args in ((q.cpu(), k, v, 1, 1), (q, k[:, :1], v, 1, 1), (q, k, v, 1, 2), (q, k, v, 1, -1),
                 (q, k, v, 2 ** 40, 1), (q, k, v, 1.5, 1), (q, k, None, 1, 1),
                 (q.transpose(1, 2).contiguous().transpose(1, 2), k, v, 1, 1)):
        with pytest.raises(ValueError):
            c.rope_kv_append(*args)
    both = torch.empty(2 * q.numel(), dtype=q.dtype, device="cuda")
    a, b = both[: q.numel()].view_as(q), both[64: 64 + q.numel()].view_as(q)
    with pytest.raises(binding.UnstepError):
        c.rope_kv_append(q, a, v, 1, 1, q_out=b)
    with pytest.raises(ValueError):
        c.window_attn(q, 1, out=q[:, :, :1])
    assert c.frames_written == 1 and c.last_chunk == (0, 1)
    with pytest.raises(ValueError):
        c.read_frames(0, 1, k_out=torch.empty(1, device="cuda", dtype=torch.bfloat16))


def test_side_stream_and_graph(cuda_lib):
    """A step on a side stream, and captured once and replayed on other inputs, gives the eager
    results; two layers share one scratch in the graph."""
    shape = shape_of(1, 3, 128, 10, 30, (44, 42, 42), 3)
    caches = [R.make_cache(shape, 6, 6)]
    caches.append(R.make_cache(shape, 6, 6, scratch=caches[0].scratch))
    first = [draw(shape, 60 + i) for i in range(2)]
    second = [draw(shape, 70 + i) for i in range(2)]

    def step(bufs, stream=None):
        outs = []
        for c, (q, k, v, qo) in zip(caches, bufs):
            c.rope_kv_append(q, k, v, 3, 3, q_out=qo, stream=stream)
            outs.append((c.window_attn(qo, 6, stream=stream), *c.read_frames(1, 5, stream=stream)))
        return outs

    for c, x in zip(caches, first):
        c.rope_kv_append(*(t.clone() for t in x), 0, 3)
    bufs = [(*(t.clone() for t in x), torch.empty_like(x[0])) for x in second]
    want = step(bufs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(bufs, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step(bufs)
    other = [draw(shape, 80 + i) for i in range(2)]
    for rep, inputs in enumerate((other, second, other)):
        for b, x in zip(bufs, inputs):
            for t, y in zip(b, x):
                t.copy_(y)
        g.replay()
        got = [[t.clone() for t in h] for h in held]
        want = step(bufs)
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), rep
    assert all(c.device_error() == 0 for c in caches)
