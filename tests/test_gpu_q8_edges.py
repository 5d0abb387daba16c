"""The 8-bit cache's calls at their edges: what the documentation allows and the main tests leave out."""
import pytest
import torch

from causal_video_diffusion_b200 import binding
from tests import q8_reference as R
from tests.test_gpu_q8 import draw, shape_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,split,H", [(64, (24, 20, 20), 3), (128, (44, 42, 42), 8), (128, (44, 42, 42), 1)])
@pytest.mark.parametrize("onto", ["k", "v"])
def test_rotated_queries_onto_k_or_v(cuda_lib, D, split, H, onto):
    """q_out may be k or v: each is read before its place is written, also right behind the norm that
    wrote it."""
    shape = shape_of(2, H, D, 7, 9, split, 2)
    cache, twin = R.make_cache(shape, 4, 8), R.make_cache(shape, 4, 8)
    n = binding.Norm("rms", 1e-6)
    rows = lambda t: t.view(shape.B, shape.L, H * D)  # noqa: E731
    for c in range(4):
        q, k, v = draw(shape, 40 + c)
        apart = [binding.norm_modulate(rows(t), n).view_as(t) for t in (k, v)]
        torch.cuda.synchronize()
        want = twin.rope_kv_append(q, *apart, 2 * c, 2, q_out=torch.empty_like(q))
        want_out = twin.window_attn(want, min(4, 2 * c + 2))
        torch.cuda.synchronize()
        over = k if onto == "k" else v
        for t in (k, v):
            binding.norm_modulate(rows(t), n, out=rows(t))
        assert cache.rope_kv_append(q, k, v, 2 * c, 2, q_out=over) is over
        out = cache.window_attn(over, min(4, 2 * c + 2))
        assert torch.equal(over, want) and torch.equal(out, want_out)
        for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
            assert torch.equal(getattr(cache, name).view(torch.uint8), getattr(twin, name).view(torch.uint8))


def test_attention_onto_its_queries_is_refused(cuda_lib):
    shape = shape_of(1, 2, 64, 4, 6, (24, 20, 20), 1)
    cache = R.make_cache(shape, 2, 4)
    q, k, v = draw(shape, 3)
    cache.rope_kv_append(q, k, v, 0, 1)
    for f in (lambda: cache.window_attn(q, 1, out=q),
              lambda: cache.read_frames(0, 1, k_out=(t := torch.empty((1, 2, 24, 64), dtype=q.dtype,
                                                                      device="cuda")), v_out=t)):
        with pytest.raises(binding.UnstepError) as e:
            f()
        assert e.value.status == binding.UNSTEP_ERR_ARG


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens,use_scratch", [(40, True), (200, True), (1500, True), (1500, False)])
def test_scores_beyond_fp32(cuda_lib, D, tokens, use_scratch):
    """Keys whose scores overflow, in one tile or in all of them.  To minus infinity: the key has no
    weight, and a row with no other key has no softmax (NaN).  To plus infinity: infinity over
    infinity (NaN).  Frame 0 on a temporal axis alone is not rotated, and both values are powers of
    two, so the stored keys are exact."""
    shape = shape_of(1, 4, D, 1, tokens, (D, 0, 0))
    cache = R.make_cache(shape, 1, 1, use_scratch=use_scratch)
    q, k, v = draw(shape, tokens, strong=False)
    q[..., 0] = 2.0 ** 100
    k[..., 0] = 0.0
    far = torch.zeros_like(k)
    far[..., 0] = -(2.0 ** 100)                 # a score of -2^200
    n = torch.arange(tokens, device="cuda")
    # head 0: every third key; head 1: all but the last; head 2: every key; head 3: one above
    gone = torch.stack([n % 3 == 1, n < tokens - 1, n >= 0, n < 0])
    for h in range(3):
        k[0, gone[h], h] = far[0, gone[h], h]
    k[0, tokens // 2, 3] = -far[0, tokens // 2, 3]
    cache.rope_kv_append(q, k, v, 0, 1)
    out = cache.window_attn(q, 1)
    torch.cuda.synchronize()
    assert cache.device_error() == 0
    kd, vd = (t.double() for t in cache.read_frames(0, 1))
    for h in (0, 1):
        keep = ~gone[h]
        want, bound = R.attention(q[:, :, h:h + 1], kd[:, h:h + 1, keep], vd[:, h:h + 1, keep])
        assert bool(((out[:, :, h:h + 1].double() - want).abs() <= bound).all()), h
    assert bool(torch.isnan(out[:, :, 2:]).all())


@pytest.mark.parametrize("D,split", [(64, (24, 20, 20)), (128, (44, 42, 42))])
@pytest.mark.parametrize("Tf", [1, 127, 128, 129, 255, 257])
def test_rows_behind_the_last_key(cuda_lib, D, split, Tf):
    """NaN in every ring row outside the window, on both sides of it, and NaN left in shared memory by
    the call before: the output keeps its bits.  The window ends inside a key tile."""
    shape = shape_of(1, 2, D, 1, Tf, split)
    cache = R.make_cache(shape, 5, 9)
    for c in range(9):
        q, k, v = draw(shape, 7 * c + Tf)
        cache.rope_kv_append(q, k, v, c, 1)
    parts = [cache.k_codes.view(torch.uint8), cache.v_codes.view(torch.uint8),
             cache.k_scale.view(torch.uint8), cache.v_scale.view(torch.uint8)]
    kept = [t.clone() for t in parts]
    for window in (1, 2, 3):                    # slots 3; 2, 3; 1, 2, 3 of five
        for t, was in zip(parts, kept):
            t.copy_(was)
        want = cache.window_attn(q, window)
        inside = R.ring_rows(shape, 5, 9 - window, window, "cuda")
        for t, was, fill in zip(parts, kept, (0x7F, 0xFF, 255, 255)):
            t[:] = fill
            t[:, :, inside] = was[:, :, inside]
        assert bool(torch.isnan(cache.window_attn(q, 5)).all())
        assert torch.equal(cache.window_attn(q, window), want), window
    assert cache.device_error() == 0


def test_host_steps(cuda_lib):
    """Steps fed from host memory give the device steps' bits; the query rotation inside the attention,
    which an 8-bit cache does not have, is refused before anything is copied."""
    shape = shape_of(1, 2, 64, 4, 6, (24, 20, 20), 2)
    cache, twin = R.make_cache(shape, 4, 8), R.make_cache(shape, 4, 8)
    bufs = {n: torch.full((1, 48, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
            for n in ("q", "k", "v", "out")}
    host = lambda t: t.cpu().pin_memory()  # noqa: E731
    q, k, v = draw(shape, 5)
    out = torch.zeros((1, 48, 2, 64), dtype=torch.bfloat16).pin_memory()
    with pytest.raises(ValueError):
        binding.HostStepPipeline(cache, rope_q_in_attn=True)
    for args in ((host(q), host(k), host(v), 0, 2, 2, out, bufs),
                 (host(q), host(k), host(v), 0, 2, 2, out, bufs, None)):
        with pytest.raises(ValueError):
            cache.step_from_host(*args, rope_q_in_attn=True)
    with pytest.raises(ValueError):
        cache.step_from_host(*args, True)
    torch.cuda.synchronize()
    assert all(bool((t == 7.0).all()) for t in bufs.values()) and cache.frames_written == 0
    qo = twin.rope_kv_append(q, k, v, 0, 2, q_out=torch.empty_like(q))
    want = twin.window_attn(qo, 2).cpu()
    cache.step_from_host(host(q), host(k), host(v), 0, 2, 2, out, bufs)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    binding.HostStepPipeline(cache).run(host(q), host(k), host(v), 0, 2, 2, out, 3)
    assert torch.equal(out, want) and cache.device_error() == 0
