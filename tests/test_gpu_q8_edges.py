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
