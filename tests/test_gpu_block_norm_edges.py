"""The norm calls at their edges: what the documentation allows and the main tests leave out."""
import pytest
import torch

from causal_video_diffusion_b200 import binding
from causal_video_diffusion_b200.binding import Norm
from tests.test_gpu_block_norm import EV, make_norm, near, norm64, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def test_views_of_one_buffer(cuda_lib):
    """Outputs between, beside and in place of the rows they are made from; a shifted view is refused
    and nothing is written."""
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    C, rows = 72, 40
    buf = rand(g, rows, 4 * C).to(BF)
    n, gate = make_norm(g, "layer", C, 4, F32, True, True)
    keep = buf.clone()
    x, y = buf[:, :C], buf[:, C:2 * C]
    want, ev = norm64(n, x.double(), 4)
    binding.norm_modulate(x, n, out=buf[:, 2 * C:3 * C])
    near(buf[:, 2 * C:3 * C], want, ev)
    # x_out and h beside x and y, all four blocks of the same rows; y is also x's neighbour
    v = x.double() + gate.double().repeat_interleave(10, 0) * y.double()
    ev = EV * (v - x.double()).abs() + 2.0 ** -23 * v.abs()
    binding.gate_residual_norm(x, y, gate=gate, next=Norm("rms"), x_out=buf[:, 2 * C:3 * C],
                               out=buf[:, 3 * C:])
    near(buf[:, 2 * C:3 * C], v, ev)
    assert torch.equal(buf[:, :2 * C], keep[:, :2 * C])
    # rows of another stride in the gaps
    flat = buf.view(-1)
    a, b = flat.as_strided((10, C), (2 * C, 1)), flat.as_strided((10, C), (4 * C, 1), C)
    want, ev = norm64(Norm("rms"), a.double(), 1)
    near(binding.norm_modulate(a, Norm("rms"), out=b), want, ev)
    # x as both inputs
    z, _ = binding.gate_residual_norm(x, x, x_out=torch.empty_like(x))
    near(z, 2 * x.double(), 2.0 ** -23 * x.double().abs())
    keep = buf.clone()
    s = torch.empty((rows + 1, C), dtype=BF, device="cuda").copy_(rand(g, rows + 1, C))
    held = s.clone()
    bad = [lambda: binding.norm_modulate(s[1:], Norm(), out=s[:-1]),
           lambda: binding.norm_modulate(s[:-1], Norm(), out=s[1:]),
           lambda: binding.norm_modulate(buf[:, :C], n, out=buf[:, 8:C + 8]),
           lambda: binding.gate_residual_norm(s[1:], y, x_out=s[:-1]),
           lambda: binding.gate_residual_norm(s[1:], y, next=n, out=s[:-1]),
           lambda: binding.gate_residual_norm(x, s[1:], next=n, out=s[:-1], x_out=torch.empty_like(x)),
           lambda: binding.norm_modulate(y, Norm(weight=s[3], shift=s[:1]), out=s[:-1])]
    for f in bad:
        with pytest.raises(binding.UnstepError) as e:
            f()
        assert e.value.status == binding.UNSTEP_ERR_ARG
    torch.cuda.synchronize()
    assert torch.equal(s, held) and torch.equal(buf, keep)


def test_channels_past_32_bits_are_refused(cuda_lib):
    """2^32 + 64 channels are not 64."""
    x = torch.zeros((1, 2 ** 32 + 64), dtype=BF, device="cuda")
    for f in (lambda: binding.norm_modulate(x, Norm(), out=x),
              lambda: binding.gate_residual_norm(x, x.clone(), next=Norm(), out=torch.empty_like(x))):
        with pytest.raises(binding.UnstepError) as e:
            f()
        assert e.value.status == binding.UNSTEP_ERR_UNSUPPORTED
