"""Norm + modulation and gated residual + norm on the GPU against their formulas in 64 bits."""
import pytest
import torch

from causal_video_diffusion_b200 import binding
from causal_video_diffusion_b200.binding import Norm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# evaluation in fp32: a row's sums take at most 64 terms a thread and a tree of 14 levels, and an
# element passes fewer than 32 further operations: under 128 roundings of 2^-24
EV = 2.0 ** -17


def norm64(n, x, G):
    """(value, fp32 evaluation bound) of a Norm of x [rows][C] (fp64)."""
    per = x.shape[0] // G
    mean = x.mean(1, keepdim=True) if n.kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + n.eps)
    v = (x - mean) * rstd
    e = EV * ((x.abs() + x.abs().mean(1, keepdim=True)) * rstd)
    if n.weight is not None:
        v, e = v * n.weight.double(), e * n.weight.double().abs()
    if n.bias is not None:
        v, e = v + n.bias.double(), e + EV * n.bias.double().abs()
    if n.scale is not None:
        s = 1 + n.scale.double().repeat_interleave(per, 0)
        v, e = v * s, e * s.abs() + EV * v.abs()
    if n.shift is not None:
        t = n.shift.double().repeat_interleave(per, 0)
        v, e = v + t, e + EV * t.abs()
    return v, e + EV * v.abs()


def moved(n, x, dx, G):
    """How far a Norm of x can move when every element moves by up to dx (first order, doubled)."""
    per = x.shape[0] // G
    mean = x.mean(1, keepdim=True) if n.kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + n.eps)
    d = rstd * (dx + dx.mean(1, keepdim=True)) + \
        ((x - mean) * rstd).abs() * rstd * dx.square().mean(1, keepdim=True).sqrt()
    if n.weight is not None:
        d = d * n.weight.double().abs()
    if n.scale is not None:
        d = d * (1 + n.scale.double().repeat_interleave(per, 0)).abs()
    return 2 * d


def near(got, want, ev):
    half = {BF: 2.0 ** -8, F32: 2.0 ** -24}[got.dtype]
    err = (got.double() - want).abs()
    bound = ev + half * (want.abs() + ev) + 1e-37
    assert bool((err <= bound).all()), (err / bound).max()


def rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def make_norm(g, kind, C, G, p, affine, modulate, eps=1e-6):
    table = (0.3 * rand(g, G, 6, C)).to(p)
    return Norm(kind, eps, weight=(1 + 0.2 * rand(g, C)).to(p) if affine else None,
                bias=(0.2 * rand(g, C)).to(p) if affine and kind == "layer" else None,
                scale=table[:, 1] if modulate else None, shift=table[:, 0] if modulate else None), \
        table[:, 2]


# rows (a multiple of groups), C, groups; C at and around each variant's limits
SIZES = [(1, 8, 1), (3, 64, 3), (5, 72, 1), (6, 128, 2), (17, 136, 1), (30, 256, 3), (4, 264, 2),
         (9, 504, 3), (10, 512, 5), (7, 520, 1), (333, 1024, 3), (5, 1032, 5), (149, 1536, 1),
         (4, 2040, 2), (6, 2048, 3), (3, 2056, 1), (3, 4096, 3), (2, 4104, 1), (4, 8192, 2),
         (2, 8200, 1), (3, 16384, 1), (1200, 1536, 3)]


@pytest.mark.parametrize("x_type", [BF, F32])
@pytest.mark.parametrize("rows,C,G", SIZES)
def test_norm_modulate(cuda_lib, rows, C, G, x_type):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * C)
    x = (rand(g, rows, C) * 3 + rand(g, C)).to(x_type)
    for i, (kind, p, affine, mod) in enumerate([("layer", F32, False, True), ("rms", BF, True, False),
                                                ("layer", BF, True, True), ("rms", F32, True, True),
                                                ("layer", F32, False, False)]):
        n, _ = make_norm(g, kind, C, G, p, affine, mod)
        groups = G if mod else 1
        want, ev = norm64(n, x.double(), groups)
        near(binding.norm_modulate(x, n), want, ev)


@pytest.mark.parametrize("x_type", [BF, F32])
@pytest.mark.parametrize("rows,C,G", SIZES)
def test_gate_residual_norm(cuda_lib, rows, C, G, x_type):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * C + 1)
    x = (rand(g, rows, C) * 3 + rand(g, C)).to(x_type)
    y = (rand(g, rows, C) * 2).to(BF)
    per = rows // G
    for post, kind, p, affine, mod, gated, s in [
            (None, "layer", F32, False, True, True, 1.0), ("rms", "rms", BF, True, False, True, 0.5),
            ("layer", "layer", BF, True, True, False, 0.125), (None, None, F32, False, False, True, 1.0),
            ("rms", None, F32, True, False, False, -2.0)]:
        post_n = make_norm(g, post, C, G, p, True, False)[0] if post else None
        next_n, gate = make_norm(g, kind or "rms", C, G, p, affine, mod)
        yv, ye = y.double(), torch.zeros_like(y, dtype=torch.float64)
        if post:
            yv, ye = norm64(post_n, yv, 1)
        gv = gate.double().repeat_interleave(per, 0) if gated else 1.0
        v = x.double() + s * gv * yv
        ev = (s * gv * torch.ones_like(v)).abs() * (ye + EV * yv.abs()) + 2.0 ** -23 * v.abs()
        x0 = x.clone()
        x_out, h = binding.gate_residual_norm(x, y, gate=gate if gated else None, res_scale=s,
                                              post=post_n, next=next_n if kind else None,
                                              x_out=torch.empty_like(x))
        assert torch.equal(x, x0)
        near(x_out, v, ev)
        if kind:
            want, eh = norm64(next_n, v, G)
            near(h, want, eh + moved(next_n, v, ev, G))
        else:
            assert h is None
        # in place: the same bits
        again, h2 = binding.gate_residual_norm(x0, y, gate=gate if gated else None, res_scale=s,
                                               post=post_n, next=next_n if kind else None)
        assert again is x0 and torch.equal(x0, x_out) and (h is None or torch.equal(h, h2))


def test_strided_rows_and_surroundings(cuda_lib):
    """Queries and keys inside a fused projection's output, read and written in place as column
    blocks; everything around them stays."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    C = 384
    qkv = rand(g, 2, 50, 3 * C).to(BF)
    keep = qkv.clone()
    n, _ = make_norm(g, "rms", C, 1, BF, True, False)
    q, k = qkv[..., :C], qkv[..., C:2 * C]
    want, ev = norm64(n, keep[..., :C].reshape(-1, C).double(), 1)
    out = torch.full((2, 50, C + 64), 3.0, dtype=BF, device="cuda")
    binding.norm_modulate(q, n, out=out[..., 32:32 + C])
    near(out[..., 32:32 + C].reshape(-1, C), want, ev)
    assert bool((out[..., :32] == 3).all()) and bool((out[..., 32 + C:] == 3).all())
    assert torch.equal(qkv, keep)
    assert binding.norm_modulate(q, n, out=q) is q
    assert torch.equal(q, out[..., 32:32 + C])
    assert torch.equal(qkv[..., C:], keep[..., C:])
    binding.norm_modulate(k, n, out=k)
    assert torch.equal(qkv[..., 2 * C:], keep[..., 2 * C:]) and torch.equal(q, out[..., 32:32 + C])
    x = torch.full((100, C + 8), 9.0, dtype=F32, device="cuda")
    x[:, :C] = rand(g, 100, C)
    x0 = x.clone()
    y = qkv.view(100, 3 * C)[:, C:2 * C]
    h = torch.full((100, C + 16), 5.0, dtype=BF, device="cuda")
    binding.gate_residual_norm(x[:, :C], y, next=n, out=h[:, :C])
    near(x[:, :C], x0[:, :C].double() + y.double(), 2.0 ** -23 * x[:, :C].double().abs())
    assert bool((x[:, C:] == 9).all()) and bool((h[:, C:] == 5).all())


@pytest.mark.parametrize("C", [72, 1536, 2056])
def test_fp32_off_32_bytes(cuda_lib, C):
    """fp32 rows and parameters on 16-byte but not 32-byte addresses: the same bits as on 32."""
    g = torch.Generator(device="cuda")
    g.manual_seed(C)

    def off(t, by=4):
        flat = torch.full((t.numel() + 16,), 7.0, dtype=t.dtype, device="cuda")
        view = flat[by: by + t.numel()].view(t.shape)
        view.copy_(t)
        return view, flat

    x, y, w = rand(g, 6, C), rand(g, 6, C).to(BF), rand(g, C)
    tab = rand(g, 3, C)
    n = Norm("layer", 1e-6, w, w, tab, tab)
    m = Norm("layer", 1e-6, off(w)[0], off(w, 12)[0], off(tab)[0], off(tab, 12)[0])
    want = binding.norm_modulate(x, n)
    assert torch.equal(binding.norm_modulate(off(x)[0], m), want)
    assert torch.equal(binding.norm_modulate(x, m), want)
    assert torch.equal(binding.norm_modulate(off(x, 12)[0], n), want)
    want = binding.gate_residual_norm(x, y, gate=tab, post=n, next=n, x_out=torch.empty_like(x))
    xo, flat = off(torch.zeros_like(x), 12)
    got = binding.gate_residual_norm(off(x)[0], y, gate=off(tab)[0], post=m, next=m, x_out=xo)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((flat[:12] == 7).all()) and bool((flat[12 + xo.numel():] == 7).all())


def test_difficult_rows(cuda_lib):
    """Constant rows, zeros, one large channel, a large common offset, NaN and infinity in one row
    of several that share a CTA; eps 0 on a row with variance."""
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    for C in (64, 1536, 4096):
        x = rand(g, 12, C)
        x[0] = 2.0
        x[1] = 0.0
        x[2, 5] = 1e18
        x[3] += 4096.0
        x[4] *= 1e-12
        x[6, 1] = float("nan")
        x[7, 2] = float("inf")
        fine = [i for i in range(12) if i not in (6, 7)]
        for kind in ("layer", "rms"):
            n = Norm(kind, 1e-6)
            h = binding.norm_modulate(x, n)
            want, ev = norm64(n, x[fine].double(), 1)
            near(h[fine], want, ev)
            assert bool(torch.isnan(h[6]).all()) and bool(torch.isnan(h[7, 2]).all())
        n = Norm("layer", 0.0)
        want, ev = norm64(n, x[8:].double(), 1)
        near(binding.norm_modulate(x[8:], n), want, ev)


def test_rows_of_none_and_of_many_groups(cuda_lib):
    z = torch.empty((0, 64), dtype=BF, device="cuda")
    assert binding.norm_modulate(z, Norm()).shape == (0, 64)
    x_out, h = binding.gate_residual_norm(z, z, next=Norm())
    assert x_out is z and h.shape == (0, 64)
    m = torch.zeros((3, 64), device="cuda")
    assert binding.norm_modulate(z, Norm(scale=m, shift=m)).shape == (0, 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    # a modulation for every row, and one shared by expanding it
    x = rand(g, 70000, 16).to(BF)
    m = rand(g, 70000, 16)
    n = Norm("rms", 1e-6, shift=m)
    want, ev = norm64(n, x.double(), 70000)
    near(binding.norm_modulate(x, n), want, ev)
    one = m[:1].expand(7, 16)
    n = Norm("rms", 1e-6, scale=one, shift=one)
    want, ev = norm64(n, x.double(), 7)
    near(binding.norm_modulate(x, n), want, ev)


def test_offsets_past_32_bits(cuda_lib):
    """Rows whose byte and element offsets pass 2^32 and 2^31 (rows far apart in one buffer)."""
    C, rows, ld = 64, 5, 600_000_000
    buf = torch.empty(((rows - 1) * ld + C,), dtype=BF, device="cuda")
    x = buf.as_strided((rows, C), (ld, 1))
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x.copy_(rand(g, rows, C))
    n = Norm("layer", 1e-6)
    want, ev = norm64(n, x.double(), 1)
    near(binding.norm_modulate(x, n), want, ev)
    x0 = x.double()
    binding.gate_residual_norm(x, want.to(BF))
    near(x.contiguous(), x0 + want.to(BF).double(), 2.0 ** -23 * x0.abs())


def test_side_stream_and_graph(cuda_lib):
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    C, G = 1536, 3
    x, y = rand(g, 300, C), rand(g, 300, C).to(BF)
    n, gate = make_norm(g, "layer", C, G, F32, True, True)
    x_out, h = torch.empty_like(x), torch.empty_like(y)

    def step(stream=None, **kw):
        return binding.gate_residual_norm(x, y, gate=gate, next=n, stream=stream, **kw)

    want = step(x_out=torch.empty_like(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s, x_out=torch.empty_like(x))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x_out=x_out, out=h)
        hm = binding.norm_modulate(x, n)
    for _ in range(3):
        x.copy_(rand(g, 300, C))
        graph.replay()
        want = step(x_out=torch.empty_like(x))
        assert torch.equal(want[0], x_out) and torch.equal(want[1], h)
        assert torch.equal(hm, binding.norm_modulate(x, n))


def test_binding_refusals(cuda_lib):
    x = torch.zeros((6, 64), dtype=BF, device="cuda")
    v, w2 = torch.zeros(64, device="cuda"), torch.zeros((2, 64), device="cuda")
    bad = [
        lambda: binding.norm_modulate(x.half(), Norm()),
        lambda: binding.norm_modulate(x.cpu(), Norm()),
        lambda: binding.norm_modulate(x[0], Norm()),
        lambda: binding.norm_modulate(x[:, ::2], Norm()),
        lambda: binding.norm_modulate(x[:1].expand(6, 64), Norm()),
        lambda: binding.norm_modulate(torch.zeros((4, 6, 64), dtype=BF, device="cuda")[:, ::2][:, :2], Norm()),
        lambda: binding.norm_modulate(x, Norm("batch")),
        lambda: binding.norm_modulate(x, Norm(weight=v, shift=w2.to(BF))),
        lambda: binding.norm_modulate(x, Norm(weight=v.half())),
        lambda: binding.norm_modulate(x, Norm(weight=v[:32])),
        lambda: binding.norm_modulate(x, Norm(weight=v.cpu())),
        lambda: binding.norm_modulate(x, Norm(scale=v)),
        lambda: binding.norm_modulate(x, Norm(scale=torch.zeros((4, 64), device="cuda"))),
        lambda: binding.norm_modulate(x, Norm(scale=w2, shift=torch.zeros((3, 64), device="cuda"))),
        lambda: binding.norm_modulate(x, Norm(scale=w2, shift=torch.zeros((2, 72), device="cuda")[:, :64])),
        lambda: binding.norm_modulate(x, Norm(), out=torch.zeros((6, 64), device="cuda")),
        lambda: binding.norm_modulate(x, Norm(), out=torch.zeros((5, 64), dtype=BF, device="cuda")),
        lambda: binding.gate_residual_norm(x, x.float()),
        lambda: binding.gate_residual_norm(x, x[:5].clone()),
        lambda: binding.gate_residual_norm(x, x.clone(), gate=v),
        lambda: binding.gate_residual_norm(x, x.clone(), gate=w2, next=Norm(scale=torch.zeros((3, 64), device="cuda"))),
        lambda: binding.gate_residual_norm(x, x.clone(), out=x.clone()),
        lambda: binding.gate_residual_norm(x, x.clone(), x_out=x.float()),
        lambda: binding.gate_residual_norm(x, x.clone(), x_out=x.cpu()),
        lambda: binding.gate_residual_norm(x, x.clone(), res_scale="1"),
        lambda: binding.norm_modulate(x, ("layer", 1e-6)),
        lambda: binding.norm_modulate(x, Norm(3)),
        lambda: binding.norm_modulate(x, Norm(weight=1.0)),
        lambda: binding.norm_modulate(x, Norm(eps=None)),
        lambda: binding.norm_modulate([1.0], Norm()),
        lambda: binding.norm_modulate(torch.zeros((), dtype=BF, device="cuda"), Norm()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(str(i))
    odd = torch.zeros((6, 60), dtype=BF, device="cuda")
    shifted = torch.zeros(6 * 64 + 4, dtype=BF, device="cuda")[4:].view(6, 64)
    for f, want in ((lambda: binding.norm_modulate(odd, Norm()), binding.UNSTEP_ERR_SHAPE),
                    (lambda: binding.norm_modulate(shifted, Norm()), binding.UNSTEP_ERR_ALIGN),
                    (lambda: binding.norm_modulate(x, Norm(eps=-1.0)), binding.UNSTEP_ERR_ARG),
                    (lambda: binding.gate_residual_norm(x, x), binding.UNSTEP_ERR_ARG),
                    (lambda: binding.gate_residual_norm(x, x.clone(), next=Norm(), out=x),
                     binding.UNSTEP_ERR_ARG)):
        with pytest.raises(binding.UnstepError) as e:
            f()
        assert e.value.status == want
