"""The norms and the 8-bit cache's calls as a DiT block makes them: each after the other on one stream,
every call's result against its definition in 64 bits, with and without waits between the calls, and
in a graph."""
import pytest
import torch

from causal_video_diffusion_b200 import binding, clip
from causal_video_diffusion_b200 import workloads as W
from causal_video_diffusion_b200.binding import Norm
from tests import q8_reference as R
from tests.test_gpu_block_norm import EV, moved, near, norm64
from tests.test_gpu_q8 import check_attn, check_rows, shape_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Block:
    """norm + modulation, fused q k v projection, RMS norms of q and k inside it, append, attention
    over the window, projection, gated residual and the next norm."""

    def __init__(self, shape, cap, frames_max, x_type=F32, seed=0):
        self.shape, self.C = shape, shape.H * shape.D
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        C, F = self.C, shape.chunk_frames
        self.w_qkv = (r(C, 3 * C) / C ** 0.5).to(BF)
        self.w_out = (r(C, C) / C ** 0.5).to(BF)
        self.table = 0.3 * r(F * shape.B, 6, C)
        self.q_norm = Norm("rms", 1e-6, weight=(1 + 0.2 * r(C)).to(BF))
        self.pre = Norm("layer", 1e-6, scale=self.table[:, 1], shift=self.table[:, 0])
        self.next = Norm("layer", 1e-6, scale=self.table[:, 4], shift=self.table[:, 3])
        self.cache = R.make_cache(shape, cap, frames_max)
        self.x_type, self.rand = x_type, r

    def forward(self, x, first, window, wait=lambda: None, seen=None):
        s, C = self.shape, self.C
        h = binding.norm_modulate(x, self.pre)
        wait()
        qkv = h @ self.w_qkv
        q, k, v = qkv[..., :C], qkv[..., C:2 * C], qkv[..., 2 * C:]
        raw = qkv.clone() if seen is not None else None
        binding.norm_modulate(q, self.q_norm, out=q)
        wait()
        binding.norm_modulate(k, self.q_norm, out=k)
        wait()
        heads = [t.contiguous().view(s.B, s.L, s.H, s.D) for t in (q, k, v)]
        rotated = self.cache.rope_kv_append(heads[0], heads[1], heads[2], first, s.chunk_frames,
                                            q_out=torch.empty_like(heads[0]))
        wait()
        out = self.cache.window_attn(rotated, window)
        wait()
        y = out.view(s.B, s.L, C) @ self.w_out
        x_new, h_next = binding.gate_residual_norm(x, y, gate=self.table[:, 2], next=self.next,
                                                   x_out=torch.empty_like(x))
        wait()
        if seen is not None:
            seen.update(h=h, raw=raw, qkv=qkv, heads=heads, rotated=rotated, out=out, y=y)
        return x_new, h_next


@pytest.mark.parametrize("x_type", [BF, F32])
@pytest.mark.parametrize("dims", [(1, 4, 64, 6, 7, (24, 20, 20), 2), (2, 3, 128, 3, 5, (44, 42, 42), 3),
                                  (1, 2, 64, 1, 1, (64, 0, 0), 1), (1, 12, 128, 10, 13, (44, 42, 42), 3)])
def test_block_against_64_bits(cuda_lib, dims, x_type):
    shape = shape_of(*dims)
    F, C = shape.chunk_frames, shape.H * shape.D
    b = Block(shape, 2 * F + 1, 4 * F, x_type)
    x = b.rand(shape.B, shape.L, C).to(x_type)
    G = F * shape.B
    for c in range(4):
        seen = {}
        x_new, h_next = b.forward(x, c * F, min(2 * F + 1, F + c * F), seen=seen)
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        want, ev = norm64(b.pre, flat(x).double(), G)
        near(flat(seen["h"]), want, ev)
        for i in (0, 1):
            col = slice(i * C, (i + 1) * C)
            want, ev = norm64(b.q_norm, flat(seen["raw"])[:, col].double(), 1)
            near(flat(seen["qkv"])[:, col], want, ev)
        assert torch.equal(seen["raw"][..., 2 * C:], seen["qkv"][..., 2 * C:])
        check_rows(shape, b.cache, seen["heads"][1], seen["heads"][2], c * F, F)
        check_attn(shape, b.cache, seen["rotated"], min(2 * F + 1, F + c * F), out=seen["out"])
        gate = b.table[:, 2].double().repeat_interleave(shape.B * shape.L // G, 0)
        v = flat(x).double() + gate * flat(seen["y"]).double()
        ev = EV * (gate * flat(seen["y"]).double()).abs() + 2.0 ** -23 * v.abs()
        near(flat(x_new), v, ev)
        want, eh = norm64(b.next, v, G)
        near(flat(h_next), want, eh + moved(b.next, v, ev, G))
        x = x_new
    assert b.cache.device_error() == 0


def test_calls_in_a_row_need_no_waits(cuda_lib):
    """Small chunks, where a kernel is set up while its predecessor runs: eight layers in a row, many
    times, give the bits of the same calls with a wait after each."""
    shape = shape_of(1, 2, 64, 4, 6, (24, 20, 20), 1)
    results = []
    for wait in (torch.cuda.synchronize, lambda: None):
        layers = [Block(shape, 6, 40, seed=i) for i in range(8)]
        x = layers[0].rand(1, shape.L, layers[0].C)
        got = []
        for c in range(30):
            for b in layers:
                x, h = b.forward(x, c, min(6, c + 1), wait=wait)
            got += [x, h, *layers[-1].cache.read_frames(max(0, c - 5), min(6, c + 1))]
        torch.cuda.synchronize()
        assert all(b.cache.device_error() == 0 for b in layers)
        results.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_norms_around_the_projections(cuda_lib):
    """Norms before and after the library's own products, which also start while their predecessor
    ends: many in a row give the bits of the same calls with a wait after each."""
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    w1, w2 = r(192, 256) / 16, r(256, 192) / 14
    x0, n = r(300, 256), Norm("layer", 1e-6, weight=1 + r(256) / 8)
    results = []
    for wait in (torch.cuda.synchronize, lambda: None):
        x, got = x0.clone(), []
        for _ in range(40):
            h = binding.norm_modulate(x, n)
            wait()
            y = binding.lowrank_linear(h, w1, w2)
            wait()
            x, h = binding.gate_residual_norm(x, y, res_scale=0.5, next=n, x_out=torch.empty_like(x))
            wait()
            got += [x, h]
        torch.cuda.synchronize()
        results.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_inputs_from_another_stream(cuda_lib):
    """Rows made on a side stream while the main stream's norms run, joined by an event, eagerly and
    as a fork and join in a graph: no norm sees them before they are there."""
    g = torch.Generator(device="cuda")
    g.manual_seed(13)
    rows, C = 3000, 512
    src = torch.randn((rows, C), generator=g, device="cuda")
    busy, x = torch.zeros((rows, C), device="cuda"), torch.zeros((rows, C), device="cuda")
    n, side = Norm("layer", 1e-6), torch.cuda.Stream()
    scratch = torch.empty_like(busy, dtype=BF)

    def run(out):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            t = src
            for _ in range(20):
                t = t * 1.5 - src
            x.copy_(t)
        for _ in range(3):
            binding.norm_modulate(busy, n, out=scratch)
        main.wait_stream(side)
        binding.norm_modulate(x, n, out=out)
        # and back: the side stream overwrites the rows once the norm has read them
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x.zero_()
        main.wait_stream(side)

    t = src
    for _ in range(20):
        t = t * 1.5 - src
    want, out = binding.norm_modulate(t, n), torch.empty_like(scratch)
    for _ in range(20):
        out.zero_()
        run(out)
        assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    for _ in range(20):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_block_in_a_graph(cuda_lib):
    """Three layers captured once and replayed on new inputs, against eager calls on a second set."""
    shape = shape_of(1, 3, 64, 5, 9, (24, 20, 20), 2)
    layers, twins = ([Block(shape, 6, 8, seed=i) for i in range(3)] for _ in range(2))
    x0 = layers[0].rand(1, shape.L, layers[0].C)
    for b in layers + twins:
        b.forward(x0, 0, 2)
    x = x0.clone()
    g = torch.cuda.CUDAGraph()

    def run(blocks, x):
        for b in blocks:
            x, h = b.forward(x, 2, 4)
        return x, h

    run(layers, x)          # allocations and the frames' first append, outside the capture
    run(twins, x)
    with torch.cuda.graph(g):
        held = run(layers, x)
    for seed in range(3):
        x.copy_(layers[0].rand(1, shape.L, layers[0].C))
        g.replay()
        want = run(twins, x)
        assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1])


def test_clip_with_8bit_caches(cuda_lib):
    """The clip driver's layers on 8-bit caches: the last forward's attention against the definition,
    and the graph against the eager clip."""
    wl = W.WORKLOADS["clip30"]
    with pytest.raises(ValueError):
        clip.ClipDriver(wl, layers=1, cache="fp4")
    drv = clip.ClipDriver(wl, layers=2, seed=4, cache="q8")
    pristine = [[q.clone() for (q, _, _) in row] for row in drv.inputs]
    drv.run()
    torch.cuda.synchronize()
    eager = [o.clone() for o in drv.outs]
    for layer, cache in enumerate(drv.caches):
        assert cache.device_error() == 0 and isinstance(cache, binding.LayerCacheQ8)
        q = drv.inputs[-1][layer][0]
        first, frames = cache.last_chunk
        k, v = cache.read_frames(first + frames - wl.window, wl.window)
        for h in (0, 7):
            want, bound = R.attention(q[:, :, h:h + 1], k[:, h:h + 1].double(), v[:, h:h + 1].double())
            assert bool(((eager[layer][:, :, h:h + 1].double() - want).abs() <= bound).all())
    for row, qs in zip(drv.inputs, pristine):
        for (q, _, _), was in zip(row, qs):
            q.copy_(was)
    drv.reset()
    drv.capture()
    drv.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, drv.outs))
