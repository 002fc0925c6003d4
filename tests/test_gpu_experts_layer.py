"""The operators on unquantized experts together, as a training step and a
decode step use them: route, gate/up with SwiGLU, down, combine, and the whole
backward pass down to the router logits, against autograd of the same layer in
fp64; the same in a captured graph, replayed; and the packed layers beside it."""
import pytest
import torch

from experts_util import F64
from gpu_util import DEV, log
from nvfp4_weight_only_moe_amd import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Layer:
    def __init__(self, T, H, I, E, k, seed, skew=0.0):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def rnd(*s, scale=1.0):
            return (torch.randn(s, generator=g, device=DEV) * scale).to(BF)
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.x, self.dout = rnd(T, H), rnd(T, H)
        self.gate, self.up, self.down = rnd(E, I, H, scale=H ** -0.5), rnd(E, I, H, scale=H ** -0.5), rnd(E, H, I, scale=I ** -0.5)
        self.logits = torch.randn((T, E), generator=g, device=DEV) - skew * torch.log(torch.arange(1, E + 1, device=DEV).float())

    def step(self):
        """Forward and backward: out and every gradient."""
        r = B.moe_route_topk(self.logits, self.k)
        h, a, b = B.moe_grouped_swiglu(self.x, self.gate, self.up, r.offsets, r.sorted_slots, self.k, save=True)
        y = B.moe_grouped_linear(h, self.down, r.offsets)
        out = B.moe_combine(y, r.slot_pos, self.k, r.topk_w)
        dy, _, dlogits = B.moe_combine_backward(self.dout, y, r.slot_pos, r.topk_w, r.topk_ids, self.E)
        ddown = B.moe_grouped_linear_wgrad(dy, h, r.offsets)
        da, db = B.moe_grouped_swiglu_dgrad(dy, self.down, a, b, r.offsets)
        dgate = B.moe_grouped_linear_wgrad(da, self.x, r.offsets, r.sorted_slots, self.k)
        dup = B.moe_grouped_linear_wgrad(db, self.x, r.offsets, r.sorted_slots, self.k)
        dx = B.moe_combine(B.moe_grouped_linear_dgrad(da, self.gate, r.offsets, db, self.up), r.slot_pos, self.k)
        return dict(out=out, dx=dx, dgate=dgate, dup=dup, ddown=ddown, dlogits=dlogits)

    def reference(self):
        leaf = {n: getattr(self, n).to(F64).requires_grad_() for n in ("x", "gate", "up", "down", "logits")}
        top = torch.topk(leaf["logits"], self.k, dim=1)
        w = torch.softmax(top.values, 1)
        out = torch.zeros((self.T, self.H), dtype=F64, device=DEV)
        for e in range(self.E):
            t, j = (top.indices == e).nonzero(as_tuple=True)
            if len(t):
                a, b = leaf["x"][t] @ leaf["gate"][e].t(), leaf["x"][t] @ leaf["up"][e].t()
                y = (a * torch.sigmoid(a) * b) @ leaf["down"][e].t()
                out = out.index_add(0, t, w[t, j, None] * y)
        out.backward(self.dout.to(F64))
        return dict(out=out.detach(), dx=leaf["x"].grad, dgate=leaf["gate"].grad, dup=leaf["up"].grad,
                    ddown=leaf["down"].grad, dlogits=leaf["logits"].grad)


def close(got, ref, name):
    """Each value passes at most six independent roundings to bf16 on its way
    (x' weights: a, b, h, y, dy, da/db, dx), each at most 2^-8 relative and
    uniform in the half step, so 2^-8 / sqrt(3) of the norm: the norm of their
    sum stays below sqrt(6) / sqrt(3) 2^-8 = 5.6e-3 times the sensitivity of
    SwiGLU's factors (1.1)."""
    ref = ref.to(F64)
    rel = ((got.to(F64) - ref).norm() / ref.norm().clamp_min(1e-300)).item()
    log(f"{name}: rel {rel:.2e}")
    assert torch.isfinite(got).all() and rel <= 6.2e-3, (name, rel)


@pytest.mark.parametrize("T,H,I,E,k,skew", [(1, 64, 32, 4, 2, 0.0), (5, 72, 40, 3, 3, 0.0), (130, 256, 136, 8, 2, 1.5),
                                            (700, 128, 64, 4, 1, 3.0), (257, 512, 256, 70, 8, 0.0)])
def test_forward_and_backward(T, H, I, E, k, skew):
    m = Layer(T, H, I, E, k, seed=T + H, skew=skew)
    got, ref = m.step(), m.reference()
    for n in ref:
        if n == "dlogits" and k == 1:                      # the softmax of one is constant
            assert (got[n] == 0).all()
            continue
        close(got[n], ref[n], n)


def test_gradient_against_differences():
    """<gradient, direction> against a central difference of the fp64 loss along it."""
    m = Layer(40, 64, 48, 5, 2, seed=9)
    got = m.step()
    g = torch.Generator(device=DEV).manual_seed(10)

    def loss(delta):
        n = Layer.__new__(Layer)
        n.__dict__.update(m.__dict__)
        for name, d in delta.items():
            setattr(n, name, getattr(m, name).to(F64) + d)
        return (n.reference()["out"] * m.dout.to(F64)).sum().item()

    for name in ("x", "gate", "up", "down"):
        d = torch.randn(getattr(m, name).shape, generator=g, device=DEV, dtype=F64) * 1e-4
        diff = (loss({name: d}) - loss({name: -d})) / 2
        grad = got["d" + name].to(F64)
        # relative 6.2e-3 of the gradient's norm (close()), seen along a random
        # direction of norm |d|: at most four standard deviations of it
        slack = 4 * 6.2e-3 * grad.norm().item() * d.norm().item() / d.numel() ** 0.5
        assert abs((grad * d).sum().item() - diff) <= slack, name


def test_captured_step_replays():
    m = Layer(260, 256, 128, 16, 4, seed=12, skew=0.8)
    want = {n: t.clone() for n, t in m.step().items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        m.step()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = m.step()
    for _ in range(4):
        for t in got.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), n
        eager = m.step()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(eager[n], want[n]), n
    m.x.copy_(m.x * 0.5)                                   # new inputs in the same buffers
    m.logits.copy_(m.logits.roll(1, 0))
    fresh = m.step()
    graph.replay()
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], fresh[n]), n


def test_two_streams_at_once():
    a, b = Layer(300, 256, 136, 8, 2, seed=21), Layer(33, 520, 64, 4, 4, seed=22)
    want = [{n: t.clone() for n, t in m.step().items()} for m in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for m, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(m.step())
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for n in w:
                assert torch.equal(w[n], g[n]), n


@pytest.mark.parametrize("T", [1, 8, 200])
def test_beside_the_packed_layers(T):
    """The unquantized layer on the weights that the packed ones stand for:
    moe_w4a16_forward on NVFP4 stacks against the grouped products on their
    dequantized values, and moe_int4_linear against grouped products on int4's."""
    H, I, E, k = 1024, 512, 16, 4
    m = Layer(T, H, I, E, k, seed=31)
    r = B.moe_route_topk(m.logits, k)
    packed = [B.moe_w4a16_quantize_pack(w.float()) for w in (m.gate, m.up, m.down)]
    layer = B.moe_w4a16_forward(m.x, *packed, r).view(BF)
    w = [B.moe_w4a16_dequantize(p) for p in packed]        # fp32; its rounding to bf16 is one more 2^-8 per weight
    h = B.moe_grouped_swiglu(m.x, w[0].to(BF), w[1].to(BF), r.offsets, r.sorted_slots, k)
    out = B.moe_combine(B.moe_grouped_linear(h, w[2].to(BF), r.offsets), r.slot_pos, k, r.topk_w)
    close(out, layer, "NVFP4 layer")
    q = [B.moe_int4_quantize_pack(v.float(), 64) for v in (m.gate, m.up, m.down)]
    a, b = (B.moe_int4_linear(m.x, v, r.offsets, r.sorted_slots, k) for v in q[:2])
    d = [B.moe_int4_dequantize(v) for v in q]
    h4 = (torch.nn.functional.silu(a.float()) * b.float()).to(BF)
    out4 = B.moe_combine(B.moe_int4_linear(h4, q[2], r.offsets), r.slot_pos, k, r.topk_w)
    h = B.moe_grouped_swiglu(m.x, d[0].to(BF), d[1].to(BF), r.offsets, r.sorted_slots, k)
    ref4 = B.moe_combine(B.moe_grouped_linear(h, d[2].to(BF), r.offsets), r.slot_pos, k, r.topk_w)
    close(out4, ref4, "int4 layer")
