"""Measured cases of the operators on unquantized and 4-bit integer experts.

Four operators, each with its directions:
  * grouped matrix products over expert-sorted rows of ragged counts: the
    product (``linear``), the gated pair with SwiGLU (``swiglu``), the input
    gradient (``dgrad``), the same through SwiGLU (``swiglu_dgrad``), the
    weight gradient (``wgrad``);
  * products with 4-bit integer weights and group scales, dense or by expert
    (``int4``);
  * the routing-weighted combine of the experts' rows (``combine``) and its
    gradients (``combine_backward``), the router's logits among them.

``run`` computes them in elementary torch operations in fp32, or, where
``own`` is true, through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
LARGEST_FLOPS = 5.2e11          # of the largest listed case; no drawn case costs more
LARGEST_VALUES = 6.0e8          # of the largest listed weight stack or set of rows


def listed():
    return [
        # the smallest layer this repository runs: 16 tokens, launch latency counts
        dict(name="linear tiny", op="linear", T=16, k=2, E=8, K=256, N=128, skew=0.0, gather=True),
        # decode of 8 sequences through one rank's 64 experts, gate and up with SwiGLU: weight streaming
        dict(name="swiglu decode 8", op="swiglu", T=8, k=8, E=64, K=5120, N=1536, skew=0.0, gather=True),
        # down product of a prefill chunk of 1024 tokens over 32 local experts
        dict(name="linear prefill 1024", op="linear", T=1024, k=8, E=32, K=1536, N=5120, skew=0.0, gather=False),
        # gate and up of a 2048-token chunk with a skewed router: some experts long, some nearly empty
        dict(name="swiglu prefill 2048 skewed", op="swiglu", T=2048, k=8, E=32, K=5120, N=1536, skew=1.1, gather=True),
        # training step, backward: through the down product and SwiGLU, an odd token count
        dict(name="swiglu dgrad 1021", op="swiglu_dgrad", T=1021, k=8, E=32, K=1536, N=5120, skew=0.0),
        # training step, backward: the gate and up products' input gradient, summed
        dict(name="dgrad pair 1021", op="dgrad", T=1021, k=8, E=32, K=5120, N=1536, skew=1.1, pair=True),
        # training step: weight gradient of the gate projection, token rows gathered
        dict(name="wgrad 1024 gathered", op="wgrad", T=1024, k=8, E=32, K=5120, N=1536, skew=0.0, gather=True),
        # training step: weight gradient of the router, one group with a long reduction
        dict(name="wgrad router 8195", op="wgrad", T=8195, k=1, E=1, K=5120, N=256, skew=0.0, gather=False),
        # one decode token through a dense 4-bit projection, groups of 128
        dict(name="int4 dense 1", op="int4", T=1, k=1, E=1, K=5120, N=5120, G=128, zeros=True, skew=0.0),
        # decode of 8 sequences through 64 4-bit experts, groups of 32
        dict(name="int4 experts 8", op="int4", T=8, k=8, E=64, K=5120, N=1536, G=32, zeros=False, skew=0.0),
        # the experts' rows back to 4099 tokens
        dict(name="combine 4099", op="combine", T=4099, k=8, E=256, H=5120, skew=0.0),
        # training step: gradients of the combine, routing weights and router logits
        dict(name="combine backward 2048", op="combine_backward", T=2048, k=8, E=256, H=5120, skew=1.1),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) // step * step))) // step * step


def draw(rng):
    op = rng.choice(["linear", "swiglu", "dgrad", "swiglu_dgrad", "wgrad", "int4", "int4", "combine", "combine_backward"])
    E = _log(rng, 1, 64)
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 8192)
    skew = rng.choice([0.0, 0.0, 0.7, 1.1])
    if op in ("combine", "combine_backward"):
        H = _log(rng, 64, 8192, 8)
        return dict(op=op, T=max(1, min(T, int(LARGEST_VALUES / 3 / (k * H)))), k=k, E=max(E, k), H=H, skew=skew)
    if op == "int4":
        T = _log(rng, 1, 256)
        c = dict(op=op, E=E, k=k, K=_log(rng, 128, 8192, 128), N=_log(rng, 16, 5200), G=rng.choice([32, 64, 128]),
                 zeros=rng.random() < 0.5, skew=skew)
    else:
        c = dict(op=op, E=E, k=k, K=_log(rng, 64, 5120, 8), N=_log(rng, 64, 5120, 8), skew=skew)
    if op in ("linear", "swiglu", "wgrad"):
        c["gather"] = rng.random() < 0.5
    if op == "dgrad":
        c["pair"] = rng.random() < 0.5
    c["E"] = max(k, min(E, int(LARGEST_VALUES / 2.4 / (c["K"] * c["N"]))))
    c["k"] = k = min(k, c["E"])
    T = min(T, int(LARGEST_FLOPS / (4.0 * k * c["K"] * c["N"])), int(LARGEST_VALUES / (c["E"] * max(c["K"], c["N"]))))
    c["T"] = max(1, T)
    return c


def _routing(c, gen):
    """Top-k of skewed random logits, and the expert-sorted order of the (token, slot) pairs."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn((T, E), generator=gen, device=DEV)
    rank = torch.randperm(E, generator=gen, device=DEV) + 1
    top = torch.topk(logits - c["skew"] * torch.log(rank.float()), k, dim=1)
    ids = top.indices.to(torch.int32)
    order = torch.sort(ids.reshape(-1), stable=True).indices.to(torch.int32)
    pos = torch.empty_like(order)
    pos[order.long()] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return dict(ids=ids, w=torch.softmax(top.values, dim=1), offsets=offsets, sorted_slots=order, slot_pos=pos,
                cap=int(counts.max()))


def _randn(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=BF16) * scale).to(BF16)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = _routing(c, gen)
    s["op"], s["k"], s["E"] = c["op"], c["k"], c["E"]
    op, T, k, E, M = c["op"], c["T"], c["k"], c["E"], c["T"] * c["k"]
    if op in ("combine", "combine_backward"):
        s["y"] = _randn(gen, M, c["H"])
        if op == "combine_backward":
            s["dout"] = _randn(gen, T, c["H"])
        return s
    K, N = c["K"], c["N"]
    if op == "int4":
        s["x"], s["G"] = _randn(gen, T, K), c["G"]
        s["codes"] = torch.randint(0, 256, (E, N, K // 2), generator=gen, device=DEV, dtype=torch.uint8)
        s["scales"] = ((0.5 + torch.rand((E, N, K // c["G"]), generator=gen, device=DEV)) * 0.004).to(BF16)
        s["zeros"] = torch.randint(0, 16, (E, N, K // c["G"]), generator=gen, device=DEV, dtype=torch.uint8) if c["zeros"] else None
        return s
    rows = T if c.get("gather") else M
    s["slots"] = s["sorted_slots"] if c.get("gather") else None
    if op in ("linear", "swiglu", "wgrad"):
        s["x"] = _randn(gen, rows, K)
    if op != "wgrad":
        s["w"] = _randn(gen, E, N, K, scale=K ** -0.5)
    if op == "swiglu" or (op == "dgrad" and c["pair"]):
        s["w2"] = _randn(gen, E, N, K, scale=K ** -0.5)
    if op in ("dgrad", "swiglu_dgrad", "wgrad"):
        s["dy"] = _randn(gen, M, N)
    if op == "dgrad" and c["pair"]:
        s["dy2"] = _randn(gen, M, N)
    if op == "swiglu_dgrad":
        s["a"], s["b"] = _randn(gen, M, K), _randn(gen, M, K)
    return s


# ------------------------------------------------------------------ plain forms
def _place(s):
    """Expert and place inside the expert of every sorted row."""
    M = s["ids"].numel()
    r = torch.arange(M, device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
    return e, r - s["offsets"].long()[e]


def _padded(s, rows, e, p):
    out = torch.zeros((s["E"], s["cap"], rows.shape[1]), dtype=torch.float32, device=DEV)
    out[e, p] = rows.float()
    return out


def _rows(s, x):
    return x if s["slots"] is None else x[(s["slots"] // s["k"]).long()]


def _silu_parts(a):
    sig = 1.0 / (1.0 + torch.exp(-a))
    return sig, a * sig


def _plain(s):
    op, k = s["op"], s["k"]
    if op == "combine":
        return (s["w"][:, :, None] * s["y"][s["slot_pos"].long()].float().view(*s["w"].shape, -1)).sum(1).to(BF16)
    if op == "combine_backward":
        yr = s["y"][s["slot_pos"].long()].float().view(*s["w"].shape, -1)
        dout, w = s["dout"].float(), s["w"]
        dy = torch.empty_like(s["y"])
        dy[s["slot_pos"].long()] = (w[:, :, None] * dout[:, None, :]).to(BF16).view(-1, yr.shape[-1])
        dw = (dout[:, None, :] * yr).sum(-1)
        dl = torch.zeros((w.shape[0], s["E"]), device=DEV)
        dl.scatter_add_(1, s["ids"].long(), w * (dw - (w * dw).sum(-1, keepdim=True)))
        return dy, dw, dl
    e, p = _place(s)
    if op == "int4":
        codes = s["codes"]
        q = torch.stack((codes & 15, codes >> 4), dim=-1).view(*codes.shape[:2], -1, s["G"]).float()
        z = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
        w = ((q - z) * s["scales"].float()[..., None]).view(*codes.shape[:2], -1)
        xp = _padded(s, s["x"][(s["sorted_slots"] // k).long()], e, p)
        return torch.bmm(xp, w.transpose(1, 2))[e, p].to(BF16)
    if op == "linear":
        return torch.bmm(_padded(s, _rows(s, s["x"]), e, p), s["w"].float().transpose(1, 2))[e, p].to(BF16)
    if op == "swiglu":
        xp = _padded(s, _rows(s, s["x"]), e, p)
        a = torch.bmm(xp, s["w"].float().transpose(1, 2))[e, p]
        b = torch.bmm(xp, s["w2"].float().transpose(1, 2))[e, p]
        return (_silu_parts(a)[1] * b).to(BF16), a.to(BF16), b.to(BF16)
    dyp = _padded(s, s["dy"], e, p)
    if op == "dgrad":
        dx = torch.bmm(dyp, s["w"].float())[e, p]
        if "w2" in s:
            dx = dx + torch.bmm(_padded(s, s["dy2"], e, p), s["w2"].float())[e, p]
        return dx.to(BF16)
    if op == "swiglu_dgrad":
        dh = torch.bmm(dyp, s["w"].float())[e, p]
        a, b = s["a"].float(), s["b"].float()
        sig, act = _silu_parts(a)
        return (dh * b * (sig + act * (1.0 - sig))).to(BF16), (dh * act).to(BF16)
    return torch.bmm(dyp.transpose(1, 2), _padded(s, _rows(s, s["x"]), e, p))


def _own(s):
    from nvfp4_weight_only_moe_amd import binding as B
    op, k = s["op"], s["k"]
    if op == "linear":
        return B.moe_grouped_linear(s["x"], s["w"], s["offsets"], s["slots"], k)
    if op == "swiglu":
        return B.moe_grouped_swiglu(s["x"], s["w"], s["w2"], s["offsets"], s["slots"], k, save=True)
    if op == "dgrad":
        return B.moe_grouped_linear_dgrad(s["dy"], s["w"], s["offsets"], s.get("dy2"), s.get("w2"))
    if op == "swiglu_dgrad":
        return B.moe_grouped_swiglu_dgrad(s["dy"], s["w"], s["a"], s["b"], s["offsets"])
    if op == "wgrad":
        return B.moe_grouped_linear_wgrad(s["dy"], s["x"], s["offsets"], s["slots"], k)
    if op == "int4":
        w = B.Int4Tensor(s["codes"], s["scales"], s["zeros"])
        if s["E"] == 1 and k == 1:
            return B.moe_int4_linear(s["x"], w)
        return B.moe_int4_linear(s["x"], w, s["offsets"], s["sorted_slots"], k)
    if op == "combine":
        return B.moe_combine(s["y"], s["slot_pos"], k, s["w"])
    return B.moe_combine_backward(s["dout"], s["y"], s["slot_pos"], s["w"], s["ids"], s["E"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = dict(case)
    T, k, E = c["T"], c["k"], c["E"]
    M = T * k
    if c["op"] == "combine":
        return dict(bytes=2.0 * M * c["H"] + 2.0 * T * c["H"] + 8.0 * M, flops=2.0 * M * c["H"])
    if c["op"] == "combine_backward":
        return dict(bytes=2.0 * T * c["H"] + 4.0 * M * c["H"] + 16.0 * M + 4.0 * T * E, flops=3.0 * M * c["H"])
    K, N = c["K"], c["N"]
    touched = E * (1.0 - (1.0 - k / E) ** T)            # expected, for a router without skew
    rows = T if c.get("gather") else M
    if c["op"] == "int4":
        per = 0.5 + (3.0 if c["zeros"] else 2.0) / c["G"]
        return dict(bytes=touched * N * K * per + 2.0 * T * K + 2.0 * M * N + 8.0 * M, flops=2.0 * M * N * K)
    if c["op"] == "linear":
        return dict(bytes=2.0 * (touched * N * K + rows * K + M * N), flops=2.0 * M * N * K)
    if c["op"] == "swiglu":
        return dict(bytes=2.0 * (2 * touched * N * K + rows * K + 3 * M * N), flops=4.0 * M * N * K)
    if c["op"] == "dgrad":
        n = 2 if c["pair"] else 1
        return dict(bytes=2.0 * (n * touched * N * K + n * M * N + M * K), flops=2.0 * n * M * N * K)
    if c["op"] == "swiglu_dgrad":
        return dict(bytes=2.0 * (touched * N * K + M * N + 4 * M * K), flops=2.0 * M * N * K)
    return dict(bytes=4.0 * E * N * K + 2.0 * (M * N + rows * K), flops=2.0 * M * N * K)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    """One expert (or one slot of all tokens) at a time, in fp64, from the definitions."""
    s = prepare(case, seed)
    op, k, E = s["op"], s["k"], s["E"]
    T = s["ids"].shape[0]
    d = torch.float64
    if op == "combine":
        out = torch.zeros((T, s["y"].shape[1]), dtype=d, device=DEV)
        for j in range(k):
            out += s["w"][:, j, None].to(d) * s["y"].to(d)[s["slot_pos"].view(T, k)[:, j].long()]
        return out
    if op == "combine_backward":
        dy = torch.zeros(s["y"].shape, dtype=d, device=DEV)
        dw = torch.zeros((T, k), dtype=d, device=DEV)
        dl = torch.zeros((T, E), dtype=d, device=DEV)
        w = s["w"].to(d)
        for j in range(k):
            at = s["slot_pos"].view(T, k)[:, j].long()
            dy[at] = w[:, j, None] * s["dout"].to(d)
            dw[:, j] = (s["dout"].to(d) * s["y"].to(d)[at]).sum(1)
        for i in range(k):                                # d w_j / d logit_i = w_j (delta_ij - w_i)
            for j in range(k):
                g = dw[:, j] * w[:, j] * ((1.0 if i == j else 0.0) - w[:, i])
                dl[torch.arange(T, device=DEV), s["ids"][:, i].long()] += g
        return dy, dw, dl
    off = s["offsets"].tolist()
    rows = (s["sorted_slots"] // k).long()
    K = case["K"]
    M, N = T * k, case["N"]

    def stack(width, n=1):
        return [torch.zeros((M, width), dtype=d, device=DEV) for _ in range(n)]

    def source(lo, hi):
        x = s["x"].to(d)
        return x[rows[lo:hi]] if op == "int4" or s["slots"] is not None else x[lo:hi]

    if op == "wgrad":
        dw = torch.zeros((E, N, K), dtype=d, device=DEV)
        for e in range(E):
            dw[e] = s["dy"][off[e]:off[e + 1]].to(d).t() @ source(off[e], off[e + 1])
        return dw
    outs = {"linear": lambda: stack(N), "int4": lambda: stack(N), "swiglu": lambda: stack(N, 3), "dgrad": lambda: stack(K),
            "swiglu_dgrad": lambda: stack(K, 2)}[op]()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        if op == "int4":
            w = torch.empty((N, K), dtype=d, device=DEV)
            w[:, 0::2] = (s["codes"][e] % 16).to(d)
            w[:, 1::2] = torch.div(s["codes"][e], 16, rounding_mode="floor").to(d)
            z = torch.full_like(s["scales"][e], 8).to(d) if s["zeros"] is None else s["zeros"][e].to(d)
            w = (w - z.repeat_interleave(s["G"], 1)) * s["scales"][e].to(d).repeat_interleave(s["G"], 1)
            outs[0][lo:hi] = source(lo, hi) @ w.t()
            continue
        w = s["w"][e].to(d)
        if op == "linear":
            outs[0][lo:hi] = source(lo, hi) @ w.t()
        elif op == "swiglu":
            a, b = source(lo, hi) @ w.t(), source(lo, hi) @ s["w2"][e].to(d).t()
            outs[0][lo:hi], outs[1][lo:hi], outs[2][lo:hi] = a / (1 + torch.exp(-a)) * b, a, b
        else:
            dx = s["dy"][lo:hi].to(d) @ w
            if op == "dgrad":
                outs[0][lo:hi] = dx + (s["dy2"][lo:hi].to(d) @ s["w2"][e].to(d) if "w2" in s else 0.0)
            else:
                a, b = s["a"][lo:hi].to(d), s["b"][lo:hi].to(d)
                sig = torch.sigmoid(a)
                outs[0][lo:hi], outs[1][lo:hi] = dx * b * sig * (1 + a * (1 - sig)), dx * a * sig
    return outs[0] if len(outs) == 1 else tuple(outs)
