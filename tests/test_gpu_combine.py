"""The combine and its gradients against plain fp64 forms."""
import pytest
import torch

from experts_util import BF16_HALF, F64, U32, assert_within, rounded
from gpu_util import DEV
from nvfp4_weight_only_moe_amd import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
CASES = [(1, 1, 8), (1, 8, 5120), (3, 2, 2056), (17, 32, 264), (130, 8, 1024), (1000, 3, 72)]


def problem(T, k, H, drop):
    g = torch.Generator(device=DEV).manual_seed(T * 100 + k + H)
    M = T * k + 3
    pos = torch.randperm(M, generator=g, device=DEV)[: T * k].to(torch.int32)
    if drop:
        gone = torch.rand(T * k, generator=g, device=DEV) < 0.4
        gone[:k] = True                                    # a token with no slot left
        pos[gone] = torch.where(torch.rand(int(gone.sum()), generator=g, device=DEV) < 0.5, -1, M).to(torch.int32)
    y = torch.randn((M, H), generator=g, device=DEV).to(BF)
    w = torch.rand((T, k), generator=g, device=DEV)
    w = w / w.sum(1, keepdim=True)
    dout = torch.randn((T, H), generator=g, device=DEV).to(BF)
    ids = torch.randint(0, 40, (T, k), generator=g, device=DEV, dtype=torch.int32)   # the same expert twice, too
    live = (pos >= 0) & (pos < M)
    named = torch.zeros(M, dtype=torch.bool, device=DEV)
    named[pos[live].long()] = True
    y[~named] = float("nan")                               # rows that no slot names
    return M, pos, y, w, dout, ids, live, named


def rows_of(y, pos, live):
    return torch.where(live[:, None], y.to(F64)[torch.where(live, pos, 0).long()], 0.0)


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("T,k,H", CASES)
def test_combine(T, k, H, weights, drop):
    M, pos, y, w, _, _, live, _ = problem(T, k, H, drop)
    got = B.moe_combine(y, pos, k, w if weights else None)
    terms = rows_of(y, pos, live).view(T, k, H) * (w.to(F64)[..., None] if weights else 1.0)
    ref = terms.sum(1)
    assert_within(got, ref, rounded(ref, 2 * k * U32 * terms.abs().sum(1)), "combine")
    if drop:
        assert (got[0] == 0).all()


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("T,k,H", CASES)
def test_combine_backward(T, k, H, drop):
    M, pos, y, w, dout, ids, live, named = problem(T, k, H, drop)
    dy = torch.full((M, H), 9.0, dtype=BF, device=DEV)
    dy, dw, dl = B.moe_combine_backward(dout, y, pos, w, ids, 40, dy=dy)
    yr = rows_of(y, pos, live).view(T, k, H)
    d = dout.to(F64)[:, None, :]
    want = torch.full((M, H), 9.0, dtype=F64, device=DEV)
    want[pos[live].long()] = (w.to(F64)[..., None] * d).view(T * k, H)[live]
    assert_within(dy, want, rounded(want, U32 * want.abs()), "dy")
    assert (dy[~named] == 9.0).all()
    dot, mag = (d * yr).sum(-1), (d * yr).abs().sum(-1)
    e = H * U32 * mag
    assert_within(dw, dot, e, "dw")
    assert (dw.view(-1)[~live] == 0).all()
    w64 = w.to(F64)
    g = w64 * (dot - (w64 * dot).sum(-1, keepdim=True))
    eg = w64 * (e + (w64 * e).sum(-1, keepdim=True)) + (k + 4) * U32 * w64 * (dot.abs() + (w64 * dot).abs().sum(-1, keepdim=True))
    ref, err = (torch.zeros((T, 40), dtype=F64, device=DEV) for _ in range(2))
    ref.scatter_add_(1, ids.long(), g)
    err.scatter_add_(1, ids.long(), eg + k * U32 * g.abs())
    assert_within(dl, ref, err, "dlogits")


def test_logits_gradient_against_differences():
    """dlogits of the whole chain softmax over the selected -> combine, against central differences in fp64."""
    T, E, k, H = 3, 9, 4, 64
    g = torch.Generator(device=DEV).manual_seed(11)
    logits = torch.randn((T, E), generator=g, device=DEV)
    r = B.moe_route_topk(logits, k)
    y = torch.randn((T * k, H), generator=g, device=DEV).to(BF)
    dout = torch.randn((T, H), generator=g, device=DEV).to(BF)
    _, _, dl = B.moe_combine_backward(dout, y, r.slot_pos, r.topk_w, r.topk_ids, E)
    yr = y.to(F64)[r.slot_pos.view(T, k).long()]

    def loss(z):
        p = torch.softmax(z.gather(1, r.topk_ids.long()), 1)
        return ((p[..., None] * yr).sum(1) * dout.to(F64)).sum().item()

    z, h = logits.to(F64), 1e-5
    for t in range(T):
        for e in range(E):
            up, dn = z.clone(), z.clone()
            up[t, e] += h
            dn[t, e] -= h
            diff = (loss(up) - loss(dn)) / (2 * h)
            # weights in fp32 (2^-23 k of sums below 64 * 4 sigma^2), differences h^2
            assert abs(dl[t, e].item() - diff) < 1e-3, (t, e)


def test_zero_tokens_and_no_rows():
    y = torch.empty((0, 64), dtype=BF, device=DEV)
    none = torch.empty((0,), dtype=torch.int32, device=DEV)
    assert B.moe_combine(y, none, 4).shape == (0, 64)
    gone = torch.full((6,), -1, dtype=torch.int32, device=DEV)
    assert (B.moe_combine(torch.empty((1, 64), dtype=BF, device=DEV), gone, 3) == 0).all()
    assert (B.moe_combine(y, gone, 3) == 0).all()          # no rows at all
    w = torch.full((2, 3), 1 / 3, device=DEV)
    dy, dw = B.moe_combine_backward(torch.ones((2, 64), dtype=BF, device=DEV), y, gone, w)
    assert dy.shape == (0, 64) and (dw == 0).all()
    dy, dw = B.moe_combine_backward(torch.ones((2, 64), dtype=BF, device=DEV), torch.ones((1, 64), dtype=BF, device=DEV), gone, w)
    assert dy.shape == (1, 64) and (dw == 0).all()
