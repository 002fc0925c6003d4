"""Grouped products of bf16 experts and their gradients against plain fp64
forms, inside the summation and rounding bounds (experts_util)."""
import pytest
import torch

from experts_util import (BF16_HALF, F64, U32, assert_within, experts_rows, offsets_of, product, rounded, source_rows,
                          swiglu, swiglu_error)
from gpu_util import DEV, log
from nvfp4_weight_only_moe_amd import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# rows per expert, K, N: empty experts, one row, tile edges of 64, 128 and 256
# rows, odd counts, K and N off every tile size, more experts than lanes
CASES = [
    ([1], 8, 8), ([1], 64, 16), ([3, 0, 1], 72, 40), ([0, 0, 5], 256, 128), ([17, 64, 65, 0], 136, 264),
    ([127, 128, 129], 264, 72), ([255, 256, 257, 1], 200, 520), ([600, 2, 0, 31], 320, 256),
    ([2] * 70 + [0] * 30 + [1] * 30, 128, 64), ([40] * 3, 1032, 1024), ([300], 64, 1288),
    # many tiles of every height (one to nine 16-row subtiles a wave), each way
    ([255, 256, 257, 288, 289, 190, 170, 130, 96, 80, 64, 33, 17, 1, 0] * 4, 72, 1288),
    ([288, 240, 161, 96, 1] * 8, 1800, 72), ([3] * 200 + [0] * 40, 80, 520),
    # few rows and a long sum: slices, also across the two products of a pair
    ([5, 0, 70], 4104, 136), ([90], 136, 4104),
    ([1, 0, 2, 0] * 256, 64, 40),                         # as many experts as there may be
]
IDS = [f"{len(c)}x{max(c)}-K{k}-N{n}" for c, k, n in CASES]


def randn(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(BF)


def gen_of(*key):
    return torch.Generator(device=DEV).manual_seed(hash(key) % (1 << 31))


def problem(counts, K, N, pad=0, seed=0):
    """Rows with `pad` rows of NaN in front of the first and behind the last expert."""
    g = gen_of(len(counts), sum(counts), K, N, pad, seed)
    off = offsets_of(counts, pad)
    M = sum(counts) + 2 * pad
    live = slice(pad, M - pad)
    return g, off, M, live


def with_nan(t, live):
    out = torch.full_like(t, float("nan"))
    out[live] = t[live]
    return out


@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("counts,K,N", CASES, ids=IDS)
def test_linear(counts, K, N, pad):
    g, off, M, live = problem(counts, K, N, pad)
    x, w = with_nan(randn(g, M, K), live), randn(g, len(counts), N, K, scale=K ** -0.5)
    out = torch.full((M, N), 7.0, dtype=BF, device=DEV)
    B.moe_grouped_linear(x, w, off, out=out)
    ref, mag = product(x.to(F64), w, off)
    assert_within(out, ref, rounded(ref, K * U32 * mag), "linear", live)
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[live] = False
    assert (out[keep] == 7.0).all(), "rows outside the experts were written"


@pytest.mark.parametrize("counts,K,N", CASES, ids=IDS)
@pytest.mark.parametrize("k", [1, 3])
def test_linear_gathered(counts, K, N, k):
    g, off, M, live = problem(counts, K, N, seed=k)
    X = M // k + 2
    x = randn(g, X, K)
    slots = torch.randint(0, X * k, (M,), generator=g, device=DEV, dtype=torch.int32)
    slots[M // 2] = -1                                    # outside: read as zeros
    slots[M - 1] = X * k
    used = torch.zeros(X, dtype=torch.bool, device=DEV)
    used[(slots[(slots >= 0) & (slots < X * k)] // k).long()] = True
    x[~used] = float("nan")                               # tokens that no row names
    w = randn(g, len(counts), N, K, scale=K ** -0.5)
    got = B.moe_grouped_linear(x.view(torch.int16), w.view(torch.int16), off, slots, k)
    assert got.dtype == torch.int16
    ref, mag = product(source_rows(x.nan_to_num(), slots, k, M), w, off)
    assert_within(got.view(BF), ref, rounded(ref, K * U32 * mag), "linear gathered")


@pytest.mark.parametrize("counts,K,N", CASES, ids=IDS)
@pytest.mark.parametrize("save", [False, True])
def test_swiglu(counts, K, N, save):
    g, off, M, live = problem(counts, K, N, seed=7)
    x = randn(g, M, K, scale=3.0)
    gate, up = (randn(g, len(counts), N, K, scale=K ** -0.5) for _ in range(2))
    got = B.moe_grouped_swiglu(x, gate, up, off, save=save)
    a, am = product(x.to(F64), gate, off)
    b, bm = product(x.to(F64), up, off)
    ea, eb = K * U32 * am, K * U32 * bm
    h = swiglu(a, b)
    assert_within(got[0] if save else got, h, rounded(h, swiglu_error(a, ea, b, eb)), "h")
    if save:
        assert_within(got[1], a, rounded(a, ea), "a")
        assert_within(got[2], b, rounded(b, eb), "b")


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("counts,K,N", CASES, ids=IDS)
def test_dgrad(counts, K, N, pair, pad):
    g, off, M, live = problem(counts, K, N, pad, seed=2)
    dy = [with_nan(randn(g, M, N), live) for _ in range(1 + pair)]
    w = [randn(g, len(counts), N, K, scale=N ** -0.5) for _ in range(1 + pair)]
    out = torch.full((M, K), 7.0, dtype=BF, device=DEV)
    B.moe_grouped_linear_dgrad(dy[0], w[0], off, *((dy[1], w[1]) if pair else ()), out=out)
    ref = mag = 0
    for d, v in zip(dy, w):
        r, m = product(d.to(F64), v, off, transpose=False)
        ref, mag = ref + r, mag + m
    assert_within(out, ref, rounded(ref, (1 + pair) * N * U32 * mag), "dgrad", live)
    assert (out[:pad] == 7.0).all() and (out[M - pad:] == 7.0).all()


@pytest.mark.parametrize("scale", [1.0, 40.0])
@pytest.mark.parametrize("counts,K,N", CASES, ids=IDS)
def test_swiglu_dgrad(counts, K, N, scale):
    g, off, M, live = problem(counts, K, N, seed=3)
    dy, w = randn(g, M, N), randn(g, len(counts), N, K, scale=N ** -0.5)
    a, b = randn(g, M, K, scale=scale), randn(g, M, K, scale=scale)
    da, db = B.moe_grouped_swiglu_dgrad(dy, w, a, b, off)
    dh, mag = product(dy.to(F64), w, off, transpose=False)
    e = N * U32 * mag
    a, b = a.to(F64), b.to(F64)
    s = torch.sigmoid(a)
    fa, fb = b * s * (1 + a * (1 - s)), a * s
    # the factors in fp32: relative error of s at most (|a| + 8) 2^-22, of
    # 1 - s the same against s; 2^-100 covers factors below fp32's normals
    rel = (a.abs() + 8) * 2.0 ** -22
    ga = b.abs() * s * (1 + a.abs()) * 4 * rel + b.abs() * 2.0 ** -100
    gb = (a * s).abs() * 2 * rel + 2.0 ** -100
    assert_within(da, dh * fa, rounded(dh * fa, e * fa.abs() + (dh.abs() + e) * ga), "da")
    assert_within(db, dh * fb, rounded(dh * fb, e * fb.abs() + (dh.abs() + e) * gb), "db")


def wgrad_ref(dy, rows, off, N, K):
    E = off.numel() - 1
    ref = torch.zeros((E, N, K), dtype=F64, device=DEV)
    mag = torch.zeros_like(ref)
    n = torch.zeros((E, 1, 1), dtype=F64, device=DEV)
    for e, lo, hi in experts_rows(off):
        d = dy[lo:hi].to(F64).t().contiguous()
        ref[e], mag[e] = d @ rows[lo:hi], d.abs() @ rows[lo:hi].abs()
        n[e] = hi - lo
    return ref, mag, n


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("counts,K,N", CASES + [([5000], 136, 72), ([3000, 1, 2500], 64, 264), ([700, 200, 400], 136, 256),
                                                  ([4999], 72, 512)],
                         ids=IDS + ["1x5000", "3x3000", "3x700", "1x4999"])
def test_wgrad(counts, K, N, pad):
    g, off, M, live = problem(counts, K, N, pad, seed=4)
    dy, x = with_nan(randn(g, M, N), live), with_nan(randn(g, M, K), live)
    got = B.moe_grouped_linear_wgrad(dy, x, off)
    ref, mag, n = wgrad_ref(dy, x.to(F64), off, N, K)
    assert_within(got, ref, n * U32 * mag, "wgrad")
    before = torch.randn(got.shape, generator=g, device=DEV)
    acc = before.clone()
    assert B.moe_grouped_linear_wgrad(dy, x, off, out=acc, accumulate=True) is acc
    want = before.to(F64) + ref
    assert_within(acc, want, n * U32 * mag + 2 * U32 * (before.abs() + ref.abs()), "wgrad accumulated")
    empty = torch.tensor([c == 0 for c in counts], device=DEV)
    assert (got[empty] == 0).all() and torch.equal(acc[empty], before[empty])


@pytest.mark.parametrize("counts,K,N", CASES + [([5000], 136, 72), ([4999, 1100], 264, 512)], ids=IDS + ["1x5000", "2x4999"])
@pytest.mark.parametrize("k", [1, 7])
def test_wgrad_gathered(counts, K, N, k):
    g, off, M, live = problem(counts, K, N, seed=5 + k)
    X = M // k + 3
    x, dy = randn(g, X, K), randn(g, M, N)
    slots = torch.randint(0, X * k, (M,), generator=g, device=DEV, dtype=torch.int32)
    slots[0] = -5
    slots[M // 3] = X * k + 1
    got = B.moe_grouped_linear_wgrad(dy, x, off, slots, k)
    ref, mag, n = wgrad_ref(dy, source_rows(x, slots, k, M), off, N, K)
    assert_within(got, ref, n * U32 * mag, "wgrad gathered")


@pytest.mark.parametrize("counts", [[500, 0, 1301, 700], [300, 1, 0, 640]], ids=["long", "mean 235"])
@pytest.mark.parametrize("gather", [False, True])
def test_wgrad_wide(counts, gather):
    """More tiles than CUs, none of them full at the edges: no slices."""
    K, N, k = 4104, 1000, 3
    g, off, M, live = problem(counts, K, N, seed=9)
    assert B.moe_grouped_linear_wgrad_workspace_size(M, N, K, len(counts)) == 0
    dy = randn(g, M, N)
    if gather:
        x = randn(g, M // k + 1, K)
        slots = torch.randint(0, x.shape[0] * k, (M,), generator=g, device=DEV, dtype=torch.int32)
        slots[2] = -1
        rows, got = source_rows(x, slots, k, M), B.moe_grouped_linear_wgrad(dy, x, off, slots, k)
    else:
        x = randn(g, M, K)
        rows, got = x.to(F64), B.moe_grouped_linear_wgrad(dy, x, off)
    ref, mag, n = wgrad_ref(dy, rows, off, N, K)
    assert_within(got, ref, n * U32 * mag, "wgrad wide")


def test_offsets_outside_are_clamped():
    """Offsets below 0 or past M count as 0 or M; descending ones hold no rows."""
    g = gen_of(1)
    M, K, N = 100, 64, 64
    x, w = randn(g, M, K), randn(g, 4, N, K)
    bad = torch.tensor([-7, 30, 20, 60, 1 << 30], dtype=torch.int32, device=DEV)
    good = torch.tensor([0, 30, 30, 60, 100], dtype=torch.int32, device=DEV)
    out = torch.zeros((M, N), dtype=BF, device=DEV)
    y = B.moe_grouped_linear(x, w, bad, out=out.clone())
    ref, mag = product(x.to(F64), w, good)
    r2, m2 = product(x.to(F64)[20:60], w[2:3], offsets_of([40]))
    # rows 20..29 belong to experts 0 and 2 at once: either result
    err, e2 = rounded(ref, K * U32 * mag), rounded(r2, K * U32 * m2)
    assert_within(y, ref, err, "clamped", slice(30, 100))
    assert_within(y[:20], ref[:20], err[:20], "clamped first")
    assert_within(y[20:60], torch.where(((y[20:60].to(F64) - r2).abs() <= e2), r2, ref[20:60]),
                  torch.maximum(e2, err[20:60]), "overlap")


def test_zero_rows_and_all_empty():
    g = gen_of(2)
    w = randn(g, 3, 16, 24)
    none = torch.empty((0, 24), dtype=BF, device=DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert B.moe_grouped_linear(none, w, off).shape == (0, 16)
    assert B.moe_grouped_swiglu(none, w, w, off).shape == (0, 16)
    dy0 = torch.empty((0, 16), dtype=BF, device=DEV)
    assert B.moe_grouped_linear_dgrad(dy0, w, off).shape == (0, 24)
    dw = B.moe_grouped_linear_wgrad(dy0, none, off)
    assert dw.shape == (3, 16, 24) and (dw == 0).all()
    x = randn(g, 9, 24)
    out = torch.full((9, 16), 3.0, dtype=BF, device=DEV)
    assert (B.moe_grouped_linear(x, w, off, out=out) == 3.0).all()


def test_infinities_stay_in_their_rows():
    """A row with an infinity or NaN gives its own row nothing finite and leaves every other row as it was."""
    g = gen_of(3)
    counts, K, N = [70, 200], 72, 136
    off = offsets_of(counts)
    x, w = randn(g, 270, K), randn(g, 2, N, K)
    clean = B.moe_grouped_linear(x, w, off)
    bad = x.clone()
    bad[5, 3], bad[100, 71], bad[269, 0] = float("inf"), float("nan"), float("-inf")
    got = B.moe_grouped_linear(bad, w, off)
    rows = torch.ones(270, dtype=torch.bool, device=DEV)
    rows[[5, 100, 269]] = False
    assert torch.equal(got[rows], clean[rows])
    assert not torch.isfinite(got[~rows]).any()


def test_repeatable_and_on_another_stream():
    g = gen_of(4)
    counts, K, N = [300, 5, 0, 130], 520, 264
    off = offsets_of(counts)
    M = sum(counts)
    x, w, dy = randn(g, M, K), randn(g, 4, N, K), randn(g, M, N)
    want = B.moe_grouped_linear(x, w, off), B.moe_grouped_linear_dgrad(dy, w, off), B.moe_grouped_linear_wgrad(dy, x, off)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = (B.moe_grouped_linear(x, w, off, stream=side), B.moe_grouped_linear_dgrad(dy, w, off, stream=side),
               B.moe_grouped_linear_wgrad(dy, x, off, stream=side))
        side.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_long_rows_pass_31_bits():
    """Rows whose byte offset passes 2^32 (not gathered: the rows' base moves with the tile)."""
    K, N, M = 8192, 16, 262144 + 40                       # M * K * 2 = 4.3 GB
    g = gen_of(5)
    x = torch.zeros((M, K), dtype=BF, device=DEV)
    x[-40:] = randn(g, 40, K)
    x[:40] = randn(g, 40, K)
    w = randn(g, 2, N, K, scale=K ** -0.5)
    off = torch.tensor([0, M - 39, M], dtype=torch.int32, device=DEV)
    got = B.moe_grouped_linear(x, w, off)
    rows = torch.cat((torch.arange(40, device=DEV), torch.arange(M - 40, M, device=DEV)))
    small = x[rows].to(F64)
    ref, mag = product(small, w, torch.tensor([0, 41, 80], dtype=torch.int32, device=DEV))
    assert_within(got[rows], ref, rounded(ref, K * U32 * mag), "long rows")
    dw = B.moe_grouped_linear_wgrad(got, x, off)
    ref, mag, n = wgrad_ref(got[rows], small, torch.tensor([0, 41, 80], dtype=torch.int32, device=DEV), N, K)
    assert_within(dw, ref, 80 * U32 * mag, "long rows wgrad")
    log(f"rows of {M * K * 2 / 2 ** 30:.1f} GiB")


def test_gathered_rows_past_the_offset_range_are_refused():
    x = torch.empty((1, 1 << 20), dtype=BF, device=DEV)
    w = torch.empty((1, 8, 1 << 20), dtype=BF, device=DEV)
    off, slots = offsets_of([1]), torch.zeros(1, dtype=torch.int32, device=DEV)
    L = B.lib()
    out = torch.empty((1, 8), dtype=BF, device=DEV)
    st = L.moe_grouped_linear(x.data_ptr(), 4096, 1 << 20, w.data_ptr(), 1, 8, off.data_ptr(), slots.data_ptr(), 1, 1,
                              out.data_ptr(), None, 0, None)
    assert B.STATUS[st] == "MOE_ERR_SHAPE"
