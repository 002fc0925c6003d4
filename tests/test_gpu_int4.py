"""4-bit integer weights: packing bit for bit against its definition, and the
products against plain fp64 forms inside the summation and rounding bounds."""
import numpy as np
import pytest
import torch

from experts_util import F64, U32, assert_within, experts_rows, offsets_of, rounded, source_rows
from gpu_util import DEV
from nvfp4_weight_only_moe_amd import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def bf16_rne(a):
    return torch.from_numpy(a).to(BF).to(torch.float32).numpy()


def pack_ref(w, G, zeros):
    """The definition in numpy fp32 (correctly rounded operations)."""
    E, N, K = w.shape
    v = w.reshape(E, N, K // G, G).astype(np.float32)
    lo, hi = np.minimum(v.min(-1), 0), np.maximum(v.max(-1), 0)
    s = bf16_rne(((hi - lo) / np.float32(15)) if zeros else (np.maximum(hi, -lo) / np.float32(7)))
    s = np.where(s == 0, np.float32(1), s)
    z = np.clip(np.rint(-lo / s), 0, 15) if zeros else np.full_like(s, 8)
    c = np.clip(np.rint(v / s[..., None]) + z[..., None], 0, 15).astype(np.uint8).reshape(E, N, K)
    return c[..., 0::2] | (c[..., 1::2] << 4), s, z.astype(np.uint8)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("E,N,K,G", [(1, 1, 128, 128), (2, 5, 256, 32), (3, 17, 384, 64)])
def test_pack(E, N, K, G, zeros):
    rng = np.random.default_rng([E, N, K, G])
    w = (rng.standard_normal((E, N, K)) * 0.02).astype(np.float32)
    w[0, 0, :G] = 0.0                                     # a group of zeros
    if N > 1:
        w[0, 1, :G] = np.abs(w[0, 1, :G])                 # one sign only
    t = B.moe_int4_quantize_pack(torch.from_numpy(w).to(DEV), G, zeros)
    codes, s, z = pack_ref(w, G, zeros)
    assert np.array_equal(t.codes.cpu().numpy(), codes)
    assert np.array_equal(t.scales.float().cpu().numpy(), s)
    if zeros:
        assert np.array_equal(t.zeros.cpu().numpy(), z)
    c = np.stack((codes & 15, codes >> 4), -1).reshape(E, N, K // G, G).astype(np.float32)
    deq = ((c - z[..., None].astype(np.float32)) * s[..., None]).reshape(E, N, K)
    assert np.array_equal(B.moe_int4_dequantize(t).cpu().numpy(), deq)


def weights(g, E, N, K, G, zeros):
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = ((torch.rand((E, N, K // G), generator=g, device=DEV) - 0.3) * 0.01).to(BF)
    z = torch.randint(0, 16, (E, N, K // G), generator=g, device=DEV, dtype=torch.uint8) if zeros else None
    return B.Int4Tensor(codes, scales, z)


def reference(rows, t, off):
    E, N, K = t.shape
    G = t.group
    c = torch.stack((t.codes & 15, t.codes >> 4), -1).view(E, N, K // G, G).to(F64)
    z = 8.0 if t.zeros is None else t.zeros.to(F64)[..., None]
    s = t.scales.to(F64)[..., None]
    w = ((c - z) * s).view(E, N, K)
    # magnitudes that the sums meet: 128 + code, and the offset times the row's sum
    m = ((128 + c) * s.abs() + (128 + z) * s.abs()).view(E, N, K)
    ref = torch.zeros((rows.shape[0], N), dtype=F64, device=DEV)
    mag = torch.zeros_like(ref)
    for e, lo, hi in experts_rows(off):
        ref[lo:hi] = rows[lo:hi] @ w[e].t().contiguous()
        mag[lo:hi] = rows[lo:hi].abs() @ m[e].t().contiguous()
    return ref, mag


def check(got, rows, t, off, what, live=slice(None)):
    ref, mag = reference(rows, t, off)
    # inside a group (group + 4 roundings), then one per group
    n = t.group + 4 + t.shape[2] // t.group
    assert_within(got, ref, rounded(ref, n * U32 * mag), what, live)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("T,K,N", [(1, 128, 1), (1, 1024, 512), (2, 384, 33), (5, 640, 100), (16, 256, 64),
                                   (17, 512, 48), (33, 1152, 130), (64, 256, 256), (100, 384, 272), (300, 128, 17)])
def test_dense(T, K, N, G, zeros):
    g = torch.Generator(device=DEV).manual_seed(T * 7919 + K + N + G)
    t = weights(g, 1, N, K, G, zeros)
    x = torch.randn((T, K), generator=g, device=DEV).to(BF)
    check(B.moe_int4_linear(x, t), x.to(F64), t, offsets_of([T]), "dense")


@pytest.mark.parametrize("zeros,G", [(False, 32), (True, 64), (True, 128)])
@pytest.mark.parametrize("counts,K,N", [([1, 0, 2], 256, 40), ([16, 17, 1, 0, 0, 3], 128, 64),
                                        ([0, 90, 33], 384, 24), ([1] * 70, 128, 16), ([200, 1], 256, 272)])
@pytest.mark.parametrize("k", [0, 1, 4])
def test_experts(counts, K, N, G, zeros, k):
    g = torch.Generator(device=DEV).manual_seed(sum(counts) * 31 + K + N + G + k)
    t = weights(g, len(counts), N, K, G, zeros)
    M, pad = sum(counts) + 4, 2
    off = offsets_of(counts, pad)
    live = slice(pad, M - pad)
    out = torch.full((M, N), 5.0, dtype=BF, device=DEV)
    if k == 0:
        x = torch.randn((M, K), generator=g, device=DEV).to(BF)
        x[:pad] = float("nan")
        x[M - pad:] = float("nan")
        B.moe_int4_linear(x, t, off, out=out)
        rows = x.to(F64)
    else:
        X = M // k + 1
        x = torch.randn((X, K), generator=g, device=DEV).to(BF)
        slots = torch.randint(0, X * k, (M,), generator=g, device=DEV, dtype=torch.int32)
        slots[pad] = -3
        B.moe_int4_linear(x, t, off, slots, k, out=out)
        rows = source_rows(x, slots, k, M)
    check(out, rows, t, off, "experts", live)
    assert (out[:pad] == 5.0).all() and (out[M - pad:] == 5.0).all()


@pytest.mark.parametrize("zeros,G", [(False, 32), (True, 64), (True, 128)])
@pytest.mark.parametrize("counts,K,N", [([3, 0, 16, 5] * 10, 640, 500), ([3, 0, 17, 5] * 10, 256, 250),
                                        ([3, 0, 16, 5] * 10, 4224, 130), ([3, 0, 16, 5] * 10, 384, 100),
                                        ([20, 31, 33, 1] * 4, 640, 1500), ([20, 31, 33, 1] * 4, 1152, 750),
                                        ([60, 65, 40, 1, 0, 100] * 4, 640, 2000)])
def test_experts_wide_tiles(counts, K, N, G, zeros):
    """Enough experts and columns for every width of a tile, none of them a multiple of it."""
    g = torch.Generator(device=DEV).manual_seed(sum(counts) + K + N + G)
    t = weights(g, len(counts), N, K, G, zeros)
    M, k = sum(counts), 2
    x = torch.randn((M // k + 1, K), generator=g, device=DEV).to(BF)
    slots = torch.randint(0, x.shape[0] * k, (M,), generator=g, device=DEV, dtype=torch.int32)
    slots[1] = -1
    off = offsets_of(counts)
    check(B.moe_int4_linear(x, t, off, slots, k), source_rows(x, slots, k, M), t, off, "wide")


@pytest.mark.parametrize("T,K,N", [(1000, 640, 2900), (16, 128, 20500), (40, 384, 6300)])
def test_dense_wide_tiles(T, K, N):
    g = torch.Generator(device=DEV).manual_seed(T + K + N)
    t = weights(g, 1, N, K, 128, True)
    x = torch.randn((T, K), generator=g, device=DEV).to(BF)
    check(B.moe_int4_linear(x, t), x.to(F64), t, offsets_of([T]), "dense wide")


def test_large_common_offset_of_x():
    """Rows far from zero: the offset's sum is large against the result."""
    g = torch.Generator(device=DEV).manual_seed(3)
    t = weights(g, 1, 64, 1024, 128, True)
    x = (torch.randn((4, 1024), generator=g, device=DEV) + 50.0).to(BF)
    check(B.moe_int4_linear(x, t), x.to(F64), t, offsets_of([4]), "offset")


def test_pack_then_product_matches_the_masters():
    g = torch.Generator(device=DEV).manual_seed(4)
    w = torch.randn((1, 96, 512), generator=g, device=DEV) * 0.02
    x = torch.randn((3, 512), generator=g, device=DEV).to(BF)
    for zeros in (False, True):
        t = B.moe_int4_quantize_pack(w, 32, zeros)
        # a code is at most 0.5 + its clamp away: |w - deq| <= s (one step covers both)
        s = t.scales.to(F64).repeat_interleave(32, -1)[0]
        ref = x.to(F64) @ w[0].to(F64).t().contiguous()
        slack = x.to(F64).abs() @ s.t().contiguous()
        assert_within(B.moe_int4_linear(x, t), ref, rounded(ref, slack), "packed")
