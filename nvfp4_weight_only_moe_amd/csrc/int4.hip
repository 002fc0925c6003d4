// 4-bit integer weights with group scales and zero points: packing, and the
// product with bf16 rows, dense or by expert.
//
//   out[p][n] = sum_g s[n][g] sum_{k in g} (code[n][k] - z[n][g]) x[src(p)][k]
//
// The matrix units see 128 + code, exact in bf16 and one AND-OR per pair of
// codes (0x4300 is bf16's 128, whose last mantissa bit weighs 1); the offset
// 128 + z leaves with the group's sum of x, which a second MFMA against ones
// gives in the same registers.  Both sums are exact products accumulated in
// fp32; their difference loses at most the bits that 128 has over |code - z|
// (about 2^-19 of sum |code - z||x|, against the output's rounding of 2^-9).
// The group's scale multiplies in fp32: no weight is rounded.
#include "device_common.h"
#include "internal.h"

namespace moe {
namespace {

// ---------------------------------------------------------------- packing
__global__ void __launch_bounds__(256) k_int4_pack(const float* __restrict__ w, int64_t groups, int G,
                                                   uint8_t* __restrict__ codes, uint16_t* __restrict__ scales,
                                                   uint8_t* __restrict__ zeros) {
    const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (g >= groups) return;
    const float* v = w + g * G;
    float lo = 0.0f, hi = 0.0f;
    for (int i = 0; i < G; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(v + i);
        lo = fminf(fminf(fminf(lo, f.x), fminf(f.y, f.z)), f.w);
        hi = fmaxf(fmaxf(fmaxf(hi, f.x), fmaxf(f.y, f.z)), f.w);
    }
    const uint16_t sb = f32_to_bf16_rne(zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f);
    const float s = bf16_bits_to_f32(sb) > 0.0f ? bf16_bits_to_f32(sb) : 1.0f;
    const float z = zeros ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 8.0f;
    scales[g] = f32_to_bf16_rne(s);
    if (zeros) zeros[g] = (uint8_t)z;
    for (int i = 0; i < G; i += 8) {
        uint32_t word = 0;
        for (int j = 0; j < 8; ++j) {
            const float c = fminf(fmaxf(rintf(v[i + j] / s) + z, 0.0f), 15.0f);
            word |= (uint32_t)c << (4 * j);
        }
        *reinterpret_cast<uint32_t*>(codes + (g * G + i) / 2) = word;
    }
}

__global__ void __launch_bounds__(256) k_int4_dequant(const uint8_t* __restrict__ codes,
                                                      const uint16_t* __restrict__ scales,
                                                      const uint8_t* __restrict__ zeros, int64_t words, int G,
                                                      float* __restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= words) return;
    const uint32_t u = reinterpret_cast<const uint32_t*>(codes)[i];
    const int64_t g = i * 8 / G;
    const float s = bf16_bits_to_f32(scales[g]), z = zeros ? (float)zeros[g] : 8.0f;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = ((float)((u >> (4 * j)) & 15u) - z) * s;
    *reinterpret_cast<float4*>(out + i * 8) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(out + i * 8 + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// ---------------------------------------------------------------- product
struct Int4Params {
    const uint16_t* x;
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;
    const int32_t* offsets;       // null: one expert, rows 0 .. M - 1
    const int32_t* slots;
    int E, M, X, k, N, K, G;
    uint16_t* out;
};

constexpr int kIntWaves = 4;
constexpr int kTB = 16;           // rows per block of a workgroup

__device__ __forceinline__ u32x4 transpose4(u32x4 v) {
    // word j of lane row i (16 lanes) -> word i of lane row j
    auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{(uint32_t)c[0], (uint32_t)c[1], (uint32_t)d[0], (uint32_t)d[1]};
}

// 128 + code of the 8 codes of a word, in the order k0 k4 k1 k5 k2 k6 k3 k7
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t w) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    return __builtin_bit_cast(bf16x8, r);
}
// eight bf16 in that order
__device__ __forceinline__ bf16x8 order_x(uint4 v) {
    u32x4 r;
    r[0] = __builtin_amdgcn_perm(v.z, v.x, 0x05040100u);
    r[1] = __builtin_amdgcn_perm(v.z, v.x, 0x07060302u);
    r[2] = __builtin_amdgcn_perm(v.w, v.y, 0x05040100u);
    r[3] = __builtin_amdgcn_perm(v.w, v.y, 0x07060302u);
    return __builtin_bit_cast(bf16x8, r);
}

// One workgroup: 16 weight rows of one expert against up to 16 of its rows
// at a time; the four waves take the 128-code chunks of K in turn and join
// their sums through LDS.
template <int G>
__global__ void __launch_bounds__(kIntWaves * kWave) k_int4_mm(Int4Params P) {
    __shared__ floatx4 s_acc[kIntWaves][kWave];
    const int e = blockIdx.y;
    int p0 = 0, cnt = P.M;
    if (P.offsets) {
        p0 = max(P.offsets[e], 0);
        cnt = min(P.offsets[e + 1], P.M) - p0;
    }
    if (cnt <= 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lrow = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 16, n = min(n0 + lrow, P.N - 1);
    const int64_t wrow = (int64_t)e * P.N + n;
    const uint8_t* codes = P.codes + wrow * (P.K / 2) + q * 16;
    const uint16_t* scales = P.scales + wrow * (P.K / G);
    const uint8_t* zeros = P.zeros ? P.zeros + wrow * (P.K / G) : nullptr;
    const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
    const floatx4 zero4 = {0, 0, 0, 0};
    for (int r0 = 0; r0 < cnt; r0 += kTB) {
        int src = min(r0 + lrow, cnt - 1) + p0;
        bool ok = true;
        if (P.slots) {
            const int slot = P.slots[src];
            src = slot / P.k;
            ok = slot >= 0 && src < P.X;
        }
        const uint16_t* x = P.x + (int64_t)(ok ? src : 0) * P.K + q * 8;
        floatx4 acc = zero4;
        for (int c = wave; c < P.K / 128; c += kIntWaves) {
            const uint4 raw = *reinterpret_cast<const uint4*>(codes + (int64_t)c * 64);
            const u32x4 w = transpose4(u32x4{raw.x, raw.y, raw.z, raw.w});
            floatx4 dot = zero4, sum = zero4;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint4 xv = *reinterpret_cast<const uint4*>(x + c * 128 + ks * 32);
                if (!ok) xv = make_uint4(0, 0, 0, 0);
                const bf16x8 xf = order_x(xv);
                dot = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, codes_bf16(w[ks]), dot, 0, 0, 0);
                sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, ones, sum, 0, 0, 0);
                if ((ks + 1) % (G / 32) == 0) {
                    const int g = (c * 128 + ks * 32) / G;
                    const float s = bf16_bits_to_f32(scales[g]);
                    const float off = 128.0f + (zeros ? (float)zeros[g] : 8.0f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = fmaf(s, fmaf(-off, sum[i], dot[i]), acc[i]);
                    dot = zero4;
                    sum = zero4;
                }
            }
        }
        __syncthreads();
        s_acc[wave][lane] = acc;
        __syncthreads();
        // wave i writes rows 4 q + i of the block
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < kIntWaves; ++j) v += s_acc[j][lane][wave];
        const int r = r0 + q * 4 + wave;
        if (r < cnt && n0 + lrow < P.N) P.out[(int64_t)(p0 + r) * P.N + n0 + lrow] = f32_to_bf16_rne(v);
    }
}

}  // namespace

moe_status launch_int4_pack(const float* w, const moe_int4_tensor* t, hipStream_t s) {
    const int64_t groups = (int64_t)t->E * t->N * (t->K / t->group);
    MOE_LAUNCH("int4_pack", k_int4_pack, dim3((unsigned)((groups + 255) / 256)), dim3(256), 0, s, w, groups, t->group,
               t->codes, t->scales, t->zeros);
    return MOE_OK;
}

moe_status launch_int4_dequant(const moe_int4_tensor* t, float* out, hipStream_t s) {
    const int64_t words = (int64_t)t->E * t->N * t->K / 8;
    MOE_LAUNCH("int4_dequant", k_int4_dequant, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, s,
               (const uint8_t*)t->codes, (const uint16_t*)t->scales, (const uint8_t*)t->zeros, words, t->group, out);
    return MOE_OK;
}

moe_status launch_int4_linear(const uint16_t* x, int X, const moe_int4_tensor* t, const int32_t* offsets,
                              const int32_t* slots, int k, int M, uint16_t* out, hipStream_t s) {
    const Int4Params P{x, t->codes, t->scales, t->zeros, offsets, slots, t->E, M, X, k, t->N, t->K, t->group, out};
    const dim3 grid((t->N + 15) / 16, t->E), block(kIntWaves * kWave);
    if (t->group == 32) MOE_LAUNCH("int4_linear", k_int4_mm<32>, grid, block, 0, s, P);
    else if (t->group == 64) MOE_LAUNCH("int4_linear", k_int4_mm<64>, grid, block, 0, s, P);
    else MOE_LAUNCH("int4_linear", k_int4_mm<128>, grid, block, 0, s, P);
    return MOE_OK;
}

}  // namespace moe
