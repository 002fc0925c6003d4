// The routing-weighted combine of the experts' rows, and its gradients.
//
//   out[t]          = sum_j w[t][j] y[pos[t][j]]
//   dy[pos[t][j]]   = w[t][j] dout[t]
//   dw[t][j]        = <dout[t], y[pos[t][j]]>
//   dlogits[t][e]   = sum_{j: ids[t][j] = e} w[t][j] (dw[t][j] - sum_i w[t][i] dw[t][i])
// (the last: w is the softmax over the k selected logits).  A slot whose
// position lies outside [0, M) was dropped: it adds nothing, its dw is 0.
// Sums in fp32 in slot order, one rounding to bf16 per output.
#include "device_common.h"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = kThreads * 8;       // columns per pass of a workgroup

__device__ __forceinline__ void widen8(uint4 v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_bits_to_f32(u[i] & 0xFFFFu);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = (uint32_t)f32_to_bf16_rne(f[2 * i]) | ((uint32_t)f32_to_bf16_rne(f[2 * i + 1]) << 16);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__global__ void __launch_bounds__(kThreads) k_combine_rows(const uint16_t* __restrict__ y, int M, int H,
                                                           const int32_t* __restrict__ pos,
                                                           const float* __restrict__ w, int k,
                                                           uint16_t* __restrict__ out) {
    const int64_t t = blockIdx.x;
    const int c = (blockIdx.y * kThreads + threadIdx.x) * 8;
    if (c >= H) return;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j = 0; j < k; ++j) {
        const int p = pos[t * k + j];
        if ((unsigned)p >= (unsigned)M) continue;
        const float wj = w ? w[t * k + j] : 1.0f;
        float f[8];
        widen8(*reinterpret_cast<const uint4*>(y + (int64_t)p * H + c), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(wj, f[i], acc[i]);
    }
    *reinterpret_cast<uint4*>(out + t * H + c) = narrow8(acc);
}

struct CombineBwd {
    const uint16_t* dout;
    const uint16_t* y;
    const int32_t* pos;
    const float* w;
    const int32_t* ids;
    int M, H, k, E;
    uint16_t* dy;
    float* dw;
    float* dlogits;
};

// One workgroup per token: dout's row is read once and meets the k rows.
__global__ void __launch_bounds__(kThreads) k_combine_bwd(CombineBwd P) {
    __shared__ float s_part[kThreads / kWave][MOE_MAX_TOPK];
    __shared__ float s_dw[MOE_MAX_TOPK], s_g[MOE_MAX_TOPK];
    __shared__ int s_id[MOE_MAX_TOPK];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j = 0; j < P.k; ++j) {
        const int p = P.pos[t * P.k + j];
        const bool ok = (unsigned)p < (unsigned)P.M;
        const float wj = P.w ? P.w[t * P.k + j] : 1.0f;
        float dot = 0.0f;
        for (int c = threadIdx.x * 8; ok && c < P.H; c += kCols) {
            float d[8], o[8];
            widen8(*reinterpret_cast<const uint4*>(P.dout + t * P.H + c), d);
            if (P.dw || P.dlogits) {
                float f[8];
                widen8(*reinterpret_cast<const uint4*>(P.y + (int64_t)p * P.H + c), f);
#pragma unroll
                for (int i = 0; i < 8; ++i) dot = fmaf(d[i], f[i], dot);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = wj * d[i];
            *reinterpret_cast<uint4*>(P.dy + (int64_t)p * P.H + c) = narrow8(o);
        }
        dot = wave_sum_dpp(dot);
        if (lane == 0) s_part[wave][j] = dot;
    }
    if (!P.dw && !P.dlogits) return;
    __syncthreads();
    if ((int)threadIdx.x < P.k) {
        float v = 0.0f;
        for (int i = 0; i < kThreads / kWave; ++i) v += s_part[i][threadIdx.x];
        s_dw[threadIdx.x] = v;
        if (P.dw) P.dw[t * P.k + threadIdx.x] = v;
    }
    if (!P.dlogits) return;
    __syncthreads();
    if ((int)threadIdx.x < P.k) {
        float mean = 0.0f;
        for (int i = 0; i < P.k; ++i) mean = fmaf(P.w[t * P.k + i], s_dw[i], mean);
        s_g[threadIdx.x] = P.w[t * P.k + threadIdx.x] * (s_dw[threadIdx.x] - mean);
        s_id[threadIdx.x] = P.ids[t * P.k + threadIdx.x];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < P.E; e += kThreads) {
        float v = 0.0f;
        for (int j = 0; j < P.k; ++j) v += s_id[j] == e ? s_g[j] : 0.0f;
        P.dlogits[t * P.E + e] = v;
    }
}

}  // namespace

moe_status launch_combine_rows(const uint16_t* y, int M, int H, const int32_t* pos, const float* w, int T, int k,
                               uint16_t* out, hipStream_t s) {
    MOE_LAUNCH("combine_rows", k_combine_rows, dim3(T, (H + kCols - 1) / kCols), dim3(kThreads), 0, s, y, M, H, pos, w,
               k, out);
    return MOE_OK;
}

moe_status launch_combine_bwd(const uint16_t* dout, const uint16_t* y, const int32_t* pos, const float* w,
                              const int32_t* ids, int T, int M, int H, int k, int E, uint16_t* dy, float* dw,
                              float* dlogits, hipStream_t s) {
    CombineBwd P{dout, y, pos, w, ids, M, H, k, E, dy, dw, dlogits};
    MOE_LAUNCH("combine_bwd", k_combine_bwd, dim3(T), dim3(kThreads), 0, s, P);
    return MOE_OK;
}

}  // namespace moe
