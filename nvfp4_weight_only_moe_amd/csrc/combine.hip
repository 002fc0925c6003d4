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

constexpr int kMaxThreads = 512;
constexpr int kSlots = 8;                 // slots whose rows are loaded together

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

__device__ __forceinline__ uint4 load_row(const uint16_t* p) { return load_stream16(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void store_row(uint16_t* p, uint4 v) {
    __builtin_nontemporal_store(nt_u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<nt_u32x4*>(p));
}

// One workgroup per token, eight columns a thread and pass.  HBM-bound: the
// rows of eight slots are requested before any is used (a dropped slot reads
// row 0 and drops it: no branch between the loads), past the caches, since each
// is used once.  4099 tokens, 8 slots of 5120: 79.7 us with the loads in a loop
// over the slots, 67.8 us so (378 MB: 5.6 TB/s; a copy reaches 5.1).
__global__ void __launch_bounds__(kMaxThreads) k_combine_rows(const uint16_t* __restrict__ y, int M, int H,
                                                              const int32_t* __restrict__ pos,
                                                              const float* __restrict__ w, int k,
                                                              uint16_t* __restrict__ out) {
    const int64_t t = blockIdx.x;
    for (int c = threadIdx.x * 8; c < H; c += blockDim.x * 8) {
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int j0 = 0; M > 0 && j0 < k; j0 += kSlots) {
            uint4 v[kSlots];
            float wj[kSlots];
            bool ok[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                const int64_t s = t * k + min(j0 + j, k - 1);
                const int p = pos[s];
                ok[j] = j0 + j < k && (unsigned)p < (unsigned)M;
                wj[j] = w ? w[s] : 1.0f;
                v[j] = load_row(y + (int64_t)(ok[j] ? p : 0) * H + c);
            }
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                if (!ok[j]) continue;                     // the same for the whole workgroup
                float f[8];
                widen8(v[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(wj[j], f[i], acc[i]);
            }
        }
        *reinterpret_cast<uint4*>(out + t * H + c) = narrow8(acc);
    }
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

// One workgroup per token: a piece of dout's row meets the rows of eight
// slots at a time (requested together, as above), whose dy rows leave at once
// (2048 tokens, 8 slots of 5120: 84 -> 72 us, 5.0 TB/s).
template <bool DOT>
__global__ void __launch_bounds__(kMaxThreads) k_combine_bwd(CombineBwd P) {
    __shared__ float s_part[kMaxThreads / kWave][MOE_MAX_TOPK];
    __shared__ float s_dw[MOE_MAX_TOPK], s_g[MOE_MAX_TOPK];
    __shared__ int s_id[MOE_MAX_TOPK];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j0 = 0; j0 < P.k; j0 += kSlots) {
        int64_t row[kSlots];
        float wj[kSlots], dot[kSlots];
        bool ok[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int64_t s = t * P.k + min(j0 + j, P.k - 1);
            const int p = P.pos[s];
            ok[j] = j0 + j < P.k && (unsigned)p < (unsigned)P.M;
            wj[j] = P.w ? P.w[s] : 1.0f;
            row[j] = (int64_t)(ok[j] ? p : 0) * P.H;
            dot[j] = 0.0f;
        }
        for (int c = threadIdx.x * 8; c < P.H; c += blockDim.x * 8) {
            const uint4 dv = *reinterpret_cast<const uint4*>(P.dout + t * P.H + c);
            uint4 v[kSlots];
            if constexpr (DOT) {
                if (P.M > 0)
#pragma unroll
                    for (int j = 0; j < kSlots; ++j) v[j] = load_row(P.y + row[j] + c);
            }
            float d[8];
            widen8(dv, d);
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                if (!ok[j]) continue;                     // the same for the whole workgroup
                float o[8];
                if constexpr (DOT) {
                    float f[8];
                    widen8(v[j], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[j] = fmaf(d[i], f[i], dot[j]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = wj[j] * d[i];
                store_row(P.dy + row[j] + c, narrow8(o));
            }
        }
        if constexpr (DOT) {
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                const float sum = wave_sum_dpp(dot[j]);
                if (lane == 0 && j0 + j < P.k) s_part[wave][j0 + j] = sum;
            }
        }
    }
    if constexpr (!DOT) return;
    __syncthreads();
    if ((int)threadIdx.x < P.k) {
        float v = 0.0f;
        for (int i = 0; i < (int)blockDim.x / kWave; ++i) v += s_part[i][threadIdx.x];
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
    for (int e = threadIdx.x; e < P.E; e += blockDim.x) {
        float v = 0.0f;
        for (int j = 0; j < P.k; ++j) v += s_id[j] == e ? s_g[j] : 0.0f;
        P.dlogits[t * P.E + e] = v;
    }
}

// Threads of a workgroup: whole waves, H / 8 shared out over as few equal passes as 512 allow.
dim3 row_threads(int H) {
    const int passes = (H / 8 + kMaxThreads - 1) / kMaxThreads;
    return dim3(((H / 8 + passes - 1) / passes + kWave - 1) / kWave * kWave);
}

}  // namespace

moe_status launch_combine_rows(const uint16_t* y, int M, int H, const int32_t* pos, const float* w, int T, int k,
                               uint16_t* out, hipStream_t s) {
    MOE_LAUNCH("combine_rows", k_combine_rows, dim3(T), row_threads(H), 0, s, y, M, H, pos, w, k, out);
    return MOE_OK;
}

moe_status launch_combine_bwd(const uint16_t* dout, const uint16_t* y, const int32_t* pos, const float* w,
                              const int32_t* ids, int T, int M, int H, int k, int E, uint16_t* dy, float* dw,
                              float* dlogits, hipStream_t s) {
    CombineBwd P{dout, y, pos, w, ids, M, H, k, E, dy, dw, dlogits};
    if (dw || dlogits) MOE_LAUNCH("combine_bwd", k_combine_bwd<true>, dim3(T), row_threads(H), 0, s, P);
    else MOE_LAUNCH("combine_bwd", k_combine_bwd<false>, dim3(T), row_threads(H), 0, s, P);
    return MOE_OK;
}

}  // namespace moe
