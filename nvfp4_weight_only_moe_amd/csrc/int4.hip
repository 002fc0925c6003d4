// 4-bit integer weights with group scales and zero points: packing, and the
// product with bf16 rows, dense or by expert.
//
//   out[p][n] = sum_g s[n][g] sum_{k in g} (code[n][k] - z[n][g]) x[src(p)][k]
//
// The matrix units see 128 + code, exact in bf16 and one AND-OR per pair of
// codes (0x4300 is bf16's 128, whose last mantissa bit weighs 1); the offset
// 128 + z leaves with the group's sum of x.  Products are exact and accumulate
// in fp32; their difference loses at most the bits that 128 has over |code - z|
// (about 2^-19 of sum |code - z||x|, against the output's rounding of 2^-9).
// The group's scale multiplies in fp32: no weight is rounded.
#include "device_common.h"
#include "expert_rows.h"
#include "internal.h"

#include <algorithm>

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
    int E, M, X, k, N, K;
    uint32_t kmagic;
    int ntn;                      // column tiles
    uint16_t* out;
};

constexpr int kIntThreads = 512, kIntWaves = kIntThreads / kWave;
constexpr int kRing = 4;          // chunks of a wave on their way, a power of two
constexpr int kSlot = 1024;       // bytes of a chunk's codes: 16 rows x 64
constexpr int kMeta = 256;        // a word per lane of scales and zero points

__device__ __forceinline__ u32x4 transpose4(u32x4 v) {
    // word j of lane row i (16 lanes) -> word i of lane row j
    auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{(uint32_t)c[0], (uint32_t)c[1], (uint32_t)d[0], (uint32_t)d[1]};
}

// 128 + code, two codes of a word at a time.  The constants sit in vector
// registers, so that the AND-OR is one instruction: it has room for one
// constant of another kind, and with both the compiler splits it.
struct Codes128 {
    uint32_t low4 = 0x000F000Fu, base = 0x43004300u;
    __device__ __forceinline__ Codes128() { asm("" : "+v"(low4), "+v"(base)); }
    __device__ __forceinline__ uint32_t pair(uint32_t w, int i) const { return ((w >> (4 * i)) & low4) | base; }
    // the 8 codes of a word, in the order k0 k4 k1 k5 k2 k6 k3 k7
    __device__ __forceinline__ bf16x8 word(uint32_t w) const {
        return __builtin_bit_cast(bf16x8, u32x4{pair(w, 0), pair(w, 1), pair(w, 2), pair(w, 3)});
    }
};
// eight bf16 in that order
__device__ __forceinline__ uint4 order_x(uint4 v) {
    return make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                      __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
}

// LDS of a workgroup against 16 TT rows of x: x (slab by slab of K), the
// groups' sums of it, the rings of weights.
template <int G, int RT, int TT, bool ZP>
struct Int4Lds {
    static constexpr int kUnits = TT <= 2 ? 4 : 8;               // 16-byte units of x a thread brings per slab
    static constexpr int kX = kUnits * kIntThreads * 16 + 16 * TT * 16;      // rows are 16 bytes longer than a slab
    static constexpr int kSums = 4096;
    static constexpr int kMetas = G == 32 && ZP ? 2 : 1;         // words per lane of a pair of chunks
    static constexpr int kCodes = kRing * RT * kSlot;            // of a wave, then its kRing / 2 pairs' words
    static constexpr int kWave1 = kCodes + kRing / 2 * RT * kMetas * kMeta, kRings = kIntWaves * kWave1;
    static constexpr int kBytes = kX + kSums + kRings;
    static_assert(kIntWaves * RT * TT * 1024 <= kX + kSums + kRings, "the K parts meet in the same memory");
};

// One workgroup: 16 RT WR weight rows of one expert against 16 TT of its rows.
// The eight waves are WR along the weight rows by WK = 8 / WR along K, in
// chunks of 128 codes in turn; the K parts meet in LDS at the end.
//
// Weights: a wave's chunks run through a ring of its own in LDS, kRing deep,
// by LDS-DMA (16 rows x 64 bytes; the scales and zero points of two chunks in
// a word per lane: with a word per lane and chunk, 64 experts, 1536 x 5120,
// 8 rows of x, group 32: 50 us, 45 so), so that the loop over chunks stays rolled: unrolled
// with its loads in registers its code is fetched as slowly as the weights
// (one row of x, 5120 x 5120: 11.6 us).
// x: a slab of its columns at a time, the next slab's loads issued before this
// slab's products, stored in the order of the decoded codes with the sum of
// every group.
// The MFMA's A operand is x, so a lane's outputs belong to one weight row,
// whose scale it reads: dot starts from -(128 + z) * sum(x), takes the
// group's products and joins acc times the scale.
template <int G, int RT, int TT, int WR, bool ZP>
__global__ void __launch_bounds__(kIntThreads, TT > 1 ? 2 : 4) k_int4_mm(Int4Params P) {
    constexpr int WK = kIntWaves / WR, TOK = 16 * TT, GC = 128 / G, kNR = 16 * RT * WR;
    using Lds = Int4Lds<G, RT, TT, ZP>;
    constexpr int XU = Lds::kUnits, MI = Lds::kMetas;
    extern __shared__ __align__(16) uint8_t smem[];
    float* sums = reinterpret_cast<float*>(smem + Lds::kX);      // [group of the slab][stok]

    int e = 0, p0, cnt, tile;
    if (P.offsets) {
        const Piece f = find_piece<false>(P.offsets, P.E, P.M, TOK, P.ntn, blockIdx.x);
        if (f.e < 0) return;
        e = f.e;
        tile = f.idx % P.ntn;
        p0 = f.lo + f.idx / P.ntn * TOK;
        cnt = min(f.lo + f.n - p0, TOK);
    } else {
        const int t = xcd_tile(blockIdx.x, (P.M + TOK - 1) / TOK * P.ntn);
        if (t < 0) return;
        tile = t % P.ntn;
        p0 = t / P.ntn * TOK;
        cnt = min(P.M - p0, TOK);
    }
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave / WK, wk = wave % WK;
    const int lrow = lane & 15, q = lane >> 4;
    const int n0 = tile * kNR + wr * 16 * RT;
    const int chunks = P.K / 128, groups = P.K / G;

    // x: XU units a thread per slab; rows to a power of two
    const int cap = TT > 1 ? TOK : cnt <= 2 ? 2 : cnt <= 4 ? 4 : cnt <= 8 ? 8 : 16;
    const int ushift = 31 - __builtin_clz(XU * kIntThreads / cap);           // units of a row: 2^ushift
    const int slab = 8 << ushift, stride = slab * 2 + 16;
    const int stok = cap < 4 ? 4 : cap;
    const uint16_t* xbase = P.slots ? P.x : P.x + (int64_t)p0 * P.K;
    uint32_t xoff[XU];                                           // gathered rows of x end below 2^32 bytes
    uint32_t xreal = 0;
    const auto unit = [&](int j) { return (tid + j * kIntThreads) & ((1 << ushift) - 1); };
#pragma unroll
    for (int j = 0; j < XU; ++j) {
        const int r = min((tid + j * kIntThreads) >> ushift, cnt - 1);
        int src = r;
        bool ok = true;
        if (P.slots) {
            const int slot = P.slots[p0 + r];
            src = slot_token(slot, P.k, P.kmagic);
            ok = slot >= 0 && src < P.X;
        }
        xoff[j] = (uint32_t)(ok ? src : 0) * (uint32_t)P.K;
        xreal |= (uint32_t)ok << j;
    }
    uint4 xv[XU];
    const auto load_x = [&](int k0) {
#pragma unroll
        for (int j = 0; j < XU; ++j)                             // past the end of K: some column, not stored
            xv[j] = *reinterpret_cast<const uint4*>(xbase + xoff[j] + (k0 + unit(j) * 8 < P.K ? k0 + unit(j) * 8 : 0));
    };
    const auto store_x = [&](int k0) {
#pragma unroll
        for (int j = 0; j < XU; ++j) {
            const int r = (tid + j * kIntThreads) >> ushift, u = unit(j);
            const uint4 v = (xreal >> j) & 1 ? xv[j] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = dot2_bf16(w[i], 0x3F803F80u, sum);
            // over the G / 8 lanes of a group (K and a row's units are multiples of 16)
            sum += dpp_f32<0xB1>(0.0f, sum);                            // lanes 1 apart
            sum += dpp_f32<0x4E>(0.0f, sum);                            // 2 apart
            if constexpr (G >= 64) sum += dpp_f32<0x141>(0.0f, sum);    // mirrored in 8
            if constexpr (G >= 128) sum += dpp_f32<0x140>(0.0f, sum);   // mirrored in 16
            if (r < cnt && k0 + u * 8 < P.K) {
                *reinterpret_cast<uint4*>(smem + r * stride + u * 16) = order_x(v);
                if (u % (G / 8) == 0) sums[u / (G / 8) * stok + r] = ZP ? sum : -136.0f * sum;
            }
        }
    };
    load_x(0);

    // weights: chunk i of the wave is chunk wk + i * WK of K
    uint8_t* ring = smem + Lds::kX + Lds::kSums + wave * Lds::kWave1;
    const uint32_t ring0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)ring;
    const uint8_t* wbase[RT];
    int64_t moff[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t row = (int64_t)e * P.N + min(n0 + r * 16 + lrow, P.N - 1);
        wbase[r] = P.codes + row * (P.K / 2) + q * 16;
        moff[r] = row * groups;
    }
    const int mine = max((chunks - wk + WK - 1) / WK, 0), pairs = (mine + 1) / 2;      // the wave's chunks
    // words of lane rows 0 .. 3: group 32: the two of a chunk's scales, then
    // those of the pair's second chunk (zero points: in words of their own);
    // else the pair's scales, then its zero points.  Aligned down to a word.
    const auto issue_meta = [&](int pair) {
        const uint32_t slot = ring0 + Lds::kCodes + (pair & (kRing / 2 - 1)) * (RT * MI * kMeta);
        const auto group = [&](int r, int h) { return moff[r] + (int64_t)(wk + min(2 * pair + h, mine - 1) * WK) * GC; };
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const uint8_t* at = reinterpret_cast<const uint8_t*>(P.scales);
            if constexpr (G == 32) at += group(r, q >> 1) * 2 + (q & 1) * 4;
            else if (ZP && q >= 2) at = P.zeros + (group(r, q & 1) & ~3ll);
            else at += group(r, q & 1) * 2 & ~3ll;
            lds_dma4(at, (lds_void*)(uintptr_t)(slot + r * MI * kMeta));
            if constexpr (MI == 2) lds_dma4(P.zeros + group(r, q & 1), (lds_void*)(uintptr_t)(slot + r * MI * kMeta + kMeta));
        }
    };
    // chunk i; the second of a pair brings the pair's words
    const auto issue = [&](int i) {
        if (i & 1) issue_meta(i >> 1);
        if (i < mine) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
                lds_dma16(wbase[r] + (int64_t)(wk + i * WK) * 64,
                          (lds_void*)(uintptr_t)(ring0 + ((i & (kRing - 1)) * RT + r) * kSlot));
        }
    };
    int done = 0;
#pragma unroll 1
    for (int i = 0; i < min(2 * pairs, kRing); ++i) issue(i);

    const Codes128 decode;
    const floatx4 zero4 = {0, 0, 0, 0};
    floatx4 acc[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = zero4;
    int xrow[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) xrow[t] = min(t * 16 + lrow, cnt - 1) * stride;

#pragma unroll 1
    for (int k0 = 0; k0 < P.K; k0 += slab) {
        const int first = k0 / 128, last = min(chunks, first + slab / 128) - 1;
        if (k0) wait_lds_barrier();                              // the slab before is no longer read
        store_x(k0);
        wait_lds_barrier();
        if (k0 + slab < P.K) load_x(k0 + slab);
#pragma unroll 1
        for (int c = first + wk; c <= last; c += WK) {
            // the oldest chunk and its pair's words are in LDS: of what was
            // asked for later, three chunks and one pair's words are left
            if (mine - done >= kRing) wait_vmem_at_most<(kRing - 1 + MI) * RT>();
            else wait_vmem_at_most<0>();
            const uint8_t* slot = ring + (done & (kRing - 1)) * (RT * kSlot);
            const uint32_t* words = reinterpret_cast<const uint32_t*>(
                ring + Lds::kCodes + ((done >> 1) & (kRing / 2 - 1)) * (RT * MI * kMeta)) + lrow;
            const int base = (c - first) * 128, h = done & 1;
            u32x4 w[RT];
            uint32_t sc[RT][GC > 1 ? GC / 2 : 1], zp[RT];
            int odd[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint4 v = *reinterpret_cast<const uint4*>(slot + r * kSlot + lane * 16);
                const uint32_t* meta = words + r * MI * (kMeta / 4);
                sc[r][0] = meta[(GC == 4 ? 2 * h : h) * 16];
                if constexpr (GC == 4) sc[r][1] = meta[(2 * h + 1) * 16];
                if constexpr (ZP) zp[r] = meta[GC == 4 ? 64 + h * 16 : 32 + h * 16];
                odd[r] = GC == 4 ? 0 : (int)(moff[r] + c * GC) & 3;     // the first group inside its words
                // with one group a chunk the order of K inside it is free:
                // lane row q then takes codes 32 q .. + 31 as loaded
                w[r] = G == 128 ? u32x4{v.x, v.y, v.z, v.w} : transpose4(u32x4{v.x, v.y, v.z, v.w});
            }
            floatx4 dot[RT][TT];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                constexpr int kSteps = G / 32;                   // k-steps of a group
                // the steps' loads together do not fit the registers (4096 rows,
                // 5120 x 5120, zero points: 648 us, 530 so)
                if (G == 32 && RT * TT == 8 && ks) __builtin_amdgcn_sched_barrier(0);
                const int g = ks / kSteps, kb = (base + (G == 128 ? q * 32 + ks * 8 : ks * 32 + q * 8)) * 2;
                bf16x8 wf[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) wf[r] = decode.word(w[r][ks]);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const bf16x8 xf = *reinterpret_cast<const bf16x8*>(smem + xrow[t] + kb);
                    floatx4 init = zero4;
                    if (ks % kSteps == 0)
                        init = *reinterpret_cast<const floatx4*>(sums + (base / G + g) * stok + t * 16 + q * 4);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        if (ks % kSteps == 0) {
                            dot[r][t] = init;
                            if constexpr (ZP) {
                                const float off = -128.0f - (float)((zp[r] >> (8 * (odd[r] + g))) & 0xFFu);
#pragma unroll
                                for (int j = 0; j < 4; ++j) dot[r][t][j] *= off;
                            }
                        }
                        dot[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, wf[r], dot[r][t], 0, 0, 0);
                        if ((ks + 1) % kSteps == 0) {
                            // G == 128: the scale is the word's low or high half
                            const uint32_t word = sc[r][g / 2];
                            const bool high = GC == 1 ? odd[r] & 1 : g & 1;
                            const float s = __uint_as_float(high ? word & 0xFFFF0000u : word << 16);
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[r][t][j] = fmaf(s, dot[r][t][j], acc[r][t][j]);
                        }
                    }
                }
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);                  // lgkmcnt 0: the slot has been read
            if (done + kRing < 2 * pairs) issue(done + kRing);
            ++done;
        }
    }
    wait_vmem_at_most<0>();                                      // nothing more lands in the rings
    wait_lds_barrier();

    // join the K parts: [wr][r][t][wk][lane]
    floatx4* part = reinterpret_cast<floatx4*>(smem);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) part[(((wr * RT + r) * TT + t) * WK + wk) * kWave + lane] = acc[r][t];
    wait_lds_barrier();
    for (int i = tid; i < WR * RT * TT * kWave; i += kIntThreads) {
        const int l = i & 63, b = i >> 6;                        // b = (wr * RT + r) * TT + t
        floatx4 v = zero4;
#pragma unroll
        for (int j = 0; j < WK; ++j) v += part[(b * WK + j) * kWave + l];
        const int n = tile * kNR + b / TT * 16 + (l & 15), r = b % TT * 16 + (l >> 4) * 4;
        if (n >= P.N) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r + j < cnt) P.out[(int64_t)(p0 + r + j) * P.N + n] = f32_to_bf16_rne(v[j]);
    }
}

// ---- a dense projection of one or two rows: vector dot products, no LDS but
// for the join.  Half a wave reads 1024 columns of one weight row, 16 bytes
// (32 codes of one group) a lane, the wave eight rows in four such loads, all
// in flight at once beside x's 32 values, which stay in registers in the order
// of the decoded codes.  The waves of a workgroup take the blocks of 1024
// columns.  Less of a wait before the first product than k_int4_mm (one row,
// 5120 x 5120: 6.4 us against 9.3; four rows: 14.6 against 11.0), and few
// rows, because unrolled code is fetched as slowly as weights (16 rows: 14.6 us).
constexpr int kVecRows = 8;       // weight rows of a workgroup
constexpr int kVecWaves = 8;

template <int T, bool ZP>
__global__ void __launch_bounds__(kVecWaves * kWave, 4) k_int4_vec(Int4Params P, int G) {
    __shared__ float part[kVecWaves * kVecRows * T];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, waves = blockDim.x >> 6, n0 = blockIdx.x * kVecRows;
    const int gshift = __builtin_ctz(G), groups = P.K >> gshift;
    const Codes128 decode;
    float acc[kVecRows / 2][T];
#pragma unroll
    for (int r = 0; r < kVecRows / 2; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[r][t] = 0.0f;
    for (int k0 = wave * 1024; k0 < P.K; k0 += waves * 1024) {
        // every load is unconditional (a lane past the end of K reads column
        // 0 and drops it), so that none waits behind a branch
        const int col = k0 + (lane & 31) * 32;
        const bool in = col < P.K;
        const int c = in ? col : 0, g = c >> gshift;
        uint4 xv[T][4], codes[kVecRows / 2];
        uint32_t sc[kVecRows / 2], zp[kVecRows / 2];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) xv[t][i] = *reinterpret_cast<const uint4*>(P.x + (int64_t)t * P.K + c + i * 8);
#pragma unroll
        for (int r = 0; r < kVecRows / 2; ++r) {
            const int64_t row = min(n0 + 2 * r + half, P.N - 1);
            codes[r] = load_stream16(reinterpret_cast<const uint4*>(P.codes + row * (P.K / 2) + c / 2));
            sc[r] = P.scales[row * groups + g];
            zp[r] = 8u;
            if constexpr (ZP) zp[r] = P.zeros[row * groups + g];
        }
        float sum[T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            sum[t] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xv[t][i] = in ? order_x(xv[t][i]) : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {xv[t][i].x, xv[t][i].y, xv[t][i].z, xv[t][i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[t] = dot2_bf16(w[j], 0x3F803F80u, sum[t]);
            }
        }
#pragma unroll
        for (int r = 0; r < kVecRows / 2; ++r) {
            const float s = in ? bf16_bits_to_f32(sc[r]) : 0.0f, off = -128.0f - (float)zp[r];
            const uint32_t cw[4] = {codes[r].x, codes[r].y, codes[r].z, codes[r].w};
            float dot[T];
#pragma unroll
            for (int t = 0; t < T; ++t) dot[t] = off * sum[t];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t pair = decode.pair(cw[i], j);
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        const uint32_t xw = j == 0 ? xv[t][i].x : j == 1 ? xv[t][i].y : j == 2 ? xv[t][i].z : xv[t][i].w;
                        dot[t] = dot2_bf16(pair, xw, dot[t]);
                    }
                }
#pragma unroll
            for (int t = 0; t < T; ++t) acc[r][t] = fmaf(s, dot[t], acc[r][t]);
        }
    }
    // lane 31: the first row of each pair, lane 63: the second
#pragma unroll
    for (int r = 0; r < kVecRows / 2; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float v = row_prefix_sum(acc[r][t]);
            v += dpp_f32<kDppRowBcast15, 0xA>(0.0f, v);
            if ((lane & 31) == 31) part[(wave * kVecRows + 2 * r + half) * T + t] = v;
        }
    wait_lds_barrier();
    const int i = threadIdx.x;
    if (i < kVecRows * T) {
        float v = 0.0f;
        for (int w = 0; w < waves; ++w) v += part[w * kVecRows * T + i];
        const int n = n0 + i / T, t = i % T;
        if (n < P.N) P.out[(int64_t)t * P.N + n] = f32_to_bf16_rne(v);
    }
}

template <int T>
moe_status launch_int4_vec(const Int4Params& P, int G, hipStream_t s) {
    const dim3 grid((P.N + kVecRows - 1) / kVecRows), block(std::min((P.K + 1023) / 1024, kVecWaves) * kWave);
    if (P.zeros) MOE_LAUNCH("int4_linear", (k_int4_vec<T, true>), grid, block, 0, s, P, G);
    else MOE_LAUNCH("int4_linear", (k_int4_vec<T, false>), grid, block, 0, s, P, G);
    return MOE_OK;
}

template <int G, int RT, int TT, int WR, bool ZP>
moe_status launch_int4_z(Int4Params P, hipStream_t s) {
    constexpr int NR = 16 * RT * WR, TOK = 16 * TT;
    P.ntn = (P.N + NR - 1) / NR;
    const int64_t blocks = P.offsets ? P.M / TOK + (int64_t)std::min(P.E, P.M) : (P.M + TOK - 1) / TOK;
    if (blocks * P.ntn >= (1 << 22)) return MOE_ERR_SHAPE;
    const size_t lds = Int4Lds<G, RT, TT, ZP>::kBytes;
    moe_status st = allow_dynamic_lds(reinterpret_cast<const void*>(&k_int4_mm<G, RT, TT, WR, ZP>), lds);
    if (st != MOE_OK) return st;
    MOE_LAUNCH("int4_linear", (k_int4_mm<G, RT, TT, WR, ZP>), dim3((unsigned)xcd_grid(blocks * P.ntn)),
               dim3(kIntThreads), lds, s, P);
    return MOE_OK;
}
template <int G, int RT, int TT, int WR>
moe_status launch_int4(const Int4Params& P, hipStream_t s) {
    return P.zeros ? launch_int4_z<G, RT, TT, WR, true>(P, s) : launch_int4_z<G, RT, TT, WR, false>(P, s);
}

// The tile.  A workgroup reads all of its rows of x for 16 RT WR weight rows,
// so a wide tile saves cache traffic, and one that leaves CUs empty costs more
// than it saves.  The widest that fills most of the CUs is taken.  Bounds where
// the two sides were measured (us; group 128 with zero points; "experts": 64):
//   64 rows against 32: a tile costs 5/3 (experts of 75 rows, 1536 x 5120: 251
//     against 238, of 256 rows: 480 against 606).  Its LDS leaves one to a CU:
//     320 of them take two turns (1024 rows, 5120 x 5120: 132 against 120).
//   32 rows against 16 (5120 x 1536): experts of 12 rows 79 against 73, of 20
//     rows 86 against 114.
//   WR 8 against 4, half the waves along K (8 rows of x, top 8): 8192 x 768 45
//     against 68, 4096 x 2048 49 against 60, 2048 x 4096 50 against 52 (group 32
//     56 against 54), 1536 x 5120 44 against 41.
//   too few: 16 rows, 160 of WR 2 13.2 against 320 of WR 1 15.6 (5120 x 5120);
//     128 of WR 2 31 against 256 of WR 1 26 (4096 x 14336).
template <int G>
moe_status launch_int4_group(const Int4Params& P, hipStream_t s) {
    if (!P.offsets && P.M == 1) return launch_int4_vec<1>(P, G, s);
    if (!P.offsets && P.M == 2) return launch_int4_vec<2>(P, G, s);
    const int64_t experts = P.offsets ? std::max<int64_t>(std::min(P.E, P.M), 1) : 1, rows = P.M / experts;
    const auto tiles = [&](int64_t tok, int64_t nr) {            // 0: half of the tile's weight rows do not exist
        return 2 * (int64_t)P.N > nr ? experts * ((rows + tok - 1) / tok) * ((P.N + nr - 1) / nr) : 0;
    };
    if (5 * ((rows + 63) / 64) < 3 * ((rows + 31) / 32)) {
        const int64_t t = tiles(64, 256), turns = (t + 255) / 256;
        if (t >= 192 && 10 * t >= 7 * 256 * turns) return launch_int4<G, 2, 4, 8>(P, s);
    }
    if (rows > (P.offsets ? 12 : 16)) {
        if (tiles(32, 128) >= 192) return launch_int4<G, 1, 2, 8>(P, s);
        if (tiles(32, 64) >= 192) return launch_int4<G, 1, 2, 4>(P, s);
    }
    if (P.K < 4096 && tiles(16, 128) >= 160) return launch_int4<G, 1, 1, 8>(P, s);
    if (tiles(16, 64) >= 160) return launch_int4<G, 1, 1, 4>(P, s);
    if (tiles(16, 32) >= 160) return launch_int4<G, 1, 1, 2>(P, s);
    return launch_int4<G, 1, 1, 1>(P, s);
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
    Int4Params P{};
    P.x = x;
    P.codes = t->codes; P.scales = t->scales; P.zeros = t->zeros;
    P.offsets = offsets;
    P.slots = slots;
    P.E = t->E; P.M = M; P.X = X; P.k = k; P.N = t->N; P.K = t->K;
    P.kmagic = div_magic(k);
    P.out = out;
    return t->group == 32 ? launch_int4_group<32>(P, s) : t->group == 64 ? launch_int4_group<64>(P, s) : launch_int4_group<128>(P, s);
}

}  // namespace moe
