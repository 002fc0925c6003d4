// Matrix products of bf16 expert weights over expert-sorted rows: the product,
// the gate/up pair with SwiGLU, the input gradients and the weight gradient.
//
// With rows p of expert e = the e-th run of d_offsets, all sums in fp32 on
// v_mfma_f32_16x16x32_bf16:
//   k_rows_mm<kNT>      y[p][n]  = sum_k x[src(p)][k] W[e][n][k]
//   k_rows_mm<kGateUp>  the same with gate and up, h = silu(a) b
//   k_rows_mm<kNN>      dx[p][k] = sum_n dy[p][n] W[e][n][k]   (and a second pair)
//   k_wgrad             dW[e][n][k] = sum_{p in e} dy[p][n] x[src(p)][k]
//
// An operand's tile of one stage (64 steps of the reduction) goes from memory
// straight to LDS (buffer loads with the LDS as destination: 16 bytes a lane,
// lanes outside the matrix get an offset past the descriptor and read zeros).
// Two layouts, by how the operand lies in memory:
//   reduction contiguous ("RC"): LDS rows of 64 values (128 bytes); 16-byte
//     unit u of row r sits at unit u ^ (r >> 1 & 7), so the 16 rows of a
//     fragment read hit 16 different 16-byte bank groups;
//   reduction outermost ("RO"): LDS rows of 256 output positions (512 bytes),
//     read through the LDS transpose load (4 x 16 blocks); 32-byte chunk c of
//     row r sits at chunk c ^ (r & 3 | r >> 1 & 4), so the eight rows that
//     half a wave reads hit eight different 32-byte bank groups.
// Counters show no bank conflict for either.  The output position that is
// contiguous in memory is the A operand of the MFMA: a lane then holds four
// neighbouring outputs of one row.
//
// What bounds it.  Tiles of 256 x 256 on eight waves read 12 fragments (12 KB)
// from LDS per 32 MFMAs and wave, 96 of the 128 bytes a clock that LDS gives,
// and 64 KB from L2 per stage and CU.  8192^3: 1150-1200 TFLOP/s forward,
// 1200-1280 input gradient, 1080-1170 weight gradient, 1300-1400 gate/up,
// against 1340-1400 of the library's product on the same boxes; zeros run
// faster, so the clock under load is part of that.  With about 256 rows an
// expert the weights' stream from HBM (one 32 KB stage a CU per 1.5 us with all
// CUs) and the matrix units (1.2 us) take turns being the limit; with few rows
// it is HBM alone (64 experts, 32 tokens: 6.2 TB/s).
#include "device_common.h"
#include "expert_rows.h"
#include "internal.h"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

constexpr int kThreads = 512;             // 8 waves: 2 along the rows x 4 along the columns
constexpr int kWaves = kThreads / kWave;
constexpr int kBN = 256;                  // output columns per tile, 64 per wave
constexpr int kNI = 4;                    // 16-column subtiles per wave
constexpr int kBK = 64;                   // reduction steps per stage
constexpr uint32_t kOutside = 0xFFFFFFFFu;
constexpr uint32_t kRecords = 0xFFFFFF00u;   // descriptor size: every real offset is below it

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

// x . W^T | x . gate^T and x . up^T | dy . W
enum Form { kNT = 0, kGateUp = 1, kNN = 2 };
// rounded outputs | SwiGLU, or its gradient (kNN) | fp32 sums of one slice of the reduction
enum Epilogue { kPlain = 0, kSwiglu = 1, kPart = 2 };

// 16 bytes per lane from (base + voff) to LDS at ldst + 16 * lane; lanes whose
// voff lies outside the descriptor write zeros.  Inline assembly for the same
// reason as lds_dma16: the compiler would wait for it before every LDS read.
__device__ __forceinline__ void lds_dma16_buf(const void* base, uint32_t voff, uint32_t ldst) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    u32x4 rsrc;
    rsrc[0] = (uint32_t)b;
    rsrc[1] = (uint32_t)(b >> 32) & 0xFFFFu;
    rsrc[2] = kRecords;
    rsrc[3] = 0x00020000u;
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "{m0}"(ldst) : "memory");
}

__device__ __forceinline__ const uint16_t* uniform_ptr(const uint16_t* p) {
    const uint64_t b = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    return reinterpret_cast<const uint16_t*>(((uint64_t)hi << 32) | lo);
}

// The stages of a tile, through rings of NSA and NSB LDS buffers for the two
// operands.  Fragments are read
// one k-step ahead: while the MFMAs of a stage's first half run, its second
// half is read (in place, a fragment as soon as its four MFMAs are issued);
// then every wave has read all of the stage, its buffers take the stages NSA
// and NSB later, and the next stage's first half is read under the second half's
// MFMAs.  OPSA, OPSB: DMAs of a wave per stage, which complete in order.
template <int OPS>
__device__ __forceinline__ void wait_stages_behind(int n) {
    if (n <= 0) wait_vmem_at_most<0>();
    else if (n == 1) wait_vmem_at_most<OPS>();
    else if (n == 2) wait_vmem_at_most<2 * OPS>();
    else wait_vmem_at_most<3 * OPS>();
}

template <int NSA, int NSB, int U, int NI, int OPSA, int OPSB, int READS_A, int READS_B, class DmaA, class DmaB,
          class ReadA, class ReadB, class Acc>
__device__ __forceinline__ void run_stages(int nstages, DmaA&& dma_a, DmaB&& dma_b, ReadA&& ra, ReadB&& rb, Acc& acc) {
    constexpr int OPS = OPSA + OPSB;
    static_assert(NSB == NSA || (NSA == 2 && NSB == 3), "the waits below");
#pragma unroll
    for (int i = 0; i < NSB; ++i) {
        if (i < NSA && i < nstages) dma_a(i);
        if (i < nstages) dma_b(i);
    }
    if constexpr (NSA == NSB) wait_stages_behind<OPS>(min(NSA, nstages) - 1);
    else if (nstages > 2) wait_vmem_at_most<OPS + OPSB>();
    else wait_stages_behind<OPS>(nstages - 1);
    wait_lds_barrier();
    bf16x8 af[U], b0[NI], b1[NI];
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) b0[ni] = rb(0, 0, ni);
#pragma unroll
    for (int mi = 0; mi < U; ++mi) af[mi] = ra(0, 0, mi);
    int bufa = 0, bufb = 0;
    for (int s = 0; s < nstages; ++s) {
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) b1[ni] = rb(bufb, 1, ni);
#pragma unroll
        for (int mi = 0; mi < U; ++mi) {
#pragma unroll
            for (int ni = 0; ni < NI; ++ni)
                acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b0[ni], af[mi], acc[mi][ni], 0, 0, 0);
            af[mi] = ra(bufa, 1, mi);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, NI * READS_B, 0);
#pragma unroll
        for (int mi = 0; mi < U; ++mi) {
            __builtin_amdgcn_sched_group_barrier(0x008, NI, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, READS_A, 0);
        }
        // stage s + 1 is in LDS (stages behind it may be in flight) and nobody reads stage s any more
        if constexpr (NSA != NSB) wait_stages_behind<OPSB>(min(1, nstages - 2 - s));
        else if constexpr (NSA == 2) wait_vmem_at_most<0>();
        else wait_stages_behind<OPS>(min(NSA - 2, nstages - 2 - s));
        wait_lds_barrier();
        if (s + NSA < nstages) dma_a(s + NSA);
        if (s + NSB < nstages) dma_b(s + NSB);
        bufa = bufa + 1 == NSA ? 0 : bufa + 1;
        bufb = bufb + 1 == NSB ? 0 : bufb + 1;
        // behind the last stage this reads a buffer whose values nobody uses
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) b0[ni] = rb(bufb, 0, ni);
#pragma unroll
        for (int mi = 0; mi < U; ++mi) {
#pragma unroll
            for (int ni = 0; ni < NI; ++ni)
                acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b1[ni], af[mi], acc[mi][ni], 0, 0, 0);
            af[mi] = ra(bufa, 0, mi);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, NI * READS_B, 0);
#pragma unroll
        for (int mi = 0; mi < U; ++mi) {
            __builtin_amdgcn_sched_group_barrier(0x008, NI, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, READS_A, 0);
        }
    }
}

// The same with stages of one k-step and one ring of NS buffers (each holds
// both operands): while a stage's MFMAs run, the next one is read.
template <int NS, int U, int NI, int OPS, int READS_A, int READS_B, class Dma, class ReadA, class ReadB, class Acc>
__device__ __forceinline__ void run_steps(int nstages, Dma&& dma, ReadA&& ra, ReadB&& rb, Acc& acc) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (i < nstages) dma(i);
    wait_stages_behind<OPS>(min(NS, nstages) - 1);
    wait_lds_barrier();
    bf16x8 af[U], b0[NI], b1[NI];
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) b0[ni] = rb(0, ni);
#pragma unroll
    for (int mi = 0; mi < U; ++mi) af[mi] = ra(0, mi);
    int buf = 0;
    const auto step = [&](int s, bf16x8 (&now)[NI], bf16x8 (&then)[NI]) {
        wait_stages_behind<OPS>(min(NS - 2, nstages - 2 - s));   // stage s + 1 is in LDS
        wait_lds_barrier();                                      // and stage s has been read
        if (s + NS < nstages) dma(s + NS);
        buf = buf + 1 == NS ? 0 : buf + 1;
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) then[ni] = rb(buf, ni);
#pragma unroll
        for (int mi = 0; mi < U; ++mi) {
#pragma unroll
            for (int ni = 0; ni < NI; ++ni)
                acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now[ni], af[mi], acc[mi][ni], 0, 0, 0);
            af[mi] = ra(buf, mi);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, NI * READS_B, 0);
#pragma unroll
        for (int mi = 0; mi < U; ++mi) {
            __builtin_amdgcn_sched_group_barrier(0x008, NI, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, READS_A, 0);
        }
    };
    for (int s = 0; s < nstages; s += 2) {
        step(s, b0, b1);
        if (s + 1 < nstages) step(s + 1, b1, b0);
    }
}

struct MmParams {
    const uint16_t* a0;           // row operand: x, or dy
    const uint16_t* a1;           // NN: the second pair's dy, or null
    const uint16_t* w0;           // weights (kSwiglu on NT: gate)
    const uint16_t* w1;           // kSwiglu on NT: up; NN: the second pair's weights, or null
    const int32_t* offsets;
    const int32_t* slots;         // NT: sorted slots, or null (row p is x's row p)
    int E, M, X, k;
    uint32_t kmagic;
    int R, C;                     // reduction length, output columns
    int pairs;
    uint16_t *o0, *o1, *o2;       // y | h, a, b | dx | da, db
    const uint16_t *i0, *i1;      // kSwiglu on NN: the saved a, b
    int ntc;                      // column tiles
    int slices;                   // kPart: the reduction's slices
    float* part;                  // kPart: [slices][1, gate/up: 2][M][C]
};

constexpr int kMGroup = 8;        // row tiles that run beside each other, sharing weight columns in L2

struct RowTile {
    int e, p0, rows, ct;          // expert (-1: none), first row, rows of the tile, column tile
    int slice;
};

// Tile of workgroup `bid`: inside an expert, kMGroup row tiles by all column
// tiles after each other, each with its slices of the reduction.
template <int BM, bool SLICED>
__device__ __forceinline__ RowTile find_tile(const MmParams& P, int bid) {
    const Piece f = find_piece<false, BM * 5 / 8>(P.offsets, P.E, P.M, BM, SLICED ? P.ntc * P.slices : P.ntc, bid);
    if (f.e < 0) return RowTile{-1, 0, 0, 0, 0};
    const int idx = SLICED ? f.idx / P.slices : f.idx, slice = SLICED ? f.idx % P.slices : 0;
    const int full = f.pieces / kMGroup * kMGroup;
    int m, c;
    if (idx < full * P.ntc) {
        const int g = idx / (kMGroup * P.ntc), r = idx % (kMGroup * P.ntc);
        c = r / kMGroup;
        m = g * kMGroup + r % kMGroup;
    } else {
        const int r = idx - full * P.ntc, last = f.pieces - full;
        c = r / last;
        m = full + r % last;
    }
    // equal heights, whole subtiles: tiles that share weight columns then move
    // through them in step and find each other's stages in L2
    const int h = ((f.n + f.pieces - 1) / f.pieces + 15) & ~15;
    return RowTile{f.e, f.lo + m * h, min(h, f.n - m * h), c, slice};
}

// ---- fragments: lane l holds output position l & 15, reduction steps
// 8 (l >> 4) .. + 7 of the k-step
__device__ __forceinline__ bf16x8 frag_rc(const lds_u8* tile, int lane_off, int sub) {
    return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8*>(tile + lane_off + sub * (16 * kBK * 2));
}
// LDS unit (16 bytes) of unit u of row r: u ^ rc_swizzle(r)
__device__ __forceinline__ int rc_swizzle(int r) { return (r >> 1) & 7; }
template <int ROW>                          // bytes of an LDS row
__device__ __forceinline__ bf16x8 frag_ro(const lds_u8* tile, int lane_off) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(tile + lane_off));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(tile + lane_off + 4 * ROW));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ int ro_swizzle(int row) { return (row & 3) | ((row >> 1) & 4); }

// Two floats to a bf16 pair, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_rne(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2){lo, hi}, bf16x2));
}
// sigmoid with the reciprocal and exponential instructions (a few 2^-23 relative)
__device__ __forceinline__ float sigmoid(float a) { return __builtin_amdgcn_rcpf(1.0f + __expf(-a)); }

// dh through silu(a) b: da = dh b s (1 + a (1 - s)), db = dh a s, s = sigmoid(a)
__device__ __forceinline__ void swiglu_grad(float dh, float a, float b, float& da, float& db) {
    const float s = sigmoid(a), act = a * s;
    db = dh * act;
    da = dh * b * (s + act * (1.0f - s));
}

// A lane's four columns of two neighbouring 16-column subtiles <-> eight
// columns of one of them: lane rows (16 lanes) 0 and 1 trade halves, and 2 and
// 3.  Afterwards lane row q holds columns 8 (q >> 1) .. + 7 of subtile q & 1,
// 16 bytes of bf16.  The exchange undoes itself.
struct Pair4 {
    uint32_t a0, a1, b0, b1;      // subtile a: columns 0, 1 | 2, 3; subtile b the same
};
__device__ __forceinline__ uint4 exchange(Pair4 v) {
    const auto x = __builtin_amdgcn_permlane16_swap(v.a0, v.b0, false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(v.a1, v.b1, false, false);
    return make_uint4(x[0], y[0], x[1], y[1]);
}
__device__ __forceinline__ Pair4 exchange_back(uint4 v) {
    const auto x = __builtin_amdgcn_permlane16_swap(v.x, v.z, false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(v.y, v.w, false, false);
    return Pair4{x[0], y[0], x[1], y[1]};
}
__device__ __forceinline__ uint4 pack_pair(floatx4 a, floatx4 b) {
    return exchange(Pair4{pack_rne(a[0], a[1]), pack_rne(a[2], a[3]), pack_rne(b[0], b[1]), pack_rne(b[2], b[3])});
}
__device__ __forceinline__ floatx4 widen4(uint32_t lo, uint32_t hi) {
    return floatx4{bf16_bits_to_f32(lo & 0xFFFFu), __uint_as_float(lo & 0xFFFF0000u), bf16_bits_to_f32(hi & 0xFFFFu),
                   __uint_as_float(hi & 0xFFFF0000u)};
}

constexpr int rows_lds(int BM, int NSA, int NSB) { return (NSA * BM + NSB * kBN) * kBK * 2; }

// One tile of up to BM rows by 256 columns on eight waves, two along the rows
// by four along the columns: U 16-row subtiles a wave.  The two waves of a
// SIMD take the tile's subtiles in turn, so a short tile costs both the same.
template <int FORM, int EPI, int BM, int U, int NSA, int NSB>
__device__ __forceinline__ void rows_tile(const MmParams& P, const RowTile& t, uint8_t* smem) {
    constexpr int kRowBytes = BM * kBK * 2, kColStage = kBN * kBK * 2, kColRing = NSA * kRowBytes;
    constexpr int kADma = kRowBytes / 1024 / kWaves, kBDma = kColStage / 1024 / kWaves;
    constexpr int kDmaRows = 512 / kBK, kUnits = kBK / 8;       // rows of a DMA, 16-byte units of a row (RC)
    constexpr bool RC = FORM != kNN, GU = FORM == kGateUp;    // GU: 128 gate + 128 up columns per tile
    constexpr int kTileCols = GU ? kBN / 2 : kBN;             // output columns per tile
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int lrow = lane & 15, q = lane >> 4;
    const int c0 = t.ct * kTileCols;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8*)smem;

    // row operand: per-lane byte offset of its rows (one per DMA); all slots are
    // asked for at once
    uint32_t aoff[kADma];
    int aunit[kADma], slot[kADma];
    const int64_t abase = P.slots ? 0 : (int64_t)t.p0 * P.R;
    const auto row = [&](int i) { return (i * kWaves + wave) * kDmaRows + lane / kUnits; };
    if (P.slots) {
#pragma unroll
        for (int i = 0; i < kADma; ++i) slot[i] = P.slots[t.p0 + min(row(i), t.rows - 1)];
    }
#pragma unroll
    for (int i = 0; i < kADma; ++i) {
        const int r = row(i);
        aunit[i] = (lane % kUnits) ^ rc_swizzle(r);
        int src = r;
        bool ok = r < t.rows;
        if (P.slots) {
            src = slot_token(slot[i], P.k, P.kmagic);
            ok = ok && slot[i] >= 0 && src < P.X;
        }
        aoff[i] = ok ? (uint32_t)src * (uint32_t)P.R * 2u + aunit[i] * 16 : kOutside;
    }
    // column operand
    uint32_t boff[kBDma];
    int bpos[kBDma];                                // RC: unit; RO: reduction row inside the stage
    const int64_t wbase = RC ? ((int64_t)t.e * P.C + c0) * P.R : (int64_t)t.e * P.R * P.C + c0;
#pragma unroll
    for (int i = 0; i < kBDma; ++i) {
        if constexpr (RC) {
            const int r = (i * kWaves + wave) * kDmaRows + lane / kUnits;
            const int n = GU ? r & (kBN / 2 - 1) : r;
            bpos[i] = (lane % kUnits) ^ rc_swizzle(r);
            boff[i] = c0 + n < P.C ? (uint32_t)n * (uint32_t)P.R * 2u + bpos[i] * 16 : kOutside;
        } else {
            const int r = (i * kWaves + wave) * 2 + (lane >> 5);
            const int pos = lane & 31, col = (((pos >> 1) ^ ro_swizzle(r)) << 4) + ((pos & 1) << 3);
            bpos[i] = r;
            boff[i] = c0 + col < P.C ? (uint32_t)r * (uint32_t)P.C * 2u + col * 2 : kOutside;
        }
    }

    const int spp = (P.R + kBK - 1) / kBK;            // stages per pair
    const int all = spp * P.pairs;
    const int first = EPI == kPart ? (int)((int64_t)all * t.slice / P.slices) : 0;
    const int nstages = (EPI == kPart ? (int)((int64_t)all * (t.slice + 1) / P.slices) : all) - first;
    const auto dma_a = [&](int s) {
        const int pair = FORM == kNN && first + s >= spp ? 1 : 0;
        const int r0 = (first + s - pair * spp) * kBK;
        const uint16_t* a = uniform_ptr((pair ? P.a1 : P.a0) + abase + r0);
        const uint32_t buf = lds0 + (s % NSA) * kRowBytes;
#pragma unroll
        for (int i = 0; i < kADma; ++i) {
            const uint32_t vo = r0 + aunit[i] * 8 < P.R ? aoff[i] : kOutside;
            lds_dma16_buf(a, vo, buf + (i * kWaves + wave) * 1024);
        }
    };
    const auto dma_b = [&](int s) {
        const int pair = FORM == kNN && first + s >= spp ? 1 : 0;
        const int r0 = (first + s - pair * spp) * kBK;
        const uint32_t buf = lds0 + kColRing + (s % NSB) * kColStage;
#pragma unroll
        for (int i = 0; i < kBDma; ++i) {
            const bool up = GU && i >= kBDma / 2;
            const uint16_t* w = uniform_ptr((pair || up ? P.w1 : P.w0) + wbase + (RC ? (int64_t)r0 : (int64_t)r0 * P.C));
            const bool ok = RC ? r0 + bpos[i] * 8 < P.R : r0 + bpos[i] < P.R;
            lds_dma16_buf(w, ok ? boff[i] : kOutside, buf + (i * kWaves + wave) * 1024);
        }
    };

    // lane offsets of the fragments
    int aread[kBK / 32], bread[kBK / 32], bchunk[kNI];
#pragma unroll
    for (int ks = 0; ks < kBK / 32; ++ks) {
        const int u = ((ks * 4 + q) ^ rc_swizzle(lrow)) * 16;
        aread[ks] = (wm * 16 + lrow) * kBK * 2 + u;
        if constexpr (RC)
            bread[ks] = ((GU ? wn * 32 : wn * 64) + lrow) * kBK * 2 + u;
        else
            bread[ks] = (ks * 32 + q * 8 + (lrow >> 2)) * 512 + (lrow & 3) * 8;
    }
    const int bsw = (lrow >> 2) | ((q & 1) << 2);   // ro_swizzle of the lane's rows
#pragma unroll
    for (int ni = 0; ni < kNI; ++ni) bchunk[ni] = ((wn * 4 + ni) ^ bsw) * 32;

    floatx4 acc[U][kNI];
#pragma unroll
    for (int mi = 0; mi < U; ++mi)
#pragma unroll
        for (int ni = 0; ni < kNI; ++ni) acc[mi][ni] = floatx4{0, 0, 0, 0};
    const auto read_a = [&](int buf, int ks, int mi) {
        return frag_rc((const lds_u8*)smem + buf * kRowBytes, aread[ks], 2 * mi);
    };
    const auto read_b = [&](int buf, int ks, int ni) {
        const lds_u8* bs = (const lds_u8*)smem + kColRing + buf * kColStage;
        if constexpr (RC) return frag_rc(bs, bread[ks], GU && ni >= 2 ? ni + 6 : ni);
        else return frag_ro<512>(bs, bread[ks] + bchunk[ni]);
    };
    constexpr int kReadsB = RC ? 1 : 2;
    run_stages<NSA, NSB, U, kNI, kADma, kBDma, 1, kReadsB>(nstages, dma_a, dma_b, read_a, read_b, acc);

    if constexpr (EPI == kPart) {
#pragma unroll
        for (int mi = 0; mi < U; ++mi) {
            const int r = (mi * 2 + wm) * 16 + lrow;
            if (r >= t.rows) continue;
#pragma unroll
            for (int ni = 0; ni < kNI; ++ni) {
                const int up = GU && ni >= 2 ? 1 : 0, c = c0 + (GU ? wn * 32 + ni % 2 * 16 : wn * 64 + ni * 16) + q * 4;
                if (c >= P.C) continue;
                const int64_t at = ((int64_t)(t.slice * (GU ? 2 : 1) + up) * P.M + t.p0 + r) * P.C + c;
                *reinterpret_cast<floatx4*>(P.part + at) = acc[mi][ni];
            }
        }
        return;
    }
    // One rounding to bf16 per output; a lane stores eight columns of one row.
    // Every lane takes part in the exchanges, also those that store nothing.
    constexpr int kPairs = GU ? 1 : 2;
    // The saved a and b: those of kAhead subtiles requested at once, in the
    // registers that the fragments leave (one at a time, each behind the
    // stores before it, 640 tiles of one stage took 112 us against 100).
    constexpr bool kGrad = FORM == kNN && EPI == kSwiglu;
    constexpr int kAhead = U > 8 ? 3 : 4;
    uint4 asave[kGrad ? kAhead : 1][kPairs], bsave[kGrad ? kAhead : 1][kPairs];
#pragma unroll
    for (int mi = 0; mi < U; ++mi) {
        const int r = (mi * 2 + wm) * 16 + lrow;
        if constexpr (kGrad) {
            if (mi % kAhead == 0)
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) {
                        // lanes outside read the tile's last row or columns, so
                        // that no load waits behind a branch
                        const int ra = min(((mi + i) * 2 + wm) * 16 + lrow, t.rows - 1);
                        const int ca = min(c0 + wn * 64 + j * 32 + (q & 1) * 16 + (q >> 1) * 8, P.C - 8);
                        const int64_t at = (int64_t)(t.p0 + ra) * P.C + ca;
                        asave[i][j] = *reinterpret_cast<const uint4*>(P.i0 + at);
                        bsave[i][j] = *reinterpret_cast<const uint4*>(P.i1 + at);
                    }
        }
        const int64_t row = (int64_t)(t.p0 + r) * P.C;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const int c = c0 + (GU ? wn * 32 : wn * 64 + j * 32) + (q & 1) * 16 + (q >> 1) * 8;
            const bool ok = r < t.rows && c < P.C;
            if constexpr (GU) {
                floatx4 h[2];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[n][i] = acc[mi][n][i] * sigmoid(acc[mi][n][i]) * acc[mi][n + 2][i];
                const uint4 hv = pack_pair(h[0], h[1]);
                if (ok) *reinterpret_cast<uint4*>(P.o0 + row + c) = hv;
                if (P.o1) {
                    const uint4 av = pack_pair(acc[mi][0], acc[mi][1]), bv = pack_pair(acc[mi][2], acc[mi][3]);
                    if (ok) {
                        *reinterpret_cast<uint4*>(P.o1 + row + c) = av;
                        *reinterpret_cast<uint4*>(P.o2 + row + c) = bv;
                    }
                }
            } else if constexpr (EPI == kSwiglu) {
                const Pair4 ap = exchange_back(asave[mi % kAhead][j]), bp = exchange_back(bsave[mi % kAhead][j]);
                const floatx4 a[2] = {widen4(ap.a0, ap.a1), widen4(ap.b0, ap.b1)};
                const floatx4 b[2] = {widen4(bp.a0, bp.a1), widen4(bp.b0, bp.b1)};
                floatx4 da[2], db[2];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x, y;                              // (elements of a vector bind to no reference)
                        swiglu_grad(acc[mi][2 * j + n][i], a[n][i], b[n][i], x, y);
                        da[n][i] = x;
                        db[n][i] = y;
                    }
                const uint4 av = pack_pair(da[0], da[1]), bv = pack_pair(db[0], db[1]);
                if (ok) {
                    *reinterpret_cast<uint4*>(P.o0 + row + c) = av;
                    *reinterpret_cast<uint4*>(P.o1 + row + c) = bv;
                }
            } else {
                const uint4 v = pack_pair(acc[mi][2 * j], acc[mi][2 * j + 1]);
                if (ok) *reinterpret_cast<uint4*>(P.o0 + row + c) = v;
            }
        }
    }
}

// Tiles of up to BM rows, by their rows: a short tile waits for memory, not
// for the matrix units, and its smaller stages leave room for more of them in
// flight.  The weights, which come from HBM, have a stage more in flight than
// the rows, which come from L2.
template <int FORM, int EPI, int BM>
__global__ void __launch_bounds__(kThreads, 2) k_rows_mm(MmParams P) {
    extern __shared__ __align__(16) uint8_t smem[];
    const RowTile t = find_tile<BM, EPI == kPart>(P, blockIdx.x);
    if (t.e < 0) return;
    if (t.rows <= 32) rows_tile<FORM, EPI, 64, 1, 4, 4>(P, t, smem);
    else if (BM == 64 || t.rows <= 64) rows_tile<FORM, EPI, 64, 2, 4, 4>(P, t, smem);
    else if constexpr (BM > 64) {
        if (t.rows <= 96) rows_tile<FORM, EPI, 128, 3, 3, 3>(P, t, smem);
        else if (t.rows <= 128) rows_tile<FORM, EPI, 128, 4, 3, 3>(P, t, smem);
        else if (t.rows <= 160) rows_tile<FORM, EPI, 192, 5, 2, 3>(P, t, smem);
        else if (t.rows <= 192) rows_tile<FORM, EPI, 192, 6, 2, 3>(P, t, smem);
        else if (t.rows <= 224) rows_tile<FORM, EPI, 256, 7, 2, 3>(P, t, smem);
        else if (t.rows <= 256) rows_tile<FORM, EPI, 256, 8, 2, 3>(P, t, smem);
        else rows_tile<FORM, EPI, 320, 9, 2, 2>(P, t, smem);
    }
}

// The slices' sums of the experts' rows, in order, and the epilogue: EPI and
// GU as above (kSwiglu without GU: the gradient).  Eight columns a thread.
template <bool GU, int EPI>
__global__ void __launch_bounds__(256) k_rows_join(MmParams P) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8, size = (int64_t)P.M * P.C;
    if (i >= size) return;
    const int64_t row = i / P.C;
    if (row < P.offsets[0] || row >= P.offsets[P.E]) return;
    const auto sum = [&](int which, float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        for (int s = 0; s < P.slices; ++s) {
            const float* p = P.part + (int64_t)(s * (GU ? 2 : 1) + which) * size + i;
            const floatx4 a = *reinterpret_cast<const floatx4*>(p), b = *reinterpret_cast<const floatx4*>(p + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] += a[j];
                v[4 + j] += b[j];
            }
        }
    };
    const auto put = [&](uint16_t* o, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(o + i) = make_uint4(pack_rne(v[0], v[1]), pack_rne(v[2], v[3]), pack_rne(v[4], v[5]), pack_rne(v[6], v[7]));
    };
    float v[8];
    sum(0, v);
    if constexpr (GU) {
        float u[8], h[8];
        sum(1, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = v[j] * sigmoid(v[j]) * u[j];
        put(P.o0, h);
        if (P.o1) {
            put(P.o1, v);
            put(P.o2, u);
        }
    } else if constexpr (EPI == kSwiglu) {
        const uint4 av = *reinterpret_cast<const uint4*>(P.i0 + i), bv = *reinterpret_cast<const uint4*>(P.i1 + i);
        const floatx4 a[2] = {widen4(av.x, av.y), widen4(av.z, av.w)}, b[2] = {widen4(bv.x, bv.y), widen4(bv.z, bv.w)};
        float da[8], db[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) swiglu_grad(v[j], a[j / 4][j % 4], b[j / 4][j % 4], da[j], db[j]);
        put(P.o0, da);
        put(P.o1, db);
    } else {
        put(P.o0, v);
    }
}

// ---------------------------------------------------------------- weight gradient
struct WgradParams {
    const uint16_t* dy;           // [M][N]
    const uint16_t* x;            // [X][K]
    const int32_t* offsets;
    const int32_t* slots;
    int E, M, X, k;
    uint32_t kmagic;
    int N, K, ntn, ntk;
    int slice;                    // rows of a slice of the reduction
    int accumulate;
    int shared_lines;             // 64-byte lines of dW that two tiles share: through the L2
    float* dw;                    // [E][N][K]
    float* part;                  // fp32 [N][K] per slice of the experts that have two or more
    int parts;                    // how many fit (offsets that are not ascending could ask for more)
};

constexpr int kSrcRows = 1024;    // gathered rows whose places in x are kept in LDS at a time

constexpr int kTurnRow = 272;     // bytes of a row of 64 sums in LDS, 16 apart in banks

constexpr int wgrad_lds(int WM, int WN, int MI, int NI, int BK, int NSA, int NSB) {
    return (NSA * MI * WM * 16 + NSB * NI * WN * 16) * BK * 2 + (NSA == NSB ? kSrcRows * 4 : 0);
}

// One workgroup of WM waves along n by WN along k: a tile of 16 WM MI x 16 WN
// NI of one expert's dW over one slice of its rows, in stages of BK rows,
// NSA of dy's and NSB of x's in LDS (NSB > NSA: nothing is gathered, and the
// table of gathered rows has no room; x, the wider one, is then a stage more
// ahead).
template <int WM, int WN, int MI, int NI, int BK, int NSA, int NSB>
__global__ void __launch_bounds__(WM * WN * kWave, 2) k_wgrad(WgradParams P) {
    constexpr int W = WM * WN, TM = WM * MI * 16, TN = WN * NI * 16;   // waves; rows n, columns k of the tile
    constexpr int kABytes = TM * BK * 2, kBBytes = TN * BK * 2, kBRing = NSA * kABytes;
    constexpr int kADma = kABytes / 1024 / W, kBDma = kBBytes / 1024 / W;
    constexpr int kARows = 512 / TM, kBRows = 512 / TN;             // LDS rows per DMA
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t* srcs = reinterpret_cast<uint32_t*>(smem + kBRing + NSB * kBBytes);
    constexpr bool kGather = NSA == NSB;
    const int per = P.ntn * P.ntk;
    const Piece f = find_piece<true>(P.offsets, P.E, P.M, P.slice, per, blockIdx.x);
    if (f.e < 0) return;
    const int e = f.e, sl = f.idx / per, tile = f.idx % per;
    // along k first: tiles that run together then write runs of whole rows (32
    // experts of 256 rows, 5120 x 1536: 249 us the other way, 237 so)
    const int n0 = tile / P.ntk * TM, k0 = tile % P.ntk * TN;
    const int p0 = f.lo + sl * P.slice, cnt = min(f.n - sl * P.slice, P.slice);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int lrow = lane & 15, q = lane >> 4;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8*)smem;

    // a lane's LDS row and the columns that it fetches, per DMA
    uint32_t aoff[kADma], xcol[kBDma];
    int arow[kADma], xrow[kBDma];
    const auto column = [&](int r, int pos) { return (((pos >> 1) ^ ro_swizzle(r)) << 4) + ((pos & 1) << 3); };
#pragma unroll
    for (int i = 0; i < kADma; ++i) {
        const int r = (i * W + wave) * kARows + lane / (64 / kARows), col = column(r, lane % (64 / kARows));
        arow[i] = r;
        aoff[i] = n0 + col < P.N ? (uint32_t)r * (uint32_t)P.N * 2u + col * 2 : kOutside;
    }
#pragma unroll
    for (int i = 0; i < kBDma; ++i) {
        const int r = (i * W + wave) * kBRows + lane / (64 / kBRows), col = column(r, lane % (64 / kBRows));
        xrow[i] = r;
        xcol[i] = k0 + col < P.K ? (uint32_t)col * 2u : kOutside;
    }
    const int nstages = (cnt + BK - 1) / BK;
    // Gathered: the byte offsets in x of the next kSrcRows rows (kOutside:
    // none), looked up ahead of the stages, since a load in line with their
    // DMAs would wait for all of them.
    const auto look_up = [&](int s) {
        for (int i = threadIdx.x; i < kSrcRows; i += W * kWave) {
            const int r = s * BK + i, slot = P.slots[min(p0 + r, P.M - 1)], src = slot_token(slot, P.k, P.kmagic);
            srcs[i] = r < cnt && slot >= 0 && src < P.X ? (uint32_t)src * (uint32_t)P.K * 2u : kOutside;
        }
        wait_lds_barrier();
    };
    const auto dma_a = [&](int s) {
        const int r0 = s * BK;
        const uint32_t buf = lds0 + (s % NSA) * kABytes;
        const uint16_t* a = uniform_ptr(P.dy + (int64_t)(p0 + r0) * P.N + n0);
#pragma unroll
        for (int i = 0; i < kADma; ++i)
            lds_dma16_buf(a, r0 + arow[i] < cnt ? aoff[i] : kOutside, buf + (i * W + wave) * 1024);
    };
    const auto dma_b = [&](int s) {
        const int r0 = s * BK;
        const uint32_t buf = lds0 + kBRing + (s % NSB) * kBBytes;
        if (kGather && P.slots && r0 % kSrcRows == 0) look_up(s);
        const uint16_t* x = uniform_ptr(P.x + (kGather && P.slots ? 0 : (int64_t)(p0 + r0) * P.K) + k0);
#pragma unroll
        for (int i = 0; i < kBDma; ++i) {
            const uint32_t row = kGather && P.slots ? srcs[(r0 + xrow[i]) % kSrcRows]
                                         : r0 + xrow[i] < cnt ? (uint32_t)xrow[i] * (uint32_t)P.K * 2u : kOutside;
            lds_dma16_buf(x, row != kOutside && xcol[i] != kOutside ? row + xcol[i] : kOutside,
                          buf + (i * W + wave) * 1024);
        }
    };

    int ard[BK / 32], brd[BK / 32], ac[MI], bc[NI];
    const int sw = (lrow >> 2) | ((q & 1) << 2);
#pragma unroll
    for (int ks = 0; ks < BK / 32; ++ks) {
        const int r = ks * 32 + q * 8 + (lrow >> 2);
        ard[ks] = r * TM * 2 + (lrow & 3) * 8;
        brd[ks] = r * TN * 2 + (lrow & 3) * 8;
    }
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) ac[mi] = ((wm * MI + mi) ^ sw) * 32;
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) bc[ni] = ((wn * NI + ni) ^ sw) * 32;

    floatx4 acc[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = floatx4{0, 0, 0, 0};

    const auto read_a = [&](int buf, int ks, int mi) {
        return frag_ro<TM * 2>((const lds_u8*)smem + buf * kABytes, ard[ks] + ac[mi]);
    };
    const auto read_b = [&](int buf, int ks, int ni) {
        return frag_ro<TN * 2>((const lds_u8*)smem + kBRing + buf * kBBytes, brd[ks] + bc[ni]);
    };
    if (nstages > 0) {
        if constexpr (BK == 64)
            run_stages<NSA, NSB, MI, NI, kADma, kBDma, 2, 2>(nstages, dma_a, dma_b, read_a, read_b, acc);
        else
            run_steps<NSA, MI, NI, kADma + kBDma, 2, 2>(
                nstages, [&](int s) { dma_a(s); dma_b(s); }, [&](int buf, int mi) { return read_a(buf, 0, mi); },
                [&](int buf, int ni) { return read_b(buf, 0, ni); }, acc);
    }
    const bool whole = f.pieces == 1;
    if (!whole && f.cut_before + sl >= P.parts) return;
    float* base = whole ? P.dw + (int64_t)e * P.N * P.K : P.part + (int64_t)(f.cut_before + sl) * P.N * P.K;
    const bool add = whole && P.accumulate;
    // A wave turns sixteen rows at a time around in LDS of its own, so that a
    // store instruction writes 256 bytes of four rows and not 64 of sixteen
    // (128 bytes of eight: 64 rows 184 us against 177, 256 rows 267 against 249;
    // no better with 1 KB).
    static_assert(NI == 4 && W * 16 * kTurnRow <= kBRing + NSB * kBBytes, "the stages' memory");
    uint8_t* turn = smem + wave * 16 * kTurnRow;
    const auto store = [&](auto shared_lines) {
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
            for (int ni = 0; ni < NI; ++ni)
                *reinterpret_cast<floatx4*>(turn + lrow * kTurnRow + ni * 64 + q * 16) = acc[mi][ni];
            const int c = k0 + wn * 64 + lrow * 4;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int n = n0 + (wm * MI + mi) * 16 + h * 4 + q;
                floatx4 w = *reinterpret_cast<const floatx4*>(turn + (h * 4 + q) * kTurnRow + lrow * 16);
                if (n >= P.N || c >= P.K) continue;
                floatx4* p = reinterpret_cast<floatx4*>(base + (int64_t)n * P.K + c);
                if (add) w += *p;
                if constexpr (decltype(shared_lines)::value) {
                    // floats by which the wave's columns begin inside a line of 64 bytes
                    const int skew = ((int)(reinterpret_cast<uintptr_t>(p) >> 2) - lrow * 4) & 15;
                    const bool shared = lrow * 4 < (-skew & 15) || lrow * 4 >= 64 - skew;
                    // these first: after the others of their rows they cost half as
                    // much again (179 us against 141); the comments between them
                    // keep the compiler from making one store of the two
                    if (shared) *p = w;
                    asm volatile("; whole lines" ::: "memory");
                    if (!shared) __builtin_nontemporal_store(w, p);
                    asm volatile("; next rows" ::: "memory");
                } else {
                    __builtin_nontemporal_store(w, p);
                }
            }
        }
    };
    if (P.shared_lines) store(std::true_type{});
    else store(std::false_type{});
}

// dW of the experts whose rows were cut into slices: the slices' sums, in order.
__global__ void __launch_bounds__(256) k_wgrad_join(WgradParams P) {
    const int lane = threadIdx.x & 63, e = blockIdx.y;
    int before = 0, pieces = 0;
    for (int b = 0; b <= e; b += kWave) {
        int k = 0;
        if (b + lane <= e) {
            const int lo = max(P.offsets[b + lane], 0), n = min(P.offsets[b + lane + 1], P.M) - lo;
            k = (max(n, 0) + P.slice - 1) / P.slice;
            if (k <= 1) k = 0;
        }
        if (b + kWave > e) {
            pieces = __builtin_amdgcn_readlane(k, e - b);
            if (lane >= e - b) k = 0;
        }
        before += __builtin_amdgcn_readlane(wave_inclusive_scan_dpp(k), 63);
    }
    pieces = min(pieces, P.parts - before);
    if (pieces <= 1) return;
    const int64_t size = (int64_t)P.N * P.K, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= size) return;
    const float* part = P.part + before * size + i;
    float* dw = P.dw + e * size + i;
    floatx4 v = {0, 0, 0, 0};
    if (P.accumulate) v = *reinterpret_cast<const floatx4*>(dw);
    for (int s = 0; s < pieces; ++s) v += *reinterpret_cast<const floatx4*>(part + s * size);
    *reinterpret_cast<floatx4*>(dw) = v;
}

// Workgroups of a row-tiled launch: at most floor(M / BM) + min(E, M) row
// tiles exist (one partial tile per expert); the ones beyond leave at once.
int64_t row_tiles_bound(int M, int E, int BM) { return M / BM + (int64_t)std::min(E, M); }

// How a row product of M rows of E experts runs: tiles of up to 64 or 288
// rows, and its reduction's slices.
struct RowsPlan {
    int bm, slices;
    size_t part_bytes;
};

// From the mean rows of an expert; the offsets are not known here.  A tile
// goes through its reduction stage by stage (64 steps: 1.2 us for 256 rows;
// for 64 rows 0.5 us with the other CUs quiet, 0.65 us with all of them
// busy), so where tiles are few it is cut into slices, whose fp32 sums are
// joined (4.5 TB/s, and another launch).  512 rows of one expert, 5120 x 512:
// 106 us in two tiles, 47 us in 16, 17 us in 16 of 8 slices; 80 rows of two
// experts, 5120 x 1536: 60 us whole, 17.6 us in slices; 8 experts of 256 rows,
// 5120 x 1536, 105 us in 48 tiles and 55 us in 192 without slices.
// With a tile for every CU the height follows the mean (64 experts of uneven
// rows, 288 against 64: mean 24, 5120 x 1536, 183 against 189 us; 56, 1536 x
// 5120, 198 against 212; 100, 768 x 2048, 42 against 54).
RowsPlan rows_plan(int M, int E, int R, int C, int pairs, int outs, int ntc) {
    const int64_t experts = std::max(1, std::min(E, M)), mean = (M + experts - 1) / experts;
    const int64_t t288 = experts * ((mean + 287) / 288) * ntc, t64 = experts * ((mean + 63) / 64) * ntc;
    const int stages = (R + kBK - 1) / kBK * pairs;
    RowsPlan best{mean > 48 ? 288 : 64, 1, 0};
    if ((mean > 48 ? t288 : t64) >= 256) return best;
    double least = 1e30;
    for (const int bm : {64, 288}) {
        if (bm == 288 && mean <= 48) break;
        const int64_t tiles = bm == 64 ? t64 : t288;
        for (int n = 1; n <= 16; ++n) {
            if (n > 1 && (n * 4 > stages || tiles * n > 512)) break;
            // a short 288-tile costs what its rows do
            const double stage = bm == 64 ? 0.5 + 0.15 * std::min(1.0, tiles * n / 256.0)
                                          : 0.3 + 0.9 * std::min<double>(mean, 288) / 256;
            const double bytes = (double)n * outs * M * C * 4;
            const double us = (double)((tiles * n + 255) / 256) * ((stages + n - 1) / n) * stage +
                              (n > 1 ? 4 + 2 * bytes / 4.5e6 : 0);
            if (us < least) {
                least = us;
                best = RowsPlan{bm, n, n > 1 ? (size_t)bytes : 0};
            }
        }
    }
    return best;
}

template <int FORM, int EPI, int BM>
moe_status launch_rows(const MmParams& P, const char* name, hipStream_t s) {
    const int64_t grid = xcd_grid(row_tiles_bound(P.M, P.E, BM) * P.ntc * (EPI == kPart ? P.slices : 1));
    constexpr size_t lds = rows_lds(256, 2, 3);
    static_assert(rows_lds(64, 4, 4) <= lds && rows_lds(128, 3, 3) <= lds && rows_lds(320, 2, 2) <= lds,
                  "one size");
    moe_status st = allow_dynamic_lds(reinterpret_cast<const void*>(&k_rows_mm<FORM, EPI, BM>), lds);
    if (st != MOE_OK) return st;
    MOE_LAUNCH(name, (k_rows_mm<FORM, EPI, BM>), dim3((unsigned)grid), dim3(kThreads), lds, s, P);
    return MOE_OK;
}

template <int FORM, int EPI>
moe_status launch_rows_any(MmParams P, const char* name, void* ws, hipStream_t s) {
    const RowsPlan p = rows_plan(P.M, P.E, P.R, P.C, P.pairs, FORM == kGateUp ? 2 : 1, P.ntc);
    if (p.slices > 1) {
        P.slices = p.slices;
        P.part = static_cast<float*>(ws);
        const moe_status st = p.bm == 64 ? launch_rows<FORM, kPart, 64>(P, name, s) : launch_rows<FORM, kPart, 288>(P, name, s);
        if (st != MOE_OK) return st;
        MOE_LAUNCH("grouped_join", (k_rows_join<FORM == kGateUp, EPI>), dim3((unsigned)(((int64_t)P.M * P.C + 2047) / 2048)),
                   dim3(256), 0, s, P);
        return MOE_OK;
    }
    return p.bm == 64 ? launch_rows<FORM, EPI, 64>(P, name, s) : launch_rows<FORM, EPI, 288>(P, name, s);
}

int column_tiles(int C, bool gate_up) { return gate_up ? (C + kBN / 2 - 1) / (kBN / 2) : (C + kBN - 1) / kBN; }

// Tile of a weight gradient (rows n, columns k) and rows of a slice of its reduction.
struct WgradPlan {
    int tn, tk, ntn, ntk, slice, parts;
    int64_t tiles, part_bytes;
};

WgradPlan wgrad_plan(int M, int N, int K, int E, bool gathered) {
    WgradPlan p{};
    const auto tile = [&](int tn, int tk) {
        p.tn = tn;
        p.tk = tk;
        p.ntn = (N + tn - 1) / tn;
        p.ntk = (K + tk - 1) / tk;
        return (int64_t)p.ntn * p.ntk;
    };
    // the tile of 256 n reads x half as often; the one of 128 leaves room for
    // two workgroups a CU, one storing while the other multiplies, and wastes
    // less on a small N (32 experts, 5120 x 1536, us in tiles of 128 and 256:
    // 128 rows 176, 187, 256 rows 213, 235, 384 rows 275, 280, 512 rows 325,
    // 322; gathered, where each tile looks its rows up: 192 rows 222, 223, 256
    // rows 246, 244, 512 rows 356, 338)
    const bool big = M / E >= 192 && (N + 127) / 128 % 2 == 0;
    const int64_t slots = big ? 256 : 512;
    int64_t per = tile(big ? 256 : 128, 256);
    p.slice = 1 << 30;
    // Few tiles: slices of at least 8 stages (the join and its partial sums
    // cost as much), so that their number comes near the workgroups that run
    // at once.  Of 256 x 128 tiles half as many slices do it, and their partial
    // sums are half as many bytes (one group of 8195 rows, 256 x 5120: 45 -> 38 us).
    if (2 * per * E <= slots) {
        if (big) per = tile(256, 128);
        const int64_t want = std::max<int64_t>(1, slots / per), stages = (M + kBK - 1) / kBK;
        const int64_t rows = std::max<int64_t>((stages + want - 1) / want, 8) * kBK;
        if (rows < M) p.slice = (int)rows;
    }
    if (p.slice >= M && big && !gathered && M / E < 448) per = tile(128, 256);    // (no slices: no workspace either way)
    p.parts = p.slice < M ? 2 * (M / p.slice) + 2 : 0;
    p.part_bytes = (int64_t)p.parts * N * K * 4;
    p.tiles = (p.slice < M ? M / p.slice + (int64_t)E : E) * per;
    return p;
}

template <int WM, int WN, int MI, int NI, int BK, int NSA, int NSB>
moe_status launch_wgrad(const WgradParams& P, int64_t tiles, hipStream_t s) {
    constexpr size_t lds = wgrad_lds(WM, WN, MI, NI, BK, NSA, NSB);
    moe_status st = allow_dynamic_lds(reinterpret_cast<const void*>(&k_wgrad<WM, WN, MI, NI, BK, NSA, NSB>), lds);
    if (st != MOE_OK) return st;
    MOE_LAUNCH("grouped_wgrad", (k_wgrad<WM, WN, MI, NI, BK, NSA, NSB>), dim3((unsigned)xcd_grid(tiles)), dim3(WM * WN * kWave),
               lds, s, P);
    return MOE_OK;
}

}  // namespace

bool grouped_grid_fits(int M, int E, int C) {
    return (M / 64 + (int64_t)std::min(E, M)) * ((C + 127) / 128) < (1 << 22);
}

bool wgrad_grid_fits(int N, int K, int E) { return (int64_t)E * ((N + 127) / 128) * ((K + 127) / 128) < (1 << 22); }

size_t grouped_rows_workspace_bytes(int M, int E, int R, int C, int pairs, bool gate_up) {
    return rows_plan(M, E, R, C, pairs, gate_up ? 2 : 1, column_tiles(C, gate_up)).part_bytes;
}

moe_status launch_grouped_fwd(const GroupedArgs& g, void* ws, hipStream_t s) {
    MmParams P{};
    P.a0 = g.x;
    P.w0 = g.w;
    P.w1 = g.w2;
    P.offsets = g.offsets;
    P.slots = g.slots;
    P.E = g.E; P.M = g.M; P.X = g.X; P.k = g.k;
    P.kmagic = div_magic(g.k);
    P.R = g.K; P.C = g.N;
    P.pairs = 1;
    P.o0 = g.o0; P.o1 = g.o1; P.o2 = g.o2;
    P.ntc = column_tiles(g.N, g.w2 != nullptr);
    if (g.w2) return launch_rows_any<kGateUp, kSwiglu>(P, "grouped_swiglu", ws, s);
    return launch_rows_any<kNT, kPlain>(P, "grouped_linear", ws, s);
}

moe_status launch_grouped_dgrad(const GroupedArgs& g, void* ws, hipStream_t s) {
    MmParams P{};
    P.a0 = g.dy;
    P.a1 = g.dy2;
    P.w0 = g.w;
    P.w1 = g.w2;
    P.offsets = g.offsets;
    P.E = g.E; P.M = g.M; P.X = g.M; P.k = 1;
    P.R = g.N; P.C = g.K;
    P.pairs = g.dy2 ? 2 : 1;
    P.o0 = g.o0; P.o1 = g.o1;
    P.i0 = g.a; P.i1 = g.b;
    P.ntc = column_tiles(g.K, false);
    if (g.a) return launch_rows_any<kNN, kSwiglu>(P, "grouped_swiglu_dgrad", ws, s);
    return launch_rows_any<kNN, kPlain>(P, "grouped_dgrad", ws, s);
}

size_t grouped_wgrad_workspace_bytes(int M, int N, int K, int E) {
    return (size_t)wgrad_plan(M, N, K, E, false).part_bytes;    // the same where rows are gathered
}

moe_status launch_grouped_wgrad(const GroupedArgs& g, float* dw, bool accumulate, void* ws, hipStream_t s) {
    const WgradPlan p = wgrad_plan(g.M, g.N, g.K, g.E, g.slots != nullptr);
    WgradParams P{};
    P.dy = g.dy;
    P.x = g.x;
    P.offsets = g.offsets;
    P.slots = g.slots;
    P.E = g.E; P.M = g.M; P.X = g.X; P.k = g.k;
    P.kmagic = div_magic(g.k);
    P.N = g.N; P.K = g.K;
    P.ntn = p.ntn;
    P.ntk = p.ntk;
    P.slice = p.slice;
    P.accumulate = accumulate;
    // Rows of dW that begin inside a 64-byte line: the lines between two waves'
    // columns leave by plain stores, to be whole when the L2 writes them; past
    // the caches each half costs a read as well (64 experts, 656 x 4824, 32 rows:
    // 241 us against 143; 54 experts, 1896 x 504: 68 against 43, 256 rows 73
    // against 67).  With much to write and to read they leave the L2 before that
    // (656 x 4824, 128 rows: 243 us against 231, 256 rows 311 against 243).
    P.shared_lines = g.K % 16 != 0 && (g.M / g.E <= 64 || (int64_t)g.E * g.N * g.K * 4 <= 1 << 29);
    P.dw = dw;
    P.part = static_cast<float*>(ws);
    P.parts = p.parts;
    const moe_status st = p.tn == 128   ? launch_wgrad<1, 4, 8, 4, 32, 3, 3>(P, p.tiles, s)
                          : p.tk == 128 ? launch_wgrad<4, 2, 4, 4, 64, 3, 3>(P, p.tiles, s)
                          : P.slots     ? launch_wgrad<2, 4, 8, 4, 64, 2, 2>(P, p.tiles, s)
                                        : launch_wgrad<2, 4, 8, 4, 64, 2, 3>(P, p.tiles, s);
    if (st != MOE_OK || p.part_bytes == 0) return st;
    MOE_LAUNCH("grouped_wgrad_join", k_wgrad_join, dim3((unsigned)(((int64_t)g.N * g.K + 1023) / 1024), g.E), dim3(256),
               0, s, P);
    return MOE_OK;
}

}  // namespace moe
