// Rows sorted by expert: which piece of which expert's rows a workgroup
// takes, and which token a sorted slot belongs to.
#pragma once

#include "device_common.h"

namespace moe {

// slot / k for 0 <= slot < 2^31, with magic = floor(2^32 / k) (k > 1) or 0
// (k == 1): the estimate is at most one too small.
__device__ __forceinline__ int slot_token(int slot, int k, uint32_t magic) {
    if (magic == 0) return slot;
    uint32_t q = __umulhi((uint32_t)slot, magic);
    if ((uint32_t)slot - q * (uint32_t)k >= (uint32_t)k) ++q;
    return (int)q;
}

inline uint32_t div_magic(int k) { return k <= 1 ? 0u : (uint32_t)((1ull << 32) / (uint32_t)k); }

// Number of workgroup `bid` among `total` tiles, or -1: the eight XCDs (which
// the workgroups go to in turn, 32 CUs each) take equal runs of at most 32
// tiles in turn, so that neighbours meet in one L2, no XCD gets all the long
// experts and none gets a run more than another.
__device__ __forceinline__ int xcd_tile(int bid, int total) {
    const int rounds = max((total + 255) >> 8, 1), run = (total + 8 * rounds - 1) / (8 * rounds), idx = bid >> 3;
    const int t = ((idx / max(run, 1)) * 8 + (bid & 7)) * run + idx % max(run, 1);
    return t < total ? t : -1;
}
// workgroups that number at most `total` tiles that way
inline int64_t xcd_grid(int64_t total) { return total + 8 * ((total + 255) / 256) + 8; }

// The expert that holds the tile of workgroup `bid`, when every expert with n
// rows has ceil(n / H) pieces (one, if n is 0 and EMPTY) of `per_piece` tiles:
// its rows, the tile's number inside the expert, and how many pieces the
// experts before it have that are cut in two or more.  Offsets are clamped to
// [0, M], so no piece leaves the buffers.
// TALL: experts whose pieces, cut to equal heights, are taller than that come
// first.  Workgroups start in order, so short ones then fill the last round
// (32 experts of about 255 rows, 6 column tiles: 240 -> 218 us).
struct Piece {
    int e, lo, n, pieces, idx, cut_before;
};
template <bool EMPTY, int TALL = 0>
__device__ __forceinline__ Piece find_piece(const int32_t* __restrict__ offsets, int E, int M, int H, int per_piece,
                                            int bid) {
    const int lane = threadIdx.x & 63;
    const int per = (E + kWave - 1) / kWave, b = lane * per;
    const auto rows = [&](int e, int& lo) {
        lo = max(offsets[e], 0);
        return max(min(offsets[e + 1], M) - lo, 0);
    };
    const auto pieces = [&](int n) { return EMPTY ? max((n + H - 1) / H, 1) : (n + H - 1) / H; };
    const auto is_tall = [&](int n, int k) { return TALL && n > TALL * k; };
    int local = 0, tall = 0, cut = 0, lo = 0, n = 0;
#pragma unroll 1
    for (int i = 0; i < per; ++i)
        if (b + i < E) {
            n = rows(b + i, lo);
            const int k = pieces(n);
            (is_tall(n, k) ? tall : local) += k;
            cut += k > 1 ? k : 0;
        }
    // offsets that are not ascending could ask for more tiles than an int counts
    const int most = (1 << 23) / per_piece;
    local = min(local, most);
    tall = min(tall, most);
    int incl = wave_inclusive_scan_dpp(local), mine = local;
    const int cincl = EMPTY ? wave_inclusive_scan_dpp(cut) : 0;
    const int tincl = TALL ? wave_inclusive_scan_dpp(tall) : 0;
    const int first_tiles = __builtin_amdgcn_readlane(tincl, 63) * per_piece;
    int t = xcd_tile(bid, first_tiles + __builtin_amdgcn_readlane(incl, 63) * per_piece);
    if (t < 0) return Piece{-1, 0, 0, 0, 0, 0};
    const bool in_tall = t < first_tiles;
    if (in_tall) {
        incl = tincl;
        mine = tall;
    } else {
        t -= first_tiles;
    }
    const int src = __ffsll((unsigned long long)__ballot(incl * per_piece > t)) - 1;
    int first = __builtin_amdgcn_readlane(incl - mine, src) * per_piece;
    int before = __builtin_amdgcn_readlane(cincl - cut, src);
    if (per == 1)                                  // the lane's expert is still at hand
        return Piece{src, __builtin_amdgcn_readlane(lo, src), __builtin_amdgcn_readlane(n, src),
                     __builtin_amdgcn_readlane(mine, src), t - first, before};
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const int e = src * per + i;
        n = rows(e, lo);
        const int k = pieces(n);
        if (is_tall(n, k) == in_tall) {
            if (t < first + k * per_piece)
                return Piece{__builtin_amdgcn_readfirstlane(e), __builtin_amdgcn_readfirstlane(lo),
                             __builtin_amdgcn_readfirstlane(n), __builtin_amdgcn_readfirstlane(k),
                             __builtin_amdgcn_readfirstlane(t - first), __builtin_amdgcn_readfirstlane(before)};
            first += k * per_piece;
        }
        before += k > 1 ? k : 0;
    }
    return Piece{-1, 0, 0, 0, 0, 0};
}

}  // namespace moe
