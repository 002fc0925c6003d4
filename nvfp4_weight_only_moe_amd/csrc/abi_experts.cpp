// C ABI of the operators on unquantized and 4-bit integer experts: argument
// checking and dispatch.  As in abi.cpp every check runs on the host before
// anything is enqueued.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "abi_common.h"
#include "internal.h"

using namespace moe;

namespace {

constexpr int32_t kMaxDim = 1 << 20;                    // N, K, H
constexpr int64_t kMaxRows = INT32_MAX / 2;             // M, T * k
constexpr int64_t kMaxGatherBytes = 0xFFFFFF00ll;       // x addressed by 32-bit offsets when rows are gathered

struct Buf {
    const void* p;
    size_t bytes;
};

moe_status check_present(std::initializer_list<Buf> bufs) {
    for (const Buf& b : bufs)
        if (!b.p) return MOE_ERR_INVALID_ARG;
    for (const Buf& b : bufs)
        if (!aligned16(b.p)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

// Every output (null: absent) apart from the inputs and the other outputs.
moe_status check_apart(std::initializer_list<Buf> outs, std::initializer_list<Buf> ins) {
    for (const Buf* o = outs.begin(); o != outs.end(); ++o) {
        if (!o->p) continue;
        if (!aligned16(o->p)) return MOE_ERR_ALIGN;
        for (const Buf& i : ins)
            if (i.p && ranges_overlap(o->p, o->bytes, i.p, i.bytes)) return MOE_ERR_INVALID_ARG;
        for (const Buf* q = outs.begin(); q != o; ++q)
            if (q->p && ranges_overlap(o->p, o->bytes, q->p, q->bytes)) return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}

inline size_t b16(int64_t rows, int64_t cols) { return (size_t)rows * (size_t)cols * 2; }

// Shapes of a grouped product: M rows, N x K weights of E experts.
moe_status check_group_shape(int32_t M, int32_t N, int32_t K, int32_t E) {
    if (M < 0 || N < 1 || K < 1 || E < 1) return MOE_ERR_SHAPE;
    if (E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    if (N % 8 || K % 8 || N > kMaxDim || K > kMaxDim || M > kMaxRows) return MOE_ERR_SHAPE;
    if (!grouped_grid_fits(M, E, N) || !grouped_grid_fits(M, E, K)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

// A workspace of `need` bytes, apart from the call's buffers.
moe_status check_ws(void* d_ws, size_t ws_bytes, size_t need, std::initializer_list<Buf> bufs) {
    if (need == 0) return MOE_OK;
    if (!d_ws || ws_bytes < need) return MOE_ERR_WORKSPACE;
    return check_apart({Buf{d_ws, need}}, bufs);
}

// x's rows: gathered through sorted slots (slot / k), or row p for row p.
moe_status check_rows(int32_t X, int32_t M, int32_t K, const int32_t* slots, int32_t k) {
    if (X < 0) return MOE_ERR_SHAPE;
    if (!slots) return X == M ? MOE_OK : MOE_ERR_SHAPE;
    if (k < 1) return MOE_ERR_SHAPE;
    if (k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    if (X < 1 || (int64_t)X * K * 2 > kMaxGatherBytes) return MOE_ERR_SHAPE;
    if (!aligned16(slots)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

moe_status check_int4(const moe_int4_tensor* t) {
    if (!t) return MOE_ERR_INVALID_ARG;
    if (t->E < 1 || t->N < 1 || t->K < 1 || t->K % 128 || t->N > kMaxDim || t->K > kMaxDim) return MOE_ERR_SHAPE;
    if (t->group != 32 && t->group != 64 && t->group != 128) return MOE_ERR_SHAPE;
    if (t->E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)t->E * t->N * t->K > ((int64_t)1 << 34)) return MOE_ERR_SHAPE;
    if (!t->codes || !t->scales) return MOE_ERR_INVALID_ARG;
    if (!aligned16(t->codes) || !aligned16(t->scales) || !aligned16(t->zeros)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

size_t int4_codes_bytes(const moe_int4_tensor* t) { return (size_t)t->E * t->N * t->K / 2; }
size_t int4_groups(const moe_int4_tensor* t) { return (size_t)t->E * t->N * (t->K / t->group); }

}  // namespace

extern "C" {

size_t moe_grouped_workspace_size(int32_t M, int32_t E, int32_t R, int32_t C, int32_t products) {
    if (products < 1 || products > 3 || check_group_shape(M, C, R, E) != MOE_OK || M == 0) return 0;
    return grouped_rows_workspace_bytes(M, E, R, C, products == MOE_GROUPED_PAIR ? 2 : 1, products == MOE_GROUPED_SWIGLU);
}

moe_status moe_grouped_linear(const uint16_t* d_x, int32_t X, int32_t K, const uint16_t* d_w, int32_t E, int32_t N,
                              const int32_t* d_offsets, const int32_t* d_sorted_slots, int32_t k, int32_t M,
                              uint16_t* d_y, void* d_ws, size_t ws_bytes, hipStream_t stream) {
    moe_status st = check_group_shape(M, N, K, E);
    if (st != MOE_OK) return st;
    if (M == 0) return MOE_OK;
    if ((st = check_rows(X, M, K, d_sorted_slots, k)) != MOE_OK) return st;
    const Buf x{d_x, b16(X, K)}, w{d_w, b16((int64_t)E * N, K)}, off{d_offsets, (size_t)(E + 1) * 4},
        slots{d_sorted_slots, (size_t)M * 4}, y{d_y, b16(M, N)};
    if ((st = check_present({x, w, off, y})) != MOE_OK) return st;
    if ((st = check_apart({y}, {x, w, off, slots})) != MOE_OK) return st;
    if ((st = check_ws(d_ws, ws_bytes, grouped_rows_workspace_bytes(M, E, K, N, 1, false), {x, w, off, slots, y})) != MOE_OK)
        return st;
    GroupedArgs g{};
    g.x = d_x; g.w = d_w; g.offsets = d_offsets; g.slots = d_sorted_slots;
    g.E = E; g.M = M; g.X = X; g.k = d_sorted_slots ? k : 1; g.N = N; g.K = K;
    g.o0 = d_y;
    return launch_grouped_fwd(g, d_ws, stream);
}

moe_status moe_grouped_swiglu(const uint16_t* d_x, int32_t X, int32_t K, const uint16_t* d_gate,
                              const uint16_t* d_up, int32_t E, int32_t N, const int32_t* d_offsets,
                              const int32_t* d_sorted_slots, int32_t k, int32_t M, uint16_t* d_h, uint16_t* d_a,
                              uint16_t* d_b, void* d_ws, size_t ws_bytes, hipStream_t stream) {
    moe_status st = check_group_shape(M, N, K, E);
    if (st != MOE_OK) return st;
    if (M == 0) return MOE_OK;
    if ((st = check_rows(X, M, K, d_sorted_slots, k)) != MOE_OK) return st;
    if ((d_a == nullptr) != (d_b == nullptr)) return MOE_ERR_INVALID_ARG;
    const Buf x{d_x, b16(X, K)}, gate{d_gate, b16((int64_t)E * N, K)}, up{d_up, b16((int64_t)E * N, K)},
        off{d_offsets, (size_t)(E + 1) * 4}, slots{d_sorted_slots, (size_t)M * 4}, h{d_h, b16(M, N)},
        a{d_a, b16(M, N)}, b{d_b, b16(M, N)};
    if ((st = check_present({x, gate, up, off, h})) != MOE_OK) return st;
    if ((st = check_apart({h, a, b}, {x, gate, up, off, slots})) != MOE_OK) return st;
    if ((st = check_ws(d_ws, ws_bytes, grouped_rows_workspace_bytes(M, E, K, N, 1, true),
                       {x, gate, up, off, slots, h, a, b})) != MOE_OK)
        return st;
    GroupedArgs g{};
    g.x = d_x; g.w = d_gate; g.w2 = d_up; g.offsets = d_offsets; g.slots = d_sorted_slots;
    g.E = E; g.M = M; g.X = X; g.k = d_sorted_slots ? k : 1; g.N = N; g.K = K;
    g.o0 = d_h; g.o1 = d_a; g.o2 = d_b;
    return launch_grouped_fwd(g, d_ws, stream);
}

moe_status moe_grouped_linear_dgrad(const uint16_t* d_dy, const uint16_t* d_w, const uint16_t* d_dy2,
                                    const uint16_t* d_w2, int32_t M, int32_t N, int32_t E, int32_t K,
                                    const int32_t* d_offsets, uint16_t* d_dx, void* d_ws, size_t ws_bytes,
                                    hipStream_t stream) {
    moe_status st = check_group_shape(M, N, K, E);
    if (st != MOE_OK) return st;
    if (M == 0) return MOE_OK;
    if ((d_dy2 == nullptr) != (d_w2 == nullptr)) return MOE_ERR_INVALID_ARG;
    const Buf dy{d_dy, b16(M, N)}, w{d_w, b16((int64_t)E * N, K)}, dy2{d_dy2, b16(M, N)},
        w2{d_w2, b16((int64_t)E * N, K)}, off{d_offsets, (size_t)(E + 1) * 4}, dx{d_dx, b16(M, K)};
    if ((st = check_present({dy, w, off, dx})) != MOE_OK) return st;
    if (!aligned16(d_dy2) || !aligned16(d_w2)) return MOE_ERR_ALIGN;
    if ((st = check_apart({dx}, {dy, w, dy2, w2, off})) != MOE_OK) return st;
    if ((st = check_ws(d_ws, ws_bytes, grouped_rows_workspace_bytes(M, E, N, K, d_dy2 ? 2 : 1, false),
                       {dy, w, dy2, w2, off, dx})) != MOE_OK)
        return st;
    GroupedArgs g{};
    g.dy = d_dy; g.dy2 = d_dy2; g.w = d_w; g.w2 = d_w2; g.offsets = d_offsets;
    g.E = E; g.M = M; g.N = N; g.K = K;
    g.o0 = d_dx;
    return launch_grouped_dgrad(g, d_ws, stream);
}

moe_status moe_grouped_swiglu_dgrad(const uint16_t* d_dy, const uint16_t* d_w, int32_t M, int32_t N, int32_t E,
                                    int32_t K, const int32_t* d_offsets, const uint16_t* d_a, const uint16_t* d_b,
                                    uint16_t* d_da, uint16_t* d_db, void* d_ws, size_t ws_bytes,
                                    hipStream_t stream) {
    moe_status st = check_group_shape(M, N, K, E);
    if (st != MOE_OK) return st;
    if (M == 0) return MOE_OK;
    const Buf dy{d_dy, b16(M, N)}, w{d_w, b16((int64_t)E * N, K)}, off{d_offsets, (size_t)(E + 1) * 4},
        a{d_a, b16(M, K)}, b{d_b, b16(M, K)}, da{d_da, b16(M, K)}, db{d_db, b16(M, K)};
    if ((st = check_present({dy, w, off, a, b, da, db})) != MOE_OK) return st;
    if ((st = check_apart({da, db}, {dy, w, off, a, b})) != MOE_OK) return st;
    if ((st = check_ws(d_ws, ws_bytes, grouped_rows_workspace_bytes(M, E, N, K, 1, false),
                       {dy, w, off, a, b, da, db})) != MOE_OK)
        return st;
    GroupedArgs g{};
    g.dy = d_dy; g.w = d_w; g.offsets = d_offsets;
    g.E = E; g.M = M; g.N = N; g.K = K;
    g.a = d_a; g.b = d_b; g.o0 = d_da; g.o1 = d_db;
    return launch_grouped_dgrad(g, d_ws, stream);
}

size_t moe_grouped_linear_wgrad_workspace_size(int32_t M, int32_t N, int32_t K, int32_t E) {
    if (check_group_shape(M, N, K, E) != MOE_OK || !wgrad_grid_fits(N, K, E) || M == 0) return 0;
    return grouped_wgrad_workspace_bytes(M, N, K, E);
}

moe_status moe_grouped_linear_wgrad(const uint16_t* d_dy, int32_t M, int32_t N, const uint16_t* d_x, int32_t X,
                                    int32_t K, int32_t E, const int32_t* d_offsets, const int32_t* d_sorted_slots,
                                    int32_t k, int32_t accumulate, float* d_dw, void* d_ws, size_t ws_bytes,
                                    hipStream_t stream) {
    moe_status st = check_group_shape(M, N, K, E);
    if (st != MOE_OK) return st;
    if (!wgrad_grid_fits(N, K, E)) return MOE_ERR_SHAPE;
    if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
    const Buf dw{d_dw, (size_t)E * N * K * 4}, off{d_offsets, (size_t)(E + 1) * 4};
    if ((st = check_present({off, dw})) != MOE_OK) return st;
    const Buf dy{d_dy, b16(M, N)}, x{d_x, b16(X, K)}, slots{d_sorted_slots, (size_t)M * 4};
    if (M > 0) {
        if ((st = check_rows(X, M, K, d_sorted_slots, k)) != MOE_OK) return st;
        if ((st = check_present({dy, x})) != MOE_OK) return st;
        if ((st = check_apart({dw}, {dy, x, off, slots})) != MOE_OK) return st;
        if ((st = check_ws(d_ws, ws_bytes, grouped_wgrad_workspace_bytes(M, N, K, E), {dy, x, off, slots, dw})) != MOE_OK)
            return st;
    }
    GroupedArgs g{};
    g.dy = d_dy; g.x = d_x; g.offsets = d_offsets; g.slots = M > 0 ? d_sorted_slots : nullptr;
    g.E = E; g.M = M; g.X = X; g.k = g.slots ? k : 1; g.N = N; g.K = K;
    return launch_grouped_wgrad(g, d_dw, accumulate != 0, d_ws, stream);
}

moe_status moe_int4_quantize_pack(const float* d_w, const moe_int4_tensor* out, hipStream_t stream) {
    moe_status st = check_int4(out);
    if (st != MOE_OK) return st;
    const Buf w{d_w, (size_t)out->E * out->N * out->K * 4};
    if ((st = check_present({w})) != MOE_OK) return st;
    if ((st = check_apart({Buf{out->codes, int4_codes_bytes(out)}, Buf{out->scales, int4_groups(out) * 2},
                           Buf{out->zeros, int4_groups(out)}}, {w})) != MOE_OK)
        return st;
    return launch_int4_pack(d_w, out, stream);
}

moe_status moe_int4_dequantize(const moe_int4_tensor* t, float* d_w_out, hipStream_t stream) {
    moe_status st = check_int4(t);
    if (st != MOE_OK) return st;
    const Buf w{d_w_out, (size_t)t->E * t->N * t->K * 4};
    if ((st = check_present({w})) != MOE_OK) return st;
    if ((st = check_apart({w}, {Buf{t->codes, int4_codes_bytes(t)}, Buf{t->scales, int4_groups(t) * 2},
                                Buf{t->zeros, int4_groups(t)}})) != MOE_OK)
        return st;
    return launch_int4_dequant(t, d_w_out, stream);
}

moe_status moe_int4_linear(const uint16_t* d_x, int32_t X, const moe_int4_tensor* w, const int32_t* d_offsets,
                           const int32_t* d_sorted_slots, int32_t k, int32_t M, uint16_t* d_out,
                           hipStream_t stream) {
    moe_status st = check_int4(w);
    if (st != MOE_OK) return st;
    if (M < 0 || M > kMaxRows) return MOE_ERR_SHAPE;
    if (!d_offsets && (w->E != 1 || d_sorted_slots)) return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    if ((st = check_rows(X, M, w->K, d_sorted_slots, k)) != MOE_OK) return st;
    const Buf x{d_x, b16(X, w->K)}, off{d_offsets, (size_t)(w->E + 1) * 4}, slots{d_sorted_slots, (size_t)M * 4},
        out{d_out, b16(M, w->N)};
    if ((st = check_present({x, out})) != MOE_OK) return st;
    if (!aligned16(d_offsets)) return MOE_ERR_ALIGN;
    if ((st = check_apart({out}, {x, off, slots, Buf{w->codes, int4_codes_bytes(w)},
                                  Buf{w->scales, int4_groups(w) * 2}, Buf{w->zeros, int4_groups(w)}})) != MOE_OK)
        return st;
    return launch_int4_linear(d_x, X, w, d_offsets, d_sorted_slots, d_sorted_slots ? k : 1, M, d_out, stream);
}

moe_status moe_combine(const uint16_t* d_y, int32_t M, int32_t H, const int32_t* d_slot_pos, const float* d_w,
                       int32_t T, int32_t k, uint16_t* d_out, hipStream_t stream) {
    if (T < 0 || M < 0 || k < 1 || H < 8 || H % 8 || H > kMaxDim || T > (1 << 22) || M > kMaxRows) return MOE_ERR_SHAPE;
    if (k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    const Buf y{d_y, b16(M, H)}, pos{d_slot_pos, (size_t)T * k * 4}, w{d_w, (size_t)T * k * 4}, out{d_out, b16(T, H)};
    moe_status st = check_present({pos, out});
    if (st != MOE_OK) return st;
    if (M > 0 && !d_y) return MOE_ERR_INVALID_ARG;
    if (!aligned16(d_y) || !aligned16(d_w)) return MOE_ERR_ALIGN;
    if ((st = check_apart({out}, {y, pos, w})) != MOE_OK) return st;
    return launch_combine_rows(d_y, M, H, d_slot_pos, d_w, T, k, d_out, stream);
}

moe_status moe_combine_backward(const uint16_t* d_dout, int32_t T, int32_t H, const uint16_t* d_y, int32_t M,
                                const int32_t* d_slot_pos, const float* d_w, const int32_t* d_topk_ids, int32_t k,
                                int32_t E, uint16_t* d_dy, float* d_dw, float* d_dlogits, hipStream_t stream) {
    if (T < 0 || M < 0 || k < 1 || H < 8 || H % 8 || H > kMaxDim || T > (1 << 22) || M > kMaxRows) return MOE_ERR_SHAPE;
    if (k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    if (d_dlogits) {
        if (E < 1) return MOE_ERR_SHAPE;
        if (E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
        if (!d_w || !d_topk_ids) return MOE_ERR_INVALID_ARG;
    }
    if (T == 0) return MOE_OK;
    const size_t tk = (size_t)T * k * 4;
    const Buf dout{d_dout, b16(T, H)}, y{d_y, b16(M, H)}, pos{d_slot_pos, tk}, w{d_w, tk}, ids{d_topk_ids, tk},
        dy{d_dy, b16(M, H)}, dw{d_dw, tk}, dl{d_dlogits, d_dlogits ? (size_t)T * E * 4 : 0};
    moe_status st = check_present({dout, pos});
    if (st != MOE_OK) return st;
    if (M > 0 && (!d_dy || ((d_dw || d_dlogits) && !d_y))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(d_y) || !aligned16(d_w) || !aligned16(d_topk_ids)) return MOE_ERR_ALIGN;
    if ((st = check_apart({dy, dw, dl}, {dout, y, pos, w, ids})) != MOE_OK) return st;
    return launch_combine_bwd(d_dout, d_y, d_slot_pos, d_w, d_topk_ids, T, M, H, k, E, d_dy, d_dw, d_dlogits, stream);
}

}  // extern "C"
