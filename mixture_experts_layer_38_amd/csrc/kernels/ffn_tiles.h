// Pieces of the tiled expert-GEMM kernels (ffn_prefill.hip): the
// XCD-partitioned, expert-grouped tile order, the swizzle of 128-byte LDS tile
// rows, and explicit wait counts.
#pragma once

#include <type_traits>

#include "../device_common.h"

namespace moe {

constexpr int PF_GM = 8;   // row tiles per group in the tile order
constexpr int PF_XCD = 8;  // XCDs: workgroup b runs on XCD b % 8

// Swizzle of the eight 16-byte chunks of a 128-byte tile row: row r keeps
// chunk c in slot c ^ pf_swz(r), so fragment reads of consecutive rows (one
// chunk each) fall in distinct banks.
__device__ __forceinline__ int pf_swz(int r) { return (r ^ (r >> 3)) & 7; }

// s_waitcnt immediate: vmcnt <= n, no wait on the other counters.
#define PF_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | (15 << 8) | ((((n) >> 4) & 3) << 14))
// s_waitcnt immediate: lgkmcnt == 0, no wait on the other counters.
#define PF_WAIT_LGKM0() __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14))

// The 32 bits of an accumulator element as a float (for stores that move both kinds).
__device__ __forceinline__ float pf_bits(float v) { return v; }
__device__ __forceinline__ float pf_bits(int v) { return __builtin_bit_cast(float, v); }

// v itself, passed through an empty asm statement (no instruction): the
// compiler keeps it after the memory operations issued before it, so a load
// whose value goes through it is waited for only here.
__device__ __forceinline__ int pf_opaque_v(int v) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(v));
#endif
    return v;
}

// The lane index, computed anew at this point: the compiler cannot reuse an
// earlier copy (which it would keep in a register across the main loop).
__device__ __forceinline__ int pf_lane_fresh() {
    int v = 0;
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(v));
#endif
    return v;
}

// The tiled kernel's per-wave block counts, encoded in one compile-time
// value v: v < PF_HT, 4 weight blocks x v token blocks (32 rows each) per
// wave (the 2 x 2 layout); v = PF_HT + n, the 1 x 4 layout's 2 weight blocks
// x n token blocks, in which a stage loads only the tile's first n token
// blocks (load instruction j fills token rows [32 j, 32 j + 32)).
constexpr int PF_HT = 16;
__host__ __device__ constexpr int pf_tblocks(int v) { return v >= PF_HT ? v - PF_HT : v; }
__host__ __device__ constexpr int pf_wblocks(int v) { return v >= PF_HT ? 2 : 4; }
__host__ __device__ constexpr int pf_aloads(int v, int nja) { return v >= PF_HT ? v - PF_HT : nja; }

// Tile t of the grouped order: row tile mt (of expert e, rows [row0, row_end))
// and weight tile nt.  A group of g row tiles starting at row tile m0 owns
// tiles [m0 n_nt, (m0 + g) n_nt), row tile fastest, so tile t lies in the
// group of row tile t / n_nt.
struct PfTile {
    int mt, nt, e, row0, row_end;
};
__device__ __forceinline__ PfTile pf_tile(int t, int n_mt, int n_nt, const int32_t* mt_expert,
                                          const int32_t* mt_row0, const int32_t* offsets, int n_rows) {
    PfTile r;
    const int m = t / n_nt;
    const int v = mt_expert[m];
    const int gsize = ((v >> 11) & 7) + 1;
    const int first = m - ((v >> 14) & 7);
    const int rem = t - first * n_nt;
    r.mt = first + rem % gsize;
    r.nt = rem / gsize;
    r.e = mt_expert[r.mt] & 0x7FF;
    r.row0 = mt_row0[r.mt];
    r.row_end = min(offsets[r.e + 1], n_rows);
    return r;
}

// Row tiles the plan may produce for n_rows grouped rows over E experts (tiles
// of at least 128 rows, one partial tile per expert).
int prefill_max_mtiles(int n_rows, int E);

// Row tiles of every expert's group, bm rows each (an expert's last one partly
// filled), in device memory: *mt_count tiles, packed as ffn_plan_kernel says.
struct RowPlan {
    const int32_t *mt_count = nullptr, *mt_expert = nullptr, *mt_row0 = nullptr;
};
// The row tiles of the groups as a wave sees them: from a plan, or, for up to
// 64 experts, found by the wave itself from the group offsets (lane e holds
// expert e), which saves a launch and the chain of loads through the plan.  The
// order is the plan's: an expert's tiles in groups of at most PF_GM, of balanced
// sizes, the groups of one expert after another.
struct GroupTiles {
    static constexpr int kMax = kWave;
    RowPlan plan;
    const int32_t* offsets;
    int bm, count;
    int beg = 0, nt = 0, incl = 0;  // lane e: first row, tiles, tiles up to and with expert e
    __device__ GroupTiles(const RowPlan& p, int E, int bm_, const int32_t* offs) : plan(p), offsets(offs), bm(bm_) {
        if (plan.mt_count != nullptr) {
            count = *plan.mt_count;
            return;
        }
        const int e = lane_id();
        beg = e < E ? offs[e] : 0;
        nt = e < E ? (max(offs[e + 1] - beg, 0) + bm - 1) / bm : 0;
        incl = nt;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const int v = __shfl_up(incl, o);
            if (e >= o) incl += v;
        }
        count = __builtin_amdgcn_readlane(incl, kWave - 1);
    }
    // Row tile m (< count) of the list: expert, its tiles before m and all of them.
    __device__ void find(int m, int& e, int& j, int& n) const {
        e = __popcll(__ballot(incl <= m));
        n = __builtin_amdgcn_readlane(nt, e);
        j = m - (__builtin_amdgcn_readlane(incl, e) - n);
    }
    // The same tile's expert and first row.
    __device__ void rows(int m, int& e, int& row0) const {
        if (plan.mt_count != nullptr) {
            e = plan.mt_expert[m] & 0x7FF;
            row0 = plan.mt_row0[m];
            return;
        }
        int j, n;
        find(m, e, j, n);
        row0 = __builtin_amdgcn_readlane(beg, e) + j * bm;
    }
    __device__ PfTile tile(int t, int n_nt, int n_rows) const {
        if (plan.mt_count != nullptr) return pf_tile(t, count, n_nt, plan.mt_expert, plan.mt_row0, offsets, n_rows);
        PfTile r;
        const int m = __builtin_amdgcn_readfirstlane(t / n_nt);
        int j, n;
        find(m, r.e, j, n);
        const int ng = (n + PF_GM - 1) / PF_GM, base = n / ng, extra = n % ng;
        const int big = extra * (base + 1);  // group g: base + (g < extra) tiles
        const int g = j < big ? j / (base + 1) : extra + (j - big) / base;
        const int gsize = base + (g < extra ? 1 : 0), first = g * base + min(g, extra);
        const int rem = t - (m - j + first) * n_nt;
        r.mt = m - j + first + rem % gsize;
        r.nt = rem / gsize;
        r.row0 = __builtin_amdgcn_readlane(beg, r.e) + (first + rem % gsize) * bm;
        r.row_end = min(offsets[r.e + 1], n_rows);
        return r;
    }
};

// What a variant of the expert-GEMM kernels takes beyond the layer's forward
// pass:
// PfKeep (gate/up GEMM of the training pass): both projections are stored too,
// rounded to bf16; PfScales (8-bit rows and weights): sums of int8 products in
// int32, scaled by the row's and the weight row's factor in the epilogue.
struct PfKeep {
    bf16 *gate, *up;
};
struct PfScales {
    const float *rows, *wa, *wb;
};
template <typename... X>
constexpr bool pf_keeps = (std::is_same<X, PfKeep>::value || ...);
template <typename... X>
constexpr bool pf_int8 = (std::is_same<X, PfScales>::value || ...);
// The extra argument of type T (T() when the variant has none).
template <typename T>
__device__ __forceinline__ T pf_extra() {
    return T{};
}
template <typename T, typename X>
__device__ __forceinline__ T pf_extra(X x) {
    if constexpr (std::is_same<T, X>::value) return x;
    else return T{};
}

// Most row tiles there can be (the plan's grid bound).
inline int row_plan_tiles(int n_rows, int E, int bm) { return n_rows / bm + E + 1; }
size_t row_plan_bytes(int n_rows, int E);
hipError_t launch_row_plan(int n_rows, int E, int bm, const int32_t* offsets, void* ws, RowPlan* plan, hipStream_t s);

}  // namespace moe
