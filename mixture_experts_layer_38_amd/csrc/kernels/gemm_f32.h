// Grouped matrix products in fp32: square output tiles on the fp32 MFMA
// (v_mfma_f32_32x32x2_f32, exact products, fp32 sums in a fixed order), for
// the fp32 layer and for operands that must not be rounded to bf16.  bf16
// operands are widened on the way into the LDS.
//
//   GM_NT  C[r][n] = sum_k A[r][k] B[n][k]     rows r of one expert's group
//   GM_NN  C[r][n] = sum_k A[r][k] B[k][n]
//   GM_TN  C[m][n] = sum_r A[r][m] B[r][n]     the sum runs over the group's rows
//
// A workgroup of four waves (2 x 2) owns a tile of 64, of which more fit on a
// compute unit and hide each other's loads, or of 128, with half the LDS reads
// per MFMA, once there are many.  A tile of 32 is for few: each wave multiplies
// all of it over its own quarter of a step's k, and the four sums are joined in
// order at the end, so the chain of MFMAs is a quarter as long and four times
// as many workgroups run.
// Operands go through registers (the next k step is loaded while the present
// one is multiplied) into LDS tiles [k][row], padded so that the
// column reads of the MFMA operands and the transposing writes fall in
// distinct banks.
#pragma once

#include "../device_common.h"
#include "ffn_tiles.h"

namespace moe {

constexpr int GM_K = 32;  // k per step
// The tile for a launch of `tiles` tiles of 128 (FFN backward, 16384 rows, 8
// experts: d 1024, F 2048, 512 to 1024 tiles a product: 3.84 ms with 64, 4.00
// with 128 where the sum is over k, 3.68 where it is over rows; d 2048, F 4096,
// 2048 tiles: 15.38, 14.75 and 14.74 ms).
inline int gm_tile(long tiles) { return tiles < 1536 ? 64 : 128; }
enum { GM_NT, GM_NN, GM_TN };

// One product of every group.  a[1], b[1]: the second factor pair where the
// kernel takes two (DUAL: two products of the same rows; SEGS = 2: the sum of
// two products; GM_TN: the second half of the grid's z takes a[1]).
template <typename TA, typename TB>
struct GemmArgs {
    const TA* a[2];
    const TB* b[2];
    int lda, ldb;
    size_t b_stride;  // elements from one expert's B to the next's (GM_NT, GM_NN)
    int M, N, K;      // GM_TN: C is [M][N]; else K is the reduction length
    int n_rows;       // grouped rows
    int E;            // experts (GM_TN: the grid's z counts them, once or twice)
    RowPlan plan;     // row tiles of the groups (mt_count NULL: up to 64 experts, see GroupTiles)
    const int32_t* offsets;  // NULL: one group of n_rows rows; GM_TN then cuts it into gridDim.z parts
};

// Eight consecutive elements of a row as floats; zeros past `left` elements.
template <typename T, bool VEC>
__device__ __forceinline__ void gm_load8(float (&r)[8], const T* p, int left) {
    if (VEC) {  // left is at most 0 or at least 8
        if (left > 0) {
            if constexpr (sizeof(T) == 4) {
                const f32x4 u = *reinterpret_cast<const f32x4*>(p);
                const f32x4 v = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    r[j] = u[j];
                    r[4 + j] = v[j];
                }
            } else {
                const bf16x8 u = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = (float)u[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = 0.0f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = j < left ? to_f32(p[j]) : 0.0f;
    }
}

// VA, VB: rows of A (B) are whole 8-element vectors.  Epi: called as
// epi(e, sel, m, n, N, v) for four consecutive columns n .. n + 3 of row m
// (grouped row, or A's column for GM_TN) with the sums v[0] (and v[1] of the
// second product).
template <int GM_T, int LAYOUT, bool DUAL, int SEGS, bool VA, bool VB, typename TA, typename TB, typename Epi>
__global__ __launch_bounds__(256) void gemm_f32_kernel(GemmArgs<TA, TB> g, Epi epi) {
    constexpr int NB = DUAL ? 2 : 1;
    constexpr bool KSPLIT = GM_T == 32;          // each wave the whole tile, over a quarter of a step's k
    constexpr int SK = KSPLIT ? 4 * GM_K : GM_K;  // k per step
    // padded LDS rows (floats); a tile of 32 that is written column by column
    // takes an odd row, else the writes of all k would share a bank
    constexpr int LA = KSPLIT && LAYOUT != GM_TN ? 33 : GM_T + 4;
    constexpr int LB = KSPLIT && LAYOUT == GM_NT ? 33 : GM_T + 4;
    constexpr int GM_H = GM_T * SK / 8 / 256;    // 8-element vectors per thread and operand
    constexpr int BL = KSPLIT ? 1 : GM_T / 64;   // 32 x 32 blocks per wave and side
    static_assert(!KSPLIT || 4 * GM_T * GM_T * NB <= SK * (LA + NB * LB), "the waves' sums fit the operands' LDS");
    __shared__ __align__(16) float lds[SK * (LA + NB * LB)];
    float(*const sA)[LA] = reinterpret_cast<float(*)[LA]>(lds);
    float(*const sB)[LB] = reinterpret_cast<float(*)[LB]>(lds + SK * LA);  // product i: rows SK i on
    const int tid = threadIdx.x;
    const int lane = lane_id();
    const int wave = tid / kWave;
    // row tiles lie along x, which alone may pass 65535
    const int n0 = (LAYOUT == GM_TN ? blockIdx.x : blockIdx.y) * GM_T;
    int e = 0, sel = 0, m0, m_end, k_beg = 0, k_end = g.K;
    if constexpr (LAYOUT == GM_TN) {
        m0 = blockIdx.y * GM_T;
        m_end = g.M;
        if (g.offsets != nullptr) {
            e = blockIdx.z % g.E;
            sel = blockIdx.z / g.E;
            k_beg = min(max(g.offsets[e], 0), g.n_rows);
            k_end = min(g.offsets[e + 1], g.n_rows);
        } else {
            e = blockIdx.z;
            k_beg = (int)((long long)g.n_rows * e / gridDim.z);
            k_end = (int)((long long)g.n_rows * (e + 1) / gridDim.z);
        }
    } else if (g.offsets != nullptr) {
        const GroupTiles gt(g.plan, g.E, GM_T, g.offsets);
        if ((int)blockIdx.x >= gt.count) return;
        gt.rows(blockIdx.x, e, m0);
        m_end = min(g.offsets[e + 1], g.n_rows);
    } else {
        m0 = blockIdx.x * GM_T;
        m_end = g.n_rows;
    }

    // a [rows][k] tile: row (and every KR on) and first k of this thread
    constexpr int KT = SK / 8, KR = 256 / KT;
    const int kr = tid / KT, kc = (tid % KT) * 8;
    // a [k][columns] tile: k (and every SR on) and first column
    constexpr int ST = GM_T / 8, SR = 256 / ST;
    const int sr = tid / ST, sc = (tid % ST) * 8;
    float ra[GM_H][8], rb[NB][GM_H][8];
    auto load = [&](int seg, int k0) {
        const TA* A = g.a[LAYOUT == GM_TN ? sel : seg];
#pragma unroll
        for (int h = 0; h < GM_H; ++h) {
            if constexpr (LAYOUT == GM_TN) {
                const int r = k0 + sr + SR * h;
                gm_load8<TA, VA>(ra[h], A + (size_t)r * g.lda + m0 + sc, r < k_end ? g.M - m0 - sc : 0);
            } else {
                const int r = m0 + kr + KR * h;
                gm_load8<TA, VA>(ra[h], A + (size_t)r * g.lda + k0 + kc, r < m_end ? k_end - k0 - kc : 0);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const TB* B = g.b[DUAL ? i : (LAYOUT == GM_TN ? 0 : seg)];
                if constexpr (LAYOUT == GM_NT) {
                    const int r = n0 + kr + KR * h;
                    gm_load8<TB, VB>(rb[i][h], B + e * g.b_stride + (size_t)r * g.ldb + k0 + kc,
                                     r < g.N ? k_end - k0 - kc : 0);
                } else {
                    const int r = k0 + sr + SR * h;
                    gm_load8<TB, VB>(rb[i][h],
                                     B + (LAYOUT == GM_TN ? 0 : e * g.b_stride) + (size_t)r * g.ldb + n0 + sc,
                                     r < k_end ? g.N - n0 - sc : 0);
                }
            }
        }
    };
    auto store_rows = [&](auto s, const float (&r)[GM_H][8]) {
#pragma unroll
        for (int h = 0; h < GM_H; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[kc + j][kr + KR * h] = r[h][j];
    };
    auto store_cols = [&](auto s, const float (&r)[GM_H][8]) {
#pragma unroll
        for (int h = 0; h < GM_H; ++h) {
            *reinterpret_cast<f32x4*>(&s[sr + SR * h][sc]) = f32x4{r[h][0], r[h][1], r[h][2], r[h][3]};
            *reinterpret_cast<f32x4*>(&s[sr + SR * h][sc + 4]) = f32x4{r[h][4], r[h][5], r[h][6], r[h][7]};
        }
    };

    const int wm = KSPLIT ? 0 : (wave & 1) * (GM_T / 2), wn = KSPLIT ? 0 : (wave >> 1) * (GM_T / 2);
    const int wk = KSPLIT ? wave * GM_K : 0;
    const int fr = lane & 31, fk = lane >> 5;
    f32x16 acc[NB][BL][BL];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int a = 0; a < BL; ++a)
#pragma unroll
            for (int b = 0; b < BL; ++b)
#pragma unroll
                for (int q = 0; q < 16; ++q) acc[i][a][b][q] = 0.0f;

    const int per = (k_end - k_beg + SK - 1) / SK;  // steps of one segment
    const int steps = per * SEGS;
    if (steps > 0) load(0, k_beg);
    for (int st = 0; st < steps; ++st) {
        __syncthreads();
        if constexpr (LAYOUT == GM_TN) store_cols(sA, ra);
        else store_rows(sA, ra);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if constexpr (LAYOUT == GM_NT) store_rows(sB + SK * i, rb[i]);
            else store_cols(sB + SK * i, rb[i]);
        }
        __syncthreads();
        if (st + 1 < steps) {
            const int seg = SEGS > 1 && st + 1 >= per ? 1 : 0;
            load(seg, k_beg + (st + 1 - seg * per) * SK);
        }
#pragma unroll
        for (int k = 0; k < GM_K; k += 2) {
            float a[BL];
#pragma unroll
            for (int mb = 0; mb < BL; ++mb) a[mb] = sA[wk + k + fk][wm + mb * 32 + fr];
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int nb = 0; nb < BL; ++nb) {
                    const float b = sB[SK * i + wk + k + fk][wn + nb * 32 + fr];
#pragma unroll
                    for (int mb = 0; mb < BL; ++mb)
                        acc[i][nb][mb] = __builtin_amdgcn_mfma_f32_32x32x2f32(b, a[mb], acc[i][nb][mb], 0, 0, 0);
                }
        }
    }
    // element i of block (nb, mb): column 8 (i / 4) + 4 (lane / 32) + i % 4, row lane % 32
    if constexpr (KSPLIT) {  // wave q joins the four sums of elements 4 q .. 4 q + 3 and hands them on
        f32x4* const sum = reinterpret_cast<f32x4*>(lds);  // [product][wave][q][lane]
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                sum[((i * 4 + wave) * 4 + q) * kWave + lane] = f32x4{acc[i][0][0][4 * q], acc[i][0][0][4 * q + 1], acc[i][0][0][4 * q + 2],
                                              acc[i][0][0][4 * q + 3]};
        __syncthreads();
        const int m = m0 + fr, n = n0 + 8 * wave + 4 * fk;
        if (m >= m_end || n >= g.N) return;
        f32x4 v[2];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            f32x4 t = sum[(i * 16 + wave) * kWave + lane];
#pragma unroll
            for (int w = 1; w < 4; ++w) {
                const f32x4 u = sum[((i * 4 + w) * 4 + wave) * kWave + lane];
#pragma unroll
                for (int j = 0; j < 4; ++j) t[j] += u[j];
            }
            v[i] = t;
        }
        epi(e, sel, m, n, g.N, v);
        return;
    }
#pragma unroll
    for (int mb = 0; mb < BL; ++mb) {
        const int m = m0 + wm + mb * 32 + fr;
        if (m >= m_end) continue;
#pragma unroll
        for (int nb = 0; nb < BL; ++nb)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = n0 + wn + nb * 32 + 8 * q + 4 * fk;
                f32x4 v[2];
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    v[i] = f32x4{acc[i][nb][mb][4 * q], acc[i][nb][mb][4 * q + 1], acc[i][nb][mb][4 * q + 2],
                                 acc[i][nb][mb][4 * q + 3]};
                if (n < g.N) epi(e, sel, m, n, g.N, v);
            }
    }
}

// Four consecutive elements of a row (16-byte fp32 or 8-byte bf16 accesses).
template <typename T> struct Vec4;
template <> struct Vec4<float> { typedef f32x4 type; };
template <> struct Vec4<bf16> { typedef bf16x4 type; };
template <typename T>
__device__ __forceinline__ f32x4 load_f32x4(const T* p) {
    const typename Vec4<T>::type v = *reinterpret_cast<const typename Vec4<T>::type*>(p);
    return f32x4{to_f32(v[0]), to_f32(v[1]), to_f32(v[2]), to_f32(v[3])};
}
template <typename T>
__device__ __forceinline__ void store_f32x4(T* p, f32x4 v) {
    *reinterpret_cast<typename Vec4<T>::type*>(p) =
        typename Vec4<T>::type{from_f32<T>(v[0]), from_f32<T>(v[1]), from_f32<T>(v[2]), from_f32<T>(v[3])};
}

}  // namespace moe
