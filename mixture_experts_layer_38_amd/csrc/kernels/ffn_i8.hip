// Grouped gated FFN on 8-bit integers.  Rows a (quantised per row to a_q, s_a)
// against weights quantised per output channel (w_q, s_w):
//   g = (sum_k a_q w1_q) s_a s1,  u likewise,  act = bf16(silu(g) u),
//   h = (sum_f act_q w2_q) s_act s2
// The integer sums are exact in 32 bits (at most 65536 * 127 * 127 < 2^31),
// so their order does not matter; scales and the gate are fp32.  act is rounded
// to bf16 before its quantisation because it is an output of the call; that
// rounding (at most 2^-8 of the value) is no larger than the half step, 1 / 254
// of the row's maximum, that the quantisation rounds by.
//
// Decode batches stream the weights (ffn_decode.hip), larger ones use the tiled
// GEMMs (ffn_prefill.hip), whose stages then hold twice the values: Mixtral
// shape, 32 tokens 261 us (bf16 weights: 483), 8192 tokens 2.68 ms, 2150 TOP/s
// over the whole call (bf16: 4.75 ms).
#include "../device_common.h"
#include "../launch.h"
#include "ffn_tiles.h"

namespace moe {

size_t prefill_ws_bytes(int n_rows, int E, int d);
int launch_plan_i8(int n_rows, int E, const int32_t* offsets, void* ws, RowPlan* plan, hipError_t* err, hipStream_t s);
hipError_t launch_prefill_i8(bool gated, int n_rows, int E, int N, int K, int bm, const int8_t* A, const float* rows,
                             const int32_t* rowmap, int topk, const int32_t* offsets, const int8_t* wa,
                             const float* sa, const int8_t* wb, const float* sb, bf16* out, void* ws, hipStream_t s);
hipError_t launch_decode_i8(bool gated, int n_rows, int E, int N, int K, const int8_t* A, const float* rows,
                            const int32_t* rowmap, int topk, const int32_t* offsets, const int8_t* wa, const float* sa,
                            const int8_t* wb, const float* sb, bf16* out, hipStream_t s);

namespace {



constexpr int I8_ALIGN = 128;  // the quantised rows are padded with zeros to whole 128-byte lines
constexpr int I8_BM = 128;     // rows per pass of the kernel below
constexpr int I8_DECODE_TOKENS = 64;  // as the bf16 layer's choice

// Reductions shorter than a stage of the tiled GEMM (16 to 112 values).  One
// wave: 16 weight rows against 128 rows of a row tile at a time, 64 k per step;
// lane l feeds row l % 16 and k (l / 16) * 16 .. + 15 of both operands.
template <bool GATED>
__global__ __launch_bounds__(256) void ffn_i8_kernel(int n_rows, int N, int K, int lda, const int8_t* __restrict__ A,
                                                    const float* __restrict__ sa, const int32_t* __restrict__ rowmap,
                                                    int topk, RowPlan plan, int bm, const int32_t* __restrict__ offsets,
                                                    const int8_t* __restrict__ wa, const float* __restrict__ swa,
                                                    const int8_t* __restrict__ wb, const float* __restrict__ swb,
                                                    bf16* __restrict__ out) {
    constexpr int NG = GATED ? 2 : 1, NB = I8_BM / 16;
    if ((int)blockIdx.x >= *plan.mt_count) return;
    const int e = plan.mt_expert[blockIdx.x] & 0x7FF;
    const int tile0 = plan.mt_row0[blockIdx.x];
    const int row_end = min(offsets[e + 1], n_rows);
    const int lane = lane_id();
    const int n0 = blockIdx.y * 64 + (threadIdx.x / kWave) * 16;
    if (n0 >= N) return;
    const int rl = lane & 15, kg = (lane >> 4) * 16;
    const size_t wrow = (size_t)e * N + n0 + rl;  // N is a multiple of 16
    const int8_t* pw[2] = {wa + wrow * K, GATED ? wb + wrow * K : nullptr};
    for (int row0 = tile0; row0 < min(tile0 + bm, row_end); row0 += I8_BM) {
        const int8_t* pa[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
            pa[b] = A + (size_t)src_row(rowmap, topk, min(row0 + 16 * b + rl, row_end - 1)) * lda;
        i32x4 acc[NG][NB];
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[i][b] = i32x4{0, 0, 0, 0};
        for (int k = kg; k < lda; k += 64) {
            i32x4 w[NG];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const i32x4 zero = {0, 0, 0, 0};
                w[i] = k < K ? *reinterpret_cast<const i32x4*>(pw[i] + k) : zero;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const i32x4 a = *reinterpret_cast<const i32x4*>(pa[b] + k);
#pragma unroll
                for (int i = 0; i < NG; ++i) acc[i][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i], a, acc[i][b], 0, 0, 0);
            }
        }
        // element i of a block: weight row n0 + 4 (lane / 16) + i, grouped row lane % 16
        const int n = n0 + 4 * (lane >> 4);
        const f32x4 s1 = *reinterpret_cast<const f32x4*>(swa + (size_t)e * N + n);
        f32x4 s3 = {0, 0, 0, 0};
        if (GATED) s3 = *reinterpret_cast<const f32x4*>(swb + (size_t)e * N + n);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = row0 + 16 * b + rl;
            if (r >= row_end) continue;
            const float s = sa[src_row(rowmap, topk, r)];
            bf16x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float g = (float)acc[0][b][i] * s * s1[i];
                if constexpr (GATED) v[i] = (bf16)(silu(g) * ((float)acc[1][b][i] * s * s3[i]));
                else v[i] = (bf16)g;
            }
            *reinterpret_cast<bf16x4*>(out + (size_t)r * N + n) = v;
        }
    }
}

struct I8Layout {
    int ldx, ldf;
    size_t xq, xs, aq, as, plan, total;
};
I8Layout i8_layout(int n_x, int n, int E, int d, int F) {
    I8Layout L;
    L.ldx = (int)align_up(d, I8_ALIGN);
    L.ldf = (int)align_up(F, I8_ALIGN);
    L.xq = 0;
    L.xs = L.xq + align_up((size_t)n_x * L.ldx, 256);
    L.aq = L.xs + align_up((size_t)n_x * sizeof(float), 256);
    L.as = L.aq + align_up((size_t)n * L.ldf, 256);
    L.plan = L.as + align_up((size_t)n * sizeof(float), 256);
    L.total = L.plan + prefill_ws_bytes(n, E, d);
    return L;
}

}  // namespace

size_t ffn_i8_ws_bytes(int T, int K, int E, int d, int F, bool by_token) {
    return i8_layout(by_token ? T : T * K, T * K, E, d, F).total;
}

hipError_t launch_ffn_i8(int T, int K, int E, int d, int F, const void* x, const int32_t* rowmap,
                         const int32_t* offsets, const moe_i8_weights& w, void* act, void* h, void* ws, hipStream_t s) {
    const int n = T * K, n_x = rowmap ? T : n;
    const I8Layout L = i8_layout(n_x, n, E, d, F);
    char* base = (char*)ws;
    int8_t *xq = (int8_t*)base + L.xq, *aq = (int8_t*)base + L.aq;
    float *xs = (float*)(base + L.xs), *as = (float*)(base + L.as);
    void* plan_ws = base + L.plan;
    const bool decode = T <= I8_DECODE_TOKENS;
    // the tiled GEMM takes reductions of one whole 128-byte stage or more
    const bool tiled_d = !decode && d >= I8_ALIGN, tiled_f = !decode && F >= I8_ALIGN;
    RowPlan plan;
    int bm = 0;
    hipError_t err = hipSuccess;
    timer_before(MOE_KERNEL_FFN_I8, s);
    if (!decode) bm = launch_plan_i8(n, E, offsets, plan_ws, &plan, &err, s);
    if (err != hipSuccess) return err;
    const unsigned mt = decode ? 0 : (unsigned)row_plan_tiles(n, E, bm);
    // grouped rows past the last group are not read; token rows all are
    err = launch_quantize_rows(n_x, d, L.ldx, tiled_d, MOE_DTYPE_BF16, x, xq, xs, rowmap ? nullptr : offsets + E, s);
    if (err != hipSuccess) return err;
    if (decode) {
        err = launch_decode_i8(true, n, E, F, d, xq, xs, rowmap, K, offsets, w.w1, w.s1, w.w3, w.s3, (bf16*)act, s);
    } else if (tiled_d) {
        err = launch_prefill_i8(true, n, E, F, d, bm, xq, xs, rowmap, K, offsets, w.w1, w.s1, w.w3, w.s3, (bf16*)act,
                                plan_ws, s);
    } else {
        ffn_i8_kernel<true><<<dim3(mt, (F + 63) / 64), 256, 0, s>>>(n, F, d, L.ldx, xq, xs, rowmap, K, plan, bm,
                                                                   offsets, w.w1, w.s1, w.w3, w.s3, (bf16*)act);
        err = hipGetLastError();
    }
    if (err != hipSuccess) return err;
    err = launch_quantize_rows(n, F, L.ldf, tiled_f, MOE_DTYPE_BF16, act, aq, as, offsets + E, s);
    if (err != hipSuccess) return err;
    if (decode) {
        err = launch_decode_i8(false, n, E, d, F, aq, as, nullptr, 1, offsets, w.w2, w.s2, nullptr, nullptr, (bf16*)h, s);
    } else if (tiled_f) {
        err = launch_prefill_i8(false, n, E, d, F, bm, aq, as, nullptr, 1, offsets, w.w2, w.s2, nullptr, nullptr,
                                (bf16*)h, plan_ws, s);
    } else {
        ffn_i8_kernel<false><<<dim3(mt, (d + 63) / 64), 256, 0, s>>>(n, d, F, L.ldf, aq, as, nullptr, 1, plan, bm,
                                                                    offsets, w.w2, w.s2, nullptr, nullptr, (bf16*)h);
        err = hipGetLastError();
    }
    if (err == hipSuccess) timer_after(MOE_KERNEL_FFN_I8, s);
    return err;
}

}  // namespace moe
