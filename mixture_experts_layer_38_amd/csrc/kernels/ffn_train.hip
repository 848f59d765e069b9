// The grouped gated FFN in training: the forward pass that keeps the gate and
// up projections, and the backward pass.  With the rows a of expert e
//   g = W1 a,  u = W3 a,  act = silu(g) u,  h = W2 act
//   da = W2^T dh;  dg, du from da, g, u (gated.h)
//   dx = W1^T dg + W3^T du;  dW1 = sum dg a^T;  dW3 = sum du a^T;  dW2 = sum dh act^T
// g and u are stored in the layer type; act is formed again from them in the
// backward pass (two stored rows of F instead of three).  da stays fp32; dg, du
// and act are rounded to bf16 once, as operands of the matrix instructions: over
// a sum their errors average, and a gradient is off by 1.4 times its own rounding.
//
// Paths of the forward pass in bf16: batches of up to 64 tokens stream the
// weights (ffn_decode.hip); widths that are multiples of 64 take the layer's
// tiled GEMMs with two more stores in the epilogue (ffn_prefill.hip; 8192 tokens,
// Mixtral shape: 4.7 ms, 1220 TFLOP/s); others ffn_train_tiles.hip, which also
// holds the backward pass.  fp32: gemm_f32.h.
#include <algorithm>
#include <type_traits>

#include "../device_common.h"
#include "../launch.h"
#include "ffn_tiles.h"
#include "gated.h"
#include "gemm_f32.h"

namespace moe {

size_t prefill_ws_bytes(int n_rows, int E, int d);
hipError_t launch_ffn_prefill_keep(int n_rows, int E, int d, int F, const bf16* x, const int32_t* offsets,
                                   const bf16* w1, const bf16* w3, const bf16* w2, bf16* gate, bf16* up, bf16* act,
                                   bf16* h, void* ws, hipStream_t s);
size_t ffn_train_tiles_ws_bytes(int n, int E, int d, int F);
hipError_t launch_ffn_train_tiles(int n, int E, int d, int F, const bf16* x, const int32_t* offsets, const bf16* w1,
                                  const bf16* w3, const bf16* w2, bf16* gate, bf16* up, bf16* act, bf16* h, void* ws,
                                  hipStream_t s);
hipError_t launch_decode_keep(int n_rows, int E, int d, int F, const bf16* x, const int32_t* offsets, const bf16* w1,
                              const bf16* w3, const bf16* w2, bf16* gate, bf16* up, bf16* act, bf16* h, hipStream_t s);

size_t ffn_grad_ws_bytes(int n, int E, int d, int F);
hipError_t launch_ffn_grad(int n, int E, int d, int F, const bf16* x, const int32_t* offsets, const bf16* w1,
                           const bf16* w3, const bf16* w2, const bf16* gate, const bf16* up, const bf16* dh, bf16* dx,
                           bf16* dw1, bf16* dw3, bf16* dw2, bf16* dgate, bf16* dup, bf16* act, void* ws,
                           hipStream_t s);

namespace {

// ---- fp32 path -------------------------------------------------------------------
template <typename T>
struct EpiGate {
    T *gate, *up, *act;
    __device__ void operator()(int, int, int m, int n, int N, const f32x4 (&v)[2]) const {
        const size_t i = (size_t)m * N + n;
        store_f32x4(gate + i, v[0]);
        store_f32x4(up + i, v[1]);
        f32x4 a;
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = silu(v[0][j]) * v[1][j];
        store_f32x4(act + i, a);
    }
};
template <typename T>
struct EpiRows {  // C rows are grouped rows
    T* out;
    __device__ void operator()(int, int, int m, int n, int N, const f32x4 (&v)[2]) const {
        store_f32x4(out + (size_t)m * N + n, v[0]);
    }
};
template <typename T>
struct EpiGateGrad {
    const T *gate, *up;
    T *dgate, *dup, *act;
    __device__ void operator()(int, int, int m, int n, int N, const f32x4 (&v)[2]) const {
        const size_t i = (size_t)m * N + n;
        const f32x4 g = load_f32x4(gate + i), u = load_f32x4(up + i);
        f32x4 dg, du, a;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const GatedGrad r = gated_grad(g[j], u[j], v[0][j]);
            dg[j] = r.dg;
            du[j] = r.du;
            a[j] = r.act;
        }
        store_f32x4(dgate + i, dg);
        store_f32x4(dup + i, du);
        store_f32x4(act + i, a);
    }
};
template <typename T>
struct EpiWeights {  // C is one expert's [M][N]
    T *out0, *out1;
    int M;
    __device__ void operator()(int e, int sel, int m, int n, int N, const f32x4 (&v)[2]) const {
        store_f32x4((sel ? out1 : out0) + ((size_t)e * M + m) * N + n, v[0]);
    }
};

// Calls f with the tile for this many rows and columns as a compile-time constant.
template <typename F>
hipError_t with_tile(int tile, F f) {
    return tile == 64 ? f(std::integral_constant<int, 64>{}) : f(std::integral_constant<int, 128>{});
}
template <bool FWD, typename F>
hipError_t with_rows_tile(int tile, F f) {
    if (tile == 32) return f(std::integral_constant<int, 32>{});
    if constexpr (FWD) return f(std::integral_constant<int, 64>{});
    else return with_tile(tile, f);
}
unsigned tiles_of(int v, int tile) { return (unsigned)((v + tile - 1) / tile); }
// Row tiles.  32 where those of 64 would leave compute units idle (64 tokens,
// 8 experts, K 2, d 128, F 256, 22 tiles of 64: the forward pass 13.9 us with 32,
// 19.3 with 64; 256 tokens, d 256, F 512: 20.7 and 34.3; 1024 tokens, d 512, F
// 1024, 328 tiles: 117 and 112).
bool small_tiles(int n, int E, int cols) {
    return E <= GroupTiles::kMax && (long)row_plan_tiles(n, E, 64) * tiles_of(cols, 64) < 256;
}
// The forward pass's: tiles of 128 lose however many there are (8192 tokens, 8
// experts, K 2, d 2048, F 4096: 7.31 ms with 64, 7.71 with 128).
int train_tile(int n, int E, int cols) { return small_tiles(n, E, cols) ? 32 : 64; }
int grad_tile(int n, int E, int cols) {
    return small_tiles(n, E, cols) ? 32 : gm_tile((long)row_plan_tiles(n, E, 128) * tiles_of(cols, 128));
}

template <int LAYOUT, bool DUAL, int SEGS, typename Epi>
hipError_t rows_product(int tile, const GemmArgs<float, float>& g, Epi epi, hipStream_t s) {
    return with_rows_tile<LAYOUT == GM_NT>(tile, [&](auto t) {
        constexpr int T = decltype(t)::value;
        gemm_f32_kernel<T, LAYOUT, DUAL, SEGS, true, true>
            <<<dim3((unsigned)row_plan_tiles(g.n_rows, g.E, T), tiles_of(g.N, T)), 256, 0, s>>>(g, epi);
        return hipGetLastError();
    });
}
hipError_t weight_product(const GemmArgs<float, float>& g, int sels, EpiWeights<float> epi, hipStream_t s) {
    const int tile = gm_tile((long)tiles_of(g.M, 128) * tiles_of(g.N, 128) * g.E * sels);
    return with_tile(tile, [&](auto t) {
        constexpr int T = decltype(t)::value;
        gemm_f32_kernel<T, GM_TN, false, 1, true, true>
            <<<dim3(tiles_of(g.N, T), tiles_of(g.M, T), g.E * sels), 256, 0, s>>>(g, epi);
        return hipGetLastError();
    });
}

// tile: rows of the row tiles, which are the products' tiles too.
hipError_t train_gemms(int n, int E, int d, int F, const float* x, const int32_t* offsets, const float* w1,
                       const float* w3, const float* w2, float* gate, float* up, float* act, float* h, int tile,
                       const RowPlan& plan, hipStream_t s) {
    typedef float T;
    GemmArgs<T, T> g{{x, nullptr}, {w1, w3}, d, d, (size_t)F * d, 0, F, d, n, E, plan, offsets};
    const hipError_t err = rows_product<GM_NT, true, 1>(tile, g, EpiGate<T>{gate, up, act}, s);
    if (err != hipSuccess) return err;
    GemmArgs<T, T> g2{{act, nullptr}, {w2, nullptr}, F, F, (size_t)F * d, 0, d, F, n, E, plan, offsets};
    return rows_product<GM_NT, false, 1>(tile, g2, EpiRows<T>{h}, s);
}

hipError_t backward_gemms(int n, int E, int d, int F, const float* x, const int32_t* offsets, const float* w1,
                          const float* w3, const float* w2, const float* gate, const float* up, const float* dh,
                          float* dx, float* dw1, float* dw3, float* dw2, float* dgate, float* dup, float* act,
                          int tile, const RowPlan& plan, hipStream_t s) {
    typedef float T;
    const size_t ws = (size_t)F * d;
    GemmArgs<T, T> ga{{dh, nullptr}, {w2, nullptr}, d, F, ws, 0, F, d, n, E, plan, offsets};
    hipError_t err = rows_product<GM_NN, false, 1>(tile, ga, EpiGateGrad<T>{gate, up, dgate, dup, act}, s);
    if (err != hipSuccess) return err;
    if (dw2 != nullptr) {
        GemmArgs<T, T> g{{dh, nullptr}, {act, nullptr}, d, F, 0, d, F, 0, n, E, RowPlan{}, offsets};
        if ((err = weight_product(g, 1, EpiWeights<T>{dw2, nullptr, d}, s)) != hipSuccess) return err;
        GemmArgs<T, T> g13{{dgate, dup}, {x, nullptr}, F, d, 0, F, d, 0, n, E, RowPlan{}, offsets};
        if ((err = weight_product(g13, 2, EpiWeights<T>{dw1, dw3, F}, s)) != hipSuccess) return err;
    }
    if (dx != nullptr) {
        GemmArgs<T, T> g{{dgate, dup}, {w1, w3}, F, d, ws, 0, d, F, n, E, plan, offsets};
        err = rows_product<GM_NN, false, 2>(tile, g, EpiRows<T>{dx}, s);
    }
    return err;
}

}  // namespace

// act, then the row plan (bf16: the tiled GEMMs' workspace)
size_t ffn_train_ws_bytes(int T, int K, int E, int d, int F, int dtype) {
    const size_t es = dtype == MOE_DTYPE_F32 ? 4 : 2;
    return align_up((size_t)T * K * F * es, 256) +
           (dtype == MOE_DTYPE_F32 ? row_plan_bytes(T * K, E)
                                   : std::max(ffn_train_tiles_ws_bytes(T * K, E, d, F), prefill_ws_bytes(T * K, E, d)));
}

hipError_t launch_ffn_train(int T, int K, int E, int d, int F, int dtype, const void* x, const int32_t* offsets,
                            const void* w1, const void* w3, const void* w2, void* gate, void* up, void* h, void* ws,
                            hipStream_t s) {
    const int n = T * K;
    const size_t es = dtype == MOE_DTYPE_F32 ? 4 : 2;
    char* base = (char*)ws;
    void* rest = base + align_up((size_t)n * F * es, 256);
    hipError_t err;
    timer_before(MOE_KERNEL_FFN_TRAIN, s);
    if (dtype == MOE_DTYPE_F32) {
        RowPlan plan;
        const int tile = train_tile(n, E, std::min(d, F));
        if (E > GroupTiles::kMax && (err = launch_row_plan(n, E, tile, offsets, rest, &plan, s)) != hipSuccess) return err;
        err = train_gemms(n, E, d, F, (const float*)x, offsets, (const float*)w1, (const float*)w3, (const float*)w2,
                          (float*)gate, (float*)up, (float*)base, (float*)h, tile, plan, s);
    } else if (T <= 64) {  // the forward pass's choice: few rows per expert, bound by the weights
        err = launch_decode_keep(n, E, d, F, (const bf16*)x, offsets, (const bf16*)w1, (const bf16*)w3, (const bf16*)w2,
                                 (bf16*)gate, (bf16*)up, (bf16*)base, (bf16*)h, s);
    } else if (d % 64 != 0 || F % 64 != 0) {
        err = launch_ffn_train_tiles(n, E, d, F, (const bf16*)x, offsets, (const bf16*)w1, (const bf16*)w3,
                                     (const bf16*)w2, (bf16*)gate, (bf16*)up, (bf16*)base, (bf16*)h, rest, s);
    } else {
        err = launch_ffn_prefill_keep(n, E, d, F, (const bf16*)x, offsets, (const bf16*)w1, (const bf16*)w3,
                                      (const bf16*)w2, (bf16*)gate, (bf16*)up, (bf16*)base, (bf16*)h, rest, s);
    }
    if (err == hipSuccess) timer_after(MOE_KERNEL_FFN_TRAIN, s);
    return err;
}

// dgate, dup, act, then the row plan (bf16: and what the weights' products need)
size_t ffn_backward_ws_bytes(int T, int K, int E, int d, int F, int dtype) {
    const size_t es = dtype == MOE_DTYPE_F32 ? 4 : 2;
    return 3 * align_up((size_t)T * K * F * es, 256) +
           (dtype == MOE_DTYPE_F32 ? row_plan_bytes(T * K, E) : ffn_grad_ws_bytes(T * K, E, d, F));
}

hipError_t launch_ffn_backward(int T, int K, int E, int d, int F, int dtype, const void* x, const int32_t* offsets,
                               const void* w1, const void* w3, const void* w2, const void* gate, const void* up,
                               const void* dh, void* dx, void* dw1, void* dw3, void* dw2, void* ws, hipStream_t s) {
    const int n = T * K;
    const size_t es = dtype == MOE_DTYPE_F32 ? 4 : 2;
    const size_t one = align_up((size_t)n * F * es, 256);
    char* base = (char*)ws;
    void *dgate = base, *dup = base + one, *act = base + 2 * one, *rest = base + 3 * one;
    hipError_t err;
    timer_before(MOE_KERNEL_FFN_BACKWARD, s);
    if (dtype == MOE_DTYPE_F32) {
        RowPlan plan;
        const int tile = grad_tile(n, E, std::min(d, F));
        if (E > GroupTiles::kMax && (err = launch_row_plan(n, E, tile, offsets, rest, &plan, s)) != hipSuccess) return err;
        err = backward_gemms(n, E, d, F, (const float*)x, offsets, (const float*)w1, (const float*)w3,
                             (const float*)w2, (const float*)gate, (const float*)up, (const float*)dh, (float*)dx,
                             (float*)dw1, (float*)dw3, (float*)dw2, (float*)dgate, (float*)dup, (float*)act, tile, plan,
                             s);
    } else {
        err = launch_ffn_grad(n, E, d, F, (const bf16*)x, offsets, (const bf16*)w1, (const bf16*)w3, (const bf16*)w2,
                              (const bf16*)gate, (const bf16*)up, (const bf16*)dh, (bf16*)dx, (bf16*)dw1, (bf16*)dw3,
                              (bf16*)dw2, (bf16*)dgate, (bf16*)dup, (bf16*)act, rest, s);
    }
    if (err == hipSuccess) timer_after(MOE_KERNEL_FFN_BACKWARD, s);
    return err;
}

}  // namespace moe
