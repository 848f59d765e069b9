// Backward pass of routing.  The routing weights are the softmax over all
// experts renormalised over the K chosen ones, which is a softmax over the K
// chosen scores, so
//   dl[t, id_k]  = w_k (dw_k - sum_j w_j dw_j)                     (0 for the mean combine)
// To it come the load-balancing loss aux = E sum_e f_e P_e (f_e taken as
// constant) and the z-loss (1/T) sum_t lse_t^2 with their coefficients:
//   dl[t, e] += d_aux E / T p_e (f_e - sum_j f_j p_j) + d_z 2 / T lse_t softmax(l_t)_e
// Then dx[t] = sum_k dx_perm[row(t,k)] + sum_e dl[t,e] W_r[:,e] and
// dW_r = x^T dl.  dl stays fp32 throughout.
#include <algorithm>

#include "../device_common.h"
#include "../launch.h"
#include "gemm_f32.h"

namespace moe {

namespace {

// One wave per token; lane l holds the scores of experts l + 64 j.
template <int MAXV>
__global__ __launch_bounds__(256) void route_dlogits_kernel(int T, int E, int K, int flags, const float* __restrict__ logits,
                                                           const float* __restrict__ bias,
                                                           const int32_t* __restrict__ ids, const float* __restrict__ w,
                                                           const float* __restrict__ dw,
                                                           const int32_t* __restrict__ counts, float d_aux, float d_z,
                                                           float* __restrict__ dl) {
    const int lane = lane_id();
    for (int t = blockIdx.x * 4 + threadIdx.x / kWave; t < T; t += gridDim.x * 4) {
        float g[MAXV];
    #pragma unroll
        for (int j = 0; j < MAXV; ++j) g[j] = 0.0f;
        if (d_aux != 0.0f || d_z != 0.0f) {
            float l[MAXV];
    #pragma unroll
            for (int j = 0; j < MAXV; ++j) {
                const int e = lane + j * kWave;
                l[j] = e < E ? logits[(size_t)t * E + e] : -INFINITY;
            }
            if (d_aux != 0.0f) {
                const bool biased = bias != nullptr && !(flags & MOE_FLAG_BIAS_SELECT_ONLY);
                float p[MAXV], f[MAXV], m = -INFINITY;
    #pragma unroll
                for (int j = 0; j < MAXV; ++j) {
                    const int e = lane + j * kWave;
                    p[j] = biased && e < E ? l[j] + bias[e] : l[j];
                    f[j] = e < E ? (float)counts[e] : 0.0f;
                    m = fmaxf(m, p[j]);
                }
                m = wave_max(m);
                float sum = 0.0f, fp = 0.0f;
    #pragma unroll
                for (int j = 0; j < MAXV; ++j) {
                    p[j] = expf(p[j] - m);
                    sum += p[j];
                    fp = fmaf(p[j], f[j], fp);
                }
                sum = wave_sum(sum);
                fp = wave_sum(fp) / sum;
                const float c = d_aux * (float)E / (float)T / ((float)T * (float)K) / sum;
    #pragma unroll
                for (int j = 0; j < MAXV; ++j) g[j] += c * p[j] * (f[j] - fp);
            }
            if (d_z != 0.0f) {
                float m = -INFINITY;
    #pragma unroll
                for (int j = 0; j < MAXV; ++j) m = fmaxf(m, l[j]);
                m = wave_max(m);
                float sum = 0.0f;
    #pragma unroll
                for (int j = 0; j < MAXV; ++j) {
                    l[j] = expf(l[j] - m);
                    sum += l[j];
                }
                sum = wave_sum(sum);
                const float c = d_z * 2.0f / (float)T * (m + logf(sum)) / sum;
    #pragma unroll
                for (int j = 0; j < MAXV; ++j) g[j] = fmaf(c, l[j], g[j]);
            }
        }
        if (dw != nullptr && !(flags & MOE_FLAG_COMBINE_MEAN)) {
            const bool in = lane < K;
            const int id = in ? ids[(size_t)t * K + lane] : -1;
            const float wk = in ? w[(size_t)t * K + lane] : 0.0f;
            const float dk = in ? dw[(size_t)t * K + lane] : 0.0f;
            const float mean = wave_sum(wk * dk);
            const float v = wk * (dk - mean);
            for (int k = 0; k < K; ++k) {
                const int ek = __shfl(id, k);
                const float vk = __shfl(v, k);
    #pragma unroll
                for (int j = 0; j < MAXV; ++j) g[j] += lane + j * kWave == ek ? vk : 0.0f;
            }
        }
    #pragma unroll
        for (int j = 0; j < MAXV; ++j) {
            const int e = lane + j * kWave;
            if (e < E) dl[(size_t)t * E + e] = g[j];
        }
    }
}

// dx row: the product's sum plus the gradients of the token's grouped rows, slot by slot.
template <typename T>
struct EpiTokenGrad {
    const T* rows;  // may be NULL
    const int32_t* assign_row;
    int K, n;
    T* out;
    __device__ void operator()(int, int, int m, int c, int N, const f32x4 (&v)[2]) const {
        f32x4 sum = v[0];
        if (rows != nullptr)
            for (int k = 0; k < K; ++k) {
                const int r = assign_row[(size_t)m * K + k];
                if ((unsigned)r < (unsigned)n) sum += load_f32x4(rows + (size_t)r * N + c);
            }
        store_f32x4(out + (size_t)m * N + c, sum);
    }
};
struct EpiPart {  // fp32 partial sums [part][M][N]
    float* out;
    int M;
    __device__ void operator()(int part, int, int m, int n, int N, const f32x4 (&v)[2]) const {
        float* o = out + ((size_t)part * M + m) * N + n;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < N) o[j] = v[0][j];
    }
};

// Adds the parts in order.
template <typename T>
__global__ __launch_bounds__(256) void route_dw_reduce_kernel(size_t n, int parts, const float* __restrict__ part,
                                                             T* __restrict__ out) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        float v = part[i];
        for (int p = 1; p < parts; ++p) v += part[(size_t)p * n + i];
        out[i] = from_f32<T>(v);
    }
}

// Parts of the sum over the tokens: enough workgroups for two per compute
// unit, at least 128 tokens each.
int dw_parts(int T, int d, int E) {
    const int tiles = ((d + GM_T - 1) / GM_T) * ((E + GM_T - 1) / GM_T);
    return std::max(1, std::min((512 + tiles - 1) / tiles, (T + 127) / 128));
}

template <typename T, bool VEC>
hipError_t route_products(int n_tok, int d, int E, int K, const T* x, const T* wr, const T* dx_perm,
                          const int32_t* assign_row, const float* dl, T* dx, T* dwr, float* part, hipStream_t s) {
    const unsigned td = (d + GM_T - 1) / GM_T;
    hipError_t err;
    if (dx != nullptr) {
        GemmArgs<float, T> g{{dl, nullptr}, {wr, nullptr}, E, E, 0, 0, d, E, n_tok, 1, RowPlan{}, nullptr};
        gemm_f32_kernel<GM_NT, false, 1, VEC, VEC><<<dim3((n_tok + GM_T - 1) / GM_T, td), 256, 0, s>>>(
            g, EpiTokenGrad<T>{dx_perm, assign_row, K, n_tok * K, dx});
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    if (dwr != nullptr) {
        const int parts = dw_parts(n_tok, d, E);
        GemmArgs<T, float> g{{x, nullptr}, {dl, nullptr}, d, E, 0, d, E, 0, n_tok, 1, RowPlan{}, nullptr};
        gemm_f32_kernel<GM_TN, false, 1, true, VEC><<<dim3((E + GM_T - 1) / GM_T, td, parts), 256, 0, s>>>(
            g, EpiPart{part, d});
        if ((err = hipGetLastError()) != hipSuccess) return err;
        const size_t n = (size_t)d * E;
        route_dw_reduce_kernel<T><<<(unsigned)std::min<size_t>((n + 255) / 256, 4096), 256, 0, s>>>(n, parts, part,
                                                                                                   dwr);
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

size_t route_backward_ws_bytes(int T, int d, int E) {
    return align_up((size_t)dw_parts(T, d, E) * d * E * sizeof(float), 256);
}

hipError_t launch_route_backward(int T, int d, int E, int K, int dtype, int flags, const void* x, const void* wr,
                                 const float* bias, const float* logits, const int32_t* ids, const float* w,
                                 const float* dw, const int32_t* counts, float d_aux, float d_z, const void* dx_perm,
                                 const int32_t* assign_row, float* dl, void* dx, void* dwr, void* ws, hipStream_t s) {
    const unsigned grid = (unsigned)std::min((T + 3) / 4, 1 << 20);
    timer_before(MOE_KERNEL_ROUTE_BACKWARD, s);
    if (E <= kWave)
        route_dlogits_kernel<1><<<grid, 256, 0, s>>>(T, E, K, flags, logits, bias, ids, w, dw, counts, d_aux, d_z, dl);
    else if (E <= 4 * kWave)
        route_dlogits_kernel<4><<<grid, 256, 0, s>>>(T, E, K, flags, logits, bias, ids, w, dw, counts, d_aux, d_z, dl);
    else
        route_dlogits_kernel<16><<<grid, 256, 0, s>>>(T, E, K, flags, logits, bias, ids, w, dw, counts, d_aux, d_z, dl);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    float* part = (float*)ws;
    const bool vec = E % 8 == 0;
    if (dtype == MOE_DTYPE_F32)
        err = vec ? route_products<float, true>(T, d, E, K, (const float*)x, (const float*)wr, (const float*)dx_perm,
                                                assign_row, dl, (float*)dx, (float*)dwr, part, s)
                  : route_products<float, false>(T, d, E, K, (const float*)x, (const float*)wr, (const float*)dx_perm,
                                                 assign_row, dl, (float*)dx, (float*)dwr, part, s);
    else
        err = vec ? route_products<bf16, true>(T, d, E, K, (const bf16*)x, (const bf16*)wr, (const bf16*)dx_perm,
                                               assign_row, dl, (bf16*)dx, (bf16*)dwr, part, s)
                  : route_products<bf16, false>(T, d, E, K, (const bf16*)x, (const bf16*)wr, (const bf16*)dx_perm,
                                                assign_row, dl, (bf16*)dx, (bf16*)dwr, part, s);
    if (err == hipSuccess) timer_after(MOE_KERNEL_ROUTE_BACKWARD, s);
    return err;
}

}  // namespace moe
