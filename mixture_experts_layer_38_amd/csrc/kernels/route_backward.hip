// Backward pass of routing.  The routing weights are the softmax over all
// experts renormalised over the K chosen ones, which is a softmax over the K
// chosen scores, so
//   dl[t, id_k]  = w_k (dw_k - sum_j w_j dw_j)                     (0 for the mean combine)
// To it come the load-balancing loss aux = E sum_e f_e P_e (f_e taken as
// constant) and the z-loss (1/T) sum_t lse_t^2 with their coefficients:
//   dl[t, e] += d_aux E / T p_e (f_e - sum_j f_j p_j) + d_z 2 / T lse_t softmax(l_t)_e
// Then dx[t] = sum_k dx_perm[row(t,k)] + sum_e dl[t,e] W_r[:,e] and
// dW_r = x^T dl.  dl stays fp32 throughout.
//
// Bound by memory where tokens are many: 4096 tokens, 256 experts, eight slots,
// d 7168 in bf16 take 202 us: scores 9, dx 128 (0.59 GB, 4.6 TB/s), dW_r 56 and
// the sum of its four parts 6.
#include <algorithm>
#include <type_traits>

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

struct EpiProduct {  // fp32 rows of the product
    float* out;
    __device__ void operator()(int, int, int m, int n, int N, const f32x4 (&v)[2]) const {
        store_f32x4(out + (size_t)m * N + n, v[0]);
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

// Adds the parts in order (n is a multiple of 8).
template <typename T>
__global__ __launch_bounds__(256) void route_dw_reduce_kernel(size_t n, int parts, const float* __restrict__ part,
                                                             T* __restrict__ out) {
    for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (size_t)gridDim.x * 1024) {
        f32x4 v = *reinterpret_cast<const f32x4*>(part + i);
        for (int p = 1; p < parts; ++p) v += *reinterpret_cast<const f32x4*>(part + (size_t)p * n + i);
        store_f32x4(out + i, v);
    }
}

// Eight columns (from c on) of the sum of a token's grouped rows, slot by slot, added to v.
template <typename T>
__device__ __forceinline__ void add_rows(float (&v)[8], const T* rows, const int32_t* slots, int K, int n, int d, int c) {
    constexpr int KC = 8;  // rows whose loads go out together
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int k0 = 0; k0 < K; k0 += KC) {
        int r[KC];
        T x[KC][8];
#pragma unroll
        for (int k = 0; k < KC; ++k) r[k] = k0 + k < K ? slots[k0 + k] : -1;
#pragma unroll
        for (int k = 0; k < KC; ++k)
            if ((unsigned)r[k] < (unsigned)n) __builtin_memcpy(x[k], rows + (size_t)r[k] * d + c, sizeof x[k]);
#pragma unroll
        for (int k = 0; k < KC; ++k)
            if ((unsigned)r[k] < (unsigned)n)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += to_f32(x[k][j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += sum[j];
}

// fp32 layer: adds the grouped rows to the product in dx.
__global__ __launch_bounds__(256) void route_add_rows_kernel(int T, int K, int d, const float* __restrict__ rows,
                                                            const int32_t* __restrict__ assign_row,
                                                            float* __restrict__ dx) {
    const size_t per = d / 8, total = (size_t)T * per;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)gridDim.x * 256) {
        const int t = (int)(i / per), c = (int)(i - (size_t)t * per) * 8;
        float* o = dx + (size_t)t * d + c;
        float v[8];
        __builtin_memcpy(v, o, sizeof v);
        add_rows(v, rows, assign_row + (size_t)t * K, K, T * K, d, c);
        __builtin_memcpy(o, v, sizeof v);
    }
}

// ---- bf16: products on the bf16 MFMAs ------------------------------------------
// An fp32 score gradient enters as two bf16 values, hi = bf16(v) and lo =
// bf16(v - hi), each rounding at most 2^-8 of what it rounds, so the product with
// exact bf16 factors is off by at most 2^-16 of its terms, a 256th of the result's
// own rounding.
__device__ __forceinline__ void split8(const float (&v)[8], bf16x8& hi, bf16x8& lo) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        hi[j] = (bf16)v[j];
        lo[j] = (bf16)(v[j] - (float)hi[j]);
    }
}
// Elements [e, e + 8) of a row of E: one vector each where E is a multiple of 8.
template <bool VEC>
__device__ __forceinline__ void load_scores(float (&v)[8], const float* row, int e, int E, bool on) {
    gm_load8<float, VEC>(v, row + e, on ? E - e : 0);
}
template <bool VEC>
__device__ __forceinline__ bf16x8 load_weights(const bf16* row, int e, int E) {
    bf16x8 r;
    if (VEC) {
        const u32x4 z = {0, 0, 0, 0};
        r = as_bf16x8(e < E ? load16(row + e) : z);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = e + j < E ? row[e + j] : (bf16)0.0f;
    }
    return r;
}

// dx: a workgroup owns 64 tokens x 128 columns.  The score gradients pass
// through the LDS (64 experts at a time, split), the router weights come
// straight from cache; the products then lie in the LDS as fp32 rows (chunks
// swizzled by row), to which each wave adds the tokens' grouped rows, whole
// lines at a time.  Bound by those rows (T K d elements); their loads are in
// flight while the products run (after them: 183 us instead of 133).
constexpr int RX_K = 8;  // grouped rows of a token whose loads go out together
constexpr int RX_T = 64, RX_C = 128, RX_E = 64, RX_LD = RX_E + 8;
template <bool VEC>
__global__ __launch_bounds__(256) void route_dx_kernel(int T, int d, int E, int K, const float* __restrict__ dl,
                                                      const bf16* __restrict__ wr, const bf16* __restrict__ rows,
                                                      const int32_t* __restrict__ assign_row, bf16* __restrict__ dx) {
    __shared__ __align__(16) float sP[RX_T * RX_C];
    __shared__ int32_t sRow[RX_T * 32];  // the tokens' grouped rows (K is at most 32)
    bf16* const sH = reinterpret_cast<bf16*>(sP);  // before sP is filled
    bf16* const sL = sH + RX_T * RX_LD;
    // column tiles first: the tokens' grouped rows are read whole at about the
    // same time (token tiles first, in pieces of 256 bytes, took 190 us
    // instead of 183)
    const unsigned tc = (d + RX_C - 1) / RX_C;
    const int t0 = blockIdx.x / tc * RX_T, c0 = blockIdx.x % tc * RX_C;
    const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
    if (rows != nullptr)
        for (int i = tid; i < RX_T * K; i += 256)
            sRow[i] = t0 + i / K < T ? assign_row[(size_t)t0 * K + i] : -1;
    const int fr = lane & 31, fk = (lane >> 5) * 8;
    f32x16 acc[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[b][i] = 0.0f;
    const int lr = tid >> 2, lc = (tid & 3) * 16;  // row and first column of this thread's part of a chunk
    const bf16* wrow = wr + (size_t)min(c0 + wave * 32 + fr, d - 1) * E;
    const bool on = t0 + lr < T;
    const float* drow = dl + (size_t)min(t0 + lr, T - 1) * E;
    bf16x8 w[4];
    float v[2][8];
    auto load = [&](int e0) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) w[ks] = load_weights<VEC>(wrow, e0 + ks * 16 + fk, E);
#pragma unroll
        for (int h = 0; h < 2; ++h) load_scores<VEC>(v[h], drow, e0 + lc + 8 * h, E, on);
    };
    // the wave's 16 tokens, four at a time; the lane's eight columns
    const int c = c0 + (lane & 15) * 8, cc = min(c, d - 8);
    const int n = T * K;
    u32x4 raw[2][RX_K];
    uint32_t own[2];  // which of raw are the token's
    auto fetch = [&](int i) {
        const int32_t* slots = sRow + (wave * (RX_T / 4) + 4 * i + (lane >> 4)) * K;
        own[i & 1] = 0;
#pragma unroll
        for (int k = 0; k < RX_K; ++k) {
            const int r = k < K ? slots[k] : -1;
            const bool in = (unsigned)r < (unsigned)n;
            own[i & 1] |= in ? 1u << k : 0u;
            // not read again: past the caches, which keep the score gradients (4096
            // tokens, 256 experts: 220 -> 210 us for the backward pass)
            const bf16* p = rows + (size_t)(in ? r : 0) * d + cc;  // (row 0 is never added then)
            raw[i & 1][k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
        }
    };
    float sum[RX_T / 16][8];
    auto add = [&](int i, float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll
        for (int k = 0; k < RX_K; ++k) {
            const bf16x8 x = as_bf16x8(raw[i & 1][k]);
            if (own[i & 1] >> k & 1)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += (float)x[j];
        }
        if (K > RX_K)
            add_rows(v, rows, sRow + (wave * (RX_T / 4) + 4 * i + (lane >> 4)) * K + RX_K, K - RX_K, n, d, cc);
    };
    auto chunk = [&](int e0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8 hi, lo;
            split8(v[h], hi, lo);
            *reinterpret_cast<bf16x8*>(sH + lr * RX_LD + lc + 8 * h) = hi;
            *reinterpret_cast<bf16x8*>(sL + lr * RX_LD + lc + 8 * h) = lo;
        }
        bf16x8 cw[4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) cw[ks] = w[ks];
        __syncthreads();
        if (e0 + RX_E < E) load(e0 + RX_E);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            if (e0 + ks * 16 < E)
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    const bf16x8 hi = *reinterpret_cast<const bf16x8*>(sH + (tb * 32 + fr) * RX_LD + ks * 16 + fk);
                    const bf16x8 lo = *reinterpret_cast<const bf16x8*>(sL + (tb * 32 + fr) * RX_LD + ks * 16 + fk);
                    acc[tb] = mfma32(cw[ks], hi, acc[tb]);
                    acc[tb] = mfma32(cw[ks], lo, acc[tb]);
                }
        __syncthreads();
    };
    load(0);
    if (rows != nullptr) {
        __syncthreads();  // sRow
        // the next fetch and a chunk of experts under each fetch's latency
        fetch(0);
#pragma unroll
        for (int i = 0; i < RX_T / 16; ++i) {
            if (i + 1 < RX_T / 16) fetch(i + 1);
            if (i * RX_E < E) chunk(i * RX_E);
            add(i, sum[i]);
        }
    }
    for (int e0 = rows != nullptr ? RX_T / 16 * RX_E : 0; e0 < E; e0 += RX_E) chunk(e0);
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int ch = wave * 8 + 2 * q + (lane >> 5), t = tb * 32 + fr;
            *reinterpret_cast<f32x4*>(sP + t * RX_C + ((ch ^ (t & 31)) << 2)) =
                f32x4{acc[tb][4 * q], acc[tb][4 * q + 1], acc[tb][4 * q + 2], acc[tb][4 * q + 3]};
        }
    __syncthreads();
    const int ch = 2 * (lane & 15);
    if (c >= d) return;
#pragma unroll
    for (int i = 0; i < RX_T / 16; ++i) {
        const int tl = wave * (RX_T / 4) + 4 * i + (lane >> 4), t = t0 + tl;
        if (t >= T) break;
        const f32x4 a = *reinterpret_cast<const f32x4*>(sP + tl * RX_C + ((ch ^ (tl & 31)) << 2));
        const f32x4 b = *reinterpret_cast<const f32x4*>(sP + tl * RX_C + (((ch + 1) ^ (tl & 31)) << 2));
        const float p[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        bf16x8 o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = (bf16)(rows != nullptr ? sum[i][j] + p[j] : p[j]);
        *reinterpret_cast<bf16x8*>(dx + (size_t)t * d + c) = o;
    }
}

// dW_r: a workgroup owns 128 columns of x x 128 experts over one part of the
// tokens, 64 tokens a step (the next step's loads in flight meanwhile: with 32
// each step waited for them, 74 us).  Both operands lie across the reduction: LDS rows
// [token][column] with the chunk swizzle and transposing reads of the FFN's
// weight gradients; the score gradients are split on the way in.
constexpr int RW_T = 128, RW_K = 64, RW_H = RW_K / 16;
template <bool VEC>
__global__ __launch_bounds__(256) void route_dw_kernel(int T, int d, int E, const bf16* __restrict__ x,
                                                      const float* __restrict__ dl, float* __restrict__ part,
                                                      bf16* __restrict__ out) {
    __shared__ __align__(16) bf16 sX[RW_K * RW_T], sH[RW_K * RW_T], sL[RW_K * RW_T];
    const int e0 = blockIdx.x * RW_T, c0 = blockIdx.y * RW_T;
    const int t_beg = (int)((long long)T * blockIdx.z / gridDim.z);
    const int t_end = (int)((long long)T * (blockIdx.z + 1) / gridDim.z);
    const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
    u32x4 rx[RW_H];
    float rd[RW_H][8];
    const int lr = tid >> 4, lch = tid & 15;  // token (and those 16, 32, 48 on) and chunk of this thread
    auto load = [&](int t) {
#pragma unroll
        for (int h = 0; h < RW_H; ++h) {
            const int r = t + lr + 16 * h;
            const bool on = r < t_end;
            rx[h] = load16_or_zero(x + (size_t)r * d + c0 + lch * 8, on && c0 + lch * 8 < d);
            load_scores<VEC>(rd[h], dl + (size_t)r * E, e0 + lch * 8, E, on);
        }
    };
    auto store = [&]() {
#pragma unroll
        for (int h = 0; h < RW_H; ++h) {
            const int at = (lr + 16 * h) * RW_T + ((lch ^ ((lr & 3) << 2)) << 3);
            bf16x8 hi, lo;
            split8(rd[h], hi, lo);
            store16(&sX[at], rx[h]);
            *reinterpret_cast<bf16x8*>(&sH[at]) = hi;
            *reinterpret_cast<bf16x8*>(&sL[at]) = lo;
        }
    };
    const int wm = wave & 1, wn = wave >> 1;
    const int fhalf = lane >> 5, g16 = (lane >> 4) & 1, rr = (lane >> 2) & 3, cc = lane & 3;
    int off[2][2];  // [x or scores][block]
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int in = 2 * g16 + (cc >> 1);
        off[0][b] = (8 * fhalf + rr) * RW_T + (((8 * wm + 4 * b + in) ^ (rr << 2)) << 3) + (cc & 1) * 4;
        off[1][b] = (8 * fhalf + rr) * RW_T + (((8 * wn + 4 * b + in) ^ (rr << 2)) << 3) + (cc & 1) * 4;
    }
    auto frag = [&](const bf16* s, int o, int q) {
        return read_tr(s + o + 16 * q * RW_T, s + o + (16 * q + 4) * RW_T);
    };
    f32x16 acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.0f;
    load(t_beg);
    for (int t = t_beg; t < t_end; t += RW_K) {
        store();
        __syncthreads();
        if (t + RW_K < t_end) load(t + RW_K);
#pragma unroll
        for (int q = 0; q < RW_K / 16; ++q) {
            bf16x8 m[2], hi[2], lo[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                m[b] = frag(sX, off[0][b], q);
                hi[b] = frag(sH, off[1][b], q);
                lo[b] = frag(sL, off[1][b], q);
            }
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int mb = 0; mb < 2; ++mb) {
                    acc[nb][mb] = mfma32(hi[nb], m[mb], acc[nb][mb]);
                    acc[nb][mb] = mfma32(lo[nb], m[mb], acc[nb][mb]);
                }
        }
        __syncthreads();
    }
    const EpiPart epi{part, d};
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
        const int c = c0 + wm * 64 + mb * 32 + (lane & 31);
        if (c >= d) continue;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int e = e0 + wn * 64 + nb * 32 + 8 * q + 4 * fhalf;
                const f32x16& a = acc[nb][mb];
                const f32x4 v[2] = {f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]}, f32x4{}};
                if (e >= E) continue;
                if (gridDim.z > 1) {
                    epi(blockIdx.z, 0, c, e, E, v);
                } else {  // one part: the result itself
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (e + j < E) out[(size_t)c * E + e + j] = (bf16)v[0][j];
                }
            }
    }
}

// Parts of the sum over the tokens: at most two workgroups per compute unit,
// which all run at once (five parts instead of four on 112 tiles, 560
// workgroups: 83 us), at least 128 tokens each.
int dw_parts(int T, int d, int E) {
    const int tiles = ((d + 127) / 128) * ((E + 127) / 128);
    return std::max(1, std::min(512 / tiles, (T + 127) / 128));
}

template <bool VEC>
hipError_t route_products(int n_tok, int d, int E, int K, const float* x, const float* wr, const float* dx_perm,
                          const int32_t* assign_row, const float* dl, float* dx, float* dwr, float* part, int parts,
                          hipStream_t s) {
    const auto tiles = [](int v, int t) { return (unsigned)((v + t - 1) / t); };
    const auto with_tile = [](int tile, auto f) {
        return tile == 64 ? f(std::integral_constant<int, 64>{}) : f(std::integral_constant<int, 128>{});
    };
    hipError_t err;
    if (dx != nullptr) {
        GemmArgs<float, float> g{{dl, nullptr}, {wr, nullptr}, E, E, 0, 0, d, E, n_tok, 1, RowPlan{}, nullptr};
        err = with_tile(gm_tile((long)tiles(n_tok, 128) * tiles(d, 128)), [&](auto t) {
            constexpr int T = decltype(t)::value;
            gemm_f32_kernel<T, GM_NT, false, 1, VEC, VEC><<<dim3(tiles(n_tok, T), tiles(d, T)), 256, 0, s>>>(g,
                                                                                                         EpiProduct{dx});
            return hipGetLastError();
        });
        if (err != hipSuccess) return err;
        if (dx_perm != nullptr) {
            const size_t vecs = (size_t)n_tok * d / 8;
            route_add_rows_kernel<<<(unsigned)std::min<size_t>((vecs + 255) / 256, 1 << 20), 256, 0, s>>>(
                n_tok, K, d, dx_perm, assign_row, dx);
            if ((err = hipGetLastError()) != hipSuccess) return err;
        }
    }
    if (dwr != nullptr) {
        GemmArgs<float, float> g{{x, nullptr}, {dl, nullptr}, d, E, 0, d, E, 0, n_tok, 1, RowPlan{}, nullptr};
        constexpr int t = 64;  // (4096 tokens, 256 experts, d 7168: the pass 524 us with 64 in both products, 548 with 128)
        gemm_f32_kernel<t, GM_TN, false, 1, true, VEC><<<dim3(tiles(E, t), tiles(d, t), parts), 256, 0, s>>>(
            g, EpiPart{parts > 1 ? part : dwr, d});
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    return hipSuccess;
}

template <bool VEC>
hipError_t route_products(int n_tok, int d, int E, int K, const bf16* x, const bf16* wr, const bf16* dx_perm,
                          const int32_t* assign_row, const float* dl, bf16* dx, bf16* dwr, float* part, int parts,
                          hipStream_t s) {
    hipError_t err;
    if (dx != nullptr) {
        route_dx_kernel<VEC><<<(unsigned)((n_tok + RX_T - 1) / RX_T) * ((d + RX_C - 1) / RX_C), 256, 0, s>>>(
            n_tok, d, E, K, dl, wr, dx_perm, assign_row, dx);
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    if (dwr != nullptr) {
        route_dw_kernel<VEC><<<dim3((E + RW_T - 1) / RW_T, (d + RW_T - 1) / RW_T, parts), 256, 0, s>>>(
            n_tok, d, E, x, dl, part, dwr);
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    return hipSuccess;
}

template <typename T>
hipError_t route_gradients(int n_tok, int d, int E, int K, const void* x, const void* wr, const void* dx_perm,
                           const int32_t* assign_row, const float* dl, void* dx, void* dwr, float* part, hipStream_t s) {
    const int parts = dw_parts(n_tok, d, E);
    const auto run = [&](auto vec) {  // rows of E elements in whole vectors or not
        return route_products<decltype(vec)::value>(n_tok, d, E, K, (const T*)x, (const T*)wr, (const T*)dx_perm,
                                                    assign_row, dl, (T*)dx, (T*)dwr, part, parts, s);
    };
    const hipError_t err = E % 8 == 0 ? run(std::true_type{}) : run(std::false_type{});
    if (err != hipSuccess || dwr == nullptr || parts == 1) return err;
    const size_t n = (size_t)d * E;
    route_dw_reduce_kernel<T><<<(unsigned)std::min<size_t>((n + 1023) / 1024, 4096), 256, 0, s>>>(n, parts, part, (T*)dwr);
    return hipGetLastError();
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
    err = dtype == MOE_DTYPE_F32
              ? route_gradients<float>(T, d, E, K, x, wr, dx_perm, assign_row, dl, dx, dwr, part, s)
              : route_gradients<bf16>(T, d, E, K, x, wr, dx_perm, assign_row, dl, dx, dwr, part, s);
    if (err == hipSuccess) timer_after(MOE_KERNEL_ROUTE_BACKWARD, s);
    return err;
}

}  // namespace moe
