// Symmetric 8-bit quantisation of rows: scale = max(amax |x| / 127, 2^-126)
// and q = x / scale rounded to the nearest integer, ties to even.  Bound by
// memory (each element read once from HBM, one byte written).
//
// The quotient is rounded exactly: half of a row's maximum falls on the border
// 63.5 up to the rounding of the scale, so a rounded fp32 quotient would
// decide such elements by chance.  n = floor(|x| / scale) comes from a rounded
// product, and the sign of |x| - (n + 0.5) scale, which one fma gives exactly,
// decides between n and n + 1.
#include <algorithm>

#include "../device_common.h"
#include "../launch.h"

namespace moe {

namespace {

__device__ __forceinline__ int quantize_one(float x, float scale, float inv) {
    const float a = fabsf(x);
    const float n = floorf(a * inv);
    const float t = fmaf(-(n + 0.5f), scale, a);
    const int lo = (int)n;
    const int q = t > 0.0f || (t == 0.0f && (lo & 1)) ? lo + 1 : lo;
    return x < 0.0f ? -q : q;
}

// TPR threads per row, 8 elements per thread and step; the second walk over
// the row reads cached lines.  A row holding a NaN or an infinity gets a NaN
// scale (its bits pass every finite value's) and zeros, so what is computed
// from it is NaN.  live: rows at or past *live are left alone (NULL: none);
// bytes [cols, ldq) of q are written as zeros; byte p of q at or past split
// (a multiple of 128, cols - split < 128) holds column p - split + cols - 128,
// zero where that lies before split.
template <typename T, int TPR>
__global__ __launch_bounds__(256) void quantize_rows_kernel(int64_t rows, int cols, int ldq, int split, const T* __restrict__ x,
                                                           int8_t* __restrict__ q, float* __restrict__ scale,
                                                           const int32_t* __restrict__ live) {
    constexpr int RPB = 256 / TPR;  // rows per block
    __shared__ uint32_t part[4];
    const int i = threadIdx.x % TPR;
    const int64_t n = live != nullptr ? min(rows, (int64_t)*live) : rows;
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < n; r0 += (int64_t)gridDim.x * RPB) {
        const int64_t r = r0 + threadIdx.x / TPR;
        const bool on = r < n;
        const T* row = x + (on ? r : 0) * cols;
        auto load8 = [&](int c, float (&v)[8]) {
            if constexpr (sizeof(T) == 4) {
                const f32x4 a = *reinterpret_cast<const f32x4*>(row + c), b = *reinterpret_cast<const f32x4*>(row + c + 4);
    #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = a[j];
                    v[4 + j] = b[j];
                }
            } else {
                const bf16x8 a = *reinterpret_cast<const bf16x8*>(row + c);
    #pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = (float)a[j];
            }
        };
        uint32_t m = 0;
        if (on)
            for (int c = i * 8; c < cols; c += TPR * 8) {
                float v[8];
                load8(c, v);
    #pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
            }
    #pragma unroll
        for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
        if constexpr (TPR > kWave) {
            if (lane_id() == 0) part[threadIdx.x / kWave] = m;
            __syncthreads();
            m = max(max(part[0], part[1]), max(part[2], part[3]));
            __syncthreads();  // part is written again for the next row
        }
        if (!on) continue;  // a whole wave, and no barrier follows it
        const bool finite = m < 0x7F800000u;
        const float s = fmaxf(__builtin_bit_cast(float, m) / 127.0f, 0x1p-126f);
        const float inv = finite ? 1.0f / s : 0.0f;
        if (i == 0) scale[r] = finite ? s : __builtin_nanf("");
        for (int b = i * 8; b < ldq; b += TPR * 8) {
            const int c = b < split ? b : b - split + cols - 128;
            uint32_t lo = 0, hi = 0;
            if ((b < split || c >= split) && c < cols && finite) {
                float v[8];
                load8(c, v);
    #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    lo |= ((uint32_t)quantize_one(v[j], s, inv) & 0xFFu) << (8 * j);
                    hi |= ((uint32_t)quantize_one(v[4 + j], s, inv) & 0xFFu) << (8 * j);
                }
            }
            *reinterpret_cast<u32x2*>(q + r * ldq + b) = u32x2{lo, hi};
        }
    }
}

template <typename T>
hipError_t quantize_t(int64_t rows, int cols, int ldq, int split, const void* x, int8_t* q, float* scale, const int32_t* live,
                      hipStream_t s) {
    const int64_t blocks = std::min<int64_t>(cols <= 2048 ? (rows + 3) / 4 : rows, 1 << 20);
    if (cols <= 2048)
        quantize_rows_kernel<T, 64><<<(unsigned)blocks, 256, 0, s>>>(rows, cols, ldq, split, (const T*)x, q, scale,
                                                                              live);
    else
        quantize_rows_kernel<T, 256><<<(unsigned)blocks, 256, 0, s>>>(rows, cols, ldq, split, (const T*)x, q, scale, live);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(int64_t rows, int cols, int ldq, bool overlap, int dtype, const void* x, int8_t* q,
                                float* scale, const int32_t* live, hipStream_t s) {
    const int split = overlap && cols % 128 != 0 ? cols / 128 * 128 : ldq;
    timer_before(MOE_KERNEL_QUANTIZE, s);
    const hipError_t err = dtype == MOE_DTYPE_F32 ? quantize_t<float>(rows, cols, ldq, split, x, q, scale, live, s)
                                                  : quantize_t<bf16>(rows, cols, ldq, split, x, q, scale, live, s);
    if (err == hipSuccess) timer_after(MOE_KERNEL_QUANTIZE, s);
    return err;
}

}  // namespace moe
