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

// Eight columns of a row as loaded (16 bytes of bf16, 32 of fp32).
template <typename T>
struct Eight;
template <>
struct Eight<bf16> {
    bf16x8 v;
    __device__ void load(const bf16* p) { v = *reinterpret_cast<const bf16x8*>(p); }
    __device__ float operator[](int j) const { return (float)v[j]; }
};
template <>
struct Eight<float> {
    f32x4 a, b;
    __device__ void load(const float* p) {
        a = *reinterpret_cast<const f32x4*>(p);
        b = *reinterpret_cast<const f32x4*>(p + 4);
    }
    __device__ float operator[](int j) const { return j < 4 ? a[j] : b[j - 4]; }
};

// TPR threads per row, NV vectors of eight columns each, held in registers
// between the maximum and the rounding (16384 rows of 14336 columns: 158 us, 4.5
// TB/s; 180 us when the rounding read the row again; NV = 0: longer rows, which
// are read twice).  A row holding a NaN or an infinity gets
// a NaN scale (its bits pass every finite value's) and zeros, so what is
// computed from it is NaN.  live: rows at or past *live are left alone (NULL:
// none).  Columns from split on go to byte split + c - (cols - 128); zeros fill
// the nz / 8 vectors from byte z0 on.
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(256) void quantize_rows_kernel(int64_t rows, int cols, int ldq, int split, int z0, int nz,
                                                           const T* __restrict__ x, int8_t* __restrict__ q,
                                                           float* __restrict__ scale, const int32_t* __restrict__ live) {
    constexpr int RPB = 256 / TPR;  // rows per block
    __shared__ uint32_t part[2][4];
    const int i = threadIdx.x % TPR;
    const int64_t n = live != nullptr ? min(rows, (int64_t)*live) : rows;
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < n; r0 += (int64_t)gridDim.x * RPB, turn ^= 1) {
        const int64_t r = r0 + threadIdx.x / TPR;
        const bool on = r < n;
        const T* row = x + (on ? r : 0) * cols;
        Eight<T> held[NV > 0 ? NV : 1];
        uint32_t m = 0;
        auto max8 = [&](const Eight<T>& v) {
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
        };
        if constexpr (NV > 0) {
            // loads at clamped columns, so that they go out together
#pragma unroll
            for (int k = 0; k < NV; ++k) held[k].load(row + min((i + k * TPR) * 8, cols - 8));
#pragma unroll
            for (int k = 0; k < NV; ++k) max8(held[k]);
        } else {
            for (int c = i * 8; c < cols; c += TPR * 8) {
                held[0].load(row + c);
                max8(held[0]);
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
        if constexpr (TPR > kWave) {  // the parts of two rows in turn: one barrier a row
            if (lane_id() == 0) part[turn][threadIdx.x / kWave] = m;
            __syncthreads();
            m = max(max(part[turn][0], part[turn][1]), max(part[turn][2], part[turn][3]));
        }
        if (!on) continue;  // a whole wave, and no barrier follows it
        const bool finite = m < 0x7F800000u;
        const float s = fmaxf(__builtin_bit_cast(float, m) / 127.0f, 0x1p-126f);
        const float inv = 1.0f / s;
        if (i == 0) scale[r] = finite ? s : __builtin_nanf("");
        int8_t* out = q + r * ldq;
        auto store = [&](int c, const Eight<T>& v) {
            uint32_t lo = 0, hi = 0;
            if (finite) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    lo |= ((uint32_t)quantize_one(v[j], s, inv) & 0xFFu) << (8 * j);
                    hi |= ((uint32_t)quantize_one(v[4 + j], s, inv) & 0xFFu) << (8 * j);
                }
            }
            *reinterpret_cast<u32x2*>(out + (c < split ? c : split + c - (cols - 128))) = u32x2{lo, hi};
        };
        if constexpr (NV > 0) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (i + k * TPR) * 8;
                if (c < cols) store(c, held[k]);
            }
        } else {
            for (int c = i * 8; c < cols; c += TPR * 8) {
                held[0].load(row + c);
                store(c, held[0]);
            }
        }
        if (i * 8 < nz) *reinterpret_cast<u32x2*>(out + z0 + i * 8) = u32x2{0, 0};
    }
}

template <typename T, int TPR, int NV>
hipError_t quantize_launch(int64_t rows, int cols, int ldq, int split, int z0, int nz, const T* x, int8_t* q,
                           float* scale, const int32_t* live, hipStream_t s) {
    const int64_t blocks = std::min<int64_t>((rows + 256 / TPR - 1) / (256 / TPR), 1 << 20);
    quantize_rows_kernel<T, TPR, NV><<<(unsigned)blocks, 256, 0, s>>>(rows, cols, ldq, split, z0, nz, x, q, scale, live);
    return hipGetLastError();
}

// A wave per row up to 4096 columns, a block beyond, or where there are too few
// rows for every compute unit to have its waves (64 rows of 4096: 8.1 us with a
// wave each, 4.9 with a block).
template <typename T>
hipError_t quantize_t(int64_t rows, int cols, int ldq, int split, const T* x, int8_t* q, float* scale,
                      const int32_t* live, hipStream_t s) {
    const bool over = split < ldq;
    const int z0 = over ? split : cols, nz = over ? split - (cols - 128) : ldq - cols;
    const bool few = rows < 2048 && cols > 1024;
    const auto go = cols <= 1024            ? quantize_launch<T, 64, 2>
                    : cols <= 2048 && !few  ? quantize_launch<T, 64, 4>
                    : cols <= 4096 && !few  ? quantize_launch<T, 64, 8>
                    : cols <= 4096          ? quantize_launch<T, 256, 2>
                    : cols <= 8192          ? quantize_launch<T, 256, 4>
                    : cols <= 16384         ? quantize_launch<T, 256, 8>
                                            : quantize_launch<T, 256, 0>;
    return go(rows, cols, ldq, split, z0, nz, x, q, scale, live, s);
}

}  // namespace

hipError_t launch_quantize_rows(int64_t rows, int cols, int ldq, bool overlap, int dtype, const void* x, int8_t* q,
                                float* scale, const int32_t* live, hipStream_t s) {
    const int split = overlap && cols % 128 != 0 ? cols / 128 * 128 : ldq;
    timer_before(MOE_KERNEL_QUANTIZE, s);
    const hipError_t err = dtype == MOE_DTYPE_F32 ? quantize_t<float>(rows, cols, ldq, split, (const float*)x, q, scale, live, s)
                                                  : quantize_t<bf16>(rows, cols, ldq, split, (const bf16*)x, q, scale, live, s);
    if (err == hipSuccess) timer_after(MOE_KERNEL_QUANTIZE, s);
    return err;
}

}  // namespace moe
