// Backward pass of the weighted combine y[t] = sum_k w[t,k] h[row(t,k)]:
//   dh[row(t,k)] = w[t,k] dy[t],   dw[t,k] = <dy[t], h[row(t,k)]>
// Bound by memory: h is read and dh written once (2 T K d elements), dy is
// read once from HBM and K times from cache.  4096 tokens, eight slots, d 7168:
// 204 us for 1.0 GB, 4.9 TB/s, what a large copy reaches.
#include <algorithm>

#include "../device_common.h"
#include "../launch.h"

namespace moe {

// One wave per (token, slot): the lanes walk the row in 16-byte vectors; the
// 64 partial dot products meet in a fixed-order butterfly.
template <typename T>
__global__ __launch_bounds__(256) void combine_backward_kernel(int n_slots, int K, int d, const T* __restrict__ dy,
                                                              const T* __restrict__ h,
                                                              const int32_t* __restrict__ assign_row,
                                                              const float* __restrict__ w, T* __restrict__ dh,
                                                              float* __restrict__ dw) {
    constexpr int VEC = 16 / sizeof(T);
    const int lane = lane_id();
    for (int a = blockIdx.x * 4 + threadIdx.x / kWave; a < n_slots; a += gridDim.x * 4) {
        const int r = assign_row[a];
        if ((unsigned)r >= (unsigned)n_slots) {  // a dropped slot
            if (dw != nullptr && lane == 0) dw[a] = 0.0f;
            continue;
        }
        const float wk = w[a];
        const T* py = dy + (size_t)(a / K) * d;
        const T* ph = dw != nullptr ? h + (size_t)r * d : nullptr;
        T* po = dh + (size_t)r * d;
        float sum = 0.0f;
        for (int c = lane * VEC; c < d; c += kWave * VEC) {
            const u32x4 vy = load16(py + c);
            const T* y = reinterpret_cast<const T*>(&vy);
            if (dw != nullptr) {
                const u32x4 vh = load16(ph + c);
                const T* x = reinterpret_cast<const T*>(&vh);
    #pragma unroll
                for (int j = 0; j < VEC; ++j) sum = fmaf(to_f32(y[j]), to_f32(x[j]), sum);
            }
            u32x4 out;
            T* o = reinterpret_cast<T*>(&out);
    #pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] = from_f32<T>(wk * to_f32(y[j]));
            store16(po + c, out);
        }
        if (dw != nullptr) {
            sum = wave_sum(sum);
            if (lane == 0) dw[a] = sum;
        }
    }
}

hipError_t launch_combine_backward(int T, int K, int d, int dtype, const void* dy, const void* h,
                                   const int32_t* assign_row, const float* w, void* dh, float* dw, hipStream_t s) {
    const int n = T * K;
    const unsigned grid = (unsigned)std::min((n + 3) / 4, 1 << 20);
    if (dtype == MOE_DTYPE_F32)
        MOE_TIMED_LAUNCH(MOE_KERNEL_COMBINE_BACKWARD, s,
                         combine_backward_kernel<float><<<grid, 256, 0, s>>>(n, K, d, (const float*)dy, (const float*)h,
                                                                             assign_row, w, (float*)dh, dw));
    else
        MOE_TIMED_LAUNCH(MOE_KERNEL_COMBINE_BACKWARD, s,
                         combine_backward_kernel<bf16><<<grid, 256, 0, s>>>(n, K, d, (const bf16*)dy, (const bf16*)h,
                                                                            assign_row, w, (bf16*)dh, dw));
    return hipGetLastError();
}

}  // namespace moe
