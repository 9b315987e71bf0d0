// mx4.cu -- microscaled 4-bit floating point: rows to e2m1 elements with one
// power-of-two scale per 32 of them, and back to values.
//
//   s = max(floor(log2 max|x|) - 2, -127),  q = e2m1(x * 2^-s)
#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}

// One warp quantises 32 values, one per lane; lanes 0, 2, ... write their bytes.
__device__ __forceinline__ void warp_quantize(float v, uint8_t *q, uint8_t *sf, int lane) {
    // fmaxf drops a NaN, so a block with one is found by a vote
    const bool odd = __any_sync(0xffffffffu, !(fabsf(v) < INFINITY));
    const uint32_t s = odd ? 255u : mx4_scale(warp_max(fabsf(v)));
    const float a = odd ? 0.0f : v * mx4_inverse(s);
    const float b = __shfl_down_sync(0xffffffffu, a, 1);
    if ((lane & 1) == 0) q[lane >> 1] = static_cast<uint8_t>(e2m1x2(a, b));
    if (lane == 0) *sf = static_cast<uint8_t>(s);
}

template <typename T>
__global__ void __launch_bounds__(256)
    quantize_kernel(const T *x, const int32_t *row_idx, int64_t n_rows, int64_t T_rows, int64_t blocks, uint8_t *q,
                    uint8_t *sf, int32_t *err) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (i >= n_rows * blocks) return;
    const int64_t r = i / blocks, b = i % blocks;
    const int64_t src = row_idx ? row_idx[r] : r;
    float v = 0.0f;
    if (src >= 0 && src < T_rows)
        v = to_f32(x[(src * blocks + b) * MX_BLOCK + lane]);
    else if (err && lane == 0)
        atomicExch(err, kErrDeviceFlag);
    warp_quantize(v, q + i * (MX_BLOCK / 2), sf + i, lane);
}

template <typename T>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const uint8_t *q, const uint8_t *sf, int64_t bytes, T *out) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= bytes) return;
    const float f = mx4_factor(sf[i / 16]);
    out[2 * i] = from_f32<T>(e2m1_value(q[i] & 15u) * f);
    out[2 * i + 1] = from_f32<T>(e2m1_value(q[i] >> 4) * f);
}

}  // namespace

cudaError_t launch_quantize_mx4(const void *x, const int32_t *row_idx, int64_t n_rows, int64_t T, int64_t K,
                                int dtype, uint8_t *q, uint8_t *sf, int32_t *err, cudaStream_t stream) {
    const int64_t blocks = K / MX_BLOCK, warps = n_rows * blocks;
    const dim3 grid(static_cast<unsigned>((warps + 7) / 8));
    if (dtype == kF32)
        return launch_pdl(quantize_kernel<float>, grid, dim3(256), 0, stream, static_cast<const float *>(x), row_idx,
                          n_rows, T, blocks, q, sf, err);
    if (dtype == kBF16)
        return launch_pdl(quantize_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream,
                          static_cast<const __nv_bfloat16 *>(x), row_idx, n_rows, T, blocks, q, sf, err);
    return launch_pdl(quantize_kernel<__half>, grid, dim3(256), 0, stream, static_cast<const __half *>(x), row_idx,
                      n_rows, T, blocks, q, sf, err);
}

cudaError_t launch_dequantize_mx4(const uint8_t *q, const uint8_t *sf, int64_t n_rows, int64_t K, int dtype, void *out,
                                  cudaStream_t stream) {
    const int64_t bytes = n_rows * (K / 2);
    const dim3 grid(static_cast<unsigned>((bytes + 255) / 256));
    if (dtype == kF32)
        return launch_pdl(dequantize_kernel<float>, grid, dim3(256), 0, stream, q, sf, bytes,
                          static_cast<float *>(out));
    if (dtype == kBF16)
        return launch_pdl(dequantize_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, q, sf, bytes,
                          static_cast<__nv_bfloat16 *>(out));
    return launch_pdl(dequantize_kernel<__half>, grid, dim3(256), 0, stream, q, sf, bytes, static_cast<__half *>(out));
}

}  // namespace moe
