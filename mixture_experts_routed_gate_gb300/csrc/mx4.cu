// mx4.cu -- microscaled 4-bit floating point: rows to e2m1 elements with one
// power-of-two scale per 32 of them, and back to values.
//
//   s = max(floor(log2 max|x|) - 2, -127),  q = e2m1(x * 2^-s)
//
// Quantising is bound by instruction issue (72% of the slots, about 0.4 a warp
// and element): 4096 x 7168 bf16 to bits and back in 28 us, 22 at the copy rate;
// 32,768 rows that 4096 tokens repeat, 105 us (one CTA a token that looks up its
// rows: 90 to 104, the search eats what it saves).
#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"

namespace moe {
namespace {

constexpr int MX_THREADS = 128;
constexpr int MX_UNIT = 8;    // elements per thread and step: four lanes hold a block
constexpr int MX_STEPS = 8;   // loads in flight per thread: a row of up to 8192 elements in one go
constexpr int MX_BACK_STEPS = 4;

template <typename T> struct Unit;  // 8 elements as loaded
template <> struct Unit<float> {
    uint4 w[2];
    __device__ __forceinline__ void load(const float *p) {
        w[0] = __ldg(reinterpret_cast<const uint4 *>(p));
        w[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        const uint32_t b[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(b[i]);
    }
    // the bits of the largest magnitude: they order like the values, with
    // infinities and then NaNs at the top
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t b[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) t = max(t, b[i] & 0x7fffffffu);
        return t;
    }
    static __device__ __forceinline__ float top_value(uint32_t t) { return __uint_as_float(t); }
    __device__ __forceinline__ void clear() { w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u); }
};
template <int DT> struct HalfUnit {
    uint4 w;
    __device__ __forceinline__ void load(const void *p) { w = __ldg(static_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<DT>(b[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t a = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), b = __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu);
        const uint32_t c = __vmaxu2(a, b);
        return max(c >> 16, c & 0xffffu);
    }
    static __device__ __forceinline__ float top_value(uint32_t t) { return unpack2<DT>(t).x; }
    __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
};
template <> struct Unit<__half> : HalfUnit<kF16> {};
template <> struct Unit<__nv_bfloat16> : HalfUnit<kBF16> {};

// Four lanes quantise 32 values, 8 each (every lane of the warp takes part):
// returns the lane's 4 bytes of elements and, through s, the scale byte.
template <typename T> __device__ __forceinline__ uint32_t quad_quantize(const Unit<T> &raw, uint32_t &s) {
    uint32_t top = raw.top();
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    s = mx4_scale(Unit<T>::top_value(top));
    const float inv = s == 255u ? 0.0f : mx4_inverse(s);
    float v[8];
    raw.values(v);
    const uint32_t q = e2m1x8(v, inv);
    return s == 255u ? 0u : q;
}

// A CTA holds rows_per_cta rows at a time, `width` threads (a power of two,
// at least four) on each.  Memory bound: 2 bytes in, 0.53 out per 16-bit
// element, every access 16 (4 out) bytes a lane and contiguous over the warp.
template <typename T>
__global__ void __launch_bounds__(MX_THREADS)
    quantize_kernel(const T *__restrict__ x, const int32_t *__restrict__ row_idx, int64_t n_rows, int64_t T_rows,
                    int units, int width, uint8_t *__restrict__ q, uint8_t *__restrict__ sf, int32_t *err) {
    griddep_wait();
    griddep_launch_dependents();
    const int rows_per_cta = MX_THREADS / width;
    const int u0 = threadIdx.x & (width - 1);
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows_per_cta; r0 < n_rows;
         r0 += static_cast<int64_t>(gridDim.x) * rows_per_cta) {
        const int64_t r = r0 + threadIdx.x / width;
        const bool here = r < n_rows;
        int64_t src = here ? (row_idx ? static_cast<int64_t>(__ldg(row_idx + r)) : r) : 0;
        const bool in = here && src >= 0 && src < T_rows;
        if (here && !in && err && u0 == 0) atomicExch(err, kErrDeviceFlag);
        const T *row = x + (in ? src : 0) * units * MX_UNIT;
        uint32_t *qr = reinterpret_cast<uint32_t *>(q) + (here ? r : 0) * units;
        uint8_t *sr = sf + (here ? r : 0) * (units / 4);
        for (int u = u0; u - u0 < units; u += width * MX_STEPS) {  // every lane the same number of steps
            Unit<T> raw[MX_STEPS];
#pragma unroll
            for (int i = 0; i < MX_STEPS; ++i) {
                if (in && u + i * width < units)
                    raw[i].load(row + static_cast<int64_t>(u + i * width) * MX_UNIT);
                else
                    raw[i].clear();
            }
#pragma unroll
            for (int i = 0; i < MX_STEPS; ++i) {
                const int at = u + i * width;
                if (at - u0 >= units) break;  // the same for the whole CTA
                uint32_t s;
                const uint32_t w = quad_quantize(raw[i], s);
                if (here && at < units) {
                    qr[at] = w;
                    if ((at & 3) == 0) sr[at >> 2] = static_cast<uint8_t>(s);
                }
            }
        }
    }
}

// 8 elements a thread
template <typename T>
__global__ void __launch_bounds__(MX_THREADS)
    dequantize_kernel(const uint32_t *__restrict__ q, const uint8_t *__restrict__ sf, int64_t words, T *__restrict__ out) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (MX_THREADS * MX_BACK_STEPS) + threadIdx.x;
    uint32_t w[MX_BACK_STEPS], s[MX_BACK_STEPS];
#pragma unroll
    for (int i = 0; i < MX_BACK_STEPS; ++i) {
        const int64_t at = first + i * MX_THREADS;
        if (at < words) {
            w[i] = __ldg(q + at);
            s[i] = __ldg(sf + (at >> 2));
        }
    }
#pragma unroll
    for (int i = 0; i < MX_BACK_STEPS; ++i) {
        const int64_t at = first + i * MX_THREADS;
        if (at >= words) return;
        const float f = mx4_factor(s[i]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 pair = e2m1x2_values((w[i] >> (8 * j)) & 255u);
            v[2 * j] = pair.x * f;
            v[2 * j + 1] = pair.y * f;
        }
        uint4 *dst = reinterpret_cast<uint4 *>(out + at * MX_UNIT);
        if constexpr (sizeof(T) == 4) {
            dst[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            dst[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
        } else {
            constexpr int DT = std::is_same<T, __half>::value ? kF16 : kBF16;
            dst[0] = make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
        }
    }
}

template <typename T>
cudaError_t launch_quantize_typed(const void *x, const int32_t *row_idx, int64_t n_rows, int64_t T_rows, int64_t K,
                                  uint8_t *q, uint8_t *sf, int32_t *err, cudaStream_t stream) {
    const int units = static_cast<int>(K / MX_UNIT);
    int width = 4;
    while (width < units && width < MX_THREADS) width *= 2;
    const int64_t groups = (n_rows + MX_THREADS / width - 1) / (MX_THREADS / width);
    const int64_t most = static_cast<int64_t>(device_sm_count()) * 512;
    return launch_pdl(quantize_kernel<T>, dim3(static_cast<unsigned>(groups < most ? groups : most)), dim3(MX_THREADS),
                      0, stream, static_cast<const T *>(x), row_idx, n_rows, T_rows, units, width, q, sf, err);
}

template <typename T>
cudaError_t launch_dequantize_typed(const uint8_t *q, const uint8_t *sf, int64_t words, void *out, cudaStream_t stream) {
    constexpr int64_t per_cta = MX_THREADS * MX_BACK_STEPS;
    return launch_pdl(dequantize_kernel<T>, dim3(static_cast<unsigned>((words + per_cta - 1) / per_cta)),
                      dim3(MX_THREADS), 0, stream, reinterpret_cast<const uint32_t *>(q), sf, words,
                      static_cast<T *>(out));
}

}  // namespace

cudaError_t launch_quantize_mx4(const void *x, const int32_t *row_idx, int64_t n_rows, int64_t T, int64_t K,
                                int dtype, uint8_t *q, uint8_t *sf, int32_t *err, cudaStream_t stream) {
    if (dtype == kF32) return launch_quantize_typed<float>(x, row_idx, n_rows, T, K, q, sf, err, stream);
    if (dtype == kBF16) return launch_quantize_typed<__nv_bfloat16>(x, row_idx, n_rows, T, K, q, sf, err, stream);
    return launch_quantize_typed<__half>(x, row_idx, n_rows, T, K, q, sf, err, stream);
}

cudaError_t launch_dequantize_mx4(const uint8_t *q, const uint8_t *sf, int64_t n_rows, int64_t K, int dtype, void *out,
                                  cudaStream_t stream) {
    const int64_t words = n_rows * (K / MX_UNIT);
    if (dtype == kF32) return launch_dequantize_typed<float>(q, sf, words, out, stream);
    if (dtype == kBF16) return launch_dequantize_typed<__nv_bfloat16>(q, sf, words, out, stream);
    return launch_dequantize_typed<__half>(q, sf, words, out, stream);
}

}  // namespace moe
