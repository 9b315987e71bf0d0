// mx4.cu -- microscaled 4-bit floating point: rows to e2m1 elements with one
// power-of-two scale per 32 of them, and back to values.
//
//   s = max(floor(log2 max|x|) - 2, -127),  q = e2m1(x * 2^-s)
//
// A thread quantises whole blocks of 32, so the scale is worked out once for
// them and no lane asks another.  32,768 rows of 7168 bf16 that 4096 tokens
// repeat: 61 to 68 us, 125 MB written, bound by L1 (86% of its rate: a warp's loads
// are 64 bytes apart); when it took 68, two lanes a block took 77, four
// 100 (the loads are then contiguous over the warp, but the scale and the lanes'
// maximum are most of the instructions); CTAs of 64 threads 68, of 256 80.  One
// CTA a token that looks up its rows was no faster at four lanes a block (90 to
// 104): the search eats what it saves.  4096 x 7168 to bits and back in 28 us, 22
// at the copy rate.
#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"

namespace moe {
namespace {

constexpr int MX_THREADS = 128;
constexpr int MX_UNIT = 32;  // a thread quantises whole blocks
constexpr int MX_BACK_STEPS = 4;

template <typename T> struct Unit {  // a block's elements, packed
    static constexpr int DT = std::is_same<T, __half>::value ? kF16 : kBF16;
    static constexpr int VECS = MX_UNIT * static_cast<int>(sizeof(T)) / 16, WORDS = 4 * VECS;
    static constexpr int STEPS = 8 / VECS;  // blocks in flight a thread: 128 bytes
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    // The bits of the largest magnitude: they order like the values, with
    // infinities and then NaNs at the top.
    __device__ __forceinline__ float top() const {
        uint32_t t = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) t = max(t, w[i] & 0x7fffffffu);
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) t = __vmaxu2(t, w[i] & 0x7fff7fffu);
            t = max(t >> 16, t & 0xffffu);
        }
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(t);
        else
            return unpack2<DT>(t).x;
    }
    // eight elements times `by`, a power of two, as a word of 4-bit ones
    __device__ __forceinline__ uint32_t word(int i, float by) const {
        float v[8];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[8 * i + j]) * by;
        } else if constexpr (DT == kBF16) {
            // two at a time: exact but for results that are zero in 4 bits anyway
            const __nv_bfloat162 by2 = __float2bfloat162_rn(by);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                __nv_bfloat162 x;
                memcpy(&x, &w[4 * i + j], 4);
                x = __hmul2(x, by2);
                uint32_t bits;
                memcpy(&bits, &x, 4);
                const float2 f = unpack2<kBF16>(bits);
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack2<kF16>(w[4 * i + j]);
                v[2 * j] = f.x * by;
                v[2 * j + 1] = f.y * by;
            }
        }
        return e2m1x8(v, 1.0f);
    }
};

// A CTA holds rows_per_cta rows at a time, `width` threads (a power of two) on
// each.
template <typename T>
__global__ void __launch_bounds__(MX_THREADS)
    quantize_kernel(const T *__restrict__ x, const int32_t *__restrict__ row_idx, int64_t n_rows, int64_t T_rows,
                    int units, int width, uint8_t *__restrict__ q, uint8_t *__restrict__ sf, int32_t *err) {
    using U = Unit<T>;
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
        uint8_t *qr = q + (here ? r : 0) * units * 16;
        uint8_t *sr = sf + (here ? r : 0) * units;
        const int have = in ? units : 0, store = here ? units : 0;
        for (int u = u0; u < store; u += width * U::STEPS) {
            U raw[U::STEPS];
#pragma unroll
            for (int i = 0; i < U::STEPS; ++i) {
                if (u + i * width < have)
                    raw[i].load(row + (u + i * width) * MX_UNIT);
                else
                    raw[i].clear();
            }
#pragma unroll
            for (int i = 0; i < U::STEPS; ++i) {
                const int at = u + i * width;
                if (at >= store) break;
                const uint32_t s = mx4_scale(raw[i].top());
                const bool bad = s == 255u;
                const float by = bad ? 0.0f : mx4_inverse(s);
                uint32_t out[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    out[j] = raw[i].word(j, by);
                    out[j] = bad ? 0u : out[j];
                }
                reinterpret_cast<uint4 *>(qr)[at] = make_uint4(out[0], out[1], out[2], out[3]);
                sr[at] = static_cast<uint8_t>(s);
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
        uint4 *dst = reinterpret_cast<uint4 *>(out + at * 8);
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
    int width = 1;
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
    const int64_t words = n_rows * (K / 8);
    if (dtype == kF32) return launch_dequantize_typed<float>(q, sf, words, out, stream);
    if (dtype == kBF16) return launch_dequantize_typed<__nv_bfloat16>(q, sf, words, out, stream);
    return launch_dequantize_typed<__half>(q, sf, words, out, stream);
}

}  // namespace moe
