// mx8.cu -- 8-bit rows (e4m3 elements, one power-of-two scale per 32): from
// values, back to values, and sorted by expert.
//
//   s = least power of two, 2^-127 at least, with max|x| / s <= 448
//   q = e4m3(x / s)
//
// All three are bound by the bytes they move.  4096 x 7168: from bf16 14.8 us (90 MB,
// 13.2 at the copy rate), from fp32 22.7 (148 MB, 21.8); to bf16 11.4 (13.1; part of the
// result stays in L2), to fp32 32.5 (21.8); sorted for 8 experts a token 42 us (273 MB,
// 40; the stores wait in the queue to L1), 64 tokens of 2048 for 6 experts 2.1 us, a
// launch.
#include "common.cuh"
#include "internal.h"
#include "mx8.cuh"

namespace moe {
namespace {

constexpr int M8_THREADS = 256;
constexpr int M8_STEPS = 4;  // units in flight a thread

// 8 consecutive elements
template <typename T> struct Eight {
    static constexpr int DT = std::is_same<T, __half>::value ? kF16 : kBF16;
    float v[8];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<DT>(u[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(p) =
                make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
        }
    }
};

// Four lanes a block.  Units past the end count as zeros, so that all lanes of
// a warp take part in the blocks' maxima.
template <typename T>
__global__ void __launch_bounds__(M8_THREADS)
    quantize_kernel(const T *__restrict__ x, int64_t units, uint8_t *__restrict__ q, uint8_t *__restrict__ sf) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (M8_THREADS * M8_STEPS) + threadIdx.x;
    Eight<T> e[M8_STEPS];
#pragma unroll
    for (int i = 0; i < M8_STEPS; ++i) {
        const int64_t at = first + i * M8_THREADS;
        if (at < units) {
            e[i].load(x + at * 8);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) e[i].v[j] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < M8_STEPS; ++i) {
        const int64_t at = first + i * M8_THREADS;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, magnitude_bits(e[i].v[j]));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t s = mx8_scale(top);
        const float by = mx8_inverse(s);
        const bool bad = s == 255u;
        const float(&v)[8] = e[i].v;
        if (at < units) {
            reinterpret_cast<uint2 *>(q)[at] =
                make_uint2(e4m3x4(v[0], v[1], v[2], v[3], by, bad), e4m3x4(v[4], v[5], v[6], v[7], by, bad));
            if ((threadIdx.x & 3) == 0) sf[at >> 2] = static_cast<uint8_t>(s);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(M8_THREADS)
    dequantize_kernel(const uint2 *__restrict__ q, const uint8_t *__restrict__ sf, int64_t units, T *__restrict__ out) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (M8_THREADS * M8_STEPS) + threadIdx.x;
    uint2 w[M8_STEPS];
    uint32_t s[M8_STEPS];
#pragma unroll
    for (int i = 0; i < M8_STEPS; ++i) {
        const int64_t at = first + i * M8_THREADS;
        if (at < units) {
            w[i] = __ldg(q + at);
            s[i] = __ldg(sf + (at >> 2));
        }
    }
#pragma unroll
    for (int i = 0; i < M8_STEPS; ++i) {
        const int64_t at = first + i * M8_THREADS;
        if (at >= units) return;
        const float f = mx8_factor(s[i]);
        Eight<T> e;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 pair = e4m3x2_values((j < 2 ? w[i].x : w[i].y) >> (16 * (j & 1)));
            e.v[2 * j] = pair.x * f;
            e.v[2 * j + 1] = pair.y * f;
        }
        e.store(out + at * 8);
    }
}

// A CTA a token: its row is read once and stored once for each of its rows.
template <typename SF>
__global__ void __launch_bounds__(M8_THREADS)
    sort_kernel(const uint4 *__restrict__ q, const SF *__restrict__ sf, const int32_t *__restrict__ pos, int k,
                int64_t n_rows, int vecs, int words, uint4 *__restrict__ q_out, SF *__restrict__ sf_out) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = blockIdx.x;
    for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
        const uint4 w = __ldg(q + t * vecs + v);
        for (int j = 0; j < k; ++j) {
            const int32_t r = __ldg(pos + t * k + j);
            if (r >= 0 && r < n_rows) q_out[static_cast<int64_t>(r) * vecs + v] = w;
        }
    }
    for (int v = threadIdx.x; v < words; v += blockDim.x) {
        const SF w = sf[t * words + v];
        for (int j = 0; j < k; ++j) {
            const int32_t r = __ldg(pos + t * k + j);
            if (r >= 0 && r < n_rows) sf_out[static_cast<int64_t>(r) * words + v] = w;
        }
    }
}

dim3 flat_grid(int64_t units) {
    constexpr int64_t per_cta = M8_THREADS * M8_STEPS;
    return dim3(static_cast<unsigned>((units + per_cta - 1) / per_cta));
}

template <typename T>
cudaError_t quantize_typed(const void *x, int64_t units, uint8_t *q, uint8_t *sf, cudaStream_t stream) {
    return launch_pdl(quantize_kernel<T>, flat_grid(units), dim3(M8_THREADS), 0, stream, static_cast<const T *>(x), units, q, sf);
}

template <typename T>
cudaError_t dequantize_typed(const uint8_t *q, const uint8_t *sf, int64_t units, void *out, cudaStream_t stream) {
    return launch_pdl(dequantize_kernel<T>, flat_grid(units), dim3(M8_THREADS), 0, stream,
                      reinterpret_cast<const uint2 *>(q), sf, units, static_cast<T *>(out));
}

}  // namespace

cudaError_t launch_quantize_mx8(const void *x, int64_t n_rows, int64_t K, int dtype, uint8_t *q, uint8_t *sf,
                                cudaStream_t stream) {
    const int64_t units = n_rows * (K / 8);
    if (dtype == kF32) return quantize_typed<float>(x, units, q, sf, stream);
    if (dtype == kBF16) return quantize_typed<__nv_bfloat16>(x, units, q, sf, stream);
    return quantize_typed<__half>(x, units, q, sf, stream);
}

cudaError_t launch_dequantize_mx8(const uint8_t *q, const uint8_t *sf, int64_t n_rows, int64_t K, int dtype, void *out,
                                  cudaStream_t stream) {
    const int64_t units = n_rows * (K / 8);
    if (dtype == kF32) return dequantize_typed<float>(q, sf, units, out, stream);
    if (dtype == kBF16) return dequantize_typed<__nv_bfloat16>(q, sf, units, out, stream);
    return dequantize_typed<__half>(q, sf, units, out, stream);
}

cudaError_t launch_sort_rows_mx8(const uint8_t *q, const uint8_t *sf, const int32_t *pos, int64_t T, int64_t k,
                                 int64_t n_rows, int64_t K, uint8_t *q_out, uint8_t *sf_out, cudaStream_t stream) {
    const int vecs = static_cast<int>(K / 16), words = static_cast<int>(K / 32);
    const bool four = K % 128 == 0 && ((reinterpret_cast<uintptr_t>(sf) | reinterpret_cast<uintptr_t>(sf_out)) & 3u) == 0;
    const dim3 grid(static_cast<unsigned>(T)), block(M8_THREADS);
    const uint4 *from = reinterpret_cast<const uint4 *>(q);
    uint4 *to = reinterpret_cast<uint4 *>(q_out);
    if (four)
        return launch_pdl(sort_kernel<uint32_t>, grid, block, 0, stream, from, reinterpret_cast<const uint32_t *>(sf), pos,
                          static_cast<int>(k), n_rows, vecs, words / 4, to, reinterpret_cast<uint32_t *>(sf_out));
    return launch_pdl(sort_kernel<uint8_t>, grid, block, 0, stream, from, sf, pos, static_cast<int>(k), n_rows, vecs, words,
                      to, sf_out);
}

}  // namespace moe
