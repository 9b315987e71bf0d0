// mx4.cu -- microscaled 4-bit floating point: rows to e2m1 elements with one
// power-of-two scale per 32 of them, back to values, and the grouped product
// of two such matrices over the dispatch tables.
//
//   s = max(floor(log2 max|x|) - 2, -127),  q = e2m1(x * 2^-s)
//   C[r, n] = sum over k of (qa 2^sa)[r, k] * (qb 2^sb)[expert of r][n, k]
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int MX_BLOCK = 32;

// the scale byte of a block whose largest magnitude is `top`: floor(log2) is
// in the exponent field; 255 for a NaN or an infinity
__device__ __forceinline__ uint32_t mx4_scale(float top) {
    const int field = static_cast<int>(__float_as_uint(top) >> 23) & 255;
    if (field == 255) return 255u;
    return static_cast<uint32_t>(max(field - 2, 0));
}

// 2^(127 - byte) for byte <= 252, exact
__device__ __forceinline__ float mx4_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^(byte - 127); byte 255 is NaN
__device__ __forceinline__ float mx4_factor(uint32_t byte) {
    if (byte == 255u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(byte ? byte << 23 : 1u << 22);
}

// two elements to a byte, `lo` in the low nibble: nearest even, limited to 6
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float e2m1_value(uint32_t code) {
    const uint32_t m = code & 7u;
    const float v = m < 4u ? 0.5f * m : (m < 6u ? m - 2.0f : 2.0f * m - 8.0f);
    return (code & 8u) ? -v : v;
}

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

// sum over K of one row of A against one row of B
__device__ __forceinline__ float mx4_dot(const uint8_t *qa, const uint8_t *sa, const uint8_t *qb, const uint8_t *sb,
                                         int64_t K) {
    float acc = 0.0f;
    for (int64_t b = 0; b < K / MX_BLOCK; ++b) {
        float s = 0.0f;
        for (int j = 0; j < 16; ++j) {
            const uint32_t va = qa[b * 16 + j], vb = qb[b * 16 + j];
            s += e2m1_value(va & 15u) * e2m1_value(vb & 15u) + e2m1_value(va >> 4) * e2m1_value(vb >> 4);
        }
        acc += s * (mx4_factor(sa[b]) * mx4_factor(sb[b]));
    }
    return acc;
}

struct Block {
    int g, m_start, rows;
};

__device__ __forceinline__ Block block_of(const Mx4Tables &t, int bx) {
    Block b;
    b.g = t.gidx[bx];
    const int off = bx * 128 - t.padded[b.g];
    b.m_start = off + t.offsets[b.g];
    b.rows = max(0, min(t.sizes[b.g] - off, 128));
    return b;
}

// grid (N / 32, M blocks); a warp's lanes are 32 columns of one row
template <typename TOut>
__global__ void __launch_bounds__(256)
    grouped_kernel(const uint8_t *qa, const uint8_t *sa, const uint8_t *qb, const uint8_t *sb, Mx4Tables tab,
                   int64_t N, int64_t K, TOut *C) {
    griddep_wait();
    griddep_launch_dependents();
    const Block b = block_of(tab, blockIdx.y);
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
    if (n >= N) return;
    const int64_t w = b.g * N + n;
    for (int i = threadIdx.x >> 5; i < b.rows; i += 8) {
        const int64_t r = b.m_start + i;
        C[r * N + n] = from_f32<TOut>(
            mx4_dot(qa + r * (K / 2), sa + r * (K / 32), qb + w * (K / 2), sb + w * (K / 32), K));
    }
}

__global__ void __launch_bounds__(256)
    grouped_gate_up_kernel(const uint8_t *qa, const uint8_t *sa, const uint8_t *qg, const uint8_t *sg,
                           const uint8_t *qu, const uint8_t *su, Mx4Tables tab, int64_t d_e, int64_t K, uint8_t *qh,
                           uint8_t *sh) {
    griddep_wait();
    griddep_launch_dependents();
    const Block b = block_of(tab, blockIdx.y);
    const int lane = threadIdx.x & 31;
    const int64_t w = b.g * d_e + static_cast<int64_t>(blockIdx.x) * 32 + lane;
    for (int i = threadIdx.x >> 5; i < b.rows; i += 8) {
        const int64_t r = b.m_start + i;
        const uint8_t *q = qa + r * (K / 2), *s = sa + r * (K / 32);
        const float g = mx4_dot(q, s, qg + w * (K / 2), sg + w * (K / 32), K);
        const float u = mx4_dot(q, s, qu + w * (K / 2), su + w * (K / 32), K);
        const int64_t o = r * (d_e / 32) + blockIdx.x;
        warp_quantize(g / (1.0f + __expf(-g)) * u, qh + o * 16, sh + o, lane);
    }
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

cudaError_t launch_grouped_gemm_mx4(const uint8_t *q_a, const uint8_t *sf_a, const uint8_t *q_b, const uint8_t *sf_b,
                                    const Mx4Tables &tab, int64_t m_blocks, int64_t n_rows, int64_t N, int64_t K,
                                    int64_t E, int out_dtype, void *C, int32_t *err, cudaStream_t stream) {
    (void)n_rows;
    (void)E;
    (void)err;
    const dim3 grid(static_cast<unsigned>((N + 31) / 32), static_cast<unsigned>(m_blocks));
    if (out_dtype == kF32)
        return launch_pdl(grouped_kernel<float>, grid, dim3(256), 0, stream, q_a, sf_a, q_b, sf_b, tab, N, K,
                          static_cast<float *>(C));
    if (out_dtype == kBF16)
        return launch_pdl(grouped_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, q_a, sf_a, q_b, sf_b, tab, N, K,
                          static_cast<__nv_bfloat16 *>(C));
    return launch_pdl(grouped_kernel<__half>, grid, dim3(256), 0, stream, q_a, sf_a, q_b, sf_b, tab, N, K,
                      static_cast<__half *>(C));
}

cudaError_t launch_grouped_gate_up_silu_mx4(const uint8_t *q_a, const uint8_t *sf_a, const uint8_t *q_gate,
                                            const uint8_t *sf_gate, const uint8_t *q_up, const uint8_t *sf_up,
                                            const Mx4Tables &tab, int64_t m_blocks, int64_t n_rows, int64_t d_h,
                                            int64_t d_e, int64_t E, uint8_t *q_h, uint8_t *sf_h, int32_t *err,
                                            cudaStream_t stream) {
    (void)n_rows;
    (void)E;
    (void)err;
    const dim3 grid(static_cast<unsigned>(d_e / 32), static_cast<unsigned>(m_blocks));
    return launch_pdl(grouped_gate_up_kernel, grid, dim3(256), 0, stream, q_a, sf_a, q_gate, sf_gate, q_up, sf_up, tab,
                      d_e, d_h, q_h, sf_h);
}

}  // namespace moe
