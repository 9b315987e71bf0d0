// mx8_gemm.cu -- the grouped product of 8-bit rows with 8-bit expert weights:
//
//   C[r, n] = sum over k of (qa 2^sa)[r, k] * (qb 2^sb)[expert of r][n, k]
//
// and the gate/up form, h = silu(A Wg^T) * (A Wu^T), quantised to 8 bits.
//
// A warp holds 32 columns of a row, a lane a column; sums in fp32.
#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"
#include "mx8.cuh"

namespace moe {
namespace {

constexpr int G8_WARPS = 8;

__device__ __forceinline__ float block_sum(const uint8_t *a, const uint8_t *b, float s) {
    const uint4 *va = reinterpret_cast<const uint4 *>(a), *vb = reinterpret_cast<const uint4 *>(b);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 x = __ldg(va + i), y = __ldg(vb + i);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
                const float2 f = e4m3x2_values(xs[j] >> h), g = e4m3x2_values(ys[j] >> h);
                s = fmaf(f.x, g.x, s);
                s = fmaf(f.y, g.y, s);
            }
    }
    return s;
}

template <typename TOut, bool GATE_UP>
__global__ void __launch_bounds__(G8_WARPS * 32)
    mx8_gemm_kernel(const uint8_t *q_a, const uint8_t *sf_a, const uint8_t *q_b0, const uint8_t *sf_b0, const uint8_t *q_b1,
                    const uint8_t *sf_b1, const MxTables tab, int64_t N, int64_t K, TOut *out, uint8_t *q_h, uint8_t *sf_h) {
    griddep_wait();
    griddep_launch_dependents();
    const Mx4Block b = mx4_block_of(tab, blockIdx.y);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + lane, kb = K / 32;
    const int64_t f = static_cast<int64_t>(b.g) * N + (n < N ? n : N - 1);
    for (int i = warp; i < b.rows; i += G8_WARPS) {
        const int64_t r = static_cast<int64_t>(b.m_start) + i;
        float s0 = 0.0f, s1 = 0.0f;
        for (int64_t c = 0; c < kb; ++c) {
            const float sa = mx8_factor(__ldg(sf_a + r * kb + c));
            s0 = fmaf(block_sum(q_a + r * K + c * 32, q_b0 + f * K + c * 32, 0.0f) * sa, mx8_factor(__ldg(sf_b0 + f * kb + c)), s0);
            if (GATE_UP)
                s1 = fmaf(block_sum(q_a + r * K + c * 32, q_b1 + f * K + c * 32, 0.0f) * sa, mx8_factor(__ldg(sf_b1 + f * kb + c)), s1);
        }
        if constexpr (GATE_UP) {
            const float h = __fdividef(s0, 1.0f + __expf(-s0)) * s1;
            const uint32_t s = mx8_scale(__reduce_max_sync(0xffffffffu, magnitude_bits(h)));
            q_h[r * N + n] = static_cast<uint8_t>(e4m3x4(h, 0.0f, 0.0f, 0.0f, mx8_inverse(s), s == 255u));
            if (lane == 0) sf_h[r * (N / 32) + blockIdx.x] = static_cast<uint8_t>(s);
        } else if (n < N) {
            out[r * N + n] = from_f32<TOut>(s0);
        }
    }
}

template <typename TOut>
cudaError_t launch_product(const uint8_t *q_a, const uint8_t *sf_a, const uint8_t *q_b, const uint8_t *sf_b, const MxTables &tab,
                           int64_t m_blocks, int64_t N, int64_t K, void *C, cudaStream_t stream) {
    return launch_pdl(mx8_gemm_kernel<TOut, false>, dim3(static_cast<unsigned>((N + 31) / 32), static_cast<unsigned>(m_blocks)),
                      dim3(G8_WARPS * 32), 0, stream, q_a, sf_a, q_b, sf_b, q_b, sf_b, tab, N, K, static_cast<TOut *>(C),
                      static_cast<uint8_t *>(nullptr), static_cast<uint8_t *>(nullptr));
}

}  // namespace

cudaError_t launch_grouped_gemm_mx8(const uint8_t *q_a, const uint8_t *sf_a, const uint8_t *q_b, const uint8_t *sf_b,
                                    const MxTables &tab, int64_t m_blocks, int64_t n_rows, int64_t N, int64_t K,
                                    int64_t E, int out_dtype, void *C, int32_t *err, cudaStream_t stream) {
    if (out_dtype == kF32) return launch_product<float>(q_a, sf_a, q_b, sf_b, tab, m_blocks, N, K, C, stream);
    if (out_dtype == kBF16) return launch_product<__nv_bfloat16>(q_a, sf_a, q_b, sf_b, tab, m_blocks, N, K, C, stream);
    return launch_product<__half>(q_a, sf_a, q_b, sf_b, tab, m_blocks, N, K, C, stream);
}

cudaError_t launch_grouped_gate_up_silu_mx8(const uint8_t *q_a, const uint8_t *sf_a, const uint8_t *q_gate,
                                            const uint8_t *sf_gate, const uint8_t *q_up, const uint8_t *sf_up,
                                            const MxTables &tab, int64_t m_blocks, int64_t n_rows, int64_t d_h,
                                            int64_t d_e, int64_t E, uint8_t *q_h, uint8_t *sf_h, int32_t *err,
                                            cudaStream_t stream) {
    return launch_pdl(mx8_gemm_kernel<float, true>, dim3(static_cast<unsigned>(d_e / 32), static_cast<unsigned>(m_blocks)),
                      dim3(G8_WARPS * 32), 0, stream, q_a, sf_a, q_gate, sf_gate, q_up, sf_up, tab, d_e, d_h,
                      static_cast<float *>(nullptr), q_h, sf_h);
}

}  // namespace moe
