// rows_back.cu -- the gradient of the combine out[t] = sum_j w[t,j] x[pos[t,j]]:
//
//   d_x[r]   = (sum of w[t,j] over the j with pos[t,j] = r) * d_out[t],  t = token of row r
//   d_w[t,j] = sum over h of x[pos[t,j], h] * d_out[t, h]
//
// and zeros for rows that no pair names and pairs that name no row.
//
// A row belongs to the token that sorted_token_idx gives it, so only that
// token's CTA writes it, whatever the positions hold: nothing is added by
// atomics and the same inputs give the same bits.  A CTA takes a token: d_out's
// row is read once and stays in registers over the token's rows.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int BACK_THREADS = 256;
constexpr int BACK_MAX_K = 32;

// 8 consecutive elements as floats
template <typename T> __device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        constexpr int DT = std::is_same<T, __half>::value ? kF16 : kBF16;
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

template <typename T> __device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        constexpr int DT = std::is_same<T, __half>::value ? kF16 : kBF16;
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
    }
}

// One warp, before the token's rows: what to do for each of its pairs.
struct BackPairs {
    int32_t read[BACK_MAX_K];   // row whose product with d_out is the weight's gradient, or -1
    int32_t write[BACK_MAX_K];  // row to write, or -1
    float w[BACK_MAX_K];        // with this factor
};

__device__ __forceinline__ void read_pairs(BackPairs &s, int64_t t, const int32_t *pos, const float *w, const int32_t *token,
                                           int k, int64_t n_rows, int32_t *err) {
    const int j = threadIdx.x;
    const int32_t r = j < k ? __ldg(pos + t * k + j) : -1;
    const bool in = r >= 0 && r < n_rows;
    const bool mine = in && __ldg(token + (in ? r : 0)) == t;
    if (err && ((!in && r != -1) || (in && !mine))) atomicExch(err, kErrDeviceFlag);
    const uint32_t same = __match_any_sync(0xffffffffu, r);
    const float wj = j < k ? (w ? __ldg(w + t * k + j) : 1.0f) : 0.0f;
    float sum = 0.0f;
    for (int i = 0; i < k; ++i) {
        const float wi = __shfl_sync(0xffffffffu, wj, i);
        if (same >> i & 1) sum += wi;
    }
    s.read[j] = in ? r : -1;
    s.write[j] = mine && (same & ((1u << j) - 1u)) == 0 ? r : -1;  // a row that two pairs name: the first writes it
    s.w[j] = sum;
}

template <typename TX, typename TD>
__global__ void __launch_bounds__(BACK_THREADS)
    reduce_backward_kernel(const TD *__restrict__ d_out, const TX *__restrict__ x, const int32_t *__restrict__ pos,
                           const float *__restrict__ w, const int32_t *__restrict__ token, int64_t T, int k, int H,
                           int64_t n_rows, int64_t rows_per_cta, TX *__restrict__ d_x, float *__restrict__ d_w, int32_t *err) {
    __shared__ BackPairs pairs;
    __shared__ float sums[BACK_THREADS / 32][BACK_MAX_K];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (t < T) {
        if (warp == 0) read_pairs(pairs, t, pos, w, token, k, n_rows, err);
        sums[warp][lane] = 0.0f;
        __syncthreads();
        for (int h0 = 0; h0 < H; h0 += BACK_THREADS * 8) {
            const int h = h0 + threadIdx.x * 8;
            const bool in = h < H;
            float d[8];
            if (in) load8(d_out + t * H + h, d);
            for (int j = 0; j < k; ++j) {
                const int32_t from = pairs.read[j], to = pairs.write[j];
                float s = 0.0f;
                if (in && d_w && from >= 0) {
                    float v[8];
                    load8(x + static_cast<int64_t>(from) * H + h, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s = fmaf(v[i], d[i], s);
                }
                if (in && to >= 0) {
                    float v[8];
                    const float f = pairs.w[j];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = f * d[i];
                    store8(d_x + static_cast<int64_t>(to) * H + h, v);
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane == 0) sums[warp][j] += s;
            }
        }
        __syncthreads();
        if (d_w && threadIdx.x < k) {
            float s = 0.0f;
            for (int i = 0; i < BACK_THREADS / 32; ++i) s += sums[i][threadIdx.x];
            d_w[t * k + threadIdx.x] = s;
        }
    }
    // rows that no pair names, of this CTA's share
    const int64_t r0 = t * rows_per_cta, r1 = min(r0 + rows_per_cta, n_rows);
    for (int64_t r = r0 + warp; r < r1; r += BACK_THREADS / 32) {
        const int32_t u = __ldg(token + r);
        const bool named = u >= 0 && u < T && lane < k && __ldg(pos + static_cast<int64_t>(u) * k + lane) == r;
        if (__any_sync(0xffffffffu, named)) continue;
        const float zero[8] = {};
        for (int h = lane * 8; h < H; h += 256) store8(d_x + r * H + h, zero);
    }
}

template <typename TX, typename TD>
cudaError_t launch_typed(const void *d_out, const void *x, const int32_t *pos, const float *w, const int32_t *token, int64_t T,
                         int64_t k, int64_t H, int64_t n_rows, void *d_x, float *d_w, int32_t *err, cudaStream_t stream) {
    const int64_t ctas = T > 0 ? T : (n_rows + 7) / 8;
    return launch_pdl(reduce_backward_kernel<TX, TD>, dim3(static_cast<unsigned>(ctas)), dim3(BACK_THREADS), 0, stream,
                      static_cast<const TD *>(d_out), static_cast<const TX *>(x), pos, w, token, T, static_cast<int>(k),
                      static_cast<int>(H), n_rows, (n_rows + ctas - 1) / ctas, static_cast<TX *>(d_x), d_w, err);
}

}  // namespace

cudaError_t launch_reduce_backward(const void *d_out, const void *x, const int32_t *pos, const float *w, const int32_t *token,
                                   int64_t T, int64_t k, int64_t H, int64_t n_rows, int x_dtype, int out_dtype, void *d_x,
                                   float *d_w, int32_t *err, cudaStream_t stream) {
    using bf16 = __nv_bfloat16;
    if (x_dtype == kF16) return launch_typed<__half, __half>(d_out, x, pos, w, token, T, k, H, n_rows, d_x, d_w, err, stream);
    if (x_dtype == kBF16) return launch_typed<bf16, bf16>(d_out, x, pos, w, token, T, k, H, n_rows, d_x, d_w, err, stream);
    if (out_dtype == kF16) return launch_typed<float, __half>(d_out, x, pos, w, token, T, k, H, n_rows, d_x, d_w, err, stream);
    if (out_dtype == kBF16) return launch_typed<float, bf16>(d_out, x, pos, w, token, T, k, H, n_rows, d_x, d_w, err, stream);
    return launch_typed<float, float>(d_out, x, pos, w, token, T, k, H, n_rows, d_x, d_w, err, stream);
}

}  // namespace moe
