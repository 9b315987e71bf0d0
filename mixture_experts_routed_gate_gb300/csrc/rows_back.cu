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
//
// Bound by its bytes: 4096 tokens, 8 rows of 7168 bf16 each, 157 us (999 MB, 147 at
// the copy rate); 333 tokens, 5 rows of 2304 fp32, 6.1 us (4.8); 64 tokens, 6 rows of
// 2048 fp16, 2.9 us.  What it takes is bytes in flight: 8 elements a thread and
// row, 191 us; four pieces of 16 bytes, one row at a time, four CTAs an SM, 157
// (two rows at a time 154, but 4096 x 6 x 2048 37 us for 35; three CTAs 160; two 173).
// Fewer tokens than twice the SMs: a piece a thread where that covers a row, and
// the token's rows over several CTAs (64 tokens: 4.6 us by one CTA a token; 1
// token, 8 rows of 7168: 6.9, so 2.8).
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int BACK_THREADS = 256;
constexpr int BACK_MAX_K = 32;

// 16 bytes of a row of x's type, and the elements of d_out that go with them
template <typename TX, typename TD> struct Piece {
    static constexpr int N = 16 / sizeof(TX);  // elements
    [[maybe_unused]] static constexpr int DT = std::is_same<TX, __half>::value ? kF16 : kBF16;
    uint4 v;  // d_out: as x where the types are the same, else widened to fp32
    __device__ __forceinline__ void load(const TX *p) { v = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void load_d(const TD *p) {
        if constexpr (std::is_same<TX, TD>::value) {
            v = __ldg(reinterpret_cast<const uint4 *>(p));
        } else {
            constexpr int D = std::is_same<TD, __half>::value ? kF16 : kBF16;
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
            const float2 a = unpack2<D>(w.x), b = unpack2<D>(w.y);
            v = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
        }
    }
    __device__ __forceinline__ float dot(const Piece &d, float s) const {
        const uint32_t x[4] = {v.x, v.y, v.z, v.w}, y[4] = {d.v.x, d.v.y, d.v.z, d.v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(TX) == 4) {
                s = fmaf(__uint_as_float(x[i]), __uint_as_float(y[i]), s);
            } else {  // products of 16-bit values are exact in fp32
                s = fma_mixed<DT, false>(x[i], y[i], s);
                s = fma_mixed<DT, true>(x[i], y[i], s);
            }
        }
        return s;
    }
    // f * this, rounded once
    __device__ __forceinline__ void store_times(float f, TX *p) const {
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(TX) == 4) {
                o[i] = __float_as_uint(f * __uint_as_float(x[i]));
            } else {
                const float2 t = unpack2<DT>(x[i]);
                o[i] = pack2<DT>(f * t.x, f * t.y);
            }
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
    }
};

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

// PIECES 16-byte pieces a thread and row, AT_ONCE rows in flight; CTA (t, y) takes
// `share` of token t's pairs.
template <typename TX, typename TD, int PIECES, int AT_ONCE>
__global__ void __launch_bounds__(BACK_THREADS, 4)
    reduce_backward_kernel(const TD *__restrict__ d_out, const TX *__restrict__ x, const int32_t *__restrict__ pos,
                           const float *__restrict__ w, const int32_t *__restrict__ token, int64_t T, int k, int H,
                           int64_t n_rows, int share, int64_t rows_per_cta, TX *__restrict__ d_x, float *__restrict__ d_w, int32_t *err) {
    using P = Piece<TX, TD>;
    __shared__ BackPairs pairs;
    __shared__ float sums[BACK_THREADS / 32][BACK_MAX_K];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int step = blockDim.x * P::N;
    const int first = blockIdx.y * share, last = min(first + share, k);
    if (t < T) {
        P d[PIECES];
        auto load_d = [&](int h0) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int h = h0 + i * step;
                if (h < H)
                    d[i].load_d(d_out + t * H + h);
                else
                    d[i].v = make_uint4(0u, 0u, 0u, 0u);
            }
        };
        load_d(threadIdx.x * P::N);
        if (warp == 0) read_pairs(pairs, t, pos, w, token, k, n_rows, err);
        sums[warp][lane] = 0.0f;
        __syncthreads();
        for (int h0 = threadIdx.x * P::N; h0 - static_cast<int>(threadIdx.x) * P::N < H; h0 += PIECES * step) {
            if (h0 >= PIECES * step) load_d(h0);
            for (int j0 = first; j0 < last; j0 += AT_ONCE) {
                P v[AT_ONCE][PIECES];
                bool read[AT_ONCE];
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u) {
                    const int32_t from = j0 + u < last ? pairs.read[j0 + u] : -1;
                    read[u] = d_w && from >= 0;
                    if (read[u]) {
#pragma unroll
                        for (int i = 0; i < PIECES; ++i) {
                            const int h = h0 + i * step;
                            if (h < H) v[u][i].load(x + static_cast<int64_t>(from) * H + h);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u) {
                    const int32_t to = j0 + u < last ? pairs.write[j0 + u] : -1;
                    if (to >= 0) {
                        const float f = pairs.w[j0 + u];
#pragma unroll
                        for (int i = 0; i < PIECES; ++i) {
                            const int h = h0 + i * step;
                            if (h < H) d[i].store_times(f, d_x + static_cast<int64_t>(to) * H + h);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u) {
                    if (!read[u]) continue;
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < PIECES; ++i)
                        if (h0 + i * step < H) s = v[u][i].dot(d[i], s);
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                    if (lane == 0) sums[warp][j0 + u] += s;
                }
            }
        }
        __syncthreads();
        if (d_w && warp == 0 && lane >= first && lane < last) {
            float s = 0.0f;
            for (int i = 0; i < warps; ++i) s += sums[i][lane];
            d_w[t * k + lane] = s;
        }
    }
    // rows that no pair names, of this CTA's share
    const int64_t r0 = (t * gridDim.y + blockIdx.y) * rows_per_cta, r1 = min(r0 + rows_per_cta, n_rows);
    for (int64_t r = r0 + warp; r < r1; r += warps) {
        const int32_t u = __ldg(token + r);
        const bool named = u >= 0 && u < T && lane < k && __ldg(pos + static_cast<int64_t>(u) * k + lane) == r;
        if (__any_sync(0xffffffffu, named)) continue;
        for (int h = lane * P::N; h < H; h += 32 * P::N) *reinterpret_cast<uint4 *>(d_x + r * H + h) = make_uint4(0u, 0u, 0u, 0u);
    }
}

template <typename TX, typename TD>
cudaError_t launch_typed(const void *d_out, const void *x, const int32_t *pos, const float *w, const int32_t *token, int64_t T,
                         int64_t k, int64_t H, int64_t n_rows, void *d_x, float *d_w, int32_t *err, cudaStream_t stream) {
    // few tokens: a token's pairs over as many CTAs as fill the GPU twice
    const int64_t room = 2 * device_sm_count(), parts = T >= room ? 1 : T > 0 ? (room / T < k ? room / T : k) : 1;
    const int share = static_cast<int>((k + parts - 1) / parts);
    const dim3 grid(static_cast<unsigned>(T > 0 ? T : (n_rows + 7) / 8), static_cast<unsigned>((k + share - 1) / share));
    const int64_t ctas = static_cast<int64_t>(grid.x) * grid.y;
    const int64_t pieces = H * static_cast<int64_t>(sizeof(TX)) / 16;
    auto launch = [&](auto kern, int each) {
        const int64_t threads = (pieces + each - 1) / each;
        return launch_pdl(kern, grid, dim3(static_cast<unsigned>(threads < BACK_THREADS ? (threads + 31) / 32 * 32 : BACK_THREADS)), 0,
                          stream, static_cast<const TD *>(d_out), static_cast<const TX *>(x), pos, w, token, T,
                          static_cast<int>(k), static_cast<int>(H), n_rows, share, (n_rows + ctas - 1) / ctas,
                          static_cast<TX *>(d_x), d_w, err);
    };
    if (T < room && pieces <= BACK_THREADS) return launch(reduce_backward_kernel<TX, TD, 1, 2>, 1);
    return launch(reduce_backward_kernel<TX, TD, 4, 1>, 4);
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
