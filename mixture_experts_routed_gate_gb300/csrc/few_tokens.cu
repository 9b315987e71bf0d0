// few_tokens.cu -- the whole routed-expert layer for a few tokens.
//
//   out_t = sum over the k experts e of token t of p_te * W_down[e] h_te,
//   h_te  = silu(W_gate[e] x_t) * (W_up[e] x_t)
// with the routing of moe_gate_topk.  One warp per dot product; h is kept,
// scaled by its routing weight, as a 16-bit value and the rest of it.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int FEW_WARPS = 8;

template <int DT>
__device__ __forceinline__ float dot8(const uint4 &a, const uint4 &b, float c) {
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c = fma_mixed<DT, false>(av[i], bv[i], c);
        c = fma_mixed<DT, true>(av[i], bv[i], c);
    }
    return c;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

// Order-preserving key of a logit: larger is better, 0 is below every logit's.
// -0 counts as +0, a NaN comes first, so whatever the logits hold, k distinct
// experts in [0, E) are chosen.
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (v != v) return 0xffffffffu;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The k best of one token's E logits (descending, ties to the lower id) and
// their softmax weights, by one warp; lane j < k gets slot j.
template <int SLOTS>
__device__ __forceinline__ void warp_route(const float *row, int E, int k, int lane, int *my_e, float *my_w) {
    float v[SLOTS];
    uint32_t key[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        const int e = s * 32 + lane;
        v[s] = e < E ? row[e] : 0.0f;
        key[s] = e < E ? logit_key(v[s]) : 0u;
    }
    float top = 0.0f, mine = 0.0f;
    int id = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
        int slot = 0;
        float val = 0.0f;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (key[s] > best) {
                best = key[s];
                slot = s;
                val = v[s];
            }
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == most ? slot * 32u + lane : 0xffffffffu);
        val = __shfl_sync(0xffffffffu, val, e & 31u);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (s * 32u + lane == e) key[s] = 0u;
        if (j == 0) top = val;
        if (j == lane) {
            mine = val;
            id = static_cast<int>(e);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
        if (s * 32 + lane < E) sum += expf(v[s] - top);
    sum = warp_sum(sum);
    *my_e = id;
    *my_w = expf(mine - top) / sum;
}

__global__ void __launch_bounds__(32) few_route_kernel(const float *logits, int E, int k, int32_t *idx, float *w) {
    griddep_wait();
    griddep_launch_dependents();
    int e;
    float p;
    warp_route<32>(logits + static_cast<int64_t>(blockIdx.x) * E, E, k, threadIdx.x, &e, &p);
    if (static_cast<int>(threadIdx.x) < k) {
        idx[blockIdx.x * k + threadIdx.x] = e;
        w[blockIdx.x * k + threadIdx.x] = p;
    }
}

// one warp per (routed pair, feature)
template <int DT>
__global__ void __launch_bounds__(FEW_WARPS * 32)
    few_gate_up_kernel(const void *x, const void *w_gate, const void *w_up, const int32_t *idx, const float *w,
                       int pairs, int k, int d_h, int d_e, void *h_hi, void *h_lo) {
    using T = typename Elem<DT>::T;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t job = static_cast<int64_t>(blockIdx.x) * FEW_WARPS + (threadIdx.x >> 5);
    const int pair = static_cast<int>(job / d_e), f = static_cast<int>(job % d_e);
    if (pair >= pairs) return;
    const int64_t row = (static_cast<int64_t>(idx[pair]) * d_e + f) * d_h;
    const uint4 *xr = reinterpret_cast<const uint4 *>(static_cast<const T *>(x) + static_cast<int64_t>(pair / k) * d_h);
    const uint4 *gr = reinterpret_cast<const uint4 *>(static_cast<const T *>(w_gate) + row);
    const uint4 *ur = reinterpret_cast<const uint4 *>(static_cast<const T *>(w_up) + row);
    float g = 0.0f, u = 0.0f;
    for (int c = lane; c < d_h / 8; c += 32) {
        const uint4 xv = xr[c];
        g = dot8<DT>(xv, gr[c], g);
        u = dot8<DT>(xv, ur[c], u);
    }
    g = warp_sum(g);
    u = warp_sum(u);
    if (lane == 0) {
        const float h = g / (1.0f + __expf(-g)) * u * w[pair];
        const T hi = from_f32<T>(h);
        const int64_t o = static_cast<int64_t>(pair) * d_e + f;
        static_cast<T *>(h_hi)[o] = hi;
        static_cast<T *>(h_lo)[o] = from_f32<T>(h - to_f32(hi));
    }
}

// one warp per (token, output)
template <int DT>
__global__ void __launch_bounds__(FEW_WARPS * 32)
    few_down_kernel(const void *h_hi, const void *h_lo, const void *w_down, const int32_t *idx, int tokens, int k,
                    int d_h, int d_e, void *out) {
    using T = typename Elem<DT>::T;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t job = static_cast<int64_t>(blockIdx.x) * FEW_WARPS + (threadIdx.x >> 5);
    const int t = static_cast<int>(job / d_h), j = static_cast<int>(job % d_h);
    if (t >= tokens) return;
    float acc = 0.0f;
    for (int s = 0; s < k; ++s) {
        const int64_t pair = static_cast<int64_t>(t) * k + s;
        const uint4 *hi = reinterpret_cast<const uint4 *>(static_cast<const T *>(h_hi) + pair * d_e);
        const uint4 *lo = reinterpret_cast<const uint4 *>(static_cast<const T *>(h_lo) + pair * d_e);
        const uint4 *wr = reinterpret_cast<const uint4 *>(static_cast<const T *>(w_down) +
                                                          (static_cast<int64_t>(idx[pair]) * d_h + j) * d_e);
        for (int c = lane; c < d_e / 8; c += 32) {
            acc = dot8<DT>(hi[c], wr[c], acc);
            acc = dot8<DT>(lo[c], wr[c], acc);
        }
    }
    acc = warp_sum(acc);
    if (lane == 0) static_cast<T *>(out)[static_cast<int64_t>(t) * d_h + j] = from_f32<T>(acc);
}

template <int DT>
cudaError_t launch_typed(const void *x, const void *w_gate, const void *w_up, const void *w_down, int64_t T,
                         int64_t d_h, int64_t d_e, int64_t k, const int32_t *idx, const float *w, void *h_hi,
                         void *h_lo, void *out, cudaStream_t stream) {
    const int64_t pairs = T * k;
    cudaError_t e = launch_pdl(few_gate_up_kernel<DT>, dim3(static_cast<unsigned>((pairs * d_e + FEW_WARPS - 1) / FEW_WARPS)),
                               dim3(FEW_WARPS * 32), 0, stream, x, w_gate, w_up, idx, w, (int)pairs, (int)k,
                               (int)d_h, (int)d_e, h_hi, h_lo);
    if (e != cudaSuccess) return e;
    return launch_pdl(few_down_kernel<DT>, dim3(static_cast<unsigned>((T * d_h + FEW_WARPS - 1) / FEW_WARPS)),
                      dim3(FEW_WARPS * 32), 0, stream, (const void *)h_hi, (const void *)h_lo, w_down, idx, (int)T,
                      (int)k, (int)d_h, (int)d_e, out);
}

size_t round_up(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t forward_few_ws_bytes(int64_t T, int64_t d_h, int64_t d_e, int64_t E, int64_t k) {
    (void)d_h;
    return round_up(static_cast<size_t>(T * E) * 4) + 2 * round_up(static_cast<size_t>(T * k) * 4) +
           2 * round_up(static_cast<size_t>(T * k * d_e) * 2);
}

cudaError_t launch_forward_few(const void *x, const void *w_g, const float *bias, const void *w_gate, const void *w_up,
                               const void *w_down, int64_t T, int64_t d_h, int64_t d_e, int64_t E, int64_t k,
                               int dtype, void *ws, void *out, int32_t *err, cudaStream_t stream) {
    char *at = static_cast<char *>(ws);
    float *logits = reinterpret_cast<float *>(at);
    at += round_up(static_cast<size_t>(T * E) * 4);
    int32_t *idx = reinterpret_cast<int32_t *>(at);
    at += round_up(static_cast<size_t>(T * k) * 4);
    float *w = reinterpret_cast<float *>(at);
    at += round_up(static_cast<size_t>(T * k) * 4);
    void *h_hi = at;
    void *h_lo = at + round_up(static_cast<size_t>(T * k * d_e) * 2);
    cudaError_t e = launch_gate_topk(x, w_g, bias, T, d_h, E, k, dtype, logits, idx, w, nullptr, err, stream);
    if (e != cudaSuccess) return e;
    e = launch_pdl(few_route_kernel, dim3(static_cast<unsigned>(T)), dim3(32), 0, stream, (const float *)logits, (int)E,
                   (int)k, idx, w);
    if (e != cudaSuccess) return e;
    if (dtype == kBF16)
        return launch_typed<kBF16>(x, w_gate, w_up, w_down, T, d_h, d_e, k, idx, w, h_hi, h_lo, out, stream);
    return launch_typed<kF16>(x, w_gate, w_up, w_down, T, d_h, d_e, k, idx, w, h_hi, h_lo, out, stream);
}

}  // namespace moe
