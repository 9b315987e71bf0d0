// norm.cu -- the norms before and after a block, fused with its gate and
// residual scale, and their gradients.
//
// Forward, per row of H elements in fp32:
//   z = y * rstd(y) * w_post;  out = res + alpha * gate * z;
//   u = out * rstd(out) * w_next;  rstd(v) = 1 / sqrt(mean(v^2) + eps).
// Backward, with v = d_u * w_next, r = rstd(out), r2 = rstd(y):
//   d   = d_out + r * v - out * r^3 / H * sum(v * out)
//   dz  = alpha * gate * d,  v2 = dz * w_post
//   d_y = r2 * v2 - y * r2^3 / H * sum(v2 * y)
// and the weights' and the gate's gradients are column (or row) sums of
// products of these.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int NORM_THREADS = 256;

struct NormParams {
    const void *y, *res, *w_post, *gate, *w_next;
    const void *d_out, *d_u, *saved_out;
    const float *r_post, *r_next;
    void *out, *u, *d_res, *d_y, *d_gate;
    float *rstd_post, *rstd_next, *d_w_post, *d_w_next;
    float *row_sum;  // backward: r^3 / H * sum(v * out) of each row
    int gate_kind;
    float alpha, eps;
    int64_t T;
    int H;
};

template <typename T> __device__ __forceinline__ float at(const void *p, int64_t i) {
    return to_f32(static_cast<const T *>(p)[i]);
}

template <typename T> __device__ __forceinline__ float gate_at(const NormParams &p, int64_t t, int h) {
    if (p.gate_kind == 1) return at<T>(p.gate, h);
    if (p.gate_kind == 2) return at<T>(p.gate, t);
    if (p.gate_kind == 3) return at<T>(p.gate, t * p.H + h);
    return 1.0f;
}

__device__ __forceinline__ float cta_sum(float v, float *scratch) {
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < NORM_THREADS / 32; ++w) total += scratch[w];
    return total;
}

template <typename T>
__global__ void __launch_bounds__(NORM_THREADS) norm_kernel(NormParams p) {
    __shared__ float scratch[NORM_THREADS / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = blockIdx.x, base = t * p.H;
    float r2 = 1.0f;
    if (p.w_post) {
        float s = 0.0f;
        for (int h = threadIdx.x; h < p.H; h += NORM_THREADS) {
            const float v = at<T>(p.y, base + h);
            s += v * v;
        }
        r2 = 1.0f / sqrtf(cta_sum(s, scratch) / static_cast<float>(p.H) + p.eps);
        if (p.rstd_post && threadIdx.x == 0) p.rstd_post[t] = r2;
    }
    auto value = [&](int h) {
        float o = at<T>(p.res, base + h);
        if (p.y) {
            float z = at<T>(p.y, base + h);
            if (p.w_post) z = z * r2 * at<T>(p.w_post, h);
            o += p.alpha * gate_at<T>(p, t, h) * z;
        }
        return o;
    };
    float r = 0.0f;
    if (p.w_next) {
        float s = 0.0f;
        for (int h = threadIdx.x; h < p.H; h += NORM_THREADS) {
            const float o = value(h);
            s += o * o;
        }
        r = 1.0f / sqrtf(cta_sum(s, scratch) / static_cast<float>(p.H) + p.eps);
        if (p.rstd_next && threadIdx.x == 0) p.rstd_next[t] = r;
    }
    for (int h = threadIdx.x; h < p.H; h += NORM_THREADS) {
        const float o = value(h);
        if (p.w_next) static_cast<T *>(p.u)[base + h] = from_f32<T>(o * r * at<T>(p.w_next, h));
        if (p.y) static_cast<T *>(p.out)[base + h] = from_f32<T>(o);
    }
}

// d at one element, given the row's sum term
template <typename T>
__device__ __forceinline__ float upstream(const NormParams &p, int64_t t, int h, float sum) {
    const int64_t i = t * p.H + h;
    float d = p.d_out ? at<T>(p.d_out, i) : 0.0f;
    if (p.w_next) d += p.r_next[t] * at<T>(p.d_u, i) * at<T>(p.w_next, h) - at<T>(p.saved_out, i) * sum;
    return d;
}

template <typename T>
__global__ void __launch_bounds__(NORM_THREADS) norm_backward_rows(NormParams p) {
    __shared__ float scratch[NORM_THREADS / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = blockIdx.x, base = t * p.H;
    float sum1 = 0.0f;
    if (p.w_next) {
        float s = 0.0f;
        for (int h = threadIdx.x; h < p.H; h += NORM_THREADS)
            s += at<T>(p.d_u, base + h) * at<T>(p.w_next, h) * at<T>(p.saved_out, base + h);
        const float r = p.r_next[t];
        sum1 = cta_sum(s, scratch) * (r * r * r / static_cast<float>(p.H));
        if (threadIdx.x == 0) p.row_sum[t] = sum1;
    }
    const float r2 = p.w_post ? p.r_post[t] : 1.0f;
    float sum2 = 0.0f, dg = 0.0f;
    if (p.y) {
        for (int h = threadIdx.x; h < p.H; h += NORM_THREADS) {
            const float d = upstream<T>(p, t, h, sum1), y = at<T>(p.y, base + h);
            const float w = p.w_post ? at<T>(p.w_post, h) : 1.0f;
            dg += d * (y * r2 * w);
            sum2 += p.alpha * gate_at<T>(p, t, h) * d * w * y;
        }
        sum2 = cta_sum(sum2, scratch) * (r2 * r2 * r2 / static_cast<float>(p.H));
        if (p.gate_kind == 2 && p.d_gate) {
            dg = cta_sum(dg, scratch);
            if (threadIdx.x == 0) static_cast<float *>(p.d_gate)[t] = p.alpha * dg;
        }
    }
    for (int h = threadIdx.x; h < p.H; h += NORM_THREADS) {
        const float d = upstream<T>(p, t, h, sum1);
        if (p.y) {
            const float y = at<T>(p.y, base + h), w = p.w_post ? at<T>(p.w_post, h) : 1.0f;
            const float dz = p.alpha * gate_at<T>(p, t, h) * d;
            static_cast<T *>(p.d_y)[base + h] = from_f32<T>(p.w_post ? r2 * dz * w - y * sum2 : dz);
            if (p.gate_kind == 3 && p.d_gate) static_cast<T *>(p.d_gate)[base + h] = from_f32<T>(p.alpha * d * (y * r2 * w));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(32) norm_backward_columns(NormParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int h = blockIdx.x * 32 + threadIdx.x;
    if (h >= p.H) return;
    float dwn = 0.0f, dwp = 0.0f, dg = 0.0f;
    for (int64_t t = 0; t < p.T; ++t) {
        const int64_t i = t * p.H + h;
        const float d = upstream<T>(p, t, h, p.w_next ? p.row_sum[t] : 0.0f);
        if (p.w_next) dwn += at<T>(p.d_u, i) * at<T>(p.saved_out, i) * p.r_next[t];
        if (p.y) {
            const float n = at<T>(p.y, i) * (p.w_post ? p.r_post[t] : 1.0f);
            dwp += p.alpha * gate_at<T>(p, t, h) * d * n;
            dg += p.alpha * d * n * (p.w_post ? at<T>(p.w_post, h) : 1.0f);
        }
        static_cast<T *>(p.d_res)[i] = from_f32<T>(d);  // after its last read of d_out: they may be one buffer
    }
    if (p.d_w_next) p.d_w_next[h] = dwn;
    if (p.d_w_post) p.d_w_post[h] = dwp;
    if (p.gate_kind == 1 && p.d_gate) static_cast<float *>(p.d_gate)[h] = dg;
}

template <typename T> cudaError_t launch_forward(const NormParams &p, cudaStream_t stream) {
    return launch_pdl(norm_kernel<T>, dim3(static_cast<unsigned>(p.T)), dim3(NORM_THREADS), 0, stream, p);
}

template <typename T> cudaError_t launch_backward(const NormParams &p, cudaStream_t stream) {
    if (p.T > 0) {
        cudaError_t e = launch_pdl(norm_backward_rows<T>, dim3(static_cast<unsigned>(p.T)), dim3(NORM_THREADS), 0,
                                   stream, p);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(norm_backward_columns<T>, dim3((p.H + 31) / 32), dim3(32), 0, stream, p);
}

}  // namespace

cudaError_t launch_residual_norm(const void *y, const void *res, const void *w_post, const void *gate, int gate_kind,
                                 float alpha, const void *w_next, float eps, int64_t T, int64_t H, int dtype,
                                 void *out, void *u, float *rstd_post, float *rstd_next, cudaStream_t stream) {
    NormParams p{};
    p.y = y;
    p.res = res;
    p.w_post = w_post;
    p.gate = gate;
    p.gate_kind = gate_kind;
    p.alpha = alpha;
    p.w_next = w_next;
    p.eps = eps;
    p.T = T;
    p.H = static_cast<int>(H);
    p.out = out;
    p.u = u;
    p.rstd_post = rstd_post;
    p.rstd_next = rstd_next;
    if (dtype == kF32) return launch_forward<float>(p, stream);
    if (dtype == kBF16) return launch_forward<__nv_bfloat16>(p, stream);
    return launch_forward<__half>(p, stream);
}

size_t residual_norm_backward_ws_bytes(int64_t T, int64_t H) {
    (void)H;
    return static_cast<size_t>(T) * 4 + 16;
}

cudaError_t launch_residual_norm_backward(const void *d_out, const void *d_u, const void *y, const void *out,
                                          const void *w_post, const void *gate, int gate_kind, float alpha,
                                          const void *w_next, const float *rstd_post, const float *rstd_next,
                                          int64_t T, int64_t H, int dtype, void *d_res, void *d_y, void *d_gate,
                                          float *d_w_post, float *d_w_next, void *ws, cudaStream_t stream) {
    NormParams p{};
    p.d_out = d_out;
    p.d_u = d_u;
    p.y = y;
    p.saved_out = out;
    p.w_post = w_post;
    p.gate = gate;
    p.gate_kind = gate_kind;
    p.alpha = alpha;
    p.w_next = w_next;
    p.r_post = rstd_post;
    p.r_next = rstd_next;
    p.T = T;
    p.H = static_cast<int>(H);
    p.d_res = d_res;
    p.d_y = d_y;
    p.d_gate = d_gate;
    p.d_w_post = d_w_post;
    p.d_w_next = d_w_next;
    p.row_sum = static_cast<float *>(ws);
    if (dtype == kF32) return launch_backward<float>(p, stream);
    if (dtype == kBF16) return launch_backward<__nv_bfloat16>(p, stream);
    return launch_backward<__half>(p, stream);
}

}  // namespace moe
