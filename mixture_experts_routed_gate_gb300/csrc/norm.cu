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
//
// Memory bound: every tensor is read once and written once.  A CTA holds one
// row at a time in registers, 8 (wide rows: 16) elements a thread, and walks
// the rows with the grid's stride; the rows to come arrive through a ring of
// shared-memory stages by bulk copies, so loads go on under the row's two
// reductions.  Rows whose bytes are no multiple of 16, and rows too wide for
// two stages, are loaded by the threads themselves.  The backward pass keeps
// the column sums of its rows in registers; a second kernel adds the CTAs'
// sums in a fixed order.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int NORM_MAX_TENSORS = 5;
constexpr int NORM_MAX_STAGES = 8;
constexpr int NORM_RING_BYTES = 200 * 1024;  // of one SM, shared by its CTAs

struct NormParams {
    const void *y, *res, *w_post, *gate, *w_next;
    const void *d_out, *d_u, *saved_out;
    const float *r_post, *r_next;
    void *out, *u, *d_res, *d_y, *d_gate;
    float *rstd_post, *rstd_next, *d_w_post, *d_w_next;
    float *partial;  // backward: [CTAs][3][H] column sums of d_w_next, d_w_post, d_gate
    int gate_kind;
    float alpha, eps;
    int64_t T;
    int H;
    int stages, tensors;  // the ring: tensors a row (in the order of the kernel's reads)
    const void *ring[NORM_MAX_TENSORS];
};

// A thread's EPT elements of a row.  RING: 16-byte vectors, `threads` apart,
// kept packed; otherwise single elements, `threads` apart, in fp32.
template <typename T, int EPT, bool RING> struct Part;

template <typename T, int EPT> struct Part<T, EPT, true> {
    static constexpr int EV = 16 / sizeof(T), V = EPT / EV;
    static constexpr int DT = std::is_same<T, __half>::value ? kF16 : kBF16;
    uint4 q[V];
    static __device__ __forceinline__ int at(int v) { return (v * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * EV; }
    __device__ __forceinline__ void load(const void *row, int H) {  // global or shared
#pragma unroll
        for (int v = 0; v < V; ++v)
            q[v] = at(v) < H ? *reinterpret_cast<const uint4 *>(static_cast<const T *>(row) + at(v)) : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void put(void *row, int H) const {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (at(v) < H) *reinterpret_cast<uint4 *>(static_cast<T *>(row) + at(v)) = q[v];
    }
    __device__ __forceinline__ void fill(float v) {
        uint32_t w;
        if constexpr (sizeof(T) == 4)
            w = __float_as_uint(v);
        else
            w = pack2<DT>(v, v);
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = make_uint4(w, w, w, w);
    }
    // The packed words as if read anew: otherwise the compiler keeps the
    // unpacked values across the reductions, twice the registers, and spills.
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int v = 0; v < V; ++v) asm volatile("" : "+r"(q[v].x), "+r"(q[v].y), "+r"(q[v].z), "+r"(q[v].w));
    }
    __device__ __forceinline__ uint32_t word(int i) const {  // the one that holds element i
        const uint4 &w = q[i / EV];
        const int j = i % EV * static_cast<int>(sizeof(T)) / 4;
        return j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(word(i));
        } else {
            const float2 f = unpack2<DT>(word(i));
            return i & 1 ? f.y : f.x;
        }
    }
    // this[i] * o[i], exact for 16-bit types: one mixed FMA, no unpacking
    __device__ __forceinline__ float times(const Part &o, int i) const {
        if constexpr (sizeof(T) == 4)
            return get(i) * o.get(i);
        else
            return i & 1 ? fma_mixed<DT, true>(word(i), o.word(i), 0.0f) : fma_mixed<DT, false>(word(i), o.word(i), 0.0f);
    }
    static __device__ __forceinline__ void store(void *row, int H, const float (&f)[EPT]) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (at(v) >= H) continue;
            uint4 w;
            if constexpr (sizeof(T) == 4) {
                w = make_uint4(__float_as_uint(f[4 * v]), __float_as_uint(f[4 * v + 1]), __float_as_uint(f[4 * v + 2]),
                               __float_as_uint(f[4 * v + 3]));
            } else {
                w = make_uint4(pack2<DT>(f[8 * v], f[8 * v + 1]), pack2<DT>(f[8 * v + 2], f[8 * v + 3]),
                               pack2<DT>(f[8 * v + 4], f[8 * v + 5]), pack2<DT>(f[8 * v + 6], f[8 * v + 7]));
            }
            *reinterpret_cast<uint4 *>(static_cast<T *>(row) + at(v)) = w;
        }
    }
    static __device__ __forceinline__ void store_sums(float *row, int H, const float (&f)[EPT]) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < EV; j += 4)
                if (at(v) < H)
                    *reinterpret_cast<float4 *>(row + at(v) + j) =
                        make_float4(f[v * EV + j], f[v * EV + j + 1], f[v * EV + j + 2], f[v * EV + j + 3]);
    }
};

template <typename T, int EPT> struct Part<T, EPT, false> {
    float f[EPT];
    static __device__ __forceinline__ int at(int i) { return i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x); }
    __device__ __forceinline__ void load(const void *row, int H) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) f[i] = at(i) < H ? to_f32(static_cast<const T *>(row)[at(i)]) : 0.0f;
    }
    __device__ __forceinline__ void put(void *, int) const {}
    __device__ __forceinline__ void fill(float v) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) f[i] = v;
    }
    __device__ __forceinline__ void again() {}
    __device__ __forceinline__ float get(int i) const { return f[i]; }
    __device__ __forceinline__ float times(const Part &o, int i) const { return f[i] * o.f[i]; }
    static __device__ __forceinline__ void store(void *row, int H, const float (&v)[EPT]) {
#pragma unroll
        for (int i = 0; i < EPT; ++i)
            if (at(i) < H) static_cast<T *>(row)[at(i)] = from_f32<T>(v[i]);
    }
    static __device__ __forceinline__ void store_sums(float *row, int H, const float (&v)[EPT]) {
#pragma unroll
        for (int i = 0; i < EPT; ++i)
            if (at(i) < H) row[at(i)] = v[i];
    }
};

// Sums over the CTA with one barrier each: two scratch buffers in turn.
struct RowSums {
    float2 *scratch;  // [2][32]
    int turn = 0;
    __device__ __forceinline__ float2 *barrier(float a, float b) {
        float2 *buf = scratch + turn * 32;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        return buf;
    }
    static __device__ __forceinline__ float lanes(float v) {
#pragma unroll
        for (int s = 16; s >= 1; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
        return v;
    }
    __device__ __forceinline__ float one(float a) {
        const float2 *buf = barrier(lanes(a), 0.0f);
        const int lane = threadIdx.x & 31;
        return lanes(lane < static_cast<int>(blockDim.x) >> 5 ? buf[lane].x : 0.0f);
    }
    __device__ __forceinline__ float2 two(float a, float b) {
        const float2 *buf = barrier(lanes(a), lanes(b));
        const int lane = threadIdx.x & 31;
        const float2 v = lane < static_cast<int>(blockDim.x) >> 5 ? buf[lane] : make_float2(0.0f, 0.0f);
        return make_float2(lanes(v.x), lanes(v.y));
    }
};

// The rows of p.ring's tensors, this CTA's in order.  next() waits for the
// next row's stage; refill() is called once every thread has read it.
template <bool RING> struct RowRing;

template <> struct RowRing<true> {
    const NormParams &p;
    uint8_t *smem;
    uint32_t bars, row_bytes, stage_bytes;
    int64_t row, ahead;  // the current row; the next one to ask for
    int stage = -1;
    uint32_t phase = 0;
    __device__ __forceinline__ RowRing(const NormParams &p, uint8_t *smem, uint64_t *bar, int elem)
        : p(p), smem(smem), bars(smem_u32(bar)), row_bytes(static_cast<uint32_t>(p.H * elem)),
          stage_bytes(row_bytes * p.tensors), row(blockIdx.x), ahead(blockIdx.x) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < p.stages; ++i) mbar_init(bars + 8u * i, 1);
            fence_mbar_init();
        }
        __syncthreads();
    }
    __device__ __forceinline__ void ask(int st) {  // thread 0
        if (ahead >= p.T) return;
        const uint32_t bar = bars + 8u * st, dst = smem_u32(smem) + st * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes);
        for (int i = 0; i < p.tensors; ++i)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             dst + i * row_bytes),
                         "l"(static_cast<const uint8_t *>(p.ring[i]) + ahead * row_bytes), "r"(row_bytes), "r"(bar)
                         : "memory");
        ahead += gridDim.x;
    }
    __device__ __forceinline__ void start() {
        if (threadIdx.x == 0)
            for (int i = 0; i < p.stages; ++i) ask(i);
    }
    // A copy of this CTA's own, asked for before: bounded, and without an
    // error word to report to a row that never came would be left as it is.
    __device__ __forceinline__ bool next() {
        if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
        }
        for (int i = 0; i < 64; ++i)  // before the slow read of the timer
            if (mbar_try_wait(bars + 8u * stage, phase)) return true;
        const unsigned long long start = global_timer_ns();
        while (!mbar_try_wait(bars + 8u * stage, phase))
            if (global_timer_ns() - start > kWaitTimeoutNs) return false;
        return true;
    }
    __device__ __forceinline__ const void *tensor(int i) const { return smem + stage * stage_bytes + i * row_bytes; }
    __device__ __forceinline__ void refill() {
        if (threadIdx.x == 0) ask(stage);
    }
};

template <> struct RowRing<false> {
    const NormParams &p;
    int64_t row, bytes;
    bool first = true;
    __device__ __forceinline__ RowRing(const NormParams &p, uint8_t *, uint64_t *, int elem)
        : p(p), row(blockIdx.x), bytes(static_cast<int64_t>(p.H) * elem) {}
    __device__ __forceinline__ void start() {}
    __device__ __forceinline__ bool next() { return true; }
    __device__ __forceinline__ const void *tensor(int i) const { return static_cast<const uint8_t *>(p.ring[i]) + row * bytes; }
    __device__ __forceinline__ void refill() {}
};

// The [H] tensors (weights, gate per channel): with the ring, a thread keeps
// its elements in shared memory after the stages, else it reads them again for
// every row; either way they take no registers between their uses.
template <typename P, bool RING>
__device__ __forceinline__ const void *keep_row(const void *row, uint8_t *&room, int H, int elem) {
    if (!RING || !row) return row;
    P part;
    part.load(row, H);
    uint8_t *at = room;
    room += H * elem;
    part.put(at, H);
    return at;
}

template <typename T, int EPT, bool RING, int MAX_THREADS, int MIN_CTAS>
__global__ void __launch_bounds__(MAX_THREADS, MIN_CTAS) norm_kernel(const __grid_constant__ NormParams p) {
    using P = Part<T, EPT, RING>;
    extern __shared__ __align__(128) uint8_t norm_smem[];
    __shared__ float2 scratch[64];
    __shared__ uint64_t bars[NORM_MAX_STAGES];
    RowRing<RING> ring(p, norm_smem, bars, sizeof(T));
    RowSums sums{scratch};
    griddep_wait();
    griddep_launch_dependents();
    ring.start();
    const int H = p.H;
    const bool has_y = p.y != nullptr, post = p.w_post != nullptr, nxt = p.w_next != nullptr;
    const float per = 1.0f / static_cast<float>(H);
    uint8_t *room = norm_smem + static_cast<int64_t>(p.stages) * p.tensors * H * sizeof(T);
    const void *w_post = keep_row<P, RING>(p.w_post, room, H, sizeof(T));
    const void *w_next = keep_row<P, RING>(p.w_next, room, H, sizeof(T));
    const void *gate_row = keep_row<P, RING>(p.gate_kind == 1 ? p.gate : nullptr, room, H, sizeof(T));
    for (; ring.row < p.T; ring.row += gridDim.x) {
        const int64_t t = ring.row, base = t * H;
        if (!ring.next()) return;
        float scale = p.alpha;
        if (p.gate_kind == 2) scale *= to_f32(static_cast<const T *>(p.gate)[t]);
        P res, y, gate;
        res.load(ring.tensor(0), H);
        if (has_y) y.load(ring.tensor(1), H);
        bool read = false;  // every thread has read the stage
        float o[EPT];
        if (has_y) {
            // what is absent counts as ones: no test per element
            if (p.gate_kind == 3)
                gate.load(ring.tensor(2), H);
            else if (p.gate_kind == 1)
                gate.load(gate_row, H);
            else
                gate.fill(1.0f);
            P w;
            float r2 = 1.0f;
            if (post) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < EPT; ++i) s = fmaf(y.get(i), y.get(i), s);
                r2 = rsqrtf(sums.one(s) * per + p.eps);
                if (p.rstd_post && threadIdx.x == 0) p.rstd_post[t] = r2;
                ring.refill();
                read = true;
                w.load(w_post, H);
            } else {
                w.fill(1.0f);
            }
#pragma unroll
            for (int i = 0; i < EPT; ++i) o[i] = fmaf(scale, y.get(i) * r2 * w.get(i) * gate.get(i), res.get(i));
            P::store(static_cast<T *>(p.out) + base, H, o);
        } else {
#pragma unroll
            for (int i = 0; i < EPT; ++i) o[i] = res.get(i);
        }
        if (nxt) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < EPT; ++i) s = fmaf(o[i], o[i], s);
            const float r = rsqrtf(sums.one(s) * per + p.eps);
            if (p.rstd_next && threadIdx.x == 0) p.rstd_next[t] = r;
            if (!read) ring.refill();
            read = true;
            P w;
            w.load(w_next, H);
#pragma unroll
            for (int i = 0; i < EPT; ++i) o[i] = o[i] * r * w.get(i);
            P::store(static_cast<T *>(p.u) + base, H, o);
        }
        if (!read) {
            if (RING) __syncthreads();
            ring.refill();
        }
    }
}

// The instructions of a row take as long as its bytes, so what a call has or
// lacks is no test per element: an absent weight is a row of ones, and the
// gate's three forms (a row, of ones where there is none; one factor a token;
// a factor an element) are three kernels.  4096 x 7168 bf16: 117 us with the
// tests, 84 us without.
template <typename T, int EPT, bool RING, int GATE, int MAX_THREADS, int MIN_CTAS>
__global__ void __launch_bounds__(MAX_THREADS, MIN_CTAS) norm_backward_kernel(const __grid_constant__ NormParams p) {
    using P = Part<T, EPT, RING>;
    constexpr bool TOKEN = GATE == 2, FULL = GATE == 3, ROW = !TOKEN && !FULL;
    extern __shared__ __align__(128) uint8_t norm_smem[];
    __shared__ float2 scratch[64];
    __shared__ uint64_t bars[NORM_MAX_STAGES];
    RowRing<RING> ring(p, norm_smem, bars, sizeof(T));
    RowSums sums{scratch};
    griddep_wait();
    griddep_launch_dependents();
    ring.start();
    const int H = p.H;
    const bool has_y = p.y != nullptr, post = p.w_post != nullptr, nxt = p.w_next != nullptr;
    const float per = 1.0f / static_cast<float>(H);
    uint8_t *room = norm_smem + static_cast<int64_t>(p.stages) * p.tensors * H * sizeof(T);
    const void *w_post = keep_row<P, RING>(p.w_post, room, H, sizeof(T));
    const void *w_next = keep_row<P, RING>(p.w_next, room, H, sizeof(T));
    const void *gate_row = keep_row<P, RING>(p.gate_kind == 1 ? p.gate : nullptr, room, H, sizeof(T));
    float sum_next[EPT], sum_post[EPT], sum_gate[EPT];  // columns, over this CTA's rows
#pragma unroll
    for (int i = 0; i < EPT; ++i) sum_next[i] = sum_post[i] = sum_gate[i] = 0.0f;
    for (; ring.row < p.T; ring.row += gridDim.x) {
        const int64_t t = ring.row, base = t * H;
        if (!ring.next()) return;
        int at = 0;
        bool read = false;  // every thread has read the stage
        float d[EPT];
        P d_out, d_u, out, y, gate, w;
        if (p.d_out)
            d_out.load(ring.tensor(at++), H);
        else
            d_out.fill(0.0f);
        if (nxt) {
            d_u.load(ring.tensor(at++), H);
            out.load(ring.tensor(at++), H);
        }
        if (has_y) y.load(ring.tensor(at++), H);
        if (FULL) gate.load(ring.tensor(at), H);
        if (nxt) {
            const float r = p.r_next[t];
            float s = 0.0f;
            w.load(w_next, H);
#pragma unroll
            for (int i = 0; i < EPT; ++i) s = fmaf(d_u.times(w, i), out.get(i), s);
            const float back = -(sums.one(s) * (r * r * r * per));
            ring.refill();
            read = true;
            d_u.again();
            w.again();
            out.again();
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                d[i] = fmaf(out.get(i), back, fmaf(r, d_u.times(w, i), d_out.get(i)));
                sum_next[i] = fmaf(r, d_u.times(out, i), sum_next[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPT; ++i) d[i] = d_out.get(i);
        }
        P::store(static_cast<T *>(p.d_res) + base, H, d);
        if (has_y) {
            const float r2 = post ? p.r_post[t] : 1.0f;
            const float factor = TOKEN ? p.alpha * to_f32(static_cast<const T *>(p.gate)[t]) : p.alpha;
            float s = 0.0f, sg = 0.0f;
            if (post)
                w.load(w_post, H);
            else
                w.fill(1.0f);
            if (ROW) {
                if (p.gate_kind == 1)
                    gate.load(gate_row, H);
                else
                    gate.fill(1.0f);
            }
            if (FULL && p.d_gate) {
                float dg[EPT];
#pragma unroll
                for (int i = 0; i < EPT; ++i) dg[i] = p.alpha * d[i] * (r2 * y.times(w, i));
                P::store(static_cast<T *>(p.d_gate) + base, H, dg);
            }
            const float alpha2 = p.alpha * r2;
#pragma unroll
            for (int i = 0; i < EPT; ++i) {  // d becomes dz * w_post
                if (ROW) sum_gate[i] = fmaf(alpha2 * d[i], y.times(w, i), sum_gate[i]);
                if (TOKEN) sg = fmaf(alpha2 * d[i], y.times(w, i), sg);
                float dz = factor * d[i];
                if (!TOKEN) dz *= gate.get(i);
                sum_post[i] = fmaf(dz * r2, y.get(i), sum_post[i]);
                d[i] = dz * w.get(i);
                s = fmaf(d[i], y.get(i), s);
            }
            if (post || TOKEN) {
                const float2 row = TOKEN ? sums.two(s, sg) : make_float2(sums.one(s), 0.0f);
                if (!read) ring.refill();
                read = true;
                if (TOKEN && p.d_gate && threadIdx.x == 0) static_cast<float *>(p.d_gate)[t] = row.y;
                if (post) {
                    const float back = -(row.x * (r2 * r2 * r2 * per));
                    y.again();
#pragma unroll
                    for (int i = 0; i < EPT; ++i) d[i] = fmaf(y.get(i), back, r2 * d[i]);
                }
            }
            P::store(static_cast<T *>(p.d_y) + base, H, d);
        }
        if (!read) {
            if (RING) __syncthreads();
            ring.refill();
        }
    }
    float *part = p.partial + static_cast<int64_t>(blockIdx.x) * 3 * H;
    if (p.d_w_next) P::store_sums(part, H, sum_next);
    if (p.d_w_post) P::store_sums(part + H, H, sum_post);
    if (p.gate_kind == 1 && p.d_gate) P::store_sums(part + 2 * H, H, sum_gate);
}

// The CTAs' column sums added: 32 columns a CTA, 8 threads a column each with
// every 8th CTA's sum, then those in order.
__global__ void __launch_bounds__(256) norm_columns_kernel(const __grid_constant__ NormParams p, int ctas) {
    __shared__ float part[8][33];
    griddep_wait();
    griddep_launch_dependents();
    const int which = blockIdx.y, c = threadIdx.x & 31, k = threadIdx.x >> 5, h = blockIdx.x * 32 + c;
    float *dst = which == 0 ? p.d_w_next : which == 1 ? p.d_w_post : (p.gate_kind == 1 ? static_cast<float *>(p.d_gate) : nullptr);
    if (!dst) return;
    float s = 0.0f;
    if (h < p.H) {
        const float *src = p.partial + static_cast<int64_t>(which) * p.H + h;
#pragma unroll 8
        for (int i = k; i < ctas; i += 8) s += src[static_cast<int64_t>(i) * 3 * p.H];
    }
    part[k][c] = s;
    __syncthreads();
    if (k == 0 && h < p.H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][c];
        dst[h] = s;
    }
}

// Threads of a CTA, CTAs of an SM and of the grid, and whether the rows go
// through the ring, by H, the type and the tensors of a row.
struct NormShape {
    int ept, threads, ctas, stages;
    bool ring;
    size_t smem;
};

NormShape norm_shape(const NormParams &p, int elem, bool backward) {
    NormShape s{};
    const int64_t row_bytes = static_cast<int64_t>(p.H) * elem, stage = row_bytes * p.tensors;
    const int kept = (p.w_post ? 1 : 0) + (p.w_next ? 1 : 0) + (p.gate_kind == 1 ? 1 : 0);
    int64_t room = 0;
    int per_sm = 1;
    auto size = [&](int ept) {
        s.ept = ept;
        s.threads = ((p.H + ept - 1) / ept + 31) / 32 * 32;
        // narrow rows: several CTAs an SM (the backward pass holds more registers)
        per_sm = (backward ? 896 : 1024) / s.threads;
        per_sm = per_sm < 1 || (backward && ept == 16) ? 1 : per_sm > 16 ? 16 : per_sm;
        room = NORM_RING_BYTES / per_sm - kept * row_bytes;
        s.ring = row_bytes % 16 == 0 && room >= 2 * stage;
    };
    // Forward: 16 elements a thread above 4096, for two CTAs an SM.  Backward:
    // 8 with the ring as long as the registers allow (72 at 896 threads).
    size(p.H <= (backward ? 7168 : 4096) ? 8 : 16);
    if (!s.ring && p.H > 4096) size(16);
    const int64_t all = static_cast<int64_t>(device_sm_count()) * per_sm;
    s.ctas = static_cast<int>(p.T < all ? p.T : all);
    if (s.ring) {
        const int64_t rows = (p.T + s.ctas - 1) / (s.ctas > 0 ? s.ctas : 1), fit = room / stage;
        s.stages = static_cast<int>(fit < NORM_MAX_STAGES ? fit : NORM_MAX_STAGES);
        if (rows < s.stages) s.stages = static_cast<int>(rows);
        s.smem = static_cast<size_t>(s.stages * stage + kept * row_bytes);
    }
    return s;
}

cudaError_t launch_kernel(void (*kern)(NormParams), std::atomic<bool> *attr_done, const NormParams &p, const NormShape &s,
                          cudaStream_t stream) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (s.ring && (dev < 0 || dev >= 64 || !attr_done[dev])) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, NORM_RING_BYTES);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    return launch_pdl(kern, dim3(static_cast<unsigned>(s.ctas)), dim3(static_cast<unsigned>(s.threads)), s.smem, stream, p);
}

template <typename T, int EPT, bool RING, int MAX_THREADS, int MIN_CTAS>
cudaError_t launch_forward(const NormParams &p, const NormShape &s, cudaStream_t stream) {
    static std::atomic<bool> attr_done[64];  // zero-initialised; several host threads may launch
    return launch_kernel(norm_kernel<T, EPT, RING, MAX_THREADS, MIN_CTAS>, attr_done, p, s, stream);
}

template <typename T, int EPT, bool RING, int MAX_THREADS, int MIN_CTAS>
cudaError_t launch_backward(const NormParams &p, const NormShape &s, cudaStream_t stream) {
    static std::atomic<bool> attr_done[3][64];  // zero-initialised; several host threads may launch
    if (p.gate_kind == 2)
        return launch_kernel(norm_backward_kernel<T, EPT, RING, 2, MAX_THREADS, MIN_CTAS>, attr_done[1], p, s, stream);
    if (p.gate_kind == 3)
        return launch_kernel(norm_backward_kernel<T, EPT, RING, 3, MAX_THREADS, MIN_CTAS>, attr_done[2], p, s, stream);
    return launch_kernel(norm_backward_kernel<T, EPT, RING, 1, MAX_THREADS, MIN_CTAS>, attr_done[0], p, s, stream);
}

// Registers by the CTA's threads: the forward pass has 64; the backward pass
// 80 up to 256 threads, 128 up to 512, 72 up to 896 (rows of 7168), 64 above.
template <typename T> cudaError_t launch_shape(const NormParams &p, const NormShape &s, bool backward, cudaStream_t stream) {
    if (!backward) {
        if (s.ept == 16) {
            if (s.threads <= 512)
                return s.ring ? launch_forward<T, 16, true, 512, 2>(p, s, stream) : launch_forward<T, 16, false, 512, 2>(p, s, stream);
            return s.ring ? launch_forward<T, 16, true, 1024, 1>(p, s, stream) : launch_forward<T, 16, false, 1024, 1>(p, s, stream);
        }
        return s.ring ? launch_forward<T, 8, true, 512, 2>(p, s, stream) : launch_forward<T, 8, false, 512, 2>(p, s, stream);
    }
    if (s.ept == 16) {
        if (s.threads <= 512)
            return s.ring ? launch_backward<T, 16, true, 512, 1>(p, s, stream) : launch_backward<T, 16, false, 512, 1>(p, s, stream);
        return s.ring ? launch_backward<T, 16, true, 1024, 1>(p, s, stream) : launch_backward<T, 16, false, 1024, 1>(p, s, stream);
    }
    if (!s.ring) return launch_backward<T, 8, false, 512, 1>(p, s, stream);
    if (s.threads <= 256) return launch_backward<T, 8, true, 256, 3>(p, s, stream);
    if (s.threads <= 512) return launch_backward<T, 8, true, 512, 1>(p, s, stream);
    return launch_backward<T, 8, true, 896, 1>(p, s, stream);
}

template <typename T> cudaError_t launch_typed(NormParams p, bool backward, cudaStream_t stream) {
    const NormShape s = norm_shape(p, sizeof(T), backward);
    p.stages = s.stages;
    if (p.T > 0) {
        const cudaError_t e = launch_shape<T>(p, s, backward, stream);
        if (e != cudaSuccess) return e;
    }
    if (!backward || (!p.d_w_next && !p.d_w_post && !(p.d_gate && p.gate_kind == 1))) return cudaSuccess;
    return launch_pdl(norm_columns_kernel, dim3(static_cast<unsigned>((p.H + 31) / 32), 3), dim3(256), 0, stream, p, s.ctas);
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
    p.ring[p.tensors++] = res;
    if (y) p.ring[p.tensors++] = y;
    if (gate_kind == 3) p.ring[p.tensors++] = gate;
    if (dtype == kF32) return launch_typed<float>(p, false, stream);
    if (dtype == kBF16) return launch_typed<__nv_bfloat16>(p, false, stream);
    return launch_typed<__half>(p, false, stream);
}

size_t residual_norm_backward_ws_bytes(int64_t T, int64_t H) {
    // three rows of column sums for each CTA of the largest grid
    const int64_t ctas = static_cast<int64_t>(device_sm_count()) * 16;
    return static_cast<size_t>((T < ctas ? T : ctas) * 3 * H * 4 + 16);
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
    p.partial = static_cast<float *>(ws);
    // in the order of the kernel's reads
    if (d_out) p.ring[p.tensors++] = d_out;
    if (w_next) {
        p.ring[p.tensors++] = d_u;
        p.ring[p.tensors++] = out;
    }
    if (y) p.ring[p.tensors++] = y;
    if (gate_kind == 3) p.ring[p.tensors++] = gate;
    if (dtype == kF32) return launch_typed<float>(p, true, stream);
    if (dtype == kBF16) return launch_typed<__nv_bfloat16>(p, true, stream);
    return launch_typed<__half>(p, true, stream);
}

}  // namespace moe
