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
// row at a time, 8 (wide rows: 16) elements a thread, and walks the rows with
// the grid's stride; the rows to come arrive through a ring of shared-memory
// slots, one tensor's row each, by bulk copies, so loads go on under the row's
// two reductions.  Rows that start on 16 bytes are read from there as 16-byte
// vectors, others (an odd H) element by element.  The backward pass keeps the
// column sums of its rows in registers; a second kernel adds the CTAs' sums in
// a fixed order.
//
// 4096 x 7168 bf16: forward 39 us (235 MB at 6.0 TB/s, against 35 at this
// card's copy rate; 67% of the issue slots), gradients 88 us (52 at the copy
// rate; 57% of the issue slots at about 500 instructions a warp and row, and the
// largest stall, 2.8 warps an issue, is on the row's statistics and gate, read
// from memory in the row they serve).  fp32: 81 and 131 us of 69 and 104; two
// rows' slots do not fit, so the slots are single tensors', a part of a row
// ahead if need be (147 and 315 us with such rows read from memory).  Rows of
// 7167 bf16, by elements: 68 and 150 us (from memory 154 and 465).
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int NORM_MAX_TENSORS = 5;
constexpr int NORM_MAX_SLOTS = 32, NORM_MAX_BARS = NORM_MAX_SLOTS + 2;
constexpr int NORM_RING_BYTES = 224 * 1024;  // of one SM, shared by its CTAs

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
    int slots, tensors;  // the ring; tensors a row (in the order of the kernel's reads)
    int bars;
    uint32_t slot_bytes, ring_bytes;
    const void *ring[NORM_MAX_TENSORS];
};

// How rows are read: through the ring, as 16-byte vectors or (rows that do not
// all start on 16 bytes) by elements; or, too wide for the ring, from memory.
enum class Rows { kVectors, kOdd, kMemory };

// A thread's EPT elements of a row, packed in registers.  VEC: 16-byte vectors,
// `threads` apart, of a row that starts on 16 bytes; otherwise single
// elements, `threads` apart.
template <typename T, int EPT, bool VEC> struct Part {
    static constexpr int DT = std::is_same<T, __half>::value ? kF16 : kBF16;
    static constexpr int PER = 4 / sizeof(T), WORDS = EPT / PER;  // elements of a word
    static constexpr int RUN = VEC ? 16 / sizeof(T) : 1;          // consecutive elements
    using Bits = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
    uint32_t w[WORDS];
    // the row's index of the thread's element i
    static __device__ __forceinline__ int at(int i) {
        return (i / RUN * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * RUN + i % RUN;
    }
    __device__ __forceinline__ void load(const void *row, int H) {  // global or shared
        if constexpr (VEC) {
#pragma unroll
            for (int v = 0; v < WORDS / 4; ++v) {
                const int i = at(v * RUN);
                const uint4 q = i < H ? *reinterpret_cast<const uint4 *>(static_cast<const T *>(row) + i) : make_uint4(0u, 0u, 0u, 0u);
                w[4 * v] = q.x;
                w[4 * v + 1] = q.y;
                w[4 * v + 2] = q.z;
                w[4 * v + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < WORDS; ++k) {
                w[k] = 0u;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int i = at(k * PER + j);
                    if (i < H) w[k] |= static_cast<uint32_t>(static_cast<const Bits *>(row)[i]) << (16 * j);
                }
            }
        }
    }
    __device__ __forceinline__ void put(void *row, int H) const {
        if constexpr (VEC) {
#pragma unroll
            for (int v = 0; v < WORDS / 4; ++v)
                if (at(v * RUN) < H)
                    *reinterpret_cast<uint4 *>(static_cast<T *>(row) + at(v * RUN)) =
                        make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                if (at(i) < H) static_cast<Bits *>(row)[at(i)] = static_cast<Bits>(w[i / PER] >> (16 * (i % PER)));
        }
    }
    __device__ __forceinline__ void fill(float v) {
        uint32_t x;
        if constexpr (sizeof(T) == 4)
            x = __float_as_uint(v);
        else
            x = pack2<DT>(v, v);
#pragma unroll
        for (int k = 0; k < WORDS; ++k) w[k] = x;
    }
    // the thread's words of its own in shared memory, and back
    __device__ __forceinline__ void keep(uint8_t *room) const {
        constexpr int N = VEC ? 4 : 1;
#pragma unroll
        for (int k = 0; k < WORDS; k += N) {
            uint8_t *at = room + (k * blockDim.x + threadIdx.x * N) * 4;
            if constexpr (VEC)
                *reinterpret_cast<uint4 *>(at) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
            else
                *reinterpret_cast<uint32_t *>(at) = w[k];
        }
    }
    __device__ __forceinline__ void again(const void *room) {
        constexpr int N = VEC ? 4 : 1;
#pragma unroll
        for (int k = 0; k < WORDS; k += N) {
            const uint8_t *at = static_cast<const uint8_t *>(room) + (k * blockDim.x + threadIdx.x * N) * 4;
            if constexpr (VEC) {
                const uint4 q = *reinterpret_cast<const uint4 *>(at);
                w[k] = q.x;
                w[k + 1] = q.y;
                w[k + 2] = q.z;
                w[k + 3] = q.w;
            } else {
                w[k] = *reinterpret_cast<const uint32_t *>(at);
            }
        }
    }
    // The packed words as if read anew: otherwise the compiler keeps the
    // unpacked values across the reductions, twice the registers, and spills.
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int k = 0; k < WORDS; ++k) asm volatile("" : "+r"(w[k]));
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w[i]);
        } else {
            const float2 f = unpack2<DT>(w[i / 2]);
            return i & 1 ? f.y : f.x;
        }
    }
    // this[i] * o[i], exact for 16-bit types: one mixed FMA, no unpacking
    __device__ __forceinline__ float times(const Part &o, int i) const {
        if constexpr (sizeof(T) == 4)
            return get(i) * o.get(i);
        else
            return i & 1 ? fma_mixed<DT, true>(w[i / 2], o.w[i / 2], 0.0f) : fma_mixed<DT, false>(w[i / 2], o.w[i / 2], 0.0f);
    }
    static __device__ __forceinline__ void store(void *row, int H, const float (&f)[EPT]) {
        Part out;
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            if constexpr (sizeof(T) == 4)
                out.w[k] = __float_as_uint(f[k]);
            else
                out.w[k] = pack2<DT>(f[2 * k], f[2 * k + 1]);
        }
        out.put(row, H);
    }
    static __device__ __forceinline__ void store_sums(float *row, int H, const float (&f)[EPT]) {
#pragma unroll
        for (int i = 0; i < EPT; i += VEC ? 4 : 1) {
            if (at(i) >= H) continue;
            if constexpr (VEC)
                *reinterpret_cast<float4 *>(row + at(i)) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
            else
                row[at(i)] = f[i];
        }
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
// next row; refill() is called once every thread has read it.
// Thread 0's: the next copy is the row at this byte of the tensors, of this
// tensor, into this shared-memory address and for this barrier.  In shared
// memory, as registers are what the backward pass lacks.
struct RowAsk {
    int64_t from;
    int tensor;
    uint32_t slot, bar;
};
struct RowState {
    uint64_t bars[NORM_MAX_BARS];
    RowAsk ask;
    int lost;  // a wait gave up
};

template <Rows MODE> struct RowRing;

template <> struct RowRing<Rows::kMemory> {
    const NormParams &p;
    int64_t row, row_bytes;
    __device__ __forceinline__ RowRing(const NormParams &p, uint8_t *, RowState &, int elem)
        : p(p), row(blockIdx.x), row_bytes(static_cast<int64_t>(p.H) * elem) {}
    __device__ __forceinline__ void start() {}
    __device__ __forceinline__ void next() { tensor = 0; }
    template <typename T> __device__ __forceinline__ void finish(bool) {}
    int tensor = 0;
    __device__ __forceinline__ const void *take() { return static_cast<const uint8_t *>(p.ring[tensor++]) + row * row_bytes; }
    __device__ __forceinline__ void refill() {}
};

// p.slots slots of one tensor's row each, filled in the order of the reads, a
// row ahead as far as they go (not a whole number of rows), and a barrier for
// each row in flight.  kOdd copies from the 16 bytes a row starts in to those
// it ends in; what is left of the tensors after their last whole 16 bytes is
// copied by the threads, into slots that no bulk copy fills again (the rows that
// come after have nothing left to copy).
template <Rows MODE> struct RowRing {
    const NormParams &p;
    uint8_t *smem;
    uint32_t bars;
    int64_t row_bytes, row;
    RowState &state;
    uint32_t slot = 0;  // of the next tensor, in bytes
    int bar = -1;       // the row's
    uint32_t phase = 0;
    __device__ __forceinline__ RowRing(const NormParams &p, uint8_t *smem, RowState &state, int elem)
        : p(p), smem(smem), bars(smem_u32(state.bars)), row_bytes(static_cast<int64_t>(p.H) * elem), row(blockIdx.x),
          state(state) {
        if (threadIdx.x == 0) {
            state.ask = RowAsk{blockIdx.x * row_bytes, 0, smem_u32(smem), bars};
            state.lost = 0;
            for (int i = 0; i < p.bars; ++i) mbar_init(bars + 8u * i, 1);
            fence_mbar_init();
        }
        __syncthreads();
    }
    __device__ __forceinline__ void ask(int copies) {
        const int64_t total = p.T * row_bytes;
        RowAsk a = state.ask;
        for (int i = 0; i < copies && a.from < total; ++i) {
            int64_t from = a.from;
            uint32_t bytes = static_cast<uint32_t>(row_bytes);
            if constexpr (MODE == Rows::kOdd) {
                int64_t to = (from + row_bytes + 15) & ~int64_t{15};
                to = to < total ? to : total & ~int64_t{15};
                from &= ~int64_t{15};
                bytes = static_cast<uint32_t>(to - from);
            }
            if (a.tensor == 0) mbar_arrive_expect_tx(a.bar, bytes * p.tensors);
            if (MODE != Rows::kOdd || bytes > 0)
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(a.slot),
                             "l"(static_cast<const uint8_t *>(p.ring[a.tensor]) + from), "r"(bytes), "r"(a.bar)
                             : "memory");
            a.slot += p.slot_bytes;
            if (a.slot == smem_u32(smem) + p.ring_bytes) a.slot = smem_u32(smem);
            if (++a.tensor == p.tensors) {
                a.tensor = 0;
                a.from += gridDim.x * row_bytes;
                a.bar += 8;
                if (a.bar == bars + 8u * p.bars) a.bar = bars;
            }
        }
        state.ask = a;
    }
    __device__ __forceinline__ bool lost() const { return *static_cast<volatile int *>(&state.lost) != 0; }
    __device__ __forceinline__ void start() {
        if (threadIdx.x == 0) ask(p.slots);
    }
    // For this CTA's own copies, asked for before; bounded all the same.  There is
    // no error word to report to: once a wait gives up, nothing more is asked for,
    // the CTA runs on with what its slots hold, and ends in finish().
    __device__ __forceinline__ void wait() {
        for (int i = 0; i < 64; ++i)  // before the slow read of the timer
            if (mbar_try_wait(bars + 8u * bar, phase & 1u) || lost()) return;
        const unsigned long long begin = global_timer_ns();
        while (!mbar_try_wait(bars + 8u * bar, phase & 1u) && !lost())
            if (global_timer_ns() - begin > kWaitTimeoutNs) *static_cast<volatile int *>(&state.lost) = 1;
    }
    // After the last row.  If a row was lost: NaN for all of the CTA's rows and its
    // column sums, and the copies still on their way land before shared memory
    // goes (2 s in all).
    template <typename T> __device__ __forceinline__ void finish(bool backward) {
        __syncthreads();
        if (!lost()) return;
        T *const wide[] = {static_cast<T *>(backward ? p.d_res : p.out), static_cast<T *>(backward ? p.d_y : p.u),
                           static_cast<T *>(p.gate_kind == 3 ? p.d_gate : nullptr)};
        float *const narrow[] = {p.rstd_post, p.rstd_next, static_cast<float *>(p.gate_kind == 2 ? p.d_gate : nullptr)};
#pragma unroll 1
        for (int i = 0; i < 3; ++i) {
#pragma unroll 1
            for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
#pragma unroll 1
                for (int h = threadIdx.x; wide[i] && h < p.H; h += blockDim.x) wide[i][t * p.H + h] = from_f32<T>(NAN);
                if (narrow[i] && threadIdx.x == 0) narrow[i][t] = NAN;
            }
        }
#pragma unroll 1
        for (int h = threadIdx.x; backward && h < 3 * p.H; h += blockDim.x)
            p.partial[static_cast<int64_t>(blockIdx.x) * 3 * p.H + h] = NAN;
        const int asked = static_cast<int>((state.ask.from / row_bytes - blockIdx.x) / gridDim.x) + (state.ask.tensor != 0);
        const unsigned long long begin = global_timer_ns();
#pragma unroll 1
        for (int k = max(0, asked - p.bars); k < asked && threadIdx.x == 0; ++k)
            while (!mbar_try_wait(bars + 8u * (k % p.bars), (k / p.bars) & 1))
                if (global_timer_ns() - begin > kWaitTimeoutNs) return;
    }
    __device__ __forceinline__ void next() {
        if (++bar == p.bars) {
            bar = 0;
            phase ^= 1u;
        }
        wait();
        if constexpr (MODE == Rows::kOdd) {
            // rows of less than 16 bytes: several may reach past the last whole 16
            const int64_t whole = p.T * row_bytes / 16 * 16;
            if ((row + 1) * row_bytes > whole) {
                int64_t from = whole - row * row_bytes;
                from = from < 0 ? 0 : from;
                const uint32_t first = slot;
                for (int i = 0; i < p.tensors; ++i) {
                    uint8_t *to = take();
                    if (threadIdx.x < row_bytes - from)
                        to[from + threadIdx.x] = static_cast<const uint8_t *>(p.ring[i])[row * row_bytes + from + threadIdx.x];
                }
                slot = first;
                __syncthreads();
            }
        }
    }
    // the row's tensors in their order
    __device__ __forceinline__ uint8_t *take() {
        uint8_t *at = smem + slot;
        slot += p.slot_bytes;
        if (slot == p.ring_bytes) slot = 0;
        return MODE == Rows::kOdd ? at + (row * row_bytes & 15) : at;
    }
    __device__ __forceinline__ void refill() {
        if (threadIdx.x == 0 && !lost()) ask(p.tensors);
    }
};

// The [H] tensors (weights, gate per channel): with the ring, a thread keeps
// its elements in shared memory after the slots, else it reads them again for
// every row; either way they take no registers between their uses.
template <typename P, Rows MODE> struct Kept {
    const void *at = nullptr;
    __device__ __forceinline__ Kept(const void *row, uint8_t *&room, int H) {
        if constexpr (MODE == Rows::kMemory) {
            at = row;
        } else if (row) {
            P part;
            part.load(row, H);
            at = room;
            part.keep(room);
            room += P::WORDS * 4 * blockDim.x;
        }
    }
    __device__ __forceinline__ void load(P &part, int H) const {
        if constexpr (MODE == Rows::kMemory)
            part.load(at, H);
        else
            part.again(at);
    }
};

template <typename T, int EPT, Rows MODE, int MAX_THREADS, int MIN_CTAS>
__global__ void __launch_bounds__(MAX_THREADS, MIN_CTAS) norm_kernel(const __grid_constant__ NormParams p) {
    using P = Part<T, EPT, MODE == Rows::kVectors>;
    extern __shared__ __align__(128) uint8_t norm_smem[];
    __shared__ float2 scratch[64];
    __shared__ RowState state;
    RowRing<MODE> ring(p, norm_smem, state, sizeof(T));
    RowSums sums{scratch};
    griddep_wait();
    griddep_launch_dependents();
    ring.start();
    const int H = p.H;
    const bool has_y = p.y != nullptr, post = p.w_post != nullptr, nxt = p.w_next != nullptr;
    const float per = 1.0f / static_cast<float>(H);
    uint8_t *room = norm_smem + p.ring_bytes;
    const Kept<P, MODE> w_post(p.w_post, room, H);
    const Kept<P, MODE> w_next(p.w_next, room, H);
    const Kept<P, MODE> gate_row(p.gate_kind == 1 ? p.gate : nullptr, room, H);
    for (; ring.row < p.T; ring.row += gridDim.x) {
        const int64_t t = ring.row, base = t * H;
        ring.next();
        float scale = p.alpha;
        if (p.gate_kind == 2) scale *= to_f32(static_cast<const T *>(p.gate)[t]);
        P res, y, gate;
        res.load(ring.take(), H);
        if (has_y) y.load(ring.take(), H);
        bool read = false;  // every thread has read the row's slots
        float o[EPT];
        if (has_y) {
            // what is absent counts as ones: no test per element
            if (p.gate_kind == 3)
                gate.load(ring.take(), H);
            else if (p.gate_kind == 1)
                gate_row.load(gate, H);
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
                w_post.load(w, H);
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
            w_next.load(w, H);
#pragma unroll
            for (int i = 0; i < EPT; ++i) o[i] = o[i] * r * w.get(i);
            P::store(static_cast<T *>(p.u) + base, H, o);
        }
        if (!read) {
            __syncthreads();
            ring.refill();
        }
    }
    ring.template finish<T>(false);
}

// The instructions of a row take longer than its bytes, so what a call has or
// lacks is no test per element: an absent weight is a row of ones, and the
// gate's three forms (a row, of ones where there is none; one factor a token;
// a factor an element) are three kernels.  4096 x 7168 bf16: 117 us with the
// tests, 88 us without.
template <typename T, int EPT, Rows MODE, int GATE, int MAX_THREADS, int MIN_CTAS>
__global__ void __launch_bounds__(MAX_THREADS, MIN_CTAS) norm_backward_kernel(const __grid_constant__ NormParams p) {
    using P = Part<T, EPT, MODE == Rows::kVectors>;
    constexpr bool TOKEN = GATE == 2, FULL = GATE == 3, ROW = !TOKEN && !FULL;
    extern __shared__ __align__(128) uint8_t norm_smem[];
    __shared__ float2 scratch[64];
    __shared__ RowState state;
    RowRing<MODE> ring(p, norm_smem, state, sizeof(T));
    RowSums sums{scratch};
    griddep_wait();
    griddep_launch_dependents();
    ring.start();
    const int H = p.H;
    const bool has_y = p.y != nullptr, post = p.w_post != nullptr, nxt = p.w_next != nullptr;
    const float per = 1.0f / static_cast<float>(H);
    uint8_t *room = norm_smem + p.ring_bytes;
    const Kept<P, MODE> w_post(p.w_post, room, H);
    const Kept<P, MODE> w_next(p.w_next, room, H);
    const Kept<P, MODE> gate_row(p.gate_kind == 1 ? p.gate : nullptr, room, H);
    float sum_next[EPT], sum_post[EPT], sum_gate[EPT];  // columns, over this CTA's rows
#pragma unroll
    for (int i = 0; i < EPT; ++i) sum_next[i] = sum_post[i] = sum_gate[i] = 0.0f;
    for (; ring.row < p.T; ring.row += gridDim.x) {
        const int64_t t = ring.row, base = t * H;
        ring.next();
        bool read = false;  // every thread has read the row's slots
        float d[EPT];
        P d_out, d_u, out, y, gate, w;
        if (p.d_out)
            d_out.load(ring.take(), H);
        else
            d_out.fill(0.0f);
        if (nxt) {
            d_u.load(ring.take(), H);
            out.load(ring.take(), H);
        }
        if (has_y) y.load(ring.take(), H);
        if (FULL) gate.load(ring.take(), H);
        if (nxt) {
            const float r = p.r_next[t];
            float s = 0.0f;
            w_next.load(w, H);
#pragma unroll
            for (int i = 0; i < EPT; ++i) s = fmaf(d_u.times(w, i), out.get(i), s);
            const float back = -(sums.one(s) * r * per) * r;  // r^3 alone leaves fp32 at an rms of 1e13
            ring.refill();
            read = true;
            d_u.again();
            w.again();
            out.again();
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                d[i] = fmaf(r, fmaf(out.get(i), back, d_u.times(w, i)), d_out.get(i));
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
                w_post.load(w, H);
            else
                w.fill(1.0f);
            if (ROW) {
                if (p.gate_kind == 1)
                    gate_row.load(gate, H);
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
                    const float back = -(row.x * r2 * per) * r2;
                    y.again();
#pragma unroll
                    for (int i = 0; i < EPT; ++i) d[i] = r2 * fmaf(y.get(i), back, d[i]);
                }
            }
            P::store(static_cast<T *>(p.d_y) + base, H, d);
        }
        if (!read) {
            __syncthreads();
            ring.refill();
        }
    }
    float *part = p.partial + static_cast<int64_t>(blockIdx.x) * 3 * H;
    if (p.d_w_next) P::store_sums(part, H, sum_next);
    if (p.d_w_post) P::store_sums(part + H, H, sum_post);
    if (p.gate_kind == 1 && p.d_gate) P::store_sums(part + 2 * H, H, sum_gate);
    ring.template finish<T>(true);
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

// Threads of a CTA, CTAs of an SM and of the grid, and the ring, by H, the
// type and the tensors of a row.
struct NormShape {
    int ept, threads, ctas;
    Rows mode;
    size_t smem;
};

// Backward: 8 elements a thread as long as the registers allow (72 at 896
// threads); narrow rows: several CTAs an SM (fewer than in the forward pass, as
// it holds more registers).
int norm_threads(int64_t H, int ept) { return static_cast<int>(((H + ept - 1) / ept + 31) / 32 * 32); }
int backward_ept(int64_t H) { return H <= 7168 ? 8 : 16; }
int backward_per_sm(int64_t H) {
    const int n = backward_ept(H) == 16 ? 1 : 896 / norm_threads(H, 8);
    return n < 1 ? 1 : n > 16 ? 16 : n;
}

NormShape norm_shape(NormParams &p, int elem, bool backward) {
    NormShape s{};
    const int64_t row_bytes = static_cast<int64_t>(p.H) * elem, padded = (row_bytes + 15) / 16 * 16;
    // Forward, 16-bit types: 16 elements a thread above 4096, for two CTAs an
    // SM (4096 x 7168 bf16 with its graph's overhead 46 us, one CTA of 8 elements
    // a thread 62); fp32 rows that wide leave two CTAs no room for a ring (81 us
    // with one CTA, 145 with two).
    s.ept = backward ? backward_ept(p.H) : p.H <= (elem == 4 ? 8192 : 4096) ? 8 : 16;
    s.threads = norm_threads(p.H, s.ept);
    int per_sm = 1024 / s.threads;
    per_sm = backward ? backward_per_sm(p.H) : per_sm < 1 ? 1 : per_sm > 16 ? 16 : per_sm;
    const int64_t kept = ((p.w_post ? 1 : 0) + (p.w_next ? 1 : 0) + (p.gate_kind == 1 ? 1 : 0)) *
                         static_cast<int64_t>(s.ept) * s.threads * elem;
    const bool odd = row_bytes % 16 != 0;
    p.slot_bytes = static_cast<uint32_t>(odd ? padded + 16 : row_bytes);
    auto fit = [&](int ctas) { return (NORM_RING_BYTES / ctas - 2048 - kept) / static_cast<int64_t>(p.slot_bytes); };
    while (per_sm > 1 && fit(per_sm) < p.tensors) --per_sm;
    const int64_t all = static_cast<int64_t>(device_sm_count()) * per_sm;
    s.ctas = static_cast<int>(p.T < all ? p.T : all);
    const int64_t rows = (p.T + s.ctas - 1) / s.ctas;
    int64_t slots = fit(per_sm);
    if (slots > NORM_MAX_SLOTS) slots = NORM_MAX_SLOTS;
    if (slots < p.tensors) {
        s.mode = Rows::kMemory;
        return s;
    }
    if (slots > rows * p.tensors) slots = rows * p.tensors;
    s.mode = odd ? Rows::kOdd : Rows::kVectors;
    p.slots = static_cast<int>(slots);
    p.ring_bytes = p.slots * p.slot_bytes;
    p.bars = p.slots / p.tensors + 2;  // the rows in the slots, wholly or in part, and the current one's
    s.smem = static_cast<size_t>(p.ring_bytes + kept);
    return s;
}

cudaError_t launch_kernel(void (*kern)(NormParams), std::atomic<bool> *attr_done, const NormParams &p, const NormShape &s,
                          cudaStream_t stream) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    // 48 KB need no leave, the kernel's own arrays included
    if (s.smem > 40 * 1024 && (dev < 0 || dev >= 64 || !attr_done[dev])) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, NORM_RING_BYTES);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    return launch_pdl(kern, dim3(static_cast<unsigned>(s.ctas)), dim3(static_cast<unsigned>(s.threads)), s.smem, stream, p);
}

template <typename T, int EPT, Rows MODE, int MAX_THREADS, int MIN_CTAS>
cudaError_t launch_forward(const NormParams &p, const NormShape &s, cudaStream_t stream) {
    static std::atomic<bool> attr_done[64];  // zero-initialised; several host threads may launch
    return launch_kernel(norm_kernel<T, EPT, MODE, MAX_THREADS, MIN_CTAS>, attr_done, p, s, stream);
}

template <typename T, int EPT, Rows MODE, int MAX_THREADS, int MIN_CTAS>
cudaError_t launch_backward(const NormParams &p, const NormShape &s, cudaStream_t stream) {
    static std::atomic<bool> attr_done[3][64];  // zero-initialised; several host threads may launch
    if (p.gate_kind == 2)
        return launch_kernel(norm_backward_kernel<T, EPT, MODE, 2, MAX_THREADS, MIN_CTAS>, attr_done[1], p, s, stream);
    if (p.gate_kind == 3)
        return launch_kernel(norm_backward_kernel<T, EPT, MODE, 3, MAX_THREADS, MIN_CTAS>, attr_done[2], p, s, stream);
    return launch_kernel(norm_backward_kernel<T, EPT, MODE, 1, MAX_THREADS, MIN_CTAS>, attr_done[0], p, s, stream);
}

// Registers by the CTA's threads: the forward pass has 64; the backward pass
// 80 up to 256 threads, 128 up to 512, 72 up to 896 (rows of 7168), 64 above.
template <typename T> cudaError_t launch_shape(const NormParams &p, const NormShape &s, bool backward, cudaStream_t stream) {
    constexpr Rows kVectors = Rows::kVectors, kOdd = Rows::kOdd, kMemory = Rows::kMemory;
    const bool odd = s.mode == kOdd;
    if (!backward) {
        if constexpr (sizeof(T) == 4)  // 16-bit rows of 16384, the widest, fit the ring
            if (s.mode == kMemory) return launch_forward<T, 16, kMemory, 1024, 1>(p, s, stream);
        if (s.ept == 16) {
            if constexpr (sizeof(T) == 2)
                if (s.threads <= 512)
                    return odd ? launch_forward<T, 16, kOdd, 512, 2>(p, s, stream)
                               : launch_forward<T, 16, kVectors, 512, 2>(p, s, stream);
            return odd ? launch_forward<T, 16, kOdd, 1024, 1>(p, s, stream) : launch_forward<T, 16, kVectors, 1024, 1>(p, s, stream);
        }
        if constexpr (sizeof(T) == 4)
            if (s.threads > 512)
                return odd ? launch_forward<T, 8, kOdd, 1024, 1>(p, s, stream) : launch_forward<T, 8, kVectors, 1024, 1>(p, s, stream);
        return odd ? launch_forward<T, 8, kOdd, 512, 2>(p, s, stream) : launch_forward<T, 8, kVectors, 512, 2>(p, s, stream);
    }
    if (s.mode == kMemory) return launch_backward<T, 16, kMemory, 1024, 1>(p, s, stream);
    if (s.ept == 16) {
        if (s.threads <= 512)
            return odd ? launch_backward<T, 16, kOdd, 512, 1>(p, s, stream) : launch_backward<T, 16, kVectors, 512, 1>(p, s, stream);
        return odd ? launch_backward<T, 16, kOdd, 1024, 1>(p, s, stream) : launch_backward<T, 16, kVectors, 1024, 1>(p, s, stream);
    }
    if (s.threads <= 256)
        return odd ? launch_backward<T, 8, kOdd, 256, 3>(p, s, stream) : launch_backward<T, 8, kVectors, 256, 3>(p, s, stream);
    if (s.threads <= 512)
        return odd ? launch_backward<T, 8, kOdd, 512, 1>(p, s, stream) : launch_backward<T, 8, kVectors, 512, 1>(p, s, stream);
    return odd ? launch_backward<T, 8, kOdd, 896, 1>(p, s, stream) : launch_backward<T, 8, kVectors, 896, 1>(p, s, stream);
}

template <typename T> cudaError_t launch_typed(NormParams p, bool backward, cudaStream_t stream) {
    int ctas = 0;  // no rows: no tensors to shape a ring for, and column sums of zero
    if (p.T > 0) {
        const NormShape s = norm_shape(p, sizeof(T), backward);
        const cudaError_t e = launch_shape<T>(p, s, backward, stream);
        if (e != cudaSuccess) return e;
        ctas = s.ctas;
    }
    if (!backward || (!p.d_w_next && !p.d_w_post && !(p.d_gate && p.gate_kind == 1))) return cudaSuccess;
    return launch_pdl(norm_columns_kernel, dim3(static_cast<unsigned>((p.H + 31) / 32), 3), dim3(256), 0, stream, p, ctas);
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
    // three rows of column sums for each CTA of the largest grid at this width
    const int64_t ctas = static_cast<int64_t>(device_sm_count()) * backward_per_sm(H);
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
