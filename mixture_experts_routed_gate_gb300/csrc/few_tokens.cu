// few_tokens.cu -- the whole routed-expert layer for a few tokens (T <= 16).
//
//   out_t = sum over the k experts e of token t of p_te * W_down[e] h_te,
//   h_te  = silu(W_gate[e] x_t) * (W_up[e] x_t)
// with the routing of moe_gate_topk.  The weights of the chosen experts are
// the cost: each is read once and meets at most 16 tokens.  Two launches:
//
// 1. few_logits_kernel: a warp per expert, all tokens, in the gate's fixed
//    summation order.
// 2. few_layer_kernel: one CTA per SM.  Every CTA chooses the experts from the
//    logits itself (T warps' work, no further launch), then takes tiles from a
//    shared counter: first the stage-1 tiles (8 features of an expert: 8 gate
//    and 8 up rows), then the stage-2 tiles (16 output rows, all experts).
//    A tile is 16 weight rows, streamed 512 columns at a time through a ring
//    of shared-memory stages: one warp copies weights (two 8-row boxes of TMA,
//    each eight 64-column slabs with the 128-byte swizzle), another the rows
//    that meet them (x, or h once its expert's tiles are done), so the weights
//    of a stage-2 tile are under way before h is.  Two groups of eight warps
//    take the stages in turn (one group needs about 600 cycles a stage, and
//    16 KB arrive every 370 ns), each warp its 64-column slab, with m16n8k16 MMAs (weights as the 16
//    rows, tokens as the 8 columns; 1 or 2 column groups): the tensor path
//    only has to keep up with the stream, and 16 rows suit short tiles.  Four
//    more warps join their sums in a fixed order.
//    h is scaled by its routing weight and kept as a 16-bit value and the
//    16-bit rest, both multiplied, so that the stage-2 accumulators hold the
//    weighted sum over the experts and the output is rounded once.  The weights
//    are a softmax over all experts, about 1 / E, and fp16 has few bits below
//    2^-14, so a token's weights are scaled by the power of two that brings its
//    largest to [0.5, 1), undone when the sums are joined, and in fp16 the rest
//    is kept times 2^11, with sums of its own: h is held to 2^-22 of itself or
//    2^-35, bf16's to 2^-17 of itself (its outputs round by 2^-9).  Without the
//    scales an h of 1e-3 among 256 experts was off by up to 0.8%.
// Tiles are taken in order, so a stage-2 tile waits only on tiles that running
// CTAs hold: the launch completes whether or not all CTAs are resident.
//
// Bound by the weights' bytes once there are many: 2 tokens at 7168 / 2048, 256
// experts, top-8, bf16: 1.39 GB in 198 us, 7.0 TB/s (a copy runs at 6.8); 8 at
// 2048 / 768, 64 experts, top-6, fp16: 331 MB in 67 us, 4.9 TB/s.  There stage 2
// is 128 tiles, each 16 rows of all 35 or so chosen experts (860 KB, about 19 us
// at a CTA's share of the memory), so 24 CTAs are idle for the last quarter.
// One token there (57 MB, 8.4 us at the copy rate) takes 20 us: two launches, the
// routing (about 2 us), the first loads' latency and h on its way from CTA to
// CTA.  When the first two of these took 210 and 72 us, stages of 256 columns
// took 343 and 117, of 1024 columns 206 and 74, and three groups of multiplying
// warps 212 and 79.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int FEW_COLS = 512;                        // columns of a stage
constexpr int FEW_ROW = FEW_COLS * 2 + 16;           // bytes of an x or h row; the pad puts the rows in other banks
constexpr int FEW_HALF = 8 * FEW_COLS * 2;           // bytes of eight weight rows
constexpr int FEW_SLABS = 8;                         // multiplying warps on a stage, 64 columns each
constexpr int FEW_GROUPS = 2;                        // groups of them, which take the stages in turn
constexpr int FEW_CONSUMERS = FEW_SLABS * FEW_GROUPS;
constexpr int FEW_FINISHERS = 4;                     // warps that join the multiplying warps' sums
constexpr int FEW_THREADS = (FEW_CONSUMERS + 2 + FEW_FINISHERS) * 32;
constexpr int FEW_PARTS = 2;                         // tiles whose sums may wait to be joined
constexpr int FEW_MAX_STAGES = 12;
constexpr int FEW_QUEUE = 4;                         // tiles handed from the copying to the other warps
constexpr int FEW_BARS = 2 * FEW_MAX_STAGES + 2 * FEW_QUEUE + 2 * FEW_PARTS;
constexpr int FEW_SMEM_MAX = 232448 - 1024;
constexpr int LOGIT_WARPS = 4;

template <int DT> constexpr float FEW_REST = DT == kF16 ? 2048.0f : 1.0f;  // scale of h's rest: at most as large as h

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

// logits[t, e] in the gate's fixed order (lane L sums its 8-element chunks
// L, L + 32, ... in ascending order, then the butterfly), a warp for one expert
// and TT tokens; also clears the counters of the second launch.
template <int DT, int TT>
__global__ void __launch_bounds__(LOGIT_WARPS * 32)
    few_logits_kernel(const uint4 *__restrict__ x, const uint4 *__restrict__ w_g, const float *__restrict__ bias,
                      int tokens, int chunks, int E, float *__restrict__ logits, int *__restrict__ counters,
                      int n_counters) {
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, e = blockIdx.x * LOGIT_WARPS + (threadIdx.x >> 5), t0 = blockIdx.y * TT;
    const uint4 *w = w_g + static_cast<int64_t>(e < E ? e : 0) * chunks;
    for (int c = lane * 8; c < chunks; c += 256)  // 128 bytes a lane
        asm volatile("prefetch.global.L2 [%0];" ::"l"(w + c));
    griddep_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < n_counters; i += LOGIT_WARPS * 32) counters[i] = 0;
    if (e >= E) return;
    constexpr int U = TT == 1 ? 8 : (TT == 2 ? 6 : 4);  // chunks in flight, each of w and of TT tokens
    float acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.0f;
    for (int c0 = lane; c0 < chunks; c0 += 32 * U) {
        uint4 wv[U], xv[TT][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * u < chunks) wv[u] = __ldg(w + c0 + 32 * u);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + 32 * u < chunks)
                    xv[t][u] = __ldg(x + static_cast<int64_t>(min(t0 + t, tokens - 1)) * chunks + c0 + 32 * u);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + 32 * u < chunks) acc[t] = dot8<DT>(xv[t][u], wv[u], acc[t]);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        float l = warp_sum(acc[t]);
        if (bias) l = l + bias[e];
        if (lane == 0 && t0 + t < tokens) logits[static_cast<int64_t>(t0 + t) * E + e] = l;
    }
}

// The k best of one token's E logits (descending, ties to the lower id) and
// their softmax weights, by one warp; lane j < k gets slot j.
template <int SLOTS>
__device__ __forceinline__ void warp_route(const float *row, int E, int k, int lane, int *my_e, float *my_w) {
    uint32_t key[SLOTS], most = 0u;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        const int e = s * 32 + lane;
        key[s] = e < E ? order_key(__ldcg(row + e)) : 0u;
        most = max(most, key[s]);
    }
    const float top = key_value(__reduce_max_sync(0xffffffffu, most));
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
        if (s * 32 + lane < E) sum += expf(key_value(key[s]) - top);
    sum = warp_sum(sum);
    uint32_t mine = 0u;
    int id = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
        int slot = 0;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (key[s] > best) {
                best = key[s];
                slot = s;
            }
        const uint32_t win = __reduce_max_sync(0xffffffffu, best);
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == win ? slot * 32u + lane : 0xffffffffu);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (s * 32u + lane == e) key[s] = 0u;
        if (j == lane) {
            mine = win;
            id = static_cast<int>(e);
        }
    }
    *my_e = id;
    *my_w = expf(key_value(mine) - top) / sum;
}

// Waits until counter `a` has reached `target` and returns the last expert up
// to which all have (a - 1 when the wait gave up).  The lanes look at 32
// counters at once: one at a time, each look cost its latency (about 1 us an
// expert, in the way of the copies).
__device__ __forceinline__ int experts_ready(const int *counters, int a, int n_act, int target, int lane,
                                             volatile int *abort_flag, int *err) {
    const unsigned long long start = global_timer_ns();
    for (;;) {
        const bool yes = a + lane < n_act && counter_load_acquire(counters + a + lane) >= target;
        const uint32_t done = __ballot_sync(0xffffffffu, yes);
        if (done & 1u) {
            // every lane's copies of h come after every lane's look at the
            // counters, and read through the async proxy
            __syncwarp();
            asm volatile("fence.proxy.async.global;" ::: "memory");
            return a + __ffs(~done) - 2 + (done == 0xffffffffu ? 33 : 0);
        }
        const bool late = *abort_flag || global_timer_ns() - start > kWaitTimeoutNs;
        if (__any_sync(0xffffffffu, late)) {
            *abort_flag = 1;
            if (err && lane == 0) atomicExch(err, kErrTimeout);
            return a - 1;
        }
        __nanosleep(50);
    }
}

// After an abort: copies in flight land before shared memory goes away; a
// stage that the other copying warp never filled stays open, 10 ms each.
// `stage`, `phase`: where the copying warp would go on.
__device__ __forceinline__ void few_drain(uint32_t full_bars, int stages, int stage, uint32_t phase) {
    for (int i = 0; i < stages; ++i) {
        const int st = (stage + i) % stages;
        const uint32_t par = stage + i < stages ? phase ^ 1u : phase;
        const unsigned long long start = global_timer_ns();
        while (!mbar_try_wait(full_bars + 8u * st, par) && global_timer_ns() - start < 10000000ull) {
        }
    }
}

struct FewParams {
    const void *x, *w_gate, *w_up, *w_down;
    const float *logits;
    int *counters;  // the next tile, then per chosen expert the stage-1 warps that stored h
    void *h_hi, *h_lo, *out;
    int32_t *err;
    int T, k, E, d_h, d_e;
    int ring_bytes;
};

// D (16 x 8 fp32) += A (16 x 16) B (16 x 8)
template <int DT>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    if constexpr (DT == kBF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// four 8 x 8 matrices, each lane giving the address of one row of one of them
__device__ __forceinline__ uint4 ldmatrix_x4(uint32_t addr) {
    uint4 r;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(addr)
                 : "memory");
    return r;
}

__device__ __forceinline__ void row_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// shared memory after the ring: chosen experts and pairs (at most T * k of each)
struct FewSmem {
    uint8_t *ring, *zeros;  // zeros: a row of x or h for a token that is not routed here
    uint64_t *bars;
    float4 *partial;  // [FEW_PARTS][FEW_CONSUMERS][NT][32]
    int *queue, *act_e, *act_base, *topk_e;
    uint32_t *act_mask;
    float *pair_w, *topk_w;  // times the token's power of two
    float *undo;             // [16] and back
};
__host__ __device__ constexpr int few_stage_bytes(int tokens) {
    return (2 * FEW_HALF + 2 * tokens * FEW_ROW + 1023) / 1024 * 1024;
}
__host__ __device__ constexpr int few_fixed_bytes(int nt, int pairs) {
    return FEW_BARS * 8 + FEW_ROW + FEW_PARTS * FEW_CONSUMERS * nt * 512 + FEW_QUEUE * 4 + pairs * 24 + 64;
}

// One output of token t from its own experts alone, by a warp (every lane gets
// it): the joining warps' way back from products that are not finite.
template <int DT>
__device__ __forceinline__ float few_output(const FewParams &p, const FewSmem &sm, int n_act, int t, int row, int lane) {
    using El = typename Elem<DT>::T;
    float s = 0.0f;
#pragma unroll 1
    for (int a = 0; a < n_act; ++a) {
        const uint32_t m = sm.act_mask[a];
        if (!((m >> t) & 1u)) continue;
        const int r = sm.act_base[a] + __popc(m & ((1u << t) - 1u));
        if (sm.pair_w[r] != sm.pair_w[r]) return sm.pair_w[r];
        const El *w = static_cast<const El *>(p.w_down) + (static_cast<int64_t>(sm.act_e[a]) * p.d_h + row) * p.d_e;
        const El *hi = static_cast<const El *>(p.h_hi) + static_cast<int64_t>(r) * p.d_e;
        const El *lo = static_cast<const El *>(p.h_lo) + static_cast<int64_t>(r) * p.d_e;
#pragma unroll 1
        for (int c = lane; c < p.d_e; c += 32)  // h comes from other CTAs: past L1
            s = fmaf(fmaf(to_f32(__ldcg(lo + c)), 1.0f / FEW_REST<DT>, to_f32(__ldcg(hi + c))), to_f32(__ldg(w + c)), s);
    }
    return warp_sum(s);
}

static_assert(1024 + FEW_GROUPS * few_stage_bytes(16) + few_fixed_bytes(2, 16 * 32) <= FEW_SMEM_MAX,
              "a stage for each group at least");
static_assert(FEW_MAX_STAGES % FEW_GROUPS == 0, "stages belong to groups");

template <int DT, int NT>
__global__ void __launch_bounds__(FEW_THREADS, 1)
    few_layer_kernel(const __grid_constant__ CUtensorMap tm_gate, const __grid_constant__ CUtensorMap tm_up,
                     const __grid_constant__ CUtensorMap tm_down, const FewParams p) {
    using El = typename Elem<DT>::T;
    extern __shared__ uint8_t few_unaligned[];
    uint8_t *few_raw = few_unaligned + ((1024u - (smem_u32(few_unaligned) & 1023u)) & 1023u);
    const int pairs = p.T * p.k;
    FewSmem sm;
    sm.ring = few_raw;
    sm.bars = reinterpret_cast<uint64_t *>(few_raw + p.ring_bytes);
    sm.zeros = reinterpret_cast<uint8_t *>(sm.bars + FEW_BARS);
    sm.partial = reinterpret_cast<float4 *>(sm.zeros + FEW_ROW);
    sm.queue = reinterpret_cast<int *>(sm.partial + FEW_PARTS * FEW_CONSUMERS * NT * 32);
    sm.act_e = sm.queue + FEW_QUEUE;
    sm.act_base = sm.act_e + pairs;
    sm.topk_e = sm.act_base + pairs;
    sm.act_mask = reinterpret_cast<uint32_t *>(sm.topk_e + pairs);
    sm.pair_w = reinterpret_cast<float *>(sm.act_mask + pairs);
    sm.topk_w = sm.pair_w + pairs;
    sm.undo = sm.topk_w + pairs;
    __shared__ int abort_word, n_act_word, most_word;
    volatile int *abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar0 = smem_u32(sm.bars);
    auto full_bar = [&](int i) { return bar0 + 8u * i; };
    auto empty_bar = [&](int i) { return bar0 + 8u * (FEW_MAX_STAGES + i); };
    auto tqf_bar = [&](int i) { return bar0 + 8u * (2 * FEW_MAX_STAGES + i); };
    auto tqe_bar = [&](int i) { return bar0 + 8u * (2 * FEW_MAX_STAGES + FEW_QUEUE + i); };
    auto pf_bar = [&](int i) { return bar0 + 8u * (2 * FEW_MAX_STAGES + 2 * FEW_QUEUE + i); };
    auto pe_bar = [&](int i) { return bar0 + 8u * (2 * FEW_MAX_STAGES + 2 * FEW_QUEUE + FEW_PARTS + i); };
    uint32_t *mask = reinterpret_cast<uint32_t *>(sm.ring);  // [E] while routing
    if (threadIdx.x == 0) {
        for (int i = 0; i < FEW_MAX_STAGES; ++i) {
            mbar_init(full_bar(i), 2);  // the weights' and the rows' copying warps
            mbar_init(empty_bar(i), FEW_SLABS);
        }
        for (int i = 0; i < FEW_QUEUE; ++i) {
            mbar_init(tqf_bar(i), 1);
            mbar_init(tqe_bar(i), FEW_CONSUMERS + 1 + FEW_FINISHERS);
        }
        for (int i = 0; i < FEW_PARTS; ++i) {
            mbar_init(pf_bar(i), FEW_CONSUMERS);
            mbar_init(pe_bar(i), FEW_FINISHERS);
        }
        abort_word = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_gate);
        tma_prefetch_desc(&tm_up);
        tma_prefetch_desc(&tm_down);
    }
    for (int e = threadIdx.x; e < p.E; e += FEW_THREADS) mask[e] = 0u;
    for (int i = threadIdx.x; i < FEW_ROW / 4; i += FEW_THREADS) reinterpret_cast<uint32_t *>(sm.zeros)[i] = 0u;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    // ------------------------------- routing -------------------------------
    for (int t = warp; t < p.T; t += FEW_THREADS / 32) {
        const float *row = p.logits + static_cast<int64_t>(t) * p.E;
        int e;
        float w;
        if (p.E <= 64)
            warp_route<2>(row, p.E, p.k, lane, &e, &w);
        else if (p.E <= 256)
            warp_route<8>(row, p.E, p.k, lane, &e, &w);
        else
            warp_route<32>(row, p.E, p.k, lane, &e, &w);
        // the largest, in [2^(field - 127), 2^(field - 126)); a NaN stays one
        const uint32_t field = min((__float_as_uint(__shfl_sync(0xffffffffu, w, 0)) >> 23) & 255u, 252u);
        if (lane < p.k) {
            sm.topk_e[t * p.k + lane] = e;
            sm.topk_w[t * p.k + lane] = w * __uint_as_float((253u - field) << 23);
            atomicOr(&mask[e], 1u << t);
        }
        if (lane == 0) sm.undo[t] = __uint_as_float((field + 1u) << 23);
    }
    __syncthreads();
    if (warp == 0) {  // the chosen experts in ascending order, their tokens, their first row of h
        int n = 0, base = 0, most = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            const uint32_t m = e < p.E ? mask[e] : 0u;
            const uint32_t has = __ballot_sync(0xffffffffu, m != 0u);
            if (has == 0u) continue;
            const int rows = __popc(m);
            int before = rows;
            most = max(most, rows);
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, before, s);
                if (lane >= s) before += v;
            }
            if (m != 0u) {
                const int a = n + __popc(has & ((1u << lane) - 1u));
                sm.act_e[a] = e;
                sm.act_mask[a] = m;
                sm.act_base[a] = base + before - rows;
                mask[e] = static_cast<uint32_t>(a);
            }
            n += __popc(has);
            base += __shfl_sync(0xffffffffu, before, 31);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            n_act_word = n;
            most_word = most;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += FEW_THREADS) {
        const uint32_t a = mask[sm.topk_e[i]];
        sm.pair_w[sm.act_base[a] + __popc(sm.act_mask[a] & ((1u << (i / p.k)) - 1u))] = sm.topk_w[i];
    }
    // the ring was written through the generic proxy; bulk copies follow
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    const int n_act = n_act_word;
    // a stage holds 16 weight rows and the rows of the expert with the most tokens
    const int stage_bytes = few_stage_bytes(most_word);
    // A multiple of the groups, so that a stage always belongs to one group: a
    // group a whole ring ahead of another on the other's stage would take the
    // barrier's phase before last for its own (they have the same parity).
    const int stages = min(FEW_MAX_STAGES, p.ring_bytes / stage_bytes) / FEW_GROUPS * FEW_GROUPS;
    const uint32_t ring = smem_u32(sm.ring);
    const int tiles_e = p.d_e / 8;           // stage-1 tiles of an expert
    const int n1 = n_act * tiles_e, total = n1 + p.d_h / 16;
    const int steps1 = (p.d_h + FEW_COLS - 1) / FEW_COLS, steps2 = (p.d_e + FEW_COLS - 1) / FEW_COLS;
    // A tile takes an even number of stages, so that its steps go to the groups
    // in the same way in whatever order the tiles are taken: the order of the
    // sums, and with it the result's bits, does not depend on it.
    static_assert(FEW_GROUPS == 2, "padding to an even count");
    auto pad_steps = [&](int tile) { return (tile < n1 ? steps1 : n_act * steps2) & 1; };

    if (warp == FEW_CONSUMERS) {
        // -------------------- weights: one thread, no broadcasts --------------------
        // (a whole warp with its shuffles took about 900 cycles a step and
        // was what paced the stream)
        if (lane != 0) return;
        const uint64_t policy = l2_policy_evict_first();
        int stage = 0, slot = 0;
        uint32_t phase = 0, qphase = 0;
        bool ok = true;
        // 512 columns of 16 weight rows: 8 from row r0 of map m0, 8 from row r1
        // of map m1 (columns past the end read as zeros)
        auto copy = [&](const CUtensorMap *m0, const CUtensorMap *m1, int r0, int r1, int steps) {
            for (int c = 0; c < steps; ++c) {
                if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) return false;
                const uint32_t dst = ring + stage * stage_bytes, bar = full_bar(stage);
                mbar_arrive_expect_tx(bar, 2 * FEW_HALF);
                tma_load_3d_hint(dst, m0, bar, 0, r0, c * (FEW_COLS / 64), policy);
                tma_load_3d_hint(dst + FEW_HALF, m1, bar, 0, r1, c * (FEW_COLS / 64), policy);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            return true;
        };
        // the step that makes a tile's count even (see pad_steps)
        auto pad = [&]() {
            if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) return false;
            mbar_arrive(full_bar(stage));
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
            return true;
        };
        int next = atomicAdd(p.counters, 1);
        while (ok) {
            ok = mbar_wait_bounded(tqe_bar(slot), qphase ^ 1u, abort_flag, p.err);
            if (!ok) break;
            const int tile = next;
            sm.queue[slot] = tile;
            mbar_arrive(tqf_bar(slot));
            if (tile >= total) break;
            // Claimed before the copies of a short stage-1 tile, under which the
            // latency passes; after those of a stage-2 tile, which are a CTA's
            // last 5 to 20 us: claimed ahead, some CTAs held two while others had
            // none (8 x 2048 fp16 then took 68 or 89 us, by chance).
            if (tile < n1) next = atomicAdd(p.counters, 1);
            if (++slot == FEW_QUEUE) {
                slot = 0;
                qphase ^= 1u;
            }
            if (tile < n1) {
                const int a = tile / tiles_e, row = sm.act_e[a] * p.d_e + (tile - a * tiles_e) * 8;
                ok = copy(&tm_gate, &tm_up, row, row, steps1);
            } else {
                for (int a = 0; a < n_act && ok; ++a) {
                    const int row = sm.act_e[a] * p.d_h + (tile - n1) * 16;
                    ok = copy(&tm_down, &tm_down, row, row + 8, steps2);
                }
            }
            for (int i = pad_steps(tile); i > 0 && ok; --i) ok = pad();
            if (tile >= n1) next = atomicAdd(p.counters, 1);
        }
        if (*abort_flag) few_drain(bar0, stages, stage, phase);
        return;
    }

    // the other warps take every tile and run whole; every lane polls, which on the usual
    // first try needs no broadcast
    int slot = 0, local = 0;
    uint32_t qphase = 0;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag, p.err)) != 0;
    };
    auto take = [&]() {  // the next tile, `total` or more when there is none
        if (!wait(tqf_bar(slot), qphase)) return total;
        const int tile = sm.queue[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(tqe_bar(slot));
        if (++slot == FEW_QUEUE) {
            slot = 0;
            qphase ^= 1u;
        }
        return tile;
    };
    if (warp == FEW_CONSUMERS + 1) {
        // ------------------ the rows that meet the weights: x or h ------------------
        const uint64_t policy = l2_policy_evict_last();
        int stage = 0, ready = -1;  // ready: experts up to here have their h
        uint32_t phase = 0;
        bool ok = true;
        // `n` rows of K columns from each lane's src, step by step.  The
        // lanes' copies may start before lane 0 has announced their bytes: its
        // arrival is what lets the phase complete
        auto copy = [&](int n, int K, const uint8_t *src, int steps) {
            for (int c = 0; c < steps; ++c) {
                if (!wait(empty_bar(stage), phase ^ 1u)) return false;
                const uint32_t bytes = static_cast<uint32_t>(min(FEW_COLS, K - c * FEW_COLS)) * 2u, bar = full_bar(stage);
                if (lane == 0) mbar_arrive_expect_tx(bar, n * bytes);  // no rows: a padding step
                if (lane < n)
                    row_copy(ring + stage * stage_bytes + 2 * FEW_HALF + lane * FEW_ROW, src + c * FEW_COLS * 2, bytes, bar, policy);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            return true;
        };
        for (int tile = take(); tile < total && ok; tile = take()) {
            if (tile < n1) {
                const uint32_t m = sm.act_mask[tile / tiles_e];
                const int n = __popc(m), t = lane < n ? static_cast<int>(__fns(m, 0, lane + 1)) : 0;
                ok = copy(n, p.d_h, static_cast<const uint8_t *>(p.x) + static_cast<int64_t>(t) * p.d_h * 2, steps1);
            } else {
                for (int a = 0; a < n_act && ok; ++a) {
                    const int rows = __popc(sm.act_mask[a]);
                    const int r = sm.act_base[a] + (lane < rows ? lane : lane - rows);
                    if (a > ready) {  // h of this expert: every stage-1 warp has stored it
                        ready = experts_ready(p.counters + 1, a, n_act, tiles_e * 2, lane, abort_flag, p.err);
                        ok = ready >= a;
                    }
                    const void *h = lane < rows ? p.h_hi : p.h_lo;
                    ok = ok && copy(2 * rows, p.d_e, static_cast<const uint8_t *>(h) + static_cast<int64_t>(r) * p.d_e * 2, steps2);
                }
            }
            if (ok && pad_steps(tile)) ok = copy(0, 0, nullptr, 1);
        }
        if (*abort_flag && lane == 0) few_drain(bar0, stages, stage, phase);
        return;
    }

    if (warp >= FEW_CONSUMERS + 2) {
        // -------------------------------- joining --------------------------------
        const int fin = warp - FEW_CONSUMERS - 2;
        for (int tile = take(); tile < total; tile = take(), ++local) {
            const int buf = local % FEW_PARTS;
            if (!wait(pf_bar(buf), static_cast<uint32_t>(local / FEW_PARTS) & 1u)) break;
            const float *f = reinterpret_cast<const float *>(sm.partial + buf * FEW_CONSUMERS * NT * 32);
            // the sums are free for the next tile as soon as they are read:
            // making h visible takes 1 to 2 us, and two pairs of warps take
            // the stage-1 tiles in turn for the same reason
            auto release = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(pe_bar(buf));
            };
            if (tile < n1) {
                if ((fin >> 1) != (local & 1)) {
                    release();
                    continue;
                }
                const int a = tile / tiles_e, i = (fin & 1) * 32 + lane, feat = i & 7, t8 = i >> 3;
                float gate[NT], up[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int at = (n * 32 + feat * 4 + (t8 >> 1)) * 4 + (t8 & 1);
                    gate[n] = up[n] = 0.0f;
#pragma unroll
                    for (int w = 0; w < FEW_CONSUMERS; ++w) {
                        gate[n] += f[w * NT * 128 + at];
                        up[n] += f[w * NT * 128 + at + 2];
                    }
                }
                release();
                const uint32_t m = sm.act_mask[a];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int t = n * 8 + t8;
                    if (!((m >> t) & 1u)) continue;
                    const int r = sm.act_base[a] + __popc(m & ((1u << t) - 1u));
                    const float h = gate[n] / (1.0f + __expf(-gate[n])) * up[n] * sm.pair_w[r];
                    const El top = from_f32<El>(h);
                    const int64_t o = static_cast<int64_t>(r) * p.d_e + (tile - a * tiles_e) * 8 + feat;
                    const float t32 = to_f32(top);
                    static_cast<El *>(p.h_hi)[o] = top;
                    static_cast<El *>(p.h_lo)[o] = from_f32<El>(fabsf(t32) == INFINITY ? 0.0f : (h - t32) * FEW_REST<DT>);
                }
                asm volatile("fence.proxy.async.global;" ::: "memory");
                __syncwarp();  // the publishing add releases the whole warp's stores
                if (lane == 0) counter_publish(p.counters + 1 + a);
            } else {
                const int i = fin * 32 + lane, r = i & 15, t8 = i >> 4;
                float v[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int at = (n * 32 + (r & 7) * 4 + (t8 >> 1)) * 4 + (t8 & 1) + (r >> 3) * 2;
                    v[n] = 0.0f;
#pragma unroll
                    for (int w = 0; w < FEW_CONSUMERS; ++w) v[n] += f[w * NT * 128 + at];
                }
                release();
                // A token takes part in every chosen expert's products, as a row of zeros
                // where it is not routed: an infinity or a NaN among the weights would
                // reach it.  And an infinite weight times h's two parts may be inf - inf.
                // So an output that is not finite is summed again from the token's own
                // experts, unless its routing is NaN already.
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const bool odd = n * 8 + t8 < p.T && !(fabsf(v[n]) < INFINITY);
                    for (uint32_t todo = __ballot_sync(0xffffffffu, odd); todo != 0u; todo &= todo - 1u) {
                        const int src = __ffs(todo) - 1, at = fin * 32 + src;
                        const float whole = few_output<DT>(p, sm, n_act, n * 8 + (at >> 4), (tile - n1) * 16 + (at & 15), lane);
                        if (lane == src) v[n] = whole;
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int t = n * 8 + t8;
                    if (t < p.T)
                        static_cast<El *>(p.out)[static_cast<int64_t>(t) * p.d_h + (tile - n1) * 16 + r] = from_f32<El>(v[n] * sm.undo[t]);
                }
            }
        }
        return;
    }

    // ------------------------------ multiplying ------------------------------
    // a lane gives the address of row lane % 8 of matrix lane / 8.  Weights:
    // the matrices are rows 0-7, then 8-15, of 8 columns, then of the next 8;
    // tokens: four times 8 columns
    const int mrow = lane & 7, mat = lane >> 3;
    const uint32_t zeros = smem_u32(sm.zeros) + mat * 16;
    const int slab = warp % FEW_SLABS;
    const uint32_t wrow = (mat & 1) * FEW_HALF + slab * 1024 + mrow * 128;
    const uint32_t trow = 2 * FEW_HALF + slab * 128 + mat * 16;
    int stage = 0, turn = warp / FEW_SLABS;  // turn 0: the next stage is this group's
    uint32_t phase = 0;
    bool ok = true;
    auto advance = [&]() {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
        turn = turn == 0 ? FEW_GROUPS - 1 : turn - 1;
    };
    for (int tile = take(); tile < total; tile = take(), ++local) {
        // four independent chains of MMAs a column group: in one chain their
        // latencies add up to most of a step
        float acc[NT][4][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[n][i >> 2][i & 3] = 0.0f;
        const bool first = tile < n1;
        const int a0 = first ? tile / tiles_e : 0, a1 = first ? a0 + 1 : n_act;
        const int K = first ? p.d_h : p.d_e, steps = first ? steps1 : steps2;
        for (int a = a0; a < a1 && ok; ++a) {
            const uint32_t m = sm.act_mask[a];
            const uint32_t rest = __popc(m) * FEW_ROW;  // from a row of h to its rest
            uint32_t token[NT];                         // the lane's token's row in a stage
            bool here[NT], any[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int t = n * 8 + mrow;
                here[n] = (m >> t) & 1u;
                any[n] = ((m >> (8 * n)) & 255u) != 0u;
                token[n] = trow + __popc(m & ((1u << t) - 1u)) * FEW_ROW;
            }
            for (int c = 0; c < steps; ++c, advance()) {
                if (turn != 0) continue;
                ok = wait(full_bar(stage), phase);
                if (!ok) break;
                if (slab * 64 < K - c * FEW_COLS) {
                    const uint32_t st = ring + stage * stage_bytes;
                    uint4 w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = ldmatrix_x4(st + wrow + (((2 * j + (mat >> 1)) ^ mrow) << 4));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (!any[n]) continue;
                        const uint32_t b = here[n] ? st + token[n] : zeros;
                        if (first) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint4 v = ldmatrix_x4(b + j * 64);
                                mma_16816<DT>(acc[n][j], w[2 * j], v.x, v.y);
                                mma_16816<DT>(acc[n][2 + j], w[2 * j + 1], v.z, v.w);
                            }
                        } else {  // chains 0 and 1: h's values, 2 and 3: their rests
                            const uint32_t b2 = here[n] ? b + rest : zeros;
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                uint4 v = ldmatrix_x4(b + j * 64);
                                mma_16816<DT>(acc[n][0], w[2 * j], v.x, v.y);
                                mma_16816<DT>(acc[n][1], w[2 * j + 1], v.z, v.w);
                                v = ldmatrix_x4(b2 + j * 64);
                                mma_16816<DT>(acc[n][2], w[2 * j], v.x, v.y);
                                mma_16816<DT>(acc[n][3], w[2 * j + 1], v.z, v.w);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty_bar(stage));
            }
        }
        if (ok && pad_steps(tile)) {
            if (turn == 0) {
                ok = wait(full_bar(stage), phase);
                if (ok && lane == 0) mbar_arrive(empty_bar(stage));
            }
            advance();
        }
        if (!ok) break;
        const int buf = local % FEW_PARTS;
        if (!wait(pe_bar(buf), (static_cast<uint32_t>(local / FEW_PARTS) & 1u) ^ 1u)) break;
        float4 *part = sm.partial + buf * FEW_CONSUMERS * NT * 32;
        const float unscale = first ? 1.0f : 1.0f / FEW_REST<DT>;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fmaf(acc[n][2][i] + acc[n][3][i], unscale, acc[n][0][i] + acc[n][1][i]);
            part[(warp * NT + n) * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(pf_bar(buf));
    }
}

size_t round_up(size_t v) { return (v + 255) / 256 * 256; }

template <int DT, int TT>
cudaError_t launch_logits(const void *x, const void *w_g, const float *bias, int64_t T, int64_t d_h, int64_t E,
                          float *logits, int *counters, int n_counters, cudaStream_t stream) {
    return launch_pdl(few_logits_kernel<DT, TT>, dim3(static_cast<unsigned>((E + LOGIT_WARPS - 1) / LOGIT_WARPS), static_cast<unsigned>((T + TT - 1) / TT)),
                      dim3(LOGIT_WARPS * 32), 0, stream, static_cast<const uint4 *>(x), static_cast<const uint4 *>(w_g),
                      bias, (int)T, (int)(d_h / 8), (int)E, logits, counters, n_counters);
}

// [E, N, K] weights as 64 columns x (E N) rows x K / 64 slabs; a box is 8 rows
// of 8 slabs, slab by slab
bool weight_map(CUtensorMap *m, const void *w, int64_t E, int64_t N, int64_t K) {
    const uint64_t dims[3] = {64, static_cast<uint64_t>(E * N), static_cast<uint64_t>(K / 64)};
    const uint64_t strides[2] = {static_cast<uint64_t>(K) * 2, 128};
    const uint32_t box[3] = {64, 8, FEW_COLS / 64};
    return encode_tma_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, w, dims, strides, box, 1);
}

template <int DT, int NT> cudaError_t launch_layer(FewParams p, cudaStream_t stream) {
    const int pairs = p.T * p.k;
    p.ring_bytes = (FEW_SMEM_MAX - 1024 - few_fixed_bytes(NT, pairs)) / 1024 * 1024;
    const int smem = 1024 + p.ring_bytes + few_fixed_bytes(NT, pairs);
    CUtensorMap maps[3];
    if (!weight_map(&maps[0], p.w_gate, p.E, p.d_e, p.d_h) || !weight_map(&maps[1], p.w_up, p.E, p.d_e, p.d_h) ||
        !weight_map(&maps[2], p.w_down, p.E, p.d_h, p.d_e))
        return cudaErrorInvalidValue;
    auto kern = few_layer_kernel<DT, NT>;
    static std::atomic<bool> attr_done[64];  // zero-initialised; several host threads may launch
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, FEW_SMEM_MAX);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    const int64_t experts = pairs < p.E ? pairs : p.E;
    const int64_t tiles = experts * (p.d_e / 8) + p.d_h / 16;
    return launch_pdl(kern, dim3(static_cast<unsigned>(mlp_grid(tiles))), dim3(FEW_THREADS), static_cast<size_t>(smem),
                      stream, maps[0], maps[1], maps[2], p);
}

template <int DT>
cudaError_t launch_typed(const void *w_g, const float *bias, FewParams p, float *logits, int n_counters,
                         cudaStream_t stream) {
    auto run = [&](auto logits_of) { return logits_of(p.x, w_g, bias, p.T, p.d_h, p.E, logits, p.counters, n_counters, stream); };
    // few warps: one token each; more: a row of w for two or four tokens
    const int64_t dots = static_cast<int64_t>(p.T) * p.E;
    cudaError_t e = dots <= 1024 ? run(launch_logits<DT, 1>) : dots <= 2048 ? run(launch_logits<DT, 2>) : run(launch_logits<DT, 4>);
    if (e != cudaSuccess) return e;
    return p.T <= 8 ? launch_layer<DT, 1>(p, stream) : launch_layer<DT, 2>(p, stream);
}

}  // namespace

size_t forward_few_ws_bytes(int64_t T, int64_t d_h, int64_t d_e, int64_t E, int64_t k) {
    (void)d_h;
    return round_up(static_cast<size_t>(T * E) * 4) + round_up(static_cast<size_t>(T * k + 1) * 4) +
           2 * round_up(static_cast<size_t>(T * k * d_e) * 2);
}

cudaError_t launch_forward_few(const void *x, const void *w_g, const float *bias, const void *w_gate, const void *w_up,
                               const void *w_down, int64_t T, int64_t d_h, int64_t d_e, int64_t E, int64_t k,
                               int dtype, void *ws, void *out, int32_t *err, cudaStream_t stream) {
    char *at = static_cast<char *>(ws);
    float *logits = reinterpret_cast<float *>(at);
    at += round_up(static_cast<size_t>(T * E) * 4);
    FewParams p{};
    p.x = x;
    p.w_gate = w_gate;
    p.w_up = w_up;
    p.w_down = w_down;
    p.logits = logits;
    p.counters = reinterpret_cast<int *>(at);
    at += round_up(static_cast<size_t>(T * k + 1) * 4);
    p.h_hi = at;
    p.h_lo = at + round_up(static_cast<size_t>(T * k * d_e) * 2);
    p.out = out;
    p.err = err;
    p.T = static_cast<int>(T);
    p.k = static_cast<int>(k);
    p.E = static_cast<int>(E);
    p.d_h = static_cast<int>(d_h);
    p.d_e = static_cast<int>(d_e);
    const int n_counters = static_cast<int>(T * k + 1);
    if (dtype == kBF16) return launch_typed<kBF16>(w_g, bias, p, logits, n_counters, stream);
    return launch_typed<kF16>(w_g, bias, p, logits, n_counters, stream);
}

}  // namespace moe
