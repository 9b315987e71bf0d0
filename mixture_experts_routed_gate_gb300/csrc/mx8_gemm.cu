// mx8_gemm.cu -- the grouped product of 8-bit rows with 8-bit expert weights on
// the block-scaled tensor cores (tcgen05.mma kind::mxf8f6f4), on pairs of SMs:
//
//   C[r, n] = sum over k of (qa 2^sa)[r, k] * (qb 2^sb)[expert of r][n, k]
//
// and the gate/up form, h = silu(A Wg^T) * (A Wu^T), quantised to 8 bits.
//
// The weights are the M = 256 operand (128 rows in each SM), up to 128 or 256
// rows of an expert the N operand (in steps of 32, half in each SM): a tile costs
// what its rows cost, and every weight byte enters one SM's shared memory once a
// tile.  The accumulator holds features in lanes and rows in columns, so a warp
// stores 32 consecutive features of a row.
//
// A persistent pair works on tiles of such rows by 256 features (128 in the
// gate/up form: 64 of W_gate and 64 of W_up in each SM).  Roles in each CTA:
//   warp 0      TMA: 256-element slices of its weights and of its half of the
//               rows into a ring of 128-byte-swizzled stages, completing on the
//               even CTA's barriers;
//   warp 1      (even CTA) one elected lane: eight K = 32 MMAs a slice;
//   warps 2-9   epilogue, from one of two accumulators while the other fills;
//   warps 10-17 scales, a unit of two slices at a time, two groups in turn: each
//               thread loads a weight row's and a row's 16 scale bytes, two units
//               ahead; through shared memory each warp gets every row's and
//               stores them to its quarter of tensor memory.  Both CTAs hold all
//               rows' scales.  The units have their own ring, of eight (wide
//               tiles: four), so that their way into tensor memory runs ahead of
//               the slices: as a part of each slice it bound the kernel (1124 us
//               where units took 788; without any scales 810).
//
// 32,768 rows, 256 experts, 7168 x 2048, bf16 out: 718 us for 4.25 GB (627 at the
// copy rate); its tiles bring 5.9 GB from L2 into shared memory, which gives out at
// 10 to 12 TB/s (16 experts of 2048 rows: 3.8 GB in 317 us, 3.0 PFLOP/s), and the
// tensor pipe is active for a quarter of the time.  What paces a slice is the one
// thread that asks for its copies: issued by one lane of a branch, each operand
// is moved to it first (770 us), and any work more between them shows in all sizes
// (chunks of shared memory handed out by need, so that a fourth narrow slice fits
// the wide tiles' ring, 8 to 10% slower).  8192 rows: 600 us, 95% of the copy rate;
// the gate/up form of those 1200 us, twice the bytes.  384 rows of 64 experts, 2048 x
// 768, fp16: 23 us for 100 MB (15 at the copy rate): about 7 us are the unit list, the
// first copies, the last epilogue and the exit, and 192 tiles are 2.5 rounds of 76
// pairs.
//
// Slower, at 384 rows through both forms (63 us with the sort): the last round's
// tiles cut by features into 2 or 4 parts 69; the weights' first slices
// prefetched into L2 before the wait for the kernel ahead 65.5 (65.4 then).
#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"
#include "mx8.cuh"

namespace moe {
namespace {

constexpr int G8_SLICE = 256;               // elements (bytes) of K per stage: two 128-byte halves
constexpr int G8_A_HALF = 128 * 128;        // 128 weight rows of one half
constexpr int G8_THREADS = 576;
constexpr int G8_EPI_WARP0 = 2, G8_EPI_WARPS = 8, G8_SF_WARP0 = 10, G8_SF_GROUPS = 2;
constexpr int G8_LIST = 512;                // units of rows that the shared-memory list holds
constexpr int G8_ACC = 128;                 // columns of an accumulator slot; wider units take both
constexpr int G8_UNIT = 2;                  // slices whose scales are stored together
constexpr int G8_AHEAD = 2;                 // units of scales in registers ahead of tensor memory's, a group
constexpr int G8_EXCHANGE = 4 * 2 * 2 * 8 * 32 * 4;  // gate/up: four pairs of epilogue warps, 8 rows by 32 features each way, twice

// NT: the most rows of a tile, 128 or 256
template <int NT> struct G8Layout {
    static constexpr int B_HALF = NT / 2 * 128;  // up to NT / 2 rows of one half
    static constexpr int STAGE = 2 * (G8_A_HALF + B_HALF);
    static constexpr int STAGES = NT == 128 ? 4 : 3;
    static constexpr int UNITS = NT == 128 ? 8 : 4;  // units of scales in tensor memory
    static constexpr int ROWS = NT / 128;           // rows whose scales a thread loads
    // a slice's scales: two halves of 4 columns for the weights, then two of 4 for each 128 rows
    static constexpr int SF_COLS = 8 + 8 * ROWS, UNIT_COLS = G8_UNIT * SF_COLS;
    static constexpr int SF_BYTES = UNIT_COLS * 128;
    static constexpr int SF_COL0 = 2 * G8_ACC;
    static constexpr int FIXED = 1024 + 512 + G8_LIST * 8 + G8_SF_GROUPS * SF_BYTES + G8_EXCHANGE;
    static constexpr int SMEM = STAGES * STAGE + FIXED;
    static_assert(SMEM <= 232448 - 256, "shared memory");
    static_assert(SF_COL0 + UNITS * UNIT_COLS <= 512, "tensor memory");
    static_assert(UNITS % G8_SF_GROUPS == 0, "the groups alternate");
    static_assert((2 * STAGES + 2 * UNITS + 4) * 8 <= 512, "barriers");
};

struct G8Params {
    const uint8_t *sf_a, *sf_b0, *sf_b1;  // b1: the up weights of the gate/up form
    MxTables tab;
    void *out;
    uint8_t *q_h, *sf_h;
    int32_t *err;
    int m_blocks, n_tiles, slices, units;
    int64_t N, K;
};

struct G8Tile {
    int g, m_start, rows, n0;
    bool single;  // the expert's only unit of rows
};

// Whether the tables name rows past the call's, into the error word; by a warp of each
// CTA that has nothing else left to do (in the loop over the entries that every CTA
// starts with it took 0.24 us a launch).
__device__ __forceinline__ void g8_flag_rows_past(const MxTables &t, int lane, int32_t *err) {
    if (!err) return;
    bool past = false;
    for (int g = static_cast<int>(blockIdx.x) * 32 + lane; g < t.E; g += static_cast<int>(gridDim.x) * 32) {
        const int size = t.sizes[g], first = t.offsets[g];
        past |= (size > 0) & (rows_there(t, size, first) < size);
    }
    if (past) atomicExch(err, kErrDeviceFlag);
}

// The accumulator slots in turn; a unit of more rows than a slot's columns takes
// both.  Every role follows the same sequence of tiles, and so of slots.
struct G8Slots {
    int cur = 0;
    uint32_t used = 0;  // a bit a slot: how often, modulo 2
    int first;
    bool both;
    __device__ __forceinline__ void take(int columns) {
        both = columns > G8_ACC;
        first = both ? 0 : cur;
        cur = both ? 0 : cur ^ 1;
    }
    __device__ __forceinline__ uint32_t parity(int slot) const { return used >> slot & 1u; }
    __device__ __forceinline__ void done() { used ^= both ? 3u : 1u << first; }
};

// kind::mxf8f6f4: e4m3 by e4m3 (format 0), e8m0 scales; the scale ids (which of
// a cell's four bytes) are added per MMA.
//   bits 4-5 B scale id; 7-9 A format, 10-12 B format; 17-22 N >> 3; 23 scale
//   type (1 = e8m0); 24-28 M >> 4; 29-30 A scale id
__device__ __forceinline__ uint32_t idesc_mxf8(uint32_t M, uint32_t N) { return ((N >> 3) << 17) | (1u << 23) | ((M >> 4) << 24); }

// The MMA warp runs whole and one elected lane issues, so that the operands come
// from uniform registers.
__device__ __forceinline__ void tc_mma2_mxf8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tc_commit2_both_elect(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// The copies' warp runs whole too.
__device__ __forceinline__ void expect_elect(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_2d_elect(uint32_t dst, const void *map, uint32_t bar_cluster, int c0, int c1, uint64_t policy) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;\n\t}" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)),
                 "r"(bar_cluster), "r"(c0), "r"(c1), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void copy_3d_elect(uint32_t dst, const void *map, uint32_t bar_cluster, int c0, int c1, int c2,
                                              uint64_t policy) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;\n\t}" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)),
                 "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
                 : "memory");
}

// A barrier of COUNT threads: whether `yes` holds in all of them.
template <int COUNT> __device__ __forceinline__ bool g8_all(int id, bool yes) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.and.aligned.pred q, %1, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(id), "r"(yes ? 1u : 0u), "n"(COUNT)
        : "memory");
    return all != 0;
}

// the scales of rows i, 32 + i, 64 + i and 96 + i, p at row i
__device__ __forceinline__ uint4 quarter_scales(const uint8_t *p) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
    return make_uint4(w[0], w[32], w[64], w[96]);
}

// 8 consecutive columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint4 &a, const uint4 &b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(a.x),
                 "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

__device__ __forceinline__ void g8_drain(uint32_t bar, uint32_t parity) {
    const unsigned long long start = global_timer_ns();
    while (!mbar_try_wait_cluster(bar, parity))
        if (global_timer_ns() - start > kWaitTimeoutNs) return;
}

// A unit's scale bytes of a row, WORDS words of 128 elements, from byte `at` on of a
// row of kb bytes (null: zeros); bytes past kb are 0 (their elements are not
// multiplied).  V: the load width that kb and the bases' alignment allow.
template <int V, int WORDS>
__device__ __forceinline__ void load_scales(uint32_t (&w)[WORDS], const uint8_t *row, int kb, int at) {
    constexpr int STEP = V < 4 ? 1 : V / 4;
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < WORDS; i += STEP) {
            const int byte = at + 4 * i;
            const bool in = row != nullptr && byte < kb;
            const uint8_t *p = row + byte;
            if constexpr (V == 16) {
                const uint4 v = in ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0u, 0u, 0u, 0u);
                w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
            } else if constexpr (V == 8) {
                const uint2 v = in ? __ldg(reinterpret_cast<const uint2 *>(p)) : make_uint2(0u, 0u);
                w[i] = v.x, w[i + 1] = v.y;
            } else {
                w[i] = in ? __ldg(reinterpret_cast<const uint32_t *>(p)) : 0u;
            }
        }
    } else {
        // rows that start anywhere: the aligned words that hold their bytes (a word
        // with one of the row's bytes lies in its allocation), shifted together
        const uintptr_t first = reinterpret_cast<uintptr_t>(row) + at;
        const uint32_t *p = reinterpret_cast<const uint32_t *>(first & ~uintptr_t{3});
        const int skip = static_cast<int>(first & 3), have = row != nullptr ? kb - at : 0;  // the row's bytes from `at` on
        uint32_t last = have > 0 ? __ldg(p) : 0u;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            const uint32_t next = have > 4 * (i + 1) - skip ? __ldg(p + i + 1) : 0u;
            const int left = have - 4 * i;
            const uint32_t v = __funnelshift_r(last, next, 8 * skip);
            w[i] = left >= 4 ? v : left <= 0 ? 0u : v & ((1u << (8 * left)) - 1u);
            last = next;
        }
    }
}

// TOut void: the gate/up form
template <typename TOut, int NT, int V>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(G8_THREADS, 1)
    mx8_gemm_kernel(const __grid_constant__ CUtensorMap tmA16, const __grid_constant__ CUtensorMap tmA32,
                    const __grid_constant__ CUtensorMap tmA64, const __grid_constant__ CUtensorMap tmB0,
                    const __grid_constant__ CUtensorMap tmB1, const G8Params p) {
    using L = G8Layout<NT>;
    constexpr bool GATE_UP = std::is_same<TOut, void>::value;
    constexpr int OWN = GATE_UP ? 64 : 128;  // features of a CTA's tile
    extern __shared__ uint8_t g8_smem_raw[];
    uint8_t *smem = g8_smem_raw + ((1024u - (smem_u32(g8_smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::STAGES * L::STAGE);
    int2 *list = reinterpret_cast<int2 *>(smem + L::STAGES * L::STAGE + 512);  // first row; expert, only block, row count
    uint8_t *staging0 = smem + L::STAGES * L::STAGE + 512 + G8_LIST * 8;
    float *exchange = reinterpret_cast<float *>(staging0 + G8_SF_GROUPS * L::SF_BYTES);
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word, warp_blocks[G8_THREADS / 32];
    volatile int *abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_cta_rank();
    const bool leader = rank == 0;
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int i) { return bar0 + 8u * i; };  // the even CTA's, both CTAs' copies
    auto empty_bar = [&](int i) { return bar0 + 8u * (L::STAGES + i); };
    auto tfull_bar = [&](int i) { return bar0 + 8u * (2 * L::STAGES + i); };
    auto tempty_bar = [&](int i) { return bar0 + 8u * (2 * L::STAGES + 2 + i); };  // the even CTA's
    auto sfull_bar = [&](int i) { return bar0 + 8u * (2 * L::STAGES + 4 + i); };   // the even CTA's, both CTAs' scales
    auto sempty_bar = [&](int i) { return bar0 + 8u * (2 * L::STAGES + 4 + L::UNITS + i); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::STAGES; ++i) {
            mbar_init(full_bar(i), 1);
            mbar_init(empty_bar(i), 1);
        }
        for (int i = 0; i < L::UNITS; ++i) {
            mbar_init(sfull_bar(i), 2 * 4);  // a group's warps of each CTA
            mbar_init(sempty_bar(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull_bar(i), 1);
            mbar_init(tempty_bar(i), 2 * G8_EPI_WARPS);
        }
        abort_word = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA16);
        tma_prefetch_desc(&tmA32);
        tma_prefetch_desc(&tmA64);
        tma_prefetch_desc(&tmB0);
        if (GATE_UP) tma_prefetch_desc(&tmB1);
    }
    if (warp == 1) {
        tmem_alloc2(smem_u32(&tmem_slot), 512);
        tmem_relinquish2();
    }
    tc_fence_before();
    cluster_sync_all();  // the other CTA's barriers are initialised before any use
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
    griddep_wait();
    griddep_launch_dependents();

    // the units that hold rows, in order, when they fit the list: each thread looks
    // at an expert (its three entries need one round trip; through the blocks'
    // expert they need two, 0.6 us more), and a scan places its units; both CTAs of
    // a pair build the same list
    int n_blocks = 0;
    for (int e0 = 0; e0 < p.tab.E && n_blocks <= G8_LIST; e0 += G8_THREADS) {
        const int g = e0 + static_cast<int>(threadIdx.x);
        const bool in = g < p.tab.E;
        const int size = in ? __ldg(p.tab.sizes + g) : 0, m = in ? __ldg(p.tab.offsets + g) : 0;
        const int blocks = p.m_blocks - (in ? __ldg(p.tab.padded + g) / 128 : 0);  // more hold no more rows than 2^24 - 1
        const int rows = max(0, min(rows_there(p.tab, size, m), min(max(blocks, 0), (1 << 24) - 1) * 128));
        const int mine = rows / NT + (rows % NT ? 1 : 0);
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int before = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? before : 0;
        }
        if (lane == 31) warp_blocks[warp] = upto;
        __syncthreads();
        int at = n_blocks + upto - mine;
        for (int w = 0; w < G8_THREADS / 32; ++w) {
            at += w < warp ? warp_blocks[w] : 0;
            n_blocks += warp_blocks[w];
        }
        for (int u = 0; u < mine && at + u < G8_LIST; ++u)
            list[at + u] = make_int2(m + u * NT, g << 10 | (mine == 1 ? 512 : 0) | min(rows - u * NT, NT));
        __syncthreads();
    }
    const int listed = n_blocks <= G8_LIST ? n_blocks : -1;
    // Tile b * n_tiles + n is unit (or block) b by feature tile n; a pair takes every
    // `pairs`-th.
    const int n_units = listed >= 0 ? listed : p.m_blocks, pairs = static_cast<int>(gridDim.x >> 1);
    const int step_b = pairs / p.n_tiles, step_n = pairs % p.n_tiles;
    struct Cursor {
        int b, n;
    };
    const Cursor first = {static_cast<int>(blockIdx.x >> 1) / p.n_tiles, static_cast<int>(blockIdx.x >> 1) % p.n_tiles};
    auto live = [&](const Cursor &c) { return c.b < n_units; };
    auto advance = [&](Cursor &c) {
        c.b += step_b;
        c.n += step_n;
        if (c.n >= p.n_tiles) {
            c.n -= p.n_tiles;
            ++c.b;
        }
    };
    auto tile_at = [&](const Cursor &c) {
        G8Tile ti;
        ti.n0 = c.n * (2 * OWN) + static_cast<int>(rank) * OWN;
        if (listed >= 0) {
            const int2 e = list[c.b];
            ti.g = e.y >> 10;
            ti.m_start = e.x;
            ti.rows = e.y & 511;
            ti.single = (e.y & 512) != 0;
        } else {
            const Mx4Block k = mx_unit_of<NT>(p.tab, c.b, p.m_blocks);
            ti.g = k.g;
            ti.m_start = k.m_start;
            ti.rows = k.rows;
            ti.single = p.tab.sizes[k.g] <= NT;
        }
        return ti;
    };
    auto columns_of = [](const G8Tile &ti) { return (ti.rows + 31) & ~31; };

    if (warp == 0) {
        // -------------------------------- copies --------------------------------
        const uint64_t keep = l2_policy_evict_last(), pass = l2_policy_evict_first();
        const uint32_t ring = smem_u32(smem), full_leader = smem_map_rank(full_bar(0), 0);
        int stage = 0;
        uint32_t phase = 0;
        long issued = 0;
        bool ok = true;
        for (Cursor t = first; live(t) && ok; advance(t)) {
            const G8Tile ti = tile_at(t);
            const int columns = __shfl_sync(0xffffffffu, columns_of(ti), 0);
            if (columns == 0) continue;
            const int half = columns / 2;  // a multiple of 16 rows
            const int row0 = __shfl_sync(0xffffffffu, ti.m_start, 0) + static_cast<int>(rank) * half;
            const int g = __shfl_sync(0xffffffffu, ti.g, 0), n0 = ti.n0;
            const uint64_t pol = __shfl_sync(0xffffffffu, ti.single ? 1 : 0, 0) ? pass : keep;  // an only unit's weights are read once
            for (int s = 0; s < p.slices; ++s) {
                ok = __all_sync(0xffffffffu, mbar_wait_cluster_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) != 0;
                if (!ok) break;
                const uint32_t a = ring + stage * L::STAGE, b = a + 2 * G8_A_HALF, fb = full_leader + 8u * stage;
                const int halves = s * G8_SLICE + 128 < p.K ? 2 : 1;
                if (leader) expect_elect(full_bar(stage), 2 * halves * (G8_A_HALF + half * 128));
                for (int h = 0; h < halves; ++h) {
                    const int k0 = s * G8_SLICE + h * 128;
                    copy_3d_elect(a + h * G8_A_HALF, &tmB0, fb, k0, n0, g, pol);
                    if (GATE_UP) copy_3d_elect(a + h * G8_A_HALF + G8_A_HALF / 2, &tmB1, fb, k0, n0, g, pol);
                    // copies of 64, 32 and 16 rows; the wide tiles' without a loop, which paces
                    // them (32768 rows 744 us with it, 718 without), the others' with one
                    // (384 rows 60.5 us with it, 61.0 without)
                    uint32_t to = b + h * L::B_HALF;
                    if constexpr (NT == 256) {
                        int r = row0;
                        if (half >= 64) {
                            copy_2d_elect(to, &tmA64, fb, k0, r, keep);
                            to += 64 * 128;
                            r += 64;
                            if (half == 128) copy_2d_elect(to, &tmA64, fb, k0, r, keep);
                        }
                        if (half & 32) {
                            copy_2d_elect(to, &tmA32, fb, k0, r, keep);
                            to += 32 * 128;
                            r += 32;
                        }
                        if (half & 16) copy_2d_elect(to, &tmA16, fb, k0, r, keep);
                    } else {
                        for (int i = 0; i < half; i += 64) {
                            const int have = half - i;
                            const uint32_t at = to + i * 128;
                            if (have >= 64) {
                                copy_2d_elect(at, &tmA64, fb, k0, row0 + i, keep);
                            } else {
                                if (have & 32) copy_2d_elect(at, &tmA32, fb, k0, row0 + i, keep);
                                if (have & 16) copy_2d_elect(at + (have & 32) * 128, &tmA16, fb, k0, row0 + i + (have & 32), keep);
                            }
                        }
                    }
                }
                ++issued;
                if (++stage == L::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (leader && lane == 0 && (!ok || *abort_flag)) {
            // both CTAs' copies in flight land before shared memory goes away
            for (long j = 1; j <= L::STAGES && j <= issued; ++j) {
                const long i = issued - j;
                g8_drain(full_bar(static_cast<int>(i % L::STAGES)), static_cast<uint32_t>((i / L::STAGES) & 1));
            }
        }
        __syncwarp();
        g8_flag_rows_past(p.tab, lane, p.err);
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        if (leader) {
            const uint32_t ring = smem_u32(smem);
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return __all_sync(0xffffffffu, mbar_wait_cluster_bounded(bar, parity, abort_flag, p.err)) != 0;
            };
            int stage = 0, unit = 0;
            G8Slots slots;
            uint32_t phase = 0, uphase = 0, last_bar = 0, last_parity = 0;
            bool ok = true, committed = false;
            for (Cursor t = first; live(t) && ok; advance(t)) {
                const int columns = __shfl_sync(0xffffffffu, columns_of(tile_at(t)), 0);
                if (columns == 0) continue;
                const uint32_t idesc = idesc_mxf8(256, static_cast<uint32_t>(columns));
                slots.take(columns);
                ok = wait(tempty_bar(slots.first), slots.parity(slots.first) ^ 1u);
                if (slots.both) ok = ok && wait(tempty_bar(1), slots.parity(1) ^ 1u);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(slots.first * G8_ACC);
                for (int s = 0; s < p.slices; ++s) {
                    const int in_unit = s % G8_UNIT;
                    if (in_unit == 0) ok = wait(sfull_bar(unit), uphase);
                    ok = ok && wait(full_bar(stage), phase);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = ring + stage * L::STAGE;
                    const uint64_t a_desc = smem_desc_sw128(a), b_desc = smem_desc_sw128(a + 2 * G8_A_HALF);
                    const uint32_t sfa = tmem + L::SF_COL0 + unit * L::UNIT_COLS + in_unit * L::SF_COLS, sfb = sfa + 8u;
                    const int left = static_cast<int>(p.K) - s * G8_SLICE;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (k * 32 >= left) break;
                        const uint32_t id = k & 3, h = k >> 2;
                        tc_mma2_mxf8(d, a_desc + (G8_A_HALF >> 4) * h + 2u * id, b_desc + (L::B_HALF >> 4) * h + 2u * id,
                                     idesc | (id << 29) | (id << 4), sfa + 4u * h, sfb + 4u * L::ROWS * h, (s | k) != 0 ? 1u : 0u);
                    }
                    tc_commit2_both_elect(empty_bar(stage));  // frees the stage in both CTAs
                    last_bar = empty_bar(stage);
                    last_parity = phase;
                    committed = true;
                    if (++stage == L::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (in_unit == G8_UNIT - 1 || s == p.slices - 1) {
                        tc_commit2_both_elect(sempty_bar(unit));
                        if (++unit == L::UNITS) {
                            unit = 0;
                            uphase ^= 1u;
                        }
                    }
                }
                if (!ok) break;
                tc_commit2_both_elect(tfull_bar(slots.first));
                slots.done();
            }
            if (!ok && committed && lane == 0) g8_drain(last_bar, last_parity);
        }
    } else if (warp >= G8_SF_WARP0) {
        // -------------------------------- scales --------------------------------
        // groups of four warps take the units in turn
        const int r = (threadIdx.x - G8_SF_WARP0 * 32) & 127;
        const int group = (warp - G8_SF_WARP0) >> 2;
        const int kb = static_cast<int>(p.K / 32), span = p.units * 8 * G8_UNIT;
        uint8_t *const staging = staging0 + group * L::SF_BYTES;
        constexpr int WORDS = 2 * G8_UNIT;
        uint32_t vw[G8_AHEAD][WORDS], vr[G8_AHEAD][L::ROWS][WORDS];  // weights', rows'
        Cursor lt = first;                      // next unit to load: its tile, its scale bytes
        int at = group * 8 * G8_UNIT;           // byte offset of that unit in its row
        const uint8_t *pw = nullptr, *pr[L::ROWS];  // the thread's rows; null where there is none
        auto next_tile = [&]() {
            for (; live(lt); advance(lt)) {
                const G8Tile ti = tile_at(lt);
                if (ti.rows == 0) continue;
                if (at >= span) {  // past this tile: the units go on in the next one
                    at -= span;
                    continue;
                }
                const bool up = GATE_UP && r >= OWN;
                const int64_t f = ti.n0 + (up ? r - OWN : r);
                pw = f < p.N ? (up ? p.sf_b1 : p.sf_b0) + (static_cast<int64_t>(ti.g) * p.N + f) * kb : nullptr;
#pragma unroll
                for (int i = 0; i < L::ROWS; ++i)
                    pr[i] = 128 * i + r < ti.rows ? p.sf_a + (static_cast<int64_t>(ti.m_start) + 128 * i + r) * kb : nullptr;
                return;
            }
        };
        next_tile();
        auto load = [&](uint32_t(&w)[WORDS], uint32_t(&x)[L::ROWS][WORDS]) {
            load_scales<V>(w, pw, kb, at);
#pragma unroll
            for (int i = 0; i < L::ROWS; ++i) load_scales<V>(x[i], pr[i], kb, at);
            at += 8 * G8_UNIT * G8_SF_GROUPS;
            if (at >= span) next_tile();
        };
        int ahead = 0;  // units in registers
#pragma unroll
        for (int j = 0; j < G8_AHEAD; ++j)
            if (live(lt)) {
                load(vw[j], vr[j]);
                ++ahead;
            }
        int unit = group;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && ahead > 0) {
#pragma unroll
            for (int j = 0; j < G8_AHEAD; ++j) {
                if (!ok || ahead == 0) continue;
                // a slice's 512 bytes for each half of the weights, then for each half and
                // 128 rows: a row's word at 4 r
                uint32_t *const mine = reinterpret_cast<uint32_t *>(staging) + r;
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    uint32_t *const slice = mine + (i >> 1) * L::SF_COLS * 32;
                    slice[(i & 1) * 128] = vw[j][i];
#pragma unroll
                    for (int n = 0; n < L::ROWS; ++n) slice[(2 + (i & 1) * L::ROWS + n) * 128] = vr[j][n][i];
                }
                int free = 1;
                if (lane == 0) free = mbar_wait_cluster_bounded(sempty_bar(unit), phase ^ 1u, abort_flag, p.err) ? 1 : 0;
                free = __shfl_sync(0xffffffffu, free, 0);
                // every thread of the group has stored.  A warp whose wait gave up
                // comes here too and takes the group along
                ok = g8_all<128>(1 + group, free != 0);
                if (!ok) continue;
                // each warp puts all rows' scales into its own lane quarter:
                // lane i, column c holds row 32 c + i
                tc_fence_after();
                const uint32_t col = tmem + ((warp & 3u) << 21) + L::SF_COL0 + unit * L::UNIT_COLS;
#pragma unroll
                for (int i = 0; i < L::UNIT_COLS / 8; ++i)
                    tmem_st8(col + 8u * i, quarter_scales(staging + 1024 * i + lane * 4), quarter_scales(staging + 1024 * i + 512 + lane * 4));
                tmem_st_wait();
                tc_fence_before();
                g8_all<128>(1 + group, true);  // the group has read: the next unit may be stored
                if (lane == 0) {
                    if (leader)
                        mbar_arrive(sfull_bar(unit));
                    else
                        mbar_arrive_remote(smem_map_rank(sfull_bar(unit), 0));
                }
                unit += G8_SF_GROUPS;
                if (unit >= L::UNITS) {
                    unit -= L::UNITS;
                    phase ^= 1u;
                }
                --ahead;
                if (live(lt)) {
                    load(vw[j], vr[j]);
                    ++ahead;
                }
            }
        }
    } else {
        // ------------------------------- epilogue -------------------------------
        // two warps to a lane quarter, each with every other 32 (gate/up: 16) columns,
        // rows of the block; a lane is a feature
        const int q = warp & 3, set = (warp - G8_EPI_WARP0) >> 2;
        const uint32_t tempty_leader = smem_map_rank(tempty_bar(0), 0);  // + 8 * acc
        // gate/up: quarters q and q + 2 hold the same features' gate and up sums
        const int pair = set * 2 + (q & 1);
        const bool up = GATE_UP && q >= 2;
        float *send = exchange + pair * 1024 + (up ? 256 : 0), *take = exchange + pair * 1024 + (up ? 0 : 256);
        G8Slots slots;
        uint32_t fills = 0;  // a bit a slot, modulo 2: a unit in both fills the first one's barrier only
        for (Cursor t = first; live(t); advance(t)) {
            const G8Tile ti = tile_at(t);
            if (ti.rows == 0) continue;
            slots.take(columns_of(ti));
            const int acc = slots.first;
            int ready = 1;
            if (lane == 0) ready = mbar_wait_cluster_bounded(tfull_bar(acc), fills >> acc & 1u, abort_flag, p.err) ? 1 : 0;
            fills ^= 1u << acc;
            ready = __shfl_sync(0xffffffffu, ready, 0);
            if constexpr (GATE_UP) ready = g8_all<64>(1 + G8_SF_GROUPS + pair, ready != 0);  // both or neither go on
            if (!ready) break;
            tc_fence_after();
            const uint32_t d = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * G8_ACC);
            if constexpr (GATE_UP) {
                const int f0 = ti.n0 + (q & 1) * 32;
                uint8_t *const q_h = p.q_h + static_cast<int64_t>(ti.m_start) * p.N + f0 + lane;
                uint8_t *const sf_h = p.sf_h + static_cast<int64_t>(ti.m_start) * (p.N / 32) + f0 / 32;
                if (f0 < p.N) {
                    uint32_t v[16];
                    int buffer = 0;
                    if (set * 16 < ti.rows) tmem_ld16(d + set * 16, v);
#pragma unroll 1
                    for (int c = set * 16; c < ti.rows; c += 32) {
                        tmem_ld_wait();
                        // the gate's warp takes the first 8 rows, up's the others; two
                        // buffers in turn, so the next exchange's stores cannot pass
                        // this one's reads
#pragma unroll
                        for (int i = 0; i < 8; ++i) send[buffer + i * 32 + lane] = __uint_as_float(up ? v[i] : v[8 + i]);
                        float own[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) own[i] = __uint_as_float(up ? v[8 + i] : v[i]);
                        if (c + 32 < ti.rows) tmem_ld16(d + c + 32, v);
                        g8_all<64>(1 + G8_SF_GROUPS + pair, true);
                        const int row0 = c + (up ? 8 : 0);
                        uint32_t scale = 0;
                        uint8_t *to = q_h + static_cast<int64_t>(row0) * p.N;
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {  // two rows at a time
                            float h[2];
                            uint32_t s[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float other = take[buffer + (i + j) * 32 + lane];
                                const float g = up ? other : own[i + j], u = up ? own[i + j] : other;
                                // silu from exp(-|g|), which neither overflows nor leaves the quotient's range
                                const float e = __expf(-fabsf(g));
                                h[j] = __fdividef(g < 0.0f ? g * e : g, 1.0f + e) * u;
                                s[j] = mx8_scale(__reduce_max_sync(0xffffffffu, magnitude_bits(h[j])));
                                scale = lane == i + j ? s[j] : scale;
                            }
                            const uint32_t e = e4m3x2(h[0] * mx8_inverse(s[0]), h[1] * mx8_inverse(s[1]));
                            if (row0 + i < ti.rows) *to = static_cast<uint8_t>(s[0] == 255u ? 0u : e);
                            to += p.N;
                            if (row0 + i + 1 < ti.rows) *to = static_cast<uint8_t>(s[1] == 255u ? 0u : e >> 8);
                            to += p.N;
                        }
                        if (lane < 8 && row0 + lane < ti.rows)
                            sf_h[static_cast<int64_t>(row0 + lane) * (p.N / 32)] = static_cast<uint8_t>(scale);
                        buffer ^= 512;
                    }
                }
            } else {
                const int64_t f = ti.n0 + q * 32 + lane;
                TOut *const out = static_cast<TOut *>(p.out) + static_cast<int64_t>(ti.m_start) * p.N + f;
#pragma unroll 1
                for (int c = set * 32; c < ti.rows; c += 64) {
                    uint32_t v[32];
                    tmem_ld32(d + c, v);
                    tmem_ld_wait();
                    if (f < p.N) {
                        // a running pointer: with an address worked out for each store
                        // this loop took longer than the stores (32768 rows of 16
                        // experts, 7168 x 2048: 400 us, so 340)
                        TOut *to = out + static_cast<int64_t>(c) * p.N;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (c + i < ti.rows) *to = from_f32<TOut>(__uint_as_float(v[i]));
                            to += p.N;
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                for (int i = acc; i <= (slots.both ? 1 : acc); ++i) {
                    if (leader)
                        mbar_arrive(tempty_bar(i));
                    else
                        mbar_arrive_remote(tempty_leader + 8u * static_cast<uint32_t>(i));
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // neither CTA leaves while the pair's MMAs or arrivals may touch it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc2(tmem, 512);
    }
}

bool rows_map(CUtensorMap *m, const uint8_t *q, int64_t K, int64_t rows, uint32_t box_rows) {
    const uint64_t dims[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {static_cast<uint64_t>(K)};
    const uint32_t box[2] = {128, box_rows};
    return encode_tma_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q, dims, strides, box, 1);
}

// of 16, 32 and 64 rows
bool rows_maps(CUtensorMap *m, const uint8_t *q, int64_t K, int64_t rows) {
    return rows_map(m, q, K, rows, 16) && rows_map(m + 1, q, K, rows, 32) && rows_map(m + 2, q, K, rows, 64);
}

bool weights_map(CUtensorMap *m, const uint8_t *q, int64_t K, int64_t N, int64_t E, uint32_t box_rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E)};
    const uint64_t strides[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N * K)};
    const uint32_t box[3] = {128, box_rows, 1};
    return encode_tma_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, q, dims, strides, box, 1);
}

template <typename TOut, int NT, int V>
cudaError_t launch_v(const CUtensorMap *maps, G8Params p, cudaStream_t stream) {
    using L = G8Layout<NT>;
    p.units = (p.slices + G8_UNIT - 1) / G8_UNIT;
    auto kern = mx8_gemm_kernel<TOut, NT, V>;
    static std::atomic<bool> attr_done[64];  // zero-initialised; several host threads may launch
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    const int64_t tiles = static_cast<int64_t>(p.m_blocks) * p.n_tiles, pairs = device_sm_count() / 2;
    return launch_pdl(kern, dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs))), dim3(G8_THREADS), L::SMEM, stream,
                      maps[0], maps[1], maps[2], maps[3], maps[4], p);
}

// the widest scale loads that K and the bases' alignment allow
template <typename TOut, int NT>
cudaError_t launch_n(const CUtensorMap *maps, const G8Params &p, cudaStream_t stream) {
    const uintptr_t bases = reinterpret_cast<uintptr_t>(p.sf_a) | reinterpret_cast<uintptr_t>(p.sf_b0) |
                            reinterpret_cast<uintptr_t>(p.sf_b1);
    if (p.K % 512 == 0 && (bases & 15u) == 0) return launch_v<TOut, NT, 16>(maps, p, stream);
    if (p.K % 256 == 0 && (bases & 7u) == 0) return launch_v<TOut, NT, 8>(maps, p, stream);
    if (p.K % 128 == 0 && (bases & 3u) == 0) return launch_v<TOut, NT, 4>(maps, p, stream);
    return launch_v<TOut, NT, 1>(maps, p, stream);
}

// Tiles of up to 256 rows where experts have many: the weights enter shared
// memory half as often.  They leave three stages for four, and the wide tiles'
// epilogue runs alone (both accumulator slots are one tile's), which a long K earns
// back, and a shorter one only when there are several rounds of tiles: the product
// from K of 1024, the gate/up form, whose epilogue is longer, from 2048 and 512 rows
// an expert; tiles that do not fill a round are better narrow, and more.  Narrow / wide, us,
// of groups whose sizes differ as routing makes them (rows on average):
//   7168 x 2048, 256 experts, 128 rows each: 828 / 730, gate/up 1730 / 1455
//   7168 x 2048, 64 experts: 32 rows each 166 / 165 and 316 / 313, 64 rows 177 / 174
//   and 331 / 326, 256 rows 321 / 244 and 678 / 520; 16 experts, 2048 rows 515 / 370
//   2048 x 768, 64 experts: 128 rows each 29 / 30, gate/up 61 / 65; 384 rows 57.5 / 62.5,
//   124 / 128; gate/up 768 rows 222 / 210, 1024 rows 295 / 269
//   2048 x 2048: 8 experts, 4096 rows 158 / 125, gate/up 352 / 327; gate/up 1024 rows
//   97 / 90, 64 experts, 256 rows 221 / 223
//   32 experts, 1024 rows, 1024 x 2048: 95.6 / 90.8, gate/up 248 / 274; 512 x 2048: 68.9 /
//   70.0, gate/up 219 / 235; 64 experts, 128 rows, 256 x 4096: 43.8 / 48.9
//   rounds of wide tiles: 0.2 (600 rows, 7168 x 512) 24 / 26, 0.4 (4096 rows) 24 / 28,
//   gate/up 0.8 of them 44 / 33; 1.7 (16 experts, 500 rows, 2048 x 1024) 28 / 30
template <typename TOut>
cudaError_t launch_typed(const CUtensorMap *maps, const G8Params &p, int64_t n_rows, int64_t E, cudaStream_t stream) {
    const int64_t tiles = (n_rows + 255) / 256 * p.n_tiles, pairs = device_sm_count() / 2;
    const bool deep = std::is_same<TOut, void>::value ? p.K >= 2048 && n_rows >= 512 * E : p.K >= 1024;
    const bool pays = p.K >= 4096 ? 4 * tiles >= 3 * pairs : deep && tiles >= 4 * pairs;
    if (n_rows > 64 * E && pays) return launch_n<TOut, 256>(maps, p, stream);
    return launch_n<TOut, 128>(maps, p, stream);
}

G8Params params(const uint8_t *sf_a, const uint8_t *sf_b0, const uint8_t *sf_b1, const MxTables &tab, int64_t m_blocks,
                int64_t N, int64_t K, int tile, int32_t *err) {
    G8Params p{};
    p.sf_a = sf_a;
    p.sf_b0 = sf_b0;
    p.sf_b1 = sf_b1;
    p.tab = tab;
    p.m_blocks = static_cast<int>(m_blocks);
    p.N = N;
    p.K = K;
    p.n_tiles = static_cast<int>((N + tile - 1) / tile);
    p.slices = static_cast<int>((K + G8_SLICE - 1) / G8_SLICE);
    p.err = err;
    return p;
}

}  // namespace

cudaError_t launch_grouped_gemm_mx8(const uint8_t *q_a, const uint8_t *sf_a, const uint8_t *q_b, const uint8_t *sf_b,
                                    const MxTables &tab, int64_t m_blocks, int64_t n_rows, int64_t N, int64_t K,
                                    int64_t E, int out_dtype, void *C, int32_t *err, cudaStream_t stream) {
    CUtensorMap maps[5];
    if (!rows_maps(maps, q_a, K, n_rows) || !weights_map(&maps[3], q_b, K, N, E, 128)) return cudaErrorInvalidValue;
    maps[4] = maps[3];
    G8Params p = params(sf_a, sf_b, sf_b, tab, m_blocks, N, K, 256, err);
    p.out = C;
    if (out_dtype == kF32) return launch_typed<float>(maps, p, n_rows, E, stream);
    if (out_dtype == kBF16) return launch_typed<__nv_bfloat16>(maps, p, n_rows, E, stream);
    return launch_typed<__half>(maps, p, n_rows, E, stream);
}

cudaError_t launch_grouped_gate_up_silu_mx8(const uint8_t *q_a, const uint8_t *sf_a, const uint8_t *q_gate,
                                            const uint8_t *sf_gate, const uint8_t *q_up, const uint8_t *sf_up,
                                            const MxTables &tab, int64_t m_blocks, int64_t n_rows, int64_t d_h,
                                            int64_t d_e, int64_t E, uint8_t *q_h, uint8_t *sf_h, int32_t *err,
                                            cudaStream_t stream) {
    CUtensorMap maps[5];
    if (!rows_maps(maps, q_a, d_h, n_rows) || !weights_map(&maps[3], q_gate, d_h, d_e, E, 64) ||
        !weights_map(&maps[4], q_up, d_h, d_e, E, 64))
        return cudaErrorInvalidValue;
    G8Params p = params(sf_a, sf_gate, sf_up, tab, m_blocks, d_e, d_h, 128, err);
    p.q_h = q_h;
    p.sf_h = sf_h;
    return launch_typed<void>(maps, p, n_rows, E, stream);
}

}  // namespace moe
