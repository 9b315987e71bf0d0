// mx4_gemm.cu -- the grouped product of 4-bit rows with 4-bit expert weights
// on the block-scaled tensor cores (tcgen05.mma kind::mxf4):
//
//   C[r, n] = sum over k of (qa 2^sa)[r, k] * (qb 2^sb)[expert of r][n, k]
//
// and the gate/up form, h = silu(A Wg^T) * (A Wu^T), whose epilogue quantises
// h (a thread holds 32 consecutive features of a row: one scale block).
//
// A persistent CTA works on tiles of 128 rows of a dispatch block by BN
// columns.  Roles:
//   warp 0      TMA: 128-byte (256-element) slices of the rows and the weights
//               into a ring of 128-byte-swizzled stages;
//   warps 10-17 scales, two groups in turn: each thread loads its row's 8 scale
//               bytes of a slice, several slices ahead; through shared memory
//               each warp gets every row's and stores them to its quarter of
//               tensor memory;
//   warp 1      one elected lane: four K = 64 MMAs a slice;
//   warps 2-9   epilogue, from one of two accumulators while the other fills.
//
// 32,768 rows, 256 experts, 7168 x 2048, bf16 out: 423 us, 2.3 PFLOP/s (323 us
// for its bytes).  Shared memory bounds a full tile: a 128 x 192 slice brings 40 KB
// in and the tensor cores read them once, 640 of its about 950 cycles at 128
// bytes each, against 340 for its MMAs alone; the rest is the hand-over between
// the roles.  And blocks are not full: 256 groups make 409 blocks of 128, 60%
// more rows than there are, each reading all of its expert's weights.  192
// columns take the tensor memory that two accumulators and the stages' scales
// leave; when that took 452 us, 128 columns took 690, 256 with a single
// accumulator 462.  The gate/up form, twice the columns: 869 us.
#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"

namespace moe {
namespace {

constexpr int MG_BM = 128;
constexpr int MG_SLICE = 256;       // elements of K per stage: 128 bytes of a row
constexpr int MG_A_BYTES = MG_BM * 128;
constexpr int MG_THREADS = 576;
constexpr int MG_EPI_WARP0 = 2, MG_EPI_WARPS = 8, MG_SF_WARP0 = 10, MG_SF_GROUPS = 2;
constexpr int MG_AHEAD = 4;         // slices of scales in registers ahead of the ring
constexpr int MG_LIST = 512;        // M blocks with rows that the shared-memory list holds
constexpr int MG_BN = 192;         // columns of a tile
constexpr int MG_BOX_ROWS = 32;     // rows of a copy: a block loads as many as hold its rows

template <int BN> struct MgLayout {
    static constexpr int B_BYTES = BN * 128;
    static constexpr int STAGE = MG_A_BYTES + B_BYTES;
    static constexpr int SF_HALVES = (BN + 127) / 128;          // 128-row groups of B's scales
    static constexpr int SF_BYTES = 2 * (1 + SF_HALVES) * 512;  // a slice's scales: two 128-element groups of K
    static constexpr int SF_COLS = 2 * 4 * (1 + SF_HALVES);     // and their tensor-memory columns
    static constexpr int LIST_BYTES = MG_LIST * 8;
    static constexpr int FIXED = 1024 + 512 + LIST_BYTES + 2 * MG_SF_GROUPS * SF_BYTES;
    static constexpr int STAGES = (232448 - 256 - FIXED) / STAGE;
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static constexpr int SF_COL0 = 2 * BN;                      // after the two accumulators
    static_assert(SF_COL0 + STAGES * SF_COLS <= 512, "tensor memory");
    static_assert(STAGE % 1024 == 0, "swizzle atoms");
    static_assert(STAGES > MG_SF_GROUPS, "the groups work on different stages");
};

struct MgParams {
    const uint8_t *sf_a, *sf_b0, *sf_b1;  // b1: the up weights of the gate/up form
    MxTables tab;
    void *out;
    uint8_t *q_h, *sf_h;
    int32_t *err;
    int m_blocks, n_tiles, slices;
    int wide;  // rows of out start 32-byte aligned
    int64_t N, K;
};

struct MgTile {
    int g, m_start, rows, n0;
};

// kind::mxf4: e2m1 by e2m1, e8m0 scales; the scale id (0 or 2: which two of a
// cell's four bytes) is added per MMA.
//   bits 4-5 B scale id; 7-9 A format, 10-12 B format (1 = e2m1); 17-22 N >> 3;
//   23 scale type (1 = e8m0); 24-28 M >> 4; 29-30 A scale id; 31 K (0 = 64)
__host__ __device__ constexpr uint32_t idesc_mxf4(uint32_t M, uint32_t N) {
    return (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (1u << 23) | ((M >> 4) << 24);
}

// The MMA warp runs whole, its operands the same in every lane, and one
// elected lane issues: the operands then come from uniform registers.  Issued
// by one lane of a divergent branch instead, each operand is moved there
// first, and an MMA took 113 cycles to issue, a copy 71.
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tc_commit_elect(uint32_t bar) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar) : "memory");
}

// A barrier of one scale group: whether `yes` holds in all its 128 threads.
__device__ __forceinline__ bool mg_group_all(int id, bool yes) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.and.aligned.pred q, %1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(id), "r"(yes ? 1u : 0u)
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

__device__ __forceinline__ void mg_drain(uint32_t bar, uint32_t parity) {
    const unsigned long long start = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - start > kWaitTimeoutNs) return;
}

// Whether the blocks name rows past the call's, into the error word; by a warp of each
// CTA that has nothing else left to do.  By blocks: weights may have more experts than
// the tables have entries, as long as no block is one's.
__device__ __forceinline__ void mg_flag_rows_past(const MxTables &t, int m_blocks, int lane, int32_t *err) {
    if (!err) return;
    bool past = false;
    for (int bx = static_cast<int>(blockIdx.x) * 32 + lane; bx < m_blocks; bx += static_cast<int>(gridDim.x) * 32) {
        const int g = static_cast<int>(min(static_cast<unsigned>(t.gidx[bx]), static_cast<unsigned>(t.E - 1)));
        const int off = static_cast<int>(static_cast<uint32_t>(bx) * 128u - static_cast<uint32_t>(t.padded[g]));
        const int named = min(t.sizes[g] - off, 128);
        past |= (named > 0) & (rows_there(t, named, off + t.offsets[g]) < named);
    }
    if (past) atomicExch(err, kErrDeviceFlag);
}

// 8 scale bytes from byte `at` on of a row of kb of them (null: zeros); bytes
// past kb are 0 (their elements are zeros too).  V: the load width that kb and
// the bases' alignment allow.
template <int V> __device__ __forceinline__ uint2 load_scales(const uint8_t *row, int kb, int at) {
    uint2 v = make_uint2(0u, 0u);
    if (!row) return v;
    const uint8_t *p = row + at;
    if constexpr (V == 8) {
        v = __ldg(reinterpret_cast<const uint2 *>(p));
    } else if constexpr (V == 4) {
        v.x = __ldg(reinterpret_cast<const uint32_t *>(p));
        if (at + 4 < kb) v.y = __ldg(reinterpret_cast<const uint32_t *>(p + 4));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (at + i < kb) v.x |= static_cast<uint32_t>(__ldg(p + i)) << (8 * i);
            if (at + 4 + i < kb) v.y |= static_cast<uint32_t>(__ldg(p + 4 + i)) << (8 * i);
        }
    }
    return v;
}

__device__ __forceinline__ void store_32_bytes(void *dst, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 32 values of one row, whose place is 32-byte aligned: whole sectors a store
template <typename TOut> __device__ __forceinline__ void store_row(TOut *dst, const uint32_t (&r)[32]) {
    constexpr int per = 32 / sizeof(TOut);
#pragma unroll
    for (int i = 0; i < 32 / per; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (sizeof(TOut) == 4) {
                w[j] = r[8 * i + j];
            } else {
                constexpr int DT = std::is_same<TOut, __half>::value ? kF16 : kBF16;
                w[j] = pack2<DT>(__uint_as_float(r[16 * i + 2 * j]), __uint_as_float(r[16 * i + 2 * j + 1]));
            }
        }
        store_32_bytes(dst + per * i, w);
    }
}

// A warp's `rows` rows (one a lane) by `cols` of 32 columns, where rows are
// not 32-byte aligned or the columns end.  More than a few rows: 8 x 8 blocks
// transposed among the lanes, so that a store writes 8 columns of 4 rows; with
// one element of 32 rows a store, a 28 MB result of odd width took 166 us.
template <typename TOut>
__device__ __forceinline__ void store_block(TOut *dst, int64_t ld, const uint32_t (&r)[32], int rows, int cols, int lane) {
    if (rows <= 8) {
        if (lane < rows) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < cols) dst[lane * ld + i] = from_f32<TOut>(__uint_as_float(r[i]));
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < 32; c += 8) {
        if (c >= cols) return;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = r[c + i];
#pragma unroll
        for (int s = 4; s >= 1; s >>= 1) {
            const bool high = lane & s;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j & s) continue;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w[j] : w[j | s], s);
                if (high)
                    w[j] = got;
                else
                    w[j | s] = got;
            }
        }
        const int col = c + (lane & 7);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = (lane & 24) + i;
            if (row < rows && col < cols) dst[row * ld + col] = from_f32<TOut>(__uint_as_float(w[i]));
        }
    }
}

template <typename TOut, bool GATE_UP, int BN, int V>
__global__ void __launch_bounds__(MG_THREADS, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                    const __grid_constant__ CUtensorMap tmB1, const MgParams p) {
    using L = MgLayout<BN>;
    constexpr int OUT_N = GATE_UP ? BN / 2 : BN;  // output columns of a tile
    extern __shared__ uint8_t mg_smem_raw[];
    uint8_t *smem = mg_smem_raw + ((1024u - (smem_u32(mg_smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::STAGES * L::STAGE);
    int2 *list = reinterpret_cast<int2 *>(smem + L::STAGES * L::STAGE + 512);  // first row; expert and row count
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word, warp_blocks[MG_THREADS / 32];
    volatile int *abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int i) { return bar0 + 8u * i; };
    auto empty_bar = [&](int i) { return bar0 + 8u * (L::STAGES + i); };
    auto tfull_bar = [&](int i) { return bar0 + 8u * (2 * L::STAGES + i); };
    auto tempty_bar = [&](int i) { return bar0 + 8u * (2 * L::STAGES + 2 + i); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::STAGES; ++i) {
            mbar_init(full_bar(i), 1 + 4);  // the copies' thread and a group's scale warps
            mbar_init(empty_bar(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull_bar(i), 1);
            mbar_init(tempty_bar(i), MG_EPI_WARPS);
        }
        abort_word = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), 512);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB0);
    }
    griddep_wait();
    griddep_launch_dependents();

    // the blocks that hold rows, in order, when they fit the list (the whole
    // CTA looks at MG_THREADS blocks at a time: the tables' latency is paid once)
    int n_blocks = 0;
    for (int b0 = 0; b0 < p.m_blocks && n_blocks <= MG_LIST; b0 += MG_THREADS) {
        const int bx = b0 + static_cast<int>(threadIdx.x);
        const Mx4Block b = bx < p.m_blocks ? mx_unit_of<128>(p.tab, bx, p.m_blocks) : Mx4Block{0, 0, 0};
        const uint32_t has = __ballot_sync(0xffffffffu, b.rows > 0);
        if (lane == 0) warp_blocks[warp] = __popc(has);
        __syncthreads();
        int at = n_blocks + __popc(has & ((1u << lane) - 1u));
        for (int w = 0; w < MG_THREADS / 32; ++w) {
            at += w < warp ? warp_blocks[w] : 0;
            n_blocks += warp_blocks[w];
        }
        if (b.rows > 0 && at < MG_LIST) list[at] = make_int2(b.m_start, b.g << 8 | b.rows);
        __syncthreads();
    }
    const int listed = n_blocks <= MG_LIST ? n_blocks : -1;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
    const int64_t total = static_cast<int64_t>(listed >= 0 ? listed : p.m_blocks) * p.n_tiles;
    auto tile_at = [&](int64_t t) {
        const int b = static_cast<int>(t / p.n_tiles);
        MgTile ti;
        ti.n0 = static_cast<int>(t - static_cast<int64_t>(b) * p.n_tiles) * OUT_N;
        if (listed >= 0) {
            const int2 e = list[b];
            ti.g = e.y >> 8;
            ti.m_start = e.x;
            ti.rows = e.y & 255;
        } else {
            const Mx4Block k = mx_unit_of<128>(p.tab, b, p.m_blocks);
            ti.g = k.g;
            ti.m_start = k.m_start;
            ti.rows = k.rows;
        }
        return ti;
    };

    if (warp == 0) {
        // -------------------------------- copies --------------------------------
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_last(), pass = l2_policy_evict_first();
            int stage = 0;
            uint32_t phase = 0;
            long issued = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const MgTile ti = tile_at(t);
                if (ti.rows == 0) continue;
                const int boxes = (ti.rows + MG_BOX_ROWS - 1) / MG_BOX_ROWS;
                // a short block is most often its expert's only one: its weights are read once
                const uint64_t pol_b = boxes == 1 ? pass : keep;
                for (int s = 0; s < p.slices; ++s) {
                    if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a = smem_u32(smem + stage * L::STAGE), b = a + MG_A_BYTES, fb = full_bar(stage);
                    mbar_arrive_expect_tx(fb, boxes * MG_BOX_ROWS * 128 + L::B_BYTES);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d_hint(a + i * MG_BOX_ROWS * 128, &tmA, fb, s * 128, ti.m_start + i * MG_BOX_ROWS, keep);
                    if (GATE_UP) {
                        tma_load_3d_hint(b, &tmB0, fb, s * 128, ti.n0, ti.g, pol_b);
                        tma_load_3d_hint(b + L::B_BYTES / 2, &tmB1, fb, s * 128, ti.n0, ti.g, pol_b);
                    } else {
                        tma_load_3d_hint(b, &tmB0, fb, s * 128, ti.n0, ti.g, pol_b);
                    }
                    ++issued;
                    if (++stage == L::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok || *abort_flag) {
                // copies in flight land before shared memory goes away (a
                // stage whose scales never came stays incomplete: bounded)
                for (long j = 1; j <= L::STAGES && j <= issued; ++j) {
                    const long i = issued - j;
                    mg_drain(full_bar(static_cast<int>(i % L::STAGES)), static_cast<uint32_t>((i / L::STAGES) & 1));
                }
            }
        }
        __syncwarp();
        mg_flag_rows_past(p.tab, p.m_blocks, lane, p.err);
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        constexpr uint32_t IDESC = idesc_mxf4(MG_BM, BN);
        const uint32_t ring = smem_u32(smem);
        auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag, p.err)) != 0;
        };
        int stage = 0, local = 0;
        uint32_t phase = 0, last_bar = 0, last_parity = 0;
        bool ok = true, committed = false;
        for (int64_t t = blockIdx.x; t < total && ok; t += gridDim.x) {
            if (__all_sync(0xffffffffu, tile_at(t).rows == 0)) continue;
            const int acc = local & 1;
            ok = wait(tempty_bar(acc), (static_cast<uint32_t>(local >> 1) & 1u) ^ 1u);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + static_cast<uint32_t>(acc * BN);
            for (int s = 0; s < p.slices; ++s) {
                ok = wait(full_bar(stage), phase);
                if (!ok) break;
                tc_fence_after();
                const uint32_t a = ring + stage * L::STAGE;
                const uint64_t a_desc = smem_desc_sw128(a), b_desc = smem_desc_sw128(a + MG_A_BYTES);
                const uint32_t sfa = tmem + L::SF_COL0 + stage * L::SF_COLS, sfb = sfa + 8u;
                const int left = static_cast<int>(p.K) - s * MG_SLICE;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k * 64 >= left) break;
                    const uint32_t id = (k & 1) * 2u;
                    tc_mma_mxf4(d, a_desc + 2u * k, b_desc + 2u * k, IDESC | (id << 29) | (id << 4),
                                sfa + 4u * (k >> 1), sfb + 4u * L::SF_HALVES * (k >> 1), (s | k) != 0 ? 1u : 0u);
                }
                tc_commit_elect(empty_bar(stage));
                last_bar = empty_bar(stage);
                last_parity = phase;
                committed = true;
                if (++stage == L::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            tc_commit_elect(tfull_bar(acc));
            ++local;
        }
        if (!ok && committed && lane == 0) mg_drain(last_bar, last_parity);
    } else if (warp >= MG_SF_WARP0) {
        // -------------------------------- scales --------------------------------
        // groups of four warps take the slices in turn
        const int r = (threadIdx.x - MG_SF_WARP0 * 32) & 127;
        const int group = (warp - MG_SF_WARP0) >> 2;
        const int kb = static_cast<int>(p.K / 32);
        const uint32_t cell = r * 4u;  // of row r within 512 bytes
        uint8_t *staging = smem + L::STAGES * L::STAGE + 512 + L::LIST_BYTES + group * 2 * L::SF_BYTES;
        static_assert(MG_AHEAD % 2 == 0, "the staging buffers alternate");
        uint2 va[MG_AHEAD], vb[MG_AHEAD][L::SF_HALVES];
        int64_t lt = blockIdx.x;  // next slice to load: its tile, its scale bytes
        int at = group * 8;       // byte offset of that slice in its row
        const uint8_t *pa = nullptr, *pb[L::SF_HALVES];  // the thread's rows; null where there is none
        auto next_tile = [&]() {
            for (; lt < total; lt += gridDim.x) {
                const MgTile ti = tile_at(lt);
                if (ti.rows == 0) continue;
                if (at >= p.slices * 8) {  // past this tile: the slices go on in the next one
                    at -= p.slices * 8;
                    continue;
                }
                pa = r < ti.rows ? p.sf_a + (static_cast<int64_t>(ti.m_start) + r) * kb : nullptr;
#pragma unroll
                for (int h = 0; h < L::SF_HALVES; ++h) {
                    const int n = h * 128 + r;  // row of the stage's B box
                    const bool up = GATE_UP && n >= OUT_N;
                    const int64_t f = ti.n0 + (up ? n - OUT_N : n);
                    pb[h] = n < BN && f < p.N ? (up ? p.sf_b1 : p.sf_b0) + (static_cast<int64_t>(ti.g) * p.N + f) * kb
                                              : nullptr;
                }
                return;
            }
        };
        next_tile();
        auto load = [&](uint2 &a, uint2(&b)[L::SF_HALVES]) {
            a = load_scales<V>(pa, kb, at);
#pragma unroll
            for (int h = 0; h < L::SF_HALVES; ++h) b[h] = load_scales<V>(pb[h], kb, at);
            at += 8 * MG_SF_GROUPS;
            if (at >= p.slices * 8) next_tile();
        };
        int ahead = 0;  // slices in registers
#pragma unroll
        for (int j = 0; j < MG_AHEAD; ++j)
            if (lt < total) {
                load(va[j], vb[j]);
                ++ahead;
            }
        int stage = group;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && ahead > 0) {
#pragma unroll
            for (int j = 0; j < MG_AHEAD; ++j) {
                if (!ok || ahead == 0) continue;
                int free = 1;
                if (lane == 0) free = mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.err) ? 1 : 0;
                free = __shfl_sync(0xffffffffu, free, 0);
                uint8_t *sf = staging + (j & 1) * L::SF_BYTES;
                *reinterpret_cast<uint32_t *>(sf + cell) = va[j].x;
                *reinterpret_cast<uint32_t *>(sf + 512 + cell) = va[j].y;
#pragma unroll
                for (int h = 0; h < L::SF_HALVES; ++h) {
                    *reinterpret_cast<uint32_t *>(sf + 1024 + h * 512 + cell) = vb[j][h].x;
                    *reinterpret_cast<uint32_t *>(sf + 1024 + (L::SF_HALVES + h) * 512 + cell) = vb[j][h].y;
                }
                // every thread of the group has stored; two buffers in turn, so
                // the next slice's stores cannot pass this one's reads.  A warp
                // whose wait gave up comes here too and takes the group along
                ok = mg_group_all(1 + group, free != 0);
                if (!ok) continue;
                // each warp puts all rows' scales into its own lane quarter:
                // lane i, column c holds row 32 c + i
                tc_fence_after();
                const uint32_t col = tmem + ((warp & 3u) << 21) + L::SF_COL0 + stage * L::SF_COLS;
#pragma unroll
                for (int i = 0; i < L::SF_COLS / 8; ++i)
                    tmem_st8(col + 8u * i, quarter_scales(sf + 1024 * i + lane * 4),
                             quarter_scales(sf + 1024 * i + 512 + lane * 4));
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(full_bar(stage));
                stage += MG_SF_GROUPS;
                if (stage >= L::STAGES) {
                    stage -= L::STAGES;
                    phase ^= 1u;
                }
                --ahead;
                if (lt < total) {
                    load(va[j], vb[j]);
                    ++ahead;
                }
            }
        }
    } else {
        // ------------------------------- epilogue -------------------------------
        // two warps to a lane quarter, each with half of the columns
        const int q = warp & 3;  // the lane quarter this warp may read
        constexpr int HALF = (OUT_N / 2 + 31) / 32 * 32;
        const int c0 = ((warp - MG_EPI_WARP0) >> 2) * HALF, c1 = c0 + HALF < OUT_N ? c0 + HALF : OUT_N;
        const int row = q * 32 + lane;
        int local = 0;
        for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
            const MgTile ti = tile_at(t);
            if (ti.rows == 0) continue;
            const int acc = local & 1;
            int ready = 1;
            if (lane == 0)
                ready = mbar_wait_bounded(tfull_bar(acc), static_cast<uint32_t>(local >> 1) & 1u, abort_flag, p.err) ? 1 : 0;
            ready = __shfl_sync(0xffffffffu, ready, 0);
            if (!ready) break;
            tc_fence_after();
            const uint32_t d = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
            const int64_t r = static_cast<int64_t>(ti.m_start) + row;
            const bool valid = row < ti.rows;
            if (q * 32 < ti.rows) {
#pragma unroll 1
                for (int c = c0; c < c1; c += 32) {
                    const int64_t n = ti.n0 + c;
                    if (n >= p.N) break;
                    uint32_t v[32];
                    tmem_ld32(d + c, v);
                    if constexpr (GATE_UP) {
                        uint32_t u[32];
                        tmem_ld32(d + OUT_N + c, u);
                        tmem_ld_wait();
                        float top = 0.0f;
                        bool odd = false;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float g = __uint_as_float(v[i]);
                            const float h = __fdividef(g, 1.0f + __expf(-g)) * __uint_as_float(u[i]);
                            odd |= !(fabsf(h) < INFINITY);
                            top = fmaxf(top, fabsf(h));
                            v[i] = __float_as_uint(h);
                        }
                        const uint32_t s = odd ? 255u : mx4_scale(top);
                        const float inv = odd ? 0.0f : mx4_inverse(s);
                        uint32_t w[4] = {0u, 0u, 0u, 0u};
                        if (!odd) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float eight[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) eight[i] = __uint_as_float(v[8 * j + i]);
                                w[j] = e2m1x8(eight, inv);
                            }
                        }
                        if (valid) {
                            const int64_t o = r * (p.N / 32) + n / 32;
                            *reinterpret_cast<uint4 *>(p.q_h + o * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                            p.sf_h[o] = static_cast<uint8_t>(s);
                        }
                    } else {
                        tmem_ld_wait();
                        TOut *out = static_cast<TOut *>(p.out);
                        if (p.wide && p.N - n >= 32) {
                            if (valid) store_row(out + r * p.N + n, v);
                        } else {
                            const int64_t left = p.N - n;
                            store_block(out + (static_cast<int64_t>(ti.m_start) + q * 32) * p.N + n, p.N, v, ti.rows - q * 32,
                                        left < 32 ? static_cast<int>(left) : 32, lane);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(acc));
            ++local;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

bool rows_map(CUtensorMap *m, const uint8_t *q, int64_t K, int64_t rows, uint32_t box_rows) {
    const uint64_t dims[2] = {static_cast<uint64_t>(K / 2), static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {static_cast<uint64_t>(K / 2)};
    const uint32_t box[2] = {128, box_rows};
    return encode_tma_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q, dims, strides, box, 1);
}

bool weights_map(CUtensorMap *m, const uint8_t *q, int64_t K, int64_t N, int64_t E, uint32_t box_rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(K / 2), static_cast<uint64_t>(N), static_cast<uint64_t>(E)};
    const uint64_t strides[2] = {static_cast<uint64_t>(K / 2), static_cast<uint64_t>(N * (K / 2))};
    const uint32_t box[3] = {128, box_rows, 1};
    return encode_tma_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, q, dims, strides, box, 1);
}

template <typename TOut, bool GATE_UP, int BN, int V>
cudaError_t launch_v(const CUtensorMap *maps, const MgParams &p, cudaStream_t stream) {
    using L = MgLayout<BN>;
    auto kern = mx4_gemm_kernel<TOut, GATE_UP, BN, V>;
    static std::atomic<bool> attr_done[64];  // zero-initialised; several host threads may launch
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev] = true;
    }
    const int64_t tiles = static_cast<int64_t>(p.m_blocks) * p.n_tiles;
    const int64_t grid = tiles < device_sm_count() ? tiles : device_sm_count();
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(MG_THREADS), L::SMEM, stream, maps[0], maps[1],
                      maps[2], p);
}

// the widest scale loads that K and the bases' alignment allow
template <typename TOut, bool GATE_UP, int BN>
cudaError_t launch_n(const CUtensorMap *maps, const MgParams &p, cudaStream_t stream) {
    const uintptr_t bases = reinterpret_cast<uintptr_t>(p.sf_a) | reinterpret_cast<uintptr_t>(p.sf_b0) |
                            reinterpret_cast<uintptr_t>(p.sf_b1);
    if (p.K % 256 == 0 && (bases & 7u) == 0) return launch_v<TOut, GATE_UP, BN, 8>(maps, p, stream);
    if (p.K % 128 == 0 && (bases & 3u) == 0) return launch_v<TOut, GATE_UP, BN, 4>(maps, p, stream);
    return launch_v<TOut, GATE_UP, BN, 1>(maps, p, stream);
}

MgParams params(const uint8_t *sf_a, const MxTables &tab, int64_t m_blocks, int64_t N, int64_t K, int out_n,
                int32_t *err) {
    MgParams p{};
    p.sf_a = sf_a;
    p.tab = tab;
    p.m_blocks = static_cast<int>(m_blocks);
    p.N = N;
    p.K = K;
    p.n_tiles = static_cast<int>((N + out_n - 1) / out_n);
    p.slices = static_cast<int>((K + MG_SLICE - 1) / MG_SLICE);
    p.err = err;
    return p;
}

}  // namespace

cudaError_t launch_grouped_gemm_mx4(const uint8_t *q_a, const uint8_t *sf_a, const uint8_t *q_b, const uint8_t *sf_b,
                                    const MxTables &tab, int64_t m_blocks, int64_t n_rows, int64_t N, int64_t K,
                                    int64_t E, int out_dtype, void *C, int32_t *err, cudaStream_t stream) {
    constexpr int BN = MG_BN;
    CUtensorMap maps[3];
    if (!rows_map(&maps[0], q_a, K, n_rows, MG_BOX_ROWS) || !weights_map(&maps[1], q_b, K, N, E, BN))
        return cudaErrorInvalidValue;
    maps[2] = maps[1];
    MgParams p = params(sf_a, tab, m_blocks, N, K, BN, err);
    p.sf_b0 = sf_b;
    p.sf_b1 = sf_b;
    p.out = C;
    const int64_t row_bytes = N * (out_dtype == kF32 ? 4 : 2);
    p.wide = row_bytes % 32 == 0 && reinterpret_cast<uintptr_t>(C) % 32 == 0;
    if (out_dtype == kF32) return launch_n<float, false, BN>(maps, p, stream);
    if (out_dtype == kBF16) return launch_n<__nv_bfloat16, false, BN>(maps, p, stream);
    return launch_n<__half, false, BN>(maps, p, stream);
}

cudaError_t launch_grouped_gate_up_silu_mx4(const uint8_t *q_a, const uint8_t *sf_a, const uint8_t *q_gate,
                                            const uint8_t *sf_gate, const uint8_t *q_up, const uint8_t *sf_up,
                                            const MxTables &tab, int64_t m_blocks, int64_t n_rows, int64_t d_h,
                                            int64_t d_e, int64_t E, uint8_t *q_h, uint8_t *sf_h, int32_t *err,
                                            cudaStream_t stream) {
    constexpr int BN = MG_BN;
    CUtensorMap maps[3];
    if (!rows_map(&maps[0], q_a, d_h, n_rows, MG_BOX_ROWS) || !weights_map(&maps[1], q_gate, d_h, d_e, E, BN / 2) ||
        !weights_map(&maps[2], q_up, d_h, d_e, E, BN / 2))
        return cudaErrorInvalidValue;
    MgParams p = params(sf_a, tab, m_blocks, d_e, d_h, BN / 2, err);
    p.sf_b0 = sf_gate;
    p.sf_b1 = sf_up;
    p.q_h = q_h;
    p.sf_h = sf_h;
    return launch_n<float, true, BN>(maps, p, stream);
}

}  // namespace moe
