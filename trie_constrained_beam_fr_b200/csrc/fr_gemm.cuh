// fr_gemm.cuh -- the persistent, warp-specialised tcgen05 tile loop that the
// cross-entropy and 8-bit kernels share.
//
// A cluster of two CTAs walks output tiles of 256 x 256 values
// (cta_group::2): each CTA stages 128 rows of A and 128 of B per K stage (128
// bytes of K wide) and holds 128 rows of the accumulator in its tensor memory.
// The pair reads each operand value once where two single CTAs with 128 x 256
// tiles would read B twice: 32 KB instead of 48 KB per stage and CTA, which is
// what bounds the 8-bit products (L2 to shared memory).  Calls of at most 128 rows
// use single CTAs with tiles of 128 x 256 instead: half of a pair's rows would be
// empty.
// In each CTA warp 0 lane 0 copies its part of the stage into a ring with TMA
// (arrivals on the first CTA's barrier); in the first CTA warp 1 lane 0 issues
// the stage's four tcgen05.mma into one of two tensor-memory accumulators;
// warps 4..11 (a tensor-memory lane quarter and half of the columns each, one
// output row per thread; with four warps the exponentials of a log-sum-exp
// epilogue took longer than an 8-bit tile's products) run the kernel's epilogue
// on the finished accumulator while the next tile's products run.  What differs
// between kernels is a policy:
//
//   struct P {
//     static constexpr bool I8;            // 8-bit integers (int32 sums) or bf16 (fp32 sums)
//     static constexpr bool PAIR;          // CTA pairs or single CTAs
//     static constexpr bool STAGED;        // the epilogue stores through shared memory
//     static constexpr int STAGES;         // ring depth
//     static constexpr bool DYNAMIC;       // tiles of unequal length: the pairs take the next one from a counter
//     __device__ void prefetch() const;              // its tensor maps
//     struct Tile { int nk; uint32_t idesc; ... };   // K stages; instruction descriptor
//     struct State { ... };                          // what begin() read after the previous kernel
//     __device__ State begin() const;
//     __device__ bool tile(const State&, uint32_t g, Tile&) const;  // tile g (< 2^31) of the launch; false behind the last
//     __device__ int32_t* counter() const;           // DYNAMIC: zero before the launch; tiles fit an int32
//     __device__ void load(const Tile&, int kb, int rank, uint8_t* a, uint8_t* b, uint32_t bar) const;
//     __device__ uint32_t stage_bytes(const Tile&) const;       // that load() copies into the pair's CTAs (or the one)
//     __device__ bool a_mn(const Tile&) const, b_mn(const Tile&) const;  // operand stored MN-major
//     // the first or second half of one row's columns; gives the accumulator back
//     // as soon as it has been read
//     __device__ void epilogue(const State&, const Tile&, uint32_t taddr, int row_in_tile, int half, const GmStage&,
//                              GmRelease&) const;
//   };
//
// Every wait on a barrier is bounded, and a whole warp's ends alike in all its lanes;
// on expiry the kernel records FR_ERR_DEVICE, stops issuing, drains the copies and
// products already issued, frees its tensor memory and returns.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>

#include "fr_internal.cuh"
#include "fr_tc.cuh"

namespace fr {

constexpr int GM_TILE = 256;         // columns of a tile, and rows of a pair's
constexpr int GM_HALF = 128;         // rows of A that one CTA stages, and of a single CTA's tile: the tensor-memory lanes
constexpr int GM_KB_BYTES = 128;     // K bytes per stage: one 128-byte swizzle span
constexpr int GM_THREADS = 384;      // 12 warps, 8 of them for the epilogue
constexpr int GM_EPI_WARPS = 8;
constexpr int GM_EPI_COLS = 128;     // columns of a tile that one epilogue warp takes
constexpr int GM_OP_BYTES = GM_HALF * GM_KB_BYTES;  // 128 rows of an operand per stage
constexpr int GM_STAGE_BUF = 32 * 128;              // one staged store: 32 rows x 128 bytes
constexpr uint32_t GM_TMEM_COLS = 2 * GM_TILE;      // two accumulators

// Instruction descriptor: accumulator type at bits 4-5 (1 = fp32, 2 = int32),
// A and B types at bits 7-9 and 10-12 (kind::f16: 1 = bf16; kind::i8: 1 =
// signed), "MN-major" flags of A and B at bits 15 and 16, N >> 3 at bits
// 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t gm_idesc(bool i8, bool pair, bool a_mn = false, bool b_mn = false, int n = GM_TILE) {
    return ((i8 ? 2u : 1u) << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)((pair ? GM_TILE : GM_HALF) >> 4) << 24);
}

// Shared-memory descriptor of an MN-major bf16 tile with the 128-byte
// swizzle, stored as blocks of 64 MN elements (128 bytes) x 64 K rows, 8 KB
// each: leading-dimension offset = the next block of 64 MN elements (8,192
// bytes), stride-dimension offset = the next 8 K rows (1,024 bytes).  The
// k-th 16-row slice starts 2,048 * k bytes further.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

#define GM_UMMA(GROUP, KIND)                                                                           \
    asm volatile(                                                                                      \
        "{\n\t.reg .pred p;\n\t"                                                                        \
        "setp.ne.b32 p, %4, 0;\n\t"                                                                    \
        "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),       \
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)                                            \
        : "memory")
template <bool I8, bool PAIR>
__device__ __forceinline__ void gm_umma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    if constexpr (PAIR) {
        if constexpr (I8)
            GM_UMMA("2", "i8");
        else
            GM_UMMA("2", "f16");
    } else {
        if constexpr (I8)
            GM_UMMA("1", "i8");
        else
            GM_UMMA("1", "f16");
    }
}
#undef GM_UMMA

// Arrives on the barrier (of a pair: at this offset in both CTAs) once every
// product issued so far by this thread has completed.
template <bool PAIR>
__device__ __forceinline__ void gm_commit(uint64_t* bar) {
    if constexpr (!PAIR) return tc_umma_commit(bar);
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ uint32_t gm_cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Address of `p`'s counterpart in the pair's first CTA.
__device__ __forceinline__ uint32_t gm_in_first(const void* p) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}

// Arrives on the other CTA's barrier after reads (of tensor memory, of a slot):
// releasing this CTA's writes to the cluster as well would wait for its stores
// on their way (a quarter of a dW tile's time with few rows).
__device__ __forceinline__ void gm_arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Arrives on the other CTA's barrier and publishes this thread's writes.
__device__ __forceinline__ void gm_publish_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void gm_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// 2-D tiled TMA load into this CTA that arrives on the first (or only) CTA's barrier.
template <bool PAIR>
__device__ __forceinline__ void gm_tma_load(const CUtensorMap* map, void* dst, uint32_t bar, int32_t x, int32_t y) {
    if constexpr (!PAIR) {
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
        return;
    }
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// A warp's staging buffer of 32 rows x 128 bytes, written out with TMA
// (128-byte swizzle: 16-byte piece j of row l lies at piece j ^ (l & 7), which
// also spreads the lanes' writes over the banks).
struct GmStage {
    uint8_t* buf;
    __device__ __forceinline__ uint8_t* row(int lane) const {
        // the buffer's last store has read its data
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        return buf + lane * 128;
    }
    __device__ __forceinline__ void put(uint8_t* row, int lane, int piece, uint4 v) const {
        *reinterpret_cast<uint4*>(row + ((piece ^ (lane & 7)) << 4)) = v;
    }
    // Stores the buffer's 32 rows at (x, y), or adds them (fp32), clipped to
    // the map's extent.
    template <bool ADD>
    __device__ __forceinline__ void send(const CUtensorMap* map, int lane, int32_t x, int32_t y) const {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            if (ADD)
                asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                                 reinterpret_cast<uint64_t>(map)),
                             "r"(x), "r"(y), "r"(smem_u32(buf))
                             : "memory");
            else
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                                 reinterpret_cast<uint64_t>(map)),
                             "r"(x), "r"(y), "r"(smem_u32(buf))
                             : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
};

// Bounded wait that also acquires what the other CTA of the pair wrote.
__device__ __forceinline__ bool gm_wait_pair(uint64_t* bar, uint32_t parity, volatile int32_t* abort_flag, int32_t* err,
                                             uint64_t limit_ns) {
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 1000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*abort_flag) return false;
        if (it == 0) t0 = tc_now_ns();
        if ((it & 63u) == 63u && tc_now_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            set_error(err, FR_ERR_DEVICE);
            return false;
        }
    }
}

// Address of `p`'s counterpart in the pair's CTA `rank`.
__device__ __forceinline__ uint32_t gm_in_cta(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

constexpr int GM_SLOTS = 4;  // tiles published ahead of the last reader

// Fetches a tensor map (a kernel argument) ahead of the first copy that goes by it.
__device__ __forceinline__ void gm_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Gives an accumulator back to the products: an epilogue calls it (the whole warp)
// after its last read of it, before it converts and stores what it read.
template <bool PAIR>
struct GmRelease {
    uint64_t* bar;
    uint32_t first_bar;  // the barrier in the pair's first CTA
    int lane;
    bool done;
    __device__ __forceinline__ void operator()() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if constexpr (PAIR)
                gm_arrive_remote(first_bar);
            else
                tc_arrive(bar);
        }
        done = true;
    }
};

template <int STAGES>
struct GmSmem {
    uint64_t full[STAGES];      // used in the first CTA: both CTAs' copies of a stage have landed
    uint64_t empty[STAGES];     // the stage's products are done
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];     // used in the first CTA: both CTAs' epilogues have read the accumulator
    uint64_t mma_done;          // every product the pair issued has completed
    uint64_t tile_full[GM_SLOTS];   // DYNAMIC: the slot's tile has been published
    uint64_t tile_empty[GM_SLOTS];  // used in the first CTA: everyone has read the slot
    int32_t tile_id[GM_SLOTS];
    uint32_t tmem_base;
    int32_t abort_flag;
};

// Tile g of an m_tiles x n_tiles grid, m fastest within groups of 32 tile rows:
// pairs running together share the B tile, and the A tiles of a group (8,192
// rows) stay in L2 while B passes by.
__device__ __forceinline__ void gm_grouped(uint32_t g, uint32_t m_tiles, uint32_t n_tiles, int32_t& m, int32_t& n) {
    const uint32_t group = m_tiles <= 32 ? 0 : g / (32 * n_tiles), m0 = group * 32, rows = min(32u, m_tiles - m0);
    const uint32_t at = g - m0 * n_tiles, q = at / rows;
    m = (int32_t)(m0 + at - q * rows);
    n = (int32_t)q;
}

// What every policy's kernel passes along.
struct GmCtl {
    int32_t* err;
    uint64_t wait_ns;  // limit of the bounded waits
    int32_t starve;    // test setting: no copies are issued, so the waits expire
};

template <class P>
__host__ __device__ constexpr size_t gm_smem_bytes() {
    return 1024 + (size_t)P::STAGES * (P::PAIR ? 2 : 3) * GM_OP_BYTES + (P::STAGED ? GM_EPI_WARPS * GM_STAGE_BUF : 0) + sizeof(GmSmem<P::STAGES>);
}

template <class P>
__device__ __forceinline__ void gm_run(const P& p, const GmCtl& ctl) {
    extern __shared__ uint8_t gm_smem_raw[];
    constexpr int STAGES = P::STAGES;
    constexpr bool PAIR = P::PAIR;
    constexpr int B_BYTES = (PAIR ? 1 : 2) * GM_OP_BYTES;  // 128 or 256 rows of B
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(gm_smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* ringA = base;
    uint8_t* ringB = base + STAGES * GM_OP_BYTES;
    uint8_t* stage = ringB + STAGES * B_BYTES;
    GmSmem<STAGES>* sm = reinterpret_cast<GmSmem<STAGES>*>(stage + (P::STAGED ? GM_EPI_WARPS * GM_STAGE_BUF : 0));
    volatile int32_t* abort_flag = &sm->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? gm_cta_rank() : 0;
    const uint32_t pair = PAIR ? blockIdx.x >> 1 : blockIdx.x, pairs = PAIR ? gridDim.x >> 1 : gridDim.x;  // (or single CTAs)

    if (threadIdx.x == 32) p.prefetch();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            tc_mbar_init(&sm->full[s], 1);
            tc_mbar_init(&sm->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc_mbar_init(&sm->tmem_full[i], 1);
            tc_mbar_init(&sm->tmem_empty[i], (PAIR ? 2 : 1) * GM_EPI_WARPS);
        }
        tc_mbar_init(&sm->mma_done, 1);
        for (int i = 0; i < GM_SLOTS; ++i) {
            tc_mbar_init(&sm->tile_full[i], 1);
            // the epilogue warps, the products, the other producer
            tc_mbar_init(&sm->tile_empty[i], PAIR ? 2 * GM_EPI_WARPS + 2 : GM_EPI_WARPS + 1);
        }
        sm->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem_base)),
                         "r"(GM_TMEM_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem_base)),
                         "r"(GM_TMEM_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) gm_cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    griddep_wait();
    griddep_launch_dependents();
    const typename P::State st = p.begin();

    // The i-th tile of this pair.  Taken in turn, or published by the first
    // CTA's producer: `whole` warps read it together, else one lane does.
    typename P::Tile t;
    const auto next = [&](int i, bool whole) -> bool {
        if (!P::DYNAMIC) return p.tile(st, pair + i * pairs, t);
        const int s = i % GM_SLOTS;
        // only the second CTA's readers need to synchronise with another CTA
        const bool there = rank == 0 ? tc_wait(&sm->tile_full[s], (i / GM_SLOTS) & 1, abort_flag, ctl.err, ctl.wait_ns)
                                     : gm_wait_pair(&sm->tile_full[s], (i / GM_SLOTS) & 1, abort_flag, ctl.err, ctl.wait_ns);
        if (!(whole ? __all_sync(0xffffffffu, there) : there)) return false;
        const int32_t g = *(volatile int32_t*)&sm->tile_id[s];
        if (whole) __syncwarp();
        if (!whole || lane == 0) {
            if (rank == 0)
                tc_arrive(&sm->tile_empty[s]);
            else
                gm_arrive_remote(gm_in_first(&sm->tile_empty[s]));
        }
        return p.tile(st, g, t);
    };
    // The first CTA's producer publishes the tile after the one that it takes
    // itself, so that nobody waits for it, and asks for the one behind that,
    // whose answer comes while this one is copied.  The first two are static.
    uint32_t cur = pair, coming = pair + pairs;
    const auto publish = [&](int i, uint32_t g) -> bool {
        const int s = i % GM_SLOTS;
        if (i >= GM_SLOTS &&
            !gm_wait_pair(&sm->tile_empty[s], ((i / GM_SLOTS) & 1) ^ 1, abort_flag, ctl.err, ctl.wait_ns))
            return false;
        *(volatile int32_t*)&sm->tile_id[s] = (int32_t)g;
        tc_arrive(&sm->tile_full[s]);
        if constexpr (!PAIR) return true;
        asm volatile("st.relaxed.cluster.shared::cluster.s32 [%0], %1;" ::"r"(gm_in_cta(&sm->tile_id[s], 1)), "r"((int32_t)g)
                     : "memory");
        gm_publish_remote(gm_in_cta(&sm->tile_full[s], 1));
        return true;
    };
    const auto take = [&](int i) -> bool {
        if (!P::DYNAMIC) return p.tile(st, pair + i * pairs, t);
        if (rank != 0) return next(i, false);
        if (i == 0 && !publish(0, cur)) return false;
        if (!p.tile(st, cur, t)) return false;
        if (!publish(i + 1, coming)) return false;
        cur = coming;
        coming = (uint32_t)atomicAdd(p.counter(), 1) + 2 * pairs;
        return true;
    };
    if (warp == 0) {
        if (lane == 0 && !ctl.starve) {
            uint32_t it = 0;
            bool ok = true;
            for (int i = 0; ok && take(i); ++i) {
                for (int kb = 0; kb < t.nk; ++kb, ++it) {
                    const uint32_t s = it % STAGES;
                    if (it >= (uint32_t)STAGES &&
                        !tc_wait(&sm->empty[s], ((it / STAGES) & 1u) ^ 1u, abort_flag, ctl.err, ctl.wait_ns)) {
                        ok = false;
                        break;
                    }
                    // the first CTA's barrier counts both CTAs' bytes
                    if (rank == 0) tc_arrive_expect_tx(&sm->full[s], p.stage_bytes(t));
                    p.load(t, kb, (int)rank, ringA + s * GM_OP_BYTES, ringB + s * B_BYTES, PAIR ? gm_in_first(&sm->full[s]) : smem_u32(&sm->full[s]));
                }
            }
            // The last copies land before the CTAs end.  Normally the first
            // CTA's barriers say so for both; after an abort the pair's CTAs
            // may have issued different stages, so each also gives its own
            // copies a millisecond.
            if (rank == 0)
                for (uint32_t j = (it > (uint32_t)STAGES ? it - STAGES : 0u); ok && j < it; ++j)
                    tc_wait_drain(&sm->full[j % STAGES], (j / STAGES) & 1u);
            if (!ok || *abort_flag) {
                const uint64_t t0 = tc_now_ns();
                for (uint32_t k = 0; k < (1u << 20) && tc_now_ns() - t0 < 1000000ull; ++k) __nanosleep(200);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            uint32_t it = 0;
            bool ok = true;
            bool more = next(0, false);
            for (int i = 0; ok && more; ++i) {
                const typename P::Tile now = t;
                const int acc = i & 1;
                if (i >= 2 && !tc_wait(&sm->tmem_empty[acc], ((i >> 1) & 1) ^ 1, abort_flag, ctl.err, ctl.wait_ns)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem + (uint32_t)(acc * GM_TILE);
                const bool amn = p.a_mn(now), bmn = p.b_mn(now);
                // address fields count 16-byte units: the K slices are 32 bytes (K-major) or 2,048 (MN-major) apart
                const uint32_t ia = amn ? 2048 >> 4 : 32 >> 4, ib = bmn ? 2048 >> 4 : 32 >> 4;
                for (int kb = 0; kb < now.nk; ++kb, ++it) {
                    const uint32_t s = it % STAGES;
                    if (!tc_wait(&sm->full[s], (it / STAGES) & 1u, abort_flag, ctl.err, ctl.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ringA + s * GM_OP_BYTES), sb = smem_u32(ringB + s * B_BYTES);
                    const uint64_t da = amn ? smem_desc_mn_sw128(sa) : smem_desc_sw128(sa);
                    const uint64_t db = bmn ? smem_desc_mn_sw128(sb) : smem_desc_sw128(sb);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        gm_umma<P::I8, PAIR>(d_tmem, da + (uint64_t)(kk * ia), db + (uint64_t)(kk * ib), now.idesc,
                                       (kb | kk) != 0 ? 1u : 0u);
                    gm_commit<PAIR>(&sm->empty[s]);  // the stage is free in both CTAs once these products are done
                    // worked out while this tile's products run
                    if (!P::DYNAMIC && kb == 0) more = next(i + 1, false);
                }
                if (P::DYNAMIC || now.nk == 0) more = ok && next(i + 1, false);
                gm_commit<PAIR>(&sm->tmem_full[acc]);  // the accumulators are complete (or, on abort, quiet)
            }
            // the tensor memory is freed only after every product issued here is done
            gm_commit<PAIR>(&sm->mma_done);
        }
        // in both CTAs: the commits' arrivals reach no CTA that has ended
        if (lane == 0) tc_wait_drain(&sm->mma_done, 0);
    } else if (warp >= 4) {
        const int q = warp & 3, half = (warp - 4) >> 2;
        GmStage sg{stage + (warp - 4) * GM_STAGE_BUF};
        const uint32_t empty0 = PAIR ? gm_in_first(&sm->tmem_empty[0]) : 0, empty1 = PAIR ? gm_in_first(&sm->tmem_empty[1]) : 0;
        for (int i = 0; next(i, true); ++i) {
            const int acc = i & 1;
            if (!tc_wait_warp(&sm->tmem_full[acc], (i >> 1) & 1, abort_flag, ctl.err, ctl.wait_ns)) break;
            tc_fence_after();
            GmRelease<PAIR> release{&sm->tmem_empty[acc], acc ? empty1 : empty0, lane, false};
            p.epilogue(st, t, tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * GM_TILE), (int)rank * GM_HALF + q * 32 + lane,
                       half, sg, release);
            if (!release.done) release();
        }
        if (P::STAGED && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) gm_cluster_sync();  // nobody's copies, products or arrivals reach a CTA that has ended
    if (warp == 2) {
        tc_fence_after();
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(GM_TMEM_COLS) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(GM_TMEM_COLS) : "memory");
    }
}

// 64 consecutive columns: two loads, one wait.
__device__ __forceinline__ void gm_ld64(uint32_t taddr, float (&v)[64]) {
    uint32_t r[64];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
            "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
            : "=r"(r[32 * h + 0]), "=r"(r[32 * h + 1]), "=r"(r[32 * h + 2]), "=r"(r[32 * h + 3]), "=r"(r[32 * h + 4]),
              "=r"(r[32 * h + 5]), "=r"(r[32 * h + 6]), "=r"(r[32 * h + 7]), "=r"(r[32 * h + 8]), "=r"(r[32 * h + 9]),
              "=r"(r[32 * h + 10]), "=r"(r[32 * h + 11]), "=r"(r[32 * h + 12]), "=r"(r[32 * h + 13]), "=r"(r[32 * h + 14]),
              "=r"(r[32 * h + 15]), "=r"(r[32 * h + 16]), "=r"(r[32 * h + 17]), "=r"(r[32 * h + 18]), "=r"(r[32 * h + 19]),
              "=r"(r[32 * h + 20]), "=r"(r[32 * h + 21]), "=r"(r[32 * h + 22]), "=r"(r[32 * h + 23]), "=r"(r[32 * h + 24]),
              "=r"(r[32 * h + 25]), "=r"(r[32 * h + 26]), "=r"(r[32 * h + 27]), "=r"(r[32 * h + 28]), "=r"(r[32 * h + 29]),
              "=r"(r[32 * h + 30]), "=r"(r[32 * h + 31])
            : "r"(taddr + 32 * h));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// Maximum that keeps a NaN.
__device__ __forceinline__ float gm_max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Folds 32 values into a running (max m, sum s of e^(x - m)); a NaN stays in
// both.  Maximum and sum go through four chains: with two epilogue warps per
// scheduler one chain's latency shows where a tile's products are short.
__device__ __forceinline__ void gm_lse_fold(const float (&v)[32], float& m, float& s) {
    constexpr float L2E = 1.4426950408889634f;
    float c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        c[k] = gm_max_nan(v[k], v[k + 4]);
#pragma unroll
        for (int i = 8; i < 32; i += 4) c[k] = gm_max_nan(c[k], v[i + k]);
    }
    const float cm = gm_max_nan(gm_max_nan(gm_max_nan(c[0], c[1]), gm_max_nan(c[2], c[3])), m);
    if (cm != m) {
        s = (m == -INFINITY) ? 0.f : s * tc_ex2((m - cm) * L2E);
        m = cm;
    }
    if (m != -INFINITY) {
        const float nm = -m * L2E;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c[k] = tc_ex2(fmaf(v[k], L2E, nm));
#pragma unroll
            for (int i = 4; i < 32; i += 4) c[k] += tc_ex2(fmaf(v[i + k], L2E, nm));
        }
        s += (c[0] + c[1]) + (c[2] + c[3]);
    }
}

// A warp's log-sum-exp of one row's n (max, scaled sum) partials (every lane
// returns it).  Two passes: the terms of the second do not wait for one another.
__device__ __forceinline__ float gm_lse_combine(const float2* p, int32_t n) {
    constexpr float L2E = 1.4426950408889634f;
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, s = 0.f;
#pragma unroll 8
    for (int i = lane; i < n; i += 32) m = gm_max_nan(m, p[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = gm_max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) return m;
#pragma unroll 8
    for (int i = lane; i < n; i += 32) {
        const float2 q = p[i];
        s += q.y * tc_ex2((q.x - m) * L2E);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return m + logf(s);
}

// Rounds 8 values to bf16 (round to nearest even).
__device__ __forceinline__ uint4 gm_pack8(const float* v) {
    uint4 o;
    uint32_t* w = &o.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    return o;
}

// Puts 64 values as bf16, or 32 as fp32, into this lane's row of the buffer.
__device__ __forceinline__ void gm_put(const GmStage& sg, int lane, const float (&v)[64]) {
    uint8_t* row = sg.row(lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) sg.put(row, lane, j, gm_pack8(v + 8 * j));
}
__device__ __forceinline__ void gm_put(const GmStage& sg, int lane, const float (&v)[32]) {
    uint8_t* row = sg.row(lane);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sg.put(row, lane, j, make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                                        __float_as_uint(v[4 * j + 3])));
}

// Writes columns [from, to) of the buffer's first `rows` rows of T to dst with
// plain stores, a row at a time: for rows that TMA cannot address (15 us of 29 on
// 333 x 1,003 fp32 values were a lane's stores to its own row).
template <class T>
__device__ __forceinline__ void gm_write_plain(const GmStage& sg, int lane, T* dst, int64_t ld, int rows, int to,
                                               int from = 0) {
    __syncwarp();
    if (sizeof(T) == 2 && from <= 0 && to >= 64 && ((reinterpret_cast<uintptr_t>(dst) | (uintptr_t)(ld * 2)) & 3) == 0) {
        // whole rows of two-byte values that start on words: 4 bytes a lane (loss and
        // gradients of 13 rows x 41,365 tokens x 1,814 values: 171 us, 202 with 2; rows that
        // start between words were slower so, shifted, than with 2)
#pragma unroll 4
        for (int r = 0; r < rows; ++r)
            *reinterpret_cast<uint32_t*>(dst + r * ld + 2 * lane) =
                *reinterpret_cast<const uint32_t*>(sg.buf + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
        return;
    }
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
#pragma unroll
        for (int c = lane; c < 128 / (int)sizeof(T); c += 32) {
            const int at = c * (int)sizeof(T);
            if (c >= from && c < to)
                dst[r * ld + c] = *reinterpret_cast<const T*>(sg.buf + r * 128 + (((at >> 4) ^ (r & 7)) << 4) + (at & 15));
        }
    }
}

// Tile width (columns): the rounds that `units` pairs or CTAs need times a tile's
// cost, its columns and about 64 columns' worth of start and end.  Fewer columns
// than 256 where that leaves units without a tile, or its last round short.
inline int32_t gm_width(int64_t m_tiles, int64_t columns, int64_t units, int32_t step, int32_t least = 64) {
    int32_t best = GM_TILE;
    int64_t cost = INT64_MAX;
    for (int32_t bn = GM_TILE; bn >= least; bn -= step) {
        const int64_t tiles = m_tiles * ((columns + bn - 1) / bn), c = (tiles + units - 1) / units * (bn + 64);
        if (c < cost) cost = c, best = bn;
    }
    return best;
}

// Sends 64 bf16 columns of the warp's 32 rows to (x, y) of `map`.
__device__ __forceinline__ void gm_stage64(const GmStage& sg, const CUtensorMap* map, int lane, const float (&v)[64], int x, int y) {
    gm_put(sg, lane, v);
    sg.send<false>(map, lane, x, y);
}

// Sends (or adds) 32 fp32 columns of the warp's 32 rows to (x, y) of `map`.
template <bool ADD>
__device__ __forceinline__ void gm_stage32(const GmStage& sg, const CUtensorMap* map, int lane, const float (&v)[32], int x, int y) {
    gm_put(sg, lane, v);
    sg.send<ADD>(map, lane, x, y);
}

// Rows of a single CTA's A copies when there are `rows` of them.  The products'
// other rows are whatever the stage held and reach nothing.  Copies of 128 rows would
// have most of them filled in, which takes longer than copying (4 rows x 129,820
// tokens x 1,212 values: 77 us for the loss, 63 without).
inline int32_t gm_a_rows(int32_t rows) { return std::min((rows + 7) / 8 * 8, GM_HALF); }

// 2-D row-major tensor map: `rows` x `cols` elements of `esize` bytes (1: 8-bit
// integers, 2: bf16, 4: fp32), row pitch `pitch` bytes, box box_rows x 128
// bytes, 128-byte swizzle, zero fill out of bounds.
inline bool gm_encode(CUtensorMap* map, int esize, const void* ptr, int64_t rows, int64_t cols, int64_t pitch,
                      uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / esize), box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType type = esize == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : esize == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    return fn(map, type, 2, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Columns of a row of `cols` elements that whole 128-byte TMA stores may write:
// a store that the map clips fills up its last 16 bytes (with zeros, measured),
// so a row that ends inside them keeps its last group for plain stores.
inline int32_t gm_staged_columns(int32_t cols, int esize) {
    return (int64_t)cols * esize % 16 == 0 ? cols : cols / (128 / esize) * (128 / esize);
}

// kernel<<<grid, block, smem, s>>>(args...) with programmatic stream
// serialisation: the kernel waits with griddep_wait before it touches memory.
template <class... KArgs, class... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), int64_t grid, int block, size_t smem, cudaStream_t s,
                              Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

// Raises a gm_run kernel's shared-memory limit on the current device.
template <class P>
inline cudaError_t gm_setup(void (*kernel)(P, GmCtl)) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)gm_smem_bytes<P>());
}

// A gm_run kernel over `tiles` tiles: CTA pairs (clusters of two) or single CTAs,
// at most one CTA per SM.
template <class P>
inline cudaError_t gm_launch(void (*kernel)(P, GmCtl), int64_t tiles, int32_t sms, cudaStream_t s, const P& p,
                             const GmCtl& ctl) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)(P::PAIR ? 2 * std::min<int64_t>(tiles, sms / 2) : std::min<int64_t>(tiles, sms)));
    cfg.blockDim = dim3(GM_THREADS);
    cfg.dynamicSmemBytes = gm_smem_bytes<P>();
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = P::PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, ctl);
}

}  // namespace fr
