// fr_gemm.cuh -- the persistent, warp-specialised tcgen05 tile loop that the
// cross-entropy and 8-bit kernels share.
//
// A kernel walks output tiles of 128 x BN values: warp 0 lane 0 copies each
// K stage's operand tiles (128 bytes of K wide) into a ring with TMA, warp 1
// lane 0 issues the stage's four tcgen05.mma into one of two tensor-memory
// accumulators, warps 4..7 (one tensor-memory lane quarter each, one output
// row per thread) run the kernel's epilogue on the finished accumulator while
// the next tile's products run.  What differs between kernels is a policy:
//
//   struct P {
//     static constexpr bool I8;            // 8-bit integers (int32 sums) or bf16 (fp32 sums)
//     static constexpr int BN, STAGES;     // tile columns, ring depth
//     struct Tile { int nk; uint32_t idesc; ... };   // K stages; instruction descriptor
//     struct State { ... };                          // what begin() read after the previous kernel
//     __device__ State begin() const;
//     __device__ bool tile(const State&, int i, Tile&) const;      // the i-th tile of this CTA
//     __device__ void load(const Tile&, int kb, uint8_t* a, uint8_t* b, uint64_t* bar) const;
//     __device__ bool a_mn(const Tile&) const, b_mn(const Tile&) const;  // operand stored MN-major
//     __device__ void epilogue(const State&, const Tile&, uint32_t taddr, int row_in_tile) const;
//   };
//
// Every wait is bounded; on expiry the kernel records FR_ERR_DEVICE, stops
// issuing, drains the copies and products already issued, frees its tensor
// memory and returns.
#pragma once

#include <cuda_bf16.h>

#include "fr_internal.cuh"
#include "fr_tc.cuh"

namespace fr {

constexpr int GM_BM = 128;           // rows per tile: the tensor-memory lanes
constexpr int GM_KB_BYTES = 128;     // K bytes per stage: one 128-byte swizzle span
constexpr int GM_THREADS = 256;      // 8 warps
constexpr int GM_A_BYTES = GM_BM * GM_KB_BYTES;

// Instruction descriptor: accumulator type at bits 4-5 (1 = fp32, 2 = int32),
// A and B types at bits 7-9 and 10-12 (kind::f16: 1 = bf16; kind::i8: 1 =
// signed), "MN-major" flags of A and B at bits 15 and 16, N >> 3 at bits
// 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t gm_idesc(bool i8, int n, bool a_mn = false, bool b_mn = false) {
    return ((i8 ? 2u : 1u) << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(GM_BM >> 4) << 24);
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

template <bool I8>
__device__ __forceinline__ void gm_umma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    if (I8)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

template <int STAGES>
struct GmSmem {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];
    uint64_t mma_done;  // every product this CTA issued has completed
    uint32_t tmem_base;
    int32_t abort_flag;
};

// What every policy's kernel passes along.
struct GmCtl {
    int32_t* err;
    uint64_t wait_ns;  // limit of the bounded waits
    int32_t starve;    // test setting: no copies are issued, so the waits expire
};

template <class P>
__host__ __device__ constexpr size_t gm_smem_bytes() {
    return 1024 + (size_t)P::STAGES * (GM_A_BYTES + P::BN * GM_KB_BYTES) + sizeof(GmSmem<P::STAGES>);
}

// Tensor-memory columns of the two accumulators (a power of two, at least 32).
template <class P>
__host__ __device__ constexpr uint32_t gm_tmem_cols() {
    uint32_t c = 32;
    while (c < 2u * P::BN) c *= 2;
    return c;
}

template <class P>
__device__ __forceinline__ void gm_run(const P& p, const GmCtl& ctl) {
    extern __shared__ uint8_t gm_smem_raw[];
    constexpr int STAGES = P::STAGES, BN = P::BN, B_BYTES = BN * GM_KB_BYTES;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(gm_smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* ringA = base;
    uint8_t* ringB = base + STAGES * GM_A_BYTES;
    GmSmem<STAGES>* sm = reinterpret_cast<GmSmem<STAGES>*>(ringB + STAGES * B_BYTES);
    volatile int32_t* abort_flag = &sm->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            tc_mbar_init(&sm->full[s], 1);
            tc_mbar_init(&sm->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc_mbar_init(&sm->tmem_full[i], 1);
            tc_mbar_init(&sm->tmem_empty[i], 4 * 32);
        }
        tc_mbar_init(&sm->mma_done, 1);
        sm->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem_base)),
                     "r"(gm_tmem_cols<P>())
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    griddep_wait();
    griddep_launch_dependents();
    const typename P::State st = p.begin();

    typename P::Tile t;
    if (warp == 0) {
        if (lane == 0 && !ctl.starve) {
            uint32_t it = 0;
            bool ok = true;
            for (int i = 0; ok && p.tile(st, i, t); ++i) {
                for (int kb = 0; kb < t.nk; ++kb, ++it) {
                    const uint32_t s = it % STAGES;
                    if (it >= (uint32_t)STAGES &&
                        !tc_wait(&sm->empty[s], ((it / STAGES) & 1u) ^ 1u, abort_flag, ctl.err, ctl.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_arrive_expect_tx(&sm->full[s], (uint32_t)(GM_A_BYTES + B_BYTES));
                    p.load(t, kb, ringA + s * GM_A_BYTES, ringB + s * B_BYTES, &sm->full[s]);
                }
            }
            // the last copies land before the CTA ends, whoever waits for them
            for (uint32_t j = (it > (uint32_t)STAGES ? it - STAGES : 0u); j < it; ++j)
                tc_wait_drain(&sm->full[j % STAGES], (j / STAGES) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int i = 0; ok && p.tile(st, i, t); ++i) {
                const int acc = i & 1;
                if (i >= 2 && !tc_wait(&sm->tmem_empty[acc], ((i >> 1) & 1) ^ 1, abort_flag, ctl.err, ctl.wait_ns)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem + (uint32_t)(acc * BN);
                const bool amn = p.a_mn(t), bmn = p.b_mn(t);
                for (int kb = 0; kb < t.nk; ++kb, ++it) {
                    const uint32_t s = it % STAGES;
                    if (!tc_wait(&sm->full[s], (it / STAGES) & 1u, abort_flag, ctl.err, ctl.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ringA + s * GM_A_BYTES), sb = smem_u32(ringB + s * B_BYTES);
                    const uint64_t da = amn ? smem_desc_mn_sw128(sa) : smem_desc_sw128(sa);
                    const uint64_t db = bmn ? smem_desc_mn_sw128(sb) : smem_desc_sw128(sb);
                    // address fields count 16-byte units: the K slices are 32 bytes (K-major) or 2,048 (MN-major) apart
                    const uint32_t ia = amn ? 2048 >> 4 : 32 >> 4, ib = bmn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        gm_umma<P::I8>(d_tmem, da + (uint64_t)(kk * ia), db + (uint64_t)(kk * ib), t.idesc,
                                       (kb | kk) != 0 ? 1u : 0u);
                    tc_umma_commit(&sm->empty[s]);  // the stage is free once these products are done
                }
                tc_umma_commit(&sm->tmem_full[acc]);  // the accumulator is complete (or, on abort, quiet)
            }
            // the tensor memory is freed only after every product issued here is done
            tc_umma_commit(&sm->mma_done);
            tc_wait_drain(&sm->mma_done, 0);
        }
    } else if (warp >= 4) {
        const int q = warp & 3;
        for (int i = 0; p.tile(st, i, t); ++i) {
            const int acc = i & 1;
            if (!tc_wait(&sm->tmem_full[acc], (i >> 1) & 1, abort_flag, ctl.err, ctl.wait_ns)) break;
            tc_fence_after();
            p.epilogue(st, t, tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN), q * 32 + lane);
            tc_fence_before();
            tc_arrive(&sm->tmem_empty[acc]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(gm_tmem_cols<P>()) : "memory");
    }
}

// 32 consecutive accumulator words of this thread's lane.
__device__ __forceinline__ void gm_ld32_i32(uint32_t taddr, int32_t (&v)[32]) {
    float f[32];
    tc_tmem_ld32(taddr, f);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __float_as_int(f[i]);
}

// Maximum that keeps a NaN.
__device__ __forceinline__ float gm_max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Folds 32 values into a running (max m, sum s of e^(x - m)); a NaN stays in
// both.
__device__ __forceinline__ void gm_lse_fold(const float (&v)[32], float& m, float& s) {
    constexpr float L2E = 1.4426950408889634f;
    float cm = v[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) cm = gm_max_nan(cm, v[i]);
    cm = gm_max_nan(cm, m);
    if (cm != m) {
        s = (m == -INFINITY) ? 0.f : s * tc_ex2((m - cm) * L2E);
        m = cm;
    }
    if (m != -INFINITY) {
        const float nm = -m * L2E;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += tc_ex2(fmaf(v[i], L2E, nm));
    }
}

// A warp's log-sum-exp of one row's n (max, scaled sum) partials, combined in
// lane order (every lane returns it).
__device__ __forceinline__ float gm_lse_combine(const float2* p, int32_t n) {
    constexpr float L2E = 1.4426950408889634f;
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, s = 0.f;
    for (int i = lane; i < n; i += 32) {
        const float2 q = p[i];
        const float M = gm_max_nan(m, q.x);
        if (M != -INFINITY) {
            s = (m == M ? s : s * tc_ex2((m - M) * L2E)) + (q.x == M ? q.y : q.y * tc_ex2((q.x - M) * L2E));
            m = M;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        const float M = gm_max_nan(m, m2);
        if (M != -INFINITY) {
            s = (m == M ? s : s * tc_ex2((m - M) * L2E)) + (m2 == M ? s2 : s2 * tc_ex2((m2 - M) * L2E));
            m = M;
        }
    }
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

// Stores the first n (<= 32) of 32 values of one row; `vec`: dst and the row
// pitch are multiples of 16 bytes, so whole 16-byte groups go out at once.
__device__ __forceinline__ void gm_store32(__nv_bfloat16* dst, const float (&v)[32], int n, bool vec) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            if (i + 8 <= n) {
                *reinterpret_cast<uint4*>(dst + i) = gm_pack8(v + i);
            } else {
#pragma unroll
                for (int j = i; j < i + 8; ++j)
                    if (j < n) dst[j] = __float2bfloat16_rn(v[j]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) dst[i] = __float2bfloat16_rn(v[i]);
    }
}

__device__ __forceinline__ void gm_store32(float* dst, const float (&v)[32], int n, bool vec) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            if (i + 4 <= n) {
                *reinterpret_cast<float4*>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            } else {
#pragma unroll
                for (int j = i; j < i + 4; ++j)
                    if (j < n) dst[j] = v[j];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) dst[i] = v[i];
    }
}

// 2-D row-major tensor map: `rows` x `cols` elements of `esize` bytes, row
// pitch `pitch` bytes, box box_rows x 128 bytes, 128-byte swizzle, zero fill
// out of bounds.
inline bool gm_encode(CUtensorMap* map, bool i8, const void* ptr, int64_t rows, int64_t cols, int64_t pitch,
                      uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)(i8 ? 128 : 64), box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

}  // namespace fr
