// fr_embed.cu -- token embedding with scaling, and its gradient by sorted
// tokens.
//
//   out_i = scale * T[tok_i]          (zeros for token -1)
//   dT_v (+)= scale * sum_{i: tok_i = v} g_i
//
// Both only move memory: the lookup reads and writes n rows, the gradient
// reads n rows and writes V (or the touched ones).
//
//   k_em_lookup   a warp per row, 8 elements a lane at a time.
//   k_em_hist / k_em_scatter   stable radix sort of the tokens with their
//                 positions, 9 bits a pass (two passes up to 2^18 tokens).
//   k_em_sum      the sorted positions in chunks of EM_CHUNK: a CTA adds the
//                 rows of a chunk, a column group per thread, and writes the
//                 finished tokens; a token that reaches over a chunk's edge
//                 leaves fp32 partials.
//   k_em_join     adds such a token's partials in chunk order.
//
// The sort is stable and the partials are joined in order, so a sum's order
// depends on the tokens alone: no floating-point atomics.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "fr.h"
#include "fr_gemm.cuh"
#include "fr_handles.h"
#include "fr_internal.cuh"

namespace fr {
namespace {

constexpr int EM_THREADS = 256;
constexpr int EM_WARPS = EM_THREADS / 32;
constexpr int EM_TILE = 2048;       // tokens per CTA of the sort
constexpr int EM_BITS = 9;          // most digit bits of a sort pass
constexpr int EM_CHUNK = 32;        // sorted positions per CTA of the sum

// VEC consecutive elements (1, or 8 that start on 16 bytes) as fp32, and back.
template <int VEC>
__device__ __forceinline__ void em_load(const float* p, float (&v)[VEC]) {
    if (VEC == 8) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x, v[1 % VEC] = a.y, v[2 % VEC] = a.z, v[3 % VEC] = a.w;
        v[4 % VEC] = b.x, v[5 % VEC] = b.y, v[6 % VEC] = b.z, v[7 % VEC] = b.w;
    } else {
        v[0] = *p;
    }
}
template <int VEC>
__device__ __forceinline__ void em_load(const __nv_bfloat16* p, float (&v)[VEC]) {
    if (VEC == 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[(2 * i) % VEC] = __uint_as_float(w[i] << 16);
            v[(2 * i + 1) % VEC] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        v[0] = __bfloat162float(*p);
    }
}
template <int VEC>
__device__ __forceinline__ void em_store(float* p, const float (&v)[VEC]) {
    if (VEC == 8) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1 % VEC], v[2 % VEC], v[3 % VEC]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4 % VEC], v[5 % VEC], v[6 % VEC], v[7 % VEC]);
    } else {
        *p = v[0];
    }
}
template <int VEC>
__device__ __forceinline__ void em_store(__nv_bfloat16* p, const float (&v)[VEC]) {
    if (VEC == 8)
        *reinterpret_cast<uint4*>(p) = gm_pack8(v);
    else
        *p = __float2bfloat16_rn(v[0]);
}

// The token as a sort key: V for -1 and for a value that is no token (which
// is recorded).
__device__ __forceinline__ uint32_t em_key(int32_t t, int32_t V, int32_t* err) {
    if (t >= 0 && t < V) return (uint32_t)t;
    if (t != -1) set_error(err, FR_ERR_CODE_RANGE);
    return (uint32_t)V;
}

template <class TI, class TO, int VEC>
__global__ void __launch_bounds__(EM_THREADS) k_em_lookup(const TI* __restrict__ table, int64_t ldt, int32_t V, int32_t d,
                                                          const int32_t* __restrict__ tokens, int32_t n, float scale,
                                                          TO* __restrict__ out, int64_t ldo, int32_t* __restrict__ err) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * EM_WARPS + (threadIdx.x >> 5);
    if (i >= n) return;
    const uint32_t t = em_key(tokens[i], V, err);
    const bool live = t < (uint32_t)V;
    const TI* src = table + (int64_t)(live ? t : 0) * ldt;
    TO* dst = out + i * ldo;
#pragma unroll 4
    for (int32_t j = lane * VEC; j < d; j += 32 * VEC) {
        float v[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = 0.f;
        if (live) em_load<VEC>(src + j, v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = live ? v[k] * scale : 0.f;
        em_store<VEC>(dst + j, v);
    }
}

// Digit counts of one tile: counts[digit * tiles + tile].  The first pass
// reads the tokens themselves (kin null).
__global__ void __launch_bounds__(EM_THREADS) k_em_hist(const int32_t* __restrict__ tokens,
                                                        const uint32_t* __restrict__ kin, int32_t n, int32_t V,
                                                        int32_t shift, int32_t bits, int32_t tiles,
                                                        int32_t* __restrict__ counts, int32_t* __restrict__ err) {
    __shared__ int32_t h[1 << EM_BITS];
    griddep_wait();
    griddep_launch_dependents();
    const int bins = 1 << bits;
    for (int b = threadIdx.x; b < bins; b += EM_THREADS) h[b] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * EM_TILE;
#pragma unroll
    for (int k = 0; k < EM_TILE; k += EM_THREADS) {
        const int64_t i = i0 + k + threadIdx.x;
        if (i < n) {
            const uint32_t key = kin ? kin[i] : em_key(tokens[i], V, err);
            atomicAdd(&h[(key >> shift) & (bins - 1)], 1);
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += EM_THREADS) counts[(int64_t)b * tiles + blockIdx.x] = h[b];
}

// Stable scatter of one tile: each warp takes 256 consecutive keys, 32 at a
// time, and ranks equal digits by lane order; the warps' digit counts are
// scanned in warp order.  offs: exclusive prefix of the counts.
__global__ void __launch_bounds__(EM_THREADS) k_em_scatter(const int32_t* __restrict__ tokens,
                                                           const uint32_t* __restrict__ kin,
                                                           const int32_t* __restrict__ pin, int32_t n, int32_t V,
                                                           int32_t shift, int32_t bits, int32_t tiles,
                                                           const int32_t* __restrict__ offs, uint32_t* __restrict__ kout,
                                                           int32_t* __restrict__ pout, int32_t* __restrict__ err) {
    constexpr int PER = EM_TILE / EM_THREADS;  // keys per lane
    __shared__ int32_t cnt[EM_WARPS][1 << EM_BITS];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << bits;
    for (int b = threadIdx.x; b < EM_WARPS * bins; b += EM_THREADS) cnt[b / bins][b % bins] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * EM_TILE + warp * (PER * 32);
    uint32_t key[PER];
    int32_t pos[PER], rank[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int64_t i = i0 + k * 32 + lane;
        key[k] = i < n ? (kin ? kin[i] : em_key(tokens[i], V, err)) : 0u;
        pos[k] = i < n ? (pin ? pin[i] : (int32_t)i) : 0;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const bool live = i0 + k * 32 + lane < n;
        const uint32_t dig = live ? (key[k] >> shift) & (bins - 1) : 0xFFFFFFFFu;
        const uint32_t same = __match_any_sync(0xffffffffu, dig);
        const int before = __popc(same & ((1u << lane) - 1u));
        int32_t base = 0;
        if (live) base = cnt[warp][dig];
        __syncwarp();
        if (live && before == 0) cnt[warp][dig] = base + __popc(same);
        __syncwarp();
        rank[k] = base + before;
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += EM_THREADS) {
        int32_t at = offs[(int64_t)b * tiles + blockIdx.x];
#pragma unroll
        for (int w = 0; w < EM_WARPS; ++w) {
            const int32_t c = cnt[w][b];
            cnt[w][b] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (i0 + k * 32 + lane < n) {
            const int32_t o = cnt[warp][(key[k] >> shift) & (bins - 1)] + rank[k];
            kout[o] = key[k];
            pout[o] = pos[k];
        }
    }
}

// One finished column group of a table row.
template <class TT, int VEC>
__device__ __forceinline__ void em_write(TT* dst, const float (&sum)[VEC], float scale, bool accumulate) {
    float v[VEC];
    if (accumulate) em_load<VEC>(dst, v);
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = accumulate ? fmaf(scale, sum[k], v[k]) : scale * sum[k];
    em_store<VEC>(dst, v);
}

// Chunk c holds the sorted positions [c * EM_CHUNK, ...).  Its partials:
// part[2c] the run that began in an earlier chunk, part[2c + 1] the run that
// begins here and goes on.
template <class TG, class TT, int VEC>
__global__ void __launch_bounds__(EM_THREADS)
    k_em_sum(const TG* __restrict__ grad, int64_t ldg, int32_t d, const uint32_t* __restrict__ keys,
             const int32_t* __restrict__ order, int32_t n, int32_t V, float scale, TT* __restrict__ table, int64_t ldt,
             int32_t accumulate, float* __restrict__ part, int64_t pitch) {
    __shared__ uint32_t key_s[EM_CHUNK + 2];  // the chunk's keys between its neighbours'
    __shared__ int32_t ord_s[EM_CHUNK];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t i0 = (int64_t)blockIdx.x * EM_CHUNK;
    for (int k = threadIdx.x; k < EM_CHUNK + 2; k += EM_THREADS) {
        const int64_t i = i0 + k - 1;
        key_s[k] = i >= 0 && i < n ? keys[i] : 0xFFFFFFFFu;
        if (k >= 1 && k <= EM_CHUNK) ord_s[k - 1] = i < n ? order[i] : 0;
    }
    __syncthreads();
    const int m = (int)min((int64_t)EM_CHUNK, n - i0);
    for (int32_t j = threadIdx.x * VEC; j < d; j += EM_THREADS * VEC) {
        float sum[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) sum[q] = 0.f;
        bool from_before = key_s[0] == key_s[1];
        for (int k0 = 0; k0 < m; k0 += 4) {
            float v[4][VEC];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (k0 + u < m && key_s[k0 + u + 1] < (uint32_t)V)
                    em_load<VEC>(grad + (int64_t)ord_s[k0 + u] * ldg + j, v[u]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = k0 + u;
                if (k >= m) break;
                const uint32_t key = key_s[k + 1];
                if (key >= (uint32_t)V) break;  // tokens that do not count are sorted last
#pragma unroll
                for (int q = 0; q < VEC; ++q) sum[q] += v[u][q];
                const bool ends = key_s[k + 2] != key;
                if (ends || k == m - 1) {
                    if (ends && !from_before) {
                        em_write<TT, VEC>(table + (int64_t)key * ldt + j, sum, scale, accumulate != 0);
                    } else {
                        float* o = part + (2 * (int64_t)blockIdx.x + (from_before ? 0 : 1)) * pitch + j;
                        em_store<VEC>(o, sum);
                    }
                    from_before = false;
#pragma unroll
                    for (int q = 0; q < VEC; ++q) sum[q] = 0.f;
                }
            }
        }
    }
}

// The run that begins in chunk c and goes on: its partials in chunk order.
template <class TT, int VEC>
__global__ void __launch_bounds__(EM_THREADS)
    k_em_join(const uint32_t* __restrict__ keys, int32_t n, int32_t V, int32_t d, float scale, TT* __restrict__ table,
              int64_t ldt, int32_t accumulate, const float* __restrict__ part, int64_t pitch) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t c = blockIdx.x, last = c * EM_CHUNK + EM_CHUNK - 1;
    if (last + 1 >= n) return;
    const uint32_t key = keys[last];
    if (key >= (uint32_t)V || keys[last + 1] != key) return;
    if (c > 0 && keys[c * EM_CHUNK - 1] == key) return;  // begins in an earlier chunk
    // the last chunk that the run reaches
    int64_t e = c + 1;
    while ((e + 1) * EM_CHUNK < n && keys[(e + 1) * EM_CHUNK] == key) ++e;
    for (int32_t j = threadIdx.x * VEC; j < d; j += EM_THREADS * VEC) {
        float sum[VEC];
        em_load<VEC>(part + (2 * c + 1) * pitch + j, sum);
        for (int64_t k = c + 1; k <= e; ++k) {
            float v[VEC];
            em_load<VEC>(part + 2 * k * pitch + j, v);
#pragma unroll
            for (int q = 0; q < VEC; ++q) sum[q] += v[q];
        }
        em_write<TT, VEC>(table + (int64_t)key * ldt + j, sum, scale, accumulate != 0);
    }
}

}  // namespace
}  // namespace fr

struct fr_embed {
    int32_t V = 0, d = 0, max_tokens = 0, device = 0;
    uint32_t* keys[2] = {};
    int32_t* pos[2] = {};
    int32_t* counts = nullptr;
    int32_t* temp = nullptr;
    float* part = nullptr;  // [2 * chunks, pitch]
    int64_t pitch = 0;
    int32_t* err = nullptr;
    cudaStream_t last_stream = nullptr;
};

namespace {

int64_t em_ceil(int64_t x, int64_t q) { return (x + q - 1) / q; }

// Whether rows of 8 elements of `size` bytes start on 16 bytes everywhere.
bool em_vec(const void* p, int64_t ld, int size, int32_t d) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * size) % 16 == 0 && d % 8 == 0;
}

bool em_bad(const void* p, fr_dtype t, int64_t ld, int32_t d) {
    return !p || (t != FR_F32 && t != FR_BF16) || ld < d || (reinterpret_cast<uintptr_t>(p) & (t == FR_F32 ? 3u : 1u));
}

bool em_on_device(const fr_embed* h) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == h->device;
}

void em_free(fr_embed* h) {
    cudaFree(h->keys[0]);
    cudaFree(h->counts);
    cudaFree(h->part);
    cudaFree(h->err);
    delete h;
}

template <class TI, class TO>
cudaError_t em_lookup(fr_embed* h, const void* table, int64_t ldt, const int32_t* tokens, int32_t n, float scale, void* out,
                      int64_t ldo, cudaStream_t s) {
    const bool vec = em_vec(table, ldt, sizeof(TI), h->d) && em_vec(out, ldo, sizeof(TO), h->d);
    auto k = vec ? fr::k_em_lookup<TI, TO, 8> : fr::k_em_lookup<TI, TO, 1>;
    return fr::launch_pdl(k, em_ceil(n, fr::EM_WARPS), fr::EM_THREADS, 0, s, (const TI*)table, ldt, h->V, h->d, tokens, n,
                          scale, (TO*)out, ldo, h->err);
}

template <class TG, class TT>
cudaError_t em_sum(fr_embed* h, const void* grad, int64_t ldg, const uint32_t* keys, const int32_t* order, int32_t n,
                   float scale, void* table, int64_t ldt, int32_t accumulate, cudaStream_t s) {
    const bool vec = em_vec(grad, ldg, sizeof(TG), h->d) && em_vec(table, ldt, sizeof(TT), h->d);
    const int64_t chunks = em_ceil(n, fr::EM_CHUNK);
    auto ks = vec ? fr::k_em_sum<TG, TT, 8> : fr::k_em_sum<TG, TT, 1>;
    cudaError_t e = fr::launch_pdl(ks, chunks, fr::EM_THREADS, 0, s, (const TG*)grad, ldg, h->d, keys, order, n, h->V, scale,
                                   (TT*)table, ldt, accumulate, h->part, h->pitch);
    if (e != cudaSuccess) return e;
    auto kj = vec ? fr::k_em_join<TT, 8> : fr::k_em_join<TT, 1>;
    return fr::launch_pdl(kj, chunks, fr::EM_THREADS, 0, s, keys, n, h->V, h->d, scale, (TT*)table, ldt, accumulate,
                          (const float*)h->part, h->pitch);
}

}  // namespace

extern "C" fr_status fr_embed_init(int32_t V, int32_t d, int32_t max_tokens, fr_embed** out) {
    if (!out) return FR_ERR_INVALID_ARG;
    *out = nullptr;
    if (V < 1 || d < 1 || max_tokens < 1 || max_tokens >= (1 << 30)) return FR_ERR_INVALID_ARG;
    fr_embed* h = new (std::nothrow) fr_embed();
    if (!h) return FR_ERR_OOM;
    h->V = V;
    h->d = d;
    h->max_tokens = max_tokens;
    h->pitch = em_ceil(d, 8) * 8;
    if (cudaGetDevice(&h->device) != cudaSuccess) {
        (void)cudaGetLastError();
        delete h;
        return FR_ERR_CUDA;
    }
    const int64_t n = max_tokens, cells = (int64_t)em_ceil(n, fr::EM_TILE) << fr::EM_BITS;
    cudaError_t e = cudaMalloc(&h->keys[0], n * 16);
    if (e == cudaSuccess) e = cudaMalloc(&h->counts, (cells + fr::scan_temp_elems(cells)) * 4);
    if (e == cudaSuccess) e = cudaMalloc(&h->part, (size_t)em_ceil(n, fr::EM_CHUNK) * 2 * h->pitch * 4);
    if (e == cudaSuccess) e = cudaMalloc(&h->err, sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMemset(h->err, 0, sizeof(int32_t));
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        em_free(h);
        return e == cudaErrorMemoryAllocation ? FR_ERR_OOM : FR_ERR_CUDA;
    }
    h->keys[1] = h->keys[0] + n;
    h->pos[0] = reinterpret_cast<int32_t*>(h->keys[1] + n);
    h->pos[1] = h->pos[0] + n;
    h->temp = h->counts + cells;
    *out = h;
    return FR_OK;
}

extern "C" fr_status fr_embed_lookup(fr_embed* h, const void* table_dev, int64_t ldt, fr_dtype table_dtype,
                                     const int32_t* tokens_dev, int32_t n, float scale, void* out_dev, int64_t ldo,
                                     fr_dtype out_dtype, fr_stream stream) {
    if (!h || em_bad(table_dev, table_dtype, ldt, h->d) || em_bad(out_dev, out_dtype, ldo, h->d) || !tokens_dev ||
        (reinterpret_cast<uintptr_t>(tokens_dev) & 3u) || n < 0 || n > h->max_tokens || !em_on_device(h))
        return FR_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    h->last_stream = s;
    if (n == 0) return FR_OK;
    cudaError_t e;
    if (table_dtype == FR_F32)
        e = out_dtype == FR_F32 ? em_lookup<float, float>(h, table_dev, ldt, tokens_dev, n, scale, out_dev, ldo, s)
                                : em_lookup<float, __nv_bfloat16>(h, table_dev, ldt, tokens_dev, n, scale, out_dev, ldo, s);
    else
        e = out_dtype == FR_F32
                ? em_lookup<__nv_bfloat16, float>(h, table_dev, ldt, tokens_dev, n, scale, out_dev, ldo, s)
                : em_lookup<__nv_bfloat16, __nv_bfloat16>(h, table_dev, ldt, tokens_dev, n, scale, out_dev, ldo, s);
    FR_CUDA_TRY(e);
    return FR_OK;
}

extern "C" fr_status fr_embed_grad(fr_embed* h, const void* grad_out_dev, int64_t ldg, fr_dtype grad_dtype,
                                   const int32_t* tokens_dev, int32_t n, float scale, void* grad_table_dev, int64_t ldt,
                                   fr_dtype table_dtype, int32_t accumulate, fr_stream stream) {
    if (!h || em_bad(grad_out_dev, grad_dtype, ldg, h->d) || em_bad(grad_table_dev, table_dtype, ldt, h->d) ||
        !tokens_dev || (reinterpret_cast<uintptr_t>(tokens_dev) & 3u) || n < 0 || n > h->max_tokens ||
        (accumulate != 0 && accumulate != 1) || !em_on_device(h))
        return FR_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    h->last_stream = s;
    const size_t tsize = table_dtype == FR_F32 ? 4 : 2;
    if (!accumulate)
        FR_CUDA_TRY(cudaMemset2DAsync(grad_table_dev, ldt * tsize, 0, h->d * tsize, h->V, s));
    if (n == 0) return FR_OK;
    // keys run over [0, V]: V stands for tokens that do not count
    int total_bits = 1;
    while (total_bits < 32 && ((uint64_t)h->V >> total_bits) != 0) ++total_bits;
    const int passes = (total_bits + fr::EM_BITS - 1) / fr::EM_BITS, bits = (total_bits + passes - 1) / passes;
    const int32_t tiles = (int32_t)em_ceil(n, fr::EM_TILE);
    for (int p = 0; p < passes; ++p) {
        const uint32_t* kin = p ? h->keys[(p - 1) & 1] : nullptr;
        const int32_t* pin = p ? h->pos[(p - 1) & 1] : nullptr;
        FR_CUDA_TRY(fr::launch_pdl(fr::k_em_hist, tiles, fr::EM_THREADS, 0, s, tokens_dev, kin, n, h->V, p * bits, bits, tiles,
                                   h->counts, h->err));
        FR_CUDA_TRY(fr::scan_exclusive_i32(h->counts, h->counts, (int64_t)tiles << bits, h->temp, nullptr, s));
        FR_CUDA_TRY(fr::launch_pdl(fr::k_em_scatter, tiles, fr::EM_THREADS, 0, s, tokens_dev, kin, pin, n, h->V, p * bits,
                                   bits, tiles, (const int32_t*)h->counts, h->keys[p & 1], h->pos[p & 1], h->err));
    }
    const uint32_t* keys = h->keys[(passes - 1) & 1];
    const int32_t* order = h->pos[(passes - 1) & 1];
    cudaError_t e;
    if (grad_dtype == FR_F32)
        e = table_dtype == FR_F32
                ? em_sum<float, float>(h, grad_out_dev, ldg, keys, order, n, scale, grad_table_dev, ldt, accumulate, s)
                : em_sum<float, __nv_bfloat16>(h, grad_out_dev, ldg, keys, order, n, scale, grad_table_dev, ldt, accumulate, s);
    else
        e = table_dtype == FR_F32
                ? em_sum<__nv_bfloat16, float>(h, grad_out_dev, ldg, keys, order, n, scale, grad_table_dev, ldt, accumulate, s)
                : em_sum<__nv_bfloat16, __nv_bfloat16>(h, grad_out_dev, ldg, keys, order, n, scale, grad_table_dev, ldt,
                                                       accumulate, s);
    FR_CUDA_TRY(e);
    return FR_OK;
}

extern "C" fr_status fr_embed_status(fr_embed* h) {
    if (!h) return FR_ERR_INVALID_ARG;
    FR_CUDA_TRY(cudaStreamSynchronize(h->last_stream));
    int32_t err = 0;
    FR_CUDA_TRY(cudaMemcpy(&err, h->err, sizeof(int32_t), cudaMemcpyDeviceToHost));
    return (fr_status)err;
}

extern "C" fr_status fr_embed_clear_status(fr_embed* h, fr_stream stream) {
    if (!h) return FR_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    FR_CUDA_TRY(cudaMemsetAsync(h->err, 0, sizeof(int32_t), s));
    h->last_stream = s;
    return FR_OK;
}

extern "C" void fr_embed_destroy(fr_embed* h) {
    if (!h) return;
    em_free(h);
}
