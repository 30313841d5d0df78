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
//   k_em_small    the gradient of few tokens in one kernel.
//   k_em_hist / k_em_scatter   otherwise a stable radix sort of the tokens with
//                 their positions, 9 bits a pass (two passes for V < 2^18).
//   k_em_sum      the sorted positions in chunks of EM_CHUNK: a CTA adds a
//                 chunk's rows, a column group per thread, and writes the
//                 finished tokens; a token that reaches over a chunk's edge
//                 leaves fp32 partials, which the last chunk to arrive adds in
//                 order, in two levels.  More CTAs zero the rows that no token
//                 fell on.
//
// The sort is stable and the partials are joined in order, so a sum's order
// depends on the tokens and d alone: no floating-point atomics.
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
constexpr int EM_TILE = 1024;       // tokens that a sorting CTA ranks at a time
constexpr int EM_BITS = 9;          // most digit bits of a sort pass
constexpr int EM_SORT_CTAS = 128;   // most CTAs of a sort pass
constexpr int EM_CHUNK = 32;        // sorted positions per CTA of the sum
constexpr int EM_JOIN = 32;         // chunks of a long run that are added together first
// Rows in flight per thread of the sum: more cost registers and so CTAs per SM (20,257
// unaligned fp32 rows of 837 added to bf16: 8 rows 100 us, 16 rows 117).
template <int VEC>
constexpr int EM_UNROLL = VEC == 8 ? 4 : 8;
constexpr int EM_ZERO_ROWS = 128;   // table rows per CTA that zeros
constexpr int EM_SMALL = 2048;      // most tokens of the gradient in one kernel, and most
constexpr int64_t EM_SMALL_READS = 1 << 24;  // tokens that its CTAs may read together
constexpr int EM_SMALL_THREADS = 128;
template <int VEC>
constexpr int EM_SMALL_GROUPS = VEC == 8 ? 1 : 4;  // groups of 32 * VEC columns per CTA of that form

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
// The same past L1: what other CTAs wrote.
template <int VEC>
__device__ __forceinline__ void em_load_cg(const float* p, float (&v)[VEC]) {
    if (VEC == 8) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(p)), b = __ldcg(reinterpret_cast<const float4*>(p + 4));
        v[0] = a.x, v[1 % VEC] = a.y, v[2 % VEC] = a.z, v[3 % VEC] = a.w;
        v[4 % VEC] = b.x, v[5 % VEC] = b.y, v[6 % VEC] = b.z, v[7 % VEC] = b.w;
    } else {
        v[0] = __ldcg(p);
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

// Lanes whose digit equals this lane's (digits of `bits` bits; lanes that are
// not live match nobody).  A ballot per bit: __match_any_sync takes a round per
// distinct value, twice as long on spread tokens.
__device__ __forceinline__ uint32_t em_match(uint32_t digit, int bits, bool live) {
    uint32_t same = __ballot_sync(0xffffffffu, live);
    for (int b = 0; b < bits; ++b) {
        const uint32_t set = __ballot_sync(0xffffffffu, digit >> b & 1u);
        same &= digit >> b & 1u ? set : ~set;
    }
    return same;
}

// Digit counts of the `per` keys of each CTA: counts[cta * bins + digit].  The
// first pass reads the tokens themselves (kin null).  Also clears the sum's counters.
__global__ void __launch_bounds__(EM_THREADS) k_em_hist(const int32_t* __restrict__ tokens,
                                                        const uint32_t* __restrict__ kin, int32_t n, int32_t per, int32_t V,
                                                        int32_t shift, int32_t bits, int32_t* __restrict__ counts,
                                                        int32_t* __restrict__ err, int32_t* __restrict__ arrived, int64_t n_arrived) {
    __shared__ int32_t h[1 << EM_BITS];
    griddep_wait();
    griddep_launch_dependents();
    const int bins = 1 << bits;
    for (int b = threadIdx.x; b < bins; b += EM_THREADS) h[b] = 0;
    for (int64_t c = blockIdx.x * EM_THREADS + threadIdx.x; c < n_arrived; c += gridDim.x * EM_THREADS) arrived[c] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * per, i1 = min(i0 + per, (int64_t)n);
#pragma unroll 4
    for (int64_t i = i0 + threadIdx.x; i < i1; i += EM_THREADS) {
        const uint32_t key = kin ? kin[i] : em_key(tokens[i], V, err);
        atomicAdd(&h[(key >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += EM_THREADS) counts[blockIdx.x * bins + b] = h[b];
}

// Stable scatter of each CTA's keys, EM_TILE at a time: a warp takes 128
// consecutive keys, 32 at a time, and ranks equal digits by lane order; the
// warps' digit counts are scanned in warp order.  Where a digit begins is
// summed from all CTAs' counts by every CTA (at most EM_SORT_CTAS x 512 reads),
// which saves a scan kernel between the two.
__global__ void __launch_bounds__(EM_THREADS) k_em_scatter(const int32_t* __restrict__ tokens,
                                                           const uint32_t* __restrict__ kin,
                                                           const int32_t* __restrict__ pin, int32_t n, int32_t per,
                                                           int32_t V, int32_t shift, int32_t bits,
                                                           const int32_t* __restrict__ counts, uint32_t* __restrict__ kout,
                                                           int32_t* __restrict__ pout, int32_t* __restrict__ err) {
    constexpr int PER = EM_TILE / EM_THREADS;             // keys per lane
    constexpr int BPT = (1 << EM_BITS) / EM_THREADS;      // digits per thread
    __shared__ int32_t cnt[EM_WARPS][1 << EM_BITS];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << bits;
    int32_t base[BPT], total = 0;  // of digits threadIdx.x * BPT + k
#pragma unroll
    for (int k = 0; k < BPT; ++k) {
        const int b = threadIdx.x * BPT + k;
        int32_t before = 0, all = 0;
        if (b < bins) {
#pragma unroll 8
            for (int t = 0; t < (int)gridDim.x; ++t) {
                const int32_t c = counts[t * bins + b];
                all += c;
                if (t < (int)blockIdx.x) before += c;
            }
        }
        base[k] = total + before;
        total += all;
    }
    int sum;
    const int32_t first = block_excl_scan(total, &sum);
#pragma unroll
    for (int k = 0; k < BPT; ++k) base[k] += first;
    const int64_t end = min((int64_t)blockIdx.x * per + per, (int64_t)n);
    for (int64_t tile = (int64_t)blockIdx.x * per; tile < end; tile += EM_TILE) {
        __syncthreads();
        for (int b = threadIdx.x; b < EM_WARPS * bins; b += EM_THREADS) cnt[b >> bits][b & (bins - 1)] = 0;
        __syncthreads();
        const int64_t i0 = tile + warp * (PER * 32);
        uint32_t key[PER];
        int32_t pos[PER], rank[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int64_t i = i0 + k * 32 + lane;
            key[k] = i < end ? (kin ? kin[i] : em_key(tokens[i], V, err)) : 0u;
            pos[k] = i < end ? (pin ? pin[i] : (int32_t)i) : 0;
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const bool live = i0 + k * 32 + lane < end;
            const uint32_t dig = (key[k] >> shift) & (bins - 1);
            const uint32_t same = em_match(dig, bits, live);
            const int before = __popc(same & ((1u << lane) - 1u));
            int32_t at = 0;
            if (live) at = cnt[warp][dig];
            __syncwarp();
            if (live && before == 0) cnt[warp][dig] = at + __popc(same);
            __syncwarp();
            rank[k] = at + before;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < BPT; ++k) {
            const int b = threadIdx.x * BPT + k;
            if (b < bins) {
#pragma unroll
                for (int w = 0; w < EM_WARPS; ++w) {
                    const int32_t c = cnt[w][b];
                    cnt[w][b] = base[k];
                    base[k] += c;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (i0 + k * 32 + lane < end) {
                const int32_t o = cnt[warp][(key[k] >> shift) & (bins - 1)] + rank[k];
                kout[o] = key[k];
                pout[o] = pos[k];
            }
        }
    }
}

// Zeros the rows of [v0, v1) that `touched` (in shared memory) does not mark, 16
// bytes a lane.  Rows that start anywhere (VEC = 1) have single elements before the
// first 16-byte border and behind the last (111,448 rows of 1,654 fp32 values: 164
// us, 268 with single elements throughout).
template <class TT, int VEC>
__device__ __forceinline__ void em_zero_rows(TT* table, int64_t ldt, int32_t d, int32_t v0, int32_t v1,
                                             const uint8_t* touched) {
    constexpr int32_t PIECE = 16 / (int32_t)sizeof(TT);
    const int lane = threadIdx.x & 31;
    for (int32_t v = v0 + (threadIdx.x >> 5); v < v1; v += blockDim.x >> 5) {
        if (touched[v - v0]) continue;
        TT* row = table + (int64_t)v * ldt;
        if (VEC == 8) {
            float zero[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) zero[k] = 0.f;
#pragma unroll 4
            for (int32_t j = lane * VEC; j < d; j += 32 * VEC) em_store<VEC>(row + j, zero);
        } else {
            const int32_t head = min(d, (int32_t)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) % 16 / sizeof(TT)));
            const int32_t pieces = (d - head) / PIECE, tail = head + pieces * PIECE;
            uint4* body = reinterpret_cast<uint4*>(row + head);
#pragma unroll 4
            for (int32_t j = lane; j < pieces; j += 32) body[j] = make_uint4(0u, 0u, 0u, 0u);
            if (lane < head) row[lane] = TT(0.f);
            if (lane < d - tail) row[tail + lane] = TT(0.f);
        }
    }
}

// One finished column group of a table row; `old` is what it held, where the sum is
// added to it (loaded beside the gradients: behind the sum its latency would show for
// every token).
template <class TT, int VEC>
__device__ __forceinline__ void em_write(TT* dst, const float (&sum)[VEC], const float (&old)[VEC], float scale, bool accumulate) {
    float v[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = accumulate ? fmaf(scale, sum[k], old[k]) : scale * sum[k];
    em_store<VEC>(dst, v);
}

// First sorted position whose key is at least `key`: 32 probes at a time (a whole
// warp).
__device__ __forceinline__ int32_t em_lower_bound(const uint32_t* __restrict__ keys, int32_t n, uint32_t key) {
    const int lane = threadIdx.x & 31;
    int32_t lo = 0, hi = n;  // the answer lies in [lo, hi]
    while (hi > lo) {
        const int32_t step = (hi - lo + 31) / 32;
        const int64_t at = lo + (int64_t)lane * step;
        const bool below = at < hi && keys[at] < key;
        const int c = __popc(__ballot_sync(0xffffffffu, below));  // probes 0 .. c - 1 lie below
        if (c == 0) return lo;
        hi = (int32_t)min((int64_t)hi, lo + (int64_t)c * step);
        lo = lo + (c - 1) * step + 1;
    }
    return lo;
}

// Chunk c holds the sorted positions [c * EM_CHUNK, ...).  Its partials:
// part[2c] the run that began in an earlier chunk, part[2c + 1] the run that
// begins here and goes on.  The chunks of a run are taken in groups of EM_JOIN
// (by chunk number).  The last of a group to arrive adds its partials in chunk
// order; the last group to arrive adds the groups' sums, so the order does not
// depend on who is last, and a token that fills the batch (padding that was not
// marked) does not leave one CTA to add all of it (65,536 equal tokens of 2,048
// bf16 values: 225 us, 544 in one level).  The CTAs behind the chunks' zero the
// rows that no token fell on, beside the sums' reads.  A CTA has as many threads
// as the columns need: latency bounds short rows (524,288 tokens of 64 values:
// 149 us, 665 with 256 threads and a search for each run's ends).  Grid: chunks
// x column blocks, then the zeroing CTAs.
template <class TG, class TT, int VEC>
__global__ void __launch_bounds__(EM_THREADS)
    k_em_sum(const TG* __restrict__ grad, int64_t ldg, int32_t d, const uint32_t* __restrict__ keys,
             const int32_t* __restrict__ order, int32_t n, int32_t V, float scale, TT* __restrict__ table, int64_t ldt,
             int32_t accumulate, float* part, int64_t pitch, int32_t* arrived, int32_t chunks, int32_t blocks) {
    __shared__ uint8_t touched[EM_ZERO_ROWS];
    __shared__ uint32_t key_s[EM_CHUNK + 2];  // the chunk's keys between its neighbours'
    __shared__ int32_t ord_s[EM_CHUNK];
    __shared__ int32_t last_s;
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x >= (uint32_t)chunks * blocks) {
        const int32_t v0 = (blockIdx.x - chunks * blocks) * EM_ZERO_ROWS, v1 = min(v0 + EM_ZERO_ROWS, V);
        for (int k = threadIdx.x; k < EM_ZERO_ROWS; k += blockDim.x) touched[k] = 0;
        __syncthreads();
        const int32_t begin = em_lower_bound(keys, n, (uint32_t)v0), end = em_lower_bound(keys, n, (uint32_t)v1);
        if (end - begin <= 16 * (int32_t)blockDim.x) {
            for (int32_t i = begin + threadIdx.x; i < end; i += blockDim.x) touched[keys[i] - v0] = 1;
        } else {
            // many tokens on few rows: a search for each row (65,536 equal tokens of 256
            // values: 50 us, 399 by reading all of them)
            for (int32_t v = v0 + threadIdx.x; v < v1; v += blockDim.x) {
                int32_t lo = begin, hi = end;
                while (lo < hi) {
                    const int32_t mid = lo + (hi - lo) / 2;
                    if (keys[mid] < (uint32_t)v)
                        lo = mid + 1;
                    else
                        hi = mid;
                }
                touched[v - v0] = lo < end && keys[lo] == (uint32_t)v;
            }
        }
        __syncthreads();
        em_zero_rows<TT, VEC>(table, ldt, d, v0, v1, touched);
        return;
    }
    const int32_t chunk = blockIdx.x / blocks, block = blockIdx.x - chunk * blocks;
    const int64_t i0 = (int64_t)chunk * EM_CHUNK;
    const int32_t j = (block * (int32_t)blockDim.x + threadIdx.x) * VEC;  // this thread's columns
    for (int k = threadIdx.x; k < EM_CHUNK + 2; k += blockDim.x) {
        const int64_t i = i0 + k - 1;
        key_s[k] = i >= 0 && i < n ? keys[i] : 0xFFFFFFFFu;
        if (k >= 1 && k <= EM_CHUNK) ord_s[k - 1] = i < n ? order[i] : 0;
    }
    __syncthreads();
    int m = (int)min((int64_t)EM_CHUNK, n - i0);
    while (m > 0 && key_s[m] >= (uint32_t)V) --m;  // tokens that do not count are sorted last
    if (m == 0) return;
    const bool head = key_s[0] == key_s[1], tail = key_s[m + 1] == key_s[m];
    // how far the first key's run reaches back and the last key's goes on: a warp's
    // probes, or a search where those are not enough
    const int64_t back = i0 - 1 - (threadIdx.x & 31), on = i0 + m + (threadIdx.x & 31);
    const uint32_t not_back = __ballot_sync(0xffffffffu, !(head && back >= 0 && keys[back] == key_s[1]));
    const uint32_t not_on = __ballot_sync(0xffffffffu, !(tail && on < n && keys[on] == key_s[m]));
    if (j < d) {
        float sum[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) sum[q] = 0.f;
        bool from_before = head;
        constexpr int U = EM_UNROLL<VEC>;
        for (int k0 = 0; k0 < m; k0 += U) {
            float v[U][VEC], old[U][VEC];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k0 + u < m) em_load<VEC>(grad + (int64_t)ord_s[k0 + u] * ldg + j, v[u]);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (accumulate && k0 + u < m && key_s[k0 + u + 2] != key_s[k0 + u + 1])
                    em_load<VEC>(table + (int64_t)key_s[k0 + u + 1] * ldt + j, old[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u;
                if (k >= m) break;
                const uint32_t key = key_s[k + 1];
#pragma unroll
                for (int q = 0; q < VEC; ++q) sum[q] += v[u][q];
                const bool ends = key_s[k + 2] != key;
                if (ends || k == m - 1) {
                    if (ends && !from_before)
                        em_write<TT, VEC>(table + (int64_t)key * ldt + j, sum, old[u], scale, accumulate != 0);
                    else
                        em_store<VEC>(part + (2 * (int64_t)chunk + (from_before ? 0 : 1)) * pitch + j, sum);
                    from_before = false;
#pragma unroll
                    for (int q = 0; q < VEC; ++q) sum[q] = 0.f;
                }
            }
        }
    }
    // the runs that reach over this chunk's edges: the first key's and, unless
    // it is the same run, the last key's
    const bool one = head && tail && key_s[1] == key_s[m];
    // whether this CTA is the last of 1 + others to come here
    const auto last = [&](int32_t* counter, int64_t others) -> bool {
        if (others == 0) return true;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) last_s = atomicAdd(counter, 1) == (int32_t)others;
        __syncthreads();
        if (!last_s) return false;
        __threadfence();
        return true;
    };
    for (int r = 0; r < 2; ++r) {
        if (!(r == 0 ? head : tail && !one)) continue;
        const uint32_t key = r == 0 ? key_s[1] : key_s[m];
        int64_t c = chunk, e = chunk;  // the run's chunks
        if (r == 0) c = (not_back ? i0 - (__ffs(not_back) - 1) : em_lower_bound(keys, n, key)) / EM_CHUNK;
        if (r == 1 || one) e = ((not_on ? i0 + m + (__ffs(not_on) - 1) : em_lower_bound(keys, n, key + 1)) - 1) / EM_CHUNK;
        const auto partial = [&](int64_t k) { return part + (2 * k + (k == c ? 1 : 0)) * pitch + j; };
        // the run's chunks of this group.  A group's counter is its first chunk's: where
        // another run begins there too, this one has no other chunk in the group.
        const int64_t k0 = max(c, (int64_t)chunk / EM_JOIN * EM_JOIN), k1 = min(e, (int64_t)chunk / EM_JOIN * EM_JOIN + EM_JOIN - 1);
        if (!last(arrived + k0 * blocks + block, k1 - k0)) continue;
        float sum[VEC];
        if (j < d) {
            em_load_cg<VEC>(partial(k0), sum);
#pragma unroll 8
            for (int64_t k = k0 + 1; k <= k1; ++k) {
                float v[VEC];
                em_load_cg<VEC>(part + 2 * k * pitch + j, v);
#pragma unroll
                for (int q = 0; q < VEC; ++q) sum[q] += v[q];
            }
        }
        const int64_t g0 = c / EM_JOIN, g1 = e / EM_JOIN;
        if (g0 != g1) {
            if (j < d) em_store<VEC>(partial(k0), sum);
            if (!last(arrived + ((int64_t)chunks + c) * blocks + block, g1 - g0)) continue;
            if (j < d) {
                em_load_cg<VEC>(partial(c), sum);
#pragma unroll 8
                for (int64_t g = g0 + 1; g <= g1; ++g) {
                    float v[VEC];
                    em_load_cg<VEC>(part + 2 * g * EM_JOIN * pitch + j, v);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) sum[q] += v[q];
                }
            }
        }
        if (j < d) {
            float old[VEC];
            if (accumulate) em_load<VEC>(table + (int64_t)key * ldt + j, old);
            em_write<TT, VEC>(table + (int64_t)key * ldt + j, sum, old, scale, accumulate != 0);
        }
    }
}

// The whole gradient of at most EM_SMALL tokens in one kernel, without a sort:
// CTA (i, column block) compares token i with all tokens; the first occurrence
// of a token adds its rows in order, four warps a quarter of the list each (256
// columns, 128 of rows that start anywhere), joined in warp order.  The CTAs behind
// those zero the rows that no token fell on.  Bound by latency: up to EM_SMALL_READS
// that costs less than the sort's launches (2,000 tokens x 391 bf16 values 17.8 us
// instead of 30.6, half as many reads 13 instead of 28; twice as many, 2,000 x 2,048:
// 31.5 and 33.6), and up to EM_SMALL tokens if few of them are common (2,000 tokens of
// which 14 differ: 25 and 28 us; all alike: 83 and 29).
template <class TG, class TT, int VEC>
__global__ void __launch_bounds__(EM_SMALL_THREADS)
    k_em_small(const TG* __restrict__ grad, int64_t ldg, int32_t d, const int32_t* __restrict__ tokens, int32_t n, int32_t V,
               float scale, TT* __restrict__ table, int64_t ldt, int32_t accumulate, int32_t blocks,
               int32_t* __restrict__ err) {
    constexpr int WARPS = EM_SMALL_THREADS / 32;
    static_assert(EM_SMALL / 32 <= EM_SMALL_THREADS, "a thread per word of hits");
    constexpr int G = EM_SMALL_GROUPS<VEC>;  // groups of 32 * VEC columns
    __shared__ uint8_t touched[EM_ZERO_ROWS];
    __shared__ uint16_t list[EM_SMALL];
    __shared__ uint32_t hits[EM_SMALL / 32];  // bit per token: it is this CTA's
    __shared__ int32_t cnt[WARPS];
    __shared__ float sums[WARPS][32 * VEC * G];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if ((int)blockIdx.x >= n * blocks) {
        const int32_t v0 = (blockIdx.x - n * blocks) * EM_ZERO_ROWS, v1 = min(v0 + EM_ZERO_ROWS, V);
        for (int k = threadIdx.x; k < EM_ZERO_ROWS; k += EM_SMALL_THREADS) touched[k] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += EM_SMALL_THREADS) {
            const int32_t t = tokens[i];
            if (t >= v0 && t < v1) touched[t - v0] = 1;
        }
        __syncthreads();
        em_zero_rows<TT, VEC>(table, ldt, d, v0, v1, touched);
        return;
    }
    const int i = blockIdx.x / blocks, j = (blockIdx.x % blocks) * 32 * VEC * G + lane * VEC;
    const uint32_t t = em_key(tokens[i], V, err);
    if (t >= (uint32_t)V) return;
    bool earlier = false;
#pragma unroll 8
    for (int k = threadIdx.x; k < ((n + 31) & ~31); k += EM_SMALL_THREADS) {
        const bool same = k < n && (uint32_t)tokens[k] == t;
        earlier |= same && k < i;
        const uint32_t hit = __ballot_sync(0xffffffffu, same);
        if (lane == 0) hits[k >> 5] = hit;
    }
    if (__syncthreads_or(earlier)) return;
    // thread w lists the tokens of word w
    uint32_t hit = threadIdx.x < (n + 31) / 32 ? hits[threadIdx.x] : 0u;
    int at = __popc(hit);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int below = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += below;
    }
    if (lane == 31) cnt[warp] = at;
    __syncthreads();
    int m = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) at += cnt[w];
        m += cnt[w];
    }
    for (at -= __popc(hit); hit; hit &= hit - 1) list[at++] = (uint16_t)(threadIdx.x * 32 + __ffs(hit) - 1);
    __syncthreads();
    float sum[G][VEC];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int q = 0; q < VEC; ++q) sum[g][q] = 0.f;
    // a warp finishes every fourth group
    float old[G][VEC];
#pragma unroll
    for (int g = 0; g < G; ++g)
        if (accumulate && g % WARPS == warp && j + g * 32 * VEC < d)
            em_load<VEC>(table + (int64_t)t * ldt + j + g * 32 * VEC, old[g]);
    const int k0 = m * warp / WARPS, k1 = m * (warp + 1) / WARPS;
#pragma unroll 4
    for (int k = k0; k < k1; ++k) {
        const TG* src = grad + (int64_t)list[k] * ldg + j;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float v[VEC];
            if (j + g * 32 * VEC < d) {
                em_load<VEC>(src + g * 32 * VEC, v);
#pragma unroll
                for (int q = 0; q < VEC; ++q) sum[g][q] += v[q];
            }
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int q = 0; q < VEC; ++q) sums[warp][(g * VEC + q) * 32 + lane] = sum[g][q];
    __syncthreads();
#pragma unroll
    for (int g = 0; g < G; ++g) {
        if (g % WARPS != warp || j + g * 32 * VEC >= d) continue;
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            sum[g][q] = sums[0][(g * VEC + q) * 32 + lane];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) sum[g][q] += sums[w][(g * VEC + q) * 32 + lane];
        }
        em_write<TT, VEC>(table + (int64_t)t * ldt + j + g * 32 * VEC, sum[g], old[g], scale, accumulate != 0);
    }
}

}  // namespace
}  // namespace fr

struct fr_embed {
    int32_t V = 0, d = 0, max_tokens = 0, device = 0;
    uint32_t* keys[2] = {};
    int32_t* pos[2] = {};
    int32_t* counts = nullptr;
    float* part = nullptr;       // [2 * chunks, pitch]
    int32_t* arrived = nullptr;  // [2, chunks, column blocks] chunks of a group, groups of a run that have arrived
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

// The keys run over [0, V]: V stands for tokens that do not count.
cudaError_t em_sort(fr_embed* h, const int32_t* tokens, int32_t n, const uint32_t** keys, const int32_t** order,
                    cudaStream_t s) {
    int total_bits = 1;
    while (total_bits < 32 && ((uint64_t)h->V >> total_bits) != 0) ++total_bits;
    const int passes = (total_bits + fr::EM_BITS - 1) / fr::EM_BITS, bits = (total_bits + passes - 1) / passes;
    const int32_t per = (int32_t)(em_ceil(em_ceil(n, fr::EM_SORT_CTAS), fr::EM_TILE) * fr::EM_TILE);
    const int64_t ctas = em_ceil(n, per);
    for (int p = 0; p < passes; ++p) {
        const uint32_t* kin = p ? h->keys[(p - 1) & 1] : nullptr;
        const int32_t* pin = p ? h->pos[(p - 1) & 1] : nullptr;
        cudaError_t e = fr::launch_pdl(fr::k_em_hist, ctas, fr::EM_THREADS, 0, s, tokens, kin, n, per, h->V, p * bits, bits,
                                       h->counts, h->err, h->arrived, p ? 0 : 2 * em_ceil(n, fr::EM_CHUNK) * em_ceil(h->d, fr::EM_THREADS));
        if (e != cudaSuccess) return e;
        e = fr::launch_pdl(fr::k_em_scatter, ctas, fr::EM_THREADS, 0, s, tokens, kin, pin, n, per, h->V, p * bits, bits,
                           (const int32_t*)h->counts, h->keys[p & 1], h->pos[p & 1], h->err);
        if (e != cudaSuccess) return e;
    }
    *keys = h->keys[(passes - 1) & 1];
    *order = h->pos[(passes - 1) & 1];
    return cudaSuccess;
}

template <class TG, class TT, int VEC>
cudaError_t em_grad(fr_embed* h, const void* grad, int64_t ldg, const int32_t* tokens, int32_t n, float scale, void* table,
                    int64_t ldt, int32_t accumulate, cudaStream_t s) {
    const int32_t blocks = (int32_t)em_ceil(h->d, 32 * VEC * fr::EM_SMALL_GROUPS<VEC>);
    const int64_t zeros = accumulate ? 0 : em_ceil(h->V, fr::EM_ZERO_ROWS);
    // By n and d alone: the two forms add in different orders, and where rows start may
    // not change a sum.  The price is paid by rows of a d that is a multiple of 8 which
    // start off 16 bytes all the same: their CTAs have 128 columns, and twice as many read
    // (1,400 tokens x 2,048 bf16 values from 2 bytes on: 50 us here, 26 sorted; added 40 and 27).
    if (n <= fr::EM_SMALL && (int64_t)n * n * em_ceil(h->d, h->d % 8 ? 128 : 256) <= fr::EM_SMALL_READS) {
        if (n * (int64_t)blocks + zeros == 0) return cudaSuccess;
        return fr::launch_pdl(fr::k_em_small<TG, TT, VEC>, n * (int64_t)blocks + zeros, fr::EM_SMALL_THREADS, 0, s,
                              (const TG*)grad, ldg, h->d, tokens, n, h->V, scale, (TT*)table, ldt, accumulate, blocks, h->err);
    }
    const uint32_t* keys;
    const int32_t* order;
    cudaError_t e = em_sort(h, tokens, n, &keys, &order, s);
    if (e != cudaSuccess) return e;
    const int32_t threads = (int32_t)std::min<int64_t>(em_ceil(em_ceil(h->d, VEC), 32) * 32, fr::EM_THREADS);
    const int64_t chunks = em_ceil(n, fr::EM_CHUNK), wide = em_ceil(h->d, threads * VEC);
    return fr::launch_pdl(fr::k_em_sum<TG, TT, VEC>, chunks * wide + zeros, threads, 0, s, (const TG*)grad, ldg, h->d, keys,
                          order, n, h->V, scale, (TT*)table, ldt, accumulate, h->part, h->pitch, h->arrived, (int32_t)chunks, (int32_t)wide);
}

template <class TG, class TT>
cudaError_t em_grad_any(fr_embed* h, const void* grad, int64_t ldg, const int32_t* tokens, int32_t n, float scale,
                        void* table, int64_t ldt, int32_t accumulate, cudaStream_t s) {
    const bool vec = em_vec(grad, ldg, sizeof(TG), h->d) && em_vec(table, ldt, sizeof(TT), h->d);
    return vec ? em_grad<TG, TT, 8>(h, grad, ldg, tokens, n, scale, table, ldt, accumulate, s)
               : em_grad<TG, TT, 1>(h, grad, ldg, tokens, n, scale, table, ldt, accumulate, s);
}

}  // namespace

extern "C" fr_status fr_embed_init(int32_t V, int32_t d, int32_t max_tokens, fr_embed** out) {
    if (!out) return FR_ERR_INVALID_ARG;
    *out = nullptr;
    if (V < 1 || V > (1 << 30) || d < 1 || d > (1 << 24) || max_tokens < 1 || max_tokens >= (1 << 30)) return FR_ERR_INVALID_ARG;
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
    const int64_t n = max_tokens;
    cudaError_t e = cudaMalloc(&h->keys[0], n * 16);
    if (e == cudaSuccess) e = cudaMalloc(&h->counts, ((size_t)(fr::EM_SORT_CTAS << fr::EM_BITS) + 2 * em_ceil(n, fr::EM_CHUNK) * em_ceil(d, fr::EM_THREADS)) * sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMalloc(&h->part, (size_t)em_ceil(n, fr::EM_CHUNK) * 2 * h->pitch * 4);
    if (e == cudaSuccess) e = fr::new_status_word(&h->err);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        em_free(h);
        return e == cudaErrorMemoryAllocation ? FR_ERR_OOM : FR_ERR_CUDA;
    }
    h->keys[1] = h->keys[0] + n;
    h->pos[0] = reinterpret_cast<int32_t*>(h->keys[1] + n);
    h->pos[1] = h->pos[0] + n;
    h->arrived = h->counts + (fr::EM_SORT_CTAS << fr::EM_BITS);
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
    auto run = grad_dtype == FR_F32 ? (table_dtype == FR_F32 ? em_grad_any<float, float> : em_grad_any<float, __nv_bfloat16>)
                                    : (table_dtype == FR_F32 ? em_grad_any<__nv_bfloat16, float>
                                                             : em_grad_any<__nv_bfloat16, __nv_bfloat16>);
    FR_CUDA_TRY(run(h, grad_out_dev, ldg, tokens_dev, n, scale, grad_table_dev, ldt, accumulate, s));
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
