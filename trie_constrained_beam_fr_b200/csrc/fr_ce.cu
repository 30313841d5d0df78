// fr_ce.cu -- softmax cross entropy of the lm_head projection, and its
// gradients, without keeping the [rows, V] logits.
//
//   x = h W^T,  lse_r = log sum_v e^(x_rv),  loss_r = lse_r - x_{r, t_r}
//   G_rv = g_r (e^(x_rv - lse_r) - [v = t_r]),  dh = G W,  dW = G^T h
//
// Rows whose target is -1 take no part: they are left out of the products
// altogether (the other rows are packed together first), so a NaN in an
// ignored row's hidden state reaches nothing and a batch that is mostly
// prompt costs only its counted rows.
//
//   k_ce_gather   packs the counted rows: hidden states, targets, (gradients:
//                 lse and g) and their row numbers.
//   k_ce_loss     tcgen05 tiles of x (256 rows x 256 tokens); the epilogue
//                 keeps a (max, scaled sum) partial per row and tile and the
//                 target's logit.  k_ce_combine: lse and loss.
//   k_ce_grad     works through the vocabulary in pieces: for a piece, tiles
//                 of x are computed again and turned into G (bf16, the only
//                 piece that is kept), then dh += G W_piece (fp32 partials
//                 over the pieces) and dW_piece = G^T h.  One launch runs the
//                 products of one piece and the G tiles of the next, so that
//                 no tile type leaves SMs idle at its end.  The transposed
//                 operands are read in place: their shared-memory tiles are
//                 MN-major.
//   k_ce_finish, k_ce_finish_few   dh = sum of the fp32 partials, rounded, at the
//                 original rows.
//
// G is rounded to bf16, the operand type of the products: half a step (2^-8)
// of each entry, the same as one rounding of the inputs.  What is rounded is
// G / scale, where the scale is max |g| times a power of two (ce_scale); it
// multiplies the fp32 sums.  So the entries at the targets, which carry most of
// a gradient whose probabilities are spread, are p - 1 times a power of two,
// without g's own rounding, when all rows have the same g (a mean), and a small
// or large g neither underflows nor overflows.  A probability below 2^-126 counts
// as 0 (the exponential flushes).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "fr.h"
#include "fr_gemm.cuh"
#include "fr_handles.h"
#include "fr_internal.cuh"

namespace fr {
namespace {

// Tokens per piece of the gradient: at least CE_PIECE_MIN, and as many as keep
// a piece of G within CE_PIECE_BYTES.  Every launch costs its start and its
// uneven end: pieces of 128, 256 and 512 MB took 11.62, 11.49 and 11.39 ms for
// the gradients of 8,192 rows (d 2,048, V 151,936).
constexpr int CE_PIECE_MIN = 4096;
constexpr int64_t CE_PIECE_BYTES = 512 << 20;
constexpr int64_t CE_PARTIALS_MORE = 1 << 16;  // for narrow tiles of small calls
constexpr float CE_L2E = 1.4426950408889634f;

// The packed rows and what belongs to them.
struct CeRows {
    __nv_bfloat16* h;  // [cap, pitch]
    int64_t pitch;
    int32_t* tgt;      // [cap]
    float* lse;        // [cap]
    float* g;          // [cap]
    int32_t* idx;      // [cap] original row
    int32_t* n;        // [1] counted rows
    float* gscale;     // [1] what g is divided by (ce_scale)
};

// What the incoming gradients are divided by before G is rounded, given the largest
// finite |g| of a counted row: that value times a power of two (so an entry p - 1 of
// equal g's still carries no rounding of g), below 2 unless it is above 2^65.  A
// quotient by the value itself would push the small g's of a mixed batch below 2^-126
// (beside 1e30, a g of 1e-10 lost all but a bit or two).  What is kept is at most
// 2^64, so no sum of the products overflows before its result does.
__device__ __forceinline__ float ce_scale(float largest) {
    if (largest == 0.f) return 1.f;
    return largest < 2.f ? largest : scalbnf(largest, -min(ilogbf(largest), 64));
}

// Rows that dW's K stages (64 rows each, at least one) run over.
__device__ __forceinline__ int32_t ce_k_rows(int32_t n) { return max((n + 63) / 64, 1) * 64; }

// A CTA packs `per` consecutive rows, CE_GATHER_ROWS at a time.  Each counts the
// counted rows before its own and in all by reading every target, so no CTA waits
// for another; four CTAs per SM at most keep those reads to a few KB for each row.
constexpr int CE_GATHER_ROWS = 8;  // a warp each
constexpr int CE_GATHER_THREADS = 256;
constexpr int CE_GATHER_CTAS = 16;  // of the gradient, at least: they share the zero rows
__global__ void __launch_bounds__(CE_GATHER_THREADS)
    k_ce_gather(const __nv_bfloat16* __restrict__ hidden, int64_t ldh, const int32_t* __restrict__ targets,
                const float* __restrict__ lse, const float* __restrict__ grad_loss, int32_t rows, int32_t per, int32_t V,
                int32_t d, CeRows out, float* __restrict__ loss_out, float* __restrict__ lse_out,
                __nv_bfloat16* __restrict__ grad_hidden, int64_t ldgh, int32_t* __restrict__ counters, int32_t n_counters,
                int32_t* __restrict__ err) {
    __shared__ int32_t before_s, total_s, pos_s[CE_GATHER_ROWS];
    __shared__ uint32_t gmax_s;
    griddep_wait();
    griddep_launch_dependents();
    const int32_t first = blockIdx.x * per, last = min(first + per, rows);
    const int32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) before_s = 0, total_s = 0, gmax_s = 0u;
    __syncthreads();
    int32_t before = 0, total = 0;
#pragma unroll 8
    for (int32_t i = tid; i < rows; i += CE_GATHER_THREADS) {
        const int32_t live = (uint32_t)targets[i] < (uint32_t)V;
        total += live;
        before += i < first ? live : 0;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) {
        atomicAdd(&before_s, before);
        atomicAdd(&total_s, total);
    }
    __syncthreads();
    const int32_t vecs = d >> 3;  // rows start on 16 bytes (checked by the caller)
    for (int32_t r0 = first; r0 < last; r0 += CE_GATHER_ROWS) {
        if (warp == 0) {
            const int32_t r = r0 + lane;
            const bool mine = lane < CE_GATHER_ROWS && r < last;
            const int32_t t = mine ? targets[r] : -1;
            const bool live = (uint32_t)t < (uint32_t)V;
            const uint32_t m = __ballot_sync(0xffffffffu, live);
            const int32_t pos = before_s + __popc(m & ((1u << lane) - 1u));
            __syncwarp();
            if (lane == 0) before_s += __popc(m);
            if (lane < CE_GATHER_ROWS) pos_s[lane] = live ? pos : -1;
            if (live) {
                out.tgt[pos] = t;
                out.idx[pos] = r;
                if (lse) {
                    out.lse[pos] = lse[r];
                    out.g[pos] = grad_loss[r];
                }
            } else if (mine) {
                const bool bad = t != -1;
                if (bad) set_error(err, FR_ERR_CODE_RANGE);
                if (loss_out) {
                    loss_out[r] = bad ? NAN : 0.f;
                    lse_out[r] = bad ? NAN : 0.f;
                }
            }
        }
        __syncthreads();
        for (int k = warp; k < CE_GATHER_ROWS && r0 + k < last; k += CE_GATHER_THREADS / 32) {
            const int32_t r = r0 + k, pos = pos_s[k];
            if (pos >= 0) {
                const uint4* src = reinterpret_cast<const uint4*>(hidden + r * ldh);
                uint4* dst = reinterpret_cast<uint4*>(out.h + pos * out.pitch);
                for (int32_t i = lane; i < vecs; i += 256) {
                    uint4 v[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (i + 32 * u < vecs) v[u] = src[i + 32 * u];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (i + 32 * u < vecs) dst[i + 32 * u] = v[u];
                }
                for (int32_t j = (vecs << 3) + lane; j < d; j += 32) out.h[pos * out.pitch + j] = hidden[r * ldh + j];
            } else if (grad_hidden) {
                for (int32_t j = lane; j < d; j += 32) grad_hidden[r * ldgh + j] = __float2bfloat16_rn(0.f);
            }
        }
        __syncthreads();
    }
    // dW's last K stage reads zeros behind the counted rows (the pitch is a multiple
    // of 8 elements)
    const int32_t n = total_s, end = lse ? ce_k_rows(n) : n;
    for (int32_t r = n + blockIdx.x; r < end; r += gridDim.x) {
        uint4* dst = reinterpret_cast<uint4*>(out.h + r * out.pitch);
        for (int32_t i = tid; i < out.pitch / 8; i += CE_GATHER_THREADS) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (blockIdx.x == 0) {
        if (tid == 0) *out.n = n;
        for (int32_t i = tid; i < n_counters; i += CE_GATHER_THREADS) counters[i] = 0;
    }
    if (lse && blockIdx.x == gridDim.x - 1) {
        float m = 0.f;
#pragma unroll 8
        for (int32_t i = tid; i < rows; i += CE_GATHER_THREADS) {
            const float g = fabsf(grad_loss[i]);
            if ((uint32_t)targets[i] < (uint32_t)V && g < INFINITY) m = fmaxf(m, g);
        }
        // non-negative floats order as their bits
        const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if (lane == 0) atomicMax(&gmax_s, w);
        __syncthreads();
        if (tid == 0) *out.gscale = ce_scale(__uint_as_float(gmax_s));
    }
}

// Rows of a tile: a pair's, or a single CTA's where there are at most 128 rows.
template <bool PAIR_>
constexpr int CE_TM = PAIR_ ? GM_TILE : GM_HALF;

// A copy of bn rows of a K-major B operand in boxes of half of them: a CTA's half,
// or both.
template <bool PAIR_>
__device__ __forceinline__ void ce_load_b(const CUtensorMap* map, uint8_t* b, uint32_t bar, int k, int n, int rank, int bn) {
    gm_tma_load<PAIR_>(map, b, bar, k, n + rank * (bn / 2));
    if constexpr (!PAIR_) gm_tma_load<PAIR_>(map, b + bn / 2 * GM_KB_BYTES, bar, k, n + bn / 2);
}

// The same of an MN-major B operand, `share` columns a CTA in boxes of 64.
template <bool PAIR_>
__device__ __forceinline__ void ce_load_b_mn(const CUtensorMap* map, uint8_t* b, uint32_t bar, int n, int k, int rank, int share) {
#pragma unroll
    for (int j = 0; j < (PAIR_ ? 2 : 4); ++j)
        if (j * 64 < share) gm_tma_load<PAIR_>(map, b + j * 8192, bar, n + rank * share + j * 64, k);
}

// BN: tokens of a tile, known to the compiler (256) or not (0: narrow_bn).  Known,
// 2,048 rows x 151,936 tokens x 2,048 values took 915 us instead of 950.
template <bool PAIR_, int BN>
struct CeLoss {
    static constexpr bool I8 = false, STAGED = false, DYNAMIC = false, PAIR = PAIR_;
    static constexpr int STAGES = PAIR ? 7 : 4, TM = CE_TM<PAIR_>;
    struct Tile {
        int nk, m0, n, n0;
        uint32_t idesc;
    };
    struct State {
        int32_t n, m_tiles;
    };
    CUtensorMap map_h, map_w;
    CeRows rows;
    int32_t V, k_blocks, n_tiles;
    int32_t narrow_bn;
    int32_t single_a_rows;  // rows of a single CTA's copy of h
    float2* partial;  // [rows, 2 * n_tiles] (max, scaled sum) of half a tile's tokens each
    float* xt;        // [cap] the target's logit

    __device__ __forceinline__ int bn() const { return BN ? BN : narrow_bn; }
    __device__ __forceinline__ int a_rows() const { return PAIR ? GM_HALF : single_a_rows; }
    __device__ __forceinline__ void prefetch() const {
        gm_prefetch(&map_h);
        gm_prefetch(&map_w);
    }
    __device__ __forceinline__ State begin() const {
        const int32_t n = *rows.n;
        return {n, (n + TM - 1) / TM};
    }
    __device__ __forceinline__ int32_t* counter() const { return nullptr; }
    __device__ __forceinline__ bool tile(const State& st, uint32_t g, Tile& t) const {
        if (g >= (uint32_t)st.m_tiles * (uint32_t)n_tiles) return false;
        int32_t m, n;
        gm_grouped(g, st.m_tiles, n_tiles, m, n);
        t.m0 = m * TM;
        t.n = n;
        t.n0 = n * bn();
        t.nk = k_blocks;
        t.idesc = gm_idesc(false, PAIR, false, false, bn());
        return true;
    }
    __device__ __forceinline__ uint32_t stage_bytes(const Tile&) const { return ((PAIR ? 2 : 1) * a_rows() + bn()) * GM_KB_BYTES; }
    __device__ __forceinline__ bool a_mn(const Tile&) const { return false; }
    __device__ __forceinline__ bool b_mn(const Tile&) const { return false; }
    __device__ __forceinline__ void load(const Tile& t, int kb, int rank, uint8_t* a, uint8_t* b, uint32_t bar) const {
        gm_tma_load<PAIR>(&map_h, a, bar, kb * 64, t.m0 + rank * GM_HALF);
        ce_load_b<PAIR>(&map_w, b, bar, kb * 64, t.n0, rank, bn());
    }
    __device__ __forceinline__ void epilogue(const State& st, const Tile& t, uint32_t taddr, int r, int half, const GmStage&,
                                             GmRelease<PAIR>& release) const {
        const int cols = (bn() / 2 + 31) & ~31, c1 = min((half + 1) * cols, bn());
        const int row = t.m0 + r;
        if (row - (int)(threadIdx.x & 31) >= st.n) return;
        const int32_t tgt = row < st.n ? rows.tgt[row] : -1;
        float m = -INFINITY, s = 0.f;
#pragma unroll 1
        for (int c = half * cols; c < c1 && t.n0 + c < V; c += 32) {
            const int n = t.n0 + c;
            float v[32];
            tc_tmem_ld32(taddr + (uint32_t)c, v);
            if (c + 32 == c1) release();
            if ((uint32_t)(tgt - n) < 32u) {
                float x = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (n + i == tgt) x = v[i];
                xt[row] = x;
            }
            if (n + 32 > V) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (n + i >= V) v[i] = -INFINITY;
            }
            gm_lse_fold(v, m, s);
        }
        if (row < st.n) partial[(int64_t)row * 2 * n_tiles + 2 * t.n + half] = make_float2(m, s);
    }
};

template <class P>
__global__ void __launch_bounds__(GM_THREADS, 1) k_ce_loss(const __grid_constant__ P p, const GmCtl ctl) {
    gm_run(p, ctl);
}

__global__ void __launch_bounds__(256) k_ce_combine(const float2* __restrict__ partial, int32_t n_parts, CeRows rows,
                                                    const float* __restrict__ xt, float* __restrict__ loss,
                                                    float* __restrict__ lse, int32_t* __restrict__ err) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t c = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (c >= *rows.n) return;
    const float v = gm_lse_combine(partial + c * n_parts, n_parts);
    if ((threadIdx.x & 31) == 0) {
        const int32_t r = rows.idx[c];
        if (!isfinite(v)) set_error(err, FR_ERR_NAN_LOGIT);
        lse[r] = v;
        loss[r] = v - xt[c];
    }
}

// One launch of the gradient: the products of one piece (tokens [v0, v1)) and
// the G tiles of the next (tokens [w0, w1), into the other buffer).  Empty ranges
// leave their part out.
template <bool PAIR_, int BN>
struct CeGrad {
    static constexpr bool I8 = false, STAGED = true, DYNAMIC = true, PAIR = PAIR_;
    static constexpr int STAGES = PAIR ? 6 : 4, TM = CE_TM<PAIR_>;
    enum { DH, DW, GT };
    struct Tile {
        int nk, type, m0, n0, k0, split;
        uint32_t idesc;
    };
    struct State {
        int32_t n, m_tiles, dh_tiles, dw_tiles, g_tiles, dw_nk, dh_per;
        bool dw_first;
        float scale;
    };
    CUtensorMap map_h_k, map_h_mn;   // packed rows: K-major (128 x 64) and MN-major (64 x 64) boxes
    CUtensorMap map_w_k, map_w_mn;   // weight: K-major (128 x 64) and MN-major (64 x 64) boxes
    CUtensorMap map_g_k, map_g_mn;   // G, two buffers' rows one after another
    CUtensorMap map_g_out;           // the same: 32 x 64 boxes
    CUtensorMap map_dw;              // the caller's dW, where its rows start on 16 bytes: 32 x 64 boxes
    CeRows rows;
    int32_t* next_tile;              // tiles taken so far beyond the pairs' first two
    int32_t V, d, d_tiles, splits, first;
    int32_t v0, v1, w0, w1;
    int32_t narrow_bn;               // tokens of a G tile where BN is 0, a multiple of 64
    int32_t single_a_rows;           // rows of a single CTA's copy of h or G (K-major)
    int32_t g_read, g_write;         // first rows of the buffers whose products run / whose tiles are computed
    CUtensorMap map_dh;              // [splits, dh_rows] rows of fp32 partials: 32 x 32 boxes
    int32_t dh, dh_rows;             // whether dh is wanted; rows of one split
    __nv_bfloat16* dw;               // the caller's dW, null: no dW
    int64_t ldw;
    int32_t dw_staged;               // columns of dW that go out through shared memory and TMA

    __device__ __forceinline__ int bn() const { return BN ? BN : narrow_bn; }
    __device__ __forceinline__ int a_rows() const { return PAIR ? GM_HALF : single_a_rows; }
    __device__ __forceinline__ void prefetch() const {
        gm_prefetch(&map_h_k);
        gm_prefetch(&map_w_k);
        gm_prefetch(&map_g_k);
        gm_prefetch(&map_w_mn);
        gm_prefetch(&map_g_mn);
        gm_prefetch(&map_h_mn);
        gm_prefetch(&map_g_out);
    }
    __device__ __forceinline__ State begin() const {
        State st;
        st.n = *rows.n;
        st.scale = *rows.gscale;
        st.m_tiles = max((st.n + TM - 1) / TM, 1);
        st.dh_tiles = dh && v1 > v0 && st.n ? st.m_tiles * d_tiles * splits : 0;
        st.dw_tiles = dw && v1 > v0 ? (v1 - v0 + TM - 1) / TM * d_tiles : 0;
        st.g_tiles = w1 > w0 ? (w1 - w0 + bn() - 1) / bn() * st.m_tiles : 0;
        st.dw_nk = ce_k_rows(st.n) / 64;
        st.dh_per = ((v1 - v0 + 63) / 64 + splits - 1) / splits;
        st.dw_first = st.dw_nk > st.dh_per;
        return st;
    }
    __device__ __forceinline__ int32_t* counter() const { return next_tile; }
    // The longest tiles first (dh or dW by their K stages, then G), so that the
    // short ones even out the pairs' ends.
    __device__ __forceinline__ bool tile(const State& st, uint32_t at, Tile& t) const {
        if (at >= (uint32_t)(st.dh_tiles + st.dw_tiles + st.g_tiles)) return false;
        int g = (int)at;
        if (st.dw_first && g < st.dh_tiles + st.dw_tiles) g += g < st.dw_tiles ? st.dh_tiles : -st.dw_tiles;
        if (g < st.dh_tiles) {
            const int kb = (v1 - v0 + 63) / 64, per = st.dh_per;
            t.type = DH;
            // d fastest: pairs running together read each row of G once
            t.n0 = g % d_tiles * GM_TILE;
            g /= d_tiles;
            t.m0 = g % st.m_tiles * TM;
            t.split = g / st.m_tiles;
            t.k0 = t.split * per;
            t.nk = max(min(per, kb - t.k0), 0);
            t.idesc = gm_idesc(false, PAIR, false, true, width(t));
            return true;
        }
        g -= st.dh_tiles;
        if (g < st.dw_tiles) {
            t.type = DW;
            t.n0 = g % d_tiles * GM_TILE;
            t.m0 = g / d_tiles * TM;
            t.k0 = 0;
            t.nk = st.dw_nk;
            t.idesc = gm_idesc(false, PAIR, true, true, width(t));
            return true;
        }
        g -= st.dw_tiles;
        t.type = GT;
        int32_t m, n;
        // last tokens first: the weight's end is what the loss left in L2, and its
        // start is what dh's first tiles then find there
        const int32_t n_tiles = (w1 - w0 + bn() - 1) / bn();
        gm_grouped(g, st.m_tiles, n_tiles, m, n);
        t.m0 = m * TM;
        t.n0 = (n_tiles - 1 - n) * bn();
        t.k0 = 0;
        t.nk = (d + 63) / 64;
        t.idesc = gm_idesc(false, PAIR, false, false, bn());
        return true;
    }
    // Columns of a dh or dW tile: in the small calls' kernels those that are there,
    // rounded up to a multiple of 32; else all (gradients of 8,192 rows x 151,936 tokens:
    // 11.4 ms, and 12.6 with a width that the compiler does not know).
    __device__ __forceinline__ int width(const Tile& t) const { return BN ? GM_TILE : min((d - t.n0 + 31) & ~31, GM_TILE); }
    __device__ __forceinline__ uint32_t stage_bytes(const Tile& t) const {
        constexpr int CTAS = PAIR ? 2 : 1;
        if (BN) return CTAS * 2 * GM_OP_BYTES;
        if (t.type == GT) return (CTAS * a_rows() + bn()) * GM_KB_BYTES;
        return CTAS * ((t.type == DW ? GM_HALF : a_rows()) + ((width(t) / CTAS + 63) & ~63)) * GM_KB_BYTES;
    }
    __device__ __forceinline__ bool a_mn(const Tile& t) const { return t.type == DW; }
    __device__ __forceinline__ bool b_mn(const Tile& t) const { return t.type != GT; }
    __device__ __forceinline__ void load(const Tile& t, int kb, int rank, uint8_t* a, uint8_t* b, uint32_t bar) const {
        const int k = (t.k0 + kb) * 64, m = t.m0 + rank * GM_HALF;
        if (t.type == GT) {
            gm_tma_load<PAIR>(&map_h_k, a, bar, k, m);
            ce_load_b<PAIR>(&map_w_k, b, bar, k, w0 + t.n0, rank, bn());
        } else if (t.type == DH) {
            gm_tma_load<PAIR>(&map_g_k, a, bar, k, g_read + m);
            ce_load_b_mn<PAIR>(&map_w_mn, b, bar, t.n0, v0 + k, rank, width(t) / (PAIR ? 2 : 1));
        } else {
            gm_tma_load<PAIR>(&map_g_mn, a, bar, m, g_read + k);
            gm_tma_load<PAIR>(&map_g_mn, a + 8192, bar, m + 64, g_read + k);
            ce_load_b_mn<PAIR>(&map_h_mn, b, bar, t.n0, k, rank, width(t) / (PAIR ? 2 : 1));
        }
    }
    __device__ __forceinline__ void epilogue(const State& st, const Tile& t, uint32_t taddr, int r, int half, const GmStage& sg,
                                             GmRelease<PAIR>& release) const {
        const int c0 = half * GM_EPI_COLS;
        const int row = t.m0 + r, lane = threadIdx.x & 31, row0 = row - lane;
        if (t.type == GT) {
            if (row0 >= ce_k_rows(st.n)) return;  // rows that no product sums over
            const int cols = (bn() / 2 + 63) & ~63, c1 = min((half + 1) * cols, bn());
            const bool live = row < st.n;
            const float g = live ? __fdiv_rn(rows.g[row], st.scale) : 0.f, nl = live ? -rows.lse[row] * CE_L2E : 0.f;
            const int32_t tgt = live ? rows.tgt[row] - w0 - t.n0 : -1;  // column in the tile
            const int width = w1 - w0 - t.n0;  // columns of this tile that are tokens
#pragma unroll 1
            for (int c = half * cols; c < c1 && c < width; c += 64) {
                float v[64];
                gm_ld64(taddr + (uint32_t)c, v);
                if (c + 64 == c1) release();
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const float p = tc_ex2(fmaf(v[i], CE_L2E, nl)) - (c + i == tgt ? 1.f : 0.f);
                    v[i] = live && c + i < width ? p * g : 0.f;  // zeros feed the products' ragged ends
                }
                gm_stage64(sg, &map_g_out, lane, v, t.n0 + c, g_write + row0);
            }
        } else if (t.type == DH) {
            if (t.nk == 0 && !first) return;  // a split without tokens adds nothing
#pragma unroll 1
            for (int c = c0; c < c0 + GM_EPI_COLS && t.n0 + c < d; c += 32) {
                float v[32];
                tc_tmem_ld32(taddr + (uint32_t)c, v);
                if (c + 32 == c0 + GM_EPI_COLS) release();
                if (t.nk == 0) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
                }
                // one addition per launch and value: the order is that of the pieces
                if (first)
                    gm_stage32<false>(sg, &map_dh, lane, v, t.n0 + c, t.split * dh_rows + row0);
                else
                    gm_stage32<true>(sg, &map_dh, lane, v, t.n0 + c, t.split * dh_rows + row0);
            }
        } else {
            const int v = v0 + row0;  // the warp's first row
#pragma unroll 1
            for (int c = c0; c < c0 + GM_EPI_COLS && t.n0 + c < d; c += 64) {
                float x[64];
                gm_ld64(taddr + (uint32_t)c, x);
                if (c + 64 == c0 + GM_EPI_COLS) release();
#pragma unroll
                for (int i = 0; i < 64; ++i) x[i] *= st.scale;
                if (v >= v1) continue;
                if (t.n0 + c < dw_staged) {
                    gm_stage64(sg, &map_dw, lane, x, t.n0 + c, v);
                } else {
                    gm_put(sg, lane, x);
                    gm_write_plain(sg, lane, dw + v * ldw + t.n0 + c, ldw, min(32, v1 - v), min(64, d - t.n0 - c));
                }
            }
        }
    }
};

template <class P>
__global__ void __launch_bounds__(GM_THREADS, 1) k_ce_grad(const __grid_constant__ P p, const GmCtl ctl) {
    gm_run(p, ctl);
}

// x += y.
__device__ __forceinline__ void ce_add(float4& x, const float4& y) {
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
}

// 4 columns of dh: times G's scale, rounded.
__device__ __forceinline__ void ce_put(__nv_bfloat16* dst, int32_t j, int32_t d, float4 x, float scale, bool vec) {
    x.x *= scale;
    x.y *= scale;
    x.z *= scale;
    x.w *= scale;
    if (vec && j + 4 <= d) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
        *reinterpret_cast<uint2*>(dst + j) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
        dst[j] = __float2bfloat16_rn(x.x);
        if (j + 1 < d) dst[j + 1] = __float2bfloat16_rn(x.y);
        if (j + 2 < d) dst[j + 2] = __float2bfloat16_rn(x.z);
        if (j + 3 < d) dst[j + 3] = __float2bfloat16_rn(x.w);
    }
}

// A CTA per packed row: the splits' partials in split order, one rounding.
constexpr int CE_FINISH_THREADS = 256;
__global__ void __launch_bounds__(CE_FINISH_THREADS)
    k_ce_finish(const float* __restrict__ dh, int64_t dh_split, int32_t splits, int32_t d, CeRows rows,
                __nv_bfloat16* __restrict__ grad_hidden, int64_t ldgh, int32_t vec) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t c = blockIdx.x;
    if (c >= *rows.n) return;
    const float scale = *rows.gscale;
    const float* src = dh + c * rows.pitch;
    __nv_bfloat16* dst = grad_hidden + rows.idx[c] * ldgh;
    for (int32_t j = threadIdx.x * 4; j < d; j += 4 * CE_FINISH_THREADS) {
        float4 x = *reinterpret_cast<const float4*>(src + j);
#pragma unroll 8
        for (int k = 1; k < splits; ++k) ce_add(x, *reinterpret_cast<const float4*>(src + k * dh_split + j));
        ce_put(dst, j, d, x, scale, vec != 0);
    }
}

// The same for few rows with several splits: `groups` threads share the splits of 4
// columns (each takes consecutive ones) and are joined in order, and a row's columns
// are shared by `col_ctas` CTAs (13 rows x 1,815 values x 32 splits: 20.6 us by the
// kernel above, 6.6 by this one; 6,400 rows x 1,000 values x 2 splits: 11.0 and 16.8).
__global__ void __launch_bounds__(CE_FINISH_THREADS)
    k_ce_finish_few(const float* __restrict__ dh, int64_t dh_split, int32_t splits, int32_t groups, int32_t col_ctas,
                    int32_t d, CeRows rows, __nv_bfloat16* __restrict__ grad_hidden, int64_t ldgh, int32_t vec) {
    __shared__ float4 sums[CE_FINISH_THREADS];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t c = blockIdx.x / col_ctas;
    if (c >= *rows.n) return;
    const int32_t width = CE_FINISH_THREADS / groups, q = threadIdx.x % width, group = threadIdx.x / width;
    const int32_t k0 = splits * group / groups, k1 = splits * (group + 1) / groups;
    const int32_t j = (blockIdx.x % col_ctas * width + q) * 4;
    const float* src = dh + c * rows.pitch;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < d) {
#pragma unroll 8
        for (int k = k0; k < k1; ++k) ce_add(x, *reinterpret_cast<const float4*>(src + k * dh_split + j));
    }
    sums[threadIdx.x] = x;
    __syncthreads();
    if (group != 0 || j >= d) return;
    for (int k = 1; k < groups; ++k) ce_add(x, sums[k * width + q]);
    ce_put(grad_hidden + rows.idx[c] * ldgh, j, d, x, *rows.gscale, vec != 0);
}

int64_t ce_round(int64_t x, int64_t q) { return (x + q - 1) / q * q; }

// Splits of dh's token axis within a piece of kb K stages when there are few rows
// (then dh's tiles are few and long): four tiles for every unit (pair or single
// CTA) up to 32 splits, more while units have none, tiles of four stages at least.
int32_t ce_splits(int32_t units, int64_t m_tiles, int64_t d_tiles, int64_t kb) {
    const int64_t tiles = m_tiles * d_tiles;
    int64_t splits = std::max(std::min<int64_t>(32, 4 * units / tiles), units / tiles);
    splits = std::max<int64_t>(1, std::min(splits, (kb + 3) / 4));
    const int64_t per = (kb + splits - 1) / splits;
    return (int32_t)((kb + per - 1) / per);  // none of them empty
}

}  // namespace
}  // namespace fr

struct fr_ce {
    int32_t V = 0, d = 0, max_rows = 0, n_tiles = 0, sms = 0, device = 0, piece = 0;
    int64_t cap = 0;
    fr::CeRows rows{};
    float2* partial = nullptr;       // partials values: at least [cap, 2 * n_tiles]
    int64_t partials = 0;
    float* xt = nullptr;             // [cap]
    __nv_bfloat16* g = nullptr;      // two buffers (one if V is one piece) of g_elems values
    int64_t g_elems = 0;
    float* dh = nullptr;             // fp32 partials of dh
    int32_t* counters = nullptr;     // [pieces + 1] tile counters of the gradient's launches
    int32_t* err = nullptr;
    cudaStream_t last_stream = nullptr;
    uint64_t wait_ns = FR_WAIT_LIMIT_NS;
    int32_t starve = 0;
};

namespace {

void ce_free(fr_ce* h) {
    cudaFree(h->rows.h);
    cudaFree(h->rows.tgt);
    cudaFree(h->partial);
    cudaFree(h->g);
    cudaFree(h->dh);
    cudaFree(h->err);
    delete h;
}

// What the loss and the gradient both ask of their arguments.
bool ce_bad_inputs(const fr_ce* h, const void* hidden, int64_t ldh, const void* weight, int64_t ldw,
                   const int32_t* targets, int32_t rows, const void* lse) {
    return !h || !hidden || !weight || !targets || !lse || rows < 0 || rows > h->max_rows || ldh < h->d || ldw < h->d ||
           (ldh & 7) || (ldw & 7) || (reinterpret_cast<uintptr_t>(hidden) & 15u) ||
           (reinterpret_cast<uintptr_t>(weight) & 15u) || (reinterpret_cast<uintptr_t>(targets) & 3u) ||
           (reinterpret_cast<uintptr_t>(lse) & 3u);
}

bool ce_on_device(const fr_ce* h) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == h->device;
}

// Rows per CTA of k_ce_gather.
int32_t ce_gather_rows(const fr_ce* h, int32_t rows) {
    return (int32_t)fr::ce_round(std::max((rows + 4 * h->sms - 1) / (4 * h->sms), 1), fr::CE_GATHER_ROWS);
}

// Tokens of a tile of x.  How many rows count, and so how many rounds the pairs have,
// is not known here: narrow tiles where a round is not full in any case, and for the
// single CTAs, whose one row tile is certain.
int32_t ce_width(const fr_ce* h, int32_t rows, int32_t step) {
    if (rows <= fr::GM_HALF) return fr::gm_width(1, h->V, h->sms, step);
    const int64_t m_tiles = fr::ce_round(rows, fr::GM_TILE) / fr::GM_TILE, units = h->sms / 2;
    return m_tiles * h->n_tiles > units ? fr::GM_TILE : fr::gm_width(m_tiles, h->V, units, step);
}

template <bool PAIR, int BN>
fr_status ce_run_loss(fr_ce* h, int32_t bn, const void* hidden_dev, int64_t ldh, const void* weight_dev, int64_t ldw,
                      const int32_t* targets_dev, int32_t rows, float* loss_dev, float* lse_dev, cudaStream_t s) {
    constexpr int TM = fr::CE_TM<PAIR>;
    fr::CeLoss<PAIR, BN> p{};
    const int64_t m_tiles = fr::ce_round(rows, TM) / TM;
    p.narrow_bn = bn;
    if (!fr::gm_encode(&p.map_w, 2, weight_dev, h->V, h->d, ldw * 2, bn / 2)) return FR_ERR_CUDA;
    p.single_a_rows = fr::gm_a_rows(rows);
    if (!fr::gm_encode(&p.map_h, 2, h->rows.h, h->cap, h->d, h->rows.pitch * 2, PAIR ? fr::GM_HALF : p.single_a_rows)) return FR_ERR_CUDA;
    p.rows = h->rows;
    p.V = h->V;
    p.k_blocks = (h->d + 63) / 64;
    p.n_tiles = (h->V + bn - 1) / bn;
    p.partial = h->partial;
    p.xt = h->xt;
    const int32_t per = ce_gather_rows(h, rows);
    FR_CUDA_TRY(fr::launch_pdl(fr::k_ce_gather, (rows + per - 1) / per, fr::CE_GATHER_THREADS, 0, s,
                               (const __nv_bfloat16*)hidden_dev, ldh, targets_dev, (const float*)nullptr,
                               (const float*)nullptr, rows, per, h->V, h->d, h->rows, loss_dev, lse_dev, (__nv_bfloat16*)nullptr, (int64_t)0, (int32_t*)nullptr, 0, h->err));
    fr::GmCtl ctl{h->err, h->wait_ns, h->starve};
    FR_CUDA_TRY(fr::gm_launch(fr::k_ce_loss<fr::CeLoss<PAIR, BN>>, m_tiles * p.n_tiles, h->sms, s, p, ctl));
    FR_CUDA_TRY(fr::launch_pdl(fr::k_ce_combine, ((int64_t)rows + 7) / 8, 256, 0, s, (const float2*)h->partial, 2 * p.n_tiles,
                               h->rows, (const float*)h->xt, loss_dev, lse_dev, h->err));
    return FR_OK;
}

template <bool PAIR, int BN>
fr_status ce_run_grad(fr_ce* h, int32_t piece, int32_t bn, const void* hidden_dev, int64_t ldh, const void* weight_dev, int64_t ldw,
                      const int32_t* targets_dev, const float* lse_dev, const float* grad_loss_dev, int32_t rows,
                      void* grad_hidden_dev, int64_t ldgh, void* grad_weight_dev, int64_t ldgw, cudaStream_t s) {
    constexpr int TM = fr::CE_TM<PAIR>;
    fr::CeGrad<PAIR, BN> p{};
    __nv_bfloat16* gh = (__nv_bfloat16*)grad_hidden_dev;
    const int64_t m_tiles = fr::ce_round(std::max(rows, 1), TM) / TM;  // no rows: dW is still written (zeros)
    const int64_t g_rows = fr::ce_round(std::max(rows, 1), fr::GM_TILE);
    const int32_t pieces = (h->V + piece - 1) / piece;
    const int64_t g_all = std::min(pieces, 2) * g_rows, g_pitch = (int64_t)piece * 2;
    const int32_t units = PAIR ? h->sms / 2 : h->sms;
    p.narrow_bn = bn;
    if (!fr::gm_encode(&p.map_w_k, 2, weight_dev, h->V, h->d, ldw * 2, bn / 2) ||
        !fr::gm_encode(&p.map_w_mn, 2, weight_dev, h->V, h->d, ldw * 2, 64))
        return FR_ERR_CUDA;
    p.single_a_rows = fr::gm_a_rows(std::max(rows, 1));
    if (!fr::gm_encode(&p.map_g_k, 2, h->g, g_all, piece, g_pitch, PAIR ? fr::GM_HALF : p.single_a_rows) ||
        !fr::gm_encode(&p.map_g_mn, 2, h->g, g_all, piece, g_pitch, 64) ||
        !fr::gm_encode(&p.map_g_out, 2, h->g, g_all, piece, g_pitch, 32))
        return FR_ERR_CUDA;
    if (!fr::gm_encode(&p.map_h_k, 2, h->rows.h, h->cap, h->d, h->rows.pitch * 2, PAIR ? fr::GM_HALF : p.single_a_rows) ||
        !fr::gm_encode(&p.map_h_mn, 2, h->rows.h, h->cap, h->d, h->rows.pitch * 2, 64))
        return FR_ERR_CUDA;
    p.rows = h->rows;
    p.V = h->V;
    p.d = h->d;
    p.d_tiles = (h->d + fr::GM_TILE - 1) / fr::GM_TILE;
    p.splits = fr::ce_splits(units, m_tiles, p.d_tiles, (std::min(piece, h->V) + 63) / 64);
    p.dh = gh != nullptr;
    p.dh_rows = (int32_t)(m_tiles * TM);
    if (!fr::gm_encode(&p.map_dh, 4, h->dh, (int64_t)p.splits * p.dh_rows, h->rows.pitch, h->rows.pitch * 4, 32))
        return FR_ERR_CUDA;
    p.dw = (__nv_bfloat16*)grad_weight_dev;
    p.ldw = ldgw;
    if (p.dw && (reinterpret_cast<uintptr_t>(grad_weight_dev) & 15u) == 0 && (ldgw & 7) == 0)
        p.dw_staged = fr::gm_staged_columns(h->d, 2);
    if (p.dw_staged && !fr::gm_encode(&p.map_dw, 2, grad_weight_dev, h->V, h->d, ldgw * 2, 32)) return FR_ERR_CUDA;
    const int32_t per = ce_gather_rows(h, rows);
    FR_CUDA_TRY(fr::launch_pdl(fr::k_ce_gather, std::max((rows + per - 1) / per, fr::CE_GATHER_CTAS), fr::CE_GATHER_THREADS, 0, s,
                               (const __nv_bfloat16*)hidden_dev, ldh, targets_dev, lse_dev, grad_loss_dev, rows, per, h->V,
                               h->d, h->rows, (float*)nullptr, (float*)nullptr, gh, ldgh, h->counters, pieces + 1, h->err));
    fr::GmCtl ctl{h->err, h->wait_ns, h->starve};
    for (int32_t k = 0; k <= pieces; ++k) {
        p.v0 = p.v1 = p.w0 = p.w1 = 0;
        int64_t tiles = 0;
        if (k > 0) {
            p.v0 = (k - 1) * piece;
            p.v1 = std::min(h->V, k * piece);
            p.first = k == 1;
            p.g_read = (int32_t)((k - 1) % 2 * g_rows);
            if (gh) tiles += m_tiles * p.d_tiles * p.splits;
            if (p.dw) tiles += (int64_t)(p.v1 - p.v0 + TM - 1) / TM * p.d_tiles;
        }
        if (k < pieces) {
            p.w0 = k * piece;
            p.w1 = std::min(h->V, (k + 1) * piece);
            p.g_write = (int32_t)(k % 2 * g_rows);
            tiles += (int64_t)(p.w1 - p.w0 + bn - 1) / bn * m_tiles;
        }
        p.next_tile = h->counters + k;
        FR_CUDA_TRY(fr::gm_launch(fr::k_ce_grad<fr::CeGrad<PAIR, BN>>, tiles, h->sms, s, p, ctl));
    }
    if (gh && rows > 0) {
        // more threads for a row's splits while they leave SMs without a CTA
        int32_t groups = 1;
        int64_t col_ctas = 1;
        while (groups < 16 && 2 * groups <= p.splits && rows * col_ctas < 4 * h->sms) {
            groups *= 2;
            col_ctas = fr::ce_round(h->d, fr::CE_FINISH_THREADS * 4 / groups) / (fr::CE_FINISH_THREADS * 4 / groups);
        }
        const int32_t vec = (reinterpret_cast<uintptr_t>(gh) & 7u) == 0 && (ldgh & 3) == 0;
        if (groups == 1)
            FR_CUDA_TRY(fr::launch_pdl(fr::k_ce_finish, (int64_t)rows, fr::CE_FINISH_THREADS, 0, s, (const float*)h->dh,
                                       p.dh_rows * h->rows.pitch, p.splits, h->d, h->rows, gh, ldgh, vec));
        else
            FR_CUDA_TRY(fr::launch_pdl(fr::k_ce_finish_few, rows * col_ctas, fr::CE_FINISH_THREADS, 0, s, (const float*)h->dh,
                                       p.dh_rows * h->rows.pitch, p.splits, groups, (int32_t)col_ctas, h->d, h->rows, gh,
                                       ldgh, vec));
    }
    return FR_OK;
}

}  // namespace

extern "C" fr_status fr_ce_init(int32_t V, int32_t d, int32_t max_rows, fr_ce** out) {
    if (!out) return FR_ERR_INVALID_ARG;
    *out = nullptr;
    if (V < 1 || d < 1 || d > (1 << 20) || max_rows < 1 || max_rows > (1 << 24) || V > (1 << 24) ||
        (int64_t)max_rows * V > ((int64_t)1 << 44))
        return FR_ERR_INVALID_ARG;
    fr_ce* h = new (std::nothrow) fr_ce();
    if (!h) return FR_ERR_OOM;
    h->V = V;
    h->d = d;
    h->max_rows = max_rows;
    h->cap = fr::ce_round(max_rows, fr::GM_TILE);
    h->n_tiles = (V + fr::GM_TILE - 1) / fr::GM_TILE;
    h->piece = (int32_t)std::min(std::max<int64_t>(fr::CE_PIECE_MIN, fr::CE_PIECE_BYTES / (2 * h->cap) / fr::GM_TILE * fr::GM_TILE),
                                 fr::ce_round(V, fr::GM_TILE));
    h->g_elems = h->cap * h->piece;
    h->rows.pitch = fr::ce_round(d, 8);
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
        fr::gm_setup(fr::k_ce_loss<fr::CeLoss<true, fr::GM_TILE>>) != cudaSuccess ||
        fr::gm_setup(fr::k_ce_loss<fr::CeLoss<true, 0>>) != cudaSuccess ||
        fr::gm_setup(fr::k_ce_loss<fr::CeLoss<false, 0>>) != cudaSuccess ||
        fr::gm_setup(fr::k_ce_grad<fr::CeGrad<true, fr::GM_TILE>>) != cudaSuccess ||
        fr::gm_setup(fr::k_ce_grad<fr::CeGrad<true, 0>>) != cudaSuccess ||
        fr::gm_setup(fr::k_ce_grad<fr::CeGrad<false, 0>>) != cudaSuccess) {
        (void)cudaGetLastError();
        delete h;
        return FR_ERR_CUDA;
    }
    const size_t cap = (size_t)h->cap, pitch = (size_t)h->rows.pitch;
    const size_t d_tiles = (d + fr::GM_TILE - 1) / fr::GM_TILE;
    // dh partials: one plane of all rows, or, where there are more splits, at most
    // 4 * units / d_tiles tiles (ce_splits) of pairs or single CTAs
    const size_t dh_rows = std::max({cap, 2 * h->sms / d_tiles * fr::GM_TILE, 4 * h->sms / d_tiles * fr::GM_HALF});
    cudaError_t e = cudaMalloc(&h->rows.h, cap * pitch * 2);
    if (e == cudaSuccess) e = cudaMalloc(&h->rows.tgt, cap * 4 * 5 + 8 + ((V + h->piece - 1) / h->piece + 1) * 4);
    h->partials = h->cap * 2 * h->n_tiles + fr::CE_PARTIALS_MORE;
    if (e == cudaSuccess) e = cudaMalloc(&h->partial, (size_t)h->partials * sizeof(float2));
    if (e == cudaSuccess) e = cudaMalloc(&h->g, (size_t)h->g_elems * (h->piece < V ? 2 : 1) * 2);
    if (e == cudaSuccess) e = cudaMalloc(&h->dh, dh_rows * pitch * 4);
    if (e == cudaSuccess) e = fr::new_status_word(&h->err);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        ce_free(h);
        return e == cudaErrorMemoryAllocation ? FR_ERR_OOM : FR_ERR_CUDA;
    }
    h->rows.lse = reinterpret_cast<float*>(h->rows.tgt + cap);
    h->rows.g = h->rows.lse + cap;
    h->xt = h->rows.g + cap;
    h->rows.idx = reinterpret_cast<int32_t*>(h->xt + cap);
    h->rows.n = h->rows.idx + cap;
    h->rows.gscale = reinterpret_cast<float*>(h->rows.n + 1);
    h->counters = h->rows.n + 2;
    *out = h;
    return FR_OK;
}

extern "C" fr_status fr_ce_loss(fr_ce* h, const void* hidden_dev, int64_t ldh, const void* weight_dev, int64_t ldw,
                                const int32_t* targets_dev, int32_t rows, float* loss_dev, float* lse_dev,
                                fr_stream stream) {
    if (ce_bad_inputs(h, hidden_dev, ldh, weight_dev, ldw, targets_dev, rows, lse_dev) || !loss_dev ||
        (reinterpret_cast<uintptr_t>(loss_dev) & 3u) || !ce_on_device(h))
        return FR_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    h->last_stream = s;
    if (rows == 0) return FR_OK;
    int32_t bn = ce_width(h, rows, 32);
    if ((int64_t)rows * 2 * ((h->V + bn - 1) / bn) > h->partials) bn = fr::GM_TILE;
    const auto run = rows <= fr::GM_HALF ? ce_run_loss<false, 0> : bn == fr::GM_TILE ? ce_run_loss<true, fr::GM_TILE> : ce_run_loss<true, 0>;
    return run(h, bn, hidden_dev, ldh, weight_dev, ldw, targets_dev, rows, loss_dev, lse_dev, s);
}

extern "C" fr_status fr_ce_grad(fr_ce* h, const void* hidden_dev, int64_t ldh, const void* weight_dev, int64_t ldw,
                                const int32_t* targets_dev, const float* lse_dev, const float* grad_loss_dev,
                                int32_t rows, void* grad_hidden_dev, int64_t ldgh, void* grad_weight_dev, int64_t ldgw,
                                fr_stream stream) {
    if (ce_bad_inputs(h, hidden_dev, ldh, weight_dev, ldw, targets_dev, rows, lse_dev) || !grad_loss_dev ||
        (reinterpret_cast<uintptr_t>(grad_loss_dev) & 3u) || (!grad_hidden_dev && !grad_weight_dev) ||
        (grad_hidden_dev && (ldgh < h->d || (reinterpret_cast<uintptr_t>(grad_hidden_dev) & 1u))) ||
        (grad_weight_dev && (ldgw < h->d || (reinterpret_cast<uintptr_t>(grad_weight_dev) & 1u))) ||
        !ce_on_device(h))
        return FR_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    h->last_stream = s;
    // as many tokens a piece as these rows leave room for in a buffer
    const int64_t fit = h->g_elems / fr::ce_round(std::max(rows, 1), fr::GM_TILE) / fr::GM_TILE * fr::GM_TILE;
    const int32_t piece = (int32_t)std::min(std::max<int64_t>(fit, h->piece), fr::ce_round(h->V, fr::GM_TILE));
    // (beside products, G tiles of any width leave no unit idle)
    const int32_t bn = piece >= h->V ? ce_width(h, rows, 64) : fr::GM_TILE;
    const auto run = rows <= fr::GM_HALF ? ce_run_grad<false, 0> : bn == fr::GM_TILE ? ce_run_grad<true, fr::GM_TILE> : ce_run_grad<true, 0>;
    return run(h, piece, bn, hidden_dev, ldh, weight_dev, ldw, targets_dev, lse_dev, grad_loss_dev, rows, grad_hidden_dev, ldgh,
               grad_weight_dev, ldgw, s);
}

extern "C" fr_status fr_ce_status(fr_ce* h) {
    if (!h) return FR_ERR_INVALID_ARG;
    FR_CUDA_TRY(cudaStreamSynchronize(h->last_stream));
    int32_t err = 0;
    FR_CUDA_TRY(cudaMemcpy(&err, h->err, sizeof(int32_t), cudaMemcpyDeviceToHost));
    return (fr_status)err;
}

extern "C" fr_status fr_ce_clear_status(fr_ce* h, fr_stream stream) {
    if (!h) return FR_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    FR_CUDA_TRY(cudaMemsetAsync(h->err, 0, sizeof(int32_t), s));
    h->last_stream = s;
    return FR_OK;
}

extern "C" fr_status fr_ce_set_wait_test(fr_ce* h, uint64_t wait_limit_ns, int32_t starve_copies) {
    if (!h || (wait_limit_ns != 0 && (wait_limit_ns < 1000ull || wait_limit_ns > 60000000000ull)) ||
        (starve_copies != 0 && starve_copies != 1))
        return FR_ERR_INVALID_ARG;
    h->wait_ns = wait_limit_ns ? wait_limit_ns : FR_WAIT_LIMIT_NS;
    h->starve = starve_copies;
    return FR_OK;
}

extern "C" void fr_ce_destroy(fr_ce* h) {
    if (!h) return;
    ce_free(h);
}
