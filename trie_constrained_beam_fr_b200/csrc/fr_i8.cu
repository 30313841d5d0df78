// fr_i8.cu -- the lm_head product in 8-bit integers with a scale for each
// token and each output channel.
//
//   scale_r = max_j |x_rj| / 127,  q_rj = rne(x_rj / scale_r)
//   y_rn    = (sum_j q_rj w_nj) * scale_r * wscale_n
//
// The sums are int32 (exact: d <= 131,071), so only the two products by the
// scales round.  The row and channel scales factor out of the sum, which is
// why the whole product runs on integers.
//
//   k_i8_quantize  a warp or a CTA per row: maximum, then values, held in registers.
//   k_i8_few       one or two tokens of long rows: a stream over the weight (__dp4a).
//   k_i8<I8Out>    tcgen05 kind::i8 tiles of up to 256 rows x 256 channels; the
//                  epilogue scales and writes logits (bf16 or fp32).
//   k_i8<I8Lse>    the same product whose epilogue reduces each row to
//                  (max, scaled sum) partials and writes the SID slice, for
//                  the step from rows; k_i8_combine merges the partials.
#include <cuda.h>
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

// q of one value: the quotient x / scale (IEEE) rounded to nearest even.  x times
// the reciprocal is within 2^-15 of the quotient (two roundings of a value of at
// most 128), so it rounds to the same integer unless it lies that near a half;
// only then is the division carried out (28 -> 22 us on 8,192 x 2,048 values with
// a warp per row).
// A row whose scale is zero or not finite quantises to zeros (a scale that is not
// finite makes every product of the row NaN or infinite).
__device__ __forceinline__ int32_t i8_quant(float x, float scale, float inv, bool live) {
    const float t = x * inv, r = rintf(t);
    float q = r;
    if (!(fabsf(fabsf(t - r) - 0.5f) > 0x1p-14f)) q = rintf(__fdiv_rn(x, scale));
    return live ? __float2int_rn(fminf(fmaxf(q, -127.f), 127.f)) : 0;
}

__device__ __forceinline__ void i8_load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void i8_load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ float i8_load1(const float* p) { return *p; }
__device__ __forceinline__ float i8_load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// TPR threads per row: a warp for short rows, else a CTA of 128 (8,192 rows of 521
// bf16 values: 8.6 us a warp each, 10.2 a CTA each; of 2,048 values: 21.9 and 17.9).
// VEC: rows start on 16 bytes (x) and 8 bytes (q), so 8 values move at once.
constexpr int QT_SHORT = 1024;
template <class T, bool VEC, int TPR>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR)
    k_i8_quantize(const T* __restrict__ x, int64_t ldx, int32_t rows, int32_t d, int8_t* __restrict__ q, int64_t ldq,
                  float* __restrict__ scale) {
    constexpr int HELD = 4;  // groups of 8 values that a thread keeps between the two passes
    __shared__ uint32_t max_s[4];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x % TPR;
    const int64_t r = (int64_t)blockIdx.x * (blockDim.x / TPR) + threadIdx.x / TPR;
    if (r >= rows) return;  // (whole warps, or nobody)
    const T* xr = x + r * ldx;
    int8_t* qr = q + r * ldq;
    const int32_t groups = VEC ? d >> 3 : 0, rest = groups << 3;
    float held[HELD][8];
    // absolute values order as their bits, a NaN above infinity
    uint32_t m = 0u;
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
        const int32_t g = k * TPR + tid;
        if (VEC && g < groups) i8_load8(xr + 8 * (int64_t)g, held[k]);
    }
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
        if (VEC && k * TPR + tid < groups) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(held[k][i]) & 0x7FFFFFFFu);
        }
    }
#pragma unroll 4
    for (int32_t g = HELD * TPR + tid; VEC && g < groups; g += TPR) {
        float v[8];
        i8_load8(xr + 8 * (int64_t)g, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
#pragma unroll 4
    for (int32_t j = rest + tid; j < d; j += TPR) m = max(m, __float_as_uint(i8_load1(xr + j)) & 0x7FFFFFFFu);
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (TPR != 32) {
        if ((tid & 31) == 0) max_s[tid >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) m = max(m, max_s[w]);
    }
    const float s = __fdiv_rn(__uint_as_float(m), 127.f);
    const bool live = s > 0.f && isfinite(s);
    const float inv = s > 0x1p-120f ? __frcp_rn(s) : NAN;  // NaN: every value divides
    const auto put8 = [&](int32_t g, const float (&v)[8]) {
        uint32_t lo = 0u, hi = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo |= (uint32_t)(i8_quant(v[i], s, inv, live) & 0xFF) << (8 * i);
            hi |= (uint32_t)(i8_quant(v[4 + i], s, inv, live) & 0xFF) << (8 * i);
        }
        *reinterpret_cast<uint2*>(qr + 8 * (int64_t)g) = make_uint2(lo, hi);
    };
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
        const int32_t g = k * TPR + tid;
        if (VEC && g < groups) put8(g, held[k]);
    }
    for (int32_t g = HELD * TPR + tid; VEC && g < groups; g += TPR) {
        float v[8];
        i8_load8(xr + 8 * (int64_t)g, v);
        put8(g, v);
    }
#pragma unroll 4
    for (int32_t j = rest + tid; j < d; j += TPR) qr[j] = (int8_t)i8_quant(i8_load1(xr + j), s, inv, live);
    if (tid == 0) scale[r] = s;
}

// The product for one or two tokens of long rows: bound by the weight's bytes, which
// go straight to registers (16 bytes a lane, 4 channels x 2,048 values per warp in
// flight); the tokens lie in shared memory (zeros behind d), __dp4a multiplies and
// one warp reduction per value adds the lanes.  A warp takes 4 channels at a time,
// so the channels spread evenly over the SMs.  151,936 channels x 2,048 values:
// 50 and 51 us for 1 and 2 tokens (6.2 TB/s) where the tiles take 60.  On the other
// side, 4 tokens of 2,048 values: 60 and 62 (__dp4a begins to bind; of 1,536 values 50
// and 45); one token of 1,536 values: 44 and 44, of 700: 39 and 29 (too few loads in
// flight at a row's end).
constexpr int FEW_ROWS = 2;
constexpr int FEW_LEAST = 1537;  // least d
constexpr int FEW_THREADS = 256;
constexpr int FEW_CH = 4;
constexpr int FEW_STEPS = 4;
constexpr int FEW_SMEM = 64 * 1024;  // most bytes of tokens

// 16 bytes of the weight, read once.
__device__ __forceinline__ int4 few_load(const int8_t* p) {
    int4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <int R, class T>
__global__ void __launch_bounds__(FEW_THREADS) k_i8_few(const int8_t* __restrict__ xq, int64_t ldx,
                                                        const float* __restrict__ xs, const int8_t* __restrict__ wq,
                                                        int64_t ldw, const float* __restrict__ ws, int32_t N, int32_t d,
                                                        T* __restrict__ out, int64_t ldo) {
    extern __shared__ __align__(16) int8_t few_x[];  // [R][pitch]
    const int32_t pieces = (d + 15) >> 4, pitch = pieces << 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();
    griddep_launch_dependents();
    for (int32_t i = threadIdx.x; i < R * pieces; i += FEW_THREADS) {
        const int32_t r = i / pieces, k = (i - r * pieces) << 4;
        const int8_t* src = xq + r * ldx + k;
        int4 v = make_int4(0, 0, 0, 0);
        if (k + 16 <= d) {
            v = *reinterpret_cast<const int4*>(src);
        } else {
            int8_t* b = reinterpret_cast<int8_t*>(&v);
            for (int j = 0; j < d - k; ++j) b[j] = src[j];
        }
        *reinterpret_cast<int4*>(few_x + r * pitch + k) = v;
    }
    __syncthreads();
    const int32_t groups = (N + FEW_CH - 1) / FEW_CH;
    for (int32_t g = blockIdx.x * (FEW_THREADS / 32) + warp; g < groups; g += gridDim.x * (FEW_THREADS / 32)) {
        const int32_t n0 = g * FEW_CH;
        int32_t acc[FEW_CH][R];
#pragma unroll
        for (int c = 0; c < FEW_CH; ++c)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[c][r] = 0;
        const int8_t* src[FEW_CH];
#pragma unroll
        for (int c = 0; c < FEW_CH; ++c) src[c] = wq + min(n0 + c, N - 1) * ldw;
        const auto add = [&](const int4 (&w)[FEW_CH], int32_t k) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int4 x = *reinterpret_cast<const int4*>(few_x + r * pitch + k);
#pragma unroll
                for (int c = 0; c < FEW_CH; ++c) {
                    acc[c][r] = __dp4a(w[c].x, x.x, acc[c][r]);
                    acc[c][r] = __dp4a(w[c].y, x.y, acc[c][r]);
                    acc[c][r] = __dp4a(w[c].z, x.z, acc[c][r]);
                    acc[c][r] = __dp4a(w[c].w, x.w, acc[c][r]);
                }
            }
        };
        // FEW_STEPS x 512 values at a time, all their loads in flight; then what is
        // left in one go.  A row's last piece may reach into its padding (the tokens
        // hold zeros there), but not behind the last row.
        int32_t k = lane << 4;
        for (; k - (lane << 4) + FEW_STEPS * 512 <= d; k += FEW_STEPS * 512) {
            int4 w[FEW_STEPS][FEW_CH];
#pragma unroll
            for (int u = 0; u < FEW_STEPS; ++u)
#pragma unroll
                for (int c = 0; c < FEW_CH; ++c) w[u][c] = few_load(src[c] + k + u * 512);
#pragma unroll
            for (int u = 0; u < FEW_STEPS; ++u) add(w[u], k + u * 512);
        }
        const bool last_row = n0 + FEW_CH >= N && d < pitch;
        if (k - (lane << 4) < d) {
            int4 w[FEW_STEPS][FEW_CH];
#pragma unroll
            for (int u = 0; u < FEW_STEPS; ++u)
#pragma unroll
                for (int c = 0; c < FEW_CH; ++c) {
                    w[u][c] = make_int4(0, 0, 0, 0);
                    if (k + u * 512 < (last_row ? d & ~15 : pitch)) w[u][c] = few_load(src[c] + k + u * 512);
                }
#pragma unroll
            for (int u = 0; u < FEW_STEPS; ++u)
                if (k + u * 512 < pitch) add(w[u], k + u * 512);
        }
        if (last_row && lane == 0) {
            int4 w[FEW_CH];
#pragma unroll
            for (int c = 0; c < FEW_CH; ++c) {
                w[c] = make_int4(0, 0, 0, 0);
                int8_t* b = reinterpret_cast<int8_t*>(&w[c]);
#pragma unroll
                for (int j = 0; j < 15; ++j)
                    if ((d & ~15) + j < d) b[j] = src[c][(d & ~15) + j];
            }
            add(w, d & ~15);
        }
        int32_t mine = 0;  // lane r * FEW_CH + c keeps token r's channel c
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < FEW_CH; ++c) {
                const int32_t sum = __reduce_add_sync(0xffffffffu, acc[c][r]);
                if (lane == r * FEW_CH + c) mine = sum;
            }
        const int32_t r = lane / FEW_CH, n = n0 + lane % FEW_CH;
        if (r < R && n < N) {
            const float y = (float)mine * xs[r] * __ldg(ws + n);
            if constexpr (sizeof(T) == 4)
                out[r * ldo + n] = y;
            else
                out[r * ldo + n] = __float2bfloat16_rn(y);
        }
    }
}

constexpr int64_t I8_PARTIALS_MORE = 1 << 16;  // for narrow tiles of small calls

// Tile walk shared by the two products.  BN: columns of a tile, known to the compiler
// (256) or not (0).
template <bool PAIR_, int BN>
struct I8Base {
    static constexpr bool I8 = true, DYNAMIC = false, PAIR = PAIR_;
    static constexpr int TM = PAIR ? GM_TILE : GM_HALF;  // rows of a tile
    __device__ __forceinline__ int32_t* counter() const { return nullptr; }
    struct Tile {
        int nk, m0, n, n0;
        uint32_t idesc;
    };
    struct State {};
    CUtensorMap map_x, map_w;
    __device__ __forceinline__ void prefetch() const {
        gm_prefetch(&map_x);
        gm_prefetch(&map_w);
    }
    int32_t rows, N, k_blocks, m_tiles, n_tiles;
    int32_t narrow_bn;      // columns of a tile where BN is 0
    int32_t single_a_rows;  // rows of a single CTA's copy of x
    __device__ __forceinline__ int bn() const { return BN ? BN : narrow_bn; }
    __device__ __forceinline__ int a_rows() const { return PAIR ? GM_HALF : single_a_rows; }
    const float* xs;
    const float* ws;
    int32_t ws_vec;  // ws starts on 16 bytes
    int32_t small;   // |sums| <= 2^22 (d <= 256)

    __device__ __forceinline__ State begin() const { return {}; }
    __device__ __forceinline__ bool tile(const State&, uint32_t g, Tile& t) const {
        if (g >= (uint32_t)m_tiles * (uint32_t)n_tiles) return false;
        int32_t m, n;
        gm_grouped(g, m_tiles, n_tiles, m, n);
        t.m0 = m * TM;
        t.n = n;
        t.n0 = n * bn();
        t.nk = k_blocks;
        t.idesc = gm_idesc(true, PAIR, false, false, bn());
        return true;
    }
    __device__ __forceinline__ uint32_t stage_bytes(const Tile&) const { return ((PAIR ? 2 : 1) * a_rows() + bn()) * GM_KB_BYTES; }
    __device__ __forceinline__ bool a_mn(const Tile&) const { return false; }
    __device__ __forceinline__ bool b_mn(const Tile&) const { return false; }
    __device__ __forceinline__ void load(const Tile& t, int kb, int rank, uint8_t* a, uint8_t* b, uint32_t bar) const {
        gm_tma_load<PAIR>(&map_x, a, bar, kb * GM_KB_BYTES, t.m0 + rank * GM_HALF);
        // a box is half a tile's columns: the CTA's, or both
        gm_tma_load<PAIR>(&map_w, b, bar, kb * GM_KB_BYTES, t.n0 + rank * (bn() / 2));
        if constexpr (!PAIR) gm_tma_load<PAIR>(&map_w, b + bn() / 2 * GM_KB_BYTES, bar, kb * GM_KB_BYTES, t.n0 + bn() / 2);
    }
    // y of CW columns from n on: the row's scale first, then the channel's
    template <int CW>
    __device__ __forceinline__ void scaled(uint32_t taddr, int n, float xscale, float (&v)[CW], bool last,
                                           GmRelease<PAIR>& release) const {
        float4 w[CW / 4];  // loaded before the accumulator is waited for
        if (ws_vec && n + CW <= N) {
#pragma unroll
            for (int i = 0; i < CW / 4; ++i) w[i] = __ldg(reinterpret_cast<const float4*>(ws + n) + i);
        } else {
#pragma unroll
            for (int i = 0; i < CW; ++i) (&w[i / 4].x)[i % 4] = n + i < N ? __ldg(ws + n + i) : 0.f;
        }
        if constexpr (CW == 64)
            gm_ld64(taddr, v);
        else
            tc_tmem_ld32(taddr, v);
        if (last) release();
        if (small) {
            // sums up to 2^22 become fp32 by 1.5 * 2^23 and its subtraction (exact): the
            // conversion instruction runs at the exponential's quarter rate, which
            // shows where few K stages hide it
#pragma unroll
            for (int i = 0; i < CW; ++i)
                v[i] = (__int_as_float(__float_as_int(v[i]) + 0x4B400000) - 12582912.f) * xscale * (&w[i / 4].x)[i % 4];
        } else {
#pragma unroll
            for (int i = 0; i < CW; ++i) v[i] = (float)__float_as_int(v[i]) * xscale * (&w[i / 4].x)[i % 4];
        }
    }
};

template <class T, bool PAIR_, int BN>
struct I8Out : I8Base<PAIR_, BN> {
    using Base = I8Base<PAIR_, BN>;
    using typename Base::State;
    using typename Base::Tile;
    using Base::bn;
    using Base::N;
    using Base::rows;
    using Base::xs;
    using Base::scaled;
    static constexpr bool STAGED = true;
    static constexpr int STAGES = PAIR_ ? 6 : 4;
    CUtensorMap map_out;
    T* out;
    int64_t ldo;
    // Columns below `staged` go out through shared memory and TMA: none unless
    // rows start on 16 bytes; all when rows are whole 16-byte pieces, else the
    // whole groups of columns (a clipped TMA store fills its last 16 bytes).
    int32_t staged;
    __device__ __forceinline__ void epilogue(const State&, const Tile& t, uint32_t taddr, int r, int half, const GmStage& sg,
                                             GmRelease<PAIR_>& release) const {
        constexpr int CW = 128 / sizeof(T);  // columns per staged store
        const int row = t.m0 + r, lane = threadIdx.x & 31, row0 = row - lane;
        const int cols = (bn() / 2 + CW - 1) / CW * CW, c1 = min((half + 1) * cols, bn());
        if (row0 >= rows) return;
        const float xscale = row < rows ? xs[row] : 0.f;
#pragma unroll 1
        for (int c = half * cols; c < c1 && t.n0 + c < N; c += CW) {
            float v[CW];
            scaled(taddr + (uint32_t)c, t.n0 + c, xscale, v, c + CW == c1, release);
            gm_put(sg, lane, v);
            if (t.n0 + c < staged)
                sg.send<false>(&map_out, lane, t.n0 + c, row0);
            else
                gm_write_plain(sg, lane, out + row0 * ldo + t.n0 + c, ldo, min(32, rows - row0), min(CW, N - t.n0 - c));
        }
    }
};

template <bool PAIR_, int BN>
struct I8Lse : I8Base<PAIR_, BN> {
    using Base = I8Base<PAIR_, BN>;
    using typename Base::State;
    using typename Base::Tile;
    using Base::bn;
    using Base::N;
    using Base::rows;
    using Base::xs;
    using Base::scaled;
    static constexpr bool STAGED = true;
    static constexpr int STAGES = PAIR_ ? 6 : 4;
    float2* partial;  // [rows, n_parts] (max, scaled sum) of half a tile's columns each
    int32_t n_parts;
    float* slice;     // [rows, sid_span]
    int32_t sid_base, sid_span;
    __device__ __forceinline__ void epilogue(const State&, const Tile& t, uint32_t taddr, int r, int half, const GmStage& sg,
                                             GmRelease<PAIR_>& release) const {
        const int cols = (bn() / 2 + 31) & ~31, c1 = min((half + 1) * cols, bn());
        const int row = t.m0 + r, lane = threadIdx.x & 31, row0 = row - lane;
        if (row0 >= rows) return;
        const float xscale = row < rows ? xs[row] : 0.f;
        float m = -INFINITY, s = 0.f;
#pragma unroll 1
        for (int c = half * cols; c < c1 && t.n0 + c < N; c += 32) {
            const int n = t.n0 + c;
            float v[32];
            scaled(taddr + (uint32_t)c, n, xscale, v, c + 32 == c1, release);
            // the slice's columns of this chunk, a row at a time (a lane's stores to
            // its own row took 267 us instead of 117 on 5,555 rows x 4,757 slice columns)
            const int lo = max(n, sid_base), hi = min(n + 32, sid_base + sid_span);
            if (lo < hi) {
                gm_put(sg, lane, v);
                gm_write_plain(sg, lane, slice + (int64_t)row0 * sid_span - sid_base + n, sid_span, min(32, rows - row0), hi - n,
                               lo - n);
            }
            if (n + 32 > N) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (n + i >= N) v[i] = -INFINITY;
            }
            gm_lse_fold(v, m, s);
        }
        if (row < rows) partial[(int64_t)row * n_parts + 2 * t.n + half] = make_float2(m, s);
    }
};

template <class P>
__global__ void __launch_bounds__(GM_THREADS, 1) k_i8(const __grid_constant__ P p, const GmCtl ctl) {
    gm_run(p, ctl);
}

__global__ void __launch_bounds__(256) k_i8_combine(const float2* __restrict__ partial, int32_t rows, int32_t n_parts,
                                                    float* __restrict__ lse, int32_t* __restrict__ err) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    const float v = gm_lse_combine(partial + r * n_parts, n_parts);
    if ((threadIdx.x & 31) == 0) {
        if (!isfinite(v)) set_error(err, FR_ERR_NAN_LOGIT);
        lse[r] = v;
    }
}

}  // namespace
}  // namespace fr

struct fr_i8 {
    const int8_t* wq = nullptr;
    const float* ws = nullptr;
    int64_t ldw = 0;
    int32_t N = 0, d = 0, max_rows = 0, sid_base = 0, sid_span = 0, sms = 0, device = 0;
    float2* partial = nullptr;  // partials values: at least [max_rows, 2 * (tiles of 256 columns)]
    int64_t partials = 0;
    int32_t* err = nullptr;
    cudaStream_t last_stream = nullptr;
    uint64_t wait_ns = FR_WAIT_LIMIT_NS;
    int32_t starve = 0;
};

namespace {

bool i8_on_device(const fr_i8* h) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == h->device;
}

template <bool PAIR, int BN>
fr_status i8_base(fr_i8* h, const int8_t* xq, int64_t ldx, const float* xs, int32_t rows, int32_t bn, fr::I8Base<PAIR, BN>* b) {
    constexpr int TM = fr::I8Base<PAIR, BN>::TM;
    b->single_a_rows = fr::gm_a_rows(rows);
    if (!fr::gm_encode(&b->map_x, 1, xq, rows, h->d, ldx, PAIR ? fr::GM_HALF : b->single_a_rows) ||
        !fr::gm_encode(&b->map_w, 1, h->wq, h->N, h->d, h->ldw, bn / 2))
        return FR_ERR_CUDA;
    b->narrow_bn = bn;
    b->rows = rows;
    b->N = h->N;
    b->k_blocks = (h->d + fr::GM_KB_BYTES - 1) / fr::GM_KB_BYTES;
    b->m_tiles = (rows + TM - 1) / TM;
    b->n_tiles = (h->N + bn - 1) / bn;
    b->xs = xs;
    b->ws = h->ws;
    b->small = h->d <= 256;  // 128 * 128 * 256 = 2^22
    b->ws_vec = (reinterpret_cast<uintptr_t>(h->ws) & 15u) == 0;
    return FR_OK;
}

// Tile width of a call.
int32_t i8_width(const fr_i8* h, int32_t rows, int32_t step) {
    if (rows <= fr::GM_HALF) return fr::gm_width(1, h->N, h->sms, step);
    return fr::gm_width((rows + fr::GM_TILE - 1) / fr::GM_TILE, h->N, h->sms / 2, step);
}

template <class P>
fr_status i8_launch(fr_i8* h, const P& p, cudaStream_t s) {
    fr::GmCtl ctl{h->err, h->wait_ns, h->starve};
    FR_CUDA_TRY(fr::gm_launch(fr::k_i8<P>, (int64_t)p.m_tiles * p.n_tiles, h->sms, s, p, ctl));
    return FR_OK;
}

template <class T, bool PAIR, int BN>
fr_status i8_tiles(fr_i8* h, int32_t bn, const int8_t* xq, int64_t ldx, const float* xs, int32_t rows, void* out, int64_t ldo,
                   cudaStream_t s) {
    fr::I8Out<T, PAIR, BN> p{};
    const fr_status st = i8_base<PAIR, BN>(h, xq, ldx, xs, rows, bn, &p);
    if (st != FR_OK) return st;
    p.out = (T*)out;
    p.ldo = ldo;
    if ((reinterpret_cast<uintptr_t>(out) & 15u) == 0 && (ldo * sizeof(T)) % 16 == 0)
        p.staged = fr::gm_staged_columns(h->N, sizeof(T));
    if (p.staged && !fr::gm_encode(&p.map_out, sizeof(T), out, rows, h->N, ldo * sizeof(T), 32)) return FR_ERR_CUDA;
    return i8_launch(h, p, s);
}

template <class T>
fr_status i8_out(fr_i8* h, const int8_t* xq, int64_t ldx, const float* xs, int32_t rows, void* out, int64_t ldo,
                 cudaStream_t s) {
    if (rows <= fr::FEW_ROWS && h->d >= fr::FEW_LEAST) {
        // as long as the tokens fit into shared memory
        const size_t smem = (size_t)rows * ((h->d + 15) / 16 * 16);
        if (smem <= (size_t)fr::FEW_SMEM) {
            auto k = rows == 1 ? fr::k_i8_few<1, T> : fr::k_i8_few<2, T>;
            const int64_t groups = (h->N + fr::FEW_CH - 1) / fr::FEW_CH, warps = fr::FEW_THREADS / 32;
            FR_CUDA_TRY(fr::launch_pdl(k, std::min<int64_t>((groups + warps - 1) / warps, 3 * (int64_t)h->sms), fr::FEW_THREADS,
                                       smem, s, xq, ldx, xs, h->wq, h->ldw, h->ws, h->N, h->d, (T*)out, ldo));
            return FR_OK;
        }
    }
    const int32_t bn = i8_width(h, rows, 128 / sizeof(T));  // (whole staged stores)
    const auto run = rows <= fr::GM_HALF ? i8_tiles<T, false, 0> : bn == fr::GM_TILE ? i8_tiles<T, true, fr::GM_TILE> : i8_tiles<T, true, 0>;
    return run(h, bn, xq, ldx, xs, rows, out, ldo, s);
}

template <bool PAIR, int BN>
fr_status i8_rows_lse(fr_i8* h, int32_t bn, const int8_t* xq, int64_t ldx, const float* xs, int32_t rows, float* lse, float* slice,
                      cudaStream_t s) {
    fr::I8Lse<PAIR, BN> p{};
    const fr_status st = i8_base<PAIR, BN>(h, xq, ldx, xs, rows, bn, &p);
    if (st != FR_OK) return st;
    p.partial = h->partial;
    p.n_parts = 2 * p.n_tiles;
    p.slice = slice;
    p.sid_base = h->sid_base;
    p.sid_span = h->sid_span;
    const fr_status run = i8_launch(h, p, s);
    if (run != FR_OK) return run;
    FR_CUDA_TRY(fr::launch_pdl(fr::k_i8_combine, ((int64_t)rows + 7) / 8, 256, 0, s, (const float2*)h->partial, rows, p.n_parts,
                               lse, h->err));
    return FR_OK;
}

template <class T>
cudaError_t i8_setup_few() {
    for (auto k : {fr::k_i8_few<1, T>, fr::k_i8_few<2, T>}) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, fr::FEW_SMEM);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <bool PAIR, int BN>
cudaError_t i8_setup_tiles() {
    cudaError_t e = fr::gm_setup(fr::k_i8<fr::I8Out<float, PAIR, BN>>);
    if (e == cudaSuccess) e = fr::gm_setup(fr::k_i8<fr::I8Out<__nv_bfloat16, PAIR, BN>>);
    if (e == cudaSuccess) e = fr::gm_setup(fr::k_i8<fr::I8Lse<PAIR, BN>>);
    return e;
}

template <class T, bool VEC>
cudaError_t i8_quantize(const void* x, int64_t ldx, int32_t rows, int32_t d, int8_t* q, int64_t ldq, float* scale,
                        cudaStream_t s) {
    if (d <= fr::QT_SHORT)
        return fr::launch_pdl(fr::k_i8_quantize<T, VEC, 32>, ((int64_t)rows + 7) / 8, 256, 0, s, (const T*)x, ldx, rows, d, q,
                              ldq, scale);
    return fr::launch_pdl(fr::k_i8_quantize<T, VEC, 128>, rows, 128, 0, s, (const T*)x, ldx, rows, d, q, ldq, scale);
}

bool i8_bad_x(const fr_i8* h, const int8_t* xq, int64_t ldx, const float* xs, int32_t rows) {
    return !h || !xq || !xs || rows < 0 || rows > h->max_rows || ldx < h->d || (ldx & 15) ||
           (reinterpret_cast<uintptr_t>(xq) & 15u) || (reinterpret_cast<uintptr_t>(xs) & 3u);
}

}  // namespace

extern "C" fr_status fr_i8_quantize(const void* x_dev, int64_t ldx, fr_dtype dtype, int32_t rows, int32_t d,
                                    int8_t* q_dev, int64_t ldq, float* scale_dev, fr_stream stream) {
    if (!x_dev || !q_dev || !scale_dev || rows < 0 || d < 1 || d > (1 << 30) || ldx < d || ldq < d ||
        (dtype != FR_F32 && dtype != FR_BF16) ||
        (reinterpret_cast<uintptr_t>(x_dev) & (dtype == FR_F32 ? 3u : 1u)) ||
        (reinterpret_cast<uintptr_t>(scale_dev) & 3u))
        return FR_ERR_INVALID_ARG;
    if (rows == 0) return FR_OK;
    const cudaStream_t s = (cudaStream_t)stream;
    const uintptr_t bytes = reinterpret_cast<uintptr_t>(x_dev) | (uintptr_t)(ldx * (dtype == FR_F32 ? 4 : 2));
    const bool vec = bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(q_dev) | (uintptr_t)ldq) % 8 == 0;
    const auto run = dtype == FR_F32 ? (vec ? i8_quantize<float, true> : i8_quantize<float, false>)
                                     : (vec ? i8_quantize<__nv_bfloat16, true> : i8_quantize<__nv_bfloat16, false>);
    FR_CUDA_TRY(run(x_dev, ldx, rows, d, q_dev, ldq, scale_dev, s));
    return FR_OK;
}

extern "C" fr_status fr_i8_init(const int8_t* weight_dev, int64_t ldw, const float* wscale_dev, int32_t N, int32_t d,
                                int32_t max_rows, int32_t sid_base, int32_t sid_span, fr_i8** out) {
    if (!out) return FR_ERR_INVALID_ARG;
    *out = nullptr;
    if (!weight_dev || !wscale_dev || N < 1 || d < 1 || d > 131071 || ldw < d || max_rows < 1 || sid_base < 0 ||
        sid_span < 0 || (int64_t)sid_base + sid_span > N || max_rows > (1 << 24) || N > (1 << 24) ||
        (int64_t)max_rows * N > ((int64_t)1 << 44))
        return FR_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(weight_dev) & 15u) || (ldw & 15) || (reinterpret_cast<uintptr_t>(wscale_dev) & 3u))
        return FR_ERR_INVALID_ARG;
    fr_i8* h = new (std::nothrow) fr_i8();
    if (!h) return FR_ERR_OOM;
    h->wq = weight_dev;
    h->ws = wscale_dev;
    h->ldw = ldw;
    h->N = N;
    h->d = d;
    h->max_rows = max_rows;
    h->sid_base = sid_base;
    h->sid_span = sid_span;
    h->partials = (int64_t)max_rows * 2 * ((N + fr::GM_TILE - 1) / fr::GM_TILE) + fr::I8_PARTIALS_MORE;
    CUtensorMap map;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
        !fr::gm_encode(&map, 1, weight_dev, N, d, ldw, fr::GM_HALF) ||
        i8_setup_few<float>() != cudaSuccess || i8_setup_few<__nv_bfloat16>() != cudaSuccess ||
        i8_setup_tiles<true, fr::GM_TILE>() != cudaSuccess || i8_setup_tiles<true, 0>() != cudaSuccess ||
        i8_setup_tiles<false, 0>() != cudaSuccess) {
        (void)cudaGetLastError();
        delete h;
        return FR_ERR_CUDA;
    }
    cudaError_t e = cudaMalloc(&h->partial, sizeof(float2) * (size_t)h->partials);
    if (e == cudaSuccess) e = fr::new_status_word(&h->err);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        cudaFree(h->partial);
        cudaFree(h->err);
        delete h;
        return e == cudaErrorMemoryAllocation ? FR_ERR_OOM : FR_ERR_CUDA;
    }
    *out = h;
    return FR_OK;
}

extern "C" fr_status fr_i8_matmul(fr_i8* h, const int8_t* xq_dev, int64_t ldx, const float* xscale_dev, int32_t rows,
                                  void* out_dev, int64_t ldo, fr_dtype out_dtype, fr_stream stream) {
    if (i8_bad_x(h, xq_dev, ldx, xscale_dev, rows) || !out_dev || ldo < h->N ||
        (out_dtype != FR_F32 && out_dtype != FR_BF16))
        return FR_ERR_INVALID_ARG;
    const int esize = out_dtype == FR_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(out_dev) & (esize - 1)) return FR_ERR_INVALID_ARG;
    if (!i8_on_device(h)) return FR_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    h->last_stream = s;
    if (rows == 0) return FR_OK;
    return out_dtype == FR_F32 ? i8_out<float>(h, xq_dev, ldx, xscale_dev, rows, out_dev, ldo, s)
                               : i8_out<__nv_bfloat16>(h, xq_dev, ldx, xscale_dev, rows, out_dev, ldo, s);
}

extern "C" fr_status fr_i8_lse(fr_i8* h, const int8_t* xq_dev, int64_t ldx, const float* xscale_dev, int32_t rows,
                               float* lse_dev, float* slice_dev, fr_stream stream) {
    if (i8_bad_x(h, xq_dev, ldx, xscale_dev, rows) || !lse_dev || (h->sid_span > 0 && !slice_dev) ||
        (reinterpret_cast<uintptr_t>(lse_dev) & 3u) || (reinterpret_cast<uintptr_t>(slice_dev) & 3u))
        return FR_ERR_INVALID_ARG;
    if (!i8_on_device(h)) return FR_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    h->last_stream = s;
    if (rows == 0) return FR_OK;
    int32_t bn = i8_width(h, rows, 32);
    if ((int64_t)rows * 2 * ((h->N + bn - 1) / bn) > h->partials) bn = fr::GM_TILE;
    const auto run = rows <= fr::GM_HALF ? i8_rows_lse<false, 0> : bn == fr::GM_TILE ? i8_rows_lse<true, fr::GM_TILE> : i8_rows_lse<true, 0>;
    return run(h, bn, xq_dev, ldx, xscale_dev, rows, lse_dev, slice_dev, s);
}

extern "C" fr_status fr_i8_status(fr_i8* h) {
    if (!h) return FR_ERR_INVALID_ARG;
    FR_CUDA_TRY(cudaStreamSynchronize(h->last_stream));
    int32_t err = 0;
    FR_CUDA_TRY(cudaMemcpy(&err, h->err, sizeof(int32_t), cudaMemcpyDeviceToHost));
    return (fr_status)err;
}

extern "C" fr_status fr_i8_clear_status(fr_i8* h, fr_stream stream) {
    if (!h) return FR_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    FR_CUDA_TRY(cudaMemsetAsync(h->err, 0, sizeof(int32_t), s));
    h->last_stream = s;
    return FR_OK;
}

extern "C" fr_status fr_i8_set_wait_test(fr_i8* h, uint64_t wait_limit_ns, int32_t starve_copies) {
    if (!h || (wait_limit_ns != 0 && (wait_limit_ns < 1000ull || wait_limit_ns > 60000000000ull)) ||
        (starve_copies != 0 && starve_copies != 1))
        return FR_ERR_INVALID_ARG;
    h->wait_ns = wait_limit_ns ? wait_limit_ns : FR_WAIT_LIMIT_NS;
    h->starve = starve_copies;
    return FR_OK;
}

extern "C" void fr_i8_destroy(fr_i8* h) {
    if (!h) return;
    cudaFree(h->partial);
    cudaFree(h->err);
    delete h;
}
