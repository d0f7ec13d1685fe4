// gm_window.cuh - causal attention with a sliding window and always-visible first tokens
// ("sinks"): what its kernels share, and the fp32 kernels.
//
// Query i of a sequence sees key t <= i iff i - t < window or t < sinks. With
// s(i, t) = scale <q_i, k_t>, P(i, t) = exp(s(i, t) - lse_i), lse_i = ln sum_t exp(s(i, t)):
//   forward   o_i = sum_t P(i, t) v_t
//   backward  delta_i = <dout_i, o_i>,  dS(i, t) = P(i, t) (<dout_i, v_t> - delta_i)
//             dq_i = scale sum_t dS(i, t) k_t,  dk_t = scale sum_i dS(i, t) q_i,
//             dv_t = sum_i P(i, t) dout_i   (dk, dv summed over the query heads of the group)
//
// The keys that a block of query rows [i0, i1) can see are two ranges: the window part
// [lo, i1) with lo = max(0, i0 - window + 1), and the sinks that lie before it,
// [0, min(sinks, lo)). The kernels walk exactly those ranges in key blocks, so the work follows
// the visible pairs and not n^2.
//
// fp32 kernels (this file). Packed FFMA tiles of 16 R rows x 64 columns: 256 threads in a 16 x 16
// grid, each holding an R x 4 piece of the scores and R rows x D/16 columns of the output. Rows
// are queries in the forward and in dq, keys in dk and dv. R = 4 has the fewest shared-memory
// reads per product; R = 2 and 1 make more and shorter blocks where a call would leave SMs idle
// (B=1 n=128, two heads: 125 us with R = 4, 53 us with R = 1, forward and backward).
// Bound by the fp32 pipes; there is no tensor-core type that keeps fp32's 24 bits. The backward
// is two kernels without atomics: one per query block (dq) and one per key block (dk, dv, summed
// over the group's heads in the block), so every gradient is written once, in a fixed order. Key
// blocks with sinks, which every query sees, are cut into pieces of about the other blocks' length
// whose sums a last kernel adds (B=4 n=1000, 4/2 heads, d=128, window 200, 2 sinks: 659 -> 349 us for
// the backward). At a size that fills the GPU, B=8 n=4096, 16/8 heads, d=128, window 512, 4 sinks:
// forward 4.43 ms, backward 13.9 ms, 29 and 33 of the 74 TFLOP/s that the pipes have at 1965 MHz
// (4 d and 14 d operations per visible pair and head).
#pragma once

#include <math.h>

#include "gm_common.cuh"

namespace gm {

// Host code clamps window and sinks to n, so no sum below leaves 32 bits (n < 2^30).
struct WinArgs {
    const void *q, *k, *v;   // [B, n, hq | hkv, D]
    const int32_t *lens;     // [B] tokens of each sequence, or null: n each
    const void *o_in, *dout; // backward
    const float *lse_in;     // backward: [B, n, hq]
    void *o;                 // forward
    float *lse;
    void *dq, *dk, *dv;
    float *delta;            // backward workspace: [B, hq, n] (sum_d dout o)
    int B, n, hq, hkv, G;
    int window, sinks;
    float scale;
    int nblk;                // blocks along the sequence
    int lone;                // backward: the first rows that see one key alone (1, or n with window 1 and no sinks)
    // fp32 dk, dv: the first sink_blocks key blocks are cut into `chunks` pieces of `steps` query tiles,
    // whose sums go to part [piece][dk, dv][rows][D]
    int sink_blocks, chunks, steps;
    float *part;
};

__device__ __forceinline__ int win_len(const WinArgs &a, int b)
{
    return a.lens ? min(max(__ldg(a.lens + b), 0), a.n) : a.n;
}

__device__ __forceinline__ bool win_sees(int i, int t, int window, int sinks)
{
    return t <= i && (i - t < window || t < sinks);
}

// Key blocks of a block of query rows: the sinks before the window first, then the window.
struct KeyBlocks {
    int na, nb;       // blocks of each part
    int lo, hi, aend; // window part [lo, hi), sink part [0, aend)
    __device__ __forceinline__ KeyBlocks(int i0, int rows, int len, int window, int sinks, int bn)
    {
        hi = min(i0 + rows, len);
        lo = max(0, i0 - window + 1);
        aend = min(sinks, lo);
        na = hi > i0 ? (aend + bn - 1) / bn : 0;
        nb = hi > i0 ? (hi - lo + bn - 1) / bn : 0;
    }
    __device__ __forceinline__ int start(int j, int bn) const { return j < na ? j * bn : lo + (j - na) * bn; }
    __device__ __forceinline__ int end(int j, int bn) const
    {
        return j < na ? min(j * bn + bn, aend) : min(lo + (j - na) * bn + bn, hi);
    }
};

// One past the last query that can see a key of [t0, t1).
__device__ __forceinline__ int query_end(int t0, int t1, int len, int window, int sinks)
{
    return t0 < sinks ? len : min(len, t1 - 1 + window);
}

// ---- fp32 tiles -----------------------------------------------------------------------------

constexpr int WT = 64;    // columns of a tile
constexpr int WLP = 68;   // padded row of a score tile, floats

template <int D, int R> struct WinF32 {
    static constexpr int ROWS = 16 * R;
    static constexpr int LD = D + 4;  // padded feature row, floats: rows 4 banks apart
    static constexpr int NC = D / 64; // float4 column groups per thread
    static constexpr size_t fwd_smem = (size_t)((ROWS + 2 * WT) * LD + ROWS * WLP) * 4;
    static constexpr size_t dq_smem = (size_t)((2 * ROWS + 2 * WT) * LD + ROWS * WLP) * 4;
    static constexpr size_t dkv_smem = (size_t)((2 * ROWS + 2 * WT) * LD + 2 * ROWS * WLP) * 4;
};

// Rows [r0, r0 + N) of one head of a [.., heads, D] tensor into a tile; rows at or past `end`
// (padding may hold anything) become zeros.
template <int D, int N>
__device__ __forceinline__ void load_tile(float *dst, const float *src, size_t row_stride, int r0, int end)
{
    constexpr int C = D / 4, PER = (N * C + 255) / 256;
    float4 f[PER];
#pragma unroll
    for (int y = 0; y < PER; ++y) {
        const int x = threadIdx.x + 256 * y, r = x / C, c = x - r * C;
        f[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (x < N * C && r0 + r < end) f[y] = __ldg(reinterpret_cast<const float4 *>(src + (size_t)(r0 + r) * row_stride) + c);
    }
#pragma unroll
    for (int y = 0; y < PER; ++y) {
        const int x = threadIdx.x + 256 * y, r = x / C, c = x - r * C;
        if (x < N * C) *reinterpret_cast<float4 *>(dst + r * (D + 4) + c * 4) = f[y];
    }
}

__device__ __forceinline__ float2 lower(const float4 &f) { return make_float2(f.x, f.y); }
__device__ __forceinline__ float2 upper(const float4 &f) { return make_float2(f.z, f.w); }

// acc[i][j] = <a[row ty*R + i], b[row tx + 16 j]>; even and odd elements sum apart, then together.
template <int D, int R>
__device__ __forceinline__ void tile_dots(const float *a, const float *b, int ty, int tx, float (&acc)[R][4])
{
    constexpr int LD = D + 4;
    float2 s[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 x[R], y[4];
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const float4 *>(a + (ty * R + i) * LD + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * LD + d);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = __ffma2_rn(lower(x[i]), lower(y[j]), s[i][j]);
                s[i][j] = __ffma2_rn(upper(x[i]), upper(y[j]), s[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = s[i][j].x + s[i][j].y;
}

// acc[i][c] += sum_r w[row ty*R + i][r] f[r][tx*4 + 64 c ..+3]
template <int D, int R>
__device__ __forceinline__ void tile_accumulate(const float *w, const float *f, int ty, int tx, float4 (&acc)[R][D / 64])
{
    constexpr int LD = D + 4, NC = D / 64;
#pragma unroll 2
    for (int r = 0; r < WT; r += 4) {
        float4 p[R];
#pragma unroll
        for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4 *>(w + (ty * R + i) * WLP + r);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const float4 y = *reinterpret_cast<const float4 *>(f + (r + e) * LD + tx * 4 + 64 * c);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float pe = (&p[i].x)[e];
                    const float2 lo = __ffma2_rn(make_float2(pe, pe), lower(y), lower(acc[i][c]));
                    const float2 hi = __ffma2_rn(make_float2(pe, pe), upper(y), upper(acc[i][c]));
                    acc[i][c] = make_float4(lo.x, lo.y, hi.x, hi.y);
                }
            }
    }
}

template <int R, int NC> __device__ __forceinline__ void zero(float4 (&acc)[R][NC])
{
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[i][c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}

// Sum / maximum over the 16 threads of a tile row (tx), every one of them gets it.
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
    return x;
}
__device__ __forceinline__ float row_max(float x)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(FULL, x, o));
    return x;
}

// This thread's rows of an output tile, times f; rows at or past n are not written.
template <int D, int R>
__device__ __forceinline__ void store_tile(float *dst, size_t row_stride, int r0, int n, int ty, int tx,
                                           const float4 (&acc)[R][D / 64], const float (&f)[R])
{
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (r0 + ty * R + i < n) {
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                *reinterpret_cast<float4 *>(dst + (size_t)(r0 + ty * R + i) * row_stride + tx * 4 + 64 * c) =
                    make_float4(acc[i][c].x * f[i], acc[i][c].y * f[i], acc[i][c].z * f[i], acc[i][c].w * f[i]);
        }
}

template <int D, int R> __global__ void __launch_bounds__(256) win_fwd_f32_kernel(WinArgs a)
{
    using S = WinF32<D, R>;
    constexpr int NC = S::NC, ROWS = S::ROWS;
    extern __shared__ __align__(16) float wsm[];
    float *sq = wsm, *sk = sq + ROWS * S::LD, *sv = sk + WT * S::LD, *sp = sv + WT * S::LD;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    // the blocks with the longest prefix first
    const int per = a.B * a.hq;
    const int blk = a.nblk - 1 - (int)(blockIdx.x / (unsigned)per);
    const int bh = (int)(blockIdx.x % (unsigned)per);
    const int b = bh / a.hq, hq = bh - b * a.hq, h = hq / a.G;
    const int len = win_len(a, b), i0 = blk * ROWS;
    const size_t qs = (size_t)a.hq * D, ks = (size_t)a.hkv * D;
    const float *q = (const float *)a.q + (size_t)b * a.n * qs + (size_t)hq * D;
    const float *k = (const float *)a.k + (size_t)b * a.n * ks + (size_t)h * D;
    const float *v = (const float *)a.v + (size_t)b * a.n * ks + (size_t)h * D;
    const KeyBlocks kb(i0, ROWS, len, a.window, a.sinks, WT);
    const float sl2 = a.scale * LOG2E;

    load_tile<D, ROWS>(sq, q, qs, i0, len);
    float4 acc[R][NC];
    zero(acc);
    float m[R], l[R];
#pragma unroll
    for (int i = 0; i < R; ++i) m[i] = -INFINITY, l[i] = 0.0f;
    for (int j = 0; j < kb.na + kb.nb; ++j) {
        const int t0 = kb.start(j, WT), t1 = kb.end(j, WT);
        __syncthreads();
        load_tile<D, WT>(sk, k, ks, t0, t1);
        load_tile<D, WT>(sv, v, ks, t0, t1);
        __syncthreads();
        float s[R][4];
        tile_dots<D, R>(sq, sk, ty, tx, s);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int qi = i0 + ty * R + i;
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int t = t0 + tx + 16 * c;
                const bool see = qi < len && t < t1 && win_sees(qi, t, a.window, a.sinks);
                s[i][c] = see ? s[i][c] * sl2 : -INFINITY;
                mx = fmaxf(mx, s[i][c]);
            }
            const float mn = fmaxf(m[i], row_max(mx));
            const float base = mn == -INFINITY ? 0.0f : mn;
            const float f = exp2f(m[i] - base);
            float sum = 0.0f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = exp2f(s[i][c] - base);
                sum += p;
                sp[(ty * R + i) * WLP + tx + 16 * c] = p;
            }
            l[i] = l[i] * f + sum;
            m[i] = mn;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                acc[i][c].x *= f;
                acc[i][c].y *= f;
                acc[i][c].z *= f;
                acc[i][c].w *= f;
            }
        }
        __syncwarp();  // a score row belongs to one half of a warp
        tile_accumulate<D, R>(sp, sv, ty, tx, acc);
    }
    float inv[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int qi = i0 + ty * R + i;
        const float sum = row_sum(l[i]);
        inv[i] = qi < len ? 1.0f / sum : 0.0f;
        if (a.lse && tx == 0 && qi < a.n)
            a.lse[((size_t)b * a.n + qi) * a.hq + hq] = qi < len ? m[i] * LN2 + logf(sum) : -INFINITY;
    }
    store_tile<D, R>((float *)a.o + (size_t)b * a.n * qs + (size_t)hq * D, qs, i0, a.n, ty, tx, acc, inv);
}

// delta[b, hq, i] = <dout[b, i, hq], o[b, i, hq]>; one warp per row.
template <int D> __global__ void __launch_bounds__(256) win_delta_kernel(WinArgs a)
{
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);  // (b, i, hq)
    const int lane = threadIdx.x & 31;
    if (row >= (int64_t)a.B * a.n * a.hq) return;
    constexpr int C = D / 4;
    const float4 *o = (const float4 *)((const float *)a.o_in + row * D), *g = (const float4 *)((const float *)a.dout + row * D);
    float x = 0.0f;
    if (lane < C) {
        const float4 fo = __ldg(o + lane), fg = __ldg(g + lane);
        x = fo.x * fg.x + fo.y * fg.y + fo.z * fg.z + fo.w * fg.w;
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(FULL, x, s);
    if (lane == 0) {
        const int64_t bi = row / a.hq;
        const int hq = (int)(row - bi * a.hq);
        const int64_t b = bi / a.n;
        a.delta[(b * a.hq + hq) * a.n + (bi - b * a.n)] = x;
    }
}

template <int D, int R> __global__ void __launch_bounds__(256) win_dq_f32_kernel(WinArgs a)
{
    using S = WinF32<D, R>;
    constexpr int NC = S::NC, ROWS = S::ROWS;
    extern __shared__ __align__(16) float wsm[];
    float *sq = wsm, *sdo = sq + ROWS * S::LD, *sk = sdo + ROWS * S::LD, *sv = sk + WT * S::LD, *sd = sv + WT * S::LD;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int per = a.B * a.hq;
    const int blk = a.nblk - 1 - (int)(blockIdx.x / (unsigned)per);
    const int bh = (int)(blockIdx.x % (unsigned)per);
    const int b = bh / a.hq, hq = bh - b * a.hq, h = hq / a.G;
    const int len = win_len(a, b), i0 = blk * ROWS;
    const size_t qs = (size_t)a.hq * D, ks = (size_t)a.hkv * D;
    const size_t qo = (size_t)b * a.n * qs + (size_t)hq * D, ko = (size_t)b * a.n * ks + (size_t)h * D;
    const KeyBlocks kb(i0, ROWS, len, a.window, a.sinks, WT);
    load_tile<D, ROWS>(sq, (const float *)a.q + qo, qs, i0, len);
    load_tile<D, ROWS>(sdo, (const float *)a.dout + qo, qs, i0, len);
    float nl[R], dl[R], scale[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int qi = i0 + ty * R + i;
        nl[i] = qi < len ? -LOG2E * __ldg(a.lse_in + ((size_t)b * a.n + qi) * a.hq + hq) : 0.0f;
        dl[i] = qi < len ? a.delta[((size_t)b * a.hq + hq) * a.n + qi] : 0.0f;
        scale[i] = a.scale;
    }
    float4 acc[R][NC];
    zero(acc);
    for (int j = 0; j < kb.na + kb.nb; ++j) {
        const int t0 = kb.start(j, WT), t1 = kb.end(j, WT);
        __syncthreads();
        load_tile<D, WT>(sk, (const float *)a.k + ko, ks, t0, t1);
        load_tile<D, WT>(sv, (const float *)a.v + ko, ks, t0, t1);
        __syncthreads();
        float s[R][4], dp[R][4];
        tile_dots<D, R>(sq, sk, ty, tx, s);
        tile_dots<D, R>(sdo, sv, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int qi = i0 + ty * R + i;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int t = t0 + tx + 16 * c;
                const bool see = qi < len && qi >= a.lone && t < t1 && win_sees(qi, t, a.window, a.sinks);
                const float p = exp2f(fmaf(s[i][c], a.scale * LOG2E, nl[i]));
                sd[(ty * R + i) * WLP + tx + 16 * c] = see ? p * (dp[i][c] - dl[i]) : 0.0f;
            }
        }
        __syncwarp();
        tile_accumulate<D, R>(sd, sk, ty, tx, acc);
    }
    store_tile<D, R>((float *)a.dq + qo, qs, i0, a.n, ty, tx, acc, scale);
}

template <int D, int R> __global__ void __launch_bounds__(256) win_dkv_f32_kernel(WinArgs a)
{
    using S = WinF32<D, R>;
    constexpr int NC = S::NC, ROWS = S::ROWS;
    extern __shared__ __align__(16) float wsm[];
    float *sk = wsm, *sv = sk + ROWS * S::LD, *sq = sv + ROWS * S::LD, *sdo = sq + WT * S::LD;
    float *sp = sdo + WT * S::LD, *sd = sp + ROWS * WLP;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const unsigned per = (unsigned)(a.B * a.hkv), pieces = per * (unsigned)(a.sink_blocks * a.chunks);
    const bool cut = blockIdx.x < pieces;  // a piece of a block that (nearly) every query sees; those come first
    const unsigned x = cut ? blockIdx.x / (unsigned)a.chunks : blockIdx.x - pieces;
    const int chunk = cut ? (int)(blockIdx.x - x * (unsigned)a.chunks) : 0;
    const int blk = (cut ? 0 : a.sink_blocks) + (int)(x / per);
    const int bh = (int)(x % per);
    const int b = bh / a.hkv, h = bh - b * a.hkv;
    const int len = win_len(a, b), t0 = blk * ROWS, t1 = min(t0 + ROWS, len);
    const size_t qs = (size_t)a.hq * D, ks = (size_t)a.hkv * D;
    const size_t ko = (size_t)b * a.n * ks + (size_t)h * D;
    load_tile<D, ROWS>(sk, (const float *)a.k + ko, ks, t0, len);
    load_tile<D, ROWS>(sv, (const float *)a.v + ko, ks, t0, len);
    float4 gk[R][NC], gv[R][NC];
    zero(gk);
    zero(gv);
    const int qend = t1 > t0 ? query_end(t0, t1, len, a.window, a.sinks) : t0;
    const int nq = (qend - t0 + WT - 1) / WT;  // query tiles per head
    const int j0 = cut ? min(chunk * a.steps, nq * a.G) : 0, j1 = cut ? min(j0 + a.steps, nq * a.G) : nq * a.G;
    {
        for (int j = j0; j < j1; ++j) {
            const int g = j / nq, hq = h * a.G + g, i0 = t0 + (j - g * nq) * WT;
            const size_t qo = (size_t)b * a.n * qs + (size_t)hq * D;
            __syncthreads();
            load_tile<D, WT>(sq, (const float *)a.q + qo, qs, i0, len);
            load_tile<D, WT>(sdo, (const float *)a.dout + qo, qs, i0, len);
            float nl[4], dl[4];  // of queries i0 + tx + 16 c
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int qi = i0 + tx + 16 * c;
                nl[c] = qi < len ? -LOG2E * __ldg(a.lse_in + ((size_t)b * a.n + qi) * a.hq + hq) : 0.0f;
                dl[c] = qi < len ? a.delta[((size_t)b * a.hq + hq) * a.n + qi] : 0.0f;
            }
            __syncthreads();
            float s[R][4], dp[R][4];
            tile_dots<D, R>(sk, sq, ty, tx, s);
            tile_dots<D, R>(sv, sdo, ty, tx, dp);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int t = t0 + ty * R + i;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int qi = i0 + tx + 16 * c;
                    const bool see = qi < len && t < len && win_sees(qi, t, a.window, a.sinks);
                    const float p = see ? exp2f(fmaf(s[i][c], a.scale * LOG2E, nl[c])) : 0.0f;
                    sp[(ty * R + i) * WLP + tx + 16 * c] = p;
                    sd[(ty * R + i) * WLP + tx + 16 * c] = see && qi >= a.lone ? p * (dp[i][c] - dl[c]) : 0.0f;
                }
            }
            __syncwarp();
            tile_accumulate<D, R>(sp, sdo, ty, tx, gv);
            tile_accumulate<D, R>(sd, sq, ty, tx, gk);
        }
    }
    float scale[R], one[R];
#pragma unroll
    for (int i = 0; i < R; ++i) scale[i] = a.scale, one[i] = 1.0f;
    if (cut) {
        float *part = a.part + (size_t)blockIdx.x * (2 * ROWS * D);
        store_tile<D, R>(part, D, 0, ROWS, ty, tx, gk, scale);
        store_tile<D, R>(part + ROWS * D, D, 0, ROWS, ty, tx, gv, one);
    } else {
        store_tile<D, R>((float *)a.dk + ko, ks, t0, a.n, ty, tx, gk, scale);
        store_tile<D, R>((float *)a.dv + ko, ks, t0, a.n, ty, tx, gv, one);
    }
}

// dk and dv of the key blocks that were cut: their pieces added in order, four elements per thread.
template <int D, int R> __global__ void __launch_bounds__(256) win_dkv_join_f32_kernel(WinArgs a)
{
    constexpr int ROWS = 16 * R, PER = 2 * ROWS * D / 4;
    const unsigned x = (blockIdx.x * 256u + threadIdx.x) / PER;  // (block, sequence, head)
    const int e = (int)((blockIdx.x * 256u + threadIdx.x) - x * PER), kv = e / (PER / 2), at = (e - kv * (PER / 2)) * 4;
    const unsigned per = (unsigned)(a.B * a.hkv);
    const int blk = (int)(x / per), bh = (int)(x % per), b = bh / a.hkv, h = bh - b * a.hkv;
    const int t = blk * ROWS + at / D;
    if (t >= a.n) return;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = 0; c < a.chunks; ++c) {  // a piece without steps holds zeros
        const float4 v = *reinterpret_cast<const float4 *>(
            a.part + ((size_t)x * a.chunks + c) * (2 * ROWS * D) + (size_t)kv * ROWS * D + at);
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    float *dst = (float *)(kv ? a.dv : a.dk) + (((size_t)b * a.n + t) * a.hkv + h) * D + at % D;
    *reinterpret_cast<float4 *>(dst) = sum;
}

}  // namespace gm
