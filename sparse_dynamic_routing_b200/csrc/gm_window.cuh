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
// fp32 kernels (this file). Plain FFMA tiles of 64 queries x 64 keys: 256 threads in a 16 x 16
// grid, each holding a 4 x 4 piece of the scores and 4 rows x D/16 columns of the output.
// Bound by the fp32 pipes; there is no tensor-core type that keeps fp32's 24 bits. The backward
// is two kernels without atomics: one per query block (dq) and one per key block (dk, dv, summed
// over the group's heads in the block), so every gradient is written once, in a fixed order.
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

constexpr int WT = 64;    // rows and columns of a tile
constexpr int WLP = 68;   // padded row of a score tile, floats

template <int D> struct WinF32 {
    static constexpr int LD = D + 4;  // padded feature row, floats: rows 4 banks apart
    static constexpr int NC = D / 64; // float4 column groups per thread
    static constexpr size_t fwd_smem = (size_t)(3 * WT * LD + WT * WLP) * 4;
    static constexpr size_t bwd_smem = (size_t)(4 * WT * LD + 2 * WT * WLP) * 4;
};

// Rows [r0, r0 + 64) of one head of a [.., heads, D] tensor into a tile; rows at or past `end`
// (padding may hold anything) become zeros.
template <int D>
__device__ __forceinline__ void load_tile(float *dst, const float *src, size_t row_stride, int r0, int end)
{
    constexpr int C = D / 4;
    for (int x = threadIdx.x; x < WT * C; x += 256) {
        const int r = x / C, c = x - r * C;
        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r0 + r < end) f = __ldg(reinterpret_cast<const float4 *>(src + (size_t)(r0 + r) * row_stride) + c);
        *reinterpret_cast<float4 *>(dst + r * WinF32<D>::LD + c * 4) = f;
    }
}

// acc[i][j] += <a[row ty*4 + i], b[row tx + 16 j]>
template <int D> __device__ __forceinline__ void tile_dots(const float *a, const float *b, int ty, int tx, float (&acc)[4][4])
{
    constexpr int LD = WinF32<D>::LD;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(a + (ty * 4 + i) * LD + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * LD + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] += x[i].x * y[j].x + x[i].y * y[j].y + x[i].z * y[j].z + x[i].w * y[j].w;
    }
}

// acc[i][c] += sum_r w(ty*4 + i, r) f[r][tx*4 + 64 c ..+3], the weights stored [row][r]
// (ROWS) or transposed, [r][row].
template <int D, bool ROWS>
__device__ __forceinline__ void tile_accumulate(const float *w, const float *f, int ty, int tx,
                                                float4 (&acc)[4][WinF32<D>::NC])
{
    constexpr int LD = WinF32<D>::LD, NC = WinF32<D>::NC;
#pragma unroll 4
    for (int r = 0; r < WT; ++r) {
        float p[4];
        if (ROWS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = w[(ty * 4 + i) * WLP + r];
        } else {
            const float4 t = *reinterpret_cast<const float4 *>(w + r * WLP + ty * 4);
            p[0] = t.x, p[1] = t.y, p[2] = t.z, p[3] = t.w;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float4 y = *reinterpret_cast<const float4 *>(f + r * LD + tx * 4 + 64 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i][c].x += p[i] * y.x;
                acc[i][c].y += p[i] * y.y;
                acc[i][c].z += p[i] * y.z;
                acc[i][c].w += p[i] * y.w;
            }
        }
    }
}

template <int NC> __device__ __forceinline__ void zero(float4 (&acc)[4][NC])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
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

template <int D> __global__ void __launch_bounds__(256) win_fwd_f32_kernel(WinArgs a)
{
    using S = WinF32<D>;
    constexpr int NC = S::NC;
    extern __shared__ __align__(16) float wsm[];
    float *sq = wsm, *sk = sq + WT * S::LD, *sv = sk + WT * S::LD, *sp = sv + WT * S::LD;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    // the blocks with the longest prefix first
    const int per = a.B * a.hq;
    const int blk = a.nblk - 1 - (int)(blockIdx.x / (unsigned)per);
    const int bh = (int)(blockIdx.x % (unsigned)per);
    const int b = bh / a.hq, hq = bh - b * a.hq, h = hq / a.G;
    const int len = win_len(a, b), i0 = blk * WT;
    const size_t qs = (size_t)a.hq * D, ks = (size_t)a.hkv * D;
    const float *q = (const float *)a.q + (size_t)b * a.n * qs + (size_t)hq * D;
    const float *k = (const float *)a.k + (size_t)b * a.n * ks + (size_t)h * D;
    const float *v = (const float *)a.v + (size_t)b * a.n * ks + (size_t)h * D;
    const KeyBlocks kb(i0, WT, len, a.window, a.sinks, WT);
    const float sl2 = a.scale * LOG2E;

    load_tile<D>(sq, q, qs, i0, len);
    float4 acc[4][NC];
    zero(acc);
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.0f;
    for (int j = 0; j < kb.na + kb.nb; ++j) {
        const int t0 = kb.start(j, WT), t1 = kb.end(j, WT);
        __syncthreads();
        load_tile<D>(sk, k, ks, t0, t1);
        load_tile<D>(sv, v, ks, t0, t1);
        __syncthreads();
        float s[4][4] = {};
        tile_dots<D>(sq, sk, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int qi = i0 + ty * 4 + i;
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
                sp[(ty * 4 + i) * WLP + tx + 16 * c] = p;
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
        tile_accumulate<D, true>(sp, sv, ty, tx, acc);
    }
    float *o = (float *)a.o + (size_t)b * a.n * qs + (size_t)hq * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int qi = i0 + ty * 4 + i;
        const float sum = row_sum(l[i]);
        if (qi >= a.n) continue;
        const float inv = qi < len ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
            *reinterpret_cast<float4 *>(o + (size_t)qi * qs + tx * 4 + 64 * c) =
                make_float4(acc[i][c].x * inv, acc[i][c].y * inv, acc[i][c].z * inv, acc[i][c].w * inv);
        if (a.lse && tx == 0)
            a.lse[((size_t)b * a.n + qi) * a.hq + hq] = qi < len ? m[i] * LN2 + logf(sum) : -INFINITY;
    }
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

// P and dS of one 64 x 64 tile (queries i0 + ty*4 + i, keys t0 + tx + 16 c), written to sp / sd.
template <int D, bool WANT_P>
__device__ __forceinline__ void bwd_scores(const WinArgs &a, const float *sq, const float *sk, const float *sdo,
                                           const float *sv, float *sp, float *sd, int i0, int len, int t0, int t1,
                                           const float (&nl)[4], const float (&dl)[4], int ty, int tx)
{
    float s[4][4] = {}, dp[4][4] = {};
    tile_dots<D>(sq, sk, ty, tx, s);
    tile_dots<D>(sdo, sv, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int qi = i0 + ty * 4 + i;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int t = t0 + tx + 16 * c;
            const bool see = qi < len && t < t1 && win_sees(qi, t, a.window, a.sinks);
            const float p = see ? exp2f(fmaf(s[i][c], a.scale * LOG2E, nl[i])) : 0.0f;
            if (WANT_P) sp[(ty * 4 + i) * WLP + tx + 16 * c] = p;
            sd[(ty * 4 + i) * WLP + tx + 16 * c] = see ? p * (dp[i][c] - dl[i]) : 0.0f;
        }
    }
}

// -log2(e) lse and delta of the thread's four query rows (0 past the sequence's end).
__device__ __forceinline__ void row_stats(const WinArgs &a, int b, int hq, int i0, int len, int ty, float (&nl)[4], float (&dl)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int qi = i0 + ty * 4 + i;
        const bool in = qi < len;
        nl[i] = in ? -LOG2E * __ldg(a.lse_in + ((size_t)b * a.n + qi) * a.hq + hq) : 0.0f;
        dl[i] = in ? a.delta[((size_t)b * a.hq + hq) * a.n + qi] : 0.0f;
    }
}

template <int D> __global__ void __launch_bounds__(256) win_dq_f32_kernel(WinArgs a)
{
    using S = WinF32<D>;
    constexpr int NC = S::NC;
    extern __shared__ __align__(16) float wsm[];
    float *sq = wsm, *sdo = sq + WT * S::LD, *sk = sdo + WT * S::LD, *sv = sk + WT * S::LD, *sd = sv + WT * S::LD;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int per = a.B * a.hq;
    const int blk = a.nblk - 1 - (int)(blockIdx.x / (unsigned)per);
    const int bh = (int)(blockIdx.x % (unsigned)per);
    const int b = bh / a.hq, hq = bh - b * a.hq, h = hq / a.G;
    const int len = win_len(a, b), i0 = blk * WT;
    const size_t qs = (size_t)a.hq * D, ks = (size_t)a.hkv * D;
    const size_t qo = (size_t)b * a.n * qs + (size_t)hq * D, ko = (size_t)b * a.n * ks + (size_t)h * D;
    const KeyBlocks kb(i0, WT, len, a.window, a.sinks, WT);
    load_tile<D>(sq, (const float *)a.q + qo, qs, i0, len);
    load_tile<D>(sdo, (const float *)a.dout + qo, qs, i0, len);
    float nl[4], dl[4];
    row_stats(a, b, hq, i0, len, ty, nl, dl);
    float4 acc[4][NC];
    zero(acc);
    for (int j = 0; j < kb.na + kb.nb; ++j) {
        const int t0 = kb.start(j, WT), t1 = kb.end(j, WT);
        __syncthreads();
        load_tile<D>(sk, (const float *)a.k + ko, ks, t0, t1);
        load_tile<D>(sv, (const float *)a.v + ko, ks, t0, t1);
        __syncthreads();
        bwd_scores<D, false>(a, sq, sk, sdo, sv, nullptr, sd, i0, len, t0, t1, nl, dl, ty, tx);
        __syncwarp();
        tile_accumulate<D, true>(sd, sk, ty, tx, acc);
    }
    float *dq = (float *)a.dq + qo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int qi = i0 + ty * 4 + i;
        if (qi >= a.n) continue;
#pragma unroll
        for (int c = 0; c < NC; ++c)
            *reinterpret_cast<float4 *>(dq + (size_t)qi * qs + tx * 4 + 64 * c) =
                make_float4(
                acc[i][c].x * a.scale, acc[i][c].y * a.scale, acc[i][c].z * a.scale, acc[i][c].w * a.scale);
    }
}

template <int D> __global__ void __launch_bounds__(256) win_dkv_f32_kernel(WinArgs a)
{
    using S = WinF32<D>;
    constexpr int NC = S::NC;
    extern __shared__ __align__(16) float wsm[];
    float *sk = wsm, *sv = sk + WT * S::LD, *sq = sv + WT * S::LD, *sdo = sq + WT * S::LD;
    float *sp = sdo + WT * S::LD, *sd = sp + WT * WLP;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int per = a.B * a.hkv;
    const int blk = (int)(blockIdx.x / (unsigned)per);  // the keys that most queries see first
    const int bh = (int)(blockIdx.x % (unsigned)per);
    const int b = bh / a.hkv, h = bh - b * a.hkv;
    const int len = win_len(a, b), t0 = blk * WT, t1 = min(t0 + WT, len);
    const size_t qs = (size_t)a.hq * D, ks = (size_t)a.hkv * D;
    const size_t ko = (size_t)b * a.n * ks + (size_t)h * D;
    load_tile<D>(sk, (const float *)a.k + ko, ks, t0, len);
    load_tile<D>(sv, (const float *)a.v + ko, ks, t0, len);
    float4 gk[4][NC], gv[4][NC];
    zero(gk);
    zero(gv);
    const int qend = t1 > t0 ? query_end(t0, t1, len, a.window, a.sinks) : t0;
    for (int g = 0; g < a.G; ++g) {
        const int hq = h * a.G + g;
        const size_t qo = (size_t)b * a.n * qs + (size_t)hq * D;
        for (int i0 = t0; i0 < qend; i0 += WT) {
            __syncthreads();
            load_tile<D>(sq, (const float *)a.q + qo, qs, i0, len);
            load_tile<D>(sdo, (const float *)a.dout + qo, qs, i0, len);
            float nl[4], dl[4];
            row_stats(a, b, hq, i0, len, ty, nl, dl);
            __syncthreads();
            bwd_scores<D, true>(a, sq, sk, sdo, sv, sp, sd, i0, len, t0, t1, nl, dl, ty, tx);
            __syncthreads();
            tile_accumulate<D, false>(sp, sdo, ty, tx, gv);
            tile_accumulate<D, false>(sd, sq, ty, tx, gk);
        }
    }
    float *dk = (float *)a.dk + ko, *dv = (float *)a.dv + ko;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + ty * 4 + i;
        if (t >= a.n) continue;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            *reinterpret_cast<float4 *>(dk + (size_t)t * ks + tx * 4 + 64 * c) =
                make_float4(
                gk[i][c].x * a.scale, gk[i][c].y * a.scale, gk[i][c].z * a.scale, gk[i][c].w * a.scale);
            *reinterpret_cast<float4 *>(dv + (size_t)t * ks + tx * 4 + 64 * c) = gv[i][c];
        }
    }
}

}  // namespace gm
