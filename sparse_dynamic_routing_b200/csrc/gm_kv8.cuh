// gm_kv8.cuh - a paged key/value cache held in 8 bits, and the attention that reads it.
//
// Pages kq, vq [num_pages, hkv, page, D] hold e4m3 values; kscale, vscale [num_pages, hkv] one
// fp32 scale per (page, KV head): an element stands for value * scale. Scales are powers of
// two, 2^e with the smallest e >= -100 such that the block's largest magnitude is at most
// 448 * 2^e (448: the largest e4m3 value), so dividing by one is exact and an element is off by
// e4m3's own half step and nothing else. A block that was given a non-finite value has the
// scale NaN, and so has everything that reads it.
//
// table [B, max_pages] lists each sequence's pages in order. Token p of sequence b is row
// p % page of page table[b, p / page].
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gm_common.cuh"

namespace gm {

struct Kv8 {
    uint8_t *kq, *vq;
    float *kscale, *vscale;
    const int32_t *table;  // [B, max_pages]
    const int32_t *lens;   // [B]
    int num_pages, max_pages, shift;  // page = 1 << shift tokens
};

constexpr int KV8_MIN_EXP = -100;

// The smallest power of two (exponent at least KV8_MIN_EXP) that 448 times is not below amax,
// from amax's fp32 bits; NaN for infinities and NaN. 448 = 1.75 * 2^8, so a significand above
// 1.75 (fraction bits above 0x600000) takes the next power.
__device__ __forceinline__ float kv8_scale(uint32_t amax_bits)
{
    if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
    const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, KV8_MIN_EXP) + 127) << 23);
}

// Two fp32 values to two e4m3 bytes, round to nearest even (callers pass at most 448).
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    return to_e4m3x2(a, b) | (to_e4m3x2(c, d) << 16);
}

// Largest magnitude so far and in a 16-byte chunk; NaN once there is one. bf16 goes two at a time.
__device__ __forceinline__ __nv_bfloat162 chunk_amax(__nv_bfloat162 m, const uint4 &u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[x])));
    return m;
}
__device__ __forceinline__ uint32_t chunk_amax(uint32_t m, const uint4 &u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) m = max(m, w[x] & 0x7fffffffu);
    return m;
}
// The magnitude's fp32 bits (an infinity or NaN: at least 0x7f800000).
__device__ __forceinline__ uint32_t amax_bits(__nv_bfloat162 m)
{
    return max((uint32_t)__bfloat16_as_ushort(m.x) << 16, (uint32_t)__bfloat16_as_ushort(m.y) << 16) & 0x7fffffffu;
}
__device__ __forceinline__ uint32_t amax_bits(uint32_t m) { return m; }
template <typename T> struct AmaxOf { using type = uint32_t; };
template <> struct AmaxOf<__nv_bfloat16> { using type = __nv_bfloat162; };

// A chunk's elements times a power of two, as e4m3 bytes. (bf16 products are exact; what they lose
// below 2^-126 is 0 in e4m3.)
__device__ __forceinline__ uint2 chunk_e4m3(const uint4 &u, float inv, __nv_bfloat16 *)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    const __nv_bfloat162 f = __float2bfloat162_rn(inv);
    uint32_t r[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w[x]), f);
        const uint32_t b = *reinterpret_cast<const uint32_t *>(&y);
        r[x] = to_e4m3x2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
    }
    return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}
__device__ __forceinline__ uint32_t chunk_e4m3(const uint4 &u, float inv, float *)
{
    return to_e4m3x4(__uint_as_float(u.x) * inv, __uint_as_float(u.y) * inv, __uint_as_float(u.z) * inv,
                     __uint_as_float(u.w) * inv);
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t two)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return __half22float2(__half2(h));
}

// ---- appending tokens ---------------------------------------------------------------------------
//
// One block per (sequence, touched page, KV head, K or V). The page's new rows stay in registers
// between the pass that finds their largest magnitude and the pass that rounds them, so every
// new element is read once and written once: the kernel moves what it must (bound by HBM; for
// single tokens by launch latency). When a partly filled page's scale grows, its older bytes
// are rounded again at the new scale.

struct Kv8AppendArgs {
    Kv8 c;
    const void *k, *v;        // [B, t, hkv, D]
    const int32_t *new_lens;  // [B] rows of each sequence that are its own, or null: t each
    int B, t, hkv, touch;     // touch: pages a sequence may touch
};

template <typename T, int D, int PAGE> __global__ void __launch_bounds__(256) kv8_append_kernel(Kv8AppendArgs a)
{
    constexpr int VEC = Vec<T>::N, C = D / VEC;       // 16-byte chunks per row
    constexpr int NCH = (PAGE * C + 255) / 256;       // chunks per thread
    __shared__ uint32_t samax[8];
    const int kv = blockIdx.x & 1;
    unsigned x = blockIdx.x >> 1;
    const int h = (int)(x % (unsigned)a.hkv);
    x /= (unsigned)a.hkv;
    const int jp = (int)(x % (unsigned)a.touch), b = (int)(x / (unsigned)a.touch);
    const int have = __ldg(a.c.lens + b);
    const int n = a.new_lens ? min(max(__ldg(a.new_lens + b), 0), a.t) : a.t;
    if (n == 0) return;
    if (have < 0) {
        if (threadIdx.x == 0) raise_index_error();
        return;
    }
    const int pg = (have >> a.c.shift) + jp;  // page of the sequence, and its rows this call writes
    const int64_t first = (int64_t)pg << a.c.shift;
    const int r0 = (int)max((int64_t)have - first, (int64_t)0);
    const int r1 = (int)min((int64_t)have + n - first, (int64_t)PAGE);
    if (r1 <= r0) return;
    int id = -1;
    if (pg < a.c.max_pages) id = __ldg(a.c.table + (size_t)b * a.c.max_pages + pg);
    if (id < 0 || id >= a.c.num_pages) {
        if (threadIdx.x == 0) raise_index_error();
        return;
    }
    const size_t blk = (size_t)id * a.hkv + h;
    // row r of the page is new token first + r - have
    const T *src = (const T *)(kv ? a.v : a.k) + (((size_t)b * a.t + (size_t)(first - have + r0)) * a.hkv + h) * D;
    uint4 u[NCH];
    const int nch = (r1 - r0) * C;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int ch = threadIdx.x + 256 * i, r = ch / C;
        u[i] = make_uint4(0, 0, 0, 0);
        if (ch < nch) u[i] = ld16_stream(src + (size_t)r * a.hkv * D + (ch - r * C) * VEC);
    }
    typename AmaxOf<T>::type big{};
#pragma unroll
    for (int i = 0; i < NCH; ++i) big = chunk_amax(big, u[i]);
    uint32_t amax = __reduce_max_sync(FULL, amax_bits(big));
    if ((threadIdx.x & 31) == 0) samax[threadIdx.x >> 5] = amax;
    float *scales = kv ? a.c.vscale : a.c.kscale;
    const float old = r0 > 0 ? scales[blk] : 0.0f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, samax[i]);
    float scale = kv8_scale(amax);
    // an older block keeps its scale unless the new rows need a larger one (NaN stays)
    if (r0 > 0 && !(scale > old) && scale == scale) scale = old;
    if (r0 > 0 && old != old) scale = old;
    if (threadIdx.x == 0) scales[blk] = scale;
    uint8_t *dst = (kv ? a.c.vq : a.c.kq) + blk * ((size_t)PAGE * D);
    if (r0 > 0 && scale != old && scale == scale) {
        const float f = old / scale;  // a power of two
        for (int ch = threadIdx.x; ch < r0 * D / 16; ch += 256) {
            uint4 w = *(reinterpret_cast<uint4 *>(dst) + ch);
            uint32_t *wp = &w.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 lo = from_e4m3x2(wp[e] & 0xffffu), hi = from_e4m3x2(wp[e] >> 16);
                wp[e] = to_e4m3x4(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
            }
            *(reinterpret_cast<uint4 *>(dst) + ch) = w;
        }
    }
    // the elements of a block whose scale is NaN are 0: no byte of a token is itself a NaN, so a
    // reader's weight of 0 always gives 0
    const bool whole = scale == scale;
    const float inv = whole ? 1.0f / scale : 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int ch = threadIdx.x + 256 * i;
        if (ch < nch) {
            auto w = chunk_e4m3(u[i], inv, (T *)nullptr);
            if (!whole) w = decltype(w){};
            // rows of a block are contiguous
            *reinterpret_cast<decltype(w) *>(dst + (size_t)r0 * D + (size_t)ch * VEC) = w;
        }
    }
}

// ---- attention over the cache ---------------------------------------------------------------------
//
// Query row x < q_lens[b] of sequence b stands at position lens[b] - q_lens[b] + x and sees the
// cached tokens that the windowed attention's rule allows (t <= i, i - t < window or t < sinks).
//
// A call reads every visible byte of K and V once, so HBM bounds it. One row tile (up to
// 8 NT query rows of one KV head: the group's heads times the sequence's rows) is split over
// `splits` blocks of four warps; every warp takes every (4 splits)-th unit of 32 keys (two pieces
// of 16, each inside one page), copies it into its own two-stage ring in shared memory while it
// computes the one before, and keeps its own softmax maximum and sum. A warp's computation on a
// unit is one long chain of dependent steps, so bandwidth comes from many warps: 12 per SM, and
// two pieces per step (one piece per step: 1400 cycles a piece whatever the memory does). The
// warps are joined in shared memory; with more than one split the blocks write partial outputs
// to the workspace and a second kernel joins those, in a fixed order. (A cluster that joins
// through distributed shared memory needs no workspace, but a GPU holds only 7 clusters of 16 such
// blocks, and one sequence of 8 KV heads then waits for two rounds: 72 us against 33 us for 65536
// tokens.)
//
// Arithmetic. mma.sync m16n8k16 with fp16 operands and fp32 sums, computed transposed
// (S^T = K q^T, O^T = V^T P^T) so that the 16-row operand is the cache and a single token's few
// query rows fill an 8-column operand. The bytes go from global memory to registers in the
// order the operands want (any permutation of d, and of the output's columns, is as good) and
// become fp16, which holds every e4m3 value. Query rows are scaled by a power of two into fp16's upper
// range (bf16's 8 bits fit its 11; what falls below fp16's subnormals is 2^-38 of the row's largest
// element), probabilities by 2^14 likewise. The fp16 rounding of a probability (half a step, 2^-11) lies
// below the bf16 rounding of the output (2^-8): one token over 65536 gives 0.0017 against 64 bits in the
// 2-norm, as probabilities in fp32 do. fp32 queries and probabilities are split in two fp16 terms, which
// leaves 2^-22: a third term would cost another product per key for the last two of fp32's 24 bits.

struct Kv8AttnArgs {
    Kv8 c;
    const void *q;          // [B, t, hq, D]
    const int32_t *q_lens;  // [B] or null: t each
    void *o;                // [B, t, hq, D]
    float *lse;             // [B, t, hq] or null
    int t, hq, hkv, G, tiles;  // row tiles per (sequence, KV head)
    int window, sinks;
    float sl2;              // scale * log2(e)
    int splits;             // blocks per row tile
    float *part;            // splits > 1: [items, splits, 8 NT, D] outputs, scaled by each split's own sum
    float2 *ml;             // [items, splits, 8 NT] maximum (base 2) and sum
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

// The two low / high e4m3 bytes of a word as fp16 values, exactly. The conversion runs at half
// rate; building the same bits with shifts and masks takes four such instructions.
__device__ __forceinline__ uint32_t half2_lo(uint32_t w)
{
    uint32_t h;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ uint32_t half2_hi(uint32_t w)
{
    uint32_t h;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(h) : "r"(w));
    return h;
}

__device__ __forceinline__ uint32_t pack_half2(float x, float y)
{
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// x and y less the fp16 values packed in `hi`
__device__ __forceinline__ uint32_t pack_rest(float x, float y, uint32_t hi)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return pack_half2(x - f.x, y - f.y);
}

__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4_at(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}

// Four elements of a query row's output, and its lse (by the thread of column 0).
template <typename T>
__device__ __forceinline__ void kv8_store_row(const Kv8AttnArgs &a, size_t row, int D, int d, float4 o, float mx, float sum,
                                              bool none)
{
    const float inv = none ? 0.0f : 1.0f / sum;
    o = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>((float *)a.o + row * D + d) = o;
    } else {
        const __nv_bfloat162 x[2] = {__floats2bfloat162_rn(o.x, o.y), __floats2bfloat162_rn(o.z, o.w)};
        *reinterpret_cast<uint2 *>((__nv_bfloat16 *)a.o + row * D + d) = *reinterpret_cast<const uint2 *>(x);
    }
    if (a.lse && d == 0) a.lse[row] = none ? -INFINITY : (mx + lg2(sum)) * LN2;
}

// A weight 2^(s - m) is multiplied by vf 2^(m - mv) 2^14 (vf: the value scale, m: the row's largest
// score, mv: the largest of score + log2 vf). While vf 2^(m - mv) is at most 2^KV8_FAR that product is
// taken as it stands: the factor is far inside fp32's range, and a weight that is flushed below 2^-126
// would have been below 2^-48 of fp16's 2^14. A block of zeros (vf = 2^-100) that holds the largest
// score, beside one of large values, has factors past fp32's range.
constexpr float KV8_FAR = 64.0f;
constexpr int KV8_W = 4;       // warps per block
constexpr int KV8_PER_SM = 3;  // blocks per SM (shared memory: the rings)

template <int D, int NT, bool SPLIT> struct Kv8Smem {
    static constexpr int ROWS = 8 * NT;
    static constexpr int QTERMS = SPLIT ? 2 : 1;
    union {
        uint8_t ring[KV8_W][2][2][2][16 * D];  // [stage][piece][K, V]: rows, 16-byte chunks swizzled
        float part[KV8_W][ROWS][D + 4];        // afterwards: the warps' outputs
    };
    float scales[KV8_W][2][2][2];
    __half q[QTERMS][ROWS][D + 8];  // rows 4 banks apart
    float qscale[ROWS];             // score factor of a row (powers of two undone)
    int pos[ROWS];                  // position, -1: no such row
    float m[KV8_W][ROWS], l[KV8_W][ROWS];
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(KV8_W * 32, KV8_PER_SM) kv8_attention_kernel(Kv8AttnArgs a)
{
    constexpr int W = KV8_W;
    constexpr bool SPLIT = sizeof(T) == 4;
    using Smem = Kv8Smem<D, NT, SPLIT>;
    constexpr int ROWS = Smem::ROWS;
    constexpr int NK = D / 64;            // 16-byte chunks of a key row per lane
    constexpr int VW = D / 32;            // 4-byte words of a value row per lane
    extern __shared__ __align__(16) unsigned char kv8_smem[];
    Smem &sm = *reinterpret_cast<Smem *>(kv8_smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    unsigned x = blockIdx.x / (unsigned)a.splits;
    const int rank = (int)(blockIdx.x - x * (unsigned)a.splits);
    const unsigned item = x;
    const int rt = (int)(x % (unsigned)a.tiles);
    x /= (unsigned)a.tiles;
    const int h = (int)(x % (unsigned)a.hkv), b = (int)(x / (unsigned)a.hkv);

    int len = __ldg(a.c.lens + b);
    const int64_t room = (int64_t)a.c.max_pages << a.c.shift;
    if (len < 0 || len > room) {
        if (threadIdx.x == 0 && rank == 0) raise_index_error();
        len = len < 0 ? 0 : (int)room;
    }
    const int ql = a.q_lens ? min(max(__ldg(a.q_lens + b), 0), a.t) : a.t;
    const int nrows = min(a.t * a.G - rt * ROWS, ROWS);  // rows of this tile that the tensors have

    // ---- query rows to shared memory, scaled into fp16 ------------------------------------
    for (int r = warp; r < ROWS; r += W) {
        const int f = rt * ROWS + r, xq = f / a.G, hq = h * a.G + f - xq * a.G;
        const int pos = r < nrows && xq < ql ? len - ql + xq : -1;
        constexpr int PER = D / 32;
        float v[PER];
        float big = 0.0f;
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = 0.0f;
        if (pos >= 0) {
            const T *q = (const T *)a.q + (((size_t)b * a.t + xq) * a.hq + hq) * D + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; ++e) v[e] = (float)q[e];
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) big = fmaxf(big, fabsf(v[e]));
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) big = fmaxf(big, __shfl_xor_sync(FULL, big, s));
        // 2^(14 - exponent of the largest), the exponent held in [-100, 127]
        const int e2 = max((int)(__float_as_uint(big) >> 23) - 127, -100);
        const float up = __uint_as_float((uint32_t)(127 + 14 - min(e2, 127)) << 23);
        const float down = __uint_as_float((uint32_t)(127 - 14 + min(e2, 127)) << 23);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const __half hi = __float2half_rn(v[e] * up);
            sm.q[0][r][lane * PER + e] = hi;
            if constexpr (SPLIT) sm.q[1][r][lane * PER + e] = __float2half_rn(v[e] * up - __half2float(hi));
        }
        if (lane == 0) {
            sm.qscale[r] = down * a.sl2;
            sm.pos[r] = pos;
        }
    }
    __syncthreads();

    // ---- the pieces of 16 keys that some row sees --------------------------------------------
    // rows are in ascending position, so the first and last of the tile bound them
    const int xa = rt * ROWS / a.G, xb = min((rt * ROWS + nrows - 1) / a.G, ql - 1);
    const int pmin = max(len - ql + xa, 0), pmax = len - ql + xb;
    int na = 0, p0 = 0, np = 0;
    if (xa <= xb && pmax >= 0) {
        const int lo = max(0, pmin - a.window + 1);
        p0 = lo >> 4;
        na = min((min(a.sinks, lo) + 15) >> 4, p0);
        np = na + (pmax >> 4) + 1 - p0;
    }
    const int nu = (np + 1) >> 1;  // units of two pieces
    const int stride = a.splits * W;

    int mypos[NT][2];
    float myq[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mypos[n][e] = sm.pos[n * 8 + 2 * c + e];
            myq[n][e] = sm.qscale[n * 8 + 2 * c + e];
        }
    float m[NT][2], mv[NT][2], l[NT][2];
    float acc[NT][D / 16][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) m[n][e] = -INFINITY, mv[n][e] = -INFINITY, l[n][e] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][j][e] = 0.0f;
    }

    const auto piece = [&](int i) { return i < na ? i : p0 + i - na; };
    const auto raw_page = [&](int i) {  // page of piece i (0 past the end), not yet checked
        return i < np ? __ldg(a.c.table + (size_t)b * a.c.max_pages + ((piece(i) << 4) >> a.c.shift)) : 0;
    };
    bool bad = false;
    const uint32_t ring = smem_u32(&sm.ring[warp][0][0][0][0]);
    constexpr int CH = D / 16;  // 16-byte chunks of a row
    // Unit u into its stage. Chunk col of row r sits at col ^ f(r), which spreads the rows that
    // one load instruction of the computation reads over the banks.
    const auto issue = [&](int u, int st, const int (&ids)[2]) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int i = 2 * u + p;
            int id = ids[p];
            if (i >= np) continue;
            if (id < 0 || id >= a.c.num_pages) {  // read page 0 and raise the flag
                bad = true;
                id = 0;
            }
            const size_t blk = (size_t)id * a.hkv + h;
            const size_t at = ((blk << a.c.shift) + (size_t)((piece(i) << 4) & ((1 << a.c.shift) - 1))) * D;
            const uint32_t dst = ring + (st * 2 + p) * (32 * D);
            const uint8_t *ks = a.c.kq + at + lane * 16, *vs = a.c.vq + at + lane * 16;
#pragma unroll
            for (int y = 0; y < CH / 2; ++y) {
                const int x = lane + 32 * y, r = x / CH, col = x - r * CH;
                const int fk = D == 128 ? (r & 1) * 4 : 0, fv = D == 128 ? ((r >> 1) & 3) * 2 : (r >> 1) & 3;
                cp_async16_at(dst + r * D + (col ^ fk) * 16, ks + y * 512);
                cp_async16_at(dst + 16 * D + r * D + (col ^ fv) * 16, vs + y * 512);
            }
            if (lane < 2) cp_async4_at(smem_u32(&sm.scales[warp][st][p][lane]), (lane ? a.c.vscale : a.c.kscale) + blk);
        }
        cp_async_commit();
    };

    int u = rank * W + warp;
    int ids[2] = {raw_page(2 * u), raw_page(2 * u + 1)};
    issue(u, 0, ids);
    ids[0] = raw_page(2 * (u + stride));
    ids[1] = raw_page(2 * (u + stride) + 1);
    for (int st = 0; u < nu; u += stride, st ^= 1) {
        __syncwarp();  // every lane is done with the other stage
        issue(u + stride, st ^ 1, ids);
        ids[0] = raw_page(2 * (u + 2 * stride));
        ids[1] = raw_page(2 * (u + 2 * stride) + 1);
        cp_async_wait<1>();
        __syncwarp();  // the unit is complete
        // a second piece past the end starts past every position (max_pages * page < 2^31, so a
        // sequence's last one is at most 2^31 - 17), where nothing is seen; its 16 rows stay within 32 bits
        const int t0[2] = {piece(2 * u) << 4, 2 * u + 1 < np ? piece(2 * u + 1) << 4 : 0x7ffffff0};
        const float kf[2] = {sm.scales[warp][st][0][0], sm.scales[warp][st][1][0]};
        const float vf[2] = {sm.scales[warp][st][0][1], sm.scales[warp][st][1][1]};
        // S^T = K q^T
        float s[2][NT][4];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[p][n][e] = 0.0f;
#pragma unroll
        for (int e = 0; e < NK; ++e) {
            uint4 kr[2][2];  // [piece][keys g, g + 8]: this lane's chunk
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    kr[p][y] = *reinterpret_cast<const uint4 *>(
                        &sm.ring[warp][st][p][0][(g + 8 * y) * D + ((c + 4 * e) ^ (D == 128 ? (g & 1) * 4 : 0)) * 16]);
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
                const int d = e * 64 + c * 16 + k4 * 4;
                uint2 q0[NT], q1[SPLIT ? NT : 1];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    q0[n] = *reinterpret_cast<const uint2 *>(&sm.q[0][n * 8 + g][d]);
                    if constexpr (SPLIT) q1[n] = *reinterpret_cast<const uint2 *>(&sm.q[1][n * 8 + g][d]);
                }
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint32_t w0 = (&kr[p][0].x)[k4], w1 = (&kr[p][1].x)[k4];
                    const uint32_t a0 = half2_lo(w0), a2 = half2_hi(w0);
                    const uint32_t a1 = half2_lo(w1), a3 = half2_hi(w1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_f16(s[p][n], a0, a1, a2, a3, q0[n].x, q0[n].y);
                        if constexpr (SPLIT) mma_f16(s[p][n], a0, a1, a2, a3, q1[n].x, q1[n].y);
                    }
                }
            }
        }
        // softmax: rows 2c + e, keys t0 + g and t0 + g + 8 of both pieces
        float lv[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) lv[p] = (float)((int)((__float_as_uint(vf[p]) >> 23) & 255u) - 127);
        uint32_t pt[2][NT][2], pl[2][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float mb[2], vb[2], up[2][2], f[2];
            bool see[2][4], moved = false, far = false;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = t0[p] + g + 8 * (e >> 1), ps = mypos[n][e & 1];
                    see[p][e] = t <= ps && (ps - t < a.window || t < a.sinks);
                    s[p][n][e] = see[p][e] ? s[p][n][e] * (myq[n][e & 1] * kf[p]) : -INFINITY;
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float m0 = fmaxf(s[0][n][e], s[0][n][e + 2]), m1 = fmaxf(s[1][n][e], s[1][n][e + 2]);
#pragma unroll
                for (int sft = 4; sft < 32; sft <<= 1) {
                    m0 = fmaxf(m0, __shfl_xor_sync(FULL, m0, sft));
                    m1 = fmaxf(m1, __shfl_xor_sync(FULL, m1, sft));
                }
                const float mn = fmaxf(m[n][e], fmaxf(m0, m1)), vn = fmaxf(mv[n][e], fmaxf(m0 + lv[0], m1 + lv[1]));
                vb[e] = vn == -INFINITY ? 0.0f : vn;
                mb[e] = mn == -INFINITY ? 0.0f : mn;
                l[n][e] *= ex2_ftz(m[n][e] - mb[e]);
                f[e] = ex2_ftz(mv[n][e] - vb[e]);
                moved |= vn != mv[n][e];
                far |= fmaxf(lv[0], lv[1]) + (mb[e] - vb[e]) > KV8_FAR;
                m[n][e] = mn;
                mv[n][e] = vn;
                const float x = ex2_ftz(mb[e] - vb[e]) * 0x1p14f;
                up[0][e] = vf[0] * x;
                up[1][e] = vf[1] * x;
            }
            if (__any_sync(FULL, far)) {
                // a factor that could overflow gives up 2^over to the exponential it multiplies, which
                // is then at most 2^-KV8_FAR: s + lv <= vb for every key that is seen
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float over = fmaxf(lv[p] + (mb[e] - vb[e]) - KV8_FAR, 0.0f);
                        up[p][e] = vf[p] * (ex2_ftz(mb[e] - vb[e] - over) * 0x1p14f);
#pragma unroll
                        for (int y = 0; y < 4; y += 2) {
                            const float x = s[p][n][e + y] - mb[e];
                            l[n][e] += see[p][e + y] ? ex2_ftz(x) : 0.0f;
                            s[p][n][e + y] = see[p][e + y] ? ex2_ftz(x + over) * up[p][e] : 0.0f;
                        }
                    }
            } else {
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = see[p][e] ? ex2_ftz(s[p][n][e] - mb[e & 1]) : 0.0f;
                        l[n][e & 1] += x;
                        s[p][n][e] = see[p][e] ? x * up[p][e & 1] : 0.0f;  // a NaN scale reaches only rows that see its block
                    }
            }
            if (__any_sync(FULL, moved)) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[n][j][e] *= f[e & 1];
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t h0 = pack_half2(s[p][n][0], s[p][n][1]), h1 = pack_half2(s[p][n][2], s[p][n][3]);
                pt[p][n][0] = transpose8x8(h0);
                pt[p][n][1] = transpose8x8(h1);
                if constexpr (SPLIT) {
                    pl[p][n][0] = transpose8x8(pack_rest(s[p][n][0], s[p][n][1], h0));
                    pl[p][n][1] = transpose8x8(pack_rest(s[p][n][2], s[p][n][3], h1));
                }
            }
        }
        // O^T += V^T P^T
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint8_t *vp = sm.ring[warp][st][p][1];
            uint32_t vr[4][VW];  // keys 2c, 2c+1, 2c+8, 2c+9: columns g * (D/8) ..
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int r = 2 * c + (y & 1) + 8 * (y >> 1);
                if constexpr (VW == 4) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(vp + r * D + (g ^ (((r >> 1) & 3) * 2)) * 16);
                    vr[y][0] = x.x, vr[y][1] = x.y, vr[y][2] = x.z, vr[y][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(vp + r * D + ((g >> 1) ^ ((r >> 1) & 3)) * 16 + (g & 1) * 8);
                    vr[y][0] = x.x, vr[y][1] = x.y;
                }
            }
            if (t0[p] > len - 16) {  // rows past the sequence's end may hold any bytes, NaN among them
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (t0[p] + 2 * c + (y & 1) + 8 * (y >> 1) >= len) {
#pragma unroll
                        for (int z = 0; z < VW; ++z) vr[y][z] = 0;
                    }
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {  // output columns g * (D/8) + 2j and + 2j + 1
                // byte pairs (key, next key) of column 2j in the low half, of column 2j + 1 in the high
                const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
                const uint32_t x = __byte_perm(vr[0][j >> 1], vr[1][j >> 1], sel);
                const uint32_t y = __byte_perm(vr[2][j >> 1], vr[3][j >> 1], sel);
                const uint32_t a0 = half2_lo(x), a1 = half2_hi(x);
                const uint32_t a2 = half2_lo(y), a3 = half2_hi(y);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_f16(acc[n][j], a0, a1, a2, a3, pt[p][n][0], pt[p][n][1]);
                    if constexpr (SPLIT) mma_f16(acc[n][j], a0, a1, a2, a3, pl[p][n][0], pl[p][n][1]);
                }
            }
        }
    }
    if (bad && lane == 0) raise_index_error();
    cp_async_wait<0>();
    __syncthreads();  // the rings become the warps' outputs

    // ---- join the warps ---------------------------------------------------------------------
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = n * 8 + 2 * c + e;
#pragma unroll
            for (int sft = 4; sft < 32; sft <<= 1) l[n][e] += __shfl_xor_sync(FULL, l[n][e], sft);
            if (r < nrows) {
                // back from the values' own maximum and the weights' 2^14
                const float x = m[n][e] == -INFINITY ? 0.0f : ex2_ftz(mv[n][e] - m[n][e]) * 0x1p-14f;
                if (g == 0) {
                    sm.m[warp][r] = m[n][e];
                    sm.l[warp][r] = l[n][e];
                }
                float *dst = &sm.part[warp][r][g * (D / 8)];
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    *reinterpret_cast<float2 *>(dst + 2 * j) = make_float2(acc[n][j][e] * x, acc[n][j][2 + e] * x);
            }
        }
    __syncthreads();
    for (int y = threadIdx.x; y < nrows * (D / 4); y += W * 32) {
        const int r = y / (D / 4), d = (y - r * (D / 4)) * 4;
        float mx = sm.m[0][r];
#pragma unroll
        for (int w = 1; w < W; ++w) mx = fmaxf(mx, sm.m[w][r]);
        const float mb = mx == -INFINITY ? 0.0f : mx;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = ex2_ftz(sm.m[w][r] - mb);
            const float4 v = *reinterpret_cast<const float4 *>(&sm.part[w][r][d]);
            o.x += v.x * f, o.y += v.y * f, o.z += v.z * f, o.w += v.w * f;
            sum += sm.l[w][r] * f;
        }
        if (a.splits > 1) {
            const size_t at = ((size_t)item * a.splits + rank) * ROWS + r;
            *reinterpret_cast<float4 *>(a.part + at * D + d) = o;
            if (d == 0) a.ml[at] = make_float2(mx, sum);
        } else {
            const int f = rt * ROWS + r, xq = f / a.G, hq = h * a.G + f - xq * a.G;
            kv8_store_row<T>(a, ((size_t)b * a.t + xq) * a.hq + hq, D, d, o, mx, sum, sm.pos[r] < 0);
        }
    }
}

// Joins the splits of every row tile: one block per row, its warps taking splits in turn, lanes
// across D.
template <typename T, int D, int NT> __global__ void __launch_bounds__(128) kv8_join_kernel(Kv8AttnArgs a)
{
    constexpr int ROWS = 8 * NT;
    __shared__ float4 so[4][D / 4];
    __shared__ float sm[4], sl[4];
    const int64_t row = blockIdx.x;  // (b, x, hq)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = lane * 4;
    const int64_t bx = row / a.hq;
    const int hq = (int)(row - bx * a.hq), h = hq / a.G;
    const int64_t b = bx / a.t;
    const int f = (int)(bx - b * a.t) * a.G + hq - h * a.G;  // row of the (sequence, KV head)
    const size_t at = (((size_t)(b * a.hkv + h) * a.tiles + f / ROWS) * a.splits) * ROWS + f % ROWS;
    pdl_wait();
    float mx = -INFINITY;
    for (int s = warp * 32 + lane; s < a.splits; s += 128) mx = fmaxf(mx, a.ml[at + (size_t)s * ROWS].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
    if (lane == 0) sm[warp] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    const float mb = mx == -INFINITY ? 0.0f : mx;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
#pragma unroll 4
    for (int s = warp; s < a.splits; s += 4) {
        const float2 ml = a.ml[at + (size_t)s * ROWS];
        const float w = ex2_ftz(ml.x - mb);
        sum += ml.y * w;
        if (d < D) {
            const float4 v = *reinterpret_cast<const float4 *>(a.part + (at + (size_t)s * ROWS) * D + d);
            o.x += v.x * w, o.y += v.y * w, o.z += v.z * w, o.w += v.w * w;
        }
    }
    if (d < D) so[warp][lane] = o;
    if (lane == 0) sl[warp] = sum;
    __syncthreads();
    if (warp > 0 || d >= D) return;
    sum = (sl[0] + sl[1]) + (sl[2] + sl[3]);
#pragma unroll
    for (int w = 1; w < 4; ++w) {
        const float4 v = so[w][lane];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    kv8_store_row<T>(a, (size_t)row, D, d, o, mx, sum, sum == 0.0f);
}

// ---- sparse edge attention over the cache -----------------------------------------------------------
//
// As gm_sea_forward for the last rows of each sequence: row x has edges idx/w [B, t, hkv, s] into
// the cached tokens, z_j = scale <q, k_{t_j}> + ln w_j, o = sum softmax(z)_j v_{t_j}.
//
// The same operands as in the attention above, with 16 gathered slots in the place of 16 keys: a
// tile is RT consecutive rows (b, x, KV head), their slots in the 16-row operand and their query
// heads in the 8-column one (4 rows of 4 slots and 2 heads fill both). Scores and weights off
// the rows' own diagonal blocks are masked away; the tensor cores have the time. Against fp32
// multiplications on the gathered bytes this takes a fifth of the instructions, which had been
// the bound. Weights enter as two fp16 terms (22 bits; the second costs a tile 8 of its 24 mma),
// so the output's rounding is the only one that shows. Weights get a power of two per query row
// that puts the largest product of weight and value scale at 2^14.
//
// A slot's chain of dependent loads (edge -> page -> scales) is walked one step per tile, three
// tiles ahead, one lane per slot; the rows themselves and the queries are copied into the warp's
// two-stage buffer in shared memory while the tile before them is computed.

struct Kv8SeaArgs {
    Kv8 c;
    const void *q;
    const int32_t *idx;
    const float *w;
    const int32_t *q_lens;
    void *o;
    float *lse;
    int t, hkv, G, s;
    int s_shift, g_shift;  // slots and heads of a row take 1 << shift operand rows and columns
    int rt;                // rows per tile
    int64_t rows, tiles;   // B * t * hkv, and tiles of rt rows
    FastDiv div_h, div_t;
    float sl2;             // scale * log2(e)
};

// A slot on its way: (1) its edge and its sequence's length, (2) its page, (3) its scales.
struct Kv8Edge {
    float w;
    int t, len, x, ql, b;  // target; the sequence's length, the query row, the sequence's query rows
    uint32_t h;
};
struct Kv8Paged {
    float w;
    int t, id;
    uint32_t h;
};
// What a slot adds: its row of the pool (NONE: inactive), score factor, weight, value scale.
struct Kv8Slot {
    static constexpr uint32_t NONE = 0xffffffffu;
    uint32_t row;
    float ks, w, vs;
};

__device__ __forceinline__ Kv8Edge kv8_edge(const Kv8SeaArgs &a, bool in, int64_t at, int j)
{
    Kv8Edge s{0.0f, 0, 0, 0, 0, 0, 0};  // no slot: as a row of an empty sequence
    if (!in || at >= a.rows || j >= a.s) return s;
    const uint32_t row = (uint32_t)at;  // rows < 2^31
    const uint32_t bx = a.div_h.div(row);
    s.h = row - bx * a.div_h.d;
    s.b = (int)a.div_t.div(bx);
    s.x = (int)(bx - (uint32_t)s.b * a.div_t.d);
    s.w = __ldg(a.w + (size_t)row * a.s + j);
    s.t = __ldg(a.idx + (size_t)row * a.s + j);
    s.len = __ldg(a.c.lens + s.b);
    s.ql = a.q_lens ? __ldg(a.q_lens + s.b) : a.t;
    return s;
}

__device__ __forceinline__ Kv8Paged kv8_paged(const Kv8SeaArgs &a, const Kv8Edge &e, bool report, int checked)
{
    Kv8Paged s{0.0f, e.t, 0, e.h};
    const int64_t room = (int64_t)a.c.max_pages << a.c.shift;
    int len = e.len;
    if (len < 0 || len > room) {
        if (report) raise_index_error();
        len = len < 0 ? 0 : (int)room;
    }
    const int ql = min(max(e.ql, 0), a.t), pos = e.x < ql ? len - ql + e.x : -1;
    if (checked && report && pos >= 0) {
        const bool bad_w = !(e.w >= 0.0f) || isinf(e.w);
        if (bad_w || (e.w > 0.0f && e.t > pos)) atomicOr(&g_error_flag, ERR_EDGE_INVALID);
    }
    if (pos < 0 || !(e.w > 0.0f)) return s;
    if (e.t < 0 || e.t >= len) {
        if (report) raise_index_error();
        return s;
    }
    s.w = e.w;
    s.id = __ldg(a.c.table + (size_t)e.b * a.c.max_pages + (e.t >> a.c.shift));
    return s;
}

__device__ __forceinline__ Kv8Slot kv8_slot(const Kv8SeaArgs &a, const Kv8Paged &p, bool report)
{
    Kv8Slot s{Kv8Slot::NONE, 0.0f, 1.0f, 0.0f};
    if (p.w == 0.0f) return s;
    if (p.id < 0 || p.id >= a.c.num_pages) {
        if (report) raise_index_error();
        return s;
    }
    const uint32_t blk = (uint32_t)p.id * (uint32_t)a.hkv + p.h;  // pool rows < 2^32
    s.row = (blk << a.c.shift) + (uint32_t)(p.t & ((1 << a.c.shift) - 1));
    s.ks = __ldg(a.c.kscale + blk);
    s.vs = __ldg(a.c.vscale + blk);
    s.w = p.w;
    return s;
}

template <typename T, int D, int NP> struct Kv8SeaSmem {  // of one warp
    uint8_t k[2][NP][16 * D], v[2][NP][16 * D];  // 16-byte chunks swizzled as in the attention's ring
    T q[2][8 * D];                               // chunk x of row r at x ^ (r & 1)
};

// NP: pieces of 16 slots per row (2 for more than 16 slots).
template <typename T, int D, int NP>
__global__ void __launch_bounds__(128) kv8_sea_kernel(Kv8SeaArgs a, int checked)
{
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr int VEC = Vec<T>::N, KS = D / 16, NK = D / 64, VW = D / 32, CH = D / 16;
    constexpr int QC = D / VEC;   // 16-byte chunks of a query row
    constexpr int QV = 16 / VEC;  // of 16 query elements
    extern __shared__ __align__(16) unsigned char kv8_smem[];
    auto &sm = reinterpret_cast<Kv8SeaSmem<T, D, NP> *>(kv8_smem)[threadIdx.x >> 5];
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // steps: tiles, and within a tile the groups of eight heads
    const int hg = (a.G + 7) / 8;
    const int64_t nstep = a.tiles * hg, stride = (int64_t)gridDim.x * 4;
    int64_t it = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (it >= nstep) return;
    // slot `lane & 15` of a tile: row (lane & 15) >> ssh (at most 16 slots per piece)
    const int ssh = min(a.s_shift, 4), sr = (lane & 15) >> ssh, sj = (lane & 15) & ((1 << ssh) - 1);
    const auto tile_of = [&](int64_t i) { return hg == 1 ? i : i / hg; };
    const auto first = [&](int64_t i) { return hg == 1 || i % hg == 0; };  // errors are raised once per tile

    Kv8Edge edge[NP];
    Kv8Paged paged[NP];
    Kv8Slot slot[NP], cur[NP];
    const auto step1 = [&](int64_t i) {
#pragma unroll
        for (int p = 0; p < NP; ++p) edge[p] = kv8_edge(a, i < nstep && sr < a.rt, tile_of(i) * a.rt + sr, p * 16 + sj);
    };
    const auto step2 = [&](int64_t i) {
#pragma unroll
        for (int p = 0; p < NP; ++p) paged[p] = kv8_paged(a, edge[p], lane < 16 && first(i), checked);
    };
    const auto step3 = [&](int64_t i) {
#pragma unroll
        for (int p = 0; p < NP; ++p) slot[p] = kv8_slot(a, paged[p], lane < 16 && first(i));
    };
    // column n of step i: row n >> g_shift of the tile, head g0 + (n & (2^g_shift - 1))
    const auto column = [&](int64_t i, int n, int64_t &row, int &head) {
        const int64_t ti = tile_of(i);
        row = ti * a.rt + (n >> a.g_shift);
        head = (int)(i - ti * hg) * 8 + (n & ((1 << a.g_shift) - 1));
        return (n >> a.g_shift) < a.rt && row < a.rows && head < a.G;
    };
    const auto issue = [&](int64_t i, int st) {  // `slot` is step i's
        if (i < nstep) {
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int y = 0; y < CH / 2; ++y) {
                    const int x = lane + 32 * y, r = x / CH, col = x - r * CH;
                    const uint32_t row = __shfl_sync(FULL, slot[p].row, r);
                    const bool on = row != Kv8Slot::NONE;  // an inactive slot's rows are zeros
                    const size_t at = on ? (size_t)row * D + col * 16 : 0;
                    const int fk = D == 128 ? (r & 1) * 4 : 0, fv = D == 128 ? ((r >> 1) & 3) * 2 : (r >> 1) & 3;
                    cp_async16_zfill(&sm.k[st][p][r * D + (col ^ fk) * 16], a.c.kq + at, on);
                    cp_async16_zfill(&sm.v[st][p][r * D + (col ^ fv) * 16], a.c.vq + at, on);
                }
#pragma unroll
            for (int y = 0; y < QC / 4; ++y) {
                const int x = lane + 32 * y, n = x / QC, col = x - n * QC;
                int64_t row;
                int head;
                const bool in = column(i, n, row, head);
                cp_async16_zfill(&sm.q[st][n * D + (col ^ (n & 1)) * VEC],
                                 (const T *)a.q + (in ? ((size_t)row * a.G + head) * D + col * VEC : 0), in);
            }
        }
        cp_async_commit();
    };

    step1(it);
    step2(it);
    step3(it);
    issue(it, 0);
#pragma unroll
    for (int p = 0; p < NP; ++p) cur[p] = slot[p];
    step1(it + stride);
    step2(it + stride);
    step3(it + stride);
    step1(it + 2 * stride);
    step2(it + 2 * stride);
    step1(it + 3 * stride);
    for (int st = 0; it < nstep; it += stride, st ^= 1) {
        __syncwarp();  // every lane is done with the other stage
        issue(it + stride, st ^ 1);
        Kv8Slot after[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) after[p] = slot[p];
        step3(it + 2 * stride);
        step2(it + 3 * stride);
        step1(it + 4 * stride);
        cp_async_wait<1>();
        __syncwarp();  // the step's rows are complete

        // ---- queries: column g, scaled into fp16 --------------------------------------------------
        uint32_t qh[KS][2], ql[SPLIT ? KS : 1][2];
        float qdown;
        {
            uint4 x[NK][QV];
            float big = 0.0f;
#pragma unroll
            for (int e = 0; e < NK; ++e)
#pragma unroll
                for (int y = 0; y < QV; ++y) {
                    x[e][y] = *reinterpret_cast<const uint4 *>(
                        &sm.q[st][g * D + (((e * 64 + c * 16) / VEC + y) ^ (g & 1)) * VEC]);
                    float f[VEC];
                    unpack<T>(x[e][y], f);
#pragma unroll
                    for (int z = 0; z < VEC; ++z) big = fmaxf(big, fabsf(f[z]));
                }
            big = fmaxf(big, __shfl_xor_sync(FULL, big, 1));
            big = fmaxf(big, __shfl_xor_sync(FULL, big, 2));
            const int e2 = min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 127);
            const float up = __uint_as_float((uint32_t)(127 + 14 - e2) << 23);
            qdown = __uint_as_float((uint32_t)(127 - 14 + e2) << 23) * a.sl2;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float f[VEC];
                unpack<T>(x[ks >> 2][(ks & 3) * 4 / VEC], f);
                const int o = (ks & 3) * 4 % VEC;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float lo = f[o + 2 * y] * up, hi = f[o + 2 * y + 1] * up;
                    qh[ks][y] = pack_half2(lo, hi);
                    if constexpr (SPLIT) ql[ks][y] = pack_rest(lo, hi, qh[ks][y]);
                }
            }
        }
        // ---- scores of slots g, g + 8 for columns 2c, 2c + 1 ------------------------------------
        float z[NP][4];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            uint4 kr[2][NK];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < NK; ++e)
                    kr[y][e] = *reinterpret_cast<const uint4 *>(
                        &sm.k[st][p][(g + 8 * y) * D + ((c + 4 * e) ^ (D == 128 ? (g & 1) * 4 : 0)) * 16]);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[p][e] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint32_t w0 = (&kr[0][ks >> 2].x)[ks & 3], w1 = (&kr[1][ks >> 2].x)[ks & 3];
                const uint32_t a0 = half2_lo(w0), a2 = half2_hi(w0);
                const uint32_t a1 = half2_lo(w1), a3 = half2_hi(w1);
                mma_f16(z[p], a0, a1, a2, a3, qh[ks][0], qh[ks][1]);
                if constexpr (SPLIT) mma_f16(z[p], a0, a1, a2, a3, ql[ks][0], ql[ks][1]);
            }
        }
        const float qd[2] = {__shfl_sync(FULL, qdown, 8 * c), __shfl_sync(FULL, qdown, 8 * c + 4)};
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, mu[2] = {0.0f, 0.0f}, vs[NP][2];
        bool see[NP][4];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const float mylw = lg2(cur[p].w);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = g + 8 * s;
                const bool on = __shfl_sync(FULL, cur[p].row, k) != Kv8Slot::NONE;
                const float ks = __shfl_sync(FULL, cur[p].ks, k), lw = __shfl_sync(FULL, mylw, k);
                vs[p][s] = __shfl_sync(FULL, cur[p].vs, k);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    see[p][2 * s + e] = on && (k >> ssh) == ((2 * c + e) >> a.g_shift);
                    z[p][2 * s + e] = see[p][2 * s + e] ? fmaf(z[p][2 * s + e], qd[e] * ks, lw) : -INFINITY;
                    m[e] = fmaxf(m[e], z[p][2 * s + e]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(FULL, m[e], o));
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = ex2_ftz(z[p][e] - (m[e & 1] == -INFINITY ? 0.0f : m[e & 1]));
                l[e & 1] += x;
                z[p][e] = see[p][e] ? x * vs[p][e >> 1] : 0.0f;
                mu[e & 1] = fmaxf(mu[e & 1], z[p][e]);
            }
        float up[2], inv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l[e] += __shfl_xor_sync(FULL, l[e], o);
                mu[e] = fmaxf(mu[e], __shfl_xor_sync(FULL, mu[e], o));
            }
            const int e2 = min(max((int)(__float_as_uint(mu[e]) >> 23) - 127, -100), 127);
            up[e] = __uint_as_float((uint32_t)(127 + 14 - e2) << 23);
            // an empty row is 0, a NaN stays
            inv[e] = l[e] == 0.0f ? 0.0f : __uint_as_float((uint32_t)(127 - 14 + e2) << 23) / l[e];
        }
        // ---- output ---------------------------------------------------------------------------------
        float acc[D / 16][4];
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            uint32_t vr[4][VW];  // slots 2c, 2c+1, 2c+8, 2c+9: columns g * (D/8) ..
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int r = 2 * c + (y & 1) + 8 * (y >> 1);
                if constexpr (VW == 4) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(&sm.v[st][p][r * D + (g ^ (((r >> 1) & 3) * 2)) * 16]);
                    vr[y][0] = x.x, vr[y][1] = x.y, vr[y][2] = x.z, vr[y][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(
                        &sm.v[st][p][r * D + ((g >> 1) ^ ((r >> 1) & 3)) * 16 + (g & 1) * 8]);
                    vr[y][0] = x.x, vr[y][1] = x.y;
                }
            }
            const float p0 = z[p][0] * up[0], p1 = z[p][1] * up[1], p2 = z[p][2] * up[0], p3 = z[p][3] * up[1];
            const uint32_t h0 = pack_half2(p0, p1), h1 = pack_half2(p2, p3);
            const uint32_t b0 = transpose8x8(h0), b1 = transpose8x8(h1);
            const uint32_t r0 = transpose8x8(pack_rest(p0, p1, h0)), r1 = transpose8x8(pack_rest(p2, p3, h1));
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
                const uint32_t x = __byte_perm(vr[0][j >> 1], vr[1][j >> 1], sel);
                const uint32_t y = __byte_perm(vr[2][j >> 1], vr[3][j >> 1], sel);
                const uint32_t a0 = half2_lo(x), a1 = half2_hi(x);
                const uint32_t a2 = half2_lo(y), a3 = half2_hi(y);
                mma_f16(acc[j], a0, a1, a2, a3, b0, b1);
                mma_f16(acc[j], a0, a1, a2, a3, r0, r1);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            int64_t row;
            int head;
            if (!column(it, 2 * c + e, row, head)) continue;
            const size_t ro = (size_t)row * a.G + head;  // row of o: (b, x, query head)
            T *dst = (T *)a.o + ro * D + g * (D / 8);
#pragma unroll
            for (int y = 0; y < D / 8 / VEC; ++y) {
                float f[VEC];
#pragma unroll
                for (int x = 0; x < VEC; ++x) {
                    const int d = y * VEC + x;  // column g * (D/8) + d of the output
                    f[x] = acc[d >> 1][(d & 1) * 2 + e] * inv[e];
                }
                *reinterpret_cast<uint4 *>(dst + y * VEC) = pack<T>(f);
            }
            if (a.lse && g == 0) a.lse[ro] = l[e] == 0.0f ? -INFINITY : (m[e] + lg2(l[e])) * LN2;
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) cur[p] = after[p];
    }
}

}  // namespace gm
