// gm_window_umma.cuh - the windowed attention's bf16 kernels, on the tensor cores (tcgen05).
//
// Forward. A CTA works on two tiles of 128 query rows that share their keys: two heads of one
// group over the same rows (groups of even size), or one head's next 256 rows. Per block of 128
// keys and tile: S = Q K^T into TMEM; one thread per query row reads its scores, keeps the running
// maximum and sum, and writes P as bf16 over S; O += P V with P as the TMEM operand. While one
// tile's rows are in the softmax, the tensor cores work on the other's. P is rounded because both
// operands of a product have one type, and V comes in bf16: at most half a step, 2^-8, of a weight.
// Against 64 bits the output is off by 0.0022 in the 2-norm at window 512, with P in fp32 it would be by
// 0.0016 (the output's own rounding).
//   warps 0-3, 4-7  softmax of tile 0, 1 (and their output)
//   warp 8          TMA loads: Q per item, K and V through their stages
//   warp 9          MMA issue
// TMEM: S0, S1 (128 columns each), O0, O1 (D columns each).
//
// A thread reads its scores twice, 32 columns at a time, once for the maximum and once for the
// exponentials: 128 of them kept in registers spill, or with the registers split among the
// warpgroups (56 and 224) do not but take 222 us against 205 (window 512). P is handed over
// in two halves, so that the first half's products run under the second half's exponentials.
// With the softmax replaced by nothing the kernel takes 738 us for n = 16384 (16 heads, full), with
// it 935: the products (at 90 % of the measured bf16 rate when alone) bound it, then the wait for
// each block's exponentials (16 per SM and cycle). A quarter of them therefore runs on the FMA pipe
// (ex2_poly; the idea was published in 2025 for attention on this generation of GPUs), in blocks that
// are seen whole: window 512 224 -> 206 us, n = 16384 1063 -> 1002 us in turn; an eighth gives 223 and
// 1046, three eighths 206 and 1031. Blocks of 64 keys with two score buffers per tile remove the wait
// but run the products at N = 64, 976 us alone.
//
// The grid is one CTA per SM; each takes item after item (longest first, every second round in
// reverse order), so the next item's loads and first scores run under the output of the one
// before (window 512, B=8 n=4096: 276 us with a CTA per item, 240 us at that time).
//
// 16/8 heads, d=128, 4 sinks beside a window; back to back on the same tensors, in brackets a single
// call with a cold L2: B=8 n=4096 window 512 200 us (224), window 1024 307 us (314); B=1 n=16384 full
// 1030 us (960; back to back it runs at the power limit, 1.1 PFLOP/s). At window 1024 the tensor pipe is
// busy 47 % of the time, the exponential unit 34 %, the issue slots 38 %: what is left is the chain
// scores - maximum - exponentials - product of one tile, which the other tile covers only in part, and
// the blocks seen in part at both ends of a window.
//
// The running maximum (the online softmax of Milakov and Gimelshein, 2018) is allowed to lag, an idea
// published beside the one above: O is rescaled only when a row's maximum has grown by more than 2^8
// since the last time (P then stays below 2^8, far inside fp32's and bf16's range), so O rarely leaves
// TMEM before the end. Key blocks are the two ranges of gm_window.cuh; a block narrower than 128 keys (a few sinks) takes only as many 32-column pieces as it has keys, and
// pieces that none of a warp's rows sees are skipped. The path of blocks that are seen in part
// stays a rolled loop: unrolled like the other it costs more in instruction fetches than it saves
// (225 against 243 us).
//
// Rows at or past the sequence's end may hold anything: scores of such keys are masked by
// selection, and their rows of the V tile are zeroed in shared memory before the MMA (only a
// sequence's last key block can have any).
//
// Every wait is bounded (gm_common.cuh, mbar_wait).
#pragma once

#include <cuda.h>

#include "gm_common.cuh"
#include "gm_umma.cuh"
#include "gm_window.cuh"

namespace gm {

constexpr int UW = 128;                 // rows of a tile, keys of a block in the backward
constexpr int UATOM = UW * 128;         // bytes of one 64-column block of a tile
constexpr int FK = 128;                 // keys of a block in the forward
constexpr int FATOM = FK * 128;

template <int D> struct WinFwdGeom {
    static constexpr int NA = D / 64;
    static constexpr int TILE = NA * UATOM;           // bytes of one 128 x D tile
    static constexpr int KTILE = NA * FATOM;          // of a key block
    static constexpr int NST = D == 128 ? 2 : 4;      // stages of K and of V
    static constexpr int OFF_K = 2 * TILE;
    static constexpr int OFF_V = OFF_K + NST * KTILE;
    static constexpr int OFF_OUT = OFF_V + NST * KTILE;  // per tile: 64 columns of output on their way
    static constexpr int OFF_BAR = OFF_OUT + 2 * UATOM;
    static constexpr int NBAR = 3 + 4 * NST + 2 + 4 + 2 + 2 + 2 + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
    static constexpr int THREADS = 320;
    static_assert(SMEM > 114 * 1024, "one CTA per SM: a second would wait for TMEM columns");
};

// Work items of the 128-row kernels: pairs of tiles.
struct WinPairs {
    int per;      // pairs of one (sequence, block): B * hkv * G/2, or B * hq
    bool heads;   // the pair is two heads of the group (else two row blocks of one head)
    int64_t items;
};

// One pair of tiles and the keys it sees.
struct WinItem {
    int b, h, hq0, hq1, i0, i1, len, nt;
    KeyBlocks kb;
    __device__ __forceinline__ WinItem(const WinArgs &a, const WinPairs &wp, int64_t item, int bn)
        : kb(0, 0, 0, 1, 0, 1)
    {
        const int blk = a.nblk - 1 - (int)(item / wp.per);  // longest prefixes first
        const int x = (int)(item % wp.per);
        int rows;
        if (wp.heads) {
            const int hp = a.hq / 2;
            b = x / hp;
            hq0 = 2 * (x - b * hp);
            hq1 = hq0 + 1;
            i0 = i1 = blk * UW;
            rows = UW;
        } else {
            b = x / a.hq;
            hq0 = hq1 = x - b * a.hq;
            i0 = blk * 2 * UW;
            i1 = i0 + UW;
            rows = 2 * UW;
        }
        h = hq0 / a.G;
        len = win_len(a, b);
        kb = KeyBlocks(i0, rows, len, a.window, a.sinks, bn);
        nt = kb.na + kb.nb;
    }
};

// The item of round k for this CTA: rounds alternate their direction.
__device__ __forceinline__ int64_t win_round(int64_t k)
{
    return k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Columns c of [base, base + 32) with c <= hi and (c >= lo or c < sink), as a bit mask.
__device__ __forceinline__ uint32_t column_mask(int base, int lo, int hi, int sink)
{
    const auto below = [&](int x) {  // bits of columns < x
        x -= base;
        return x <= 0 ? 0u : (x >= 32 ? 0xffffffffu : (1u << x) - 1u);
    };
    return below(hi + 1) & (~below(lo) | below(sink));
}

// Whether rows [r0, r0 + 32) see all, some or none of the 32 keys from t on (keys end at t1).
enum class Piece { none, some, all };
__device__ __forceinline__ Piece key_piece(int r0, int t, int t1, int len, int window, int sinks)
{
    const int last = min(r0 + 31, len - 1);  // the last row that is one
    if (t >= t1 || t > last || (t + 31 <= r0 - window && t >= sinks)) return Piece::none;
    if (t + 31 < t1 && t + 31 <= r0 && r0 + 31 < len && (t > r0 + 31 - window || t + 31 < sinks)) return Piece::all;
    return Piece::some;
}

// Whole warp: zeroes rows [first, ROWS) of a ROWS x D tile.
template <int NA, int ROWS> __device__ __forceinline__ void zero_rows(uint8_t *tile, int first, int lane)
{
    const int per = (ROWS - first) * 8;
    for (int y = lane; y < NA * per; y += 32) {
        const int at = y / per, z = y - at * per;
        *reinterpret_cast<uint4 *>(tile + at * (ROWS * 128) + first * 128 + z * 16) = make_uint4(0, 0, 0, 0);
    }
}

// This thread's row of a TMEM accumulator (columns [c0, c1) of 32s), times f, as bf16 into a
// swizzled tile; zeros where `keep` is false.
__device__ __forceinline__ void stage_row(uint8_t *tile, uint32_t taddr, int r, int c0, int c1, float f, bool keep)
{
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
        uint32_t o[32];
        umma::tmem_ld32(taddr + c * 32, o);
        umma::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t x[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
                x[y] = keep ? bf16_pair(__uint_as_float(o[e * 8 + 2 * y]) * f, __uint_as_float(o[e * 8 + 2 * y + 1]) * f)
                            : 0u;
            *reinterpret_cast<uint4 *>(tile + (c / 2) * UATOM + r * 128 + ((((c & 1) * 4 + e) ^ (r & 7)) * 16)) =
                make_uint4(x[0], x[1], x[2], x[3]);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(WinFwdGeom<D>::THREADS, 1)
win_fwd_umma_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmo, WinArgs a,
                    WinPairs wp)
{
    using Geo = WinFwdGeom<D>;
    constexpr int NA = Geo::NA, NST = Geo::NST, TILE = Geo::TILE, KTILE = Geo::KTILE;
    extern __shared__ __align__(1024) uint8_t wdsm[];
    const uint32_t raw = smem_u32(wdsm);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *sm = wdsm + (base - raw);
    const uint32_t sq = base, sk = base + Geo::OFF_K, sv = base + Geo::OFF_V, sb = base + Geo::OFF_BAR;
    const uint32_t q_full = sb, q_empty = sb + 8, tail = sb + 16, k_full = sb + 24, k_empty = k_full + 8 * NST;
    const uint32_t v_full = k_empty + 8 * NST, v_empty = v_full + 8 * NST;
    const uint32_t s_full = v_empty + 8 * NST;                            // [tile]
    const uint32_t p_full = s_full + 16;                                  // [tile][half]
    const uint32_t pv_done = p_full + 32, o_empty = pv_done + 16, out_sync = o_empty + 16;  // [tile]
    const uint32_t mma_done = out_sync + 16, tslot = base + Geo::OFF_BAR + Geo::NBAR * 8;
    const uint32_t *tslot_p = reinterpret_cast<const uint32_t *>(sm + Geo::OFF_BAR + Geo::NBAR * 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(tail, 1);
#pragma unroll
        for (int s = 0; s < NST; ++s) {
            mbar_init(k_full + 8 * s, 1);
            mbar_init(k_empty + 8 * s, 1);
            mbar_init(v_full + 8 * s, 1);
            mbar_init(v_empty + 8 * s, 1);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + 8 * t, 1);
            mbar_init(p_full + 16 * t, UW);
            mbar_init(p_full + 16 * t + 8, UW);
            mbar_init(out_sync + 8 * t, UW);
            mbar_init(pv_done + 8 * t, 1);
            mbar_init(o_empty + 8 * t, UW);
        }
        mbar_init(mma_done, 1);
        mbar_init_fence();
    }
    if (warp == 9) umma::tmem_alloc(tslot, 512);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = *tslot_p;

    if (warp == 8) {
        // ---- loads ------------------------------------------------------------------------
        uint32_t kc = 0, fixes = 0;  // key blocks so far
        int qc = 0;                  // items with keys so far
        bool ok = true;
        for (int64_t k = 0; ok && k * gridDim.x < wp.items; ++k) {
            const int64_t item = win_round(k);
            if (item >= wp.items) continue;
            const WinItem w(a, wp, item, FK);
            if (w.nt == 0) continue;
            if (lane == 0 && qc > 0) ok = mbar_wait(q_empty, (qc - 1) & 1);
            ok = __shfl_sync(FULL, ok, 0);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect(q_full, 2 * TILE);
#pragma unroll
                for (int at = 0; at < NA; ++at) {
                    umma::tma_load_4d(sq + at * UATOM, &tmq, at * 64, w.hq0, w.i0, w.b, q_full);
                    umma::tma_load_4d(sq + TILE + at * UATOM, &tmq, at * 64, w.hq1, w.i1, w.b, q_full);
                }
            }
            ++qc;
            for (int j = 0; ok && j < w.nt; ++j, ++kc) {
                const uint32_t s = kc % NST, ph = kc / NST;
                const int t0 = w.kb.start(j, FK);
                if (lane == 0 && kc >= NST) ok = mbar_wait(k_empty + 8 * s, (ph - 1) & 1);
                if (lane == 0 && ok) {
                    mbar_arrive_expect(k_full + 8 * s, KTILE);
#pragma unroll
                    for (int at = 0; at < NA; ++at)
                        umma::tma_load_4d(sk + s * KTILE + at * FATOM, &tmk, at * 64, w.h, t0, w.b, k_full + 8 * s);
                }
                if (lane == 0 && ok && kc >= NST) ok = mbar_wait(v_empty + 8 * s, (ph - 1) & 1);
                ok = __shfl_sync(FULL, ok, 0);
                if (!ok) break;
                const bool fix = t0 + FK > w.len && w.len < a.n;  // the last block alone
                const uint32_t bar = fix ? tail : v_full + 8 * s;
                if (lane == 0) {
                    mbar_arrive_expect(bar, KTILE);
#pragma unroll
                    for (int at = 0; at < NA; ++at)
                        umma::tma_load_4d(sv + s * KTILE + at * FATOM, &tmv, at * 64, w.h, t0, w.b, bar);
                }
                if (fix) {
                    ok = __all_sync(FULL, mbar_wait(tail, fixes++ & 1));
                    if (ok) zero_rows<NA, FK>(sm + Geo::OFF_V + s * KTILE, max(w.len - t0, 0), lane);
                    umma::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0 && ok) mbar_arrive(v_full + 8 * s);
                }
            }
        }
        if (lane == 0 && !ok && qc > 0) {  // gave up: copies in flight land before the CTA ends (bounded)
            mbar_wait(q_full, (qc - 1) & 1);
            for (uint32_t y = kc > NST ? kc - NST : 0; y < kc; ++y) {
                mbar_wait(k_full + 8 * (y % NST), (y / NST) & 1);
                mbar_wait(v_full + 8 * (y % NST), (y / NST) & 1);
            }
        }
    } else if (warp == 9) {
        // ---- MMAs (the whole warp runs along, one lane issues) ----------------------------
        constexpr uint32_t idesc_pv = umma::idesc_bf16_f32_bmn(UW, D);
        const uint32_t lead = umma::elect_lead();
        const uint32_t q_lo = umma::sdesc_lo(sq, umma::KMAJOR), k_lo = umma::sdesc_lo(sk, umma::KMAJOR);
        const uint32_t v_lo = umma::sdesc_lo(sv, FATOM);
        uint32_t kc = 0;  // step 0 of the item, over all items
        int qc = 0;
        bool ok = true;
        for (int64_t k = 0; ok && k * gridDim.x < wp.items; ++k) {
            const int64_t item = win_round(k);
            if (item >= wp.items) continue;
            const WinItem w(a, wp, item, FK);
            if (w.nt == 0) continue;
            const auto width = [&](int j) { return (w.kb.end(j, FK) - w.kb.start(j, FK) + 31) & ~31; };
            const auto scores = [&](int t, int j) {  // S_t(j) = Q_t K_j^T
                const uint32_t y = kc + j, s = y % NST;
                const uint32_t idesc = umma::idesc_bf16_f32(UW, width(j));
                const uint32_t d = tmem + t * 128;
                const uint32_t al = q_lo + t * (TILE >> 4), bl = k_lo + s * (KTILE >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    umma::mma_ss(lead, d, al + (((ks / 4) * UATOM + (ks % 4) * 32) >> 4),
                                 bl + (((ks / 4) * FATOM + (ks % 4) * 32) >> 4), idesc, ks > 0);
                umma::commit_if(lead, s_full + 8 * t);
                if (t == 1) {
                    umma::commit_if(lead, k_empty + 8 * s);
                    if (j == w.nt - 1) umma::commit_if(lead, q_empty);
                }
            };
            ok = mbar_wait_warp(q_full, qc & 1) && mbar_wait_warp(k_full + 8 * (kc % NST), (kc / NST) & 1);
            if (!ok) break;
            umma::fence_after_sync();
            scores(0, 0);
            scores(1, 0);
            for (int j = 0; ok && j < w.nt; ++j) {
                const uint32_t y = kc + j, s = y % NST;
                const int wd = width(j);
                ok = mbar_wait_warp(v_full + 8 * s, (y / NST) & 1);
                if (ok && j + 1 < w.nt) ok = mbar_wait_warp(k_full + 8 * ((y + 1) % NST), ((y + 1) / NST) & 1);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (ok && j == 0 && qc > 0) ok = mbar_wait_warp(o_empty + 8 * t, (qc - 1) & 1);
                    const uint32_t d = tmem + 256 + t * D, bl = v_lo + s * (KTILE >> 4);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (ok) ok = mbar_wait_warp(p_full + 16 * t + 8 * half, y & 1);
                        if (!ok) break;
                        umma::fence_after_sync();
#pragma unroll
                        for (int ks = half * 4; ks < half * 4 + 4; ++ks)  // O_t += P_t V_j
                            if (ks < 2 || ks * 16 < wd)
                                umma::mma_ts(lead, d, tmem + t * 128 + ks * 8, bl + (ks * 2048 >> 4), idesc_pv, j > 0 || ks > 0);
                    }
                    if (!ok) break;
                    umma::commit_if(lead, pv_done + 8 * t);
                    if (t == 1) umma::commit_if(lead, v_empty + 8 * s);
                    if (j + 1 < w.nt) scores(t, j + 1);
                }
            }
            kc += w.nt;
            ++qc;
        }
        // every MMA issued has completed before the CTA releases its tensor memory
        umma::commit_if(lead, mma_done);
        mbar_wait_warp(mma_done, 0);
    } else {
        // ---- softmax: thread = query row = TMEM lane ----------------------------------------
        const int t = warp >> 2, r = (warp & 3) * 32 + lane;
        const float sl2 = a.scale;  // log2(e) folded in by the host, never 0
        const float hide = sl2 > 0.0f ? -INFINITY : INFINITY;
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t to = trow + 256 + t * D;
        const bool leader = (threadIdx.x & (UW - 1)) == 0;
        uint32_t kc = 0, syncs = 0;
        bool ok = true;
        // the tile's 128 threads meet (a barrier with a limit: a warp that gave up never comes)
        const auto meet = [&]() {
            mbar_arrive(out_sync + 8 * t);
            return __all_sync(FULL, mbar_wait(out_sync + 8 * t, syncs++ & 1)) != 0;
        };
        for (int64_t k = 0; ok && k * gridDim.x < wp.items; ++k) {
            const int64_t item = win_round(k);
            if (item >= wp.items) continue;
            const WinItem w(a, wp, item, FK);
            const int len = w.len, it = t ? w.i1 : w.i0, i = it + r, hq = t ? w.hq1 : w.hq0, r0 = it + (warp & 3) * 32;
            const bool valid = i < len;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < w.nt; ++j) {
                const uint32_t y = kc + j;
                ok = mbar_wait_warp(s_full + 8 * t, y & 1);
                if (!ok) break;
                umma::fence_after_sync();
                const uint32_t ts = trow + t * 128;
                const int t0 = w.kb.start(j, FK), t1 = w.kb.end(j, FK), nch = (t1 - t0 + 31) / 32;
                const bool whole = t1 - t0 == FK && t1 - 1 <= r0 && r0 + 32 <= len &&
                                   (t0 > r0 + 31 - a.window || t1 <= a.sinks);
                // ---- maximum over the visible columns ------------------------------------------
                float m4[4] = {hide, hide, hide, hide};
                const auto maximum = [&](const uint32_t(&x)[32]) {
                    if (sl2 > 0.0f) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            m4[(e >> 1) & 3] = fmaxf(fmaxf(m4[(e >> 1) & 3], __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) m4[e & 3] = fminf(m4[e & 3], __uint_as_float(x[e]));
                    }
                };
                // columns the row sees: c <= hi and (c >= lo or c < sinks - t0)
                const int hi = valid ? min(i, t1 - 1) - t0 : -1, lo = i - a.window + 1 - t0;
                uint32_t s[2][32];
                if (whole) {
                    umma::tmem_ld32(ts, s[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        umma::tmem_wait_ld32(s[c & 1]);
                        if (c < 3) umma::tmem_ld32(ts + (c + 1) * 32, s[(c + 1) & 1]);
                        maximum(s[c & 1]);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < nch; ++c) {
                        const Piece piece = key_piece(r0, t0 + c * 32, t1, len, a.window, a.sinks);
                        if (piece == Piece::none) continue;
                        umma::tmem_ld32(ts + c * 32, s[0]);
                        umma::tmem_wait_ld32(s[0]);
                        if (piece == Piece::some) {
                            const uint32_t mask = column_mask(c * 32, lo, hi, a.sinks - t0);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((mask >> e) & 1)) s[0][e] = __float_as_uint(hide);
                            umma::tmem_st32(ts + c * 32, s[0]);  // for the second reading
                        }
                        maximum(s[0]);
                    }
                    umma::tmem_wait_st();
                }
                float mx = sl2 > 0.0f ? fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]))
                                      : fminf(fminf(m4[0], m4[1]), fminf(m4[2], m4[3]));
                mx *= sl2;
                const bool grow = mx > m + 8.0f;
                if (__any_sync(FULL, grow)) {
                    const float f = grow ? ex2_ftz(m - mx) : 1.0f;  // the first visible block: 2^-inf = 0
                    if (grow) m = mx;
                    l *= f;
                    if (j > 0) {
                        // S_t(j) was issued after P_t(j-1) V, so O_t is at rest until this block's P
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            umma::tmem_ld16(to + c * 16, o);
                            umma::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            umma::tmem_st16(to + c * 16, o);
                        }
                    }
                }
                // ---- P = 2^(sl2 S - m), piece c over scores of pieces already read --------------
                const float nm = m == -INFINITY ? 0.0f : -m;
                const float2 sl22 = make_float2(sl2, sl2), nm2 = make_float2(nm, nm);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                // a hidden score is an infinity of the sign that gives 2^-inf = 0 (not by ex2_poly)
                const auto exponentials = [&](const uint32_t(&v)[32], uint32_t(&p)[16], bool all) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 x = make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                        x = __ffma2_rn(x, sl22, nm2);
                        x = all ? ex2_pair<4>(x, e) : ex2_pair<0>(x, e);
                        sum[e & 1] = __fadd2_rn(sum[e & 1], x);
                        p[e] = bf16_pair(x.x, x.y);
                    }
                };
                const auto hand_over = [&](int half) {  // half of the block is ready for the tensor cores
                    umma::tmem_wait_st();
                    umma::fence_before_sync();
                    mbar_arrive(p_full + 16 * t + 8 * half);
                };
                uint32_t p[16];
                if (whole) {
                    umma::tmem_ld32(ts, s[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        umma::tmem_wait_ld32(s[c & 1]);
                        if (c < 3) umma::tmem_ld32(ts + (c + 1) * 32, s[(c + 1) & 1]);
                        exponentials(s[c & 1], p, true);
                        umma::tmem_st16(ts + c * 16, p);
                        if (c & 1) hand_over(c >> 1);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        if (key_piece(r0, t0 + c * 32, t1, len, a.window, a.sinks) != Piece::none) {
                            umma::tmem_ld32(ts + c * 32, s[0]);
                            umma::tmem_wait_ld32(s[0]);
                            exponentials(s[0], p, false);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) p[e] = 0;
                        }
                        if (c < nch) umma::tmem_st16(ts + c * 16, p);
                        if (c & 1) hand_over(c >> 1);
                    }
                }
                sum[0] = __fadd2_rn(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
            }
            kc += w.nt;
            if (!ok) break;
            // ---- output: 64 columns at a time through the tile's buffer, out by TMA ----------------
            if (w.nt > 0) {
                ok = mbar_wait_warp(pv_done + 8 * t, (kc - 1) & 1);
                if (!ok) break;
                umma::fence_after_sync();
            }
            const float inv = valid ? 1.0f / l : 0.0f;
            uint8_t *out = sm + Geo::OFF_OUT + t * UATOM;
#pragma unroll 1
            for (int at = 0; at < NA; ++at) {
                if (leader) umma::tma_store_wait_read();
                ok = meet();  // the buffer is free
                if (!ok) break;
                stage_row(out - at * UATOM, to, r, at * 2, at * 2 + 2, inv, valid);
                if (at == NA - 1 && w.nt > 0) {  // O has been read
                    umma::fence_before_sync();
                    mbar_arrive(o_empty + 8 * t);
                }
                umma::fence_proxy_async();
                ok = meet();
                if (!ok) break;
                if (leader && it < a.n) {
                    umma::tma_store_4d(&tmo, base + Geo::OFF_OUT + t * UATOM, at * 64, hq, it, w.b);
                    umma::tma_store_commit();
                }
            }
            if (a.lse && i < a.n)
                a.lse[((size_t)w.b * a.n + i) * a.hq + hq] = valid ? (m + log2f(l)) * LN2 : -INFINITY;
        }
        if (leader) umma::tma_store_wait_read();
    }

    umma::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, 512);
    }
}

}  // namespace gm
