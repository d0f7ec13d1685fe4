// gm_window_umma.cuh - the windowed attention's bf16 kernels, on the tensor cores (tcgen05).
//
// Forward. One CTA works on two tiles of 128 query rows that share their keys: two heads of one
// group over the same rows (groups of even size), or one head's next 256 rows. Per key block of
// 128 and tile: S = Q K^T into TMEM; one thread per query row reads its 128 scores, keeps the
// running maximum and sum, and writes P as bf16 over S; O += P V with P as the TMEM operand. While
// one tile's rows are in the softmax, the tensor cores work on the other's.
//   warps 0-3, 4-7  softmax of tile 0, 1 (and their output)
//   warp 8          TMA loads: Q once, then K and V through separate stages
//   warp 9          MMA issue
// A thread reads its scores twice, 32 columns at a time, once for the maximum and once for the
// exponentials: 128 of them kept in registers spill, and TMEM has the bandwidth.
// P is handed over in two halves, so that the first half's products run under the second half's
// exponentials.
// TMEM: S0, S1 (128 columns each), O0, O1 (D columns each).
//
// The running maximum is allowed to lag: O is rescaled only when a row's maximum has grown by
// more than 2^8 since the last time (P then stays below 2^8, far inside fp32's and bf16's range),
// so O rarely leaves TMEM before the end. Key blocks are the two ranges of gm_window.cuh; a block
// narrower than 128 keys (a few sinks) takes only as many 32-column pieces as it has keys.
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

constexpr int UW = 128;                 // rows of a tile, keys of a block
constexpr int UATOM = UW * 128;         // bytes of one 64-column block of a tile

template <int D> struct WinFwdGeom {
    static constexpr int NA = D / 64;
    static constexpr int TILE = NA * UATOM;           // bytes of one 128 x D tile
    static constexpr int NST = D == 128 ? 2 : 4;      // stages of K and of V
    static constexpr int OFF_K = 2 * TILE;
    static constexpr int OFF_V = OFF_K + NST * TILE;
    static constexpr int OFF_BAR = OFF_V + NST * TILE;
    static constexpr int NBAR = 2 + 4 * NST + 2 + 4 + 2 + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
    static constexpr int THREADS = 320;
};

// Work items of the 128-row kernels: pairs of tiles.
struct WinPairs {
    int per;      // pairs of one (sequence, block): B * hkv * G/2, or B * hq
    bool heads;   // the pair is two heads of the group (else two row blocks of one head)
};

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

__device__ __forceinline__ void named_sync(int id, int count)
{
    asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(count) : "memory");
}

template <int D>
__global__ void __launch_bounds__(WinFwdGeom<D>::THREADS, 1)
win_fwd_umma_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmo, WinArgs a,
                    WinPairs wp)
{
    using Geo = WinFwdGeom<D>;
    constexpr int NA = Geo::NA, NST = Geo::NST, TILE = Geo::TILE;
    extern __shared__ __align__(1024) uint8_t wdsm[];
    const uint32_t raw = smem_u32(wdsm);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *sm = wdsm + (base - raw);
    const uint32_t sq = base, sk = base + Geo::OFF_K, sv = base + Geo::OFF_V, sb = base + Geo::OFF_BAR;
    const uint32_t q_full = sb, tail = sb + 8, k_full = sb + 16, k_empty = k_full + 8 * NST;
    const uint32_t v_full = k_empty + 8 * NST, v_empty = v_full + 8 * NST, s_full = v_empty + 8 * NST;
    const uint32_t p_full = s_full + 16, o_full = p_full + 32, mma_done = o_full + 16, tslot = mma_done + 8;
    const uint32_t *tslot_p = reinterpret_cast<const uint32_t *>(sm + Geo::OFF_BAR + Geo::NBAR * 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blk = a.nblk - 1 - (int)(blockIdx.x / (unsigned)wp.per);  // longest prefixes first
    int x = (int)(blockIdx.x % (unsigned)wp.per);
    int b, h, hq0, hq1, i0, i1, rows;
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
    const int len = win_len(a, b);
    const KeyBlocks kb(i0, rows, len, a.window, a.sinks, UW);
    const int nt = kb.na + kb.nb;

    if (nt == 0) {  // nothing but padding: rows of zeros
        for (int y = threadIdx.x; y < 2 * UW * (D / 8); y += Geo::THREADS) {
            const int r = y / (D / 8), c = y - r * (D / 8);
            const int i = (r < UW ? i0 : i1) + (r & (UW - 1)), hq = r < UW ? hq0 : hq1;
            if (i < a.n) {
                const size_t row = ((size_t)b * a.n + i) * a.hq + hq;
                *reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.o + row * D + c * 8) = make_uint4(0, 0, 0, 0);
                if (c == 0 && a.lse) a.lse[row] = -INFINITY;
            }
        }
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
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
            mbar_init(o_full + 8 * t, 1);
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
        const auto load = [&](uint32_t dst, const CUtensorMap *m, int head, int row, uint32_t bar) {
#pragma unroll
            for (int at = 0; at < NA; ++at) umma::tma_load_4d(dst + at * UATOM, m, at * 64, head, row, b, bar);
        };
        if (lane == 0) {
            mbar_arrive_expect(q_full, 2 * TILE);
            load(sq, &tmq, hq0, i0, q_full);
            load(sq + TILE, &tmq, hq1, i1, q_full);
        }
        bool ok = true;
        for (int j = 0; ok && j < nt; ++j) {
            const int s = j % NST, t0 = kb.start(j, UW);
            if (lane == 0 && j >= NST) ok = mbar_wait(k_empty + 8 * s, ((j / NST) - 1) & 1);
            if (lane == 0 && ok) {
                mbar_arrive_expect(k_full + 8 * s, TILE);
                load(sk + s * TILE, &tmk, h, t0, k_full + 8 * s);
            }
            if (lane == 0 && ok && j >= NST) ok = mbar_wait(v_empty + 8 * s, ((j / NST) - 1) & 1);
            ok = __shfl_sync(FULL, ok, 0);
            if (!ok) break;
            const bool fix = t0 + UW > len && len < a.n;  // the last block alone
            const uint32_t bar = fix ? tail : v_full + 8 * s;
            if (lane == 0) {
                mbar_arrive_expect(bar, TILE);
                load(sv + s * TILE, &tmv, h, t0, bar);
            }
            if (fix) {
                ok = __all_sync(FULL, mbar_wait(tail, 0));
                uint4 *tile = reinterpret_cast<uint4 *>(sm + Geo::OFF_V + s * TILE);
                const int first = max(len - t0, 0);
                for (int y = lane; ok && y < NA * (UW - first) * 8; y += 32) {
                    const int at = y / ((UW - first) * 8), z = y - at * ((UW - first) * 8);
                    tile[at * (UATOM / 16) + first * 8 + z] = make_uint4(0, 0, 0, 0);
                }
                umma::fence_proxy_async();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(v_full + 8 * s);
            }
        }
        // copies still in flight land before the CTA ends: the MMA warp waits for every one
        // that it uses; after a wait that gave up, this drains the rest
        if (lane == 0 && !ok) {
            mbar_wait(q_full, 0);
            for (int s = 0; s < NST; ++s) {
                mbar_wait(k_full + 8 * s, 0);
                mbar_wait(v_full + 8 * s, 0);
            }
        }
    } else if (warp == 9) {
        // ---- MMAs -------------------------------------------------------------------------
        if (lane == 0) {
            const auto scores = [&](int t, int j, int n) {  // S_t = Q_t K_j^T
                const uint32_t idesc = umma::idesc_bf16_f32(UW, n);
                const int s = j % NST;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = (ks / 4) * UATOM + (ks % 4) * 32;
                    umma::mma_bf16(tmem + t * UW, umma::sdesc_sw128_kmajor(sq + t * TILE + off),
                                   umma::sdesc_sw128_kmajor(sk + s * TILE + off), idesc, ks > 0);
                }
            };
            const auto width = [&](int j) { return (kb.end(j, UW) - kb.start(j, UW) + 31) & ~31; };
            constexpr uint32_t idesc_pv = umma::idesc_bf16_f32_bmn(UW, D);
            bool ok = mbar_wait(q_full, 0) && mbar_wait(k_full, 0);
            if (ok) {
                umma::fence_after_sync();
                const int n = width(0);
                scores(0, 0, n);
                umma::commit(s_full);
                scores(1, 0, n);
                umma::commit(s_full + 8);
                umma::commit(k_empty);
            }
            for (int j = 0; ok && j < nt; ++j) {
                const int s = j % NST, w = width(j);
                const int n = j + 1 < nt ? width(j + 1) : 0;
                ok = mbar_wait(v_full + 8 * s, (j / NST) & 1);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (ok) ok = mbar_wait(p_full + 16 * t + 8 * half, j & 1);
                        if (!ok) break;
                        umma::fence_after_sync();
                        for (int ks = half * 4; ks < min(w / 16, half * 4 + 4); ++ks)  // O_t += P_t V_j
                            umma::mma_bf16_ta(tmem + 2 * UW + t * D, tmem + t * UW + ks * 8,
                                              umma::sdesc_sw128_mnmajor(sv + s * TILE + ks * 2048, UATOM), idesc_pv,
                                              j > 0 || ks > 0);
                    }
                    if (!ok) break;
                    if (t == 1) umma::commit(v_empty + 8 * s);
                    if (n > 0) {
                        if (t == 0) {
                            ok = mbar_wait(k_full + 8 * ((j + 1) % NST), ((j + 1) / NST) & 1);
                            if (!ok) break;
                            umma::fence_after_sync();
                        }
                        scores(t, j + 1, n);
                        umma::commit(s_full + 8 * t);
                        if (t == 1) umma::commit(k_empty + 8 * ((j + 1) % NST));
                    } else {
                        umma::commit(o_full + 8 * t);
                    }
                }
            }
            // every MMA issued has completed before the CTA releases its tensor memory
            umma::commit(mma_done);
            mbar_wait(mma_done, 0);
        }
    } else {
        // ---- softmax: thread = query row = TMEM lane ----------------------------------------
        const int t = warp >> 2, r = (warp & 3) * 32 + lane;
        const int it = t ? i1 : i0, i = it + r, hq = t ? hq1 : hq0, r0 = it + (warp & 3) * 32;
        const bool valid = i < len;
        const float sl2 = a.scale;  // log2(e) folded in by the host, never 0
        const float hide = sl2 > 0.0f ? -INFINITY : INFINITY;
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = trow + t * UW, to = trow + 2 * UW + t * D;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            ok = __all_sync(FULL, mbar_wait(s_full + 8 * t, j & 1));
            if (!ok) break;
            umma::fence_after_sync();
            const int t0 = kb.start(j, UW), t1 = kb.end(j, UW), nch = (t1 - t0 + 31) / 32;
            const bool whole = t1 - t0 == UW && t1 - 1 <= it && it + UW <= len &&
                               (t0 > it + UW - 1 - a.window || t1 <= a.sinks);
            // ---- maximum over the visible columns ------------------------------------------------
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
                    }
                    maximum(s[0]);
                }
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
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        umma::tmem_ld32(to + c * 32, o);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        umma::tmem_st32(to + c * 32, o);
                    }
                }
            }
            // ---- P = 2^(sl2 S - m), piece c over scores of pieces already read --------------------
            const float nm = m == -INFINITY ? 0.0f : -m;
            const float2 sl22 = make_float2(sl2, sl2), nm2 = make_float2(nm, nm);
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            const auto exponentials = [&](const uint32_t(&y)[32], uint32_t(&p)[16], uint32_t mask, bool masked) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float2 x = make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]));
                    x = __ffma2_rn(x, sl22, nm2);
                    x.x = ex2_ftz(x.x);
                    x.y = ex2_ftz(x.y);
                    if (masked) {
                        x.x = (mask >> (2 * e)) & 1 ? x.x : 0.0f;
                        x.y = (mask >> (2 * e + 1)) & 1 ? x.y : 0.0f;
                    }
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
                    exponentials(s[c & 1], p, 0, false);
                    umma::tmem_st16(ts + c * 16, p);
                    if (c & 1) hand_over(c >> 1);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    const Piece piece = key_piece(r0, t0 + c * 32, t1, len, a.window, a.sinks);
                    if (piece != Piece::none) {
                        umma::tmem_ld32(ts + c * 32, s[0]);
                        umma::tmem_wait_ld32(s[0]);
                        if (piece == Piece::all)
                            exponentials(s[0], p, 0, false);
                        else
                            exponentials(s[0], p, column_mask(c * 32, lo, hi, a.sinks - t0), true);
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
        // ---- output -----------------------------------------------------------------------
        if (ok) ok = __all_sync(FULL, mbar_wait(o_full + 8 * t, 0));
        if (ok) {
            umma::fence_after_sync();
            const float inv = valid ? 1.0f / l : 0.0f;
            // the tile's Q rows are free now: the output goes there and out by TMA
            uint8_t *row = sm + t * TILE + r * 128;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                umma::tmem_ld32(to + c * 32, o);
                umma::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        w[y] = valid ? bf16_pair(__uint_as_float(o[e * 8 + 2 * y]) * inv,
                                                 __uint_as_float(o[e * 8 + 2 * y + 1]) * inv)
                                     : 0u;
                    *reinterpret_cast<uint4 *>(row + (c / 2) * UATOM + ((((c & 1) * 4 + e) ^ (r & 7)) * 16)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (a.lse && i < a.n)
                a.lse[((size_t)b * a.n + i) * a.hq + hq] = valid ? (m + log2f(l)) * LN2 : -INFINITY;
            umma::fence_proxy_async();
        }
        named_sync(1 + t, UW);
        if ((threadIdx.x & (UW - 1)) == 0 && ok && it < a.n) {
#pragma unroll
            for (int at = 0; at < NA; ++at)
                umma::tma_store_4d(&tmo, sq + t * TILE + at * UATOM, at * 64, hq, it, b);
            umma::tma_store_commit();
            umma::tma_store_wait_read();
        }
    }

    umma::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, 512);
    }
}

}  // namespace gm
