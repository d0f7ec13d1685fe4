// gm_window_bwd_umma.cuh - the windowed attention's bf16 backward, on the tensor cores (tcgen05).
//
// Two kernels, so that every gradient is summed by one CTA in a fixed order and written once (no
// atomics, no fp32 buffer in HBM), at the price of computing S and dP twice: seven products per
// pair of blocks where a single kernel with atomics has five.
//
//   dq    one CTA per 128 query rows of a head, over the key blocks they see. TMEM lane = query:
//         S = Q K^T and dP = dO V^T land in TMEM, the threads turn them into
//         dS = P (dP - delta), P = 2^(sl2 S + nl), written as bf16 over dP, and dQ += dS K takes
//         it from there. dP has two buffers, S one that is free again once read, so the tensor
//         cores run a block ahead of the threads.
//   dkv   one CTA per 128 keys of a KV head, over the query blocks that see them and the group's
//         heads. TMEM lane = key: S^T = K Q^T, dP^T = V dO^T; P^T goes over S^T for dV += P^T dO,
//         dS^T over dP^T for dK += dS^T Q. The MMAs of a step run in the order dV(j), S(j+1),
//         dK(j), dP(j+1): the threads compute P(j+1) under dK(j) and dP(j+1), and dS(j+1) under
//         dV(j+1) and S(j+2).
//
// In both, two groups of four warps share the 128 lanes and take half of the columns each, each
// keeping its bf16 results inside its own half of the fp32 tile. nl = -lse log2(e) and
// delta = <dout, o> come from a pass over o and dout, laid out [B, hq, npad] with npad a
// multiple of 128; rows at or past the sequence's end have nl = -inf (P = 0) and delta = 0.
// Such rows of the tiles are zeroed in shared memory where a product sums over them.
//
// Every wait is bounded (gm_common.cuh, mbar_wait).
#pragma once

#include "gm_window_umma.cuh"

namespace gm {

struct WinBwdArgs {
    WinArgs w;          // w.scale: scale * log2(e) (never 0)
    float scale;
    const float *nl;    // [B, hq, npad]
    const float *ndelta;  // -delta
    int npad;
};

template <int D> struct WinBwdGeom {
    static constexpr int NA = D / 64;
    static constexpr int TILE = NA * UATOM;
    static constexpr int N3 = 3, N2 = 2;               // stages of the two streamed operands
    static constexpr int OFF_3 = 2 * TILE;             // after the two resident tiles
    static constexpr int OFF_2 = OFF_3 + N3 * TILE;
    static constexpr int OFF_NL = OFF_2 + N2 * TILE;   // dkv: nl with the first operand's stages
    static constexpr int OFF_DELTA = OFF_NL + N3 * 512;
    static constexpr int OFF_BAR = OFF_DELTA + N2 * 512;
    static constexpr int NBAR = 24;
    static constexpr int NEED = OFF_BAR + NBAR * 8 + 16;
    // more than half of the SM's shared memory: a second CTA would wait there for TMEM columns
    static constexpr int SMEM = NEED < 120 * 1024 ? 120 * 1024 : NEED;
    static constexpr int THREADS = 320;
    static_assert(SMEM <= 232448, "shared memory of one CTA");
};

// nl and -delta of every row; D/8 lanes per row.
template <int D> __global__ void __launch_bounds__(256) win_stats_kernel(WinBwdArgs a, float *nl, float *ndelta)
{
    constexpr int C = D / 8, RPB = 256 / C;
    const WinArgs &w = a.w;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / C;  // (b, i < npad, hq)
    const int c = threadIdx.x % C;
    const int64_t bi = row / w.hq;
    const int hq = (int)(row - bi * w.hq);
    const int b = (int)(bi / a.npad), i = (int)(bi - (int64_t)b * a.npad);
    const bool in = b < w.B;
    const bool valid = in && i < win_len(w, b);
    float x = 0.0f;
    if (valid) {
        const size_t at = (((size_t)b * w.n + i) * w.hq + hq) * D + c * 8;
        float fo[8], fg[8];
        unpack<__nv_bfloat16>(ld16((const __nv_bfloat16 *)w.o_in + at), fo);
        unpack<__nv_bfloat16>(ld16((const __nv_bfloat16 *)w.dout + at), fg);
#pragma unroll
        for (int e = 0; e < 8; ++e) x += fo[e] * fg[e];
    }
    x = seg_sum<C>(x);
    if (in && c == 0) {
        const size_t to = ((size_t)b * w.hq + hq) * a.npad + i;
        nl[to] = valid ? -LOG2E * __ldg(w.lse_in + ((size_t)b * w.n + i) * w.hq + hq) : -INFINITY;
        ndelta[to] = -x;
    }
}

// Whether queries [i, i + 32) see all, some or none of keys [k0, k0 + 32). Queries past the end
// need no mask: their P is 0 by nl.
__device__ __forceinline__ Piece query_piece(int k0, int i, int len, int window, int sinks)
{
    if (i + 31 < k0 || i >= len || k0 >= len || (i > k0 + 31 + window - 1 && k0 >= sinks)) return Piece::none;
    if (i >= k0 + 31 && (i + 31 <= k0 + window - 1 || k0 + 32 <= sinks)) return Piece::all;
    return Piece::some;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Whole warp: A x B^T of two K-major tiles (128 x D and n x D) into TMEM at `d`; the descriptors'
// low words.
template <int D> __device__ __forceinline__ void mma_tiles(uint32_t lead, uint32_t d, uint32_t a_lo, uint32_t b_lo, int n)
{
    const uint32_t idesc = umma::idesc_bf16_f32(UW, n);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = ((ks / 4) * UATOM + (ks % 4) * 32) >> 4;
        umma::mma_ss(lead, d, a_lo + off, b_lo + off, idesc, ks > 0);
    }
}

// Whole warp: TMEM operand (bf16 pairs: columns 0-63 at +0, columns 64-127 at +64) x rows [0, k) of
// a tile taken MN-major, added to the D columns at `d`. k: a multiple of 32.
template <int D>
__device__ __forceinline__ void mma_accumulate(uint32_t lead, uint32_t d, uint32_t ta, uint32_t b_lo, int k, bool add)
{
    constexpr uint32_t idesc = umma::idesc_bf16_f32_bmn(UW, D);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
        if (ks < 2 || ks * 16 < k)
            umma::mma_ts(lead, d, ta + (ks < 4 ? ks * 8 : 64 + (ks - 4) * 8), b_lo + (ks * 2048 >> 4), idesc, add || ks > 0);
}

template <int D>
__global__ void __launch_bounds__(WinBwdGeom<D>::THREADS, 1)
win_dq_umma_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmdo,
                   const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                   const __grid_constant__ CUtensorMap tmdq, WinBwdArgs ba)
{
    using Geo = WinBwdGeom<D>;
    constexpr int NA = Geo::NA, TILE = Geo::TILE, NK = Geo::N3, NV = Geo::N2;
    const WinArgs &a = ba.w;
    extern __shared__ __align__(1024) uint8_t wdsm[];
    uint8_t *sm = wdsm;
    const uint32_t base = smem_u32(sm);
    const uint32_t sq = base, sdo = base + TILE, sk = base + Geo::OFF_3, sv = base + Geo::OFF_2;
    const uint32_t sb = base + Geo::OFF_BAR;
    const uint32_t q_full = sb, tail = sb + 8, k_full = sb + 16, k_empty = k_full + 8 * NK, v_full = k_empty + 8 * NK;
    const uint32_t v_empty = v_full + 8 * NV, s_full = v_empty + 8 * NV, s_empty = s_full + 8, dp_full = s_empty + 8;
    const uint32_t ds_full = dp_full + 16, dq_full = ds_full + 16, mma_done = dq_full + 8, tslot = base + Geo::OFF_BAR + Geo::NBAR * 8;
    const uint32_t *tslot_p = reinterpret_cast<const uint32_t *>(sm + Geo::OFF_BAR + Geo::NBAR * 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = a.B * a.hq;
    const int blk = a.nblk - 1 - (int)(blockIdx.x / (unsigned)per);
    const int bh = (int)(blockIdx.x % (unsigned)per);
    const int b = bh / a.hq, hq = bh - b * a.hq, h = hq / a.G, i0 = blk * UW;
    const int len = win_len(a, b);
    const KeyBlocks kb(i0, UW, len, a.window, a.sinks, UW);
    const int nt = kb.na + kb.nb;
    if (nt == 0) {
        for (int y = threadIdx.x; y < UW * (D / 8); y += Geo::THREADS) {
            const int r = y / (D / 8), c = y - r * (D / 8);
            if (i0 + r < a.n)
                *reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.dq + (((size_t)b * a.n + i0 + r) * a.hq + hq) * D + c * 8) =
                    make_uint4(0, 0, 0, 0);
        }
        return;
    }
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(tail, 1);
#pragma unroll
        for (int s = 0; s < NK; ++s) mbar_init(k_full + 8 * s, 1), mbar_init(k_empty + 8 * s, 1);
#pragma unroll
        for (int s = 0; s < NV; ++s) mbar_init(v_full + 8 * s, 1), mbar_init(v_empty + 8 * s, 1);
        mbar_init(s_full, 1);
        mbar_init(s_empty, 256);
#pragma unroll
        for (int s = 0; s < 2; ++s) mbar_init(dp_full + 8 * s, 1), mbar_init(ds_full + 8 * s, 256);
        mbar_init(dq_full, 1);
        mbar_init(mma_done, 1);
        mbar_init_fence();
    }
    if (warp == 9) umma::tmem_alloc(tslot, 512);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = *tslot_p;
    const uint32_t tS = tmem, tP = tmem + 128, tQ = tmem + 384;  // S, two dP / dS buffers, dQ

    if (warp == 8) {
        const auto load = [&](uint32_t dst, const CUtensorMap *m, int head, int row, uint32_t bar) {
#pragma unroll
            for (int at = 0; at < NA; ++at) umma::tma_load_4d(dst + at * UATOM, m, at * 64, head, row, b, bar);
        };
        if (lane == 0) {
            mbar_arrive_expect(q_full, 2 * TILE);
            load(sq, &tmq, hq, i0, q_full);
            load(sdo, &tmdo, hq, i0, q_full);
        }
        bool ok = true;
        for (int j = 0; ok && j < nt; ++j) {
            const int s3 = j % NK, s2 = j % NV, t0 = kb.start(j, UW);
            if (lane == 0 && j >= NK) ok = mbar_wait(k_empty + 8 * s3, ((j / NK) - 1) & 1);
            ok = __shfl_sync(FULL, ok, 0);
            if (!ok) break;
            const bool fix = t0 + UW > len && len < a.n;  // the last block alone: dQ sums over K's rows
            const uint32_t bar = fix ? tail : k_full + 8 * s3;
            if (lane == 0) {
                mbar_arrive_expect(bar, TILE);
                load(sk + s3 * TILE, &tmk, h, t0, bar);
            }
            if (fix) {
                ok = __all_sync(FULL, mbar_wait(tail, 0));
                if (ok) zero_rows<NA, UW>(sm + Geo::OFF_3 + s3 * TILE, max(len - t0, 0), lane);
                umma::fence_proxy_async();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(k_full + 8 * s3);
            }
            if (lane == 0 && ok && j >= NV) ok = mbar_wait(v_empty + 8 * s2, ((j / NV) - 1) & 1);
            if (lane == 0 && ok) {
                mbar_arrive_expect(v_full + 8 * s2, TILE);
                load(sv + s2 * TILE, &tmv, h, t0, v_full + 8 * s2);
            }
            ok = __shfl_sync(FULL, ok, 0);
        }
        if (lane == 0 && !ok) {  // gave up: copies in flight land before the CTA ends (bounded)
            mbar_wait(q_full, 0);
            for (int s = 0; s < NK; ++s) mbar_wait(k_full + 8 * s, 0);
            for (int s = 0; s < NV; ++s) mbar_wait(v_full + 8 * s, 0);
        }
    } else if (warp == 9) {
        // ---- MMAs (the whole warp runs along, one lane issues) ----------------------------
        const uint32_t lead = umma::elect_lead();
        const uint32_t q_lo = umma::sdesc_lo(sq, umma::KMAJOR), do_lo = umma::sdesc_lo(sdo, umma::KMAJOR);
        const uint32_t k_lo = umma::sdesc_lo(sk, umma::KMAJOR), kt_lo = umma::sdesc_lo(sk, UATOM);
        const uint32_t v_lo = umma::sdesc_lo(sv, umma::KMAJOR);
        const auto width = [&](int j) { return (kb.end(j, UW) - kb.start(j, UW) + 31) & ~31; };
        const auto first = [&](int j) {  // S(j), then dP(j)
            const int n = width(j), s3 = j % NK, s2 = j % NV;
            bool ok = mbar_wait_warp(k_full + 8 * s3, (j / NK) & 1);
            if (ok && j > 0) ok = mbar_wait_warp(s_empty, (j - 1) & 1);
            if (!ok) return false;
            umma::fence_after_sync();
            mma_tiles<D>(lead, tS, q_lo, k_lo + s3 * (TILE >> 4), n);
            umma::commit_if(lead, s_full);
            if (!mbar_wait_warp(v_full + 8 * s2, (j / NV) & 1)) return false;
            umma::fence_after_sync();
            mma_tiles<D>(lead, tP + (j & 1) * 128, do_lo, v_lo + s2 * (TILE >> 4), n);
            umma::commit_if(lead, dp_full + 8 * (j & 1));
            umma::commit_if(lead, v_empty + 8 * s2);
            return true;
        };
        bool ok = mbar_wait_warp(q_full, 0) && first(0);
        for (int j = 0; ok && j < nt; ++j) {
            if (j + 1 < nt) ok = first(j + 1);
            if (ok) ok = mbar_wait_warp(ds_full + 8 * (j & 1), (j >> 1) & 1);
            if (!ok) break;
            umma::fence_after_sync();
            mma_accumulate<D>(lead, tQ, tP + (j & 1) * 128, kt_lo + (j % NK) * (TILE >> 4), width(j), j > 0);
            umma::commit_if(lead, k_empty + 8 * (j % NK));
        }
        if (ok) umma::commit_if(lead, dq_full);
        umma::commit_if(lead, mma_done);
        mbar_wait_warp(mma_done, 0);
    } else {
        const int wg = warp >> 2, r = (warp & 3) * 32 + lane, i = i0 + r;
        const bool valid = i < len;
        const size_t st = ((size_t)b * a.hq + hq) * ba.npad + i;  // i < npad
        const float nl = valid ? __ldg(ba.nl + st) : 0.0f, dl = valid ? __ldg(ba.ndelta + st) : 0.0f;
        const float sl2 = a.scale;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            const int t0 = kb.start(j, UW), t1 = kb.end(j, UW);
            const int c0 = wg * 64, nch = min(max((t1 - t0 - c0 + 31) / 32, 0), 2);  // this group's pieces
            const bool whole = ((t1 - t0) & 31) == 0 && t1 - 1 <= i0 && i0 + UW <= len &&
                               (t0 > i0 + UW - 1 - a.window || t1 <= a.sinks);
            ok = __all_sync(FULL, mbar_wait(s_full, j & 1));
            if (!ok) break;
            umma::fence_after_sync();
            uint32_t s[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (c < nch) umma::tmem_ld32(tS + lane_off + c0 + c * 32, s[c]);
            umma::tmem_wait_ld();
            umma::fence_before_sync();
            mbar_arrive(s_empty);
            Piece piece[2];
            uint32_t mask[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = c0 + c * 32;
                piece[c] = whole ? Piece::all : key_piece(i0 + (warp & 3) * 32, t0 + col, t1, len, a.window, a.sinks);
                mask[c] = piece[c] == Piece::some ? column_mask(col, i - a.window + 1 - t0, valid ? min(i, t1 - 1) - t0 : -1,
                                                                a.sinks - t0)
                                                  : 0u;
                if (piece[c] == Piece::none) continue;
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                                make_float2(sl2, sl2), make_float2(nl, nl));
                    s[c][e] = __float_as_uint(ex2_ftz(x.x));
                    s[c][e + 1] = __float_as_uint(ex2_ftz(x.y));
                }
            }
            ok = __all_sync(FULL, mbar_wait(dp_full + 8 * (j & 1), (j >> 1) & 1));
            if (!ok) break;
            umma::fence_after_sync();
            const uint32_t tp = tP + (j & 1) * 128 + lane_off + c0;
            uint32_t d[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (piece[c] != Piece::none) umma::tmem_ld32(tp + c * 32, d[c]);
            umma::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t x[16];
                if (piece[c] == Piece::none) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = 0u;
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 p = make_float2(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1]));
                        const float2 y =
                            __fmul2_rn(p, __fadd2_rn(make_float2(__uint_as_float(d[c][2 * e]), __uint_as_float(d[c][2 * e + 1])),
                                                     make_float2(dl, dl)));
                        x[e] = bf16_pair(y.x, y.y);
                    }
                    if (piece[c] == Piece::some) {  // hidden keys' dS is dropped, whatever their rows held
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const uint32_t lo = (mask[c] >> (2 * e)) & 1 ? 0x0000ffffu : 0u;
                            const uint32_t hi = (mask[c] >> (2 * e + 1)) & 1 ? 0xffff0000u : 0u;
                            x[e] &= lo | hi;
                        }
                    }
                }
                if (c < nch) umma::tmem_st16(tp + c * 16, x);
            }
            umma::tmem_wait_st();
            umma::fence_before_sync();
            mbar_arrive(ds_full + 8 * (j & 1));
        }
        if (ok) ok = __all_sync(FULL, mbar_wait(dq_full, 0));
        if (ok) {
            umma::fence_after_sync();
            // the tile's Q rows are free now
            stage_row(sm, tQ + lane_off, r, wg * (D / 64), (wg + 1) * (D / 64), ba.scale, valid);
            umma::fence_proxy_async();
        }
        named_sync(1, 256);
        if (threadIdx.x == 0 && ok) {
#pragma unroll
            for (int at = 0; at < NA; ++at) umma::tma_store_4d(&tmdq, sq + at * UATOM, at * 64, hq, i0, b);
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

template <int D>
__global__ void __launch_bounds__(WinBwdGeom<D>::THREADS, 1)
win_dkv_umma_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmdo,
                    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                    const __grid_constant__ CUtensorMap tmdk, const __grid_constant__ CUtensorMap tmdv, WinBwdArgs ba)
{
    using Geo = WinBwdGeom<D>;
    constexpr int NA = Geo::NA, TILE = Geo::TILE, NQ = Geo::N3, ND = Geo::N2;
    const WinArgs &a = ba.w;
    extern __shared__ __align__(1024) uint8_t wdsm[];
    uint8_t *sm = wdsm;
    const uint32_t base = smem_u32(sm);
    const uint32_t sk = base, sv = base + TILE, sq = base + Geo::OFF_3, sdo = base + Geo::OFF_2;
    const uint32_t sb = base + Geo::OFF_BAR;
    const uint32_t kv_full = sb, tail = sb + 8, q_full = sb + 16, q_empty = q_full + 8 * NQ, do_full = q_empty + 8 * NQ;
    const uint32_t do_empty = do_full + 8 * ND, s_full = do_empty + 8 * ND, dp_full = s_full + 8, p_full = dp_full + 8;
    const uint32_t ds_full = p_full + 8, acc_full = ds_full + 8, mma_done = acc_full + 8, tslot = base + Geo::OFF_BAR + Geo::NBAR * 8;
    const uint32_t *tslot_p = reinterpret_cast<const uint32_t *>(sm + Geo::OFF_BAR + Geo::NBAR * 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = a.B * a.hkv;
    const int blk = (int)(blockIdx.x / (unsigned)per);  // the keys that most queries see first
    const int bh = (int)(blockIdx.x % (unsigned)per);
    const int b = bh / a.hkv, h = bh - b * a.hkv, t0 = blk * UW;
    const int len = win_len(a, b);
    const int t1 = min(t0 + UW, len);
    const int qend = t1 > t0 ? query_end(t0, t1, len, a.window, a.sinks) : t0;
    const int nq = (qend - t0 + UW - 1) / UW, nt = nq * a.G;  // query blocks per head, steps
    if (nt == 0) {
        for (int y = threadIdx.x; y < UW * (D / 8); y += Geo::THREADS) {
            const int r = y / (D / 8), c = y - r * (D / 8);
            if (t0 + r < a.n) {
                const size_t at = (((size_t)b * a.n + t0 + r) * a.hkv + h) * D + c * 8;
                *reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.dk + at) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.dv + at) = make_uint4(0, 0, 0, 0);
            }
        }
        return;
    }
    if (threadIdx.x == 0) {
        mbar_init(kv_full, 1);
        mbar_init(tail, 1);
#pragma unroll
        for (int s = 0; s < NQ; ++s) mbar_init(q_full + 8 * s, 1), mbar_init(q_empty + 8 * s, 1);
#pragma unroll
        for (int s = 0; s < ND; ++s) mbar_init(do_full + 8 * s, 1), mbar_init(do_empty + 8 * s, 1);
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_full, 256);
        mbar_init(ds_full, 256);
        mbar_init(acc_full, 1);
        mbar_init(mma_done, 1);
        mbar_init_fence();
    }
    if (warp == 9) umma::tmem_alloc(tslot, 512);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = *tslot_p;
    const uint32_t tS = tmem, tP = tmem + 128, tV = tmem + 256, tK = tmem + 256 + D;

    if (warp == 8) {
        const auto load = [&](uint32_t dst, const CUtensorMap *m, int head, int row, uint32_t bar) {
#pragma unroll
            for (int at = 0; at < NA; ++at) umma::tma_load_4d(dst + at * UATOM, m, at * 64, head, row, b, bar);
        };
        if (lane == 0) {
            mbar_arrive_expect(kv_full, 2 * TILE);
            load(sk, &tmk, h, t0, kv_full);
            load(sv, &tmv, h, t0, kv_full);
        }
        bool ok = true;
        int fixes = 0;
        for (int j = 0; ok && j < nt; ++j) {
            const int s3 = j % NQ, s2 = j % ND, g = j / nq, i0 = t0 + (j - g * nq) * UW, hq = h * a.G + g;
            const float *nl = ba.nl + ((size_t)b * a.hq + hq) * ba.npad + i0;
            const float *dl = ba.ndelta + ((size_t)b * a.hq + hq) * ba.npad + i0;
            const bool fix = i0 + UW > len && len < a.n;  // dK and dV sum over these rows
            if (lane == 0 && j >= NQ) ok = mbar_wait(q_empty + 8 * s3, ((j / NQ) - 1) & 1);
            if (lane == 0 && ok && j >= ND) ok = mbar_wait(do_empty + 8 * s2, ((j / ND) - 1) & 1);
            ok = __shfl_sync(FULL, ok, 0);
            if (!ok) break;
            if (lane == 0) {
                const uint32_t bq = fix ? tail : q_full + 8 * s3, bd = fix ? tail : do_full + 8 * s2;
                if (fix) {
                    mbar_arrive_expect(tail, 2 * (TILE + 512));
                } else {
                    mbar_arrive_expect(bq, TILE + 512);
                    mbar_arrive_expect(bd, TILE + 512);
                }
                load(sq + s3 * TILE, &tmq, hq, i0, bq);
                bulk_load(base + Geo::OFF_NL + s3 * 512, nl, 512, bq);
                load(sdo + s2 * TILE, &tmdo, hq, i0, bd);
                bulk_load(base + Geo::OFF_DELTA + s2 * 512, dl, 512, bd);
            }
            if (fix) {
                ok = __all_sync(FULL, mbar_wait(tail, fixes++ & 1));
                if (ok) {
                    zero_rows<NA, UW>(sm + Geo::OFF_3 + s3 * TILE, max(len - i0, 0), lane);
                    zero_rows<NA, UW>(sm + Geo::OFF_2 + s2 * TILE, max(len - i0, 0), lane);
                }
                umma::fence_proxy_async();
                __syncwarp();
                if (lane == 0 && ok) {
                    mbar_arrive(q_full + 8 * s3);
                    mbar_arrive(do_full + 8 * s2);
                }
            }
        }
        if (lane == 0 && !ok) {
            mbar_wait(kv_full, 0);
            for (int s = 0; s < NQ; ++s) mbar_wait(q_full + 8 * s, 0);
            for (int s = 0; s < ND; ++s) mbar_wait(do_full + 8 * s, 0);
        }
    } else if (warp == 9) {
        // ---- MMAs (the whole warp runs along, one lane issues) ----------------------------
        const uint32_t lead = umma::elect_lead();
        const uint32_t k_lo = umma::sdesc_lo(sk, umma::KMAJOR), v_lo = umma::sdesc_lo(sv, umma::KMAJOR);
        const uint32_t q_lo = umma::sdesc_lo(sq, umma::KMAJOR), qt_lo = umma::sdesc_lo(sq, UATOM);
        const uint32_t do_lo = umma::sdesc_lo(sdo, umma::KMAJOR), dot_lo = umma::sdesc_lo(sdo, UATOM);
        const auto scores = [&](int j) {
            if (!mbar_wait_warp(q_full + 8 * (j % NQ), (j / NQ) & 1)) return false;
            umma::fence_after_sync();
            mma_tiles<D>(lead, tS, k_lo, q_lo + (j % NQ) * (TILE >> 4), UW);
            umma::commit_if(lead, s_full);
            return true;
        };
        const auto dps = [&](int j) {
            if (!mbar_wait_warp(do_full + 8 * (j % ND), (j / ND) & 1)) return false;
            umma::fence_after_sync();
            mma_tiles<D>(lead, tP, v_lo, do_lo + (j % ND) * (TILE >> 4), UW);
            umma::commit_if(lead, dp_full);
            return true;
        };
        bool ok = mbar_wait_warp(kv_full, 0) && scores(0) && dps(0);
        for (int j = 0; ok && j < nt; ++j) {
            ok = mbar_wait_warp(p_full, j & 1);
            if (!ok) break;
            umma::fence_after_sync();
            mma_accumulate<D>(lead, tV, tS, dot_lo + (j % ND) * (TILE >> 4), UW, j > 0);
            if (j + 1 < nt) ok = scores(j + 1);
            if (ok) ok = mbar_wait_warp(ds_full, j & 1);
            if (!ok) break;
            umma::fence_after_sync();
            mma_accumulate<D>(lead, tK, tP, qt_lo + (j % NQ) * (TILE >> 4), UW, j > 0);
            umma::commit_if(lead, q_empty + 8 * (j % NQ));
            umma::commit_if(lead, do_empty + 8 * (j % ND));
            if (j + 1 < nt) ok = dps(j + 1);
        }
        if (ok) umma::commit_if(lead, acc_full);
        umma::commit_if(lead, mma_done);
        mbar_wait_warp(mma_done, 0);
    } else {
        const int wg = warp >> 2, r = (warp & 3) * 32 + lane, t = t0 + r;
        const bool valid = t < len;
        const float sl2 = a.scale;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const int c0 = wg * 64;
        const int last = t < a.sinks ? len - 1 : min(len - 1, t + a.window - 1);  // last query that sees the key
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            const int g = j / nq, i0 = t0 + (j - g * nq) * UW;
            const bool whole = i0 >= t0 + UW - 1 && (i0 + UW - 1 <= t0 + a.window - 1 || t0 + UW <= a.sinks);
            ok = __all_sync(FULL, mbar_wait(q_full + 8 * (j % NQ), (j / NQ) & 1) && mbar_wait(s_full, j & 1));
            if (!ok) break;
            umma::fence_after_sync();
            const float4 *nl = reinterpret_cast<const float4 *>(sm + Geo::OFF_NL + (j % NQ) * 512) + wg * 16;
            // pieces of 32 queries: which keys of the warp's 32 rows do they see?
            Piece piece[2];
            uint32_t mask[2], s[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                piece[c] = whole ? Piece::all : query_piece(t0 + (warp & 3) * 32, i0 + c0 + c * 32, len, a.window, a.sinks);
                mask[c] = piece[c] == Piece::some ? column_mask(c0 + c * 32, t - i0, last - i0, 0) : 0u;
                if (piece[c] != Piece::none) umma::tmem_ld32(tS + lane_off + c0 + c * 32, s[c]);
            }
            umma::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t x[16];
                if (piece[c] == Piece::none) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = 0u;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 y = nl[c * 8 + e];
                        const float2 x0 = __ffma2_rn(make_float2(__uint_as_float(s[c][4 * e]), __uint_as_float(s[c][4 * e + 1])),
                                                     make_float2(sl2, sl2), make_float2(y.x, y.y));
                        const float2 x1 = __ffma2_rn(make_float2(__uint_as_float(s[c][4 * e + 2]), __uint_as_float(s[c][4 * e + 3])),
                                                     make_float2(sl2, sl2), make_float2(y.z, y.w));
                        s[c][4 * e] = __float_as_uint(ex2_ftz(x0.x));
                        s[c][4 * e + 1] = __float_as_uint(ex2_ftz(x0.y));
                        s[c][4 * e + 2] = __float_as_uint(ex2_ftz(x1.x));
                        s[c][4 * e + 3] = __float_as_uint(ex2_ftz(x1.y));
                    }
                    if (piece[c] == Piece::some) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((mask[c] >> e) & 1)) s[c][e] = 0u;
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        x[e] = bf16_pair(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1]));
                }
                umma::tmem_st16(tS + lane_off + c0 + c * 16, x);
            }
            umma::tmem_wait_st();
            umma::fence_before_sync();
            mbar_arrive(p_full);
            ok = __all_sync(FULL, mbar_wait(do_full + 8 * (j % ND), (j / ND) & 1) && mbar_wait(dp_full, j & 1));
            if (!ok) break;
            umma::fence_after_sync();
            const float4 *dl = reinterpret_cast<const float4 *>(sm + Geo::OFF_DELTA + (j % ND) * 512) + wg * 16;  // -delta
            uint32_t d[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (piece[c] != Piece::none) umma::tmem_ld32(tP + lane_off + c0 + c * 32, d[c]);
            umma::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t x[16];
                if (piece[c] == Piece::none) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = 0u;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 y = dl[c * 8 + e];
                        const float2 x0 = __fmul2_rn(make_float2(__uint_as_float(s[c][4 * e]), __uint_as_float(s[c][4 * e + 1])),
                                                     __fadd2_rn(make_float2(__uint_as_float(d[c][4 * e]), __uint_as_float(d[c][4 * e + 1])),
                                                                make_float2(y.x, y.y)));
                        const float2 x1 = __fmul2_rn(make_float2(__uint_as_float(s[c][4 * e + 2]), __uint_as_float(s[c][4 * e + 3])),
                                                     __fadd2_rn(make_float2(__uint_as_float(d[c][4 * e + 2]), __uint_as_float(d[c][4 * e + 3])),
                                                                make_float2(y.z, y.w)));
                        x[2 * e] = bf16_pair(x0.x, x0.y);
                        x[2 * e + 1] = bf16_pair(x1.x, x1.y);
                    }
                }
                umma::tmem_st16(tP + lane_off + c0 + c * 16, x);
            }
            umma::tmem_wait_st();
            umma::fence_before_sync();
            mbar_arrive(ds_full);
        }
        if (ok) ok = __all_sync(FULL, mbar_wait(acc_full, 0));
        if (ok) {
            umma::fence_after_sync();
            // the K and V tiles are free now: dk goes out through the first, dv through the second
            stage_row(sm + wg * TILE, (wg ? tV : tK) + lane_off, r, 0, D / 32, wg ? 1.0f : ba.scale, valid);
            umma::fence_proxy_async();
        }
        named_sync(1, 256);
        if (threadIdx.x == 0 && ok) {
#pragma unroll
            for (int at = 0; at < NA; ++at) {
                umma::tma_store_4d(&tmdk, sk + at * UATOM, at * 64, h, t0, b);
                umma::tma_store_4d(&tmdv, sv + at * UATOM, at * 64, h, t0, b);
            }
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
