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
// keeping its bf16 results inside its own half of the fp32 tile. P and dS are rounded to bf16, at most
// half a step (2^-8) each, because both operands of a product have one type and the other one comes in
// bf16: against 64 bits forward and backward together are off by 0.0024 in the 2-norm at window 1024,
// in fp32 with one rounding at the end by 0.0017.
//
// nl = -lse log2(e) and delta = <dout, o> come from a pass over o and dout, laid out [B, hq, npad] with
// npad a multiple of 128; rows at or past the sequence's end have nl = -inf (P <= 2^-126) and delta = 0.
// Such rows of the tiles are zeroed in shared memory where a product sums over them. An eighth of the
// exponentials runs on the FMA pipe (n = 16384 3661 -> 3547 us, window 1024 1266 -> 1254 us in turn;
// three sixteenths 3609, 1262).
//
// The threads read scores and dP from TMEM 32 columns at a time, the next under the arithmetic of the
// one before (window 1024 1207 -> 1163 us in turn; all 64 at once need fewer waits but hold every
// warp at the same place).
//
// 16/8 heads, d=128, 4 sinks beside a window; back to back on the same tensors (at the power limit), in
// brackets a single call with a cold L2: B=8 n=4096 window 512 790 us (720), window 1024 1150 us (1030);
// B=1 n=16384 full 3470 us (3060). The tensor pipe is busy half of the time (dq 50 %): a step's products
// wait for its elements and the other way round, at one CTA per SM.
//
// Both kernels run one CTA per SM, which takes item after item from a counter in the workspace
// (items differ in length, by the mask and by the sequences): the loads, S and dP of the next item
// start under the last elements and the output of the one before. Output rows go from registers to
// global memory, 16 bytes at a time: all of shared memory holds operands.
//
// dkv with few keys that many queries see (sinks; few sequences): the steps of one key block are
// cut into chunks, each an item of its own that writes fp32 partial sums to the workspace, and
// win_dkv_join_kernel adds those in chunk order.
//
// A row that sees one key has P = 1 whatever its score: its dS is 0, not the difference of two equal
// sums (WinArgs::lone).
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
    int64_t items;        // work items of the kernel that is launched
    int *next;            // its counter, 0 at the launch
    // dkv: the first `sink_blocks` key blocks are cut into sink_chunks, the others into chunks pieces of
    // at most sink_steps / steps steps; pieces of cut blocks go to `part` [piece][dk, dv][128][D]
    int sink_blocks, sink_chunks, chunks, sink_steps, steps;
    float *part;
};

// One piece of one key block's work in dkv.
struct DkvItem {
    int b, h, t0, len, nq, j0, j1;  // query blocks per head; steps [j0, j1) of nq * G
    bool cut;
    int64_t slot;                   // of the piece in `part`
    __device__ __forceinline__ DkvItem(const WinBwdArgs &ba, int64_t item)
    {
        const WinArgs &a = ba.w;
        const int64_t per = (int64_t)a.B * a.hkv, sink_items = per * ba.sink_blocks * ba.sink_chunks;
        int blk, chunk, most;
        int64_t x;
        if (item < sink_items) {  // a block's pieces are neighbours
            chunk = (int)(item % ba.sink_chunks);
            x = item / ba.sink_chunks;
            blk = (int)(x / per);
            most = ba.sink_steps;
            cut = ba.sink_chunks > 1;
            slot = item;
        } else {
            const int64_t y = item - sink_items;
            chunk = (int)(y % ba.chunks);
            x = y / ba.chunks;
            blk = ba.sink_blocks + (int)(x / per);
            most = ba.steps;
            cut = ba.chunks > 1;
            slot = (ba.sink_chunks > 1 ? sink_items : 0) + y;
        }
        const int bh = (int)(x % per);
        b = bh / a.hkv;
        h = bh - b * a.hkv;
        t0 = blk * UW;
        len = win_len(a, b);
        const int t1 = min(t0 + UW, len);
        const int qend = t1 > t0 ? query_end(t0, t1, len, a.window, a.sinks) : t0;
        nq = (qend - t0 + UW - 1) / UW;
        const int64_t first = (int64_t)chunk * most;  // 64 bits: steps of an uncut block are unlimited
        const int all = nq * a.G;
        j0 = (int)(first < all ? first : all);
        j1 = (int)(first + most < all ? first + most : all);
    }
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
    static constexpr int NBAR = 32;                    // the last eight: the item queue's
    static constexpr int OFF_QUEUE = OFF_BAR + NBAR * 8 + 16;
    static constexpr int NEED = OFF_QUEUE + 16;
    // more than half of the SM's shared memory: a second CTA would wait there for TMEM columns
    static constexpr int SMEM = NEED < 120 * 1024 ? 120 * 1024 : NEED;
    static constexpr int THREADS = 384;                // warps 10 and 11 only fill their warpgroup
    // Registers per thread: at the launch, of warps 8-11, of warps 0-7. At 168 the dq threads spill
    // (window 512 868 -> 805 us, window 128 567 -> 509 us in turn with the split).
    static constexpr int REGS = 168, REGS_LOAD = 88, REGS_ELEM = 208;
    static_assert(REGS_LOAD + 2 * REGS_ELEM <= 3 * REGS, "a split above the launch's registers would wait forever");
    static_assert(SMEM <= 232448, "shared memory of one CTA");
};

// -delta of the first `few` rows of a sequence, those that see at most FEW keys.
//
// delta = <dout, o> inherits the rounding of o to bf16, an error that reaches dS as P times a
// constant of the row. Averaged over many keys it is lost in the other roundings, but a row of
// few keys has o as large as v and dS = P (dP - delta) as a difference of near values. Such rows
// get delta = sum_t P dP from q, k, v and dout (2-norm error of dq at windows of 2 to 8 keys:
// 0.0034 -> 0.0023, two roundings to bf16 alone give 0.0023). D/8 lanes per row, two keys at a
// time so that their loads overlap.
constexpr int FEW = 24;

template <int D> __device__ __forceinline__ void few_rows(const WinBwdArgs &a, const FastDiv &div_hq, int b,
                                                          uint32_t y0, int few, float *ndelta)
{
    constexpr int C = D / 8, N = 2;
    const WinArgs &w = a.w;
    const int c = threadIdx.x % C;
    const uint32_t y = y0 + threadIdx.x / C;
    const uint32_t real = (uint32_t)min(win_len(w, b), few) * w.hq;
    const uint32_t i = div_hq.div(y), hq = y - i * div_hq.d;
    const size_t row = (size_t)b * w.n * w.hq + y;
    const bool in = y < real;
    const int keys = in ? (int)min((int64_t)i + 1, (int64_t)w.window + w.sinks) : 0;
    const int lo = max((int)i - w.window + 1, 0), ns = min(w.sinks, lo);  // sinks before the window
    float fq[8], fg[8], sum = 0.0f;
    unpack<__nv_bfloat16>(in ? ld16((const __nv_bfloat16 *)w.q + row * D + c * 8) : make_uint4(0, 0, 0, 0), fq);
    unpack<__nv_bfloat16>(in ? ld16((const __nv_bfloat16 *)w.dout + row * D + c * 8) : make_uint4(0, 0, 0, 0), fg);
    const float nl = in ? -LOG2E * __ldg(w.lse_in + row) : 0.0f;
    const int most = __reduce_max_sync(FULL, keys);
    for (int u0 = 0; u0 < most; u0 += N) {
        uint4 uk[N], uv[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int u = u0 + e, t = u < ns ? u : lo + u - ns;
            const size_t at = (((size_t)b * w.n + t) * w.hkv + hq / w.G) * D + c * 8;
            uk[e] = uv[e] = make_uint4(0, 0, 0, 0);
            if (u < keys) uk[e] = ld16((const __nv_bfloat16 *)w.k + at), uv[e] = ld16((const __nv_bfloat16 *)w.v + at);
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float fk[8], fv[8];
            float2 dots = make_float2(0.0f, 0.0f);
            unpack<__nv_bfloat16>(uk[e], fk);
            unpack<__nv_bfloat16>(uv[e], fv);
#pragma unroll
            for (int z = 0; z < 8; ++z) {
                dots.x += fq[z] * fk[z];
                dots.y += fg[z] * fv[z];
            }
            dots = seg_sum2<C>(dots);
            if (u0 + e < keys) sum += ex2_ftz(fmaf(dots.x, w.scale, nl)) * dots.y;
        }
    }
    if (in && c == 0) ndelta[((size_t)b * w.hq + hq) * a.npad + i] = -sum;
}

// nl and -delta of every row (b, i < npad, hq); D/8 lanes per row, each taking two rows so that
// four 16-byte loads are in flight. A block stays within one sequence, whose rows are contiguous.
// Also sets both counters to 0. Bound by HBM: o and dout once (B=8 n=4096, 16 heads: 47 us).
// The first few_blocks blocks take few_rows, few_per_seq of them per sequence: they start with the
// others and are bound by latency, so they end within the others' time at large sizes.
template <int D> __global__ void __launch_bounds__(256, 5)
win_stats_kernel(WinBwdArgs a, FastDiv div_hq, unsigned per_seq, int few, unsigned few_per_seq, unsigned few_blocks,
                 float *nl, float *ndelta)
{
    if (blockIdx.x == 0 && threadIdx.x < 2) a.next[threadIdx.x] = 0;
    constexpr int C = D / 8, RPB = 256 / C, N = 2;
    if (blockIdx.x < few_blocks) {
        const unsigned b = blockIdx.x / few_per_seq;
        few_rows<D>(a, div_hq, (int)b, (blockIdx.x - b * few_per_seq) * RPB, few, ndelta);
        return;
    }
    const WinArgs &w = a.w;
    const unsigned bx = blockIdx.x - few_blocks;
    const int c = threadIdx.x % C, b = (int)(bx / per_seq);
    const uint32_t y0 = (bx - (uint32_t)b * per_seq) * (RPB * N) + threadIdx.x / C;  // row of the sequence
    const uint32_t rows = (uint32_t)a.npad * w.hq, real = (uint32_t)win_len(w, b) * w.hq;
    const uint32_t skip = min((uint32_t)few * w.hq, real);  // rows that few_rows takes
    const size_t first = (size_t)b * w.n * w.hq;
    uint4 uo[N], ug[N];
    float lse[N];
#pragma unroll
    for (int r = 0; r < N; ++r) {
        const uint32_t y = y0 + r * RPB;
        uo[r] = ug[r] = make_uint4(0, 0, 0, 0);
        lse[r] = 0.0f;
        if (y >= skip && y < real) {
            uo[r] = ld16_stream((const __nv_bfloat16 *)w.o_in + (first + y) * D + c * 8);
            ug[r] = ld16((const __nv_bfloat16 *)w.dout + (first + y) * D + c * 8);
        }
        if (y < real && c == 0) lse[r] = __ldg(w.lse_in + first + y);
    }
#pragma unroll
    for (int r = 0; r < N; ++r) {
        const uint32_t y = y0 + r * RPB;
        float fo[8], fg[8], x = 0.0f;
        unpack<__nv_bfloat16>(uo[r], fo);
        unpack<__nv_bfloat16>(ug[r], fg);
#pragma unroll
        for (int e = 0; e < 8; ++e) x += fo[e] * fg[e];
        x = seg_sum<C>(x);
        if (y < rows && c == 0) {
            const uint32_t i = div_hq.div(y), hq = y - i * div_hq.d;
            const size_t to = ((size_t)b * w.hq + hq) * a.npad + i;
            nl[to] = y < real ? -LOG2E * lse[r] : -INFINITY;
            if (y >= skip) ndelta[to] = -x;
        }
    }
}

// Whether queries [i, i + 32) see all, some or none of keys [k0, k0 + 32). Queries past the end
// need no mask: their P is at most 2^-126 by nl and their rows of the tiles are 0.
__device__ __forceinline__ Piece query_piece(int k0, int i, int len, int window, int sinks)
{
    if (i + 31 < k0 || i >= len || k0 >= len || (i > k0 + 31 + window - 1 && k0 >= sinks)) return Piece::none;
    if (i >= k0 + 31 && (i + 31 <= k0 + window - 1 || k0 + 32 <= sinks)) return Piece::all;
    return Piece::some;
}

// The CTA's queue of work items: the load warp takes them from the counter and passes them on, up
// to four ahead of the slowest reader. Item `items` or more ends the work.
struct ItemQueue {
    uint32_t full, empty;    // barriers of the four slots
    volatile int *slots;
    uint32_t n = 0;
    __device__ __forceinline__ ItemQueue(uint32_t bars, void *mem) : full(bars), empty(bars + 32), slots((volatile int *)mem) {}
    // By one thread, before the others read.
    __device__ __forceinline__ void init() const
    {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 9);  // eight element warps and the MMA warp
        }
    }
    // By the load warp: passes `item` on; false after a wait that gave up.
    __device__ __forceinline__ bool push(int item, int lane)
    {
        const uint32_t s = n % 4;
        bool ok = true;
        if (lane == 0) {
            if (n >= 4) ok = mbar_wait(empty + 8 * s, ((n / 4) - 1) & 1);
            if (ok) {
                slots[s] = item;
                mbar_arrive(full + 8 * s);
            }
        }
        ++n;
        return __shfl_sync(FULL, ok, 0);
    }
    // By a reading warp: the next item, or -1 after a wait that gave up.
    __device__ __forceinline__ int pop(int lane)
    {
        const uint32_t s = n % 4;
        if (!mbar_wait_warp(full + 8 * s, (n / 4) & 1)) return -1;
        const int item = slots[s];
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * s);
        ++n;
        return item;
    }
};

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

// This thread's row of a TMEM accumulator, columns [32 c0, 32 c1), times f, as bf16 (or fp32) to
// global memory; nothing where `keep` is 0, zeros where it is 1, the values where it is 2.
template <typename T>
__device__ __forceinline__ void store_row(T *dst, uint32_t taddr, int c0, int c1, float f, int keep)
{
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
        uint32_t o[32];
        umma::tmem_ld32(taddr + c * 32, o);
        umma::tmem_wait_ld();
        if (keep) {
            constexpr int V = 16 / sizeof(T);
#pragma unroll
            for (int e = 0; e < 32 / V; ++e) {
                float x[V];
#pragma unroll
                for (int y = 0; y < V; ++y) x[y] = keep == 2 ? __uint_as_float(o[e * V + y]) * f : 0.0f;
                *reinterpret_cast<uint4 *>(dst + c * 32 + e * V) = pack<T>(x);
            }
        }
        __syncwarp();
    }
}

template <int D>
__global__ void __launch_bounds__(WinBwdGeom<D>::THREADS, 1)
win_dq_umma_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmdo,
                   const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, WinBwdArgs ba)
{
    using Geo = WinBwdGeom<D>;
    constexpr int NA = Geo::NA, TILE = Geo::TILE, NK = Geo::N3, NV = Geo::N2;
    const WinArgs &a = ba.w;
    extern __shared__ __align__(1024) uint8_t wdsm[];
    uint8_t *sm = wdsm;
    const uint32_t base = smem_u32(sm);
    const uint32_t sq = base, sdo = base + TILE, sk = base + Geo::OFF_3, sv = base + Geo::OFF_2;
    const uint32_t sb = base + Geo::OFF_BAR;
    const uint32_t q_full = sb, q_empty = sb + 8, tail = sb + 16, k_full = sb + 24, k_empty = k_full + 8 * NK;
    const uint32_t v_full = k_empty + 8 * NK, v_empty = v_full + 8 * NV, s_full = v_empty + 8 * NV, s_empty = s_full + 8;
    const uint32_t dp_full = s_empty + 8, ds_full = dp_full + 16, dq_full = ds_full + 16, dq_empty = dq_full + 8;
    const uint32_t do_full = dq_empty + 8, do_empty = do_full + 8, mma_done = do_empty + 8, tslot = base + Geo::OFF_BAR + Geo::NBAR * 8;
    const uint32_t *tslot_p = reinterpret_cast<const uint32_t *>(sm + Geo::OFF_BAR + Geo::NBAR * 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ItemQueue queue(base + Geo::OFF_BAR + (Geo::NBAR - 8) * 8, sm + Geo::OFF_QUEUE);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(do_full, 1);
        mbar_init(do_empty, 1);
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
        mbar_init(dq_empty, 256);
        mbar_init(mma_done, 1);
        queue.init();
        mbar_init_fence();
    }
    if (warp == 9) umma::tmem_alloc(tslot, 512);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = *tslot_p;
    const uint32_t tS = tmem, tP = tmem + 128, tQ = tmem + 384;  // S, two dP / dS buffers, dQ

    // item: (query block, longest prefixes first; sequence; head)
    const int per = a.B * a.hq;
    struct Item {
        int b, hq, h, i0, len, nt;
        KeyBlocks kb;
        __device__ __forceinline__ Item(const WinArgs &a, int64_t item, int per) : kb(0, 0, 0, 1, 0, 1)
        {
            const int x = (int)(item % per);
            b = x / a.hq;
            hq = x - b * a.hq;
            h = hq / a.G;
            i0 = (a.nblk - 1 - (int)(item / per)) * UW;
            len = win_len(a, b);
            kb = KeyBlocks(i0, UW, len, a.window, a.sinks, UW);
            nt = kb.na + kb.nb;
        }
    };

    if (warp >= 8) {
        umma::regs_dec<Geo::REGS_LOAD>();
        if (warp == 8) {
            uint32_t kc = 0, fixes = 0;
            int qc = 0;
            bool ok = true;
            // the first item by position, the others from the counter, asked for one item ahead
            int item = (int)blockIdx.x, ahead = lane == 0 ? (int)gridDim.x + atomicAdd(ba.next, 1) : 0;
            for (;;) {
                ok = queue.push(item, lane);
                if (!ok || item >= ba.items) break;
                const Item w(a, item, per);
                item = __shfl_sync(FULL, ahead, 0);
                if (lane == 0) ahead = (int)gridDim.x + atomicAdd(ba.next, 1);
                if (w.nt == 0) continue;
                const auto load = [&](uint32_t dst, const CUtensorMap *m, int head, int row, uint32_t bar) {
    #pragma unroll
                    for (int at = 0; at < NA; ++at) umma::tma_load_4d(dst + at * UATOM, m, at * 64, head, row, w.b, bar);
                };
                if (lane == 0 && qc > 0) ok = mbar_wait(q_empty, (qc - 1) & 1);
                ok = __shfl_sync(FULL, ok, 0);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect(q_full, TILE);
                    load(sq, &tmq, w.hq, w.i0, q_full);
                    if (qc > 0) ok = mbar_wait(do_empty, (qc - 1) & 1);
                    mbar_arrive_expect(do_full, TILE);
                    load(sdo, &tmdo, w.hq, w.i0, do_full);
                }
                ok = __shfl_sync(FULL, ok, 0);
                ++qc;
                for (int j = 0; ok && j < w.nt; ++j, ++kc) {
                    const uint32_t s3 = kc % NK, s2 = kc % NV;
                    const int t0 = w.kb.start(j, UW);
                    if (lane == 0 && kc >= NK) ok = mbar_wait(k_empty + 8 * s3, ((kc / NK) - 1) & 1);
                    ok = __shfl_sync(FULL, ok, 0);
                    if (!ok) break;
                    const bool fix = t0 + UW > w.len && w.len < a.n;  // the last block alone: dQ sums over K's rows
                    const uint32_t bar = fix ? tail : k_full + 8 * s3;
                    if (lane == 0) {
                        mbar_arrive_expect(bar, TILE);
                        load(sk + s3 * TILE, &tmk, w.h, t0, bar);
                    }
                    if (fix) {
                        ok = mbar_wait_warp(tail, fixes++ & 1);
                        if (ok) zero_rows<NA, UW>(sm + Geo::OFF_3 + s3 * TILE, max(w.len - t0, 0), lane);
                        umma::fence_proxy_async();
                        __syncwarp();
                        if (lane == 0 && ok) mbar_arrive(k_full + 8 * s3);
                    }
                    if (lane == 0 && ok && kc >= NV) ok = mbar_wait(v_empty + 8 * s2, ((kc / NV) - 1) & 1);
                    if (lane == 0 && ok) {
                        mbar_arrive_expect(v_full + 8 * s2, TILE);
                        load(sv + s2 * TILE, &tmv, w.h, t0, v_full + 8 * s2);
                    }
                    ok = __shfl_sync(FULL, ok, 0);
                }
                if (!ok) break;
            }
            if (lane == 0 && !ok && qc > 0) {  // gave up: copies in flight land before the CTA ends (bounded)
                mbar_wait(q_full, (qc - 1) & 1);
                mbar_wait(do_full, (qc - 1) & 1);
                for (uint32_t y = kc > NK ? kc - NK : 0; y < kc; ++y) mbar_wait(k_full + 8 * (y % NK), (y / NK) & 1);
                for (uint32_t y = kc > NV ? kc - NV : 0; y < kc; ++y) mbar_wait(v_full + 8 * (y % NV), (y / NV) & 1);
            }
        } else if (warp == 9) {
            // ---- MMAs (the whole warp runs along, one lane issues) ----------------------------
            const uint32_t lead = umma::elect_lead();
            const uint32_t q_lo = umma::sdesc_lo(sq, umma::KMAJOR), do_lo = umma::sdesc_lo(sdo, umma::KMAJOR);
            const uint32_t k_lo = umma::sdesc_lo(sk, umma::KMAJOR), kt_lo = umma::sdesc_lo(sk, UATOM);
            const uint32_t v_lo = umma::sdesc_lo(sv, umma::KMAJOR);
            uint32_t kc = 0;
            int qc = 0;
            bool ok = true;
            while (ok) {
                const int item = queue.pop(lane);
                if (item < 0 || item >= ba.items) break;
                const Item w(a, item, per);
                if (w.nt == 0) continue;
                const auto width = [&](int j) { return (w.kb.end(j, UW) - w.kb.start(j, UW) + 31) & ~31; };
                const auto first = [&](int j) {  // S(j), then dP(j)
                    const uint32_t y = kc + j, s3 = y % NK, s2 = y % NV;
                    const int n = width(j);
                    bool ok = mbar_wait_warp(k_full + 8 * s3, (y / NK) & 1);
                    if (ok && y > 0) ok = mbar_wait_warp(s_empty, (y - 1) & 1);
                    if (!ok) return false;
                    umma::fence_after_sync();
                    mma_tiles<D>(lead, tS, q_lo, k_lo + s3 * (TILE >> 4), n);
                    umma::commit_if(lead, s_full);
                    if (j == w.nt - 1) umma::commit_if(lead, q_empty);
                    if (j == 0 && !mbar_wait_warp(do_full, qc & 1)) return false;
                    if (!mbar_wait_warp(v_full + 8 * s2, (y / NV) & 1)) return false;
                    umma::fence_after_sync();
                    mma_tiles<D>(lead, tP + (y & 1) * 128, do_lo, v_lo + s2 * (TILE >> 4), n);
                    umma::commit_if(lead, dp_full + 8 * (y & 1));
                    umma::commit_if(lead, v_empty + 8 * s2);
                    if (j == w.nt - 1) umma::commit_if(lead, do_empty);
                    return true;
                };
                ok = mbar_wait_warp(q_full, qc & 1) && first(0);
                for (int j = 0; ok && j < w.nt; ++j) {
                    const uint32_t y = kc + j;
                    if (j + 1 < w.nt) ok = first(j + 1);
                    if (ok && j == 0 && qc > 0) ok = mbar_wait_warp(dq_empty, (qc - 1) & 1);
                    if (ok) ok = mbar_wait_warp(ds_full + 8 * (y & 1), (y >> 1) & 1);
                    if (!ok) break;
                    umma::fence_after_sync();
                    mma_accumulate<D>(lead, tQ, tP + (y & 1) * 128, kt_lo + (y % NK) * (TILE >> 4), width(j), j > 0);
                    umma::commit_if(lead, k_empty + 8 * (y % NK));
                }
                if (ok) umma::commit_if(lead, dq_full);
                kc += w.nt;
                ++qc;
            }
            // every MMA issued has completed before the CTA releases its tensor memory
            umma::commit_if(lead, mma_done);
            mbar_wait_warp(mma_done, 0);
        }
    } else {
        umma::regs_inc<Geo::REGS_ELEM>();
        const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
        const float sl2 = a.scale;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        uint32_t kc = 0;
        int qc = 0;
        bool ok = true;
        // an item is taken, and its row's statistics asked for, before the output of the one before
        int item = queue.pop(lane);
        float nl = 0.0f, dl = 0.0f;
        const auto statistics = [&](const Item &w) {
            const size_t st = ((size_t)w.b * a.hq + w.hq) * ba.npad + w.i0 + r;  // rows are padded to npad
            nl = __ldg(ba.nl + st);
            dl = __ldg(ba.ndelta + st);
        };
        if (item >= 0 && item < ba.items) statistics(Item(a, item, per));
        while (item >= 0 && item < ba.items) {
            const Item w(a, item, per);
            const int len = w.len, i0 = w.i0, i = i0 + r;
            const bool valid = i < len;
            for (int j = 0; j < w.nt; ++j) {
                const uint32_t y = kc + j;
                const int t0 = w.kb.start(j, UW), t1 = w.kb.end(j, UW);
                const int c0 = wg * 64, nch = min(max((t1 - t0 - c0 + 31) / 32, 0), 2);  // this group's pieces
                const bool whole = ((t1 - t0) & 31) == 0 && t1 - 1 <= i0 && i0 + UW <= len &&
                                   (t0 > i0 + UW - 1 - a.window || t1 <= a.sinks);
                ok = mbar_wait_warp(s_full, y & 1);
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
                    piece[c] = key_piece(i0 + (warp & 3) * 32, t0 + col, t1, len, a.window, a.sinks);
                    if (whole) piece[c] = c < nch ? Piece::all : Piece::none;
                    mask[c] = piece[c] == Piece::some ? column_mask(col, i - a.window + 1 - t0,
                                                                    valid && i >= a.lone ? min(i, t1 - 1) - t0 : -1, a.sinks - t0)
                                                      : 0u;
                    if (piece[c] == Piece::none) continue;
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                                    make_float2(sl2, sl2), make_float2(nl, nl));
                        const float2 p = ex2_pair<2>(x, e / 2);
                        s[c][e] = __float_as_uint(p.x);
                        s[c][e + 1] = __float_as_uint(p.y);
                    }
                }
                ok = mbar_wait_warp(dp_full + 8 * (y & 1), (y >> 1) & 1);
                if (!ok) break;
                umma::fence_after_sync();
                const uint32_t tp = tP + (y & 1) * 128 + lane_off + c0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[16], d[32];
                    if (piece[c] == Piece::none) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] = 0u;
                    } else {
                        umma::tmem_ld32(tp + c * 32, d);
                        umma::tmem_wait_ld32(d);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 p = make_float2(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1]));
                            const float2 z = __fmul2_rn(
                                p, __fadd2_rn(make_float2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])),
                                              make_float2(dl, dl)));
                            x[e] = bf16_pair(z.x, z.y);
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
                mbar_arrive(ds_full + 8 * (y & 1));
            }
            kc += w.nt;
            if (!ok) break;
            item = queue.pop(lane);
            if (item >= 0 && item < ba.items) statistics(Item(a, item, per));
            if (w.nt > 0) {
                ok = mbar_wait_warp(dq_full, qc & 1);
                if (!ok) break;
                umma::fence_after_sync();
            }
            __nv_bfloat16 *row = (__nv_bfloat16 *)a.dq + (((size_t)w.b * a.n + i) * a.hq + w.hq) * D;
            store_row(row, tQ + lane_off, wg * (D / 64), (wg + 1) * (D / 64), ba.scale, i >= a.n ? 0 : valid ? 2 : 1);
            if (w.nt > 0) {
                umma::fence_before_sync();
                mbar_arrive(dq_empty);
                ++qc;
            }
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
                    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, WinBwdArgs ba)
{
    using Geo = WinBwdGeom<D>;
    constexpr int NA = Geo::NA, TILE = Geo::TILE, NQ = Geo::N3, ND = Geo::N2;
    const WinArgs &a = ba.w;
    extern __shared__ __align__(1024) uint8_t wdsm[];
    uint8_t *sm = wdsm;
    const uint32_t base = smem_u32(sm);
    const uint32_t sk = base, sv = base + TILE, sq = base + Geo::OFF_3, sdo = base + Geo::OFF_2;
    const uint32_t sb = base + Geo::OFF_BAR;
    const uint32_t kv_full = sb, kv_empty = sb + 8, tail = sb + 16, q_full = sb + 24, q_empty = q_full + 8 * NQ;
    const uint32_t do_full = q_empty + 8 * NQ, do_empty = do_full + 8 * ND, s_full = do_empty + 8 * ND, dp_full = s_full + 8;
    const uint32_t p_full = dp_full + 8, ds_full = p_full + 8, acc_full = ds_full + 8, acc_empty = acc_full + 8;
    const uint32_t mma_done = acc_empty + 8, tslot = base + Geo::OFF_BAR + Geo::NBAR * 8;
    const uint32_t *tslot_p = reinterpret_cast<const uint32_t *>(sm + Geo::OFF_BAR + Geo::NBAR * 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ItemQueue queue(base + Geo::OFF_BAR + (Geo::NBAR - 8) * 8, sm + Geo::OFF_QUEUE);

    if (threadIdx.x == 0) {
        mbar_init(kv_full, 1);
        mbar_init(kv_empty, 1);
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
        mbar_init(acc_empty, 256);
        mbar_init(mma_done, 1);
        queue.init();
        mbar_init_fence();
    }
    if (warp == 9) umma::tmem_alloc(tslot, 512);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = *tslot_p;
    const uint32_t tS = tmem, tP = tmem + 128, tV = tmem + 256, tK = tmem + 256 + D;

    if (warp >= 8) {
        umma::regs_dec<Geo::REGS_LOAD>();
        if (warp == 8) {
            uint32_t kc = 0, fixes = 0;  // steps so far
            int qc = 0;                  // items with steps so far
            bool ok = true;
            // the first item by position, the others from the counter, asked for one item ahead
            int item = (int)blockIdx.x, ahead = lane == 0 ? (int)gridDim.x + atomicAdd(ba.next, 1) : 0;
            for (;;) {
                ok = queue.push(item, lane);
                if (!ok || item >= ba.items) break;
                const DkvItem w(ba, item);
                item = __shfl_sync(FULL, ahead, 0);
                if (lane == 0) ahead = (int)gridDim.x + atomicAdd(ba.next, 1);
                if (w.j1 <= w.j0) continue;
                const auto load = [&](uint32_t dst, const CUtensorMap *m, int head, int row, uint32_t bar) {
    #pragma unroll
                    for (int at = 0; at < NA; ++at) umma::tma_load_4d(dst + at * UATOM, m, at * 64, head, row, w.b, bar);
                };
                if (lane == 0 && qc > 0) ok = mbar_wait(kv_empty, (qc - 1) & 1);
                ok = __shfl_sync(FULL, ok, 0);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect(kv_full, 2 * TILE);
                    load(sk, &tmk, w.h, w.t0, kv_full);
                    load(sv, &tmv, w.h, w.t0, kv_full);
                }
                ++qc;
                for (int j = w.j0; ok && j < w.j1; ++j, ++kc) {
                    const uint32_t s3 = kc % NQ, s2 = kc % ND;
                    const int g = j / w.nq, i0 = w.t0 + (j - g * w.nq) * UW, hq = w.h * a.G + g;
                    const float *nl = ba.nl + ((size_t)w.b * a.hq + hq) * ba.npad + i0;
                    const float *dl = ba.ndelta + ((size_t)w.b * a.hq + hq) * ba.npad + i0;
                    const bool fix = i0 + UW > w.len && w.len < a.n;  // dK and dV sum over these rows
                    if (lane == 0 && kc >= NQ) ok = mbar_wait(q_empty + 8 * s3, ((kc / NQ) - 1) & 1);
                    if (lane == 0 && ok && kc >= ND) ok = mbar_wait(do_empty + 8 * s2, ((kc / ND) - 1) & 1);
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
                        ok = mbar_wait_warp(tail, fixes++ & 1);
                        if (ok) {
                            zero_rows<NA, UW>(sm + Geo::OFF_3 + s3 * TILE, max(w.len - i0, 0), lane);
                            zero_rows<NA, UW>(sm + Geo::OFF_2 + s2 * TILE, max(w.len - i0, 0), lane);
                        }
                        umma::fence_proxy_async();
                        __syncwarp();
                        if (lane == 0 && ok) {
                            mbar_arrive(q_full + 8 * s3);
                            mbar_arrive(do_full + 8 * s2);
                        }
                    }
                }
                if (!ok) break;
            }
            if (lane == 0 && !ok && qc > 0) {  // gave up: copies in flight land before the CTA ends (bounded)
                mbar_wait(kv_full, (qc - 1) & 1);
                for (uint32_t y = kc > NQ ? kc - NQ : 0; y < kc; ++y) mbar_wait(q_full + 8 * (y % NQ), (y / NQ) & 1);
                for (uint32_t y = kc > ND ? kc - ND : 0; y < kc; ++y) mbar_wait(do_full + 8 * (y % ND), (y / ND) & 1);
            }
        } else if (warp == 9) {
            // ---- MMAs (the whole warp runs along, one lane issues) ----------------------------
            const uint32_t lead = umma::elect_lead();
            const uint32_t k_lo = umma::sdesc_lo(sk, umma::KMAJOR), v_lo = umma::sdesc_lo(sv, umma::KMAJOR);
            const uint32_t q_lo = umma::sdesc_lo(sq, umma::KMAJOR), qt_lo = umma::sdesc_lo(sq, UATOM);
            const uint32_t do_lo = umma::sdesc_lo(sdo, umma::KMAJOR), dot_lo = umma::sdesc_lo(sdo, UATOM);
            const auto scores = [&](uint32_t y) {
                if (!mbar_wait_warp(q_full + 8 * (y % NQ), (y / NQ) & 1)) return false;
                umma::fence_after_sync();
                mma_tiles<D>(lead, tS, k_lo, q_lo + (y % NQ) * (TILE >> 4), UW);
                umma::commit_if(lead, s_full);
                return true;
            };
            const auto dps = [&](uint32_t y, bool last) {
                if (!mbar_wait_warp(do_full + 8 * (y % ND), (y / ND) & 1)) return false;
                umma::fence_after_sync();
                mma_tiles<D>(lead, tP, v_lo, do_lo + (y % ND) * (TILE >> 4), UW);
                umma::commit_if(lead, dp_full);
                if (last) umma::commit_if(lead, kv_empty);
                return true;
            };
            uint32_t kc = 0;
            int qc = 0;
            bool ok = true;
            while (ok) {
                const int item = queue.pop(lane);
                if (item < 0 || item >= ba.items) break;
                const DkvItem w(ba, item);
                const int nt = w.j1 - w.j0;
                if (nt <= 0) continue;
                ok = mbar_wait_warp(kv_full, qc & 1) && scores(kc) && dps(kc, nt == 1);
                for (int j = 0; ok && j < nt; ++j) {
                    const uint32_t y = kc + j;
                    if (j == 0 && qc > 0) ok = mbar_wait_warp(acc_empty, (qc - 1) & 1);
                    if (ok) ok = mbar_wait_warp(p_full, y & 1);
                    if (!ok) break;
                    umma::fence_after_sync();
                    mma_accumulate<D>(lead, tV, tS, dot_lo + (y % ND) * (TILE >> 4), UW, j > 0);
                    if (j + 1 < nt) ok = scores(y + 1);
                    if (ok) ok = mbar_wait_warp(ds_full, y & 1);
                    if (!ok) break;
                    umma::fence_after_sync();
                    mma_accumulate<D>(lead, tK, tP, qt_lo + (y % NQ) * (TILE >> 4), UW, j > 0);
                    umma::commit_if(lead, q_empty + 8 * (y % NQ));
                    umma::commit_if(lead, do_empty + 8 * (y % ND));
                    if (j + 1 < nt) ok = dps(y + 1, j + 2 == nt);
                }
                if (ok) umma::commit_if(lead, acc_full);
                kc += nt;
                ++qc;
            }
            // every MMA issued has completed before the CTA releases its tensor memory
            umma::commit_if(lead, mma_done);
            mbar_wait_warp(mma_done, 0);
        }
    } else {
        umma::regs_inc<Geo::REGS_ELEM>();
        const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
        const float sl2 = a.scale;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const int c0 = wg * 64;
        uint32_t kc = 0;
        int qc = 0;
        bool ok = true;
        while (ok) {
            const int item = queue.pop(lane);
            if (item < 0 || item >= ba.items) break;
            const DkvItem w(ba, item);
            const int len = w.len, t0 = w.t0, t = t0 + r;
            const bool valid = t < len;
            const int last = t < a.sinks ? len - 1 : min(len - 1, t + a.window - 1);  // last query that sees the key
            for (int j = w.j0; j < w.j1; ++j) {
                const uint32_t y = kc + j - w.j0;
                const int g = j / w.nq, i0 = t0 + (j - g * w.nq) * UW;
                const bool whole = i0 >= t0 + UW - 1 && (i0 + UW - 1 <= t0 + a.window - 1 || t0 + UW <= a.sinks);
                ok = mbar_wait_warp(q_full + 8 * (y % NQ), (y / NQ) & 1) && mbar_wait_warp(s_full, y & 1);
                if (!ok) break;
                umma::fence_after_sync();
                const float4 *nl = reinterpret_cast<const float4 *>(sm + Geo::OFF_NL + (y % NQ) * 512) + wg * 16;
                // pieces of 32 queries: which keys of the warp's 32 rows do they see?
                Piece piece[2];
                uint32_t mask[2], s[2][32];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    piece[c] = whole ? Piece::all : query_piece(t0 + (warp & 3) * 32, i0 + c0 + c * 32, len, a.window, a.sinks);
                    mask[c] = piece[c] == Piece::some ? column_mask(c0 + c * 32, t - i0, last - i0, 0) : 0u;
                }
                if (piece[0] != Piece::none) umma::tmem_ld32(tS + lane_off + c0, s[0]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    umma::tmem_wait_ld32(s[c]);
                    if (c == 0 && piece[1] != Piece::none) umma::tmem_ld32(tS + lane_off + c0 + 32, s[1]);
                    uint32_t x[16];
                    if (piece[c] == Piece::none) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] = 0u;
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 z = nl[c * 8 + e];
                            const float2 x0 = __ffma2_rn(make_float2(__uint_as_float(s[c][4 * e]), __uint_as_float(s[c][4 * e + 1])),
                                                         make_float2(sl2, sl2), make_float2(z.x, z.y));
                            const float2 x1 = __ffma2_rn(make_float2(__uint_as_float(s[c][4 * e + 2]), __uint_as_float(s[c][4 * e + 3])),
                                                         make_float2(sl2, sl2), make_float2(z.z, z.w));
                            const float2 p0 = ex2_pair<2>(x0, 2 * e), p1 = ex2_pair<2>(x1, 2 * e + 1);
                            s[c][4 * e] = __float_as_uint(p0.x);
                            s[c][4 * e + 1] = __float_as_uint(p0.y);
                            s[c][4 * e + 2] = __float_as_uint(p1.x);
                            s[c][4 * e + 3] = __float_as_uint(p1.y);
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
                ok = mbar_wait_warp(do_full + 8 * (y % ND), (y / ND) & 1) && mbar_wait_warp(dp_full, y & 1);
                if (!ok) break;
                umma::fence_after_sync();
                const float4 *dl = reinterpret_cast<const float4 *>(sm + Geo::OFF_DELTA + (y % ND) * 512) + wg * 16;  // -delta
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[16], d[32];
                    if (piece[c] == Piece::none) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] = 0u;
                    } else {
                        umma::tmem_ld32(tP + lane_off + c0 + c * 32, d);
                        umma::tmem_wait_ld32(d);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 z = dl[c * 8 + e];
                            const float2 x0 = __fmul2_rn(make_float2(__uint_as_float(s[c][4 * e]), __uint_as_float(s[c][4 * e + 1])),
                                                         __fadd2_rn(make_float2(__uint_as_float(d[4 * e]), __uint_as_float(d[4 * e + 1])),
                                                                    make_float2(z.x, z.y)));
                            const float2 x1 = __fmul2_rn(make_float2(__uint_as_float(s[c][4 * e + 2]), __uint_as_float(s[c][4 * e + 3])),
                                                         __fadd2_rn(make_float2(__uint_as_float(d[4 * e + 2]), __uint_as_float(d[4 * e + 3])),
                                                                    make_float2(z.z, z.w)));
                            x[2 * e] = bf16_pair(x0.x, x0.y);
                            x[2 * e + 1] = bf16_pair(x1.x, x1.y);
                        }
                        if (i0 + c0 + c * 32 < a.lone) {  // queries that see one key
                            x[0] &= 0xffff0000u;
                            if (a.lone > 1) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[e] = 0u;
                            }
                        }
                    }
                    // dS of piece c lies over dP of this or an earlier piece of the group
                    umma::tmem_st16(tP + lane_off + c0 + c * 16, x);
                }
                umma::tmem_wait_st();
                umma::fence_before_sync();
                mbar_arrive(ds_full);
            }
            const int nt = w.j1 - w.j0;
            kc += nt;
            if (!ok) break;
            if (nt > 0) {
                ok = mbar_wait_warp(acc_full, qc & 1);
                if (!ok) break;
                umma::fence_after_sync();
            }
            // one group writes dk, the other dv
            if (w.cut) {
                if (nt > 0) store_row(ba.part + ((size_t)w.slot * 2 + wg) * (UW * D) + (size_t)r * D, (wg ? tV : tK) + lane_off, 0,
                                      D / 32, wg ? 1.0f : ba.scale, 2);
            } else {
                __nv_bfloat16 *row = (__nv_bfloat16 *)(wg ? a.dv : a.dk) + (((size_t)w.b * a.n + t) * a.hkv + w.h) * D;
                store_row(row, (wg ? tV : tK) + lane_off, 0, D / 32, wg ? 1.0f : ba.scale, t >= a.n ? 0 : valid ? 2 : 1);
            }
            if (nt > 0) {
                umma::fence_before_sync();
                mbar_arrive(acc_empty);
                ++qc;
            }
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, 512);
    }
}

// dk and dv of key blocks that were cut: their pieces' partial sums, added in order. One thread per
// four elements; first_item: the block's first piece.
template <int D> __global__ void __launch_bounds__(256) win_dkv_join_kernel(WinBwdArgs ba, int64_t first_item, int chunks)
{
    const WinArgs &a = ba.w;
    constexpr int PER = 2 * UW * D / 4;  // threads per key block
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t block = x / PER;
    const int e = (int)(x - block * PER), kv = e / (UW * D / 4), at = (e - kv * (UW * D / 4)) * 4;
    const int r = at / D, d = at - r * D;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const DkvItem w(ba, first_item + block * chunks);
    const int t = w.t0 + r;
    if (t >= a.n) return;
    if (t < w.len) {
        for (int c = 0; c < chunks; ++c) {
            const DkvItem y(ba, first_item + block * chunks + c);
            if (y.j1 <= y.j0) break;
            const float4 v = *reinterpret_cast<const float4 *>(ba.part + ((size_t)y.slot * 2 + kv) * (UW * D) + at);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
    }
    const __nv_bfloat162 p[2] = {__floats2bfloat162_rn(sum.x, sum.y), __floats2bfloat162_rn(sum.z, sum.w)};
    __nv_bfloat16 *row = (__nv_bfloat16 *)(kv ? a.dv : a.dk) + (((size_t)w.b * a.n + t) * a.hkv + w.h) * D + d;
    *reinterpret_cast<uint2 *>(row) = *reinterpret_cast<const uint2 *>(p);
}

}  // namespace gm
