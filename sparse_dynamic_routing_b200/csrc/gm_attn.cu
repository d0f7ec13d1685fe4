// gm_attn.cu - host side of the windowed-attention and 8-bit-cache calls of include/gm.h:
// argument checks, choice of the kernel, launch on the caller's stream. A translation unit of
// its own so that it compiles beside gm_api.cu.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/gm.h"
#include "gm_common.cuh"
#include "gm_host.cuh"
#include "gm_kv8.cuh"
#include "gm_window.cuh"
#include "gm_window_bwd_umma.cuh"
#include "gm_window_umma.cuh"

#ifndef GM_CHECKED
#define GM_CHECKED 0
#endif

// Whether this library's calls of this file were ever made: before the first, their error word needs no
// reading (a copy from the device, 12 us, and the loading of their kernels).
static std::atomic<bool> g_attn_used{false};

bool gm_attn_take_errors(unsigned *flag)
{
    *flag = 0;
    if (!g_attn_used.load()) return true;
    if (cudaMemcpyFromSymbol(flag, gm::g_error_flag, sizeof(*flag)) != cudaSuccess) return false;
    const unsigned zero = 0;
    return *flag == 0 || cudaMemcpyToSymbol(gm::g_error_flag, &zero, sizeof(zero)) == cudaSuccess;
}

namespace {

// Lets a kernel have `bytes` of dynamic shared memory on the current device; asked of the runtime
// once per kernel and device. A kernel that splits its registers among warpgroups also says how many
// per thread a launch has to bring: with fewer, warps would wait for registers without end.
template <auto KERNEL> bool raise_smem(size_t bytes, int regs = 0)
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    cudaFuncAttributes attr;
    if (regs > 0 && (cudaFuncGetAttributes(&attr, KERNEL) != cudaSuccess || attr.numRegs < regs)) return false;
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Kernels take exponentials in base 2: the factor with log2(e) in it has to be finite as well.
bool good_scale(float scale) { return std::isfinite(scale * gm::LOG2E); }

// ---- windowed attention -------------------------------------------------------------------------

gm_status check_window(gm_dtype dtype, int B, int n, int hq, int hkv, int d, int window, int sinks, float scale)
{
    if (B < 0 || n < 0 || hq < 1 || hkv < 1 || d < 1 || hq % hkv != 0) return GM_ERR_INVALID_ARG;
    if (window < 1 || sinks < 0 || !good_scale(scale)) return GM_ERR_INVALID_ARG;
    if (dtype != GM_F32 && dtype != GM_BF16) return GM_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GM_ERR_UNSUPPORTED;
    if (n >= (1 << 30) || (int64_t)B * n >= MAX_ROWS || (int64_t)B * n * hq >= MAX_ROWS) return GM_ERR_UNSUPPORTED;
    return GM_OK;
}

gm::WinArgs window_args(int B, int n, int hq, int hkv, int window, int sinks, float scale, const int32_t *lens)
{
    gm::WinArgs a{};
    a.B = B;
    a.n = n;
    a.hq = hq;
    a.hkv = hkv;
    a.G = hq / hkv;
    a.window = std::min(window, n);
    a.sinks = std::min(sinks, n);
    a.lone = a.window + a.sinks == 1 ? n : 1;
    a.scale = scale;
    a.lens = lens;
    return a;
}

// Rows per thread of the fp32 kernels: 4 where blocks of 64 rows fill the SMs one and a half times,
// else 2 or 1 (gm_window.cuh).
int f32_rows(int n, int64_t heads)
{
    const int64_t blocks = (n + 63) / 64 * heads;
    return blocks >= 222 ? 4 : blocks >= 74 ? 2 : 1;
}

template <int D, int R> gm_status window_forward_f32(gm::WinArgs a, cudaStream_t st)
{
    using S = gm::WinF32<D, R>;
    constexpr auto kern = gm::win_fwd_f32_kernel<D, R>;
    if (!raise_smem<kern>(S::fwd_smem)) return GM_ERR_CUDA;
    a.nblk = (a.n + S::ROWS - 1) / S::ROWS;
    kern<<<(unsigned)((int64_t)a.nblk * a.B * a.hq), 256, S::fwd_smem, st>>>(a);
    return launched();
}

template <int D> gm_status window_forward(const gm::WinArgs &a, cudaStream_t st)
{
    const int r = f32_rows(a.n, (int64_t)a.B * a.hq);
    return r == 4 ? window_forward_f32<D, 4>(a, st) : r == 2 ? window_forward_f32<D, 2>(a, st) : window_forward_f32<D, 1>(a, st);
}

template <int D, int R> gm_status window_dq_f32(gm::WinArgs a, cudaStream_t st)
{
    using S = gm::WinF32<D, R>;
    constexpr auto kern = gm::win_dq_f32_kernel<D, R>;
    if (!raise_smem<kern>(S::dq_smem)) return GM_ERR_CUDA;
    a.nblk = (a.n + S::ROWS - 1) / S::ROWS;
    kern<<<(unsigned)((int64_t)a.nblk * a.B * a.hq), 256, S::dq_smem, st>>>(a);
    return launched();
}

// The fp32 dk, dv kernel's cut of key blocks with sinks (gm_window.cuh).
struct WinF32Plan {
    int rows, nblk, sink_blocks, chunks, steps;  // rows: per thread
    size_t delta_bytes, bytes;                   // workspace: delta, then the pieces
};

WinF32Plan window_f32_plan(int B, int n, int hq, int hkv, int d, int window, int sinks)
{
    WinF32Plan p{};
    const int G = hq / hkv;
    window = std::min(window, n);
    sinks = std::min(sinks, n);
    p.rows = f32_rows(n, (int64_t)B * hkv);
    const int tile = 16 * p.rows;
    p.nblk = (n + tile - 1) / tile;
    // query tiles of the longest block, with and without sinks
    const int all = (n + gm::WT - 1) / gm::WT;
    const int near = (int)std::min<int64_t>(all, ((int64_t)tile - 1 + window + gm::WT - 1) / gm::WT);
    p.steps = std::max(near * G, 4);
    p.chunks = (all * G + p.steps - 1) / p.steps;
    // Pieces take 2 x tile x d fp32 sums of workspace each. Eight per SM fill the GPU whatever their
    // length; with sinks in many blocks more of them would only let the workspace grow with n^2.
    const int sink_blocks = std::min(p.nblk, (sinks + tile - 1) / tile);
    const int64_t whole = (int64_t)B * hkv * sink_blocks;
    if (whole > 0) p.chunks = (int)std::min<int64_t>(p.chunks, std::max<int64_t>(1, 8 * 148 / whole));
    p.steps = std::max(p.steps, (all * G + p.chunks - 1) / p.chunks);
    p.sink_blocks = p.chunks > 1 ? sink_blocks : 0;
    p.delta_bytes = ((size_t)B * n * hq * 4 + 15) / 16 * 16;
    p.bytes = p.delta_bytes + (size_t)B * hkv * p.sink_blocks * p.chunks * 2 * tile * d * 4;
    return p;
}

template <int D, int R> gm_status window_dkv_f32(gm::WinArgs a, const WinF32Plan &p, cudaStream_t st)
{
    using S = gm::WinF32<D, R>;
    constexpr auto kern = gm::win_dkv_f32_kernel<D, R>;
    if (!raise_smem<kern>(S::dkv_smem)) return GM_ERR_CUDA;
    a.nblk = p.nblk;
    a.sink_blocks = p.sink_blocks;
    a.chunks = p.chunks;
    a.steps = p.steps;
    a.part = (float *)((char *)a.delta + p.delta_bytes);
    const int64_t per = (int64_t)a.B * a.hkv;
    const int64_t grid = per * (a.nblk - a.sink_blocks) + per * a.sink_blocks * a.chunks;
    kern<<<(unsigned)grid, 256, S::dkv_smem, st>>>(a);  // no more blocks than rows of k, and the pieces
    if (a.sink_blocks > 0)
        gm::win_dkv_join_f32_kernel<D, R><<<(unsigned)(per * a.sink_blocks * (2 * S::ROWS * D / 4) / 256), 256, 0, st>>>(a);
    return launched();
}

template <int D> gm_status window_backward(const gm::WinArgs &a, cudaStream_t st)
{
    gm::win_delta_kernel<D><<<(unsigned)(((int64_t)a.B * a.n * a.hq + 7) / 8), 256, 0, st>>>(a);
    const int rq = f32_rows(a.n, (int64_t)a.B * a.hq);
    const gm_status s = rq == 4   ? window_dq_f32<D, 4>(a, st)
                        : rq == 2 ? window_dq_f32<D, 2>(a, st)
                                  : window_dq_f32<D, 1>(a, st);
    if (s != GM_OK) return s;
    const WinF32Plan p = window_f32_plan(a.B, a.n, a.hq, a.hkv, D, a.window, a.sinks);
    return p.rows == 4 ? window_dkv_f32<D, 4>(a, p, st) : p.rows == 2 ? window_dkv_f32<D, 2>(a, p, st) : window_dkv_f32<D, 1>(a, p, st);
}

// A bf16 feature tensor [B, n, heads, d] as a 4-d TMA map whose boxes are 64 elements of d (128
// bytes, the swizzle width) x 1 head x box_rows rows of one sequence; rows past n read as zeros and are
// not written.
bool sequence_tmap(CUtensorMap &m, const void *ptr, int B, int n, int heads, int d, int box_rows = gm::UW)
{
    const EncodeTiledFn f = encode_tiled();
    if (f == nullptr) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n, (cuuint64_t)B};
    const cuuint64_t row = (cuuint64_t)heads * d * 2;
    const cuuint64_t strides[3] = {(cuuint64_t)d * 2, row, row * n};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return f(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Score factor in base 2. A scale of 0 becomes one so small that every score rounds to 0 after
// the maximum is taken off: the kernels hide keys with an infinite score, which 0 would make NaN.
float base2_scale(float scale)
{
    const float s = scale * gm::LOG2E;
    return s == 0.0f ? 0x1p-120f : s;
}

// Pairs of 128-row tiles that share their keys (gm_window_umma.cuh).
int64_t window_pairs(gm::WinArgs &a, gm::WinPairs &p)
{
    p.heads = a.G % 2 == 0;
    p.per = p.heads ? a.B * (a.hq / 2) : a.B * a.hq;
    const int rows = p.heads ? gm::UW : 2 * gm::UW;
    a.nblk = (a.n + rows - 1) / rows;
    return (int64_t)a.nblk * p.per;
}

template <int D> gm_status window_forward_bf16(gm::WinArgs a, cudaStream_t st)
{
    using Geo = gm::WinFwdGeom<D>;
    CUtensorMap tq, tk, tv, to;
    if (!sequence_tmap(tq, a.q, a.B, a.n, a.hq, D) || !sequence_tmap(tk, a.k, a.B, a.n, a.hkv, D, gm::FK) ||
        !sequence_tmap(tv, a.v, a.B, a.n, a.hkv, D, gm::FK) || !sequence_tmap(to, a.o, a.B, a.n, a.hq, D))
        return GM_ERR_CUDA;
    constexpr auto kern = gm::win_fwd_umma_kernel<D>;
    if (!raise_smem<kern>(Geo::SMEM)) return GM_ERR_CUDA;
    gm::WinPairs wp;
    wp.items = window_pairs(a, wp);
    a.scale = base2_scale(a.scale);
    kern<<<(unsigned)std::min<int64_t>(wp.items, 148), Geo::THREADS, Geo::SMEM, st>>>(tq, tk, tv, to, a, wp);
    return launched();
}

// How the key blocks of a backward are cut (gm_window_bwd_umma.cuh, WinBwdArgs), and the workspace.
struct WinBwdPlan {
    int nblk, sink_blocks, sink_chunks, chunks, sink_steps, steps;
    int64_t sink_items, items;
    size_t stats_bytes, bytes;  // nl and -delta and two counters, then the pieces' partial sums
};

WinBwdPlan window_backward_plan(int B, int n, int hq, int hkv, int d, int window, int sinks)
{
    WinBwdPlan p{};
    const int G = hq / hkv;
    window = std::min(window, n);
    sinks = std::min(sinks, n);
    p.nblk = (n + gm::UW - 1) / gm::UW;
    const int64_t per = (int64_t)B * hkv;
    // steps (128 queries of one head) of the block that is seen longest, with and without sinks
    const int64_t near = std::min<int64_t>(p.nblk, (127 + (int64_t)window + 127) / 128);
    p.sink_blocks = near < p.nblk ? std::min(p.nblk, (sinks + 127) / 128) : 0;
    const int64_t sink_most = (int64_t)p.nblk * G, most = near * G;
    int64_t total = 0;
    for (int64_t b = 0; b < p.nblk; ++b) total += (b < p.sink_blocks ? p.nblk - b : std::min(near, p.nblk - b)) * G;
    total *= per;
    // Blocks are cut where the longest would take half as long again as an SM's share of it all, sink
    // blocks, of which there are few, at half of that share (B=1 n=32768 window 512 with sinks: 1520 ->
    // 900 us); elsewhere the writes and reads of 2 x 128 x d fp32 sums per piece cost more than the
    // balance gives (B=1 n=4096 full: 275 -> 356 us).
    const int64_t share = (total + 147) / 148;
    const auto pieces = [&](int64_t steps, int64_t longest, int64_t piece) {
        return (int)(steps >= 16 && steps > longest ? (steps + std::max<int64_t>(8, piece) - 1) / std::max<int64_t>(8, piece) : 1);
    };
    p.sink_chunks = p.sink_blocks ? pieces(sink_most, share / 2, share / 4) : 1;
    p.chunks = pieces(most, 3 * share / 2, share / 2);
    p.sink_steps = p.sink_chunks > 1 ? (int)((sink_most + p.sink_chunks - 1) / p.sink_chunks) : INT32_MAX;
    p.steps = p.chunks > 1 ? (int)((most + p.chunks - 1) / p.chunks) : INT32_MAX;
    p.sink_items = per * p.sink_blocks * p.sink_chunks;
    p.items = p.sink_items + per * (p.nblk - p.sink_blocks) * p.chunks;
    const int64_t cut = (p.sink_chunks > 1 ? p.sink_items : 0) + (p.chunks > 1 ? p.items - p.sink_items : 0);
    p.stats_bytes = (size_t)B * p.nblk * gm::UW * hq * 8 + 16;
    p.bytes = p.stats_bytes + (size_t)cut * 2 * gm::UW * d * 4;
    return p;
}

// Whether the bf16 backward takes the shape: its statistics pass counts the padded rows of a sequence in
// 32 bits and takes 32 or more of them per block, its items are counted in 32 bits.
bool window_backward_fits(gm_dtype dtype, int B, int n, int hq)
{
    const int64_t rows = ((int64_t)n + gm::UW - 1) / gm::UW * gm::UW * hq;
    return dtype != GM_BF16 || (rows < MAX_ROWS && B * rows < (int64_t)1 << 36);
}

template <int D> gm_status window_backward_bf16(const gm::WinArgs &w, cudaStream_t st)
{
    using Geo = gm::WinBwdGeom<D>;
    CUtensorMap tq, tdo, tk, tv;
    if (!sequence_tmap(tq, w.q, w.B, w.n, w.hq, D) || !sequence_tmap(tdo, w.dout, w.B, w.n, w.hq, D) ||
        !sequence_tmap(tk, w.k, w.B, w.n, w.hkv, D) || !sequence_tmap(tv, w.v, w.B, w.n, w.hkv, D))
        return GM_ERR_CUDA;
    constexpr auto kq = gm::win_dq_umma_kernel<D>;
    constexpr auto kkv = gm::win_dkv_umma_kernel<D>;
    if (!raise_smem<kq>(Geo::SMEM, Geo::REGS) || !raise_smem<kkv>(Geo::SMEM, Geo::REGS)) return GM_ERR_CUDA;
    const WinBwdPlan p = window_backward_plan(w.B, w.n, w.hq, w.hkv, D, w.window, w.sinks);
    gm::WinBwdArgs a{};
    a.w = w;
    a.scale = w.scale;
    a.w.scale = base2_scale(w.scale);
    a.w.nblk = p.nblk;
    a.npad = p.nblk * gm::UW;
    a.sink_blocks = p.sink_blocks;
    a.sink_chunks = p.sink_chunks;
    a.chunks = p.chunks;
    a.sink_steps = p.sink_steps;
    a.steps = p.steps;
    const int64_t rows = (int64_t)w.B * a.npad * w.hq;
    float *nl = w.delta, *ndelta = w.delta + rows;
    a.nl = nl;
    a.ndelta = ndelta;
    a.next = (int *)(ndelta + rows);
    a.part = (float *)((char *)w.delta + p.stats_bytes);
    const unsigned per_seq = (unsigned)(((int64_t)a.npad * w.hq * (D / 8) + 511) / 512);  // blocks of 512 / (D / 8) rows
    // rows that see few keys: all of them, or those at a sequence's start
    const int few = (int64_t)w.window + w.sinks <= gm::FEW ? w.n : std::min(w.n, gm::FEW);
    const unsigned few_per_seq = (unsigned)(((int64_t)few * w.hq * (D / 8) + 255) / 256);
    const unsigned few_blocks = (unsigned)w.B * few_per_seq;
    gm::win_stats_kernel<D><<<few_blocks + (unsigned)w.B * per_seq, 256, 0, st>>>(
        a, gm::FastDiv((uint32_t)w.hq), per_seq, few, few_per_seq, few_blocks, nl, ndelta);
    a.items = (int64_t)p.nblk * w.B * w.hq;
    kq<<<(unsigned)std::min<int64_t>(a.items, 148), Geo::THREADS, Geo::SMEM, st>>>(tq, tdo, tk, tv, a);
    a.items = p.items;
    a.next += 1;
    kkv<<<(unsigned)std::min<int64_t>(a.items, 148), Geo::THREADS, Geo::SMEM, st>>>(tq, tdo, tk, tv, a);
    const int64_t per = (int64_t)w.B * w.hkv, threads = 2 * gm::UW * D / 4;  // per key block
    if (p.sink_chunks > 1)
        gm::win_dkv_join_kernel<D><<<(unsigned)(per * p.sink_blocks * threads / 256), 256, 0, st>>>(a, 0, p.sink_chunks);
    if (p.chunks > 1)
        gm::win_dkv_join_kernel<D><<<(unsigned)(per * (p.nblk - p.sink_blocks) * threads / 256), 256, 0, st>>>(a, p.sink_items, p.chunks);
    return launched();
}

// ---- 8-bit cache -----------------------------------------------------------------------------------

// The sizes of a call over the cache, without its pool.
gm_status check_cache_sizes(int B, int t, int heads, int hkv, int d, int page, int max_pages)
{
    if (B < 0 || t < 0 || heads < 1 || hkv < 1 || d < 1 || heads % hkv != 0) return GM_ERR_INVALID_ARG;
    if (max_pages < 0 || page < 1) return GM_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GM_ERR_UNSUPPORTED;
    if (page != 16 && page != 32 && page != 64 && page != 128) return GM_ERR_UNSUPPORTED;
    if ((int64_t)max_pages * page >= MAX_ROWS) return GM_ERR_UNSUPPORTED;
    // two factors at a time: B * t * heads alone can pass 64 bits
    if ((int64_t)B * t >= MAX_ROWS || (int64_t)B * t * heads >= MAX_ROWS) return GM_ERR_UNSUPPORTED;
    return GM_OK;
}

gm_status check_cache(gm::Kv8 &c, void *kq, void *vq, float *kscale, float *vscale, int num_pages, int page,
                      const int32_t *table, int max_pages, const int32_t *lens, int B, int t, int heads, int hkv, int d,
                      gm_dtype dtype)
{
    if (num_pages < 0 || (dtype != GM_F32 && dtype != GM_BF16)) return GM_ERR_INVALID_ARG;
    const gm_status sizes = check_cache_sizes(B, t, heads, hkv, d, page, max_pages);
    if (sizes != GM_OK) return sizes;
    // pool rows are counted in 32 bits (2^32 of them are 256 GB and more)
    if ((int64_t)num_pages * hkv >= ((int64_t)1 << 32) / page) return GM_ERR_UNSUPPORTED;
    if ((int64_t)B * t == 0) return GM_OK;
    if (!lens || (max_pages > 0 && !table)) return GM_ERR_INVALID_ARG;
    if (num_pages > 0 && (!kq || !vq || !kscale || !vscale)) return GM_ERR_INVALID_ARG;
    if (!aligned16(kq) || !aligned16(vq)) return GM_ERR_INVALID_ARG;
    c.kq = (uint8_t *)kq;
    c.vq = (uint8_t *)vq;
    c.kscale = kscale;
    c.vscale = vscale;
    c.table = table;
    c.lens = lens;
    c.num_pages = num_pages;
    c.max_pages = num_pages > 0 ? max_pages : 0;  // an empty pool holds no token
    c.shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    return GM_OK;
}

template <typename T, int D> gm_status kv8_append(const gm::Kv8AppendArgs &a, unsigned grid, cudaStream_t st)
{
    switch (a.c.shift) {
    case 4: gm::kv8_append_kernel<T, D, 16><<<grid, 256, 0, st>>>(a); break;
    case 5: gm::kv8_append_kernel<T, D, 32><<<grid, 256, 0, st>>>(a); break;
    case 6: gm::kv8_append_kernel<T, D, 64><<<grid, 256, 0, st>>>(a); break;
    default: gm::kv8_append_kernel<T, D, 128><<<grid, 256, 0, st>>>(a); break;
    }
    return launched();
}

// How a call of gm_kv8_attention_forward is cut up: row tiles of 8 nt query rows, and the blocks
// that share the keys of one (gm_kv8.cuh).
struct Kv8Plan {
    int nt, tiles, splits;
    int64_t items;
    size_t part_bytes, bytes;  // workspace: partial outputs, then maxima and sums
};

Kv8Plan kv8_plan(int B, int t, int hq, int hkv, int d, int64_t keys)
{
    Kv8Plan p{};
    const int64_t flat = (int64_t)t * (hq / hkv);
    p.nt = flat <= 8 ? 1 : 2;
    p.tiles = (int)((flat + 8 * p.nt - 1) / (8 * p.nt));
    p.items = (int64_t)B * hkv * p.tiles;
    // Rounds of blocks that the GPU takes, times what one round lasts: a block's units of 32 keys
    // per warp and a start and end worth about four of them. The splits with the least of it.
    const int64_t room = 148 * gm::KV8_PER_SM, units = (keys + 31) / 32;
    const int64_t most = std::min<int64_t>(room, std::max<int64_t>(1, units / (2 * gm::KV8_W)));
    // Tried: no split, and as many as fill one to eight rounds.
    int64_t best = INT64_MAX;
    for (int64_t rounds = 0; rounds <= 8; ++rounds) {
        const int64_t s = rounds == 0 ? 1 : std::min(most, rounds * room / p.items);
        if (s < 1) continue;
        const int64_t cost = ((p.items * s + room - 1) / room) * ((units + s * gm::KV8_W - 1) / (s * gm::KV8_W) + 4);
        if (cost < best) {
            best = cost;
            p.splits = (int)s;
        }
        if (rounds > 0 && s == most) break;
    }
    if (p.splits > 1) {
        const size_t rows = (size_t)p.items * p.splits * 8 * p.nt;
        p.part_bytes = rows * d * 4;
        p.bytes = p.part_bytes + rows * 8;
    }
    return p;
}

// Keys that one row tile can see at most.
int64_t kv8_keys(int64_t room, int window, int sinks, int t)
{
    return std::min<int64_t>(room, (int64_t)window + sinks + t);
}

template <typename T, int D, int NT> gm_status launch_kv8_attention(const gm::Kv8AttnArgs &a, int B, int64_t items, cudaStream_t st)
{
    using Smem = gm::Kv8Smem<D, NT, sizeof(T) == 4>;
    constexpr auto kern = gm::kv8_attention_kernel<T, D, NT>;
    if (!raise_smem<kern>(sizeof(Smem))) return GM_ERR_CUDA;
    kern<<<(unsigned)(items * a.splits), gm::KV8_W * 32, sizeof(Smem), st>>>(a);
    if (a.splits > 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((int64_t)B * a.t * a.hq));
        cfg.blockDim = dim3(128);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        (void)cudaLaunchKernelEx(&cfg, gm::kv8_join_kernel<T, D, NT>, a);
    }
    return launched();
}

template <typename T, int D> gm_status kv8_attention(const gm::Kv8AttnArgs &a, int B, const Kv8Plan &p, cudaStream_t st)
{
    return p.nt == 1 ? launch_kv8_attention<T, D, 1>(a, B, p.items, st) : launch_kv8_attention<T, D, 2>(a, B, p.items, st);
}

template <typename T, int D, int NP> gm_status launch_kv8_sea(const gm::Kv8SeaArgs &a, cudaStream_t st)
{
    constexpr int smem = 4 * (int)sizeof(gm::Kv8SeaSmem<T, D, NP>);
    constexpr auto kern = gm::kv8_sea_kernel<T, D, NP>;
    if (!raise_smem<kern>(smem)) return GM_ERR_CUDA;
    // as many warps as the GPU holds at once, each taking step after step
    const int per_sm = std::max(1, std::min(4, (227 * 1024) / (smem + 1024)));
    const int64_t steps = a.tiles * ((a.G + 7) / 8);
    kern<<<(unsigned)std::min<int64_t>((steps + 3) / 4, 148 * per_sm), 128, smem, st>>>(a, GM_CHECKED);
    return launched();
}

template <typename T, int D> gm_status kv8_sea(const gm::Kv8SeaArgs &a, cudaStream_t st)
{
    return a.s <= 16 ? launch_kv8_sea<T, D, 1>(a, st) : launch_kv8_sea<T, D, 2>(a, st);
}

}  // namespace

extern "C" {

gm_status gm_window_attention_forward(const void *q, const void *k, const void *v, gm_dtype dtype, const int32_t *lens,
                                      int B, int n, int hq, int hkv, int d, int window, int sinks, float scale,
                                      void *o, float *lse, cudaStream_t stream)
{
    const gm_status st = check_window(dtype, B, n, hq, hkv, d, window, sinks, scale);
    if (st != GM_OK || (int64_t)B * n == 0) return st;
    if (!q || !k || !v || !o) return GM_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return GM_ERR_INVALID_ARG;
    g_attn_used = true;
    gm::WinArgs a = window_args(B, n, hq, hkv, window, sinks, scale, lens);
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    a.lse = lse;
    if (dtype == GM_F32) return d == 64 ? window_forward<64>(a, stream) : window_forward<128>(a, stream);
    return d == 64 ? window_forward_bf16<64>(a, stream) : window_forward_bf16<128>(a, stream);
}

size_t gm_window_attention_backward_workspace_size(gm_dtype dtype, int B, int n, int hq, int hkv, int d, int window, int sinks)
{
    if (check_window(dtype, B, n, hq, hkv, d, window, sinks, 1.0f) != GM_OK || (int64_t)B * n == 0) return 0;
    if (!window_backward_fits(dtype, B, n, hq)) return 0;
    if (dtype == GM_F32) return window_f32_plan(B, n, hq, hkv, d, window, sinks).bytes;
    return window_backward_plan(B, n, hq, hkv, d, window, sinks).bytes;
}

gm_status gm_window_attention_backward(const void *q, const void *k, const void *v, const void *o, const void *dout,
                                       const float *lse, gm_dtype dtype, const int32_t *lens, int B, int n, int hq,
                                       int hkv, int d, int window, int sinks, float scale, void *dq, void *dk, void *dv,
                                       void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    const gm_status st = check_window(dtype, B, n, hq, hkv, d, window, sinks, scale);
    if (st != GM_OK || (int64_t)B * n == 0) return st;
    if (!window_backward_fits(dtype, B, n, hq)) return GM_ERR_UNSUPPORTED;
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace) return GM_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, o, dout, (const void *)dq, (const void *)dk, (const void *)dv, (const void *)workspace})
        if (!aligned16(p)) return GM_ERR_INVALID_ARG;
    if (workspace_bytes < gm_window_attention_backward_workspace_size(dtype, B, n, hq, hkv, d, window, sinks))
        return GM_ERR_INVALID_ARG;
    g_attn_used = true;
    gm::WinArgs a = window_args(B, n, hq, hkv, window, sinks, scale, lens);
    a.q = q;
    a.k = k;
    a.v = v;
    a.o_in = o;
    a.dout = dout;
    a.lse_in = lse;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.delta = (float *)workspace;
    if (dtype == GM_F32) return d == 64 ? window_backward<64>(a, stream) : window_backward<128>(a, stream);
    return d == 64 ? window_backward_bf16<64>(a, stream) : window_backward_bf16<128>(a, stream);
}

gm_status gm_kv8_append(const void *k, const void *v, gm_dtype dtype, int B, int t, int hkv, int d, void *kq, void *vq,
                        float *kscale, float *vscale, int num_pages, int page, const int32_t *table, int max_pages,
                        const int32_t *lens, const int32_t *new_lens, cudaStream_t stream)
{
    gm::Kv8AppendArgs a{};
    const gm_status st = check_cache(a.c, kq, vq, kscale, vscale, num_pages, page, table, max_pages, lens, B, t, hkv, hkv,
                                     d, dtype);
    if (st != GM_OK || (int64_t)B * t == 0) return st;
    if (!k || !v || !aligned16(k) || !aligned16(v)) return GM_ERR_INVALID_ARG;
    g_attn_used = true;
    a.k = k;
    a.v = v;
    a.new_lens = new_lens;
    a.B = B;
    a.t = t;
    a.hkv = hkv;
    a.touch = (int)(((int64_t)t + page - 2) / page + 1);
    const int64_t grid = (int64_t)B * a.touch * hkv * 2;
    if (grid >= MAX_ROWS) return GM_ERR_UNSUPPORTED;
    if (dtype == GM_F32)
        return d == 64 ? kv8_append<float, 64>(a, (unsigned)grid, stream) : kv8_append<float, 128>(a, (unsigned)grid, stream);
    return d == 64 ? kv8_append<__nv_bfloat16, 64>(a, (unsigned)grid, stream)
                   : kv8_append<__nv_bfloat16, 128>(a, (unsigned)grid, stream);
}

size_t gm_kv8_attention_workspace_size(int B, int t, int hq, int hkv, int d, int page, int max_pages, int window, int sinks)
{
    if (check_cache_sizes(B, t, hq, hkv, d, page, max_pages) != GM_OK || (int64_t)B * t == 0 || window < 1 || sinks < 0) return 0;
    return kv8_plan(B, t, hq, hkv, d, kv8_keys((int64_t)max_pages * page, window, sinks, t)).bytes;
}

gm_status gm_kv8_attention_forward(const void *q, gm_dtype dtype, int B, int t, int hq, int hkv, int d, const void *kq,
                                   const void *vq, const float *kscale, const float *vscale, int num_pages, int page,
                                   const int32_t *table, int max_pages, const int32_t *lens, const int32_t *q_lens,
                                   int window, int sinks, float scale, void *o, float *lse, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream)
{
    gm::Kv8AttnArgs a{};
    const gm_status st = check_cache(a.c, const_cast<void *>(kq), const_cast<void *>(vq), const_cast<float *>(kscale),
                                     const_cast<float *>(vscale), num_pages, page, table, max_pages, lens, B, t, hq, hkv,
                                     d, dtype);
    if (window < 1 || sinks < 0 || !good_scale(scale)) return GM_ERR_INVALID_ARG;
    if (st != GM_OK || (int64_t)B * t == 0) return st;
    if (!q || !o || !aligned16(q) || !aligned16(o)) return GM_ERR_INVALID_ARG;
    const Kv8Plan p = kv8_plan(B, t, hq, hkv, d, kv8_keys((int64_t)max_pages * page, window, sinks, t));
    if (p.items * p.splits >= MAX_ROWS) return GM_ERR_UNSUPPORTED;
    if (p.bytes > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < p.bytes)) return GM_ERR_INVALID_ARG;
    g_attn_used = true;
    a.q = q;
    a.q_lens = q_lens;
    a.o = o;
    a.lse = lse;
    a.t = t;
    a.hq = hq;
    a.hkv = hkv;
    a.G = hq / hkv;
    a.tiles = p.tiles;
    a.splits = p.splits;
    a.part = (float *)workspace;
    a.ml = (float2 *)((char *)workspace + p.part_bytes);
    const int64_t room = (int64_t)a.c.max_pages * page;
    a.window = (int)std::min<int64_t>(window, std::max<int64_t>(room, 1));
    a.sinks = (int)std::min<int64_t>(sinks, room);
    a.sl2 = scale * gm::LOG2E;
    if (dtype == GM_F32)
        return d == 64 ? kv8_attention<float, 64>(a, B, p, stream) : kv8_attention<float, 128>(a, B, p, stream);
    return d == 64 ? kv8_attention<__nv_bfloat16, 64>(a, B, p, stream) : kv8_attention<__nv_bfloat16, 128>(a, B, p, stream);
}

gm_status gm_kv8_sea_forward(const void *q, gm_dtype dtype, const int32_t *idx, const float *w, int s, int B, int t,
                             int hq, int hkv, int d, const void *kq, const void *vq, const float *kscale,
                             const float *vscale, int num_pages, int page, const int32_t *table, int max_pages,
                             const int32_t *lens, const int32_t *q_lens, float scale, void *o, float *lse,
                             cudaStream_t stream)
{
    gm::Kv8SeaArgs a{};
    const gm_status st = check_cache(a.c, const_cast<void *>(kq), const_cast<void *>(vq), const_cast<float *>(kscale),
                                     const_cast<float *>(vscale), num_pages, page, table, max_pages, lens, B, t, hq, hkv,
                                     d, dtype);
    if (s < 1 || s > 32 || !good_scale(scale)) return GM_ERR_INVALID_ARG;
    if (st != GM_OK || (int64_t)B * t == 0) return st;
    if (!q || !o || !idx || !w || !aligned16(q) || !aligned16(o)) return GM_ERR_INVALID_ARG;
    g_attn_used = true;
    a.q = q;
    a.idx = idx;
    a.w = w;
    a.q_lens = q_lens;
    a.o = o;
    a.lse = lse;
    a.t = t;
    a.hkv = hkv;
    a.G = hq / hkv;
    a.s = s;
    while ((1 << a.s_shift) < s) ++a.s_shift;
    a.rows = (int64_t)B * t * hkv;
    while (a.g_shift < 3 && (1 << a.g_shift) < a.G) ++a.g_shift;
    a.rt = std::min(std::max(16 >> a.s_shift, 1), 8 >> a.g_shift);
    a.tiles = (a.rows + a.rt - 1) / a.rt;
    a.div_h = gm::FastDiv((uint32_t)hkv);
    a.div_t = gm::FastDiv((uint32_t)t);
    a.sl2 = scale * gm::LOG2E;
    if (dtype == GM_F32) return d == 64 ? kv8_sea<float, 64>(a, stream) : kv8_sea<float, 128>(a, stream);
    return d == 64 ? kv8_sea<__nv_bfloat16, 64>(a, stream) : kv8_sea<__nv_bfloat16, 128>(a, stream);
}

}  // extern "C"
