// tree_tc.cu -- attention of drafted tokens over a paged cache on the
// 5th-generation tensor cores (bf16 pools; tree.cuh says what is computed and
// how the work is cut into shares).
//
// One CTA per SM takes a share of the work line.  A unit's rows are one or two
// MMA tiles of 128 rows; K and V come in tiles of 128 tokens, worked through in
// halves of 64.  Two streams, each with its own four softmax warps, two S / P
// buffers and an O accumulator in tensor memory, keep the tensor cores and the
// exponentials busy at once:
//   more than 128 rows: stream w owns row tile w and takes every half, so K and V
//                       are read once for up to 256 rows;
//   up to 128 rows:     both streams hold the same rows, stream w takes half w of
//                       every tile; the epilogue joins the two.
// Step k of a stream (buffer k % 2) is
//   S = Q . K^T   (M = 128 rows, N = 64 tokens, K = d)
//   softmax       (online, base 2, lazy rescale of O in tensor memory)
//   O += P . V    (M = 128, N = d, K = 64 tokens; P as a bf16 pair hi + lo,
//                  written over S: about 16 significant bits, so that the
//                  weights' rounding stays below the output's)
// While a stream's warps work on step k, the tensor cores do PV(k - 1) and S(k + 1)
// in the other buffer.  (One buffer of 128 tokens per stream, which is what tensor
// memory holds next to two O of d = 128, took 266 against 260 us on 64 sequences of
// 128 to 8191 tokens with up to 132 rows per kv head, and 461 against 474 us on 8 of
// 8192 to 32768 tokens with up to 512.)
//
// K and V tiles go through one ring of five 32 KB slots in the order K0 V0 K1
// V1 ...; a K slot is free again once its S are done, so up to 160 KB are in
// flight or in use.  Two loader warps, one for K and one for V, run ahead into
// the CTA's next runs.  One bulk copy brings a whole block, or 64
// columns of a block of four tokens (64 copies per slot at d = 128, which bound the
// kernel: 64 130 tokens of one sequence, 40 / 8 heads, take 167 us; 1155 us on the
// CUDA cores).  Next to busy softmax
// warps a loader needs 2150 cycles for a slot of 8-token blocks (460 alone): one
// warp for both pools held an SM at 22 GB/s.
//
// Per 128-token tile: 64 KB of K and V, 1.5 us at an SM's share of the measured
// copy bandwidth; per 128 rows 768 (S: 48 cycles per MMA at N = 64) + 1024 tensor
// cycles and 1024 cycles of exponentials on each SM quarter.  Up to 128 rows the
// kernel is bound by HBM; 256 rows take 3600 tensor cycles per tile, 1.9 us.
//
// Every wait is bounded: on a timeout the CTA raises PA_DEVERR_TIMEOUT, skips
// what is left, lets its copies and MMAs drain, frees its tensor memory and
// returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_tma.h"
#include "pa_umma.cuh"
#include "tree.cuh"

namespace pa {
namespace {

constexpr int TT_M = 128;               // rows of a stream: the MMA's M
constexpr int TT_ROWS = 2 * TT_M;       // rows of a unit
constexpr int TT_KT = 128;              // tokens of a K or V tile
constexpr int TT_HT = TT_KT / 2;         // tokens of a step
constexpr int TT_SLOTS = 5;             // ring slots (one K or V tile each)
constexpr int TT_MASKS = 4;             // tiles whose token masks are kept
constexpr int TT_SOFTMAX_WARPS = 8;     // warps 0-3: stream 0, 4-7: stream 1
constexpr int TT_SOFTMAX = TT_SOFTMAX_WARPS * 32;
constexpr int TT_MMA_WARP = 8;
constexpr int TT_K_WARP = 9;            // copies of K, of V
constexpr int TT_V_WARP = 10;
constexpr int TT_THREADS = (TT_SOFTMAX_WARPS + 3) * 32;
constexpr int TT_TMEM_COLS = 512;
constexpr int TT_Q_BARRIER = 1;         // Q in shared memory, O read: softmax + MMA warps
constexpr int TT_ML_BARRIER = 2;        // the streams' (max, sum) exchanged: softmax warps
constexpr int TT_MASK_WORDS = TT_KT / 32;
// Steps whose P.V meet in one accumulator.  An accumulating MMA cuts its sum off at 24 bits
// instead of rounding it, so O shrinks a little with every product: by 1e-7 of itself per
// step (measured; 8 products each), 5e-5 over a run of 512 steps.  After this many steps O
// is folded into a sum in the workspace, which rounds: 9e-6 of error however long the run.
// (8 sequences of 8192 to 32768 tokens, 512 rows per kv head: 593 us without folds, 606 us
// with one every 64 steps, 623 us every 32.)
constexpr int TT_FOLD = 64;

template <int D>
struct TreeGeom {
    static constexpr int NH = D / 64;
    static constexpr int Q_HALF = TT_M * 128;          // 128 rows x 64 columns, 128-byte swizzle
    static constexpr int Q_TILE = NH * Q_HALF;
    // K and V: 8-row groups of NH 64-column halves, as the copies lay blocks out
    static constexpr int GROUP = NH * 1024;
    static constexpr int SLOT = TT_KT / 8 * GROUP;
    static constexpr int OFF_SLOTS = 2 * Q_TILE;
    static constexpr int BYTES = OFF_SLOTS + TT_SLOTS * SLOT;
    // tensor memory columns: S / P of stream w, buffer b at 128 w + 64 b, O of stream w
    // behind them
    static constexpr int O_COL = 4 * TT_HT;
    static_assert(O_COL + 2 * D <= TT_TMEM_COLS, "tensor memory");
    static_assert(TREE_WINDOWS_MAX * 4 <= TT_SLOTS * SLOT, "window sums fit the ring");
};

constexpr uint32_t TT_IDESC_S = umma_idesc_bf16(TT_M, TT_HT, 0, 0);

struct TreeShared {
    uint64_t full[TT_SLOTS], empty[TT_SLOTS];
    uint64_t masked[TT_MASKS];     // the tile's token mask is written
    uint64_t s_full[2][2];         // [stream][buffer]: S of the step is in tensor memory
    uint64_t p_full[2][2];         // its weights are (128 arrivals)
    uint64_t o_done[2][2];         // its P.V has finished
    uint64_t drain;
    int odd_run;                   // last run (counted from 1) with a non-finite value element among its nodes
    alignas(16) uint32_t mask[TT_MASKS][TT_MASK_WORDS];
    uint32_t tmem;
    int abort_flag;
};

// Bulk tensor copy of box (0, 0, part, block) of a map of half groups.
__device__ __forceinline__ void tt_load_half_group_elected(uint32_t elected, uint32_t dst, const void* tensor_map, uint32_t bar,
                                                           int part, int block) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %6, 0;\n\t"
        "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %3, %4, %5}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tensor_map)), "r"(bar), "r"(0), "r"(part), "r"(block), "r"(elected)
        : "memory");
}

// Bounds a loop of polls: true once WAIT_LIMIT_NS have passed since the first
// of them.  The global timer is slow to read: only every 256th poll looks.
struct PollLimit {
    uint32_t polls = 0;
    uint64_t t0 = 0;
    __device__ __forceinline__ bool out() {
        if (++polls & 255u) return false;
        const uint64_t t = global_timer_ns();
        if (t0 == 0) t0 = t;
        return t - t0 > WAIT_LIMIT_NS;
    }
};

__device__ __forceinline__ bool tt_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* dev_err) {
    const uint32_t b = smem_u32(bar);
    PollLimit limit;
    while (!mbar_try_wait(b, parity)) {
        if (*abort_flag) return false;
        if (limit.out()) {
            *abort_flag = 1;
            flag_error(dev_err, PA_DEVERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

// A row's maximum was raised before chunk c of a step: scales what was summed with
// the old one, O (when scale_o, once `bar` says that none of the stream's P.V runs)
// and the step's weights before chunk c, which are rounded to their 16 bits again.  Out of
// line: it is rare, and the loop that calls it has to stay small for the
// instruction caches (inlined, the softmax took 1.3 times as long).
template <int D>
__device__ __noinline__ bool tt_rescale(uint32_t o_col, uint32_t s_col, float alpha, int c, bool scale_o, uint64_t* bar,
                                        uint32_t parity, volatile int* abort_flag, int32_t* dev_err) {
    if (scale_o) {
        const bool done = tt_wait(bar, parity, abort_flag, dev_err);
        if (!__all_sync(FULL_MASK, done)) return false;
        tmem_fence_after_sync();
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            tmem_load32(o_col + c0, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= alpha;
            tmem_store32(o_col + c0, o);
        }
    }
    if (c > 0) {
        tmem_await_stores();
        const uint32_t col = s_col + 32 * (c - 1);
        uint32_t pw[32];
        tmem_issue32(col, pw);
        tmem_await32(pw);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float p = (bf16_lo(pw[k]) + bf16_lo(pw[16 + k])) * alpha;
            const float q = (bf16_hi(pw[k]) + bf16_hi(pw[16 + k])) * alpha;
            pw[k] = pack_bf16(p, q);
            pw[16 + k] = pack_bf16(p - bf16_lo(pw[k]), q - bf16_hi(pw[k]));
        }
        tmem_store32_bits(col, pw);
    }
    return true;
}

// Moves a row's O, which belongs to the running maximum m, into its sum in the workspace,
// once `bar` says that none of the stream's P.V runs (fresh: the run's first fold), or,
// back: adds that sum to O.  `at` keeps the sum's maximum.  Sum and maximum are
// the thread's own.  Out of line like tt_rescale.
template <int D>
__device__ __noinline__ bool tt_fold(uint32_t o_col, float4* sum, int stride, float* at, float m, bool fresh, bool back, bool valid,
                                     uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* dev_err) {
    const bool done = tt_wait(bar, parity, abort_flag, dev_err);
    if (!__all_sync(FULL_MASK, done)) return false;
    tmem_fence_after_sync();
    float e = 0.f;
    if (valid && !fresh) {
        const float before = *at;
        e = before == NEG_INF ? 0.f : exp2_approx(before - m);
    }
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = valid && !fresh ? __ldcg(sum + (c / 4 + k) * stride) : make_float4(0.f, 0.f, 0.f, 0.f);
        float o[32];
        tmem_load32(o_col + c, o);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            o[4 * k + 0] = fmaf(v[k].x, e, o[4 * k + 0]);
            o[4 * k + 1] = fmaf(v[k].y, e, o[4 * k + 1]);
            o[4 * k + 2] = fmaf(v[k].z, e, o[4 * k + 2]);
            o[4 * k + 3] = fmaf(v[k].w, e, o[4 * k + 3]);
        }
        if (back) {
            tmem_store32(o_col + c, o);
        } else if (valid) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                __stcg(sum + (c / 4 + k) * stride, make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
        }
        __syncwarp();
    }
    if (valid && !back) *at = m;
    return true;
}

// Both bf16 halves, non-finite ones as 0.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v) {
    if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
    if ((v & 0x7f800000u) == 0x7f800000u) v &= 0x0000ffffu;
    return v;
}

// Adds the non-finite value elements of the nodes at positions [from, to) that a row
// sees to columns [c0, c0 + cols) of its O (times a positive weight they stay what
// they are).  Read from the pool again, a row per thread of the warp: this is for
// models that have come apart.
template <int D>
__device__ __noinline__ void tt_add_odd(const void* v_cache, int num_blocks, int num_kv_heads, int log2_block, uint32_t o_col,
                                        int c0, int cols, const int32_t* table, int kvh, const uint32_t* mrow, int words,
                                        int pre, int from, int to, bool valid) {
#pragma unroll 1
    for (int c = c0; c < c0 + cols; c += 32) {
        float o[32];
        tmem_load32(o_col + c, o);
        for (int p = from; p < to; ++p) {
            if (!valid || !(tree_bits(mrow, words, p - pre) & 1u)) continue;
            const int b = table[p >> log2_block];
            if (b < 0 || b >= num_blocks) continue;
            const uint32_t* v = reinterpret_cast<const uint32_t*>(
                static_cast<const __nv_bfloat16*>(v_cache) +
                (((static_cast<size_t>(b) * num_kv_heads + kvh) << log2_block) + (p & ((1 << log2_block) - 1))) * D + c);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint32_t w = v[k], odd = w ^ finite_bf16x2(w);
                if ((odd & 0xffffu) != 0u) o[2 * k] += bf16_lo(w);
                if ((odd >> 16) != 0u) o[2 * k + 1] += bf16_hi(w);
            }
        }
        __syncwarp();
        tmem_store32(o_col + c, o);
    }
}

template <int D>
__global__ void __launch_bounds__(TT_THREADS, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const TreeArgs a) {
    using Geo = TreeGeom<D>;
    constexpr int NH = Geo::NH, KS = D / 16;
    constexpr uint32_t IDESC_O = umma_idesc_bf16(TT_M, D, 0, 1);

    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    __shared__ TreeShared sh;
    volatile int* abort_flag = &sh.abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        sh.abort_flag = 0;
        sh.odd_run = 0;
        for (int i = 0; i < TT_SLOTS; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < TT_MASKS; ++i) mbar_init(smem_u32(&sh.masked[i]), 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_u32(&sh.s_full[i >> 1][i & 1]), 1);
            mbar_init(smem_u32(&sh.p_full[i >> 1][i & 1]), TT_M);
            mbar_init(smem_u32(&sh.o_done[i >> 1][i & 1]), 1);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        fence_barrier_init();
        prefetch_tensor_map(&tm_k);
        prefetch_tensor_map(&tm_v);
    }
    if (warp == 0) tmem_alloc(smem_u32(&sh.tmem), TT_TMEM_COLS);
    pdl_wait();
    pdl_launch_dependents();
    TreeWalker<TT_M, 2, TT_KT> walk;
    tree_begin(a, reinterpret_cast<int*>(smem + Geo::OFF_SLOTS), walk);
    fence_proxy_async_smem();   // the window sums lie where copies land next
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const uint32_t sQ = smem_u32(smem), sSlots = smem_u32(smem + Geo::OFF_SLOTS);
    const int B = a.block_size;

    TreeRun r;
    if (warp == TT_K_WARP || warp == TT_V_WARP) {
        // ---- copies ---------------------------------------------------------
        const bool is_v = warp == TT_V_WARP;
        const CUtensorMap* map = is_v ? &tm_v : &tm_k;
        uint32_t ring = is_v ? 1 : 0, tiles = 0;   // ring position and tiles passed so far
        bool ok = true;
        const uint32_t leader = elect_one();
        const int per = TT_KT / B;      // blocks of a tile: one lane each
        const uint32_t slots = __shfl_sync(FULL_MASK, sSlots, 0);
        while (ok && walk.next(a, r)) {
            if (r.starts && !is_v && lane == 0) tree_record(a, r);
            const int32_t* table = a.block_tables + static_cast<size_t>(r.s) * a.max_blocks;
            auto entry_at = [&](int t) {   // the lane's block-table entry of tile t, -2 past the context
                const int p = t * TT_KT + lane * B;
                return t < r.t1 && lane < per && p < r.ctx ? table[p >> a.log2_block] : -2;
            };
            int entry = entry_at(r.t0);
            for (int t = r.t0; t < r.t1; ++t) {
                const int next = entry_at(t + 1);
                const bool bad = entry != -2 && (entry < 0 || entry >= a.num_blocks);
                const bool here = entry >= 0 && !bad;
                if (bad) flag_error(a.dev_err, PA_DEVERR_BLOCK_ID);
                const uint32_t valid = __ballot_sync(FULL_MASK, here);
                const uint32_t bytes = __popc(valid) * NH * static_cast<uint32_t>(B) * 128u;
                const int group = here ? (entry * a.num_kv_heads + r.kvh) * (B < 8 ? 1 : B / 8) : 0;
                const uint32_t slot = ring % TT_SLOTS;
                bool w = true;
                if (ring >= TT_SLOTS) w = tt_wait(&sh.empty[slot], ((ring / TT_SLOTS) - 1) & 1u, abort_flag, a.dev_err);
                if (!__all_sync(FULL_MASK, w)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_u32(&sh.full[slot]);
                mbar_arrive_expect_tx_elected(leader, bar, bytes);
                const uint32_t dst = slots + slot * Geo::SLOT;
                for (int i = 0; i < per; i += 4) {   // four at a time: their shuffles overlap
                    int at[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) at[u] = __shfl_sync(FULL_MASK, group, i + u);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (B >= 8) {
                            tma_load_group_elected(leader & (valid >> (i + u)), dst + (i + u) * (B / 8) * Geo::GROUP, map, bar, at[u]);
                            continue;
                        }
#pragma unroll
                        for (int h = 0; h < NH; ++h)
                            tt_load_half_group_elected(leader & (valid >> (i + u)),
                                                       dst + ((i + u) >> 1) * Geo::GROUP + h * 1024 + (u & 1) * 512, map, bar, h, at[u]);
                    }
                }
                if (!is_v) {
                    // tokens of the tile that take part: in the context and in a valid
                    // block.  The mask's ring entry is free: the slot of K was last
                    // used two tiles and a half ago, by a tile whose step (and those
                    // before it) has been through softmax.
                    const int left = r.ctx - t * TT_KT - lane * B;
                    uint32_t part = 0;
                    if (here) part = left >= B ? (B == 32 ? 0xffffffffu : (1u << B) - 1u) : (1u << left) - 1u;
                    const int lanes_per_word = 32 / B;
                    part <<= (lane % lanes_per_word) * B;
                    for (int o = 1; o < lanes_per_word; o <<= 1) part |= __shfl_xor_sync(FULL_MASK, part, o);
                    if (lane < per && lane % lanes_per_word == 0) sh.mask[tiles % TT_MASKS][lane / lanes_per_word] = part;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.masked[tiles % TT_MASKS]));
                }
                ring += 2;
                ++tiles;
                entry = next;
            }
        }
        // after a timeout: the latest copy into every slot must have landed
        if (*abort_flag && lane == 0) {
            for (uint32_t g = ring; g >= 2 && ring - g < 2 * TT_SLOTS; g -= 2)
                mbar_wait_bounded(smem_u32(&sh.full[(g - 2) % TT_SLOTS]), ((g - 2) / TT_SLOTS) & 1u, DRAIN_LIMIT_NS);
        }
    } else if (warp == TT_MMA_WARP) {
        // ---- MMAs -----------------------------------------------------------
        // The whole warp runs this loop and one elected lane issues.
        const uint32_t leader = elect_one();
        const uint32_t utmem = __shfl_sync(FULL_MASK, tmem, 0);
        const uint64_t q_desc = umma_desc_sw128(__shfl_sync(FULL_MASK, sQ, 0), 16, 1024);
        const uint64_t k_desc = umma_desc_sw128(__shfl_sync(FULL_MASK, sSlots, 0), 16, Geo::GROUP);
        const uint64_t v_desc = umma_desc_sw128(__shfl_sync(FULL_MASK, sSlots, 0), 1024, Geo::GROUP);
        const uint32_t bars = __shfl_sync(FULL_MASK, smem_u32(&sh), 0);
        auto bar_at = [&](const uint64_t* first, uint32_t i) {
            return bars + static_cast<uint32_t>(reinterpret_cast<const uint8_t*>(first) - reinterpret_cast<const uint8_t*>(&sh)) + 8u * i;
        };
        auto passed = [&](uint32_t bar, uint32_t parity) { return __all_sync(FULL_MASK, mbar_test_wait(bar, parity)); };
        uint32_t base = 0;                    // steps of each stream in earlier runs (the same for both)
        uint32_t k_slot = 0, k_phase = 0;     // ring slot of the next S's K and its phase
        uint32_t v_slot = 1, v_phase = 0;     // of the next P.V's V
        auto advance = [](uint32_t& slot, uint32_t& phase) {
            slot += 2;
            if (slot >= TT_SLOTS) {
                slot -= TT_SLOTS;
                phase ^= 1u;
            }
        };
        while (walk.next(a, r)) {
            named_barrier_sync(TT_Q_BARRIER, TT_SOFTMAX + 32);   // Q written, O of the last run read
            const bool two = __shfl_sync(FULL_MASK, r.per_tile, 0) == 2;   // every half is a step of both streams
            const int nt = __shfl_sync(FULL_MASK, r.t1 - r.t0, 0);
            const int last = two ? 3 : 1, steps = (last + 1) * nt;   // i & last == last: a tile's last step
            if (__any_sync(FULL_MASK, *abort_flag)) continue;
            tmem_fence_after_sync();
            // Step i of the run: stream i % 2, its step base + i / 2, whose parity is
            // the buffer and whose half is the buffer's phase.  S(i) needs its K and
            // P.V(i - 4) done with the buffer; P.V(i) needs its weights and its V.  The
            // first stream to end, whose last P.V is steps - 2, writes the next run's Q
            // over both tiles: that P.V comes after the other stream's last S (whose K
            // is in the same tile), so that its commit stands for both.
            // Each goes in order; the barriers are tested without blocking.
            int ns = 0, no = 0;
            bool k_here = false, v_here = false;   // the slot's copy was seen to have landed
            PollLimit limit;
            while (no < steps) {
                bool progressed = false;
                if (ns < steps && ns < no + 4 && (k_here || (k_here = passed(bar_at(sh.full, k_slot), k_phase)))) {
                    const uint32_t w = ns & 1, use = base + (ns >> 1), buf = use & 1u;
                    if (ns < 4 || passed(bar_at(&sh.o_done[0][0], 2 * w + buf), ((use >> 1) & 1u) ^ 1u)) {
                        tmem_fence_after_sync();
                        const uint32_t half = two ? (ns >> 1) & 1 : w;
                        const uint64_t qd = q_desc + (two && w ? Geo::Q_TILE >> 4 : 0);
                        const uint64_t kd = k_desc + ((k_slot * Geo::SLOT + half * (Geo::SLOT / 2)) >> 4);
                        const uint32_t s_tmem = utmem + TT_KT * w + TT_HT * buf;
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            // k-step inside a 128-byte row, 64-column half
                            constexpr int STEP = 32 >> 4;
                            umma_bf16_elected(leader, s_tmem, qd + (ks % 4) * STEP + (ks / 4) * (Geo::Q_HALF >> 4),
                                              kd + (ks % 4) * STEP + (ks / 4) * (1024 >> 4), TT_IDESC_S,
                                              ks > 0 ? 1u : 0u);
                        }
                        umma_commit_elected(leader, bar_at(&sh.s_full[0][0], 2 * w + buf));
                        if ((ns & last) == last) {   // K's last reader
                            umma_commit_elected(leader, bar_at(sh.empty, k_slot));
                            advance(k_slot, k_phase);
                            k_here = false;
                        }
                        ++ns;
                        progressed = true;
                    }
                }
                if (no < ns && (no + 2 != steps || ns == steps)) {
                    const uint32_t w = no & 1, use = base + (no >> 1), buf = use & 1u;
                    if (passed(bar_at(&sh.p_full[0][0], 2 * w + buf), (use >> 1) & 1u) &&
                        (v_here || (v_here = passed(bar_at(sh.full, v_slot), v_phase)))) {
                        tmem_fence_after_sync();
                        const uint32_t half = two ? (no >> 1) & 1 : w;
                        const uint64_t vd = v_desc + ((v_slot * Geo::SLOT + half * (Geo::SLOT / 2)) >> 4);
                        const uint32_t p_tmem = utmem + TT_KT * w + TT_HT * buf;
                        const uint32_t o_tmem = utmem + Geo::O_COL + D * w;
                        // 0: the stream's first step of the run, or the first since O was folded
                        const uint32_t more = ((no >> 1) & (TT_FOLD - 1)) != 0 ? 1u : 0u;
#pragma unroll
                        for (int kk = 0; kk < TT_HT / 16; ++kk) {
                            const uint32_t p = p_tmem + 32 * (kk / 2) + 8 * (kk % 2);
                            umma_bf16_tmem_a_elected(leader, o_tmem, p, vd + kk * (2 * Geo::GROUP >> 4), IDESC_O, kk > 0 ? 1u : more);
                            umma_bf16_tmem_a_elected(leader, o_tmem, p + 16, vd + kk * (2 * Geo::GROUP >> 4), IDESC_O, 1u);
                        }
                        if ((no & last) == last) {
                            umma_commit_elected(leader, bar_at(sh.empty, v_slot));
                            advance(v_slot, v_phase);
                            v_here = false;
                        }
                        umma_commit_elected(leader, bar_at(&sh.o_done[0][0], 2 * w + buf));
                        ++no;
                        progressed = true;
                    }
                }
                if (progressed) {
                    limit = PollLimit();
                    continue;
                }
                // Nothing to issue: sleep on what most likely comes next (the weights of
                // the step in turn, or K), but not long, since anything may.  Polling
                // without a pause takes issue slots from the softmax warps beside it.
                if (no < ns) {
                    const uint32_t w = no & 1, use = base + (no >> 1);
                    mbar_try_wait_for(bar_at(&sh.p_full[0][0], 2 * w + (use & 1u)), (use >> 1) & 1u, 200);
                } else {
                    mbar_try_wait_for(bar_at(sh.full, k_slot), k_phase, 200);
                }
                __syncwarp();
                if (__any_sync(FULL_MASK, *abort_flag)) {
                    break;
                } else if (__any_sync(FULL_MASK, limit.out())) {
                    *abort_flag = 1;
                    if (leader) flag_error(a.dev_err, PA_DEVERR_TIMEOUT);
                    break;
                }
            }
            base += steps / 2;
        }
        if (__any_sync(FULL_MASK, *abort_flag)) {   // every MMA issued so far
            umma_commit_elected(leader, smem_u32(&sh.drain));
            mbar_wait_bounded(smem_u32(&sh.drain), 0, DRAIN_LIMIT_NS);
        }
    } else {
        // ---- softmax --------------------------------------------------------
        const int w = warp >> 2;                  // stream
        const int row = tid & (TT_M - 1);         // row of the stream's tile = tensor memory lane
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t o_col = lanes + Geo::O_COL + D * w;
        // a zero scale would turn the masked -inf into NaN: the smallest normal
        // numbers leave every weight of a row at 1 just as well
        const float sl2 = a.scale_log2 == 0.f ? 1e-37f : a.scale_log2;
        uint32_t ring = 0, tiles = 0, use = 0;    // ring position and tile of the run's start; the stream's steps
        int run = 0;                              // runs so far
        while (walk.next(a, r)) {
            ++run;
            const bool two = r.per_tile == 2;
            const int nt = r.t1 - r.t0;
            // Q: one or two tiles of 128 rows; rows past the unit's are zero.  A thread
            // loads chunk ch of every STRIDE-th row; (node, head) step along.
            {
                constexpr int CH = D / 8, STRIDE = TT_SOFTMAX / CH, BATCH = 8;
                const int ch = tid % CH, G = a.group;
                const int by_node = STRIDE / G, by_head = STRIDE - by_node * G;
                int rr = tid / CH;
                int node = (r.row0 + rr) / G, head = r.row0 + rr - node * G;
                const uint4* q = reinterpret_cast<const uint4*>(a.q) + ch;
                const int rows = two ? 2 * TT_M : TT_M;
                while (rr < rows) {
                    uint4 v[BATCH];
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        v[k] = make_uint4(0u, 0u, 0u, 0u);
                        if (rr + k * STRIDE < r.rows)
                            v[k] = __ldg(q + (static_cast<size_t>(r.first + node) * a.num_heads + r.kvh * G + head) * CH);
                        node += by_node;
                        head += by_head;
                        if (head >= G) {
                            head -= G;
                            ++node;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const int i = rr + k * STRIDE;
                        if (i < rows)
                            *reinterpret_cast<uint4*>(smem + (i / TT_M) * Geo::Q_TILE + (ch / 8) * Geo::Q_HALF +
                                                      (i % TT_M) * 128 + (((ch % 8) ^ (i & 7)) << 4)) = v[k];
                    }
                    rr += BATCH * STRIDE;
                }
            }
            fence_proxy_async_smem();
            tmem_fence_before_sync();   // the last run's O was read
            named_barrier_sync(TT_Q_BARRIER, TT_SOFTMAX + 32);

            const int R = (two ? w * TT_M : 0) + row;       // row of the unit
            const bool valid = R < r.rows;
            const bool busy = R - (row & 31) < r.rows;      // the warp has a valid row
            const int node = valid ? (r.row0 + R) / a.group : 0;
            const uint32_t* mrow = a.tree_mask + static_cast<size_t>(r.first + node) * a.mask_words32;
            const int pre = r.ctx - r.n;
            float m = NEG_INF, l = 0.f;
            bool ok = __all_sync(FULL_MASK, !*abort_flag);
            const int steps = two ? 2 * nt : nt;
            // O's folded sum: in the run's partial, where nothing lies yet (a run that leaves
            // none uses the last one's), a row for every row of both streams
            auto fold = [&](bool fresh, bool back) {
                const int slot = 2 * blockIdx.x + (r.starts ? 0 : 1), i = two ? R : w * (a.part_rows / 2) + row;
                return tt_fold<D>(o_col, reinterpret_cast<float4*>(tree_part(a, slot, D)) + i, a.part_rows,
                                  &a.part_ml[static_cast<size_t>(slot) * a.part_rows + i].x, m, fresh, back, valid,
                                  &sh.o_done[w][(use - 1) & 1u], ((use - 1) >> 1) & 1u, abort_flag, a.dev_err);
            };
            for (int step = 0; step < steps && ok; ++step, ++use) {
                const int j = two ? step >> 1 : step, h = two ? step & 1 : w;   // tile of the run, half of the tile
                const uint32_t s_col = lanes + TT_KT * w + TT_HT * (use & 1u);
                const uint32_t mi = (tiles + j) % TT_MASKS;
                const uint32_t vg = ring + 2 * j + 1, vslot = vg % TT_SLOTS;
                bool ready = tt_wait(&sh.masked[mi], ((tiles + j) / TT_MASKS) & 1u, abort_flag, a.dev_err);
                const uint2 in = *reinterpret_cast<const uint2*>(&sh.mask[mi][2 * h]);
                ready = ready && tt_wait(&sh.s_full[w][use & 1u], (use >> 1) & 1u, abort_flag, a.dev_err);
                const bool all_in = (in.x & in.y) == 0xffffffffu;
                const int p0 = (r.t0 + j) * TT_KT + h * TT_HT;
                const bool every = all_in && p0 + TT_HT <= pre;   // every token seen by every row
                if (!every) ready = ready && tt_wait(&sh.full[vslot], (vg / TT_SLOTS) & 1u, abort_flag, a.dev_err);
                if (!__all_sync(FULL_MASK, ready)) {
                    ok = false;
                    break;
                }
                tmem_fence_after_sync();
                // Value rows of tokens that take no part may hold anything, NaN too: zero
                // them, so that 0 * V stays 0.  A node's non-finite value elements must
                // not reach the rows that do not see it (weight 0) either: they become
                // zero, and the epilogue gives them to the rows that do.  (Two row tiles
                // share the half: stream 0's P.V comes first, and its warps do it.)
                if (!every && (!two || w == 0)) {
                    uint8_t* vs = smem + Geo::OFF_SLOTS + vslot * Geo::SLOT + h * (Geo::SLOT / 2);
                    bool odd = false;
                    for (int i = row; i < TT_HT * NH * 8; i += TT_M) {
                        const int tok = i / (NH * 8), ch = i % (NH * 8);
                        uint4* at = reinterpret_cast<uint4*>(vs + (tok / 8) * Geo::GROUP + (ch / 8) * 1024 + (tok % 8) * 128 + (ch % 8) * 16);
                        if (!(((tok < 32 ? in.x : in.y) >> (tok & 31)) & 1u)) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                        } else if (p0 + tok >= pre) {
                            const uint4 v = *at;
                            const uint4 f = make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z), finite_bf16x2(v.w));
                            if (((v.x ^ f.x) | (v.y ^ f.y) | (v.z ^ f.z) | (v.w ^ f.w)) != 0u) {
                                *at = f;
                                odd = true;
                            }
                        }
                    }
                    if (odd) *const_cast<volatile int*>(&sh.odd_run) = run;
                    fence_proxy_async_smem();
                }
                if (busy) {
                    const float unseen = sl2 >= 0.f ? NEG_INF : INFINITY;   // times the scale: -inf
                    // One pass over S, 32 columns at a time with the next 32 under way:
                    // the running maximum is raised lazily (by more than
                    // RESCALE_THRESHOLD), and then everything before the chunk is scaled
                    // down: the sum, O, and the step's weights already written.
                    // That is rare after a run's first tiles; a pass of its own for the
                    // maximum took a quarter of the softmax's time.
                    f32x2 sum(0.f, 0.f);
                    uint32_t x[32];
                    tmem_issue32(s_col, x);
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        tmem_await32(x);
                        if (!every) {
                            const uint32_t seen = (c ? in.y : in.x) & tree_bits(mrow, a.mask_words32, p0 + 32 * c - pre);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((seen >> k) & 1u)) x[k] = __float_as_uint(unseen);
                        }
                        // the largest x * sl2: the largest x, or the smallest under a negative scale
                        float top[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) top[k] = __uint_as_float(x[k]);
                        if (sl2 >= 0.f) {
#pragma unroll
                            for (int k = 4; k < 28; k += 8)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    top[i] = max3(top[i], __uint_as_float(x[k + i]), __uint_as_float(x[k + 4 + i]));
#pragma unroll
                            for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], __uint_as_float(x[28 + i]));
                            top[0] = fmaxf(max3(top[0], top[1], top[2]), top[3]);
                        } else {
#pragma unroll
                            for (int k = 4; k < 32; ++k) top[k & 3] = fminf(top[k & 3], __uint_as_float(x[k]));
                            top[0] = fminf(fminf(top[0], top[1]), fminf(top[2], top[3]));
                        }
                        const float mx = top[0] * sl2;
                        const bool up = mx > m + RESCALE_THRESHOLD;
                        if (__any_sync(FULL_MASK, up)) {
                            const float alpha = up ? exp2_approx(m - mx) : 1.f;
                            if (up) m = mx;
                            l *= alpha;
                            sum = fma2(sum, f32x2(alpha, alpha), f32x2(0.f, 0.f));
                            // O may be scaled only when none of this stream's P.V runs
                            ok &= tt_rescale<D>(o_col, s_col, alpha, c, step > 0, &sh.o_done[w][(use - 1) & 1u],
                                                ((use - 1) >> 1) & 1u, abort_flag, a.dev_err);
                        }
                        // weights over S: 16 columns of hi = bf16(p), then 16 of lo = bf16(p - hi)
                        const float base = m == NEG_INF ? 0.f : m;
                        const f32x2 mul(sl2, sl2), sub(-base, -base), minus(-1.f, -1.f);
                        uint32_t pw[32];
                        f32x2 part[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float p, q;
                            fma2(f32x2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), mul, sub).get(p, q);
                            p = exp2_approx(p);
                            q = exp2_approx(q);
                            const f32x2 pq(p, q);
                            part[k & 1] = add2(part[k & 1], pq);
                            pw[k] = pack_bf16(p, q);
                            fma2(f32x2(bf16_lo(pw[k]), bf16_hi(pw[k])), minus, pq).get(p, q);
                            pw[16 + k] = pack_bf16(p, q);
                        }
                        sum = add2(sum, add2(part[0], part[1]));
                        if (c == 0) tmem_issue32(s_col + 32, x);
                        tmem_issue_store32(s_col + 32 * c, pw);
                    }
                    tmem_await_stores();
                    float s0, s1;
                    sum.get(s0, s1);
                    l += s0 + s1;
                    if (step > 0 && step % TT_FOLD == 0) ok &= fold(step == TT_FOLD, false);
                }
                tmem_fence_before_sync();
                mbar_arrive(smem_u32(&sh.p_full[w][use & 1u]));
            }
            // the run's last P.V of this stream
            if (ok) ok = tt_wait(&sh.o_done[w][(use - 1) & 1u], ((use - 1) >> 1) & 1u, abort_flag, a.dev_err);
            tmem_fence_after_sync();
            if (steps > TT_FOLD && busy && __all_sync(FULL_MASK, ok)) ok = fold(false, true);

            // epilogue.  Two row tiles: every stream stores its own rows.  One:
            // both streams hold a part of the same rows; each stores half of the
            // columns of both parts together.
            float M = m, L = l, c0 = 1.f, c1 = 0.f;
            if (!two) {
                float2* ml = reinterpret_cast<float2*>(smem + Geo::Q_TILE);   // the row tile that is not in use
                ml[w * TT_M + row] = make_float2(m, l);
                tmem_fence_before_sync();
                named_barrier_sync(TT_ML_BARRIER, TT_SOFTMAX);
                tmem_fence_after_sync();
                const float2 x0 = ml[row], x1 = ml[TT_M + row];
                // read by all before a warp without rows, which has no epilogue, writes the
                // next run's Q there
                named_barrier_sync(TT_ML_BARRIER, TT_SOFTMAX);
                M = fmaxf(x0.x, x1.x);
                c0 = M == NEG_INF ? 0.f : exp2_approx(x0.x - M);
                c1 = M == NEG_INF ? 0.f : exp2_approx(x1.x - M);
                L = c0 * x0.y + c1 * x1.y;
            }
            const bool go = __all_sync(FULL_MASK, ok && !*abort_flag);
            if (go && busy) {
                const bool whole = r.t0 == 0 && r.t1 == r.nt;
                const int slot = 2 * blockIdx.x + (r.starts ? 0 : 1);
                const int col0 = two ? 0 : w * (D / 2), cols = two ? D : D / 2;
                const uint32_t first = lanes + Geo::O_COL + (two ? D * w : 0);
                const float inv = whole ? (L > 0.f ? 1.f / L : 0.f) : 1.f;
                // a row that has seen nothing: its O is zero whatever the buffer holds
                const float f0 = c0 * inv, f1 = c1 * inv;
                const size_t at = valid ? tree_out_row(a, r.first, r.kvh, r.row0 + R) * D : 0;
                float4* acc = reinterpret_cast<float4*>(tree_part(a, slot, D)) + R;
                if (*const_cast<volatile int*>(&sh.odd_run) == run)   // to the stream that counts more
                    tt_add_odd<D>(a.v_cache, a.num_blocks, a.num_kv_heads, a.log2_block, first + (!two && c1 > c0 ? D : 0),
                                  col0, cols, a.block_tables + static_cast<size_t>(r.s) * a.max_blocks, r.kvh, mrow,
                                  a.mask_words32, pre,
                                  max(max(0, pre), r.t0 * TT_KT), min(r.ctx, r.t1 * TT_KT), valid);
#pragma unroll 1
                for (int c = col0; c < col0 + cols; c += 32) {
                    float o[32];
                    tmem_load32(first + c, o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] *= f0;
                    if (!two) {
                        float o1[32];
                        tmem_load32(first + D + c, o1);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = fmaf(o1[k], f1, o[k]);
                    }
                    if (valid && !whole) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            acc[(c / 4 + k) * a.part_rows] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    } else if (valid && a.out_f32) {
                        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + c);
#pragma unroll
                        for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    } else if (valid) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at + c);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            dst[k] = make_uint4(pack_bf16(o[8 * k], o[8 * k + 1]), pack_bf16(o[8 * k + 2], o[8 * k + 3]),
                                                pack_bf16(o[8 * k + 4], o[8 * k + 5]), pack_bf16(o[8 * k + 6], o[8 * k + 7]));
                    }
                    __syncwarp();
                }
                if (valid && !whole && (two || w == 0)) a.part_ml[static_cast<size_t>(slot) * a.part_rows + R] = make_float2(M, L);
            }
            ring += 2 * nt;
            tiles += nt;
        }
    }

    __syncwarp();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    if (warp == 0) tmem_free(tmem, TT_TMEM_COLS);
}

template <int D>
int launch(const TreeArgs& a, int ctas, cudaStream_t st) {
    static KernelSlot slot;
    CUtensorMap tk, tv;
    auto encode = [&](CUtensorMap* m, const void* pool) {
        return a.block_size < 8 ? encode_half_group_map(m, pool, a.num_blocks, a.num_kv_heads, D)
                                : encode_block_map(m, pool, a.num_blocks, a.num_kv_heads, a.block_size, D);
    };
    if (!encode(&tk, a.k_cache) || !encode(&tv, a.v_cache)) return PA_ERR_CUDA;
    const int smem = TreeGeom<D>::BYTES + 1024;
    auto kern = tree_tc_kernel<D>;
    if (prepare_kernel(slot, reinterpret_cast<const void*>(kern), TT_THREADS, smem) <= 0) return PA_ERR_CUDA;
    return launch_status(launch_pdl(kern, dim3(ctas), dim3(TT_THREADS), smem, st, tk, tv, a));
}

}  // namespace

bool tree_tc_eligible(pa_dtype dtype, int block_size) {
    return dtype == PA_BF16 && (block_size == 4 || block_size == 8 || block_size == 16 || block_size == 32);
}

int tree_tc_rows() { return TT_ROWS; }

int launch_tree_tc(const TreeArgs& a, int head_dim, int ctas, cudaStream_t st) {
    return head_dim == 128 ? launch<128>(a, ctas, st) : launch<64>(a, ctas, st);
}

}  // namespace pa
