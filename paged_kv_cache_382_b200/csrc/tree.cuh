// tree.cuh -- attention of drafted tokens over a paged cache (pa_tree_decode):
// what its two attend kernels share (tree_decode.cu on the CUDA cores, fp32 pools;
// tree_tc.cu on the tensor cores, bf16 pools).
//
// What is computed: new token ("node") i of sequence s, one of n_s, sees every
// position below context_len - n_s (the prefix) and the nodes its mask names:
//   out = softmax(scale * q . K[seen]^T) . V[seen].
//
// Work line.  A unit is one row block of one (sequence, kv head): up to ROWS
// query rows (row r = node r / g, head r % g of the group), all of which read
// the same K/V.  It takes ceil(context / KT) K/V tiles, at least one, and a tile
// costs one step per HALF rows (a kernel that works through ROWS = 2 HALF rows
// needs twice the time for more than HALF of them); starting and finishing a unit
// costs another TREE_UNIT_STEPS, behind its tiles.  The units' steps in a row
// (sequence, kv head, row block) form a line of W steps that the CTAs cut into
// equal shares: CTA c of G takes the tiles whose first step lies in [c W / G,
// (c + 1) W / G).  Ragged contexts and drafts need no other balancing, few rows
// over a long context are split as finely as there are SMs, and a CTA leaves at
// most two units unfinished: a partial (max, sum, unnormalised output) for its
// first run and one for its last, whatever the batch.  A second kernel joins
// each cut unit's partials in CTA order.  The cuts depend on the whole batch, so a
// row's rounding may differ in another batch; a batch gives the same bits every
// time.
#pragma once

#include "pa_device.cuh"
#include "pa_host.h"

namespace pa {

// The run a CTA's share starts with, for the join (none: t0 = 0, begin = -1).
struct TreeRecord {
    int begin;                   // the unit's first step on the line
    int first, kvh, row0, rows;  // its rows (see TreeRun)
    int t0, nt, per_tile;        // the run's first tile, the unit's tiles, steps per tile
};

struct TreeArgs {
    void* out;
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_start;
    const uint32_t* tree_mask;   // [num_tokens][mask_words32]
    int32_t* dev_err;
    TreeRecord* recs;            // [CTA]: the unit each CTA's share starts in
    int* line;                   // W
    float* part_acc;             // [2 * CTA][head_dim / 4][part_rows][4]
    float2* part_ml;             // [2 * CTA][part_rows]
    int part_rows;               // rows a partial has room for
    int mask_words32;            // 32-bit words per mask row
    int num_seqs, num_tokens, num_heads, num_kv_heads, group;
    int block_size, log2_block, num_blocks, max_blocks, cap;
    float scale_log2;
    int out_f32;
};

// CTAs a launch may have (and partial pairs the workspace holds): one per SM on the
// tensor cores, two on the CUDA cores.
constexpr int TREE_TC_CTAS = 160, TREE_SIMT_CTAS = 2 * TREE_TC_CTAS, TREE_CTAS_MAX = TREE_SIMT_CTAS;
// Sequences are found in windows of 32; the windows' sums sit in shared memory.
constexpr int TREE_WINDOWS_MAX = 4096;
// What a unit costs besides its tiles (the host bounds W by INT_MAX).
constexpr int TREE_UNIT_STEPS = 2;

// One sequence as the work line sees it; a malformed one (rows outside q) has none.
struct TreeSeq {
    int first, n, ctx;   // first row of q, nodes, context
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int s, bool report) {
    TreeSeq t{0, 0, 0};
    if (s >= a.num_seqs) return t;
    const int q0 = a.query_start[s], q1 = a.query_start[s + 1], raw = a.context_lens[s];
    t.ctx = clamp_context(raw, a.cap);
    if (q0 < 0 || q1 < q0 || q1 > a.num_tokens) {
        if (report) flag_error(a.dev_err, PA_DEVERR_CONTEXT);
        return t;
    }
    t.first = q0;
    t.n = q1 - q0;
    if (report && (raw != t.ctx || t.n > t.ctx || t.n > 32 * a.mask_words32)) flag_error(a.dev_err, PA_DEVERR_CONTEXT);
    return t;
}

template <int KT>
__device__ __forceinline__ int tree_tiles(int ctx) {
    return ctx > 0 ? (ctx - 1) / KT + 1 : 1;   // an empty context still writes its zero rows
}

// Row blocks of a sequence and kv head, in halves of HALF rows; all blocks but the
// last have HALVES of them.
template <int HALF>
__device__ __forceinline__ int tree_halves(const TreeArgs& a, int n) {
    return (n * a.group + HALF - 1) / HALF;
}
// Steps of one kv head's units.
template <int HALF, int HALVES, int KT>
__device__ __forceinline__ int tree_head_steps(const TreeArgs& a, const TreeSeq& t) {
    const int halves = tree_halves<HALF>(a, t.n);
    return halves * tree_tiles<KT>(t.ctx) + (halves + HALVES - 1) / HALVES * TREE_UNIT_STEPS;
}

// A run of one unit's tiles.
struct TreeRun {
    int s, first, n, ctx;   // the sequence
    int kvh, row0, rows;    // kv head; the unit's first row and rows within (node, head) rows
    int t0, t1, nt;         // tiles [t0, t1) of the unit's nt
    int per_tile;           // steps per tile (1 or 2)
    int begin;              // the unit's first step on the line
    bool starts;            // the CTA's first run
};

// Walks the runs of one CTA; every warp that needs them keeps its own walker
// (lane l holds the window's l-th sequence).
template <int HALF, int HALVES, int KT>
struct TreeWalker {
    static_assert(HALVES == 1 || HALVES == 2, "steps per tile");
    int w, w_end;           // position on the line, the end of the CTA's share
    int seq0;               // the window's first sequence
    bool started;           // a run was given out
    TreeSeq mine;
    int start, cost;        // the lane's sequence on the line

    __device__ __forceinline__ void load(const TreeArgs& a, int first_seq, int at) {
        const int lane = threadIdx.x & 31;
        seq0 = first_seq;
        mine = tree_seq(a, seq0 + lane, false);
        cost = tree_head_steps<HALF, HALVES, KT>(a, mine) * a.num_kv_heads;
        start = at + warp_inclusive_scan(cost) - cost;
    }

    // The next run, or false at the end of the CTA's share.  Called by all lanes.
    __device__ __forceinline__ bool next(const TreeArgs& a, TreeRun& r) {
        while (w < w_end) {
            unsigned past;
            while ((past = __ballot_sync(FULL_MASK, w < start + cost)) == 0u) {
                if (seq0 + 32 >= a.num_seqs) return false;   // lengths changed under the launch
                load(a, seq0 + 32, __shfl_sync(FULL_MASK, start + cost, 31));
            }
            const int l = __ffs(past) - 1;
            r.s = seq0 + l;
            r.first = __shfl_sync(FULL_MASK, mine.first, l);
            r.n = __shfl_sync(FULL_MASK, mine.n, l);
            r.ctx = __shfl_sync(FULL_MASK, mine.ctx, l);
            r.nt = tree_tiles<KT>(r.ctx);
            unsigned off = w - __shfl_sync(FULL_MASK, start, l);
            const unsigned seq_steps = __shfl_sync(FULL_MASK, cost, l);
            // overlapping ranges of a malformed query_start can overflow the line:
            // nothing outside a sequence's own steps is ever a run
            if (off >= seq_steps) return false;
            const unsigned head_steps = seq_steps / a.num_kv_heads;
            r.kvh = off / head_steps;
            off -= r.kvh * head_steps;
            const unsigned block_steps = HALVES * r.nt + TREE_UNIT_STEPS;
            const int block = off / block_steps;
            off -= block * block_steps;
            r.per_tile = min(HALVES, tree_halves<HALF>(a, r.n) - HALVES * block);
            r.row0 = block * HALF * HALVES;
            r.rows = min(HALF * HALVES, r.n * a.group - r.row0);
            r.begin = w - off;
            // tiles whose first step is in the share
            const int unit_steps = r.per_tile * r.nt + TREE_UNIT_STEPS;
            const int end = min(unit_steps, w_end - r.begin);
            r.t0 = min(r.nt, (static_cast<int>(off) + r.per_tile - 1) / r.per_tile);
            r.t1 = min(r.nt, (end + r.per_tile - 1) / r.per_tile);
            if (r.begin + end <= w) return false;
            w = r.begin + end;
            if (r.t0 >= r.t1) continue;   // the share holds no tile's first step of this unit
            r.starts = !started;
            started = true;
            return true;
        }
        return false;
    }
};

// CTAs that share a line of W steps, and the first step of CTA c's share.
__device__ __forceinline__ int tree_sharers(int W, int ctas) { return W / 2 < ctas ? (W > 1 ? W / 2 : 1) : ctas; }
__device__ __forceinline__ int tree_share(int W, int sharers, int c) {
    return c >= sharers ? W : W / sharers * c + W % sharers * c / sharers;
}

// Line length and the CTA's walker.  Called by the whole CTA; `sums` (shared
// memory, a word per window of 32 sequences) is free again after the caller's
// next barrier.  CTA 0 reports malformed sequences and keeps the length for the
// join.
template <int HALF, int HALVES, int KT>
__device__ __forceinline__ void tree_begin(const TreeArgs& a, int* sums, TreeWalker<HALF, HALVES, KT>& walk) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    const int windows = (a.num_seqs + 31) / 32;
    for (int v = warp; v < windows; v += nwarps) {
        int c = tree_head_steps<HALF, HALVES, KT>(a, tree_seq(a, 32 * v + lane, blockIdx.x == 0)) * a.num_kv_heads;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(FULL_MASK, c, o);
        if (lane == 0) sums[v] = c;
    }
    __syncthreads();
    int total = 0;
    for (int v = lane; v < windows; v += 32) total += sums[v];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(FULL_MASK, total, o);
    const int sharers = tree_sharers(total, gridDim.x);
    walk.w = tree_share(total, sharers, blockIdx.x);
    walk.w_end = tree_share(total, sharers, blockIdx.x + 1);
    walk.started = false;
    // the window that holds the first step of the share
    int at = 0, v = 0;
    while (v + 1 < windows && at + sums[v] <= walk.w) at += sums[v++];
    walk.load(a, 32 * v, at);
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) *a.line = total;
        a.recs[blockIdx.x] = TreeRecord{-1, 0, 0, 0, 0, 0, 0, 1};
    }
}

// Called after the barrier that follows tree_begin, by one thread.
__device__ __forceinline__ void tree_record(const TreeArgs& a, const TreeRun& r) {
    a.recs[blockIdx.x] = TreeRecord{r.begin, r.first, r.kvh, r.row0, r.rows, r.t0, r.nt, r.per_tile};
}

__device__ __forceinline__ float* tree_part(const TreeArgs& a, int slot, int D) {
    return a.part_acc + static_cast<size_t>(slot) * a.part_rows * D;
}

// Row of q / out ([num_tokens][num_heads] rows) of row R of a sequence's (node, head) rows.
__device__ __forceinline__ size_t tree_out_row(const TreeArgs& a, int first, int kvh, int R) {
    const int node = R / a.group;
    return static_cast<size_t>(first + node) * a.num_heads + kvh * a.group + (R - node * a.group);
}

// Bits k of the result: node `from` + k of the row's mask; nodes before 0 (the
// prefix) are seen, nodes past the words are not.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* row, int words, int from) {
    if (from <= -32) return 0xffffffffu;
    if (from < 0) return (words > 0 ? row[0] << -from : 0u) | ((1u << -from) - 1u);
    const int i = from >> 5;
    const uint32_t lo = i < words ? row[i] : 0u, hi = i + 1 < words ? row[i + 1] : 0u;
    return __funnelshift_r(lo, hi, from & 31);
}

// Attend on the tensor cores (tree_tc.cu): bf16 pools, head_dim 64 or 128,
// blocks of 4, 8, 16 or 32 tokens, any group.
bool tree_tc_eligible(pa_dtype dtype, int block_size);
int tree_tc_rows();
int launch_tree_tc(const TreeArgs& a, int head_dim, int ctas, cudaStream_t st);

}  // namespace pa
