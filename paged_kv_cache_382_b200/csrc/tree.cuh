// tree.cuh -- attention of drafted tokens over a paged cache (pa_tree_decode):
// what its two attend kernels share (tree_decode.cu on the CUDA cores, any pool;
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
// needs twice the time for more than HALF of them).  The units' steps in a row
// (sequence, kv head, row block) form a line of W steps that the CTAs cut into
// equal shares: CTA c of G takes the tiles whose first step lies in [c W / G,
// (c + 1) W / G).  Ragged contexts and drafts need no other balancing, few rows
// over a long context are split as finely as there are SMs, and a CTA leaves at
// most two units unfinished: a partial (max, sum, unnormalised output) for its
// first run and one for its last, whatever the batch.  A second kernel joins
// each cut unit's partials in CTA order.  Shares have at least two steps, so that
// each holds the start of a tile.  The cuts depend on the whole batch, so a row's
// rounding may differ in another batch; a batch gives the same bits every time.
#pragma once

#include "pa_device.cuh"
#include "pa_host.h"

namespace pa {

// The run a CTA's share starts with, for the join.
struct TreeRecord {
    long long begin;             // the unit's first step on the line
    int first, kvh, row0, rows;  // its rows (see TreeRun)
    int t0, nt, per_tile;        // the run's first tile, the unit's tiles, steps per tile
    int pad;
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
    long long* line;             // W
    float* part_acc;             // [2 * CTA][head_dim / 4][part_rows][4]
    float2* part_ml;             // [2 * CTA][part_rows]
    int part_rows;               // rows a partial has room for
    int mask_words32;            // 32-bit words per mask row
    int num_seqs, num_tokens, num_heads, num_kv_heads, group;
    int block_size, log2_block, num_blocks, max_blocks, cap;
    float scale_log2;
    int out_f32;
};

// CTAs a launch may have (and partial pairs the workspace holds).
constexpr int TREE_CTAS_MAX = 160;
// Sequences are found in windows of 32; the windows' sums sit in shared memory.
constexpr int TREE_WINDOWS_MAX = 4096;

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

// Steps of a sequence's units, and of one kv head's: row blocks of two halves,
// the last one of one half when that holds its rows.
template <int HALF>
__device__ __forceinline__ int tree_halves(const TreeArgs& a, int n) {
    return (n * a.group + HALF - 1) / HALF;
}
template <int HALF, int KT>
__device__ __forceinline__ long long tree_cost(const TreeArgs& a, const TreeSeq& t) {
    return static_cast<long long>(tree_halves<HALF>(a, t.n)) * a.num_kv_heads * tree_tiles<KT>(t.ctx);
}

// A run of one unit's tiles.
struct TreeRun {
    int s, first, n, ctx;   // the sequence
    int kvh, row0, rows;    // kv head; the unit's first row and rows within (node, head) rows
    int t0, t1, nt;         // tiles [t0, t1) of the unit's nt
    int per_tile;           // steps per tile (1 or 2)
    long long begin;        // the unit's first step on the line
    bool starts;            // the CTA's first run
};

// Walks the runs of one CTA; every warp that needs them keeps its own walker
// (lane l holds the window's l-th sequence).
template <int HALF, int HALVES, int KT>
struct TreeWalker {
    static_assert(HALVES == 1 || HALVES == 2, "steps per tile");
    long long w, w_end;     // position on the line, the end of the CTA's share
    int seq0;               // the window's first sequence
    bool started;           // a run was given out
    TreeSeq mine;
    long long start, cost;  // the lane's sequence on the line

    __device__ __forceinline__ void load(const TreeArgs& a, int first_seq, long long at) {
        const int lane = threadIdx.x & 31;
        seq0 = first_seq;
        mine = tree_seq(a, seq0 + lane, false);
        cost = tree_cost<HALF, KT>(a, mine);
        long long inc = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(FULL_MASK, inc, o);
            if (lane >= o) inc += v;
        }
        start = at + inc - cost;
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
            const long long seq_start = __shfl_sync(FULL_MASK, start, l);
            r.nt = tree_tiles<KT>(r.ctx);
            // kv head, then row block: all of HALVES steps per tile but the last
            const int halves = tree_halves<HALF>(a, r.n);
            const long long head_steps = static_cast<long long>(halves) * r.nt;
            long long off = w - seq_start;
            r.kvh = static_cast<int>(off / head_steps);
            off -= r.kvh * head_steps;
            const long long block_steps = static_cast<long long>(HALVES) * r.nt;
            const int block = static_cast<int>(off / block_steps);
            off -= block * block_steps;
            r.per_tile = min(HALVES, halves - HALVES * block);
            r.row0 = block * HALF * HALVES;
            r.rows = min(HALF * HALVES, r.n * a.group - r.row0);
            r.begin = w - off;
            // tiles whose first step is in the share
            const long long unit_steps = static_cast<long long>(r.per_tile) * r.nt;
            const long long end = r.begin + unit_steps < w_end ? unit_steps : w_end - r.begin;
            r.t0 = static_cast<int>((off + r.per_tile - 1) / r.per_tile);
            r.t1 = static_cast<int>((end + r.per_tile - 1) / r.per_tile);
            w = r.begin + end;
            if (r.t0 >= r.t1) continue;   // only the second step of a tile whose first is another CTA's
            r.starts = !started;
            started = true;
            return true;
        }
        return false;
    }
};

// CTAs that share a line of W steps, and the first step of CTA c's share.
__device__ __forceinline__ int tree_sharers(long long W, int ctas) {
    return W / 2 < ctas ? (W > 1 ? static_cast<int>(W / 2) : 1) : ctas;
}
__device__ __forceinline__ long long tree_share(long long W, int sharers, int c) {
    return c >= sharers ? W : W / sharers * c + (W % sharers) * c / sharers;
}

// Line length and the CTA's walker.  Called by the whole CTA; `sums` (shared
// memory, a word per window of 32 sequences) is free again after the caller's
// next barrier.  CTA 0 reports malformed sequences and keeps the length for the
// join.
template <int HALF, int HALVES, int KT>
__device__ __forceinline__ void tree_begin(const TreeArgs& a, long long* sums, TreeWalker<HALF, HALVES, KT>& walk) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    const int windows = (a.num_seqs + 31) / 32;
    for (int v = warp; v < windows; v += nwarps) {
        long long c = tree_cost<HALF, KT>(a, tree_seq(a, 32 * v + lane, blockIdx.x == 0));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(FULL_MASK, c, o);
        if (lane == 0) sums[v] = c;
    }
    __syncthreads();
    long long total = 0;
    for (int v = lane; v < windows; v += 32) total += sums[v];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(FULL_MASK, total, o);
    const int sharers = tree_sharers(total, gridDim.x);
    walk.w = tree_share(total, sharers, blockIdx.x);
    walk.w_end = tree_share(total, sharers, blockIdx.x + 1);
    walk.started = false;
    // the window that holds the first step of the share
    long long at = 0;
    int v = 0;
    while (v + 1 < windows && at + sums[v] <= walk.w) at += sums[v++];
    walk.load(a, 32 * v, at);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.line = total;
}

__device__ __forceinline__ void tree_record(const TreeArgs& a, const TreeRun& r) {
    a.recs[blockIdx.x] = TreeRecord{r.begin, r.first, r.kvh, r.row0, r.rows, r.t0, r.nt, r.per_tile, 0};
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
// blocks of 8, 16 or 32 tokens, any group.
bool tree_tc_eligible(pa_dtype dtype, int block_size);
int tree_tc_rows();
int launch_tree_tc(const TreeArgs& a, int head_dim, int ctas, cudaStream_t st);

}  // namespace pa
