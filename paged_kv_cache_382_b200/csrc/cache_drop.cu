// cache_drop.cu -- dropping tokens from a paged KV cache:
//   pa_select_tokens: which tokens of each sequence and kv head to keep, from
//     running totals of their attention weights (pa_decode_weights).
//   pa_compact: moves the kept tokens' K, V and totals to consecutive
//     positions, in place or into other blocks.  Also moves up the accepted
//     path of a verified tree of drafted tokens (pa_tree_decode).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>

#include "pa_device.cuh"
#include "pa_host.h"

namespace cg = cooperative_groups;

namespace pa {

// ---------------------------------------------------------------------------
// select
//
// Row (s, h) holds n = context_lens[s] totals.  The last min(recent, budget)
// positions are kept; of the m others the k = budget - recent with the largest
// totals (ties: the lowest positions).  The k-th largest key is found by a
// radix descent (11 + 11 + 10 bits) over order-preserving integer keys, then
// one ordered pass writes the positions whose key is above it and the first
// ones equal to it.
//
// A row is split over a cluster of CTAs, each with a contiguous segment.  In a pass
// every CTA counts its segment's digits in shared memory and adds its counts to
// the leader's through distributed shared memory (adds return nothing, so nobody
// waits for them); the leader finds the digit and writes it to every CTA.  Reading
// all CTAs' counts from every CTA instead took most of a pass.  Keys that share the
// first digit with the sought one are few, as a rule: they go to the leader, which
// finds the other digits among them alone (a pass over the cluster costs 6000
// cycles, half of them barriers).  Only where they are too many for its list, as
// when most totals are equal, the cluster makes the other passes too.  A segment's
// keys are read once, all loads at the same time, and stay with their threads, in
// registers or, 32 to a thread, in shared memory (up to 131072 candidates to a row;
// longer rows are read again, from L2: that takes 74 us instead of 56 on 64 rows of
// 131072; 64 rows of 200000 take 114 us, 8 of them 41 us).
// ---------------------------------------------------------------------------

constexpr int SEL_THREADS = 512;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_BINS = 2048;
constexpr int SEL_PER = SEL_BINS / SEL_THREADS;   // bins per thread
constexpr int SEL_MAX_CLUSTER = 8;
constexpr int SEL_LIST = 6144;      // keys the leader's list holds
// Keys of a CTA that holds them: 4 Q of each thread.
constexpr int SEL_Q_SHORT = 2, SEL_Q_MIDDLE = 4, SEL_Q_LONG = 8;
constexpr int sel_keys(int q) { return 4 * q * SEL_THREADS; }

struct SelectArgs {
    int32_t* keep;
    int32_t* keep_lens;
    const float* weights;
    const int32_t* context_lens;
    const int32_t* budgets;
    int32_t* dev_err;
    int num_kv_heads, weights_stride, keep_stride, recent;
};

// Order-preserving integer of a total: larger totals, larger keys.  NaN counts
// as -inf, -0 as 0.
__device__ __forceinline__ uint32_t total_key(float w) {
    const float v = w != w ? NEG_INF : w + 0.f;
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Keys i .. i + 3 of a segment (i a multiple of 4); those past `len` are 0, the
// key of no total.
struct SegmentKeys {
    const float* w;
    int len;
    bool vec;          // w is 16-byte aligned
    __device__ __forceinline__ uint4 load(int i) const {
        if (vec && i + 4 <= len) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(w + i));
            return make_uint4(total_key(f.x), total_key(f.y), total_key(f.z), total_key(f.w));
        }
        uint32_t k[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = i + j < len ? total_key(__ldg(w + i + j)) : 0u;
        return make_uint4(k[0], k[1], k[2], k[3]);
    }
};

// Q > 0: the segment's keys are held, Q groups of four per thread (32 registers of
// them would leave one CTA per SM: those go to shared memory, 16 bytes a thread and
// group).  Q = 0: read again where they are needed.
template <int Q>
__global__ void __launch_bounds__(SEL_THREADS, 2) select_kernel(const SelectArgs a) {
    __shared__ uint32_t hist[2][SEL_BINS];   // by pass parity: one is cleared while the other is in use
    __shared__ int s_scan[33];
    __shared__ uint32_t s_found[3];          // the pass's digit, how many keys lie above it, how many have it
    __shared__ uint32_t s_list[SEL_LIST];    // the leader's: keys with the first digit
    __shared__ uint32_t s_listed;
    __shared__ int2 s_warp[SEL_WARPS];       // (above, equal) of each warp's sub-segment
    __shared__ int2 s_cta;                   // and of the segment, read by the cluster
    __shared__ int2 s_base;                  // and of the segments before it
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / CL;
    const int s = row / a.num_kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#pragma unroll
    for (int i = 0; i < 2 * SEL_PER; ++i) hist[i / SEL_PER][(i % SEL_PER) * SEL_THREADS + tid] = 0;
    if (tid == 0) s_listed = 0;
    auto sync_all = [&]() {
        if (CL > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    pdl_wait();
    pdl_launch_dependents();

    const int raw_n = a.context_lens[s], raw_b = a.budgets[s];
    const int n = clamp_context(raw_n, a.weights_stride);
    const int budget = clamp_context(raw_b, a.keep_stride);
    if (tid == 0 && row == s * a.num_kv_heads && rank == 0 && (n != raw_n || budget != raw_b))
        flag_error(a.dev_err, PA_DEVERR_CONTEXT);
    const int kept = min(n, budget);
    const int recent = min(a.recent, kept);
    const int m = n - recent, k = kept - recent;   // candidates, and how many of them stay
    int32_t* out = a.keep + static_cast<size_t>(row) * a.keep_stride;
    if (tid == 0 && row == s * a.num_kv_heads && rank == 0) a.keep_lens[s] = kept;

    // the latest positions, shared out over the cluster
    for (int i = rank * SEL_THREADS + tid; i < recent; i += CL * SEL_THREADS) out[k + i] = m + i;
    if (k == m || k == 0) {   // every candidate stays, or none (all CTAs of the row agree)
        for (int i = rank * SEL_THREADS + tid; i < k; i += CL * SEL_THREADS) out[i] = i;
        return;
    }

    const int seg = ((m + CL - 1) / CL + 31) & ~31;
    const int lo = min(m, rank * seg), len = min(m, lo + seg) - lo;
    SegmentKeys keys;
    keys.w = a.weights + static_cast<size_t>(row) * a.weights_stride + lo;
    keys.len = len;
    keys.vec = (reinterpret_cast<uintptr_t>(keys.w) & 15u) == 0;
    // warp w takes a contiguous part of the segment, a lane four keys at a time
    const int part = Q > 0 ? 128 * Q : ((len + SEL_WARPS - 1) / SEL_WARPS + 127) & ~127;
    const int w0 = min(len, warp * part), w1 = min(len, w0 + part);
    extern __shared__ __align__(16) uint4 s_held[];   // [Q][SEL_THREADS] for Q = SEL_Q_LONG
    constexpr bool IN_SHARED = Q == SEL_Q_LONG;
    uint4 held[Q > 0 && !IN_SHARED ? Q : 1];
    if constexpr (Q > 0) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const uint4 k4 = keys.load(w0 + 128 * q + 4 * lane);
            if constexpr (IN_SHARED)
                s_held[q * SEL_THREADS + tid] = k4;
            else
                held[q] = k4;
        }
    }
    // f(four keys, index of the first) for the lane's keys, in order
    auto each = [&](auto&& f) {
        if constexpr (IN_SHARED) {
#pragma unroll 2
            for (int q = 0; q < Q; ++q) f(s_held[q * SEL_THREADS + tid], w0 + 128 * q + 4 * lane);
        } else if constexpr (Q > 0) {
#pragma unroll
            for (int q = 0; q < Q; ++q) f(held[q], w0 + 128 * q + 4 * lane);
        } else {
#pragma unroll 2
            for (int i0 = w0; i0 < w1; i0 += 128) f(keys.load(i0 + 4 * lane), i0 + 4 * lane);
        }
    };
    sync_all();                // cleared counts (the leader's before anybody adds)

    uint32_t prefix = 0;       // digits found so far
    uint32_t want = k;         // rank of the sought key among those with the prefix
    int shift = 32;
    // counts the digits (of `bits` bits, above `shift`) of four keys that have the prefix
    auto count4 = [&](uint32_t* h, const uint4& k4, int i, int end, int pass, int hi_shift, uint32_t mask) {
        const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w};
        // neighbours with one digit (zeros above all) add once
        uint32_t at = 0, count = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = i + j < end && (pass == 0 || (kk[j] >> hi_shift) == prefix);
            if (!in) continue;
            const uint32_t d = (kk[j] >> shift) & mask;
            if (count != 0 && d != at) {
                atomicAdd(&h[at], count);
                count = 0;
            }
            at = d;
            ++count;
        }
        if (count != 0) atomicAdd(&h[at], count);
    };
    // the digit that holds the wanted rank, told to CTAs 0 .. tell - 1; whole CTA, counts complete
    auto find = [&](const uint32_t* h, int tell) {
        // thread t owns SEL_PER bins counted from the top
        uint32_t cnt[SEL_PER], sum = 0;
#pragma unroll
        for (int j = 0; j < SEL_PER; ++j) {
            cnt[j] = h[SEL_BINS - 1 - (tid * SEL_PER + j)];
            sum += cnt[j];
        }
        int total;
        uint32_t before = static_cast<uint32_t>(cta_exclusive_scan(static_cast<int>(sum), &total, s_scan));
#pragma unroll
        for (int j = 0; j < SEL_PER; ++j) {
            if (before < want && want <= before + cnt[j]) {   // exactly one thread and bin
                for (int c = 0; c < tell; ++c) {
                    uint32_t* to = cluster.map_shared_rank(s_found, c);
                    to[0] = SEL_BINS - 1 - (tid * SEL_PER + j);
                    to[1] = before;
                    to[2] = cnt[j];
                }
            }
            before += cnt[j];
        }
        __syncthreads();
    };
    bool done = false;
#pragma unroll 1
    for (int pass = 0; pass < 3 && !done; ++pass) {
        const int bits = pass < 2 ? 11 : 10;
        const int hi_shift = shift;
        shift -= bits;
        const uint32_t mask = (1u << bits) - 1u;
        uint32_t* h = hist[pass & 1];
        each([&](const uint4& k4, int i) { count4(h, k4, i, w1, pass, hi_shift, mask); });
        __syncthreads();
        if (CL > 1) {
            if (rank != 0) {
                uint32_t* lead = cluster.map_shared_rank(h, 0);
#pragma unroll
                for (int j = 0; j < SEL_PER; ++j) {
                    const uint32_t c = h[j * SEL_THREADS + tid];
                    if (c != 0) atomicAdd(lead + j * SEL_THREADS + tid, c);
                }
            }
            cluster.sync();    // the leader has every segment's counts
        }
        if (rank == 0) find(h, CL);
#pragma unroll
        for (int j = 0; j < SEL_PER; ++j) h[j * SEL_THREADS + tid] = 0;   // for the pass after the next
        sync_all();            // the digit is known
        prefix = (prefix << bits) | s_found[0];
        want -= s_found[1];
        if (pass > 0 || s_found[2] > SEL_LIST) continue;

        // few enough: the leader takes the keys with this digit and goes on alone
        done = true;
        int mine = 0;
        each([&](const uint4& k4, int i) {
            const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) mine += i + j < w1 && (kk[j] >> shift) == prefix;
        });
        const int upto = warp_inclusive_scan(mine);
        uint32_t at = 0;
        if (lane == 31 && upto > 0) at = atomicAdd(cluster.map_shared_rank(&s_listed, 0), static_cast<uint32_t>(upto));
        at = __shfl_sync(FULL_MASK, at, 31) + upto - mine;
        uint32_t* list = cluster.map_shared_rank(s_list, 0);
        each([&](const uint4& k4, int i) {
            const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < w1 && (kk[j] >> shift) == prefix) list[at++] = kk[j];
        });
        sync_all();            // the list is complete
        if (rank == 0) {
            const int n_list = static_cast<int>(s_listed);
#pragma unroll 1
            for (int p = 1; p < 3; ++p) {
                const int b = p < 2 ? 11 : 10, hi = shift;
                shift -= b;
                for (int i = tid; i < n_list; i += SEL_THREADS)
                    if ((s_list[i] >> hi) == prefix) atomicAdd(&hist[p & 1][(s_list[i] >> shift) & ((1u << b) - 1u)], 1u);
                __syncthreads();
                find(hist[p & 1], 1);
                prefix = (prefix << b) | s_found[0];
                want -= s_found[1];
                __syncthreads();   // s_found is written again
            }
            if (tid < CL) {
                uint32_t* to = cluster.map_shared_rank(s_found, tid);
                to[0] = prefix;
                to[1] = want;
            }
        }
        sync_all();
        prefix = s_found[0];
        want = s_found[1];
    }
    // want = how many of the keys equal to prefix stay, the first ones by position

    auto tell = [&](const uint4& k4, int i, int (&up)[4], int (&eq)[4]) {
        const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            up[j] = i + j < w1 && kk[j] > prefix;
            eq[j] = i + j < w1 && kk[j] == prefix;
        }
    };
    int above = 0, equal = 0;
    each([&](const uint4& k4, int i) {
        int up[4], eq[4];
        tell(k4, i, up, eq);
        above += up[0] + up[1] + up[2] + up[3];
        equal += eq[0] + eq[1] + eq[2] + eq[3];
    });
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        above += __shfl_xor_sync(FULL_MASK, above, off);
        equal += __shfl_xor_sync(FULL_MASK, equal, off);
    }
    if (lane == 0) s_warp[warp] = make_int2(above, equal);
    __syncthreads();
    if (warp == 0) {
        const int2 x = lane < SEL_WARPS ? s_warp[lane] : make_int2(0, 0);
        const int ix = warp_inclusive_scan(x.x), iy = warp_inclusive_scan(x.y);
        if (lane < SEL_WARPS) s_warp[lane] = make_int2(ix - x.x, iy - x.y);
        if (lane == 31) s_cta = make_int2(ix, iy);
    }
    sync_all();
    if (warp == 0) {
        int2 x = make_int2(0, 0);
        if (lane < rank) x = *cluster.map_shared_rank(&s_cta, lane);
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) {
            x.x += __shfl_xor_sync(FULL_MASK, x.x, off);
            x.y += __shfl_xor_sync(FULL_MASK, x.y, off);
        }
        if (lane == 0) s_base = x;
    }
    sync_all();       // and s_cta is no longer read by the cluster
    int base_above = s_warp[warp].x + s_base.x, base_equal = s_warp[warp].y + s_base.y;
    const int quota = static_cast<int>(want);
    each([&](const uint4& k4, int i) {
        int up[4], eq[4];
        tell(k4, i, up, eq);
        const int nu = up[0] + up[1] + up[2] + up[3], ne = eq[0] + eq[1] + eq[2] + eq[3];
        // both counts of a lane in one scan: at most 128 each
        const int inc = warp_inclusive_scan(nu | (ne << 16));
        int bu = base_above + (inc & 0xffff) - nu, be = base_equal + (inc >> 16) - ne;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (up[j] || (eq[j] && be < quota)) out[bu + min(be, quota)] = lo + i + j;
            bu += up[j];
            be += eq[j];
        }
        const int all = __shfl_sync(FULL_MASK, inc, 31);
        base_above += all & 0xffff;
        base_equal += all >> 16;
    });
}

// ---------------------------------------------------------------------------
// compact
//
// Destination position starts[s] + j of (s, h) receives position keep[s][h][j].
// Positions only move down (keep[j] >= starts + j, checked), so in place it is
// enough that, within one (s, h), chunk c of destinations is written after the
// sources of chunks 0 .. c were read: later chunks' sources lie above every
// destination of chunk c.  One CTA walks the chunks of one (s, h) in order,
// loads running ahead of the stores; other CTAs take the other pool, other 16-byte
// columns of the same rows, and the totals, which never meet.
//
// A thread finds the pool rows of one (source, destination) pair of a page of
// THREADS pairs, its position and table entries fetched one and two pages ahead;
// the threads that move a row's columns read the pair from shared memory.  Every
// column's thread finding the rows itself took 1.6 times as long (64 sequences of 128
// to 2048 tokens cut to a half, 32 kv heads: 306 against 194 us).
// With many walks that is bound by HBM.  With few (a CTA per SM or less) the round
// trips of a chunk would bound it: compact_few_kernel's CTAs have 1024 threads,
// find 8192 pairs at once and keep four chunks of rows in flight.  One sequence of 8
// kv heads, d 128, bf16, to a quarter: 32768 tokens 20 against 43 us, 4096 tokens 5.3
// against 6.4 us (in place 20 against 39).
// ---------------------------------------------------------------------------

constexpr int CMP_THREADS = 256, CMP_FEW_THREADS = 1024;
constexpr int CMP_FEW_PAIRS = 8, CMP_FEW_DEPTH = 4;   // pairs per thread and page, chunks in flight
constexpr int CMP_ROWS = 2;     // rows per thread and chunk
constexpr int CMP_TOTALS = 4;   // totals per thread and chunk

struct CompactArgs {
    uint4* k_cache;           // [NB][Hkv][B][d] as 16-byte vectors
    uint4* v_cache;
    float* w_out;
    const float* w_in;
    const int32_t* src_tables;
    const int32_t* dst_tables;
    const int32_t* keep;
    const int32_t* starts;
    const int32_t* keep_lens;
    int32_t* dev_err;
    int num_kv_heads, keep_heads, keep_stride, w_stride;
    int src_blocks, dst_blocks;   // table widths
    int num_blocks, block_size, log2_block, row_vecs;
    int log2_vecs;            // 16-byte columns per CTA: 1 << log2_vecs
    int slices;               // CTAs along a row: row_vecs >> log2_vecs
    int walks;                // CTAs per (s, h): 2 pools x slices, and one for the totals if there are any
};

// What a walk knows of its (s, h).
struct CompactRow {
    const int32_t* keep;
    const int32_t* src_table;
    const int32_t* dst_table;
    int n, start;
};

// Position keep[j], or -1 when it may not move (past the row's end: silently).
__device__ __forceinline__ int compact_source(const CompactArgs& a, const CompactRow& r, int j, int pos, bool report) {
    if (j >= r.n) return -1;
    const long long d = static_cast<long long>(r.start) + j;
    if (pos < d || pos >= (static_cast<long long>(a.src_blocks) << a.log2_block) ||
        d >= (static_cast<long long>(a.dst_blocks) << a.log2_block)) {
        if (report) flag_error(a.dev_err, PA_DEVERR_COPY);
        return -1;
    }
    return pos;
}

// blockIdx.x = (s * Hkv + h) * walks + walk: the CTA's (s, h); false if it has nothing to do.
__device__ __forceinline__ bool compact_begin(const CompactArgs& a, CompactRow& r, int& h, int& walk, int& row) {
    row = blockIdx.x / a.walks;
    walk = blockIdx.x - row * a.walks;
    const int s = row / a.num_kv_heads;
    h = row - s * a.num_kv_heads;
    const int raw = a.keep_lens[s];
    r.n = clamp_context(raw, a.keep_stride);
    r.start = a.starts != nullptr ? a.starts[s] : 0;
    if (walk == 0 && threadIdx.x == 0 && h == 0 && (raw != r.n || r.start < 0)) flag_error(a.dev_err, PA_DEVERR_CONTEXT);
    if (r.start < 0 || r.n == 0) return false;
    r.keep = a.keep + (static_cast<size_t>(s) * a.keep_heads + (a.keep_heads > 1 ? h : 0)) * a.keep_stride;
    r.src_table = a.src_tables + static_cast<size_t>(s) * a.src_blocks;
    r.dst_table = a.dst_tables + static_cast<size_t>(s) * a.dst_blocks;
    return true;
}

// The walk of one (s, h)'s totals: a thread per position.
__device__ __forceinline__ void compact_totals(const CompactArgs& a, const CompactRow& r, int row) {
    const float* in = a.w_in + static_cast<size_t>(row) * a.w_stride;
    float* out = a.w_out + static_cast<size_t>(row) * a.w_stride;
    const int chunk = blockDim.x * CMP_TOTALS;
    for (int j0 = 0; j0 < r.n; j0 += chunk) {
        float t[CMP_TOTALS];
        int at[CMP_TOTALS];
#pragma unroll
        for (int u = 0; u < CMP_TOTALS; ++u) {
            const int j = j0 + u * blockDim.x + threadIdx.x;
            const int pos = compact_source(a, r, j, j < r.n ? r.keep[j] : -1, false);
            at[u] = -1;
            if (pos < 0 || pos >= a.w_stride) continue;
            const int d = r.start + j, sb = r.src_table[pos >> a.log2_block], db = r.dst_table[d >> a.log2_block];
            if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) continue;   // its K and V stay, too
            t[u] = __ldcg(in + pos);
            at[u] = d;
        }
        __syncthreads();      // every thread has read its sources of the chunk
#pragma unroll
        for (int u = 0; u < CMP_TOTALS; ++u)
            if (at[u] >= 0) __stcg(out + at[u], t[u]);
    }
}

// Pool rows (source, destination) of pair j, from its source position's offset in
// the block (-1: none) and its table entries; source -1 if nothing moves.  Rows of a
// pool fit 31 bits.
__device__ __forceinline__ int2 compact_pair(const CompactArgs& a, const CompactRow& r, int h, int j, int off, int sb,
                                             int db, bool report) {
    if (off < 0) return make_int2(-1, 0);
    if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
        if (report) flag_error(a.dev_err, PA_DEVERR_BLOCK_ID);
        return make_int2(-1, 0);
    }
    const int from = (sb * a.num_kv_heads + h) * a.block_size + off;
    const int dest = (db * a.num_kv_heads + h) * a.block_size + ((r.start + j) & (a.block_size - 1));
    return make_int2(from == dest ? -1 : from, dest);
}

__global__ void __launch_bounds__(CMP_FEW_THREADS, 1) compact_few_kernel(const CompactArgs a) {
    constexpr int T = CMP_FEW_THREADS, PAGE = T * CMP_FEW_PAIRS, DEPTH = CMP_FEW_DEPTH;
    extern __shared__ int2 s_page[];   // [PAGE]
    pdl_wait();
    pdl_launch_dependents();
    CompactRow r;
    int h, walk, row;
    if (!compact_begin(a, r, h, walk, row)) return;
    if (walk == 2 * a.slices) {
        compact_totals(a, r, row);
        return;
    }
    const bool lead = walk == 0;
    const int vecs = 1 << a.log2_vecs, r0 = threadIdx.x >> a.log2_vecs, rows_per = T >> a.log2_vecs;
    uint4* pool = ((walk & 1) ? a.v_cache : a.k_cache) + (walk >> 1) * vecs + (threadIdx.x & (vecs - 1));
    for (int j0 = 0; j0 < r.n; j0 += PAGE) {
        int off[CMP_FEW_PAIRS], sb[CMP_FEW_PAIRS], db[CMP_FEW_PAIRS];
#pragma unroll
        for (int u = 0; u < CMP_FEW_PAIRS; ++u) {
            const int j = j0 + u * T + threadIdx.x;
            off[u] = j < r.n ? r.keep[j] : -1;
        }
#pragma unroll
        for (int u = 0; u < CMP_FEW_PAIRS; ++u) {
            const int j = j0 + u * T + threadIdx.x;
            const int p = compact_source(a, r, j, off[u], lead);
            off[u] = p < 0 ? -1 : p & (a.block_size - 1);
            if (p < 0) continue;
            sb[u] = r.src_table[p >> a.log2_block];
            db[u] = r.dst_table[(r.start + j) >> a.log2_block];
        }
        __syncthreads();   // the last page's pairs are no longer read
#pragma unroll
        for (int u = 0; u < CMP_FEW_PAIRS; ++u)
            s_page[u * T + threadIdx.x] = compact_pair(a, r, h, j0 + u * T + threadIdx.x, off[u], sb[u], db[u], lead);
        __syncthreads();
        // chunk c: the page's pairs [c * rows_per, ...), a thread's row r0 of each
        const int chunks = (min(PAGE, r.n - j0) + rows_per - 1) / rows_per;
        uint4 v[DEPTH];
        int to[DEPTH];
        auto load = [&](int c, uint4& vv, int& tt) {
            tt = -1;
            if (c >= chunks) return;
            const int2 pair = s_page[c * rows_per + r0];
            if (pair.x < 0) return;
            tt = pair.y;
            vv = __ldcg(pool + static_cast<size_t>(pair.x) * a.row_vecs);
        };
#pragma unroll
        for (int u = 0; u < DEPTH - 1; ++u) load(u, v[u], to[u]);
        for (int c0 = 0; c0 < chunks; c0 += DEPTH) {
#pragma unroll
            for (int u = 0; u < DEPTH; ++u) {
                load(c0 + u + DEPTH - 1, v[(u + DEPTH - 1) % DEPTH], to[(u + DEPTH - 1) % DEPTH]);
                __syncthreads();   // every thread has read its source of chunk c0 + u
                if (to[u] >= 0) __stcg(pool + static_cast<size_t>(to[u]) * a.row_vecs, v[u]);
            }
        }
    }
}

__global__ void __launch_bounds__(CMP_THREADS, 6) compact_kernel(const CompactArgs a) {
    constexpr int THREADS = CMP_THREADS;
    pdl_wait();
    pdl_launch_dependents();
    CompactRow r;
    int h, walk, row;
    if (!compact_begin(a, r, h, walk, row)) return;
    if (walk == 2 * a.slices) {
        compact_totals(a, r, row);
        return;
    }
    const int slice = walk >> 1;
    const bool lead = walk == 0;  // reports what it skips
    const int vecs = 1 << a.log2_vecs;
    const int r0 = threadIdx.x >> a.log2_vecs;
    const int rows_per = THREADS >> a.log2_vecs, chunk = rows_per * CMP_ROWS;
    const int per_page = vecs / CMP_ROWS;   // chunks of a page of THREADS pairs
    uint4* pool = ((walk & 1) ? a.v_cache : a.k_cache) + slice * vecs + (threadIdx.x & (vecs - 1));
    const int nchunks = (r.n + chunk - 1) / chunk;
    __shared__ int2 s_pair[2][THREADS];     // (source row, destination row) of the pool, source -1: nothing to move

    // the thread's pair of a page: position and table entries under way
    int pos, off = -1, sb = 0, db = 0;
    auto load_pos = [&](int page) {
        const int j = page * THREADS + threadIdx.x;
        pos = j < r.n ? r.keep[j] : -1;
    };
    auto load_entries = [&](int page) {
        const int j = page * THREADS + threadIdx.x;
        const int p = compact_source(a, r, j, pos, lead);
        off = p < 0 ? -1 : p & (a.block_size - 1);
        if (p < 0) return;
        sb = r.src_table[p >> a.log2_block];
        db = r.dst_table[(r.start + j) >> a.log2_block];
    };
    auto write_pair = [&](int page) {
        s_pair[page & 1][threadIdx.x] = compact_pair(a, r, h, page * THREADS + threadIdx.x, off, sb, db, lead);
    };

    uint4 v[CMP_ROWS];
    int to[CMP_ROWS];
    auto load_rows = [&](int c) {
        const int2* pairs = s_pair[(c / per_page) & 1] + c % per_page * chunk + r0;
#pragma unroll
        for (int u = 0; u < CMP_ROWS; ++u) {
            const int2 pair = pairs[u * rows_per];
            to[u] = pair.x < 0 ? -1 : pair.y;
            if (pair.x >= 0) v[u] = __ldcg(pool + static_cast<size_t>(pair.x) * a.row_vecs);
        }
    };

    load_pos(0);
    load_entries(0);
    load_pos(1);
    write_pair(0);
    load_entries(1);
    load_pos(2);
    __syncthreads();
    load_rows(0);
    for (int c = 0; c < nchunks; ++c) {
        uint4 cv[CMP_ROWS];
        int cto[CMP_ROWS];
#pragma unroll
        for (int u = 0; u < CMP_ROWS; ++u) {
            cv[u] = v[u];
            cto[u] = to[u];
        }
        if (c % per_page == 0) {   // page p begins: page p + 1's pairs are due
            const int page = c / per_page;
            write_pair(page + 1);
            load_entries(page + 2);
            load_pos(page + 3);
            __syncthreads();
        }
        if (c + 1 < nchunks) load_rows(c + 1);
        __syncthreads();   // every thread has read its sources of chunk c
#pragma unroll
        for (int u = 0; u < CMP_ROWS; ++u)
            if (cto[u] >= 0) __stcg(pool + static_cast<size_t>(cto[u]) * a.row_vecs, cv[u]);
    }
}

}  // namespace pa

using namespace pa;

// Whether two arrays of n share an element.
static bool overlap(const int32_t* a, const int32_t* b, int n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b), bytes = sizeof(int32_t) * static_cast<size_t>(n);
    return x < y + bytes && y < x + bytes;
}

extern "C" int pa_select_tokens(int32_t* keep, int32_t* keep_lens, const float* weights, const int32_t* context_lens,
                                const int32_t* budgets, int num_seqs, int num_kv_heads, int weights_stride,
                                int keep_stride, int recent, int32_t* dev_err, pa_stream stream) {
    if (num_seqs < 0 || num_kv_heads <= 0 || weights_stride <= 0 || keep_stride <= 0 || recent < 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!keep || !keep_lens || !weights || !context_lens || !budgets) return PA_ERR_INVALID_ARG;
    if (!aligned_to(keep, 4) || !aligned_to(keep_lens, 4) || !aligned_to(weights, 4) || !aligned_to(context_lens, 4) ||
        !aligned_to(budgets, 4))
        return PA_ERR_INVALID_ARG;
    const long long rows = static_cast<long long>(num_seqs) * num_kv_heads;
    if (rows * SEL_MAX_CLUSTER > INT_MAX || weights_stride > MAX_POSITIONS || keep_stride > MAX_POSITIONS)
        return PA_ERR_UNSUPPORTED;
    // one CTA writes a sequence's keep_lens while those of its other heads still read the inputs
    if (overlap(keep_lens, context_lens, num_seqs) || overlap(keep_lens, budgets, num_seqs)) return PA_ERR_INVALID_ARG;
    if (const int rc = device_check(weights)) return rc;
    SelectArgs a;
    a.keep = keep;
    a.keep_lens = keep_lens;
    a.weights = weights;
    a.context_lens = context_lens;
    a.budgets = budgets;
    a.dev_err = dev_err;
    a.num_kv_heads = num_kv_heads;
    a.weights_stride = weights_stride;
    a.keep_stride = keep_stride;
    a.recent = recent;
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    // As few CTAs to a row as hold its keys, then more while that leaves SMs idle: a
    // cluster's barriers cost more than longer segments do (2048 rows of 4097: 85 us with
    // one CTA, 147 with two; 64 rows of 32768: 17 us with two or four, 25 with eight; 8
    // rows of 4097: 9.3 us with one, 8.7 with two).
    int cluster = 1;
    auto segment = [&](int c) { return ((weights_stride + c - 1) / c + 31) & ~31; };
    while (cluster < SEL_MAX_CLUSTER && segment(cluster) > sel_keys(SEL_Q_LONG)) cluster *= 2;
    while (cluster < SEL_MAX_CLUSTER && rows * cluster < sms && segment(cluster) > sel_keys(SEL_Q_SHORT)) cluster *= 2;
    const int seg = segment(cluster);
    auto kern = seg <= sel_keys(SEL_Q_SHORT)    ? select_kernel<SEL_Q_SHORT>
                : seg <= sel_keys(SEL_Q_MIDDLE) ? select_kernel<SEL_Q_MIDDLE>
                : seg <= sel_keys(SEL_Q_LONG)   ? select_kernel<SEL_Q_LONG>
                                                : select_kernel<0>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
    cfg.blockDim = dim3(SEL_THREADS);
    if (seg > sel_keys(SEL_Q_MIDDLE) && seg <= sel_keys(SEL_Q_LONG)) {
        static KernelSlot slot;
        cfg.dynamicSmemBytes = sel_keys(SEL_Q_LONG) * 4;
        if (prepare_kernel(slot, reinterpret_cast<const void*>(kern), SEL_THREADS, sel_keys(SEL_Q_LONG) * 4) <= 0)
            return PA_ERR_CUDA;
    }
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launch_status(cudaLaunchKernelEx(&cfg, kern, a));
}

extern "C" int pa_compact(void* k_cache, void* v_cache, float* weights_out, const float* weights_in, int weights_stride,
                          const int32_t* src_tables, const int32_t* dst_tables, int src_max_blocks, int dst_max_blocks,
                          const int32_t* keep, int keep_heads, int keep_stride, const int32_t* starts,
                          const int32_t* keep_lens, int num_seqs, int num_kv_heads, int head_dim, int block_size,
                          int num_blocks, pa_dtype dtype, int32_t* dev_err, pa_stream stream) {
    if (num_seqs < 0 || num_kv_heads <= 0 || num_blocks <= 0 || src_max_blocks <= 0 || dst_max_blocks <= 0 ||
        keep_stride <= 0 || !valid_dtype(dtype))
        return PA_ERR_INVALID_ARG;
    if (keep_heads != 1 && keep_heads != num_kv_heads) return PA_ERR_INVALID_ARG;
    if (!(head_dim == 64 || head_dim == 128)) return PA_ERR_UNSUPPORTED;
    if (!(block_size == 4 || block_size == 8 || block_size == 16 || block_size == 32)) return PA_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_blocks) * num_kv_heads * block_size > INT_MAX || keep_stride > MAX_POSITIONS)
        return PA_ERR_UNSUPPORTED;
    if (static_cast<long long>(src_max_blocks) * block_size > INT_MAX ||
        static_cast<long long>(dst_max_blocks) * block_size > INT_MAX)
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!k_cache || !v_cache || !src_tables || !dst_tables || !keep || !keep_lens) return PA_ERR_INVALID_ARG;
    if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(src_tables, 4) ||
        !aligned_to(dst_tables, 4) || !aligned_to(keep, 4) || !aligned_to(keep_lens, 4) ||
        (starts && !aligned_to(starts, 4)))
        return PA_ERR_INVALID_ARG;
    if ((weights_out == nullptr) != (weights_in == nullptr)) return PA_ERR_INVALID_ARG;
    // every destination that has a source fits when the source rows do
    if (weights_out && (!aligned_to(weights_out, 4) || !aligned_to(weights_in, 4) || weights_stride <= 0))
        return PA_ERR_INVALID_ARG;
    const int row_vecs = head_dim * element_bytes(dtype) / 16;
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    // Whole rows per CTA while (sequences x heads x pools) fill the GPU; below
    // that rows are cut into slices of at least 32 bytes (a memory sector).  One
    // sequence of 8 kv heads, 32768 tokens to 8192: 20 us with 32-byte slices, 40 with 128,
    // 70 with whole rows of 256; 8 sequences of 4096 to 1024: 20, 18 and 25 us.
    int log2_vecs = 0;
    while ((1 << log2_vecs) < row_vecs) ++log2_vecs;
    const long long pairs = 2LL * num_seqs * num_kv_heads;
    while (log2_vecs > 1 && pairs * (row_vecs >> log2_vecs) < 4LL * sms) --log2_vecs;
    CompactArgs a;
    a.k_cache = static_cast<uint4*>(k_cache);
    a.v_cache = static_cast<uint4*>(v_cache);
    a.w_out = weights_out;
    a.w_in = weights_in;
    a.src_tables = src_tables;
    a.dst_tables = dst_tables;
    a.keep = keep;
    a.starts = starts;
    a.keep_lens = keep_lens;
    a.dev_err = dev_err;
    a.num_kv_heads = num_kv_heads;
    a.keep_heads = keep_heads;
    a.keep_stride = keep_stride;
    a.w_stride = weights_stride;
    a.src_blocks = src_max_blocks;
    a.dst_blocks = dst_max_blocks;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.log2_block = block_size == 4 ? 2 : block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
    a.row_vecs = row_vecs;
    a.log2_vecs = log2_vecs;
    a.slices = row_vecs >> log2_vecs;
    a.walks = 2 * a.slices + (weights_out != nullptr ? 1 : 0);
    const long long ctas = static_cast<long long>(num_seqs) * num_kv_heads * a.walks;
    if (ctas > INT_MAX) return PA_ERR_UNSUPPORTED;
    if (const int rc = device_check(k_cache)) return rc;
    const cudaStream_t st = as_stream(stream);
    if (ctas <= sms) {
        static KernelSlot slot;
        const int smem = CMP_FEW_THREADS * CMP_FEW_PAIRS * static_cast<int>(sizeof(int2));
        if (prepare_kernel(slot, reinterpret_cast<const void*>(compact_few_kernel), CMP_FEW_THREADS, smem) <= 0)
            return PA_ERR_CUDA;
        return launch_status(launch_pdl(compact_few_kernel, dim3(static_cast<unsigned>(ctas)), dim3(CMP_FEW_THREADS),
                                        smem, st, a));
    }
    return launch_status(launch_pdl(compact_kernel, dim3(static_cast<unsigned>(ctas)), dim3(CMP_THREADS), 0, st, a));
}
