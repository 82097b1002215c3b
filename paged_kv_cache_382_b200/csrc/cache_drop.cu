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
// A row is split over a cluster of CTAs, each with a contiguous segment; a
// pass adds the segments' histograms through distributed shared memory, so
// every CTA knows the digit without another launch.  The segment's keys stay
// in shared memory over the passes (one read of the totals); only rows whose
// segments do not fit are read again (from L2).
// ---------------------------------------------------------------------------

constexpr int SEL_THREADS = 512;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_BINS = 2048;
constexpr int SEL_MAX_CLUSTER = 8;
constexpr int SEL_SMEM_KEYS = 48 * 1024;   // keys a CTA can hold (192 KB)

struct SelectArgs {
    int32_t* keep;
    int32_t* keep_lens;
    const float* weights;
    const int32_t* context_lens;
    const int32_t* budgets;
    int32_t* dev_err;
    int num_kv_heads, weights_stride, keep_stride, recent;
    int cached_keys;   // segment keys held in shared memory (0: read again from global memory)
};

// Order-preserving integer of a total: larger totals, larger keys.  NaN counts
// as -inf, -0 as 0.
__device__ __forceinline__ uint32_t total_key(float w) {
    const float v = w != w ? NEG_INF : w + 0.f;
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__global__ void __launch_bounds__(SEL_THREADS) select_kernel(const SelectArgs a) {
    extern __shared__ uint32_t s_keys[];
    __shared__ uint32_t hist[SEL_BINS];
    __shared__ int s_scan[33];
    __shared__ uint32_t s_digit, s_above;
    __shared__ int2 s_warp[SEL_WARPS];   // (above, equal) of each warp's sub-segment
    __shared__ int2 s_cta;               // and of the segment, read by the cluster
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / CL;
    const int s = row / a.num_kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    const float* w = a.weights + static_cast<size_t>(row) * a.weights_stride + lo;
    const bool cached = seg <= a.cached_keys;
    auto key_at = [&](int i) { return cached ? s_keys[i] : total_key(__ldg(w + i)); };
    if (cached) {
        for (int i = tid; i < len; i += SEL_THREADS) s_keys[i] = total_key(__ldg(w + i));
        __syncthreads();
    }

    uint32_t prefix = 0;       // digits found so far
    uint32_t want = k;         // rank of the sought key among those with the prefix
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10;
        const int hi_shift = shift;
        shift -= bits;
        const uint32_t mask = (1u << bits) - 1u;
        for (int i = tid; i < SEL_BINS; i += SEL_THREADS) hist[i] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < len; i0 += SEL_THREADS) {
            const int i = i0 + tid;
            const uint32_t key = i < len ? key_at(i) : 0u;
            const bool in = i < len && (pass == 0 || (key >> hi_shift) == prefix);
            const uint32_t d = (key >> shift) & mask;
            // totals that repeat (zeros above all) would add to one bin 32 times over
            const unsigned live = __ballot_sync(FULL_MASK, in);
            if (live == 0u) continue;
            const uint32_t first = __shfl_sync(FULL_MASK, d, __ffs(live) - 1);
            const unsigned same = __ballot_sync(FULL_MASK, in && d == first);
            if (lane == __ffs(live) - 1) atomicAdd(&hist[first], __popc(same));
            if (in && d != first) atomicAdd(&hist[d], 1u);
        }
        cluster.sync();        // every segment's histogram is complete
        // thread t owns bins [t * PER, (t + 1) * PER) counted from the top
        constexpr int PER = SEL_BINS / SEL_THREADS;
        uint32_t cnt[PER], sum = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            cnt[j] = 0;
            const int bin = SEL_BINS - 1 - (tid * PER + j);
            for (int c = 0; c < CL; ++c) cnt[j] += *cluster.map_shared_rank(&hist[bin], c);
            sum += cnt[j];
        }
        int total;
        uint32_t before = static_cast<uint32_t>(cta_exclusive_scan(static_cast<int>(sum), &total, s_scan));
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (before < want && want <= before + cnt[j]) {   // exactly one thread and bin
                s_digit = SEL_BINS - 1 - (tid * PER + j);
                s_above = before;
            }
            before += cnt[j];
        }
        cluster.sync();        // digit known; no CTA still reads another's histogram
        prefix = (prefix << bits) | s_digit;
        want -= s_above;
    }
    // want = how many of the keys equal to prefix stay, the first ones by position

    // warp w takes a contiguous part of the segment
    const int part = ((len + SEL_WARPS - 1) / SEL_WARPS + 31) & ~31;
    const int w0 = min(len, warp * part), w1 = min(len, w0 + part);
    int above = 0, equal = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t key = key_at(i);
        above += key > prefix;
        equal += key == prefix;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        above += __shfl_xor_sync(FULL_MASK, above, off);
        equal += __shfl_xor_sync(FULL_MASK, equal, off);
    }
    if (lane == 0) s_warp[warp] = make_int2(above, equal);
    __syncthreads();
    if (tid == 0) {
        int2 t = make_int2(0, 0);
        for (int i = 0; i < SEL_WARPS; ++i) {
            const int2 x = s_warp[i];
            s_warp[i] = t;
            t.x += x.x;
            t.y += x.y;
        }
        s_cta = t;
    }
    cluster.sync();
    int base_above = s_warp[warp].x, base_equal = s_warp[warp].y;
    for (int c = 0; c < rank; ++c) {
        const int2 t = *cluster.map_shared_rank(&s_cta, c);
        base_above += t.x;
        base_equal += t.y;
    }
    const int quota = static_cast<int>(want);
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < w1 ? key_at(i) : 0u;
        const bool up = i < w1 && key > prefix, eq = i < w1 && key == prefix;
        const unsigned bu = __ballot_sync(FULL_MASK, up), be = __ballot_sync(FULL_MASK, eq);
        const unsigned below = (1u << lane) - 1u;
        const int eq_before = base_equal + __popc(be & below);
        if (up || (eq && eq_before < quota))
            out[base_above + __popc(bu & below) + min(eq_before, quota)] = lo + i;
        base_above += __popc(bu);
        base_equal += __popc(be);
    }
    cluster.sync();   // s_cta is read by the cluster until here
}

// ---------------------------------------------------------------------------
// compact
//
// Destination position starts[s] + j of (s, h) receives position keep[s][h][j].
// Positions only move down (keep[j] >= starts + j, checked), so in place it is
// enough that, within one (s, h), chunk c of destinations is written after the
// sources of chunks 0 .. c were read: later chunks' sources lie above every
// destination of chunk c.  One CTA walks the chunks of one (s, h) in order,
// loads running ahead of the stores; other CTAs take the other pool and other
// 16-byte columns of the same rows, which never meet.
// ---------------------------------------------------------------------------

constexpr int CMP_THREADS = 256;
constexpr int CMP_ROWS = 4;   // rows per thread and chunk

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
};

__global__ void __launch_bounds__(CMP_THREADS) compact_kernel(const CompactArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    // blockIdx.x = ((s * Hkv + h) * 2 + pool) * slices + slice
    int b = blockIdx.x;
    const int slice = b % a.slices;
    b /= a.slices;
    const int which = b & 1;
    const int row = b >> 1, s = row / a.num_kv_heads, h = row - s * a.num_kv_heads;
    const int raw = a.keep_lens[s];
    const int n = clamp_context(raw, a.keep_stride);
    const int start = a.starts != nullptr ? a.starts[s] : 0;
    const bool lead = slice == 0 && which == 0;   // the CTA that reports and moves the totals
    if (lead && threadIdx.x == 0 && h == 0 && (raw != n || start < 0)) flag_error(a.dev_err, PA_DEVERR_CONTEXT);
    if (start < 0 || n == 0) return;

    const int vecs = 1 << a.log2_vecs;
    const int col = threadIdx.x & (vecs - 1), r0 = threadIdx.x >> a.log2_vecs;
    const int rows_per = CMP_THREADS >> a.log2_vecs, chunk = rows_per * CMP_ROWS;
    const int32_t* keep = a.keep + (static_cast<size_t>(s) * a.keep_heads + (a.keep_heads > 1 ? h : 0)) * a.keep_stride;
    const int32_t* src_table = a.src_tables + static_cast<size_t>(s) * a.src_blocks;
    const int32_t* dst_table = a.dst_tables + static_cast<size_t>(s) * a.dst_blocks;
    uint4* pool = (which ? a.v_cache : a.k_cache) + slice * vecs + col;
    const long long src_cap = static_cast<long long>(a.src_blocks) << a.log2_block;
    const long long dst_cap = static_cast<long long>(a.dst_blocks) << a.log2_block;
    const float* w_in = a.w_in != nullptr ? a.w_in + static_cast<size_t>(row) * a.w_stride : nullptr;
    float* w_out = a.w_out != nullptr ? a.w_out + static_cast<size_t>(row) * a.w_stride : nullptr;
    const bool totals = lead && col == 0 && w_out != nullptr;
    const int nchunks = (n + chunk - 1) / chunk;

    // three stages ahead of the store: positions, table entries, rows
    int pos[CMP_ROWS];
    int sb[CMP_ROWS], db[CMP_ROWS], sp[CMP_ROWS];
    uint4 v[CMP_ROWS];
    float tw[CMP_ROWS];
    long long to[CMP_ROWS];   // destination vector, or -1
    int wt[CMP_ROWS];         // destination position of the total, or -1

    auto load_pos = [&](int c) {
#pragma unroll
        for (int u = 0; u < CMP_ROWS; ++u) {
            const int j = c * chunk + u * rows_per + r0;
            pos[u] = j < n ? keep[j] : -1;
        }
    };
    auto load_entries = [&](int c) {
#pragma unroll
        for (int u = 0; u < CMP_ROWS; ++u) {
            const int j = c * chunk + u * rows_per + r0;
            const long long d = static_cast<long long>(start) + j;
            sp[u] = -1;
            sb[u] = db[u] = -1;
            if (j >= n) continue;
            if (pos[u] < d || pos[u] >= src_cap || d >= dst_cap) {
                if (lead) flag_error(a.dev_err, PA_DEVERR_COPY);
                continue;
            }
            sp[u] = pos[u];
            sb[u] = src_table[pos[u] >> a.log2_block];
            db[u] = dst_table[d >> a.log2_block];
        }
    };
    auto load_rows = [&](int c) {
#pragma unroll
        for (int u = 0; u < CMP_ROWS; ++u) {
            const int j = c * chunk + u * rows_per + r0;
            to[u] = -1;
            wt[u] = -1;
            if (sp[u] < 0) continue;
            if (sb[u] < 0 || sb[u] >= a.num_blocks || db[u] < 0 || db[u] >= a.num_blocks) {
                if (lead) flag_error(a.dev_err, PA_DEVERR_BLOCK_ID);
                continue;
            }
            const int d = start + j, off = a.block_size - 1;
            const long long from = ((static_cast<long long>(sb[u]) * a.num_kv_heads + h) * a.block_size + (sp[u] & off)) * a.row_vecs;
            const long long dest = ((static_cast<long long>(db[u]) * a.num_kv_heads + h) * a.block_size + (d & off)) * a.row_vecs;
            if (totals && (w_in != w_out || sp[u] != d) && sp[u] < a.w_stride) {
                tw[u] = __ldcg(w_in + sp[u]);
                wt[u] = d;
            }
            if (from == dest) continue;
            v[u] = __ldcg(pool + from);
            to[u] = dest;
        }
    };

    load_pos(0);
    load_entries(0);
    if (nchunks > 1) load_pos(1);
    load_rows(0);
    for (int c = 0; c < nchunks; ++c) {
        uint4 cv[CMP_ROWS];
        float ct[CMP_ROWS];
        long long cto[CMP_ROWS];
        int cwt[CMP_ROWS];
#pragma unroll
        for (int u = 0; u < CMP_ROWS; ++u) {
            cv[u] = v[u];
            cto[u] = to[u];
            ct[u] = tw[u];
            cwt[u] = wt[u];
        }
        if (c + 1 < nchunks) {
            load_entries(c + 1);
            if (c + 2 < nchunks) load_pos(c + 2);
            load_rows(c + 1);
        }
        __syncthreads();   // every thread has read its sources of chunk c
#pragma unroll
        for (int u = 0; u < CMP_ROWS; ++u) {
            if (cto[u] >= 0) __stcg(pool + cto[u], cv[u]);
            if (cwt[u] >= 0) __stcg(w_out + cwt[u], ct[u]);
        }
    }
}

}  // namespace pa

using namespace pa;

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
    if (rows * SEL_MAX_CLUSTER > INT_MAX) return PA_ERR_UNSUPPORTED;
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
    int cluster = 1;
    while (cluster < SEL_MAX_CLUSTER && weights_stride / cluster > 4096) cluster *= 2;
    const int seg = ((weights_stride + cluster - 1) / cluster + 31) & ~31;
    a.cached_keys = seg <= SEL_SMEM_KEYS ? seg : 0;
    const int smem = a.cached_keys * 4;
    static KernelSlot slot;
    if (prepare_kernel(slot, reinterpret_cast<const void*>(select_kernel), SEL_THREADS, SEL_SMEM_KEYS * 4) <= 0)
        return PA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
    cfg.blockDim = dim3(SEL_THREADS);
    cfg.dynamicSmemBytes = smem;
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
    return launch_status(cudaLaunchKernelEx(&cfg, select_kernel, a));
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
    // that rows are cut into slices of at least 32 bytes (a memory sector).
    int log2_vecs = 0;
    while ((1 << log2_vecs) < row_vecs) ++log2_vecs;
    const long long walks = 2LL * num_seqs * num_kv_heads;
    while (log2_vecs > 1 && walks * (row_vecs >> log2_vecs) < 4LL * sms) --log2_vecs;
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
    const long long ctas = walks * a.slices;
    if (ctas > INT_MAX) return PA_ERR_UNSUPPORTED;
    if (const int rc = device_check(k_cache)) return rc;
    return launch_status(launch_pdl(compact_kernel, dim3(static_cast<unsigned>(ctas)), dim3(CMP_THREADS), 0,
                                    as_stream(stream), a));
}
