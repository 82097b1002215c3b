// tree_decode.cu -- pa_tree_decode: attention of a tree of drafted tokens over
// a paged cache.  The entry point, the attend kernel on the CUDA cores (fp32
// pools), the join of cut units, and the host-side construction of masks from
// parents (pa_tree_mask).  tree.cuh says what is computed and how the work is cut.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>
#include <cmath>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_host.h"
#include "tree.cuh"

namespace pa {
namespace {

// ---------------------------------------------------------------------------
// attend on the CUDA cores
//
// Bound by fp32 FMAs (4 rows d per token and kv head).  256 threads, 16 x 16:
// thread (ty, tx) holds rows 4 ty .. 4 ty + 3 of S for tokens 4 tx .. and of O
// for D / 16 columns, so each operand read from shared memory feeds four FMAs.
// Q and K are stored transposed ([d][row]) for that; softmax statistics of a row
// live in the 16 threads that share it.  The weights take K's place once S is
// complete, so that two CTAs fit an SM and one loads while the other computes.
// ---------------------------------------------------------------------------

constexpr int TS_ROWS = 64;
constexpr int TS_KT = 64;
constexpr int TS_THREADS = 256;
constexpr int TS_PAD = 68;   // floats per transposed row: 16-byte aligned, columns spread over the banks

template <int D>
constexpr int tree_simt_smem() {
    return (2 * D * TS_PAD + TS_KT * D) * 4;
}

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

template <int D>
__global__ void __launch_bounds__(TS_THREADS, 2) tree_simt_kernel(const TreeArgs a) {
    constexpr int OC = D / 16;   // output columns per thread
    extern __shared__ __align__(16) uint8_t smem_dyn[];
    float* sQ = reinterpret_cast<float*>(smem_dyn);   // [D][TS_PAD]
    float* sK = sQ + D * TS_PAD;                      // [D][TS_PAD]
    float* sV = sK + D * TS_PAD;                      // [TS_KT][D]
    float* sP = sK;                                   // [TS_ROWS][TS_PAD], once S is complete
    __shared__ int s_row[TS_KT];                      // pool row of each token of the tile, or -1
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const float* q = static_cast<const float*>(a.q);
    const float* kc = static_cast<const float*>(a.k_cache);
    const float* vc = static_cast<const float*>(a.v_cache);
    pdl_wait();
    pdl_launch_dependents();
    TreeWalker<TS_ROWS, 1, TS_KT> walk;
    tree_begin(a, reinterpret_cast<int*>(smem_dyn), walk);
    __syncthreads();

    TreeRun r;
    while (walk.next(a, r)) {
        if (r.starts && tid == 0) tree_record(a, r);
        // Q, scaled into the log2 domain
        for (int i = tid; i < TS_ROWS * (D / 4); i += TS_THREADS) {
            const int row = i % TS_ROWS, c = i / TS_ROWS * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < r.rows) v = load4(q + tree_out_row(a, r.first, r.kvh, r.row0 + row) * D + c);
            sQ[(c + 0) * TS_PAD + row] = v.x;
            sQ[(c + 1) * TS_PAD + row] = v.y;
            sQ[(c + 2) * TS_PAD + row] = v.z;
            sQ[(c + 3) * TS_PAD + row] = v.w;
        }
        const uint32_t* mrow[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mrow[i] = a.tree_mask + static_cast<size_t>(r.first + min(r.n - 1, (r.row0 + 4 * ty + i) / a.group)) * a.mask_words32;
        const int pre = r.ctx - r.n;   // positions below it: the prefix
        float m[4], l[4], o[4][OC];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = NEG_INF;
            l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < OC; ++j) o[i][j] = 0.f;
        }
        for (int t = r.t0; t < r.t1; ++t) {
            const int p0 = t * TS_KT;
            __syncthreads();   // the previous tile is no longer read
            if (tid < TS_KT) {
                int at = -1;
                if (p0 + tid < r.ctx) {
                    const int b = a.block_tables[static_cast<size_t>(r.s) * a.max_blocks + ((p0 + tid) >> a.log2_block)];
                    if (b < 0 || b >= a.num_blocks)
                        flag_error(a.dev_err, PA_DEVERR_BLOCK_ID);
                    else
                        at = (b * a.num_kv_heads + r.kvh) * a.block_size + ((p0 + tid) & (a.block_size - 1));
                }
                s_row[tid] = at;
            }
            __syncthreads();
            for (int i = tid; i < TS_KT * (D / 4); i += TS_THREADS) {
                const int tok = i % TS_KT, c = i / TS_KT * 4;
                const int at = s_row[tok];
                float4 k4 = make_float4(0.f, 0.f, 0.f, 0.f);
                if (at >= 0) k4 = load4(kc + static_cast<size_t>(at) * D + c);
                sK[(c + 0) * TS_PAD + tok] = k4.x;
                sK[(c + 1) * TS_PAD + tok] = k4.y;
                sK[(c + 2) * TS_PAD + tok] = k4.z;
                sK[(c + 3) * TS_PAD + tok] = k4.w;
            }
            int odd = 0;
            for (int i = tid; i < TS_KT * (D / 4); i += TS_THREADS) {
                const int tok = i / (D / 4), c = i % (D / 4) * 4;
                const int at = s_row[tok];
                float4 v4 = make_float4(0.f, 0.f, 0.f, 0.f);   // tokens that take no part: 0 * 0
                if (at >= 0) v4 = load4(vc + static_cast<size_t>(at) * D + c);
                // a node's non-finite value must not meet the zero weight of a row that
                // does not see it
                if (p0 + tok >= pre) odd |= !(isfinite(v4.x) && isfinite(v4.y) && isfinite(v4.z) && isfinite(v4.w));
                *reinterpret_cast<float4*>(sV + tok * D + c) = v4;
            }
            const bool guarded = __syncthreads_or(odd);
            float x[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; ++d) {
                const float4 qv = *reinterpret_cast<const float4*>(sQ + d * TS_PAD + 4 * ty);
                const float4 kv = *reinterpret_cast<const float4*>(sK + d * TS_PAD + 4 * tx);
                const float qa[4] = {qv.x, qv.y, qv.z, qv.w}, ka[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[i][j] = fmaf(qa[i], ka[j], x[i][j]);
            }
            __syncthreads();   // K is no longer read: P goes there
            uint32_t in = 0;   // tokens of this thread that take part
#pragma unroll
            for (int j = 0; j < 4; ++j) in |= (s_row[4 * tx + j] >= 0 ? 1u : 0u) << j;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t seen = in & tree_bits(mrow[i], a.mask_words32, p0 + 4 * tx - pre);
                float mx = NEG_INF;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = (seen >> j) & 1u ? x[i][j] * a.scale_log2 : NEG_INF;
                    mx = fmaxf(mx, x[i][j]);
                }
#pragma unroll
                for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, off));
                const float mn = fmaxf(m[i], mx);
                const float base = mn == NEG_INF ? 0.f : mn;
                const float al = exp2_approx(m[i] - base);
                m[i] = mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = exp2_approx(x[i][j] - base);
                    sum += x[i][j];
                }
#pragma unroll
                for (int off = 1; off < 16; off <<= 1) sum += __shfl_xor_sync(FULL_MASK, sum, off);
                l[i] = fmaf(l[i], al, sum);
#pragma unroll
                for (int j = 0; j < OC; ++j) o[i][j] *= al;
                *reinterpret_cast<float4*>(sP + (4 * ty + i) * TS_PAD + 4 * tx) =
                    make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
            }
            __syncwarp();   // a row's 16 threads share a warp
            auto add_values = [&](auto skip_zero) {
#pragma unroll 2
                for (int tok = 0; tok < TS_KT; tok += 4) {
                    float p[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = *reinterpret_cast<const float4*>(sP + (4 * ty + i) * TS_PAD + tok);
                        p[i][0] = v.x;
                        p[i][1] = v.y;
                        p[i][2] = v.z;
                        p[i][3] = v.w;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int j = 0; j < OC; j += 4) {
                            const float4 v = *reinterpret_cast<const float4*>(sV + (tok + k) * D + 16 * j + 4 * tx);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (decltype(skip_zero)::value && p[i][k] == 0.f) continue;
                                o[i][j + 0] = fmaf(p[i][k], v.x, o[i][j + 0]);
                                o[i][j + 1] = fmaf(p[i][k], v.y, o[i][j + 1]);
                                o[i][j + 2] = fmaf(p[i][k], v.z, o[i][j + 2]);
                                o[i][j + 3] = fmaf(p[i][k], v.w, o[i][j + 3]);
                            }
                        }
                    }
                }
            };
            if (guarded)
                add_values(std::true_type());
            else
                add_values(std::false_type());
        }
        const bool whole = r.t0 == 0 && r.t1 == r.nt;
        const int slot = 2 * blockIdx.x + (r.starts ? 0 : 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * ty + i;
            if (row >= r.rows) continue;
            if (whole) {
                const size_t at = tree_out_row(a, r.first, r.kvh, r.row0 + row) * D;
                const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
                for (int j = 0; j < OC; j += 4)
                    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + 16 * j + 4 * tx) =
                        make_float4(o[i][j] * inv, o[i][j + 1] * inv, o[i][j + 2] * inv, o[i][j + 3] * inv);
            } else {
                float4* acc = reinterpret_cast<float4*>(tree_part(a, slot, D));
#pragma unroll
                for (int j = 0; j < OC; j += 4)
                    acc[(4 * j + tx) * a.part_rows + row] = make_float4(o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]);
                if (tx == 0) a.part_ml[static_cast<size_t>(slot) * a.part_rows + row] = make_float2(m[i], l[i]);
            }
        }
        __syncthreads();   // sQ and sP are written again for the next run
    }
}

template <int D>
int launch_tree_simt(const TreeArgs& a, int ctas, cudaStream_t st) {
    static KernelSlot slot;
    auto kern = tree_simt_kernel<D>;
    if (prepare_kernel(slot, reinterpret_cast<const void*>(kern), TS_THREADS, tree_simt_smem<D>()) <= 0) return PA_ERR_CUDA;
    return launch_status(launch_pdl(kern, dim3(ctas), dim3(TS_THREADS), tree_simt_smem<D>(), st, a));
}

// ---------------------------------------------------------------------------
// join: the partials of each unit that the shares cut, in CTA order.  The
// unit's first cut lies at the start of some CTA's share: that CTA's row of
// the grid joins it.
// ---------------------------------------------------------------------------

constexpr int TJ_THREADS = 256;
constexpr int TJ_ROWS = 16;   // rows per CTA: two float4 per thread at d = 128, so that all loads go out at once

template <int D>
__global__ void __launch_bounds__(TJ_THREADS) tree_join_kernel(const TreeArgs a, int ctas) {
    __shared__ float s_coef[TJ_ROWS][TREE_CTAS_MAX + 1];   // weight of each partial
    __shared__ int s_slot[TREE_CTAS_MAX];
    __shared__ int s_parts;
    pdl_wait();
    pdl_launch_dependents();
    const int c = blockIdx.x + 1;   // share 0 starts no cut
    const int W = *a.line;
    const TreeRecord r = a.recs[c];
    const int g = tree_sharers(W, ctas);
    if (c >= g || r.t0 == 0) return;                     // no share, or it starts with a unit
    const int row0 = blockIdx.y * TJ_ROWS, here = min(TJ_ROWS, r.rows - row0);
    if (here <= 0) return;
    // the tiles [t0, t1) that share x holds of this unit
    auto first_tile = [&](int x) {
        const int off = tree_share(W, g, x) - r.begin;
        return off <= 0 ? 0 : min(r.nt, (off + r.per_tile - 1) / r.per_tile);
    };
    // the unit's tile 0 lies in the nearest share before c that holds a tile of it;
    // c joins the unit if that one is it, i.e. starts with or before the unit
    int head = c - 1;
    while (first_tile(head) == r.t0) --head;             // no tile of its own
    if (first_tile(head) > 0) return;                    // not the unit's first cut
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int head_slot = 2 * head + (a.recs[head].begin == r.begin ? 0 : 1);
        int n = 1;
        if (lane == 0) s_slot[0] = head_slot;
        for (int x0 = c; x0 < g && first_tile(x0) < r.nt; x0 += 32) {
            const int x = x0 + lane;
            const bool has = x < g && first_tile(x) < first_tile(x + 1);
            const unsigned all = __ballot_sync(FULL_MASK, has);
            if (has) s_slot[n + __popc(all & ((1u << lane) - 1u))] = 2 * x;
            n += __popc(all);
        }
        if (lane == 0) s_parts = n;
    }
    __syncthreads();
    const int parts = s_parts;
    // coefficients: half a warp per row, a lane per partial
    const int sub = threadIdx.x & 15, rr = threadIdx.x >> 4;
    if (rr < here) {
        const size_t row = row0 + rr;
        float M = NEG_INF, L = 0.f;
        float2 ml0 = make_float2(NEG_INF, 0.f);
        if (sub < parts) ml0 = a.part_ml[static_cast<size_t>(s_slot[sub]) * a.part_rows + row];
        M = ml0.x;
        for (int p = sub + 16; p < parts; p += 16)
            M = fmaxf(M, a.part_ml[static_cast<size_t>(s_slot[p]) * a.part_rows + row].x);
        const unsigned half = 0xffffu << (threadIdx.x & 16);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(half, M, off));
        for (int p = sub; p < parts; p += 16) {
            const float2 ml = p == sub ? ml0 : a.part_ml[static_cast<size_t>(s_slot[p]) * a.part_rows + row];
            const float e = M == NEG_INF ? 0.f : exp2_approx(ml.x - M);
            s_coef[rr][p] = e;
            L = fmaf(e, ml.y, L);
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) L += __shfl_xor_sync(half, L, off);
        const float inv = L > 0.f ? 1.f / L : 0.f;
        for (int p = sub; p < parts; p += 16) s_coef[rr][p] *= inv;
    }
    __syncthreads();
    constexpr int ITEMS = TJ_ROWS * (D / 4) / TJ_THREADS, U = 4;
    const int i0 = threadIdx.x % TJ_ROWS;   // row, fastest over the threads: the partials' order
    if (i0 >= here) return;
    float4 o[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += U) {
        float4 v[U][ITEMS];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
                if (p0 + u < parts)
                    v[u][k] = reinterpret_cast<const float4*>(tree_part(a, s_slot[p0 + u], D))
                        [(threadIdx.x / TJ_ROWS + k * (TJ_THREADS / TJ_ROWS)) * a.part_rows + row0 + i0];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p0 + u >= parts) break;
            const float e = s_coef[i0][p0 + u];
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                o[k].x = fmaf(e, v[u][k].x, o[k].x);
                o[k].y = fmaf(e, v[u][k].y, o[k].y);
                o[k].z = fmaf(e, v[u][k].z, o[k].z);
                o[k].w = fmaf(e, v[u][k].w, o[k].w);
            }
        }
    }
    const size_t at = tree_out_row(a, r.first, r.kvh, r.row0 + row0 + i0) * D;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const size_t col = at + 4 * (threadIdx.x / TJ_ROWS + k * (TJ_THREADS / TJ_ROWS));
        if (a.out_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + col) = o[k];
        else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + col) =
                make_uint2(pack_bf16(o[k].x, o[k].y), pack_bf16(o[k].z, o[k].w));
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct TreeWs {
    size_t line, recs, ml, acc, total;
    int tc_rows, simt_rows;   // rows of a partial
};

inline TreeWs tree_ws(long long num_tokens, int num_heads, int head_dim) {
    TreeWs w;
    const long long rows = num_tokens * num_heads;   // no unit has more
    // on the tensor cores a row of every stream: both may hold the same rows
    w.tc_rows = static_cast<int>(2 * rows < tree_tc_rows() ? 2 * rows : tree_tc_rows());
    w.simt_rows = static_cast<int>(rows < TS_ROWS ? rows : TS_ROWS);
    const size_t tc = 2ull * TREE_TC_CTAS * w.tc_rows, simt = 2ull * TREE_SIMT_CTAS * w.simt_rows;
    const size_t most = tc > simt ? tc : simt;
    w.line = 0;
    w.recs = 256;
    w.ml = w.recs + up256(TREE_CTAS_MAX * sizeof(TreeRecord));
    w.acc = w.ml + up256(most * sizeof(float2));
    w.total = w.acc + up256(most * head_dim * sizeof(float));
    return w;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_tree_workspace_bytes(int num_tokens, int num_heads, int head_dim) {
    if (num_tokens < 0 || num_heads <= 0 || head_dim <= 0) return 0;
    return tree_ws(num_tokens, num_heads, head_dim).total;
}

extern "C" int pa_tree_uses_tensor_cores(pa_dtype dtype, int block_size) { return tree_tc_eligible(dtype, block_size) ? 1 : 0; }

extern "C" int pa_tree_decode(void* out, pa_dtype out_dtype, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
                              const int64_t* tree_mask, int mask_words, int num_seqs, int num_tokens, int num_heads,
                              int num_kv_heads, int head_dim, int block_size, int num_blocks, int max_blocks_per_seq,
                              int max_context_len, float scale, void* workspace, size_t workspace_bytes, pa_dtype dtype,
                              int32_t* dev_err, pa_stream stream) {
    if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || max_context_len < 0 || num_heads % num_kv_heads != 0 || !valid_dtype(dtype) ||
        !valid_dtype(out_dtype) || !std::isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (out_dtype != PA_F32 && out_dtype != dtype) return PA_ERR_UNSUPPORTED;
    if (!(head_dim == 64 || head_dim == 128)) return PA_ERR_UNSUPPORTED;
    if (!(block_size == 4 || block_size == 8 || block_size == 16 || block_size == 32)) return PA_ERR_UNSUPPORTED;
    if (mask_words < 1) return PA_ERR_INVALID_ARG;
    if (mask_words > PA_TREE_MAX_WORDS) return PA_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_blocks) * num_kv_heads * block_size > INT_MAX ||
        static_cast<long long>(num_tokens) * num_heads > INT_MAX || num_seqs > 32 * TREE_WINDOWS_MAX)
        return PA_ERR_UNSUPPORTED;
    if (static_cast<long long>(max_blocks_per_seq) * block_size > INT_MAX) return PA_ERR_INVALID_ARG;
    long long cap = static_cast<long long>(max_blocks_per_seq) * block_size;
    if (max_context_len > 0 && max_context_len < cap) cap = max_context_len;
    if (cap > MAX_POSITIONS) return PA_ERR_UNSUPPORTED;
    // the work line is counted in 32 bits: at most this many half row blocks, each
    // with a step per 64-token tile
    const long long halves = static_cast<long long>(num_tokens) * num_heads / TS_ROWS +
                             static_cast<long long>(num_seqs) * num_kv_heads;
    if (halves > INT_MAX / (cap / TS_KT + 1 + TREE_UNIT_STEPS)) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (num_seqs == 0) return PA_ERR_INVALID_ARG;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || !tree_mask || !workspace)
        return PA_ERR_INVALID_ARG;
    if (!aligned_to(out, 16) || !aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
        !aligned_to(block_tables, 4) || !aligned_to(context_lens, 4) || !aligned_to(query_start, 4) ||
        !aligned_to(tree_mask, 8) || !aligned_to(workspace, 256))
        return PA_ERR_INVALID_ARG;
    const TreeWs L = tree_ws(num_tokens, num_heads, head_dim);
    if (workspace_bytes < L.total) return PA_ERR_WORKSPACE;

    TreeArgs a;
    a.out = out;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.tree_mask = reinterpret_cast<const uint32_t*>(tree_mask);
    a.dev_err = dev_err;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.line = reinterpret_cast<int*>(ws + L.line);
    a.recs = reinterpret_cast<TreeRecord*>(ws + L.recs);
    a.part_ml = reinterpret_cast<float2*>(ws + L.ml);
    a.part_acc = reinterpret_cast<float*>(ws + L.acc);
    const bool tc = tree_tc_eligible(dtype, block_size);
    a.part_rows = tc ? L.tc_rows : L.simt_rows;
    a.mask_words32 = 2 * mask_words;
    a.num_seqs = num_seqs;
    a.num_tokens = num_tokens;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = num_heads / num_kv_heads;
    a.block_size = block_size;
    a.log2_block = block_size == 4 ? 2 : block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
    a.num_blocks = num_blocks;
    a.max_blocks = max_blocks_per_seq;
    a.cap = static_cast<int>(cap);
    a.scale_log2 = scale * LOG2E;
    a.out_f32 = out_dtype == PA_F32;
    const cudaStream_t st = as_stream(stream);
    if (const int rc = device_check(k_cache)) return rc;
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const int ctas = tc ? (sms < TREE_TC_CTAS ? sms : TREE_TC_CTAS) : (2 * sms < TREE_SIMT_CTAS ? 2 * sms : TREE_SIMT_CTAS);
    int rc;
    if (tc)
        rc = launch_tree_tc(a, head_dim, ctas, st);
    else
        rc = head_dim == 128 ? launch_tree_simt<128>(a, ctas, st) : launch_tree_simt<64>(a, ctas, st);
    if (rc != PA_OK || ctas < 2) return rc;
    const long long rows = static_cast<long long>(num_tokens) * num_heads;   // no unit has more
    const int unit_rows = rows < a.part_rows ? static_cast<int>(rows) : a.part_rows;
    const dim3 grid(ctas - 1, (unit_rows + TJ_ROWS - 1) / TJ_ROWS);
    return launch_status(head_dim == 128 ? launch_pdl(tree_join_kernel<128>, grid, dim3(TJ_THREADS), 0, st, a, ctas)
                                         : launch_pdl(tree_join_kernel<64>, grid, dim3(TJ_THREADS), 0, st, a, ctas));
}

extern "C" int pa_tree_mask(const int32_t* parents, int num_nodes, int mask_words, int64_t* mask) {
    if (num_nodes < 0 || mask_words < 1) return PA_ERR_INVALID_ARG;
    if (mask_words > PA_TREE_MAX_WORDS || num_nodes > 64 * mask_words) return PA_ERR_UNSUPPORTED;
    if (num_nodes > 0 && (!parents || !mask)) return PA_ERR_INVALID_ARG;
    for (int i = 0; i < num_nodes; ++i)
        if (parents[i] >= i) return PA_ERR_INVALID_ARG;   // parents come first
    for (int i = 0; i < num_nodes; ++i) {
        uint64_t* row = reinterpret_cast<uint64_t*>(mask) + static_cast<size_t>(i) * mask_words;
        const uint64_t* up = parents[i] >= 0 ? reinterpret_cast<const uint64_t*>(mask) + static_cast<size_t>(parents[i]) * mask_words : nullptr;
        for (int w = 0; w < mask_words; ++w) row[w] = up ? up[w] : 0u;
        row[i / 64] |= 1ull << (i % 64);
    }
    return PA_OK;
}
