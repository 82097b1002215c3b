// pa_tma.h -- host-side tensor-map set-up for the bulk tensor copies of the
// paged pools (driver entry point looked up through the runtime, so the
// library needs no link against the driver library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace pa {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled_fn() {
    static std::atomic<EncodeTiledFn> fn{nullptr};
    EncodeTiledFn f = fn.load(std::memory_order_acquire);
    if (f) return f;
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || ptr == nullptr)
        return nullptr;
    f = reinterpret_cast<EncodeTiledFn>(ptr);
    fn.store(f, std::memory_order_release);
    return f;
}

// Tensor map over one bf16 pool viewed as rows of head_dim elements
// (row = (block * Hkv + kv_head) * B + slot), boxes of 64 columns x rb rows.
inline bool encode_pool_map(CUtensorMap* m, const void* pool, int num_blocks, int Hkv, int B, int D,
                            int rb) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D),
                                static_cast<cuuint64_t>(num_blocks) * Hkv * B};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * 2};
    const cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(rb)};
    const cuuint32_t estr[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same pool as 8-row groups of 64-column parts: one box brings a whole block
// of one kv head (B a multiple of 8) and lays it out as [8-row group][64-column
// part][8 rows][64 columns], so that consecutive blocks continue one another with
// one group stride.
inline bool encode_block_map(CUtensorMap* m, const void* pool, int num_blocks, int Hkv, int B, int D) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
    const cuuint64_t dims[4] = {64u, 8u, static_cast<cuuint64_t>(D / 64),
                                static_cast<cuuint64_t>(num_blocks) * Hkv * (B / 8)};
    const cuuint64_t strides[3] = {row, 128u, 8 * row};
    const cuuint32_t box[4] = {64u, 8u, static_cast<cuuint32_t>(D / 64), static_cast<cuuint32_t>(B / 8)};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for blocks of four tokens, half a group: one box is a 64-column part of
// a block, and two blocks share a group.  (The 128-byte swizzle goes by the address
// in shared memory, so the second half of a group is swizzled as its rows 4 to 7.)
inline bool encode_half_group_map(CUtensorMap* m, const void* pool, int num_blocks, int Hkv, int D) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
    const cuuint64_t dims[4] = {64u, 4u, static_cast<cuuint64_t>(D / 64), static_cast<cuuint64_t>(num_blocks) * Hkv};
    const cuuint64_t strides[3] = {row, 128u, 4 * row};
    const cuuint32_t box[4] = {64u, 4u, 1u, 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pa
