// Host-side construction of TMA tensor maps (cuTensorMapEncodeTiled, reached through the
// runtime's driver entry point so the library needs no direct libcuda link).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "pa_common.cuh"

namespace pa {
namespace {
std::once_flag g_encode_once;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}
}  // namespace

// 3-D bf16 view [outer][heads][128 dims] (dims innermost); box = 64 dims x box_heads x box_rows;
// 128-byte swizzle; zero fill outside the tensor.
bool make_map_heads(CUtensorMap* map, const void* base, uint64_t outer, uint64_t heads,
                    uint32_t box_heads, uint32_t box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {128, heads, outer};
  cuuint64_t strides[2] = {256, heads * 256};
  cuuint32_t box[3] = {64, box_heads, box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same with a box of one head.
bool make_map_3d(CUtensorMap* map, const void* base, uint64_t outer, uint64_t heads,
                 uint32_t box_rows) {
  return make_map_heads(map, base, outer, heads, 1, box_rows);
}

// A page pool [num_pages][16 tokens][heads][128 dims] as 5-D [head][8 tokens' group][half of the dims][8
// tokens][64 dims]; box = one head's page, which arrives as two groups of 8 tokens, each 1 KB of the first
// 64 dims and 1 KB of the others: whole swizzle atoms at one stride however many pages stand behind each
// other. 128-byte swizzle.
bool make_map_pages(CUtensorMap* map, const void* base, uint64_t num_pages, uint64_t heads) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[5] = {64, 8, 2, num_pages * 2, heads};
  cuuint64_t strides[4] = {heads * 256, 128, 8 * heads * 256, 256};
  cuuint32_t box[5] = {64, 8, 2, 2, 1};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D bf16 matrix [rows][cols] with a row stride in bytes; box = 64 columns x box_rows rows;
// 128-byte swizzle; zero fill outside the matrix.
bool make_map_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                 uint64_t row_stride_bytes, uint32_t box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {row_stride_bytes};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pa
