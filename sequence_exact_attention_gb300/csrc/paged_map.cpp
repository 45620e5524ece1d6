// TMA tensor maps of the paged key/value cache. The driver's encoder is looked
// up once through the runtime, so the library links no driver library directly.
#include <mutex>

#include "paged_internal.h"

namespace ra {
namespace {

using EncodeTiledFn = decltype(&cuTensorMapEncodeTiled);

EncodeTiledFn encoder() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

}  // namespace

bool make_page_map(CUtensorMap* m, const PagePool& p, const void* ptr, int box_rows,
                   int box_parts) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  const cuuint64_t size = p.quant ? 1 : 2, cols = p.quant ? p.D : 64;
  cuuint64_t dims[4] = {cols, (cuuint64_t)p.page, p.D / cols, (cuuint64_t)p.n_pages * p.H_kv};
  cuuint64_t strides[3] = {p.D * size, cols * size, p.D * size * p.page};
  cuuint32_t box[4] = {(cuuint32_t)cols, (cuuint32_t)box_rows, (cuuint32_t)box_parts, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, p.quant ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             p.quant && p.D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_query_map(CUtensorMap* m, const void* q, int rows, int H_q, int D, int heads,
                    int tokens) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H_q, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H_q * D * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ra
