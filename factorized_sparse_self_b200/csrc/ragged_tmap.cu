// Tensor maps of token-row tensors for the ragged kernels. They are encoded in
// every call (a few hundred nanoseconds each): callers' buffers come and go.
#include <cuda.h>

#include "ragged_tc.cuh"

namespace st {
namespace rag {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// [outer][rows][heads][d] (strides in rows of d elements) with boxes of `heads_box`
// heads x `rows_box` rows x 64 columns.
bool encode(CUtensorMap* out, const void* base, bool f16, int d, int heads, int head, int rows, int row,
            int outer, int64_t outer_stride, int heads_box, int rows_box) {
  const EncodeTiledFn enc = encode_fn();
  const cuuint64_t es = (cuuint64_t)d * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)outer};
  const cuuint64_t strides[3] = {head * es, row * es, (cuuint64_t)outer_stride * es};
  const cuuint32_t box[4] = {64, (cuuint32_t)heads_box, (cuuint32_t)rows_box, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc && enc(out, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                    const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool make_key_maps(TileMaps& m, const Geo& g, const void* k, const void* v, bool f16) {
  m.nat_rows = m.sum_rows = 0;
  if (g.kv_lens) {
    // boxes of the largest power of two that divides the page, from 8 rows on
    const int r = g.page_size & -g.page_size;
    if (r < 8 || g.k.head < 1 || g.k.tok < 1 || g.k.page < 1) return true;
    m.nat_rows = r < 128 ? r : 128;
    return encode(&m.k, k, f16, g.d, g.Hkv, g.k.head, g.page_size, g.k.tok, g.num_pages, g.k.page, 1, m.nat_rows) &&
           encode(&m.v, v, f16, g.d, g.Hkv, g.v.head, g.page_size, g.v.tok, g.num_pages, g.v.page, 1, m.nat_rows);
  }
  m.nat_rows = 128;
  if (!encode(&m.k, k, f16, g.d, g.Hkv, 1, g.total, g.k.tok, 1, (int64_t)g.total * g.k.tok, 1, 128) ||
      !encode(&m.v, v, f16, g.d, g.Hkv, 1, g.total, g.v.tok, 1, (int64_t)g.total * g.v.tok, 1, 128))
    return false;
  if (g.c % 8 == 0 && 128 % g.c == 0) {
    m.sum_rows = g.c;
    return encode(&m.ksum, k, f16, g.d, g.Hkv, 1, g.total, g.k.tok, 1, (int64_t)g.total * g.k.tok, 1, g.c) &&
           encode(&m.vsum, v, f16, g.d, g.Hkv, 1, g.total, g.v.tok, 1, (int64_t)g.total * g.v.tok, 1, g.c);
  }
  return true;
}

bool make_query_map(CUtensorMap* out, TileMaps& m, const Geo& g, const Rows& rows, const void* base, bool f16) {
  m.q_tokens = 0;
  if (g.split || 128 % g.G) return true;
  m.q_tokens = 128 / g.G;
  return encode(out, base, f16, g.d, g.H, 1, g.total, rows.tok, 1, (int64_t)g.total * rows.tok, g.G, m.q_tokens);
}

}  // namespace rag
}  // namespace st
