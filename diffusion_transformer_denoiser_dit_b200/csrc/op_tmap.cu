// Tensor maps over strided views (the packed-layer building blocks' operands).
#include "internal.h"
#include "ops.h"

namespace dit {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    return nullptr;
  }();
  return fn;
}

bool make_tmap_view(CUtensorMap* map, int dtype, const void* base, int rank, const uint64_t* dims,
                    const uint64_t* strides_bytes, const uint32_t* box) {
  const EncodeTiledFn fn = encode_tiled();
  const uint32_t es = dtype == DIT_DTYPE_F32 ? 4 : 2;
  if (fn == nullptr || rank < 2 || rank > 4 || (reinterpret_cast<uintptr_t>(base) & 15u) != 0 || box[0] * es != 128)
    return false;
  cuuint64_t d[4], s[4];
  cuuint32_t b[4], e[4];
  for (int i = 0; i < rank; ++i) {
    if (dims[i] == 0 || box[i] == 0 || box[i] > 256) return false;
    d[i] = dims[i];
    b[i] = box[i];
    e[i] = 1;
    if (i + 1 < rank) {
      s[i] = strides_bytes[i];
      if (s[i] == 0 || s[i] % 16 != 0 || s[i] >= (1ull << 40)) return false;
    }
  }
  const CUtensorMapDataType t = dtype == DIT_DTYPE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : dtype == DIT_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(map, t, rank, const_cast<void*>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dit
