// Tensor maps for the TMA-staged kernels: the driver's cuTensorMapEncodeTiled,
// looked up once (the CUDA runtime is linked statically, so the driver entry
// point is resolved at run time), and a bf16 encoder on top of it.
#include <mutex>

#include "cmr_internal.cuh"

namespace cmr {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

bool encode(CUtensorMap* map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle,
            CUtensorMapL2promotion promotion, void* base, int rank, const uint64_t* dims,
            const uint64_t* strides_bytes, const uint32_t* box) {
  const EncodeTiledFn enc = encoder();
  if (enc == nullptr || rank < 1 || rank > 5) return false;
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], unit[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    unit[i] = 1;
    if (i + 1 < rank) st[i] = strides_bytes[i];
  }
  return enc(map, type, static_cast<cuuint32_t>(rank), base, d, st, b, unit,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool encode_bf16_tensor_map(CUtensorMap* map, void* base, int rank, const uint64_t* dims,
                            const uint64_t* strides_bytes, const uint32_t* box,
                            bool swizzle_128b) {
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                swizzle_128b ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_NONE, base, rank, dims, strides_bytes, box);
}

bool encode_u8_tensor_map(CUtensorMap* map, void* base, int rank, const uint64_t* dims,
                          const uint64_t* strides_bytes, const uint32_t* box,
                          int swizzle_bytes) {
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                swizzle_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B, base, rank, dims, strides_bytes, box);
}

int64_t device_l2_bytes() {
  static std::mutex mu;
  static int64_t cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (cached[dev & 63] == 0) {
    int l2 = 0;
    if (cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    cached[dev & 63] = l2 > 0 ? l2 : 1;
  }
  return cached[dev & 63];
}

}  // namespace cmr
