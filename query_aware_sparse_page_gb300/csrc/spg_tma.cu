// Host side of the TMA tensor tiles: encodes the tensor maps through which the
// kernels copy tiles of pools, queries and matrices.  cuTensorMapEncodeTiled comes from
// the runtime's driver entry-point lookup, so the library does not link
// against the driver library itself.
#include <cudaTypedefs.h>

#include <mutex>

#include "spg_internal.h"

namespace spg {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

}  // namespace

bool encode_tmap(CUtensorMap* map, CUtensorMapDataType dtype, int rank, const void* base, const uint64_t* dims,
                 const uint64_t* strides, const uint32_t* box) {
  const auto fn = encode_fn();
  if (!fn || rank < 2 || rank > 4) return false;
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i + 1 < rank) s[i] = strides[i];
  }
  const auto encode = [&] {
    return fn(map, dtype, rank, const_cast<void*>(base), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r != CUDA_SUCCESS && r != CUDA_ERROR_INVALID_VALUE) {
    // The encoder is a driver call and wants a context, which a host thread only
    // gets with its first work in the runtime: a thread whose first work is this
    // call takes the current device's.
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = encode();
  }
  return r == CUDA_SUCCESS;
}

bool make_kv_tmap(CUtensorMap* map, const void* pool, int kv_dtype, long long rows, int head_dim,
                  int page_size, bool* whole_page) {
  const int esz = kv_dtype == SPG_I8 ? 1 : 2;
  if (kv_dtype != SPG_F16 && kv_dtype != SPG_BF16 && kv_dtype != SPG_I8) return false;
  if ((head_dim * esz) % 128 != 0 || page_size < 8 || page_size > 256) return false;
  if (rows < 1 || rows > 0x7fffffffLL) return false;  // int32 row coordinates
  if ((reinterpret_cast<uintptr_t>(pool) & 15u) != 0) return false;
  const CUtensorMapDataType dt = kv_dtype == SPG_F16    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                 : kv_dtype == SPG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const uint64_t row_bytes = static_cast<uint64_t>(head_dim) * esz;
  const uint32_t nt = static_cast<uint32_t>(row_bytes / 128);  // 128-byte slices of a row
  const uint32_t slice = 128u / static_cast<uint32_t>(esz);
  // Whole page in one copy: a 3-D view (x: the 128 bytes of a slice, y: rows,
  // z: slices), so that a box of [128 bytes][page_size rows][nt slices] lands
  // as nt tiles of [page_size rows][128 bytes], the same layout (and 128-byte
  // swizzle) as nt separate 2-D tile copies.
  {
    const uint64_t dims[3] = {slice, static_cast<uint64_t>(rows), nt}, strides[2] = {row_bytes, 128};
    const uint32_t box[3] = {slice, static_cast<uint32_t>(page_size), nt};
    if (encode_tmap(map, dt, 3, pool, dims, strides, box)) {
      *whole_page = true;
      return true;
    }
  }
  // else one 2-D tile of [page_size rows][128 bytes] per slice
  *whole_page = false;
  const uint64_t dims[2] = {static_cast<uint64_t>(head_dim), static_cast<uint64_t>(rows)};
  const uint32_t box[2] = {slice, static_cast<uint32_t>(page_size)};  // 128-byte rows
  return encode_tmap(map, dt, 2, pool, dims, &row_bytes, box);
}

bool make_q_tmap(CUtensorMap* map, const void* q, const spg_params& p, int total_q, int rows) {
  const uint64_t d = p.head_dim, G = p.num_q_heads / p.num_kv_heads, Hkv = p.num_kv_heads;
  const uint64_t dims[4] = {d, G, Hkv, static_cast<uint64_t>(total_q)};
  const uint64_t strides[3] = {d * 2, G * d * 2, Hkv * G * d * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(G), 1, static_cast<uint32_t>(rows / G)};
  return encode_tmap(map, p.q_dtype == SPG_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, q,
                     dims, strides, box);
}

}  // namespace spg
