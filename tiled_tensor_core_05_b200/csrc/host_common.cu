// Host-side helpers shared by the libraries (linked into each of them):
// per-device state, driver entry points, pointer checks, TMA tensor-map
// encoding and the programmatic-launch attribute.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstdlib>
#include <mutex>

#include "../../include/gemm_f16.h"
#include "extent.h"
#include "internal.h"

namespace ttc {

// One status word per device (first device-side error wins; 0 = none).
__device__ int g_device_status;

namespace {

constexpr uint64_t kDefaultTimeoutNs = 1000ull * 1000ull * 1000ull;  // 1 s per wait
constexpr int kMaxDevices = 64;

struct DeviceEntry {
  bool ready = false;
  bool supported = false;
  int sm_count = 0;
  int* status = nullptr;
};

std::mutex g_devices_mutex;
DeviceEntry g_devices[kMaxDevices];

// ------------------------------------------------------ driver entry points ---
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
typedef CUresult (*AddressRangeFn)(CUdeviceptr*, size_t*, CUdeviceptr);
typedef CUresult (*PointerAttrsFn)(unsigned int, CUpointer_attribute*, void**, CUdeviceptr);

EncodeTiledFn g_encode = nullptr;
AddressRangeFn g_addr_range = nullptr;
PointerAttrsFn g_ptr_attrs = nullptr;
std::once_flag g_entry_once;

// Device memory of the current device (or managed memory) only.
bool is_device_pointer(const void* p, int device) {
  cudaPointerAttributes attr;
  if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
    cudaGetLastError();  // clear the sticky-free error state of this query
    return false;
  }
  if (attr.type == cudaMemoryTypeManaged) return true;
  return attr.type == cudaMemoryTypeDevice && attr.device == device;
}

// The bytes [p, p + span) lie in one allocation.
bool extent_in_allocation(const void* p, uint64_t span) {
  if (g_addr_range == nullptr) return true;  // cannot check; TMA bounds still apply
  CUdeviceptr base = 0;
  size_t size = 0;
  if (g_addr_range(&base, &size, reinterpret_cast<CUdeviceptr>(p)) != CUDA_SUCCESS) return false;
  return span_inside(reinterpret_cast<uint64_t>(p), span, base, size);
}

}  // namespace

void load_entry_points() {
  std::call_once(g_entry_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_addr_range = reinterpret_cast<AddressRangeFn>(fn);
    fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuPointerGetAttributes", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_ptr_attrs = reinterpret_cast<PointerAttrsFn>(fn);
  });
}

// ------------------------------------------------------------ device state ---
int get_device(DeviceCtx* ctx) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return runtime_error();
  if (dev < 0 || dev >= kMaxDevices) return GEMM_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lock(g_devices_mutex);
  DeviceEntry& e = g_devices[dev];
  if (!e.ready) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return runtime_error();
    e.supported = (major == 10 && minor == 0);
    e.sm_count = sms;
    if (e.supported) {
      // The symbol's device address for this device (host code cannot use the
      // symbol itself as a pointer).
      void* p = nullptr;
      if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return runtime_error();
      e.status = static_cast<int*>(p);
    }
    e.ready = true;
  }
  if (!e.supported) return GEMM_ERR_UNSUPPORTED_DEVICE;
  ctx->device = dev;
  ctx->sm_count = e.sm_count;
  ctx->status = e.status;
  ctx->timeout_ns = kDefaultTimeoutNs;
  return GEMM_OK;
}

// One driver query for memory type, owning device and allocation range.
// Returns -1 when the query itself is unavailable (caller falls back).
int query_pointer(const void* p, int device, uint64_t span) {
  if (g_ptr_attrs == nullptr) return -1;
  unsigned int mem_type = 0;
  int ordinal = -1;
  unsigned int managed = 0;
  CUdeviceptr base = 0;
  size_t size = 0;
  CUpointer_attribute attrs[5] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE,
                                  CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL,
                                  CU_POINTER_ATTRIBUTE_IS_MANAGED,
                                  CU_POINTER_ATTRIBUTE_RANGE_START_ADDR,
                                  CU_POINTER_ATTRIBUTE_RANGE_SIZE};
  void* data[5] = {&mem_type, &ordinal, &managed, &base, &size};
  if (g_ptr_attrs(5, attrs, data, reinterpret_cast<CUdeviceptr>(p)) != CUDA_SUCCESS) return 0;
  const bool on_device = (mem_type == CU_MEMORYTYPE_DEVICE && ordinal == device) || managed != 0;
  if (!on_device || size == 0) return 0;
  return span_inside(reinterpret_cast<uint64_t>(p), span, base, size) ? 1 : 0;
}

int check_device_range(const void* p, int device, uint64_t span) {
  const int q = query_pointer(p, device, span);
  if (q == 0) return GEMM_ERR_INVALID_ARG;
  if (q < 0 && (!is_device_pointer(p, device) || !extent_in_allocation(p, span)))
    return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

int encode_tmap_f16_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer,
                       uint64_t ld, uint32_t box_inner, uint32_t box_outer) {
  load_entry_points();
  if (g_encode == nullptr) return GEMM_ERR_LAUNCH;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {ld * 2u};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estrides[2] = {1, 1};
  // (L2 promotion none / 128 B / 256 B measured alike on the pair kernels:
  // the same DRAM bytes and time)
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base),
                              dims, strides, box, estrides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

int encode_tmap_u8_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer,
                      uint64_t ld, uint32_t box_outer) {
  load_entry_points();
  if (g_encode == nullptr) return GEMM_ERR_LAUNCH;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {ld};
  const cuuint32_t box[2] = {128, box_outer};
  const cuuint32_t estrides[2] = {1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                              strides, box, estrides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

int encode_tmap_scales(CUtensorMap* map, const void* base, uint64_t tiles, uint32_t box_tiles) {
  load_entry_points();
  if (g_encode == nullptr) return GEMM_ERR_LAUNCH;
  const cuuint64_t dims[2] = {128, tiles};
  const cuuint64_t strides[1] = {512};
  const cuuint32_t box[2] = {128, box_tiles};
  const cuuint32_t estrides[2] = {1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, const_cast<void*>(base), dims,
                              strides, box, estrides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

int encode_tmap_rows(CUtensorMap* map, const void* base, int bytes, uint64_t inner, uint64_t outer,
                     uint64_t ld, uint32_t box_inner, uint32_t box_outer) {
  load_entry_points();
  if (g_encode == nullptr) return GEMM_ERR_LAUNCH;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {ld * static_cast<unsigned>(bytes)};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estrides[2] = {1, 1};
  const CUresult r = g_encode(
      map, bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
      const_cast<void*>(base), dims, strides, box, estrides, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

bool pdl_enabled() {
  static const bool on = [] {
    const char* s = std::getenv("TTC_PDL");
    return !(s != nullptr && s[0] == '0');
  }();
  return on;
}

int pdl_attribute(cudaLaunchAttribute* attr) {
  if (!pdl_enabled()) return 0;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  return 1;
}

}  // namespace ttc
