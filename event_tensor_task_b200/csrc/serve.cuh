// serve.cuh — what the serving operators' kernels share: 16-bit element types,
// the paged cache's view, the status word and launches with attributes.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <string>

#include "device.cuh"
#include "serve.hpp"

namespace mk {

// two 16-bit elements <-> fp32
template <class T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};

__device__ __forceinline__ void report_bounds(int* status) {
  if (status) *status = MK_ERR_DEVICE_BOUNDS;
}

// The page that holds position t of sequence b, or -1 (reported) where the
// table names none or one outside the pool.
__device__ __forceinline__ int page_of(const mk_kv_pages& P, int b, int page_index, int* status) {
  int page = -1;
  if (page_index < P.table_width) page = __ldg(P.page_table + (long long)b * P.table_stride + page_index);
  if (page < 0 || page >= P.n_pages) {
    report_bounds(status);
    return -1;
  }
  return page;
}

// What a launch needs of the current device: its number and SM count (asked for once per device and process).
struct Device {
  int id = 0, sms = 0;
};
inline cudaError_t current_device(Device& d) {
  static std::atomic<int> sms[64];
  cudaError_t e = cudaGetDevice(&d.id);
  if (e != cudaSuccess) return e;
  const int slot = d.id & 63;
  d.sms = d.id < 64 ? sms[slot].load(std::memory_order_relaxed) : 0;
  if (d.sms == 0) {
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, d.id);
    if (e == cudaSuccess && d.id < 64) sms[slot].store(d.sms, std::memory_order_relaxed);
  }
  return e;
}

// A kernel's opt-in shared memory (and, where asked, clusters above 8 blocks), set once per device.
template <auto Kernel>
cudaError_t allow(const Device& d, int smem, bool large_clusters = false) {
  static std::atomic<unsigned long long> done{0};
  const unsigned long long bit = d.id < 64 ? 1ull << d.id : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && large_clusters) e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// A map of 16-bit elements [dims...] with element strides (of dimension 1 on), read in boxes of 64 x box under the
// 128-byte swizzle.  A dimension of one element has no stride of its own.
inline bool encode_map(CUtensorMap* map, int dtype, const void* p, int rank, const long long* dims, const long long* strides,
            const int* box) {
  EncodeTiledFn enc = encode_tiled();
  cuuint64_t d[4], st[3];
  cuuint32_t b[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    b[i] = (cuuint32_t)box[i];
    if (i) st[i - 1] = (cuuint64_t)(dims[i] == 1 ? dims[0] : strides[i - 1]) * 2;
  }
  return enc && enc(map, dtype == MK_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                    const_cast<void*>(p), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The maps of a pool's keys and values, read in boxes of 64 elements x `rows` rows of one (page, head): coordinates
// (element, row, head, page); what lies behind a page or the pool reads as zeros.
inline bool encode_pages(CUtensorMap* k, CUtensorMap* v, const mk_kv_pages& g, int rows) {
  const long long dims[4] = {g.head_dim, g.page_size, g.n_kv_heads, g.n_pages};
  const long long strides[3] = {g.row_stride, g.head_stride, g.page_stride};
  const int box[4] = {64, rows, 1, 1};
  return encode_map(k, g.dtype, g.k, 4, dims, strides, box) && encode_map(v, g.dtype, g.v, 4, dims, strides, box);
}

// Launches that may begin while the kernel before them on the stream still runs (programmatic dependent launch; a
// captured graph keeps it).  Such a kernel sets up what concerns nobody else, waits for what came before (dep_wait),
// and only then lets the next one begin (dep_launch): whatever runs early therefore finds all but the last kernel done.
// `early` is for calls that leave SMs idle, where the launch is a good part of the time (one row of logits 7.8 -> 5.5
// us a call, one sequence's decode 8.2 -> 7.0); behind a full device it costs more than it gives (32 sequences' decode
// 53 -> 63 us, eight packed prompts 202 -> 207).
template <class... P, class... A>
cudaError_t launch(bool early, void (*kernel)(P...), dim3 grid, int block, int smem, cudaStream_t s, int cluster, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  if (early) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 0) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = cluster;
    at[cfg.numAttrs].val.clusterDim.y = 1;
    at[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  cfg.attrs = at;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

inline mk_status cuda_result(cudaError_t e, const char* what, std::string& err) {
  if (e == cudaSuccess) return MK_OK;
  err = std::string(what) + ": " + cudaGetErrorString(e);
  return MK_ERR_CUDA;
}

}  // namespace mk
