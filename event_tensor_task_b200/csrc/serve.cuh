// serve.cuh — what the serving operators' kernels share: 16-bit element types,
// the paged cache's view, the status word and launches with attributes.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

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

inline mk_status cuda_result(cudaError_t e, const char* what, std::string& err) {
  if (e == cudaSuccess) return MK_OK;
  err = std::string(what) + ": " + cudaGetErrorString(e);
  return MK_ERR_CUDA;
}

}  // namespace mk
