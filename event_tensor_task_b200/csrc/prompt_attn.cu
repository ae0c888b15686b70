// prompt_attn.cu — mk_prompt_attention: attention of packed prompts over packed
// or paged keys.
//
// A warp per (query row, head): its lanes hold the row's dimensions, the keys
// pass one after the other with a running maximum and sum.  Right for every
// case; bound by its instructions (a warp reduction per key).
#include <cmath>

#include "serve.cuh"

namespace mk {
namespace {

constexpr int kWarps = 8;

struct PromptParams {
  mk_prompt_args a;
  float scale_log2;
};

template <class T, int D>
__global__ void __launch_bounds__(kWarps * 32) prompt_kernel(const __grid_constant__ PromptParams P) {
  constexpr int E = D / 32;
  const mk_prompt_args& a = P.a;
  const mk_kv_pages& g = a.pages;
  const int lane = threadIdx.x & 31, head = blockIdx.y;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.n_tokens) return;
  int b = 0;
  for (int i = lane; i < a.batch; i += 32) b += __ldg(a.cu_q + i + 1) <= t;
  b = __reduce_add_sync(~0u, b);
  if (b >= a.batch) return;
  int q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
  if (q0 > t) return;
  if (q0 < 0 || q1 > a.n_tokens) {
    report_bounds(a.status);
    q0 = max(q0, 0);
    q1 = min(q1, a.n_tokens);
  }
  int k0 = 0, m;
  if (g.page_table) {
    const int cap = g.table_width * g.page_size;
    m = __ldg(a.kv_lens + b);
    if (m < 0 || m > cap) {
      report_bounds(a.status);
      m = m < 0 ? 0 : cap;
    }
  } else {
    k0 = __ldg(a.cu_k + b);
    int k1 = __ldg(a.cu_k + b + 1);
    if (k0 < 0 || k1 > g.page_size || k1 < k0) {
      report_bounds(a.status);
      k0 = min(max(k0, 0), g.page_size);
      k1 = max(min(k1, g.page_size), k0);
    }
    m = k1 - k0;
  }
  const int seen = a.causal ? min(m, max(0, t - q0 + 1 + m - (q1 - q0))) : m;
  const int kvh = head / (a.n_q_heads / g.n_kv_heads);
  float q[E], o[E] = {};
#pragma unroll
  for (int e = 0; e < E; ++e)
    q[e] = static_cast<float>(static_cast<const T*>(a.q)[t * a.q_row_stride + head * a.q_head_stride + lane * E + e]) * P.scale_log2;
  float top = -INFINITY, sum = 0.f;
  for (int j = 0; j < seen; ++j) {
    long long off = (long long)(k0 + j) * g.row_stride;
    bool live = true;
    if (g.page_table) {
      const int page = page_of(g, b, j / g.page_size, a.status);
      live = page >= 0;
      off = live ? page * g.page_stride + (long long)(j % g.page_size) * g.row_stride : 0;
    }
    off += kvh * g.head_stride + lane * E;
    float s = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      s += live ? q[e] * static_cast<float>(static_cast<const T*>(g.k)[off + e]) : 0.f;
      v[e] = live ? static_cast<float>(static_cast<const T*>(g.v)[off + e]) : 0.f;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    const float up = fmaxf(top, s), f = exp2f(top - up), p = exp2f(s - up);
    sum = sum * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * v[e];
    top = up;
  }
  const float inv = seen > 0 ? 1.f / sum : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    static_cast<T*>(a.out)[t * a.o_row_stride + head * a.o_head_stride + lane * E + e] = static_cast<T>(o[e] * inv);
}

}  // namespace

mk_status launch_prompt(const mk_prompt_args& a, void* stream, std::string& err) {
  PromptParams P;
  P.a = a;
  const int D = a.pages.head_dim;
  P.scale_log2 = (a.scale > 0.f ? a.scale : 1.f / std::sqrt((float)D)) * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((a.n_tokens + kWarps - 1) / kWarps, a.n_q_heads);
  if (a.pages.dtype == MK_DTYPE_BF16) {
    if (D == 64) prompt_kernel<__nv_bfloat16, 64><<<grid, kWarps * 32, 0, s>>>(P);
    else prompt_kernel<__nv_bfloat16, 128><<<grid, kWarps * 32, 0, s>>>(P);
  } else {
    if (D == 64) prompt_kernel<__half, 64><<<grid, kWarps * 32, 0, s>>>(P);
    else prompt_kernel<__half, 128><<<grid, kWarps * 32, 0, s>>>(P);
  }
  return cuda_result(cudaGetLastError(), "mk_prompt_attention launch", err);
}

}  // namespace mk
