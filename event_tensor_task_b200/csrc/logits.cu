// logits.cu — mk_process_logits: penalties for repeated tokens, biases and a
// grammar's mask on logits, and the choice of the largest.
//
// One row is the work of one thread-block cluster; each of its blocks takes a
// range of the vocabulary in tiles of kTile ids.  For a tile a block counts in
// shared memory how often each of its ids stands in the row's history (integer
// atomics, so their order does not matter) and adds the row's biases up there
// in list order, then makes one pass over the tile's logits, which it had
// loaded into registers beforehand.  Nothing but logits, history, bias list
// and mask bits is read, and no count ever exists in device memory.  The
// blocks' best (value, id) keys meet in the first block through distributed
// shared memory: no workspace, no atomics on device memory, one launch.
//
// Bound: memory (logits in, logits out) for a batch; for a single row the
// latency of its dependent steps (history, logits, cluster barrier).
#include <cooperative_groups.h>

#include "serve.cuh"

namespace mk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kPer = 16;                 // ids a thread holds of a tile
constexpr int kTile = kThreads * kPer;   // 8192 ids: 32 KB of counts, 32 KB of biases
constexpr int kMaxCluster = 16;

template <class T>
__device__ __forceinline__ float to_f32(T v) { return static_cast<float>(v); }

// VEC: rows of logits and out start on 16 bytes (8 for 16-bit logits), so four
// ids go per access; else one id per access, neighbouring lanes on neighbouring ids.
template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ mk_logits_args a, int per_block) {
  extern __shared__ uint32_t dyn[];
  uint32_t* count = dyn;                                     // [kTile]: answer occurrences * 2 + stands in the history
  float* bias = reinterpret_cast<float*>(dyn + kTile);       // [kTile], present only with a bias list
  __shared__ unsigned long long best_key[kThreads / 32 + 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int row = blockIdx.y, tid = threadIdx.x;
  const T* src = static_cast<const T*>(a.logits) + row * a.logits_stride;
  float* dst = a.out ? a.out + row * a.out_stride : nullptr;
  const uint32_t* mask = a.mask ? a.mask + row * a.mask_stride : nullptr;

  int len = 0, first = 0;
  float rep = 1.f, freq = 0.f, pres = 0.f;
  if (a.history) {
    len = a.history_lens ? __ldg(a.history_lens + row) : a.history_width;
    if (len < 0 || len > a.history_width) {
      if (tid == 0) report_bounds(a.status);
      len = len < 0 ? 0 : a.history_width;
    }
    first = a.prompt_lens ? __ldg(a.prompt_lens + row) : 0;
    if (a.repetition) rep = __ldg(a.repetition + row);
    if (a.frequency) freq = __ldg(a.frequency + row);
    if (a.presence) pres = __ldg(a.presence + row);
  }
  int b0 = 0, b1 = 0;
  if (a.bias_indptr) {
    b0 = __ldg(a.bias_indptr + row);
    b1 = __ldg(a.bias_indptr + row + 1);
    if (b0 < 0 || b1 > a.bias_count || b0 > b1) {
      if (tid == 0) report_bounds(a.status);
      b0 = b1 = 0;
    }
  }
  const bool counted = len > 0 && (a.repetition || a.frequency || a.presence);
  const int* history = a.history + (a.history ? row * a.history_stride : 0);

  unsigned long long best = 0;
  const int block_lo = min((long long)a.vocab, (long long)blockIdx.x * per_block);
  const int block_hi = min((long long)a.vocab, (long long)block_lo + per_block);
  for (int lo = block_lo; lo < block_hi; lo += kTile) {
    const int n = min(kTile, block_hi - lo);
    // id of element j of this thread: VEC 4 * (tid + kThreads * (j / 4)) + j % 4, else tid + kThreads * j
    float x[kPer];
    if (VEC) {
#pragma unroll
      for (int g = 0; g < kPer / 4; ++g) {
        const int at = 4 * (tid + kThreads * g);
        if (at + 4 <= n) {
          if constexpr (sizeof(T) == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src + lo + at);
            x[4 * g] = v.x, x[4 * g + 1] = v.y, x[4 * g + 2] = v.z, x[4 * g + 3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src + lo + at);
            const float2 p = Elem<T>::unpack(v.x), q = Elem<T>::unpack(v.y);
            x[4 * g] = p.x, x[4 * g + 1] = p.y, x[4 * g + 2] = q.x, x[4 * g + 3] = q.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * g + e] = at + e < n ? to_f32(src[lo + at + e]) : 0.f;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int at = tid + kThreads * j;
        x[j] = at < n ? to_f32(src[lo + at]) : 0.f;
      }
    }
    if (counted) {
      for (int i = tid; i < n; i += kThreads) count[i] = 0;
    }
    if (b1 > b0) {
      for (int i = tid; i < n; i += kThreads) bias[i] = 0.f;
    }
    if (counted || b1 > b0) __syncthreads();
    if (counted) {
      for (int i = tid; i < len; i += kThreads) {
        const unsigned at = (unsigned)__ldg(history + i) - (unsigned)lo;  // (a negative id wraps past every tile)
        if (at < (unsigned)n) {
          if (i >= first) atomicAdd(count + at, 2u);
          else atomicOr(count + at, 1u);
        }
      }
    }
    if (b1 > b0 && tid < 32) {
      // one warp, 32 entries at a time in list order: the first lane of each id adds its group's values in lane order
      for (int i = b0; i < b1; i += 32) {
        const bool live = i + tid < b1;
        const int id = live ? __ldg(a.bias_ids + i + tid) : -1;
        const float v = live ? __ldg(a.bias_values + i + tid) : 0.f;
        const unsigned at = (unsigned)id - (unsigned)lo;
        const bool here = at < (unsigned)n;
        const unsigned same = __match_any_sync(~0u, here ? (int)at : -1);
        const bool lead = here && (__ffs(same) - 1) == tid;
        float sum = lead ? bias[at] : 0.f;
        for (int l = 0; l < 32; ++l) {
          const float other = __shfl_sync(~0u, v, l);
          if (lead && (same >> l & 1)) sum += other;
        }
        if (lead) bias[at] = sum;
        __syncwarp();
      }
    }
    if (counted || b1 > b0) __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int at = VEC ? 4 * (tid + kThreads * (j / 4)) + j % 4 : tid + kThreads * j;
      if (at >= n) continue;
      float v = x[j];
      if (counted) {
        const uint32_t c = count[at];
        if (c) {
          const float s = (float)(c >> 1);
          if (a.repetition) v = v > 0.f ? v / rep : v * rep;
          if (c > 1) v = v - freq * s - pres;
        }
      }
      if (b1 > b0) v += bias[at];
      if (mask && !(__ldg(mask + ((lo + at) >> 5)) >> ((lo + at) & 31) & 1)) v = -INFINITY;
      x[j] = v;
      if (v > -INFINITY) {
        const unsigned long long key = argmax_key(v + 0.f, lo + at);  // (-0 ties with 0)
        best = key > best ? key : best;
      }
    }
    if (dst) {
      if (VEC) {
#pragma unroll
        for (int g = 0; g < kPer / 4; ++g) {
          const int at = 4 * (tid + kThreads * g);
          if (at + 4 <= n) *reinterpret_cast<float4*>(dst + lo + at) = make_float4(x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]);
          else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (at + e < n) dst[lo + at + e] = x[4 * g + e];
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int at = tid + kThreads * j;
          if (at < n) dst[lo + at] = x[j];
        }
      }
    }
    if (lo + kTile < block_hi && (counted || b1 > b0)) __syncthreads();  // the counts are cleared for the next tile
  }
  if (!a.next_tokens) return;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const unsigned long long other = __shfl_xor_sync(~0u, best, d);
    best = other > best ? other : best;
  }
  if ((tid & 31) == 0) best_key[tid >> 5] = best;
  __syncthreads();
  if (tid < 32) {
    best = tid < kThreads / 32 ? best_key[tid] : 0;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const unsigned long long other = __shfl_xor_sync(~0u, best, d);
      best = other > best ? other : best;
    }
    if (tid == 0) best_key[kThreads / 32] = best;
  }
  cluster.sync();
  if (cluster.block_rank() == 0 && tid < 32) {
    best = tid < (int)cluster.num_blocks() ? *cluster.map_shared_rank(best_key + kThreads / 32, tid) : 0;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const unsigned long long other = __shfl_xor_sync(~0u, best, d);
      best = other > best ? other : best;
    }
    if (tid == 0) a.next_tokens[row] = best ? argmax_key_index(best) : -1;
  }
  cluster.sync();  // no block leaves while its key may still be read
}

template <class T, bool VEC>
mk_status launch(const mk_logits_args& a, cudaStream_t s, std::string& err) {
  const int smem = kTile * (a.bias_indptr ? 8 : 4);
  Device dev;
  cudaError_t e = current_device(dev);
  if (e == cudaSuccess) e = allow<logits_kernel<T, VEC>>(dev, kTile * 8, true);
  if (e != cudaSuccess) return cuda_result(e, "mk_process_logits attributes", err);
  int cluster = 1;
  while (cluster < kMaxCluster && (a.vocab + cluster - 1) / cluster > 2048 && a.rows * cluster < 512) cluster *= 2;
  const int per_block = ((a.vocab + cluster - 1) / cluster + 127) / 128 * 128;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster, a.rows);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_result(cudaLaunchKernelEx(&cfg, logits_kernel<T, VEC>, a, per_block), "mk_process_logits launch", err);
}

template <class T>
mk_status pick(const mk_logits_args& a, cudaStream_t s, std::string& err) {
  const uintptr_t in = reinterpret_cast<uintptr_t>(a.logits), out = reinterpret_cast<uintptr_t>(a.out);
  const bool vec = in % (4 * sizeof(T)) == 0 && out % 16 == 0 && (a.rows == 1 || (a.logits_stride % 4 == 0 && (!a.out || a.out_stride % 4 == 0)));
  return vec ? launch<T, true>(a, s, err) : launch<T, false>(a, s, err);
}

}  // namespace

mk_status launch_logits(const mk_logits_args& a, void* stream, std::string& err) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.dtype == MK_DTYPE_FP32) return pick<float>(a, s, err);
  return a.dtype == MK_DTYPE_BF16 ? pick<__nv_bfloat16>(a, s, err) : pick<__half>(a, s, err);
}

}  // namespace mk
