// logits.cu — mk_process_logits: penalties for repeated tokens, biases and a
// grammar's mask on logits, and the choice of the largest.
//
// One row is the work of one thread-block cluster; each of its blocks takes a
// range of the vocabulary.  First a block marks in shared memory, a word per id
// of its range, how often the id stands in the row's history (integer atomics,
// so their order does not matter) and whether the bias list names it; then it
// streams its logits once, the first of them loaded before the marks are made.
// Nothing but logits, history, bias list and mask bits is read, and no count
// ever exists in device memory.  A mark leads to its id's
// entry of the bias list; for an id that the list names twice the sum is taken
// from the list, in its order, by the thread that has the id.  The blocks' best (value, id) keys meet
// in the first block through distributed shared memory: no workspace, no
// atomics on device memory, one launch.
//
// Bound: memory (logits in, logits out) for a batch; for a single row the
// latency of its dependent steps (lengths, history, logits, cluster barrier).
#include <cooperative_groups.h>

#include <algorithm>

#include "serve.cuh"

namespace mk {
namespace {

namespace cg = cooperative_groups;

constexpr int kPer = 8;                  // ids a thread has in flight
constexpr int kThreads = 512;
constexpr int kMaxTile = 16384;          // ids marked at a time: 64 KB of marks, so that an SM holds two blocks
// The mark of an id.  Bit 0: it stands in the history; from bit 1: its
// occurrences in the answer; kBias: the bias list names it, kTwice: more than
// once.  The entry's place in the row's list lies in bits 14-29 as long as
// history and list are short enough for that, else (WIDE) in a second word.
constexpr uint32_t kBias = 1u << 30, kTwice = 1u << 31;
constexpr int kPlaceBit = 14, kShortHistory = (1 << 13) - 1, kShortList = 1 << 16;

template <class T>
__device__ __forceinline__ float to_f32(T v) { return static_cast<float>(v); }

// VEC: rows of logits and out start on 16 bytes (8 for 16-bit logits), so four
// ids go per access; else one id per access, neighbouring lanes on neighbouring ids.
// Element j of a thread is id VEC ? 4 * (tid + NT * (j / 4)) + j % 4 : tid + NT * j of its batch.
template <class T, bool VEC>
struct Batch {
  static constexpr int NT = kThreads, kIds = NT * kPer;
  static __device__ __forceinline__ int at(int j) { return VEC ? 4 * (threadIdx.x + NT * (j / 4)) + j % 4 : threadIdx.x + NT * j; }
  static __device__ __forceinline__ void load(float (&x)[kPer], const T* src, int n) {
#pragma unroll
    for (int j = 0; j < kPer; j += VEC ? 4 : 1) {
      if constexpr (VEC) {
        if (at(j) + 4 <= n) {
          if constexpr (sizeof(T) == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src + at(j));
            x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src + at(j));
            const float2 p = Elem<T>::unpack(v.x), q = Elem<T>::unpack(v.y);
            x[j] = p.x, x[j + 1] = p.y, x[j + 2] = q.x, x[j + 3] = q.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[j + e] = at(j) + e < n ? to_f32(src[at(j) + e]) : 0.f;
        }
      } else {
        x[j] = at(j) < n ? to_f32(src[at(j)]) : 0.f;
      }
    }
  }
};

// The row's bias values with this id, added in list order by a warp.
__device__ __forceinline__ float sum_of_id(const mk_logits_args& a, int b0, int b1, int id) {
  float sum = 0.f;
#pragma unroll 2
  for (int i = b0 + (int)(threadIdx.x & 31); i - (int)(threadIdx.x & 31) < b1; i += 32) {
    const bool match = i < b1 && __ldg(a.bias_ids + i) == id;
    const float v = match ? __ldg(a.bias_values + i) : 0.f;
    for (unsigned m = __ballot_sync(~0u, match); m; m &= m - 1) sum += __shfl_sync(~0u, v, __ffs(m) - 1);
  }
  return sum;
}

template <class T, bool VEC, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) logits_kernel(const __grid_constant__ mk_logits_args a, int per_block, int tile) {
  using B = Batch<T, VEC>;
  constexpr int NT = kThreads;
  constexpr uint32_t kCounts = WIDE ? kBias - 1 : (1u << kPlaceBit) - 1;
  extern __shared__ __align__(16) uint32_t marks[];  // [tile]
  uint32_t* const place = marks + tile;              // WIDE: [tile]
  __shared__ unsigned long long best_key[NT / 32 + 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int row = blockIdx.y, tid = threadIdx.x;
  const T* src = static_cast<const T*>(a.logits) + row * a.logits_stride;
  float* dst = a.out ? a.out + row * a.out_stride : nullptr;
  const uint32_t* mask = a.mask ? a.mask + row * a.mask_stride : nullptr;
  const int block_lo = (int)min((long long)a.vocab, (long long)blockIdx.x * per_block);
  const int block_hi = (int)min((long long)a.vocab, (long long)block_lo + per_block);

  float x[kPer];
  B::load(x, src + block_lo, block_hi - block_lo);

  // the first ids of the history, before its length is known (a row holds history_width ids)
  const bool penalised = a.repetition || a.frequency || a.presence;
  const int* history = a.history + (a.history ? row * a.history_stride : 0);
  int id[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) id[e] = penalised && tid + e * NT < a.history_width ? __ldg(history + tid + e * NT) : -1;

  int len = 0, first = 0, b0 = 0, b1 = 0;
  float rep = 1.f, freq = 0.f, pres = 0.f;
  if (penalised) {
    len = a.history_lens ? __ldg(a.history_lens + row) : a.history_width;
    first = a.prompt_lens ? __ldg(a.prompt_lens + row) : 0;
    if (a.repetition) rep = __ldg(a.repetition + row);
    if (a.frequency) freq = __ldg(a.frequency + row);
    if (a.presence) pres = __ldg(a.presence + row);
  }
  if (a.bias_indptr) {
    b0 = __ldg(a.bias_indptr + row);
    b1 = __ldg(a.bias_indptr + row + 1);
  }
  if (len < 0 || len > a.history_width) {
    if (tid == 0) report_bounds(a.status);
    len = len < 0 ? 0 : a.history_width;
  }
  if (b0 < 0 || b1 > a.bias_count || b0 > b1) {
    if (tid == 0) report_bounds(a.status);
    b0 = b1 = 0;
  }
  const bool marked = len > 0 || b1 > b0;

  float best_value = -INFINITY;
  int best_id = -1;
  for (int lo = block_lo; lo < block_hi; lo += tile) {
    const int n = min(tile, block_hi - lo);
    if (lo != block_lo) B::load(x, src + lo, n);
    if (marked) {
      if (lo != block_lo) __syncthreads();  // (the marks of the tile before are done with)
      for (int i = tid; i < (n + 3) / 4; i += NT) reinterpret_cast<uint4*>(marks)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      for (int i0 = tid; i0 < len; i0 += 8 * NT) {  // (8 loads in flight a thread)
        if (len > 8 * NT && (i0 != tid || lo != block_lo)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) id[e] = i0 + e * NT < len ? __ldg(history + i0 + e * NT) : -1;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const unsigned at = (unsigned)id[e] - (unsigned)lo;
          if (id[e] >= 0 && at < (unsigned)n && i0 + e * NT < len) {
            if (i0 + e * NT >= first) atomicAdd(marks + at, 2u);
            else atomicOr(marks + at, 1u);
          }
        }
      }
      for (int i = b0 + tid; i < b1; i += NT) {
        const int id = __ldg(a.bias_ids + i);
        const unsigned at = (unsigned)id - (unsigned)lo;
        if (id >= 0 && at < (unsigned)n) {
          if (WIDE) place[at] = i - b0;
          if (atomicOr(marks + at, WIDE ? kBias : kBias | (uint32_t)(i - b0) << kPlaceBit) & kBias) atomicOr(marks + at, kTwice);
        }
      }
      __syncthreads();
    }
    for (int done = 0; done < n; done += B::kIds) {
      const int left = n - done, base = lo + done;
      float y[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) y[j] = x[j];
      if (left > B::kIds) B::load(x, src + base + B::kIds, left - B::kIds);  // the next batch, while this one is worked on
      uint32_t allowed[VEC ? kPer / 4 : kPer];  // (lo is a multiple of 128: four ids from a multiple of 4 share a word)
      if (mask) {
#pragma unroll
        for (int j = 0; j < kPer; j += VEC ? 4 : 1) allowed[VEC ? j / 4 : j] = B::at(j) < left ? __ldg(mask + ((base + B::at(j)) >> 5)) : 0u;
      }
#pragma unroll
      for (int g = 0; g < kPer / 4; ++g) {
        uint32_t mark[4] = {0, 0, 0, 0};
        if (marked) {
          if (VEC) {  // (one 16-byte read: four ids in a row a lane, no bank twice)
            if (B::at(4 * g) < left) *reinterpret_cast<uint4*>(mark) = *reinterpret_cast<const uint4*>(marks + done + B::at(4 * g));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) mark[e] = B::at(4 * g + e) < left ? marks[done + B::at(4 * g + e)] : 0u;
          }
        }
        float twice[4] = {0.f, 0.f, 0.f, 0.f};
        if (__any_sync(~0u, (mark[0] | mark[1] | mark[2] | mark[3]) & kTwice)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int mine = base + B::at(4 * g + e);
            for (unsigned need = __ballot_sync(~0u, mark[e] & kTwice); need; need &= need - 1) {
              const float sum = sum_of_id(a, b0, b1, __shfl_sync(~0u, mine, __ffs(need) - 1));
              if ((tid & 31) == __ffs(need) - 1) twice[e] = sum;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 4 * g + e, at = B::at(j);
          float v = y[j];
          if (mark[e]) {
            const uint32_t c = mark[e] & kCounts;
            if (c) {
              if (a.repetition) v = v > 0.f ? v / rep : v * rep;
              if (c > 1) v = v - freq * (float)(c >> 1) - pres;
            }
            if (mark[e] & kTwice) {
              v += twice[e];
            } else if (mark[e] & kBias) {
              v += __ldg(a.bias_values + b0 + (WIDE ? place[done + at] : mark[e] >> kPlaceBit & (kShortList - 1)));
            }
          }
          if (mask && !(allowed[VEC ? g : j] >> ((base + at) & 31) & 1)) v = -INFINITY;
          y[j] = v;
          if (v > best_value && at < left) {  // (a thread's ids ascend: the lowest of equal ones stays; NaN and -inf never win)
            best_value = v;
            best_id = base + at;
          }
        }
      }
      if (dst) {
#pragma unroll
        for (int j = 0; j < kPer; j += VEC ? 4 : 1) {
          float* out = dst + base + B::at(j);
          if (VEC && B::at(j) + 4 <= left) *reinterpret_cast<float4*>(out) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
          else {
#pragma unroll
            for (int e = 0; e < (VEC ? 4 : 1); ++e)
              if (B::at(j + e) < left) out[e] = y[j + e];
          }
        }
      }
    }
  }
  if (!a.next_tokens) return;
  unsigned long long best = best_id >= 0 ? argmax_key(best_value + 0.f, best_id) : 0;  // (-0 ties with 0)
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const unsigned long long other = __shfl_xor_sync(~0u, best, d);
    best = other > best ? other : best;
  }
  if ((tid & 31) == 0) best_key[tid >> 5] = best;
  __syncthreads();
  if (tid < 32) {
    best = tid < NT / 32 ? best_key[tid] : 0;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const unsigned long long other = __shfl_xor_sync(~0u, best, d);
      best = other > best ? other : best;
    }
    if (tid == 0) best_key[NT / 32] = best;
  }
  cluster.sync();
  if (cluster.block_rank() == 0 && tid < 32) {
    best = tid < (int)cluster.num_blocks() ? *cluster.map_shared_rank(best_key + NT / 32, tid) : 0;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const unsigned long long other = __shfl_xor_sync(~0u, best, d);
      best = other > best ? other : best;
    }
    if (tid == 0) a.next_tokens[row] = best ? argmax_key_index(best) : -1;
  }
  cluster.sync();  // no block leaves while its key may still be read
}

template <class T, bool VEC, bool WIDE>
mk_status launch(const mk_logits_args& a, int cluster, const Device& dev, cudaStream_t s, std::string& err) {
  cudaError_t e = allow<logits_kernel<T, VEC, WIDE>>(dev, kMaxTile * 8, true);
  if (e != cudaSuccess) return cuda_result(e, "mk_process_logits attributes", err);
  const int per_block = ((a.vocab - 1) / cluster + 128) / 128 * 128;
  const int tile = std::min(per_block, kMaxTile);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster, a.rows);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = a.history || a.bias_indptr ? tile * (WIDE ? 8 : 4) : 0;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_result(cudaLaunchKernelEx(&cfg, logits_kernel<T, VEC, WIDE>, a, per_block, tile), "mk_process_logits launch", err);
}

// Blocks of a row (a cluster): enough for two on each SM, as long as each has 2048 ids or more.  A cluster lies within
// one group of SMs: of 16 blocks hardly one fits a group, so 16 is for one to four rows.
template <class T, bool VEC>
mk_status size_up(const mk_logits_args& a, cudaStream_t s, std::string& err) {
  Device dev;
  cudaError_t e = current_device(dev);
  if (e != cudaSuccess) return cuda_result(e, "mk_process_logits device query", err);
  const int most = a.rows <= 4 ? 16 : 8;
  int cluster = 1;
  while (cluster < most && a.vocab > 2048 * cluster && (long long)a.rows * cluster * 2 < dev.sms * 3) cluster *= 2;
  if (a.history_width > kShortHistory || a.bias_count > kShortList) return launch<T, VEC, true>(a, cluster, dev, s, err);
  return launch<T, VEC, false>(a, cluster, dev, s, err);
}

template <class T>
mk_status pick(const mk_logits_args& a, cudaStream_t s, std::string& err) {
  const uintptr_t in = reinterpret_cast<uintptr_t>(a.logits), out = reinterpret_cast<uintptr_t>(a.out);
  const bool vec = in % (4 * sizeof(T)) == 0 && out % 16 == 0 && (a.rows == 1 || (a.logits_stride % 4 == 0 && (!a.out || a.out_stride % 4 == 0)));
  return vec ? size_up<T, true>(a, s, err) : size_up<T, false>(a, s, err);
}

}  // namespace

mk_status launch_logits(const mk_logits_args& a, void* stream, std::string& err) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.dtype == MK_DTYPE_FP32) return pick<float>(a, s, err);
  return a.dtype == MK_DTYPE_BF16 ? pick<__nv_bfloat16>(a, s, err) : pick<__half>(a, s, err);
}

}  // namespace mk
