// logits.cu — mk_process_logits: penalties for repeated tokens, biases and a
// grammar's mask on logits, and the choice of the largest.
//
// One row is the work of one thread-block cluster; each of its blocks takes a
// range of the vocabulary.  First a block marks in shared memory, 16 bits per
// id of its range, how often the id stands in the row's history (integer
// atomics, so their order does not matter) and whether the bias list names it;
// then it streams its logits once, the first of them loaded before the marks
// are made.  Ids with a bias, few, pass unchanged there and are seen to
// afterwards by the list's entries, each id by one of them; where the list
// names an id twice, its values add up in list order.  Nothing but logits,
// history, bias list and mask bits is read, and no count ever exists in device
// memory.  The blocks' best (value, id) keys meet in the first block through
// distributed shared memory: no workspace, no atomics on device memory, one
// launch.
//
// Bound: memory (logits in, logits out) for a batch; for a single row the
// latency of its dependent steps (lengths, history, logits, cluster barrier).
// Measured (one B200, inputs that change from call to call and are not in L2):
// 64 rows of 128,256 with 4,096 ids of history, 64 biases and a mask each in
// 26 us, 2.6 TB/s (20 on inputs that L2 holds).  Their stream alone takes 15
// (a copy of the logits 14), the history with it 18, the biases 17, the mask
// 21: the marks are made before the stream and hardly overlap it, and each
// batch waits for its mask words.  One row with 1,500 ids in 5.5 us.
#include <cooperative_groups.h>

#include <algorithm>

#include "serve.cuh"

namespace mk {
namespace {

namespace cg = cooperative_groups;

constexpr int kPer = 8;                  // ids a thread has in flight
constexpr int kThreads = 1024;
constexpr int kMarkBytes = 128 * 1024;   // marks of the ids that a block takes at a time
// The mark of an id (M: 16 bits, or 32 for a history above kShortHistory ids).
// Bit 0: it stands in the history; from bit 1: its occurrences in the answer;
// the two highest: the bias list names it, and more than once.
constexpr int kShortHistory = (1 << 13) - 1;
template <class M>
struct Mark {
  static constexpr int kBits = 8 * sizeof(M), kPerWord = 32 / kBits;
  static constexpr uint32_t kBias = 1u << (kBits - 2), kTwice = 1u << (kBits - 1), kCounts = kBias - 1;
  // the word that holds the mark of id `at`, and the mark's place in it
  static __device__ __forceinline__ int shift(unsigned at) { return sizeof(M) == 2 ? (at & 1) * 16 : 0; }
  static __device__ __forceinline__ uint32_t* word(uint32_t* marks, unsigned at) { return marks + at / kPerWord; }
  static __device__ __forceinline__ uint32_t get(const uint32_t* marks, unsigned at) { return reinterpret_cast<const M*>(marks)[at]; }
};

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
__device__ __noinline__ float sum_of_id(const mk_logits_args& a, int b0, int b1, int id) {
  float sum = 0.f;
#pragma unroll 2
  for (int i = b0 + (int)(threadIdx.x & 31); i - (int)(threadIdx.x & 31) < b1; i += 32) {
    const bool match = i < b1 && __ldg(a.bias_ids + i) == id;
    const float v = match ? __ldg(a.bias_values + i) : 0.f;
    for (unsigned m = __ballot_sync(~0u, match); m; m &= m - 1) sum += __shfl_sync(~0u, v, __ffs(m) - 1);
  }
  return sum;
}

template <class T, bool VEC, class M>
__global__ void __launch_bounds__(kThreads, 1) logits_kernel(const __grid_constant__ mk_logits_args a, int per_block, int tile) {
  using B = Batch<T, VEC>;
  using K = Mark<M>;
  constexpr int NT = kThreads;
  extern __shared__ __align__(16) uint32_t marks[];  // [tile] of M
  __shared__ unsigned long long best_key[NT / 32 + 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int row = blockIdx.y, tid = threadIdx.x;
  const T* src = static_cast<const T*>(a.logits) + row * a.logits_stride;
  float* dst = a.out ? a.out + row * a.out_stride : nullptr;
  const uint32_t* mask = a.mask ? a.mask + row * a.mask_stride : nullptr;
  const int block_lo = (int)min((long long)a.vocab, (long long)blockIdx.x * per_block);
  const int block_hi = (int)min((long long)a.vocab, (long long)block_lo + per_block);

  dep_wait();
  dep_launch();
  float x[kPer];
  B::load(x, src + block_lo, block_hi - block_lo);

  // the first ids of the history, before its length is known (a row holds history_width ids)
  const bool penalised = a.repetition || a.frequency || a.presence;
  const int* history = a.history + (a.history ? row * a.history_stride : 0);
  int id[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) id[e] = penalised && tid + e * NT < a.history_width ? __ldg(history + tid + e * NT) : -1;

  int len = 0, first = 0, b0 = 0, b1 = 0;
  float rep = 1.f, inv_rep = 1.f, freq = 0.f, pres = 0.f;
  if (penalised) {
    len = a.history_lens ? __ldg(a.history_lens + row) : a.history_width;
    first = a.prompt_lens ? __ldg(a.prompt_lens + row) : 0;
    if (a.repetition) rep = __ldg(a.repetition + row);
    if (a.frequency) freq = __ldg(a.frequency + row);
    if (a.presence) pres = __ldg(a.presence + row);
    inv_rep = 1.f / rep;
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

  // x after the penalties that a mark asks for
  auto penalise = [&](float v, uint32_t mark) {
    const uint32_t c = mark & K::kCounts;
    const float scaled = v > 0.f ? v * inv_rep : v * rep;
    v = c ? scaled : v;
    return c > 1 ? v - freq * (float)(c >> 1) - pres : v;
  };
  float best_value = -INFINITY;
  int best_id = -1;
  for (int lo = block_lo; lo < block_hi; lo += tile) {
    const int n = min(tile, block_hi - lo);
    if (lo != block_lo) B::load(x, src + lo, n);
    if (marked) {
      for (int i = tid; i < (n + 4 * K::kPerWord - 1) / (4 * K::kPerWord); i += NT) reinterpret_cast<uint4*>(marks)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      for (int i0 = tid; i0 < len; i0 += 4 * NT) {  // (4 loads in flight a thread)
        if (len > 4 * NT && (i0 != tid || lo != block_lo)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) id[e] = i0 + e * NT < len ? __ldg(history + i0 + e * NT) : -1;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const unsigned at = (unsigned)id[e] - (unsigned)lo;
          if (id[e] >= 0 && at < (unsigned)n && i0 + e * NT < len) {
            if (i0 + e * NT >= first) atomicAdd(K::word(marks, at), 2u << K::shift(at));
            else atomicOr(K::word(marks, at), 1u << K::shift(at));
          }
        }
      }
      for (int i = b0 + tid; i < b1; i += NT) {
        const int which = __ldg(a.bias_ids + i);
        const unsigned at = (unsigned)which - (unsigned)lo;
        if (which >= 0 && at < (unsigned)n) {
          const uint32_t old = atomicOr(K::word(marks, at), K::kBias << K::shift(at));
          if (old >> K::shift(at) & K::kBias) atomicOr(K::word(marks, at), K::kTwice << K::shift(at));
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
#pragma unroll
      for (int g = 0; g < kPer / 4; ++g) {
        uint32_t mark[4] = {0, 0, 0, 0}, allowed[4] = {1, 1, 1, 1};
        if (VEC) {  // (lo is a multiple of 128: four ids from a multiple of 4 share a mask word)
          const int at = B::at(4 * g);
          if (marked && at < left) {
            if constexpr (sizeof(M) == 4) {
              *reinterpret_cast<uint4*>(mark) = *reinterpret_cast<const uint4*>(marks + done + at);
            } else {
              const uint2 two = *reinterpret_cast<const uint2*>(marks + (done + at) / 2);
              mark[0] = two.x & 0xffff, mark[1] = two.x >> 16, mark[2] = two.y & 0xffff, mark[3] = two.y >> 16;
            }
          }
          if (mask) {
            const uint32_t word = at < left ? __ldg(mask + ((base + at) >> 5)) >> ((base + at) & 31) : 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) allowed[e] = word >> e & 1;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = B::at(4 * g + e);
            if (marked && at < left) mark[e] = K::get(marks, done + at);
            if (mask) allowed[e] = at < left ? __ldg(mask + ((base + at) >> 5)) >> ((base + at) & 31) & 1 : 0u;
          }
        }
        if (mark[0] | mark[1] | mark[2] | mark[3]) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(mark[e] & K::kBias)) y[4 * g + e] = penalise(y[4 * g + e], mark[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 4 * g + e, at = B::at(j);
          const bool later = mark[e] & K::kBias;
          if (!allowed[e] && !later) y[j] = -INFINITY;
          if (y[j] > best_value && !later && at < left) {  // (a thread's ids ascend: the lowest of equal ones stays; NaN and -inf never win)
            best_value = y[j];
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
    if (b1 > b0) {
      // ---- ids with a bias, each by the first entry that takes its mark off (whole warps come here)
      __syncthreads();  // (their values as they were are written by now)
      for (int i = b0 + tid; i - (tid & 31) < b1; i += NT) {
        const int which = i < b1 ? __ldg(a.bias_ids + i) : -1;
        const unsigned at = (unsigned)which - (unsigned)lo;
        uint32_t mark = 0;
        if (which >= 0 && at < (unsigned)n) mark = atomicAnd(K::word(marks, at), ~(K::kBias << K::shift(at))) >> K::shift(at);
        const bool mine = mark & K::kBias;
        float add = mine && !(mark & K::kTwice) ? __ldg(a.bias_values + i) : 0.f;
        for (unsigned need = __ballot_sync(~0u, mine && (mark & K::kTwice)); need; need &= need - 1) {
          const float sum = sum_of_id(a, b0, b1, __shfl_sync(~0u, which, __ffs(need) - 1));
          if ((tid & 31) == __ffs(need) - 1) add = sum;
        }
        if (!mine) continue;
        float v = penalise(to_f32(src[which]), mark) + add;
        if (mask && !(__ldg(mask + (which >> 5)) >> (which & 31) & 1)) v = -INFINITY;
        if (dst) dst[which] = v;
        if (v > best_value || (v == best_value && which < best_id)) {
          best_value = v;
          best_id = which;
        }
      }
    }
    if (marked && lo + tile < block_hi) __syncthreads();  // (the marks are cleared for the next tile)
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

template <class T, bool VEC, class M>
mk_status launch(const mk_logits_args& a, int cluster, const Device& dev, cudaStream_t s, std::string& err) {
  cudaError_t e = allow<logits_kernel<T, VEC, M>>(dev, kMarkBytes, true);
  if (e != cudaSuccess) return cuda_result(e, "mk_process_logits attributes", err);
  const int per_block = ((a.vocab - 1) / cluster + 128) / 128 * 128;
  const int tile = std::min<int>(per_block, kMarkBytes / sizeof(M));
  e = mk::launch(cluster * a.rows < dev.sms, logits_kernel<T, VEC, M>, dim3(cluster, a.rows), kThreads,
                 a.history || a.bias_indptr ? (int)(tile * sizeof(M)) : 0, s, cluster, a, per_block, tile);
  return cuda_result(e, "mk_process_logits launch", err);
}

// Blocks of a row (a cluster): one for each SM, as long as each has 2048 ids or more.  A cluster lies within one group
// of SMs: of 16 blocks hardly one fits a group, so 16 is for one to four rows.
template <class T, bool VEC>
mk_status size_up(const mk_logits_args& a, cudaStream_t s, std::string& err) {
  Device dev;
  cudaError_t e = current_device(dev);
  if (e != cudaSuccess) return cuda_result(e, "mk_process_logits device query", err);
  const int most = a.rows <= 4 ? 16 : 8;
  int cluster = 1;
  while (cluster < most && a.vocab > 2048 * cluster && (long long)a.rows * cluster * 2 <= dev.sms) cluster *= 2;
  if (a.history_width > kShortHistory) return launch<T, VEC, uint32_t>(a, cluster, dev, s, err);
  return launch<T, VEC, uint16_t>(a, cluster, dev, s, err);
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
