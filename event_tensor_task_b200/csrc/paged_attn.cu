// paged_attn.cu — mk_paged_attention: attention of one new token per sequence
// over its cached keys, in pages.
//
// Mathematics: out = sum_j p_j v_j / sum_j p_j with p_j = 2^(c (q.k_j) - m),
// c = scale log2 e, m a running maximum: one pass over keys and values, parts
// with their own (m, l = sum p, O = sum p v) joined exactly as in the loop.
//
// Bound: memory; every cached row is read once, G = n_q_heads / n_kv_heads
// query heads share it.  So:
//  - the keys of all (sequence, kv head) pairs are laid end to end in units of
//    64 and cut into equal shares, one per resident block, whatever the
//    sequences' lengths; a block's share begins and ends inside a pair, so it
//    leaves at most two partial results, and a second kernel joins them;
//  - a warp owns 16 keys of each unit and runs alone: its own ring of stages
//    in shared memory (TMA boxes of 16 rows out of the pages, or rows gathered
//    by cp.async where pages are no multiple of 16 rows), its own running
//    maximum, sum and output in registers; the block's four warps meet only
//    where a pair ends;
//  - the products are warp MMAs (m16n8k16, the group's heads as rows): at most
//    16 rows make a tile too small for tcgen05, whose M is 64 or more, and the
//    tensor pipe is nearly idle either way.  With G <= 8 the spare rows carry
//    what rounding takes off the probabilities (value and remainder), above 8
//    the remainders take a second MMA: the sum sees ~16 bits of p.
// Measured (one B200, calls one after the other on inputs that are not in L2):
// 475 MB of keys and values in 90 us, 5.3 TB/s (the first kernel alone, under
// the profiler, 85); 286 MB of 32 sequences in 57 us; one sequence of 1,025
// keys, 32/8 heads, in 7 us.  About 8 us of a call are launch, search, the
// first round trips and the join, whatever its size.
#include <algorithm>
#include <cmath>

#include "serve.cuh"
#include "waits.hpp"

namespace mk {
namespace {

constexpr int kThreads = 128, kWarps = 4;
constexpr int kKeys = 16;               // keys of a warp's piece of a unit
constexpr int kUnit = kKeys * kWarps;   // keys of a unit
constexpr int kRows = 16;               // query heads of a tile
constexpr unsigned long long kWaitNs = 2000000000ull;  // limit of a wait
constexpr int kMaxCtas = 640;           // the workspace holds two partials of each

// FULL: 9 to 16 heads in a tile (both halves of the MMA's rows are heads)
template <int D, bool FULL>
struct Shape {
  static constexpr int kPiece = kKeys * D * 2 * 2;  // bytes of a warp's keys and values
  // D = 128: three blocks of two stages rather than two of three (32 ragged sequences 57 -> 53 us, 200 short ones
  // 55 -> 46 us, one long cache 84 -> 85 us), where the registers allow three
  static constexpr int kStages = D == 64 ? 4 : FULL ? 3 : 2;
  static constexpr int kBlocksPerSm = D == 64 || !FULL ? 3 : 2;
  static constexpr int kMerge = kRows * D * 4;       // two half output tiles in fp32
  static constexpr int kSmem = kWarps * kStages * kPiece + kMerge + 1024;
};
template <int D>
constexpr int kPartial = 2 * kRows + kRows * D;  // floats of a partial result: m, l, O

struct PagedParams {
  CUtensorMap tk, tv;  // (page_size a multiple of 16)
  mk_paged_attn_args a;
  float scale_log2;
  int group, tiles;    // G; tiles of 16 heads per kv head
  int n_cta;
  int by_pair;         // how the join's blocks are laid out
  float* partial;      // [n_cta][2][kPartial<D>]
};

template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 bytes global -> shared, zeros where !live
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// a warp that waits for a phase of an mbarrier (wait_together)
struct Landing {
  uint64_t* bar;
  uint32_t parity;
  __device__ __forceinline__ bool there() const { return mbar_try(bar, parity); }
  __device__ __forceinline__ bool all(bool p) const { return __all_sync(~0u, p); }
  __device__ __forceinline__ bool any(bool p) const { return __any_sync(~0u, p); }
  __device__ __forceinline__ unsigned long long now() const { return global_ns(); }
};

// keys of sequence b that are there to see
__device__ __forceinline__ int keys_of(const mk_paged_attn_args& a, int b) {
  const int n = __ldg(a.kv_lens + b), cap = a.pages.table_width * a.pages.page_size;
  if (n < 0 || n > cap) {
    report_bounds(a.status);
    return n < 0 ? 0 : cap;
  }
  return n;
}

// The units of all sequences end to end (below 2^31: the launch sees to that).
// Called by a whole block of NT threads, each of which counts `per` sequences;
// `scratch` receives the units before each thread's, and the total last.
template <int NT>
__device__ __forceinline__ int scan_units(const PagedParams& P, int* scratch, int& per) {
  const int B = P.a.batch, pairs = P.a.pages.n_kv_heads * P.tiles;
  per = (B + NT - 1) / NT;
  int mine = 0;
  for (int b = threadIdx.x * per; b < min(B, (int)(threadIdx.x + 1) * per); ++b)
    mine += (keys_of(P.a, b) + kUnit - 1) / kUnit * pairs;
  // exclusive sums over the block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, sum, d);
    if (lane >= d) sum += o;
  }
  __shared__ int warp_sum[NT / 32];
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  int base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) base += warp_sum[w];
    total += warp_sum[w];
  }
  scratch[threadIdx.x] = base + sum - mine;
  if (threadIdx.x == 0) scratch[NT] = total;
  __syncthreads();
  return total;
}

// Block c's share of `total` units: equal shares, the first total % n of them one unit longer.
struct Shares {
  int base, longer;
  __device__ __forceinline__ Shares(int total, int n) : base(total / n), longer(total - total / n * n) {}
  __device__ __forceinline__ int begin(int c) const { return c * base + min(c, longer); }
  __device__ __forceinline__ int of(int unit) const {  // the share that holds a unit
    const int cut = longer * (base + 1);
    return unit < cut ? unit / (base + 1) : longer + (unit - cut) / base;
  }
};

// One pair's place in the flattened order: sequence b, head tile h (kv head * tiles + tile).
struct Walk {
  int b, h, tile, ntile, len;
  __device__ __forceinline__ void enter(const PagedParams& P, int seq) {
    b = seq;
    for (;;) {
      len = b < P.a.batch ? keys_of(P.a, b) : 0;
      ntile = (len + kUnit - 1) / kUnit;
      if (ntile > 0 || b >= P.a.batch) break;
      ++b;
    }
    h = tile = 0;
  }
  __device__ __forceinline__ void next(const PagedParams& P) {
    if (++tile < ntile) return;
    tile = 0;
    if (++h < P.a.pages.n_kv_heads * P.tiles) return;
    enter(P, b + 1);
  }
};

// The place of unit `u` (below the total), by a block of NT threads' sums in `scratch` (scan_units).
template <int NT>
__device__ __forceinline__ Walk walk_to(const PagedParams& P, const int* scratch, int per, int u) {
  // the last group of sequences that begins at or before u
  int lo = 0, hi = NT - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (scratch[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  int at = scratch[lo];
  const int pairs = P.a.pages.n_kv_heads * P.tiles;
  Walk w;
  w.enter(P, lo * per);
  while (at + w.ntile * pairs <= u) {
    at += w.ntile * pairs;
    w.enter(P, w.b + 1);
  }
  w.h = (u - at) / w.ntile;
  w.tile = (u - at) % w.ntile;
  return w;
}

// first element of key `t` of the pair's rows; -1: no such key (zeros)
__device__ __forceinline__ long long row_offset(const PagedParams& P, const Walk& w, int t) {
  if (t >= w.len) return -1;
  const mk_kv_pages& g = P.a.pages;
  const unsigned page_index = (unsigned)t / (unsigned)g.page_size, row = (unsigned)t % (unsigned)g.page_size;
  const int page = page_of(g, w.b, page_index, P.a.status);
  if (page < 0) return -1;
  return page * g.page_stride + (long long)(w.h / P.tiles) * g.head_stride + row * g.row_stride;
}

// TMA: page_size is a multiple of 16, so a warp's 16 keys lie in one page and
// come as boxes of 64 dimensions x 16 rows; else the rows are gathered one by one.
template <class T, int D, bool FULL, bool TMA>
__global__ void __launch_bounds__(kThreads, Shape<D, FULL>::kBlocksPerSm) paged_kernel(const __grid_constant__ PagedParams P) {
  using S = Shape<D, FULL>;
  constexpr int CH = D / 8;  // 16-byte chunks of a row
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);  // (the swizzle goes by address)
  __shared__ uint64_t landed[kWarps][S::kStages];
  __shared__ int scratch[kThreads + 1];
  __shared__ float part_m[kWarps][kRows], part_l[kWarps][kRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quad = lane >> 2, sub = lane & 3;
  float* merge = reinterpret_cast<float*>(smem + kWarps * S::kStages * S::kPiece);
  const uint32_t ring = smem_u32(smem) + warp * S::kStages * S::kPiece;

  if (TMA && tid == 0) {
    prefetch_map(&P.tk);
    prefetch_map(&P.tv);
  }
  dep_wait();
  dep_launch();
  int per;
  const int total = scan_units<kThreads>(P, scratch, per);
  const Shares shares(total, P.n_cta);
  const int u0 = shares.begin(blockIdx.x), u1 = shares.begin(blockIdx.x + 1);
  // sequences without keys have zero rows; each block sees to some of them, after its share
  auto clear_empty = [&]() {
    for (int b = blockIdx.x; b < P.a.batch; b += gridDim.x) {
      if (keys_of(P.a, b) > 0) continue;
      for (int i = tid; i < P.a.n_q_heads * D; i += kThreads)
        static_cast<T*>(P.a.out)[b * P.a.o_row_stride + i / D * P.a.o_head_stride + i % D] = static_cast<T>(0.f);
    }
  };
  if (u0 >= u1) {
    clear_empty();
    return;
  }

  Walk load = walk_to<kThreads>(P, scratch, per, u0);
  Walk use = load;
  const int n_units = u1 - u0;

  // The piece that is loaded next, its page looked up one unit ahead.  A piece holds its keys' 16 rows, then its
  // values', each as halves of 64 dimensions: 128 bytes a row, 16-byte chunks swizzled by the row's low three bits.
  constexpr int kHalf = kKeys * 128, kRowsOfKeys = kKeys * D * 2;
  const int my_key = warp * kKeys + (TMA ? 0 : (lane & 15));
  long long off = 0;
  int page = 0, row = 0;
  auto look_up = [&]() {
    const int t = load.tile * kUnit + my_key;
    if (TMA) {
      const unsigned ps = P.a.pages.page_size;
      page = t < load.len ? page_of(P.a.pages, load.b, (unsigned)t / ps, P.a.status) : -1;
      row = (unsigned)t % ps;
    } else {
      off = row_offset(P, load, t);
    }
  };
  look_up();
  int issued = 0;
  bool lost = false;  // a wait has run out: the rest is computed without waiting, the status word tells
  auto issue = [&]() {
    if (issued < n_units) {
      const int stage = issued % S::kStages;
      const uint32_t st = ring + stage * S::kPiece;
      if (TMA) {
        if (lane == 0) {
          unsigned char* dst = smem + (warp * S::kStages + stage) * S::kPiece;
          const int head = load.h / P.tiles, p = page < 0 ? P.a.pages.n_pages : page;  // (no such page: zeros)
          mbar_arrive_expect_tx(&landed[warp][stage], S::kPiece);
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            tma_load_4d(dst + h * kHalf, &P.tk, 64 * h, row, head, p, &landed[warp][stage]);
            tma_load_4d(dst + kRowsOfKeys + h * kHalf, &P.tv, 64 * h, row, head, p, &landed[warp][stage]);
          }
        }
        __syncwarp();
      } else {
        const char* kbase = static_cast<const char*>(P.a.pages.k);
        const char* vbase = static_cast<const char*>(P.a.pages.v);
#pragma unroll
        for (int i = 0; i < kKeys * CH / 32; ++i) {
          const int r = (i * 32 + lane) / CH, c = (i * 32 + lane) % CH;
          const long long o = __shfl_sync(~0u, off, r);
          const uint32_t d = st + (c / 8) * kHalf + r * 128 + (((c % 8) ^ (r & 7)) << 4);
          const long long byte = (o + c * 8) * 2;
          cp16(d, o < 0 ? P.a.q : kbase + byte, o >= 0);  // (no such row: zeros, nothing is read)
          cp16(d + kRowsOfKeys, o < 0 ? P.a.q : vbase + byte, o >= 0);
        }
      }
      ++issued;
      if (issued < n_units) {
        load.next(P);
        look_up();
      }
    }
    if (!TMA) cp_commit();
  };
  if (TMA) {
    if (lane == 0) {
      for (int i = 0; i < S::kStages; ++i) mbar_init(&landed[warp][i], 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
  }
  // the lane's place in the 8 x 8 matrices of a 16 x 16 block: row and chunk, the swizzle applied; chunk 2k is ^ (k << 5)
  const int kr = (lane & 7) + ((lane >> 4) << 3), vr = lane & 15;
  const uint32_t kat = kr * 128 + ((((lane >> 3) & 1) ^ (kr & 7)) << 4), vat = kRowsOfKeys + vr * 128 + (((lane >> 4) ^ (vr & 7)) << 4);
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) issue();

  int slot = 0;  // the partial that the next unfinished pair goes to
  for (int u = 0; u < n_units;) {
    // ---- one pair's part: its units in this share
    const int n_here = min(use.ntile - use.tile, n_units - u);
    const int first_head = (use.h / P.tiles) * P.group + (use.h % P.tiles) * kRows;
    const int heads = min(kRows, P.group - (use.h % P.tiles) * kRows);
    uint32_t q[D / 16][4];
    {
      const T* row0 = static_cast<const T*>(P.a.q) + use.b * P.a.q_row_stride + (first_head + quad) * P.a.q_head_stride;
      const T* row1 = row0 + 8 * P.a.q_head_stride;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][0] = quad < heads ? __ldg(reinterpret_cast<const uint32_t*>(row0 + 16 * k + 2 * sub)) : 0u;
        q[k][2] = quad < heads ? __ldg(reinterpret_cast<const uint32_t*>(row0 + 16 * k + 8 + 2 * sub)) : 0u;
        if (FULL) {
          q[k][1] = quad + 8 < heads ? __ldg(reinterpret_cast<const uint32_t*>(row1 + 16 * k + 2 * sub)) : 0u;
          q[k][3] = quad + 8 < heads ? __ldg(reinterpret_cast<const uint32_t*>(row1 + 16 * k + 8 + 2 * sub)) : 0u;
        } else {
          q[k][1] = q[k][0];
          q[k][3] = q[k][2];
        }
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int i = 0; i < n_here; ++i, ++u) {
      issue();
      const uint32_t at = ring + (u % S::kStages) * S::kPiece;
      if (TMA) {
        Landing piece{&landed[warp][u % S::kStages], (uint32_t)(u / S::kStages) & 1};
        if (!lost && !wait_together(piece, kWaitNs)) {
          if (P.a.status) *P.a.status = MK_ERR_DEVICE_TIMEOUT;
          lost = true;
        }
      } else {
        cp_wait<S::kStages - 1>();
      }
      __syncwarp();
      float s[2][4] = {};
      // matrices: (keys 0-7, dims 0-7), (keys 0-7, dims 8-15), (keys 8-15, dims 0-7), (keys 8-15, dims 8-15)
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldsm4(b, (at + (k / 4) * kHalf + kat) ^ ((k % 4) << 5));
        mma16816<T>(s[0], q[k], b[0], b[1]);
        mma16816<T>(s[1], q[k], b[2], b[3]);
      }
      const int left = use.len - (use.tile + i) * kUnit - warp * kKeys;  // keys of the piece that exist
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = t * 8 + 2 * sub + (e & 1);
          s[t][e] = key < left ? s[t][e] * P.scale_log2 : -INFINITY;
        }
      float n0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      n0 = fmaxf(n0, __shfl_xor_sync(~0u, n0, 1));
      n0 = fmaxf(m0, fmaxf(n0, __shfl_xor_sync(~0u, n0, 2)));
      float n1 = n0;
      if (FULL) {
        n1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
        n1 = fmaxf(n1, __shfl_xor_sync(~0u, n1, 1));
        n1 = fmaxf(m1, fmaxf(n1, __shfl_xor_sync(~0u, n1, 2)));
      }
      if (__any_sync(~0u, n0 > m0 || n1 > m1)) {
        // a maximum moved: what was summed is brought to it (exp2f(-inf) = 0 at the first piece)
        const float f0 = n0 > m0 ? exp2f(m0 - n0) : 1.f, f1 = FULL ? (n1 > m1 ? exp2f(m1 - n1) : 1.f) : f0;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          o[k][0] *= f0;
          o[k][1] *= f0;
          o[k][2] *= f1;
          o[k][3] *= f1;
        }
        m0 = n0;
        m1 = n1;
      }
      const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float p0 = exp2f(s[t][0] - z0), p1 = exp2f(s[t][1] - z0);
        l0 += p0 + p1;
        hi[2 * t] = Elem<T>::pack(p0, p1);
        float2 h = Elem<T>::unpack(hi[2 * t]);
        const uint32_t rest0 = Elem<T>::pack(p0 - h.x, p1 - h.y);
        if (FULL) {
          const float p2 = exp2f(s[t][2] - z1), p3 = exp2f(s[t][3] - z1);
          l1 += p2 + p3;
          hi[2 * t + 1] = Elem<T>::pack(p2, p3);
          h = Elem<T>::unpack(hi[2 * t + 1]);
          lo[2 * t] = rest0;
          lo[2 * t + 1] = Elem<T>::pack(p2 - h.x, p3 - h.y);
        } else {
          hi[2 * t + 1] = rest0;  // rows 8 to 15: the remainders of rows 0 to 7
        }
      }
      // A row behind the last key may hold anything, NaN too, and has probability 0: it is left out of the product.
      // (Gathered rows behind the last key are zeros already.)
      const bool ragged = TMA && left < kKeys;
      const uint32_t live0 = (2 * sub < left ? 0xffffu : 0u) | (2 * sub + 1 < left ? 0xffff0000u : 0u);
      const uint32_t live1 = (2 * sub + 8 < left ? 0xffffu : 0u) | (2 * sub + 9 < left ? 0xffff0000u : 0u);
      // transposed: (keys 0-7, dims 0-7), (keys 8-15, dims 0-7), (keys 0-7, dims 8-15), (keys 8-15, dims 8-15)
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldsm4_trans(b, (at + (k / 4) * kHalf + vat) ^ ((k % 4) << 5));
        if (ragged) {
          b[0] &= live0;
          b[1] &= live1;
          b[2] &= live0;
          b[3] &= live1;
        }
        mma16816<T>(o[2 * k], hi, b[0], b[1]);
        mma16816<T>(o[2 * k + 1], hi, b[2], b[3]);
        if (FULL) {
          mma16816<T>(o[2 * k], lo, b[0], b[1]);
          mma16816<T>(o[2 * k + 1], lo, b[2], b[3]);
        }
      }
      __syncwarp();  // the stage is read before the next copy into it is issued
    }

    // ---- the four warps' parts meet
    l0 += __shfl_xor_sync(~0u, l0, 1);
    l0 += __shfl_xor_sync(~0u, l0, 2);
    if (FULL) {
      l1 += __shfl_xor_sync(~0u, l1, 1);
      l1 += __shfl_xor_sync(~0u, l1, 2);
    } else {
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        o[k][0] += o[k][2];
        o[k][1] += o[k][3];
      }
    }
    if (sub == 0) {
      part_m[warp][quad] = m0;
      part_l[warp][quad] = l0;
      if (FULL) {
        part_m[warp][quad + 8] = m1;
        part_l[warp][quad + 8] = l1;
      }
    }
    __syncthreads();
    float top0 = -INFINITY, top1 = -INFINITY, sum0 = 0.f, sum1 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      top0 = fmaxf(top0, part_m[w][quad]);
      if (FULL) top1 = fmaxf(top1, part_m[w][quad + 8]);
    }
    // (unit 0 of a part always holds a key, so the tops are finite; a warp without one has weight 0)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum0 += part_l[w][quad] * exp2f(part_m[w][quad] - top0);
      if (FULL) sum1 += part_l[w][quad + 8] * exp2f(part_m[w][quad + 8] - top1);
    }
    const float f0 = exp2f(m0 - top0), f1 = FULL ? exp2f(m1 - top1) : 0.f;
    // outputs add up two by two through shared memory: all of the 8 rows at once, or 16 rows in two halves of D
    constexpr int ROWS = FULL ? 16 : 8, PARTS = FULL ? 2 : 1, W = D / PARTS, KN = W / 8;
    float* buf = merge + (warp & 1) * ROWS * W;
    const float* other = merge + ROWS * W;
    const bool whole = n_here == use.ntile;
    float* part = P.partial + ((long long)blockIdx.x * 2 + slot) * kPartial<D>;
    T* row0 = static_cast<T*>(P.a.out) + use.b * P.a.o_row_stride + (first_head + quad) * P.a.o_head_stride;
    T* row1 = row0 + 8 * P.a.o_head_stride;
    const float i0 = 1.f / sum0, i1 = FULL ? 1.f / sum1 : 0.f;
    if (warp == 0 && sub == 0 && !whole) {
      part[quad] = top0;
      part[kRows + quad] = sum0;
      if (FULL) {
        part[quad + 8] = top1;
        part[kRows + quad + 8] = sum1;
      }
    }
#pragma unroll
    for (int h = 0; h < PARTS; ++h) {
      if (h) __syncthreads();
      if (warp >= 2) {
#pragma unroll
        for (int k = 0; k < KN; ++k) {
          const float(&x)[4] = o[h * KN + k];
          *reinterpret_cast<float2*>(buf + quad * W + 8 * k + 2 * sub) = make_float2(x[0] * f0, x[1] * f0);
          if (FULL) *reinterpret_cast<float2*>(buf + (quad + 8) * W + 8 * k + 2 * sub) = make_float2(x[2] * f1, x[3] * f1);
        }
      }
      __syncthreads();
      if (warp < 2) {
#pragma unroll
        for (int k = 0; k < KN; ++k) {
          float(&x)[4] = o[h * KN + k];
          float2* p = reinterpret_cast<float2*>(buf + quad * W + 8 * k + 2 * sub);
          x[0] = x[0] * f0 + p->x;
          x[1] = x[1] * f0 + p->y;
          if (warp == 1) *p = make_float2(x[0], x[1]);
          if (FULL) {
            p = reinterpret_cast<float2*>(buf + (quad + 8) * W + 8 * k + 2 * sub);
            x[2] = x[2] * f1 + p->x;
            x[3] = x[3] * f1 + p->y;
            if (warp == 1) *p = make_float2(x[2], x[3]);
          }
        }
      }
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int k = 0; k < KN; ++k) {
          const int col = h * W + 8 * k + 2 * sub;
          const float(&x)[4] = o[h * KN + k];
          float2 y0 = *reinterpret_cast<const float2*>(other + quad * W + 8 * k + 2 * sub), y1 = make_float2(0.f, 0.f);
          y0 = make_float2(x[0] + y0.x, x[1] + y0.y);
          if (FULL) {
            y1 = *reinterpret_cast<const float2*>(other + (quad + 8) * W + 8 * k + 2 * sub);
            y1 = make_float2(x[2] + y1.x, x[3] + y1.y);
          }
          if (whole) {
            if (quad < heads) *reinterpret_cast<uint32_t*>(row0 + col) = Elem<T>::pack(y0.x * i0, y0.y * i0);
            if (FULL && quad + 8 < heads) *reinterpret_cast<uint32_t*>(row1 + col) = Elem<T>::pack(y1.x * i1, y1.y * i1);
          } else {
            *reinterpret_cast<float2*>(part + 2 * kRows + quad * D + col) = y0;
            if (FULL) *reinterpret_cast<float2*>(part + 2 * kRows + (quad + 8) * D + col) = y1;
          }
        }
      }
    }
    slot = 1;
    // on to the next pair (warps 1 to 3 may run ahead: the merge buffers are written again only behind a barrier)
    use.tile += n_here - 1;
    use.next(P);
  }
  if (TMA && lost) {  // no copy is in flight when the block leaves, if that can be had
    const unsigned long long t0 = global_ns();
    for (int i = max(0, n_units - S::kStages); i < n_units; ++i)
      while (!mbar_try(&landed[warp][i % S::kStages], (i / S::kStages) & 1) && global_ns() - t0 < kWaitNs) {}
  }
  clear_empty();
}

// The parts of one (sequence, query head) joined.  A block for each of them, as
// long as these are few (by_pair); else a block for each row of the pair that a
// share's end cuts, which works if that is the pair's first cut (4,000
// sequences of 200 keys: 2.26 -> 0.43 ms; 32 sequences: 53 -> 55 us, so the few
// keep the first way).  Launched while the first kernel runs (programmatic
// dependent launch): it finds its place, then waits for the parts.  A thread
// takes every GROUPS-th part, four at a time so that their loads travel
// together, and keeps a running maximum.
constexpr int kJoinThreads = 128;

template <class T, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ PagedParams P) {
  constexpr int LANES = D / 4, GROUPS = kJoinThreads / LANES;  // threads of a part's row, 4 values each
  __shared__ int scratch[kJoinThreads + 1];
  __shared__ float4 group_o[GROUPS][LANES];
  __shared__ float group_m[GROUPS], group_l[GROUPS];
  const int tid = threadIdx.x;
  int per;
  const int total = scan_units<kJoinThreads>(P, scratch, per);
  const Shares shares(total, P.n_cta);
  const int pairs = P.a.pages.n_kv_heads * P.tiles;
  int b = 0, head = 0, row = 0, p0 = 0, c0 = 0, c1 = 0;  // the pair's first unit, its first and last share
  if (P.by_pair) {
    b = blockIdx.y;
    head = blockIdx.x;
    const int ntile = (keys_of(P.a, b) + kUnit - 1) / kUnit, in_group = head % P.group;
    int at = scratch[b / per];
    for (int i = b / per * per; i < b; ++i) at += (keys_of(P.a, i) + kUnit - 1) / kUnit * pairs;
    row = in_group % kRows;
    p0 = at + ((head / P.group) * P.tiles + in_group / kRows) * ntile;
    if (ntile > 0) {
      c0 = shares.of(p0);
      c1 = shares.of(p0 + ntile - 1);
    }
  } else {
    const int cut = shares.begin(blockIdx.y + 1);
    if (cut < total) {
      const Walk w = walk_to<kJoinThreads>(P, scratch, per, cut);
      row = blockIdx.x;
      b = w.b;
      head = (w.h / P.tiles) * P.group + (w.h % P.tiles) * kRows + row;
      p0 = cut - w.tile;
      c0 = blockIdx.y;
      // (not cut, or not here first, or no such head: nothing to do)
      c1 = w.tile > 0 && shares.begin(c0) <= p0 && row < P.group - (w.h % P.tiles) * kRows ? shares.of(p0 + w.ntile - 1) : c0;
    }
  }
  dep_wait();
  dep_launch();
  if (c0 == c1) return;  // one block had it all and wrote it
  const int g = tid / LANES, c = tid % LANES;
  T* out = static_cast<T*>(P.a.out) + b * P.a.o_row_stride + head * P.a.o_head_stride;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = c0 + g; k0 <= c1; k0 += 4 * GROUPS) {
    float pm[4], pl[4];
    float4 po[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = k0 + e * GROUPS;
      pm[e] = -INFINITY;
      pl[e] = 0.f;
      po[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k <= c1) {
        // a share that begins before the pair ends with its part of it
        const float* part = P.partial + ((long long)k * 2 + (shares.begin(k) < p0 ? 1 : 0)) * kPartial<D>;
        pm[e] = part[row];
        pl[e] = part[kRows + row];
        po[e] = *reinterpret_cast<const float4*>(part + 2 * kRows + row * D + 4 * c);
      }
    }
    const float up = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])), m), f = exp2f(m - up);
    l *= f;
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float w = exp2f(pm[e] - up);
      l += w * pl[e];
      o.x += w * po[e].x, o.y += w * po[e].y, o.z += w * po[e].z, o.w += w * po[e].w;
    }
    m = up;
  }
  if (c == 0) {
    group_m[g] = m;
    group_l[g] = l;
  }
  group_o[g][c] = o;
  __syncthreads();
  if (g == 0) {
    float top = m;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) top = fmaxf(top, group_m[i]);
    float f = exp2f(m - top);
    l *= f;
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) {
      const float4 v = group_o[i][c];
      f = exp2f(group_m[i] - top);
      l += f * group_l[i];
      o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
    }
    const float inv = 1.f / l;
    *reinterpret_cast<uint2*>(out + 4 * c) = make_uint2(Elem<T>::pack(o.x * inv, o.y * inv), Elem<T>::pack(o.z * inv, o.w * inv));
  }
}

template <class T, int D, bool FULL, bool TMA>
mk_status launch(PagedParams& P, cudaStream_t s, std::string& err) {
  using S = Shape<D, FULL>;
  Device dev;
  cudaError_t e = current_device(dev);
  if (e == cudaSuccess) e = allow<paged_kernel<T, D, FULL, TMA>>(dev, S::kSmem);
  if (e != cudaSuccess) return cuda_result(e, "mk_paged_attention attributes", err);
  P.n_cta = std::min(kMaxCtas, dev.sms * S::kBlocksPerSm);
  P.by_pair = (long long)P.a.batch * P.a.n_q_heads <= 2048;
  const long long units = ((long long)P.a.pages.table_width * P.a.pages.page_size + kUnit - 1) / kUnit * P.a.batch *
                          P.a.pages.n_kv_heads * P.tiles;
  e = mk::launch(units <= P.n_cta, paged_kernel<T, D, FULL, TMA>, dim3(P.n_cta), kThreads, S::kSmem, s, 0, P);
  if (e != cudaSuccess) return cuda_result(e, "mk_paged_attention launch", err);
  const dim3 grid = P.by_pair ? dim3(P.a.n_q_heads, P.a.batch) : dim3(std::min(P.group, kRows), P.n_cta - 1);
  e = mk::launch(true, join_kernel<T, D>, grid, kJoinThreads, 0, s, 0, P);
  return cuda_result(e, "mk_paged_attention join launch", err);
}
template <class T, int D>
mk_status pick(PagedParams& P, cudaStream_t s, std::string& err) {
  const mk_kv_pages& g = P.a.pages;
  // (no tensor map of the pool's strides, as where heads share their rows: gathered)
  if (g.page_size % kKeys == 0 && g.n_pages > 0 && encode_pages(&P.tk, &P.tv, g, kKeys))
    return P.group > 8 ? launch<T, D, true, true>(P, s, err) : launch<T, D, false, true>(P, s, err);
  return P.group > 8 ? launch<T, D, true, false>(P, s, err) : launch<T, D, false, false>(P, s, err);
}

}  // namespace

size_t paged_workspace_bytes(int, int, int, int head_dim) {
  return (size_t)kMaxCtas * 2 * (head_dim <= 64 ? kPartial<64> : kPartial<128>) * sizeof(float);
}

mk_status launch_paged(const mk_paged_attn_args& a, void* stream, std::string& err) {
  PagedParams P;
  P.a = a;
  P.group = a.n_q_heads / a.pages.n_kv_heads;
  P.tiles = (P.group + kRows - 1) / kRows;
  const long long units = ((long long)a.pages.table_width * a.pages.page_size + kUnit - 1) / kUnit;
  if (units * a.batch * a.pages.n_kv_heads * P.tiles > 0x7fffffffll) {
    err = "batch, heads and page table reach 2^31 units of 64 keys";
    return MK_ERR_UNSUPPORTED;
  }
  const float scale = a.scale > 0.f ? a.scale : 1.f / std::sqrt((float)a.pages.head_dim);
  P.scale_log2 = scale * 1.4426950408889634f;
  P.partial = static_cast<float*>(a.workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = a.pages.head_dim == 128;
  if (a.pages.dtype == MK_DTYPE_BF16)
    return wide ? pick<__nv_bfloat16, 128>(P, s, err) : pick<__nv_bfloat16, 64>(P, s, err);
  return wide ? pick<__half, 128>(P, s, err) : pick<__half, 64>(P, s, err);
}

}  // namespace mk
