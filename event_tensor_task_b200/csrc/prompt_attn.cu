// prompt_attn.cu — mk_prompt_attention: attention of packed prompts over packed
// or paged keys, on tcgen05.
//
// Mathematics: out_i = sum_j p_ij v_j / sum_j p_ij, p_ij = 2^(c (q_i.k_j) - m_i),
// c = scale log2 e, in one pass over the keys with a running reference m_i.
// m_i follows the running maximum only when that has grown by more than 2^8:
// the probabilities then stay below 2^8, exact in the same way, and the
// accumulated output is rescaled a few times a row instead of at every tile.
//
// Rows: the G = n_q_heads / n_kv_heads query heads that share a kv head are
// stacked, so a tile of 128 rows is floor(128 / G) tokens times G heads (one
// TMA box [tokens][G][64]); a short prompt fills a tile G times better and the
// causal diagonal is G times narrower than with one head per tile.
//
// A block holds two such tiles (256 rows) and streams the keys past both:
//   warps 0-3 / 4-7: softmax of tile 0 / 1, a thread per row: S from TMEM to
//                    registers, maximum, exponentials, P (16 bit) back to TMEM
//                    over S, at the end O / l to global memory;
//   warp 8:          one thread issues the MMAs, S = Q K^T (Q, K from shared
//                    memory, both K-major) and O += P V (P from TMEM, V from
//                    shared memory, its N = dimensions contiguous);
//   warp 9:          TMA loads, K and V tiles of 128 keys in a ring
//                    (warps 10 and 11 fill up the warpgroup whose registers
//                    the softmax warps take over).
// While one tile is in its softmax, the other has the tensor pipe.
//
// Bound: at D = 128 the two products and the exponentials take the same time
// (128 x 128 scores: 1,024 cycles of the tensor pipe, 1,024 of the MUFU); at
// D = 64 the exponentials take twice the products' time.
#include <algorithm>
#include <cmath>

#include "serve.cuh"

namespace mk {
namespace {

constexpr int kRows = 128;   // rows of a tile, keys of a tile
constexpr int kTiles64 = 1;           // row tiles of a block at D = 64
constexpr int kParts = 2;            // parts of a P tile, handed to the MMAs one by one
constexpr float kSlack = 8.f;  // log2 growth of the maximum that is left to the probabilities
constexpr unsigned long long kWaitNs = 2000000000ull;  // limit of every wait

// TILES: row tiles of a block
template <int D, int TILES>
struct Shape {
  static constexpr int kSoftmaxWarps = 4 * TILES;
  static constexpr int kThreads = (kSoftmaxWarps + 4) * 32;  // (registers move between whole warpgroups)
  static constexpr int kBlocksPerSm = TILES == 1 ? 2 : 1;
  // registers of a thread: at launch 64K / (threads of an SM), then softmax and other warps
  static constexpr int kMore = TILES == 1 ? 200 : 208, kLess = TILES == 1 ? 56 : 80;
  static constexpr int kTmem = TILES == 1 ? 256 : 512;       // columns
  static constexpr int kTile = kRows * D * 2;        // bytes of 128 rows
  static constexpr int kStages = D == 64 ? (TILES == 1 ? 5 : 8) : 4;  // ring of K and V tiles
  static constexpr int kFma = D == 64 ? 2 : 1;       // of 8 exponentials, how many go over the FMA pipes
  static constexpr int kSmem = (TILES + kStages) * kTile + 1024;
};

struct PromptParams {
  CUtensorMap tq, tk, tv;
  mk_prompt_args a;
  float scale_log2;
  int group, tokens;   // G; tokens of a row tile
  int blocks;          // upper bound on blocks of row tiles of all sequences
  int span, per_span;  // keys of a page (or of all), key tiles that cover them
  int box;             // key rows of a TMA box
};

struct Control {
  uint64_t q_full, kv_full[8], kv_empty[8], s_full[2], p_full[2][kParts], pv_done[2], v_tail;
  uint32_t tmem;
  int abort;
  int warp_sum[8];
  int found;
  int seq, pair;
};

// A whole warp waits for a phase; false (for all its lanes) after the limit or once another role has given up.
__device__ __forceinline__ bool await_lane(Control& c, uint64_t* bar, uint32_t parity, int* status) {
  if (mbar_try(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&c.abort)) return false;
    if (global_ns() - t0 > kWaitNs) {
      *reinterpret_cast<volatile int*>(&c.abort) = 1;
      if (status) *status = MK_ERR_DEVICE_TIMEOUT;
      return false;
    }
  }
}

__device__ __forceinline__ bool await(Control& c, uint64_t* bar, uint32_t parity, int* status) {
  return __all_sync(~0u, await_lane(c, bar, parity, status));
}
// Waits for copies in flight, whatever became of the other roles.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = global_ns();
  while (!mbar_try(bar, parity) && global_ns() - t0 < kWaitNs) {}
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Shared-memory descriptors under the 128-byte swizzle, the upper half the
// same for all: 8-row (8-k) groups 1024 bytes apart, version 1, 128-byte
// swizzle.  The lower half holds the address and the leading offset, both / 16:
// for a K-major operand (Q, K: 64 elements of k in a row) that is unused (1)
// and a 16-k step is 32 bytes further; for V, whose rows are k and hold 64 of
// its N dimensions, it leads to the next 64 dimensions and a 16-k step is
// 2048 bytes further.
constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(const void* tile, uint32_t leading) {
  return ((smem_u32(tile) >> 4) & 0x3FFFu) | (leading << 16);
}
// kind::f16 instruction descriptor: fp32 D, A and B bf16 (format 1) or fp16
// (format 0), bit 16: B with N contiguous.
template <class T>
__device__ constexpr uint32_t idesc(int n, bool b_mn) {
  const uint32_t f = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
// D[tmem] (+)= A . B, A from shared memory or from TMEM
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(id), "r"((uint32_t)accumulate), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t id, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(id), "r"((uint32_t)accumulate), "n"(kDescHi)
      : "memory");
}

#define MK_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define MK_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 consecutive columns of the thread's TMEM lane (no wait)
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : MK_R8(r, 0), MK_R8(r, 8), MK_R8(r, 16), MK_R8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      MK_W8(r, 0), MK_W8(r, 8), MK_W8(r, 16), MK_W8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      MK_W8(r, 0), MK_W8(r, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// two fp32 values in one register pair: one instruction for both
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 2^x of a pair on the FMA pipes, for x in [-125, 64] (smaller x as -125):
// x = n + f with n whole and |f| <= 1/2 (Cody-Waite reduction by adding
// 1.5 2^23), 2^f by a degree-4 polynomial, n into the exponent.  The
// coefficients are those of the least relative error on [-1/2, 1/2] (Remez
// exchange): 2^-18.5, far below a 16-bit probability's half step.
__device__ __forceinline__ float2 ex2_fma(uint64_t x) {
  float2 v = both(x);
  x = pair(fmaxf(v.x, -125.f), fmaxf(v.y, -125.f));
  const uint64_t magic = pair(12582912.f, 12582912.f);
  const uint64_t t = add2(x, magic);
  const uint64_t f = fma2(add2(t, pair(-12582912.f, -12582912.f)), pair(-1.f, -1.f), x);
  uint64_t p = fma2(pair(0.009570102f, 0.009570102f), f, pair(0.055917859f, 0.055917859f));
  p = fma2(p, f, pair(0.24024744f, 0.24024744f));
  p = fma2(p, f, pair(0.69312179f, 0.69312179f));
  p = fma2(p, f, pair(0.99999928f, 0.99999928f));
  const float2 n = both(t), y = both(p);
  return make_float2(__uint_as_float(__float_as_uint(y.x) + (__float_as_uint(n.x) << 23)),
                     __uint_as_float(__float_as_uint(y.y) + (__float_as_uint(n.y) << 23)));
}
// p = 2^(c s - m) of the 128 scores in x, 16-bit pairs to TMEM at `dst`, each
// part announced on `ready` when it is there; returns their sum.  FMA of 8 pairs go over the FMA pipes, the others over
// the MUFU.
template <class T, int FMA>
__device__ __forceinline__ float exponentials(const uint32_t* x, float c, float m, uint32_t dst, uint64_t* ready, int lane) {
  const uint64_t cc = pair(c, c), mm = pair(-m, -m);
  uint64_t sum[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kRows; i += 32) {
    uint32_t p[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint64_t u = fma2(pair(__uint_as_float(x[i + 2 * e]), __uint_as_float(x[i + 2 * e + 1])), cc, mm);
      float2 y;
      if ((e * FMA) / 8 != ((e + 1) * FMA) / 8) {
        y = ex2_fma(u);
      } else {
        y = both(u);
        y = make_float2(ex2(y.x), ex2(y.y));
      }
      sum[e & 1] = add2(sum[e & 1], pair(y.x, y.y));
      p[e] = Elem<T>::pack(y.x, y.y);
    }
    tmem_st16(dst + i / 2, p);
    if ((i + 32) % (kRows / kParts) == 0) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ready + i / (kRows / kParts));
    }
  }
  const float2 a = both(add2(sum[0], sum[1]));
  return a.x + a.y;
}

// One sequence: its query rows, key rows and where they lie.
struct Seq {
  int q0, n;   // first query row, queries
  int k0, m;   // first key row (packed), keys
  __device__ __forceinline__ void load(const PromptParams& P, int b) {
    const mk_prompt_args& a = P.a;
    const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1);
    q0 = min(max(c0, 0), a.n_tokens);
    n = max(min(c1, a.n_tokens), q0) - q0;
    bool fine = c0 == q0 && c1 == q0 + n;
    if (a.pages.page_table) {
      const int cap = a.pages.table_width * a.pages.page_size, l = __ldg(a.kv_lens + b);
      k0 = 0;
      m = min(max(l, 0), cap);
      fine = fine && l == m;
    } else {
      const int e0 = __ldg(a.cu_k + b), e1 = __ldg(a.cu_k + b + 1);
      k0 = min(max(e0, 0), a.pages.page_size);
      m = max(min(e1, a.pages.page_size), k0) - k0;
      fine = fine && e0 == k0 && e1 == k0 + m;
    }
    if (!fine) report_bounds(a.status);
  }
  // keys that query i sees
  __device__ __forceinline__ int limit(const PromptParams& P, int i) const {
    return P.a.causal ? min(m, max(0, i + 1 + m - n)) : m;
  }
};

template <class T, int D, int TILES>
__global__ void __launch_bounds__(Shape<D, TILES>::kThreads, Shape<D, TILES>::kBlocksPerSm)
    prompt_kernel(const __grid_constant__ PromptParams P) {
  using S = Shape<D, TILES>;
  constexpr int HALVES = D / 64, kSoftmaxWarps = S::kSoftmaxWarps, kO = 128 * TILES;
  extern __shared__ unsigned char raw[];
  __shared__ Control c;
  unsigned char* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  unsigned char* sq = smem;                      // [TILES][HALVES][128][64]
  unsigned char* ring = smem + TILES * S::kTile; // [kStages][HALVES][128][64]
  const mk_prompt_args& a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kvh = blockIdx.x % a.pages.n_kv_heads;
  const int want = P.blocks - 1 - (int)(blockIdx.x / a.pages.n_kv_heads);  // long rows (the last) first

  // ---- which sequence and pair of row tiles: counted over the sequences, 256 at a time
  if (tid == 0) {
    c.abort = 0;
    c.found = 0;
  }
  __syncthreads();
  int base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kSoftmaxWarps * 32) {
    int mine = 0, sum = 0;
    if (warp < kSoftmaxWarps) {
      const int b = b0 + tid;
      if (b < a.batch) {
        const int q0 = min(max(__ldg(a.cu_q + b), 0), a.n_tokens), q1 = min(__ldg(a.cu_q + b + 1), a.n_tokens);
        mine = (max(q1 - q0, 0) + TILES * P.tokens - 1) / (TILES * P.tokens);
      }
      sum = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(~0u, sum, d);
        if (lane >= d) sum += o;
      }
      if (lane == 31) c.warp_sum[warp] = sum;
    }
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kSoftmaxWarps; ++w) {
      if (w < warp) sum += c.warp_sum[w];
      total += c.warp_sum[w];
    }
    if (warp < kSoftmaxWarps && want >= base + sum - mine && want < base + sum) {
      c.seq = b0 + tid;
      c.pair = want - (base + sum - mine);
      c.found = 1;
    }
    __syncthreads();
    base += total;
    if (c.found) break;
  }
  if (!c.found) return;

  Seq s;
  s.load(P, c.seq);
  const int first = c.pair * TILES * P.tokens;  // the block's first query
  int tiles[TILES], n_tiles = 0;            // key tiles of each row tile
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    const int last = min(s.n, first + (t + 1) * P.tokens) - 1;
    const int seen = last >= first + t * P.tokens ? s.limit(P, last) : 0;
    const int full = seen > 0 ? (seen - 1) / P.span : 0;
    tiles[t] = seen > 0 ? full * P.per_span + (seen - full * P.span + kRows - 1) / kRows : 0;
    n_tiles = max(n_tiles, tiles[t]);
  }
  // the key tile that the sequence ends inside, where this block reads it: the last one
  int ragged = -1;
  if (n_tiles > 0 && s.m - (((n_tiles - 1) / P.per_span) * P.span + ((n_tiles - 1) % P.per_span) * kRows) < kRows) ragged = n_tiles - 1;

  if (tid == 0) {
    mbar_init(&c.q_full, 1);
    mbar_init(&c.v_tail, 1);
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&c.kv_full[i], 1);
      mbar_init(&c.kv_empty[i], 1);
    }
    for (int t = 0; t < TILES; ++t) {
      mbar_init(&c.s_full[t], 1);
      for (int i = 0; i < kParts; ++i) mbar_init(&c.p_full[t][i], 4);
      mbar_init(&c.pv_done[t], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kSoftmaxWarps) tmem_alloc(&c.tmem, S::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;  // S of tile t at column 128 t, O at kO + D t

  // (registers of a block, two tiles: 256 x 208 + 128 x 80 <= 384 x 168 at launch; one: 128 x (200 + 56) = 256 x 128)
  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kLess));
    if (warp == kSoftmaxWarps + 1) {
    // ---- loads
    if (n_tiles > 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(&c.q_full, (uint32_t)(TILES * HALVES * 128) * P.tokens * P.group);
        for (int t = 0; t < TILES; ++t)
          for (int h = 0; h < HALVES; ++h)
            tma_load_3d(sq + t * S::kTile + h * (kRows * 128), &P.tq, 64 * h, kvh * P.group, s.q0 + first + t * P.tokens,
                        &c.q_full);
      }
      const int boxes = kRows / P.box;
      const int pages = a.pages.page_table ? (s.m + a.pages.page_size - 1) / a.pages.page_size : 1;
      int issued = 0;
      bool fine = true;
      for (int i = 0; i < 2 * n_tiles && fine; ++i) {
        const int stage = i % S::kStages, j = i >> 1;
        if (i >= S::kStages) fine = await(c, &c.kv_empty[stage], (i / S::kStages - 1) & 1, a.status);
        if (!fine) break;
        uint64_t* full = i == 2 * ragged + 1 ? &c.v_tail : &c.kv_full[stage];
        if (lane == 0) mbar_arrive_expect_tx(full, S::kTile);
        __syncwarp();
        if (lane < boxes) {
          int page = 0, row;
          if (!a.pages.page_table) {
            row = s.k0 + j * kRows;
          } else {
            const int key = (j / P.per_span) * P.span + (j % P.per_span) * kRows + lane * P.box;
            const int at = key / a.pages.page_size;
            row = key % a.pages.page_size;
            page = at < pages ? page_of(a.pages, c.seq, at, a.status) : -1;
            if (page < 0) page = a.pages.n_pages;  // out of range: the box reads as zeros
          }
          unsigned char* dst = ring + stage * S::kTile + lane * P.box * 128;
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            tma_load_4d(dst + h * (kRows * 128), (i & 1) ? &P.tv : &P.tk, 64 * h, row, kvh, page, full);
        }
        __syncwarp();
        issued = i + 1;
      }
      // no copy is in flight when the block leaves, even if another role has given up
      drain(&c.q_full, 0);
      for (int i = max(0, issued - S::kStages); i < issued; ++i) {
        if (i == 2 * ragged + 1) drain(&c.v_tail, 0);
        else drain(&c.kv_full[i % S::kStages], (i / S::kStages) & 1);
      }
    }
    } else if (warp == kSoftmaxWarps) {
      // ---- MMAs, by one thread (elect.sync: the compiler keeps the descriptors in uniform registers)
      if (n_tiles > 0 && elect_one()) {
        constexpr uint32_t id_qk = idesc<T>(kRows, false), id_pv = idesc<T>(D, true);
        const uint32_t q_lo = desc_lo(sq, 1), k_lo = desc_lo(ring, 1), v_lo = desc_lo(ring, kRows * 128 / 16);
        auto qk = [&](int t, int stage) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k / 4) * (kRows * 128) + (k % 4) * 32) / 16;
            umma_ss(tmem + 128u * t, q_lo + t * (S::kTile / 16) + off, k_lo + stage * (S::kTile / 16) + off, id_qk, k != 0);
          }
          umma_commit(&c.s_full[t]);
        };
        auto pv = [&](int t, int stage, int part, bool more) {
#pragma unroll
          for (int i = 0; i < kRows / 16 / kParts; ++i) {
            const int k = part * (kRows / 16 / kParts) + i;
            umma_ts(tmem + kO + D * t, tmem + 128u * t + 8u * k, v_lo + stage * (S::kTile / 16) + 128u * k, id_pv, more || i);
          }
        };
        bool fine = await_lane(c, &c.q_full, 0, a.status) && await_lane(c, &c.kv_full[0], 0, a.status);
        if (fine) {
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < TILES; ++t)
            if (tiles[t] > 0) qk(t, 0);
          umma_commit(&c.kv_empty[0]);
        }
        for (int j = 0; j < n_tiles && fine; ++j) {
          const int iv = 2 * j + 1, ik = 2 * j + 2, sv = iv % S::kStages, sk = ik % S::kStages;
          fine = await_lane(c, &c.kv_full[sv], (iv / S::kStages) & 1, a.status);
          if (!fine) break;
          bool k_here = false;
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            if (j < tiles[t]) {
#pragma unroll
              for (int i = 0; i < kParts; ++i) {
                fine = fine && await_lane(c, &c.p_full[t][i], j & 1, a.status);
                if (!fine) break;
                tc_fence_after();
                pv(t, sv, i, j > 0 || i > 0);
              }
              if (!fine) break;
              umma_commit(&c.pv_done[t]);
            }
            if (j + 1 < tiles[t]) {
              if (!k_here) fine = await_lane(c, &c.kv_full[sk], (ik / S::kStages) & 1, a.status);
              if (!fine) break;
              tc_fence_after();
              k_here = true;
              qk(t, sk);
            }
          }
          umma_commit(&c.kv_empty[sv]);
          if (j + 1 < n_tiles) umma_commit(&c.kv_empty[sk]);
        }
      }
      __syncwarp();
    } else if (warp == kSoftmaxWarps + 2) {
      // ---- value rows behind the sequence's last key may hold anything, NaN too, and meet probabilities of zero:
      // cleared, before the tile counts as full
      if (ragged >= 0 && await(c, &c.v_tail, 0, a.status)) {
        const int live = s.m - ((ragged / P.per_span) * P.span + (ragged % P.per_span) * kRows);
        unsigned char* v = ring + (2 * ragged + 1) % S::kStages * S::kTile + live * 128;
        for (int i = lane; i < (kRows - live) * 8; i += 32)
#pragma unroll
          for (int h = 0; h < HALVES; ++h) *reinterpret_cast<uint4*>(v + h * (kRows * 128) + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.kv_full[(2 * ragged + 1) % S::kStages]);
      }
    }
  } else {
    // ---- softmax: a thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kMore));
    const int t = warp >> 2, r = tid & 127;
    const uint32_t ts = tmem + ((uint32_t)(warp & 3) << 21) + 128u * t;
    const uint32_t to = tmem + ((uint32_t)(warp & 3) << 21) + kO + D * t;
    const int token = first + t * P.tokens + r / P.group;
    const bool row_live = r < P.tokens * P.group && token < s.n;
    const int limit = row_live ? s.limit(P, token) : 0;
    float m = 0.f, l = 0.f;
    bool fine = true;
    for (int j = 0; j < tiles[t] && fine; ++j) {
      fine = await(c, &c.s_full[t], j & 1, a.status);
      if (!fine) break;
      tc_fence_after();
      uint32_t x[kRows];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, x + 32 * i);
      tmem_wait_ld();
      const int sub = (j % P.per_span) * kRows;
      const int live = min(limit - ((j / P.per_span) * P.span + sub), P.span - sub);  // columns the row sees
      const bool masked = __any_sync(~0u, live < kRows);
      if (masked) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (i >= live) x[i] = 0xff800000u;
      }
      float part[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kRows; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          part[e] = fmaxf(fmaxf(part[e], __uint_as_float(x[i + e])), __uint_as_float(x[i + 4 + e]));
      float top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
      top *= P.scale_log2;
      if (j == 0) {
        m = top == -INFINITY ? 0.f : top;
      } else if (__any_sync(~0u, top > m + kSlack)) {
        fine = await(c, &c.pv_done[t], (j - 1) & 1, a.status);
        if (!fine) break;
        tc_fence_after();
        const float up = top > m + kSlack ? top : m, f = ex2(m - up);
        m = up;
        l *= f;
#pragma unroll
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          tmem_ld32(to + i, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tmem_st32(to + i, o);
        }
      }
      // (a masked score's probability is an exact zero only over the MUFU)
      l += masked ? exponentials<T, 0>(x, P.scale_log2, m, ts, c.p_full[t], lane)
                  : exponentials<T, S::kFma>(x, P.scale_log2, m, ts, c.p_full[t], lane);
    }
    if (tiles[t] > 0 && fine) {
      fine = await(c, &c.pv_done[t], (tiles[t] - 1) & 1, a.status);
      tc_fence_after();
    }
    if (fine) {
      const float inv = limit > 0 ? 1.f / l : 0.f;
      T* out = static_cast<T*>(a.out) + (long long)(s.q0 + token) * a.o_row_stride +
               (long long)(kvh * P.group + r % P.group) * a.o_head_stride;
#pragma unroll
      for (int i = 0; i < D; i += 32) {
        uint32_t o[32];
        if (tiles[t] > 0) {
          tmem_ld32(to + i, o);
          tmem_wait_ld();
        }
        if (row_live) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (limit > 0) {
              w.x = Elem<T>::pack(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
              w.y = Elem<T>::pack(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
              w.z = Elem<T>::pack(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
              w.w = Elem<T>::pack(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
            }
            *reinterpret_cast<uint4*>(out + i + e) = w;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmem);
  }
}

template <class T, int D, int TILES>
mk_status launch(PromptParams& P, cudaStream_t s, std::string& err) {
  using S = Shape<D, TILES>;
  const long long blocks = (long long)P.a.n_tokens / (TILES * P.tokens) + P.a.batch;
  if (blocks * P.a.pages.n_kv_heads > 0x7fffffffll) {
    err = "too many row tiles for one launch";
    return MK_ERR_UNSUPPORTED;
  }
  P.blocks = (int)blocks;
  Device dev;
  cudaError_t e = current_device(dev);
  if (e == cudaSuccess) e = allow<prompt_kernel<T, D, TILES>>(dev, S::kSmem);
  if (e != cudaSuccess) return cuda_result(e, "mk_prompt_attention attributes", err);
  prompt_kernel<T, D, TILES><<<P.blocks * P.a.pages.n_kv_heads, S::kThreads, S::kSmem, s>>>(P);
  return cuda_result(cudaGetLastError(), "mk_prompt_attention launch", err);
}

}  // namespace

mk_status launch_prompt(const mk_prompt_args& a, void* stream, std::string& err) {
  PromptParams P;
  P.a = a;
  const mk_kv_pages& g = a.pages;
  const int D = g.head_dim;
  P.scale_log2 = (a.scale > 0.f ? a.scale : 1.f / std::sqrt((float)D)) * 1.4426950408889634f;
  P.group = a.n_q_heads / g.n_kv_heads;
  P.tokens = kRows / P.group;
  const bool paged = g.page_table != nullptr;
  P.box = paged && g.page_size < kRows ? g.page_size : kRows;
  P.span = paged ? std::max(g.page_size, kRows) : std::max(g.page_size, 1);
  P.per_span = (P.span + kRows - 1) / kRows;
  {
    const long long dims[3] = {D, a.n_q_heads, a.n_tokens}, strides[2] = {a.q_head_stride, a.q_row_stride};
    const int box[3] = {64, P.group, P.tokens};
    if (!encode_map(&P.tq, g.dtype, a.q, 3, dims, strides, box)) {
      err = "the driver takes no tensor map of q's strides";
      return MK_ERR_UNSUPPORTED;
    }
  }
  // (no keys at all: nothing is loaded, the maps are those of q)
  P.tk = P.tv = P.tq;
  if (g.n_pages > 0 && g.page_size > 0 && !encode_pages(&P.tk, &P.tv, g, P.box)) {
    err = "the driver takes no tensor map of the keys' strides";
    return MK_ERR_UNSUPPORTED;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (g.dtype == MK_DTYPE_BF16)
    return D == 64 ? launch<__nv_bfloat16, 64, kTiles64>(P, s, err) : launch<__nv_bfloat16, 128, 2>(P, s, err);
  return D == 64 ? launch<__half, 64, kTiles64>(P, s, err) : launch<__half, 128, 2>(P, s, err);
}

}  // namespace mk
