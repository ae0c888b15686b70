// prompt_attn.cu — mk_prompt_attention: attention of packed prompts over packed
// or paged keys, on tcgen05.
//
// Mathematics: out_i = sum_j p_ij v_j / sum_j p_ij, p_ij = 2^(c (q_i.k_j) - m_i),
// c = scale log2 e, in one pass over the keys with a running reference m_i.
// m_i follows the running maximum only when that has grown by more than 8 in
// the exponent (a published idea for attention on this GPU): the probabilities
// then stay below 2^8, exact in the same way, and the accumulated output is
// rescaled a few times a row instead of at every tile.  P is rounded to the
// type for its product, as the tensor cores take it; its sum is that of the
// unrounded values in fp32.  A remainder of P beside it, as single tokens have
// it, would be half as many MMAs again and is left out: the error is 1.25 times
// that of a form rounded once at the end (bf16 2.0e-3 against 1.6e-3, fp16
// 2.5e-4 against 2.0e-4, root mean square).
//
// Rows: the G = n_q_heads / n_kv_heads query heads that share a kv head are
// stacked, so a tile of 128 rows is floor(128 / G) tokens times G heads (one
// TMA box [tokens][G][64]); a short prompt fills a tile G times better and the
// causal diagonal is G times narrower than with one head per tile.
//
// A block holds one such tile (D = 64, two blocks an SM) or two (D = 128, one
// block) and streams the keys past them:
//   4 warps a tile:  softmax, a thread per row: S from TMEM to registers,
//                    maximum, exponentials, P (16 bit) back to TMEM, at the end
//                    O / l to global memory;
//   a warp:          one thread issues the MMAs, S = Q K^T (Q, K from shared
//                    memory, both K-major) and O += P V (P from TMEM, V from
//                    shared memory, its N = dimensions contiguous);
//   a warp:          TMA loads, K and V tiles of 128 keys in a ring;
//   a warp:          clears the rows of V behind a sequence's last key;
//   a warp:          fetches the block's next piece of work (cluster launch
//                    control: numbers of blocks that have not begun).
// While one tile is in its softmax, the other has the tensor pipe.  Where few
// rows meet many keys, the keys are cut into pieces that a second kernel joins.
//
// Bound: per tile of 128 x 128 scores the exponentials take 1,024 cycles of the
// MUFU, the products 1,024 of the tensor pipe at D = 128 and 512 at D = 64.
// Measured (one B200; packed causal prompts of 64 to 4,096 tokens, 32/8 heads):
// a block takes 1.58 us a tile at D = 64 (two blocks an SM) and 1.75 us a pair
// of tiles at D = 128, that is 1,350 and 1,500 cycles a tile: a row's chain (S
// ready, maximum, exponentials, P, the product's wait) and its ~600
// instructions on two softmax warps a scheduler.  A piece of work's way in and
// out takes 4.0 and 5.0 us more: its first loads and scores, O to memory by
// the warps that would be in the next softmax.  16k tokens, 32 heads of 128:
// 1.75 ms for a call alone (1,260 TFLOP/s), 1.94 to 2.0 when repeated (1,100
// to 1,130, the power limit).  The instances spill 68 bytes (D = 64) and 16
// (D = 128) of a thread's registers.
// Tried and slower: two threads a row (2.13 against 1.80 ms on 16k tokens), an
// eighth to a half of the exponentials as a polynomial on the FMA pipes (equal
// at an eighth, 10 % slower at 3/8), two tiles a block at D = 64 (222 against
// 204 us on eight packed prompts).
#include <algorithm>
#include <cmath>

#include "prompt_ring.hpp"
#include "serve.cuh"

namespace mk {
namespace {

constexpr int kRows = 128;       // rows of a tile, keys of a tile
constexpr int kTiles64 = 1;      // row tiles of a block at D = 64
constexpr int kParts = 2;        // halves of a P tile, handed to the MMAs one by one
constexpr int kShares = 2;       // of the work for each resident block (see find_cut)
constexpr int kMostPieces = 64;  // of a block's keys
constexpr int kLeastTiles = 6;   // key tiles of a piece: a block's way in and out costs two to three
constexpr float kSlack = 8.f;    // log2 growth of the maximum that is left to the probabilities
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
  // At D = 64 TMEM holds P beside S, so S of the next key tile is computed while this one is in its softmax; at
  // D = 128 S and O take all of it and P lies over S.
  static constexpr bool kApart = D == 64;
  static constexpr int kP = kApart ? TILES * (kRows + D) : 0, kPStep = kApart ? 64 : 128;  // P of tile t at column kP + kPStep t
  static constexpr int kTile = kRows * D * 2;        // bytes of 128 rows
  static constexpr int kStages = D == 64 ? 5 : 4;            // ring of K and V tiles
  static constexpr int kPartial = TILES * kRows * (D + 2);   // floats of a piece's result: m, l, O of each row tile
  static constexpr int kSmem = (TILES + kStages) * kTile + 1024;
};

struct PromptParams {
  CUtensorMap tq, tk, tv;
  mk_prompt_args a;
  float scale_log2;
  int group, tokens;   // G; tokens of a row tile
  int span, per_span;  // keys of a page (or of all), key tiles that cover them
  int box;             // key rows of a TMA box
  int shares;          // equal shares that the call's work is cut into
  float* partial;      // results of pieces, or NULL: no sequence is cut into pieces
  int slots;           // pieces that fit there
  int out32;           // every row of out starts on 32 bytes
};

// One piece of work: a block's row tiles of one kv head against key tiles lo .. lo + max(count).
struct Item {
  int live;           // 0: no more work
  int seq, kvh, first; // first: the block's first query within its sequence
  int q0, n, k0, m;   // of the sequence (Seq)
  int lo, count[2];   // first key tile; key tiles that each row tile sees from there
  int slot;           // where the piece's result goes, or -1: to the output
};

struct Control {
  uint64_t q_full, q_empty, kv_full[5], kv_empty[5], s_full[2], s_read[2], p_full[2][kParts], pv_done[2], v_tail[kTails];
  uint64_t item_full[2], item_empty[2], next_block;
  uint4 answer;       // of the request for the next block's number
  Item item[2];
  uint32_t tmem;
  int abort;
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
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : MK_R8(r, 0), MK_R8(r, 8)
      : "r"(addr));
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
// p = 2^(c s - m) of 64 scores, as 16-bit pairs to TMEM at `dst`, added to
// `sum` two by two.  MAX: the maximum of these 64 and of 64 more in `others`
// is taken on the way, in the issue slots that the MUFU leaves free.
template <class T, bool MAX>
__device__ __forceinline__ void exponentials(const uint32_t* x, const uint32_t* others, float c, float m, uint32_t dst,
                                             uint64_t& sum, float& top) {
  const uint64_t cc = pair(c, c), mm = pair(-m, -m);
  uint64_t part[2] = {0, 0};
  float best[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 64; i += 32) {
    uint32_t p[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int at = i + 2 * e;
      const float2 u = both(fma2(pair(__uint_as_float(x[at]), __uint_as_float(x[at + 1])), cc, mm));
      const float2 y = make_float2(ex2(u.x), ex2(u.y));
      part[e & 1] = add2(part[e & 1], pair(y.x, y.y));
      p[e] = Elem<T>::pack(y.x, y.y);
      if (MAX) {
        best[e & 1] = fmaxf(fmaxf(best[e & 1], __uint_as_float(x[at])), __uint_as_float(x[at + 1]));
        best[2 + (e & 1)] = fmaxf(fmaxf(best[2 + (e & 1)], __uint_as_float(others[at])), __uint_as_float(others[at + 1]));
      }
    }
    tmem_st16(dst + i / 2, p);
  }
  sum = add2(part[0], part[1]);
  if (MAX) top = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]));
}
// a part of P is in TMEM: announced
__device__ __forceinline__ void announce(uint64_t* ready, int lane) {
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(ready);
}

// 32 bytes to a 32-byte boundary: a whole sector a lane
__device__ __forceinline__ void store32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), MK_W8(r, 0) : "memory");
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
      // (a pool without pages holds no keys, whatever the table names: there is no tensor map of it to load by)
      const int cap = a.pages.n_pages > 0 ? a.pages.table_width * a.pages.page_size : 0, l = __ldg(a.kv_lens + b);
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

// Which of an item's key tiles the sequence ends inside: its last one or none (-1).
__device__ __forceinline__ int ragged_tile(const PromptParams& P, const Item& i, int n_tiles) {
  const int j = i.lo + n_tiles - 1;
  return n_tiles > 0 && i.m - ((j / P.per_span) * P.span + (j % P.per_span) * kRows) < kRows ? n_tiles - 1 : -1;
}

// How long rows of keys are cut: sequences whose last block sees more than
// `above` key tiles, into pieces of about `piece`.
struct Cut {
  int above, piece;
};

// How a sequence's work is laid out: row blocks, key tiles, pieces.
template <int TILES>
struct Work {
  int blocks, tiles, pieces;  // tiles: of the last block, which sees the most keys
  // key tiles that cover the first `seen` keys
  static __device__ __forceinline__ int cover(const PromptParams& P, int seen) {
    const int full = seen > 0 ? (seen - 1) / P.span : 0;
    return seen > 0 ? full * P.per_span + (seen - full * P.span + kRows - 1) / kRows : 0;
  }
  __device__ __forceinline__ void load(const PromptParams& P, const Seq& s, Cut cut) {
    blocks = (s.n + TILES * P.tokens - 1) / (TILES * P.tokens);
    tiles = blocks > 0 ? cover(P, s.m) : 0;
    pieces = blocks > 0 && tiles > cut.above ? min(kMostPieces, (tiles + cut.piece - 1) / cut.piece) : 1;
  }
  // key tiles that the row tiles of a block see, and in how many pieces: a block that sees no more than one piece's is
  // the business of its first
  __device__ __forceinline__ int seen(const PromptParams& P, const Seq& s, int block, int (&each)[2]) const {
    int most = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int first = (block * TILES + t) * P.tokens, last = min(s.n, first + P.tokens) - 1;
      each[t] = t < TILES && last >= first ? cover(P, s.limit(P, last)) : 0;
      most = max(most, each[t]);
    }
    return most;
  }
  __device__ __forceinline__ int pieces_of(int most, Cut cut) const { return most > cut.piece ? pieces : 1; }
  // the key tiles of all its blocks, as the mean of the first and the last
  __device__ __forceinline__ long long total(const PromptParams& P, const Seq& s) const {
    if (blocks == 0) return 0;
    const int head = cover(P, s.limit(P, min(s.n, TILES * P.tokens) - 1));
    return (long long)blocks * (head + tiles + 1) / 2 * P.a.pages.n_kv_heads;
  }
};

// The whole call's work in kShares shares for each block that the device holds
// gives the key tiles of a piece, not below kLeastTiles.  Sequences that see
// more are cut, but only where one sees more than twice a resident block's
// share: its blocks would be the last to end, while cutting what evens out by
// itself costs more than it gives (2,000 tokens, 24 heads of 64: 57 us cut, 42
// whole).  No more than 4 times the shares carry results to be joined (blocks *
// tiles <= 2 total, and pieces < 2 tiles / piece where there are two or more).
// Found by one warp, alike wherever it is asked for.
template <int TILES>
__device__ Cut find_cut(const PromptParams& P) {
  if (!P.partial) return {0x7fffffff, 0};  // (nothing is cut, all sequences are walked at once)
  long long sum = 0;
  int most = 0;
  for (int b = threadIdx.x & 31; b < P.a.batch; b += 32) {
    Seq s;
    s.load(P, b);
    Work<TILES> w;
    w.load(P, s, {0x7fffffff, 0});
    sum += w.total(P, s);
    most = max(most, w.tiles);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  most = __reduce_max_sync(~0u, most);
  const long long share = (sum + P.shares - 1) / P.shares;
  const int piece = (int)min(0x7fffffffll, max((long long)kLeastTiles, share));
  return {most >= 2 * kLeastTiles && most > 2 * kShares * share ? piece : 0x7fffffff, piece};
}

// A warp walks the sequences, 32 at a time, for the one that item or joined
// block number `want` falls into; numbers mostly ascend, and it goes on from
// where it was.  Sequences of more key tiles than a piece's come first, so that
// the last work to begin is short.
template <int TILES, bool JOIN>
struct Walk {
  int b0 = 0;
  bool second = false;  // the walk over the shorter sequences
  Cut cut;
  long long base = 0, slot_base = 0;  // items, and results of pieces, of the sequences before b0
  long long before, count, slots, slot_before;
  Seq s;
  Work<TILES> w;
  __device__ __forceinline__ void fill(const PromptParams& P) {
    const int lane = threadIdx.x & 31, b = b0 + lane;
    count = slots = 0;
    w.blocks = w.tiles = 0;
    w.pieces = 1;
    if (b < P.a.batch) {
      s.load(P, b);
      w.load(P, s, cut);
      const long long rows = (w.tiles > cut.piece) == second ? 0 : (long long)w.blocks * P.a.pages.n_kv_heads;
      slots = w.pieces > 1 ? rows * w.pieces : 0;
      count = JOIN ? (w.pieces > 1 ? rows : 0) : rows * w.pieces;
    }
    before = count;
    slot_before = slots;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(~0u, before, d), p = __shfl_up_sync(~0u, slot_before, d);
      if (lane >= d) {
        before += o;
        slot_before += p;
      }
    }
    before -= count;
    slot_before -= slots;
  }
  __device__ __forceinline__ void begin(const PromptParams& P) {
    cut = find_cut<TILES>(P);
    fill(P);
  }
  // the lane whose sequence holds `want`, or -1
  __device__ __forceinline__ int find(const PromptParams& P, long long want) {
    if (want < base) {
      base = slot_base = 0;
      b0 = 0;
      second = false;
      fill(P);
    }
    for (;;) {
      const unsigned hit = __ballot_sync(~0u, want >= base + before && want < base + before + count);
      if (hit) return __ffs(hit) - 1;
      const bool at_end = b0 + 32 >= P.a.batch;
      if (at_end && second) return -1;
      base += __shfl_sync(~0u, before + count, 31);
      slot_base += __shfl_sync(~0u, slot_before + slots, 31);
      b0 = at_end ? 0 : b0 + 32;
      second = second || at_end;
      fill(P);
    }
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

  if (tid == 32) {
    prefetch_map(&P.tq);
    prefetch_map(&P.tk);
    prefetch_map(&P.tv);
  }
  if (tid == 0) {
    c.abort = 0;
    mbar_init(&c.q_full, 1);
    mbar_init(&c.q_empty, 1);
    for (int i = 0; i < kTails; ++i) mbar_init(&c.v_tail[i], 1);
    mbar_init(&c.next_block, 1);
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&c.kv_full[i], 1);
      mbar_init(&c.kv_empty[i], 1);
    }
    for (int t = 0; t < TILES; ++t) {
      mbar_init(&c.s_full[t], 1);
      mbar_init(&c.s_read[t], 4);
      for (int i = 0; i < kParts; ++i) mbar_init(&c.p_full[t][i], 4);
      mbar_init(&c.pv_done[t], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.item_full[i], 1);
      mbar_init(&c.item_empty[i], kSoftmaxWarps + 3);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kSoftmaxWarps) tmem_alloc(&c.tmem, S::kTmem);
  Walk<TILES, false> walk;
  if (warp == kSoftmaxWarps + 3) {  // (every other role begins with an item that this warp hands out)
    dep_wait();
    dep_launch();
    walk.begin(P);  // (its loads travel while the block is set up)
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;  // S of tile t at column 128 t, O at kO + D t

  // Every role runs the block's items one after the other, each at its own pace: the loads of the next item begin
  // while this one is in its last softmax and on its way out.
  // (registers of a block, two tiles: 256 x 208 + 128 x 80 <= 384 x 168 at launch; one: 128 x (200 + 56) = 256 x 128)
  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kLess));
    if (warp == kSoftmaxWarps + 3) {
      // ---- items: this block's number first, then those of blocks that have not begun, taken over one at a time
      const int kv_heads = a.pages.n_kv_heads;
      long long number = blockIdx.x;
      bool fine = true;
      int k = 0;
      for (uint32_t asked = 0; fine; ++asked) {
        const int at = walk.find(P, number);
        if (at >= 0) {
          Item& it = c.item[k & 1];
          int idle = 0;
          if (lane == at) {  // (the lane that writes the item also hands it out: its arrival is behind its writes)
            const Seq& s = walk.s;
            const int numbered = walk.w.pieces, r = (int)(number - walk.base - walk.before);
            const int block = walk.w.blocks - 1 - r / (kv_heads * numbered);  // a sequence's last rows see the most keys: first
            const int kvh = r % kv_heads, piece = r / kv_heads % numbered;
            int tiles[2];
            const int n = walk.w.seen(P, s, block, tiles), pieces = walk.w.pieces_of(n, walk.cut);
            idle = piece >= pieces;
            const int lo = (int)((long long)n * piece / pieces), hi = (int)((long long)n * (piece + 1) / pieces);
            it.live = 1;
            it.first = block * TILES * P.tokens;
            it.seq = walk.b0 + lane;
            it.kvh = kvh;
            it.q0 = s.q0;
            it.n = s.n;
            it.k0 = s.k0;
            it.m = s.m;
            it.lo = lo;
#pragma unroll
            for (int t = 0; t < 2; ++t) it.count[t] = max(0, min(tiles[t], hi) - lo);
            it.slot = -1;
            if (pieces > 1) it.slot = (int)(walk.slot_base + walk.slot_before) + (block * kv_heads + kvh) * numbered + piece;
            if (!idle) mbar_arrive(&c.item_full[k & 1]);
          }
          if (!__any_sync(~0u, idle)) {
            fine = await(c, &c.item_empty[k & 1], (k >> 1) & 1, a.status);  // all roles have it; the other slot is free
            if (!fine) break;
            ++k;
          }
        }
        uint32_t taken = 0, id = 0;
        if (lane == 0) {
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(&c.next_block, 16);
          asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                           smem_u32(&c.answer)),
                       "r"(smem_u32(&c.next_block))
                       : "memory");
        }
        fine = await(c, &c.next_block, asked & 1, a.status);
        if (!fine) break;
        asm volatile(
            "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
            : "=r"(taken), "=r"(id)
            : "r"(smem_u32(&c.answer))
            : "memory");
        __syncwarp();
        if (!taken) break;
        number = id;
      }
      if (lane == 0) {
        c.item[k & 1].live = 0;
        mbar_arrive(&c.item_full[k & 1]);
      }
    } else if (warp == kSoftmaxWarps + 1) {
      // ---- loads
      int it = 0, loaded = 0, tails = 0;  // tiles of the ring, items with keys, ragged value tiles so far
      bool fine = true;
      for (int k = 0; fine; ++k) {
        fine = await(c, &c.item_full[k & 1], (k >> 1) & 1, a.status);
        if (!fine) break;
        const Item item = c.item[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.item_empty[k & 1]);
        if (!item.live) break;
        const int n_tiles = max(item.count[0], item.count[1]);
        if (n_tiles == 0) continue;
        if (loaded > 0) fine = await(c, &c.q_empty, (loaded - 1) & 1, a.status);
        if (!fine) break;
        ++loaded;
        if (lane == 0) {
          mbar_arrive_expect_tx(&c.q_full, (uint32_t)(TILES * HALVES * 128) * P.tokens * P.group);
          for (int t = 0; t < TILES; ++t)
            for (int h = 0; h < HALVES; ++h)
              tma_load_3d(sq + t * S::kTile + h * (kRows * 128), &P.tq, 64 * h, item.kvh * P.group,
                          item.q0 + item.first + t * P.tokens, &c.q_full);
        }
        const int boxes = kRows / P.box, ragged = ragged_tile(P, item, n_tiles);
        const int pages = a.pages.page_table ? (item.m + a.pages.page_size - 1) / a.pages.page_size : 1;
        for (int i = 0; i < 2 * n_tiles; ++i, ++it) {
          const bool is_v = ring_is_v<S::kApart>(i, n_tiles);
          const int stage = it % S::kStages, rel = ring_tile<S::kApart>(i, n_tiles);
          const int j = item.lo + rel;
          if (it >= S::kStages) fine = await(c, &c.kv_empty[stage], (it / S::kStages - 1) & 1, a.status);
          if (!fine) break;
          uint64_t* full = is_v && rel == ragged ? &c.v_tail[tail_slot(tails)] : &c.kv_full[stage];
          if (lane == 0) mbar_arrive_expect_tx(full, S::kTile);
          __syncwarp();
          if (lane < boxes) {
            int page = 0, row;
            if (!a.pages.page_table) {
              row = item.k0 + j * kRows;
            } else {
              const int key = (j / P.per_span) * P.span + (j % P.per_span) * kRows + lane * P.box;
              const int at = key / a.pages.page_size;
              row = key % a.pages.page_size;
              page = at < pages ? page_of(a.pages, item.seq, at, a.status) : -1;
              if (page < 0) page = a.pages.n_pages;  // out of range: the box reads as zeros
            }
            unsigned char* dst = ring + stage * S::kTile + lane * P.box * 128;
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
              tma_load_4d(dst + h * (kRows * 128), is_v ? &P.tv : &P.tk, 64 * h, row, item.kvh, page, full);
          }
          __syncwarp();
        }
        tails += ragged >= 0;
      }
      // no copy is in flight when the block leaves, even if another role has given up
      if (loaded > 0) drain(&c.q_full, (loaded - 1) & 1);
      for (int i = max(0, it - S::kStages); i < it; ++i) drain(&c.kv_full[i % S::kStages], (i / S::kStages) & 1);
    } else if (warp == kSoftmaxWarps) {
      // ---- MMAs, by one thread (elect.sync: the compiler keeps the descriptors in uniform registers)
      if (elect_one()) {
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
            umma_ts(tmem + kO + D * t, tmem + S::kP + S::kPStep * t + 8u * k, v_lo + stage * (S::kTile / 16) + 128u * k, id_pv, more || i);
          }
        };
        int it = 0, loaded = 0, done[2] = {0, 0}, asked[2] = {0, 0};  // tiles of the ring, items with keys, P and S tiles of each row tile so far
        bool fine = true;
        for (int k = 0; fine; ++k) {
          fine = await_lane(c, &c.item_full[k & 1], (k >> 1) & 1, a.status);
          if (!fine) break;
          const int live = c.item[k & 1].live;
          int count[TILES], n_tiles = 0;
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            count[t] = c.item[k & 1].count[t];
            n_tiles = max(n_tiles, count[t]);
          }
          mbar_arrive(&c.item_empty[k & 1]);
          if (!live) break;
          if (n_tiles == 0) continue;
          fine = await_lane(c, &c.q_full, loaded & 1, a.status);
          ++loaded;
          // S of key tile j of every row tile that sees it
          auto scores = [&](int j) {
            const int i = it + ring_k<S::kApart>(j);
            fine = fine && await_lane(c, &c.kv_full[i % S::kStages], (i / S::kStages) & 1, a.status);
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              if (j >= count[t] || !fine) continue;
              // the S before has been read (where P lies over S: its P has been multiplied, which is issued before this)
              if (S::kApart && asked[t] > 0) fine = await_lane(c, &c.s_read[t], (asked[t] - 1) & 1, a.status);
              if (!fine) continue;
              ++asked[t];
              tc_fence_after();
              qk(t, i % S::kStages);
            }
            umma_commit(&c.kv_empty[i % S::kStages]);
            if (j + 1 == n_tiles) umma_commit(&c.q_empty);
          };
          // O += P V of key tile j and row tile t
          auto values = [&](int t, int j, int stage) {
            // (the first P of an item is announced after O of the item before has been read)
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
              fine = fine && await_lane(c, &c.p_full[t][i], done[t] & 1, a.status);
              if (!fine) return;
              tc_fence_after();
              pv(t, stage, i, j > 0 || i > 0);
            }
            umma_commit(&c.pv_done[t]);
            ++done[t];
          };
          scores(0);
          for (int j = 0; j < n_tiles && fine; ++j) {
            const int iv = it + ring_v<S::kApart>(j, n_tiles), sv = iv % S::kStages;
            if constexpr (S::kApart) {
              if (j + 1 < n_tiles) scores(j + 1);
              fine = fine && await_lane(c, &c.kv_full[sv], (iv / S::kStages) & 1, a.status);
#pragma unroll
              for (int t = 0; t < TILES; ++t)
                if (j < count[t] && fine) values(t, j, sv);
              umma_commit(&c.kv_empty[sv]);
            } else {
              const int ik = it + ring_k<false>(j + 1), sk = ik % S::kStages;
              fine = await_lane(c, &c.kv_full[sv], (iv / S::kStages) & 1, a.status);
              bool k_here = false;
#pragma unroll
              for (int t = 0; t < TILES; ++t) {
                if (j < count[t] && fine) values(t, j, sv);
                if (j + 1 < count[t] && fine) {
                  if (!k_here) fine = await_lane(c, &c.kv_full[sk], (ik / S::kStages) & 1, a.status);
                  if (!fine) break;
                  tc_fence_after();
                  k_here = true;
                  ++asked[t];
                  qk(t, sk);
                }
              }
              umma_commit(&c.kv_empty[sv]);
              if (j + 1 < n_tiles) umma_commit(&c.kv_empty[sk]);
              if (j + 2 == n_tiles) umma_commit(&c.q_empty);
            }
          }
          it += 2 * n_tiles;
        }
      }
      __syncwarp();
    } else {
      // ---- value rows behind the sequence's last key may hold anything, NaN too, and meet probabilities of zero:
      // cleared, before the tile counts as full
      int it = 0, cleared = 0;
      for (int k = 0;; ++k) {
        if (!await(c, &c.item_full[k & 1], (k >> 1) & 1, a.status)) break;
        const Item item = c.item[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.item_empty[k & 1]);
        if (!item.live) break;
        const int n_tiles = max(item.count[0], item.count[1]), ragged = ragged_tile(P, item, n_tiles);
        if (ragged >= 0) {
          if (!await(c, &c.v_tail[tail_slot(cleared)], tail_parity(cleared), a.status)) break;
          ++cleared;
          const int j = item.lo + ragged, stage = (it + ring_v<S::kApart>(ragged, n_tiles)) % S::kStages;
          const int live = item.m - ((j / P.per_span) * P.span + (j % P.per_span) * kRows);
          unsigned char* v = ring + stage * S::kTile + live * 128;
          for (int i = lane; i < (kRows - live) * 8; i += 32)
#pragma unroll
            for (int h = 0; h < HALVES; ++h) *reinterpret_cast<uint4*>(v + h * (kRows * 128) + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.kv_full[stage]);
        }
        it += 2 * n_tiles;
      }
    }
  } else {
    // ---- softmax: a thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kMore));
    const int t = warp >> 2, r = tid & 127;
    const uint32_t ts = tmem + ((uint32_t)(warp & 3) << 21) + 128u * t;
    const uint32_t to = tmem + ((uint32_t)(warp & 3) << 21) + kO + D * t;
    const uint32_t tp = tmem + ((uint32_t)(warp & 3) << 21) + S::kP + S::kPStep * t;
    const int row_token = r / P.group, row_head = r % P.group;
    int done = 0;  // S tiles so far
    bool fine = true;
    for (int k = 0; fine; ++k) {
      fine = await(c, &c.item_full[k & 1], (k >> 1) & 1, a.status);
      if (!fine) break;
      const int live_item = c.item[k & 1].live, first = c.item[k & 1].first, kvh = c.item[k & 1].kvh, lo = c.item[k & 1].lo;
      const int n_here = c.item[k & 1].count[t], slot = c.item[k & 1].slot;
      Seq s;
      s.q0 = c.item[k & 1].q0;
      s.n = c.item[k & 1].n;
      s.m = c.item[k & 1].m;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.item_empty[k & 1]);
      if (!live_item) break;
      const int token = first + t * P.tokens + row_token;
      const bool row_live = r < P.tokens * P.group && token < s.n;
      const int limit = row_live ? s.limit(P, token) : 0;
      float m = -INFINITY, l = 0.f;  // m: the reference, -inf until the row has seen a key
      for (int j = 0; j < n_here && fine; ++j, ++done) {
        fine = await(c, &c.s_full[t], done & 1, a.status);
        if (!fine) break;
        tc_fence_after();
        uint32_t x[kRows];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, x + 32 * i);
        tmem_wait_ld();
        if (S::kApart) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.s_read[t]);
        }
        const int sub = ((lo + j) % P.per_span) * kRows;
        // columns that the row sees; a row that is none (behind the last token, or the tile's remainder by G) sees all,
        // or its warp would go through the mask at every tile
        const int live = row_live ? min(limit - (((lo + j) / P.per_span) * P.span + sub), P.span - sub) : kRows;
        if (__any_sync(~0u, live < kRows)) {
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            if (i >= live) x[i] = 0xff800000u;
        }
        if (S::kApart && j > 0) {  // the product before is complete: P may be written
          fine = await(c, &c.pv_done[t], (done - 1) & 1, a.status);
          if (!fine) break;
          tc_fence_after();
        }
        // The first half's probabilities are taken with the reference as it stands, the maximum beside them.  Where a
        // row's maximum has outgrown the reference (always at its first keys, seldom later), what is there is brought
        // to the maximum and the half is taken again.
        uint64_t sum[2];
        for (;;) {
          float top = 0.f;
          exponentials<T, true>(x, x + 64, P.scale_log2, m == -INFINITY ? 0.f : m, tp, sum[0], top);
          top *= P.scale_log2;
          const bool grown = top > m + kSlack;
          if (!__any_sync(~0u, grown)) break;
          const float up = grown ? top : m, f = grown ? ex2(m - up) : 1.f;  // (0 at the row's first keys)
          m = up;
          if (j > 0) {
            if (!S::kApart) {
              fine = await(c, &c.pv_done[t], (done - 1) & 1, a.status);
              if (!fine) break;
              tc_fence_after();
            }
            l *= f;
#pragma unroll
            for (int i = 0; i < D; i += 16) {
              uint32_t o[16];
              tmem_ld16(to + i, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(to + i, o);
            }
          }
        }
        if (!fine) break;
        announce(&c.p_full[t][0], lane);
        float unused;
        exponentials<T, false>(x + 64, nullptr, P.scale_log2, m == -INFINITY ? 0.f : m, tp + 32, sum[1], unused);
        announce(&c.p_full[t][1], lane);
        const float2 total = both(add2(sum[0], sum[1]));
        l += total.x + total.y;
      }
      if (!fine) break;
      if (n_here > 0) {
        fine = await(c, &c.pv_done[t], (done - 1) & 1, a.status);
        if (!fine) break;
        tc_fence_after();
      }
      if (slot >= 0) {
        // a piece's result: m and l of the rows, then O in chunks of 8 columns, [chunk][row][8], so that a warp's rows
        // lie next to one another
        float* part = P.partial + (long long)slot * S::kPartial + t * (kRows * (D + 2));
        const bool there = row_live && slot < P.slots;
        if (there) {
          part[r] = m;
          part[kRows + r] = l;
        }
        if (n_here > 0) {
#pragma unroll
          for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tmem_ld32(to + i, o);
            tmem_wait_ld();
            if (there) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) store32(part + 2 * kRows + ((i + e) / 8 * kRows + r) * 8, o + e);
            }
          }
        }
      } else {
        const float inv = limit > 0 ? 1.f / l : 0.f;
        T* out = static_cast<T*>(a.out) + (long long)(s.q0 + token) * a.o_row_stride + (long long)(kvh * P.group + row_head) * a.o_head_stride;
#pragma unroll
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          if (n_here > 0) {
            tmem_ld32(to + i, o);
            tmem_wait_ld();
          }
          if (row_live) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              w[e] = limit > 0 ? Elem<T>::pack(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv) : 0u;
            if (P.out32) {
              store32(out + i, w);
              store32(out + i + 16, w + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4*>(out + i + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
            }
          }
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmem);
  }
}

// The pieces of a (row block, kv head) joined, 32 rows of one of its row tiles
// at a time; launched while the first kernel runs.
constexpr int kJoinRows = 32;

template <class T, int D, int TILES>
__global__ void __launch_bounds__(256, 4) join_kernel(const __grid_constant__ PromptParams P) {
  using S = Shape<D, TILES>;
  constexpr int LANES = D / 4, PARTS = kRows / kJoinRows;  // a thread holds 4 values of a row
  __shared__ int at[6];
  const mk_prompt_args& a = P.a;
  const int tid = threadIdx.x;
  Walk<TILES, true> walk;
  if (tid < 32) walk.begin(P);
  for (long long number = blockIdx.x;; number += gridDim.x) {
    const int t = number / PARTS % TILES, first_row = number % PARTS * kJoinRows;
    if (tid < 32) {
      const int hit = walk.find(P, number / (PARTS * TILES));
      if (tid == 0) at[0] = 0;
      __syncwarp();
      if (tid == hit) {
        const int r = (int)(number / (PARTS * TILES) - walk.base - walk.before), kv_heads = a.pages.n_kv_heads;
        int tiles[2];
        const int n = walk.w.seen(P, walk.s, r / kv_heads, tiles);
        at[1] = (int)(walk.slot_base + walk.slot_before) + r * walk.w.pieces;  // (r = block * kv_heads + head)
        at[2] = r / kv_heads * TILES * P.tokens + t * P.tokens;
        at[3] = r % kv_heads;
        at[4] = walk.s.q0;
        at[5] = walk.s.n;
        at[0] = walk.w.pieces_of(n, walk.cut);
      }
    }
    __syncthreads();
    if (number == blockIdx.x) {
      dep_wait();
      dep_launch();
    }
    const int pieces = at[0], slot = at[1];
    if (pieces == 0 || slot + pieces > P.slots) return;
    if (pieces == 1) {  // (its first piece wrote the output)
      __syncthreads();
      continue;
    }
    const int rows = min(kJoinRows, min(P.tokens, at[5] - at[2]) * P.group - first_row);  // (rows of tokens that exist)
    const float* part = P.partial + (long long)slot * S::kPartial + t * (kRows * (D + 2));
    // a thread keeps a row's running maximum, sum and 4 output values, over four pieces at a time so that their loads
    // travel together; a piece in which the row sees no key (m = -inf) counts nothing: its output may not be there
    const int c = tid % LANES * 4;
#pragma unroll 1
    for (int row = first_row + tid / LANES; row < first_row + rows; row += 256 / LANES) {
      float m = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k0 = 0; k0 < pieces; k0 += 4) {
        float pm[4], pl[4];
        float4 po[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float* p = part + (long long)min(k0 + e, pieces - 1) * S::kPartial;
          pm[e] = k0 + e < pieces ? p[row] : -INFINITY;
          pl[e] = p[kRows + row];
          po[e] = *reinterpret_cast<const float4*>(p + 2 * kRows + (c / 8 * kRows + row) * 8 + c % 8);
        }
        const float up = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])), m);
        if (up == -INFINITY) continue;
        const float f = ex2(m - up);
        m = up;
        l *= f;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (pm[e] == -INFINITY) continue;
          const float w = ex2(pm[e] - up);
          l += w * pl[e];
          o.x += w * po[e].x, o.y += w * po[e].y, o.z += w * po[e].z, o.w += w * po[e].w;
        }
      }
      const float inv = m == -INFINITY ? 0.f : 1.f / l;
      T* out = static_cast<T*>(a.out) + (long long)(at[4] + at[2] + row / P.group) * a.o_row_stride +
               (long long)(at[3] * P.group + row % P.group) * a.o_head_stride + c;
      *reinterpret_cast<uint2*>(out) = make_uint2(Elem<T>::pack(o.x * inv, o.y * inv), Elem<T>::pack(o.z * inv, o.w * inv));
    }
    __syncthreads();  // (at is done with)
  }
}

// Whether a call may cut sequences into pieces: its row blocks could leave SMs
// idle at the end, and there may be keys enough.  With more than two blocks for
// each that the device holds the ends even out, and what looking and the second
// launch cost is saved (3 us; 5 of 190 on 6,000 tokens, 24 heads of 64).
bool may_cut(long long items, long long keys, int resident) { return items < 2ll * resident && keys >= 2ll * kLeastTiles * kRows; }

template <int D, int TILES>
long long items_of(const mk_prompt_args& a) {
  const int tokens = kRows / (a.n_q_heads / a.pages.n_kv_heads);
  return ((long long)a.n_tokens / (TILES * tokens) + a.batch) * a.pages.n_kv_heads;
}

// Results of pieces that a call can leave: by its work no more than 4 for each share (find_cut), and by its size no more
// than a block and head can be cut into, at kLeastTiles a piece (one prompt of 17 tokens over a cache of 2,048 rows: 6
// of them, not the 2,368 of the whole device).
long long slots_of(long long items, long long key_tiles, int shares) {
  const long long pieces = std::min<long long>(kMostPieces, (key_tiles + kLeastTiles - 1) / kLeastTiles);
  return std::min(4ll * shares, items * pieces);
}

// (Pages that are no multiple of a tile take more tiles than their keys fill, less than twice as many: a page that is cut
// holds at least one whole tile.)
template <int D, int TILES>
size_t bytes_of(const mk_prompt_args& a, long long max_keys, int sms) {
  using S = Shape<D, TILES>;
  const int resident = sms * S::kBlocksPerSm;
  const long long items = items_of<D, TILES>(a);
  if (!may_cut(items, max_keys, resident)) return 0;
  return slots_of(items, 2 * (max_keys / kRows) + 1, kShares * resident) * S::kPartial * sizeof(float);
}

template <class T, int D, int TILES>
mk_status launch(PromptParams& P, cudaStream_t s, std::string& err) {
  using S = Shape<D, TILES>;
  Device dev;
  cudaError_t e = current_device(dev);
  if (e == cudaSuccess) e = allow<prompt_kernel<T, D, TILES>>(dev, S::kSmem);
  if (e != cudaSuccess) return cuda_result(e, "mk_prompt_attention attributes", err);
  const mk_kv_pages& g = P.a.pages;
  const int resident = dev.sms * S::kBlocksPerSm;
  P.shares = kShares * resident;
  long long items = items_of<D, TILES>(P.a);
  const long long keys = g.page_table ? (long long)g.table_width * g.page_size : g.page_size;
  const long long slots = slots_of(items, keys / P.span * P.per_span + (keys % P.span + kRows - 1) / kRows, P.shares);
  if (P.a.workspace && P.a.workspace_bytes >= slots * S::kPartial * sizeof(float) && may_cut(items, keys, resident)) {
    P.partial = static_cast<float*>(P.a.workspace);
    P.slots = (int)slots;
    items += 2 * P.shares;  // pieces: at most tiles / piece_tiles + 1 each, blocks * tiles <= 2 total
  }
  if (items > 0x7fffffffll) {
    err = "too many row tiles for one launch";
    return MK_ERR_UNSUPPORTED;
  }
  e = mk::launch(items <= resident, prompt_kernel<T, D, TILES>, dim3((unsigned)items), S::kThreads, S::kSmem, s, 0, P);
  if (e != cudaSuccess || !P.partial) return cuda_result(e, "mk_prompt_attention launch", err);
  e = mk::launch(true, join_kernel<T, D, TILES>, dim3(4 * dev.sms), 256, 0, s, 0, P);
  return cuda_result(e, "mk_prompt_attention join launch", err);
}

}  // namespace

size_t prompt_workspace_bytes(int batch, int n_tokens, int n_q_heads, int n_kv_heads, int head_dim, long long max_keys) {
  Device dev;
  if (batch < 1 || n_tokens < 1 || n_kv_heads < 1 || n_q_heads < n_kv_heads || n_q_heads / n_kv_heads > kRows ||
      current_device(dev) != cudaSuccess)
    return 0;
  mk_prompt_args a = {};
  a.batch = batch;
  a.n_tokens = n_tokens;
  a.n_q_heads = n_q_heads;
  a.pages.n_kv_heads = n_kv_heads;
  if (head_dim <= 64) return bytes_of<64, kTiles64>(a, max_keys, dev.sms);
  return bytes_of<128, 2>(a, max_keys, dev.sms);
}

mk_status launch_prompt(const mk_prompt_args& a, void* stream, std::string& err) {
  PromptParams P;
  P.a = a;
  P.partial = nullptr;
  P.slots = 0;
  P.out32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.o_row_stride % 16 == 0 && a.o_head_stride % 16 == 0;
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
  // (no keys at all: nothing is loaded, see Seq; the maps are those of q)
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
