// append_kv.cu — mk_append_kv: new tokens' query and key rows turned to their
// positions, key and value rows stored in the cache's pages.
//
// Mathematics: pair (x, y) = (row[p], row[p + D/2]) of every query and key
// head becomes (x cos a - y sin a, y cos a + x sin a), a = position *
// theta^(-2p/D).  The frequency and the product are taken in double, since a
// far position times a frequency loses its fraction in fp32; the angle is
// brought into [-pi, pi] in double and only then handed to the fp32 sine and
// cosine.  One angle serves all heads of a token, so a block computes its
// tokens' angles once into shared memory and the heads read them there.
//
// Bound: memory.  Every row is read and written once, 16 bytes a thread and
// access; a thread turns 8 pairs (a 16-byte piece of each half of a head).
// Measured (one B200, in a graph, inputs that are not in L2): 8,148 tokens of
// 32/8 heads of 128 (200 MB) in 39 us, 5.1 TB/s; 64 tokens of 64 sequences in
// 3.3 us.
#include <cmath>

#include "serve.cuh"

namespace mk {
namespace {

constexpr int kThreads = 256;
// 8,148 tokens: 39 us with 4 tokens a block and 2 pieces in flight, 41 with 2
// tokens, 51 with 1, 42 with 4 or 8 tokens and 4 pieces.
constexpr int kMaxTokens = 4;   // tokens of a block
constexpr int kFewTokens = 512; // up to here one (64 tokens: 3.8 us, 6.3 with 8 a block)
constexpr int kBatch = 2;       // pieces a thread has in flight

struct AppendParams {
  mk_append_args a;
  double freq[64];  // theta^(-2p/D)
};

template <class T, int D, int TOK>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams P) {
  constexpr int H = D / 2, PIECES = D / 16;  // pairs of a head; 16-byte pieces of half a head
  const mk_append_args& a = P.a;
  __shared__ __align__(16) float2 turn[TOK][H];  // (cos, sin)
  __shared__ long long dest[TOK];          // first element of the token's row in head 0 of its page, or -1
  __shared__ int where[TOK];               // position, or -1: row behind the last sequence
  const int t0 = blockIdx.x * TOK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  dep_wait();
  dep_launch();

  // a warp per token: its sequence is the number of sequences that end at or before it
  if (warp < TOK) {
    const int t = t0 + warp;
    int n = 0;
    for (int b = lane; b < a.batch; b += 32) n += __ldg(a.cu_seqlens + b + 1) <= t;
    n = __reduce_add_sync(~0u, n);
    if (lane == 0) {
      int pos = -1;
      long long d = -1;
      if (t < a.n_tokens && n < a.batch) {
        const int begin = __ldg(a.cu_seqlens + n), ctx = __ldg(a.ctx_lens + n);
        const long long at = (long long)ctx + t - begin;
        if (begin < 0 || begin > t || ctx < 0 || at >= (long long)a.pages.table_width * a.pages.page_size) {
          if (begin <= t) report_bounds(a.status);  // (begin > t: a row before the first sequence)
        } else {
          const int page = page_of(a.pages, n, (int)(at / a.pages.page_size), a.status);
          if (page >= 0) {
            pos = (int)at;
            d = (long long)page * a.pages.page_stride + (at % a.pages.page_size) * a.pages.row_stride;
          }
        }
      }
      where[warp] = pos;
      dest[warp] = d;
    }
  } else if (blockIdx.x == 0 && warp == kThreads / 32 - 1 && a.status) {
    // meanwhile, once a call: bounds that descend or go past the rows (what they hide, no row's search can tell)
    bool bad = false;
    for (int b = lane; b < a.batch; b += 32) {
      const int begin = __ldg(a.cu_seqlens + b), end = __ldg(a.cu_seqlens + b + 1);
      bad = bad || begin < 0 || end < begin || end > a.n_tokens;
    }
    if (bad) report_bounds(a.status);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < TOK * H; i += kThreads) {
    const int tok = i / H, p = i % H;
    float2 cs = make_float2(1.f, 0.f);
    if (where[tok] > 0 && a.rope_theta != 0.0) {
      const double angle = (double)where[tok] * P.freq[p];
      const double turns = rint(angle * 0.15915494309189535);  // 1 / (2 pi)
      const float r = (float)fma(turns, -6.283185307179586, angle);
      sincosf(r, &cs.y, &cs.x);
    }
    turn[tok][p] = cs;
  }
  __syncthreads();

  // pieces: 8 elements of a head's first half and the 8 that they turn with; kBatch of them are in flight a thread
  const int hq = a.q ? a.n_q_heads : 0, hkv = a.pages.n_kv_heads;
  const int per_token = (hq + 2 * hkv) * PIECES, all = TOK * per_token;
  for (int i0 = threadIdx.x; i0 < all; i0 += kThreads * kBatch) {
    uint4 lo[kBatch], hi[kBatch];
    T* dst[kBatch];
    int turned[kBatch];  // token of the block * H + first pair, or -1: not turned
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kThreads;
      dst[u] = nullptr;
      turned[u] = -1;
      if (i >= all) continue;
      const int tok = TOK == 1 ? 0 : i / per_token, r = i - tok * per_token, head = r / PIECES, c = (r % PIECES) * 8;
      if (dest[tok] < 0) continue;
      const long long t = t0 + tok;
      const T* src;
      if (head < hq) {
        src = static_cast<const T*>(a.q) + t * a.q_row_stride + head * a.q_head_stride;
        dst[u] = static_cast<T*>(a.q_out) + t * a.qo_row_stride + head * a.qo_head_stride;
      } else if (head < hq + hkv) {
        const int h = head - hq;
        src = static_cast<const T*>(a.k) + t * a.k_row_stride + h * a.k_head_stride;
        dst[u] = static_cast<T*>(a.pages.k) + dest[tok] + h * a.pages.head_stride;
      } else {
        const int h = head - hq - hkv;
        src = static_cast<const T*>(a.v) + t * a.v_row_stride + h * a.v_head_stride;
        dst[u] = static_cast<T*>(a.pages.v) + dest[tok] + h * a.pages.head_stride;
      }
      if (head < hq + hkv && a.rope_theta != 0.0) turned[u] = tok * H + c;
      lo[u] = *reinterpret_cast<const uint4*>(src + c);
      hi[u] = *reinterpret_cast<const uint4*>(src + c + H);
      dst[u] += c;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!dst[u]) continue;
      if (turned[u] >= 0) {
        const float4* cs = reinterpret_cast<const float4*>(&turn[0][0] + turned[u]);
        uint32_t* l = &lo[u].x;
        uint32_t* h = &hi[u].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = Elem<T>::unpack(l[j]), y = Elem<T>::unpack(h[j]);
          const float4 w = cs[j];  // (cos, sin) of two pairs
          l[j] = Elem<T>::pack(x.x * w.x - y.x * w.y, x.y * w.z - y.y * w.w);
          h[j] = Elem<T>::pack(y.x * w.x + x.x * w.y, y.y * w.z + x.y * w.w);
        }
      }
      *reinterpret_cast<uint4*>(dst[u]) = lo[u];
      *reinterpret_cast<uint4*>(dst[u] + H) = hi[u];
    }
  }
}

template <class T, int D>
mk_status launch(const AppendParams& P, cudaStream_t s, std::string& err) {
  // A block's tokens share its prologue (sequence search, angles); few tokens go one to a block, so that more SMs take part.
  const int n = P.a.n_tokens;
  const cudaError_t e = n <= kFewTokens
      ? mk::launch(true, append_kernel<T, D, 1>, dim3(n), kThreads, 0, s, 0, P)
      : mk::launch(false, append_kernel<T, D, kMaxTokens>, dim3((n + kMaxTokens - 1) / kMaxTokens), kThreads, 0, s, 0, P);
  return cuda_result(e, "mk_append_kv launch", err);
}

}  // namespace

mk_status launch_append(const mk_append_args& a, void* stream, std::string& err) {
  AppendParams P;
  P.a = a;
  const int D = a.pages.head_dim;
  // theta^(-2p/D) = r^p, by squares of earlier ones (at most 12 roundings in double): 64 calls of pow would take
  // longer than the kernel does for a few tokens
  const double r = a.rope_theta != 0.0 ? std::pow(a.rope_theta, -2.0 / D) : 0.0;
  P.freq[0] = 1.0;
  for (int p = 1; p < 64; ++p) P.freq[p] = P.freq[p / 2] * P.freq[p / 2] * (p & 1 ? r : 1.0);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.pages.dtype == MK_DTYPE_BF16)
    return D == 64 ? launch<__nv_bfloat16, 64>(P, s, err) : launch<__nv_bfloat16, 128>(P, s, err);
  return D == 64 ? launch<__half, 64>(P, s, err) : launch<__half, 128>(P, s, err);
}

}  // namespace mk
