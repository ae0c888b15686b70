// prompt_ring.hpp — the order in which a block of mk_prompt_attention passes
// tiles through its ring, and which barrier and phase a ragged value tile
// takes: arithmetic that several roles of the kernel must agree on, kept free
// of CUDA so that a host model of the roles can be run over it.
#pragma once

#ifdef __CUDACC__
#define MK_RING_FN __host__ __device__ __forceinline__
#else
#define MK_RING_FN inline
#endif

namespace mk {

// An item's K and V tiles (n of each) in the ring as the MMAs take them:
// K0 V0 K1 V1 .. where P lies over S, else (APART) K0 K1 V0 K2 V1 ..
template <bool APART>
MK_RING_FN int ring_k(int j) { return APART ? (j > 0 ? 2 * j - 1 : 0) : 2 * j; }
template <bool APART>
MK_RING_FN int ring_v(int j, int n) { return APART ? (2 * j + 2 < 2 * n - 1 ? 2 * j + 2 : 2 * n - 1) : 2 * j + 1; }
// and back: what lies at place i of an item's 2 n
template <bool APART>
MK_RING_FN bool ring_is_v(int i, int n) { return APART ? i == 2 * n - 1 || (i > 0 && !(i & 1)) : i & 1; }
template <bool APART>
MK_RING_FN int ring_tile(int i, int n) {
  if (!APART) return i >> 1;
  return ring_is_v<true>(i, n) ? (i == 2 * n - 1 ? n - 1 : i / 2 - 1) : (i + 1) / 2;
}

// A value tile that its sequence ends inside lands on a barrier of its own,
// where one warp waits to clear the rows behind the end.  The loads of an item
// may begin while the last value tile of the item before is still on its way
// (nothing but its key tiles has to be there by then), but not before the
// clearing warp has done with the item before that: so the block's ragged
// tiles, counted from 0, take two barriers in turn.
constexpr int kTails = 2;
MK_RING_FN int tail_slot(int count) { return count % kTails; }
MK_RING_FN int tail_parity(int count) { return count / kTails & 1; }

}  // namespace mk
