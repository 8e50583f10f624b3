// tree_events.cuh -- which barrier tells the softmax warps of the tree kernel
// that its next event has come.  Plain arithmetic, for the kernel and for the
// host's check of it.
//
// The MMA warp numbers its events through a CTA's life: S of a tile is there, a
// tile comes back, O of a unit is complete.  After the first two it goes on only
// when every softmax warp has answered with P, but after O it does not wait: the
// next unit's S follows at once.  A softmax warp waits for a phase's parity, so
// on one barrier it would miss O where that S is complete before it has looked.
// Events therefore take two barriers in turn.  Of two events in a row one at
// least is answered (S follows O), a warp answers an event when it has seen all
// up to it, and so event e, the first to use e's barrier again after e - 2, does
// not come before every warp has seen e - 2.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define LCA_EVENT_HD __host__ __device__ __forceinline__
#else
#define LCA_EVENT_HD inline
#endif

namespace lca {

constexpr int kTreeEventBars = 2;

LCA_EVENT_HD int tree_event_bar(int event) { return event & 1; }
LCA_EVENT_HD uint32_t tree_event_parity(int event) { return (uint32_t)(event >> 1) & 1u; }

}  // namespace lca
