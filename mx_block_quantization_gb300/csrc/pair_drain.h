// pair_drain.h -- shutting down a pipeline of stages that a pair of CTAs loads together.
//
// Stage n goes to slot n % stages.  Each CTA loads its half of a stage into its own shared
// memory, and the leader's barrier of the slot counts both halves: one arrival, by the
// leader as it issues its half, that announces the bytes of both.  When a wait has run out
// the two may have stopped at different stages.  For each stage that may still be under
// way, in order, the leader makes up for what was not announced or not loaded, and waits.
// Host code as well, so that the accounting is tested without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MXQ_PAIR_FN __host__ __device__ inline
#else
#define MXQ_PAIR_FN inline
#endif

namespace mxq {

// Stages [first, end) may be under way where the leader has issued `own` stages and its
// peer `peer`: a slot is loaded again only after both halves of its last stage were used.
struct PairDrain {
  int32_t first, end;
};
MXQ_PAIR_FN PairDrain pair_drain(int32_t own, int32_t peer, int32_t stages) {
  const int32_t both = own < peer ? own : peer, most = own < peer ? peer : own;
  return {both < stages ? 0 : both - stages, most};
}

// Stage n was loaded by the peer alone: its half is still to be announced.
MXQ_PAIR_FN bool pair_unannounced(int32_t n, int32_t own) { return n >= own; }
// Stage n was loaded by the leader alone: the peer's half is announced and never comes.
MXQ_PAIR_FN bool pair_half_missing(int32_t n, int32_t peer) { return n >= peer; }

}  // namespace mxq
