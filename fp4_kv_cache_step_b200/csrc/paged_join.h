// paged_join.h -- which partials the join of paged attention reads for a pair of a
// sequence and a row block. Plain C++, so that the rule is tested on the host.
#pragma once

#ifdef __CUDACC__
#define CSA2_JOIN_FN __host__ __device__ __forceinline__
#else
#define CSA2_JOIN_FN inline
#endif

namespace csa2 {

// Each of `pieces` pieces has two slots for partials, 2 i and 2 i + 1: a pair that is cut
// leaves one in the slot `slot` of its first piece, and in 2 i of every further one.
CSA2_JOIN_FN int join_slot(int i, int first, int slot) { return i == first ? slot : 2 * i; }

// Whether {first, last, slot} is a pair's record. The piece that holds the pair's first
// tile writes it; one that gave up after a wait ran out did not, and then these are
// whatever the workspace held. With a record that holds, every join_slot(i, first, slot)
// of first <= i <= last lies in [0, 2 pieces).
CSA2_JOIN_FN bool join_record_holds(int first, int last, int slot, int pieces) {
  return first >= 0 && first <= last && last < pieces && (slot >> 1) == first;
}

}  // namespace csa2
