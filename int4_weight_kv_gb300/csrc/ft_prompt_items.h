// Which block of prompt attention an item of work is, where every sequence is a lane's (up to 32 of them): the blocks of the
// last place that any sequence has come first, then those of the place before it, and so on; within a place in the order of
// the sequences.  (No CUDA in here: the walk is also compiled for the host.)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FT_ITEM_CALL __device__ __forceinline__
#else
#define FT_ITEM_CALL inline
#endif

namespace ft {

// `have(level)`: a bit for each sequence with a block at place `level`; `count` its bits.  The walk goes on from the item
// before, since items mostly come in ascending order.  Nothing promises that they do (cluster launch control hands out CTAs
// that have not begun in any order): an item before the place where the walk stands starts it again.
struct ItemWalk {
  int top, level, above;  // the last place of all; where the walk stands, and the blocks at places above it
  FT_ITEM_CALL explicit ItemWalk(int top_) : top(top_), level(top_), above(0) {}
  // The sequences at item i's place (afterwards `level`); it is the (i - above)-th of them, from 0.
  template <class Have, class Count>
  FT_ITEM_CALL uint32_t find(int i, Have have, Count count) {
    if (i < above) level = top, above = 0;
    uint32_t some = have(level);
    while (i - above >= count(some)) {
      above += count(some);
      some = have(--level);
    }
    return some;
  }
};

}  // namespace ft

#undef FT_ITEM_CALL
