// kd_boxes.h -- which of a warp's two output boxes the GEMM epilogues stage next.
//
// A box in shared memory may be written again once the TMA transfer issued from
// it has read it, and an epilogue waits for that until at most
// BOX_READS_PENDING transfers are still reading.  So the boxes have to be taken in
// turn over everything the warp emits: a tile with an odd number of boxes (an
// odd number of 32-column blocks, as N = 72 or 200 gives) leaves the next tile to
// begin with the other box.  Plain C++ so that a host program can check it
// (tests/c/box_turn_check.cc).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KD_BOX_FN __host__ __device__ __forceinline__
#else
#define KD_BOX_FN inline
#endif

namespace kd {

constexpr int EPI_BOXES = 2;                            // boxes of a warp
constexpr int BOX_READS_PENDING = EPI_BOXES - 1;        // transfers that may still read

// The box to stage next; `turn` counts the boxes that this warp has taken, over all
// of its tiles.
KD_BOX_FN uint32_t box_take(uint32_t& turn) { return turn++ % EPI_BOXES; }

}  // namespace kd
