// When the many-row kernel's cleaning warps wait for the end of an item.
//
// They note non-finite values of item i in shared memory; the softmax warps read
// and clear the notes at the item's end, phase i of the barrier `epilogue`.  The
// cleaning warps may be two items ahead of that end, but a wait for a phase by
// its parity is only sound while the phase is the current one or the one before.
// So phase i - 1 is waited for twice: before the first note of item i, and in any
// case before the item's last tile is handed over.  The second says that item
// i - 1 has ended when they go on to item i + 1, and the item's own end cannot
// come before it; both waits then find phase i - 1 current or just over.  (Host
// code too: tests/test_paged_notes_cpu.py replays it.)
#pragma once

#ifdef __CUDACC__
#define ARMT_NOTES_FN __host__ __device__ constexpr
#else
#define ARMT_NOTES_FN constexpr
#endif

namespace armt {

// The phase of `epilogue` to wait for in item `item` (-1: none).
ARMT_NOTES_FN int notes_phase(int item) { return item - 1; }
// Whether tile `tile` of `count` is handed over only after that phase.
ARMT_NOTES_FN bool notes_hold_back(int item, int tile, int count) { return item > 0 && tile + 1 == count; }

}  // namespace armt
