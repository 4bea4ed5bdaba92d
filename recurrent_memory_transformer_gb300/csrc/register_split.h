// Registers of a block whose warps trade them (setmaxnreg).
#pragma once

namespace armt {

// Registers a thread that a kernel using `used` of them is launched with: they are
// handed out in eights.  A split that adds up to a launch with 128 also does with
// a kernel that the compiler brought to 121.
constexpr int launch_registers(int used) { return (used + 7) / 8 * 8; }

// Whether `takers` threads of `block` can go to `take` registers each, and the
// others to `keep`, when the kernel uses `used`.  If not, the takers would wait for
// registers that nobody gives back.
constexpr bool split_fits(int used, int block, int takers, int take, int keep) {
  return used > 0 && takers * take + (block - takers) * keep <= block * launch_registers(used);
}

}  // namespace armt
