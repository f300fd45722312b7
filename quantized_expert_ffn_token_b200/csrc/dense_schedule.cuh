// Arithmetic of the tiled dense products' schedule that both sides of a launch use; plain integers, so that it also runs
// on the host.
#pragma once

namespace qeffn {
namespace dense {

constexpr long long kSpinCycles = 4000000000LL;   // clock64 cycles, about two seconds: the limit of a wait on one copy or MMA

// Limit of the wait for a tile's whole product, of `k_steps` steps of 64 (8-bit: 128) reduction values.  A step takes 260
// to 700 cycles while its operands keep up and about 1,500 where every one comes from HBM; the weight gradients over
// 2^30 rows have 2^24 of them in a tile (8 x 8 matrices: 4.2 s a call, about 450 cycles a step).
__host__ __device__ constexpr long long tile_wait_cycles(long long k_steps) { return kSpinCycles + 4096 * k_steps; }

}  // namespace dense
}  // namespace qeffn
