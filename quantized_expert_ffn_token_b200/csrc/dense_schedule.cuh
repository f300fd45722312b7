// Arithmetic of the tiled dense products' schedule that both sides of a launch use; plain integers, so that it also runs
// on the host.
#pragma once

namespace qeffn {
namespace dense {

constexpr long long kSpinCycles = 4000000000LL;   // clock64 cycles, about two seconds: the limit of a wait on one copy or MMA

// Limit of the wait for a tile's whole product, of `k_steps` steps of 64 (8-bit: 128) reduction values.  A step takes 260
// to 700 cycles while its operands keep up; with every operand from HBM, 74 pairs of 64 KB a step at 3.4 KB a cycle would
// take 1,400.  The weight gradients over 2^30 rows have 2^24 steps in a tile (8 x 8 matrices: 4.2 s a call, about 450
// cycles a step).
__host__ __device__ constexpr long long tile_wait_cycles(long long k_steps) { return kSpinCycles + 4096 * k_steps; }

// The tiles of cluster c of P, in order.  A group's first `big` tiles (a product with a long reduction) are dealt round
// robin; so the first big % P clusters hold one more of them, and the others take `rounds` more of the remaining tiles,
// which are dealt round robin among those that have time.
template <bool GROUP>
struct Order {
    int c, P, n, mine = 0, rest = 0, big = 0, rounds = 0;
    bool more = false;
    __host__ __device__ Order(int tiles, int big_, int rounds_, int cluster, int clusters) : c(cluster), P(clusters), n(tiles) {
        if constexpr (GROUP) {
            big = big_;
            rounds = rounds_;
            mine = c < big ? (big - c + P - 1) / P : 0;
            const int r = big % P;
            rest = P - r;
            more = c >= r;
        }
    }
    __host__ __device__ int at(int k) const {   // -1: no more
        int t = c + k * P;
        if constexpr (GROUP)
            if (k >= mine) {
                const int j = k - mine;
                t = big + (more && j < rounds ? j * rest + c - (P - rest) : rounds * rest + (j - (more ? rounds : 0)) * P + c);
            }
        return t < n ? t : -1;
    }
};

}  // namespace dense
}  // namespace qeffn
