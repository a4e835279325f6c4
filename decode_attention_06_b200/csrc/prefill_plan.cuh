// prefill_plan.cuh -- the work plan of the chunk attention (prefill.cu), shared by its
// kernels and by the host-side planner.
//
// Sequence b brings n_b new tokens, the last n_b of its L_b cached ones. A query block
// is 4 (128 / G) tokens of one sequence (times the G heads of one group: two 256-row MMA
// tiles over a CTA pair); its keys are the tokens [0, kv_end), kv_end = the position after its last
// token, in tiles of 128. The batch's (block, key tile) pairs, ordered by sequence, group,
// block and tile, are cut into `num_splits` chunks of ceil(T / num_splits) pairs, one per
// CTA pair: every pair gets the same number of tiles although causal blocks differ in length,
// and a few rows against a long context spread over many pairs by the same rule. A block
// that falls in one chunk is finished by its pair; of one that a chunk boundary cuts, each
// piece writes a partial (slot 2c: the block began in an earlier chunk; slot 2c + 1: it
// begins in chunk c and goes on), merged by the combine.
#pragma once

#include <stdint.h>

namespace gqla {

constexpr int kPfTile = 128;        // keys per tile (two pages)
constexpr int kPfRows = 128;        // query rows of one CTA in an MMA tile
constexpr int kPfBlockRows = 512;   // query rows of a block: two MMA tiles over two CTAs

// Query tokens of a CTA's part of an MMA tile / of a block, for G heads per group.
__host__ __device__ inline int pf_tile_tokens(int G) { return kPfRows / G; }
__host__ __device__ inline int pf_block_tokens(int G) { return 4 * (kPfRows / G); }

// sum over i in [0, n) of floor((a i + b) / m), a, b >= 0: the lattice points under a line,
// by Euclid's steps on (a, m).
__host__ __device__ inline int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    int64_t sum = 0;
    while (true) {
        if (a >= m) {
            sum += (a / m) * (n * (n - 1) / 2);
            a %= m;
        }
        if (b >= m) {
            sum += (b / m) * n;
            b %= m;
        }
        const int64_t top = a * n + b;
        if (top < m) return sum;
        n = top / m;
        b = top % m;
        const int64_t t = m;
        m = a;
        a = t;
    }
}

// Key tiles of the first i query blocks (W tokens each, the last one short) of a sequence
// of L tokens whose last n are the queries: sum of ceil(kv_end / 128).
__host__ __device__ inline int64_t pf_tiles_before(int n, int L, int W, int i) {
    const int full = n / W;
    const int f = i < full ? i : full;
    int64_t s = f > 0 ? floor_sum(f, kPfTile, W, (int64_t)(L - n) + W + kPfTile - 1) : 0;
    if (i > full) s += ((int64_t)L + kPfTile - 1) / kPfTile;
    return s;
}

__host__ __device__ inline int pf_blocks(int n, int W) { return (n + W - 1) / W; }

}  // namespace gqla
