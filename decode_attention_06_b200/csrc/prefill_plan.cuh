// prefill_plan.cuh -- the work plan of the chunk attention (prefill.cu), shared by its
// kernels and by the host-side planner.
//
// Sequence b brings n_b new tokens, the last n_b of its L_b cached ones. A query block is
// 4 T tokens of one sequence, T = 128 / G (times the G heads of one group: two 256-row MMA
// tiles over a CTA pair); its keys are the tokens [0, kv_end), kv_end = the position after
// its last token, in tiles of 128.
//
// The batch's blocks, ordered by sequence, group and block, lie on a line of cost units: a
// block takes w = 2 units per key tile (1 if its tokens fit one MMA tile, whose steps take
// about half as long) and kPfBlockCost more. The line is cut into `num_splits` chunks of
// equal length, one per CTA pair; a key tile belongs to the chunk that holds its first unit.
// So every pair gets the same share although causal blocks differ in length, and a few rows
// against a long context spread over many pairs by the same rule. A block that falls in one
// chunk is finished by its pair; of one that a cut divides, each piece writes a partial (slot
// 2c: the block began in an earlier chunk; slot 2c + 1: it begins in chunk c and goes on) and
// the pair that begins it a record of the merge, which the combine carries out. With `whole`
// no block is divided: it belongs to the chunk that holds its first unit.
#pragma once

#include <stdint.h>

namespace gqla {

constexpr int kPfTile = 128;        // keys per tile (two pages)
constexpr int kPfRows = 128;        // query rows of one CTA in an MMA tile
constexpr int kPfBlockRows = 512;   // query rows of a block: two MMA tiles over two CTAs
// Units for a block's start and end: a step of two MMA tiles (2 units) takes 3500 cycles, a
// block 8000 more (fitted to the spread of the pairs' times over prompts of 130 to 8192 tokens).
constexpr int kPfBlockCost = 5;

// Query tokens of a CTA's part of an MMA tile, for G heads per group: T.
__host__ __device__ inline int pf_tile_tokens(int G) { return kPfRows / G; }

// Units per key tile of a block of `ntok` tokens.
__host__ __device__ inline int pf_weight(int ntok, int T) { return ntok > 2 * T ? 2 : 1; }

__host__ __device__ inline int pf_blocks(int n, int T) { return (n + 4 * T - 1) / (4 * T); }

// Length of a chunk: at least 2 units, so that every chunk inside a block holds a tile of it.
__host__ __device__ inline int64_t pf_chunk(int64_t total, int num_splits) {
    const int64_t k = (total + num_splits - 1) / num_splits;
    return k < 2 ? 2 : k;
}

// sum over i in [0, n) of floor((a i + b) / 128): the lattice points under a line, by Euclid's
// steps on (a, 128), the first of them with shifts. a n + b < 2^32.
__host__ __device__ inline int64_t tile_sum(uint32_t n, uint32_t a, uint32_t b) {
    static_assert(kPfTile == 128, "shifts");
    int64_t sum = (int64_t)(a >> 7) * ((int64_t)n * (n - 1) / 2) + (int64_t)(b >> 7) * n;
    uint32_t top = (a & 127) * n + (b & 127);
    uint32_t m = a & 127;  // a and m trade places
    a = 128;
    if (top < 128) return sum;
    n = top >> 7;
    b = top & 127;
    while (true) {
        sum += (int64_t)(a / m) * ((int64_t)n * (n - 1) / 2);
        a %= m;
        if (b >= m) {
            sum += (int64_t)(b / m) * n;
            b %= m;
        }
        top = a * n + b;
        if (top < m) return sum;
        n = top / m;
        b = top % m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
}

// Units of the first i query blocks of one group of a sequence of L tokens whose last n are
// the queries. All blocks but the last have 4 T tokens.
__host__ __device__ inline int64_t pf_units_before(int n, int L, int T, int i) {
    const int W = 4 * T, full = n / W;
    const int f = i < full ? i : full;
    int64_t s = (int64_t)kPfBlockCost * i;
    if (f > 0) s += 2 * tile_sum(f, W, (uint32_t)(L - n) + W + kPfTile - 1);
    if (i > full) s += (int64_t)pf_weight(n - full * W, T) * (((int64_t)L + kPfTile - 1) / kPfTile);
    return s;
}

}  // namespace gqla
