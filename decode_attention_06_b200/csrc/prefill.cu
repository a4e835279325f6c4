// prefill.cu -- attention of chunks of new tokens over the paged expanded cache (GQA
// path): every new token of a sequence attends to the cached tokens up to and including
// itself, G query heads sharing each group's [K_nope | k^R] and V (GQLA, paperlayer.ai
// summary, sec. 3 "Two equivalent decoding paths": the g K/V groups are materialised and
// attention over them is standard grouped-query attention).
//
// Bound by the tensor cores for chunks (2 (192 + 128) FLOPs per visible (row, key) pair
// against 640 bytes per key shared by 512 rows) and by HBM when a few rows meet a long
// context.
//
//  * A query block is 512 rows: two MMA tiles of 256 rows over a CTA pair (cta_group::2), each
//    CTA's 128 rows being (128 / G) tokens x G heads of one group, so that the heads of a
//    group share every key tile on chip. Per key tile of 128 tokens (two pages) and MMA tile:
//      S[256 x 128]   = q (256 x 192, smem) x K^T (192 x 128, smem: a page in each CTA)
//      O[256 x 128]  += P (256 x 128, bf16 in TMEM) x V (128 x 128, smem: 64 columns in each CTA)
//    The pair halves what a CTA loads and what the tensor core reads of B from shared memory:
//    with one CTA, q and K alone take the 128 bytes a cycle that shared memory gives, and the
//    copies come on top (2690 cycles a step against 2560 of MMA; the pair 1730).
//  * TMEM: P0 | S | P1 | O0 | O1 (64 + 128 + 64 + 128 + 128 columns). The two MMA tiles take turns
//    with S, which is free again once their softmax has it in registers, so no tile waits
//    for its own P -> O -> S chain. What paces a step is this turn-around: read, remote
//    arrive, 12 MMAs and their commit are about 1520 cycles, twice a step: 3050 to 3300 cycles
//    measured per step of two MMA tiles against 2560 of MMA.
//  * 12 warps: warp 0 TMA producer, warps 1 and 2 the issuers of S and of O (in rank 0, for the
//    pair), warp 3 TMEM owner and clears V rows past a block's last key; warps 4-7 and 8-11 the
//    softmax of tile 0 and tile 1, one query row per thread (no exchange between threads), fp32
//    online softmax in the base-2 domain, relative to a base that is set from a row's first
//    tile and raised (O rescaled) only when a later one needs it. In a block of one MMA tile
//    both softmax warpgroups take its rows, for even and odd key tiles.
//  * K and V tiles pass through rings of three stages each.
//  * Work split: prefill_plan.cuh. Every CTA derives its chunk from the device-resident
//    lengths.
//  * Every wait is bounded; a wait that runs out records GQLA_ERR_TIMEOUT and the pair
//    drains and exits.
//
// Measured (128 heads over 8 groups, back to back under the power limit): 2048 tokens after 32768
// cached ones 4.4 ms, 1290 TFLOP/s (78% of the measured burst rate of a library GEMM, 94% of its
// sustained rate); a prompt of 8192 2.15 ms, 1280 TFLOP/s.
#include <cuda.h>
#include <limits.h>

#include "common.cuh"
#include "prefill_plan.cuh"
#include "ragged.cuh"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace gqla {

namespace {

using namespace sm100;

constexpr int kPfThreads = 384;
constexpr int kPfLaunchRegs = 168;
constexpr int kPfIssueRegs = 72, kPfSoftmaxRegs = 216;
static_assert(128 * kPfIssueRegs + 256 * kPfSoftmaxRegs <= kPfThreads * kPfLaunchRegs, "register split");
// A row's base is looked at anew when a tile's sum is above 2^16 (or under a mask), and raised
// if the maximum is more than 2^8 above it. 128 scores that stay below that sum to 2^15 at most,
// so a sum above 2^16 always raises the base. P is at most 2^16 then, l and the unnormalised O at
// most 2^16 a tile (times max |V|): O stays below 2^128 for |V| up to 2^118 / L.
constexpr float kPfRise = 65536.0f, kPfRescaleLog2 = 8.0f;

constexpr int kPfBox = 64 * 128;          // one TMA box: 64 rows of 128 bytes
constexpr int kPfK = 3 * kPfBox;          // a key tile's K in one CTA: its page's 64 keys x 192
constexpr int kPfV = 2 * kPfBox;          // and V: 128 keys x its 64 columns
constexpr int kPfStages = 3;              // tiles in the rings
constexpr int kPfQBlock = kPfRows * 128;  // 64 columns of a query tile

struct PfSmem {
    static constexpr int oQ = 0;                                   // [2 tiles][3 column blocks]
    static constexpr int oK = oQ + 6 * kPfQBlock;                  // [stages]
    static constexpr int oV = oK + kPfStages * kPfK;               // [stages]
    static constexpr int oBar = oV + kPfStages * kPfV;
    // k_full/k_empty, v_full/v_empty[stages], q_full/q_empty[2], s_full[2], s_free, p_full[2],
    // pv_done[2], o_free[2], x_full, v_part[stages], drain[2]
    static constexpr int kNumBars = 5 * kPfStages + 4 + 2 + 1 + 2 + 2 + 2 + 1 + 2;
    static constexpr int kExchange = 2 * kPfRows * 4;              // m, l of the second half's rows
    static constexpr int oPlan = oBar + kNumBars * 8;              // PfPlan
    static constexpr int oList = oPlan + 48;                       // PfListed[kPfListed]
    static constexpr int oX = oList + 128 * 16;
    static constexpr int oMisc = oX + kExchange;                       // tmem base, abort flag
    static constexpr int kBytes = oMisc + 16;
    static constexpr int kAlloc = kBytes + 1024;
};
static_assert(PfSmem::kAlloc <= 227 * 1024, "shared memory");

struct PfParams {
    const int32_t *q_starts;
    const int32_t *page_table;
    const int32_t *seqlens;
    float *o_part;    // [2 num_splits][512][128]
    float *lse_part;  // [2 num_splits][512], then the merge records
    __nv_bfloat16 *out;
    float *lse_out;
    void *ws;
    int64_t total_q;
    int64_t num_slots;
    int batch, max_pages, num_pages, num_splits, heads, groups, G, tile_tokens;
    bool whole;  // no block is divided: no partials, no merge
    int drop_v;  // diagnostic: rank 0 never issues its V load of this step (-1: none)
    float scale_log2;
};

// Bounded wait of a role that may have nothing to do for whole blocks (a query tile that
// short blocks leave empty, the V rows of blocks that end on a tile): the roles that feed it
// give up after kWaitCycles and raise the abort flag; its own limit is 32 times that.
__device__ __forceinline__ bool mbar_wait_long(uint64_t *bar, uint32_t parity, volatile int *abort) {
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (clock64() - t0 > 32 * kWaitCycles) return false;
    }
}

using PfSeq = RaggedSeq;

__device__ __forceinline__ PfSeq pf_seq(const PfParams &p, int b) {
    return ragged_seq(p.q_starts, p.seqlens, b, p.total_q, p.max_pages);
}

__device__ __forceinline__ int64_t pf_seq_units(const PfParams &p, const PfSeq &s) {
    return s.n > 0 ? p.groups * pf_units_before(s.n, s.L, p.tile_tokens, pf_blocks(s.n, p.tile_tokens)) : 0;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ int64_t warp_scan64(int64_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
    }
    return v;
}

// A pair's chunk: units [start of block (g, i) of its first sequence, end) from tile t of that
// block on; `len` is the length of every chunk. Its sequences, those without new tokens left out,
// are listed in shared memory (the first kPfListed of them; the iterator reads on from there).
constexpr int kPfListed = 128;
struct PfPlan {
    int64_t u0, end, len;
    int listed, g, i, t;
};
struct PfListed {
    int b, n, L, q0;
};

// The whole CTA: the plan of chunk c. Sequences with bad numbers are reported when `report`.
__device__ void pf_plan(const PfParams &p, int c, bool report, PfPlan *plan, PfListed *list) {
    constexpr int kWarps = kPfThreads / 32;
    __shared__ int64_t sums[kWarps], first_start;
    __shared__ int counts[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the first sequence of a thread stays in registers: a batch of up to 384 is read once
    PfSeq s0{0, 0, 0, false};
    int64_t units0 = 0, total = 0;
    for (int b = threadIdx.x; b < p.batch; b += kPfThreads) {
        const PfSeq s = pf_seq(p, b);
        if (s.bad && report) report_error(p.ws, GQLA_ERR_DEVICE, b);
        const int64_t u = pf_seq_units(p, s);
        total += u;
        if (b < kPfThreads) { s0 = s; units0 = u; }
    }
    total = warp_sum64(total);
    if (lane == 0) sums[warp] = total;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kWarps; ++w) total += sums[w];
    const int64_t len = pf_chunk(total, p.num_splits), pos = c * len, end = min(total, pos + len);
    int64_t base = 0;
    int taken = 0;
    for (int b0 = 0; b0 < p.batch && base < end; b0 += kPfThreads) {
        const int b = b0 + threadIdx.x;
        PfSeq s{0, 0, 0, false};
        int64_t mine = 0;
        if (b0 == 0) { s = s0; mine = units0; }
        else if (b < p.batch) { s = pf_seq(p, b); mine = pf_seq_units(p, s); }
        const int64_t incl = warp_scan64(mine);
        __syncthreads();
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int64_t start = base + incl - mine;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) start += sums[w];
            base += sums[w];
        }
        // the sequences that the chunk meets, in order
        const bool in = mine > 0 && start < end && start + mine > pos;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        if (lane == 0) counts[warp] = __popc(m);
        __syncthreads();
        int at = taken + __popc(m & ((1u << lane) - 1));
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += counts[w];
            taken += counts[w];
        }
        if (in && at == 0) first_start = start;
        if (in && at < kPfListed) list[at] = PfListed{b, s.n, s.L, (int)s.q0};
    }
    __syncthreads();
    if (warp != 0) return;
    PfPlan r{0, 0, len, min(taken, kPfListed), 0, 0, 0};
    if (taken > 0) {
        r.end = end;
        const int n = list[0].n, L = list[0].L, T = p.tile_tokens, blocks = pf_blocks(n, T);
        const int64_t per_group = pf_units_before(n, L, T, blocks);
        int64_t off = pos - first_start;
        r.g = (int)(off / per_group);
        off -= r.g * per_group;
        // the block that holds unit `off`: the last i with units_before(i) <= off
        int lo = 0, hi = blocks;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int at = lo + (lane + 1) * step;
            const bool le = at < hi && pf_units_before(n, L, T, at) <= off;
            const int k = __popc(__ballot_sync(0xffffffffu, le));
            hi = min(hi, lo + (k + 1) * step);
            lo += k * step;
        }
        r.i = lo;
        off -= pf_units_before(n, L, T, lo);
        r.u0 = pos - off;
        const int w = pf_weight(min(n - lo * 4 * T, 4 * T), T);
        // the first tile of the chunk (past the block's last one: the next block's)
        r.t = p.whole ? (off > 0 ? INT_MAX : 0) : (int)((off + w - 1) >> (w - 1));
    }
    if (lane == 0) *plan = r;
}

// One piece: key tiles [t0, t1) of a query block.
struct PfPiece {
    int b, g;
    int64_t row0;   // query row (token) of the block's first token
    int ntok;       // its tokens
    int pos0;       // the first token's position in the sequence
    int t0, t1;     // key tiles of this chunk
    int nt;         // key tiles of the block
    int kv_end;     // keys of the block
};

// Walks the pieces of a chunk; the same in every role.
struct PfIter {
    const PfListed *list;
    int64_t u0, end;  // first unit of the next block, end of the chunk
    int64_t q0;       // the sequence's first query row
    int listed, at;   // sequences in the list, the place of this one (counted on past the list)
    int b, n, L;      // the sequence
    int g, i, t;
    bool started;
    __device__ __forceinline__ PfIter(const PfPlan &plan, const PfListed *seqs)
        : list(seqs), u0(plan.u0), end(plan.end), listed(plan.listed), at(0), g(plan.g), i(plan.i), t(plan.t),
          started(false) {
        if (listed > 0) take(list[0]);
    }
    __device__ __forceinline__ void take(const PfListed &s) {
        b = s.b;
        n = s.n;
        L = s.L;
        q0 = s.q0;
    }
    // False past the batch.
    __device__ __forceinline__ bool next_sequence(const PfParams &p) {
        if (++at < listed) {
            take(list[at]);
            return true;
        }
        while (++b < p.batch) {
            const PfSeq s = pf_seq(p, b);
            n = s.n;
            L = s.L;
            q0 = s.q0;
            if (n > 0) return true;
        }
        return false;
    }
    __device__ __forceinline__ bool next(const PfParams &p, PfPiece &o) {
        while (u0 < end) {
            if (started && ++i * 4 * p.tile_tokens >= n) {
                i = 0;
                if (++g == p.groups) {
                    g = 0;
                    if (!next_sequence(p)) end = u0;
                    if (u0 >= end) return false;
                }
            }
            started = true;
            const int first = i * 4 * p.tile_tokens;
            o.b = b;
            o.g = g;
            o.row0 = q0 + first;
            o.ntok = min(4 * p.tile_tokens, n - first);
            o.pos0 = L - n + first;
            o.kv_end = o.pos0 + o.ntok;
            o.nt = (int)(((uint32_t)o.kv_end + kPfTile - 1) / kPfTile);  // kv_end may be 2^31 - 1
            const int w = pf_weight(o.ntok, p.tile_tokens);
            o.t0 = t;
            o.t1 = p.whole ? o.nt : (int)min((int64_t)o.nt, (end - u0 + w - 1) >> (w - 1));  // w is 1 or 2
            t = 0;
            u0 += (int64_t)w * o.nt + kPfBlockCost;
            if (o.t0 < o.t1) return true;
        }
        return false;
    }
};

// The merge of the block that begins in chunk c and goes on: pieces in `parts` chunks (0: none
// does), rows of tokens [row0, row0 + ntok), group g. One record per chunk, behind the LSE rows
// of the partials.
struct PfMerge {
    int parts, row0, ntok, g;
};

__device__ __forceinline__ PfMerge *pf_merge(const PfParams &p, int c) {
    return reinterpret_cast<PfMerge *>(p.lse_part + (int64_t)2 * p.num_splits * kPfBlockRows) + c;
}

// TMEM columns: P of the two query tiles (bf16, 64 columns each) with the one S between
// them, then O. The tiles take turns with S: it is free again as soon as the softmax has
// read it, so S of the next step is formed while P of this one still is, and no tile waits
// for its own P -> O -> S chain.
constexpr int kPfColS = 64;
__device__ __forceinline__ uint32_t p_col(int q) { return q ? 192 : 0; }
__device__ __forceinline__ uint32_t o_col(int q) { return 256 + kDv * q; }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// P = 2^(s scale - mu) of a row's 128 scores, rounded to bf16, into the row's P columns;
// returns the sum of the unrounded values. (bf16 because both operands of the product P V have one
// type and V is bf16; it is the one rounding besides the output's, and the decode kernels make it
// too: outputs are 1.4 times as far from float64 as with the output's alone. l and the LSE do not
// see it.) (A share of the exponentials as polynomials on the
// FMA pipes does not pay here: the issue slots and the power that they take cost more than the
// special-function unit's time. Step of 128 keys: 3080 cycles without, 3190 with a quarter,
// 3610 with half.)
template <typename Ready>
__device__ __forceinline__ float form_p(const uint32_t (&sv)[128], float scale, float mu, uint32_t t_p, Ready ready) {
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const float2 sc = make_float2(scale, scale), sub = make_float2(-mu, -mu);
#pragma unroll
    for (int i = 0; i < 128; i += 32) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const float2 x = fma2(make_float2(__uint_as_float(sv[i + e]), __uint_as_float(sv[i + e + 1])), sc, sub);
            const float2 v = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], v);
            __nv_bfloat162 h2 = __floats2bfloat162_rn(v.x, v.y);
            w[e / 2] = *reinterpret_cast<uint32_t *>(&h2);
        }
        if (i == 0) ready();  // P of the step before has been used
        tmem_st16(t_p + i / 2, w);
    }
    const float2 t = add2(sum[0], sum[1]);
    return t.x + t.y;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPfThreads, 1)
    prefill_gqa_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap kr_map,
                       const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap q_token_map,
                       const PfParams p) {
    using SM = PfSmem;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + SM::oBar), *k_empty = k_full + kPfStages;
    uint64_t *v_full = k_empty + kPfStages, *v_empty = v_full + kPfStages;
    uint64_t *q_full = v_empty + kPfStages, *q_empty = q_full + 2;
    uint64_t *s_full = q_empty + 2, *s_free = s_full + 2, *p_full = s_free + 1, *pv_done = p_full + 2;
    uint64_t *o_free = pv_done + 2;
    uint64_t *x_full = o_free + 2, *v_part = x_full + 1, *drain = v_part + kPfStages;
    static_assert(sizeof(PfPlan) <= SM::oList - SM::oPlan && kPfListed * sizeof(PfListed) <= SM::oX - SM::oList, "plan");
    PfPlan &plan = *reinterpret_cast<PfPlan *>(smem + SM::oPlan);
    PfListed *const list = reinterpret_cast<PfListed *>(smem + SM::oList);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SM::oMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SM::oMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x >> 1;  // this pair's chunk
    const uint32_t rank = cluster_rank();
    // the barriers that the MMA issuer waits for are those of rank 0
    auto lead = [](uint64_t *bar) { return map_peer(smem_u32(bar), 0); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kPfStages; ++i) {
            mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1); mbar_init(&v_empty[i], 1);
            mbar_init(&v_part[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 8);
            mbar_init(&pv_done[i], 1); mbar_init(&o_free[i], 8);
        }
        mbar_init(s_free, 8);
        mbar_init(x_full, 4);
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&kv_map);
        prefetch_tensormap(&kr_map);
        prefetch_tensormap(&q_map);
    }
    __syncwarp();
    cluster_arrive();  // this thread's barriers are initialised
    if (warp == 3) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
        tc_fence_before();
    }
    griddep_wait();
    griddep_launch_dependents();
    pf_plan(p, c, blockIdx.x == 0, &plan, list);
    __syncthreads();
    cluster_wait();  // the other CTA's barriers are initialised too
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPfIssueRegs));
        if (warp == 0) {
            // ------------------------------------------------------------ TMA producer
            if (elect_one()) {
                uint32_t kn = 0, vn = 0, qn[2] = {0, 0};
                // the next stage of a ring, once it is free
                auto stage = [&](uint64_t *fullb, uint64_t *emptyb, uint32_t n, uint32_t bytes) -> int {
                    const int st = n % kPfStages;
                    if (!mbar_wait(&emptyb[st], ((n / kPfStages) & 1) ^ 1, abort_flag)) *abort_flag = 1;
                    if (*abort_flag) return -1;
                    if (rank == 0) mbar_arrive_expect_tx(&fullb[st], 2 * bytes);  // both CTAs' parts
                    return st;
                };
                // first cache slots of the two pages of a tile; a missing page reads as zeros (a
                // row past the end of the map)
                struct Slots { int s0, s1; };
                auto slots = [&](const PfPiece &pc, int t) -> Slots {
                    const int32_t *row = p.page_table + (int64_t)pc.b * p.max_pages;
                    const int pg = 2 * t, pages = pages_of(pc.kv_end);
                    const int a0 = row[pg], a1 = pg + 1 < pages ? row[pg + 1] : 0;
                    const bool ok0 = a0 >= 0 && a0 < p.num_pages, ok1 = a1 >= 0 && a1 < p.num_pages;
                    if (!ok0 || !ok1) report_error(p.ws, GQLA_ERR_DEVICE, pc.b);
                    return Slots{ok0 ? a0 * kPage : (int)p.num_slots,
                                 ok1 && pg + 1 < pages ? a1 * kPage : (int)p.num_slots};
                };
                // V: both pages, this CTA's 64 columns
                // (`last`: with rows past the block's keys, through warp 3)
                auto load_v = [&](int g, const Slots &sl, bool last) {
                    if (rank == 0 && (int)vn == p.drop_v) {
                        ++vn;
                        return;
                    }
                    const int st = stage(v_full, v_empty, vn, kPfV);
                    if (st < 0) return;
                    uint8_t *dst = smem + SM::oV + st * kPfV;
                    if (last) mbar_arrive_expect_tx(&v_part[st], kPfV);
                    const uint32_t bar = last ? map_peer(smem_u32(&v_part[st]), rank) : lead(&v_full[st]);
                    tma_load_3d_pair(dst, &kv_map, bar, kNope + 64 * (int)rank, sl.s0, g);
                    tma_load_3d_pair(dst + kPfBox, &kv_map, bar, kNope + 64 * (int)rank, sl.s1, g);
                    ++vn;
                };
                auto load_k = [&](int g, const Slots &sl) {
                    const int st = stage(k_full, k_empty, kn, kPfK);
                    if (st < 0) return;
                    uint8_t *dst = smem + SM::oK + st * kPfK;  // K_nope, RoPE keys of this CTA's page
                    const uint32_t bar = lead(&k_full[st]);
                    const int y = rank ? sl.s1 : sl.s0;
                    tma_load_3d_pair(dst, &kv_map, bar, 0, y, g);
                    tma_load_3d_pair(dst + kPfBox, &kv_map, bar, 64, y, g);
                    tma_load_2d_pair(dst + 2 * kPfBox, &kr_map, bar, 0, y);
                    ++kn;
                };
                // Order: K of the next step before V of this one (whose stage frees later); at the
                // end of a piece V, then the next piece's first K, and only then its queries, whose
                // place frees last.
                const uint32_t q_bytes = (uint32_t)(p.tile_tokens * p.G) * 128u;
                PfIter it(plan, list);
                PfPiece pc;
                while (!*abort_flag && it.next(p, pc)) {
                    Slots sl = slots(pc, pc.t0);
                    load_k(pc.g, sl);
                    for (int q = 0; q < 2 && 2 * q * p.tile_tokens < pc.ntok; ++q) {
                        if (!mbar_wait(&q_empty[q], (qn[q] & 1) ^ 1, abort_flag)) *abort_flag = 1;
                        if (*abort_flag) break;
                        ++qn[q];
                        if (rank == 0) mbar_arrive_expect_tx(&q_full[q], 2 * 3 * q_bytes);
                        // Tokens of this CTA's part. Where the block has none, zeros (tokens past the
                        // batch): a product of zeros takes much less power than one of whatever
                        // rows come next, and under the power limit that is time (G a multiple of
                        // 8 rows, the swizzle's period; other G load what is there).
                        const int first = (2 * q + (int)rank) * p.tile_tokens;
                        const int here = min(max(pc.ntok - first, 0), p.tile_tokens);
                        const uint32_t bar = lead(&q_full[q]);
                        for (int cb = 0; cb < 3; ++cb) {
                            uint8_t *dst = smem + SM::oQ + (3 * q + cb) * kPfQBlock;
                            if (here == p.tile_tokens || p.G % 8 != 0) {
                                tma_load_3d_pair(dst, &q_map, bar, 64 * cb, pc.g * p.G, (int)(pc.row0 + first));
                            } else if (here == 0) {
                                tma_load_3d_pair(dst, &q_map, bar, 64 * cb, pc.g * p.G, (int)p.total_q);
                            } else {
                                for (int i = 0; i < p.tile_tokens; ++i)
                                    tma_load_3d_pair(dst + i * p.G * 128, &q_token_map, bar, 64 * cb, pc.g * p.G,
                                                     i < here ? (int)(pc.row0 + first + i) : (int)p.total_q);
                            }
                        }
                    }
                    for (int t = pc.t0; t < pc.t1 && !*abort_flag; ++t) {
                        const Slots now = sl;
                        if (t + 1 < pc.t1) {
                            sl = slots(pc, t + 1);
                            load_k(pc.g, sl);
                        }
                        if (!*abort_flag) load_v(pc.g, now, t == pc.nt - 1 && pc.kv_end % kPfTile != 0);
                    }
                }
                // every copy has been used, and the other CTA's commits have arrived here
                auto drained = [&](uint64_t *emptyb, uint32_t n) {
                    for (uint32_t x = (n > kPfStages ? n - kPfStages : 0); x < n && !*abort_flag; ++x)
                        if (!mbar_wait(&emptyb[x % kPfStages], (x / kPfStages) & 1, abort_flag)) *abort_flag = 1;
                };
                drained(k_empty, kn);
                drained(v_empty, vn);
                for (int q = 0; q < 2; ++q)
                    if (qn[q] && !*abort_flag && !mbar_wait(&q_empty[q], (qn[q] - 1) & 1, abort_flag)) *abort_flag = 1;
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ S issuer
            // S_q of every step in turn, each as soon as the softmax has read the one before it
            if (rank == 0 && elect_one()) {
                constexpr uint32_t idesc = idesc_bf16(2 * kPfRows, kPfTile, 0, 0);
                // descriptor words: q and K K-major, 128-byte swizzled rows
                const uint64_t q_d = smem_desc(smem_u32(smem + SM::oQ), 16, 1024, kSw128);
                const uint32_t hi = static_cast<uint32_t>(q_d >> 32), q_lo = static_cast<uint32_t>(q_d);
                const uint32_t k_lo = static_cast<uint32_t>(smem_desc(smem_u32(smem + SM::oK), 16, 1024, kSw128));
                uint32_t qn[2] = {0, 0}, sn = 0, s = 0;
                PfIter it(plan, list);
                PfPiece pc;
                while (!*abort_flag && it.next(p, pc)) {
                    const int nq = pc.ntok > 2 * p.tile_tokens ? 2 : 1;
                    for (int t = pc.t0; t < pc.t1 && !*abort_flag; ++t, ++s) {
                        const int st = s % kPfStages;
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            if (nq == 1 && q != ((t - pc.t0) & 1)) continue;
                            const int qt = nq == 2 ? q : 0;  // query tile
                            bool ok = true;
                            if (t == pc.t0) ok = mbar_wait(&q_full[qt], qn[qt]++ & 1, abort_flag);
                            if (qt == 0) ok = ok && mbar_wait(&k_full[st], (s / kPfStages) & 1, abort_flag);
                            if (sn++ > 0) ok = ok && mbar_wait(s_free, sn & 1, abort_flag);
                            if (!ok) *abort_flag = 1;
                            tc_fence_after();
                            const uint32_t a = q_lo + qt * (3 * kPfQBlock >> 4), b = k_lo + st * (kPfK >> 4);
#pragma unroll
                            for (int ks = 0; ks < 12; ++ks)
                                mma_bf16_pair(tmem + kPfColS, a + ((ks >> 2) * kPfQBlock + (ks & 3) * 32 >> 4),
                                              b + ((ks >> 2) * kPfBox + (ks & 3) * 32 >> 4), hi, idesc, ks > 0 ? 1u : 0u);
                            mma_commit_pair(&s_full[q]);
                            if (qt == nq - 1) mma_commit_pair(&k_empty[st]);  // the step's last query tile
                            if (t == pc.t1 - 1) mma_commit_pair(&q_empty[qt]);
                        }
                    }
                }
                // nothing may still be running when TMEM is freed
                mma_commit_pair(&drain[0], 1);
                int dummy = 0;
                mbar_wait(&drain[0], 0, reinterpret_cast<volatile int *>(&dummy));
            }
        } else if (warp == 2) {
            // ------------------------------------------------------------ O issuer
            // O_q += P_q V of every step in turn
            if (rank == 0 && elect_one()) {
                constexpr uint32_t idesc = idesc_bf16(2 * kPfRows, kDv, 0, 1);
                const uint64_t v_d = smem_desc(smem_u32(smem + SM::oV), 16, 1024, kSw128);  // V MN-major
                const uint32_t hi = static_cast<uint32_t>(v_d >> 32), v_lo = static_cast<uint32_t>(v_d);
                uint32_t pn[2] = {0, 0}, on[2] = {0, 0}, s = 0;
                PfIter it(plan, list);
                PfPiece pc;
                while (!*abort_flag && it.next(p, pc)) {
                    const int nq = pc.ntok > 2 * p.tile_tokens ? 2 : 1;
                    for (int t = pc.t0; t < pc.t1 && !*abort_flag; ++t, ++s) {
                        const int st = s % kPfStages;
                        const uint32_t b = v_lo + st * (kPfV >> 4);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            if (nq == 1 && q != ((t - pc.t0) & 1)) continue;
                            const bool fresh = t - pc.t0 == (nq == 1 ? q : 0);  // O_q starts here
                            bool ok = true;
                            if (nq == 1 || q == 0) {
                                const uint32_t parity = (s / kPfStages) & 1;
                                // cleared by warp 3 of either CTA, or as the copies left it
                                ok = t == pc.nt - 1 && pc.kv_end % kPfTile != 0
                                         ? mbar_wait_cluster(&v_full[st], parity, abort_flag)
                                         : mbar_wait(&v_full[st], parity, abort_flag);
                            }
                            if (fresh) ok = ok && mbar_wait(&o_free[q], (on[q]++ & 1) ^ 1, abort_flag);
                            ok = ok && mbar_wait(&p_full[q], pn[q]++ & 1, abort_flag);
                            if (!ok) *abort_flag = 1;
                            tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks)
                                mma_bf16_ts_pair(tmem + o_col(q), tmem + p_col(q) + 8 * ks, b + (ks * 2048 >> 4), hi, idesc,
                                                 (ks > 0 || !fresh) ? 1u : 0u);
                            mma_commit_pair(&pv_done[q]);
                            if (nq == 1 || q == 1) mma_commit_pair(&v_empty[st]);
                        }
                    }
                }
                mma_commit_pair(&drain[1], 1);
                int dummy = 0;
                mbar_wait(&drain[1], 0, reinterpret_cast<volatile int *>(&dummy));
            }
        } else if (warp == 3) {
            // ------------------------------------------------------------ V rows past the keys
            // The last tile of a block ends at its last query token, rarely at the tile's end:
            // the rows past it (later tokens, or slots that hold no token and may hold NaN) meet
            // P = 0 in the product and are cleared so that 0 x NaN cannot enter it. V of such a
            // tile arrives on a barrier of this CTA, and this warp passes its bytes on to the
            // barrier that the O issuer waits for. That issuer reads shared memory of both CTAs, so
            // what orders the cleared rows before its product has cluster scope on both sides
            // (a fence here, the wait there); once per block, it costs nothing that shows.
            PfIter it(plan, list);
            PfPiece pc;
            PfMerge merge{0, 0, 0, 0};
            uint32_t s = 0, fixes = 0;
            while (it.next(p, pc)) {
                s += pc.t1 - pc.t0;
                if (pc.t0 == 0 && pc.t1 < pc.nt) {  // begins here, goes on: where does its last tile lie
                    const int64_t tail = kPfBlockCost + pf_weight(pc.ntok, p.tile_tokens);
                    merge = PfMerge{(int)((it.u0 - tail) / plan.len) - c + 1, (int)pc.row0, pc.ntok, pc.g};
                }
                const int keep = pc.kv_end % kPfTile;
                if (pc.t1 != pc.nt || keep == 0) continue;
                const int st = (s - 1) % kPfStages;
                if (!__all_sync(0xffffffffu, mbar_wait_long(&v_part[st], fixes >> st & 1, abort_flag))) break;
                fixes ^= 1u << st;
                for (int h = 0; h < 2; ++h) {
                    uint8_t *v = smem + SM::oV + st * kPfV + h * kPfBox;
                    const int r0 = min(max(keep - kPage * h, 0), kPage);  // first row to clear in this page
                    for (int i = lane; i < (kPage - r0) * 8; i += 32)
                        *reinterpret_cast<uint4 *>(v + r0 * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    fence_acq_rel_cluster();
                    mbar_complete_tx_remote(lead(&v_full[st]), kPfV);
                }
            }
            if (!p.whole && rank == 0 && lane == 0) *pf_merge(p, c) = merge;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPfSoftmaxRegs));
        // ---------------------------------------------------------------- softmax, epilogue
        const int q = (warp - 4) >> 2;             // query tile
        const int row = 32 * (warp & 3) + lane;    // this thread's query row: its TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t t_s = tmem + kPfColS + lane_off, t_p = tmem + p_col(q) + lane_off, t_o = tmem + o_col(q) + lane_off;
        const int row_tok = row / p.G, hg = row - row_tok * p.G;  // token of the part, head of the group
        float *const xm = reinterpret_cast<float *>(smem + SM::oX), *const xl = xm + kPfRows;
        uint32_t xn = 0;
        const bool in_tile = row < p.tile_tokens * p.G;
        uint32_t sn = 0, pvn = 0;  // steps seen, and products of this tile known to be complete
        PfIter it(plan, list);
        PfPiece pc;
        // A wait that runs out is not branched on (the turn-around of S would pay for the vote):
        // it raises the abort flag, later waits return at once, and nothing is stored any more.
        bool alive = true;
        const uint32_t s_free_a = lead(s_free), p_full_a = lead(&p_full[q]);
        // the first n products of this tile are complete: P may be written, O changed or read
        auto products = [&](uint32_t n) {
            if (pvn < n) {
                alive &= mbar_wait(&pv_done[q], pvn & 1, abort_flag);
                tc_fence_after();
                ++pvn;
            }
        };
        while (it.next(p, pc)) {
            // a block of one MMA tile: both warpgroups take its rows, the even and the odd key
            // tiles, and the first joins the two at the end
            const bool one = pc.ntok <= 2 * p.tile_tokens, joined = one && pc.t1 - pc.t0 > 1;
            if (one && q == 1 && !joined) continue;
            const int part = (one ? 0 : 2 * q) + (int)rank;        // 128-row part of the block
            const int tok = part * p.tile_tokens + row_tok;        // token of the block
            const bool valid = in_tile && tok < pc.ntok;
            const bool warp_valid = __any_sync(0xffffffffu, valid);
            const int last = pc.pos0 + tok;   // the last key this row sees
            float m = valid ? -INFINITY : INFINITY, l = 0.0f;  // base (log2 units) and sum of this row
            const int t_first = pc.t0 + (one ? q : 0);
            for (int t = t_first; t < pc.t1; t += one ? 2 : 1) {
                alive &= mbar_wait_long(&s_full[q], sn++ & 1, abort_flag);
                if (!alive) *abort_flag = 1;
                tc_fence_after();
                if (warp_valid) {
                    uint32_t sv[128];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld32(t_s + 32 * i, sv + 32 * i);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_relaxed(s_free_a);
                    // keys of this tile that the row sees (rows of no token are computed along, with
                    // P = 0, and never stored)
                    const int lim = valid ? last + 1 - t * kPfTile : kPfTile;
                    const bool masked = __any_sync(0xffffffffu, lim < kPfTile);
                    // P against the base so far, at once. The base of a row (its largest score when
                    // it was set, in log2 units) need not be its maximum: bf16 and fp32 have the
                    // exponents for P up to 2^16 (kPfRise), and P, O and l are all relative to it. It
                    // is set on a piece's first tile and under a mask, and again where a sum says
                    // that the scores rose too far above it (or that there was none yet, or that
                    // a score is NaN).
                    float lt;
                    for (bool fresh = t == t_first || masked;; fresh = true) {
                        if (fresh) {
                            if (masked) {
#pragma unroll
                                for (int i = 0; i < 128; i += 32) {
                                    if (!__any_sync(0xffffffffu, lim < i + 32)) continue;  // seen by all rows
#pragma unroll
                                    for (int e = i; e < i + 32; ++e)
                                        if (e >= lim) sv[e] = 0xff800000u;
                                }
                            }
                            float mt = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 128; e += 2)
                                mt = fmaxf(mt, fmaxf(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])));
                            mt *= p.scale_log2;
                            const bool rise = mt > m + kPfRescaleLog2;
                            const float a = rise ? fast_exp2(m - mt) : 1.0f;  // 0 from an empty row
                            if (rise) m = mt;
                            l *= a;
                            products(sn - 1);
                            if (t > t_first && __any_sync(0xffffffffu, rise)) {
#pragma unroll 1
                                for (int i = 0; i < kDv; i += 16) {
                                    uint32_t r[16];
                                    tmem_ld16(t_o + i, r);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * a);
                                    tmem_st16(t_o + i, r);
                                }
                            }
                            tmem_wait_st();
                        }
                        lt = form_p(sv, p.scale_log2, m == -INFINITY ? 0.0f : m, t_p, [&] { products(sn - 1); });
                        if (fresh || !__any_sync(0xffffffffu, valid && (m == -INFINITY || !(lt <= kPfRise)))) break;
                    }
                    l += lt;
                    tmem_wait_st();
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_relaxed(s_free_a);
                    products(sn - 1);
                    if (t == t_first) {  // a warp without a token: P = 0, for the power that products of it save
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = 0;
#pragma unroll
                        for (int i = 0; i < 64; i += 16) tmem_st16(t_p + i, w);
                        tmem_wait_st();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_relaxed(p_full_a);
            }
            // ---- epilogue: O / l and the LSE, to the output or to this piece's partial
            products(sn - 1);
            products(sn);
            if (joined && q == 1) {  // this half's O stays in TMEM, where the same lanes read it
                xm[row] = m;
                xl[row] = l;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(x_full);
                continue;
            }
            float a0 = 1.0f, a1 = 0.0f;
            if (joined) {
                alive &= mbar_wait(x_full, xn++ & 1, abort_flag);
                tc_fence_after();
                const float m1 = xm[row], top = fmaxf(m, m1);
                a0 = m == -INFINITY ? 0.0f : fast_exp2(m - top);
                a1 = m1 == -INFINITY ? 0.0f : fast_exp2(m1 - top);
                l = l * a0 + xl[row] * a1;
                m = top;
            }
            // l = 0: no key seen. A NaN among the scores makes l, and so the row and its LSE, NaN
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            const float lse = l != 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
            const float w0 = a0 * inv, w1 = a1 * inv;
            const bool whole = pc.t0 == 0 && pc.t1 == pc.nt;
            const int64_t prow = (int64_t)(2 * c + (pc.t0 == 0 ? 1 : 0)) * kPfBlockRows + part * kPfRows + row;
            const int64_t orow = (pc.row0 + tok) * p.heads + pc.g * p.G + hg;
            if (warp_valid) {
                if (valid && alive) {
                    if (!whole) p.lse_part[prow] = lse;
                    else if (p.lse_out) p.lse_out[orow] = lse;
                }
                // A lane's row goes out in 64-byte pieces: four lanes trade 16-byte units, so that
                // they write one piece of one row together (alone, a lane's row would touch a line
                // of its own with every store of the warp).
                char *const mine = whole ? reinterpret_cast<char *>(p.out + orow * kDv)
                                         : reinterpret_cast<char *>(p.o_part + prow * kDv);
                char *dst[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t a = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(valid && alive ? mine : nullptr),
                                                   (lane & ~3) + k);
                    dst[k] = a ? reinterpret_cast<char *>(a) + (lane & 3) * 16 : nullptr;
                }
                auto store = [&](uint32_t (&w)[16], int at) {
                    quad_transpose(w, lane);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (dst[k])
                            *reinterpret_cast<uint4 *>(dst[k] + at) =
                                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                };
#pragma unroll 2
                for (int i = 0; i < kDv; i += 32) {
                    uint32_t r[32];
                    tmem_ld32(t_o + i, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * w0);
                    if (joined) {
                        uint32_t r1[32];
                        tmem_ld32(t_o + kDv + i, r1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            r[e] = __float_as_uint(fmaf(__uint_as_float(r1[e]), w1, __uint_as_float(r[e])));
                    }
                    uint32_t w[16];
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
                            w[e] = *reinterpret_cast<uint32_t *>(&h2);
                        }
                        store(w, i * 2);
                    } else {
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = r[h + e];
                            store(w, (i + h) * 4);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_remote_relaxed(lead(&o_free[q]));
                if (joined) mbar_arrive_remote_relaxed(lead(&o_free[1]));
            }
        }
        if (!alive) *abort_flag = 1;
    }

    // Leave together: a CTA that gave up tells the other one; after the barrier none sends
    // anything new, and if either gave up both wait until what is in flight (loads, commits:
    // microseconds) has landed, and for each other once more.
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) {
        report_error(p.ws, GQLA_ERR_TIMEOUT, c);
        st_cluster_b32(map_peer(smem_u32(const_cast<int *>(abort_flag)), rank ^ 1), 1);
    }
    cluster_sync();
    if (*abort_flag) {  // the same in both CTAs
        const long long t0 = clock64();
        while (clock64() - t0 < 200000) {}
        cluster_sync();
    }
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Merge of the divided blocks: CTA (c, y) the rows 32 y .. 32 y + 31 of the block that begins
// in chunk c, if it goes on: slots 2 c + 1, 2 (c + 1), 2 (c + 2), ... Latency-bound: a warp takes
// four rows, four columns a lane, and asks for the first two partials of all of them (nearly
// always there are no more) in one round trip. Partials are added in chunk order.
// ---------------------------------------------------------------------------
constexpr int kPcRows = 32, kPcWarps = 8, kPcWarpRows = kPcRows / kPcWarps;

__global__ void __launch_bounds__(32 * kPcWarps) prefill_combine_kernel(const PfParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x, r0 = blockIdx.y * kPcRows + warp * kPcWarpRows;
    griddep_wait();
    griddep_launch_dependents();
    const PfMerge mg = *pf_merge(p, c);
    if (mg.parts == 0) return;
    bool ok[kPcWarpRows];
    float l0[kPcWarpRows], l1[kPcWarpRows];
    float4 v0[kPcWarpRows], v1[kPcWarpRows];
    auto slot = [&](int x) { return (int64_t)(2 * (c + x) + (x == 0 ? 1 : 0)) * kPfBlockRows; };
    auto load = [&](int64_t row) { return *reinterpret_cast<const float4 *>(p.o_part + row * kDv + 4 * lane); };
#pragma unroll
    for (int i = 0; i < kPcWarpRows; ++i) {
        const int in_tile = (r0 + i) % kPfRows;
        ok[i] = in_tile < p.tile_tokens * p.G && (r0 + i) / kPfRows * p.tile_tokens + in_tile / p.G < mg.ntok;
        if (!ok[i]) continue;
        l0[i] = p.lse_part[slot(0) + r0 + i];
        l1[i] = p.lse_part[slot(1) + r0 + i];
        v0[i] = load(slot(0) + r0 + i);
        v1[i] = load(slot(1) + r0 + i);
    }
#pragma unroll
    for (int i = 0; i < kPcWarpRows; ++i) {
        if (!ok[i]) continue;
        float M = fmaxf(l0[i], l1[i]);
        float w0 = l0[i] == -INFINITY ? 0.0f : expf(l0[i] - M), w1 = l1[i] == -INFINITY ? 0.0f : expf(l1[i] - M);
        float den = w0 + w1;
        float4 acc = make_float4(w0 * v0[i].x + w1 * v1[i].x, w0 * v0[i].y + w1 * v1[i].y, w0 * v0[i].z + w1 * v1[i].z,
                                 w0 * v0[i].w + w1 * v1[i].w);
#pragma unroll 4
        for (int x = 2; x < mg.parts; ++x) {
            const float l = p.lse_part[slot(x) + r0 + i];
            const float4 v = load(slot(x) + r0 + i);
            const float top = fmaxf(M, l);
            const float a = M == -INFINITY ? 0.0f : expf(M - top), w = l == -INFINITY ? 0.0f : expf(l - top);
            M = top;
            den = den * a + w;
            acc = make_float4(acc.x * a + w * v.x, acc.y * a + w * v.y, acc.z * a + w * v.z, acc.w * a + w * v.w);
        }
        const int in_tile = (r0 + i) % kPfRows, tok = (r0 + i) / kPfRows * p.tile_tokens + in_tile / p.G;
        const float inv = den != 0.0f ? 1.0f / den : 0.0f;
        const int64_t orow = (int64_t)(mg.row0 + tok) * p.heads + mg.g * p.G + in_tile % p.G;
        *reinterpret_cast<uint2 *>(p.out + orow * kDv + 4 * lane) =
            pack_bf16x4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (lane == 0 && p.lse_out) p.lse_out[orow] = den != 0.0f ? M + logf(den) : -INFINITY;
    }
}

}  // namespace

extern thread_local int g_drop_v_unit;  // set by gqla_debug_drop_v_load

cudaError_t launch_prefill_gqa(const void *q, int64_t total_q, const int32_t *q_starts, int heads, int num_groups,
                               const void *kv, const void *k_rope, int64_t num_slots, const gqla_kv_index *idx,
                               int num_splits, bool whole, float scale, float *o_part, float *lse_part, void *out,
                               float *lse_out, void *ws, cudaStream_t stream) {
    const int G = heads / num_groups;
    PfParams p;
    p.q_starts = q_starts;
    p.page_table = idx->page_table;
    p.seqlens = idx->seqlens;
    p.o_part = o_part;
    p.lse_part = lse_part;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse_out = lse_out;
    p.ws = ws;
    p.total_q = total_q;
    p.num_slots = num_slots;
    p.batch = idx->batch;
    p.max_pages = idx->max_pages_per_seq;
    p.num_pages = idx->num_pages;
    p.num_splits = num_splits;
    p.whole = whole;
    p.drop_v = g_drop_v_unit;
    g_drop_v_unit = -1;
    p.heads = heads;
    p.groups = num_groups;
    p.G = G;
    p.tile_tokens = pf_tile_tokens(G);
    p.scale_log2 = scale * kLog2e;
    CUtensorMap kvm, krm, qm, qtm;
    {
        const uint64_t dims[3] = {(uint64_t)kKv, (uint64_t)num_slots, (uint64_t)num_groups};
        const uint64_t strides[2] = {(uint64_t)kKv * 2, (uint64_t)num_slots * kKv * 2};
        const uint32_t box[3] = {64, 64, 1};
        if (!make_bf16_map(&kvm, kv, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    }
    {
        const uint64_t dims[2] = {(uint64_t)kRope, (uint64_t)num_slots};
        const uint64_t strides[1] = {(uint64_t)kRope * 2};
        const uint32_t box[2] = {64, 64};
        if (!make_bf16_map(&krm, k_rope, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    }
    {  // a box is the G heads of one group for the tokens of one MMA tile
        const uint64_t dims[3] = {(uint64_t)kQk, (uint64_t)heads, (uint64_t)total_q};
        const uint64_t strides[2] = {(uint64_t)kQk * 2, (uint64_t)heads * kQk * 2};
        const uint32_t box[3] = {64, (uint32_t)G, (uint32_t)p.tile_tokens};
        const uint32_t one[3] = {64, (uint32_t)G, 1};
        if (!make_bf16_map(&qm, q, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_bf16_map(&qtm, q, 3, dims, strides, one, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = once_per_device(ready, [] {
        cudaError_t r = cudaFuncSetAttribute(prefill_gqa_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             PfSmem::kAlloc);
        cudaFuncAttributes fa;
        if (r == cudaSuccess) r = cudaFuncGetAttributes(&fa, prefill_gqa_kernel);
        if (r != cudaSuccess) return r;
        // the register split must not ask for more than the launch gives
        return 128 * kPfIssueRegs + 256 * kPfSoftmaxRegs > kPfThreads * fa.numRegs ? cudaErrorInvalidConfiguration
                                                                                     : cudaSuccess;
    });
    if (e != cudaSuccess) return e;
    e = launch_dependent(prefill_gqa_kernel, dim3(2 * num_splits), dim3(kPfThreads), PfSmem::kAlloc, stream, kvm, krm, qm,
                         qtm, p);
    if (e != cudaSuccess || whole) return e;
    return launch_dependent(prefill_combine_kernel, dim3(num_splits - 1, kPfBlockRows / kPcRows),
                            dim3(32 * kPcWarps), 0, stream, p);
}

}  // namespace gqla
