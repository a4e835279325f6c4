// pages.cu -- the pages of a paged cache: copied, forked, extended, freed, compacted.
//
// page_refs[p] counts the used page-table entries that name page p; 0 is a free page. New
// pages are always the lowest free ones, in list order, so every result is the same on
// every run (reference counts change by integer atomics, whose order does not matter).
//
// The table calls are latency-bound, one launch each: 256 forks of sequences of 1500 tokens 9 us,
// 288 sequences extended 6.8 us, a pool of 2048 pages compacted 11 us. Fork and compact run as
// one cluster of eight CTAs, whose first CTA scans the reference counts while the others wait
// at the cluster barrier, and which then rewrite the table rows together. Of larger pools the scan
// of one CTA shows: 20000 pages 27 us to compact and 10 us for 64 forks, 200000 pages 216 and 19 us;
// extend, which stops where it has found enough, stays at 7 us.
#include <limits.h>

#include "common.cuh"
#include "sm100.cuh"

namespace gqla {

namespace {

using namespace sm100;

constexpr int kPgThreads = 1024;
constexpr int kPgCluster = 8;

struct PgPool {
    int32_t *table, *lens, *refs;
    int batch, max_pages, num_pages;
    void *ws;
};

// Sum of v over the block's threads before this one; *total the sum over all. The warps'
// sums go through `part` (32 + 1 values).
template <typename T>
__device__ __forceinline__ T block_excl_scan(T v, T *part, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        T w = lane < (int)(blockDim.x >> 5) ? part[lane] : 0;
        T s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T n = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += n;
        }
        part[lane] = s - w;
        if (lane == 31) part[32] = s;
    }
    __syncthreads();
    const T r = part[warp] + incl - v;
    *total = part[32];
    __syncthreads();
    return r;
}

// ---------------------------------------------------------------------------
// Copy. Every cache is cut into 8 KB pieces (a latent page is nine of them, a group's plane
// of a page four, the RoPE keys one); piece after piece passes through a ring in shared
// memory by bulk copies (global -> shared -> global), driven by one thread per CTA, so that
// up to 80 KB per SM are on their way. Bound by HBM: 490 pages (337 MB read and written) 53 us,
// 6.4 TB/s. What the pairs may not do -- write a page twice, or read one that another pair
// writes -- would make the result depend on timing: each CTA marks the written pages in a
// bitmap first and leaves such pairs out (reported).
// ---------------------------------------------------------------------------
constexpr int kCpThreads = 256;
constexpr int kCpPiece = 8192;
constexpr int kCpStages = 10, kCpLag = 6;  // stages; loads issued ahead of the stores
constexpr int kLatPieces = kPage * kRow * 2 / kCpPiece;   // 9
constexpr int kKvPieces = kPage * kKv * 2 / kCpPiece;     // 4 per group
static_assert(kPage * kRow * 2 % kCpPiece == 0 && kPage * kKv * 2 % kCpPiece == 0, "pieces");
constexpr int kCpMaxPages = 1 << 19;  // two bitmaps of 64 KB

struct CpParams {
    const int2 *pairs;
    uint8_t *latent, *kv, *rope;
    void *ws;
    int64_t n, num_pages;
    int pieces, lat_pieces, kv_pieces, words;
};

__device__ __forceinline__ int ld_cluster_b32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Where piece `x` of page `page` lies.
__device__ __forceinline__ uint8_t *piece_ptr(const CpParams &p, int x, int64_t page) {
    if (x < p.lat_pieces) return p.latent + (page * kLatPieces + x) * kCpPiece;
    x -= p.lat_pieces;
    if (x < p.kv_pieces)
        return p.kv + (((int64_t)(x / kKvPieces) * p.num_pages + page) * kKvPieces + x % kKvPieces) * kCpPiece;
    return p.rope + page * kCpPiece;
}

__global__ void __launch_bounds__(kCpThreads, 1) copy_pages_kernel(const CpParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *ring = smem;
    uint32_t *written = reinterpret_cast<uint32_t *>(smem + kCpStages * kCpPiece), *twice = written + p.words;
    __shared__ uint64_t full[kCpStages];
    __shared__ uint8_t *from[kCpThreads], *to[kCpThreads];
    __shared__ int count, stop, part[33];
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < kCpStages; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
        stop = 0;
    }
    for (int i = tid; i < 2 * p.words; i += kCpThreads) written[i] = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    auto inside = [&](int2 v) {
        return v.x >= 0 && v.y >= 0 && v.x < p.num_pages && v.y < p.num_pages && v.x != v.y;
    };
    for (int64_t i = tid; i < p.n; i += kCpThreads) {
        const int2 v = p.pairs[i];
        if (!inside(v)) continue;
        const uint32_t bit = 1u << (v.y & 31);
        if (atomicOr(&written[v.y >> 5], bit) & bit) atomicOr(&twice[v.y >> 5], bit);
    }
    __syncthreads();
    const int64_t units = p.n * p.pieces;
    uint32_t done = 0;  // pieces that passed through the ring
    for (int64_t u0 = blockIdx.x; u0 < units; u0 += (int64_t)kCpThreads * gridDim.x) {
        // the next 256 pieces of this CTA, those of pairs that move nothing left out
        const int64_t u = u0 + (int64_t)tid * gridDim.x;
        bool go = false;
        uint8_t *src = nullptr, *dst = nullptr;
        if (u < units) {
            const int64_t pr = u / p.pieces;
            const int x = (int)(u - pr * p.pieces);
            const int2 v = p.pairs[pr];
            const bool unused = v.x < 0 || v.x == v.y;
            go = inside(v);
            if (go) {
                const bool clash = (twice[v.y >> 5] >> (v.y & 31) & 1) || (written[v.x >> 5] >> (v.x & 31) & 1);
                if (clash && x == 0) report_error(p.ws, GQLA_ERR_DEVICE, (int)pr);
                go = !clash;
            } else if (!unused && x == 0) {
                report_error(p.ws, GQLA_ERR_DEVICE, (int)pr);
            }
            if (go) {
                src = piece_ptr(p, x, v.x);
                dst = piece_ptr(p, x, v.y);
            }
        }
        int total;
        const int at = block_excl_scan<int>(go ? 1 : 0, part, &total);
        if (go) {
            from[at] = src;
            to[at] = dst;
        }
        if (tid == 0) count = total;
        __syncthreads();
        if (tid == 0 && !stop) {
            const int n = count;
            for (int k = 0; k < n + kCpLag && !stop; ++k) {
                if (k < n) {
                    const uint32_t st = (done + k) % kCpStages;
                    // the store that used this stage, kCpStages pieces ago, has read it: at most
                    // the kCpStages - kCpLag - 1 stores after it are still pending
                    bulk_wait_group_read<kCpStages - kCpLag - 1>();
                    mbar_arrive_expect_tx(&full[st], kCpPiece);
                    bulk_load(ring + st * kCpPiece, from[k], kCpPiece, &full[st]);
                }
                const int j = k - kCpLag;
                if (j >= 0) {
                    const uint32_t q = done + j, st = q % kCpStages;
                    if (!mbar_wait(&full[st], (q / kCpStages) & 1, &stop)) {
                        stop = 1;
                        report_error(p.ws, GQLA_ERR_TIMEOUT, (int)blockIdx.x);
                        int dummy = 0;  // never leave with copies in flight
                        for (int i = j + 1; i <= k && i < n; ++i)
                            mbar_wait(&full[(done + i) % kCpStages], ((done + i) / kCpStages) & 1,
                                      reinterpret_cast<volatile int *>(&dummy));
                        break;
                    }
                    bulk_store(to[j], ring + st * kCpPiece, kCpPiece);
                    bulk_commit_group();
                }
            }
            done += n;
        }
        __syncthreads();
    }
    if (tid == 0) bulk_wait_group<0>();
}

// ---------------------------------------------------------------------------
// Fork. forks[i] = {parent, child}: the child (an empty sequence) gets the parent's full
// pages, and a fresh page in place of a partly filled last one, whose copy is left to the
// caller as pairs[i] = {parent's page, fresh page} (-1, -1: nothing to copy).
// ---------------------------------------------------------------------------
struct FkParams {
    PgPool pool;
    const int2 *forks;
    int2 *pairs;
    int n;
};

// One block: the free pages from page `*cursor` on, in ascending order, up to `need` of them, into
// `list` (if not null). Returns how many there are; *cursor ends at the pages looked at last. A warp
// looks at 256 consecutive pages at a time, 32 with each load.
constexpr int kPgList = 2048;  // pages that a list in shared memory holds

__device__ int collect_free(const PgPool &p, int need, int *cursor, int *list, int *part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int found = 0;
    for (int base = *cursor; base < p.num_pages && found < need; base += kPgThreads * 8) {
        const int first = base + warp * 256;
        uint32_t mask[8];
        int mine = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int page = first + 32 * j + lane;
            mask[j] = __ballot_sync(0xffffffffu, page < p.num_pages && p.refs[page] == 0);
            mine += __popc(mask[j]);
        }
        __syncthreads();  // part and list were read
        if (lane == 0) part[warp] = mine;
        __syncthreads();
        const int of_warp = part[lane];
        const int incl = warp_incl_scan(of_warp);
        int rank = found + __shfl_sync(0xffffffffu, incl - of_warp, warp);
        found += __shfl_sync(0xffffffffu, incl, 31);
        if (list) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = rank + __popc(mask[j] & ((1u << lane) - 1));
                if ((mask[j] >> lane & 1) && r < need) list[r] = first + 32 * j + lane;
                rank += __popc(mask[j]);
            }
        }
        *cursor = base;
    }
    __syncthreads();
    return min(found, need);
}

__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    fork_kernel(const FkParams p) {
    extern __shared__ uint8_t smem[];
    const PgPool &pool = p.pool;
    const int words = (pool.batch + 31) / 32;
    uint32_t *child_bit = reinterpret_cast<uint32_t *>(smem), *twice = child_bit + words;
    uint8_t *state = reinterpret_cast<uint8_t *>(twice + words);  // per fork: 0 refused, 1 no copy, 2 one page
    __shared__ int part[33];
    const int tid = threadIdx.x, rank = cluster_rank();
    for (int i = tid; i < 2 * words; i += kPgThreads) child_bit[i] = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    for (int i = tid; i < p.n; i += kPgThreads) {
        const int ch = p.forks[i].y;
        if (ch < 0 || ch >= pool.batch) continue;
        const uint32_t bit = 1u << (ch & 31);
        if (atomicOr(&child_bit[ch >> 5], bit) & bit) atomicOr(&twice[ch >> 5], bit);
    }
    __syncthreads();
    // every CTA judges all forks (they read the lengths before any CTA writes one)
    int need = 0;
    for (int i0 = 0; i0 < p.n; i0 += kPgThreads) {
        const int i = i0 + tid;
        int st = 0, src = -1;
        if (i < p.n) {
            const int2 f = p.forks[i];
            if (f.x >= 0 && f.y >= 0 && f.x < pool.batch && f.y < pool.batch && f.x != f.y &&
                !(twice[f.y >> 5] >> (f.y & 31) & 1) && !(child_bit[f.x >> 5] >> (f.x & 31) & 1)) {
                const int L = pool.lens[f.x];
                if (L >= 0 && pool.lens[f.y] == 0 && (int64_t)L <= (int64_t)pool.max_pages * kPage) {
                    st = 1;
                    if (L % kPage) {
                        src = pool.table[(int64_t)f.x * pool.max_pages + L / kPage];
                        st = src >= 0 && src < pool.num_pages ? 2 : 0;
                    }
                }
            }
            state[i] = (uint8_t)st;
            if (rank == 0) {
                if (!st) report_error(pool.ws, GQLA_ERR_DEVICE, i);
                p.pairs[i] = make_int2(st == 2 ? src : -1, -1);
            }
        }
        need += __syncthreads_count(st == 2);
    }
    if (rank == 0 && need > 0) {
        // the takers in list order, 1024 forks at a time: rank of a fork -> fork
        __shared__ int taker[kPgThreads], list[kPgThreads];
        int cursor = 0;
        for (int i0 = 0; i0 < p.n; i0 += kPgThreads) {
            const int i = i0 + tid;
            const bool takes = i < p.n && state[i] == 2;
            int total;
            const int r = block_excl_scan<int>(takes ? 1 : 0, part, &total);
            if (takes) taker[r] = i;
            __syncthreads();
            const int given = collect_free(pool, total, &cursor, list, part);
            if (tid < given) {
                p.pairs[taker[tid]].y = list[tid];
                pool.refs[list[tid]] = 1;
            }
            for (int k = given + tid; k < total; k += kPgThreads) {  // the pool is full
                p.pairs[taker[k]] = make_int2(-1, -1);
                report_error(pool.ws, GQLA_ERR_DEVICE, taker[k]);
            }
            __syncthreads();  // the next forks' pages are looked for among refs as they are now
        }
    }
    cluster_sync();
    // rows, a warp to a fork
    const int lane = tid & 31;
    for (int i = (rank * kPgThreads + tid) >> 5; i < p.n; i += kPgCluster * kPgThreads / 32) {
        const int st = state[i];
        if (st == 0) continue;
        const int2 f = p.forks[i];
        const int fresh = st == 2 ? __ldcg(&p.pairs[i].y) : -1;
        if (st == 2 && fresh < 0) continue;
        const int L = pool.lens[f.x];
        const int32_t *from = pool.table + (int64_t)f.x * pool.max_pages;
        int32_t *to = pool.table + (int64_t)f.y * pool.max_pages;
        for (int j = lane; j < L / kPage; j += 32) {
            const int page = from[j];
            to[j] = page;
            if (page >= 0 && page < pool.num_pages) atomicAdd(&pool.refs[page], 1);
            else report_error(pool.ws, GQLA_ERR_DEVICE, i);
        }
        if (lane == 0) {
            if (st == 2) to[L / kPage] = fresh;
            pool.lens[f.y] = L;
        }
    }
}

// ---------------------------------------------------------------------------
// Extend: new_tokens[b] more tokens for every sequence, and the pages they need.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPgThreads) extend_kernel(const PgPool p, const int32_t *new_tokens) {
    __shared__ int part[33], before[kPgThreads], owner_pages[kPgThreads], list[kPgList];
    __shared__ long long part64[33];
    const int tid = threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    bool full = false;  // a sequence found too few pages: it and those after it that need one get none
    int cursor = 0;     // no free page lies below
    for (int b0 = 0; b0 < p.batch; b0 += kPgThreads) {
        const int b = b0 + tid;
        int add = 0, have = 0;
        int64_t len = 0;
        bool grow = false;
        if (b < p.batch) {
            const int L = p.lens[b], n = new_tokens[b];
            len = (int64_t)L + n;
            grow = n > 0 && L >= 0 && len <= min((int64_t)p.max_pages * kPage, (int64_t)INT_MAX);
            if (n != 0 && !grow) report_error(p.ws, GQLA_ERR_DEVICE, b);
            have = pages_of(L);
            add = grow ? (int)((len + kPage - 1) / kPage) - have : 0;
        }
        // 64 bits: what is asked for may pass 2^31 pages, what there is does not
        long long all;
        const long long mine = block_excl_scan<long long>(add, part64, &all);
        const int total = (int)min(all, (long long)INT_MAX);
        before[tid] = (int)min(mine, (long long)INT_MAX);
        owner_pages[tid] = have;
        // how many of the pages that these sequences need there are; up to kPgList of them are
        // in the list already
        const bool listed = total <= kPgList;
        int there = 0, from = cursor;
        if (!full && total > 0) there = collect_free(p, total, &from, listed ? list : nullptr, part);
        // granted: the sequences whose pages end within those
        const bool ok = mine + add <= there;
        if (grow) {
            if (add == 0 || ok) p.lens[b] = (int)len;
            else report_error(p.ws, GQLA_ERR_DEVICE, b);
        }
        // the grants are a prefix of the ranks; its end
        int limit = add > 0 && ok ? (int)mine + add : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) limit = max(limit, __shfl_xor_sync(0xffffffffu, limit, o));
        __syncthreads();
        if ((tid & 31) == 0) part[tid >> 5] = limit;
        __syncthreads();
        limit = part[tid & 31];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) limit = max(limit, __shfl_xor_sync(0xffffffffu, limit, o));
        for (int given = 0; given < limit;) {
            const int n = listed ? limit : collect_free(p, min(limit - given, kPgList), &cursor, list, part);
            if (n == 0) {  // pages that were counted are gone: another call is taking them meanwhile
                if (tid == 0) report_error(p.ws, GQLA_ERR_DEVICE, b0);
                break;
            }
            for (int k = tid; k < n; k += kPgThreads) {
                const int r = given + k;
                int lo = 0, hi = kPgThreads;  // the last sequence whose ranks start at or before r
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (before[mid] <= r) lo = mid;
                    else hi = mid;
                }
                p.table[(int64_t)(b0 + lo) * p.max_pages + owner_pages[lo] + r - before[lo]] = list[k];
                p.refs[list[k]] = 1;
            }
            given += n;
            __syncthreads();
        }
        full = full || there < total;
        if (listed) cursor = max(cursor, from);  // all free pages before it are taken, or `full` is set
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Free: a warp per listed sequence. A sequence listed twice is freed once (the exchange of
// its length lets one warp through).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) free_kernel(const PgPool p, const int32_t *ids, int n) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int i = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (i >= n) return;
    const int b = ids[i];
    if (b < 0 || b >= p.batch) {
        if (lane == 0) report_error(p.ws, GQLA_ERR_DEVICE, i);
        return;
    }
    int L = 0;
    if (lane == 0) L = atomicExch(&p.lens[b], 0);
    L = __shfl_sync(0xffffffffu, L, 0);
    if ((int64_t)L > (int64_t)p.max_pages * kPage) {
        if (lane == 0) report_error(p.ws, GQLA_ERR_DEVICE, i);
        L = p.max_pages * kPage;
    }
    for (int j = lane; j < pages_of(L); j += 32) {
        const int page = p.table[(int64_t)b * p.max_pages + j];
        if (page < 0 || page >= p.num_pages) {
            report_error(p.ws, GQLA_ERR_DEVICE, i);
        } else if (atomicSub(&p.refs[page], 1) <= 0) {  // it was free: put the count back
            atomicAdd(&p.refs[page], 1);
            report_error(p.ws, GQLA_ERR_DEVICE, i);
        }
    }
}

// ---------------------------------------------------------------------------
// Compact: with N live pages, the live pages of index >= N move to the free ones below N,
// ascending to ascending; pairs lists the moves (their copy is left to the caller) and the
// table and the counts come out rewritten. In between, refs_out of a page that moves holds
// its new index, of a free page above N -1.
// ---------------------------------------------------------------------------
struct CmParams {
    PgPool pool;
    int32_t *table_out, *refs_out;
    int2 *pairs;
    int32_t *counts;  // {live pages, moves}
};

__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    compact_kernel(const CmParams p) {
    __shared__ unsigned long long part[33];
    __shared__ int s_live;
    const PgPool &pool = p.pool;
    const int tid = threadIdx.x, rank = cluster_rank(), N = pool.num_pages;
    constexpr int kPer = 8;
    griddep_wait();
    griddep_launch_dependents();
    if (rank == 0) {
        int mine = 0;
        for (int i = tid; i < N; i += kPgThreads) mine += pool.refs[i] > 0;
        unsigned long long total;
        block_excl_scan<unsigned long long>(mine, part, &total);
        const int live = (int)total;
        unsigned long long done = 0;  // moves found so far: high word sources, low word targets
        for (int base = 0; base < N; base += kPgThreads * kPer) {
            const int first = base + tid * kPer;
            uint32_t src = 0, dst = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int page = first + j;
                if (page >= N) break;
                const bool used = pool.refs[page] > 0;
                if (used && page >= live) src |= 1u << j;
                if (!used && page < live) dst |= 1u << j;
            }
            const unsigned long long at =
                done + block_excl_scan<unsigned long long>(((unsigned long long)__popc(src) << 32) | __popc(dst), part, &total);
            int a = (int)(at >> 32), b = (int)(at & 0xffffffffu);
            for (; src; src &= src - 1) p.pairs[a++].x = first + __ffs(src) - 1;
            for (; dst; dst &= dst - 1) p.pairs[b++].y = first + __ffs(dst) - 1;
            done += total;
        }
        const int moves = (int)(done >> 32);
        __syncthreads();
        for (int i = tid; i < N; i += kPgThreads) {
            const int r = pool.refs[i];
            if (i < live) {
                if (r > 0) p.refs_out[i] = r;
            } else if (r <= 0) {
                p.refs_out[i] = -1;
            }
        }
        __syncthreads();
        for (int i = tid; i < max(1, N / 2); i += kPgThreads) {
            if (i < moves) {
                const int2 v = p.pairs[i];
                p.refs_out[v.y] = pool.refs[v.x];
                p.refs_out[v.x] = v.y;
            } else {
                p.pairs[i] = make_int2(-1, -1);
            }
        }
        if (tid == 0) {
            p.counts[0] = live;
            p.counts[1] = moves;
            s_live = live;
        }
    }
    cluster_sync();
    const int live = ld_cluster_b32(map_peer(smem_u32(&s_live), 0));
    // table rows, a warp to a sequence
    const int lane = tid & 31;
    for (int b = (rank * kPgThreads + tid) >> 5; b < pool.batch; b += kPgCluster * kPgThreads / 32) {
        const int used = min(pages_of(pool.lens[b]), pool.max_pages);
        if (pages_of(pool.lens[b]) > pool.max_pages && lane == 0) report_error(pool.ws, GQLA_ERR_DEVICE, b);
        for (int j = lane; j < pool.max_pages; j += 32) {
            const int64_t at = (int64_t)b * pool.max_pages + j;
            int page = pool.table[at];
            if (j < used) {
                if (page < 0 || page >= N) {
                    report_error(pool.ws, GQLA_ERR_DEVICE, b);
                } else if (page >= live) {
                    const int to = __ldcg(&p.refs_out[page]);
                    if (to < 0) report_error(pool.ws, GQLA_ERR_DEVICE, b);  // a used page whose count is 0
                    else page = to;
                }
            }
            p.table_out[at] = page;
        }
    }
    cluster_sync();
    for (int i = live + rank * kPgThreads + tid; i < N; i += kPgCluster * kPgThreads) p.refs_out[i] = 0;
}

PgPool make_pool(const gqla_page_pool *pool, void *ws) {
    return PgPool{pool->page_table, pool->seqlens, pool->page_refs, pool->batch, pool->max_pages_per_seq,
                  pool->num_pages, ws};
}

}  // namespace

int64_t copy_pages_limit() { return kCpMaxPages; }

cudaError_t launch_copy_pages(const int32_t *pairs, int64_t n, int num_pages, int num_groups, void *latent, void *kv,
                              void *k_rope, void *ws, cudaStream_t stream) {
    CpParams p;
    p.pairs = reinterpret_cast<const int2 *>(pairs);
    p.latent = static_cast<uint8_t *>(latent);
    p.kv = static_cast<uint8_t *>(kv);
    p.rope = static_cast<uint8_t *>(k_rope);
    p.ws = ws;
    p.n = n;
    p.num_pages = num_pages;
    p.lat_pieces = latent ? kLatPieces : 0;
    p.kv_pieces = kv ? num_groups * kKvPieces : 0;
    p.pieces = p.lat_pieces + p.kv_pieces + (k_rope ? 1 : 0);
    p.words = (num_pages + 31) / 32;
    const int bytes = kCpStages * kCpPiece + 2 * p.words * 4;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = once_per_device(ready, [] {
        return cudaFuncSetAttribute(copy_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kCpStages * kCpPiece + 2 * (kCpMaxPages / 32) * 4);
    });
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t units = n * p.pieces;
    return launch_dependent(copy_pages_kernel, dim3((unsigned)(units < sms ? units : sms)), dim3(kCpThreads), bytes,
                            stream, p);
}

cudaError_t launch_fork(const gqla_page_pool *pool, const int32_t *forks, int n, int32_t *pairs, void *ws,
                        cudaStream_t stream) {
    FkParams p{make_pool(pool, ws), reinterpret_cast<const int2 *>(forks), reinterpret_cast<int2 *>(pairs), n};
    const int bytes = 2 * ((pool->batch + 31) / 32) * 4 + n;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = once_per_device(ready, [] {
        return cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(fork_kernel, dim3(kPgCluster), dim3(kPgThreads), bytes, stream, p);
}

cudaError_t launch_extend(const gqla_page_pool *pool, const int32_t *new_tokens, void *ws, cudaStream_t stream) {
    return launch_dependent(extend_kernel, dim3(1), dim3(kPgThreads), 0, stream, make_pool(pool, ws), new_tokens);
}

cudaError_t launch_free(const gqla_page_pool *pool, const int32_t *ids, int n, void *ws, cudaStream_t stream) {
    return launch_dependent(free_kernel, dim3((unsigned)((n + 7) / 8)), dim3(256), 0, stream, make_pool(pool, ws), ids, n);
}

cudaError_t launch_compact(const gqla_page_pool *pool, int32_t *table_out, int32_t *refs_out, int32_t *pairs,
                           int32_t *counts, void *ws, cudaStream_t stream) {
    CmParams p{make_pool(pool, ws), table_out, refs_out, reinterpret_cast<int2 *>(pairs), counts};
    return launch_dependent(compact_kernel, dim3(kPgCluster), dim3(kPgThreads), 0, stream, p);
}

}  // namespace gqla
