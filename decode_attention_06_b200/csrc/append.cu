// append.cu -- the rows of new tokens into the pages of the caches: the latent row itself,
// and for the GQA path its per-group projections K_nope = c W_UK_g, V = c W_UV_g and the
// shared RoPE key (GQLA, paperlayer.ai summary, sec. 3 "Two equivalent decoding paths": what
// the one-shot expansion does to a whole cache, done to the tokens of one step or prompt).
//
//   D[256 rows x NC] = A[256 x 512] * B[512 x NC],  B = [W_UK_g | W_UV_g] (NC = 256) or one of
//   the two (NC = 128)
//
// A CTA pair (cta_group::2) takes 256 rows and a share of the products: each CTA holds its 128
// rows of A (K-major, 128 KB) for all of them and streams one half of B's columns (MN-major,
// the weights as stored) through a ring of 64-row slabs, so that the weights cross from L2
// once per 256 rows; two TMEM accumulators let the epilogue of one product run during the
// next. The cache slot of a row follows from q_starts, the lengths and the page table; the
// threads look theirs up while the operands are on their way. Two warps copy the latent rows
// and the RoPE keys.
//
// Bound by the tensor cores for many rows (2.1 MFLOP a row at 8 groups against 6.5 KB) and by
// latency for a step's rows: 7752 rows 20.4 us (798 TFLOP/s, 2.6 TB/s: four groups a pair in one
// wave, 9 us of MMA, the rest the launch, the first operands' way in and the last group's out),
// 128 rows 7.5 us. Into the latent cache alone (2304 bytes a row, no product): 7752 rows 6.1 us
// against 2.7 of HBM, 128 rows 4.8 us: launch, the rows' slots, one copy in and one out.
#include <cuda.h>

#include "common.cuh"
#include "ragged.cuh"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace gqla {

namespace {

using namespace sm100;

constexpr int kApRows = 128;               // rows of one CTA
constexpr int kApThreads = 384;
constexpr int kApBoxA = kApRows * 128;     // [128 rows][64 latent columns]
constexpr int kApA = 8 * kApBoxA;
constexpr int kApSlab = 64;                // K rows of B per ring stage
constexpr int kApBoxB = kApSlab * 128;     // [64 K rows][64 columns]
constexpr int kApStages = 4;
constexpr int kApSlabs = kLatent / kApSlab;
constexpr int kApCopyRows = 16;            // rows copied at a time by the two copying warps
constexpr int kApCopyBytes = kApCopyRows / 2 * kRow * 2;  // one warp's

template <int NC>
struct ApSmem {
    static constexpr int kStage = NC / 128 * kApBoxB;  // one CTA's NC / 2 columns
    static constexpr int oA = 0;
    static constexpr int oB = oA + kApA;
    static constexpr int oCopy = oB + kApStages * kStage;
    static constexpr int oBar = oCopy + 2 * kApCopyBytes;
    // a_full[8], b_full/b_empty[kApStages], acc_full/acc_empty[2], drain, copy[2]
    static constexpr int kNumBars = 8 + 2 * kApStages + 4 + 1 + 2;
    static constexpr int oMisc = oBar + kNumBars * 8;
    static constexpr int kAlloc = oMisc + 16 + 1024;
};
static_assert(ApSmem<256>::kAlloc <= 227 * 1024, "shared memory");

struct ApParams {
    const uint4 *rows;            // [total][576] bf16
    const int32_t *q_starts, *seqlens, *page_table;
    uint4 *latent;                // [num_slots][576] bf16, or null
    __nv_bfloat16 *kv;            // [g][num_slots][256], or null
    uint4 *k_rope;                // [num_slots][64] bf16, or null
    void *ws;
    int64_t total, num_slots;
    int batch, max_pages, num_pages;
    int products;                 // products (of NC columns) of one pair
};

// Cache slot of row r (of no row where !has), or -1 if it belongs to no (valid) sequence or its
// page is outside the pool (reported when `report`). By the whole warp: each lane bisects for
// the last b with q_starts[b] <= r; rows that this leaves without a sequence are looked for in
// all of them if the starts do not ascend (then a valid sequence may lie beside the bad ones).
__device__ int64_t ap_slot(const ApParams &p, int64_t r, bool has, bool report) {
    int lo = 0, hi = p.batch;  // q_starts[lo] <= r < q_starts[hi], where they ascend
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.q_starts[mid] <= r) lo = mid;
        else hi = mid;
    }
    auto owns = [&](const RaggedSeq &s) { return r >= s.q0 && r < s.q0 + s.n; };
    RaggedSeq s = ragged_seq(p.q_starts, p.seqlens, lo, p.total, p.max_pages);
    bool found = owns(s);
    if (__any_sync(0xffffffffu, has && !found)) {
        bool falls = false;
        for (int b = threadIdx.x & 31; b < p.batch; b += 32) falls |= p.q_starts[b + 1] < p.q_starts[b];
        if (__any_sync(0xffffffffu, falls))
            for (int b = 0; b < p.batch && has && !found; ++b) {
                s = ragged_seq(p.q_starts, p.seqlens, lo = b, p.total, p.max_pages);
                found = owns(s);
            }
        __syncwarp();
    }
    if (!has || !found) return -1;
    const int t = s.L - s.n + (int)(r - s.q0);
    const int page = p.page_table[(int64_t)lo * p.max_pages + t / kPage];
    if (page < 0 || page >= p.num_pages) {
        if (report) report_error(p.ws, GQLA_ERR_DEVICE, lo);
        return -1;
    }
    return (int64_t)page * kPage + t % kPage;
}

// One warp of two: this CTA's share of its tile's latent rows and RoPE keys, eight rows at a
// time through shared memory by bulk copies (one in, one or two out per row). Row by row
// through registers the copies took twice as long as the products beside them.
__device__ __forceinline__ void ap_copy(const ApParams &p, int64_t row0, int w, uint8_t *stage, uint64_t *bar,
                                        volatile int *abort_flag) {
    constexpr int kRowBytes = kRow * 2;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int b = 32 * w + lane; b < p.batch; b += 64)
            if (ragged_seq(p.q_starts, p.seqlens, b, p.total, p.max_pages).bad) report_error(p.ws, GQLA_ERR_DEVICE, b);
    uint32_t n = 0;
    for (int r0 = blockIdx.y * kApCopyRows; r0 < kApRows; r0 += gridDim.y * kApCopyRows, ++n) {
        const int64_t r = row0 + r0 + w * kApCopyRows / 2;
        const int rows = (int)min((int64_t)kApCopyRows / 2, p.total - r);
        if (rows <= 0) break;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar, rows * kRowBytes);
            bulk_load(stage, reinterpret_cast<const uint8_t *>(p.rows) + r * kRowBytes, rows * kRowBytes, bar);
        }
        const int64_t s = ap_slot(p, r + lane, lane < rows, true);
        if (!__all_sync(0xffffffffu, mbar_wait(bar, n & 1, abort_flag))) {
            *abort_flag = 1;
            int dummy = 0;  // never leave with a copy in flight
            mbar_wait(bar, n & 1, &dummy);
            break;
        }
        if (s >= 0) {
            const uint8_t *row = stage + lane * kRowBytes;
            if (p.latent) bulk_store(reinterpret_cast<uint8_t *>(p.latent) + s * kRowBytes, row, kRowBytes);
            if (p.k_rope) bulk_store(reinterpret_cast<uint8_t *>(p.k_rope) + s * kRope * 2, row + kLatent * 2, kRope * 2);
        }
        bulk_commit_group();
        bulk_wait_group_read<0>();
        __syncwarp();
    }
    bulk_wait_group<0>();
}

// Latent cache only (no expansion).
__global__ void __launch_bounds__(64) append_latent_kernel(const ApParams p) {
    __shared__ __align__(128) uint8_t stage[2][kApCopyBytes];
    __shared__ uint64_t bar[2];
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar[0], 1);
        mbar_init(&bar[1], 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int w = threadIdx.x >> 5;
    ap_copy(p, (int64_t)blockIdx.x * kApRows, w, stage[w], &bar[w], &abort_flag);
    __syncthreads();
    if (threadIdx.x == 0 && abort_flag) report_error(p.ws, GQLA_ERR_TIMEOUT, (int)blockIdx.x);
}

template <int NC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kApThreads, 1)
    append_kernel(const __grid_constant__ CUtensorMap row_map, const __grid_constant__ CUtensorMap wuk_map,
                  const __grid_constant__ CUtensorMap wuv_map, const ApParams p) {
    using SM = ApSmem<NC>;
    constexpr int ST = kApStages;
    const int64_t row0 = (int64_t)blockIdx.x * kApRows;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *a_full = reinterpret_cast<uint64_t *>(smem + SM::oBar);
    uint64_t *b_full = a_full + 8, *b_empty = b_full + ST, *acc_full = b_empty + ST, *acc_empty = acc_full + 2;
    uint64_t *drain = acc_empty + 2, *copy_bar = drain + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SM::oMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SM::oMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int first = blockIdx.y * p.products;  // this pair's first product
    // the barriers that the MMA issuer waits for are those of rank 0
    auto lead = [](uint64_t *bar) { return map_peer(smem_u32(bar), 0); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(&a_full[i], 1);
        for (int i = 0; i < ST; ++i) { mbar_init(&b_full[i], 1); mbar_init(&b_empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 16); }
        mbar_init(drain, 1);
        mbar_init(&copy_bar[0], 1);
        mbar_init(&copy_bar[1], 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&row_map);
        prefetch_tensormap(&wuk_map);
        prefetch_tensormap(&wuv_map);
    }
    __syncwarp();
    cluster_arrive();  // this thread's barriers are initialised
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
        tc_fence_before();
    }
    __syncthreads();
    cluster_wait();  // the other CTA's are too
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch_dependents();

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (elect_one()) {
            int u = 0;
            for (int x = 0; x < p.products && !*abort_flag; ++x) {
                // this CTA's columns: of W_UK_g or W_UV_g, all 128 (NC = 256) or 64 of them
                const int v = first + x, g = v * NC / kKv;
                const CUtensorMap *w_map = (NC == 256 ? (int)rank : v & 1) ? &wuv_map : &wuk_map;
                for (int kb = 0; kb < kApSlabs; ++kb, ++u) {
                    if (x == 0) {  // a box of A with each slab of the first product
                        if (rank == 0) mbar_arrive_expect_tx(&a_full[kb], 2 * kApBoxA);
                        tma_load_2d_pair(smem + SM::oA + kb * kApBoxA, &row_map, lead(&a_full[kb]), 64 * kb, (int)row0);
                    }
                    const int st = u % ST;
                    if (!mbar_wait(&b_empty[st], ((u / ST) & 1) ^ 1, abort_flag)) *abort_flag = 1;
                    if (*abort_flag) break;
                    uint8_t *dst = smem + SM::oB + st * SM::kStage;
                    if (rank == 0) mbar_arrive_expect_tx(&b_full[st], 2 * SM::kStage);
                    const int y = g * kLatent + kb * kApSlab;
                    if (NC == 256) {
                        tma_load_2d_pair(dst, w_map, lead(&b_full[st]), 0, y);
                        tma_load_2d_pair(dst + kApBoxB, w_map, lead(&b_full[st]), 64, y);
                    } else {
                        tma_load_2d_pair(dst, w_map, lead(&b_full[st]), 64 * (int)rank, y);
                    }
                }
            }
            // every copy has been used, and the other CTA's commits have arrived here
            for (int i = u > ST ? u - ST : 0; i < u && !*abort_flag; ++i)
                if (!mbar_wait(&b_empty[i % ST], (i / ST) & 1, abort_flag)) *abort_flag = 1;
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = idesc_bf16(2 * kApRows, NC, 0, 1);
            // A K-major, 64-column boxes; B MN-major, atoms of 64 columns
            const uint64_t a_d = smem_desc(smem_u32(smem + SM::oA), kApBoxB, 1024, kSw128);
            const uint32_t b_lo0 = static_cast<uint32_t>(smem_desc(smem_u32(smem + SM::oB), kApBoxB, 1024, kSw128));
            const uint32_t a_lo = static_cast<uint32_t>(a_d), hi = static_cast<uint32_t>(a_d >> 32);
            int u = 0;
            for (int x = 0; x < p.products && !*abort_flag; ++x) {
                const int ab = x & 1;
                if (!mbar_wait(&acc_empty[ab], ((x >> 1) & 1) ^ 1, abort_flag)) *abort_flag = 1;
                for (int kb = 0; kb < kApSlabs; ++kb, ++u) {
                    const int st = u % ST;
                    bool ok = x > 0 || mbar_wait(&a_full[kb], 0, abort_flag);
                    ok = ok && mbar_wait(&b_full[st], (u / ST) & 1, abort_flag);
                    if (!ok) *abort_flag = 1;
                    tc_fence_after();
                    const uint32_t a = a_lo + (kb * kApBoxA >> 4), b = b_lo0 + (st * SM::kStage >> 4);
#pragma unroll
                    for (int ks = 0; ks < kApSlab / 16; ++ks)
                        mma_bf16_pair(tmem + 256 * ab, a + (ks * 32 >> 4), b + (ks * 2048 >> 4), hi, idesc,
                                      (kb > 0 || ks > 0) ? 1u : 0u);
                    mma_commit_pair(&b_empty[st]);
                }
                mma_commit_pair(&acc_full[ab]);
            }
            mma_commit_pair(drain, 1);
            int dummy = 0;
            mbar_wait(drain, 0, reinterpret_cast<volatile int *>(&dummy));
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- epilogue
        // two warps to a TMEM lane quadrant, one for each half of the columns
        const int quad = warp & 3, col0 = (warp - 4) >> 2 ? NC / 2 : 0;
        const int64_t r = row0 + 32 * quad + lane;
        const uint32_t lane_off = static_cast<uint32_t>(32 * quad) << 16;
        const int64_t slot = ap_slot(p, r, r < p.total, false);
        // four lanes trade 16-byte units, so that they write 64 bytes of one row together
        int64_t to[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) to[k] = __shfl_sync(0xffffffffu, slot, (lane & ~3) + k);
        for (int x = 0; x < p.products; ++x) {
            const int ab = x & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[ab], (x >> 1) & 1, abort_flag))) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const int v = first + x;
            __nv_bfloat16 *base = p.kv + (int64_t)(v * NC / kKv) * p.num_slots * kKv + v * NC % kKv + (lane & 3) * 8;
#pragma unroll 2
            for (int cc = col0; cc < col0 + NC / 2; cc += 32) {
                uint32_t o[32], w[16];
                tmem_ld32(tmem + 256 * ab + lane_off + cc, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    __nv_bfloat162 t = __floats2bfloat162_rn(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                    w[i] = *reinterpret_cast<uint32_t *>(&t);
                }
                quad_transpose(w, lane);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (to[k] >= 0)
                        *reinterpret_cast<uint4 *>(base + to[k] * kKv + cc) =
                            make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(lead(&acc_empty[ab]));
        }
    } else {
        ap_copy(p, row0, warp - 2, smem + SM::oCopy + (warp - 2) * kApCopyBytes, &copy_bar[warp - 2], abort_flag);
    }
    // Leave together: as in prefill.cu, after the first barrier neither CTA sends anything new
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) {
        report_error(p.ws, GQLA_ERR_TIMEOUT, (int)blockIdx.x);
        st_cluster_b32(map_peer(smem_u32(const_cast<int *>(abort_flag)), rank ^ 1), 1);
    }
    cluster_sync();
    if (*abort_flag) {  // the same in both CTAs
        const long long t0 = clock64();
        while (clock64() - t0 < 200000) {}
        cluster_sync();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

template <int NC>
cudaError_t launch_append_nc(const CUtensorMap &rm, const CUtensorMap &wuk, const CUtensorMap &wuv, const ApParams &p,
                             dim3 grid, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = once_per_device(ready, [] {
        return cudaFuncSetAttribute(append_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, ApSmem<NC>::kAlloc);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(append_kernel<NC>, grid, dim3(kApThreads), ApSmem<NC>::kAlloc, stream, rm, wuk, wuv, p);
}

}  // namespace

cudaError_t launch_append(const void *rows, int64_t total, const int32_t *q_starts, const void *w_uk,
                          const void *w_uv, int num_groups, void *latent, void *kv, void *k_rope, int64_t num_slots,
                          const gqla_kv_index *idx, void *ws, cudaStream_t stream) {
    ApParams p;
    p.rows = static_cast<const uint4 *>(rows);
    p.q_starts = q_starts;
    p.seqlens = idx->seqlens;
    p.page_table = idx->page_table;
    p.latent = static_cast<uint4 *>(latent);
    p.kv = static_cast<__nv_bfloat16 *>(kv);
    p.k_rope = static_cast<uint4 *>(k_rope);
    p.ws = ws;
    p.total = total;
    p.num_slots = num_slots;
    p.batch = idx->batch;
    p.max_pages = idx->max_pages_per_seq;
    p.num_pages = idx->num_pages;
    p.products = 0;
    const unsigned tiles = (unsigned)((total + kApRows - 1) / kApRows);
    if (!kv) return launch_dependent(append_latent_kernel, dim3(tiles, 8), dim3(64), 0, stream, p);
    CUtensorMap rm, wuk, wuv;
    {
        const uint64_t dims[2] = {(uint64_t)kRow, (uint64_t)total};
        const uint64_t strides[1] = {(uint64_t)kRow * 2};
        const uint32_t box[2] = {64, (uint32_t)kApRows};
        if (!make_bf16_map(&rm, rows, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    }
    {
        const uint64_t dims[2] = {(uint64_t)kNope, (uint64_t)num_groups * kLatent};
        const uint64_t strides[1] = {(uint64_t)kNope * 2};
        const uint32_t box[2] = {64, (uint32_t)kApSlab};
        if (!make_bf16_map(&wuk, w_uk, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_bf16_map(&wuv, w_uv, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // The products over as many pairs as one wave holds. Few rows: half a group's columns to a
    // pair, so that the weights' 2 MB come in through as many SMs as there are (128 rows: 9.2 us
    // with a group to a pair, 7.5 us so); many: whole groups, N = 256, which reads A from shared
    // memory half as often.
    const int64_t pairs = (tiles + 1) / 2;
    if (pairs * 2 * num_groups <= sms / 2) {
        p.products = 1;
        return launch_append_nc<128>(rm, wuk, wuv, p, dim3((unsigned)(2 * pairs), 2 * num_groups), stream);
    }
    int split = 1;
    while (split * 2 <= num_groups && num_groups % (split * 2) == 0 && pairs * split * 2 <= sms / 2) split *= 2;
    p.products = num_groups / split;
    return launch_append_nc<256>(rm, wuk, wuv, p, dim3((unsigned)(2 * pairs), split), stream);
}

}  // namespace gqla
