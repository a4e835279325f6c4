// append.cu -- the rows of new tokens into the pages of the caches: the latent row itself,
// and for the GQA path its per-group projections K_nope = c W_UK_g, V = c W_UV_g and the
// shared RoPE key (GQLA, paperlayer.ai summary, sec. 3 "Two equivalent decoding paths": what
// the one-shot expansion does to a whole cache, done to the tokens of one step or prompt).
//
//   D[128 rows x NC] = A[128 x 512] * B[512 x NC],  NC = 256: B = [W_UK_g | W_UV_g], or
//   NC = 128: one of the two
//
// A CTA takes 128 rows (A, K-major, 128 KB, stays in shared memory) and a share of the
// groups; B streams through a ring of 32-row slabs (MN-major, the weights as stored); two
// TMEM accumulators let the epilogue of one product run during the next. The cache slot of
// a row follows from q_starts, the lengths and the page table; each epilogue thread looks
// its own row's up while the operands are on their way. One more CTA per 128 rows copies the
// latent rows and the RoPE keys.
#include <cuda.h>

#include "common.cuh"
#include "ragged.cuh"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace gqla {

namespace {

using namespace sm100;

constexpr int kApRows = 128;               // rows per tile (MMA M)
constexpr int kApThreads = 192;
constexpr int kApBoxA = kApRows * 128;     // [128 rows][64 latent columns]
constexpr int kApA = 8 * kApBoxA;
constexpr int kApSlab = 32;                // K rows of B per ring stage
constexpr int kApBoxB = kApSlab * 128;     // [32 K rows][64 columns]
constexpr int kApSlabs = kLatent / kApSlab;

template <int NC>
struct ApSmem {
    static constexpr int kStage = NC / 64 * kApBoxB;
    static constexpr int kStages = 4 * 256 / NC;
    static constexpr int oA = 0;
    static constexpr int oB = oA + kApA;
    static constexpr int oBar = oB + kStages * kStage;
    // a_full[8], b_full/b_empty[kStages], acc_full/acc_empty[2], drain
    static constexpr int kNumBars = 8 + 2 * kStages + 4 + 1;
    static constexpr int oMisc = oBar + kNumBars * 8;
    static constexpr int kAlloc = oMisc + 16 + 1024;
};
static_assert(ApSmem<256>::kAlloc <= 227 * 1024 && ApSmem<128>::kAlloc <= 227 * 1024, "shared memory");

struct ApParams {
    const uint4 *rows;            // [total][576] bf16
    const int32_t *q_starts, *seqlens, *page_table;
    uint4 *latent;                // [num_slots][576] bf16, or null
    __nv_bfloat16 *kv;            // [g][num_slots][256], or null
    uint4 *k_rope;                // [num_slots][64] bf16, or null
    void *ws;
    int64_t total, num_slots;
    int batch, max_pages, num_pages;
    int products;                 // products (of NC columns) of one CTA
};

// Cache slot of row r, or -1 if it belongs to no (valid) sequence or its page is outside the
// pool (reported when `report`): the last b with q_starts[b] <= r, by bisection.
__device__ int64_t ap_slot(const ApParams &p, int64_t r, bool report) {
    int lo = 0, hi = p.batch;  // q_starts[lo] <= r < q_starts[hi], where they ascend
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.q_starts[mid] <= r) lo = mid;
        else hi = mid;
    }
    const RaggedSeq s = ragged_seq(p.q_starts, p.seqlens, lo, p.total, p.max_pages);
    if (r < s.q0 || r >= s.q0 + s.n) return -1;
    const int t = s.L - s.n + (int)(r - s.q0);
    const int page = p.page_table[(int64_t)lo * p.max_pages + t / kPage];
    if (page < 0 || page >= p.num_pages) {
        if (report) report_error(p.ws, GQLA_ERR_DEVICE, lo);
        return -1;
    }
    return (int64_t)page * kPage + t % kPage;
}

// The copying CTA of a tile: its rows' latent rows and RoPE keys, 16 bytes a thread.
__device__ void ap_copy(const ApParams &p, int64_t row0) {
    __shared__ int64_t slot[kApRows];
    const int tid = threadIdx.x;
    if (blockIdx.x == 0)
        for (int b = tid; b < p.batch; b += kApThreads)
            if (ragged_seq(p.q_starts, p.seqlens, b, p.total, p.max_pages).bad) report_error(p.ws, GQLA_ERR_DEVICE, b);
    if (tid < kApRows) slot[tid] = row0 + tid < p.total ? ap_slot(p, row0 + tid, true) : -1;
    __syncthreads();
    constexpr int kChunks = kRow / 8, kFirstRope = kLatent / 8;  // 16-byte pieces of a row
    const int lead = p.latent ? 0 : kFirstRope;                  // without a latent cache: the RoPE keys only
    const int per = kChunks - lead;
#pragma unroll 4
    for (int i = tid; i < kApRows * per; i += kApThreads) {
        const int r = i / per, ch = lead + i % per;
        const int64_t s = slot[r];
        if (s < 0) continue;
        const uint4 v = p.rows[(row0 + r) * kChunks + ch];
        if (p.latent) p.latent[s * kChunks + ch] = v;
        if (p.k_rope && ch >= kFirstRope) p.k_rope[s * (kRope / 8) + ch - kFirstRope] = v;
    }
}

template <int NC>
__global__ void __launch_bounds__(kApThreads, 1)
    append_kernel(const __grid_constant__ CUtensorMap row_map, const __grid_constant__ CUtensorMap wuk_map,
                  const __grid_constant__ CUtensorMap wuv_map, const ApParams p) {
    using SM = ApSmem<NC>;
    constexpr int ST = SM::kStages;
    const int64_t row0 = (int64_t)blockIdx.x * kApRows;
    if (blockIdx.y == 0) {  // one CTA of a tile copies
        griddep_wait();
        griddep_launch_dependents();
        ap_copy(p, row0);
        return;
    }
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *a_full = reinterpret_cast<uint64_t *>(smem + SM::oBar);
    uint64_t *b_full = a_full + 8, *b_empty = b_full + ST, *acc_full = b_empty + ST, *acc_empty = acc_full + 2;
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SM::oMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SM::oMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = (blockIdx.y - 1) * p.products;  // this CTA's first product: group first * NC / 256

    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(&a_full[i], 1);
        for (int i = 0; i < ST; ++i) { mbar_init(&b_full[i], 1); mbar_init(&b_empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 4); }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&row_map);
        prefetch_tensormap(&wuk_map);
        prefetch_tensormap(&wuv_map);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch_dependents();

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (elect_one()) {
            int u = 0, boxes = 0;
            for (int x = 0; x < p.products && !*abort_flag; ++x) {
                const int col = (first + x) * NC % kKv, wrow = (first + x) * NC / kKv * kLatent;
                for (int kb = 0; kb < kApSlabs; ++kb, ++u) {
                    // A with the first product's B, two slabs of B to a box of A
                    if (x == 0 && kb % 2 == 0) {
                        mbar_arrive_expect_tx(&a_full[kb / 2], kApBoxA);
                        tma_load_2d(smem + SM::oA + kb / 2 * kApBoxA, &row_map, &a_full[kb / 2], 32 * kb, (int)row0);
                        ++boxes;
                    }
                    const int st = u % ST;
                    if (!mbar_wait(&b_empty[st], ((u / ST) & 1) ^ 1, abort_flag)) *abort_flag = 1;
                    if (*abort_flag) break;
                    uint8_t *dst = smem + SM::oB + st * SM::kStage;
                    mbar_arrive_expect_tx(&b_full[st], SM::kStage);
                    const int y = wrow + kb * kApSlab;
#pragma unroll
                    for (int h = 0; h < NC / 64; ++h) {
                        const int cc = col + 64 * h;
                        tma_load_2d(dst + h * kApBoxB, cc < kNope ? &wuk_map : &wuv_map, &b_full[st], cc % kNope, y);
                    }
                }
            }
            // never leave with copies in flight
            int dummy = 0;
            volatile int *no_abort = reinterpret_cast<volatile int *>(&dummy);
            for (int i = u > ST ? u - ST : 0; i < u; ++i) mbar_wait(&b_full[i % ST], (i / ST) & 1, no_abort);
            for (int i = 0; i < boxes; ++i) mbar_wait(&a_full[i], 0, no_abort);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_bf16(kApRows, NC, 0, 1);
            const uint64_t a_d0 = smem_desc(smem_u32(smem + SM::oA), 16, 1024, kSw128);
            const uint64_t b_d0 = smem_desc(smem_u32(smem + SM::oB), kApBoxB, 1024, kSw128);
            int u = 0;
            for (int x = 0; x < p.products && !*abort_flag; ++x) {
                const int ab = x & 1;
                if (!mbar_wait(&acc_empty[ab], ((x >> 1) & 1) ^ 1, abort_flag)) *abort_flag = 1;
                for (int kb = 0; kb < kApSlabs; ++kb, ++u) {
                    const int st = u % ST;
                    if (x == 0 && !mbar_wait(&a_full[kb / 2], 0, abort_flag)) *abort_flag = 1;
                    if (!mbar_wait(&b_full[st], (u / ST) & 1, abort_flag)) *abort_flag = 1;
                    tc_fence_after();
                    if (!*abort_flag) {
#pragma unroll
                        for (int ks = 0; ks < kApSlab / 16; ++ks) {
                            const int k = kb * kApSlab + ks * 16;
                            mma_bf16(tmem + 256 * ab, desc_advance(a_d0, (k >> 6) * kApBoxA + ((k & 63) >> 3) * 16),
                                     desc_advance(b_d0, st * SM::kStage + ks * 16 * 128), idesc,
                                     (kb > 0 || ks > 0) ? 1u : 0u);
                        }
                    }
                    mma_commit(&b_empty[st]);
                }
                mma_commit(&acc_full[ab]);
            }
            mma_commit(drain);
            int dummy = 0;
            mbar_wait(drain, 0, reinterpret_cast<volatile int *>(&dummy));
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        const int quad = warp & 3;
        const int64_t r = row0 + 32 * quad + lane;
        const uint32_t lane_off = static_cast<uint32_t>(32 * quad) << 16;
        const int64_t slot = r < p.total ? ap_slot(p, r, false) : -1;
        for (int x = 0; x < p.products; ++x) {
            const int ab = x & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[ab], (x >> 1) & 1, abort_flag))) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const int col = (first + x) * NC % kKv, g = (first + x) * NC / kKv;
            uint4 *dst = reinterpret_cast<uint4 *>(p.kv + ((int64_t)g * p.num_slots + slot) * kKv + col);
#pragma unroll 1
            for (int cc = 0; cc < NC; cc += 32) {
                uint32_t v[32];
                tmem_ld32(tmem + 256 * ab + lane_off + cc, v);
                tmem_wait_ld();
                if (slot < 0) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint2 lo = pack_bf16x4(__uint_as_float(v[8 * i]), __uint_as_float(v[8 * i + 1]),
                                                 __uint_as_float(v[8 * i + 2]), __uint_as_float(v[8 * i + 3]));
                    const uint2 hi = pack_bf16x4(__uint_as_float(v[8 * i + 4]), __uint_as_float(v[8 * i + 5]),
                                                 __uint_as_float(v[8 * i + 6]), __uint_as_float(v[8 * i + 7]));
                    dst[cc / 8 + i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[ab]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) report_error(p.ws, GQLA_ERR_TIMEOUT, (int)blockIdx.x);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int NC>
cudaError_t launch_append_nc(const CUtensorMap &rm, const CUtensorMap &wuk, const CUtensorMap &wuv, const ApParams &p,
                             dim3 grid, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(append_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         ApSmem<NC>::kAlloc);
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
    CUtensorMap rm = {}, wuk = {}, wuv = {};
    const unsigned tiles = (unsigned)((total + kApRows - 1) / kApRows);
    if (!kv) return launch_append_nc<256>(rm, wuk, wuv, p, dim3(tiles, 1), stream);
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
    // Few tiles: a CTA per 128 output columns, so that the weights' 2 MB are read by as many
    // SMs as there are; otherwise a CTA takes whole groups, as many as leave one wave.
    if ((int64_t)tiles * 2 * num_groups <= sms) {
        p.products = 1;
        return launch_append_nc<128>(rm, wuk, wuv, p, dim3(tiles, 1 + 2 * num_groups), stream);
    }
    int split = 1;
    while (split * 2 <= num_groups && num_groups % (split * 2) == 0 && (int64_t)tiles * split * 2 <= sms) split *= 2;
    p.products = num_groups / split;
    return launch_append_nc<256>(rm, wuk, wuv, p, dim3(tiles, 1 + split), stream);
}

}  // namespace gqla
