// Grouped and block-scaled products, many rows an expert: pairs of CTAs on tiles of
// 256 tokens x 256 channels (tcgen05 cta_group::2, M = 256), the tokens on the
// accumulator's lanes.
//
// A tile's channels are two halves of 128, each with two accumulators and four
// summing warps of its own in either CTA.  With block scales a block of 128 in k is
// a product of its own for each half; a summing warp's thread is one token and half
// a tile's channels, so its factor sx sw is one number a block, and 128 sums stay in
// its registers.  In bf16 the accumulators are summed over all of k and alternate
// between tiles.
#include <limits.h>

#include <algorithm>

#include "grouped.cuh"

namespace gdn {

using namespace tc;

GDN_DECLARE_STATUS_WORD(g_status_grouped_wide)
GDN_STATUS_READER(read_status_grouped_wide, g_status_grouped_wide)

cudaError_t set_grouped_wide_limit(uint64_t limit_ns, cudaStream_t s) {
    return cudaMemcpyToSymbolAsync(tc::g_wait_limit_ns, &limit_ns, sizeof(limit_ns), 0, cudaMemcpyHostToDevice, s);
}

namespace {

constexpr int kGwStages = 6, kGwEpiWarps = 8, kGwThreads = 128 + 32 * kGwEpiWarps;
constexpr int kGwRows = 256, kGwChannels = 256;
// Registers of a thread: 168 at launch; the first warpgroup gives up what the summing
// ones take (72 x 128 + 216 x 256 = 168 x 384).
constexpr int kGwRegsFew = 72, kGwRegsMany = 216;
constexpr uint32_t kGwX = 128 * 128, kGwHalf = 64 * 128, kGwStage = kGwX + 2 * kGwHalf;
constexpr uint32_t kGwRowBytes = 80;     // a staging row: 64 bytes of y, and 16 that keep 8 rows off each other's banks
constexpr uint32_t kGwStaging = 32 * kGwRowBytes;
constexpr uint32_t kGwSmem = kGwStages * kGwStage + kGwEpiWarps * kGwStaging;

// Loads into this CTA's shared memory, their bytes counted on a barrier of either CTA.
__device__ __forceinline__ void pair_load_2d(void *dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void pair_load_3d(void *dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y,
                                             int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void pair_gather4(void *dst, const CUtensorMap *map, uint32_t bar, int32_t x, const int4 &r) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
        : "memory");
}
// Arrives on the barrier at this offset in both CTAs (mask 3) or the leader (1) once
// the products issued so far by this thread are done.
__device__ __forceinline__ void pair_commit(uint64_t *bar, uint16_t mask = 3) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(mask)
        : "memory");
}
template <bool kE4m3>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (kE4m3)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// A warp's 32 rows x 128 channels out: 64 bytes of each row at a time through its
// staging rows, so that neighbouring lanes write neighbouring bytes.
template <typename O>
__device__ __forceinline__ void wide_store(const F2 (&acc)[64], uint8_t *staging, const GroupedCall &c, int row0, int r1,
                                           int n0, bool there, int lane) {
    constexpr int COLS = 64 / sizeof(O);
    const int rows = r1 - row0;                        // of the warp's 32, those that there are (or more)
    O *y = reinterpret_cast<O *>(c.y) + (int64_t)row0 * c.ys + n0;
#pragma unroll
    for (int ch = 0; ch < 128 / COLS; ++ch) {
        const int left = c.n_out - n0 - ch * COLS;     // channels
        if (left <= 0 || rows <= 0) break;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 *p = acc + (ch * COLS + i * (COLS / 4)) / 2;
            uint4 v;
            if constexpr (sizeof(O) == 2) {
                const float2 a = f2_get(p[0]), b = f2_get(p[1]), d = f2_get(p[2]), e = f2_get(p[3]);
                v = make_uint4(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y), pack_bf16(d.x, d.y), pack_bf16(e.x, e.y));
            } else {
                const float2 a = f2_get(p[0]), b = f2_get(p[1]);
                v = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
            }
            if (!there) v = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(staging + lane * kGwRowBytes + i * 16) = v;
        }
        __syncwarp();
        if (c.vec16) {
            const int piece = lane & 3;
            if (piece * (16 / (int)sizeof(O)) < left) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 8 + (lane >> 2);
                    const uint4 v = *reinterpret_cast<const uint4 *>(staging + r * kGwRowBytes + piece * 16);
                    if (r < rows) *reinterpret_cast<uint4 *>(y + r * c.ys + ch * COLS + piece * (16 / sizeof(O))) = v;
                }
            }
        } else {
            const int col = lane % COLS;
            if (col < left) {
#pragma unroll 8
                for (int r = lane / COLS; r < 32; r += 32 / COLS) {
                    const O v = *reinterpret_cast<const O *>(staging + r * kGwRowBytes + col * sizeof(O));
                    if (r < rows) y[r * c.ys + ch * COLS + col] = v;
                }
            }
        }
    }
}

template <bool kBlock, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGwThreads, 1)
grouped_wide_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                    const __grid_constant__ GroupedCall c, int keep) {
    constexpr int S = kGwStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ GroupTable table;
    __shared__ uint64_t full[S], empty[S], acc_full[2][2], acc_empty[2][2], drained;   // [half][accumulator]
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = (int)cta_rank();
    constexpr int kElems = kBlock ? 128 : 64;
    const int nk = (c.n_in + kElems - 1) / kElems, nn = (c.n_out + kGwChannels - 1) / kGwChannels;
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    volatile int *abort = &abort_flag;

    if (tid == 0) {
        prefetch_tensormap(&mx);
        prefetch_tensormap(&mw);
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&acc_full[i >> 1][i & 1], 1);
            mbar_init(&acc_empty[i >> 1][i & 1], kGwEpiWarps);     // four warps of either CTA
        }
        mbar_init(&drained, 1);
        abort_flag = (smem_u32(smem) & 1023u) != 0;
        fence_mbar_init();
    }
    griddep_wait();            // nothing is read, and no tensor memory asked for, before the kernel in front has ended
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    bool bad;
    const int tiles = build_group_table(table, c, kGwRows, &bad) * nn;     // has barriers
    cluster_arrive_relaxed();  // both CTAs' barriers and tensor memory are ready
    cluster_wait();
    tc_fence_after();
    if (bad && tid == 0 && blockIdx.x == 0) flag_status(GDN_DEVSTAT_BAD_SEQLEN);

    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGwRegsFew));
    if (warp == 0) {
        // This CTA's 128 rows of x and half of each half's weight rows, counted on the leader's barrier.
        const bool one = elect_lane();
        const uint32_t lead = peer_smem(smem_u32(full), 0);
        int s = 0, i = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            const GroupTile a = find_group_tile(table, c.n_experts, t, nn, kGwRows);
            const int r0 = a.r0 + rank * 128, n0 = a.n * kGwChannels;
            const bool both = n0 + 128 < c.n_out;
            int4 rows;
            if (c.rows) {
                const int r = r0 + lane * 4;
                rows = make_int4(group_x_row(c, r, a.r1), group_x_row(c, r + 1, a.r1), group_x_row(c, r + 2, a.r1),
                                 group_x_row(c, r + 3, a.r1));
            }
            const uint32_t bytes = 2 * (kGwX + kGwHalf + (both ? kGwHalf : 0));
#pragma unroll 1
            for (int k = 0; k < nk; ++k, ++i) {
                if (i >= S && !mbar_wait_all(&empty[s], phase, abort)) {
                    ok = false;
                    break;
                }
                uint8_t *st = smem + s * kGwStage;
                const uint32_t bar = lead + s * 8;
                if (i < keep) {
                    if (one) {
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                        if (!c.rows) pair_load_2d(st, &mx, bar, k * kElems, r0);
                        pair_load_3d(st + kGwX, &mw, bar, k * kElems, n0 + rank * 64, a.e);
                        if (both) pair_load_3d(st + kGwX + kGwHalf, &mw, bar, k * kElems, n0 + 128 + rank * 64, a.e);
                    }
                    __syncwarp();
                    if (c.rows) pair_gather4(st + lane * 512, &mx, bar, k * kElems, rows);
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        griddep_launch();
        // the last stages' releases have come
        for (int j = i > S ? i - S : 0; ok && j < i; ++j) ok = mbar_wait_all(&empty[j % S], (j / S) & 1, abort);
        if (one && (!ok || *abort)) {
            // Given up: the copies in flight land before the CTA ends.  The leader waits on
            // the barriers that count them; the peer, which has none, longer than a copy takes.
            if (rank == 0) {
                for (int j = i > S ? i - S : 0; j < min(i, keep); ++j) mbar_drain(&full[j % S], (j / S) & 1);
            } else {
                let_copies_land();
            }
        }
    } else if (warp == 1 && rank == 0) {
        constexpr uint32_t idesc = kBlock ? idesc_e4m3(256, 128) : idesc_bf16(256, 128);
        const uint64_t desc = sdesc_sw128(0, 0, 1024);
        const uint32_t base = smem_u32(smem) >> 4, sums = tmem_base;
        int s = 0, u[2] = {0, 0};          // accumulators of a half used so far
        uint32_t phase = 0;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            const GroupTile a = find_group_tile(table, c.n_experts, t, nn, kGwRows);
            const bool both = a.n * kGwChannels + 128 < c.n_out;
#pragma unroll 1
            for (int k = 0; k < nk && ok; ++k) {
                if (!mbar_wait_all(&full[s], phase, abort)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1 && !both) continue;
                    const int b = u[h] & 1;
                    if ((kBlock || k == 0) && u[h] >= 2 &&
                        !mbar_wait_all(&acc_empty[h][b], ((u[h] >> 1) - 1) & 1, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_lane()) {
                        const uint32_t st = base + s * (kGwStage >> 4), d = sums + (b * 2 + h) * 128;
                        const uint64_t da = desc | st, db = desc | (st + ((kGwX + h * kGwHalf) >> 4));
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            pair_mma<kBlock>(d, da + 2 * q, db + 2 * q, idesc, q > 0 || (!kBlock && k > 0));
                        if (kBlock || k == nk - 1) pair_commit(&acc_full[h][b]);
                    }
                    __syncwarp();
                    if (kBlock || k == nk - 1) ++u[h];
                }
                if (ok && elect_lane()) pair_commit(&empty[s]);
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        // every arrival of the peer's has come, every product is done, before the pair may end
#pragma unroll
        for (int h = 0; h < 2; ++h)
            for (int j = max(0, u[h] - 2); ok && j < u[h]; ++j) ok = mbar_wait_all(&acc_empty[h][j & 1], (j >> 1) & 1, abort);
        if (elect_lane()) {
            pair_commit(&drained, 1);
            mbar_drain(&drained, 0);
        }
        __syncwarp();
    } else if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGwRegsMany));
        // Accumulator lane 32 q + l is token row 32 q + l of this CTA's 128.
        const int q = warp & 3, h = (warp - 4) >> 2;
        uint8_t *staging = smem + S * kGwStage + (warp - 4) * kGwStaging;
        int u = 0;
        bool ok = true, wrong = false;
        for (int t = pair; t < tiles && ok; t += pairs) {
            const GroupTile a = find_group_tile(table, c.n_experts, t, nn, kGwRows);
            const int n0 = a.n * kGwChannels + h * 128;
            if (n0 >= c.n_out) continue;
            const int row0 = a.r0 + rank * 128 + q * 32;
            const int xr = group_x_row(c, row0 + lane, a.r1);
            if (c.rows && row0 + lane < a.r1) wrong |= c.rows[row0 + lane] >= c.n_x;
            const bool there = xr < c.n_x;
            const float *sx = kBlock ? c.sx + (int64_t)(there ? xr : 0) * c.kb : nullptr;
            const float *sw = kBlock ? c.sw + ((int64_t)a.e * c.nb + n0 / 128) * c.kb : nullptr;
            F2 acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = f2(0.f, 0.f);
            // factors two blocks ahead
            float f0 = kBlock ? sx[0] * sw[0] : 1.f, a1 = 0.f, b1 = 0.f;
            if (kBlock && nk > 1) {
                a1 = sx[1];
                b1 = sw[1];
            }
#pragma unroll 1
            for (int k = 0; k < (kBlock ? nk : 1); ++k, ++u) {
                const F2 f = f2(f0, f0);
                float a2 = 0.f, b2 = 0.f;
                if (kBlock && k + 2 < nk) {
                    a2 = sx[k + 2];
                    b2 = sw[k + 2];
                }
                const int b = u & 1;
                if (!mbar_wait_all(&acc_full[h][b], (u >> 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t from = tmem_addr(tmem_base, q * 32, (b * 2 + h) * 128);
                uint32_t r[2][32];
                tmem_ask32(from, r[0]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    tmem_wait32(r[j & 1]);
                    if (j < 3) {
                        tmem_ask32(from + (j + 1) * 32, r[(j + 1) & 1]);
                    } else {                               // all of it has been read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(peer_smem(smem_u32(&acc_empty[h][b]), 0));
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const F2 v = f2_bits(r[j & 1][2 * i], r[j & 1][2 * i + 1]);
                        acc[j * 16 + i] = kBlock ? f2_fma(v, f, acc[j * 16 + i]) : v;
                    }
                }
                f0 = a1 * b1;
                a1 = a2;
                b1 = b2;
            }
            if (!ok) break;
            wide_store<O>(acc, staging, c, row0, a.r1, n0, there, lane);
        }
        if (wrong) flag_status(GDN_DEVSTAT_BAD_INDEX);
        tc_fence_before();
    }
    __syncthreads();
    // Neither CTA ends while the other may reach its memory: every arrival from the other
    // one has been waited for above, so nothing is handed over, unless the pair has given up.
    if (*abort) cluster_arrive();
    else cluster_arrive_relaxed();
    cluster_wait();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
    if (tid == 0 && abort_flag) {
        flag_status(GDN_DEVSTAT_TIMEOUT);
        let_copies_land();     // arrivals that were not waited for
    }
}

template <bool kBlock, typename O> gdn_status launch(const GroupedCall &c, int drop, cudaStream_t s) {
    CUtensorMap mx, mw;
    if (!encode_tmap_rows(&mx, c, 128) || !encode_tmap_experts(&mw, c, 64)) return GDN_ERR_CUDA;
    auto kernel = grouped_wide_kernel<kBlock, O>;
    static SmemAllowed allowed;
    cudaError_t e = allowed.ask(kernel, kGwSmem);
    const int64_t nn = (c.n_out + kGwChannels - 1) / kGwChannels;
    const int64_t tiles = (((int64_t)c.n_rows + kGwRows - 1) / kGwRows + (c.offsets ? std::min(c.n_experts, c.n_rows) : 0)) * nn;
    if (tiles >= (1ll << 31)) return GDN_ERR_UNSUPPORTED;
    if (e == cudaSuccess)
        e = launch_after(kernel, dim3((unsigned)std::min<int64_t>(2 * tiles, sm_count() / 2 * 2)), dim3(kGwThreads), kGwSmem,
                         s, mx, mw, c, drop == kDropNone ? INT_MAX : drop & kDropAll ? 0 : (c.n_in + (kBlock ? 127 : 63)) / (kBlock ? 128 : 64));
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

}  // namespace

gdn_status launch_grouped_wide(const GroupedCall &c, int drop, cudaStream_t s) {
    if (c.e4m3) return c.out_f32 ? launch<true, float>(c, drop, s) : launch<true, __nv_bfloat16>(c, drop, s);
    return c.out_f32 ? launch<false, float>(c, drop, s) : launch<false, __nv_bfloat16>(c, drop, s);
}

}  // namespace gdn
