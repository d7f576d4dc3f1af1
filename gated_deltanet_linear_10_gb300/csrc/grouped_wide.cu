// Grouped and block-scaled products, many rows an expert: pairs of CTAs on tiles of
// 256 tokens x 256 channels (tcgen05 cta_group::2, M = 256), the tokens on the
// accumulator's lanes.
//
// With block scales every block of 128 in k is a product of its own, which eight
// warps of either CTA take out of tensor memory and add, times its factor, to sums in
// registers.  A thread is one token and 128 channels, so the factor sx sw is one
// number a block and half a tile.  The half tiles of 128 channels have two
// accumulators each: the way from a product's issue over its sums' reading to the
// accumulator's release is longer than two products of a whole tile take, but not
// than four of a half.  In bf16 the accumulators are summed over all of k and
// alternate between tiles.
//
// Where rows are gathered, two warps copy them to shared memory in pieces of 16 bytes:
// a TMA gather of four rows took 84 cycles (20668 x 10 rows 2048 x 1024 e4m3: 2780
// cycles a block of 128, of which 1750 for the rows to come).
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

constexpr int kGwStages = 4, kGwEpiWarps = 8, kGwThreads = 128 + 32 * kGwEpiWarps;
constexpr int kGwRows = 256, kGwChannels = 256;
// Registers of a thread: 168 at launch; the first warpgroup gives up what the summing
// ones take (88 x 128 + 208 x 256 = 168 x 384).
constexpr int kGwRegsFew = 88, kGwRegsMany = 208;
constexpr uint32_t kGwX = 128 * 128, kGwHalf = 64 * 128, kGwStage = kGwX + 2 * kGwHalf;
// Staging of a warp: two tiles of 32 rows x 128 bytes in the 128-byte swizzle.
constexpr uint32_t kGwStaging = 2 * 4096;
constexpr uint32_t kGwSmem = kGwStages * kGwStage + kGwEpiWarps * kGwStaging;
constexpr int kGwLag = 2;                // gathered stages in flight behind the one being asked for

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
// 16 bytes of global into shared memory, those from `bytes` on as zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// A warp's 32 rows x 64 channels of the tile's halves out, through its staging tiles:
// by a TMA store that goes on behind the call; where the expert ends within the rows,
// in pieces of 16 bytes, and where rows are no whole pieces, element by element.  n0:
// the warp's channels of half 0, those of half 1 are 128 on.  (Rows of bulk copies, one
// a lane, took 5,500 cycles a tile and held up the loads behind them.)
template <typename O>
__device__ __forceinline__ void wide_store(const F2 (&acc)[2][32], uint8_t *staging, const CUtensorMap *my,
                                           const GroupedCall &c, int row0, int r1, int n0, bool there, int lane) {
    constexpr int COLS = 128 / sizeof(O), TILES = 64 / COLS;          // channels of a tile, tiles of a half
    const int rows = r1 - row0;                        // of the warp's 32, those that there are (or more)
    O *y = reinterpret_cast<O *>(c.y) + (int64_t)row0 * c.ys;
    uint8_t *mine = staging + lane * 128;
#pragma unroll
    for (int i = 0; i < 2 * TILES; ++i) {
        const int h = i / TILES, n = n0 + h * 128 + i % TILES * COLS, left = c.n_out - n;
        if (left <= 0 || rows <= 0) break;
        uint8_t *tile = staging + i % 2 * 4096, *row = mine + i % 2 * 4096;
        if (i % 2 == 0) {                              // the last stores have read the tiles
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const F2 *p = acc[h] + (i % TILES * COLS + j * (16 / (int)sizeof(O))) / 2;
            uint4 v;
            if constexpr (sizeof(O) == 2) {
                const float2 a = f2_get(p[0]), b = f2_get(p[1]), d = f2_get(p[2]), e = f2_get(p[3]);
                v = make_uint4(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y), pack_bf16(d.x, d.y), pack_bf16(e.x, e.y));
            } else {
                const float2 a = f2_get(p[0]), b = f2_get(p[1]);
                v = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
            }
            if (!there) v = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(row + ((j ^ (lane & 7)) << 4)) = v;
        }
        if (c.vec16 && rows >= 32) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(my, tile, n, row0);
                bulk_commit();
            }
            continue;
        }
        __syncwarp();
        if (c.vec16) {
            const int piece = lane & 7;
            if (piece * (16 / (int)sizeof(O)) < left) {
                for (int r = lane >> 3; r < min(32, rows); r += 4)
                    *reinterpret_cast<uint4 *>(y + r * c.ys + n + piece * (16 / sizeof(O))) =
                        *reinterpret_cast<const uint4 *>(tile + r * 128 + ((piece ^ (r & 7)) << 4));
            }
        } else {
#pragma unroll 4
            for (int r = 0; r < min(32, rows); ++r)
#pragma unroll
                for (int col = lane; col < COLS; col += 32) {
                    const uint32_t at = col * (uint32_t)sizeof(O);
                    if (col < left)
                        y[r * c.ys + n + col] = *reinterpret_cast<const O *>(tile + r * 128 + ((at >> 4 ^ (r & 7)) << 4) + (at & 15));
                }
        }
        __syncwarp();
    }
}

// A tile as the loads and the products need it, looked up one tile ahead.
struct WideTile {
    int e, r0, r1, n0;
    bool both;                                         // channels in both halves
};
__device__ __forceinline__ WideTile wide_tile(const GroupTable &g, const GroupedCall &c, int tile, int tiles, int nn) {
    WideTile w = {};
    if (tile < tiles) {
        const GroupTile t = find_group_tile(g, c.n_experts, tile, nn, kGwRows);
        w = {t.e, t.r0, t.r1, t.n * kGwChannels, t.n * kGwChannels + 128 < c.n_out};
    }
    return w;
}

template <bool kBlock, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGwThreads, 1)
grouped_wide_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                    const __grid_constant__ CUtensorMap my, const __grid_constant__ GroupedCall c, int keep) {
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
            mbar_init(&full[s], c.rows ? 5 : 1);       // the loads by TMA, two gathering warps of either CTA
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&acc_full[i >> 1][i & 1], 1);
            mbar_init(&acc_empty[i >> 1][i & 1], 2 * kGwEpiWarps);
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
        // Half of the weight rows and this CTA's 128 rows of x, counted on the leader's barrier.
        const bool one = elect_lane();
        const uint32_t lead = peer_smem(smem_u32(full), 0);
        int s = 0, i = 0;
        uint32_t phase = 1;
        bool ok = true;
        WideTile a = wide_tile(table, c, pair, tiles, nn), next = a;
        for (int t = pair; t < tiles && ok; t += pairs, a = next) {
            // the product of a whole tile takes channels 0 .. 127 from the leader, that of a half 0 .. 63
            const bool whole = !kBlock && a.both;
            const int n0 = a.n0 + rank * (whole ? 128 : 64), n1 = n0 + (whole ? 64 : 128);
            const uint32_t bytes = 2 * ((c.rows ? 0 : kGwX) + kGwHalf + (a.both ? kGwHalf : 0));
#pragma unroll 1
            for (int k = 0; k < nk; ++k, ++i) {
                if (i >= S && !mbar_wait_all(&empty[s], phase, abort)) {
                    ok = false;
                    break;
                }
                uint8_t *st = smem + s * kGwStage;
                const uint32_t bar = lead + s * 8;
                if (i < keep && one) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                    if (!c.rows) pair_load_2d(st, &mx, bar, k * kElems, a.r0 + rank * 128);
                    pair_load_3d(st + kGwX, &mw, bar, k * kElems, n0, a.e);
                    if (a.both) pair_load_3d(st + kGwX + kGwHalf, &mw, bar, k * kElems, n1, a.e);
                }
                __syncwarp();
                if (k == 0) next = wide_tile(table, c, t + pairs, tiles, nn);
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
            // the barriers that count them; the peer, which has none, and a leader whose rows
            // are gathered (its barriers count these too), longer than a copy takes.
            if (rank == 0 && !c.rows) {
                for (int j = i > S ? i - S : 0; j < min(i, keep); ++j) mbar_drain(&full[j % S], (j / S) & 1);
            } else {
                let_copies_land();
            }
        }
    } else if (warp == 1 && rank == 0) {
        constexpr uint32_t half = kBlock ? idesc_e4m3(256, 128) : idesc_bf16(256, 128);
        constexpr uint32_t full_tile = idesc_bf16(256, 256);
        const uint64_t desc = sdesc_sw128(0, 0, 1024);
        const uint32_t base = smem_u32(smem) >> 4, sums = tmem_base;
        int s = 0, u[2] = {0, 0};          // accumulators of a half used so far
        uint32_t phase = 0, st = base;
        bool ok = true, both = wide_tile(table, c, pair, tiles, nn).both, next = both;
        for (int t = pair; t < tiles && ok; t += pairs, both = next) {
#pragma unroll 1
            for (int k = 0; k < nk; ++k) {
                if (!mbar_wait_all(&full[s], phase, abort)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int h = 0; h < (kBlock ? 2 : 1); ++h) {
                    if (h == 1 && !both) break;
                    const int b = u[h] & 1;
                    if (kBlock || k == 0) {
                        if (u[h] >= 2 && !mbar_wait_all(&acc_empty[h][b], ((u[h] >> 1) - 1) & 1, abort)) ok = false;
                        if (!ok) break;
                    }
                    tc_fence_after();
                    const bool last = kBlock || k == nk - 1;
                    if (elect_lane()) {
                        const uint32_t d = sums + (b * 2 + h) * 128;
                        const uint64_t da = desc | st, db = desc | (st + ((kGwX + h * kGwHalf) >> 4));
                        const uint32_t idesc = kBlock || !both ? half : full_tile;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            pair_mma<kBlock>(d, da + 2 * q, db + 2 * q, idesc, q > 0 || (!kBlock && k > 0));
                        if (last) pair_commit(&acc_full[h][b]);
                        if (!kBlock || h == 1 || !both) pair_commit(&empty[s]);
                    }
                    __syncwarp();
                    if (last) ++u[h];
                }
                if (!ok) break;
                st += kGwStage >> 4;
                if (++s == S) {
                    s = 0;
                    st = base;
                    phase ^= 1;
                }
                if (k == 0) next = wide_tile(table, c, t + pairs, tiles, nn).both;   // behind the products
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
    } else if (warp == 2 || warp == 3) {
        // Gathered rows: a lane copies 16 bytes of every eighth row, a warp four whole rows
        // at a time, and hands over a stage when its copies have come.
        if (c.rows) {
            const uint32_t lead = peer_smem(smem_u32(full), 0);
            const int sub = (warp - 2) * 4 + (lane >> 3);                  // of eight rows
            const uint32_t to = smem_u32(smem) + sub * 128 + (((lane & 7) ^ sub) << 4);
            const int64_t stride = c.xs * (kBlock ? 1 : 2);
            const int bytes = c.n_in * (kBlock ? 1 : 2) - (lane & 7) * 16;  // of the row from this lane's first on
            int s = 0, i = 0;
            uint32_t phase = 1;
            bool ok = true;
            int row[16], next_row[16];
            auto look = [&](int tile, int (&r)[16]) {
                const WideTile a = wide_tile(table, c, tile, tiles, nn);
                const int r0 = a.r0 + rank * 128 + sub;
#pragma unroll
                for (int j = 0; j < 16; ++j) r[j] = tile < tiles ? group_x_row(c, r0 + j * 8, a.r1) : c.n_x;
            };
            look(pair, row);
            auto hand_over = [&](int j) {                                   // stage of block j
                // The copies lie in this CTA's own shared memory and, by the fence, before the tensor
                // core's reads there, which the leader's product starts after the arrival: a relaxed
                // one (with release at the cluster it waited for the copies still in flight, 2,000
                // cycles a block).
                fence_async_smem();
                __syncwarp();
                if (lane == 0 && j < keep) mbar_arrive_cluster(lead + j % S * 8);
            };
            for (int t = pair; t < tiles && ok; t += pairs) {
#pragma unroll 1
                for (int k = 0; k < nk; ++k, ++i) {
                    if (i >= S && !mbar_wait_all(&empty[s], phase, abort)) {
                        ok = false;
                        break;
                    }
                    const int n = min(16, max(0, bytes - k * 128));
                    const uint8_t *src = reinterpret_cast<const uint8_t *>(c.x) + k * 128 + (lane & 7) * 16;
                    if (i < keep) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const bool on = row[j] < c.n_x && n > 0;
                            copy16(to + s * kGwStage + j * 1024, on ? src + row[j] * stride : c.x, on ? n : 0);
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (i >= kGwLag) {
                        asm volatile("cp.async.wait_group %0;" ::"n"(kGwLag) : "memory");
                        hand_over(i - kGwLag);
                    }
                    if (k == 0) look(t + pairs, next_row);
                    if (++s == S) {
                        s = 0;
                        phase ^= 1;
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) row[j] = next_row[j];
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            for (int j = max(0, i - kGwLag); ok && j < i; ++j) hand_over(j);
        }
    } else if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGwRegsMany));
        // Accumulator lane 32 q + l is token row 32 q + l of this CTA's 128; the two warps
        // of a quadrant take 64 channels each of either half.
        const int q = warp & 3, part = (warp - 4) >> 2;
        uint8_t *staging = smem + S * kGwStage + (warp - 4) * kGwStaging;
        int u[2] = {0, 0};
        bool ok = true, wrong = false;
        WideTile a = wide_tile(table, c, pair, tiles, nn), next = a;
        auto x_row = [&](const WideTile &w) {
            const int r = w.r0 + rank * 128 + q * 32 + lane;
            if (c.rows && r < w.r1) wrong |= c.rows[r] >= c.n_x;
            return group_x_row(c, r, w.r1);
        };
        int xr = x_row(a), next_xr = xr;
        for (int t = pair; t < tiles && ok; t += pairs, a = next, xr = next_xr) {
            const bool there = xr < c.n_x;
            const float *sx = kBlock ? c.sx + (int64_t)(there ? xr : 0) * c.kb : nullptr;
            const float *sw = kBlock ? c.sw + ((int64_t)a.e * c.nb + a.n0 / 128) * c.kb : nullptr;
            const int second = a.both ? c.kb : 0;           // the other half's scales
            F2 acc[2][32];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i / 32][i % 32] = f2(0.f, 0.f);
            // factors two blocks ahead
            float f0 = 1.f, f1 = 1.f, xa = 0.f, wa = 0.f, wb = 0.f;
            if (kBlock) {
                f0 = sx[0] * sw[0];
                f1 = sx[0] * sw[second];
                if (nk > 1) {
                    xa = sx[1];
                    wa = sw[1];
                    wb = sw[second + 1];
                }
            }
#pragma unroll 1
            for (int k = 0; k < (kBlock ? nk : 1); ++k) {
                float xn = 0.f, wn = 0.f, wm = 0.f;
                if (kBlock && k + 2 < nk) {
                    xn = sx[k + 2];
                    wn = sw[k + 2];
                    wm = sw[second + k + 2];
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1 && !a.both) break;
                    constexpr bool kWhole = !kBlock;           // one product for both halves
                    int &uses = u[kWhole ? 0 : h];
                    const int b = uses & 1;
                    if ((!kWhole || h == 0) && !mbar_wait_all(&acc_full[kWhole ? 0 : h][b], (uses >> 1) & 1, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t from = tmem_addr(tmem_base, q * 32, (b * 2 + h) * 128 + part * 64);
                    const float f = h ? f1 : f0;
                    uint32_t r[2][32];
                    tmem_ask32(from, r[0]);
                    tmem_ask32(from + 32, r[1]);
                    tmem_wait32(r[0]);
                    tmem_wait32(r[1]);
                    tc_fence_before();                         // all of it has been read
                    __syncwarp();
                    if (!kWhole || h == 1 || !a.both) {
                        if (lane == 0) mbar_arrive_cluster(peer_smem(smem_u32(&acc_empty[kWhole ? 0 : h][b]), 0));
                        ++uses;
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const F2 v = f2_bits(r[i / 16][i % 16 * 2], r[i / 16][i % 16 * 2 + 1]);
                        acc[h][i] = kBlock ? f2_fma(v, f2(f, f), acc[h][i]) : v;
                    }
                }
                if (!ok) break;
                if (k == 0) {
                    next = wide_tile(table, c, t + pairs, tiles, nn);
                    next_xr = x_row(next);
                }
                f0 = xa * wa;
                f1 = xa * wb;
                xa = xn;
                wa = wn;
                wb = wm;
            }
            if (!ok) break;
            wide_store<O>(acc, staging, &my, c, a.r0 + rank * 128 + q * 32, a.r1, a.n0 + part * 64, there, lane);
        }
        if (lane == 0) bulk_wait_read_all();       // the staging tiles stay until they are read
        __syncwarp();
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
    CUtensorMap mx, mw, my = {};
    if (!encode_tmap_rows(&mx, c, 128) || !encode_tmap_experts(&mw, c, 64)) return GDN_ERR_CUDA;
    if (c.vec16 && !encode_tmap_2d(&my, sizeof(O) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                   c.y, c.n_out, c.n_rows, c.n_rows == 1 ? (uint64_t)c.n_out * sizeof(O) : c.ys * sizeof(O),
                                   128 / sizeof(O), 32, true))
        return GDN_ERR_CUDA;
    auto kernel = grouped_wide_kernel<kBlock, O>;
    static SmemAllowed allowed;
    cudaError_t e = allowed.ask(kernel, kGwSmem);
    const int64_t nn = (c.n_out + kGwChannels - 1) / kGwChannels;
    const int64_t tiles = (((int64_t)c.n_rows + kGwRows - 1) / kGwRows + (c.offsets ? std::min(c.n_experts, c.n_rows) : 0)) * nn;
    if (tiles >= (1ll << 31)) return GDN_ERR_UNSUPPORTED;
    if (e == cudaSuccess)
        e = launch_after(kernel, dim3((unsigned)std::min<int64_t>(2 * tiles, sm_count() / 2 * 2)), dim3(kGwThreads), kGwSmem,
                         s, mx, mw, my, c, drop == kDropNone ? INT_MAX : drop & kDropAll ? 0 : (c.n_in + (kBlock ? 127 : 63)) / (kBlock ? 128 : 64));
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
