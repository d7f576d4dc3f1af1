// Grouped and block-scaled products, many rows an expert: pairs of CTAs on tiles of
// 256 tokens x 256 channels (tcgen05 cta_group::2, M = 256), the tokens on the
// accumulator's lanes.
//
// With block scales every block of 128 in k is a product of its own, which four warps
// of either CTA take out of tensor memory and add, times its factor, to sums in
// registers.  A thread is one token and half a tile's channels, so the factor sx sw is
// one number a block.  The two halves of 128 channels are pipelines of their own: a
// warp that issues the products, two accumulators, and the warps that sum them.  What
// bounds a block is the instructions around it, each warp's in turn (a wait that finds
// its barrier done takes some 165 cycles, four products and their commits 200): one
// issuing warp for both halves took 1,100 cycles a block, the products 512.  In bf16
// the accumulators are summed over all of k and alternate between tiles.
//
// The factors come through shared memory, from a warp that reads them eight blocks at a
// time: read by the summing warps themselves, a word of 32 rows a block, they took a
// fifth of the time (gathered rows: 897 us, with one row's factors for all 697).  What
// can wait polls with one lane and sleeps: more polling warps slow the chain down.
//
// Where rows are gathered, three warps copy them to shared memory in pieces of 16 bytes:
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

constexpr int kGwEpiWarps = 8;
// Warps: 0 loads by TMA, 1 and 2 products, 3 looks up tiles and makes the factors, 4 to 11
// sums, 12 to 14 gathered rows, 15 hands them over.
constexpr int kGwThreads = 512, kGwTile = 3, kGwFirstEpi = 4, kGwFirstGather = 12, kGwGather = 3, kGwRelay = 15;
constexpr int kGwChunk = 8;              // blocks whose factors are handed over at a time
constexpr int kGwRows = 256, kGwChannels = 256;
// Registers of a thread: 128 at launch; the summing warpgroups take what the others
// give up: their sum over the four warpgroups stays 512.  (A spill in any of the loops
// costs more than it looks: with 48, 64 and 200 bf16 rows gathered took 353 us instead
// of 268.  With these, 24 to 34 bytes of a thread are still spilled.)
template <bool kBlock> struct GwRegs {
    static constexpr int kFew = kBlock ? 56 : 72, kGather = kBlock ? 88 : 72, kMany = 184;
    static_assert(kFew + kGather + 2 * kMany == 512, "registers that the launch has");
};
constexpr uint32_t kGwX = 128 * 128, kGwHalf = 64 * 128, kGwStage = kGwX + 2 * kGwHalf;
constexpr uint32_t kGwFactors = 2 * kGwChunk * 128 * 4;       // [half][block][row], fp32
// Shared memory: the ring's stages, a warp's staging tiles of 32 rows x 128 bytes of y in
// the 128-byte swizzle, the factors.  In bf16 a stage is used up in half the time, and a
// fifth one gains more than a second staging tile (64 experts of 1300 rows: 261 -> 238
// us; with block scales 301 -> 327).
template <bool kBlock> struct GwSmem {
    static constexpr int kStages = kBlock ? 4 : 5, kHold = kBlock ? 2 : 1;
    static constexpr uint32_t kStaging = kHold * 4096;
    static constexpr uint32_t kBytes = kStages * kGwStage + kGwEpiWarps * kStaging + (kBlock ? 2 * kGwFactors : 0);
};

// Loads into this CTA's shared memory, their bytes counted on a barrier of either CTA.
__device__ __forceinline__ void pair_load_2d(void *dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void pair_load_3d(void *dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y,
                                             int32_t z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
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

// A warp's 32 rows x 128 channels n0 .. out, through its staging tiles:
// by a TMA store that goes on behind the call; where the expert ends within the rows,
// in pieces of 16 bytes, and where rows are no whole pieces, by words or elements.
// (Rows of bulk copies, one a lane, took 5,500 cycles a tile and held up the loads
// behind them.)
template <typename O, int kHold>
__device__ __forceinline__ void wide_store(const F2 (&acc)[64], uint8_t *staging, const CUtensorMap *my,
                                           const GroupedCall &c, int row0, int r1, int n0, bool there, int lane) {
    constexpr int COLS = 128 / sizeof(O);              // channels of a staging tile
    const int rows = r1 - row0;                        // of the warp's 32, those that there are (or more)
    O *y = reinterpret_cast<O *>(c.y) + (int64_t)row0 * c.ys;
    uint8_t *mine = staging + lane * 128;
#pragma unroll
    for (int i = 0; i < 128 / COLS; ++i) {
        const int n = n0 + i * COLS, left = c.n_out - n;
        if (left <= 0 || rows <= 0) break;
        uint8_t *tile = staging + i % kHold * 4096, *row = mine + i % kHold * 4096;
        if (i % kHold == 0) {                          // the last stores have read the tiles
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const F2 *p = acc + (i * COLS + j * (16 / (int)sizeof(O))) / 2;
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
            // words of 4 bytes, or elements where rows are not on them; eight of a lane are read
            // before the first is written
            constexpr int E = 4 / sizeof(O);               // elements of a word
            if (E == 1 || c.vec4) {
#pragma unroll 1
                for (int r = 0; r < min(32, rows); r += 8) {
                    uint32_t v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = *reinterpret_cast<const uint32_t *>(tile + (r + j) * 128 + ((lane >> 2 ^ (j & 7)) << 4) +
                                                                   (lane & 3) * 4);
                    const int col = lane * E;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (r + j >= rows || col >= left) continue;
                        O *p = y + (r + j) * c.ys + n + col;
                        if (E == 1 || col + 1 < left) *reinterpret_cast<uint32_t *>(p) = v[j];
                        else *reinterpret_cast<uint16_t *>(p) = (uint16_t)v[j];
                    }
                }
            } else {
#pragma unroll 1
                for (int r = 0; r < min(32, rows); r += 4) {
                    uint16_t v[8];                         // 32 neighbours of a row at a time
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int row = r + (j >> 1), piece = (j & 1) * 4 + (lane >> 3);
                        v[j] = *reinterpret_cast<const uint16_t *>(tile + row * 128 + ((piece ^ (row & 7)) << 4) +
                                                                   (lane & 7) * 2);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int row = r + (j >> 1), col = (j & 1) * 32 + lane;
                        if (row < rows && col < left) reinterpret_cast<uint16_t *>(y + row * c.ys + n)[col] = v[j];
                    }
                }
            }
        }
        __syncwarp();
    }
}

// What the warps of a CTA know of a tile, by way of shared memory: one warp looks the
// tiles up, a tile ahead (in every warp that took registers which its loop over the
// blocks then missed, and 500 cycles for two divisions).
constexpr int kGwTiles = 4;
struct WideTiles {
    int4 at[kGwTiles];                  // first row, the expert's end, first channel, expert
    uint32_t there[kGwTiles][4];        // which of this CTA's 128 rows there are
    int row[kGwTiles][128];             // and the rows of x that they take
    uint64_t full[kGwTiles], empty[kGwTiles];
};
// The j-th tile of this CTA, for a whole warp, which then lets go of its place.
__device__ __forceinline__ bool take_tile(WideTiles &w, int j, int4 &a, volatile int *abort) {
    const int s = j % kGwTiles;
    if (!mbar_wait_all(&w.full[s], (j / kGwTiles) & 1, abort)) return false;
    a = w.at[s];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&w.empty[s]);
    return true;
}

template <bool kBlock, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGwThreads, 1)
grouped_wide_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                    const __grid_constant__ CUtensorMap my, const __grid_constant__ GroupedCall c, int keep) {
    using M = GwSmem<kBlock>;
    constexpr int S = M::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ GroupTable table;
    __shared__ uint64_t full[S], empty[S], gathered[S], drained[2], sc_full[2], sc_empty[2];
    __shared__ uint64_t acc_full[2][2], acc_empty[2][2];   // [half][accumulator]
    constexpr int H = kBlock ? 2 : 1;      // issuing warps; one product makes both halves in bf16
    __shared__ WideTiles wide;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = (int)cta_rank();
    constexpr int kElems = kBlock ? 128 : 64;
    const int nk = (c.n_in + kElems - 1) / kElems, nn = (c.n_out + kGwChannels - 1) / kGwChannels;
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    float *factors = reinterpret_cast<float *>(smem + S * kGwStage + kGwEpiWarps * M::kStaging);
    volatile int *abort = &abort_flag;

    if (tid == 0) {
        prefetch_tensormap(&mx);
        prefetch_tensormap(&mw);
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], c.rows ? 3 : 1);       // the loads by TMA, either CTA's gathered rows
            mbar_init(&gathered[s], 32 * kGwGather);
            mbar_init(&empty[s], H);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&acc_full[i >> 1][i & 1], 1);
            mbar_init(&acc_empty[i >> 1][i & 1], 2 * kGwEpiWarps / H);
        }
        for (int i = 0; i < kGwTiles; ++i) {
            mbar_init(&wide.full[i], 1);
            // the loads, the products, the gathered rows and the sums
            mbar_init(&wide.empty[i], 1 + (rank == 0 ? H : 0) + (c.rows ? kGwGather : 0) + kGwEpiWarps);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&drained[h], 1);
            mbar_init(&sc_full[h], 1);
            mbar_init(&sc_empty[h], kGwEpiWarps);
        }
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

    if (warp < kGwFirstEpi) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(GwRegs<kBlock>::kFew));
    if (warp >= kGwFirstGather) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(GwRegs<kBlock>::kGather));
    if (warp == 0) {
        // Half of the weight rows and this CTA's 128 rows of x, counted on the leader's barrier.
        const bool one = elect_lane();
        const uint32_t lead = peer_smem(smem_u32(full), 0);
        const uint64_t policy = c.offsets ? l2_first() : l2_normal();
        int s = 0, i = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int t = pair, j = 0; t < tiles && ok; t += pairs, ++j) {
            int4 a;
            if (!take_tile(wide, j, a, abort)) {
                ok = false;
                break;
            }
            const bool both = a.z + 128 < c.n_out;
            // the product of a whole tile takes channels 0 .. 127 from the leader, that of a half 0 .. 63
            const bool whole = !kBlock && both;
            const int n0 = a.z + rank * (whole ? 128 : 64), n1 = n0 + (whole ? 64 : 128), r0 = a.x + rank * 128;
            const uint32_t bytes = 2 * ((c.rows ? 0 : kGwX) + kGwHalf + (both ? kGwHalf : 0));
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
                    if (!c.rows) pair_load_2d(st, &mx, bar, k * kElems, r0);
                    pair_load_3d(st + kGwX, &mw, bar, k * kElems, n0, a.w, policy);
                    if (both) pair_load_3d(st + kGwX + kGwHalf, &mw, bar, k * kElems, n1, a.w, policy);
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
            // the barriers that count them; the peer, which has none, and a leader whose rows
            // are gathered (its barriers count these too), longer than a copy takes.
            if (rank == 0 && !c.rows) {
                for (int j = i > S ? i - S : 0; j < min(i, keep); ++j) mbar_drain(&full[j % S], (j / S) & 1);
            } else {
                let_copies_land();
            }
        }
    } else if (warp <= H && rank == 0) {
        const int h = warp - 1;
        constexpr uint32_t half = kBlock ? idesc_e4m3(256, 128) : idesc_bf16(256, 128);
        constexpr uint32_t full_tile = idesc_bf16(256, 256);
        const uint64_t desc = sdesc_sw128(0, 0, 1024);
        const uint32_t base = smem_u32(smem) >> 4, sums = tmem_base + h * 128, xh = (kGwX + h * kGwHalf) >> 4;
        int s = 0, u = 0;                  // u: accumulators used so far
        uint32_t phase = 0, st = base;
        bool ok = true, ready = false;     // operands and accumulator of the next block are known to be there
        for (int t = pair, j = 0; t < tiles && ok; t += pairs, ++j) {
            int4 a;
            if (!take_tile(wide, j, a, abort)) {
                ok = false;
                break;
            }
            const bool both = a.z + 128 < c.n_out;
            const uint32_t idesc = kBlock || !both ? half : full_tile;
            const bool mine = h == 0 || both;          // else the stages are handed back as they are
#pragma unroll 1
            for (int k = 0; k < nk; ++k) {
                if (!ready) {
                    // the operands first, which have mostly come: less lies behind the accumulator's release
                    ok = mbar_wait_all(&full[s], phase, abort);
                    if (ok && (kBlock || k == 0) && mine && u >= 2)
                        ok = mbar_wait_all(&acc_empty[h][u & 1], ((u >> 1) - 1) & 1, abort);
                    if (!ok) break;
                }
                tc_fence_after();
                const bool last = kBlock || k == nk - 1;
                if (elect_lane()) {
                    if (mine) {
                        if (c.rows) acquire_smem_of_cluster();         // rows that either CTA's threads have written
                        const uint32_t d = sums + (u & 1) * 256;
                        const uint64_t da = desc | st, db = desc | (st + xh);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            pair_mma<kBlock>(d, da + 2 * q, db + 2 * q, idesc, q > 0 || (!kBlock && k > 0));
                        if (last) pair_commit(&acc_full[h][u & 1]);
                    }
                    pair_commit(&empty[s]);
                }
                __syncwarp();
                if (last && mine) ++u;
                st += kGwStage >> 4;
                if (++s == S) {
                    s = 0;
                    st = base;
                    phase ^= 1;
                }
                // (a wait that finds its barrier done takes 150 cycles, two looks ahead of time hardly any)
                ready = mbar_test(&full[s], phase);
                if (last && u >= 2) ready = mbar_test(&acc_empty[h][u & 1], ((u >> 1) - 1) & 1) && ready;
                ready = __all_sync(0xffffffffu, ready);
            }
        }
        // every arrival of the peer's has come, every product is done, before the pair may end
        for (int j = max(0, u - 2); ok && j < u; ++j) ok = mbar_wait_all(&acc_empty[h][j & 1], (j >> 1) & 1, abort);
        if (elect_lane()) {
            pair_commit(&drained[h], 1);
            mbar_drain(&drained[h], 0);
        }
        __syncwarp();
    } else if (warp == kGwRelay) {
        // Gathered rows are in this CTA's shared memory; the first fence puts them before the tensor
        // core's reads there, the second before the arrival that the leader's product waits for
        // (20668 x 10 rows e4m3 568 us, without the second 565; an arrival with release at the
        // cluster waits for other copies in flight too, 2,000 cycles, and took 773, in bf16
        // 20668 x 4 rows 710 us instead of 266).
        if (c.rows) {
            const uint32_t lead = peer_smem(smem_u32(full), 0);
            int s = 0;
            uint32_t phase = 0;
            const int64_t all = tiles > pair ? (int64_t)((tiles - pair + pairs - 1) / pairs) * nk : 0;
#pragma unroll 1
            for (int64_t i = 0; i < min(all, (int64_t)keep); ++i) {
                if (!mbar_wait_all(&gathered[s], phase, abort)) break;
                fence_async_smem();
                if (lane == 0) {
                    release_smem_to_cluster();
                    mbar_arrive_cluster(lead + s * 8);
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp >= kGwFirstGather) {
        // A lane copies 16 bytes of a row, a warp four whole rows at a time and every third four.
        // Where there is no row the stage keeps what it holds: a row of the product that is not
        // written, or written as zeros.
        if (c.rows) {
            constexpr int N = (32 + kGwGather - 1) / kGwGather;
            const int first = warp - kGwFirstGather, sub = lane >> 3;       // of 32 fours; row of it
            const uint32_t to = smem_u32(smem) + sub * 128;
            // the 16 bytes' place in the swizzled rows of even fours, and of odd ones
            const uint32_t even = ((lane & 7) ^ sub) << 4, odd = ((lane & 7) ^ (sub + 4)) << 4;
            const int64_t stride = c.xs * (kBlock ? 1 : 2);
            const int bytes = c.n_in * (kBlock ? 1 : 2) - (lane & 7) * 16;  // of the row from this lane's first on
            const int whole = c.n_in * (kBlock ? 1 : 2) / 128;              // blocks of 128 bytes
            int s = 0, i = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int t = pair, tile = 0; t < tiles && ok; t += pairs, ++tile) {
                const int slot = tile % kGwTiles;
                if (!mbar_wait_all(&wide.full[slot], (tile / kGwTiles) & 1, abort)) break;
                int row[N];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int four = first + j * kGwGather;
                    row[j] = four < 32 ? wide.row[slot][four * 4 + sub] : c.n_x;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&wide.empty[slot]);
                const uint8_t *src = reinterpret_cast<const uint8_t *>(c.x) + (lane & 7) * 16;
#pragma unroll 1
                for (int k = 0; k < nk; ++k, ++i, src += 128) {
                    if (i >= S && !mbar_wait_all(&empty[s], phase, abort)) {
                        ok = false;
                        break;
                    }
                    if (i < keep) {
                        const uint32_t st = to + s * kGwStage + first * 512;
                        if (k < whole) {
#pragma unroll
                            for (int j = 0; j < N; ++j)
                                copy16_if(row[j] < c.n_x, st + j * kGwGather * 512 + ((first + j * kGwGather) & 1 ? odd : even),
                                          src + row[j] * stride);
                        } else {
                            const int n = min(16, max(0, bytes - k * 128));
#pragma unroll 1
                            for (int j = 0; j < N; ++j) {
                                int at = row[0];
#pragma unroll
                                for (int z = 1; z < N; ++z) at = z == j ? row[z] : at;      // no array in memory
                                if (at < c.n_x)
                                    copy16(st + j * kGwGather * 512 + ((first + j * kGwGather) & 1 ? odd : even),
                                           n > 0 ? src + at * stride : c.x, n);
                            }
                        }
                        copies_arrive(&gathered[s]);
                    }
                    if (++s == S) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp == kGwTile) {
        // Looks up the tiles, and makes the factors sx sw of the CTA's 128 rows, eight blocks at
        // a time, for either half.
        int v = 0;
        bool ok = true, wrong = false;
        int xr[4], next_xr[4];
        const float *sw = nullptr, *next_sw = nullptr;
        auto tell = [&](int t, int j) {
            if (t >= tiles) return true;
            const GroupTile g = find_group_tile(table, c, t, nn, kGwRows);
            const int s = j % kGwTiles, n0 = g.n * kGwChannels;
            uint32_t there[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = g.r0 + rank * 128 + i * 32 + lane;
                next_xr[i] = group_x_row(c, r, g.r1);
                if (c.rows && r < g.r1) wrong |= c.rows[r] >= c.n_x;
                there[i] = __ballot_sync(0xffffffffu, next_xr[i] < c.n_x);
            }
            if (kBlock)
                next_sw = c.sw + ((int64_t)g.e * c.nb + n0 / 128) * c.kb +
                          (lane < kGwChunk || n0 + 128 >= c.n_out ? 0 : c.kb);
            if (j >= kGwTiles && !mbar_wait_warp(&wide.empty[s], (j / kGwTiles - 1) & 1, abort)) return false;
            if (lane == 0) {
                wide.at[s] = make_int4(g.r0, g.r1, n0, g.e);
#pragma unroll
                for (int i = 0; i < 4; ++i) wide.there[s][i] = there[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wide.row[s][i * 32 + lane] = next_xr[i];
                if (next_xr[i] >= c.n_x) next_xr[i] = 0;   // whose scale is read, and not used
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&wide.full[s]);
            return true;
        };
        ok = tell(pair, 0);
        for (int t = pair, j = 0; t < tiles && ok; t += pairs, ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) xr[i] = next_xr[i];
            sw = next_sw;
            ok = tell(t + pairs, j + 1);
            for (int k0 = 0; kBlock && k0 < nk && ok; k0 += kGwChunk, ++v) {
                // lane i: the weight's scale of block k0 + i % 8 in half i / 8
                const int kw = k0 + lane % kGwChunk;
                const float w = lane < 2 * kGwChunk && kw < nk ? sw[kw] : 0.f;
                if (v >= 2 && !mbar_wait_warp(&sc_empty[v & 1], ((v >> 1) - 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                float *to = factors + (v & 1) * (kGwFactors / 4) + lane;
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    const float *sx = c.sx + (int64_t)(i < 2 ? i ? xr[1] : xr[0] : i < 3 ? xr[2] : xr[3]) * c.kb + k0;
                    float x[kGwChunk];
                    if (k0 + kGwChunk <= nk && c.sx16) {
                        const float4 p = reinterpret_cast<const float4 *>(sx)[0], q = reinterpret_cast<const float4 *>(sx)[1];
                        x[0] = p.x; x[1] = p.y; x[2] = p.z; x[3] = p.w;
                        x[4] = q.x; x[5] = q.y; x[6] = q.z; x[7] = q.w;
                    } else {
#pragma unroll
                        for (int z = 0; z < kGwChunk; ++z) x[z] = k0 + z < nk ? sx[z] : 0.f;
                    }
#pragma unroll
                    for (int z = 0; z < 2 * kGwChunk; ++z)
                        to[z * 128 + i * 32] = x[z % kGwChunk] * __shfl_sync(0xffffffffu, w, z);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[v & 1]);
            }
        }
        if (wrong) flag_status(GDN_DEVSTAT_BAD_INDEX);
    } else if (warp >= kGwFirstEpi && warp < kGwFirstGather) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(GwRegs<kBlock>::kMany));
        // Accumulator lane 32 q + l is token row 32 q + l of this CTA's 128; four warps a half.
        const int q = warp & 3, h = (warp - kGwFirstEpi) >> 2, p = kBlock ? h : 0;
        uint8_t *staging = smem + S * kGwStage + (warp - kGwFirstEpi) * M::kStaging;
        const uint32_t sums = tmem_addr(tmem_base, q * 32, h * 128), release = peer_smem(smem_u32(acc_empty[p]), 0);
        int u = 0, v = 0;                  // accumulators and chunks of factors used so far
        uint32_t r[2][32];
        bool ok = true, ready = false;     // the next accumulator is known to be there
        const int mine_tiles = tiles > pair ? (tiles - pair + pairs - 1) / pairs : 0;
        for (int tile = 0; tile < mine_tiles; ++tile) {
            const int slot = tile % kGwTiles;          // held until the tile is out: registers are short here
            if (!mbar_wait_all(&wide.full[slot], (tile / kGwTiles) & 1, abort)) break;
            const bool mine = !kBlock || h == 0 || wide.at[slot].z + 128 < c.n_out;
            F2 acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = f2(0.f, 0.f);
            const float *sc = factors + h * kGwChunk * 128 + q * 32 + lane;
#pragma unroll 1
            for (int k0 = 0; k0 < (kBlock ? nk : 1) && ok; k0 += kGwChunk) {
                const int n = kBlock ? min(nk - k0, kGwChunk) : 1;
                const float *f = sc + (v & 1) * (kGwFactors / 4);
                if (kBlock && !mbar_wait_all(&sc_full[v & 1], (v >> 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                float f0 = kBlock ? *f : 1.f;
#pragma unroll 1
                for (int k = 0; mine && k < n; ++k) {
                    if (!ready) {
                        if (!mbar_wait_all(&acc_full[p][u & 1], (u >> 1) & 1, abort)) {
                            ok = false;
                            break;
                        }
                    }
                    tc_fence_after();
                    tmem_ask(sums + (u & 1) * 256, r[0]);
                    const uint32_t from = sums + (u & 1) * 256;
                    const F2 f2x = f2(f0, f0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        tmem_wait(r[j & 1]);
                        if (j < 3) {
                            tmem_ask(from + (j + 1) * 32, r[(j + 1) & 1]);
                        } else {                           // all of it has been read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(release + (u & 1) * 8);
                            ++u;
                            if (kBlock && k + 1 < n) f0 = f[(k + 1) * 128];
                            // the next block's first columns, while this one's last are added
                            ready = mbar_test(&acc_full[p][u & 1], (u >> 1) & 1);
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const F2 x = f2_bits(r[j & 1][2 * i], r[j & 1][2 * i + 1]);
                            acc[j * 16 + i] = kBlock ? f2_fma(x, f2x, acc[j * 16 + i]) : x;
                        }
                    }
                    ready = __all_sync(0xffffffffu, ready);
                }
                if (kBlock) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sc_empty[v & 1]);
                    ++v;
                }
            }
            if (!ok) break;
            const int4 a = wide.at[slot];
            const bool there = wide.there[slot][q] >> lane & 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&wide.empty[slot]);
            if (mine) wide_store<O, M::kHold>(acc, staging, &my, c, a.x + rank * 128 + q * 32, a.y, a.z + h * 128, there, lane);
        }
        if (lane == 0) bulk_wait_read_all();       // the staging tiles stay until they are read
        __syncwarp();
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

template <bool kBlock, typename O> gdn_status launch(GroupedCall c, int drop, cudaStream_t s) {
    CUtensorMap mx, mw, my = {};
    if (!encode_tmap_rows(&mx, c, 128) || !encode_tmap_experts(&mw, c, 64)) return GDN_ERR_CUDA;
    if (c.vec16 && !encode_tmap_2d(&my, sizeof(O) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                   c.y, c.n_out, c.n_rows, c.n_rows == 1 ? (uint64_t)c.n_out * sizeof(O) : c.ys * sizeof(O),
                                   128 / sizeof(O), 32, true))
        return GDN_ERR_CUDA;
    auto kernel = grouped_wide_kernel<kBlock, O>;
    static SmemAllowed allowed;
    cudaError_t e = allowed.ask(kernel, GwSmem<kBlock>::kBytes);
    const int64_t nn = (c.n_out + kGwChannels - 1) / kGwChannels;
    const int64_t tiles = most_row_tiles(c, kGwRows) * nn;
    if (tiles >= (1ll << 31)) return GDN_ERR_UNSUPPORTED;
    c.channel_tiles(nn);
    if (e == cudaSuccess)
        e = launch_after(kernel, dim3((unsigned)std::min<int64_t>(2 * tiles, sm_count() / 2 * 2)), dim3(kGwThreads),
                         GwSmem<kBlock>::kBytes, s, mx, mw, my, c,
                         drop == kDropNone ? INT_MAX : drop & kDropAll ? 0 : (c.n_in + (kBlock ? 127 : 63)) / (kBlock ? 128 : 64));
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
