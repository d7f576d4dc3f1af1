// Grouped and block-scaled products, few rows an expert: an expert's 128 weight
// rows are the lanes of the accumulator and up to BT of its tokens the columns, so
// that a tile of few rows costs little more than reading its weights.  Of 128 rows a
// tile they change places (kTurned): a lane has one token, so that its factor sx sw is
// one number a block, not one for each column out of shared memory, and a row's part of
// y is written in pieces of 16 bytes (256 x 2048 x 8192: 12.1 -> 9.8 us).
//
// Persistent CTAs, a warp for each part: loads (tiles by TMA; gathered rows in pieces
// of 16 bytes, by a warp or, of 32 and more a tile, five: a TMA gather of four rows takes
// 150 cycles and held one token's block at 620, one warp 64 rows of a block at 900),
// products, scales, and 4 or 8 that sum the blocks.  With block scales every block of 128
// in k is a product of its own into one of four accumulators; the summing warps add it,
// times sx sw, to registers.  A block takes such a warp some 500 cycles of waits and
// latencies, so two groups of four share the columns of a tile of 32 rows or more (with four
// groups 256 x 2048 x 8192 took half a microsecond longer).  Where there are few tiles, a
// cluster's CTAs share the blocks of one (64 x 4096 x 2048: 12.4 -> 8.5 us, 16 x 16384 x
// 256: 40 -> 10).
#include <limits.h>

#include <algorithm>

#include "grouped.cuh"

namespace gdn {

using namespace tc;

GDN_DECLARE_STATUS_WORD(g_status_grouped_narrow)
GDN_STATUS_READER(read_status_grouped_narrow, g_status_grouped_narrow)

cudaError_t set_grouped_narrow_limit(uint64_t limit_ns, cudaStream_t s) {
    return cudaMemcpyToSymbolAsync(tc::g_wait_limit_ns, &limit_ns, sizeof(limit_ns), 0, cudaMemcpyHostToDevice, s);
}

namespace {

constexpr int kScaleChunk = 8;         // blocks whose scales are handed over at a time
// Warps: 0 loads by TMA, 1 products, 2 scales, 3 on sums, then gathered rows: a multiple
// of four, by which registers are shared out.
constexpr int kGnScale = 2, kGnFirstSum = 3;

template <int BT> struct GnCfg {
    static constexpr uint32_t kW = 128 * 128, kX = BT * 128, kStage = kW + kX;
    static constexpr int kStages = BT == 16 ? 11 : BT == 32 ? 10 : BT == 64 ? 8 : 6;
    static constexpr int kAccs = 4;
    static constexpr int kSums = BT >= 32 ? 8 : 4;        // summing warps, groups of four share the columns
    static constexpr int kGather = BT >= 32 ? 5 : 1;      // warps for gathered rows
    static constexpr int kWidth = BT * 4 / kSums;         // columns of one
    static constexpr int kThreads = 32 * (kGnFirstSum + kSums + kGather);
    // of 128 rows a tile, the rows are the accumulator's lanes
    static constexpr bool kTurned = BT == 128;
    static constexpr uint32_t kScales = 2 * kScaleChunk * BT * 4;
    static constexpr uint32_t kStaging = kTurned ? 2048 : 0;      // of a summing warp: 64 bytes of 32 rows
    static constexpr uint32_t kSmem = kStages * kStage + kScales + kSums * kStaging;
};

// A warp's 32 rows from row0 on, a lane each, and W channels from n0 on, by way of a few
// bytes of each row in shared memory, so that a row's neighbours go out together: 64, in
// pieces of 16 (kPieces), or 32, as elements.  (Each lane its own row, 16 bytes at a time,
// writes half sectors: 18 experts of 3000 rows, 263 x 5392 e4m3, 373 us, so 255.)
template <bool kPieces, typename O, int W>
__device__ __forceinline__ void store_lanes(const F2 (&acc)[W / 2], uint8_t *staging, const GroupedCall &c, int row0, int r1,
                                            int n0, bool there, int lane) {
    constexpr int V = 16 / sizeof(O), P = kPieces ? 4 : 2, N = P * V;    // channels of 16 bytes, of a round
    O *y = reinterpret_cast<O *>(c.y) + (int64_t)row0 * c.ys + n0;
    const int rows = r1 - row0, left = c.n_out - n0;
#pragma unroll
    for (int i = 0; i < W; i += N) {
        if (i >= left) break;
        __syncwarp();                                  // the last round's are read
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const F2 *p = acc + (i + j * V) / 2;
            uint4 v;
            if constexpr (sizeof(O) == 2) {
                const float2 a = f2_get(p[0]), b = f2_get(p[1]), d = f2_get(p[2]), e = f2_get(p[3]);
                v = make_uint4(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y), pack_bf16(d.x, d.y), pack_bf16(e.x, e.y));
            } else {
                const float2 a = f2_get(p[0]), b = f2_get(p[1]);
                v = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
            }
            if (!there) v = make_uint4(0u, 0u, 0u, 0u);
            reinterpret_cast<uint4 *>(staging)[lane * P + (kPieces ? j ^ (lane >> 1 & 3) : j)] = v;
        }
        __syncwarp();
        if (kPieces) {
            const int first = lane >> 2, piece = lane & 3;                 // eight rows at a time
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = reinterpret_cast<const uint4 *>(staging)[(j * 8 + first) * 4 + (piece ^ (first >> 1 & 3))];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j * 8 + first < rows && i + piece * V < left)
                    *reinterpret_cast<uint4 *>(y + (j * 8 + first) * c.ys + i + piece * V) = v[j];
        } else {
            const int first = lane / N, ch = lane % N;                     // 32 / N rows at a time
            O e[N];                                    // all read before the first is written
#pragma unroll
            for (int j = 0; j < N; ++j) e[j] = reinterpret_cast<const O *>(staging)[j * 32 + lane];
            O *to = y + first * c.ys + i + ch;
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j * (32 / N) + first < rows && i + ch < left) to[j * (32 / N) * c.ys] = e[j];
        }
    }
    __syncwarp();
}

template <int BT, bool kBlock, bool kPieces>
__global__ void __launch_bounds__(GnCfg<BT>::kThreads)
grouped_narrow_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                      const __grid_constant__ GroupedCall c, int cut, int keep) {
    using C = GnCfg<BT>;
    constexpr int S = C::kStages, A = C::kAccs;
    constexpr bool kTurned = C::kTurned;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ GroupTable table;
    __shared__ uint64_t full[S], empty[S], acc_full[A], acc_empty[A], sc_full[2], sc_empty[2], drained;
    __shared__ uint32_t valid[2][BT < 32 ? 1 : BT / 32];   // rows that there are, with the scales
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    constexpr int kElems = kBlock ? 128 : 64;
    const int nn = (c.n_out + 127) / 128;
    // Blocks kb0 .. nk - 1 are this CTA's: all, or its part where 2^cut CTAs, a cluster, share
    // a tile (one each at most).
    const bool shared = cut > 0;
    const int rank = shared ? (int)cta_rank() : 0, split = shared ? 1 << cut : 1;
    int kb0 = 0, nk = (c.n_in + kElems - 1) / kElems, tile0 = blockIdx.x, tile_step = gridDim.x;
    if (shared) {
        kb0 = nk * rank >> cut;
        nk = nk * (rank + 1) >> cut;
        tile0 >>= cut;
        tile_step >>= cut;
    }
    float *scales = reinterpret_cast<float *>(smem + S * C::kStage);
    volatile int *abort = &abort_flag;

    if (tid == 0) {
        prefetch_tensormap(&mx);
        prefetch_tensormap(&mw);
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], c.rows ? 1 + 32 * C::kGather : 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < A; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], C::kSums);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_empty[i], C::kSums);
        }
        mbar_init(&drained, 1);
        abort_flag = (smem_u32(smem) & 1023u) != 0;
        fence_mbar_init();
        fence_async_smem();
    }
    griddep_wait();
    if (warp == 1) {
        tmem_alloc(&tmem_base, A * BT);
        tmem_relinquish();
    }
    tc_fence_before();
    bool bad;
    const int tiles = build_group_table(table, c, BT, &bad) * nn;    // has barriers
    tc_fence_after();
    if (bad && tid == 0 && blockIdx.x == 0) flag_status(GDN_DEVSTAT_BAD_SEQLEN);

    if (warp == 0) {
        const bool one = elect_lane();
        int s = 0, i = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int t = tile0; t < tiles && ok; t += tile_step) {
            const GroupTile a = find_group_tile(table, c, t, nn, BT);
            const uint32_t bytes = c.rows ? C::kW : C::kStage;
#pragma unroll 1
            for (int k = kb0; k < nk; ++k, ++i) {
                if (i >= S && !mbar_wait_all(&empty[s], phase, abort)) {
                    ok = false;
                    break;
                }
                uint8_t *st = smem + s * C::kStage;
                if (i < keep && one) {
                    mbar_arrive_expect_tx(&full[s], bytes);
                    tma_load_3d(st, &mw, smem_u32(&full[s]), k * kElems, a.n * 128, a.e);
                    if (!c.rows) tma_load_2d(st + C::kW, &mx, &full[s], k * kElems, a.r0);
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        griddep_launch();
        for (int j = i > S ? i - S : 0; ok && j < i; ++j) ok = mbar_wait_all(&empty[j % S], (j / S) & 1, abort);
        if (one && (!ok || *abort)) {      // given up: the copies in flight land before the CTA ends
            if (c.rows) let_copies_land(); // the barriers count the gathered rows too
            else
                for (int j = i > S ? i - S : 0; j < min(i, keep); ++j) mbar_drain(&full[j % S], (j / S) & 1);
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = kBlock ? idesc_e4m3(128, BT) : idesc_bf16(128, BT);
        const uint64_t desc = sdesc_sw128(0, 0, 1024);
        const uint32_t base = smem_u32(smem) >> 4, sums = tmem_base;
        int s = 0, u = 0;                  // u: accumulators used so far
        uint32_t phase = 0;
        bool ok = true, ready = false;     // operands and accumulator of the next block are known to be there
        for (int t = tile0; t < tiles && ok; t += tile_step) {
#pragma unroll 1
            for (int k = kb0; k < nk; ++k) {
                if (!ready) {
                    ok = mbar_wait_all(&full[s], phase, abort);
                    if (ok && (kBlock || k == kb0) && u >= A) ok = mbar_wait_all(&acc_empty[u % A], (u / A - 1) & 1, abort);
                    if (!ok) break;
                }
                tc_fence_after();
                if (c.rows) fence_async_smem();           // rows that threads have written, before the product reads them
                const bool last = kBlock || k == nk - 1;
                if (elect_lane()) {
                    const uint32_t st = base + s * (C::kStage >> 4), d = sums + u % A * BT;
                    const uint32_t xt = st + (C::kW >> 4);
                    const uint64_t da = desc | (kTurned ? xt : st), db = desc | (kTurned ? st : xt);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        linear_mma<kBlock>(d, da + 2 * q, db + 2 * q, idesc, q > 0 || (!kBlock && k > kb0));
                    mma_commit(&empty[s]);
                    if (last) mma_commit(&acc_full[u % A]);
                }
                __syncwarp();
                if (last) ++u;
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
                // (a wait that finds its barrier done takes 150 cycles, two looks ahead of time hardly any)
                ready = mbar_test(&full[s], phase);
                if (last && u >= A) ready = mbar_test(&acc_empty[u % A], (u / A - 1) & 1) && ready;
                ready = __all_sync(0xffffffffu, ready);
            }
        }
        if (elect_lane()) {
            mma_commit(&drained);
            mbar_drain(&drained, 0);
        }
        __syncwarp();
    } else if (warp >= kGnFirstSum + C::kSums) {
        // A lane copies 16 bytes of a row, a warp four whole rows at a time and, of more warps,
        // every so-manieth four.  Where there is no row the stage keeps what it holds: a column
        // that is not written, or written as zeros.
        if (c.rows) {
            constexpr int G = C::kGather, N = (BT / 4 + G - 1) / G;
            const int first = warp - kGnFirstSum - C::kSums, sub = lane >> 3;   // of all fours; row of it
            const uint32_t to = smem_u32(smem) + C::kW + sub * 128;
            // the 16 bytes' place in the swizzled rows of even fours, and of odd ones
            const uint32_t even = ((lane & 7) ^ sub) << 4, odd = ((lane & 7) ^ (sub + 4)) << 4;
            const int64_t stride = c.xs * (kBlock ? 1 : 2);
            const int bytes = c.n_in * (kBlock ? 1 : 2) - (lane & 7) * 16;  // of the row from this lane's first on
            const int whole = c.n_in * (kBlock ? 1 : 2) / 128;              // blocks of 128 bytes
            int s = 0, i = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int t = tile0; t < tiles && ok; t += tile_step) {
                const GroupTile a = find_group_tile(table, c, t, nn, BT);
                int row[N];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int four = first + j * G;
                    row[j] = four < BT / 4 ? group_x_row(c, a.r0 + four * 4 + sub, a.r1) : c.n_x;
                }
                const uint8_t *src = reinterpret_cast<const uint8_t *>(c.x) + (lane & 7) * 16 + kb0 * 128;
#pragma unroll 1
                for (int k = kb0; k < nk; ++k, ++i, src += 128) {
                    if (i >= S && !mbar_wait_all(&empty[s], phase, abort)) {
                        ok = false;
                        break;
                    }
                    if (i < keep) {
                        const uint32_t st = to + s * C::kStage + first * 512;
                        if (k < whole) {
#pragma unroll
                            for (int j = 0; j < N; ++j)
                                copy16_if(row[j] < c.n_x, st + j * G * 512 + ((first + j * G) & 1 ? odd : even),
                                          src + row[j] * stride);
                        } else {
                            const int n = min(16, max(0, bytes - k * 128));
#pragma unroll 1
                            for (int j = 0; j < N; ++j) {
                                int at = row[0];
#pragma unroll
                                for (int z = 1; z < N; ++z) at = z == j ? row[z] : at;      // no array in memory
                                if (at < c.n_x)
                                    copy16(st + j * G * 512 + ((first + j * G) & 1 ? odd : even),
                                           n > 0 ? src + at * stride : c.x, n);
                            }
                        }
                        copies_arrive(&full[s]);
                    }
                    if (++s == S) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp == kGnScale) {
        // Scales of the next blocks, times the weight's, and which rows there are.
        int slot = 0, v = 0;
        bool ok = true, wrong = false;
        for (int t = tile0; t < tiles && ok; t += tile_step) {
            const GroupTile a = find_group_tile(table, c, t, nn, BT);
            constexpr int Q = (BT + 31) / 32;
            int row[Q];
            uint32_t there[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int col = q * 32 + lane, r = a.r0 + col;
                row[q] = col < BT ? group_x_row(c, r, a.r1) : c.n_x;
                if (col < BT && r < a.r1 && c.rows) wrong |= c.rows[r] >= c.n_x;
                there[q] = __ballot_sync(0xffffffffu, row[q] < c.n_x);
            }
            const float *sw = kBlock ? c.sw + ((int64_t)a.e * c.nb + a.n) * c.kb : nullptr;
            for (int k0 = kBlock ? kb0 : 0; k0 < (kBlock ? nk : 1) && ok; k0 += kScaleChunk, ++v, slot ^= 1) {
                __align__(16) float f[Q][kScaleChunk];       // written by vectors
                if (kBlock) {
                    const bool pieces = k0 + kScaleChunk <= nk && c.sx16 && k0 % 4 == 0;
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const float *sx = c.sx + (int64_t)row[q] * c.kb + k0;
                        if (pieces && row[q] < c.n_x) {
                            *reinterpret_cast<float4 *>(f[q]) = *reinterpret_cast<const float4 *>(sx);
                            *reinterpret_cast<float4 *>(f[q] + 4) = *reinterpret_cast<const float4 *>(sx + 4);
                        } else {
#pragma unroll
                            for (int i = 0; i < kScaleChunk; ++i) f[q][i] = k0 + i < nk && row[q] < c.n_x ? sx[i] : 0.f;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kScaleChunk; ++i) {
                        const float w = k0 + i < nk ? sw[k0 + i] : 0.f;
#pragma unroll
                        for (int q = 0; q < Q; ++q) f[q][i] *= w;
                    }
                }
                if (v >= 2 && !mbar_wait_all(&sc_empty[slot], (v / 2 - 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                if (kBlock) {
#pragma unroll
                    for (int i = 0; i < kScaleChunk; ++i)
#pragma unroll
                        for (int q = 0; q < Q; ++q)
                            if (q * 32 + lane < BT) scales[(slot * kScaleChunk + i) * BT + q * 32 + lane] = f[q][i];
                }
                if (lane == 0) {
#pragma unroll
                    for (int q = 0; q < Q; ++q) valid[slot][q] = there[q];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[slot]);
            }
        }
        if (wrong) flag_status(GDN_DEVSTAT_BAD_INDEX);
    } else if (warp >= kGnFirstSum) {
        // Accumulator lane 32 q + l is channel 32 q + l of the tile, turned row 32 q + l.
        constexpr int W = C::kWidth, L = W < 32 ? 16 : 32;       // columns, and of a load
        const int q = warp & 3, c0 = ((warp - kGnFirstSum) >> 2) * W;
        int u = 0, v = 0;                  // accumulators and chunks used so far
        bool ok = true, ready = false;     // the next accumulator is known to be there
        const int blocks = kBlock ? nk : 1;
        bool joined = false;               // the cluster's other parts have been waited for
        for (int t = tile0; t < tiles && ok; t += tile_step) {
            const GroupTile a = find_group_tile(table, c, t, nn, BT);
            F2 acc[W / 2];
#pragma unroll
            for (int i = 0; i < W / 2; ++i) acc[i] = f2(0.f, 0.f);
            uint32_t there[kTurned ? 1 : (W + 31) / 32];
#pragma unroll 1
            for (int k0 = kBlock ? kb0 : 0; k0 < blocks && ok; k0 += kScaleChunk, ++v) {
                const int slot = v & 1, n = min(blocks - k0, kScaleChunk);
                if (!mbar_wait_all(&sc_full[slot], (v >> 1) & 1, abort)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < (kTurned ? 1 : (W + 31) / 32); ++i) there[i] = valid[slot][kTurned ? q : c0 / 32 + i] >> (kTurned ? 0 : c0 % 32);
                const float *sc = scales + slot * kScaleChunk * BT + (kTurned ? q * 32 + lane : c0);
#pragma unroll 1
                for (int k = 0; k < n; ++k, sc += BT) {
                    if (!ready && !mbar_wait_all(&acc_full[u % A], (u / A) & 1, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float own = kTurned && kBlock ? *sc : 1.f;
                    const uint32_t from = tmem_addr(tmem_base, q * 32, u % A * BT + c0);
                    uint32_t r[W / L][L];
#pragma unroll
                    for (int j = 0; j < W / L; ++j) tmem_ask(from + j * L, r[j]);
#pragma unroll
                    for (int j = 0; j < W / L; ++j) tmem_wait(r[j]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[u % A]);
                    ++u;
                    ready = mbar_test(&acc_full[u % A], (u / A) & 1);
#pragma unroll
                    for (int i = 0; i < W; i += 4) {
                        const uint32_t *p = r[i / L] + i % L;
                        F2 &lo = acc[i / 2], &hi = acc[i / 2 + 1];
                        if (kBlock && kTurned) {
                            lo = f2_fma(f2_bits(p[0], p[1]), f2(own, own), lo);
                            hi = f2_fma(f2_bits(p[2], p[3]), f2(own, own), hi);
                        } else if (kBlock) {
                            const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(sc + i);
                            lo = f2_fma(f2_bits(p[0], p[1]), f.x, lo);
                            hi = f2_fma(f2_bits(p[2], p[3]), f.y, hi);
                        } else {
                            lo = f2_bits(p[0], p[1]);
                            hi = f2_bits(p[2], p[3]);
                        }
                    }
                    ready = __all_sync(0xffffffffu, ready);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_empty[slot]);
            }
            if (!ok) break;
            if (shared) {
                // The leader adds the others' sums, in their order, out of their shared memory
                // (the ring's, which nothing reads or fills any more).
                joined = true;
                const uint32_t place = smem_u32(smem) + ((warp - kGnFirstSum) * (W / 2) * 32 + lane) * 8;
                if (rank != 0) {
#pragma unroll
                    for (int i = 0; i < W / 2; ++i)
                        asm volatile("st.shared.b64 [%0], %1;" ::"r"(place + i * 256), "l"(acc[i]) : "memory");
                }
                __syncwarp();
                cluster_arrive();
                cluster_wait();
                if (rank != 0) break;
                for (int j = 1; j < split; ++j) {
                    const uint32_t from = peer_smem(place, j);
                    int gone;
                    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(gone) : "r"(peer_smem(smem_u32(&abort_flag), j)) : "memory");
                    if (gone) *abort = 1;                  // what it has is no sum
#pragma unroll
                    for (int i = 0; i < W / 2; ++i) {
                        F2 x;
                        asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(x) : "r"(from + i * 256) : "memory");
                        acc[i] = f2_add(acc[i], x);
                    }
                }
                if (*abort) break;
            }
            if constexpr (kTurned) {
                const bool is = there[0] >> lane & 1;
                uint8_t *staging = smem + S * C::kStage + C::kScales + (warp - kGnFirstSum) * C::kStaging;
                if (c.out_f32) store_lanes<kPieces, float, W>(acc, staging, c, a.r0 + q * 32, a.r1, a.n * 128 + c0, is, lane);
                else store_lanes<kPieces, __nv_bfloat16, W>(acc, staging, c, a.r0 + q * 32, a.r1, a.n * 128 + c0, is, lane);
            } else {
                const int n = a.n * 128 + q * 32 + lane, cnt = min(W, a.r1 - a.r0 - c0);
                if (n < c.n_out) {
                    const int64_t at = (int64_t)(a.r0 + c0) * c.ys + n;
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const float2 f = f2_get(acc[i / 2]);
                        const float val = there[i / 32] >> (i % 32) & 1 ? (i & 1 ? f.y : f.x) : 0.f;
                        if (i < cnt) {
                            if (c.out_f32) reinterpret_cast<float *>(c.y)[at + i * c.ys] = val;
                            else reinterpret_cast<__nv_bfloat16 *>(c.y)[at + i * c.ys] = __float2bfloat16_rn(val);
                        }
                    }
                }
            }
        }
        if (shared && !joined) {
            __syncwarp();
            cluster_arrive();
            cluster_wait();
        }
        tc_fence_before();
    }
    if (shared) {
        __syncwarp();
        if (warp < kGnFirstSum || warp >= kGnFirstSum + C::kSums) {
            cluster_arrive();
            cluster_wait();
        }
        // no CTA ends while the leader may read its sums; one that has given up does not use what
        // it asked for, and waits for it here
        if (*abort) cluster_arrive();
        else cluster_arrive_relaxed();
        cluster_wait();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, A * BT);
    if (tid == 0 && abort_flag) flag_status(GDN_DEVSTAT_TIMEOUT);
}

template <int BT, bool kBlock, bool kPieces = true> gdn_status launch(GroupedCall c, int cut, int drop, cudaStream_t s) {
    using C = GnCfg<BT>;
    CUtensorMap mx, mw;
    if (!encode_tmap_rows(&mx, c, BT) || !encode_tmap_experts(&mw, c, 128)) return GDN_ERR_CUDA;
    auto kernel = grouped_narrow_kernel<BT, kBlock, kPieces>;
    static SmemAllowed allowed;
    cudaError_t e = allowed.ask(kernel, C::kSmem);
    const int64_t nn = (c.n_out + 127) / 128;
    const int64_t tiles = most_row_tiles(c, BT) * nn;
    if (tiles >= (1ll << 31)) return GDN_ERR_UNSUPPORTED;
    c.channel_tiles(nn);
    const int keep = drop == kDropNone ? INT_MAX : drop & kDropAll ? 0 : 1;
    if (e == cudaSuccess)
        e = cut > 0 ? launch_after_cluster(kernel, 1 << cut, dim3((unsigned)tiles << cut), dim3(C::kThreads), C::kSmem, s, mx,
                                           mw, c, cut, keep)
                    : launch_after(kernel, dim3((unsigned)std::min<int64_t>(tiles, sm_count())), dim3(C::kThreads), C::kSmem, s,
                                   mx, mw, c, cut, keep);
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

}  // namespace

int grouped_eights() {
    static ClustersHeld held;
    int count = 0;
    using C = GnCfg<128>;
    return held.ask(grouped_narrow_kernel<128, true, true>, 8, C::kThreads, C::kSmem, count) == cudaSuccess ? count : 0;
}

gdn_status launch_grouped_narrow(const GroupedCall &c, int tile_rows, int cut, int drop, cudaStream_t s) {
    switch (tile_rows) {
        case 16: return c.e4m3 ? launch<16, true>(c, cut, drop, s) : launch<16, false>(c, cut, drop, s);
        case 32: return c.e4m3 ? launch<32, true>(c, cut, drop, s) : launch<32, false>(c, cut, drop, s);
        case 64: return c.e4m3 ? launch<64, true>(c, cut, drop, s) : launch<64, false>(c, cut, drop, s);
        default:
            if (!c.vec16) return c.e4m3 ? launch<128, true, false>(c, cut, drop, s) : launch<128, false, false>(c, cut, drop, s);
            return c.e4m3 ? launch<128, true>(c, cut, drop, s) : launch<128, false>(c, cut, drop, s);
    }
}

}  // namespace gdn
