// Grouped and block-scaled products, few rows an expert: an expert's 128 weight
// rows are the lanes of the accumulator and up to BT of its tokens the columns, so
// that a tile of few rows costs little more than reading its weights.
//
// Persistent CTAs, a warp for each part: loads (weights as tiles, the tokens' rows
// gathered), products, scales, and four that sum the blocks.  With block scales
// every block of 128 in k is a product of its own into one of four accumulators;
// the summing warps add it, times sx sw of its column, to registers.
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
constexpr int kGnThreads = 7 * 32;

template <int BT> struct GnCfg {
    static constexpr uint32_t kW = 128 * 128, kX = BT * 128, kStage = kW + kX;
    static constexpr int kStages = BT == 16 ? 11 : BT == 32 ? 10 : BT == 64 ? 8 : 6;
    static constexpr int kAccs = 4;
    static constexpr uint32_t kScales = 2 * kScaleChunk * BT * 4;
    static constexpr uint32_t kSmem = kStages * kStage + kScales;
};

template <int BT, bool kBlock>
__global__ void __launch_bounds__(kGnThreads)
grouped_narrow_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                      const __grid_constant__ GroupedCall c, int keep) {
    using C = GnCfg<BT>;
    constexpr int S = C::kStages, A = C::kAccs;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ GroupTable table;
    __shared__ uint64_t full[S], empty[S], acc_full[A], acc_empty[A], sc_full[2], sc_empty[2], drained;
    __shared__ uint32_t valid[2][BT < 32 ? 1 : BT / 32];   // rows that there are, with the scales
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    constexpr int kElems = kBlock ? 128 : 64;
    const int nk = (c.n_in + kElems - 1) / kElems, nn = (c.n_out + 127) / 128;
    float *scales = reinterpret_cast<float *>(smem + S * C::kStage);
    volatile int *abort = &abort_flag;

    if (tid == 0) {
        prefetch_tensormap(&mx);
        prefetch_tensormap(&mw);
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < A; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_empty[i], 4);
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
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const GroupTile a = find_group_tile(table, c.n_experts, t, nn, BT);
            int4 rows;
            if (c.rows) {
                const int r = a.r0 + lane * 4;
                rows = make_int4(group_x_row(c, r, a.r1), group_x_row(c, r + 1, a.r1), group_x_row(c, r + 2, a.r1),
                                 group_x_row(c, r + 3, a.r1));
            }
#pragma unroll 1
            for (int k = 0; k < nk; ++k, ++i) {
                if (i >= S && !mbar_wait_all(&empty[s], phase, abort)) {
                    ok = false;
                    break;
                }
                uint8_t *st = smem + s * C::kStage;
                const uint32_t bar = smem_u32(&full[s]);
                if (i < keep) {
                    if (one) {
                        mbar_arrive_expect_tx(&full[s], C::kStage);
                        tma_load_3d(st, &mw, bar, k * kElems, a.n * 128, a.e);
                        if (!c.rows) tma_load_2d(st + C::kW, &mx, &full[s], k * kElems, a.r0);
                    }
                    __syncwarp();
                    if (c.rows && lane < BT / 4) tma_gather4(st + C::kW + lane * 512, &mx, bar, k * kElems, rows);
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
        if (one && (!ok || *abort))        // given up: the copies in flight land before the CTA ends
            for (int j = i > S ? i - S : 0; j < min(i, keep); ++j) mbar_drain(&full[j % S], (j / S) & 1);
    } else if (warp == 1) {
        constexpr uint32_t idesc = kBlock ? idesc_e4m3(128, BT) : idesc_bf16(128, BT);
        const uint64_t desc = sdesc_sw128(0, 0, 1024);
        const uint32_t base = smem_u32(smem) >> 4, sums = tmem_base;
        int s = 0, u = 0;                  // u: accumulators used so far
        uint32_t phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
#pragma unroll 1
            for (int k = 0; k < nk; ++k) {
                if ((kBlock || k == 0) && u >= A && !mbar_wait_all(&acc_empty[u % A], (u / A - 1) & 1, abort)) ok = false;
                if (!ok || !mbar_wait_all(&full[s], phase, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_lane()) {
                    const uint32_t st = base + s * (C::kStage >> 4), d = sums + u % A * BT;
                    const uint64_t da = desc | st, db = desc | (st + (C::kW >> 4));
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        linear_mma<kBlock>(d, da + 2 * q, db + 2 * q, idesc, q > 0 || (!kBlock && k > 0));
                    mma_commit(&empty[s]);
                    if (kBlock || k == nk - 1) mma_commit(&acc_full[u % A]);
                }
                __syncwarp();
                if (kBlock || k == nk - 1) ++u;
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        if (elect_lane()) {
            mma_commit(&drained);
            mbar_drain(&drained, 0);
        }
        __syncwarp();
    } else if (warp == 6) {
        // Scales of the next blocks, times the weight's, and which rows there are.
        int slot = 0, v = 0;
        bool ok = true, wrong = false;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const GroupTile a = find_group_tile(table, c.n_experts, t, nn, BT);
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
            for (int k0 = 0; k0 < (kBlock ? nk : 1) && ok; k0 += kScaleChunk, ++v, slot ^= 1) {
                float f[Q][kScaleChunk];
                if (kBlock) {
#pragma unroll
                    for (int i = 0; i < kScaleChunk; ++i) {
                        const float w = k0 + i < nk ? sw[k0 + i] : 0.f;
#pragma unroll
                        for (int q = 0; q < Q; ++q)
                            f[q][i] = k0 + i < nk && row[q] < c.n_x ? w * c.sx[(int64_t)row[q] * c.kb + k0 + i] : 0.f;
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
    } else {
        // Accumulator lane 32 q + l is channel 32 q + l of the tile.
        const int q = warp & 3;
        int u = 0, slot = 0, v = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const GroupTile a = find_group_tile(table, c.n_experts, t, nn, BT);
            F2 acc[BT / 2];
#pragma unroll
            for (int i = 0; i < BT / 2; ++i) acc[i] = f2(0.f, 0.f);
            uint32_t there[(BT + 31) / 32];
#pragma unroll 1
            for (int k = 0; k < (kBlock ? nk : 1); ++k, ++u) {
                if (k % kScaleChunk == 0 && !mbar_wait_all(&sc_full[slot], (v / 2) & 1, abort)) ok = false;
                if (!ok || !mbar_wait_all(&acc_full[u % A], (u / A) & 1, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t from = tmem_addr(tmem_base, q * 32, u % A * BT);
                const float *sc = scales + (slot * kScaleChunk + k % kScaleChunk) * BT;
                uint32_t r[2][16];
                tmem_ask16(from, r[0]);
#pragma unroll
                for (int j = 0; j < BT / 16; ++j) {
                    tmem_wait16(r[j & 1]);
                    if (j + 1 < BT / 16) tmem_ask16(from + (j + 1) * 16, r[(j + 1) & 1]);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const uint32_t *p = r[j & 1] + i;
                        F2 &lo = acc[j * 8 + i / 2], &hi = acc[j * 8 + i / 2 + 1];
                        if (kBlock) {
                            const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(sc + j * 16 + i);
                            lo = f2_fma(f2_bits(p[0], p[1]), f.x, lo);
                            hi = f2_fma(f2_bits(p[2], p[3]), f.y, hi);
                        } else {
                            lo = f2_bits(p[0], p[1]);
                            hi = f2_bits(p[2], p[3]);
                        }
                    }
                }
                tc_fence_before();
                if (!kBlock || k == nk - 1) {
#pragma unroll
                    for (int i = 0; i < (BT + 31) / 32; ++i) there[i] = valid[slot][i];
                }
                const bool last = !kBlock || k == nk - 1 || k % kScaleChunk == kScaleChunk - 1;
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&acc_empty[u % A]);
                    if (last) mbar_arrive(&sc_empty[slot]);
                }
                if (last) {
                    slot ^= 1;
                    ++v;
                }
            }
            if (!ok) break;
            const int n = a.n * 128 + q * 32 + lane, cnt = min(BT, a.r1 - a.r0);
            if (n < c.n_out) {
                const int64_t at = (int64_t)a.r0 * c.ys + n;
#pragma unroll
                for (int i = 0; i < BT; ++i) {
                    const float2 f = f2_get(acc[i / 2]);
                    const float val = there[i / 32] >> (i % 32) & 1 ? (i & 1 ? f.y : f.x) : 0.f;
                    if (i < cnt) {
                        if (c.out_f32) reinterpret_cast<float *>(c.y)[at + i * c.ys] = val;
                        else reinterpret_cast<__nv_bfloat16 *>(c.y)[at + i * c.ys] = __float2bfloat16_rn(val);
                    }
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, A * BT);
    if (tid == 0 && abort_flag) flag_status(GDN_DEVSTAT_TIMEOUT);
}

template <int BT, bool kBlock> gdn_status launch(const GroupedCall &c, int drop, cudaStream_t s) {
    using C = GnCfg<BT>;
    CUtensorMap mx, mw;
    if (!encode_tmap_rows(&mx, c, BT) || !encode_tmap_experts(&mw, c, 128)) return GDN_ERR_CUDA;
    auto kernel = grouped_narrow_kernel<BT, kBlock>;
    static SmemAllowed allowed;
    cudaError_t e = allowed.ask(kernel, C::kSmem);
    const int64_t nn = (c.n_out + 127) / 128;
    const int64_t tiles = (((int64_t)c.n_rows + BT - 1) / BT + (c.offsets ? std::min(c.n_experts, c.n_rows) : 0)) * nn;
    if (tiles >= (1ll << 31)) return GDN_ERR_UNSUPPORTED;
    if (e == cudaSuccess)
        e = launch_after(kernel, dim3((unsigned)std::min<int64_t>(tiles, sm_count())), dim3(kGnThreads), C::kSmem, s, mx,
                         mw, c, drop == kDropNone ? INT_MAX : drop & kDropAll ? 0 : 1);
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

}  // namespace

gdn_status launch_grouped_narrow(const GroupedCall &c, int tile_rows, int drop, cudaStream_t s) {
    switch (tile_rows) {
        case 16: return c.e4m3 ? launch<16, true>(c, drop, s) : launch<16, false>(c, drop, s);
        case 32: return c.e4m3 ? launch<32, true>(c, drop, s) : launch<32, false>(c, drop, s);
        case 64: return c.e4m3 ? launch<64, true>(c, drop, s) : launch<64, false>(c, drop, s);
        default: return c.e4m3 ? launch<128, true>(c, drop, s) : launch<128, false>(c, drop, s);
    }
}

}  // namespace gdn
