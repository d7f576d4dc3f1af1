// gdn_linear for many tokens: a persistent grid of CTA pairs, each pair on one
// tile of 256 tokens x BN channels at a time (tcgen05 cta_group::2, M = 256).
//
// A CTA of a pair loads its own 128 tokens and half of the tile's weight rows,
// so a pair reads each operand byte once from L2 and its tensor cores read
// (128 + BN) x 128 B of shared memory per 128 bytes of k where two single CTAs
// would read (128 + BN) x 128 B each for half the products.  The accumulator
// (BN fp32 columns) is doubled in tensor memory: the epilogue warps turn one
// tile into y while the next one's products run.
//
// Epilogue: a thread holds one token row and takes 128 bytes of y at a time
// (64 bf16 or 32 fp32 columns): scale, bias, activation, residual, one
// rounding, then into a 128-byte-swizzled staging row (4 KB per warp, three of
// them), from which one TMA store writes 32 rows; the residual comes through
// the same staging row by a TMA load, requested one slice ahead.  A y or residual that TMA cannot address
// (rows off 16-byte boundaries) goes through the staging row to plain accesses
// of consecutive elements.
#include <algorithm>

#include "linear.cuh"

namespace gdn {

using namespace tc;

GDN_DECLARE_STATUS_WORD(g_status_linear_wide)
GDN_STATUS_READER(read_status_linear_wide, g_status_linear_wide)

namespace {

constexpr int kTokTile = 256, kTokHalf = 128, kStagesWide = 5, kEpiWarps = 4;
constexpr int kStagingBufs = 3;
constexpr int kRaster = 8;     // token tiles of one raster group (below)

template <int BN> struct WideCfg {
    static constexpr uint32_t kA = kTokHalf * 128, kB = BN / 2 * 128, kStage = kA + kB;
    static constexpr uint32_t kStaging = kEpiWarps * kStagingBufs * 4096;
    static constexpr uint32_t kSmem = kStagesWide * kStage + kStaging + 1024;
    static constexpr uint32_t kCols = 2 * BN;
};

// Tiled load into this CTA's shared memory, its bytes counted on a barrier of
// either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar,
                                                 int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the products issued
// so far by this thread are done.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// Waits until at most N of this thread's committed stores have not read their source.
template <int N> __device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
template <bool kE4m3>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
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

// Tile order: groups of kRaster token tiles; within a group the token tile
// runs fastest, then the channel tile.  The tiles in flight at one time then
// share about as many token rows as weight rows.
struct WideTiles {
    int nt, nn;      // token and channel tiles
    __device__ __forceinline__ void at(int tile, int &t, int &n) const {
        const int per = kRaster * nn, g = tile / per, r = tile - g * per;
        const int rows = min(kRaster, nt - g * kRaster);
        n = r / rows;
        t = g * kRaster + (r - n * rows);
    }
};

template <typename O> __device__ __forceinline__ void add_chunk(float *v, const uint4 &q);
template <> __device__ __forceinline__ void add_chunk<__nv_bfloat16>(float *v, const uint4 &q) {
    float f[8];
    Vec16<__nv_bfloat16>::unpack(q, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += f[i];
}
template <> __device__ __forceinline__ void add_chunk<float>(float *v, const uint4 &q) {
    float f[4];
    Vec16<float>::unpack(q, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += f[i];
}

// 32 rows of 128 bytes between a staging buffer and memory that TMA cannot
// address, element by element: a warp's lanes take consecutive elements, and
// 16 rows are in flight at a time.
template <typename O, bool kLoad>
__device__ __forceinline__ void plain_rows(uint8_t *buf, O *p, int64_t stride, int t0, int n0,
                                           int n_tokens, int n_out, int lane) {
    constexpr int COLS = 128 / sizeof(O), PART = COLS / 32, ROWS = 16;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += ROWS) {
        if (t0 + r0 >= n_tokens) break;
        O v[ROWS][PART];
#pragma unroll
        for (int pass = 0; pass < 2; ++pass)
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int c = 0; c < PART; ++c) {
                    const int col = c * 32 + lane, t = t0 + r0 + r;
                    const bool on = t < n_tokens && n0 + col < n_out;
                    const uint32_t off = col * sizeof(O);
                    O *in_buf = reinterpret_cast<O *>(
                        buf + (r0 + r) * 128 + (((off >> 4) ^ ((r0 + r) & 7)) << 4) + (off & 15));
                    O *in_mem = p + t * stride + n0 + col;
                    if (pass == 0) {
                        if (on) v[r][c] = kLoad ? *in_mem : *in_buf;
                    } else if (on) {
                        *(kLoad ? in_buf : in_mem) = v[r][c];
                    }
                }
    }
}

struct WideFlags {
    bool y_tma, res_tma;
};

// One staging row's worth of columns of a tile: accumulator -> y values in the
// staging row.  cols: the columns' scales, then their biases, in shared memory.
template <int kAct, typename O, int BN>
__device__ __forceinline__ void wide_slice(uint32_t taddr, const float *cols, float sx, bool has_res,
                                           uint8_t *row, int r7) {
    constexpr int COLS = 128 / sizeof(O), PER = 16 / sizeof(O);
#pragma unroll
    for (int h = 0; h < COLS / 32; ++h) {
        uint32_t r[32];
        tmem_ld32(taddr + h * 32, r);
#pragma unroll
        for (int c = 0; c < 32 / PER; ++c) {
            float v[PER];
            const int j0 = h * 32 + c * PER;
#pragma unroll
            for (int i = 0; i < PER; i += 4) {
                const float4 s = *reinterpret_cast<const float4 *>(cols + j0 + i);
                const float4 b = *reinterpret_cast<const float4 *>(cols + BN + j0 + i);
                const uint32_t *a = r + c * PER + i;
                v[i] = linear_act<kAct>(fmaf(__uint_as_float(a[0]), sx * s.x, b.x));
                v[i + 1] = linear_act<kAct>(fmaf(__uint_as_float(a[1]), sx * s.y, b.y));
                v[i + 2] = linear_act<kAct>(fmaf(__uint_as_float(a[2]), sx * s.z, b.z));
                v[i + 3] = linear_act<kAct>(fmaf(__uint_as_float(a[3]), sx * s.w, b.w));
            }
            uint4 *chunk = reinterpret_cast<uint4 *>(row + (((j0 / PER) ^ r7) << 4));
            if (has_res) add_chunk<O>(v, *chunk);
            Vec16<O>::store(reinterpret_cast<O *>(chunk), v);
        }
    }
}

template <int BN, bool kE4m3, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(256, 1)
linear_wide_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                   const __grid_constant__ CUtensorMap my, const __grid_constant__ CUtensorMap mres,
                   const __grid_constant__ LinearEpi ep, int n_in, WideTiles tiles, WideFlags flags) {
    using C = WideCfg<BN>;
    constexpr int S = kStagesWide, COLS = 128 / sizeof(O), SLICES = BN / COLS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[S], empty[S], acc_full[2], acc_empty[2], res_full[kEpiWarps][kStagingBufs], drained;
    __shared__ __align__(16) float cols[2][2 * BN];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cta_rank();
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int kElems = kE4m3 ? 128 : 64;                 // k per block of 128 bytes
    const int nk = (n_in + kElems - 1) / kElems;
    const int n_tiles = tiles.nt * tiles.nn, pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&mx);
        prefetch_tensormap(&mw);
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kEpiWarps);
        }
        for (int w = 0; w < kEpiWarps; ++w)
            for (int b = 0; b < kStagingBufs; ++b) mbar_init(&res_full[w][b], 1);
        mbar_init(&drained, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_base)),
                     "r"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync_all();        // both CTAs' barriers and tensor memory are ready
    tc_fence_after();
    griddep_wait();            // launched behind the kernel that writes x: nothing is read before it
    volatile int *abort = &abort_flag;

    if (warp == 0 && lane == 0) {
        // Loads: this CTA's half of both operands, counted on the leader's barrier.
        int i = 0;
        bool ok = true;
        for (int tile = pair; tile < n_tiles && ok; tile += pairs) {
            int tt, tn;
            tiles.at(tile, tt, tn);
            const int t0 = tt * kTokTile + (int)rank * kTokHalf, n0 = tn * BN + (int)rank * (BN / 2);
            for (int k = 0; k < nk; ++k, ++i) {
                const int s = i % S;
                if (i >= S && !mbar_wait(&empty[s], ((i / S) - 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                uint8_t *st = smem + s * C::kStage;
                const uint32_t bar = peer_smem(smem_u32(&full[s]), 0);
                if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);
                tma_load_2d_pair(st, &mx, bar, k * kElems, t0);
                tma_load_2d_pair(st + C::kA, &mw, bar, k * kElems, n0);
            }
        }
        if (!ok || *abort) {
            // Given up: the copies in flight land before the CTA ends.  The leader
            // waits on the barriers that count them; the peer, which has none of
            // its own, waits far longer (10 ms) than a copy takes.
            if (rank == 0) {
                for (int j = i > S ? i - S : 0; j < i; ++j) mbar_drain(&full[j % S], (j / S) & 1);
            } else {
                const uint64_t t = globaltimer_ns();
                while (globaltimer_ns() - t < 10000000ull) {
                }
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        constexpr uint32_t idesc = kE4m3 ? idesc_e4m3(256, BN) : idesc_bf16(256, BN);
        int i = 0, u = 0;
        bool ok = true;
        for (int tile = pair; tile < n_tiles && ok; tile += pairs, ++u) {
            const int b = u & 1;
            if (u >= 2 && !mbar_wait(&acc_empty[b], ((u >> 1) - 1) & 1, abort)) break;
            tc_fence_after();
            const uint32_t d = tmem_base + b * BN;
            for (int k = 0; k < nk; ++k, ++i) {
                const int s = i % S;
                if (!mbar_wait(&full[s], (i / S) & 1, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = smem_u32(smem + s * C::kStage);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    mma_pair<kE4m3>(d, sdesc_sw128(st + q * 32, 0, 1024),
                                    sdesc_sw128(st + C::kA + q * 32, 0, 1024), idesc, k > 0 || q > 0);
                mma_commit_pair(&empty[s]);
            }
            if (ok) mma_commit_pair(&acc_full[b]);
        }
        mma_commit_pair(&drained);      // every product issued is done before the pair ends
        mbar_drain(&drained, 0);
    } else if (warp >= 4) {
        const int q = warp & 3, etid = tid - 128;
        uint8_t *staging = smem + S * C::kStage + q * (kStagingBufs * 4096);
        uint64_t *rbar = res_full[q];
        const bool has_res = ep.res != nullptr, res_tma = has_res && flags.res_tma;
        int u = 0, sl = 0;              // sl: slices so far; a slice's staging buffer is sl % 3
        int asked = 0, seen = 0;        // residual slices requested and waited for
        // Requests a slice's residual into its buffer, which the store of three
        // slices before has read (the bulk_wait_read before each call).
        auto ask = [&](int slice, int nc, int t0) {
            if (lane == 0) {
                uint64_t *bar = &rbar[slice % kStagingBufs];
                mbar_arrive_expect_tx(bar, 4096);
                tma_load_2d(staging + (slice % kStagingBufs) * 4096, &mres, bar, nc, t0);
            }
            ++asked;
        };
        for (int tile = pair; tile < n_tiles; tile += pairs, ++u) {
            const int b = u & 1;
            int tt, tn;
            tiles.at(tile, tt, tn);
            const int t0 = tt * kTokTile + (int)rank * kTokHalf + q * 32, n0 = tn * BN;
            const int t = t0 + lane;
            float *cb = cols[b];
            for (int c = etid; c < BN; c += 128) {
                const bool on = n0 + c < ep.n_out;
                cb[c] = on && ep.sw ? ep.sw[n0 + c] : 1.0f;
                cb[BN + c] = on && ep.bias ? ep.bias[n0 + c] : 0.0f;
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const float sx = ep.sx && t < ep.n_tokens ? ep.sx[t] : 1.0f;
            if (lane == 0) bulk_wait_read<2>();
            if (res_tma) ask(sl, n0, t0);
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[b], (u >> 1) & 1, abort))) break;
            tc_fence_after();
#pragma unroll 1
            for (int s = 0; s < SLICES; ++s, ++sl) {
                uint8_t *buf = staging + (sl % kStagingBufs) * 4096;
                uint8_t *my_row = buf + lane * 128;
                const int nc = n0 + s * COLS;
                // free the next slice's buffer: the store of two slices ago has read it
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
                if (has_res) {
                    if (res_tma) {
                        if (s + 1 < SLICES) ask(sl + 1, nc + COLS, t0);
                        if (__all_sync(0xffffffffu, mbar_wait(&rbar[sl % kStagingBufs], (sl / kStagingBufs) & 1, abort)))
                            ++seen;
                    } else {
                        plain_rows<O, true>(buf, reinterpret_cast<O *>(const_cast<void *>(ep.res)), ep.rs,
                                            t0, nc, ep.n_tokens, ep.n_out, lane);
                        __syncwarp();
                    }
                }
                const uint32_t ta = tmem_addr(tmem_base, q * 32, b * BN + s * COLS);
                const float *cs = cb + s * COLS;
                if (ep.act == GDN_ACT_SILU)
                    wide_slice<GDN_ACT_SILU, O, BN>(ta, cs, sx, has_res, my_row, lane & 7);
                else if (ep.act == GDN_ACT_GELU)
                    wide_slice<GDN_ACT_GELU, O, BN>(ta, cs, sx, has_res, my_row, lane & 7);
                else
                    wide_slice<GDN_ACT_NONE, O, BN>(ta, cs, sx, has_res, my_row, lane & 7);
                if (s == SLICES - 1) {   // the accumulator is read out
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(peer_smem(smem_u32(&acc_empty[b]), 0));
                }
                if (flags.y_tma) {
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (nc < ep.n_out && t0 < ep.n_tokens) tma_store_2d(&my, buf, nc, t0);
                        bulk_commit();
                    }
                } else {
                    __syncwarp();
                    plain_rows<O, false>(buf, reinterpret_cast<O *>(ep.y), ep.ys, t0, nc, ep.n_tokens,
                                         ep.n_out, lane);
                    // the next user of the buffer may be a copy of the async proxy
                    fence_async_smem();
                    __syncwarp();
                }
            }
        }
        tc_fence_before();
        if (lane == 0) {
            // given up: residual copies in flight land before the CTA ends
            for (int j = seen; j < asked; ++j) mbar_drain(&rbar[j % kStagingBufs], (j / kStagingBufs) & 1);
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
        __syncwarp();
    }
    __syncwarp();
    cluster_sync_all();        // neither CTA ends while the other may reach its memory
    tc_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(C::kCols)
                     : "memory");
    if (tid == 0 && abort_flag) flag_status(GDN_DEVSTAT_TIMEOUT);
}

template <typename O> constexpr CUtensorMapDataType tmap_type() {
    return sizeof(O) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// Whether TMA can address these rows: 16-byte aligned, the stride too.
bool tma_rows(const void *p, int64_t stride, size_t elem) {
    return (uintptr_t)p % 16 == 0 && (stride * (int64_t)elem) % 16 == 0 && stride < (1ll << 36);
}

template <int BN, bool kE4m3, typename O> gdn_status launch_wide(const LinearCall &c) {
    using C = WideCfg<BN>;
    const LinearEpi &e = c.e;
    CUtensorMap mx, mw, my = {}, mres = {};
    WideFlags f = {tma_rows(e.y, e.ys, sizeof(O)), e.res && tma_rows(e.res, e.rs, sizeof(O))};
    if (!encode_tmap_operand(&mx, c.x, c.n_in, e.n_tokens, c.xs, kTokHalf, kE4m3) ||
        !encode_tmap_operand(&mw, c.w, c.n_in, e.n_out, c.ws, BN / 2, kE4m3))
        return GDN_ERR_CUDA;
    constexpr uint32_t box = 128 / sizeof(O);
    if (f.y_tma && !encode_tmap_2d(&my, tmap_type<O>(), e.y, e.n_out, e.n_tokens, e.ys * sizeof(O), box, 32, true))
        return GDN_ERR_CUDA;
    if (f.res_tma &&
        !encode_tmap_2d(&mres, tmap_type<O>(), e.res, e.n_out, e.n_tokens, e.rs * sizeof(O), box, 32, true))
        return GDN_ERR_CUDA;
    auto kernel = linear_wide_kernel<BN, kE4m3, O>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    const WideTiles tiles = {(e.n_tokens + kTokTile - 1) / kTokTile, (e.n_out + BN - 1) / BN};
    const int64_t n = (int64_t)tiles.nt * tiles.nn;
    const int pairs = (int)std::min<int64_t>(n, std::max(1, sm_count() / 2));
    if (err == cudaSuccess)
        err = launch_after(kernel, dim3(2 * pairs), dim3(256), C::kSmem, c.stream, mx, mw, my, mres, e,
                           c.n_in, tiles, f);
    if (err != cudaSuccess) {
        set_last_cuda_error(err);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

}  // namespace

gdn_status launch_linear_wide(const LinearCall &c, bool e4m3) {
    if (e4m3) return c.e.out_f32 ? launch_wide<256, true, float>(c) : launch_wide<256, true, __nv_bfloat16>(c);
    return c.e.out_f32 ? launch_wide<256, false, float>(c) : launch_wide<256, false, __nv_bfloat16>(c);
}

}  // namespace gdn
