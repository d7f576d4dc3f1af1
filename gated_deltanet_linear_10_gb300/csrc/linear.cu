// gdn_linear: the matrix product of the block's projections with scales, bias,
// activation and residual in its epilogue.
//
// The products run on tcgen05 with both operands loaded by TMA in the 128-byte
// swizzle and the accumulator in tensor memory; k is cut into blocks of 128
// bytes (64 bf16 or 128 e4m3), which a ring of shared-memory stages holds.
// The weights' rows are the 128 lanes of the accumulator and the tokens its
// columns, so that a single token costs one narrow product per weight tile and
// the tile follows the number of tokens.
#include <limits.h>

#include <algorithm>

#include "grouped.cuh"
#include "linear.cuh"

namespace gdn {

using namespace tc;

GDN_DECLARE_STATUS_WORD(g_status_linear)
GDN_STATUS_READER(read_status_linear, g_status_linear)

// Test control of the failure path (gdn_debug_set_wait_limit).
static std::atomic<int> g_linear_drop{kDropNone};
cudaError_t set_linear_failure(uint64_t limit_ns, int drop, cudaStream_t s) {
    g_linear_drop.store(drop, std::memory_order_relaxed);
    cudaError_t e = cudaMemcpyToSymbolAsync(tc::g_wait_limit_ns, &limit_ns, sizeof(limit_ns), 0,
                                            cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = set_linear_wide_limit(limit_ns, s);
    if (e == cudaSuccess) e = set_grouped_narrow_limit(limit_ns, s);
    return e != cudaSuccess ? e : set_grouped_wide_limit(limit_ns, s);
}
int linear_drop() { return g_linear_drop.load(std::memory_order_relaxed); }

bool encode_tmap_operand(CUtensorMap *map, const void *base, int64_t cols, int64_t rows,
                         int64_t row_stride_elems, uint32_t box_rows, bool e4m3) {
    const int elem = e4m3 ? 1 : 2;
    if (rows == 1) row_stride_elems = (cols + 15) / 16 * 16;   // never stepped over
    return encode_tmap_2d(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                          base, cols, rows, row_stride_elems * elem, 128 / elem, box_rows, true);
}

// BT: tokens per tile (the product's N).  A cluster of `splits` CTAs per
// 128 x BT tile, each on its part of k.
template <int BT> struct NarrowCfg {
    static constexpr uint32_t kW = 128 * 128, kX = BT * 128, kStage = kW + kX;
    static constexpr int kStages = BT >= 128 ? 5 : BT >= 64 ? 3 : 4;
    static constexpr uint32_t kSums = BT * 512;          // BT tokens x 128 channels, fp32
    static constexpr uint32_t kSmem = kStages * kStage + kSums;
    static_assert(kStages * kStage >= kSums, "a CTA's own sums fit its stages");
};
constexpr int kNarrowThreads = 256;

// Copy of this CTA's shared memory into another CTA's of the cluster, its bytes
// counted on a barrier of that CTA (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_send(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "r"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Channels of a thread, in pairs i = 0 .. 3: 8 in a row where rows are vectors of
// 8, else one pair of every 32, so that a token's 16 threads access neighbours.
__device__ __forceinline__ int narrow_channel(bool vec, int g, int i) { return vec ? g * 8 + 2 * i : g * 2 + 32 * i; }

// The residual of a thread's channels n + narrow_channel of token t, as loaded: a
// vector (bf16: the first 16 bytes), or a channel a word.
struct Res8 {
    uint4 q[2];
    template <typename O> __device__ __forceinline__ void load_as(const LinearEpi &ep, bool vec, int t, int n, int g) {
        const O *p = reinterpret_cast<const O *>(ep.res) + t * ep.rs + n;
        if (vec) {
            const uint4 *v = reinterpret_cast<const uint4 *>(p + g * 8);
            q[0] = v[0];
            if (sizeof(O) == 4) q[1] = v[1];
        } else {
            uint32_t *w = reinterpret_cast<uint32_t *>(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = narrow_channel(false, g, i / 2) + i % 2;
                if (n + c >= ep.n_out) continue;
                if constexpr (sizeof(O) == 4) w[i] = reinterpret_cast<const uint32_t *>(p)[c];
                else w[i] = reinterpret_cast<const uint16_t *>(p)[c];
            }
        }
    }
    __device__ __forceinline__ void load(const LinearEpi &ep, bool vec, int t, int n, int g) {
        if (ep.out_f32) load_as<float>(ep, vec, t, n, g);
        else load_as<__nv_bfloat16>(ep, vec, t, n, g);
    }
};

// A thread's channels of tokens t[0], t[1] (t[u] < 0: none) out: residual, one
// rounding, store.  y may be residual: it is read before it is written.
template <typename O>
__device__ __forceinline__ void narrow_out(F2 (&v)[2][4], const LinearEpi &ep, const int (&t)[2], int n, int g,
                                           bool vec, const Res8 (&r)[2]) {
    O *y = reinterpret_cast<O *>(ep.y) + n;
    if (vec) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (t[u] < 0) continue;
            if (ep.res) {
                RawVec<O, 8> raw;
                F2 q[4];
                raw.r[0] = r[u].q[0];
                if constexpr (sizeof(O) == 4) raw.r[1] = r[u].q[1];
                raw.pairs(q);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[u][i] = f2_add(v[u][i], q[i]);
            }
            float f[8];
            unpair<8>(v[u], f);
            store_row<8>(y + g * 8 + t[u] * ep.ys, f);
        }
    } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (t[u] < 0) continue;
            const uint32_t *w = reinterpret_cast<const uint32_t *>(r[u].q);
            float f[8];
            unpair<8>(v[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = narrow_channel(false, g, i / 2) + i % 2;
                if (n + c >= ep.n_out) continue;
                if (ep.res) f[i] += __uint_as_float(sizeof(O) == 4 ? w[i] : w[i] << 16);
                Io<O>::store(y + t[u] * ep.ys + c, f[i]);
            }
        }
    }
}

template <int kAct> __device__ __forceinline__ void narrow_act(F2 (&v)[2][4]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i / 4][i % 4] = linear_act<kAct>(v[i / 4][i % 4]);
}

// grid (channel tiles * splits, token tiles); the `splits` CTAs of a tile are a
// cluster, CTA r of it on the k blocks [r nk / splits, (r + 1) nk / splits).
// Its sums go from tensor memory to its shared memory as rows of 128 channels.
// With splits > 1, CTA r collects the tokens [r BT / splits, (r + 1) BT / splits)
// of every CTA by bulk copies and adds them in the order of the CTAs, so the
// result has one order of sums; with one, it has them all.  Then 16 threads
// write a token's 128 channels.
//
// Where a wait has run out, the exchange takes place all the same, with whatever
// there is, so that every copy has a CTA that counts it; nothing is written to y.
// keep: k blocks of a CTA that are loaded, all of them but for tests of that path.
//
// What bounds it at 256 x 4096 x 2048 (8.8 us with the weights in L2, 10.2 with weights
// from HBM; at the memory's rate 3.1): 2,000 cycles to the
// first products, 5,500 to 6,500 of products (16 blocks, held by their copies: 256
// lines of 128 bytes at some 1.6 cycles each; the products alone would take 256
// cycles a block), 3,200 of exchange (48 KB a CTA, 1,500 of it latency), 3,500 to
// write the sums and the output.  One token (1 x 2048 x 8192, 6.9 to 7.2 us, from HBM
// 8.6; 4.9) waits for the weights.
// The code behind the products runs once per CTA, so it is kept short and
// rolled: unrolled over 32 tokens with its variants it took 3 to 20 us of
// instruction fetches and dependent loads at 256 tokens.
template <int BT, bool kE4m3>
__global__ void __launch_bounds__(kNarrowThreads)
linear_narrow_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                     const __grid_constant__ LinearEpi ep, int n_in, int splits, int keep) {
    using C = NarrowCfg<BT>;
    constexpr int S = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[S], empty[S], done, arrived;
    __shared__ float sxs[BT];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    // the warp's number by a shuffle, so that it is known to be one for the warp
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = splits > 1 ? (int)cta_rank() : 0;
    const int n0 = blockIdx.x / splits * 128, t0 = blockIdx.y * BT;
    constexpr int kElems = kE4m3 ? 128 : 64;                 // k per block of 128 bytes
    const int blocks = (n_in + kElems - 1) / kElems;
    const int k0 = (int)((int64_t)blocks * rank / splits);
    const int nk = (int)((int64_t)blocks * (rank + 1) / splits) - k0;
    const int nload = min(nk, keep);
    volatile int *abort = &abort_flag;
    const bool one = warp < 2 && elect_lane();
    auto load = [&](int i, int s) {
        uint8_t *st = smem + s * C::kStage;
        mbar_arrive_expect_tx(&full[s], C::kStage);
        tma_load_2d(st, &mw, &full[s], (k0 + i) * kElems, n0);
        tma_load_2d(st + C::kW, &mx, &full[s], (k0 + i) * kElems, t0);
    };

    if (warp == 0) {
        if (one) {
            prefetch_tensormap(&mx);
            prefetch_tensormap(&mw);
            for (int s = 0; s < S; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            mbar_init(&done, 1);
            mbar_init(&arrived, 1);
            abort_flag = (smem_u32(smem) & 1023u) != 0;   // the swizzle needs the alignment asked for above
            fence_mbar_init();
            fence_async_smem();
            griddep_wait();   // launched behind the kernel that writes x: nothing is read before it
            for (int i = 0; i < min(S, nload); ++i) load(i, i);
        }
        __syncwarp();
    }
    if (warp == 1) {
        griddep_wait();       // no tensor memory is held while an earlier kernel may still ask for its own
        tmem_alloc(&tmem_base, BT);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (splits > 1) cluster_arrive_relaxed();      // waited for before the first copy to another CTA
    griddep_wait();

    int issued = min(S, nload);                              // of warp 0
    if (warp == 0) {
        int s = 0;
        uint32_t phase = 0;
#pragma unroll 1
        for (; issued < nload; ++issued) {
            if (!mbar_wait_all(&empty[s], phase, abort)) break;
            if (one) load(issued, s);
            __syncwarp();
            if (++s == S) {
                s = 0;
                phase ^= 1;
            }
        }
        griddep_launch();   // what is launched behind this kernel may set itself up
    } else if (warp == 1) {
        constexpr uint32_t idesc = kE4m3 ? idesc_e4m3(128, BT) : idesc_bf16(128, BT);
        const uint64_t desc = sdesc_sw128(0, 0, 1024);
        // What a product is issued with is read from memory once and known to be one for
        // the warp, and the lane is elected on the spot: 64 cycles for 128 x 128 x 16, where
        // rereading the base and testing a kept flag took 140.
        const uint32_t base = smem_u32(smem) >> 4, sums = tmem_base;
        uint32_t phase = 0;
        int s = 0;
#pragma unroll 1
        for (int i = 0; i < nk; ++i) {
            if (!mbar_wait_all(&full[s], phase, abort)) break;
            tc_fence_after();
            if (elect_lane()) {
                const uint32_t st = base + s * (C::kStage >> 4);
                const uint64_t da = desc | st, db = desc | (st + (C::kW >> 4));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    linear_mma<kE4m3>(sums, da + 2 * k, db + 2 * k, idesc, i > 0 || k > 0);
                mma_commit(&empty[s]);
            }
            __syncwarp();
            if (++s == S) {
                s = 0;
                phase ^= 1;
            }
        }
        if (one) {
            mma_commit(&done);
            mbar_drain(&done, 0);
        }
    } else {
        for (int t = tid - 64; t < BT; t += kNarrowThreads - 64)
            sxs[t] = ep.sx && t0 + t < ep.n_tokens ? ep.sx[t0 + t] : 1.0f;
    }
    __syncwarp();

    const int per = BT / splits;                         // tokens that a CTA collects
    const int first = t0 + rank * per, cnt = min(per, ep.n_tokens - first);   // those it writes (cnt <= 0: none)
    float *own = reinterpret_cast<float *>(smem);        // where the operands were
    float *got = reinterpret_cast<float *>(smem + S * C::kStage);
    const int g = tid & 15;                              // this thread's channels below
    const bool vec = ep.vec8;
    F2 sw[4], bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = n0 + narrow_channel(vec, g, i);
        const bool on = n < ep.n_out, on1 = n + 1 < ep.n_out;
        sw[i] = f2(on && ep.sw ? ep.sw[n] : 1.0f, on1 && ep.sw ? ep.sw[n + 1] : 1.0f);
        bias[i] = f2(on && ep.bias ? ep.bias[n] : 0.0f, on1 && ep.bias ? ep.bias[n + 1] : 0.0f);
    }
    // the residual of two of its items ahead: the first two before the sums are there
    const bool any = !vec || n0 + g * 8 < ep.n_out;
    Res8 res[2];
    auto ask = [&](int i) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int tok = (i + u * kNarrowThreads) >> 4;
            if (ep.res && any && tok < cnt) res[u].load(ep, vec, first + tok, n0, g);
        }
    };
    ask(tid);
    if (warp >= 2 && warp < 6 && mbar_wait_all(&done, 0, abort)) {
        // accumulator lane 32 q + l is channel n0 + 32 q + l, its columns the tokens
        tc_fence_after();
        const int quad = warp & 3;
        float *col = own + quad * 32 + lane;
#pragma unroll 1
        for (int c = 0; c < BT && t0 + c < ep.n_tokens; c += 32) {
            uint32_t r[32];
            tmem_ld32(tmem_addr(tmem_base, quad * 32, c), r);
#pragma unroll
            for (int j = 0; j < 32; ++j) col[(c + j) * 128] = __uint_as_float(r[j]);
        }
        tc_fence_before();
        fence_async_smem();
    }
    if (splits > 1) {
        __syncwarp();
        cluster_wait();                                  // every CTA of the cluster has its barriers
    }
    __syncthreads();
    if (splits > 1) {
        if (tid == 0) {
            if (cnt > 0) mbar_arrive_expect_tx(&arrived, (splits - 1) * cnt * 512);
            for (int o = 1; o < splits; ++o) {           // each starts with another one
                const int to = (rank + o) & (splits - 1);
                const int tokens = min(per, ep.n_tokens - t0 - to * per);
                if (tokens > 0)
                    bulk_send(peer_smem(smem_u32(got + rank * per * 128), to), smem_u32(own + to * per * 128),
                              tokens * 512, peer_smem(smem_u32(&arrived), to));
            }
        }
        if (cnt > 0 && !mbar_wait(&arrived, 0, abort)) mbar_drain(&arrived, 0);
        // This CTA has what was sent to it, or tells the others that it has given up: then
        // none ends before all copies have had their time.
        if (tid == 0 && *abort) {
            for (int o = 0; o < splits; ++o) set_peer_flag(&abort_flag, o);
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
        }
        __syncwarp();
        cluster_arrive_relaxed();
    }
    if (!*abort) {
#pragma unroll 1
        for (int i = tid; i < cnt * 16; i += 2 * kNarrowThreads) {
            const int tok[2] = {i >> 4, (i + kNarrowThreads) >> 4};
            const int tok1 = min(tok[1], cnt - 1);
            F2 v[2][4] = {};
#pragma unroll 1
            for (int r = 0; r < splits; ++r) {
                const float *p = (r == rank ? own : got) + r * per * 128;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float *q = p + (u ? tok1 : tok[0]) * 128;
                    if (vec) {
                        const ulonglong2 *q4 = reinterpret_cast<const ulonglong2 *>(q + g * 8);
                        const ulonglong2 a = q4[0], b = q4[1];
                        v[u][0] = f2_add(v[u][0], a.x);
                        v[u][1] = f2_add(v[u][1], a.y);
                        v[u][2] = f2_add(v[u][2], b.x);
                        v[u][3] = f2_add(v[u][3], b.y);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[u][i] = f2_add(v[u][i], *reinterpret_cast<const F2 *>(q + narrow_channel(false, g, i)));
                    }
                }
            }
            const Res8 cur[2] = {res[0], res[1]};
            ask(i + 2 * kNarrowThreads);
            const float sx0 = sxs[rank * per + tok[0]], sx1 = sxs[rank * per + tok1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[0][j] = f2_fma(v[0][j], f2_mul(f2(sx0, sx0), sw[j]), bias[j]);
                v[1][j] = f2_fma(v[1][j], f2_mul(f2(sx1, sx1), sw[j]), bias[j]);
            }
            if (ep.act == GDN_ACT_SILU) narrow_act<GDN_ACT_SILU>(v);
            else if (ep.act == GDN_ACT_GELU) narrow_act<GDN_ACT_GELU>(v);
            if (any) {
                const int t[2] = {first + tok[0], tok[1] < cnt ? first + tok[1] : -1};
                if (ep.out_f32) narrow_out<float>(v, ep, t, n0, g, vec, cur);
                else narrow_out<__nv_bfloat16>(v, ep, t, n0, g, vec, cur);
            }
        }
    }
    __syncwarp();
    if (splits > 1) cluster_wait();                      // and the others what it sent
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, BT);
    if (tid == 0 && abort_flag) {
        flag_status(GDN_DEVSTAT_TIMEOUT);
        // the copies in flight land before the CTA ends
        for (int j = max(0, issued - S); j < issued; ++j) mbar_drain(&full[j % S], (j / S) & 1);
        if (splits > 1) let_copies_land();
    }
}

// How a product of these sizes is cut over narrow tiles, and what that takes in
// SM cycles by the estimate below.
struct NarrowPlan {
    int nn, nt, splits;
    int64_t cycles;
};

// Fitted, with the weights in L2, to 1 to 2000 tokens on products of 256 x 2048 to 8192 x 1024, with k in one,
// two, four and eight, bf16 and e4m3: what this estimate picks takes 0.5 % longer
// than the best of them in the mean, and 7 % at the worst (on sizes it was not fitted
// to, 17 % in one of 264).  A k block of 128 tokens takes 425 cycles, its copies from
// L2, and 800 where rows are off the memory's lines (128 x 2056 x 8192, k whole: 16.2
// us, on lines 12.9); what goes before and after the loop grows with the tokens, and
// with the CTAs that start at once.  Every cluster that the device cannot hold at once
// waits for a whole one.
template <int BT, bool kE4m3> static cudaError_t plan_narrow(const LinearCall &c, NarrowPlan &best) {
    using C = NarrowCfg<BT>;
    static ClustersHeld held[4];
    auto kernel = linear_narrow_kernel<BT, kE4m3>;
    const int nn = (c.e.n_out + 127) / 128, nt = (c.e.n_tokens + BT - 1) / BT;
    const int blocks = (c.n_in + (kE4m3 ? 127 : 63)) / (kE4m3 ? 128 : 64);
    best.cycles = INT64_MAX;
    for (int i = 0; i < 4 && (i == 0 || blocks >= 2 << i); ++i) {   // at least two blocks for a CTA
        int fit = 0;
        const cudaError_t e = held[i].ask(kernel, 1 << i, kNarrowThreads, C::kSmem, fit);
        if (e != cudaSuccess) return e;
        if (fit <= 0) continue;
        const int block = c.lines() ? (BT == 128 ? 425 : 300) : BT == 128 ? 800 : BT == 64 ? 530 : 360;
        constexpr int kEnds = BT == 128 ? 8700 : 5000;
        constexpr int kExchange[4] = {0, 300, 300, 900}, kCtaCycles = 17;
        const int64_t tiles = (int64_t)nn * nt, waves = (tiles + fit - 1) / fit;
        const int64_t cycles = waves * (kEnds + kExchange[i] + kCtaCycles * (std::min<int64_t>(tiles, fit) << i) +
                                        ((blocks + (1 << i) - 1) >> i) * block);
        if (cycles < best.cycles) best = {nn, nt, 1 << i, cycles};
    }
    return cudaSuccess;
}

template <int BT, bool kE4m3>
static gdn_status launch_narrow(const LinearCall &c, const NarrowPlan &plan) {
    using C = NarrowCfg<BT>;
    CUtensorMap mx, mw;
    if (!encode_tmap_operand(&mx, c.x, c.n_in, c.e.n_tokens, c.xs, BT, kE4m3) ||
        !encode_tmap_operand(&mw, c.w, c.n_in, c.e.n_out, c.ws, 128, kE4m3))
        return GDN_ERR_CUDA;
    const cudaError_t e = launch_after_cluster(linear_narrow_kernel<BT, kE4m3>, plan.splits,
                                               dim3(plan.nn * plan.splits, plan.nt), dim3(kNarrowThreads),
                                               C::kSmem, c.stream, mx, mw, c.e, c.n_in, plan.splits,
                                               c.drop == kDropNone ? INT_MAX : c.drop & kDropAll ? 0 : 1);
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

// The narrow tiles for up to 128 tokens; beyond, whichever estimate is shorter
// (narrow and wide measured, bf16: 256 x 4096 x 2048 9.0 and 14.7 us, 512 x 4096 x
// 2048 12.5 and 16.0, 512 x 2048 x 8192 24.4 and 16.7, 640 x 2048 x 2048 10.5 and
// 10.4, 256 x 8192 x 1024 11.7 and 25.6; e4m3: 256 x 2048 x 8192 8.6 and 8.1).
template <bool kE4m3> static gdn_status launch_linear(const LinearCall &c) {
    const int t = c.e.n_tokens;
    NarrowPlan plan = {};
    cudaError_t e = t <= 32   ? plan_narrow<32, kE4m3>(c, plan)
                    : t <= 64 ? plan_narrow<64, kE4m3>(c, plan)
                              : plan_narrow<128, kE4m3>(c, plan);
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_CUDA;
    }
    if (plan.nt > 65535) plan.cycles = INT64_MAX;      // token tiles are a grid dimension
    if (t > 128) {
        WidePlan wide;
        if (plan_linear_wide(c, wide) < plan.cycles) return launch_linear_wide(c, wide);
    }
    if (plan.cycles == INT64_MAX) return GDN_ERR_UNSUPPORTED;
    if (t <= 32) return launch_narrow<32, kE4m3>(c, plan);
    if (t <= 64) return launch_narrow<64, kE4m3>(c, plan);
    return launch_narrow<128, kE4m3>(c, plan);
}

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_linear(const void *x, int64_t x_row_stride, const float *x_scale,
                                 const void *w, int64_t w_row_stride, const float *w_scale,
                                 const float *bias, const void *residual,
                                 int64_t residual_row_stride, int64_t n_tokens, int32_t n_in,
                                 int32_t n_out, int32_t act, void *y, int64_t y_row_stride,
                                 int32_t dtype, int32_t y_dtype, void *stream) {
    GDN_REQUIRE(dtype == GDN_F32 || dtype == GDN_BF16 || dtype == GDN_E4M3, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(y_dtype == GDN_F32 || y_dtype == GDN_BF16, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(dtype != GDN_F32, GDN_ERR_UNSUPPORTED);
    GDN_REQUIRE(act >= GDN_ACT_NONE && act <= GDN_ACT_GELU, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_tokens >= 0 && n_in > 0 && n_out > 0, GDN_ERR_INVALID_ARG);
    // token tiles of the wide kernel; a tile's sum over k (0.2 s at 2^24, with operands from
    // HBM) stays far below the second that the waits for it allow
    GDN_REQUIRE(n_tokens <= 65535 * 256 && n_out <= (1 << 30) && n_in <= (1 << 24), GDN_ERR_UNSUPPORTED);
    if (n_tokens == 0) return GDN_OK;
    GDN_REQUIRE(x && w && y && y != x && y != w, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(x_row_stride >= n_in && w_row_stride >= n_in && y_row_stride >= n_out &&
                    (!residual || residual_row_stride >= n_out),
                GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(y != residual || n_tokens == 1 || y_row_stride == residual_row_stride, GDN_ERR_INVALID_ARG);
    // the operands' rows start on 16-byte boundaries (TMA); a single row has no stride
    const int64_t per = dtype == GDN_E4M3 ? 16 : 8;
    GDN_REQUIRE((uintptr_t)x % 16 == 0 && (uintptr_t)w % 16 == 0 &&
                    (n_tokens == 1 || x_row_stride % per == 0) && (n_out == 1 || w_row_stride % per == 0),
                GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(x_row_stride < (1ll << 36) && w_row_stride < (1ll << 36) && y_row_stride < (1ll << 36) &&
                    residual_row_stride < (1ll << 36),
                GDN_ERR_UNSUPPORTED);
    const uintptr_t ye = y_dtype == GDN_F32 ? 4 : 2;
    GDN_REQUIRE((uintptr_t)y % ye == 0 && (uintptr_t)residual % ye == 0 && (uintptr_t)x_scale % 4 == 0 &&
                    (uintptr_t)w_scale % 4 == 0 && (uintptr_t)bias % 4 == 0,
                GDN_ERR_INVALID_ARG);
    LinearCall c;
    c.x = x;
    c.w = w;
    c.xs = x_row_stride;
    c.ws = w_row_stride;
    c.n_in = n_in;
    c.e4m3 = dtype == GDN_E4M3;
    c.stream = (cudaStream_t)stream;
    c.drop = g_linear_drop.load(std::memory_order_relaxed);
    c.e = {x_scale, w_scale, bias, residual, residual_row_stride, y, y_row_stride,
           (int)n_tokens, n_out, act, y_dtype == GDN_F32, false};
    // 8 channels at a time: 16 bytes of bf16, 32 of fp32
    c.e.vec8 = n_out % 8 == 0 && (uintptr_t)y % 16 == 0 && y_row_stride * (int64_t)ye % 16 == 0 &&
               (!residual || ((uintptr_t)residual % 16 == 0 && residual_row_stride * (int64_t)ye % 16 == 0));
    return dtype == GDN_E4M3 ? launch_linear<true>(c) : launch_linear<false>(c);
}
