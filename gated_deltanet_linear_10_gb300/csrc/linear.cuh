// The matrix product with its epilogue (internal header):
//   y[t][n] = act(sx[t] sw[n] sum_k x[t][k] w[n][k] + bias[n]) + residual[t][n]
#pragma once

#include <algorithm>
#include <atomic>

#include "quant.cuh"
#include "tc.cuh"

namespace gdn {

// The epilogue's inputs and the output; null pointers leave a part out.
struct LinearEpi {
    const float *sx, *sw, *bias;
    const void *res;
    int64_t rs;
    void *y;
    int64_t ys;
    int n_tokens, n_out, act;
    bool out_f32;
    bool vec8;            // rows of y and residual on 16-byte boundaries
};

// The activations run beside the products and take issue slots from the warps
// that feed them, so they are kept short.

// Two values at a time, with one reciprocal for both: 1 / a = b / (a b), the
// factors at most 2^63, so that their product stays finite.
__device__ __forceinline__ F2 rcp_pair(float a, float b) {
    const float r = rcp_approx(a * b);
    return f2_mul(f2(r, r), f2(b, a));
}

// v / (1 + e^-v).  Below -43.6 (e^-v = 2^63) it stays at the value there, -5e-18.
// A NaN stays out of the factors, which the other value shares.
__device__ __forceinline__ F2 silu_short(float a, float b) {
    constexpr float kLeast = -43.6f;
    return f2_mul(f2(max_nan(a, kLeast), max_nan(b, kLeast)),
                  rcp_pair(1.0f + ex2_approx(-kLog2e * fmaxf(a, kLeast)), 1.0f + ex2_approx(-kLog2e * fmaxf(b, kLeast))));
}

// GELU(v) = v Phi(v) by erfc(x) / 2 = t P(t) exp(-x^2), t = 1 / (1 + p x), at x =
// |v| / sqrt(2) >= 0 (the form of Abramowitz and Stegun, Handbook of Mathematical
// Functions, 7.1.26).  P is a fit of its own, of degree 7, to the least largest
// relative error over x in [0, 9.6] (least squares with Lawson's weights at 4000
// Chebyshev points; p = 0.58 gives the least, 2.7e-7), so that the small values below
// zero keep their digits too: with the roundings the result's relative error is at
// most 2^-19 (1 + v^2 / 16).  The handbook's own five terms hold an absolute 1.5e-7,
// 4e-3 of GELU(-6), and take 2 to 3 % less time where the epilogue bounds a call (14261 x
// 692 x 909 e4m3: 35.9 us, with these eight 36.9; 20668 x 2048 x 8192: the same).
// Values below 2^-126 become 0 (v < -13.1).
__device__ __forceinline__ F2 gelu_short(float a, float b) {
    constexpr float kP = 0.58f * 0.70710678118f, kMost = 9.2e18f;
    constexpr float kC[8] = {0.163665797f, 0.162445677f, 0.14720637f, 0.0243334345f,
                             0.180663089f, -0.329384131f, 0.190333878f, -0.039263981f};
    const F2 v = f2(a, b);
    const F2 t = rcp_pair(fminf(fmaf(fabsf(a), kP, 1.0f), kMost), fminf(fmaf(fabsf(b), kP, 1.0f), kMost));
    F2 p = f2(kC[7], kC[7]);
#pragma unroll
    for (int i = 6; i >= 0; --i) p = f2_fma(p, t, f2(kC[i], kC[i]));
    const float2 e = f2_get(f2_mul(f2_mul(v, v), f2(-0.5f * kLog2e, -0.5f * kLog2e)));
    const float2 half_erfc = f2_get(f2_mul(f2_mul(p, t), f2(ex2_approx(e.x), ex2_approx(e.y))));
    return f2_mul(v, f2(a > 0.0f ? 1.0f - half_erfc.x : half_erfc.x, b > 0.0f ? 1.0f - half_erfc.y : half_erfc.y));
}

template <int kAct> __device__ __forceinline__ F2 linear_act(F2 v) {
    if constexpr (kAct == GDN_ACT_NONE) return v;
    const float2 f = f2_get(v);
    return kAct == GDN_ACT_SILU ? silu_short(f.x, f.y) : gelu_short(f.x, f.y);
}

// Instruction descriptor, kind::f8f6f4: e4m3 A and B, fp32 accumulator (the
// type fields of A and B are 0 for e4m3; the rest is laid out as for f16).
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D(tmem) (+)= A(smem) * B(smem), 32 bytes of K: 16 bf16 or 32 e4m3.
template <bool kE4m3>
__device__ __forceinline__ void linear_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
    if constexpr (kE4m3)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        tc::mma_ss(d, a, b, idesc, accumulate);
}

// ------------------------------------------------------------ clusters --
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Relaxed, where there is nothing to pass on but that the arrival happened (or
// barriers' initialisation, which fence_mbar_init has released): with release
// every warp first waited for its stores and loads to be done.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Relaxed: it says that something has been read out, or follows the release below.  (With
// release of its own it first waited for the thread's stores to reach the cluster, 2,000
// cycles a tile.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Hands over what is in this CTA's shared memory, with a relaxed arrival behind the one and
// the other behind the wait for it: a release and an acquire at the cluster that order shared
// memory alone, and so do not wait for copies and stores elsewhere.
__device__ __forceinline__ void release_smem_to_cluster() {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}
__device__ __forceinline__ void acquire_smem_of_cluster() {
    asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}
// Sets an int of this name in CTA `rank`'s shared memory.
__device__ __forceinline__ void set_peer_flag(int *flag, uint32_t rank) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_smem(tc::smem_u32(flag), rank)), "r"(1) : "memory");
}
// True in one lane of the (whole, converged) warp.  The warp that issues the
// products stays converged and issues them under this predicate: from a branch
// that one lane took alone (lane == 0) the same loop issued 155 cycles a
// product, in this form it keeps up with the 128 that the tensor cores take
// (256 x 256 x 16 by a pair of CTAs).
__device__ __forceinline__ bool elect_lane() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(e));
    return e != 0;
}
// mbar_wait by a whole warp, with one answer.
__device__ __forceinline__ bool mbar_wait_all(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort));
}

// mbar_wait for a copy or product that is in flight already when the CTA has
// given up: it does not return at once on the abort flag, but it is bounded.
__device__ __forceinline__ void mbar_drain(uint64_t *bar, uint32_t parity) {
    volatile int give_up = 0;
    tc::mbar_wait(bar, parity, &give_up);
}

// A cluster that has given up, once all of its CTAs have sent what they send: far
// longer than a copy takes.
__device__ __forceinline__ void let_copies_land() {
    const uint64_t t = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t < 10000000ull) {
    }
}

// mbar_wait for a whole warp that has time: one lane looks, and sleeps between looks.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
    int ok = 1;
    if ((threadIdx.x & 31) == 0 && !tc::mbar_try_wait(bar, parity)) {
        const uint64_t t0 = tc::globaltimer_ns(), limit = *(volatile uint64_t *)&tc::g_wait_limit_ns;
        while (!tc::mbar_try_wait(bar, parity)) {
            if (*abort || tc::globaltimer_ns() - t0 > limit) {
                *abort = 1;
                ok = 0;
                break;
            }
            __nanosleep(100);
        }
    }
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// The product's 2-D operand: rows of `cols` elements of 2 bytes (bf16) or 1
// (e4m3), loaded as boxes of 128 bytes x box_rows in the 128-byte swizzle.
bool encode_tmap_operand(CUtensorMap *map, const void *base, int64_t cols, int64_t rows,
                         int64_t row_stride_elems, uint32_t box_rows, bool e4m3);

// cudaFuncSetAttribute for a kernel's dynamic shared memory, asked for once per
// device (a call of its own takes as long as the argument checks).
struct SmemAllowed {
    std::atomic<uint64_t> devices{0};
    template <typename K> cudaError_t ask(K kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (devices.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// A cluster launch's configuration, behind the kernel before it in the stream.
struct ClusterLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    ClusterLaunch(int cluster, dim3 grid, dim3 block, size_t smem, cudaStream_t s) {
        cfg.gridDim = grid;
        cfg.blockDim = block;
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
};

// How many clusters of a kernel the device holds at once; the kernel's dynamic
// shared memory is allowed on the way.  Asked for once per device.
struct ClustersHeld {
    static constexpr int kDevices = 16;
    std::atomic<int> held[kDevices] = {};   // count + 1
    template <typename K> cudaError_t ask(K kernel, int cluster, int threads, int smem, int &count) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const int known = dev < kDevices ? held[dev].load(std::memory_order_acquire) : 0;
        if (known) {
            count = known - 1;
            return cudaSuccess;
        }
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        // as much shared memory as there is: two CTAs of an SM where they fit
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        ClusterLaunch l(cluster, dim3(cluster), dim3(threads), smem, nullptr);
        l.cfg.numAttrs = 1;                 // the cluster's size
        e = cudaOccupancyMaxActiveClusters(&count, kernel, &l.cfg);
        // which counts one CTA of an SM.  Two run there where shared memory and
        // registers allow: 64 x 4096 x 2048 with k cut over 16 clusters of 8 took
        // 14.8 us with tiles of 128 KB (15 clusters at once) and 8.6 us with 104 KB.
        int sm_smem = 0, sm_regs = 0;
        cudaFuncAttributes a;
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sm_smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sm_regs, cudaDevAttrMaxRegistersPerMultiprocessor, dev);
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, kernel);
        if (e != cudaSuccess) return e;
        const int per_sm = std::min(sm_smem / (int)(smem + a.sharedSizeBytes + 1024),
                                    sm_regs / ((a.numRegs + 7) / 8 * 8 * threads));
        count *= std::max(1, std::min(2, per_sm));
        if (e == cudaSuccess && dev < kDevices) held[dev].store(count + 1, std::memory_order_release);
        return e;
    }
};

template <typename... KArgs, typename... Args>
inline cudaError_t launch_after_cluster(void (*kernel)(KArgs...), int cluster, dim3 grid, dim3 block,
                                        size_t smem, cudaStream_t s, Args &&...args) {
    const ClusterLaunch l(cluster, grid, block, smem, s);
    return cudaLaunchKernelEx(&l.cfg, kernel, std::forward<Args>(args)...);
}

// Test control of the failure path: loads that a call does not issue, so that its
// waits for them run out.  Behind the first: all but a pair's first tile, or a narrow
// CTA's first block.
enum LinearDrop { kDropNone = 0, kDropAll = 1, kDropBehindFirst = 2 };   // 3: as all

struct LinearCall {
    const void *x, *w;
    int64_t xs, ws;
    int n_in;
    bool e4m3;
    LinearEpi e;
    cudaStream_t stream;
    int drop;       // the failure path's test control (LinearDrop), 0 otherwise
    // whether 128 bytes of a row of x and w are one line of memory, and not parts of two
    bool lines() const {
        const int64_t elem = e4m3 ? 1 : 2;
        return (((uintptr_t)x | (uintptr_t)w | (uint64_t)(xs * elem) | (uint64_t)(ws * elem)) & 127) == 0;
    }
};

// The tiles: token rows [0, nt_full) in channel tiles of 256, the token
// rows behind them in channel tiles of tail_w.  Order: groups of eight token
// tiles; within a group the token tile runs fastest, then the channel tile, so
// the tiles in flight at one time share about as many token rows as weight rows
// (all token tiles in one group: 9 % slower at 20668 x 2048 x 8192).
struct WidePlan {
    int nt_full, nt, nn, n_full, tail_w, n_tiles;
};

// linear_wide.cu: the product on CTA pairs; its plan, with the cycles of an SM that
// it takes by estimate (INT64_MAX: not built), and its launch.
int64_t plan_linear_wide(const LinearCall &c, WidePlan &plan);
cudaError_t set_linear_wide_limit(uint64_t limit_ns, cudaStream_t s);
gdn_status launch_linear_wide(const LinearCall &c, const WidePlan &plan);

}  // namespace gdn
