// The layer's gated RMSNorm with an 8-bit output: per (token, V head) row
//   y = o / sqrt(mean(o^2) + eps) * w * SiLU(z)
// as in gdn_gated_rmsnorm, then e4m3 with one fp32 scale per token over all
// its heads (a token is one row of the output projection that reads it).
//
// One CTA per token at a time; a thread holds kVecs vectors of 8 elements, and
// the dv / 8 lanes of a head lie within one warp, so the head's mean square is
// a warp shuffle and only the token's maximum crosses warps.  A token's loads
// are issued before the one in front of it is worked on.  SiLU takes the fast
// power of two and reciprocal (a few fp32 ulp, far below half an e4m3 step, and
// within what a scale in fp32 has to keep).
//
// What bounds it: HBM.  20668 x 32 x 128 bf16 takes 64.7 us, 6.55 TB/s of its 423
// MB (0.96 of the copy rate); with one vector a thread for up to 512 vectors,
// and so twice the threads at a token's barrier, 72.7 us; before the loads went
// ahead and the arithmetic in pairs, 95.9 us, by issue slots.
#include <algorithm>

#include "quant.cuh"

namespace gdn {

constexpr int kGatedMaxRow = 16384;   // hv * dv

// Resident threads of an SM with one vector each: 42 registers, fp32 64.
constexpr int gated_sm_threads(size_t elem) { return elem == 4 ? 1024 : 1536; }

// kThreads: the most of a launch; with two vectors each 64 registers for 1024, 128 for 512.
template <typename T, int DV, int kVecs, int kThreads>
__global__ void __launch_bounds__(kThreads, kVecs == 1 ? gated_sm_threads(sizeof(T)) / 256 : 1)
gated_quant_kernel(const T *__restrict__ o, const T *__restrict__ z, int64_t zs,
                   const float *__restrict__ w, int n_tokens, int row, float eps,
                   bool z16, uint8_t *__restrict__ y, float *__restrict__ y_scale) {
    constexpr int N = 8, P = N / 2, LANES = DV / N;
    __shared__ float2 part[2][32];
    griddep_wait();    // launched behind the kernel that writes o: nothing is read before it
    griddep_launch();  // what is launched behind this kernel may set itself up
    const int tid = threadIdx.x;
    F2 wv[P];                                     // the lane's place in a head is the same for every vector
#pragma unroll
    for (int i = 0; i < P; ++i) wv[i] = f2(w[(tid % LANES) * N + 2 * i], w[(tid % LANES) * N + 2 * i + 1]);
    RawVec<T, N> a[kVecs], b[kVecs];
    auto load = [&](int t) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = (tid + k * blockDim.x) * N;
            if (e < row) {
                const T *op = o + (int64_t)t * row + e, *zp = z + (int64_t)t * zs + e;
                if (z16) {
                    a[k].load(op);
                    b[k].load(zp);
                } else {
                    a[k].load_half(op);
                    b[k].load_half(zp);
                }
            }
        }
    };
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        a[k].zero();
        b[k].zero();
    }
    int t = blockIdx.x, flip = 0;
    if (t < n_tokens) load(t);
    for (; t < n_tokens; t += gridDim.x, flip ^= 1) {
        F2 v[kVecs][P], g[kVecs][P];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            a[k].pairs(v[k]);
            b[k].pairs(g[k]);
        }
        if (t + (int)gridDim.x < n_tokens) load(t + gridDim.x);
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            F2 ss2 = f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                ss2 = f2_fma(v[k][i], v[k][i], ss2);
                // SiLU(z) = z / (1 + 2^(-z log2 e)); 1 / infinity = 0 for z << 0
                const float2 e = f2_get(f2_mul(g[k][i], f2(-kLog2e, -kLog2e)));
                const float2 d = f2_get(f2_add(f2(ex2_approx(e.x), ex2_approx(e.y)), f2(1.0f, 1.0f)));
                const F2 gate = f2_mul(g[k][i], f2(rcp_approx(d.x), rcp_approx(d.y)));
                v[k][i] = f2_mul(f2_mul(v[k][i], wv[i]), gate);
            }
            const float2 sum = f2_get(ss2);
            float ss = sum.x + sum.y;
#pragma unroll
            for (int off = LANES / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float inv = rsqrtf(ss * (1.0f / DV) + eps);
            const F2 inv2 = f2(inv, inv);
            const bool on = (tid + k * blockDim.x) * N < row;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                v[k][i] = f2_mul(v[k][i], inv2);
                const float2 f = f2_get(v[k][i]);
                if (on) mx = max_abs_nan(mx, f.x, f.y);
            }
        }
        const float scale = e4m3_scale(block_max(mx, part[flip]));
        const float q = 1.0f / scale;
        const F2 q2 = f2(q, q);
        if (tid == 0) y_scale[t] = scale;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = (tid + k * blockDim.x) * N;
            if (e >= row) continue;
#pragma unroll
            for (int i = 0; i < P; ++i) v[k][i] = f2_mul(v[k][i], q2);
            float f[N];
            unpair<N>(v[k], f);
            store_row<N>(reinterpret_cast<E4m3 *>(y) + (int64_t)t * row + e, f);
        }
    }
}

// fp32 takes twice the registers a vector: at 42 and 64 of them it spilled (20668 x
// 3 x 256: 26.8 us, at 64 22.9; 5000 x 32 x 256: 79.8 us, at 128 55.5).  Beyond 1024
// vectors there is only the 64 (5000 x 64 x 256: 165 us, 4.5 TB/s).
template <typename T, int DV>
static cudaError_t launch_gated_quant(const void *o, const void *z, int64_t zs, const float *w,
                                      int n_tokens, int hv, float eps, bool z16, void *y,
                                      float *y_scale, cudaStream_t s) {
    const int row = hv * DV, vecs = row / 8;
    auto go = [&](auto kernel, int per, int resident) {
        const int threads = ((vecs + per - 1) / per + 31) / 32 * 32;
        const int grid = std::min(n_tokens, sm_count() * std::min(32, std::max(1, resident / threads)));
        return launch_after(kernel, dim3(grid), dim3(threads), 0, s, (const T *)o, (const T *)z, zs,
                            w, n_tokens, row, eps, z16, (uint8_t *)y, y_scale);
    };
    if (vecs <= 256) return go(gated_quant_kernel<T, DV, 1, 256>, 1, gated_sm_threads(sizeof(T)));
    if (sizeof(T) == 4 && vecs <= 1024) return go(gated_quant_kernel<T, DV, 2, 512>, 2, 512);
    return go(gated_quant_kernel<T, DV, 2, 1024>, 2, 1024);
}

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_gated_rmsnorm_quant(const void *o, const void *z, int64_t z_row_stride,
                                              const float *weight, int64_t n_tokens, int32_t hv,
                                              int32_t dv, float eps, void *y, float *y_scale,
                                              int32_t dtype, void *stream) {
    GDN_REQUIRE(dtype == GDN_F32 || dtype == GDN_BF16, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_tokens >= 0 && hv > 0 && eps >= 0.f, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(dv == 16 || dv == 32 || dv == 64 || dv == 128 || dv == 256, GDN_ERR_UNSUPPORTED);
    // a token plus the grid stays within 32 bits
    GDN_REQUIRE((int64_t)hv * dv <= kGatedMaxRow && n_tokens < (1ll << 31) - (1 << 20), GDN_ERR_UNSUPPORTED);
    if (n_tokens == 0) return GDN_OK;
    GDN_REQUIRE(o && z && weight && y && y_scale && y != o && y != z, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(z_row_stride >= (int64_t)hv * dv, GDN_ERR_INVALID_ARG);
    const uintptr_t elem = dtype == GDN_F32 ? 4 : 2;
    GDN_REQUIRE((uintptr_t)o % (4 * elem) == 0 && (uintptr_t)z % (4 * elem) == 0 &&
                    z_row_stride % 4 == 0 && (uintptr_t)y % 8 == 0 && (uintptr_t)weight % 4 == 0 &&
                    (uintptr_t)y_scale % 4 == 0,
                GDN_ERR_INVALID_ARG);
    const bool z16 = (uintptr_t)o % 16 == 0 && (uintptr_t)z % 16 == 0 &&
                     (z_row_stride * (int64_t)elem) % 16 == 0;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
#define GDN_GQ(T, DV) \
    launch_gated_quant<T, DV>(o, z, z_row_stride, weight, (int)n_tokens, hv, eps, z16, y, y_scale, s)
#define GDN_GQ_DV(T)                          \
    switch (dv) {                             \
        case 16: e = GDN_GQ(T, 16); break;    \
        case 32: e = GDN_GQ(T, 32); break;    \
        case 64: e = GDN_GQ(T, 64); break;    \
        case 128: e = GDN_GQ(T, 128); break;  \
        default: e = GDN_GQ(T, 256); break;   \
    }
    if (dtype == GDN_BF16) {
        GDN_GQ_DV(__nv_bfloat16)
    } else {
        GDN_GQ_DV(float)
    }
#undef GDN_GQ_DV
#undef GDN_GQ
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}
