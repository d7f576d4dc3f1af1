// The layer's gated RMSNorm with an 8-bit output: per (token, V head) row
//   y = o / sqrt(mean(o^2) + eps) * w * SiLU(z)
// as in gdn_gated_rmsnorm, then e4m3 with one fp32 scale per token over all
// its heads (a token is one row of the output projection that reads it).
//
// One CTA per token at a time; a thread holds kVecs vectors of 8 elements, and
// the dv / 8 lanes of a head lie within one warp, so the head's mean square is
// a warp shuffle and only the token's maximum crosses warps.  SiLU takes the
// fast exponential and division (a few fp32 ulp, far below half an e4m3 step).
#include <algorithm>

#include "quant.cuh"

namespace gdn {

constexpr int kGatedMaxRow = 16384;   // hv * dv

template <typename T, int DV, int kVecs>
__global__ void __launch_bounds__(kVecs == 1 ? 512 : 1024)
gated_quant_kernel(const T *__restrict__ o, const T *__restrict__ z, int64_t zs,
                                   const float *__restrict__ w, int n_tokens, int row, float eps,
                                   bool z16, uint8_t *__restrict__ y, float *__restrict__ y_scale) {
    constexpr int N = 8, LANES = DV / N;
    __shared__ float2 part[2][32];
    griddep_wait();   // launched behind the kernel that writes o: nothing is read before it
    const int tid = threadIdx.x;
    float wv[N];                                  // the lane's place in a head is the same for every vector
#pragma unroll
    for (int c = 0; c < N; ++c) wv[c] = w[(tid % LANES) * N + c];
    int flip = 0;
    for (int t = blockIdx.x; t < n_tokens; t += gridDim.x, flip ^= 1) {
        RawVec<T, N> a[kVecs], b[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = (tid + k * blockDim.x) * N;
            a[k].zero();
            b[k].zero();
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
        float v[kVecs][N], mx = 0.f;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            float g[N], ss = 0.f;
            a[k].get(v[k]);
            b[k].get(g);
#pragma unroll
            for (int c = 0; c < N; ++c) ss = fmaf(v[k][c], v[k][c], ss);
#pragma unroll
            for (int off = LANES / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float inv = rsqrtf(ss * (1.0f / DV) + eps);
            const bool on = (tid + k * blockDim.x) * N < row;
#pragma unroll
            for (int c = 0; c < N; ++c) {
                v[k][c] = v[k][c] * inv * wv[c] * silu_f(g[c]);
                if (on) mx = max_nan(mx, fabsf(v[k][c]));
            }
        }
        const float scale = e4m3_scale(block_sum_max(0.f, mx, part[flip]).y);
        const float q = 1.0f / scale;
        if (tid == 0) y_scale[t] = scale;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = (tid + k * blockDim.x) * N;
            if (e >= row) continue;
#pragma unroll
            for (int c = 0; c < N; ++c) v[k][c] *= q;
            store_row<N>(reinterpret_cast<E4m3 *>(y) + (int64_t)t * row + e, v[k]);
        }
    }
}

template <typename T, int DV>
static cudaError_t launch_gated_quant(const void *o, const void *z, int64_t zs, const float *w,
                                      int n_tokens, int hv, float eps, bool z16, void *y,
                                      float *y_scale, cudaStream_t s) {
    const int row = hv * DV, vecs = row / 8;
    auto go = [&](auto kernel, int per) {
        const int threads = ((vecs + per - 1) / per + 31) / 32 * 32;
        const int grid = std::min(n_tokens, sm_count() * std::max(1, 2048 / threads));
        return launch_after(kernel, dim3(grid), dim3(threads), 0, s, (const T *)o, (const T *)z, zs,
                            w, n_tokens, row, eps, z16, (uint8_t *)y, y_scale);
    };
    return vecs <= 512 ? go(gated_quant_kernel<T, DV, 1>, 1) : go(gated_quant_kernel<T, DV, 2>, 2);
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
    GDN_REQUIRE((int64_t)hv * dv <= kGatedMaxRow && n_tokens < (1ll << 31), GDN_ERR_UNSUPPORTED);
    if (n_tokens == 0) return GDN_OK;
    GDN_REQUIRE(o && z && weight && y && y_scale, GDN_ERR_INVALID_ARG);
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
