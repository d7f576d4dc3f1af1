// Activations to 8 bits with one fp32 scale for each block of 128 channels of a
// row, as the products with block scales read them:
//   v = x, or SiLU(x[:n]) x[n:]
//   scale[t][b] = max(max_{j in block b} |v_tj| / 448, 2^-126), q = v / scale
// 16 lanes hold a block, 8 channels each; the block's maximum is four shuffles.  Bound by
// the memory and, with SiLU, nearly by instructions (83 % of the slots): 206680 x 512 gate
// and up in bf16 take 81 us, 0.97 of a copy's rate.  32 registers a thread, so that an SM has
// 2048 threads whose loads are under way.
//
// SiLU takes the fast exponential and division, and the quotient is a product with 1 / scale:
// of 1e6 gated values one lies so near to the middle between two steps of e4m3 (within 2^-21)
// that it goes to the other one than with every operation rounded by itself, which is no
// nearer to the formula.  That (expf, and one step from the remainder behind each of the two
// quotients) takes 48 registers and 128 us here, and 28 instead of 25 for 20668 x 2048
// bf16 without the gate.
#include <algorithm>

#include "quant.cuh"

namespace gdn {

constexpr int kQuantBlock = 128;

// kVec: rows and blocks on vectors of 8 channels; else lane l holds channels l + 16 i.
template <typename T, bool kGlu, bool kVec>
__global__ void __launch_bounds__(256)
block_quant_kernel(const T *__restrict__ x, int64_t xs, int64_t items, int n, int blocks, QuickDiv by_blocks,
                   uint8_t *__restrict__ y, int64_t ys, float *__restrict__ y_scale) {
    griddep_wait();
    griddep_launch();
    const int l = threadIdx.x & 15;
    const int64_t step = (int64_t)gridDim.x * 16;
    const bool small = items < (1ll << 31);
    // whole warps stay in the loop: their shuffles take both halves
    const int64_t half = (threadIdx.x >> 4) & 1;
    for (int64_t i = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); i - half < items; i += step) {
        const bool on = i < items;
        const int64_t t = !on ? 0 : small ? by_blocks((uint32_t)i) : i / blocks;
        const int c = (on ? (int)(i - t * blocks) : 0) * kQuantBlock + (kVec ? l * 8 : l);
        const T *p = x + t * xs + c;
        float v[8] = {};
        if (kVec) {
            RawVec<T, 8> gate, up;
            gate.zero();
            up.zero();
            if (on && c < n) {
                gate.load(p);
                if (kGlu) up.load(p + n);
            }
            F2 a[4], b[4];
            gate.pairs(a);
            if (kGlu) {
                up.pairs(b);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 g = f2_get(a[j]);
                    a[j] = f2_mul(f2(silu_f(g.x), silu_f(g.y)), b[j]);
                }
            }
            unpair<8>(a, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (on && c + 16 * j < n) {
                    v[j] = Io<T>::load(p + 16 * j);
                    if (kGlu) v[j] = silu_f(v[j]) * Io<T>::load(p + n + 16 * j);
                }
        }
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < 8; j += 2) mx = max_abs_nan(mx, v[j], v[j + 1]);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float scale = e4m3_scale(mx), q = 1.0f / scale;
        if (!on) continue;
        if (l == 0) y_scale[i] = scale;
        uint8_t *o = y + t * ys + c;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= q;
        if (kVec) {
            if (c < n) store_row<8>(reinterpret_cast<E4m3 *>(o), v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + 16 * j < n) store_row<1>(reinterpret_cast<E4m3 *>(o + 16 * j), v + j);
        }
    }
}

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_block_quant(const void *x, int64_t x_row_stride, int64_t n_rows, int32_t n, int32_t glu, void *y,
                                      int64_t y_row_stride, float *y_scale, int32_t dtype, void *stream) {
    GDN_REQUIRE(dtype == GDN_F32 || dtype == GDN_BF16, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_rows >= 0 && n > 0, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n <= (1 << 29) && n_rows < (1ll << 31), GDN_ERR_UNSUPPORTED);
    if (n_rows == 0) return GDN_OK;
    const int64_t width = glu ? 2 * (int64_t)n : n;
    GDN_REQUIRE(x && y && y_scale && y != x && (const void *)y_scale != x && (void *)y_scale != y, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_rows == 1 || (x_row_stride >= width && y_row_stride >= n), GDN_ERR_INVALID_ARG);
    const uintptr_t elem = dtype == GDN_F32 ? 4 : 2;
    GDN_REQUIRE((uintptr_t)x % elem == 0 && (uintptr_t)y_scale % 4 == 0, GDN_ERR_INVALID_ARG);
    const bool vec = n % 8 == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)y % 8 == 0 &&
                     (n_rows == 1 || (x_row_stride * (int64_t)elem % 16 == 0 && y_row_stride % 8 == 0));
    const int blocks = (n + kQuantBlock - 1) / kQuantBlock;
    const int64_t items = n_rows * blocks;
    const int grid = (int)std::min<int64_t>((items + 15) / 16, (int64_t)sm_count() * 64);
    auto go = [&](auto kernel, auto one) {
        using T = decltype(one);
        return launch_after(kernel, dim3(grid), dim3(256), 0, (cudaStream_t)stream, (const T *)x, x_row_stride, items, n,
                            blocks, QuickDiv(blocks), (uint8_t *)y, y_row_stride, y_scale);
    };
    cudaError_t e;
#define GDN_BQ(T)                                                                       \
    (glu ? (vec ? go(block_quant_kernel<T, true, true>, T()) : go(block_quant_kernel<T, true, false>, T())) \
         : (vec ? go(block_quant_kernel<T, false, true>, T()) : go(block_quant_kernel<T, false, false>, T())))
    e = dtype == GDN_F32 ? GDN_BQ(float) : GDN_BQ(__nv_bfloat16);
#undef GDN_BQ
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}
