// Products of rows with the weights of their expert, in bf16 or in e4m3 with an
// fp32 scale for each block of 128 in k, and the product of all rows with one
// weight in the latter form:
//   y_r = sum_b sx[x row of r][b] sw[e][n / 128][b] sum_{k in b} x[x row of r][k] w[e][n][k]
// for offsets[e] <= r < offsets[e + 1].
#include <algorithm>

#include "linear.cuh"
#include "grouped.cuh"

namespace gdn {

GDN_DECLARE_STATUS_WORD(g_status_grouped)
GDN_STATUS_READER(read_status_grouped, g_status_grouped)

template <bool kE4m3> __device__ __forceinline__ float grouped_value(const void *p, int64_t i) {
    if constexpr (kE4m3) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(reinterpret_cast<const __nv_fp8_storage_t *>(p)[i], __NV_E4M3);
        return __half2float(*reinterpret_cast<const __half *>(&h));
    } else {
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
    }
}

// Tiles of 64 rows x 64 channels; 4 x 4 of them a thread.
template <bool kE4m3, typename O>
__global__ void __launch_bounds__(256) grouped_simple_kernel(const GroupedCall c) {
    constexpr int KS = 32;
    __shared__ float xs[KS][65], ws[KS][65];
    __shared__ int found[3];
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, n0 = blockIdx.x * 64;
    if (tid == 0) {
        int first = 0, end = c.n_rows, e = 0, left = blockIdx.y;
        bool bad = false;
        if (c.offsets) {
            int at = -1, r0 = 0, r1 = 0;
            for (int i = 0; i < c.n_experts; ++i) {
                const int a = c.offsets[i], b = c.offsets[i + 1];
                bad |= a < 0 || b < a || b > c.n_rows;
                const int tiles = (b - a + 63) / 64;
                if (at < 0 && left < tiles) {
                    at = i;
                    r0 = a;
                    r1 = b;
                }
                if (at < 0) left -= tiles;
            }
            e = at;
            first = r0;
            end = r1;
        }
        if (bad) flag_status(GDN_DEVSTAT_BAD_SEQLEN);
        found[0] = bad ? -1 : e;
        found[1] = first + left * 64;
        found[2] = end;
    }
    __syncthreads();
    const int e = found[0], r0 = found[1], r1 = found[2];
    if (e < 0) return;
    const int tx = tid & 15, ty = tid >> 4;
    float sum[4][4] = {}, part[4][4] = {};
    int64_t xrow[4];
    auto x_row = [&](int r) -> int64_t {
        if (r >= r1) return -1;
        if (!c.rows) return r;
        const int64_t v = c.rows[r];
        if (v >= c.n_x) flag_status(GDN_DEVSTAT_BAD_INDEX);
        return v >= 0 && v < c.n_x ? v : -1;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) xrow[i] = x_row(r0 + ty * 4 + i);
    for (int k0 = 0; k0 < c.n_in; k0 += KS) {
        for (int i = tid; i < 64 * KS; i += 256) {
            const int k = i % KS, r = i / KS;
            const int64_t xr = x_row(r0 + r);
            xs[k][r] = xr >= 0 && k0 + k < c.n_in ? grouped_value<kE4m3>(c.x, xr * c.xs + k0 + k) : 0.f;
            ws[k][r] = n0 + r < c.n_out && k0 + k < c.n_in
                           ? grouped_value<kE4m3>(c.w, e * c.we + (int64_t)(n0 + r) * c.ws + k0 + k) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) part[i][j] = fmaf(xs[k][ty * 4 + i], ws[k][tx + 16 * j], part[i][j]);
        __syncthreads();
        if (!kE4m3 || k0 % 128 == 96 || k0 + KS >= c.n_in) {
            const int b = k0 / 128;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f = 1.0f;
                    const int n = n0 + tx + 16 * j;
                    if (kE4m3 && xrow[i] >= 0 && n < c.n_out)
                        f = c.sx[xrow[i] * c.kb + b] * c.sw[((int64_t)e * c.nb + n / 128) * c.kb + b];
                    sum[i][j] = fmaf(part[i][j], f, sum[i][j]);
                    part[i][j] = 0.f;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + ty * 4 + i, n = n0 + tx + 16 * j;
            if (r < r1 && n < c.n_out)
                Io<O>::store(reinterpret_cast<O *>(c.y) + r * c.ys + n, xrow[i] < 0 ? 0.f : sum[i][j]);
        }
}

static gdn_status launch_grouped(const GroupedCall &c, cudaStream_t s) {
    const int tiles = (int)std::min<int64_t>(65535, ((int64_t)c.n_rows + 63) / 64 + (c.offsets ? c.n_experts : 0));
    auto go = [&](auto kernel) {
        return launch_after(kernel, dim3((c.n_out + 63) / 64, tiles), dim3(256), 0, s, c);
    };
    const cudaError_t e = c.e4m3 ? (c.out_f32 ? go(grouped_simple_kernel<true, float>) : go(grouped_simple_kernel<true, __nv_bfloat16>))
                                 : (c.out_f32 ? go(grouped_simple_kernel<false, float>) : go(grouped_simple_kernel<false, __nv_bfloat16>));
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

}  // namespace gdn

using namespace gdn;

static gdn_status grouped_check(const GroupedCall &c, int64_t n_rows, int64_t n_x, int32_t dtype, int32_t y_dtype) {
    GDN_REQUIRE(c.x && c.w && c.y && c.y != c.x && c.y != c.w, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE((n_x == 1 || c.xs >= c.n_in) && (c.n_out == 1 || c.ws >= c.n_in) && (n_rows == 1 || c.ys >= c.n_out),
                GDN_ERR_INVALID_ARG);
    // the operands' rows start on 16-byte boundaries (TMA); a single row has no stride
    const int64_t per = c.e4m3 ? 16 : 8;
    GDN_REQUIRE((uintptr_t)c.x % 16 == 0 && (uintptr_t)c.w % 16 == 0 && (n_x == 1 || c.xs % per == 0) &&
                    (c.n_out == 1 || c.ws % per == 0) && (c.n_experts == 1 || c.we % per == 0),
                GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(c.n_experts == 1 || c.we >= (c.n_out - 1) * c.ws + c.n_in, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(c.xs < (1ll << 36) && c.ws < (1ll << 36) && c.we < (1ll << 36) && c.ys < (1ll << 36), GDN_ERR_UNSUPPORTED);
    GDN_REQUIRE((uintptr_t)c.y % (c.out_f32 ? 4 : 2) == 0 && (uintptr_t)c.sx % 4 == 0 && (uintptr_t)c.sw % 4 == 0 &&
                    (uintptr_t)c.offsets % 4 == 0 && (uintptr_t)c.rows % 4 == 0,
                GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(c.e4m3 ? c.sx && c.sw : !c.sx && !c.sw, GDN_ERR_INVALID_ARG);
    return GDN_OK;
}

extern "C" gdn_status gdn_linear_block(const void *x, int64_t x_row_stride, const float *x_scale, const void *w,
                                       int64_t w_row_stride, const float *w_scale, int64_t n_tokens, int32_t n_in,
                                       int32_t n_out, void *y, int64_t y_row_stride, int32_t y_dtype, void *stream) {
    GDN_REQUIRE(y_dtype == GDN_F32 || y_dtype == GDN_BF16, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_tokens >= 0 && n_in > 0 && n_out > 0, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_tokens <= kGroupedRows && n_out <= kGroupedOut && n_in <= kGroupedIn, GDN_ERR_UNSUPPORTED);
    if (n_tokens == 0) return GDN_OK;
    const GroupedCall c = {x, w, x_row_stride, w_row_stride, 0, x_scale, w_scale, nullptr, nullptr, y, y_row_stride,
                           (int)n_tokens, (int)n_tokens, 1, n_in, n_out, (n_in + 127) / 128, (n_out + 127) / 128, true,
                           y_dtype == GDN_F32};
    const gdn_status st = grouped_check(c, n_tokens, n_tokens, GDN_E4M3, y_dtype);
    return st == GDN_OK ? launch_grouped(c, (cudaStream_t)stream) : st;
}

extern "C" gdn_status gdn_grouped_linear(const void *x, int64_t x_row_stride, const float *x_scale, int64_t n_x,
                                         const int32_t *rows, const void *w, int64_t w_row_stride,
                                         int64_t w_expert_stride, const float *w_scale, const int32_t *offsets,
                                         int32_t n_experts, int64_t n_rows, int32_t n_in, int32_t n_out, void *y,
                                         int64_t y_row_stride, int32_t dtype, int32_t y_dtype, void *stream) {
    GDN_REQUIRE(dtype == GDN_F32 || dtype == GDN_BF16 || dtype == GDN_E4M3, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(y_dtype == GDN_F32 || y_dtype == GDN_BF16, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(dtype != GDN_F32, GDN_ERR_UNSUPPORTED);
    GDN_REQUIRE(n_rows >= 0 && n_x >= 0 && n_in > 0 && n_out > 0 && n_experts > 0, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_rows <= kGroupedRows && n_x <= kGroupedRows && n_out <= kGroupedOut && n_in <= kGroupedIn &&
                    n_experts <= kGroupedExperts,
                GDN_ERR_UNSUPPORTED);
    if (n_rows == 0) return GDN_OK;
    GDN_REQUIRE(offsets && n_x > 0 && (rows || n_x == n_rows), GDN_ERR_INVALID_ARG);
    const GroupedCall c = {x, w, x_row_stride, w_row_stride, w_expert_stride, x_scale, w_scale, offsets, rows, y,
                           y_row_stride, (int)n_rows, (int)n_x, n_experts, n_in, n_out, (n_in + 127) / 128,
                           (n_out + 127) / 128, dtype == GDN_E4M3, y_dtype == GDN_F32};
    const gdn_status st = grouped_check(c, n_rows, n_x, dtype, y_dtype);
    return st == GDN_OK ? launch_grouped(c, (cudaStream_t)stream) : st;
}
