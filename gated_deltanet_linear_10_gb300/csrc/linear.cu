// gdn_linear: the matrix product of the block's projections with scales, bias,
// activation and residual in its epilogue.
//
// The products run on tcgen05 with both operands loaded by TMA in the 128-byte
// swizzle and the accumulator in tensor memory; k is cut into blocks of 128
// bytes (64 bf16 or 128 e4m3), which a ring of shared-memory stages holds.
// The weights' rows are the 128 lanes of the accumulator and the tokens its
// columns, so that a single token costs one narrow product per weight tile and
// the tile follows the number of tokens.
#include <algorithm>

#include "linear.cuh"

namespace gdn {

using namespace tc;

GDN_DECLARE_STATUS_WORD(g_status_linear)
GDN_STATUS_READER(read_status_linear, g_status_linear)

bool encode_tmap_operand(CUtensorMap *map, const void *base, int64_t cols, int64_t rows,
                         int64_t row_stride_elems, uint32_t box_rows, bool e4m3) {
    const int elem = e4m3 ? 1 : 2;
    if (rows == 1) row_stride_elems = (cols + 15) / 16 * 16;   // never stepped over
    return encode_tmap_2d(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                          base, cols, rows, row_stride_elems * elem, 128 / elem, box_rows, true);
}

// BT: tokens per tile (the product's N).  One CTA per 128 x BT tile.
template <int BT> struct NarrowCfg {
    static constexpr uint32_t kW = 128 * 128, kX = BT * 128, kStage = kW + kX;
    static constexpr int kStages = BT >= 256 ? 4 : BT >= 128 ? 6 : 8;
    static constexpr uint32_t kSmem = kStages * kStage + 1024;
    static constexpr uint32_t kCols = BT < 32 ? 32 : BT;
};

// COLS accumulator columns of one weight row n, tokens t0 ..: scale, bias,
// activation, residual, store.  A warp's 32 lanes are 32 consecutive n.  The
// residual is read for all columns before the first store (y may be residual).
template <int COLS, int kAct, typename O>
__device__ __forceinline__ void narrow_store(const uint32_t (&r)[32], const LinearEpi &ep, int n,
                                             int t0, float swn, float bn) {
    O *y = reinterpret_cast<O *>(ep.y) + t0 * ep.ys + n;
    const O *res = reinterpret_cast<const O *>(ep.res) + t0 * ep.rs + n;
    const int cnt = min(COLS, ep.n_tokens - t0);
    float rv[COLS];
#pragma unroll
    for (int j = 0; j < COLS; ++j) rv[j] = ep.res && j < cnt ? Io<O>::load(res + j * ep.rs) : 0.0f;
#pragma unroll
    for (int j = 0; j < COLS; ++j) {
        if (j < cnt) {
            const float sc = ep.sx ? ep.sx[t0 + j] * swn : swn;
            Io<O>::store(y + j * ep.ys, linear_act<kAct>(fmaf(__uint_as_float(r[j]), sc, bn)) + rv[j]);
        }
    }
}

template <int COLS, typename O>
__device__ __forceinline__ void narrow_store_act(const uint32_t (&r)[32], const LinearEpi &ep, int n,
                                                 int t0, float swn, float bn) {
    if (ep.act == GDN_ACT_SILU) narrow_store<COLS, GDN_ACT_SILU, O>(r, ep, n, t0, swn, bn);
    else if (ep.act == GDN_ACT_GELU) narrow_store<COLS, GDN_ACT_GELU, O>(r, ep, n, t0, swn, bn);
    else narrow_store<COLS, GDN_ACT_NONE, O>(r, ep, n, t0, swn, bn);
}

template <int BT, bool kE4m3>
__global__ void __launch_bounds__(192)
linear_narrow_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                     const __grid_constant__ LinearEpi ep, int n_in) {
    using C = NarrowCfg<BT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[C::kStages], empty[C::kStages], done;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int n0 = blockIdx.x * 128, t0 = blockIdx.y * BT;
    constexpr int kElems = kE4m3 ? 128 : 64;                 // k per block of 128 bytes
    const int nk = (n_in + kElems - 1) / kElems;

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&mx);
        prefetch_tensormap(&mw);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&done, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, C::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();   // launched behind the kernel that writes x: nothing is read before it
    volatile int *abort = &abort_flag;

    if (warp == 0 && lane == 0) {
        int i = 0;
        for (; i < nk; ++i) {
            const int s = i % C::kStages;
            if (i >= C::kStages && !mbar_wait(&empty[s], ((i / C::kStages) - 1) & 1, abort)) break;
            uint8_t *st = smem + s * C::kStage;
            mbar_arrive_expect_tx(&full[s], C::kStage);
            tma_load_2d(st, &mw, &full[s], i * kElems, n0);
            tma_load_2d(st + C::kW, &mx, &full[s], i * kElems, t0);
        }
        if (*abort)
            for (int j = i > C::kStages ? i - C::kStages : 0; j < i; ++j)
                mbar_drain(&full[j % C::kStages], (j / C::kStages) & 1);
    } else if (warp == 1 && lane == 0) {
        constexpr uint32_t idesc = kE4m3 ? idesc_e4m3(128, BT) : idesc_bf16(128, BT);
        for (int i = 0; i < nk; ++i) {
            const int s = i % C::kStages;
            if (!mbar_wait(&full[s], (i / C::kStages) & 1, abort)) break;
            tc_fence_after();
            const uint32_t st = smem_u32(smem + s * C::kStage);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                linear_mma<kE4m3>(tmem_base, sdesc_sw128(st + k * 32, 0, 1024),
                                  sdesc_sw128(st + C::kW + k * 32, 0, 1024), idesc, i > 0 || k > 0);
            mma_commit(&empty[s]);
        }
        mma_commit(&done);
        mbar_drain(&done, 0);
    } else if (warp >= 2) {
        // lane l of the quadrant q reads accumulator lane 32 q + l: one weight row
        const uint32_t quad = warp & 3;
        const int n = n0 + quad * 32 + lane;
        const bool on = n < ep.n_out;
        const float swn = on && ep.sw ? ep.sw[n] : 1.0f;
        const float bn = on && ep.bias ? ep.bias[n] : 0.0f;
        if (mbar_wait(&done, 0, abort)) {
            tc_fence_after();
            constexpr int COLS = BT < 32 ? BT : 32;
            for (int c = 0; c < BT && t0 + c < ep.n_tokens; c += 32) {
                uint32_t r[32];
                tmem_ld32(tmem_addr(tmem_base, quad * 32, c), r);   // at least 32 columns are allocated
                if (!on) continue;
                if (ep.out_f32) narrow_store_act<COLS, float>(r, ep, n, t0 + c, swn, bn);
                else narrow_store_act<COLS, __nv_bfloat16>(r, ep, n, t0 + c, swn, bn);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, C::kCols);
    if (tid == 0 && abort_flag) flag_status(GDN_DEVSTAT_TIMEOUT);
}

template <int BT, bool kE4m3>
static gdn_status launch_narrow(const LinearCall &c) {
    using C = NarrowCfg<BT>;
    CUtensorMap mx, mw;
    if (!encode_tmap_operand(&mx, c.x, c.n_in, c.e.n_tokens, c.xs, BT, kE4m3) ||
        !encode_tmap_operand(&mw, c.w, c.n_in, c.e.n_out, c.ws, 128, kE4m3))
        return GDN_ERR_CUDA;
    auto kernel = linear_narrow_kernel<BT, kE4m3>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e == cudaSuccess)
        e = launch_after(kernel, dim3((c.e.n_out + 127) / 128, (c.e.n_tokens + BT - 1) / BT), dim3(192),
                         C::kSmem, c.stream, mx, mw, c.e, c.n_in);
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

template <bool kE4m3> static gdn_status launch_linear(const LinearCall &c) {
    const int t = c.e.n_tokens;
    if (t >= 512) return launch_linear_wide(c, kE4m3);
    if (t <= 16) return launch_narrow<16, kE4m3>(c);
    if (t <= 32) return launch_narrow<32, kE4m3>(c);
    if (t <= 64) return launch_narrow<64, kE4m3>(c);
    if (t <= 128) return launch_narrow<128, kE4m3>(c);
    return launch_narrow<256, kE4m3>(c);
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
    // token tiles are a grid dimension of at most 65,535
    GDN_REQUIRE(n_tokens <= 65535 * 256 && n_out <= (1 << 30) && n_in <= (1 << 30), GDN_ERR_UNSUPPORTED);
    if (n_tokens == 0) return GDN_OK;
    GDN_REQUIRE(x && w && y, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(x_row_stride >= n_in && w_row_stride >= n_in && y_row_stride >= n_out &&
                    (!residual || residual_row_stride >= n_out),
                GDN_ERR_INVALID_ARG);
    // the operands' rows start on 16-byte boundaries (TMA); a single row has no stride
    const int64_t per = dtype == GDN_E4M3 ? 16 : 8;
    GDN_REQUIRE((uintptr_t)x % 16 == 0 && (uintptr_t)w % 16 == 0 &&
                    (n_tokens == 1 || x_row_stride % per == 0) && (n_out == 1 || w_row_stride % per == 0),
                GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(x_row_stride < (1ll << 36) && w_row_stride < (1ll << 36), GDN_ERR_UNSUPPORTED);
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
    c.stream = (cudaStream_t)stream;
    c.e = {x_scale, w_scale, bias, residual, residual_row_stride, y, y_row_stride,
           (int)n_tokens, n_out, act, y_dtype == GDN_F32};
    return dtype == GDN_E4M3 ? launch_linear<true>(c) : launch_linear<false>(c);
}
