// The block's input norm: the residual's addition and the RMSNorm of the sum,
// per token row of `hidden` elements,
//   s = x + residual,  residual_out = s,
//   y = s / sqrt(mean(s^2) + eps) * (weight_offset + weight),
// with y in x's type or as e4m3 with one fp32 scale per token ("RMSNorm" and
// "Gemma RMSNorm", the (1 + w)-scaled form, "[model] Support Qwen3next",
// LightLLM issue 1097, Highlights; no formula is printed there).
//
// s stays in fp32 registers from the loads to the stores: the norm reads the
// unrounded sum, and residual_out is its one rounding to the stream's type.
// The maximum that the 8-bit scale needs is taken over |s (offset + w)| in the
// same pass as the sum of squares, since 1 / rms is one factor of the row.
//
// One CTA works on a row at a time, or, up to 32 vectors of 16 bytes wide, each
// of its 8 warps; kVecs vectors per thread.  The weights stay in registers over
// the rows of a thread, and a row's loads are issued before the row in front of
// it is reduced, so that there is always a row in flight.
//
// Rows that start within 16 bytes, all of a token's alike (packed rows of an odd
// width are), are cut at their memory's 16-byte boundaries all the same (kShift):
// vector v of a row holds elements v N - p .. v N - p + N - 1, with p where the row
// starts, and the two ends go element by element.  The grid is a multiple of N
// rows, so that p and with it the weights are the same for all rows of a thread.
//
// What bounds it: HBM for many rows.  20668 x 2048 bf16 to e4m3 with the
// residual takes 46.1 us, 6.43 TB/s of its 296 MB (0.95 of the copy rate); 61.9
// us before the loads went ahead.  With 1024 or 2048 resident threads an SM
// instead of 1536 it takes 48.2 and 51.2 us.  A few rows take 1.7 to 2.4 us, a
// launch and two dependent trips to memory.
#include <algorithm>

#include "quant.cuh"

namespace gdn {

constexpr int kRmsMaxHidden = 16384;

// T: x, residual and residual_out.  O: y (T or E4m3).  N: elements per vector
// (16 bytes of T, or 1 where a row is not on 16-byte boundaries).
constexpr int rms_threads(int n, int vecs, size_t elem) {   // the most a launch below takes
    if (n == 1 || (vecs == 4 && elem == 4)) return 1024;
    if (vecs == 4) return 512;
    return n * vecs <= 8 ? 768 : 704;
}
constexpr int kRmsSmThreads = 1536;   // resident threads of an SM: 42 registers each

template <typename T, typename O, int N, int kVecs, bool kShift, int kRows>
__global__ void __launch_bounds__(rms_threads(N, kVecs, sizeof(T)),
                                  kRmsSmThreads / rms_threads(N, kVecs, sizeof(T)) * (N * kVecs <= 8 ? 1 : 0) +
                                      (N * kVecs <= 8 ? 0 : 1))
add_rmsnorm_kernel(const T *x, int64_t xs, const T *res, int64_t rs, const float *__restrict__ w,
                   float offset, int n_rows, int hidden, float eps, T *res_out, int64_t ros, O *y,
                   int64_t ys, float *__restrict__ y_scale, int first, int step) {
    __shared__ float2 part[2][32];
    constexpr bool kQuant = sizeof(O) == 1;
    constexpr int P = (N + 1) / 2;
    griddep_wait();    // launched behind the kernel that writes x: nothing is read before it
    griddep_launch();  // what is launched behind this kernel may set itself up
    const int tid = threadIdx.x;
    // kRows rows at a time: one, or each a warp's
    int row = kRows == 1 ? blockIdx.x : blockIdx.x * kRows + threadIdx.y, flip = 0;
    const int p = kShift ? (int)((first + (uint64_t)row * step) % N) : 0;
    auto at = [&](int k) { return (int)(tid + k * blockDim.x) * N - p; };
    // a whole vector, or (kShift) one of the two ends of a row
    auto whole = [&](int e) { return e < hidden && (!kShift || (e >= 0 && e + N <= hidden)); };
    auto part_of = [&](int e) { return kShift && e < hidden && !(e >= 0 && e + N <= hidden); };
    F2 wv[kVecs][P];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int e = at(k);
        float f[2 * P] = {};
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (kShift ? e + c >= 0 && e + c < hidden : e < hidden) f[c] = offset + w[e + c];
#pragma unroll
        for (int i = 0; i < P; ++i) wv[k][i] = f2(f[2 * i], f[2 * i + 1]);
    }
    RawVec<T, N> a[kVecs], b[kVecs];
    // An end of a row.  bf16: the whole vector, with what lies beside the row, unless
    // that is beside all rows; elements, two to a register, would be waited for here
    // (20668 x 2047 to bf16: 67.9 us, with the vector 57.7; 54.7 with few stores of
    // the ends, 55.3 at 2048).
    constexpr bool kBeside = kShift && sizeof(T) == 2;
    auto load_end = [&](RawVec<T, N> &v, const T *p, int row, int e) {
        if (kBeside && (e >= 0 || row > 0) && (e + N <= hidden || row + 1 < n_rows)) v.load(p);
        else v.load_part(p, -e, hidden - e);
    };
    auto load = [&](int row) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = at(k);
            if (whole(e)) {
                a[k].load(x + row * xs + e);
                if (res) b[k].load(res + row * rs + e);
            } else if (part_of(e)) {
                load_end(a[k], x + row * xs + e, row, e);
                if (res) load_end(b[k], res + row * rs + e, row, e);
            }
        }
    };
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        a[k].zero();
        b[k].zero();
    }
    if (row < n_rows) load(row);
    for (; row < n_rows; row += gridDim.x * kRows, flip ^= 1) {
        F2 s[kVecs][P], ss = f2(0.f, 0.f);
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            F2 r[P];
            a[k].pairs(s[k]);
            b[k].pairs(r);
#pragma unroll
            for (int i = 0; i < P; ++i) s[k][i] = f2_add(s[k][i], r[i]);
            if (kBeside && part_of(at(k))) {         // what lies beside the row is not its own
                const int lo = -at(k), hi = hidden + lo;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float2 v = f2_get(s[k][i]);
                    s[k][i] = f2(2 * i < lo || 2 * i >= hi ? 0.f : v.x, 2 * i + 1 < lo || 2 * i + 1 >= hi ? 0.f : v.y);
                }
            }
        }
        if (row + (int)gridDim.x * kRows < n_rows) load(row + gridDim.x * kRows);
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = at(k);
            if (res_out && e < hidden) {
                float f[2 * P];
                unpair<2 * P>(s[k], f);
                if (whole(e)) store_row<N>(res_out + row * ros + e, f);
                else store_part<N>(res_out + row * ros + e, f, -e, hidden - e);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                ss = f2_fma(s[k][i], s[k][i], ss);
                s[k][i] = f2_mul(s[k][i], wv[k][i]);
                if constexpr (kQuant) {
                    const float2 v = f2_get(s[k][i]);
                    mx = max_abs_nan(mx, v.x, v.y);
                }
            }
        }
        const float2 sum = f2_get(ss), red = block_sum_max(sum.x + sum.y, mx, part[flip]);
        const float inv = rsqrtf(red.x / (float)hidden + eps);
        const F2 inv2 = f2(inv, inv);
        F2 q2 = inv2;
        if constexpr (kQuant) {
            const float scale = e4m3_scale(red.y * inv), q = 1.0f / scale;
            q2 = f2(q, q);
            if (tid == 0) y_scale[row] = scale;
        }
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = at(k);
            if (e >= hidden) continue;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                s[k][i] = f2_mul(s[k][i], inv2);
                if constexpr (kQuant) s[k][i] = f2_mul(s[k][i], q2);
            }
            float f[2 * P];
            unpair<2 * P>(s[k], f);
            if (whole(e)) store_row<N>(y + row * ys + e, f);
            else store_part<N>(y + row * ys + e, f, -e, hidden - e);
        }
    }
}

// Where rows start: on vectors; first + row * step elements behind one, all
// alike; or anywhere.
struct RmsRows {
    enum { kVector, kShifted, kAny } kind;
    int first, step;
};

template <typename T, typename O, int N, int kVecs, bool kShift, int kRows>
static cudaError_t launch_rms_n(RmsRows at, const void *x, int64_t xs, const void *res, int64_t rs,
                                const float *w, float offset, int n_rows, int hidden, float eps,
                                void *res_out, int64_t ros, void *y, int64_t ys, float *y_scale,
                                cudaStream_t s) {
    const int per = N * kVecs;
    const int threads = (((hidden + (kShift ? N - 1 : 0) + per - 1) / per) + 31) / 32 * 32;
    const int resident = N * kVecs <= 8 ? kRmsSmThreads : rms_threads(N, kVecs, sizeof(T));
    int grid = std::min((n_rows + kRows - 1) / kRows, sm_count() * std::max(1, resident / (threads * kRows)));
    if (kShift && grid < n_rows) grid = std::max(N, grid / N * N);
    return launch_after(add_rmsnorm_kernel<T, O, N, kVecs, kShift, kRows>, dim3(grid), dim3(threads, kRows), 0, s,
                        (const T *)x, xs, (const T *)res, rs, w, offset, n_rows, hidden, eps,
                        (T *)res_out, ros, (O *)y, ys, y_scale, at.first, at.step);
}

// One vector per thread while that fits a CTA of 768 threads, two of which an SM
// holds at 42 registers; two per thread up to 704 (bf16, 88 registers) or 768
// threads, four beyond.  A CTA of 544 threads beats one of 288 with twice the
// vectors and registers: 10000 x 4095 bf16 to e4m3 took 77 us, with two 121 (60
// since the rows' ends are cheaper); 5000 x 8191 at two vectors 73 us, at four 95 (56
// since).  A warp per row up to 32 vectors (20000 rows of 203 bf16 to e4m3: 12.3 us, by CTAs
// of a warp 16.7; with two and four vectors a lane it loses: 301 fp32 43 us, by
// CTAs of 96 threads 18).  Shifted bf16 rows of less than 128 elements go element
// by element, their ends being most of them (101: 9.0 us, on vectors 11.3).
template <typename T, typename O>
static cudaError_t launch_rms(RmsRows at, const void *x, int64_t xs, const void *res, int64_t rs,
                              const float *w, float offset, int n_rows, int hidden, float eps,
                              void *res_out, int64_t ros, void *y, int64_t ys, float *y_scale,
                              cudaStream_t s) {
    constexpr int N = 16 / sizeof(T);
    constexpr int kOne = rms_threads(N, 1, sizeof(T)) * N, kTwo = rms_threads(N, 2, sizeof(T)) * 2 * N;
#define GDN_RMS(n, v, shift) GDN_RMS_ROWS(n, v, shift, 1)
#define GDN_RMS_ROWS(n, v, shift, rows)                                                                     \
    launch_rms_n<T, O, n, v, shift, rows>(at, x, xs, res, rs, w, offset, n_rows, hidden, eps, res_out, ros, y, ys, \
                                    y_scale, s)
    if (at.kind == RmsRows::kVector) {
        if (hidden <= 32 * N) return GDN_RMS_ROWS(N, 1, false, 8);
        if (hidden <= kOne) return GDN_RMS(N, 1, false);
        if (hidden <= kTwo) return GDN_RMS(N, 2, false);
        return GDN_RMS(N, 4, false);
    }
    if (at.kind == RmsRows::kShifted && hidden >= (sizeof(T) == 4 ? N : 128)) {   // no vector with both ends
        if (hidden + N - 1 <= 32 * N) return GDN_RMS_ROWS(N, 1, true, 8);
        if (hidden + N - 1 <= kOne) return GDN_RMS(N, 1, true);
        if (hidden + N - 1 <= kTwo) return GDN_RMS(N, 2, true);
        if (hidden + N - 1 <= (sizeof(T) == 4 ? 1024 : 512) * N * 4) return GDN_RMS(N, 4, true);
    }
    if (hidden <= 128) return GDN_RMS_ROWS(1, 4, false, 8);
    if (hidden <= 4096) return GDN_RMS(1, 4, false);
    return GDN_RMS(1, 16, false);
#undef GDN_RMS_ROWS
#undef GDN_RMS
}

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_add_rmsnorm(const void *x, int64_t x_row_stride, const void *residual,
                                      int64_t residual_row_stride, const float *weight,
                                      float weight_offset, int64_t n_tokens, int32_t hidden,
                                      float eps, void *residual_out,
                                      int64_t residual_out_row_stride, void *y,
                                      int64_t y_row_stride, float *y_scale, int32_t dtype,
                                      int32_t y_dtype, void *stream) {
    GDN_REQUIRE(dtype == GDN_F32 || dtype == GDN_BF16, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(y_dtype == dtype || y_dtype == GDN_E4M3, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_tokens >= 0 && hidden > 0 && eps >= 0.f, GDN_ERR_INVALID_ARG);
    // a row plus the grid stays within 32 bits
    GDN_REQUIRE(hidden <= kRmsMaxHidden && n_tokens < (1ll << 31) - (1 << 20), GDN_ERR_UNSUPPORTED);
    if (n_tokens == 0) return GDN_OK;
    GDN_REQUIRE(x && weight && y && y != residual_out, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE((y_scale != nullptr) == (y_dtype == GDN_E4M3), GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(x_row_stride >= hidden && y_row_stride >= hidden, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(!residual || residual_row_stride >= hidden, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(!residual_out || residual_out_row_stride >= hidden, GDN_ERR_INVALID_ARG);
    const uintptr_t elem = dtype == GDN_F32 ? 4 : 2, yelem = y_dtype == GDN_E4M3 ? 1 : elem;
    GDN_REQUIRE((uintptr_t)x % elem == 0 && (uintptr_t)residual % elem == 0 &&
                    (uintptr_t)residual_out % elem == 0 && (uintptr_t)y % yelem == 0 &&
                    (uintptr_t)weight % 4 == 0 && (uintptr_t)y_scale % 4 == 0,
                GDN_ERR_INVALID_ARG);
    // in place a row lies on the one it is made from: another row's CTA would overwrite it
    auto own_row = [&](const void *out, int64_t out_bytes, const void *in, int64_t in_bytes) {
        return out != in || !in || n_tokens == 1 || out_bytes == in_bytes;
    };
    const int64_t yb = y_row_stride * (int64_t)yelem, rob = residual_out_row_stride * (int64_t)elem;
    const int64_t xb = x_row_stride * (int64_t)elem, rb = residual_row_stride * (int64_t)elem;
    GDN_REQUIRE(own_row(y, yb, x, xb) && own_row(y, yb, residual, rb) && own_row(residual_out, rob, x, xb) &&
                    own_row(residual_out, rob, residual, rb),
                GDN_ERR_INVALID_ARG);
    // 16-byte vectors of the stream (and the y elements that belong to one)
    const uint64_t n = 16 / elem;
    const uint64_t first = (uintptr_t)x / elem % n, step = (uint64_t)x_row_stride % n;
    auto alike = [&](const void *p, uintptr_t size, int64_t stride) {
        return !p || ((uintptr_t)p / size % n == first && (n_tokens == 1 || (uint64_t)stride % n == step));
    };
    RmsRows at = {RmsRows::kAny, (int)first, (int)step};
    if (alike(residual, elem, residual_row_stride) && alike(residual_out, elem, residual_out_row_stride) &&
        alike(y, yelem, y_row_stride))
        at.kind = first == 0 && hidden % n == 0 && (step == 0 || n_tokens == 1) ? RmsRows::kVector : RmsRows::kShifted;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
#define GDN_RMS(T, O)                                                                           \
    launch_rms<T, O>(at, x, x_row_stride, residual, residual_row_stride, weight, weight_offset, \
                     (int)n_tokens, hidden, eps, residual_out, residual_out_row_stride, y,        \
                     y_row_stride, y_scale, s)
    if (dtype == GDN_BF16)
        e = y_dtype == GDN_E4M3 ? GDN_RMS(__nv_bfloat16, E4m3) : GDN_RMS(__nv_bfloat16, __nv_bfloat16);
    else
        e = y_dtype == GDN_E4M3 ? GDN_RMS(float, E4m3) : GDN_RMS(float, float);
#undef GDN_RMS
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}
