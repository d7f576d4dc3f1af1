// The ends of a mixture of experts: the router, which picks each token's experts
// and sorts the pairs (token, choice) by expert, and the weighted sum that brings
// the experts' rows back to the tokens.
//
// Router.  One warp a token.  The order of the logits is that of 32-bit keys
// (key_of), ties by the lowest index; the k largest are taken one after the
// other.  The sort is a counting sort: a chunk of 64 tokens keeps, per expert, a
// word of 64 bits with the tokens that ask for it, so that a pair's place within
// its chunk is a population count of the bits below it.  That order (by expert,
// then by token) depends on no timing.
#include <algorithm>

#include "quant.cuh"

namespace gdn {

GDN_DECLARE_STATUS_WORD(g_status_moe)
GDN_STATUS_READER(read_status_moe, g_status_moe)

constexpr int kMaxExperts = 1024, kMaxTop = 32;
constexpr int kChunk = 64;                 // tokens of a chunk
constexpr int kRouteThreads = 256;

// Larger logits have larger keys; -0 equals 0 and a NaN is above everything.
// 0 is no logit's key.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return v != v ? 0xffffffffu : b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k == 0xffffffffu ? 0x7fffffffu : k ^ ((int)k < 0 ? 0x80000000u : 0xffffffffu));
}

// A warp's token: lane j < top gets the j-th choice.  PER: experts of a lane.
template <typename T, int PER>
__device__ __forceinline__ void route_token(const T *row, int experts, int top, bool renorm, int lane, int &id,
                                            float &weight) {
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        key[i] = e < experts ? key_of(Io<T>::load(row + e)) : 0u;
    }
    float all = 0.f;
    uint32_t mine = 0, first = 0;
    id = 0;
    for (int j = 0; j < top; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        int at = kMaxExperts;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (key[i] == best) at = i * 32 + lane;
        at = __reduce_min_sync(0xffffffffu, at);
        if (j == 0) {
            first = best;
            if (!renorm) {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (key[i]) all += expf(key_value(key[i]) - key_value(first));
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (at == i * 32 + lane) key[i] = 0;
        if (lane == j) {
            mine = best;
            id = at;
        }
    }
    const float top1 = key_value(first);
    const float p = lane < top ? expf(key_value(mine) - top1) : 0.f;
    if (renorm) all = p;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
    weight = top1 == -INFINITY ? 0.f : p / all;      // no expert is open to the token
}

// A chunk's tokens: ids and weights out, and per expert how many ask for it.
template <typename T, int PER>
__global__ void __launch_bounds__(kRouteThreads)
route_top_kernel(const T *__restrict__ logits, int64_t ls, int n_tokens, int experts, int top, bool renorm,
                 int32_t *__restrict__ ids, float *__restrict__ weights, int32_t *__restrict__ counts) {
    __shared__ int count[kMaxExperts];
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, t0 = blockIdx.x * kChunk;
    for (int e = tid; e < experts; e += kRouteThreads) count[e] = 0;
    __syncthreads();
    for (int t = t0 + (tid >> 5); t < min(t0 + kChunk, n_tokens); t += kRouteThreads / 32) {
        int id;
        float w;
        route_token<T, PER>(logits + t * ls, experts, top, renorm, lane, id, w);
        if (lane < top) {
            ids[(int64_t)t * top + lane] = id;
            weights[(int64_t)t * top + lane] = w;
            atomicAdd(&count[id], 1);
        }
    }
    __syncthreads();
    griddep_launch();
    for (int e = tid; e < experts; e += kRouteThreads) counts[(int64_t)blockIdx.x * experts + e] = count[e];
}

// Per expert the sum over the chunks in front of each one, in place, and over all
// of them.  32 experts a CTA, each by 32 threads, a run of chunks for a thread.
__global__ void __launch_bounds__(1024)
route_scan_kernel(int32_t *__restrict__ counts, int chunks, int experts, int32_t *__restrict__ totals) {
    __shared__ int part[32][33];
    griddep_wait();
    const int x = threadIdx.x & 31, g = threadIdx.x >> 5, e = blockIdx.x * 32 + x;
    const int a = (int)((int64_t)chunks * g / 32), b = (int)((int64_t)chunks * (g + 1) / 32);
    int sum = 0;
    if (e < experts)
        for (int c = a; c < b; ++c) sum += counts[(int64_t)c * experts + e];
    part[g][x] = sum;
    __syncthreads();
    griddep_launch();
    int before = 0;
    for (int i = 0; i < g; ++i) before += part[i][x];
    if (e >= experts) return;
    if (g == 31) totals[e] = before + sum;
    for (int c = a; c < b; ++c) {
        const int n = counts[(int64_t)c * experts + e];
        counts[(int64_t)c * experts + e] = before;
        before += n;
    }
}

// Each pair to its place.
__global__ void __launch_bounds__(kRouteThreads)
route_place_kernel(const int32_t *__restrict__ ids, const int32_t *__restrict__ counts,
                   const int32_t *__restrict__ totals, int n_tokens, int experts, int top,
                   int32_t *__restrict__ offsets, int32_t *__restrict__ rows, int32_t *__restrict__ slots) {
    __shared__ unsigned long long mask[kMaxExperts];
    __shared__ int base[kMaxExperts], warp_sum[kRouteThreads / 32];
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t0 = blockIdx.x * kChunk;
    const int n = min(kChunk, n_tokens - t0) * top;           // pairs (none: only the offsets)
    // experts in front of each one, four of them a thread
    constexpr int Q = kMaxExperts / kRouteThreads;
    int v[Q], sum = 0;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const int e = tid * Q + i;
        v[i] = sum;
        sum += e < experts && totals ? totals[e] : 0;
    }
    int scan = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, scan, off);
        if (lane >= off) scan += o;
    }
    if (lane == 31) warp_sum[warp] = scan;
    for (int e = tid; e < experts; e += kRouteThreads) mask[e] = 0;
    __syncthreads();
    int front = scan - sum;
    for (int i = 0; i < warp; ++i) front += warp_sum[i];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const int e = tid * Q + i;
        if (e < experts) {
            base[e] = front + v[i] + (n > 0 ? counts[(int64_t)blockIdx.x * experts + e] : 0);
            if (blockIdx.x == 0) offsets[e] = front + v[i];
        }
    }
    if (blockIdx.x == 0 && tid == kRouteThreads - 1) offsets[experts] = front + sum;
    for (int i = tid; i < n; i += kRouteThreads) atomicOr(&mask[ids[(int64_t)t0 * top + i]], 1ull << (i / top));
    __syncthreads();
    for (int i = tid; i < n; i += kRouteThreads) {
        const int t = i / top, e = ids[(int64_t)t0 * top + i];
        const int r = base[e] + __popcll(mask[e] & ((1ull << t) - 1));
        rows[r] = t0 + t;
        slots[(int64_t)t0 * top + i] = r;
    }
}

template <typename T>
static cudaError_t launch_top(const void *logits, int64_t ls, int n, int experts, int top, bool renorm, int32_t *ids,
                              float *weights, int32_t *counts, cudaStream_t s) {
    auto go = [&](auto kernel) {
        return launch_after(kernel, dim3((n + kChunk - 1) / kChunk), dim3(kRouteThreads), 0, s, (const T *)logits, ls, n,
                            experts, top, renorm, ids, weights, counts);
    };
    const int per = (experts + 31) / 32;
    if (per <= 1) return go(route_top_kernel<T, 1>);
    if (per <= 2) return go(route_top_kernel<T, 2>);
    if (per <= 4) return go(route_top_kernel<T, 4>);
    if (per <= 8) return go(route_top_kernel<T, 8>);
    if (per <= 16) return go(route_top_kernel<T, 16>);
    return go(route_top_kernel<T, 32>);
}

// y = residual + the weighted rows of a token, one thread a vector of N channels.
template <typename T, int N>
__global__ void __launch_bounds__(256)
combine_kernel(const T *__restrict__ x, int64_t xs, int64_t n_rows, const int32_t *__restrict__ slots,
               const float *__restrict__ weights, const T *res, int64_t rs, int top, int64_t items, int vecs, T *y,
               int64_t ys) {
    griddep_wait();
    griddep_launch();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= items) return;
    const int64_t t = i / vecs;
    const int c = (int)(i - t * vecs) * N;
    constexpr int P = (N + 1) / 2;
    F2 sum[P];
#pragma unroll
    for (int p = 0; p < P; ++p) sum[p] = f2(0.f, 0.f);
    for (int j = 0; j < top; ++j) {
        const int64_t r = slots[t * top + j];
        if (r < 0) continue;
        if (r >= n_rows) {
            flag_status(GDN_DEVSTAT_BAD_INDEX);
            continue;
        }
        const float w = weights[t * top + j];
        RawVec<T, N> raw;
        raw.load(x + r * xs + c);
        F2 v[P];
        raw.pairs(v);
#pragma unroll
        for (int p = 0; p < P; ++p) sum[p] = f2_fma(f2(w, w), v[p], sum[p]);
    }
    if (res) {
        RawVec<T, N> raw;
        raw.load(res + t * rs + c);
        F2 v[P];
        raw.pairs(v);
#pragma unroll
        for (int p = 0; p < P; ++p) sum[p] = f2_add(sum[p], v[p]);
    }
    float f[N];
    unpair<N>(sum, f);
    store_row<N>(y + t * ys + c, f);
}

}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_moe_route_workspace_size(int64_t n_tokens, int32_t n_experts) {
    if (n_tokens <= 0 || n_experts <= 0) return 0;
    return (size_t)((n_tokens + kChunk - 1) / kChunk + 1) * n_experts * sizeof(int32_t);
}

extern "C" gdn_status gdn_moe_route(const void *logits, int64_t logits_row_stride, int64_t n_tokens, int32_t n_experts,
                                    int32_t top_k, int32_t renormalize, int32_t *ids, float *weights, int32_t *offsets,
                                    int32_t *rows, int32_t *slots, int32_t dtype, void *workspace,
                                    size_t workspace_bytes, void *stream) {
    GDN_REQUIRE(dtype == GDN_F32 || dtype == GDN_BF16, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_tokens >= 0 && n_experts > 0 && top_k > 0 && top_k <= n_experts, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_experts <= kMaxExperts && top_k <= kMaxTop && n_tokens * top_k < (1ll << 31) - (1 << 20),
                GDN_ERR_UNSUPPORTED);
    GDN_REQUIRE(offsets && (uintptr_t)offsets % 4 == 0, GDN_ERR_INVALID_ARG);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (n_tokens == 0) {
        e = launch_after(route_place_kernel, dim3(1), dim3(kRouteThreads), 0, s, (const int32_t *)nullptr,
                         (const int32_t *)nullptr, (const int32_t *)nullptr, 0, n_experts, top_k, offsets, rows, slots);
    } else {
        GDN_REQUIRE(logits && ids && weights && rows && slots && workspace, GDN_ERR_INVALID_ARG);
        GDN_REQUIRE(n_tokens == 1 || logits_row_stride >= n_experts, GDN_ERR_INVALID_ARG);
        GDN_REQUIRE((uintptr_t)logits % (dtype == GDN_F32 ? 4 : 2) == 0 && (uintptr_t)ids % 4 == 0 &&
                        (uintptr_t)weights % 4 == 0 && (uintptr_t)rows % 4 == 0 && (uintptr_t)slots % 4 == 0 &&
                        (uintptr_t)workspace % 16 == 0,
                    GDN_ERR_INVALID_ARG);
        GDN_REQUIRE(workspace_bytes >= gdn_moe_route_workspace_size(n_tokens, n_experts), GDN_ERR_INVALID_ARG);
        const int n = (int)n_tokens, chunks = (n + kChunk - 1) / kChunk;
        int32_t *totals = (int32_t *)workspace, *counts = totals + n_experts;
        e = dtype == GDN_F32 ? launch_top<float>(logits, logits_row_stride, n, n_experts, top_k, renormalize != 0, ids,
                                                 weights, counts, s)
                             : launch_top<__nv_bfloat16>(logits, logits_row_stride, n, n_experts, top_k,
                                                         renormalize != 0, ids, weights, counts, s);
        if (e == cudaSuccess)
            e = launch_after(route_scan_kernel, dim3((n_experts + 31) / 32), dim3(1024), 0, s, counts, chunks, n_experts,
                             totals);
        if (e == cudaSuccess)
            e = launch_after(route_place_kernel, dim3(chunks), dim3(kRouteThreads), 0, s, (const int32_t *)ids,
                             (const int32_t *)counts, (const int32_t *)totals, n, n_experts, top_k, offsets, rows, slots);
    }
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

extern "C" gdn_status gdn_moe_combine(const void *x, int64_t x_row_stride, int64_t n_rows, const int32_t *slots,
                                      const float *weights, const void *residual, int64_t residual_row_stride,
                                      int64_t n_tokens, int32_t top_k, int32_t hidden, void *y, int64_t y_row_stride,
                                      int32_t dtype, void *stream) {
    GDN_REQUIRE(dtype == GDN_F32 || dtype == GDN_BF16, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_tokens >= 0 && n_rows >= 0 && top_k > 0 && hidden > 0, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_rows < (1ll << 31) && n_tokens * top_k < (1ll << 31) && top_k <= kMaxExperts, GDN_ERR_UNSUPPORTED);
    if (n_tokens == 0) return GDN_OK;
    GDN_REQUIRE(slots && weights && y && (x || n_rows == 0) && y != x, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE((n_rows <= 1 || x_row_stride >= hidden) && (n_tokens == 1 || y_row_stride >= hidden) &&
                    (!residual || n_tokens == 1 || residual_row_stride >= hidden),
                GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(y != residual || n_tokens == 1 || y_row_stride == residual_row_stride, GDN_ERR_INVALID_ARG);
    const uintptr_t elem = dtype == GDN_F32 ? 4 : 2;
    GDN_REQUIRE((uintptr_t)x % elem == 0 && (uintptr_t)y % elem == 0 && (uintptr_t)residual % elem == 0 &&
                    (uintptr_t)slots % 4 == 0 && (uintptr_t)weights % 4 == 0,
                GDN_ERR_INVALID_ARG);
    const int64_t n = 16 / (int64_t)elem;
    const bool vec = hidden % n == 0 && ((uintptr_t)x | (uintptr_t)y | (uintptr_t)residual) % 16 == 0 &&
                     (n_rows <= 1 || x_row_stride % n == 0) && (n_tokens == 1 || y_row_stride % n == 0) &&
                     (!residual || n_tokens == 1 || residual_row_stride % n == 0);
    const int vecs = vec ? (int)(hidden / n) : hidden;
    const int64_t items = n_tokens * vecs, blocks = (items + 255) / 256;
    GDN_REQUIRE(blocks < (1ll << 31), GDN_ERR_UNSUPPORTED);
    auto go = [&](auto kernel, auto one) {
        using T = decltype(one);
        return launch_after(kernel, dim3((unsigned)blocks), dim3(256), 0, (cudaStream_t)stream, (const T *)x, x_row_stride,
                            n_rows, slots, weights, (const T *)residual, residual_row_stride, top_k, items, vecs, (T *)y,
                            y_row_stride);
    };
    cudaError_t e;
    if (dtype == GDN_F32) e = vec ? go(combine_kernel<float, 4>, 0.0f) : go(combine_kernel<float, 1>, 0.0f);
    else e = vec ? go(combine_kernel<__nv_bfloat16, 8>, __nv_bfloat16()) : go(combine_kernel<__nv_bfloat16, 1>, __nv_bfloat16());
    if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}
