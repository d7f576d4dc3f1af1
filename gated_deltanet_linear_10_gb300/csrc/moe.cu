// The ends of a mixture of experts: the router, which picks each token's experts
// and sorts the pairs (token, choice) by expert, and the weighted sum that brings
// the experts' rows back to the tokens.
//
// Router.  One warp a token, the logits as 32-bit keys of the same order (key_of).
// The top-th largest of the lanes' largest keys is a bound that at least `top`
// experts reach and few others do; these go to shared memory, and an expert's place
// among them is the number of larger ones (ties: of lower index).
//
// The sort is a counting sort in three launches: a CTA has a run of tokens and counts,
// per expert, who asks for it; sums over the runs in front; places, 64 tokens at a time:
// per expert a word of 64 bits with those that ask for it, so that a pair's place is a
// population count of the bits below it.  That order (by expert, then by token) depends
// on no timing.  Up to 512 tokens are one launch of one cluster, whose CTAs read each
// other's words.  (With runs in clusters too, that add up their counts, the second
// launch goes, but 20668 tokens take 28 us instead of 24.)
#include <algorithm>

#include "linear.cuh"
#include "quant.cuh"

namespace gdn {

GDN_DECLARE_STATUS_WORD(g_status_moe)
GDN_STATUS_READER(read_status_moe, g_status_moe)

constexpr int kMaxExperts = 1024, kMaxTop = 32;
constexpr int kChunk = 64;                 // tokens placed at a time
constexpr int kRouteThreads = 256;
// Tokens of a run: a round of a CTA's eight warps, more once the CTAs fill a wave of four
// an SM (20668 tokens in runs of 64, half a wave: 31 us where this took 26).
constexpr int kWave = 608;
static int run_of(int64_t n) {
    return (int)std::max<int64_t>(kRouteThreads / 32, (n + kWave - 1) / kWave);
}
static int runs_of(int64_t n) { return (int)((n + run_of(n) - 1) / run_of(n)); }
// The most of the single launch, eight chunks.  512 tokens of 512 experts in fp32 take
// 11.5 us so and 7.9 in three launches, 256 tokens 7.8 and 7.7; but three launches and a
// workspace are 5 us more on the host, which is what a call outside a graph waits for.
constexpr int kClusterTokens = 512;

// Larger logits have larger keys; -0 equals 0 (by the addition, which also makes every
// NaN the same, above everything).  0 is no logit's key.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((int)k < 0 ? 0x80000000u : 0xffffffffu));
}

// What a lane keeps of an expert, and the word by which experts are ordered: the key,
// then the index turned round, so that of equal logits the lowest index has the largest
// word.  A bf16 logit's key has 16 bits, and one word of 32 is both.
template <typename T> struct Choice;
template <> struct Choice<float> {
    using Word = unsigned long long;
    static constexpr uint32_t kLeast = 1;      // no logit keeps less
    static __device__ __forceinline__ Word word(uint32_t kept, int e) { return (Word)kept << 32 | (uint32_t)~e; }
    static __device__ __forceinline__ float value(uint32_t kept) { return key_value(kept); }
    static __device__ __forceinline__ float value_of(Word w) { return key_value((uint32_t)(w >> 32)); }
    static __device__ __forceinline__ int index_of(Word w) { return (int)~(uint32_t)w; }
    static __device__ __forceinline__ Word warp_max(Word w) {
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(w >> 32));
        return (Word)hi << 32 | __reduce_max_sync(0xffffffffu, (uint32_t)(w >> 32) == hi ? (uint32_t)w : 0u);
    }
};
template <> struct Choice<__nv_bfloat16> {
    using Word = uint32_t;
    static constexpr uint32_t kLeast = 1u << 16;
    static __device__ __forceinline__ Word word(uint32_t kept, int) { return kept; }
    static __device__ __forceinline__ float value(uint32_t kept) {
        return __uint_as_float(__float_as_uint(key_value(kept)) & 0xffff0000u);
    }
    static __device__ __forceinline__ float value_of(Word w) { return value(w); }
    static __device__ __forceinline__ int index_of(Word w) { return 0xffff - (int)(w & 0xffffu); }
    static __device__ __forceinline__ Word warp_max(Word w) { return __reduce_max_sync(0xffffffffu, w); }
};

// A lane's logits of a token as they are in memory: PER experts, VEC of them neighbours.
template <typename T, int PER, int VEC> struct RawLogits {
    static constexpr int W = (PER * (int)sizeof(T) + 3) / 4;
    uint32_t w[W];
    static __device__ __forceinline__ int index(int i, int lane) { return i / VEC * VEC * 32 + lane * VEC + i % VEC; }
    __device__ __forceinline__ void load(const T *row, int experts, int lane) {
        if constexpr (VEC > 1) {
#pragma unroll
            for (int i = 0; i < PER; i += VEC) {
                const int e = index(i, lane);
                const uint4 v = e < experts ? *reinterpret_cast<const uint4 *>(row + e) : make_uint4(0u, 0u, 0u, 0u);
                uint32_t *to = w + i / VEC * 4;
                to[0] = v.x;
                to[1] = v.y;
                to[2] = v.z;
                to[3] = v.w;
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                w[i] = index(i, lane) < experts ? *reinterpret_cast<const uint32_t *>(row + index(i, lane)) : 0u;
        } else {
            auto half = [&](int i) {
                const int e = index(i, lane);
                return i < PER && e < experts ? *reinterpret_cast<const uint16_t *>(row + e) : (uint16_t)0;
            };
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = half(2 * i) | (uint32_t)half(2 * i + 1) << 16;
        }
    }
};

// Two bf16 logits at a time, in the halves of a word: what a token takes in instructions
// is what the router is bound by (one at a time: 20668 x 512 experts 26 us).
__device__ __forceinline__ uint32_t key_of_two(uint32_t v) {
    uint32_t b, sign;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v), "r"(0u));
    asm("prmt.b32 %0, %1, %1, 0xbb99;" : "=r"(sign) : "r"(b));        // each half's sign in all its bits
    return b ^ (sign | 0x80008000u);
}
__device__ __forceinline__ uint32_t max_of_two(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// What a lane keeps of its experts, and of the largest one (of no expert: less than kLeast).
template <int PER, int VEC>
__device__ __forceinline__ uint32_t keep_logits(const RawLogits<float, PER, VEC> &raw, int experts, int lane,
                                                uint32_t (&kept)[PER]) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        kept[i] = raw.index(i, lane) < experts ? key_of(__uint_as_float(raw.w[i])) : 0u;
        most = max(most, kept[i]);
    }
    return most;
}
template <int PER, int VEC>
__device__ __forceinline__ uint32_t keep_logits(const RawLogits<__nv_bfloat16, PER, VEC> &raw, int experts, int lane,
                                                uint32_t (&kept)[PER]) {
    uint32_t two = 0;
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
        const int e = raw.index(i, lane), f = raw.index(i + 1, lane);
        uint32_t k = e < experts ? key_of_two(raw.w[i / 2]) : 0u;
        if ((VEC == 1 && f >= experts) || PER == 1) k &= 0xffffu;
        two = max_of_two(two, k);
        kept[i] = __byte_perm(k, 0xffff - e, 0x1054);
        if constexpr (PER > 1) kept[i + 1] = __byte_perm(k, 0xffff - f, 0x3254);
    }
    return max(two << 16, two & 0xffff0000u);
}

// The top-th largest of the lanes' `most`, or a little less: at least `top` experts keep as
// much, where there are so many.  space: 128 bytes of the warp's own.
template <typename T>
__device__ __forceinline__ uint32_t bound_of(uint32_t most, int top, int lane, void *space) {
    __syncwarp();                              // the last token's are read
    if constexpr (sizeof(T) == 4) {
        uint32_t *lanes = reinterpret_cast<uint32_t *>(space);
        lanes[lane] = most;
        __syncwarp();
        int place = 0;                         // lanes with more
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const uint4 q = *reinterpret_cast<const uint4 *>(lanes + j);
            place += (q.x > most) + (q.y > most) + (q.z > most) + (q.w > most);
        }
        return __reduce_min_sync(0xffffffffu, place < top ? most : 0xffffffffu);
    } else {
        // 15 bits of each: the difference's highest bit says which is larger, of two lanes at a time
        const uint32_t mine = most >> 17, twice = (mine | 0x8000u) * 0x10001u;
        reinterpret_cast<uint16_t *>(space)[lane] = (uint16_t)mine;
        __syncwarp();
        uint32_t less = 0;                     // a bit for each lane that has no more
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 q = reinterpret_cast<const uint4 *>(space)[j];
            uint32_t a, b;
            asm("prmt.b32 %0, %1, %2, 0xfdb9;" : "=r"(a) : "r"(twice - q.x), "r"(twice - q.y));
            asm("prmt.b32 %0, %1, %2, 0xfdb9;" : "=r"(b) : "r"(twice - q.z), "r"(twice - q.w));
            less |= (a & (0x01010101u << 2 * j)) | (b & (0x02020202u << 2 * j));
        }
        const int place = 32 - __popc(less);
        return __reduce_min_sync(0xffffffffu, place < top ? mine : 0x7fffu) << 17;
    }
}
constexpr int kCands = 64;                 // candidates of a token that are kept
constexpr int kCandSpace = kCands + 4;     // words, some behind them of zeros

// A warp's token: its `top` choices to ids and weights, each(expert, place) for every one
// of them.  space: kCandSpace words of the warp's own, for the candidates.
template <typename T, int PER, int VEC, typename F>
__device__ __forceinline__ void route_token(const RawLogits<T, PER, VEC> &raw, int experts, int top, bool renorm, int lane,
                                            uint64_t *space, int32_t *ids, float *weights, F each) {
    using C = Choice<T>;
    using Word = typename C::Word;
    uint32_t kept[PER];
    const uint32_t most = keep_logits(raw, experts, lane, kept);
    auto index = [&](int i) { return raw.index(i, lane); };
    // (no lane's, where fewer lanes than choices have an expert: all experts)
    const uint32_t bound = max(bound_of<T>(most, top, lane, space), C::kLeast);
    const uint32_t most_of_all = __reduce_max_sync(0xffffffffu, most);
    const float top1 = C::value(most_of_all);
    float all = 0.f;
    if (!renorm) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (kept[i] >= C::kLeast) all += expf(C::value(kept[i]) - top1);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
    }
    auto count = [&](uint32_t from) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) n += kept[i] >= from;
        return n;
    };
    auto sum_before = [&](int n) {             // with a lane's own
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, n, off);
            if (lane >= off) n += o;
        }
        return n;
    };
    uint32_t from = bound;
    int cnt = count(from), scan = sum_before(cnt), total = __shfl_sync(0xffffffffu, scan, 31);
    if (total > kCands) {
        // too many (most of the lanes' largest were needed): between the bound and the largest
        // (100000 x 1024 top 32: 1657 us one after the other, 246 so)
        uint32_t past = most_of_all;
        while (total > kCands && past - from > 1) {
            const uint32_t mid = from + (past - from) / 2;
            const int c = count(mid), n = __reduce_add_sync(0xffffffffu, c);
            if (n >= top) {
                from = mid;
                cnt = c;
                total = n;
            } else {
                past = mid;
            }
        }
        scan = sum_before(cnt);
    }
    Word *cands = reinterpret_cast<Word *>(space);
    __syncwarp();                              // the lanes' largest are read
    if (total <= kCands) {
        Word *to = cands + scan - cnt;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (kept[i] >= from) *to++ = C::word(kept[i], index(i));
    } else {                                   // many alike: the largest, one after the other
        for (int j = 0; j < top; ++j) {
            Word best = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const Word w = kept[i] >= C::kLeast ? C::word(kept[i], index(i)) : 0;
                best = w > best ? w : best;
            }
            best = C::warp_max(best);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (C::word(kept[i], index(i)) == best) kept[i] = 0;
            if (lane == 0) cands[j] = best;
        }
    }
    const int n = total <= kCands ? total : top;
    if (lane < 4) cands[n + lane] = 0;
    __syncwarp();
    float p[kCands / 32];
    int rank[kCands / 32];
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kCands / 32; ++q) {
        rank[q] = kCands;
        if (q * 32 >= n) continue;
        const Word mine = q * 32 + lane < n ? cands[q * 32 + lane] : 0;
        int r = 0;
        for (int j = 0; j < n; j += 4) {
            __align__(16) Word w[4];                     // written by vectors
            if constexpr (sizeof(Word) == 4) {
                *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(cands + j);
            } else {
                *reinterpret_cast<ulonglong2 *>(w) = *reinterpret_cast<const ulonglong2 *>(cands + j);
                *reinterpret_cast<ulonglong2 *>(w + 2) = *reinterpret_cast<const ulonglong2 *>(cands + j + 2);
            }
            r += (w[0] > mine) + (w[1] > mine) + (w[2] > mine) + (w[3] > mine);
        }
        rank[q] = mine ? r : kCands;
        p[q] = rank[q] < top ? expf(C::value_of(mine) - top1) : 0.f;
        sum += p[q];
    }
    if (renorm) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        all = sum;
    }
#pragma unroll
    for (int q = 0; q < kCands / 32; ++q)
        if (rank[q] < top) {
            const int id = C::index_of(cands[q * 32 + lane]);
            ids[rank[q]] = id;
            weights[rank[q]] = top1 == -INFINITY ? 0.f : p[q] / all;      // no expert is open to the token
            each(id, rank[q]);
        }
}

// A run of tokens: ids and weights out, and per expert how many ask for it.
template <typename T, int PER, int VEC>
__global__ void __launch_bounds__(kRouteThreads, PER <= 16 ? 4 : 2)
route_top_kernel(const T *__restrict__ logits, int64_t ls, int n_tokens, int run, int experts, int top, bool renorm,
                 int32_t *__restrict__ ids, float *__restrict__ weights, int32_t *__restrict__ counts) {
    __shared__ int count[kMaxExperts];
    __shared__ __align__(16) uint64_t cands[kRouteThreads / 32][kCandSpace];
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, t0 = blockIdx.x * run;
    for (int e = tid; e < experts; e += kRouteThreads) count[e] = 0;
    __syncthreads();
    // few registers: the next token's logits are on their way while one is worked on
    constexpr bool kNext = RawLogits<T, PER, VEC>::W <= 8;
    const int end = min(t0 + run, n_tokens);
    RawLogits<T, PER, VEC> raw, next;
    int t = t0 + (tid >> 5);
    if (kNext && t < end) next.load(logits + t * ls, experts, lane);
    for (; t < end; t += kRouteThreads / 32) {
        if (kNext) {
            raw = next;
            if (t + kRouteThreads / 32 < end) next.load(logits + (t + kRouteThreads / 32) * ls, experts, lane);
        } else {
            raw.load(logits + t * ls, experts, lane);
        }
        route_token(raw, experts, top, renorm, lane, cands[tid >> 5], ids + (int64_t)t * top, weights + (int64_t)t * top,
                    [&](int id, int) { atomicAdd(&count[id], 1); });
    }
    __syncthreads();
    griddep_launch();
    for (int e = tid; e < experts; e += kRouteThreads) counts[(int64_t)blockIdx.x * experts + e] = count[e];
}

// Experts' sums in front of each one, by the whole CTA: v[i] of expert tid * Q + i becomes
// the sum of those before it; returns the sum of all.
template <int Q> __device__ __forceinline__ int scan_experts(int (&v)[Q], int *warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const int x = v[i];
        v[i] = sum;
        sum += x;
    }
    int scan = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, scan, off);
        if (lane >= off) scan += o;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int front = scan - sum, all = 0;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) {
        if (i < warp) front += warp_sum[i];
        all += warp_sum[i];
    }
#pragma unroll
    for (int i = 0; i < Q; ++i) v[i] += front;
    return all;
}

__device__ __forceinline__ uint64_t load_of_rank(const void *p, uint32_t rank) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer_smem(tc::smem_u32(p), rank)) : "memory");
    return v;
}
// Up to kClusterTokens tokens in one launch: a cluster of 1, 2, 4 or 8 CTAs, a chunk each.
constexpr int kClusterThreads = 1024;
template <typename T, int PER, int VEC>
__global__ void __launch_bounds__(kClusterThreads)
route_cluster_kernel(const T *__restrict__ logits, int64_t ls, int n_tokens, int experts, int top, bool renorm,
                     int32_t *__restrict__ ids, float *__restrict__ weights, int32_t *__restrict__ offsets,
                     int32_t *__restrict__ rows, int32_t *__restrict__ slots) {
    __shared__ unsigned long long mask[kMaxExperts];
    __shared__ int base[kMaxExperts], warp_sum[32];
    __shared__ __align__(16) uint64_t cands[kClusterThreads / 32][kCandSpace];
    __shared__ uint16_t pick[kChunk * kMaxTop];
    static_assert(kClusterThreads >= kMaxExperts, "a thread an expert");
    const int tid = threadIdx.x, lane = tid & 31, ctas = gridDim.x;
    const uint32_t rank = cta_rank();
    const int per = (n_tokens + ctas - 1) / ctas, t0 = rank * per, n = max(0, min(per, n_tokens - t0));
    mask[tid] = 0;
    griddep_wait();
    griddep_launch();
    __syncthreads();
    for (int t = tid >> 5; t < n; t += kClusterThreads / 32) {
        int32_t *to = ids + (int64_t)(t0 + t) * top;
        RawLogits<T, PER, VEC> raw;
        raw.load(logits + (t0 + t) * ls, experts, lane);
        route_token(raw, experts, top, renorm, lane, cands[tid >> 5], to, weights + (int64_t)(t0 + t) * top,
                    [&](int id, int place) {
                        atomicOr(&mask[id], 1ull << t);
                        pick[t * top + place] = (uint16_t)id;
                    });
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    int v[1] = {0}, before = 0;
    if (tid < experts) {
        uint64_t word[8];                       // all asked for before the first is counted
#pragma unroll
        for (int r = 0; r < 8; ++r) word[r] = r < ctas ? load_of_rank(&mask[tid], r) : 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            v[0] += __popcll(word[r]);
            if (r < (int)rank) before += __popcll(word[r]);
        }
    }
    const int all = scan_experts(v, warp_sum);
    if (tid < experts) {
        base[tid] = v[0] + before;
        if (rank == 0) offsets[tid] = v[0];
    }
    if (rank == 0 && tid == 0) offsets[experts] = all;
    __syncthreads();
    for (int i = tid; i < n * top; i += kClusterThreads) {
        const int t = i / top, e = pick[i];
        const int r = base[e] + __popcll(mask[e] & ((1ull << t) - 1));
        rows[r] = t0 + t;
        slots[(int64_t)t0 * top + i] = r;
    }
    cluster_arrive_relaxed();
    cluster_wait();                             // no CTA ends while another one may read its words
}

// Per expert the sum over the runs in front of each one, in place, and over all of them.
// 8 experts a CTA, each by 128 threads, a few runs for a thread.
constexpr int kScanExperts = 8, kScanParts = 1024 / kScanExperts, kScanRuns = (kWave + kScanParts - 1) / kScanParts;
__global__ void __launch_bounds__(1024)
route_scan_kernel(int32_t *__restrict__ counts, int runs, int experts, int32_t *__restrict__ totals) {
    __shared__ int sums[32][kScanExperts];
    griddep_wait();
    griddep_launch();
    const int x = threadIdx.x % kScanExperts, part = threadIdx.x / kScanExperts, e = blockIdx.x * kScanExperts + x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = runs * part / kScanParts, end = e < experts ? runs * (part + 1) / kScanParts : 0;
    int32_t *own = counts + (int64_t)first * experts + e;
    int n[kScanRuns], sum = 0;
#pragma unroll
    for (int i = 0; i < kScanRuns; ++i) {
        n[i] = first + i < end ? own[(int64_t)i * experts] : 0;
        sum += n[i];
    }
    // the four parts of a warp, then the warps
    int scan = sum;
#pragma unroll
    for (int off = kScanExperts; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, scan, off);
        if (lane >= off) scan += o;
    }
    if (lane >= 32 - kScanExperts) sums[warp][x] = scan;
    __syncthreads();
    int before = scan - sum, all = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
        if (w < warp) before += sums[w][x];
        all += sums[w][x];
    }
    if (part == 0 && e < experts) totals[e] = all;
#pragma unroll
    for (int i = 0; i < kScanRuns; ++i) {
        if (first + i < end) own[(int64_t)i * experts] = before;
        before += n[i];
    }
}

// Each pair to its place.
__global__ void __launch_bounds__(kRouteThreads)
route_place_kernel(const int32_t *__restrict__ ids, const int32_t *__restrict__ counts,
                   const int32_t *__restrict__ totals, int n_tokens, int run, int experts, int top,
                   int32_t *__restrict__ offsets, int32_t *__restrict__ rows, int32_t *__restrict__ slots) {
    constexpr int Q = kMaxExperts / kRouteThreads;          // experts of a thread
    __shared__ unsigned long long mask[kMaxExperts];
    __shared__ int base[kMaxExperts], warp_sum[kRouteThreads / 32];
    const int tid = threadIdx.x;
    for (int e = tid; e < experts; e += kRouteThreads) mask[e] = 0;
    griddep_wait();
    griddep_launch();
    int v[Q], before[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const int e = tid * Q + i;
        v[i] = e < experts ? totals[e] : 0;
        before[i] = e < experts ? counts[(int64_t)blockIdx.x * experts + e] : 0;
    }
    const int all = scan_experts(v, warp_sum);
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const int e = tid * Q + i;
        if (e < experts) {
            base[e] = v[i] + before[i];
            if (blockIdx.x == 0) offsets[e] = v[i];
        }
    }
    if (blockIdx.x == 0 && tid == 0) offsets[experts] = all;
    const int end = min((int)(blockIdx.x + 1) * run, n_tokens);
    for (int t0 = blockIdx.x * run; t0 < end; t0 += kChunk) {
        const int n = min(kChunk, end - t0) * top;          // pairs
        const int32_t *from = ids + (int64_t)t0 * top;
        for (int i = tid; i < n; i += kRouteThreads) atomicOr(&mask[from[i]], 1ull << (i / top));
        __syncthreads();
        for (int i = tid; i < n; i += kRouteThreads) {
            const int t = i / top, e = from[i];
            const int r = base[e] + __popcll(mask[e] & ((1ull << t) - 1));
            rows[r] = t0 + t;
            slots[(int64_t)t0 * top + i] = r;
        }
        if (t0 + kChunk < end) {
            __syncthreads();
            for (int e = tid; e < experts; e += kRouteThreads) {
                base[e] += __popcll(mask[e]);
                mask[e] = 0;
            }
            __syncthreads();
        }
    }
}

// go(kernels of PER experts a lane, VEC of them neighbours): vectors of 16 bytes where the
// rows allow them, else an expert a lane and step.
template <typename T, typename F> static cudaError_t for_experts(const void *logits, int64_t ls, int n, int experts, F go) {
    constexpr int V = Vec16<T>::N;
    const bool vec = experts % V == 0 && (uintptr_t)logits % 16 == 0 && (n == 1 || ls % V == 0);
    const int per = (experts + 31) / 32;
#define GDN_EXPERTS(PER) (PER >= V && vec ? go.template operator()<PER, (PER >= V ? V : 1)>() : go.template operator()<PER, 1>())
    if (per <= 1) return GDN_EXPERTS(1);
    if (per <= 2) return GDN_EXPERTS(2);
    if (per <= 4) return GDN_EXPERTS(4);
    if (per <= 8) return GDN_EXPERTS(8);
    if (per <= 16) return GDN_EXPERTS(16);
    return GDN_EXPERTS(32);
#undef GDN_EXPERTS
}

struct RouteCall {
    const void *logits;
    int64_t ls;
    int n, experts, top;
    bool renorm;
    int32_t *ids;
    float *weights;
    int32_t *offsets, *rows, *slots, *counts, *totals;
    cudaStream_t s;
};
template <typename T> struct LaunchTop {
    const RouteCall &c;
    template <int PER, int VEC> cudaError_t operator()() const {
        return launch_after(route_top_kernel<T, PER, VEC>, dim3(runs_of(c.n)), dim3(kRouteThreads), 0, c.s,
                            (const T *)c.logits, c.ls, c.n, run_of(c.n), c.experts, c.top, c.renorm, c.ids, c.weights, c.counts);
    }
};
template <typename T> struct LaunchCluster {
    const RouteCall &c;
    template <int PER, int VEC> cudaError_t operator()() const {
        const int ctas = c.n <= 32 ? 1 : c.n <= 64 ? 2 : c.n <= 128 ? 4 : 8;       // a token a warp, or two
        return launch_after_cluster(route_cluster_kernel<T, PER, VEC>, ctas, dim3(ctas), dim3(kClusterThreads), 0, c.s,
                                    (const T *)c.logits, c.ls, c.n, c.experts, c.top, c.renorm, c.ids, c.weights, c.offsets,
                                    c.rows, c.slots);
    }
};
template <typename T> static cudaError_t launch_route(const RouteCall &c) {
    if (c.n <= kClusterTokens) return for_experts<T>(c.logits, c.ls, c.n, c.experts, LaunchCluster<T>{c});
    cudaError_t e = for_experts<T>(c.logits, c.ls, c.n, c.experts, LaunchTop<T>{c});
    if (e == cudaSuccess)
        e = launch_after(route_scan_kernel, dim3((c.experts + kScanExperts - 1) / kScanExperts), dim3(1024), 0, c.s,
                         c.counts, runs_of(c.n), c.experts, c.totals);
    if (e == cudaSuccess)
        e = launch_after(route_place_kernel, dim3(runs_of(c.n)), dim3(kRouteThreads), 0, c.s, (const int32_t *)c.ids,
                         (const int32_t *)c.counts, (const int32_t *)c.totals, c.n, run_of(c.n), c.experts, c.top,
                         c.offsets, c.rows, c.slots);
    return e;
}

// y = residual + the weighted rows of a token, one thread a vector of N channels, kAhead
// rows asked for before the first is added.  Bound by the memory: 20668 x 10 rows of 2048
// bf16 take 163 us, 0.92 of a copy's rate; 256 x 10 take 3.3, a launch and two trips.
// `split`: CTAs of a token, or 0 where a CTA has `per` whole tokens.
constexpr int kAhead = 5, kCombineThreads = 256;
template <typename T, int N>
__global__ void __launch_bounds__(kCombineThreads, 4)
combine_kernel(const T *__restrict__ x, int64_t xs, int64_t n_rows, const int32_t *__restrict__ slots,
               const float *__restrict__ weights, const T *res, int64_t rs, int n_tokens, int top, uint32_t vecs,
               uint32_t split, uint32_t per, T *y, int64_t ys) {
    griddep_wait();
    griddep_launch();
    const uint32_t own = split ? 0 : threadIdx.x / vecs;
    const int64_t t = split ? blockIdx.x / split : (int64_t)blockIdx.x * per + own;
    const uint32_t v = split ? blockIdx.x % split * kCombineThreads + threadIdx.x : threadIdx.x - own * vecs;
    if (t >= n_tokens || v >= vecs || own >= (split ? 1 : per)) return;
    const int64_t c = (int64_t)v * N;
    const int32_t *s = slots + t * top;
    const float *w = weights + t * top;
    constexpr int P = (N + 1) / 2;
    RawVec<T, N> last;
    if (res) last.load(res + t * rs + c);
    F2 sum[P];
#pragma unroll
    for (int p = 0; p < P; ++p) sum[p] = f2(0.f, 0.f);
    for (int j0 = 0; j0 < top; j0 += kAhead) {
        RawVec<T, N> raw[kAhead];
        float f[kAhead];
        bool on[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t r = j0 + j < top ? s[j0 + j] : -1;
            on[j] = r >= 0 && r < n_rows;
            if (r >= n_rows) flag_status(GDN_DEVSTAT_BAD_INDEX);
            if (on[j]) {
                f[j] = w[j0 + j];
                raw[j].load(x + r * xs + c);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (on[j]) {
                F2 q[P];
                raw[j].pairs(q);
#pragma unroll
                for (int p = 0; p < P; ++p) sum[p] = f2_fma(f2(f[j], f[j]), q[p], sum[p]);
            }
    }
    if (res) {
        F2 q[P];
        last.pairs(q);
#pragma unroll
        for (int p = 0; p < P; ++p) sum[p] = f2_add(sum[p], q[p]);
    }
    float f[N];
    unpair<N>(sum, f);
    store_row<N>(y + t * ys + c, f);
}

}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_moe_route_workspace_size(int64_t n_tokens, int32_t n_experts) {
    if (n_tokens <= kClusterTokens || n_experts <= 0) return 0;
    return (size_t)(runs_of(n_tokens) + 1) * n_experts * sizeof(int32_t);
}

extern "C" gdn_status gdn_moe_route(const void *logits, int64_t logits_row_stride, int64_t n_tokens, int32_t n_experts,
                                    int32_t top_k, int32_t renormalize, int32_t *ids, float *weights, int32_t *offsets,
                                    int32_t *rows, int32_t *slots, int32_t dtype, void *workspace,
                                    size_t workspace_bytes, void *stream) {
    GDN_REQUIRE(dtype == GDN_F32 || dtype == GDN_BF16, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_tokens >= 0 && n_experts > 0 && top_k > 0 && top_k <= n_experts, GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(n_experts <= kMaxExperts && top_k <= kMaxTop && n_tokens < (1ll << 31) &&
                    n_tokens * top_k < (1ll << 31) - (1 << 20),
                GDN_ERR_UNSUPPORTED);
    GDN_REQUIRE(offsets && (uintptr_t)offsets % 4 == 0, GDN_ERR_INVALID_ARG);
    cudaStream_t s = (cudaStream_t)stream;
    const bool space = n_tokens > kClusterTokens;
    if (n_tokens > 0) {                                     // none: only the offsets
        GDN_REQUIRE(logits && ids && weights && rows && slots && (workspace || !space), GDN_ERR_INVALID_ARG);
        GDN_REQUIRE(n_tokens == 1 || logits_row_stride >= n_experts, GDN_ERR_INVALID_ARG);
        GDN_REQUIRE((uintptr_t)logits % (dtype == GDN_F32 ? 4 : 2) == 0 && (uintptr_t)ids % 4 == 0 &&
                        (uintptr_t)weights % 4 == 0 && (uintptr_t)rows % 4 == 0 && (uintptr_t)slots % 4 == 0,
                    GDN_ERR_INVALID_ARG);
        GDN_REQUIRE(!space || ((uintptr_t)workspace % 16 == 0 &&
                               workspace_bytes >= gdn_moe_route_workspace_size(n_tokens, n_experts)),
                    GDN_ERR_INVALID_ARG);
    }
    int32_t *counts = (int32_t *)workspace, *totals = space ? counts + (int64_t)runs_of(n_tokens) * n_experts : nullptr;
    const RouteCall c = {logits, logits_row_stride, (int)n_tokens, n_experts, top_k, renormalize != 0, ids, weights,
                         offsets, rows, slots, counts, totals, s};
    const cudaError_t e = dtype == GDN_F32 ? launch_route<float>(c) : launch_route<__nv_bfloat16>(c);
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
    GDN_REQUIRE(n_rows < (1ll << 31) && n_tokens < (1ll << 31) && n_tokens * top_k < (1ll << 31) && top_k <= kMaxExperts,
                GDN_ERR_UNSUPPORTED);
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
    const uint32_t vecs = vec ? (uint32_t)(hidden / n) : (uint32_t)hidden;
    const uint32_t split = vecs >= kCombineThreads ? (vecs + kCombineThreads - 1) / kCombineThreads : 0;
    const uint32_t per = split ? 1 : kCombineThreads / vecs;
    const int64_t blocks = split ? n_tokens * split : (n_tokens + per - 1) / per;
    GDN_REQUIRE(blocks < (1ll << 31), GDN_ERR_UNSUPPORTED);
    auto go = [&](auto kernel, auto one) {
        using T = decltype(one);
        return launch_after(kernel, dim3((unsigned)blocks), dim3(kCombineThreads), 0, (cudaStream_t)stream, (const T *)x,
                            x_row_stride, n_rows, slots, weights, (const T *)residual, residual_row_stride, (int)n_tokens,
                            top_k, vecs, split, per, (T *)y, y_row_stride);
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
