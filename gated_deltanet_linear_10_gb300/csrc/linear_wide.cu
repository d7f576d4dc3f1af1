// gdn_linear for many tokens: a persistent grid of CTA pairs, each pair on one
// tile of 256 tokens x up to 256 channels at a time (tcgen05 cta_group::2,
// M = 256).
//
// A CTA of a pair loads its own 128 tokens and half of the tile's weight rows,
// so a pair reads each operand byte once from L2.  The accumulator is doubled
// in tensor memory: the epilogue warps turn one tile into y while the next
// one's products run.
//
// What bounds it from n_in = 1024 on is the tensor cores' rate and then the
// power: 256 x 256 x 16 take a pair 128 cycles.  20668 x 2048 x 8192 bf16 is
// 574,000 cycles of them and takes some 590,000, at 1.5 GHz (1.9 without the load):
// 353 to 365 us, 1,950 TFLOP/s; over seconds 411 to 425 us.  20668 x 4096 x 2048 e4m3
// with a residual: 104 to 114 us, 3,340 TFLOP/s at best, over seconds 120 to 124, one of
// its nine waves half full.
// What it took, in cycles of a tile (n_in 2048; 16,400 of products): issuing from
// a converged warp 2,900, six stages instead of five 900 (the ring's latency: with
// four, 3,300), a converged producer warp 700.  At n_in = 256 a tile is its
// epilogue: four chunks of 1,000 cycles for a warp (8000 x 256 x 4096: 24 us, 72 MB).
//
// Epilogue: a thread holds a token row and takes 32 channels at a time to a
// swizzled staging row of 128 bytes, from which one TMA store writes 32 rows; the
// residual comes straight from memory, whole sectors of 32 bytes.  Stores from
// registers instead of staging rows were 4 % slower.  Rows off 16-byte boundaries
// are turned in shared memory, so that a warp's lanes access neighbours.
#include <limits.h>

#include <algorithm>

#include "linear.cuh"

namespace gdn {

using namespace tc;

GDN_DECLARE_STATUS_WORD(g_status_linear_wide)
GDN_STATUS_READER(read_status_linear_wide, g_status_linear_wide)

cudaError_t set_linear_wide_limit(uint64_t limit_ns, cudaStream_t s) {
    return cudaMemcpyToSymbolAsync(tc::g_wait_limit_ns, &limit_ns, sizeof(limit_ns), 0, cudaMemcpyHostToDevice, s);
}

namespace {

constexpr int kTokTile = 256, kTokHalf = 128, kChTile = 256, kStagesWide = 6, kEpiWarps = 8;
constexpr int kWideThreads = 128 + 32 * kEpiWarps;
constexpr int kRaster = 8;     // token tiles of one raster group (below)
constexpr uint32_t kStaging = 4096;   // per warp: 32 rows of 128 bytes, or 32 x 32 floats to turn
constexpr uint32_t kStageA = kTokHalf * 128, kStageBytes = kStageA + kChTile / 2 * 128;
constexpr uint32_t kWideSmem = kStagesWide * kStageBytes + kEpiWarps * kStaging;

// Tiled load into this CTA's shared memory, its bytes counted on a barrier of
// either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar,
                                                 int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// Arrives on the barrier at this offset in the CTAs of the mask (1: the leader, 3: both)
// once the products issued so far by this thread are done.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar, uint16_t mask = 3) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(mask)
        : "memory");
}
template <bool kE4m3>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    if constexpr (kE4m3)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// A pair's walk over the tiles: every `pairs`-th one.  Steps instead of
// divisions: two of them in every warp cost some 500 cycles a tile.
struct WideWalk {
    int tile, base, r;       // base: first token tile of the group, r: tile within the group (tail: within it)
    __device__ __forceinline__ void start(const WidePlan &p, int first) {
        tile = r = first;
        base = 0;
        settle(p);
    }
    __device__ __forceinline__ void next(const WidePlan &p, int pairs) {
        tile += pairs;
        r += pairs;
        settle(p);
    }
    __device__ __forceinline__ void settle(const WidePlan &p) {
        while (base < p.nt_full) {
            const int size = min(kRaster, p.nt_full - base) * p.nn;
            if (r < size) break;
            r -= size;
            base += min(kRaster, p.nt_full - base);
        }
    }
    __device__ __forceinline__ bool more(const WidePlan &p) const { return tile < p.n_tiles; }
    __device__ __forceinline__ void at(const WidePlan &p, int n_out, int &t0, int &n0, int &box, int &width) const {
        const bool full = base < p.nt_full;
        const int rows = full ? min(kRaster, p.nt_full - base) : p.nt - p.nt_full;
        const int n = rows == kRaster ? r / kRaster : r / rows;
        box = full ? kChTile : p.tail_w;
        t0 = (base + r - n * rows) * kTokTile;
        n0 = n * box;
        width = min(box, (n_out - n0 + 31) / 32 * 32);   // the product's N: no wider than the channels left
    }
};

// Where the rows of y and the residual start: on 32, 16 or 4 bytes, or anywhere;
// kRowsOdd: on 2 bytes, y's and the residual's rows alike.
enum WideRows { kRows32, kRows16, kRows4, kRowsOdd, kRowsPlain };

// 32 bytes of a row into registers.
__device__ __forceinline__ void load32(uint32_t *r, const void *p, int rows) {
    if (rows == kRows32) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                       "=r"(r[7])
                     : "l"(p)
                     : "memory");
    } else {
        const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
        r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
        r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
    }
}
// A value of O as 32 bits, so that loads stay in flight until it is used.
template <typename O> __device__ __forceinline__ uint32_t load_bits(const O *p) {
    if constexpr (sizeof(O) == 4) return *reinterpret_cast<const uint32_t *>(p);
    else return *reinterpret_cast<const uint16_t *>(p);
}
template <typename O> __device__ __forceinline__ float bits_value(uint32_t b) {
    return __uint_as_float(sizeof(O) == 4 ? b : b << 16);
}

// 32 channels n .. of a row: whole vectors, or element by element behind which
// the row ends.
template <typename O>
__device__ __forceinline__ void load_row(uint32_t *r, const O *p, int n, int n_out, int rows) {
    constexpr int E = 4 / sizeof(O);                 // elements of a word
    if (n + 32 <= n_out) {
#pragma unroll
        for (int i = 0; i < 32 / E; i += 8) load32(r + i, p + i * E, rows);
    } else {
#pragma unroll
        for (int i = 0; i < 32 / E; ++i) {
            r[i] = n + i * E < n_out ? load_bits(p + i * E) : 0u;
            if (E == 2 && n + i * E + 1 < n_out) r[i] |= load_bits(p + i * E + 1) << 16;
        }
    }
}

// The residual of a warp's 32 token rows x 32 channels n .., a channel a lane;
// in bounds for every lane and row.
template <typename O>
__device__ __forceinline__ void plain_ask(uint32_t *rv, const LinearEpi &ep, int t0, int n, int lane) {
    const O *res = reinterpret_cast<const O *>(ep.res) + min(n + lane, ep.n_out - 1);
    const int last = ep.n_tokens - 1;
#pragma unroll
    for (int i = 0; i < 32; ++i) rv[i] = load_bits(res + min(t0 + i, last) * ep.rs);
}

// A warp's 32 token rows x 32 channels of values (r: one token row a lane) to
// rows that start anywhere: turned through a 32 x 32 buffer (columns permuted
// by the row, so that both ways touch every bank once), then a lane is a
// channel.  rv: their residual.
template <typename O>
__device__ __forceinline__ void wide_plain(const uint32_t (&r)[32], const uint32_t (&rv)[32], float *turn,
                                           const LinearEpi &ep, int t0, int n, int lane) {
    __syncwarp();                                    // the buffer's last values are read
#pragma unroll
    for (int j = 0; j < 32; ++j) turn[lane * 32 + (j ^ lane)] = __uint_as_float(r[j]);
    __syncwarp();
    const int rows = n + lane < ep.n_out ? ep.n_tokens - t0 : 0;
    O *y = reinterpret_cast<O *>(ep.y) + n + lane + t0 * ep.ys;
    float v[32];                                     // all read in front of the first store
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = turn[i * 32 + (lane ^ i)];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (ep.res) v[i] += bits_value<O>(rv[i]);
        if (i < rows) Io<O>::store(y, v[i]);
        y += ep.ys;
    }
}

// The same for bf16 rows that start on 4 bytes or, kOdd, some on 2: a lane holds
// two channels of a row and the warp two rows at a time, half of wide_plain's
// accesses to memory (11036 x 84 x 4854 with a residual: 105 us, with wide_plain
// 138; words of 8 bytes gain nothing more).  An odd row, which starts between two
// words, gives channels n - 1 .. n + 30 instead, so that these are words too; the
// last chunk of a run adds the one that is left, and of the tile's first word only
// the upper half is its own (12183 x 538 x 5715 with a residual: 146 us; with both
// ends of every chunk apart 179, with wide_plain 203).
template <bool kOdd> struct WideWords {
    int h, w;                                              // row of the pair, word of the row
    bool odd, mine, edge, last;                            // rows of h odd; row t0 + lane odd; half a word; end of a run
    __device__ __forceinline__ WideWords(const LinearEpi &ep, int t0, int n, int c, int width, int lane) {
        h = lane >> 4;
        w = lane & 15;
        odd = mine = edge = last = false;
        if constexpr (kOdd) {
            const uint64_t at = ((uintptr_t)ep.y >> 1) + (uint64_t)t0 * ep.ys + n;
            odd = (at + h * ep.ys) & 1;
            mine = (at + lane * ep.ys) & 1;
            edge = odd && w == 0 && c == 0;
            last = c + 32 >= width || n + 64 > ep.n_out;
        }
    }
    // rv[k]: the residual's word of row 2 k + h; rv[16]: that of the channel left over in row t0 + lane
    __device__ __forceinline__ void ask(uint32_t *rv, const LinearEpi &ep, int t0, int n, int lane) const {
        const __nv_bfloat16 *res = reinterpret_cast<const __nv_bfloat16 *>(ep.res);
        const __nv_bfloat16 *p = res + (t0 + h) * ep.rs + n + 2 * w - odd;
        const int rows = ep.n_tokens - t0 - h;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if (2 * k < rows) {
                if (kOdd && edge) rv[k] = load_bits(p + 1);      // shifted when it is used, not before it is here
                else rv[k] = *reinterpret_cast<const uint32_t *>(p);
            }
            p += 2 * ep.rs;
        }
        if (kOdd && last && mine && t0 + lane < ep.n_tokens) rv[16] = load_bits(res + (t0 + lane) * ep.rs + n + 31);
    }
    // before: the value of channel n - 1
    __device__ __forceinline__ void out(const uint32_t (&r)[32], uint32_t before, const uint32_t (&rv)[32], uint8_t *turn,
                                        const LinearEpi &ep, int t0, int n, int lane) const {
        __syncwarp();                                      // the buffer's last values are read
        auto v = [&](int j) { return kOdd && mine ? (j ? r[j - 1] : before) : r[j]; };
#pragma unroll
        for (int q = 0; q < 8; ++q)                        // 16 bytes at a time, permuted by the row
            *reinterpret_cast<uint4 *>(turn + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                make_uint4(v(4 * q), v(4 * q + 1), v(4 * q + 2), v(4 * q + 3));
        __syncwarp();
        const int rows = ep.n_tokens - t0 - h;
        __nv_bfloat16 *y = reinterpret_cast<__nv_bfloat16 *>(ep.y);
        if (kOdd && last && mine && t0 + lane < ep.n_tokens) {
            float v = __uint_as_float(r[31]);
            if (ep.res) v += bits_value<__nv_bfloat16>(rv[16]);
            Io<__nv_bfloat16>::store(y + (t0 + lane) * ep.ys + n + 31, v);
        }
        y += (t0 + h) * ep.ys + n + 2 * w - odd;
        // All of them are read in front of the first store, which the compiler will not
        // read behind.
        float2 f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)                       // row 2 k + h, its word w
            f[k] = *reinterpret_cast<const float2 *>(turn + k * 256 + h * 128 + (w & 1) * 8 +
                                                     (((w >> 1) ^ h ^ (2 * k & 7)) << 4));
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            float a = f[k].x, b = f[k].y;
            if (ep.res) {
                a += bits_value<__nv_bfloat16>(rv[k]);
                b += __uint_as_float(kOdd && edge ? rv[k] << 16 : rv[k] & 0xffff0000u);
            }
            const uint32_t q = pack_bf16(a, b);
            if (2 * k < rows) {
                if (kOdd && edge) *reinterpret_cast<uint16_t *>(y + 1) = (uint16_t)(q >> 16);
                else *reinterpret_cast<uint32_t *>(y) = q;
            }
            y += 2 * ep.ys;
        }
    }
};

// 32 accumulators of one token row -> act(sx sw acc + bias), in place.  cols:
// the columns' scales in shared memory, their biases kChTile floats on.
template <int kAct, bool kCols>
__device__ __forceinline__ void wide_values(uint32_t (&r)[32], const float *cols, float sx) {
    const F2 sx2 = f2(sx, sx);
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        F2 v[2] = {f2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                   f2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]))};
        if constexpr (kCols) {
            const ulonglong2 s = *reinterpret_cast<const ulonglong2 *>(cols + j);
            const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(cols + kChTile + j);
            v[0] = f2_fma(v[0], f2_mul(sx2, s.x), b.x);
            v[1] = f2_fma(v[1], f2_mul(sx2, s.y), b.y);
        } else {
            v[0] = f2_mul(v[0], sx2);
            v[1] = f2_mul(v[1], sx2);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 f = f2_get(linear_act<kAct>(v[i]));
            r[j + 2 * i] = __float_as_uint(f.x);
            r[j + 2 * i + 1] = __float_as_uint(f.y);
        }
    }
}

// The second of a pair of them, from both: the activations share a reciprocal, so a
// channel's last bits depend on the one that it is paired with.
__device__ __forceinline__ uint32_t wide_second(F2 v, int act, const float *cols, bool has_cols, float sx) {
    const F2 sx2 = f2(sx, sx);
    if (has_cols)
        v = f2_fma(v, f2_mul(sx2, *reinterpret_cast<const F2 *>(cols)), *reinterpret_cast<const F2 *>(cols + kChTile));
    else v = f2_mul(v, sx2);
    if (act == GDN_ACT_SILU) v = linear_act<GDN_ACT_SILU>(v);
    else if (act == GDN_ACT_GELU) v = linear_act<GDN_ACT_GELU>(v);
    return __float_as_uint(f2_get(v).y);
}

// Two columns of 32 lanes of tensor memory.
__device__ __forceinline__ F2 tmem_ld2(uint32_t taddr) {
    uint32_t a, b;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a), "=r"(b)
        : "r"(taddr)
        : "memory");
    return f2_bits(a, b);
}

template <bool kE4m3, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
linear_wide_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                   const __grid_constant__ CUtensorMap mw_tail, const __grid_constant__ CUtensorMap my,
                   const __grid_constant__ LinearEpi ep, int n_in, WidePlan plan, int rows, int keep) {
    constexpr int S = kStagesWide;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[S], empty[S], acc_full[2], acc_empty[2], drained;
    __shared__ __align__(16) float cols[2 * kChTile];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = cta_rank();
    constexpr int kElems = kE4m3 ? 128 : 64;                 // k per block of 128 bytes
    const int nk = (n_in + kElems - 1) / kElems;
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&mx);
        prefetch_tensormap(&mw);
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kEpiWarps);
        }
        mbar_init(&drained, 1);
        abort_flag = (smem_u32(smem) & 1023u) != 0;   // the swizzle needs the alignment asked for above
        fence_mbar_init();
    }
    if (warp == 2) {
        griddep_wait();        // no tensor memory is held while an earlier kernel may still ask for its own
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_base)),
                     "r"(2 * kChTile)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_arrive_relaxed();  // both CTAs' barriers and tensor memory are ready
    cluster_wait();
    tc_fence_after();
    griddep_wait();            // launched behind the kernel that writes x: nothing is read before it
    volatile int *abort = &abort_flag;

    if (warp == 0) {
        // Loads: this CTA's half of both operands, counted on the leader's barrier.
        const bool one = elect_lane();
        const uint32_t lead = peer_smem(smem_u32(full), 0);
        int s = 0, i = 0;
        uint32_t phase = 1;              // of the stage's last release; the first S have none
        bool ok = true;
        WideWalk walk;
        for (walk.start(plan, pair); walk.more(plan) && ok; walk.next(plan, pairs)) {
            const bool go = one && i < keep;   // all tiles' loads, but for tests of the failure path
            int t0, n0, box, width;
            walk.at(plan, ep.n_out, t0, n0, box, width);
            const CUtensorMap *map = box == kChTile ? &mw : &mw_tail;
            const uint32_t bytes = 2 * (kStageA + box / 2 * 128);
            const int tr = t0 + (int)rank * kTokHalf, nr = n0 + (int)rank * (width / 2);
            int kc = 0;
#pragma unroll 1
            for (int k = 0; k < nk; ++k, ++i, kc += kElems) {
                if (i >= S && !mbar_wait_all(&empty[s], phase, abort)) {
                    ok = false;
                    break;
                }
                if (go) {
                    uint8_t *st = smem + s * kStageBytes;
                    const uint32_t bar = lead + s * 8;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                    tma_load_2d_pair(st, &mx, bar, kc, tr);
                    tma_load_2d_pair(st + kStageA, map, bar, kc, nr);
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        griddep_launch();      // what is launched behind this kernel may set itself up
        // the last stages' releases have come
        for (int j = i > S ? i - S : 0; ok && j < i; ++j) ok = mbar_wait_all(&empty[j % S], (j / S) & 1, abort);
        if (one && (!ok || *abort)) {
            // Given up: the copies in flight land before the CTA ends.  The leader
            // waits on the barriers that count them; the peer, which has none of
            // its own, waits far longer (10 ms) than a copy takes.
            if (rank == 0) {
                for (int j = i > S ? i - S : 0; j < i; ++j) mbar_drain(&full[j % S], (j / S) & 1);
            } else {
                let_copies_land();
            }
        }
    } else if (warp == 1 && rank == 0) {
        const bool one = elect_lane();
        const uint32_t first = smem_u32(smem) >> 4;       // descriptors count in 16 bytes
        const uint64_t desc = sdesc_sw128(0, 0, 1024);
        const uint32_t idesc0 = kE4m3 ? idesc_e4m3(256, 0) : idesc_bf16(256, 0);
        int t0, n0, box, width, s = 0;
        uint32_t phase = 0, st = first;
        bool ok = true;
        WideWalk walk;
        walk.start(plan, pair);
        walk.at(plan, ep.n_out, t0, n0, box, width);
        for (int u = 0; walk.more(plan) && ok; ++u) {
            const int b = u & 1;
            if (u >= 2 && !mbar_wait_all(&acc_empty[b], ((u >> 1) - 1) & 1, abort)) break;
            tc_fence_after();
            const uint32_t d = tmem_base + b * kChTile, idesc = idesc0 | ((uint32_t)(width >> 3) << 17);
#pragma unroll 1
            for (int k = 0; k < nk; ++k) {
                if (!mbar_wait_all(&full[s], phase, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_lane()) {
                    const uint64_t da = desc | st, db = desc | (st + (kStageA >> 4));
#pragma unroll
                    for (int q = 0; q < 4; ++q) mma_pair<kE4m3>(d, da + 2 * q, db + 2 * q, idesc, k > 0 || q > 0);
                    mma_commit_pair(&empty[s]);
                }
                __syncwarp();
                st += kStageBytes >> 4;
                if (++s == S) {
                    s = 0;
                    st = first;
                    phase ^= 1;
                }
                if (k == 0) {                             // the next tile, behind this one's products
                    walk.next(plan, pairs);
                    if (walk.more(plan)) walk.at(plan, ep.n_out, t0, n0, box, width);
                }
            }
            if (ok && one) mma_commit_pair(&acc_full[b]);
            __syncwarp();
        }
        if (one) {
            mma_commit_pair(&drained, 1);     // every product issued is done before the leader lets the pair end
            mbar_drain(&drained, 0);
        }
    } else if (warp >= 4) {
        // Accumulator lane 32 q + l is token row 32 q + l of this CTA's half; the
        // two warps of a quadrant take alternate slices of 128 bytes of y.
        constexpr int COLS = 128 / sizeof(O), PARTS = COLS / 32, WORDS = 8 * sizeof(O);
        constexpr int STEP = kEpiWarps / 4 * COLS;
        const int q = warp & 3, half = (warp - 4) >> 2, etid = tid - 128;
        uint8_t *staging = smem + S * kStageBytes + (warp - 4) * kStaging;
        const bool has_cols = ep.sw || ep.bias || ep.act != GDN_ACT_NONE;
        const O *res = reinterpret_cast<const O *>(ep.res);
        const int start = half * COLS;
        // What a tile needs besides its sums is asked for a tile ahead: the columns'
        // scales and biases and the row's scale into registers, the residual to L2
        // and, a chunk ahead, into registers.
        struct Ahead {
            int t0, n0, width;
            float sx, sw, bias;
        } cur, nxt;
        WideWalk walk;
        auto ahead = [&](Ahead &a) {                    // for the tile that the walk has reached
            int box;
            a.width = 0;
            if (!walk.more(plan)) return;
            walk.at(plan, ep.n_out, a.t0, a.n0, box, a.width);
            a.t0 += (int)rank * kTokHalf + q * 32;
            const int t = a.t0 + lane, n = a.n0 + etid;
            a.sx = ep.sx && t < ep.n_tokens ? ep.sx[t] : 1.0f;
            if (has_cols) {
                a.sw = n < ep.n_out && ep.sw ? ep.sw[n] : 1.0f;
                a.bias = n < ep.n_out && ep.bias ? ep.bias[n] : 0.0f;
            }
            if (ep.res && t < ep.n_tokens && half == 0) {
                const O *p = res + t * ep.rs + a.n0;
                const int span = min(a.width, ep.n_out - a.n0);
                for (int i = 0; i < span; i += 128 / (int)sizeof(O))
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i));
            }
        };
        uint32_t rv[32];
        auto ask = [&](const Ahead &a, int c) {         // the residual of a chunk
            const int t0 = a.t0, n = a.n0 + c;
            if (n >= ep.n_out) return;
            if (rows <= kRows16) {
                const int t = t0 + lane;
                if (t < ep.n_tokens) load_row<O>(rv, res + t * ep.rs + n, n, ep.n_out, rows);
                return;
            }
            if constexpr (sizeof(O) == 2) {
                if (n + 32 <= ep.n_out && rows != kRowsPlain) {
                    if (rows == kRows4) WideWords<false>(ep, t0, n, c, a.width, lane).ask(rv, ep, t0, n, lane);
                    else WideWords<true>(ep, t0, n, c, a.width, lane).ask(rv, ep, t0, n, lane);
                    return;
                }
            }
            plain_ask<O>(rv, ep, t0, n, lane);
        };
        static_assert(32 * kEpiWarps == kChTile, "a thread holds one column's scale and bias");
        walk.start(plan, pair);
        ahead(cur);
        if (ep.res && start < cur.width) ask(cur, start);
        // A warp that has given up walks the tiles that are left without work: the others
        // may have seen this tile's sums and wait for it at the barriers of the next.
        bool gone = false;
        for (int u = 0; cur.width > 0; ++u, cur = nxt) {
            const int b = u & 1, t0 = cur.t0, n0 = cur.n0, width = cur.width;
            const float sx = cur.sx;
            if (has_cols) {
                asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");   // the last tile's are read
                cols[etid] = cur.sw;
                cols[kChTile + etid] = cur.bias;
                asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
            }
            walk.next(plan, pairs);
            ahead(nxt);
            gone = gone || !mbar_wait_warp(&acc_full[b], (u >> 1) & 1, abort);
            if (gone) continue;
            tc_fence_after();
#pragma unroll 1
            for (int c = start, part = 0; c < width;) {
                const int n = n0 + c;
                const int next_c = part + 1 < PARTS && c + 32 < width ? c + 32 : c - part * 32 + STEP;
                uint32_t r[32], before = 0;
                tmem_ld32(tmem_addr(tmem_base, q * 32, b * kChTile + c), r);
                if (rows == kRowsOdd && c > 0)
                    before = wide_second(tmem_ld2(tmem_addr(tmem_base, q * 32, b * kChTile + c - 2)), ep.act,
                                         cols + c - 2, has_cols, sx);
                if (ep.act == GDN_ACT_SILU) wide_values<GDN_ACT_SILU, true>(r, cols + c, sx);
                else if (ep.act == GDN_ACT_GELU) wide_values<GDN_ACT_GELU, true>(r, cols + c, sx);
                else if (has_cols) wide_values<GDN_ACT_NONE, true>(r, cols + c, sx);
                else wide_values<GDN_ACT_NONE, false>(r, cols + c, sx);
                if (rows <= kRows16) {
                    if (res) {
#pragma unroll
                        for (int i = 0; i < WORDS; ++i) {
                            if constexpr (sizeof(O) == 2) {
                                const float2 f = unpack_bf16(rv[i]);
                                r[2 * i] = __float_as_uint(__uint_as_float(r[2 * i]) + f.x);
                                r[2 * i + 1] = __float_as_uint(__uint_as_float(r[2 * i + 1]) + f.y);
                            } else {
                                r[i] = __float_as_uint(__uint_as_float(r[i]) + __uint_as_float(rv[i]));
                            }
                        }
                    }
                } else if (n < ep.n_out) {
                    if (sizeof(O) == 4 || rows == kRowsPlain || n + 32 > ep.n_out) {
                        wide_plain<O>(r, rv, reinterpret_cast<float *>(staging), ep, t0, n, lane);
                    } else if constexpr (sizeof(O) == 2) {
                        if (rows == kRows4)
                            WideWords<false>(ep, t0, n, c, width, lane).out(r, 0, rv, staging, ep, t0, n, lane);
                        else
                            WideWords<true>(ep, t0, n, c, width, lane).out(r, before, rv, staging, ep, t0, n, lane);
                    }
                }
                if (res) {
                    if (next_c < width) ask(cur, next_c);
                    else if (start < nxt.width) ask(nxt, start);
                }
                if (rows <= kRows16) {
                    if constexpr (sizeof(O) == 2) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            r[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                    }
                    if (part == 0) {                    // the last store has read the staging rows
                        if (lane == 0) bulk_wait_read_all();
                        __syncwarp();
                    }
#pragma unroll
                    for (int i = 0; i < WORDS / 4; ++i)
                        *reinterpret_cast<uint4 *>(staging + lane * 128 +
                                                   (((part * WORDS / 4 + i) ^ (lane & 7)) << 4)) =
                            make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                    if (part + 1 == PARTS || c + 32 >= width) {
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (t0 < ep.n_tokens) tma_store_2d(&my, staging, n - part * 32, t0);
                            bulk_commit();
                        }
                    }
                }
                part = next_c == c + 32 && PARTS > 1 ? 1 : 0;
                c = next_c;
            }
            if (ep.res && start >= width && start < nxt.width) ask(nxt, start);   // no chunk here
            tc_fence_before();                          // this warp has read its part of the accumulator
            __syncwarp();
            // the tile after next waits for it (an arrival that nobody waits for could come too late)
            if (lane == 0 && walk.tile + pairs < plan.n_tiles) mbar_arrive_cluster(peer_smem(smem_u32(&acc_empty[b]), 0));
        }
        if (lane == 0) bulk_wait_read_all();    // the staging rows stay until they are read
        __syncwarp();
        tc_fence_before();
    }
    __syncthreads();
    // Neither CTA ends while the other may reach its memory: every arrival from the
    // other one has been waited for above, so nothing is handed over here, unless the
    // pair has given up.  (With release a CTA waited for its stores to y first, some
    // 1,200 cycles.)
    if (*abort) cluster_arrive();
    else cluster_arrive_relaxed();
    cluster_wait();
    tc_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(2 * kChTile)
                     : "memory");
    if (tid == 0 && abort_flag) {
        flag_status(GDN_DEVSTAT_TIMEOUT);
        let_copies_land();     // arrivals that were not waited for
    }
}

// The plan with the shortest estimate, and that in cycles of a k block.  A block
// takes 512 cycles of a pair on 256 channels, the rate of the tensor cores; on
// fewer it is the operands' copies that hold it (512 x 2048 x 8192 in channel
// tiles of 192, 128 and 64: 445, 410 and 410), and where rows are off the memory's
// lines, on 256 too (512 x 2056 x 8192: 18.4 us, on lines 16.5).  The last `rows`
// token tiles are cut into channel tiles of w where that fills the last wave of
// pairs better (8000 x 2048 x 2048: 40.4 us, in tiles of 256 alone 42.9, of 192 44.1).
int64_t plan_wide(const LinearCall &call, int pairs, WidePlan &best) {
    constexpr int kBlockCycles[2][4] = {{424, 540, 640, 750}, {410, 410, 445, 512}};
    const int n_tokens = call.e.n_tokens, n_out = call.e.n_out, *cycles = kBlockCycles[call.lines()];
    const int nt = (n_tokens + kTokTile - 1) / kTokTile, nn = (n_out + kChTile - 1) / kChTile;
    auto waves = [&](int64_t tiles) { return (tiles + pairs - 1) / pairs; };
    int64_t cost = INT64_MAX;
    for (int rows = 0; rows <= std::min(nt, 16); ++rows)
        for (int w = 64; w <= (rows ? kChTile - 64 : 64); w += 64) {   // whole staging rows
            const int64_t full = (int64_t)(nt - rows) * nn, tail = (int64_t)rows * ((n_out + w - 1) / w);
            const int64_t c = waves(full) * cycles[3] + waves(tail) * cycles[w / 64 - 1];
            if (c < cost) {
                cost = c;
                best = {nt - rows, nt, nn, (int)full, w, (int)(full + tail)};
            }
        }
    return cost;
}

// Whether the tiles can be counted in 32 bits.
bool wide_fits(const LinearEpi &e) {
    return ((int64_t)e.n_tokens + 255) / 256 * (((int64_t)e.n_out + 31) / 32) < (1 << 30);
}

template <bool kE4m3, typename O> gdn_status launch_wide(const LinearCall &c, const WidePlan &plan) {
    const LinearEpi &e = c.e;
    const int sms = sm_count() / 2 * 2;
    CUtensorMap mx, mw, mt, my = {};
    if (!encode_tmap_operand(&mx, c.x, c.n_in, e.n_tokens, c.xs, kTokHalf, kE4m3) ||
        !encode_tmap_operand(&mw, c.w, c.n_in, e.n_out, c.ws, kChTile / 2, kE4m3) ||
        !encode_tmap_operand(&mt, c.w, c.n_in, e.n_out, c.ws, plan.tail_w / 2, kE4m3))
        return GDN_ERR_CUDA;
    auto at = [&](int64_t bytes) {
        return (uintptr_t)e.y % bytes == 0 && e.ys * (int64_t)sizeof(O) % bytes == 0 &&
               (!e.res || ((uintptr_t)e.res % bytes == 0 && e.rs * (int64_t)sizeof(O) % bytes == 0));
    };
    const bool alike = !e.res || ((((uintptr_t)e.y ^ (uintptr_t)e.res) & 3) == 0 && ((e.ys ^ e.rs) & 1) == 0);
    // a TMA store writes whole 16 bytes: it would reach behind rows that end within some
    const bool whole = (int64_t)e.n_out * sizeof(O) % 16 == 0;
    const int rows = whole && at(32)       ? kRows32
                     : whole && at(16)     ? kRows16
                     : sizeof(O) == 4      ? kRowsPlain
                     : at(4)               ? kRows4
                     : alike               ? kRowsOdd
                                           : kRowsPlain;
    if (rows <= kRows16 &&
        !encode_tmap_2d(&my, sizeof(O) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, e.y,
                        e.n_out, e.n_tokens, e.ys * sizeof(O), 128 / sizeof(O), 32, true))
        return GDN_ERR_CUDA;
    const int keep = c.drop == kDropNone ? INT_MAX : c.drop & kDropAll ? 0 : (c.n_in + (kE4m3 ? 127 : 63)) / (kE4m3 ? 128 : 64);
    auto kernel = linear_wide_kernel<kE4m3, O>;
    static SmemAllowed allowed;
    cudaError_t err = allowed.ask(kernel, kWideSmem);
    if (err == cudaSuccess)
        err = launch_after(kernel, dim3(std::min(2 * plan.n_tiles, sms)), dim3(kWideThreads), kWideSmem,
                           c.stream, mx, mw, mt, my, e, c.n_in, plan, rows, keep);
    if (err != cudaSuccess) {
        set_last_cuda_error(err);
        return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

}  // namespace

// 8,700 cycles in front of the first product and behind the last.
int64_t plan_linear_wide(const LinearCall &c, WidePlan &plan) {
    const int pairs = sm_count() / 2;
    if (pairs < 1 || !wide_fits(c.e)) return INT64_MAX;
    const int64_t blocks = (c.n_in + (c.e4m3 ? 127 : 63)) / (c.e4m3 ? 128 : 64);
    return 8700 + plan_wide(c, pairs, plan) * blocks;
}

gdn_status launch_linear_wide(const LinearCall &c, const WidePlan &plan) {
    if (c.e4m3) return c.e.out_f32 ? launch_wide<true, float>(c, plan) : launch_wide<true, __nv_bfloat16>(c, plan);
    return c.e.out_f32 ? launch_wide<false, float>(c, plan) : launch_wide<false, __nv_bfloat16>(c, plan);
}

}  // namespace gdn
