// The products grouped by expert and with block scales (internal header):
//   y_r = sum_b sx[i][b] sw[e][n / 128][b] sum_{k in b} x[i][k] w[e][n][k],
//   i = rows[r], offsets[e] <= r < offsets[e + 1]
// (bf16: no scales and one block).  The product of all rows with one weight is
// the case of one expert, without offsets.
#pragma once

#include "linear.cuh"

namespace gdn {

constexpr int64_t kGroupedRows = 65535 * 256;
constexpr int kGroupRaster = 8;
constexpr int kGroupedOut = 1 << 20, kGroupedIn = 1 << 20, kGroupedExperts = 1024;

struct GroupedCall {
    const void *x, *w;
    int64_t xs, ws, we;              // strides of a row of x, of w, and of an expert
    const float *sx, *sw;            // [n_x][kb], [n_experts][nb][kb]
    const int32_t *offsets, *rows;   // null: one group of all rows; row r of x
    void *y;
    int64_t ys;
    int n_rows, n_x, n_experts, n_in, n_out, kb, nb;
    bool e4m3, out_f32;
    bool vec16;                      // rows of y on 16-byte boundaries, whole 16 bytes of them
    bool vec4;                       // rows of y on 4-byte boundaries
    bool sx16;                       // rows of sx on 16-byte boundaries
    QuickDiv by_channels, by_raster; // by a row of channel tiles, by kGroupRaster of them
    void channel_tiles(int64_t nn);  // sets these
};

// grouped_narrow.cu: a tile's weight rows on the accumulator's lanes, its tokens the
// columns; grouped_wide.cu: tokens on the lanes, a pair of CTAs a tile.
// 2^cut CTAs share a tile, each a part of k: only with at least as many blocks, and where
// that is one wave of CTAs.
int64_t most_row_tiles(const GroupedCall &c, int tile_rows);      // that there can be
int grouped_eights();                // clusters of eight of its CTAs that the device holds at once
gdn_status launch_grouped_narrow(const GroupedCall &c, int tile_rows, int cut, int drop, cudaStream_t s);
gdn_status launch_grouped_wide(const GroupedCall &c, int drop, cudaStream_t s);
cudaError_t set_grouped_narrow_limit(uint64_t limit_ns, cudaStream_t s);
cudaError_t set_grouped_wide_limit(uint64_t limit_ns, cudaStream_t s);
int linear_drop();                   // the failure path's test control (LinearDrop)

// The operands' maps, in boxes of 128 bytes x box_rows: w as [n_experts][n_out][n_in],
// x as rows (not used where they are gathered).
bool encode_tmap_experts(CUtensorMap *map, const GroupedCall &c, uint32_t box_rows);
bool encode_tmap_rows(CUtensorMap *map, const GroupedCall &c, uint32_t box_rows);

// ------------------------------------------------------------ device side --
// Which rows an expert has and how many tiles of rows lie in front of it, in shared
// memory; built by the whole CTA from the offsets.
struct GroupTable {
    int first[kGroupedExperts + 1], start[kGroupedExperts + 1];
    int part[32];
    int bad;
};

// All threads; returns the number of row tiles, 0 where the offsets are no offsets
// (then *bad).  Ends with a barrier.
__device__ __forceinline__ int build_group_table(GroupTable &g, const GroupedCall &c, int tile_rows, bool *bad) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    *bad = false;
    if (!c.offsets) {
        if (tid == 0) {
            g.first[0] = g.start[0] = 0;
            g.first[1] = (c.n_rows + tile_rows - 1) / tile_rows;
            g.start[1] = c.n_rows;
        }
        __syncthreads();
        return g.first[1];
    }
    // as many experts a thread as it takes (at least 256 threads), their offsets asked for together
    constexpr int Q = 4;
    const int per = (c.n_experts + nt - 1) / nt, e0 = tid * per, e1 = min(e0 + per, c.n_experts);
    int sum = 0, wrong = 0;
    if (e0 < e1) {
        int o[Q + 1];
#pragma unroll
        for (int i = 0; i <= Q; ++i) o[i] = c.offsets[min(e0 + i, e1)];
        wrong |= o[0] < 0;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            wrong |= o[i + 1] < o[i] || o[i + 1] > c.n_rows;
            sum += (o[i + 1] - o[i] + tile_rows - 1) / tile_rows;
            if (e0 + i <= e1) g.start[e0 + i] = o[i];
        }
        if (e0 + Q <= e1) g.start[e0 + Q] = o[Q];
    }
    wrong = __syncthreads_or(wrong);
    int scan = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, scan, off);
        if (lane >= off) scan += o;
    }
    if (lane == 31) g.part[warp] = scan;
    __syncthreads();
    int front = scan - sum;
    for (int i = 0; i < warp; ++i) front += g.part[i];
    for (int e = e0; e < e1; ++e) {
        g.first[e] = front;
        front += (g.start[e + 1] - g.start[e] + tile_rows - 1) / tile_rows;
    }
    if (e0 < e1 && e1 == c.n_experts) g.first[e1] = front;
    __syncthreads();
    *bad = wrong != 0;
    return wrong ? 0 : g.first[c.n_experts];
}

// A tile: rows r0 .. r1 - 1 (r1: the expert's end, not the tile's), channel tile n.
struct GroupTile {
    int e, r0, r1, n;
};

// By a whole warp.  Within an expert groups of kGroupRaster row tiles take the channel
// tiles one after the other, row tiles fastest: the tiles in flight share weights and rows.
// (Three quotients by division are most of 900 cycles, which the sums of a tile wait for.)
__device__ __forceinline__ GroupTile find_group_tile(const GroupTable &g, const GroupedCall &c, int tile, int nn,
                                                     int tile_rows) {
    const int experts = c.n_experts, lane = threadIdx.x & 31, rt = c.by_channels(tile);
    const int hi = __popc(__ballot_sync(0xffffffffu, g.first[min(32 * (lane + 1), experts)] <= rt));
    const int e = 32 * hi + __popc(__ballot_sync(0xffffffffu, g.first[min(32 * hi + lane + 1, experts)] <= rt));
    GroupTile t;
    t.e = e;
    const int f = g.first[e], tiles = g.first[e + 1] - f, r = tile - f * nn;
    const int base = r < kGroupRaster * nn ? 0 : c.by_raster(r) * kGroupRaster, rr = r - base * nn;
    const int rows = min(kGroupRaster, tiles - base);
    // 2^32 / rows, rounded up: exact below 2^29
    constexpr uint32_t kInverse[kGroupRaster + 1] = {0,       0,          1u << 31,   1431655766u, 1u << 30,
                                                     858993460u, 715827883u, 613566757u, 1u << 29};
    t.n = rr;
#pragma unroll
    for (int i = 2; i <= kGroupRaster; ++i)
        if (rows == i) t.n = __umulhi((uint32_t)rr, kInverse[i]);
    t.r0 = g.start[e] + (base + rr - t.n * rows) * tile_rows;
    t.r1 = g.start[e + 1];
    return t;
}

// The row of x that sorted row r takes, n_x (which reads as zeros) where there is none.
__device__ __forceinline__ int group_x_row(const GroupedCall &c, int r, int r1) {
    if (r >= r1) return c.n_x;
    if (!c.rows) return r;
    const int i = c.rows[r];
    return i < 0 || i >= c.n_x ? c.n_x : i;
}

// How long what is read or written should stay in L2.
__device__ __forceinline__ uint64_t l2_first() {     // it makes room first
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t l2_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// 16 bytes of global into shared memory, those from `bytes` on as zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// (the size as a register makes that a slow sequence)
__device__ __forceinline__ void copy16_if(bool on, uint32_t dst, const void *src) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}\n" ::"r"(dst),
        "l"(src), "r"((uint32_t)on)
        : "memory");
}
// Arrives on a barrier, whose count has it already, when this thread's copies so far have come.
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
// Whether a phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Columns of 32 lanes of tensor memory, on their way until every load of the thread
// has come (tmem_wait; r is named there so that nothing reads it before).
__device__ __forceinline__ void tmem_ask(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :);
}
__device__ __forceinline__ void tmem_ask(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :);
}

}  // namespace gdn
