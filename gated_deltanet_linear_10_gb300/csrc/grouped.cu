// Products of rows with the weights of their expert, in bf16 or in e4m3 with an
// fp32 scale for each block of 128 in k, and the product of all rows with one
// weight in the latter form: argument checks, operand maps and the choice of a kernel.
#include <limits.h>

#include <algorithm>
#include <atomic>

#include "grouped.cuh"

namespace gdn {

void GroupedCall::channel_tiles(int64_t nn) {
    by_channels = QuickDiv((uint32_t)nn);
    by_raster = QuickDiv((uint32_t)nn * kGroupRaster);
}

// A single row (or expert) has no stride; a map wants one all the same.
bool encode_tmap_experts(CUtensorMap *map, const GroupedCall &c, uint32_t box_rows) {
    const int64_t elem = c.e4m3 ? 1 : 2, row = ((int64_t)c.n_in + 15) / 16 * 16;
    const int64_t ws = c.n_out == 1 ? row : c.ws, we = c.n_experts == 1 ? ws * c.n_out : c.we;
    return encode_tmap_3d(map, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, c.w, c.n_in,
                          c.n_out, c.n_experts, ws * elem, we * elem, 128 / (uint32_t)elem, box_rows);
}
bool encode_tmap_rows(CUtensorMap *map, const GroupedCall &c, uint32_t box_rows) {
    return encode_tmap_operand(map, c.x, c.n_in, c.n_x, c.xs, box_rows, c.e4m3);
}

// Of R rows floor(R / r) tiles are full at most, and each expert with rows may have one more.
int64_t most_row_tiles(const GroupedCall &c, int tile_rows) {
    const int64_t n = c.n_rows;
    return c.offsets ? std::min(n, n / tile_rows + std::min<int64_t>(c.n_experts, n)) : (n + tile_rows - 1) / tile_rows;
}

// Test control (gdn_debug_set_grouped_tile): the tile's rows, 0 for the estimate's choice,
// and 16 bits up the cut + 1.
static std::atomic<int> g_grouped_tile{0};

// The choice of a tile: the shortest by an estimate of waves of tiles, each of as many
// blocks of 128 bytes in k.  The figures (in 10 ns: a call's ends, a tile's, what rows of y
// off 16 bytes add to that, a block) come from a fit, but for the blocks of e4m3 tiles of 32
// rows, which were raised by hand (256 x 10 rows of 512 experts: 138.4 -> 135.7 us; of 408
// e4m3 products 19 change, and take 1.9 % longer than their best tile instead of 3.5).
// Measured with every tile and cut on 626 products (1 to 4096 tokens, 2 to 400 rows for each of
// 8, 60 and 256 experts, random ones of 64 to 4096 in, 33 to 8192 out), the choice takes
// 2.2 % longer than the best, more than 15 % for one in twenty (most of them calls under 6 us
// of one or two blocks), 40 % at worst (6481 x 110 x 4283 to fp32: 53.7 us on pairs, 38.3 in
// tiles of 128).  Of an expert's rows the host knows the mean: tiles of r rows take mean /
// r + 1/2 of them, at least one.  (256 experts of 82 rows gathered, 1000 x 700 e4m3, in the five tiles: 193,
// 154, 81, 84 and 105 us; 256 x 2048 x 8192 in those of 64, 128 and 256: 15.8, 9.8, 13.4.)
static gdn_status launch_grouped(GroupedCall c, cudaStream_t s) {
    const int64_t ye = c.out_f32 ? 4 : 2;
    c.vec16 = (uintptr_t)c.y % 16 == 0 && c.n_out * ye % 16 == 0 && (c.n_rows == 1 || c.ys * ye % 16 == 0);
    c.vec4 = (uintptr_t)c.y % 4 == 0 && (c.n_rows == 1 || c.ys * ye % 4 == 0);
    c.sx16 = (uintptr_t)c.sx % 16 == 0 && c.kb % 4 == 0;
    struct Tile {
        int rows, channels, ends, tile, odd[2], block[2][2];   // odd, block: bf16, e4m3; block: rows in place, gathered
    };
    constexpr Tile kTiles[] = {{16, 128, 280, 90, {0, 0}, {{26, 31}, {30, 33}}},
                               {32, 128, 310, 70, {0, 0}, {{26, 31}, {31, 35}}},
                               {64, 128, 270, 90, {0, 0}, {{30, 38}, {36, 42}}},
                               {128, 128, 290, 90, {60, 60}, {{33, 37}, {31, 41}}},
                               // (pairs write such rows slowly, and with block scales sum nothing meanwhile)
                               {256, 256, 450, 90, {180, 190}, {{39, 39}, {47, 61}}}};
    constexpr int kJoin = 40, kJoinRows = 21;          // k in parts: a call's, 16 rows of a part
    const int sms = sm_count(), experts = c.offsets ? std::min(c.n_experts, c.n_rows) : 1;
    const int64_t blocks = c.e4m3 ? c.kb : (c.n_in + 63) / 64;
    const int wanted = g_grouped_tile.load(std::memory_order_relaxed), only_rows = wanted & 0xffff, only_cut = (wanted >> 16) - 1;
    int best = 0, best_cut = 0;
    int64_t least = INT64_MAX;
    for (const Tile &t : kTiles) {
        if (only_rows && t.rows != only_rows) continue;
        const int64_t halves = c.offsets ? std::max<int64_t>(2 * (int64_t)experts, 2 * (int64_t)c.n_rows / t.rows + experts)
                                         : 2 * (((int64_t)c.n_rows + t.rows - 1) / t.rows);
        const int64_t tiles = (halves + 1) / 2 * ((c.n_out + t.channels - 1) / t.channels);
        if (tiles >= (1ll << 30)) continue;                // (so many are not launched)
        const int64_t most = most_row_tiles(c, t.rows) * ((c.n_out + t.channels - 1) / t.channels);
        const int64_t slots = t.rows == 256 ? std::max(1, sms / 2) : sms, block = t.block[c.e4m3][c.rows != nullptr];
        const int64_t rest = t.tile + (c.vec16 ? 0 : t.odd[c.e4m3]);
        for (int cut = 0; cut <= 3; ++cut) {
            // k in parts, a block each at least
            if (cut > 0 && (t.rows == 256 || blocks >> cut < 1 || most << cut >= (1ll << 31))) break;
            // ... in one wave, four blocks a CTA at least (16 clusters of eight, where 15
            // fit, are two waves: 1 x 4096 x 2048 11.9 us, in clusters of four 6.9)
            if (cut > 0 && only_cut < 0 && (most << cut > sms || blocks >> cut < 4)) break;
            if (cut == 3 && only_cut < 0 && most > grouped_eights()) break;
            if (only_cut >= 0 && cut != only_cut) continue;
            const int64_t cost = t.ends + (tiles + slots - 1) / slots * (rest + ((blocks + (1 << cut) - 1) >> cut) * block) +
                                 (cut > 0 ? kJoin + (t.rows << cut) * kJoinRows / 16 : 0);
            if (cost >= least) continue;
            least = cost;
            best = t.rows;
            best_cut = cut;
        }
    }
    if (best == 0) return GDN_ERR_UNSUPPORTED;
    return best == 256 ? launch_grouped_wide(c, linear_drop(), s) : launch_grouped_narrow(c, best, best_cut, linear_drop(), s);
}

}  // namespace gdn

using namespace gdn;

static gdn_status grouped_check(const GroupedCall &c, int64_t n_rows, int64_t n_x) {
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

extern "C" gdn_status gdn_debug_set_grouped_tile(int32_t tile_rows, int32_t cut) {
    GDN_REQUIRE(tile_rows == 0 || tile_rows == 16 || tile_rows == 32 || tile_rows == 64 || tile_rows == 128 || tile_rows == 256,
                GDN_ERR_INVALID_ARG);
    GDN_REQUIRE(cut >= -1 && cut <= (tile_rows == 256 ? 0 : 3) && (tile_rows || cut == -1), GDN_ERR_INVALID_ARG);
    g_grouped_tile.store(tile_rows | (cut + 1) << 16, std::memory_order_relaxed);
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
    const gdn_status st = grouped_check(c, n_tokens, n_tokens);
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
    const gdn_status st = grouped_check(c, n_rows, n_x);
    return st == GDN_OK ? launch_grouped(c, (cudaStream_t)stream) : st;
}
