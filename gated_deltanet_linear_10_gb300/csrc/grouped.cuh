// The products grouped by expert and with block scales (internal header).
#pragma once

#include "common.cuh"

namespace gdn {

constexpr int64_t kGroupedRows = 65535 * 256;
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
};

}  // namespace gdn
