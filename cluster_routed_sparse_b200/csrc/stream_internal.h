// stream_internal.h -- host side of the streaming operators: argument blocks and
// kernel launchers.
#pragma once

#include <algorithm>

#include "ac_internal.h"

namespace ac {

// Error words of the streaming operators, one pair per device (they have no
// context).  `timeout` holds the number of the launch whose bounded wait
// expired, so that the other CTAs of that launch give up early; `bits` holds
// DEV_ERR_* until ac_ops_status reads it.
struct OpErr {
    uint32_t timeout, bits;
};
cudaError_t op_err_address(OpErr **out);
uint32_t next_launch_id();

struct View {  // [B, H, L, d], d contiguous; strides in elements
    void *p;
    int64_t b, h, l;
};

struct WinRule {
    int left, right, sinks, g;
};

struct RopeArgs {
    View x[2], y[2];
    int H[2], B, L, d, P;       // P rotated pairs
    const int *pos;             // [L, n_axes], plus pos_b per sequence
    int64_t pos_b;
    int n_axes;
    uint64_t turns[128];        // turns per step of each pair, 0.64 fixed point
    uint8_t axis[128];
    int interleaved, inverse;
};
cudaError_t launch_rope(int dtype, const RopeArgs &a, cudaStream_t s);

struct AppendArgs {
    uint8_t *k8, *v8;
    float *ks, *vs;
    View k, v;
    const int *table, *start, *counts;
    int pages, Hk, T, d, B, n, max_pages;
    OpErr *err;
};
cudaError_t launch_cache8_append(const AppendArgs &a, cudaStream_t s);

// Attention over bf16 keys (k, v) or, when k8 is set, over the paged 8-bit cache.
struct WinArgs {
    View q, k, v, o;
    const uint8_t *k8, *v8;
    const float *ks, *vs;
    const int *table;
    int pages, T, max_pages;
    float *lse;                 // [B, Hq, Lq]; may be null
    const int *q_lens, *k_lens;
    int B, Hq, Hk, G, Lq, Lk, d;
    WinRule w;
    float scale;
    void *ws;
    OpErr *err;
};
cudaError_t launch_window_simple(const WinArgs &a, cudaStream_t s);

struct WinBwdArgs {
    WinArgs f;                  // q, k, v, o, lse as the forward left them
    View go, dq, dk, dv;
};
cudaError_t launch_window_bwd_simple(const WinBwdArgs &a, cudaStream_t s);

}  // namespace ac
