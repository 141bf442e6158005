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

// Launches a kernel of several that make up one call, never the first of them: it may
// begin before the one in front of it has ended.  It reads the call's inputs at once,
// and waits (wait_predecessor) before it touches anything that the call writes.
template <class... P, class... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, A &&...args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid, c.blockDim = dim3(block), c.dynamicSmemBytes = smem, c.stream = s;
    c.attrs = &at, c.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, kern, P(args)...);
    if (e == cudaSuccess) AC_NOTE_LAUNCH();
    return e;
}

struct View {  // [B, H, L, d], d contiguous; strides in elements
    void *p;
    int64_t b, h, l;
};

struct WinRule {
    int left, right, sinks, g;
};

// Most tiles of `bn` keys that any `tokens` consecutive queries see.
inline int64_t window_tiles(const WinRule &w, int64_t tokens, int Lq, int Lk, int bn) {
    tokens = std::min<int64_t>(std::max(tokens, int64_t(1)), std::max(Lq, 1));
    if (w.left < 0 || w.right < 0) return (Lk + bn - 1) / bn;
    const int64_t blocks = (tokens - 1 + w.g - 1) / w.g + 1 + (int64_t)w.left + w.right;
    const int64_t span = blocks > Lk / w.g ? Lk : std::min<int64_t>(blocks * w.g, Lk);
    const int64_t sinks = std::min<int64_t>(w.sinks, Lk);
    return std::min<int64_t>(span / bn + 2 + (sinks + bn - 1) / bn, (Lk + bn - 1) / bn);
}

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
int64_t window_mma_workspace(const WinArgs &a);   // any number of rows
cudaError_t launch_window_mma(const WinArgs &a, cudaStream_t s);
int64_t window_few_workspace(const WinArgs &a);   // a few times 8 rows for each key head
cudaError_t launch_window_few(const WinArgs &a, cudaStream_t s);
cudaError_t launch_combine(const float *part_o, const float *part_lse, const WinArgs &a, int nsplit, cudaStream_t s);

cudaError_t launch_cache8_expand(const WinArgs &a, __nv_bfloat16 *k, __nv_bfloat16 *v, cudaStream_t s);

struct WinBwdArgs {
    WinArgs f;                  // q, k, v, o, lse as the forward left them
    View go, dq, dk, dv;
};
int64_t window_bwd_workspace(const WinArgs &a);
cudaError_t launch_window_bwd(const WinBwdArgs &a, cudaStream_t s);

}  // namespace ac
