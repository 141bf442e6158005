// window_simple.cu -- gradients of the window attention straight from the
// definition: one warp per query row (dQ) or key row (dK, dV), fp32 throughout.
#include "stream_device.cuh"

namespace ac {
namespace {

constexpr int kWarps = 4;

// Address of key row j (bf16) of (b, hk).
__device__ __forceinline__ const bf16 *row_bf16(const View &v, int b, int h, int j) {
    return static_cast<const bf16 *>(v.p) + b * v.b + h * v.h + (int64_t)j * v.l;
}

// x[0..N) of this lane: elements lane * N .. of a key or value row.
template <int N>
__device__ __forceinline__ void load_row(const WinArgs &a, bool v, int b, int hk, int j, int lane, float (&x)[N]) {
    const bf16 *r = row_bf16(v ? a.v : a.k, b, hk, j) + lane * N;
    for (int i = 0; i < N; ++i) x[i] = bf2f(r[i]);
}

__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

template <int N>
__device__ __forceinline__ float dot(const float (&a)[N], const float (&b)[N]) {
    float s = 0.f;
    for (int i = 0; i < N; ++i) s = fmaf(a[i], b[i], s);
    return warp_sum(s);
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) k_simple_dq(const WinBwdArgs g) {
    constexpr int N = D / 32;
    const WinArgs &a = g.f;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (int64_t)a.B * a.Hq * a.Lq) return;
    const int i = (int)(row % a.Lq), h = (int)(row / a.Lq % a.Hq), b = (int)(row / a.Lq / a.Hq), hk = h / a.G;
    const int ql = seq_len(a.q_lens, b, a.Lq, a.err), kl = seq_len(a.k_lens, b, a.Lk, a.err);
    RowRange r{0, 0};
    if (i < ql) r = row_range(a.w, i + kl - ql, kl);
    float q[N], go[N], dq[N], k[N], x[N];
    for (int e = 0; e < N; ++e) {
        q[e] = bf2f(row_bf16(a.q, b, h, i)[lane * N + e]);
        go[e] = bf2f(row_bf16(g.go, b, h, i)[lane * N + e]);
        x[e] = bf2f(row_bf16(a.o, b, h, i)[lane * N + e]);
        dq[e] = 0.f;
    }
    const float delta = dot(go, x), lse = a.lse[row];
    for (int j = min(a.w.sinks, r.lo) > 0 ? 0 : r.lo; j < r.hi; ++j) {
        if (j >= a.w.sinks && j < r.lo) j = r.lo;
        if (j >= r.hi) break;
        load_row(a, false, b, hk, j, lane, k);
        load_row(a, true, b, hk, j, lane, x);
        const float ds = __expf(dot(q, k) * a.scale - lse) * (dot(go, x) - delta) * a.scale;
        for (int e = 0; e < N; ++e) dq[e] += ds * k[e];
    }
    bf16 *dst = static_cast<bf16 *>(g.dq.p) + b * g.dq.b + h * g.dq.h + (int64_t)i * g.dq.l + lane * N;
    for (int e = 0; e < N; ++e) dst[e] = __float2bfloat16_rn(dq[e]);
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) k_simple_dkv(const WinBwdArgs g) {
    constexpr int N = D / 32;
    const WinArgs &a = g.f;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (int64_t)a.B * a.Hk * a.Lk) return;
    const int j = (int)(row % a.Lk), hk = (int)(row / a.Lk % a.Hk), b = (int)(row / a.Lk / a.Hk);
    const int ql = seq_len(a.q_lens, b, a.Lq, a.err), kl = seq_len(a.k_lens, b, a.Lk, a.err);
    float k[N], v[N], q[N], go[N], x[N], dk[N] = {}, dv[N] = {};
    load_row(a, false, b, hk, j, lane, k);
    load_row(a, true, b, hk, j, lane, v);
    for (int i = 0; i < ql; ++i) {
        const RowRange r = row_range(a.w, i + kl - ql, kl);
        if (j >= r.hi || (j < r.lo && j >= a.w.sinks)) continue;
        for (int h = hk * a.G; h < (hk + 1) * a.G; ++h) {
            for (int e = 0; e < N; ++e) {
                q[e] = bf2f(row_bf16(a.q, b, h, i)[lane * N + e]);
                go[e] = bf2f(row_bf16(g.go, b, h, i)[lane * N + e]);
                x[e] = bf2f(row_bf16(a.o, b, h, i)[lane * N + e]);
            }
            const float p = __expf(dot(q, k) * a.scale - a.lse[((int64_t)b * a.Hq + h) * a.Lq + i]);
            const float ds = p * (dot(go, v) - dot(go, x)) * a.scale;
            for (int e = 0; e < N; ++e) dv[e] += p * go[e], dk[e] += ds * q[e];
        }
    }
    bf16 *pk = static_cast<bf16 *>(g.dk.p) + b * g.dk.b + hk * g.dk.h + (int64_t)j * g.dk.l + lane * N;
    bf16 *pv = static_cast<bf16 *>(g.dv.p) + b * g.dv.b + hk * g.dv.h + (int64_t)j * g.dv.l + lane * N;
    for (int e = 0; e < N; ++e) pk[e] = __float2bfloat16_rn(dk[e]), pv[e] = __float2bfloat16_rn(dv[e]);
}

unsigned blocks(int64_t rows) { return (unsigned)((rows + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_window_bwd_simple(const WinBwdArgs &g, cudaStream_t s) {
    const WinArgs &a = g.f;
    const unsigned nq = blocks((int64_t)a.B * a.Hq * a.Lq), nk = blocks((int64_t)a.B * a.Hk * a.Lk);
    auto go = [&](auto kern, unsigned n) {
        if (n == 0) return;
        kern<<<n, 32 * kWarps, 0, s>>>(g);
        AC_NOTE_LAUNCH();
    };
    if (a.d == 128)
        go(k_simple_dq<128>, nq), go(k_simple_dkv<128>, nk);
    else
        go(k_simple_dq<64>, nq), go(k_simple_dkv<64>, nk);
    return cudaGetLastError();
}

}  // namespace ac
