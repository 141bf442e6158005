// rope_axes.cu -- rotary positions with several axes (time, height, width).
//
// Pair p of a token belongs to one axis a(p) and turns by the angle
// pos[a(p)] * freq[p]:  (x, y) -> (x cos - y sin, x sin + y cos); the inverse
// (the transpose, hence also the gradient) turns the other way.
//
// The angle is kept in turns as a 0.64 fixed-point number: freq / (2 pi) is
// rounded to 2^-64 once on the host, and pos * turns modulo 2^64 is exact for
// every 32-bit position, so a position of a million loses nothing (in fp32 the
// angle itself would be off by 2^-24 relative, 0.06 rad there).  sincospif
// takes the top 32 bits, rounded, as a float; the up to 7 bits that a float does not hold
// turn its sine and cosine a little further, which leaves 2^-32 turns of error.
//
// Bound by memory: every element is read and written once.  A thread owns one
// token and one 16-byte chunk (two chunks when the pair's halves lie d/2 apart),
// computes its sines and cosines once and then walks over the heads of q and
// k, four loads in flight.  Projections leave [B, L, H, d], the attention layer
// takes [B, H, L, d]; both are views here, so the change of order costs nothing.
// Q and K of 40 heads, 75,600 tokens, d = 128, bf16 (3.1 GB): 510 us, 6.1 TB/s, 94% of a
// copy; fp32, halves, 30 heads, 17,550 tokens, d = 64 (0.54 GB): 88.6 us, 94%; one token
// of 40 heads: 3.4 us in a graph.
#include "stream_device.cuh"

namespace ac {
namespace {

template <class T>
struct Vec;  // 16 bytes of T as floats and back
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&f)[4]) {
        f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct Vec<bf16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&f)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Vec<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&f)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            f[2 * i] = v.x, f[2 * i + 1] = v.y;
        }
    }
    static __device__ __forceinline__ uint32_t two(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
    }
};

__device__ __forceinline__ void pair_sincos(const RopeArgs &a, const int *pos, int p, float &s, float &c) {
    const uint64_t t = (uint64_t)(int64_t)pos[a.axis[p]] * a.turns[p];
    const int32_t units = (int32_t)((t + (1ull << 31)) >> 32);  // of 2^-31 half turns
    const float f = __int2float_rz(units);  // (towards 0: within int32 again)
    sincospif(f * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
    const float rest = (float)(units - __float2int_rz(f)) * 1.4629180792671596e-9f;  // pi 2^-31
    const float s0 = s;
    s = fmaf(c, rest, s), c = fmaf(-s0, rest, c);
    if (a.inverse) s = -s;
}

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// One thread: token l, chunk c, heads [h0, h1) of the heads of q and then k.
template <class T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) k_rope(const __grid_constant__ RopeArgs a, int heads_per_block) {
    constexpr int N = Vec<T>::N;
    constexpr int M = INTERLEAVED ? 1 : 2;           // chunks of a thread
    constexpr int NP = INTERLEAVED ? N / 2 : N;      // pairs of a thread
    const int R = 2 * a.P;                           // rotated elements
    // chunks per row: interleaved d / N; halves: P / N that rotate, (d - R) / N / 2 rounded up that only move
    const int rot_units = INTERLEAVED ? a.d / N : a.P / N;
    const int units = INTERLEAVED ? rot_units : rot_units + ((a.d - R) / N + 1) / 2;
    const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t row = idx / units;
    const int u = (int)(idx % units);
    if (row >= (int64_t)a.B * a.L) return;
    const int b = (int)(row / a.L), l = (int)(row % a.L);
    const int *pos = a.pos + b * a.pos_b + (int64_t)l * a.n_axes;

    float sn[NP], cs[NP];
    int e0, e1 = 0;  // first element of each chunk
    bool second = true;
    int live = NP;  // pairs of this thread that turn; what lies behind them moves as it is
    if (INTERLEAVED) {
        e0 = u * N;
        live = a.P - e0 / 2;
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (i < live) pair_sincos(a, pos, e0 / 2 + i, sn[i], cs[i]);
    } else if (u < rot_units) {
        e0 = u * N, e1 = a.P + u * N;
#pragma unroll
        for (int i = 0; i < NP; ++i) pair_sincos(a, pos, e0 + i, sn[i], cs[i]);
    } else {
        e0 = R + (u - rot_units) * 2 * N, e1 = e0 + N;
        second = e1 < a.d;
        live = 0;
    }

    const int h0 = blockIdx.y * heads_per_block, h1 = min(h0 + heads_per_block, a.H[0] + a.H[1]);
    for (int h = h0; h < h1; h += kUnroll) {
        uint4 w[kUnroll][M];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
            if (h + j < h1) {
                const int t = h + j >= a.H[0], hh = h + j - (t ? a.H[0] : 0);
                const View &v = a.x[t];
                const T *src = static_cast<const T *>(v.p) + b * v.b + hh * v.h + l * v.l;
                w[j][0] = *reinterpret_cast<const uint4 *>(src + e0);
                if (M == 2 && second) w[j][M - 1] = *reinterpret_cast<const uint4 *>(src + e1);
            }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
            if (h + j < h1) {
                const int t = h + j >= a.H[0], hh = h + j - (t ? a.H[0] : 0);
                const View &v = a.y[t];
                T *dst = static_cast<T *>(v.p) + b * v.b + hh * v.h + l * v.l;
                float f[M][N];
#pragma unroll
                for (int m = 0; m < M; ++m) Vec<T>::unpack(w[j][m], f[m]);
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    if (i >= live) break;
                    float &x = INTERLEAVED ? f[0][(2 * i) % N] : f[0][i % N];
                    float &y = INTERLEAVED ? f[0][(2 * i + 1) % N] : f[M - 1][i % N];
                    const float r = x * cs[i] - y * sn[i], q = x * sn[i] + y * cs[i];
                    x = r, y = q;
                }
                *reinterpret_cast<uint4 *>(dst + e0) = Vec<T>::pack(f[0]);
                if (M == 2 && second) *reinterpret_cast<uint4 *>(dst + e1) = Vec<T>::pack(f[M - 1]);
            }
    }
}

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ float ld(const bf16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ld(const __half *p) { return __half2float(*p); }
__device__ __forceinline__ void st(float *p, float v) { *p = v; }
__device__ __forceinline__ void st(bf16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void st(__half *p, float v) { *p = __float2half_rn(v); }

// Any strides and any number of pairs: a thread owns one pair, or one element
// pair behind the rotated ones, and walks over the heads.  Taken when a view is
// not 16-byte aligned or when halves of P pairs do not fall on 16 bytes.
template <class T>
__global__ void __launch_bounds__(kThreads) k_rope_any(const __grid_constant__ RopeArgs a, int heads_per_block) {
    const int units = a.d / 2;
    const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t row = idx / units;
    const int u = (int)(idx % units);
    if (row >= (int64_t)a.B * a.L) return;
    const int b = (int)(row / a.L), l = (int)(row % a.L);
    const bool turns = u < a.P;
    float sn = 0.f, cs = 1.f;
    if (turns) pair_sincos(a, a.pos + b * a.pos_b + (int64_t)l * a.n_axes, u, sn, cs);
    const bool halves = !a.interleaved && turns;
    const int e0 = halves ? u : 2 * u, e1 = halves ? a.P + u : 2 * u + 1;
    const int h0 = blockIdx.y * heads_per_block, h1 = min(h0 + heads_per_block, a.H[0] + a.H[1]);
    for (int h = h0; h < h1; ++h) {
        const int t = h >= a.H[0], hh = h - (t ? a.H[0] : 0);
        const T *src = static_cast<const T *>(a.x[t].p) + b * a.x[t].b + hh * a.x[t].h + l * a.x[t].l;
        T *dst = static_cast<T *>(a.y[t].p) + b * a.y[t].b + hh * a.y[t].h + l * a.y[t].l;
        const float x = ld(src + e0), y = ld(src + e1);
        st(dst + e0, turns ? x * cs - y * sn : x);
        st(dst + e1, turns ? x * sn + y * cs : y);
    }
}

template <class T>
cudaError_t go(const RopeArgs &a, cudaStream_t s) {
    constexpr int N = Vec<T>::N;
    bool vec = a.d % N == 0 && (a.interleaved || a.P % N == 0);
    for (int t = 0; t < 2; ++t) {
        if (!a.H[t]) continue;
        for (const View *v : {&a.x[t], &a.y[t]})
            if ((reinterpret_cast<uintptr_t>(v->p) & 15u) || (a.B > 1 && v->b % N) || (a.H[t] > 1 && v->h % N) ||
                (a.L > 1 && v->l % N))
                vec = false;
    }
    const int H = a.H[0] + a.H[1];
    const int units = !vec ? a.d / 2 : a.interleaved ? a.d / N : a.P / N + ((a.d - 2 * a.P) / N + 1) / 2;
    const int64_t blocks = ((int64_t)a.B * a.L * units + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    // Heads per block: as many as leave 8 blocks for each of the 148 SMs, 16 at
    // most (the sines of a thread then cost a small part of its loads).
    int hpb = 16;
    while (hpb > 1 && blocks * ((H + hpb - 1) / hpb) < 148 * 8) hpb /= 2;
    const dim3 grid((unsigned)blocks, (H + hpb - 1) / hpb);
    if (!vec)
        k_rope_any<T><<<grid, kThreads, 0, s>>>(a, hpb);
    else if (a.interleaved)
        k_rope<T, true><<<grid, kThreads, 0, s>>>(a, hpb);
    else
        k_rope<T, false><<<grid, kThreads, 0, s>>>(a, hpb);
    AC_NOTE_LAUNCH();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(int dtype, const RopeArgs &a, cudaStream_t s) {
    if (dtype == AC_DTYPE_BF16) return go<bf16>(a, s);
    if (dtype == AC_DTYPE_F16) return go<__half>(a, s);
    return go<float>(a, s);
}

}  // namespace ac
