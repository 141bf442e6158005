// window_few.cu -- the same attention for few query rows: single tokens, or a
// few, with G * Lq <= 16 rows for each key head, over bf16 keys or the 8-bit cache.
//
// Bound by reading K and V once.  A warp takes 16 keys at a time: S = Q K^T with
// m16n8k16 products (the 16 rows are the packed (token, head) rows of one key
// head), the running softmax of window_attn.cu, and O += P V.  K and V go from
// global memory straight into the products' operand registers: the order of the
// contraction over d, and of the output columns, is free, so each thread owns d / 4
// consecutive elements of a key row (K) and d / 8 of four value rows (V), loads
// them 16 bytes at a time, and the rows of a warp are read whole.  The tile
// kernel would spend its time on the 112 or more empty rows of its products; here
// the products are a small part of the issue slots.
//
// The next K rows are loaded as soon as the products of the present ones have
// taken theirs, and the same for V: every warp has one of the two in flight.
// The keys are split over CTAs (k_combine joins them) and, within a CTA, over
// four warps, which are joined in shared memory.
//
// Types, scales and roundings as in the tile kernel: bf16 over bf16 keys, fp16 with
// the scales in the exponents over the 8-bit cache.
#include "stream_device.cuh"

namespace ac {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kChunk = 16;

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct FewParams {
    WinArgs a;
    int nsplit;
    float scale_log2;
    float *part_o, *part_lse;
};

// N 16-byte words (8 bytes for N = 0) from global memory, read once.
template <int BYTES>
__device__ __forceinline__ void load_bytes(uint32_t (&r)[BYTES / 4], const void *src, bool live) {
    if constexpr (BYTES == 8) {
        uint2 w = make_uint2(0, 0);
        if (live) w = __ldg(static_cast<const uint2 *>(src));
        r[0] = w.x, r[1] = w.y;
    } else {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live) w = __ldg(static_cast<const uint4 *>(src) + i);
            r[4 * i] = w.x, r[4 * i + 1] = w.y, r[4 * i + 2] = w.z, r[4 * i + 3] = w.w;
        }
    }
}

template <int D, bool C8>
__global__ void __launch_bounds__(kThreads, C8 ? 3 : 2) k_window_few(const __grid_constant__ FewParams fp) {
    const WinArgs &p = fp.a;
    constexpr int ES = C8 ? 1 : 2;        // bytes of a stored element
    constexpr int KB = D / 4 * ES;        // bytes of a key row that a thread owns
    constexpr int VB = D / 8 * ES;        // of a value row
    constexpr int KS = D / 16;            // k16 steps of S
    constexpr int NT = D / 8;             // n8 tiles of O
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;

    int idx = blockIdx.x;
    const int sp = idx % fp.nsplit;
    idx /= fp.nsplit;
    const int hk = idx % p.Hk, b = idx / p.Hk;
    const int ql = seq_len(p.q_lens, b, p.Lq, p.err), kl = seq_len(p.k_lens, b, p.Lk, p.err);
    const int off = kl - ql, rows = p.G * p.Lq;
    int lo_c = 0, hi_c = 0;
    if (ql > 0) {
        lo_c = row_range(p.w, off, kl).lo;
        hi_c = row_range(p.w, ql - 1 + off, kl).hi;
    }
    const int sink_c = min(p.w.sinks, hi_c);
    const int w0 = lo_c / kChunk, w1 = (hi_c + kChunk - 1) / kChunk;
    const int nsink = min((sink_c + kChunk - 1) / kChunk, w0);
    const int n_all = hi_c > 0 ? nsink + w1 - w0 : 0;
    const int j0 = (int)((long long)n_all * sp / fp.nsplit), j1 = (int)((long long)n_all * (sp + 1) / fp.nsplit);
    auto chunk_base = [&](int j) { return (j < nsink ? j : w0 + (j - nsink)) * kChunk; };

    // ---- this thread's two rows, g8 and g8 + 8
    RowRange rr[2];
    int sink[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = g8 + 8 * e, i = r / p.G;
        rr[e] = RowRange{0, 0x7FFFFFFF};  // a row that does not exist never asks for a mask
        if (r < rows && i < ql) rr[e] = row_range(p.w, i + off, kl);
        else if (r < rows) rr[e] = RowRange{0, 0};
        sink[e] = min(p.w.sinks, rr[e].hi);
    }
    // ---- Q as the A operand: k16 step s holds elements t4 D/4 + 4 s + {0..3} of the rows
    uint32_t aq[KS][4];
    float row_c[2];  // scale log2(e), times the power of two taken out of the row
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = g8 + 8 * e;
        uint32_t w[D / 8];
        const bool live = r < rows && r / p.G < ql;
        const bf16 *src = static_cast<const bf16 *>(p.q.p);
        if (live) src += b * p.q.b + (int64_t)(hk * p.G + r % p.G) * p.q.h + (int64_t)(r / p.G) * p.q.l + t4 * (D / 4);
        load_bytes<D / 2>(w, src, live);
        row_c[e] = fp.scale_log2;
        if constexpr (C8) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int ex = min(max((int)(top >> 7) - 127, -120), 120);  // |q| < 2^(ex + 1)
            row_c[e] *= exp2i(ex);
            const float dn = exp2i(-ex);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                w[i] = pack_half2(__uint_as_float(w[i] << 16) * dn, __uint_as_float(w[i] & 0xFFFF0000u) * dn);
            }
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) aq[s][e] = w[2 * s], aq[s][2 + e] = w[2 * s + 1];
    }

    // ---- addresses of a chunk's rows
    const int *table = C8 ? p.table + (int64_t)b * p.max_pages : nullptr;
    float ks = 1.f, vs_next = 1.f;
    struct Rows {
        const uint8_t *k, *v;  // row 0 of the chunk; null: zeros
    };
    auto rows_of = [&](int base, float &ksc, float &vsc) -> Rows {
        if constexpr (C8) {
            const int page = table[base / p.T];
            if (page < 0 || page >= p.pages) {
                if (lane == 0) atomicOr(&p.err->bits, DEV_ERR_BOUNDS);
                ksc = vsc = 1.f;
                return Rows{nullptr, nullptr};
            }
            const int64_t slot = (int64_t)page * p.Hk + hk;
            ksc = __ldg(p.ks + slot), vsc = __ldg(p.vs + slot);
            const int64_t at = (slot * p.T + base % p.T) * D;
            return Rows{p.k8 + at, vsc >= kMinScale ? p.v8 + at : nullptr};
        } else {
            const bf16 *k = static_cast<const bf16 *>(p.k.p) + b * p.k.b + hk * p.k.h + (int64_t)base * p.k.l;
            const bf16 *v = static_cast<const bf16 *>(p.v.p) + b * p.v.b + hk * p.v.h + (int64_t)base * p.v.l;
            return Rows{reinterpret_cast<const uint8_t *>(k), reinterpret_cast<const uint8_t *>(v)};
        }
    };
    const int64_t krow = C8 ? D : p.k.l * 2, vrow = C8 ? D : p.v.l * 2;  // bytes from row to row
    uint32_t kw[2][KB / 4], vw[4][VB / 4];
    auto load_k = [&](const Rows &r, int base) {  // keys g8 and g8 + 8
#pragma unroll
        for (int u = 0; u < 2; ++u)
            load_bytes<KB>(kw[u], r.k + (g8 + 8 * u) * krow + t4 * KB, r.k != nullptr && base + g8 + 8 * u < kl);
    };
    auto load_v = [&](const Rows &r, int base) {  // keys 2 t4, 2 t4 + 1, and 8 on
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int key = 2 * t4 + (u & 1) + 8 * (u >> 1);
            load_bytes<VB>(vw[u], r.v + key * vrow + g8 * VB, r.v != nullptr && base + key < kl);
        }
    };

    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    int j = j0 + warp;
    float vs = 1.f, ks_next = 1.f;
    Rows cur{nullptr, nullptr};
    if (j < j1) {
        cur = rows_of(chunk_base(j), ks, vs);
        load_k(cur, chunk_base(j));
        load_v(cur, chunk_base(j));
    }
    for (; j < j1; j += kWarps) {
        const int base = chunk_base(j);
        const bool more = j + kWarps < j1;
        const int base2 = more ? chunk_base(j + kWarps) : 0;
        Rows nxt{nullptr, nullptr};
        if (more) nxt = rows_of(base2, ks_next, vs_next);

        float s[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][e] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if constexpr (C8) {
                    const uint32_t w = kw[u][k];  // 4 codes: one k16 step's share
                    mma_f16(s[u], aq[k], e4m3x2_to_half2(w & 0xFFFFu), e4m3x2_to_half2(w >> 16));
                } else {
                    mma_bf16(s[u], aq[k], kw[u][2 * k], kw[u][2 * k + 1]);
                }
            }
        }
        if (more) load_k(nxt, base2);

        // scores in log2 units; s[u][2 e + c]: row g8 + 8 e, key 8 u + 2 t4 + c
        bool full = true;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            full = full && base + kChunk <= rr[e].hi && (base >= rr[e].lo || base + kChunk <= sink[e]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float c = C8 ? row_c[e] * ks : row_c[e];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int x = 0; x < 2; ++x) s[u][2 * e + x] *= c;
        }
        if (!full) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int key = base + 8 * u + 2 * t4 + x;
                        const bool see = key < rr[e].hi && (key >= rr[e].lo || key < sink[e]);
                        s[u][2 * e + x] = see ? s[u][2 * e + x] : -INFINITY;
                    }
        }
        const float ev = C8 ? fmaxf(__log2f(vs), kMinLogScale) : 0.f;  // exponent of the scale of V
        float top[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) top[e] = ev + fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
        // The maximum moves when some row's grew by more than 2^8 (or is the first).
        if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = top[e];
                x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
                const float mn = fmaxf(m[e], x);
                const float al = mn > m[e] ? ex2_approx(m[e] - mn) : 1.f;
                m[e] = mn;
                l[e] *= al;
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][2 * e] *= al, acc[n][2 * e + 1] *= al;
            }
        }
        uint32_t ap[4];
        const float inv_vs = C8 ? ex2_approx(-ev) : 1.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float mu = (m[e] == -INFINITY ? 0.f : m[e]) - ev;
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float p0 = ex2_approx(s[u][2 * e] - mu), p1 = ex2_approx(s[u][2 * e + 1] - mu);
                sum += p0 + p1;
                ap[2 * u + e] = C8 ? pack_half2(p0, p1) : pack_bf16x2(p0, p1);
            }
            l[e] = C8 ? fmaf(sum, inv_vs, l[e]) : l[e] + sum;
        }
        // n8 tile n, column g8 is output element g8 D/8 + n
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
            uint32_t b0[2], b1[2];
            if constexpr (C8) {
                const int word = n / 4, odd = (n / 2) & 1;  // bytes n, n + 1 of the four rows
                const uint32_t sel = odd ? 0x7362 : 0x5140;
                const uint32_t x = __byte_perm(vw[0][word], vw[1][word], sel), y = __byte_perm(vw[2][word], vw[3][word], sel);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    b0[i] = e4m3x2_to_half2((x >> (16 * i)) & 0xFFFFu), b1[i] = e4m3x2_to_half2((y >> (16 * i)) & 0xFFFFu);
            } else {
                const uint32_t r0 = vw[0][n / 2], r1 = vw[1][n / 2], r2 = vw[2][n / 2], r3 = vw[3][n / 2];
                b0[0] = __byte_perm(r0, r1, 0x5410), b0[1] = __byte_perm(r0, r1, 0x7632);
                b1[0] = __byte_perm(r2, r3, 0x5410), b1[1] = __byte_perm(r2, r3, 0x7632);
            }
            if constexpr (C8) {
                mma_f16(acc[n], ap, b0[0], b1[0]);
                mma_f16(acc[n + 1], ap, b0[1], b1[1]);
            } else {
                mma_bf16(acc[n], ap, b0[0], b1[0]);
                mma_bf16(acc[n + 1], ap, b0[1], b1[1]);
            }
        }
        if (more) load_v(nxt, base2);
        ks = ks_next, vs = vs_next;
    }

    // ---- join the four warps
    __shared__ float s_m[kWarps][16], s_l[kWarps][16];
    __shared__ __align__(16) float s_o[kWarps][16][D + 4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
        l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
        if (t4 == 0) s_m[warp][g8 + 8 * e] = m[e], s_l[warp][g8 + 8 * e] = l[e];
        // columns 2 t4 and 2 t4 + 1 of the n8 tiles: elements (2 t4 + x) D/8 + n
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int n = 0; n < NT; ++n) s_o[warp][g8 + 8 * e][(2 * t4 + x) * NT + n] = acc[n][2 * e + x];
    }
    __syncthreads();
    constexpr int TPR = kThreads / 16;      // threads of a row
    constexpr int EPT = D / TPR;            // elements of a thread
    const int r = tid / TPR, e0 = (tid % TPR) * EPT;
    if (r >= rows) return;
    float top = -INFINITY, sum = 0.f, wgt[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        wgt[w] = s_m[w][r] == -INFINITY ? 0.f : ex2_approx(s_m[w][r] - top);
        sum += wgt[w] * s_l[w][r];
    }
    const int i = r / p.G, h = hk * p.G + r % p.G;
    const bool some = i < ql && sum > 0.f;
    const float inv = some ? 1.f / sum : 0.f;
    const float lse = some ? (top + __log2f(sum)) * 0.693147180559945f : -INFINITY;
    const int64_t all = (int64_t)p.B * p.Hq * p.Lq, orow = ((int64_t)b * p.Hq + h) * p.Lq + i;
    float o[EPT];
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
        o[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) o[e] += wgt[w] * s_o[w][r][e0 + e];
        o[e] = some ? o[e] * inv : 0.f;
    }
    if (fp.nsplit > 1) {
        float *dst = fp.part_o + (sp * all + orow) * D + e0;
#pragma unroll
        for (int e = 0; e < EPT; e += 4) *reinterpret_cast<float4 *>(dst + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        if (e0 == 0) fp.part_lse[sp * all + orow] = lse;
    } else {
        bf16 *dst = static_cast<bf16 *>(p.o.p) + b * p.o.b + h * p.o.h + (int64_t)i * p.o.l + e0;
#pragma unroll
        for (int e = 0; e < EPT; e += 8)
            *reinterpret_cast<uint4 *>(dst + e) = make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]),
                                                             pack_bf16x2(o[e + 4], o[e + 5]), pack_bf16x2(o[e + 6], o[e + 7]));
        if (p.lse && e0 == 0) p.lse[orow] = lse;
    }
}

// CTAs for eight waves of single CTAs on the 148 SMs, but no part below 512 keys.
int few_split(const WinArgs &a) {
    const int64_t n = window_tiles(a.w, a.Lq, a.Lq, a.Lk, kChunk);
    const int64_t want = (148 * 8 + (int64_t)a.B * a.Hk - 1) / ((int64_t)a.B * a.Hk);
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, n / 32));
}

}  // namespace

int64_t window_few_workspace(const WinArgs &a) {
    const int s = few_split(a);
    return s > 1 ? (int64_t)s * a.B * a.Hq * a.Lq * (a.d + 1) * 4 : 0;
}

cudaError_t launch_window_few(const WinArgs &a, cudaStream_t s) {
    FewParams p{};
    p.a = a;
    p.nsplit = few_split(a);
    p.scale_log2 = a.scale * 1.44269504088896f;
    if (p.nsplit > 1) {
        p.part_o = static_cast<float *>(a.ws);
        p.part_lse = p.part_o + (int64_t)p.nsplit * a.B * a.Hq * a.Lq * a.d;
    }
    const int64_t grid = (int64_t)a.B * a.Hk * p.nsplit;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (a.d == 128) {
        if (a.k8) k_window_few<128, true><<<(unsigned)grid, kThreads, 0, s>>>(p);
        else k_window_few<128, false><<<(unsigned)grid, kThreads, 0, s>>>(p);
    } else {
        if (a.k8) k_window_few<64, true><<<(unsigned)grid, kThreads, 0, s>>>(p);
        else k_window_few<64, false><<<(unsigned)grid, kThreads, 0, s>>>(p);
    }
    AC_NOTE_LAUNCH();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.nsplit == 1) return e;
    return launch_combine(p.part_o, p.part_lse, a, p.nsplit, s);
}

}  // namespace ac
