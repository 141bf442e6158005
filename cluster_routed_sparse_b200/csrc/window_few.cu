// window_few.cu -- the same attention for few query rows: single tokens, or a few,
// with 8 rows (G heads x tokens) of a key head to a CTA, over bf16 keys or the 8-bit cache.
//
// Bound by reading K and V once.  A warp takes 16 keys at a time, and its 8 rows are
// the short side of m16n8k16 products: S^T = K Q^T, the running softmax of
// window_attn.cu, O^T += V^T P^T, with P^T transposed in registers.  K and V go from
// global memory straight into the products' operand registers: the order of the
// contraction over d, and of the output rows, is free, so each thread owns d / 4
// consecutive elements of two key rows and d / 8 of four value rows, loads them
// 16 bytes at a time, and the rows of a warp are read whole.
//
// The next K rows are loaded as soon as the products of the present ones have
// taken theirs, and the same for V: every warp has one of the two in flight.
// The keys are split over CTAs (k_combine joins them) and, within a CTA, over
// four warps, which are joined in shared memory.
//
// One token of four sequences over 16,384 of 32,760 bf16 keys and 128 first ones, 40
// heads (1.35 GB): 209 us in a graph, the rate of a copy.  One token of eight sequences
// over 32,760 cached tokens, 8 key heads for 40 (0.54 GB): 108 us, 5.0 TB/s, 77% of it:
// a warp waits for its loads and then works, and converting V to bf16 takes 8 us of that,
// the second part of the weights 3 (fp16 codes and weights took 95, and lost weights;
// integer steps instead of the two conversions 116; 5 CTAs on an SM spill, 152).
// More rows take as many CTAs, which find the keys in the L2 cache: 200 us for 16 rows over
// a cache of that size, 281 for 24.
//
// Over the 8-bit cache K enters its product as fp16 codes (one conversion for two of them), with
// the scale of its page taken into the scores and Q divided by a power of two per row to fit:
// fp16 then holds its elements down to 2^-31 of the row's largest exactly.  Where one is
// smaller, the CTA takes K as bf16 codes and Q as it is (three conversions more; the branch
// costs 1 us of 107, a loop of its own for each 6).  V: bf16 codes.
// Rounding: a weight is a sum of two bf16 values, hence off by 2^-17 at most, over
// fp32's whole range of exponents; over the cache it takes the scale of V's page first, a power of
// two, and the sum of the weights does without.  (In fp16 small weights lost their bits
// beside a page of large values.)  The second value's products are hidden behind the loads.
// O is rounded once at the end; everything else is fp32.
#include "stream_device.cuh"

namespace ac {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kChunk = 16;

// m16n8k16 with fp32 sums, fp16 or bf16 operands.
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 matrix of 16-bit values, lane (g, t) holding row g, columns 2 t and 2 t + 1, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

struct FewParams {
    WinArgs a;
    int nsplit, groups;
    float scale_log2;
    float *part_o, *part_lse;
};

// BYTES bytes (8, or a multiple of 16) from global memory, read once; zeros where not live.
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

// The CTAs of the 8-row groups of a key head stand side by side.
template <int D, bool C8>
__global__ void __launch_bounds__(kThreads, C8 ? 4 : 3) k_window_few(const __grid_constant__ FewParams fp) {
    const WinArgs &p = fp.a;
    constexpr int ES = C8 ? 1 : 2;        // bytes of a stored element
    constexpr int KB = D / 4 * ES;        // bytes of a key row that a thread owns
    constexpr int VB = D / 8 * ES;        // of a value row
    constexpr int KS = D / 16;            // k16 steps of S
    constexpr int DT = D / 16;            // m16 tiles of O^T
    constexpr int NR = 2;                 // rows of a thread
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;

    release_successor();
    int idx = blockIdx.x;
    const int row0 = idx % fp.groups * 8;  // the CTA's first row: token row / G, head row % G
    idx /= fp.groups;
    const int sp = idx % fp.nsplit;
    idx /= fp.nsplit;
    const int hk = idx % p.Hk, b = idx / p.Hk;
    const int ql = seq_len(p.q_lens, b, p.Lq, p.err), kl = seq_len(p.k_lens, b, p.Lk, p.err);
    const int off = kl - ql, rows = p.G * p.Lq - row0;
    int lo_c = 0, hi_c = 0;
    if (row0 / p.G < ql) {
        lo_c = row_range(p.w, row0 / p.G + off, kl).lo;
        hi_c = row_range(p.w, min((row0 + 7) / p.G, ql - 1) + off, kl).hi;
    }
    const int sink_c = min(p.w.sinks, hi_c);
    const int w0 = lo_c / kChunk, w1 = (hi_c + kChunk - 1) / kChunk;
    const int nsink = min((sink_c + kChunk - 1) / kChunk, w0);
    const int n_all = hi_c > 0 ? nsink + w1 - w0 : 0;
    const int j0 = (int)((long long)n_all * sp / fp.nsplit), j1 = (int)((long long)n_all * (sp + 1) / fp.nsplit);
    auto chunk_base = [&](int j) { return (j < nsink ? j : w0 + (j - nsink)) * kChunk; };

    // ---- Q^T as the B operand: k16 step s holds elements t4 D/4 + 4 s + {0..3} of row g8
    uint32_t bq[KS][2];
    bool wide = false;          // over the cache: Q stays bf16
    float g_c = fp.scale_log2;  // scale log2(e), times the power of two taken out of that row
    {
        uint32_t w[D / 8];
        const int i = (row0 + g8) / p.G, g = (row0 + g8) % p.G;
        const bool live = g8 < rows && i < ql;
        const bf16 *src = static_cast<const bf16 *>(p.q.p);
        if (live) src += b * p.q.b + (int64_t)(hk * p.G + g) * p.q.h + (int64_t)i * p.q.l + t4 * (D / 4);
        load_bytes<D / 2>(w, src, live);
        if constexpr (C8) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int ex = (top ? min(max((int)(top >> 7) - 127, -112), 120) : 0) - 14;  // |q| < 2^(ex + 15)
            uint32_t least = 0xFFFFu;  // the smallest that is not 0 (0 - 1 is the largest)
#pragma unroll
            for (int i = 0; i < D / 8; ++i) least = min(least, min(((w[i] & 0x7FFFu) - 1u) & 0xFFFFu, (((w[i] >> 16) & 0x7FFFu) - 1u) & 0xFFFFu));
            wide = __any_sync(0xFFFFFFFFu, (int)((least + 1u) >> 7) - 127 < ex - 17) != 0;
            if (!wide) {
                g_c *= exp2i(ex);
                const float dn = exp2i(-ex);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) w[i] = pack_half2(__uint_as_float(w[i] << 16) * dn, __uint_as_float(w[i] & 0xFFFF0000u) * dn);
            }
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) bq[s][0] = w[2 * s], bq[s][1] = w[2 * s + 1];
    }
    // ---- this thread's rows of the scores: e is row 2 t4 + e
    RowRange rr[NR];
    int sink[NR];
    float row_c[NR];
#pragma unroll
    for (int e = 0; e < NR; ++e) {
        const int r = 2 * t4 + e, i = (row0 + r) / p.G;
        rr[e] = RowRange{0, 0x7FFFFFFF};  // a row that does not exist never asks for a mask
        if (r < rows && i < ql) rr[e] = row_range(p.w, i + off, kl);
        else if (r < rows) rr[e] = RowRange{0, 0};
        sink[e] = min(p.w.sinks, rr[e].hi);
        row_c[e] = __shfl_sync(0xFFFFFFFFu, g_c, 4 * (2 * t4 + e));
    }

    // ---- addresses of a chunk's rows.  The table entry is loaded one chunk ahead.
    const int *table = C8 ? p.table + (int64_t)b * p.max_pages : nullptr;
    const int log_t = C8 ? 31 - __clz(p.T) : 0;
    auto entry_of = [&](int j) -> int { return C8 && j < j1 ? __ldg(table + (chunk_base(j) >> log_t)) : 0; };
    struct Rows {
        const uint8_t *k, *v;  // row 0 of the chunk; null: zeros
    };
    auto rows_of = [&](int base, int page, float &ksc, float &vsc) -> Rows {
        if constexpr (C8) {
            if (page < 0 || page >= p.pages) {
                if (lane == 0) atomicOr(&p.err->bits, DEV_ERR_BOUNDS);
                ksc = vsc = 1.f;
                return Rows{nullptr, nullptr};
            }
            const int64_t slot = (int64_t)page * p.Hk + hk;
            ksc = __ldg(p.ks + slot), vsc = __ldg(p.vs + slot);
            const int64_t at = (slot * p.T + (base & (p.T - 1))) * D;
            return Rows{p.k8 + at, p.v8 + at};
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

    float acc[DT][4];
#pragma unroll
    for (int n = 0; n < DT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    float m[NR], l[NR];
#pragma unroll
    for (int e = 0; e < NR; ++e) m[e] = -INFINITY, l[e] = 0.f;

    int j = j0 + warp;
    float ks = 1.f, vs = 1.f, ks_next = 1.f, vs_next = 1.f;
    int entry = entry_of(j + kWarps);
    if (j < j1) {
        const Rows cur = rows_of(chunk_base(j), entry_of(j), ks, vs);
        load_k(cur, chunk_base(j));
        load_v(cur, chunk_base(j));
    }
    for (; j < j1; j += kWarps) {
        const int base = chunk_base(j);
        const bool more = j + kWarps < j1;
        const int base2 = more ? chunk_base(j + kWarps) : 0;
        Rows nxt{nullptr, nullptr};
        if (more) nxt = rows_of(base2, entry, ks_next, vs_next);
        entry = entry_of(j + 2 * kWarps);

        // S^T: s[2 u + e] is key g8 + 8 u, row 2 t4 + e
        float s[4] = {};
        if (C8 && wide) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint32_t x = kw[0][k], y = kw[1][k];  // 4 codes: one k16 step's share
                mma<false>(s, e4m3x2_to_bf16x2(x & 0xFFFFu), e4m3x2_to_bf16x2(y & 0xFFFFu), e4m3x2_to_bf16x2(x >> 16),
                           e4m3x2_to_bf16x2(y >> 16), bq[k][0], bq[k][1]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t a[4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if constexpr (C8) {
                        const uint32_t w = kw[u][k];
                        a[u] = e4m3x2_to_half2(w & 0xFFFFu), a[2 + u] = e4m3x2_to_half2(w >> 16);
                    } else {
                        a[u] = kw[u][2 * k], a[2 + u] = kw[u][2 * k + 1];
                    }
                }
                mma<C8>(s, a[0], a[1], a[2], a[3], bq[k][0], bq[k][1]);
            }
        }
        if (more) load_k(nxt, base2);

        // scores in log2 units, without V's scale
        bool full = true;
#pragma unroll
        for (int e = 0; e < NR; ++e) {
            full = full && base + kChunk <= rr[e].hi && (base >= rr[e].lo || base + kChunk <= sink[e]);
            s[e] *= row_c[e], s[2 + e] *= row_c[e];
            if (C8) s[e] *= ks, s[2 + e] *= ks;  // (one after the other: the two factors' product may overflow where s is 0)
        }
        if (!full) {
#pragma unroll
            for (int e = 0; e < NR; ++e)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int key = base + g8 + 8 * u;
                    float &x = s[2 * u + e];
                    x = key < rr[e].hi && (key >= rr[e].lo || key < sink[e]) ? x : -INFINITY;
                }
        }
        float top[NR];
        bool grows = false;
#pragma unroll
        for (int e = 0; e < NR; ++e) {
            top[e] = fmaxf(s[e], s[2 + e]);
            grows = grows || top[e] > m[e] + 8.f;
        }
        // The maximum moves when some row's grew by more than 2^8 (or is the first).
        if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
            for (int e = 0; e < NR; ++e) {
                float x = top[e];
#pragma unroll
                for (int o = 4; o < 32; o *= 2) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
                const float mn = fmaxf(m[e], x);
                const float al = mn > m[e] ? ex2_approx(m[e] - mn) : 1.f;
                m[e] = mn;
                l[e] *= al;
#pragma unroll
                for (int n = 0; n < DT; ++n) acc[n][e] *= al, acc[n][2 + e] *= al;
            }
        }
        // weights, and P^T as the B operand: keys 8 u + 2 t4 + {0, 1} of row g8
        uint32_t bp[2][2];  // [high and low part][u]
        float pr[2][2];
#pragma unroll
        for (int e = 0; e < NR; ++e) {
            const float mu = m[e] == -INFINITY ? 0.f : m[e];
            pr[0][e] = ex2_approx(s[e] - mu), pr[1][e] = ex2_approx(s[2 + e] - mu);
            l[e] += pr[0][e] + pr[1][e];
            if (C8) pr[0][e] *= vs, pr[1][e] *= vs;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t hi = pack_bf16x2(pr[u][0], pr[u][1]);
            bp[0][u] = transpose8x8(hi);
            bp[1][u] = transpose8x8(pack_bf16x2(pr[u][0] - __uint_as_float(hi << 16), pr[u][1] - __uint_as_float(hi & 0xFFFF0000u)));
        }
        // O^T: row g8 of m16 tile n is element g8 D/8 + 2 n, row g8 + 8 the next one.
        // Four tiles at a time: the products of a weight's two parts, which add up in one
        // accumulator, stand apart (one token over 32,760 cached tokens, 64 heads: 114 us side by side, 106).
        constexpr int GRP = 4;
#pragma unroll
        for (int n0 = 0; n0 < DT; n0 += GRP) {
            uint32_t a[GRP][4];
#pragma unroll
            for (int i = 0; i < GRP; ++i) {
                const int n = n0 + i;
                if constexpr (C8) {
                    const int word = n / 2;  // bytes 2 n, 2 n + 1 of the four rows
                    const uint32_t sel = n & 1 ? 0x7362 : 0x5140;
                    const uint32_t x = __byte_perm(vw[0][word], vw[1][word], sel), y = __byte_perm(vw[2][word], vw[3][word], sel);
                    a[i][0] = e4m3x2_to_bf16x2(x & 0xFFFFu), a[i][1] = e4m3x2_to_bf16x2(x >> 16);
                    a[i][2] = e4m3x2_to_bf16x2(y & 0xFFFFu), a[i][3] = e4m3x2_to_bf16x2(y >> 16);
                } else {
                    a[i][0] = __byte_perm(vw[0][n], vw[1][n], 0x5410), a[i][1] = __byte_perm(vw[0][n], vw[1][n], 0x7632);
                    a[i][2] = __byte_perm(vw[2][n], vw[3][n], 0x5410), a[i][3] = __byte_perm(vw[2][n], vw[3][n], 0x7632);
                }
            }
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int i = 0; i < GRP; ++i) mma<false>(acc[n0 + i], a[i][0], a[i][1], a[i][2], a[i][3], bp[part][0], bp[part][1]);
        }
        if (more) load_v(nxt, base2);
        ks = ks_next, vs = vs_next;
    }

    // ---- join the four warps
    __shared__ float s_m[kWarps][8], s_l[kWarps][8];
    __shared__ __align__(16) float s_o[kWarps][8][D + 4];
#pragma unroll
    for (int e = 0; e < NR; ++e) {
        const int r = 2 * t4 + e;
#pragma unroll
        for (int o = 4; o < 32; o *= 2) l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], o);
        if (g8 == 0) s_m[warp][r] = m[e], s_l[warp][r] = l[e];
#pragma unroll
        for (int n = 0; n < DT; ++n)
            *reinterpret_cast<float2 *>(&s_o[warp][r][g8 * (D / 8) + 2 * n]) =
                make_float2(acc[n][e], acc[n][2 + e]);
    }
    __syncthreads();
    constexpr int TPR = kThreads / 8;       // threads of a row
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
    const int i = (row0 + r) / p.G, h = hk * p.G + (row0 + r) % p.G;
    const bool some = i < ql && sum != 0.f;  // a row that sees nothing has a sum of exactly 0; a NaN is no such row
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
        for (int e = 0; e < EPT; e += 4)
            *reinterpret_cast<uint2 *>(dst + e) = make_uint2(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]));
        if (p.lse && e0 == 0) p.lse[orow] = lse;
    }
}

int few_groups(const WinArgs &a) { return (int)(((int64_t)a.G * a.Lq + 7) / 8); }

// Parts of the keys: as many as make the waves of CTAs come out full, a CTA costing
// its 16-key chunks and about ten more for its start and end, no part below 256 keys.
// (32,760 cached tokens, 64 key heads in all: 180, 109, 111, 114 and 125 us with 4, 9,
// 18, 27 and 37 parts.)
int few_split(const WinArgs &a) {
    const int64_t n = window_tiles(a.w, a.Lq, a.Lq, a.Lk, kChunk), units = (int64_t)a.B * a.Hk * few_groups(a);
    const int64_t slots = 148 * (a.k8 ? 4 : 3);
    int64_t best = INT64_MAX;
    int parts = 1;
    for (int64_t waves = 0; waves <= 8; ++waves) {
        const int64_t s = std::min(std::max<int64_t>(waves * slots / units, 1), std::max<int64_t>(n / 16, 1));
        const int64_t t = ((units * s + slots - 1) / slots) * ((n + s - 1) / s + 10);
        if (t < best) best = t, parts = (int)s;
    }
    return parts;
}

}  // namespace

int64_t window_few_workspace(const WinArgs &a) {
    const int s = few_split(a);
    return s > 1 ? (int64_t)s * a.B * a.Hq * a.Lq * (a.d + 1) * 4 : 0;
}

cudaError_t launch_window_few(const WinArgs &a, cudaStream_t s) {
    FewParams p{};
    p.a = a;
    p.nsplit = few_split(a), p.groups = few_groups(a);
    p.scale_log2 = a.scale * 1.44269504088896f;
    if (p.nsplit > 1) {
        p.part_o = static_cast<float *>(a.ws);
        p.part_lse = p.part_o + (int64_t)p.nsplit * a.B * a.Hq * a.Lq * a.d;
    }
    const int64_t grid = (int64_t)a.B * a.Hk * p.nsplit * p.groups;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    auto go = [&](auto kern) { kern<<<(unsigned)grid, kThreads, 0, s>>>(p); };
    if (a.d == 128) a.k8 ? go(k_window_few<128, true>) : go(k_window_few<128, false>);
    else a.k8 ? go(k_window_few<64, true>) : go(k_window_few<64, false>);
    AC_NOTE_LAUNCH();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.nsplit == 1) return e;
    return launch_combine(p.part_o, p.part_lse, a, p.nsplit, s);
}

}  // namespace ac
