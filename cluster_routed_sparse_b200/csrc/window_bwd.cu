// window_bwd.cu -- gradients of the window attention on tcgen05 / TMEM.
//
// With P = 2^(s c - lse) from the forward's log-sum-exp, and per row
// delta = sum_j P dP:
//   dP = dO V^T    dS = P (dP - delta)    dV = P^T dO    dK = s dS^T Q    dQ = s dS K
// One kernel in two roles, each with four 128 x 128 products per tile:
//   rows = queries, tiles = keys:     S = Q K^T, dP = dO V^T, A1 += P K,    A2 += dS K
//   rows = keys,    tiles = queries:  S = K Q^T, dP = V dO^T, A1 += P dO,   A2 += dS Q
// (the second holds the transposes of S, P, dP, dS).  Every output row belongs to
// one CTA: no atomic sums, and the same bits from run to run.  Query rows are
// packed over the heads of a key head as in window_attn.cu, so the gradients of
// shared heads add up in the accumulator.
//
// The row sum delta0 = sum dO o that the first role starts from uses o as the
// forward rounded it, off by 2^-8 |dO| |o| at most: over thousands of keys that error,
// times sum_j P_j k_j, would be the largest in dQ (1.2e-2 of its norm measured over
// 5,000 keys, against 2e-3 from all other roundings).  Since sum_j dS_j = 0 for the
// true delta, r = sum_j dS_j tells the error, and dQ = s (A2 - r A1) takes it
// out; that is what A1 = P K is for.  There r sums dS as rounded to bf16, so that the
// part of those roundings which is common to all keys leaves too.  The second role
// takes delta0 plus the sum of dS before its rounding, which is the true delta (with
// the rounded sum the error of dK is up to a fifth larger where rows see few keys).
//
// A key tile that many queries see (first tokens; early keys without a left bound)
// would keep one SM busy after the others are done: its query tiles are split into
// parts of at most `chunk`, whose fp32 dK and dV k_sum_parts adds, in order.
//
// Schedule: A1(j), S(j+1), A2(j), dP(j+1) on the tensor core; 256 threads (row
// t mod 128, column half t / 128) turn S(j+1) into P while A2(j) and dP(j+1) run,
// and dP into dS while A1(j+1) and S(j+2) run.  Tensor memory (512 columns):
// S | dP | A1 | A2, each bf16 operand in the half of its scores that its own
// threads have read; the products of each half start when its four warps are done.
// P and dS are rounded to bf16, the operand type: 2^-8 of each at most and random over
// the sum, so each gradient is as far off from that as from its own rounding to bf16
// (2.3e-3 of its norm instead of 1.7e-3).  All else is fp32.  Masks as in
// window_attn.cu: one column interval per thread.
//
// Bound by the tensor core and the hand-offs: 8 products of 128 x 128 x d per tile and
// role pair where 5 are the gradient's own: S and dP are formed twice because each output
// row has one owner (dQ summed across key tiles, by atomics or in turns, would save them), and
// A1 = P K only takes the rounding of o out again.  32,760 queries in frames of 1,560 over three
// frames and the first, 12 heads, d = 128: 4.66 TFLOP in 3.8 ms, 1.22 PFLOP/s, 72% of
// the measured cuBLAS rate; 2,830 cycles a tile in the first role and 3,000 in the
// second where the products take 2,048 (the scores' wait 500, P 1,380, of which the
// exponentials 1,024, dS 670, and in the second role the statistics 420).  Short loops
// (clips) pay for their start: 4,800 cycles until the first tiles are there, a tile and
// a half.  Dropped: P and dS in column halves of 64 that go round on their own (5,264
// us with the forward, against 5,100); a barrier for each fixed tile, and
// an eighth to a third of the exponentials as a quartic on the FMA pipe (no difference).
#include "stream_device.cuh"
#include "stream_host.h"

namespace ac {
namespace {

constexpr int NTHREADS = 384;
constexpr uint32_t kRegsMath = 208, kRegsOther = 88;
static_assert(2 * 128 * kRegsMath + 128 * kRegsOther <= NTHREADS * 168, "register split exceeds the launch");
constexpr int kStats = 256;  // floats per query tile: -lse log2(e) of 128 rows, then delta

template <int D>
struct Layout {
    static constexpr int HALVES = D / 64;
    static constexpr uint32_t TILE = HALVES * 128 * 128;
    static constexpr uint32_t OFF_F = 0;               // fixed tiles F0, F1
    static constexpr uint32_t OFF_L0 = 2 * TILE;       // [2] looped tiles
    static constexpr uint32_t OFF_L1 = OFF_L0 + 2 * TILE;
    static constexpr uint32_t OFF_ST = OFF_L1 + 2 * TILE;  // [2][kStats] statistics of the looped queries
    static constexpr uint32_t OFF_R = OFF_ST + 2 * kStats * 4;  // [2][256] row sums
    static constexpr uint32_t OFF_BAR = OFF_R + 2 * 256 * 4;
    static constexpr uint32_t SMEM = OFF_BAR + 256 + 1024;
};

enum {
    B_FF = 0,   // fixed tiles filled
    B_0F = 1,   // [2] L0 stage filled
    B_0E = 3,   // [2] L0 stage free
    B_1F = 5,   // [2] L1 stage filled
    B_1E = 7,   // [2] L1 stage free
    B_SF = 9,   // S written
    B_DPF = 10, // dP written
    B_PF = 12,  // [2] half of P written by its four warps
    B_DF = 14,  // [2] half of dS written by its four warps
    B_Z0 = 16,  // rows behind the sequence zeroed in the last L0, L1 tile
    B_Z1 = 17,
    B_AF = 18,  // accumulators complete
    NBAR = 19
};

struct BwdMaps {
    CUtensorMap f0, f1, l0, l1;
};

struct BwdParams {
    View dq, dk, dv;
    float *stats;  // [B Hk][tiles_q][kStats]
    float *parts;  // [B Hk][part_tiles][max_parts][2][128][d]: dV, dK of key tiles in parts
    int chunk, max_parts, part_tiles;  // query tiles of a part; key tiles of a head that may have parts
    const int *q_lens, *k_lens;
    int B, Hq, Hk, G, TT, Lq, Lk, tiles_q, tiles_k;
    WinRule w;
    float scale, scale_log2;
    uint32_t launch;
    OpErr *err;
};

__device__ __forceinline__ uint32_t low_mask(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Tokens of a sequence that see key j: [lo, hi).
__device__ __forceinline__ RowRange key_range(const WinRule &w, int j, int off, int ql, int kl) {
    if (j >= kl) return RowRange{0, 0};
    const long long bj = w.g == 1 ? j : j / w.g;
    long long lo = w.right < 0 ? 0 : (bj - w.right) * w.g - off;
    long long hi = w.left < 0 || j < w.sinks ? ql : (bj + w.left + 1) * w.g - off;
    lo = lo < 0 ? 0 : lo > ql ? ql : lo;
    hi = hi < lo ? lo : hi > ql ? ql : hi;
    return RowRange{(int)lo, (int)hi};
}

// Query tiles [lo, lo + n) that see the key tile at key r0, and the parts they come in.
struct KeyTile {
    int lo, n, parts;
};
__device__ __forceinline__ KeyTile key_tile(const BwdParams &p, int r0, int ql, int kl) {
    KeyTile t{0, 0, 1};
    if (r0 < kl) {
        const RowRange a = key_range(p.w, r0, kl - ql, ql, kl);
        const RowRange z = key_range(p.w, min(r0 + 127, kl - 1), kl - ql, ql, kl);
        const int hi = max(a.hi, z.hi);
        if (hi > a.lo) t.lo = a.lo / p.TT, t.n = (hi + p.TT - 1) / p.TT - t.lo;
    }
    if (r0 / 128 < p.part_tiles) t.parts = max(1, min((t.n + p.chunk - 1) / p.chunk, p.max_parts));
    return t;
}

// -lse log2(e) (-inf for a row without keys, so that its P is 0) and
// delta0 = sum dO o of every row of the query tiles, in the order of the tiles.
// A CTA takes a query tile, D / 8 lanes a row; bound by reading dO and o once (9,360
// tokens of 12 heads, d = 128, 57 MB: 15 us).
template <int D>
__global__ void __launch_bounds__(256) k_row_stats(View go, View o, const float *__restrict__ lse, BwdParams p) {
    constexpr int LPR = D / 8, RPP = 256 / LPR, N = 4;  // lanes of a row, rows of a pass, passes with loads in flight
    release_successor();
    const int qt = blockIdx.x % (unsigned)p.tiles_q, bh = blockIdx.x / (unsigned)p.tiles_q;
    const int b = bh / p.Hk, hk = bh % p.Hk;
    const int part = threadIdx.x % LPR, first = threadIdx.x / LPR;
    const int ql = seq_len(p.q_lens, b, p.Lq, p.err);
    const bf16 *gb = static_cast<const bf16 *>(go.p) + b * go.b + hk * p.G * go.h, *ob = static_cast<const bf16 *>(o.p) + b * o.b + hk * p.G * o.h;
    const float *lb = lse + ((int64_t)b * p.Hq + hk * p.G) * p.Lq;
    float *st = p.stats + ((int64_t)bh * p.tiles_q + qt) * kStats;
    for (int r0 = first; r0 < 128; r0 += N * RPP) {
        uint4 x[N], y[N];
        float l[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int row = r0 + k * RPP, i = qt * p.TT + row / p.G, g = row % p.G;
            x[k] = y[k] = make_uint4(0, 0, 0, 0), l[k] = -INFINITY;
            if (row < p.G * p.TT && i < ql) {
                x[k] = *(reinterpret_cast<const uint4 *>(gb + g * go.h + i * go.l) + part);
                y[k] = *(reinterpret_cast<const uint4 *>(ob + g * o.h + i * o.l) + part);
                l[k] = lb[(int64_t)g * p.Lq + i];
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t xs[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, ys[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), s);
                s = fmaf(__uint_as_float(xs[e] & 0xFFFF0000u), __uint_as_float(ys[e] & 0xFFFF0000u), s);
            }
#pragma unroll
            for (int m = LPR / 2; m; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
            if (part == 0) {
                const int row = r0 + k * RPP;
                st[row] = l[k] == -INFINITY ? -INFINITY : -l[k] * 1.44269504088896f;  // (a NaN stays one)
                st[128 + row] = s;
            }
        }
    }
}

// KEYS: rows are keys, tiles are queries (dK, dV); otherwise rows are queries (dQ).
template <int D, bool KEYS>
__global__ void __launch_bounds__(NTHREADS, 1) k_window_bwd(const __grid_constant__ BwdMaps maps,
                                                           const __grid_constant__ BwdParams p) {
    using LY = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- work item: (sequence and key head, row tile).  The row tiles with the most
    // columns first, those of all heads: early keys (first tokens; no left bound), late queries
    // (frames, three and the first: 5,090 -> 4,930 us with the forward; a clip 133 -> 125).  Without
    // bounds head after head, as in window_attn.cu.
    const int tiles = KEYS ? p.tiles_k : p.tiles_q;
    const int part = KEYS ? blockIdx.x % p.max_parts : 0, item = KEYS ? blockIdx.x / p.max_parts : blockIdx.x;
    const bool spread = p.w.left >= 0 || p.w.right >= 0;
    const int bh = spread ? item % (p.B * p.Hk) : item / tiles, nth = spread ? item / (p.B * p.Hk) : item % tiles;
    const int rt = KEYS ? nth : tiles - 1 - nth;
    const int b = bh / p.Hk, hk = bh % p.Hk;
    const int ql = seq_len(p.q_lens, b, p.Lq, p.err), kl = seq_len(p.k_lens, b, p.Lk, p.err);
    const int off = kl - ql;
    const int r0 = KEYS ? rt * 128 : rt * p.TT;  // first key, or first token

    int lo_c = 0, n_tiles = 0, nsink = 0;  // lo_c: first tile (behind the first tokens' tiles)
    bool tail = false;                     // the last tile holds rows behind the sequence that TMA does not zero
    int tail_row = 0;
    int parts = 1;
    if (KEYS) {
        const KeyTile t = key_tile(p, r0, ql, kl);
        parts = t.parts;
        if (part >= parts) return;  // (the whole CTA, before it holds anything)
        const int j0 = (int)((long long)t.n * part / parts), j1 = (int)((long long)t.n * (part + 1) / parts);
        lo_c = t.lo + j0, n_tiles = j1 - j0;
        tail = n_tiles > 0 && (lo_c + n_tiles) * p.TT > ql && ql < p.Lq;
        tail_row = (ql - (lo_c + n_tiles - 1) * p.TT) * p.G;
    } else if (r0 < ql) {
        const int lo = row_range(p.w, r0 + off, kl).lo;
        const int hi = row_range(p.w, min(r0 + p.TT, ql) - 1 + off, kl).hi;
        if (hi > 0) {
            lo_c = lo / 128;
            nsink = min((min(p.w.sinks, hi) + 127) / 128, lo_c);
            n_tiles = nsink + (hi + 127) / 128 - lo_c;
            tail = (hi + 127) / 128 * 128 > kl && kl < p.Lk;
            tail_row = kl - (hi + 127) / 128 * 128 + 128;
        }
    }
    // first key of key tile j, or first token of query tile j
    auto tile_base = [&](int j) { return KEYS ? (lo_c + j) * p.TT : (j < nsink ? j : lo_c + j - nsink) * 128; };

    const uint32_t bar0 = sbase + LY::OFF_BAR;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
    // (a local pointer: with the expression in the call the compiler spills more)
    uint32_t *noted = &p.err->timeout;
    auto wait = [&](uint32_t bar, uint32_t parity) { return wait_or_note(bar, parity, noted, p.launch); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + LY::OFF_BAR + 8 * NBAR);

    const int packed = p.G * p.TT;  // rows of a query tile
    const uint32_t qbytes = LY::HALVES * packed * 128;
    // L0 (t = 0, with the statistics of its queries) or L1 tile j, by the producer thread
    auto load_tile = [&](int t, int j) {
        const int s = j & 1, base = tile_base(j);
        const uint32_t bar = BAR((t ? B_1F : B_0F) + s);
        mbar_arrive_expect_tx(bar, (KEYS ? qbytes : LY::TILE) + (KEYS && t == 0 ? kStats * 4 : 0));
        for (int hf = 0; hf < LY::HALVES; ++hf) {
            const uint32_t dst = sbase + (t ? LY::OFF_L1 : LY::OFF_L0) + s * LY::TILE + hf * 128 * 128;
            if (KEYS) tma_load_5d(dst, t ? &maps.l1 : &maps.l0, hf * 64, 0, base, hk, b, bar);
            else tma_load_4d(dst, t ? &maps.l1 : &maps.l0, hf * 64, base, hk, b, bar);
        }
    };
    auto load_stats = [&](int j) {
        const int s = j & 1;
        bulk_load(sbase + LY::OFF_ST + s * kStats * 4, p.stats + ((int64_t)bh * p.tiles_q + lo_c + j) * kStats, kStats * 4, BAR(B_0F + s));
    };
    if (tid == 8 * 32) {  // (the producer, so that the first loads start before the other warps are there)
        mbar_init(BAR(B_FF), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(BAR(B_0F + i), 1);
            mbar_init(BAR(B_0E + i), 1);
            mbar_init(BAR(B_1F + i), 1);
            mbar_init(BAR(B_1E + i), 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(BAR(B_PF + h), 4);
            mbar_init(BAR(B_DF + h), 4);
        }
        mbar_init(BAR(B_SF), 1);
        mbar_init(BAR(B_DPF), 1);
        mbar_init(BAR(B_Z0), 1);
        mbar_init(BAR(B_Z1), 1);
        mbar_init(BAR(B_AF), 1);
        fence_mbar_init();
        if (n_tiles > 0) {
            mbar_arrive_expect_tx(BAR(B_FF), 2 * (KEYS ? LY::TILE : qbytes));
            for (int t = 0; t < 2; ++t)
                for (int hf = 0; hf < LY::HALVES; ++hf) {
                    const uint32_t dst = sbase + LY::OFF_F + t * LY::TILE + hf * 128 * 128;
                    if (KEYS) tma_load_4d(dst, t ? &maps.f1 : &maps.f0, hf * 64, r0, hk, b, BAR(B_FF));
                    else tma_load_5d(dst, t ? &maps.f1 : &maps.f0, hf * 64, 0, r0, hk, b, BAR(B_FF));
                }
            for (int j = 0; j < 2 && j < n_tiles; ++j) load_tile(0, j), load_tile(1, j);
            if (KEYS) {
                wait_predecessor();
                for (int j = 0; j < 2 && j < n_tiles; ++j) load_stats(j);
            }
        }
    }
    __syncwarp();
    if (KEYS && packed < 128) {
        // The rows of the query stages that no load fills enter products over
        // the rows: zeros.
        for (int t = tid; t < 4 * LY::HALVES * (128 - packed) * 8; t += NTHREADS) {
            const int i = t % ((128 - packed) * 8), blk = t / ((128 - packed) * 8);
            *reinterpret_cast<uint4 *>(sm + LY::OFF_L0 + blk * 128 * 128 + packed * 128 + i * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    release_successor();
    constexpr uint32_t tS = 0, tP = 128, tA1 = 256, tA2 = 384;  // (all 512 columns are this CTA's: they start at 0)
    bool ok = true;

    if (warp >= 8) {
        reg_dealloc<kRegsOther>();
        if (warp == 9) {
            // ------------------------------------------------ MMA issuer
            // (the whole warp, with the same values in every lane: see stream_device.cuh)
            const int n = uniform(n_tiles), clean = uniform(tail);
            if (n > 0) {
                constexpr uint32_t ISS = idesc_bf16_f32(128, 128, false);
                constexpr uint32_t ITS = idesc_bf16_f32(128, D, true);
                constexpr uint32_t STEP = LY::TILE >> 4;
                const uint32_t leader = elect_one();
                const Desc f0 = make_desc(sdesc_sw128(sbase + LY::OFF_F, 16, 1024));
                const Desc f1 = make_desc(sdesc_sw128(sbase + LY::OFF_F + LY::TILE, 16, 1024));
                const Desc k0 = make_desc(sdesc_sw128(sbase + LY::OFF_L0, 16, 1024));  // as K-major operands
                const Desc k1 = make_desc(sdesc_sw128(sbase + LY::OFF_L1, 16, 1024));
                const Desc m0 = make_desc(sdesc_sw128(sbase + LY::OFF_L0, 128 * 128, 1024));  // as MN-major operands
                const Desc m1 = make_desc(sdesc_sw128(sbase + LY::OFF_L1, 128 * 128, 1024));
                auto wait_all = [&](int bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(BAR(bar), parity)) != 0; };
                auto cleaned = [&](int bar, int j) { return !clean || j + 1 < n || wait_all(bar, 0); };
                bool go = wait_all(B_FF, 0) && wait_all(B_0F, 0) && cleaned(B_Z0, 0);
                tc_fence_after();
                if (go) {
                    mma_rows<D>(leader, tS, f0, k0, ISS);
                    commit(leader, BAR(B_SF));
                    go = wait_all(B_1F, 0) && cleaned(B_Z1, 0);
                    tc_fence_after();
                    if (go) {
                        mma_rows<D>(leader, tP, f1, k1, ISS);
                        commit(leader, BAR(B_DPF));
                    }
                }
                for (int j = 0; j < n && go; ++j) {
                    const bool more = j + 1 < n;
                    const int s = j & 1, s2 = s ^ 1, ph2 = ((j + 1) >> 1) & 1;
                    const Desc x1 = KEYS ? m1 : m0;
                    if (more && !(go = wait_all(B_0F + s2, ph2) && cleaned(B_Z0, j + 1))) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!(go = wait_all(B_PF + h, j & 1))) break;
                        tc_fence_after();
                        mma_weights<64>(leader, tA1, tS, Desc{x1.lo + s * STEP, x1.hi}, ITS, j > 0 || h > 0 ? 1u : 0u, h);
                    }
                    if (!go) break;
                    if (more) {
                        mma_rows<D>(leader, tS, f0, Desc{k0.lo + s2 * STEP, k0.hi}, ISS);
                        commit(leader, BAR(B_SF));
                    }
                    commit(leader, BAR(B_1E + s));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!(go = wait_all(B_DF + h, j & 1))) break;
                        tc_fence_after();
                        mma_weights<64>(leader, tA2, tP, Desc{m0.lo + s * STEP, m0.hi}, ITS, j > 0 || h > 0 ? 1u : 0u, h);
                    }
                    if (!go) break;
                    commit(leader, BAR(B_0E + s));
                    if (more) {
                        if (!(go = wait_all(B_1F + s2, ph2) && cleaned(B_Z1, j + 1))) break;
                        tc_fence_after();
                        mma_rows<D>(leader, tP, f1, Desc{k1.lo + s2 * STEP, k1.hi}, ISS);
                        commit(leader, BAR(B_DPF));
                    }
                }
                commit(leader, BAR(B_AF));
                mbar_wait(BAR(B_AF), 0);
            }
        } else if (warp == 8 && n_tiles > 0) {
          if (lane == 0) {
            // ------------------------------------------------ TMA producer
            int done[2] = {min(2, n_tiles), min(2, n_tiles)};
            for (int j = 2; j < n_tiles && ok; ++j) {
                for (int t = 0; t < 2; ++t) {
                    if (!(ok = wait(BAR((t ? B_1E : B_0E) + (j & 1)), ((j >> 1) - 1) & 1))) break;
                    load_tile(t, j);
                    if (KEYS && t == 0) load_stats(j);
                    ++done[t];
                }
            }
            // Loads still in flight must land before the CTA exits.
            for (int t = 0; t < 2; ++t)
                for (int j = max(done[t] - 2, 0); j < done[t]; ++j) mbar_wait(BAR((t ? B_1F : B_0F) + (j & 1)), (j >> 1) & 1);
            mbar_wait(BAR(B_FF), 0);
          }
          __syncwarp();
          if (tail && __shfl_sync(0xFFFFFFFFu, (int)ok, 0)) {
            // ------------------------------------------------ rows behind the sequence
            // (by the producer, which has followed every phase of the stages)
            const int j = n_tiles - 1, s = j & 1;
            for (int t = 0; t < 2; ++t) {
                mbar_wait(BAR((t ? B_1F : B_0F) + s), (j >> 1) & 1);
                for (int hf = 0; hf < LY::HALVES; ++hf)
                    for (int i = max(tail_row, 0) * 8 + lane; i < 128 * 8; i += 32)
                        *reinterpret_cast<uint4 *>(sm + (t ? LY::OFF_L1 : LY::OFF_L0) + s * LY::TILE + hf * 128 * 128 + i * 16) =
                            make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(t ? B_Z1 : B_Z0));
            }
          }
        }
        __syncwarp();
    } else {
        reg_alloc<kRegsMath>();
        // ------------------------------------------------ P and dS; epilogue
        const int half = warp >> 2, row = tid & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t mS = tmem + lane_off + tS + half * 64, mP = tmem + lane_off + tP + half * 64;
        float *row_sum = reinterpret_cast<float *>(sm + LY::OFF_R);
        // KEYS: key r0 + row, its visible tokens; otherwise token and head of the row, its visible keys
        const int g = row % p.G, i = r0 + row / p.G;
        RowRange rr{0, 0x7FFFFFFF};  // a row that is not live never makes its warp mask
        int sink = 0;
        bool live;
        float nl = -INFINITY, delta = 0.f, rsum = 0.f;
        uint64_t true_sum = f2_pack(0.f, 0.f);
        float *stat = p.stats + ((int64_t)bh * p.tiles_q + rt) * kStats;
        wait_predecessor();
        if (KEYS) {
            live = r0 + row < kl;
            if (live) rr = key_range(p.w, r0 + row, off, ql, kl);
        } else {
            live = row < packed && i < ql;
            if (live) {
                rr = row_range(p.w, i + off, kl);
                sink = min(p.w.sinks, rr.hi);
                nl = stat[row], delta = stat[128 + row];
            }
        }
        const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
        for (int j = 0; j < n_tiles; ++j) {
            const int s = j & 1, base = tile_base(j);
            // columns of this thread that it sees: [c_lo, c_hi) and, of keys, the first ones
            int c_lo, c_hi, c_sink = 0;
            bool full;
            if (KEYS) {
                const long long lo = (long long)(rr.lo - base) * p.G, hi = (long long)(rr.hi - base) * p.G;
                full = lo <= 0 && hi >= packed;  // columns behind the packed ones have P = 0
                c_lo = (int)max(min(lo, 1024ll), -1024ll) - half * 64, c_hi = (int)max(min(hi, 1024ll), -1024ll) - half * 64;
            } else {
                full = base + 128 <= rr.hi && (base >= rr.lo || base + 128 <= sink);
                c_lo = rr.lo - base - half * 64, c_hi = rr.hi - base - half * 64, c_sink = sink - base - half * 64;
            }
            if (!live) full = true;
            const bool masked = !__all_sync(0xFFFFFFFFu, full);
            const float *st = reinterpret_cast<const float *>(sm + LY::OFF_ST + s * kStats * 4) + half * 64;
            bool got = true;
            float nls[KEYS ? 64 : 1];
            if (KEYS) {  // the statistics came with L0, before S
                got = wait(BAR(B_0F + s), (j >> 1) & 1);
#pragma unroll
                for (int e = 0; e < 64; e += 4) *reinterpret_cast<float4 *>(nls + (KEYS ? e : 0)) = *reinterpret_cast<const float4 *>(st + e);
            }
            got = wait(BAR(B_SF), j & 1) && got;
            if (!__all_sync(0xFFFFFFFFu, got)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t x[2][32], pk[32];
            tmem_ld32(mS, x[0]);
            tmem_ld32(mS + 32, x[1]);
            tmem_ld_wait();
            // ---- P = 2^(s c - lse)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float n0 = KEYS ? nls[KEYS ? c * 32 + e : 0] : nl, n1 = KEYS ? nls[KEYS ? c * 32 + e + 1 : 0] : nl;
                    float y0, y1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), c2, f2_pack(n0, n1)), y0, y1);
                    x[c][e] = __float_as_uint(ex2_approx(y0)), x[c][e + 1] = __float_as_uint(ex2_approx(y1));
                }
                if (masked) {
                    const uint32_t vm = (low_mask(c_hi - 32 * c) & ~low_mask(c_lo - 32 * c)) | low_mask(c_sink - 32 * c);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[c][e] = ((vm >> e) & 1u) ? x[c][e] : 0u;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    pk[c * 16 + e / 2] = pack_bf16x2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
            }
            tmem_st32(mS, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(B_PF + half));
            // ---- dS = P (dP - delta)
            if (!__all_sync(0xFFFFFFFFu, wait(BAR(B_DPF), j & 1))) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t d[32];
                tmem_ld32(mP + c * 32, d);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    float4 d4 = make_float4(delta, delta, delta, delta);
                    if (KEYS) d4 = *reinterpret_cast<const float4 *>(st + 128 + c * 32 + e);
                    const uint64_t y01 = f2_mul(f2_pack(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])),
                                                f2_sub(f2_pack(__uint_as_float(d[e]), __uint_as_float(d[e + 1])), f2_pack(d4.x, d4.y)));
                    const uint64_t y23 = f2_mul(f2_pack(__uint_as_float(x[c][e + 2]), __uint_as_float(x[c][e + 3])),
                                                f2_sub(f2_pack(__uint_as_float(d[e + 2]), __uint_as_float(d[e + 3])), f2_pack(d4.z, d4.w)));
                    float y[4];
                    f2_unpack(y01, y[0], y[1]), f2_unpack(y23, y[2], y[3]);
                    const uint32_t w0 = pack_bf16x2(y[0], y[1]), w1 = pack_bf16x2(y[2], y[3]);
                    pk[c * 16 + e / 2] = w0, pk[c * 16 + e / 2 + 1] = w1;
                    if (!KEYS) {
                        rsum += (__uint_as_float(w0 << 16) + __uint_as_float(w0 & 0xFFFF0000u)) +
                                (__uint_as_float(w1 << 16) + __uint_as_float(w1 & 0xFFFF0000u));
                        true_sum = f2_add(true_sum, f2_add(y01, y23));
                    }
                }
            }
            tmem_st32(mP, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(B_DF + half));
        }
        if (ok && n_tiles > 0 && !__all_sync(0xFFFFFFFFu, wait(BAR(B_AF), 0))) ok = false;
        tc_fence_after();
        if (!KEYS) {
            float t0, t1;
            f2_unpack(true_sum, t0, t1);
            row_sum[tid] = rsum, row_sum[256 + tid] = t0 + t1;
            asm volatile("bar.sync 2, 256;" ::: "memory");
            rsum = row_sum[row] + row_sum[128 + row];
            if (half == 0 && live && n_tiles > 0) stat[128 + row] = delta + (row_sum[256 + row] + row_sum[384 + row]);
        }
        const bool some = live && n_tiles > 0;
        if (KEYS) {
            // half 0: dV = A1; half 1: dK = scale A2
            const View &v = half ? p.dk : p.dv;
            const float f = half ? p.scale : 1.f;
            const bool store = ok && r0 + row < p.Lk;
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<bf16 *>(v.p) + b * v.b + hk * v.h + (int64_t)(r0 + row) * v.l);
            float4 *dst4 = nullptr;
            if (parts > 1)
                dst4 = reinterpret_cast<float4 *>(
                    p.parts + (((((int64_t)bh * p.part_tiles + rt) * p.max_parts + part) * 2 + half) * 128 + row) * D);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (n_tiles > 0) {
                    tmem_ld32(tmem + lane_off + (half ? tA2 : tA1) + c * 32, o);
                    tmem_ld_wait();
                }
                if (store && parts > 1) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float *x = reinterpret_cast<const float *>(o + 4 * q);
                        dst4[c * 8 + q] = some ? make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                } else if (store) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float *x = reinterpret_cast<const float *>(o + 8 * q);
                        dst[c * 4 + q] = some ? make_uint4(pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f),
                                                           pack_bf16x2(x[4] * f, x[5] * f), pack_bf16x2(x[6] * f, x[7] * f))
                                              : make_uint4(0, 0, 0, 0);
                    }
                }
                __syncwarp();
            }
        } else {
            // dQ = scale (A2 - r A1), half the columns each
            const bool store = ok && row < packed && i < p.Lq;
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<bf16 *>(p.dq.p) + b * p.dq.b + (int64_t)(hk * p.G + g) * p.dq.h +
                                                   (int64_t)i * p.dq.l + half * (D / 2));
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
                uint32_t a1[32], a2[32];
                if (n_tiles > 0) {
                    tmem_ld32(tmem + lane_off + tA1 + half * (D / 2) + c * 32, a1);
                    tmem_ld32(tmem + lane_off + tA2 + half * (D / 2) + c * 32, a2);
                    tmem_ld_wait();
                }
                if (store) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            y[e] = p.scale * fmaf(-rsum, __uint_as_float(a1[8 * q + e]), __uint_as_float(a2[8 * q + e]));
                        dst[c * 4 + q] = some ? make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                           pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]))
                                              : make_uint4(0, 0, 0, 0);
                    }
                }
            }
        }
    }
#undef BAR
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// dV and dK of the key tiles in parts: the parts' sums in order.  One thread for four
// elements of a row.
template <int D>
__global__ void __launch_bounds__(256) k_sum_parts(const BwdParams p) {
    const int tile = blockIdx.x % p.part_tiles, bh = blockIdx.x / p.part_tiles;
    const int b = bh / p.Hk, hk = bh % p.Hk, r0 = tile * 128;
    const int ql = seq_len(p.q_lens, b, p.Lq, p.err), kl = seq_len(p.k_lens, b, p.Lk, p.err);
    const int parts = key_tile(p, r0, ql, kl).parts;
    wait_predecessor();  // (always: the end of this kernel stands for the end of the one before)
    if (parts == 1) return;
    const float4 *src = reinterpret_cast<const float4 *>(p.parts + ((int64_t)bh * p.part_tiles + tile) * p.max_parts * 2 * 128 * D);
    for (int t = blockIdx.y * 256 + threadIdx.x; t < 2 * 128 * D / 4; t += gridDim.y * 256) {
        const int half = t / (128 * D / 4), row = t / (D / 4) % 128, e = t % (D / 4) * 4;
        if (r0 + row >= p.Lk) continue;
        float4 s = src[t];
#pragma unroll 4
        for (int i = 1; i < parts; ++i) {
            const float4 x = src[(int64_t)i * (2 * 128 * D / 4) + t];
            s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
        }
        const View &v = half ? p.dk : p.dv;
        *reinterpret_cast<uint2 *>(static_cast<bf16 *>(v.p) + b * v.b + hk * v.h + (int64_t)(r0 + row) * v.l + e) =
            make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    }
}

int64_t query_tiles(const WinArgs &a) {
    const int TT = 128 / a.G;
    return (a.Lq + TT - 1) / TT;
}

}  // namespace

namespace {

// Parts of the key tiles' work.  A part takes at most half of what an SM has to do on
// average, and eight query tiles at least.
struct Parts {
    int chunk, max_parts, part_tiles;
};

Parts plan_parts(const WinArgs &a) {
    const int64_t all = query_tiles(a), tiles_k = (a.Lk + 127) / 128, heads = (int64_t)a.B * a.Hk;
    Parts pt{1 << 30, 1, 0};
    if (all == 0 || tiles_k == 0) return pt;
    WinRule w = a.w;
    w.sinks = 0;  // (a key that is no first token is seen by its window alone)
    const int64_t window = std::min(all, window_tiles(w, 128, a.Lk, a.Lq, 128 / a.G));  // of keys without the first tokens
    const int64_t first = a.w.left < 0 ? tiles_k : std::min<int64_t>(tiles_k, (a.w.sinks + (int64_t)127) / 128);
    const int64_t total = a.w.left < 0 ? heads * tiles_k * (a.w.right < 0 ? all : (all + 1) / 2)
                                       : heads * (first * all + (tiles_k - first) * window);
    const int64_t chunk = std::max<int64_t>(8, (total + 2 * 148 - 1) / (2 * 148));
    const int64_t most = first > 0 ? all : window;
    if (most <= chunk) return pt;
    pt.chunk = (int)chunk;
    pt.max_parts = (int)std::min<int64_t>((most + chunk - 1) / chunk, 64);
    pt.part_tiles = (int)(window > chunk ? tiles_k : first);
    return pt;
}

int64_t stats_floats(const WinArgs &a) { return (int64_t)a.B * a.Hk * query_tiles(a) * kStats; }

}  // namespace

int64_t window_bwd_workspace(const WinArgs &a) {
    const Parts pt = plan_parts(a);
    return (stats_floats(a) + (int64_t)a.B * a.Hk * pt.part_tiles * pt.max_parts * 2 * 128 * a.d) * 4;
}

cudaError_t launch_window_bwd(const WinBwdArgs &g, cudaStream_t s) {
    const WinArgs &a = g.f;
    BwdParams p{};
    p.dq = g.dq, p.dk = g.dk, p.dv = g.dv;
    p.stats = static_cast<float *>(a.ws);
    p.q_lens = a.q_lens, p.k_lens = a.k_lens;
    p.B = a.B, p.Hq = a.Hq, p.Hk = a.Hk, p.G = a.G, p.TT = 128 / a.G, p.Lq = a.Lq, p.Lk = a.Lk;
    p.tiles_q = (int)query_tiles(a), p.tiles_k = (a.Lk + 127) / 128;
    p.w = a.w, p.scale = a.scale, p.scale_log2 = a.scale * 1.44269504088896f;
    p.launch = next_launch_id(), p.err = a.err;
    const Parts pt = plan_parts(a);
    p.parts = p.stats + stats_floats(a);
    p.chunk = pt.chunk, p.max_parts = pt.max_parts, p.part_tiles = pt.part_tiles;
    const int64_t nq = (int64_t)a.B * a.Hk * p.tiles_q, nk = (int64_t)a.B * a.Hk * p.tiles_k * pt.max_parts;
    if (nq > 0x7FFFFFFF || nk > 0x7FFFFFFF) return cudaErrorInvalidValue;
    BwdMaps mq{}, mk{};  // rows = queries; rows = keys
    cudaError_t e = cudaSuccess;
    auto qmap = [&](CUtensorMap *m, const View &v) {
        if (e == cudaSuccess && a.Lq > 0) e = map_rows_packed(m, v, a.B, a.Hk, a.G, a.Lq, a.d, p.TT);
    };
    auto kmap = [&](CUtensorMap *m, const View &v) {
        if (e == cudaSuccess && a.Lk > 0) e = map_rows(m, v, a.B, a.Hk, a.Lk, a.d, 128);
    };
    qmap(&mq.f0, a.q), qmap(&mq.f1, g.go), kmap(&mq.l0, a.k), kmap(&mq.l1, a.v);
    if (e != cudaSuccess) return e;
    mk.f0 = mq.l0, mk.f1 = mq.l1, mk.l0 = mq.f0, mk.l1 = mq.f1;
    auto go = [&](auto kern, uint32_t smem, const BwdMaps &m, int64_t grid) {
        if (e != cudaSuccess || grid == 0) return;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return;
        if (nq > 0) {
            e = launch_after(kern, (unsigned)grid, NTHREADS, smem, s, m, p);
        } else {  // the stream's previous kernel is not one of this call
            kern<<<(unsigned)grid, NTHREADS, smem, s>>>(m, p);
            AC_NOTE_LAUNCH();
            e = cudaGetLastError();
        }
    };
    if (nq > 0) {
        if (a.d == 128)
            k_row_stats<128><<<(unsigned)nq, 256, 0, s>>>(g.go, a.o, a.lse, p);
        else
            k_row_stats<64><<<(unsigned)nq, 256, 0, s>>>(g.go, a.o, a.lse, p);
        AC_NOTE_LAUNCH();
        e = cudaGetLastError();
    }
    if (a.d == 128) {
        go(k_window_bwd<128, false>, Layout<128>::SMEM, mq, nq);
        go(k_window_bwd<128, true>, Layout<128>::SMEM, mk, nk);
    } else {
        go(k_window_bwd<64, false>, Layout<64>::SMEM, mq, nq);
        go(k_window_bwd<64, true>, Layout<64>::SMEM, mk, nk);
    }
    if (e == cudaSuccess && pt.part_tiles > 0) {
        const dim3 grid((unsigned)((int64_t)a.B * a.Hk * pt.part_tiles), 8);
        e = launch_after(a.d == 128 ? k_sum_parts<128> : k_sum_parts<64>, grid, 256, 0, s, p);
    }
    return e;
}

}  // namespace ac
