// window_attn.cu -- attention within a window and over a few first tokens, on
// tcgen05 / TMEM, over bf16 keys or over the paged 8-bit cache.
//
// One pass over the visible keys with the running maximum and sum of a softmax:
// S = Q K^T, P = 2^(S c - m), O += P V, with c = scale log2(e); O is divided by
// the sum at the end.
//
// A CTA takes 256 query rows as two 128-row tiles that share every K/V tile.
// Rows are packed token by token over the G query heads of one key head (row r
// of a tile: token r / G, head r % G; TT = floor(128 / G) tokens), so shared
// heads read their keys once and a tile spans few tokens, hence few keys.  The
// visible keys of a row are one interval and the first tokens; the CTA walks
// the 128-key tiles that meet any of its rows' and masks columns only in tiles
// where some row of the warp does not see all of them.
//
// Warp roles (three warpgroups; five over 8-bit keys):
//   warps 0-3 / 4-7  softmax + epilogue of row tile 0 / 1; thread t owns row t (bf16 keys, one
//                    row tile: of its even / odd key tiles)
//   warp 8           TMA producer (Q; bf16 keys: K and V, and in the last tile it
//                    zeroes the V rows behind the sequence: 0 x garbage would be NaN)
//   warp 9           TMEM allocator and tcgen05.mma issuer
//   8-bit keys: warps 12-15 load the codes of K and warps 16-19 those of V into
//               registers and store them, times their pages' scales, as bf16 (exact)
//               in the swizzled layout that the products read.  The codes of
//               the next tile are in flight while a thread waits for its stage, and
//               the scales and page numbers of the ones after that too.  Each thread
//               keeps its place within 16 rows, so that a tile costs few address
//               computations: the issue slots, and the instruction cache, are
//               shared with the softmax.
// Tensor memory (512 columns): S_0 | S_1 | O_0 | O_1; each half of P overwrites
// the first half of the scores it came from.
// Few query tiles: the key tiles are split over several CTAs, whose partial O
// and log-sum-exp k_combine joins.
//
// Rounding: P to bf16, the operand type of the product, off by 2^-8 relative at most
// and random over the keys; over the cache too, because only bf16 has the exponents for
// weights far below the largest and for pages of very different scales.  (fp16
// with the scales in the exponents of P loses a weight 2^-25 below the largest one times its
// page's scale, which the sum still counts.)  O once at the end; everything else is fp32.
// Bound by the softmax's chain: a pair of row tiles takes 3,500 cycles per key tile (S
// 1,100 waited for, its load 150, maximum 320, exponentials 1,310, P 285, per row tile)
// where the products take 2,048.  Frame-causal, 32,760 tokens in frames of 1,560, three
// frames and the first, 12 heads, d = 128 (1.17 TFLOP): 1,040 us alone, 1.12 PFLOP/s, 67%
// of the measured cuBLAS rate; 1,200 us in a long loop under the power limit.  1,560
// rows over 18,720 keys, 12 heads (0.18 TFLOP): 204 us; over the codes of the 8-bit cache
// 252, because every CTA converts them anew and reads its scores twice (registers go to
// the converting threads): many rows take the cache as bf16 rows instead.  Dropped, in us
// of the two workloads (codes): two threads a row (1,266 in the loop; 595), a quarter of the
// exponentials as a polynomial on the FMA pipe (no difference), a persistent CTA (1,059
// against 1,028; 440 against 349 then), S in 64-key halves that go round on their own
// (1,215 in the loop; 341), each converting register refilled as soon as it is free (17 rows:
// 258 -> 290).
//
// Every mbarrier wait is bounded; on timeout the CTA notes it, waits for the loads and
// products that it issued (for a bounded time too) and frees its TMEM.
#include <type_traits>

#include "stream_device.cuh"
#include "stream_host.h"

namespace ac {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int NS = 2;  // K/V stages
template <bool C8>
struct Split {  // threads and registers: bf16 keys launch with 168 each, 8-bit keys with 96
    static constexpr int THREADS = C8 ? 640 : 384;
    static constexpr uint32_t SOFTMAX = C8 ? 152 : 200, OTHER = C8 ? 48 : 72, CONVERT = 64;
    static_assert(2 * SOFTMAX + OTHER + (C8 ? 2 * CONVERT : 0) <= THREADS / 128 * (C8 ? 96 : 168), "register split exceeds the launch");
};
constexpr float kRescaleLog2 = 8.0f;
constexpr int kConverters = 128;  // threads that convert K, and as many V

template <int D, bool C8>
struct Layout {
    static constexpr int HALVES = D / 64;  // 128-byte column halves of a row
    static constexpr uint32_t TILE = HALVES * 128 * 128;
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_K = 2 * TILE;
    static constexpr uint32_t OFF_V = OFF_K + NS * TILE;
    static constexpr uint32_t OFF_ROW = OFF_V + NS * TILE;  // [2][128] float2: maximum and sum of a row in each warpgroup
    static constexpr uint32_t OFF_BAR = OFF_ROW + (C8 ? 0 : 2 * 128 * 8);
    static constexpr uint32_t SMEM = OFF_BAR + 256 + 1024;  // 1024-byte alignment slack
};
static_assert(Layout<128, false>::SMEM <= 232448, "shared memory");

enum {
    B_KF = 0,     // [NS] K stage filled
    B_KE = 2,     // [NS] K stage free (MMA commit after both S products)
    B_VF = 4,     // [NS] V stage filled
    B_VE = 6,     // [NS] V stage free (MMA commit after both PV products)
    B_QF = 8,     // query tiles filled
    B_SF = 9,     // [2] S_i written (MMA commit)
    B_PF = 11,    // [2][2] half of P_i written (+ O_i rescaled) by the four softmax warps
    B_OF = 15,    // [2] last PV_i complete (MMA commit)
    B_DONE = 17,  // every MMA complete
    B_VZ = 18,    // V rows behind the sequence zeroed (bf16 keys)
    NBAR = 19
};

struct WinMaps {
    CUtensorMap q, k, v;
};

struct WinParams {
    View o;
    float *lse;
    float *part_o, *part_lse;  // [nsplit][B Hq Lq] partials when nsplit > 1
    const int *q_lens, *k_lens;
    int B, Hq, Hk, G, TT, Lq, Lk, tiles_q, nsplit;
    WinRule w;
    float scale_log2;
    const uint8_t *k8, *v8;
    const float *ks, *vs;
    const int *table;
    int pages, T, max_pages;
    uint32_t launch;
    OpErr *err;
};

__device__ __forceinline__ uint32_t low_mask(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

__device__ __forceinline__ uint4 load_codes(const uint8_t *src) {
    uint4 w;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(src));
    return w;
}

// C8: over the codes of the 8-bit cache.
template <int D, bool C8>
__global__ void __launch_bounds__(Split<C8>::THREADS, 1) k_window_attn(const __grid_constant__ WinMaps maps,
                                                            const __grid_constant__ WinParams p) {
    using LY = Layout<D, C8>;
    // The half of a tile's keys whose weights come first: over the cache the one that the
    // search for the maximum has read last.
    constexpr int FIRST_HALF = C8 ? 1 : 0;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- work item: (sequence and key head, pair of row tiles, part of the keys).
    // All heads' late tiles first: they see the most keys (16,384 tokens, causal, 12 heads: 751
    // -> 652 us).  Without bounds all see the same, and head after head keeps the keys in the L2
    // cache (1,593 against 1,666 us).
    int idx = blockIdx.x;
    const int sp = idx % p.nsplit;
    idx /= p.nsplit;
    const bool spread = p.w.left >= 0 || p.w.right >= 0;
    const int bh = spread ? idx % (p.B * p.Hk) : idx / p.tiles_q;
    const int qt = p.tiles_q - 1 - (spread ? idx / (p.B * p.Hk) : idx % p.tiles_q);
    const int b = bh / p.Hk, hk = bh % p.Hk;
    const int i0 = qt * 2 * p.TT;
    const int ql = seq_len(p.q_lens, b, p.Lq, p.err), kl = seq_len(p.k_lens, b, p.Lk, p.err);
    const int off = kl - ql;
    int lo_c = 0, hi_c = 0;
    if (i0 < ql) {
        lo_c = row_range(p.w, i0 + off, kl).lo;
        hi_c = row_range(p.w, min(i0 + 2 * p.TT, ql) - 1 + off, kl).hi;
    }
    const bool has1 = i0 + p.TT < ql;
    // One row tile alone: its key tiles go to the two warpgroups in turn, which are joined at the
    // end.  (17 rows over 32,760 bf16 keys, 64 heads: 214 -> 167 us.  Not over the cache, where the
    // code that this takes costs full pairs of tiles more than it gains: 299 -> 258 us, but a frame
    // of 1,560 tokens 317 -> 332.)
    const bool pair = C8 || has1;
    const int step = pair ? 1 : 2;
    const int sink_c = min(p.w.sinks, hi_c);
    const int wt0 = lo_c / BN, wt1 = (hi_c + BN - 1) / BN;
    const int nsink = min((sink_c + BN - 1) / BN, wt0);
    const int n_all = hi_c > 0 ? nsink + wt1 - wt0 : 0;
    const int j0 = (int)((long long)n_all * sp / p.nsplit), j1 = (int)((long long)n_all * (sp + 1) / p.nsplit);
    const int n_tiles = j1 - j0;
    auto tile_base = [&](int j) { return (j0 + j < nsink ? j0 + j : wt0 + (j0 + j - nsink)) * BN; };
    // rows of V behind the sequence that are not behind the tensor (which TMA fills with zeros)
    const bool tail = !C8 && n_tiles > 0 && j1 == n_all && wt1 * BN > kl && kl < p.Lk;

    const uint32_t bar0 = sbase + LY::OFF_BAR;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
    // (a local pointer: with the expression in the call the compiler spills more)
    uint32_t *noted = &p.err->timeout;
    auto wait = [&](uint32_t bar, uint32_t parity) { return wait_or_note(bar, parity, noted, p.launch); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + LY::OFF_BAR + 8 * NBAR);

    // K and V tiles j of the producer thread
    auto load_tile = [&](bool v, int j) {
        const int s = j % NS;
        const uint32_t bar = BAR((v ? B_VF : B_KF) + s);
        mbar_arrive_expect_tx(bar, LY::TILE);
        for (int hf = 0; hf < LY::HALVES; ++hf)
            tma_load_4d(sbase + (v ? LY::OFF_V : LY::OFF_K) + s * LY::TILE + hf * BN * 128, v ? &maps.v : &maps.k, hf * 64,
                        tile_base(j), hk, b, bar);
    };
    if (tid == 8 * 32) {  // (the producer, so that the first loads start before the other warps are there)
        for (int i = 0; i < NS; ++i) {
            mbar_init(BAR(B_KF + i), C8 ? kConverters : 1);
            mbar_init(BAR(B_KE + i), 1);
            mbar_init(BAR(B_VF + i), C8 ? kConverters : 1);
            mbar_init(BAR(B_VE + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(BAR(B_SF + i), 1);
            mbar_init(BAR(B_PF + 2 * i), 4);
            mbar_init(BAR(B_PF + 2 * i + 1), 4);
            mbar_init(BAR(B_OF + i), 1);
        }
        mbar_init(BAR(B_QF), 1);
        mbar_init(BAR(B_DONE), 1);
        mbar_init(BAR(B_VZ), 1);
        fence_mbar_init();
        if (n_tiles > 0) {
            const uint32_t bytes = LY::HALVES * p.G * p.TT * 128;
            mbar_arrive_expect_tx(BAR(B_QF), (has1 ? 2 : 1) * bytes);
            for (int t = 0; t < (has1 ? 2 : 1); ++t)
                for (int hf = 0; hf < LY::HALVES; ++hf)
                    tma_load_5d(sbase + LY::OFF_Q + t * LY::TILE + hf * BM * 128, &maps.q, hf * 64, 0, i0 + t * p.TT, hk, b,
                                BAR(B_QF));
            if (!C8)
                for (int j = 0; j < NS && j < n_tiles; ++j) load_tile(false, j), load_tile(true, j);
        }
    }
    __syncwarp();
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    release_successor();
    bool ok = true;

    if (C8 && warp >= 12) {
        reg_dealloc<Split<C8>::CONVERT>();
        if constexpr (C8) {
            // ------------------------------------------------ 8-bit pages to bf16 tiles
            const bool is_v = warp >= 16;
            const int ct = tid & 127, log_t = 31 - __clz(p.T);
            const int *table = p.table + (int64_t)b * p.max_pages;
            const float *scales = (is_v ? p.vs : p.ks) + hk;
            // A thread converts 16 codes of every 16 RS-th row: row r0 + RS k of a tile, chunk e.
            constexpr int CPR = D / 16, RS = kConverters / CPR, NCH = BN / RS;
            const int r0 = ct / CPR, e = ct % CPR;
            // Lane i < 8: table entry of keys 16 i .. 16 i + 15 of tile j, -1 where this CTA sees none
            // of them (then the table may hold anything); and the page, -1 when there is none.
            auto entry_of = [&](int j) -> int {
                if (lane >= 8 || j >= n_tiles) return -1;
                const int key = (tile_base(j) + 16 * lane) >> log_t << log_t;
                if (!((key < hi_c && key + p.T > lo_c) || key < sink_c)) return -1;
                const int page = __ldg(table + (key >> log_t));
                return page == -1 ? -2 : page;
            };
            auto page_of = [&](int entry) -> int {
                if (entry >= 0 && entry < p.pages) return entry;
                if (entry != -1) atomicOr(&p.err->bits, DEV_ERR_BOUNDS);
                return -1;
            };
            auto scale_of = [&](int page) { return page >= 0 ? __ldg(scales + (int64_t)page * p.Hk) : 1.f; };
            uint4 w[NCH];
            // Codes of tile j; `page`: of this lane's group of 16 keys.
            auto load = [&](int j, int page) {
                const uint8_t *group = nullptr;  // the group's first row
                if (page >= 0) group = (is_v ? p.v8 : p.k8) + (((int64_t)page * p.Hk + hk) * p.T + (16 * lane & (p.T - 1))) * D;
                const int rows = kl - tile_base(j);
#pragma unroll
                for (int k = 0; k < NCH; ++k) {
                    const unsigned long long at = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(group), (r0 + RS * k) >> 4);
                    w[k] = make_uint4(0, 0, 0, 0);
                    if (at && r0 + RS * k < rows) w[k] = load_codes(reinterpret_cast<const uint8_t *>(at) + (r0 & 15) * D + e * 16);
                }
            };
            // 128-byte rows of a column half, 16-byte pieces swizzled by the row
            uint8_t *dst = sm + (is_v ? LY::OFF_V : LY::OFF_K) + (e / 4) * BN * 128 + r0 * 128;
            const int sw0 = (((e % 4) * 2) ^ (r0 & 7)) << 4, sw1 = (((e % 4) * 2 + 1) ^ (r0 & 7)) << 4;
            if (n_tiles > 0) {
                // The codes of tile j + 1 are loaded one tile ahead, its scales two, its table entry three:
                // nothing here waits for a load that was just issued.
                int entry = entry_of(1), page = page_of(entry_of(0));
                float scale = scale_of(page), scale1;  // of this lane's page of tile j, and of tile j + 1
                load(0, page);
                page = page_of(entry);
                scale1 = scale_of(page);
                entry = entry_of(2);
                for (int j = 0; j < n_tiles; ++j) {
                    const int s = j % NS;
                    if (!__all_sync(0xFFFFFFFFu, j < NS || wait(BAR((is_v ? B_VE : B_KE) + s), ((j / NS) - 1) & 1))) {
                        ok = false;
                        break;
                    }
                    uint8_t *d = dst + s * LY::TILE;
#pragma unroll
                    for (int k = 0; k < NCH; ++k) {
                        const float f = __shfl_sync(0xFFFFFFFFu, scale, (r0 + RS * k) >> 4);
                        *reinterpret_cast<uint4 *>(d + k * RS * 128 + sw0) =
                            make_uint4(e4m3x2_to_bf16x2(w[k].x & 0xFFFFu, f), e4m3x2_to_bf16x2(w[k].x >> 16, f),
                                       e4m3x2_to_bf16x2(w[k].y & 0xFFFFu, f), e4m3x2_to_bf16x2(w[k].y >> 16, f));
                        *reinterpret_cast<uint4 *>(d + k * RS * 128 + sw1) =
                            make_uint4(e4m3x2_to_bf16x2(w[k].z & 0xFFFFu, f), e4m3x2_to_bf16x2(w[k].z >> 16, f),
                                       e4m3x2_to_bf16x2(w[k].w & 0xFFFFu, f), e4m3x2_to_bf16x2(w[k].w >> 16, f));
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(BAR((is_v ? B_VF : B_KF) + s));
                    if (j + 1 < n_tiles) {
                        load(j + 1, page);
                        scale = scale1;
                        page = page_of(entry);
                        scale1 = scale_of(page);
                        entry = entry_of(j + 3);
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        reg_dealloc<Split<C8>::OTHER>();
        if (warp == 9) {
            // ------------------------------------------------ MMA issuer
            // (the whole warp, with the same values in every lane: see stream_device.cuh)
            const int n = uniform(n_tiles), two = uniform(has1), solo = uniform(!pair), turn = solo ? 2 : 1, clean = uniform(tail);
            if (n > 0) {
                constexpr uint32_t IQK = idesc_bf16_f32(BM, BN, false);
                constexpr uint32_t IPV = idesc_bf16_f32(BM, D, true);
                constexpr uint32_t STEP = LY::TILE >> 4;
                const uint32_t leader = elect_one();
                const Desc dq0 = make_desc(sdesc_sw128(sbase + LY::OFF_Q, 16, 1024));
                const Desc dk0 = make_desc(sdesc_sw128(sbase + LY::OFF_K, 16, 1024));
                const Desc dv0 = make_desc(sdesc_sw128(sbase + LY::OFF_V, BN * 128, 1024));
                auto wait_all = [&](int bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(BAR(bar), parity)) != 0; };
                // (all 512 columns are this CTA's: tensor memory starts at address 0)
                auto issue_s = [&](int i, int j) {
                    mma_rows<D>(leader, i * BN, Desc{dq0.lo + (solo ? 0 : i) * STEP, dq0.hi}, Desc{dk0.lo + (j % NS) * STEP, dk0.hi}, IQK);
                    commit(leader, BAR(B_SF + i));
                };
                // the products of 64 keys, half h of P_i(j)
                auto issue_pv = [&](int i, int j, int h) {
                    mma_weights<64>(leader, 256 + i * 128, i * BN, Desc{dv0.lo + (j % NS) * STEP, dv0.hi}, IPV,
                                    j >= turn || h != FIRST_HALF ? 1u : 0u, h);
                };
                bool go = wait_all(B_QF, 0) && wait_all(B_KF, 0);
                tc_fence_after();
                if (go) {
                    issue_s(0, 0);
                    if (two) issue_s(1, 0);
                    commit(leader, BAR(B_KE));
                }
                if (go && solo && n > 1) {
                    go = wait_all(B_KF + 1, 0);
                    tc_fence_after();
                    if (go) {
                        issue_s(1, 1);
                        commit(leader, BAR(B_KE + 1));
                    }
                }
                for (int j = 0; j < n && go; ++j) {
                    const int next = j + turn;  // the tile whose scores take the place of tile j's weights
                    const bool more = next < n;
                    // V and the next K are there long before P
                    if (!(go = wait_all(B_VF + j % NS, (j / NS) & 1) && (!clean || j + 1 < n || wait_all(B_VZ, 0)) &&
                               (!more || wait_all(B_KF + next % NS, (next / NS) & 1))))
                        break;
                    for (int i = solo ? j & 1 : 0; i < (solo ? (j & 1) + 1 : two ? 2 : 1); ++i) {
                        for (int hh = 0; hh < 2 && go; ++hh) {
                            const int h = hh ^ FIRST_HALF;
                            if (!(go = wait_all(B_PF + 2 * i + h, (solo ? j >> 1 : j) & 1))) break;
                            tc_fence_after();
                            issue_pv(i, j, h);
                        }
                        if (!go) break;
                        if (more) issue_s(i, next);
                        else commit(leader, BAR(B_OF + i));
                    }
                    if (!go) break;
                    if (more) commit(leader, BAR(B_KE + next % NS));
                    commit(leader, BAR(B_VE + j % NS));
                }
                commit(leader, BAR(B_DONE));
                mbar_wait(BAR(B_DONE), 0);
            }
            __syncwarp();
        } else if (warp == 8 && lane == 0 && n_tiles > 0) {
            if (!C8) {
                // -------------------------------------------- K/V producer
                int kd = min(NS, n_tiles), vd = kd;
                // One row tile: K runs a tile ahead of V, because S is issued two tiles ahead of P V.
                const int lag = step - 1;
                for (int j = NS; j < n_tiles + lag; ++j) {
                    if (j < n_tiles) {
                        if (!(ok = wait(BAR(B_KE + j % NS), ((j / NS) - 1) & 1))) break;
                        load_tile(false, j);
                        ++kd;
                    }
                    const int jv = j - lag;
                    if (jv >= NS) {
                        if (!(ok = wait(BAR(B_VE + jv % NS), ((jv / NS) - 1) & 1))) break;
                        load_tile(true, jv);
                        ++vd;
                    }
                }
                // Loads still in flight must land before the CTA exits.
                for (int j = max(kd - NS, 0); j < kd; ++j) mbar_wait(BAR(B_KF + j % NS), (j / NS) & 1);
                for (int j = max(vd - NS, 0); j < vd; ++j) mbar_wait(BAR(B_VF + j % NS), (j / NS) & 1);
                mbar_wait(BAR(B_QF), 0);
            }
        }
        if (!C8 && warp == 8 && tail) {
            // V rows behind the sequence, by the producer, which has followed every phase
            __syncwarp();
            const int j = n_tiles - 1, s = j % NS, r0 = kl - tile_base(j);
            if (__shfl_sync(0xFFFFFFFFu, (int)ok, 0)) {
                mbar_wait(BAR(B_VF + s), (j / NS) & 1);
                for (int hf = 0; hf < LY::HALVES; ++hf)
                    for (int i = r0 * 8 + lane; i < BN * 8; i += 32)
                        *reinterpret_cast<uint4 *>(sm + LY::OFF_V + s * LY::TILE + hf * BN * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(B_VZ));
            }
        }
        if (C8 && warp == 8 && lane == 0 && n_tiles > 0) mbar_wait(BAR(B_QF), 0);  // in flight until then
        __syncwarp();
    } else {
        reg_alloc<Split<C8>::SOFTMAX>();
        // ------------------------------------------------ softmax + epilogue
        const int wg = warp >> 2;
        const int row = tid & 127;
        const int g = row % p.G, i = i0 + (pair ? wg * p.TT : 0) + row / p.G;
        const bool mine = row < p.G * p.TT && i < p.Lq;
        const bool live = mine && i < ql;
        // A row that is not live computes something that is not used: it sees
        // every column, so that it never makes its warp mask.
        RowRange rr{0, 0x7FFFFFFF};
        if (live) rr = row_range(p.w, i + off, kl);
        const int sink = min(p.w.sinks, rr.hi);
        float m_run = -INFINITY, l_run = 0.f;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + wg * BN;
        const uint32_t tO = tmem + lane_off + 256 + wg * 128;
        const bool active = C8 ? n_tiles > 0 && (wg == 0 || has1) : n_tiles > (has1 ? 0 : wg);
        float2 *row_s = reinterpret_cast<float2 *>(sm + LY::OFF_ROW);
        if (active) {
            const float sl2 = p.scale_log2;
            for (int j = pair ? 0 : wg; j < n_tiles && ok; j += step) {
                // Wait outcomes are combined across the warp: the TMEM loads and
                // stores below are warp-collective, so a warp leaves together.
                if (!__all_sync(0xFFFFFFFFu, wait(BAR(B_SF + wg), (pair ? j : j >> 1) & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int base = tile_base(j);
                const bool full = base + BN <= rr.hi && (base >= rr.lo || base + BN <= sink);
                const bool masked = !__all_sync(0xFFFFFFFFu, full);
                // The scores are read 64 columns at a time.  Over bf16 keys all 128 stay
                // in registers; over the cache, whose converting threads need registers
                // too, the first 64 are read again for the exponentials.
                constexpr int KEEP = C8 ? 1 : 2;
                uint32_t r[KEEP][2][32];
                auto load = [&](int h) {
                    tmem_ld32(tS + h * 64, r[h % KEEP][0]);
                    tmem_ld32(tS + h * 64 + 32, r[h % KEEP][1]);
                };
                auto mask = [&](int h) {
                    uint32_t(&x)[2][32] = r[h % KEEP];
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int cb = base + h * 64 + c * 32;
                            const uint32_t vm = (low_mask(rr.hi - cb) & ~low_mask(rr.lo - cb)) | low_mask(sink - cb);
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[c][e] = ((vm >> e) & 1u) ? x[c][e] : 0xFF800000u;
                        }
                    }
                };
                float m_new = m_run;
                auto maximum = [&](int h) {
                    const uint32_t(&x)[2][32] = r[h % KEEP];
                    float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // (four independent ones)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            pm[(e >> 1) & 3] = fmax3(pm[(e >> 1) & 3], __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
                    m_new = fmaxf(m_new, fmax3(pm[0], pm[1], fmaxf(pm[2], pm[3])) * sl2);
                };
                if (C8) {
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        load(h);
                        tmem_ld_wait();
                        mask(h);
                        maximum(h);
                    }
                } else {
                    load(0), load(1);
                    tmem_ld_wait();
                    mask(0), mask(1);
                    maximum(0), maximum(1);
                }
                // The rescale touches TMEM with warp-collective loads and stores, so
                // the whole warp moves when one live row's maximum grew by more than 2^8.
                if (__any_sync(0xFFFFFFFFu, j < step || (live && m_new > m_run + kRescaleLog2))) {
                    if (j >= step) {
                        const float alpha = m_new > m_run ? ex2_approx(m_run - m_new) : 1.f;
                        l_run *= alpha;
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tO + c * 32, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(tO + c * 32, o);
                        }
                        tmem_st_wait();
                    }
                    m_run = m_new;
                }
                const float m_use = m_run == -INFINITY ? 0.f : m_run;  // nothing seen yet: every p is 0
                auto weights = [&](int h) {
                    const uint32_t(&x)[2][32] = r[h % KEEP];
                    const uint64_t sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(-m_use, -m_use);
                    uint64_t ps2[4];
#pragma unroll
                    for (int a = 0; a < 4; ++a) ps2[a] = f2_pack(0.f, 0.f);
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const uint64_t x2 = f2_fma(f2_pack(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), sl2x2, negm2);
                            float p0, p1;
                            f2_unpack(x2, p0, p1);
                            p0 = ex2_approx(p0), p1 = ex2_approx(p1);
                            ps2[(e >> 1) & 3] = f2_add(ps2[(e >> 1) & 3], f2_pack(p0, p1));
                            pk[c * 16 + (e >> 1)] = pack_bf16x2(p0, p1);
                        }
                    tmem_st32(tS + h * 64, pk);
                    float a0, a1;
                    f2_unpack(f2_add(f2_add(ps2[0], ps2[1]), f2_add(ps2[2], ps2[3])), a0, a1);
                    l_run += a0 + a1;
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(B_PF + 2 * wg + h));
                };
                if (C8) {
#pragma unroll 1
                    for (int h = FIRST_HALF; h >= 0; --h) {
                        if (h != FIRST_HALF) {
                            load(h);
                            tmem_ld_wait();
                            mask(h);
                        }
                        weights(h);
                    }
                } else {
                    weights(0), weights(1);
                }
            }
            if (ok && !__all_sync(0xFFFFFFFFu, wait(BAR(B_OF + wg), 0))) ok = false;
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        // (one row tile: each warpgroup reads both accumulators)
        if (!pair && n_tiles > 1 - wg && ok && !__all_sync(0xFFFFFFFFu, wait(BAR(B_OF + 1 - wg), 0))) ok = false;
        tc_fence_after();
        // Columns [c0, c1) of 32 to store; one row tile: half each, of w0 O_0 + w1 O_1.
        int c0 = 0, c1 = D / 32;
        float w0 = 1.f, w1 = 0.f;
        if (!pair) {
            row_s[wg * 128 + row] = make_float2(ok ? m_run : NAN, l_run);
            asm volatile("bar.sync 2, 256;" ::: "memory");
            const float2 a = row_s[row], c = row_s[128 + row];
            ok = ok && a.x == a.x && c.x == c.x;
            m_run = fmaxf(a.x, c.x);
            w0 = a.x > -INFINITY ? ex2_approx(a.x - m_run) : 0.f;
            w1 = c.x > -INFINITY ? ex2_approx(c.x - m_run) : 0.f;
            l_run = a.y * w0 + c.y * w1;
            c0 = wg * (D / 64), c1 = c0 + D / 64;
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        const bool read = C8 ? active : n_tiles > 0;
        // A row that sees nothing has a sum of exactly 0.  (Its maximum does not tell: the maximum passes over a NaN.)
        const bool some = read && live && l_run != 0.f;
        const float il = some ? 1.f / l_run : 0.f;
        const int64_t orow = ((int64_t)b * p.Hq + hk * p.G + g) * p.Lq + i;
        if (ok && mine && (pair || wg == 0)) {
            const float lse = some ? (m_run + __log2f(l_run)) * 0.693147180559945f : -INFINITY;
            if (p.nsplit > 1)
                p.part_lse[(int64_t)sp * p.B * p.Hq * p.Lq + orow] = lse;
            else if (p.lse)
                p.lse[orow] = lse;
        }
        if (ok) {
            float4 *dst4 = reinterpret_cast<float4 *>(p.part_o + ((int64_t)sp * p.B * p.Hq * p.Lq + orow) * D);
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<bf16 *>(p.o.p) + b * p.o.b + (int64_t)(hk * p.G + g) * p.o.h + i * p.o.l);
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                uint32_t o[32];
                if (read) {
                    tmem_ld32((pair ? tO : tmem + lane_off + 256) + c * 32, o);
                    tmem_ld_wait();
                }
                if (!pair && read) {
                    uint32_t o1[32];
                    tmem_ld32(tmem + lane_off + 256 + 128 + c * 32, o1);
                    tmem_ld_wait();
                    // (what a warpgroup that saw nothing of the row left there does not count)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint((w0 > 0.f ? __uint_as_float(o[e]) * w0 : 0.f) + (w1 > 0.f ? __uint_as_float(o1[e]) * w1 : 0.f));
                }
                if (mine && p.nsplit > 1) {
                    if (some) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float *f = reinterpret_cast<const float *>(o + 4 * q);
                            dst4[c * 8 + q] = make_float4(f[0] * il, f[1] * il, f[2] * il, f[3] * il);
                        }
                    }
                } else if (mine) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float *f = reinterpret_cast<const float *>(o + 8 * q);
                        dst[c * 4 + q] = some ? make_uint4(pack_bf16x2(f[0] * il, f[1] * il), pack_bf16x2(f[2] * il, f[3] * il),
                                                           pack_bf16x2(f[4] * il, f[5] * il), pack_bf16x2(f[6] * il, f[7] * il))
                                              : make_uint4(0, 0, 0, 0);
                    }
                }
            }
        }
        if (!pair && wg == 1) {
            // the rows of the second tile, all behind the sequence
            const int i1 = i + p.TT;
            if (row < p.G * p.TT && i1 < p.Lq) {
                if (p.nsplit > 1) {
                    p.part_lse[(int64_t)sp * p.B * p.Hq * p.Lq + orow + p.TT] = -INFINITY;
                } else {
                    if (p.lse) p.lse[orow + p.TT] = -INFINITY;
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<bf16 *>(p.o.p) + b * p.o.b + (int64_t)(hk * p.G + g) * p.o.h + i1 * p.o.l);
#pragma unroll 1
                    for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
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

// Joins the partial results of a row: O = sum_s w_s O_s with w_s = e^(lse_s - lse).  A
// part that saw nothing has lse_s = -inf and no O_s; one with a NaN makes the row NaN.  WARPS warps per row, each with the
// loads of eight parts in flight; bound by their latency.  (One row of 100,000 keys, 390
// parts: 101 us in all when one warp read the parts one after the other, 17 now.)
template <int D, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : 32 * WARPS) k_combine(const float *__restrict__ part_o, const float *__restrict__ part_lse,
                                                 View o, float *lse, int64_t rows, int nsplit, int Hq, int Lq) {
    constexpr int N = D / 32;
    typedef typename std::conditional<N == 4, float4, float2>::type Vec;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = WARPS == 1 ? 0 : warp;
    const int64_t row = WARPS == 1 ? (int64_t)blockIdx.x * 4 + warp : blockIdx.x;
    if (row >= rows) return;
    wait_predecessor();
    float mine;  // log-sum-exp of part s0 + lane of the group
    Vec f[8];    // (loaded whatever they hold, so that all are in flight)
    auto load = [&](int s0) {
        const int n = min(8, nsplit - s0);
        mine = lane < n ? part_lse[(s0 + lane) * rows + row] : -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = *reinterpret_cast<const Vec *>(part_o + ((s0 + min(i, n - 1)) * rows + row) * D + lane * N);
    };
    if (w0 * 8 < nsplit) load(w0 * 8);
    float top = -INFINITY;
    bool seen = false;
    for (int s = lane; s < nsplit; s += 32) {
        const float x = part_lse[s * rows + row];
        top = fmaxf(top, x), seen = seen || x != -INFINITY;
    }
    for (int m = 16; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    float acc[N] = {}, sum = 0.f;
    if (__any_sync(0xFFFFFFFFu, seen)) {
        for (int s0 = w0 * 8; s0 < nsplit; s0 += WARPS * 8) {
            if (s0 != w0 * 8) load(s0);
            const float weight = mine == -INFINITY ? -1.f : __expf(mine - top);  // (-1: no O_s)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = __shfl_sync(0xFFFFFFFFu, weight, i);
                const float *x = reinterpret_cast<const float *>(&f[i]);
                sum = w < 0.f ? sum : sum + w;
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] = w < 0.f ? acc[e] : fmaf(w, x[e], acc[e]);
            }
        }
    }
    if constexpr (WARPS > 1) {
        __shared__ float s_acc[WARPS][D], s_sum[WARPS];
#pragma unroll
        for (int e = 0; e < N; ++e) s_acc[warp][lane * N + e] = acc[e];
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
            sum += s_sum[w];
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += s_acc[w][lane * N + e];
        }
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const uint32_t r = (uint32_t)row, i = r % (uint32_t)Lq, bh = r / (uint32_t)Lq, h = bh % (uint32_t)Hq;  // (at most 2^32 rows)
    const int64_t b = bh / (uint32_t)Hq;
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<bf16 *>(o.p) + b * o.b + h * o.h + i * o.l) + lane * (N / 2);
#pragma unroll
    for (int e = 0; e < N; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lse && lane == 0) lse[row] = sum != 0.f ? top + __logf(sum) : -INFINITY;
}

// Parts of the key tiles.  A CTA takes about (tiles + 4) tile times (its start
// and end cost as much as four), 148 run at once, and joining reads and writes
// the partial O; a tile time is about 1.9 us, 2.6 us over the cache's codes.  (Us with 1, 2,
// 3, 5, 8 and 14 parts: 1,560 rows of 12 heads over 18,720 keys 261, 227, 204, 199, 228,
// 261; 300 rows of 8 heads over 8,192 keys 118, 68, 52, 38, 30, 37; 1,560 rows of 40
// heads over those 241, 302, 323, 353, 409, 539.)
struct Plan {
    int TT, tiles_q, nsplit;
};

Plan plan(const WinArgs &a) {
    Plan pl;
    pl.TT = 128 / a.G;
    pl.tiles_q = (a.Lq + 2 * pl.TT - 1) / (2 * pl.TT);
    const int64_t ctas = (int64_t)a.B * a.Hk * pl.tiles_q;
    const int64_t n = window_tiles(a.w, 2 * pl.TT, a.Lq, a.Lk, BN);
    const double rows_us = (double)a.B * a.Hq * a.Lq * a.d * 8 / 5e6;
    pl.nsplit = 1;
    double best = 1e30;
    for (int s = 1; s <= 64 && s <= std::max<int64_t>(n, 1); ++s) {
        const double t = (double)((ctas * s + 147) / 148) * ((n + s - 1) / s + 4) * (a.k8 ? 2.6 : 1.9) + (s > 1 ? 4.0 + rows_us * s : 0.0);
        if (t < best) best = t, pl.nsplit = s;
    }
    return pl;
}

}  // namespace

int64_t window_mma_workspace(const WinArgs &a) {
    const Plan pl = plan(a);
    return pl.nsplit > 1 ? (int64_t)pl.nsplit * a.B * a.Hq * a.Lq * (a.d + 1) * 4 : 0;
}

cudaError_t launch_combine(const float *part_o, const float *part_lse, const WinArgs &a, int nsplit, cudaStream_t s) {
    const int64_t rows = (int64_t)a.B * a.Hq * a.Lq;
    // Several warps where there are more parts than one has loads in flight, and few rows.
    const bool several = nsplit > 8 && rows <= 148 * 8;
    const unsigned grid = (unsigned)(several ? rows : (rows + 3) / 4);
    auto kern = a.d == 128 ? (several ? k_combine<128, 8> : k_combine<128, 1>) : several ? k_combine<64, 8> : k_combine<64, 1>;
    return launch_after(kern, grid, several ? 256 : 128, 0, s, part_o, part_lse, a.o, a.lse, rows, nsplit, a.Hq, a.Lq);
}

cudaError_t launch_window_mma(const WinArgs &a, cudaStream_t s) {
    const Plan pl = plan(a);
    WinParams p{};
    p.o = a.o, p.lse = a.lse;
    p.q_lens = a.q_lens, p.k_lens = a.k_lens;
    p.B = a.B, p.Hq = a.Hq, p.Hk = a.Hk, p.G = a.G, p.TT = pl.TT, p.Lq = a.Lq, p.Lk = a.Lk;
    p.tiles_q = pl.tiles_q, p.nsplit = pl.nsplit;
    p.w = a.w;
    p.scale_log2 = a.scale * 1.44269504088896f;
    p.k8 = a.k8, p.v8 = a.v8, p.ks = a.ks, p.vs = a.vs;
    p.table = a.table, p.pages = a.pages, p.T = a.T, p.max_pages = a.max_pages;
    p.launch = next_launch_id(), p.err = a.err;
    const int64_t rows = (int64_t)a.B * a.Hq * a.Lq;
    if (pl.nsplit > 1) {
        p.part_o = static_cast<float *>(a.ws);
        p.part_lse = p.part_o + pl.nsplit * rows * a.d;
    }
    const int64_t grid = (int64_t)a.B * a.Hk * pl.tiles_q * pl.nsplit;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    WinMaps maps;
    cudaError_t e = map_rows_packed(&maps.q, a.q, a.B, a.Hk, a.G, a.Lq, a.d, pl.TT);
    if (e == cudaSuccess && !a.k8 && a.Lk > 0) e = map_rows(&maps.k, a.k, a.B, a.Hk, a.Lk, a.d, BN);
    if (e == cudaSuccess && !a.k8 && a.Lk > 0) e = map_rows(&maps.v, a.v, a.B, a.Hk, a.Lk, a.d, BN);
    if (e != cudaSuccess) return e;
    auto go = [&](auto kern, uint32_t smem) -> cudaError_t {
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess) return err;
        kern<<<(unsigned)grid, a.k8 ? Split<true>::THREADS : Split<false>::THREADS, smem, s>>>(maps, p);
        AC_NOTE_LAUNCH();
        return cudaGetLastError();
    };
    if (a.d == 128)
        e = a.k8 ? go(k_window_attn<128, true>, Layout<128, true>::SMEM) : go(k_window_attn<128, false>, Layout<128, false>::SMEM);
    else
        e = a.k8 ? go(k_window_attn<64, true>, Layout<64, true>::SMEM) : go(k_window_attn<64, false>, Layout<64, false>::SMEM);
    if (e != cudaSuccess || pl.nsplit == 1) return e;
    return launch_combine(p.part_o, p.part_lse, a, pl.nsplit, s);
}

}  // namespace ac
