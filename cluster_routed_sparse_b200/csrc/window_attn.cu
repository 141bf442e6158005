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
// Warp roles (384 threads, three warpgroups):
//   warps 0-3 / 4-7  softmax + epilogue of row tile 0 / 1; thread t owns row t
//   warp 9           TMEM allocator and the single-thread tcgen05.mma issuer
//   bf16 keys:  warp 8 TMA producer; in the last tile it zeroes the V rows behind
//               the sequence (0 x garbage would be NaN)
//   8-bit keys: warps 8, 10, 11 convert: pages land as codes in a staging
//               buffer (cp.async.bulk), are multiplied by their scale into bf16
//               (exact: 4 significant bits, a power of two) and stored in the
//               swizzled layout that the products read
// Tensor memory (512 columns): S_0 | S_1 | O_0 | O_1; P overwrites S as bf16.
// Few query tiles: the key tiles are split over several CTAs, whose partial O
// and log-sum-exp k_combine joins.
//
// Rounding: P to bf16 (the operand type of the product, 2^-9 relative, random
// over the keys), O once at the end; everything else is fp32.
// Every mbarrier wait is bounded; on timeout the CTA notes it, drains what it
// issued and frees its TMEM.
#include "stream_device.cuh"
#include "stream_host.h"

namespace ac {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int NS = 2;  // K/V stages
constexpr int NTHREADS = 384;
constexpr uint32_t kRegsSoftmax = 200, kRegsOther = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsOther <= NTHREADS * 168, "register split exceeds the launch");
constexpr float kRescaleLog2 = 8.0f;
constexpr int kConverters = 96;

template <int D, bool C8>
struct Layout {
    static constexpr int HALVES = D / 64;  // 128-byte column halves of a row
    static constexpr uint32_t TILE = HALVES * 128 * 128;
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_K = 2 * TILE;
    static constexpr uint32_t OFF_V = OFF_K + NS * TILE;
    static constexpr uint32_t OFF_ST = OFF_V + NS * TILE;  // 8-bit staging: K codes, V codes
    static constexpr uint32_t STAGING = C8 ? BN * D : 0;
    static constexpr uint32_t OFF_BAR = OFF_ST + 2 * STAGING;
    static constexpr uint32_t SMEM = OFF_BAR + 256 + 1024;  // 1024-byte alignment slack
};
static_assert(Layout<128, true>::SMEM <= 232448, "shared memory");

enum {
    B_KF = 0,     // [NS] K stage filled
    B_KE = 2,     // [NS] K stage free (MMA commit after both S products)
    B_VF = 4,     // [NS] V stage filled
    B_VE = 6,     // [NS] V stage free (MMA commit after both PV products)
    B_QF = 8,     // query tiles filled
    B_SF = 9,     // [2] S_i written (MMA commit)
    B_PF = 11,    // [2] P_i written (+ O_i rescaled) by the 128 softmax threads
    B_OF = 13,    // [2] last PV_i complete (MMA commit)
    B_DONE = 15,  // every MMA complete
    B_VZ = 16,    // V rows behind the sequence zeroed (bf16 keys)
    B_ST = 17,    // [2] staging of K / V codes filled (8-bit keys)
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

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void converters_sync() { asm volatile("bar.sync 1, 96;" ::: "memory"); }

template <int D, bool C8>
__global__ void __launch_bounds__(NTHREADS, 1) k_window_attn(const __grid_constant__ WinMaps maps,
                                                            const __grid_constant__ WinParams p) {
    using LY = Layout<D, C8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- work item: (sequence and key head, pair of row tiles, part of the keys).
    // Late tiles first: without a left bound they see the most keys.
    int idx = blockIdx.x;
    const int sp = idx % p.nsplit;
    idx /= p.nsplit;
    const int qt = p.tiles_q - 1 - idx % p.tiles_q;
    const int bh = idx / p.tiles_q;
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
    uint32_t *abort_word = &p.err->timeout;
    // Bounded wait; the first to expire notes the launch, which ends the others' waits early.
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        const long long c0 = clock64();
        for (uint32_t it = 0;; ++it) {
            if (mbar_try_wait(bar, parity)) return true;
            if ((it & 255u) == 255u) {
                if (*reinterpret_cast<const volatile uint32_t *>(abort_word) == p.launch) return false;
                if (globaltimer_ns() - t0 > kWaitLimitNs || clock64() - c0 > kWaitLimitCycles || it > kWaitLimitPolls) {
                    *reinterpret_cast<volatile uint32_t *>(abort_word) = p.launch;
                    return false;
                }
            }
        }
    };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + LY::OFF_BAR + 8 * NBAR);

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(BAR(B_KF + i), C8 ? kConverters : 1);
            mbar_init(BAR(B_KE + i), 1);
            mbar_init(BAR(B_VF + i), C8 ? kConverters : 1);
            mbar_init(BAR(B_VE + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(BAR(B_SF + i), 1);
            mbar_init(BAR(B_PF + i), BM);
            mbar_init(BAR(B_OF + i), 1);
            mbar_init(BAR(B_ST + i), 1);
        }
        mbar_init(BAR(B_QF), 1);
        mbar_init(BAR(B_DONE), 1);
        mbar_init(BAR(B_VZ), 1);
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    if (warp >= 8) {
        reg_dealloc<kRegsOther>();
        if (warp == 9) {
            // ------------------------------------------------ MMA issuer
            if (lane == 0 && n_tiles > 0) {
                constexpr uint32_t IQK = idesc_bf16_f32(BM, BN, false);
                constexpr uint32_t IPV = idesc_bf16_f32(BM, D, true);
                const uint64_t dq0 = sdesc_sw128(sbase + LY::OFF_Q, 16, 1024);
                const uint64_t dk0 = sdesc_sw128(sbase + LY::OFF_K, 16, 1024);
                const uint64_t dv0 = sdesc_sw128(sbase + LY::OFF_V, BN * 128, 1024);
                auto issue_s = [&](int i, int j) {
                    const uint64_t dq = dq0 + (uint64_t)((i * LY::TILE) >> 4);
                    const uint64_t dk = dk0 + (uint64_t)(((j % NS) * LY::TILE) >> 4);
                    if constexpr (D == 128) {
                        constexpr uint32_t H = (BM * 128) >> 4;  // second column half
                        mma8_ss<2, 4, 6, H, H + 2, H + 4, H + 6, 2, 4, 6, H, H + 2, H + 4, H + 6>(tmem + i * BN, dq, dk, IQK, 0u);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc_mma_bf16(tmem + i * BN, dq + (uint64_t)(kk * 2), dk + (uint64_t)(kk * 2), IQK, kk > 0 ? 1u : 0u);
                    }
                    tc_commit(BAR(B_SF + i));
                };
                auto issue_pv = [&](int i, int j) {
                    const uint64_t dv = dv0 + (uint64_t)(((j % NS) * LY::TILE) >> 4);
                    mma8_ts<2048 / 16>(tmem + 256 + i * 128, tmem + i * BN, dv, IPV, j > 0 ? 1u : 0u);
                };
                ok = wait(BAR(B_QF), 0) && wait(BAR(B_KF), 0);
                tc_fence_after();
                if (ok) {
                    issue_s(0, 0);
                    if (has1) issue_s(1, 0);
                    tc_commit(BAR(B_KE));
                }
                for (int j = 0; j < n_tiles && ok; ++j) {
                    const bool more = j + 1 < n_tiles;
                    if (!wait(BAR(B_PF), j & 1) || !wait(BAR(B_VF + j % NS), (j / NS) & 1) ||
                        (tail && !more && !wait(BAR(B_VZ), 0))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    issue_pv(0, j);
                    if (!more) tc_commit(BAR(B_OF));
                    if (more) {
                        if (!wait(BAR(B_KF + (j + 1) % NS), ((j + 1) / NS) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        issue_s(0, j + 1);
                    }
                    if (has1) {
                        if (!wait(BAR(B_PF + 1), j & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        issue_pv(1, j);
                        if (!more) tc_commit(BAR(B_OF + 1));
                        if (more) issue_s(1, j + 1);
                    }
                    if (more) tc_commit(BAR(B_KE + (j + 1) % NS));
                    tc_commit(BAR(B_VE + j % NS));
                }
                tc_commit(BAR(B_DONE));
                wait(BAR(B_DONE), 0);
            }
            __syncwarp();
        } else if (warp == 8 && lane == 0 && n_tiles > 0) {
            // ------------------------------------------------ query tiles
            const uint32_t bytes = LY::HALVES * p.G * p.TT * 128;
            mbar_arrive_expect_tx(BAR(B_QF), (has1 ? 2 : 1) * bytes);
            for (int t = 0; t < (has1 ? 2 : 1); ++t)
                for (int hf = 0; hf < LY::HALVES; ++hf)
                    tma_load_5d(sbase + LY::OFF_Q + t * LY::TILE + hf * BM * 128, &maps.q, hf * 64, 0, i0 + t * p.TT, hk, b,
                                BAR(B_QF));
            if (!C8) {
                // -------------------------------------------- K/V producer
                int kd = 0, vd = 0;
                for (int j = 0; j < n_tiles; ++j) {
                    const int s = j % NS, base = tile_base(j);
                    if (j >= NS && !(ok = wait(BAR(B_KE + s), ((j / NS) - 1) & 1))) break;
                    mbar_arrive_expect_tx(BAR(B_KF + s), LY::TILE);
                    for (int hf = 0; hf < LY::HALVES; ++hf)
                        tma_load_4d(sbase + LY::OFF_K + s * LY::TILE + hf * BN * 128, &maps.k, hf * 64, base, hk, b, BAR(B_KF + s));
                    ++kd;
                    if (j >= NS && !(ok = wait(BAR(B_VE + s), ((j / NS) - 1) & 1))) break;
                    mbar_arrive_expect_tx(BAR(B_VF + s), LY::TILE);
                    for (int hf = 0; hf < LY::HALVES; ++hf)
                        tma_load_4d(sbase + LY::OFF_V + s * LY::TILE + hf * BN * 128, &maps.v, hf * 64, base, hk, b, BAR(B_VF + s));
                    ++vd;
                }
                // Loads still in flight must land before the CTA exits.
                for (int j = max(kd - NS, 0); j < kd; ++j) wait(BAR(B_KF + j % NS), (j / NS) & 1);
                for (int j = max(vd - NS, 0); j < vd; ++j) wait(BAR(B_VF + j % NS), (j / NS) & 1);
                wait(BAR(B_QF), 0);
            }
        }
        if (!C8 && warp == 8 && tail) {
            // V rows behind the sequence, by the producer, which has followed every phase
            __syncwarp();
            const int j = n_tiles - 1, s = j % NS, r0 = kl - tile_base(j);
            if (__shfl_sync(0xFFFFFFFFu, (int)ok, 0)) {
                wait(BAR(B_VF + s), (j / NS) & 1);
                for (int hf = 0; hf < LY::HALVES; ++hf)
                    for (int i = r0 * 8 + lane; i < BN * 8; i += 32)
                        *reinterpret_cast<uint4 *>(sm + LY::OFF_V + s * LY::TILE + hf * BN * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(B_VZ));
            }
        }
        if (C8 && warp != 9 && n_tiles > 0) {
            // ------------------------------------------------ 8-bit pages to bf16 tiles
            __syncwarp();
            const int ct = (warp == 8 ? 0 : warp - 9) * 32 + lane;  // 0..95
            const int ppt = BN / p.T;                               // pages of a tile
            const int *table = p.table + (int64_t)b * p.max_pages;
            // Page of the keys from `key` on: -1 where no row of this CTA sees any of
            // them, -2 when it is visible but its index is out of range.
            auto page_of = [&](int key) -> int {
                if (!((key < hi_c && key + p.T > lo_c) || key < sink_c)) return -1;
                const int page = table[key / p.T];
                return page < 0 || page >= p.pages ? -2 : page;
            };
            auto fetch = [&](int which, int j) {  // thread 0: codes of tile j into the staging
                const int base = tile_base(j);
                uint32_t bytes = 0;
                for (int i = 0; i < ppt; ++i) {
                    const int page = page_of(base + i * p.T);
                    if (page >= 0) bytes += p.T * D;
                    if (page == -2) atomicOr(&p.err->bits, DEV_ERR_BOUNDS);
                }
                mbar_arrive_expect_tx(BAR(B_ST + which), bytes);
                for (int i = 0; i < ppt; ++i) {
                    const int page = page_of(base + i * p.T);
                    if (page >= 0)
                        bulk_load(sbase + LY::OFF_ST + which * LY::STAGING + i * p.T * D,
                                  (which ? p.v8 : p.k8) + ((int64_t)page * p.Hk + hk) * p.T * D, p.T * D, BAR(B_ST + which));
                }
            };
            if (ct == 0) {
                fetch(0, 0);
                fetch(1, 0);
            }
            int fetched[2] = {1, 1};
            for (int j = 0; j < n_tiles && ok; ++j) {
                const int s = j % NS, base = tile_base(j);
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    const bool got = wait(BAR(B_ST + which), j & 1) &&
                                     (j < NS || wait(BAR((which ? B_VE : B_KE) + s), ((j / NS) - 1) & 1));
                    // the 96 threads leave together
                    int all = got;
                    asm volatile("{\n\t.reg .pred q, r;\n\tsetp.ne.b32 q, %1, 0;\n\tbarrier.cta.red.and.pred r, 1, 96, q;\n\t"
                                 "selp.b32 %0, 1, 0, r;\n\t}" : "=r"(all) : "r"((int)got) : "memory");
                    if (!all) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = sm + (which ? LY::OFF_V : LY::OFF_K) + s * LY::TILE;
                    const uint8_t *src = sm + LY::OFF_ST + which * LY::STAGING;
                    constexpr int CPR = D / 16;  // 16-code chunks of a row
                    for (int c = ct; c < BN * CPR; c += kConverters) {
                        const int r = c / CPR, e = c % CPR;
                        const int page = base + r < kl ? page_of((base + r) / p.T * p.T) : -1;
                        uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
                        if (page >= 0) {
                            const float sc = (which ? p.vs : p.ks)[(int64_t)page * p.Hk + hk];
                            const uint4 w = *reinterpret_cast<const uint4 *>(src + c * 16);
                            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                            uint32_t q[8];
                            const uint64_t sc2 = f2_pack(sc, sc);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float2 f = e4m3x2_to_float2((u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
                                float x, y;
                                f2_unpack(f2_mul(f2_pack(f.x, f.y), sc2), x, y);
                                q[i] = pack_bf16x2(x, y);
                            }
                            w0 = make_uint4(q[0], q[1], q[2], q[3]), w1 = make_uint4(q[4], q[5], q[6], q[7]);
                        }
                        // 128-byte rows of a column half, 16-byte pieces swizzled by the row
                        uint8_t *row = dst + (e / 4) * BN * 128 + r * 128;
                        const int a = (e % 4) * 2;
                        *reinterpret_cast<uint4 *>(row + ((a ^ (r & 7)) << 4)) = w0;
                        *reinterpret_cast<uint4 *>(row + (((a + 1) ^ (r & 7)) << 4)) = w1;
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(BAR((which ? B_VF : B_KF) + s));
                    converters_sync();  // the staging has been read
                    if (ct == 0 && j + 1 < n_tiles) {
                        fetch(which, j + 1);
                        ++fetched[which];
                    }
                }
            }
            if (ct == 0) {
                // Loads still in flight must land before the CTA exits.
                for (int which = 0; which < 2; ++which) wait(BAR(B_ST + which), (fetched[which] - 1) & 1);
                wait(BAR(B_QF), 0);
            }
        }
        __syncwarp();
    } else {
        reg_alloc<kRegsSoftmax>();
        // ------------------------------------------------ softmax + epilogue
        const int wg = warp >> 2;
        const int row = tid & 127;
        const int g = row % p.G, i = i0 + wg * p.TT + row / p.G;
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
        const bool active = n_tiles > 0 && (wg == 0 || has1);
        if (active) {
            const float sl2 = p.scale_log2;
            for (int j = 0; j < n_tiles; ++j) {
                // Wait outcomes are combined across the warp: the TMEM loads and
                // stores below are warp-collective, so a warp leaves together.
                if (!__all_sync(0xFFFFFFFFu, wait(BAR(B_SF + wg), j & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t r[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, r[c]);
                const int base = tile_base(j);
                const bool full = base + BN <= rr.hi && (base >= rr.lo || base + BN <= sink);
                const bool masked = !__all_sync(0xFFFFFFFFu, full);
                tmem_ld_wait();
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int cb = base + 32 * c;
                        const uint32_t vm = (low_mask(rr.hi - cb) & ~low_mask(rr.lo - cb)) | low_mask(sink - cb);
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[c][e] = ((vm >> e) & 1u) ? r[c][e] : 0xFF800000u;
                    }
                }
                float pm[8];
#pragma unroll
                for (int a = 0; a < 8; ++a) pm[a] = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        pm[(e >> 1) & 7] = fmax3(pm[(e >> 1) & 7], __uint_as_float(r[c][e]), __uint_as_float(r[c][e + 1]));
                const float tmax = fmax3(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
                const float m_new = fmaxf(m_run, tmax * sl2);
                // The rescale touches TMEM with warp-collective loads and stores, so
                // the whole warp moves when one live row's maximum grew by more than 2^8.
                if (__any_sync(0xFFFFFFFFu, j == 0 || (live && m_new > m_run + kRescaleLog2))) {
                    if (j > 0) {
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
                const uint64_t sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(-m_use, -m_use);
                uint64_t ps2[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) ps2[a] = f2_pack(0.f, 0.f);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        const int c = half * 2 + cc;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const uint64_t x2 = f2_fma(f2_pack(__uint_as_float(r[c][e]), __uint_as_float(r[c][e + 1])), sl2x2, negm2);
                            float x0, x1;
                            f2_unpack(x2, x0, x1);
                            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                            ps2[(e >> 1) & 3] = f2_add(ps2[(e >> 1) & 3], f2_pack(p0, p1));
                            pk[cc * 16 + (e >> 1)] = pack_bf16x2(p0, p1);
                        }
                    }
                    tmem_st32(tS + half * 32, pk);
                }
                float ps[8];
#pragma unroll
                for (int a = 0; a < 4; ++a) f2_unpack(ps2[a], ps[2 * a], ps[2 * a + 1]);
                tmem_st_wait();
                l_run += ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
                tc_fence_before();
                mbar_arrive(BAR(B_PF + wg));
            }
            if (ok && !__all_sync(0xFFFFFFFFu, wait(BAR(B_OF + wg), 0))) ok = false;
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
        }
        const bool some = active && live && l_run > 0.f;
        const float il = some ? 1.f / l_run : 0.f;
        const int64_t orow = ((int64_t)b * p.Hq + hk * p.G + g) * p.Lq + i;
        if (ok && mine) {
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
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (active) {
                    tmem_ld32(tO + c * 32, o);
                    tmem_ld_wait();
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
    }
#undef BAR
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partial results of a row: O = sum_s w_s O_s with w_s = 2^(lse_s - lse)
// (natural logarithms).  A part that saw nothing has lse_s = -inf and no O_s.
// One warp per row; bound by reading the partials once.
template <int D>
__global__ void __launch_bounds__(128) k_combine(const float *__restrict__ part_o, const float *__restrict__ part_lse,
                                                 View o, float *lse, int64_t rows, int nsplit, int Hq, int Lq) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    float top = -INFINITY;
    for (int s = lane; s < nsplit; s += 32) top = fmaxf(top, part_lse[s * rows + row]);
    for (int m = 16; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    float acc[N] = {}, sum = 0.f;
    if (top > -INFINITY) {
        for (int s = 0; s < nsplit; ++s) {
            const float ls = part_lse[s * rows + row];
            if (ls == -INFINITY) continue;
            const float w = __expf(ls - top);
            sum += w;
            const float *src = part_o + (s * rows + row) * D + lane * N;
            if constexpr (N == 4) {
                const float4 f = *reinterpret_cast<const float4 *>(src);
                acc[0] += w * f.x, acc[1] += w * f.y, acc[2] += w * f.z, acc[3] += w * f.w;
            } else {
                const float2 f = *reinterpret_cast<const float2 *>(src);
                acc[0] += w * f.x, acc[1] += w * f.y;
            }
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int i = (int)(row % Lq), h = (int)(row / Lq % Hq);
    const int64_t b = row / Lq / Hq;
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<bf16 *>(o.p) + b * o.b + h * o.h + i * o.l) + lane * (N / 2);
#pragma unroll
    for (int e = 0; e < N; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lse && lane == 0) lse[row] = sum > 0.f ? top + __logf(sum) : -INFINITY;
}

// Parts of the key tiles.  A CTA takes about (tiles + 4) tile times (its start
// and end cost as much as four), 148 run at once, and joining reads and writes
// the partial O: one tile time is about 1.1 us.
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
        const double t = (double)((ctas * s + 147) / 148) * ((n + s - 1) / s + 4) * 1.1 + (s > 1 ? 2.5 + rows_us * s : 0.0);
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
    const unsigned grid = (unsigned)((rows + 3) / 4);
    if (a.d == 128)
        k_combine<128><<<grid, 128, 0, s>>>(part_o, part_lse, a.o, a.lse, rows, nsplit, a.Hq, a.Lq);
    else
        k_combine<64><<<grid, 128, 0, s>>>(part_o, part_lse, a.o, a.lse, rows, nsplit, a.Hq, a.Lq);
    AC_NOTE_LAUNCH();
    return cudaGetLastError();
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
        kern<<<(unsigned)grid, NTHREADS, smem, s>>>(maps, p);
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
