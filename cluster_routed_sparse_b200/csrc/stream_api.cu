// stream_api.cu -- C ABI of the streaming operators: checks of arguments,
// argument blocks and the error words.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <thread>

#include "stream_device.cuh"

using namespace ac;

namespace {

__device__ OpErr g_op_err;
std::atomic<uint32_t> g_launch_id{0};

ac_status refuse(const char *what, ac_status st = AC_ERR_INVALID_ARG) {
    set_static_error(what);
    return st;
}

ac_status cuda_refuse(const char *fn, cudaError_t e) {
    char buf[256];
    snprintf(buf, sizeof(buf), "%s: %s", fn, cudaGetErrorString(e));
    set_static_error(buf);
    return AC_ERR_CUDA;
}

// The kernels are built for sm_100a only.
ac_status check_device(const char *fn) {
    int dev = 0, major = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e != cudaSuccess) return cuda_refuse(fn, e);
    if (major != 10) return refuse("the streaming operators need an sm_100 device", AC_ERR_UNSUPPORTED);
    return AC_OK;
}

constexpr int kMaxLen = 1 << 30;

// Few query rows for each key head are bound by reading the keys: they go to the kernel
// whose products take 8 rows.  It reads the keys once for every 8 rows, from the L2
// cache after the first time, at a cost that grows with the rows; the tile kernel's is that
// of 128, and over the cache that of converting every code to 16 bits.  Us of the two,
// d = 128, few rows / tiles:
//                                  8 rows       16 rows      24 rows      32 rows      64 rows
//   bf16   32,768 keys, 64 heads   166 / 165    281 / 166                 541 / 166
//           2,048 keys, 160 heads   38 / 48      57 / 49                   98 / 51
//           2,048 keys, 8 heads    9.0 / 10.0   9.2 / 10.0                11.6 / 10.2  17.0 / 11.1
//             320 keys, 2 heads    5.7 / 8.3    5.8 / 8.4                 5.9 / 8.4    5.9 / 8.3
//   8 bits 32,768 keys, 64 heads   110 / 280    200 / 277    281 / 277    371 / 276    698 / 278
//           2,048 keys, 160 heads   26 / 70      44 / 72      56 / 72      83 / 75     139 / 78
//             320 keys, 2 heads    9.1 / 10.9   9.3 / 12.1                9.5 / 17.9   9.3 / 11.6
bool few_rows(const WinArgs &a) {
    const int64_t rows = (int64_t)a.G * a.Lq;
    return rows <= (a.k8 ? 24 : 8) || (rows <= 64 && window_tiles(a.w, a.Lq, a.Lq, a.Lk, 16) <= 32);
}
// Many rows over the cache: its visible part is written out as bf16 once, instead of
// being converted by every CTA for its 256 rows.  Us of the two, d = 128, codes / bf16:
//                            512 rows     768         1,024       1,560       3,120
//    16,384 keys, 12 heads    75 / 87    100 / 107   128 / 131   233 / 219   443 / 367
//     8,192 keys, 32 heads   102 / 118   147 / 156   173 / 167   321 / 287   481 / 411
//     2,048 keys, 8 heads     22 / 25     25 / 29     28 / 30     43 / 39     50 / 45
//       512 keys, 2 heads     12 / 14                 12 / 14     12 / 15     14 / 17   (d = 64)
// A call that would need more than 1 GiB for it (262,144 tokens of 8 heads) reads the codes.
constexpr int64_t kExpandRows = 1024, kExpandKeys = 16384, kExpandMost = int64_t(1) << 30;
int64_t expand_bytes(const WinArgs &a) { return (int64_t)a.B * a.Hk * a.Lk * a.d * 4; }
bool expands(const WinArgs &a) {
    return a.k8 && !few_rows(a) && (int64_t)a.G * a.Lq > kExpandRows && (int64_t)a.B * a.Hk * a.Lk >= kExpandKeys &&
           expand_bytes(a) <= kExpandMost;
}
// The call over the rows written out, which stand in front of its own workspace.
WinArgs expanded(const WinArgs &a) {
    WinArgs x = a;
    const int64_t n = (int64_t)a.Hk * a.Lk * a.d, half = expand_bytes(a) / 2;
    x.k = View{a.ws, n, (int64_t)a.Lk * a.d, a.d};
    x.v = View{static_cast<char *>(a.ws) + half, n, (int64_t)a.Lk * a.d, a.d};
    x.ws = static_cast<char *>(a.ws) + 2 * half;
    x.k8 = x.v8 = nullptr;
    return x;
}
int64_t window_workspace(const WinArgs &a) {
    if (expands(a)) return expand_bytes(a) + window_mma_workspace(expanded(a));
    return few_rows(a) ? window_few_workspace(a) : window_mma_workspace(a);
}
cudaError_t launch_window(const WinArgs &a, cudaStream_t s) {
    if (expands(a)) {
        const WinArgs x = expanded(a);
        const cudaError_t e = launch_cache8_expand(a, static_cast<bf16 *>(x.k.p), static_cast<bf16 *>(x.v.p), s);
        return e == cudaSuccess ? launch_window_mma(x, s) : e;
    }
    return few_rows(a) ? launch_window_few(a, s) : launch_window_mma(a, s);
}

// f / (2 pi) modulo 1 in units of 2^-64, to the nearest; 0 from |f| = 2^126 on.  f is a 53-bit
// integer times a power of two, and 1 / (2 pi) is held to 192 bits, so whole turns leave
// exactly and the fraction keeps all its bits.
uint64_t turns_of(double f) {
    constexpr uint64_t kInv[3] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull};  // of 2^-64, 2^-128, 2^-192
    int x;
    const double m = std::frexp(std::fabs(f), &x);
    if (m == 0.0 || x < -62 || x > 126) return 0;
    const uint64_t i = (uint64_t)std::ldexp(m, 53);
    x -= 53;  // |f| = i 2^x
    // i / (2 pi) modulo 2^64 in words: the whole turns, and three of the fraction
    uint64_t w[4];
    unsigned __int128 carry = 0;
    for (int k = 2; k >= 0; --k) {
        const unsigned __int128 p = (unsigned __int128)i * kInv[k] + carry;
        w[k + 1] = (uint64_t)p;
        carry = p >> 64;
    }
    w[0] = (uint64_t)carry;
    // the 64 bits behind the point, once that has moved by x, and the bit after them
    const int from = 64 + x;  // bit position in w, from its top
    auto bit_word = [&](int at) -> uint64_t {  // 64 bits that begin at position `at`, zeros in front of w and behind it
        uint64_t r = 0;
        for (int k = 0; k < 4; ++k) {
            const int d = at - 64 * k;
            if (d >= 0 && d < 64) r |= w[k] << d;
            else if (d < 0 && d > -64) r |= w[k] >> -d;
        }
        return r;
    };
    const uint64_t units = bit_word(from) + (bit_word(from + 64) >> 63);
    return f < 0 ? 0 - units : units;
}

// The same of n frequencies.  The last ones' stay at hand: 0.5 us of a call of 8 us.
bool turns_of(const double *freq, int n, uint64_t *turns) {
    thread_local double last[128];
    thread_local uint64_t last_turns[128];
    thread_local int last_n = -1;
    if (n != last_n || memcmp(freq, last, n * sizeof(double))) {
        last_n = -1;
        for (int k = 0; k < n; ++k) {
            if (!std::isfinite(freq[k])) return false;
            last_turns[k] = turns_of(freq[k]);
            last[k] = freq[k];
        }
        last_n = n;
    }
    memcpy(turns, last_turns, n * sizeof(uint64_t));
    return true;
}

View view_of(const ac_view *v) { return View{v->data, v->stride_b, v->stride_h, v->stride_l}; }

// 16-byte rows: what the vector and bulk tensor loads need.  A stride of a
// dimension of one entry is never used.
bool rows16(const ac_view *v, int B, int H, int L) {
    if (!v || !v->data || (reinterpret_cast<uintptr_t>(v->data) & 15u)) return false;
    const int64_t st[3] = {v->stride_b, v->stride_h, v->stride_l};
    const int n[3] = {B, H, L};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (st[i] <= 0 || st[i] % 8 || st[i] >= (int64_t(1) << 38))) return false;
    return true;
}

// Workspaces hold float4 parts and rows that bulk copies read.
ac_status check_workspace(const char *what, const void *ws, int64_t bytes, int64_t need) {
    if (need == 0) return AC_OK;
    if (!ws || bytes < need) return refuse(what, AC_ERR_WORKSPACE);
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return refuse("the workspace must be 256-byte aligned");
    return AC_OK;
}

ac_status window_rule(const ac_window *w, int d, WinRule *out, float *scale) {
    if (!w || w->left < -1 || w->right < -1 || w->sinks < 0 || w->block < 1 || !std::isfinite(w->scale) ||
        w->scale < 0.f)
        return refuse("window: left and right must be >= -1, sinks >= 0, block >= 1 and the scale finite and >= 0");
    *out = WinRule{w->left, w->right, w->sinks, w->block};
    *scale = w->scale != 0.f ? w->scale : 1.f / sqrtf((float)d);
    return AC_OK;
}

ac_status check_sizes(int B, int Hq, int Hk, int Lq, int Lk, int d) {
    if (d != 64 && d != 128) return refuse("window attention: d must be 64 or 128", AC_ERR_UNSUPPORTED);
    if (B < 0 || Hq < 1 || Hk < 1 || Lq < 0 || Lk < 0 || Lq > kMaxLen || Lk > kMaxLen)
        return refuse("window attention: bad sizes");
    if (Hq % Hk || Hq / Hk > 128)
        return refuse("window attention: query heads must be a multiple of the key heads, at most 128 for each");
    const int64_t rows = (int64_t)B * Hq * (int64_t)std::max(Lq, 1), keys = (int64_t)B * Hk * (int64_t)std::max(Lk, 1);
    if (B > 65535 || Hq > 65535 || rows > (int64_t(1) << 32) || keys > (int64_t(1) << 32))
        return refuse("window attention: at most 2^32 rows of queries and of keys");
    return AC_OK;
}

}  // namespace

cudaError_t ac::op_err_address(OpErr **out) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(out), g_op_err);
}

uint32_t ac::next_launch_id() {
    uint32_t id;
    do id = g_launch_id.fetch_add(1, std::memory_order_relaxed) + 1;
    while (id == 0);
    return id;
}

namespace {
__global__ void k_ops_wait_check(OpErr *err, uint32_t launch, uint64_t limit_ns) {
    __shared__ alignas(8) uint64_t bar;
    mbar_init(smem_u32(&bar), 1);
    fence_mbar_init();
    wait_or_note(smem_u32(&bar), 0, &err->timeout, launch, limit_ns);
}
}  // namespace

extern "C" ac_status ac_ops_check_wait_timeout(int32_t limit_us, void *stream) {
    if (limit_us < 1 || limit_us > 2000000) return refuse("ac_ops_check_wait_timeout: limit_us outside 1 .. 2,000,000");
    OpErr *p = nullptr;
    cudaError_t e = op_err_address(&p);
    if (e == cudaSuccess) {
        k_ops_wait_check<<<1, 1, 0, (cudaStream_t)stream>>>(p, next_launch_id(), (uint64_t)limit_us * 1000ull);
        AC_NOTE_LAUNCH();
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? AC_OK : cuda_refuse("ac_ops_check_wait_timeout", e);
}

// What was noted is taken and cleared in one step, so that no note of another stream's kernels
// gets lost in between.  An expired wait comes first; the bits then stay for the next call.
namespace {
constexpr int kSlots = 64;  // calls at once
__device__ OpErr g_taken[kSlots];
std::atomic<uint64_t> g_slots{0};  // those in use

__global__ void k_ops_take(OpErr *err, int slot) {
    OpErr t{atomicExch(&err->timeout, 0u), 0u};
    if (!t.timeout) t.bits = atomicExch(&err->bits, 0u);
    g_taken[slot] = t;
}

struct Slot {
    int i;
    Slot() {
        uint64_t used = g_slots.load(std::memory_order_relaxed);
        for (;;) {
            if (used == ~uint64_t(0)) {
                std::this_thread::yield();
                used = g_slots.load(std::memory_order_relaxed);
                continue;
            }
            i = __builtin_ctzll(~used);
            if (g_slots.compare_exchange_weak(used, used | uint64_t(1) << i, std::memory_order_acquire)) return;
        }
    }
    ~Slot() { g_slots.fetch_and(~(uint64_t(1) << i), std::memory_order_release); }
};
}  // namespace

extern "C" ac_status ac_ops_status(void *stream) {
    OpErr *p = nullptr, h{};
    void *taken = nullptr;
    cudaStream_t s = (cudaStream_t)stream;
    const Slot slot;
    cudaError_t e = op_err_address(&p);
    if (e == cudaSuccess) e = cudaGetSymbolAddress(&taken, g_taken);
    if (e == cudaSuccess) {
        k_ops_take<<<1, 1, 0, s>>>(p, slot.i);
        AC_NOTE_LAUNCH();
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = cudaMemcpyAsync(&h, static_cast<OpErr *>(taken) + slot.i, sizeof(h), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_refuse("ac_ops_status", e);
    if (h.timeout) return refuse("a bounded in-kernel wait expired", AC_ERR_TIMEOUT);
    if (h.bits) return refuse("a length or a page index on the device is out of range", AC_ERR_BOUNDS);
    return AC_OK;
}

extern "C" ac_status ac_rope_axes(int32_t dtype, const ac_view *x, const ac_view *y, int32_t H, const ac_view *x2,
                                  const ac_view *y2, int32_t H2, int32_t B, int32_t L, int32_t d,
                                  const int32_t *positions, int64_t pos_stride_b, const double *freq,
                                  const int32_t *pairs, int32_t n_axes, int32_t interleaved, int32_t inverse,
                                  void *stream) {
    if (dtype < AC_DTYPE_BF16 || dtype > AC_DTYPE_F32) return refuse("ac_rope_axes: unknown dtype", AC_ERR_UNSUPPORTED);
    if (d < 2 || d > 256 || d % 2) return refuse("ac_rope_axes: d must be even and at most 256", AC_ERR_UNSUPPORTED);
    if (!freq || !pairs || n_axes < 1 || n_axes > 8 || B < 0 || L < 0 || H < 0 || H2 < 0 || H > 65535 || H2 > 65535)
        return refuse("ac_rope_axes: invalid argument");
    RopeArgs a;
    a.P = 0;
    for (int i = 0; i < n_axes; ++i) {
        if (pairs[i] < 0 || pairs[i] > d / 2 - a.P) return refuse("ac_rope_axes: the axes' pairs must fit in d / 2");
        for (int k = 0; k < pairs[i]; ++k) a.axis[a.P++] = (uint8_t)i;
    }
    if (!turns_of(freq, a.P, a.turns)) return refuse("ac_rope_axes: frequencies must be finite");
    if (B == 0 || L == 0 || H + H2 == 0) return AC_OK;
    if (!positions || (H && (!x || !y || !x->data || !y->data)) || (H2 && (!x2 || !y2 || !x2->data || !y2->data)))
        return refuse("ac_rope_axes: NULL tensor");
    a.H[0] = H, a.H[1] = H2;
    for (int t = 0; t < 2; ++t) {
        const ac_view *in = t ? x2 : x, *out = t ? y2 : y;
        a.x[t] = a.H[t] ? view_of(in) : View{};
        a.y[t] = a.H[t] ? view_of(out) : View{};
    }
    for (int t = 0; t < 2; ++t)
        if ((B > 1 && a.H[t] && !a.y[t].b) || (a.H[t] > 1 && !a.y[t].h) || (L > 1 && a.H[t] && !a.y[t].l))
            return refuse("ac_rope_axes: an output cannot be a broadcast tensor");
    a.B = B, a.L = L, a.d = d;
    a.pos = positions, a.pos_b = pos_stride_b, a.n_axes = n_axes;
    a.interleaved = interleaved != 0, a.inverse = inverse != 0;
    const ac_status st = check_device("ac_rope_axes");
    if (st != AC_OK) return st;
    const cudaError_t e = launch_rope(dtype, a, (cudaStream_t)stream);
    return e == cudaSuccess ? AC_OK : cuda_refuse("ac_rope_axes", e);
}

// ---------------------------------------------------------------- window attention
extern "C" ac_status ac_window_attn_workspace(int32_t B, int32_t Hq, int32_t Hk, int32_t Lq, int32_t Lk, int32_t d,
                                              const ac_window *w, int64_t *bytes) {
    if (!bytes) return refuse("ac_window_attn_workspace: NULL argument");
    ac_status st = check_sizes(B, Hq, Hk, Lq, Lk, d);
    WinRule r;
    float scale;
    if (st == AC_OK) st = window_rule(w, d, &r, &scale);
    if (st != AC_OK) return st;
    WinArgs a{};
    a.B = B, a.Hq = Hq, a.Hk = Hk, a.G = Hq / Hk, a.Lq = Lq, a.Lk = Lk, a.d = d, a.w = r;
    *bytes = B && Lq ? window_workspace(a) : 0;
    return AC_OK;
}

extern "C" ac_status ac_window_attn(const ac_view *q, const ac_view *k, const ac_view *v, const ac_view *o, float *lse,
                                    int32_t B, int32_t Hq, int32_t Hk, int32_t Lq, int32_t Lk, int32_t d,
                                    const int32_t *q_lens, const int32_t *k_lens, const ac_window *w, void *workspace,
                                    int64_t workspace_bytes, void *stream) {
    ac_status st = check_sizes(B, Hq, Hk, Lq, Lk, d);
    WinArgs a{};
    if (st == AC_OK) st = window_rule(w, d, &a.w, &a.scale);
    int64_t need = 0;
    if (st == AC_OK) st = ac_window_attn_workspace(B, Hq, Hk, Lq, Lk, d, w, &need);
    if (st != AC_OK) return st;
    if (B == 0 || Lq == 0) return AC_OK;
    if (!rows16(q, B, Hq, Lq) || !rows16(o, B, Hq, Lq) || (Lk > 0 && (!rows16(k, B, Hk, Lk) || !rows16(v, B, Hk, Lk))))
        return refuse("ac_window_attn: tensors must be 16-byte aligned with positive strides in multiples of 8");
    if ((st = check_workspace("ac_window_attn: workspace too small", workspace, workspace_bytes, need)) != AC_OK) return st;
    if ((st = check_device("ac_window_attn")) != AC_OK) return st;
    a.q = view_of(q), a.o = view_of(o);
    if (Lk > 0) a.k = view_of(k), a.v = view_of(v);
    a.lse = lse, a.q_lens = q_lens, a.k_lens = k_lens;
    a.B = B, a.Hq = Hq, a.Hk = Hk, a.G = Hq / Hk, a.Lq = Lq, a.Lk = Lk, a.d = d;
    a.ws = workspace;
    cudaError_t e = op_err_address(&a.err);
    if (e == cudaSuccess) e = launch_window(a, (cudaStream_t)stream);
    return e == cudaSuccess ? AC_OK : cuda_refuse("ac_window_attn", e);
}

extern "C" ac_status ac_window_attn_backward_workspace(int32_t B, int32_t Hq, int32_t Hk, int32_t Lq, int32_t Lk,
                                                       int32_t d, const ac_window *w, int64_t *bytes) {
    if (!bytes) return refuse("ac_window_attn_backward_workspace: NULL argument");
    ac_status st = check_sizes(B, Hq, Hk, Lq, Lk, d);
    WinArgs a{};
    if (st == AC_OK) st = window_rule(w, d, &a.w, &a.scale);
    if (st != AC_OK) return st;
    a.B = B, a.Hq = Hq, a.Hk = Hk, a.G = Hq / Hk, a.Lq = Lq, a.Lk = Lk, a.d = d;
    *bytes = window_bwd_workspace(a);
    return AC_OK;
}

extern "C" ac_status ac_window_attn_backward(const ac_view *d_o, const ac_view *q, const ac_view *k, const ac_view *v,
                                             const ac_view *o, const float *lse, const ac_view *dq, const ac_view *dk,
                                             const ac_view *dv, int32_t B, int32_t Hq, int32_t Hk, int32_t Lq,
                                             int32_t Lk, int32_t d, const int32_t *q_lens, const int32_t *k_lens,
                                             const ac_window *w, void *workspace, int64_t workspace_bytes,
                                             void *stream) {
    ac_status st = check_sizes(B, Hq, Hk, Lq, Lk, d);
    WinBwdArgs g{};
    WinArgs &a = g.f;
    if (st == AC_OK) st = window_rule(w, d, &a.w, &a.scale);
    int64_t need = 0;
    if (st == AC_OK) st = ac_window_attn_backward_workspace(B, Hq, Hk, Lq, Lk, d, w, &need);
    if (st != AC_OK) return st;
    if (B == 0 || (Lq == 0 && Lk == 0)) return AC_OK;
    if ((Lq > 0 && (!lse || !rows16(q, B, Hq, Lq) || !rows16(o, B, Hq, Lq) || !rows16(d_o, B, Hq, Lq) ||
                    !rows16(dq, B, Hq, Lq))) ||
        (Lk > 0 && (!rows16(k, B, Hk, Lk) || !rows16(v, B, Hk, Lk) || !rows16(dk, B, Hk, Lk) || !rows16(dv, B, Hk, Lk))))
        return refuse("ac_window_attn_backward: tensors must be 16-byte aligned with positive strides in multiples of 8");
    if ((st = check_workspace("ac_window_attn_backward: workspace too small", workspace, workspace_bytes, need)) != AC_OK) return st;
    if ((st = check_device("ac_window_attn_backward")) != AC_OK) return st;
    if (Lq > 0) a.q = view_of(q), a.o = view_of(o), g.go = view_of(d_o), g.dq = view_of(dq);
    if (Lk > 0) a.k = view_of(k), a.v = view_of(v), g.dk = view_of(dk), g.dv = view_of(dv);
    a.lse = const_cast<float *>(lse), a.q_lens = q_lens, a.k_lens = k_lens;
    a.B = B, a.Hq = Hq, a.Hk = Hk, a.G = Hq / Hk, a.Lq = Lq, a.Lk = Lk, a.d = d;
    a.ws = workspace;
    cudaError_t e = op_err_address(&a.err);
    if (e == cudaSuccess) e = launch_window_bwd(g, (cudaStream_t)stream);
    return e == cudaSuccess ? AC_OK : cuda_refuse("ac_window_attn_backward", e);
}

// ---------------------------------------------------------------- 8-bit cache
namespace {
ac_status check_cache(const ac_cache8 *c, int max_pages) {
    if (!c || c->pages < 0 || c->heads < 1 || max_pages < 0) return refuse("8-bit cache: invalid argument");
    if (c->d != 64 && c->d != 128) return refuse("8-bit cache: d must be 64 or 128", AC_ERR_UNSUPPORTED);
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return refuse("8-bit cache: pages must hold 16, 32, 64 or 128 tokens", AC_ERR_UNSUPPORTED);
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || (reinterpret_cast<uintptr_t>(c->k) & 15u) ||
        (reinterpret_cast<uintptr_t>(c->v) & 15u))
        return refuse("8-bit cache: codes must be 16-byte aligned");
    if ((int64_t)max_pages * c->page_tokens > kMaxLen) return refuse("8-bit cache: sequences of at most 2^30 tokens");
    return AC_OK;
}
}  // namespace

extern "C" ac_status ac_cache8_append(const ac_cache8 *cache, const ac_view *k, const ac_view *v, int32_t B, int32_t n,
                                      const int32_t *page_table, int32_t max_pages, const int32_t *start,
                                      const int32_t *counts, void *stream) {
    ac_status st = check_cache(cache, max_pages);
    if (st != AC_OK) return st;
    if (B < 0 || n < 0 || n > kMaxLen) return refuse("ac_cache8_append: bad sizes");
    if (B == 0 || n == 0) return AC_OK;
    if (!page_table || !start) return refuse("ac_cache8_append: NULL page table or lengths");
    if (!rows16(k, B, cache->heads, n) || !rows16(v, B, cache->heads, n))
        return refuse("ac_cache8_append: tensors must be 16-byte aligned with positive strides in multiples of 8");
    if ((st = check_device("ac_cache8_append")) != AC_OK) return st;
    AppendArgs a{cache->k, cache->v, cache->k_scale, cache->v_scale, view_of(k), view_of(v), page_table, start, counts,
                 cache->pages, cache->heads, cache->page_tokens, cache->d, B, n, max_pages, nullptr};
    cudaError_t e = op_err_address(&a.err);
    if (e == cudaSuccess) e = launch_cache8_append(a, (cudaStream_t)stream);
    return e == cudaSuccess ? AC_OK : cuda_refuse("ac_cache8_append", e);
}

extern "C" ac_status ac_cache8_attn_workspace(const ac_cache8 *cache, int32_t B, int32_t Hq, int32_t Lq,
                                              int32_t max_pages, const ac_window *w, int64_t *bytes) {
    if (!bytes) return refuse("ac_cache8_attn_workspace: NULL argument");
    ac_status st = check_cache(cache, max_pages);
    if (st == AC_OK) st = check_sizes(B, Hq, cache->heads, Lq, max_pages * cache->page_tokens, cache->d);
    WinRule r;
    float scale;
    if (st == AC_OK) st = window_rule(w, cache->d, &r, &scale);
    if (st != AC_OK) return st;
    WinArgs a{};
    a.B = B, a.Hq = Hq, a.Hk = cache->heads, a.G = Hq / cache->heads, a.Lq = Lq, a.d = cache->d, a.w = r;
    a.Lk = max_pages * cache->page_tokens, a.T = cache->page_tokens, a.k8 = cache->k;
    *bytes = B && Lq ? window_workspace(a) : 0;
    return AC_OK;
}

extern "C" ac_status ac_cache8_attn(const ac_cache8 *cache, const ac_view *q, const ac_view *o, float *lse, int32_t B,
                                    int32_t Hq, int32_t Lq, const int32_t *page_table, int32_t max_pages,
                                    const int32_t *q_lens, const int32_t *k_lens, const ac_window *w, void *workspace,
                                    int64_t workspace_bytes, void *stream) {
    int64_t need = 0;
    ac_status st = ac_cache8_attn_workspace(cache, B, Hq, Lq, max_pages, w, &need);
    if (st != AC_OK) return st;
    if (B == 0 || Lq == 0) return AC_OK;
    if (!k_lens || (max_pages > 0 && !page_table)) return refuse("ac_cache8_attn: NULL page table or lengths");
    if (!rows16(q, B, Hq, Lq) || !rows16(o, B, Hq, Lq))
        return refuse("ac_cache8_attn: tensors must be 16-byte aligned with positive strides in multiples of 8");
    if ((st = check_workspace("ac_cache8_attn: workspace too small", workspace, workspace_bytes, need)) != AC_OK) return st;
    if ((st = check_device("ac_cache8_attn")) != AC_OK) return st;
    WinArgs a{};
    if ((st = window_rule(w, cache->d, &a.w, &a.scale)) != AC_OK) return st;
    a.q = view_of(q), a.o = view_of(o);
    a.k8 = cache->k, a.v8 = cache->v, a.ks = cache->k_scale, a.vs = cache->v_scale;
    a.table = page_table, a.pages = cache->pages, a.T = cache->page_tokens, a.max_pages = max_pages;
    a.lse = lse, a.q_lens = q_lens, a.k_lens = k_lens;
    a.B = B, a.Hq = Hq, a.Hk = cache->heads, a.G = Hq / cache->heads, a.Lq = Lq;
    a.Lk = max_pages * cache->page_tokens, a.d = cache->d;
    a.ws = workspace;
    cudaError_t e = op_err_address(&a.err);
    if (e == cudaSuccess) e = launch_window(a, (cudaStream_t)stream);
    return e == cudaSuccess ? AC_OK : cuda_refuse("ac_cache8_attn", e);
}
