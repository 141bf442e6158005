// fast_binding.cpp -- the streaming operators' calls from Python without the
// interpreter's share: a single-token call's kernels take 3 us, reading four
// tensors' attributes in Python takes 15.
//
// Each function here takes the common case (tensors on the current CUDA device
// with the right types and shapes, new outputs) through the C ABI of libac; for
// everything else, wrong arguments and tensors that autograd records included, it returns
// None, and the caller in streaming.py goes its own way, which checks and explains.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ac.h"

namespace {

using at::Tensor;

const Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const Tensor &t, at::ScalarType type, c10::DeviceIndex dev) {
    return t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided;
}

// A [B, H, L, d] tensor with d contiguous.
bool rows(const Tensor &t, at::ScalarType type, c10::DeviceIndex dev, ac_view *v) {
    if (!on(t, type, dev) || t.dim() != 4 || (t.stride(3) != 1 && t.size(3) > 1)) return false;
    *v = ac_view{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
    return true;
}

bool same(const Tensor &t, int64_t a, int64_t b, int64_t c, int64_t d) {
    return t.size(0) == a && t.size(1) == b && t.size(2) == c && t.size(3) == d;
}

// int32 lengths [B], or None.
bool lens(PyObject *o, int64_t B, c10::DeviceIndex dev, const int32_t **p) {
    *p = nullptr;
    if (o == Py_None) return true;
    const Tensor *t = tensor(o);
    if (!t || !on(*t, at::kInt, dev) || t->dim() != 1 || t->size(0) != B || !t->is_contiguous()) return false;
    *p = static_cast<const int32_t *>(t->data_ptr());
    return true;
}

bool integers(PyObject *const *args, int n, int64_t *out) {
    for (int i = 0; i < n; ++i) {
        if (!PyLong_Check(args[i])) return false;
        out[i] = PyLong_AsLongLong(args[i]);
        if (out[i] == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            return false;
        }
    }
    return true;
}

bool fits(int64_t v) { return v >= -0x7FFFFFFF && v <= 0x7FFFFFFF; }

Tensor like(const Tensor &t, at::IntArrayRef shape, at::ScalarType type) {
    return at::empty(shape, t.options().dtype(type));
}

// Whether autograd records what is done with the tensor: backwards, or its tangent forwards.
bool recorded(const Tensor &t) {
    return (at::GradMode::is_enabled() && t.requires_grad()) || t._fw_grad(0).defined();
}

void *stream(c10::DeviceIndex dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

PyObject *none() { Py_RETURN_NONE; }

PyObject *error(ac_status st) { return PyLong_FromLong(st); }  // the caller raises

PyObject *two(const Tensor &a, const Tensor &b) {
    PyObject *t = PyTuple_New(2);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
    return t;
}

// rope(q, k, positions, freq address, pairs address, axes, pairs' sum, interleaved, inverse)
PyObject *rope(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS  // (torch's own exceptions: out of memory is torch.OutOfMemoryError)
    int64_t i[6];
    if (n != 9 || !integers(args + 3, 6, i)) return none();
    const Tensor *q = tensor(args[0]), *k = tensor(args[1]), *pos = tensor(args[2]);
    if (!q || !pos || !q->is_cuda() || (!k && args[1] != Py_None) || recorded(*q) || (k && recorded(*k))) return none();
    const c10::DeviceIndex dev = q->get_device();
    if (dev != c10::cuda::current_device()) return none();
    const at::ScalarType type = q->scalar_type();
    const int32_t dtype = type == at::kBFloat16 ? AC_DTYPE_BF16 : type == at::kHalf ? AC_DTYPE_F16 : type == at::kFloat ? AC_DTYPE_F32 : -1;
    ac_view vq, vk{}, oq, ok{};
    if (dtype < 0 || !rows(*q, type, dev, &vq)) return none();
    const int64_t B = q->size(0), Hq = q->size(1), L = q->size(2), d = q->size(3), axes = i[2];
    int64_t Hk = 0;
    if (k) {
        if (!rows(*k, type, dev, &vk)) return none();
        Hk = k->size(1);
        if (!same(*k, B, Hk, L, d)) return none();
    }
    if (!on(*pos, at::kInt, dev) || !pos->is_contiguous()) return none();
    const bool per_sequence = pos->dim() == 3;
    if (per_sequence ? pos->size(0) != B || pos->size(1) != L || pos->size(2) != axes
                     : pos->dim() != 2 || pos->size(0) != L || pos->size(1) != axes)
        return none();
    if (!fits(B) || !fits(Hq) || !fits(Hk) || !fits(L) || !fits(d)) return none();
    const Tensor yq = like(*q, {B, Hq, L, d}, type);
    const Tensor yk = k ? like(*k, {B, Hk, L, d}, type) : Tensor();
    oq = ac_view{yq.data_ptr(), Hq * L * d, L * d, d};
    if (k) ok = ac_view{yk.data_ptr(), Hk * L * d, L * d, d};
    const ac_status st = ac_rope_axes(dtype, &vq, &oq, (int32_t)Hq, &vk, &ok, (int32_t)Hk, (int32_t)B, (int32_t)L, (int32_t)d,
                                      static_cast<const int32_t *>(pos->data_ptr()), per_sequence ? L * axes : 0,
                                      reinterpret_cast<const double *>(i[0]), reinterpret_cast<const int32_t *>(i[1]),
                                      (int32_t)axes, i[4] != 0, i[5] != 0, stream(dev));
    if (st != AC_OK) return error(st);
    return k ? two(yq, yk) : THPVariable_Wrap(yq);
    END_HANDLE_TH_ERRORS
}

struct Window {
    ac_window w;
    bool read(PyObject *const *args) {  // left, right, sinks, block, scale
        int64_t i[4];
        if (!integers(args, 4, i) || !fits(i[0]) || !fits(i[1]) || !fits(i[2]) || !fits(i[3]) || !PyFloat_Check(args[4])) return false;
        w = ac_window{(int32_t)i[0], (int32_t)i[1], (int32_t)i[2], (int32_t)i[3], (float)PyFloat_AS_DOUBLE(args[4])};
        return true;
    }
};

// window(q, k, v, left, right, sinks, block, scale, q_lens, k_lens, lse wanted)
PyObject *window(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Window win;
    if (n != 11 || !win.read(args + 3)) return none();
    const Tensor *q = tensor(args[0]), *k = tensor(args[1]), *v = tensor(args[2]);
    if (!q || !k || !v || !q->is_cuda() || recorded(*q) || recorded(*k) || recorded(*v)) return none();
    const c10::DeviceIndex dev = q->get_device();
    ac_view vq, vk, vv;
    if (dev != c10::cuda::current_device() || !rows(*q, at::kBFloat16, dev, &vq) || !rows(*k, at::kBFloat16, dev, &vk) ||
        !rows(*v, at::kBFloat16, dev, &vv))
        return none();
    const int64_t B = q->size(0), Hq = q->size(1), Lq = q->size(2), d = q->size(3), Hk = k->size(1), Lk = k->size(2);
    const int32_t *ql, *kl;
    if (!same(*k, B, Hk, Lk, d) || !same(*v, B, Hk, Lk, d) || !lens(args[8], B, dev, &ql) || !lens(args[9], B, dev, &kl) ||
        !fits(B) || !fits(Hq) || !fits(Hk) || !fits(Lq) || !fits(Lk) || !fits(d))
        return none();
    const bool want = args[10] == Py_True;
    int64_t bytes = 0;
    ac_status st = ac_window_attn_workspace((int32_t)B, (int32_t)Hq, (int32_t)Hk, (int32_t)Lq, (int32_t)Lk, (int32_t)d, &win.w, &bytes);
    if (st != AC_OK) return error(st);
    const Tensor o = like(*q, {B, Hq, Lq, d}, at::kBFloat16);
    const Tensor lse = want ? like(*q, {B, Hq, Lq}, at::kFloat) : Tensor();
    const Tensor ws = bytes ? like(*q, {bytes}, at::kByte) : Tensor();
    const ac_view vo{o.data_ptr(), Hq * Lq * d, Lq * d, d};
    st = ac_window_attn(&vq, &vk, &vv, &vo, want ? static_cast<float *>(lse.data_ptr()) : nullptr, (int32_t)B, (int32_t)Hq,
                        (int32_t)Hk, (int32_t)Lq, (int32_t)Lk, (int32_t)d, ql, kl, &win.w, bytes ? ws.data_ptr() : nullptr,
                        bytes, stream(dev));
    if (st != AC_OK) return error(st);
    return want ? two(o, lse) : THPVariable_Wrap(o);
    END_HANDLE_TH_ERRORS
}

// backward(d_out, q, k, v, o, lse, left, right, sinks, block, scale, q_lens, k_lens)
PyObject *backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Window win;
    if (n != 13 || !win.read(args + 6)) return none();
    const Tensor *t[6];
    for (int i = 0; i < 6; ++i)
        if (!(t[i] = tensor(args[i])) || !t[i]->is_cuda() || recorded(*t[i])) return none();
    const c10::DeviceIndex dev = t[1]->get_device();
    ac_view v[5];
    if (dev != c10::cuda::current_device()) return none();
    for (int i = 0; i < 5; ++i)
        if (!rows(*t[i], at::kBFloat16, dev, &v[i])) return none();
    const int64_t B = t[1]->size(0), Hq = t[1]->size(1), Lq = t[1]->size(2), d = t[1]->size(3);
    const int64_t Hk = t[2]->size(1), Lk = t[2]->size(2);
    const Tensor &lse = *t[5];
    const int32_t *ql, *kl;
    if (!same(*t[0], B, Hq, Lq, d) || !same(*t[4], B, Hq, Lq, d) || !same(*t[2], B, Hk, Lk, d) || !same(*t[3], B, Hk, Lk, d) ||
        !on(lse, at::kFloat, dev) || lse.dim() != 3 || lse.size(0) != B || lse.size(1) != Hq || lse.size(2) != Lq ||
        !lse.is_contiguous() || !lens(args[11], B, dev, &ql) || !lens(args[12], B, dev, &kl) || !fits(B) || !fits(Hq) ||
        !fits(Hk) || !fits(Lq) || !fits(Lk) || !fits(d))
        return none();
    int64_t bytes = 0;
    ac_status st = ac_window_attn_backward_workspace((int32_t)B, (int32_t)Hq, (int32_t)Hk, (int32_t)Lq, (int32_t)Lk, (int32_t)d,
                                                     &win.w, &bytes);
    if (st != AC_OK) return error(st);
    const Tensor dq = like(*t[1], {B, Hq, Lq, d}, at::kBFloat16), dk = like(*t[1], {B, Hk, Lk, d}, at::kBFloat16),
                 dv = like(*t[1], {B, Hk, Lk, d}, at::kBFloat16);
    const Tensor ws = bytes ? like(*t[1], {bytes}, at::kByte) : Tensor();
    const ac_view vdq{dq.data_ptr(), Hq * Lq * d, Lq * d, d}, vdk{dk.data_ptr(), Hk * Lk * d, Lk * d, d},
        vdv{dv.data_ptr(), Hk * Lk * d, Lk * d, d};
    st = ac_window_attn_backward(&v[0], &v[1], &v[2], &v[3], &v[4], static_cast<const float *>(lse.data_ptr()), &vdq, &vdk, &vdv,
                                 (int32_t)B, (int32_t)Hq, (int32_t)Hk, (int32_t)Lq, (int32_t)Lk, (int32_t)d, ql, kl, &win.w,
                                 bytes ? ws.data_ptr() : nullptr, bytes, stream(dev));
    if (st != AC_OK) return error(st);
    PyObject *r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(dq));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(dk));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(dv));
    return r;
    END_HANDLE_TH_ERRORS
}

// The tensors of a cache: k, v, k_scale, v_scale.
bool cache_of(PyObject *const *args, c10::DeviceIndex dev, ac_cache8 *c) {
    const Tensor *t[4];
    for (int i = 0; i < 4; ++i) {
        t[i] = tensor(args[i]);
        if (!t[i] || !on(*t[i], i < 2 ? at::kFloat8_e4m3fn : at::kFloat, dev) || t[i]->dim() != (i < 2 ? 4 : 2) || !t[i]->is_contiguous())
            return false;
    }
    const int64_t pages = t[0]->size(0), heads = t[0]->size(1), T = t[0]->size(2), d = t[0]->size(3);
    if (!same(*t[1], pages, heads, T, d) || !fits(pages) || !fits(heads) || !fits(T) || !fits(d)) return false;
    for (int i = 2; i < 4; ++i)
        if (t[i]->size(0) != pages || t[i]->size(1) != heads) return false;
    *c = ac_cache8{static_cast<uint8_t *>(t[0]->data_ptr()), static_cast<uint8_t *>(t[1]->data_ptr()),
                   static_cast<float *>(t[2]->data_ptr()), static_cast<float *>(t[3]->data_ptr()),
                   (int32_t)pages, (int32_t)heads, (int32_t)T, (int32_t)d};
    return true;
}

bool table_of(PyObject *o, int64_t B, c10::DeviceIndex dev, const int32_t **p, int32_t *per) {
    const Tensor *t = tensor(o);
    if (!t || !on(*t, at::kInt, dev) || t->dim() != 2 || t->size(0) != B || !t->is_contiguous() || !fits(t->size(1))) return false;
    *p = static_cast<const int32_t *>(t->data_ptr());
    *per = (int32_t)t->size(1);
    return true;
}

// append(k, v, cache's four tensors, page_table, start, counts): True when done
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) return none();
    const Tensor *k = tensor(args[0]), *v = tensor(args[1]);
    if (!k || !v || !k->is_cuda() || recorded(*k) || recorded(*v)) return none();
    const c10::DeviceIndex dev = k->get_device();
    ac_view vk, vv;
    ac_cache8 c;
    if (dev != c10::cuda::current_device() || !rows(*k, at::kBFloat16, dev, &vk) || !rows(*v, at::kBFloat16, dev, &vv) ||
        !cache_of(args + 2, dev, &c))
        return none();
    const int64_t B = k->size(0), H = k->size(1), len = k->size(2), d = k->size(3);
    const int32_t *table, *start, *counts;
    int32_t per;
    if (!same(*v, B, H, len, d) || H != c.heads || d != c.d || !fits(B) || !fits(len) || !table_of(args[6], B, dev, &table, &per) ||
        args[7] == Py_None || !lens(args[7], B, dev, &start) || !lens(args[8], B, dev, &counts))
        return none();
    const ac_status st = ac_cache8_append(&c, &vk, &vv, (int32_t)B, (int32_t)len, table, per, start, counts, stream(dev));
    if (st != AC_OK) return error(st);
    Py_RETURN_TRUE;
    END_HANDLE_TH_ERRORS
}

// cache_attn(q, cache's four tensors, page_table, k_lens, left, right, sinks, block, scale, q_lens, lse wanted)
PyObject *cache_attn(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Window win;
    if (n != 14 || !win.read(args + 7)) return none();
    const Tensor *q = tensor(args[0]);
    if (!q || !q->is_cuda() || recorded(*q)) return none();
    const c10::DeviceIndex dev = q->get_device();
    ac_view vq;
    ac_cache8 c;
    if (dev != c10::cuda::current_device() || !rows(*q, at::kBFloat16, dev, &vq) || !cache_of(args + 1, dev, &c)) return none();
    const int64_t B = q->size(0), Hq = q->size(1), Lq = q->size(2), d = q->size(3);
    const int32_t *table, *ql, *kl;
    int32_t per;
    if (d != c.d || !fits(B) || !fits(Hq) || !fits(Lq) || !table_of(args[5], B, dev, &table, &per) || args[6] == Py_None ||
        !lens(args[6], B, dev, &kl) || !lens(args[12], B, dev, &ql))
        return none();
    const bool want = args[13] == Py_True;
    int64_t bytes = 0;
    ac_status st = ac_cache8_attn_workspace(&c, (int32_t)B, (int32_t)Hq, (int32_t)Lq, per, &win.w, &bytes);
    if (st != AC_OK) return error(st);
    const Tensor o = like(*q, {B, Hq, Lq, d}, at::kBFloat16);
    const Tensor lse = want ? like(*q, {B, Hq, Lq}, at::kFloat) : Tensor();
    const Tensor ws = bytes ? like(*q, {bytes}, at::kByte) : Tensor();
    const ac_view vo{o.data_ptr(), Hq * Lq * d, Lq * d, d};
    st = ac_cache8_attn(&c, &vq, &vo, want ? static_cast<float *>(lse.data_ptr()) : nullptr, (int32_t)B, (int32_t)Hq, (int32_t)Lq,
                        table, per, ql, kl, &win.w, bytes ? ws.data_ptr() : nullptr, bytes, stream(dev));
    if (st != AC_OK) return error(st);
    return want ? two(o, lse) : THPVariable_Wrap(o);
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, nullptr},
    {"window", (PyCFunction)(void (*)(void))window, METH_FASTCALL, nullptr},
    {"backward", (PyCFunction)(void (*)(void))backward, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"cache_attn", (PyCFunction)(void (*)(void))cache_attn, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast(void) { return PyModule_Create(&module); }
