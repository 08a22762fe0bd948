// pa_torch.cpp -- the plain calls of pa_window_attention, pa_rope_write_kv and
// pa_copy_blocks from Python straight into libpa.so.
//
// A small step's kernels take 2 to 8 us; reading fifteen tensors' types, devices,
// shapes and pointers through Python attributes took 6 us and ctypes one more (a call
// of pa_window_attention 10.0 us of host time, 3.4 here; of pa_rope_write_kv 9.9 and
// 2.7).  Here they are read from the tensors themselves.  A call whose arguments are all as
// documented goes to the library; any other (a wrong type, shape, layout or
// device, a staging area, a workspace that is too small) comes back as "not
// plain", and the package's own checks say what is wrong or serve it.  Nothing is
// kept from one call for the next.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pa.h"

namespace {

decltype(&pa_window_attention) g_window = nullptr;
decltype(&pa_rope_write_kv) g_rope = nullptr;
decltype(&pa_copy_blocks) g_copy = nullptr;

// The arguments of a call; `plain` turns false at the first that is not as
// documented.
struct Args {
    PyObject *const *a;
    bool plain = true;
    int device = -1;

    void need(bool ok) { plain = plain && ok; }
    bool none(int i) const { return a[i] == Py_None; }
    const at::Tensor *tensor(int i) {
        if (!plain || !THPVariable_Check(a[i])) {
            plain = false;
            return nullptr;
        }
        return &THPVariable_Unpack(a[i]);
    }
    // A contiguous tensor of this type on the call's device (the first one's).
    const at::Tensor *dense(int i, at::ScalarType type) {
        const at::Tensor *t = tensor(i);
        if (!t) return nullptr;
        if (device < 0 && t->is_cuda()) device = t->get_device();
        need(t->scalar_type() == type && t->is_cuda() && t->get_device() == device &&
             t->is_contiguous());
        return plain ? t : nullptr;
    }
    int64_t integer(int i) {
        if (!plain || !PyLong_Check(a[i])) {
            plain = false;
            return 0;
        }
        int overflow = 0;
        const long long v = PyLong_AsLongLongAndOverflow(a[i], &overflow);
        need(!overflow && v >= INT32_MIN && v <= INT32_MAX);
        return v;
    }
    double number(int i) {
        if (plain && PyFloat_Check(a[i])) return PyFloat_AS_DOUBLE(a[i]);
        return static_cast<double>(integer(i));
    }
    // [T, H, d] bf16 with contiguous rows; *stride = elements between tokens
    const at::Tensor *token_rows(int i, int64_t *stride) {
        const at::Tensor *t = tensor(i);
        if (!t) return nullptr;
        if (device < 0 && t->is_cuda()) device = t->get_device();
        need(t->scalar_type() == at::kBFloat16 && t->is_cuda() && t->get_device() == device &&
             t->dim() == 3);
        if (!plain) return nullptr;
        need(t->stride(2) == 1 && (t->stride(1) == t->size(2) || t->size(1) <= 1));
        *stride = t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
        return plain ? t : nullptr;
    }
    // the pool of k_cache (argument i), v_cache (i + 1) and its scales (s, s + 1)
    void pool(int i, int s, pa_kv_desc *kv) {
        const at::Tensor *k = tensor(i);
        if (!k) return;
        const bool codes = k->scalar_type() == at::kByte || k->scalar_type() == at::kFloat8_e4m3fn;
        k = dense(i, codes ? k->scalar_type() : at::kBFloat16);
        const at::Tensor *v = k ? dense(i + 1, k->scalar_type()) : nullptr;
        if (!v || k->dim() != 4 || v->sizes() != k->sizes()) {
            plain = false;
            return;
        }
        for (int d = 0; d < 4; ++d) need(k->size(d) <= INT32_MAX);
        kv->k_cache = k->data_ptr();
        kv->v_cache = v->data_ptr();
        kv->num_blocks = static_cast<int32_t>(k->size(0));
        kv->num_kv_heads = static_cast<int32_t>(k->size(1));
        kv->block_size = static_cast<int32_t>(k->size(2));
        kv->head_dim = static_cast<int32_t>(k->size(3));
        kv->kv_dtype = codes ? PA_KV_FP8_E4M3 : PA_KV_BF16;
        if (!codes) {
            need(none(s) && none(s + 1));
            return;
        }
        const at::Tensor *ks = dense(s, at::kFloat), *vs = dense(s + 1, at::kFloat);
        need(ks && vs && ks->numel() == kv->num_kv_heads && vs->numel() == kv->num_kv_heads);
        if (!plain) return;
        kv->k_scale = static_cast<const float *>(ks->data_ptr());
        kv->v_scale = static_cast<const float *>(vs->data_ptr());
    }
    void *stream(int i) {
        if (!plain || device != c10::cuda::current_device()) {
            plain = false;
            return nullptr;
        }
        if (none(i)) return c10::cuda::getCurrentCUDAStream(device).stream();
        PyObject *h = PyObject_GetAttrString(a[i], "cuda_stream");
        void *p = h ? PyLong_AsVoidPtr(h) : nullptr;
        Py_XDECREF(h);
        need(!PyErr_Occurred());
        PyErr_Clear();
        return p;
    }
};

template <typename T>
T *data(const at::Tensor *t) {
    return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}

// -1: not a plain call; else the library's code.
PyObject *finish(int rc) { return PyLong_FromLong(rc); }

// The library call without the interpreter's lock (a full launch queue blocks it).
template <typename F>
PyObject *launch(F &&call) {
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = call();
    Py_END_ALLOW_THREADS;
    return finish(rc);
}

// q, k_cache, v_cache, block_tables, query_start_loc, context_lens, seq_lens, scale,
// window, num_sinks, out, lse, workspace, stream, k_scale, v_scale
PyObject *window_attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 16 || !g_window) return finish(-1);
    try {
        Args a{args};
        pa_kv_desc kv{};
        const at::Tensor *q = a.dense(0, at::kBFloat16);
        a.pool(1, 14, &kv);
        const at::Tensor *tables = a.dense(3, at::kInt), *qsl = a.dense(4, at::kInt),
                         *ctx = a.dense(5, at::kInt), *seq = a.dense(6, at::kInt);
        const double scale = a.number(7);
        const int64_t window = a.integer(8), sinks = a.integer(9);
        const at::Tensor *out = a.dense(10, at::kBFloat16);
        const at::Tensor *lse = a.none(11) ? nullptr : a.dense(11, at::kFloat);
        const at::Tensor *ws = a.tensor(12);
        if (!a.plain) return finish(-1);
        a.need(q->dim() == 3 && out->sizes() == q->sizes() && tables->dim() == 2 &&
               ws->is_cuda() && ws->get_device() == a.device && ws->is_contiguous());
        if (!a.plain) return finish(-1);
        const int64_t T = q->size(0), hq = q->size(1), B = seq->numel();
        a.need(q->size(2) == kv.head_dim && tables->size(0) == B && ctx->numel() == B &&
               qsl->numel() == B + 1 && (!lse || lse->numel() == T * hq) && T <= INT32_MAX &&
               hq <= INT32_MAX && B <= INT32_MAX && tables->size(1) <= INT32_MAX);
        void *stream = a.stream(13);
        if (!a.plain) return finish(-1);
        void *qp = q->data_ptr(), *op = out->data_ptr(), *wp = ws->data_ptr();
        const int32_t *tp = data<int32_t>(tables), *qslp = data<int32_t>(qsl),
                      *cp = data<int32_t>(ctx), *sp = data<int32_t>(seq);
        float *lp = data<float>(lse);
        const int64_t width = tables->size(1);
        const size_t bytes = ws->nbytes();
        return launch([&] {
            return g_window(qp, &kv, tp, static_cast<int32_t>(width), qslp, cp, sp,
                            static_cast<int32_t>(B), static_cast<int32_t>(T),
                            static_cast<int32_t>(hq), static_cast<float>(scale),
                            static_cast<int32_t>(window), static_cast<int32_t>(sinks), op, lp, wp,
                            bytes, stream);
        });
    } catch (...) {  // a tensor without storage, no device: the package's checks explain
        PyErr_Clear();
        return finish(-1);
    }
}

// q, k, v, positions, inv_freq, axis, slot_mapping, k_cache, v_cache, q_out, adjacent,
// attn_factor, stream, k_scale, v_scale
PyObject *rope_write_kv(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 15 || !g_rope) return finish(-1);
    try {
        Args a{args};
        pa_kv_desc kv{};
        int64_t ks = 0, vs = 0, qs = 0;
        const at::Tensor *k = a.token_rows(1, &ks), *v = a.token_rows(2, &vs);
        const at::Tensor *q = a.none(0) ? nullptr : a.token_rows(0, &qs);
        const at::Tensor *pos = a.dense(3, at::kInt), *freq = a.dense(4, at::kDouble),
                         *axis = a.none(5) ? nullptr : a.dense(5, at::kInt),
                         *slots = a.dense(6, at::kLong);
        a.pool(7, 13, &kv);
        const at::Tensor *q_out = a.none(9) ? nullptr : a.dense(9, at::kBFloat16);
        a.need(PyBool_Check(args[10]));
        const double factor = a.number(11);
        if (!a.plain) return finish(-1);
        const int64_t T = k->size(0), half = freq->numel();
        a.need(k->size(1) == kv.num_kv_heads && k->size(2) == kv.head_dim &&
               v->sizes() == k->sizes() && (q != nullptr) == (q_out != nullptr) &&
               (!q || (q->size(0) == T && q->size(2) == kv.head_dim &&
                       q_out->sizes() == q->sizes())) &&
               (pos->dim() == 1 || pos->dim() == 2) && pos->size(-1) == T &&
               slots->numel() == T && (!axis || axis->numel() == half) && T <= INT32_MAX &&
               half <= INT32_MAX / 2 && (!q || q->size(1) <= INT32_MAX) &&
               (pos->dim() == 1 || pos->size(0) <= INT32_MAX));
        void *stream = a.stream(12);
        if (!a.plain) return finish(-1);
        pa_rope_desc rope{};
        rope.inv_freq = data<double>(freq);
        rope.axis = data<int32_t>(axis);
        rope.rot_dim = static_cast<int32_t>(2 * half);
        rope.num_axes = pos->dim() == 1 ? 1 : static_cast<int32_t>(pos->size(0));
        rope.adjacent = args[10] == Py_True;
        rope.attn_factor = static_cast<float>(factor);
        void *qp = q ? q->data_ptr() : nullptr, *kp = k->data_ptr(), *vp = v->data_ptr();
        void *op = q_out ? q_out->data_ptr() : nullptr;
        const int32_t *pp = data<int32_t>(pos);
        const int64_t *sp = data<int64_t>(slots);
        const int32_t hq = q ? static_cast<int32_t>(q->size(1)) : 0;
        return launch([&] {
            return g_rope(qp, qs, kp, ks, vp, vs, pp, &rope, sp, static_cast<int32_t>(T), hq, &kv,
                          op, stream);
        });
    } catch (...) {
        PyErr_Clear();
        return finish(-1);
    }
}

// address and count of the layers' descriptors, their device, pairs, stream
PyObject *copy_blocks(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 5 || !g_copy) return finish(-1);
    try {
        Args a{args};
        const int64_t layers = a.integer(1);
        a.device = static_cast<int>(a.integer(2));
        a.need(PyLong_Check(args[0]) && layers > 0 && a.device >= 0);
        const at::Tensor *pairs = a.dense(3, at::kInt);
        if (!a.plain) return finish(-1);
        a.need(pairs->dim() == 2 && pairs->size(1) == 2 && pairs->size(0) <= INT32_MAX);
        void *stream = a.stream(4);
        const pa_kv_desc *descs = static_cast<const pa_kv_desc *>(PyLong_AsVoidPtr(args[0]));
        a.need(!PyErr_Occurred());
        PyErr_Clear();
        if (!a.plain) return finish(-1);
        const int32_t *pp = data<int32_t>(pairs);
        const int32_t count = static_cast<int32_t>(pairs->size(0));
        return launch([&] { return g_copy(descs, static_cast<int32_t>(layers), pp, count, stream); });
    } catch (...) {
        PyErr_Clear();
        return finish(-1);
    }
}

// bind(addresses of pa_window_attention, pa_rope_write_kv and pa_copy_blocks of the loaded
// libpa.so)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "bind(window_attention, rope_write_kv, copy_blocks)");
        return nullptr;
    }
    void *w = PyLong_AsVoidPtr(args[0]), *r = PyLong_AsVoidPtr(args[1]),
         *c = PyLong_AsVoidPtr(args[2]);
    if (PyErr_Occurred()) return nullptr;
    g_window = reinterpret_cast<decltype(g_window)>(w);
    g_rope = reinterpret_cast<decltype(g_rope)>(r);
    g_copy = reinterpret_cast<decltype(g_copy)>(c);
    Py_RETURN_NONE;
}

// METH_FASTCALL functions have a wider type than the table's field
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"bind", fast<bind>(), METH_FASTCALL, nullptr},
    {"window_attention", fast<window_attention>(), METH_FASTCALL, nullptr},
    {"rope_write_kv", fast<rope_write_kv>(), METH_FASTCALL, nullptr},
    {"copy_blocks", fast<copy_blocks>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_torch() { return PyModule_Create(&module); }
