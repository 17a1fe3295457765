// fa_torch.cpp -- the Python binding's short way into the library for the
// ordinary call: contiguous (or evenly strided) CUDA tensors of one device and
// one 16-bit type on the current device and stream.
//
// A call through ctypes costs the host 10 to 30 us, most of it in Python: a
// decoding step's kernels run for 3 to 10.  Here the tensors' fields are read
// and the outputs allocated in C++, and the same C entry point is called.  Each
// function returns None for anything out of the ordinary -- another device,
// shape, type or layout -- and the Python path then takes the call, with its
// checks and messages; a status other than FA_OK comes back as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>

#include "fa.h"

namespace {

// A contiguous CUDA tensor of the given device.
const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool plain(const at::Tensor &t, at::ScalarType type, int dev) {
    return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.is_contiguous();
}

// Element strides (batch, row, head) of a [B, S, H, D] input: zeros if it is
// contiguous; false if the tensor loads cannot take it as it lies.
bool strides(const at::Tensor &t, long long (&st)[3]) {
    st[0] = st[1] = st[2] = 0;
    if (t.is_contiguous()) return true;
    if (t.stride(3) != 1 || (reinterpret_cast<uintptr_t>(t.data_ptr()) & 15u)) return false;
    for (int i = 0; i < 3; ++i) {
        st[i] = t.size(i) == 1 ? 8 : t.stride(i);
        if (st[i] <= 0 || (st[i] & 7) || st[i] >= (1LL << 39)) return false;
    }
    return true;
}

PyObject *none() { Py_RETURN_NONE; }

// The current device; -1 where there is none.
int current() {
    c10::DeviceIndex d = -1;
    return c10::cuda::GetDevice(&d) == cudaSuccess ? d : -1;
}

struct Call {   // what the forward and the backward share
    const at::Tensor *q, *k, *v;
    int B, Sq, Sk, Hq, Hkv, D, dev;
    float scale;
    int causal;
    fa_dtype dtype;
    fa_ext ext;
};

// q, k, v, scale or None, causal, softcap, ranges buffer or None, its B and S
bool open_call(PyObject *const *a, Call &c) {
    c.q = tensor(a[0]), c.k = tensor(a[1]), c.v = tensor(a[2]);
    if (!c.q || !c.k || !c.v || c.q->dim() != 4 || c.k->dim() != 4 || !c.q->is_cuda()) return false;
    c.dev = c.q->get_device();
    if (c.dev != current()) return false;
    const at::ScalarType ty = c.q->scalar_type();
    if (ty != at::kBFloat16 && ty != at::kHalf) return false;
    c.dtype = ty == at::kBFloat16 ? FA_BF16 : FA_FP16;
    for (const at::Tensor *t : {c.k, c.v})
        if (!t->is_cuda() || t->get_device() != c.dev || t->scalar_type() != ty) return false;
    if (c.v->sizes() != c.k->sizes() || c.q->size(0) != c.k->size(0) || c.q->size(3) != c.k->size(3)) return false;
    c.B = (int)c.q->size(0), c.Sq = (int)c.q->size(1), c.Hq = (int)c.q->size(2), c.D = (int)c.q->size(3);
    c.Sk = (int)c.k->size(1), c.Hkv = (int)c.k->size(2);
    if (c.q->numel() == 0 || c.k->numel() == 0) return false;
    if (a[3] == Py_None) {
        c.scale = (float)(1.0 / std::sqrt((double)c.D));
    } else {
        c.scale = (float)PyFloat_AsDouble(a[3]);
    }
    c.causal = PyObject_IsTrue(a[4]);
    const double cap = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) return false;
    std::memset(&c.ext, 0, sizeof(c.ext));
    c.ext.window_left = c.ext.window_right = -1;
    c.ext.softcap = (float)cap;
    if (a[6] != Py_None) {
        const at::Tensor *r = tensor(a[6]);
        if (!r || !plain(*r, at::kByte, c.dev)) return false;
        if (PyLong_AsLong(a[7]) != c.B || PyLong_AsLong(a[8]) != c.Sq || c.Sq != c.Sk) return false;
        c.ext.mask_ranges = r->data_ptr();
        c.ext.mask_ranges_bytes = (size_t)r->numel();
    }
    return strides(*c.q, c.ext.q_stride) && strides(*c.k, c.ext.k_stride) && strides(*c.v, c.ext.v_stride);
}

cudaStream_t stream(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

PyObject *pair(at::Tensor a, at::Tensor b) {
    PyObject *t = PyTuple_New(2);
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(a)));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(b)));
    return t;
}

// A C++ exception (an allocation that failed) becomes a Python one.
template <typename F>
PyObject *guarded(F &&f) {
    try {
        PyObject *r = f();
        if (PyErr_Occurred()) {   // an argument was no number: the Python path says so
            PyErr_Clear();
            Py_XDECREF(r);
            return none();
        }
        return r;
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// agree(q, k, v, o, dout, dq, dk, dv, lse, cu_q, cu_k) -> True if the tensors of a
// call (None: not of it) have the shapes, types and GPU that q and k say
PyObject *agree(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 11) return none();
    return guarded([&]() -> PyObject * {
        const at::Tensor *t[11];
        for (int i = 0; i < 11; ++i) {
            t[i] = a[i] == Py_None ? nullptr : tensor(a[i]);
            if (!t[i] && a[i] != Py_None) return none();
        }
        if (!t[0] || !t[1] || !t[2]) return none();
        const at::Tensor &q = *t[0], &k = *t[1], &v = *t[2];
        const int64_t d = q.dim();
        if ((d != 3 && d != 4) || k.dim() != d || v.dim() != d || !q.is_cuda() || k.size(d - 1) != q.size(d - 1) ||
            (d == 4 && k.size(0) != q.size(0)))
            return none();
        const at::IntArrayRef qs = q.sizes(), ks = k.sizes();
        auto like = [&](const at::Tensor &x, at::IntArrayRef rows, int64_t last) {
            return x.is_cuda() && x.get_device() == q.get_device() && x.scalar_type() == q.scalar_type() &&
                   x.dim() == d && x.size(d - 1) == last && x.sizes().slice(0, d - 1) == rows.slice(0, d - 1);
        };
        const int64_t D = q.size(d - 1), Dv = v.size(d - 1);
        const at::IntArrayRef rows[8] = {qs, ks, ks, qs, qs, qs, ks, ks};
        const int64_t last[8] = {D, D, Dv, Dv, Dv, D, D, Dv};
        for (int i = 1; i < 8; ++i)
            if (t[i] && !like(*t[i], rows[i], last[i])) return none();
        if (const at::Tensor *l = t[8])
            if (!l->is_cuda() || l->get_device() != q.get_device() || l->scalar_type() != at::kFloat ||
                l->numel() * D != q.numel())
                return none();
        if (!t[9] != !t[10]) return none();
        for (int i = 9; i < 11; ++i)
            if (t[i] && (!plain(*t[i], at::kInt, (int)q.get_device()) || t[i]->dim() != 1 ||
                         t[i]->sizes() != t[9]->sizes()))
                return none();
        Py_RETURN_TRUE;
    });
}

// fwd(q, k, v, scale, causal, softcap, ranges, B, S) -> (o, lse)
PyObject *fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        if (!open_call(a, c)) return none();
        at::Tensor o = at::empty(c.q->sizes(), c.q->options().memory_format(at::MemoryFormat::Contiguous));
        at::Tensor lse = at::empty({c.B, c.Hq, c.Sq}, c.q->options().dtype(at::kFloat));
        const fa_status st = fa_fwd_ext(c.q->data_ptr(), c.k->data_ptr(), c.v->data_ptr(), o.data_ptr(),
                                        (float *)lse.data_ptr(), c.B, c.Sq, c.Sk, c.Hq, c.Hkv, c.D, c.scale, c.causal,
                                        nullptr, nullptr, &c.ext, c.dtype, stream(c.dev));
        return st == FA_OK ? pair(std::move(o), std::move(lse)) : PyLong_FromLong(st);
    });
}

// bwd(q, k, v, scale, causal, softcap, ranges, B, S, o, dout, lse) -> (dq, dk, dv), scratch from the library's pool
PyObject *bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 12) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        if (!open_call(a, c)) return none();
        const at::Tensor *o = tensor(a[9]), *g = tensor(a[10]), *lse = tensor(a[11]);
        if (!o || !g || !lse) return none();
        for (const at::Tensor *t : {o, g})
            if (!t->is_cuda() || t->get_device() != c.dev || t->scalar_type() != c.q->scalar_type() ||
                t->sizes() != c.q->sizes())
                return none();
        if (!plain(*lse, at::kFloat, c.dev) || lse->numel() != (int64_t)c.B * c.Hq * c.Sq) return none();
        if (!strides(*o, c.ext.o_stride) || !strides(*g, c.ext.dout_stride)) return none();
        at::Tensor d[3] = {at::empty(c.q->sizes(), c.q->options().memory_format(at::MemoryFormat::Contiguous)),
                           at::empty(c.k->sizes(), c.q->options().memory_format(at::MemoryFormat::Contiguous)),
                           at::empty(c.k->sizes(), c.q->options().memory_format(at::MemoryFormat::Contiguous))};
        const fa_status st =
            fa_bwd_ext(c.q->data_ptr(), c.k->data_ptr(), c.v->data_ptr(), o->data_ptr(), g->data_ptr(),
                       (const float *)lse->data_ptr(), d[0].data_ptr(), d[1].data_ptr(), d[2].data_ptr(), c.B, c.Sq,
                       c.Sk, c.Hq, c.Hkv, c.D, c.scale, c.causal, nullptr, nullptr, &c.ext, 0, c.dtype, nullptr, 0,
                       stream(c.dev));
        if (st != FA_OK) return PyLong_FromLong(st);
        PyObject *t = PyTuple_New(3);
        for (int i = 0; i < 3; ++i) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(std::move(d[i])));
        return t;
    });
}

// mask_ranges(B, S, doc_ids, prefix_len, causal) -> buffer
PyObject *mask_ranges(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 5) return none();
    return guarded([&]() -> PyObject * {
        const long B = PyLong_AsLong(a[0]), S = PyLong_AsLong(a[1]);
        const at::Tensor *doc = a[2] == Py_None ? nullptr : tensor(a[2]);
        const at::Tensor *pre = a[3] == Py_None ? nullptr : tensor(a[3]);
        if (PyErr_Occurred() || B <= 0 || S <= 0 || B > 0x7fffffffL || S > 0x7fffffffL) return none();
        if ((!doc && a[2] != Py_None) || (!pre && a[3] != Py_None)) return none();
        const int dev = current();
        if (dev < 0) return none();
        if (doc && (!plain(*doc, at::kInt, dev) || doc->dim() != 2 || doc->size(0) != B || doc->size(1) != S))
            return none();
        if (pre && (!plain(*pre, at::kInt, dev) || pre->size(0) != B || pre->dim() > 2 ||
                    (pre->dim() == 2 && pre->size(1) != S)))
            return none();
        const size_t need = fa_mask_ranges_bytes((int)B, (int)S);
        if (need == 0) return none();
        at::Tensor r = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev));
        const fa_status st = fa_mask_ranges(doc ? (const int *)doc->data_ptr() : nullptr,
                                            pre ? (const int *)pre->data_ptr() : nullptr, pre && pre->dim() == 2,
                                            (int)B, (int)S, PyObject_IsTrue(a[4]), -1, -1, r.data_ptr(), need,
                                            stream(dev));
        return st == FA_OK ? THPVariable_Wrap(std::move(r)) : PyLong_FromLong(st);
    });
}

// cache(k, v, k_scale, v_scale, block_table) -> True if they make a cache on the current device
PyObject *cache(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 5) return none();
    return guarded([&]() -> PyObject * {
        const at::Tensor *t[5];
        for (int i = 0; i < 5; ++i)
            if (!(t[i] = tensor(a[i]))) return none();
        const int dev = current();
        if (t[0]->dim() != 4 || t[1]->dim() != 4 || t[4]->dim() != 2) return none();
        const int64_t P = t[0]->size(0), H = t[0]->size(1), ps = t[0]->size(2), D = t[0]->size(3);
        if (!plain(*t[0], at::kFloat8_e4m3fn, dev) || !plain(*t[1], at::kFloat8_e4m3fn, dev) ||
            !plain(*t[2], at::kFloat, dev) || !plain(*t[3], at::kFloat, dev) || !plain(*t[4], at::kInt, dev))
            return none();
        if (t[1]->sizes() != at::IntArrayRef({P, H, D, ps}) || t[2]->sizes() != at::IntArrayRef({P, H}) ||
            t[3]->sizes() != at::IntArrayRef({P, H}))
            return none();
        Py_RETURN_TRUE;
    });
}

const fa_kv_cache *cache_struct(PyObject *o) {
    return reinterpret_cast<const fa_kv_cache *>(PyLong_AsUnsignedLongLong(o));
}

// append(cache struct's address, B, device, cache_len, k_new, v_new, cu_new, max_new) -> status
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 8) return none();
    return guarded([&]() -> PyObject * {
        const fa_kv_cache *kc = cache_struct(a[0]);
        const long B = PyLong_AsLong(a[1]), dev = PyLong_AsLong(a[2]);
        const at::Tensor *len = tensor(a[3]), *k = tensor(a[4]), *v = tensor(a[5]);
        const at::Tensor *cu = a[6] == Py_None ? nullptr : tensor(a[6]);
        if (PyErr_Occurred() || !len || !k || !v || (!cu && a[6] != Py_None)) return none();
        if (dev != current()) return none();
        const at::ScalarType ty = k->scalar_type();
        if ((ty != at::kBFloat16 && ty != at::kHalf) || !plain(*k, ty, (int)dev) || !plain(*v, ty, (int)dev) ||
            k->sizes() != v->sizes() || !plain(*len, at::kInt, (int)dev) || len->dim() != 1 || len->size(0) != B)
            return none();
        const int64_t d = k->dim();
        if (d != (cu ? 3 : 4) || k->size(d - 2) != kc->Hkv || k->size(d - 1) != kc->D) return none();
        long max_new;
        if (cu) {
            if (!plain(*cu, at::kInt, (int)dev) || cu->dim() != 1 || cu->size(0) != B + 1) return none();
            max_new = PyLong_AsLong(a[7]);   // (None: the Python path refuses)
            if (PyErr_Occurred()) return none();
        } else {
            if (k->size(0) != B) return none();
            max_new = (long)k->size(1);
        }
        const int64_t rows = cu ? k->size(0) : (int64_t)B * max_new;
        if (max_new <= 0 || max_new > 0x7fffffffL || rows <= 0 || rows > 0x7fffffffL) return none();
        return PyLong_FromLong(fa_kvcache_append(kc, (const int *)len->data_ptr(), k->data_ptr(), v->data_ptr(),
                                                 cu ? (const int *)cu->data_ptr() : nullptr, (int)rows, (int)B, (int)max_new,
                                                 ty == at::kBFloat16 ? FA_BF16 : FA_FP16, stream((int)dev)));
    });
}

// attend(cache struct's address, B, device, q, cache_len, scale, softcap, window_left) -> (o, lse)
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 8) return none();
    return guarded([&]() -> PyObject * {
        const fa_kv_cache *kc = cache_struct(a[0]);
        const long B = PyLong_AsLong(a[1]), dev = PyLong_AsLong(a[2]);
        const at::Tensor *q = tensor(a[3]), *len = tensor(a[4]);
        if (PyErr_Occurred() || !q || !len || dev != current()) return none();
        const at::ScalarType ty = q->scalar_type();
        if ((ty != at::kBFloat16 && ty != at::kHalf) || !plain(*q, ty, (int)dev) || q->dim() != 4 ||
            q->size(0) != B || q->size(3) != kc->D || q->numel() == 0 || !plain(*len, at::kInt, (int)dev) ||
            len->dim() != 1 || len->size(0) != B)
            return none();
        const float scale = a[5] == Py_None ? (float)(1.0 / std::sqrt((double)kc->D)) : (float)PyFloat_AsDouble(a[5]);
        const float cap = (float)PyFloat_AsDouble(a[6]);
        const long window = PyLong_AsLong(a[7]);
        if (PyErr_Occurred() || window > 0x7fffffffL || window < -0x7fffffffL) return none();
        const size_t bytes = fa_fwd_kvcache_workspace_bytes(kc->D);
        if (bytes == 0) return none();
        at::Tensor o = at::empty(q->sizes(), q->options());
        at::Tensor lse = at::empty({q->size(0), q->size(2), q->size(1)}, q->options().dtype(at::kFloat));
        at::Tensor ws = at::empty({(int64_t)bytes}, q->options().dtype(at::kByte));
        const fa_status st =
            fa_fwd_kvcache(q->data_ptr(), kc, (const int *)len->data_ptr(), o.data_ptr(), (float *)lse.data_ptr(),
                           (int)B, (int)q->size(1), (int)q->size(2), scale, cap, (int)window,
                           ty == at::kBFloat16 ? FA_BF16 : FA_FP16, ws.data_ptr(), bytes, stream((int)dev));
        return st == FA_OK ? pair(std::move(o), std::move(lse)) : PyLong_FromLong(st);
    });
}

#define FN(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FN(agree), FN(fwd), FN(bwd), FN(mask_ranges), FN(cache), FN(append), FN(attend), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&module); }
