// marshal.cpp -- the serving-step calls from torch tensors to the C ABI, as a
// CPython module.
//
// These calls run for 4 to 8 us on the GPU at the sizes of a decode step and
// pass up to sixteen tensors each; described one by one in Python they take
// 20 us of host time.  Here a call takes about 3.  Nothing but marshalling
// happens: arguments are checked as the Python path checks them (binding.py),
// every other check and all work is the library's.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <dlfcn.h>
#include <stdint.h>

#include <exception>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "spd.h"

namespace {

decltype(&paged_assign_slots) p_assign = nullptr;
decltype(&paged_norm_rope_store) p_store = nullptr;
decltype(&paged_prefill_attention) p_dense = nullptr;
decltype(&paged_sparse_prefill_attention) p_sparse = nullptr;
decltype(&paged_norm_rope_store_block_scaled) p_store_bs = nullptr;
decltype(&paged_decode_attention_block_scaled) p_decode_bs = nullptr;
decltype(&paged_sparse_decode_attention_block_scaled) p_sparse_decode_bs = nullptr;
decltype(&paged_prefill_attention_block_scaled) p_dense_bs = nullptr;
decltype(&paged_sparse_prefill_attention_block_scaled) p_sparse_bs = nullptr;
decltype(&spd_last_error) p_error = nullptr;
PyObject *raise_last = nullptr;  // Python callable that raises the library's last error

int dtype_code(c10::ScalarType t) {
    switch (t) {
    case c10::ScalarType::Float: return SPD_F32;
    case c10::ScalarType::BFloat16: return SPD_BF16;
    case c10::ScalarType::Half: return SPD_F16;
    case c10::ScalarType::Float8_e4m3fn: return SPD_E4M3;
    case c10::ScalarType::Int: return SPD_I32;
    default: return -1;
    }
}

// The arguments of one call, taken in order; a failed take leaves a Python
// error and makes the later ones do nothing.
struct Args {
    PyObject *const *a;
    Py_ssize_t n, at = 0;
    int device;
    bool ok = true;
    spd_tensor d[16];
    int used = 0;

    Args(PyObject *const *args, Py_ssize_t count, Py_ssize_t want) : a(args), n(count) {
        if (count != want) {
            PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, count);
            ok = false;
        }
        device = c10::cuda::device_count() > 0 ? static_cast<int>(c10::cuda::current_device()) : -2;
    }

    const spd_tensor *tensor(const char *name) {
        if (!ok) return nullptr;
        PyObject *o = a[at++];
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) return fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
        const at::Tensor &t = THPVariable_Unpack(o);
        const int code = dtype_code(t.scalar_type());
        if (code < 0) return fail(PyExc_TypeError, "%s: its dtype is not supported by libspd", name);
        const int64_t dims = t.dim();
        if (dims > 4) return fail(PyExc_ValueError, "%s has more than 4 dims", name);
        if (t.numel() > 0 && (!t.is_cuda() || t.get_device() != device))
            return fail(PyExc_ValueError, "%s must be a CUDA tensor on the current device", name);
        spd_tensor &x = d[used++];
        x.data = t.numel() > 0 ? t.data_ptr() : nullptr;
        x.dtype = code;
        x.ndim = static_cast<int32_t>(dims);
        for (int64_t i = 0; i < 4; ++i) {
            x.shape[i] = i < dims ? t.size(i) : 0;
            x.stride[i] = i < dims ? t.stride(i) : 0;
        }
        return &x;
    }

    int32_t integer() {
        if (!ok) return 0;
        const long v = PyLong_AsLong(a[at++]);
        if (v == -1 && PyErr_Occurred()) {
            ok = false;
        } else if (v < INT32_MIN || v > INT32_MAX) {
            PyErr_SetString(PyExc_OverflowError, "integer argument outside 32 bits");
            ok = false;
        }
        return static_cast<int32_t>(v);
    }

    float real() {
        if (!ok) return 0.f;
        const double v = PyFloat_AsDouble(a[at++]);
        if (v == -1.0 && PyErr_Occurred()) ok = false;
        return static_cast<float>(v);
    }

    void *workspace(size_t *bytes) {
        *bytes = 0;
        if (!ok) return nullptr;
        PyObject *o = a[at++];
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda() || THPVariable_Unpack(o).get_device() != device) {
            fail(PyExc_TypeError, "%s must be a CUDA tensor on the current device", "workspace");
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_contiguous()) {  // its bytes are used as one run
            fail(PyExc_ValueError, "%s must be contiguous", "workspace");
            return nullptr;
        }
        *bytes = t.nbytes();
        return t.data_ptr();
    }

    spd_stream_t stream() {
        if (!ok) return nullptr;
        PyObject *o = a[at++];
        if (o == Py_None)
            return device >= 0 ? reinterpret_cast<spd_stream_t>(c10::cuda::getCurrentCUDAStream().stream()) : nullptr;
        const unsigned long long v = PyLong_AsUnsignedLongLong(o);
        if (PyErr_Occurred()) ok = false;
        return reinterpret_cast<spd_stream_t>(v);
    }

    const spd_tensor *fail(PyObject *type, const char *format, const char *name) {
        PyErr_Format(type, format, name);
        ok = false;
        return nullptr;
    }
};

PyObject *done() {
    if (p_error(nullptr, 0) != 0) return PyObject_CallNoArgs(raise_last);
    Py_RETURN_NONE;
}

template <typename F>
PyObject *guarded(F &&f) {
    if (p_error == nullptr) {
        PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
        return nullptr;
    }
    try {
        return f();
    } catch (const std::exception &e) {  // a tensor without storage, and the like
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject *assign(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Args x(a, n, 17);
        const auto *nw = x.tensor("new_lens"), *pre = x.tensor("prefix_lens"), *sid = x.tensor("slot_ids"),
                   *fp = x.tensor("free_pages"), *fc = x.tensor("free_count");
        const int32_t pages = x.integer(), bs = x.integer(), bq = x.integer();
        const auto *bt = x.tensor("block_table"), *cu = x.tensor("cu_seqlens"), *cub = x.tensor("cu_seqblocks_q"),
                   *sl = x.tensor("seq_lens"), *req = x.tensor("req_idx"), *tl = x.tensor("token_lens"),
                   *slots = x.tensor("slots"), *left = x.tensor("free_left");
        const spd_stream_t s = x.stream();
        if (!x.ok) return nullptr;
        p_assign(nw, pre, sid, fp, fc, pages, bs, bq, bt, cu, cub, sl, req, tl, slots, left, s);
        return done();
    });
}

PyObject *store(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Args x(a, n, 17);
        const auto *q = x.tensor("q"), *k = x.tensor("k"), *v = x.tensor("v"), *wq = x.tensor("q_weight"),
                   *wk = x.tensor("k_weight"), *cs = x.tensor("cos_sin"), *tl = x.tensor("token_lens"),
                   *slots = x.tensor("slots"), *qo = x.tensor("q_out"), *kc = x.tensor("k_cache"), *vc = x.tensor("v_cache");
        const float eps = x.real();
        const int32_t inter = x.integer(), bs = x.integer();
        const float ks = x.real(), vs = x.real();
        const spd_stream_t s = x.stream();
        if (!x.ok) return nullptr;
        p_store(q, k, v, wq, wk, cs, tl, slots, qo, kc, vc, eps, inter, bs, ks, vs, s);
        return done();
    });
}

PyObject *attention(PyObject *const *a, Py_ssize_t n, bool sparse) {
    return guarded([&]() -> PyObject * {
        Args x(a, n, sparse ? 18 : 15);
        const auto *q = x.tensor("q"), *k = x.tensor("k_cache"), *v = x.tensor("v_cache"), *bt = x.tensor("block_table"),
                   *sid = x.tensor("slot_ids"), *cu = x.tensor("cu_seqlens"), *sl = x.tensor("seq_lens"),
                   *pre = x.tensor("prefix_lens");
        const spd_tensor *tk = nullptr, *cub = nullptr;
        int32_t bq = 0;
        if (sparse) {
            tk = x.tensor("topk_idx");
            bq = x.integer();
            cub = x.tensor("cu_seqblocks_q");
        }
        const auto *out = x.tensor("out");
        const float sm = x.real();
        const int32_t bs = x.integer();
        const float ks = x.real(), vs = x.real();
        size_t bytes = 0;
        void *ws = x.workspace(&bytes);
        const spd_stream_t s = x.stream();
        if (!x.ok) return nullptr;
        if (sparse) p_sparse(q, k, v, bt, sid, cu, sl, pre, tk, bq, cub, out, sm, bs, ks, vs, ws, bytes, s);
        else p_dense(q, k, v, bt, sid, cu, sl, pre, out, sm, bs, ks, vs, ws, bytes, s);
        return done();
    });
}

PyObject *dense_attention(PyObject *, PyObject *const *a, Py_ssize_t n) { return attention(a, n, false); }
PyObject *sparse_attention(PyObject *, PyObject *const *a, Py_ssize_t n) { return attention(a, n, true); }

PyObject *store_block(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Args x(a, n, 17);
        const auto *q = x.tensor("q"), *k = x.tensor("k"), *v = x.tensor("v"), *wq = x.tensor("q_weight"),
                   *wk = x.tensor("k_weight"), *cs = x.tensor("cos_sin"), *tl = x.tensor("token_lens"),
                   *slots = x.tensor("slots"), *qo = x.tensor("q_out"), *kc = x.tensor("k_cache"),
                   *vc = x.tensor("v_cache"), *ks = x.tensor("k_scales"), *vs = x.tensor("v_scales");
        const float eps = x.real();
        const int32_t inter = x.integer(), bs = x.integer();
        const spd_stream_t s = x.stream();
        if (!x.ok) return nullptr;
        p_store_bs(q, k, v, wq, wk, cs, tl, slots, qo, kc, vc, ks, vs, eps, inter, bs, s);
        return done();
    });
}

PyObject *decode_block(PyObject *const *a, Py_ssize_t n, bool sparse) {
    return guarded([&]() -> PyObject * {
        Args x(a, n, sparse ? 14 : 13);
        const auto *q = x.tensor("q"), *k = x.tensor("k_cache"), *v = x.tensor("v_cache"), *ks = x.tensor("k_scales"),
                   *vs = x.tensor("v_scales"), *bt = x.tensor("block_table"), *sl = x.tensor("seq_lens"),
                   *ri = x.tensor("req_idx");
        const spd_tensor *tk = sparse ? x.tensor("topk_idx") : nullptr;
        const auto *out = x.tensor("out");
        const float sm = x.real();
        const int32_t bs = x.integer();
        size_t bytes = 0;
        void *ws = x.workspace(&bytes);
        const spd_stream_t s = x.stream();
        if (!x.ok) return nullptr;
        if (sparse) p_sparse_decode_bs(q, k, v, ks, vs, bt, sl, ri, tk, out, sm, bs, ws, bytes, s);
        else p_decode_bs(q, k, v, ks, vs, bt, sl, ri, out, sm, bs, ws, bytes, s);
        return done();
    });
}

PyObject *attention_block(PyObject *const *a, Py_ssize_t n, bool sparse) {
    return guarded([&]() -> PyObject * {
        Args x(a, n, sparse ? 18 : 15);
        const auto *q = x.tensor("q"), *k = x.tensor("k_cache"), *v = x.tensor("v_cache"), *ks = x.tensor("k_scales"),
                   *vs = x.tensor("v_scales"), *bt = x.tensor("block_table"), *sid = x.tensor("slot_ids"),
                   *cu = x.tensor("cu_seqlens"), *sl = x.tensor("seq_lens"), *pre = x.tensor("prefix_lens");
        const spd_tensor *tk = nullptr, *cub = nullptr;
        int32_t bq = 0;
        if (sparse) {
            tk = x.tensor("topk_idx");
            bq = x.integer();
            cub = x.tensor("cu_seqblocks_q");
        }
        const auto *out = x.tensor("out");
        const float sm = x.real();
        const int32_t bs = x.integer();
        size_t bytes = 0;
        void *ws = x.workspace(&bytes);
        const spd_stream_t s = x.stream();
        if (!x.ok) return nullptr;
        if (sparse) p_sparse_bs(q, k, v, ks, vs, bt, sid, cu, sl, pre, tk, bq, cub, out, sm, bs, ws, bytes, s);
        else p_dense_bs(q, k, v, ks, vs, bt, sid, cu, sl, pre, out, sm, bs, ws, bytes, s);
        return done();
    });
}

PyObject *decode_block_dense(PyObject *, PyObject *const *a, Py_ssize_t n) { return decode_block(a, n, false); }
PyObject *decode_block_sparse(PyObject *, PyObject *const *a, Py_ssize_t n) { return decode_block(a, n, true); }
PyObject *attention_block_dense(PyObject *, PyObject *const *a, Py_ssize_t n) { return attention_block(a, n, false); }
PyObject *attention_block_sparse(PyObject *, PyObject *const *a, Py_ssize_t n) { return attention_block(a, n, true); }

// bind(path of libspd.so, callable that raises its last error)
PyObject *bind(PyObject *, PyObject *args) {
    const char *path = nullptr;
    PyObject *raise = nullptr;
    if (!PyArg_ParseTuple(args, "sO", &path, &raise)) return nullptr;
    void *lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (lib == nullptr) {
        PyErr_Format(PyExc_RuntimeError, "dlopen: %s", dlerror());
        return nullptr;
    }
    auto get = [&](const char *name) { return dlsym(lib, name); };
    p_assign = reinterpret_cast<decltype(p_assign)>(get("paged_assign_slots"));
    p_store = reinterpret_cast<decltype(p_store)>(get("paged_norm_rope_store"));
    p_dense = reinterpret_cast<decltype(p_dense)>(get("paged_prefill_attention"));
    p_sparse = reinterpret_cast<decltype(p_sparse)>(get("paged_sparse_prefill_attention"));
    p_store_bs = reinterpret_cast<decltype(p_store_bs)>(get("paged_norm_rope_store_block_scaled"));
    p_decode_bs = reinterpret_cast<decltype(p_decode_bs)>(get("paged_decode_attention_block_scaled"));
    p_sparse_decode_bs =
        reinterpret_cast<decltype(p_sparse_decode_bs)>(get("paged_sparse_decode_attention_block_scaled"));
    p_dense_bs = reinterpret_cast<decltype(p_dense_bs)>(get("paged_prefill_attention_block_scaled"));
    p_sparse_bs = reinterpret_cast<decltype(p_sparse_bs)>(get("paged_sparse_prefill_attention_block_scaled"));
    auto error = reinterpret_cast<decltype(p_error)>(get("spd_last_error"));
    if (!p_assign || !p_store || !p_dense || !p_sparse || !p_store_bs || !p_decode_bs || !p_sparse_decode_bs ||
        !p_dense_bs || !p_sparse_bs || !error) {
        PyErr_SetString(PyExc_RuntimeError, "libspd.so lacks a serving-step call");
        return nullptr;
    }
    Py_INCREF(raise);
    Py_XDECREF(raise_last);
    raise_last = raise;
    p_error = error;
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         FAST("paged_assign_slots", assign),
                         FAST("paged_norm_rope_store", store),
                         FAST("paged_prefill_attention", dense_attention),
                         FAST("paged_sparse_prefill_attention", sparse_attention),
                         FAST("paged_norm_rope_store_block_scaled", store_block),
                         FAST("paged_decode_attention_block_scaled", decode_block_dense),
                         FAST("paged_sparse_decode_attention_block_scaled", decode_block_sparse),
                         FAST("paged_prefill_attention_block_scaled", attention_block_dense),
                         FAST("paged_sparse_prefill_attention_block_scaled", attention_block_sparse),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
