// binding.cpp -- the Python calls of the rotated appends and of the 4-bit attention, as a CPython module.
//
// These calls take a few microseconds on the GPU (one decode step of an append: two), so their host
// side counts: checking and marshalling a dozen tensors costs 8 us in Python and 4 us more through
// ctypes, about 1 us here. The module only checks arguments, takes PyTorch memory for outputs that the
// caller does not give, and calls the C ABI (include/kvdecode.h) on the current stream; the functions
// of the same names in the package's __init__.py document them.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kvdecode.h"

namespace {

PyObject* g_error = nullptr;  // the package's KvdError(status, where)

struct Refused {  // an argument that is not what the call needs
    PyObject* type;
    std::string what;
};
[[noreturn]] void type_error(const std::string& what) { throw Refused{PyExc_TypeError, what}; }
[[noreturn]] void value_error(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

std::string list(c10::IntArrayRef s) {
    std::ostringstream o;
    o << s;
    return o.str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        type_error(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

// The type, shape and device that the call's leading tensor sets or follows from it.
void check(const at::Tensor& t, const char* name, int dev, at::ScalarType dtype,
           c10::IntArrayRef shape) {
    if (t.scalar_type() != dtype)
        type_error(std::string(name) + " must be " + c10::toString(dtype) + ", got " +
                   c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
        value_error(std::string(name) + " must be " + list(shape) + ", got " + list(t.sizes()));
    if (t.get_device() != dev)
        value_error(std::string(name) + " must be on the device of the other tensors");
}

// A dense tensor's address; null for None where that is allowed.
void* dense(PyObject* o, const char* name, int dev, at::ScalarType dtype, c10::IntArrayRef shape) {
    const at::Tensor& t = tensor(o, name);
    check(t, name, dev, dtype, shape);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return t.data_ptr();
}
void* dense_or_null(PyObject* o, const char* name, int dev, at::ScalarType dtype,
                    c10::IntArrayRef shape) {
    return o == Py_None ? nullptr : dense(o, name, dev, dtype, shape);
}

// [T, H, D] with dense heads: address, and elements between tokens.
void* tokens(PyObject* o, const char* name, int dev, at::ScalarType dtype, c10::IntArrayRef shape,
             long long* stride) {
    const at::Tensor& t = tensor(o, name);
    check(t, name, dev, dtype, shape);
    const int64_t T = shape[0], H = shape[1], D = shape[2];
    if (t.numel() && (t.stride(2) != 1 || (H > 1 && t.stride(1) != D)))
        value_error(std::string(name) + " must have dense heads (strides " + std::to_string(D) +
                    ", 1 in a token)");
    *stride = T > 1 ? t.stride(0) : H * D;
    return t.data_ptr();
}

int dtype_of(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kFloat) return KVD_F32;
    if (t.scalar_type() == at::kBFloat16) return KVD_BF16;
    type_error(std::string(name) + " must be float32 or bfloat16");
}

// Sizes are int in the C ABI.
int narrow(int64_t x, const char* what) {
    if (x < 0 || x > INT32_MAX) value_error(std::string(what) + " is out of range");
    return static_cast<int>(x);
}
int integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};  // the error is set
    if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " is out of range");
    return static_cast<int>(v);
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{nullptr, ""};
    return v != 0;
}

// Page size of a 4-bit pool [num_pages, Hkv, page bytes]; 0 if it is none.
int64_t q4_page_size(const at::Tensor& pool, int64_t D) {
    if (pool.dim() != 3 || (D != 64 && D != 128)) return 0;
    const int64_t per = D / 2 + D / 16, bytes = pool.size(2);
    return bytes % per == 0 ? bytes / per : 0;
}

// The stream of the call: a handle, or the device's current one.
cudaStream_t stream_of(PyObject* o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev));
    const unsigned long long h = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) throw Refused{nullptr, ""};
    return reinterpret_cast<cudaStream_t>(h);
}

template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Refused& r) {
        if (r.type) PyErr_SetString(r.type, r.what.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject* failed(int status, const char* where) {
    PyObject* e = PyObject_CallFunction(g_error, "is", status, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

// rope_append(q4, q, k_new, v_new, cos_sin, k_pool, v_pool, block_table, seq_lens, cu_seqlens, window,
//             n_sink, interleaved, q_out, k_out, v_out, err, stream) -> q_out or None
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 18) type_error("rope_append takes 18 arguments");
        const bool q4 = truth(a[0]);
        const at::Tensor& k = tensor(a[2], "k_new");
        if (k.dim() != 3) value_error("k_new must be [T, Hkv, D]");
        const int dtype = dtype_of(k, "k_new");
        const at::ScalarType dt = k.scalar_type();
        const int dev = static_cast<int>(k.get_device());
        const int64_t T = k.size(0), Hkv = k.size(1), D = k.size(2);
        const at::Tensor& pool = tensor(a[5], "k_pool");
        const at::ScalarType pool_dt = q4 ? at::kByte : dt;
        if (pool.scalar_type() != pool_dt)
            type_error(std::string("k_pool must be ") + c10::toString(pool_dt) + ", got " +
                       c10::toString(pool.scalar_type()));
        const int64_t P = q4 ? q4_page_size(pool, D) : pool.dim() == 4 ? pool.size(2) : 0;
        if (P < 1 || pool.size(1) != Hkv || (!q4 && pool.size(3) != D))
            value_error(q4 ? "k_pool must be [num_pages, Hkv, q4_page_bytes(page_size, D)]"
                           : "k_pool must be [num_pages, Hkv, page_size, D]");
        const at::Tensor& bt = tensor(a[7], "block_table");
        const at::Tensor& cs = tensor(a[4], "cos_sin");
        if (bt.dim() != 2) value_error("block_table must have 2 dims");
        if (cs.dim() != 2) value_error("cos_sin must have 2 dims");
        const int64_t B = bt.size(0);
        long long qs = 0, ks = 0, vs = 0;
        void* kp = tokens(a[2], "k_new", dev, dt, k.sizes(), &ks);
        void* vp = tokens(a[3], "v_new", dev, dt, k.sizes(), &vs);
        void *qp = nullptr, *qo = nullptr;
        int64_t Hq = 0;
        at::Tensor made;
        if (a[1] != Py_None) {
            const at::Tensor& q = tensor(a[1], "q");
            if (q.dim() != 3) value_error("q must be [T, Hq, D]");
            Hq = q.size(1);
            const int64_t shape[3] = {T, Hq, D};
            qp = tokens(a[1], "q", dev, dt, shape, &qs);
            if (a[13] == Py_None) {
                made = at::empty(shape, q.options());
                qo = made.data_ptr();
            } else {
                qo = dense(a[13], "q_out", dev, dt, shape);
            }
        } else if (a[13] != Py_None) {
            value_error("q_out needs q");
        }
        if (a[9] == Py_None && T != B)
            value_error("without cu_seqlens there is one token of each sequence");
        const int32_t* cu =
            static_cast<const int32_t*>(dense_or_null(a[9], "cu_seqlens", dev, at::kInt, {B + 1}));
        const float* csp =
            static_cast<const float*>(dense(a[4], "cos_sin", dev, at::kFloat, cs.sizes()));
        const int32_t* btp =
            static_cast<const int32_t*>(dense(a[7], "block_table", dev, at::kInt, bt.sizes()));
        const int32_t* sl =
            static_cast<const int32_t*>(dense(a[8], "seq_lens", dev, at::kInt, {B}));
        void* kpool = dense(a[5], "k_pool", dev, pool_dt, pool.sizes());
        void* vpool = dense(a[6], "v_pool", dev, pool_dt, pool.sizes());
        int* err = static_cast<int*>(dense_or_null(a[16], "err", dev, at::kInt, {1}));
        const int b = narrow(B, "B"), t = narrow(T, "T"), hq = narrow(Hq, "Hq"),
                  hkv = narrow(Hkv, "Hkv"), d = narrow(D, "D"), rot = narrow(cs.size(1), "rot_dim"),
                  max_pos = narrow(cs.size(0), "positions"), ps = narrow(P, "page_size"),
                  mp = narrow(bt.size(1), "max_pages"), np = narrow(pool.size(0), "num_pages"),
                  window = integer(a[10], "window"), n_sink = integer(a[11], "n_sink");
        const int inter = truth(a[12]);
        const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(dev));
        const cudaStream_t stream = stream_of(a[17], dev);
        int st;
        if (q4) {
            void* ko = dense_or_null(a[14], "k_out", dev, dt, k.sizes());
            void* vo = dense_or_null(a[15], "v_out", dev, dt, k.sizes());
            st = kvd_rope_append_q4(qp, kp, vp, csp, cu, btp, sl, qo, kpool, vpool, ko, vo, b, t,
                                    hq, hkv, d, qs, ks, vs, rot, inter, max_pos, ps, mp, np, dtype,
                                    window, n_sink, err, stream);
        } else {
            st = kvd_rope_append(qp, kp, vp, csp, cu, btp, sl, qo, kpool, vpool, b, t, hq, hkv, d,
                                 qs, ks, vs, rot, inter, max_pos, ps, mp, np, dtype, window, n_sink,
                                 err, stream);
        }
        if (st != KVD_OK) return failed(st, q4 ? "kvd_rope_append_q4" : "kvd_rope_append");
        if (made.defined()) return THPVariable_Wrap(made);
        return Py_NewRef(a[13]);
    });
}

// attn_decode_gqa_q4(q, k_pool, v_pool, block_table, seq_lens, window, n_sink_tokens, ring, sink_logit,
//                    scale, out, lse_out, workspace, err, stream) -> out
PyObject* attn_decode_gqa_q4_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 15) type_error("attn_decode_gqa_q4 takes 15 arguments");
        const at::Tensor& q = tensor(a[0], "q");
        if (q.dim() != 3) value_error("q must be [B, Hq, D]");
        const int dtype = dtype_of(q, "q");
        const at::ScalarType dt = q.scalar_type();
        const int dev = static_cast<int>(q.get_device());
        const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
        const at::Tensor& pool = tensor(a[1], "k_pool");
        if (pool.scalar_type() != at::kByte)
            type_error(std::string("k_pool must be ") + c10::toString(at::kByte) + ", got " +
                       c10::toString(pool.scalar_type()));
        const int64_t P = q4_page_size(pool, D);
        if (P < 1) value_error("k_pool must be [num_pages, Hkv, q4_page_bytes(page_size, D)]");
        const at::Tensor& bt = tensor(a[3], "block_table");
        if (bt.dim() != 2) value_error("block_table must have 2 dims");
        const int64_t max_pages = bt.size(1);
        const void* qp = dense(a[0], "q", dev, dt, q.sizes());
        const void* kp = dense(a[1], "k_pool", dev, at::kByte, pool.sizes());
        const void* vp = dense(a[2], "v_pool", dev, at::kByte, pool.sizes());
        const int32_t* btp = static_cast<const int32_t*>(
            dense(a[3], "block_table", dev, at::kInt, {B, max_pages}));
        const int32_t* sl =
            static_cast<const int32_t*>(dense(a[4], "seq_lens", dev, at::kInt, {B}));
        const float* sink = static_cast<const float*>(
            dense_or_null(a[8], "sink_logit", dev, at::kFloat, {Hq}));
        float* lse =
            static_cast<float*>(dense_or_null(a[11], "lse_out", dev, at::kFloat, {B, Hq}));
        int* err = static_cast<int*>(dense_or_null(a[13], "err", dev, at::kInt, {1}));
        const int b = narrow(B, "B"), hq = narrow(Hq, "Hq"), hkv = narrow(pool.size(1), "Hkv"),
                  d = narrow(D, "D"), ps = narrow(P, "page_size"),
                  mp = narrow(max_pages, "max_pages"), np = narrow(pool.size(0), "num_pages"),
                  window = integer(a[5], "window"), n_sink = integer(a[6], "n_sink_tokens");
        const int ring = truth(a[7]);
        double scale = 1.0 / std::sqrt(static_cast<double>(D));
        if (a[9] != Py_None) {
            scale = PyFloat_AsDouble(a[9]);
            if (scale == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
        }
        at::Tensor made, ws;
        void* out;
        if (a[10] == Py_None) {
            made = at::empty(q.sizes(), q.options());
            out = made.data_ptr();
        } else {
            out = dense(a[10], "out", dev, dt, q.sizes());
        }
        if (a[12] == Py_None) {
            size_t bytes = 0;
            if (static_cast<int64_t>(mp) * ps <= INT32_MAX)
                bytes = kvd_workspace_size(KVD_OP_GQA_Q4, b, hq, hkv, d, mp * ps, 0, 0, 0);
            // (a shape that the call refuses needs none)
            ws = at::empty({static_cast<int64_t>(bytes > 0 ? bytes : 1)}, pool.options());
        } else {
            ws = tensor(a[12], "workspace");
            dense(a[12], "workspace", dev, at::kByte, {ws.numel()});
        }
        const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(dev));
        const int st = attn_decode_gqa_q4(qp, kp, vp, btp, sl, out, lse, b, hq, hkv, d, ps, mp, np,
                                          static_cast<float>(scale), dtype, window, n_sink, ring,
                                          sink, ws.data_ptr(), static_cast<size_t>(ws.numel()), err,
                                          stream_of(a[14], dev));
        if (st != KVD_OK) return failed(st, "attn_decode_gqa_q4");
        if (made.defined()) return THPVariable_Wrap(made);
        return Py_NewRef(a[10]);
    });
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_XSETREF(g_error, Py_NewRef(type));
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(rope_append)),
     METH_FASTCALL, nullptr},
    {"attn_decode_gqa_q4",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(attn_decode_gqa_q4_py)),
     METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&module);
    // the PyTorch whose tensors this module can read (build.py gives it): the package compares
    if (m && PyModule_AddStringConstant(m, "built_for", KVD_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
