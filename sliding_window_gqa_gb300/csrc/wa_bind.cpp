// wa_bind.cpp — the drafted-token calls' short way from Python to the C ABI.
//
// A call for one sequence runs for five to twenty microseconds on the GPU, and the checks of its tensors as
// Python expressions took as long again.  This module does them on the tensors themselves (under a
// microsecond) for the ordinary call: contiguous tensors of the right types on the current device, its current
// stream.  For any other call, valid or not, each function returns None and the package's own checks, which name
// what is wrong, take it from there.  On success a function returns the call's tensors, and a WA_E* code as an
// int where the library refused it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "wa.h"

namespace {

using at::Tensor;

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// An ordinary tensor: contiguous, of this type, on CUDA device `dev`.
bool plain(const Tensor* t, at::ScalarType type, int64_t dev) {
    return t && t->defined() && t->is_cuda() && t->scalar_type() == type && t->get_device() == dev && t->is_contiguous();
}

bool sized(const Tensor* t, std::initializer_list<int64_t> want) { return t->sizes() == at::IntArrayRef(want.begin(), want.size()); }

PyObject* none() { Py_RETURN_NONE; }

// Runs `f` (which returns a new reference) with any C++ or Python error turned into None, and none left set: a
// conversion that failed (win = 1024.0) leaves one behind although f has returned.
template <class F>
PyObject* guarded(F&& f) {
    PyObject* r = nullptr;
    try {
        r = f();
    } catch (...) {
        r = nullptr;
    }
    if (!r || PyErr_Occurred()) {
        Py_XDECREF(r);
        PyErr_Clear();
        return none();
    }
    return r;
}

Tensor make(at::IntArrayRef sizes, at::ScalarType type, const Tensor& like) {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

// The caller's workspace, if it is an ordinary byte buffer, or a new one.
bool workspace(PyObject* o, size_t bytes, const Tensor& like, Tensor& ws) {
    if (o == Py_None) {
        ws = make({static_cast<int64_t>(bytes < 256 ? 256 : bytes)}, at::kByte, like);
        return true;
    }
    const Tensor* t = tensor(o);
    if (!plain(t, at::kByte, like.get_device())) return false;
    ws = *t;
    return true;
}

// tree_decode(q, k_ring, v_ring, k_tree, v_tree, pos, parent, win, n, scale, out, ws)
PyObject* tree_decode(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject* {
        if (nargs != 12) return none();
        const Tensor *q = tensor(arg[0]), *k = tensor(arg[1]), *v = tensor(arg[2]), *kt = tensor(arg[3]), *vt = tensor(arg[4]),
                     *pos = tensor(arg[5]), *parent = tensor(arg[6]);
        if (!q || !q->defined() || !q->is_cuda() || q->dim() != 4 || !k || !k->defined() || k->dim() != 4) return none();
        const int64_t dev = q->get_device(), rows = q->size(0), nodes = q->size(1), hq = q->size(2), d = q->size(3);
        const int64_t ring = k->size(1), hkv = k->size(2);
        for (const Tensor* t : {q, k, v, kt, vt})
            if (!plain(t, at::kBFloat16, dev)) return none();
        if (!plain(pos, at::kInt, dev) || !plain(parent, at::kInt, dev)) return none();
        if (!sized(k, {rows, ring, hkv, d}) || !sized(v, {rows, ring, hkv, d}) || !sized(kt, {rows, nodes, hkv, d}) ||
            !sized(vt, {rows, nodes, hkv, d}) || !sized(pos, {rows}) || !sized(parent, {rows, nodes}))
            return none();
        for (int64_t x : {rows, nodes, hq, d, ring, hkv})
            if (x > INT32_MAX) return none();
        const Tensor* n = arg[8] == Py_None ? nullptr : tensor(arg[8]);
        if (arg[8] != Py_None && (!plain(n, at::kInt, dev) || !sized(n, {rows}))) return none();
        const long win = PyLong_AsLong(arg[7]);
        const double scale = PyFloat_AsDouble(arg[9]);
        if (PyErr_Occurred() || win < INT32_MIN || win > INT32_MAX) return none();
        if (dev != c10::cuda::current_device()) return none();
        Tensor out, ws;
        if (arg[10] == Py_None) {
            out = make(q->sizes(), at::kBFloat16, *q);
        } else {
            const Tensor* o = tensor(arg[10]);
            if (!plain(o, at::kBFloat16, dev) || o->sizes() != q->sizes()) return none();
            out = *o;
        }
        const size_t need = wa_tree_decode_ws_bytes(rows, nodes, hq, hkv, d, win, ring);
        if (!workspace(arg[11], need, *q, ws)) return none();
        int rc;
        cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev).stream();
        Py_BEGIN_ALLOW_THREADS
        rc = wa_tree_decode(q->data_ptr(), k->data_ptr(), v->data_ptr(), kt->data_ptr(), vt->data_ptr(),
                            static_cast<const int32_t*>(pos->data_ptr()), static_cast<const int32_t*>(parent->data_ptr()),
                            n ? static_cast<const int32_t*>(n->data_ptr()) : nullptr, rows, nodes, hq, hkv, d, win, ring,
                            static_cast<float>(scale), nullptr, out.data_ptr(), ws.data_ptr(), ws.numel(), s);
        Py_END_ALLOW_THREADS
        if (rc != WA_OK) return PyLong_FromLong(rc);
        if (arg[10] != Py_None) {
            Py_INCREF(arg[10]);
            return arg[10];
        }
        return THPVariable_Wrap(std::move(out));
    });
}

// tree_verify(target, parent, tokens, u, draft, n, ws) -> (path, length, token)
PyObject* tree_verify(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject* {
        if (nargs != 7) return none();
        const Tensor *target = tensor(arg[0]), *parent = tensor(arg[1]), *tokens = tensor(arg[2]), *u = tensor(arg[3]);
        if (!target || !target->defined() || !target->is_cuda() || target->dim() != 3) return none();
        const int64_t dev = target->get_device(), rows = target->size(0), nodes = target->size(1), vocab = target->size(2);
        for (int64_t x : {rows, nodes, vocab})
            if (x > INT32_MAX) return none();
        const Tensor* draft = arg[4] == Py_None ? nullptr : tensor(arg[4]);
        const Tensor* n = arg[5] == Py_None ? nullptr : tensor(arg[5]);
        if (!plain(target, at::kFloat, dev) || !plain(parent, at::kInt, dev) || !plain(tokens, at::kInt, dev) ||
            !plain(u, at::kFloat, dev) || !sized(parent, {rows, nodes}) || !sized(tokens, {rows, nodes}) || !sized(u, {rows, nodes}))
            return none();
        if (arg[4] != Py_None && (!plain(draft, at::kFloat, dev) || draft->sizes() != target->sizes())) return none();
        if (arg[5] != Py_None && (!plain(n, at::kInt, dev) || !sized(n, {rows}))) return none();
        if (dev != c10::cuda::current_device()) return none();
        Tensor ws;
        if (!workspace(arg[6], WA_TREE_WS_BYTES, *target, ws)) return none();
        Tensor path = make({rows, nodes}, at::kInt, *target), length = make({rows}, at::kInt, *target),
               token = make({rows}, at::kInt, *target);
        int rc;
        cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev).stream();
        Py_BEGIN_ALLOW_THREADS
        rc = wa_tree_verify(static_cast<const float*>(target->data_ptr()), draft ? static_cast<const float*>(draft->data_ptr()) : nullptr,
                            static_cast<const int32_t*>(parent->data_ptr()), static_cast<const int32_t*>(tokens->data_ptr()),
                            n ? static_cast<const int32_t*>(n->data_ptr()) : nullptr, static_cast<const float*>(u->data_ptr()), rows,
                            nodes, vocab, nullptr, static_cast<int32_t*>(path.data_ptr()), static_cast<int32_t*>(length.data_ptr()),
                            static_cast<int32_t*>(token.data_ptr()), ws.data_ptr(), ws.numel(), s);
        Py_END_ALLOW_THREADS
        if (rc != WA_OK) return PyLong_FromLong(rc);
        return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(path)), THPVariable_Wrap(std::move(length)),
                             THPVariable_Wrap(std::move(token)));
    });
}

// The tensors of one argument of tree_commit: a tensor, or a list or tuple of them.  False: something else.
bool layers(PyObject* o, const Tensor* (&t)[WA_COMMIT_MAX_LAYERS], int& count) {
    PyObject* const* item = &o;
    Py_ssize_t size = 1;
    if (PyList_Check(o) || PyTuple_Check(o)) {
        size = PySequence_Fast_GET_SIZE(o);
        item = PySequence_Fast_ITEMS(o);
    }
    if (size < 1 || size > WA_COMMIT_MAX_LAYERS) return false;
    for (Py_ssize_t i = 0; i < size; ++i)
        if (!(t[i] = tensor(item[i])) || !t[i]->defined()) return false;
    count = static_cast<int>(size);
    return true;
}

// tree_commit(k_tree, v_tree, k_ring, v_ring, path, length, pos, ws) -> ws
PyObject* tree_commit(PyObject*, PyObject* const* arg, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject* {
        if (nargs != 8) return none();
        const Tensor* t[4][WA_COMMIT_MAX_LAYERS];
        int count[4];
        for (int i = 0; i < 4; ++i)
            if (!layers(arg[i], t[i], count[i]) || count[i] != count[0]) return none();
        const int L = count[0];
        const Tensor &first = *t[0][0], *path = tensor(arg[4]), *length = tensor(arg[5]), *pos = tensor(arg[6]);
        if (!first.is_cuda() || first.dim() != 4 || !path || !path->defined() || path->dim() != 2) return none();
        const int64_t dev = first.get_device(), rows = first.size(0), nodes = first.size(1), hkv = first.size(2), d = first.size(3);
        const int64_t most = path->size(1);
        for (int64_t x : {rows, nodes, hkv, d, most})
            if (x > INT32_MAX) return none();
        void* p[4][WA_COMMIT_MAX_LAYERS];
        int32_t ring[WA_COMMIT_MAX_LAYERS];
        for (int l = 0; l < L; ++l) {
            for (int i = 0; i < 4; ++i) {
                if (!plain(t[i][l], at::kBFloat16, dev) || t[i][l]->dim() != 4) return none();
                p[i][l] = t[i][l]->data_ptr();
            }
            const int64_t slots = t[2][l]->size(1);
            if (slots > INT32_MAX || t[0][l]->sizes() != first.sizes() || t[1][l]->sizes() != first.sizes() ||
                !sized(t[2][l], {rows, slots, hkv, d}) || !sized(t[3][l], {rows, slots, hkv, d}))
                return none();
            ring[l] = static_cast<int32_t>(slots);
        }
        if (!plain(path, at::kInt, dev) || !plain(length, at::kInt, dev) || !plain(pos, at::kInt, dev) ||
            !sized(path, {rows, most}) || !sized(length, {rows}) || !sized(pos, {rows}))
            return none();
        if (dev != c10::cuda::current_device()) return none();
        Tensor ws;
        if (!workspace(arg[7], WA_TREE_WS_BYTES, first, ws)) return none();
        int rc;
        cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev).stream();
        Py_BEGIN_ALLOW_THREADS
        rc = wa_tree_commit(L, p[0], p[1], p[2], p[3], ring, rows, nodes, hkv, d, nullptr, static_cast<const int32_t*>(path->data_ptr()),
                            most, static_cast<const int32_t*>(length->data_ptr()), static_cast<const int32_t*>(pos->data_ptr()),
                            ws.data_ptr(), ws.numel(), s);
        Py_END_ALLOW_THREADS
        if (rc != WA_OK) return PyLong_FromLong(rc);
        if (arg[7] != Py_None) {
            Py_INCREF(arg[7]);
            return arg[7];
        }
        return THPVariable_Wrap(std::move(ws));
    });
}

PyMethodDef methods[] = {
    {"tree_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree_decode)), METH_FASTCALL, nullptr},
    {"tree_verify", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree_verify)), METH_FASTCALL, nullptr},
    {"tree_commit", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree_commit)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "wa_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `built_for`: the PyTorch and Python whose headers this was compiled against; the package uses it with no others.
PyMODINIT_FUNC PyInit_wa_bind() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", WA_BIND_FOR) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
