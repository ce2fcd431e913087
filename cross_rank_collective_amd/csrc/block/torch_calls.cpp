// torch_calls.cpp -- the tensor-level block-boundary calls, natively.
//
// The kernels of a single token take 4 us and less; reading a dozen tensors'
// shapes, strides and pointers from Python and marshalling them takes 10.
// This extension module reads them from the tensors themselves.  It takes only
// calls whose tensors all fit as they are (types, shapes, devices, plain
// strides, torch's current stream or a handle) and returns the library's
// status; for anything else it returns None, and the Python code in block.py
// looks again, makes the call or raises the error.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "ptored_block.h"

namespace {

struct Misfit {};

// A call that does not fit, or that torch itself refuses.
template <typename F>
PyObject* guarded(F call) {
    try {
        return PyLong_FromLong(call());
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) throw Misfit{};
    return THPVariable_Unpack(o);
}

float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Misfit{};
    return (float)v;
}

int code_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return PTORED_F32;
        case at::kBFloat16: return PTORED_BF16;
        case at::kHalf: return PTORED_F16;
        default: throw Misfit{};
    }
}

int64_t blocks_of(int64_t cols) {
    return (cols + PTORED_CHECKPOINT_BLOCK - 1) / PTORED_CHECKPOINT_BLOCK;
}

// What a call's tensors share.
struct Group {
    int64_t rows, cols;
    at::ScalarType type;
    int device;
    int code;

    explicit Group(const at::Tensor& t) {
        if (t.dim() != 2 || !t.is_cuda()) throw Misfit{};
        rows = t.size(0);
        cols = t.size(1);
        type = t.scalar_type();
        code = code_of(type);
        device = t.get_device();
        if (rows == 0 || cols == 0) throw Misfit{};
        int current = -1;
        if (hipGetDevice(&current) != hipSuccess || current != device) throw Misfit{};
    }

    ptored_rows rows_of(const at::Tensor& t, int64_t r, int64_t c, at::ScalarType ty) const {
        if (t.scalar_type() != ty || t.dim() != 2 || t.size(0) != r || t.size(1) != c ||
            !t.is_cuda() || t.get_device() != device || t.stride(1) != 1 || t.stride(0) < c)
            throw Misfit{};
        return {t.data_ptr(), t.stride(0)};
    }
    ptored_rows mat(PyObject* o) const {
        if (o == Py_None) return {nullptr, 0};
        return rows_of(tensor(o), rows, cols, type);
    }
    void* vec(PyObject* o, int64_t n, at::ScalarType ty) const {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor(o);
        if (t.scalar_type() != ty || t.dim() != 1 || t.size(0) != n || !t.is_cuda() ||
            t.get_device() != device || t.stride(0) != 1)
            throw Misfit{};
        return t.data_ptr();
    }
    // A gate or its gradient: [D] or [G, D].
    ptored_rows gate(PyObject* o, int64_t& g) const {
        g = 0;
        if (o == Py_None) return {nullptr, 0};
        const at::Tensor& t = tensor(o);
        if (t.dim() == 1) {
            g = 1;
            return {vec(o, cols, type), cols};
        }
        if (t.dim() != 2 || t.size(0) == 0 || rows % t.size(0) != 0) throw Misfit{};
        g = t.size(0);
        return rows_of(t, g, cols, type);
    }
    ptored_checkpoint kept(PyObject* o, int64_t c) const {
        if (o == Py_None) return {nullptr, 0, nullptr, 0};
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) throw Misfit{};
        const ptored_rows q = rows_of(tensor(PyTuple_GET_ITEM(o, 0)), rows, c, at::kChar);
        const ptored_rows s = rows_of(tensor(PyTuple_GET_ITEM(o, 1)), rows, blocks_of(c), at::kByte);
        return {q.data, q.ld, s.data, s.ld};
    }
    hipStream_t stream(PyObject* o) const {
        if (o == Py_None) return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
        void* p = PyLong_AsVoidPtr(o);
        if (p == nullptr && PyErr_Occurred()) throw Misfit{};
        return static_cast<hipStream_t>(p);
    }
    // post_weight, gate, pre_weight, eps, weight_offset, branch_scale, residual_scale
    ptored_block_params params(PyObject* const* a, at::ScalarType& weights) const {
        PyObject* first = a[0] != Py_None ? a[0] : a[2];
        weights = first == Py_None ? type : tensor(first).scalar_type();
        if (weights != type && weights != at::kFloat) throw Misfit{};
        ptored_block_params p{};
        p.rows = rows;
        p.cols = cols;
        p.post_weight = vec(a[0], cols, weights);
        p.pre_weight = vec(a[2], cols, weights);
        p.gate = gate(a[1], p.gate_rows);
        p.eps = number(a[3]);
        p.weight_offset = number(a[4]);
        p.branch_scale = number(a[5]);
        p.residual_scale = number(a[6]);
        p.dtype = code;
        p.weight_dtype = code_of(weights);
        return p;
    }
    // The caller's workspace, or one from torch on the current stream.
    at::Tensor workspace(PyObject* given, PyObject* stream, int64_t bytes) const {
        if (given != Py_None) {
            const at::Tensor& t = tensor(given);
            if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous()) throw Misfit{};
            return t;
        }
        if (bytes == 0) return at::Tensor();
        if (stream != Py_None) throw Misfit{};
        return at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(
                                      at::Device(at::kCUDA, (c10::DeviceIndex)device)));
    }
};

// Outputs (None, tensors or kept pairs) of a call that was made: as after torch's
// own in-place operations, autograd then finds a tensor changed that it saved
// before.
int wrote(int status, std::initializer_list<PyObject*> outputs) {
    if (status != PTORED_OK) return status;
    auto changed = [](PyObject* o) {
        const at::Tensor& t = tensor(o);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    };
    for (PyObject* o : outputs) {
        if (o == Py_None) continue;
        if (PyTuple_Check(o)) {
            changed(PyTuple_GET_ITEM(o, 0));
            changed(PyTuple_GET_ITEM(o, 1));
        } else {
            changed(o);
        }
    }
    return status;
}

void want(Py_ssize_t got, Py_ssize_t n) {
    if (got != n) throw Misfit{};
}

// parts, x, x_out, z, <params: 7>, h, post_rstd, pre_rstd, h_kept, x_kept, z_kept, stream
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 18);
        const Group g(tensor(a[1]));
        if (!PyList_Check(a[0]) && !PyTuple_Check(a[0])) throw Misfit{};
        const Py_ssize_t nranks = PySequence_Fast_GET_SIZE(a[0]);
        if (nranks > PTORED_MAX_RANKS) throw Misfit{};
        const void* parts[PTORED_MAX_RANKS];
        int64_t part_ld = g.cols;
        for (Py_ssize_t r = 0; r < nranks; ++r) {
            const ptored_rows y = g.mat(PySequence_Fast_GET_ITEM(a[0], r));
            if (r == 0) part_ld = y.ld;
            // the pitch of a single row is any
            if (y.data == nullptr || (g.rows > 1 && y.ld != part_ld)) throw Misfit{};
            parts[r] = y.data;
        }
        at::ScalarType weights;
        const ptored_block_params p = g.params(a + 4, weights);
        ptored_block_io io{};
        io.x = g.mat(a[1]);
        io.x_out = g.mat(a[2]);
        io.z = g.mat(a[3]);
        io.h = g.mat(a[11]);
        io.post_rstd = static_cast<float*>(g.vec(a[12], g.rows, at::kFloat));
        io.pre_rstd = static_cast<float*>(g.vec(a[13], g.rows, at::kFloat));
        io.h_kept = g.kept(a[14], g.cols);
        io.x_kept = g.kept(a[15], g.cols);
        io.z_kept = g.kept(a[16], g.cols);
        return wrote(ptored_block_norm(parts, (int)nranks, part_ld, &p, &io, g.stream(a[17])),
                     {a[2], a[3], a[11], a[12], a[13], a[14], a[15], a[16]});
    });
}

// dz, dx_out, x_out, pre_rstd, dx, dh, h, post_rstd, <params: 7>, dpost_weight, dgate,
// dpre_weight, workspace, stream
PyObject* block_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 20);
        const Group g(tensor(a[0] != Py_None ? a[0] : a[1]));
        at::ScalarType weights;
        const ptored_block_params p = g.params(a + 8, weights);
        ptored_block_grad_io io{};
        io.dz = g.mat(a[0]);
        io.dx_out = g.mat(a[1]);
        if (PyTuple_Check(a[2]) || PyTuple_Check(a[6])) {
            io.x_kept = g.kept(a[2], g.cols);
            io.h_kept = g.kept(a[6], g.cols);
        } else {
            io.x_out = g.mat(a[2]);
            io.h = g.mat(a[6]);
        }
        io.pre_rstd = static_cast<float*>(g.vec(a[3], g.rows, at::kFloat));
        io.post_rstd = static_cast<float*>(g.vec(a[7], g.rows, at::kFloat));
        io.dx = g.mat(a[4]);
        io.dh = g.mat(a[5]);
        io.dpost_weight = g.vec(a[15], g.cols, weights);
        io.dpre_weight = g.vec(a[17], g.cols, weights);
        int64_t dgate_rows;
        io.dgate = g.gate(a[16], dgate_rows);
        if (dgate_rows != 0 && dgate_rows != p.gate_rows) throw Misfit{};
        int64_t bytes = 0;
        if (io.dpost_weight || io.dpre_weight || io.dgate.data) {
            if (ptored_block_norm_backward_workspace(g.rows, g.cols, dgate_rows, &bytes) != PTORED_OK)
                throw Misfit{};
        }
        const at::Tensor ws = g.workspace(a[18], a[19], bytes);
        if (ws.defined()) {
            io.workspace = ws.data_ptr();
            io.workspace_bytes = (int64_t)ws.nbytes();
        }
        return wrote(ptored_block_norm_backward(&p, &io, g.stream(a[19])),
                     {a[4], a[5], a[15], a[16], a[17]});
    });
}

// x, kept, stream
PyObject* checkpoint_pack(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 3);
        const Group g(tensor(a[0]));
        if (a[1] == Py_None) throw Misfit{};
        return wrote(ptored_checkpoint_pack(g.mat(a[0]), g.rows, g.cols, g.code,
                                            g.kept(a[1], g.cols), g.stream(a[2])),
                     {a[1]});
    });
}

// kept, out, stream
PyObject* checkpoint_unpack(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 3);
        const Group g(tensor(a[1]));
        if (a[0] == Py_None) throw Misfit{};
        return wrote(ptored_checkpoint_unpack(g.kept(a[0], g.cols), g.rows, g.cols, g.code,
                                              g.mat(a[1]), g.stream(a[2])),
                     {a[1]});
    });
}

// dy, kept, dw, accumulate, workspace, stream
PyObject* checkpoint_wgrad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 6);
        const Group g(tensor(a[0]));
        const at::Tensor& dw = tensor(a[2]);
        if (a[1] == Py_None || dw.dim() != 2) throw Misfit{};
        const int64_t cols = dw.size(1);
        if (cols == 0) throw Misfit{};
        const int code = code_of(dw.scalar_type());
        if (code != PTORED_F32 && code != g.code) throw Misfit{};
        const int accumulate = PyObject_IsTrue(a[3]);
        if (accumulate < 0) throw Misfit{};
        int64_t bytes = 0;
        if (ptored_checkpoint_wgrad_workspace(g.rows, g.cols, cols, g.code, &bytes) != PTORED_OK)
            throw Misfit{};
        const ptored_rows out = g.rows_of(dw, g.cols, cols, dw.scalar_type());
        const ptored_checkpoint x = g.kept(a[1], cols);
        const at::Tensor ws = g.workspace(a[4], a[5], bytes);
        return wrote(ptored_checkpoint_wgrad(g.mat(a[0]), x, g.rows, g.cols, cols, g.code, out, code,
                                             accumulate, ws.defined() ? ws.data_ptr() : nullptr,
                                             ws.defined() ? (int64_t)ws.nbytes() : 0,
                                             g.stream(a[5])),
                     {a[2]});
    });
}

#define PTORED_CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    PTORED_CALL(block_norm),        PTORED_CALL(block_norm_backward), PTORED_CALL(checkpoint_pack),
    PTORED_CALL(checkpoint_unpack), PTORED_CALL(checkpoint_wgrad),    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
