// torch_calls.cpp -- the tensor-level calls of the block boundary and of the
// step's operators, natively.
//
// The kernels of a single token take 4 us and less; reading a dozen tensors'
// shapes, strides and pointers from Python and marshalling them takes 10.
// This extension module reads them from the tensors themselves.  It takes only
// calls whose tensors all fit as they are (types, shapes, devices, plain
// strides, torch's current stream or a handle) and returns the library's
// status; for anything else it returns None, and the Python code in block.py or
// step.py looks again, makes the call or raises the error.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <vector>

#include "ptored_step.h"

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
    // A matrix of the group's type and another shape, or None.
    ptored_rows of(PyObject* o, int64_t r, int64_t c) const {
        if (o == Py_None) return {nullptr, 0};
        return rows_of(tensor(o), r, c, type);
    }
    // The ranks' partial outputs; returns how many.
    int parts(PyObject* list, const void** to, int64_t& part_ld) const {
        if (!PyList_Check(list) && !PyTuple_Check(list)) throw Misfit{};
        const Py_ssize_t nranks = PySequence_Fast_GET_SIZE(list);
        if (nranks > PTORED_MAX_RANKS) throw Misfit{};
        part_ld = cols;
        for (Py_ssize_t r = 0; r < nranks; ++r) {
            const ptored_rows y = mat(PySequence_Fast_GET_ITEM(list, r));
            if (r == 0) part_ld = y.ld;
            // the pitch of a single row is any
            if (y.data == nullptr || (rows > 1 && y.ld != part_ld)) throw Misfit{};
            to[r] = y.data;
        }
        return (int)nranks;
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
        const void* parts[PTORED_MAX_RANKS];
        int64_t part_ld;
        const int nranks = g.parts(a[0], parts, part_ld);
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
        return wrote(ptored_block_norm(parts, nranks, part_ld, &p, &io, g.stream(a[17])),
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

// The type that weights (None among them) share; float32 without any.
at::ScalarType weight_type(const Group& g, std::initializer_list<PyObject*> weights) {
    for (PyObject* o : weights) {
        if (o == Py_None) continue;
        const at::ScalarType t = tensor(o).scalar_type();
        if (t != g.type && t != at::kFloat) throw Misfit{};
        return t;
    }
    return at::kFloat;
}

// parts, x, x_out, z, weight, bias, eps, mean, rstd, stream
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 10);
        const Group g(tensor(a[1]));
        const void* parts[PTORED_MAX_RANKS];
        int64_t part_ld;
        const int nranks = g.parts(a[0], parts, part_ld);
        const at::ScalarType weights = weight_type(g, {a[4], a[5]});
        ptored_layer_norm_params p{};
        p.rows = g.rows;
        p.cols = g.cols;
        p.weight = g.vec(a[4], g.cols, weights);
        p.bias = g.vec(a[5], g.cols, weights);
        p.eps = number(a[6]);
        p.dtype = g.code;
        p.weight_dtype = code_of(weights);
        return wrote(ptored_layer_norm(parts, nranks, part_ld, &p, g.mat(a[1]), g.mat(a[2]),
                                       g.mat(a[3]),
                                       static_cast<float*>(g.vec(a[7], g.rows, at::kFloat)),
                                       static_cast<float*>(g.vec(a[8], g.rows, at::kFloat)),
                                       g.stream(a[9])),
                     {a[2], a[3], a[7], a[8]});
    });
}

// dz, dx_out, x_out, mean, rstd, dx, weight, dweight, dbias, workspace, stream
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 11);
        const Group g(tensor(a[0]));
        if (a[2] == Py_None || a[3] == Py_None || a[4] == Py_None) throw Misfit{};
        const at::ScalarType weights = weight_type(g, {a[6], a[7], a[8]});
        ptored_layer_norm_params p{};
        p.rows = g.rows;
        p.cols = g.cols;
        p.weight = g.vec(a[6], g.cols, weights);
        p.dtype = g.code;
        p.weight_dtype = code_of(weights);
        void* const dw = g.vec(a[7], g.cols, weights);
        void* const db = g.vec(a[8], g.cols, weights);
        int64_t bytes = 0;
        if ((dw || db) && ptored_layer_norm_backward_workspace(g.rows, g.cols, &bytes) != PTORED_OK)
            throw Misfit{};
        const ptored_rows dz = g.mat(a[0]), dxo = g.mat(a[1]), x = g.mat(a[2]), dx = g.mat(a[5]);
        const void* const mean = g.vec(a[3], g.rows, at::kFloat);
        const void* const rstd = g.vec(a[4], g.rows, at::kFloat);
        const at::Tensor ws = g.workspace(a[9], a[10], bytes);
        return wrote(ptored_layer_norm_backward(
                         &p, dz, dxo, x, static_cast<const float*>(mean),
                         static_cast<const float*>(rstd), dx, dw, db,
                         ws.defined() ? ws.data_ptr() : nullptr,
                         ws.defined() ? (int64_t)ws.nbytes() : 0, g.stream(a[10])),
                     {a[5], a[7], a[8]});
    });
}

int whole(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Misfit{};
    return (int)v;
}

// x, w_gate, w_up, y, activation, gate, up, workspace, stream
PyObject* gated_ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 9);
        const Group g(tensor(a[0]));
        const at::Tensor& out = tensor(a[3]);
        if (out.dim() != 2 || out.size(1) == 0) throw Misfit{};
        const int64_t wide = out.size(1);
        const ptored_ffn_params p{g.rows, g.cols, wide, g.code, whole(a[4])};
        const ptored_rows x = g.mat(a[0]), wg = g.of(a[1], wide, g.cols), wu = g.of(a[2], wide, g.cols);
        const ptored_rows y = g.of(a[3], g.rows, wide), gate = g.of(a[5], g.rows, wide);
        const ptored_rows up = g.of(a[6], g.rows, wide);
        int64_t bytes = 0;
        if (ptored_gated_ffn_workspace(g.rows, g.cols, wide, g.code, &bytes) != PTORED_OK) throw Misfit{};
        const at::Tensor ws = g.workspace(a[7], a[8], bytes);
        return wrote(ptored_gated_ffn(&p, x, wg, wu, y, gate, up, ws.defined() ? ws.data_ptr() : nullptr,
                                      ws.defined() ? (int64_t)ws.nbytes() : 0, g.stream(a[8])),
                     {a[3], a[5], a[6]});
    });
}

// dy, gate, up, dgate, dup, activation, x, w_gate, w_up, dx, dw_gate, dw_up, accumulate, workspace,
// stream
PyObject* gated_ffn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 15);
        const Group g(tensor(a[0]));
        for (int i = 1; i <= 4; ++i)
            if (a[i] == Py_None) throw Misfit{};
        const int64_t wide = g.cols;
        int64_t cols = 0;
        for (const int i : {6, 9, 7, 8}) {
            if (a[i] == Py_None) continue;
            const at::Tensor& t = tensor(a[i]);
            if (t.dim() != 2 || t.size(1) == 0) throw Misfit{};
            cols = t.size(1);
            break;
        }
        const ptored_ffn_params p{g.rows, cols, wide, g.code, whole(a[5])};
        ptored_ffn_grad_io io{};
        io.dy = g.mat(a[0]);
        io.gate = g.mat(a[1]);
        io.up = g.mat(a[2]);
        io.dgate = g.mat(a[3]);
        io.dup = g.mat(a[4]);
        io.x = g.of(a[6], g.rows, cols);
        io.w_gate = g.of(a[7], wide, cols);
        io.w_up = g.of(a[8], wide, cols);
        io.dx = g.of(a[9], g.rows, cols);
        at::ScalarType weights = g.type;
        if (a[10] != Py_None || a[11] != Py_None)
            weights = tensor(a[a[10] != Py_None ? 10 : 11]).scalar_type();
        if (weights != g.type && weights != at::kFloat) throw Misfit{};
        if (a[10] != Py_None) io.dw_gate = g.rows_of(tensor(a[10]), wide, cols, weights);
        if (a[11] != Py_None) io.dw_up = g.rows_of(tensor(a[11]), wide, cols, weights);
        if ((io.dx.data && !(io.w_gate.data && io.w_up.data)) ||
            ((io.dw_gate.data || io.dw_up.data) && !io.x.data))
            throw Misfit{};
        io.dw_dtype = code_of(weights);
        io.accumulate = PyObject_IsTrue(a[12]);
        if (io.accumulate < 0) throw Misfit{};
        int64_t bytes = 0;
        if ((io.dx.data || io.dw_gate.data || io.dw_up.data) &&
            ptored_gated_ffn_backward_workspace(g.rows, cols, wide, g.code, &bytes) != PTORED_OK)
            throw Misfit{};
        const at::Tensor ws = g.workspace(a[13], a[14], bytes);
        if (ws.defined()) {
            io.workspace = ws.data_ptr();
            io.workspace_bytes = (int64_t)ws.nbytes();
        }
        return wrote(ptored_gated_ffn_backward(&p, &io, g.stream(a[14])),
                     {a[3], a[4], a[9], a[10], a[11]});
    });
}

// The gradients of a call that all lie as they are: filling a range of memory
// in their order, or 2-D with unit column stride; outs alike.
struct Gradients {
    std::vector<ptored_grad> list;
    const at::Tensor& norm;
    PyObject* outs;
    Group g;

    Gradients(PyObject* grads, PyObject* norm_, PyObject* outs_)
        : norm(tensor(norm_)), outs(outs_), g(on_device(norm)) {
        if (!(PyList_Check(grads) || PyTuple_Check(grads))) throw Misfit{};
        const bool into = outs != nullptr && outs != Py_None;
        if (into && !(PyList_Check(outs) || PyTuple_Check(outs))) throw Misfit{};
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(grads);
        if (into && PySequence_Fast_GET_SIZE(outs) != n) throw Misfit{};
        list.resize((size_t)n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const at::Tensor& t = tensor(PySequence_Fast_GET_ITEM(grads, i));
            const at::Tensor& o = into ? tensor(PySequence_Fast_GET_ITEM(outs, i)) : t;
            ptored_grad& e = list[(size_t)i];
            if (t.layout() != at::kStrided || o.layout() != at::kStrided || !t.is_cuda() ||
                !o.is_cuda() || t.get_device() != g.device || o.get_device() != g.device)
                throw Misfit{};
            e.dtype = code_of(t.scalar_type());
            e.out_dtype = code_of(o.scalar_type());
            if (e.out_dtype != PTORED_F32 && e.out_dtype != e.dtype) throw Misfit{};
            if (into && t.sizes() != o.sizes()) throw Misfit{};
            const int64_t elems = t.numel();
            if (elems == 0) throw Misfit{};
            e.data = t.data_ptr();
            e.out = o.data_ptr();
            if (t.is_contiguous() && o.is_contiguous()) {
                e.rows = 1;
                e.cols = e.ld = e.out_ld = elems;
                continue;
            }
            if (t.dim() != 2) throw Misfit{};
            e.rows = t.size(0);
            e.cols = t.size(1);
            e.ld = t.stride(0);
            e.out_ld = o.stride(0);
            if (t.stride(1) != 1 || o.stride(1) != 1 || e.ld < e.cols || e.out_ld < e.cols)
                throw Misfit{};
        }
    }
    static Group on_device(const at::Tensor& norm) {
        if (norm.numel() != 1 || norm.scalar_type() != at::kFloat) throw Misfit{};
        return Group(norm.reshape({1, 1}));
    }
    at::Tensor workspace(PyObject* given, PyObject* stream) const {
        int64_t bytes = 0;
        if (ptored_grad_norm_workspace(list.data(), (int64_t)list.size(), &bytes) != PTORED_OK)
            throw Misfit{};
        return g.workspace(given, stream, bytes);
    }
    int wrote_outs(int status, PyObject* grads) const {
        PyObject* o = outs == Py_None ? grads : outs;
        for (Py_ssize_t i = 0; status == PTORED_OK && i < PySequence_Fast_GET_SIZE(o); ++i)
            wrote(status, {PySequence_Fast_GET_ITEM(o, i)});
        return status;
    }
};

// grads, norm, workspace, stream
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 4);
        const Gradients v(a[0], a[1], nullptr);
        const at::Tensor ws = v.workspace(a[2], a[3]);
        return wrote(ptored_grad_norm(v.list.data(), (int64_t)v.list.size(),
                                      static_cast<float*>(v.norm.data_ptr()),
                                      ws.defined() ? ws.data_ptr() : nullptr,
                                      ws.defined() ? (int64_t)ws.nbytes() : 0, v.g.stream(a[3])),
                     {a[1]});
    });
}

// grads, norm, max_norm, outs, workspace, stream
PyObject* grad_scale(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 6);
        const Gradients v(a[0], a[1], a[3]);
        const float most = number(a[2]);
        const at::Tensor ws = v.workspace(a[4], a[5]);
        return v.wrote_outs(ptored_grad_scale(v.list.data(), (int64_t)v.list.size(),
                                              static_cast<const float*>(v.norm.data_ptr()), most,
                                              ws.defined() ? ws.data_ptr() : nullptr,
                                              ws.defined() ? (int64_t)ws.nbytes() : 0,
                                              v.g.stream(a[5])),
                            a[0]);
    });
}

// grads, max_norm, norm, outs, workspace, stream
PyObject* grad_clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        want(n, 6);
        const Gradients v(a[0], a[2], a[3]);
        const float most = number(a[1]);
        const at::Tensor ws = v.workspace(a[4], a[5]);
        const int status = ptored_grad_clip(v.list.data(), (int64_t)v.list.size(), most,
                                            static_cast<float*>(v.norm.data_ptr()),
                                            ws.defined() ? ws.data_ptr() : nullptr,
                                            ws.defined() ? (int64_t)ws.nbytes() : 0, v.g.stream(a[5]));
        return v.wrote_outs(wrote(status, {a[2]}), a[0]);
    });
}

#define PTORED_CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    PTORED_CALL(block_norm),        PTORED_CALL(block_norm_backward), PTORED_CALL(checkpoint_pack),
    PTORED_CALL(checkpoint_unpack), PTORED_CALL(checkpoint_wgrad),    PTORED_CALL(layer_norm),
    PTORED_CALL(layer_norm_backward), PTORED_CALL(gated_ffn),         PTORED_CALL(gated_ffn_backward),
    PTORED_CALL(grad_norm),         PTORED_CALL(grad_scale),          PTORED_CALL(grad_clip),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
