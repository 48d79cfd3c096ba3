// torch_calls.cpp -- the operators of moe_ops.h on torch tensors, for the usual
// call: exact tensors on the current device, the current stream, nothing to report.
//
// A call on a few tokens is as long on the host as on the GPU, and most of that is
// the interpreter asking each tensor for its properties and allocating the output.
// Here the same checks and the allocation are C++ (host time of a one-token linear on
// a Grace core: 3.6 us, 11 through ctypes). Whatever is not the usual call (another device or stream, a tensor
// subclass, an input that asks for a gradient, any argument that does not fit)
// returns None, and ops.py goes on from there with its own checks and messages.
// Compiled against the installed torch, without the CUDA library: ops.py passes in
// the addresses of its entry points.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe_ops.h"

namespace {

decltype(&moe_linear) fn_linear;
decltype(&moe_grouped_linear) fn_grouped;
decltype(&moe_group_slots) fn_slots;
decltype(&moe_combine_slots) fn_combine;

PyObject *other() { Py_RETURN_NONE; }

// whether autograd would have to record a call on this tensor, backwards or forwards
bool differentiated(const at::Tensor &t) {
    return (t.requires_grad() && c10::GradMode::is_enabled()) || t._fw_grad(0).defined();
}

// the tensor of a plain torch.Tensor argument (a null pointer for None), or false
bool tensor(PyObject *o, const at::Tensor **t) {
    *t = nullptr;
    if (o == Py_None) return true;
    if (!THPVariable_CheckExact(o)) return false;
    *t = &THPVariable_Unpack(o);
    return (*t)->defined() && (*t)->layout() == at::kStrided && !differentiated(**t);
}

// [n, cols] (n < 0: any) of type dt on CUDA device dev with adjacent columns
bool rows(const at::Tensor &t, int64_t n, int64_t cols, at::ScalarType dt, int dev, int64_t *ld) {
    if (t.dim() != 2 || t.size(1) != cols || (n >= 0 && t.size(0) != n)) return false;
    if (t.scalar_type() != dt || !t.is_cuda() || t.get_device() != dev) return false;
    if (t.is_contiguous()) *ld = cols;
    else if (t.stride(1) != 1 && cols > 1) return false;
    else *ld = t.size(0) > 1 ? t.stride(0) : cols;
    return true;
}

bool dense(const at::Tensor &t, at::ScalarType dt, int dev) {
    return t.scalar_type() == dt && t.is_cuda() && t.get_device() == dev && t.is_contiguous();
}

// the result of a call: the tensor, or the status as a number. (An output that was given
// counts as written, for whoever keeps it for a backward pass.)
PyObject *result(moe_status st, const at::Tensor &out, PyObject *given) {
    if (st != MOE_OK) return PyLong_FromLong(st);
    if (given != Py_None) {
        if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(out);
}

at::ScalarType type_of(int dtype) { return dtype == MOE_DTYPE_BF16 ? at::kBFloat16 : at::kHalf; }

// Whether a product's weights (w, w_up, bias, bias_up: tensors or None) are still what
// *p says of them: a tensor may have been given another storage, shape or device.
bool weights(PyObject *o, const moe_product *p, int dev) {
    if (!p || !PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) return false;
    const void *at[4] = {p->w, p->w_up, p->bias, p->bias_up};
    const at::ScalarType dt = type_of(p->dtype);
    for (int i = 0; i < 4; ++i) {
        PyObject *w = PyTuple_GET_ITEM(o, i);
        if (w == Py_None) {
            if (at[i]) return false;
            continue;
        }
        if (!THPVariable_Check(w)) return false;
        const at::Tensor &t = THPVariable_Unpack(w);
        if (!t.defined() || t.layout() != at::kStrided || differentiated(t) || t.scalar_type() != dt || !t.is_cuda() ||
            t.get_device() != dev || t.const_data_ptr() != at[i])
            return false;
        const int64_t d = t.dim();
        if (i < 2) {
            if ((d != 2 && d != 3) || t.size(d - 1) != p->K || t.size(d - 2) != p->N || (d == 3 ? t.size(0) : 1) != p->E)
                return false;
            if ((t.stride(d - 1) != 1 && p->K > 1) || (p->N > 1 && t.stride(d - 2) != p->ldw) ||
                (p->E > 1 && t.stride(0) != p->stride_e))
                return false;
        } else if (t.numel() != (int64_t)p->E * p->N || !t.is_contiguous()) {
            return false;
        }
    }
    return true;
}

// linear(product address, device, x, residual, out, weights)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (n_args != 6) return other();
    const auto *p = static_cast<const moe_product *>(PyLong_AsVoidPtr(a[0]));
    const int dev = (int)PyLong_AsLong(a[1]);
    if (dev < 0 || !weights(a[5], p, dev)) return other();
    const at::Tensor *x, *res, *given;
    if (!tensor(a[2], &x) || !x || !tensor(a[3], &res) || !tensor(a[4], &given)) return other();
    const at::ScalarType dt = type_of(p->dtype);
    int64_t ldx, ldr = 0, ldo = p->N;
    if (!rows(*x, -1, p->K, dt, dev, &ldx)) return other();
    const int64_t n = x->size(0);
    if (n == 0 || n > INT32_MAX || (res && !rows(*res, n, p->N, dt, dev, &ldr)) ||
        (given && !rows(*given, n, p->N, dt, dev, &ldo)) || c10::cuda::current_device() != dev)
        return other();
    const at::Tensor out = given ? *given : at::empty({n, p->N}, x->options());
    const moe_status st = fn_linear(p, x->const_data_ptr(), ldx, (int)n, res ? res->const_data_ptr() : nullptr, ldr,
                                    out.mutable_data_ptr(), ldo, c10::cuda::getCurrentCUDAStream(dev).stream());
    return result(st, out, a[4]);
    END_HANDLE_TH_ERRORS
}

// grouped(product address, device, x, offsets, row_token, out, weights)
PyObject *grouped(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (n_args != 7) return other();
    const auto *p = static_cast<const moe_product *>(PyLong_AsVoidPtr(a[0]));
    const int dev = (int)PyLong_AsLong(a[1]);
    if (dev < 0 || !weights(a[6], p, dev)) return other();
    const at::Tensor *x, *off, *token, *given;
    if (!tensor(a[2], &x) || !x || !tensor(a[3], &off) || !off || !tensor(a[4], &token) ||
        !tensor(a[5], &given))
        return other();
    const at::ScalarType dt = type_of(p->dtype);
    int64_t ldx, ldo = p->N;
    if (!rows(*x, -1, p->K, dt, dev, &ldx) || !dense(*off, at::kInt, dev) || off->dim() != 1 ||
        off->size(0) != p->E + 1 || (token && (!dense(*token, at::kInt, dev) || token->dim() != 1)))
        return other();
    const int64_t x_rows = x->size(0), n = token ? token->size(0) : x_rows;
    if (n == 0 || x_rows == 0 || n > INT32_MAX || x_rows > INT32_MAX ||
        (given && !rows(*given, n, p->N, dt, dev, &ldo)) || c10::cuda::current_device() != dev)
        return other();
    const at::Tensor out = given ? *given : at::empty({n, p->N}, x->options());
    const moe_status st = fn_grouped(p, off->const_data_ptr<int32_t>(), token ? token->const_data_ptr<int32_t>() : nullptr,
                                     x->const_data_ptr(), ldx, (int)x_rows, (int)n, out.mutable_data_ptr(), ldo,
                                     c10::cuda::getCurrentCUDAStream(dev).stream());
    return result(st, out, a[5]);
    END_HANDLE_TH_ERRORS
}

// slots(topk_idx, E, begin, end): (offsets, slot_token, slot_k, slot_of)
PyObject *slots(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (n_args != 4) return other();
    const at::Tensor *idx;
    if (!tensor(a[0], &idx) || !idx || !PyLong_Check(a[1]) || !PyLong_Check(a[2]) || !PyLong_Check(a[3]))
        return other();
    const long E = PyLong_AsLong(a[1]), lo = PyLong_AsLong(a[2]), hi = PyLong_AsLong(a[3]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return other();
    }
    if (idx->dim() != 2 || idx->numel() == 0 || idx->numel() > INT32_MAX || E < 1 || E > (1 << 20) || lo < 0 || lo > E ||
        hi < 0 || hi > E || !idx->is_cuda() || !dense(*idx, at::kInt, idx->get_device()) ||
        c10::cuda::current_device() != idx->get_device())
        return other();
    const int64_t S = idx->numel();
    const at::Tensor all = at::empty({3 * S + E + 1}, idx->options());
    // One allocation, and four tensors on its storage, each with the values that it
    // alone covers: a call of 8 x 8 ids takes 5.2 us of the host, 7.8 with four
    // allocations. The storage lives as long as any of the four.
    auto part = [&](int64_t first, at::IntArrayRef sizes) {
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
        t.unsafeGetTensorImpl()->set_storage_offset(first);
        t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
        return t;
    };
    const at::Tensor token = part(0, {S}), rank = part(S, {S}), of = part(2 * S, idx->sizes()),
                     offsets = part(3 * S, {E + 1});
    const moe_status st =
        fn_slots(idx->const_data_ptr<int32_t>(), (int)idx->size(0), (int)idx->size(1), (int)E, (int)lo, (int)hi,
                 offsets.mutable_data_ptr<int32_t>(), token.mutable_data_ptr<int32_t>(),
                 rank.mutable_data_ptr<int32_t>(), of.mutable_data_ptr<int32_t>(),
                 c10::cuda::getCurrentCUDAStream(idx->get_device()).stream());
    if (st != MOE_OK) return PyLong_FromLong(st);
    PyObject *t = PyTuple_New(4);
    if (!t) return nullptr;
    const at::Tensor *parts[4] = {&offsets, &token, &rank, &of};
    for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(*parts[i]));
    return t;
    END_HANDLE_TH_ERRORS
}

// combine(y, slot_of, topk_w, residual, out)
PyObject *combine(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (n_args != 5) return other();
    const at::Tensor *y, *of, *w, *res, *given;
    if (!tensor(a[0], &y) || !y || !tensor(a[1], &of) || !of || !tensor(a[2], &w) || !w || !tensor(a[3], &res) ||
        !tensor(a[4], &given))
        return other();
    if (y->dim() != 2 || !y->is_cuda() || of->dim() != 2) return other();
    const at::ScalarType dt = y->scalar_type();
    const int dev = (int)y->get_device();
    const int64_t r = y->size(0), N = y->size(1), n = of->size(0), k = of->size(1);
    int64_t ldy, ldr = 0, ldo = N;
    if ((dt != at::kBFloat16 && dt != at::kHalf) || r == 0 || N == 0 || n == 0 || k == 0 || r > INT32_MAX ||
        N > INT32_MAX || n > INT32_MAX || k > INT32_MAX || !rows(*y, -1, N, dt, dev, &ldy) ||
        !dense(*of, at::kInt, dev) || !dense(*w, at::kFloat, dev) || w->sizes() != of->sizes() ||
        (res && !rows(*res, n, N, dt, dev, &ldr)) || (given && !rows(*given, n, N, dt, dev, &ldo)) ||
        c10::cuda::current_device() != dev)
        return other();
    const at::Tensor out = given ? *given : at::empty({n, N}, y->options());
    const moe_status st = fn_combine(dt == at::kHalf ? MOE_DTYPE_F16 : MOE_DTYPE_BF16, y->const_data_ptr(), ldy, (int)r,
                                     of->const_data_ptr<int32_t>(), w->const_data_ptr<float>(), (int)n, (int)k, (int)N,
                                     res ? res->const_data_ptr() : nullptr, ldr, out.mutable_data_ptr(), ldo,
                                     c10::cuda::getCurrentCUDAStream(dev).stream());
    return result(st, out, a[4]);
    END_HANDLE_TH_ERRORS
}

// bind(addresses of the four entry points)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (n_args != 4) {
        PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
        return nullptr;
    }
    fn_linear = reinterpret_cast<decltype(fn_linear)>(PyLong_AsVoidPtr(a[0]));
    fn_grouped = reinterpret_cast<decltype(fn_grouped)>(PyLong_AsVoidPtr(a[1]));
    fn_slots = reinterpret_cast<decltype(fn_slots)>(PyLong_AsVoidPtr(a[2]));
    fn_combine = reinterpret_cast<decltype(fn_combine)>(PyLong_AsVoidPtr(a[3]));
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
constexpr PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<linear>("linear"),   method<grouped>("grouped"), method<slots>("slots"),
                         method<combine>("combine"), method<bind>("bind"),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
