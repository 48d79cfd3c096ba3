// torch_calls.cpp -- the operators of moe_ops.h on torch tensors, for the usual
// call: exact tensors on the current device, the current stream, nothing to report.
//
// A call on a few tokens is as long on the host as on the GPU, and most of that is
// the interpreter asking each tensor for its properties and allocating the output.
// Here the same checks and the allocation are C++ (host time of a one-token linear on
// a Grace core: 2.9 us, 11 through ctypes). Whatever is not the usual call (another device
// or stream, a tensor subclass, an input that asks for a gradient, outputs that torch would
// fill, any argument that does not fit) returns None, and ops.py goes on from there with its own checks and messages.
// Compiled against the installed torch, without the CUDA library: ops.py passes in
// the addresses of its entry points.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
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
decltype(&moe_route) fn_route;
decltype(&moe_quantize_rows) fn_quantize;
decltype(&moe_linear_q8) fn_linear_q8;
decltype(&moe_grouped_linear_q8) fn_grouped_q8;

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

// Whether torch fills new memory (torch.use_deterministic_algorithms): torch.empty does, what is
// below does not, and such a call is not the usual one.
bool fills() {
    const at::Context &c = at::globalContext();
    return c.deterministicAlgorithms() && c.deterministicFillUninitializedMemory();
}

// Memory on the current device for an output, from torch's allocator, and a tensor of `type`
// and these sizes on it from byte `at` on. (at::empty finds its way to the same allocator in
// about 1 us more; several outputs share a storage, which lives as long as any of them.)
c10::Storage memory(int64_t bytes) {
    c10::Allocator *a = c10::cuda::CUDACachingAllocator::get();
    return c10::Storage(c10::Storage::use_byte_size_t(), bytes, a->allocate(bytes), a, true);
}
at::Tensor part_of(const c10::Storage &all, at::ScalarType type, int64_t at, at::IntArrayRef sizes) {
    const auto meta = c10::scalarTypeToTypeMeta(type);
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all), c10::DispatchKeySet(c10::DispatchKey::CUDA), meta);
    t.unsafeGetTensorImpl()->set_storage_offset(at / (int64_t)meta.itemsize());
    t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    return t;
}
at::Tensor empty(int64_t n, int64_t cols, at::ScalarType type) {
    return part_of(memory(n * cols * (int64_t)c10::elementSize(type)), type, 0, {n, cols});
}

at::ScalarType type_of(int dtype) { return dtype == MOE_DTYPE_BF16 ? at::kBFloat16 : at::kHalf; }

// tensors that a struct keeps the addresses of (None where it has no address)
template <int N> struct Kept {
    const void *at[N];
    at::ScalarType type[N];
};
Kept<4> kept(const moe_product *p) {
    const at::ScalarType dt = type_of(p->dtype);
    return {{p->w, p->w_up, p->bias, p->bias_up}, {dt, dt, dt, dt}};
}
Kept<6> kept(const moe_product_q8 *p) {
    const at::ScalarType dt = type_of(p->dtype);
    return {{p->w, p->w_up, p->scale, p->scale_up, p->bias, p->bias_up},
            {at::kChar, at::kChar, at::kFloat, at::kFloat, dt, dt}};
}

// whether `w` is still the tensor of type dt at address `at`, on the device
bool still(PyObject *w, const void *at, at::ScalarType dt, int dev) {
    if (!THPVariable_Check(w)) return false;
    const at::Tensor &t = THPVariable_Unpack(w);
    return t.defined() && t.layout() == at::kStrided && !differentiated(t) && t.scalar_type() == dt && t.is_cuda() &&
           t.get_device() == dev && t.const_data_ptr() == at;
}

// Whether a product's weights (w, w_up, then vectors of E N values: tensors or None) are
// still what *p says of them: a tensor may have been given another storage, shape or device.
template <typename P> bool weights(PyObject *o, const P *p, int dev) {
    constexpr int N = sizeof(decltype(kept(p))::at) / sizeof(void *);
    // (another number: the weights of another kind of product, and p no P)
    if (!p || !PyTuple_Check(o) || PyTuple_GET_SIZE(o) != N) return false;
    const auto k = kept(p);
    for (int i = 0; i < N; ++i) {
        PyObject *w = PyTuple_GET_ITEM(o, i);
        if (w == Py_None) {
            if (k.at[i]) return false;
            continue;
        }
        if (!still(w, k.at[i], k.type[i], dev)) return false;
        const at::Tensor &t = THPVariable_Unpack(w);
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
    if (!given && fills()) return other();
    const at::Tensor out = given ? *given : empty(n, p->N, dt);
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
    if (!given && fills()) return other();
    const at::Tensor out = given ? *given : empty(n, p->N, dt);
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
    if (fills()) return other();
    const int64_t S = idx->numel();
    // one allocation, and four tensors on its storage, each with the values that it alone covers
    const c10::Storage all = memory(4 * (3 * S + E + 1));
    const at::Tensor token = part_of(all, at::kInt, 0, {S}), rank = part_of(all, at::kInt, 4 * S, {S}),
                     of = part_of(all, at::kInt, 8 * S, idx->sizes()), offsets = part_of(all, at::kInt, 12 * S, {E + 1});
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
    if (!given && fills()) return other();
    const at::Tensor out = given ? *given : empty(n, N, dt);
    const moe_status st = fn_combine(dt == at::kHalf ? MOE_DTYPE_F16 : MOE_DTYPE_BF16, y->const_data_ptr(), ldy, (int)r,
                                     of->const_data_ptr<int32_t>(), w->const_data_ptr<float>(), (int)n, (int)k, (int)N,
                                     res ? res->const_data_ptr() : nullptr, ldr, out.mutable_data_ptr(), ldo,
                                     c10::cuda::getCurrentCUDAStream(dev).stream());
    return result(st, out, a[4]);
    END_HANDLE_TH_ERRORS
}

// two results of a call as a `type` (a subclass of tuple without members), or its status as a number
PyObject *results(moe_status st, PyTypeObject *type, const at::Tensor &first, const at::Tensor &second) {
    if (st != MOE_OK) return PyLong_FromLong(st);
    PyObject *t = type->tp_alloc(type, 2);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(first));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(second));
    return t;
}

bool tuple_type(PyObject *o) { return PyType_Check(o) && PyType_IsSubtype((PyTypeObject *)o, &PyTuple_Type); }

// route(router address, logits, (bias,), type): type of (topk_idx, topk_w)
PyObject *route(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (n_args != 4 || !PyTuple_Check(a[2]) || PyTuple_GET_SIZE(a[2]) != 1 || !tuple_type(a[3])) return other();
    const auto *r = static_cast<const moe_router *>(PyLong_AsVoidPtr(a[0]));
    const at::Tensor *l;
    if (!r || !tensor(a[1], &l) || !l || l->dim() != 2 || !l->is_cuda()) return other();
    const int dev = (int)l->get_device();
    PyObject *bias = PyTuple_GET_ITEM(a[2], 0);
    if (bias == Py_None ? r->bias != nullptr
                        : !still(bias, r->bias, at::kFloat, dev) || THPVariable_Unpack(bias).numel() != r->E ||
                              !THPVariable_Unpack(bias).is_contiguous())
        return other();
    const at::ScalarType dt = l->scalar_type();
    int64_t ldl;
    const int64_t n = l->size(0), k = r->top_k;
    if ((dt != at::kBFloat16 && dt != at::kHalf && dt != at::kFloat) || !rows(*l, -1, r->E, dt, dev, &ldl) || n == 0 ||
        n > INT32_MAX || k < 1 || k > 1024 || c10::cuda::current_device() != dev)
        return other();
    if (fills()) return other();
    const c10::Storage all = memory(8 * n * k);
    const at::Tensor idx = part_of(all, at::kInt, 0, {n, k}), w = part_of(all, at::kFloat, 4 * n * k, {n, k});
    const moe_status st = fn_route(r, dt == at::kFloat ? MOE_DTYPE_F32 : dt == at::kHalf ? MOE_DTYPE_F16 : MOE_DTYPE_BF16,
                                   l->const_data_ptr(), ldl, (int)n, idx.mutable_data_ptr<int32_t>(),
                                   w.mutable_data_ptr<float>(), c10::cuda::getCurrentCUDAStream(dev).stream());
    return results(st, (PyTypeObject *)a[3], idx, w);
    END_HANDLE_TH_ERRORS
}

// quantize(x, type): type of (codes, scale)
PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    const at::Tensor *x;
    if (n_args != 2 || !tuple_type(a[1]) || !tensor(a[0], &x) || !x || x->dim() != 2 || !x->is_cuda()) return other();
    const int dev = (int)x->get_device();
    const at::ScalarType dt = x->scalar_type();
    const int64_t n = x->size(0), K = x->size(1);
    int64_t ldx;
    if ((dt != at::kBFloat16 && dt != at::kHalf) || n == 0 || K == 0 || n > INT32_MAX || K > INT32_MAX ||
        !rows(*x, -1, K, dt, dev, &ldx) || c10::cuda::current_device() != dev)
        return other();
    if (fills()) return other();
    const int64_t at_scale = (n * K + 15) / 16 * 16;
    const c10::Storage all = memory(at_scale + 4 * n);
    const at::Tensor codes = part_of(all, at::kChar, 0, {n, K}), scale = part_of(all, at::kFloat, at_scale, {n});
    const moe_status st = fn_quantize(dt == at::kHalf ? MOE_DTYPE_F16 : MOE_DTYPE_BF16, x->const_data_ptr(), ldx, (int)n,
                                      (int)K, codes.mutable_data_ptr<int8_t>(), K, scale.mutable_data_ptr<float>(),
                                      c10::cuda::getCurrentCUDAStream(dev).stream());
    return results(st, (PyTypeObject *)a[1], codes, scale);
    END_HANDLE_TH_ERRORS
}

// (codes [rows, K], the scale of each row)
bool coded(PyObject *o, int64_t K, int dev, const at::Tensor **x, const at::Tensor **scale, int64_t *ldx) {
    return PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2 && tensor(PyTuple_GET_ITEM(o, 0), x) && *x &&
           tensor(PyTuple_GET_ITEM(o, 1), scale) && *scale && rows(**x, -1, K, at::kChar, dev, ldx) &&
           dense(**scale, at::kFloat, dev) && (*scale)->dim() == 1 && (*scale)->size(0) == (*x)->size(0);
}

// linear_q8(product address, device, (codes, scale), residual, out, weights)
PyObject *linear_q8(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (n_args != 6) return other();
    const auto *p = static_cast<const moe_product_q8 *>(PyLong_AsVoidPtr(a[0]));
    const int dev = (int)PyLong_AsLong(a[1]);
    if (dev < 0 || !weights(a[5], p, dev) || p->E != 1) return other();
    const at::Tensor *x, *scale, *res, *given;
    int64_t ldx, ldr = 0, ldo = p->N;
    if (!coded(a[2], p->K, dev, &x, &scale, &ldx) || !tensor(a[3], &res) || !tensor(a[4], &given)) return other();
    const at::ScalarType dt = type_of(p->dtype);
    const int64_t n = x->size(0);
    if (n == 0 || n > INT32_MAX || (res && !rows(*res, n, p->N, dt, dev, &ldr)) ||
        (given && !rows(*given, n, p->N, dt, dev, &ldo)) || c10::cuda::current_device() != dev)
        return other();
    if (!given && fills()) return other();
    const at::Tensor out = given ? *given : empty(n, p->N, dt);
    const moe_status st =
        fn_linear_q8(p, x->const_data_ptr<int8_t>(), ldx, scale->const_data_ptr<float>(), (int)n,
                     res ? res->const_data_ptr() : nullptr, ldr, out.mutable_data_ptr(), ldo,
                     c10::cuda::getCurrentCUDAStream(dev).stream());
    return result(st, out, a[4]);
    END_HANDLE_TH_ERRORS
}

// grouped_q8(product address, device, (codes, scale), offsets, row_token, out, weights)
PyObject *grouped_q8(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (n_args != 7) return other();
    const auto *p = static_cast<const moe_product_q8 *>(PyLong_AsVoidPtr(a[0]));
    const int dev = (int)PyLong_AsLong(a[1]);
    if (dev < 0 || !weights(a[6], p, dev)) return other();
    const at::Tensor *x, *scale, *off, *token, *given;
    int64_t ldx, ldo = p->N;
    if (!coded(a[2], p->K, dev, &x, &scale, &ldx) || !tensor(a[3], &off) || !off || !tensor(a[4], &token) ||
        !tensor(a[5], &given))
        return other();
    if (!dense(*off, at::kInt, dev) || off->dim() != 1 || off->size(0) != p->E + 1 ||
        (token && (!dense(*token, at::kInt, dev) || token->dim() != 1)))
        return other();
    const at::ScalarType dt = type_of(p->dtype);
    const int64_t x_rows = x->size(0), n = token ? token->size(0) : x_rows;
    if (n == 0 || x_rows == 0 || n > INT32_MAX || x_rows > INT32_MAX ||
        (given && !rows(*given, n, p->N, dt, dev, &ldo)) || c10::cuda::current_device() != dev)
        return other();
    if (!given && fills()) return other();
    const at::Tensor out = given ? *given : empty(n, p->N, dt);
    const moe_status st = fn_grouped_q8(
        p, off->const_data_ptr<int32_t>(), token ? token->const_data_ptr<int32_t>() : nullptr,
        x->const_data_ptr<int8_t>(), ldx, scale->const_data_ptr<float>(), (int)x_rows, (int)n, out.mutable_data_ptr(), ldo,
        c10::cuda::getCurrentCUDAStream(dev).stream());
    return result(st, out, a[5]);
    END_HANDLE_TH_ERRORS
}

// bind(addresses of the eight entry points)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (n_args != 8) {
        PyErr_SetString(PyExc_TypeError, "bind takes eight addresses");
        return nullptr;
    }
    fn_route = reinterpret_cast<decltype(fn_route)>(PyLong_AsVoidPtr(a[4]));
    fn_quantize = reinterpret_cast<decltype(fn_quantize)>(PyLong_AsVoidPtr(a[5]));
    fn_linear_q8 = reinterpret_cast<decltype(fn_linear_q8)>(PyLong_AsVoidPtr(a[6]));
    fn_grouped_q8 = reinterpret_cast<decltype(fn_grouped_q8)>(PyLong_AsVoidPtr(a[7]));
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
                         method<combine>("combine"), method<route>("route"),     method<quantize>("quantize"),
                         method<linear_q8>("linear_q8"), method<grouped_q8>("grouped_q8"), method<bind>("bind"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
