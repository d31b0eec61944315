// binding.cpp -- CPython module _native: the tensor side of the routed and
// grouped operators (checks, outputs, the call into include/gemm_coll_grouped.h).
//
// A call on a few tokens takes the device 4 to 10 us.  Through ctypes, with
// the checks and the allocations in Python, the host took 7 to 12 us for it
// and set the pace; here it takes about half of that, most of it the kernel
// launches.  Nothing is computed here.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "gemm_coll_grouped.h"

namespace {

using at::Tensor;

// Thrown with a Python error set.
struct Refused {
};

std::string text(at::IntArrayRef s)
{
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i)
        r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

[[noreturn]] void refuse(PyObject *kind, const std::string &what)
{
    PyErr_SetString(kind, what.c_str());
    throw Refused{};
}

const char *type_name(at::ScalarType t)
{
    return t == at::kBFloat16 ? "torch.bfloat16" : t == at::kFloat ? "torch.float32" : "torch.int32";
}

const Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// The current device, looked up at the first tensor of a call (-1: not yet).
thread_local int t_device;

// Refuses a tensor that is not on the current device, whose stream the call
// is launched on.
void here(const Tensor &t, const char *name)
{
    if (!t.is_cuda())
        refuse(PyExc_ValueError, std::string(name) + " must be a device tensor");
    if (t_device < 0)
        t_device = c10::impl::getDeviceGuardImpl(c10::DeviceType::CUDA)->getDevice().index();
    if (t.get_device() != t_device)
        refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() +
                                     ", the current device is cuda:" + std::to_string(t_device));
}

// A contiguous tensor of the given type on the current device.
const Tensor &dense(PyObject *o, const char *name, at::ScalarType type)
{
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, std::string(name) + " must be " + type_name(type) + ", got torch." +
                                    c10::toString(t.scalar_type()));
    here(t, name);
    if (!t.is_contiguous())
        refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t;
}

const Tensor &dense(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape)
{
    const Tensor &t = dense(o, name, type);
    if (t.sizes() != shape)
        refuse(PyExc_ValueError,
               std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
    return t;
}

void dims(const Tensor &t, const char *name, int64_t n, const char *form)
{
    if (t.dim() != n)
        refuse(PyExc_ValueError, std::string(name) + " must be " + form + ", got " + text(t.sizes()));
}

int64_t whole(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Refused{};
    return v;
}

int small(PyObject *o, const char *name)
{
    const int64_t v = whole(o);
    if (v < INT32_MIN || v > INT32_MAX)
        refuse(PyExc_ValueError, std::string(name) + " is out of range");
    return (int)v;
}

void *address(PyObject *o)
{
    return o == Py_None ? nullptr : (void *)(uintptr_t)whole(o);
}

void done(int code, const char *what)
{
    if (code != GC_OK)
        refuse(PyExc_RuntimeError, std::string(what) + ": " + gemm_coll_strerror(code) + " (code " +
                                       std::to_string(code) + ")");
}

// Output of shape {rows, cols}: the caller's, or a new one beside `like`.
Tensor output(PyObject *o, const Tensor &like, int64_t rows, int64_t cols)
{
    if (o == Py_None)
        return at::empty({rows, cols}, like.options());
    return dense(o, "out", at::kBFloat16, {rows, cols});
}

// Returns the given output object itself, or the new tensor.
PyObject *give(PyObject *o, Tensor t)
{
    if (o != Py_None) {
        Py_INCREF(o);
        return o;
    }
    return THPVariable_Wrap(std::move(t));
}

// A tensor of its own over part of another's memory, which it keeps alive
// (through the dispatcher a view costs as much as an allocation).
Tensor part(const Tensor &buf, at::ScalarType type, int64_t byte, at::IntArrayRef shape)
{
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(),
                                                        c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(byte / 4);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return t;
}

template <class F>
PyObject *guarded(PyObject *const *a, Py_ssize_t n, Py_ssize_t want, F &&f)
{
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    t_device = -1;
    try {
        return f(a);
    } catch (const Refused &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (logits, k, score, bias, renormalize, scale, stream, workspace, bytes)
PyObject *moe_route(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    return guarded(args, nargs, 9, [](PyObject *const *a) -> PyObject * {
        const Tensor &x = tensor(a[0], "logits");
        const at::ScalarType type = x.scalar_type();
        if (x.dim() != 2 || (type != at::kFloat && type != at::kBFloat16))
            refuse(PyExc_TypeError, std::string("logits must be float32 or bfloat16 [T, E], got ") +
                                        c10::toString(type) + " " + text(x.sizes()));
        here(x, "logits");
        const int64_t T = x.size(0), E = x.size(1);
        const int k = small(a[1], "k");
        if (E > 1 && T > 0 && x.stride(1) != 1)
            refuse(PyExc_ValueError, "logits: the experts of a row must be contiguous");
        if (k < 1 || E < 1 || E > GC_GROUPS_MAX || k > GC_TOPK_MAX)
            done(GC_EINVAL, "moe_route");
        const float *bias = nullptr;
        if (a[3] != Py_None)
            bias = dense(a[3], "bias", at::kFloat, {E}).const_data_ptr<float>();
        const int renormalize = PyObject_IsTrue(a[4]);
        if (renormalize < 0)
            throw Refused{};
        const double scale = PyFloat_AsDouble(a[5]);
        if (scale == -1.0 && PyErr_Occurred())
            throw Refused{};
        // one allocation for the five outputs, each on a 256-byte boundary
        const int64_t pairs = (T * k * 4 + 255) / 256 * 256;
        const Tensor buf = at::empty({pairs + E / 64 * 64 + 64}, x.options().dtype(at::kInt));
        Tensor ids = part(buf, at::kInt, 0, {T, k}), weights = part(buf, at::kFloat, pairs, {T, k});
        Tensor rows = part(buf, at::kInt, 2 * pairs, {T * k}), slots = part(buf, at::kInt, 3 * pairs, {T, k});
        Tensor offsets = part(buf, at::kInt, 4 * pairs, {E + 1});
        done(gemm_coll_moe_route(x.const_data_ptr(), type == at::kBFloat16 ? GC_BF16 : GC_F32,
                                 T > 1 ? x.stride(0) : E, T, (int)E, k, small(a[2], "score"), bias,
                                 renormalize, (float)scale, ids.data_ptr<int32_t>(),
                                 weights.data_ptr<float>(), offsets.data_ptr<int32_t>(),
                                 rows.data_ptr<int32_t>(), slots.data_ptr<int32_t>(), address(a[7]),
                                 (uint64_t)whole(a[8]), address(a[6])),
             "moe_route");
        PyObject *r = PyTuple_New(5);
        if (!r)
            throw Refused{};
        Tensor *all[5] = {&ids, &weights, &offsets, &rows, &slots};
        for (int i = 0; i < 5; ++i)
            PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(*all[i])));
        return r;
    });
}

// (ids, groups, stream, workspace, bytes)
PyObject *group_rows(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    return guarded(args, nargs, 5, [](PyObject *const *a) -> PyObject * {
        const Tensor &t = tensor(a[0], "ids");
        if (t.dim() != 1 && t.dim() != 2)
            refuse(PyExc_ValueError, "ids must be [T] or [T, k], got " + text(t.sizes()));
        const Tensor &ids = dense(a[0], "ids", at::kInt);
        const int64_t T = ids.size(0), k = ids.dim() == 2 ? ids.size(1) : 1;
        const int groups = small(a[1], "groups");
        if (groups < 1 || groups > GC_GROUPS_MAX || k < 1)
            done(GC_EINVAL, "group_rows");
        Tensor offsets = at::empty({groups + 1}, ids.options()), rows = at::empty({T * k}, ids.options());
        Tensor slots = at::empty(ids.sizes(), ids.options());
        done(k > INT32_MAX ? GC_ENOTSUP
                           : gemm_coll_group_rows(ids.const_data_ptr<int32_t>(), T, (int)k, groups,
                                                  offsets.data_ptr<int32_t>(), rows.data_ptr<int32_t>(),
                                                  slots.data_ptr<int32_t>(), address(a[3]),
                                                  (uint64_t)whole(a[4]), address(a[2])),
             "group_rows");
        PyObject *r = PyTuple_New(3);
        if (!r)
            throw Refused{};
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(offsets)));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(rows)));
        PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(slots)));
        return r;
    });
}

// (X, W, offsets, rows, out, act, stream, workspace, bytes)
PyObject *grouped_gemm(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    return guarded(args, nargs, 9, [](PyObject *const *a) -> PyObject * {
        dims(tensor(a[0], "X"), "X", 2, "[T, K]");
        dims(tensor(a[1], "W"), "W", 3, "[E, K, N]");
        const Tensor &X = dense(a[0], "X", at::kBFloat16);
        const int64_t T = X.size(0), K = X.size(1);
        const int64_t E = tensor(a[1], "W").size(0), N = tensor(a[1], "W").size(2);
        const Tensor &W = dense(a[1], "W", at::kBFloat16, {E, K, N});
        const Tensor &offsets = dense(a[2], "offsets", at::kInt, {E + 1});
        const int32_t *rows = nullptr;
        int64_t S = T;
        if (a[3] != Py_None) {
            const Tensor &r = dense(a[3], "rows", at::kInt);
            dims(r, "rows", 1, "[S]");
            rows = r.const_data_ptr<int32_t>();
            S = r.size(0);
        }
        const int act = small(a[5], "act");
        Tensor out = output(a[4], X, S, act == GC_ACT_SILU_GLU ? N / 2 : N);
        done(E > GC_GROUPS_MAX
                 ? GC_EINVAL
                 : gemm_coll_grouped_gemm((const gc_bf16 *)X.const_data_ptr(), T,
                                          (const gc_bf16 *)W.const_data_ptr(),
                                          offsets.const_data_ptr<int32_t>(), rows, S, K, N, (int)E, act,
                                          (gc_bf16 *)out.data_ptr(), address(a[7]), (uint64_t)whole(a[8]),
                                          address(a[6])),
             "grouped_gemm");
        return give(a[4], std::move(out));
    });
}

// (Y, slots, weights, partials, out, stream)
PyObject *moe_combine(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    return guarded(args, nargs, 6, [](PyObject *const *a) -> PyObject * {
        dims(tensor(a[0], "Y"), "Y", 2, "[S, N]");
        dims(tensor(a[1], "slots"), "slots", 2, "[T, k]");
        const Tensor &Y = dense(a[0], "Y", at::kBFloat16);
        const Tensor &slots = dense(a[1], "slots", at::kInt);
        const int64_t S = Y.size(0), N = Y.size(1), T = slots.size(0), k = slots.size(1);
        const Tensor &weights = dense(a[2], "weights", at::kFloat, {T, k});
        const gc_bf16 *pp = nullptr;
        int64_t npeers = 0, stride = 0;
        if (a[3] != Py_None) {
            const Tensor &p = tensor(a[3], "partials");
            if (p.scalar_type() != at::kBFloat16 || p.dim() != 3 || p.size(1) != T || p.size(2) != N)
                refuse(PyExc_ValueError, "partials: expected bf16 [npeers, " + std::to_string(T) + ", " +
                                             std::to_string(N) + "], got " + c10::toString(p.scalar_type()) +
                                             " " + text(p.sizes()));
            if (p.size(0) > 0) {
                // (on another device too, where this one can reach its memory)
                if (!p.is_cuda())
                    refuse(PyExc_ValueError, "partials must be a device tensor");
                if (T * N > 0 && (p.stride(2) != 1 || (T > 1 && p.stride(1) != N)))
                    refuse(PyExc_ValueError, "partials: rows must be contiguous");
                npeers = p.size(0);
                stride = p.stride(0);
                pp = (const gc_bf16 *)p.const_data_ptr();
            }
        }
        Tensor out = output(a[4], Y, T, N);
        done(k > GC_TOPK_MAX || npeers > 15
                 ? GC_EINVAL
                 : gemm_coll_moe_combine((const gc_bf16 *)Y.const_data_ptr(), S,
                                         slots.const_data_ptr<int32_t>(), weights.const_data_ptr<float>(), T,
                                         (int)k, N, pp, (int)npeers, stride, (gc_bf16 *)out.data_ptr(),
                                         address(a[5])),
             "moe_combine");
        return give(a[4], std::move(out));
    });
}

// (base, X, down, up, scale, offsets, rows, out, stream, workspace, bytes)
PyObject *lora_add(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    return guarded(args, nargs, 11, [](PyObject *const *a) -> PyObject * {
        dims(tensor(a[1], "X"), "X", 2, "[M, K]");
        dims(tensor(a[2], "down"), "down", 3, "[G, K, r]");
        dims(tensor(a[3], "up"), "up", 3, "[G, r, N]");
        const Tensor &X = dense(a[1], "X", at::kBFloat16);
        const int64_t M = X.size(0), K = X.size(1);
        const int64_t G = tensor(a[2], "down").size(0), r = tensor(a[2], "down").size(2);
        const int64_t N = tensor(a[3], "up").size(2);
        const Tensor &down = dense(a[2], "down", at::kBFloat16, {G, K, r});
        const Tensor &up = dense(a[3], "up", at::kBFloat16, {G, r, N});
        const Tensor &base = dense(a[0], "base", at::kBFloat16, {M, N});
        const Tensor &scale = dense(a[4], "scale", at::kFloat, {G});
        const Tensor &offsets = dense(a[5], "offsets", at::kInt, {G + 1});
        const Tensor &rows = dense(a[6], "rows", at::kInt, {M});
        Tensor out = output(a[7], base, M, N);
        done(G >= GC_GROUPS_MAX || r > 128
                 ? GC_EINVAL
                 : gemm_coll_lora_add((const gc_bf16 *)base.const_data_ptr(),
                                      (const gc_bf16 *)X.const_data_ptr(),
                                      (const gc_bf16 *)down.const_data_ptr(),
                                      (const gc_bf16 *)up.const_data_ptr(), scale.const_data_ptr<float>(),
                                      offsets.const_data_ptr<int32_t>(), rows.const_data_ptr<int32_t>(), M, K,
                                      N, (int)r, (int)G, (gc_bf16 *)out.data_ptr(), address(a[9]),
                                      (uint64_t)whole(a[10]), address(a[8])),
             "lora_add");
        return give(a[7], std::move(out));
    });
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(moe_route), FAST(group_rows), FAST(grouped_gemm), FAST(moe_combine),
                         FAST(lora_add), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr,
                          nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module_def); }
