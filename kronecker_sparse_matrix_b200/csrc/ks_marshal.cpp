// The calls of the Python binding whose own time counts (adapters, AdamW): checks and
// reads torch tensors and calls the library.  Type, device, contiguity, shape and
// address of each tensor come through the DLPack exchange functions that torch.Tensor
// publishes (__dlpack_c_exchange_api__), so that no torch type is needed here.  The same
// checks as attribute reads from Python take 18 us for a list of 60 tensors, an order of
// magnitude more than here, and a step has up to seven lists; for one adapter call they
// take half of a single token's time.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>

#include <cstdint>
#include <cstring>

#include "ks.h"

namespace {

const DLPackExchangeAPI *g_api = nullptr;
PyTypeObject *g_tensor = nullptr;

// Type codes of the table: what ks_dtype and state_bits are chosen by.
enum Kind { kNone = -1, kF32 = 0, kBF16 = 1, kE4M3 = 2, kI32 = 3 };

int kind_of(const DLDataType &t) {
    if (t.lanes != 1) return kNone;
    if (t.code == kDLFloat && t.bits == 32) return kF32;
    if (t.code == kDLBfloat && t.bits == 16) return kBF16;
    if (t.code == kDLInt && t.bits == 32) return kI32;
    if (t.code == kDLFloat8_e4m3fn && t.bits == 8) return kE4M3;
    return kNone;
}

const char *kind_name(int k) {
    return k == kF32 ? "torch.float32" : k == kBF16 ? "torch.bfloat16" : k == kE4M3 ? "torch.float8_e4m3fn" : "other";
}

struct Info {
    uint64_t ptr;
    int64_t numel;
    int kind, device;  // device: CUDA index, or -1
    int ndim;
    int64_t shape[3];  // of the first three dimensions
    bool contiguous;
};

bool read(PyObject *o, Info *out) {
    if (!PyObject_TypeCheck(o, g_tensor)) {
        PyErr_SetString(PyExc_TypeError, "expected torch tensors");
        return false;
    }
    DLTensor t;
    if (g_api->dltensor_from_py_object_no_sync(o, &t) != 0) return false;
    out->ptr = (uint64_t)(uintptr_t)t.data + t.byte_offset;
    out->kind = kind_of(t.dtype);
    out->device = t.device.device_type == kDLCUDA ? t.device.device_id : -1;
    int64_t n = 1;
    bool c = true;
    for (int d = t.ndim - 1; d >= 0; --d) {
        if (t.strides && t.shape[d] > 1 && t.strides[d] != n) c = false;
        n *= t.shape[d];
    }
    out->ndim = t.ndim;
    for (int d = 0; d < 3; ++d) out->shape[d] = d < t.ndim ? t.shape[d] : 1;
    out->numel = n;
    out->contiguous = c || n == 0;
    return true;
}

// The current stream of a CUDA device, as torch has it; false with an error set.
bool current_stream(int device, unsigned long long *out) {
    void *st = nullptr;
    if (g_api->current_work_stream(kDLCUDA, device, &st) != 0) return false;
    *out = (unsigned long long)(uintptr_t)st;
    return true;
}

// The integers of args[0 .. n); false with an error set.
bool integers(PyObject *const *args, int n, long long *out) {
    for (int k = 0; k < n; ++k) {
        out[k] = PyLong_AsLongLong(args[k]);
        if (out[k] == -1 && PyErr_Occurred()) return false;
    }
    return true;
}

// The sizes of a pattern's product.
struct Sizes {
    long long in_f, out_f, nvals;
};
bool sizes_of(const long long *p, Sizes *o) {
    if (__builtin_mul_overflow(p[0], p[3], &o->out_f) || __builtin_mul_overflow(o->out_f, p[2], &o->in_f) ||
        __builtin_mul_overflow(o->out_f, p[1], &o->out_f) || __builtin_mul_overflow(o->in_f, p[1], &o->nvals)) {
        PyErr_SetString(PyExc_ValueError, "the pattern's sizes overflow");
        return false;
    }
    return true;
}

// The ks_dtype of tensors of kind k from a pair (of float32 tensors, of bfloat16 ones or -1).
bool dtype_of(PyObject *pair, int k, int *out) {
    int d[2];
    if (!PyArg_ParseTuple(pair, "ii", &d[0], &d[1])) return false;
    *out = d[k == kBF16];
    if (*out < 0) PyErr_SetString(PyExc_ValueError, "tf32 applies to fp32 tensors only");
    return *out >= 0;
}

// The stream of a call: the handle given, or for None the device's current one.
bool stream_of(PyObject *given, int device, unsigned long long *out) {
    if (given == Py_None) return current_stream(device, out);
    *out = PyLong_AsUnsignedLongLong(given);
    return !PyErr_Occurred();
}

// A new tensor of the given shape with the dtype and device of `like`.
PyObject *new_empty(PyObject *like, const int64_t *shape, int ndim, Info *info) {
    PyObject *args = ndim == 2 ? Py_BuildValue("((LL))", (long long)shape[0], (long long)shape[1])
                               : Py_BuildValue("((LLL))", (long long)shape[0], (long long)shape[1], (long long)shape[2]);
    PyObject *make = args ? PyObject_GetAttrString(like, "new_empty") : nullptr;
    PyObject *out = make ? PyObject_CallObject(make, args) : nullptr;
    Py_XDECREF(make);
    Py_XDECREF(args);
    if (out && !read(out, info)) Py_CLEAR(out);
    return out;
}

void *address(const Info &o) { return reinterpret_cast<void *>((uintptr_t)o.ptr); }

const char *const kNames[7] = {"params", "grads", "exp_avgs", "exp_avg_sqs", "masters", "exp_avg_scales",
                               "exp_avg_sq_scales"};
constexpr int64_t kBlock = 256;  // elements that share a scale in an 8-bit state

// The buffer of list c (kNames) of a tensor.
void set_buffer(ks_adamw_tensor *t, int c, void *p) {
    switch (c) {
        case 0: t->param = p; break;
        case 1: t->grad = p; break;
        case 2: t->exp_avg = p; break;
        case 3: t->exp_avg_sq = p; break;
        case 4: t->master = static_cast<float *>(p); break;
        case 5: t->exp_avg_scale = static_cast<float *>(p); break;
        default: t->exp_avg_sq_scale = static_cast<float *>(p); break;
    }
}

// A tensor of one element of the given type (kind kNone: int64) on the device, or false with an error set.
template <typename T>
bool scalar_of(PyObject *o, const char *name, int kind, int device, const T **out) {
    Info t;
    DLTensor d;
    if (!read(o, &t) || g_api->dltensor_from_py_object_no_sync(o, &d) != 0) return false;
    const bool type = kind == kNone ? d.dtype.code == kDLInt && d.dtype.bits == 64 && d.dtype.lanes == 1 : t.kind == kind;
    if (!type || t.device != device || t.numel != 1) {
        PyErr_Format(PyExc_ValueError, "%s as a tensor must hold one %s on cuda:%d", name,
                     kind == kNone ? "torch.int64" : kind_name(kind), device);
        return false;
    }
    *out = reinterpret_cast<const T *>((uintptr_t)t.ptr);
    return true;
}

// A step's numbers, args: lr, step, grad_scale (each a number or a tensor; grad_scale may be
// None), beta1, beta2, eps, weight_decay.
bool options_of(PyObject *const *args, int device, ks_adamw_options *o) {
    *o = ks_adamw_options{};
    double *const number[4] = {&o->beta1, &o->beta2, &o->eps, &o->weight_decay};
    for (int k = 0; k < 4; ++k) {
        *number[k] = PyFloat_AsDouble(args[3 + k]);
        if (PyErr_Occurred()) return false;
    }
    if (PyObject_TypeCheck(args[0], g_tensor)) {
        if (!scalar_of(args[0], "lr", kF32, device, &o->lr_ptr)) return false;
    } else {
        o->lr = PyFloat_AsDouble(args[0]);
    }
    if (PyErr_Occurred()) return false;
    if (PyObject_TypeCheck(args[1], g_tensor)) {
        if (!scalar_of(args[1], "step", kNone, device, &o->step_ptr)) return false;
    } else {
        o->step = PyLong_AsLongLong(args[1]);
    }
    if (PyErr_Occurred()) return false;
    return args[2] == Py_None || scalar_of(args[2], "grad_scale", kF32, device, &o->grad_scale);
}

// adamw_step(function, params, grads, exp_avgs, exp_avg_sqs, masters, exp_avg_scales, exp_avg_sq_scales,
//            lr, step, grad_scale, beta1, beta2, eps, weight_decay, dtypes, stream) -> status
// Checks the tensors and numbers and calls ks_adamw_step (function: its address;
// dtypes and stream: dtype_of, stream_of).  Lists of equal lengths; masters and scales may be None.
PyObject *adamw_step(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs != 17) return PyErr_Format(PyExc_TypeError, "adamw_step takes 17 arguments");
    const auto function = reinterpret_cast<decltype(&ks_adamw_step)>(PyLong_AsVoidPtr(args[0]));
    if (!function) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "no function");
    PyObject *const *const options = args + 8;
    ++args;
    PyObject *list[7] = {}, *table = nullptr, *result = nullptr;
    ks_adamw_options opt;
    int ks_dtype = 0, status = 0;
    Py_ssize_t count = 0;
    int dtype = kNone, state = kNone, device = -1;
    ks_adamw_tensor *tensors = nullptr;
    unsigned long long stream = 0;
    for (int c = 0; c < 7; ++c) {
        if (args[c] == Py_None && c >= 4) continue;
        list[c] = PySequence_Fast(args[c], "expected lists of tensors");
        if (!list[c]) goto done;
        if (c == 0) {
            count = PySequence_Fast_GET_SIZE(list[0]);
        } else if (PySequence_Fast_GET_SIZE(list[c]) != count) {
            PyErr_Format(PyExc_ValueError, "%s must have one tensor for each parameter", kNames[c]);
            goto done;
        }
    }
    table = PyBytes_FromStringAndSize(nullptr, count * (Py_ssize_t)sizeof(ks_adamw_tensor));
    if (!table) goto done;
    tensors = reinterpret_cast<ks_adamw_tensor *>(PyBytes_AS_STRING(table));
    memset(static_cast<void *>(tensors), 0, (size_t)count * sizeof(ks_adamw_tensor));
    for (int c = 0; c < 7; ++c) {
        if (!list[c]) continue;
        PyObject **items = PySequence_Fast_ITEMS(list[c]);
        for (Py_ssize_t k = 0; k < count; ++k) {
            Info t;
            if (!read(items[k], &t)) goto done;
            if (c == 0 && k == 0) {
                dtype = t.kind;
                device = t.device;
                if (dtype != kF32 && dtype != kBF16) {
                    PyErr_SetString(PyExc_TypeError, "unsupported dtype of params: use float32 or bfloat16");
                    goto done;
                }
                if (device < 0) {
                    PyErr_SetString(PyExc_ValueError, "params must be CUDA tensors");
                    goto done;
                }
            }
            if (c == 2 && k == 0) {
                state = t.kind;
                if (state != kF32 && state != kE4M3) {
                    PyErr_SetString(PyExc_TypeError, "unsupported dtype of exp_avgs: use float32 or float8_e4m3fn");
                    goto done;
                }
            }
            const int want = c < 2 ? dtype : c < 4 ? state : kF32;
            if (t.kind != want || t.device != device) {
                PyErr_Format(PyExc_ValueError, "%s must be %s tensors on cuda:%d", kNames[c], kind_name(want), device);
                goto done;
            }
            if (!t.contiguous) {
                PyErr_Format(PyExc_ValueError, "%s must be contiguous", kNames[c]);
                goto done;
            }
            if (c == 0) {
                tensors[k].n = t.numel;
            } else {
                const int64_t n = tensors[k].n;
                if (t.numel != (c < 5 ? n : (n + kBlock - 1) / kBlock)) {
                    PyErr_Format(PyExc_ValueError,
                                 "%s must have the parameters' element counts (scales: one for each 256)", kNames[c]);
                    goto done;
                }
            }
            set_buffer(&tensors[k], c, address(t));
        }
    }
    if (count == 0) {
        result = PyLong_FromLong(0);
        goto done;
    }
    if ((state == kE4M3) != (list[5] != nullptr) || (list[5] != nullptr) != (list[6] != nullptr)) {
        PyErr_SetString(PyExc_ValueError,
                        "8-bit states need exp_avg_scales and exp_avg_sq_scales, 32-bit states take none");
        goto done;
    }
    if (!options_of(options, device, &opt) || !dtype_of(options[7], dtype, &ks_dtype) ||
        !stream_of(options[8], device, &stream))
        goto done;
    Py_BEGIN_ALLOW_THREADS
    status = function(tensors, count, ks_dtype, state == kE4M3 ? 8 : 32, &opt, reinterpret_cast<void *>((uintptr_t)stream));
    Py_END_ALLOW_THREADS
    result = PyLong_FromLong(status);
done:
    Py_XDECREF(table);
    for (PyObject *l : list) Py_XDECREF(l);
    return result;
}

// Reads and checks the tensors of an adapter call, args: x, values, A, B, ids, scales, bias.
// x: (rows, width), called `name` in messages; values, ids, scales and bias may be None.
bool check_adapters(PyObject *const *args, long long width, long long in_f, long long out_f, long long nvals,
                    const char *name, Info (&t)[7]) {
    for (int k = 0; k < 7; ++k) {
        t[k] = Info{};
        if (args[k] == Py_None && k != 0 && k != 2 && k != 3) continue;
        if (!read(args[k], &t[k])) return false;
    }
    const Info &x = t[0], &A = t[2], &B = t[3];
    const auto given = [&](int k) { return args[k] != Py_None; };
    const auto like_x = [&](const Info &o) { return o.kind == x.kind && o.device == x.device && o.contiguous; };
    const long long s = A.shape[0], r = A.shape[1];
    if (x.kind != kF32 && x.kind != kBF16)
        PyErr_Format(PyExc_TypeError, "unsupported dtype of %s: use float32 or bfloat16", name);
    else if (x.ndim != 2 || x.device < 0 || !x.contiguous || x.shape[1] != width)
        PyErr_Format(PyExc_ValueError, "%s must be a contiguous CUDA tensor of shape (batch, %lld)", name, width);
    else if (A.ndim != 3 || A.shape[2] != in_f || s == 0 || r == 0)
        PyErr_Format(PyExc_ValueError, "A must have shape (adapters, rank, %lld)", in_f);
    else if (B.ndim != 3 || B.shape[0] != s || B.shape[1] != out_f || B.shape[2] != r)
        PyErr_Format(PyExc_ValueError, "B must have shape (%lld, %lld, %lld)", s, out_f, r);
    else if (!like_x(A) || !like_x(B) || (given(1) && !like_x(t[1])))
        PyErr_Format(PyExc_ValueError, "values, A and B must be contiguous, with %s's dtype and device", name);
    else if (given(1) && t[1].numel != nvals)
        PyErr_Format(PyExc_ValueError, "values must have %lld elements", nvals);
    else if (given(4) && (t[4].kind != kI32 || t[4].device != x.device || t[4].ndim != 1 ||
                          t[4].shape[0] != x.shape[0] || !t[4].contiguous))
        PyErr_SetString(PyExc_ValueError,
                        "ids must be a contiguous int32 tensor with one entry per row, on the same device");
    else if (given(5) && (t[5].kind != kF32 || t[5].device != x.device || t[5].ndim != 1 || t[5].shape[0] != s ||
                          !t[5].contiguous))
        PyErr_SetString(PyExc_ValueError,
                        "scales must be a contiguous float32 tensor with one entry per adapter, on the same device");
    else if (given(6) && (!like_x(t[6]) || t[6].numel != out_f))
        PyErr_Format(PyExc_ValueError, "bias must be a contiguous tensor of %lld elements with x's dtype and device",
                     out_f);
    else
        return true;
    return false;
}

// adapter_matmul(function, x, values, A, B, ids, scales, bias, out, a, b, c, d, activation, dtypes, stream)
//   -> (status, out)
// Checks the tensors, makes out (None: a new tensor) and calls ks_adapter_matmul
// (function: its address; dtypes and stream: dtype_of, stream_of).  Through ctypes the
// call alone takes 2 us more.
PyObject *adapter_matmul(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs != 16) return PyErr_Format(PyExc_TypeError, "adapter_matmul takes 16 arguments");
    const auto function = reinterpret_cast<decltype(&ks_adapter_matmul)>(PyLong_AsVoidPtr(args[0]));
    if (!function) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "no function");
    long long n[5];  // a, b, c, d, activation
    Sizes z;
    Info t[7], y;
    int dtype = 0;
    unsigned long long stream = 0;
    if (!integers(args + 9, 5, n) || !sizes_of(n, &z) ||
        !check_adapters(args + 1, z.in_f, z.in_f, z.out_f, z.nvals, "x", t) || !dtype_of(args[14], t[0].kind, &dtype) ||
        !stream_of(args[15], t[0].device, &stream))
        return nullptr;
    const Info &x = t[0];
    const int64_t shape[2] = {x.shape[0], z.out_f};
    PyObject *out = args[8];
    if (out == Py_None) {
        out = new_empty(args[1], shape, 2, &y);
        if (!out) return nullptr;
    } else {
        if (!read(out, &y)) return nullptr;
        if (y.kind != x.kind || y.device != x.device || !y.contiguous || y.ndim != 2 || y.shape[0] != shape[0] ||
            y.shape[1] != shape[1])
            return PyErr_Format(PyExc_ValueError, "out must be a contiguous (%lld, %lld) tensor with x's dtype and device",
                                (long long)shape[0], (long long)shape[1]);
        Py_INCREF(out);
    }
    int status = 0;
    Py_BEGIN_ALLOW_THREADS
    status = function(address(x), address(t[1]), n[0], n[1], n[2], n[3], x.shape[0], address(y), dtype, address(t[6]),
                      (int)n[4], address(t[2]), address(t[3]), static_cast<const float *>(address(t[5])),
                      static_cast<const int32_t *>(address(t[4])), t[2].shape[0], t[2].shape[1],
                      reinterpret_cast<void *>((uintptr_t)stream));
    Py_END_ALLOW_THREADS
    return Py_BuildValue("iN", status, out);
}

// adapter_backward(function, dy, values, A, B, ids, scales, x, a, b, c, d, need_dx, need_da, need_db, dtypes, stream)
//   -> (status, dx, da, db)
// The same for ks_adapter_backward; gradients that are not needed are None.
PyObject *adapter_backward(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs != 17) return PyErr_Format(PyExc_TypeError, "adapter_backward takes 17 arguments");
    const auto function = reinterpret_cast<decltype(&ks_adapter_backward)>(PyLong_AsVoidPtr(args[0]));
    if (!function) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "no function");
    long long n[4];
    Sizes z;
    Info t[7], x{}, g[3] = {};
    int dtype = 0, need[3];
    unsigned long long stream = 0;
    for (int k = 0; k < 3; ++k)
        if ((need[k] = PyObject_IsTrue(args[12 + k])) < 0) return nullptr;
    PyObject *const in[7] = {args[1], args[2], args[3], args[4], args[5], args[6], Py_None};
    if (!integers(args + 8, 4, n) || !sizes_of(n, &z) ||
        !check_adapters(in, z.out_f, z.in_f, z.out_f, z.nvals, "dy", t) || !dtype_of(args[15], t[0].kind, &dtype) ||
        !stream_of(args[16], t[0].device, &stream))
        return nullptr;
    const Info &dy = t[0];
    if (need[0] && args[2] == Py_None) return PyErr_Format(PyExc_ValueError, "dX needs the values");
    if (need[1] || need[2]) {
        if (args[7] != Py_None && !read(args[7], &x)) return nullptr;
        if (args[7] == Py_None || x.ndim != 2 || x.shape[0] != dy.shape[0] || x.shape[1] != z.in_f ||
            x.kind != dy.kind || x.device != dy.device || !x.contiguous)
            return PyErr_Format(PyExc_ValueError, "x must be a contiguous (%lld, %lld) tensor with dy's dtype and device",
                                (long long)dy.shape[0], z.in_f);
    }
    const int64_t shape[3][3] = {{dy.shape[0], z.in_f, 0},
                                 {t[2].shape[0], t[2].shape[1], t[2].shape[2]},
                                 {t[3].shape[0], t[3].shape[1], t[3].shape[2]}};
    PyObject *grad[3] = {};
    for (int k = 0; k < 3; ++k) {
        grad[k] = need[k] ? new_empty(args[1], shape[k], k ? 3 : 2, &g[k]) : Py_NewRef(Py_None);
        if (!grad[k]) {
            for (int j = 0; j < k; ++j) Py_DECREF(grad[j]);
            return nullptr;
        }
    }
    int status = 0;
    Py_BEGIN_ALLOW_THREADS
    status = function(address(dy), address(x), address(t[1]), n[0], n[1], n[2], n[3], dy.shape[0], dtype, address(t[2]),
                      address(t[3]), static_cast<const float *>(address(t[5])),
                      static_cast<const int32_t *>(address(t[4])), t[2].shape[0], t[2].shape[1], address(g[0]),
                      address(g[1]), address(g[2]), reinterpret_cast<void *>((uintptr_t)stream));
    Py_END_ALLOW_THREADS
    return Py_BuildValue("iNNN", status, grad[0], grad[1], grad[2]);
}

PyMethodDef kMethods[] = {
    {"adapter_matmul", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(adapter_matmul)), METH_FASTCALL,
     "ks_adapter_matmul on torch tensors."},
    {"adapter_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(adapter_backward)), METH_FASTCALL,
     "ks_adapter_backward on torch tensors."},
    {"adamw_step", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(adamw_step)), METH_FASTCALL,
     "ks_adamw_step on lists of torch tensors."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ks_marshal", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__ks_marshal(void) {
    PyObject *torch = PyImport_ImportModule("torch");
    if (!torch) return nullptr;
    PyObject *type = PyObject_GetAttrString(torch, "Tensor");
    Py_DECREF(torch);
    if (!type) return nullptr;
    PyObject *capsule = PyObject_GetAttrString(type, "__dlpack_c_exchange_api__");
    if (!capsule) {
        Py_DECREF(type);
        return nullptr;
    }
    const auto *api = static_cast<const DLPackExchangeAPI *>(PyCapsule_GetPointer(capsule, "dlpack_exchange_api"));
    Py_DECREF(capsule);
    if (api && (api->header.version.major != DLPACK_MAJOR_VERSION || !api->dltensor_from_py_object_no_sync ||
                !api->current_work_stream)) {
        PyErr_SetString(PyExc_ImportError, "torch's DLPack exchange functions have another version than this build");
        api = nullptr;
    }
    if (!api) {
        Py_DECREF(type);
        return nullptr;
    }
    g_api = api;
    g_tensor = reinterpret_cast<PyTypeObject *>(type);  // kept
    return PyModule_Create(&kModule);
}
