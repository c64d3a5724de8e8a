// Checks and reads torch tensors for the Python binding (the table of
// ks_adamw_step, the arguments of the adapter calls): type, device, contiguity,
// shape and address of each tensor through the DLPack exchange functions that
// torch.Tensor publishes (__dlpack_c_exchange_api__), so that no torch type is
// needed here.  The same checks as attribute reads from Python take 18 us for a
// list of 60 tensors, an order of magnitude more than here, and a step has up to
// seven lists; for one adapter call they take half of a single token's time.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>

#include <cstdint>
#include <cstring>

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

const char *const kNames[7] = {"params", "grads", "exp_avgs", "exp_avg_sqs", "masters", "exp_avg_scales",
                               "exp_avg_sq_scales"};
constexpr int64_t kBlock = 256;  // elements that share a scale in an 8-bit state

// adamw_table(params, grads, exp_avgs, exp_avg_sqs, masters, exp_avg_scales, exp_avg_sq_scales)
//   -> (table, tensors, dtype kind, state kind, device index, its current stream)
// Lists of equal lengths; the last three may be None.
PyObject *adamw_table(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs != 7) return PyErr_Format(PyExc_TypeError, "adamw_table takes 7 lists");
    PyObject *list[7] = {}, *table = nullptr, *result = nullptr;
    Py_ssize_t count = 0;
    int dtype = kNone, state = kNone, device = -1;
    uint64_t *words = nullptr;
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
    table = PyBytes_FromStringAndSize(nullptr, count * 64);  // ks_adamw_tensor: eight 64-bit words
    if (!table) goto done;
    words = reinterpret_cast<uint64_t *>(PyBytes_AS_STRING(table));
    memset(words, 0, (size_t)count * 64);
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
                words[8 * k + 7] = (uint64_t)t.numel;
            } else {
                const int64_t n = (int64_t)words[8 * k + 7];
                if (t.numel != (c < 5 ? n : (n + kBlock - 1) / kBlock)) {
                    PyErr_Format(PyExc_ValueError,
                                 "%s must have the parameters' element counts (scales: one for each 256)", kNames[c]);
                    goto done;
                }
            }
            words[8 * k + c] = t.ptr;
        }
    }
    if (current_stream(device, &stream)) result = Py_BuildValue("OniiiK", table, count, dtype, state, device, stream);
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

// The integers of args[0 .. n); false with an error set.
bool integers(PyObject *const *args, int n, long long *out) {
    for (int k = 0; k < n; ++k) {
        out[k] = PyLong_AsLongLong(args[k]);
        if (out[k] == -1 && PyErr_Occurred()) return false;
    }
    return true;
}

// adapter_args(x, values, A, B, ids, scales, bias, width, in_f, out_f, nvals, name)
//   -> (rows, adapters, rank, dtype kind, device, its current stream, x, values, A, B, ids, scales, bias)
// The addresses of tensors that are None are 0.
PyObject *adapter_args(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs != 12) return PyErr_Format(PyExc_TypeError, "adapter_args takes 12 arguments");
    long long size[4];
    Info t[7];
    const char *name = PyUnicode_AsUTF8(args[11]);
    if (!name || !integers(args + 7, 4, size) || !check_adapters(args, size[0], size[1], size[2], size[3], name, t))
        return nullptr;
    unsigned long long stream = 0;
    if (!current_stream(t[0].device, &stream)) return nullptr;
    return Py_BuildValue("LLLiiKKKKKKKK", (long long)t[0].shape[0], (long long)t[2].shape[0], (long long)t[2].shape[1],
                         t[0].kind, t[0].device, stream, (unsigned long long)t[0].ptr, (unsigned long long)t[1].ptr,
                         (unsigned long long)t[2].ptr, (unsigned long long)t[3].ptr, (unsigned long long)t[4].ptr,
                         (unsigned long long)t[5].ptr, (unsigned long long)t[6].ptr);
}

// adapter_matmul(function, x, values, A, B, ids, scales, bias, out, a, b, c, d, activation, dtypes, stream)
//   -> (status, out)
// Checks the tensors, makes out (None: a new tensor) and calls ks_adapter_matmul
// (function: its address).  dtypes: (ks_dtype of float32 tensors, of bfloat16 ones or
// -1); stream: None for the current one.  Through ctypes the call alone takes 2 us more.
using AdapterMatmul = int (*)(const void *, const void *, int64_t, int64_t, int64_t, int64_t, int64_t, void *, int,
                              const void *, int, const void *, const void *, const float *, const int32_t *, int64_t,
                              int64_t, void *);
PyObject *adapter_matmul(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs != 16) return PyErr_Format(PyExc_TypeError, "adapter_matmul takes 16 arguments");
    const auto function = reinterpret_cast<AdapterMatmul>(PyLong_AsVoidPtr(args[0]));
    if (!function) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "no function");
    long long n[5];  // a, b, c, d, activation
    int dtypes[2];
    if (!integers(args + 9, 5, n) || !PyArg_ParseTuple(args[14], "ii", &dtypes[0], &dtypes[1])) return nullptr;
    long long in_f, out_f, nvals;
    if (__builtin_mul_overflow(n[0], n[3], &out_f) || __builtin_mul_overflow(out_f, n[2], &in_f) ||
        __builtin_mul_overflow(out_f, n[1], &out_f) || __builtin_mul_overflow(in_f, n[1], &nvals))
        return PyErr_Format(PyExc_ValueError, "the pattern's sizes overflow");
    Info t[7];
    if (!check_adapters(args + 1, in_f, in_f, out_f, nvals, "x", t)) return nullptr;
    const Info &x = t[0];
    const int dtype = dtypes[x.kind == kBF16];
    if (dtype < 0) return PyErr_Format(PyExc_ValueError, "tf32 applies to fp32 tensors only");
    unsigned long long stream = 0;
    if (args[15] == Py_None) {
        if (!current_stream(x.device, &stream)) return nullptr;
    } else {
        stream = PyLong_AsUnsignedLongLong(args[15]);
        if (PyErr_Occurred()) return nullptr;
    }
    PyObject *out = nullptr;
    if (args[8] == Py_None) {
        PyObject *shape = Py_BuildValue("((LL))", (long long)x.shape[0], out_f);
        PyObject *make = shape ? PyObject_GetAttrString(args[1], "new_empty") : nullptr;
        if (make) out = PyObject_CallObject(make, shape);
        Py_XDECREF(make);
        Py_XDECREF(shape);
    } else {
        out = args[8];
        Py_INCREF(out);
    }
    if (!out) return nullptr;
    Info y;
    if (!read(out, &y)) {
        Py_DECREF(out);
        return nullptr;
    }
    if (y.kind != x.kind || y.device != x.device || !y.contiguous || y.ndim != 2 || y.shape[0] != x.shape[0] ||
        y.shape[1] != out_f) {
        Py_DECREF(out);
        return PyErr_Format(PyExc_ValueError, "out must be a contiguous (%lld, %lld) tensor with x's dtype and device",
                            (long long)x.shape[0], out_f);
    }
    const auto ptr = [](const Info &o) { return reinterpret_cast<void *>((uintptr_t)o.ptr); };
    int status = 0;
    Py_BEGIN_ALLOW_THREADS
    status = function(ptr(x), ptr(t[1]), n[0], n[1], n[2], n[3], x.shape[0], ptr(y), dtype, ptr(t[6]), (int)n[4],
                      ptr(t[2]), ptr(t[3]), static_cast<const float *>(ptr(t[5])), static_cast<const int32_t *>(ptr(t[4])),
                      t[2].shape[0], t[2].shape[1], reinterpret_cast<void *>((uintptr_t)stream));
    Py_END_ALLOW_THREADS
    return Py_BuildValue("iN", status, out);
}

PyMethodDef kMethods[] = {
    {"adapter_args", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(adapter_args)), METH_FASTCALL,
     "Checked arguments of an adapter call."},
    {"adapter_matmul", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(adapter_matmul)), METH_FASTCALL,
     "ks_adapter_matmul on torch tensors."},
    {"adamw_table", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(adamw_table)), METH_FASTCALL,
     "The table of ks_adamw_step from lists of tensors."},
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
