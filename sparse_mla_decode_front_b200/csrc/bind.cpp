// Native argument marshalling of the routed experts' Python binding (experts.py): the same
// checks that the ctypes binding makes (device, dtype, contiguity, shape), the tensors'
// addresses and torch's current stream, then one call of the C ABI. A decode loop makes these
// calls by the thousand, and the smallest kernels take 2 to 4 us: with the checks in Python and
// ctypes a loop of calls ran at 6.5 us (quantise, gather of one token) to 9 us (sort) a call, with
// these at 3.0 to 4.3, which is the launch and the kernel.
//
// Every function takes positional arguments (experts.py gives them their names, defaults and
// documentation) and returns the C ABI's code; what does not fit raises ValueError. The entry
// points' addresses come from the library that _lib.lib() loaded (set_entries).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "moe_experts.h"

namespace {

using at::ScalarType;

struct Entries {
    decltype(&mla_moe_sort) sort;
    decltype(&mla_moe_gather) gather;
    decltype(&mla_moe_combine) combine;
    decltype(&mla_moe_combine_backward) combine_backward;
    decltype(&mla_fp8_quantize) quantize;
    decltype(&mla_fp8_matmul) matmul;
    decltype(&mla_fp8_grouped_matmul) grouped_matmul;
} g_entry;

struct Refused {};   // a Python error is set

std::string text_of(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}
const char* name_of(ScalarType t) {
    switch (t) {
        case ScalarType::Float: return "torch.float32";
        case ScalarType::Half: return "torch.float16";
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Int: return "torch.int32";
        case ScalarType::Byte: return "torch.uint8";
        case ScalarType::Float8_e4m3fn: return "torch.float8_e4m3fn";
        default: return c10::toString(t);
    }
}

// A tensor argument that must be there.
const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_ValueError, "%s is %s, expected a tensor", name, o == Py_None ? "None" : Py_TYPE(o)->tp_name);
        throw Refused();
    }
    return THPVariable_Unpack(o);
}
// One that gives a call some of its sizes: its rank, and sizes that fit the ABI's.
const at::Tensor& sized(const char* name, PyObject* o, int dims) {
    const at::Tensor& t = tensor(name, o);
    if (t.dim() != dims) {
        PyErr_Format(PyExc_ValueError, "%s must have %d dimensions, got shape %s", name, dims, text_of(t.sizes()).c_str());
        throw Refused();
    }
    for (const int64_t d : t.sizes())
        if (d > INT32_MAX) {
            PyErr_Format(PyExc_ValueError, "%s has shape %s: a dimension is beyond the library's 32-bit sizes", name,
                         text_of(t.sizes()).c_str());
            throw Refused();
        }
    return t;
}
// The device of a call: its first tensor's.
int device_of(const char* name, const at::Tensor& t) {
    if (!t.is_cuda()) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
        throw Refused();
    }
    return t.get_device();
}
int dtype_code(const char* name, const at::Tensor& t) {
    switch (t.scalar_type()) {
        case ScalarType::BFloat16: return MLA_DTYPE_BF16;
        case ScalarType::Half: return MLA_DTYPE_FP16;
        case ScalarType::Float: return MLA_DTYPE_FP32;
        default:
            PyErr_Format(PyExc_ValueError, "%s must be bfloat16, float16 or float32, got %s", name,
                         name_of(t.scalar_type()));
            throw Refused();
    }
}
// The tensor's address after every check.
template <class T = void>
T* address(const char* name, PyObject* o, ScalarType type, std::initializer_list<int64_t> shape, int dev) {
    const at::Tensor& t = tensor(name, o);
    const at::IntArrayRef want(shape.begin(), shape.size());
    if (!t.is_cuda())
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
    else if (t.scalar_type() != type)
        PyErr_Format(PyExc_ValueError, "%s must be %s, got %s", name, name_of(type), name_of(t.scalar_type()));
    else if (t.sizes() != want)
        PyErr_Format(PyExc_ValueError, "%s has shape %s, expected %s", name, text_of(t.sizes()).c_str(),
                     text_of(want).c_str());
    else if (t.get_device() != dev)
        PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, expected cuda:%d", name, (int)t.get_device(), dev);
    else if (!t.is_contiguous())
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    else
        return static_cast<T*>(t.data_ptr());
    throw Refused();
}
template <class T = void>
T* optional(const char* name, PyObject* o, ScalarType type, std::initializer_list<int64_t> shape, int dev) {
    return o == Py_None ? nullptr : address<T>(name, o, type, shape, dev);
}

int int_of(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "an integer argument is beyond the library's 32 bits");
        throw Refused();
    }
    return (int)v;
}
bool truth_of(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v != 0;
}
float float_of(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return (float)v;
}
int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

// `stream`: None (torch's current one of the device), a torch stream, or a handle.
void* stream_of(PyObject* o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
    if (!handle) {
        PyErr_Clear();
        handle = o;
        Py_INCREF(handle);
    }
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!p && PyErr_Occurred()) throw Refused();
    return p;
}

// Run `call` with `dev` current and without the interpreter's lock (a launch can block).
template <class F>
PyObject* run(int dev, F call) {
    int rc;
    PyThreadState* state = PyEval_SaveThread();
    try {
        const int before = c10::cuda::current_device();
        if (before != dev) c10::cuda::set_device((c10::DeviceIndex)dev);
        rc = call();
        if (before != dev) c10::cuda::set_device((c10::DeviceIndex)before);
    } catch (...) {
        PyEval_RestoreThread(state);
        throw;
    }
    PyEval_RestoreThread(state);
    return PyLong_FromLong(rc);
}

PyObject* do_sort(PyObject* const* a) {
    const at::Tensor& idx = sized("topk_idx", a[0], 2);
    const int dev = device_of("topk_idx", idx);
    const int64_t T = idx.size(0), K = idx.size(1), E = sized("expert_offsets", a[1], 1).size(0) - 1;
    int64_t total = 0, ws_bytes = 0;
    const void* aff = nullptr;
    float* w = nullptr;
    void* ws = nullptr;
    if ((a[6] == Py_None) != (a[7] == Py_None)) {
        PyErr_SetString(PyExc_ValueError, "affinities and weights come together");
        throw Refused();
    }
    if (a[6] != Py_None) {
        total = sized("affinities", a[6], 2).size(1);
        aff = address("affinities", a[6], ScalarType::BFloat16, {T, total}, dev);
        w = address<float>("weights", a[7], ScalarType::Float, {T, K}, dev);
    }
    if (a[4] != Py_None) {
        const at::Tensor& t = tensor("workspace", a[4]);
        ws_bytes = t.numel();
        ws = address("workspace", a[4], ScalarType::Byte, {ws_bytes}, dev);
    }
    const int32_t* ip = address<int32_t>("topk_idx", a[0], ScalarType::Int, {T, K}, dev);
    int32_t* off = address<int32_t>("expert_offsets", a[1], ScalarType::Int, {E + 1}, dev);
    int32_t* row = address<int32_t>("row_of", a[2], ScalarType::Int, {T, K}, dev);
    int32_t* src = address<int32_t>("source_of", a[3], ScalarType::Int, {T * K}, dev);
    const int first = int_of(a[5]), normalize = truth_of(a[8]);
    const float scale = float_of(a[9]);
    void* s = stream_of(a[10], dev);
    return run(dev, [&] {
        return g_entry.sort(ip, aff, (int)T, (int)K, (int)total, first, (int)E, normalize, scale, off, row, src, w, ws,
                            (size_t)ws_bytes, s);
    });
}

PyObject* do_gather(PyObject* const* a) {
    const at::Tensor& x = sized("x", a[0], 2);
    const int dev = device_of("x", x), code = dtype_code("x", x);
    const int64_t T = x.size(0), H = x.size(1), K = sized("row_of", a[1], 2).size(1), R = sized("rows", a[2], 2).size(0);
    const void* xp = address("x", a[0], x.scalar_type(), {T, H}, dev);
    const int32_t* row = address<int32_t>("row_of", a[1], ScalarType::Int, {T, K}, dev);
    float* sc = optional<float>("scales", a[3], ScalarType::Float, {blocks_of(H), R}, dev);
    void* rows = address("rows", a[2], a[3] == Py_None ? x.scalar_type() : ScalarType::Float8_e4m3fn, {R, H}, dev);
    void* s = stream_of(a[4], dev);
    return run(dev, [&] { return g_entry.gather(xp, code, row, (int)T, (int)K, (int)H, (int)R, rows, sc, s); });
}

PyObject* do_combine(PyObject* const* a) {
    const at::Tensor& rows = sized("rows", a[0], 2);
    const int dev = device_of("rows", rows), code = dtype_code("rows", rows);
    const int64_t R = rows.size(0), H = rows.size(1);
    const at::Tensor& ro = sized("row_of", a[1], 2);
    const int64_t T = ro.size(0), K = ro.size(1);
    const void* rp = address("rows", a[0], rows.scalar_type(), {R, H}, dev);
    const int32_t* row = address<int32_t>("row_of", a[1], ScalarType::Int, {T, K}, dev);
    const float* w = optional<float>("weights", a[2], ScalarType::Float, {T, K}, dev);
    void* out = address("out", a[3], rows.scalar_type(), {T, H}, dev);
    void* s = stream_of(a[4], dev);
    return run(dev, [&] { return g_entry.combine(rp, code, row, w, (int)T, (int)K, (int)H, (int)R, out, s); });
}

PyObject* do_combine_backward(PyObject* const* a) {
    const at::Tensor& g = sized("grad_out", a[0], 2);
    const int dev = device_of("grad_out", g), code = dtype_code("grad_out", g);
    const int64_t T = g.size(0), H = g.size(1), K = sized("row_of", a[2], 2).size(1);
    if (a[4] == Py_None && a[5] == Py_None) {
        PyErr_SetString(PyExc_ValueError, "grad_rows and grad_weights are both None");
        throw Refused();
    }
    if (a[1] == Py_None && a[5] != Py_None) {
        PyErr_SetString(PyExc_ValueError, "grad_weights needs rows");
        throw Refused();
    }
    const bool has_rows = a[1] != Py_None;
    const int64_t R = sized(has_rows ? "rows" : "grad_rows", a[has_rows ? 1 : 4], 2).size(0);
    const void* gp = address("grad_out", a[0], g.scalar_type(), {T, H}, dev);
    const void* rows = optional("rows", a[1], g.scalar_type(), {R, H}, dev);
    const int32_t* row = address<int32_t>("row_of", a[2], ScalarType::Int, {T, K}, dev);
    const float* w = optional<float>("weights", a[3], ScalarType::Float, {T, K}, dev);
    void* gr = optional("grad_rows", a[4], g.scalar_type(), {R, H}, dev);
    float* gw = optional<float>("grad_weights", a[5], ScalarType::Float, {T, K}, dev);
    void* s = stream_of(a[6], dev);
    return run(dev, [&] {
        return g_entry.combine_backward(gp, rows, code, row, w, (int)T, (int)K, (int)H, (int)R, gr, gw, s);
    });
}

PyObject* do_quantize(PyObject* const* a) {
    const at::Tensor& x = sized("x", a[0], 2);
    const int dev = device_of("x", x), code = dtype_code("x", x);
    const at::Tensor& qt = sized("q", a[1], 2);
    const int64_t R = qt.size(0), C = qt.size(1);
    const int gated = truth_of(a[3]);
    const void* xp = address("x", a[0], x.scalar_type(), {R, gated ? 2 * C : C}, dev);
    void* q = address("q", a[1], ScalarType::Float8_e4m3fn, {R, C}, dev);
    float* sc = address<float>("scales", a[2], ScalarType::Float, {blocks_of(C), R}, dev);
    const int32_t* valid = optional<int32_t>("valid_rows", a[4], ScalarType::Int, {1}, dev);
    void* s = stream_of(a[5], dev);
    return run(dev, [&] { return g_entry.quantize(xp, code, (int)R, (int)C, gated, valid, q, sc, s); });
}

PyObject* do_matmul(PyObject* const* a) {
    const at::Tensor& x = sized("x", a[0], 2);
    const int dev = device_of("x", x);
    const int64_t M = x.size(0), K = x.size(1), N = sized("w", a[2], 2).size(0);
    const at::Tensor& ot = tensor("out", a[4]);
    const int code = dtype_code("out", ot);
    const void* xp = address("x", a[0], ScalarType::Float8_e4m3fn, {M, K}, dev);
    const float* xs = address<float>("x_scales", a[1], ScalarType::Float, {blocks_of(K), M}, dev);
    const void* w = address("w", a[2], ScalarType::Float8_e4m3fn, {N, K}, dev);
    const float* ws = address<float>("w_scales", a[3], ScalarType::Float, {blocks_of(N), blocks_of(K)}, dev);
    void* out = address("out", a[4], ot.scalar_type(), {M, N}, dev);
    int32_t* status = optional<int32_t>("status", a[5], ScalarType::Int, {1}, dev);
    void* s = stream_of(a[6], dev);
    return run(dev, [&] { return g_entry.matmul(xp, xs, w, ws, (int)M, (int)N, (int)K, out, code, status, s); });
}

PyObject* do_grouped_matmul(PyObject* const* a) {
    const at::Tensor& x = sized("x", a[0], 2);
    const int dev = device_of("x", x);
    const at::Tensor& wt = sized("w", a[2], 3);
    const int64_t M = x.size(0), K = x.size(1), E = wt.size(0), N = wt.size(1);
    const at::Tensor& ot = tensor("out", a[5]);
    const int code = dtype_code("out", ot);
    const void* xp = address("x", a[0], ScalarType::Float8_e4m3fn, {M, K}, dev);
    const float* xs = address<float>("x_scales", a[1], ScalarType::Float, {blocks_of(K), M}, dev);
    const void* w = address("w", a[2], ScalarType::Float8_e4m3fn, {E, N, K}, dev);
    const float* ws = address<float>("w_scales", a[3], ScalarType::Float, {E, blocks_of(N), blocks_of(K)}, dev);
    const int32_t* off = address<int32_t>("expert_offsets", a[4], ScalarType::Int, {E + 1}, dev);
    void* out = address("out", a[5], ot.scalar_type(), {M, N}, dev);
    int32_t* status = optional<int32_t>("status", a[6], ScalarType::Int, {1}, dev);
    void* s = stream_of(a[7], dev);
    return run(dev, [&] {
        return g_entry.grouped_matmul(xp, xs, w, ws, off, (int)M, (int)E, (int)N, (int)K, out, code, status, s);
    });
}

// No C++ exception leaves this module.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* set_entries(PyObject*, PyObject* const* args, Py_ssize_t n) {
    void* p[7];
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "set_entries takes 7 addresses");
        return nullptr;
    }
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point's address is 0");
            return nullptr;
        }
    }
    g_entry = {reinterpret_cast<decltype(g_entry.sort)>(p[0]),
               reinterpret_cast<decltype(g_entry.gather)>(p[1]),
               reinterpret_cast<decltype(g_entry.combine)>(p[2]),
               reinterpret_cast<decltype(g_entry.combine_backward)>(p[3]),
               reinterpret_cast<decltype(g_entry.quantize)>(p[4]),
               reinterpret_cast<decltype(g_entry.matmul)>(p[5]),
               reinterpret_cast<decltype(g_entry.grouped_matmul)>(p[6])};
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef g_methods[] = {
    {"set_entries", FAST(set_entries), METH_FASTCALL, "addresses of the C ABI's entry points, in this module's order"},
    {"moe_sort", FAST((guarded<do_sort, 11>)), METH_FASTCALL, nullptr},
    {"moe_gather", FAST((guarded<do_gather, 5>)), METH_FASTCALL, nullptr},
    {"moe_combine", FAST((guarded<do_combine, 5>)), METH_FASTCALL, nullptr},
    {"moe_combine_backward", FAST((guarded<do_combine_backward, 7>)), METH_FASTCALL, nullptr},
    {"fp8_quantize", FAST((guarded<do_quantize, 6>)), METH_FASTCALL, nullptr},
    {"fp8_matmul", FAST((guarded<do_matmul, 7>)), METH_FASTCALL, nullptr},
    {"fp8_grouped_matmul", FAST((guarded<do_grouped_matmul, 8>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_bind", "native argument marshalling of experts.py", -1, g_methods};

}  // namespace

// The module says which torch and Python its inline layouts are from (BIND_TAG, given by the build);
// experts.py compares that with the ones that load it.
PyMODINIT_FUNC PyInit__bind(void) {
    PyObject* m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "built_for", BIND_TAG) < 0) Py_CLEAR(m);
    return m;
}
