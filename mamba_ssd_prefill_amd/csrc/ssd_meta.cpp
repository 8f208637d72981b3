// ssd_meta.cpp -- Python module mamba_ssd_prefill_amd._meta: the selective binding's dealings with torch's tensors and
// with the library, each in one call.
//
// meta(*tensors) -> (key, pointers): `key` holds every tensor's type, device, sizes and strides as bytes (None has an
// entry of its own), so that two calls with equal keys pass the same checks; `pointers` their addresses (None for
// None).  Reading these through the tensors' Python attributes took 0.5 us a tensor, longer than the launch
// itself for the eleven of a scan step.
// new(*layouts) -> tensors: uninitialised tensors, each of a layout that `meta` gives as the key of one tensor.
// call(function, *arguments) -> status: a function of the library by its address, with pointers and sizes as integers
// (None: a null pointer), without the interpreter's lock.  A tensor stands for its address and is taken to be written by the
// call: its version goes up, so that autograd refuses a backward pass that needs what it held before.  ctypes took 0.6 us
// more for the twelve of a scan step.
#include <Python.h>
#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <array>
#include <utility>

static PyObject* meta(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    THPObjectPtr ptrs(PyTuple_New(n));
    if (!ptrs) return nullptr;
    c10::SmallVector<int64_t, 160> key;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (args[i] == Py_None) {
            key.push_back(-1);
            Py_INCREF(Py_None);
            PyTuple_SET_ITEM(ptrs.get(), i, Py_None);
            continue;
        }
        if (!THPVariable_Check(args[i])) {
            PyErr_Format(PyExc_TypeError, "expected a tensor or None, got %s", Py_TYPE(args[i])->tp_name);
            return nullptr;
        }
        const at::Tensor& t = THPVariable_Unpack(args[i]);
        if (t.layout() != at::kStrided) {
            PyErr_SetString(PyExc_ValueError, "expected a strided tensor");
            return nullptr;
        }
        const c10::Device d = t.device();
        key.push_back((int64_t)t.dim() << 32 | (int64_t)(uint8_t)t.scalar_type() << 16 | (int64_t)(uint8_t)d.type() << 8 |
                      (uint8_t)d.index());
        for (int64_t s : t.sizes()) key.push_back(s);
        for (int64_t s : t.strides()) key.push_back(s);
        PyObject* p = PyLong_FromUnsignedLongLong((unsigned long long)(uintptr_t)t.data_ptr());
        if (!p) return nullptr;
        PyTuple_SET_ITEM(ptrs.get(), i, p);
    }
    THPObjectPtr bytes(PyBytes_FromStringAndSize((const char*)key.data(), (Py_ssize_t)(key.size() * sizeof(int64_t))));
    return bytes ? PyTuple_Pack(2, bytes.get(), ptrs.get()) : nullptr;
    END_HANDLE_TH_ERRORS
}

static PyObject* new_tensors(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    THPObjectPtr out(PyTuple_New(n));
    if (!out) return nullptr;
    for (Py_ssize_t i = 0; i < n; ++i) {
        const int64_t* v = PyBytes_Check(args[i]) ? (const int64_t*)PyBytes_AS_STRING(args[i]) : nullptr;
        const Py_ssize_t words = v ? PyBytes_GET_SIZE(args[i]) / (Py_ssize_t)sizeof(int64_t) : 0;
        const int64_t dim = words ? v[0] >> 32 : -1;
        if (dim < 0 || words != 1 + 2 * dim) {
            PyErr_SetString(PyExc_ValueError, "expected the layout of one tensor");
            return nullptr;
        }
        const c10::Device device((c10::DeviceType)(uint8_t)(v[0] >> 8), (c10::DeviceIndex)(int8_t)v[0]);
        const auto options = at::TensorOptions().dtype((at::ScalarType)(uint8_t)(v[0] >> 16)).device(device);
        PyObject* t = THPVariable_Wrap(
            at::empty_strided(at::IntArrayRef(v + 1, (size_t)dim), at::IntArrayRef(v + 1 + dim, (size_t)dim), options));
        if (!t) return nullptr;
        PyTuple_SET_ITEM(out.get(), i, t);
    }
    return out.release();
    END_HANDLE_TH_ERRORS
}

// Every argument of the library's functions is a pointer or a size_t, one integer register or stack slot each, so a
// function of n arguments is called through a type with n integers.
constexpr size_t kMaxArgs = 32;
typedef int (*Call)(void*, const uintptr_t*);
template <size_t... I> static int call_n(void* f, const uintptr_t* a, std::index_sequence<I...>) {
    return ((int (*)(decltype((void)I, uintptr_t())...))f)(a[I]...);
}
template <size_t N> static int call_with(void* f, const uintptr_t* a) { return call_n(f, a, std::make_index_sequence<N>()); }
template <size_t... N> static constexpr std::array<Call, sizeof...(N)> call_table(std::index_sequence<N...>) {
    return {&call_with<N>...};
}
constexpr auto kCalls = call_table(std::make_index_sequence<kMaxArgs + 1>());

static PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    uintptr_t v[kMaxArgs + 1];
    if (n < 1 || n > (Py_ssize_t)kMaxArgs + 1) {
        PyErr_SetString(PyExc_TypeError, "expected a function and up to 32 arguments");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        v[i] = 0;
        if (i && args[i] == Py_None) continue;
        if (i && !PyLong_CheckExact(args[i]) && THPVariable_Check(args[i])) {
            const at::Tensor& t = THPVariable_Unpack(args[i]);
            v[i] = (uintptr_t)t.data_ptr();
            if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
            continue;
        }
        const unsigned long long u = PyLong_AsUnsignedLongLong(args[i]);
        if (u == (unsigned long long)-1 && PyErr_Occurred()) return nullptr;
        v[i] = (uintptr_t)u;
    }
    if (!v[0]) {
        PyErr_SetString(PyExc_ValueError, "expected the address of a function");
        return nullptr;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = kCalls[(size_t)n - 1]((void*)v[0], v + 1);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

static PyMethodDef methods[] = {
    {"meta", (PyCFunction)(void (*)(void))meta, METH_FASTCALL, "meta(*tensors) -> (key, pointers)"},
    {"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, "call(function, *arguments) -> status"},
    {"new", (PyCFunction)(void (*)(void))new_tensors, METH_FASTCALL, "new(*layouts) -> uninitialised tensors"},
    {nullptr, nullptr, 0, nullptr},
};
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_meta", "Tensors' metadata, new tensors and library calls.", -1, methods,
                             nullptr, nullptr, nullptr, nullptr};
PyMODINIT_FUNC PyInit__meta(void) { return PyModule_Create(&module); }
