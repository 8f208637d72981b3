// ssd_meta.cpp -- Python module mamba_ssd_prefill_amd._meta: what a call of the selective binding depends on of its
// tensors, read in one call.
//
// meta(*tensors) -> (key, pointers): `key` holds every tensor's type, device, sizes and strides as bytes (None has an
// entry of its own), so that two calls with equal keys pass the same checks; `pointers` their addresses (None
// for None).  Reading these through the tensors' Python attributes took 0.5 us a tensor, longer than the
// launch itself for the eleven of a scan step.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

static PyObject* meta(PyObject*, PyObject* const* args, Py_ssize_t n) {
    PyObject* ptrs = PyTuple_New(n);
    if (!ptrs) return nullptr;
    try {
        c10::SmallVector<int64_t, 160> key;
        for (Py_ssize_t i = 0; i < n; ++i) {
            if (args[i] == Py_None) {
                key.push_back(-1);
                Py_INCREF(Py_None);
                PyTuple_SET_ITEM(ptrs, i, Py_None);
                continue;
            }
            if (!THPVariable_Check(args[i])) {
                PyErr_Format(PyExc_TypeError, "expected a tensor or None, got %s", Py_TYPE(args[i])->tp_name);
                Py_DECREF(ptrs);
                return nullptr;
            }
            const at::Tensor& t = THPVariable_Unpack(args[i]);
            if (t.layout() != at::kStrided) {
                PyErr_SetString(PyExc_ValueError, "expected a strided tensor");
                Py_DECREF(ptrs);
                return nullptr;
            }
            const c10::Device d = t.device();
            key.push_back((int64_t)t.dim() << 32 | (int64_t)(uint8_t)t.scalar_type() << 16 |
                          (int64_t)(uint8_t)d.type() << 8 | (uint8_t)d.index());
            for (int64_t s : t.sizes()) key.push_back(s);
            for (int64_t s : t.strides()) key.push_back(s);
            PyObject* p = PyLong_FromUnsignedLongLong((unsigned long long)(uintptr_t)t.data_ptr());
            if (!p) {
                Py_DECREF(ptrs);
                return nullptr;
            }
            PyTuple_SET_ITEM(ptrs, i, p);
        }
        PyObject* bytes = PyBytes_FromStringAndSize((const char*)key.data(), (Py_ssize_t)(key.size() * sizeof(int64_t)));
        PyObject* out = bytes ? PyTuple_Pack(2, bytes, ptrs) : nullptr;
        Py_XDECREF(bytes);
        Py_DECREF(ptrs);
        return out;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "a tensor could not be read");
    }
    Py_DECREF(ptrs);
    return nullptr;
}

static PyMethodDef methods[] = {
    {"meta", (PyCFunction)(void (*)(void))meta, METH_FASTCALL, "meta(*tensors) -> (key, pointers)"},
    {nullptr, nullptr, 0, nullptr},
};
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_meta", "Tensors' metadata in one call.", -1, methods,
                             nullptr, nullptr, nullptr, nullptr};
PyMODINIT_FUNC PyInit__meta(void) { return PyModule_Create(&module); }
