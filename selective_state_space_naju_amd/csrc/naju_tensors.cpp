// naju_tensors.cpp -- lists of torch tensors as a table of addresses, for the calls of the
// binding that take many tensors.
//
// In Python a property of a tensor takes 40 ns: the update of 27 tensors took 58 us a call with
// the checks there and takes 11 with them here (its kernel 6), that of 157 tensors with 8-bit
// states 425 and 35.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstring>

#include <ATen/core/Tensor.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

enum Kind { kSameCount = 0, kSameShape = 1, kBlocks = 2 };

// table(width, device, block, lists): lists is a tuple of (column, list, dtype, kind), the first
// one the tensors that the others go with.  Returns bytes: for each tensor of the first list
// `width` words of 8 bytes, its number of elements and in each list's column the address of that
// list's tensor; or None if a tensor is missing, or not contiguous, of the dtype and on the GPU
// `device`, with as many elements (kind 0), the same shape (1), or one element for each `block`
// elements (2) of the first list's.
PyObject *table(PyObject *, PyObject *args)
{
    Py_ssize_t width, device, block;
    PyObject *lists;
    if (!PyArg_ParseTuple(args, "nnnO!", &width, &device, &block, &PyTuple_Type, &lists))
        return nullptr;
    const Py_ssize_t fields = PyTuple_GET_SIZE(lists);
    if (fields < 1 || width < 1 || block < 1) {
        PyErr_SetString(PyExc_ValueError, "table: no lists, or no width");
        return nullptr;
    }
    PyObject *out = nullptr, *first = nullptr;
    Py_ssize_t n = 0;
    for (Py_ssize_t j = 0; j < fields; ++j) {
        Py_ssize_t column, kind;
        PyObject *list, *dtype;
        if (!PyArg_ParseTuple(PyTuple_GET_ITEM(lists, j), "nOOn", &column, &list, &dtype, &kind) ||
            !(PyList_Check(list) || PyTuple_Check(list)) || !THPDtype_Check(dtype) || column < 1 ||
            column >= width) {
            Py_XDECREF(out);
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "table: lists of tensors");
            return nullptr;
        }
        const at::ScalarType type = reinterpret_cast<THPDtype *>(dtype)->scalar_type;
        if (j == 0) {
            first = list;
            n = PySequence_Fast_GET_SIZE(list);
            out = PyBytes_FromStringAndSize(nullptr, n * width * 8);
            if (out == nullptr) return nullptr;
            std::memset(PyBytes_AS_STRING(out), 0, (size_t)(n * width * 8));
        }
        bool fits = PySequence_Fast_GET_SIZE(list) == n;
        uint64_t *words = reinterpret_cast<uint64_t *>(PyBytes_AS_STRING(out));
        try {
            for (Py_ssize_t i = 0; fits && i < n; ++i) {
                PyObject *obj = PySequence_Fast_GET_ITEM(list, i);
                if (!(fits = THPVariable_Check(obj))) break;
                const at::Tensor &t = THPVariable_Unpack(obj);
                const at::Tensor &f = THPVariable_Unpack(PySequence_Fast_GET_ITEM(first, i));
                const int64_t count = f.numel();
                fits = t.is_cuda() && t.device().index() == device && t.scalar_type() == type &&
                       t.layout() == at::kStrided && t.is_contiguous() &&
                       t.numel() == (kind == kBlocks ? (count + block - 1) / block : count) &&
                       (kind != kSameShape || t.sizes() == f.sizes());
                if (!fits) break;
                words[i * width] = (uint64_t)count;
                words[i * width + column] = (uint64_t)(uintptr_t)t.data_ptr();
            }
        } catch (const std::exception &e) {  // (a tensor without memory of its own)
            Py_DECREF(out);
            PyErr_SetString(PyExc_ValueError, e.what());
            return nullptr;
        }
        if (!fits) {
            Py_DECREF(out);
            Py_RETURN_NONE;
        }
    }
    return out;
}

PyMethodDef methods[] = {{"table", table, METH_VARARGS, "Addresses of lists of tensors."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
