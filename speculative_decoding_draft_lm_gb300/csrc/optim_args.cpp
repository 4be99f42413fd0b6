// The checks of the update's gradients, for Python: a step takes hundreds of tensors,
// and four attributes of each read in Python cost 0.4 us a tensor (96 tensors: 43 us
// a step, of which the GPU needs 7), here 19 ns.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "domino_rollout.h"

namespace {

// the tensor of a list's entry; nullptr: none
const at::Tensor* tensor_at(PyObject* fast, Py_ssize_t i) {
    PyObject* o = PySequence_Fast_GET_ITEM(fast, i);
    return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// the library's name of a tensor's type; false: it has none
bool type_code(const at::Tensor& t, int* code) {
    if (t.scalar_type() == at::kBFloat16) *code = DOMINO_DTYPE_BF16;
    else if (t.scalar_type() == at::kFloat) *code = DOMINO_DTYPE_FP32;
    else return false;
    return true;
}

// whether g is what the gradient of p has to be; *code: its type
bool good(const at::Tensor& g, const at::Tensor& p, long device, int* code) {
    return g.layout() == c10::kStrided && g.get_device() == device && type_code(g, code) && g.sizes() == p.sizes() &&
           g.is_contiguous();
}

// whether p still is `n` elements in a row, of type `code`
bool same(const at::Tensor& p, int64_t n, int code) {
    int its;
    return p.numel() == n && type_code(p, &its) && its == code && p.is_contiguous();
}

// the array at the address that is an argument; sets Python's error if it is no integer
template <typename T>
T* array(PyObject* address) {
    return reinterpret_cast<T*>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLongMask(address)));
}

// gradients(params, grads, device, held, addresses, dtypes[, sizes, types, buffers, buffers_held]) -> int
//
// (Arguments are taken one by one: a format string takes 0.1 us a call.)
//
// params: list of tensors; grads: list of a tensor or None for each, or None for their .grad.  The gradients'
// addresses (0: none) go to the uint64 array at `addresses`, their types to the int array at `dtypes`.  Returns -1,
// or the place of the first gradient that is not contiguous, bf16 or fp32, of its parameter's shape and on `device`,
// or -2 - the place of the first parameter whose elements are not at its address in the uint64 array at `held`, or
// not as many as the int64 array at `sizes` has it, of the type in the int array at `types` and contiguous.  After the
// parameters come the tensors of the list `buffers`: address and bytes of each in the uint64 array at `buffers_held`.
PyObject* gradients(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if ((nargs != 6 && nargs != 10) || !PyList_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "gradients: want a list and 5 or 9 more arguments");
        return nullptr;
    }
    PyObject *params = args[0], *grads = args[1], *buffers = nargs == 10 ? args[8] : Py_None;
    const long device = PyLong_AsLong(args[2]);
    const uint64_t* at = array<const uint64_t>(args[3]);
    uint64_t* to = array<uint64_t>(args[4]);
    int* codes = array<int>(args[5]);
    const int64_t* n_of = nargs == 10 ? array<const int64_t>(args[6]) : nullptr;
    const int* type_of = nargs == 10 ? array<const int>(args[7]) : nullptr;
    const uint64_t* buffer_at = nargs == 10 ? array<const uint64_t>(args[9]) : nullptr;
    if (PyErr_Occurred()) return nullptr;
    const Py_ssize_t n = PyList_GET_SIZE(params);
    PyObject* fast = nullptr;
    if (grads != Py_None) {
        fast = PySequence_Fast(grads, "grads: want a list of tensors");
        if (!fast) return nullptr;
        if (PySequence_Fast_GET_SIZE(fast) != n) {
            Py_DECREF(fast);
            PyErr_Format(PyExc_ValueError, "grads: want %zd tensors (or None)", n);
            return nullptr;
        }
    }
    Py_ssize_t bad = -1, moved = -1;
    try {
        for (Py_ssize_t i = 0; bad < 0 && i < n; ++i) {
            const at::Tensor* p = tensor_at(params, i);
            at::Tensor own;
            const at::Tensor* g = nullptr;
            bool none = false;
            if (!p || reinterpret_cast<uintptr_t>(p->data_ptr()) != at[i] ||
                (n_of && type_of && !same(*p, n_of[i], type_of[i]))) {
                moved = i;
                break;
            }
            if (!fast) {
                own = p->grad();
                none = !own.defined();
                g = &own;
            } else {
                none = PySequence_Fast_GET_ITEM(fast, i) == Py_None;
                g = tensor_at(fast, i);
            }
            to[i] = 0;
            codes[i] = DOMINO_DTYPE_FP32;
            if (none) continue;
            if (!g || !good(*g, *p, device, &codes[i])) bad = i;
            else to[i] = static_cast<uint64_t>(reinterpret_cast<uintptr_t>(g->data_ptr()));
        }
        for (Py_ssize_t i = 0; bad < 0 && moved < 0 && PyList_Check(buffers) && i < PyList_GET_SIZE(buffers); ++i) {
            const at::Tensor* b = tensor_at(buffers, i);
            if (!b || reinterpret_cast<uintptr_t>(b->data_ptr()) != buffer_at[2 * i] || b->nbytes() != buffer_at[2 * i + 1] ||
                !b->is_contiguous())
                moved = n + i;
        }
    } catch (const std::exception& e) {
        Py_XDECREF(fast);
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    Py_XDECREF(fast);
    return PyLong_FromSsize_t(moved >= 0 ? -2 - moved : bad);
}

// written(params, addresses): the parameters whose address is not 0 were changed in place
PyObject* written(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 2 || !PyList_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "written: want a list and an address");
        return nullptr;
    }
    PyObject* params = args[0];
    const uint64_t* at = array<const uint64_t>(args[1]);
    if (PyErr_Occurred()) return nullptr;
    try {
        for (Py_ssize_t i = 0; i < PyList_GET_SIZE(params); ++i) {
            const at::Tensor* p = tensor_at(params, i);
            if (p && at[i] && !p->is_inference()) p->unsafeGetTensorImpl()->bump_version();
        }
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"gradients", fast(gradients), METH_FASTCALL, "addresses and types of a step's gradients"},
                         {"written", fast(written), METH_FASTCALL, "counts the change of the parameters"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_optim_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__optim_args() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", DOMINO_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
