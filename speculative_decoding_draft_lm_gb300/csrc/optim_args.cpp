// The checks of the update's gradients, for Python: a step takes hundreds of tensors,
// and four attributes of each read in Python cost 0.4 us a tensor (96 tensors: 43 us
// a step, of which the GPU needs 7), here 19 ns.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <new>

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

template <typename T>
T* array(unsigned long long address) {
    return reinterpret_cast<T*>(static_cast<uintptr_t>(address));
}

// What a context's calls have in common.  The lists are borrowed: who has the plan keeps them (a reference here would
// be one that Python's collector of cycles does not see).
struct Plan {
    PyObject *params, *buffers;  // lists; buffers may be null
    long device;
    const uint64_t* held;
    uint64_t* addresses;
    int* dtypes;
    const int64_t* sizes;
    const int* types;
    const uint64_t* buffers_held;
};

// Puts the gradients' addresses (0: none) and types into the plan's arrays; grads: list of a tensor or None for each
// parameter, or None for their .grad.  Returns -1, or the place of the first gradient that is not contiguous, bf16 or
// fp32, of its parameter's shape and on `device`, or -2 - the place of the first parameter whose elements are not at
// its address in `held`, or not as many as `sizes` has it, of the type in `types` and contiguous.  After the parameters
// come the buffers: address and bytes of each in `buffers_held`.
PyObject* read(const Plan& plan, PyObject* grads) {
    PyObject* const params = plan.params;
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
            if (!p || reinterpret_cast<uintptr_t>(p->data_ptr()) != plan.held[i] ||
                (plan.sizes && !same(*p, plan.sizes[i], plan.types[i]))) {
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
            plan.addresses[i] = 0;
            plan.dtypes[i] = DOMINO_DTYPE_FP32;
            if (none) continue;
            if (!g || !good(*g, *p, plan.device, &plan.dtypes[i])) bad = i;
            else plan.addresses[i] = static_cast<uint64_t>(reinterpret_cast<uintptr_t>(g->data_ptr()));
        }
        const Py_ssize_t buffers = plan.buffers ? PyList_GET_SIZE(plan.buffers) : 0;
        for (Py_ssize_t i = 0; bad < 0 && moved < 0 && i < buffers; ++i) {
            const at::Tensor* b = tensor_at(plan.buffers, i);
            const uint64_t* was = plan.buffers_held + 2 * i;
            if (!b || reinterpret_cast<uintptr_t>(b->data_ptr()) != was[0] || b->nbytes() != was[1] || !b->is_contiguous())
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

// Counts the change of the parameters whose address is not 0.
PyObject* count_change(PyObject* params, const uint64_t* addresses) {
    try {
        for (Py_ssize_t i = 0; i < PyList_GET_SIZE(params); ++i) {
            const at::Tensor* p = tensor_at(params, i);
            if (p && addresses[i] && !p->is_inference()) p->unsafeGetTensorImpl()->bump_version();
        }
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    Py_RETURN_NONE;
}

// gradients(params, grads, device, held, addresses, dtypes) -> int: one call's, of params as they are
PyObject* gradients(PyObject*, PyObject* args) {
    Plan plan = {};
    PyObject* grads;
    unsigned long long held, addresses, dtypes;
    if (!PyArg_ParseTuple(args, "O!OlKKK", &PyList_Type, &plan.params, &grads, &plan.device, &held, &addresses, &dtypes))
        return nullptr;
    plan.held = array<const uint64_t>(held);
    plan.addresses = array<uint64_t>(addresses);
    plan.dtypes = array<int>(dtypes);
    return read(plan, grads);
}

// written(params, addresses)
PyObject* written(PyObject*, PyObject* args) {
    PyObject* params;
    unsigned long long addresses;
    if (!PyArg_ParseTuple(args, "O!K", &PyList_Type, &params, &addresses)) return nullptr;
    return count_change(params, array<const uint64_t>(addresses));
}

// plan(params, device, held, addresses, dtypes, sizes, types, buffers, buffers_held) -> (f(grads), g()): what a context
// calls in every step, with nothing to take apart (0.3 us less than `gradients` with all these).
const char kPlan[] = "_optim_args.plan";
const Plan* plan_of(PyObject* capsule) { return static_cast<const Plan*>(PyCapsule_GetPointer(capsule, kPlan)); }
PyObject* planned_read(PyObject* self, PyObject* grads) {
    const Plan* plan = plan_of(self);
    return plan ? read(*plan, grads) : nullptr;
}
PyObject* planned_written(PyObject* self, PyObject*) {
    const Plan* plan = plan_of(self);
    return plan ? count_change(plan->params, plan->addresses) : nullptr;
}
PyMethodDef read_method = {"read", planned_read, METH_O, "addresses and types of a step's gradients"};
PyMethodDef written_method = {"written", planned_written, METH_NOARGS, "counts the change of the parameters"};

PyObject* make_plan(PyObject*, PyObject* args) {
    Plan plan = {};
    unsigned long long held, addresses, dtypes, sizes, types, buffers_held;
    if (!PyArg_ParseTuple(args, "O!lKKKKKO!K", &PyList_Type, &plan.params, &plan.device, &held, &addresses, &dtypes, &sizes,
                          &types, &PyList_Type, &plan.buffers, &buffers_held))
        return nullptr;
    plan.held = array<const uint64_t>(held);
    plan.addresses = array<uint64_t>(addresses);
    plan.dtypes = array<int>(dtypes);
    plan.sizes = array<const int64_t>(sizes);
    plan.types = array<const int>(types);
    plan.buffers_held = array<const uint64_t>(buffers_held);
    Plan* kept = new (std::nothrow) Plan(plan);
    if (!kept) return PyErr_NoMemory();
    PyObject* capsule =
        PyCapsule_New(kept, kPlan, [](PyObject* c) { delete static_cast<Plan*>(PyCapsule_GetPointer(c, kPlan)); });
    if (!capsule) {
        delete kept;
        return nullptr;
    }
    PyObject* read_call = PyCFunction_New(&read_method, capsule);
    PyObject* written_call = PyCFunction_New(&written_method, capsule);
    Py_DECREF(capsule);
    PyObject* both = read_call && written_call ? PyTuple_Pack(2, read_call, written_call) : nullptr;
    Py_XDECREF(read_call);
    Py_XDECREF(written_call);
    return both;
}

PyMethodDef methods[] = {{"gradients", gradients, METH_VARARGS, "addresses and types of a step's gradients"},
                         {"written", written, METH_VARARGS, "counts the change of the parameters"},
                         {"plan", make_plan, METH_VARARGS, "both of these for the tensors of a context"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_optim_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__optim_args() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", DOMINO_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
