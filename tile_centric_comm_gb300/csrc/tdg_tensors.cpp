// tdg_tensors.cpp -- the tensor checks of the attention calls' binding, as a
// CPython module that reads torch's tensors directly.
//
// A call of one token takes the GPU 4 us, and checking its up to ten tensors
// took Python 6: a frame and five or six attribute calls for each.  Here a
// tensor that passes costs 0.1 us.  One that does not pass, or is not a plain
// torch.Tensor, goes to the Python function of the same checks, which accepts
// it or raises the error.
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject *tensor_type, *checked_rows, *checked_table, *checked_flat;

// the plain tensor behind `o`, of the type and on the device; NULL for any other
const at::Tensor *plain(PyObject *o, at::ScalarType type, PyObject *device)
{
    if (reinterpret_cast<PyObject *>(Py_TYPE(o)) != tensor_type || !THPDevice_Check(device))
        return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    const bool ok = t.defined() && t.layout() == at::kStrided && t.scalar_type() == type &&
                    t.device() == reinterpret_cast<THPDevice *>(device)->device;
    return ok ? &t : nullptr;
}

long long address(const at::Tensor &t) { return reinterpret_cast<long long>(t.data_ptr()); }

// No exception of torch's leaves a function below: what throws goes to Python.
template <class F> PyObject *run(F native, PyObject *checked, PyObject *const *args, Py_ssize_t n)
{
    PyObject *r = nullptr;
    try {
        r = native();
    } catch (...) {
        r = nullptr;
    }
    return r || PyErr_Occurred() ? r : PyObject_Vectorcall(checked, args, static_cast<size_t>(n), nullptr);
}

// rows(tensor, name, device) -> (address, row stride, rows, heads, D)
PyObject *rows(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return run(
        [&]() -> PyObject * {
            const at::Tensor *t = n == 3 ? plain(args[0], at::kBFloat16, args[2]) : nullptr;
            if (!t || t->dim() != 3)
                return nullptr;
            const long long rows = t->size(0), heads = t->size(1), D = t->size(2);
            long long stride = t->stride(0);
            if (rows <= 1 || !heads)
                stride = heads * D; // no second row, no stride
            if (rows && heads && ((t->stride(2) != 1 && D > 1) || (t->stride(1) != D && heads > 1)))
                return nullptr;
            return Py_BuildValue("(LLLLL)", address(*t), stride, rows, heads, D);
        },
        checked_rows, args, n);
}

// table(tensor, name, device) -> (address, entries, row stride, sequences)
PyObject *table(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return run(
        [&]() -> PyObject * {
            const at::Tensor *t = n == 3 ? plain(args[0], at::kInt, args[2]) : nullptr;
            if (!t || t->dim() != 2)
                return nullptr;
            const long long sequences = t->size(0), entries = t->size(1);
            if (entries > 1 && t->stride(1) != 1)
                return nullptr;
            return Py_BuildValue("(LLLL)", address(*t), entries, sequences <= 1 ? entries : static_cast<long long>(t->stride(0)),
                                 sequences);
        },
        checked_table, args, n);
}

// flat(tensor, name, dtype, elements, device) -> address
PyObject *flat(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return run(
        [&]() -> PyObject * {
            if (n != 5 || !THPDtype_Check(args[2]) || !PyLong_CheckExact(args[3]))
                return nullptr;
            const at::Tensor *t = plain(args[0], reinterpret_cast<THPDtype *>(args[2])->scalar_type, args[4]);
            int overflow = 0;
            const long long want = PyLong_AsLongLongAndOverflow(args[3], &overflow);
            if (!t || overflow || !t->is_contiguous() || t->numel() < want)
                return nullptr;
            return PyLong_FromLongLong(address(*t));
        },
        checked_flat, args, n);
}

// setup(Tensor, rows, table, flat): torch's class and the Python functions
PyObject *setup(PyObject *, PyObject *args)
{
    PyObject *o[4];
    if (!PyArg_ParseTuple(args, "OOOO", &o[0], &o[1], &o[2], &o[3]))
        return nullptr;
    PyObject **const to[4] = {&tensor_type, &checked_rows, &checked_table, &checked_flat};
    for (int i = 0; i < 4; ++i) {
        Py_INCREF(o[i]);
        Py_XDECREF(*to[i]);
        *to[i] = o[i];
    }
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)> PyMethodDef fast(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, nullptr}, fast<rows>("rows"), fast<table>("table"), fast<flat>("flat"), {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "tdg_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit_tdg_tensors() { return PyModule_Create(&module); }
