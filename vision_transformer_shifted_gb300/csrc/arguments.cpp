// The binding's checks of a tensor argument (type, shape, contiguous, on the call's
// device) and its address, from PyTorch's own tensor objects: 0.09 us a tensor and 0.39
// in Python, which on one row is the time of a call (layer norm 1 x 2048, six tensors:
// 5.6 us of host and 3.7; its kernel alone takes 1.4).  Whatever is not a plain tensor
// that passes goes to the Python functions of the same names and signatures, which say
// what is wrong with it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

namespace {

struct {
    PyObject *tensor, *parameter;   // the types a plain tensor has
    PyObject *dtypes[3];            // torch.bfloat16, .float32, .float8_e4m3fn
    PyObject *arg, *rows;           // the functions in Python
    PyObject *current_device;
    PyObject *C;                    // "C"
} py;
constexpr at::ScalarType TYPES[3] = {at::kBFloat16, at::kFloat, at::kFloat8_e4m3fn};

const at::Tensor *plain(PyObject *o)
{
    PyObject *type = reinterpret_cast<PyObject *>(Py_TYPE(o));
    return type == py.tensor || type == py.parameter ? &THPVariable_Unpack(o) : nullptr;
}
bool of_type(const at::Tensor &t, PyObject *dtype)
{
    for (int i = 0; i < 3; ++i)
        if (dtype == py.dtypes[i]) return t.scalar_type() == TYPES[i];
    return false;
}
bool of_shape(const at::Tensor &t, PyObject *shape)
{
    if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != t.dim()) return false;
    for (int64_t i = 0; i < t.dim(); ++i)
        if (PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)) != t.size(i)) return false;
    return true;
}

// arg(name, t, dtype, shape, dev): the address
PyObject *arg(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n == 5) {
        try {
            const at::Tensor *t = plain(a[1]);
            if (t && of_type(*t, a[2]) && of_shape(*t, a[3]) && t->is_contiguous() && t->is_cuda() &&
                t->get_device() == PyLong_AsLong(a[4]))
                return PyLong_FromVoidPtr(t->data_ptr());
        } catch (...) {
        }
        PyErr_Clear();
    }
    return PyObject_Vectorcall(py.arg, a, n, nullptr);
}

// rows(h, x, dtype, name): rows, shape, device and address of the tokens x [..., C]
PyObject *rows(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n == 4) {
        PyObject *C = PyObject_GetAttr(a[0], py.C), *now = nullptr, *shape = nullptr;
        try {
            const at::Tensor *t = plain(a[1]);
            const int64_t c = C ? PyLong_AsLongLong(C) : 0;
            if (t && c > 0 && t->dim() > 0 && t->size(-1) == c && of_type(*t, a[2]) && t->is_contiguous() && t->is_cuda() &&
                t->numel() / c <= 0x7fffffff && (now = PyObject_CallNoArgs(py.current_device)) &&
                PyLong_AsLong(now) == t->get_device() && (shape = PyObject_GetAttrString(a[1], "shape"))) {
                PyObject *r = Py_BuildValue("(LOOK)", (long long)(t->numel() / c), shape, now,
                                            (unsigned long long)(uintptr_t)t->data_ptr());
                Py_XDECREF(C);
                Py_XDECREF(now);
                Py_XDECREF(shape);
                return r;
            }
        } catch (...) {
        }
        Py_XDECREF(C);
        Py_XDECREF(now);
        Py_XDECREF(shape);
        PyErr_Clear();
    }
    return PyObject_Vectorcall(py.rows, a, n, nullptr);
}

// setup(tensor, parameter, bfloat16, float32, float8_e4m3fn, arg, rows, current_device)
PyObject *setup(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "setup takes eight arguments");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) Py_INCREF(a[i]);   // (for the process)
    py = {a[0], a[1], {a[2], a[3], a[4]}, a[5], a[6], a[7], PyUnicode_InternFromString("C")};
    if (!py.C) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"arg", (PyCFunction)(void (*)())arg, METH_FASTCALL, nullptr},
                         {"rows", (PyCFunction)(void (*)())rows, METH_FASTCALL, nullptr},
                         {"setup", (PyCFunction)(void (*)())setup, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_arguments", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

// (The binding uses it under the PyTorch that it was built against only: it reads the
// tensor objects' layout from that one's headers.)
PyMODINIT_FUNC PyInit__arguments()
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_BUILT) < 0) Py_CLEAR(m);
    return m;
}
