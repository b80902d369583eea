// w4a16_call.cpp -- the decode-step operators as CPython functions: the C entries of the same names with
// their arguments in order, and the status as the result.
//
// A decode step is a chain of calls of a few microseconds each, and converting 31 arguments through
// ctypes took longer than the launch.  A pointer argument is None, an address, or an object with
// data_ptr() (a torch tensor) or .ctypes.data (a numpy array).  Integers outside the parameter's range raise
// OverflowError.  The lock is released during the call, as a launch may wait for room in its queue.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "w4a16.h"

namespace {

PyObject *name_data_ptr, *name_ctypes, *name_data;

bool as_address(PyObject *o, void *&out)
{
    if (o == Py_None) {
        out = nullptr;
        return true;
    }
    if (PyLong_Check(o)) {
        out = PyLong_AsVoidPtr(o);
        return !PyErr_Occurred();
    }
    PyObject *r = PyObject_CallMethodNoArgs(o, name_data_ptr);
    if (!r && PyErr_ExceptionMatches(PyExc_AttributeError)) {
        PyErr_Clear();
        PyObject *c = PyObject_GetAttr(o, name_ctypes);
        if (c) {
            r = PyObject_GetAttr(c, name_data);
            Py_DECREF(c);
        }
    }
    if (!r)
        return false;
    out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

template <class T>
bool convert(PyObject *o, T &out)
{
    if constexpr (std::is_pointer_v<T>) {
        void *p = nullptr;
        const bool ok = as_address(o, p);
        out = static_cast<T>(p);
        return ok;
    } else if constexpr (std::is_floating_point_v<T>) {
        const double d = PyFloat_AsDouble(o);
        out = static_cast<T>(d);
        return d != -1.0 || !PyErr_Occurred();
    } else if constexpr (std::is_same_v<T, size_t>) {
        PyObject *i = PyNumber_Index(o); // PyLong_AsSize_t takes ints alone, PyLong_AsLongLong what counts as one
        if (!i)
            return false;
        out = PyLong_AsSize_t(i);
        Py_DECREF(i);
        return out != static_cast<size_t>(-1) || !PyErr_Occurred();
    } else {
        static_assert(std::is_integral_v<T>);
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred())
            return false;
        out = static_cast<T>(v);
        if (static_cast<long long>(out) != v) {
            PyErr_SetString(PyExc_OverflowError, "an argument does not fit its parameter");
            return false;
        }
        return true;
    }
}

template <class... A, size_t... I>
PyObject *forward(int (*entry)(A...), PyObject *const *args, std::index_sequence<I...>)
{
    std::tuple<A...> values;
    if (!(convert(args[I], std::get<I>(values)) && ...))
        return nullptr;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = entry(std::get<I>(values)...);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

template <class... A>
PyObject *checked(int (*entry)(A...), PyObject *const *args, Py_ssize_t n)
{
    if (n != static_cast<Py_ssize_t>(sizeof...(A))) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", static_cast<int>(sizeof...(A)), n);
        return nullptr;
    }
    return forward(entry, args, std::index_sequence_for<A...>());
}

template <auto entry>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return checked(entry, args, n);
}

template <auto entry>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<entry>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<&w4a16_rope_append>("w4a16_rope_append"),
    method<&w4a16_paged_attention>("w4a16_paged_attention"),
    method<&w4a16_moe_layer>("w4a16_moe_layer"),
    method<&w4a16_norm_rope_append>("w4a16_norm_rope_append"),
    method<&w4a16_kv4_append>("w4a16_kv4_append"),
    method<&w4a16_kv4_attention>("w4a16_kv4_attention"),
    method<&w4a16_sample>("w4a16_sample"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w4a16_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__w4a16_call(void)
{
    name_data_ptr = PyUnicode_InternFromString("data_ptr");
    name_ctypes = PyUnicode_InternFromString("ctypes");
    name_data = PyUnicode_InternFromString("data");
    if (!name_data_ptr || !name_ctypes || !name_data)
        return nullptr;
    return PyModule_Create(&module);
}
