// Python calls of libdsa.so's entry points (include/dsa.h) without ctypes.
//
// A launch takes about 3 us on the host; marshalling 24 arguments through ctypes and
// reading ten tensors' addresses in Python took 5 more, which is what a decode step
// of small kernels then waits for. Here an argument costs some tens of nanoseconds:
// a pointer is None, an integer address or an object with data_ptr() (a tensor), the
// conversions follow from the C declarations, and the status is returned as it is.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "../../include/dsa.h"

namespace {

PyObject *g_data_ptr;                                 // "data_ptr"

template <typename T>
bool get(PyObject *o, T *&out) {
    if (o == Py_None) {
        out = nullptr;
        return true;
    }
    PyObject *address = PyLong_Check(o) ? Py_NewRef(o) : PyObject_CallMethodNoArgs(o, g_data_ptr);
    if (!address) return false;
    out = static_cast<T *>(PyLong_AsVoidPtr(address));
    Py_DECREF(address);
    return !PyErr_Occurred();
}

template <typename T>
std::enable_if_t<std::is_integral_v<T>, bool> get(PyObject *o, T &out) {
    PyObject *index = PyLong_Check(o) ? Py_NewRef(o) : PyNumber_Index(o);
    if (!index) return false;
    const long long v = PyLong_AsLongLong(index);
    Py_DECREF(index);
    if (v == -1 && PyErr_Occurred()) return false;
    out = static_cast<T>(v);
    if (static_cast<long long>(out) != v || (std::is_unsigned_v<T> && v < 0)) {
        PyErr_SetString(PyExc_OverflowError, "an integer argument does not fit its C type");
        return false;
    }
    return true;
}

bool get(PyObject *o, float &out) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return false;
    out = static_cast<float>(v);
    return true;
}

template <auto Fn>
struct Call;

template <typename... A, int (*Fn)(A...)>
struct Call<Fn> {
    template <size_t... I>
    static PyObject *go(PyObject *const *args, std::index_sequence<I...>) {
        std::tuple<A...> v;
        if (!(get(args[I], std::get<I>(v)) && ...)) return nullptr;
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = Fn(std::get<I>(v)...);
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(status);
    }
    static PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
        if (n != (Py_ssize_t)sizeof...(A)) {
            PyErr_Format(PyExc_TypeError, "%zd arguments, the entry point takes %zd", n, (Py_ssize_t)sizeof...(A));
            return nullptr;
        }
        return go(args, std::index_sequence_for<A...>{});
    }
};

#define ENTRY(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&Call<&name>::call)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    ENTRY(dsa_selftest_bounded_wait),
    ENTRY(dsa_head_gate),
    ENTRY(dsa_kpool_compress),
    ENTRY(dsa_indexer_store),
    ENTRY(dsa_kpool_compress_tokens),
    ENTRY(dsa_index_scores),
    ENTRY(dsa_topk_expand),
    ENTRY(dsa_topk_expand_tail),
    ENTRY(dsa_indexer_select),
    ENTRY(dsa_sparse_mla_decode),
    ENTRY(dsa_sparse_mla_decode_noalloc),
    ENTRY(dsa_sparse_mla_decode_paged),
    ENTRY(dsa_sparse_mla_decode_paged_fp8),
    ENTRY(dsa_latent_append_paged),
    ENTRY(dsa_latent_append_paged_fp8),
    ENTRY(dsa_prefix_mla_decode_paged),
    ENTRY(dsa_prefix_mla_decode_paged_fp8),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dsacall", "libdsa.so's entry points; each returns its status.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dsacall(void) {
    g_data_ptr = PyUnicode_InternFromString("data_ptr");
    return g_data_ptr ? PyModule_Create(&module) : nullptr;
}
