// Python extension of the bindings in aware_conv_amd/adamw.py and gscan.py:
// checks tensors and reads what the library takes of them, in one call for
// several tensors, and tells autograd of those that were written.  What is wrong is put into words by the caller.
//
// A step over a hundred small tensors has several hundred of them to check and
// look up; attribute by attribute from Python that takes longer than the step
// itself does on the GPU (96 us for 90 tensors of 4 lists; the GPU takes 13),
// and a single decoded token's call is mostly that, too.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/util/Exception.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

constexpr int kColumns = 8;  // of a row, 64 bits each: seven addresses, then the number of elements

// A method whose C++ exceptions become Python's.  Asking a tensor for its memory
// throws where it has none of its own, as inside torch's function transforms; past
// the interpreter's frames, which are C, an exception would end the process.
template <PyObject* (*body)(PyObject*)>
PyObject* guarded(PyObject*, PyObject* args) {
    try {
        return body(args);
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// What is wrong with a list, for the caller to put into words.
enum { OK, COUNT, NOT_TENSOR, DTYPE, DEVICE, LAYOUT, SIZE };

// column(tensors, table, rows, column, dtype, device, block) -> (code, index)
//
// tensors: a list or tuple, which the caller keeps as long as the table is
// used (nothing else is taken: an iterator's tensors would be gone with it).
// table: address of `rows` rows.  column: where the addresses go.  block: 0
// writes the numbers of elements to the last column; k > 0 expects
// ceil(n / k) elements for the n found there.
PyObject* column(PyObject* args) {
    PyObject *list, *dtype;
    unsigned long long table;
    Py_ssize_t rows;
    int col, device;
    long long block;
    if (!PyArg_ParseTuple(args, "OKniOiL", &list, &table, &rows, &col, &dtype, &device, &block))
        return nullptr;
    if (!THPDtype_Check(dtype) || col < 0 || col >= kColumns - 1 || block < 0) {
        PyErr_SetString(PyExc_ValueError, "column: bad arguments");
        return nullptr;
    }
    const at::ScalarType type = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    if (!PyList_Check(list) && !PyTuple_Check(list)) {
        PyErr_SetString(PyExc_TypeError, "expected a list or tuple of tensors");
        return nullptr;
    }
    int code = PySequence_Fast_GET_SIZE(list) == rows ? OK : COUNT;
    Py_ssize_t i = 0;
    if (code == OK) {
        PyObject** items = PySequence_Fast_ITEMS(list);
        long long* row = reinterpret_cast<long long*>(table);
        for (; i < rows; ++i, row += kColumns) {
            if (!THPVariable_Check(items[i])) {
                code = NOT_TENSOR;
                break;
            }
            const at::Tensor& t = THPVariable_Unpack(items[i]);
            if (t.scalar_type() != type) code = DTYPE;
            else if (!t.is_cuda() || t.device().index() != device) code = DEVICE;
            else if (t.layout() != at::kStrided || !t.is_contiguous()) code = LAYOUT;
            if (code != OK) break;
            const long long n = t.numel();
            if (block == 0) {
                row[kColumns - 1] = n;
            } else if (n != (row[kColumns - 1] + block - 1) / block) {
                code = SIZE;
                break;
            }
            row[col] = reinterpret_cast<long long>(t.data_ptr());
        }
    }
    return Py_BuildValue("in", code, i);
}

// Whether each row (the last axis; the planes of a 4-D tensor) is one run.
bool adjacent(const at::Tensor& t) {
    if (t.is_contiguous() || t.numel() == 0) return true;
    const int64_t n = t.dim();
    if (n == 4 && !(t.size(2) == 1 || t.stride(2) == t.size(3))) return false;
    return t.size(n - 1) == 1 || t.stride(n - 1) == 1;
}

// views(tensors, address) -> index of the first that does not fit, or -1
//
// tensors: a tuple whose first is a CUDA tensor of two to four axes; the others
// are None or of its shape, dtype and device, and all have adjacent rows.
// Writes (pointer, stride of axis 0, stride of axis 1) of each, 64 bits each;
// zeros for None.
PyObject* views(PyObject* args) {
    PyObject* tuple;
    unsigned long long address;
    if (!PyArg_ParseTuple(args, "O!K", &PyTuple_Type, &tuple, &address)) return nullptr;
    long long* out = reinterpret_cast<long long*>(address);
    const Py_ssize_t n = PyTuple_GET_SIZE(tuple);
    const at::Tensor* x = nullptr;
    for (Py_ssize_t i = 0; i < n; ++i, out += 3) {
        PyObject* o = PyTuple_GET_ITEM(tuple, i);
        if (i > 0 && o == Py_None) {
            out[0] = out[1] = out[2] = 0;
            continue;
        }
        if (!THPVariable_Check(o)) return PyLong_FromSsize_t(i);
        const at::Tensor& t = THPVariable_Unpack(o);
        if (i == 0) x = &t;
        if (!t.is_cuda() || t.layout() != at::kStrided || t.dim() < 2 || t.dim() > 4 ||
            t.scalar_type() != x->scalar_type() || t.device() != x->device() ||
            t.sizes() != x->sizes() || !adjacent(t))
            return PyLong_FromSsize_t(i);
        out[0] = reinterpret_cast<long long>(t.data_ptr());
        out[1] = t.stride(0);
        out[2] = t.stride(1);
    }
    return PyLong_FromLong(-1);
}

// flat(tensor, dtype, device, n0, n1) -> address, None for None, False if it
// does not fit: contiguous, of that dtype on that CUDA device, of the shape
// (n0, n1), or (n0,) for a negative n1.
PyObject* flat(PyObject* args) {
    PyObject *o, *dtype;
    int device;
    long long n0, n1;
    if (!PyArg_ParseTuple(args, "OOiLL", &o, &dtype, &device, &n0, &n1)) return nullptr;
    if (o == Py_None) Py_RETURN_NONE;
    if (!THPVariable_Check(o) || !THPDtype_Check(dtype)) Py_RETURN_FALSE;
    const at::Tensor& t = THPVariable_Unpack(o);
    const int dims = n1 < 0 ? 1 : 2;
    if (t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type || !t.is_cuda() ||
        t.device().index() != device || t.layout() != at::kStrided || t.dim() != dims ||
        t.size(0) != n0 || (dims == 2 && t.size(1) != n1) || !t.is_contiguous())
        Py_RETURN_FALSE;
    return PyLong_FromUnsignedLongLong(reinterpret_cast<unsigned long long>(t.data_ptr()));
}

// written(tensors...) -- advances the version counters of what a call has
// written through its addresses, so that autograd sees a change of what it
// saved.  Each argument: a tensor, None, or a list or tuple of tensors.
PyObject* written(PyObject* args) {
    auto bump = [](PyObject* o) {
        if (!THPVariable_Check(o)) return;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();  // those have no counter
    };
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(args); ++i) {
        PyObject* o = PyTuple_GET_ITEM(args, i);
        if (!PyList_Check(o) && !PyTuple_Check(o)) {
            bump(o);
            continue;
        }
        for (Py_ssize_t k = 0; k < PySequence_Fast_GET_SIZE(o); ++k) bump(PySequence_Fast_GET_ITEM(o, k));
    }
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"views", guarded<views>, METH_VARARGS, "Checks strided activations and writes their views."},
                         {"flat", guarded<flat>, METH_VARARGS, "Checks a contiguous tensor and returns its address."},
                         {"column", guarded<column>, METH_VARARGS, "Checks a list of tensors and writes their addresses."},
                         {"written", guarded<written>, METH_VARARGS, "Advances tensors' version counters."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lists() { return PyModule_Create(&module); }
