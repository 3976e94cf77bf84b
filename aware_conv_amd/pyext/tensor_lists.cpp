// Python extension of the AdamW binding (aware_conv_amd/adamw.py): checks the
// tensors of a list and writes their addresses into a host table, in one call.
//
// A step over a hundred small tensors has several hundred of them to check and
// look up; attribute by attribute from Python that takes longer than the step
// itself does on the GPU (96 us for 90 tensors of 4 lists; the GPU takes 13).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

constexpr int kColumns = 8;  // of a row, 64 bits each: seven addresses, then the number of elements

// What is wrong with a list, for the caller to put into words.
enum { OK, COUNT, NOT_TENSOR, DTYPE, DEVICE, LAYOUT, SIZE };

// column(tensors, table, rows, column, dtype, device, block) -> (code, index)
//
// tensors: a list or tuple.  table: address of `rows` rows.  column: where the
// addresses go.  block: 0 writes the numbers of elements to the last column;
// k > 0 expects ceil(n / k) elements for the n found there.
PyObject* column(PyObject*, PyObject* args) {
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
    PyObject* seq = PySequence_Fast(list, "expected a list of tensors");
    if (!seq) return nullptr;
    int code = PySequence_Fast_GET_SIZE(seq) == rows ? OK : COUNT;
    Py_ssize_t i = 0;
    if (code == OK) {
        PyObject** items = PySequence_Fast_ITEMS(seq);
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
    Py_DECREF(seq);
    return Py_BuildValue("in", code, i);
}

PyMethodDef methods[] = {{"column", column, METH_VARARGS, "Checks a list of tensors and writes their addresses."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lists() { return PyModule_Create(&module); }
