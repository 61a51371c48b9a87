// tensors.cpp -- the Python binding's look at torch tensors, for calls that
// take several tensors per worker: types, devices, shapes and strides checked
// and addresses packed in one pass. (Through Python's attributes the same
// takes 0.5 us a tensor: 16 us of a call with 8 workers' four tensors, as
// long as such a call's kernels run.) Host code; addresses and counts go on
// to the C ABI as bytes.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

namespace {

// The binding's type codes (the first two are ga_dtype).
constexpr at::ScalarType kTypes[] = {at::kFloat, at::kBFloat16, at::kInt, at::kByte, at::kBool};
constexpr int kNumTypes = 5;

// A sequence of tensors; throws nothing, sets Python's error.
struct Tensors {
    PyObject* seq = nullptr;
    Py_ssize_t n = 0;
    bool open(PyObject* o, const char* what) {
        seq = PySequence_Fast(o, "one tensor per worker, as a sequence");
        if (!seq) return false;
        n = PySequence_Fast_GET_SIZE(seq);
        for (Py_ssize_t i = 0; i < n; i++)
            if (!THPVariable_Check(PySequence_Fast_GET_ITEM(seq, i))) {
                PyErr_Format(PyExc_TypeError, "%s must be tensors", what);
                return false;
            }
        return true;
    }
    const at::Tensor& operator[](Py_ssize_t i) const { return THPVariable_Unpack(PySequence_Fast_GET_ITEM(seq, i)); }
    ~Tensors() { Py_XDECREF(seq); }
};

int device_of(const at::Tensor& t) { return t.is_cuda() ? (int)t.get_device() : -1; }

// A tensor whose memory holds its values (no sparse one, no lazy negation).
bool usable(const at::Tensor& t, const char* what) {
    if (t.defined() && t.layout() == at::kStrided && t.has_storage() && !t.is_neg()) return true;
    PyErr_Format(PyExc_TypeError, "%s must be strided tensors with values of their own", what);
    return false;
}

bool same_kind(const at::Tensor& t, const char* what, int type, int device) {
    if (!usable(t, what)) return false;
    if (t.scalar_type() == kTypes[type] && device_of(t) == device) return true;
    const std::string d = t.device().str();
    PyErr_Format(PyExc_TypeError, "%s must be %s on cuda:%d, not %s on %s", what, c10::toString(kTypes[type]), device,
                 c10::toString(t.scalar_type()), d.c_str());
    return false;
}

// The row stride of matrices of rows[i] x cols; -1 with an error set.
int64_t row_stride(const Tensors& ts, const char* what, const int64_t* rows, int64_t cols) {
    int64_t ld = -1;
    for (Py_ssize_t i = 0; i < ts.n; i++) {
        const at::Tensor& t = ts[i];
        if (t.dim() != 2 || t.size(0) != rows[i] || t.size(1) != cols) {
            PyErr_Format(PyExc_ValueError, "%s of worker %zd must be a matrix of %lld x %lld", what, i,
                         (long long)rows[i], (long long)cols);
            return -1;
        }
        if (rows[i] && cols > 1 && t.stride(1) != 1) {
            PyErr_Format(PyExc_ValueError, "%s must have consecutive columns", what);
            return -1;
        }
        if (rows[i] > 1) {
            if (t.stride(0) < cols || (ld >= 0 && t.stride(0) != ld)) {
                PyErr_Format(PyExc_ValueError, "all workers' %s need the same row stride, of at least a row", what);
                return -1;
            }
            ld = t.stride(0);
        }
    }
    return ld < 0 ? cols : ld;
}

PyObject* pointers(const Tensors& ts) {
    PyObject* b = PyBytes_FromStringAndSize(nullptr, ts.n * (Py_ssize_t)sizeof(void*));
    if (!b) return nullptr;
    void** p = reinterpret_cast<void**>(PyBytes_AS_STRING(b));
    for (Py_ssize_t i = 0; i < ts.n; i++) p[i] = ts[i].data_ptr();
    return b;
}

// The row counts packed by logits(), checked against a sequence's length.
const int64_t* rows_of(PyObject* o, Py_ssize_t n, const char* what) {
    if (!PyBytes_Check(o)) {
        PyErr_SetString(PyExc_TypeError, "row counts must be bytes");
        return nullptr;
    }
    if (PyBytes_GET_SIZE(o) != n * (Py_ssize_t)sizeof(int64_t)) {
        PyErr_Format(PyExc_ValueError, "%zd %s for %zd workers", n, what,
                     PyBytes_GET_SIZE(o) / (Py_ssize_t)sizeof(int64_t));
        return nullptr;
    }
    return reinterpret_cast<const int64_t*>(PyBytes_AS_STRING(o));
}

// logits(tensors) -> (pointers, row counts, rows, columns, stride, type, device)
PyObject* logits(PyObject* o) {
    Tensors ts;
    if (!ts.open(o, "logits")) return nullptr;
    if (!ts.n) {
        PyErr_SetString(PyExc_ValueError, "no workers");
        return nullptr;
    }
    const at::Tensor& t0 = ts[0];
    const int type = t0.scalar_type() == at::kFloat ? 0 : t0.scalar_type() == at::kBFloat16 ? 1 : -1;
    if (type < 0) {
        PyErr_Format(PyExc_TypeError, "logits are float32 or bfloat16, not %s", c10::toString(t0.scalar_type()));
        return nullptr;
    }
    if (!t0.is_cuda()) {
        PyErr_SetString(PyExc_ValueError, "logits must be GPU tensors");
        return nullptr;
    }
    const int device = device_of(t0);
    std::vector<int64_t> rows(ts.n);
    int64_t sum = 0;
    for (Py_ssize_t i = 0; i < ts.n; i++) {
        if (!same_kind(ts[i], "logits", type, device)) return nullptr;
        if (ts[i].dim() != 2) {
            PyErr_SetString(PyExc_ValueError, "logits are matrices, rows x columns");
            return nullptr;
        }
        sum += rows[i] = ts[i].size(0);
    }
    const int64_t cols = t0.size(1), ld = row_stride(ts, "logits", rows.data(), cols);
    if (ld < 0) return nullptr;
    PyObject* p = pointers(ts);
    if (!p) return nullptr;
    return Py_BuildValue("Ny#LLLii", p, (const char*)rows.data(), (Py_ssize_t)(ts.n * sizeof(int64_t)),
                         (long long)sum, (long long)cols, (long long)ld, type, device);
}

// matrices(tensors, what, type, device, row counts, columns) -> (pointers, stride)
PyObject* matrices(PyObject* o, const char* what, int type, int device, PyObject* counts, long long cols) {
    Tensors ts;
    if (!ts.open(o, what)) return nullptr;
    const int64_t* rows = rows_of(counts, ts.n, what);
    if (!rows) return nullptr;
    for (Py_ssize_t i = 0; i < ts.n; i++)
        if (!same_kind(ts[i], what, type, device)) return nullptr;
    const int64_t ld = row_stride(ts, what, rows, cols);
    if (ld < 0) return nullptr;
    PyObject* p = pointers(ts);
    return p ? Py_BuildValue("NL", p, (long long)ld) : nullptr;
}

// dense(tensors, what, type, device, row counts, columns) -> pointers of dense
// matrices, or (columns < 0) vectors
PyObject* dense(PyObject* o, const char* what, int type, int device, PyObject* counts, long long cols) {
    Tensors ts;
    if (!ts.open(o, what)) return nullptr;
    const int64_t* rows = rows_of(counts, ts.n, what);
    if (!rows) return nullptr;
    for (Py_ssize_t i = 0; i < ts.n; i++) {
        const at::Tensor& t = ts[i];
        if (!same_kind(t, what, type, device)) return nullptr;
        const bool shape = cols < 0 ? t.dim() == 1 && t.size(0) == rows[i]
                                    : t.dim() == 2 && t.size(0) == rows[i] && t.size(1) == cols;
        if (!shape || !t.is_contiguous()) {
            PyErr_Format(PyExc_ValueError, "%s of worker %zd must be dense, %lld rows of %lld", what, i,
                         (long long)rows[i], cols < 0 ? 1 : cols);
            return nullptr;
        }
    }
    return pointers(ts);
}

// one(tensor, what, type, device, numel) -> address of a dense tensor
PyObject* one(PyObject* o, const char* what, int type, int device, long long numel) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
        return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!same_kind(t, what, type, device)) return nullptr;
    if (t.numel() != numel || !t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be %lld dense values", what, numel);
        return nullptr;
    }
    return PyLong_FromVoidPtr(t.data_ptr());
}

// written(tensor, tensors, None, truth value, ...): the version of every tensor
// goes up, so that a backward pass that saved what stood there before is
// refused. (Tensors of inference mode have none.)
PyObject* written(PyObject* args) {
    auto bump = [](const at::Tensor& t) {
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    };
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(args); i++) {
        PyObject* o = PyTuple_GET_ITEM(args, i);
        if (o == Py_None || PyBool_Check(o)) continue;
        if (THPVariable_Check(o)) {
            bump(THPVariable_Unpack(o));
            continue;
        }
        Tensors ts;
        if (!ts.open(o, "outputs")) return nullptr;
        for (Py_ssize_t k = 0; k < ts.n; k++) bump(ts[k]);
    }
    Py_RETURN_NONE;
}

// No C++ exception leaves the module.
template <class F> PyObject* guarded(F f) {
    try {
        return f();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

bool type_ok(int type) {
    if (type >= 0 && type < kNumTypes) return true;
    PyErr_Format(PyExc_ValueError, "unknown type code %d", type);
    return false;
}

PyObject* py_logits(PyObject*, PyObject* o) {
    return guarded([&] { return logits(o); });
}

template <PyObject* F(PyObject*, const char*, int, int, PyObject*, long long)>
PyObject* py_list(PyObject*, PyObject* args) {
    PyObject *o, *rows;
    const char* what;
    int type, device;
    long long cols;
    if (!PyArg_ParseTuple(args, "OsiiOL", &o, &what, &type, &device, &rows, &cols) || !type_ok(type)) return nullptr;
    return guarded([&] { return F(o, what, type, device, rows, cols); });
}

PyObject* py_one(PyObject*, PyObject* args) {
    PyObject* o;
    const char* what;
    int type, device;
    long long numel;
    if (!PyArg_ParseTuple(args, "OsiiL", &o, &what, &type, &device, &numel) || !type_ok(type)) return nullptr;
    return guarded([&] { return one(o, what, type, device, numel); });
}

PyObject* py_written(PyObject*, PyObject* args) {
    return guarded([&] { return written(args); });
}

PyMethodDef kMethods[] = {
    {"logits", py_logits, METH_O, "(pointers, row counts, rows, columns, stride, type, device) of the workers' logits"},
    {"matrices", py_list<matrices>, METH_VARARGS, "(pointers, stride) of matrices that match the logits' rows"},
    {"dense", py_list<dense>, METH_VARARGS, "pointers of dense matrices or vectors that match the logits' rows"},
    {"one", py_one, METH_VARARGS, "address of a dense tensor"},
    {"written", py_written, METH_VARARGS, "the versions of tensors that were given and written go up"},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_tensors", "Checks and addresses of torch tensors.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&kModule); }
