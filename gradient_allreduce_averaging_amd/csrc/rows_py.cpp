// The tensors of a call over rows of tokens, checked and laid out as the C
// calls take them (rms_norm*, distill_*): the Python module _rows.  A call on
// small tensors is bound by this work, and a tensor's address, type and strides
// cost a tenth of a microsecond each from Python and a few nanoseconds here: the
// norm of one token takes 5.4 us for the whole call and took 9.6, the gradient of
// 8 ranks of 2 tokens 15 and took 32.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/TensorBase.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

namespace {

// What an operand may hold, and the code of each type as the C calls take it
// (an index: its bytes).
enum : long { kMaskF32 = 1, kMaskBF16 = 2, kMaskI8 = 4, kMaskE4M3 = 8, kMaskI32 = 16, kMaskI64 = 32 };
struct Type {
    long mask;
    int code;
};
Type type_of(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return {kMaskF32, 0};
    case at::kBFloat16: return {kMaskBF16, 1};
    case at::kChar: return {kMaskI8, 2};
    case at::kFloat8_e4m3fn: return {kMaskE4M3, 3};
    case at::kInt: return {kMaskI32, 4};
    case at::kLong: return {kMaskI64, 8};
    default: return {0, -1};
    }
}

const at::Tensor *tensor_of(PyObject *o, const char *what)
{
    if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
    PyErr_Format(PyExc_TypeError, "%s: a tensor is required", what);
    return nullptr;
}

bool on_device(const at::Tensor &t, long device, const char *what)
{
    if (t.is_cuda() && t.get_device() == device) return true;
    PyErr_Format(PyExc_ValueError, "%s: tensor is not on %s GPU", what, t.is_cuda() ? "the current" : "a");
    return false;
}

bool type_ok(const at::Tensor &t, long mask, const char *what, int *code)
{
    const Type ty = type_of(t.scalar_type());
    *code = ty.code;
    if (ty.mask & mask) return true;
    PyErr_Format(PyExc_TypeError, "%s: unsupported dtype %s", what, at::toString(t.scalar_type()));
    return false;
}

// Elements from row to row of a tensor taken as rows of its last dimension;
// false where the rows are not one fixed distance apart.
bool row_stride(const at::Tensor &t, int64_t *pitch)
{
    const auto size = t.sizes(), stride = t.strides();
    const int64_t last = (int64_t)size.size() - 1;
    int64_t rows = 1;
    for (int64_t d = last - 1; d >= 0; --d) {
        if (size[d] == 1) continue;
        if (rows == 1)
            *pitch = stride[d];
        else if (stride[d] != rows * *pitch)
            return false;
        rows *= size[d];
    }
    return true;
}

// An operand's form, where it is not a width of its own.
enum : long { kLike = -1, kRows = -2, kWidth = -3, kOwn = -4 };

// An object that this code owns.
struct Ref {
    PyObject *o = nullptr;
    ~Ref() { Py_XDECREF(o); }
};

// The layout of one call under way.
struct Call {
    long device;
    Py_ssize_t n = 0;              // ranks
    int64_t width = 0, own = 0;    // of kLike and kOwn operands
    int64_t *words = nullptr, *next = nullptr;
};

// The rows and the width of rank r's tensor of the first operand.
bool set_rows(Call &c, const at::Tensor &t, const char *what, Py_ssize_t r)
{
    const auto size = t.sizes();
    if (size.empty()) {
        PyErr_Format(PyExc_ValueError, "%s: a rank's tensor needs a dimension for the width", what);
        return false;
    }
    if (r == 0) c.width = size.back();
    if (c.width < 1) {
        PyErr_Format(PyExc_ValueError, "%s: the width is 0", what);
        return false;
    }
    c.words[r] = size.back() ? t.numel() / size.back() : 0;
    return true;
}

// One matrix operand: its addresses, then its ddp_rows_t, whose address is
// returned; 0 with an error set.
int64_t matrix(Call &c, PyObject **ts, const char *what, long mask, int64_t width, int *code, bool first)
{
    int64_t *const rank = c.next;
    int64_t stride = -1;
    for (Py_ssize_t r = 0; r < c.n; ++r) {
        const at::Tensor *t = tensor_of(ts[r], what);
        if (!t || !on_device(*t, c.device, what)) return 0;
        int mine;
        if (!type_ok(*t, mask, what, &mine)) return 0;
        if (r == 0) *code = mine;
        if (mine != *code) {
            PyErr_Format(PyExc_ValueError, "%s: the ranks differ in dtype", what);
            return 0;
        }
        if (first) {
            if (!set_rows(c, *t, what, r)) return 0;
            width = c.width;
        }
        const int64_t rows = c.words[r];
        const auto size = t->sizes();
        if (size.empty() || size.back() != width || t->numel() != rows * width) {
            PyErr_Format(PyExc_ValueError, "%s: %lld rows of %lld elements are required", what, (long long)rows,
                         (long long)width);
            return 0;
        }
        if (rows > 0) {
            if (width > 1 && t->strides().back() != 1) {
                PyErr_Format(PyExc_ValueError, "%s: the elements of a row are not consecutive", what);
                return 0;
            }
            int64_t pitch = width;
            if (!row_stride(*t, &pitch)) {
                PyErr_Format(PyExc_ValueError, "%s: the rows are not one fixed distance apart", what);
                return 0;
            }
            if (rows > 1 && pitch != stride) {
                if (stride >= 0) {
                    PyErr_Format(PyExc_ValueError, "%s: the ranks differ in row stride", what);
                    return 0;
                }
                stride = pitch;
            }
        }
        *c.next++ = (int64_t)(intptr_t)t->data_ptr();
    }
    int64_t *const m = c.next;
    *c.next++ = (int64_t)(intptr_t)rank;
    *c.next++ = stride >= 0 ? stride : width;
    return (int64_t)(intptr_t)m;
}

int64_t vectors(Call &c, PyObject **ts, const char *what, long mask, bool per_row, int *code)
{
    int64_t *const rank = c.next;
    for (Py_ssize_t r = 0; r < c.n; ++r) {
        const at::Tensor *t = tensor_of(ts[r], what);
        if (!t || !on_device(*t, c.device, what)) return 0;
        int mine;
        if (!type_ok(*t, mask, what, &mine)) return 0;
        if (r == 0) *code = mine;
        if (mine != *code) {
            PyErr_Format(PyExc_ValueError, "%s: the ranks differ in dtype", what);
            return 0;
        }
        const int64_t want = per_row ? c.words[r] : c.width;
        if (t->numel() != want || !t->is_contiguous()) {
            PyErr_Format(PyExc_ValueError, "%s: %lld contiguous elements are required", what, (long long)want);
            return 0;
        }
        *c.next++ = (int64_t)(intptr_t)t->data_ptr();
    }
    return (int64_t)(intptr_t)rank;
}

// pack(device, (tensors, name, types, form), ...): each operand is None or one
// tensor for each rank, of one of `types`, in the form
//   LIKE    a matrix like the first operand's: its last dimension is the width, the
//           others are the rank's rows (tokens)
//   ROWS    a vector of one element for each row
//   WIDTH   a vector of as many elements as the width
//   OWN     a matrix of another width, the same for all of this form
// Returns (words, ranks, width, OWN width, address of the row counts, then a type
// code and an address for each operand).  `words` holds the row counts, the pointer
// arrays and the ddp_rows_t: it has to outlive the call.
PyObject *pack_operands(PyObject *const *args, Py_ssize_t nargs)
{
    constexpr Py_ssize_t kMost = 10;
    const Py_ssize_t ops = nargs - 1;
    if (ops < 1 || ops > kMost) return PyErr_Format(PyExc_TypeError, "pack: 1 to %zd operands", kMost);
    Call c;
    c.device = PyLong_AsLong(args[0]);
    if (c.device == -1 && PyErr_Occurred()) return nullptr;
    Ref seq[kMost];   // the sequences' items, until the return
    const char *what[kMost];
    long mask[kMost], form[kMost];
    for (Py_ssize_t k = 0; k < ops; ++k) {
        PyObject *ts;
        if (!PyTuple_Check(args[k + 1]) || !PyArg_ParseTuple(args[k + 1], "Osll", &ts, &what[k], &mask[k], &form[k]))
            return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_TypeError, "pack: a tuple is required");
        if (ts == Py_None && k > 0) continue;
        seq[k].o = PySequence_Fast(ts, "one tensor per rank is required");
        if (!seq[k].o) return nullptr;
        const Py_ssize_t len = PySequence_Fast_GET_SIZE(seq[k].o);
        if (k == 0) {
            c.n = len;
            if (len == 0) return PyErr_Format(PyExc_ValueError, "%s: no ranks", what[k]);
        } else if (len != c.n) {
            return PyErr_Format(PyExc_ValueError, "%s: one tensor per rank is required", what[k]);
        }
    }
    PyObject *words = PyByteArray_FromStringAndSize(nullptr, 8 * (c.n + ops * (c.n + 2)));
    if (!words) return nullptr;
    Ref out{PyTuple_New(5 + 2 * ops)};
    if (!out.o) {
        Py_DECREF(words);
        return nullptr;
    }
    PyTuple_SET_ITEM(out.o, 0, words);
    c.words = reinterpret_cast<int64_t *>(PyByteArray_AS_STRING(words));
    c.next = c.words + c.n;
    for (Py_ssize_t k = 0; k < ops; ++k) {
        PyObject *code = Py_None, *address = Py_None;
        if (seq[k].o) {
            PyObject **ts = PySequence_Fast_ITEMS(seq[k].o);
            int type = 0;
            int64_t at = 0;
            if (form[k] == kRows || form[k] == kWidth) {
                at = vectors(c, ts, what[k], mask[k], form[k] == kRows, &type);
            } else {
                if (form[k] == kOwn && c.own == 0) {
                    const at::Tensor *t = tensor_of(ts[0], what[k]);
                    if (t && t->dim() > 0) c.own = t->size(-1);
                }
                if (!PyErr_Occurred())
                    at = matrix(c, ts, what[k], mask[k], form[k] == kOwn ? c.own : c.width, &type, k == 0);
            }
            if (!at) return nullptr;
            code = PyLong_FromLong(type);
            address = PyLong_FromLongLong(at);
        } else {
            Py_INCREF(code);
            Py_INCREF(address);
        }
        PyTuple_SET_ITEM(out.o, 5 + 2 * k, code);
        PyTuple_SET_ITEM(out.o, 6 + 2 * k, address);
    }
    PyTuple_SET_ITEM(out.o, 1, PyLong_FromSsize_t(c.n));
    PyTuple_SET_ITEM(out.o, 2, PyLong_FromLongLong(c.width));
    PyTuple_SET_ITEM(out.o, 3, PyLong_FromLongLong(c.own));
    PyTuple_SET_ITEM(out.o, 4, PyLong_FromLongLong((int64_t)(intptr_t)c.words));
    for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(out.o); ++k)
        if (!PyTuple_GET_ITEM(out.o, k)) return nullptr;   // no memory
    Py_INCREF(out.o);
    return out.o;
}

// span(device, tensor, name, types, length): (type code, address, bytes) of a
// contiguous tensor that every rank shares; (0, None, 0) for None.  length -1: any;
// types 0: any.
PyObject *span_of(PyObject *const *args, Py_ssize_t nargs)
{
    if (nargs != 5) return PyErr_Format(PyExc_TypeError, "span: 5 arguments");
    if (args[1] == Py_None) return Py_BuildValue("iOi", 0, Py_None, 0);
    const long device = PyLong_AsLong(args[0]), mask = PyLong_AsLong(args[3]);
    const long long length = PyLong_AsLongLong(args[4]);
    const char *what = PyUnicode_AsUTF8(args[2]);
    if (PyErr_Occurred()) return nullptr;
    const at::Tensor *t = tensor_of(args[1], what);
    if (!t || !on_device(*t, device, what)) return nullptr;
    int code = 0;
    if (mask && !type_ok(*t, mask, what, &code)) return nullptr;
    if (length >= 0 && t->numel() != length)
        return PyErr_Format(PyExc_ValueError, "%s: %lld elements are required, got %lld", what, length,
                            (long long)t->numel());
    if (!t->is_contiguous()) return PyErr_Format(PyExc_ValueError, "%s: tensor is not contiguous", what);
    return Py_BuildValue("iLL", code, (long long)(intptr_t)t->data_ptr(), (long long)t->nbytes());
}

// No C++ exception (a tensor without storage, say) leaves the module.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    try {
        return F(args, nargs);
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyMethodDef kMethods[] = {
    {"pack", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&guarded<pack_operands>)), METH_FASTCALL,
     "The operands of one call over rows of tokens, as the C call takes them."},
    {"span", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&guarded<span_of>)), METH_FASTCALL,
     "A tensor that every rank shares."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_rows", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rows()
{
    PyObject *m = PyModule_Create(&kModule);
    if (!m) return nullptr;
    const struct { const char *name; long value; } constants[] = {
        {"F32", kMaskF32}, {"BF16", kMaskBF16}, {"I8", kMaskI8}, {"E4M3", kMaskE4M3}, {"I32", kMaskI32},
        {"I64", kMaskI64}, {"LIKE", kLike}, {"ROWS", kRows}, {"WIDTH", kWidth}, {"OWN", kOwn}};
    for (const auto &k : constants)
        if (PyModule_AddIntConstant(m, k.name, k.value) < 0) {
            Py_DECREF(m);
            return nullptr;
        }
    return m;
}
