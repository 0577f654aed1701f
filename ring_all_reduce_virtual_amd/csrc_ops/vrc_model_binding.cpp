// vrc_model_binding.cpp -- the Python binding of include/vrc_model.h as a compiled
// module (_vrc_model.so): it checks tensors, allocates outputs and workspaces from
// torch's allocator and calls libvrc_ops.so.  A small call's time is its host's: of
// an all-reduced token (8 ranks: 16 tensors checked, 11 allocated) the same steps
// take 26 us in Python.  model.py holds the documented functions.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

#include "vrc_model.h"
#include "vrc_ops.h"

namespace {

constexpr int kMaxRanks = 16;

// An error that is already set in the interpreter.
struct Set {};

[[noreturn]] void fail(PyObject* type, const char* where, const char* text)
{
    PyErr_Format(type, "%s: %s", where, text);
    throw Set{};
}
[[noreturn]] void refuse(const char* where, const char* text) { fail(PyExc_ValueError, where, text); }

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* where, const char* what)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_ValueError, "%s: %s must be a tensor", where, what);
        throw Set{};
    }
    return THPVariable_Unpack(o);
}

typedef c10::SmallVector<int64_t, 6> Shape;

int64_t product(const Shape& s)
{
    int64_t p = 1;
    for (const int64_t k : s) p *= k;
    return p;
}

// What every tensor of a call shares, from its first.
struct Like {
    at::ScalarType type;
    at::Device device;
    int dtype;  // vrc_dtype_t
    at::TensorOptions options(at::ScalarType t) const { return at::TensorOptions().dtype(t).device(device); }
};

Like like(const at::Tensor& t, const char* where)
{
    if (!t.is_cuda()) refuse(where, "tensors must live on the GPU");
    const auto type = t.scalar_type();
    int code = -1;
    if (type == at::kFloat) code = VRC_FP32;
    else if (type == at::kHalf) code = VRC_FP16;
    else if (type == at::kBFloat16) code = VRC_BF16;
    else fail(PyExc_TypeError, where, "unsupported dtype");
    return {type, t.device(), code};
}

std::string text(const Shape& s)
{
    std::string t = "[";
    for (size_t i = 0; i < s.size(); i++) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

// One contiguous tensor of a shape, type and device.
const at::Tensor& same(PyObject* o, const Shape& shape, at::ScalarType type, const Like& l, const char* where, const char* what)
{
    const at::Tensor& t = tensor(o, where, what);
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || t.device() != l.device || !t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s: %s must be contiguous %s of the call's type, on the inputs' device", where, what,
                     text(shape).c_str());
        throw Set{};
    }
    return t;
}

// The items of a list or tuple (borrowed); throws on anything else.
struct Items {
    PyObject** at = nullptr;
    Py_ssize_t n = 0;
    Items(PyObject* o, const char* where, const char* what)
    {
        if (!PyList_Check(o) && !PyTuple_Check(o)) {
            PyErr_Format(PyExc_ValueError, "%s: %s must be a list of one tensor per rank", where, what);
            throw Set{};
        }
        at = PySequence_Fast_ITEMS(o);
        n = PySequence_Fast_GET_SIZE(o);
    }
};

// One tensor per rank, all of one shape: their pointers.  The first is `t0`.
int ranks(PyObject* o, const char* where, void** p, const at::Tensor** t0)
{
    const Items items(o, where, "the first argument");
    if (items.n == 0) refuse(where, "expected a non-empty list of tensors, one per rank");
    if (items.n > kMaxRanks) refuse(where, "at most 16 ranks");
    const at::Tensor& first = tensor(items.at[0], where, "every rank's argument");
    if (!first.is_cuda()) refuse(where, "tensors must live on the GPU");
    for (Py_ssize_t r = 0; r < items.n; r++) {
        const at::Tensor& t = tensor(items.at[r], where, "every rank's argument");
        if (t.scalar_type() != first.scalar_type() || t.sizes() != first.sizes() || t.device() != first.device())
            refuse(where, "all ranks need the same dtype, shape and device");
        if (!t.is_contiguous()) refuse(where, "tensors must be contiguous");
        p[r] = t.data_ptr();
    }
    *t0 = &first;
    return (int)items.n;
}

// What there is one of per part: a list, or a single tensor where all ranks share it.
void parts(PyObject* o, const std::vector<Shape>& shapes, at::ScalarType type, const Like& l, bool one, const char* where,
           const char* what, void** p)
{
    if (one) {
        p[0] = same(o, shapes[0], type, l, where, what).data_ptr();
        return;
    }
    const Items items(o, where, what);
    if (items.n != (Py_ssize_t)shapes.size()) {
        PyErr_Format(PyExc_ValueError, "%s: %s must be one tensor per rank", where, what);
        throw Set{};
    }
    for (Py_ssize_t i = 0; i < items.n; i++) p[i] = same(items.at[i], shapes[i], type, l, where, what).data_ptr();
}

PyObject* none()
{
    Py_INCREF(Py_None);
    return Py_None;
}

// An owned reference.
struct Ref {
    PyObject* o = nullptr;
    explicit Ref(PyObject* p) : o(p)
    {
        if (!p) throw Set{};
    }
    Ref(Ref&& r) : o(r.o) { r.o = nullptr; }
    Ref(const Ref&) = delete;
    ~Ref() { Py_XDECREF(o); }
    PyObject* take()
    {
        PyObject* p = o;
        o = nullptr;
        return p;
    }
};

// New tensors, each with a storage of its own (one that is resized in place, kept or
// saved then reaches no other): a list, or the tensor itself where all ranks share it.
Ref allocate(const std::vector<Shape>& shapes, at::ScalarType type, const Like& l, bool one, void** p)
{
    const auto options = l.options(type);
    if (one) {
        const at::Tensor t = at::empty(shapes[0], options);
        p[0] = t.data_ptr();
        return Ref(THPVariable_Wrap(t));
    }
    Ref list(PyList_New((Py_ssize_t)shapes.size()));
    for (size_t i = 0; i < shapes.size(); i++) {
        const at::Tensor t = at::empty(shapes[i], options);
        p[i] = t.data_ptr();
        PyList_SET_ITEM(list.o, (Py_ssize_t)i, Ref(THPVariable_Wrap(t)).take());
    }
    return list;
}

// Outputs that the caller may bring.
Ref outputs(PyObject* given_, const std::vector<Shape>& shapes, at::ScalarType type, const Like& l, bool one, const char* where,
            const char* what, void** p)
{
    if (!given(given_)) return allocate(shapes, type, l, one, p);
    parts(given_, shapes, type, l, one, where, what, p);
    Py_INCREF(given_);
    return Ref(given_);
}

at::Tensor workspace(size_t bytes, const Like& l) { return at::empty({(int64_t)bytes}, l.options(at::kByte)); }

// The stream to enqueue on: a handle, or that of the device's current stream.
PyObject* g_current_stream = nullptr;  // model.py's, of a device index
vrc_stream_t stream_of(PyObject* o, const Like& l)
{
    PyObject* handle = o;
    Ref found = given(o) ? (Py_INCREF(o), Ref(o)) : Ref(PyObject_CallFunction(g_current_stream, "i", (int)l.device.index()));
    handle = found.o;
    void* p = PyLong_AsVoidPtr(handle);
    if (!p && PyErr_Occurred()) throw Set{};
    return (vrc_stream_t)p;
}

double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Set{};
    return v;
}

long whole(PyObject* o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Set{};
    return v;
}

bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Set{};
    return v != 0;
}

void expect(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    throw Set{};
}

PyObject* g_out_of_memory = nullptr;  // torch's exception
PyObject* g_done = nullptr;           // model.py's: raises for a status that is an error
void done(vrc_status_t st, const char* where)
{
    if (st == VRC_OK) return;
    Ref r(PyObject_CallFunction(g_done, "is", (int)st, where));
    fail(PyExc_RuntimeError, where, "failed");
}

template <class F>
void call(const char* where, F f)
{
    vrc_status_t st;
    Py_BEGIN_ALLOW_THREADS st = f();
    Py_END_ALLOW_THREADS done(st, where);
}

template <class F>
PyObject* guarded(F f)
{
    try {
        return f();
    } catch (const Set&) {
    } catch (const c10::Error& e) {  // the allocator's, as torch's own calls raise it
        const bool memory = dynamic_cast<const c10::OutOfMemoryError*>(&e) != nullptr;
        PyErr_SetString(memory && g_out_of_memory ? g_out_of_memory : PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// ---------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------
struct NormShapes {
    int64_t rows, width;
    std::vector<Shape> parts, outs, lines;  // of h; of y; of mean and rstd
    bool one;
};

NormShapes norm_shapes(const at::Tensor& t, int n, int join, const char* where)
{
    if (t.dim() == 0) refuse(where, "tensors need at least one dimension");
    NormShapes s;
    const Shape shape(t.sizes().begin(), t.sizes().end()), line(shape.begin(), shape.end() - 1);
    s.width = shape.back();
    s.rows = product(line);
    s.one = join == VRC_NORM_SUM;
    if (join == VRC_NORM_SCATTER) {
        for (int c = 0; c < n; c++) {
            const int64_t each = s.rows / n, k = c + 1 < n ? each : s.rows - each * (n - 1);
            s.parts.push_back({k, s.width});
            s.lines.push_back({k});
        }
        s.outs = s.parts;
    } else {
        s.parts.assign(s.one ? 1 : n, shape);
        s.lines.assign(s.one ? 1 : n, line);
        s.outs.assign(n, shape);
    }
    return s;
}

const at::Tensor& norm_weight(PyObject* o, int64_t width, const Like& l, const char* where)
{
    const at::Tensor& w = tensor(o, where, "weight");
    if (w.scalar_type() != l.type && w.scalar_type() != at::kFloat)
        fail(PyExc_TypeError, where, "weight must be of the rows' dtype or float32");
    return same(o, Shape{width}, w.scalar_type(), l, where, "weight");
}

vrc_layer_norm_t norm_of(const NormShapes& s, const Like& l, const at::Tensor& w, int join, bool center, double eps)
{
    return {(size_t)s.rows, (size_t)s.width, (vrc_dtype_t)l.dtype, w.scalar_type() == at::kFloat ? VRC_FP32 : (vrc_dtype_t)l.dtype,
            (vrc_norm_join_t)join, center, eps};
}

// (send, weight, bias, eps, residual, join, center, recv, sum, stream) -> (y, h, mean, rstd)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded([&]() -> PyObject* {
        const char* where = "vrc_layer_norm";
        expect(count, 10);
        const int join = (int)whole(a[5]);
        const bool center = truth(a[6]);
        void *x[kMaxRanks], *res[kMaxRanks], *y[kMaxRanks], *h[kMaxRanks], *mean[kMaxRanks], *rstd[kMaxRanks];
        const at::Tensor* t0;
        const int n = ranks(a[0], where, x, &t0);
        const Like l = like(*t0, where);
        const NormShapes s = norm_shapes(*t0, n, join, where);
        const at::Tensor& w = norm_weight(a[1], s.width, l, where);
        const void* b = given(a[2]) ? same(a[2], Shape{s.width}, w.scalar_type(), l, where, "bias").data_ptr() : nullptr;
        const bool residual = given(a[4]), added = residual || join != VRC_NORM_EACH;
        if (residual) parts(a[4], s.parts, l.type, l, s.one, where, "residual", res);
        if (given(a[8]) && !added) refuse(where, "without a residual each rank's rows are their own sum");
        const vrc_layer_norm_t d = norm_of(s, l, w, join, center, number(a[3]));
        const vrc_stream_t st = stream_of(a[9], l);
        Ref ys = outputs(a[7], s.outs, l.type, l, false, where, "recv", y);
        // rows that nothing is added to are their own sum, unless y takes their place
        bool over = false;
        for (int r = 0; r < n && !added; r++) over |= s.rows && s.width && y[r] == x[r];
        Ref hs = added ? outputs(a[8], s.parts, l.type, l, s.one, where, "sum", h) : over ? Ref(none()) : (Py_INCREF(a[0]), Ref(a[0]));
        Ref means = center ? allocate(s.lines, at::kFloat, l, s.one, mean) : Ref(none());
        Ref rstds = allocate(s.lines, at::kFloat, l, s.one, rstd);
        call(where, [&] {
            return vrc_layer_norm(&d, x, residual ? res : nullptr, w.data_ptr(), b, y, added ? h : nullptr,
                                  center ? (float* const*)mean : nullptr, (float* const*)rstd, n, st);
        });
        return PyTuple_Pack(4, ys.o, hs.o, means.o, rstds.o);
    });
}

// (dy, h, weight, mean, rstd, dh, join, bias, recv, stream) -> (dx, dweight, dbias)
PyObject* layer_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded([&]() -> PyObject* {
        const char* where = "vrc_layer_norm_grad";
        expect(count, 10);
        const int join = (int)whole(a[6]);
        const bool center = given(a[3]), residual = given(a[5]), bias = truth(a[7]);
        void *dy[kMaxRanks], *h[kMaxRanks], *mean[kMaxRanks], *rstd[kMaxRanks], *res[kMaxRanks], *dx[kMaxRanks], *dw, *db = nullptr;
        const at::Tensor* t0;
        const int n = ranks(a[0], where, dy, &t0);
        const Like l = like(*t0, where);
        const NormShapes s = norm_shapes(*t0, n, join, where);
        const at::Tensor& w = norm_weight(a[2], s.width, l, where);
        parts(a[1], s.parts, l.type, l, s.one, where, "h", h);
        if (center) parts(a[3], s.lines, at::kFloat, l, s.one, where, "mean", mean);
        parts(a[4], s.lines, at::kFloat, l, s.one, where, "rstd", rstd);
        if (residual) parts(a[5], s.parts, l.type, l, s.one, where, "dh", res);
        const vrc_layer_norm_t d = norm_of(s, l, w, join, center, 0.0);
        const vrc_stream_t st = stream_of(a[9], l);
        size_t bytes = 0;
        done(vrc_layer_norm_grad_workspace(&d, n, &bytes), where);
        Ref dxs = outputs(a[8], s.outs, l.type, l, false, where, "recv", dx);
        const std::vector<Shape> row(1, Shape{s.width});
        Ref dws = allocate(row, w.scalar_type(), l, true, &dw);
        Ref dbs = bias ? allocate(row, w.scalar_type(), l, true, &db) : Ref(none());
        const at::Tensor space = workspace(bytes, l);
        call(where, [&] {
            return vrc_layer_norm_grad(&d, dy, h, center ? (const float* const*)mean : nullptr, (const float* const*)rstd, w.data_ptr(),
                                       residual ? res : nullptr, dx, dw, db, n, space.data_ptr(), bytes, st);
        });
        return PyTuple_Pack(3, dxs.o, dws.o, dbs.o);
    });
}

// ---------------------------------------------------------------------------
// Cross entropy
// ---------------------------------------------------------------------------
struct Entropy {
    vrc_cross_entropy_t d;
    size_t vocab[kMaxRanks];
    void* weight[kMaxRanks];
    int n;
    const at::Tensor* hidden;
    Shape lead;
    std::vector<Shape> shapes;  // of the weights
    const long long* target = nullptr;
};

Like entropy(PyObject* hidden, PyObject* weight, PyObject* target, PyObject* ignore, const char* where, Entropy* e)
{
    const Items items(weight, where, "weight");
    if (items.n < 1 || items.n > kMaxRanks) refuse(where, "weight must be one tensor per rank, 16 at most");
    const at::Tensor& h = tensor(hidden, where, "hidden");
    const Like l = like(h, where);
    if (!h.is_contiguous()) refuse(where, "tensors must be contiguous");
    if (h.dim() == 0 || h.sizes().back() == 0) refuse(where, "hidden must be [..., width]");
    const int64_t width = h.sizes().back();
    e->n = (int)items.n;
    e->hidden = &h;
    e->lead.assign(h.sizes().begin(), h.sizes().end() - 1);
    for (int r = 0; r < e->n; r++) {
        const at::Tensor& w = tensor(items.at[r], where, "every rank's weight");
        if (w.dim() != 2 || w.size(1) != width) refuse(where, "every rank's weight must be [rows of the vocabulary, hidden's width]");
        e->shapes.push_back({w.size(0), width});
        same(items.at[r], e->shapes.back(), l.type, l, where, "every rank's weight");
        e->vocab[r] = (size_t)w.size(0);
        e->weight[r] = w.data_ptr();
    }
    if (given(target)) {
        const at::Tensor& t = tensor(target, where, "target");
        if (t.scalar_type() != at::kLong || t.sizes() != at::IntArrayRef(e->lead))
            refuse(where, "target must be int64 of hidden's leading shape");
        if (t.device() != l.device || !t.is_contiguous()) refuse(where, "target must be contiguous on hidden's device");
        e->target = (const long long*)t.data_ptr();
    }
    const long long skip = PyLong_AsLongLong(ignore);
    if (skip == -1 && PyErr_Occurred()) {
        if (!PyErr_ExceptionMatches(PyExc_OverflowError)) throw Set{};
        PyErr_Clear();
        refuse(where, "ignore_index must be a signed 64-bit number");
    }
    e->d = {(size_t)product(e->lead), (size_t)width, e->vocab, (vrc_dtype_t)l.dtype, skip};
    return l;
}

// (hidden, weight, target, ignore_index, stream) -> (loss, lse)
PyObject* cross_entropy(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded([&]() -> PyObject* {
        const char* where = "vrc_cross_entropy";
        expect(count, 5);
        Entropy e;
        const Like l = entropy(a[0], a[1], a[2], a[3], where, &e);
        const vrc_stream_t st = stream_of(a[4], l);
        size_t bytes = 0;
        done(vrc_cross_entropy_workspace(&e.d, e.hidden->data_ptr(), e.weight, e.n, &bytes), where);
        const std::vector<Shape> lead(1, e.lead);
        void *loss = nullptr, *lse;
        Ref lses = allocate(lead, at::kFloat, l, true, &lse);
        Ref losses = e.target || given(a[2]) ? allocate(lead, at::kFloat, l, true, &loss) : Ref(none());
        const at::Tensor space = workspace(bytes, l);
        call(where, [&] {
            return vrc_cross_entropy(&e.d, e.hidden->data_ptr(), e.weight, e.target, (float*)loss, (float*)lse, e.n, space.data_ptr(),
                                     bytes, st);
        });
        return PyTuple_Pack(2, losses.o, lses.o);
    });
}

// (hidden, weight, target, lse, dloss, dlse, ignore_index, need_hidden, need_weight, dhidden, dweight, stream) -> (dhidden, dweight)
PyObject* cross_entropy_grad(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded([&]() -> PyObject* {
        const char* where = "vrc_cross_entropy_grad";
        expect(count, 12);
        if (!given(a[2])) refuse(where, "target is missing");
        Entropy e;
        const Like l = entropy(a[0], a[1], a[2], a[6], where, &e);
        const void* lse = same(a[3], e.lead, at::kFloat, l, where, "lse").data_ptr();
        const void* dloss = same(a[4], e.lead, at::kFloat, l, where, "dloss").data_ptr();
        const void* dlse = given(a[5]) ? same(a[5], e.lead, at::kFloat, l, where, "dlse").data_ptr() : nullptr;
        const bool need_hidden = truth(a[7]), need_weight = truth(a[8]);
        const vrc_stream_t st = stream_of(a[11], l);
        size_t bytes = 0;
        done(vrc_cross_entropy_grad_workspace(&e.d, e.hidden->data_ptr(), e.weight, need_hidden, e.n, &bytes), where);
        void *dh = nullptr, *dw[kMaxRanks];
        const std::vector<Shape> shape(1, Shape(e.hidden->sizes().begin(), e.hidden->sizes().end()));
        Ref dhs = need_hidden ? outputs(a[9], shape, l.type, l, true, where, "recv's dhidden", &dh) : Ref(none());
        Ref dws = need_weight ? outputs(a[10], e.shapes, l.type, l, false, where, "recv's dweight", dw) : Ref(none());
        const at::Tensor space = workspace(bytes, l);
        call(where, [&] {
            return vrc_cross_entropy_grad(&e.d, e.hidden->data_ptr(), e.weight, e.target, (const float*)lse, (const float*)dloss,
                                          (const float*)dlse, dh, need_weight ? dw : nullptr, e.n, space.data_ptr(), bytes, st);
        });
        return PyTuple_Pack(2, dhs.o, dws.o);
    });
}

// (current_stream, done, out_of_memory): model.py's callbacks and torch's exception.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded([&]() -> PyObject* {
        expect(count, 3);
        for (int i = 0; i < 3; i++) Py_INCREF(a[i]);
        Py_XSETREF(g_current_stream, a[0]);
        Py_XSETREF(g_done, a[1]);
        Py_XSETREF(g_out_of_memory, a[2]);
        return PyLong_FromLong(vrc_ops_version());
    });
}

PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, nullptr},
    {"layer_norm", (PyCFunction)(void (*)(void))layer_norm, METH_FASTCALL, nullptr},
    {"layer_norm_grad", (PyCFunction)(void (*)(void))layer_norm_grad, METH_FASTCALL, nullptr},
    {"cross_entropy", (PyCFunction)(void (*)(void))cross_entropy, METH_FASTCALL, nullptr},
    {"cross_entropy_grad", (PyCFunction)(void (*)(void))cross_entropy_grad, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_vrc_model", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__vrc_model(void) { return PyModule_Create(&module); }
