// Native half of the Python binding of the group norm and gradient calls:
// checks the tensors, allocates what the caller did not give, and passes
// pointers and the current stream to the C ABI (libnorm_group.h,
// libnorm_grad.h). These calls are short and many (a step of a small network,
// lists of hundreds of gradients); marshalling them through ctypes took three
// to five times as long as their kernels.
//
// Everything runs on the current stream of the tensors' device. Outputs and
// workspaces come from torch's caching allocator, which hands a block out
// again on the same stream only, so a workspace may be released as soon as
// the call has queued its kernels.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/SmallVector.h>

#include <cstdint>
#include <exception>
#include <limits>
#include <stdexcept>
#include <string>
#include <unordered_map>
#include <vector>

#include "libnorm_grad.h"
#include "libnorm_group.h"

namespace {

struct BadType : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PythonError {};  // an error is set already

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw BadType(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

int64_t whole(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}

double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return v;
}

norm_dtype dtype_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return NORM_F32;
        case at::kBFloat16: return NORM_BF16;
        case at::kHalf: return NORM_F16;
        default: throw BadType("libnorm supports float32, bfloat16 and float16, got " + std::string(c10::toString(t.scalar_type())));
    }
}

void* ptr(const at::Tensor& t) { return t.defined() && t.numel() > 0 ? t.mutable_data_ptr() : nullptr; }

// New tensors come straight from the caching allocator: gn_fwd with its three
// new outputs takes 5.6 us of the host, 8.0 through the dispatcher.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like) {
    return at::Tensor(at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt));
}
at::Tensor new_f32(at::IntArrayRef shape, const at::Tensor& like) { return fresh(shape, at::kFloat, like); }

// The caller's fp32 tensor of n values, checked; `name` for the message.
at::Tensor given_f32(PyObject* o, int64_t n, const at::Tensor& x, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kFloat || t.numel() != n || !t.is_contiguous() || t.device() != x.device())
        refuse(std::string(name) + " must be a contiguous fp32 tensor of " + std::to_string(n) + " elements on " + x.device().str());
    return t;
}
at::Tensor f32(PyObject* o, at::IntArrayRef shape, const at::Tensor& x, const char* name) {
    return o == Py_None ? new_f32(shape, x) : given_f32(o, c10::multiply_integers(shape), x, name);
}

at::Tensor param(PyObject* o, const at::Tensor& x, int64_t C, const char* name) {
    const at::Tensor& p = tensor(o, name);
    if (p.device() != x.device() || p.scalar_type() != x.scalar_type())
        refuse(std::string(name) + " must be on " + x.device().str() + " with dtype " + c10::toString(x.scalar_type()));
    if (p.numel() != C) refuse(std::string(name) + " must have " + std::to_string(C) + " elements, got " + std::to_string(p.numel()));
    return p.is_contiguous() ? p : p.contiguous();
}

at::Tensor scratch(PyObject* o, size_t bytes, const at::Tensor& x) {
    if (o == Py_None)
        return bytes ? fresh({static_cast<int64_t>(bytes)}, at::kByte, x) : at::Tensor();
    const at::Tensor& t = tensor(o, "workspace");
    if (t.device() != x.device() || !t.is_contiguous()) refuse("workspace must be a contiguous tensor on " + x.device().str());
    return t;
}
size_t bytes_of(const at::Tensor& t) { return t.defined() ? static_cast<size_t>(t.nbytes()) : 0; }

// ------------------------------------------------------------ group norm
// A [B, ..., C] tensor as positions: S of them per sample, `row` elements
// apart, samples `batch` apart.
struct Rows {
    int64_t S = 1, batch = 0, row = 0;
};
bool rows_of(const at::Tensor& t, Rows* out) {
    const int64_t n = t.dim(), B = t.size(0), C = t.size(-1);
    Rows r;
    r.row = C;
    bool any = false;
    for (int64_t d = n - 2; d >= 1; --d) {
        const int64_t size = t.size(d);
        if (size == 1) continue;
        if (!any) {
            r.row = t.stride(d);
            any = true;
        } else if (t.stride(d) != r.row * r.S) {
            return t.numel() == 0 ? (*out = Rows{0, 0, C}, true) : false;
        }
        r.S *= size;
    }
    if (t.numel() == 0) {
        *out = Rows{B == 0 ? r.S : 0, 0, C};
        return true;
    }
    const int64_t span = (r.S - 1) * r.row + C;
    r.batch = B > 1 ? t.stride(0) : span;
    if ((C > 1 && t.stride(-1) != 1) || r.row < C || r.batch < span) return false;
    *out = r;
    return true;
}

struct Call {
    at::Tensor x, gamma, beta;
    norm_dtype dtype;
    norm_act act;
    int64_t B, C, G;
    Rows rows;
};

// Checks shared by forward and backward; x is copied where its strides allow
// no common pitches.
void read_call(Call* c, PyObject* x, PyObject* gamma, PyObject* beta, PyObject* groups, PyObject* act, const char* what) {
    c->x = tensor(x, "x");
    if (!c->x.is_cuda()) refuse(std::string(what) + " needs a CUDA tensor");
    c->dtype = dtype_of(c->x);
    if (c->x.dim() < 2) refuse("x must be [B, ..., C]: samples first, channels last");
    c->B = c->x.size(0);
    c->C = c->x.size(-1);
    c->G = whole(groups);
    if (c->G < 1 || c->C < 1 || c->C % c->G != 0)
        refuse(std::to_string(c->C) + " channels do not form " + std::to_string(c->G) + " groups");
    c->act = static_cast<norm_act>(whole(act));
    c->gamma = param(gamma, c->x, c->C, "gamma");
    c->beta = param(beta, c->x, c->C, "beta");
}

void read_rows(at::Tensor* t, Rows* r) {
    if (rows_of(*t, r)) return;
    *t = t->contiguous();
    rows_of(*t, r);
}

at::Tensor output(PyObject* o, const at::Tensor& x, Rows* r, const char* name) {
    at::Tensor y;
    if (o == Py_None) {
        y = fresh(x.sizes(), x.scalar_type(), x);
    } else {
        y = tensor(o, name);
        if (y.sizes() != x.sizes() || y.scalar_type() != x.scalar_type() || y.device() != x.device())
            refuse(std::string(name) + " must have x's shape, dtype and device");
    }
    if (!rows_of(y, r))
        refuse(std::string(name) + " must have evenly strided positions and samples with unit channel stride");
    return y;
}

struct Key {
    int64_t B, S, C, G;
    int kind;
    bool operator==(const Key& o) const { return B == o.B && S == o.S && C == o.C && G == o.G && kind == o.kind; }
};
struct KeyHash {
    size_t operator()(const Key& k) const {
        uint64_t h = 1469598103934665603ull;
        for (uint64_t v : {uint64_t(k.B), uint64_t(k.S), uint64_t(k.C), uint64_t(k.G), uint64_t(k.kind)}) h = (h ^ v) * 1099511628211ull;
        return static_cast<size_t>(h ^ (h >> 29));
    }
};

int sm_count(int device) {
    static int cache[64] = {};
    if (device >= 0 && device < 64 && cache[device] > 0) return cache[device];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n <= 0)
        throw std::runtime_error("the device's SM count cannot be read");
    if (device >= 0 && device < 64) cache[device] = n;
    return n;
}

// The workspace size of a shape, kept (sizes only; the interpreter's lock
// guards the table). Shapes the library refuses get 0: the call then says why.
size_t gn_bytes(const Call& c, bool backward, const gn_plan* plan) {
    size_t n = 0;
    if (plan) {
        const norm_status st = gn_workspace_bytes(c.B, c.rows.S, c.C, c.G, c.dtype, backward, 0, plan, &n);
        return st == NORM_OK ? n : 0;
    }
    static std::unordered_map<Key, size_t, KeyHash> table;
    const Key key{c.B, c.rows.S, c.C, c.G, (c.x.get_device() * 4 + c.dtype) * 2 + backward};
    const auto it = table.find(key);
    if (it != table.end()) return it->second;
    if (gn_workspace_bytes(c.B, c.rows.S, c.C, c.G, c.dtype, backward, sm_count(c.x.get_device()), nullptr, &n) != NORM_OK) return 0;
    if (table.size() > 4096) table.clear();
    table.emplace(key, n);
    return n;
}

PyObject* gn_fwd_py(PyObject* const* a) {
    // x gamma beta groups eps act out mean rstd stats workspace plan
    Call c;
    read_call(&c, a[0], a[1], a[2], a[3], a[5], "gn_fwd");
    const float eps = static_cast<float>(real(a[4]));
    const c10::cuda::CUDAGuard guard(c.x.device());
    Rows yr;
    const at::Tensor y = output(a[6], c.x, &yr, "out");
    read_rows(&c.x, &c.rows);
    at::Tensor mean, rstd;
    if (a[9] == Py_True) {
        mean = f32(a[7], {c.B, c.G}, c.x, "mean");
        rstd = f32(a[8], {c.B, c.G}, c.x, "rstd");
        if (c.rows.S == 0) {  // no call writes the statistics of no values: NaN, as the formula gives them
            if (a[7] == Py_None) mean.fill_(std::numeric_limits<float>::quiet_NaN());
            if (a[8] == Py_None) rstd.fill_(std::numeric_limits<float>::quiet_NaN());
        }
    }
    const gn_plan* plan = a[11] == Py_None ? nullptr : static_cast<const gn_plan*>(PyLong_AsVoidPtr(a[11]));
    const at::Tensor ws = scratch(a[10], a[10] == Py_None ? gn_bytes(c, false, plan) : 0, c.x);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.x.get_device()).stream();
    norm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = gn_fwd_planned(ptr(c.x), c.rows.batch, c.rows.row, ptr(c.gamma), ptr(c.beta), ptr(y), yr.batch, yr.row,
                        static_cast<float*>(ptr(mean)), static_cast<float*>(ptr(rstd)), ptr(ws), bytes_of(ws), c.B,
                        c.rows.S, c.C, c.G, eps, c.act, c.dtype, stream, plan);
    Py_END_ALLOW_THREADS
    if (st != NORM_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(3);
    if (!out) throw PythonError{};
    PyTuple_SET_ITEM(out, 0, a[6] == Py_None ? THPVariable_Wrap(y) : Py_NewRef(a[6]));
    PyTuple_SET_ITEM(out, 1, !mean.defined() ? Py_NewRef(Py_None) : a[7] == Py_None ? THPVariable_Wrap(mean) : Py_NewRef(a[7]));
    PyTuple_SET_ITEM(out, 2, !rstd.defined() ? Py_NewRef(Py_None) : a[8] == Py_None ? THPVariable_Wrap(rstd) : Py_NewRef(a[8]));
    return out;
}

PyObject* gn_bwd_py(PyObject* const* a) {
    // dy x gamma beta mean rstd groups act dx dgamma dbeta workspace plan
    Call c;
    read_call(&c, a[1], a[2], a[3], a[6], a[7], "gn_bwd");
    at::Tensor dy = tensor(a[0], "dy");
    if (dy.sizes() != c.x.sizes() || dy.scalar_type() != c.x.scalar_type() || dy.device() != c.x.device())
        refuse("dy must have x's shape, dtype and device");
    const at::Tensor mean = given_f32(a[4], c.B * c.G, c.x, "mean"), rstd = given_f32(a[5], c.B * c.G, c.x, "rstd");
    const c10::cuda::CUDAGuard guard(c.x.device());
    Rows dxr, dyr;
    const at::Tensor dx = output(a[8], c.x, &dxr, "dx");
    read_rows(&c.x, &c.rows);
    read_rows(&dy, &dyr);
    const at::Tensor dgamma = f32(a[9], {c.C}, c.x, "dgamma"), dbeta = f32(a[10], {c.C}, c.x, "dbeta");
    const gn_plan* plan = a[12] == Py_None ? nullptr : static_cast<const gn_plan*>(PyLong_AsVoidPtr(a[12]));
    const at::Tensor ws = scratch(a[11], a[11] == Py_None ? gn_bytes(c, true, plan) : 0, c.x);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.x.get_device()).stream();
    norm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = gn_bwd_planned(ptr(dy), dyr.batch, dyr.row, ptr(c.x), c.rows.batch, c.rows.row, ptr(c.gamma), ptr(c.beta),
                        static_cast<float*>(ptr(mean)), static_cast<float*>(ptr(rstd)), ptr(dx), dxr.batch, dxr.row,
                        static_cast<float*>(ptr(dgamma)), static_cast<float*>(ptr(dbeta)), ptr(ws), bytes_of(ws), c.B,
                        c.rows.S, c.C, c.G, c.act, c.dtype, stream, plan);
    Py_END_ALLOW_THREADS
    if (st != NORM_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(3);
    if (!out) throw PythonError{};
    PyTuple_SET_ITEM(out, 0, a[8] == Py_None ? THPVariable_Wrap(dx) : Py_NewRef(a[8]));
    PyTuple_SET_ITEM(out, 1, a[9] == Py_None ? THPVariable_Wrap(dgamma) : Py_NewRef(a[9]));
    PyTuple_SET_ITEM(out, 2, a[10] == Py_None ? THPVariable_Wrap(dbeta) : Py_NewRef(a[10]));
    return out;
}

// ------------------------------------------------------------ gradients
struct Items {
    PyObject* seq;
    Items(PyObject* o, const char* name) : seq(PySequence_Fast(o, (std::string(name) + " must be a sequence of tensors").c_str())) {
        if (!seq) throw PythonError{};
    }
    ~Items() { Py_DECREF(seq); }
    Items(const Items&) = delete;
    Items& operator=(const Items&) = delete;
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
    PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

PyObject* grad_py(PyObject* const* a) {
    // grads out max_norm norm workspace; max_norm None: the norm alone
    const bool clip = a[2] != Py_None;
    const char* what = clip ? "grad_clip" : "grad_norm";
    const Items grads(a[0], "grads");
    const Py_ssize_t n = grads.size();
    if (n == 0) refuse(std::string(what) + " needs at least one tensor");
    const at::Tensor first = tensor(grads[0], "a gradient");
    if (!first.is_cuda()) refuse(std::string(what) + " needs CUDA tensors");
    std::vector<norm_tensor> table(static_cast<size_t>(n));
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor& t = tensor(grads[i], "a gradient");
        if (t.device() != first.device()) refuse("every gradient must be on " + first.device().str());
        norm_tensor& e = table[static_cast<size_t>(i)];
        e.dtype = dtype_of(t);
        if (!t.is_contiguous() && !t.is_non_overlapping_and_dense())
            refuse("gradient " + std::to_string(i) + " must be dense (no gaps or overlaps between its values)");
        e.numel = t.numel();
        e.data = e.out = ptr(t);
        e.reserved = 0;
    }
    if (a[1] != Py_None && a[1] != a[0]) {
        const Items outs(a[1], "out");
        if (outs.size() != n)
            refuse("out must hold one tensor per gradient (" + std::to_string(n) + "), got " + std::to_string(outs.size()));
        for (Py_ssize_t i = 0; i < n; ++i) {
            const at::Tensor &t = THPVariable_Unpack(grads[i]), &o = tensor(outs[i], "an out");
            if (o.sizes() != t.sizes() || o.strides() != t.strides() || o.scalar_type() != t.scalar_type() || o.device() != t.device())
                refuse("out " + std::to_string(i) + " must have its gradient's shape, strides, dtype and device");
            table[static_cast<size_t>(i)].out = ptr(o);
        }
    }
    const float max_norm = clip ? static_cast<float>(real(a[2])) : 0.f;
    const c10::cuda::CUDAGuard guard(first.device());
    const at::Tensor norm = f32(a[3], {}, first, "norm");
    size_t bytes = 0;
    if (a[4] == Py_None) grad_workspace_bytes(table.data(), n, sm_count(first.get_device()), &bytes);
    const at::Tensor ws = scratch(a[4], bytes, first);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(first.get_device()).stream();
    norm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = clip ? grad_clip(table.data(), n, max_norm, static_cast<float*>(ptr(norm)), ptr(ws), bytes_of(ws), stream)
              : grad_norm(table.data(), n, static_cast<float*>(ptr(norm)), ptr(ws), bytes_of(ws), stream);
    Py_END_ALLOW_THREADS
    if (st != NORM_OK) return PyLong_FromLong(st);
    return a[3] == Py_None ? THPVariable_Wrap(norm) : Py_NewRef(a[3]);
}

// No C++ exception leaves a call: each becomes the Python error it stands for.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        if (n != N) throw BadType("wrong number of arguments");
        return F(args);
    } catch (const PythonError&) {
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const BadType& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (...) {  // torch's own, with the types its calls raise (torch.OutOfMemoryError), and any other
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"gn_fwd", fast(entry<gn_fwd_py, 12>), METH_FASTCALL, nullptr},
    {"gn_bwd", fast(entry<gn_bwd_py, 13>), METH_FASTCALL, nullptr},
    {"grad", fast(entry<grad_py, 5>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
