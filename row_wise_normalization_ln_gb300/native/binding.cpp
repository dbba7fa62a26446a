// Native half of the Python binding of the group norm, gradient, head norm and
// dropout calls: checks the tensors, allocates what the caller did not give,
// and passes pointers and the current stream to the C ABI (libnorm_group.h,
// libnorm_grad.h, libnorm_rope.h, libnorm_dropout.h). These calls are short and many (a step of a small network,
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

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <exception>
#include <limits>
#include <stdexcept>
#include <string>
#include <unordered_map>
#include <vector>

#include "libnorm_dropout.h"
#include "libnorm_grad.h"
#include "libnorm_group.h"
#include "libnorm_rope.h"

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

// ------------------------------------------------------------ head norms with rotation
// Heads [T, heads, D] or [B, S, heads, D] with unit stride of their values.
bool heads_of(const at::Tensor& t, norm_heads* h) {
    const int64_t n = t.dim();
    h->data = ptr(t);
    h->batch = n == 4 ? t.stride(0) : 0;
    h->token = t.stride(n - 3);
    h->head = t.stride(n - 2);
    return t.size(n - 1) == 1 || t.stride(n - 1) == 1 || t.numel() == 0;
}

// Whether a tensor of one position per token lists them in the tokens' order:
// flat, or, for [B, S, heads, D], as [B, S] (dimensions of one value aside).
// [S, B] has as many values, in another order.
bool in_token_order(const at::Tensor& p, const at::Tensor& q) {
    if (q.dim() == 3) return true;
    c10::SmallVector<int64_t, 4> have, want;
    for (int64_t n : p.sizes())
        if (n != 1) have.push_back(n);
    for (int64_t n : {q.size(0), q.size(1)})
        if (n != 1) want.push_back(n);
    return have.size() <= 1 || have == want;
}

struct HeadCall {
    at::Tensor x[2], dy[2], w[2], out[2], dw[2], cos, sin, positions;  // queries, keys
    norm_rope_side side[2] = {};
    norm_rope_angles angles = {};
    norm_dtype dtype;
    int64_t B = 1, S, D;
};

const char* const kHeadNames[2] = {"q", "k"};

void same_kind(const at::Tensor& t, const at::Tensor& x, const std::string& name) {
    if (t.device() != x.device() || t.scalar_type() != x.scalar_type())
        refuse(name + " must be on " + x.device().str() + " with dtype " + c10::toString(x.scalar_type()));
}

// Checks shared by forward and backward; inputs whose values lie apart are copied.
void read_heads(HeadCall* c, PyObject* const* x, PyObject* const* w, PyObject* cos, PyObject* sin, PyObject* positions,
                PyObject* interleaved, const char* what) {
    for (int i = 0; i < 2; ++i) {
        if (i == 1 && x[1] == Py_None) {
            if (w[1] != Py_None) refuse("wk is given without k");
            break;
        }
        c->x[i] = tensor(x[i], kHeadNames[i]);
        const at::Tensor& t = c->x[i];
        if (!t.is_cuda()) refuse(std::string(what) + " needs CUDA tensors");
        if (t.dim() != 3 && t.dim() != 4) refuse(std::string(kHeadNames[i]) + " must be [tokens, heads, D] or [B, S, heads, D]");
        if (i == 0) {
            c->dtype = dtype_of(t);
            c->D = t.size(-1);
            c->S = t.size(t.dim() - 3);
            c->B = t.dim() == 4 ? t.size(0) : 1;
        } else {
            same_kind(t, c->x[0], "k");
            if (t.dim() != c->x[0].dim() || t.size(-1) != c->D || t.size(t.dim() - 3) != c->S || (t.dim() == 4 && t.size(0) != c->B))
                refuse("k must have q's tokens and head width");
        }
        c->w[i] = param(w[i], t, c->D, i == 0 ? "wq" : "wk");
        c->side[i].heads = t.size(t.dim() - 2);
        c->side[i].w = ptr(c->w[i]);
        if (!heads_of(t, &c->side[i].x)) {
            c->x[i] = t.contiguous();
            heads_of(c->x[i], &c->side[i].x);
        }
    }
    const at::Tensor& q = c->x[0];
    c->cos = tensor(cos, "cos");
    c->sin = tensor(sin, "sin");
    for (const at::Tensor* t : {&c->cos, &c->sin}) {
        if (t->scalar_type() != at::kFloat || t->dim() != 2 || t->device() != q.device() || t->sizes() != c->cos.sizes())
            refuse("cos and sin must be fp32 tables [positions, R / 2] of one shape on " + q.device().str());
        if (2 * t->size(1) > c->D) refuse("cos and sin have " + std::to_string(t->size(1)) + " angles, a head of " + std::to_string(c->D) + " values has room for " + std::to_string(c->D / 2));
    }
    const auto rows = [](const at::Tensor& t) {  // the pitch of a table's rows; -1: not rows
        if (t.size(1) > 1 && t.stride(1) != 1) return int64_t(-1);
        if (t.size(0) <= 1) return std::max<int64_t>(t.size(1), 1);
        return t.stride(0) >= t.size(1) ? t.stride(0) : int64_t(-1);
    };
    if (rows(c->cos) < 0 || rows(c->cos) != rows(c->sin)) {
        c->cos = c->cos.contiguous();
        c->sin = c->sin.contiguous();
    }
    c->angles.cos = static_cast<const float*>(ptr(c->cos));
    c->angles.sin = static_cast<const float*>(ptr(c->sin));
    c->angles.table_pitch = rows(c->cos);
    c->angles.P = c->cos.size(0);
    c->angles.R = static_cast<int32_t>(2 * c->cos.size(1));
    c->angles.interleaved = interleaved == Py_True;
    if (c->angles.R > 0 && c->angles.P == 0 && q.numel() > 0) refuse("cos and sin have no positions");
    if (positions != Py_None) {
        c->positions = tensor(positions, "positions");
        const at::ScalarType st = c->positions.scalar_type();
        if ((st != at::kLong && st != at::kInt) || c->positions.device() != q.device() || c->positions.numel() != c->B * c->S || !in_token_order(c->positions, q))
            refuse("positions must be int64 or int32 with one value per token (" + std::to_string(c->B * c->S) + "), flat or [B, S], on " + q.device().str());
        if (!c->positions.is_contiguous()) c->positions = c->positions.contiguous();
        c->angles.positions = ptr(c->positions);
        c->angles.position_bytes = st == at::kLong ? 8 : 4;
    }
}

// Whether some address belongs to two values of t, heads of unit stride.
bool shares_memory(const at::Tensor& t) {
    if (t.numel() == 0) return false;
    struct Dim {
        int64_t size, stride;
    };
    c10::SmallVector<Dim, 4> d;
    for (int64_t i = 0; i + 1 < t.dim(); ++i)
        if (t.size(i) > 1) d.push_back({t.size(i), t.stride(i)});
    std::sort(d.begin(), d.end(), [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    int64_t span = t.size(-1);  // of the dimensions so far: nested ones share nothing
    bool nested = true;
    for (const Dim& k : d) {
        nested = nested && k.stride >= span;
        span += (k.size - 1) * k.stride;
    }
    if (nested) return false;
    // Two heads share memory if a sum of steps i_k stride_k, not all 0, is less
    // than a head: every choice of the shorter dimensions' steps (of one sign
    // for the first of them), and the nearest steps of the longest.
    std::sort(d.begin(), d.end(), [](const Dim& a, const Dim& b) { return a.size < b.size; });
    while (d.size() < 3) d.insert(d.begin(), {1, 0});
    const Dim a = d[0], b = d[1], c = d[2];
    if (c.stride == 0) return true;
    for (int64_t i = 0; i < a.size; ++i)
        for (int64_t j = i == 0 ? 0 : 1 - b.size; j < b.size; ++j) {
            const int64_t at = i * a.stride + j * b.stride, near = -at / c.stride;
            for (int64_t k = std::max(near - 1, 1 - c.size); k <= std::min(near + 1, c.size - 1); ++k)
                if ((i || j || k) && std::abs(at + k * c.stride) < t.size(-1)) return true;
        }
    return false;
}

void read_head_outputs(HeadCall* c, PyObject* const* out, const char* const* names) {
    for (int i = 0; i < 2; ++i) {
        const at::Tensor& x = c->x[i];
        if (!x.defined()) {
            if (out[i] != Py_None) refuse(std::string(names[i]) + " is given without k");
            continue;
        }
        if (out[i] == Py_None) {
            c->out[i] = fresh(x.sizes(), x.scalar_type(), x);
        } else {
            c->out[i] = tensor(out[i], names[i]);
            if (c->out[i].sizes() != x.sizes() || c->out[i].scalar_type() != x.scalar_type() || c->out[i].device() != x.device())
                refuse(std::string(names[i]) + " must have " + kHeadNames[i] + "'s shape, dtype and device");
        }
        if (!heads_of(c->out[i], &c->side[i].y) || (out[i] != Py_None && shares_memory(c->out[i]))) refuse(std::string(names[i]) + " must have heads of unit stride that do not share memory");
    }
}

PyObject* given_or(PyObject* given, const at::Tensor& t) {
    return !t.defined() ? Py_NewRef(Py_None) : given == Py_None ? THPVariable_Wrap(t) : Py_NewRef(given);
}

PyObject* rope_fwd_py(PyObject* const* a) {
    // q k wq wk cos sin positions eps interleaved q_out k_out plan
    HeadCall c;
    read_heads(&c, a, a + 2, a[4], a[5], a[6], a[8], "rms_fwd_rope");
    const float eps = static_cast<float>(real(a[7]));
    const c10::cuda::CUDAGuard guard(c.x[0].device());
    static const char* const names[2] = {"q_out", "k_out"};
    read_head_outputs(&c, a + 9, names);
    const norm_rope_plan* plan = a[11] == Py_None ? nullptr : static_cast<const norm_rope_plan*>(PyLong_AsVoidPtr(a[11]));
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.x[0].get_device()).stream();
    norm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = rms_fwd_rope_planned(&c.side[0], &c.side[1], &c.angles, c.B, c.S, c.D, eps, c.dtype, stream, plan);
    Py_END_ALLOW_THREADS
    if (st != NORM_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(2);
    if (!out) throw PythonError{};
    for (int i = 0; i < 2; ++i) PyTuple_SET_ITEM(out, i, given_or(a[9 + i], c.out[i]));
    return out;
}

PyObject* rope_bwd_py(PyObject* const* a) {
    // dq dk q k wq wk cos sin positions eps interleaved dq_out dk_out dwq dwk workspace plan
    HeadCall c;
    read_heads(&c, a + 2, a + 4, a[6], a[7], a[8], a[10], "rms_bwd_rope");
    const float eps = static_cast<float>(real(a[9]));
    const at::Tensor& q = c.x[0];
    const c10::cuda::CUDAGuard guard(q.device());
    for (int i = 0; i < 2; ++i) {
        if (!c.x[i].defined()) {
            if (a[i] != Py_None || a[14] != Py_None) refuse("dk or dwk is given without k");
            continue;
        }
        const std::string name = i == 0 ? "dq" : "dk";
        c.dy[i] = tensor(a[i], name.c_str());
        same_kind(c.dy[i], q, name);
        if (c.dy[i].sizes() != c.x[i].sizes()) refuse(name + " must have " + kHeadNames[i] + "'s shape");
        if (!heads_of(c.dy[i], &c.side[i].dy)) {
            c.dy[i] = c.dy[i].contiguous();
            heads_of(c.dy[i], &c.side[i].dy);
        }
        c.dw[i] = f32(a[13 + i], {c.D}, q, i == 0 ? "dwq" : "dwk");
        if (c.side[i].heads == 0) c.dw[i].zero_();
        c.side[i].dw = static_cast<float*>(ptr(c.dw[i]));
    }
    static const char* const names[2] = {"dq_out", "dk_out"};
    read_head_outputs(&c, a + 11, names);
    const norm_rope_plan* plan = a[16] == Py_None ? nullptr : static_cast<const norm_rope_plan*>(PyLong_AsVoidPtr(a[16]));
    size_t bytes = 0;
    if (a[15] == Py_None)
        rope_workspace_bytes(c.B * c.S, c.side[0].heads, c.side[1].heads, c.D, sm_count(q.get_device()), plan, &bytes);
    const at::Tensor ws = scratch(a[15], bytes, q);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(q.get_device()).stream();
    norm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = rms_bwd_rope_planned(&c.side[0], &c.side[1], &c.angles, ptr(ws), bytes_of(ws), c.B, c.S, c.D, eps, c.dtype, stream, plan);
    Py_END_ALLOW_THREADS
    if (st != NORM_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(4);
    if (!out) throw PythonError{};
    for (int i = 0; i < 2; ++i) {
        PyTuple_SET_ITEM(out, i, given_or(a[11 + i], c.out[i]));
        PyTuple_SET_ITEM(out, 2 + i, given_or(a[13 + i], c.dw[i]));
    }
    return out;
}

// ------------------------------------------------------------ dropout, add and norm
struct RowCall {
    at::Tensor x;  // the rows' type, device and shape
    norm_dtype dtype;
    int64_t M, N;
};

void read_shape(RowCall* c, const at::Tensor& x, const char* what) {
    if (!x.is_cuda()) refuse(std::string(what) + " needs CUDA tensors");
    c->x = x;
    c->dtype = dtype_of(x);
    if (x.dim() == 0) refuse("rows need at least one dimension");
    c->N = x.size(-1);
    if (c->N == 0) refuse("rows must have at least one element");
    c->M = x.numel() / c->N;
}

// A tensor of the rows' shape, type and device, made contiguous.
at::Tensor rows_like(PyObject* o, const RowCall& c, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (t.sizes() != c.x.sizes() || t.scalar_type() != c.x.scalar_type() || t.device() != c.x.device())
        refuse(std::string(name) + " must have the rows' shape, dtype and device");
    return t.is_contiguous() ? t : t.contiguous();
}

at::Tensor rows_out(PyObject* o, const RowCall& c, const char* name) {
    if (o == Py_None) return fresh(c.x.sizes(), c.x.scalar_type(), c.x);
    const at::Tensor& t = tensor(o, name);
    if (t.sizes() != c.x.sizes() || t.scalar_type() != c.x.scalar_type() || t.device() != c.x.device() || !t.is_contiguous())
        refuse(std::string(name) + " must be a contiguous tensor of the rows' shape, dtype and device");
    return t;
}

// Where the random numbers come from: (seed, offset), or a CUDA tensor of both.
const norm_rng* read_rng(PyObject* o, const RowCall& c, norm_rng* out) {
    if (o == Py_None) return nullptr;
    *out = norm_rng{0, 0, nullptr};
    if (THPVariable_Check(o)) {
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.scalar_type() != at::kLong || t.numel() != 2 || !t.is_contiguous() || t.device() != c.x.device())
            refuse("rng must be (seed, offset) or a contiguous int64 tensor of both on " + c.x.device().str());
        out->device = static_cast<const uint64_t*>(ptr(t));
        return out;
    }
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) throw BadType("rng must be (seed, offset) or an int64 tensor of both");
    uint64_t* to[2] = {&out->seed, &out->offset};
    for (int i = 0; i < 2; ++i) {
        *to[i] = PyLong_AsUnsignedLongLongMask(PyTuple_GET_ITEM(o, i));
        if (PyErr_Occurred()) throw PythonError{};
    }
    return out;
}

PyObject* drop_fwd_py(PyObject* const* a) {
    // ln x residual gamma beta p rng eps h_out out mean rstd stats plan
    const bool ln = a[0] == Py_True;
    RowCall c;
    read_shape(&c, tensor(a[1], "x"), ln ? "ln_fwd_dropout_add" : "rms_fwd_dropout_add");
    const at::Tensor gamma = param(a[3], c.x, c.N, ln ? "gamma" : "w"), beta = ln ? param(a[4], c.x, c.N, "beta") : at::Tensor();
    const double p = real(a[5]);
    const float eps = static_cast<float>(real(a[7]));
    norm_rng rng;
    const norm_rng* r = read_rng(a[6], c, &rng);
    const c10::cuda::CUDAGuard guard(c.x.device());
    const at::Tensor x = rows_like(a[1], c, "x"), res = rows_like(a[2], c, "residual");
    const at::Tensor h = rows_out(a[8], c, "h_out"), y = rows_out(a[9], c, "out");
    at::Tensor mean, rstd;
    if (ln && a[12] == Py_True) {
        mean = f32(a[10], {c.M}, c.x, "mean");
        rstd = f32(a[11], {c.M}, c.x, "rstd");
    }
    const norm_plan* plan = a[13] == Py_None ? nullptr : static_cast<const norm_plan*>(PyLong_AsVoidPtr(a[13]));
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.x.get_device()).stream();
    norm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = drop_fwd_planned(ln, ptr(x), ptr(res), ptr(gamma), ptr(beta), p, r, ptr(h), ptr(y), static_cast<float*>(ptr(mean)),
                          static_cast<float*>(ptr(rstd)), c.M, c.N, eps, c.dtype, stream, plan);
    Py_END_ALLOW_THREADS
    if (st != NORM_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(ln ? 4 : 2);
    if (!out) throw PythonError{};
    PyTuple_SET_ITEM(out, 0, given_or(a[8], h));
    PyTuple_SET_ITEM(out, 1, given_or(a[9], y));
    if (ln) {
        PyTuple_SET_ITEM(out, 2, given_or(a[10], mean));
        PyTuple_SET_ITEM(out, 3, given_or(a[11], rstd));
    }
    return out;
}

PyObject* drop_bwd_py(PyObject* const* a) {
    // ln dropout dy dh h gamma mean rstd p rng eps dx dresidual dgamma dbeta workspace plan
    const bool ln = a[0] == Py_True, dropout = a[1] == Py_True;
    RowCall c;
    const char* what = ln ? (dropout ? "ln_bwd_dropout_add" : "ln_bwd_add") : (dropout ? "rms_bwd_dropout_add" : "rms_bwd_add");
    read_shape(&c, tensor(a[4], "h"), what);
    const at::Tensor gamma = param(a[5], c.x, c.N, ln ? "gamma" : "w");
    const double p = real(a[8]);
    const float eps = static_cast<float>(real(a[10]));
    norm_rng rng;
    const norm_rng* r = read_rng(a[9], c, &rng);
    const c10::cuda::CUDAGuard guard(c.x.device());
    const at::Tensor dy = rows_like(a[2], c, "dy"), h = rows_like(a[4], c, "h");
    const at::Tensor dh = a[3] == Py_None ? at::Tensor() : rows_like(a[3], c, "dh");
    at::Tensor mean, rstd, dx;
    if (ln) {
        mean = given_f32(a[6], c.M, c.x, "mean");
        rstd = given_f32(a[7], c.M, c.x, "rstd");
    }
    if (dropout) dx = rows_out(a[11], c, "dx");
    const at::Tensor dres = rows_out(a[12], c, "dresidual");
    const at::Tensor dgamma = f32(a[13], {c.N}, c.x, ln ? "dgamma" : "dw");
    const at::Tensor dbeta = ln ? f32(a[14], {c.N}, c.x, "dbeta") : at::Tensor();
    const norm_plan* plan = a[16] == Py_None ? nullptr : static_cast<const norm_plan*>(PyLong_AsVoidPtr(a[16]));
    size_t bytes = 0;
    if (a[15] == Py_None) drop_workspace_bytes(c.M, c.N, c.dtype, ln, sm_count(c.x.get_device()), plan, &bytes);
    const at::Tensor ws = scratch(a[15], bytes, c.x);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c.x.get_device()).stream();
    norm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = drop_bwd_planned(ln, ptr(dy), ptr(dh), ptr(h), ptr(gamma), static_cast<float*>(ptr(mean)), static_cast<float*>(ptr(rstd)), p, r,
                          ptr(dx), ptr(dres), static_cast<float*>(ptr(dgamma)), static_cast<float*>(ptr(dbeta)), ptr(ws), bytes_of(ws),
                          c.M, c.N, eps, c.dtype, stream, plan);
    Py_END_ALLOW_THREADS
    if (st != NORM_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(2 + dropout + ln);
    if (!out) throw PythonError{};
    Py_ssize_t i = 0;
    if (dropout) PyTuple_SET_ITEM(out, i++, given_or(a[11], dx));
    PyTuple_SET_ITEM(out, i++, given_or(a[12], dres));
    PyTuple_SET_ITEM(out, i++, given_or(a[13], dgamma));
    if (ln) PyTuple_SET_ITEM(out, i++, given_or(a[14], dbeta));
    return out;
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
    {"rms_fwd_rope", fast(entry<rope_fwd_py, 12>), METH_FASTCALL, nullptr},
    {"rms_bwd_rope", fast(entry<rope_bwd_py, 17>), METH_FASTCALL, nullptr},
    {"drop_fwd", fast(entry<drop_fwd_py, 14>), METH_FASTCALL, nullptr},
    {"drop_bwd", fast(entry<drop_bwd_py, 17>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
