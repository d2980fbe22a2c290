// CPython binding of the rotary and paged calls of include/cca.h: argument checks and
// marshalling only, as api.py does for the others through ctypes.  A decoding step makes many
// small calls, and looking at a tensor costs about 0.1 us per attribute from Python, a call
// 20-60 us in all; here it is 2-4 us besides the launches.  The library's functions are not
// linked: api.py hands over their addresses with bind().
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <cstring>
#include <unordered_set>
#include <vector>

#include "../../include/cca.h"

namespace {

struct Library {
    decltype(&cca_rope) rope;
    decltype(&cca_rope_append) rope_append;
    decltype(&cca_tree_fwd) tree_fwd;
    decltype(&cca_tree_workspace_size) tree_workspace_size;
    decltype(&cca_pool_pages) pool_pages;
    decltype(&cca_pages_reserve) pages_reserve;
    decltype(&cca_pages_reserve_workspace_size) pages_reserve_workspace_size;
    decltype(&cca_pages_fork) pages_fork;
    decltype(&cca_pages_free) pages_free;
    decltype(&cca_pages_copy) pages_copy;
    decltype(&cca_pages_compact) pages_compact;
} lib;
PyObject *error_class = nullptr;  // api.CcaError(status, what)

// A check that failed has set a Python error and throws this; every entry point catches it.
struct Refused {};

template <typename... Args>
[[noreturn]] void refuse(const char *format, Args... args) {
    PyErr_Format(PyExc_ValueError, format, args...);
    throw Refused();
}

void set_error(int status, const char *what) {
    PyObject *e = PyObject_CallFunction(error_class, "is", status, what);
    if (e != nullptr) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
}

void check(int status, const char *what) {
    if (status == CCA_OK) return;
    set_error(status, what);
    throw Refused();
}

// The same where autograd's threads may be the callers: the error travels with the exception.
void check_anywhere(int status, const char *what) {
    if (status == CCA_OK) return;
    python_error e;
    const PyGILState_STATE gil = PyGILState_Ensure();
    set_error(status, what);
    e.persist();
    PyGILState_Release(gil);
    throw e;
}

bool none(PyObject *o) { return o == nullptr || o == Py_None; }

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (o == nullptr || !THPVariable_Check(o)) refuse("%s must be a CUDA tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    return t;
}

std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

// A tensor of the call's device, type and shape.
const at::Tensor &same(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int dev) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type) refuse("%s has dtype %s, expected %s", name, at::toString(t.scalar_type()), at::toString(type));
    if (t.sizes() != shape) refuse("%s has shape %s, expected %s", name, text(t.sizes()).c_str(), text(shape).c_str());
    if (t.get_device() != dev) refuse("%s is on cuda:%d, expected cuda:%d", name, static_cast<int>(t.get_device()), dev);
    return t;
}

// Pointer of such a tensor that is contiguous; null for None.
template <typename T = void>
T *ptr(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int dev) {
    if (none(o)) return nullptr;
    const at::Tensor &t = same(o, name, type, shape, dev);
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    return static_cast<T *>(t.data_ptr());
}
int32_t *words(PyObject *o, const char *name, at::IntArrayRef shape, int dev) {
    return ptr<int32_t>(o, name, at::kInt, shape, dev);
}

// A tensor that the call is given to write.  Autograd learns of it as of any write in place: what it
// has saved of the tensor is out of date.  Where the write would have to be differentiated it is refused.
void to_write(PyObject *o, const char *name) {
    if (none(o)) return;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.requires_grad() && c10::GradMode::is_enabled())
        refuse("%s requires a gradient: it cannot be written in place outside torch.no_grad()", name);
}
void wrote(PyObject *o) {
    if (none(o)) return;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

int64_t integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("%s must be a 64-bit integer", name);
    }
    return v;
}
int int32(PyObject *o, const char *name) {
    const int64_t v = integer(o, name);
    if (v < INT32_MIN || v > INT32_MAX) refuse("%s is out of range", name);
    return static_cast<int>(v);
}
int size32(int64_t v, const char *name) {
    if (v > INT32_MAX) refuse("%s is too large", name);
    return static_cast<int>(v);
}
bool flag(PyObject *o, const char *name) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        refuse("%s must be true or false", name);
    }
    return v == 1;
}
float real(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("%s must be a number", name);
    }
    return static_cast<float>(v);
}

int dtype_of(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kBFloat16) return CCA_BF16;
    if (t.scalar_type() == at::kFloat) return CCA_F32;
    refuse("unsupported dtype %s of %s", at::toString(t.scalar_type()), name);
}

// The tensor that says where a call runs, [.., .., .., ..] of bf16 or f32.
const at::Tensor &leader(PyObject *o, const char *name, int64_t dims = 4) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != dims) refuse("%s has shape %s", name, text(t.sizes()).c_str());
    return t;
}

// Makes the tensors' device the current one for the call; its current stream.
struct Place {
    c10::cuda::CUDAGuard guard;
    int dev;
    void *stream;
    explicit Place(const at::Tensor &t)
        : guard(t.device()), dev(t.get_device()), stream(c10::cuda::getCurrentCUDAStream(t.get_device()).stream()) {}
};

int64_t columns(PyObject *o, const char *name) {
    if (o == nullptr || !THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 2) refuse("%s must be a matrix", name);
    return THPVariable_Unpack(o).size(1);
}

// A pool [pages, Hkv, rows, d] ([layers, pages, ...] where allowed) and its table.
cca_pages_t pool(PyObject *K, PyObject *V, PyObject *table, int64_t B, int64_t heads, int64_t d, at::ScalarType type, int dev,
                 const char *what, bool layers) {
    const at::Tensor &k = tensor(K, what);
    const bool deep = layers && k.dim() == 5;
    if (k.dim() != 4 && !deep) refuse("%s must be [%spages, Hkv, rows, d]", what, layers ? "layers, " : "");
    if (k.size(-3) != heads || k.size(-1) != d)
        refuse("%s has shape %s, expected [pages, %lld, rows, %lld]", what, text(k.sizes()).c_str(), static_cast<long long>(heads),
               static_cast<long long>(d));
    cca_pages_t p = {};
    p.K = ptr(K, what, type, k.sizes(), dev);
    p.V = ptr(V, what, type, k.sizes(), dev);
    p.n_pages = size32(k.size(-4), what);
    p.rows = size32(k.size(-2), what);
    p.layers = deep ? size32(k.size(0), what) : 1;
    if (!none(table)) {
        p.cols = size32(columns(table, "table"), "table");
        p.table = words(table, "table", {B, p.cols}, dev);
    }
    return p;
}

cca_params_t params(int64_t B, int64_t Hq, int64_t Hkv, int64_t d, int dtype, int32_t *status) {
    cca_params_t p = {};
    p.B = size32(B, "batch");
    p.Hq = size32(Hq, "heads");
    p.Hkv = size32(Hkv, "heads");
    p.d = size32(d, "head dimension");
    p.g = p.w = 1;
    p.dtype = dtype;
    p.dev_status = status;
    return p;
}

// A caller's workspace, or one for this call alone (on its stream, so it may be handed back at once).
struct Workspace {
    at::Tensor own;
    void *p;
    uint64_t bytes;
    Workspace(PyObject *o, uint64_t need, const at::Tensor &like) {
        if (none(o)) {
            bytes = need < 16 ? 16 : need;
            own = at::empty({static_cast<int64_t>(bytes)}, like.options().dtype(at::kByte));
            p = own.data_ptr();
        } else {
            const at::Tensor &t = tensor(o, "workspace");
            bytes = t.nbytes();
            if (t.get_device() != like.get_device() || !t.is_contiguous() || bytes < need)
                refuse("workspace must be a buffer of at least %llu bytes on cuda:%d", static_cast<unsigned long long>(need),
                       static_cast<int>(like.get_device()));
            p = t.data_ptr();
        }
    }
};

// ---------------------------------------------------------------- rotary

cca_rope_tensor_t rows(const at::Tensor &x, const at::Tensor *y, const char *name) {
    if (x.stride(3) != 1 || (y != nullptr && y->stride(3) != 1)) refuse("%s must be contiguous in its last dimension", name);
    cca_rope_tensor_t r = {};
    r.x = x.data_ptr();
    r.y = y != nullptr ? y->data_ptr() : nullptr;
    r.H = size32(x.size(1), name);
    for (int i = 0; i < 3; ++i) {
        r.x_stride[i] = x.stride(i);
        r.y_stride[i] = y != nullptr ? y->stride(i) : 0;
    }
    return r;
}

void frequencies(PyObject *o, int64_t d, int dev, cca_rope_params_t &p) {
    if (none(o)) return;
    const at::Tensor &f = tensor(o, "inv_freq");
    if (f.dim() != 1 || 2 * f.numel() > d) refuse("inv_freq must be [rot/2] with rot <= %lld", static_cast<long long>(d));
    p.inv_freq = ptr<double>(o, "inv_freq", at::kDouble, f.sizes(), dev);
    p.rot = static_cast<int>(2 * f.numel());
}

int layout(PyObject *o) {
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "half") == 0) return 0;
        if (PyUnicode_CompareWithASCIIString(o, "interleaved") == 0) return 1;
    }
    refuse("layout must be 'half' or 'interleaved'");
}

// What a rotation needs besides the tensors it turns.
struct Turn {
    at::Tensor inv_freq, positions;  // positions: undefined without
    int64_t start = 0;
    int layout = 0;
    float factor = 1.f;
    bool inverse = false;
    // Q, K, inv_freq, positions, start, layout, factor
    Turn(PyObject *const *a, const at::Tensor &q, int dev) {
        cca_rope_params_t p = {};
        frequencies(a[2], q.size(3), dev, p);
        if (!none(a[2])) inv_freq = THPVariable_Unpack(a[2]);
        start = integer(a[4], "start");
        if (!none(a[3])) {
            if (start != 0) refuse("start and positions exclude each other");
            positions = tensor(a[3], "positions");
            if (positions.dim() == 1) words(a[3], "positions", {q.size(2)}, dev);
            else words(a[3], "positions", {q.size(0), q.size(2)}, dev);
        }
        layout = ::layout(a[5]);
        factor = real(a[6], "factor");
    }
    Turn() = default;
    cca_rope_params_t params(const at::Tensor &q, int dtype) const {
        cca_rope_params_t p = {};
        p.B = static_cast<int32_t>(q.size(0));
        p.N = static_cast<int32_t>(q.size(2));
        p.d = static_cast<int32_t>(q.size(3));
        p.dtype = dtype;
        if (inv_freq.defined()) {
            p.inv_freq = static_cast<const double *>(inv_freq.data_ptr());
            p.rot = static_cast<int32_t>(2 * inv_freq.numel());
        }
        if (positions.defined()) {
            p.positions = static_cast<const int32_t *>(positions.data_ptr());
            p.pos_stride = positions.dim() == 1 ? 0 : p.N;
        }
        p.start = start;
        p.layout = layout;
        p.factor = factor;
        p.inverse = inverse;
        return p;
    }
};

// Queries and (where there are any) keys that belong together.
int check_pair(PyObject *const *a, const at::Tensor &q, int dev) {
    size32(q.size(0), "batch"), size32(q.size(2), "rows"), size32(q.size(3), "head dimension");
    if (!none(a[1])) same(a[1], "K", q.scalar_type(), {q.size(0), leader(a[1], "K").size(1), q.size(2), q.size(3)}, dev);
    return dtype_of(q, "Q");
}

// Q, K, inv_freq, positions, start, layout, factor, inverse, out Q, out K
PyObject *rope(PyObject *const *a) {
    const at::Tensor &q = leader(a[0], "Q");
    const Place at(q);
    const int dtype = check_pair(a, q, at.dev);
    Turn turn(a, q, at.dev);
    turn.inverse = flag(a[7], "inverse");
    const bool two = !none(a[1]);
    if ((!two && !none(a[9])) || (two && none(a[8]) != none(a[9]))) refuse("out must hold one tensor for each input");
    at::Tensor outs[2];
    cca_rope_tensor_t t[2];
    for (int i = 0; i < (two ? 2 : 1); ++i) {
        const at::Tensor &x = THPVariable_Unpack(a[i]);
        outs[i] = none(a[8 + i]) ? at::empty(x.sizes(), q.options()) : same(a[8 + i], "out", q.scalar_type(), x.sizes(), at.dev);
        t[i] = rows(x, &outs[i], i == 0 ? "Q" : "K");
        to_write(a[8 + i], "out");
    }
    const cca_rope_params_t p = turn.params(q, dtype);
    check(lib.rope(t, two ? 2 : 1, &p, at.stream), "cca_rope");
    wrote(a[8]), wrote(a[9]);
    PyObject *first = THPVariable_Wrap(outs[0]);
    if (two) return Py_BuildValue("(NN)", first, THPVariable_Wrap(outs[1]));
    return Py_BuildValue("(NO)", first, Py_None);
}

// A leaf's gradient is accumulated on the stream where an earlier graph that still lives first used
// the leaf.  Inside a capture the default stream cannot be waited for, and autograd ends the process
// when it tries, so a captured backward pass that would come there is refused before it does.
void refuse_uncapturable_leaves() {
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return;
    const auto here = torch::autograd::get_current_node();
    std::vector<torch::autograd::Node *> todo{here.get()};
    std::unordered_set<torch::autograd::Node *> seen;
    while (!todo.empty()) {
        torch::autograd::Node *node = todo.back();
        todo.pop_back();
        if (node == nullptr || !seen.insert(node).second) continue;
        if (dynamic_cast<torch::autograd::AccumulateGrad *>(node) != nullptr) {
            const auto stream = node->stream();
            TORCH_CHECK(!stream || !stream->device().is_cuda() || c10::cuda::CUDAStream(*stream).stream() != nullptr,
                        "a backward pass is being captured, but a graph made outside the capture still holds one of its "
                        "leaves on the default stream: let go of that graph's outputs first");
        }
        for (size_t i = 0; i < node->num_outputs(); ++i)  // where this pass goes on
            if (node->task_should_compute_output(i)) todo.push_back(node->next_edge(i).function.get());
    }
}

// Autograd of the rotation.  It is linear: the gradient is the rotation back, by the same kernel,
// and can be differentiated again.  The backward pass runs on the engine's thread, without Python.
struct RopeFunction : torch::autograd::Function<RopeFunction> {
    using List = torch::autograd::variable_list;

    // x itself where its rows can be read in place, a contiguous copy otherwise
    static at::Tensor ready(const at::Tensor &x) {
        const int64_t es = x.element_size();
        const bool in_place = x.stride(3) == 1 && (x.stride(0) | x.stride(1) | x.stride(2)) * es % 16 == 0 &&
                              reinterpret_cast<uintptr_t>(x.data_ptr()) % 16 == 0;
        return in_place ? x : x.contiguous();
    }

    static List turned(const Turn &turn, const List &in) {
        const c10::cuda::CUDAGuard guard(in[0].device());
        List out;
        cca_rope_tensor_t t[2];
        List held;
        for (size_t i = 0; i < in.size(); ++i) {
            held.push_back(ready(in[i]));
            out.push_back(at::empty(in[i].sizes(), in[i].options()));
            cca_rope_tensor_t &r = t[i];
            r = {};
            r.x = held[i].data_ptr();
            r.y = out[i].data_ptr();
            r.H = static_cast<int32_t>(in[i].size(1));
            for (int k = 0; k < 3; ++k) {
                r.x_stride[k] = held[i].stride(k);
                r.y_stride[k] = out[i].stride(k);
            }
        }
        const cca_rope_params_t p = turn.params(in[0], in[0].scalar_type() == at::kBFloat16 ? CCA_BF16 : CCA_F32);
        const int status = lib.rope(t, static_cast<int>(in.size()), &p, c10::cuda::getCurrentCUDAStream(in[0].get_device()).stream());
        check_anywhere(status, "cca_rope");
        return out;
    }

    static List forward(torch::autograd::AutogradContext *ctx, const at::Tensor &q, const c10::optional<at::Tensor> &k,
                        const at::Tensor &inv_freq, const c10::optional<at::Tensor> &positions, int64_t start, int64_t layout,
                        double factor, bool inverse) {
        ctx->save_for_backward({inv_freq, positions.has_value() ? *positions : at::Tensor()});
        ctx->saved_data["start"] = start;
        ctx->saved_data["layout"] = layout;
        ctx->saved_data["factor"] = factor;
        ctx->saved_data["inverse"] = inverse;
        ctx->saved_data["two"] = k.has_value();
        Turn turn;
        turn.inv_freq = inv_freq;
        if (positions.has_value()) turn.positions = *positions;
        turn.start = start;
        turn.layout = static_cast<int>(layout);
        turn.factor = static_cast<float>(factor);
        turn.inverse = inverse;
        return turned(turn, k.has_value() ? List{q, *k} : List{q});
    }

    static List backward(torch::autograd::AutogradContext *ctx, const List &grads) {
        refuse_uncapturable_leaves();
        const List saved = ctx->get_saved_variables();
        const bool two = ctx->saved_data["two"].toBool();
        Turn turn;
        turn.inv_freq = saved[0];
        turn.positions = saved[1];
        turn.start = ctx->saved_data["start"].toInt();
        turn.layout = static_cast<int>(ctx->saved_data["layout"].toInt());
        turn.factor = static_cast<float>(ctx->saved_data["factor"].toDouble());
        turn.inverse = !ctx->saved_data["inverse"].toBool();
        // the gradients that this pass asks for: of Q, K or both
        const auto here = torch::autograd::get_current_node();
        List in;
        for (int k = 0; k < (two ? 2 : 1); ++k)
            if (here == nullptr || here->task_should_compute_output(k)) in.push_back(grads[k]);
        List g;
        if (in.empty()) {
        } else if (c10::GradMode::is_enabled()) {
            g = apply(in[0], in.size() == 2 ? c10::optional<at::Tensor>(in[1]) : c10::nullopt, turn.inv_freq,
                      turn.positions.defined() ? c10::optional<at::Tensor>(turn.positions) : c10::nullopt, turn.start,
                      static_cast<int64_t>(turn.layout), static_cast<double>(turn.factor), turn.inverse);
        } else {
            g = turned(turn, in);
        }
        List out(8);
        for (size_t k = 0, n = 0; n < g.size(); ++k)
            if (here == nullptr || here->task_should_compute_output(k)) out[k] = g[n++];
        return out;
    }
};

// Q, K, inv_freq, positions, start, layout, factor
PyObject *rope_grad(PyObject *const *a) {
    const at::Tensor &q = leader(a[0], "Q");
    const Place at(q);
    check_pair(a, q, at.dev);
    const Turn turn(a, q, at.dev);
    if (!turn.inv_freq.defined()) refuse("inv_freq must be a CUDA tensor");
    const bool two = !none(a[1]);
    const auto out = RopeFunction::apply(
        q, two ? c10::optional<at::Tensor>(THPVariable_Unpack(a[1])) : c10::nullopt, turn.inv_freq,
        turn.positions.defined() ? c10::optional<at::Tensor>(turn.positions) : c10::nullopt, turn.start,
        static_cast<int64_t>(turn.layout), static_cast<double>(turn.factor), false);
    PyObject *first = THPVariable_Wrap(out[0]);
    if (two) return Py_BuildValue("(NN)", first, THPVariable_Wrap(out[1]));
    return Py_BuildValue("(NO)", first, Py_None);
}

PyObject *check_leaves(PyObject *const *) {
    refuse_uncapturable_leaves();
    Py_RETURN_NONE;
}

// Q, K, V, Kp, Vp, table, lens, inv_freq, parents, counts, layout, factor, out, dev_status
PyObject *rope_append(PyObject *const *a) {
    const at::Tensor &k = leader(a[1], "K");
    const Place at(k);
    const int64_t B = k.size(0), H = k.size(1), T = k.size(2), d = k.size(3);
    cca_rope_params_t p = {};
    p.B = size32(B, "batch");
    p.N = size32(T, "tokens");
    p.d = size32(d, "head dimension");
    p.dtype = dtype_of(k, "K");
    frequencies(a[7], d, at.dev, p);
    p.layout = layout(a[10]);
    p.factor = real(a[11], "factor");
    const at::Tensor &v = same(a[2], "V", k.scalar_type(), k.sizes(), at.dev);
    const cca_rope_tensor_t kt = rows(k, nullptr, "K"), vt = rows(v, nullptr, "V");
    const cca_pages_t raw = pool(a[3], a[4], a[5], B, H, d, k.scalar_type(), at.dev, "raw pool", false);
    int32_t *lens = words(a[6], "lens", {B}, at.dev), *parents = words(a[8], "parents", {B, T}, at.dev),
            *counts = words(a[9], "counts", {B}, at.dev), *status = words(a[13], "dev_status", {1}, at.dev);
    at::Tensor out;
    cca_rope_tensor_t qt = {};
    const bool has_q = !none(a[0]);
    if (has_q) {
        const at::Tensor &q = leader(a[0], "Q");
        same(a[0], "Q", k.scalar_type(), {B, q.size(1), T, d}, at.dev);
        out = none(a[12]) ? at::empty(q.sizes(), k.options()) : same(a[12], "out", k.scalar_type(), q.sizes(), at.dev);
        qt = rows(q, &out, "Q");
    } else if (!none(a[12])) {
        refuse("out without Q");
    }
    to_write(a[3], "raw pool"), to_write(a[4], "raw pool"), to_write(a[12], "out");
    check(lib.rope_append(has_q ? &qt : nullptr, &kt, &vt, &raw, lens, parents, counts, status, &p, at.stream), "cca_rope_append");
    wrote(a[3]), wrote(a[4]), wrote(a[12]);
    if (has_q) return THPVariable_Wrap(out);
    Py_RETURN_NONE;
}

// ---------------------------------------------------------------- paged attention and pooling

// Q, Kp, Vp, table, Kcp, Vcp, core_table, lens, g, w, parents, O, LSE, workspace, scale, dev_status, window_mode
PyObject *tree_fwd(PyObject *const *a) {
    const at::Tensor &q = leader(a[0], "Q");
    const Place at(q);
    const int64_t B = q.size(0), H = q.size(1), T = q.size(2), d = q.size(3);
    const int64_t Hkv = leader(a[1], "raw pool").size(1);
    cca_params_t p = params(B, H, Hkv, d, dtype_of(q, "Q"), words(a[15], "dev_status", {1}, at.dev));
    p.g = int32(a[8], "g");
    p.w = int32(a[9], "w");
    p.scale = real(a[14], "scale");
    p.window_mode = int32(a[16], "window_mode");
    const void *qp = ptr(a[0], "Q", q.scalar_type(), q.sizes(), at.dev);
    const cca_pages_t raw = pool(a[1], a[2], a[3], B, Hkv, d, q.scalar_type(), at.dev, "raw pool", false);
    const cca_pages_t core = pool(a[4], a[5], a[6], B, Hkv, d, q.scalar_type(), at.dev, "core pool", false);
    int32_t *lens = words(a[7], "lens", {B}, at.dev), *parents = words(a[10], "parents", {B, T}, at.dev);
    at::Tensor O, LSE;
    if (none(a[11])) O = at::empty(q.sizes(), q.options());
    else ptr(a[11], "O", q.scalar_type(), q.sizes(), at.dev), O = THPVariable_Unpack(a[11]);
    if (none(a[12])) LSE = at::empty({B, H, T}, q.options().dtype(at::kFloat));
    else ptr(a[12], "LSE", at::kFloat, {B, H, T}, at.dev), LSE = THPVariable_Unpack(a[12]);
    to_write(a[11], "O"), to_write(a[12], "LSE");
    const int nodes = size32(T, "nodes");
    const Workspace ws(a[13], lib.tree_workspace_size(&p, nodes), q);
    check(lib.tree_fwd(qp, &raw, &core, lens, parents, nodes, O.data_ptr(), static_cast<float *>(LSE.data_ptr()), &p, ws.p, ws.bytes,
                       at.stream),
          "cca_tree_fwd");
    wrote(a[11]), wrote(a[12]);
    PyObject *first = THPVariable_Wrap(O);
    return Py_BuildValue("(NN)", first, THPVariable_Wrap(LSE));
}

// Q, Kp, Vp, table, Kcp, Vcp, core_table, lens, accepted, g, path, scale, dev_status, pool_mode
PyObject *pool_pages(PyObject *const *a) {
    const at::Tensor &q = leader(a[0], "Q");
    const Place at(q);
    const int64_t B = q.size(0), H = q.size(1), T = q.size(2), d = q.size(3);
    const int64_t Hkv = leader(a[1], "raw pool").size(1);
    cca_params_t p = params(B, H, Hkv, d, dtype_of(q, "Q"), words(a[12], "dev_status", {1}, at.dev));
    p.g = int32(a[9], "g");
    p.scale = real(a[11], "scale");
    p.pool_mode = int32(a[13], "pool_mode");
    const void *qp = ptr(a[0], "Q", q.scalar_type(), q.sizes(), at.dev);
    const cca_pages_t raw = pool(a[1], a[2], a[3], B, Hkv, d, q.scalar_type(), at.dev, "raw pool", false);
    const cca_pages_t core = pool(a[4], a[5], a[6], B, Hkv, d, q.scalar_type(), at.dev, "core pool", false);
    const int64_t A = none(a[10]) ? T : columns(a[10], "path");
    to_write(a[4], "core pool"), to_write(a[5], "core pool");
    check(lib.pool_pages(qp, &raw, &core, words(a[7], "lens", {B}, at.dev), words(a[8], "accepted", {B}, at.dev),
                         words(a[10], "path", {B, A}, at.dev), size32(A, "path"), size32(T, "tokens"), &p, at.stream),
          "cca_pool_pages");
    wrote(a[4]), wrote(a[5]);
    Py_RETURN_NONE;
}

// ---------------------------------------------------------------- the pages' book

struct Book {
    const at::Tensor &refs;
    Place at;
    int n, B, cols;
    int32_t *r, *t;
    Book(PyObject *refs_, PyObject *table)
        : refs(leader(refs_, "refs", 1)), at(refs), n(size32(refs.size(0), "refs")), cols(size32(columns(table, "table"), "table")) {
        B = size32(THPVariable_Unpack(table).size(0), "table");
        r = words(refs_, "refs", {n}, at.dev);
        t = words(table, "table", {B, cols}, at.dev);
    }
};

// refs, table, lens, extra, rows, pairs, workspace, dev_status
PyObject *pages_reserve(PyObject *const *a) {
    const Book k(a[0], a[1]);
    const int dev = k.at.dev;
    at::Tensor pairs;
    if (none(a[5])) pairs = at::empty({k.B, 2}, k.refs.options());
    else words(a[5], "pairs", {k.B, 2}, dev), pairs = THPVariable_Unpack(a[5]);
    const Workspace ws(a[6], lib.pages_reserve_workspace_size(k.B, k.cols), k.refs);
    check(lib.pages_reserve(k.r, k.n, k.t, k.B, k.cols, int32(a[4], "rows"), words(a[2], "lens", {k.B}, dev),
                            words(a[3], "extra", {k.B}, dev), static_cast<int32_t *>(pairs.data_ptr()), ws.p, ws.bytes,
                            words(a[7], "dev_status", {1}, dev), k.at.stream),
          "cca_pages_reserve");
    wrote(a[0]), wrote(a[1]), wrote(a[5]);
    return THPVariable_Wrap(pairs);
}

// refs, table, src, dst, lens, rows, dev_status
PyObject *pages_fork(PyObject *const *a) {
    const Book k(a[0], a[1]);
    const int dev = k.at.dev;
    const int64_t n = tensor(a[2], "src").numel();
    check(lib.pages_fork(k.r, k.n, k.t, k.B, k.cols, int32(a[5], "rows"), words(a[2], "src", {n}, dev), words(a[3], "dst", {n}, dev),
                         size32(n, "src"), words(a[4], "lens", {k.B}, dev), words(a[6], "dev_status", {1}, dev), k.at.stream),
          "cca_pages_fork");
    wrote(a[0]), wrote(a[1]);
    Py_RETURN_NONE;
}

// refs, table, first, last, dev_status
PyObject *pages_free(PyObject *const *a) {
    const Book k(a[0], a[1]);
    const int dev = k.at.dev;
    check(lib.pages_free(k.r, k.n, k.t, k.B, k.cols, words(a[2], "first", {k.B}, dev), words(a[3], "last", {k.B}, dev),
                         words(a[4], "dev_status", {1}, dev), k.at.stream),
          "cca_pages_free");
    wrote(a[0]), wrote(a[1]);
    Py_RETURN_NONE;
}

const at::Tensor &pool_leader(PyObject *o) {
    const at::Tensor &k = tensor(o, "pool");
    if (k.dim() != 4 && k.dim() != 5) refuse("pool must be [layers, pages, Hkv, rows, d] or [pages, Hkv, rows, d]");
    return k;
}

// Kp, Vp, pairs, dev_status
PyObject *pages_copy(PyObject *const *a) {
    const at::Tensor &k = pool_leader(a[0]);
    const Place at(k);
    const cca_params_t p = params(1, k.size(-3), k.size(-3), k.size(-1), dtype_of(k, "pool"), words(a[3], "dev_status", {1}, at.dev));
    const cca_pages_t pages = pool(a[0], a[1], nullptr, 1, k.size(-3), k.size(-1), k.scalar_type(), at.dev, "pool", true);
    if (columns(a[2], "pairs") != 2) refuse("pairs must be [n, 2]");
    const int64_t n = THPVariable_Unpack(a[2]).size(0);
    to_write(a[0], "pool"), to_write(a[1], "pool");
    check(lib.pages_copy(&pages, words(a[2], "pairs", {n, 2}, at.dev), size32(n, "pairs"), &p, at.stream), "cca_pages_copy");
    wrote(a[0]), wrote(a[1]);
    Py_RETURN_NONE;
}

// Kp, Vp, table, lens, path, accepted, dev_status
PyObject *pages_compact(PyObject *const *a) {
    const at::Tensor &k = pool_leader(a[0]);
    const Place at(k);
    const int64_t A = columns(a[4], "path"), B = THPVariable_Unpack(a[4]).size(0);
    const cca_params_t p = params(B, k.size(-3), k.size(-3), k.size(-1), dtype_of(k, "pool"), words(a[6], "dev_status", {1}, at.dev));
    const cca_pages_t pages = pool(a[0], a[1], a[2], B, k.size(-3), k.size(-1), k.scalar_type(), at.dev, "pool", true);
    to_write(a[0], "pool"), to_write(a[1], "pool");
    check(lib.pages_compact(&pages, words(a[3], "lens", {B}, at.dev), words(a[4], "path", {B, A}, at.dev), size32(A, "path"),
                            words(a[5], "accepted", {B}, at.dev), &p, at.stream),
          "cca_pages_compact");
    wrote(a[0]), wrote(a[1]);
    Py_RETURN_NONE;
}

// ---------------------------------------------------------------- module

template <PyObject *(*call)(PyObject *const *), Py_ssize_t count>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != count) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, count);
        return nullptr;
    }
    try {
        return call(args);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// bind(error class, {name: address})
PyObject *bind(PyObject *, PyObject *args) {
    PyObject *cls, *table;
    if (!PyArg_ParseTuple(args, "OO!", &cls, &PyDict_Type, &table)) return nullptr;
    Library l = {};
    const struct {
        const char *name;
        void *to;
    } all[] = {{"cca_rope", &l.rope}, {"cca_rope_append", &l.rope_append}, {"cca_tree_fwd", &l.tree_fwd},
               {"cca_tree_workspace_size", &l.tree_workspace_size}, {"cca_pool_pages", &l.pool_pages},
               {"cca_pages_reserve", &l.pages_reserve}, {"cca_pages_reserve_workspace_size", &l.pages_reserve_workspace_size},
               {"cca_pages_fork", &l.pages_fork}, {"cca_pages_free", &l.pages_free}, {"cca_pages_copy", &l.pages_copy},
               {"cca_pages_compact", &l.pages_compact}};
    for (const auto &f : all) {
        PyObject *address = PyDict_GetItemString(table, f.name);
        void *p = address == nullptr ? nullptr : PyLong_AsVoidPtr(address);
        if (p == nullptr) {
            PyErr_Format(PyExc_ValueError, "no address of %s", f.name);
            return nullptr;
        }
        std::memcpy(f.to, &p, sizeof p);
    }
    lib = l;
    Py_INCREF(cls);
    Py_XSETREF(error_class, cls);
    Py_RETURN_NONE;
}

#define CCA_ENTRY(name, count) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<name, count>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CCA_ENTRY(rope, 10),
                         CCA_ENTRY(rope_grad, 7),
                         CCA_ENTRY(check_leaves, 0),
                         CCA_ENTRY(rope_append, 14),
                         CCA_ENTRY(tree_fwd, 17),
                         CCA_ENTRY(pool_pages, 14),
                         CCA_ENTRY(pages_reserve, 8),
                         CCA_ENTRY(pages_fork, 7),
                         CCA_ENTRY(pages_free, 5),
                         CCA_ENTRY(pages_copy, 4),
                         CCA_ENTRY(pages_compact, 7),
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
