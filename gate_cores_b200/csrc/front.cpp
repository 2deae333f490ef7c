// Tensor front end of layer norm, rotary positions and the expert permutation:
// PyTorch CUDA tensors in, PyTorch CUDA tensors out, as cores.py documents
// them.  Marshalling only: checks, shapes, strides and outputs; every step of
// the computation is in the C entry points.  A call runs on its tensors' device
// and that device's current stream.
//
// In C++ because a call of few tokens takes the GPU less time than Python takes
// to prepare it.  On B200, us a pass with this in Python over ctypes and here:
// layer norm of 128 x 4096 9.3 and 4.5; rotary positions of 128 tokens 13.9 and
// 5.2; sort, dispatch and combine of 128 tokens 29.1 and 12.6 (about what the
// GPU takes); the gradients of 777 tokens' rows 19.6 and 8.4.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <limits>
#include <optional>
#include <string>

#include "muse_cores.h"

namespace {

using at::Tensor;

PyObject* g_fail = nullptr;  // _lib._fail(status, name), which raises

const Tensor& tensor(PyObject* o, const char* what) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a tensor");
    return THPVariable_Unpack(o);
}
const Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

void same_device(const Tensor& x, std::initializer_list<const Tensor*> ts) {
    TORCH_CHECK_VALUE(x.is_cuda(), "tensors must live on a CUDA device");
    for (const Tensor* t : ts) TORCH_CHECK_VALUE(!t || t->device() == x.device(), "tensors must live on one CUDA device");
}

// The device and the stream of a call.
struct On {
    c10::cuda::CUDAGuard guard;
    cudaStream_t stream;
    explicit On(const Tensor& x) : guard(x.device()), stream(c10::cuda::getCurrentCUDAStream(x.get_device()).stream()) {}
};

muse_dtype dtype_of(const Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return MUSE_DTYPE_BF16;
    TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, "unsupported dtype ", t.scalar_type(), "; use bfloat16 or float32");
    return MUSE_DTYPE_F32;
}

template <typename T> T* at_of(const Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

Tensor contiguous(const Tensor& t) { return t.is_contiguous() ? t : t.contiguous(); }

// Straight from PyTorch's allocator (through the dispatcher an output takes 0.1 to 0.2 us longer), unless something is
// on that sees new tensors there: deterministic algorithms, which fill them, or a dispatch mode.
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
    if (at::globalContext().deterministicAlgorithms() || c10::impl::TorchDispatchModeTLS::any_modes_set())
        return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
    return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// `out`, checked against `like`, or a new contiguous tensor of its shape and type.
Tensor output(const Tensor& like, const Tensor* out, const char* what) {
    if (!out) return empty(like.sizes(), like.scalar_type(), like);
    TORCH_CHECK_VALUE(out->sizes() == like.sizes() && out->scalar_type() == like.scalar_type(), what,
                      " must have the shape and dtype of the tensor it belongs to");
    return *out;
}

// An FP32 vector of `hidden` channels.
std::optional<Tensor> channels(const Tensor* p, int64_t hidden, const char* what) {
    if (!p) return std::nullopt;
    TORCH_CHECK_TYPE(p->scalar_type() == at::kFloat, what, " must be float32");
    TORCH_CHECK_VALUE(p->dim() == 1 && p->size(0) == hidden, what, " must be [", std::to_string(hidden), "]");
    return contiguous(*p);
}
template <typename T> T* at_of(const std::optional<Tensor>& t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

// A tensor of rows; one row has the stride of its width, none too.
struct Rows {
    int64_t rows, hidden, stride;
};
Rows row_view(const Tensor& t, const char* what) {
    TORCH_CHECK_VALUE(t.dim() >= 1 && t.size(-1) >= 1, what, " must have a last dimension of at least one element");
    const int64_t hidden = t.size(-1);
    if (t.is_contiguous()) return {t.numel() / hidden, hidden, hidden};
    TORCH_CHECK_VALUE(t.dim() == 2, what, " must be contiguous unless it has two dimensions");
    TORCH_CHECK_VALUE(t.stride(1) == 1 || hidden == 1, "the last dimension of ", what, " must be contiguous");
    return {t.size(0), hidden, t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), hidden)};
}
Rows matrix(const Tensor& t, const char* what) {
    TORCH_CHECK_VALUE(t.dim() == 2, what, " must be [rows, hidden]");
    return row_view(t, what);
}

// Bytes of a caller's workspace, which have to be its own and enough.
size_t workspace_bytes(const Tensor& ws, size_t need) {
    const size_t n = (size_t)ws.numel() * ws.element_size();
    TORCH_CHECK_VALUE(n >= need && ws.is_contiguous(), "workspace needs ", std::to_string(need), " contiguous bytes");
    return n;
}

// Runs an entry point without the interpreter's lock; a status other than OK raises.
template <typename F> void call(const char* name, F&& f) {
    muse_status status;
    Py_BEGIN_ALLOW_THREADS
    status = f();
    Py_END_ALLOW_THREADS
    if (status == MUSE_OK) return;
    PyObject* r = PyObject_CallFunction(g_fail, "is", (int)status, name);
    Py_XDECREF(r);
    throw python_error();
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
    TORCH_CHECK_TYPE(n == want, "takes ", std::to_string(want), " arguments (", std::to_string(n), " given)");
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap(const std::optional<Tensor>& t) { return t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None); }

// (x, gain, bias, gain_offset, eps, out) -> y
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 6);
    const Tensor& x = tensor(a[0], "x");
    const Tensor *gain = maybe(a[1], "gain"), *bias = maybe(a[2], "bias"), *out = maybe(a[5], "out");
    const float offset = (float)number(a[3]), eps = (float)number(a[4]);
    same_device(x, {gain, bias, out});
    const On on(x);
    const muse_dtype dt = dtype_of(x);
    const Rows xr = row_view(x, "x");
    const auto g = channels(gain, xr.hidden, "gain"), b = channels(bias, xr.hidden, "bias");
    const Tensor y = output(x, out, "out");
    const Rows yr = row_view(y, "out");
    const void* px = x.data_ptr();
    void* py = y.data_ptr();
    const float *pg = at_of<const float>(g), *pb = at_of<const float>(b);
    call("muse_layer_norm", [&] {
        return muse_layer_norm(px, py, dt, xr.rows, xr.hidden, xr.stride, yr.stride, pg, offset, pb, eps, on.stream);
    });
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

// (x, dy, gain, gain_offset, eps, dx, want_dgain, want_dbias, workspace) -> (dx, dgain, dbias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 9);
    const Tensor &x = tensor(a[0], "x"), &dy = tensor(a[1], "dy");
    const Tensor *gain = maybe(a[2], "gain"), *into = maybe(a[5], "dx"), *ws = maybe(a[8], "workspace");
    const float offset = (float)number(a[3]), eps = (float)number(a[4]);
    const bool want_dgain = truth(a[6]), want_dbias = truth(a[7]);
    same_device(x, {&dy, gain, into, ws});
    const On on(x);
    TORCH_CHECK_VALUE(dy.sizes() == x.sizes() && dy.scalar_type() == x.scalar_type(), "dy must match x");
    const muse_dtype dt = dtype_of(x);
    const Rows xr = row_view(x, "x");
    const int64_t dys = row_view(dy, "dy").stride;
    const auto g = channels(gain, xr.hidden, "gain");
    const Tensor dx = output(x, into, "dx");
    const int64_t dxs = row_view(dx, "dx").stride;
    std::optional<Tensor> dgain, dbias, own;
    if (want_dgain && g) dgain = empty({xr.hidden}, at::kFloat, x);
    if (want_dbias) dbias = empty({xr.hidden}, at::kFloat, x);
    size_t ws_bytes = 0;
    if (dgain || dbias) {
        const size_t need = muse_norm_backward_workspace_bytes(xr.rows, xr.hidden);
        if (ws) ws_bytes = workspace_bytes(*ws, need);
        else own = empty({(int64_t)(ws_bytes = std::max<size_t>(need, 16))}, at::kByte, x), ws = &*own;
    }
    const void *px = x.data_ptr(), *pdy = dy.data_ptr();
    void *pdx = dx.data_ptr(), *pws = ws_bytes ? ws->data_ptr() : nullptr;
    const float* pg = at_of<const float>(g);
    float *pdg = at_of<float>(dgain), *pdb = at_of<float>(dbias);
    call("muse_layer_norm_backward", [&] {
        return muse_layer_norm_backward(px, pdy, pdx, dt, xr.rows, xr.hidden, xr.stride, dys, dxs, pg, offset, eps, pdg,
                                        pdb, pws, ws_bytes, on.stream);
    });
    return Py_BuildValue("(NNN)", wrap(dx), wrap(dgain), wrap(dbias));
    END_HANDLE_TH_ERRORS
}

// Elements between tokens of [T, heads, d] or [B, S, heads, d]; strides of dimensions of one entry do not count.
int64_t head_stride(const Tensor& t, int64_t heads, int64_t d, int64_t tokens) {
    if (t.is_contiguous()) return heads * d;
    const auto st = t.strides(), sh = t.sizes();
    const size_t n = st.size();
    TORCH_CHECK_VALUE((d <= 1 || st[n - 1] == 1) && (heads <= 1 || st[n - 2] == d),
                      "each token's heads must be contiguous ([.., heads, head_dim])");
    if (tokens <= 1) return heads * d;
    if (n == 3 || sh[0] == 1) return st[n - 3];
    if (sh[1] == 1) return st[0];
    TORCH_CHECK_VALUE(st[0] == sh[1] * st[1], "BSHD tensors need a uniform token stride");
    return st[1];
}

int32_t as_int32(int64_t v) { return (int32_t)std::min<int64_t>(v, std::numeric_limits<int32_t>::max()); }

// (q, k, inv_freq, positions, cu_seqlens, pairing, attention_scale, q_out, k_out, backward) -> (q', k')
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 10);
    const Tensor &q = tensor(a[0], "q"), &freq = tensor(a[2], "inv_freq");
    const Tensor *k = maybe(a[1], "k"), *positions = maybe(a[3], "positions"), *cu = maybe(a[4], "cu_seqlens");
    const Tensor *q_out = maybe(a[7], "q's output"), *k_out = maybe(a[8], "k's output");
    const long pairing = PyLong_AsLong(a[5]);
    if (pairing == -1 && PyErr_Occurred()) throw python_error();
    const float scale = (float)number(a[6]);
    const bool backward = truth(a[9]);
    same_device(q, {k, &freq, positions, cu, q_out, k_out});
    const On on(q);
    const int64_t dims = q.dim();
    TORCH_CHECK_VALUE(dims == 3 || dims == 4, "q must be [B,S,Hq,D] or [T,Hq,D]");
    TORCH_CHECK_TYPE(freq.scalar_type() == at::kDouble && freq.dim() == 1, "inv_freq must be a float64 vector");
    const muse_dtype dt = dtype_of(q);
    const int64_t hq = q.size(-2), d = q.size(-1);
    muse_layout layout = MUSE_LAYOUT_BSHD;
    int64_t batch, seqlen, tokens;
    if (dims == 4) {
        TORCH_CHECK_VALUE(!cu, "cu_seqlens belongs to packed tensors [T,H,D]");
        batch = q.size(0), seqlen = q.size(1), tokens = batch * seqlen;
        if (seqlen == 0) batch = 0;
    } else {
        tokens = seqlen = q.size(0), batch = tokens ? 1 : 0;
    }
    Tensor cu_held, pos_held;
    const int32_t *pcu = nullptr, *ppos = nullptr;
    int64_t num_seqs = 0;
    if (cu) {
        TORCH_CHECK_VALUE(cu->scalar_type() == at::kInt && cu->dim() == 1, "cu_seqlens must be an int32 vector");
        layout = MUSE_LAYOUT_THD;
        cu_held = contiguous(*cu);
        pcu = at_of<const int32_t>(&cu_held);
        num_seqs = std::max<int64_t>(cu->numel() - 1, 0);
    }
    if (positions) {
        TORCH_CHECK_VALUE(positions->scalar_type() == at::kInt && positions->numel() == tokens,
                          "positions must be int32 with one entry per token");
        pos_held = contiguous(*positions);
        ppos = at_of<const int32_t>(&pos_held);
    }
    const Tensor f = contiguous(freq);
    const int64_t qs = head_stride(q, hq, d, tokens);
    int64_t hk = 0, ks = 0, kos = 0;
    if (k) {
        hk = k->dim() == dims ? k->size(-2) : 0;
        TORCH_CHECK_VALUE(k->dim() == dims && k->scalar_type() == q.scalar_type() && k->size(-1) == d &&
                              k->sizes().slice(0, dims - 2) == q.sizes().slice(0, dims - 2),
                          "k must match q's leading dims, head_dim and dtype");
        ks = head_stride(*k, hk, d, tokens);
    } else {
        TORCH_CHECK_VALUE(!k_out, "an output for k without k");
    }
    const Tensor qo = output(q, q_out, "q's output");
    const int64_t qos = head_stride(qo, hq, d, tokens);
    std::optional<Tensor> ko;
    if (k) {
        ko = output(*k, k_out, "k's output");
        kos = head_stride(*ko, hk, d, tokens);
    }
    const void *pq = q.data_ptr(), *pk = at_of<const void>(k);
    void *pqo = qo.data_ptr(), *pko = at_of<void>(ko);
    const double* pf = at_of<const double>(&f);
    const auto entry = backward ? muse_rope_backward : muse_rope;
    call(backward ? "muse_rope_backward" : "muse_rope", [&] {
        return entry(pq, pk, pqo, pko, dt, layout, batch, seqlen, pcu, as_int32(num_seqs), tokens, ppos, as_int32(hq),
                     as_int32(hk), as_int32(d), as_int32(2 * f.numel()), (muse_rope_pairing)pairing, qs, ks, qos, kos, pf,
                     scale, on.stream);
    });
    return Py_BuildValue("(NN)", wrap(qo), wrap(ko));
    END_HANDLE_TH_ERRORS
}

// (expert_ids, num_experts, workspace) -> (group_offsets, row_of_slot, slot_of_row)
PyObject* expert_sort(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 3);
    const Tensor& choices = tensor(a[0], "expert_ids");
    const int64_t experts = PyLong_AsLongLong(a[1]);
    if (experts == -1 && PyErr_Occurred()) throw python_error();
    const Tensor* ws = maybe(a[2], "workspace");
    same_device(choices, {ws});
    const On on(choices);
    TORCH_CHECK_VALUE(choices.dim() == 2 && choices.size(1) >= 1, "expert_ids must be [tokens, top_k]");
    const bool wide = choices.scalar_type() == at::kLong;
    TORCH_CHECK_TYPE(wide || choices.scalar_type() == at::kInt, "expert_ids must be int32 or int64");
    TORCH_CHECK_VALUE(experts >= 1, "num_experts must be positive");
    const int32_t E = as_int32(experts);
    const Tensor ids = contiguous(choices);
    const int64_t tokens = ids.size(0), top_k = ids.size(1), slots = tokens * top_k;
    // (more than the library takes: it refuses before any of them is written)
    const Tensor offsets = empty({std::min<int64_t>(experts, 1 << 20) + 1}, at::kInt, ids);
    const Tensor rows = empty({tokens, top_k}, at::kInt, ids), back = empty({slots}, at::kInt, ids);
    const size_t need = muse_expert_sort_workspace_bytes(slots, E);
    size_t ws_bytes = 0;
    std::optional<Tensor> own;
    if (ws) ws_bytes = workspace_bytes(*ws, need);
    else if (need) own = empty({(int64_t)(ws_bytes = need)}, at::kByte, ids), ws = &*own;
    const void* pi = ids.data_ptr();
    int32_t *po = at_of<int32_t>(&offsets), *pr = at_of<int32_t>(&rows), *pb = at_of<int32_t>(&back);
    void* pws = ws ? ws->data_ptr() : nullptr;
    call("muse_expert_sort", [&] {
        return muse_expert_sort(pi, wide ? MUSE_INDEX_I64 : MUSE_INDEX_I32, tokens, as_int32(top_k), E, po, pr, pb, pws,
                                ws_bytes, on.stream);
    });
    return Py_BuildValue("(NNN)", wrap(offsets), wrap(rows), wrap(back));
    END_HANDLE_TH_ERRORS
}

// row_of_slot, of `tokens` lines where that is given (not negative).
Tensor slots_of(const Tensor& t, int64_t tokens = -1) {
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.dim() == 2 && t.size(1) >= 1, "row_of_slot must be int32 [tokens, top_k]");
    TORCH_CHECK_VALUE(tokens < 0 || t.size(0) == tokens, "row_of_slot must have a line for each token");
    return contiguous(t);
}
std::optional<Tensor> weights_of(const Tensor* w, const Tensor& slots) {
    if (!w) return std::nullopt;
    TORCH_CHECK_TYPE(w->scalar_type() == at::kFloat, "weights must be float32");
    TORCH_CHECK_VALUE(w->sizes() == slots.sizes(), "weights must be shaped like row_of_slot");
    return contiguous(*w);
}

// (x, row_of_slot, out) -> rows
PyObject* expert_dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 3);
    const Tensor &x = tensor(a[0], "x"), &slots = tensor(a[1], "row_of_slot");
    const Tensor* into = maybe(a[2], "out");
    same_device(x, {&slots, into});
    const On on(x);
    const Rows xr = matrix(x, "x");
    const muse_dtype dt = dtype_of(x);
    const Tensor row = slots_of(slots, xr.rows);
    const Tensor out = into ? *into : empty({row.numel(), xr.hidden}, x.scalar_type(), x);
    const Rows orr = matrix(out, "out");
    TORCH_CHECK_VALUE(orr.hidden == xr.hidden && out.scalar_type() == x.scalar_type(), "out must have x's dtype and width");
    const void* px = x.data_ptr();
    void* po = out.data_ptr();
    const int32_t* pr = at_of<const int32_t>(&row);
    const int32_t top_k = as_int32(row.size(1));
    call("muse_expert_dispatch", [&] {
        return muse_expert_dispatch(px, po, dt, xr.rows, xr.hidden, top_k, orr.rows, xr.stride, orr.stride, pr, on.stream);
    });
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// (rows, row_of_slot, weights, out, dispatch's backward) -> y, or dx
PyObject* expert_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 5);
    const Tensor &rows = tensor(a[0], "the rows"), &slots = tensor(a[1], "row_of_slot");
    const Tensor *weights = maybe(a[2], "weights"), *into = maybe(a[3], "out");
    const bool backward = truth(a[4]);
    same_device(rows, {&slots, weights, into});
    const On on(rows);
    const Rows rr = matrix(rows, "the rows");
    const muse_dtype dt = dtype_of(rows);
    const Tensor row = slots_of(slots);
    const int64_t tokens = row.size(0);
    const auto w = weights_of(weights, row);
    TORCH_CHECK_VALUE(!into || (into->dim() == 2 && into->size(0) == tokens && into->size(1) == rr.hidden &&
                                into->scalar_type() == rows.scalar_type()),
                      "out must be [tokens, hidden] in the rows' dtype");
    const Tensor y = into ? *into : empty({tokens, rr.hidden}, rows.scalar_type(), rows);
    const int64_t ys = matrix(y, "out").stride;
    const void* pin = rows.data_ptr();
    void* py = y.data_ptr();
    const int32_t* pr = at_of<const int32_t>(&row);
    const float* pw = at_of<const float>(w);
    const int32_t top_k = as_int32(row.size(1));
    if (backward)
        call("muse_expert_dispatch_backward", [&] {
            return muse_expert_dispatch_backward(pin, py, dt, tokens, rr.hidden, top_k, rr.rows, rr.stride, ys, pr, on.stream);
        });
    else
        call("muse_expert_combine", [&] {
            return muse_expert_combine(pin, py, dt, tokens, rr.hidden, top_k, rr.rows, rr.stride, ys, pr, pw, on.stream);
        });
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

// (rows, dy, row_of_slot, weights, drows, want_dweights) -> (drows, dweights)
PyObject* expert_combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 6);
    const Tensor &rows = tensor(a[0], "the rows"), &dy = tensor(a[1], "dy"), &slots = tensor(a[2], "row_of_slot");
    const Tensor *weights = maybe(a[3], "weights"), *into = maybe(a[4], "drows");
    const bool want = truth(a[5]);
    same_device(dy, {&rows, &slots, weights, into});
    const On on(dy);
    const Rows yr = matrix(dy, "dy"), rr = matrix(rows, "the rows");
    TORCH_CHECK_VALUE(rr.hidden == yr.hidden && rows.scalar_type() == dy.scalar_type(), "rows and dy must share their dtype and width");
    const muse_dtype dt = dtype_of(dy);
    const Tensor row = slots_of(slots, yr.rows);
    const auto w = weights_of(weights, row);
    const Tensor drows = output(rows, into, "drows");
    const int64_t ds = matrix(drows, "drows").stride;
    std::optional<Tensor> dw;
    if (want) dw = empty(row.sizes(), at::kFloat, dy);
    const void *pin = rows.data_ptr(), *pdy = dy.data_ptr();
    void* pd = drows.data_ptr();
    const int32_t* pr = at_of<const int32_t>(&row);
    const float* pw = at_of<const float>(w);
    float* pdw = at_of<float>(dw);
    const int32_t top_k = as_int32(row.size(1));
    call("muse_expert_combine_backward", [&] {
        return muse_expert_combine_backward(pin, pdy, pd, dt, yr.rows, yr.hidden, top_k, rr.rows, rr.stride, yr.stride, ds,
                                            pr, pw, pdw, on.stream);
    });
    return Py_BuildValue("(NN)", wrap(drows), wrap(dw));
    END_HANDLE_TH_ERRORS
}

#define FRONT(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FRONT(layer_norm),      FRONT(layer_norm_backward), FRONT(rope),
                          FRONT(expert_sort),     FRONT(expert_dispatch),     FRONT(expert_combine),
                          FRONT(expert_combine_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_front", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__front() {
    PyObject* lib = PyImport_ImportModule("gate_cores_b200._lib");
    if (!lib) return nullptr;
    g_fail = PyObject_GetAttrString(lib, "_fail");
    Py_DECREF(lib);
    return g_fail ? PyModule_Create(&kModule) : nullptr;
}
