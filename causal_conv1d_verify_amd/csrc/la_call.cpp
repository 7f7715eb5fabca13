// The short way from torch tensors to liblinattn.so: one C function per group of entry points
// that reads the tensors' sizes and strides, fills the shape and calls the C ABI on torch's
// current stream.  It takes the calls that are plainly in order and answers None to every other
// (a check that fails, another device or stream, no tokens): those go through the binding in
// linear_attention.py, which checks again and says what is wrong.  A single-token call is a few
// microseconds on the GPU, less than the same marshalling takes in Python (15 us).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <exception>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "linear_attention.h"

namespace {

using at::Tensor;

// None: no tensor.  Anything else that is not a tensor: `ok` becomes false.
const Tensor *tensor(PyObject *o, bool &ok) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
        ok = false;
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}

int dtype_code(const Tensor &t) {
    return t.scalar_type() == at::kFloat ? CV_F32 : t.scalar_type() == at::kBFloat16 ? CV_BF16 : -1;
}

bool rows_in_order(const Tensor &t) { return t.size(-1) == 1 || t.stride(-1) == 1; }
int64_t stride(const Tensor &t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }

bool int32_vec(const Tensor *t, int64_t n) {
    return !t || (t->scalar_type() == at::kInt && t->dim() == 1 && t->size(0) == n && (n <= 1 || t->stride(0) == 1));
}

bool weights(const Tensor *t, int64_t dim) {
    return !t || (t->dim() == 1 && t->size(0) == dim && (dim == 1 || t->stride(0) == 1));
}

// All on one GPU, the current one.
bool one_gpu(std::initializer_list<const Tensor *> ts, c10::Device *dev) {
    bool first = true;
    for (const Tensor *t : ts) {
        if (!t) continue;
        if (first) *dev = t->device(), first = false;
        else if (t->device() != *dev) return false;
    }
    return !first && dev->is_cuda() && dev->index() == c10::hip::current_device();
}

void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

bool number(PyObject *o, double *x) {
    if (PyFloat_CheckExact(o)) *x = PyFloat_AS_DOUBLE(o);
    else if (PyLong_CheckExact(o)) *x = PyLong_AsDouble(o);
    else return false;
    return !PyErr_Occurred();
}

enum { PREFILL, UPDATE, VERIFY, COMMIT };

// attn(kind, q, k, v, g, state, out, cu_seqlens, max_len, scale, slot_idx, has_initial_state,
//      num_tokens, workspace) -> the C ABI's return code, or None: not taken
PyObject *attn(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    if (n_args != 14) Py_RETURN_NONE;
    bool ok = true;
    const long kind = PyLong_AsLong(args[0]);
    const Tensor *q = tensor(args[1], ok), *k = tensor(args[2], ok), *v = tensor(args[3], ok), *g = tensor(args[4], ok),
                 *state = tensor(args[5], ok), *out = tensor(args[6], ok), *cu = tensor(args[7], ok),
                 *slot = tensor(args[10], ok), *init = tensor(args[11], ok), *num = tensor(args[12], ok),
                 *workspace = tensor(args[13], ok);
    const bool packed = kind == PREFILL, both = kind != COMMIT;
    if (!ok || !k || !v || !state || (both && (!q || !out)) || packed != (cu != nullptr)) Py_RETURN_NONE;
    c10::Device dev(c10::kCPU);
    if (!one_gpu({state, q, k, v, g, out, cu, slot, init, num, workspace}, &dev)) Py_RETURN_NONE;
    const int64_t lead = packed ? 1 : 2;
    if (k->dim() != lead + 2 || v->dim() != lead + 2 || state->dim() != 4) Py_RETURN_NONE;
    for (int64_t d = 0; d < lead; ++d)
        if (k->size(d) != v->size(d) || v->size(d) == 0) Py_RETURN_NONE;
    if (both && (q->sizes() != k->sizes() || out->sizes() != v->sizes())) Py_RETURN_NONE;
    for (const Tensor *t : {q, k, v, out})
        if (t && (t->scalar_type() != v->scalar_type() || !rows_in_order(*t))) Py_RETURN_NONE;
    la_shape_t s{};
    s.q_heads = (int32_t)k->size(lead);
    s.dk = (int32_t)k->size(lead + 1);
    s.v_heads = (int32_t)v->size(lead);
    s.dv = (int32_t)v->size(lead + 1);
    int64_t below = 1;
    for (int64_t d = 3; d > 0; below *= state->size(d), --d)
        if (state->size(d) != (d == 3 ? s.dv : d == 2 ? s.dk : s.v_heads) || (state->size(d) > 1 && state->stride(d) != below))
            Py_RETURN_NONE;
    if (g) {
        if (g->scalar_type() != at::kFloat || g->dim() < 1 || g->size(-1) != s.v_heads || !rows_in_order(*g)) Py_RETURN_NONE;
        if (g->dim() > 1) {
            if (g->dim() != lead + 1) Py_RETURN_NONE;
            for (int64_t d = 0; d < lead; ++d)
                if (g->size(d) != v->size(d)) Py_RETURN_NONE;
            s.g_tok_stride = stride(*g, lead - 1);
            s.g_seq_stride = packed ? 0 : stride(*g, 0);
        }
    }
    if (packed) {
        if (workspace && !workspace->is_contiguous()) Py_RETURN_NONE;
        if (cu->dim() != 1 || cu->size(0) < 1 || !PyLong_CheckExact(args[8])) Py_RETURN_NONE;
        const int64_t rows = cu->size(0) - 1;
        const long long longest = PyLong_AsLongLong(args[8]);
        if (PyErr_Occurred()) PyErr_Clear(), ok = false;
        if (!ok || longest > INT32_MAX || rows > INT32_MAX || !int32_vec(cu, rows + 1) || !int32_vec(init, rows)) Py_RETURN_NONE;
        s.n_seq = (int32_t)rows;
        s.T = longest < 1 ? 1 : (int32_t)longest;
        s.tokens = v->size(0);
    } else {
        if (v->size(0) > INT32_MAX || v->size(1) > INT32_MAX || !int32_vec(num, v->size(0))) Py_RETURN_NONE;
        s.n_seq = (int32_t)v->size(0);
        s.T = (int32_t)v->size(1);
    }
    if (!int32_vec(slot, s.n_seq) || state->size(0) > INT32_MAX) Py_RETURN_NONE;
    double scale = 0.0;
    if (args[9] == Py_None) scale = std::pow((double)s.dk, -0.5);
    else if (!number(args[9], &scale)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    s.scale = (float)scale;
    s.x_dtype = dtype_code(*v);
    s.state_dtype = dtype_code(*state);
    if (s.x_dtype < 0 || s.state_dtype < 0) Py_RETURN_NONE;
    s.n_slots = (int32_t)state->size(0);
    const int64_t tok = lead - 1, head = lead;
    if (q) {
        s.q_seq_stride = packed ? 0 : stride(*q, 0);
        s.q_tok_stride = stride(*q, tok);
        s.q_head_stride = stride(*q, head);
    }
    s.k_seq_stride = packed ? 0 : stride(*k, 0);
    s.k_tok_stride = stride(*k, tok);
    s.k_head_stride = stride(*k, head);
    s.v_seq_stride = packed ? 0 : stride(*v, 0);
    s.v_tok_stride = stride(*v, tok);
    s.v_head_stride = stride(*v, head);
    if (out) {
        s.out_seq_stride = packed ? 0 : stride(*out, 0);
        s.out_tok_stride = stride(*out, tok);
        s.out_head_stride = stride(*out, head);
    }
    s.state_slot_stride = stride(*state, 0);
    hipStream_t stream = c10::hip::getCurrentHIPStream(dev.index()).stream();
    const float *gp = static_cast<const float *>(ptr(g));
    const int32_t *slots = static_cast<const int32_t *>(ptr(slot));
    int rc;
    if (kind == PREFILL) {
        const int64_t need = linattn_prefill_workspace(&s);
        if (need < 0) return PyLong_FromLongLong(need);
        Tensor made;
        if (need > 0 && !workspace) {
            made = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(dev));
            workspace = &made;
        }
        rc = linattn_prefill(&s, ptr(q), ptr(k), ptr(v), gp, ptr(state), slots, static_cast<const int32_t *>(ptr(cu)),
                             static_cast<const int32_t *>(ptr(init)), ptr(out), ptr(workspace),
                             workspace ? workspace->numel() * workspace->element_size() : 0, stream);
    } else if (kind == COMMIT) {
        rc = linattn_commit(&s, ptr(k), ptr(v), gp, ptr(state), slots, static_cast<const int32_t *>(ptr(num)), stream);
    } else {
        rc = (kind == UPDATE ? linattn_update(&s, ptr(q), ptr(k), ptr(v), gp, ptr(state), slots, ptr(out), stream)
                             : linattn_verify(&s, ptr(q), ptr(k), ptr(v), gp, ptr(state), slots, ptr(out), stream));
    }
    return PyLong_FromLong(rc);
}

// gated(y, gate, weight, out, eps, activation, gate_first): likewise
PyObject *gated(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    if (n_args != 7) Py_RETURN_NONE;
    bool ok = true;
    const Tensor *y = tensor(args[0], ok), *gate = tensor(args[1], ok), *w = tensor(args[2], ok), *out = tensor(args[3], ok);
    if (!ok || !y || !w || !out || (y->dim() != 2 && y->dim() != 3) || y->numel() == 0) Py_RETURN_NONE;
    c10::Device dev(c10::kCPU);
    if (!one_gpu({y, gate, w, out}, &dev) || out->sizes() != y->sizes() || (gate && gate->sizes() != y->sizes())) Py_RETURN_NONE;
    for (const Tensor *t : {y, gate, w, out})
        if (t && (t->scalar_type() != y->scalar_type() || !rows_in_order(*t))) Py_RETURN_NONE;
    la_norm_shape_t s{};
    double eps;
    const long act = PyLong_AsLong(args[5]);
    if (!weights(w, y->size(-1)) || y->size(-1) > INT32_MAX || !number(args[4], &eps)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const bool heads = y->dim() == 3;
    s.rows = y->size(0);
    s.heads = heads ? (int32_t)y->size(1) : 1;
    s.dim = (int32_t)y->size(-1);
    s.eps = (float)eps;
    s.scale = 1.0f;
    s.x_dtype = s.res_dtype = dtype_code(*y);
    s.activation = (int32_t)act;
    s.gate_first = args[6] == Py_True;
    if (s.x_dtype < 0 || (heads && y->size(1) > INT32_MAX) || !PyBool_Check(args[6])) Py_RETURN_NONE;
    s.y_row_stride = stride(*y, 0);
    s.y_head_stride = heads ? stride(*y, 1) : 0;
    if (gate) {
        s.gate_row_stride = stride(*gate, 0);
        s.gate_head_stride = heads ? stride(*gate, 1) : 0;
    }
    s.out_row_stride = stride(*out, 0);
    s.out_head_stride = heads ? stride(*out, 1) : 0;
    return PyLong_FromLong(norm_gated(&s, ptr(y), ptr(gate), ptr(w), ptr(out), c10::hip::getCurrentHIPStream(dev.index()).stream()));
}

// residual(y, residual, pre_weight, out, post_weight, gate, scale, residual_out, eps): likewise
PyObject *residual(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    if (n_args != 9) Py_RETURN_NONE;
    bool ok = true;
    const Tensor *y = tensor(args[0], ok), *res = tensor(args[1], ok), *w = tensor(args[2], ok), *out = tensor(args[3], ok),
                 *post = tensor(args[4], ok), *gate = tensor(args[5], ok), *res_out = tensor(args[7], ok);
    if (!ok || !y || !res || !w != !out || y->dim() != 2 || y->numel() == 0) Py_RETURN_NONE;
    if (!res_out) res_out = res;
    c10::Device dev(c10::kCPU);
    if (!one_gpu({y, res, w, out, post, gate, res_out}, &dev)) Py_RETURN_NONE;
    const int64_t dim = y->size(1);
    if (res->sizes() != y->sizes() || res_out->sizes() != y->sizes() || (out && out->sizes() != y->sizes())) Py_RETURN_NONE;
    const bool each = gate && gate->dim() == 2;    // a gate for each token
    if (gate && (each ? gate->sizes() != y->sizes() : gate->dim() != 1 || gate->size(0) != dim)) Py_RETURN_NONE;
    for (const Tensor *t : {y, post, gate, w, out})
        if (t && t->scalar_type() != y->scalar_type()) Py_RETURN_NONE;
    for (const Tensor *t : {y, gate, res, res_out, out})
        if (t && !rows_in_order(*t)) Py_RETURN_NONE;
    double scale, eps;
    if (res->scalar_type() != res_out->scalar_type() || !weights(post, dim) || !weights(w, dim) || dim > INT32_MAX ||
        !number(args[6], &scale) || !number(args[8], &eps)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    la_norm_shape_t s{};
    s.rows = y->size(0);
    s.heads = 1;
    s.dim = (int32_t)dim;
    s.eps = (float)eps;
    s.scale = (float)scale;
    s.x_dtype = dtype_code(*y);
    s.res_dtype = dtype_code(*res);
    if (s.x_dtype < 0 || s.res_dtype < 0) Py_RETURN_NONE;
    s.y_row_stride = stride(*y, 0);
    s.gate_row_stride = each ? stride(*gate, 0) : 0;
    s.out_row_stride = out ? stride(*out, 0) : 0;
    s.res_row_stride = stride(*res, 0);
    s.res_out_row_stride = stride(*res_out, 0);
    return PyLong_FromLong(norm_residual(&s, ptr(y), ptr(post), ptr(gate), ptr(res), ptr(res_out), ptr(w), ptr(out),
                                         c10::hip::getCurrentHIPStream(dev.index()).stream()));
}

// No exception of torch's (out of memory, a tensor without storage) leaves through C: the long way
// meets it again and raises it.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n_args) {
    try {
        return F(self, args, n_args);
    } catch (const std::exception &) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<f>))
PyMethodDef methods[] = {{"attn", FAST(attn), METH_FASTCALL, nullptr},
                         {"gated", FAST(gated), METH_FASTCALL, nullptr},
                         {"residual", FAST(residual), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lacall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__lacall(void) { return PyModule_Create(&module); }
