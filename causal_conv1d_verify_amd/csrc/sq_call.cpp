// The short way from torch tensors to libseqops.so, as la_call.cpp has it for liblinattn.so: one C
// function per group of entry points.  It takes the calls that are plainly in order and answers None to
// every other; those go through the binding in sequence_ops.py, which checks again and says what is
// wrong.
#include "call_tensors.h"

#include "sequence_ops.h"

namespace {

enum { PREFILL, UPDATE, VERIFY, COMMIT };

bool table(const Tensor *t, int64_t rows, int64_t cols) {   // [rows, cols] int32, rows apart
    return !t || (t->scalar_type() == at::kInt && t->dim() == 2 && t->size(0) == rows && t->size(1) == cols && rows_in_order(*t));
}
bool floats(const Tensor *t, int64_t n) { return !t || (t->scalar_type() == at::kFloat && weights(t, n)); }

Tensor workspace_of(int64_t bytes, c10::Device dev) {
    return at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(dev));
}
int64_t bytes_of(const Tensor *t) { return t ? t->numel() * t->element_size() : 0; }

// scan(kind, x, dt, A, B, C, state, out, cu_seqlens, max_len, z, D, dt_bias, dt_softplus, slot_idx,
//      has_initial_state, num_tokens, workspace) -> the C ABI's return code, or None: not taken
PyObject *scan(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    if (n_args != 18) Py_RETURN_NONE;
    bool ok = true;
    const long kind = PyLong_AsLong(args[0]);
    const Tensor *x = tensor(args[1], ok), *dt = tensor(args[2], ok), *A = tensor(args[3], ok), *B = tensor(args[4], ok),
                 *C = tensor(args[5], ok), *state = tensor(args[6], ok), *out = tensor(args[7], ok), *cu = tensor(args[8], ok),
                 *z = tensor(args[10], ok), *D = tensor(args[11], ok), *bias = tensor(args[12], ok), *slot = tensor(args[14], ok),
                 *init = tensor(args[15], ok), *num = tensor(args[16], ok), *workspace = tensor(args[17], ok);
    const bool packed = kind == PREFILL, both = kind != COMMIT;
    if (!ok || !x || !dt || !A || !B || !state || (both && (!C || !out)) || packed != (cu != nullptr) || !PyBool_Check(args[13]))
        Py_RETURN_NONE;
    c10::Device dev(c10::kCPU);
    if (!one_gpu({state, x, dt, A, B, C, out, z, D, bias, cu, slot, init, num, workspace}, &dev)) Py_RETURN_NONE;
    const int64_t lead = packed ? 1 : 2;
    if (x->dim() != lead + 1 || B->dim() != lead + 1 || state->dim() != 3) Py_RETURN_NONE;
    for (int64_t i = 0; i < lead; ++i)
        if (x->size(i) == 0 || B->size(i) != x->size(i)) Py_RETURN_NONE;
    const int64_t d = x->size(lead), N = B->size(lead);
    if (dt->sizes() != x->sizes() || (z && z->sizes() != x->sizes()) || (out && out->sizes() != x->sizes()) ||
        (C && C->sizes() != B->sizes()) || d > INT32_MAX || N > INT32_MAX)
        Py_RETURN_NONE;
    for (const Tensor *t : {x, dt, B, C, z, out})
        if (t && (t->scalar_type() != x->scalar_type() || !rows_in_order(*t))) Py_RETURN_NONE;
    if (A->scalar_type() != at::kFloat || A->dim() != 2 || A->size(0) != d || A->size(1) != N || !A->is_contiguous() ||
        !floats(D, d) || !floats(bias, d))
        Py_RETURN_NONE;
    if (state->size(1) != d || state->size(2) != N || (N > 1 && state->stride(2) != 1) || (d > 1 && state->stride(1) != N))
        Py_RETURN_NONE;
    sq_scan_shape_t s{};
    s.d = (int32_t)d;
    s.d_state = (int32_t)N;
    s.softplus = args[13] == Py_True;
    if (packed) {
        if (workspace && !workspace->is_contiguous()) Py_RETURN_NONE;
        if (cu->dim() != 1 || cu->size(0) < 1 || !PyLong_CheckExact(args[9])) Py_RETURN_NONE;
        const int64_t rows = cu->size(0) - 1;
        const long long longest = PyLong_AsLongLong(args[9]);
        if (PyErr_Occurred()) PyErr_Clear(), ok = false;
        if (!ok || longest > INT32_MAX || rows > INT32_MAX || !int32_vec(cu, rows + 1) || !int32_vec(init, rows)) Py_RETURN_NONE;
        s.n_seq = (int32_t)rows;
        s.T = longest < 1 ? 1 : (int32_t)longest;
        s.tokens = x->size(0);
    } else {
        if (x->size(0) > INT32_MAX || x->size(1) > INT32_MAX || !int32_vec(num, x->size(0))) Py_RETURN_NONE;
        s.n_seq = (int32_t)x->size(0);
        s.T = (int32_t)x->size(1);
    }
    if (!int32_vec(slot, s.n_seq) || state->size(0) > INT32_MAX) Py_RETURN_NONE;
    s.x_dtype = dtype_code(*x);
    s.state_dtype = dtype_code(*state);
    if (s.x_dtype < 0 || s.state_dtype < 0) Py_RETURN_NONE;
    s.n_slots = (int32_t)state->size(0);
    auto strides = [&](const Tensor *t, int64_t *seq, int64_t *tok) {
        if (!t) return;
        *seq = packed ? 0 : stride(*t, 0);
        *tok = stride(*t, lead - 1);
    };
    strides(x, &s.x_seq_stride, &s.x_tok_stride);
    strides(dt, &s.dt_seq_stride, &s.dt_tok_stride);
    strides(z, &s.z_seq_stride, &s.z_tok_stride);
    strides(B, &s.b_seq_stride, &s.b_tok_stride);
    strides(C, &s.c_seq_stride, &s.c_tok_stride);
    strides(out, &s.out_seq_stride, &s.out_tok_stride);
    s.state_slot_stride = stride(*state, 0);
    const sq_scan_data_t p{ptr(x), ptr(dt), ptr(z), ptr(B), ptr(C), static_cast<const float *>(ptr(A)),
                           static_cast<const float *>(ptr(D)), static_cast<const float *>(ptr(bias))};
    hipStream_t stream = c10::hip::getCurrentHIPStream(dev.index()).stream();
    const int32_t *slots = static_cast<const int32_t *>(ptr(slot));
    int rc;
    if (kind == PREFILL) {
        const int64_t need = selscan_prefill_workspace(&s);
        if (need < 0) return PyLong_FromLongLong(need);
        Tensor made;
        if (need > 0 && !workspace) made = workspace_of(need, dev), workspace = &made;
        rc = selscan_prefill(&s, &p, ptr(state), slots, static_cast<const int32_t *>(ptr(cu)),
                             static_cast<const int32_t *>(ptr(init)), ptr(out), ptr(workspace), bytes_of(workspace), stream);
    } else if (kind == COMMIT) {
        rc = selscan_commit(&s, &p, ptr(state), slots, static_cast<const int32_t *>(ptr(num)), stream);
    } else {
        rc = kind == UPDATE ? selscan_update(&s, &p, ptr(state), slots, ptr(out), stream)
                            : selscan_verify(&s, &p, ptr(state), slots, ptr(out), stream);
    }
    return PyLong_FromLong(rc);
}

// rotary(q, k, positions, inv_freq, q_out, k_out, q_weight, k_weight, eps, interleaved): likewise
PyObject *rotary(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    if (n_args != 10) Py_RETURN_NONE;
    bool ok = true;
    const Tensor *q = tensor(args[0], ok), *k = tensor(args[1], ok), *pos = tensor(args[2], ok), *freq = tensor(args[3], ok),
                 *qo = tensor(args[4], ok), *ko = tensor(args[5], ok), *qw = tensor(args[6], ok), *kw = tensor(args[7], ok);
    if (!ok || !q || !qo || !k != !ko || (kw && !k) || !pos != !freq || q->dim() != 3 || q->numel() == 0 || !PyBool_Check(args[9]))
        Py_RETURN_NONE;
    c10::Device dev(c10::kCPU);
    if (!one_gpu({q, k, pos, freq, qo, ko, qw, kw}, &dev) || qo->sizes() != q->sizes()) Py_RETURN_NONE;
    const int64_t dim = q->size(2);
    if (k && (k->dim() != 3 || k->size(0) != q->size(0) || k->size(2) != dim || k->numel() == 0 || ko->sizes() != k->sizes() ||
              k->size(1) > INT32_MAX))
        Py_RETURN_NONE;
    for (const Tensor *t : {q, k, qo, ko})
        if (t && (t->scalar_type() != q->scalar_type() || !rows_in_order(*t))) Py_RETURN_NONE;
    for (const Tensor *t : {qw, kw})
        if (t && t->scalar_type() != q->scalar_type()) Py_RETURN_NONE;
    double eps;
    if (!weights(qw, dim) || !weights(kw, dim) || dim > INT32_MAX || q->size(1) > INT32_MAX || !number(args[8], &eps)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    sq_rotary_shape_t s{};
    if (freq) {
        if (pos->dim() != 1 || pos->size(0) != q->size(0) || (pos->size(0) > 1 && pos->stride(0) != 1) || freq->dim() != 1 ||
            (freq->size(0) > 1 && freq->stride(0) != 1) || freq->scalar_type() != at::kFloat || freq->size(0) > dim)
            Py_RETURN_NONE;
        if (pos->scalar_type() != at::kInt && pos->scalar_type() != at::kLong) Py_RETURN_NONE;
        s.wide_positions = pos->scalar_type() == at::kLong;
        s.rot = (int32_t)(2 * freq->size(0));
    }
    s.tokens = q->size(0);
    s.q_heads = (int32_t)q->size(1);
    s.k_heads = k ? (int32_t)k->size(1) : 0;
    s.dim = (int32_t)dim;
    s.eps = (float)eps;
    s.x_dtype = dtype_code(*q);
    s.interleaved = args[9] == Py_True;
    if (s.x_dtype < 0) Py_RETURN_NONE;
    s.q_tok_stride = stride(*q, 0), s.q_head_stride = stride(*q, 1);
    s.q_out_tok_stride = stride(*qo, 0), s.q_out_head_stride = stride(*qo, 1);
    if (k) {
        s.k_tok_stride = stride(*k, 0), s.k_head_stride = stride(*k, 1);
        s.k_out_tok_stride = stride(*ko, 0), s.k_out_head_stride = stride(*ko, 1);
    }
    return PyLong_FromLong(norm_rotary(&s, ptr(q), ptr(k), ptr(qw), ptr(kw), ptr(pos), static_cast<const float *>(ptr(freq)),
                                       ptr(qo), ptr(ko), c10::hip::getCurrentHIPStream(dev.index()).stream()));
}

// accept(tokens, target, uniform, num_tokens, next_token, draft, parent, window_index, path, slot_idx,
//        workspace): likewise
PyObject *accept(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    if (n_args != 11) Py_RETURN_NONE;
    bool ok = true;
    const Tensor *tokens = tensor(args[0], ok), *target = tensor(args[1], ok), *uniform = tensor(args[2], ok),
                 *num = tensor(args[3], ok), *next = tensor(args[4], ok), *draft = tensor(args[5], ok),
                 *parent = tensor(args[6], ok), *last = tensor(args[7], ok), *path = tensor(args[8], ok),
                 *slot = tensor(args[9], ok), *workspace = tensor(args[10], ok);
    if (!ok || !tokens || !target || !uniform || !num || !next || target->dim() != 3 || target->numel() == 0) Py_RETURN_NONE;
    c10::Device dev(c10::kCPU);
    if (!one_gpu({target, tokens, uniform, num, next, draft, parent, last, path, slot, workspace}, &dev)) Py_RETURN_NONE;
    const int64_t n = target->size(0), T = target->size(1), V = target->size(2);
    if (n > INT32_MAX || T > INT32_MAX || V > INT32_MAX || !rows_in_order(*target)) Py_RETURN_NONE;
    if (!table(tokens, n, T) || !table(parent, n, T) || !table(path, n, T) || !int32_vec(num, n) || !int32_vec(next, n) ||
        !int32_vec(last, n) || !int32_vec(slot, n))
        Py_RETURN_NONE;
    if (uniform->scalar_type() != at::kFloat || uniform->dim() != 2 || uniform->size(0) != n || uniform->size(1) != T ||
        !rows_in_order(*uniform) || (workspace && !workspace->is_contiguous()))
        Py_RETURN_NONE;
    if (draft && (draft->dim() != 3 || draft->size(0) != n || draft->size(1) != T - 1 || draft->size(2) != V ||
                  draft->scalar_type() != target->scalar_type() || !rows_in_order(*draft) || T < 2))
        Py_RETURN_NONE;
    sq_accept_shape_t s{};
    s.n_seq = (int32_t)n;
    s.T = (int32_t)T;
    s.vocab = (int32_t)V;
    s.p_dtype = dtype_code(*target);
    if (s.p_dtype < 0) Py_RETURN_NONE;
    s.tokens_stride = stride(*tokens, 0);
    s.uniform_stride = stride(*uniform, 0);
    if (parent) s.parent_stride = stride(*parent, 0);
    if (path) s.path_stride = stride(*path, 0);
    s.target_seq_stride = stride(*target, 0), s.target_tok_stride = stride(*target, 1);
    if (draft) s.draft_seq_stride = stride(*draft, 0), s.draft_tok_stride = stride(*draft, 1);
    const int64_t need = accept_drafts_workspace(&s);
    if (need < 0) return PyLong_FromLongLong(need);
    Tensor made;
    if (need > 0 && !workspace) made = workspace_of(need, dev), workspace = &made;
    auto ints = [](const Tensor *t) { return static_cast<int32_t *>(ptr(t)); };
    return PyLong_FromLong(accept_drafts(&s, ints(tokens), ints(parent), ptr(target), ptr(draft),
                                         static_cast<const float *>(ptr(uniform)), ints(slot), ints(num), ints(next),
                                         ints(last), ints(path), ptr(workspace), bytes_of(workspace),
                                         c10::hip::getCurrentHIPStream(dev.index()).stream()));
}

PyMethodDef methods[] = {{"scan", FAST(scan), METH_FASTCALL, nullptr},
                         {"rotary", FAST(rotary), METH_FASTCALL, nullptr},
                         {"accept", FAST(accept), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sqcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__sqcall(void) { return PyModule_Create(&module); }
