// The calls that are bound by what they cost the host -- single tokens, small
// layers -- without the interpreter's share: module _pycall, used by binding.py.
// Each function takes a call whose arguments are as they nearly always are
// (plain tensors of the right type, shape and device, dense where they have to
// be), allocates its outputs and calls the C ABI.  Anything else it leaves to the
// binding's own path, which names what is wrong: it then returns NotImplemented
// and has done nothing.
#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstdlib>

#include "../../include/ssmscan.h"

namespace {

// entry points of libssmscan.so, as loaded by the binding
struct Calls {
    decltype(&ssm_conv_fwd) conv_fwd;
    decltype(&ssm_conv_bwd) conv_bwd;
    decltype(&ssm_ckpt8_pack) pack;
    decltype(&ssm_ckpt8_unpack) unpack;
    decltype(&ssm_tokens_conv) tokens_conv;
    decltype(&ssm_tokens_scan) tokens_scan;
    decltype(&ssm_gated_fwd) gated_fwd;
    decltype(&ssm_gated_bwd) gated_bwd;
    decltype(&ssm_tokens_gated) tokens_gated;
    decltype(&ssm_group_norm_fwd) norm_fwd;
    decltype(&ssm_group_norm_bwd) norm_bwd;
    decltype(&ssm_tokens_pack8) pack_rows;
    decltype(&ssm_tokens_mm8) mm8;
    decltype(&ssm_workspace_bytes) bytes;
} g{};
constexpr int kCalls = 14;

// The arguments of one call, checked one by one; `ok` turns false at the first that is not as expected.
struct Args {
    PyObject* const* a;
    Py_ssize_t n, i = 0;
    bool ok = true;
    int dev = -1;
    at::ScalarType dt = at::kFloat;

    PyObject* next() { return a[i++]; }
    int flag() {
        const int v = PyObject_IsTrue(next());
        if (v < 0) {
            PyErr_Clear();
            ok = false;
        }
        return v == 1;
    }
    int64_t whole() { return PyLong_AsLongLong(next()); }
    // a count, and a real number (nothing else is taken for one: the binding's own path says what is wrong with it)
    int64_t count() {
        PyObject* o = next();
        if (!PyLong_CheckExact(o)) {
            ok = false;
            return 0;
        }
        const int64_t v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    float real() {
        PyObject* o = next();
        if (!PyFloat_CheckExact(o)) {
            ok = false;
            return 0.0f;
        }
        return (float)PyFloat_AS_DOUBLE(o);
    }
    // the next argument as a tensor of the call's device; null for None (or where not ok)
    const at::Tensor* tensor(bool required) {
        PyObject* o = next();
        if (o == Py_None) {
            if (required) ok = false;
            return nullptr;
        }
        if (!THPVariable_CheckExact(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor* t = &THPVariable_Unpack(o);
        if (!t->is_cuda() || t->layout() != at::kStrided || t->get_device() != dev) {
            ok = false;
            return nullptr;
        }
        return t;
    }
    const void* dense(at::ScalarType type, at::IntArrayRef shape, bool required = false) {
        const at::Tensor* t = tensor(required);
        if (!t) return nullptr;
        if (t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    // a matrix of rows, contiguous each, any stride from one to the next
    const void* rows(at::ScalarType type, int64_t T, int64_t D, int64_t* stride) {
        const at::Tensor* t = tensor(true);
        if (!t) return nullptr;
        if (t->scalar_type() != type || t->dim() != 2 || t->size(0) != T || t->size(1) != D ||
            (t->stride(1) != 1 && D > 1)) {
            ok = false;
            return nullptr;
        }
        *stride = t->stride(0);
        return t->data_ptr();
    }
};
bool stream_type(at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16; }
int32_t code(at::ScalarType t) { return t == at::kBFloat16 ? SSM_BF16 : SSM_F32; }

PyObject* none_of_these() { Py_RETURN_NOTIMPLEMENTED; }
PyObject* wrapped(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev));
}
// a workspace, 256-byte aligned
struct Scratch {
    at::Tensor t;
    void* p = nullptr;
    size_t n = 0;
    int get(int op, const void* args, int dev) {
        if (int rc = g.bytes(op, args, &n)) return rc;
        if (n) {
            t = fresh({(int64_t)n + 256}, at::kByte, dev);
            p = (void*)(((uintptr_t)t.data_ptr() + 255) & ~(uintptr_t)255);
        }
        return SSM_OK;
    }
};
template <typename F>
PyObject* guarded(F f) {   // what C++ throws reaches the interpreter as torch's exceptions: no memory as OutOfMemoryError
    HANDLE_TH_ERRORS
    return f();
    END_HANDLE_TH_ERRORS
}

// sequences of a packed-row call: seq_start, slot, fresh, pool; pool (slots, D, inner), or (slots, D) with inner -1
struct Seq {
    const int32_t *start, *slot;
    const uint8_t* fresh;
    void* pool;
    int64_t S, slots, stride;
};
bool sequences(Args& in, int64_t T, int64_t D, int64_t inner, at::ScalarType pool_type, Seq* q) {
    const at::Tensor* start = in.tensor(false);
    q->S = T;
    q->start = nullptr;
    if (!in.ok) return false;
    if (start) {
        if (start->scalar_type() != at::kInt || start->dim() != 1 || start->size(0) < 1 || !start->is_contiguous())
            return in.ok = false;
        q->S = start->size(0) - 1;
        q->start = (const int32_t*)start->data_ptr();
    }
    q->slot = (const int32_t*)in.dense(at::kInt, {q->S});
    const at::Tensor* fr = in.tensor(false);
    q->fresh = nullptr;
    if (!in.ok) return false;
    if (fr) {
        if ((fr->scalar_type() != at::kBool && fr->scalar_type() != at::kByte) || fr->dim() != 1 ||
            fr->size(0) != q->S || !fr->is_contiguous())
            return in.ok = false;
        q->fresh = (const uint8_t*)fr->data_ptr();
    }
    const at::Tensor* pool = in.tensor(true);
    if (!pool) return false;
    if (pool->scalar_type() != pool_type || pool->dim() != (inner < 0 ? 2 : 3) || pool->size(1) != D || pool->numel() == 0 ||
        (pool->stride(1) != std::abs(inner) && D > 1) ||
        (inner >= 0 && (pool->size(2) != inner || (pool->stride(2) != 1 && inner > 1))))
        return in.ok = false;
    q->pool = pool->data_ptr();
    q->slots = pool->size(0);
    q->stride = pool->stride(0);
    return true;
}
// the output's rows: the caller's tensor, or a new one
void* out_rows(Args& in, at::ScalarType type, int64_t T, int64_t D, int64_t* stride, at::Tensor* made) {
    if (in.a[in.i] == Py_None) {
        ++in.i;
        if (!in.ok) return nullptr;
        *made = fresh({T, D}, type, in.dev);
        *stride = D;
        return made->data_ptr();
    }
    void* p = const_cast<void*>(in.rows(type, T, D, stride));
    if (in.ok && T > 1 && *stride < D) in.ok = false;
    return p;
}

// Every function: (device, stream, ...) -> its tensors, a status where the library refused the call, or
// NotImplemented.

// x, w, bias, silu, seq_start, slot, fresh, pool, y -> y
PyObject* tokens_conv(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        ssm_tokens_conv_args a{};
        const at::Tensor* x = in.tensor(true);
        if (!x || x->dim() != 2 || !stream_type(x->scalar_type())) return none_of_these();
        const int64_t T = x->size(0), D = x->size(1);
        if (x->stride(1) != 1 && D > 1) return none_of_these();
        const at::Tensor* w = in.tensor(true);
        if (!w || w->dim() != 2 || w->size(0) != D || w->scalar_type() != at::kFloat || !w->is_contiguous())
            return none_of_these();
        a.dtype = code(x->scalar_type());
        a.tokens = T; a.channels = D; a.width = w->size(1);
        a.x = x->data_ptr(); a.x_stride = x->stride(0);
        a.w = (const float*)w->data_ptr();
        a.bias = (const float*)in.dense(at::kFloat, {D});
        a.silu = in.flag();
        Seq q;
        if (!in.ok || !sequences(in, T, D, a.width - 1, x->scalar_type(), &q)) return none_of_these();
        at::Tensor y;
        a.y = out_rows(in, x->scalar_type(), T, D, &a.y_stride, &y);
        if (!in.ok) return none_of_these();
        a.seq_start = q.start; a.slot = q.slot; a.fresh = q.fresh; a.pool = q.pool;
        a.sequences = q.S; a.slots = q.slots; a.pool_stride = q.stride;
        if (int rc = g.tokens_conv(&a, stream)) return PyLong_FromLong(rc);
        return wrapped(y);
    });
}

// x, A, delta, Bm, C, z, skip, delta_bias, delta_softplus, seq_start, slot, fresh, pool, y -> y
PyObject* tokens_scan(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        ssm_tokens_scan_args a{};
        const at::Tensor* x = in.tensor(true);
        if (!x || x->dim() != 2 || !stream_type(x->scalar_type())) return none_of_these();
        const at::ScalarType dt = x->scalar_type();
        const int64_t T = x->size(0), D = x->size(1);
        if (x->stride(1) != 1 && D > 1) return none_of_these();
        const at::Tensor* A = in.tensor(true);
        if (!A || A->dim() != 2 || A->size(0) != D || A->scalar_type() != at::kFloat || !A->is_contiguous())
            return none_of_these();
        const int64_t N = A->size(1);
        a.dtype = code(dt);
        a.tokens = T; a.channels = D; a.state = N;
        a.x = x->data_ptr(); a.x_stride = x->stride(0);
        a.A = (const float*)A->data_ptr();
        a.delta = in.rows(dt, T, D, &a.delta_stride);
        a.Bm = in.rows(dt, T, N, &a.Bm_stride);
        a.C = in.rows(dt, T, N, &a.C_stride);
        if (in.a[in.i] == Py_None) ++in.i;
        else a.z = in.rows(dt, T, D, &a.z_stride);
        a.skip = (const float*)in.dense(at::kFloat, {D});
        a.delta_bias = (const float*)in.dense(at::kFloat, {D});
        a.delta_softplus = in.flag();
        Seq q;
        if (!in.ok || !sequences(in, T, D, N, at::kFloat, &q)) return none_of_these();
        at::Tensor y;
        a.y = out_rows(in, dt, T, D, &a.y_stride, &y);
        if (!in.ok) return none_of_these();
        a.seq_start = q.start; a.slot = q.slot; a.fresh = q.fresh; a.pool = (float*)q.pool;
        a.sequences = q.S; a.slots = q.slots; a.pool_stride = q.stride;
        Scratch ws;
        if (q.start)
            if (int rc = ws.get(SSM_OP_TOKENS_SCAN, &a, in.dev)) return PyLong_FromLong(rc);
        if (int rc = g.tokens_scan(&a, ws.p, ws.n, stream)) return PyLong_FromLong(rc);
        return wrapped(y);
    });
}

// the input of a convolution: x, or x8 and x8_scale with the stream's type from `like`; then w, bias, init, silu
bool conv_input(Args& in, const at::Tensor* like, ssm_conv_args* a, at::ScalarType* dt) {
    const at::Tensor* x = in.tensor(false);
    const at::Tensor* x8 = in.tensor(false);
    const at::Tensor* sc = in.tensor(false);
    if (!in.ok || !x == !x8) return false;
    const at::Tensor* s = x ? x : x8;
    if (s->dim() != 3 || !s->is_contiguous()) return false;
    a->batch = s->size(0); a->channels = s->size(1); a->length = s->size(2);
    if (x) {
        *dt = x->scalar_type();
        a->x = x->data_ptr();
        if (like && like->scalar_type() != *dt) return false;
    } else {
        if (!sc || !like || x8->scalar_type() != at::kChar || sc->scalar_type() != at::kFloat || !sc->is_contiguous() ||
            sc->sizes() != at::IntArrayRef({a->batch, a->channels, (a->length + SSM_CKPT8_BLOCK - 1) / SSM_CKPT8_BLOCK}))
            return false;
        *dt = like->scalar_type();
        a->x8 = (const int8_t*)x8->data_ptr();
        a->x8_scale = (const float*)sc->data_ptr();
    }
    if (!stream_type(*dt)) return false;
    a->dtype = code(*dt);
    const at::Tensor* w = in.tensor(true);
    if (!w || w->dim() != 2 || w->size(0) != a->channels || w->scalar_type() != at::kFloat || !w->is_contiguous())
        return false;
    a->width = w->size(1);
    a->w = (const float*)w->data_ptr();
    a->bias = (const float*)in.dense(at::kFloat, {a->channels});
    a->init = in.dense(*dt, {a->batch, a->channels, a->width - 1});
    a->silu = in.flag();
    return in.ok && a->width > 0;
}

// x, None, None, w, bias, init, silu, want_y, want_last, want_ckpt8 -> (y, last, x8, x8_scale)
PyObject* conv_fwd(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        ssm_conv_args a{};
        at::ScalarType dt;
        if (!conv_input(in, nullptr, &a, &dt)) return none_of_these();
        ssm_conv_fwd_out o{};
        at::Tensor y, last, x8, sc;
        const int64_t B = a.batch, D = a.channels, L = a.length;
        const int want_y = in.flag(), want_last = in.flag(), want_ckpt8 = in.flag();
        if (!in.ok) return none_of_these();
        if (want_y) o.y = (y = fresh({B, D, L}, dt, in.dev)).data_ptr();
        if (want_last) o.last = (last = fresh({B, D, a.width - 1}, dt, in.dev)).data_ptr();
        if (want_ckpt8) {
            o.x8 = (int8_t*)(x8 = fresh({B, D, L}, at::kChar, in.dev)).data_ptr();
            o.x8_scale = (float*)(sc = fresh({B, D, (L + SSM_CKPT8_BLOCK - 1) / SSM_CKPT8_BLOCK}, at::kFloat, in.dev))
                             .data_ptr();
        }
        if (int rc = g.conv_fwd(&a, &o, stream)) return PyLong_FromLong(rc);
        return Py_BuildValue("(NNNN)", wrapped(y), wrapped(last), wrapped(x8), wrapped(sc));
    });
}

// gy, glast, x, x8, x8_scale, w, bias, init, silu, and which of gx, gw, gbias, ginit -> these
PyObject* conv_bwd(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        const at::Tensor* gy = in.tensor(true);
        const at::Tensor* glast = in.tensor(false);
        ssm_conv_args a{};
        at::ScalarType dt;
        if (!in.ok || !gy->is_contiguous() || !conv_input(in, gy, &a, &dt)) return none_of_these();
        const int64_t B = a.batch, D = a.channels, L = a.length, W = a.width;
        if (gy->sizes() != at::IntArrayRef({B, D, L})) return none_of_these();
        if (glast && (glast->scalar_type() != dt || glast->sizes() != at::IntArrayRef({B, D, W - 1}) ||
                      !glast->is_contiguous()))
            return none_of_these();
        ssm_conv_grads o{};
        at::Tensor gx, gw, gb, gi;
        if (in.flag()) o.gx = (gx = fresh({B, D, L}, dt, in.dev)).data_ptr();
        if (in.flag()) o.gw = (float*)(gw = fresh({D, W}, at::kFloat, in.dev)).data_ptr();
        if (in.flag()) o.gbias = (float*)(gb = fresh({D}, at::kFloat, in.dev)).data_ptr();
        if (in.flag()) o.ginit = (gi = fresh({B, D, W - 1}, dt, in.dev)).data_ptr();
        Scratch ws;
        if (int rc = ws.get(SSM_OP_CONV_BWD, &a, in.dev)) return PyLong_FromLong(rc);
        if (int rc = g.conv_bwd(&a, gy->data_ptr(), glast ? glast->data_ptr() : nullptr, &o, ws.p, ws.n, stream))
            return PyLong_FromLong(rc);
        return Py_BuildValue("(NNNN)", wrapped(gx), wrapped(gw), wrapped(gb), wrapped(gi));
    });
}

// x -> (x8, x8_scale)
PyObject* ckpt8_pack(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        const at::Tensor* x = in.tensor(true);
        if (!x || x->dim() != 3 || !stream_type(x->scalar_type()) || !x->is_contiguous()) return none_of_these();
        ssm_ckpt8_args a{};
        a.dtype = code(x->scalar_type());
        a.batch = x->size(0); a.channels = x->size(1); a.length = x->size(2);
        at::Tensor x8 = fresh(x->sizes(), at::kChar, in.dev);
        at::Tensor sc = fresh({a.batch, a.channels, (a.length + SSM_CKPT8_BLOCK - 1) / SSM_CKPT8_BLOCK}, at::kFloat, in.dev);
        if (int rc = g.pack(&a, x->data_ptr(), (int8_t*)x8.data_ptr(), (float*)sc.data_ptr(), stream))
            return PyLong_FromLong(rc);
        return Py_BuildValue("(NN)", wrapped(x8), wrapped(sc));
    });
}

// x8, x8_scale, 1 for bf16 -> y
PyObject* ckpt8_unpack(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        const at::Tensor* x8 = in.tensor(true);
        if (!x8 || x8->dim() != 3 || x8->scalar_type() != at::kChar || !x8->is_contiguous()) return none_of_these();
        ssm_ckpt8_args a{};
        a.batch = x8->size(0); a.channels = x8->size(1); a.length = x8->size(2);
        const void* sc = in.dense(at::kFloat, {a.batch, a.channels, (a.length + SSM_CKPT8_BLOCK - 1) / SSM_CKPT8_BLOCK}, true);
        if (!in.ok) return none_of_these();
        const at::ScalarType dt = in.flag() ? at::kBFloat16 : at::kFloat;
        a.dtype = code(dt);
        at::Tensor y = fresh(x8->sizes(), dt, in.dev);
        if (int rc = g.unpack(&a, (const int8_t*)x8->data_ptr(), (const float*)sc, y.data_ptr(), stream))
            return PyLong_FromLong(rc);
        return wrapped(y);
    });
}

// x, r, i, lam, r_bias, i_bias, power, h0 of a gated recurrence over dense streams
bool gated_input(Args& in, ssm_gated_args* a, at::ScalarType* dt) {
    const at::Tensor* x = in.tensor(true);
    if (!x || x->dim() != 3 || !stream_type(x->scalar_type()) || !x->is_contiguous()) return false;
    *dt = x->scalar_type();
    a->dtype = code(*dt);
    const int64_t B = a->batch = x->size(0), D = a->channels = x->size(1), L = a->length = x->size(2);
    a->x = x->data_ptr();
    a->r = in.dense(*dt, {B, D, L}, true);
    a->i = in.dense(*dt, {B, D, L}, true);
    a->lam = (const float*)in.dense(at::kFloat, {D}, true);
    a->r_bias = (const float*)in.dense(at::kFloat, {D});
    a->i_bias = (const float*)in.dense(at::kFloat, {D});
    a->power = in.real();
    a->h0 = (const float*)in.dense(at::kFloat, {B, D});
    for (int64_t* s : {a->x_stride, a->r_stride, a->i_stride}) {
        s[0] = D * L;
        s[1] = L;
    }
    return in.ok;
}
int64_t gated_chunks(int64_t L) { return (L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK; }

// x, r, i, lam, r_bias, i_bias, power, h0, want_y, want_h_last, want_ckpt -> (y, h_last, ckpt)
PyObject* gated_fwd(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        ssm_gated_args a{};
        at::ScalarType dt;
        if (!gated_input(in, &a, &dt)) return none_of_these();
        ssm_gated_fwd_out o{};
        at::Tensor y, last, ck;
        const int want_y = in.flag(), want_last = in.flag(), want_ckpt = in.flag();
        if (!in.ok) return none_of_these();
        if (want_y) o.y = (y = fresh({a.batch, a.channels, a.length}, dt, in.dev)).data_ptr();
        if (want_last) o.h_last = (float*)(last = fresh({a.batch, a.channels}, at::kFloat, in.dev)).data_ptr();
        if (want_ckpt)
            o.ckpt = (float*)(ck = fresh({a.batch, a.channels, gated_chunks(a.length)}, at::kFloat, in.dev)).data_ptr();
        o.y_stride[0] = a.channels * a.length;
        o.y_stride[1] = a.length;
        if (int rc = g.gated_fwd(&a, &o, stream)) return PyLong_FromLong(rc);
        return Py_BuildValue("(NNN)", wrapped(y), wrapped(last), wrapped(ck));
    });
}

// gy, gh_last, ckpt, x, r, i, lam, r_bias, i_bias, power, h0, and which of gx, gr, gi, glam, gr_bias, gi_bias, gh0 -> these
PyObject* gated_bwd(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        const at::Tensor* gy = in.tensor(true);
        const at::Tensor* gl = in.tensor(false);
        const at::Tensor* ck = in.tensor(false);
        ssm_gated_args a{};
        at::ScalarType dt;
        if (!in.ok || !gated_input(in, &a, &dt)) return none_of_these();
        const int64_t B = a.batch, D = a.channels, L = a.length;
        if (gy->scalar_type() != dt || gy->sizes() != at::IntArrayRef({B, D, L}) || !gy->is_contiguous() ||
            (gl && (gl->scalar_type() != at::kFloat || gl->sizes() != at::IntArrayRef({B, D}) || !gl->is_contiguous())) ||
            (ck && (ck->scalar_type() != at::kFloat || ck->sizes() != at::IntArrayRef({B, D, gated_chunks(L)}) ||
                    !ck->is_contiguous())))
            return none_of_these();
        ssm_gated_bwd_in b{gy->data_ptr(), gl ? (const float*)gl->data_ptr() : nullptr,
                           ck ? (const float*)ck->data_ptr() : nullptr, {D * L, L}};
        ssm_gated_grads o{};
        at::Tensor t[7];
        void** streams[3] = {&o.gx, &o.gr, &o.gi};
        float** par[4] = {&o.glam, &o.gr_bias, &o.gi_bias, &o.gh0};
        for (int k = 0; k < 3; ++k)
            if (in.flag()) *streams[k] = (t[k] = fresh({B, D, L}, dt, in.dev)).data_ptr();
        for (int k = 0; k < 4; ++k)
            if (in.flag()) {
                t[3 + k] = k == 3 ? fresh({B, D}, at::kFloat, in.dev) : fresh({D}, at::kFloat, in.dev);
                *par[k] = (float*)t[3 + k].data_ptr();
            }
        for (int64_t* s : {o.gx_stride, o.gr_stride, o.gi_stride}) {
            s[0] = D * L;
            s[1] = L;
        }
        Scratch ws;
        if (int rc = ws.get(SSM_OP_GATED_BWD, &a, in.dev)) return PyLong_FromLong(rc);
        if (int rc = g.gated_bwd(&a, &b, &o, ws.p, ws.n, stream)) return PyLong_FromLong(rc);
        return Py_BuildValue("(NNNNNNN)", wrapped(t[0]), wrapped(t[1]), wrapped(t[2]), wrapped(t[3]), wrapped(t[4]),
                             wrapped(t[5]), wrapped(t[6]));
    });
}

// x, r, i, lam, r_bias, i_bias, power, seq_start, slot, fresh, pool, y -> y
PyObject* tokens_gated(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        ssm_tokens_gated_args a{};
        const at::Tensor* x = in.tensor(true);
        if (!x || x->dim() != 2 || !stream_type(x->scalar_type())) return none_of_these();
        const at::ScalarType dt = x->scalar_type();
        const int64_t T = x->size(0), D = x->size(1);
        if (x->stride(1) != 1 && D > 1) return none_of_these();
        a.dtype = code(dt);
        a.tokens = T; a.channels = D;
        a.x = x->data_ptr(); a.x_stride = x->stride(0);
        a.r = in.rows(dt, T, D, &a.r_stride);
        a.i = in.rows(dt, T, D, &a.i_stride);
        a.lam = (const float*)in.dense(at::kFloat, {D}, true);
        a.r_bias = (const float*)in.dense(at::kFloat, {D});
        a.i_bias = (const float*)in.dense(at::kFloat, {D});
        a.power = in.real();
        Seq q;
        if (!in.ok || !sequences(in, T, D, -1, at::kFloat, &q)) return none_of_these();
        at::Tensor y;
        a.y = out_rows(in, dt, T, D, &a.y_stride, &y);
        if (!in.ok) return none_of_these();
        a.seq_start = q.start; a.slot = q.slot; a.fresh = q.fresh; a.pool = (float*)q.pool;
        a.sequences = q.S; a.slots = q.slots; a.pool_stride = q.stride;
        Scratch ws;
        if (q.start)
            if (int rc = ws.get(SSM_OP_TOKENS_GATED, &a, in.dev)) return PyLong_FromLong(rc);
        if (int rc = g.tokens_gated(&a, ws.p, ws.n, stream)) return PyLong_FromLong(rc);
        return wrapped(y);
    });
}

// x, groups, w, bias, eps, silu, z of a group norm
bool norm_input(Args& in, ssm_group_norm_args* a, at::ScalarType* dt) {
    const at::Tensor* x = in.tensor(true);
    if (!x || x->dim() != 2 || !stream_type(x->scalar_type()) || (x->stride(1) != 1 && x->size(1) > 1)) return false;
    *dt = x->scalar_type();
    a->dtype = code(*dt);
    const int64_t T = a->rows = x->size(0), C = a->channels = x->size(1);
    a->x = x->data_ptr(); a->x_stride = x->stride(0);
    a->groups = in.count();
    a->w = (const float*)in.dense(at::kFloat, {C});
    a->bias = (const float*)in.dense(at::kFloat, {C});
    a->eps = in.real();
    a->silu = in.flag();
    if (in.a[in.i] == Py_None) ++in.i;
    else a->z = in.rows(*dt, T, C, &a->z_stride);
    return in.ok;
}
// x, groups, w, bias, eps, silu, z, y -> y
PyObject* group_norm_fwd(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        ssm_group_norm_args a{};
        at::ScalarType dt;
        if (!norm_input(in, &a, &dt)) return none_of_these();
        at::Tensor y;
        int64_t sy = 0;
        void* p = out_rows(in, dt, a.rows, a.channels, &sy, &y);
        if (!in.ok) return none_of_these();
        if (int rc = g.norm_fwd(&a, p, sy, stream)) return PyLong_FromLong(rc);
        return wrapped(y);
    });
}
// gy, x, groups, w, bias, eps, silu, z, and which of gx, gz, gw, gbias -> these
PyObject* group_norm_bwd(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        const at::Tensor* gy = in.tensor(true);
        ssm_group_norm_args a{};
        at::ScalarType dt;
        if (!in.ok || !norm_input(in, &a, &dt)) return none_of_these();
        const int64_t T = a.rows, C = a.channels;
        if (gy->scalar_type() != dt || gy->sizes() != at::IntArrayRef({T, C}) || (gy->stride(1) != 1 && C > 1))
            return none_of_these();
        ssm_group_norm_grads o{};
        at::Tensor gx, gz, gw, gb;
        if (in.flag()) o.gx = (gx = fresh({T, C}, dt, in.dev)).data_ptr();
        if (in.flag()) o.gz = (gz = fresh({T, C}, dt, in.dev)).data_ptr();
        if (in.flag()) o.gw = (float*)(gw = fresh({C}, at::kFloat, in.dev)).data_ptr();
        if (in.flag()) o.gbias = (float*)(gb = fresh({C}, at::kFloat, in.dev)).data_ptr();
        o.gx_stride = o.gz_stride = C;
        Scratch ws;
        if (int rc = ws.get(SSM_OP_GROUP_NORM_BWD, &a, in.dev)) return PyLong_FromLong(rc);
        if (int rc = g.norm_bwd(&a, gy->data_ptr(), gy->stride(0), &o, ws.p, ws.n, stream)) return PyLong_FromLong(rc);
        return Py_BuildValue("(NNNN)", wrapped(gx), wrapped(gz), wrapped(gw), wrapped(gb));
    });
}

// x -> (x8, x8_scale)
PyObject* tokens_pack8(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        const at::Tensor* x = in.tensor(true);
        if (!x || x->dim() != 2 || !stream_type(x->scalar_type()) || (x->stride(1) != 1 && x->size(1) > 1))
            return none_of_these();
        ssm_tokens_pack8_args a{};
        a.dtype = code(x->scalar_type());
        a.tokens = x->size(0); a.channels = x->size(1);
        a.x = x->data_ptr(); a.x_stride = x->stride(0);
        at::Tensor x8 = fresh(x->sizes(), at::kChar, in.dev), sc = fresh({a.tokens}, at::kFloat, in.dev);
        a.x8 = (int8_t*)x8.data_ptr(); a.x8_scale = (float*)sc.data_ptr();
        a.x8_stride = a.channels;
        if (int rc = g.pack_rows(&a, stream)) return PyLong_FromLong(rc);
        return Py_BuildValue("(NN)", wrapped(x8), wrapped(sc));
    });
}

// x8, x8_scale, w8, w8_scale, bias, 1 for bf16, y -> y
PyObject* tokens_mm8(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    return guarded([&]() -> PyObject* {
        Args in{argv, argc};
        in.dev = (int)in.whole();
        void* stream = (void*)(intptr_t)in.whole();
        ssm_tokens_mm8_args a{};
        const at::Tensor* x = in.tensor(true);
        if (!x || x->dim() != 2 || x->scalar_type() != at::kChar || (x->stride(1) != 1 && x->size(1) > 1))
            return none_of_these();
        const int64_t T = a.tokens = x->size(0), K = a.inputs = x->size(1);
        a.x8 = (const int8_t*)x->data_ptr(); a.x8_stride = x->stride(0);
        a.x8_scale = (const float*)in.dense(at::kFloat, {T}, true);
        const at::Tensor* w = in.tensor(true);
        if (!in.ok || w->dim() != 2 || w->scalar_type() != at::kChar || w->size(1) != K || (w->stride(1) != 1 && K > 1))
            return none_of_these();
        const int64_t N = a.outputs = w->size(0);
        a.w8 = (const int8_t*)w->data_ptr(); a.w8_stride = w->stride(0);
        a.w8_scale = (const float*)in.dense(at::kFloat, {N}, true);
        a.bias = (const float*)in.dense(at::kFloat, {N});
        const at::ScalarType dt = in.flag() ? at::kBFloat16 : at::kFloat;
        a.dtype = code(dt);
        at::Tensor y;
        a.y = out_rows(in, dt, T, N, &a.y_stride, &y);
        if (!in.ok) return none_of_these();
        if (int rc = g.mm8(&a, stream)) return PyLong_FromLong(rc);
        return wrapped(y);
    });
}

// addresses of the library's functions, in the order of Calls
PyObject* bind(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
    if (argc != kCalls) {
        PyErr_SetString(PyExc_TypeError, "bind takes the addresses of Calls");
        return nullptr;
    }
    void* p[kCalls];
    for (int i = 0; i < kCalls; ++i) {
        p[i] = PyLong_AsVoidPtr(argv[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "address 0");
            return nullptr;
        }
    }
    g = Calls{(decltype(g.conv_fwd))p[0],     (decltype(g.conv_bwd))p[1],    (decltype(g.pack))p[2],
              (decltype(g.unpack))p[3],       (decltype(g.tokens_conv))p[4], (decltype(g.tokens_scan))p[5],
              (decltype(g.gated_fwd))p[6],    (decltype(g.gated_bwd))p[7],   (decltype(g.tokens_gated))p[8],
              (decltype(g.norm_fwd))p[9],     (decltype(g.norm_bwd))p[10],   (decltype(g.pack_rows))p[11],
              (decltype(g.mm8))p[12],         (decltype(g.bytes))p[13]};
    Py_RETURN_NONE;
}

// A METH_FASTCALL function with the number of its arguments checked.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int N>
PyObject* counted(PyObject* self, PyObject* const* argv, Py_ssize_t argc) {
    if (argc != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, argc);
        return nullptr;
    }
    if (!g.bytes) {
        PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
        return nullptr;
    }
    return F(self, argv, argc);
}
PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"tokens_conv", (PyCFunction)(void (*)(void))counted<tokens_conv, 11>, METH_FASTCALL, nullptr},
    {"tokens_scan", (PyCFunction)(void (*)(void))counted<tokens_scan, 16>, METH_FASTCALL, nullptr},
    {"conv_fwd", (PyCFunction)(void (*)(void))counted<conv_fwd, 12>, METH_FASTCALL, nullptr},
    {"conv_bwd", (PyCFunction)(void (*)(void))counted<conv_bwd, 15>, METH_FASTCALL, nullptr},
    {"ckpt8_pack", (PyCFunction)(void (*)(void))counted<ckpt8_pack, 3>, METH_FASTCALL, nullptr},
    {"ckpt8_unpack", (PyCFunction)(void (*)(void))counted<ckpt8_unpack, 5>, METH_FASTCALL, nullptr},
    {"gated_fwd", (PyCFunction)(void (*)(void))counted<gated_fwd, 13>, METH_FASTCALL, nullptr},
    {"gated_bwd", (PyCFunction)(void (*)(void))counted<gated_bwd, 20>, METH_FASTCALL, nullptr},
    {"tokens_gated", (PyCFunction)(void (*)(void))counted<tokens_gated, 14>, METH_FASTCALL, nullptr},
    {"group_norm_fwd", (PyCFunction)(void (*)(void))counted<group_norm_fwd, 10>, METH_FASTCALL, nullptr},
    {"group_norm_bwd", (PyCFunction)(void (*)(void))counted<group_norm_bwd, 14>, METH_FASTCALL, nullptr},
    {"tokens_pack8", (PyCFunction)(void (*)(void))counted<tokens_pack8, 3>, METH_FASTCALL, nullptr},
    {"tokens_mm8", (PyCFunction)(void (*)(void))counted<tokens_mm8, 9>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pycall() { return PyModule_Create(&module); }
