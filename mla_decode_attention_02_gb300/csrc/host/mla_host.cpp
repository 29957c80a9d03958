// Argument marshalling of the tree step's and the chunk step's calls in C++ (a CPython
// extension on torch's own tensor objects).
//
// A call of a small operator takes 2-5 us on the GPU; checking a dozen tensors
// from Python and passing them through ctypes takes 10-20 us, so such calls were
// bound by their marshalling.  Each function below checks its arguments, makes
// the outputs that the caller did not bring and calls the C ABI (the addresses
// come from the binding, see bind()).  It returns
//   the outputs   if the call was made,
//   an int        the C ABI's status, if that refused the call,
//   None          if the arguments are not the plain case (a wrong type, shape or
//                 device, another device than the current one, ...): nothing was
//                 done, and the binding's own checks name the reason.
// No CUDA kernel and no arithmetic is here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>

#include "mla_chunk.h"
#include "mla_fp8.h"
#include "mla_tree.h"

namespace {

struct Entry {
    decltype(&mla_query) query;
    decltype(&mla_cache_append) append, append_fp8;
    decltype(&mla_tree_workspace_size) tree_workspace_size;
    decltype(&mla_tree_plan) tree_plan;
    decltype(&mla_tree_decode) tree_decode;
    decltype(&mla_tree_decode_fp8) tree_decode_fp8;
    decltype(&mla_cache_commit) commit;
    decltype(&mla_rotate) rotate;
    decltype(&mla_residual_norm) residual_norm;
    decltype(&mla_residual_norm_fp8) residual_norm_fp8;
    decltype(&mla_chunk_workspace_size) chunk_workspace_size;
    decltype(&mla_chunk_plan) chunk_plan;
    decltype(&mla_chunk_attend) chunk_attend;
    decltype(&mla_chunk_attend_fp8) chunk_attend_fp8;
};
Entry g_entry;
bool g_bound = false;

constexpr int64_t kH = MLA_NUM_HEADS, kL = MLA_D_LATENT, kR = MLA_D_ROPE, kN = 128, kP = MLA_PAGE_SIZE;
constexpr int64_t kRow = kL + kR;

// An argument's tensor, or null.
const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool is(const at::Tensor &t, at::ScalarType type, c10::IntArrayRef shape, int dev, uintptr_t align) {
    return t.scalar_type() == type && t.sizes() == shape && t.is_cuda() && t.get_device() == dev && t.is_contiguous() &&
           (reinterpret_cast<uintptr_t>(t.data_ptr()) & (align - 1)) == 0;
}

// Address of a dense argument, or null.
void *dense(PyObject *o, at::ScalarType type, c10::IntArrayRef shape, int dev, uintptr_t align) {
    const at::Tensor *t = tensor(o);
    return t && is(*t, type, shape, dev, align) ? t->data_ptr() : nullptr;
}

// Address of a bf16 argument whose last dimension is contiguous, or null; its other strides.
void *strided(PyObject *o, c10::IntArrayRef shape, int dev, int64_t *strides) {
    const at::Tensor *t = tensor(o);
    if (!t || t->scalar_type() != at::kBFloat16 || t->sizes() != shape || !t->is_cuda() || t->get_device() != dev ||
        (reinterpret_cast<uintptr_t>(t->data_ptr()) & 15))
        return nullptr;
    const size_t n = shape.size();
    if (t->stride((int64_t)n - 1) != 1) return nullptr;
    for (size_t i = 0; i + 1 < n; ++i) {
        int64_t v = t->stride((int64_t)i);
        if (i == 0 && shape[0] == 1) v = 8;   // of one element: never used
        if (v < 1 || v % 8 || v >= (int64_t)1 << 31) return nullptr;
        strides[i] = v;
    }
    return t->data_ptr();
}

at::Tensor make(c10::IntArrayRef shape, at::ScalarType type, int dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
}

// The caller's output or a new one; false if the caller's does not fit.
bool output(PyObject *o, at::ScalarType type, c10::IntArrayRef shape, int dev, at::Tensor *t) {
    if (o == Py_None) {
        *t = make(shape, type, dev);
        return true;
    }
    const at::Tensor *given = tensor(o);
    if (!given || !is(*given, type, shape, dev, type == at::kInt ? 4 : 16)) return false;
    *t = *given;
    return true;
}

bool status_word(PyObject *o, int dev, at::Tensor *t) {
    if (o == Py_None) {
        *t = at::zeros({1}, at::TensorOptions().dtype(at::kInt).device(at::kCUDA, (c10::DeviceIndex)dev));
        return true;
    }
    return output(o, at::kInt, {1}, dev, t);
}

// Whether the tensor fixes a device that is the current one.
bool here(const at::Tensor *t) {
    return g_bound && t && t->is_cuda() && t->get_device() == c10::cuda::current_device();
}

mla_stream_t stream_of(int dev) {
    return reinterpret_cast<mla_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}

// The plan owns its workspace and may be dropped while calls on this stream are still queued, and
// it may have been made on another stream: the allocator gives the memory out again only after them.
// (Nothing is done if it was allocated on this stream, or not by the allocator.)
void used_here(const at::Tensor &workspace, int dev) {
    c10::cuda::CUDACachingAllocator::recordStream(workspace.storage().data_ptr(),
                                                  c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev));
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

PyObject *status_error(mla_status st) { return PyLong_FromLong(st); }

bool cache_shape(const at::Tensor *t, bool fp8, bool layers) {
    if (!t) return false;
    const int64_t d = t->dim();
    return (d == 3 || (layers && d == 4)) && t->size(d - 2) == kP && t->size(d - 1) == (fp8 ? MLA_FP8_ROW_BYTES : kRow) &&
           t->numel() > 0;
}

// Every function: no C++ exception leaves it (torch's become its Python ones, out of memory too).
template <typename F>
PyObject *guarded(F f) {
    HANDLE_TH_ERRORS
    return f();
    END_HANDLE_TH_ERRORS
}
#define MLA_NOT_PLAIN Py_RETURN_NONE

// q_nope, q_pe, w_uk, positions, table, q_latent, q_rope, status -> (q_latent, q_rope, status)
PyObject *py_query(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const at::Tensor *q = n == 8 ? tensor(a[0]) : nullptr;
        if (!here(q) || q->dim() != 3 || q->size(0) < 1 || q->size(0) > INT32_MAX) MLA_NOT_PLAIN;
        const int dev = q->get_device();
        const int64_t T = q->size(0);
        int64_t ns[2], ps[2];
        void *qn = strided(a[0], {T, kH, kN}, dev, ns), *qp = strided(a[1], {T, kH, kR}, dev, ps);
        void *w = dense(a[2], at::kBFloat16, {kH, kN, kL}, dev, 16), *pos = dense(a[3], at::kInt, {T}, dev, 4);
        void *table = dense(a[4], at::kFloat, {64}, dev, 4);
        if (!qn || !qp || !w || !pos || !table) MLA_NOT_PLAIN;
        at::Tensor ql, qr, st;
        if (!output(a[5], at::kBFloat16, {T, kH, kL}, dev, &ql) || !output(a[6], at::kBFloat16, {T, kH, kR}, dev, &qr) ||
            !status_word(a[7], dev, &st))
            MLA_NOT_PLAIN;
        const mla_status rc =
            g_entry.query((int32_t)T, qn, ns[0], ns[1], qp, ps[0], ps[1], w, (const float *)table, (const int32_t *)pos,
                          ql.data_ptr(), qr.data_ptr(), (int32_t *)st.data_ptr(), stream_of(dev));
        if (rc != MLA_OK) return status_error(rc);
        return Py_BuildValue("(NNN)", wrap(ql), wrap(qr), wrap(st));
    });
}

// fp8, kv_latent, k_pe, gamma, cache, block_table, seq_lens, offsets, positions, rms_eps, table, status -> status
PyObject *py_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const at::Tensor *x = n == 12 ? tensor(a[1]) : nullptr;
        if (!here(x) || x->dim() != 2 || x->size(0) < 1 || x->size(0) > INT32_MAX) MLA_NOT_PLAIN;
        const bool fp8 = a[0] == Py_True;
        const int dev = x->get_device();
        const int64_t T = x->size(0);
        int64_t ls, ks;
        void *lat = strided(a[1], {T, kL}, dev, &ls), *pe = strided(a[2], {T, kR}, dev, &ks);
        void *gamma = dense(a[3], at::kBFloat16, {kL}, dev, 16);
        const at::Tensor *cache = tensor(a[4]), *bt = tensor(a[5]);
        if (!lat || !pe || !gamma || !cache_shape(cache, fp8, false) || !bt || bt->dim() != 2 || bt->numel() < 1 ||
            bt->size(0) >= INT32_MAX || bt->size(1) > INT32_MAX ||
            !is(*cache, fp8 ? at::kByte : at::kBFloat16, cache->sizes(), dev, 16) ||
            !is(*bt, at::kInt, bt->sizes(), dev, 4))
            MLA_NOT_PLAIN;
        const int64_t B = bt->size(0);
        void *sl = dense(a[6], at::kInt, {B}, dev, 4), *off = dense(a[7], at::kInt, {B + 1}, dev, 4);
        void *pos = a[8] == Py_None ? nullptr : dense(a[8], at::kInt, {T}, dev, 4);
        void *table = dense(a[10], at::kFloat, {64}, dev, 4);
        if (!sl || !off || (!pos && a[8] != Py_None) || !table || !PyFloat_Check(a[9])) MLA_NOT_PLAIN;
        at::Tensor st;
        if (!status_word(a[11], dev, &st)) MLA_NOT_PLAIN;
        const mla_ragged prob = {(int32_t)B, (int32_t)T, (int32_t)kH, (int32_t)kP, (int32_t)bt->size(1), 0};
        const mla_status rc = (fp8 ? g_entry.append_fp8 : g_entry.append)(
            &prob, lat, ls, pe, ks, gamma, (float)PyFloat_AS_DOUBLE(a[9]), (const float *)table, (const int32_t *)pos,
            cache->data_ptr(), cache->size(0), (const int32_t *)bt->data_ptr(), (const int32_t *)sl, (const int32_t *)off,
            (int32_t *)st.data_ptr(), stream_of(dev));
        if (rc != MLA_OK) return status_error(rc);
        return wrap(st);
    });
}

// seq_lens, offsets, masks, max_pages, workspace -> workspace
PyObject *py_tree_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const at::Tensor *lens = n == 5 ? tensor(a[0]) : nullptr, *masks = n == 5 ? tensor(a[2]) : nullptr;
        if (!here(lens) || lens->dim() != 1 || !masks || masks->dim() != 1 || lens->numel() < 1 || masks->numel() < 1 ||
            lens->numel() >= INT32_MAX || masks->numel() > INT32_MAX || !PyLong_CheckExact(a[3]))
            MLA_NOT_PLAIN;
        const int dev = lens->get_device();
        const int64_t B = lens->size(0), T = masks->size(0);
        int overflow = 0;
        const long pages = PyLong_AsLongAndOverflow(a[3], &overflow);
        void *sl = dense(a[0], at::kInt, {B}, dev, 4), *off = dense(a[1], at::kInt, {B + 1}, dev, 4);
        void *m = dense(a[2], at::kLong, {T}, dev, 8);
        if (!sl || !off || !m || overflow || pages < 1 || pages > INT32_MAX) MLA_NOT_PLAIN;
        const mla_ragged prob = {(int32_t)B, (int32_t)T, (int32_t)kH, (int32_t)kP, (int32_t)pages, 0};
        at::Tensor ws;
        if (a[4] == Py_None) {
            size_t bytes = 0;
            const mla_status rc = g_entry.tree_workspace_size(&prob, &bytes);
            if (rc != MLA_OK) return status_error(rc);
            ws = make({(int64_t)bytes}, at::kByte, dev);
        } else {
            const at::Tensor *given = tensor(a[4]);
            if (!given || !is(*given, at::kByte, given->sizes(), dev, 16)) MLA_NOT_PLAIN;
            ws = *given;
            used_here(ws, dev);
        }
        const mla_status rc = g_entry.tree_plan(&prob, (const int32_t *)sl, (const int32_t *)off, (const uint64_t *)m,
                                                ws.data_ptr(), (size_t)ws.numel(), stream_of(dev));
        if (rc != MLA_OK) return status_error(rc);
        return wrap(ws);
    });
}

// batch, tokens, max_pages, workspace, q_latent, q_rope, cache, block_table, scale, out, lse, flags, fp8, scratch
// (None: none; a positive int: so many bytes are made) -> (out, lse), or False, nothing done, if they could not be
PyObject *py_tree_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const at::Tensor *ws = n == 14 ? tensor(a[3]) : nullptr;
        if (!here(ws) || !PyFloat_Check(a[8])) MLA_NOT_PLAIN;
        const int dev = ws->get_device();
        const int64_t B = PyLong_AsLongLong(a[0]), T = PyLong_AsLongLong(a[1]), pages = PyLong_AsLongLong(a[2]);
        const long flags = PyLong_AsLong(a[11]);
        const int64_t room = PyLong_Check(a[13]) ? PyLong_AsLongLong(a[13]) : 1;
        if (PyErr_Occurred()) {
            PyErr_Clear();
            MLA_NOT_PLAIN;
        }
        if (B < 1 || B > INT32_MAX || T < 1 || T > INT32_MAX || pages < 1 || pages > INT32_MAX || room < 1) MLA_NOT_PLAIN;
        const bool fp8 = a[12] == Py_True;
        void *ql = dense(a[4], at::kBFloat16, {T, kH, kL}, dev, 16), *qr = dense(a[5], at::kBFloat16, {T, kH, kR}, dev, 16);
        const at::Tensor *cache = tensor(a[6]);
        void *bt = dense(a[7], at::kInt, {B, pages}, dev, 4);
        if (!ql || !qr || !bt || !cache_shape(cache, fp8, false) ||
            !is(*cache, fp8 ? at::kByte : at::kBFloat16, cache->sizes(), dev, 16) ||
            !is(*ws, at::kByte, ws->sizes(), dev, 16))
            MLA_NOT_PLAIN;
        at::Tensor out, lse, scratch;
        if (!output(a[9], at::kBFloat16, {T, kH, kL}, dev, &out) || !output(a[10], at::kFloat, {T, kH}, dev, &lse))
            MLA_NOT_PLAIN;
        if (PyLong_Check(a[13])) {
            try {
                scratch = make({room}, at::kByte, dev);
            } catch (const c10::OutOfMemoryError &) {
                Py_RETURN_FALSE;
            }
        } else if (a[13] != Py_None) {
            const at::Tensor *given = tensor(a[13]);
            if (!given || !is(*given, at::kByte, given->sizes(), dev, 16)) MLA_NOT_PLAIN;
            scratch = *given;
        }
        used_here(*ws, dev);
        const mla_ragged prob = {(int32_t)B, (int32_t)T, (int32_t)kH, (int32_t)kP, (int32_t)pages, (int32_t)flags};
        const float scale = (float)PyFloat_AS_DOUBLE(a[8]);
        const mla_status rc =
            fp8 ? g_entry.tree_decode_fp8(&prob, ql, qr, cache->data_ptr(), cache->size(0), (const int32_t *)bt, scale,
                                          out.data_ptr(), (float *)lse.data_ptr(), ws->data_ptr(), (size_t)ws->numel(),
                                          scratch.defined() ? scratch.data_ptr() : nullptr,
                                          scratch.defined() ? (size_t)scratch.numel() : 0, stream_of(dev))
                : g_entry.tree_decode(&prob, ql, qr, cache->data_ptr(), cache->size(0), (const int32_t *)bt, scale,
                                      out.data_ptr(), (float *)lse.data_ptr(), ws->data_ptr(), (size_t)ws->numel(),
                                      stream_of(dev));
        if (rc != MLA_OK) return status_error(rc);
        return Py_BuildValue("(NN)", wrap(out), wrap(lse));
    });
}

// fp8, cache, block_table, seq_lens, offsets, paths, path_lens, new_seq_lens, status -> (new_seq_lens, status)
PyObject *py_commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const at::Tensor *bt = n == 9 ? tensor(a[2]) : nullptr;
        if (!here(bt) || bt->dim() != 2 || bt->numel() < 1 || bt->size(0) >= INT32_MAX || bt->size(1) > INT32_MAX)
            MLA_NOT_PLAIN;
        const bool fp8 = a[0] == Py_True;
        const int dev = bt->get_device();
        const int64_t B = bt->size(0);
        const at::Tensor *cache = tensor(a[1]), *paths = tensor(a[5]);
        void *sl = dense(a[3], at::kInt, {B}, dev, 4), *off = dense(a[4], at::kInt, {B + 1}, dev, 4);
        void *lens = dense(a[6], at::kInt, {B}, dev, 4);
        if (!sl || !off || !lens || !paths || paths->dim() != 2 || paths->size(1) < 1 || paths->size(1) > INT32_MAX ||
            !is(*paths, at::kInt, {B, paths->size(1)}, dev, 4) || !is(*bt, at::kInt, bt->sizes(), dev, 4) ||
            !cache_shape(cache, fp8, true) || !is(*cache, fp8 ? at::kByte : at::kBFloat16, cache->sizes(), dev, 16))
            MLA_NOT_PLAIN;
        at::Tensor after, st;
        if (!output(a[7], at::kInt, {B}, dev, &after) || !status_word(a[8], dev, &st)) MLA_NOT_PLAIN;
        const int64_t layers = cache->dim() == 4 ? cache->size(0) : 1, pages = cache->size(cache->dim() - 3);
        if (layers > INT32_MAX) MLA_NOT_PLAIN;
        const int32_t row = fp8 ? MLA_FP8_ROW_BYTES : (int32_t)(2 * kRow);
        // the offsets alone say how many nodes there are: any bound on them will do
        const mla_ragged prob = {(int32_t)B, (1 << 24) - 1, (int32_t)kH, (int32_t)kP, (int32_t)bt->size(1), 0};
        const mla_status rc = g_entry.commit(
            &prob, cache->data_ptr(), (int32_t)layers, pages * kP * row, row, pages, (const int32_t *)bt->data_ptr(),
            (const int32_t *)sl, (const int32_t *)off, (const int32_t *)paths->data_ptr(), (int32_t)paths->size(1),
            (const int32_t *)lens, (int32_t *)after.data_ptr(), (int32_t *)st.data_ptr(), stream_of(dev));
        if (rc != MLA_OK) return status_error(rc);
        return Py_BuildValue("(NN)", wrap(after), wrap(st));
    });
}

// x, positions, table, layout, inverse, magnitude, out -> out
PyObject *py_rotate(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const at::Tensor *x = n == 7 ? tensor(a[0]) : nullptr;
        if (!here(x) || x->dim() != 3 || x->numel() < 1 || x->size(0) > INT32_MAX || x->size(1) > INT32_MAX ||
            !PyFloat_Check(a[5]))
            MLA_NOT_PLAIN;
        const int dev = x->get_device();
        const int64_t T = x->size(0), H = x->size(1), D = x->size(2);
        if (D != 16 && D != 32 && D != 64 && D != 128 && D != 256) MLA_NOT_PLAIN;
        const long layout = PyLong_AsLong(a[3]);
        int64_t xs[2], os[2] = {H * D, D};
        void *src = strided(a[0], {T, H, D}, dev, xs), *pos = dense(a[1], at::kInt, {T}, dev, 4);
        void *table = dense(a[2], at::kFloat, {D}, dev, 4);
        if (!src || !pos || !table) MLA_NOT_PLAIN;
        at::Tensor out;
        if (a[6] == Py_None) {
            out = make({T, H, D}, at::kBFloat16, dev);
        } else {
            if (!strided(a[6], {T, H, D}, dev, os)) MLA_NOT_PLAIN;
            out = *tensor(a[6]);
        }
        const mla_status rc = g_entry.rotate((int32_t)T, (int32_t)H, (int32_t)D, src, xs[0], xs[1], (const int32_t *)pos,
                                             (const float *)table, (int32_t)layout, a[4] == Py_True,
                                             (float)PyFloat_AS_DOUBLE(a[5]), out.data_ptr(), os[0], os[1], stream_of(dev));
        if (rc != MLA_OK) return status_error(rc);
        return wrap(out);
    });
}

// x, residual, weight, rms_eps, group (-1: bf16), out (codes), scales, residual_out -> (out, scales, residual_out)
PyObject *py_residual_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const at::Tensor *x = n == 8 ? tensor(a[0]) : nullptr;
        if (!here(x) || x->dim() != 2 || x->numel() < 1 || x->size(0) > INT32_MAX || x->size(1) > 16384 ||
            x->size(1) % 8 || !PyFloat_Check(a[3]) || !PyLong_Check(a[4]))
            MLA_NOT_PLAIN;
        const int dev = x->get_device();
        const int64_t T = x->size(0), N = x->size(1);
        const long group = PyLong_AsLong(a[4]);
        const bool added = a[1] != Py_None, fp8 = group >= 0;
        int64_t xs, rs = 8;
        void *src = strided(a[0], {T, N}, dev, &xs), *res = added ? strided(a[1], {T, N}, dev, &rs) : nullptr;
        void *w = dense(a[2], at::kBFloat16, {N}, dev, 16);
        if (!src || (added && !res) || !w || (!added && a[7] != Py_None)) MLA_NOT_PLAIN;
        at::Tensor out, scales, kept;
        if (!output(a[5], fp8 ? at::kFloat8_e4m3fn : at::kBFloat16, {T, N}, dev, &out) ||
            (fp8 && !output(a[6], at::kFloat, {T, group ? (N + group - 1) / group : 1}, dev, &scales)) ||
            (added && !output(a[7], at::kBFloat16, {T, N}, dev, &kept)))
            MLA_NOT_PLAIN;
        const float eps = (float)PyFloat_AS_DOUBLE(a[3]);
        void *to = added ? kept.data_ptr() : nullptr;
        const mla_status rc =
            fp8 ? g_entry.residual_norm_fp8((int32_t)T, (int32_t)N, src, xs, res, rs, w, eps, (int32_t)group,
                                            out.data_ptr(), (float *)scales.data_ptr(), to, stream_of(dev))
                : g_entry.residual_norm((int32_t)T, (int32_t)N, src, xs, res, rs, w, eps, out.data_ptr(), to,
                                        stream_of(dev));
        if (rc != MLA_OK) return status_error(rc);
        auto or_none = [](const at::Tensor &t) {
            if (t.defined()) return wrap(t);
            Py_INCREF(Py_None);
            return Py_None;
        };
        return Py_BuildValue("(NNN)", wrap(out), or_none(scales), or_none(kept));
    });
}

// seq_lens, offsets, tokens, max_pages, kv_tokens, workspace -> workspace
PyObject *py_chunk_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const at::Tensor *lens = n == 6 ? tensor(a[0]) : nullptr;
        if (!here(lens) || lens->dim() != 1 || lens->numel() < 1 || lens->numel() >= INT32_MAX) MLA_NOT_PLAIN;
        const int dev = lens->get_device();
        const int64_t B = lens->size(0);
        const int64_t T = PyLong_AsLongLong(a[2]), pages = PyLong_AsLongLong(a[3]), kv = PyLong_AsLongLong(a[4]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            MLA_NOT_PLAIN;
        }
        void *sl = dense(a[0], at::kInt, {B}, dev, 4), *off = dense(a[1], at::kInt, {B + 1}, dev, 4);
        if (!sl || !off || T < 1 || T > INT32_MAX || pages < 1 || pages > INT32_MAX) MLA_NOT_PLAIN;
        const mla_chunk prob = {(int32_t)B, (int32_t)T, (int32_t)kH, (int32_t)kP, (int32_t)pages, 0, kv};
        at::Tensor ws;
        if (a[5] == Py_None) {
            size_t bytes = 0;
            const mla_status rc = g_entry.chunk_workspace_size(&prob, &bytes);
            if (rc != MLA_OK) return status_error(rc);
            ws = make({(int64_t)bytes}, at::kByte, dev);
        } else {
            const at::Tensor *given = tensor(a[5]);
            if (!given || !is(*given, at::kByte, given->sizes(), dev, 16)) MLA_NOT_PLAIN;
            ws = *given;
            used_here(ws, dev);
        }
        const mla_status rc = g_entry.chunk_plan(&prob, (const int32_t *)sl, (const int32_t *)off, ws.data_ptr(),
                                                 (size_t)ws.numel(), stream_of(dev));
        if (rc != MLA_OK) return status_error(rc);
        return wrap(ws);
    });
}

// batch, tokens, max_pages, kv_tokens, workspace, q_nope, q_rope, w_uk, w_uv, cache, block_table, scale, out, lse,
// scratch (a tensor, or how many bytes of it to make), fp8 -> out
PyObject *py_chunk_attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const at::Tensor *ws = n == 16 ? tensor(a[4]) : nullptr;
        if (!here(ws) || !PyFloat_Check(a[11])) MLA_NOT_PLAIN;
        const int dev = ws->get_device();
        const int64_t B = PyLong_AsLongLong(a[0]), T = PyLong_AsLongLong(a[1]), pages = PyLong_AsLongLong(a[2]);
        const int64_t kv = PyLong_AsLongLong(a[3]), room = PyLong_Check(a[14]) ? PyLong_AsLongLong(a[14]) : 1;
        if (PyErr_Occurred()) {
            PyErr_Clear();
            MLA_NOT_PLAIN;
        }
        if (B < 1 || B > INT32_MAX || T < 1 || T > INT32_MAX || pages < 1 || pages > INT32_MAX || room < 1) MLA_NOT_PLAIN;
        const bool fp8 = a[15] == Py_True;
        int64_t ns[2], rs[2];
        void *qn = strided(a[5], {T, kH, kN}, dev, ns), *qr = strided(a[6], {T, kH, kR}, dev, rs);
        void *uk = dense(a[7], at::kBFloat16, {kH, kN, kL}, dev, 16), *uv = dense(a[8], at::kBFloat16, {kH, kN, kL}, dev, 16);
        const at::Tensor *cache = tensor(a[9]);
        void *bt = dense(a[10], at::kInt, {B, pages}, dev, 4);
        void *lse = a[13] == Py_None ? nullptr : dense(a[13], at::kFloat, {T, kH}, dev, 4);
        if (!qn || !qr || !uk || !uv || !bt || (!lse && a[13] != Py_None) || !cache_shape(cache, fp8, false) ||
            !is(*cache, fp8 ? at::kByte : at::kBFloat16, cache->sizes(), dev, 16) ||
            !is(*ws, at::kByte, ws->sizes(), dev, 16))
            MLA_NOT_PLAIN;
        at::Tensor out, scratch;
        if (!output(a[12], at::kBFloat16, {T, kH, kN}, dev, &out)) MLA_NOT_PLAIN;
        if (PyLong_Check(a[14])) {
            scratch = make({room}, at::kByte, dev);
        } else {
            const at::Tensor *given = tensor(a[14]);
            if (!given || !is(*given, at::kByte, given->sizes(), dev, 128)) MLA_NOT_PLAIN;
            scratch = *given;
        }
        used_here(*ws, dev);
        const mla_chunk prob = {(int32_t)B, (int32_t)T, (int32_t)kH, (int32_t)kP, (int32_t)pages, 0, kv};
        const mla_status rc = (fp8 ? g_entry.chunk_attend_fp8 : g_entry.chunk_attend)(
            &prob, qn, ns[0], ns[1], qr, rs[0], rs[1], uk, uv, cache->data_ptr(), cache->size(0), (const int32_t *)bt,
            (float)PyFloat_AS_DOUBLE(a[11]), out.data_ptr(), (float *)lse, ws->data_ptr(), (size_t)ws->numel(),
            scratch.data_ptr(), (size_t)scratch.numel(), stream_of(dev));
        if (rc != MLA_OK) return status_error(rc);
        return wrap(out);
    });
}

// The C ABI's addresses, in the order of Entry.
PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr int kEntries = sizeof(Entry) / sizeof(void *);
    if (n != kEntries) {
        PyErr_SetString(PyExc_TypeError, "bind: one address per entry point");
        return nullptr;
    }
    void *p[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return nullptr;
        }
    }
    static_assert(sizeof(p) == sizeof(g_entry), "entry table");
    memcpy(&g_entry, p, sizeof p);
    g_bound = true;
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(py_bind), METH_FASTCALL, nullptr},
    {"query", reinterpret_cast<PyCFunction>(py_query), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(py_append), METH_FASTCALL, nullptr},
    {"tree_plan", reinterpret_cast<PyCFunction>(py_tree_plan), METH_FASTCALL, nullptr},
    {"tree_decode", reinterpret_cast<PyCFunction>(py_tree_decode), METH_FASTCALL, nullptr},
    {"commit", reinterpret_cast<PyCFunction>(py_commit), METH_FASTCALL, nullptr},
    {"rotate", reinterpret_cast<PyCFunction>(py_rotate), METH_FASTCALL, nullptr},
    {"residual_norm", reinterpret_cast<PyCFunction>(py_residual_norm), METH_FASTCALL, nullptr},
    {"chunk_plan", reinterpret_cast<PyCFunction>(py_chunk_plan), METH_FASTCALL, nullptr},
    {"chunk_attend", reinterpret_cast<PyCFunction>(py_chunk_attend), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_mla_host", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mla_host() { return PyModule_Create(&kModule); }
