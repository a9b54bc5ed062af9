// hs_binding.cpp -- the usual calls of the paged-cache entry points from
// Python without the interpreter in between: a decode step's kernel runs for
// ten microseconds, and checking and converting thirty arguments in Python and
// ctypes took as long again (13.4 us a call of hs_paged_decode, 5.5 here;
// hs_evict 14.2 and 3.7).  So did those of a step of several new tokens
// (hs_paged_extend, hs_rope_append, hs_paged_prefill).
//
// Each function looks at its tensors and makes the C call if everything is as
// in the common case: right types and shapes, contiguous, on the given device.
// Where anything is not, it returns None without having done anything, and
// hs.py goes through its own checks, which say what is wrong or take the
// general way (strided tensors, a workspace to allocate).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "hs_api.h"

namespace {

// One tensor's facts; `ok` only for a contiguous CUDA tensor on the device asked
// for, with at most four dimensions.
struct Tensor {
    at::ScalarType dtype = at::ScalarType::Undefined;
    int64_t dim[4] = {0, 0, 0, 0};
    int ndim = 0;
    void* ptr = nullptr;
    int64_t bytes = 0;
    bool ok = false;
};

bool as_int(PyObject* o, int64_t* out) {
    if (o == nullptr || !PyLong_CheckExact(o)) return false;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    *out = v;
    return true;
}

bool as_i32(PyObject* o, int32_t* out) {
    int64_t v;
    if (!as_int(o, &v) || v < INT32_MIN || v > INT32_MAX) return false;
    *out = int32_t(v);
    return true;
}

bool as_float(PyObject* o, float* out) {
    if (!PyFloat_Check(o) && !PyLong_CheckExact(o)) return false;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return false;
    *out = float(v);
    return true;
}

Tensor look(PyObject* o, int64_t device) {
    Tensor x;
    if (!THPVariable_Check(o)) return x;
    try {
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.get_device() != device || t.dim() > 4 || !t.is_contiguous())
            return x;
        x.dtype = t.scalar_type();
        x.ndim = int(t.dim());
        for (int i = 0; i < x.ndim; ++i) x.dim[i] = t.size(i);
        x.ptr = t.data_ptr();
        x.bytes = int64_t(t.nbytes());
        x.ok = true;
    } catch (const std::exception&) {  // no storage of its own, symbolic sizes
    }
    return x;
}

// Rows [tokens, heads, d] whose heads are packed; tokens may be strided.
struct Rows {
    at::ScalarType dtype = at::ScalarType::Undefined;
    int64_t n = 0, heads = 0, d = 0, stride = 0;
    void* ptr = nullptr;
    bool ok = false;
};

Rows look_rows(PyObject* o, int64_t device) {
    Rows x;
    if (!THPVariable_Check(o)) return x;
    try {
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.get_device() != device || t.dim() != 3) return x;
        x.dtype = t.scalar_type();
        x.n = t.size(0);
        x.heads = t.size(1);
        x.d = t.size(2);
        if (x.n > INT32_MAX || x.heads > INT32_MAX || x.d > INT32_MAX || t.stride(2) != 1 ||
            (x.heads > 1 && t.stride(1) != x.d))
            return x;
        x.stride = x.n > 1 ? t.stride(0) : x.heads * x.d;
        x.ptr = t.data_ptr();
        x.ok = x.dtype == at::kBFloat16 || x.dtype == at::kHalf;
    } catch (const std::exception&) {
    }
    return x;
}

// A paged cache pair [pages, page_size, kv_heads, d].
struct Cache {
    Tensor k, v;
    int64_t page_stride = 0, row_stride = 0, head_stride = 0;
    int element = -1;
};

bool look_cache(PyObject* k, PyObject* v, int64_t device, Cache* c);

// An optional status word: false where the common case does not apply.
bool look_status(PyObject* o, int64_t device, int32_t** out);

bool vector(const Tensor& t, at::ScalarType dtype, int64_t n) {
    return t.ok && t.dtype == dtype && t.ndim == 1 && t.dim[0] == n;
}
bool matrix(const Tensor& t, at::ScalarType dtype, int64_t rows, int64_t cols) {
    return t.ok && t.dtype == dtype && t.ndim == 2 && t.dim[0] == rows && t.dim[1] >= cols;
}
bool same_shape(const Tensor& a, const Tensor& b) {
    if (a.ndim != b.ndim) return false;
    for (int i = 0; i < a.ndim; ++i)
        if (a.dim[i] != b.dim[i]) return false;
    return true;
}

// The common case does not apply: leave everything to hs.py.
PyObject* general() {
    PyErr_Clear();
    Py_RETURN_NONE;
}

int element(at::ScalarType dtype) {
    return dtype == at::kBFloat16 ? HS_BF16 : dtype == at::kHalf ? HS_FP16 : dtype == at::kFloat8_e4m3fn ? HS_E4M3 : -1;
}

bool look_cache(PyObject* k, PyObject* v, int64_t device, Cache* c) {
    c->k = look(k, device);
    c->v = look(v, device);
    c->element = c->k.ok ? element(c->k.dtype) : -1;
    if (c->element < 0 || c->k.ndim != 4 || !c->v.ok || c->v.dtype != c->k.dtype ||
        !same_shape(c->k, c->v))
        return false;
    const int64_t* n = c->k.dim;
    for (int i = 0; i < 4; ++i)
        if (n[i] > INT32_MAX) return false;
    c->page_stride = n[0] > 1 ? n[1] * n[2] * n[3] : 0;
    c->row_stride = n[1] > 1 ? n[2] * n[3] : 0;
    c->head_stride = n[2] > 1 ? n[3] : 0;
    return true;
}

bool look_status(PyObject* o, int64_t device, int32_t** out) {
    *out = nullptr;
    if (o == Py_None) return true;
    const Tensor s = look(o, device);
    if (!s.ok || s.dtype != at::kInt || s.bytes < 4) return false;
    *out = static_cast<int32_t*>(s.ptr);
    return true;
}

// An optional fp32 vector of n entries.
bool look_scale(PyObject* o, int64_t device, int64_t n, const float** out) {
    *out = nullptr;
    if (o == Py_None) return true;
    const Tensor s = look(o, device);
    if (!vector(s, at::kFloat, n)) return false;
    *out = static_cast<const float*>(s.ptr);
    return true;
}

template <typename T>
T* as(const Tensor& t) {
    return static_cast<T*>(t.ptr);
}

// paged_extend(device, stream, new_lens, seq_lens, block_table, free_ring,
// ring_pos, page_size, max_tokens, lens_out, attend_lens, ring_out, cu_new, slot,
// row_req, positions, status): the arguments of hs.paged_extend; lens_out and
// ring_out may be None.
PyObject* paged_extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t device, stream;
    int32_t page_size, max_tokens;
    int32_t* status;
    if (n != 17 || !as_int(a[0], &device) || device < 0 || !as_int(a[1], &stream) ||
        !as_i32(a[7], &page_size) || !as_i32(a[8], &max_tokens) || max_tokens < 0)
        return general();
    const Tensor fresh = look(a[2], device), lens = look(a[3], device);
    const Tensor table = look(a[4], device), ring = look(a[5], device), pos = look(a[6], device);
    if (!fresh.ok || fresh.ndim != 1 || fresh.dtype != at::kInt || fresh.dim[0] > INT32_MAX)
        return general();
    const int64_t rows = fresh.dim[0];
    if (!vector(lens, at::kInt, rows) || !matrix(table, at::kInt, rows, 0) ||
        table.dim[1] > INT32_MAX || !ring.ok || ring.ndim != 1 || ring.dtype != at::kInt ||
        ring.dim[0] > INT32_MAX || !vector(pos, at::kLong, 2))
        return general();
    const Tensor lens_out = a[9] == Py_None ? lens : look(a[9], device);
    const Tensor attend = look(a[10], device);
    const Tensor ring_out = a[11] == Py_None ? pos : look(a[11], device);
    const Tensor cu = look(a[12], device), slot = look(a[13], device);
    const Tensor row = look(a[14], device), at = look(a[15], device);
    if (!vector(lens_out, at::kInt, rows) || !vector(attend, at::kInt, rows) ||
        !vector(ring_out, at::kLong, 2) || !vector(cu, at::kInt, rows + 1) ||
        !vector(slot, at::kInt, max_tokens) || !vector(row, at::kInt, max_tokens) ||
        !vector(at, at::kInt, max_tokens) || !look_status(a[16], device, &status))
        return general();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = hs_paged_extend(as<const int32_t>(fresh), as<const int32_t>(lens), as<int32_t>(table),
                         table.dim[1], int32_t(rows), int32_t(table.dim[1]), as<int32_t>(ring),
                         int32_t(ring.dim[0]), as<const int64_t>(pos), page_size, max_tokens,
                         as<int32_t>(lens_out), as<int32_t>(attend), as<int64_t>(ring_out),
                         as<int32_t>(cu), as<int32_t>(slot), as<int32_t>(row), as<int32_t>(at),
                         status, reinterpret_cast<hs_stream_t>(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

// rope_append(device, stream, q, k, v, positions, slot, turns, k_cache, v_cache,
// interleaved, mscale, k_scale, v_scale, q_out, status): the arguments of
// hs.rope_append with everything given but the scales and status.
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t device, stream;
    float mscale;
    const float *ks, *vs;
    int32_t* status;
    Cache c;
    if (n != 16 || !as_int(a[0], &device) || device < 0 || !as_int(a[1], &stream) ||
        !PyBool_Check(a[10]) || !as_float(a[11], &mscale))
        return general();
    const Rows q = look_rows(a[2], device), k = look_rows(a[3], device), v = look_rows(a[4], device);
    const Rows out = look_rows(a[14], device);
    const Tensor pos = look(a[5], device), slot = look(a[6], device), turns = look(a[7], device);
    if (!q.ok || !k.ok || !v.ok || !out.ok || k.dtype != q.dtype || v.dtype != q.dtype ||
        out.dtype != q.dtype || k.n != q.n || v.n != q.n || out.n != q.n || k.d != q.d ||
        v.d != q.d || out.d != q.d || v.heads != k.heads || out.heads != q.heads ||
        !vector(pos, at::kInt, q.n) || !vector(slot, at::kInt, q.n) || !turns.ok ||
        turns.ndim != 1 || turns.dtype != at::kLong || turns.dim[0] > INT32_MAX / 2 ||
        !look_cache(a[8], a[9], device, &c) || c.k.dim[2] != k.heads || c.k.dim[3] != q.d ||
        !look_scale(a[12], device, k.heads, &ks) || !look_scale(a[13], device, k.heads, &vs) ||
        !look_status(a[15], device, &status))
        return general();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = hs_rope_append(q.ptr, q.stride, k.ptr, k.stride, v.ptr, v.stride, element(q.dtype),
                        int32_t(q.n), int32_t(q.heads), int32_t(k.heads), int32_t(q.d),
                        as<const int32_t>(pos), as<const int32_t>(slot), as<const int64_t>(turns),
                        int32_t(2 * turns.dim[0]), a[10] == Py_True, mscale, out.ptr, out.stride,
                        c.k.ptr, c.v.ptr, c.element, c.page_stride, c.row_stride, c.head_stride,
                        int32_t(c.k.dim[0]), int32_t(c.k.dim[1]), ks, vs, status,
                        reinterpret_cast<hs_stream_t>(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

// paged_prefill(device, stream, q, k_cache, v_cache, block_table, cu_new,
// seq_lens, scale, window, num_sinks, max_len, k_scale, v_scale, out, lse,
// workspace, status)
PyObject* paged_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t device, stream;
    int32_t window, sinks;
    float scale;
    const float *ks, *vs;
    int32_t* status;
    Cache c;
    if (n != 18 || !as_int(a[0], &device) || device < 0 || !as_int(a[1], &stream) ||
        !as_float(a[8], &scale) || !as_i32(a[9], &window) || !as_i32(a[10], &sinks) ||
        a[14] == Py_None || a[15] == Py_None || a[16] == Py_None)
        return general();
    const Rows q = look_rows(a[2], device);
    const Tensor table = look(a[5], device), cu = look(a[6], device), lens = look(a[7], device);
    const Tensor out = look(a[14], device), lse = look(a[15], device), ws = look(a[16], device);
    if (!q.ok || !look_cache(a[3], a[4], device, &c) || c.k.dim[3] != q.d || !lens.ok ||
        lens.ndim != 1 || lens.dtype != at::kInt || lens.dim[0] > INT32_MAX)
        return general();
    const int64_t rows = lens.dim[0];
    if (!matrix(table, at::kInt, rows, 0) || table.dim[1] > INT32_MAX ||
        !vector(cu, at::kInt, rows + 1) || !out.ok || out.dtype != q.dtype || out.ndim != 3 ||
        out.dim[0] != q.n || out.dim[1] != q.heads || out.dim[2] != q.d ||
        !matrix(lse, at::kFloat, q.n, q.heads) || lse.dim[1] != q.heads || !ws.ok ||
        !look_scale(a[12], device, c.k.dim[2], &ks) || !look_scale(a[13], device, c.k.dim[2], &vs) ||
        !look_status(a[17], device, &status))
        return general();
    int64_t max_len = table.dim[1] * c.k.dim[1];
    if (a[11] != Py_None && !as_int(a[11], &max_len)) return general();
    if (max_len < 0 || max_len > INT32_MAX) return general();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = hs_paged_prefill(q.ptr, q.stride, element(q.dtype), int32_t(q.n), c.k.ptr, c.v.ptr,
                          c.element, c.page_stride, c.row_stride, c.head_stride,
                          int32_t(c.k.dim[0]), int32_t(c.k.dim[1]), as<const int32_t>(table),
                          table.dim[1], int32_t(table.dim[1]), int32_t(max_len),
                          as<const int32_t>(cu), as<const int32_t>(lens), ks, vs, int32_t(rows),
                          int32_t(q.heads), int32_t(c.k.dim[2]), int32_t(q.d), window, sinks, scale,
                          out.ptr, as<float>(lse), ws.ptr, ws.bytes, status,
                          reinterpret_cast<hs_stream_t>(stream));
    Py_END_ALLOW_THREADS
    if (rc == HS_ERR_CAPACITY) return general();  // a larger workspace is wanted
    return PyLong_FromLong(rc);
}

// paged_decode(device, stream, q, k_cache, v_cache, block_table, seq_lens,
// scale, window, num_sinks, max_len, k_scale, v_scale, score, score_decay,
// out, lse, workspace, status)
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t device, stream;
    int32_t window, sinks;
    float scale, decay;
    if (n != 19 || !as_int(a[0], &device) || device < 0 || !as_int(a[1], &stream) ||
        !as_float(a[7], &scale) || !as_i32(a[8], &window) || !as_i32(a[9], &sinks) ||
        !as_float(a[14], &decay) || a[15] == Py_None || a[16] == Py_None || a[17] == Py_None)
        return general();
    const Tensor q = look(a[2], device), k = look(a[3], device), v = look(a[4], device);
    const Tensor table = look(a[5], device), lens = look(a[6], device);
    const Tensor out = look(a[15], device), lse = look(a[16], device), ws = look(a[17], device);
    const int qe = q.ok ? element(q.dtype) : -1, ke = k.ok ? element(k.dtype) : -1;
    if (qe < 0 || qe == HS_E4M3 || ke < 0 || q.ndim != 3 || k.ndim != 4 || !v.ok ||
        v.dtype != k.dtype || !same_shape(k, v) || k.dim[3] != q.dim[2])
        return general();
    for (const Tensor* t : {&q, &k, &table})
        for (int i = 0; i < t->ndim; ++i)
            if (t->dim[i] > INT32_MAX) return general();
    const int64_t rows = q.dim[0], heads = q.dim[1], d = q.dim[2];
    const int64_t pages = k.dim[0], page = k.dim[1], kvh = k.dim[2];
    if (!matrix(table, at::kInt, rows, 0) || !vector(lens, at::kInt, rows) || !out.ok ||
        out.dtype != q.dtype || !same_shape(out, q) || !matrix(lse, at::kFloat, rows, heads) ||
        lse.dim[1] != heads || !ws.ok)
        return general();
    const int64_t blocks = table.dim[1];
    int64_t max_len = blocks * page;
    Tensor score, ks, vs;
    if (a[13] != Py_None) {
        score = look(a[13], device);
        if (!matrix(score, at::kFloat, rows, 0)) return general();
        if (score.dim[1] < max_len) max_len = score.dim[1];
    }
    if (a[10] != Py_None && !as_int(a[10], &max_len)) return general();
    if (max_len < 0 || max_len > INT32_MAX || (score.ok && score.dim[1] < max_len))
        return general();
    if (a[11] != Py_None) {
        ks = look(a[11], device);
        if (!vector(ks, at::kFloat, kvh)) return general();
    }
    if (a[12] != Py_None) {
        vs = look(a[12], device);
        if (!vector(vs, at::kFloat, kvh)) return general();
    }
    void* status = nullptr;
    if (a[18] != Py_None) {
        const Tensor s = look(a[18], device);
        if (!s.ok || s.dtype != at::kInt || s.bytes < 4) return general();
        status = s.ptr;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS  // a launch may wait for room in its stream
    rc = hs_paged_decode(
        q.ptr, heads * d, qe, k.ptr, v.ptr, ke, pages > 1 ? page * kvh * d : 0,
        page > 1 ? kvh * d : 0, kvh > 1 ? d : 0, int32_t(pages), int32_t(page),
        static_cast<const int32_t*>(table.ptr), blocks, int32_t(blocks), int32_t(max_len),
        static_cast<const int32_t*>(lens.ptr), static_cast<const float*>(ks.ptr),
        static_cast<const float*>(vs.ptr), int32_t(rows), int32_t(heads), int32_t(kvh), int32_t(d),
        window, sinks, scale, static_cast<float*>(score.ptr), score.ok ? score.dim[1] : 0, decay,
        out.ptr, static_cast<float*>(lse.ptr), ws.ptr, ws.bytes, static_cast<int32_t*>(status),
        reinterpret_cast<hs_stream_t>(stream));
    Py_END_ALLOW_THREADS
    if (rc == HS_ERR_CAPACITY) return general();  // a larger workspace is wanted
    return PyLong_FromLong(rc);
}

// evict(device, stream, score, seq_lens, budget, k_cache, v_cache, block_table,
// max_len, recent, num_sinks, positions, next_pos, score_out, positions_out,
// lens_out, (move_src, move_dst, move_count), status): the arguments of
// hs.evict, None where it has a default.
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t device, stream, max_len;
    int32_t budget, recent, sinks;
    if (n != 18 || !as_int(a[0], &device) || device < 0 || !as_int(a[1], &stream) ||
        !as_i32(a[4], &budget) || !as_i32(a[9], &recent) || !as_i32(a[10], &sinks) ||
        !PyTuple_CheckExact(a[16]) || PyTuple_GET_SIZE(a[16]) != 3)
        return general();
    const Tensor score = look(a[2], device), lens = look(a[3], device);
    if (!score.ok || score.ndim != 2 || score.dtype != at::kFloat || score.dim[0] > INT32_MAX ||
        score.dim[1] > INT32_MAX)
        return general();
    const int64_t rows = score.dim[0];
    max_len = score.dim[1];
    if (a[8] != Py_None && !as_int(a[8], &max_len)) return general();
    if (max_len < 0 || max_len > score.dim[1] || !vector(lens, at::kInt, rows)) return general();
    Tensor pos, next, so = score, po, lo = lens;
    if (a[11] != Py_None) {
        pos = look(a[11], device);
        if (!matrix(pos, at::kInt, rows, max_len)) return general();
    }
    po = pos;
    if (a[12] != Py_None) {
        next = look(a[12], device);
        if (!vector(next, at::kInt, rows)) return general();
    }
    if (a[13] != Py_None) {
        so = look(a[13], device);
        if (!matrix(so, at::kFloat, rows, max_len)) return general();
    }
    if (a[14] != Py_None) {
        po = look(a[14], device);
        if (!matrix(po, at::kInt, rows, max_len)) return general();
    }
    if (a[15] != Py_None) {
        lo = look(a[15], device);
        if (!vector(lo, at::kInt, rows)) return general();
    }
    const Tensor src = look(PyTuple_GET_ITEM(a[16], 0), device);
    const Tensor dst = look(PyTuple_GET_ITEM(a[16], 1), device);
    const Tensor count = look(PyTuple_GET_ITEM(a[16], 2), device);
    const Tensor k = look(a[5], device), table = look(a[7], device);
    if (!matrix(src, at::kInt, rows, 0) || src.dim[1] > INT32_MAX || !matrix(dst, at::kInt, rows, 0) ||
        dst.dim[1] != src.dim[1] || !vector(count, at::kInt, rows) || !k.ok || k.ndim != 4 ||
        !matrix(table, at::kInt, rows, 0))
        return general();
    Tensor v;
    if (a[6] != Py_None) {
        v = look(a[6], device);
        if (!v.ok || v.dtype != k.dtype || !same_shape(k, v)) return general();
    }
    int64_t e;
    if (element(k.dtype) >= 0) {
        e = k.dtype == at::kFloat8_e4m3fn ? 1 : 2;
    } else {
        return general();
    }
    const int64_t pages = k.dim[0], page = k.dim[1], kvh = k.dim[2], row = k.dim[3] * e;
    for (int i = 0; i < 4; ++i)
        if (k.dim[i] > INT32_MAX / 2) return general();
    if (table.dim[1] > INT32_MAX) return general();
    void* status = nullptr;
    if (a[17] != Py_None) {
        const Tensor s = look(a[17], device);
        if (!s.ok || s.dtype != at::kInt || s.bytes < 4) return general();
        status = s.ptr;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = hs_evict(
        static_cast<const float*>(score.ptr), score.dim[1], static_cast<const int32_t*>(pos.ptr),
        pos.ok ? pos.dim[1] : 0, static_cast<const int32_t*>(lens.ptr),
        static_cast<const int32_t*>(next.ptr), int32_t(rows), int32_t(max_len), budget, recent,
        sinks, static_cast<float*>(so.ptr), so.dim[1], static_cast<int32_t*>(po.ptr),
        po.ok ? po.dim[1] : 0, static_cast<int32_t*>(lo.ptr), static_cast<int32_t*>(src.ptr),
        static_cast<int32_t*>(dst.ptr), static_cast<int32_t*>(count.ptr), int32_t(src.dim[1]),
        k.ptr, v.ptr, pages > 1 ? page * kvh * row : 0, page > 1 ? kvh * row : 0,
        kvh > 1 ? row : 0, int32_t(kvh), int32_t(row), int32_t(pages), int32_t(page),
        static_cast<const int32_t*>(table.ptr), table.dim[1], int32_t(table.dim[1]),
        static_cast<int32_t*>(status), reinterpret_cast<hs_stream_t>(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"paged_decode", fast(paged_decode), METH_FASTCALL, nullptr},
                         {"evict", fast(evict), METH_FASTCALL, nullptr},
                         {"paged_extend", fast(paged_extend), METH_FASTCALL, nullptr},
                         {"rope_append", fast(rope_append), METH_FASTCALL, nullptr},
                         {"paged_prefill", fast(paged_prefill), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hs_binding", nullptr, -1, methods,
                      nullptr,               nullptr,       nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hs_binding() { return PyModule_Create(&module); }
