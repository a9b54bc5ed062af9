// hs_binding.cpp -- the usual calls of the paged-cache entry points from
// Python without the interpreter in between: a decode step's kernel runs for
// ten microseconds, and checking and converting thirty arguments in Python and
// ctypes took as long again (13.4 us a call of hs_paged_decode, 5.5 here;
// hs_evict 14.2 and 3.7).
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
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hs_binding", nullptr, -1, methods,
                      nullptr,               nullptr,       nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hs_binding() { return PyModule_Create(&module); }
