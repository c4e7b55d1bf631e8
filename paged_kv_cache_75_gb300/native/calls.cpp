// CPython module _native: the argument checks and the marshalling of the calls
// that a decode step makes (once a layer pa_qk_norm_rope, pa_qk_norm_rope_write,
// pa_decode_window, pa_prefill_varlen_window, pa_varlen_cascade; once pa_beam_select,
// pa_beam_reorder).  The same as a ctypes call would do,
// in a third of the time: through ctypes the checks and conversions took 8 of the 11
// microseconds of a small call.
//
// It knows tensors by their Python attributes alone (shape, dtype, data_ptr(), ...)
// and the library by the addresses of its functions, so it is built against neither.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include "pa_kv.h"

namespace {

PyObject *n_shape, *n_dtype, *n_get_device, *n_is_contiguous, *n_data_ptr, *n_stride, *n_numel, *n_element_size;
// set by setup(): torch's dtypes, its current-device and stream queries
PyObject *t_f16, *t_bf16, *t_e4m3, *t_i32, *t_i64, *t_f32, *f_get_device, *f_set_device, *f_stream;
decltype(&pa_qk_norm_rope) c_rope;
decltype(&pa_qk_norm_rope_write) c_write;
decltype(&pa_decode_window) c_decode;
decltype(&pa_prefill_varlen_window) c_prefill;
// set by setup_beams(), with torch's types of what ended
decltype(&pa_varlen_cascade) c_cascade;
decltype(&pa_beam_select) c_select;
decltype(&pa_beam_reorder) c_reorder;
PyObject *t_u8, *t_bool;

struct Tensor {
    Py_ssize_t dim;
    int64_t size[4];
    PyObject* dtype;  // borrowed: torch keeps its dtypes
    void* ptr;
};

bool as_int(PyObject* o, int64_t* out, int64_t lo = INT32_MIN, int64_t hi = INT32_MAX) {
    PyObject* i = PyNumber_Index(o);
    if (i == nullptr) return false;
    *out = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (*out == -1 && PyErr_Occurred()) return false;
    if (*out < lo || *out > hi) {
        PyErr_SetString(PyExc_OverflowError, "an argument does not fit 32 bits");
        return false;
    }
    return true;
}

bool as_float(PyObject* o, float* out) {
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) return false;
    *out = static_cast<float>(d);
    return true;
}

bool call_int(PyObject* o, PyObject* method, int64_t* out) {
    PyObject* r = PyObject_CallMethodNoArgs(o, method);
    if (r == nullptr) return false;
    *out = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return !(*out == -1 && PyErr_Occurred());
}

bool call_ptr(PyObject* o, void** out) {
    PyObject* r = PyObject_CallMethodNoArgs(o, n_data_ptr);
    if (r == nullptr) return false;
    *out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return !(*out == nullptr && PyErr_Occurred());
}

bool call_true(PyObject* o, PyObject* method, bool* out) {
    PyObject* r = PyObject_CallMethodNoArgs(o, method);
    if (r == nullptr) return false;
    *out = r == Py_True;
    Py_DECREF(r);
    return true;
}

bool sizes(PyObject* t, Py_ssize_t* dim, int64_t* out) {
    if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) > 4) return false;
    *dim = PyTuple_GET_SIZE(t);
    for (Py_ssize_t i = 0; i < *dim; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        if (out[i] == -1 && PyErr_Occurred()) return false;
    }
    return true;
}

// a tensor of at most four dimensions on device `index` (-1: any GPU's, which
// *index then becomes); contiguous, unless its strides are asked for
bool load(PyObject* o, const char* name, int64_t* index, Tensor* t, int64_t* strides = nullptr) {
    PyObject* shape = PyObject_GetAttr(o, n_shape);
    if (shape == nullptr) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        return false;
    }
    const bool ok = sizes(shape, &t->dim, t->size);
    Py_DECREF(shape);
    if (!ok) {
        if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s has too many dimensions", name);
        return false;
    }
    t->dtype = PyObject_GetAttr(o, n_dtype);
    if (t->dtype == nullptr) return false;
    Py_DECREF(t->dtype);
    int64_t dev;
    if (!call_int(o, n_get_device, &dev)) return false;
    if (*index < 0) *index = dev;
    if (dev < 0 || dev != *index) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor on the queries' device", name);
        return false;
    }
    if (strides != nullptr) {
        PyObject* s = PyObject_CallMethodNoArgs(o, n_stride);
        if (s == nullptr) return false;
        Py_ssize_t n;
        const bool fine = sizes(s, &n, strides);
        Py_DECREF(s);
        if (!fine) return false;
    } else {
        bool contiguous;
        if (!call_true(o, n_is_contiguous, &contiguous)) return false;
        if (!contiguous) {
            PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
            return false;
        }
    }
    return call_ptr(o, &t->ptr);
}

// contiguous, of that type and shape (n1 < 0: a vector)
bool load_as(PyObject* o, const char* name, int64_t* index, PyObject* dtype, int64_t n0, int64_t n1, Tensor* t) {
    if (!load(o, name, index, t)) return false;
    if (t->dtype != dtype) {
        PyErr_Format(PyExc_TypeError, "%s must be %R, got %R", name, dtype, t->dtype);
        return false;
    }
    if (t->dim != (n1 < 0 ? 1 : 2) || t->size[0] != n0) {
        PyErr_Format(PyExc_ValueError, "%s must have %lld %s", name, static_cast<long long>(n0),
                     n1 < 0 ? "entries" : "rows");
        return false;
    }
    return true;
}

bool code_of(PyObject* dtype, pa_dtype* code) {
    if (dtype == t_f16) *code = PA_F16;
    else if (dtype == t_bf16) *code = PA_BF16;
    else if (dtype == t_e4m3) *code = PA_FP8_E4M3;
    else {
        PyErr_Format(PyExc_TypeError, "unsupported dtype %R", dtype);
        return false;
    }
    return true;
}

// [T, heads, head_size] rows whose tokens may be strided -> the token stride
bool rows(PyObject* o, const char* name, int64_t* index, Tensor* t, int64_t* stride, const Tensor* like,
          int64_t heads) {
    int64_t s[4];
    if (!load(o, name, index, t, s)) return false;
    if (t->dim != 3) {
        PyErr_Format(PyExc_ValueError, "%s must be [tokens, heads, head_size]", name);
        return false;
    }
    if (like != nullptr && (t->dtype != like->dtype || t->size[0] != like->size[0] || t->size[2] != like->size[2] ||
                            (heads >= 0 && t->size[1] != heads))) {
        PyErr_Format(PyExc_ValueError, "%s must have the queries' type, tokens and head size, and its head count", name);
        return false;
    }
    const int64_t n = t->size[1], d = t->size[2];
    if ((d > 1 && s[2] != 1) || (n > 1 && s[1] != d)) {
        PyErr_Format(PyExc_ValueError, "the heads of a token of %s must be contiguous", name);
        return false;
    }
    // (a single token's stride says nothing)
    *stride = t->size[0] > 1 || s[0] > n * d ? s[0] : n * d;
    return true;
}

bool cache_of(PyObject* const* a, int64_t* index, pa_kv_cache* c) {
    Tensor k, v;
    if (!load(a[0], "k_cache", index, &k) || !load(a[1], "v_cache", index, &v)) return false;
    if (k.dim != 4 || v.dim != 4 || k.dtype != v.dtype || k.size[0] != v.size[0] || k.size[1] != v.size[1] ||
        k.size[2] != v.size[2] || k.size[3] != v.size[3]) {
        PyErr_SetString(PyExc_ValueError, "k_cache and v_cache must match");
        return false;
    }
    pa_dtype code;
    if (!code_of(k.dtype, &code)) return false;
    *c = {k.ptr, v.ptr, k.size[0], static_cast<int32_t>(k.size[2]), static_cast<int32_t>(k.size[1]),
          static_cast<int32_t>(k.size[3]), code, 1.f, 1.f};
    return as_float(a[2], &c->k_scale) && as_float(a[3], &c->v_scale);
}

bool status_of(PyObject* o, int64_t* index, int32_t** p) {
    *p = nullptr;
    if (o == Py_None) return true;
    Tensor t;
    if (!load(o, "dev_status", index, &t)) return false;
    if (t.dtype != t_i32) {
        PyErr_SetString(PyExc_ValueError, "dev_status must be int32");
        return false;
    }
    *p = static_cast<int32_t*>(t.ptr);
    return true;
}

// what a QKTransform hands over: (q_weight, k_weight, turns, eps, factor, interleaved)
bool transform_of(PyObject* o, int64_t* index, int64_t head_size, pa_qk_transform* tr) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 6) {
        PyErr_SetString(PyExc_TypeError, "transform must be a QKTransform");
        return false;
    }
    *tr = {nullptr, nullptr, 0.f, nullptr, 1.f, 0, 0};
    const char* names[3] = {"q_weight", "k_weight", "rope.turns"};
    for (int i = 0; i < 3; ++i) {
        PyObject* w = PyTuple_GET_ITEM(o, i);
        if (w == Py_None) continue;
        Tensor t;
        if (!load(w, names[i], index, &t)) return false;
        if (t.dim != 1 || t.dtype != (i < 2 ? t_f32 : t_i64) || (i < 2 && t.size[0] != head_size)) {
            PyErr_Format(PyExc_ValueError, "%s must have the rows' head size", names[i]);
            return false;
        }
        if (i == 0) tr->q_weight = static_cast<const float*>(t.ptr);
        else if (i == 1) tr->k_weight = static_cast<const float*>(t.ptr);
        else {
            tr->turns = static_cast<const uint64_t*>(t.ptr);
            tr->rotary_dim = static_cast<int32_t>(2 * t.size[0]);
        }
    }
    tr->interleaved = PyTuple_GET_ITEM(o, 5) == Py_True ? 1 : 0;
    return as_float(PyTuple_GET_ITEM(o, 3), &tr->eps) && as_float(PyTuple_GET_ITEM(o, 4), &tr->rope_factor);
}

// call(stream) on the device `index` and its current stream -> the status
template <typename Call>
PyObject* on_device(int64_t index, Call call) {
    PyObject* want = PyLong_FromLongLong(index);
    PyObject* cur = want != nullptr ? PyObject_CallNoArgs(f_get_device) : nullptr;
    PyObject* s = cur != nullptr ? PyObject_CallOneArg(f_stream, want) : nullptr;
    PyObject* result = nullptr;
    if (s != nullptr) {
        const int64_t now = PyLong_AsLongLong(cur);
        const pa_stream_t stream = PyErr_Occurred() ? nullptr : static_cast<pa_stream_t>(PyLong_AsVoidPtr(s));
        if (!PyErr_Occurred()) {
            // (from here to the device's restoring nothing but these two can fail:
            // no Python code runs with an error pending)
            PyObject* set = now != index ? PyObject_CallOneArg(f_set_device, want) : Py_NewRef(Py_None);
            if (set != nullptr) {
                pa_status st;
                Py_BEGIN_ALLOW_THREADS;
                st = call(stream);
                Py_END_ALLOW_THREADS;
                PyObject* back = now != index ? PyObject_CallOneArg(f_set_device, cur) : Py_NewRef(Py_None);
                if (back != nullptr) result = PyLong_FromLong(st);
                Py_XDECREF(back);
            }
            Py_XDECREF(set);
        }
    }
    Py_XDECREF(s);
    Py_XDECREF(cur);
    Py_XDECREF(want);
    return result;
}

bool count(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, got);
    return got == want;
}

// (q_out, k_out, q, k, positions, transform)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t dev = -1, qs, ks, qos, kos;
    Tensor q, k, qo, ko, pos{};
    pa_dtype dt;
    pa_qk_transform tr;
    if (!count(n, 6) || !rows(a[2], "q", &dev, &q, &qs, nullptr, -1) || !rows(a[3], "k", &dev, &k, &ks, &q, -1) ||
        !rows(a[0], "q_out", &dev, &qo, &qos, &q, q.size[1]) || !rows(a[1], "k_out", &dev, &ko, &kos, &q, k.size[1]) ||
        !code_of(q.dtype, &dt) ||
        (a[4] != Py_None && !load_as(a[4], "positions", &dev, t_i64, q.size[0], -1, &pos)) ||
        !transform_of(a[5], &dev, q.size[2], &tr))
        return nullptr;
    const auto T = q.size[0];
    const auto H = static_cast<int32_t>(q.size[1]), Hkv = static_cast<int32_t>(k.size[1]);
    const auto D = static_cast<int32_t>(q.size[2]);
    return on_device(dev, [&](pa_stream_t s) {
        return c_rope(qo.ptr, ko.ptr, q.ptr, k.ptr, dt, T, H, Hkv, D, qs, ks, qos, kos,
                      static_cast<const int64_t*>(pos.ptr), &tr, s);
    });
}

// (q_out, q, k, v, k_cache, v_cache, k_scale, v_scale, positions, slot_mapping, transform, dev_status)
PyObject* qk_norm_rope_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t dev = -1, qs, ks, vs, qos;
    Tensor q, k, v, qo, pos{}, slots;
    pa_dtype dt;
    pa_kv_cache c;
    pa_qk_transform tr;
    int32_t* status;
    if (!count(n, 12) || !rows(a[1], "q", &dev, &q, &qs, nullptr, -1) || !cache_of(a + 4, &dev, &c)) return nullptr;
    if (c.head_size != q.size[2]) {
        PyErr_SetString(PyExc_ValueError, "the cache must have the queries' head size");
        return nullptr;
    }
    if (!rows(a[2], "k", &dev, &k, &ks, &q, c.num_kv_heads) || !rows(a[3], "v", &dev, &v, &vs, &q, c.num_kv_heads) ||
        !rows(a[0], "q_out", &dev, &qo, &qos, &q, q.size[1]) || !code_of(q.dtype, &dt) ||
        (a[8] != Py_None && !load_as(a[8], "positions", &dev, t_i64, q.size[0], -1, &pos)) ||
        !load_as(a[9], "slot_mapping", &dev, t_i64, q.size[0], -1, &slots) ||
        !transform_of(a[10], &dev, q.size[2], &tr) || !status_of(a[11], &dev, &status))
        return nullptr;
    return on_device(dev, [&](pa_stream_t s) {
        return c_write(qo.ptr, q.ptr, k.ptr, v.ptr, dt, &c, q.size[0], static_cast<int32_t>(q.size[1]), qs, ks, vs, qos,
                       static_cast<const int64_t*>(pos.ptr), static_cast<const int64_t*>(slots.ptr), &tr, status, s);
    });
}

// contiguous q and out [rows, num_heads, head_size] beside the cache
bool queries(PyObject* out, PyObject* q, PyObject* const* cache, int64_t* dev, Tensor* tq, Tensor* to, pa_dtype* dt,
             pa_kv_cache* c) {
    if (!load(q, "q", dev, tq) || !load(out, "out", dev, to) || !code_of(tq->dtype, dt) || !cache_of(cache, dev, c))
        return false;
    if (tq->dim != 3 || to->dim != 3 || to->dtype != tq->dtype || to->size[0] != tq->size[0] ||
        to->size[1] != tq->size[1] || to->size[2] != tq->size[2] || c->head_size != tq->size[2]) {
        PyErr_SetString(PyExc_ValueError, "q and out must be [rows, num_heads, head_size] of one type, the cache of that "
                                          "head size");
        return false;
    }
    return true;
}

// (out, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, max_seq_len, scale, window, num_sinks,
// partition_size, workspace, dev_status)
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t dev = -1, max_len, window, sinks, part, ws_bytes = 0, elem;
    Tensor q, out, table, lens, ws{};
    pa_dtype dt;
    pa_kv_cache c;
    float scale;
    int32_t* status;
    if (!count(n, 15) || !queries(a[0], a[1], a + 2, &dev, &q, &out, &dt, &c) ||
        !load_as(a[6], "block_table", &dev, t_i32, q.size[0], 0, &table) ||
        !load_as(a[7], "seq_lens", &dev, t_i32, q.size[0], -1, &lens) || !as_int(a[8], &max_len) ||
        !as_float(a[9], &scale) || !as_int(a[10], &window) || !as_int(a[11], &sinks) || !as_int(a[12], &part) ||
        !status_of(a[14], &dev, &status))
        return nullptr;
    if (a[13] != Py_None) {
        if (!load(a[13], "workspace", &dev, &ws) || !call_int(a[13], n_numel, &ws_bytes) ||
            !call_int(a[13], n_element_size, &elem))
            return nullptr;
        ws_bytes *= elem;
    }
    return on_device(dev, [&](pa_stream_t s) {
        return c_decode(out.ptr, q.ptr, dt, &c, static_cast<const int32_t*>(table.ptr),
                        static_cast<int32_t>(table.size[1]), static_cast<const int32_t*>(lens.ptr),
                        static_cast<int32_t>(q.size[0]), static_cast<int32_t>(max_len),
                        static_cast<int32_t>(q.size[1]), scale, static_cast<int32_t>(window),
                        static_cast<int32_t>(sinks), static_cast<int32_t>(part), ws.ptr,
                        static_cast<size_t>(ws_bytes), status, s);
    });
}

// (out, q, k_cache, v_cache, k_scale, v_scale, block_table, cu_seq_lens_q, cu_seq_lens_k, max_seqlen_q,
// max_seqlen_k, scale, window, num_sinks, dev_status)
PyObject* prefill_varlen_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t dev = -1, max_q, max_k, window, sinks;
    Tensor q, out, table, cu_q, cu_k;
    pa_dtype dt;
    pa_kv_cache c;
    float scale;
    int32_t* status;
    if (!count(n, 15) || !queries(a[0], a[1], a + 2, &dev, &q, &out, &dt, &c) ||
        !load(a[7], "cu_seq_lens_q", &dev, &cu_q))
        return nullptr;
    const int64_t rows1 = cu_q.dim == 1 ? cu_q.size[0] : 0;
    if (rows1 < 1) {
        PyErr_SetString(PyExc_ValueError, "cu_seq_lens_q must have num_seqs + 1 entries");
        return nullptr;
    }
    if (!load_as(a[7], "cu_seq_lens_q", &dev, t_i32, rows1, -1, &cu_q) ||
        !load_as(a[8], "cu_seq_lens_k", &dev, t_i32, rows1, -1, &cu_k) ||
        !load_as(a[6], "block_table", &dev, t_i32, rows1 - 1, 0, &table) || !as_int(a[9], &max_q) ||
        !as_int(a[10], &max_k) || !as_float(a[11], &scale) || !as_int(a[12], &window) || !as_int(a[13], &sinks) ||
        !status_of(a[14], &dev, &status))
        return nullptr;
    return on_device(dev, [&](pa_stream_t s) {
        return c_prefill(out.ptr, q.ptr, dt, &c, static_cast<const int32_t*>(table.ptr),
                         static_cast<int32_t>(table.size[1]), static_cast<const int32_t*>(cu_q.ptr),
                         static_cast<const int32_t*>(cu_k.ptr), static_cast<int32_t>(rows1 - 1),
                         static_cast<int32_t>(max_q), static_cast<int32_t>(max_k), static_cast<int32_t>(q.size[1]), scale,
                         static_cast<int32_t>(window), static_cast<int32_t>(sinks), status, s);
    });
}

// contiguous, of that type and shape: n1 < 0 a vector, -2 in n0 any length
bool exact(PyObject* o, const char* name, int64_t* index, PyObject* dtype, int64_t n0, int64_t n1, Tensor* t) {
    if (!load(o, name, index, t)) return false;
    if (t->dtype != dtype) {
        PyErr_Format(PyExc_TypeError, "%s must be %R, got %R", name, dtype, t->dtype);
        return false;
    }
    if (t->dim != (n1 < 0 ? 1 : 2) || (n0 >= 0 && t->size[0] != n0) || (n1 >= 0 && t->size[1] != n1)) {
        if (n1 < 0) PyErr_Format(PyExc_ValueError, "%s must have %lld entries", name, static_cast<long long>(n0));
        else PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld]", name, static_cast<long long>(n0),
                          static_cast<long long>(n1));
        return false;
    }
    return true;
}

bool workspace_of(PyObject* o, int64_t* index, void** ptr, int64_t* bytes) {
    *ptr = nullptr;
    *bytes = 0;
    if (o == Py_None) return true;
    Tensor t;
    int64_t elem;
    if (!load(o, "workspace", index, &t) || !call_int(o, n_numel, bytes) || !call_int(o, n_element_size, &elem)) return false;
    *ptr = t.ptr;
    *bytes *= elem;
    return true;
}

bool fits32(int64_t n, const char* name) {
    if (n <= INT32_MAX) return true;
    PyErr_Format(PyExc_ValueError, "%s is too large", name);
    return false;
}

// (out, q, k_cache, v_cache, k_scale, v_scale, block_table, cu_seq_lens_q, cu_seq_lens_k, max_seqlen_q,
// max_seqlen_k, scale, cu_groups, shared_lens, max_group_size, max_shared_len, workspace, dev_status)
PyObject* varlen_cascade(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t dev = -1, max_q, max_k, max_group, max_shared, ws_bytes;
    Tensor q, out, table, cu_q, cu_k, cu_g, shared;
    pa_dtype dt;
    pa_kv_cache c;
    float scale;
    int32_t* status;
    void* ws;
    if (!count(n, 18) || !load(a[1], "q", &dev, &q) || !load(a[0], "out", &dev, &out)) return nullptr;
    if (out.dtype != q.dtype) {
        PyErr_Format(PyExc_TypeError, "out must be %R, got %R", q.dtype, out.dtype);
        return nullptr;
    }
    if (!queries(a[0], a[1], a + 2, &dev, &q, &out, &dt, &c) ||
        !exact(a[7], "cu_seq_lens_q", &dev, t_i32, -2, -1, &cu_q) || !exact(a[13], "shared_lens", &dev, t_i32, -2, -1, &shared))
        return nullptr;
    if (cu_q.size[0] < 1) {
        PyErr_SetString(PyExc_ValueError, "cu_seq_lens_q must have num_seqs + 1 entries");
        return nullptr;
    }
    if (!fits32(cu_q.size[0], "the batch") || !exact(a[8], "cu_seq_lens_k", &dev, t_i32, cu_q.size[0], -1, &cu_k) ||
        !load_as(a[6], "block_table", &dev, t_i32, cu_q.size[0] - 1, 0, &table) ||
        !exact(a[12], "cu_groups", &dev, t_i32, shared.size[0] + 1, -1, &cu_g) || !as_int(a[9], &max_q) ||
        !as_int(a[10], &max_k) || !as_float(a[11], &scale) || !as_int(a[14], &max_group) || !as_int(a[15], &max_shared) ||
        !workspace_of(a[16], &dev, &ws, &ws_bytes) || !status_of(a[17], &dev, &status))
        return nullptr;
    return on_device(dev, [&](pa_stream_t s) {
        return c_cascade(out.ptr, q.ptr, dt, &c, static_cast<const int32_t*>(table.ptr), static_cast<int32_t>(table.size[1]),
                         static_cast<const int32_t*>(cu_q.ptr), static_cast<const int32_t*>(cu_k.ptr),
                         static_cast<int32_t>(cu_q.size[0] - 1), q.size[0], static_cast<int32_t>(max_q),
                         static_cast<int32_t>(max_k), static_cast<int32_t>(q.size[1]), scale,
                         static_cast<const int32_t*>(cu_g.ptr), static_cast<const int32_t*>(shared.ptr),
                         static_cast<int32_t>(shared.size[0]), static_cast<int32_t>(max_group),
                         static_cast<int32_t>(max_shared), ws, static_cast<size_t>(ws_bytes), status, s);
    });
}

// (scores_out, rows_out, tokens_out, logits, scores, cu_beams, allowed, ended, end_token, workspace, dev_status)
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t dev = -1, stride[4], end_token, ws_bytes;
    Tensor x, scores, cu, so, ro, to, allowed{}, ended{};
    int32_t* status;
    void* ws;
    if (!count(n, 11) || !load(a[3], "logits", &dev, &x, stride)) return nullptr;
    pa_dtype dt;
    if (x.dtype == t_f32) dt = PA_F32;
    else if (x.dtype == t_f16) dt = PA_F16;
    else if (x.dtype == t_bf16) dt = PA_BF16;
    else {
        PyErr_Format(PyExc_TypeError, "unsupported dtype %R", x.dtype);
        return nullptr;
    }
    if (x.dim != 2 || (x.size[1] > 1 && stride[1] != 1)) {
        PyErr_SetString(PyExc_ValueError, "logits must be [num_rows, vocab], the tokens of a row contiguous");
        return nullptr;
    }
    const int64_t R = x.size[0], V = x.size[1], words = (V + 31) / 32;
    if (!fits32(R, "num_rows") || !fits32(V, "vocab") || !exact(a[5], "cu_beams", &dev, t_i32, -2, -1, &cu)) return nullptr;
    const int64_t B = cu.size[0] - 1;
    if (B < 0 || !fits32(B, "num_requests")) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "cu_beams must have num_requests + 1 entries");
        return nullptr;
    }
    if (!load(a[0], "scores_out", &dev, &so)) return nullptr;
    if (so.dim != 2) {
        PyErr_SetString(PyExc_ValueError, "scores_out must be [num_requests, num_select]");
        return nullptr;
    }
    const int64_t K = so.size[1];
    if (!fits32(K, "num_select") || !exact(a[0], "scores_out", &dev, t_f32, B, K, &so) ||
        !exact(a[1], "rows_out", &dev, t_i32, B, K, &ro) || !exact(a[2], "tokens_out", &dev, t_i32, B, K, &to) ||
        !exact(a[4], "scores", &dev, t_f32, R, -1, &scores) ||
        (a[6] != Py_None && !exact(a[6], "allowed", &dev, t_i32, R, words, &allowed)) || !as_int(a[8], &end_token) ||
        !workspace_of(a[9], &dev, &ws, &ws_bytes) || !status_of(a[10], &dev, &status))
        return nullptr;
    if (a[7] != Py_None) {
        if (!load(a[7], "ended", &dev, &ended)) return nullptr;
        if (ended.dtype != t_u8 && ended.dtype != t_bool) {
            PyErr_SetString(PyExc_TypeError, "ended must be uint8 or bool");
            return nullptr;
        }
        if (ended.dim != 1 || ended.size[0] != R) {
            PyErr_SetString(PyExc_ValueError, "ended must have an entry for each row");
            return nullptr;
        }
    }
    return on_device(dev, [&](pa_stream_t s) {
        return c_select(static_cast<float*>(so.ptr), static_cast<int32_t*>(ro.ptr), static_cast<int32_t*>(to.ptr), x.ptr, dt,
                        R > 1 ? stride[0] : V, static_cast<int32_t>(V), static_cast<int32_t>(R),
                        static_cast<const float*>(scores.ptr), static_cast<const int32_t*>(cu.ptr), static_cast<int32_t>(B),
                        static_cast<const uint32_t*>(allowed.ptr), words, static_cast<const uint8_t*>(ended.ptr),
                        static_cast<int32_t>(end_token), static_cast<int32_t>(K), ws, static_cast<size_t>(ws_bytes), status,
                        s);
    });
}

// (address of the layers' pa_kv_cache array, their number, the first layer's k_cache, parents, block_table, seq_lens,
// spare_blocks, block_table_out, seq_lens_out, slot_mapping_out, spare_used_out, dev_status)
PyObject* beam_reorder(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int64_t dev = -1, layers;
    Tensor k, parents, table, lens, spare, t2, l2, slots, used;
    int32_t* status;
    if (!count(n, 12)) return nullptr;
    const auto* caches = static_cast<const pa_kv_cache*>(PyLong_AsVoidPtr(a[0]));
    if (caches == nullptr) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no layers");
        return nullptr;
    }
    if (!as_int(a[1], &layers) || !load(a[2], "k_cache", &dev, &k) ||
        !exact(a[3], "parents", &dev, t_i32, -2, -1, &parents) || !load(a[4], "block_table", &dev, &table))
        return nullptr;
    if (table.dim != 2 || table.dtype != t_i32) {
        PyErr_SetString(table.dim != 2 ? PyExc_ValueError : PyExc_TypeError, "block_table must be int32 [rows, max_blocks]");
        return nullptr;
    }
    const int64_t m = parents.size[0], rows = table.size[0], width = table.size[1];
    if (!fits32(m, "num_rows") || !fits32(rows, "num_rows_in") || !fits32(width, "max_blocks") ||
        !exact(a[5], "seq_lens", &dev, t_i32, rows, -1, &lens) || !exact(a[6], "spare_blocks", &dev, t_i32, m, -1, &spare) ||
        !exact(a[7], "block_table_out", &dev, t_i32, m, width, &t2) || !exact(a[8], "seq_lens_out", &dev, t_i32, m, -1, &l2) ||
        !exact(a[9], "slot_mapping_out", &dev, t_i64, m, -1, &slots) ||
        !exact(a[10], "spare_used_out", &dev, t_i32, m, -1, &used) || !status_of(a[11], &dev, &status))
        return nullptr;
    return on_device(dev, [&](pa_stream_t s) {
        return c_reorder(caches, static_cast<int32_t>(layers), static_cast<const int32_t*>(parents.ptr),
                         static_cast<int32_t>(m), static_cast<const int32_t*>(table.ptr), static_cast<int32_t>(rows),
                         static_cast<int32_t>(width), static_cast<const int32_t*>(lens.ptr),
                         static_cast<const int32_t*>(spare.ptr), static_cast<int32_t*>(t2.ptr), static_cast<int32_t*>(l2.ptr),
                         static_cast<int64_t*>(slots.ptr), static_cast<int32_t*>(used.ptr), status, s);
    });
}

// setup_beams(uint8, bool; addresses of pa_varlen_cascade, pa_beam_select, pa_beam_reorder), after setup()
PyObject* setup_beams(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 5)) return nullptr;
    void* f[3];
    for (int i = 0; i < 3; ++i) {
        f[i] = PyLong_AsVoidPtr(a[2 + i]);
        if (f[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function's address is missing");
            return nullptr;
        }
    }
    t_u8 = Py_NewRef(a[0]);
    t_bool = Py_NewRef(a[1]);
    c_cascade = reinterpret_cast<decltype(c_cascade)>(f[0]);
    c_select = reinterpret_cast<decltype(c_select)>(f[1]);
    c_reorder = reinterpret_cast<decltype(c_reorder)>(f[2]);
    Py_RETURN_NONE;
}

// setup(dtypes: float16, bfloat16, float8_e4m3fn, int32, int64, float32; get_device, set_device, get_stream;
// addresses of pa_qk_norm_rope, pa_qk_norm_rope_write, pa_decode_window, pa_prefill_varlen_window)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 13)) return nullptr;
    PyObject** keep[9] = {&t_f16, &t_bf16, &t_e4m3, &t_i32, &t_i64, &t_f32, &f_get_device, &f_set_device, &f_stream};
    for (int i = 0; i < 9; ++i) *keep[i] = Py_NewRef(a[i]);
    void* f[4];
    for (int i = 0; i < 4; ++i) {
        f[i] = PyLong_AsVoidPtr(a[9 + i]);
        if (f[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function's address is missing");
            return nullptr;
        }
    }
    c_rope = reinterpret_cast<decltype(c_rope)>(f[0]);
    c_write = reinterpret_cast<decltype(c_write)>(f[1]);
    c_decode = reinterpret_cast<decltype(c_decode)>(f[2]);
    c_prefill = reinterpret_cast<decltype(c_prefill)>(f[3]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* ready(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (c_rope == nullptr) {
        PyErr_SetString(PyExc_RuntimeError, "setup() has not been called");
        return nullptr;
    }
    return F(self, a, n);
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* beams_ready(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (c_rope == nullptr || c_cascade == nullptr) {
        PyErr_SetString(PyExc_RuntimeError, "setup() and setup_beams() have not been called");
        return nullptr;
    }
    return F(self, a, n);
}

#define PA_METHOD(NAME, F) {NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_METHOD("setup", setup),
                         PA_METHOD("qk_norm_rope", ready<qk_norm_rope>),
                         PA_METHOD("qk_norm_rope_write", ready<qk_norm_rope_write>),
                         PA_METHOD("decode_window", ready<decode_window>),
                         PA_METHOD("prefill_varlen_window", ready<prefill_varlen_window>),
                         PA_METHOD("setup_beams", setup_beams),
                         PA_METHOD("varlen_cascade", beams_ready<varlen_cascade>),
                         PA_METHOD("beam_select", beams_ready<beam_select>),
                         PA_METHOD("beam_reorder", beams_ready<beam_reorder>),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() {
    const struct {
        PyObject** to;
        const char* name;
    } names[] = {{&n_shape, "shape"},       {&n_dtype, "dtype"},     {&n_get_device, "get_device"},
                 {&n_is_contiguous, "is_contiguous"}, {&n_data_ptr, "data_ptr"}, {&n_stride, "stride"},
                 {&n_numel, "numel"},       {&n_element_size, "element_size"}};
    for (const auto& x : names) {
        *x.to = PyUnicode_InternFromString(x.name);
        if (*x.to == nullptr) return nullptr;
    }
    return PyModule_Create(&module);
}
