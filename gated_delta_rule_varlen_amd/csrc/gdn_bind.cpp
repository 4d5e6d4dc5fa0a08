// gdn_bind.cpp -- argument marshalling of the softmax-attention operators, the 4-bit cache and the block's norms as a
// CPython extension (_bind.so): from tensors to descriptors and addresses, with the checks of the Python binding's other
// functions.
//
// These operators are called once a layer and token, where the host's time per call is the operator's: one token's
// attention takes 6.2 us of it, and with the same checks in Python 11.6, more than the kernels of a small step.  The entry
// points of libgdn.so are handed in as addresses (connect), so nothing here is linked against it.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "gdn.h"

namespace {

decltype(&gdn_qk_norm_rope_varlen) rope_fn;
decltype(&gdn_attention_varlen) attention_fn;
decltype(&gdn_attention_prefix_varlen) prefix_fn;
decltype(&gdn_attention_workspace_bytes) workspace_fn, fp4_workspace_fn;
decltype(&gdn_cache_write_fp4_varlen) fp4_write_fn;
decltype(&gdn_cache_read_fp4_varlen) fp4_read_fn;
decltype(&gdn_attention_fp4_varlen) fp4_attention_fn;
decltype(&gdn_residual_norm) residual_fn;
decltype(&gdn_gated_norm) gated_fn;

int dtype_code(at::ScalarType t) {
    return t == at::kFloat ? GDN_F32 : t == at::kBFloat16 ? GDN_BF16 : t == at::kHalf ? GDN_F16 : -1;
}

// What a call's tensors have in common, and whether an argument was refused (the Python error is set then).
struct Call {
    int64_t D = 0;
    int dev = 0;
    at::ScalarType dtype = at::kFloat;
    bool failed = false;

    template <typename... A>
    void refuse(PyObject* type, const char* format, A... a) {
        if (!failed) PyErr_Format(type, format, a...);
        failed = true;
    }
    const at::Tensor* tensor(PyObject* o, const char* what) {
        if (failed) return nullptr;  // nothing may be asked of Python with an error set
        if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
        refuse(PyExc_TypeError, "%s must be a tensor", what);
        return nullptr;
    }
    bool placed(const at::Tensor& t, at::ScalarType want, const char* what) {
        if (t.scalar_type() != want) {
            refuse(PyExc_TypeError, "%s must be %s, got %s", what, at::toString(want), at::toString(t.scalar_type()));
            return false;
        }
        if (!t.is_cuda() || t.get_device() != dev) {
            refuse(PyExc_ValueError, "%s must be on device cuda:%d", what, dev);
            return false;
        }
        return true;
    }
    // The queries say which device, type and head width the others have to have.
    const at::Tensor* queries(PyObject* o) { return leader(o, "q", 3); }
    // The tensor of `axes` axes that says so.
    const at::Tensor* leader(PyObject* o, const char* what, int axes) {
        const at::Tensor* q = tensor(o, what);
        if (q == nullptr) return nullptr;
        if (q->dim() != axes) {
            refuse(PyExc_ValueError, "%s must be %s, got %d axes", what, axes == 3 ? "[N, heads, D]" : "[N, C]", (int)q->dim());
        } else if (!q->is_cuda()) {
            refuse(PyExc_ValueError, "%s must be a device tensor", what);
        } else if (dtype_code(q->scalar_type()) < 0) {
            refuse(PyExc_TypeError, "%s: unsupported dtype %s", what, at::toString(q->scalar_type()));
        }
        if (failed) return nullptr;
        D = q->size(axes - 1);
        dev = q->get_device();
        dtype = q->scalar_type();
        return q;
    }
    // A [rows, heads, D] tensor with contiguous heads: its address, its strides into `stride` and its rows.
    struct Rows {
        void* p = nullptr;
        int64_t rows = 0;
    };
    Rows head_rows(const at::Tensor* t, int64_t heads, int64_t* stride, const char* what) {
        if (t == nullptr || !placed(*t, dtype, what)) return {};
        if (t->dim() != 3 || t->size(1) != heads || t->size(2) != D) {
            refuse(PyExc_ValueError, "%s must be [rows, %lld heads, %lld]", what, (long long)heads, (long long)D);
            return {};
        }
        if (t->stride(2) != 1 && D != 1) {
            refuse(PyExc_ValueError, "%s: the elements of a head must be contiguous", what);
            return {};
        }
        // the stride of an axis of one entry names nothing
        stride[0] = t->size(0) > 1 ? t->stride(0) : heads * D;
        stride[1] = heads > 1 ? t->stride(1) : D;
        return {t->data_ptr(), t->size(0)};
    }
    // Address of a contiguous vector of n entries; None is no vector.
    void* flat(PyObject* o, int64_t n, at::ScalarType want, const char* what) {
        if (o == Py_None) return nullptr;
        const at::Tensor* t = tensor(o, what);
        if (t == nullptr || !placed(*t, want, what)) return nullptr;
        if (t->numel() != n || !t->is_contiguous()) {
            refuse(PyExc_ValueError, "%s must be contiguous with %lld entries", what, (long long)n);
            return nullptr;
        }
        return t->data_ptr();
    }
    // A [N, width] tensor with contiguous rows: its address and its row stride.
    void* row_view(const at::Tensor* t, int64_t N, at::ScalarType want, int64_t* stride, const char* what) {
        if (t == nullptr || !placed(*t, want, what)) return nullptr;
        if (t->dim() != 2 || t->size(0) != N || t->size(1) != D || (D != 1 && t->stride(1) != 1)) {
            refuse(PyExc_ValueError, "%s must be [%lld, %lld] with contiguous rows", what, (long long)N, (long long)D);
            return nullptr;
        }
        *stride = N > 1 ? t->stride(0) : D;
        return t->data_ptr();
    }
    // The four tensors of a 4-bit cache of D elements a head; as many heads as the first one has.
    bool cache(PyObject* o, gdn_fp4_cache* to, int64_t* of_heads) {
        if (failed) return false;
        if (!(PyTuple_Check(o) || PyList_Check(o)) || PySequence_Fast_GET_SIZE(o) != 4) {
            refuse(PyExc_TypeError, "cache must be a tuple of four tensors: k_codes, k_scales, v_codes, v_scales");
        } else {
            static const char* const names[4] = {"cache: k_codes", "cache: k_scales", "cache: v_codes", "cache: v_scales"};
            void** const to_p[4] = {&to->k_codes, &to->k_scales, &to->v_codes, &to->v_scales};
            int64_t* const to_s[4] = {to->k_codes_stride, to->k_scales_stride, to->v_codes_stride, to->v_scales_stride};
            for (int i = 0; i < 4 && !failed; ++i) {
                const at::Tensor* t = tensor(PySequence_Fast_GET_ITEM(o, i), names[i]);
                if (t == nullptr || !placed(*t, at::kByte, names[i])) break;
                const int64_t width = i % 2 == 0 ? D / 2 : D / 32;
                if (i == 0) *of_heads = t->dim() == 3 ? t->size(1) : 0;
                const int64_t heads = *of_heads;
                if (t->dim() != 3 || t->size(1) != heads || t->size(2) != width || (i > 0 && t->size(0) != to->rows)) {
                    refuse(PyExc_ValueError, "%s must be [rows, %lld heads, %lld], with the same rows in all four", names[i],
                           (long long)heads, (long long)width);
                } else if (width != 1 && t->stride(2) != 1) {
                    refuse(PyExc_ValueError, "%s: the bytes of a head must be contiguous", names[i]);
                } else {
                    to->rows = t->size(0);
                    to_s[i][0] = t->size(0) > 1 ? t->stride(0) : heads * width;
                    to_s[i][1] = heads > 1 ? t->stride(1) : width;
                    *to_p[i] = t->data_ptr();
                }
            }
        }
        return !failed;
    }
    int32_t narrow(int64_t x, const char* what) {
        if (x < 0 || x > INT32_MAX) refuse(PyExc_ValueError, "%s does not fit 32 bits", what);
        return (int32_t)x;
    }
    void rows_are(bool same, const char* what) {
        if (!failed && !same) refuse(PyExc_ValueError, "%s", what);
    }
};

// A new tensor, as an object and to look at.
struct Made {
    PyObject* object;
    at::Tensor t;
    Made(PyObject* given, at::IntArrayRef shape, const at::Tensor& like, at::ScalarType dtype) {
        if (given != Py_None) {
            Py_INCREF(given);
            object = given;
        } else {
            t = at::empty(shape, like.options().dtype(dtype).requires_grad(false));
            object = THPVariable_Wrap(t);
        }
    }
    Made(const Made&) = delete;
    ~Made() { Py_XDECREF(object); }
    PyObject* release() {
        PyObject* o = object;
        object = nullptr;
        return o;
    }
};

hipStream_t stream_of(PyObject* o) { return reinterpret_cast<hipStream_t>(PyLong_AsVoidPtr(o)); }

// rope(q, k, v, offsets, inv_freq, q_weight, k_weight, eps, interleaved, past, positions, kv_begin, q_out, k_out, v_out,
//      dev_status, stream) -> (status, q_out, k_out, v_out)
PyObject* rope(PyObject*, PyObject* const* x, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != 17 || rope_fn == nullptr) {
        PyErr_SetString(PyExc_TypeError, "rope: 17 arguments, after connect");
        return nullptr;
    }
    Call c;
    const at::Tensor* q = c.queries(x[0]);
    const at::Tensor *k = c.tensor(x[1], "k"), *off = c.tensor(x[3], "offsets");
    const at::Tensor* freq = c.tensor(x[4], "inv_freq");
    if (!c.failed && k->dim() != 3) c.refuse(PyExc_ValueError, "k must be [N, heads, D]");
    if (c.failed) return nullptr;
    const bool has_v = x[2] != Py_None, paged = x[11] != Py_None;
    if (paged && (x[13] == Py_None || (has_v && x[14] == Py_None))) {
        PyErr_SetString(PyExc_ValueError, "k_out and v_out are required with kv_begin");
        return nullptr;
    }
    if (!has_v && x[14] != Py_None) {
        PyErr_SetString(PyExc_ValueError, "v_out without v");
        return nullptr;
    }
    gdn_rope_desc d{};
    const int64_t N = q->size(0), H = q->size(1), HK = k->size(1), B = off->numel() - 1;
    Made q_out(x[12], {N, H, c.D}, *q, c.dtype), k_out(x[13], {N, HK, c.D}, *q, c.dtype);
    Made v_out(has_v ? x[14] : Py_True, {N, HK, c.D}, *q, c.dtype);
    d.B = c.narrow(B, "B");
    d.N = c.narrow(N, "N");
    d.H = c.narrow(H, "H");
    d.HK = c.narrow(HK, "HK");
    d.D = c.narrow(c.D, "D");
    d.rot = c.narrow(2 * freq->numel(), "rot");
    d.dtype = dtype_code(c.dtype);
    d.flags = PyObject_IsTrue(x[8]) == 1 ? GDN_ROPE_INTERLEAVED : 0;
    d.eps = (float)PyFloat_AsDouble(x[7]);
    if (c.failed || PyErr_Occurred()) return nullptr;
    const auto qr = c.head_rows(q, H, d.q_stride, "q"), kr = c.head_rows(k, HK, d.k_stride, "k");
    const auto qo = c.head_rows(c.tensor(q_out.object, "q_out"), H, d.q_out_stride, "q_out");
    const auto ko = c.head_rows(c.tensor(k_out.object, "k_out"), HK, d.k_out_stride, "k_out");
    Call::Rows vr, vo;
    c.rows_are(kr.rows == N && qo.rows == N, "q, k and q_out must have one row per token");
    if (has_v) {
        vr = c.head_rows(c.tensor(x[2], "v"), HK, d.v_stride, "v");
        vo = c.head_rows(c.tensor(v_out.object, "v_out"), HK, d.v_out_stride, "v_out");
        c.rows_are(vr.rows == N && vo.rows == ko.rows, "v must have one row per token and v_out as many rows as k_out");
    }
    d.cache_rows = ko.rows;
    const auto inv_freq = (const float*)c.flat(x[4], freq->numel(), at::kFloat, "inv_freq");
    const auto q_weight = (const float*)c.flat(x[5], c.D, at::kFloat, "q_weight");
    const auto k_weight = (const float*)c.flat(x[6], c.D, at::kFloat, "k_weight");
    const auto offsets = (const int32_t*)c.flat(x[3], B + 1, at::kInt, "offsets");
    const auto past = (const int32_t*)c.flat(x[9], B, at::kInt, "past");
    const auto positions = (const int32_t*)c.flat(x[10], B, at::kInt, "positions");
    const auto kv_begin = (const int64_t*)c.flat(x[11], B, at::kLong, "kv_begin");
    const auto status = (int32_t*)c.flat(x[15], 1, at::kInt, "dev_status");
    const hipStream_t stream = stream_of(x[16]);
    if (c.failed || PyErr_Occurred()) return nullptr;
    const gdn_status st = rope_fn(&d, qr.p, kr.p, vr.p, inv_freq, q_weight, k_weight, offsets, past, positions, kv_begin,
                                  qo.p, ko.p, vo.p, status, stream);
    if (!has_v) {
        Py_DECREF(v_out.release());
        Py_INCREF(Py_None);
        v_out.object = Py_None;
    }
    return Py_BuildValue("iNNN", (int)st, q_out.release(), k_out.release(), v_out.release());
    END_HANDLE_TH_ERRORS
}

// attention(q, prefix_k, prefix_v, k, v, offsets, kv_len, kv_begin, max_q, scale, out, lse, return_lse, workspace,
//           dev_status, stream) -> (status, out, lse)
PyObject* attention(PyObject*, PyObject* const* x, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != 16 || attention_fn == nullptr) {
        PyErr_SetString(PyExc_TypeError, "attention: 16 arguments, after connect");
        return nullptr;
    }
    Call c;
    const at::Tensor* q = c.queries(x[0]);
    const at::Tensor *k = c.tensor(x[3], "k"), *v = c.tensor(x[4], "v"), *off = c.tensor(x[5], "offsets");
    if (!c.failed && k->dim() != 3) c.refuse(PyExc_ValueError, "k must be [rows, heads, D]");
    if (c.failed) return nullptr;
    gdn_attn_desc d{};
    const int64_t N = q->size(0), H = q->size(1), HK = k->size(1), B = off->numel() - 1;
    const bool prefix = x[1] != Py_None;
    d.B = c.narrow(B, "B");
    d.N = c.narrow(N, "N");
    d.H = c.narrow(H, "H");
    d.HK = c.narrow(HK, "HK");
    d.D = c.narrow(c.D, "D");
    d.dtype = dtype_code(c.dtype);
    if (x[8] == Py_None) {
        d.max_q = d.N;
    } else {
        const long long most = PyLong_AsLongLong(x[8]);
        if (most == -1 && PyErr_Occurred()) return nullptr;
        d.max_q = (int32_t)std::max(-1ll, std::min<long long>(most, N));
    }
    d.scale = (float)PyFloat_AsDouble(x[9]);
    if (c.failed || PyErr_Occurred()) return nullptr;
    const auto qr = c.head_rows(q, H, d.q_stride, "q");
    const auto kr = c.head_rows(k, HK, d.k_stride, "k"), vr = c.head_rows(v, HK, d.v_stride, "v");
    c.rows_are(kr.rows == vr.rows, "k and v must have the same rows");
    d.kv_rows = kr.rows;
    Call::Rows pk, pv;
    if (prefix) {
        pk = c.head_rows(c.tensor(x[1], "prefix_k"), HK, d.prefix_k_stride, "prefix_k");
        pv = c.head_rows(c.tensor(x[2], "prefix_v"), HK, d.prefix_v_stride, "prefix_v");
        c.rows_are(pk.rows == pv.rows, "prefix_k and prefix_v must have the same rows");
        d.prefix_len = c.narrow(pk.rows, "the prefix");
    }
    const auto offsets = (const int32_t*)c.flat(x[5], B + 1, at::kInt, "offsets");
    const auto kv_len = (const int32_t*)c.flat(x[6], B, at::kInt, "kv_len");
    const auto kv_begin = (const int64_t*)c.flat(x[7], B, at::kLong, "kv_begin");
    const auto status = (int32_t*)c.flat(x[14], 1, at::kInt, "dev_status");
    const hipStream_t stream = stream_of(x[15]);
    if (c.failed || PyErr_Occurred()) return nullptr;

    Made out(x[10], {N, H, c.D}, *q, c.dtype);
    const auto o = c.head_rows(c.tensor(out.object, "out"), H, d.out_stride, "out");
    c.rows_are(o.rows == N, "out must have one row per token");
    const int asked = PyObject_IsTrue(x[12]);
    if (c.failed || asked < 0) return nullptr;
    const bool with_lse = x[11] != Py_None || asked == 1;
    Made lse(with_lse ? x[11] : Py_True, {N, H}, *q, at::kFloat);
    auto stats = with_lse ? (float*)c.flat(lse.object, N * H, at::kFloat, "lse") : nullptr;
    at::Tensor scratch;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (x[13] != Py_None) {
        const at::Tensor* t = c.tensor(x[13], "workspace");
        if (t != nullptr && (!t->is_cuda() || t->get_device() != c.dev || !t->is_contiguous()))
            c.refuse(PyExc_ValueError, "workspace must be a contiguous tensor on device cuda:%d", c.dev);
        if (c.failed) return nullptr;
        ws = t->data_ptr();
        ws_bytes = t->nbytes();
    }
    if (c.failed) return nullptr;
    gdn_status st = GDN_OK;
    if (x[13] == Py_None && (st = workspace_fn(&d, &ws_bytes)) == GDN_OK && ws_bytes > 0) {
        scratch = at::empty({(int64_t)ws_bytes}, q->options().dtype(at::kByte).requires_grad(false));
        ws = scratch.data_ptr();
    }
    if (st == GDN_OK)
        st = prefix ? prefix_fn(&d, qr.p, pk.p, pv.p, kr.p, vr.p, offsets, kv_begin, kv_len, o.p, stats, ws, ws_bytes,
                                status, stream)
                    : attention_fn(&d, qr.p, kr.p, vr.p, offsets, kv_begin, kv_len, o.p, stats, ws, ws_bytes, status,
                                   stream);
    if (!with_lse) {
        Py_DECREF(lse.release());
        Py_INCREF(Py_None);
        lse.object = Py_None;
    }
    return Py_BuildValue("iNN", (int)st, out.release(), lse.release());
    END_HANDLE_TH_ERRORS
}

// fp4_rows(read, k, v, offsets, cache, past, kv_begin, dev_status, stream) -> status
PyObject* fp4_rows(PyObject*, PyObject* const* x, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != 9 || fp4_write_fn == nullptr) {
        PyErr_SetString(PyExc_TypeError, "fp4_rows: 9 arguments, after connect");
        return nullptr;
    }
    Call c;
    const bool read = x[0] == Py_True;
    const at::Tensor* k = c.leader(x[1], read ? "k_out" : "k", 3);
    const at::Tensor *v = c.tensor(x[2], read ? "v_out" : "v"), *off = c.tensor(x[3], "offsets");
    if (c.failed) return nullptr;
    gdn_fp4_rows_desc d{};
    gdn_fp4_cache cache{};
    const int64_t N = k->size(0), HK = k->size(1), B = off->numel() - 1;
    d.B = c.narrow(B, "B");
    d.N = c.narrow(N, "N");
    d.HK = c.narrow(HK, "HK");
    d.D = c.narrow(c.D, "D");
    d.dtype = dtype_code(c.dtype);
    const auto kr = c.head_rows(k, HK, d.k_stride, read ? "k_out" : "k"), vr = c.head_rows(v, HK, d.v_stride, read ? "v_out" : "v");
    c.rows_are(vr.rows == N, "k and v must have one row per token");
    int64_t heads = 0;
    if (!c.cache(x[4], &cache, &heads)) return nullptr;
    c.rows_are(heads == HK, "the cache must have as many heads as k and v");
    const auto offsets = (const int32_t*)c.flat(x[3], B + 1, at::kInt, "offsets");
    const auto past = (const int32_t*)c.flat(x[5], B, at::kInt, "past");
    const auto kv_begin = (const int64_t*)c.flat(x[6], B, at::kLong, "kv_begin");
    const auto status = (int32_t*)c.flat(x[7], 1, at::kInt, "dev_status");
    const hipStream_t stream = stream_of(x[8]);
    if (c.failed || PyErr_Occurred()) return nullptr;
    const c10::DeviceGuard on(k->device());
    return PyLong_FromLong(read ? fp4_read_fn(&d, &cache, offsets, past, kv_begin, kr.p, vr.p, status, stream)
                                : fp4_write_fn(&d, kr.p, vr.p, offsets, past, kv_begin, &cache, status, stream));
    END_HANDLE_TH_ERRORS
}

// fp4_read(cache, offsets, N, past, kv_begin, dtype, dev_status, stream) -> (status, k, v), with new k and v
PyObject* fp4_read(PyObject*, PyObject* const* x, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != 8 || fp4_read_fn == nullptr) {
        PyErr_SetString(PyExc_TypeError, "fp4_read: 8 arguments, after connect");
        return nullptr;
    }
    Call c;
    if (!(PyTuple_Check(x[0]) || PyList_Check(x[0])) || PySequence_Fast_GET_SIZE(x[0]) != 4)
        c.refuse(PyExc_TypeError, "cache must be a tuple of four tensors: k_codes, k_scales, v_codes, v_scales");
    const at::Tensor* codes = c.failed ? nullptr : c.tensor(PySequence_Fast_GET_ITEM(x[0], 0), "cache: k_codes");
    const at::Tensor* off = c.tensor(x[1], "offsets");
    if (!c.failed && (codes->dim() != 3 || !codes->is_cuda())) c.refuse(PyExc_ValueError, "cache: k_codes must be a device tensor [rows, heads, D/2]");
    if (!c.failed && !THPDtype_Check(x[5])) c.refuse(PyExc_TypeError, "dtype must be a torch.dtype");
    if (c.failed) return nullptr;
    c.dtype = reinterpret_cast<THPDtype*>(x[5])->scalar_type;
    c.dev = codes->get_device();
    c.D = 2 * codes->size(2);
    if (dtype_code(c.dtype) < 0) c.refuse(PyExc_TypeError, "dtype: unsupported dtype %s", at::toString(c.dtype));
    const int64_t N = PyLong_AsLongLong(x[2]), HK = codes->size(1), B = off->numel() - 1;
    if (c.failed || PyErr_Occurred()) return nullptr;
    gdn_fp4_rows_desc d{};
    gdn_fp4_cache cache{};
    int64_t heads = 0;
    d.B = c.narrow(B, "B");
    d.N = c.narrow(N, "N");
    d.HK = c.narrow(HK, "HK");
    d.D = c.narrow(c.D, "D");
    d.dtype = dtype_code(c.dtype);
    if (!c.cache(x[0], &cache, &heads)) return nullptr;
    const auto offsets = (const int32_t*)c.flat(x[1], B + 1, at::kInt, "offsets");
    const auto past = (const int32_t*)c.flat(x[3], B, at::kInt, "past");
    const auto kv_begin = (const int64_t*)c.flat(x[4], B, at::kLong, "kv_begin");
    const auto status = (int32_t*)c.flat(x[6], 1, at::kInt, "dev_status");
    const hipStream_t stream = stream_of(x[7]);
    if (c.failed || PyErr_Occurred()) return nullptr;
    const c10::DeviceGuard on(codes->device());
    Made k(Py_None, {N, HK, c.D}, *codes, c.dtype), v(Py_None, {N, HK, c.D}, *codes, c.dtype);
    for (int64_t* s : {d.k_stride, d.v_stride}) s[0] = HK * c.D, s[1] = c.D;
    const gdn_status st = fp4_read_fn(&d, &cache, offsets, past, kv_begin, k.t.data_ptr(), v.t.data_ptr(), status, stream);
    return Py_BuildValue("iNN", (int)st, k.release(), v.release());
    END_HANDLE_TH_ERRORS
}

// attention_fp4(q, cache, offsets, kv_len, kv_begin, max_q, scale, out, lse, return_lse, workspace, dev_status, stream)
//   -> (status, out, lse)
PyObject* attention_fp4(PyObject*, PyObject* const* x, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != 13 || fp4_attention_fn == nullptr) {
        PyErr_SetString(PyExc_TypeError, "attention_fp4: 13 arguments, after connect");
        return nullptr;
    }
    Call c;
    const at::Tensor *q = c.queries(x[0]), *off = c.tensor(x[2], "offsets");
    if (c.failed) return nullptr;
    gdn_attn_desc d{};
    gdn_fp4_cache cache{};
    const int64_t N = q->size(0), H = q->size(1), B = off->numel() - 1;
    int64_t HK = 0;
    if (!c.cache(x[1], &cache, &HK)) return nullptr;
    d.B = c.narrow(B, "B");
    d.N = c.narrow(N, "N");
    d.H = c.narrow(H, "H");
    d.HK = c.narrow(HK, "HK");
    d.D = c.narrow(c.D, "D");
    d.dtype = dtype_code(c.dtype);
    if (x[5] == Py_None) {
        d.max_q = d.N;
    } else {
        const long long most = PyLong_AsLongLong(x[5]);
        if (most == -1 && PyErr_Occurred()) return nullptr;
        d.max_q = (int32_t)std::max(-1ll, std::min<long long>(most, N));
    }
    d.scale = (float)PyFloat_AsDouble(x[6]);
    if (c.failed || PyErr_Occurred()) return nullptr;
    const auto qr = c.head_rows(q, H, d.q_stride, "q");
    d.kv_rows = cache.rows;
    const auto offsets = (const int32_t*)c.flat(x[2], B + 1, at::kInt, "offsets");
    const auto kv_len = (const int32_t*)c.flat(x[3], B, at::kInt, "kv_len");
    const auto kv_begin = (const int64_t*)c.flat(x[4], B, at::kLong, "kv_begin");
    const auto status = (int32_t*)c.flat(x[11], 1, at::kInt, "dev_status");
    const hipStream_t stream = stream_of(x[12]);
    const int asked = c.failed ? -1 : PyObject_IsTrue(x[9]);
    if (c.failed || asked < 0 || PyErr_Occurred()) return nullptr;

    const c10::DeviceGuard on(q->device());
    Made out(x[7], {N, H, c.D}, *q, c.dtype);
    const auto o = c.head_rows(c.tensor(out.object, "out"), H, d.out_stride, "out");
    c.rows_are(o.rows == N, "out must have one row per token");
    if (c.failed) return nullptr;
    const bool with_lse = x[8] != Py_None || asked == 1;
    Made lse(with_lse ? x[8] : Py_True, {N, H}, *q, at::kFloat);
    auto stats = with_lse ? (float*)c.flat(lse.object, N * H, at::kFloat, "lse") : nullptr;
    at::Tensor scratch;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (x[10] != Py_None) {
        const at::Tensor* t = c.tensor(x[10], "workspace");
        if (t != nullptr && (!t->is_cuda() || t->get_device() != c.dev || !t->is_contiguous()))
            c.refuse(PyExc_ValueError, "workspace must be a contiguous tensor on device cuda:%d", c.dev);
        if (c.failed) return nullptr;
        ws = t->data_ptr();
        ws_bytes = t->nbytes();
    }
    if (c.failed) return nullptr;
    gdn_status st = GDN_OK;
    if (x[10] == Py_None && (st = fp4_workspace_fn(&d, &ws_bytes)) == GDN_OK && ws_bytes > 0) {
        scratch = at::empty({(int64_t)ws_bytes}, q->options().dtype(at::kByte).requires_grad(false));
        ws = scratch.data_ptr();
    }
    if (st == GDN_OK)
        st = fp4_attention_fn(&d, qr.p, &cache, offsets, kv_begin, kv_len, o.p, stats, ws, ws_bytes, status, stream);
    if (!with_lse) {
        Py_DECREF(lse.release());
        Py_INCREF(Py_None);
        lse.object = Py_None;
    }
    return Py_BuildValue("iNN", (int)st, out.release(), lse.release());
    END_HANDLE_TH_ERRORS
}

// residual_norm(x, residual, weight, post_weight, scale, channel_scale, eps, out, residual_out, write_residual, stream)
//   -> (status, out, residual_out)
PyObject* residual_norm(PyObject*, PyObject* const* x, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != 11 || residual_fn == nullptr) {
        PyErr_SetString(PyExc_TypeError, "residual_norm: 11 arguments, after connect");
        return nullptr;
    }
    Call c;
    const at::Tensor* t = c.leader(x[0], "x", 2);
    const at::Tensor* r = x[1] != Py_None ? c.tensor(x[1], "residual") : nullptr;
    const at::Tensor* ro = x[8] != Py_None ? c.tensor(x[8], "residual_out") : nullptr;
    if (c.failed) return nullptr;
    gdn_residual_norm_desc d{};
    const int64_t N = t->size(0);
    const at::ScalarType stream_type = r != nullptr ? r->scalar_type() : ro != nullptr ? ro->scalar_type() : c.dtype;
    d.N = c.narrow(N, "N");
    d.C = c.narrow(c.D, "C");
    d.dtype = dtype_code(c.dtype);
    d.residual_dtype = dtype_code(stream_type);
    d.scale = (float)PyFloat_AsDouble(x[4]);
    d.eps = (float)PyFloat_AsDouble(x[6]);
    if (c.failed || PyErr_Occurred()) return nullptr;
    if (stream_type != c.dtype && stream_type != at::kFloat) c.refuse(PyExc_TypeError, "residual must be of x's type or float32");
    const int write = c.failed ? -1 : PyObject_IsTrue(x[9]);
    if (c.failed || write < 0) return nullptr;
    const auto xp = c.row_view(t, N, c.dtype, &d.x_stride, "x");
    const auto rp = r != nullptr ? c.row_view(r, N, stream_type, &d.residual_stride, "residual") : nullptr;
    const auto weight = (const float*)c.flat(x[2], c.D, at::kFloat, "weight");
    const auto post = (const float*)c.flat(x[3], c.D, at::kFloat, "post_weight");
    const auto channel = (const float*)c.flat(x[5], c.D, at::kFloat, "channel_scale");
    const hipStream_t stream = stream_of(x[10]);
    if (c.failed || PyErr_Occurred()) return nullptr;
    const c10::DeviceGuard on(t->device());
    const bool with_residual = ro != nullptr || write == 1;
    Made out(x[7], {N, c.D}, *t, c.dtype), next(with_residual ? x[8] : Py_True, {N, c.D}, *t, stream_type);
    const auto op = c.row_view(c.tensor(out.object, "out"), N, c.dtype, &d.out_stride, "out");
    const auto np = with_residual ? c.row_view(c.tensor(next.object, "residual_out"), N, stream_type, &d.residual_out_stride,
                                               "residual_out") : nullptr;
    if (c.failed) return nullptr;
    const gdn_status st = residual_fn(&d, xp, rp, post, channel, weight, op, np, stream);
    if (!with_residual) {
        Py_DECREF(next.release());
        Py_INCREF(Py_None);
        next.object = Py_None;
    }
    return Py_BuildValue("iNN", (int)st, out.release(), next.release());
    END_HANDLE_TH_ERRORS
}

// gated_norm(x, gate, weight, eps, flags, out, stream) -> (status, out)
PyObject* gated_norm(PyObject*, PyObject* const* x, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != 7 || gated_fn == nullptr) {
        PyErr_SetString(PyExc_TypeError, "gated_norm: 7 arguments, after connect");
        return nullptr;
    }
    Call c;
    const at::Tensor *t = c.leader(x[0], "x", 3), *z = c.tensor(x[1], "gate");
    if (c.failed) return nullptr;
    gdn_gated_norm_desc d{};
    const int64_t N = t->size(0), H = t->size(1);
    d.N = c.narrow(N, "N");
    d.H = c.narrow(H, "H");
    d.V = c.narrow(c.D, "V");
    d.dtype = dtype_code(c.dtype);
    d.eps = (float)PyFloat_AsDouble(x[3]);
    d.flags = (uint32_t)PyLong_AsUnsignedLong(x[4]);
    if (c.failed || PyErr_Occurred()) return nullptr;
    const auto xr = c.head_rows(t, H, d.x_stride, "x"), zr = c.head_rows(z, H, d.gate_stride, "gate");
    c.rows_are(zr.rows == N, "gate must have one row per token");
    const auto weight = (const float*)c.flat(x[2], c.D, at::kFloat, "weight");
    const hipStream_t stream = stream_of(x[6]);
    if (c.failed || PyErr_Occurred()) return nullptr;
    const c10::DeviceGuard on(t->device());
    Made out(x[5], {N, H, c.D}, *t, c.dtype);
    const auto o = c.head_rows(c.tensor(out.object, "out"), H, d.out_stride, "out");
    c.rows_are(o.rows == N, "out must have one row per token");
    if (c.failed) return nullptr;
    const gdn_status st = gated_fn(&d, xr.p, zr.p, weight, o.p, stream);
    return Py_BuildValue("iN", (int)st, out.release());
    END_HANDLE_TH_ERRORS
}

// connect(the addresses of libgdn.so's entry points): rope, attention, attention over a prefix, its workspace; cache write
// and read, attention over it, its workspace; residual norm, gated norm.
PyObject* connect(PyObject*, PyObject* args) {
    unsigned long long a[10];
    if (!PyArg_ParseTuple(args, "KKKKKKKKKK", a, a + 1, a + 2, a + 3, a + 4, a + 5, a + 6, a + 7, a + 8, a + 9)) return nullptr;
    auto set = [](auto& f, unsigned long long at) { f = reinterpret_cast<std::decay_t<decltype(f)>>((uintptr_t)at); };
    set(rope_fn, a[0]);
    set(attention_fn, a[1]);
    set(prefix_fn, a[2]);
    set(workspace_fn, a[3]);
    set(fp4_write_fn, a[4]);
    set(fp4_read_fn, a[5]);
    set(fp4_attention_fn, a[6]);
    set(fp4_workspace_fn, a[7]);
    set(residual_fn, a[8]);
    set(gated_fn, a[9]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, nullptr},
                         {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
                         {"fp4_rows", (PyCFunction)(void (*)(void))fp4_rows, METH_FASTCALL, nullptr},
                         {"fp4_read", (PyCFunction)(void (*)(void))fp4_read, METH_FASTCALL, nullptr},
                         {"attention_fp4", (PyCFunction)(void (*)(void))attention_fp4, METH_FASTCALL, nullptr},
                         {"residual_norm", (PyCFunction)(void (*)(void))residual_norm, METH_FASTCALL, nullptr},
                         {"gated_norm", (PyCFunction)(void (*)(void))gated_norm, METH_FASTCALL, nullptr},
                         {"connect", connect, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&module); }
