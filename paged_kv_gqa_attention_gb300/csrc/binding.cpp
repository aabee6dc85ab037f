// Python binding of the rotary-position and 4-bit-cache calls: reads torch
// tensors, checks them and passes addresses, sizes and the current stream to
// the qa_* entry point of the same name (qa.h).
//
// These calls are made once a layer and token, and a small one's kernel is
// done in 2 to 7 us.  Marshalled in Python, eight tensors' attributes, the
// structs and the ctypes call take 13 to 18 us on a Grace core; here a call
// takes about 4, most of it the launch.  Nothing of a call's arguments is
// kept for the next one (the library keeps the frequency table of a thread's
// last rope theta, rope.cu).
//
// A function returns its outputs, or the status as an int where the call was
// refused.  Arguments of the wrong kind raise TypeError or ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/core/Stream.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <optional>

#include "qa.h"

namespace {

constexpr int64_t kHeadBytes = 1280;  // one KV head of a 4-bit page

struct ArgError {
    PyObject *type;
    char text[256];
};

[[noreturn]] void refuse(PyObject *type, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
[[noreturn]] void refuse(PyObject *type, const char *fmt, ...) {
    ArgError e;
    e.type = type;
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(e.text, sizeof e.text, fmt, ap);
    va_end(ap);
    throw e;
}

int current_device() {  // -1 without a GPU: every tensor is refused then
    c10::DeviceIndex device = -1;
    return c10::cuda::GetDevice(&device) == cudaSuccess ? (int)device : -1;
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

void on_device(const at::Tensor &t, const char *name, int device) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
    if (t.get_device() != device)
        refuse(PyExc_ValueError, "tensors must be on the current CUDA device (%d), %s is on device %d", device, name,
               (int)t.get_device());
}

// A contiguous tensor's address; host: page-locked host memory will do too.
void *address(const at::Tensor &t, const char *name, at::ScalarType type, int64_t ndim, int device, bool host = false) {
    if (!(host && t.is_cpu() && t.is_pinned())) on_device(t, name, device);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be torch.%s", name,
                                        type == at::kBFloat16 ? "bfloat16" : type == at::kInt ? "int32" : type == at::kByte ? "uint8" : "float32");
    if (t.dim() != ndim) refuse(PyExc_ValueError, "%s must have %d dims", name, (int)ndim);
    return t.data_ptr();
}

// A bf16 [rows, heads, head_dim] tensor whose rows are packed inside, but may
// lie apart (views into a fused projection's rows).
struct Rows {
    void *p;
    long long ld;
};
Rows rows(const at::Tensor &t, const char *name, int device) {
    on_device(t, name, device);
    if (t.scalar_type() != at::kBFloat16) refuse(PyExc_TypeError, "%s must be torch.bfloat16", name);
    if (t.dim() != 3) refuse(PyExc_ValueError, "%s must have 3 dims", name);
    const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
    if (n > 0 && (t.stride(2) != 1 || (h > 1 && t.stride(1) != d)))
        refuse(PyExc_ValueError, "%s must be contiguous within each row", name);
    if (n > 1 && t.stride(0) < h * d) refuse(PyExc_ValueError, "%s has rows that overlap", name);
    return {t.data_ptr(), n > 1 ? (long long)t.stride(0) : 0};
}

bool shape_is(const at::Tensor &t, int64_t a, int64_t b, int64_t c) {
    return t.dim() == 3 && t.size(0) == a && t.size(1) == b && t.size(2) == c;
}

int as_int(int64_t x, const char *name) {
    if (x < 0 || x > 0x7fffffff) refuse(PyExc_ValueError, "%s %lld is outside [0, 2^31)", name, (long long)x);
    return (int)x;
}

long as_long(PyObject *o, const char *name) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_TypeError, "%s must be an integer", name);
    }
    return x;
}

bool as_bool(PyObject *o, const char *name) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) {
        PyErr_Clear();
        refuse(PyExc_TypeError, "%s must be true or false", name);
    }
    return x;
}

double as_double(PyObject *o, const char *name) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_TypeError, "%s must be a number", name);
    }
    return x;
}

// The stream a call runs on: the current one, or the torch.cuda.Stream given.
// Buffers made inside a call are allocated (and zeroed, and later reused) in
// its order.
struct Stream {
    std::optional<c10::cuda::CUDAStream> given;
    void *raw;
};
Stream stream_of(PyObject *o, int device) {
    Stream s;
    if (o == Py_None) {
        s.raw = c10::cuda::getCurrentCUDAStream(device).stream();
        return s;
    }
    long long part[3];
    const char *const names[3] = {"stream_id", "device_index", "device_type"};
    for (int i = 0; i < 3; ++i) {
        PyObject *v = PyObject_GetAttrString(o, names[i]);
        part[i] = v ? PyLong_AsLongLong(v) : 0;
        Py_XDECREF(v);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            refuse(PyExc_TypeError, "stream must be a torch.cuda.Stream");
        }
    }
    if (part[1] != device) refuse(PyExc_ValueError, "stream must be of the current CUDA device (%d)", device);
    s.given = c10::cuda::CUDAStream::unpack3(part[0], (c10::DeviceIndex)part[1], (c10::DeviceType)part[2]);
    s.raw = s.given->stream();
    return s;
}
at::Tensor made(const Stream &s, at::IntArrayRef shape, at::ScalarType type, int device, bool zeros = false) {
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    if (s.given) guard.emplace(*s.given);
    const c10::Device where(c10::kCUDA, (c10::DeviceIndex)device);
    if (zeros) return at::zeros(shape, at::TensorOptions().dtype(type).device(where));
    return at::Tensor(at::detail::empty_cuda(shape, type, where, std::nullopt));  // past the dispatcher: half the time
}

qa_attn_params params_of(int64_t hq, int64_t hkv, int64_t d, int64_t pages, int64_t width, double scale, void *stream,
                         PyObject *debug, PyObject *stable) {
    qa_attn_params p = qa_attn_default_params();
    p.n_q_heads = as_int(hq, "n_q_heads");
    p.n_kv_heads = as_int(hkv, "n_kv_heads");
    p.head_dim = as_int(d, "head_dim");
    p.num_pages = as_int(pages, "num_pages");
    p.max_pages_per_seq = as_int(width, "max_pages");
    p.scale = (float)scale;
    p.stream = stream;
    p.debug_checks = as_bool(debug, "debug_checks") ? 1 : 0;
    p.stable_metadata = as_int(as_long(stable, "stable_metadata"), "stable_metadata");
    return p;
}

// The qa_rope struct; `axes` holds what its pair_axis points to.
struct Rope {
    qa_rope r;
    uint8_t axes[64];
};
void rope_of(Rope &out, PyObject *positions, int64_t n_rows, PyObject *q_gain, PyObject *k_gain, PyObject *pair_axis, int64_t d,
             PyObject *eps, PyObject *theta, int device) {
    qa_rope &r = out.r;
    std::memset(&r, 0, sizeof r);
    const auto gain = [&](PyObject *o, const char *name) -> const float * {
        if (o == Py_None) return nullptr;
        const at::Tensor &t = tensor(o, name);
        const float *p = static_cast<const float *>(address(t, name, at::kFloat, 1, device));
        if (t.size(0) != d) refuse(PyExc_ValueError, "gains must be [head_dim]");
        return p;
    };
    r.q_gain = gain(q_gain, "q_gain");
    r.k_gain = gain(k_gain, "k_gain");
    r.rms_eps = (float)as_double(eps, "rms_eps");
    r.theta = (float)as_double(theta, "rope_theta");
    r.n_axes = 1;
    if (positions != Py_None) {
        const at::Tensor &t = tensor(positions, "positions");
        if ((t.dim() != 1 && t.dim() != 2) || t.size(t.dim() - 1) != n_rows)
            refuse(PyExc_ValueError, "positions must be [rows] or [n_axes, rows] with %lld rows", (long long)n_rows);
        r.positions = static_cast<const int32_t *>(address(t, "positions", at::kInt, t.dim(), device));
        if (t.dim() == 2) r.n_axes = as_int(t.size(0), "n_axes");
    }
    if (pair_axis == Py_None) return;
    const char *const what = "pair_axis must be head_dim / 2 integers";
    if (d / 2 > (int64_t)sizeof out.axes) refuse(PyExc_ValueError, "%s", what);
    Py_buffer view;
    if (PyObject_CheckBuffer(pair_axis) && PyObject_GetBuffer(pair_axis, &view, PyBUF_SIMPLE) == 0) {
        const bool bytes = view.itemsize == 1 && view.len == d / 2;
        if (bytes) std::memcpy(out.axes, view.buf, (size_t)view.len);
        const bool wrong = view.itemsize == 1 && !bytes;
        PyBuffer_Release(&view);
        if (wrong) refuse(PyExc_ValueError, "%s", what);
        if (bytes) {
            r.pair_axis = out.axes;
            return;
        }
    }
    PyErr_Clear();
    PyObject *seq = PySequence_Fast(pair_axis, what);
    if (!seq) {
        PyErr_Clear();
        refuse(PyExc_TypeError, "%s", what);
    }
    bool ok = PySequence_Fast_GET_SIZE(seq) == d / 2;
    for (Py_ssize_t i = 0; ok && i < d / 2; ++i) {
        const long x = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
        if (x < 0 || x > 255) ok = false;  // an error too
        else out.axes[i] = (uint8_t)x;
    }
    PyErr_Clear();
    Py_DECREF(seq);
    if (!ok) refuse(PyExc_ValueError, "%s", what);
    r.pair_axis = out.axes;
}

// A qa_* call, with other Python threads running meanwhile: a launch waits
// where the stream's queue is full, and a checked call for the GPU.  Nothing
// in it may throw, so arguments are checked before.
template <typename F>
qa_status call(F f) {
    qa_status st;
    static_assert(noexcept(f()), "an exception would leave the interpreter's lock released");
    Py_BEGIN_ALLOW_THREADS st = f();
    Py_END_ALLOW_THREADS return st;
}

// An output's Python object: the one that was given, or a new one.
PyObject *object_of(PyObject *given, at::Tensor &&made) {
    return given != Py_None ? Py_NewRef(given) : THPVariable_Wrap(std::move(made));
}
PyObject *pair_of(PyObject *a, PyObject *b) {
    PyObject *t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return t;
}

// (q, k, positions, q_out, k_out, q_gain, k_gain, rms_eps, rope_theta, pair_axis, stream, debug_checks, stable_metadata)
PyObject *rope_rows(PyObject *const *a) {
    const int device = current_device();
    const at::Tensor &q = tensor(a[0], "q");
    const Rows rq = rows(q, "q", device);
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    if (a[2] == Py_None) refuse(PyExc_ValueError, "positions are required");
    const Stream s = stream_of(a[10], device);
    at::Tensor q_made, k_made;
    Rows ro, rk = {nullptr, 0}, rko = {nullptr, 0};
    if (a[3] == Py_None) {
        q_made = made(s, {T, Hq, D}, at::kBFloat16, device);
        ro = {q_made.data_ptr(), 0};
    } else {
        const at::Tensor &t = tensor(a[3], "q_out");
        ro = rows(t, "q_out", device);
        if (!shape_is(t, T, Hq, D)) refuse(PyExc_ValueError, "outputs must have their inputs' shapes");
    }
    int64_t Hkv = 1;
    if (a[1] != Py_None) {
        const at::Tensor &k = tensor(a[1], "k");
        rk = rows(k, "k", device);
        Hkv = k.size(1);
        if (!shape_is(k, T, Hkv, D)) refuse(PyExc_ValueError, "inconsistent rope shapes");
        if (a[4] == Py_None) {
            k_made = made(s, {T, Hkv, D}, at::kBFloat16, device);
            rko = {k_made.data_ptr(), 0};
        } else {
            const at::Tensor &t = tensor(a[4], "k_out");
            rko = rows(t, "k_out", device);
            if (!shape_is(t, T, Hkv, D)) refuse(PyExc_ValueError, "outputs must have their inputs' shapes");
        }
    }
    Rope r;
    rope_of(r, a[2], T, a[5], a[6], a[9], D, a[7], a[8], device);
    const qa_attn_params p = params_of(Hq, Hkv, D, 0, 0, 0.0, s.raw, a[11], a[12]);
    const int n = as_int(T, "rows");
    const qa_status st = call([&]() noexcept {
        return qa_rope_rows(rq.p, rq.ld, rk.p, rk.ld, n, ro.p, ro.ld, rko.p, rko.ld, &r.r, &p);
    });
    if (st != QA_STATUS_OK) return PyLong_FromLong(st);
    return pair_of(object_of(a[3], std::move(q_made)),
                   a[1] == Py_None ? Py_NewRef(a[4]) : object_of(a[4], std::move(k_made)));
}

struct Pools {
    void *k, *v;
    int64_t pages, hkv;
};
Pools pools_of(PyObject *ko, PyObject *vo, int device) {
    const at::Tensor &k = tensor(ko, "k_pages"), &v = tensor(vo, "v_pages");
    if (k.dim() != 2 || v.dim() != 2 || k.size(1) == 0 || k.size(1) % kHeadBytes || k.sizes() != v.sizes())
        refuse(PyExc_ValueError, "4-bit pools must be uint8 [num_pages, qa_kvq_page_bytes(n_kv_heads)], of one shape");
    return {address(k, "k_pages", at::kByte, 2, device), address(v, "v_pages", at::kByte, 2, device), k.size(0),
            k.size(1) / kHeadBytes};
}

// What says which rows of which requests lie where.
struct RowArgs {
    const int32_t *cu, *past, *table;
    int64_t batch, width;
};
RowArgs row_args(PyObject *cu_o, PyObject *past_o, PyObject *table_o, int device) {
    RowArgs r;
    const at::Tensor &cu = tensor(cu_o, "cu_seqlens"), &table = tensor(table_o, "page_table");
    r.cu = static_cast<const int32_t *>(address(cu, "cu_seqlens", at::kInt, 1, device));
    r.table = static_cast<const int32_t *>(address(table, "page_table", at::kInt, 2, device));
    r.batch = table.size(0), r.width = table.size(1);
    r.past = nullptr;
    bool fits = cu.size(0) == r.batch + 1;
    if (past_o != Py_None) {
        const at::Tensor &past = tensor(past_o, "n_past");
        r.past = static_cast<const int32_t *>(address(past, "n_past", at::kInt, 1, device));
        fits = fits && past.size(0) == r.batch;
    }
    if (!fits) refuse(PyExc_ValueError, "page_table must be [batch, max_pages], cu_seqlens [batch + 1] and n_past [batch]");
    return r;
}

// (k, v, cu_seqlens, page_table, k_pages, v_pages, n_past, stream, debug_checks, stable_metadata)
PyObject *kvq_write(PyObject *const *a) {
    const int device = current_device();
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const Pools pools = pools_of(a[4], a[5], device);
    const Rows rk = rows(k, "k", device), rv = rows(v, "v", device);
    if (k.sizes() != v.sizes() || k.size(1) != pools.hkv) refuse(PyExc_ValueError, "inconsistent 4-bit write shapes");
    const RowArgs r = row_args(a[2], a[6], a[3], device);
    const Stream s = stream_of(a[7], device);
    const qa_attn_params p = params_of(pools.hkv, pools.hkv, k.size(2), pools.pages, r.width, 0.0, s.raw, a[8], a[9]);
    const int T = as_int(k.size(0), "total_tokens"), batch = as_int(r.batch, "batch");
    const qa_status st = call([&]() noexcept {
        return qa_kvq_write(rk.p, rk.ld, rv.p, rv.ld, r.cu, r.past, batch, T, r.table, pools.k, pools.v, &p);
    });
    if (st != QA_STATUS_OK) return PyLong_FromLong(st);
    Py_RETURN_NONE;
}

// (k_pages, v_pages, page_table, cu_seqlens, total_tokens, k_out, v_out, n_past, stream, debug_checks, stable_metadata)
PyObject *kvq_read(PyObject *const *a) {
    const int device = current_device();
    const Pools pools = pools_of(a[0], a[1], device);
    const RowArgs r = row_args(a[3], a[7], a[2], device);
    const int T = as_int(as_long(a[4], "total_tokens"), "total_tokens");
    const Stream s = stream_of(a[8], device);
    at::Tensor buf[2];
    void *out[2];
    for (int i = 0; i < 2; ++i) {
        const char *name = i ? "v_out" : "k_out";
        if (a[5 + i] == Py_None) {
            buf[i] = made(s, {T, pools.hkv, 128}, at::kBFloat16, device);
            out[i] = buf[i].data_ptr();
        } else {
            const at::Tensor &t = tensor(a[5 + i], name);
            out[i] = address(t, name, at::kBFloat16, 3, device);
            if (!shape_is(t, T, pools.hkv, 128)) refuse(PyExc_ValueError, "k_out and v_out must be [total_tokens, n_kv_heads, 128]");
        }
    }
    const qa_attn_params p = params_of(pools.hkv, pools.hkv, 128, pools.pages, r.width, 0.0, s.raw, a[9], a[10]);
    const int batch = as_int(r.batch, "batch");
    const qa_status st = call([&]() noexcept {
        return qa_kvq_read(pools.k, pools.v, r.table, r.cu, r.past, batch, T, out[0], out[1], &p);
    });
    if (st != QA_STATUS_OK) return PyLong_FromLong(st);
    return pair_of(object_of(a[5], std::move(buf[0])), object_of(a[6], std::move(buf[1])));
}

// (q, k_pages, v_pages, page_table, seq_lens, out, workspace, scale, stream, debug_checks, stable_metadata), and for the
// step also (k, v, q_gain, k_gain, positions, pair_axis, rms_eps, rope_theta)
PyObject *decode(PyObject *const *a, bool step) {
    const int device = current_device();
    const at::Tensor &q = tensor(a[0], "q");
    if (q.dim() != 3) refuse(PyExc_ValueError, "q must have 3 dims");
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
    const Pools pools = pools_of(a[1], a[2], device);
    const at::Tensor &table = tensor(a[3], "page_table"), &lens = tensor(a[4], "seq_lens");
    const int32_t *tp = static_cast<const int32_t *>(address(table, "page_table", at::kInt, 2, device, true));
    const int32_t *lp = static_cast<const int32_t *>(address(lens, "seq_lens", at::kInt, 1, device, true));
    if (table.size(0) != B || lens.size(0) != B) refuse(PyExc_ValueError, "inconsistent decode shapes");
    const Stream s = stream_of(a[8], device);
    at::Tensor out_made, ws_made;
    void *out;
    if (a[5] == Py_None) {
        out_made = made(s, {B, Hq, D}, at::kBFloat16, device);
        out = out_made.data_ptr();
    } else {
        const at::Tensor &t = tensor(a[5], "out");
        out = address(t, "out", at::kBFloat16, 3, device, true);
        if (!shape_is(t, B, Hq, D)) refuse(PyExc_ValueError, "out must have q's shape");
    }
    qa_attn_params p = params_of(Hq, pools.hkv, D, pools.pages, table.size(1), as_double(a[7], "scale"), s.raw, a[9], a[10]);
    const int batch = as_int(B, "batch");
    if (a[6] == Py_None) {
        const size_t need = qa_kvq_decode_workspace_size(batch, 0, &p);
        if (!need) return PyLong_FromLong(QA_STATUS_INVALID_PARAMS);
        ws_made = made(s, {(int64_t)need}, at::kByte, device, true);
        p.workspace = ws_made.data_ptr();
        p.workspace_bytes = need;
    } else {
        const at::Tensor &t = tensor(a[6], "workspace");
        on_device(t, "workspace", device);
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
        p.workspace = t.data_ptr();
        p.workspace_bytes = (size_t)t.nbytes();
    }
    qa_status st;
    if (!step) {
        const void *qp = address(q, "q", at::kBFloat16, 3, device, true);
        st = call([&]() noexcept { return qa_kvq_decode_attn(qp, pools.k, pools.v, tp, lp, batch, out, &p); });
    } else {
        const at::Tensor &k = tensor(a[11], "k"), &v = tensor(a[12], "v");
        const Rows rq = rows(q, "q", device), rk = rows(k, "k", device), rv = rows(v, "v", device);
        if (!shape_is(k, B, pools.hkv, D) || !shape_is(v, B, pools.hkv, D)) refuse(PyExc_ValueError, "inconsistent decode-step shapes");
        const long long width = pools.hkv * D;
        if ((rk.ld ? rk.ld : width) != (rv.ld ? rv.ld : width)) refuse(PyExc_ValueError, "k and v must have the same row stride");
        Rope r;
        rope_of(r, a[15], B, a[13], a[14], a[16], D, a[17], a[18], device);
        st = call([&]() noexcept { return qa_kvq_decode_step(rq.p, rq.ld, rk.p, rv.p, rk.ld, &r.r, pools.k, pools.v, tp, lp, batch, out, &p); });
    }
    if (st != QA_STATUS_OK) return PyLong_FromLong(st);
    return object_of(a[5], std::move(out_made));
}
PyObject *kvq_decode_attn(PyObject *const *a) { return decode(a, false); }
PyObject *kvq_decode_step(PyObject *const *a) { return decode(a, true); }

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const ArgError &e) {
        PyErr_SetString(e.type, e.text);
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(rope_rows, 13), ENTRY(kvq_write, 10), ENTRY(kvq_read, 11), ENTRY(kvq_decode_attn, 11),
                         ENTRY(kvq_decode_step, 19), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
