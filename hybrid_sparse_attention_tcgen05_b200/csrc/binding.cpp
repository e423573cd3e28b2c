// Native half of the Python binding of the calls over ragged batches and
// paged caches (ragged.py): checks the torch tensors, allocates what the
// caller left out and calls the C ABI on the tensors' device and that
// device's current stream.  A decode step makes several of these calls for a
// few microseconds of work each; from Python through ctypes the checks and
// conversions took longer than the launch.
//
// Positional arguments only, in the order that ragged.py passes them.  The
// library is the one that _lib.py has loaded: bind() gets the addresses.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <climits>

#include "hysparse.h"

namespace {

PyObject *g_check = nullptr;   // check(status, call): raises for a status that is not ok
decltype(&hysparse_rope) g_rope = nullptr;
decltype(&hysparse_cache_write) g_cache_write = nullptr;
decltype(&hysparse_cache_read) g_cache_read = nullptr;
decltype(&hysparse_ragged_workspace_size) g_workspace_size = nullptr;
decltype(&hysparse_packed_attn) g_packed_attn = nullptr;
decltype(&hysparse_chunk_attn_paged) g_chunk_attn = nullptr;

at::Tensor tensor(PyObject *o, const char *what) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a tensor");
    return THPVariable_Unpack(o);
}
at::Tensor maybe_tensor(PyObject *o, const char *what) {
    return o == Py_None ? at::Tensor() : tensor(o, what);
}

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
int as_int(int64_t v, const char *what) {
    TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, what, " is out of range");
    return (int)v;
}

// The one CUDA device that all the tensors are on.
class Device {
  public:
    template <typename... Ts>
    explicit Device(const Ts &...ts) { (add(ts), ...); }
    void add(const at::Tensor &t) {
        if (!t.defined()) return;
        TORCH_CHECK_VALUE(t.is_cuda(), "hysparse runs on CUDA tensors only (no CPU path)");
        TORCH_CHECK_VALUE(index_ < 0 || t.get_device() == index_, "all tensors must be on the same device");
        index_ = t.get_device();
    }
    c10::DeviceIndex index() const { return (c10::DeviceIndex)index_; }

  private:
    int64_t index_ = -1;
};

const void *ptr(const at::Tensor &t) { return t.defined() ? t.const_data_ptr() : nullptr; }
void *mut(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// A packed [T, H, d] tensor; ld: elements from one row to the next.
struct Rows {
    int T, H, d;
    long long ld;
};
Rows rows_of(const at::Tensor &t, const char *what) {
    TORCH_CHECK_VALUE(t.dim() == 3, what, " must be [T, H, d]");
    Rows r;
    r.T = as_int(t.size(0), what);
    r.H = as_int(t.size(1), what);
    r.d = as_int(t.size(2), what);
    TORCH_CHECK_VALUE(r.T == 0 || ((r.d <= 1 || t.stride(2) == 1) && (r.H <= 1 || t.stride(1) == r.d)), what,
                      ": the heads of a row must be contiguous");
    r.ld = r.T > 1 ? t.stride(0) : (long long)r.H * r.d;
    return r;
}

// `out` checked against t, or allocated.
at::Tensor like(const at::Tensor &out, const at::Tensor &t, const char *what) {
    if (!out.defined()) return at::empty(t.sizes(), t.options());
    TORCH_CHECK_VALUE(out.sizes() == t.sizes() && out.scalar_type() == t.scalar_type(), what);
    return out;
}

int code_of(at::ScalarType t) {
    TORCH_CHECK_TYPE(t == at::kFloat || t == at::kBFloat16, "unsupported dtype ", t);
    return t == at::kFloat ? HS_F32 : HS_BF16;
}

void dense(const at::Tensor &t, const char *what, at::ScalarType dtype, at::IntArrayRef shape) {
    if (!t.defined()) return;
    TORCH_CHECK_TYPE(t.scalar_type() == dtype, what, " must be ", dtype);
    TORCH_CHECK_VALUE(t.sizes() == shape, what, " must have shape ", shape);
    TORCH_CHECK_VALUE(t.is_contiguous(), what, " must be contiguous");
}

int rot_of(const at::Tensor &inv_freq, int d) {
    if (!inv_freq.defined()) return 0;
    TORCH_CHECK_TYPE(inv_freq.scalar_type() == at::kDouble && inv_freq.dim() == 1 && inv_freq.is_contiguous(),
                     "inv_freq must be a contiguous float64 vector");
    const int64_t rot = 2 * inv_freq.numel();
    TORCH_CHECK_VALUE(rot >= 2 && rot <= d, "inv_freq holds one angle per rotated pair: 1 to d / 2 of them");
    return (int)rot;
}

// The checked paged cache of these tensors; Hkv and d of its pages.
struct Pages {
    hs_paged_cache c{};
    int Hkv = 0, d = 0;
};
Pages pages_of(const at::Tensor &k, const at::Tensor &v, const at::Tensor &cu, const at::Tensor &kv_len,
               const at::Tensor &table, const at::Tensor &ks, const at::Tensor &vs) {
    TORCH_CHECK_VALUE(k.dim() == 4 && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type(),
                      "k_pages, v_pages: [num_pages, page_size, Hkv, d], alike");
    TORCH_CHECK_VALUE(k.is_contiguous() && v.is_contiguous(), "page pools must be contiguous");
    Pages p;
    p.c.cache_dtype = k.scalar_type() == at::kFloat8_e4m3fn ? (int)HS_E4M3 : code_of(k.scalar_type());
    TORCH_CHECK_TYPE(table.dim() == 2 && table.scalar_type() == at::kInt && table.is_contiguous(),
                     "block_table must be a contiguous int32 [B, max_pages]");
    p.c.B = as_int(table.size(0), "B");
    p.c.max_pages = as_int(table.size(1), "max_pages");
    p.c.num_pages = as_int(k.size(0), "num_pages");
    p.c.page_size = as_int(k.size(1), "page_size");
    p.Hkv = as_int(k.size(2), "Hkv");
    p.d = as_int(k.size(3), "d");
    dense(cu, "cu_seqlens", at::kInt, {table.size(0) + 1});
    dense(kv_len, "kv_len", at::kInt, {table.size(0)});
    if (p.c.cache_dtype == HS_E4M3) {
        TORCH_CHECK_VALUE(ks.defined() && vs.defined(), "8-bit pages need k_scale and v_scale");
        dense(ks, "k_scale", at::kByte, {k.size(0), k.size(2), k.size(1)});
        dense(vs, "v_scale", at::kByte, {k.size(0), k.size(2), k.size(1)});
    } else {
        TORCH_CHECK_VALUE(!ks.defined() && !vs.defined(), "k_scale and v_scale belong to 8-bit pages");
    }
    p.c.cu_rows = (const int32_t *)ptr(cu);
    p.c.kv_len = (const int32_t *)ptr(kv_len);
    p.c.block_table = (const int32_t *)ptr(table);
    p.c.k_pages = mut(k);
    p.c.v_pages = mut(v);
    p.c.k_scale = (uint8_t *)mut(ks);
    p.c.v_scale = (uint8_t *)mut(vs);
    return p;
}

void status_ws(const at::Tensor &ws) {
    TORCH_CHECK_VALUE(!ws.defined() || (ws.is_contiguous() && ws.nbytes() >= 256),
                      "ws must be contiguous and hold at least 256 bytes");
}

// Marks the caller's tensors as changed, as torch's own writes do, so that a
// backward pass that saved one of them raises instead of using what was written
// over it.  (Tensors made in inference mode keep no count of changes.)
template <typename... Ts> void changed(const Ts &...ts) {
    auto mark = [](const at::Tensor &t) {
        if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    };
    (mark(ts), ...);
}

// Runs call(stream) on the device and its current stream, without the
// interpreter's lock; false with the library's error raised.
template <typename F>
bool run(const Device &dev, const char *what, F call) {
    int st;
    {
        const c10::cuda::CUDAGuard guard(dev.index());
        hs_stream_t stream = (hs_stream_t)c10::cuda::getCurrentCUDAStream(dev.index()).stream();
        Py_BEGIN_ALLOW_THREADS;
        st = call(stream);
        Py_END_ALLOW_THREADS;
    }
    if (st == HS_OK) return true;
    Py_XDECREF(PyObject_CallFunction(g_check, "is", st, what));
    return false;
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b) {
    PyObject *t = PyTuple_New(2);
    if (t == nullptr) throw python_error();
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
    return t;
}

void need_args(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// rope(q, positions, inv_freq, k, interleaved, inverse, factor, out, out_k)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    need_args(n, 9);
    const at::Tensor q = tensor(a[0], "q"), positions = tensor(a[1], "positions"), f = tensor(a[2], "inv_freq");
    const at::Tensor k = maybe_tensor(a[3], "k");
    const int flags = (truth(a[4]) ? HS_ROPE_INTERLEAVED : 0) | (truth(a[5]) ? HS_ROPE_INVERSE : 0);
    const float factor = (float)number(a[6]);
    at::Tensor out = maybe_tensor(a[7], "out"), out_k = maybe_tensor(a[8], "out_k");
    Device dev(q, positions, f, k, out, out_k);
    const Rows rq = rows_of(q, "q");
    const int rot = rot_of(f, rq.d);
    TORCH_CHECK_TYPE(positions.scalar_type() == at::kInt && positions.dim() == 1 && positions.size(0) == rq.T &&
                         positions.is_contiguous(),
                     "positions must be a contiguous int32 vector, one per row");
    const int code = code_of(q.scalar_type());
    out = like(out, q, "out must be like q");
    const Rows ro = rows_of(out, "out");
    Rows rk{0, 0, 0, 0}, rok{0, 0, 0, 0};
    if (k.defined()) {
        rk = rows_of(k, "k");
        TORCH_CHECK_VALUE(rk.T == rq.T && rk.d == rq.d && k.scalar_type() == q.scalar_type(),
                          "q and k disagree on rows, head dim or dtype");
        out_k = like(out_k, k, "out_k must be like k");
        rok = rows_of(out_k, "out_k");
    } else {
        TORCH_CHECK_VALUE(!out_k.defined(), "out_k without k");
    }
    if (!run(dev, "hysparse_rope", [&](hs_stream_t st) {
        return g_rope(rq.T, rq.H, rk.H, rq.d, code, ptr(q), rq.ld, ptr(k), rk.ld, (const int32_t *)ptr(positions),
                             (const double *)ptr(f), rot, flags, factor, mut(out), ro.ld, mut(out_k), rok.ld, st);
    })) return nullptr;
    changed(out, out_k);
    return k.defined() ? pair(out, out_k) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// cache_write(k, v, k_pages, v_pages, cu, kv_len, table, k_scale, v_scale, inv_freq, interleaved, factor, ws)
PyObject *cache_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    need_args(n, 13);
    const at::Tensor k = tensor(a[0], "k"), v = tensor(a[1], "v"), kp = tensor(a[2], "k_pages"), vp = tensor(a[3], "v_pages");
    const at::Tensor cu = tensor(a[4], "cu_seqlens"), kv = tensor(a[5], "kv_len"), table = tensor(a[6], "block_table");
    const at::Tensor ks = maybe_tensor(a[7], "k_scale"), vs = maybe_tensor(a[8], "v_scale"), f = maybe_tensor(a[9], "inv_freq");
    const int flags = truth(a[10]) ? HS_ROPE_INTERLEAVED : 0;
    const float factor = (float)number(a[11]);
    const at::Tensor ws = maybe_tensor(a[12], "ws");
    Device dev(k, v, kp, vp, cu, kv, table, ks, vs, f, ws);
    const Rows rk = rows_of(k, "k"), rv = rows_of(v, "v");
    const Pages p = pages_of(kp, vp, cu, kv, table, ks, vs);
    TORCH_CHECK_VALUE(rv.T == rk.T && rv.H == rk.H && rv.d == rk.d && rk.H == p.Hkv && rk.d == p.d &&
                          k.scalar_type() == v.scalar_type(),
                      "k, v and the pages disagree on rows, heads, head dim or dtype");
    const int rot = rot_of(f, rk.d), code = code_of(k.scalar_type());
    status_ws(ws);
    if (!run(dev, "hysparse_cache_write", [&](hs_stream_t st) {
        return g_cache_write(&p.c, rk.T, rk.H, rk.d, code, ptr(k), rk.ld, ptr(v), rv.ld, (const double *)ptr(f), rot,
                                    flags, factor, mut(ws), st);
    })) return nullptr;
    changed(kp, vp, ks, vs);
    return Py_NewRef(Py_None);
    END_HANDLE_TH_ERRORS
}

// cache_read(k_pages, v_pages, cu, table, total, start, k_scale, v_scale, bf16, out_k, out_v, ws)
PyObject *cache_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    need_args(n, 12);
    const at::Tensor kp = tensor(a[0], "k_pages"), vp = tensor(a[1], "v_pages"), cu = tensor(a[2], "cu_rows"),
                     table = tensor(a[3], "block_table");
    const int total = as_int(integer(a[4]), "total");
    TORCH_CHECK_VALUE(total >= 0, "total must not be negative");
    const at::Tensor start = maybe_tensor(a[5], "start"), ks = maybe_tensor(a[6], "k_scale"), vs = maybe_tensor(a[7], "v_scale");
    const at::ScalarType dtype = truth(a[8]) ? at::kBFloat16 : at::kFloat;
    at::Tensor ok = maybe_tensor(a[9], "out_k"), ov = maybe_tensor(a[10], "out_v");
    const at::Tensor ws = maybe_tensor(a[11], "ws");
    Device dev(kp, vp, cu, table, start, ks, vs, ok, ov, ws);
    const Pages p = pages_of(kp, vp, cu, at::Tensor(), table, ks, vs);
    dense(start, "start", at::kInt, {table.size(0)});
    const int64_t shape[3] = {total, p.Hkv, p.d};
    if (!ok.defined()) ok = at::empty(shape, kp.options().dtype(dtype));
    if (!ov.defined()) ov = at::empty(shape, kp.options().dtype(dtype));
    dense(ok, "out_k", dtype, shape);
    dense(ov, "out_v", dtype, shape);
    status_ws(ws);
    if (!run(dev, "hysparse_cache_read", [&](hs_stream_t st) {
        return g_cache_read(&p.c, (const int32_t *)ptr(start), total, p.Hkv, p.d, code_of(dtype), mut(ok), mut(ov),
                                   mut(ws), st);
    })) return nullptr;
    changed(ok, ov);
    return pair(ok, ov);
    END_HANDLE_TH_ERRORS
}

// out, lse and scratch of the attention calls: checked, or allocated.
struct AttnBuffers {
    Rows q;
    at::Tensor out, lse, ws;
};
AttnBuffers attn_buffers(const at::Tensor &q, int Hkv, int B, int max_q, int max_len, PyObject *out, PyObject *lse,
                         PyObject *ws) {
    AttnBuffers b;
    b.q = rows_of(q, "q");
    TORCH_CHECK_TYPE(q.scalar_type() == at::kBFloat16, "q must be bfloat16");
    b.out = maybe_tensor(out, "out");
    b.lse = maybe_tensor(lse, "lse");
    b.ws = maybe_tensor(ws, "ws");
    if (b.out.defined()) {
        dense(b.out, "out", at::kBFloat16, q.sizes());
    } else {
        b.out = at::empty(q.sizes(), q.options());
    }
    const int64_t lse_shape[2] = {b.q.H, b.q.T};
    if (b.lse.defined()) {
        dense(b.lse, "lse", at::kFloat, lse_shape);
    } else {
        b.lse = at::empty(lse_shape, q.options().dtype(at::kFloat));
    }
    if (b.ws.defined()) {
        TORCH_CHECK_VALUE(b.ws.is_contiguous(), "ws must be contiguous");
    } else {       // scratch for this call only: its status word is not read
        const size_t n = g_workspace_size(B, b.q.T, b.q.H, Hkv, b.q.d, max_q, max_len);
        b.ws = at::empty({(int64_t)n}, q.options().dtype(at::kByte));
    }
    return b;
}

// packed_attn(q, k, v, cu, max_len (None or 0: T), scale, out, lse, ws)
PyObject *packed_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    need_args(n, 9);
    const at::Tensor q = tensor(a[0], "q"), k = tensor(a[1], "k"), v = tensor(a[2], "v"), cu = tensor(a[3], "cu_seqlens");
    const float scale = (float)number(a[5]);
    Device dev(q, k, v, cu);
    for (int i = 6; i < 9; ++i) dev.add(maybe_tensor(a[i], "out, lse, ws"));
    const Rows rk = rows_of(k, "k"), rv = rows_of(v, "v");
    TORCH_CHECK_VALUE(rv.T == rk.T && rv.H == rk.H && rv.d == rk.d && q.dim() == 3 && q.size(0) == rk.T && q.size(2) == rk.d,
                      "q, k and v disagree on rows, heads or head dim");
    TORCH_CHECK_TYPE(k.scalar_type() == at::kBFloat16 && v.scalar_type() == at::kBFloat16, "k and v must be bfloat16");
    TORCH_CHECK_VALUE(cu.dim() == 1 && cu.size(0) >= 2, "cu_seqlens must hold B + 1 entries");
    dense(cu, "cu_seqlens", at::kInt, {cu.size(0)});
    const int B = as_int(cu.size(0) - 1, "B");
    int longest = a[4] == Py_None ? 0 : as_int(integer(a[4]), "max_len");
    if (longest == 0) longest = rk.T;
    const AttnBuffers b = attn_buffers(q, rk.H, B, longest, longest, a[6], a[7], a[8]);
    if (!run(dev, "hysparse_packed_attn", [&](hs_stream_t st) {
        return g_packed_attn((const int32_t *)ptr(cu), B, b.q.T, b.q.H, rk.H, b.q.d, longest, scale, ptr(q), b.q.ld,
                                    ptr(k), rk.ld, ptr(v), rv.ld, mut(b.out), (float *)mut(b.lse), mut(b.ws), b.ws.nbytes(),
                                    st);
    })) return nullptr;
    changed(b.out, b.lse);
    return pair(b.out, b.lse);
    END_HANDLE_TH_ERRORS
}

// chunk_attn_paged(q, k_pages, v_pages, cu, kv_len, table, max_q, max_len, k_scale, v_scale, scale, out, lse, ws)
PyObject *chunk_attn_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    need_args(n, 14);
    const at::Tensor q = tensor(a[0], "q"), kp = tensor(a[1], "k_pages"), vp = tensor(a[2], "v_pages"),
                     cu = tensor(a[3], "cu_seqlens"), kv = tensor(a[4], "kv_len"), table = tensor(a[5], "block_table");
    const at::Tensor ks = maybe_tensor(a[8], "k_scale"), vs = maybe_tensor(a[9], "v_scale");
    const float scale = (float)number(a[10]);
    Device dev(q, kp, vp, cu, kv, table, ks, vs);
    for (int i = 11; i < 14; ++i) dev.add(maybe_tensor(a[i], "out, lse, ws"));
    const Pages p = pages_of(kp, vp, cu, kv, table, ks, vs);
    TORCH_CHECK_VALUE(q.dim() == 3 && q.size(2) == p.d, "q and the pages disagree on head dim");
    const int most = a[6] == Py_None ? as_int(q.size(0), "T") : as_int(integer(a[6]), "max_q");
    int longest = a[7] == Py_None ? 0 : as_int(integer(a[7]), "max_len");
    if (longest == 0) longest = as_int((int64_t)p.c.max_pages * p.c.page_size, "max_pages * page_size");
    const AttnBuffers b = attn_buffers(q, p.Hkv, p.c.B, most, longest, a[11], a[12], a[13]);
    if (!run(dev, "hysparse_chunk_attn_paged", [&](hs_stream_t st) {
        return g_chunk_attn(&p.c, b.q.T, b.q.H, p.Hkv, b.q.d, most, longest, scale, ptr(q), b.q.ld, mut(b.out),
                                         (float *)mut(b.lse), mut(b.ws), b.ws.nbytes(), st);
    })) return nullptr;
    changed(b.out, b.lse);
    return pair(b.out, b.lse);
    END_HANDLE_TH_ERRORS
}

// bind(check, address of each library call used here, in the order below)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    need_args(n, 7);
    void *fn[6];
    for (int i = 0; i < 6; ++i) fn[i] = (void *)integer(a[1 + i]);
    g_rope = (decltype(g_rope))fn[0];
    g_cache_write = (decltype(g_cache_write))fn[1];
    g_cache_read = (decltype(g_cache_read))fn[2];
    g_workspace_size = (decltype(g_workspace_size))fn[3];
    g_packed_attn = (decltype(g_packed_attn))fn[4];
    g_chunk_attn = (decltype(g_chunk_attn))fn[5];
    Py_INCREF(a[0]);
    Py_XDECREF(g_check);
    g_check = a[0];
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rope), FAST(cache_write), FAST(cache_read), FAST(packed_attn), FAST(chunk_attn_paged),
                         FAST(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Native half of ragged.py", -1, methods, nullptr, nullptr, nullptr,
                      nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
    PyObject *m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "TORCH_VERSION", TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
