// binding.cpp — the short way from Python into the paged-cache and rotary entry
// points.
//
// The calls of a decoding step take 2 to 10 us on the GPU.  Checked and
// marshalled in Python they took the host 9 to 25 us (an allocation 2 to 3, a
// ctypes call 4); the same checks here take less than half.  Each function
// handles the ordinary call: every argument as documented, outputs and
// workspace given or from the allocator, the current stream and device.  For
// anything else, a refusal included, it returns None without having done
// anything, and the Python function of the same name goes on: it has all the
// checks and messages.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "gbattn.h"

namespace {

decltype(&attn_page_table) page_table_fn;
decltype(&attn_cache_append) cache_append_fn;
decltype(&attn_fwd_paged) fwd_paged_fn;
decltype(&attn_fwd_paged_workspace_size) workspace_fn;
decltype(&attn_rope) rope_fn;
decltype(&attn_cache_append_rope) append_rope_fn;
decltype(&attn_cache_append_fp8) append_fp8_fn;
decltype(&attn_fwd_paged_fp8) fwd_paged_fp8_fn;

// A failed check: None to the caller.
struct NotHandled {};
void need(bool ok) {
    if (!ok) throw NotHandled{};
}

const at::Tensor& tensor(PyObject* o) {
    need(THPVariable_CheckExact(o));
    return THPVariable_Unpack(o);
}

int integer(PyObject* o) {
    need(PyLong_CheckExact(o));
    int overflow = 0;
    const long v = PyLong_AsLongAndOverflow(o, &overflow);
    need(overflow == 0 && v >= INT32_MIN && v <= INT32_MAX);
    return static_cast<int>(v);
}

// The device of a call: t's, which has to be the current one.
c10::Device call_device(const at::Tensor& t) {
    need(t.is_cuda() && t.get_device() == c10::cuda::current_device());
    return t.device();
}

template <typename T>
T* index_ptr(const at::Tensor& t, at::ScalarType type, int64_t n, c10::Device dev) {
    need(t.scalar_type() == type && t.device() == dev && t.dim() == 1 && t.size(0) == n && t.is_contiguous());
    return static_cast<T*>(t.data_ptr());
}

int32_t* table_ptr(const at::Tensor& t, c10::Device dev) {
    need(t.scalar_type() == at::kInt && t.device() == dev && t.dim() == 2 && t.is_contiguous());
    return static_cast<int32_t*>(t.data_ptr());
}

int* status_ptr(PyObject* o, c10::Device dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == at::kInt && t.device() == dev && t.numel() >= 1 && t.is_contiguous());
    return static_cast<int*>(t.data_ptr());
}

attn_dtype dtype_of(const at::Tensor& t) {
    need(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf);
    return t.scalar_type() == at::kBFloat16 ? ATTN_DTYPE_BF16 : ATTN_DTYPE_FP16;
}

bool same_layout(const at::Tensor& a, const at::Tensor& b) {
    if (!a.sizes().equals(b.sizes())) return false;
    for (int64_t i = 0; i < a.dim(); ++i)
        if (a.size(i) > 1 && a.stride(i) != b.stride(i)) return false;
    return true;
}

// [num_pages, Hkv, page_size, d] caches of the given type on x's device, laid out alike.
void check_caches(const at::Tensor& k, const at::Tensor& v, const at::Tensor& x, int64_t d, at::ScalarType type) {
    need(k.dim() == 4 && k.scalar_type() == type && v.scalar_type() == type &&
         k.device() == x.device() && v.device() == x.device() && k.size(3) == d && k.stride(3) == 1 &&
         v.dim() == 4 && v.stride(3) == 1 && same_layout(k, v));
    for (int64_t i = 0; i < 3; ++i) need(k.size(i) <= INT32_MAX);
}

// Scales of a cache of e4m3.
float* scale_ptr(const at::Tensor& t, const at::Tensor& cache) {
    need(t.scalar_type() == at::kFloat && t.device() == cache.device() && t.dim() == 2 &&
         t.size(0) == cache.size(0) && t.size(1) == cache.size(1) && t.is_contiguous());
    return static_cast<float*>(t.data_ptr());
}

double number(PyObject* o) {
    need(PyFloat_CheckExact(o));
    return PyFloat_AS_DOUBLE(o);
}

// An output: what the caller gave, or a new tensor.
at::Tensor output(PyObject* given, at::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
    if (given == Py_None) return at::empty(sizes, at::TensorOptions().dtype(type).device(dev));
    const at::Tensor& t = tensor(given);
    need(t.scalar_type() == type && t.device() == dev && t.sizes().equals(sizes) && t.is_contiguous());
    return t;
}

// call(stream) without the interpreter's lock: a launch can wait for the GPU.
template <typename Call>
void launch(c10::Device dev, Call&& call) {
    void* stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    PyThreadState* state = PyEval_SaveThread();
    const attn_status st = call(stream);
    PyEval_RestoreThread(state);
    need(st == ATTN_OK);   // the Python function calls again and raises
}

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (out == nullptr) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t));
    return out;
}

template <typename Body>
PyObject* guarded(Body&& body) {
    try {
        return body();
    } catch (...) {   // no C++ exception may leave; the Python function finds out what is wrong
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// page_table(cached_lens, new_lens, page_table, free_pages, num_free, page_size, max_tokens, cu_seqlens_q,
// seq_lens, slots, pages_taken, dev_status) -> the four outputs
PyObject* page_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == 12);
        const at::Tensor &cached = tensor(a[0]), &fresh = tensor(a[1]), &table = tensor(a[2]), &free = tensor(a[3]),
                         &num_free = tensor(a[4]);
        const int page_size = integer(a[5]), max_tokens = integer(a[6]);
        const c10::Device dev = call_device(table);
        int32_t* const table_p = table_ptr(table, dev);
        const int64_t B = table.size(0);
        need(B >= 1 && B <= INT32_MAX && table.size(1) <= INT32_MAX && free.dim() == 1 &&
             free.size(0) <= INT32_MAX && max_tokens >= 1);
        const int32_t* const cached_p = index_ptr<int32_t>(cached, at::kInt, B, dev);
        const int32_t* const fresh_p = index_ptr<int32_t>(fresh, at::kInt, B, dev);
        const int32_t* const free_p = index_ptr<int32_t>(free, at::kInt, free.size(0), dev);
        const int32_t* const num_p = index_ptr<int32_t>(num_free, at::kInt, 1, dev);
        int* const status = status_ptr(a[11], dev);
        const at::Tensor cu = output(a[7], {B + 1}, at::kInt, dev), lens = output(a[8], {B}, at::kInt, dev),
                         slots = output(a[9], {max_tokens}, at::kLong, dev),
                         taken = output(a[10], {1}, at::kInt, dev);
        launch(dev, [&](void* stream) {
            return page_table_fn(cached_p, fresh_p, table_p, free_p, num_p, static_cast<int32_t*>(cu.data_ptr()),
                                 static_cast<int32_t*>(lens.data_ptr()), static_cast<int64_t*>(slots.data_ptr()),
                                 static_cast<int32_t*>(taken.data_ptr()), static_cast<int>(B),
                                 static_cast<int>(table.size(1)), page_size, max_tokens,
                                 static_cast<int>(free.size(0)), status, stream);
        });
        return tuple_of({cu, lens, slots, taken});
    });
}

// A step's K and V rows: [T, Hkv, d], d innermost, laid out alike.
void check_rows(const at::Tensor& k, const at::Tensor& v) {
    need(k.dim() == 3 && k.stride(2) == 1 && v.dim() == 3 && v.stride(2) == 1 && v.device() == k.device() &&
         v.scalar_type() == k.scalar_type() && same_layout(k, v) && k.size(0) <= INT32_MAX &&
         k.size(2) <= INT32_MAX);
}

// cache_append(k, v, k_cache, v_cache, slots, dev_status) -> True; cache_append_fp8 has the scales behind them
template <bool kFp8>
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == (kFp8 ? 8 : 6));
        const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]), &kc = tensor(a[2]), &vc = tensor(a[3]),
                         &slots = tensor(a[4]);
        const c10::Device dev = call_device(k);
        check_rows(k, v);
        check_caches(kc, vc, k, k.size(2), kFp8 ? at::kFloat8_e4m3fn : k.scalar_type());
        need(kc.size(1) == k.size(1));
        const int64_t* const slots_p = index_ptr<int64_t>(slots, at::kLong, k.size(0), dev);
        const attn_dtype dtype = dtype_of(k);
        int* const status = status_ptr(a[5], dev);
        const int T = static_cast<int>(k.size(0)), Hkv = static_cast<int>(k.size(1)), d = static_cast<int>(k.size(2)),
                  pages = static_cast<int>(kc.size(0)), page_size = static_cast<int>(kc.size(2));
        float *ks = nullptr, *vs = nullptr;
        if (kFp8) {
            ks = scale_ptr(tensor(a[6]), kc);
            vs = scale_ptr(tensor(a[7]), kc);
        }
        launch(dev, [&](void* stream) {
            return kFp8 ? append_fp8_fn(k.data_ptr(), v.data_ptr(), kc.data_ptr(), vc.data_ptr(), ks, vs, slots_p, T,
                                        Hkv, d, dtype, k.stride(0), k.stride(1), pages, page_size, kc.stride(0),
                                        kc.stride(1), kc.stride(2), status, stream)
                        : cache_append_fn(k.data_ptr(), v.data_ptr(), kc.data_ptr(), vc.data_ptr(), slots_p, T, Hkv,
                                          d, dtype, k.stride(0), k.stride(1), pages, page_size, kc.stride(0),
                                          kc.stride(1), kc.stride(2), status, stream);
        });
        Py_RETURN_TRUE;
    });
}

// fwd_paged(q, k_cache, v_cache, page_table, seq_lens, cu_seqlens_q, max_seqlen_q, causal, window, scale, out,
// lse, workspace, dev_status) -> (out, lse); fwd_paged_fp8 has the scales behind them
template <bool kFp8>
PyObject* fwd_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == (kFp8 ? 16 : 14));
        const at::Tensor &q = tensor(a[0]), &kc = tensor(a[1]), &vc = tensor(a[2]), &table = tensor(a[3]),
                         &lens = tensor(a[4]), &cu = tensor(a[5]);
        const int max_q = integer(a[6]), window = integer(a[8]);
        need(PyBool_Check(a[7]) && (a[9] == Py_None || PyFloat_CheckExact(a[9])));
        const c10::Device dev = call_device(q);
        need(q.dim() == 3 && q.stride(2) == 1 && q.size(0) <= INT32_MAX && q.size(1) <= INT32_MAX &&
             q.size(2) >= 1 && q.size(2) <= INT32_MAX);
        check_caches(kc, vc, q, q.size(2), kFp8 ? at::kFloat8_e4m3fn : q.scalar_type());
        float *ks = nullptr, *vs = nullptr;
        if (kFp8) {
            ks = scale_ptr(tensor(a[14]), kc);
            vs = scale_ptr(tensor(a[15]), kc);
        }
        const int total_q = static_cast<int>(q.size(0)), H = static_cast<int>(q.size(1)),
                  d = static_cast<int>(q.size(2)), Hkv = static_cast<int>(kc.size(1)),
                  page_size = static_cast<int>(kc.size(2)), pages = static_cast<int>(kc.size(0));
        const int32_t* const table_p = table_ptr(table, dev);
        const int64_t B = table.size(0);
        need(B >= 1 && B < INT32_MAX && table.size(1) <= INT32_MAX);
        const int max_pages = static_cast<int>(table.size(1));
        const int32_t* const lens_p = index_ptr<int32_t>(lens, at::kInt, B, dev);
        const int32_t* const cu_p = index_ptr<int32_t>(cu, at::kInt, B + 1, dev);
        const attn_dtype dtype = dtype_of(q);
        const float scale = static_cast<float>(a[9] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d))
                                                               : PyFloat_AS_DOUBLE(a[9]));
        int* const status = status_ptr(a[13], dev);
        const at::Tensor out = output(a[10], {total_q, H, d}, q.scalar_type(), dev),
                         lse_t = output(a[11], {H, total_q}, at::kFloat, dev);
        at::Tensor workspace;
        size_t bytes = 0;
        if (a[12] == Py_None) {
            bytes = workspace_fn(static_cast<int>(B), H, Hkv, total_q, max_q, max_pages, page_size, d);
            if (bytes > 0) workspace = output(Py_None, {static_cast<int64_t>(bytes)}, at::kByte, dev);
        } else {
            workspace = tensor(a[12]);
            need(workspace.device() == dev && workspace.is_contiguous());
            bytes = workspace.nbytes();
        }
        void* const ws = workspace.defined() ? workspace.data_ptr() : nullptr;
        float* const lse = static_cast<float*>(lse_t.data_ptr());
        launch(dev, [&](void* stream) {
            return kFp8 ? fwd_paged_fp8_fn(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ks, vs, out.data_ptr(), lse,
                                           cu_p, lens_p, table_p, static_cast<int>(B), H, Hkv, total_q, max_q, pages,
                                           page_size, max_pages, d, dtype, q.stride(0), q.stride(1), kc.stride(0),
                                           kc.stride(1), kc.stride(2), scale, a[7] == Py_True, window, ws, bytes,
                                           status, stream)
                        : fwd_paged_fn(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), out.data_ptr(), lse, cu_p, lens_p,
                                       table_p, static_cast<int>(B), H, Hkv, total_q, max_q, pages, page_size,
                                       max_pages, d, dtype, q.stride(0), q.stride(1), kc.stride(0), kc.stride(1),
                                       kc.stride(2), scale, a[7] == Py_True, window, ws, bytes, status, stream);
        });
        return tuple_of({out, lse_t});
    });
}

// Rows of queries or keys: [B, heads, N, d], or packed [tokens, heads, d].
struct Rows {
    int64_t B, heads, N, d, batch, head, token;   // strides
    explicit Rows(const at::Tensor& t) {
        const bool packed = t.dim() == 3;
        need((packed || t.dim() == 4) && t.stride(-1) == 1);
        B = packed ? 1 : t.size(0);
        heads = t.size(1);
        N = t.size(packed ? 0 : 2);
        d = t.size(-1);
        batch = packed ? 0 : t.stride(0);
        head = t.stride(1);
        token = t.stride(packed ? 0 : 2);
        need(B <= INT32_MAX && heads <= INT32_MAX && N <= INT32_MAX && d <= INT32_MAX);
    }
};

// An output like t: what the caller gave, with any strides, or a new tensor.
at::Tensor output_like(PyObject* given, const at::Tensor& t) {
    if (given == Py_None) return at::empty(t.sizes(), at::TensorOptions().dtype(t.scalar_type()).device(t.device()));
    const at::Tensor& o = tensor(given);
    need(o.scalar_type() == t.scalar_type() && o.device() == t.device() && o.sizes().equals(t.sizes()));
    return o;
}

const float* frequencies(const at::Tensor& t, c10::Device dev, int& rotary_dim) {
    need(t.scalar_type() == at::kFloat && t.device() == dev && t.dim() == 1 && t.is_contiguous() &&
         t.size(0) <= (1 << 20));
    rotary_dim = static_cast<int>(2 * t.size(0));
    return static_cast<const float*>(t.data_ptr());
}

// rope(q, k, inv_freq, positions, interleaved, inverse, scaling, q_out, k_out) -> (q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == 9 && a[1] != Py_None && PyBool_Check(a[4]) && PyBool_Check(a[5]));
        const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]);
        const c10::Device dev = call_device(q);
        const Rows x(q), y(k);
        need(k.dim() == q.dim() && k.device() == dev && k.scalar_type() == q.scalar_type() && y.B == x.B &&
             y.N == x.N && y.d == x.d && y.heads >= 1);
        const attn_dtype dtype = q.scalar_type() == at::kFloat ? ATTN_DTYPE_FP32 : dtype_of(q);
        int rotary_dim;
        const float* const freq = frequencies(tensor(a[2]), dev, rotary_dim);
        const int32_t* pos = nullptr;
        int64_t pos_batch = 0;
        if (a[3] != Py_None) {
            const at::Tensor& t = tensor(a[3]);
            if (q.dim() == 4 && t.dim() == 2) {
                need(t.size(0) == x.B && t.size(1) == x.N);
                pos = table_ptr(t, dev);
                pos_batch = x.N;
            } else {
                pos = index_ptr<int32_t>(t, at::kInt, x.N, dev);
            }
        } else {
            need(q.dim() == 4);
        }
        const float scaling = static_cast<float>(number(a[6]));
        const at::Tensor q_out = output_like(a[7], q), k_out = output_like(a[8], k);
        const Rows xo(q_out), yo(k_out);
        launch(dev, [&](void* stream) {
            return rope_fn(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), freq, pos,
                           static_cast<int>(x.B), static_cast<int>(x.heads), static_cast<int>(y.heads),
                           static_cast<int>(x.N), static_cast<int>(x.d), rotary_dim, dtype, x.batch, x.head, x.token,
                           y.batch, y.head, y.token, xo.batch, xo.head, xo.token, yo.batch, yo.head, yo.token,
                           pos_batch, scaling, a[4] == Py_True, a[5] == Py_True, stream);
        });
        return tuple_of({q_out, k_out});
    });
}

// cache_append_rope(q, k, v, k_cache, v_cache, slots, inv_freq, positions, cu_seqlens_q, seq_lens, interleaved,
// scaling, q_out, dev_status) -> q_out
PyObject* cache_append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == 14 && PyBool_Check(a[10]));
        const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]), &v = tensor(a[2]), &kc = tensor(a[3]),
                         &vc = tensor(a[4]), &slots = tensor(a[5]);
        const c10::Device dev = call_device(k);
        check_rows(k, v);
        need(q.dim() == 3 && q.device() == dev && q.scalar_type() == k.scalar_type() && q.size(0) == k.size(0) &&
             q.size(2) == k.size(2));
        const Rows x(q);
        check_caches(kc, vc, k, k.size(2), k.scalar_type());
        need(kc.size(1) == k.size(1));
        const int64_t* const slots_p = index_ptr<int64_t>(slots, at::kLong, k.size(0), dev);
        int rotary_dim;
        const float* const freq = frequencies(tensor(a[6]), dev, rotary_dim);
        const int32_t *pos = nullptr, *cu = nullptr, *lens = nullptr;
        int64_t B = 0;
        if (a[7] != Py_None) {
            pos = index_ptr<int32_t>(tensor(a[7]), at::kInt, k.size(0), dev);
        } else {
            const at::Tensor& l = tensor(a[9]);
            need(l.dim() == 1 && l.size(0) >= 1 && l.size(0) < INT32_MAX);
            B = l.size(0);
            lens = index_ptr<int32_t>(l, at::kInt, B, dev);
            cu = index_ptr<int32_t>(tensor(a[8]), at::kInt, B + 1, dev);
        }
        const attn_dtype dtype = dtype_of(k);
        const float scaling = static_cast<float>(number(a[11]));
        int* const status = status_ptr(a[13], dev);
        const at::Tensor q_out = output_like(a[12], q);
        const Rows xo(q_out);
        launch(dev, [&](void* stream) {
            return append_rope_fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), kc.data_ptr(),
                                  vc.data_ptr(), slots_p, freq, pos, cu, lens, static_cast<int>(B),
                                  static_cast<int>(x.N), static_cast<int>(x.heads), static_cast<int>(k.size(1)),
                                  static_cast<int>(x.d), rotary_dim, dtype, x.token, x.head, k.stride(0), k.stride(1),
                                  xo.token, xo.head, static_cast<int>(kc.size(0)), static_cast<int>(kc.size(2)),
                                  kc.stride(0), kc.stride(1), kc.stride(2), scaling, a[10] == Py_True, status, stream);
        });
        return THPVariable_Wrap(q_out);
    });
}

// bind(addresses of attn_page_table, attn_cache_append, attn_fwd_paged, attn_fwd_paged_workspace_size, attn_rope,
// attn_cache_append_rope, attn_cache_append_fp8, attn_fwd_paged_fp8)
PyObject* bind(PyObject*, PyObject* args) {
    unsigned long long p[8];
    if (!PyArg_ParseTuple(args, "KKKKKKKK", &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6], &p[7])) return nullptr;
    page_table_fn = reinterpret_cast<decltype(page_table_fn)>(p[0]);
    cache_append_fn = reinterpret_cast<decltype(cache_append_fn)>(p[1]);
    fwd_paged_fn = reinterpret_cast<decltype(fwd_paged_fn)>(p[2]);
    workspace_fn = reinterpret_cast<decltype(workspace_fn)>(p[3]);
    rope_fn = reinterpret_cast<decltype(rope_fn)>(p[4]);
    append_rope_fn = reinterpret_cast<decltype(append_rope_fn)>(p[5]);
    append_fp8_fn = reinterpret_cast<decltype(append_fp8_fn)>(p[6]);
    fwd_paged_fp8_fn = reinterpret_cast<decltype(fwd_paged_fp8_fn)>(p[7]);
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"page_table", fast(page_table), METH_FASTCALL, nullptr},
    {"cache_append", fast(cache_append<false>), METH_FASTCALL, nullptr},
    {"cache_append_fp8", fast(cache_append<true>), METH_FASTCALL, nullptr},
    {"cache_append_rope", fast(cache_append_rope), METH_FASTCALL, nullptr},
    {"fwd_paged", fast(fwd_paged<false>), METH_FASTCALL, nullptr},
    {"fwd_paged_fp8", fast(fwd_paged<true>), METH_FASTCALL, nullptr},
    {"rope", fast(rope), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
