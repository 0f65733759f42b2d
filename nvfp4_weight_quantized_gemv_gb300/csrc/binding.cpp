// binding.cpp -- the Python binding of the operators over the paged cache:
// PyTorch tensors to the C ABI's argument structs.
//
// A decode step's calls take a few microseconds on the GPU, and reading a dozen
// tensors' types, shapes, strides and addresses from Python takes longer than
// that: 13 us of the 15 to 18 us that a call took from Python through ctypes.
// The library itself stays free of Python and PyTorch: its functions are
// handed over by address.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "nvfp4_gemv.h"

namespace {

decltype(&nvfp4_qk_norm_rope) g_norm_rope;
decltype(&nvfp4_kv_append) g_append;
decltype(&nvfp4_attn_paged) g_attn;
decltype(&nvfp4_attn_paged_shared) g_shared;
decltype(&nvfp4_attn_shared_workspace_size) g_shared_bytes;
decltype(&nvfp4_kv_tables) g_tables;
decltype(&nvfp4_verify_drafts) g_verify;
PyObject *g_check;  // raises the library's last error for a status

struct Refused {  // a Python error is set
};
[[noreturn]] void refuse(PyObject *type, const std::string &what) {
    PyErr_SetString(type, what.c_str());
    throw Refused();
}

bool given(PyObject *o) { return o != Py_None; }

// The call's device: the current one, which the library launches on.  Unknown
// (-1) until a tensor of a GPU is met.
thread_local int t_device = -1;

const at::Tensor &tensor(const char *name, PyObject *o) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.is_cuda()) {
        if (t_device < 0) t_device = c10::cuda::current_device();
        if (t.get_device() != t_device)
            refuse(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                                         ", the current device is cuda:" + std::to_string(t_device));
    }
    return t;
}
int integer(const char *name, PyObject *o) {
    PyObject *const i = PyNumber_Index(o);
    if (!i) throw Refused();
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(i, &overflow);
    Py_DECREF(i);
    if (overflow || v > INT32_MAX || v < INT32_MIN)
        refuse(PyExc_OverflowError, std::string(name) + " does not fit 32 bits");
    return (int)v;
}
float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return (float)v;
}
int sizes32(const char *name, int64_t n) {
    if (n > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is too large");
    return (int)n;
}

// A bf16 tensor [tokens, heads, head_dim] of any strides over tokens and heads.
nvfp4_head_rows head_rows(const char *name, const at::Tensor &t) {
    if (t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.dim() != 3)
        refuse(PyExc_TypeError, std::string(name) + " must be a CUDA bfloat16 tensor [tokens, heads, head_dim]");
    if (t.stride(2) != 1 && t.size(2) > 1)
        refuse(PyExc_ValueError, std::string(name) + ": the entries of a head must be contiguous");
    return {static_cast<const uint16_t *>(t.data_ptr()), t.stride(0), t.stride(1), sizes32(name, t.size(1))};
}
at::Tensor out_rows(const char *name, PyObject *out, const at::Tensor &like) {
    if (!given(out)) return at::empty(like.sizes(), at::TensorOptions().dtype(at::kBFloat16).device(like.device()));
    const at::Tensor &t = tensor(name, out);
    if (t.scalar_type() != at::kBFloat16 || t.sizes() != like.sizes() || !t.is_cuda() || !t.is_contiguous())
        refuse(PyExc_ValueError, std::string(name) + " must be a contiguous CUDA bfloat16 tensor of the rows' shape");
    return t;
}
uint16_t *bf16_ptr(const at::Tensor &t) { return static_cast<uint16_t *>(t.data_ptr()); }

const uint16_t *weight(const char *name, PyObject *o, int64_t head_dim) {
    if (!given(o)) return nullptr;
    const at::Tensor &w = tensor(name, o);
    if (w.scalar_type() != at::kBFloat16 || !w.is_cuda() || !w.is_contiguous() || w.numel() != head_dim)
        refuse(PyExc_ValueError, std::string(name) + " must be a contiguous CUDA bfloat16 tensor [head_dim]");
    return bf16_ptr(w);
}
nvfp4_norm_rope norm_rope(int64_t head_dim, PyObject *q_weight, PyObject *k_weight, PyObject *eps, PyObject *cos_sin,
                          PyObject *interleaved) {
    nvfp4_norm_rope how = {};
    how.q_weight = weight("q_weight", q_weight, head_dim);
    how.k_weight = weight("k_weight", k_weight, head_dim);
    how.eps = number(eps);
    if (given(cos_sin)) {
        const at::Tensor &t = tensor("cos_sin", cos_sin);
        if (t.scalar_type() != at::kFloat || !t.is_cuda() || !t.is_contiguous() || t.dim() != 2)
            refuse(PyExc_ValueError, "cos_sin must be a contiguous CUDA float32 tensor [positions, rot]");
        how.cos_sin = static_cast<const float *>(t.data_ptr());
        how.table_positions = sizes32("cos_sin", t.size(0));
        how.rot = sizes32("cos_sin", t.size(1));
    }
    const int inter = PyObject_IsTrue(interleaved);
    if (inter < 0) throw Refused();
    how.interleaved = inter;
    return how;
}
const int32_t *int32s(const char *name, const at::Tensor &t) {
    if (t.scalar_type() != at::kInt || !t.is_cuda() || t.dim() < 1 || (t.stride(-1) != 1 && t.numel() > 1))
        refuse(PyExc_TypeError, std::string(name) + " must be a CUDA int32 tensor with contiguous rows");
    return static_cast<const int32_t *>(t.data_ptr());
}

nvfp4_kv_cache kv_cache(PyObject *k_cache, PyObject *v_cache, PyObject *k_scale, PyObject *v_scale) {
    const at::Tensor &k = tensor("k_cache", k_cache), &v = tensor("v_cache", v_cache);
    for (const at::Tensor *t : {&k, &v}) {
        const auto dt = t->scalar_type();
        if ((dt != at::kFloat8_e4m3fn && dt != at::kByte) || !t->is_cuda() || t->dim() != 4 || t->stride(3) != 1)
            refuse(PyExc_TypeError,
                   std::string(t == &k ? "k_cache" : "v_cache") + " must be a CUDA float8_e4m3fn or uint8 tensor "
                   "[pages, kv_heads, page_size, head_dim] with contiguous entries");
    }
    bool alike = k.sizes() == v.sizes();
    for (int i = 0; alike && i < 4; ++i)  // the stride of a dimension of one entry says nothing
        alike = k.size(i) <= 1 || k.stride(i) == v.stride(i);
    if (!alike) refuse(PyExc_ValueError, "k_cache and v_cache must have the same shape and strides");
    const int64_t pages = k.size(0), heads = k.size(1), d = k.size(3);
    nvfp4_kv_cache c = {};
    c.k = static_cast<uint8_t *>(k.data_ptr());
    c.v = static_cast<uint8_t *>(v.data_ptr());
    const char *const names[2] = {"k_scale", "v_scale"};
    for (int i = 0; i < 2; ++i) {
        const at::Tensor &t = tensor(names[i], i ? v_scale : k_scale);
        if (t.scalar_type() != at::kFloat || !t.is_cuda() || !t.is_contiguous() || t.dim() != 2 || t.size(0) != pages ||
            t.size(1) != heads)
            refuse(PyExc_ValueError, std::string(names[i]) + " must be a contiguous CUDA float32 tensor [" +
                                         std::to_string(pages) + ", " + std::to_string(heads) + "]");
        (i ? c.v_scale : c.k_scale) = static_cast<float *>(t.data_ptr());
    }
    c.page_stride = pages > 1 ? k.stride(0) : d;
    c.head_stride = heads > 1 ? k.stride(1) : d;
    c.token_stride = k.stride(2);
    c.pages = sizes32("k_cache", pages);
    c.kv_heads = sizes32("k_cache", heads);
    c.page_size = sizes32("k_cache", k.size(2));
    c.head_dim = sizes32("k_cache", d);
    return c;
}
// table_positions: what bounds max_kv_len beside the table where it is not given (0: nothing).
nvfp4_kv_batch kv_batch(PyObject *block_table, PyObject *cu_q, PyObject *kv_lens, int64_t tokens, PyObject *max_q_len,
                        PyObject *max_kv_len, const nvfp4_kv_cache &c, int table_positions) {
    const at::Tensor &table = tensor("block_table", block_table), &cu = tensor("cu_q", cu_q);
    const at::Tensor &lens = tensor("kv_lens", kv_lens);
    const int64_t b = lens.numel();
    if (table.dim() != 2 || table.size(0) != b || cu.numel() != b + 1)
        refuse(PyExc_ValueError, "shape mismatch: block_table [batch, pages], cu_q [batch + 1], kv_lens [batch]");
    const int64_t most = table.size(1) * c.page_size;
    nvfp4_kv_batch n = {};
    if (given(max_kv_len)) {
        n.max_kv_len = integer("max_kv_len", max_kv_len);
        if (n.max_kv_len > most) refuse(PyExc_ValueError, "block_table has fewer pages than max_kv_len needs");
    } else {
        const int64_t all = table_positions > 0 && table_positions < most ? table_positions : most;
        n.max_kv_len = (int)(all < INT32_MAX ? all : INT32_MAX);
    }
    n.block_table = int32s("block_table", table);
    n.cu_q = int32s("cu_q", cu);
    n.kv_lens = int32s("kv_lens", lens);
    n.batch = sizes32("kv_lens", b);
    n.table_stride = sizes32("block_table", b > 1 ? table.stride(0) : table.size(1));
    n.tokens = sizes32("tokens", tokens);
    n.max_q_len = integer("max_q_len", max_q_len);
    return n;
}

// The stream of a call: the given one (a torch stream or a handle), which is then
// the current stream until the call returns, so that outputs are allocated in its
// order; else the current one.
class Stream {
public:
    Stream(PyObject *stream, const at::Tensor &t) {
        if (!given(stream)) {
            handle_ = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
            return;
        }
        PyObject *h = PyObject_GetAttrString(stream, "cuda_stream");
        if (!h) {
            PyErr_Clear();
            h = PyNumber_Long(stream);
            if (!h) throw Refused();
        }
        handle_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
        Py_DECREF(h);
        if (!handle_ && PyErr_Occurred()) throw Refused();
        guard_.reset_stream(c10::cuda::getStreamFromExternal(handle_, t.get_device()));
    }
    cudaStream_t handle() const { return handle_; }

private:
    cudaStream_t handle_;
    c10::cuda::OptionalCUDAStreamGuard guard_;
};

void check(nvfp4_status status) {
    if (status == NVFP4_OK) return;
    PyObject *const r = PyObject_CallFunction(g_check, "i", (int)status);
    Py_XDECREF(r);
    if (r) PyErr_SetString(PyExc_RuntimeError, "the call failed");
    throw Refused();
}

void arguments(Py_ssize_t got, Py_ssize_t want) {
    t_device = -1;
    if (got != want) refuse(PyExc_TypeError, "expected " + std::to_string(want) + " arguments");
}

// (q, k, positions, cos_sin, q_weight, k_weight, eps, interleaved, q_out, k_out, stream) -> (q_out, k_out)
PyObject *py_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        arguments(n, 11);
        const at::Tensor &q = tensor("q", a[0]);
        const nvfp4_head_rows qr = head_rows("q", q);
        const Stream stream(a[10], q);
        const int64_t tokens = q.size(0), d = q.size(2);
        nvfp4_head_rows kr = {};
        at::Tensor k_out;
        if (given(a[1])) {
            const at::Tensor &k = tensor("k", a[1]);
            kr = head_rows("k", k);
            if (k.size(0) != tokens || k.size(2) != d)
                refuse(PyExc_ValueError, "shape mismatch: q [tokens, heads, head_dim], k [tokens, kv_heads, head_dim]");
            k_out = out_rows("k_out", a[9], k);
        }
        const int32_t *positions = nullptr;
        if (given(a[2])) {
            const at::Tensor &t = tensor("positions", a[2]);
            if (t.numel() != tokens) refuse(PyExc_ValueError, "positions must have one entry a token");
            positions = int32s("positions", t);
        }
        const nvfp4_norm_rope how = norm_rope(d, a[4], a[5], a[6], a[3], a[7]);
        const at::Tensor q_out = out_rows("q_out", a[8], q);
        check(g_norm_rope(&qr, given(a[1]) ? &kr : nullptr, positions, &how, sizes32("q", tokens), sizes32("q", d),
                          bf16_ptr(q_out), k_out.defined() ? bf16_ptr(k_out) : nullptr, stream.handle()));
        PyObject *const qo = THPVariable_Wrap(q_out);
        PyObject *const ko = k_out.defined() ? THPVariable_Wrap(k_out) : Py_NewRef(Py_None);
        PyObject *const both = PyTuple_Pack(2, qo, ko);
        Py_DECREF(qo);
        Py_DECREF(ko);
        return both;
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_q, kv_lens, max_q_len, cos_sin, k_weight, q, q_weight,
//  eps, interleaved, q_out, max_kv_len, stream) -> q_out or None
PyObject *py_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        arguments(n, 19);
        const at::Tensor &k = tensor("k", a[0]), &v = tensor("v", a[1]);
        const at::Tensor *const q = given(a[12]) ? &tensor("q", a[12]) : nullptr;
        const at::Tensor &cache = tensor("k_cache", a[2]);
        if (k.dim() != 3 || v.sizes() != k.sizes() || cache.dim() < 1 || cache.size(-1) != k.size(2) ||
            (q && (q->dim() != 3 || q->size(0) != k.size(0) || q->size(2) != k.size(2))))
            refuse(PyExc_ValueError, "shape mismatch: q [tokens, heads, head_dim], k and v [tokens, kv_heads, head_dim]");
        const nvfp4_head_rows kr = head_rows("k", k), vr = head_rows("v", v);
        const Stream stream(a[18], k);
        const int64_t tokens = k.size(0), d = k.size(2);
        const nvfp4_kv_cache c = kv_cache(a[2], a[3], a[4], a[5]);
        nvfp4_head_rows qr = {};
        at::Tensor q_out;
        if (q) {
            qr = head_rows("q", *q);
            q_out = out_rows("q_out", a[16], *q);
        }
        const nvfp4_norm_rope how = norm_rope(d, a[13], a[11], a[14], a[10], a[15]);
        const nvfp4_kv_batch b = kv_batch(a[6], a[7], a[8], tokens, a[9], a[17], c, how.table_positions);
        check(g_append(q ? &qr : nullptr, &kr, &vr, &how, &c, &b, q_out.defined() ? bf16_ptr(q_out) : nullptr,
                       stream.handle()));
        return q_out.defined() ? THPVariable_Wrap(q_out) : Py_NewRef(Py_None);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, k_scale, v_scale, block_table, cu_q, kv_lens, max_q_len, max_kv_len, scale, gate, out,
//  workspace, stream) -> out
PyObject *py_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        arguments(n, 15);
        const at::Tensor &q = tensor("q", a[0]);
        const nvfp4_head_rows qr = head_rows("q", q);
        const Stream stream(a[14], q);
        const nvfp4_kv_cache c = kv_cache(a[1], a[2], a[3], a[4]);
        nvfp4_head_rows gr = {};
        bool match = c.head_dim == q.size(2);
        if (given(a[11])) {
            const at::Tensor &gate = tensor("gate", a[11]);
            gr = head_rows("gate", gate);
            match = match && gate.sizes() == q.sizes();
        }
        if (!match)
            refuse(PyExc_ValueError, "shape mismatch: q and gate [tokens, heads, head_dim], the cache [.., head_dim]");
        const nvfp4_kv_batch b = kv_batch(a[5], a[6], a[7], q.size(0), a[8], a[9], c, 0);
        const float scale = given(a[10]) ? number(a[10]) : (float)(1.0 / std::sqrt((double)c.head_dim));
        const at::Tensor out = out_rows("out", a[12], q);
        void *ws = nullptr;
        size_t ws_bytes = 0;
        if (given(a[13])) {
            const at::Tensor &t = tensor("workspace", a[13]);
            if (!t.is_cuda() || !t.is_contiguous())
                refuse(PyExc_ValueError, "workspace must be a contiguous CUDA tensor");
            ws = t.data_ptr();
            ws_bytes = t.nbytes();
        }
        check(g_attn(&qr, &c, &b, scale, given(a[11]) ? &gr : nullptr, bf16_ptr(out), ws, ws_bytes, stream.handle()));
        return THPVariable_Wrap(out);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// Contiguous tensors of one allocation on the current stream: a call with many
// small outputs allocates once (1.2 us each).
class Outputs {
public:
    int add(at::ScalarType type, std::initializer_list<int64_t> sizes) {
        Piece &p = pieces_[n_];
        p.type = type;
        p.dims = 0;
        int64_t count = 1;
        for (int64_t x : sizes) {
            p.sizes[p.dims++] = x;
            count *= x;
        }
        p.at = bytes_;
        bytes_ += (count * (int64_t)c10::elementSize(type) + 15) / 16 * 16;
        return n_++;
    }
    void allocate(const at::Device &device) {
        base_ = at::empty({bytes_}, at::TensorOptions().dtype(at::kByte).device(device));
    }
    void *ptr(int i) const { return static_cast<char *>(base_.data_ptr()) + pieces_[i].at; }
    at::Tensor get(int i) const {
        const Piece &p = pieces_[i];
        c10::Storage storage = base_.storage();
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
            std::move(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(p.type));
        t.unsafeGetTensorImpl()->set_storage_offset(p.at / (int64_t)c10::elementSize(p.type));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(c10::IntArrayRef(p.sizes, p.dims));
        return t;
    }

private:
    struct Piece {
        at::ScalarType type;
        int64_t sizes[2], at;
        int dims;
    };
    Piece pieces_[8];
    int n_ = 0;
    int64_t bytes_ = 0;
    at::Tensor base_;
};
PyObject *tuple(std::initializer_list<at::Tensor> items) {
    PyObject *const all = PyTuple_New((Py_ssize_t)items.size());
    if (!all) throw Refused();
    Py_ssize_t i = 0;
    for (const at::Tensor &t : items) PyTuple_SET_ITEM(all, i++, t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None));
    return all;
}
// A contiguous CUDA tensor of one dimension and `n` entries (any number if n < 0).
const at::Tensor &vec(const char *name, PyObject *o, at::ScalarType type, int64_t n) {
    const at::Tensor &t = tensor(name, o);
    if (t.scalar_type() != type || !t.is_cuda())
        refuse(PyExc_TypeError, std::string(name) + " must be a CUDA " + c10::toString(type) + " tensor");
    if (t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous())
        refuse(PyExc_ValueError, std::string(name) + " must be contiguous and have " +
                                     (n >= 0 ? std::to_string(n) + " entries" : std::string("one dimension")));
    return t;
}
template <class T>
T *ptr(const at::Tensor &t) {
    return static_cast<T *>(t.data_ptr());
}

// (q, k_cache, v_cache, k_scale, v_scale, block_table, cu_q, kv_lens, group_cu, prefix_lens, max_q_len, max_kv_len,
//  max_group_tokens, max_own_len, scale, gate, out, workspace, stream) -> out
PyObject *py_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        arguments(n, 19);
        const at::Tensor &q = tensor("q", a[0]);
        const nvfp4_head_rows qr = head_rows("q", q);
        const Stream stream(a[18], q);
        const nvfp4_kv_cache c = kv_cache(a[1], a[2], a[3], a[4]);
        nvfp4_head_rows gr = {};
        bool match = c.head_dim == q.size(2);
        if (given(a[15])) {
            const at::Tensor &gate = tensor("gate", a[15]);
            gr = head_rows("gate", gate);
            match = match && gate.sizes() == q.sizes();
        }
        if (!match)
            refuse(PyExc_ValueError, "shape mismatch: q and gate [tokens, heads, head_dim], the cache [.., head_dim]");
        const nvfp4_kv_batch b = kv_batch(a[5], a[6], a[7], q.size(0), a[10], a[11], c, 0);
        const at::Tensor &lens = vec("prefix_lens", a[9], at::kInt, -1);
        nvfp4_kv_prefix p = {};
        p.prefix_lens = ptr<const int32_t>(lens);
        p.groups = sizes32("prefix_lens", lens.size(0));
        p.group_cu = ptr<const int32_t>(vec("group_cu", a[8], at::kInt, lens.size(0) + 1));
        p.max_group_tokens = given(a[12]) ? integer("max_group_tokens", a[12]) : b.tokens > 0 ? b.tokens : 1;
        p.max_own_len = given(a[13]) ? integer("max_own_len", a[13]) : 0;
        const float scale = given(a[14]) ? number(a[14]) : (float)(1.0 / std::sqrt((double)c.head_dim));
        const at::Tensor out = out_rows("out", a[16], q);
        at::Tensor ws;
        if (given(a[17])) {
            ws = tensor("workspace", a[17]);
            if (!ws.is_cuda() || !ws.is_contiguous())
                refuse(PyExc_ValueError, "workspace must be a contiguous CUDA tensor");
        } else {
            size_t bytes = 0;
            check(g_shared_bytes(b.tokens, qr.heads, c.head_dim, b.batch, &bytes));
            ws = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(q.device()));
        }
        check(g_shared(&qr, &c, &b, &p, scale, given(a[15]) ? &gr : nullptr, bf16_ptr(out), ws.data_ptr(), ws.nbytes(),
                       stream.handle()));
        return THPVariable_Wrap(out);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (block_table, held, free_pages, span, kv_lens, q_lens, page_size, tokens, kept, held_out, span_out, stream)
//  -> (cu_q, new_lens, positions, slots, held_out, span_out)
PyObject *py_tables(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        arguments(n, 12);
        const at::Tensor &table = tensor("block_table", a[0]);
        if (table.scalar_type() != at::kInt || !table.is_cuda())
            refuse(PyExc_TypeError, "block_table must be a CUDA Int tensor");
        if (table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
            refuse(PyExc_ValueError, "block_table must be [batch, pages] with contiguous rows");
        const Stream stream(a[11], table);
        const int64_t batch = table.size(0);
        const int tokens = integer("tokens", a[7]);
        if (tokens < 0) refuse(PyExc_ValueError, "tokens must not be negative");
        nvfp4_kv_pages p = {};
        p.block_table = ptr<int32_t>(table);
        p.table_stride = batch > 1 ? table.stride(0) : table.size(1);
        p.table_width = sizes32("block_table", table.size(1));
        p.page_size = integer("page_size", a[6]);
        p.held = ptr<int32_t>(vec("held", a[1], at::kInt, batch));
        const at::Tensor &ring = vec("free_pages", a[2], at::kInt, -1);
        p.free_pages = ptr<int32_t>(ring);
        p.ring = sizes32("free_pages", ring.size(0));
        p.span = ptr<int64_t>(vec("span", a[3], at::kLong, 2));
        const at::Tensor &kv = vec("kv_lens", a[4], at::kInt, batch), &q = vec("q_lens", a[5], at::kInt, batch);
        p.kept = given(a[8]) ? ptr<int32_t>(vec("kept", a[8], at::kInt, batch)) : nullptr;
        at::Tensor held_out, span_out;
        Outputs o;
        const int slots = o.add(at::kLong, {tokens}), positions = o.add(at::kInt, {tokens});
        const int cu = o.add(at::kInt, {batch + 1}), lens = o.add(at::kInt, {batch});
        int held_at = -1, span_at = -1;
        if (given(a[9])) {
            held_out = vec("held_out", a[9], at::kInt, batch);
            p.held_out = ptr<int32_t>(held_out);
        } else {
            held_at = o.add(at::kInt, {batch});
        }
        if (given(a[10])) {
            span_out = vec("span_out", a[10], at::kLong, 2);
            p.span_out = ptr<int64_t>(span_out);
        } else {
            span_at = o.add(at::kLong, {2});
        }
        o.allocate(table.device());
        if (held_at >= 0) {
            held_out = o.get(held_at);
            p.held_out = ptr<int32_t>(held_out);
        }
        if (span_at >= 0) {
            span_out = o.get(span_at);
            p.span_out = ptr<int64_t>(span_out);
        }
        check(g_tables(&p, sizes32("block_table", batch), ptr<int32_t>(kv), ptr<int32_t>(q), tokens,
                       static_cast<int32_t *>(o.ptr(cu)), static_cast<int32_t *>(o.ptr(lens)),
                       static_cast<int32_t *>(o.ptr(positions)), static_cast<int64_t *>(o.ptr(slots)), stream.handle()));
        return tuple({o.get(cu), o.get(lens), o.get(positions), o.get(slots), held_out, span_out});
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

const float *distributions(const char *name, const at::Tensor &t, int64_t rows, int64_t vocab) {
    if (t.scalar_type() != at::kFloat || !t.is_cuda() || t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1))
        refuse(PyExc_TypeError, std::string(name) + " must be a CUDA float32 tensor [tokens, vocab] with contiguous rows");
    if (t.size(0) != rows || t.size(1) != vocab)
        refuse(PyExc_ValueError, "shape mismatch: target and draft [tokens, vocab], ids and u_accept [tokens]");
    return ptr<const float>(t);
}

// (target, ids, cu_q, u_accept, u_next, draft, kv_lens, stream) -> (out_tokens, accepted, next, new_lens or None)
PyObject *py_verify(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        arguments(n, 8);
        const at::Tensor &target = tensor("target", a[0]);
        if (target.dim() != 2) refuse(PyExc_ValueError, "target must be [tokens, vocab]");
        const int64_t rows = target.size(0), vocab = target.size(1);
        nvfp4_draft_rows r = {};
        r.target = distributions("target", target, rows, vocab);
        r.target_stride = rows > 1 ? target.stride(0) : vocab;
        if (given(a[5])) {
            const at::Tensor &draft = tensor("draft", a[5]);
            r.draft = distributions("draft", draft, rows, vocab);
            r.draft_stride = rows > 1 ? draft.stride(0) : vocab;
        }
        const Stream stream(a[7], target);
        r.ids = ptr<const int32_t>(vec("ids", a[1], at::kInt, rows));
        r.tokens = sizes32("target", rows);
        r.vocab = sizes32("target", vocab);
        const at::Tensor &pick = vec("u_next", a[4], at::kFloat, -1);
        const int64_t batch = pick.size(0);
        const at::Tensor &cu = vec("cu_q", a[2], at::kInt, batch + 1), &u = vec("u_accept", a[3], at::kFloat, rows);
        const int32_t *const kv = given(a[6]) ? ptr<const int32_t>(vec("kv_lens", a[6], at::kInt, batch)) : nullptr;
        Outputs o;
        const int out = o.add(at::kInt, {rows}), accepted = o.add(at::kInt, {batch}), next = o.add(at::kInt, {batch});
        const int lens = given(a[6]) ? o.add(at::kInt, {batch}) : -1;
        o.allocate(target.device());
        check(g_verify(&r, ptr<const int32_t>(cu), kv, ptr<const float>(u), ptr<const float>(pick), sizes32("cu_q", batch),
                       static_cast<int32_t *>(o.ptr(out)), static_cast<int32_t *>(o.ptr(accepted)),
                       static_cast<int32_t *>(o.ptr(next)), lens >= 0 ? static_cast<int32_t *>(o.ptr(lens)) : nullptr,
                       stream.handle()));
        return tuple({o.get(out), o.get(accepted), o.get(next), lens >= 0 ? o.get(lens) : at::Tensor()});
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (addresses of nvfp4_qk_norm_rope, nvfp4_kv_append, nvfp4_attn_paged, nvfp4_attn_paged_shared,
//  nvfp4_attn_shared_workspace_size, nvfp4_kv_tables and nvfp4_verify_drafts, what raises a status)
PyObject *py_setup(PyObject *, PyObject *args) {
    unsigned long long f[7];
    PyObject *raise_status;
    if (!PyArg_ParseTuple(args, "KKKKKKKO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &raise_status)) return nullptr;
    g_norm_rope = reinterpret_cast<decltype(g_norm_rope)>(f[0]);
    g_append = reinterpret_cast<decltype(g_append)>(f[1]);
    g_attn = reinterpret_cast<decltype(g_attn)>(f[2]);
    g_shared = reinterpret_cast<decltype(g_shared)>(f[3]);
    g_shared_bytes = reinterpret_cast<decltype(g_shared_bytes)>(f[4]);
    g_tables = reinterpret_cast<decltype(g_tables)>(f[5]);
    g_verify = reinterpret_cast<decltype(g_verify)>(f[6]);
    Py_XSETREF(g_check, Py_NewRef(raise_status));
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"setup", py_setup, METH_VARARGS, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_norm_rope)), METH_FASTCALL, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_append)), METH_FASTCALL, nullptr},
    {"attn_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_attn)), METH_FASTCALL, nullptr},
    {"attn_paged_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_shared)), METH_FASTCALL, nullptr},
    {"kv_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_tables)), METH_FASTCALL, nullptr},
    {"verify_drafts", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_verify)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attn_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_binding() { return PyModule_Create(&g_module); }
