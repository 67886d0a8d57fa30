// paged_binding.cpp -- the Python binding of the paged calls as an extension module
// (dynamic_sparse_attention_est_b200._paged): checks of the torch tensors, their
// pointers and strides handed to the C ABI, outputs allocated by torch.
//
// A decoding step calls these once per layer on kernels of a few microseconds.
// Host time of a call with the attributes read in Python and the C ABI reached by
// ctypes: 27 us for the append, 30 us for attention; here 5 us and 10 to 16 us.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/StringUtil.h>

#include <cmath>

#include "minf.h"

namespace {

template <class... A>
[[noreturn]] void refuse(const A &...what) {
    const std::string text = c10::str(what...);
    PyErr_SetString(PyExc_ValueError, text.c_str());
    throw python_error();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// What the first tensor of a call fixes for the others.
struct Kind {
    c10::Device dev{c10::kCPU};
    at::ScalarType type;
    int code;  // MINF_BF16 or MINF_FP16
};

Kind kind_of(const at::Tensor &t, const char *name) {
    if (t.dim() != 3 || !t.is_cuda() || (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf))
        refuse(name, " must be a CUDA bf16 or fp16 tensor [tokens, heads, 128]");
    return {t.device(), t.scalar_type(), t.scalar_type() == at::kHalf ? MINF_FP16 : MINF_BF16};
}

void same_kind(const at::Tensor &t, const char *name, const Kind &k) {
    if (t.scalar_type() != k.type || t.device() != k.dev) refuse(name, " must be ", k.type, " on ", k.dev);
}

minf_rows rows_of(const at::Tensor &t, const char *name, const Kind &k, int64_t total, int64_t heads) {
    same_kind(t, name, k);
    if (t.dim() != 3 || t.size(0) != total || t.size(1) != heads || t.size(2) != 128 || t.stride(2) != 1)
        refuse(name, " must be [", total, ", ", heads, ", 128] with a contiguous last dimension");
    return {t.data_ptr(), t.stride(0), t.stride(1)};
}

int int32_of(int64_t x, const char *name) {
    if (x < 0 || x > 0x7fffffff) refuse(name, " out of range");
    return (int)x;
}

minf_paged_seqs seqs_of(PyObject *tables_o, PyObject *cu_o, PyObject *kv_o, int64_t max_q, int64_t total, int64_t page,
                        int64_t num_pages, const Kind &k) {
    const at::Tensor &tables = tensor(tables_o, "block_tables"), &cu = tensor(cu_o, "cu_q"),
                     &kv = tensor(kv_o, "kv_lens");
    auto check = [&](const at::Tensor &t, const char *name, int64_t nd) {
        if (t.scalar_type() != at::kInt || t.device() != k.dev || t.dim() != nd || (t.size(nd - 1) > 1 && t.stride(nd - 1) != 1))
            refuse(name, " must be a ", nd, "-D int32 tensor on ", k.dev, " with a contiguous last dimension");
    };
    check(tables, "block_tables", 2);
    check(cu, "cu_q", 1);
    check(kv, "kv_lens", 1);
    const int64_t n = kv.size(0);
    if (cu.size(0) != n + 1 || tables.size(0) != n)
        refuse("cu_q, kv_lens and block_tables disagree on the number of sequences");
    minf_paged_seqs s{};
    s.cu_q = static_cast<const int32_t *>(cu.data_ptr());
    s.kv_lens = static_cast<const int32_t *>(kv.data_ptr());
    s.block_tables = static_cast<const int32_t *>(tables.data_ptr());
    s.width = int32_of(tables.size(1), "block_tables");
    s.table_stride = n > 1 ? tables.stride(0) : s.width;
    s.n_seqs = int32_of(n, "sequences");
    s.total = int32_of(total, "tokens");
    s.max_q = int32_of(std::min(max_q, total), "max_q_len");
    s.page_size = int32_of(page, "page_size");
    s.num_pages = int32_of(num_pages, "pages");
    return s;
}

struct Cache {
    minf_paged_cache c;
    int64_t pages, hkv, page;
};

Cache cache_of(PyObject *k_o, PyObject *v_o, const Kind &kind) {
    const at::Tensor &k = tensor(k_o, "k_cache"), &v = tensor(v_o, "v_cache");
    auto check = [&](const at::Tensor &t, const char *name) {
        if (t.scalar_type() != kind.type || t.device() != kind.dev || t.dim() != 4 || t.sizes() != k.sizes() ||
            t.size(3) != 128)
            refuse(name, " must be a ", kind.type, " tensor [pages, hkv, page_size, 128] on ", kind.dev);
        if (t.stride(3) != 1 || t.stride(2) != 128 || (t.size(1) > 1 && t.stride(1) != t.size(2) * 128))
            refuse(name, " must be contiguous within a page");
    };
    check(k, "k_cache");
    check(v, "v_cache");
    Cache x{};
    x.pages = k.size(0);
    x.hkv = k.size(1);
    x.page = k.size(2);
    const int64_t least = x.hkv * x.page * 128;
    x.c = {k.data_ptr(), v.data_ptr(), x.pages > 1 ? k.stride(0) : least, x.pages > 1 ? v.stride(0) : least};
    return x;
}

// The caller's workspace, or one of `need` bytes of which the status block is zero: the
// kernels write what they read of the rest (157 MB for a chunk).
at::Tensor workspace_of(PyObject *o, size_t need, const Kind &k) {
    if (o == Py_None) {
        at::Tensor ws = at::empty({(int64_t)std::max(need, (size_t)MINF_STATUS_BYTES)},
                                  at::TensorOptions().dtype(at::kByte).device(k.dev));
        ws.narrow(0, 0, MINF_STATUS_BYTES).zero_();
        return ws;
    }
    const at::Tensor &ws = tensor(o, "ws");
    if (ws.scalar_type() != at::kByte || ws.device() != k.dev || !ws.is_contiguous())
        refuse("ws must be a contiguous uint8 tensor on ", k.dev);
    return ws;
}

minf_stream_t stream_of(const Kind &k) {
    return (minf_stream_t)c10::cuda::getCurrentCUDAStream(k.dev.index()).stream();
}

int64_t integer(PyObject *o, const char *name) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) refuse(name, " must be an integer");
    return x;
}

bool truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();  // the object's own exception
    return x != 0;
}

// out (allocated unless given) and lse (allocated if wanted) of an attention call.
struct Outputs {
    at::Tensor out, lse;
    minf_rows rows;
};
Outputs outputs_of(PyObject *out_o, bool want_lse, const Kind &k, int64_t total, int64_t hq) {
    Outputs x;
    if (out_o == Py_None) x.out = at::empty({total, hq, 128}, at::TensorOptions().dtype(k.type).device(k.dev));
    else x.out = tensor(out_o, "out");
    x.rows = rows_of(x.out, "out", k, total, hq);
    if (want_lse) x.lse = at::empty({total, hq}, at::TensorOptions().dtype(at::kFloat).device(k.dev));
    return x;
}

void count_args(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse("expected ", want, " arguments, got ", n);
}

PyObject *wrap(const at::Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject *result(int rc, const at::Tensor &a, const at::Tensor &b) {
    return Py_BuildValue("(iNN)", rc, wrap(a), wrap(b));
}

// append(k, v, k_cache, v_cache, tables, cu_q, kv_lens, max_q, rope, interleaved, q, q_out, k_bounds, ws)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_args(n, 14);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const Kind kind = kind_of(k, "k");
    const int64_t total = k.size(0);
    const Cache cache = cache_of(a[2], a[3], kind);
    const minf_paged_seqs seqs = seqs_of(a[4], a[5], a[6], integer(a[7], "max_q_len"), total, cache.page, cache.pages, kind);
    const minf_rows rk = rows_of(k, "k", kind, total, cache.hkv), rv = rows_of(v, "v", kind, total, cache.hkv);
    int64_t hq = cache.hkv;
    minf_rows rq{}, ro{};
    at::Tensor q_out;
    const bool with_q = a[10] != Py_None;
    if (with_q) {
        const at::Tensor &q = tensor(a[10], "q");
        if (q.dim() != 3) refuse("q must be [tokens, heads, 128]");
        hq = q.size(1);
        rq = rows_of(q, "q", kind, total, hq);
        if (a[11] == Py_None) q_out = at::empty({total, hq, 128}, at::TensorOptions().dtype(kind.type).device(kind.dev));
        else q_out = tensor(a[11], "q_out");
        ro = rows_of(q_out, "q_out", kind, total, hq);
    } else if (a[11] != Py_None) {
        refuse("q_out without q");
    }
    const float *rope = nullptr;
    int rows = 0, rot = 0;
    if (a[8] != Py_None) {
        const at::Tensor &t = tensor(a[8], "rope");
        if (t.scalar_type() != at::kFloat || t.device() != kind.dev || t.dim() != 2 || !t.is_contiguous())
            refuse("rope must be a contiguous fp32 tensor [positions, rot] on ", kind.dev);
        rope = static_cast<const float *>(t.data_ptr());
        rows = int32_of(t.size(0), "rope");
        rot = int32_of(t.size(1), "rope");
    }
    const bool interleaved = truth(a[9]);
    void *bounds = nullptr;
    if (a[12] != Py_None) {
        const at::Tensor &t = tensor(a[12], "k_bounds");
        if (t.scalar_type() != kind.type || t.device() != kind.dev || !t.is_contiguous() || t.dim() != 4 ||
            t.size(0) != cache.pages || t.size(1) != cache.hkv || t.size(2) != 2 || t.size(3) != 128)
            refuse("k_bounds must be a contiguous ", kind.type, " tensor [", cache.pages, ", ", cache.hkv,
                   ", 2, 128] on ", kind.dev);
        bounds = t.data_ptr();
    }
    const at::Tensor ws = workspace_of(a[13], MINF_STATUS_BYTES, kind);
    const minf_stream_t st = stream_of(kind);
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = minf_paged_append(&seqs, kind.code, (int)hq, (int)cache.hkv, 128, &rk, &rv, with_q ? &rq : nullptr,
                           with_q ? &ro : nullptr, &cache.c, bounds, rope, rows, rot, interleaved, ws.data_ptr(),
                           (size_t)ws.numel(), st);
    Py_END_ALLOW_THREADS;
    return result(rc, q_out, at::Tensor());
    END_HANDLE_TH_ERRORS
}

// attention(q, k_cache, v_cache, tables, cu_q, kv_lens, max_q, scale, out, want_lse, ws)
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_args(n, 11);
    const at::Tensor &q = tensor(a[0], "q");
    const Kind kind = kind_of(q, "q");
    const int64_t total = q.size(0), hq = q.size(1);
    const Cache cache = cache_of(a[1], a[2], kind);
    const minf_paged_seqs seqs = seqs_of(a[3], a[4], a[5], integer(a[6], "max_q_len"), total, cache.page, cache.pages, kind);
    const minf_rows rq = rows_of(q, "q", kind, total, hq);
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt(128.0) : PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) throw python_error();
    const Outputs o = outputs_of(a[8], truth(a[9]), kind, total, hq);
    const size_t need = a[10] != Py_None ? 0
                                         : minf_paged_workspace_bytes(MINF_OP_PAGED_ATTENTION, (int)hq, (int)cache.hkv, seqs.total,
                                                                      seqs.n_seqs, seqs.max_q, seqs.width, 0);
    const at::Tensor ws = workspace_of(a[10], need, kind);
    const minf_stream_t st = stream_of(kind);
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = minf_paged_attention(&seqs, kind.code, (int)hq, (int)cache.hkv, 128, &rq, &cache.c, (float)scale, &o.rows,
                              o.lse.defined() ? static_cast<float *>(o.lse.data_ptr()) : nullptr, ws.data_ptr(),
                              (size_t)ws.numel(), st);
    Py_END_ALLOW_THREADS;
    return result(rc, o.out, o.lse);
    END_HANDLE_TH_ERRORS
}

// block_estimate(q, k_bounds, tables, cu_q, kv_lens, max_q, page_size, topk, ws)
PyObject *block_estimate(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_args(n, 9);
    const at::Tensor &q = tensor(a[0], "q"), &kb = tensor(a[1], "k_bounds");
    const Kind kind = kind_of(q, "q");
    const int64_t total = q.size(0), hq = q.size(1);
    if (kb.scalar_type() != kind.type || kb.device() != kind.dev || kb.dim() != 4 || !kb.is_contiguous() ||
        kb.size(2) != 2 || kb.size(3) != 128)
        refuse("k_bounds must be a contiguous ", kind.type, " tensor [pages, hkv, 2, 128] on ", kind.dev);
    const int64_t hkv = kb.size(1);
    const minf_paged_seqs seqs =
        seqs_of(a[2], a[3], a[4], integer(a[5], "max_q_len"), total, integer(a[6], "page_size"), kb.size(0), kind);
    const minf_rows rq = rows_of(q, "q", kind, total, hq);
    const int topk = int32_of(integer(a[7], "topk"), "topk");
    const auto ints = at::TensorOptions().dtype(at::kInt).device(kind.dev);
    const at::Tensor idx = at::empty({total, hkv, topk}, ints), cnt = at::empty({total, hkv}, ints);
    const size_t need = a[8] != Py_None ? 0
                                        : minf_paged_workspace_bytes(MINF_OP_PAGED_BLOCK_ESTIMATE, (int)hq, (int)hkv, seqs.total,
                                                                     seqs.n_seqs, seqs.max_q, seqs.width, topk);
    const at::Tensor ws = workspace_of(a[8], need, kind);
    const minf_stream_t st = stream_of(kind);
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = minf_paged_block_estimate(&seqs, kind.code, (int)hq, (int)hkv, 128, &rq, kb.data_ptr(), topk,
                                   static_cast<int32_t *>(idx.data_ptr()), static_cast<int32_t *>(cnt.data_ptr()),
                                   ws.data_ptr(), (size_t)ws.numel(), st);
    Py_END_ALLOW_THREADS;
    return result(rc, idx, cnt);
    END_HANDLE_TH_ERRORS
}

// block_attention(q, k_cache, v_cache, tables, cu_q, kv_lens, max_q, blk_idx, blk_cnt, scale, out, want_lse, ws)
PyObject *block_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_args(n, 13);
    const at::Tensor &q = tensor(a[0], "q");
    const Kind kind = kind_of(q, "q");
    const int64_t total = q.size(0), hq = q.size(1);
    const Cache cache = cache_of(a[1], a[2], kind);
    const minf_paged_seqs seqs = seqs_of(a[3], a[4], a[5], integer(a[6], "max_q_len"), total, cache.page, cache.pages, kind);
    const minf_rows rq = rows_of(q, "q", kind, total, hq);
    const at::Tensor &idx = tensor(a[7], "blk_idx"), &cnt = tensor(a[8], "blk_cnt");
    if (idx.scalar_type() != at::kInt || idx.device() != kind.dev || idx.dim() != 3 || idx.size(0) != total ||
        idx.size(1) != cache.hkv || !idx.is_contiguous())
        refuse("blk_idx must be a contiguous int32 tensor [", total, ", ", cache.hkv, ", topk] on ", kind.dev);
    if (cnt.scalar_type() != at::kInt || cnt.device() != kind.dev || cnt.dim() != 2 || cnt.size(0) != total ||
        cnt.size(1) != cache.hkv || !cnt.is_contiguous())
        refuse("blk_cnt must be a contiguous int32 tensor [", total, ", ", cache.hkv, "] on ", kind.dev);
    const int topk = int32_of(idx.size(2), "topk");
    const double scale = a[9] == Py_None ? 1.0 / std::sqrt(128.0) : PyFloat_AsDouble(a[9]);
    if (PyErr_Occurred()) throw python_error();
    const Outputs o = outputs_of(a[10], truth(a[11]), kind, total, hq);
    const size_t need = a[12] != Py_None ? 0
                                         : minf_paged_workspace_bytes(MINF_OP_PAGED_BLOCK_ATTENTION, (int)hq, (int)cache.hkv,
                                                                      seqs.total, seqs.n_seqs, seqs.max_q, seqs.width, topk);
    const at::Tensor ws = workspace_of(a[12], need, kind);
    const minf_stream_t st = stream_of(kind);
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = minf_paged_block_attention(&seqs, kind.code, (int)hq, (int)cache.hkv, 128, &rq, &cache.c, (float)scale,
                                    static_cast<const int32_t *>(idx.data_ptr()),
                                    static_cast<const int32_t *>(cnt.data_ptr()), topk, &o.rows,
                                    o.lse.defined() ? static_cast<float *>(o.lse.data_ptr()) : nullptr, ws.data_ptr(),
                                    (size_t)ws.numel(), st);
    Py_END_ALLOW_THREADS;
    return result(rc, o.out, o.lse);
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)), METH_FASTCALL, nullptr},
    {"block_estimate", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(block_estimate)), METH_FASTCALL, nullptr},
    {"block_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(block_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", "Paged-cache calls of libminf.so for torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
