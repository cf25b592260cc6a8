// The Python side of libgqa_serve.so: checks of the tensors, outputs, the current device and
// stream, and the C call.  These calls may take a few microseconds on the GPU, less than the
// same checks do as Python operations.  No computation happens here.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdlib>
#include <optional>
#include <stdexcept>
#include <string>

#include "gqa_serve.h"

namespace {

// A wrong argument: becomes a ValueError.
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

std::string text(at::IntArrayRef shape) {
    std::string s = "[";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// The address of a contiguous int32 tensor of this shape on CUDA device `dev`.
int* ints(const at::Tensor& t, const char* name, at::IntArrayRef shape, int dev) {
    if (t.scalar_type() != at::kInt || t.sizes() != shape || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
        refuse(std::string(name) + " must be a contiguous int32 CUDA tensor " + text(shape) + " on the same device");
    return static_cast<int*>(t.data_ptr());
}
int* ints(PyObject* o, const char* name, at::IntArrayRef shape, int dev) { return ints(tensor(o, name), name, shape, dev); }
int* ints_or_null(PyObject* o, const char* name, at::IntArrayRef shape, int dev) {
    return o == Py_None ? nullptr : ints(o, name, shape, dev);
}

int number(int64_t x, const char* name) {
    if (x < 0 || x > 0x7fffffff) refuse(std::string(name) + " is too large");
    return (int)x;
}

// Makes the device current, and the stream argument's stream: None (the device's own current
// one) or a torch.cuda.Stream.  Outputs are allocated with that stream current: a block that was
// freed on another one may still be in use there.
class On {
public:
    On(PyObject* o, int dev) : device_((c10::DeviceIndex)dev) {
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
            return;
        }
        PyObject* x = PyObject_GetAttrString(o, "cuda_stream");
        stream = x != nullptr ? PyLong_AsVoidPtr(x) : nullptr;
        Py_XDECREF(x);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            refuse("stream must be a torch.cuda.Stream");
        }
        given_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), (c10::DeviceIndex)dev));
    }
    void* stream = nullptr;

private:
    c10::cuda::CUDAGuard device_;
    std::optional<c10::cuda::CUDAStreamGuard> given_;
};

double scale_of(PyObject* o, int64_t d) {
    if (o == Py_None) return 1.0 / std::sqrt((double)d);
    const double x = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("scale must be a number");
    }
    return x;
}

bool truth(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) {
        PyErr_Clear();
        refuse("causal must be a truth value");
    }
    return x != 0;
}

// out and lse as given or new; bf16: 1 or 0 from out_dtype (used when out is not given).
struct Outputs {
    at::Tensor out, lse;
    int code;
};
Outputs outputs(PyObject* out, PyObject* lse, bool bf16, at::IntArrayRef out_shape, at::IntArrayRef lse_shape, int dev) {
    Outputs r;
    const auto cuda = at::TensorOptions().device(at::Device(at::kCUDA, (c10::DeviceIndex)dev));
    if (out == Py_None) {
        r.out = at::empty(out_shape, cuda.dtype(bf16 ? at::kBFloat16 : at::kFloat));
    } else {
        r.out = tensor(out, "out");
        if ((r.out.scalar_type() != at::kFloat && r.out.scalar_type() != at::kBFloat16) || !r.out.is_contiguous() ||
            !r.out.is_cuda() || r.out.get_device() != dev || r.out.sizes() != out_shape)
            refuse("out must be a contiguous fp32 or bf16 tensor " + text(out_shape) + " on q's device");
    }
    if (lse == Py_None) {
        r.lse = at::empty(lse_shape, cuda.dtype(at::kFloat));
    } else {
        r.lse = tensor(lse, "lse");
        if (r.lse.scalar_type() != at::kFloat || !r.lse.is_contiguous() || !r.lse.is_cuda() ||
            r.lse.get_device() != dev || r.lse.sizes() != lse_shape)
            refuse("lse must be a contiguous fp32 tensor " + text(lse_shape) + " on q's device");
    }
    r.code = r.out.scalar_type() == at::kBFloat16 ? GQA_OUT_BF16 : GQA_OUT_F32;
    return r;
}

PyObject* g_raise = nullptr;  // called with a status that is not GQA_OK

// NULL with the Python error set, when a call did not succeed.
bool failed(gqa_status st) {
    if (st == GQA_OK) return false;
    PyObject* r = PyObject_CallFunction(g_raise, "i", (int)st);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the call failed");
    return true;
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
    PyObject* x = THPVariable_Wrap(a);
    PyObject* y = x ? THPVariable_Wrap(b) : nullptr;
    PyObject* r = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

// Runs a call: C++ exceptions become Python's.
template <class F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
    try {
        if (given != wanted) refuse("wrong number of arguments");
        return f();
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {  // (an allocation that failed, for one)
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// The row stride of a bf16 tensor [n, H, d] whose heads are contiguous (0: contiguous rows).
long long rows(const at::Tensor& t, const char* name, int64_t H, int64_t d, int dev) {
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || !t.is_cuda() || t.get_device() != dev || t.size(1) != H ||
        t.size(2) != d)
        refuse(std::string(name) + " must be a bf16 CUDA tensor [rows, " + std::to_string(H) + ", " + std::to_string(d) +
               "] on q's device");
    if (t.is_contiguous() || t.numel() == 0) return 0;
    if (t.stride(2) != 1 || (H > 1 && t.stride(1) != d))
        refuse(std::string("the heads of a row of ") + name + " must be contiguous");
    if (t.size(0) <= 1) return 0;
    if (t.stride(0) < H * d || t.stride(0) % 8)
        refuse(std::string(name) + "'s rows must not overlap, and start a multiple of 8 elements apart");
    return t.stride(0);
}

// varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse, bf16, scale, causal, stream)
PyObject* varlen(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        const at::Tensor& cq = tensor(a[3], "cu_seqlens_q");
        if (!q.is_cuda() || q.dim() != 3 || k.dim() != 3) refuse("q, k and v must be CUDA tensors [rows, heads, d]");
        const int dev = (int)q.get_device();
        const int64_t tq = q.size(0), Hq = q.size(1), d = q.size(2), tk = k.size(0), Hk = k.size(1);
        const long long qs = rows(q, "q", Hq, d, dev), ks = rows(k, "k", Hk, d, dev), vs = rows(v, "v", Hk, d, dev);
        if (v.size(0) != tk) refuse("k and v must have the same shape");
        const int64_t bounds = cq.numel();
        if (bounds < 2) refuse("cu_seqlens_q must hold at least two bounds");
        const int* cqp = ints(cq, "cu_seqlens_q", {bounds}, dev);
        if (a[4] == Py_None && tk != tq) refuse("without cu_seqlens_k, k has as many rows as q");
        const int* ckp = a[4] == Py_None ? cqp : ints(a[4], "cu_seqlens_k", {bounds}, dev);
        const On on(a[10], dev);
        Outputs o = outputs(a[5], a[6], truth(a[7]), {tq, Hq, d}, {Hq, tq}, dev);
        const gqa_status st = gqa_attn_fwd_varlen(
            q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, cqp, ckp, o.out.data_ptr(), o.code,
            static_cast<float*>(o.lse.data_ptr()), number(bounds - 1, "the batch"), number(tq, "q"), number(tk, "k"),
            number(Hq, "Hq"), number(Hk, "Hk"), number(d, "d"), (float)scale_of(a[8], d), truth(a[9]), on.stream);
        return failed(st) ? nullptr : pair(o.out, o.lse);
    });
}

// tree(q, k_cache, v_cache, tree_mask, cache_seqlens, block_table, tree_lens, out, lse, bf16, scale, stream)
PyObject* tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache");
        const at::Tensor& mask = tensor(a[3], "tree_mask");
        if (!q.is_cuda() || q.dim() != 4 || k.dim() != 4)
            refuse("q must be a CUDA tensor [B, T, Hq, d], the cache [B, Sk, Hk, d] or [num_pages, page_size, Hk, d]");
        const int dev = (int)q.get_device();
        const int64_t B = q.size(0), T = q.size(1), Hq = q.size(2), d = q.size(3), Hk = k.size(2);
        for (const at::Tensor* t : {&q, &k, &v})
            if (t->scalar_type() != at::kBFloat16 || !t->is_contiguous() || !t->is_cuda() || t->get_device() != dev)
                refuse("q, k_cache and v_cache must be contiguous bf16 CUDA tensors on one device");
        if (k.sizes() != v.sizes() || k.size(3) != d) refuse("k_cache and v_cache must have one shape, with q's d");
        const int64_t words = (T + 31) / 32;
        const bool shared = mask.dim() == 2;
        const int* mp = shared ? ints(mask, "tree_mask", {T, words}, dev) : ints(mask, "tree_mask", {B, T, words}, dev);
        const int* lens = ints(a[4], "cache_seqlens", {B}, dev);
        const int* tl = ints_or_null(a[6], "tree_lens", {B}, dev);
        const int* table = nullptr;
        int M = 0, P = 0, page = 0, Sk = 0;
        if (a[5] == Py_None) {
            if (k.size(0) != B) refuse("without a block_table the cache is [B, Sk, Hk, d]");
            Sk = number(k.size(1), "the cache");
        } else {
            const at::Tensor& bt = tensor(a[5], "block_table");
            if (bt.dim() != 2) refuse("block_table must be [B, max_pages_per_seq]");
            table = ints(bt, "block_table", {B, bt.size(1)}, dev);
            M = number(bt.size(1), "block_table");
            P = number(k.size(0), "the pool");
            page = number(k.size(1), "the page size");
        }
        const On on(a[11], dev);
        Outputs o = outputs(a[7], a[8], truth(a[9]), {B, T, Hq, d}, {B, Hq, T}, dev);
        const gqa_status st = gqa_attn_fwd_tree(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), table, M, P, page, lens, mp, shared, tl, o.out.data_ptr(), o.code,
            static_cast<float*>(o.lse.data_ptr()), number(B, "B"), number(T, "T"), Sk, number(Hq, "Hq"), number(Hk, "Hk"),
            number(d, "d"), (float)scale_of(a[10], d), on.stream);
        return failed(st) ? nullptr : pair(o.out, o.lse);
    });
}

// The arrays that describe a cache's pages, from three arguments.
struct State {
    int *table, *lens, *refs;
    int S, M, P, dev;
};
State state(PyObject* const* a) {
    const at::Tensor &t = tensor(a[0], "block_table"), &r = tensor(a[2], "page_refs");
    if (!t.is_cuda() || t.dim() != 2 || r.dim() != 1)
        refuse("block_table must be a CUDA tensor [S, max_pages_per_seq], page_refs [num_pages]");
    State s;
    s.dev = (int)t.get_device();
    s.table = ints(t, "block_table", t.sizes(), s.dev);
    s.lens = ints(a[1], "cache_seqlens", {t.size(0)}, s.dev);
    s.refs = ints(r, "page_refs", r.sizes(), s.dev);
    s.S = number(t.size(0), "block_table");
    s.M = number(t.size(1), "block_table");
    s.P = number(r.size(0), "page_refs");
    return s;
}

struct PoolArgs {
    void *k, *v;
    int layers, page;
    long long row;
};
PoolArgs pools(PyObject* const* a, const State& s) {
    const at::Tensor &k = tensor(a[0], "k_pages"), &v = tensor(a[1], "v_pages");
    const int64_t dim = k.dim();
    if (k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type() || (dim != 4 && dim != 5))
        refuse("k_pages and v_pages must have one shape and type, [num_pages, page_size, Hk, d] or [layers, ...]");
    for (const at::Tensor* t : {&k, &v})
        if (!t->is_cuda() || t->get_device() != s.dev || !t->is_contiguous())
            refuse("k_pages and v_pages must be contiguous, on block_table's device");
    if (k.size(dim - 4) != s.P) refuse("page_refs must count as many pages as the pools have");
    if (k.data_ptr() == v.data_ptr()) refuse("k_pages and v_pages must be different tensors");
    PoolArgs p;
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    p.layers = dim == 5 ? number(k.size(0), "the layers") : 1;
    p.page = number(k.size(dim - 3), "the page size");
    p.row = (long long)k.size(dim - 1) * k.size(dim - 2) * k.element_size();
    return p;
}

at::Tensor status_of(PyObject* o, int64_t n, int dev) {
    if (o != Py_None) {
        const at::Tensor& t = tensor(o, "status");
        ints(t, "status", {n}, dev);
        return t;
    }
    return at::empty({n}, at::TensorOptions().device(at::Device(at::kCUDA, (c10::DeviceIndex)dev)).dtype(at::kInt));
}

// resize(block_table, cache_seqlens, page_refs, page_size, new_lens, slots, status, stream)
PyObject* resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const State s = state(a);
        const long page = PyLong_AsLong(a[3]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            refuse("page_size must be a whole number");
        }
        const int64_t m = tensor(a[4], "new_lens").numel();
        if (a[5] == Py_None && m > s.S) refuse("without slots there are at most as many lengths as slots");
        const int* nl = ints(a[4], "new_lens", {m}, s.dev);
        const int* sl = ints_or_null(a[5], "slots", {m}, s.dev);
        const On on(a[7], s.dev);
        at::Tensor st = status_of(a[6], m, s.dev);
        const gqa_status e = gqa_cache_resize(s.table, s.lens, s.refs, s.S, s.M, s.P, number(page < 0 ? 0 : page, "page_size"),
                                              sl, nl, number(m, "new_lens"), static_cast<int*>(st.data_ptr()),
                                              on.stream);
        return failed(e) ? nullptr : THPVariable_Wrap(st);
    });
}

// fork(k_pages, v_pages, block_table, cache_seqlens, page_refs, parents, children, status, stream)
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const State s = state(a + 2);
        const PoolArgs p = pools(a, s);
        const int64_t m = tensor(a[5], "parents").numel();
        const int *pa = ints(a[5], "parents", {m}, s.dev), *ch = ints(a[6], "children", {m}, s.dev);
        const On on(a[8], s.dev);
        at::Tensor st = status_of(a[7], m, s.dev);
        const gqa_status e = gqa_cache_fork(p.k, p.v, p.layers, p.row, s.table, s.lens, s.refs, s.S, s.M, s.P, p.page, pa, ch,
                                            number(m, "parents"), static_cast<int*>(st.data_ptr()), on.stream);
        return failed(e) ? nullptr : THPVariable_Wrap(st);
    });
}

// compact(k_pages, v_pages, block_table, cache_seqlens, page_refs, keep, keep_lens, tree_lens, status, stream)
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const State s = state(a + 2);
        const PoolArgs p = pools(a, s);
        const at::Tensor& keep = tensor(a[5], "keep");
        if (keep.dim() != 2) refuse("keep must be [S, T]");
        const int64_t T = keep.size(1);
        const int *kp = ints(keep, "keep", {s.S, T}, s.dev), *kl = ints(a[6], "keep_lens", {s.S}, s.dev);
        const int* tl = ints_or_null(a[7], "tree_lens", {s.S}, s.dev);
        const On on(a[9], s.dev);
        at::Tensor st = status_of(a[8], s.S, s.dev);
        const gqa_status e =
            gqa_cache_compact(p.k, p.v, p.layers, p.row, s.table, s.lens, s.refs, s.S, s.M, s.P, p.page, kp, kl, tl,
                              number(T, "T"), static_cast<int*>(st.data_ptr()), on.stream);
        return failed(e) ? nullptr : THPVariable_Wrap(st);
    });
}

// on_error(f): f(status) raises the package's error
PyObject* on_error(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XSETREF(g_raise, f);
    Py_RETURN_NONE;
}

// nvtx(): whether GQA_NVTX asks for ranges
PyObject* nvtx(PyObject*, PyObject*) {
    const char* e = std::getenv("GQA_NVTX");
    return PyBool_FromLong(e != nullptr && e[0] != '\0' && !(e[0] == '0' && e[1] == '\0'));
}

template <class F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {
    {"varlen", fast(varlen), METH_FASTCALL, nullptr},   {"tree", fast(tree), METH_FASTCALL, nullptr},
    {"resize", fast(resize), METH_FASTCALL, nullptr},   {"fork", fast(fork), METH_FASTCALL, nullptr},
    {"compact", fast(compact), METH_FASTCALL, nullptr}, {"on_error", on_error, METH_O, nullptr},
    {"nvtx", nvtx, METH_NOARGS, nullptr},               {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve_bind() { return PyModule_Create(&module); }
