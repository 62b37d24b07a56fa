// marshal.cpp -- argument marshalling of the calls on rotated rows and 8-bit
// pools, for binding.py: checks of the tensors, the C ABI's descriptors and
// pointers, the outputs that the caller did not give, and the current stream.
// A step of a few short sequences takes the GPU 2 to 6 us; the same checks in
// Python took the host 9 to 18 us, and 52 us for the caches of 40 layers.
//
// Every call returns its output (or None); it raises ValueError where a tensor
// is not what the call takes, and binding.py's error, which bind() is given,
// where the library refused.  The library itself is libpagedkv.so, whose entry
// points bind() looks up.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <stdexcept>
#include <vector>

#include "../../include/pagedkv.h"

namespace {

decltype(&paged_kv_append_rope) p_append_rope = nullptr;
decltype(&paged_kv_append_rope_fp8) p_append_rope_fp8 = nullptr;
decltype(&paged_attention_decode_fp8) p_decode_fp8 = nullptr;
decltype(&paged_attention_workspace_bytes) p_workspace_bytes = nullptr;
decltype(&copy_blocks_fp8) p_copy_blocks_fp8 = nullptr;
PyObject* refused = nullptr;  // exception of (status, call)

// Becomes Python's ValueError.
struct BadValue : std::runtime_error {
    using std::runtime_error::runtime_error;
};
void require(bool ok, const char* what) {
    if (!ok) throw BadValue(what);
}

int32_t dtype_code(c10::ScalarType t) {
    switch (t) {
        case c10::ScalarType::BFloat16: return PKV_BF16;
        case c10::ScalarType::Half: return PKV_FP16;
        case c10::ScalarType::Float: return PKV_FP32;
        case c10::ScalarType::Float8_e4m3fn: return PKV_E4M3;
        default: return -1;  // the library refuses it
    }
}

const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) throw BadValue("a tensor is needed");
    return THPVariable_Unpack(o);
}
// None: nullptr
const at::Tensor* maybe(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }
void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// The device of a call: that of its first tensor, which all the others share.
struct Device {
    c10::DeviceIndex index = -1;
    void same(const at::Tensor& t) {
        require(t.is_cuda(), "tensors must be on one CUDA device");
        if (index < 0) index = t.get_device();
        require(t.get_device() == index, "tensors must be on one CUDA device");
    }
    void whole(const at::Tensor* t) {
        if (!t) return;
        same(*t);
        require(t->is_contiguous(), "tensors must be contiguous");
    }
};

bool shaped(const at::Tensor& t, std::initializer_list<int64_t> s) {
    return t.sizes() == c10::IntArrayRef(s.begin(), s.size());
}

int32_t narrow(int64_t v) {
    require(v >= INT32_MIN && v <= INT32_MAX, "a size does not fit 32 bits");
    return (int32_t)v;
}

pkv_cache_desc cache_of(const at::Tensor& k, const at::Tensor& v) {
    require(k.dim() == 4 && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type(),
            "caches must be [num_blocks, num_kv_heads, block_size, head_dim], K as V");
    return {k.size(0), narrow(k.size(1)), narrow(k.size(2)), narrow(k.size(3)), dtype_code(k.scalar_type())};
}

void scales_of(const at::Tensor* s, const pkv_cache_desc& c) {
    require(s && s->scalar_type() == c10::ScalarType::Float && shaped(*s, {c.num_blocks, c.num_kv_heads}),
            "scales must be fp32 [num_blocks, num_kv_heads]");
}

// Elements from one token's row to the next of q, k or v.
int64_t token_stride(const at::Tensor& t, int64_t n, int64_t heads, int64_t d, c10::ScalarType dt, Device& dev) {
    dev.same(t);
    require(t.dim() == 3 && shaped(t, {n, heads, d}) && t.scalar_type() == dt,
            "q is [num_tokens, num_q_heads, head_dim], k and v [num_tokens, num_kv_heads, head_dim], of one dtype");
    require((t.stride(2) == 1 || d == 1) && (t.stride(1) == d || heads == 1),
            "a token's heads must be contiguous in q, k and v");
    return n > 1 ? t.stride(0) : heads * d;
}

// Other threads run while a call is issued.  (The calls of the C ABI throw
// nothing; what may throw -- a tensor without memory of its own has no pointer
// to give, a size may not fit -- is evaluated before the lock is given up, and
// the lock comes back however the scope is left.)
class Unlocked {
    PyThreadState* const state_ = PyEval_SaveThread();

  public:
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state_); }
};

PyObject* result(pkv_status st, const char* call, const at::Tensor* out) {
    if (st != PKV_OK) {
        PyObject* e = PyObject_CallFunction(refused, "is", (int)st, call);
        if (e) {
            PyErr_SetObject(refused, e);
            Py_DECREF(e);
        }
        return nullptr;
    }
    if (!out) Py_RETURN_NONE;
    return THPVariable_Wrap(*out);
}

// fp8, q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, k_scales, v_scales, q_norm, k_norm, norm_eps,
// interleaved, q_out
PyObject* append_rope(PyObject* const* a) {
    const bool fp8 = a[0] == Py_True;
    const at::Tensor *q = maybe(a[1]), &k = tensor(a[2]), &v = tensor(a[3]), *positions = maybe(a[4]),
                     *cos_sin = maybe(a[5]), &slots = tensor(a[6]), &k_cache = tensor(a[7]), &v_cache = tensor(a[8]),
                     *k_scales = maybe(a[9]), *v_scales = maybe(a[10]), *q_norm = maybe(a[11]), *k_norm = maybe(a[12]);
    const double eps = PyFloat_AsDouble(a[13]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const int inter = PyObject_IsTrue(a[14]);
    if (inter < 0) return nullptr;
    const at::Tensor* q_out = maybe(a[15]);

    Device dev;
    for (const at::Tensor* t : {&k_cache, &v_cache, &slots, positions, cos_sin, k_scales, v_scales, q_norm, k_norm, q_out})
        dev.whole(t);
    const pkv_cache_desc cache = cache_of(k_cache, v_cache);
    const int64_t d = cache.head_dim, hkv = cache.num_kv_heads;
    const c10::ScalarType dt = k.scalar_type();
    require(slots.scalar_type() == c10::ScalarType::Long && slots.dim() == 1, "slot_mapping must be int64 [num_tokens]");
    const int64_t n = slots.numel();
    pkv_rope_desc rope = {};
    rope.dtype = dtype_code(dt);
    rope.k_stride = token_stride(k, n, hkv, d, dt, dev);
    rope.v_stride = token_stride(v, n, hkv, d, dt, dev);
    if (q) {
        require(q->dim() == 3, "q is [num_tokens, num_q_heads, head_dim]");
        rope.num_q_heads = narrow(q->size(1));
        rope.q_stride = token_stride(*q, n, q->size(1), d, dt, dev);
        require(!q_out || (q_out->sizes() == q->sizes() && q_out->scalar_type() == dt), "q_out is as q");
    } else {
        require(!q_out && !q_norm, "q_out and q_norm belong to q");
    }
    // without cos_sin positions may stand there (a layer that rotates nothing, called like its neighbours) unread
    require(!positions || (positions->scalar_type() == c10::ScalarType::Long && shaped(*positions, {n})),
            "positions must be int64 [num_tokens]");
    if (cos_sin) {
        require(positions, "cos_sin needs positions");
        require(cos_sin->scalar_type() == c10::ScalarType::Float && cos_sin->dim() == 2 && cos_sin->size(1) > 0,
                "cos_sin must be fp32 [max_position, rot_dim] (None: no rotation)");
        rope.max_position = cos_sin->size(0);
        rope.rot_dim = narrow(cos_sin->size(1));
    }
    for (const at::Tensor* w : {q_norm, k_norm})
        require(!w || (w->scalar_type() == dt && shaped(*w, {d})), "norm weights are [head_dim], of k's dtype");
    if (fp8) {
        scales_of(k_scales, cache);
        scales_of(v_scales, cache);
    }
    rope.interleaved = inter;
    rope.norm_eps = (float)eps;

    const c10::cuda::CUDAGuard guard(dev.index);
    at::Tensor made;
    if (q && !q_out) {
        made = at::empty(q->sizes(), q->options());
        q_out = &made;
    }
    void* stream = c10::cuda::getCurrentCUDAStream(dev.index).stream();
    void *p_q = ptr(q), *p_k = ptr(&k), *p_v = ptr(&v), *p_qn = ptr(q_norm), *p_kn = ptr(k_norm), *p_out = ptr(q_out),
         *p_kc = ptr(&k_cache), *p_vc = ptr(&v_cache);
    const auto p_pos = static_cast<const int64_t*>(ptr(positions)), p_slots = static_cast<const int64_t*>(ptr(&slots));
    const auto p_table = static_cast<const float*>(ptr(cos_sin));
    const auto p_ks = static_cast<float*>(ptr(k_scales)), p_vs = static_cast<float*>(ptr(v_scales));
    pkv_status st;
    {
        const Unlocked unlocked;
        st = fp8 ? p_append_rope_fp8(p_q, p_k, p_v, p_pos, p_table, p_qn, p_kn, p_slots, n, p_out, p_kc, p_vc, p_ks, p_vs,
                                     &cache, &rope, stream)
                 : p_append_rope(p_q, p_k, p_v, p_pos, p_table, p_qn, p_kn, p_slots, n, p_out, p_kc, p_vc, &cache, &rope,
                                 stream);
    }
    return result(st, fp8 ? "paged_kv_append_rope_fp8" : "paged_kv_append_rope", q_out);
}

// q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale, out, max_context_len, partition_size,
// workspace, out_dtype
PyObject* decode_fp8(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0]), &k_cache = tensor(a[1]), &v_cache = tensor(a[2]), &k_scales = tensor(a[3]),
                     &v_scales = tensor(a[4]), &tables = tensor(a[5]), &lens = tensor(a[6]);
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    const at::Tensor* out = maybe(a[8]);
    const int64_t asked = a[9] == Py_None ? -1 : PyLong_AsLongLong(a[9]);
    if (asked == -1 && PyErr_Occurred()) return nullptr;
    const int64_t partition = PyLong_AsLongLong(a[10]);
    if (partition == -1 && PyErr_Occurred()) return nullptr;
    const at::Tensor* workspace = maybe(a[11]);
    require(THPDtype_Check(a[12]), "out_dtype is a torch dtype");

    Device dev;
    for (const at::Tensor* t : {&q, &k_cache, &v_cache, &k_scales, &v_scales, &tables, &lens, out, workspace}) dev.whole(t);
    const pkv_cache_desc cache = cache_of(k_cache, v_cache);
    require(q.dim() == 3 && q.size(2) == cache.head_dim && (!out || out->sizes() == q.sizes()),
            "q and out are [num_seqs, num_q_heads, head_dim]");
    const int32_t num_seqs = narrow(q.size(0)), hq = narrow(q.size(1));
    require(tables.scalar_type() == c10::ScalarType::Int && tables.dim() == 2 && tables.size(0) == num_seqs,
            "block_tables must be int32 [num_seqs, max_blocks_per_seq]");
    require(lens.scalar_type() == c10::ScalarType::Int && shaped(lens, {num_seqs}), "context_lens must be int32 [num_seqs]");
    scales_of(&k_scales, cache);
    scales_of(&v_scales, cache);
    const int32_t max_len = narrow(a[9] == Py_None ? tables.size(1) * cache.block_size : asked), part = narrow(partition);

    const c10::cuda::CUDAGuard guard(dev.index);
    at::Tensor made, space;
    if (!out) {
        made = at::empty(q.sizes(), q.options().dtype(reinterpret_cast<THPDtype*>(a[12])->scalar_type));
        out = &made;
    }
    if (!workspace) {
        const size_t need = p_workspace_bytes(num_seqs, hq, cache.head_dim, max_len, part);
        if (need) {
            space = at::empty({(int64_t)need}, q.options().dtype(c10::ScalarType::Byte));
            workspace = &space;
        }
    }
    void* stream = c10::cuda::getCurrentCUDAStream(dev.index).stream();
    void *p_q = ptr(&q), *p_kc = ptr(&k_cache), *p_vc = ptr(&v_cache), *p_out = ptr(out), *p_space = ptr(workspace);
    const auto p_ks = static_cast<const float*>(ptr(&k_scales)), p_vs = static_cast<const float*>(ptr(&v_scales));
    const auto p_tables = static_cast<const int32_t*>(ptr(&tables)), p_lens = static_cast<const int32_t*>(ptr(&lens));
    const int32_t width = narrow(tables.size(1)), q_type = dtype_code(q.scalar_type()), out_type = dtype_code(out->scalar_type());
    const size_t space_bytes = workspace ? workspace->nbytes() : 0;
    pkv_status st;
    {
        const Unlocked unlocked;
        st = p_decode_fp8(p_q, q_type, p_kc, p_vc, p_ks, p_vs, p_tables, width, p_lens, num_seqs, hq, max_len, (float)scale,
                          p_out, out_type, &cache, part, p_space, space_bytes, stream);
    }
    return result(st, "paged_attention_decode_fp8", out);
}

// k_caches, v_caches, k_scales, v_scales (lists of one tensor per layer), src_dst_pairs
PyObject* copy_fp8(PyObject* const* a) {
    const at::Tensor& pairs = tensor(a[4]);
    Py_ssize_t layers = -1;
    Device dev;
    dev.whole(&pairs);
    pkv_cache_desc cache = {};
    std::vector<void*> ptrs[4];
    for (int i = 0; i < 4; ++i) {
        require(PyList_Check(a[i]), "lists of one tensor per layer");
        const Py_ssize_t n = PyList_GET_SIZE(a[i]);
        require(n > 0 && (layers < 0 || n == layers), "need one K and one V cache per layer, and their scales");
        layers = n;
        ptrs[i].reserve(n);
        for (Py_ssize_t l = 0; l < n; ++l) {
            const at::Tensor& t = tensor(PyList_GET_ITEM(a[i], l));
            dev.whole(&t);
            if (i == 0 && l == 0) cache = cache_of(t, t);
            if (i < 2)
                require(shaped(t, {cache.num_blocks, cache.num_kv_heads, cache.block_size, cache.head_dim}) &&
                            dtype_code(t.scalar_type()) == cache.dtype,
                        "the caches differ");
            else
                scales_of(&t, cache);
            ptrs[i].push_back(t.data_ptr());
        }
    }
    require(pairs.scalar_type() == c10::ScalarType::Long && pairs.numel() % 2 == 0, "src_dst_pairs must be int64 [n, 2]");
    const c10::cuda::CUDAGuard guard(dev.index);
    void* stream = c10::cuda::getCurrentCUDAStream(dev.index).stream();
    const int32_t n_layers = narrow(layers), n_pairs = narrow(pairs.numel() / 2);
    const auto p_pairs = static_cast<const int64_t*>(ptr(&pairs));
    pkv_status st;
    {
        const Unlocked unlocked;
        st = p_copy_blocks_fp8(ptrs[0].data(), ptrs[1].data(), reinterpret_cast<float* const*>(ptrs[2].data()),
                               reinterpret_cast<float* const*>(ptrs[3].data()), n_layers, p_pairs, n_pairs, &cache, stream);
    }
    return result(st, "copy_blocks_fp8", nullptr);
}

// No C++ exception passes into Python.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, and %zd are needed", n, N);
        return nullptr;
    }
    if (!p_append_rope) {
        PyErr_SetString(PyExc_RuntimeError, "bind() comes first");
        return nullptr;
    }
    try {
        return F(args);
    } catch (const BadValue& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject* bind(PyObject*, PyObject* args) {
    const char* p;
    PyObject* error;
    if (!PyArg_ParseTuple(args, "sO", &p, &error)) return nullptr;
    void* lib = dlopen(p, RTLD_NOW | RTLD_LOCAL);  // the handle that ctypes opened
    if (!lib) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    const auto find = [&](auto& f, const char* name) {
        f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(lib, name));
        return f != nullptr;
    };
    if (!find(p_workspace_bytes, "paged_attention_workspace_bytes") || !find(p_decode_fp8, "paged_attention_decode_fp8") ||
        !find(p_copy_blocks_fp8, "copy_blocks_fp8") || !find(p_append_rope_fp8, "paged_kv_append_rope_fp8") ||
        !find(p_append_rope, "paged_kv_append_rope")) {
        p_append_rope = nullptr;
        PyErr_SetString(PyExc_RuntimeError, "libpagedkv.so lacks an entry point");
        return nullptr;
    }
    Py_INCREF(error);
    Py_XSETREF(refused, error);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "Looks the entry points up in libpagedkv.so: its path, and the error of a refusal."},
    {"append_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<append_rope, 16>)), METH_FASTCALL, nullptr},
    {"decode_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<decode_fp8, 13>)), METH_FASTCALL, nullptr},
    {"copy_blocks_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<copy_fp8, 5>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
