// paged_binding.cpp -- the calls of paged.py in the usual case, without Python in between.
//
// A decode step makes a handful of calls whose kernels take 2 to 10 microseconds; checking and
// marshalling a dozen tensors in Python takes longer than that.  Each function here checks the same
// conditions as its namesake in paged.py, allocates its results and calls the C ABI.  It returns
//   None   when a condition does not hold or the call is out of the ordinary (another device is
//          current): paged.py then makes the call itself, or says what is wrong;
//   an int, the dcp_status of a call that the library refused;
//   else   the results (True where there are none).
// The library is the one paged.py loaded: set_library() takes its path.
#include <Python.h>
#include <dlfcn.h>

#include <cmath>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "dcp_paged.h"

namespace {

decltype(&dcp_paged_attention_workspace) f_workspace = nullptr;
decltype(&dcp_paged_attention) f_attention = nullptr;
decltype(&dcp_paged_attention_pack) f_attention_pack = nullptr;
decltype(&dcp_kv_append) f_append = nullptr;
decltype(&dcp_kv_weights) f_weights = nullptr;
decltype(&dcp_kv_evict) f_evict = nullptr;

PyObject *set_library(PyObject *, PyObject *path) {
    const char *name = PyUnicode_AsUTF8(path);
    if (!name) return nullptr;
    void *lib = dlopen(name, RTLD_NOW | RTLD_LOCAL);
    if (!lib) {
        PyErr_SetString(PyExc_OSError, dlerror());
        return nullptr;
    }
    f_workspace = reinterpret_cast<decltype(f_workspace)>(dlsym(lib, "dcp_paged_attention_workspace"));
    f_attention = reinterpret_cast<decltype(f_attention)>(dlsym(lib, "dcp_paged_attention"));
    f_attention_pack = reinterpret_cast<decltype(f_attention_pack)>(dlsym(lib, "dcp_paged_attention_pack"));
    f_append = reinterpret_cast<decltype(f_append)>(dlsym(lib, "dcp_kv_append"));
    f_weights = reinterpret_cast<decltype(f_weights)>(dlsym(lib, "dcp_kv_weights"));
    f_evict = reinterpret_cast<decltype(f_evict)>(dlsym(lib, "dcp_kv_evict"));
    if (!f_workspace || !f_attention || !f_attention_pack || !f_append || !f_weights || !f_evict) {
        PyErr_SetString(PyExc_OSError, "the library lacks a paged entry point");
        return nullptr;
    }
    Py_RETURN_NONE;
}

// ---- arguments: each returns false where paged.py has to look ---------------------------------
struct Args {
    PyObject *const *a;
    int device = -1;  // of every tensor so far
    bool ok = true;

    // Argument i as a CUDA tensor on the device of the others; null (and !ok) if it is none.
    const at::Tensor *tensor(int i) {
        if (!THPVariable_Check(a[i])) return ok = false, nullptr;
        const at::Tensor &t = THPVariable_Unpack(a[i]);
        if (!t.is_cuda()) return ok = false, nullptr;
        const int d = t.get_device();
        if (device < 0) device = d;
        if (d != device) return ok = false, nullptr;
        return &t;
    }
    const at::Tensor *optional(int i) { return a[i] == Py_None ? nullptr : tensor(i); }
    int64_t integer(int i) {
        if (!PyLong_Check(a[i])) return ok = false, 0;
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    int32_t small(int i) {
        const int64_t v = integer(i);
        if (v < INT32_MIN || v > INT32_MAX) ok = false;
        return static_cast<int32_t>(v);
    }
    int32_t truth(int i) {
        const int v = PyObject_IsTrue(a[i]);
        if (v < 0) {
            PyErr_Clear();
            ok = false;
        }
        return v > 0;
    }
    bool current() const { return ok && f_attention && device >= 0 && c10::cuda::current_device() == device; }
    void *stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
};

int32_t code_of(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return DCP_BF16;
        case at::kHalf: return DCP_FP16;
        case at::kFloat: return DCP_FP32;
        default: return -1;
    }
}

bool inner(const at::Tensor &t) { return t.size(-1) <= 1 || t.stride(-1) == 1; }

bool lengths(const at::Tensor *t, int64_t n) {
    return t && t->scalar_type() == at::kInt && t->dim() == 1 && t->size(0) == n && t->is_contiguous();
}

// fp32 [n0, n1, any], contiguous in its last dimension
bool rows(const at::Tensor *t, int64_t n0, int64_t n1) {
    return t && t->scalar_type() == at::kFloat && t->dim() == 3 && t->size(0) == n0 && t->size(1) == n1 && inner(*t);
}

bool cache(const at::Tensor *k, const at::Tensor *v, const at::Tensor *table, int64_t requests, dcp_paged_kv &kv) {
    if (!k || !v || !table || k->dim() != 4 || v->sizes() != k->sizes() || v->scalar_type() != k->scalar_type() ||
        !inner(*k) || !inner(*v) || table->scalar_type() != at::kInt || table->dim() != 2 ||
        table->size(0) != requests || !inner(*table))
        return false;
    const int32_t code = code_of(k->scalar_type());
    if (code < 0 || k->size(1) > INT32_MAX || k->size(2) > INT32_MAX || k->size(3) > INT32_MAX) return false;
    kv = {k->data_ptr(), v->data_ptr(), static_cast<const int32_t *>(table->data_ptr()), k->size(0), k->stride(0),
          k->stride(1), k->stride(2), v->stride(0), v->stride(1), v->stride(2), table->stride(0), table->size(1),
          static_cast<int32_t>(k->size(1)), static_cast<int32_t>(k->size(2)), static_cast<int32_t>(k->size(3)), code};
    return true;
}

const float *floats(const at::Tensor &t) { return static_cast<const float *>(t.data_ptr()); }
const int32_t *ints(const at::Tensor &t) { return static_cast<const int32_t *>(t.data_ptr()); }

// Runs f; an exception (memory, above all) leaves the call to paged.py.
template <class F>
PyObject *guarded(F &&f) {
    try {
        return f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// Workspace of one call, in the order of its stream.
struct Scratch {
    void *p = nullptr;
    Scratch(int64_t n, void *stream) {
        if (n > 0) p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(n, static_cast<cudaStream_t>(stream));
    }
    ~Scratch() {
        if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
    }
    Scratch(const Scratch &) = delete;
};

// attend(q, k, v, table, seq_lens, world_size or 0, scale or None, shard, num_shards, interleave, logits or
// None, base_e, result or None, lse or None): world_size 0 -> (result, lse) or True, else the send buffer or True
PyObject *attend(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 14) Py_RETURN_NONE;
        Args a{argv};
        const at::Tensor *q = a.tensor(0), *k = a.tensor(1), *v = a.tensor(2), *table = a.tensor(3),
                         *seq = a.tensor(4), *logits = a.optional(10), *result = a.optional(12),
                         *lse = a.optional(13);
        const int64_t world = a.integer(5);
        const int32_t shard = a.small(7), shards = a.small(8), interleave = a.small(9), base_e = a.truth(11);
        dcp_paged_kv kv;
        if (!a.current() || q->dim() != 3) Py_RETURN_NONE;
        const int64_t B = q->size(0), H = q->size(1), D = q->size(2);
        if (!cache(k, v, table, B, kv) || !lengths(seq, B) || D != kv.head_dim || D == 0 ||
            q->scalar_type() != k->scalar_type() || !inner(*q) || (logits && !rows(logits, B, H)))
            Py_RETURN_NONE;
        float scale;
        if (argv[6] == Py_None) {
            scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
        } else if (PyFloat_Check(argv[6])) {
            scale = static_cast<float>(PyFloat_AS_DOUBLE(argv[6]));
        } else {
            Py_RETURN_NONE;
        }
        const int P = kv.dtype == DCP_FP32 ? 1 : 2;
        at::Tensor out, sums;  // what this call allocates
        if (world == 0) {
            if ((result == nullptr) != (lse == nullptr)) Py_RETURN_NONE;
            if (result) {
                if (result->sizes() != q->sizes() || result->scalar_type() != q->scalar_type() ||
                    !result->is_contiguous() || lse->dim() != 2 || lse->size(0) != B || lse->size(1) != H ||
                    lse->scalar_type() != at::kFloat || !lse->is_contiguous())
                    Py_RETURN_NONE;
            } else {
                out = at::empty({B, H, D}, q->options());
                sums = at::empty({B, H}, q->options().dtype(at::kFloat));
            }
        } else {
            if (world < 1 || world > DCP_MAX_SHARDS || H % world || lse) Py_RETURN_NONE;
            if (result) {
                if (result->dim() != 4 || result->size(0) != world || result->size(1) != B ||
                    result->size(2) != H / world || result->size(3) != D + P ||
                    result->scalar_type() != q->scalar_type() || !result->is_contiguous())
                    Py_RETURN_NONE;
            } else {
                out = at::empty({world, B, H / world, D + P}, q->options());
            }
        }
        const at::Tensor &to = result ? *result : out;
        void *stream = a.stream();
        const int64_t bytes = f_workspace(H, kv.heads, kv.head_dim, kv.dtype);
        const Scratch ws(bytes, stream);
        float *lg = logits ? static_cast<float *>(logits->data_ptr()) : nullptr;
        const int64_t lb = logits ? logits->stride(0) : 0, lh = logits ? logits->stride(1) : 0,
                      cap = logits ? logits->size(2) : 0;
        int32_t st;
        if (world == 0) {
            float *ls = static_cast<float *>((lse ? *lse : sums).data_ptr());
            st = f_attention(&kv, q->data_ptr(), ints(*seq), to.data_ptr(), ls, lg, B, H, q->stride(0), q->stride(1),
                             lb, lh, cap, scale, shard, shards, interleave, base_e, ws.p, bytes, stream);
        } else {
            st = f_attention_pack(&kv, q->data_ptr(), ints(*seq), to.data_ptr(), lg, B, H,
                                  static_cast<int32_t>(world), q->stride(0), q->stride(1), lb, lh, cap, scale, shard,
                                  shards, interleave, base_e, ws.p, bytes, stream);
        }
        if (st != DCP_OK) return PyLong_FromLong(st);
        if (result) Py_RETURN_TRUE;
        if (world) return THPVariable_Wrap(out);
        PyObject *pair = PyTuple_New(2);
        if (!pair) return nullptr;
        PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(out));
        PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(sums));
        return pair;
    });
}

// append(k_new, v_new, k, v, table, seq_lens, query_start_loc, shard, num_shards, interleave) -> True
PyObject *append(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 10) Py_RETURN_NONE;
        Args a{argv};
        const at::Tensor *kn = a.tensor(0), *vn = a.tensor(1), *k = a.tensor(2), *v = a.tensor(3),
                         *table = a.tensor(4), *seq = a.tensor(5), *starts = a.tensor(6);
        const int32_t shard = a.small(7), shards = a.small(8), interleave = a.small(9);
        dcp_paged_kv kv;
        if (!a.current() || seq->dim() != 1) Py_RETURN_NONE;
        const int64_t R = seq->size(0);
        if (R > INT32_MAX || !lengths(seq, R) || !lengths(starts, R + 1) || !cache(k, v, table, R, kv)) Py_RETURN_NONE;
        for (const at::Tensor *t : {kn, vn})
            if (t->dim() != 3 || t->size(0) != kn->size(0) || t->size(1) != kv.heads || t->size(2) != kv.head_dim ||
                t->scalar_type() != k->scalar_type() || !inner(*t))
                Py_RETURN_NONE;
        const int32_t st = f_append(&kv, kn->data_ptr(), vn->data_ptr(), ints(*seq), ints(*starts), kn->size(0),
                                    static_cast<int32_t>(R), kn->stride(0), kn->stride(1), vn->stride(0),
                                    vn->stride(1), shard, shards, interleave, a.stream());
        if (st != DCP_OK) return PyLong_FromLong(st);
        Py_RETURN_TRUE;
    });
}

// weigh(logits, lse, seq_lens, weights, shard, num_shards, interleave, base_e) -> True
PyObject *weigh(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 8) Py_RETURN_NONE;
        Args a{argv};
        const at::Tensor *logits = a.tensor(0), *lse = a.tensor(1), *seq = a.tensor(2), *w = a.tensor(3);
        const int32_t shard = a.small(4), shards = a.small(5), interleave = a.small(6), base_e = a.truth(7);
        if (!a.current() || logits->dim() != 3 || w->dim() != 3) Py_RETURN_NONE;
        const int64_t B = logits->size(0), H = logits->size(1), heads = w->size(1);
        if (!rows(logits, B, H) || !rows(w, B, heads) || !lengths(seq, B) || lse->dim() != 2 || lse->size(0) != B ||
            lse->size(1) != H || lse->scalar_type() != at::kFloat)
            Py_RETURN_NONE;
        const int64_t cap = std::min(logits->size(2), w->size(2));
        const int32_t st = f_weights(floats(*logits), floats(*lse), ints(*seq), static_cast<float *>(w->data_ptr()), B,
                                     H, heads, cap, logits->stride(0), logits->stride(1), lse->stride(0),
                                     lse->stride(1), w->stride(0), w->stride(1), shard, shards, interleave, base_e,
                                     a.stream());
        if (st != DCP_OK) return PyLong_FromLong(st);
        Py_RETURN_TRUE;
    });
}

// evict(weights, k, v, table, seq_lens, k_out, v_out, new_table, keep, recent, shard, num_shards, interleave)
// -> (kept, new_lens, new_weights)
PyObject *evict(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 13) Py_RETURN_NONE;
        Args a{argv};
        const at::Tensor *w = a.tensor(0), *k = a.tensor(1), *v = a.tensor(2), *table = a.tensor(3),
                         *seq = a.tensor(4), *ko = a.tensor(5), *vo = a.tensor(6), *new_table = a.tensor(7);
        const int64_t keep = a.integer(8), recent = a.integer(9);
        const int32_t shard = a.small(10), shards = a.small(11), interleave = a.small(12);
        dcp_paged_kv src, dst;
        if (!a.current() || seq->dim() != 1 || keep < 1) Py_RETURN_NONE;
        const int64_t B = seq->size(0);
        if (!lengths(seq, B) || !cache(k, v, table, B, src) || !cache(ko, vo, new_table, B, dst) ||
            !rows(w, B, src.heads))
            Py_RETURN_NONE;
        const int64_t cap = w->size(2), new_cap = std::max(cap, keep);
        const at::Tensor kept = at::empty({B, src.heads, keep}, w->options().dtype(at::kInt));
        const at::Tensor lens = at::empty({B}, w->options().dtype(at::kInt));
        const at::Tensor nw = at::empty({B, src.heads, new_cap}, w->options());
        const int32_t st = f_evict(&src, &dst, ints(*seq), floats(*w), static_cast<float *>(nw.data_ptr()),
                                   static_cast<int32_t *>(kept.data_ptr()), static_cast<int32_t *>(lens.data_ptr()),
                                   B, cap, new_cap, w->stride(0), w->stride(1), nw.stride(0), nw.stride(1), keep,
                                   recent, shard, shards, interleave, a.stream());
        if (st != DCP_OK) return PyLong_FromLong(st);
        PyObject *all = PyTuple_New(3);
        if (!all) return nullptr;
        PyTuple_SET_ITEM(all, 0, THPVariable_Wrap(kept));
        PyTuple_SET_ITEM(all, 1, THPVariable_Wrap(lens));
        PyTuple_SET_ITEM(all, 2, THPVariable_Wrap(nw));
        return all;
    });
}

PyMethodDef methods[] = {
    {"set_library", set_library, METH_O, "Loads the entry points of the library at this path."},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"weigh", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(weigh)), METH_FASTCALL, nullptr},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(evict)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__paged_binding() { return PyModule_Create(&module); }
