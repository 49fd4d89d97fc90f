// Argument marshalling of the serving entry points for Python (latent_chunk,
// page_*, verify_drafts): torch tensors are checked, outputs are allocated and
// the C entry points of include/kda.h are called on torch's current stream.
//
// These calls are a few microseconds of GPU time, and through ctypes they took
// 14 to 16 on the host, half of it in checks, allocations and conversions that
// Python did one by one; here 6 to 8.
//
// Each function takes its arguments by position and returns its tensors, or a
// kda_status that is not KDA_OK as a number, or None where an argument is not
// as documented: the Python wrapper then says what is wrong.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <vector>

#include "kda.h"

namespace {

using at::Tensor;

constexpr int64_t STATUS_BYTES = 256;
constexpr int64_t ROW = 576, LATENT = 512, QUERY = 192, EXPANDED = 256, VALUE = 128;

bool fits(int64_t x) { return x >= 0 && x <= INT_MAX; }

// A whole number of 32 bits that is not negative.
bool whole(PyObject* o, int64_t& x) {
    if (PyFloat_Check(o)) {
        const double d = PyFloat_AS_DOUBLE(o);
        if (!(d >= 0 && d <= INT_MAX && d == (double)(int64_t)d)) return false;
        x = (int64_t)d;
        return true;
    }
    if (!PyIndex_Check(o)) return false;
    PyObject* i = PyNumber_Index(o);
    if (i == nullptr) {
        PyErr_Clear();
        return false;
    }
    int overflow = 0;
    x = PyLong_AsLongLongAndOverflow(i, &overflow);
    Py_DECREF(i);
    return overflow == 0 && fits(x);
}

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// Tensors of one call: all on one GPU.
struct Call {
    int64_t device = -1;
    bool fine = true;
    // A tensor argument of a type and number of dimensions; nullptr, and the call refused, where it is not that.
    const Tensor* take(PyObject* o, at::ScalarType type, int64_t dim) {
        const Tensor* t = tensor(o);
        if (t == nullptr || t->scalar_type() != type || t->dim() != dim || !t->is_cuda()) return refuse();
        if (device < 0) device = t->get_device();
        else if (t->get_device() != device) return refuse();
        return t;
    }
    const Tensor* ints(PyObject* o, int64_t dim) { return take(o, at::kInt, dim); }
    // One of those, or None.
    const Tensor* maybe(PyObject* o, at::ScalarType type, int64_t dim) { return o == Py_None ? nullptr : take(o, type, dim); }
    const Tensor* refuse() {
        fine = false;
        return nullptr;
    }
    bool sizes(std::initializer_list<int64_t> all) {
        for (int64_t x : all) fine = fine && fits(x);
        return fine;
    }
    // The status header, or nullptr.
    void* header(PyObject* o) {
        if (o == Py_None) return nullptr;
        const Tensor* t = memory(o);
        if (t == nullptr || (int64_t)t->nbytes() < STATUS_BYTES) return fine = false, nullptr;
        return t->data_ptr();
    }
    // A workspace of any type in one piece.
    const Tensor* memory(PyObject* o) {
        const Tensor* t = tensor(o);
        if (t == nullptr || !t->is_cuda() || t->get_device() != device || !t->is_contiguous()) return refuse();
        return t;
    }
};

Tensor fresh(at::IntArrayRef sizes, const Tensor& like, at::ScalarType type) { return at::empty(sizes, like.options().dtype(type)); }

// In one piece, on 16 bytes: the kernels read 16 at a time.
Tensor in_place(const Tensor& t) {
    Tensor c = t.contiguous();
    return reinterpret_cast<uintptr_t>(c.data_ptr()) % 16 == 0 ? c : c.clone();
}

const int32_t* i32(const Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }
int32_t* i32_out(const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

PyObject* result(kda_status status, std::initializer_list<Tensor> outputs) {
    if (status != KDA_OK) return PyLong_FromLong(status);
    PyObject* tuple = PyTuple_New((Py_ssize_t)outputs.size());
    Py_ssize_t at = 0;
    for (const Tensor& t : outputs) PyTuple_SET_ITEM(tuple, at++, THPVariable_Wrap(t));
    return tuple;
}

// A launch may have to wait for room in the stream's queue: other threads go on meanwhile.
template <typename F>
kda_status launch(F f) {
    PyThreadState* state = PyEval_SaveThread();
    const kda_status status = f();
    PyEval_RestoreThread(state);
    return status;
}

cudaStream_t stream_of(int64_t device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

#define MARSHAL(name, count)                                                             \
    PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {                        \
        HANDLE_TH_ERRORS                                                                 \
        if (n != count) {                                                                \
            PyErr_SetString(PyExc_TypeError, #name ": number of arguments");             \
            return nullptr;                                                              \
        }

// block_table, seq_lens, parents, children, refs, free_pages, free_head, page_size, fork_lens, workspace
MARSHAL(page_fork, 10)
    Call c;
    const Tensor *table = c.ints(a[0], 2), *lens = c.ints(a[1], 1), *parents = c.ints(a[2], 1), *children = c.ints(a[3], 1);
    const Tensor *refs = c.ints(a[4], 1), *list = c.ints(a[5], 1), *head = c.ints(a[6], 1), *some = c.maybe(a[8], at::kInt, 1);
    int64_t page = 0;
    if (!c.fine || !whole(a[7], page) || page < 1) Py_RETURN_NONE;
    const int64_t N = table->size(0), F = parents->size(0);
    if (lens->size(0) != N || children->size(0) != F || (some && some->size(0) != F) || head->size(0) != 1 || !table->is_contiguous() ||
        !c.sizes({N, table->size(1), refs->size(0), list->size(0), F}))
        Py_RETURN_NONE;
    void* status = c.header(a[9]);
    if (!c.fine) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    // (copies are held until the launch)
    const Tensor l = lens->contiguous(), p = parents->contiguous(), k = children->contiguous(), r = refs->contiguous(), f = list->contiguous();
    const Tensor s = some ? some->contiguous() : Tensor();
    Tensor lens_out = fresh({N}, l, at::kInt), refs_out = fresh({r.size(0)}, l, at::kInt), head_out = fresh({1}, l, at::kInt);
    Tensor pairs = fresh({F, 2}, l, at::kInt);
    const cudaStream_t stream = stream_of(c.device);
    return result(launch([&] { return kda_page_fork(i32_out(*table), (int)table->size(1), i32(l), i32(p), i32(k), some ? i32(s) : nullptr, i32(r), (int)r.size(0),
                                i32(f), (int)f.size(0), i32(*head), (int)page, i32_out(lens_out), i32_out(refs_out), i32_out(head_out),
                                i32_out(pairs), (int)N, (int)F, status, stream); }),
                  {lens_out, refs_out, head_out, pairs});
    END_HANDLE_TH_ERRORS
}

// pools (a tensor, a list or a tuple), pairs, count, workspace.  Returns an empty tuple.
MARSHAL(page_copy, 4)
    Call c;
    const Tensor *pairs = c.ints(a[1], 2), *count = c.maybe(a[2], at::kInt, 1);
    if (!c.fine || pairs->size(1) != 2 || (count && count->size(0) != 1) || !c.sizes({pairs->size(0)})) Py_RETURN_NONE;
    PyObject* const* items = a;
    Py_ssize_t several = 1;
    if (!THPVariable_Check(a[0])) {
        if (!PyList_Check(a[0]) && !PyTuple_Check(a[0])) Py_RETURN_NONE;
        several = PySequence_Fast_GET_SIZE(a[0]);
        items = PySequence_Fast_ITEMS(a[0]);
    }
    if (several < 1 || !fits(several)) Py_RETURN_NONE;
    std::vector<void*> at((size_t)several);
    const Tensor* first = tensor(items[0]);
    for (Py_ssize_t i = 0; i < several; ++i) {
        const Tensor* t = c.memory(items[i]);
        if (t == nullptr || t->dim() < 1 || t->scalar_type() != first->scalar_type() || t->sizes() != first->sizes()) Py_RETURN_NONE;
        at[(size_t)i] = t->data_ptr();
        if (reinterpret_cast<uintptr_t>(at[(size_t)i]) % 16 != 0) Py_RETURN_NONE;
    }
    const int64_t pages = first->size(0);
    if (pages < 1 || !fits(pages)) Py_RETURN_NONE;
    const int64_t bytes = (int64_t)first->nbytes() / pages;
    void* status = c.header(a[3]);
    if (!c.fine || bytes < 16 || bytes % 16 != 0) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    const Tensor p = pairs->contiguous();
    const cudaStream_t stream = stream_of(c.device);
    return result(launch([&] { return kda_page_copy(at.data(), (int)several, (int)pages, bytes, i32(p), count ? i32(*count) : nullptr, (int)p.size(0), status,
                                stream); }),
                  {});
    END_HANDLE_TH_ERRORS
}

// block_table, seq_lens, keep_lens, refs, free_pages, free_head, page_size, workspace
MARSHAL(page_free, 8)
    Call c;
    const Tensor *table = c.ints(a[0], 2), *lens = c.ints(a[1], 1), *keep = c.ints(a[2], 1), *refs = c.ints(a[3], 1);
    const Tensor *list = c.ints(a[4], 1), *head = c.ints(a[5], 1);
    int64_t page = 0;
    if (!c.fine || !whole(a[6], page) || page < 1) Py_RETURN_NONE;
    const int64_t N = table->size(0);
    if (lens->size(0) != N || keep->size(0) != N || head->size(0) != 1 || !list->is_contiguous() ||
        !c.sizes({N, table->size(1), refs->size(0), list->size(0)}))
        Py_RETURN_NONE;
    void* status = c.header(a[7]);
    if (!c.fine) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    const Tensor t = table->contiguous(), l = lens->contiguous(), k = keep->contiguous(), r = refs->contiguous();
    Tensor lens_out = fresh({N}, l, at::kInt), refs_out = fresh({r.size(0)}, l, at::kInt), head_out = fresh({1}, l, at::kInt);
    const cudaStream_t stream = stream_of(c.device);
    return result(launch([&] { return kda_page_free(i32(t), (int)t.size(1), i32(l), i32(k), i32(r), (int)r.size(0), i32_out(*list), (int)list->size(0), i32(*head),
                                (int)page, i32_out(lens_out), i32_out(refs_out), i32_out(head_out), (int)N, status, stream); }),
                  {lens_out, refs_out, head_out});
    END_HANDLE_TH_ERRORS
}

// block_table, seq_lens, refs, free_pages, free_head, page_size, workspace
MARSHAL(page_compact, 7)
    Call c;
    const Tensor *table = c.ints(a[0], 2), *lens = c.ints(a[1], 1), *refs = c.ints(a[2], 1), *list = c.ints(a[3], 1), *head = c.ints(a[4], 1);
    int64_t page = 0;
    if (!c.fine || !whole(a[5], page) || page < 1) Py_RETURN_NONE;
    const int64_t N = table->size(0), pages = refs->size(0);
    if (lens->size(0) != N || head->size(0) != 1 || !c.sizes({N, table->size(1), pages, list->size(0)})) Py_RETURN_NONE;
    void* status = c.header(a[6]);
    if (!c.fine) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    const Tensor t = table->contiguous(), l = lens->contiguous(), r = refs->contiguous(), f = list->contiguous();
    Tensor table_out = fresh({N, t.size(1)}, l, at::kInt), refs_out = fresh({pages}, l, at::kInt), free_out = fresh({f.size(0)}, l, at::kInt);
    Tensor pairs = fresh({pages / 2, 2}, l, at::kInt), count = fresh({1}, l, at::kInt), moved = fresh({pages}, l, at::kInt);
    const cudaStream_t stream = stream_of(c.device);
    return result(launch([&] { return kda_page_compact(i32(t), (int)t.size(1), i32(l), i32(r), (int)pages, i32(f), (int)f.size(0), i32(*head), (int)page,
                                   i32_out(table_out), i32_out(refs_out), i32_out(free_out), i32_out(pairs), i32_out(count), i32_out(moved), (int)N,
                                   status, stream); }),
                  {table_out, refs_out, free_out, pairs, count, moved});
    END_HANDLE_TH_ERRORS
}

// draft_tokens, target_probs, uniform, draft_probs, workspace
MARSHAL(verify_drafts, 5)
    const Tensor* probs = tensor(a[1]);
    if (probs == nullptr) Py_RETURN_NONE;
    const at::ScalarType type = probs->scalar_type();
    if (type != at::kFloat && type != at::kHalf && type != at::kBFloat16) Py_RETURN_NONE;
    Call c;
    const Tensor *drafts = c.take(a[0], at::kLong, 2), *target = c.take(a[1], type, 3), *uniform = c.take(a[2], at::kFloat, 2);
    const Tensor* draft = c.maybe(a[3], type, 3);
    if (!c.fine) Py_RETURN_NONE;
    const int64_t N = drafts->size(0), S = drafts->size(1), V = target->size(2);
    if (target->size(0) != N || target->size(1) != S + 1 || uniform->size(0) != N || uniform->size(1) != S + 1 ||
        (draft && (draft->size(0) != N || draft->size(1) != S || draft->size(2) != V)) || !c.sizes({N, S + 1, V}))
        Py_RETURN_NONE;
    void* status = c.header(a[4]);
    if (!c.fine) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    const Tensor d = drafts->contiguous(), u = uniform->contiguous();
    auto rows = [&](const Tensor& t) { return t.stride(2) == 1 || V <= 1 ? t : t.contiguous(); };
    const Tensor p = rows(*target), q = draft ? rows(*draft) : Tensor();
    const long long p_strides[2] = {p.stride(0), p.stride(1)}, q_strides[2] = {draft ? q.stride(0) : 0, draft ? q.stride(1) : 0};
    Tensor tokens = fresh({N, S + 1}, d, at::kLong), accepted = fresh({N}, d, at::kInt);
    const unsigned flags = type == at::kFloat ? KDA_FLAG_FP32 : type == at::kHalf ? KDA_FLAG_FP16 : 0u;
    const cudaStream_t stream = stream_of(c.device);
    return result(launch([&] { return kda_verify_drafts(static_cast<const int64_t*>(d.data_ptr()), draft ? q.data_ptr() : nullptr, q_strides, p.data_ptr(), p_strides,
                                    static_cast<const float*>(u.data_ptr()), static_cast<int64_t*>(tokens.data_ptr()), i32_out(accepted), (int)N,
                                    (int)S, (int)V, flags, status, stream); }),
                  {tokens, accepted});
    END_HANDLE_TH_ERRORS
}

// q, cache, block_table, seq_lens, w_up, cu_seqlens_q, num_keys, scale (a float), workspace
MARSHAL(latent_chunk, 9)
    const Tensor* first = tensor(a[0]);
    if (first == nullptr || (first->scalar_type() != at::kHalf && first->scalar_type() != at::kBFloat16)) Py_RETURN_NONE;
    const at::ScalarType type = first->scalar_type();
    Call c;
    const Tensor *query = c.take(a[0], type, 3), *cache = c.take(a[1], type, 3), *table = c.ints(a[2], 2), *lens = c.ints(a[3], 1);
    const Tensor *up = c.take(a[4], type, 3), *offsets = c.ints(a[5], 1);
    int64_t keys = 0;
    if (!c.fine || !whole(a[6], keys)) Py_RETURN_NONE;
    const int64_t T = query->size(0), H = query->size(1), N = table->size(0);
    if (query->size(2) != QUERY || cache->size(2) != ROW || !cache->is_contiguous() || up->size(0) != H || up->size(1) != EXPANDED ||
        up->size(2) != LATENT || lens->size(0) != N || offsets->size(0) != N + 1 ||
        !c.sizes({T, H, N, table->size(1), cache->size(0), cache->size(1)}))
        Py_RETURN_NONE;
    const Tensor* given = a[8] == Py_None ? nullptr : c.memory(a[8]);
    if (!c.fine) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    const Tensor q = in_place(*query), w = in_place(*up), t = table->contiguous(), l = lens->contiguous(), o = offsets->contiguous();
    const size_t need = kda_latent_chunk_workspace_bytes((int)T, (int)keys, (int)H, (int)N);
    // a workspace that is too small still gets the status
    const bool enough = given != nullptr && given->nbytes() >= need;
    const Tensor scratch = enough ? *given : fresh({(int64_t)(need > (size_t)STATUS_BYTES ? need : (size_t)STATUS_BYTES)}, l, at::kByte);
    Tensor out = fresh({T, H, VALUE}, q, type), lse = fresh({T, H}, q, at::kFloat);
    const cudaStream_t stream = stream_of(c.device);
    const float scale = (float)PyFloat_AsDouble(a[7]);
    kda_status status = launch([&] { return kda_latent_chunk(
        q.data_ptr(), cache->data_ptr(), (int)cache->size(0), (int)cache->size(1), i32(t), (int)t.size(1), i32(l), w.data_ptr(),
        scale, i32(o), (int)keys, out.data_ptr(), static_cast<float*>(lse.data_ptr()), (int)T, (int)H, (int)N,
        type == at::kHalf ? KDA_FLAG_FP16 : 0u, scratch.data_ptr(), scratch.nbytes(), stream); });
    if (status == KDA_OK && given != nullptr && !enough) {
        const size_t bytes = given->nbytes() < (size_t)STATUS_BYTES ? given->nbytes() : (size_t)STATUS_BYTES;
        if (cudaMemcpyAsync(given->data_ptr(), scratch.data_ptr(), bytes, cudaMemcpyDeviceToDevice, stream) != cudaSuccess) {
            (void)cudaGetLastError();
            status = KDA_ERR_CUDA;
        }
    }
    return result(status, {out, lse});
    END_HANDLE_TH_ERRORS
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(page_fork),     ENTRY(page_copy),    ENTRY(page_free), ENTRY(page_compact),
                         ENTRY(verify_drafts), ENTRY(latent_chunk), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kda_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kda_marshal() { return PyModule_Create(&module); }
