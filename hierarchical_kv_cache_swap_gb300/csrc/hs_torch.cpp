// hs_torch.cpp -- the page and latent calls for torch tensors: checks of types, shapes, strides and
// devices, then the C call of include/hs.h. The calls take a few microseconds on the GPU at
// small sizes, less than their arguments would take to check and marshal in Python.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <exception>
#include <initializer_list>

#include "hs.h"

namespace {

PyObject* g_error = nullptr;  // HsError

struct Refused : std::exception {};  // a Python error is set

[[noreturn]] void refuse(const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(PyExc_ValueError, fmt, ap);
    va_end(ap);
    throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

bool has(PyObject* o) { return o != Py_None; }

// A contiguous tensor of the given type and shape (-1: any extent).
void vector(const at::Tensor& x, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    bool ok = x.scalar_type() == type && x.dim() == (int64_t)shape.size() && x.is_contiguous();
    if (ok) {
        int i = 0;
        for (int64_t n : shape) {
            if (n >= 0 && x.size(i) != n) ok = false;
            ++i;
        }
    }
    if (ok) return;
    std::string want;
    for (int64_t n : shape) want += (want.empty() ? "" : ", ") + (n < 0 ? std::string("*") : std::to_string(n));
    refuse("%s must be a contiguous %s tensor of shape [%s]", name, c10::toString(type), want.c_str());
}

int dtype_code(const at::Tensor& x, const char* name) {
    if (x.scalar_type() == at::kBFloat16) return HS_BF16;
    if (x.scalar_type() == at::kHalf) return HS_F16;
    refuse("%s must be bfloat16 or float16", name);
}

struct Named {
    const char* name;
    const at::Tensor* x;
};

// Every tensor is on the calling thread's current device.
void on_device(std::initializer_list<Named> list) {
    for (const Named& t : list)
        if (t.x && !t.x->is_cuda()) refuse("%s must be on the current CUDA device, it is on the CPU", t.name);
    const int device = c10::cuda::current_device();
    for (const Named& t : list)
        if (t.x && t.x->get_device() != device)
            refuse("%s must be on the current CUDA device %d, it is on device %d", t.name, device, (int)t.x->get_device());
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}

int int_of(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    if (v < INT_MIN || v > INT_MAX) refuse("%s=%lld is out of range", name, (long long)v);
    return (int)v;
}

int int_of(int64_t v, const char* name) {
    if (v < INT_MIN || v > INT_MAX) refuse("%s=%lld is out of range", name, (long long)v);
    return (int)v;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}

// The shape as any triple (tokens, kv_heads, head_dim).
hs_page_shape shape_of(PyObject* o) {
    PyObject* seq = PySequence_Fast(o, "the page shape is (tokens, kv_heads, head_dim)");
    if (!seq) throw Refused();
    hs_page_shape s{0, 0, 0};
    const bool three = PySequence_Fast_GET_SIZE(seq) == 3;
    try {
        if (three) {
            PyObject** e = PySequence_Fast_ITEMS(seq);
            s = hs_page_shape{int_of(e[0], "tokens"), int_of(e[1], "kv_heads"), int_of(e[2], "head_dim")};
        }
    } catch (...) {
        Py_DECREF(seq);
        throw;
    }
    Py_DECREF(seq);
    if (!three) refuse("the page shape is (tokens, kv_heads, head_dim)");
    if (hs_page_bytes(&s) == 0) refuse("unsupported page shape (%d, %d, %d)", s.tokens, s.kv_heads, s.head_dim);
    return s;
}

// None: torch's current stream; an int, or an object with cuda_stream, otherwise.
hs_stream_t stream_of(PyObject* o) {
    if (!has(o)) return (hs_stream_t)c10::cuda::getCurrentCUDAStream().stream();
    if (PyLong_Check(o)) return (hs_stream_t)(uintptr_t)integer(o);
    PyObject* a = PyObject_GetAttrString(o, "cuda_stream");
    if (!a) throw Refused();
    const unsigned long long v = PyLong_AsUnsignedLongLong(a);
    Py_DECREF(a);
    if (PyErr_Occurred()) throw Refused();
    return (hs_stream_t)(uintptr_t)v;
}

// A device status word: a tensor of one int32, an address, or None.
uint32_t* status_of(PyObject* o) {
    if (!has(o)) return nullptr;
    if (PyLong_Check(o)) return (uint32_t*)(uintptr_t)integer(o);
    const at::Tensor& x = tensor(o, "status");
    vector(x, "status", at::kInt, {1});
    on_device({{"status", &x}});
    return (uint32_t*)x.data_ptr();
}

// Makes the C call without the interpreter's lock: a launch may block while the queue is full
// of work that waits for a callback into Python. Nothing of torch is asked in there: a tensor
// without memory throws when asked for its pointer, and an error is set under the lock.
template <class F>
PyObject* done(const char* what, F&& call) {
    PyThreadState* state = PyEval_SaveThread();
    const int rc = [&]() noexcept { return call(); }();
    PyEval_RestoreThread(state);
    if (rc == HS_OK) Py_RETURN_NONE;
    PyErr_Format(g_error ? g_error : PyExc_RuntimeError, "%s failed (%d): %s", what, rc, hs_last_error());
    return nullptr;
}

// Runs `f` with C++ exceptions turned into Python errors.
template <class F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

bool arity(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", want, got);
    return got == want;
}

// The stride of dimension i; a dimension of one has none that matters.
int64_t stride(const at::Tensor& x, int i) { return x.size(i) > 1 ? x.stride(i) : 0; }

// k and v [n, kv_heads, head_dim] with contiguous rows.
hs_token_rows rows_of(const hs_page_shape& s, const at::Tensor& k, const at::Tensor& v) {
    const int64_t n = k.dim() == 3 ? k.size(0) : 0;
    for (const Named& t : {Named{"k", &k}, Named{"v", &v}})
        if (t.x->dim() != 3 || t.x->size(0) != n || t.x->size(1) != s.kv_heads || t.x->size(2) != s.head_dim ||
            (t.x->stride(2) != 1 && t.x->numel() > 0))
            refuse("%s must have shape [%lld, %d, %d] with contiguous rows", t.name, (long long)n, s.kv_heads, s.head_dim);
    if (v.scalar_type() != k.scalar_type()) refuse("k and v must have one dtype");
    return hs_token_rows{k.data_ptr(), v.data_ptr(), stride(k, 0), stride(k, 1), stride(v, 0), stride(v, 1)};
}

// write_tokens(shape, k, v, dest, pages, status, stream)
PyObject* write_tokens(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arity(na, 7)) return nullptr;
    return guarded([&] {
        const hs_page_shape s = shape_of(a[0]);
        const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &dest = tensor(a[3], "dest"), &pages = tensor(a[4], "pages");
        const hs_token_rows rows = rows_of(s, k, v);
        const int type = dtype_code(k, "k");
        vector(dest, "dest", at::kLong, {k.size(0)});
        vector(pages, "pages", at::kByte, {-1, (int64_t)hs_page_bytes(&s)});
        on_device({{"k", &k}, {"v", &v}, {"dest", &dest}, {"pages", pages.is_cpu() && pages.is_pinned() ? nullptr : &pages}});
        uint32_t* const status = status_of(a[5]);
        const hs_stream_t stream = stream_of(a[6]);
        const int64_t n = k.size(0), num_pages = pages.size(0), *const to = (const int64_t*)dest.data_ptr();
        uint8_t* const at = (uint8_t*)pages.data_ptr();
        return done("hs_write_tokens", [&] { return hs_write_tokens(stream, &s, type, &rows, n, to, at, num_pages, status); });
    });
}

// append_tokens(context, shape, k, v, positions, requests, stream)
PyObject* append_tokens(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arity(na, 7)) return nullptr;
    return guarded([&] {
        const hs_page_shape s = shape_of(a[1]);
        const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v"), &pos = tensor(a[4], "positions");
        const at::Tensor* req = has(a[5]) ? &tensor(a[5], "requests") : nullptr;
        const hs_token_rows rows = rows_of(s, k, v);
        const int type = dtype_code(k, "k");
        vector(pos, "positions", at::kInt, {k.size(0)});
        if (req) vector(*req, "requests", at::kInt, {k.size(0)});
        on_device({{"k", &k}, {"v", &v}, {"positions", &pos}, {"requests", req}});
        hs_ctx* const ctx = (hs_ctx*)(uintptr_t)integer(a[0]);
        const hs_stream_t stream = stream_of(a[6]);
        const int64_t n = k.size(0);
        const int32_t *const requests = req ? (const int32_t*)req->data_ptr() : nullptr, *const positions = (const int32_t*)pos.data_ptr();
        return done("hs_append_tokens", [&] { return hs_append_tokens(ctx, stream, &s, type, &rows, n, requests, positions); });
    });
}

// Pages (or entries) [B, S, bytes]: a tensor, or (address, B, S, device) of a context's device buffer.
struct Pages {
    const uint8_t* at;
    int64_t B, S;
};
Pages rows_in_slots(PyObject* o, const char* name, int64_t bytes) {
    if (PyTuple_Check(o)) {
        if (PyTuple_GET_SIZE(o) != 4) refuse("%s must be a tensor", name);
        const int device = c10::cuda::current_device();
        if (integer(PyTuple_GET_ITEM(o, 3)) != device) refuse("the current device %d is not the context's", device);
        return Pages{(const uint8_t*)(uintptr_t)integer(PyTuple_GET_ITEM(o, 0)), integer(PyTuple_GET_ITEM(o, 1)),
                     integer(PyTuple_GET_ITEM(o, 2))};
    }
    const at::Tensor& x = tensor(o, name);
    vector(x, name, at::kByte, {-1, -1, bytes});
    on_device({{name, &x}});
    return Pages{(const uint8_t*)x.data_ptr(), x.size(0), x.size(1)};
}
Pages pages_of(PyObject* o, const hs_page_shape& s) { return rows_in_slots(o, "pages", (int64_t)hs_page_bytes(&s)); }

// read_pages(shape, pages, slots, k, v, status, stream)
PyObject* read_pages(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arity(na, 7)) return nullptr;
    return guarded([&] {
        const hs_page_shape s = shape_of(a[0]);
        const at::Tensor &slots = tensor(a[2], "slots"), &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
        const int type = dtype_code(k, "k");
        vector(slots, "slots", at::kInt, {-1, -1});
        const int64_t B = slots.size(0), n = slots.size(1);
        vector(k, "k", k.scalar_type(), {B, n * s.tokens, s.kv_heads, s.head_dim});
        vector(v, "v", k.scalar_type(), {B, n * s.tokens, s.kv_heads, s.head_dim});
        const Pages p = pages_of(a[1], s);
        if (p.B != B) refuse("pages of %lld requests, slots of %lld", (long long)p.B, (long long)B);
        on_device({{"slots", &slots}, {"k", &k}, {"v", &v}});
        const int requests = int_of(B, "B"), S = int_of(p.S, "S"), count = int_of(n, "n");
        uint32_t* const status = status_of(a[5]);
        const hs_stream_t stream = stream_of(a[6]);
        const int32_t* const from = (const int32_t*)slots.data_ptr();
        void *const ko = k.data_ptr(), *const vo = v.data_ptr();
        return done("hs_read_pages", [&] { return hs_read_pages(stream, &s, type, p.at, requests, S, from, count, ko, vo, status); });
    });
}

// attend_pages(shape, q, pages, slots, selections, lengths, o, lse, sm_scale, softcap, slopes,
//              start, prefix, status, stream)
PyObject* attend_pages(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arity(na, 15)) return nullptr;
    return guarded([&] {
        hs_page_attention p{};
        p.shape = shape_of(a[0]);
        const at::Tensor &q = tensor(a[1], "q"), &slots = tensor(a[3], "slots"), &sel = tensor(a[4], "selections"),
                         &lengths = tensor(a[5], "lengths"), &o = tensor(a[6], "o"), &lse = tensor(a[7], "lse");
        const at::Tensor* slopes = has(a[10]) ? &tensor(a[10], "slopes") : nullptr;
        const at::Tensor* start = has(a[11]) ? &tensor(a[11], "start") : nullptr;
        const at::Tensor* prefix = has(a[12]) ? &tensor(a[12], "prefix") : nullptr;
        p.dtype = dtype_code(q, "q");
        if (q.dim() != 4 || q.size(3) != p.shape.head_dim || o.sizes() != q.sizes() || o.scalar_type() != q.scalar_type() ||
            (q.numel() > 0 && (q.stride(3) != 1 || o.stride(3) != 1)))
            refuse("q and o must be [B, q_tokens, q_heads, %d] of one dtype with contiguous rows", p.shape.head_dim);
        const int64_t B = q.size(0), T = q.size(1), Hq = q.size(2);
        vector(slots, "slots", at::kInt, {B, -1});
        const int64_t k = slots.size(1);
        vector(sel, "selections", at::kInt, {B, k});
        vector(lengths, "lengths", at::kInt, {B});
        vector(lse, "lse", at::kFloat, {B, T, Hq});
        if (slopes) vector(*slopes, "slopes", at::kFloat, {Hq});
        if (start) vector(*start, "start", at::kInt, {B});
        if (prefix) vector(*prefix, "prefix", at::kInt, {B});
        const Pages pages = pages_of(a[2], p.shape);
        if (pages.B != B) refuse("pages of %lld requests, q of %lld", (long long)pages.B, (long long)B);
        on_device({{"q", &q}, {"slots", &slots}, {"selections", &sel}, {"lengths", &lengths}, {"o", &o}, {"lse", &lse},
                   {"slopes", slopes}, {"start", start}, {"prefix", prefix}});
        p.B = int_of(B, "B");
        p.S = int_of(pages.S, "S");
        p.k = int_of(k, "k");
        p.q_heads = int_of(Hq, "q_heads");
        p.q_tokens = int_of(T, "q_tokens");
        p.q = q.data_ptr();
        p.q_batch_stride = stride(q, 0);
        p.q_token_stride = stride(q, 1);
        p.q_head_stride = stride(q, 2);
        p.o = o.data_ptr();
        p.o_batch_stride = stride(o, 0);
        p.o_token_stride = stride(o, 1);
        p.o_head_stride = stride(o, 2);
        p.lse = (float*)lse.data_ptr();
        p.pages = pages.at;
        p.slots = (const int32_t*)slots.data_ptr();
        p.selections = (const int32_t*)sel.data_ptr();
        p.lengths = (const int32_t*)lengths.data_ptr();
        p.sm_scale = (float)number(a[8]);
        p.softcap = (float)number(a[9]);
        p.slopes = slopes ? (const float*)slopes->data_ptr() : nullptr;
        p.start = start ? (const int32_t*)start->data_ptr() : nullptr;
        p.prefix = prefix ? (const int32_t*)prefix->data_ptr() : nullptr;
        p.status = status_of(a[13]);
        const hs_stream_t stream = stream_of(a[14]);
        return done("hs_attend_pages", [&] { return hs_attend_pages(stream, &p); });
    });
}

// A rotation as (table, positions, halves), table None for none; `own`: the call has positions of its
// own, which stand in where these are None. nullptr where nothing is rotated.
const hs_rotation* rotation_of(PyObject* table, PyObject* positions, PyObject* halves, int64_t n, bool own, hs_rotation* r) {
    if (!has(table)) {
        if (!own && has(positions)) refuse("positions without a rotation");
        return nullptr;
    }
    const at::Tensor& t = tensor(table, "rotation");
    vector(t, "rotation", at::kFloat, {-1, 64});
    on_device({{"rotation", &t}});
    const int32_t* p = nullptr;
    if (has(positions)) {
        const at::Tensor& x = tensor(positions, "positions");
        vector(x, "positions", at::kInt, {n});
        on_device({{"positions", &x}});
        p = (const int32_t*)x.data_ptr();
    } else if (!own) {
        refuse("a rotation wants positions");
    }
    const int h = PyObject_IsTrue(halves);
    if (h < 0) throw Refused();
    *r = hs_rotation{(const float*)t.data_ptr(), t.size(0), p, h};
    return r;
}

// latent [n, 512] and rope [n, 64] with contiguous rows.
hs_latent_rows latents_of(const at::Tensor& latent, const at::Tensor& rope) {
    const int64_t n = latent.dim() == 2 ? latent.size(0) : 0;
    const struct {
        const char* name;
        const at::Tensor* x;
        int width;
    } both[] = {{"latent", &latent, 512}, {"rope", &rope, 64}};
    for (const auto& t : both)
        if (t.x->dim() != 2 || t.x->size(0) != n || t.x->size(1) != t.width || (t.x->stride(1) != 1 && n > 0))
            refuse("%s must have shape [%lld, %d] with contiguous rows", t.name, (long long)n, t.width);
    if (rope.scalar_type() != latent.scalar_type()) refuse("latent and rope must have one dtype");
    return hs_latent_rows{latent.data_ptr(), rope.data_ptr(), stride(latent, 0), stride(rope, 0)};
}

// write_latents(latent, rope, dest, entries, rotation, positions, halves, status, stream)
PyObject* write_latents(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arity(na, 9)) return nullptr;
    return guarded([&] {
        const at::Tensor &latent = tensor(a[0], "latent"), &rope = tensor(a[1], "rope"), &dest = tensor(a[2], "dest"),
                         &entries = tensor(a[3], "entries");
        const int type = dtype_code(latent, "latent");
        const hs_latent_rows rows = latents_of(latent, rope);
        const int64_t n = latent.size(0);
        vector(dest, "dest", at::kLong, {n});
        vector(entries, "entries", at::kByte, {-1, HS_LATENT_ENTRY_BYTES});
        on_device({{"latent", &latent}, {"rope", &rope}, {"dest", &dest},
                   {"entries", entries.is_cpu() && entries.is_pinned() ? nullptr : &entries}});
        hs_rotation r;
        const hs_rotation* const rot = rotation_of(a[4], a[5], a[6], n, false, &r);
        uint32_t* const status = status_of(a[7]);
        const hs_stream_t stream = stream_of(a[8]);
        const int64_t num = entries.size(0), *const to = (const int64_t*)dest.data_ptr();
        uint8_t* const at = (uint8_t*)entries.data_ptr();
        return done("hs_write_latents", [&] { return hs_write_latents(stream, type, &rows, n, rot, to, at, num, status); });
    });
}

// append_latents(context, latent, rope, positions, requests, rotation, rotation positions, halves, stream)
PyObject* append_latents(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arity(na, 9)) return nullptr;
    return guarded([&] {
        const at::Tensor &latent = tensor(a[1], "latent"), &rope = tensor(a[2], "rope"), &pos = tensor(a[3], "positions");
        const at::Tensor* req = has(a[4]) ? &tensor(a[4], "requests") : nullptr;
        const int type = dtype_code(latent, "latent");
        const hs_latent_rows rows = latents_of(latent, rope);
        const int64_t n = latent.size(0);
        vector(pos, "positions", at::kInt, {n});
        if (req) vector(*req, "requests", at::kInt, {n});
        on_device({{"latent", &latent}, {"rope", &rope}, {"positions", &pos}, {"requests", req}});
        hs_rotation r;
        const hs_rotation* const rot = rotation_of(a[5], a[6], a[7], n, true, &r);
        hs_ctx* const ctx = (hs_ctx*)(uintptr_t)integer(a[0]);
        const hs_stream_t stream = stream_of(a[8]);
        const int32_t *const requests = req ? (const int32_t*)req->data_ptr() : nullptr, *const positions = (const int32_t*)pos.data_ptr();
        return done("hs_append_latents", [&] { return hs_append_latents(ctx, stream, type, &rows, n, rot, requests, positions); });
    });
}

// read_latents(entries, slots, latent, rope, status, stream)
PyObject* read_latents(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arity(na, 6)) return nullptr;
    return guarded([&] {
        const at::Tensor &slots = tensor(a[1], "slots"), &latent = tensor(a[2], "latent"), &rope = tensor(a[3], "rope");
        const int type = dtype_code(latent, "latent");
        vector(slots, "slots", at::kInt, {-1, -1});
        const int64_t B = slots.size(0), n = slots.size(1);
        vector(latent, "latent", latent.scalar_type(), {B, n, 512});
        vector(rope, "rope", latent.scalar_type(), {B, n, 64});
        const Pages p = rows_in_slots(a[0], "entries", HS_LATENT_ENTRY_BYTES);
        if (p.B != B) refuse("entries of %lld requests, slots of %lld", (long long)p.B, (long long)B);
        on_device({{"slots", &slots}, {"latent", &latent}, {"rope", &rope}});
        const int requests = int_of(B, "B"), S = int_of(p.S, "S"), count = int_of(n, "n");
        uint32_t* const status = status_of(a[4]);
        const hs_stream_t stream = stream_of(a[5]);
        const int32_t* const from = (const int32_t*)slots.data_ptr();
        void *const lo = latent.data_ptr(), *const ro = rope.data_ptr();
        return done("hs_read_latents", [&] { return hs_read_latents(stream, type, p.at, requests, S, from, count, lo, ro, status); });
    });
}

// x [n, heads, x_width], w [heads, 128, 512] with contiguous rows, out [n, heads, out_width] contiguous.
hs_head_product product_of(const at::Tensor& x, const char* name, at::ScalarType type, int x_width, const at::Tensor& w, const at::Tensor& out,
                           int out_width) {
    if (x.dim() != 3 || x.size(2) != x_width || x.scalar_type() != type || (x.stride(2) != 1 && x.numel() > 0))
        refuse("%s must be a %s tensor of shape [*, *, %d] with contiguous rows", name, c10::toString(type), x_width);
    const int64_t n = x.size(0), H = x.size(1);
    if (w.dim() != 3 || w.size(0) != H || w.size(1) != 128 || w.size(2) != 512 || w.scalar_type() != at::kBFloat16 ||
        (w.stride(2) != 1 && w.numel() > 0))
        refuse("the matrices must be a bfloat16 tensor of shape [%lld, 128, 512] with contiguous rows", (long long)H);
    vector(out, "out", at::kBFloat16, {n, H, out_width});
    on_device({{name, &x}, {"the matrices", &w}, {"out", &out}});
    return hs_head_product{x.data_ptr(), stride(x, 0), stride(x, 1), w.data_ptr(), stride(w, 0), stride(w, 1), out.data_ptr(), n,
                           int_of(H, "heads"), nullptr};
}

// absorb_queries(q, up_k, out, rotation, positions, halves, status, stream)
PyObject* absorb_queries(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arity(na, 8)) return nullptr;
    return guarded([&] {
        const at::Tensor& q = tensor(a[0], "q");
        const hs_head_product p = product_of(q, "q", at::kBFloat16, 192, tensor(a[1], "up_k"), tensor(a[2], "out"), 576);
        hs_rotation r;
        const hs_rotation* const rot = rotation_of(a[3], a[4], a[5], p.n, false, &r);
        uint32_t* const status = status_of(a[6]);
        const hs_stream_t stream = stream_of(a[7]);
        return done("hs_absorb_queries", [&] { return hs_absorb_queries(stream, &p, rot, status); });
    });
}

// expand_outputs(o, up_v, out, status, stream)
PyObject* expand_outputs(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arity(na, 5)) return nullptr;
    return guarded([&] {
        hs_head_product p = product_of(tensor(a[0], "o"), "o", at::kFloat, 512, tensor(a[1], "up_v"), tensor(a[2], "out"), 128);
        p.status = status_of(a[3]);
        const hs_stream_t stream = stream_of(a[4]);
        return done("hs_expand_outputs", [&] { return hs_expand_outputs(stream, &p); });
    });
}

// attend_prompts(q, k, k_rope, v, q_starts, k_starts, o, lse, sm_scale, causal, status, stream)
PyObject* attend_prompts(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arity(na, 12)) return nullptr;
    return guarded([&] {
        hs_prompt_attention p{};
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &r = tensor(a[2], "k_rope"), &v = tensor(a[3], "v"),
                         &qs = tensor(a[4], "q_starts"), &ks = tensor(a[5], "k_starts"), &o = tensor(a[6], "o"), &lse = tensor(a[7], "lse");
        p.dtype = dtype_code(q, "q");
        const int64_t H = q.dim() == 3 ? q.size(1) : 0, n = k.dim() == 3 ? k.size(0) : 0, m = q.dim() == 3 ? q.size(0) : 0;
        const struct {
            const char* name;
            const at::Tensor* x;
            int64_t rows, width;
        } rows[] = {{"q", &q, m, 192}, {"o", &o, m, 128}, {"k", &k, n, 128}, {"v", &v, n, 128}};
        for (const auto& t : rows)
            if (t.x->dim() != 3 || t.x->size(0) != t.rows || t.x->size(1) != H || t.x->size(2) != t.width || t.x->scalar_type() != q.scalar_type() ||
                (t.x->stride(2) != 1 && t.x->numel() > 0))
                refuse("%s must have shape [%lld, %lld, %lld] with contiguous rows, and q's dtype", t.name, (long long)t.rows, (long long)H,
                       (long long)t.width);
        if (r.dim() != 2 || r.size(0) != n || r.size(1) != 64 || r.scalar_type() != q.scalar_type() || (r.stride(1) != 1 && n > 0))
            refuse("k_rope must have shape [%lld, 64] with contiguous rows, and q's dtype", (long long)n);
        vector(qs, "q_starts", at::kInt, {-1});
        vector(ks, "k_starts", at::kInt, {qs.size(0)});
        if (qs.size(0) < 1) refuse("q_starts and k_starts must have an element more than there are prompts");
        vector(lse, "lse", at::kFloat, {m, H});
        on_device({{"q", &q}, {"k", &k}, {"k_rope", &r}, {"v", &v}, {"q_starts", &qs}, {"k_starts", &ks}, {"o", &o}, {"lse", &lse}});
        p.B = int_of(qs.size(0) - 1, "B");
        p.heads = int_of(H, "heads");
        p.causal = PyObject_IsTrue(a[9]);
        if (p.causal < 0) throw Refused();
        p.q_rows = m;
        p.k_rows = n;
        p.q = q.data_ptr();
        p.q_token_stride = stride(q, 0);
        p.q_head_stride = stride(q, 1);
        p.k = k.data_ptr();
        p.k_token_stride = stride(k, 0);
        p.k_head_stride = stride(k, 1);
        p.k_rope = r.data_ptr();
        p.k_rope_stride = stride(r, 0);
        p.v = v.data_ptr();
        p.v_token_stride = stride(v, 0);
        p.v_head_stride = stride(v, 1);
        p.o = o.data_ptr();
        p.o_token_stride = stride(o, 0);
        p.o_head_stride = stride(o, 1);
        p.lse = (float*)lse.data_ptr();
        p.q_starts = (const int32_t*)qs.data_ptr();
        p.k_starts = (const int32_t*)ks.data_ptr();
        p.sm_scale = (float)number(a[8]);
        p.status = status_of(a[10]);
        const hs_stream_t stream = stream_of(a[11]);
        return done("hs_attend_prompts", [&] { return hs_attend_prompts(stream, &p); });
    });
}

PyObject* set_error(PyObject*, PyObject* e) {
    Py_XDECREF(g_error);
    Py_INCREF(e);
    g_error = e;
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"write_tokens", (PyCFunction)(void (*)(void))write_tokens, METH_FASTCALL, nullptr},
    {"append_tokens", (PyCFunction)(void (*)(void))append_tokens, METH_FASTCALL, nullptr},
    {"read_pages", (PyCFunction)(void (*)(void))read_pages, METH_FASTCALL, nullptr},
    {"attend_pages", (PyCFunction)(void (*)(void))attend_pages, METH_FASTCALL, nullptr},
    {"write_latents", (PyCFunction)(void (*)(void))write_latents, METH_FASTCALL, nullptr},
    {"append_latents", (PyCFunction)(void (*)(void))append_latents, METH_FASTCALL, nullptr},
    {"read_latents", (PyCFunction)(void (*)(void))read_latents, METH_FASTCALL, nullptr},
    {"absorb_queries", (PyCFunction)(void (*)(void))absorb_queries, METH_FASTCALL, nullptr},
    {"expand_outputs", (PyCFunction)(void (*)(void))expand_outputs, METH_FASTCALL, nullptr},
    {"attend_prompts", (PyCFunction)(void (*)(void))attend_prompts, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_hs_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hs_torch(void) { return PyModule_Create(&kModule); }
