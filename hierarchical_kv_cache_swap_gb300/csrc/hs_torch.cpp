// hs_torch.cpp -- the page calls for torch tensors: checks of types, shapes, strides and
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

// Pages [B, S, page bytes]: a tensor, or (address, B, S, device) of a context's device buffer.
struct Pages {
    const uint8_t* at;
    int64_t B, S;
};
Pages pages_of(PyObject* o, const hs_page_shape& s) {
    if (PyTuple_Check(o)) {
        if (PyTuple_GET_SIZE(o) != 4) refuse("pages must be a tensor");
        const int device = c10::cuda::current_device();
        if (integer(PyTuple_GET_ITEM(o, 3)) != device) refuse("the current device %d is not the context's", device);
        return Pages{(const uint8_t*)(uintptr_t)integer(PyTuple_GET_ITEM(o, 0)), integer(PyTuple_GET_ITEM(o, 1)),
                     integer(PyTuple_GET_ITEM(o, 2))};
    }
    const at::Tensor& x = tensor(o, "pages");
    vector(x, "pages", at::kByte, {-1, -1, (int64_t)hs_page_bytes(&s)});
    on_device({{"pages", &x}});
    return Pages{(const uint8_t*)x.data_ptr(), x.size(0), x.size(1)};
}

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
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_hs_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hs_torch(void) { return PyModule_Create(&kModule); }
