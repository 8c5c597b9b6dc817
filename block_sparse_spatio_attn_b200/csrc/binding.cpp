// binding.cpp -- the streaming attention calls for Python: argument marshalling only.
//
// A decoding step runs a handful of calls of a few microseconds each, so here the marshalling
// itself has to be cheap: checking a dozen tensors and filling the C structs from Python
// (ctypes) took 10-20 us a call, this module takes about 1.  Every check the C ABI cannot make
// from a pointer is made here: type, shape, contiguous rows, one CUDA device for all; strides
// and alignment are the library's to check.  The tensors' device is made current for the
// call and the current one put back.  Errors become SvgaError(status, message).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <cuda_runtime_api.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <exception>
#include <string>

#include "../../include/svga.h"

namespace {

PyObject *g_error_class = nullptr;  // svga.SvgaError

struct Refusal {
    svga_status status;
    std::string message;
};
struct PythonError {};  // a Python exception is already set

[[noreturn]] void refuse(svga_status status, const std::string &message)
{
    throw Refusal{status, message};
}

void check(svga_status rc)
{
    if (rc != SVGA_OK) refuse(rc, svga_last_error());
}

const char *type_name(at::ScalarType t)
{
    switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
    }
}

std::string tuple_of(at::IntArrayRef x)
{
    std::string s = "(";
    for (size_t i = 0; i < x.size(); ++i) s += (i ? ", " : "") + std::to_string(x[i]);
    return s + (x.size() == 1 ? ",)" : ")");
}

int dim32(int64_t x, const char *name)
{
    if (x > INT32_MAX)
        refuse(SVGA_ERR_SHAPE, std::string(name) + " has a dimension of " + std::to_string(x));
    return (int)x;
}

// The tensor arguments of one call.
class Tensors {
public:
    const at::Tensor &take(PyObject *o, const char *name)
    {
        if (!THPVariable_Check(o))
            refuse(SVGA_ERR_INVALID_ARG, std::string(name) + " must be a torch.Tensor, got " +
                                             Py_TYPE(o)->tp_name);
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.layout() != at::kStrided)
            refuse(SVGA_ERR_INVALID_ARG, std::string(name) + " must be a strided tensor");
        return t;
    }

    // the tensor whose type and shape the others follow
    const at::Tensor &lead(PyObject *o, const char *name, int dims, bool f32, svga_dtype *dt)
    {
        if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != dims)
            refuse(SVGA_ERR_SHAPE, std::string(name) + " must be a tensor of " +
                                       std::to_string(dims) + " dimensions");
        const at::Tensor &t = take(o, name);
        if (t.scalar_type() == at::kBFloat16)
            *dt = SVGA_BF16;
        else if (t.scalar_type() == at::kHalf)
            *dt = SVGA_F16;
        else if (f32 && t.scalar_type() == at::kFloat)
            *dt = SVGA_F32;
        else
            refuse(SVGA_ERR_INVALID_ARG, std::string(name) + " must be bf16 or fp16" +
                                             (f32 ? " or fp32" : "") + ", got " +
                                             type_name(t.scalar_type()));
        return t;
    }

    void match(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape)
    {
        if (t.scalar_type() != type)
            refuse(SVGA_ERR_INVALID_ARG, std::string(name) + " must be " + type_name(type) +
                                             ", got " + type_name(t.scalar_type()));
        if (t.sizes() != shape)
            refuse(SVGA_ERR_SHAPE, std::string(name) + " has shape " + tuple_of(t.sizes()) +
                                       ", expected " + tuple_of(shape));
        if (count_ < (int)seen_.size()) seen_[count_++] = {name, t.device()};
    }

    // [batch, heads, tokens, head_dim], or [batch, heads, head_dim] without tokens
    svga_view view(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape)
    {
        const at::Tensor &t = take(o, name);
        match(t, name, type, shape);
        const at::IntArrayRef s = t.strides();
        if (s.back() != 1 && t.numel() > 0)
            refuse(SVGA_ERR_INVALID_ARG,
                   std::string(name) + ": the values of a row must be contiguous");
        return {t.data_ptr(), s[0], s[1], s.size() == 4 ? s[2] : 0};
    }

    void *flat(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape)
    {
        const at::Tensor &t = take(o, name);
        match(t, name, type, shape);
        if (!t.is_contiguous())
            refuse(SVGA_ERR_INVALID_ARG, std::string(name) + " must be contiguous");
        return t.data_ptr();
    }

    void *optional(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape)
    {
        return o == Py_None ? nullptr : flat(o, name, type, shape);
    }

    // All on one CUDA device, which becomes the current one.
    void done()
    {
        for (int i = 0; i < count_; ++i) {
            if (!seen_[i].device.is_cuda())
                refuse(SVGA_ERR_INVALID_ARG,
                       std::string(seen_[i].name) + " must be on a CUDA device");
            if (seen_[i].device != seen_[0].device)
                refuse(SVGA_ERR_INVALID_ARG, std::string(seen_[i].name) + " is on " +
                                                 seen_[i].device.str() + ", " + seen_[0].name +
                                                 " on " + seen_[0].device.str());
        }
        guard_.set_device(seen_[0].device);
    }

    c10::Device device() const { return seen_[0].device; }

    // stream: None (the current stream of the device) or a torch.cuda.Stream
    cudaStream_t stream(PyObject *o)
    {
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device().index()).stream();
        given_ = true;
        PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
        PyObject *d = h ? PyObject_GetAttrString(o, "device_index") : nullptr;
        if (!d) {
            Py_XDECREF(h);
            PyErr_Clear();
            refuse(SVGA_ERR_INVALID_ARG, "stream must be a torch.cuda.Stream or None");
        }
        void *st = PyLong_AsVoidPtr(h);
        const long index = PyLong_AsLong(d);
        Py_DECREF(h);
        Py_DECREF(d);
        if (PyErr_Occurred()) throw PythonError{};
        if (index != device().index())
            refuse(SVGA_ERR_INVALID_ARG, "the stream is on cuda:" + std::to_string(index) +
                                             ", the tensors on " + device().str());
        return static_cast<cudaStream_t>(st);
    }

    // The caller's scratch, or some from torch's allocator that belongs to the call's stream
    // (and so is not handed out again before the call's kernels are done with it).
    void *workspace(PyObject *o, size_t need, cudaStream_t st, size_t *bytes)
    {
        if (o != Py_None) {
            const at::Tensor &t = take(o, "workspace");
            match(t, "workspace", at::kByte, t.sizes());
            if (!t.is_contiguous())
                refuse(SVGA_ERR_INVALID_ARG, "workspace must be contiguous");
            done();
            *bytes = (size_t)t.numel();
            return t.data_ptr();
        }
        *bytes = need;
        if (need == 0) return nullptr;
        c10::cuda::OptionalCUDAStreamGuard on;
        if (given_) on.reset_stream(c10::cuda::getStreamFromExternal(st, device().index()));
        scratch_ = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(device()));
        return scratch_.data_ptr();
    }

private:
    struct Seen {
        const char *name;
        c10::Device device{c10::DeviceType::CPU};
    };
    std::array<Seen, 16> seen_;
    int count_ = 0;
    bool given_ = false;
    at::Tensor scratch_;
    c10::cuda::OptionalCUDAGuard guard_;
};

int64_t integer(PyObject *o)
{
    PyObject *n = PyNumber_Index(o);
    if (!n) throw PythonError{};
    const long long x = PyLong_AsLongLong(n);
    Py_DECREF(n);
    if (x == -1 && PyErr_Occurred()) throw PythonError{};
    return x;
}

int integer32(PyObject *o, const char *name)
{
    const int64_t x = integer(o);
    if (x < INT32_MIN || x > INT32_MAX)
        refuse(SVGA_ERR_INVALID_ARG, std::string(name) + ": " + std::to_string(x) +
                                         " does not fit 32 bits");
    return (int)x;
}

double real(PyObject *o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw PythonError{};
    return x;
}

template <typename T>
const T *address(PyObject *o)
{
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw PythonError{};
    return static_cast<const T *>(p);
}

// spec_at, rows of its table, table
const float *table_of(Tensors &t, PyObject *table, int64_t rows)
{
    return static_cast<const float *>(t.flat(table, "table", at::kFloat, {rows, 2}));
}

void rotary_table(PyObject *const *a)  // spec_at, rows, theta, table, stream
{
    Tensors t;
    float *table = const_cast<float *>(table_of(t, a[3], integer(a[1])));
    t.done();
    check(svga_rotary_table(address<svga_rotary_spec>(a[0]), real(a[2]), table, t.stream(a[4])));
}

// src, dst, spec_at, rows, heads of its order or -1, table, positions, first, inverse, status,
// stream
void rotary(PyObject *const *a)
{
    Tensors t;
    svga_dtype dt;
    const at::Tensor &src = t.lead(a[0], "src", 4, true, &dt);
    const at::IntArrayRef n = src.sizes();
    const svga_view vs = t.view(a[0], "src", src.scalar_type(), n);
    const svga_view vd = t.view(a[1], "dst", src.scalar_type(), n);
    const float *table = table_of(t, a[5], integer(a[3]));
    const void *pos = t.optional(a[6], "positions", at::kInt, {n[0], n[2]});
    void *status = t.optional(a[9], "status", at::kInt, {1});
    const int inverse = integer32(a[8], "inverse");
    const int64_t named = integer(a[4]);
    if (named >= 0 && named != n[1])
        refuse(SVGA_ERR_SHAPE, "order names " + std::to_string(named) + " heads, src has " +
                                   std::to_string(n[1]));
    t.done();
    check(svga_rotary(&vs, &vd, dim32(n[0], "src"), dim32(n[1], "src"), dim32(n[2], "src"),
                      dim32(n[3], "src"), dt, address<svga_rotary_spec>(a[2]), table,
                      static_cast<const int32_t *>(pos), integer(a[7]), inverse,
                      static_cast<int32_t *>(status), t.stream(a[10])));
}

svga_window_problem window_problem(Tensors &t, const at::Tensor &q, const at::Tensor &k,
                                   svga_dtype dt, PyObject *mask, PyObject *q_lens,
                                   PyObject *k_lens, PyObject *status)
{
    svga_window_problem p;
    p.batch = dim32(q.size(0), "q");
    p.q_heads = dim32(q.size(1), "q");
    p.q_tokens = dim32(q.size(2), "q");
    p.head_dim = dim32(q.size(3), "q");
    p.kv_heads = dim32(k.size(1), "k");
    p.k_tokens = dim32(k.size(2), "k");
    p.dtype = dt;
    p.mask = *address<svga_window_mask>(mask);
    p.q_lens = static_cast<int32_t *>(t.optional(q_lens, "q_lens", at::kInt, {q.size(0)}));
    p.k_lens = static_cast<int32_t *>(t.optional(k_lens, "k_lens", at::kInt, {q.size(0)}));
    p.status = static_cast<int32_t *>(t.optional(status, "status", at::kInt, {1}));
    return p;
}

// q, k, v, o, lse, mask_at, scale, q_lens, k_lens, status, workspace, stream
void window_fwd(PyObject *const *a)
{
    Tensors t;
    svga_dtype dt, kt;
    const at::Tensor &q = t.lead(a[0], "q", 4, false, &dt), &k = t.lead(a[1], "k", 4, false, &kt);
    const at::ScalarType type = q.scalar_type();
    const int64_t ks[4] = {q.size(0), k.size(1), k.size(2), q.size(3)};
    const svga_window_problem p = window_problem(t, q, k, dt, a[5], a[7], a[8], a[9]);
    const svga_view vq = t.view(a[0], "q", type, q.sizes()), vk = t.view(a[1], "k", type, ks),
                    vv = t.view(a[2], "v", type, ks), vo = t.view(a[3], "o", type, q.sizes());
    float *lse = static_cast<float *>(
        t.optional(a[4], "lse", at::kFloat, {q.size(0), q.size(1), q.size(2)}));
    t.done();
    const cudaStream_t st = t.stream(a[11]);
    size_t need = 0, have;
    check(svga_window_attention_size(&p, &need, nullptr));
    void *ws = t.workspace(a[10], need, st, &have);
    check(svga_window_attention_fwd(&vq, &vk, &vv, &vo, lse, &p, (float)real(a[6]), ws, have, st));
}

// d_o, q, k, v, o, lse, dq, dk, dv, mask_at, scale, q_lens, k_lens, status, workspace, stream
void window_bwd(PyObject *const *a)
{
    Tensors t;
    svga_dtype dt, kt;
    const at::Tensor &q = t.lead(a[1], "q", 4, false, &dt), &k = t.lead(a[2], "k", 4, false, &kt);
    const at::ScalarType type = q.scalar_type();
    const at::IntArrayRef qs = q.sizes();
    const int64_t ks[4] = {q.size(0), k.size(1), k.size(2), q.size(3)};
    const svga_window_problem p = window_problem(t, q, k, dt, a[9], a[11], a[12], a[13]);
    const svga_view vdo = t.view(a[0], "d_o", type, qs), vq = t.view(a[1], "q", type, qs),
                    vk = t.view(a[2], "k", type, ks), vv = t.view(a[3], "v", type, ks),
                    vo = t.view(a[4], "o", type, qs), dq = t.view(a[6], "dq", type, qs),
                    dk = t.view(a[7], "dk", type, ks), dv = t.view(a[8], "dv", type, ks);
    const float *lse =
        static_cast<float *>(t.flat(a[5], "lse", at::kFloat, {qs[0], qs[1], qs[2]}));
    t.done();
    const cudaStream_t st = t.stream(a[15]);
    size_t need = 0, have;
    check(svga_window_attention_size(&p, nullptr, &need));
    void *ws = t.workspace(a[14], need, st, &have);
    check(svga_window_attention_bwd(&vdo, &vq, &vk, &vv, &vo, lse, &dq, &dk, &dv, &p,
                                    (float)real(a[10]), ws, have, st));
}

// a: k_pages, v_pages, page_table, lens
svga_paged_cache paged_cache(Tensors &t, PyObject *const *a, int64_t batch, PyObject *status)
{
    svga_paged_cache c;
    const at::Tensor &k = t.lead(a[0], "k_pages", 4, false, &c.dtype);
    const at::IntArrayRef n = k.sizes();
    c.k_pages = t.flat(a[0], "k_pages", k.scalar_type(), n);
    c.v_pages = t.flat(a[1], "v_pages", k.scalar_type(), n);
    c.pages = dim32(n[0], "k_pages");
    c.kv_heads = dim32(n[1], "k_pages");
    c.page_size = dim32(n[2], "k_pages");
    c.head_dim = dim32(n[3], "k_pages");
    c.batch = dim32(batch, "k or q");
    if (!THPVariable_Check(a[2]) || THPVariable_Unpack(a[2]).dim() != 2)
        refuse(SVGA_ERR_SHAPE, "page_table must be an int32 tensor [batch, pages a sequence]");
    const int64_t most = THPVariable_Unpack(a[2]).size(1);
    c.max_pages = dim32(most, "page_table");
    c.page_table = static_cast<int32_t *>(t.flat(a[2], "page_table", at::kInt, {batch, most}));
    c.lens = static_cast<int32_t *>(t.flat(a[3], "lens", at::kInt, {batch}));
    c.status = static_cast<int32_t *>(t.optional(status, "status", at::kInt, {1}));
    return c;
}

// k, v, k_pages, v_pages, page_table, lens, new_lens, spec_at or 0, rows, table, status, stream
void cache_append(PyObject *const *a)
{
    Tensors t;
    svga_dtype dt;
    const at::Tensor &k = t.lead(a[0], "k", 4, false, &dt);
    const svga_paged_cache c = paged_cache(t, a + 2, k.size(0), a[10]);
    const at::ScalarType type = c.dtype == SVGA_F16 ? at::kHalf : at::kBFloat16;
    const int64_t shape[4] = {k.size(0), c.kv_heads, k.size(2), c.head_dim};
    const svga_view vk = t.view(a[0], "k", type, shape), vv = t.view(a[1], "v", type, shape);
    const int32_t *n =
        static_cast<int32_t *>(t.optional(a[6], "new_lens", at::kInt, {k.size(0)}));
    const svga_rotary_spec *spec = address<svga_rotary_spec>(a[7]);
    const float *table = nullptr;
    if (spec)
        table = table_of(t, a[9], integer(a[8]));
    else if (a[9] != Py_None)
        refuse(SVGA_ERR_INVALID_ARG, "a table without a RotarySpec");
    t.done();
    check(svga_cache_append(&vk, &vv, dim32(k.size(2), "k"), n, &c, spec, table, t.stream(a[11])));
}

// q, k_pages, v_pages, page_table, lens, o, lse, mask_at, scale, status, stream
void cache_decode(PyObject *const *a)
{
    Tensors t;
    svga_dtype dt;
    const at::Tensor &q = t.lead(a[0], "q", 3, false, &dt);
    const svga_paged_cache c = paged_cache(t, a + 1, q.size(0), a[9]);
    const at::ScalarType type = c.dtype == SVGA_F16 ? at::kHalf : at::kBFloat16;
    const int64_t shape[3] = {q.size(0), q.size(1), c.head_dim};
    const svga_view vq = t.view(a[0], "q", type, shape), vo = t.view(a[5], "o", type, shape);
    float *lse =
        static_cast<float *>(t.optional(a[6], "lse", at::kFloat, {q.size(0), q.size(1)}));
    t.done();
    check(svga_cache_decode(&vq, &vo, lse, dim32(q.size(1), "q"), &c,
                            address<svga_window_mask>(a[7]), (float)real(a[8]), t.stream(a[10])));
}

// One Python entry: the argument count, then the call, every C++ exception turned into a
// Python one.
template <void (*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        F(args);
        Py_RETURN_NONE;
    } catch (const Refusal &r) {
        PyObject *x = g_error_class ? PyObject_CallFunction(g_error_class, "is", (int)r.status,
                                                            r.message.c_str())
                                    : nullptr;
        if (x) {
            PyErr_SetObject(g_error_class, x);
            Py_DECREF(x);
        } else if (!PyErr_Occurred()) {
            PyErr_SetString(PyExc_RuntimeError, r.message.c_str());
        }
    } catch (const PythonError &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject *set_error_class(PyObject *, PyObject *cls)
{
    Py_INCREF(cls);
    Py_XSETREF(g_error_class, cls);
    Py_RETURN_NONE;
}

#define SVGA_ENTRY(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, n>)), \
     METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {
    SVGA_ENTRY(rotary_table, 5),  SVGA_ENTRY(rotary, 11),       SVGA_ENTRY(window_fwd, 12),
    SVGA_ENTRY(window_bwd, 16),   SVGA_ENTRY(cache_append, 12), SVGA_ENTRY(cache_decode, 11),
    {"set_error_class", &set_error_class, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding",
                        "Marshalling of the streaming attention calls.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding()
{
    PyObject *m = PyModule_Create(&g_module);
    // the torch and Python it was compiled against: the importer refuses any other
    if (m && PyModule_AddStringConstant(m, "built_for", SVGA_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
