// had_cache_bind.cpp -- argument marshalling of the decoder cache's binding.
//
// A step of a decoder makes several of these calls, most of them a few
// microseconds of GPU work, so what a call costs on the host is part of the
// operator: checking a dozen tensors from Python and passing twenty numbers
// through ctypes takes 10 us, the same here 1 us.  No arithmetic of the
// method: tensors are checked, missing outputs allocated (on the current
// stream of the tensors' device), pointers passed on, and a status that is not
// HAD_OK is returned to the Python side, which raises HadError.
#include <Python.h>
#include <climits>
#include <string>

#include <ATen/Functions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "had.h"

namespace {

using at::ScalarType;
using at::Tensor;

// A Python exception to be raised at the entry point.
struct Refused {
    PyObject *type;
    std::string what;
};

[[noreturn]] void type_error(const std::string &what) { throw Refused{PyExc_TypeError, what}; }
[[noreturn]] void value_error(const std::string &what) { throw Refused{PyExc_ValueError, what}; }

// A pool of pages and the tensors that hold it.
struct Pool {
    had_cache_t c;
    int device;
    Tensor kbits, vcodes, vscale;
};

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const char *type_name(ScalarType t)
{
    switch (t) {
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    default: return c10::toString(t);
    }
}

// A contiguous CUDA tensor of `ndim` dimensions; on `device` unless that is -1.
const Tensor &cuda_tensor(PyObject *o, const char *name, int64_t ndim, int device = -1)
{
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda())
        value_error(std::string(name) + " must be a CUDA tensor (the HAD library has no CPU path)");
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    if (t.dim() != ndim)
        value_error(std::string(name) + " must have " + std::to_string(ndim) + " dimensions, got " +
                    std::to_string(t.dim()));
    if (device >= 0 && t.get_device() != device)
        value_error(std::string(name) + " is on " + t.device().str() +
                    ", the other tensors on cuda:" + std::to_string(device));
    for (int64_t n : t.sizes())
        if (n > INT_MAX) value_error(std::string(name) + " has more than 2^31 - 1 entries a dimension");
    return t;
}

const Tensor &typed(PyObject *o, const char *name, ScalarType type, int64_t ndim, int device = -1)
{
    const Tensor &t = cuda_tensor(o, name, ndim, device);
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + type_name(type) + ", got " +
                   type_name(t.scalar_type()));
    return t;
}

template <typename P>
P *shaped(PyObject *o, const char *name, ScalarType type, at::IntArrayRef shape, int device)
{
    const Tensor &t = typed(o, name, type, (int64_t)shape.size(), device);
    if (t.sizes() != shape)
        value_error(std::string(name) + " must have shape " + shape_text(shape) + ", got " +
                    shape_text(t.sizes()));
    return static_cast<P *>(t.data_ptr());
}

int32_t *ints(PyObject *o, const char *name, int64_t n, int device)
{
    return shaped<int32_t>(o, name, ScalarType::Int, {n}, device);
}

int32_t *maybe_ints(PyObject *o, const char *name, int64_t n, int device)
{
    return o == Py_None ? nullptr : ints(o, name, n, device);
}

// A whole number that the C ABI's int holds.
int number(PyObject *o, const char *name)
{
    int overflow = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (x == -1 && !overflow && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be an integer");
    }
    if (overflow || x > INT_MAX || x < INT_MIN) value_error(std::string(name) + " must fit 32 bits");
    return (int)x;
}

had_dtype_t dtype_code(const Tensor &t, const char *name)
{
    if (t.scalar_type() == ScalarType::BFloat16) return HAD_BF16;
    if (t.scalar_type() == ScalarType::Float) return HAD_F32;
    type_error(std::string(name) + " must be bfloat16 or float32, got " + type_name(t.scalar_type()));
}

// The tensors' device made current for the call, and its current stream.
struct On {
    c10::cuda::CUDAGuard guard;
    cudaStream_t stream;
    explicit On(int device)
        : guard((c10::DeviceIndex)device),
          stream(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream())
    {
    }
};

Tensor new_tensor(at::IntArrayRef shape, ScalarType type, int device)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, device));
}

// An output: the caller's, checked, or a new one.
Tensor output(PyObject *o, const char *name, ScalarType type, at::IntArrayRef shape, int device)
{
    if (o == Py_None) return new_tensor(shape, type, device);
    shaped<void>(o, name, type, shape, device);
    return THPVariable_Unpack(o);
}

constexpr const char *kPoolName = "sparse_attention_sigma_b200.cache.Pool";

void drop_pool(PyObject *capsule)
{
    delete static_cast<Pool *>(PyCapsule_GetPointer(capsule, kPoolName));
}

// The address of one of a pool's tensors now: a program may give a tensor other storage.
void *address(const Tensor &t, ScalarType type, at::IntArrayRef shape, int device)
{
    if (!t.is_cuda() || t.get_device() != device || t.scalar_type() != type || t.sizes() != shape ||
        !t.is_contiguous())
        value_error("a tensor of the cache is not what the cache was made of any more");
    return t.data_ptr();
}

const Pool &pool_of(PyObject *o)
{
    if (!PyCapsule_IsValid(o, kPoolName)) type_error("cache must be a Cache");
    Pool &p = *static_cast<Pool *>(PyCapsule_GetPointer(o, kPoolName));
    had_cache_t &c = p.c;
    c.kbits = static_cast<uint32_t *>(
        address(p.kbits, ScalarType::Int, {c.pages, c.heads, c.page, c.d / 32}, p.device));
    c.vcodes = static_cast<uint8_t *>(
        address(p.vcodes, ScalarType::Byte, {c.pages, c.heads, c.page, c.d / 2}, p.device));
    c.vscale = address(p.vscale, ScalarType::BFloat16, {c.pages, c.heads, c.page, 2}, p.device);
    return p;
}

PyObject *status_of(had_status_t s) { return PyLong_FromLong((long)s); }

// (status, outputs...)
template <typename... Ts>
PyObject *with_outputs(had_status_t s, const Ts &...ts)
{
    PyObject *r = PyTuple_New(1 + sizeof...(Ts));
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, status_of(s));
    Py_ssize_t i = 1;
    (PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(ts)), ...);
    return r;
}

// kbits, vcodes, vscale -> (capsule, pages, heads, page, d)
PyObject *make_pool(PyObject *const *a)
{
    const Tensor &kbits = typed(a[0], "kbits", ScalarType::Int, 4);
    const int device = kbits.get_device();
    const int64_t pages = kbits.size(0), heads = kbits.size(1), page = kbits.size(2), d = 32 * kbits.size(3);
    auto *codes = shaped<uint8_t>(a[1], "vcodes", ScalarType::Byte, {pages, heads, page, d / 2}, device);
    auto *scale = shaped<void>(a[2], "vscale", ScalarType::BFloat16, {pages, heads, page, 2}, device);
    if (d > INT_MAX) value_error("kbits has too long rows");
    Pool *p = new Pool{{static_cast<uint32_t *>(kbits.data_ptr()), codes, scale, (int)pages, (int)heads,
                        (int)page, (int)d}, device, kbits, THPVariable_Unpack(a[1]),
                       THPVariable_Unpack(a[2])};
    PyObject *capsule = PyCapsule_New(p, kPoolName, drop_pool);
    if (!capsule) {
        delete p;
        return nullptr;
    }
    return Py_BuildValue("Niiii", capsule, p->c.pages, p->c.heads, p->c.page, p->c.d);
}

// Address and row length of the table of B sequences.
int32_t *table_of(PyObject *o, int64_t B, int device, int *width)
{
    const Tensor &t = typed(o, "table", ScalarType::Int, 2, device);
    if (t.size(0) != B)
        value_error("table must have " + std::to_string(B) + " rows, got " + std::to_string(t.size(0)));
    *width = (int)t.size(1);
    return static_cast<int32_t *>(t.data_ptr());
}

// pool, k, v, sigma_k, table, start, counts, dev_status
PyObject *call_append(PyObject *const *a)
{
    const Pool &p = pool_of(a[0]);
    const Tensor &k = cuda_tensor(a[1], "k", 4, p.device);
    if (k.size(1) != p.c.heads || k.size(3) != p.c.d)
        value_error("k must be [B, " + std::to_string(p.c.heads) + ", T, " + std::to_string(p.c.d) +
                    "], got " + shape_text(k.sizes()));
    const had_dtype_t dt = dtype_code(k, "k");
    const int B = (int)k.size(0), T = (int)k.size(2);
    const void *v = shaped<void>(a[2], "v", k.scalar_type(), k.sizes(), p.device);
    const float *sigma = shaped<float>(a[3], "sigma_k", ScalarType::Float, {p.c.heads}, p.device);
    int width;
    const int32_t *table = table_of(a[4], B, p.device, &width);
    const int32_t *start = ints(a[5], "start", B, p.device);
    const int32_t *counts = maybe_ints(a[6], "counts", B, p.device);
    int32_t *status = maybe_ints(a[7], "dev_status", 1, p.device);
    On on(p.device);
    return status_of(had_cache_append(k.data_ptr(), v, dt, sigma, &p.c, table, width, start, counts, B,
                                      T, status, on.stream));
}

// pool, table, start, T, counts, bits, values, dev_status
PyObject *call_read(PyObject *const *a)
{
    const Pool &p = pool_of(a[0]);
    const int64_t B = typed(a[1], "table", ScalarType::Int, 2, p.device).size(0);
    int width;
    const int32_t *table = table_of(a[1], B, p.device, &width);
    const int32_t *start = ints(a[2], "start", B, p.device);
    const int T = number(a[3], "T");
    const int32_t *counts = maybe_ints(a[4], "counts", B, p.device);
    int32_t *status = maybe_ints(a[7], "dev_status", 1, p.device);
    if (T < 0) return with_outputs(HAD_ERR_INVALID_ARG);
    On on(p.device);
    const Tensor bits = output(a[5], "bits", ScalarType::Int, {B, p.c.heads, T, p.c.d / 32}, p.device);
    const Tensor values = output(a[6], "values", ScalarType::Float, {B, p.c.heads, T, p.c.d}, p.device);
    const had_status_t s = had_cache_read(&p.c, table, width, start, counts, (int)B, T,
                                          static_cast<uint32_t *>(bits.data_ptr()),
                                          static_cast<float *>(values.data_ptr()), status, on.stream);
    return with_outputs(s, bits, values);
}

// pool, q, sigma_q, table, lens, N, tau, window, sinks, counts, out, dev_status, max_len
PyObject *call_attention(PyObject *const *a)
{
    const Pool &p = pool_of(a[0]);
    const Tensor &q = cuda_tensor(a[1], "q", 4, p.device);
    if (q.size(3) != p.c.d)
        value_error("q must be [B, Hq, T, " + std::to_string(p.c.d) + "], got " + shape_text(q.sizes()));
    const had_dtype_t dt = dtype_code(q, "q");
    const int B = (int)q.size(0), Hq = (int)q.size(1), T = (int)q.size(2);
    const float *sigma = shaped<float>(a[2], "sigma_q", ScalarType::Float, {Hq}, p.device);
    int width;
    const int32_t *table = table_of(a[3], B, p.device, &width);
    const int32_t *lens = ints(a[4], "lens", B, p.device);
    const int N = number(a[5], "N");
    const double tau = PyFloat_AsDouble(a[6]);
    if (tau == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error("tau must be a number");
    }
    const int window = number(a[7], "window"), sinks = number(a[8], "sinks");
    const int max_len = number(a[12], "max_len");
    const int32_t *counts = maybe_ints(a[9], "counts", B, p.device);
    int32_t *status = maybe_ints(a[11], "dev_status", 1, p.device);
    On on(p.device);
    const Tensor out = output(a[10], "out", ScalarType::Float, q.sizes(), p.device);
    const had_status_t s = had_cache_attention(q.data_ptr(), dt, sigma, &p.c, table, width, lens, counts,
                                               B, Hq, T, N, (float)tau, window, sinks, max_len,
                                               static_cast<float *>(out.data_ptr()), status, on.stream);
    return with_outputs(s, out);
}

// The books of a call: table, refs and, unless o_lens is null, lens.
struct BookArgs {
    int device, S, width, pages;
    int32_t *table, *lens, *refs;
    BookArgs(PyObject *o_table, PyObject *o_lens, PyObject *o_refs)
    {
        const Tensor &t = typed(o_table, "table", ScalarType::Int, 2);
        device = t.get_device();
        S = (int)t.size(0);
        width = (int)t.size(1);
        table = static_cast<int32_t *>(t.data_ptr());
        lens = o_lens ? ints(o_lens, "lens", S, device) : nullptr;
        const Tensor &r = typed(o_refs, "refs", ScalarType::Int, 1, device);
        pages = (int)r.size(0);
        refs = static_cast<int32_t *>(r.data_ptr());
    }
};

// table, lens, refs, page, src, dst, dev_status
PyObject *call_fork(PyObject *const *a)
{
    const BookArgs k(a[0], a[1], a[2]);
    const int page = number(a[3], "page");
    const Tensor &src = typed(a[4], "src", ScalarType::Int, 1, k.device);
    const int32_t *dst = ints(a[5], "dst", src.size(0), k.device);
    int32_t *status = maybe_ints(a[6], "dev_status", 1, k.device);
    On on(k.device);
    return status_of(had_cache_fork(k.table, k.lens, k.refs, k.S, k.width, k.pages, page,
                                    static_cast<int32_t *>(src.data_ptr()), dst, (int)src.size(0),
                                    status, on.stream));
}

// table, lens, refs, page, grow, src, dst, dev_status
PyObject *call_reserve(PyObject *const *a)
{
    const BookArgs k(a[0], a[1], a[2]);
    const int page = number(a[3], "page");
    const int32_t *grow = ints(a[4], "grow", k.S, k.device);
    int32_t *status = maybe_ints(a[7], "dev_status", 1, k.device);
    On on(k.device);
    const Tensor src = output(a[5], "src", ScalarType::Int, {k.S}, k.device);
    const Tensor dst = output(a[6], "dst", ScalarType::Int, {k.S}, k.device);
    const had_status_t s = had_cache_reserve(k.table, k.lens, k.refs, k.S, k.width, k.pages, page, grow,
                                             static_cast<int32_t *>(src.data_ptr()),
                                             static_cast<int32_t *>(dst.data_ptr()), status, on.stream);
    return with_outputs(s, src, dst);
}

// table, lens, refs, seqs, dev_status
PyObject *call_free(PyObject *const *a)
{
    const BookArgs k(a[0], a[1], a[2]);
    const Tensor &seqs = typed(a[3], "seqs", ScalarType::Int, 1, k.device);
    int32_t *status = maybe_ints(a[4], "dev_status", 1, k.device);
    On on(k.device);
    return status_of(had_cache_free(k.table, k.lens, k.refs, k.S, k.width, k.pages,
                                    static_cast<int32_t *>(seqs.data_ptr()), (int)seqs.size(0), status,
                                    on.stream));
}

// table, lens, refs, page, window, sinks, dev_status
PyObject *call_evict(PyObject *const *a)
{
    const BookArgs k(a[0], a[1], a[2]);
    const int page = number(a[3], "page"), window = number(a[4], "window"), sinks = number(a[5], "sinks");
    int32_t *status = maybe_ints(a[6], "dev_status", 1, k.device);
    On on(k.device);
    return status_of(had_cache_evict(k.table, k.lens, k.refs, k.S, k.width, k.pages, page, window, sinks,
                                     status, on.stream));
}

// table, refs, src, dst, live, dev_status
PyObject *call_compact(PyObject *const *a)
{
    const BookArgs k(a[0], nullptr, a[1]);
    int32_t *status = maybe_ints(a[5], "dev_status", 1, k.device);
    On on(k.device);
    const Tensor src = output(a[2], "src", ScalarType::Int, {k.pages}, k.device);
    const Tensor dst = output(a[3], "dst", ScalarType::Int, {k.pages}, k.device);
    const Tensor live = output(a[4], "live", ScalarType::Int, {1}, k.device);
    const had_status_t s = had_cache_compact(k.table, k.refs, k.S, k.width, k.pages,
                                             static_cast<int32_t *>(src.data_ptr()),
                                             static_cast<int32_t *>(dst.data_ptr()),
                                             static_cast<int32_t *>(live.data_ptr()), status, on.stream);
    return with_outputs(s, src, dst, live);
}

// pool, src, dst, dev_status
PyObject *call_copy_pages(PyObject *const *a)
{
    const Pool &p = pool_of(a[0]);
    const Tensor &src = typed(a[1], "src", ScalarType::Int, 1, p.device);
    const int32_t *dst = ints(a[2], "dst", src.size(0), p.device);
    int32_t *status = maybe_ints(a[3], "dev_status", 1, p.device);
    On on(p.device);
    return status_of(had_cache_copy_pages(&p.c, static_cast<int32_t *>(src.data_ptr()), dst,
                                          (int)src.size(0), status, on.stream));
}

// One entry point: the number of arguments, and C++ exceptions as Python ones.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    HANDLE_TH_ERRORS
    try {
        return F(args);
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name)
{
    return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
                       METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<make_pool, 3>("pool"),       method<call_append, 8>("append"),
    method<call_read, 8>("read"),            method<call_attention, 13>("attention"),
    method<call_fork, 7>("fork"),            method<call_reserve, 8>("reserve"),
    method<call_free, 5>("free"),       method<call_evict, 7>("evict"),
    method<call_compact, 6>("compact"),      method<call_copy_pages, 4>("copy_pages"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache(void) { return PyModule_Create(&module); }
