// csa2_torch.cpp -- the Python binding's short calls (cache rows, dense
// attention): arguments are taken from tensors here, because on the GPU these
// calls can be shorter than the interpreter needs for the same checks (a row
// read of 129 rows: 1.7 us on the GPU, 8 us of checks and ctypes in Python).
// Marshalling only, as in the rest of the binding: every refusal is a CsaError
// (with what Python raised on the way, if anything, as its cause), no memory for a
// workspace is PyTorch's OutOfMemoryError, and no C++ exception leaves a function.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "csa2.h"

namespace {

PyObject *g_error = nullptr;      // the package's CsaError
PyObject *g_memory = nullptr;     // PyTorch's OutOfMemoryError

struct Refusal { std::string what; };
struct Raised {};                 // a Python exception is set already

[[noreturn]] void refuse(const std::string &what) { throw Refusal{what}; }

// A reference held for the time of a block (a null one: an exception is set).
struct Ref {
    PyObject *o;
    explicit Ref(PyObject *p) : o(p) { if (p == nullptr) throw Raised{}; }
    ~Ref() { Py_XDECREF(o); }
    Ref(const Ref &) = delete;
};

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// nullptr for None
const at::Tensor *maybe(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

long long whole(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

bool type_of(at::ScalarType t, csa2_dtype *out)
{
    switch (t) {
    case at::kFloat: *out = CSA2_F32; return true;
    case at::kBFloat16: *out = CSA2_BF16; return true;
    case at::kHalf: *out = CSA2_F16; return true;
    default: return false;
    }
}

template <typename T>
T *at_of(const at::Tensor *t) { return t == nullptr ? nullptr : static_cast<T *>(t->data_ptr()); }

// The current device, which all tensors must be on: a call runs on its stream.
struct Device {
    int dev;
    explicit Device(const at::Tensor &first) : dev(first.is_cuda() ? (int)first.get_device() : -1)
    {
        if (dev < 0) refuse("tensor is not on a CUDA device");
        const int now = (int)c10::cuda::current_device();
        if (dev != now)
            refuse("tensors on cuda:" + std::to_string(dev) + ", the current device is cuda:" + std::to_string(now));
    }
    void holds(const at::Tensor *t, const char *name) const
    {
        if (t != nullptr && (!t->is_cuda() || (int)t->get_device() != dev))
            refuse(std::string(name) + " is not on cuda:" + std::to_string(dev));
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

const uint32_t *counters_of(PyObject *o, const Device &d, const at::Tensor **t)
{
    *t = maybe(o, "counters");
    d.holds(*t, "counters");
    if (*t != nullptr && ((*t)->scalar_type() != at::kInt || (*t)->numel() < CSA2_NUM_COUNTERS || !(*t)->is_contiguous()))
        refuse("counters must be contiguous int32 [" + std::to_string(CSA2_NUM_COUNTERS) + "]");
    return at_of<uint32_t>(*t);
}

// csa2_cache of a Cache object; its tensors are the object's, which the caller holds.
struct CacheArg {
    csa2_cache c{};
    CacheArg(PyObject *cache, const Device &d)
    {
        static PyObject *names[10] = {};
        if (names[0] == nullptr) {
            static const char *const n[10] = {"codes", "scales", "kidx", "kscale", "seq_base", "seq_len",
                                              "cap", "batch", "d_idx", "m"};
            for (int i = 9; i >= 0; --i)
                if ((names[i] = PyUnicode_InternFromString(n[i])) == nullptr) throw Raised{};
        }
        void *p[6];
        for (int i = 0; i < 6; ++i) {
            const Ref o(PyObject_GetAttr(cache, names[i]));
            const at::Tensor *t = maybe(o.o, "cache tensor");
            if (t == nullptr && i != 2 && i != 3) refuse("a cache tensor is None");
            d.holds(t, "cache");
            p[i] = at_of<void>(t);
        }
        long long v[4];
        for (int i = 0; i < 4; ++i) {
            const Ref o(PyObject_GetAttr(cache, names[6 + i]));
            v[i] = whole(o.o);
        }
        c.codes = static_cast<uint8_t *>(p[0]);
        c.scales = static_cast<uint8_t *>(p[1]);
        c.kidx = static_cast<uint8_t *>(p[2]);
        c.kscale = static_cast<float *>(p[3]);
        c.seq_base = static_cast<const int64_t *>(p[4]);
        c.seq_len = static_cast<int32_t *>(p[5]);
        c.cap = v[0];
        c.batch = (int32_t)v[1];
        c.d_idx = (int32_t)v[2];
        c.m = (int32_t)v[3];
    }
};

void check(csa2_status s, const char *what)
{
    if (s != CSA2_OK) refuse(std::string(what) + ": " + csa2_status_string(s));
}

std::string shape_of(const at::Tensor &t)
{
    std::string s = "[";
    for (const int64_t v : t.sizes()) s += std::to_string(v) + ", ";
    return s + "]";
}

bool is(const at::Tensor &t, int64_t a, int64_t b) { return t.dim() == 2 && t.size(0) == a && t.size(1) == b; }

// Makes the Python exception that is set (a wrong type, a missing attribute) the
// cause of a CsaError of the same words; an interrupt or a lack of memory stays.
void as_refusal(PyObject *type)
{
    PyObject *const cause = PyErr_GetRaisedException();
    if (!PyErr_GivenExceptionMatches(cause, PyExc_Exception) || PyErr_GivenExceptionMatches(cause, PyExc_MemoryError)) {
        PyErr_SetRaisedException(cause);
        return;
    }
    PyErr_Format(type, "%S", cause);
    PyObject *const e = PyErr_GetRaisedException();
    PyException_SetCause(e, cause);       // (takes the reference)
    PyErr_SetRaisedException(e);
}

// Runs f, turning what it throws into a Python exception.
template <typename F>
PyObject *guarded(F f)
{
    PyObject *const type = g_error != nullptr ? g_error : PyExc_RuntimeError;
    try {
        return f();
    } catch (const Raised &) {
        as_refusal(type);
    } catch (const Refusal &r) {
        PyErr_SetString(type, r.what.c_str());
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(g_memory != nullptr ? g_memory : PyExc_MemoryError, e.what_without_backtrace());
    } catch (const c10::Error &e) {       // (a tensor without the storage or strides that a call needs)
        PyErr_SetString(type, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(type, e.what());
    } catch (...) {
        PyErr_SetString(type, "unknown error");
    }
    return nullptr;
}

void arguments(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) refuse("wrong number of arguments");
}

// (cache, rows, x, key, counters)
PyObject *row_call(PyObject *const *a, Py_ssize_t n_args, bool write)
{
    return guarded([&]() -> PyObject * {
        const char *what = write ? "csa2_cache_write" : "csa2_cache_read";
        arguments(n_args, 5);
        const at::Tensor &rows = tensor(a[1], "rows"), &x = tensor(a[2], "x");
        const at::Tensor *key = maybe(a[3], "key");
        if (rows.scalar_type() != at::kLong || rows.dim() != 1 || !rows.is_contiguous())
            refuse("rows must be contiguous int64 [n], got " + shape_of(rows));
        const int64_t n = rows.size(0);
        csa2_dtype type;
        if (!type_of(x.scalar_type(), &type)) refuse(std::string(what) + ": x must be fp32, bf16 or f16");
        if (!is(x, n, CSA2_D) || x.stride(1) != 1)
            refuse(std::string(what) + ": x must be [n][512] with contiguous rows, got " + shape_of(x));
        if (key != nullptr && key->scalar_type() != (write ? x.scalar_type() : at::kFloat))
            refuse(std::string(what) + (write ? ": key must have x's type" : ": key must be fp32"));
        const Device d(x);
        d.holds(&rows, "rows");
        d.holds(key, "key");
        const CacheArg c(a[0], d);
        if (key != nullptr && (!is(*key, n, c.c.d_idx) || key->stride(1) != 1))
            refuse(std::string(what) + ": key must be [n][d_idx] with contiguous rows, got " + shape_of(*key));
        const at::Tensor *counters;
        uint32_t *cnt = const_cast<uint32_t *>(counters_of(a[4], d, &counters));
        // (the stride of a single row says nothing)
        const int64_t ld_x = n > 1 ? x.stride(0) : CSA2_D;
        const int64_t ld_key = key == nullptr ? 0 : n > 1 ? key->stride(0) : c.c.d_idx;
        const int64_t *r = at_of<const int64_t>(&rows);
        void *xp = x.data_ptr(), *kp = at_of<void>(key), *st = d.stream();
        csa2_status s;
        Py_BEGIN_ALLOW_THREADS
        s = write ? csa2_cache_write(&c.c, r, n, xp, type, ld_x, kp, ld_key, cnt, st)
                  : csa2_cache_read(&c.c, r, n, xp, type, ld_x, static_cast<float *>(kp), ld_key, cnt, st);
        Py_END_ALLOW_THREADS
        check(s, what);
        Py_RETURN_NONE;
    });
}

PyObject *cache_write(PyObject *, PyObject *const *a, Py_ssize_t n) { return row_call(a, n, true); }
PyObject *cache_read(PyObject *, PyObject *const *a, Py_ssize_t n) { return row_call(a, n, false); }

// (cache, seq, off, length, q, out, lse, prev_out, prev_lse, sm_scale, max_n, ws, counters)
PyObject *dense_attn(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject * {
        arguments(n_args, 13);
        const at::Tensor &seq = tensor(a[1], "seq"), &off = tensor(a[2], "off");
        const at::Tensor *length = maybe(a[3], "length");
        const at::Tensor &q = tensor(a[4], "q"), &out = tensor(a[5], "out");
        const at::Tensor *lse = maybe(a[6], "lse"), *po = maybe(a[7], "prev"), *pl = maybe(a[8], "prev");
        if (q.dim() != 3 || q.size(2) != CSA2_D || out.sizes() != q.sizes())
            refuse("dense_attn: q must be [nq][H][512] and out like it, got " + shape_of(q) + ", " + shape_of(out));
        csa2_dtype q_type, out_type;
        if (!type_of(q.scalar_type(), &q_type) || q_type == CSA2_F32 || !type_of(out.scalar_type(), &out_type))
            refuse("dense_attn: q must be bf16 or f16, out fp32, bf16 or f16");
        const int64_t nq = q.size(0), H = q.size(1);
        if (nq > INT32_MAX || H > INT32_MAX) refuse("dense_attn: q is too large");
        if (!q.is_contiguous() || !out.is_contiguous()) refuse("dense_attn: q and out must be contiguous");
        auto rows_ok = [&](const at::Tensor &t) { return t.scalar_type() == at::kFloat && is(t, nq, H) && t.is_contiguous(); };
        if (lse != nullptr && !rows_ok(*lse)) refuse("dense_attn: lse must be contiguous fp32 [nq][H]");
        if ((po == nullptr) != (pl == nullptr)) refuse("dense_attn: prev is a pair (out, lse)");
        if (po != nullptr && (po->scalar_type() != at::kFloat || po->sizes() != q.sizes() || !po->is_contiguous() || !rows_ok(*pl)))
            refuse("dense_attn: prev must be contiguous fp32 [nq][H][512] and [nq][H]");
        const Device d(q);
        auto ints = [&](const at::Tensor *t, int64_t n, const char *name) {
            if (t == nullptr) return;
            if (t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
                refuse(std::string("groups: ") + name + " must be contiguous int32 [" + std::to_string(n) + "]");
            d.holds(t, name);
        };
        const int64_t ng = seq.numel();
        if (ng > INT32_MAX) refuse("dense_attn: too many groups");
        ints(&seq, ng, "seq");
        ints(&off, ng + 1, "off");
        ints(length, ng, "length");
        d.holds(&out, "out");
        d.holds(lse, "lse");
        d.holds(po, "prev");
        d.holds(pl, "prev");
        const CacheArg c(a[0], d);
        const double sm = PyFloat_AsDouble(a[9]);
        if (sm == -1.0 && PyErr_Occurred()) throw Raised{};
        const int64_t max_n = a[10] == Py_None ? c.c.cap : (int64_t)whole(a[10]);
        const at::Tensor *counters;
        uint32_t *cnt = const_cast<uint32_t *>(counters_of(a[12], d, &counters));
        const at::Tensor *ws = maybe(a[11], "ws");
        void *st = d.stream(), *wp;
        size_t bytes;
        at::DataPtr own;          // freed as the call returns: later allocations of this stream come after the kernels
        if (ws != nullptr) {
            d.holds(ws, "ws");
            if (!ws->is_contiguous()) refuse("dense_attn: ws must be contiguous");
            wp = ws->data_ptr();
            bytes = ws->nbytes();
        } else {
            bytes = csa2_dense_workspace_size((int32_t)ng, (int32_t)nq, (int32_t)H, max_n);
            own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
            wp = own.get();
        }
        const csa2_groups g{at_of<const int32_t>(&seq), at_of<const int32_t>(&off), at_of<const int32_t>(length),
                            (int32_t)ng, (int32_t)nq};
        void *qp = q.data_ptr(), *op = out.data_ptr();
        float *lp = at_of<float>(lse), *pop = at_of<float>(po), *plp = at_of<float>(pl);
        csa2_status s;
        Py_BEGIN_ALLOW_THREADS
        s = csa2_dense_attn(&c.c, &g, max_n, qp, q_type, (int32_t)H, (float)sm, pop, plp, op, out_type, lp, wp, bytes, cnt, st);
        Py_END_ALLOW_THREADS
        check(s, "csa2_dense_attn");
        Py_RETURN_NONE;
    });
}

// (codes, scales, kidx, kscale, seq_base, seq_len) -> (cap, batch, d_idx): checks that they make a cache
PyObject *check_cache(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject * {
        arguments(n_args, 6);
        const at::Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales");
        const at::Tensor *kidx = maybe(a[2], "kidx"), *kscale = maybe(a[3], "kscale");
        const at::Tensor &base = tensor(a[4], "seq_base"), &len = tensor(a[5], "seq_len");
        if (codes.scalar_type() != at::kByte || scales.scalar_type() != at::kByte ||
            (kidx != nullptr && kidx->scalar_type() != at::kByte) ||
            (kscale != nullptr && kscale->scalar_type() != at::kFloat) || base.scalar_type() != at::kLong ||
            len.scalar_type() != at::kInt)
            refuse("cache tensors: codes, scales, kidx uint8, kscale fp32, seq_base int64, seq_len int32");
        for (const at::Tensor *t : {&scales, kidx, kscale, &base, &len})
            if (t != nullptr && t->device() != codes.device())
                refuse("cache tensors on " + codes.device().str() + " and " + t->device().str());
        if (!codes.is_contiguous() || !scales.is_contiguous() || (kidx != nullptr && !kidx->is_contiguous()) ||
            (kscale != nullptr && !kscale->is_contiguous()) || !base.is_contiguous() || !len.is_contiguous())
            refuse("cache tensors must be contiguous");
        const int64_t cap = codes.dim() == 2 ? codes.size(0) : -1;
        if (!is(codes, cap, CSA2_CODE_BYTES) || !is(scales, cap, CSA2_SCALE_BYTES) ||
            (kidx == nullptr) != (kscale == nullptr) ||
            (kidx != nullptr && (kidx->dim() != 2 || kidx->size(0) != cap || kscale->numel() != cap)) ||
            base.numel() != len.numel() + 1)
            refuse("cache tensors do not fit together");
        return Py_BuildValue("LLL", (long long)cap, (long long)len.numel(),
                             (long long)(kidx != nullptr ? kidx->size(1) : 128));
    });
}

// (CsaError, torch.OutOfMemoryError)
PyObject *set_errors(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject * {
        arguments(n_args, 2);
        Py_XSETREF(g_error, Py_NewRef(a[0]));
        Py_XSETREF(g_memory, Py_NewRef(a[1]));
        Py_RETURN_NONE;
    });
}

#define CSA2_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CSA2_FAST(cache_write), CSA2_FAST(cache_read), CSA2_FAST(dense_attn), CSA2_FAST(check_cache),
                         CSA2_FAST(set_errors), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "csa2_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject *PyInit_csa2_torch() { return PyModule_Create(&module); }
