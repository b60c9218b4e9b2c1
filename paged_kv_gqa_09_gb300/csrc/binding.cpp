// binding.cpp -- the Python side of the calls a serving loop makes per layer and
// token (the 4-bit cache and windowed decode): it checks that every tensor lives
// on the current CUDA device with the dtype, layout and size the C ABI expects
// and forwards raw pointers and a stream.  ctypes did the same in about 5 us a
// call on the host; this takes a few tenths.
//
// The module holds no state but the entry points of the libpkv that the package
// has loaded, which it is given once.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <string>

#include "pkv.h"

namespace {

struct Refused {
    PyObject *type;
    std::string what;
};

struct {
    decltype(&pkv_attn_workspace_size) ws_size;
    decltype(&pkv_quant_append) append;
    decltype(&pkv_quant_read) read;
    decltype(&pkv_quant_decode) quant;
    decltype(&pkv_window_decode) window;
} lib;

const char *name_of(at::ScalarType t)
{
    return t == at::kHalf ? "torch.float16" : t == at::kInt ? "torch.int32" : t == at::kFloat ? "torch.float32" : "torch.uint8";
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        throw Refused{PyExc_TypeError, std::string(name) + " must be a torch tensor"};
    return THPVariable_Unpack(o);
}

// One call's arguments: the shape, the current device and the stream.
struct Call {
    pkv_shape_t s;
    int dev = -1;  // not looked up before there is a CUDA tensor

    explicit Call(PyObject *shape)
    {
        Py_buffer b;
        if (PyObject_GetBuffer(shape, &b, PyBUF_SIMPLE) != 0)
            throw Refused{nullptr, ""};
        const bool fits = b.len == (Py_ssize_t)sizeof s;
        if (fits)
            s = *static_cast<const pkv_shape_t *>(b.buf);
        PyBuffer_Release(&b);
        if (!fits)
            throw Refused{PyExc_TypeError, "shape must be a Shape"};
    }

    void on_device(const at::Tensor &t, const char *name)
    {
        if (!t.is_cuda())
            throw Refused{PyExc_ValueError, std::string(name) + " must be a CUDA tensor (got " + t.device().str() + ")"};
        if (dev < 0)
            dev = c10::cuda::current_device();
        if (t.get_device() != dev)
            throw Refused{PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", current device is cuda:" +
                                                std::to_string(dev)};
    }

    // Pointer of a contiguous tensor of `type` with at least n elements.
    template <class T = void>
    T *arg(PyObject *o, const char *name, at::ScalarType type, int64_t n, bool nullable = false)
    {
        if (nullable && o == Py_None)
            return nullptr;
        const at::Tensor &t = tensor(o, name);
        on_device(t, name);
        if (t.scalar_type() != type)
            throw Refused{PyExc_ValueError, std::string(name) + " must be " + name_of(type)};
        if (!t.is_contiguous())
            throw Refused{PyExc_ValueError, std::string(name) + " must be contiguous"};
        if (t.numel() < n)
            throw Refused{PyExc_ValueError, std::string(name) + " has " + std::to_string(t.numel()) + " elements, needs " +
                                                std::to_string(n)};
        return static_cast<T *>(t.data_ptr());
    }

    void *workspace(PyObject *o)
    {
        const at::Tensor &t = tensor(o, "workspace");
        on_device(t, "workspace");
        if (!t.is_contiguous())
            throw Refused{PyExc_ValueError, "workspace must be contiguous"};
        const size_t need = lib.ws_size(&s);  // 0 for a bad shape, which the call itself refuses
        if ((size_t)t.nbytes() < need)
            throw Refused{PyExc_ValueError, "workspace has " + std::to_string(t.nbytes()) + " bytes, needs " + std::to_string(need)};
        return t.data_ptr();
    }

    int32_t *table(PyObject *o) { return arg<int32_t>(o, "block_table", at::kInt, (int64_t)s.B * s.bt_stride); }
    int32_t *lens(PyObject *o, const char *name = "seq_lens", bool nullable = false) { return arg<int32_t>(o, name, at::kInt, s.B, nullable); }
    int32_t *offsets(PyObject *o, const char *name, bool nullable) { return arg<int32_t>(o, name, at::kInt, (int64_t)s.B + 1, nullable); }
    void *rows(PyObject *o, const char *name) { return arg(o, name, at::kHalf, (int64_t)s.B * s.Hq * s.d); }
    float *lse(PyObject *o) { return arg<float>(o, "lse", at::kFloat, (int64_t)s.B * s.Hq, true); }
    void *pages(PyObject *o, const char *name) { return arg(o, name, at::kHalf, (int64_t)s.num_pages * s.page_size * s.Hkv * s.d); }
    void *quant(PyObject *o)
    {
        return arg(o, "quant_cache", at::kByte, (int64_t)s.num_pages * s.Hkv * ((int64_t)s.page_size * s.d * 5 / 4));
    }

    // Packed K and V [T, Hkv, d], whose tokens may be strided (alike in both);
    // a size of one or none leaves a stride without meaning.
    void packed(PyObject *ko, PyObject *vo, const char *kname, const char *vname, void *&k, void *&v, int32_t &T, int64_t &stride)
    {
        const at::Tensor &kt = tensor(ko, kname), &vt = tensor(vo, vname);
        const int64_t n = kt.dim() == 3 ? kt.size(0) : -1;
        if (n > INT32_MAX)
            throw Refused{PyExc_ValueError, std::string(kname) + " has too many tokens"};
        T = (int32_t)n;
        stride = n > 1 ? kt.stride(0) : (int64_t)s.Hkv * s.d;
        for (int u = 0; u < 2; ++u) {
            const at::Tensor &t = u ? vt : kt;
            const char *name = u ? vname : kname;
            on_device(t, name);
            if (t.scalar_type() != at::kHalf)
                throw Refused{PyExc_ValueError, std::string(name) + " must be torch.float16"};
            if (t.dim() != 3 || t.size(0) != n || t.size(1) != s.Hkv || t.size(2) != s.d)
                throw Refused{PyExc_ValueError, std::string(name) + " must be [tokens, " + std::to_string(s.Hkv) + ", " +
                                                    std::to_string(s.d) + "], K and V alike"};
            if (n > 0 && (t.stride(2) != 1 || (s.Hkv > 1 && t.stride(1) != s.d)))
                throw Refused{PyExc_ValueError, std::string(name) + " must be contiguous within a token"};
            if (n > 1 && t.stride(0) != stride)
                throw Refused{PyExc_ValueError, std::string(kname) + " and " + vname + " must have one token stride"};
        }
        k = kt.data_ptr();
        v = vt.data_ptr();
    }

    void *stream(PyObject *o)
    {
        if (o == Py_None)
            return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        void *p = PyLong_AsVoidPtr(o);
        if (!p && PyErr_Occurred())
            throw Refused{nullptr, ""};
        return p;
    }
};

int32_t int32(PyObject *o, const char *name)
{
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred())
        throw Refused{nullptr, ""};
    if (x < INT32_MIN || x > INT32_MAX)
        throw Refused{PyExc_ValueError, std::string(name) + " does not fit an int32"};
    return (int32_t)x;
}

// Runs `f`, which checks its arguments and returns the call to make; that one
// is made without the interpreter's lock.
template <class F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F &&f)
{
    try {
        if (got != want)
            throw Refused{PyExc_TypeError, "wrong number of arguments"};
        auto call = f();
        int st = 0;
        Py_BEGIN_ALLOW_THREADS
        st = call();
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(st);
    } catch (const Refused &r) {
        if (r.type)
            PyErr_SetString(r.type, r.what.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (shape, ws, k_new, v_new, block_table, seq_lens, quant_cache, new_offsets, seq_lens_out, stream)
PyObject *quant_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [a] {
        Call c(a[0]);
        void *k, *v;
        int32_t T;
        int64_t step;
        c.packed(a[2], a[3], "k_new", "v_new", k, v, T, step);
        void *ws = c.workspace(a[1]);
        int32_t *bt = c.table(a[4]), *sl = c.lens(a[5]);
        void *cache = c.quant(a[6]);
        int32_t *off = c.offsets(a[7], "new_offsets", true);
        int32_t *out = a[8] == Py_None ? sl : c.lens(a[8], "seq_lens_out");
        void *st = c.stream(a[9]);
        return [=] { return lib.append(&c.s, ws, k, v, step, T, off, bt, sl, out, cache, st); };
    });
}

// (shape, ws, quant_cache, block_table, seq_lens, out_offsets, k_out, v_out, first, stream)
PyObject *quant_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [a] {
        Call c(a[0]);
        void *k, *v;
        int32_t T;
        int64_t step;
        c.packed(a[6], a[7], "k_out", "v_out", k, v, T, step);
        void *ws = c.workspace(a[1]), *cache = c.quant(a[2]);
        int32_t *bt = c.table(a[3]), *sl = c.lens(a[4]), *off = c.offsets(a[5], "out_offsets", false);
        int32_t *first = c.lens(a[8], "first", true);
        void *st = c.stream(a[9]);
        return [=] { return lib.read(&c.s, ws, cache, bt, sl, first, off, T, k, v, step, st); };
    });
}

// (shape, ws, q, quant_cache, block_table, seq_lens, o, lse, window, sinks, stream)
PyObject *quant_decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [a] {
        Call c(a[0]);
        void *ws = c.workspace(a[1]), *q = c.rows(a[2], "q"), *cache = c.quant(a[3]);
        int32_t *bt = c.table(a[4]), *sl = c.lens(a[5]);
        void *o = c.rows(a[6], "o");
        float *lse = c.lse(a[7]);
        const bool whole = a[8] == Py_None;
        const pkv_window_t win = {whole ? 0 : int32(a[8], "window"), int32(a[9], "sinks")};
        void *st = c.stream(a[10]);
        return [=] { return lib.quant(&c.s, whole ? nullptr : &win, ws, q, cache, bt, sl, o, lse, st); };
    });
}

// (shape, ws, q, k_cache, v_cache, block_table, seq_lens, window, sinks, o, lse, stream)
PyObject *window_decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 12, [a] {
        Call c(a[0]);
        void *ws = c.workspace(a[1]), *q = c.rows(a[2], "q");
        void *k = c.pages(a[3], "k_cache"), *v = c.pages(a[4], "v_cache");
        int32_t *bt = c.table(a[5]), *sl = c.lens(a[6]);
        const pkv_window_t win = {int32(a[7], "window"), int32(a[8], "sinks")};
        void *o = c.rows(a[9], "o");
        float *lse = c.lse(a[10]);
        void *st = c.stream(a[11]);
        return [=] { return lib.window(&c.s, &win, ws, q, k, v, bt, sl, o, lse, st); };
    });
}

// Addresses of pkv_attn_workspace_size, pkv_quant_append, pkv_quant_read, pkv_quant_decode, pkv_window_decode
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    void *p[5];
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "five addresses");
        return nullptr;
    }
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    lib.ws_size = reinterpret_cast<decltype(lib.ws_size)>(p[0]);
    lib.append = reinterpret_cast<decltype(lib.append)>(p[1]);
    lib.read = reinterpret_cast<decltype(lib.read)>(p[2]);
    lib.quant = reinterpret_cast<decltype(lib.quant)>(p[3]);
    lib.window = reinterpret_cast<decltype(lib.window)>(p[4]);
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"quant_append", fast(quant_append), METH_FASTCALL, nullptr},
                         {"quant_read", fast(quant_read), METH_FASTCALL, nullptr},
                         {"quant_decode", fast(quant_decode), METH_FASTCALL, nullptr},
                         {"window_decode", fast(window_decode), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_call(void) { return PyModule_Create(&module); }
