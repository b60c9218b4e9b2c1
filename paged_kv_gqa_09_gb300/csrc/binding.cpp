// binding.cpp -- the Python side of the calls a serving loop makes per layer and
// token (pages and slots, the 4-bit and 8-bit caches, windowed decode): it checks that every tensor lives
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
#include <initializer_list>
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
    decltype(&pkv_map_pages) map;
    decltype(&pkv_append_slots) slots;
    decltype(&pkv_byte_append) append8;
    decltype(&pkv_byte_read) read8;
    decltype(&pkv_byte_decode) decode8;
} lib;

const char *name_of(at::ScalarType t)
{
    return t == at::kHalf ? "torch.float16" : t == at::kInt ? "torch.int32" : t == at::kFloat ? "torch.float32" : t == at::kLong ? "torch.int64" : "torch.uint8";
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
    // Elements of an array of these extents, INT64_MAX where that many cannot be
    // counted; 0 with an extent of a bad shape, which the call itself refuses.
    static int64_t elements(std::initializer_list<int64_t> extents)
    {
        int64_t n = 1;
        for (int64_t x : extents)
            if (x <= 0)
                return 0;
        for (int64_t x : extents)
            if (__builtin_mul_overflow(n, x, &n))
                return INT64_MAX;
        return n;
    }

    void *rows(PyObject *o, const char *name) { return arg(o, name, at::kHalf, elements({s.B, s.Hq, s.d})); }
    float *lse(PyObject *o) { return arg<float>(o, "lse", at::kFloat, (int64_t)s.B * s.Hq, true); }
    void *pages(PyObject *o, const char *name) { return arg(o, name, at::kHalf, elements({s.num_pages, s.page_size, s.Hkv, s.d})); }
    void *quant(PyObject *o)
    {
        return arg(o, "quant_cache", at::kByte, elements({s.num_pages, s.Hkv, (int64_t)s.page_size * s.d * 5 / 4}));
    }

    void *codes(PyObject *o)
    {
        const int64_t tb = s.page_size < 64 ? s.page_size : 64, blocks = tb < 1 ? 0 : s.page_size / tb;
        return arg(o, "byte_cache", at::kByte, elements({s.num_pages, s.Hkv, blocks, 2 * tb * s.d + (tb == 64 ? 32 : 16)}));
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

// Tokens of a one-dimensional tensor that says how many a call is for.
int32_t length(const at::Tensor &t, const char *name)
{
    if (t.numel() > INT32_MAX)
        throw Refused{PyExc_ValueError, std::string(name) + " has too many entries"};
    return (int32_t)t.numel();
}

// (shape, ws, seq_lens, new_lens, block_table, free_pages, free_count, slot_map, new_offsets, seq_lens_out,
//  free_count_out, positions, stream)
PyObject *map_pages(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [a] {
        Call c(a[0]);
        void *ws = c.workspace(a[1]);
        int32_t *sl = c.lens(a[2]), *nl = c.lens(a[3], "new_lens"), *bt = c.table(a[4]);
        int32_t *fp = c.arg<int32_t>(a[5], "free_pages", at::kInt, 0);
        const int32_t cap = length(tensor(a[5], "free_pages"), "free_pages");
        int32_t *fc = c.arg<int32_t>(a[6], "free_count", at::kInt, 1);
        int64_t *slots = c.arg<int64_t>(a[7], "slot_map", at::kLong, 0);
        const int32_t T = length(tensor(a[7], "slot_map"), "slot_map");
        int32_t *off = c.offsets(a[8], "new_offsets", false);
        int32_t *out = a[9] == Py_None ? sl : c.lens(a[9], "seq_lens_out");
        int32_t *fout = a[10] == Py_None ? fc : c.arg<int32_t>(a[10], "free_count_out", at::kInt, 1);
        int32_t *pos = c.arg<int32_t>(a[11], "positions", at::kInt, T, true);
        void *st = c.stream(a[12]);
        return [=] { return lib.map(&c.s, ws, sl, nl, out, bt, fp, cap, fc, fout, off, slots, pos, T, st); };
    });
}

// (shape, ws, k_new, v_new, slot_map, k_cache, v_cache, stream)
PyObject *append_slots(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [a] {
        Call c(a[0]);
        void *k, *v;
        int32_t T;
        int64_t step;
        c.packed(a[2], a[3], "k_new", "v_new", k, v, T, step);
        void *ws = c.workspace(a[1]);
        int64_t *slots = c.arg<int64_t>(a[4], "slot_map", at::kLong, T);
        void *kc = c.pages(a[5], "k_cache"), *vc = c.pages(a[6], "v_cache");
        void *st = c.stream(a[7]);
        return [=] { return lib.slots(&c.s, ws, k, v, step, T, slots, kc, vc, st); };
    });
}

// (shape, ws, format, k_new, v_new, block_table, seq_lens, byte_cache, new_offsets, seq_lens_out, stream)
PyObject *byte_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [a] {
        Call c(a[0]);
        const int32_t format = int32(a[2], "format");
        void *k, *v;
        int32_t T;
        int64_t step;
        c.packed(a[3], a[4], "k_new", "v_new", k, v, T, step);
        void *ws = c.workspace(a[1]);
        int32_t *bt = c.table(a[5]), *sl = c.lens(a[6]);
        void *cache = c.codes(a[7]);
        int32_t *off = c.offsets(a[8], "new_offsets", true);
        int32_t *out = a[9] == Py_None ? sl : c.lens(a[9], "seq_lens_out");
        void *st = c.stream(a[10]);
        return [=] { return lib.append8(&c.s, ws, format, k, v, step, T, off, bt, sl, out, cache, st); };
    });
}

// (shape, ws, format, byte_cache, block_table, seq_lens, out_offsets, k_out, v_out, first, stream)
PyObject *byte_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [a] {
        Call c(a[0]);
        const int32_t format = int32(a[2], "format");
        void *k, *v;
        int32_t T;
        int64_t step;
        c.packed(a[7], a[8], "k_out", "v_out", k, v, T, step);
        void *ws = c.workspace(a[1]), *cache = c.codes(a[3]);
        int32_t *bt = c.table(a[4]), *sl = c.lens(a[5]), *off = c.offsets(a[6], "out_offsets", false);
        int32_t *first = c.lens(a[9], "first", true);
        void *st = c.stream(a[10]);
        return [=] { return lib.read8(&c.s, ws, format, cache, bt, sl, first, off, T, k, v, step, st); };
    });
}

// (shape, ws, format, q, byte_cache, block_table, seq_lens, o, lse, window, sinks, stream)
PyObject *byte_decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 12, [a] {
        Call c(a[0]);
        const int32_t format = int32(a[2], "format");
        void *ws = c.workspace(a[1]), *q = c.rows(a[3], "q"), *cache = c.codes(a[4]);
        int32_t *bt = c.table(a[5]), *sl = c.lens(a[6]);
        void *o = c.rows(a[7], "o");
        float *lse = c.lse(a[8]);
        const bool whole = a[9] == Py_None;
        const pkv_window_t win = {whole ? 0 : int32(a[9], "window"), int32(a[10], "sinks")};
        void *st = c.stream(a[11]);
        return [=] { return lib.decode8(&c.s, whole ? nullptr : &win, ws, format, q, cache, bt, sl, o, lse, st); };
    });
}

// Addresses of pkv_attn_workspace_size, pkv_quant_append, pkv_quant_read, pkv_quant_decode, pkv_window_decode,
// pkv_map_pages, pkv_append_slots, pkv_byte_append, pkv_byte_read, pkv_byte_decode
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    void *p[10];
    if (n != 10) {
        PyErr_SetString(PyExc_TypeError, "ten addresses");
        return nullptr;
    }
    for (int i = 0; i < 10; ++i) {
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
    lib.map = reinterpret_cast<decltype(lib.map)>(p[5]);
    lib.slots = reinterpret_cast<decltype(lib.slots)>(p[6]);
    lib.append8 = reinterpret_cast<decltype(lib.append8)>(p[7]);
    lib.read8 = reinterpret_cast<decltype(lib.read8)>(p[8]);
    lib.decode8 = reinterpret_cast<decltype(lib.decode8)>(p[9]);
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"quant_append", fast(quant_append), METH_FASTCALL, nullptr},
                         {"quant_read", fast(quant_read), METH_FASTCALL, nullptr},
                         {"quant_decode", fast(quant_decode), METH_FASTCALL, nullptr},
                         {"window_decode", fast(window_decode), METH_FASTCALL, nullptr},
                         {"map_pages", fast(map_pages), METH_FASTCALL, nullptr},
                         {"append_slots", fast(append_slots), METH_FASTCALL, nullptr},
                         {"byte_append", fast(byte_append), METH_FASTCALL, nullptr},
                         {"byte_read", fast(byte_read), METH_FASTCALL, nullptr},
                         {"byte_decode", fast(byte_decode), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_call(void) { return PyModule_Create(&module); }
