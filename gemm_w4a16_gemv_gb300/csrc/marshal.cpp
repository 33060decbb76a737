// Host side of the Python binding for the operators of a decode step: checks a
// call's tensors and makes the call, without building Python objects on the
// way.
//
// Each function takes what the binding's function of that name takes, all of
// it and in order, finds sizes and addresses, and calls the C ABI on the
// current stream of the tensors' device (or the given handle).  It returns the
// library's status; or None if an argument is not what it has to be -- then
// nothing was called, and the binding goes through its own checks, which say
// what is wrong.  On a Grace core a call of kv4_plan takes 3.5 us this way; the
// same checks in Python and ctypes took 9.8 us, where the launch takes 2.5.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "w4a16.h"

namespace {

using at::ScalarType;

// The library's entry points (bind() finds them).
decltype(&kv4_plan) p_plan = nullptr;
decltype(&w4a16_qk_norm_rope) p_rope = nullptr;
decltype(&kv4_append) p_append = nullptr;
decltype(&kv4_gather) p_gather = nullptr;
decltype(&kv4_attention) p_attention = nullptr;
decltype(&kv4_bounds) p_bounds = nullptr;
decltype(&kv4_select) p_select = nullptr;
decltype(&kv4_sparse_attention) p_sparse = nullptr;
decltype(&kv4_prefix_attention) p_prefix = nullptr;
decltype(&w4a16_sample) p_sample = nullptr;

struct Unfit {};  // an argument that the binding has to look at

const at::Tensor &tensor(PyObject *o) {
    if (!THPVariable_Check(o)) throw Unfit();
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) throw Unfit();
    return t;
}

// Address of a contiguous tensor of `type` on `device` with `count` elements
// (negative: any number).
void *address(const at::Tensor &t, ScalarType type, int device, int64_t count) {
    if (t.scalar_type() != type || t.get_device() != device || !t.is_contiguous() || (count >= 0 && t.numel() != count))
        throw Unfit();
    return t.data_ptr();
}
// The same of an object that may be None (null).
template <typename T>
T *address(PyObject *o, ScalarType type, int device, int64_t count) {
    return o == Py_None ? nullptr : static_cast<T *>(address(tensor(o), type, device, count));
}

// bfloat16 [tokens, heads, D]: heads and elements contiguous, tokens any stride.
struct Rows {
    const uint16_t *p = nullptr;
    int64_t stride = 0, T = 0, H = 0, D = 0;
    Rows() = default;
    Rows(PyObject *o, int device) {
        const at::Tensor &t = tensor(o);
        if (t.scalar_type() != ScalarType::BFloat16 || t.get_device() != device || t.dim() != 3) throw Unfit();
        T = t.size(0), H = t.size(1), D = t.size(2);
        if ((t.stride(2) != 1 && D > 1) || (t.stride(1) != D && H > 1)) throw Unfit();
        p = static_cast<const uint16_t *>(t.data_ptr());
        stride = T > 1 ? t.stride(0) : H * D;
    }
};

int64_t integer(PyObject *o) {
    if (!PyLong_CheckExact(o)) throw Unfit();
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unfit();
    }
    return v;
}
int small(int64_t v) {
    if (v < INT32_MIN || v > INT32_MAX) throw Unfit();
    return static_cast<int>(v);
}
float real(PyObject *o) {
    if (!PyFloat_Check(o)) throw Unfit();
    return static_cast<float>(PyFloat_AS_DOUBLE(o));
}

int truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        throw Unfit();
    }
    return v;
}

// The stream to launch on, with its device current while this lives.
struct Launch {
    std::optional<c10::cuda::CUDAGuard> guard;
    void *stream;
    Launch(int device, PyObject *o) {
        if (c10::cuda::current_device() != device) guard.emplace(static_cast<c10::DeviceIndex>(device));
        if (o == Py_None) stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
        else stream = reinterpret_cast<void *>(integer(o));
    }
};

struct Cache {
    uint8_t *p;
    int device, bs;
    int64_t blocks, Hkv, D;
    explicit Cache(PyObject *o) {
        const at::Tensor &t = tensor(o);
        if (t.dim() != 4 || t.size(3) % 18 != 0) throw Unfit();
        device = t.get_device();
        p = static_cast<uint8_t *>(address(t, ScalarType::Byte, device, -1));
        blocks = t.size(0), Hkv = t.size(1), bs = small(t.size(2) * 16), D = t.size(3) / 18;
    }
};

// A cos_sin table (or None) and the positions that go with it.
struct Table {
    const float *p = nullptr;
    const int32_t *positions = nullptr;
    int64_t rows = 0, rot = 0;
    Table(PyObject *o, PyObject *pos, int device, int64_t T) {
        if (o == Py_None) return;
        const at::Tensor &t = tensor(o);
        if (t.dim() != 2 || pos == Py_None) throw Unfit();
        p = static_cast<const float *>(address(t, ScalarType::Float, device, -1));
        rows = t.size(0), rot = t.size(1);
        positions = address<const int32_t>(pos, ScalarType::Int, device, T);
    }
};

// ctx_lens, new_lens, block_table, free_blocks, block_size, seq_lens, cu_new, positions, slots, taken, stream
int plan(PyObject *const *a) {
    const at::Tensor &ctx = tensor(a[0]), &table = tensor(a[2]), &free = tensor(a[3]), &pos = tensor(a[7]);
    const int device = ctx.get_device();
    const int64_t B = ctx.numel(), T = pos.numel();
    if (table.dim() != 2 || table.size(0) != B) throw Unfit();
    const ScalarType I = ScalarType::Int;
    const int32_t *pc = static_cast<int32_t *>(address(ctx, I, device, B)), *pn = address<int32_t>(a[1], I, device, B);
    int32_t *pt = static_cast<int32_t *>(address(table, I, device, -1));
    const int32_t *pf = static_cast<int32_t *>(address(free, I, device, -1));
    int32_t *ps = address<int32_t>(a[5], I, device, B), *pu = address<int32_t>(a[6], I, device, B + 1);
    int32_t *pp = static_cast<int32_t *>(address(pos, I, device, T)), *pk = address<int32_t>(a[9], I, device, 1);
    int64_t *pl = address<int64_t>(a[8], ScalarType::Long, device, T);
    const int bs = small(integer(a[4]));
    const Launch l(device, a[10]);
    return p_plan(pc, pn, small(B), pt, table.size(1), pf, free.numel(), bs, T, ps, pu, pp, pl, pk, l.stream);
}

// q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out, eps, weight_offset, interleaved, stream
int rope(PyObject *const *a) {
    const int device = tensor(a[0]).get_device();
    const Rows q(a[0], device), k(a[1], device);
    if (k.T != q.T || k.D != q.D) throw Unfit();
    const ScalarType H = ScalarType::BFloat16;
    const uint16_t *wq = address<uint16_t>(a[2], H, device, q.D), *wk = address<uint16_t>(a[3], H, device, q.D);
    const Table t(a[4], a[5], device, q.T);
    uint16_t *oq = address<uint16_t>(a[6], H, device, q.T * q.H * q.D), *ok = address<uint16_t>(a[7], H, device, k.T * k.H * k.D);
    const float eps = real(a[8]), offset = real(a[9]);
    const int interleaved = truth(a[10]);
    const Launch l(device, a[11]);
    return p_rope(q.p, q.stride, k.p, k.stride, wq, wk, t.p, t.rows, small(t.rot), t.positions, oq, ok, q.T, small(q.H),
                  small(k.H), small(q.D), eps, offset, interleaved, l.stream);
}

// k, v, cache, slots, q, q_weight, k_weight, cos_sin, positions, q_out, eps, weight_offset, interleaved, stream
int append(PyObject *const *a) {
    const Cache c(a[2]);
    const Rows k(a[0], c.device), v(a[1], c.device);
    if (k.H != c.Hkv || k.D != c.D || v.T != k.T || v.H != c.Hkv || v.D != c.D) throw Unfit();
    const ScalarType H = ScalarType::BFloat16;
    const int64_t *slots = address<int64_t>(a[3], ScalarType::Long, c.device, k.T);
    Rows q;
    uint16_t *out = nullptr;
    if (a[4] != Py_None) {
        q = Rows(a[4], c.device);
        if (q.T != k.T || q.D != c.D) throw Unfit();
        out = address<uint16_t>(a[9], H, c.device, q.T * q.H * q.D);
    }
    const uint16_t *wq = address<uint16_t>(a[5], H, c.device, c.D), *wk = address<uint16_t>(a[6], H, c.device, c.D);
    const Table t(a[7], a[8], c.device, k.T);
    const float eps = real(a[10]), offset = real(a[11]);
    const int interleaved = truth(a[12]);
    const Launch l(c.device, a[13]);
    return p_append(q.p, q.stride, k.p, k.stride, v.p, v.stride, wq, wk, t.p, t.rows, small(t.rot), t.positions, slots, out,
                    c.p, c.blocks, c.bs, k.T, small(q.H), small(c.Hkv), small(c.D), eps, offset, interleaved, l.stream);
}

// cache, slots, k, v, stream
int gather(PyObject *const *a) {
    const Cache c(a[0]);
    const at::Tensor &s = tensor(a[1]);
    const int64_t T = s.numel(), n = T * c.Hkv * c.D;
    const int64_t *slots = static_cast<int64_t *>(address(s, ScalarType::Long, c.device, T));
    uint16_t *k = address<uint16_t>(a[2], ScalarType::BFloat16, c.device, n),
             *v = address<uint16_t>(a[3], ScalarType::BFloat16, c.device, n);
    const Launch l(c.device, a[4]);
    return p_gather(c.p, c.blocks, c.bs, slots, k, v, T, small(c.Hkv), small(c.D), l.stream);
}

// q, cache, block_table, seq_lens, cu_new, scratch, out, scale, window, sinks, max_new, stream
int attention(PyObject *const *a) {
    const Cache c(a[1]);
    const Rows q(a[0], c.device);
    const at::Tensor &table = tensor(a[2]), &lens = tensor(a[3]), &scratch = tensor(a[5]);
    const int64_t B = lens.numel();
    if (q.D != c.D || table.dim() != 2 || table.size(0) != B) throw Unfit();
    const ScalarType I = ScalarType::Int;
    const int32_t *pt = static_cast<int32_t *>(address(table, I, c.device, -1));
    const int32_t *pl = static_cast<int32_t *>(address(lens, I, c.device, B)), *pu = address<int32_t>(a[4], I, c.device, B + 1);
    void *ps = address(scratch, ScalarType::Byte, c.device, -1);
    uint16_t *out = address<uint16_t>(a[6], ScalarType::BFloat16, c.device, q.T * q.H * q.D);
    const float scale = real(a[7]);
    const int64_t window = integer(a[8]), sinks = integer(a[9]), most = integer(a[10]);
    const Launch l(c.device, a[11]);
    return p_attention(q.p, q.stride, c.p, c.blocks, c.bs, pt, table.size(1), pl, pu, small(B), out, q.T, small(q.H),
                       small(c.Hkv), small(c.D), scale, window, sinks, most, ps, scratch.numel(), l.stream);
}

// cache, slots, bounds, stream
int bounds(PyObject *const *a) {
    const Cache c(a[0]);
    const at::Tensor &s = tensor(a[1]);
    const int64_t T = s.numel();
    const int64_t *slots = static_cast<int64_t *>(address(s, ScalarType::Long, c.device, T));
    uint8_t *out = static_cast<uint8_t *>(address(tensor(a[2]), ScalarType::Byte, c.device, c.blocks * c.Hkv * (2 * c.D + 16)));
    const Launch l(c.device, a[3]);
    return p_bounds(c.p, c.blocks, c.bs, slots, out, T, small(c.Hkv), small(c.D), l.stream);
}

// q, bounds, block_table, seq_lens, cu_new, block_size, top, first, recent, tables, lens, stream
int select(PyObject *const *a) {
    const at::Tensor &x = tensor(a[1]);
    const int device = x.get_device();
    const Rows q(a[0], device);
    if (x.dim() != 3 || x.size(2) != 2 * q.D + 16) throw Unfit();
    const uint8_t *px = static_cast<uint8_t *>(address(x, ScalarType::Byte, device, -1));
    const at::Tensor &table = tensor(a[2]), &lens = tensor(a[3]);
    const int64_t B = lens.numel();
    if (table.dim() != 2 || table.size(0) != B) throw Unfit();
    const ScalarType I = ScalarType::Int;
    const int32_t *pt = static_cast<int32_t *>(address(table, I, device, -1));
    const int32_t *pl = static_cast<int32_t *>(address(lens, I, device, B)), *pu = address<int32_t>(a[4], I, device, B + 1);
    const int bs = small(integer(a[5])), top = small(integer(a[6])), first = small(integer(a[7])), recent = small(integer(a[8]));
    int32_t *to = address<int32_t>(a[9], I, device, q.T * x.size(1) * top), *n = address<int32_t>(a[10], I, device, q.T);
    const Launch l(device, a[11]);
    return p_select(q.p, q.stride, px, x.size(0), bs, pt, table.size(1), pl, pu, small(B), q.T, small(q.H), small(x.size(1)),
                    small(q.D), top, first, recent, to, n, l.stream);
}

// q, cache, tables, lens, scratch, out, scale, stream
int sparse(PyObject *const *a) {
    const Cache c(a[1]);
    const Rows q(a[0], c.device);
    const at::Tensor &tables = tensor(a[2]), &scratch = tensor(a[4]);
    if (q.D != c.D || tables.dim() != 3 || tables.size(0) != q.T || tables.size(1) != c.Hkv) throw Unfit();
    const ScalarType I = ScalarType::Int;
    const int32_t *pt = static_cast<int32_t *>(address(tables, I, c.device, -1)), *pl = address<int32_t>(a[3], I, c.device, q.T);
    void *ps = address(scratch, ScalarType::Byte, c.device, -1);
    uint16_t *out = address<uint16_t>(a[5], ScalarType::BFloat16, c.device, q.T * q.H * q.D);
    const float scale = real(a[6]);
    const Launch l(c.device, a[7]);
    return p_sparse(q.p, q.stride, c.p, c.blocks, c.bs, pt, tables.size(2), pl, out, q.T, small(q.H), small(c.Hkv), small(c.D),
                    scale, ps, scratch.numel(), l.stream);
}

// q, cache, block_table, seq_lens, cu_new, prefix_lens, cu_groups, scratch, out, scale, max_new, max_group, stream
int prefix(PyObject *const *a) {
    const Cache c(a[1]);
    const Rows q(a[0], c.device);
    const at::Tensor &table = tensor(a[2]), &lens = tensor(a[3]), &prefixes = tensor(a[5]), &scratch = tensor(a[7]);
    const int64_t B = lens.numel(), N = prefixes.numel();
    if (q.D != c.D || table.dim() != 2 || table.size(0) != B) throw Unfit();
    const ScalarType I = ScalarType::Int;
    const int32_t *pt = static_cast<int32_t *>(address(table, I, c.device, -1));
    const int32_t *pl = static_cast<int32_t *>(address(lens, I, c.device, B)), *pu = address<int32_t>(a[4], I, c.device, B + 1);
    const int32_t *pp = static_cast<int32_t *>(address(prefixes, I, c.device, N)), *pg = address<int32_t>(a[6], I, c.device, N + 1);
    void *ps = address(scratch, ScalarType::Byte, c.device, -1);
    uint16_t *out = address<uint16_t>(a[8], ScalarType::BFloat16, c.device, q.T * q.H * q.D);
    const float scale = real(a[9]);
    const int64_t most = integer(a[10]), widest = integer(a[11]);
    const Launch l(c.device, a[12]);
    return p_prefix(q.p, q.stride, c.p, c.blocks, c.bs, pt, table.size(1), pl, pu, small(B), pp, pg, small(N), out, q.T,
                    small(q.H), small(c.Hkv), small(c.D), scale, most, widest, ps, scratch.numel(), l.stream);
}

// logits, u, temperature, top_k, top_p, min_p, out, stream
int sample(PyObject *const *a) {
    const at::Tensor &x = tensor(a[0]);
    const int device = x.get_device();
    const bool f32 = x.scalar_type() == ScalarType::Float;
    if (x.dim() != 2 || (!f32 && x.scalar_type() != ScalarType::BFloat16)) throw Unfit();
    const int64_t R = x.size(0), V = x.size(1);
    if (x.stride(1) != 1 && V > 1) throw Unfit();
    const ScalarType F = ScalarType::Float, I = ScalarType::Int;
    const float *u = address<float>(a[1], F, device, R), *T = address<float>(a[2], F, device, R);
    const int32_t *k = address<int32_t>(a[3], I, device, R);
    const float *p = address<float>(a[4], F, device, R), *m = address<float>(a[5], F, device, R);
    int32_t *out = address<int32_t>(a[6], I, device, R);
    const Launch l(device, a[7]);
    return p_sample(x.data_ptr(), f32 ? W4_OUT_F32 : W4_OUT_BF16, R > 1 ? x.stride(0) : V, R, V, u, T, k, p, m, out, l.stream);
}

template <int (*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, nargs);
        return nullptr;
    }
    if (!p_sample) Py_RETURN_NONE;  // not bound to the library
    try {
        return PyLong_FromLong(F(args));
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// bind(path): finds the entry points in the loaded library.
PyObject *bind(PyObject *, PyObject *path) {
    const char *s = PyUnicode_AsUTF8(path);
    if (!s) return nullptr;
    void *h = dlopen(s, RTLD_NOW);
    if (!h) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    p_plan = reinterpret_cast<decltype(p_plan)>(dlsym(h, "kv4_plan"));
    p_rope = reinterpret_cast<decltype(p_rope)>(dlsym(h, "w4a16_qk_norm_rope"));
    p_append = reinterpret_cast<decltype(p_append)>(dlsym(h, "kv4_append"));
    p_gather = reinterpret_cast<decltype(p_gather)>(dlsym(h, "kv4_gather"));
    p_attention = reinterpret_cast<decltype(p_attention)>(dlsym(h, "kv4_attention"));
    p_bounds = reinterpret_cast<decltype(p_bounds)>(dlsym(h, "kv4_bounds"));
    p_select = reinterpret_cast<decltype(p_select)>(dlsym(h, "kv4_select"));
    p_sparse = reinterpret_cast<decltype(p_sparse)>(dlsym(h, "kv4_sparse_attention"));
    p_prefix = reinterpret_cast<decltype(p_prefix)>(dlsym(h, "kv4_prefix_attention"));
    p_sample = reinterpret_cast<decltype(p_sample)>(dlsym(h, "w4a16_sample"));
    if (!p_plan || !p_rope || !p_append || !p_gather || !p_attention || !p_bounds || !p_select || !p_sparse || !p_prefix ||
        !p_sample) {
        p_sample = nullptr;
        PyErr_SetString(PyExc_RuntimeError, "the library lacks an entry point");
        return nullptr;
    }
    Py_RETURN_NONE;
}

template <int (*F)(PyObject *const *), int N>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         method<plan, 11>("kv4_plan"),
                         method<rope, 12>("w4a16_qk_norm_rope"),
                         method<append, 14>("kv4_append"),
                         method<gather, 5>("kv4_gather"),
                         method<attention, 12>("kv4_attention"),
                         method<bounds, 4>("kv4_bounds"),
                         method<select, 12>("kv4_select"),
                         method<sparse, 8>("kv4_sparse_attention"),
                         method<prefix, 13>("kv4_prefix_attention"),
                         method<sample, 8>("w4a16_sample"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
