// torch_marshal.cpp -- the short way from torch tensors to the calls of
// include/pkv_ops.h: a CPython module that reads the tensors' addresses, sizes and
// types in C++ (a few hundred ns for a call's dozen tensors, where attribute
// lookups from Python take 8 to 11 us). It only accepts what needs no explanation:
// anything unexpected returns None, and the Python face, which checks the same
// conditions one by one, raises the error (or makes the call itself).
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pkv_ops.h"

namespace {

// Addresses in libpkv.so (loaded by the package, handed over by bind()).
decltype(&pkv_rope_kv_append) g_rope;
decltype(&pkv_rope_kv_append_fp8_block) g_rope_fp8;
decltype(&pkv_paged_decode_attention_scored) g_attend;
decltype(&pkv_workspace_size_scored) g_size;

// One argument as a CUDA tensor of device `dev`; ok() of what is asked is kept.
struct Arg {
    const at::Tensor *t = nullptr;

    Arg(PyObject *o, int dev, at::ScalarType type, int dims, bool *ok, bool dense = true)
    {
        if (!THPVariable_Check(o)) {
            *ok = false;
            return;
        }
        t = &THPVariable_Unpack(o);
        *ok = *ok && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type &&
              t->dim() == dims && (!dense || t->is_contiguous());
    }
    int64_t size(int i) const { return t->size(i); }
    void *ptr() const { return t->data_ptr(); }
    // [n, heads, D] with contiguous rows: the elements between two rows, -1 if not
    int64_t row_stride() const
    {
        const int64_t n = size(0), h = size(1), d = size(2);
        if ((d > 1 && t->stride(2) != 1) || (h > 1 && t->stride(1) != d))
            return -1;
        return n > 1 ? t->stride(0) : h * d;
    }
};

bool same(const Arg &a, int64_t x, int64_t y, int64_t z)
{
    return a.size(0) == x && a.size(1) == y && a.size(2) == z;
}

PyObject *status(pkv_status st) { return PyLong_FromLong(long(st)); }

constexpr auto kBf16 = at::ScalarType::BFloat16;
constexpr auto kByte = at::ScalarType::Byte;
constexpr auto kInt = at::ScalarType::Int;
constexpr auto kLong = at::ScalarType::Long;
constexpr auto kFloat = at::ScalarType::Float;

// rope(q, k_new, v_new, positions, turns, slot_mapping, k_cache, v_cache, k_scale,
//      v_scale, q_out, interleaved, rotary_scale, device, stream) -> status or None
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 15 || !g_rope)
        Py_RETURN_NONE;
    const int interleaved = PyObject_IsTrue(a[11]);
    const double scale = PyFloat_AsDouble(a[12]);
    const int dev = int(PyLong_AsLong(a[13]));
    void *stream = PyLong_AsVoidPtr(a[14]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    bool ok = true;
    const bool fp8 = a[8] != Py_None, with_q = a[0] != Py_None;
    const auto pool = fp8 ? kByte : kBf16;
    const Arg k(a[1], dev, kBf16, 3, &ok, false), v(a[2], dev, kBf16, 3, &ok, false),
        pos(a[3], dev, kLong, 1, &ok), turns(a[4], dev, kLong, 1, &ok),
        slots(a[5], dev, kLong, 1, &ok), kc(a[6], dev, pool, 4, &ok), vc(a[7], dev, pool, 4, &ok);
    if (!ok)
        Py_RETURN_NONE;
    const int64_t nb = kc.size(0), hkv = kc.size(2), d = kc.size(3), rows = slots.size(0);
    ok = kc.size(1) == 16 && vc.t->sizes() == kc.t->sizes() && same(k, rows, hkv, d) &&
         same(v, rows, hkv, d) && pos.size(0) == rows;
    const int64_t ks = k.row_stride(), vs = v.row_stride();
    int64_t hq = 0, qs = 0;
    void *q = nullptr, *out = nullptr;
    if (with_q) {
        const Arg qi(a[0], dev, kBf16, 3, &ok, false), qo(a[10], dev, kBf16, 3, &ok);
        if (!ok)
            Py_RETURN_NONE;
        hq = qi.size(1);
        qs = qi.row_stride();
        ok = same(qi, rows, hq, d) && qo.t->sizes() == qi.t->sizes();
        q = qi.ptr();
        out = qo.ptr();
    } else {
        ok = ok && a[10] == Py_None;
    }
    if (!ok || ks < 0 || vs < 0 || qs < 0 || hkv > INT32_MAX || hq > INT32_MAX || d > INT32_MAX ||
        turns.size(0) > INT32_MAX / 2)
        Py_RETURN_NONE;
    const auto *p = static_cast<const int64_t *>(pos.ptr());
    const auto *f = static_cast<const uint64_t *>(turns.ptr());
    const auto *s = static_cast<const int64_t *>(slots.ptr());
    const int32_t r = int32_t(2 * turns.size(0));
    if (!fp8)
        return status(g_rope(q, qs, k.ptr(), ks, v.ptr(), vs, p, f, s, rows, out, kc.ptr(),
                             vc.ptr(), nb, int32_t(hq), int32_t(hkv), int32_t(d), r, interleaved,
                             float(scale), stream));
    const Arg ksc(a[8], dev, kByte, 2, &ok), vsc(a[9], dev, kByte, 2, &ok);
    if (!ok || ksc.size(0) != nb || ksc.size(1) != hkv || vsc.t->sizes() != ksc.t->sizes())
        Py_RETURN_NONE;
    return status(g_rope_fp8(q, qs, k.ptr(), ks, v.ptr(), vs, p, f, s, rows, out, kc.ptr(),
                             vc.ptr(), static_cast<uint8_t *>(ksc.ptr()),
                             static_cast<uint8_t *>(vsc.ptr()), nb, int32_t(hq), int32_t(hkv),
                             int32_t(d), r, interleaved, float(scale), stream));
}

// attend(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
//        n_query_per_seq, scale, out, softcap, alibi_slopes, window, ws, device,
//        stream) -> status or None (also where ws is None or too small)
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 16 || !g_attend || a[13] == Py_None)
        Py_RETURN_NONE;
    const long nq = PyLong_AsLong(a[7]);
    const double scale = PyFloat_AsDouble(a[8]), cap = PyFloat_AsDouble(a[10]);
    const long window = PyLong_AsLong(a[12]);
    const int dev = int(PyLong_AsLong(a[14]));
    void *stream = PyLong_AsVoidPtr(a[15]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    bool ok = true;
    const bool fp8 = a[3] != Py_None;
    const auto pool = fp8 ? kByte : kBf16;
    const Arg q(a[0], dev, kBf16, 3, &ok), kc(a[1], dev, pool, 4, &ok), vc(a[2], dev, pool, 4, &ok),
        bt(a[5], dev, kInt, 2, &ok), cl(a[6], dev, kInt, 1, &ok), ws(a[13], dev, kByte, 1, &ok);
    if (!ok || !THPVariable_Check(a[9]))
        Py_RETURN_NONE;
    const auto out_type = THPVariable_Unpack(a[9]).scalar_type();
    const Arg out(a[9], dev, out_type, 3, &ok);
    const int64_t nb = kc.size(0), hkv = kc.size(2), d = kc.size(3), seqs = cl.size(0);
    const int64_t hq = q.size(1);
    ok = ok && (out_type == kBf16 || out_type == kFloat) && kc.size(1) == 16 &&
         vc.t->sizes() == kc.t->sizes() && same(q, seqs * nq, hq, d) &&
         out.t->sizes() == q.t->sizes() && bt.size(0) == seqs && seqs <= INT32_MAX &&
         bt.size(1) <= INT32_MAX && hq <= INT32_MAX && hkv <= INT32_MAX && d <= INT32_MAX &&
         nq <= INT32_MAX && nq >= INT32_MIN && window <= INT32_MAX && window >= INT32_MIN;
    const uint8_t *ks = nullptr, *vs = nullptr;
    if (ok && fp8) {
        const Arg s0(a[3], dev, kByte, 2, &ok), s1(a[4], dev, kByte, 2, &ok);
        ok = ok && s0.size(0) == nb && s0.size(1) == hkv && s1.t->sizes() == s0.t->sizes();
        if (ok) {
            ks = static_cast<const uint8_t *>(s0.ptr());
            vs = static_cast<const uint8_t *>(s1.ptr());
        }
    } else if (a[4] != Py_None) {
        ok = false;
    }
    const float *slopes = nullptr;
    if (ok && a[11] != Py_None) {
        const Arg sl(a[11], dev, kFloat, 1, &ok);
        ok = ok && sl.size(0) == hq;
        if (ok)
            slopes = static_cast<const float *>(sl.ptr());
    }
    if (!ok || ws.size(0) < int64_t(g_size(int32_t(seqs), int32_t(nq), int32_t(hq), int32_t(hkv),
                                           int32_t(d))))
        Py_RETURN_NONE;
    return status(g_attend(q.ptr(), kc.ptr(), vc.ptr(), nb, ks, vs,
                           static_cast<const int32_t *>(bt.ptr()), int32_t(bt.size(1)),
                           static_cast<const int32_t *>(cl.ptr()), int32_t(seqs), int32_t(nq),
                           int32_t(hq), int32_t(hkv), int32_t(d), float(scale), float(cap), slopes,
                           int32_t(window), out.ptr(), out_type == kFloat ? PKV_FP32 : PKV_BF16,
                           ws.ptr(), size_t(ws.size(0)), stream));
}

// bind(rope, rope_fp8_block, attention, workspace_size): addresses in libpkv.so
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
        return nullptr;
    }
    void *p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred())
            return nullptr;
    }
    g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
    g_rope_fp8 = reinterpret_cast<decltype(g_rope_fp8)>(p[1]);
    g_attend = reinterpret_cast<decltype(g_attend)>(p[2]);
    g_size = reinterpret_cast<decltype(g_size)>(p[3]);
    Py_RETURN_NONE;
}

// No C++ exception (torch throws on odd tensors) leaves a call.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    try {
        return F(self, a, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)),
            METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<rope>("rope"), method<attend>("attend"), method<bind>("bind"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_marshal", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_marshal() { return PyModule_Create(&g_module); }
