// The calls that a serving step makes once a layer or once a step, with their
// arguments checked and taken apart here instead of in Python: the checks of a call's
// ten to fourteen tensors and its foreign-function call took longer than most of
// these kernels run (fa_rope_append for 64 tokens: 13.5 us a call, of which the
// kernel 2.5).
//
// Each function returns the call's fa_status, or kExplain where an argument is not
// exactly what the call takes (or not of the exact Python type); the Python wrapper
// then goes its own way, which finds the words for it.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

namespace {

constexpr long kExplain = 1;          // no fa_status
struct Explain {};

void need(bool ok) {
    if (!ok) throw Explain();
}

const at::Tensor& tensor(PyObject* o) {
    need(THPVariable_Check(o));
    const at::Tensor& t = THPVariable_Unpack(o);
    need(t.is_cuda());
    return t;
}

// A call's current device: every tensor has to be on it.
struct Device {
    int index;
    explicit Device(const at::Tensor& any) : index(any.get_device()) {
        need(index == (int)c10::cuda::current_device());
    }
    void here(const at::Tensor& t) const { need(t.get_device() == index); }
    // a contiguous tensor's memory
    void* whole(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape) const {
        need(t.scalar_type() == type && t.sizes() == shape && t.is_contiguous());
        here(t);
        return t.data_ptr();
    }
    void* whole(PyObject* o, at::ScalarType type, at::IntArrayRef shape) const {
        return whole(tensor(o), type, shape);
    }
    // rows of any strides, which go to `strides` (of B, H and N)
    void* rows(PyObject* o, at::IntArrayRef shape, long long* strides) const {
        const at::Tensor& t = tensor(o);
        need(t.scalar_type() == at::kBFloat16 && t.sizes() == shape && t.stride(3) == 1);
        here(t);
        for (int i = 0; i < 3; ++i) strides[i] = t.stride(i);
        return t.data_ptr();
    }
};

int whole_number(PyObject* o) {
    need(PyLong_Check(o));
    int overflow;
    const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
    need(!overflow && x >= INT32_MIN && x <= INT32_MAX);
    return (int)x;
}

int size_of(int64_t n) {
    need(n <= INT32_MAX);
    return (int)n;
}

bool truth(PyObject* o) {
    need(PyBool_Check(o));
    return o == Py_True;
}

float number(PyObject* o) {
    need(PyFloat_Check(o));
    return (float)PyFloat_AS_DOUBLE(o);
}

// None: the current stream; else a stream's handle.
fa_stream_t stream_of(PyObject* o, const Device& dev) {
    if (o == Py_None)
        return (fa_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream();
    need(PyLong_Check(o));
    return (fa_stream_t)PyLong_AsVoidPtr(o);
}

template <typename F>
PyObject* answer(Py_ssize_t n, Py_ssize_t expected, F&& f) {
    long st = kExplain;
    if (n == expected) {
        try {
            st = f();
        } catch (...) {
            st = kExplain;
        }
        if (PyErr_Occurred()) PyErr_Clear();
    }
    return PyLong_FromLong(st);
}

// The call itself, without the interpreter's lock.
template <typename F>
long launched(F&& f) {
    fa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return (long)st;
}

PyObject* kv_reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return answer(n, 12, [&]() -> long {
        const at::Tensor &table = tensor(a[0]), &free_pages = tensor(a[2]);
        const Device dev(table);
        need(table.dim() == 2 && free_pages.dim() == 1);
        const int64_t B = table.size(0), P = free_pages.size(0);
        const auto i32 = at::kInt;
        int* const t = (int*)dev.whole(table, i32, table.sizes());
        int* const f = (int*)dev.whole(free_pages, i32, {P});
        int* p[6];
        const int at[6] = {1, 3, 4, 5, 6, 7};
        for (int i = 0; i < 6; ++i)
            p[i] = (int*)dev.whole(a[at[i]], i32, {i == 1 ? 1 : i == 5 ? B + 1 : B});
        int* positions = nullptr;
        long long* slots = nullptr;
        int N = 0, total = 0;
        if (a[8] != Py_None || a[9] != Py_None) {
            const at::Tensor& s = tensor(a[9]);
            need((s.dim() == 2 && s.size(0) == B && s.size(1) >= 1) || s.dim() == 1);
            positions = (int*)dev.whole(a[8], i32, s.sizes());
            slots = (long long*)dev.whole(s, at::kLong, s.sizes());
            (s.dim() == 2 ? N : total) = size_of(s.size(s.dim() - 1));
        }
        const int ps = whole_number(a[10]);
        const fa_stream_t st = stream_of(a[11], dev);
        const int b = size_of(B), np = size_of(P), mp = size_of(table.size(1));
        return launched([&] {
            return fa_kv_reserve(t, p[0], f, p[1], p[2], p[3], p[4], p[5], positions, slots, b, N,
                                 total, np, ps, mp, st);
        });
    });
}

PyObject* kv_release(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return answer(n, 8, [&]() -> long {
        const at::Tensor &table = tensor(a[0]), &free_pages = tensor(a[2]);
        const Device dev(table);
        need(table.dim() == 2 && free_pages.dim() == 1);
        const int64_t B = table.size(0), P = free_pages.size(0);
        const auto i32 = at::kInt;
        int* const t = (int*)dev.whole(table, i32, table.sizes());
        int* const lens = (int*)dev.whole(a[1], i32, {B});
        int* const f = (int*)dev.whole(free_pages, i32, {P});
        int* const n_free = (int*)dev.whole(a[3], i32, {1});
        const int* const keep = (int*)dev.whole(a[4], i32, {B});
        const int* const pinned = a[5] == Py_None ? nullptr : (int*)dev.whole(a[5], i32, {B});
        const int ps = whole_number(a[6]);
        const fa_stream_t st = stream_of(a[7], dev);
        const int b = size_of(B), np = size_of(P), mp = size_of(table.size(1));
        return launched(
            [&] { return fa_kv_release(t, lens, f, n_free, keep, pinned, b, np, ps, mp, st); });
    });
}

// Sizes, positions and frequencies of a rotary call.
struct Rotary {
    const at::Tensor& q;
    Device dev;
    int B, H, N, d, rot;
    const int* positions;
    const unsigned long long* freqs;
    Rotary(PyObject* q_, PyObject* pos, PyObject* fr) : q(tensor(q_)), dev(q) {
        need(q.dim() == 4);
        B = size_of(q.size(0));
        H = size_of(q.size(1));
        N = size_of(q.size(2));
        d = size_of(q.size(3));
        positions = (const int*)dev.whole(pos, at::kInt, {B, N});
        const at::Tensor& f = tensor(fr);
        need(f.dim() == 1);
        freqs = (const unsigned long long*)dev.whole(f, at::kLong, f.sizes());
        rot = size_of(2 * f.size(0));
    }
};

PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return answer(n, 10, [&]() -> long {
        const Rotary r(a[0], a[4], a[5]);
        long long s[12] = {};
        const void* q = r.dev.rows(a[0], r.q.sizes(), s);
        void* qo = r.dev.rows(a[2], r.q.sizes(), s + 6);
        const void* k = nullptr;
        void* ko = nullptr;
        int Hkv = 0;
        if (a[1] != Py_None || a[3] != Py_None) {
            const at::Tensor& t = tensor(a[1]);
            need(t.dim() == 4 && t.size(0) == r.B && t.size(2) == r.N && t.size(3) == r.d);
            Hkv = size_of(t.size(1));
            k = r.dev.rows(a[1], t.sizes(), s + 3);
            ko = r.dev.rows(a[3], t.sizes(), s + 9);
        }
        const bool inter = truth(a[6]), inverse = truth(a[7]);
        const float amplitude = number(a[8]);
        const fa_stream_t st = stream_of(a[9], r.dev);
        return launched([&] {
            return fa_rope(q, k, qo, ko, r.positions, r.freqs, s, r.B, r.H, Hkv, r.N, r.d, r.rot,
                           inter, inverse, amplitude, st);
        });
    });
}

PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return answer(n, 13, [&]() -> long {
        const Rotary r(a[0], a[6], a[8]);
        const at::Tensor &pages = tensor(a[4]), &values = tensor(a[5]);
        need(pages.dim() == 4 && pages.size(3) == r.d);
        const int64_t P = pages.size(0), Hkv = pages.size(1), ps = pages.size(2);
        const bool f8 = a[11] != Py_None;
        const auto kind = f8 ? at::kFloat8_e4m3fn : at::kBFloat16;
        long long s[12];
        const void* q = r.dev.rows(a[0], r.q.sizes(), s);
        const void* k = r.dev.rows(a[1], {r.B, Hkv, r.N, r.d}, s + 3);
        const void* v = r.dev.rows(a[2], {r.B, Hkv, r.N, r.d}, s + 6);
        void* qo = r.dev.rows(a[3], r.q.sizes(), s + 9);
        void* kp = r.dev.whole(pages, kind, pages.sizes());
        void* vp = r.dev.whole(values, kind, pages.sizes());
        float* scales = f8 ? (float*)r.dev.whole(a[11], at::kFloat, {P, Hkv, 2, ps}) : nullptr;
        const long long* slots = (const long long*)r.dev.whole(a[7], at::kLong, {r.B, r.N});
        const bool inter = truth(a[9]);
        const float amplitude = number(a[10]);
        const fa_stream_t st = stream_of(a[12], r.dev);
        const int np = size_of(P), hk = size_of(Hkv), p = size_of(ps);
        return launched([&] {
            return fa_rope_append(q, k, v, qo, kp, vp, scales, r.positions, slots, r.freqs, s, r.B,
                                  r.H, hk, r.N, np, p, r.d, r.rot, inter, amplitude, st);
        });
    });
}

PyObject* cross_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return answer(n, 10, [&]() -> long {
        const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]), &ws = tensor(a[5]);
        const Device dev(q);
        need(q.dim() == 4 && k.dim() == 4 && k.size(0) == q.size(0) && k.size(3) == q.size(3));
        const auto bf = at::kBFloat16;
        const void* qp = dev.whole(q, bf, q.sizes());
        const void* kp = dev.whole(k, bf, k.sizes());
        const void* vp = dev.whole(a[2], bf, k.sizes());
        void* o = dev.whole(a[3], bf, q.sizes());
        float* lse = (float*)dev.whole(a[4], at::kFloat, q.sizes().slice(0, 3));
        dev.here(ws);
        need(ws.is_contiguous());
        const int* lens = a[8] == Py_None ? nullptr : (int*)dev.whole(a[8], at::kInt, {q.size(0)});
        const bool causal = truth(a[6]);
        const float scale = number(a[7]);
        const fa_stream_t st = stream_of(a[9], dev);
        const int B = size_of(q.size(0)), H = size_of(q.size(1)), Hkv = size_of(k.size(1)),
                  Nq = size_of(q.size(2)), Nk = size_of(k.size(2)), d = size_of(q.size(3));
        return launched([&] {
            return fa_fwd_cross_decode(qp, kp, vp, o, lse, lens, ws.data_ptr(), ws.nbytes(), B, H,
                                       Hkv, Nq, Nk, d, causal, scale, st);
        });
    });
}

// Queries and keys of two lengths, padded or (3-D, with cu_q and cu_k) packed: the tensors
// that all four calls have.
struct Cross {
    const at::Tensor &q, &k, &ws;
    Device dev;
    bool packed;
    int B, H, Hkv, Nq, Nk, d, total_q = 0, total_k = 0;
    const int *cu_q = nullptr, *cu_k = nullptr, *lens = nullptr;
    // at: the place of cu_q, cu_k, max_q and max_k (packed), of kv_lens (padded)
    Cross(PyObject* const* a, int workspace, int at, bool packed_)
        : q(tensor(a[0])), k(tensor(a[1])), ws(tensor(a[workspace])), dev(q), packed(packed_) {
        const int n = packed ? 3 : 4;
        need(q.dim() == n && k.dim() == n && k.size(n - 1) == q.size(n - 1));
        dev.here(ws);
        need(ws.is_contiguous());
        d = size_of(q.size(n - 1));
        H = size_of(q.size(n - 3));
        Hkv = size_of(k.size(n - 3));
        Nq = size_of(q.size(n - 2));
        Nk = size_of(k.size(n - 2));
        if (packed) {
            total_q = Nq;
            total_k = Nk;
            const at::Tensor &cq = tensor(a[at]), &ck = tensor(a[at + 1]);
            need(cq.dim() == 1 && cq.size(0) >= 1);
            cu_q = (const int*)dev.whole(cq, at::kInt, cq.sizes());
            cu_k = (const int*)dev.whole(ck, at::kInt, cq.sizes());
            B = size_of(cq.size(0) - 1);
            Nq = whole_number(a[at + 2]);
            Nk = whole_number(a[at + 3]);
        } else {
            need(k.size(0) == q.size(0));
            B = size_of(q.size(0));
            if (a[at] != Py_None) lens = (const int*)dev.whole(a[at], at::kInt, {q.size(0)});
        }
    }
    void* like_q(PyObject* o) const { return dev.whole(o, at::kBFloat16, q.sizes()); }
    void* like_k(PyObject* o) const { return dev.whole(o, at::kBFloat16, k.sizes()); }
    float* rows(PyObject* o) const {
        return (float*)dev.whole(o, at::kFloat, q.sizes().slice(0, q.dim() - 1));
    }
};

// (q, k, v, o, lse, workspace, causal, scale, kv_lens | cu_q, cu_k, max_q, max_k, stream)
PyObject* forward(PyObject* const* a, Py_ssize_t n, bool packed) {
    return answer(n, packed ? 13 : 10, [&]() -> long {
        const Cross c(a, 5, 8, packed);
        const void *q = c.like_q(a[0]), *k = c.like_k(a[1]), *v = c.like_k(a[2]);
        void* o = c.like_q(a[3]);
        float* lse = c.rows(a[4]);
        const bool causal = truth(a[6]);
        const float scale = number(a[7]);
        const fa_stream_t st = stream_of(a[n - 1], c.dev);
        void* const ws = c.ws.data_ptr();
        const size_t bytes = c.ws.nbytes();
        return launched([&] {
            return packed ? fa_fwd_cross_varlen(q, k, v, o, lse, c.cu_q, c.cu_k, ws, bytes, c.B,
                                                c.Nq, c.Nk, c.total_q, c.total_k, c.H, c.Hkv, c.d,
                                                causal, scale, st)
                          : fa_fwd_cross(q, k, v, o, lse, c.lens, ws, bytes, c.B, c.H, c.Hkv, c.Nq,
                                         c.Nk, c.d, causal, scale, st);
        });
    });
}

// (q, k, v, o, dout, lse, dq, dk, dv, workspace, causal, scale, as above)
PyObject* backward(PyObject* const* a, Py_ssize_t n, bool packed) {
    return answer(n, packed ? 17 : 14, [&]() -> long {
        const Cross c(a, 9, 12, packed);
        const void *q = c.like_q(a[0]), *k = c.like_k(a[1]), *v = c.like_k(a[2]);
        const void *o = c.like_q(a[3]), *dout = c.like_q(a[4]);
        const float* lse = c.rows(a[5]);
        void *dq = c.like_q(a[6]), *dk = c.like_k(a[7]), *dv = c.like_k(a[8]);
        const bool causal = truth(a[10]);
        const float scale = number(a[11]);
        const fa_stream_t st = stream_of(a[n - 1], c.dev);
        void* const ws = c.ws.data_ptr();
        const size_t bytes = c.ws.nbytes();
        return launched([&] {
            return packed ? fa_bwd_cross_varlen(q, k, v, o, dout, lse, dq, dk, dv, c.cu_q, c.cu_k,
                                                ws, bytes, c.B, c.Nq, c.Nk, c.total_q, c.total_k,
                                                c.H, c.Hkv, c.d, causal, scale, st)
                          : fa_bwd_cross(q, k, v, o, dout, lse, dq, dk, dv, c.lens, ws, bytes, c.B,
                                         c.H, c.Hkv, c.Nq, c.Nk, c.d, causal, scale, st);
        });
    });
}

PyObject* cross_forward(PyObject*, PyObject* const* a, Py_ssize_t n) { return forward(a, n, false); }
PyObject* cross_forward_varlen(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return forward(a, n, true);
}
PyObject* cross_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return backward(a, n, false);
}
PyObject* cross_backward_varlen(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return backward(a, n, true);
}

PyMethodDef methods[] = {
    {"kv_reserve", (PyCFunction)(void (*)(void))kv_reserve, METH_FASTCALL, nullptr},
    {"kv_release", (PyCFunction)(void (*)(void))kv_release, METH_FASTCALL, nullptr},
    {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, nullptr},
    {"rope_append", (PyCFunction)(void (*)(void))rope_append, METH_FASTCALL, nullptr},
    {"cross_decode", (PyCFunction)(void (*)(void))cross_decode, METH_FASTCALL, nullptr},
    {"cross_forward", (PyCFunction)(void (*)(void))cross_forward, METH_FASTCALL,
     nullptr},
    {"cross_forward_varlen", (PyCFunction)(void (*)(void))cross_forward_varlen, METH_FASTCALL,
     nullptr},
    {"cross_backward", (PyCFunction)(void (*)(void))cross_backward, METH_FASTCALL,
     nullptr},
    {"cross_backward_varlen", (PyCFunction)(void (*)(void))cross_backward_varlen, METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "fa_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa_binding() { return PyModule_Create(&module); }
