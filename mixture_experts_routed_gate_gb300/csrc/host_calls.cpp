// host_calls.cpp -- the binding's shortest calls, as a Python extension.
//
// A decode step's 8-bit calls are a few microseconds on the GPU and 15 to 28 in
// Python (checks, new tensors, ctypes).  Each function here makes one call of an
// entry point in the case that a program's inner loop makes: every tensor a
// contiguous CUDA tensor of the current device, of the right type and shape, results
// made new.  In every other case, wrong arguments among them, it makes no call and
// returns None, and the binding's Python code goes on: it has the checks' words,
// the caller's own result tensors and other devices.  So nothing is decided here
// that is not decided there, and without this extension the same calls are made.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <optional>

#include "../../include/moe_routed_gate.h"

namespace {

using at::Tensor;

// The call is not one of those above.
struct NotHere {};

void need(bool yes) {
    if (!yes) throw NotHere{};
}

const Tensor &tensor(PyObject *o) {
    need(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

// `first`, of any shape of so many dimensions: its device is the call's
const Tensor &first(PyObject *o, int64_t dims) {
    const Tensor &t = tensor(o);
    need(t.is_cuda() && t.dim() == dims && t.is_contiguous() && t.get_device() == c10::cuda::current_device());
    return t;
}

const Tensor &like(PyObject *o, const Tensor &on, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const Tensor &t = tensor(o);
    need(t.is_cuda() && t.scalar_type() == type && t.get_device() == on.get_device() && t.is_contiguous() &&
         t.sizes() == at::IntArrayRef(shape.begin(), shape.size()));
    return t;
}

// e4m3 elements and scale bytes [.., K / 32]
void scaled(PyObject *o, const Tensor &q) {
    need(q.scalar_type() == at::kFloat8_e4m3fn);
    const int64_t n = q.dim(), K = q.size(n - 1);
    need(K % 32 == 0);
    const Tensor &sf = tensor(o);
    need(sf.is_cuda() && sf.scalar_type() == at::kByte && sf.get_device() == q.get_device() && sf.is_contiguous() && sf.dim() == n &&
         sf.size(n - 1) == K / 32);
    for (int64_t i = 0; i + 1 < n; ++i) need(sf.size(i) == q.size(i));
}

Tensor made(const Tensor &on, at::ScalarType type, at::IntArrayRef shape) {
    return at::detail::empty_cuda(shape, type, on.device(), std::nullopt);
}

moe_dtype_t code(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return MOE_F16;
        case at::kBFloat16: return MOE_BF16;
        case at::kFloat: return MOE_F32;
        default: throw NotHere{};
    }
}

at::ScalarType type_of(long c) {
    need(c >= 0 && c <= 2);
    return c == 0 ? at::kHalf : c == 1 ? at::kBFloat16 : at::kFloat;
}

template <typename T> T *at_(const Tensor &t) { return static_cast<T *>(t.data_ptr()); }

moe_stream_t stream_of(const Tensor &t) {
    return reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}

int32_t *error_word(PyObject *o, const Tensor &on) {
    if (o == Py_None) return nullptr;
    const Tensor &t = tensor(o);
    need(t.is_cuda() && t.scalar_type() == at::kInt && t.is_contiguous() && t.get_device() == on.get_device());
    return at_<int32_t>(t);
}

PyObject *wrapped(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject *tuple_of(std::initializer_list<Tensor> ts) {
    PyObject *out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor &t : ts) {
        PyObject *o = wrapped(t);
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

// The entry point's status: anything but success is the Python code's to report, by
// the same call again (a refused call has launched nothing).
template <typename F> void call(F f) {
    struct OtherThreads {  // may run meanwhile, also where f ends with an exception
        PyThreadState *state = PyEval_SaveThread();
        ~OtherThreads() { PyEval_RestoreThread(state); }
    };
    moe_status_t st;
    {
        OtherThreads others;
        st = f();
    }
    need(st == MOE_OK);
}

template <typename F> PyObject *guarded(F f) {
    try {
        return f();
    } catch (const NotHere &) {
    } catch (const std::exception &) {  // no memory, among others: the Python code meets it again
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// (y, res, w_post, gate, alpha, w_next, eps, with_u, out) -> (out, u, q, sf, rstd_post, rstd_next)
PyObject *norm_mx8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        need(n == 9);
        const Tensor &res = first(a[1], 2);
        const int64_t T = res.size(0), H = res.size(1);
        const at::ScalarType type = res.scalar_type();
        const moe_dtype_t dt = code(type);
        need(H > 0 && H % 32 == 0);
        const bool has_y = a[0] != Py_None;
        const void *y = has_y ? like(a[0], res, type, {T, H}).data_ptr() : nullptr;
        const void *w_post = a[2] != Py_None ? like(a[2], res, type, {H}).data_ptr() : nullptr;
        need(has_y || (a[2] == Py_None && a[3] == Py_None && a[8] == Py_None));
        const void *gate = nullptr;
        moe_gate_t kind = MOE_GATE_NONE;
        if (a[3] != Py_None) {
            const Tensor &g = tensor(a[3]);
            const bool row = g.dim() == 1;
            kind = row ? MOE_GATE_CHANNEL : g.dim() == 2 && g.size(1) == 1 && H != 1 ? MOE_GATE_TOKEN : MOE_GATE_FULL;
            gate = (row ? like(a[3], res, type, {H}) : like(a[3], res, type, {T, kind == MOE_GATE_TOKEN ? 1 : H})).data_ptr();
        }
        need((PyFloat_Check(a[4]) || PyLong_Check(a[4])) && (PyFloat_Check(a[6]) || PyLong_Check(a[6])));
        const double alpha = PyFloat_AsDouble(a[4]), eps = PyFloat_AsDouble(a[6]);
        need(!PyErr_Occurred());
        const Tensor &w_next = like(a[5], res, type, {H});
        const int truth = PyObject_IsTrue(a[7]);
        need(truth >= 0);  // what has none is the Python code's to report
        const bool with_u = truth != 0;
        Tensor out, u, r_post;
        if (has_y) out = a[8] != Py_None ? like(a[8], res, type, {T, H}) : made(res, type, {T, H});
        if (with_u) u = made(res, type, {T, H});
        if (w_post) r_post = made(res, at::kFloat, {T});
        const Tensor q = made(res, at::kFloat8_e4m3fn, {T, H}), sf = made(res, at::kByte, {T, H / 32}), r_next = made(res, at::kFloat, {T});
        const moe_stream_t s = stream_of(res);
        call([&] {
            return moe_residual_norm_mx8(y, res.data_ptr(), w_post, gate, kind, static_cast<float>(alpha), w_next.data_ptr(),
                                         static_cast<float>(eps), T, H, dt, has_y ? out.data_ptr() : nullptr,
                                         with_u ? u.data_ptr() : nullptr, at_<uint8_t>(q), at_<uint8_t>(sf),
                                         w_post ? at_<float>(r_post) : nullptr, at_<float>(r_next), s);
        });
        return tuple_of({out, u, q, sf, r_post, r_next});
    });
}

// (q, sf, token_topk_to_pos) -> (q_out, sf_out)
PyObject *sort_rows_mx8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        need(n == 3);
        const Tensor &q = first(a[0], 2);
        scaled(a[1], q);
        const Tensor &sf = THPVariable_Unpack(a[1]), &pos = tensor(a[2]);
        const int64_t T = q.size(0), K = q.size(1);
        need(pos.dim() == 2);
        const int64_t k = pos.size(1), rows = T * k;
        like(a[2], q, at::kInt, {T, k});
        const Tensor q_out = made(q, at::kFloat8_e4m3fn, {rows, K}), sf_out = made(q, at::kByte, {rows, K / 32});
        const moe_stream_t s = stream_of(q);
        call([&] {
            return moe_sort_rows_mx8(at_<uint8_t>(q), at_<uint8_t>(sf), at_<int32_t>(pos), T, k, rows, K, at_<uint8_t>(q_out),
                                     at_<uint8_t>(sf_out), s);
        });
        return tuple_of({q_out, sf_out});
    });
}

// (d_out, x, token_topk_to_pos, topk_weights, sorted_token_idx, err) -> (d_x, d_topk_w)
PyObject *reduce_fused_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        need(n == 6);
        const Tensor &x = first(a[1], 2), &pos = tensor(a[2]), &d_out = tensor(a[0]);
        const int64_t rows = x.size(0), H = x.size(1);
        need(pos.dim() == 2);
        const int64_t T = pos.size(0), K = pos.size(1);
        like(a[2], x, at::kInt, {T, K});
        like(a[0], x, d_out.scalar_type(), {T, H});
        const float *w = a[3] != Py_None ? at_<float>(like(a[3], x, at::kFloat, {T, K})) : nullptr;
        const Tensor &token = like(a[4], x, at::kInt, {rows});
        const moe_dtype_t in = code(x.scalar_type()), out = code(d_out.scalar_type());
        int32_t *err = error_word(a[5], x);
        const Tensor d_x = made(x, x.scalar_type(), {rows, H}), d_w = made(x, at::kFloat, {T, K});
        const moe_stream_t s = stream_of(x);
        call([&] {
            return moe_reduce_fused_backward(d_out.data_ptr(), x.data_ptr(), rows, at_<int32_t>(pos), w, at_<int32_t>(token), T, K, H, in,
                                             out, d_x.data_ptr(), at_<float>(d_w), err, s);
        });
        return tuple_of({d_x, d_w});
    });
}

struct Tables {
    const int32_t *sizes, *offsets, *padded, *gidx;
    int64_t blocks;
};

// The four tables of E experts, the last one's length the blocks'.
Tables tables_of(PyObject *const *a, const Tensor &on, int64_t E) {
    Tables t;
    t.sizes = at_<int32_t>(like(a[0], on, at::kInt, {E}));
    t.offsets = at_<int32_t>(like(a[1], on, at::kInt, {E}));
    t.padded = at_<int32_t>(like(a[2], on, at::kInt, {E}));
    const Tensor &g = tensor(a[3]);
    need(g.dim() == 1);
    t.blocks = g.size(0);
    t.gidx = at_<int32_t>(like(a[3], on, at::kInt, {t.blocks}));
    return t;
}

// (q_a, sf_a, q_b, sf_b, group_sizes, group_offsets, group_padded_offsets, group_idx_for_bx, out type's code, err) -> C
PyObject *grouped_gemm_mx8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        need(n == 10);
        const Tensor &q_a = first(a[0], 2), &q_b = first(a[2], 3);
        scaled(a[1], q_a);
        scaled(a[3], q_b);
        const int64_t rows = q_a.size(0), K = q_a.size(1), E = q_b.size(0), N = q_b.size(1);
        need(q_b.size(2) == K && q_b.get_device() == q_a.get_device());
        const Tables t = tables_of(a + 4, q_a, E);
        need(PyLong_Check(a[8]));
        const long out_code = PyLong_AsLong(a[8]);
        need(!PyErr_Occurred());
        int32_t *err = error_word(a[9], q_a);
        const Tensor out = made(q_a, type_of(out_code), {rows, N}), &sf_a = THPVariable_Unpack(a[1]), &sf_b = THPVariable_Unpack(a[3]);
        const moe_stream_t s = stream_of(q_a);
        call([&] {
            return moe_grouped_gemm_mx8(at_<uint8_t>(q_a), at_<uint8_t>(sf_a), at_<uint8_t>(q_b), at_<uint8_t>(sf_b), t.sizes, t.offsets,
                                        t.padded, t.gidx, t.blocks, rows, N, K, E, static_cast<moe_dtype_t>(out_code), out.data_ptr(), err,
                                        s);
        });
        return wrapped(out);
    });
}

// (q_a, sf_a, q_gate, sf_gate, q_up, sf_up, the four tables, err) -> (q_h, sf_h)
PyObject *grouped_gate_up_silu_mx8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        need(n == 11);
        const Tensor &q_a = first(a[0], 2), &gate = first(a[2], 3), &up = first(a[4], 3);
        scaled(a[1], q_a);
        scaled(a[3], gate);
        scaled(a[5], up);
        const int64_t rows = q_a.size(0), d_h = q_a.size(1), E = gate.size(0), d_e = gate.size(1);
        need(gate.size(2) == d_h && up.sizes() == gate.sizes() && d_e % 32 == 0);
        const Tables t = tables_of(a + 6, q_a, E);
        int32_t *err = error_word(a[10], q_a);
        const Tensor q_h = made(q_a, at::kFloat8_e4m3fn, {rows, d_e}), sf_h = made(q_a, at::kByte, {rows, d_e / 32});
        const Tensor &sf_a = THPVariable_Unpack(a[1]), &sf_gate = THPVariable_Unpack(a[3]), &sf_up = THPVariable_Unpack(a[5]);
        const moe_stream_t s = stream_of(q_a);
        call([&] {
            return moe_grouped_gate_up_silu_mx8(at_<uint8_t>(q_a), at_<uint8_t>(sf_a), at_<uint8_t>(gate), at_<uint8_t>(sf_gate),
                                                at_<uint8_t>(up), at_<uint8_t>(sf_up), t.sizes, t.offsets, t.padded, t.gidx, t.blocks, rows,
                                                d_h, d_e, E, at_<uint8_t>(q_h), at_<uint8_t>(sf_h), err, s);
        });
        return tuple_of({q_h, sf_h});
    });
}

// (q_gate, sf_gate, q_up, sf_up, q_down, sf_down) -> (E, d_e, d_h), checked
PyObject *experts_mx8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        need(n == 6);
        const Tensor &gate = first(a[0], 3), &up = first(a[2], 3), &down = first(a[4], 3);
        for (int i = 0; i < 6; i += 2) scaled(a[i + 1], THPVariable_Unpack(a[i]));
        const int64_t E = gate.size(0), d_e = gate.size(1), d_h = gate.size(2);
        need(up.sizes() == gate.sizes() && down.size(0) == E && down.size(1) == d_h && down.size(2) == d_e);
        return Py_BuildValue("(LLL)", static_cast<long long>(E), static_cast<long long>(d_e), static_cast<long long>(d_h));
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)> PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"norm_mx8", fast<norm_mx8>(), METH_FASTCALL, nullptr},
    {"sort_rows_mx8", fast<sort_rows_mx8>(), METH_FASTCALL, nullptr},
    {"reduce_fused_backward", fast<reduce_fused_backward>(), METH_FASTCALL, nullptr},
    {"grouped_gemm_mx8", fast<grouped_gemm_mx8>(), METH_FASTCALL, nullptr},
    {"grouped_gate_up_silu_mx8", fast<grouped_gate_up_silu_mx8>(), METH_FASTCALL, nullptr},
    {"experts_mx8", fast<experts_mx8>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the PyTorch and the Python whose headers this file was compiled with
PyMODINIT_FUNC PyInit__host_calls() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", MOE_BUILT_FOR) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
