// marshal.cpp -- the Python binding's common path in C++ (module _marshal):
// reads the tensors of a call, allocates its outputs and calls the C ABI.
//
// A decode step of a few microseconds on the GPU is bound by the host; read
// attribute by attribute from Python, the dozen tensors of such a call cost
// about 15 us.  The functions here do the checks of ssm.py on the tensors
// themselves.  They return the call's results, the nonzero status of the
// library as an int, or None for anything that is not plainly right (a wrong
// type, shape, device or layout, an option they do not take): ssm.py then
// goes through its own checks, which name what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "../../include/ssm.h"

namespace {

using at::Tensor;

// Thrown for whatever the slow path has to look at.
struct NotPlain {};

void want(bool ok) {
    if (!ok) throw NotPlain();
}

// A size as the ABI takes it; Python names one that does not fit.
int count(int64_t v) {
    want(v >= 0 && v <= 0x7fffffff);
    return (int)v;
}

// The arguments of a call, in order.
struct Args {
    PyObject *const *p;
    Py_ssize_t n, i = 0;
    PyObject *next() {
        want(i < n);
        return p[i++];
    }
    const Tensor *optional() {
        PyObject *o = next();
        if (o == Py_None) return nullptr;
        want(THPVariable_Check(o));
        return &THPVariable_Unpack(o);
    }
    const Tensor &tensor() {
        const Tensor *t = optional();
        want(t != nullptr);
        return *t;
    }
    // what has no truth value is the slow path's to name, before anything is launched
    bool flag() {
        const int v = PyObject_IsTrue(next());
        want(v >= 0);
        return v == 1;
    }
};

int code_of(at::ScalarType t) {
    want(t == at::kBFloat16 || t == at::kFloat);
    return t == at::kBFloat16 ? SSM_BF16 : SSM_F32;
}

// Everything about one call's device: tensors have to be on the current one.
struct Device {
    int index;
    explicit Device(const Tensor &t) : index(-1) {
        want(t.is_cuda());
        index = t.get_device();
        want(index == c10::cuda::current_device());
    }
    cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }
    // address of a contiguous tensor of this type and shape
    void *data(const Tensor &t, at::ScalarType type, at::IntArrayRef shape) const {
        want(t.is_cuda() && t.get_device() == index && t.scalar_type() == type && t.sizes() == shape && t.is_contiguous());
        return t.data_ptr();
    }
    void *data(const Tensor *t, at::ScalarType type, at::IntArrayRef shape) const { return t ? data(*t, type, shape) : nullptr; }
    const float *f32(const Tensor *t, at::IntArrayRef shape) const { return static_cast<const float *>(data(t, at::kFloat, shape)); }
    const int32_t *i32(const Tensor *t, at::IntArrayRef shape) const { return static_cast<const int32_t *>(data(t, at::kInt, shape)); }
    int *status(const Tensor *t) const {
        if (!t) return nullptr;
        return static_cast<int *>(data(*t, at::kInt, t->sizes()));
    }
};

// An activation: leading axes (tokens) and contiguous, equally spaced rows.
struct Rows {
    const void *p = nullptr;
    int64_t stride = 0;
    Rows() = default;
    Rows(const Device &dev, const Tensor &t, at::ScalarType type, at::IntArrayRef lead, at::IntArrayRef row) {
        const size_t k = lead.size();
        want(t.is_cuda() && t.get_device() == dev.index && t.scalar_type() == type && (size_t)t.dim() == k + row.size());
        int64_t width = 1, tokens = 1;
        for (size_t i = 0; i < row.size(); ++i) {
            want(t.size(k + i) == row[i]);
            width *= row[i];
        }
        for (size_t i = 0; i < k; ++i) {
            want(t.size(i) == lead[i]);
            tokens *= lead[i];
        }
        p = t.data_ptr();
        stride = width;
        if (!tokens) return;
        int64_t step = 1;
        for (size_t i = row.size(); i-- > 0;) {
            want(row[i] == 1 || t.stride(k + i) == step);
            step *= row[i];
        }
        if (k == 1) {
            if (lead[0] > 1) stride = t.stride(0);
            return;
        }
        if (lead[1] > 1) stride = t.stride(1);
        else if (lead[0] > 1) stride = t.stride(0);
        want(lead[0] <= 1 || lead[1] <= 1 || t.stride(0) == lead[1] * stride);
    }
};

// Sequences of an x [nseq, L, dim], or packed [T, dim] with cu_seqlens.
struct Tokens {
    int64_t lead[2], nlead, nseq, seqlen, T, dim;
    const int32_t *cu = nullptr;
    Tokens(const Device &dev, const Tensor &x, const Tensor *cu_seqlens) {
        if (cu_seqlens) {
            want(x.dim() == 2 && cu_seqlens->dim() == 1 && cu_seqlens->size(0) >= 1);
            cu = dev.i32(cu_seqlens, cu_seqlens->sizes());
            nlead = 1;
            lead[0] = T = seqlen = x.size(0);
            nseq = cu_seqlens->size(0) - 1;
            dim = x.size(1);
        } else {
            want(x.dim() == 3);
            nlead = 2;
            lead[0] = nseq = x.size(0);
            lead[1] = seqlen = x.size(1);
            T = nseq * seqlen;
            dim = x.size(2);
        }
        count(T);
    }
    at::IntArrayRef axes() const { return at::IntArrayRef(lead, nlead); }
};

// The operands every per-channel call takes, in the order of its signature:
// x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit.
struct Operands {
    Rows x, dt, B, C, z;
    const float *A, *D;
    int64_t N, G;
    int in_code, dt_code;
    ssm_dt_params params{};
    bool has_params, gate;
    const ssm_dt_params *dt_params() const { return has_params ? &params : nullptr; }
    Operands(const Device &dev, Args &a, const Tensor &tx, at::IntArrayRef lead, int64_t dim) {
        const Tensor &tdt = a.tensor(), &tA = a.tensor(), &tB = a.tensor(), &tC = a.tensor();
        const Tensor *tD = a.optional(), *tz = a.optional(), *bias = a.optional();
        const bool softplus = a.flag();
        PyObject *limit = a.next();
        const at::ScalarType type = tx.scalar_type();
        in_code = code_of(type);
        dt_code = code_of(tdt.scalar_type());
        want(tA.dim() == 2 && (size_t)tB.dim() == lead.size() + 2);
        N = tA.size(1);
        G = tB.size(-2);
        const int64_t row[1] = {dim}, bc[2] = {G, N}, an[2] = {dim, N};
        A = dev.f32(&tA, an);
        D = dev.f32(tD, row);
        x = Rows(dev, tx, type, lead, row);
        dt = Rows(dev, tdt, tdt.scalar_type(), lead, row);
        B = Rows(dev, tB, type, lead, bc);
        C = Rows(dev, tC, type, lead, bc);
        gate = tz != nullptr;
        if (gate) z = Rows(dev, *tz, type, lead, row);
        params.dt_bias = dev.f32(bias, row);
        params.softplus = softplus;
        params.clamp = limit != Py_None;
        if (params.clamp) {
            want(PyTuple_Check(limit) && PyTuple_GET_SIZE(limit) == 2);
            double v[2];
            for (int i = 0; i < 2; ++i) {
                v[i] = PyFloat_AsDouble(PyTuple_GET_ITEM(limit, i));
                if (PyErr_Occurred()) {
                    PyErr_Clear();
                    throw NotPlain();
                }
            }
            params.dt_min = (float)v[0];
            params.dt_max = (float)v[1];
        }
        has_params = bias || softplus || params.clamp;
    }
};

Tensor fresh(const Tensor &like, at::IntArrayRef shape, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type).requires_grad(false));
}
PyObject *wrap(const Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
void *addr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// f(args), with NotPlain and any error of torch as None.
template <typename F>
PyObject *guarded(F f, PyObject *const *p, Py_ssize_t n) {
    try {
        Args a{p, n};
        return f(a);
    } catch (const NotPlain &) {
    } catch (const std::exception &) {
    }
    if (PyErr_Occurred()) PyErr_Clear();
    Py_RETURN_NONE;
}
PyObject *result(int status, std::initializer_list<PyObject *> items) {
    if (status == SSM_OK) {
        PyObject *t = PyTuple_New((Py_ssize_t)items.size());
        Py_ssize_t i = 0;
        for (PyObject *o : items) PyTuple_SET_ITEM(t, i++, o);
        return t;
    }
    for (PyObject *o : items) Py_XDECREF(o);
    return PyLong_FromLong(status);
}
PyObject *ref(const Tensor *t) { return t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None); }

// x, cu_seqlens, dt .. dt_limit, initial_state, final_state, slot_idx,
// has_initial_state, y, return_final_state, save_states, status -> (y, final_state, saved or None)
PyObject *scan_fwd(PyObject *, PyObject *const *p, Py_ssize_t n) {
    return guarded([](Args &a) {
        const Tensor &x = a.tensor();
        const Device dev(x);
        const Tokens t(dev, x, a.optional());
        const Operands o(dev, a, x, t.axes(), t.dim);
        const Tensor *init = a.optional(), *fin = a.optional(), *slots = a.optional(), *has = a.optional(), *y = a.optional();
        const bool want_final = a.flag(), save = a.flag();
        const Tensor *status = a.optional();
        const int64_t seqs[1] = {t.nseq};
        int64_t state[3] = {t.nseq, t.dim, o.N};
        Tensor made_final, made_y, saved, ws;
        if (slots) {
            const Tensor *pool = fin ? fin : init;
            want(pool && pool->dim() == 3);
            state[0] = pool->size(0);
        } else if (!fin && want_final) {
            made_final = fresh(x, state, at::kFloat);
            fin = &made_final;
        }
        if (!y) {
            made_y = fresh(x, x.sizes(), x.scalar_type());
            y = &made_y;
        }
        size_t wsb = 0;
        if (save) {
            saved = fresh(x, {(int64_t)(selective_scan_saved_size(count(t.nseq), t.T, count(t.dim), count(o.N)) / 4)}, at::kFloat);
        }
        if ((wsb = selective_scan_workspace_size(count(t.nseq), t.T, count(t.dim), count(o.N), count(o.G)))) {
            ws = fresh(x, {(int64_t)wsb}, at::kByte);
        }
        const int st = selective_scan_fwd(
            count(t.nseq), count(t.seqlen), t.cu, count(t.dim), count(o.N), count(o.G), o.in_code, o.x.p, o.x.stride, o.dt_code, o.dt.p,
            o.dt.stride, o.A, o.B.p, o.B.stride, o.C.p, o.C.stride, o.D, o.z.p, o.z.stride, o.dt_params(), dev.f32(init, state),
            static_cast<float *>(dev.data(fin, at::kFloat, state)), count(state[0]), dev.i32(slots, seqs), dev.i32(has, seqs),
            code_of(y->scalar_type()), dev.data(*y, y->scalar_type(), x.sizes()), static_cast<float *>(addr(saved)), addr(ws), wsb,
            dev.status(status), dev.stream());
        return result(st, {ref(y), ref(fin), wrap(saved)});
    }, p, n);
}

// x, cu_seqlens, dt .. dt_limit, dy, saved, dfinal_state, want_dinitial, status -> the nine gradients
PyObject *scan_bwd(PyObject *, PyObject *const *p, Py_ssize_t n) {
    return guarded([](Args &a) {
        const Tensor &x = a.tensor();
        const Device dev(x);
        const Tokens t(dev, x, a.optional());
        const Operands o(dev, a, x, t.axes(), t.dim);
        const Tensor &tdy = a.tensor(), &saved = a.tensor();
        const Tensor *dfin = a.optional();
        const bool want_init = a.flag();
        const Tensor *status = a.optional();
        want(t.nseq > 0);
        const int64_t row[1] = {t.dim}, state[3] = {t.nseq, t.dim, o.N}, an[2] = {t.dim, o.N};
        const at::ScalarType type = x.scalar_type();
        const Rows dy(dev, tdy, type, t.axes(), row);
        want((size_t)saved.numel() * 4 == selective_scan_saved_size(count(t.nseq), t.T, count(t.dim), count(o.N)));
        std::vector<int64_t> bc(t.lead, t.lead + t.nlead);
        bc.push_back(o.G);
        bc.push_back(o.N);
        Tensor dx = fresh(x, x.sizes(), type), ddt = fresh(x, x.sizes(), o.dt_code == SSM_BF16 ? at::kBFloat16 : at::kFloat),
               dA = fresh(x, an, at::kFloat), dB = fresh(x, bc, type), dC = fresh(x, bc, type), dD, dz, db, di;
        if (o.D) dD = fresh(x, row, at::kFloat);
        if (o.gate) dz = fresh(x, x.sizes(), type);
        if (o.params.dt_bias) db = fresh(x, row, at::kFloat);
        if (want_init) di = fresh(x, state, at::kFloat);
        const size_t wsb = selective_scan_bwd_workspace_size(count(t.nseq), t.T, count(t.dim), count(o.N), count(o.G));
        Tensor ws = fresh(x, {(int64_t)wsb}, at::kByte);
        const int st = selective_scan_bwd(
            count(t.nseq), count(t.seqlen), t.cu, count(t.dim), count(o.N), count(o.G), o.in_code, dy.p, dy.stride, o.x.p, o.x.stride,
            o.dt_code, o.dt.p, o.dt.stride, o.A, o.B.p, o.B.stride, o.C.p, o.C.stride, o.D, o.z.p, o.z.stride, o.dt_params(),
            dev.f32(&saved, saved.sizes()), dev.f32(dfin, state), dx.data_ptr(), ddt.data_ptr(), static_cast<float *>(dA.data_ptr()),
            dB.data_ptr(), dC.data_ptr(), static_cast<float *>(addr(dD)), addr(dz), static_cast<float *>(addr(db)),
            static_cast<float *>(addr(di)), ws.data_ptr(), wsb, dev.status(status), dev.stream());
        return result(st, {wrap(dx), wrap(ddt), wrap(dA), wrap(dB), wrap(dC), wrap(dD), wrap(dz), wrap(db), wrap(di)});
    }, p, n);
}

// x, dt .. dt_limit, state, slot_idx, y, status -> (y,)
PyObject *state_update(PyObject *, PyObject *const *p, Py_ssize_t n) {
    return guarded([](Args &a) {
        const Tensor &x = a.tensor();
        const Device dev(x);
        want(x.dim() == 2);
        const int64_t lead[1] = {x.size(0)}, dim = x.size(1);
        const Operands o(dev, a, x, lead, dim);
        const Tensor &state = a.tensor(), *slots = a.optional(), *y = a.optional(), *status = a.optional();
        want(state.dim() == 3);
        const int64_t rows[3] = {slots ? state.size(0) : lead[0], dim, o.N};
        Tensor made;
        if (!y) {
            made = at::zeros(x.sizes(), x.options().requires_grad(false));
            y = &made;
        }
        const int st = selective_state_update(
            count(lead[0]), count(dim), count(o.N), count(o.G), static_cast<float *>(dev.data(state, at::kFloat, rows)), count(rows[0]),
            dev.i32(slots, lead), o.in_code, o.x.p, o.x.stride, o.dt_code, o.dt.p, o.dt.stride, o.A, o.B.p, o.B.stride, o.C.p,
            o.C.stride, o.D, o.z.p, o.z.stride, o.dt_params(), code_of(y->scalar_type()), dev.data(*y, y->scalar_type(), x.sizes()),
            dev.status(status), dev.stream());
        return result(st, {ref(y)});
    }, p, n);
}

// x, cu_seqlens, dy, weight, bias, initial_state, dfinal_state, activation, status -> (dx, dweight, dbias, dinitial_state)
PyObject *conv1d_bwd(PyObject *, PyObject *const *p, Py_ssize_t n) {
    return guarded([](Args &a) {
        const Tensor &x = a.tensor();
        const Device dev(x);
        const Tokens t(dev, x, a.optional());
        const Tensor &dy = a.tensor(), &w = a.tensor(), *bias = a.optional(), *init = a.optional(), *dfin = a.optional();
        const long act = PyLong_AsLong(a.next());
        const Tensor *status = a.optional();
        const at::ScalarType type = x.scalar_type();
        want(w.dim() == 2 && w.size(1) >= 1);
        const int64_t K = w.size(1), row[1] = {t.dim}, wk[2] = {t.dim, K}, line[3] = {t.nseq, t.dim, K - 1};
        Tensor dx = fresh(x, x.sizes(), type), dw = fresh(x, wk, at::kFloat), db, di;
        if (bias) db = fresh(x, row, at::kFloat);
        if (init) di = fresh(x, line, type);
        const size_t wsb = causal_conv1d_bwd_workspace_size(t.T, count(t.dim), count(K));
        Tensor ws = fresh(x, {(int64_t)wsb}, at::kByte);
        const int st = causal_conv1d_bwd(
            count(t.nseq), count(t.seqlen), t.cu, count(t.dim), count(K), code_of(type), dev.data(dy, type, x.sizes()),
            dev.data(x, type, x.sizes()), dev.f32(&w, wk), dev.f32(bias, row), (int)act, dev.data(init, type, line),
            dev.data(dfin, type, line), dx.data_ptr(), static_cast<float *>(dw.data_ptr()), static_cast<float *>(addr(db)), addr(di),
            wsb ? ws.data_ptr() : nullptr, wsb, dev.status(status), dev.stream());
        return result(st, {wrap(dx), wrap(dw), wrap(db), wrap(di)});
    }, p, n);
}

// The pools of a call: a tensor, or a list or tuple of them, [max_slots, ...] with contiguous rows.
struct Pools {
    std::vector<ssm_pool> rows;
    const Tensor *first = nullptr;
    int64_t slots = 0;
    explicit Pools(PyObject *o) {
        if (THPVariable_Check(o)) {
            add(THPVariable_Unpack(o));
            return;
        }
        want(PyList_Check(o) || PyTuple_Check(o));
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
        want(n > 0);
        rows.reserve((size_t)n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            PyObject *t = PySequence_Fast_GET_ITEM(o, i);
            want(THPVariable_Check(t));
            add(THPVariable_Unpack(t));
        }
    }
    void add(const Tensor &t) {
        want(t.dim() >= 1 && t.is_cuda());
        if (!first) {
            first = &t;
            slots = t.size(0);
            want(slots > 0);
        }
        want(t.get_device() == first->get_device() && t.size(0) == slots);
        int64_t step = 1;
        for (int64_t i = t.dim() - 1; i > 0; --i) {
            want(t.size(i) == 1 || t.stride(i) == step);
            step *= t.size(i);
        }
        const int64_t size = (int64_t)t.element_size();
        rows.push_back(ssm_pool{t.data_ptr(), step * size, (slots > 1 ? t.stride(0) : step) * size});
    }
};

// pools, src_idx, dst_idx, status -> ()
PyObject *pool_copy(PyObject *, PyObject *const *p, Py_ssize_t n) {
    return guarded([](Args &a) {
        const Pools q(a.next());
        const Device dev(*q.first);
        const Tensor &src = a.tensor(), &dst = a.tensor(), *status = a.optional();
        want(src.dim() == 1);
        const int st = ssm_pool_copy(count(q.rows.size()), q.rows.data(), count(q.slots), count(src.size(0)), dev.i32(&src, src.sizes()),
                                     dev.i32(&dst, src.sizes()), dev.status(status), dev.stream());
        return result(st, {});
    }, p, n);
}

// pools, row_idx, status -> ()
PyObject *pool_zero(PyObject *, PyObject *const *p, Py_ssize_t n) {
    return guarded([](Args &a) {
        const Pools q(a.next());
        const Device dev(*q.first);
        const Tensor &rows = a.tensor(), *status = a.optional();
        want(rows.dim() == 1);
        const int st = ssm_pool_zero(count(q.rows.size()), q.rows.data(), count(q.slots), count(rows.size(0)),
                                     dev.i32(&rows, rows.sizes()), dev.status(status), dev.stream());
        return result(st, {});
    }, p, n);
}

// pools, slot_idx, status -> (live,)
PyObject *pool_compact(PyObject *, PyObject *const *p, Py_ssize_t n) {
    return guarded([](Args &a) {
        const Pools q(a.next());
        const Device dev(*q.first);
        const Tensor &table = a.tensor(), *status = a.optional();
        want(table.dim() == 1);
        int32_t *slots = static_cast<int32_t *>(dev.data(table, at::kInt, table.sizes()));
        Tensor live = fresh(table, {}, at::kInt);
        const size_t wsb = ssm_pool_compact_workspace_size(count(q.slots), count(table.size(0)));
        Tensor ws = fresh(table, {(int64_t)wsb}, at::kByte);
        const int st = ssm_pool_compact(count(q.rows.size()), q.rows.data(), count(q.slots), count(table.size(0)), slots,
                                        static_cast<int32_t *>(live.data_ptr()), ws.data_ptr(), wsb, dev.status(status), dev.stream());
        return result(st, {wrap(live)});
    }, p, n);
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(scan_fwd), ENTRY(scan_bwd), ENTRY(state_update), ENTRY(conv1d_bwd), ENTRY(pool_copy),
                         ENTRY(pool_zero), ENTRY(pool_compact), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

#ifndef SSM_TORCH_VERSION
#error "SSM_TORCH_VERSION: the torch.__version__ whose headers these are"
#endif

// torch_version: what it was built for; ssm.py uses it with no other.
PyMODINIT_FUNC PyInit__marshal(void) {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", SSM_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
