// The calls of the operators around the delta-rule kernels from Python, without the ctypes
// marshalling: a decoding step makes several of them per layer, and describing the tensors,
// allocating the outputs and crossing ctypes take longer there than the kernels run.
//
// Each function takes its binding's arguments in the binding's order and returns the result,
// the status as an int where the library refuses the call, or None, with nothing done, where
// the call is not of the plain kind (CUDA tensors on the current device, its current stream,
// dtypes and dimensions that a descriptor can hold): the binding then goes its general way.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/deltanet.h"

namespace {

struct Call {
    dn_tensor room[16];
    int used = 0;
    bool plain = true;
    c10::DeviceIndex dev = -1;                 // the current one, once there is a CUDA tensor

    void* stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
    dn_tensor* describe(const at::Tensor& t) {
        int32_t dtype = -1;
        switch (t.scalar_type()) {
            case at::kFloat: dtype = DN_F32; break;
            case at::kBFloat16: dtype = DN_BF16; break;
            case at::kInt: dtype = DN_I32; break;
            default: break;
        }
        if (t.is_cuda() && dev < 0) dev = c10::cuda::current_device();
        if (dtype < 0 || used == 16 || !t.is_cuda() || t.get_device() != dev || t.layout() != at::kStrided ||
            t.dim() < 1 || t.dim() > 4) {
            plain = false;
            return nullptr;
        }
        dn_tensor& d = room[used++];
        d = dn_tensor();
        d.data = t.data_ptr();
        d.dtype = dtype;
        d.ndim = (int32_t)t.dim();
        for (int i = 0; i < d.ndim; ++i) {
            d.shape[i] = t.size(i);
            d.stride[i] = t.stride(i);
        }
        return &d;
    }
    // None: no tensor
    dn_tensor* operator()(PyObject* o) {
        if (o == Py_None) return nullptr;
        if (THPVariable_Check(o)) return describe(THPVariable_Unpack(o));
        plain = false;
        return nullptr;
    }
    long number(PyObject* o) {
        const long x = PyLong_AsLong(o);
        if (x == -1 && PyErr_Occurred()) PyErr_Clear(), plain = false;
        return x;
    }
    float real(PyObject* o) {
        const double x = PyFloat_AsDouble(o);
        if (x == -1.0 && PyErr_Occurred()) PyErr_Clear(), plain = false;
        return (float)x;
    }
};

const at::Tensor& tensor(PyObject* o) { return THPVariable_Unpack(o); }

// An output: the caller's buffer, or one made here.
struct Out {
    PyObject* given;
    at::Tensor made;
    dn_tensor* d = nullptr;
    Out(Call& c, PyObject* o) : given(o), d(c(o)) {}
    bool wanted() const { return given == Py_None; }
    void make(Call& c, at::IntArrayRef shape, const at::TensorOptions& like) {
        made = at::empty(shape, like);
        d = c.describe(made);
    }
    PyObject* result() const {
        if (made.defined()) return THPVariable_Wrap(made);
        Py_INCREF(given);
        return given;
    }
};

template <typename F>
dn_status without_gil(F f) {
    dn_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return st;
}

PyObject* result(dn_status st, std::initializer_list<const Out*> outs) {
    if (st != DN_OK) return PyLong_FromLong(st);
    if (outs.size() == 1) return (*outs.begin())->result();
    PyObject* t = PyTuple_New((Py_ssize_t)outs.size());
    if (!t) return nullptr;
    Py_ssize_t i = 0;
    for (const Out* o : outs) {
        PyObject* x = o->result();
        if (!x) {
            Py_DECREF(t);
            return nullptr;
        }
        PyTuple_SET_ITEM(t, i++, x);
    }
    return t;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
    return false;
}

PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 9)) return nullptr;
    Call c;
    const dn_tensor *q = c(a[0]), *k = c(a[1]), *v = c(a[2]), *beta = c(a[3]), *g = c(a[5]), *slots = c(a[7]);
    dn_tensor* state = c(a[4]);
    const long nh = c.number(a[6]);
    Out out(c, a[8]);
    if (!c.plain || nh != (int)nh || !q || !v || q->ndim != 4 || v->ndim != 4) Py_RETURN_NONE;
    if (out.wanted()) out.make(c, {q->shape[0], q->shape[1], q->shape[2], v->shape[3]}, tensor(a[0]).options());
    return result(without_gil([&, s = c.stream()] { return deltanet_step(q, k, v, beta, g, (int)nh, state, slots, out.d, s); }), {&out});
    END_HANDLE_TH_ERRORS
}

PyObject* scan_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 7)) return nullptr;
    Call c;
    const dn_tensor *x = c(a[0]), *g = c(a[1]), *s0 = c(a[2]), *cu = c(a[3]);
    Out out(c, a[4]), fin(c, a[5]);
    const int want = PyObject_IsTrue(a[6]);
    if (!c.plain || want < 0 || !x || x->ndim != 3 || (cu && (cu->ndim != 1 || cu->shape[0] < 1))) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const at::Tensor& t = tensor(a[0]);
    if (out.wanted()) out.make(c, t.sizes(), t.options());
    if (fin.wanted() && want) fin.make(c, {cu ? cu->shape[0] - 1 : x->shape[0], x->shape[2]}, t.options().dtype(at::kFloat));
    return result(without_gil([&, s = c.stream()] { return deltanet_scan_fwd(x, g, s0, cu, out.d, fin.d, s); }), {&out, &fin});
    END_HANDLE_TH_ERRORS
}

PyObject* scan_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 9)) return nullptr;
    Call c;
    const dn_tensor *g = c(a[0]), *h = c(a[1]), *dh = c(a[2]), *s0 = c(a[3]), *cu = c(a[4]), *dfin = c(a[5]);
    Out dx(c, a[6]), dg(c, a[7]), dinit(c, a[8]);
    if (!c.plain || !g || !h) Py_RETURN_NONE;
    if (dx.wanted()) dx.make(c, tensor(a[1]).sizes(), tensor(a[1]).options());
    if (dg.wanted()) dg.make(c, tensor(a[0]).sizes(), tensor(a[0]).options());
    if (dinit.wanted() && s0) dinit.make(c, tensor(a[3]).sizes(), tensor(a[3]).options());
    return result(without_gil([&, s = c.stream()] { return deltanet_scan_bwd(g, h, s0, cu, dh, dfin, dx.d, dg.d, dinit.d, s); }),
                  {&dx, &dg, &dinit});
    END_HANDLE_TH_ERRORS
}

PyObject* scan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 5)) return nullptr;
    Call c;
    const dn_tensor *x = c(a[0]), *g = c(a[1]), *slots = c(a[3]);
    dn_tensor* state = c(a[2]);
    Out out(c, a[4]);
    if (!c.plain || !x) Py_RETURN_NONE;
    if (out.wanted()) out.make(c, tensor(a[0]).sizes(), tensor(a[0]).options());
    return result(without_gil([&, s = c.stream()] { return deltanet_scan_step(x, g, state, slots, out.d, s); }), {&out});
    END_HANDLE_TH_ERRORS
}

PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 10)) return nullptr;
    Call c;
    const dn_tensor *y = c(a[0]), *w = c(a[1]), *z = c(a[2]), *r = c(a[3]), *sc = c(a[4]), *nw = c(a[5]);
    const long act = c.number(a[6]);
    const float eps = c.real(a[7]);
    Out out(c, a[8]), rout(c, a[9]);
    if (!c.plain || !y) Py_RETURN_NONE;
    if (out.wanted() && (!r || nw)) out.make(c, tensor(a[0]).sizes(), tensor(a[0]).options());
    if (rout.wanted() && r) rout.make(c, tensor(a[3]).sizes(), tensor(a[3]).options());
    return result(without_gil([&, s = c.stream()] { return deltanet_norm_fwd(y, w, z, (int)act, r, sc, nw, eps, out.d, rout.d, s); }),
                  {&out, &rout});
    END_HANDLE_TH_ERRORS
}

PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 13)) return nullptr;
    Call c;
    const dn_tensor *y = c(a[0]), *dout = c(a[1]), *w = c(a[2]), *z = c(a[3]), *r = c(a[4]), *sc = c(a[5]), *nw = c(a[6]),
                    *dr = c(a[7]);
    const long act = c.number(a[8]);
    const float eps = c.real(a[9]);
    Out dy(c, a[10]), dz(c, a[11]), dres(c, a[12]), dw(c, Py_None), dsc(c, Py_None), dnw(c, Py_None), work(c, Py_None);
    if (!c.plain || !y) Py_RETURN_NONE;
    const int64_t d = y->shape[y->ndim - 1], rows = d ? tensor(a[0]).numel() / d : 0;
    const at::TensorOptions f32 = tensor(a[0]).options().dtype(at::kFloat);
    if (dy.wanted()) dy.make(c, tensor(a[0]).sizes(), tensor(a[0]).options());
    if (dz.wanted() && z) dz.make(c, tensor(a[3]).sizes(), tensor(a[3]).options());
    if (dres.wanted() && r) dres.make(c, tensor(a[4]).sizes(), tensor(a[4]).options());
    if (w) dw.make(c, {d}, f32);
    if (sc) dsc.make(c, {d}, f32);
    if (nw) dnw.make(c, {d}, f32);
    const int64_t need = w || sc || nw ? deltanet_norm_workspace(rows, d) : 0;
    if (need > 0) work.make(c, {need}, f32);
    return result(without_gil([&, s = c.stream()] {
                      return deltanet_norm_bwd(y, w, z, (int)act, r, sc, nw, eps, dout, dr, dy.d, dw.d, dz.d, dres.d, dsc.d,
                                               dnw.d, work.d, s);
                  }),
                  {&dy, &dw, &dz, &dres, &dsc, &dnw});
    END_HANDLE_TH_ERRORS
}

#define DN_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {DN_METHOD(step),      DN_METHOD(scan_fwd), DN_METHOD(scan_bwd), DN_METHOD(scan_step),
                         DN_METHOD(norm_fwd), DN_METHOD(norm_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "dn_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_dn_call(void) { return PyModule_Create(&module); }
