// Tensor checks and argument marshalling of the calls around the experts
// (moe_select_experts, moe_add_adapters, moe_block_norm) for moe.py.  Decode
// makes them once per layer and token, each with up to ten tensors: the same
// checks through Python attributes and ctypes took 6 to 9 us a call, most of what
// such a call costs; here they take less than 1 us.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <stdarg.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "moe_b200.h"

namespace {

PyObject* g_error = nullptr;         // moe.MoeError(status, message)

void raise(int status, const char* msg) {
    PyObject* e = PyObject_CallFunction(g_error, "is", status, msg);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
}

bool refuse(const char* fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    raise(MOE_ERR_INVALID_ARG, msg);
    return false;
}

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

constexpr at::ScalarType kBF16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt;
const char* name_of(at::ScalarType t) { return t == kBF16 ? "bfloat16" : t == kF32 ? "float32" : "int32"; }

// The address of a contiguous CUDA tensor of this type and shape on device dev
bool flat(const char* name, PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, int dev, const void** p) {
    const at::Tensor* t = tensor(o);
    if (t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && t->sizes() == at::IntArrayRef(shape.begin(), shape.size()) &&
        t->is_contiguous()) {
        *p = t->data_ptr();
        return true;
    }
    char dims[96] = "";
    size_t at = 0;
    for (int64_t s : shape) at += snprintf(dims + at, sizeof dims - at, "%s%lld", at ? ", " : "", (long long)s);
    return refuse("%s: need a contiguous %s tensor [%s] on cuda:%d", name, name_of(type), dims, dev);
}

// The 2-D CUDA tensor that sets a call's sizes
bool lead(const char* name, PyObject* o, int64_t* T, int64_t* W, int* dev) {
    const at::Tensor* t = tensor(o);
    if (!t || !t->is_cuda() || t->dim() != 2) return refuse("%s: need a 2-D CUDA tensor", name);
    *T = t->size(0);
    *W = t->size(1);
    *dev = t->get_device();
    if (*T > INT32_MAX || *W > INT32_MAX) return refuse("%s: too large", name);
    return true;
}

// Address and row distance of a tensor [T, W] with contiguous rows, bf16 or (where
// f32 is allowed; told by *is_f32) fp32
bool rows(const char* name, PyObject* o, bool bf16, bool f32, int64_t T, int64_t W, int dev, const void** p, int64_t* ld, int32_t* is_f32 = nullptr) {
    const at::Tensor* t = tensor(o);
    if (!t || !t->is_cuda() || t->get_device() != dev || !((bf16 && t->scalar_type() == kBF16) || (f32 && t->scalar_type() == kF32)) || t->dim() != 2 ||
        t->size(0) != T || t->size(1) != W)
        return refuse("%s: need %s%s%s [%lld, %lld] on cuda:%d", name, bf16 ? "bfloat16" : "", bf16 && f32 ? " or " : "", f32 ? "float32" : "",
                      (long long)T, (long long)W, dev);
    if (W > 1 && t->stride(1) != 1) return refuse("%s: the elements of a row must be contiguous", name);
    *p = t->data_ptr();
    *ld = T > 1 ? t->stride(0) : W;
    if (is_f32) *is_f32 = t->scalar_type() == kF32;
    return true;
}

// device dev current and its stream (None: torch's current one) for a call
struct On {
    int prev;
    moe_stream_t stream;
    bool ok = true;
    On(int dev, PyObject* s) : prev(c10::cuda::current_device()), stream(nullptr) {
        if (s == Py_None) {
            stream = reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
        } else {
            stream = reinterpret_cast<moe_stream_t>(PyLong_AsVoidPtr(s));
            ok = !PyErr_Occurred();
        }
        cur = dev;
        if (prev != dev) c10::cuda::set_device((c10::DeviceIndex)dev);
    }
    ~On() {
        if (prev != cur) c10::cuda::set_device((c10::DeviceIndex)prev);
    }
    int cur;
};

PyObject* done(moe_status s) {
    if (s == MOE_OK) Py_RETURN_NONE;
    raise(s, moe_last_error(nullptr));
    return nullptr;
}

bool count(const char* fn, Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, need %zd", fn, n, want);
    return false;
}

// C++ exceptions (torch's checks) end at the C entries
template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// init(MoeError)
PyObject* init(PyObject*, PyObject* error) {
    Py_INCREF(error);
    Py_XDECREF(g_error);
    g_error = error;
    Py_RETURN_NONE;
}

// select_experts(logits, k, address of the moe_routing, bias or None, ids, w, stream)
PyObject* select_experts(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (!count("select_experts", n, 7)) return nullptr;
        int64_t T, E, ld;
        int dev;
        const void *logits, *ids, *w, *bias;
        const long k = PyLong_AsLong(v[1]);
        const void* rule = PyLong_AsVoidPtr(v[2]);
        if (PyErr_Occurred()) return nullptr;
        if (!lead("logits", v[0], &T, &E, &dev) || !rows("logits", v[0], false, true, T, E, dev, &logits, &ld)) return nullptr;
        if (v[3] != Py_None && !flat("bias", v[3], kF32, {E}, dev, &bias)) return nullptr;
        if (!flat("ids", v[4], kI32, {T, k}, dev, &ids) || !flat("w", v[5], kF32, {T, k}, dev, &w)) return nullptr;
        On on(dev, v[6]);
        if (!on.ok) return nullptr;
        return done(moe_select_experts(static_cast<const float*>(logits), ld, (int32_t)T, (int32_t)E, (int32_t)k, static_cast<const moe_routing*>(rule),
                                       static_cast<int32_t*>(const_cast<void*>(ids)), static_cast<float*>(const_cast<void*>(w)), on.stream));
    });
}

// add_adapters(x, y, adapter_ids, a, b, scales, ranks or None, out, stream)
PyObject* add_adapters(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (!count("add_adapters", n, 9)) return nullptr;
        int64_t T, K, ld_x, ld_y, ld_out;
        int dev;
        int32_t f32, out_f32;
        const void *x, *y, *out, *ids, *a, *b, *scales, *ranks = nullptr;
        if (!lead("x", v[0], &T, &K, &dev) || !rows("x", v[0], true, false, T, K, dev, &x, &ld_x)) return nullptr;
        const at::Tensor *ta = tensor(v[3]), *tb = tensor(v[4]);
        if (!ta || ta->dim() != 3 || !tb || tb->dim() != 3) {
            refuse("a and b: need [n, R, K] and [n, N, R]");
            return nullptr;
        }
        const int64_t na = ta->size(0), R = ta->size(1), N = tb->size(1);
        if (na > INT32_MAX || R > INT32_MAX || N > INT32_MAX) {
            refuse("a and b: too large");
            return nullptr;
        }
        if (!flat("a", v[3], kBF16, {na, R, K}, dev, &a) || !flat("b", v[4], kBF16, {na, N, R}, dev, &b) || !flat("scales", v[5], kF32, {na}, dev, &scales) ||
            (v[6] != Py_None && !flat("ranks", v[6], kI32, {na}, dev, &ranks)) || !flat("adapter_ids", v[2], kI32, {T}, dev, &ids) ||
            !rows("y", v[1], true, true, T, N, dev, &y, &ld_y, &f32) || !rows("out", v[7], !f32, f32 != 0, T, N, dev, &out, &ld_out, &out_f32))
            return nullptr;
        moe_adapters ad;
        ad.a = a;
        ad.b = b;
        ad.scales = static_cast<const float*>(scales);
        ad.ranks = static_cast<const int32_t*>(ranks);
        ad.num_adapters = (int32_t)na;
        ad.R = (int32_t)R;
        ad.K = (int32_t)K;
        ad.N = (int32_t)N;
        On on(dev, v[8]);
        if (!on.ok) return nullptr;
        return done(moe_add_adapters(x, ld_x, y, ld_y, const_cast<void*>(out), ld_out, f32, (int32_t)T, static_cast<const int32_t*>(ids), &ad, on.stream));
    });
}

// block_norm(r, y, post_weight, gate, gate_sigmoid, pre_weight, eps, branch_scale,
// residual_scale, unit_offset, r_out, x_out, stream); tensors may be None but r
PyObject* block_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (!count("block_norm", n, 13)) return nullptr;
        moe_norm p = {};
        int64_t T, H;
        int dev;
        const void* q;
        int32_t out_f32;
        const int sigmoid = PyObject_IsTrue(v[4]), offset = PyObject_IsTrue(v[9]);
        p.eps = (float)PyFloat_AsDouble(v[6]);
        p.branch_scale = (float)PyFloat_AsDouble(v[7]);
        p.residual_scale = (float)PyFloat_AsDouble(v[8]);
        if (PyErr_Occurred()) return nullptr;
        p.gate_sigmoid = sigmoid;
        p.unit_offset = offset;
        if (!lead("r", v[0], &T, &H, &dev) || !rows("r", v[0], true, true, T, H, dev, &p.r, &p.ld_r, &p.r_fp32)) return nullptr;
        p.T = (int32_t)T;
        p.H = (int32_t)H;
        if (v[1] != Py_None && !rows("y", v[1], true, false, T, H, dev, &p.y, &p.ld_y)) return nullptr;
        if (v[2] != Py_None && !flat("post_weight", v[2], kBF16, {H}, dev, &p.w_post)) return nullptr;
        if (v[3] != Py_None) {
            const at::Tensor* g = tensor(v[3]);
            if (g && g->dim() == 2) {
                p.gate_kind = MOE_GATE_ELEMENT;
                if (!rows("gate", v[3], true, false, T, H, dev, &p.gate, &p.ld_gate)) return nullptr;
            } else if (g && g->scalar_type() == kF32) {
                p.gate_kind = MOE_GATE_TOKEN;
                if (!flat("gate", v[3], kF32, {T}, dev, &p.gate)) return nullptr;
            } else {
                p.gate_kind = MOE_GATE_CHANNEL;
                if (!flat("gate", v[3], kBF16, {H}, dev, &p.gate)) return nullptr;
            }
        }
        if (v[5] != Py_None && !flat("pre_weight", v[5], kBF16, {H}, dev, &p.w_pre)) return nullptr;
        if (!rows("r_out", v[10], !p.r_fp32, p.r_fp32 != 0, T, H, dev, &q, &p.ld_r_out, &out_f32)) return nullptr;
        p.r_out = const_cast<void*>(q);
        if (v[11] != Py_None) {
            if (!rows("x_out", v[11], true, false, T, H, dev, &q, &p.ld_x)) return nullptr;
            p.x_out = const_cast<void*>(q);
        }
        // a null address of an empty tensor must not read as an absent one
        if (T == 0) Py_RETURN_NONE;
        On on(dev, v[12]);
        if (!on.ok) return nullptr;
        return done(moe_block_norm(&p, on.stream));
    });
}

PyMethodDef methods[] = {
    {"init", init, METH_O, nullptr},
    {"select_experts", (PyCFunction)(void (*)(void))select_experts, METH_FASTCALL, nullptr},
    {"add_adapters", (PyCFunction)(void (*)(void))add_adapters, METH_FASTCALL, nullptr},
    {"block_norm", (PyCFunction)(void (*)(void))block_norm, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
