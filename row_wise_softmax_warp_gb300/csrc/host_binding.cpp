// host_binding.cpp - the compiled part of the Python binding (module _host): argument
// checks, outputs, the current stream and the C call of the operators whose smallest
// calls take the device a few microseconds.
//
// binding.py gives every argument by position and None for what the caller left out.  A
// wrong argument raises TypeError or ValueError; a call that the library refuses returns
// its status as an int, which binding.py raises.  Outputs are allocated by torch on the
// current stream of the tensors' device.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <string>
#include <vector>

#include "rowops.h"

namespace {

using at::ScalarType;
using Shape = c10::SmallVector<int64_t, 6>;

struct Library {
    decltype(&rowops_quantize_mx4) quantize_mx4;
    decltype(&rowops_expert_matmul_mx4_workspace) matmul_mx4_workspace;
    decltype(&rowops_expert_matmul_mx4) matmul_mx4;
    decltype(&rowops_dropout) dropout;
    decltype(&rowops_add_rmsnorm_fwd) norm_fwd;
    decltype(&rowops_add_rmsnorm_bwd_workspace) norm_bwd_workspace;
    decltype(&rowops_add_rmsnorm_bwd) norm_bwd;
} lib;

constexpr std::initializer_list<ScalarType> kFloats = {ScalarType::Float, ScalarType::Half, ScalarType::BFloat16};
constexpr std::initializer_list<ScalarType> kF32 = {ScalarType::Float};
constexpr std::initializer_list<ScalarType> kByte = {ScalarType::Byte};

int code_of(ScalarType t) {
    switch (t) {
        case ScalarType::Float: return ROWOPS_F32;
        case ScalarType::Half: return ROWOPS_F16;
        case ScalarType::BFloat16: return ROWOPS_BF16;
        default: return -1;
    }
}
const char* name_of(ScalarType t) {
    switch (t) {
        case ScalarType::Float: return "torch.float32";
        case ScalarType::Half: return "torch.float16";
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Byte: return "torch.uint8";
        case ScalarType::Int: return "torch.int32";
        case ScalarType::Long: return "torch.int64";
        case ScalarType::Float8_e4m3fn: return "torch.float8_e4m3fn";
        default: return c10::toString(t);
    }
}
std::string text_of(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

// An argument that is not what it should be.
struct Wrong {
    PyObject* kind;
    std::string what;
};
[[noreturn]] void wrong_type(const std::string& what) { throw Wrong{PyExc_TypeError, what}; }
[[noreturn]] void wrong_value(const std::string& what) { throw Wrong{PyExc_ValueError, what}; }

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) wrong_type(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor& typed(PyObject* o, const char* name, std::initializer_list<ScalarType> types) {
    const at::Tensor& t = cuda_tensor(o, name);
    bool found = false;
    for (ScalarType s : types) found |= t.scalar_type() == s;
    if (!found) {
        std::string what = std::string(name) + " must be ";
        for (const ScalarType* s = types.begin(); s != types.end(); ++s) what += (s == types.begin() ? "" : " or ") + std::string(name_of(*s));
        wrong_type(what + ", got " + name_of(t.scalar_type()));
    }
    if (!t.is_contiguous()) wrong_value(std::string(name) + " must be contiguous");
    return t;
}
// And on the device of `like`, of `shape`.
const at::Tensor& typed(PyObject* o, const char* name, std::initializer_list<ScalarType> types, const at::Tensor& like) {
    const at::Tensor& t = typed(o, name, types);
    if (t.get_device() != like.get_device())
        wrong_value(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", not on cuda:" + std::to_string(like.get_device()));
    return t;
}
const at::Tensor& typed(PyObject* o, const char* name, std::initializer_list<ScalarType> types, const at::Tensor& like,
                        at::IntArrayRef shape) {
    const at::Tensor& t = typed(o, name, types, like);
    if (t.sizes() != shape)
        wrong_value(std::string(name) + " must have shape " + text_of(shape) + ", got " + text_of(t.sizes()));
    return t;
}
void dims(const at::Tensor& t, const char* name, int64_t n) {
    if (t.dim() != n)
        wrong_value(std::string(name) + " must have " + std::to_string(n) + " dimensions, got " + std::to_string(t.dim()));
}
ScalarType dtype_of(PyObject* o) {
    if (!THPDtype_Check(o)) wrong_type("dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

// An output: the caller's, checked, or a new one.
struct Output {
    PyObject* object;  // a reference of its own, until take()
    const at::Tensor* t;
    at::Tensor made;
    Output(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape, const at::Tensor& like) : object(o) {
        if (given(o)) {
            t = &typed(o, name, {type}, like, shape);
            Py_INCREF(o);
        } else {
            made = at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
            t = &made;
            object = nullptr;
        }
    }
    Output(const Output&) = delete;
    ~Output() { Py_XDECREF(object); }
    void* ptr() const { return t->data_ptr(); }
    PyObject* take() {  // a new reference
        if (object == nullptr) object = THPVariable_Wrap(made);
        PyObject* o = object;
        object = nullptr;
        return o;
    }
};

const void* at_or_null(PyObject* o, const char* name, std::initializer_list<ScalarType> types, const at::Tensor& like,
                       at::IntArrayRef shape) {
    return given(o) ? typed(o, name, types, like, shape).const_data_ptr() : nullptr;
}
const uint64_t* rng_of(PyObject* o, double p, const at::Tensor& like) {
    if (given(o)) return static_cast<const uint64_t*>(typed(o, "rng", {ScalarType::Long}, like, {2}).const_data_ptr());
    if (p != 0 && p != 1) wrong_value("rng is needed where values drop");
    return nullptr;
}
// rows, cols of a tensor whose last dimension is the columns
struct Rows {
    int64_t rows, cols;
    Shape lead;
    explicit Rows(const at::Tensor& t) : rows(1), cols(1) {
        const at::IntArrayRef s = t.sizes();
        if (s.empty()) return;
        cols = s.back();
        lead.assign(s.begin(), s.end() - 1);
        for (int64_t n : lead) rows *= n;
    }
    Shape with(int64_t last) const {
        Shape s = lead;
        s.push_back(last);
        return s;
    }
};
struct Workspace {
    at::Tensor made;
    void* p = nullptr;
    size_t bytes = 0;
    // the caller's, or a new one of `need` bytes where that is not 0
    Workspace(PyObject* o, size_t need, const at::Tensor& like) {
        if (given(o)) {
            if (!THPVariable_Check(o) || THPVariable_Unpack(o).device() != like.device())
                wrong_value("workspace must be a tensor on " + like.device().str());
            const at::Tensor& t = THPVariable_Unpack(o);
            if (!t.is_contiguous()) wrong_value("workspace must be contiguous");
            p = t.data_ptr();
            bytes = t.nbytes();
        } else if (need) {
            made = at::Tensor(at::detail::empty_cuda({int64_t(need)}, ScalarType::Byte, like.device(), std::nullopt));
            p = made.data_ptr();
            bytes = need;
        }
    }
};

rowops_stream stream_of(const at::Tensor& t) {
    return reinterpret_cast<rowops_stream>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}

// The C call without the interpreter's lock, as ctypes makes it.  What `f` throws (a tensor
// without storage has no address to give) passes on with the lock taken again.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F>
int call(F&& f) {
    const Unlocked unlocked;
    return f();
}
PyObject* tuple_of(std::initializer_list<PyObject*> items) {  // takes the references
    PyObject* t = PyTuple_New(Py_ssize_t(items.size()));
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}
PyObject* none() {
    Py_INCREF(Py_None);
    return Py_None;
}

PyObject* quantize_mx4(PyObject* const* a) {
    const at::Tensor& x = typed(a[0], "x", kFloats);
    if (x.dim() == 0) wrong_value("x must have columns");
    c10::cuda::CUDAGuard guard(x.device());
    const Rows r(x);
    Output q(a[1], "q", ScalarType::Byte, r.with((r.cols + 1) / 2), x);
    Output scale(a[2], "scale", ScalarType::Byte, r.with((r.cols + 31) / 32), x);
    const int status = call([&] {
        return lib.quantize_mx4(x.const_data_ptr(), static_cast<uint8_t*>(q.ptr()), static_cast<uint8_t*>(scale.ptr()), r.rows,
                                r.cols, code_of(x.scalar_type()), stream_of(x));
    });
    if (status) return PyLong_FromLong(status);
    return tuple_of({q.take(), scale.take()});
}

PyObject* expert_matmul_mx4(PyObject* const* a) {
    const at::Tensor& xq = typed(a[0], "xq", kByte);
    c10::cuda::CUDAGuard guard(xq.device());
    dims(xq, "xq", 2);
    const at::Tensor& wq = typed(a[2], "wq", kByte, xq);
    dims(wq, "wq", 3);
    const int64_t slots = xq.size(0), width = xq.size(1), experts = wq.size(0), out = wq.size(1), blocks = (width + 15) / 16;
    if (wq.size(2) != width)
        wrong_value("wq must have rows of " + std::to_string(width) + " bytes, got " + text_of(wq.sizes()));
    const at::Tensor& xs = typed(a[1], "xs", kByte, xq, {slots, blocks});
    const at::Tensor& ws = typed(a[3], "ws", kByte, xq, {experts, out, blocks});
    if (!given(a[4]) && experts != 1) wrong_value("offsets may be None for one expert only");
    const void* offsets = at_or_null(a[4], "offsets", {ScalarType::Int}, xq, {experts + 1});
    const ScalarType type = given(a[5]) ? typed(a[5], "y", kFloats, xq).scalar_type() : dtype_of(a[6]);
    Output y(a[5], "y", type, {slots, out}, xq);
    size_t need = 0;
    if (!given(a[7])) {
        // The library's function sees the widths alone; what starts off a 16-byte boundary
        // needs room for a copy too.
        const uintptr_t x_at = reinterpret_cast<uintptr_t>(xq.const_data_ptr()), w_at = reinterpret_cast<uintptr_t>(wq.const_data_ptr());
        if (width % 16) need = lib.matmul_mx4_workspace(slots, 2 * width, out, experts);
        else need = (x_at % 16 ? slots * width + 512 : 0) + (w_at % 16 ? experts * out * width + 512 : 0);
    }
    Workspace w(a[7], need, xq);
    const auto bytes = [](const at::Tensor& t) { return static_cast<const uint8_t*>(t.const_data_ptr()); };
    const int status = call([&] {
        return lib.matmul_mx4(bytes(xq), bytes(xs), bytes(wq), bytes(ws), static_cast<const int32_t*>(offsets), y.ptr(), slots,
                              2 * width, out, experts, code_of(type), w.p, w.bytes, stream_of(xq));
    });
    if (status) return PyLong_FromLong(status);
    return y.take();
}

PyObject* dropout(PyObject* const* a) {
    const at::Tensor& x = typed(a[0], "x", kFloats);
    c10::cuda::CUDAGuard guard(x.device());
    const double p = number(a[2]);
    const uint64_t* rng = rng_of(a[1], p, x);
    const ScalarType type = given(a[5])   ? dtype_of(a[5])
                            : given(a[4]) ? cuda_tensor(a[4], "y").scalar_type()
                            : given(a[3]) ? cuda_tensor(a[3], "residual").scalar_type()
                                          : x.scalar_type();
    const void* residual = at_or_null(a[3], "residual", {type}, x, x.sizes());
    Output y(a[4], "y", type, x.sizes(), x);
    const Rows r(x);
    const int status = call([&] {
        return lib.dropout(x.const_data_ptr(), residual, rng, y.ptr(), r.rows, r.cols, float(p), code_of(x.scalar_type()),
                           code_of(type), stream_of(x));
    });
    if (status) return PyLong_FromLong(status);
    return y.take();
}

PyObject* add_rmsnorm_fwd(PyObject* const* a) {
    const at::Tensor& x = typed(a[0], "x", kFloats);
    c10::cuda::CUDAGuard guard(x.device());
    const Rows r(x);
    const at::Tensor& gamma = typed(a[1], "gamma", kF32, x, {r.cols});
    const double p = number(a[4]), eps = number(a[5]);
    const uint64_t* rng = rng_of(a[3], p, x);
    const void* residual = at_or_null(a[2], "residual", kFloats, x, x.sizes());
    const ScalarType h_type = given(a[2])   ? THPVariable_Unpack(a[2]).scalar_type()
                              : given(a[9]) ? cuda_tensor(a[9], "h").scalar_type()
                                            : x.scalar_type();
    const bool h_is_x = !given(a[2]) && !given(a[9]) && p == 0;  // the sum is x
    std::optional<Output> h, scale;
    if (!h_is_x) h.emplace(a[9], "h", h_type, x.sizes(), x);
    int out_type = code_of(x.scalar_type());
    ScalarType type = x.scalar_type(), scale_type = ScalarType::Float;
    Shape wide(x.sizes().begin(), x.sizes().end()), blocks;
    if (given(a[6])) {
        const char* how = PyUnicode_Check(a[6]) ? PyUnicode_AsUTF8(a[6]) : "";
        if (std::string(how) == "e4m3") {
            out_type = ROWOPS_E4M3;
            type = ScalarType::Float8_e4m3fn;
            blocks = r.with((r.cols + 127) / 128);
        } else if (std::string(how) == "mx4") {
            out_type = ROWOPS_E2M1;
            type = scale_type = ScalarType::Byte;
            wide = r.with((r.cols + 1) / 2);
            blocks = r.with((r.cols + 31) / 32);
        } else {
            wrong_value("quantize must be None, \"e4m3\" or \"mx4\"");
        }
        scale.emplace(a[8], "scale", scale_type, blocks, x);
    } else if (given(a[8])) {
        wrong_value("scale is of quantised answers only");
    }
    Output out(a[7], "out", type, wide, x);
    Output row_rms(a[10], "row_rms", ScalarType::Float, r.lead, x);
    const int status = call([&] {
        return lib.norm_fwd(x.const_data_ptr(), residual, static_cast<const float*>(gamma.const_data_ptr()), rng,
                            h ? h->ptr() : nullptr, out.ptr(), scale ? scale->ptr() : nullptr,
                            static_cast<float*>(row_rms.ptr()), r.rows, r.cols, float(eps), float(p),
                            code_of(x.scalar_type()), code_of(h_type), out_type, stream_of(x));
    });
    if (status) return PyLong_FromLong(status);
    PyObject* sum = a[0];
    if (h) sum = h->take();
    else Py_INCREF(sum);
    return tuple_of({out.take(), scale ? scale->take() : none(), sum, row_rms.take()});
}

PyObject* add_rmsnorm_bwd(PyObject* const* a) {
    const at::Tensor& dy = typed(a[0], "dy", kFloats);
    c10::cuda::CUDAGuard guard(dy.device());
    const Rows r(dy);
    const at::Tensor& gamma = typed(a[1], "gamma", kF32, dy, {r.cols});
    const at::Tensor& h = typed(a[2], "h", kFloats, dy, dy.sizes());
    const at::Tensor& row_rms = typed(a[3], "row_rms", kF32, dy, r.lead);
    const double p = number(a[6]);
    const uint64_t* rng = rng_of(a[5], p, dy);
    const ScalarType h_type = h.scalar_type();
    const void* dh = at_or_null(a[4], "dh", {h_type}, dy, dy.sizes());
    Output dresidual(a[8], "dresidual", h_type, dy.sizes(), dy);
    const bool one = !given(a[7]) && p == 0 && dy.scalar_type() == h_type;  // dx is dresidual
    std::optional<Output> dx;
    if (!one) dx.emplace(a[7], "dx", dy.scalar_type(), dy.sizes(), dy);
    Output dgamma(a[9], "dgamma", ScalarType::Float, {r.cols}, dy);
    Workspace w(a[10], given(a[10]) ? 0 : lib.norm_bwd_workspace(r.rows, r.cols), dy);
    const auto floats = [](const at::Tensor& t) { return static_cast<const float*>(t.const_data_ptr()); };
    const int status = call([&] {
        return lib.norm_bwd(dy.const_data_ptr(), floats(gamma), h.const_data_ptr(), floats(row_rms), dh, rng, dresidual.ptr(),
                            dx ? dx->ptr() : nullptr, static_cast<float*>(dgamma.ptr()), r.rows, r.cols, float(p),
                            code_of(dy.scalar_type()), code_of(h_type), w.p, w.bytes, stream_of(dy));
    });
    if (status) return PyLong_FromLong(status);
    PyObject* res = dresidual.take();
    PyObject* first = res;
    if (dx) first = dx->take();
    else Py_INCREF(first);
    return tuple_of({first, res, dgamma.take()});
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments are wanted", N);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Wrong& w) {
        PyErr_SetString(w.kind, w.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// load(path): the library whose functions are called.
PyObject* load(PyObject*, PyObject* path) {
    const char* at = PyUnicode_AsUTF8(path);
    if (at == nullptr) return nullptr;
    void* so = dlopen(at, RTLD_NOW | RTLD_LOCAL);
    if (so == nullptr) {
        PyErr_Format(PyExc_RuntimeError, "%s: %s", at, dlerror());
        return nullptr;
    }
    bool all = true;
    const auto find = [&](auto& f, const char* name) {
        f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(so, name));
        if (f == nullptr && all) {
            all = false;
            PyErr_Format(PyExc_RuntimeError, "%s has no %s", at, name);
        }
    };
    find(lib.quantize_mx4, "rowops_quantize_mx4");
    find(lib.matmul_mx4_workspace, "rowops_expert_matmul_mx4_workspace");
    find(lib.matmul_mx4, "rowops_expert_matmul_mx4");
    find(lib.dropout, "rowops_dropout");
    find(lib.norm_fwd, "rowops_add_rmsnorm_fwd");
    find(lib.norm_bwd_workspace, "rowops_add_rmsnorm_bwd_workspace");
    find(lib.norm_bwd, "rowops_add_rmsnorm_bwd");
    return all ? none() : nullptr;
}

#define ROWOPS_ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ROWOPS_ENTRY(quantize_mx4, 3),
                         ROWOPS_ENTRY(expert_matmul_mx4, 8),
                         ROWOPS_ENTRY(dropout, 6),
                         ROWOPS_ENTRY(add_rmsnorm_fwd, 11),
                         ROWOPS_ENTRY(add_rmsnorm_bwd, 11),
                         {"load", load, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() { return PyModule_Create(&module); }
