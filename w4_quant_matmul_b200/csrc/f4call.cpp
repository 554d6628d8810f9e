// f4call.cpp -- the plain calls of the f4_* Python functions, without the
// interpreter: the decode-sized operators take 2 to 6 us on the GPU, and checking
// tensors and marshalling a C call in Python takes longer than that (a call of
// f4_mm 11.5 us, f4_gemv 10.9; here 4.0 and 3.9).
//
// Every function takes what its Python namesake takes of a call with no output,
// workspace or stream of the caller's.  It makes the binding's checks -- plain
// CUDA tensors on the current device, types, exact shapes, contiguity -- and on
// anything else, or on a status other than W4_OK, returns None; the Python
// function then goes its own way, which says what is wrong.  Outputs come from
// torch's allocator on the current stream, past its dispatcher (0.4 us a tensor),
// which has nothing to add for a buffer that is written in full.  The C entry points are handed over as
// addresses, so that this module works on whichever libw4 is loaded.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "w4.h"

namespace {

struct Library {
    decltype(&f4_tensor_scale) tensor_scale = nullptr;
    decltype(&f4_quantize) quantize = nullptr;
    decltype(&f4_dequantize) dequantize = nullptr;
    decltype(&f4_embed) embed = nullptr;
    decltype(&f4_mm) mm = nullptr;
    decltype(&f4_gemv) gemv = nullptr;
    decltype(&f4_gemv_workspace_size) gemv_workspace_size = nullptr;
} lib;
PyObject* dtype_bf16 = nullptr;  // torch.bfloat16, torch.float32
PyObject* dtype_f32 = nullptr;

// The current device, -1 where there is none.
int current_device() { return c10::cuda::device_count() ? c10::cuda::current_device() : -1; }

// The tensor behind a Python object, if it is a plain contiguous CUDA tensor of
// this type on the device `dev`.
const at::Tensor* plain(PyObject* o, at::ScalarType type, int dev) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || t.scalar_type() != type ||
        t.get_device() != dev || !t.is_contiguous())
        return nullptr;
    return &t;
}

// The planes of one 4-bit matrix; g is None for MX.
struct Planes {
    const at::Tensor *codes, *scales, *g;
    int64_t rows, k;
    int format;
    const uint8_t* c() const { return codes->const_data_ptr<uint8_t>(); }
    const uint8_t* s() const { return scales->const_data_ptr<uint8_t>(); }
    const float* gp() const { return g ? g->const_data_ptr<float>() : nullptr; }
};

bool planes(Planes& p, PyObject* codes, PyObject* scales, PyObject* g, int dev) {
    p.codes = plain(codes, at::kByte, dev);
    p.scales = plain(scales, at::kByte, dev);
    p.g = nullptr;
    if (!p.codes || !p.scales || p.codes->dim() != 2 || p.scales->dim() != 3) return false;
    p.format = g == Py_None ? W4_F4_MX : W4_F4_NV;
    if (g != Py_None) {
        p.g = plain(g, at::kFloat, dev);
        if (!p.g || p.g->dim() != 1 || p.g->size(0) != 1) return false;
    }
    p.rows = p.codes->size(0);
    p.k = 2 * p.codes->size(1);
    const int64_t word = p.format == W4_F4_MX ? 128 : 64;  // k of a scale word
    return p.k % 32 == 0 && p.scales->size(0) == (p.rows + 127) / 128 &&
           p.scales->size(1) == (p.k + word - 1) / word && p.scales->size(2) == 512;
}

// out_dtype: None, torch.bfloat16 or torch.float32.
bool out_type(PyObject* o, int& code, at::ScalarType& type) {
    const bool f32 = o == dtype_f32;
    if (!f32 && o != dtype_bf16 && o != Py_None) return false;
    code = f32 ? W4_OUT_F32 : W4_OUT_BF16;
    type = f32 ? at::kFloat : at::kBFloat16;
    return true;
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

void* stream(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// f4_tensor_scale takes any of these; returns the in_dtype code or -1.
int in_type(PyObject* o, int dev, const at::Tensor*& t) {
    constexpr std::pair<at::ScalarType, int> types[] = {
        {at::kBFloat16, W4_IN_BF16}, {at::kFloat, W4_IN_F32}, {at::kHalf, W4_IN_F16}};
    for (const auto& [type, code] : types)
        if ((t = plain(o, type, dev)) && t->dim() == 2) return code;
    return -1;
}

PyObject* none() { Py_RETURN_NONE; }

// quantize(x, format, tensor_scale or None) -> (codes, scales, g)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 3) return none();
    const int dev = current_device();
    const at::Tensor* x = nullptr;
    const int in = in_type(a[0], dev, x);
    const long format = PyLong_AsLong(a[1]);
    if (in < 0 || (format != W4_F4_MX && format != W4_F4_NV)) return none();
    const int64_t R = x->size(0), K = x->size(1);
    if (K % 32 != 0) return none();
    at::Tensor g;
    bool find = false;
    if (format == W4_F4_NV) {
        if (a[2] != Py_None) {
            const at::Tensor* given = plain(a[2], at::kFloat, dev);
            if (!given || given->dim() != 1 || given->size(0) != 1) return none();
            g = *given;
        } else {
            g = make({1}, at::kFloat, *x);
            find = true;
        }
    } else if (a[2] != Py_None) {
        return none();
    }
    const int64_t word = format == W4_F4_MX ? 128 : 64;
    at::Tensor codes = make({R, K / 2}, at::kByte, *x);
    at::Tensor scales = make({(R + 127) / 128, (K + word - 1) / word, 512}, at::kByte, *x);
    void* st = stream(dev);
    float* gp = g.defined() ? static_cast<float*>(g.data_ptr()) : nullptr;
    if (find && lib.tensor_scale(x->const_data_ptr(), in, R, K, gp, st) != W4_OK) return none();
    if (lib.quantize(x->const_data_ptr(), in, R, K, (int)format, gp,
                     static_cast<uint8_t*>(codes.data_ptr()),
                     static_cast<uint8_t*>(scales.data_ptr()), st) != W4_OK)
        return none();
    PyObject* out = PyTuple_New(3);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(codes));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(scales));
    PyObject* go = find ? THPVariable_Wrap(g) : a[2];
    if (!find) Py_INCREF(go);
    PyTuple_SET_ITEM(out, 2, go);
    return out;
    END_HANDLE_TH_ERRORS
}

// dequantize(codes, scales, g, out_dtype) -> y
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 4) return none();
    const int dev = current_device();
    Planes w;
    int out;
    at::ScalarType type;
    if (!planes(w, a[0], a[1], a[2], dev) || !out_type(a[3], out, type)) return none();
    at::Tensor y = make({w.rows, w.k}, type, *w.codes);
    if (lib.dequantize(w.c(), w.s(), w.gp(), w.rows, w.k, w.format, y.data_ptr(), out, stream(dev)) !=
        W4_OK)
        return none();
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// embed(codes, scales, g, ids, scale, out_dtype) -> y
PyObject* embed(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 6) return none();
    const int dev = current_device();
    Planes w;
    int out;
    at::ScalarType type;
    const at::Tensor* ids = plain(a[3], at::kLong, dev);
    if (!planes(w, a[0], a[1], a[2], dev) || !ids || ids->dim() != 1 || !out_type(a[5], out, type))
        return none();
    const double scale = PyFloat_AsDouble(a[4]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    const int64_t T = ids->size(0);
    at::Tensor y = make({T, w.k}, type, *w.codes);
    if (lib.embed(w.c(), w.s(), w.gp(), w.rows, w.k, w.format, ids->const_data_ptr<int64_t>(), T,
                  (float)scale, y.data_ptr(), out, stream(dev)) != W4_OK)
        return none();
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// mm(codes, scales, g, qa, sa, ga, out_dtype) -> y
PyObject* mm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) return none();
    const int dev = current_device();
    Planes w, q;
    int out;
    at::ScalarType type;
    if (!planes(w, a[0], a[1], a[2], dev) || !planes(q, a[3], a[4], a[5], dev) || q.k != w.k ||
        q.format != w.format || !out_type(a[6], out, type))
        return none();
    at::Tensor y = make({q.rows, w.rows}, type, *w.codes);
    if (lib.mm(w.c(), w.s(), w.gp(), w.rows, w.k, w.format, q.c(), q.s(), q.gp(), q.rows, y.data_ptr(),
               out, stream(dev)) != W4_OK)
        return none();
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// gemv(codes, scales, g, x, out_dtype) -> y
PyObject* gemv(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5) return none();
    const int dev = current_device();
    Planes w;
    int out;
    at::ScalarType type;
    const at::Tensor* x = plain(a[3], at::kBFloat16, dev);
    if (!planes(w, a[0], a[1], a[2], dev) || !x || x->dim() != 2 || x->size(1) != w.k ||
        x->size(0) > 8 || !out_type(a[4], out, type))
        return none();
    const int64_t M = x->size(0);
    const size_t bytes = lib.gemv_workspace_size(M, w.rows, w.k, w.format);
    at::Tensor y = make({M, w.rows}, type, *w.codes), ws;
    if (bytes) ws = make({(int64_t)bytes}, at::kByte, *x);
    if (lib.gemv(w.c(), w.s(), w.gp(), w.rows, w.k, w.format,
                 static_cast<const uint16_t*>(x->const_data_ptr()), (int)M, y.data_ptr(), out,
                 bytes ? ws.data_ptr() : nullptr, bytes, stream(dev)) != W4_OK)
        return none();
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// init(address of f4_tensor_scale, f4_quantize, f4_dequantize, f4_embed, f4_mm,
// f4_gemv, f4_gemv_workspace_size, torch.bfloat16, torch.float32)
PyObject* init(PyObject*, PyObject* args) {
    unsigned long long p[7];
    PyObject *bf16, *f32;
    if (!PyArg_ParseTuple(args, "KKKKKKKOO", &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6], &bf16,
                          &f32))
        return nullptr;
    lib.tensor_scale = reinterpret_cast<decltype(lib.tensor_scale)>(p[0]);
    lib.quantize = reinterpret_cast<decltype(lib.quantize)>(p[1]);
    lib.dequantize = reinterpret_cast<decltype(lib.dequantize)>(p[2]);
    lib.embed = reinterpret_cast<decltype(lib.embed)>(p[3]);
    lib.mm = reinterpret_cast<decltype(lib.mm)>(p[4]);
    lib.gemv = reinterpret_cast<decltype(lib.gemv)>(p[5]);
    lib.gemv_workspace_size = reinterpret_cast<decltype(lib.gemv_workspace_size)>(p[6]);
    Py_INCREF(bf16);
    Py_INCREF(f32);
    Py_XSETREF(dtype_bf16, bf16);
    Py_XSETREF(dtype_f32, f32);
    Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Fast f) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL,
            nullptr};
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, nullptr}, method("quantize", quantize),
    method("dequantize", dequantize),      method("embed", embed),
    method("mm", mm),                      method("gemv", gemv),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_f4call", nullptr, -1, methods};

}  // namespace

// built_for: the torch and the Python of this build; the binding calls nothing else of
// a module that was built for others.
PyMODINIT_FUNC PyInit__f4call() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", W4_BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
