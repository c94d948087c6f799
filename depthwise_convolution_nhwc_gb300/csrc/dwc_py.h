// dwc_py.h -- what the host paths of the operators for Python share (CPython C API over PyTorch's
// tensors): argument types, allocation, the current stream, errors.
#pragma once

#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <utility>

#include "../../include/dwc_norm.h"
#include "../../include/dwc_seq.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_error = nullptr;   // DwcError(function, code), given by norm.py

struct Failed {                // a status code of the library
    const char* fn;
    int code;
};

dwc_dtype_t code_of(ScalarType t) {
    switch (t) {
        case ScalarType::Float: return DWC_F32;
        case ScalarType::BFloat16: return DWC_BF16;
        case ScalarType::Half: return DWC_F16;
        default: TORCH_CHECK_TYPE(false, "unsupported dtype ", t, " (fp32, bf16 or fp16)");
    }
}

// "none", "sigmoid" or "silu".
dwc_gate_t gate_code(PyObject* o) {
    const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    if (s != nullptr && std::strcmp(s, "none") == 0) return DWC_GATE_NONE;
    if (s != nullptr && std::strcmp(s, "sigmoid") == 0) return DWC_GATE_SIGMOID;
    TORCH_CHECK_VALUE(s != nullptr && std::strcmp(s, "silu") == 0, "act must be \"none\", \"sigmoid\" or \"silu\"");
    return DWC_GATE_SILU;
}

const Tensor& tensor(PyObject* o, const char* what) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a tensor");
    return THPVariable_Unpack(o);
}

// A new dense tensor from PyTorch's allocator (the CUDA backend's own factory: the dispatcher's way
// to it costs as much again).
Tensor new_tensor(at::IntArrayRef shape, ScalarType type, const at::Device& device) {
    return Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

// The current stream of the tensors' device, with that device current.
struct OnDevice {
    c10::cuda::OptionalCUDAGuard guard;
    dwc_stream_t stream;
    explicit OnDevice(const Tensor& t) {
        const auto index = t.get_device();
        if (index != c10::cuda::current_device()) guard.set_index(index);
        stream = c10::cuda::getCurrentCUDAStream(index).stream();
    }
};

void check(const char* fn, dwc_status_t code) {
    if (code != DWC_OK) throw Failed{fn, static_cast<int>(code)};
}

PyObject* wrap(const Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

PyObject* pack(std::initializer_list<const Tensor*> list) {
    PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(list.size()));
    if (tuple == nullptr) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor* t : list) {
        PyObject* o = wrap(*t);
        if (o == nullptr) {
            Py_DECREF(tuple);
            return nullptr;
        }
        PyTuple_SET_ITEM(tuple, i++, o);
    }
    return tuple;
}

float* fp(const Tensor& t) { return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr; }

using Fast = PyObject* (*)(PyObject* const*);

// The common frame: the number of arguments, and every C++ exception as a Python one.
template <Fast f, int kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == kArgs, "expected ", kArgs, " arguments, got ", n);
    try {
        return f(a);
    } catch (const Failed& e) {
        if (PyObject* x = PyObject_CallFunction(g_error, "si", e.fn, e.code)) {
            PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(x)), x);
            Py_DECREF(x);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <Fast f, int kArgs>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, kArgs>)), METH_FASTCALL, nullptr};
}

}  // namespace
