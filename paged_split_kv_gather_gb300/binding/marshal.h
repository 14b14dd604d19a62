// marshal.h -- what the compiled bindings share: reading tensors, sizes and streams from
// Python objects, running a call on the device of its tensors, exceptions.
#pragma once

#include <cstdint>
#include <stdexcept>
#include <string>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/fdec.h"

namespace {

using Tensor = at::Tensor;

struct Bad : std::runtime_error {  // -> ValueError
    using std::runtime_error::runtime_error;
};

void need(bool ok, const char* message) {
    if (!ok) throw Bad(message);
}

const Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw Bad(std::string(what) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// A tensor or None (an undefined tensor).
Tensor maybe(PyObject* o, const char* what) { return o == Py_None ? Tensor() : tensor(o, what); }

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Bad("");
    return v;
}

int small(PyObject* o, const char* what) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) throw Bad(std::string(what) + " does not fit 32 bits");
    return static_cast<int>(v);
}

float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Bad("");
    return static_cast<float>(v);
}

// The stream given, or the current one of the tensors' device.
cudaStream_t stream_of(PyObject* o, c10::Device device) {
    if (o == Py_None) return device.is_cuda() ? c10::cuda::getCurrentCUDAStream(device.index()).stream() : nullptr;
    if (PyLong_Check(o)) return reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(o));
    PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
    if (handle == nullptr) throw Bad("");
    void* s = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    return static_cast<cudaStream_t>(s);
}

fdec_dtype dtype_of(const Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return FDEC_BF16;
    if (t.scalar_type() == at::kHalf) return FDEC_F16;
    throw Bad(std::string("expected bfloat16 or float16, got ") + c10::toString(t.scalar_type()));
}

// FDEC_KV_SAME for a cache of the 16-bit type, FDEC_KV_E4M3 for one of 1-byte codes.
int kv_of(const Tensor& t, at::ScalarType type) {
    if (t.scalar_type() == type) return FDEC_KV_SAME;
    if (t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte) return FDEC_KV_E4M3;
    throw Bad(std::string("expected a cache of the 16-bit type or of E4M3 codes, got ") + c10::toString(t.scalar_type()));
}

int as_int(int64_t v) {
    need(v <= INT32_MAX, "a size does not fit 32 bits");
    return static_cast<int>(v);
}

// The stride of a dimension; 0 for one of a single index, whose stride may be anything.
int64_t step(const Tensor& t, int dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

// Entries between two rows of a page table.
int64_t table_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

fdec_kv_desc pool(const Tensor& t) {
    need(t.dim() == 4 && t.stride(3) == 1, "caches must be 4-D [page, kv_head, slot, dim] with a unit dim stride");
    return {t.data_ptr(), t.size(0), step(t, 0), step(t, 1), step(t, 2)};
}

fdec_rows rows(const Tensor& t) {
    need(t.dim() == 3 && t.stride(2) == 1, "rows must be [n, heads, head_dim] with a unit dim stride");
    return {t.data_ptr(), step(t, 0), step(t, 1)};
}

const int32_t* index(const Tensor& t, int64_t dim, const char* what) {
    if (t.scalar_type() != at::kInt || t.dim() != dim || (t.numel() > 0 && t.stride(dim - 1) != 1))
        throw Bad(std::string(what) + " must be an int32 tensor with contiguous rows, of " + std::to_string(dim) +
                  " dimension(s)");
    return static_cast<const int32_t*>(t.data_ptr());
}

void on(const Tensor& first, std::initializer_list<const Tensor*> others) {
    for (const Tensor* t : others)
        if (t->defined() && t->device() != first.device())
            throw Bad("tensors on " + first.device().str() + " and " + t->device().str());
}

uint32_t* error_word(const Tensor& t) {
    if (!t.defined()) return nullptr;
    need(t.element_size() == 4 && t.numel() >= 1, "device_errors must hold one 32-bit value");
    return static_cast<uint32_t*>(t.data_ptr());
}

// Token and head strides of q [B, Q, Hq, D], tokens flattened.
void q_strides(const Tensor& q, int64_t* tok, int64_t* head) {
    need(q.dim() == 4 && q.stride(3) == 1, "q must be [B, Q, Hq, D] with a unit head_dim stride");
    if (q.size(1) == 1) {
        *tok = step(q, 0);
    } else {
        need(q.size(0) <= 1 || q.stride(0) == q.size(1) * q.stride(1), "q tokens must flatten to one stride (b*q_len + i)");
        *tok = q.stride(1);
    }
    *head = step(q, 2);
}

void (*g_checks_only)(int) = nullptr;
constexpr int kChecksOnly = -1;  // the status of a call that has passed its checks and launched nothing

// The library call f(stream) on the device of its tensors.  Tensors that are not on a GPU
// go through its checks, which touch no element, and are refused where it would launch.
template <typename F>
fdec_status on_device(const Tensor& t, PyObject* stream, F&& f) {
    const cudaStream_t s = stream_of(stream, t.device());
    if (t.is_cuda()) {
        const c10::cuda::CUDAGuard guard(t.device());
        return f(s);
    }
    struct ChecksOnly {
        ChecksOnly() { g_checks_only(1); }
        ~ChecksOnly() { g_checks_only(0); }
    };
    const fdec_status st = [&] {
        const ChecksOnly scope;
        return f(s);
    }();
    need(static_cast<int>(st) != kChecksOnly, "tensors must be on a CUDA device");
    return st;
}

// Run f() -> status; C++ exceptions become Python ones.
template <typename F>
PyObject* guarded(F&& f) {
    try {
        return PyLong_FromLong(static_cast<long>(f()));
    } catch (const Bad& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

bool has(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// A function of n arguments as a method table's entry.
#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}

}  // namespace
