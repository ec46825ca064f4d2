// Marshalling for the calls of a decode step.  A token's step makes several
// small launches a layer, each of a few microseconds, and reading a dozen
// tensors' shapes, types and addresses from Python costs more than that.  The
// checks here are those of the package's Python functions, on the tensors
// themselves; each function returns the library's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <array>
#include <cmath>

#include "rfp2.h"

namespace {

// A check that failed; the Python error is set.
struct Refused {};

[[noreturn]] void refuse(PyObject *kind, const char *what) {
    PyErr_SetString(kind, what);
    throw Refused{};
}
[[noreturn]] void refuse(PyObject *kind, const char *name, const char *what) {
    PyErr_Format(kind, "%s %s", name, what);
    throw Refused{};
}

// The tensor behind `o`, on the GPU that `device` names (-1: none yet, and then it
// has to be the current one, where the library launches).
const at::Tensor &tensor(PyObject *o, const char *name, int &device) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, "must be a CUDA tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(PyExc_TypeError, name, "must be a CUDA tensor");
    const int index = t.get_device();
    if (device < 0) {
        // (with one GPU there, that is 0)
        if ((index != 0 || c10::cuda::device_count() > 1) && index != c10::cuda::current_device())
            refuse(PyExc_ValueError, name, "must be on the current device");
        device = index;
    }
    if (index != device) refuse(PyExc_ValueError, name, "must be on the other tensors' device");
    return t;
}

const at::Tensor &array(PyObject *o, const char *name, at::ScalarType type, const char *type_name, int &device) {
    const at::Tensor &t = tensor(o, name, device);
    if (t.scalar_type() != type) {
        PyErr_Format(PyExc_TypeError, "%s must be %s", name, type_name);
        throw Refused{};
    }
    if (!t.is_contiguous()) refuse(PyExc_ValueError, name, "must be contiguous");
    return t;
}

// Activations of `dims` dimensions, the last contiguous.
const at::Tensor &rows(PyObject *o, const char *name, int dims, int &device) {
    const at::Tensor &t = tensor(o, name, device);
    if (t.dim() != dims) {
        PyErr_Format(PyExc_ValueError, "%s must have %d dimensions, got %d", name, dims, (int)t.dim());
        throw Refused{};
    }
    if (t.stride(dims - 1) != 1 && t.size(dims - 1) > 1)
        refuse(PyExc_ValueError, name, "must be contiguous in its last dimension");
    return t;
}

int type_code(const at::Tensor &t, const char *name) {
    switch (t.scalar_type()) {
        case at::kFloat: return RFP2_F32;
        case at::kBFloat16: return RFP2_BF16;
        case at::kHalf: return RFP2_F16;
        default: refuse(PyExc_TypeError, name, "must be float32, bfloat16 or float16");
    }
}

// A tensor that a call writes to: what autograd has kept of it is out of date.
void wrote(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

bool same_shape(const at::Tensor &a, const at::Tensor &b) { return a.sizes() == b.sizes(); }

int32_t *status_of(PyObject *o, int &device) {
    if (o == Py_None) return nullptr;
    return array(o, "dev_status", at::kInt, "torch.int32", device).data_ptr<int32_t>();
}

rfp2_stream_t stream_of(int device) {
    return reinterpret_cast<rfp2_stream_t>(
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
}

// The cache's four arrays, passed as one sequence.
struct Cache {
    PyObject *held;
    int8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    int64_t pages, heads, page_size, D;
    std::array<const at::Tensor *, 4> arrays;

    Cache(PyObject *o, int &device) : held(PySequence_Fast(o, "cache must be four tensors")) {
        if (!held) throw Refused{};
        try {
            if (PySequence_Fast_GET_SIZE(held) != 4) refuse(PyExc_ValueError, "cache must be four tensors");
            PyObject **at = PySequence_Fast_ITEMS(held);
            const at::Tensor &kc = array(at[0], "k_codes", at::kChar, "torch.int8", device);
            const at::Tensor &ks = array(at[1], "k_scales", at::kFloat, "torch.float32", device);
            const at::Tensor &vc = array(at[2], "v_codes", at::kChar, "torch.int8", device);
            const at::Tensor &vs = array(at[3], "v_scales", at::kFloat, "torch.float32", device);
            const auto fits = [&](const at::Tensor &s) {
                return s.dim() == 4 && s.size(0) == kc.size(0) && s.size(1) == kc.size(1) &&
                       s.size(2) == kc.size(2) && s.size(3) == kc.size(3) / 32;
            };
            if (kc.dim() != 4 || !same_shape(kc, vc) || !fits(ks) || !fits(vs))
                refuse(PyExc_ValueError,
                       "the cache's codes must be [pages, heads, page_size, D], its scales "
                       "[pages, heads, page_size, D/32]");
            arrays = {&kc, &ks, &vc, &vs};
            k_codes = kc.data_ptr<int8_t>();
            k_scales = ks.data_ptr<float>();
            v_codes = vc.data_ptr<int8_t>();
            v_scales = vs.data_ptr<float>();
            pages = kc.size(0);
            heads = kc.size(1);
            page_size = kc.size(2);
            D = kc.size(3);
        } catch (...) {
            Py_DECREF(held);
            throw;
        }
    }
    ~Cache() { Py_DECREF(held); }
    Cache(const Cache &) = delete;
};

// Python numbers; an error of the conversion is the call's.
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return v;
}
int64_t whole(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

// rope(x, positions, inv_freq, out, flags, factor)
int rope(PyObject *const *a) {
    int device = -1;
    const at::Tensor &x = rows(a[0], "x", 3, device);
    const int type = type_code(x, "x");
    const at::Tensor &positions = array(a[1], "positions", at::kInt, "torch.int32", device);
    const at::Tensor &inv_freq = array(a[2], "inv_freq", at::kFloat, "torch.float32", device);
    if (positions.numel() != x.size(0)) refuse(PyExc_ValueError, "positions needs one value per token");
    const at::Tensor &out = rows(a[3], "out", 3, device);
    if (!same_shape(out, x) || out.scalar_type() != x.scalar_type())
        refuse(PyExc_ValueError, "out must have x's shape and type");
    if (x.requires_grad() && at::GradMode::is_enabled())
        refuse(PyExc_RuntimeError, "x", "requires a gradient, which a call with out= does not give");
    wrote(out);
    return rfp2_rope(x.data_ptr(), type, x.size(0), x.size(1), x.size(2), x.stride(0), x.stride(1),
                     positions.data_ptr<int32_t>(), inv_freq.data_ptr<float>(), 2 * inv_freq.numel(),
                     (float)number(a[5]), (int)whole(a[4]), out.data_ptr(), out.stride(0), out.stride(1),
                     stream_of(device));
}

// kv_write(cache, k, v, slots, positions, inv_freq, flags, factor, dev_status)
int kv_write(PyObject *const *a) {
    int device = -1;
    const Cache c(a[0], device);
    const at::Tensor &k = rows(a[1], "k", 3, device);
    const at::Tensor &v = rows(a[2], "v", 3, device);
    const int type = type_code(k, "k");
    if (k.size(1) != c.heads || k.size(2) != c.D || !same_shape(k, v) || v.scalar_type() != k.scalar_type())
        refuse(PyExc_ValueError, "k and v must be [T, heads, D] of one type, as the cache has them");
    const at::Tensor &slots = array(a[3], "slots", at::kLong, "torch.int64", device);
    if (slots.numel() != k.size(0)) refuse(PyExc_ValueError, "slots needs one value per token");
    const int32_t *positions = nullptr;
    const float *inv_freq = nullptr;
    int64_t R = 0;
    if (a[4] != Py_None) {
        const at::Tensor &p = array(a[4], "positions", at::kInt, "torch.int32", device);
        if (p.numel() != k.size(0)) refuse(PyExc_ValueError, "positions needs one value per token");
        positions = p.data_ptr<int32_t>();
    }
    if (a[5] != Py_None) {
        const at::Tensor &f = array(a[5], "inv_freq", at::kFloat, "torch.float32", device);
        inv_freq = f.data_ptr<float>();
        R = 2 * f.numel();
    }
    if (R == 0 && a[4] != Py_None && a[5] != Py_None) {  // no pairs to turn
        positions = nullptr;
        inv_freq = nullptr;
    }
    for (const at::Tensor *t : c.arrays) wrote(*t);
    return rfp2_kv_write(k.data_ptr(), v.data_ptr(), type, k.size(0), k.stride(0), k.stride(1), v.stride(0),
                         v.stride(1), slots.data_ptr<int64_t>(), positions, inv_freq, R, (float)number(a[7]),
                         (int)whole(a[6]), c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.pages, c.heads,
                         c.page_size, c.D, status_of(a[8], device), stream_of(device));
}

// kv_read(cache, slots, k, v, dev_status)
int kv_read(PyObject *const *a) {
    int device = -1;
    const Cache c(a[0], device);
    const at::Tensor &slots = array(a[1], "slots", at::kLong, "torch.int64", device);
    const int64_t shape[3] = {slots.numel(), c.heads, c.D};
    const at::Tensor &k = tensor(a[2], "k", device);
    const at::Tensor &v = tensor(a[3], "v", device);
    const int type = type_code(k, "k");
    if (v.scalar_type() != k.scalar_type()) refuse(PyExc_TypeError, "v must have k's type");
    if (!k.is_contiguous() || !v.is_contiguous() || k.sizes() != at::IntArrayRef(shape, 3) || !same_shape(k, v))
        refuse(PyExc_ValueError, "k and v must be [T, heads, D] and contiguous");
    wrote(k);
    wrote(v);
    return rfp2_kv_read(c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.pages, c.heads, c.page_size, c.D,
                        slots.data_ptr<int64_t>(), slots.numel(), type, k.data_ptr(), v.data_ptr(),
                        status_of(a[4], device), stream_of(device));
}

// attn_decode(q, cache, table, lens, scale, window, softcap, out, lse, workspace, dev_status)
int attn_decode(PyObject *const *a) {
    int device = -1;
    const Cache c(a[1], device);
    const at::Tensor &q = rows(a[0], "q", 4, device);
    const int type = type_code(q, "q");
    const at::Tensor &lens = array(a[3], "lens", at::kInt, "torch.int32", device);
    const at::Tensor &table = rows(a[2], "table", 2, device);
    if (table.scalar_type() != at::kInt) refuse(PyExc_TypeError, "table must be torch.int32");
    const int64_t B = q.size(0), nq = q.size(1), Hq = q.size(2);
    if (q.size(3) != c.D || table.size(0) != B || lens.numel() != B)
        refuse(PyExc_ValueError, "q must be [B, nq, Hq, D] with the cache's D, table [B, width], lens [B]");
    const at::Tensor &out = tensor(a[7], "out", device);
    if (out.scalar_type() != q.scalar_type()) refuse(PyExc_TypeError, "out must have q's type");
    if (!same_shape(out, q) || !out.is_contiguous()) refuse(PyExc_ValueError, "out must have q's shape, contiguous");
    const at::Tensor &lse = array(a[8], "lse", at::kFloat, "torch.float32", device);
    if (lse.dim() != 3 || lse.size(0) != B || lse.size(1) != nq || lse.size(2) != Hq)
        refuse(PyExc_ValueError, "lse must be [B, nq, Hq]");
    const at::Tensor &workspace = array(a[9], "workspace", at::kByte, "torch.uint8", device);
    const int64_t width = table.size(1), stride = B > 1 ? table.stride(0) : std::max(table.stride(0), width);
    const double scale = a[4] == Py_None ? 1.0 / std::sqrt((double)c.D) : number(a[4]);
    if (B == 0) return RFP2_OK;  // no sequence, as rotation and cache take no token
    wrote(out);
    wrote(lse);
    return rfp2_attn_decode(q.data_ptr(), type, B, nq, Hq, c.D, q.stride(0), q.stride(1), q.stride(2), c.k_codes,
                            c.k_scales, c.v_codes, c.v_scales, c.pages, c.heads, c.page_size,
                            table.data_ptr<int32_t>(), width, stride, lens.data_ptr<int32_t>(), (float)scale,
                            whole(a[5]), (float)number(a[6]), out.data_ptr(), lse.data_ptr<float>(),
                            workspace.data_ptr(), (size_t)workspace.numel(), status_of(a[10], device),
                            stream_of(device));
}

template <int (*F)(PyObject *const *), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %d", N, (int)n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

#define RFP2_METHOD(name, n) {#name, reinterpret_cast<PyCFunction>(call<name, n>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {RFP2_METHOD(rope, 6), RFP2_METHOD(kv_write, 9), RFP2_METHOD(kv_read, 5),
                         RFP2_METHOD(attn_decode, 11), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rfp2_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rfp2_binding() { return PyModule_Create(&module); }
