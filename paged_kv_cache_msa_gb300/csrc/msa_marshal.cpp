// Torch tensors to C arguments, for the calls of a layer's input side (norm, adapters, the
// producer with several rotary axes): a CPython extension that checks the tensors and makes the C
// call.  In Python the checks of ten tensors take 7 to 14 us, more than the kernels of a small
// batch; here they take under one.
//
// Each function takes the address of the C entry point (the library is loaded by the binding), the
// configuration as a ctypes structure, the tensors (None where they are optional), the launch flags
// and the stream's handle (None: the current stream of the first tensor's device), and returns the
// entry point's status.  A tensor that does not fit is a ValueError.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <sstream>
#include <stdexcept>
#include <string>

#include "msa_adapter.h"
#include "msa_norm.h"
#include "msa_producer.h"

namespace {

struct BadArgument : std::runtime_error {       // becomes a ValueError
    using std::runtime_error::runtime_error;
};

struct PythonError {};                          // already set

enum class Kind { bf16, e4m3, f32, i32, i64 };

bool is(const at::Tensor &t, Kind kind)
{
    const at::ScalarType s = t.scalar_type();
    switch (kind) {
    case Kind::bf16: return s == at::kBFloat16 || s == at::kShort;       // or raw 16-bit words
    case Kind::e4m3: return s == at::kFloat8_e4m3fn || s == at::kByte;
    case Kind::f32: return s == at::kFloat;
    case Kind::i32: return s == at::kInt;
    case Kind::i64: return s == at::kLong;
    }
    return false;
}

const char *name_of(Kind kind)
{
    switch (kind) {
    case Kind::bf16: return "bfloat16";
    case Kind::e4m3: return "float8_e4m3fn";
    case Kind::f32: return "float32";
    case Kind::i32: return "int32";
    case Kind::i64: return "int64";
    }
    return "";
}

// nullptr for None
const at::Tensor *tensor(PyObject *o, const char *name)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        throw BadArgument(std::string(name) + ": expected a tensor");
    return &THPVariable_Unpack(o);
}

const at::Tensor &required(PyObject *o, const char *name)
{
    const at::Tensor *t = tensor(o, name);
    if (!t)
        throw BadArgument(std::string(name) + " is required");
    return *t;
}

[[noreturn]] void refuse(const char *name, const at::Tensor &t, Kind kind, at::IntArrayRef shape, const char *layout,
                         at::Device dev)
{
    std::ostringstream s;
    if (t.device() != dev)
        s << name << " is on " << t.device() << ", not on " << dev;
    else
        s << name << ": expected a " << name_of(kind) << " tensor of shape " << shape << ", " << layout << ", got "
          << t.scalar_type() << " " << t.sizes() << ", strides " << t.strides();
    throw BadArgument(s.str());
}

// The first tensor of a call: its device, a CUDA one.
at::Device device_of(const at::Tensor &t, const char *name)
{
    if (!t.is_cuda()) {
        std::ostringstream s;
        s << name << " is on " << t.device() << "; the calls take CUDA tensors";
        throw BadArgument(s.str());
    }
    return t.device();
}

// A contiguous tensor's address, nullptr for None.
void *dense(PyObject *o, const char *name, at::IntArrayRef shape, Kind kind, at::Device dev)
{
    const at::Tensor *t = tensor(o, name);
    if (!t)
        return nullptr;
    if (!is(*t, kind) || t->sizes() != shape || t->device() != dev || !t->is_contiguous())
        refuse(name, *t, kind, shape, "contiguous", dev);
    return t->data_ptr();
}

// n rows of k elements, any stride apart: address and stride (nullptr and 0 for None).
struct Rows {
    void *data = nullptr;
    int64_t stride = 0;
};

Rows rows(PyObject *o, const char *name, int64_t n, int64_t k, Kind kind, at::Device dev)
{
    const at::Tensor *t = tensor(o, name);
    if (!t)
        return {};
    if (!is(*t, kind) || t->dim() != 2 || t->size(0) != n || t->size(1) != k || t->device() != dev ||
        (t->stride(1) != 1 && k > 1))
        refuse(name, *t, kind, {n, k}, "unit column stride", dev);
    return {t->data_ptr(), n > 1 ? t->stride(0) : (k + 15) / 16 * 16};       // one row has no stride
}

template <class T>
struct Cfg {                                    // a ctypes structure's memory, None: nullptr
    Py_buffer view{};
    const T *ptr = nullptr;

    Cfg(PyObject *o, const char *name)
    {
        if (o == Py_None)
            return;
        if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0)
            throw PythonError();
        if (view.len != (Py_ssize_t)sizeof(T)) {
            PyBuffer_Release(&view);
            throw BadArgument(std::string(name) + ": not the structure of this call");
        }
        ptr = static_cast<const T *>(view.buf);
    }
    ~Cfg()
    {
        if (ptr)
            PyBuffer_Release(&view);
    }
    Cfg(const Cfg &) = delete;
    Cfg &operator=(const Cfg &) = delete;
};

template <class F>
F entry(PyObject *address)
{
    void *p = PyLong_AsVoidPtr(address);
    if (!p)
        throw BadArgument("no entry point");
    return reinterpret_cast<F>(p);
}

int flags_of(PyObject *o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred())
        throw PythonError();
    if (v < INT32_MIN || v > INT32_MAX)
        throw BadArgument("launch_flags: " + std::to_string(v));
    return (int)v;
}

cudaStream_t stream_of(PyObject *o, at::Device dev)
{
    if (o == Py_None)
        return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred())
        throw PythonError();
    return static_cast<cudaStream_t>(p);
}

// Runs `body` (which returns a status) and turns what it throws into Python's errors.
template <class F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t wanted, F body)
{
    if (got != wanted)
        return PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", got, wanted);
    try {
        return PyLong_FromLong(body());
    } catch (const PythonError &) {
        return nullptr;
    } catch (const BadArgument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <class F>
int call(at::Device dev, F f)                   // on the tensors' device, without Python's lock
{
    c10::cuda::CUDAGuard guard(dev);
    PyThreadState *s = PyEval_SaveThread();
    const int status = f();
    PyEval_RestoreThread(s);
    return status;
}

// entry, cfg, x, weight, residual, residual_out, out, codes, scales, flags, stream
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    return guarded(count, 11, [&]() -> int {
        auto f = entry<decltype(&msa_norm_forward)>(a[0]);
        Cfg<msa_norm_cfg> cfg(a[1], "cfg");
        const at::Tensor &x = required(a[2], "x");
        const at::Device dev = device_of(x, "x");
        const int64_t n = x.dim() > 0 ? x.size(0) : 0, k = cfg.ptr ? cfg.ptr->hidden_size : 0;
        const Rows xs = rows(a[2], "x", n, k, Kind::bf16, dev);
        void *w = dense(a[3], "weight", {k}, Kind::bf16, dev);
        const Rows r = rows(a[4], "residual", n, k, Kind::bf16, dev), ro = rows(a[5], "residual_out", n, k, Kind::bf16, dev);
        const Rows o = rows(a[6], "out", n, k, Kind::bf16, dev), c = rows(a[7], "codes", n, k, Kind::e4m3, dev);
        void *s = dense(a[8], "scales", {n}, Kind::f32, dev);
        const int flags = flags_of(a[9]);
        const cudaStream_t stream = stream_of(a[10], dev);
        return call(dev, [&] {
            return f(cfg.ptr, n, xs.data, xs.stride, r.data, r.stride, w, ro.data, ro.stride, o.data, o.stride, c.data,
                     c.stride, static_cast<float *>(s), flags, stream);
        });
    });
}

// entry, cfg, hidden, down, up, adapter_ids, rows, out, hidden_scales, adapter_scales, workspace, flags, stream
PyObject *adapter(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    return guarded(count, 13, [&]() -> int {
        auto f = entry<decltype(&msa_adapter_forward)>(a[0]);
        Cfg<msa_adapter_cfg> cfg(a[1], "cfg");
        if (!cfg.ptr || cfg.ptr->num_slices < 1 || cfg.ptr->num_slices > MSA_ADAPTER_MAX_SLICES)
            throw BadArgument("cfg: no slices");
        const msa_adapter_cfg &g = *cfg.ptr;
        const at::Tensor &x = required(a[2], "hidden"), &d = required(a[3], "down"), &ws = required(a[10], "workspace");
        const at::Device dev = device_of(x, "hidden");
        const int64_t n = x.dim() > 0 ? x.size(0) : 0, k = g.hidden_size, na = g.num_adapters;
        const int64_t sr = (int64_t)g.num_slices * g.rank, width = g.slice_end[g.num_slices - 1];
        const Rows h = rows(a[2], "hidden", n, k, g.hidden_dtype == MSA_DTYPE_BF16 ? Kind::bf16 : Kind::e4m3, dev);
        if (!is(d, Kind::bf16) || d.dim() != 3 || d.size(0) != na || d.size(1) != sr || d.size(2) != k ||
            d.device() != dev || (d.stride(2) != 1 && k > 1) || (na > 1 && d.stride(0) != sr * d.stride(1)))
            refuse("down", d, Kind::bf16, {na, sr, k}, "its rows one stride apart", dev);
        const int64_t down_stride = na * sr > 1 ? d.stride(1) : (k + 15) / 16 * 16;
        void *up = dense(a[4], "up", {na, width, g.rank}, Kind::bf16, dev);
        void *ids = dense(a[5], "adapter_ids", {n}, Kind::i32, dev);
        const Rows in = rows(a[6], "rows", n, width, Kind::bf16, dev), out = rows(a[7], "out", n, width, Kind::bf16, dev);
        void *hs = dense(a[8], "hidden_scales", {n}, Kind::f32, dev), *as = dense(a[9], "adapter_scales", {na}, Kind::f32, dev);
        if (ws.device() != dev || !ws.is_contiguous())
            throw BadArgument("workspace: expected a contiguous tensor on hidden's device");
        const int flags = flags_of(a[11]);
        const cudaStream_t stream = stream_of(a[12], dev);
        return call(dev, [&] {
            return f(cfg.ptr, n, h.data, h.stride, static_cast<const float *>(hs), d.data_ptr(), down_stride, up,
                     static_cast<const int32_t *>(ids), static_cast<const float *>(as), in.data, in.stride, out.data,
                     out.stride, ws.data_ptr(), (int64_t)ws.nbytes(), flags, stream);
        });
    });
}

// entry, cfg, axes, qkv, positions, slot_mapping, page_table, q_norm_w, k_norm_w, idx_q_norm_w,
// idx_k_norm_w, q_out, idx_q_out, k_cache, v_cache, idx_k_cache, scales, flags, stream
PyObject *producer_axes(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    return guarded(count, 19, [&]() -> int {
        auto f = entry<decltype(&msa_producer_axes_forward)>(a[0]);
        Cfg<msa_producer_cfg> cfg(a[1], "cfg");
        Cfg<msa_rope_axes> axes(a[2], "axes");
        if (!cfg.ptr || !axes.ptr)
            throw BadArgument("cfg and axes are required");
        const msa_producer_cfg &g = *cfg.ptr;
        const at::Tensor &x = required(a[3], "qkv"), &pos = required(a[4], "positions");
        const at::Device dev = device_of(x, "qkv");
        const int64_t n = x.dim() > 0 ? x.size(0) : 0, d = g.head_dim;
        const int64_t width = ((int64_t)g.num_q_heads + 2 * (int64_t)g.num_kv_heads + g.num_idx_q_heads + g.num_idx_k_heads) * d;
        if (!is(x, Kind::bf16) || x.dim() != 2 || x.size(1) < width || (x.stride(1) != 1 && x.size(1) > 1))
            refuse("qkv", x, Kind::bf16, {n, width}, "or wider, unit column stride", dev);
        if (!is(pos, Kind::i32) || pos.dim() != 2 || pos.size(0) != axes.ptr->num_axes || pos.size(1) != n ||
            pos.device() != dev || (n > 1 && pos.stride(1) != 1) || (pos.size(0) > 1 && n > 0 && pos.stride(0) < n))
            refuse("positions", pos, Kind::i32, {axes.ptr->num_axes, n}, "unit column stride", dev);
        void *slots = dense(a[5], "slot_mapping", {n}, Kind::i64, dev);
        const at::Tensor *table = tensor(a[6], "page_table");
        void *pages = table ? dense(a[6], "page_table", table->sizes(), Kind::i32, dev) : nullptr;
        static const char *const names[4] = {"q_norm_w", "k_norm_w", "idx_q_norm_w", "idx_k_norm_w"};
        void *w[4];
        for (int i = 0; i < 4; ++i)
            w[i] = dense(a[7 + i], names[i], {d}, Kind::bf16, dev);
        void *q = dense(a[11], "q_out", {n, g.num_q_heads, d}, Kind::bf16, dev);
        void *iq = dense(a[12], "idx_q_out", {n, g.num_idx_q_heads, d}, Kind::bf16, dev);
        Cfg<msa_cache_desc> kc(a[13], "k_cache"), vc(a[14], "v_cache"), ic(a[15], "idx_k_cache");
        const at::Tensor *scales = tensor(a[16], "scales");
        if (scales) {
            const int64_t ns = g.scale_mode == MSA_SCALE_PER_HEAD ? 2 * (int64_t)g.num_kv_heads + g.num_idx_k_heads : 3;
            if (scales->dim() != 1 || scales->size(0) < ns || !is(*scales, Kind::f32) || scales->device() != dev ||
                !scales->is_contiguous())
                refuse("scales", *scales, Kind::f32, {ns}, "or more, contiguous", dev);
        }
        const int flags = flags_of(a[17]);
        const cudaStream_t stream = stream_of(a[18], dev);
        return call(dev, [&] {
            return f(cfg.ptr, axes.ptr, n, x.data_ptr(), n > 1 ? x.stride(0) : (width + 7) / 8 * 8,
                     static_cast<const int32_t *>(pos.data_ptr()), pos.size(0) > 1 ? pos.stride(0) : n,
                     static_cast<const int64_t *>(slots), static_cast<const int32_t *>(pages), table ? table->numel() : 0,
                     w[0], w[1], w[2], w[3], q, iq, kc.ptr, vc.ptr, ic.ptr,
                     scales ? static_cast<const float *>(scales->data_ptr()) : nullptr, flags, stream);
        });
    });
}

PyMethodDef methods[] = {
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm)), METH_FASTCALL, nullptr},
    {"adapter", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(adapter)), METH_FASTCALL, nullptr},
    {"producer_axes", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(producer_axes)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "msa_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_msa_marshal() { return PyModule_Create(&module); }
