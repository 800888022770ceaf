// The Python binding's native half: argument checks and marshalling of the
// calls over block-scaled pools, straight from torch tensors to the C ABI in
// pa.h.  A serving step makes several such calls, each over ten tensors or so;
// checked and unpacked in Python that cost 18 us a call, four times the C call
// itself and twice the small kernels.
//
// Every function takes its arguments by position (__init__.py gives them
// their names), runs on the tensors' device and, where no stream is given, on
// that device's current stream, and returns the call's pa_status.  A bad
// argument raises TypeError or ValueError; no C++ exception leaves this file.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>
#include <string>

#include "pa.h"

namespace {

struct BadArgument {
    PyObject *type;
    std::string what;
};
[[noreturn]] void type_error(const std::string &what) { throw BadArgument{PyExc_TypeError, what}; }
[[noreturn]] void value_error(const std::string &what) { throw BadArgument{PyExc_ValueError, what}; }
struct PythonError {};   // a Python exception is already set

// The tensors of one call: each a CUDA tensor, all on one device.
class Call {
  public:
    const at::Tensor &tensor(PyObject *o, const char *name) {
        if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
        const int dev = t.get_device();
        if (device_ < 0) device_ = dev;
        else if (dev != device_)
            value_error(std::string(name) + " is on cuda:" + std::to_string(dev) +
                        ", the tensors before it on cuda:" + std::to_string(device_));
        return t;
    }
    const at::Tensor &contiguous(PyObject *o, const char *name) {
        const at::Tensor &t = tensor(o, name);
        if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
        return t;
    }
    const at::Tensor &typed(PyObject *o, const char *name, at::ScalarType type) {
        const at::Tensor &t = contiguous(o, name);
        if (t.scalar_type() != type)
            type_error(std::string(name) + " must be " + c10::toString(type) + ", got " +
                       c10::toString(t.scalar_type()));
        return t;
    }
    int device() const { return device_; }

  private:
    int device_ = -1;
};

int32_t size32(const at::Tensor &t, int dim, const char *name) {
    const int64_t n = t.size(dim);
    if (n > INT32_MAX) value_error(std::string(name) + " is too large");
    return (int32_t)n;
}

int32_t int_arg(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    if (v > INT32_MAX || v < INT32_MIN) value_error(std::string(name) + " is out of range");
    return (int32_t)v;
}

// A stream argument: None (the device's current stream), an object with a
// cuda_stream, or the handle itself.
pa_stream_t stream_of(PyObject *o, int device) {
    if (o == Py_None)
        return reinterpret_cast<pa_stream_t>(
            c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    PyObject *h = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream")
                                                           : PyNumber_Long(o);
    if (!h) throw PythonError{};
    void *p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw PythonError{};
    return reinterpret_cast<pa_stream_t>(p);
}

bool is_fp8(const at::Tensor &t) {
    return t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn;
}

pa_dtype element_type(const at::Tensor &a, const at::Tensor &b, const char *names) {
    if (a.scalar_type() != b.scalar_type() ||
        (a.scalar_type() != at::kBFloat16 && a.scalar_type() != at::kHalf))
        type_error(std::string(names) + " must share a bf16/fp16 dtype");
    return a.scalar_type() == at::kBFloat16 ? PA_BF16 : PA_FP16;
}

// Both pools [NB, bs, Hkv, D] and, where they are given, both tables [NB, Hkv].
struct Pools {
    void *kc, *vc;
    uint8_t *ks = nullptr, *vs = nullptr;
    int32_t nb, bs, hkv, d;
    pa_dtype dtype;

    Pools(Call &c, PyObject *k, PyObject *v) {
        const at::Tensor &kt = c.contiguous(k, "key_cache"), &vt = c.contiguous(v, "value_cache");
        if (kt.dim() != 4 || kt.sizes() != vt.sizes())
            value_error("key/value caches must both be [NB, bs, Hkv, D]");
        if (is_fp8(kt) && is_fp8(vt)) dtype = PA_FP8_E4M3;
        else if (kt.scalar_type() == vt.scalar_type() && kt.scalar_type() == at::kBFloat16) dtype = PA_BF16;
        else if (kt.scalar_type() == vt.scalar_type() && kt.scalar_type() == at::kHalf) dtype = PA_FP16;
        else type_error("caches must share a bf16/fp16/FP8 dtype");
        nb = size32(kt, 0, "key_cache");
        bs = size32(kt, 1, "key_cache");
        hkv = size32(kt, 2, "key_cache");
        d = size32(kt, 3, "key_cache");
        kc = kt.data_ptr();
        vc = vt.data_ptr();
    }
    void tables(Call &c, PyObject *k, PyObject *v) {
        if (dtype != PA_FP8_E4M3) type_error("block scales belong to FP8 pools (uint8/float8_e4m3fn)");
        ks = table(c, k, "k_scales");
        vs = table(c, v, "v_scales");
    }

  private:
    uint8_t *table(Call &c, PyObject *o, const char *name) {
        const at::Tensor &t = c.typed(o, name, at::kByte);
        if (t.dim() != 2 || t.size(0) != nb || t.size(1) != hkv)
            value_error(std::string(name) + " must be [" + std::to_string(nb) + ", " +
                        std::to_string(hkv) + "] (blocks, kv heads)");
        return static_cast<uint8_t *>(t.data_ptr());
    }
};

// block_table [R, MB], starts [R + 1] and lens [R].
struct Batch {
    const int32_t *bt, *starts, *lens;
    int32_t r, mb;
    Batch(Call &c, PyObject *table, PyObject *s, const char *s_name, PyObject *l, const char *l_name) {
        const at::Tensor &t = c.typed(table, "block_table", at::kInt);
        const at::Tensor &st = c.typed(s, s_name, at::kInt), &lt = c.typed(l, l_name, at::kInt);
        if (t.dim() != 2 || st.dim() != 1 || lt.dim() != 1 || t.size(0) != lt.size(0) ||
            st.size(0) != lt.size(0) + 1)
            value_error(std::string("block_table [R, MB], ") + s_name + " [R + 1] and " + l_name +
                        " [R] must agree on R");
        r = size32(lt, 0, l_name);
        mb = size32(t, 1, "block_table");
        bt = static_cast<const int32_t *>(t.data_ptr());
        starts = static_cast<const int32_t *>(st.data_ptr());
        lens = static_cast<const int32_t *>(lt.data_ptr());
    }
};

// A [rows, heads, d] tensor's shape.
void need_rows(const at::Tensor &a, const at::Tensor &b, int32_t heads, int32_t d, const char *names) {
    if (a.dim() != 3 || a.size(1) != heads || a.size(2) != d || a.sizes() != b.sizes())
        value_error(std::string(names) + " must both be [rows, " + std::to_string(heads) + ", " +
                    std::to_string(d) + "]");
}

const float *pool_scale(Call &c, PyObject *o, const char *name) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = c.tensor(o, name);
    if (t.scalar_type() != at::kFloat || t.numel() != 1)
        type_error(std::string(name) + " must be a one-element float32 CUDA tensor");
    return static_cast<const float *>(t.data_ptr());
}

// Runs `body` (which returns a pa_status) with C++ exceptions turned into
// Python ones.
template <typename F>
PyObject *guarded(const char *fn, Py_ssize_t given, Py_ssize_t wanted, F body) {
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", fn, wanted, given);
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)body());
    } catch (const PythonError &) {
    } catch (const BadArgument &e) {
        PyErr_SetString(e.type, e.what.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_Format(PyExc_RuntimeError, "%s failed", fn);
    }
    return nullptr;
}

// key, value, key_cache, value_cache, k_scales, v_scales, block_table,
// query_start_loc, seq_lens, stream
PyObject *cache_write_scaled(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("cache_write_scaled", n, 10, [&]() -> pa_status {
        Call c;
        const at::Tensor &key = c.tensor(a[0], "key"), &value = c.tensor(a[1], "value");
        Pools p(c, a[2], a[3]);
        p.tables(c, a[4], a[5]);
        const pa_dtype dt = element_type(key, value, "key and value");
        need_rows(key, value, p.hkv, p.d, "key and value");
        const int32_t t = size32(key, 0, "key");
        int64_t stride = (int64_t)p.hkv * p.d;
        if (t > 0) {
            for (const at::Tensor *x : {&key, &value})
                if ((p.hkv > 1 && x->stride(1) != p.d) || (p.d > 1 && x->stride(2) != 1))
                    value_error("key/value rows must be [Hkv, D]-contiguous");
            if (t > 1) {
                if (key.stride(0) != value.stride(0))
                    value_error("key and value must have equal token strides");
                stride = key.stride(0);
            }
        }
        const Batch b(c, a[6], a[7], "query_start_loc", a[8], "seq_lens");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device());
        const pa_stream_t st = stream_of(a[9], c.device());
        return pa_cache_write_scaled(key.data_ptr(), value.data_ptr(), stride, p.kc, p.vc, p.ks, p.vs,
                                     b.bt, b.mb, b.starts, b.lens, b.r, t, p.hkv, p.d, p.bs, p.nb, dt,
                                     st);
    });
}

// key_cache, value_cache, block_table, first_positions, row_start_loc,
// key_out, value_out, k_scales, v_scales, k_scale, v_scale, stream
PyObject *cache_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("cache_read", n, 12, [&]() -> pa_status {
        Call c;
        Pools p(c, a[0], a[1]);
        if (a[7] != Py_None || a[8] != Py_None) p.tables(c, a[7], a[8]);
        const Batch b(c, a[2], a[4], "row_start_loc", a[3], "first_positions");
        const at::Tensor &ko = c.contiguous(a[5], "key_out"), &vo = c.contiguous(a[6], "value_out");
        const pa_dtype dt = element_type(ko, vo, "key_out and value_out");
        need_rows(ko, vo, p.hkv, p.d, "key_out and value_out");
        const float *k1 = pool_scale(c, a[9], "k_scale"), *v1 = pool_scale(c, a[10], "v_scale");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device());
        const pa_stream_t st = stream_of(a[11], c.device());
        return pa_cache_read(p.kc, p.vc, p.dtype, k1, v1, p.ks, p.vs, b.bt, b.mb, b.lens, b.starts, b.r,
                             size32(ko, 0, "key_out"), p.hkv, p.d, p.bs, p.nb, ko.data_ptr(),
                             vo.data_ptr(), dt, st);
    });
}

// key_cache, value_cache, k_scales, v_scales, src_blocks, dst_blocks, stream
PyObject *copy_blocks_scaled(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("copy_blocks_scaled", n, 7, [&]() -> pa_status {
        Call c;
        Pools p(c, a[0], a[1]);
        p.tables(c, a[2], a[3]);
        const at::Tensor &src = c.typed(a[4], "src_blocks", at::kInt);
        const at::Tensor &dst = c.typed(a[5], "dst_blocks", at::kInt);
        if (src.dim() != 1 || src.sizes() != dst.sizes())
            value_error("src_blocks and dst_blocks must be 1-D of equal length");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device());
        const pa_stream_t st = stream_of(a[6], c.device());
        return pa_copy_blocks_scaled(p.kc, p.vc, p.ks, p.vs, static_cast<int32_t *>(src.data_ptr()),
                                     static_cast<int32_t *>(dst.data_ptr()),
                                     size32(src, 0, "src_blocks"), p.bs, p.hkv, p.d, p.nb, st);
    });
}

// q, key_cache, value_cache, k_scales, v_scales, block_table, query_start_loc,
// seq_lens, max_query_len, max_seq_len, scale, out, workspace, stream, flags
PyObject *attention_scaled(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("attention_scaled", n, 15, [&]() -> pa_status {
        Call c;
        const at::Tensor &q = c.contiguous(a[0], "q");
        Pools p(c, a[1], a[2]);
        p.tables(c, a[3], a[4]);
        const at::Tensor &out = c.contiguous(a[11], "out");
        const pa_dtype dt = element_type(q, out, "q and out");
        if (q.dim() != 3) value_error("q and out must both be [T, Hq, D]");
        need_rows(q, out, size32(q, 1, "q"), p.d, "q and out");
        const Batch b(c, a[5], a[6], "query_start_loc", a[7], "seq_lens");
        const int32_t max_q = int_arg(a[8], "max_query_len"), max_seq = int_arg(a[9], "max_seq_len");
        const double scale = PyFloat_AsDouble(a[10]);
        if (scale == -1.0 && PyErr_Occurred()) throw PythonError{};
        void *ws = nullptr;
        size_t ws_bytes = 0;
        if (a[12] != Py_None) {
            const at::Tensor &w = c.contiguous(a[12], "workspace");
            ws_bytes = (size_t)w.numel() * w.element_size();
            if (ws_bytes) ws = w.data_ptr();
        }
        const unsigned long flags = PyLong_AsUnsignedLong(a[14]);
        if (flags == (unsigned long)-1 && PyErr_Occurred()) throw PythonError{};
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device());
        const pa_stream_t st = stream_of(a[13], c.device());
        return pa_attention_scaled(q.data_ptr(), p.kc, p.vc, p.ks, p.vs, b.bt, b.mb, b.starts, b.lens,
                                   b.r, size32(q, 0, "q"), max_q, max_seq, size32(q, 1, "q"), p.hkv,
                                   p.d, p.bs, p.nb, (float)scale, dt, (uint32_t)flags, out.data_ptr(),
                                   ws, ws_bytes, st);
    });
}

#define PA_FASTCALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef methods[] = {
    {"cache_write_scaled", PA_FASTCALL(cache_write_scaled), METH_FASTCALL, nullptr},
    {"cache_read", PA_FASTCALL(cache_read), METH_FASTCALL, nullptr},
    {"copy_blocks_scaled", PA_FASTCALL(copy_blocks_scaled), METH_FASTCALL, nullptr},
    {"attention_scaled", PA_FASTCALL(attention_scaled), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
