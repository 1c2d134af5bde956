// tensor_calls.cpp -- the binding's calls that a serving loop makes for every
// layer of every step, on torch tensors: argument checks and marshalling only, as
// api.py does for the others, then the C ABI's entry point.  In Python the checks
// and the conversion of some 25 arguments take 6 us of a call whose kernel runs for
// 2 (the host of a GB300, an append of 4 tokens: 10.3 us a call, 3.3 here).
//
// Each takes its tensors in the order of api.py's function and then `stream` (a raw
// handle, or None: torch's current stream), raises ValueError for what does not fit
// together, and returns the entry point's status; the attention calls return minus
// the bytes of the workspace that they need and were not given.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/pagedkv.h"

namespace {

struct Refused {};       // a Python error is set

[[noreturn]] void refuse(const char* why) {
    PyErr_SetString(PyExc_ValueError, why);
    throw Refused();
}

const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) {
        PyErr_SetString(PyExc_TypeError, "expected a torch.Tensor");
        throw Refused();
    }
    return THPVariable_Unpack(o);
}

// NULL for None.
const at::Tensor* optional(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }

long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}

int as_int(long long v) {
    if (v < -2147483647LL || v > 2147483647LL) refuse("a size beyond 32 bits");
    return (int)v;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}

// The calls launch on the current device; every tensor has to be there.
struct Here {
    int device = -1;     // asked for at the first tensor on a GPU: without one there is none
    void check(const at::Tensor& t) {
        if (t.is_cuda() && device < 0) device = (int)c10::cuda::current_device();
        if (!t.is_cuda() || t.get_device() != device)
            refuse("tensors must be on the current CUDA device");
    }
    void check_contiguous(const at::Tensor& t) {
        check(t);
        if (!t.is_contiguous()) refuse("tensors must be contiguous (q, k, v and their outputs: each token)");
    }
    void* stream(PyObject* o) const {
        if (o != Py_None) {
            const unsigned long long v = PyLong_AsUnsignedLongLong(o);
            if (v == (unsigned long long)-1 && PyErr_Occurred()) throw Refused();
            return reinterpret_cast<void*>((uintptr_t)v);
        }
        return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    }
};

// The pointers of a call are all taken ahead of Py_BEGIN_ALLOW_THREADS: data_ptr() throws
// for a tensor without storage (one of vmap's, say), and an exception needs the
// interpreter.
template <class T>
T* pointer(const at::Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}
template <class T>
T* pointer(const at::Tensor* t) {
    return t ? pointer<T>(*t) : nullptr;
}

bool same_shape(const at::Tensor& a, const at::Tensor& b) { return a.sizes() == b.sizes(); }

bool is(const at::Tensor& t, at::ScalarType type) { return t.scalar_type() == type; }

pkv_dtype dtype16(const at::Tensor& t) {
    if (is(t, at::kBFloat16)) return PKV_BF16;
    if (is(t, at::kHalf)) return PKV_F16;
    refuse("q, k and v must be float16 or bfloat16");
}

pkv_dtype dtype_out(const at::Tensor& t) { return is(t, at::kFloat) ? PKV_F32 : dtype16(t); }

// Stride of rows [T, heads, D], each contiguous.
int64_t row_stride(const at::Tensor& t) {
    const int64_t heads = t.size(1), D = t.size(2);
    if (t.size(0) <= 1 || t.is_contiguous()) {
        if (!t.is_contiguous() && ((D > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != D)))
            refuse("rows must be [tokens, heads, head_dim], each token contiguous");
        return heads * D;
    }
    if ((D > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != D))
        refuse("rows must be [tokens, heads, head_dim], each token contiguous");
    return t.stride(0);
}

void check_scales(Here& here, const at::Tensor& k_scale, const at::Tensor& v_scale, int64_t nb,
                  int64_t Hk) {
    for (const at::Tensor* t : {&k_scale, &v_scale}) {
        here.check_contiguous(*t);
        if (!is(*t, at::kFloat) || t->dim() != 2 || t->size(0) != nb || t->size(1) != Hk)
            refuse("k_scale and v_scale must be float32 [num_blocks, Hk]");
    }
}

template <class F>
PyObject* guarded(F f) {
    try {
        return PyLong_FromLongLong(f());
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
        return nullptr;
    }
}

// (k_pool, v_pool, [k_scale, v_scale,] k, v, slots, positions, rope, q, q_out, k_out,
// interleaved, stream)
long long append(PyObject* const* a, Py_ssize_t n, bool q8) {
    if (n != (q8 ? 14 : 12)) refuse("wrong number of arguments");
    Here here;
    const at::Tensor &k_pool = tensor(a[0]), &v_pool = tensor(a[1]);
    PyObject* const* b = a + (q8 ? 4 : 2);
    const at::Tensor &k = tensor(b[0]), &v = tensor(b[1]), &slots = tensor(b[2]);
    const at::Tensor *positions = optional(b[3]), *rope = optional(b[4]), *q = optional(b[5]),
                     *q_out = optional(b[6]), *k_out = optional(b[7]);
    if (k_pool.dim() != 4 || k.dim() != 3)
        refuse("pools are [num_blocks, B, Hk, D], k and v [tokens, Hk, D]");
    const int64_t nb = k_pool.size(0), B = k_pool.size(1), Hk = k_pool.size(2), D = k_pool.size(3),
                  T = k.size(0);
    const at::ScalarType type = k.scalar_type();
    const pkv_dtype dt = dtype16(k);
    const at::ScalarType held = q8 ? at::kFloat8_e4m3fn : type;
    if (!same_shape(k_pool, v_pool) || !same_shape(k, v) || k.size(1) != Hk || k.size(2) != D ||
        !is(v, type) || !is(k_pool, held) || !is(v_pool, held) || slots.dim() != 1 ||
        slots.size(0) != T)
        refuse("inconsistent shapes or dtypes");
    if (!is(slots, at::kLong)) refuse("slot_mapping must be int64");
    here.check_contiguous(k_pool);
    here.check_contiguous(v_pool);
    here.check_contiguous(slots);
    here.check(k);
    here.check(v);
    if (q8) check_scales(here, tensor(a[2]), tensor(a[3]), nb, Hk);
    if (rope) {
        if (!positions) refuse("positions are needed with rope");
        here.check_contiguous(*rope);
        here.check_contiguous(*positions);
        if (!is(*rope, at::kFloat) || rope->dim() != 2)
            refuse("rope must be float32 [positions, rotary_dim]");
        if (!is(*positions, at::kInt) || positions->dim() != 1 || positions->size(0) != T)
            refuse("positions must be int32 [tokens]");
    }
    if ((q == nullptr) != (q_out == nullptr)) refuse("q and q_out: both or neither");
    int64_t H = 0, q_row = 0, q_out_row = 0, k_out_row = 0;
    if (q) {
        if (q->dim() != 3 || q->size(0) != T || q->size(2) != D || !same_shape(*q, *q_out))
            refuse("q and q_out must be [tokens, H, D]");
        if (!is(*q, type) || !is(*q_out, type)) refuse("q and q_out must be of k's dtype");
        here.check(*q);
        here.check(*q_out);
        H = q->size(1);
        q_row = row_stride(*q);
        q_out_row = row_stride(*q_out);
    }
    if (k_out) {
        if (!same_shape(*k_out, k) || !is(*k_out, type)) refuse("k_out must be shaped like k");
        here.check(*k_out);
        k_out_row = row_stride(*k_out);
    }
    const int64_t k_row = row_stride(k), v_row = row_stride(v);
    const int inter = PyObject_IsTrue(b[8]);
    if (inter < 0) throw Refused();
    void* stream = here.stream(b[9]);
    const int rows = rope ? as_int(rope->size(0)) : 0, rot = rope ? as_int(rope->size(1)) : 0;
    const int t = as_int(T), h = as_int(H), hk = as_int(Hk), d = as_int(D), bs = as_int(B),
              blocks = as_int(nb);
    void *kp = pointer<void>(k_pool), *vp = pointer<void>(v_pool);
    const void *k_at = pointer<void>(k), *v_at = pointer<void>(v), *q_at = pointer<void>(q);
    void *q_to = q ? pointer<void>(q_out) : nullptr, *k_to = pointer<void>(k_out);
    const int64_t* slot = pointer<int64_t>(slots);
    const int32_t* pos = rope ? pointer<int32_t>(positions) : nullptr;
    const float* table = pointer<float>(rope);
    float* ks = q8 ? pointer<float>(tensor(a[2])) : nullptr;
    float* vs = q8 ? pointer<float>(tensor(a[3])) : nullptr;
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS
    if (q8)
        st = kv_append_rope_q8(kp, vp, ks, vs, k_at, k_row, v_at, v_row, dt, slot, pos, table, rows,
                               rot, inter, q_at, q_row, q_to, q_out_row, k_to, k_out_row, t, h, hk, d,
                               bs, blocks, stream);
    else
        st = kv_append_rope(kp, vp, k_at, k_row, v_at, v_row, dt, slot, pos, table, rows, rot, inter,
                            q_at, q_row, q_to, q_out_row, k_to, k_out_row, t, h, hk, d, bs, blocks,
                            stream);
    Py_END_ALLOW_THREADS
    return st;
}

// What the 8-bit attention calls share.
struct Q8 {
    const at::Tensor &out, &q, &k_pool, &v_pool, &k_scale, &v_scale, &tables, &lens;
    const at::Tensor* workspace;
    int H, nb, B, Hk, D, S;
    void* out_at = nullptr;
    const void *q_at = nullptr, *kp = nullptr, *vp = nullptr;
    const float *ks = nullptr, *vs = nullptr;
    const int32_t *table = nullptr, *len = nullptr;
    int width = 0;
    void* ws = nullptr;
    size_t ws_bytes = 0;

    Q8(Here& here, PyObject* out_, PyObject* q_, PyObject* const* pools, PyObject* workspace_)
        : out(tensor(out_)), q(tensor(q_)), k_pool(tensor(pools[0])), v_pool(tensor(pools[1])),
          k_scale(tensor(pools[2])), v_scale(tensor(pools[3])), tables(tensor(pools[4])),
          lens(tensor(pools[5])), workspace(optional(workspace_)) {
        for (const at::Tensor* t : {&out, &q, &k_pool, &v_pool, &tables, &lens})
            here.check_contiguous(*t);
        if (q.dim() != 3 || k_pool.dim() != 4)
            refuse("q is [rows, H, D], pools are [num_blocks, B, Hk, D]");
        if (q.size(2) != k_pool.size(3) || !same_shape(k_pool, v_pool) || !same_shape(out, q) ||
            !is(k_pool, at::kFloat8_e4m3fn) || !is(v_pool, at::kFloat8_e4m3fn) || tables.dim() != 2 ||
            lens.dim() != 1 || tables.size(0) != lens.size(0))
            refuse("inconsistent shapes or dtypes");
        if (!is(tables, at::kInt) || !is(lens, at::kInt))
            refuse("block_tables and context_lens must be int32");
        H = as_int(q.size(1));
        nb = as_int(k_pool.size(0));
        B = as_int(k_pool.size(1));
        Hk = as_int(k_pool.size(2));
        D = as_int(k_pool.size(3));
        S = as_int(lens.size(0));
        check_scales(here, k_scale, v_scale, nb, Hk);
        if (workspace) here.check_contiguous(*workspace);
        out_at = pointer<void>(out);
        q_at = pointer<void>(q);
        kp = pointer<void>(k_pool);
        vp = pointer<void>(v_pool);
        ks = pointer<float>(k_scale);
        vs = pointer<float>(v_scale);
        table = pointer<int32_t>(tables);
        len = pointer<int32_t>(lens);
        width = as_int(tables.size(1));
        ws = pointer<void>(workspace);
        ws_bytes = workspace ? workspace->nbytes() : 0;
    }
};

// (out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale,
// max_context_len, workspace, stream)
long long decode(PyObject* const* a, Py_ssize_t n) {
    if (n != 12) refuse("wrong number of arguments");
    Here here;
    const Q8 c(here, a[0], a[1], a + 2, a[10]);
    if (c.q.size(0) != c.S) refuse("inconsistent shapes or dtypes");
    const float scale = (float)number(a[8]);
    const int max_len = as_int(integer(a[9]));
    const pkv_dtype out_dt = dtype_out(c.out), q_dt = dtype16(c.q);
    void* stream = here.stream(a[11]);
    if (!c.workspace) {
        const size_t need =
            pkv_decode_q8_workspace_bytes(c.S, c.H, c.Hk, c.D, c.B, max_len);
        if (need) return -(long long)need;
    }
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS
    st = paged_attn_decode_q8(c.out_at, out_dt, c.q_at, q_dt, c.kp, c.vp, c.ks, c.vs, c.table,
                              c.width, c.len, c.S, c.H, c.Hk, c.D, c.B, c.nb, scale, max_len, c.ws,
                              c.ws_bytes, stream);
    Py_END_ALLOW_THREADS
    return st;
}

// (out, q, q_start, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens,
// scale, max_q_len, max_context_len, workspace, stream)
long long chunk(PyObject* const* a, Py_ssize_t n) {
    if (n != 14) refuse("wrong number of arguments");
    Here here;
    const Q8 c(here, a[0], a[1], a + 3, a[12]);
    const at::Tensor& q_start = tensor(a[2]);
    here.check_contiguous(q_start);
    if (!is(q_start, at::kInt) || q_start.dim() != 1 || q_start.size(0) != (int64_t)c.S + 1)
        refuse("q_start must be int32 [S + 1]");
    const float scale = (float)number(a[9]);
    const int max_q = as_int(integer(a[10])), max_len = as_int(integer(a[11])),
              total = as_int(c.q.size(0));
    const pkv_dtype out_dt = dtype_out(c.out), q_dt = dtype16(c.q);
    const int32_t* start = pointer<int32_t>(q_start);
    void* stream = here.stream(a[13]);
    if (!c.workspace) {
        const size_t need =
            pkv_multi_query_q8_workspace_bytes(c.S, max_q, c.H, c.Hk, c.D, c.B, max_len);
        if (need) return -(long long)need;
    }
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS
    st = paged_attn_multi_query_q8(c.out_at, out_dt, c.q_at, q_dt, start, total, max_q, c.kp, c.vp,
                                   c.ks, c.vs, c.table, c.width, c.len, c.S, c.H, c.Hk, c.D, c.B,
                                   c.nb, scale, max_len, c.ws, c.ws_bytes, stream);
    Py_END_ALLOW_THREADS
    return st;
}

PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] { return append(a, n, false); });
}
PyObject* py_append_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] { return append(a, n, true); });
}
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] { return decode(a, n); });
}
PyObject* py_chunk(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] { return chunk(a, n); });
}

template <class F>
PyCFunction fastcall(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}

PyMethodDef methods[] = {
    {"kv_append_rope", fastcall(py_append), METH_FASTCALL, nullptr},
    {"kv_append_rope_q8", fastcall(py_append_q8), METH_FASTCALL, nullptr},
    {"paged_attn_decode_q8", fastcall(py_decode), METH_FASTCALL, nullptr},
    {"paged_attn_multi_query_q8", fastcall(py_chunk), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls(void) { return PyModule_Create(&module); }
