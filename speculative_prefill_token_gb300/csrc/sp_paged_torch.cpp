// Torch side of the paged-cache operators: checks of the tensors and calls of
// the C ABI (specprefill.h). The same checks made in Python and the marshalling
// through ctypes cost 5 to 7 us of a call whose kernel takes 3: a decode step
// makes these calls for every layer.
//
// Every function takes all its arguments by position, outputs included, and
// returns the library's status; a tensor that does not fit raises ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <stdexcept>
#include <string>

#include "specprefill.h"

namespace {

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

// A Python error is already set.
struct PythonError {};

const at::Tensor* maybe(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

const at::Tensor& need(PyObject* o, const char* name) {
    const at::Tensor* t = maybe(o, name);
    if (!t) refuse(std::string(name) + " must be a tensor");
    return *t;
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}

int32_t int32(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
    return static_cast<int32_t>(v);
}

double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return v;
}

// The device of a call: that of its first tensor, which has to be the current
// CUDA device (the library launches there).
int device_of(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    const int dev = t.get_device();
    if (dev != c10::cuda::current_device()) refuse(std::string(name) + " is not on the current CUDA device");
    return dev;
}

sp_stream_t stream_of(PyObject* o, int dev) {
    if (o == Py_None)
        return reinterpret_cast<sp_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
    return reinterpret_cast<sp_stream_t>(static_cast<uintptr_t>(integer(o)));
}

bool on(const at::Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

// int32 vector of at least n entries.
int32_t* ints(const at::Tensor* t, int64_t n, const char* name, int dev) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kInt || !on(*t, dev) || t->numel() < n || !t->is_contiguous())
        refuse(std::string(name) + " must be a contiguous int32 tensor of at least " + std::to_string(n) +
               " entries on the call's device");
    return static_cast<int32_t*>(t->data_ptr());
}

int dtype_code(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return SP_DTYPE_BF16;
    if (t.scalar_type() == at::kHalf) return SP_DTYPE_F16;
    refuse(std::string(name) + " must be bfloat16 or float16");
}

struct Rows {
    uint16_t* p;
    int64_t n, heads, d, token, head;   // strides in elements
};

// [rows, heads, d], d contiguous.
Rows rows(const at::Tensor& t, at::ScalarType type, const char* name, int dev) {
    if (t.dim() != 3 || t.scalar_type() != type || t.stride(2) != 1 || !on(t, dev))
        refuse(std::string(name) +
               " must be a [rows, heads, d] tensor of the call's type and device with d contiguous");
    return {static_cast<uint16_t*>(t.data_ptr()), t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)};
}

struct Pool {
    uint16_t* p;
    int64_t blocks, bs, heads, d, token, head;
};

// [blocks, block_size, Hk, d], blocks following one another.
Pool pool(const at::Tensor& t, at::ScalarType type, const char* name, int dev) {
    if (t.dim() != 4 || t.scalar_type() != type || t.stride(3) != 1 || !on(t, dev))
        refuse(std::string(name) +
               " must be a [blocks, block_size, Hk, d] tensor of the call's type and device with d contiguous");
    // (a block of one row has no token stride of its own)
    const int64_t token = t.size(1) > 1 ? t.stride(1) : t.stride(0);
    if (t.size(0) > 1 && t.stride(0) != t.size(1) * token)
        refuse("the blocks of " + std::string(name) + " must follow one another with the token stride");
    return {static_cast<uint16_t*>(t.data_ptr()), t.size(0), t.size(1), t.size(2), t.size(3), token, t.stride(2)};
}

void same(const Pool& a, const Pool& b) {
    if (a.blocks != b.blocks || a.bs != b.bs || a.heads != b.heads || a.d != b.d)
        refuse("the pools disagree on heads, head_dim or blocks");
}

int32_t* table(const at::Tensor& t, int64_t n_seqs, int dev, int32_t* width) {
    if (t.dim() != 2 || t.scalar_type() != at::kInt || t.size(0) != n_seqs || t.size(1) < 1 || !t.is_contiguous() ||
        !on(t, dev) || t.size(1) > INT32_MAX)
        refuse("block_table must be a contiguous int32 [B, max_blocks] tensor on the call's device");
    *width = static_cast<int32_t>(t.size(1));
    return static_cast<int32_t*>(t.data_ptr());
}

int32_t count(int64_t n, const char* what) {
    if (n > INT32_MAX) refuse(std::string(what) + " has too many entries");
    return static_cast<int32_t>(n);
}

float* floats(const at::Tensor* t, const char* name, int dev) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kFloat || t->dim() != 2 || !t->is_contiguous() || !on(*t, dev))
        refuse(std::string(name) + " must be a contiguous two-dimensional float32 tensor on the call's device");
    return static_cast<float*>(t->data_ptr());
}

// (ctx_len, new_off, free_blocks, n_free, block_table, block_size, n_tokens,
//  slot_map, kv_len, n_left, status, pool_blocks, stream); n_tokens None: all
// of slot_map, pool_blocks None: as many as 31-bit slots allow.
int call_block_tables(PyObject* const* a) {
    const at::Tensor &ctx = need(a[0], "ctx_len"), &slots = need(a[7], "slot_map");
    const int dev = device_of(ctx, "ctx_len");
    sp_block_shape s;
    s.n_seqs = count(ctx.numel(), "ctx_len");
    s.block_size = int32(a[5], "block_size");
    int32_t* tab = table(need(a[4], "block_table"), s.n_seqs, dev, &s.table_stride);
    s.n_tokens = a[6] == Py_None ? count(slots.numel(), "slot_map") : int32(a[6], "n_tokens");
    const at::Tensor& free = need(a[2], "free_blocks");
    s.free_capacity = count(free.numel(), "free_blocks");
    s.pool_blocks = a[11] == Py_None ? INT32_MAX / (s.block_size > 0 ? s.block_size : 1) : int32(a[11], "pool_blocks");
    return sp_block_tables(&s, ints(&ctx, 1, "ctx_len", dev), ints(&need(a[1], "new_off"), s.n_seqs + 1ll, "new_off", dev),
                           ints(&free, 0, "free_blocks", dev), ints(&need(a[3], "n_free"), 1, "n_free", dev), tab,
                           ints(&slots, s.n_tokens, "slot_map", dev),
                           ints(&need(a[8], "kv_len"), s.n_seqs, "kv_len", dev),
                           ints(&need(a[9], "n_left"), 1, "n_left", dev), ints(maybe(a[10], "status"), 1, "status", dev),
                           stream_of(a[12], dev));
}

// (k, v, slot_map, k_pool, v_pool, q, q_out, positions, cos_sin, n_new, status,
//  stream)
int call_append_kv(PyObject* const* a) {
    const at::Tensor& kt = need(a[0], "k");
    const int dev = device_of(kt, "k");
    const at::ScalarType type = kt.scalar_type();
    sp_append_shape s = {};
    s.dtype = dtype_code(kt, "k");
    const Rows k = rows(kt, type, "k", dev), v = rows(need(a[1], "v"), type, "v", dev);
    const Pool kp = pool(need(a[3], "k_pool"), type, "k_pool", dev), vp = pool(need(a[4], "v_pool"), type, "v_pool", dev);
    same(kp, vp);
    if (v.n != k.n || v.heads != k.heads || v.d != k.d || kp.heads != k.heads || kp.d != k.d)
        refuse("k, v and the pools disagree on tokens, heads or head_dim");
    s.n_tokens = count(k.n, "k");
    s.n_kv_heads = count(k.heads, "k");
    s.head_dim = count(k.d, "k");
    s.pool_tokens = kp.blocks * kp.bs;
    s.k_stride_token = k.token, s.k_stride_head = k.head;
    s.v_stride_token = v.token, s.v_stride_head = v.head;
    s.kp_stride_token = kp.token, s.kp_stride_head = kp.head;
    s.vp_stride_token = vp.token, s.vp_stride_head = vp.head;
    const at::Tensor *qt = maybe(a[5], "q"), *qot = maybe(a[6], "q_out");
    Rows q = {}, qo = {};
    if ((qt != nullptr) != (qot != nullptr)) refuse("q and q_out go together");
    if (qt) {
        q = rows(*qt, type, "q", dev);
        qo = rows(*qot, type, "q_out", dev);
        if (q.n != k.n || q.d != k.d || qo.n != q.n || qo.heads != q.heads || qo.d != q.d)
            refuse("q, q_out and k disagree on tokens, heads or head_dim");
        s.n_q_heads = count(q.heads, "q");
        s.q_stride_token = q.token, s.q_stride_head = q.head;
        s.qo_stride_token = qo.token, s.qo_stride_head = qo.head;
    }
    const at::Tensor *pos = maybe(a[7], "positions"), *cs = maybe(a[8], "cos_sin");
    if ((pos != nullptr) != (cs != nullptr)) refuse("positions and cos_sin go together");
    const float* turn = floats(cs, "cos_sin", dev);
    if (cs) {
        s.max_pos = count(cs->size(0), "cos_sin");
        s.rotary_dim = count(cs->size(1), "cos_sin");
    }
    const int32_t* slots = ints(&need(a[2], "slot_map"), k.n, "slot_map", dev);
    const int32_t* at_pos = ints(pos, k.n, "positions", dev);
    const int32_t* n_new = ints(maybe(a[9], "n_new"), 1, "n_new", dev);
    int32_t* status = ints(maybe(a[10], "status"), 1, "status", dev);
    if (k.n == 0) return SP_OK;
    return sp_append_kv(&s, q.p, k.p, v.p, slots, at_pos, turn, n_new, qo.p, kp.p, vp.p, status, stream_of(a[11], dev));
}

// The shape of an attention call (table_stride is left to the caller).
sp_paged_shape attention_shape(const at::Tensor& qt, int64_t n_seqs, const at::Tensor& kpt, const at::Tensor* vpt,
                               const at::Tensor* ot, int dev, Rows* q, Pool* kp, Pool* vp, Rows* out) {
    const at::ScalarType type = qt.scalar_type();
    sp_paged_shape s = {};
    s.dtype = dtype_code(qt, "q");
    *q = rows(qt, type, "q", dev);
    *kp = pool(kpt, type, "k_pool", dev);
    *vp = vpt ? pool(*vpt, type, "v_pool", dev) : *kp;
    same(*kp, *vp);
    *out = ot ? rows(*ot, type, "out", dev) : Rows{nullptr, q->n, q->heads, q->d, q->heads * q->d, q->d};
    if (q->d != kp->d) refuse("q and the pools disagree on head_dim");
    if (out->n != q->n || out->heads != q->heads || out->d != q->d) refuse("out must have the shape of q");
    s.n_seqs = count(n_seqs, "kv_len");
    s.n_q_heads = count(q->heads, "q");
    s.n_kv_heads = count(kp->heads, "k_pool");
    s.head_dim = count(q->d, "q");
    s.block_size = count(kp->bs, "k_pool");
    s.table_stride = 1;
    s.n_tokens = count(q->n, "q");
    s.pool_tokens = kp->blocks * kp->bs;
    s.q_stride_token = q->token, s.q_stride_head = q->head;
    s.o_stride_token = out->token, s.o_stride_head = out->head;
    s.k_stride_token = kp->token, s.k_stride_head = kp->head;
    s.v_stride_token = vp->token, s.v_stride_head = vp->head;
    return s;
}

// (q, q_off, kv_len, block_table, k_pool, v_pool, causal, window, scale, out,
//  lse, ws, spin_limit, stream)
int call_paged_attention(PyObject* const* a) {
    const at::Tensor &qt = need(a[0], "q"), &kvt = need(a[2], "kv_len"), &ot = need(a[9], "out");
    const int dev = device_of(qt, "q");
    const int64_t n_seqs = kvt.numel();
    Rows q, out;
    Pool kp, vp;
    sp_paged_shape s = attention_shape(qt, n_seqs, need(a[4], "k_pool"), &need(a[5], "v_pool"), &ot, dev, &q, &kp, &vp, &out);
    const int32_t* kv = ints(&kvt, 1, "kv_len", dev);
    const int32_t* off = ints(&need(a[1], "q_off"), n_seqs + 1, "q_off", dev);
    const int32_t* tab = table(need(a[3], "block_table"), n_seqs, dev, &s.table_stride);
    const at::Tensor* lt = maybe(a[10], "lse");
    float* lse = floats(lt, "lse", dev);
    if (lt && (lt->size(0) != q.n || lt->size(1) != q.heads)) refuse("lse must be [T, Hq]");
    sp_attn_params p;
    const int causal = PyObject_IsTrue(a[6]);
    if (causal < 0) throw PythonError();
    p.causal = causal;
    p.window = int32(a[7], "window");
    p.scale = static_cast<float>(real(a[8]));
    p.spin_limit = int32(a[12], "spin_limit");
    const at::Tensor& ws = need(a[11], "ws");
    if (!on(ws, dev) || !ws.is_contiguous()) refuse("ws must come from make_attention_workspace on the call's device");
    return sp_paged_attention(&s, &p, off, kv, tab, q.p, kp.p, vp.p, out.p, lse, ws.data_ptr(),
                              static_cast<size_t>(ws.nbytes()), stream_of(a[13], dev));
}

// (q, n_seqs, k_pool) -> bytes of workspace, or minus the status
int64_t call_workspace(PyObject* const* a) {
    const at::Tensor& qt = need(a[0], "q");
    const int dev = device_of(qt, "q");
    Rows q, out;
    Pool kp, vp;
    const sp_paged_shape s = attention_shape(qt, integer(a[1]), need(a[2], "k_pool"), nullptr, nullptr, dev, &q, &kp, &vp, &out);
    size_t bytes = 0;
    const int rc = sp_paged_attention_workspace(&s, &bytes);
    return rc == SP_OK ? static_cast<int64_t>(bytes) : -static_cast<int64_t>(rc);
}

template <typename R, R (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "takes %d arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return PyLong_FromLongLong(kCall(args));
    } catch (const PythonError&) {
        return nullptr;
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define SP_METHOD(name, type, fn, n) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<type, fn, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    SP_METHOD("block_tables", int, call_block_tables, 13),
    SP_METHOD("append_kv", int, call_append_kv, 12),
    SP_METHOD("paged_attention", int, call_paged_attention, 14),
    SP_METHOD("workspace", int64_t, call_workspace, 3),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_torch() { return PyModule_Create(&module); }
