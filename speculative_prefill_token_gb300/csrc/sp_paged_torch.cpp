// Torch side of the paged-cache operators, the 4-bit cache and its pages among
// them: checks of the tensors and calls of the C ABI (specprefill.h). The same checks made in Python and the marshalling
// through ctypes cost 5 to 7 us of a call whose kernel takes 3: a decode step
// makes these calls for every layer.
//
// Every function takes all its arguments by position, outputs included, and
// returns the library's status; a tensor that does not fit raises ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
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

// A reference that is dropped at the end of its scope, a refusal's among them.
struct Owned {
    PyObject* o;
    explicit Owned(PyObject* object) : o(object) {}
    Owned(const Owned&) = delete;
    ~Owned() { Py_XDECREF(o); }
    PyObject* release() {
        PyObject* r = o;
        o = nullptr;
        return r;
    }
};

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

// ------------------------------------------------------------ 4-bit cache and pages

struct Pool4 {
    uint8_t* p;
    int64_t blocks, heads, bs, d, block, head;   // strides in bytes
};

// uint8 [blocks, Hk, block_size / 8, 9 d / 2], the records of a block and head
// following one another.
Pool4 pool4(const at::Tensor& t, const char* name, int dev) {
    if (t.dim() != 4 || t.scalar_type() != at::kByte || !on(t, dev) || t.size(3) % 288 != 0 || t.size(3) == 0 ||
        t.size(0) < 1 || t.size(2) < 1 || t.stride(3) != 1 || (t.size(2) > 1 && t.stride(2) != t.size(3)))
        refuse(std::string(name) +
               " must be a uint8 [blocks, Hk, block_size / 8, 9 d / 2] tensor on the call's device with its last two "
               "dimensions dense (make_pool_fp4)");
    return {static_cast<uint8_t*>(t.data_ptr()), t.size(0), t.size(1), t.size(2) * 8, t.size(3) * 2 / 9, t.stride(0), t.stride(1)};
}

void same4(const Pool4& a, const Pool4& b) {
    if (a.blocks != b.blocks || a.bs != b.bs || a.heads != b.heads || a.d != b.d)
        refuse("the pools disagree on heads, head_dim or blocks");
}

// (k, v, slot_map, k_pool, v_pool, q, q_out, positions, cos_sin, n_new, status,
//  k_scale, v_scale, stream)
int call_append_kv_fp4(PyObject* const* a) {
    const at::Tensor& kt = need(a[0], "k");
    const int dev = device_of(kt, "k");
    const at::ScalarType type = kt.scalar_type();
    sp_append_fp4_shape s = {};
    s.dtype = dtype_code(kt, "k");
    const Rows k = rows(kt, type, "k", dev), v = rows(need(a[1], "v"), type, "v", dev);
    const Pool4 kp = pool4(need(a[3], "k_pool"), "k_pool", dev), vp = pool4(need(a[4], "v_pool"), "v_pool", dev);
    same4(kp, vp);
    if (v.n != k.n || v.heads != k.heads || v.d != k.d || kp.heads != k.heads || kp.d != k.d)
        refuse("k, v and the pools disagree on tokens, heads or head_dim");
    s.n_tokens = count(k.n, "k");
    s.n_kv_heads = count(k.heads, "k");
    s.head_dim = count(k.d, "k");
    s.block_size = count(kp.bs, "k_pool");
    s.pool_blocks = kp.blocks;
    s.k_stride_token = k.token, s.k_stride_head = k.head;
    s.v_stride_token = v.token, s.v_stride_head = v.head;
    s.kp_stride_block = kp.block, s.kp_stride_head = kp.head;
    s.vp_stride_block = vp.block, s.vp_stride_head = vp.head;
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
    s.k_scale = static_cast<float>(real(a[11]));
    s.v_scale = static_cast<float>(real(a[12]));
    if (k.n == 0) return SP_OK;
    return sp_append_kv_fp4(&s, q.p, k.p, v.p, slots, at_pos, turn, n_new, qo.p, kp.p, vp.p, status, stream_of(a[13], dev));
}

// (pool, slots, out, scale, status, stream); out is [rows, Hk, d], or without slots
// [blocks, block_size, Hk, d] with the blocks following one another
int call_unpack_fp4(PyObject* const* a) {
    const at::Tensor &pt = need(a[0], "pool"), &ot = need(a[2], "out");
    const int dev = device_of(pt, "pool");
    const Pool4 p = pool4(pt, "pool", dev);
    sp_unpack_fp4_shape s = {};
    s.dtype = dtype_code(ot, "out");
    const at::Tensor* st = maybe(a[1], "slots");
    Rows out;
    if (st) {
        out = rows(ot, ot.scalar_type(), "out", dev);
    } else {
        const Pool o = pool(ot, ot.scalar_type(), "out", dev);
        if (o.blocks != p.blocks || o.bs != p.bs) refuse("out must hold every row of the pool");
        out = {o.p, o.blocks * o.bs, o.heads, o.d, o.token, o.head};
    }
    if (out.heads != p.heads || out.d != p.d) refuse("out and the pool disagree on heads or head_dim");
    const int32_t* slots = ints(st, out.n, "slots", dev);
    s.n_kv_heads = count(p.heads, "pool");
    s.head_dim = count(p.d, "pool");
    s.block_size = count(p.bs, "pool");
    s.pool_blocks = p.blocks;
    s.stride_block = p.block, s.stride_head = p.head;
    s.n_rows = out.n;
    s.o_stride_token = out.token, s.o_stride_head = out.head;
    s.scale = static_cast<float>(real(a[3]));
    int32_t* status = ints(maybe(a[4], "status"), 1, "status", dev);
    if (out.n == 0) return SP_OK;
    return sp_unpack_fp4(&s, p.p, slots, out.p, status, stream_of(a[5], dev));
}

// (pool, slots, like, scale, status): the same into a new tensor of `like`'s type, on the
// current stream (made here: 8 us of the interpreter's time less)
PyObject* new_unpack_fp4(PyObject* const* a) {
    const at::Tensor& pt = need(a[0], "pool");
    const int dev = device_of(pt, "pool");
    const Pool4 p = pool4(pt, "pool", dev);
    const at::Tensor* st = maybe(a[1], "slots");
    const at::ScalarType type = PyObject_IsTrue(a[2]) ? at::kHalf : at::kBFloat16;
    at::Tensor out;
    if (st) out = at::empty({st->numel(), p.heads, p.d}, pt.options().dtype(type));
    else out = at::empty({p.blocks, p.bs, p.heads, p.d}, pt.options().dtype(type));
    Owned o{THPVariable_Wrap(out)};
    if (!o.o) throw PythonError();
    PyObject* args[6] = {a[0], a[1], o.o, a[3], a[4], Py_None};
    const int rc = call_unpack_fp4(args);
    return rc == SP_OK ? o.release() : PyLong_FromLong(rc);
}

// The shape of an attention call over 4-bit pools (table_stride is left to the
// caller).
sp_fp4_shape fp4_shape(const at::Tensor& qt, int64_t n_seqs, const at::Tensor& kpt, const at::Tensor* vpt,
                       const at::Tensor* ot, int dev, PyObject* max_new, Rows* q, Pool4* kp, Pool4* vp, Rows* out) {
    const at::ScalarType type = qt.scalar_type();
    sp_fp4_shape s = {};
    s.dtype = dtype_code(qt, "q");
    *q = rows(qt, type, "q", dev);
    *kp = pool4(kpt, "k_pool", dev);
    *vp = vpt ? pool4(*vpt, "v_pool", dev) : *kp;
    same4(*kp, *vp);
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
    // (a bound above the rows of q is theirs)
    s.max_new = max_new == Py_None ? 0 : int32(max_new, "max_new");
    if (max_new != Py_None && s.max_new < 1) refuse("max_new must be at least 1");
    if (s.max_new > s.n_tokens) s.max_new = 0;
    s.pool_blocks = kp->blocks;
    s.q_stride_token = q->token, s.q_stride_head = q->head;
    s.o_stride_token = out->token, s.o_stride_head = out->head;
    s.k_stride_block = kp->block, s.k_stride_head = kp->head;
    s.v_stride_block = vp->block, s.v_stride_head = vp->head;
    return s;
}

// (q, q_off, kv_len, block_table, k_pool, v_pool, causal, window, scale, k_scale,
//  v_scale, out, lse, max_new, ws, dense_tokens, spin_limit, stream)
int call_paged_attention_fp4(PyObject* const* a) {
    const at::Tensor &qt = need(a[0], "q"), &kvt = need(a[2], "kv_len"), &ot = need(a[11], "out");
    const int dev = device_of(qt, "q");
    const int64_t n_seqs = kvt.numel();
    Rows q, out;
    Pool4 kp, vp;
    sp_fp4_shape s = fp4_shape(qt, n_seqs, need(a[4], "k_pool"), &need(a[5], "v_pool"), &ot, dev, a[13], &q, &kp, &vp, &out);
    const int32_t* kv = ints(&kvt, 1, "kv_len", dev);
    const int32_t* off = ints(&need(a[1], "q_off"), n_seqs + 1, "q_off", dev);
    const int32_t* tab = table(need(a[3], "block_table"), n_seqs, dev, &s.table_stride);
    const at::Tensor* lt = maybe(a[12], "lse");
    float* lse = floats(lt, "lse", dev);
    if (lt && (lt->size(0) != q.n || lt->size(1) != q.heads)) refuse("lse must be [T, Hq]");
    s.dense_tokens = integer(a[15]);
    sp_fp4_params p;
    const int causal = PyObject_IsTrue(a[6]);
    if (causal < 0) throw PythonError();
    p.causal = causal;
    p.window = int32(a[7], "window");
    p.scale = static_cast<float>(real(a[8]));
    p.k_scale = static_cast<float>(real(a[9]));
    p.v_scale = static_cast<float>(real(a[10]));
    p.spin_limit = int32(a[16], "spin_limit");
    const at::Tensor& ws = need(a[14], "ws");
    if (!on(ws, dev) || !ws.is_contiguous()) refuse("ws must come from make_attention_fp4_workspace on the call's device");
    return sp_paged_attention_fp4(&s, &p, off, kv, tab, q.p, kp.p, vp.p, out.p, lse, ws.data_ptr(),
                                  static_cast<size_t>(ws.nbytes()), stream_of(a[17], dev));
}

// (q, n_seqs, k_pool, max_new, dense_tokens) -> bytes of workspace, or minus the
// status
int64_t call_workspace_fp4(PyObject* const* a) {
    const at::Tensor& qt = need(a[0], "q");
    const int dev = device_of(qt, "q");
    Rows q, out;
    Pool4 kp, vp;
    sp_fp4_shape s = fp4_shape(qt, integer(a[1]), need(a[2], "k_pool"), nullptr, nullptr, dev, a[3], &q, &kp, &vp, &out);
    s.dense_tokens = integer(a[4]);
    size_t bytes = 0;
    const int rc = sp_paged_attention_fp4_workspace(&s, &bytes);
    return rc == SP_OK ? static_cast<int64_t>(bytes) : -static_cast<int64_t>(rc);
}

// (pools, src, dst, rows, block_table, src_off, n_used, status, stream)
int call_copy_kv(PyObject* const* a) {
    PyObject* list = PySequence_Fast(a[0], "pools must be a sequence of tensors");
    if (!list) throw PythonError();
    const Owned release{list};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(list);
    if (n < 1 || n > SP_MAX_COPY_POOLS) refuse("give 1 to " + std::to_string(SP_MAX_COPY_POOLS) + " pools");
    const at::Tensor& first = need(PySequence_Fast_GET_ITEM(list, 0), "pools");
    const int dev = device_of(first, "pools");
    sp_copy_shape s = {};
    void* ptr[SP_MAX_COPY_POOLS];
    s.fp4 = first.scalar_type() == at::kByte;
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor& t = need(PySequence_Fast_GET_ITEM(list, i), "pools");
        if (t.scalar_type() != first.scalar_type() || t.sizes() != first.sizes() || t.strides() != first.strides())
            refuse("the pools must have one type, shape and layout");
        if (s.fp4) {
            const Pool4 p = pool4(t, "a pool", dev);
            ptr[i] = p.p;
            s.pool_blocks = p.blocks;
            s.block_size = count(p.bs, "pools");
            s.n_kv_heads = count(p.heads, "pools");
            s.head_dim = count(p.d, "pools");
            s.stride_block = p.block, s.stride_head = p.head;
        } else {
            dtype_code(t, "a 16-bit pool");
            if (t.dim() != 4 || t.stride(3) != 1 || !on(t, dev) || t.size(0) < 1)
                refuse("a pool must be a [blocks, block_size, Hk, d] tensor on the call's device with d contiguous");
            ptr[i] = t.data_ptr();
            s.pool_blocks = t.size(0);
            s.block_size = count(t.size(1), "pools");
            s.n_kv_heads = count(t.size(2), "pools");
            s.head_dim = count(t.size(3), "pools");
            s.stride_block = 2 * t.stride(0), s.stride_token = 2 * t.stride(1), s.stride_head = 2 * t.stride(2);
        }
    }
    s.n_pools = static_cast<int32_t>(n);
    const at::Tensor &st = need(a[1], "src"), &dt = need(a[2], "dst");
    s.n_entries = count(st.numel(), "src");
    if (dt.numel() != st.numel()) refuse("src and dst must have the same number of entries");
    s.rows = int32(a[3], "rows");
    const at::Tensor *bt = maybe(a[4], "block_table"), *ot = maybe(a[5], "src_off");
    if ((bt != nullptr) != (ot != nullptr)) refuse("block_table and src_off go together");
    const int32_t* tab = nullptr;
    if (bt) {
        s.n_seqs = count(bt->dim() == 2 ? bt->size(0) : 0, "block_table");
        tab = table(*bt, s.n_seqs, dev, &s.table_stride);
    }
    const int32_t* off = ints(ot, s.n_seqs + 1ll, "src_off", dev);
    const int32_t *src = ints(&st, 0, "src", dev), *dst = ints(&dt, 0, "dst", dev);
    const int32_t* n_used = ints(maybe(a[6], "n"), 1, "n", dev);
    int32_t* status = ints(maybe(a[7], "status"), 1, "status", dev);
    if (s.n_entries == 0) return SP_OK;
    return sp_copy_kv(&s, ptr, src, dst, tab, off, n_used, status, stream_of(a[8], dev));
}

// Rows and blocks of a page operator.
sp_pages_shape pages_shape(const at::Tensor& ctx, PyObject* table_o, PyObject* shared_o, const at::Tensor& free,
                           PyObject* block_size, int dev, int32_t** tab, int32_t** shared) {
    sp_pages_shape s = {};
    s.n_seqs = count(ctx.numel(), "ctx_len");
    s.block_size = int32(block_size, "block_size");
    *tab = table(need(table_o, "block_table"), s.n_seqs, dev, &s.table_stride);
    const at::Tensor& sh = need(shared_o, "shared");
    s.pool_blocks = count(sh.numel(), "shared");
    *shared = ints(&sh, 1, "shared", dev);
    s.free_capacity = count(free.numel(), "free_blocks");
    return s;
}

// (src, dst, ctx_len, block_table, shared, free_blocks, n_free, block_size, kv_len,
//  copy_src, copy_dst, n_left, status, stream)
int call_fork_blocks(PyObject* const* a) {
    const at::Tensor &st = need(a[0], "src"), &dt = need(a[1], "dst"), &ctx = need(a[2], "ctx_len"), &free = need(a[5], "free_blocks");
    const int dev = device_of(ctx, "ctx_len");
    int32_t *tab, *shared;
    sp_pages_shape s = pages_shape(ctx, a[3], a[4], free, a[7], dev, &tab, &shared);
    s.n_forks = count(st.numel(), "src");
    if (dt.numel() != st.numel()) refuse("src and dst must have the same number of entries");
    return sp_fork_blocks(&s, ints(&st, 1, "src", dev), ints(&dt, 1, "dst", dev), ints(&ctx, 1, "ctx_len", dev), tab, shared,
                          ints(&free, 0, "free_blocks", dev), ints(&need(a[6], "n_free"), 1, "n_free", dev),
                          ints(&need(a[8], "kv_len"), s.n_seqs, "kv_len", dev),
                          ints(&need(a[9], "copy_src"), s.n_forks, "copy_src", dev),
                          ints(&need(a[10], "copy_dst"), s.n_forks, "copy_dst", dev),
                          ints(&need(a[11], "n_left"), 1, "n_left", dev), ints(maybe(a[12], "status"), 1, "status", dev),
                          stream_of(a[13], dev));
}

// (ctx_len, new_len, block_table, shared, free_blocks, n_free, block_size, kv_len,
//  n_left, status, alone, stream)
int call_free_blocks(PyObject* const* a) {
    const at::Tensor &ctx = need(a[0], "ctx_len"), &free = need(a[4], "free_blocks");
    const int dev = device_of(ctx, "ctx_len");
    int32_t *tab, *shared;
    sp_pages_shape s = pages_shape(ctx, a[2], a[3], free, a[6], dev, &tab, &shared);
    s.alone = PyObject_IsTrue(a[10]);
    if (s.alone < 0) throw PythonError();
    return sp_free_blocks(&s, ints(&ctx, 1, "ctx_len", dev), ints(&need(a[1], "new_len"), s.n_seqs, "new_len", dev), tab, shared,
                          ints(&free, 0, "free_blocks", dev), ints(&need(a[5], "n_free"), 1, "n_free", dev),
                          ints(&need(a[7], "kv_len"), s.n_seqs, "kv_len", dev),
                          ints(&need(a[8], "n_left"), 1, "n_left", dev), ints(maybe(a[9], "status"), 1, "status", dev),
                          stream_of(a[11], dev));
}

PyObject* wrapped(int64_t v) { return PyLong_FromLongLong(v); }
PyObject* wrapped(PyObject* o) { return o; }

template <typename R, R (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "takes %d arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return wrapped(kCall(args));
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
    SP_METHOD("append_kv_fp4", int, call_append_kv_fp4, 14),
    SP_METHOD("unpack_fp4", int, call_unpack_fp4, 6),
    SP_METHOD("new_unpack_fp4", PyObject*, new_unpack_fp4, 5),
    SP_METHOD("paged_attention_fp4", int, call_paged_attention_fp4, 18),
    SP_METHOD("workspace_fp4", int64_t, call_workspace_fp4, 5),
    SP_METHOD("copy_kv", int, call_copy_kv, 9),
    SP_METHOD("fork_blocks", int, call_fork_blocks, 14),
    SP_METHOD("free_blocks", int, call_free_blocks, 12),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_torch() { return PyModule_Create(&module); }
