// native.cpp -- argument marshalling of the rotary, windowed and ragged-batch calls
// in native code (CPython extension over torch's C++ API).  A call of the Python binding
// costs 15 to 20 us of host time, most of it tensor attribute look-ups and
// ctypes conversions, which is more than the small calls' kernels take; here it
// costs 2 to 3 us, the launch among them.
//
// Every function makes the same checks as its Python counterpart and, when all
// hold, the library call.  When one does not (another dtype, shape, stride or
// device, or an argument of another kind) it returns None without doing
// anything, and the caller goes on in Python, which says what is wrong.  Nothing
// is kept between calls but the library's function addresses.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/pagedkv.h"
#include "../../include/pagedkv_batch.h"
#include "../../include/pagedkv_rope.h"
#include "../../include/pagedkv_window.h"

namespace {

decltype(&paged_kv_write_rope) g_write_rope;
decltype(&paged_decode_attention_window) g_decode_window;
decltype(&paged_decode_step_window) g_step_window;
decltype(&paged_prefill_attention_window) g_prefill_window;
decltype(&paged_step_maps) g_step_maps;
decltype(&paged_kv_write_slots) g_write_slots;
decltype(&pkv_rows_workspace_bytes) g_rows_workspace_bytes;
decltype(&paged_cross_attention) g_cross;
decltype(&paged_decode_attention_shared) g_shared;

// Lets other Python threads run while it lives: a launch waits where the stream's queue
// is full.  (The caller holds the arguments meanwhile.)
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// The tensor of a Python argument, or null.
const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// The tensor of a Python argument on CUDA device dev, of a type and rank, contiguous.
const at::Tensor *need(PyObject *o, at::ScalarType type, int64_t ndim, int dev)
{
    const at::Tensor *t = tensor(o);
    if (!t || !t->is_cuda() || t->get_device() != dev || t->scalar_type() != type || t->dim() != ndim || !t->is_contiguous())
        return nullptr;
    return t;
}

// Elements between the tokens of t [..., heads, D]; -1: they are not one stride apart.
int64_t token_stride(const at::Tensor &t, int64_t ndim, int dev)
{
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kBFloat16 || t.dim() != ndim) return -1;
    const auto size = t.sizes(), stride = t.strides();
    const int64_t heads = size[ndim - 2], d = size[ndim - 1];
    if ((d > 1 && stride[ndim - 1] != 1) || (heads > 1 && stride[ndim - 2] != d)) return -1;
    int64_t step = heads * d;
    if (size[0] > 1) step = stride[0];
    if (ndim == 4 && size[1] > 1) {
        if (size[0] > 1 && stride[0] != size[1] * stride[1]) return -1;
        step = stride[1];
    }
    return step;
}

// An uninitialised tensor of t's sizes, contiguous, on t's device (straight from the
// allocator: through the dispatcher it takes 0.3 us longer).
at::Tensor new_like(const at::Tensor &t)
{
    return at::Tensor(at::detail::empty_cuda(t.sizes(), t.scalar_type(), t.device(), std::nullopt));
}

struct Pools {
    const at::Tensor *k, *v, *ks, *vs, *tables;
    pkv_dims dims;
    int32_t kv_dtype;
};

// The pools (with scales when they are int8) and, where a call has them, tables.
bool pools(Pools *p, PyObject *k, PyObject *v, PyObject *ks, PyObject *vs, PyObject *tables, int dev)
{
    const at::Tensor *kt = tensor(k);
    if (!kt) return false;
    const bool int8 = kt->scalar_type() == at::kChar;
    const at::ScalarType type = int8 ? at::kChar : at::kBFloat16;
    p->k = need(k, type, 4, dev);
    p->v = need(v, type, 4, dev);
    p->tables = tables ? need(tables, at::kInt, 2, dev) : nullptr;
    if (!p->k || !p->v || (tables && !p->tables) || p->v->sizes() != p->k->sizes()) return false;
    p->ks = p->vs = nullptr;
    const auto size = p->k->sizes();
    if (int8) {
        p->ks = need(ks, at::kFloat, 3, dev);
        p->vs = need(vs, at::kFloat, 3, dev);
        if (!p->ks || !p->vs || p->ks->sizes() != size.slice(0, 3) || p->vs->sizes() != size.slice(0, 3)) return false;
    } else if (ks != Py_None || vs != Py_None) {
        return false;
    }
    for (int64_t s : size)
        if (s > INT32_MAX) return false;
    p->dims = pkv_dims{(int32_t)size[0] - 1, (int32_t)size[1], (int32_t)size[2], (int32_t)size[3]};
    p->kv_dtype = int8 ? PKV_KV_INT8 : PKV_KV_BF16;
    return true;
}

template <class T>
T *ptr(const at::Tensor *t)
{
    return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}

bool small(int64_t x) { return x >= 0 && x <= INT32_MAX; }

// dev_status: None, or an int32 tensor with an element.
bool status_arg(PyObject *o, int dev, int32_t **out)
{
    *out = nullptr;
    if (o == Py_None) return true;
    const at::Tensor *t = tensor(o);
    if (!t || !t->is_cuda() || t->get_device() != dev || t->scalar_type() != at::kInt || !t->is_contiguous() || t->numel() < 1)
        return false;
    *out = t->data_ptr<int32_t>();
    return true;
}

// A rope handle: the address of its pkv_rope and the tensor of its phases (both
// held by the Python object); None where a call needs none.
bool rope_arg(PyObject *address, PyObject *phases, int dev, int64_t head_dim, const pkv_rope **out)
{
    *out = nullptr;
    if (address == Py_None) return true;
    const at::Tensor *t = tensor(phases);
    if (!t || !t->is_cuda() || t->get_device() != dev || !PyLong_Check(address)) return false;
    *out = static_cast<const pkv_rope *>(PyLong_AsVoidPtr(address));
    return *out && (*out)->rot_dim <= head_dim;
}

PyObject *status_result(int st) { return PyLong_FromLong(st); }

// (done, result): a status other than 0 is returned as an int, which the caller raises.
PyObject *none() { Py_RETURN_NONE; }

// write_rope(q, k_new, v_new, rope address, rope phases, k_pool, v_pool, tables,
//            start_pos, k_scales, v_scales, q_out, dev_status) -> q_out, a status, or None
PyObject *write_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 13) return none();
    try {
        const at::Tensor *kp = tensor(a[5]), *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]);
        if (!kp || !q || !k || !v || !kp->is_cuda()) return none();
        const int dev = kp->get_device();
        Pools p;
        if (dev != c10::cuda::current_device() || !pools(&p, a[5], a[6], a[9], a[10], a[7], dev)) return none();
        const int64_t qs = token_stride(*q, 4, dev), ks = token_stride(*k, 4, dev), vs = token_stride(*v, 4, dev);
        if (qs < 0 || ks < 0 || vs < 0) return none();
        const int64_t n_seqs = q->size(0), n_new = q->size(1), hq = q->size(2), d = q->size(3);
        const int64_t new_size[4] = {n_seqs, n_new, p.dims.n_kv_heads, p.dims.head_dim};
        const at::Tensor *sp = need(a[8], at::kInt, 1, dev);
        const pkv_rope *rope;
        int32_t *status;
        if (!sp || d != p.dims.head_dim || k->sizes() != at::IntArrayRef(new_size, 4) || v->sizes() != k->sizes() ||
            p.tables->size(0) != n_seqs || sp->size(0) != n_seqs || !small(n_seqs) || !small(n_new) || !small(hq) ||
            !small(p.tables->size(1)) || !rope_arg(a[3], a[4], dev, d, &rope) || !rope || !status_arg(a[12], dev, &status))
            return none();
        at::Tensor out;
        if (a[11] == Py_None) {
            out = new_like(*q);
        } else {
            const at::Tensor *o = need(a[11], at::kBFloat16, 4, dev);
            if (!o || o->sizes() != q->sizes()) return none();
            out = *o;
        }
        int st;
        {
            const Unlocked other_threads_run;
            st = g_write_rope(ptr<const pkv_bf16>(q), qs, (int32_t)hq, ptr<const pkv_bf16>(k), ks, ptr<const pkv_bf16>(v), vs,
                              rope, ptr<pkv_bf16>(&out), p.k->data_ptr(), p.v->data_ptr(), ptr<float>(p.ks),
                              ptr<float>(p.vs), p.kv_dtype, p.dims, ptr<const int32_t>(p.tables),
                              (int32_t)p.tables->size(1), ptr<const int32_t>(sp), (int32_t)n_seqs, (int32_t)n_new, status,
                              reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream()));
        }
        if (st != 0) return status_result(st);
        if (a[11] != Py_None) {
            Py_INCREF(a[11]);
            return a[11];
        }
        return THPVariable_Wrap(std::move(out));
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// prefill_window(q, k_pool, v_pool, tables, prefix_lens, scale, window, sinks, out,
//                lse_out, dev_status) -> out, a status, or None
PyObject *prefill_window(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 11 || !PyFloat_Check(a[5]) || !PyLong_Check(a[6]) || !PyLong_Check(a[7])) return none();
    try {
        const at::Tensor *t = tensor(a[0]);
        if (!t || !t->is_cuda()) return none();
        const int dev = t->get_device();
        const at::Tensor *q = need(a[0], at::kBFloat16, 4, dev), *pre = need(a[4], at::kInt, 1, dev);
        Pools p;
        int32_t *status;
        if (!q || !pre || dev != c10::cuda::current_device() || !pools(&p, a[1], a[2], Py_None, Py_None, a[3], dev) ||
            p.kv_dtype != PKV_KV_BF16 || q->size(3) != p.dims.head_dim || p.tables->size(0) != q->size(0) ||
            pre->size(0) != q->size(0) || !small(q->size(0)) || !small(q->size(1)) || !small(q->size(2)) ||
            !small(p.tables->size(1)) || !status_arg(a[10], dev, &status))
            return none();
        const long window = PyLong_AsLong(a[6]), sinks = PyLong_AsLong(a[7]);
        if ((window == -1 || sinks == -1) && PyErr_Occurred()) {
            PyErr_Clear();
            return none();
        }
        if (!small(window) || !small(sinks)) return none();
        float *lse = nullptr;
        if (a[9] != Py_None) {
            const at::Tensor *l = need(a[9], at::kFloat, 3, dev);
            if (!l || l->sizes() != q->sizes().slice(0, 3)) return none();
            lse = l->data_ptr<float>();
        }
        at::Tensor out;
        if (a[8] == Py_None) {
            out = new_like(*q);
        } else {
            const at::Tensor *o = need(a[8], at::kBFloat16, 4, dev);
            if (!o || o->sizes() != q->sizes()) return none();
            out = *o;
        }
        const float scale = (float)PyFloat_AS_DOUBLE(a[5]);
        int st;
        {
            const Unlocked other_threads_run;
            st = g_prefill_window(ptr<const pkv_bf16>(q), (int32_t)q->size(2), ptr<const pkv_bf16>(p.k),
                                  ptr<const pkv_bf16>(p.v), p.dims, ptr<const int32_t>(p.tables), (int32_t)p.tables->size(1),
                                  ptr<const int32_t>(pre), (int32_t)q->size(0), (int32_t)q->size(1), scale, (int32_t)window,
                                  (int32_t)sinks, ptr<pkv_bf16>(&out), lse, status,
                                  reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream()));
        }
        if (st != 0) return status_result(st);
        if (a[8] != Py_None) {
            Py_INCREF(a[8]);
            return a[8];
        }
        return THPVariable_Wrap(std::move(out));
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// The arguments of a windowed decode plan that stay the same; the plan's Python
// object holds the tensors whose addresses these are.
struct Plan {
    int dev;
    int32_t n_q_heads, n_seqs, max_blocks, kv_dtype, window, sinks;
    pkv_dims dims;
    float scale;
    void *k_pool, *v_pool;
    float *k_scales, *v_scales, *lse_out;
    const int32_t *tables, *ctx_lens;
    pkv_bf16 *out;
    int32_t *dev_status;
    const pkv_rope *rope;
};

void free_plan(PyObject *capsule) { delete static_cast<Plan *>(PyCapsule_GetPointer(capsule, "pkv_window_plan")); }

// make_plan(device, n_q_heads, rope address or 0, k_pool, v_pool, k_scales, v_scales,
//           kv_dtype, n_blocks, block_size, n_kv_heads, head_dim, tables, max_blocks,
//           ctx_lens, n_seqs, scale, window, sinks, out, lse_out, dev_status): addresses
// (0: none) and numbers that the Python plan has checked
PyObject *make_plan(PyObject *, PyObject *args)
{
    unsigned long long rope, k, v, ks, vs, tables, ctx, out, lse, status;
    Plan p{};
    if (!PyArg_ParseTuple(args, "iiKKKKKiiiiiKiKifiiKKK", &p.dev, &p.n_q_heads, &rope, &k, &v, &ks, &vs, &p.kv_dtype,
                          &p.dims.n_blocks, &p.dims.block_size, &p.dims.n_kv_heads, &p.dims.head_dim, &tables, &p.max_blocks,
                          &ctx, &p.n_seqs, &p.scale, &p.window, &p.sinks, &out, &lse, &status))
        return nullptr;
    p.rope = reinterpret_cast<const pkv_rope *>(rope);
    p.k_pool = reinterpret_cast<void *>(k);
    p.v_pool = reinterpret_cast<void *>(v);
    p.k_scales = reinterpret_cast<float *>(ks);
    p.v_scales = reinterpret_cast<float *>(vs);
    p.tables = reinterpret_cast<const int32_t *>(tables);
    p.ctx_lens = reinterpret_cast<const int32_t *>(ctx);
    p.out = reinterpret_cast<pkv_bf16 *>(out);
    p.lse_out = reinterpret_cast<float *>(lse);
    p.dev_status = reinterpret_cast<int32_t *>(status);
    return PyCapsule_New(new Plan(p), "pkv_window_plan", free_plan);
}

// run_plan(plan, q, k_new, v_new, start_pos) -> a status, or None
PyObject *run_plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 5) return none();
    try {
        const Plan *p = static_cast<const Plan *>(PyCapsule_GetPointer(a[0], "pkv_window_plan"));
        if (!p) return nullptr;
        const at::Tensor *q = tensor(a[1]);
        if (!q || !q->is_cuda() || p->dev != c10::cuda::current_device()) return none();
        const int64_t d = p->dims.head_dim, q_size[3] = {p->n_seqs, p->n_q_heads, d};
        const int64_t qs = token_stride(*q, 3, p->dev);
        if (qs < 0 || q->sizes() != at::IntArrayRef(q_size, 3)) return none();
        const auto stream = reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(p->dev).stream());
        if (a[2] == Py_None) {
            if (a[3] != Py_None || a[4] != Py_None || p->rope || !q->is_contiguous()) return none();
            int st;
            {
                const Unlocked other_threads_run;
                st = g_decode_window(ptr<const pkv_bf16>(q), p->n_q_heads, p->k_pool, p->v_pool, p->k_scales, p->v_scales,
                                     p->kv_dtype, p->dims, p->tables, p->max_blocks, p->ctx_lens, p->n_seqs, p->scale,
                                     p->window, p->sinks, p->out, p->lse_out, p->dev_status, stream);
            }
            return status_result(st);
        }
        const at::Tensor *k = tensor(a[2]), *v = tensor(a[3]), *sp = need(a[4], at::kInt, 1, p->dev);
        if (!k || !v || !sp) return none();
        const int64_t new_size[4] = {p->n_seqs, 1, p->dims.n_kv_heads, d};
        const int64_t ks = token_stride(*k, 4, p->dev), vs = token_stride(*v, 4, p->dev);
        if (ks < 0 || vs < 0 || k->sizes() != at::IntArrayRef(new_size, 4) || v->sizes() != k->sizes() ||
            sp->size(0) != p->n_seqs)
            return none();
        int st;
        {
            const Unlocked other_threads_run;
            st = g_step_window(ptr<const pkv_bf16>(k), ks, ptr<const pkv_bf16>(v), vs, ptr<const int32_t>(sp),
                               ptr<const pkv_bf16>(q), qs, p->n_q_heads, p->rope, p->k_pool, p->v_pool, p->k_scales,
                               p->v_scales, p->kv_dtype, p->dims, p->tables, p->max_blocks, p->ctx_lens, p->n_seqs, p->scale,
                               p->window, p->sinks, p->out, p->lse_out, p->dev_status, stream);
        }
        return status_result(st);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// An int32 (or int64) vector of n elements on device dev, or null.
const at::Tensor *vector(PyObject *o, int64_t n, int dev, at::ScalarType type = at::kInt)
{
    const at::Tensor *t = need(o, type, 1, dev);
    return t && t->size(0) == n ? t : nullptr;
}

pkv_stream_t current_stream(int dev) { return reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream()); }

// A non-negative Python int below 2^31, or -1.
int32_t count_arg(PyObject *o)
{
    if (!PyLong_CheckExact(o)) return -1;
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) PyErr_Clear();
    return small(x) ? (int32_t)x : -1;
}

// step_maps(lens, n_new, free_blocks, block_tables, block_size, n_blocks, n_tokens, cursor,
//           out (six tensors), dev_status) -> a status, or None
PyObject *step_maps(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 10 || !PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 6) return none();
    try {
        const at::Tensor *t = tensor(a[3]);
        if (!t || !t->is_cuda()) return none();
        const int dev = t->get_device();
        const at::Tensor *tables = need(a[3], at::kInt, 2, dev), *free = need(a[2], at::kInt, 1, dev);
        const int32_t bs = count_arg(a[4]), n_blocks = count_arg(a[5]), n_tokens = count_arg(a[6]);
        if (!tables || !free || dev != c10::cuda::current_device() || bs < 0 || n_blocks < 0 || n_tokens < 0 ||
            !small(tables->size(0)) || !small(tables->size(1)) || !small(free->size(0)))
            return none();
        const int64_t n_seqs = tables->size(0);
        const at::Tensor *lens = vector(a[0], n_seqs, dev), *n_new = vector(a[1], n_seqs, dev), *cursor = nullptr;
        if (!lens || !n_new || (a[7] != Py_None && !(cursor = vector(a[7], 1, dev)))) return none();
        const int64_t sizes[6] = {n_seqs, n_seqs + 1, n_tokens, n_tokens, n_tokens, 1};
        const at::Tensor *out[6];
        for (int i = 0; i < 6; ++i)
            if (!(out[i] = vector(PyTuple_GET_ITEM(a[8], i), sizes[i], dev, i == 4 ? at::kLong : at::kInt))) return none();
        int32_t *status;
        if (!status_arg(a[9], dev, &status)) return none();
        int st;
        {
            const Unlocked other_threads_run;
            st = g_step_maps(ptr<const int32_t>(lens), ptr<const int32_t>(n_new), (int32_t)n_seqs, ptr<const int32_t>(free),
                             (int32_t)free->size(0), ptr<const int32_t>(cursor), n_blocks, bs, ptr<int32_t>(tables),
                             (int32_t)tables->size(1), n_tokens, ptr<int32_t>(out[0]), ptr<int32_t>(out[1]), ptr<int32_t>(out[2]),
                             ptr<int32_t>(out[3]), ptr<int64_t>(out[4]), ptr<int32_t>(out[5]), status, current_stream(dev));
        }
        return status_result(st);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// write_slots(k_new, v_new, k_pool, v_pool, slots, k_scales, v_scales, dev_status) -> a
// status, or None
PyObject *write_slots(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 8) return none();
    try {
        const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *kp = tensor(a[2]);
        if (!k || !v || !kp || !kp->is_cuda()) return none();
        const int dev = kp->get_device();
        Pools p;
        if (dev != c10::cuda::current_device() || !pools(&p, a[2], a[3], a[5], a[6], nullptr, dev)) return none();
        const int64_t ks = token_stride(*k, 3, dev), vs = token_stride(*v, 3, dev);
        if (ks < 0 || vs < 0 || !small(k->size(0))) return none();
        const int64_t rows = k->size(0), size[3] = {rows, p.dims.n_kv_heads, p.dims.head_dim};
        const at::Tensor *slots = vector(a[4], rows, dev, at::kLong);
        int32_t *status;
        if (!slots || k->sizes() != at::IntArrayRef(size, 3) || v->sizes() != k->sizes() || !status_arg(a[7], dev, &status)) return none();
        int st;
        {
            const Unlocked other_threads_run;
            st = g_write_slots(ptr<const pkv_bf16>(k), ks, ptr<const pkv_bf16>(v), vs, p.k->data_ptr(), p.v->data_ptr(),
                               ptr<float>(p.ks), ptr<float>(p.vs), p.kv_dtype, p.dims, ptr<const int64_t>(slots), (int32_t)rows,
                               status, current_stream(dev));
        }
        return status_result(st);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// cross(q, q_starts, k_pool, v_pool, tables, key_lens, scale, k_scales, v_scales, out,
//       lse_out, workspace, dev_status) -> out, a status, or None
PyObject *cross(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 13 || !PyFloat_Check(a[6])) return none();
    try {
        const at::Tensor *q = tensor(a[0]);
        if (!q || !q->is_cuda()) return none();
        const int dev = q->get_device();
        Pools p;
        if (dev != c10::cuda::current_device() || !pools(&p, a[2], a[3], a[7], a[8], a[4], dev)) return none();
        const int64_t qs = token_stride(*q, 3, dev), n_seqs = p.tables->size(0);
        const at::Tensor *starts = vector(a[1], n_seqs + 1, dev), *lens = vector(a[5], n_seqs, dev);
        int32_t *status;
        if (qs < 0 || !starts || !lens || q->size(2) != p.dims.head_dim || !small(q->size(0)) || !small(q->size(1)) ||
            !small(n_seqs) || !small(p.tables->size(1)) || !status_arg(a[12], dev, &status))
            return none();
        float *lse = nullptr;
        if (a[10] != Py_None) {
            const at::Tensor *l = need(a[10], at::kFloat, 2, dev);
            if (!l || l->sizes() != q->sizes().slice(0, 2)) return none();
            lse = l->data_ptr<float>();
        }
        at::Tensor out, ws;
        if (a[9] == Py_None) {
            out = new_like(*q);
        } else {
            const at::Tensor *o = need(a[9], at::kBFloat16, 3, dev);
            if (!o || o->sizes() != q->sizes()) return none();
            out = *o;
        }
        if (a[11] == Py_None) {
            const size_t bytes = g_rows_workspace_bytes((int32_t)q->size(0), (int32_t)q->size(1), p.dims.head_dim);
            if (bytes == 0) return none();
            const int64_t size[1] = {(int64_t)bytes};
            ws = at::Tensor(at::detail::empty_cuda(at::IntArrayRef(size, 1), at::kByte, q->device(), std::nullopt));
        } else {
            const at::Tensor *w = need(a[11], at::kByte, 1, dev);
            if (!w) return none();
            ws = *w;
        }
        const float scale = (float)PyFloat_AS_DOUBLE(a[6]);
        int st;
        {
            const Unlocked other_threads_run;
            st = g_cross(ptr<const pkv_bf16>(q), qs, (int32_t)q->size(1), ptr<const int32_t>(starts), (int32_t)q->size(0),
                         p.k->data_ptr(), p.v->data_ptr(), ptr<const float>(p.ks), ptr<const float>(p.vs), p.kv_dtype, p.dims,
                         ptr<const int32_t>(p.tables), (int32_t)p.tables->size(1), ptr<const int32_t>(lens), (int32_t)n_seqs, scale,
                         ptr<pkv_bf16>(&out), lse, ws.data_ptr(), (size_t)ws.numel(), status, current_stream(dev));
        }
        if (st != 0) return status_result(st);
        if (a[9] != Py_None) {
            Py_INCREF(a[9]);
            return a[9];
        }
        return THPVariable_Wrap(std::move(out));
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// The arguments of a shared decode plan that stay the same, as Plan.
struct SharedPlan {
    int dev;
    int32_t n_q_heads, n_seqs, max_blocks, kv_dtype, n_groups, max_prefix_blocks;
    pkv_dims dims;
    float scale;
    void *k_pool, *v_pool, *workspace;
    float *k_scales, *v_scales, *lse_out;
    const int32_t *tables, *ctx_lens, *group_starts, *prefix_tables, *prefix_lens;
    pkv_bf16 *out;
    unsigned long long workspace_bytes;
    int32_t *dev_status;
};

void free_shared_plan(PyObject *capsule) { delete static_cast<SharedPlan *>(PyCapsule_GetPointer(capsule, "pkv_shared_plan")); }

// make_shared_plan(device, n_q_heads, k_pool, v_pool, k_scales, v_scales, kv_dtype, n_blocks,
//                  block_size, n_kv_heads, head_dim, tables, max_blocks, ctx_lens, n_seqs,
//                  group_starts, n_groups, prefix_tables, max_prefix_blocks, prefix_lens,
//                  scale, out, lse_out, workspace, workspace_bytes, dev_status): as make_plan
PyObject *make_shared_plan(PyObject *, PyObject *args)
{
    unsigned long long k, v, ks, vs, tables, ctx, starts, ptables, plens, out, lse, ws, status;
    SharedPlan p{};
    if (!PyArg_ParseTuple(args, "iiKKKKiiiiiKiKiKiKiKfKKKKK", &p.dev, &p.n_q_heads, &k, &v, &ks, &vs, &p.kv_dtype, &p.dims.n_blocks,
                          &p.dims.block_size, &p.dims.n_kv_heads, &p.dims.head_dim, &tables, &p.max_blocks, &ctx, &p.n_seqs,
                          &starts, &p.n_groups, &ptables, &p.max_prefix_blocks, &plens, &p.scale, &out, &lse, &ws,
                          &p.workspace_bytes, &status))
        return nullptr;
    p.k_pool = reinterpret_cast<void *>(k);
    p.v_pool = reinterpret_cast<void *>(v);
    p.k_scales = reinterpret_cast<float *>(ks);
    p.v_scales = reinterpret_cast<float *>(vs);
    p.tables = reinterpret_cast<const int32_t *>(tables);
    p.ctx_lens = reinterpret_cast<const int32_t *>(ctx);
    p.group_starts = reinterpret_cast<const int32_t *>(starts);
    p.prefix_tables = reinterpret_cast<const int32_t *>(ptables);
    p.prefix_lens = reinterpret_cast<const int32_t *>(plens);
    p.out = reinterpret_cast<pkv_bf16 *>(out);
    p.lse_out = reinterpret_cast<float *>(lse);
    p.workspace = reinterpret_cast<void *>(ws);
    p.dev_status = reinterpret_cast<int32_t *>(status);
    return PyCapsule_New(new SharedPlan(p), "pkv_shared_plan", free_shared_plan);
}

// run_shared_plan(plan, q) -> a status, or None
PyObject *run_shared_plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 2) return none();
    try {
        const SharedPlan *p = static_cast<const SharedPlan *>(PyCapsule_GetPointer(a[0], "pkv_shared_plan"));
        if (!p) return nullptr;
        const at::Tensor *q = tensor(a[1]);
        if (!q || !q->is_cuda() || p->dev != c10::cuda::current_device()) return none();
        const int64_t size[3] = {p->n_seqs, p->n_q_heads, p->dims.head_dim}, qs = token_stride(*q, 3, p->dev);
        if (qs < 0 || q->sizes() != at::IntArrayRef(size, 3)) return none();
        int st;
        {
            const Unlocked other_threads_run;
            st = g_shared(ptr<const pkv_bf16>(q), qs, p->n_q_heads, p->k_pool, p->v_pool, p->k_scales, p->v_scales, p->kv_dtype,
                          p->dims, p->tables, p->max_blocks, p->ctx_lens, p->n_seqs, p->group_starts, p->n_groups,
                          p->prefix_tables, p->max_prefix_blocks, p->prefix_lens, p->scale, p->out, p->lse_out, p->workspace,
                          (size_t)p->workspace_bytes, p->dev_status, current_stream(p->dev));
        }
        return status_result(st);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// set_functions(write_rope, decode_window, step_window, prefill_window): the
// library's entry points
PyObject *set_functions(PyObject *, PyObject *args)
{
    unsigned long long f[4];
    if (!PyArg_ParseTuple(args, "KKKK", f, f + 1, f + 2, f + 3)) return nullptr;
    g_write_rope = reinterpret_cast<decltype(g_write_rope)>(f[0]);
    g_decode_window = reinterpret_cast<decltype(g_decode_window)>(f[1]);
    g_step_window = reinterpret_cast<decltype(g_step_window)>(f[2]);
    g_prefill_window = reinterpret_cast<decltype(g_prefill_window)>(f[3]);
    Py_RETURN_NONE;
}

// set_batch_functions(step_maps, write_slots, rows_workspace_bytes, cross, shared): the
// same for those of ragged batches
PyObject *set_batch_functions(PyObject *, PyObject *args)
{
    unsigned long long f[5];
    if (!PyArg_ParseTuple(args, "KKKKK", f, f + 1, f + 2, f + 3, f + 4)) return nullptr;
    g_step_maps = reinterpret_cast<decltype(g_step_maps)>(f[0]);
    g_write_slots = reinterpret_cast<decltype(g_write_slots)>(f[1]);
    g_rows_workspace_bytes = reinterpret_cast<decltype(g_rows_workspace_bytes)>(f[2]);
    g_cross = reinterpret_cast<decltype(g_cross)>(f[3]);
    g_shared = reinterpret_cast<decltype(g_shared)>(f[4]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"set_functions", set_functions, METH_VARARGS, nullptr},
    {"set_batch_functions", set_batch_functions, METH_VARARGS, nullptr},
    {"make_shared_plan", make_shared_plan, METH_VARARGS, nullptr},
    {"run_shared_plan", (PyCFunction)(void (*)(void))run_shared_plan, METH_FASTCALL, nullptr},
    {"step_maps", (PyCFunction)(void (*)(void))step_maps, METH_FASTCALL, nullptr},
    {"write_slots", (PyCFunction)(void (*)(void))write_slots, METH_FASTCALL, nullptr},
    {"cross", (PyCFunction)(void (*)(void))cross, METH_FASTCALL, nullptr},
    {"make_plan", make_plan, METH_VARARGS, nullptr},
    {"run_plan", (PyCFunction)(void (*)(void))run_plan, METH_FASTCALL, nullptr},
    {"write_rope", (PyCFunction)(void (*)(void))write_rope, METH_FASTCALL, nullptr},
    {"prefill_window", (PyCFunction)(void (*)(void))prefill_window, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
