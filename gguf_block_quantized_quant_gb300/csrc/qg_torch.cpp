// qg_torch.cpp -- fast path of the Python binding for the decoder-layer calls: checks and marshals
// torch tensors in C++ and calls the C ABI (include/qg.h).  A call through Python's ctypes takes
// 20 to 30 us on the host of a GB300 (tensor attributes one by one), many times what its kernels
// take for a single token.
//
// Each function takes its arguments by position, returns its outputs, or an int where the C call
// returned a status; bad tensors raise ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>

#include "../../include/qg.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Bad : std::runtime_error {
    using std::runtime_error::runtime_error;
};
void need(bool ok, const char *what) {
    if (!ok) throw Bad(what);
}

const Tensor &tensor(PyObject *o, const char *what) {
    if (!THPVariable_Check(o)) throw Bad(what);
    return THPVariable_Unpack(o);
}
// A tensor or None.
const Tensor *maybe(PyObject *o, const char *what) { return o == Py_None ? nullptr : &tensor(o, what); }

int type_of(ScalarType t) {
    switch (t) {
    case ScalarType::Float: return QG_F32;
    case ScalarType::Half: return QG_F16;
    case ScalarType::BFloat16: return QG_BF16;
    case ScalarType::Char: return QG_Q8_0;
    default: return -1;
    }
}
bool is_float(ScalarType t) { return t == ScalarType::Float || t == ScalarType::Half || t == ScalarType::BFloat16; }
ScalarType dtype(PyObject *o, ScalarType none) {
    if (o == Py_None) return none;
    if (!THPDtype_Check(o)) throw Bad("a dtype is a torch.dtype");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Bad("expected a number");
    return v;
}
// The C interface counts in int: what does not fit is refused, not cut.
int narrow(int64_t v) {
    need(v == (int64_t)(int)v, "a size or an integer argument is beyond 32 bits");
    return (int)v;
}
int integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Bad("expected an integer");
    return narrow(v);
}
void on(const at::Device &d, const Tensor *t) {
    need(!t || t->device() == d, "all tensors of a call must be on one CUDA device");
}
template <class T = void>
T *ptr(const Tensor *t) {
    return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}
// The stream of a call (the current one, or the one given) and the tensors made for it.  They come from that
// stream's memory: memory of the current stream's, freed and handed out again in that stream's order, could
// meet work of the call that is still running or work of the current stream that is not done yet.
class Call {
  public:
    Call(PyObject *o, const at::Device &d) : device_(d), current_(c10::cuda::getCurrentCUDAStream(d.index())), stream_(current_.stream()) {
        if (o == Py_None) return;
        void *p = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred()) throw Bad("a stream is a torch.cuda.Stream");
        if (p == stream_) return;
        stream_ = static_cast<cudaStream_t>(p);
        guard_.reset_stream(c10::cuda::getStreamFromExternal(stream_, d.index()));
    }
    void *stream() const { return stream_; }
    // A workspace: the call is its only user.
    Tensor workspace(int64_t bytes) const { return at::detail::empty_cuda({bytes}, ScalarType::Byte, device_, std::nullopt); }
    // An output, which the caller reads on the current stream (once it has waited for the call).
    Tensor output(at::IntArrayRef shape, ScalarType t) const {
        Tensor x = at::detail::empty_cuda(shape, t, device_, std::nullopt);
        if (guard_.current_stream()) c10::cuda::CUDACachingAllocator::recordStream(x.storage().data_ptr(), current_);
        return x;
    }

  private:
    at::Device device_;
    c10::cuda::CUDAStream current_;
    cudaStream_t stream_;
    c10::cuda::OptionalCUDAStreamGuard guard_;
};
// Rows of a 2-D tensor whose last dimension is contiguous: elements between them.
int64_t rows(const Tensor &t, const char *what) {
    need(t.dim() == 2 && t.is_cuda() && (t.stride(1) == 1 || t.size(1) == 1), what);
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
}
void weight(const Tensor *w, int64_t n) {
    need(!w || (w->scalar_type() == ScalarType::Float && w->numel() == n && w->is_contiguous()),
         "norm weights are contiguous fp32 tensors of the width they scale");
}

struct Heads {
    const void *p;
    int64_t ld, hd;
};
// A (tokens, heads, dim) view, contiguous along dim.
Heads heads(const Tensor &t, const char *what) {
    need(t.dim() == 3 && t.is_cuda() && t.stride(2) == 1, what);
    const int64_t d = t.size(2);
    return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : d, t.size(1) > 1 ? t.stride(1) : d};  // a stride of one element says nothing
}

qg_paged paged(const Tensor &k, const Tensor &v, const Tensor *kd, const Tensor *vd, const Tensor &q_start, const Tensor &kv_len,
               const Tensor &pages) {
    const int type = type_of(k.scalar_type());
    // the stride of a dimension of one element says nothing
    auto strides = [](const Tensor &a, const Tensor &b) {
        for (int i = 0; i < 4; ++i)
            if (a.size(i) > 1 && a.stride(i) != b.stride(i)) return false;
        return true;
    };
    need(k.dim() == 4 && (type == QG_F16 || type == QG_BF16 || type == QG_Q8_0) && v.scalar_type() == k.scalar_type() &&
             v.sizes() == k.sizes() && strides(k, v) && k.is_cuda(),
         "cache pools are fp16, bf16 or int8 CUDA tensors (pages, kv_heads, page, dim) of one shape, type and layout");
    need(k.stride(3) == 1, "cache pools must be contiguous along the head dimension");
    const int64_t n = k.size(0), h = k.size(1), page = k.size(2), dim = k.size(3);
    qg_paged c{};
    if (type == QG_Q8_0) {
        need(kd && vd && kd->scalar_type() == ScalarType::Half && vd->scalar_type() == ScalarType::Half,
             "an int8 cache needs fp16 steps kd and vd");
        const int64_t blocks = dim / 32;
        for (const Tensor *s : {kd, vd})
            need(s->dim() == 4 && s->size(0) == n && s->size(1) == h && s->size(2) == page && s->size(3) == blocks &&
                     s->stride(3) == 1 && s->stride(2) == blocks && (h == 1 || s->stride(1) == page * blocks) && strides(*s, *kd),
                 "steps have shape (pages, kv_heads, page, dim / 32), contiguous within a page");
        c.step_stride = n > 1 ? kd->stride(0) : h * page * blocks;
    }
    for (const Tensor *t : {&q_start, &kv_len, &pages})
        need(t->scalar_type() == ScalarType::Int, "q_start, kv_len and pages are int32 tensors");
    const int64_t batch = kv_len.numel();
    need(q_start.numel() == batch + 1 && pages.dim() == 2 && pages.size(0) == batch && (pages.stride(1) == 1 || pages.size(1) == 1),
         "q_start has batch + 1 entries, kv_len batch, pages batch rows");
    need(q_start.is_contiguous() && kv_len.is_contiguous(), "q_start and kv_len must be contiguous");
    for (const Tensor *t : {&v, kd, vd, &q_start, &kv_len, &pages}) on(k.device(), t);
    c.type = type;
    c.kv_heads = narrow(h), c.dim = narrow(dim), c.page = narrow(page), c.n_pages = narrow(n);
    c.batch = narrow(batch), c.table_width = narrow(pages.size(1));
    c.slot_stride = k.stride(2);
    c.head_stride = h > 1 ? k.stride(1) : page * c.slot_stride;
    c.page_stride = n > 1 ? k.stride(0) : h * page * c.slot_stride;
    c.table_stride = batch > 1 ? pages.stride(0) : std::max(pages.size(1), pages.stride(0));
    c.k = k.data_ptr(), c.v = v.data_ptr();
    c.kd = type == QG_Q8_0 ? kd->data_ptr() : nullptr, c.vd = type == QG_Q8_0 ? vd->data_ptr() : nullptr;
    c.q_start = q_start.const_data_ptr<int32_t>(), c.kv_len = kv_len.const_data_ptr<int32_t>(), c.pages = pages.const_data_ptr<int32_t>();
    return c;
}

template <class Fn>
PyObject *guarded(Fn &&fn) {
    try {
        return fn();
    } catch (const Bad &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
bool arguments(Py_ssize_t have, Py_ssize_t want) {
    if (have == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
    return false;
}

// (y, res, w_pre, w_post, gate, alpha, eps, w_offset, x_dtype, res_out, x_out, stream)
PyObject *norm_residual(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 12)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &y = tensor(a[0], "y is a tensor");
        const Tensor *res = maybe(a[1], "res is a tensor or None"), *w_pre = maybe(a[2], "w_pre is a tensor or None");
        const Tensor *w_post = maybe(a[3], "w_post is a tensor or None"), *gate = maybe(a[4], "gate is a tensor or None");
        const Tensor *ro = maybe(a[9], "res_out is a tensor or None"), *xo = maybe(a[10], "x_out is a tensor or None");
        const int64_t ldy = rows(y, "y is a CUDA tensor (rows, width), contiguous along the width");
        const int64_t M = y.size(0), H = y.size(1);
        need(is_float(y.scalar_type()), "y is fp32, fp16 or bf16");
        for (const Tensor *t : {res, w_pre, w_post, gate, ro, xo}) on(y.device(), t);
        int64_t ldr = H, ldg = 0;
        ScalarType rt = y.scalar_type();
        if (res) {
            ldr = rows(*res, "res is a CUDA tensor (rows, width), contiguous along the width");
            need(res->sizes() == y.sizes(), "res has the shape of y");
            rt = res->scalar_type();
        }
        if (gate) {
            need(gate->scalar_type() == y.scalar_type() && gate->dim() <= 2 && gate->dim() >= 1 && gate->size(-1) == H &&
                     (gate->stride(-1) == 1 || H == 1) && (gate->dim() == 1 || gate->size(0) == 1 || gate->size(0) == M),
                 "gate has y's type and shape (rows, width) or (width,), contiguous along the width");
            if (gate->dim() == 2 && gate->size(0) > 1) ldg = gate->stride(0);
        }
        weight(w_pre, H);
        weight(w_post, H);
        const c10::cuda::CUDAGuard dev(y.device());
        const Call call(a[11], y.device());
        Tensor r, x;
        if (ro) {
            need(ro->sizes() == y.sizes() && ro->scalar_type() == rt && ro->is_contiguous(), "res_out is contiguous, with res's shape and type");
        } else {
            r = call.output({M, H}, rt);
            ro = &r;
        }
        if (xo) {
            need(xo->sizes() == y.sizes() && xo->is_contiguous() && w_pre, "x_out is contiguous, with y's shape, and needs w_pre");
        } else if (w_pre) {
            x = call.output({M, H}, dtype(a[8], y.scalar_type()));
            xo = &x;
        }
        const int rc = qg_norm_residual(y.data_ptr(), type_of(y.scalar_type()), ldy, ptr(res), type_of(rt), ldr, ptr<const float>(w_post),
                                        ptr(gate), ldg, ptr<const float>(w_pre), (float)number(a[7]), (float)number(a[5]),
                                        (float)number(a[6]), ro->data_ptr(), ptr(xo), xo ? type_of(xo->scalar_type()) : QG_F32, narrow(M), narrow(H),
                                        call.stream());
        if (rc) return PyLong_FromLong(rc);
        PyObject *pr = THPVariable_Wrap(*ro), *px = xo ? THPVariable_Wrap(*xo) : (Py_INCREF(Py_None), Py_None);
        PyObject *out = PyTuple_Pack(2, pr, px);
        Py_XDECREF(pr);
        Py_XDECREF(px);
        return out;
    });
}

// (q, nk, nv, turns, k, v, q_start, kv_len, pages, kd, vd, pairs, amp, wq, wk, eps, q_dtype, q_out, stream)
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 19)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &q = tensor(a[0], "q is a tensor"), &nk = tensor(a[1], "nk is a tensor"), &nv = tensor(a[2], "nv is a tensor");
        const Tensor *turns = maybe(a[3], "turns is a tensor or None");
        const Tensor &k = tensor(a[4], "k is a tensor"), &v = tensor(a[5], "v is a tensor");
        const Tensor *kd = maybe(a[9], "kd is a tensor or None"), *vd = maybe(a[10], "vd is a tensor or None");
        const Tensor *wq = maybe(a[13], "wq is a tensor or None"), *wk = maybe(a[14], "wk is a tensor or None");
        const Tensor *qo = maybe(a[17], "q_out is a tensor or None");
        const char *what = "q, nk and nv are CUDA tensors (tokens, heads, dim), contiguous along dim";
        const Heads hq = heads(q, what), hk = heads(nk, what), hv = heads(nv, what);
        const qg_paged c = paged(k, v, kd, vd, tensor(a[6], "q_start is a tensor"), tensor(a[7], "kv_len is a tensor"), tensor(a[8], "pages is a tensor"));
        const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
        need(is_float(q.scalar_type()) && nk.scalar_type() == q.scalar_type() && nv.scalar_type() == q.scalar_type() && nk.sizes() == nv.sizes() &&
                 nk.size(0) == T && nk.size(2) == D && nk.size(1) == k.size(1) && D == k.size(3),
             "q, nk and nv are of one float type, for the same tokens and the cache's heads");
        const ScalarType dt = k.scalar_type() == ScalarType::BFloat16 ? ScalarType::BFloat16 : ScalarType::Half;
        need(dtype(a[16], dt) == dt, "queries beside a bf16 cache are bf16, else fp16");
        need(!turns || (turns->scalar_type() == ScalarType::Long && turns->is_contiguous()), "turns is a contiguous int64 tensor");
        weight(wq, D);
        weight(wk, D);
        for (const Tensor *t : {&nk, &nv, turns, &k, wq, wk, qo}) on(q.device(), t);
        const c10::cuda::CUDAGuard dev(q.device());
        const Call call(a[18], q.device());
        Tensor o;
        if (qo) {
            need(qo->sizes() == q.sizes() && qo->scalar_type() == dt && qo->is_contiguous(), "q_out is contiguous, with q's shape");
        } else {
            o = call.output({T, H, D}, dt);
            qo = &o;
        }
        const int rc = qg_rope_append(hq.p, hq.ld, hq.hd, hk.p, hk.ld, hk.hd, hv.p, hv.ld, hv.hd, type_of(q.scalar_type()), narrow(T), narrow(H),
                                      ptr<const uint64_t>(turns), turns ? narrow(2 * turns->numel()) : 0, PyObject_IsTrue(a[11]),
                                      (float)number(a[12]), ptr<const float>(wq), ptr<const float>(wk), (float)number(a[15]), qo->data_ptr(),
                                      &c, call.stream());
        return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(*qo);
    });
}

// The longest chunk where the caller does not say: the lengths are on the device.  Tokens that divide evenly are
// taken for as many of each sequence (single tokens, drafts to verify); else for one chunk among single tokens, the
// longest there can be if every sequence has one.  Taking the mean there too sends a chunk through the row
// kernel, 8 or 16 rows at a time, over all of its context: one chunk of 193 tokens after 16000 among 63 single
// tokens of 300 to 16000, 16/8 heads of 128, fp16 401 us, now 213, and without end for longer ones; taking the
// longest for even calls too costs at most a factor of two: 64 x 2 tokens, 8-bit 230 us instead of 110.
int longest_guess(int64_t tokens, int64_t batch) {
    if (batch < 1) return 0;
    return narrow(tokens % batch == 0 ? tokens / batch : std::max(tokens - batch + 1, (tokens + batch - 1) / batch));
}

// (q, k, v, q_start, kv_len, pages, kd, vd, max_new, scale, window, out_dtype, out, lse, ws, stream)
PyObject *attn_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 16)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &q = tensor(a[0], "q is a tensor"), &k = tensor(a[1], "k is a tensor"), &v = tensor(a[2], "v is a tensor");
        const Tensor &q_start = tensor(a[3], "q_start is a tensor"), &kv_len = tensor(a[4], "kv_len is a tensor"), &pages = tensor(a[5], "pages is a tensor");
        const Tensor *kd = maybe(a[6], "kd is a tensor or None"), *vd = maybe(a[7], "vd is a tensor or None");
        const Tensor *out = maybe(a[12], "out is a tensor or None"), *lse = maybe(a[13], "lse is a tensor or None"), *ws = maybe(a[14], "ws is a tensor or None");
        const Heads hq = heads(q, "q is a CUDA tensor (tokens, heads, dim), contiguous along dim");
        const qg_paged c = paged(k, v, kd, vd, q_start, kv_len, pages);
        const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
        const ScalarType qt = q.scalar_type();
        need(D == k.size(3), "pools have shape (pages, kv_heads, page, dim) with q's dim");
        need(qt == ScalarType::Half || qt == ScalarType::BFloat16, "q is fp16 or bf16");
        for (const Tensor *t : {&k, out, lse, ws}) on(q.device(), t);
        need(!lse || (lse->dim() == 2 && lse->size(0) == T && lse->size(1) == H && lse->scalar_type() == ScalarType::Float && lse->is_contiguous()),
             "lse is a contiguous fp32 tensor (tokens, heads)");
        const c10::cuda::CUDAGuard dev(q.device());
        const Call call(a[15], q.device());
        Tensor o, w;
        if (out) {
            need(out->sizes() == q.sizes() && out->is_contiguous() && (out->scalar_type() == qt || out->scalar_type() == ScalarType::Float),
                 "out is contiguous, with q's shape, in q's type or fp32");
        } else {
            o = call.output({T, H, D}, dtype(a[11], qt));
            out = &o;
        }
        size_t nws;
        if (ws) {
            nws = ws->nbytes();
        } else {
            nws = qg_attn_workspace_size(c.dim, narrow(H), c.kv_heads, narrow(T), c.batch);
            if (nws == (size_t)-1) return PyLong_FromLong(QG_EINVAL);
            w = call.workspace((int64_t)nws);
            ws = &w;
        }
        const int max_new = a[8] == Py_None ? longest_guess(T, c.batch) : integer(a[8]);
        const double scale = a[9] == Py_None ? 1.0 / std::sqrt((double)D) : number(a[9]);
        const int rc = qg_attn_paged(hq.p, hq.ld, hq.hd, type_of(qt), narrow(T), narrow(H), max_new, (float)scale, integer(a[10]),
                                     out->data_ptr(), type_of(out->scalar_type()), ptr<float>(lse), &c, ws->data_ptr(), nws,
                                     call.stream());
        return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(*out);
    });
}

PyMethodDef methods[] = {
    {"norm_residual", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_residual)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rope_append)), METH_FASTCALL, nullptr},
    {"attn_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(attn_paged)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "qg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qg_torch(void) { return PyModule_Create(&module); }
