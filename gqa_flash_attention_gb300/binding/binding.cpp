// The Python binding of the serving operators: argument checks, outputs and streams in C++, then one call
// of the C ABI (include/sdp.h). The same work in Python with ctypes costs 17 to 39 us a call on the
// host where the smallest kernels take 7, so a decode step waits for its launches; here it takes
// a few. No arithmetic is done here, and the checks are the ABI's callers' part: what the C call itself
// refuses comes back as its status code.
//
// Functions take every argument by position (serving.py has the signatures and their documentation)
// and raise ValueError, or return (status code, results).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <stdexcept>
#include <string>

#include "sdp.h"

namespace {

// A refused argument: becomes ValueError.
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

using OptTensor = std::optional<at::Tensor>;

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        throw Refused(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

OptTensor opt_tensor(PyObject *o, const char *name)
{
    if (o == Py_None)
        return std::nullopt;
    return tensor(o, name);
}

double number(PyObject *o, const char *name)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + " must be a number");
    }
    return x;
}

bool truth(PyObject *o, const char *name)
{
    const int x = PyObject_IsTrue(o);
    if (x < 0) {
        PyErr_Clear();
        throw Refused(std::string(name) + " must be true or false");
    }
    return x != 0;
}

// A whole number that fits the ABI's int.
int whole(PyObject *o, const char *name)
{
    PyObject *i = PyNumber_Index(o);
    if (i == nullptr) {
        PyErr_Clear();
        throw Refused(std::string(name) + " must be a whole number");
    }
    const long long x = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if ((x == -1 && PyErr_Occurred()) || x > INT32_MAX || x < INT32_MIN) {
        PyErr_Clear();
        throw Refused(std::string(name) + " does not fit 32 bits");
    }
    return static_cast<int>(x);
}

int size32(int64_t n, const char *what)
{
    if (n > INT32_MAX)
        throw Refused(std::string(what) + " does not fit 32 bits");
    return static_cast<int>(n);
}

void check(bool ok, const char *what)
{
    if (!ok)
        throw Refused(what);
}

int type_code(const at::Tensor &t)
{
    switch (t.scalar_type()) {
    case at::kHalf:
        return SDP_FP16;
    case at::kBFloat16:
        return SDP_BF16;
    default:
        return -1;
    }
}

int cuda_index(const at::Tensor &t) { return t.is_cuda() ? t.get_device() : -1; }

void forward_only(std::initializer_list<const at::Tensor *> ts)
{
    if (!c10::GradMode::is_enabled())
        return;
    for (const at::Tensor *t : ts)
        check(t == nullptr || !t->requires_grad(), "forward only: detach the inputs or run under torch.no_grad()");
}

// The call's device and stream. Tensors made for a stream other than the current one come from that
// stream's own pool (a block of the current stream's pool could still be in use there) and are safe to
// free from the current one.
class Place {
  public:
    Place(int dev, PyObject *stream) : guard_(static_cast<c10::DeviceIndex>(dev)), now_(c10::cuda::getCurrentCUDAStream(dev))
    {
        if (stream == Py_None) {
            handle_ = now_.stream();
            return;
        }
        PyObject *h = stream;
        Py_INCREF(h);
        if (!PyLong_Check(h)) {
            Py_DECREF(h);
            h = PyObject_GetAttrString(stream, "cuda_stream");
            if (h == nullptr) {
                PyErr_Clear();
                throw Refused("stream must be a torch.cuda.Stream or a stream handle");
            }
        }
        handle_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
        Py_DECREF(h);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            throw Refused("stream must be a torch.cuda.Stream or a stream handle");
        }
        if (handle_ != now_.stream())
            other_ = handle_ == nullptr ? c10::cuda::getDefaultCUDAStream(dev) : c10::cuda::getStreamFromExternal(handle_, dev);
    }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const
    {
        const auto options = at::TensorOptions().dtype(type).device(at::kCUDA, now_.device_index());
        if (!other_)
            return at::empty(shape, options);
        at::Tensor t;
        {
            c10::cuda::CUDAStreamGuard g(*other_);
            t = at::empty(shape, options);
        }
        c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), now_);
        return t;
    }
    void *handle() const { return handle_; }

  private:
    c10::cuda::CUDAGuard guard_;
    c10::cuda::CUDAStream now_;
    std::optional<c10::cuda::CUDAStream> other_;
    cudaStream_t handle_ = nullptr;
};

PyObject *wrap(const OptTensor &t)
{
    if (!t)
        Py_RETURN_NONE;
    return THPVariable_Wrap(*t);
}

// (status code, results...)
PyObject *answer(long long rc, std::initializer_list<const OptTensor *> results)
{
    PyObject *r = PyTuple_New(1 + static_cast<Py_ssize_t>(results.size()));
    PyTuple_SET_ITEM(r, 0, PyLong_FromLongLong(rc));
    Py_ssize_t i = 1;
    for (const OptTensor *t : results)
        PyTuple_SET_ITEM(r, i++, wrap(*t));
    return r;
}

// A contiguous output like `q`, given or new.
at::Tensor output_like(OptTensor given, const at::Tensor &q, int dev, const Place &at)
{
    if (!given)
        return at.empty(q.sizes(), q.scalar_type());
    check(given->sizes() == q.sizes() && given->scalar_type() == q.scalar_type() && given->is_contiguous() &&
              cuda_index(*given) == dev,
          "out must be a contiguous tensor shaped and typed like q");
    return *given;
}

OptTensor lse_of(OptTensor given, bool wanted, at::IntArrayRef shape, int dev, const Place &at)
{
    if (!given) {
        if (!wanted)
            return std::nullopt;
        return at.empty(shape, at::kFloat);
    }
    check(given->sizes() == shape && given->scalar_type() == at::kFloat && given->is_contiguous() && cuda_index(*given) == dev,
          "lse must be a contiguous float32 tensor of q's rows on its device");
    return given;
}

float *lse_ptr(const OptTensor &t) { return t ? t->data_ptr<float>() : nullptr; }

const int *int32_ptr(const at::Tensor &t, int64_t n, int dev, const char *what)
{
    check(t.dim() == 1 && t.size(0) == n && t.scalar_type() == at::kInt && t.is_contiguous() && cuda_index(t) == dev, what);
    return t.data_ptr<int>();
}

// ------------------------------------------------------------------ head norms and rotation

struct Rows {
    int64_t sb, ss, sh, B, S, H;
};

Rows rows_of(const at::Tensor &t)
{
    if (t.dim() == 3)
        return Rows{0, t.stride(0), t.stride(1), 1, t.size(0), t.size(1)};
    return Rows{t.stride(0), t.stride(2), t.stride(1), t.size(0), t.size(2), t.size(1)};
}

PyObject *qk_norm_rope(PyObject *const *a)
{
    const at::Tensor &q = tensor(a[0], "q");
    const OptTensor k = opt_tensor(a[1], "k"), positions = opt_tensor(a[2], "positions");
    const OptTensor wq = opt_tensor(a[4], "q_weight"), wk = opt_tensor(a[5], "k_weight");
    OptTensor qo = opt_tensor(a[8], "q_out"), ko = opt_tensor(a[9], "k_out");
    const bool packed = q.dim() == 3;
    check(packed || q.dim() == 4, "q must be [T, H, D] or [B, H, S, D]");
    const int dev = cuda_index(q), dt = type_code(q);
    check(dev >= 0 && dt >= 0, "q must be a float16 or bfloat16 CUDA tensor");
    forward_only({&q, k ? &*k : nullptr, wq ? &*wq : nullptr, wk ? &*wk : nullptr});
    check(q.stride(-1) == 1, "the last dimension of q must be contiguous");
    const int64_t D = q.size(-1);
    const Rows rq = rows_of(q);
    const Place at(dev, a[10]);
    auto out_like = [&](OptTensor &o, const at::Tensor &x, const char *what) {
        if (!o)
            o = at.empty(x.sizes(), x.scalar_type());
        else
            check(o->sizes() == x.sizes() && o->scalar_type() == x.scalar_type() && cuda_index(*o) == dev && o->stride(-1) == 1,
                  what);
        return rows_of(*o);
    };
    const Rows oq = out_like(qo, q, "q_out must be shaped and typed like q, its last dimension contiguous");
    Rows rk{}, ok{};
    if (k) {
        check(k->dim() == q.dim() && k->scalar_type() == q.scalar_type() && cuda_index(*k) == dev && k->size(-1) == D &&
                  k->stride(-1) == 1,
              "k must have q's dimensions, dtype, device and head dim, its last dimension contiguous");
        rk = rows_of(*k);
        check(rk.B == rq.B && rk.S == rq.S, "q and k must have the same tokens");
        ok = out_like(ko, *k, "k_out must be shaped and typed like k, its last dimension contiguous");
    } else {
        check(!ko && !wk, "k_out and k_weight need k");
    }
    int64_t R = 0, sb = 0, ss = 0;
    const unsigned long long *turns = nullptr;
    const void *pos = nullptr;
    double mscale = 1.0;
    bool wide = false;
    if (a[3] != Py_None) {
        check(PyTuple_Check(a[3]) && PyTuple_GET_SIZE(a[3]) == 2, "table must be rope_table's");
        const at::Tensor &t = tensor(PyTuple_GET_ITEM(a[3], 0), "table.turns");
        mscale = number(PyTuple_GET_ITEM(a[3], 1), "table.mscale");
        check(cuda_index(t) == dev && t.scalar_type() == at::kLong && t.is_contiguous(), "table must be rope_table's, on q's device");
        R = 2 * t.numel();
        turns = reinterpret_cast<const unsigned long long *>(t.data_ptr<int64_t>());
        check(positions && cuda_index(*positions) == dev &&
                  (positions->scalar_type() == at::kInt || positions->scalar_type() == at::kLong),
              "positions must be an int32 or int64 tensor on q's device");
        if (positions->dim() == 1 && positions->size(0) == rq.S) {
            ss = positions->stride(0);
        } else {
            check(!packed && positions->dim() == 2 && positions->size(0) == rq.B && positions->size(1) == rq.S,
                  "positions must be [T], or [S] or [B, S]");
            sb = positions->stride(0);
            ss = positions->stride(1);
        }
        wide = positions->scalar_type() == at::kLong;
        pos = positions->data_ptr();
    }
    std::optional<at::ScalarType> wt;
    for (const OptTensor *w : {&wq, &wk}) {
        if (!*w)
            continue;
        check((*w)->dim() == 1 && (*w)->size(0) == D && (*w)->is_contiguous() && cuda_index(**w) == dev &&
                  ((*w)->scalar_type() == q.scalar_type() || (*w)->scalar_type() == at::kFloat),
              "weights must be contiguous [D] tensors of q's dtype or float32 on its device");
        check(!wt || *wt == (*w)->scalar_type(), "both weights must have one dtype");
        wt = (*w)->scalar_type();
    }
    const int rc = sdp_qk_norm_rope(
        q.data_ptr(), rq.sb, rq.ss, rq.sh, k ? k->data_ptr() : nullptr, rk.sb, rk.ss, rk.sh, qo->data_ptr(), oq.sb, oq.ss,
        oq.sh, ko ? ko->data_ptr() : nullptr, ok.sb, ok.ss, ok.sh, pos, sb, ss, wide, turns, size32(R, "the table"),
        static_cast<float>(mscale), wq ? wq->data_ptr() : nullptr, wk ? wk->data_ptr() : nullptr, wt && *wt == at::kFloat,
        static_cast<float>(number(a[6], "eps")), truth(a[7], "interleaved"), size32(rq.B, "B"), size32(rq.S, "S"),
        size32(rq.H, "Hq"), size32(rk.H, "Hkv"), size32(D, "D"), dt, at.handle());
    return answer(rc, {&qo, &ko});
}

// ------------------------------------------------------------------ the 4-bit paged cache

struct Pool {
    void *kc, *ks, *vc, *vs;
    const int *table;
    int pages, page, max_pages, nseq, Hkv, D;
    long long stride;
};

Pool pool_of(PyObject *cache, const at::Tensor &table, int dev)
{
    check(PyTuple_Check(cache) && PyTuple_GET_SIZE(cache) == 4, "cache must be a Cache4");
    const at::Tensor &kc = tensor(PyTuple_GET_ITEM(cache, 0), "k_codes"), &ks = tensor(PyTuple_GET_ITEM(cache, 1), "k_scales");
    const at::Tensor &vc = tensor(PyTuple_GET_ITEM(cache, 2), "v_codes"), &vs = tensor(PyTuple_GET_ITEM(cache, 3), "v_scales");
    check(kc.dim() == 4 && kc.scalar_type() == at::kByte && vc.scalar_type() == at::kByte && vc.sizes() == kc.sizes(),
          "codes must be uint8 [num_pages, Hkv, page_size, D / 2]");
    const int64_t half = kc.size(3);
    for (const at::Tensor *s : {&ks, &vs})
        check(s->dim() == 5 && s->scalar_type() == at::kBFloat16 && s->size(0) == kc.size(0) && s->size(1) == kc.size(1) &&
                  s->size(2) == kc.size(2) && s->size(3) == half / 32 && s->size(4) == 2,
              "scales must be bfloat16 [num_pages, Hkv, page_size, D / 64, 2]");
    for (const at::Tensor *t : {&kc, &ks, &vc, &vs})
        check(t->is_contiguous() && cuda_index(*t) == dev, "the cache must be contiguous on the inputs' device");
    check(table.dim() == 2 && table.scalar_type() == at::kInt && (table.size(1) <= 1 || table.stride(1) == 1) &&
              cuda_index(table) == dev,
          "block_table must be int32 [nseq, max_pages] on the inputs' device, its last dimension contiguous");
    Pool p;
    p.kc = kc.data_ptr();
    p.ks = ks.data_ptr();
    p.vc = vc.data_ptr();
    p.vs = vs.data_ptr();
    p.table = table.data_ptr<int>();
    p.stride = table.stride(0);
    p.pages = size32(kc.size(0), "num_pages");
    p.Hkv = size32(kc.size(1), "Hkv");
    p.page = size32(kc.size(2), "page_size");
    p.D = size32(2 * half, "D");
    p.nseq = size32(table.size(0), "nseq");
    p.max_pages = size32(table.size(1), "max_pages");
    return p;
}

PyObject *cache4_append(PyObject *const *a)
{
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const at::Tensor &cu = tensor(a[3], "cu_seqlens"), &lens = tensor(a[4], "cache_lens"), &table = tensor(a[5], "block_table");
    const int dev = cuda_index(k), dt = type_code(k);
    check(dev >= 0 && dt >= 0 && v.scalar_type() == k.scalar_type() && cuda_index(v) == dev,
          "k and v must be CUDA tensors on one device of one dtype, float16 or bfloat16");
    forward_only({&k, &v});
    const Pool p = pool_of(a[0], table, dev);
    check(k.dim() == 3 && v.sizes() == k.sizes() && k.size(1) == p.Hkv && k.size(2) == p.D,
          "k and v must be [tokens, Hkv, D] of the cache's heads and head dim");
    check(k.stride(2) == 1 && v.stride(2) == 1, "the last dimension of k and v must be contiguous");
    const int *cp = int32_ptr(cu, p.nseq + 1LL, dev, "cu_seqlens must be a contiguous int32 tensor [nseq + 1] on the inputs' device");
    const int *lp = int32_ptr(lens, p.nseq, dev, "cache_lens must be a contiguous int32 tensor [nseq] on the inputs' device");
    const Place at(dev, a[6]);
    if (p.nseq == 0)
        return answer(SDP_OK, {});
    const int rc = sdp_cache4_append(p.kc, p.ks, p.vc, p.vs, p.pages, p.page, p.table, p.stride, p.max_pages, k.data_ptr(),
                                     k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), cp, lp, p.nseq,
                                     size32(k.size(0), "tokens"), p.Hkv, p.D, dt, at.handle());
    return answer(rc, {});
}

PyObject *cache4_gather(PyObject *const *a)
{
    const at::Tensor &cu = tensor(a[1], "cu_seqlens"), &table = tensor(a[2], "block_table");
    const int total = whole(a[3], "total");
    check(total >= 0, "total must not be negative");
    const bool bf16 = truth(a[4], "dtype");  // serving.py has looked the dtype over
    OptTensor ko = opt_tensor(a[5], "k_out"), vo = opt_tensor(a[6], "v_out");
    const int dev = cuda_index(table);
    check(dev >= 0, "the cache and the block table must be on a CUDA device");
    const Pool p = pool_of(a[0], table, dev);
    const int *cp = int32_ptr(cu, p.nseq + 1LL, dev, "cu_seqlens must be a contiguous int32 tensor [nseq + 1] on the cache's device");
    const Place at(dev, a[7]);
    const at::ScalarType type = bf16 ? at::kBFloat16 : at::kHalf;
    const int64_t shape[3] = {total, p.Hkv, p.D};
    for (OptTensor *t : {&ko, &vo}) {
        if (!*t)
            *t = at.empty(shape, type);
        else
            check((*t)->sizes() == at::IntArrayRef(shape) && (*t)->scalar_type() == type && cuda_index(**t) == dev &&
                      (*t)->stride(2) == 1,
                  "k_out and v_out must be [total, Hkv, D] of dtype on the cache's device, the last dimension contiguous");
    }
    if (p.nseq == 0)
        return answer(SDP_OK, {&ko, &vo});
    const int rc = sdp_cache4_gather(p.kc, p.ks, p.vc, p.vs, p.pages, p.page, p.table, p.stride, p.max_pages, ko->data_ptr(),
                                     ko->stride(0), ko->stride(1), vo->data_ptr(), vo->stride(0), vo->stride(1), cp, p.nseq,
                                     total, p.Hkv, p.D, bf16 ? SDP_BF16 : SDP_FP16, at.handle());
    return answer(rc, {&ko, &vo});
}

PyObject *fwd_cache4(PyObject *const *a)
{
    const at::Tensor &q = tensor(a[0], "q"), &lens = tensor(a[2], "cache_lens"), &table = tensor(a[3], "block_table");
    check(q.dim() == 3 || q.dim() == 4, "q must be [nseq, Hq, D] or [nseq, rows, Hq, D]");
    const int dev = cuda_index(q), dt = type_code(q);
    check(dev >= 0 && dt >= 0 && q.is_contiguous(), "q must be a contiguous float16 or bfloat16 CUDA tensor");
    forward_only({&q});
    const Pool p = pool_of(a[1], table, dev);
    check(p.nseq == q.size(0) && p.D == q.size(-1), "q, the block table and the cache must agree in sequences and head dim");
    const int *lp = int32_ptr(lens, p.nseq, dev, "cache_lens must be a contiguous int32 tensor [nseq] on q's device");
    const int rows = q.dim() == 4 ? size32(q.size(1), "rows") : 1, Hq = size32(q.size(-2), "Hq");
    const Place at(dev, a[11]);
    const OptTensor out = output_like(opt_tensor(a[7], "out"), q, dev, at);
    const OptTensor lse = lse_of(opt_tensor(a[8], "lse"), truth(a[9], "return_lse"), q.sizes().slice(0, q.dim() - 1), dev, at);
    if (p.nseq == 0 || rows == 0)
        return answer(SDP_OK, {&out, &lse});
    const double scale = a[4] == Py_None ? 1.0 / std::sqrt(static_cast<double>(p.D)) : number(a[4], "scale");
    OptTensor ws = opt_tensor(a[10], "workspace");
    if (!ws) {
        const long long need = sdp_fwd_cache4_workspace_bytes(p.nseq, rows, Hq, p.Hkv, p.D, dt);
        if (need < 0)
            return answer(need, {&out, &lse});
        ws = at.empty({need}, at::kByte);
    } else {
        check(cuda_index(*ws) == dev && ws->is_contiguous(), "workspace must be a contiguous tensor on q's device");
    }
    const int rc = sdp_fwd_cache4(q.data_ptr(), p.kc, p.ks, p.vc, p.vs, p.pages, p.page, p.table, p.stride, p.max_pages, lp,
                                  out->data_ptr(), lse_ptr(lse), p.nseq, rows, Hq, p.Hkv, p.D, static_cast<float>(scale), dt,
                                  whole(a[5], "window"), whole(a[6], "sinks"), ws->data_ptr(), ws->nbytes(), at.handle());
    return answer(rc, {&out, &lse});
}

// ------------------------------------------------------------------ sliding windows

// What both window calls want of q, k and v; their device and dtype code.
std::pair<int, int> qkv(const at::Tensor &q, const at::Tensor &k, const at::Tensor &v, int64_t dim, const char *shape)
{
    check(q.dim() == dim && k.dim() == dim && v.dim() == dim, shape);
    const int dev = cuda_index(q), dt = type_code(q);
    check(dev >= 0 && cuda_index(k) == dev && cuda_index(v) == dev, "q, k, v must be CUDA tensors on one device");
    check(dt >= 0 && k.scalar_type() == q.scalar_type() && v.scalar_type() == q.scalar_type(),
          "q, k, v must share one dtype, float16 or bfloat16");
    check(q.is_contiguous() && k.is_contiguous() && v.is_contiguous(), "q, k, v must be contiguous");
    check(k.sizes() == v.sizes() && k.size(-1) == q.size(-1), "q, k and v must agree in shape");
    forward_only({&q, &k, &v});
    return {dev, dt};
}

double scale_or(PyObject *o, int64_t D) { return o == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : number(o, "scale"); }

PyObject *fwd_window(PyObject *const *a)
{
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const auto [dev, dt] = qkv(q, k, v, 4, "q, k, v must be 4-D [B, H, S, D]");
    check(k.size(0) == q.size(0), "q, k and v must have the same batch");
    const Place at(dev, a[9]);
    const OptTensor out = output_like(opt_tensor(a[6], "out"), q, dev, at);
    const OptTensor lse = lse_of(opt_tensor(a[7], "lse"), truth(a[8], "return_lse"), q.sizes().slice(0, 3), dev, at);
    const int rc = sdp_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out->data_ptr(), lse_ptr(lse),
                                  size32(q.size(0), "B"), size32(q.size(1), "Hq"), size32(k.size(1), "Hkv"),
                                  size32(q.size(2), "Sq"), size32(k.size(2), "Skv"), size32(q.size(3), "D"),
                                  static_cast<float>(scale_or(a[5], q.size(3))), dt, whole(a[3], "window"),
                                  whole(a[4], "sinks"), at.handle());
    return answer(rc, {&out, &lse});
}

PyObject *fwd_varlen_window(PyObject *const *a)
{
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const at::Tensor &cq = tensor(a[3], "cu_seqlens_q"), &ck = tensor(a[4], "cu_seqlens_k");
    const auto [dev, dt] = qkv(q, k, v, 3, "q, k, v must be 3-D [tokens, heads, D]");
    check(cq.dim() == 1 && cq.size(0) >= 2, "sequence offsets must be 1-D [nseq + 1]");
    const int64_t n = cq.size(0);
    const int *qp = int32_ptr(cq, n, dev, "cu_seqlens_q must be a contiguous int32 tensor [nseq + 1] on q's device");
    const int *kp = int32_ptr(ck, n, dev, "cu_seqlens_k must be a contiguous int32 tensor [nseq + 1] on q's device");
    const Place at(dev, a[12]);
    const OptTensor out = output_like(opt_tensor(a[9], "out"), q, dev, at);
    const int64_t shape[2] = {q.size(1), q.size(0)};
    const OptTensor lse = lse_of(opt_tensor(a[10], "lse"), truth(a[11], "return_lse"), shape, dev, at);
    const int rc = sdp_fwd_varlen_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out->data_ptr(), lse_ptr(lse), qp, kp,
                                         size32(n - 1, "nseq"), size32(q.size(1), "Hq"), size32(k.size(1), "Hkv"),
                                         size32(q.size(0), "total_q"), size32(k.size(0), "total_k"),
                                         whole(a[5], "max_seqlen_q"), size32(q.size(2), "D"),
                                         static_cast<float>(scale_or(a[8], q.size(2))), dt, whole(a[6], "window"),
                                         whole(a[7], "sinks"), at.handle());
    return answer(rc, {&out, &lse});
}

// No C++ exception leaves an entry: a refused argument is a ValueError, the rest (no memory) a RuntimeError.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments are wanted, %d were given", N, static_cast<int>(n));
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch_c = PyImport_ImportModule("torch");
        PyObject *type = torch_c == nullptr ? nullptr : PyObject_GetAttrString(torch_c, "OutOfMemoryError");
        Py_XDECREF(torch_c);
        PyErr_SetString(type == nullptr ? PyExc_MemoryError : type, e.what_without_backtrace());
        Py_XDECREF(type);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<qk_norm_rope, 11>("qk_norm_rope"),
    method<cache4_append, 7>("cache4_append"),
    method<cache4_gather, 8>("cache4_gather"),
    method<fwd_cache4, 12>("fwd_cache4"),
    method<fwd_window, 10>("fwd_window"),
    method<fwd_varlen_window, 13>("fwd_varlen_window"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__serving() { return PyModule_Create(&module_def); }
