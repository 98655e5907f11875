// Argument marshalling of block.py's calls: torch tensors to the C structs of
// include/convrot_block.h. A call checks a dozen tensors; through torch's
// Python attributes that took 8 to 12 us, more than the kernels of the smallest
// calls, and here it takes a fraction of one.
//
// Every function takes its arguments by position from block.py, raises
// TypeError or ValueError for what the C side cannot check (types, shapes,
// strides, one device for all), and returns the C call's status, made with that
// device current.
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/convrot_block.h"

namespace {

using at::Tensor;

struct Matrix {
    void *p = nullptr;
    int64_t ld = 0;
};

bool raise(PyObject *kind, const char *name, const char *what)
{
    PyErr_Format(kind, "%s %s", name, what);
    return false;
}

const Tensor *tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) {
        raise(PyExc_TypeError, name, "must be a tensor");
        return nullptr;
    }
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) {
        raise(PyExc_TypeError, name, "must be a CUDA tensor");
        return nullptr;
    }
    return &t;
}

// Every CUDA tensor of the call is on the device of `first`: the C side sees addresses alone.
bool one_device(PyObject *const *v, Py_ssize_t n, const Tensor &first)
{
    for (Py_ssize_t i = 0; i < n; ++i) {
        // (asking whether something is a tensor is slow where it is none)
        if (v[i] == Py_None || PyLong_Check(v[i]) || PyFloat_Check(v[i]) || !THPVariable_Check(v[i])) continue;
        const Tensor &t = THPVariable_Unpack(v[i]);
        if (t.is_cuda() && t.device().index() != first.device().index()) {
            PyErr_Format(PyExc_ValueError, "the tensors of a call must be on one device, not on cuda:%d and cuda:%d",
                         static_cast<int>(first.device().index()), static_cast<int>(t.device().index()));
            return false;
        }
    }
    return true;
}

bool dtype_of(const Tensor &t, const char *name, int32_t &code)
{
    switch (t.scalar_type()) {
    case at::kFloat: code = CONVROT_F32; return true;
    case at::kBFloat16: code = CONVROT_BF16; return true;
    case at::kHalf: code = CONVROT_F16; return true;
    default: return raise(PyExc_TypeError, name, "must be float32, bfloat16 or float16");
    }
}

// A [rows, cols] tensor of the type with contiguous rows. One row has no
// leading dimension of its own, so any that holds it will do.
bool matrix(PyObject *o, const char *name, at::ScalarType type, int64_t rows, int64_t cols, Matrix &m)
{
    const Tensor *t = tensor(o, name);
    if (!t) return false;
    if (t->scalar_type() != type) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor of %s, not %s", name, c10::toString(type), c10::toString(t->scalar_type()));
        return false;
    }
    if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols) {
        PyErr_Format(PyExc_ValueError, "%s must have the shape [%lld, %lld]", name, static_cast<long long>(rows), static_cast<long long>(cols));
        return false;
    }
    if (cols > 1 && t->stride(1) != 1) return raise(PyExc_ValueError, name, "must have contiguous rows");
    m.p = t->data_ptr();
    m.ld = rows > 1 ? t->stride(0) : t->stride(0) > cols ? t->stride(0) : cols;
    return true;
}

bool optional_matrix(PyObject *o, const char *name, at::ScalarType type, int64_t rows, int64_t cols, Matrix &m)
{
    m = Matrix{nullptr, cols};
    return o == Py_None || matrix(o, name, type, rows, cols, m);
}

// A contiguous vector of n elements, or None.
bool vector(PyObject *o, const char *name, at::ScalarType type, int64_t n, const void **p)
{
    *p = nullptr;
    if (o == Py_None) return true;
    const Tensor *t = tensor(o, name);
    if (!t) return false;
    if (t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || (n > 1 && t->stride(0) != 1)) {
        PyErr_Format(PyExc_TypeError, "%s must be a contiguous tensor of %lld elements of %s", name, static_cast<long long>(n), c10::toString(type));
        return false;
    }
    *p = t->data_ptr();
    return true;
}

bool status_word(PyObject *o, int32_t **p) { return vector(o, "dev_status", at::kInt, 1, const_cast<const void **>(reinterpret_cast<void **>(p))); }

// A workspace: 1-D, contiguous, uint8, or None.
bool workspace(PyObject *o, void **p, int64_t *bytes)
{
    *p = nullptr;
    *bytes = 0;
    if (o == Py_None) return true;
    const Tensor *t = tensor(o, "work");
    if (!t) return false;
    if (t->scalar_type() != at::kByte || t->dim() != 1 || !t->is_contiguous()) return raise(PyExc_ValueError, "work", "must be a contiguous 1-D uint8 tensor");
    *p = t->data_ptr();
    *bytes = t->numel();
    return true;
}

// The stream's handle: None is torch's current stream of the tensor's device.
bool stream_of(PyObject *o, const Tensor &t, cudaStream_t &s)
{
    if (o == Py_None) {
        s = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
        return true;
    }
    PyObject *v = PyObject_GetAttrString(o, "cuda_stream");
    if (!v) return false;
    s = static_cast<cudaStream_t>(PyLong_AsVoidPtr(v));
    Py_DECREF(v);
    return !PyErr_Occurred();
}

// The tensor's device is current while this lives (asking which one is costs a fraction of torch's own guard).
class DeviceOf {
public:
    explicit DeviceOf(const Tensor &t)
    {
        if (c10::cuda::current_device() != t.device().index()) guard_.set_index(t.device().index());
    }

private:
    c10::cuda::OptionalCUDAGuard guard_;
};

// Memory that a call allocates belongs to the stream that the call runs on: there, what used a block before has been
// queued before, and what is freed is used again only behind this call's kernels. Outputs, which the caller reads and
// frees on its own stream, are marked as used on that one too (record).
class OnStream {
public:
    OnStream(cudaStream_t launch, const Tensor &like) : here_(c10::cuda::getCurrentCUDAStream(like.device().index()))
    {
        if (here_.stream() != launch) guard_.reset_stream(c10::cuda::getStreamFromExternal(launch, like.device().index()));
    }
    void record(const Tensor &t) const
    {
        if (guard_.current_stream() && t.numel()) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), here_);
    }

private:
    c10::cuda::CUDAStream here_;
    c10::cuda::OptionalCUDAStreamGuard guard_;
};

// A workspace of the call alone: of its stream's memory, and back to it when the call is queued.
class Workspace {
public:
    Workspace() = default;
    Workspace(const Workspace &) = delete;
    ~Workspace()
    {
        if (p_) c10::cuda::CUDACachingAllocator::raw_delete(p_);
    }
    void *get(int64_t bytes, cudaStream_t stream)
    {
        if (bytes > 0) p_ = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(static_cast<size_t>(bytes), stream);
        return p_;
    }

private:
    void *p_ = nullptr;
};

bool integer(PyObject *o, int64_t &v)
{
    v = PyLong_AsLongLong(o);
    return !(v == -1 && PyErr_Occurred());
}

bool integer(PyObject *o, int32_t &v)
{
    int64_t w;
    if (!integer(o, w)) return false;
    v = static_cast<int32_t>(w);
    return v == w || raise(PyExc_OverflowError, "integer", "does not fit 32 bits");
}

bool real(PyObject *o, float &v)
{
    v = static_cast<float>(PyFloat_AsDouble(o));
    return !PyErr_Occurred();
}

// Rows of a sample: all m of them by default, and at most.
bool sample_rows(PyObject *o, int64_t m, int64_t &rows)
{
    const int64_t all = m > 0 ? m : 1;
    if (o == Py_None) {
        rows = all;
        return true;
    }
    if (!integer(o, rows)) return false;
    if (rows > all) rows = all;
    return true;
}

PyObject *status(convrot_status s) { return PyLong_FromLong(s); }

bool count(Py_ssize_t got, Py_ssize_t want)
{
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, got);
    return false;
}

#define REQUIRE(x)                   \
    do {                             \
        if (!(x)) return nullptr;    \
    } while (0)

// Codes: rows that start on 16 bytes. One row needs no leading dimension, but the C side asks for a multiple of 16.
bool codes(PyObject *o, const char *name, int64_t rows, int64_t cols, Matrix &m)
{
    if (!matrix(o, name, at::kFloat8_e4m3fn, rows, cols, m)) return false;
    if (rows <= 1) m.ld = (cols + 15) / 16 * 16;
    return true;
}

int64_t blocks(int64_t v) { return (v + CONVROT_FP8_BLOCK - 1) / CONVROT_FP8_BLOCK; }

// (x or q, x_scale or None, w.q, w.scale, bias, act, out, work, dev_status, stream); x_scale None: x is rows to pack
PyObject *linear(PyObject *const *v, Py_ssize_t n)
{
    REQUIRE(count(n, 10));
    const bool pack = v[1] == Py_None;
    const Tensor *x = tensor(v[0], pack ? "X" : "x.q"), *w = tensor(v[2], "w.q"), *out = tensor(v[6], "out");
    REQUIRE(x && w && out && one_device(v, n, *x));
    if (x->dim() != 2 || w->dim() != 2) {
        raise(PyExc_TypeError, "x and w", "must be 2-D tensors");
        return nullptr;
    }
    convrot_fp8_linear_args a{};
    a.m = x->size(0);
    a.k = x->size(1);
    a.n = w->size(0);
    Matrix mx, ms{nullptr, a.m}, mw, mws, my;
    if (pack) {
        REQUIRE(dtype_of(*x, "X", a.x_dtype) && matrix(v[0], "X", x->scalar_type(), a.m, a.k, mx));
    } else {
        REQUIRE(codes(v[0], "x.q", a.m, a.k, mx) && matrix(v[1], "x.scale", at::kFloat, blocks(a.k), a.m, ms));
    }
    REQUIRE(codes(v[2], "w.q", a.n, a.k, mw) && matrix(v[3], "w.scale", at::kFloat, blocks(a.n), blocks(a.k), mws));
    REQUIRE(dtype_of(*out, "out", a.y_dtype) && matrix(v[6], "out", out->scalar_type(), a.m, a.n, my));
    const void *bias;
    cudaStream_t stream;
    REQUIRE(vector(v[4], "bias", at::kFloat, a.n, &bias) && integer(v[5], a.act) && workspace(v[7], &a.work, &a.work_bytes));
    REQUIRE(status_word(v[8], &a.dev_status) && stream_of(v[9], *out, stream));
    const DeviceOf device(*x);
    a.x = mx.p;
    a.ldx = mx.ld;
    a.x_scale = static_cast<const float *>(ms.p);
    a.ld_x_scale = ms.ld;
    a.w = mw.p;
    a.ldw = mw.ld;
    a.w_scale = static_cast<const float *>(mws.p);
    a.ld_w_scale = mws.ld;
    a.bias = static_cast<const float *>(bias);
    a.y = my.p;
    a.ldy = my.ld;
    Tensor work;
    if (pack && !a.work) {
        a.work_bytes = convrot_fp8_pack_linear_work_bytes(a.m, a.n, a.k);
        if (a.work_bytes) {
            const OnStream allocate(stream, *out);
            work = at::empty({a.work_bytes}, out->options().dtype(at::kByte));
            a.work = work.data_ptr();
        }
    }
    return status(pack ? convrot_fp8_pack_linear(&a, stream) : convrot_fp8_linear(&a, stream));
}

// (X, q, scale, stream)
PyObject *pack_activations(PyObject *const *v, Py_ssize_t n)
{
    REQUIRE(count(n, 4));
    const Tensor *x = tensor(v[0], "X");
    REQUIRE(x && one_device(v, n, *x));
    if (x->dim() != 2) {
        raise(PyExc_TypeError, "X", "must be a 2-D tensor");
        return nullptr;
    }
    const int64_t m = x->size(0), k = x->size(1);
    int32_t dtype;
    Matrix mx, mq, ms;
    cudaStream_t stream;
    REQUIRE(dtype_of(*x, "X", dtype) && matrix(v[0], "X", x->scalar_type(), m, k, mx) && codes(v[1], "q", m, k, mq));
    REQUIRE(matrix(v[2], "scale", at::kFloat, blocks(k), m, ms) && stream_of(v[3], *x, stream));
    const DeviceOf device(*x);
    return status(convrot_fp8_pack_activations(mx.p, dtype, m, k, mx.ld, mq.p, mq.ld, static_cast<float *>(ms.p), ms.ld, stream));
}

// The one type of the parameters that are given: float32 or the tensors' own.
bool param_type(at::ScalarType own, std::initializer_list<PyObject *> all, at::ScalarType &type)
{
    type = at::kFloat;
    for (PyObject *o : all) {
        if (o == Py_None) continue;
        const Tensor *t = tensor(o, "parameters");
        if (!t) return false;
        type = t->scalar_type();
        return type == at::kFloat || type == own || raise(PyExc_TypeError, "parameters", "must be float32 or of x's type");
    }
    return true;
}

// Without a branch y there is nothing that its gate, weight and bias could apply to.
bool branch_for(PyObject *y, std::initializer_list<PyObject *> all)
{
    for (PyObject *o : all)
        if (y == Py_None && o != Py_None) return raise(PyExc_ValueError, "gate, post_weight and post_bias", "belong to a branch y");
    return true;
}

int32_t code_of(at::ScalarType t) { return t == at::kFloat ? CONVROT_F32 : t == at::kBFloat16 ? CONVROT_BF16 : CONVROT_F16; }

// (x, y, gate, scale, shift, rows_per_batch, res_scale, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps,
//  out_h, out_n, q, q_scale, stream)
PyObject *gated_norm(PyObject *const *v, Py_ssize_t n)
{
    REQUIRE(count(n, 19));
    const Tensor *x = tensor(v[0], "x");
    REQUIRE(x && one_device(v, n, *x));
    if (x->dim() != 2) {
        raise(PyExc_TypeError, "x", "must be a 2-D tensor");
        return nullptr;
    }
    REQUIRE(branch_for(v[1], {v[2], v[8], v[9]}));
    convrot_gated_norm_args a{};
    const at::ScalarType t = x->scalar_type();
    at::ScalarType p;
    REQUIRE(dtype_of(*x, "x", a.dtype) && param_type(t, {v[2], v[3], v[4], v[8], v[9], v[11], v[12]}, p));
    a.param_dtype = code_of(p);
    a.m = x->size(0);
    a.d = x->size(1);
    REQUIRE(sample_rows(v[5], a.m, a.rows_per_batch));
    if (a.rows_per_batch < 1) return status(CONVROT_ERR_INVALID_ARG);
    const int64_t m = a.m, d = a.d, batches = (m + a.rows_per_batch - 1) / a.rows_per_batch;
    Matrix mx, my, mg, mc, mf, mh, mn, mq{nullptr, 0}, ms{nullptr, 0};
    cudaStream_t stream;
    REQUIRE(matrix(v[0], "x", t, m, d, mx) && optional_matrix(v[1], "y", t, m, d, my) && optional_matrix(v[2], "gate", p, batches, d, mg));
    REQUIRE(optional_matrix(v[3], "scale", p, batches, d, mc) && optional_matrix(v[4], "shift", p, batches, d, mf));
    REQUIRE(real(v[6], a.res_scale) && integer(v[7], a.post) && vector(v[8], "post_weight", p, d, &a.post_weight));
    REQUIRE(vector(v[9], "post_bias", p, d, &a.post_bias) && integer(v[10], a.pre) && vector(v[11], "pre_weight", p, d, &a.pre_weight));
    REQUIRE(vector(v[12], "pre_bias", p, d, &a.pre_bias) && real(v[13], a.eps));
    REQUIRE(optional_matrix(v[14], "out_h", t, m, d, mh) && optional_matrix(v[15], "out_n", t, m, d, mn));
    if (v[16] != Py_None) REQUIRE(codes(v[16], "q", m, d, mq) && matrix(v[17], "scale", at::kFloat, blocks(d), m, ms));
    REQUIRE(stream_of(v[18], *x, stream));
    const DeviceOf device(*x);
    a.x = mx.p;
    a.ldx = mx.ld;
    a.y = my.p;
    a.ldy = my.ld;
    a.gate = mg.p;
    a.ldgate = mg.ld;
    a.scale = mc.p;
    a.ldscale = mc.ld;
    a.shift = mf.p;
    a.ldshift = mf.ld;
    a.h = mh.p;
    a.ldh = mh.ld;
    a.n = mn.p;
    a.ldn = mn.ld;
    a.q = mq.p;
    a.ldq = mq.ld;
    a.q_scale = static_cast<float *>(ms.p);
    a.ld_q_scale = ms.ld;
    return status(convrot_gated_norm(&a, stream));
}

// (h, y, dh, dn, gate, scale, shift, rows_per_batch, res_scale, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps,
//  work, stream) -> status, or the dict of gradients. They are allocated here, each for itself: whoever
// keeps one of them keeps no more than that.
PyObject *gated_norm_backward(PyObject *const *v, Py_ssize_t n)
{
    REQUIRE(count(n, 18));
    const Tensor *h = tensor(v[0], "h");
    REQUIRE(h && one_device(v, n, *h));
    if (h->dim() != 2) {
        raise(PyExc_TypeError, "h", "must be a 2-D tensor");
        return nullptr;
    }
    REQUIRE(branch_for(v[1], {v[4], v[10], v[11]}));
    convrot_gated_norm_backward_args a{};
    const at::ScalarType t = h->scalar_type();
    at::ScalarType p;
    REQUIRE(dtype_of(*h, "h", a.dtype) && param_type(t, {v[4], v[5], v[6], v[10], v[11], v[13], v[14]}, p));
    a.param_dtype = code_of(p);
    a.m = h->size(0);
    a.d = h->size(1);
    REQUIRE(sample_rows(v[7], a.m, a.rows_per_batch));
    if (a.rows_per_batch < 1) return status(CONVROT_ERR_INVALID_ARG);
    const int64_t m = a.m, d = a.d, batches = (m + a.rows_per_batch - 1) / a.rows_per_batch;
    Matrix mh, my, mdh, mdn, mg, mc, mf;
    cudaStream_t stream;
    REQUIRE(matrix(v[0], "h", t, m, d, mh) && optional_matrix(v[1], "y", t, m, d, my) && optional_matrix(v[2], "dh", t, m, d, mdh));
    REQUIRE(optional_matrix(v[3], "dn", t, m, d, mdn) && optional_matrix(v[4], "gate", p, batches, d, mg));
    REQUIRE(optional_matrix(v[5], "scale", p, batches, d, mc) && optional_matrix(v[6], "shift", p, batches, d, mf));
    REQUIRE(real(v[8], a.res_scale) && integer(v[9], a.post) && vector(v[10], "post_weight", p, d, &a.post_weight));
    REQUIRE(vector(v[11], "post_bias", p, d, &a.post_bias) && integer(v[12], a.pre) && vector(v[13], "pre_weight", p, d, &a.pre_weight));
    REQUIRE(vector(v[14], "pre_bias", p, d, &a.pre_bias) && real(v[15], a.eps));
    REQUIRE(workspace(v[16], &a.work, &a.work_bytes) && stream_of(v[17], *h, stream));
    struct Small {
        PyObject *name;
        PyObject *of;
        bool of_samples;
        float **to;
        Tensor grad;
    };
    static PyObject *const names[7] = {
        PyUnicode_InternFromString("dgate"),     PyUnicode_InternFromString("dscale"),     PyUnicode_InternFromString("dshift"),
        PyUnicode_InternFromString("dpost_weight"), PyUnicode_InternFromString("dpost_bias"), PyUnicode_InternFromString("dpre_weight"),
        PyUnicode_InternFromString("dpre_bias")};
    Small small[7] = {{names[0], v[4], true, &a.dgate, {}},         {names[1], v[5], true, &a.dscale, {}},
                      {names[2], v[6], true, &a.dshift, {}},        {names[3], v[10], false, &a.dpost_weight, {}},
                      {names[4], v[11], false, &a.dpost_bias, {}},  {names[5], v[13], false, &a.dpre_weight, {}},
                      {names[6], v[14], false, &a.dpre_bias, {}}};
    const DeviceOf device(*h);
    const OnStream allocate(stream, *h);
    // (straight from the allocator: a trip through the dispatcher for each costs as much as a launch)
    c10::Allocator *const allocator = c10::cuda::CUDACachingAllocator::get();
    auto fresh = [&](at::IntArrayRef sizes, at::ScalarType type) {
        size_t bytes = c10::elementSize(type);
        for (int64_t n : sizes) bytes *= static_cast<size_t>(n);
        Tensor t = at::detail::make_tensor<c10::TensorImpl>(
            c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes, allocator->allocate(bytes), allocator, true),
            c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
        allocate.record(t);
        return t;
    };
    Tensor dx = fresh({m, d}, t), dy = v[1] != Py_None ? fresh({m, d}, t) : Tensor();
    for (Small &s : small) {
        if (s.of == Py_None) continue;
        s.grad = s.of_samples ? fresh({batches, d}, at::kFloat) : fresh({d}, at::kFloat);
        *s.to = static_cast<float *>(s.grad.data_ptr());
    }
    Workspace work;
    if (v[16] == Py_None) {
        a.work_bytes = convrot_gated_norm_backward_work_bytes(m, d, a.rows_per_batch);
        a.work = work.get(a.work_bytes, stream);
    }
    a.h = mh.p;
    a.ldh = mh.ld;
    a.y = my.p;
    a.ldy = my.ld;
    a.dh = mdh.p;
    a.lddh = mdh.ld;
    a.dn = mdn.p;
    a.lddn = mdn.ld;
    a.gate = mg.p;
    a.ldgate = mg.ld;
    a.scale = mc.p;
    a.ldscale = mc.ld;
    a.dx = dx.data_ptr();
    a.lddx = d;
    a.dy = dy.defined() ? dy.data_ptr() : nullptr;
    a.lddy = d;
    const convrot_status st = convrot_gated_norm_backward(&a, stream);
    if (st != CONVROT_OK) return status(st);
    PyObject *dict = PyDict_New();
    bool ok = dict != nullptr;
    auto put = [&](PyObject *name, Tensor &grad) {
        if (!ok) return;
        PyObject *o = grad.defined() ? THPVariable_Wrap(std::move(grad)) : Py_NewRef(Py_None);
        ok = o && PyDict_SetItem(dict, name, o) == 0;
        Py_XDECREF(o);
    };
    static PyObject *const dx_name = PyUnicode_InternFromString("dx"), *const dy_name = PyUnicode_InternFromString("dy");
    put(dx_name, dx);
    put(dy_name, dy);
    for (Small &s : small) put(s.name, s.grad);
    if (!ok) Py_CLEAR(dict);
    return dict;
}

// A [batch, tokens, heads, head_dim] tensor like `like` but for its heads.
bool heads(PyObject *o, const char *name, const Tensor &like, void **p, int64_t &n, int64_t (&strides)[3])
{
    const Tensor *t = tensor(o, name);
    if (!t) return false;
    if (t->dim() != 4 || t->scalar_type() != like.scalar_type()) return raise(PyExc_TypeError, name, "must be 4-D and of q's type");
    if (t->size(0) != like.size(0) || t->size(1) != like.size(1) || t->size(3) != like.size(3))
        return raise(PyExc_ValueError, name, "must have q's batch, tokens and head_dim");
    if (t->size(3) > 1 && t->stride(3) != 1) return raise(PyExc_ValueError, name, "must have a contiguous last dimension");
    *p = t->data_ptr();
    n = t->size(2);
    for (int i = 0; i < 3; ++i) strides[i] = t->stride(i);
    return true;
}

// (q, k, cos, sin, positions, layout, inverse, out_q, out_k, dev_status, stream)
PyObject *rotary(PyObject *const *v, Py_ssize_t n)
{
    REQUIRE(count(n, 11));
    const Tensor *q = tensor(v[0], "q"), *cos = tensor(v[2], "cos");
    REQUIRE(q && cos && one_device(v, n, *q));
    if (q->dim() != 4 || cos->dim() != 2) {
        raise(PyExc_TypeError, "q and cos", "must be [batch, tokens, heads, head_dim] and [rows, pairs]");
        return nullptr;
    }
    convrot_rotary_args a{};
    REQUIRE(dtype_of(*q, "q", a.dtype));
    a.batch = q->size(0);
    a.tokens = q->size(1);
    if (q->size(3) > INT32_MAX || cos->size(1) > INT32_MAX / 2) return status(CONVROT_ERR_UNSUPPORTED);
    a.head_dim = static_cast<int32_t>(q->size(3));
    a.rot_dim = static_cast<int32_t>(2 * cos->size(1));
    a.table_rows = cos->size(0);
    void *qp, *kp = nullptr, *oq, *ok = nullptr;
    int64_t out_heads;
    REQUIRE(heads(v[0], "q", *q, &qp, a.q_heads, a.q_strides) && heads(v[7], "out_q", *q, &oq, out_heads, a.out_q_strides));
    bool same = out_heads == a.q_heads;
    if (v[1] != Py_None) {
        REQUIRE(heads(v[1], "k", *q, &kp, a.k_heads, a.k_strides) && heads(v[8], "out_k", *q, &ok, out_heads, a.out_k_strides));
        same = same && out_heads == a.k_heads;
    }
    if (!same) {
        raise(PyExc_ValueError, "outputs", "must have as many heads as their inputs");
        return nullptr;
    }
    Matrix mc, ms;
    REQUIRE(matrix(v[2], "cos", at::kFloat, a.table_rows, cos->size(1), mc) && matrix(v[3], "sin", at::kFloat, a.table_rows, cos->size(1), ms));
    if (a.table_rows > 1 && mc.ld != ms.ld) {
        raise(PyExc_ValueError, "cos and sin", "must have the same leading dimension");
        return nullptr;
    }
    if (v[4] != Py_None) {
        const Tensor *t = tensor(v[4], "positions");
        REQUIRE(t);
        if (t->scalar_type() != at::kInt && t->scalar_type() != at::kLong) {
            raise(PyExc_TypeError, "positions", "must be int32 or int64");
            return nullptr;
        }
        const bool shared = t->dim() == 1 && t->size(0) == a.tokens;
        if (!shared && !(t->dim() == 2 && t->size(0) == a.batch && t->size(1) == a.tokens)) {
            raise(PyExc_ValueError, "positions", "must be [batch, tokens] or [tokens]");
            return nullptr;
        }
        if (a.tokens > 1 && t->stride(t->dim() - 1) != 1) {
            raise(PyExc_ValueError, "positions", "must be contiguous along tokens");
            return nullptr;
        }
        a.positions = t->data_ptr();
        a.position_bits = t->scalar_type() == at::kLong ? 64 : 32;
        a.pos_stride = shared ? 0 : t->stride(0);
    }
    const int inverse = PyObject_IsTrue(v[6]);
    cudaStream_t stream;
    REQUIRE(integer(v[5], a.layout) && inverse >= 0 && status_word(v[9], &a.dev_status) && stream_of(v[10], *q, stream));
    const DeviceOf device(*q);
    a.inverse = inverse;
    a.q = qp;
    a.k = kp;
    a.out_q = oq;
    a.out_k = ok;
    a.cos = static_cast<const float *>(mc.p);
    a.sin = static_cast<const float *>(ms.p);
    a.ldt = mc.ld;
    return status(convrot_rotary(&a, stream));
}

// A call as Python makes it. torch's C++ side throws (out of memory, or a tensor without memory of its own, as under
// torch.vmap): what it throws becomes the Python exception that torch itself would raise, and does not leave here.
template <PyObject *(*kCall)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    try {
        return kCall(v, n);
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(linear), METHOD(pack_activations), METHOD(gated_norm), METHOD(gated_norm_backward), METHOD(rotary),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
