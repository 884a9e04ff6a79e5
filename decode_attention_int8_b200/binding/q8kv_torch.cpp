// q8kv_torch.cpp -- the compiled half of the serving operators' binding (_serving.py): checks of
// the torch tensors' type, shape, device and layout, and the call of the C entry point with
// their addresses and the stream.
//
// Why compiled: these operators run once per layer and step on a few sequences, where the
// kernel takes 3 to 6 us. With the same checks in Python and the call through ctypes the host
// needed 9 to 14 us per call (about 0.5 us per tensor checked and 0.13 us per argument passed).
//
// The library itself is not linked: bind() gets the addresses of its entry points from the
// loaded library. Functions return the q8kv_status of the call.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <sstream>
#include <string>

#include "q8kv.h"

namespace {

struct Refused {
    PyObject *type; // the Python exception
    std::string what;
};

decltype(&q8kv_decode_attn_lse) g_lse;
decltype(&q8kv_attn_mass) g_mass;
decltype(&q8kv_evict) g_evict;
decltype(&q8kv_rope_cache_write) g_rope;
decltype(&q8kv_verify_draft) g_verify;

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        throw Refused{PyExc_TypeError, std::string(name) + " must be a torch.Tensor"};
    return THPVariable_Unpack(o);
}

template <typename Sizes>
std::string text(const Sizes &sizes)
{
    std::ostringstream s;
    s << "(";
    for (auto it = sizes.begin(); it != sizes.end(); ++it)
        s << (it == sizes.begin() ? "" : ", ") << *it;
    s << ")";
    return s.str();
}

[[noreturn]] void refuse(const at::Tensor &t, const char *name, const std::string &wanted)
{
    std::ostringstream s;
    s << name << ": expected " << wanted << ", got " << t.dtype().name() << " "
      << text(t.sizes()) << " strides " << text(t.strides()) << " on " << t.device();
    throw Refused{PyExc_ValueError, s.str()};
}

// The tensor that says where a call runs and what its sizes are.
const at::Tensor &sized(PyObject *o, const char *name, int64_t dims)
{
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != dims)
        refuse(t, name, std::to_string(dims) + " dimensions");
    return t;
}

const at::Tensor &leading(PyObject *o, const char *name, int64_t dims)
{
    const at::Tensor &t = sized(o, name, dims);
    if (!t.is_cuda())
        refuse(t, name, "a CUDA tensor");
    return t;
}

// Address of a contiguous tensor of this type and shape on the call's device.
template <typename T>
T *addr(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape,
        const at::Device &dev)
{
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || t.device() != dev ||
        !t.is_contiguous()) {
        std::ostringstream s;
        s << "a contiguous " << c10::toString(type) << " tensor " << text(shape) << " on " << dev;
        refuse(t, name, s.str());
    }
    return static_cast<T *>(t.data_ptr());
}

int whole(int64_t x, const char *name)
{
    if (x < INT32_MIN || x > INT32_MAX)
        throw Refused{PyExc_ValueError, std::string(name) + ": larger than a C int"};
    return static_cast<int>(x);
}

int integer(PyObject *o, const char *name)
{
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{PyExc_TypeError, std::string(name) + " must be an integer"};
    }
    return whole(x, name);
}

float real(PyObject *o, const char *name)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{PyExc_TypeError, std::string(name) + " must be a number"};
    }
    return static_cast<float>(x);
}

int dtype_code(const at::Tensor &t, const char *name)
{
    switch (t.scalar_type()) {
    case at::kFloat:
        return Q8KV_F32;
    case at::kHalf:
        return Q8KV_F16;
    case at::kBFloat16:
        return Q8KV_BF16;
    default:
        refuse(t, name, "float32, float16 or bfloat16");
    }
}

// The stream argument: None (the device's current stream), a torch stream or a handle.
cudaStream_t stream_of(PyObject *o, const at::Device &dev)
{
    if (o == Py_None)
        return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) {
        PyErr_Clear();
        h = PyNumber_Long(o);
    }
    void *p = h ? PyLong_AsVoidPtr(h) : nullptr;
    Py_XDECREF(h);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{PyExc_TypeError, "stream must be a torch.cuda.Stream or its handle"};
    }
    return static_cast<cudaStream_t>(p);
}

// Rows [n][heads][D] whose last two dimensions have no gaps: address and token stride.
const void *token_rows(PyObject *o, const char *name, at::ScalarType type, int64_t n,
                       int64_t heads, int64_t D, const at::Device &dev, long long &stride)
{
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef({n, heads, D}) ||
        t.device() != dev || (D > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != D)) {
        std::ostringstream s;
        s << "a " << c10::toString(type) << " tensor (" << n << ", " << heads << ", " << D
          << ") on " << dev << " with contiguous rows";
        refuse(t, name, s.str());
    }
    stride = n > 1 ? t.stride(0) : heads * D;
    if (stride < heads * D && t.numel() > 0) // (an expanded token: the library's 0 means no gap)
        refuse(t, name, "a token stride of at least " + std::to_string(heads * D));
    return t.data_ptr();
}

// Probabilities [B][rows][vocab]: address and elements between rows.
const void *prob_rows(PyObject *o, const char *name, at::ScalarType type, int64_t B, int64_t rows,
                      int64_t vocab, const at::Device &dev, long long &stride)
{
    const at::Tensor &t = tensor(o, name);
    bool ok = t.scalar_type() == type && t.sizes() == at::IntArrayRef({B, rows, vocab}) &&
              t.device() == dev && (vocab <= 1 || t.stride(2) == 1);
    if (ok) {
        stride = rows > 1 ? t.stride(1) : (B > 1 ? t.stride(0) : vocab);
        ok = (rows <= 1 || B <= 1 || t.stride(0) == rows * stride) &&
             (stride >= vocab || t.numel() == 0); // (expanded rows: the library's 0 means no gap)
    }
    if (!ok) {
        std::ostringstream s;
        s << "a " << c10::toString(type) << " tensor (" << B << ", " << rows << ", " << vocab
          << ") on " << dev << " with contiguous, evenly spaced rows";
        refuse(t, name, s.str());
    }
    return t.data_ptr();
}

// Runs `call` on the device of the call's tensors, whichever is current.
template <typename Call>
PyObject *launch(const at::Device &dev, Call call)
{
    q8kv_status st;
    {
        c10::cuda::OptionalCUDAGuard guard;
        if (dev.index() != c10::cuda::current_device())
            guard.set_device(dev);
        st = call();
    }
    return PyLong_FromLong(static_cast<long>(st));
}

template <typename Body>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, Body body)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject *decode_attn_lse(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 12, [&] {
        const at::Tensor &q = leading(a[2], "q", 4), &k = sized(a[3], "k_blocks", 4);
        const at::Tensor &table = sized(a[7], "block_table", 2);
        const at::Device dev = q.device();
        const int64_t B = q.size(0), nq = q.size(1), Hq = q.size(2), D = q.size(3);
        const int64_t P = k.size(0), bs = k.size(1), Hk = k.size(2), m = table.size(1);
        void *ws = nullptr;
        size_t ws_bytes = 0;
        if (a[10] != Py_None) {
            const at::Tensor &w = tensor(a[10], "workspace");
            if (w.device() != dev || !w.is_contiguous())
                refuse(w, "workspace", "a contiguous tensor on the call's device");
            ws = w.data_ptr();
            ws_bytes = w.nbytes();
        }
        float *out = addr<float>(a[0], "out", at::kFloat, {B, nq, Hq, D}, dev);
        float *lse = addr<float>(a[1], "lse", at::kFloat, {B, nq, Hq}, dev);
        const float *qp = addr<float>(a[2], "q", at::kFloat, {B, nq, Hq, D}, dev);
        const int8_t *kp = addr<int8_t>(a[3], "k_blocks", at::kChar, {P, bs, Hk, D}, dev);
        const int8_t *vp = addr<int8_t>(a[4], "v_blocks", at::kChar, {P, bs, Hk, D}, dev);
        const float *ks = addr<float>(a[5], "kscale", at::kFloat, {P, bs, Hk}, dev);
        const float *vs = addr<float>(a[6], "vscale", at::kFloat, {P, bs, Hk}, dev);
        const int32_t *bt = addr<int32_t>(a[7], "block_table", at::kInt, {B, m}, dev);
        const int32_t *lens = addr<int32_t>(a[8], "seq_lens", at::kInt, {B}, dev);
        const float scale = real(a[9], "scale");
        const cudaStream_t st = stream_of(a[11], dev);
        const int size[8] = {whole(B, "batch"),   whole(nq, "n_queries"), whole(Hq, "heads"),
                             whole(Hk, "heads"),  whole(D, "head_dim"),   whole(bs, "block_size"),
                             whole(m, "max_blocks"), whole(P, "num_blocks")};
        return launch(dev, [&] {
            return g_lse(out, lse, qp, kp, vp, ks, vs, bt, lens, size[0], size[1], size[2], size[3],
                         size[4], size[5], size[6], size[7], scale, ws, ws_bytes, st);
        });
    });
}

PyObject *attn_mass(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&] {
        const at::Tensor &q = leading(a[1], "q", 4), &k = sized(a[3], "k_blocks", 4);
        const at::Tensor &table = sized(a[5], "block_table", 2);
        const at::Device dev = q.device();
        const int64_t B = q.size(0), nq = q.size(1), Hq = q.size(2), D = q.size(3);
        const int64_t P = k.size(0), bs = k.size(1), Hk = k.size(2), m = table.size(1);
        float *mass = addr<float>(a[0], "mass", at::kFloat, {B, Hk, m * bs}, dev);
        const float *qp = addr<float>(a[1], "q", at::kFloat, {B, nq, Hq, D}, dev);
        const float *lse = addr<float>(a[2], "lse", at::kFloat, {B, nq, Hq}, dev);
        const int8_t *kp = addr<int8_t>(a[3], "k_blocks", at::kChar, {P, bs, Hk, D}, dev);
        const float *ks = addr<float>(a[4], "kscale", at::kFloat, {P, bs, Hk}, dev);
        const int32_t *bt = addr<int32_t>(a[5], "block_table", at::kInt, {B, m}, dev);
        const int32_t *lens = addr<int32_t>(a[6], "seq_lens", at::kInt, {B}, dev);
        const float scale = real(a[7], "scale"), decay = real(a[8], "decay");
        const cudaStream_t st = stream_of(a[9], dev);
        const int size[8] = {whole(B, "batch"),   whole(nq, "n_queries"), whole(Hq, "heads"),
                             whole(Hk, "heads"),  whole(D, "head_dim"),   whole(bs, "block_size"),
                             whole(m, "max_blocks"), whole(P, "num_blocks")};
        return launch(dev, [&] {
            return g_mass(mass, qp, lse, kp, ks, bt, lens, size[0], size[1], size[2], size[3],
                          size[4], size[5], size[6], size[7], scale, decay, st);
        });
    });
}

PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 14, [&] {
        const at::Tensor &k = leading(a[0], "k_blocks", 4), &kept_t = sized(a[5], "kept", 3);
        const at::Tensor &table = sized(a[8], "block_table", 2);
        const at::Tensor &new_table = sized(a[10], "new_block_table", 2);
        const at::Device dev = k.device();
        const int64_t P = k.size(0), bs = k.size(1), Hk = k.size(2), D = k.size(3);
        const int64_t B = table.size(0), m = table.size(1), nm = new_table.size(1);
        const int64_t keep = kept_t.size(2);
        int8_t *kp = addr<int8_t>(a[0], "k_blocks", at::kChar, {P, bs, Hk, D}, dev);
        int8_t *vp = addr<int8_t>(a[1], "v_blocks", at::kChar, {P, bs, Hk, D}, dev);
        float *ks = addr<float>(a[2], "kscale", at::kFloat, {P, bs, Hk}, dev);
        float *vs = addr<float>(a[3], "vscale", at::kFloat, {P, bs, Hk}, dev);
        float *new_mass = addr<float>(a[4], "new_mass", at::kFloat, {B, Hk, nm * bs}, dev);
        int32_t *kept = addr<int32_t>(a[5], "kept", at::kInt, {B, Hk, keep}, dev);
        int32_t *new_lens = addr<int32_t>(a[6], "new_lens", at::kInt, {B}, dev);
        const float *mass = addr<float>(a[7], "mass", at::kFloat, {B, Hk, m * bs}, dev);
        const int32_t *bt = addr<int32_t>(a[8], "block_table", at::kInt, {B, m}, dev);
        const int32_t *lens = addr<int32_t>(a[9], "seq_lens", at::kInt, {B}, dev);
        const int32_t *nbt = addr<int32_t>(a[10], "new_block_table", at::kInt, {B, nm}, dev);
        const int sink = integer(a[11], "sink"), recent = integer(a[12], "recent");
        const cudaStream_t st = stream_of(a[13], dev);
        const int size[8] = {whole(B, "batch"),      whole(Hk, "heads"),
                             whole(D, "head_dim"),   whole(bs, "block_size"),
                             whole(m, "max_blocks"), whole(nm, "new max_blocks"),
                             whole(P, "num_blocks"), whole(keep, "keep")};
        return launch(dev, [&] {
            return g_evict(kp, vp, ks, vs, new_mass, kept, new_lens, mass, bt, lens, nbt, size[0],
                           size[1], size[2], size[3], size[4], size[5], size[6], size[7], sink,
                           recent, st);
        });
    });
}

PyObject *rope_cache_write(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 14, [&] {
        const at::Tensor &out = leading(a[0], "q_out", 3), &k = sized(a[1], "k_blocks", 4);
        const at::Tensor &q = tensor(a[5], "q_new"), &pos = sized(a[9], "positions", 2);
        const at::Tensor &table = sized(a[10], "cos_sin", 2);
        const at::Device dev = out.device();
        const int64_t tokens = out.size(0), Hq = out.size(1);
        const int64_t P = k.size(0), bs = k.size(1), Hk = k.size(2), D = k.size(3);
        const int64_t axes = pos.size(0), top = table.size(0), rot = table.size(1);
        const int code = dtype_code(q, "q_new");
        const at::ScalarType type = q.scalar_type();
        float *qo = addr<float>(a[0], "q_out", at::kFloat, {tokens, Hq, D}, dev);
        int8_t *kp = addr<int8_t>(a[1], "k_blocks", at::kChar, {P, bs, Hk, D}, dev);
        int8_t *vp = addr<int8_t>(a[2], "v_blocks", at::kChar, {P, bs, Hk, D}, dev);
        float *ks = addr<float>(a[3], "kscale", at::kFloat, {P, bs, Hk}, dev);
        float *vs = addr<float>(a[4], "vscale", at::kFloat, {P, bs, Hk}, dev);
        long long q_stride, k_stride, v_stride;
        const void *qn = token_rows(a[5], "q_new", type, tokens, Hq, D, dev, q_stride);
        const void *kn = token_rows(a[6], "k_new", type, tokens, Hk, D, dev, k_stride);
        const void *vn = token_rows(a[7], "v_new", type, tokens, Hk, D, dev, v_stride);
        if (k_stride != v_stride)
            throw Refused{PyExc_ValueError, "k_new and v_new must have the same token stride"};
        const int64_t *slots = addr<int64_t>(a[8], "slot_mapping", at::kLong, {tokens}, dev);
        const int32_t *ps = addr<int32_t>(a[9], "positions", at::kInt, {axes, tokens}, dev);
        const float *cs = addr<float>(a[10], "cos_sin", at::kFloat, {top, rot}, dev);
        const uint8_t *axis = nullptr;
        if (a[11] != Py_None) { // (bytes)
            char *p;
            Py_ssize_t len;
            if (PyBytes_AsStringAndSize(a[11], &p, &len) != 0) {
                PyErr_Clear();
                throw Refused{PyExc_TypeError, "pair_axis must be bytes or a sequence of integers"};
            }
            if (len != rot / 2)
                throw Refused{PyExc_ValueError, "pair_axis needs " + std::to_string(rot / 2) +
                                                    " entries, got " + std::to_string(len)};
            axis = reinterpret_cast<const uint8_t *>(p);
        }
        const int adjacent = PyObject_IsTrue(a[12]);
        if (adjacent < 0) {
            PyErr_Clear();
            throw Refused{PyExc_TypeError, "adjacent must be true or false"};
        }
        const cudaStream_t st = stream_of(a[13], dev);
        const int size[9] = {whole(tokens, "tokens"), whole(axes, "axes"),
                             whole(Hq, "heads"),      whole(Hk, "heads"),
                             whole(D, "head_dim"),    whole(rot, "rotary_dim"),
                             whole(top, "positions"), whole(bs, "block_size"),
                             whole(P, "num_blocks")};
        return launch(dev, [&] {
            return g_rope(qo, kp, vp, ks, vs, qn, kn, vn, slots, ps, cs, axis, size[0], size[1],
                          size[2], size[3], size[4], size[5], adjacent, size[6],
                          static_cast<q8kv_dtype>(code), size[7], size[8], q_stride, k_stride, st);
        });
    });
}

PyObject *verify_draft(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const at::Tensor &t = leading(a[2], "target_probs", 3);
        const at::Device dev = t.device();
        const int64_t B = t.size(0), drafts = t.size(1) - 1, vocab = t.size(2);
        const int code = dtype_code(t, "target_probs");
        const at::ScalarType type = t.scalar_type();
        long long ts = 0, ds = 0;
        const void *tp = prob_rows(a[2], "target_probs", type, B, drafts + 1, vocab, dev, ts);
        const void *dp = nullptr;
        if (a[3] != Py_None && drafts > 0)
            dp = prob_rows(a[3], "draft_probs", type, B, drafts, vocab, dev, ds);
        int32_t *accepted = addr<int32_t>(a[0], "n_accepted", at::kInt, {B}, dev);
        int32_t *tokens = addr<int32_t>(a[1], "tokens", at::kInt, {B, drafts + 1}, dev);
        const int32_t *drafted = addr<int32_t>(a[4], "draft_tokens", at::kInt, {B, drafts}, dev);
        const float *uni = addr<float>(a[5], "uniforms", at::kFloat, {B, drafts + 1}, dev);
        const int32_t *counts =
            a[6] == Py_None ? nullptr : addr<int32_t>(a[6], "n_drafts", at::kInt, {B}, dev);
        const cudaStream_t st = stream_of(a[7], dev);
        const int size[3] = {whole(B, "batch"), whole(drafts, "drafts"), whole(vocab, "vocab")};
        return launch(dev, [&] {
            return g_verify(accepted, tokens, tp, dp, drafted, counts, uni, size[0], size[1],
                            size[2], ts, ds, static_cast<q8kv_dtype>(code), st);
        });
    });
}

// bind(lse, mass, evict, rope, verify): addresses of the library's entry points
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 5, [&]() -> PyObject * {
        void *p[5];
        for (int i = 0; i < 5; ++i) {
            p[i] = PyLong_AsVoidPtr(a[i]);
            if (!p[i]) {
                PyErr_Clear();
                throw Refused{PyExc_ValueError, "bind: not an address"};
            }
        }
        g_lse = reinterpret_cast<decltype(g_lse)>(p[0]);
        g_mass = reinterpret_cast<decltype(g_mass)>(p[1]);
        g_evict = reinterpret_cast<decltype(g_evict)>(p[2]);
        g_rope = reinterpret_cast<decltype(g_rope)>(p[3]);
        g_verify = reinterpret_cast<decltype(g_verify)>(p[4]);
        Py_RETURN_NONE;
    });
}

#define METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(bind),  METHOD(decode_attn_lse),  METHOD(attn_mass),
                           METHOD(evict), METHOD(rope_cache_write), METHOD(verify_draft),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_q8kv_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__q8kv_torch()
{
    return PyModule_Create(&g_module);
}
