// ropekv_bind.cpp -- Python binding of libropekv_serving.so (include/ropekv_serving.h,
// include/ropekv_sequence.h) for torch tensors: checks type, device, layout and shape agreement, reads
// sizes and addresses, calls the C entry point on the current (or given) stream
// and returns its status. It computes nothing. A module of its own, because the
// checks of a call's ten tensors in Python take longer (20 us) than a decode-sized
// launch; here the whole call takes about 2 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <string>

#include "ropekv_sequence.h"
#include "ropekv_serving.h"

namespace {

struct Refusal {
    PyObject* type;
    std::string text;
};

[[noreturn]] void value_error(const std::string& text) { throw Refusal{PyExc_ValueError, text}; }
[[noreturn]] void type_error(const std::string& text) { throw Refusal{PyExc_TypeError, text}; }

struct PythonError {};   // a Python exception is already set

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o))
        type_error(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

const at::Tensor* optional(PyObject* o, const char* name)
{
    return o == Py_None ? nullptr : &tensor(o, name);
}

void on_device(const at::Tensor& t, const char* name, at::Device dev)
{
    if (!dev.is_cuda())
        value_error(std::string(name) + " is on " + t.device().str() + ", expected a CUDA device");
    if (t.device() != dev)
        value_error(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
}

void has_type(const at::Tensor& t, const char* name, at::ScalarType type)
{
    if (t.scalar_type() != type)
        type_error(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + ", expected " +
                   c10::toString(type));
}

template <typename T = void>
T* dense(const at::Tensor& t, const char* name, at::ScalarType type, at::Device dev)
{
    has_type(t, name, type);
    on_device(t, name, dev);
    if (!t.is_contiguous())
        value_error(std::string(name) + " must be contiguous");
    return static_cast<T*>(t.data_ptr());
}

template <typename T = void>
T* dense(const at::Tensor* t, const char* name, at::ScalarType type, at::Device dev)
{
    return t ? dense<T>(*t, name, type, dev) : nullptr;
}

// Address and token stride of a [T, H, D] float16 tensor with dense heads and dims.
const uint16_t* rows(const at::Tensor& t, const char* name, at::Device dev, int64_t& stride)
{
    has_type(t, name, at::kHalf);
    on_device(t, name, dev);
    if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != t.size(2)))
        value_error(std::string(name) + ": heads and dims must be dense (strides (*, D, 1))");
    stride = t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
    return static_cast<const uint16_t*>(t.data_ptr());
}

int format_of(const at::Tensor& t, const char* name, bool eight_bit_only)
{
    switch (t.scalar_type()) {
    case at::kHalf:
        if (!eight_bit_only)
            return ROPEKV_CACHE_F16;
        break;
    case at::kFloat8_e4m3fn: return ROPEKV_CACHE_E4M3;
    case at::kChar: return ROPEKV_CACHE_INT8;
    default: break;
    }
    type_error(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + ", expected " +
               (eight_bit_only ? "" : "float16, ") + "float8_e4m3fn or int8");
}

int32_t small(int64_t n, const char* what)
{
    if (n > INT32_MAX || n < INT32_MIN)
        value_error(std::string(what) + " is too large");
    return (int32_t)n;
}

int32_t whole(PyObject* o, const char* name)
{
    const long long n = PyLong_AsLongLong(o);
    if (n == -1 && PyErr_Occurred())
        throw PythonError{};
    return small(n, name);
}

bool is(const at::Tensor& t, std::initializer_list<int64_t> shape)
{
    return t.sizes() == c10::IntArrayRef(shape);
}

// The given torch.cuda.Stream, or the current one of the device.
c10::cuda::CUDAStream stream_of(PyObject* o, at::Device dev)
{
    if (o == Py_None)
        return c10::cuda::getCurrentCUDAStream(dev.index());
    int64_t v[3];
    const char* names[3] = {"stream_id", "device_index", "device_type"};
    for (int i = 0; i < 3; ++i) {
        PyObject* x = PyObject_GetAttrString(o, names[i]);
        if (!x)
            throw PythonError{};
        v[i] = PyLong_AsLongLong(x);
        Py_DECREF(x);
        if (v[i] == -1 && PyErr_Occurred())
            throw PythonError{};
    }
    if (v[1] != dev.index())
        value_error("stream is on device " + std::to_string(v[1]) + ", expected " + dev.str());
    return c10::cuda::CUDAStream::unpack3(v[0], (c10::DeviceIndex)v[1], (c10::DeviceType)v[2]);
}

struct WriteShape {
    int32_t T, Hq, Hkv, D;
};

WriteShape check_write(const char* fn, const at::Tensor& cosSin, const at::Tensor& q,
                       const at::Tensor& k, const at::Tensor& v, const at::Tensor& slots,
                       const at::Tensor& keyCache, const at::Tensor& valueCache,
                       const at::Tensor& qOut)
{
    if (q.dim() != 3 || k.dim() != 3 || keyCache.dim() != 4 || cosSin.dim() != 2)
        value_error("cos_sin [rows,r], q [T,Hq,D], k [T,Hkv,D], key_cache "
                    "[blocks,block_size,Hkv,D] expected");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
    if (!is(k, {T, Hkv, D}) || !is(v, {T, Hkv, D}) || !is(slots, {T}) || keyCache.size(2) != Hkv ||
        keyCache.size(3) != D || valueCache.sizes() != keyCache.sizes() || !is(qOut, {T, Hq, D}))
        value_error(std::string("inconsistent shapes for ") + fn);
    return {small(T, "T"), small(Hq, "Hq"), small(Hkv, "Hkv"), small(D, "D")};
}

template <typename F>
int on_stream(at::Device dev, F&& call)
{
    const c10::cuda::CUDAGuard guard(dev);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return rc;
}

// mrope(cos_sin, positions, freq_axis, q, k, v, slots, key_cache, value_cache, q_out, k_out, style, stream)
int mrope(PyObject* const* x)
{
    const at::Tensor &cs = tensor(x[0], "cos_sin"), &pos = tensor(x[1], "positions"),
                     &axis = tensor(x[2], "freq_axis"), &q = tensor(x[3], "q"), &k = tensor(x[4], "k"),
                     &v = tensor(x[5], "v"), &slots = tensor(x[6], "slot_mapping"),
                     &kc = tensor(x[7], "key_cache"), &vc = tensor(x[8], "value_cache"),
                     &qo = tensor(x[9], "q_out");
    const at::Tensor* ko = optional(x[10], "k_out");
    if (pos.dim() != 2)
        value_error("positions [axes, T] expected");
    const WriteShape s = check_write("rope_write_kv_mrope", cs, q, k, v, slots, kc, vc, qo);
    if (pos.size(1) != s.T)
        value_error("inconsistent shapes for rope_write_kv_mrope");
    if (ko && !is(*ko, {s.T, s.Hkv, s.D}))
        value_error("k_out [T, Hkv, D] expected");
    if (axis.scalar_type() != at::kInt || !axis.device().is_cpu() || !is(axis, {cs.size(1) / 2}) ||
        !axis.is_contiguous())
        value_error("freq_axis must be a contiguous int32 CPU tensor of r/2 elements");
    const at::Device dev = q.device();
    int64_t qs, ks, vs;
    const uint16_t *qp = rows(q, "q", dev, qs), *kp = rows(k, "k", dev, ks), *vp = rows(v, "v", dev, vs);
    const float* csp = dense<float>(cs, "cos_sin", at::kFloat, dev);
    const int64_t *pp = dense<int64_t>(pos, "positions", at::kLong, dev),
                  *sp = dense<int64_t>(slots, "slot_mapping", at::kLong, dev);
    uint16_t *kcp = dense<uint16_t>(kc, "key_cache", at::kHalf, dev),
             *vcp = dense<uint16_t>(vc, "value_cache", at::kHalf, dev),
             *qop = dense<uint16_t>(qo, "q_out", at::kHalf, dev),
             *kop = dense<uint16_t>(ko, "k_out", at::kHalf, dev);
    const int32_t* ap = static_cast<const int32_t*>(axis.data_ptr());
    const int32_t axes = small(pos.size(0), "axes"), r = small(cs.size(1), "r"), n = small(cs.size(0), "rows"),
                  bs = small(kc.size(1), "block_size"), style = whole(x[11], "style");
    const auto st = stream_of(x[12], dev);
    return on_stream(dev, [&] {
        return rope_write_kv_mrope(csp, pp, ap, axes, qp, qs, kp, ks, vp, vs, sp, kcp, vcp, qop, kop,
                                   s.T, s.Hq, s.Hkv, s.D, r, n, kc.size(0), bs, style, st.stream());
    });
}

// quant(cos_sin, positions, q, k, v, slots, key_cache, value_cache, key_scales, value_scales, q_out, style, stream)
int quant(PyObject* const* x)
{
    const at::Tensor &cs = tensor(x[0], "cos_sin"), &pos = tensor(x[1], "positions"),
                     &q = tensor(x[2], "q"), &k = tensor(x[3], "k"), &v = tensor(x[4], "v"),
                     &slots = tensor(x[5], "slot_mapping"), &kc = tensor(x[6], "key_cache"),
                     &vc = tensor(x[7], "value_cache"), &ksc = tensor(x[8], "key_scales"),
                     &vsc = tensor(x[9], "value_scales"), &qo = tensor(x[10], "q_out");
    const WriteShape s = check_write("rope_write_kv_slot_mapping_quant", cs, q, k, v, slots, kc, vc, qo);
    if (!is(pos, {s.T}))
        value_error("inconsistent shapes for rope_write_kv_slot_mapping_quant");
    if (!is(ksc, {kc.size(0), s.Hkv, kc.size(1)}) || vsc.sizes() != ksc.sizes())
        value_error("key_scales, value_scales [blocks, Hkv, block_size] expected");
    const int fmt = format_of(kc, "key_cache", true);
    const at::Device dev = q.device();
    int64_t qs, ks, vs;
    const uint16_t *qp = rows(q, "q", dev, qs), *kp = rows(k, "k", dev, ks), *vp = rows(v, "v", dev, vs);
    const float* csp = dense<float>(cs, "cos_sin", at::kFloat, dev);
    const int64_t *pp = dense<int64_t>(pos, "positions", at::kLong, dev),
                  *sp = dense<int64_t>(slots, "slot_mapping", at::kLong, dev);
    uint8_t *kcp = dense<uint8_t>(kc, "key_cache", kc.scalar_type(), dev),
            *vcp = dense<uint8_t>(vc, "value_cache", kc.scalar_type(), dev);
    float *kscp = dense<float>(ksc, "key_scales", at::kFloat, dev),
          *vscp = dense<float>(vsc, "value_scales", at::kFloat, dev);
    uint16_t* qop = dense<uint16_t>(qo, "q_out", at::kHalf, dev);
    const int32_t r = small(cs.size(1), "r"), n = small(cs.size(0), "rows"),
                  bs = small(kc.size(1), "block_size"), style = whole(x[11], "style");
    const auto st = stream_of(x[12], dev);
    return on_stream(dev, [&] {
        return rope_write_kv_slot_mapping_quant(csp, pp, qp, qs, kp, ks, vp, vs, sp, kcp, vcp, kscp, vscp,
                                                qop, s.T, s.Hq, s.Hkv, s.D, r, n, kc.size(0), bs, fmt,
                                                style, st.stream());
    });
}

struct Pool {
    int32_t pages, tpp, Hkv, D, fmt, B, M;
};

Pool check_pool(const at::Tensor& cache, const at::Tensor* scales, const at::Tensor& table)
{
    if (cache.dim() != 5 || cache.size(0) != 2 || table.dim() != 3 || table.size(1) != 2)
        value_error("kv_cache [2,P,TPP,Hkv,D] and page_table [B,2,M] expected");
    const int fmt = format_of(cache, "kv_cache", false);
    if (fmt == ROPEKV_CACHE_F16) {
        if (scales)
            value_error("a float16 cache has no kv_scales");
    } else if (!scales || !is(*scales, {2, cache.size(1), cache.size(3), cache.size(2)})) {
        value_error("kv_scales [2, P, Hkv, TPP] expected for an 8-bit cache");
    }
    return {small(cache.size(1), "P"), small(cache.size(2), "TPP"), small(cache.size(3), "Hkv"),
            small(cache.size(4), "D"), fmt, small(table.size(0), "B"), small(table.size(2), "M")};
}

// read(kv_cache, page_table, row_positions, row_sequences, k_out, v_out, kv_scales, stream)
int read(PyObject* const* x)
{
    const at::Tensor &cache = tensor(x[0], "kv_cache"), &table = tensor(x[1], "page_table"),
                     &pos = tensor(x[2], "row_positions"), &seq = tensor(x[3], "row_sequences"),
                     &ko = tensor(x[4], "k_out"), &vo = tensor(x[5], "v_out");
    const at::Tensor* scales = optional(x[6], "kv_scales");
    const Pool p = check_pool(cache, scales, table);
    if (pos.dim() != 1 || seq.sizes() != pos.sizes() || !is(ko, {pos.size(0), p.Hkv, p.D}) ||
        vo.sizes() != ko.sizes())
        value_error("row_positions, row_sequences [N] and k_out, v_out [N, Hkv, D] expected");
    const at::Device dev = cache.device();
    const void* cp = dense(cache, "kv_cache", cache.scalar_type(), dev);
    const float* sp = dense<float>(scales, "kv_scales", at::kFloat, dev);
    const int32_t *tp = dense<int32_t>(table, "page_table", at::kInt, dev),
                  *pp = dense<int32_t>(pos, "row_positions", at::kInt, dev),
                  *qp = dense<int32_t>(seq, "row_sequences", at::kInt, dev);
    uint16_t *kop = dense<uint16_t>(ko, "k_out", at::kHalf, dev), *vop = dense<uint16_t>(vo, "v_out", at::kHalf, dev);
    const int32_t n = small(pos.size(0), "N");
    const auto st = stream_of(x[7], dev);
    return on_stream(dev, [&] {
        return paged_kv_read(cp, sp, tp, pp, qp, kop, vop, n, p.B, p.Hkv, p.D, p.pages, p.M, p.tpp,
                             p.fmt, st.stream());
    });
}

ropekv_attention_dims attention_dims(const at::Tensor& q, const at::Tensor& cache,
                                     const at::Tensor* scales, const at::Tensor* prefixTable,
                                     PyObject* prefixLen, const at::Tensor& table)
{
    if (q.dim() != 4)
        value_error("q [B, S, Hq, D] expected");
    const Pool p = check_pool(cache, scales, table);
    if (q.size(0) != p.B || q.size(3) != p.D)
        value_error("q does not match page_table and kv_cache");
    if (prefixTable && (prefixTable->dim() != 2 || prefixTable->size(0) != 2))
        value_error("prefix_table [2, prefix pages] expected");
    return {p.B, small(q.size(1), "S"), small(q.size(2), "Hq"), p.Hkv, p.D, p.pages, p.tpp, p.M,
            whole(prefixLen, "prefix_len"), prefixTable ? small(prefixTable->size(1), "prefix pages") : 0,
            p.fmt};
}

// attention_workspace(q, kv_cache, prefix_table, prefix_len, page_table, kv_scales)
int64_t attention_workspace(PyObject* const* x)
{
    const ropekv_attention_dims d = attention_dims(tensor(x[0], "q"), tensor(x[1], "kv_cache"),
                                                   optional(x[5], "kv_scales"), optional(x[2], "prefix_table"),
                                                   x[3], tensor(x[4], "page_table"));
    return paged_attention_workspace_size(&d);
}

// attention(q, kv_cache, prefix_table, prefix_len, page_table, kv_lens, out, lse, kv_scales, sm_scale, workspace, stream)
int attention(PyObject* const* x)
{
    const at::Tensor &q = tensor(x[0], "q"), &cache = tensor(x[1], "kv_cache"),
                     &table = tensor(x[4], "page_table"), &lens = tensor(x[5], "kv_lens"),
                     &out = tensor(x[6], "out");
    const at::Tensor *prefix = optional(x[2], "prefix_table"), *lse = optional(x[7], "lse"),
                     *scales = optional(x[8], "kv_scales"), *given = optional(x[10], "workspace");
    const ropekv_attention_dims d = attention_dims(q, cache, scales, prefix, x[3], table);
    if (!is(lens, {d.batch}) || out.sizes() != q.sizes() ||
        (lse && !is(*lse, {q.size(0), q.size(1), q.size(2)})))
        value_error("kv_lens [B], out [B,S,Hq,D], lse [B,S,Hq] expected");
    double scale;
    if (x[9] == Py_None) {
        scale = 1.0 / std::sqrt((double)d.headDim);
    } else {
        scale = PyFloat_AsDouble(x[9]);
        if (scale == -1.0 && PyErr_Occurred())
            throw PythonError{};
    }
    const at::Device dev = q.device();
    const uint16_t* qp = dense<uint16_t>(q, "q", at::kHalf, dev);
    const void* cp = dense(cache, "kv_cache", cache.scalar_type(), dev);
    const float* sp = dense<float>(scales, "kv_scales", at::kFloat, dev);
    const int32_t *pp = dense<int32_t>(prefix, "prefix_table", at::kInt, dev),
                  *tp = dense<int32_t>(table, "page_table", at::kInt, dev),
                  *lp = dense<int32_t>(lens, "kv_lens", at::kInt, dev);
    uint16_t* op = dense<uint16_t>(out, "out", at::kHalf, dev);
    float* ep = dense<float>(lse, "lse", at::kFloat, dev);
    void* wp = dense(given, "workspace", at::kByte, dev);
    const auto st = stream_of(x[11], dev);
    at::Tensor own;                 // freed when the call returns: reuse is ordered by the stream
    int64_t size = given ? given->numel() : paged_attention_workspace_size(&d);
    if (size < 0)
        return (int)size;
    if (!given && size > 0) {
        const c10::cuda::CUDAStreamGuard guard(st);
        own = at::empty({size}, at::TensorOptions().dtype(at::kByte).device(dev));
        wp = own.data_ptr();
    }
    return on_stream(dev, [&] {
        return paged_attention_shared_prefix(qp, cp, sp, pp, tp, lp, op, ep, wp, size, &d, (float)scale,
                                             st.stream());
    });
}

double scale_of(PyObject* o, int32_t D)
{
    if (o == Py_None)
        return 1.0 / std::sqrt((double)D);
    const double scale = PyFloat_AsDouble(o);
    if (scale == -1.0 && PyErr_Occurred())
        throw PythonError{};
    return scale;
}

// A workspace of `size` bytes: the given one, or one of the stream's that is freed when
// the call returns (reuse is ordered by the stream).
struct Workspace {
    at::Tensor own;
    void* data = nullptr;
    int64_t size = 0;
    Workspace(const at::Tensor* given, int64_t need, at::Device dev, const c10::cuda::CUDAStream& st)
    {
        data = dense(given, "workspace", at::kByte, dev);
        size = given ? given->numel() : need;
        if (!given && need > 0) {
            const c10::cuda::CUDAStreamGuard guard(st);
            own = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(dev));
            data = own.data_ptr();
        }
    }
};

ropekv_prompt_dims prompt_dims(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v,
                               const at::Tensor& qStarts, const at::Tensor* kvStarts)
{
    if (q.dim() != 3 || k.dim() != 3 || q.size(2) != k.size(2) || v.sizes() != k.sizes())
        value_error("q [T,Hq,D] and k, v [Tk,Hkv,D] expected");
    if (qStarts.dim() != 1 || qStarts.size(0) < 1 || (kvStarts && kvStarts->sizes() != qStarts.sizes()))
        value_error("q_starts, kv_starts [B + 1] expected");
    if (!kvStarts && q.size(0) != k.size(0))
        value_error("kv_starts is needed where q and k differ in their numbers of tokens");
    return {small(q.size(0), "T"), small(k.size(0), "Tk"), small(qStarts.size(0) - 1, "B"),
            small(q.size(1), "Hq"), small(k.size(1), "Hkv"), small(q.size(2), "D")};
}

// prompt_workspace(q, k, v, q_starts, kv_starts)
int64_t prompt_workspace(PyObject* const* x)
{
    const ropekv_prompt_dims d = prompt_dims(tensor(x[0], "q"), tensor(x[1], "k"), tensor(x[2], "v"),
                                             tensor(x[3], "q_starts"), optional(x[4], "kv_starts"));
    return prompt_attention_workspace_size(&d);
}

// prompt(q, k, v, q_starts, out, kv_starts, lse, sm_scale, workspace, stream)
int prompt(PyObject* const* x)
{
    const at::Tensor &q = tensor(x[0], "q"), &k = tensor(x[1], "k"), &v = tensor(x[2], "v"),
                     &qStarts = tensor(x[3], "q_starts"), &out = tensor(x[4], "out");
    const at::Tensor *kvStarts = optional(x[5], "kv_starts"), *lse = optional(x[6], "lse"),
                     *given = optional(x[8], "workspace");
    const ropekv_prompt_dims d = prompt_dims(q, k, v, qStarts, kvStarts);
    if (out.sizes() != q.sizes() || (lse && !is(*lse, {q.size(0), q.size(1)})))
        value_error("out [T,Hq,D], lse [T,Hq] expected");
    const double scale = scale_of(x[7], d.headDim);
    const at::Device dev = q.device();
    int64_t qs, ks, vs;
    const uint16_t *qp = rows(q, "q", dev, qs), *kp = rows(k, "k", dev, ks), *vp = rows(v, "v", dev, vs);
    const int32_t *qsp = dense<int32_t>(qStarts, "q_starts", at::kInt, dev),
                  *ksp = dense<int32_t>(kvStarts, "kv_starts", at::kInt, dev);
    uint16_t* op = dense<uint16_t>(out, "out", at::kHalf, dev);
    float* ep = dense<float>(lse, "lse", at::kFloat, dev);
    const auto st = stream_of(x[9], dev);
    const int64_t need = prompt_attention_workspace_size(&d);
    if (need < 0)
        return (int)need;
    const Workspace ws(given, need, dev, st);
    return on_stream(dev, [&] {
        return prompt_attention(qp, qs, kp, ks, vp, vs, qsp, ksp, op, ep, ws.data, ws.size, &d, (float)scale,
                                st.stream());
    });
}

ropekv_tree_dims tree_dims(const at::Tensor& q, const at::Tensor& cache)
{
    if (q.dim() != 4 || cache.dim() != 5 || cache.size(0) != q.size(0) || cache.size(1) != 2 ||
        cache.size(4) != q.size(3))
        value_error("q [B,S,Hq,D] and kv_cache [B,2,Hkv,cap,D] expected");
    return {small(q.size(0), "B"), small(q.size(1), "S"), small(q.size(2), "Hq"), small(cache.size(2), "Hkv"),
            small(q.size(3), "D"), small(cache.size(3), "cap")};
}

// tree_workspace(q, kv_cache)
int64_t tree_workspace(PyObject* const* x)
{
    const ropekv_tree_dims d = tree_dims(tensor(x[0], "q"), tensor(x[1], "kv_cache"));
    return tree_attention_workspace_size(&d);
}

// tree(q, kv_cache, kv_cache_end_lens, out, tree_mask, lse, sm_scale, workspace, stream)
int tree(PyObject* const* x)
{
    const at::Tensor &q = tensor(x[0], "q"), &cache = tensor(x[1], "kv_cache"),
                     &lens = tensor(x[2], "kv_cache_end_lens"), &out = tensor(x[3], "out");
    const at::Tensor *mask = optional(x[4], "tree_mask"), *lse = optional(x[5], "lse"),
                     *given = optional(x[7], "workspace");
    const ropekv_tree_dims d = tree_dims(q, cache);
    if (!is(lens, {d.batch}) || out.sizes() != q.sizes() || (lse && !is(*lse, {q.size(0), q.size(1), q.size(2)})))
        value_error("kv_cache_end_lens [B], out [B,S,Hq,D], lse [B,S,Hq] expected");
    if (mask && !is(*mask, {d.batch, d.seqLen, (d.seqLen + 31) / 32}))
        value_error("tree_mask [B, S, ceil(S / 32)] expected");
    const double scale = scale_of(x[6], d.headDim);
    const at::Device dev = q.device();
    const uint16_t *qp = dense<uint16_t>(q, "q", at::kHalf, dev), *cp = dense<uint16_t>(cache, "kv_cache", at::kHalf, dev);
    const int32_t *lp = dense<int32_t>(lens, "kv_cache_end_lens", at::kInt, dev),
                  *mp = dense<int32_t>(mask, "tree_mask", at::kInt, dev);
    uint16_t* op = dense<uint16_t>(out, "out", at::kHalf, dev);
    float* ep = dense<float>(lse, "lse", at::kFloat, dev);
    const auto st = stream_of(x[8], dev);
    const int64_t need = tree_attention_workspace_size(&d);
    if (need < 0)
        return (int)need;
    const Workspace ws(given, need, dev, st);
    return on_stream(dev, [&] {
        return tree_attention(qp, cp, lp, mp, op, ep, ws.data, ws.size, &d, (float)scale, st.stream());
    });
}

// accept(kv_cache, kv_cache_end_lens, seq_len, accepted, accepted_lens, end_lens_out, stream)
int accept(PyObject* const* x)
{
    const at::Tensor &cache = tensor(x[0], "kv_cache"), &lens = tensor(x[1], "kv_cache_end_lens"),
                     &acc = tensor(x[3], "accepted"), &accLens = tensor(x[4], "accepted_lens");
    const at::Tensor* lensOut = optional(x[5], "end_lens_out");
    if (cache.dim() != 5 || cache.size(1) != 2)
        value_error("kv_cache [B,2,Hkv,cap,D] expected");
    const int64_t B = cache.size(0);
    if (!is(lens, {B}) || acc.dim() != 2 || acc.size(0) != B || !is(accLens, {B}) || (lensOut && !is(*lensOut, {B})))
        value_error("kv_cache_end_lens [B], accepted [B,A], accepted_lens [B], end_lens_out [B] expected");
    const int32_t S = whole(x[2], "seq_len"), A = small(acc.size(1), "A"), b = small(B, "B"),
                  Hkv = small(cache.size(2), "Hkv"), cap = small(cache.size(3), "cap"), D = small(cache.size(4), "D");
    const at::Device dev = cache.device();
    uint16_t* cp = dense<uint16_t>(cache, "kv_cache", at::kHalf, dev);
    const int32_t *lp = dense<int32_t>(lens, "kv_cache_end_lens", at::kInt, dev),
                  *ap = dense<int32_t>(acc, "accepted", at::kInt, dev),
                  *np = dense<int32_t>(accLens, "accepted_lens", at::kInt, dev);
    int32_t* op = dense<int32_t>(lensOut, "end_lens_out", at::kInt, dev);
    const auto st = stream_of(x[6], dev);
    return on_stream(dev, [&] {
        return kv_accept_drafts(cp, lp, ap, np, op, b, S, A, Hkv, D, cap, st.stream());
    });
}

// paged_accept(kv_cache, page_table, kv_lens, seq_len, accepted, accepted_lens, kv_lens_out, kv_scales, stream)
int paged_accept(PyObject* const* x)
{
    const at::Tensor &cache = tensor(x[0], "kv_cache"), &table = tensor(x[1], "page_table"),
                     &lens = tensor(x[2], "kv_lens"), &acc = tensor(x[4], "accepted"),
                     &accLens = tensor(x[5], "accepted_lens");
    const at::Tensor *lensOut = optional(x[6], "kv_lens_out"), *scales = optional(x[7], "kv_scales");
    const Pool p = check_pool(cache, scales, table);
    if (!is(lens, {p.B}) || acc.dim() != 2 || acc.size(0) != p.B || !is(accLens, {p.B}) || (lensOut && !is(*lensOut, {p.B})))
        value_error("kv_lens [B], accepted [B,A], accepted_lens [B], kv_lens_out [B] expected");
    const int32_t S = whole(x[3], "seq_len"), A = small(acc.size(1), "A");
    const at::Device dev = cache.device();
    void* cp = dense(cache, "kv_cache", cache.scalar_type(), dev);
    float* sp = dense<float>(scales, "kv_scales", at::kFloat, dev);
    const int32_t *tp = dense<int32_t>(table, "page_table", at::kInt, dev),
                  *lp = dense<int32_t>(lens, "kv_lens", at::kInt, dev),
                  *ap = dense<int32_t>(acc, "accepted", at::kInt, dev),
                  *np = dense<int32_t>(accLens, "accepted_lens", at::kInt, dev);
    int32_t* op = dense<int32_t>(lensOut, "kv_lens_out", at::kInt, dev);
    const auto st = stream_of(x[8], dev);
    return on_stream(dev, [&] {
        return paged_kv_accept_drafts(cp, sp, tp, lp, ap, np, op, p.B, S, A, p.Hkv, p.D, p.pages, p.M, p.tpp, p.fmt,
                                      st.stream());
    });
}

// A pool alone: as check_pool, without a page table.
Pool check_pool(const at::Tensor& cache, const at::Tensor* scales)
{
    if (cache.dim() != 5 || cache.size(0) != 2)
        value_error("kv_cache [2,P,TPP,Hkv,D] expected");
    const int fmt = format_of(cache, "kv_cache", false);
    if (fmt == ROPEKV_CACHE_F16 ? scales != nullptr
                                : !scales || !is(*scales, {2, cache.size(1), cache.size(3), cache.size(2)}))
        value_error(fmt == ROPEKV_CACHE_F16 ? "a float16 cache has no kv_scales"
                                            : "kv_scales [2, P, Hkv, TPP] expected for an 8-bit cache");
    return {small(cache.size(1), "P"), small(cache.size(2), "TPP"), small(cache.size(3), "Hkv"),
            small(cache.size(4), "D"), fmt, 0, 0};
}

// copy_pages(kv_cache, src_pages, dst_pages, kv_scales, stream)
int copy_pages(PyObject* const* x)
{
    const at::Tensor &cache = tensor(x[0], "kv_cache"), &src = tensor(x[1], "src_pages"), &dst = tensor(x[2], "dst_pages");
    const at::Tensor* scales = optional(x[3], "kv_scales");
    const Pool p = check_pool(cache, scales);
    if (src.dim() != 1 || dst.sizes() != src.sizes())
        value_error("src_pages, dst_pages [N] expected");
    const at::Device dev = cache.device();
    void* cp = dense(cache, "kv_cache", cache.scalar_type(), dev);
    float* scp = dense<float>(scales, "kv_scales", at::kFloat, dev);
    const int32_t *sp = dense<int32_t>(src, "src_pages", at::kInt, dev), *dp = dense<int32_t>(dst, "dst_pages", at::kInt, dev);
    const int32_t n = small(src.size(0), "N");
    const auto st = stream_of(x[4], dev);
    return on_stream(dev, [&] {
        return paged_kv_copy_pages(cp, scp, sp, dp, n, p.Hkv, p.D, p.pages, p.tpp, p.fmt, st.stream());
    });
}

// fork(kv_cache, page_table, kv_lens, ref_counts, parents, children, kv_scales, workspace, stream)
int fork(PyObject* const* x)
{
    const at::Tensor &cache = tensor(x[0], "kv_cache"), &table = tensor(x[1], "page_table"), &lens = tensor(x[2], "kv_lens"),
                     &refs = tensor(x[3], "ref_counts"), &parents = tensor(x[4], "parents"),
                     &children = tensor(x[5], "children");
    const at::Tensor *scales = optional(x[6], "kv_scales"), *given = optional(x[7], "workspace");
    const Pool p = check_pool(cache, scales, table);
    if (!is(lens, {p.B}) || !is(refs, {p.pages}) || parents.dim() != 1 || children.sizes() != parents.sizes())
        value_error("kv_lens [B], ref_counts [P], parents, children [N] expected");
    const at::Device dev = cache.device();
    void* cp = dense(cache, "kv_cache", cache.scalar_type(), dev);
    float* scp = dense<float>(scales, "kv_scales", at::kFloat, dev);
    int32_t *tp = dense<int32_t>(table, "page_table", at::kInt, dev), *lp = dense<int32_t>(lens, "kv_lens", at::kInt, dev),
            *rp = dense<int32_t>(refs, "ref_counts", at::kInt, dev);
    const int32_t *pp = dense<int32_t>(parents, "parents", at::kInt, dev),
                  *chp = dense<int32_t>(children, "children", at::kInt, dev);
    const int32_t n = small(parents.size(0), "N");
    const auto st = stream_of(x[8], dev);
    const int64_t need = paged_kv_fork_workspace_size(n, p.B);
    if (need < 0)
        return (int)need;
    const Workspace ws(given, need, dev, st);
    return on_stream(dev, [&] {
        return paged_kv_fork(cp, scp, tp, lp, rp, pp, chp, ws.data, ws.size, n, p.B, p.Hkv, p.D, p.pages, p.M, p.tpp,
                             p.fmt, st.stream());
    });
}

// release(page_table, kv_lens, ref_counts, sequences, tokens_per_page, keep_lens, stream)
int release(PyObject* const* x)
{
    const at::Tensor &table = tensor(x[0], "page_table"), &lens = tensor(x[1], "kv_lens"), &refs = tensor(x[2], "ref_counts"),
                     &seqs = tensor(x[3], "sequences");
    const at::Tensor* keep = optional(x[5], "keep_lens");
    if (table.dim() != 3 || table.size(1) != 2 || !is(lens, {table.size(0)}) || refs.dim() != 1)
        value_error("page_table [B,2,M], kv_lens [B], ref_counts [P] expected");
    if (seqs.dim() != 1 || (keep && keep->sizes() != seqs.sizes()))
        value_error("sequences, keep_lens [N] expected");
    const at::Device dev = table.device();
    int32_t *tp = dense<int32_t>(table, "page_table", at::kInt, dev), *lp = dense<int32_t>(lens, "kv_lens", at::kInt, dev),
            *rp = dense<int32_t>(refs, "ref_counts", at::kInt, dev);
    const int32_t *sp = dense<int32_t>(seqs, "sequences", at::kInt, dev), *kp = dense<int32_t>(keep, "keep_lens", at::kInt, dev);
    const int32_t n = small(seqs.size(0), "N"), B = small(table.size(0), "B"), M = small(table.size(2), "M"),
                  P = small(refs.size(0), "P"), tpp = whole(x[4], "tokens_per_page");
    const auto st = stream_of(x[6], dev);
    return on_stream(dev, [&] {
        return paged_kv_free(tp, lp, rp, sp, kp, n, B, P, M, tpp, st.stream());
    });
}

template <typename R, R (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        return PyLong_FromLongLong((long long)F(args));
    } catch (const Refusal& e) {
        PyErr_SetString(e.type, e.text.c_str());
    } catch (const PythonError&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <typename R, R (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<R, F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {
    method<int, mrope, 13>("mrope"),
    method<int, quant, 13>("quant"),
    method<int, read, 8>("read"),
    method<int, attention, 12>("attention"),
    method<int64_t, attention_workspace, 6>("attention_workspace"),
    method<int, prompt, 10>("prompt"),
    method<int64_t, prompt_workspace, 5>("prompt_workspace"),
    method<int, tree, 9>("tree"),
    method<int64_t, tree_workspace, 2>("tree_workspace"),
    method<int, accept, 7>("accept"),
    method<int, paged_accept, 9>("paged_accept"),
    method<int, copy_pages, 5>("copy_pages"),
    method<int, fork, 9>("fork"),
    method<int, release, 7>("release"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "ropekv_bind", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ropekv_bind()
{
    return PyModule_Create(&kModule);
}
