// The Python binding's argument marshalling: shapes, types, strides and
// devices of torch tensors are checked here and handed to the C entry points
// (include/w8a16.h), whose addresses Python passes once.  Written against the
// CPython and torch C++ interfaces because a call's attribute reads and
// argument objects in Python cost more than its launch: a decode step's
// append of three axes 11.4 us of Python and 3.5 of library and launch.
//
// Refused arguments raise ValueError; a status other than W8A16_OK is
// returned as an int, for the caller to raise.

#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "w8a16.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Raised {};      // a Python error is set

decltype(&w8a16_rope) f_rope;
decltype(&w8a16_rope_axes) f_rope_axes;
decltype(&w8a16_kv_append) f_kv_append;
decltype(&w8a16_kv_append_axes) f_kv_append_axes;
decltype(&w8a16_kv_attention) f_kv_attention;
decltype(&w8a16_kv_attention_span) f_kv_attention_span;
decltype(&w8a16_gemm_epilogue) f_gemm_epilogue;

void require(bool ok, const char *message)
{
    if (!ok)
        throw Refused(message);
}

const Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw Raised();
    }
    return THPVariable_Unpack(o);
}

bool given(PyObject *o) { return o != Py_None; }

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised();
    return v;
}

double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised();
    return v;
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised();
    return v != 0;
}

// Index of a string (or None, where names[i] is null) among `names`.
template <size_t N> uint32_t choice(PyObject *o, const char *const (&names)[N], const char *message)
{
    for (size_t i = 0; i < N; ++i)
        if (names[i] ? PyUnicode_Check(o) && PyUnicode_CompareWithASCIIString(o, names[i]) == 0 : o == Py_None)
            return (uint32_t)i;
    throw Refused(message);
}

const char *const kLayouts[] = {"half", "interleaved"};
const char *const kOrders[] = {"split", "turns", "own"};
const char *const kActivations[] = {nullptr, "relu", "silu", "gelu", "gelu_tanh"};

uint32_t dtype_code(ScalarType t)      // w8a16_dtype, 0 for others
{
    return t == ScalarType::BFloat16 ? W8A16_BF16 : t == ScalarType::Half ? W8A16_FP16
           : t == ScalarType::Float ? W8A16_FP32 : 0;
}

const char *type_name(ScalarType t)
{
    return t == ScalarType::BFloat16 ? "bfloat16" : t == ScalarType::Half ? "float16" : "float32";
}

// Tensors of a call lie on one device, the first one's.
struct Device {
    c10::Device d;
    explicit Device(const Tensor &t) : d(t.device()) {}
    bool has(const Tensor &t) const { return t.is_cuda() && t.device() == d; }
};

// A 32-bit count: what does not fit is no shape.
uint32_t u32(int64_t v) { return v < 0 || v > 0xffffffffll ? 0xffffffffu : (uint32_t)v; }

void *stream_of(PyObject *o)
{
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred())
        throw Raised();
    return p;
}

// Other Python threads run while a call is enqueued (or its workspace grows).
struct Unlocked {
    PyThreadState *const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F, class... A> int unlocked(F f, A... args)
{
    const Unlocked u;
    return f(args...);
}

struct Rows {
    int64_t token, head;
};

// Token and head strides of a [tokens, heads, dim] operand.
Rows rows(const char *name, const Tensor &t, int64_t tokens, int64_t heads, int64_t dim, ScalarType type,
          const Device &dev)
{
    if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != dim ||
        t.scalar_type() != type || !dev.has(t))
        throw Refused(std::string(name) + " must be a " + type_name(type) + " GPU tensor [" +
                      std::to_string(tokens) + ", " + std::to_string(heads) + ", " + std::to_string(dim) +
                      "] beside the others");
    if (t.stride(2) != 1 && dim > 1)
        throw Refused(std::string(name) + " needs a unit stride along head_dim");
    return {t.stride(0), t.stride(1)};
}

// A new contiguous tensor of t's type.
Tensor fresh(const Tensor &t, at::IntArrayRef sizes) { return at::empty(sizes, t.options()); }

void check_table(const Tensor &t, const Device &dev)
{
    require(t.scalar_type() == ScalarType::Float && t.dim() == 3 && t.size(2) == 2 && t.is_contiguous() &&
                dev.has(t),
            "table must be a contiguous float32 GPU tensor [positions, rot_dim/2, 2]");
}

// Positions of several axes; sections: pairs of each.
w8a16_axes_t axes(PyObject *positions, int64_t tokens, PyObject *sections, PyObject *order, int64_t table_pairs,
                  const Device &dev)
{
    w8a16_axes_t a = {};
    a.order = choice(order, kOrders, "order must be 'split', 'turns' or 'own'");
    PyObject *seq = PySequence_Fast(sections, "sections must be a sequence of pairs");
    if (!seq)
        throw Raised();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    bool ok = n >= 1 && n <= W8A16_ROPE_MAX_AXES;
    for (Py_ssize_t i = 0; ok && i < n; ++i) {
        const long long v = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
        if (v == -1 && PyErr_Occurred()) {
            Py_DECREF(seq);
            throw Raised();
        }
        ok = v >= 0 && v <= 0xffffffffll;
        a.pairs[i] = u32(v);
    }
    Py_DECREF(seq);
    require(ok, "sections must be the pairs of 1 to 4 axes");
    require(given(positions), "positions of the axes are missing");
    const Tensor &p = tensor(positions, "positions");
    require(p.scalar_type() == ScalarType::Int && p.dim() == 2 && p.size(0) == n && p.size(1) == tokens &&
                dev.has(p) && (tokens < 2 || p.stride(1) == 1),
            "positions must be an int32 GPU tensor [axes, tokens] with a unit stride along tokens");
    a.positions = static_cast<const int32_t *>(p.const_data_ptr());
    a.axis_stride = p.stride(0);
    a.count = (uint32_t)n;
    a.table_pairs = u32(table_pairs);
    return a;
}

uint32_t axes_rot(const w8a16_axes_t &a)
{
    uint64_t sum = 0;
    for (uint32_t i = 0; i < a.count; ++i)
        sum += a.pairs[i];
    return u32((int64_t)(2 * sum));
}

// Page stride of a cache tensor whose pages are contiguous inside (of a single
// page its size, whatever the tensor says).
uint64_t page_stride(const char *name, const Tensor &t)
{
    int64_t want = 1;
    for (int64_t i = t.dim() - 1; i > 0; --i) {
        if (t.size(i) > 1 && t.stride(i) != want)
            throw Refused(std::string("the inside of a ") + name + " page must be contiguous");
        want *= t.size(i);
    }
    return (uint64_t)(t.size(0) < 2 ? want : t.stride(0));
}

w8a16_kv_cache_t cache_of(PyObject *o, const Device &d)
{
    PyObject *seq = PySequence_Fast(o, "cache must be (k, v, k_scale, v_scale)");
    if (!seq)
        throw Raised();
    struct Hold {
        PyObject *p;
        ~Hold() { Py_DECREF(p); }
    } hold{seq};
    require(PySequence_Fast_GET_SIZE(seq) == 4, "cache must be (k, v, k_scale, v_scale)");
    PyObject **it = PySequence_Fast_ITEMS(seq);
    const Tensor &k = tensor(it[0], "cache.k"), &v = tensor(it[1], "cache.v"), &ks = tensor(it[2], "cache.k_scale"),
                 &vs = tensor(it[3], "cache.v_scale");
    const char *shape = "cache must be k [pages, heads, page, dim], v [pages, heads, page/16, dim, 16] and scales "
                        "[pages, heads, page/16]";
    require(k.dim() == 4, shape);
    const int64_t pages = k.size(0), heads = k.size(1), page = k.size(2), dim = k.size(3);
    const int64_t blocks = page / W8A16_KV_BLOCK;
    const int64_t vw[5] = {pages, heads, blocks, dim, W8A16_KV_BLOCK}, sw[3] = {pages, heads, blocks};
    require(v.sizes() == at::IntArrayRef(vw, 5) && ks.sizes() == at::IntArrayRef(sw, 3) && vs.sizes() == ks.sizes(),
            shape);
    auto codes = [](const Tensor &t) {
        return t.scalar_type() == ScalarType::Byte || t.scalar_type() == ScalarType::Float8_e4m3fn;
    };
    auto bytes = [](const Tensor &t) {
        return t.scalar_type() == ScalarType::Byte || t.scalar_type() == ScalarType::Float8_e8m0fnu;
    };
    require(codes(k) && codes(v) && bytes(ks) && bytes(vs),
            "cache codes must be uint8 or float8_e4m3fn, its scales uint8 or float8_e8m0fnu");
    require(d.has(k) && d.has(v) && d.has(ks) && d.has(vs), "cache must be GPU tensors");
    w8a16_kv_cache_t c;
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.k_scale = static_cast<uint8_t *>(ks.data_ptr());
    c.v_scale = static_cast<uint8_t *>(vs.data_ptr());
    c.k_page_stride = page_stride("k", k);
    c.v_page_stride = page_stride("v", v);
    c.k_scale_page_stride = page_stride("k_scale", ks);
    c.v_scale_page_stride = page_stride("v_scale", vs);
    c.pages = u32(pages);
    c.page_size = u32(page);
    c.kv_heads = u32(heads);
    c.head_dim = u32(dim);
    return c;
}

w8a16_kv_seqs_t seqs_of(PyObject *block_table, PyObject *kv_lens, PyObject *cu_seqlens, PyObject *max_new,
                        int64_t tokens, const Device &dev)
{
    const Tensor &bt = tensor(block_table, "block_table"), &lens = tensor(kv_lens, "kv_lens");
    require(bt.scalar_type() == ScalarType::Int && lens.scalar_type() == ScalarType::Int && lens.dim() == 1 &&
                bt.dim() == 2,
            "block_table must be int32 [seqs, pages] and kv_lens int32 [seqs]");
    const int64_t n = lens.size(0), width = bt.size(1);
    require(bt.size(0) == n && dev.has(bt) && dev.has(lens),
            "block_table and kv_lens must be GPU tensors of the same sequences");
    require(width < 2 || bt.stride(1) == 1, "block_table rows must be contiguous");
    require(lens.is_contiguous(), "kv_lens must be contiguous");
    w8a16_kv_seqs_t s = {};
    s.block_table = static_cast<const int32_t *>(bt.const_data_ptr());
    s.kv_lens = static_cast<const int32_t *>(lens.const_data_ptr());
    const int64_t pitch = n > 1 ? bt.stride(0) : width;
    require(pitch >= 0 && pitch <= 0xffffffffll, "block_table rows must be at most 2^32 - 1 places apart");
    s.block_table_stride = u32(pitch);
    s.block_table_width = u32(width);
    s.seqs = u32(n);
    s.tokens = u32(tokens);
    if (given(cu_seqlens)) {
        const Tensor &cu = tensor(cu_seqlens, "cu_seqlens");
        require(cu.scalar_type() == ScalarType::Int && cu.dim() == 1 && cu.size(0) == n + 1 && cu.is_contiguous() &&
                    dev.has(cu),
                "cu_seqlens must be a contiguous int32 GPU tensor [seqs + 1]");
        s.cu_seqlens = static_cast<const int32_t *>(cu.const_data_ptr());
        s.max_new = u32(given(max_new) ? integer(max_new) : tokens);
    } else {
        s.max_new = u32(given(max_new) ? integer(max_new) : tokens / (n > 1 ? n : 1));
    }
    return s;
}

PyObject *status(int st) { return PyLong_FromLong(st); }

// rope(x, table, positions, out, layout, inverse, sections, order, stream)
PyObject *rope(PyObject *const *o)
{
    const Tensor &x = tensor(o[0], "x");
    const ScalarType type = x.scalar_type();
    const uint32_t code = dtype_code(type);
    require(x.dim() == 3 && code, "x must be bfloat16, float16 or float32 [tokens, heads, head_dim]");
    const int64_t tokens = x.size(0), heads = x.size(1), dim = x.size(2);
    const Device dev(x);
    const Rows xr = rows("x", x, tokens, heads, dim, type, dev);
    const uint32_t layout = choice(o[4], kLayouts, "layout must be 'half' or 'interleaved'");
    const Tensor &table = tensor(o[1], "table");
    check_table(table, dev);
    Tensor made;
    Rows yr = {heads * dim, dim};
    if (given(o[3]))
        yr = rows("out", tensor(o[3], "out"), tokens, heads, dim, type, dev);
    else
        made = fresh(x, x.sizes());
    const Tensor &y = given(o[3]) ? THPVariable_Unpack(o[3]) : made;
    const float *tp = static_cast<const float *>(table.const_data_ptr());
    int st;
    if (given(o[6])) {
        const w8a16_axes_t a = axes(o[2], tokens, o[6], o[7], table.size(1), dev);
        st = unlocked(f_rope_axes, x.const_data_ptr(), xr.token, xr.head, y.data_ptr(), yr.token, yr.head, code,
                      u32(tokens), u32(heads), u32(dim), tp, u32(table.size(0)), &a, layout, truth(o[5]),
                      stream_of(o[8]));
    } else {
        const Tensor &p = tensor(o[2], "positions");
        require(p.dim() == 1 && p.size(0) == tokens && p.scalar_type() == ScalarType::Int && p.is_contiguous() &&
                    dev.has(p),
                "positions must be a contiguous int32 GPU tensor [tokens]");
        st = unlocked(f_rope, x.const_data_ptr(), xr.token, xr.head, y.data_ptr(), yr.token, yr.head, code,
                      u32(tokens), u32(heads), u32(dim), tp, u32(table.size(0)), u32(2 * table.size(1)),
                      static_cast<const int32_t *>(p.const_data_ptr()), layout, truth(o[5]), stream_of(o[8]));
    }
    if (st)
        return status(st);
    return given(o[3]) ? Py_NewRef(o[3]) : THPVariable_Wrap(made);
}

// kv_append(cache, k, v, block_table, kv_lens, cu_seqlens, max_new, table, layout, q, q_out, positions,
//           sections, order, stream)
PyObject *kv_append(PyObject *const *o)
{
    const Tensor &k = tensor(o[1], "k"), &v = tensor(o[2], "v");
    const ScalarType type = k.scalar_type();
    w8a16_kv_append_args_t a = {};
    a.dtype = dtype_code(type);
    require(k.dim() == 3 && a.dtype, "k must be bfloat16, float16 or float32 [tokens, kv_heads, head_dim]");
    const int64_t tokens = k.size(0), heads = k.size(1), dim = k.size(2);
    const Device dev(k);
    const w8a16_kv_cache_t c = cache_of(o[0], dev);
    require(heads == c.kv_heads && dim == c.head_dim, "k must have the cache's heads and head_dim");
    const Rows kr = rows("k", k, tokens, heads, dim, type, dev), vr = rows("v", v, tokens, heads, dim, type, dev);
    a.layout = choice(o[8], kLayouts, "layout must be 'half' or 'interleaved'");
    a.k = k.const_data_ptr();
    a.v = v.const_data_ptr();
    a.k_token_stride = kr.token;
    a.k_head_stride = kr.head;
    a.v_token_stride = vr.token;
    a.v_head_stride = vr.head;
    int64_t pairs = 0;
    if (given(o[7])) {
        const Tensor &table = tensor(o[7], "table");
        check_table(table, dev);
        pairs = table.size(1);
        a.table = static_cast<const float *>(table.const_data_ptr());
        a.table_positions = u32(table.size(0));
        a.rot_dim = u32(2 * pairs);
    }
    const w8a16_kv_seqs_t s = seqs_of(o[3], o[4], o[5], o[6], tokens, dev);
    w8a16_axes_t ax = {};
    const bool by_axes = given(o[12]);
    if (by_axes) {
        require(given(o[7]), "positions of several axes need a table");
        ax = axes(o[11], tokens, o[12], o[13], pairs, dev);
        a.rot_dim = axes_rot(ax);
    } else {
        require(!given(o[11]), "positions need sections");
    }
    Tensor made;
    const bool queries = given(o[9]);
    if (queries) {
        const Tensor &q = tensor(o[9], "q");
        const int64_t hq = q.dim() == 3 ? q.size(1) : 0;
        const Rows qr = rows("q", q, tokens, hq, dim, type, dev);
        Rows yr = {hq * dim, dim};
        if (given(o[10]))
            yr = rows("q_out", tensor(o[10], "q_out"), tokens, hq, dim, type, dev);
        else
            made = fresh(q, q.sizes());
        a.q = q.const_data_ptr();
        a.q_out = given(o[10]) ? THPVariable_Unpack(o[10]).data_ptr() : made.data_ptr();
        a.q_token_stride = qr.token;
        a.q_head_stride = qr.head;
        a.q_out_token_stride = yr.token;
        a.q_out_head_stride = yr.head;
        a.q_heads = u32(hq);
    }
    void *stream = stream_of(o[14]);
    const int st = by_axes ? unlocked(f_kv_append_axes, &c, &s, &a, &ax, stream)
                           : unlocked(f_kv_append, &c, &s, &a, stream);
    if (st)
        return status(st);
    if (!queries)
        Py_RETURN_NONE;
    return given(o[10]) ? Py_NewRef(o[10]) : THPVariable_Wrap(made);
}

// kv_attention(q, cache, block_table, kv_lens, out, cu_seqlens, max_new, max_kv, scale, causal, window, sinks,
//              shared, return_lse, plan address, stream)
PyObject *kv_attention(PyObject *const *o)
{
    const Tensor &q = tensor(o[0], "q");
    const ScalarType type = q.scalar_type();
    w8a16_kv_attention_args_t a = {};
    a.dtype = dtype_code(type);
    require(q.dim() == 3 && a.dtype, "q must be bfloat16 or float16 [tokens, q_heads, head_dim]");
    const Device dev(q);
    const w8a16_kv_cache_t c = cache_of(o[1], dev);
    const int64_t tokens = q.size(0), heads = q.size(1), dim = c.head_dim;
    const Rows qr = rows("q", q, tokens, heads, dim, type, dev);
    const int64_t window = integer(o[10]), sinks = integer(o[11]), shared = integer(o[12]);
    require(window >= 0 && sinks >= 0 && shared >= 0, "window, sinks and shared must not be negative");
    const w8a16_kv_seqs_t s = seqs_of(o[2], o[3], o[5], o[6], tokens, dev);
    a.scale = given(o[8]) ? (float)real(o[8]) : 0.f;
    Tensor made, lse;
    Rows yr = {heads * dim, dim};
    if (given(o[4]))
        yr = rows("out", tensor(o[4], "out"), tokens, heads, dim, type, dev);
    else
        made = fresh(q, q.sizes());
    if (truth(o[13])) {
        lse = at::empty({tokens, heads}, q.options().dtype(ScalarType::Float));
        a.lse = static_cast<float *>(lse.data_ptr());
    }
    a.q = q.const_data_ptr();
    a.out = given(o[4]) ? THPVariable_Unpack(o[4]).data_ptr() : made.data_ptr();
    a.q_token_stride = qr.token;
    a.q_head_stride = qr.head;
    a.out_token_stride = yr.token;
    a.out_head_stride = yr.head;
    a.plan = static_cast<const w8a16_kv_plan_t *>(stream_of(o[14]));
    if (!given(o[8]))
        a.scale = (float)(1.0 / std::sqrt((double)dim));
    a.q_heads = u32(heads);
    a.causal = truth(o[9]);
    a.window = u32(window);
    a.max_kv = given(o[7]) ? u32(integer(o[7])) : 0u;
    void *stream = stream_of(o[15]);
    int st;
    if (sinks || shared) {
        const w8a16_kv_span_t span = {u32(sinks), u32(shared)};
        st = unlocked(f_kv_attention_span, &c, &s, &a, &span, stream);
    } else {
        st = unlocked(f_kv_attention, &c, &s, &a, stream);
    }
    if (st)
        return status(st);
    PyObject *out = given(o[4]) ? Py_NewRef(o[4]) : THPVariable_Wrap(made);
    if (!lse.defined() || !out)
        return out;
    PyObject *l = THPVariable_Wrap(lse), *pair = l ? PyTuple_Pack(2, out, l) : nullptr;
    Py_DECREF(out);
    Py_XDECREF(l);
    return pair;
}

// Row stride of an [m, n] operand with unit column stride (of a single row its
// length, whatever the tensor says).
uint32_t rows2(const char *name, const Tensor &t, int64_t m, int64_t n, bool f32, const Device &dev)
{
    const bool type = t.scalar_type() == ScalarType::BFloat16 || (f32 && t.scalar_type() == ScalarType::Float);
    if (!type || t.dim() != 2 || t.size(0) != m || t.size(1) != n || !dev.has(t))
        throw Refused(std::string(name) + " must be a bfloat16 " + (f32 ? "or float32 " : "") + "GPU tensor [" +
                      std::to_string(m) + ", " + std::to_string(n) + "] beside the others");
    if (t.stride(1) != 1 && n > 1)
        throw Refused(std::string(name) + " needs a unit column stride");
    const int64_t rs = t.stride(0);
    require(m < 2 || (rs >= 0 && rs <= 0xffffffffll), "rows must be at most 2^32 - 1 elements apart");
    return u32(m > 1 ? rs : n);
}

// gemm_epilogue(a, w, scale, c, bias, activation, gate, residual, out is float32 (None: not said), stream)
PyObject *gemm_epilogue(PyObject *const *o)
{
    const Tensor &a = tensor(o[0], "a"), &w = tensor(o[1], "w"), &scale = tensor(o[2], "scale");
    require(a.dim() == 2 && w.dim() == 2, "a and w must be 2-D");
    const int64_t m = a.size(0), k = a.size(1), n = w.size(0);
    require(w.size(1) == k, "w must be [n, k] with the k of a");
    require((w.scalar_type() == ScalarType::Byte || w.scalar_type() == ScalarType::Float8_e4m3fn) && w.is_contiguous(),
            "w must be contiguous float8_e4m3fn or uint8");
    require(scale.scalar_type() == ScalarType::Float && scale.is_contiguous() &&
                scale.numel() >= (n + 127) / 128 * (k % 128 == 0 ? k / 128 : 0),
            "scale must be contiguous float32 [ceil(n/128), k/128]");
    w8a16_epilogue_t e = {};
    e.activation = choice(o[5], kActivations, "activation must be None, 'relu', 'silu', 'gelu' or 'gelu_tanh'");
    const Device dev(a);
    const uint32_t ars = rows2("a", a, m, k, false, dev);
    require(dev.has(w) && dev.has(scale), "all operands must be GPU tensors");
    Tensor made;
    uint32_t crs = u32(n);
    if (given(o[3])) {
        const Tensor &c = tensor(o[3], "c");
        crs = rows2("c", c, m, n, true, dev);
        require(!given(o[8]) || truth(o[8]) == (c.scalar_type() == ScalarType::Float), "out_dtype must be that of c");
    }
    if (given(o[4])) {
        const Tensor &bias = tensor(o[4], "bias");
        require(dtype_code(bias.scalar_type()) && bias.scalar_type() != ScalarType::Half && bias.dim() == 1 &&
                    bias.size(0) == n && bias.is_contiguous() && dev.has(bias),
                "bias must be a contiguous bfloat16 or float32 GPU tensor [n]");
        e.bias = bias.const_data_ptr();
        e.bias_dtype = dtype_code(bias.scalar_type());
    }
    if (given(o[6])) {
        const Tensor &gate = tensor(o[6], "gate");
        e.gate_row_stride = rows2("gate", gate, m, n, false, dev);
        e.gate = gate.const_data_ptr();
    }
    if (given(o[7])) {
        const Tensor &r = tensor(o[7], "residual");
        e.residual_row_stride = rows2("residual", r, m, n, true, dev);
        e.residual = r.const_data_ptr();
        e.residual_dtype = dtype_code(r.scalar_type());
    }
    if (!given(o[3]))
        made = at::empty({m, n}, given(o[8]) && truth(o[8]) ? a.options().dtype(ScalarType::Float) : a.options());
    const Tensor &c = given(o[3]) ? THPVariable_Unpack(o[3]) : made;
    e.out_dtype = dtype_code(c.scalar_type());
    const int st = unlocked(f_gemm_epilogue, a.const_data_ptr(), ars, w.const_data_ptr(),
                            static_cast<const float *>(scale.const_data_ptr()), c.data_ptr(), crs, u32(m), u32(n),
                            u32(k), &e, stream_of(o[9]));
    if (st)
        return status(st);
    return given(o[3]) ? Py_NewRef(o[3]) : THPVariable_Wrap(made);
}

// No C++ exception passes into the interpreter.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    if (count != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", N, count);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised &) {
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type)
            PyErr_SetString(type, e.what());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// bind(addresses of rope, rope_axes, kv_append, kv_append_axes, kv_attention, kv_attention_span,
//      gemm_epilogue)
PyObject *bind(PyObject *const *o)
{
    f_rope = reinterpret_cast<decltype(f_rope)>(stream_of(o[0]));
    f_rope_axes = reinterpret_cast<decltype(f_rope_axes)>(stream_of(o[1]));
    f_kv_append = reinterpret_cast<decltype(f_kv_append)>(stream_of(o[2]));
    f_kv_append_axes = reinterpret_cast<decltype(f_kv_append_axes)>(stream_of(o[3]));
    f_kv_attention = reinterpret_cast<decltype(f_kv_attention)>(stream_of(o[4]));
    f_kv_attention_span = reinterpret_cast<decltype(f_kv_attention_span)>(stream_of(o[5]));
    f_gemm_epilogue = reinterpret_cast<decltype(f_gemm_epilogue)>(stream_of(o[6]));
    Py_RETURN_NONE;
}

#define W8A16_METHOD(name, count) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, count>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {W8A16_METHOD(bind, 7), W8A16_METHOD(rope, 9), W8A16_METHOD(kv_append, 15),
                         W8A16_METHOD(kv_attention, 16), W8A16_METHOD(gemm_epilogue, 10),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// W8A16_TORCH_VERSION: of the torch it is compiled against, whose tensors it
// reads by their layout.  What is checked here works in any CPython 3.
PyMODINIT_FUNC PyInit__binding()
{
    const std::string python = std::to_string(PY_MAJOR_VERSION) + "." + std::to_string(PY_MINOR_VERSION);
    const std::string here = Py_GetVersion();
    if (here.compare(0, python.size() + 1, python + ".") != 0) {
        PyErr_Format(PyExc_ImportError, "built for Python %s, this is %.8s", python.c_str(), here.c_str());
        return nullptr;
    }
    PyObject *m = PyModule_Create(&module);
    if (m && (PyModule_AddStringConstant(m, "torch_version", W8A16_TORCH_VERSION) < 0 ||
              PyModule_AddStringConstant(m, "python_version", python.c_str()) < 0)) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
