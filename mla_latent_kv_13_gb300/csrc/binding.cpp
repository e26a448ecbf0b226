// binding.cpp -- the ragged serving calls and the pages' calls for Python: checks the tensors and
// calls the C ABI (include/mla.h). mla.py has their documentation and makes missing buffers.
//
// For small calls the host's time counts, and it was mostly marshalling: reading types, shapes and
// addresses of nine tensors attribute by attribute and a call through ctypes took 6 us of a norm
// call's 10 (its launch 2, its kernel 3); here they take about half a microsecond.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <initializer_list>
#include <limits>
#include <string>

#include "mla.h"

namespace {

constexpr int64_t D_C = MLA_D_C, D_ROPE = MLA_D_ROPE, D_QK = MLA_D_QK, BLOCK = MLA_BLOCK;

struct Raised {};  // thrown once the Python error is set

[[noreturn]] void raise(PyObject *type, const std::string &what) {
    PyErr_SetString(type, what.c_str());
    throw Raised{};
}

// What a tensor may hold; bf16 also as its bit patterns.
enum Kind { BF16, BYTES, I32, F32 };

bool is_kind(at::ScalarType t, Kind k) {
    switch (k) {
        case BF16: return t == at::kBFloat16 || t == at::kShort || t == at::kUInt16;
        case BYTES: return t == at::kByte || t == at::kChar;
        case I32: return t == at::kInt;
        case F32: return t == at::kFloat;
    }
    return false;
}

std::string shape_text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

const at::Tensor &tensor(PyObject *o) {
    if (!THPVariable_Check(o))
        raise(PyExc_TypeError, std::string("expected a tensor, got ") + Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

const at::Tensor &tensor(PyObject *o, int64_t dim) {
    const at::Tensor &t = tensor(o);
    if (t.dim() != dim)
        raise(PyExc_ValueError, "expected " + std::to_string(dim) + " dimensions, got shape " +
                                    shape_text(t.sizes()));
    return t;
}

void check_kind(const at::Tensor &t, Kind k) {
    static const char *const names[] = {"torch.bfloat16", "torch.uint8", "torch.int32",
                                        "torch.float32"};
    if (!is_kind(t.scalar_type(), k))
        raise(PyExc_TypeError, std::string("expected ") + names[k] + ", got " +
                                   c10::toString(t.scalar_type()));
}

// The device of the present call: the current one, which its launches go to.
thread_local int here = -1;
int current_device() {
    if (here < 0) here = c10::cuda::current_device();
    return here;
}
void check_device(const at::Tensor &t) {
    if (t.get_device() != current_device())
        raise(PyExc_ValueError, "tensor is on CUDA device " + std::to_string(t.get_device()) +
                                    ", the current one is " + std::to_string(here));
}
void check_place(const at::Tensor &t) {
    if (!(t.is_cuda() && t.is_contiguous()))
        raise(PyExc_ValueError, "tensor must be on a CUDA device and contiguous");
    check_device(t);
}

template <typename T = void>
T *address(const at::Tensor &t, Kind k, at::IntArrayRef shape) {
    check_kind(t, k);
    if (t.sizes() != shape)
        raise(PyExc_ValueError,
              "expected shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    check_place(t);
    return static_cast<T *>(t.data_ptr());
}
template <typename T = void>
T *address(PyObject *o, Kind k, std::initializer_list<int64_t> shape) {
    return address<T>(tensor(o), k, at::IntArrayRef(shape.begin(), shape.size()));
}

int integer(PyObject *o) {
    long long v = PyLong_Check(o) ? PyLong_AsLongLong(o) : 0;
    if (!PyLong_Check(o)) {  // numpy's, for instance
        PyObject *i = PyNumber_Index(o);
        if (!i) throw Raised{};
        v = PyLong_AsLongLong(i);
        Py_DECREF(i);
    }
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < std::numeric_limits<int>::min() || v > std::numeric_limits<int>::max())
        raise(PyExc_OverflowError, "an argument does not fit in 32 bits");
    return static_cast<int>(v);
}
int integer(int64_t v) {
    if (v > std::numeric_limits<int>::max())
        raise(PyExc_OverflowError, "a dimension does not fit in 32 bits");
    return static_cast<int>(v);
}
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
}

mla_stream_t stream_of(PyObject *o) {
    if (o == Py_None)
        return reinterpret_cast<mla_stream_t>(
            c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(current_device())).stream());
    PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Raised{};
    void *p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw Raised{};
    return static_cast<mla_stream_t>(p);
}

struct Workspace {
    void *ptr;
    size_t bytes;
    explicit Workspace(PyObject *o) {
        const at::Tensor &t = tensor(o);
        check_place(t);
        ptr = t.data_ptr();
        bytes = t.nbytes();
    }
};

// kv_cache, or kv_codes and kv_exps (None with a bf16 cache)
struct Cache {
    mla_bf16_t *rows = nullptr;
    uint8_t *codes = nullptr;
    int8_t *exps = nullptr;
    int blocks;
    Cache(PyObject *cache, PyObject *e) {
        const at::Tensor &c = tensor(cache, 3);
        const int64_t n = c.size(0);
        blocks = integer(n);
        if (e == Py_None) {
            rows = address<mla_bf16_t>(cache, BF16, {n, BLOCK, D_QK});
        } else {
            codes = address<uint8_t>(cache, BYTES, {n, BLOCK, D_QK});
            exps = address<int8_t>(e, BYTES, {n, BLOCK});
        }
    }
};

// a cache of any format: kv_cache; kv_codes, kv_exps; kv_codes, kv_exps, kv_scales, kv_keys
struct AnyCache {
    mla_bf16_t *rows = nullptr;
    uint8_t *codes = nullptr;
    int8_t *exps = nullptr;
    uint8_t *scales = nullptr;
    mla_bf16_t *keys = nullptr;
    int blocks;
    explicit AnyCache(PyObject *const *a) {
        if (a[2] == Py_None) {
            const Cache c(a[0], a[1]);
            rows = c.rows, codes = c.codes, exps = c.exps, blocks = c.blocks;
            return;
        }
        const int64_t n = tensor(a[0], 3).size(0);
        blocks = integer(n);
        codes = address<uint8_t>(a[0], BYTES, {n, BLOCK, D_C / 2});
        exps = address<int8_t>(a[1], BYTES, {n, BLOCK});
        scales = address<uint8_t>(a[2], BYTES, {n, BLOCK, D_C / 16});
        keys = address<mla_bf16_t>(a[3], BF16, {n, BLOCK, D_ROPE});
    }
};

// a rotation's plan (mla.RopePlan)
struct Plan {
    mla_rope_t p;
    explicit Plan(PyObject *o) {
        Py_buffer b;
        if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Raised{};
        const bool ok = b.len == static_cast<Py_ssize_t>(sizeof(p));
        if (ok) std::memcpy(&p, b.buf, sizeof(p));
        PyBuffer_Release(&b);
        if (!ok) raise(PyExc_TypeError, "expected what rope_plan() gave");
    }
};

struct Table {
    int32_t *ptr;
    int64_t rows, most;
    explicit Table(PyObject *o) {
        const at::Tensor &t = tensor(o, 2);
        rows = t.size(0), most = t.size(1);
        ptr = address<int32_t>(o, I32, {rows, most});
        integer(rows), integer(most);
    }
};

// the call itself without the interpreter's lock
template <typename F>
mla_status_t without_lock(const F &f) {
    mla_status_t s;
    Py_BEGIN_ALLOW_THREADS
    s = f();
    Py_END_ALLOW_THREADS
    return s;
}

// q_lat q_rope cache exps block_table q_starts seqlens max_seqlen scale window sinks out lse
// workspace stream
mla_status_t chunk(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], 3);
    const int64_t T = q.size(0), H = q.size(1);
    const auto *q_lat = address<mla_bf16_t>(a[0], BF16, {T, H, D_C});
    const auto *q_rope = address<mla_bf16_t>(a[1], BF16, {T, H, D_ROPE});
    const Cache c(a[2], a[3]);
    const Table t(a[4]);
    const auto *starts = address<int32_t>(a[5], I32, {t.rows + 1});
    const auto *lens = address<int32_t>(a[6], I32, {t.rows});
    const int most = integer(a[7]), window = integer(a[9]), sinks = integer(a[10]);
    const float scale = real(a[8]);
    auto *out = address<mla_bf16_t>(a[11], BF16, {T, H, D_C});
    auto *lse = address<float>(a[12], F32, {T, H});
    const Workspace w(a[13]);
    const int B = integer(t.rows), tokens = integer(T), heads = integer(H);
    const mla_stream_t st = stream_of(a[14]);
    return without_lock([&] {
        return c.codes ? mla_chunk_attention_fp8(q_lat, q_rope, c.codes, c.exps, c.blocks, t.ptr,
                                                 t.most, starts, lens, B, tokens, heads, most,
                                                 window, sinks, scale, w.ptr, w.bytes, out, lse, st)
                       : mla_chunk_attention(q_lat, q_rope, c.rows, c.blocks, t.ptr, t.most, starts,
                                             lens, B, tokens, heads, most, window, sinks, scale,
                                             w.ptr, w.bytes, out, lse, st);
    });
}

// What the decode calls share: queries [B, H, 512] or [B, s_q, H, 512], the cache and its table,
// lengths, outputs in the queries' layout.
struct DecodeArgs {
    const mla_bf16_t *q_lat, *q_rope;
    Cache c;
    Table t;
    const int32_t *lens;
    mla_bf16_t *out;
    float *lse;
    int B, s_q, heads;
    DecodeArgs(PyObject *ql, PyObject *qr, PyObject *cache, PyObject *exps, PyObject *table,
               PyObject *seqlens, PyObject *o, PyObject *l)
        : c(cache, exps), t(table) {
        const at::Tensor &q = tensor(ql);
        if (q.dim() != 3 && q.dim() != 4)
            raise(PyExc_ValueError, "expected q_lat [B, H, 512] or [B, s_q, H, 512], got shape " +
                                        shape_text(q.sizes()));
        const int64_t b = q.size(0);
        // q_lat's shape with another width (or, for lse, none)
        int64_t shape[4];
        const size_t n = q.dim();
        for (size_t i = 0; i < n; ++i) shape[i] = q.size(i);
        auto wide = [&](int64_t d) { return shape[n - 1] = d, at::IntArrayRef(shape, n); };
        q_lat = address<mla_bf16_t>(q, BF16, wide(D_C));
        q_rope = address<mla_bf16_t>(tensor(qr), BF16, wide(D_ROPE));
        if (t.rows != b)
            raise(PyExc_ValueError, "expected shape (" + std::to_string(b) +
                                        ", ..) of block_table, got " + shape_text({t.rows, t.most}));
        lens = address<int32_t>(seqlens, I32, {b});
        out = address<mla_bf16_t>(tensor(o), BF16, wide(D_C));
        lse = address<float>(tensor(l), F32, at::IntArrayRef(shape, n - 1));
        B = integer(b), s_q = integer(n == 4 ? q.size(1) : 1), heads = integer(q.size(-2));
    }
};

// q_lat q_rope cache exps block_table seqlens max_seqlen window sinks scale num_splits out lse
// workspace stream
mla_status_t window(PyObject *const *a) {
    const DecodeArgs d(a[0], a[1], a[2], a[3], a[4], a[5], a[11], a[12]);
    const int most = integer(a[6]), win = integer(a[7]), sinks = integer(a[8]);
    const float scale = real(a[9]);
    const int splits = integer(a[10]);
    const Workspace w(a[13]);
    const mla_stream_t st = stream_of(a[14]);
    return without_lock([&] {
        return d.c.codes
                   ? mla_decode_attention_window_fp8(d.q_lat, d.q_rope, d.c.codes, d.c.exps,
                                                     d.c.blocks, d.t.ptr, d.t.most, d.lens, d.B,
                                                     d.s_q, d.heads, most, win, sinks, scale, splits,
                                                     w.ptr, w.bytes, d.out, d.lse, st)
                   : mla_decode_attention_window(d.q_lat, d.q_rope, d.c.rows, d.c.blocks, d.t.ptr,
                                                 d.t.most, d.lens, d.B, d.s_q, d.heads, most, win,
                                                 sinks, scale, splits, w.ptr, w.bytes, d.out, d.lse,
                                                 st);
    });
}

// q_lat q_rope cache exps block_table seqlens group_starts prefix_lens max_seqlen scale out lse
// workspace stream
mla_status_t shared(PyObject *const *a) {
    const DecodeArgs d(a[0], a[1], a[2], a[3], a[4], a[5], a[10], a[11]);
    const int64_t G = tensor(a[7], 1).size(0);
    const auto *prefix = address<int32_t>(a[7], I32, {G});
    const auto *starts = address<int32_t>(a[6], I32, {G + 1});
    const int most = integer(a[8]), groups = integer(G);
    const float scale = real(a[9]);
    const Workspace w(a[12]);
    const mla_stream_t st = stream_of(a[13]);
    return without_lock([&] {
        return d.c.codes
                   ? mla_decode_attention_shared_fp8(d.q_lat, d.q_rope, d.c.codes, d.c.exps,
                                                     d.c.blocks, d.t.ptr, d.t.most, d.lens, starts,
                                                     prefix, groups, d.B, d.s_q, d.heads, most,
                                                     scale, w.ptr, w.bytes, d.out, d.lse, st)
                   : mla_decode_attention_shared(d.q_lat, d.q_rope, d.c.rows, d.c.blocks, d.t.ptr,
                                                 d.t.most, d.lens, starts, prefix, groups, d.B,
                                                 d.s_q, d.heads, most, scale, w.ptr, w.bytes, d.out,
                                                 d.lse, st);
    });
}

// x w_q w_kv q_starts seqlens block_table, what the calls with the norms begin with, and c_q
struct NormArgs {
    const mla_bf16_t *x, *w_q, *w_kv;
    const int32_t *starts, *lens;
    Table t;
    mla_bf16_t *c_q;
    int64_t pitch;
    int B, tokens, q_lora;
    NormArgs(PyObject *const *a, PyObject *out) : t(a[5]) {
        const at::Tensor &in = tensor(a[0]);
        const bool rows = in.dim() == 2 && is_kind(in.scalar_type(), BF16) && in.is_cuda();
        const int64_t T = rows ? in.size(0) : 0, width = rows ? in.size(1) : 0, ql = width - D_QK;
        pitch = rows ? T == 1 ? width : in.stride(0) : 0;
        if (!rows || ql < 0 || in.stride(1) != 1 || pitch < width)
            raise(PyExc_ValueError, "x: a CUDA tensor of bf16 rows [tokens, q_lora + 576]");
        check_device(in);
        if (ql && a[1] == Py_None) raise(PyExc_ValueError, "w_q [q_lora] is wanted");
        w_q = ql ? address<mla_bf16_t>(a[1], BF16, {ql}) : nullptr;
        w_kv = address<mla_bf16_t>(a[2], BF16, {D_C});
        starts = address<int32_t>(a[3], I32, {t.rows + 1});
        lens = address<int32_t>(a[4], I32, {t.rows});
        c_q = ql ? address<mla_bf16_t>(out, BF16, {T, ql}) : nullptr;
        x = static_cast<const mla_bf16_t *>(in.data_ptr());
        B = integer(t.rows), tokens = integer(T), q_lora = integer(ql);
    }
};

// x w_q w_kv q_starts seqlens block_table cache exps rope_theta eps c_q workspace stream
mla_status_t norm(PyObject *const *a) {
    const NormArgs n(a, a[10]);
    const Cache c(a[6], a[7]);
    const float theta = real(a[8]), eps = real(a[9]);
    const Workspace w(a[11]);
    const mla_stream_t st = stream_of(a[12]);
    return without_lock([&] {
        return c.codes ? mla_norm_rope_append_fp8(n.x, n.pitch, n.q_lora, n.w_q, n.w_kv, eps, n.starts,
                                                  n.lens, n.B, n.tokens, n.t.ptr, n.t.most, c.codes,
                                                  c.exps, c.blocks, theta, n.c_q, w.ptr, w.bytes, st)
                       : mla_norm_rope_append(n.x, n.pitch, n.q_lora, n.w_q, n.w_kv, eps, n.starts,
                                              n.lens, n.B, n.tokens, n.t.ptr, n.t.most, c.rows,
                                              c.blocks, theta, n.c_q, w.ptr, w.bytes, st);
    });
}

// x w_q w_kv q_starts seqlens block_table cache exps scales keys plan eps c_q workspace stream
mla_status_t norm_plan(PyObject *const *a) {
    const NormArgs n(a, a[12]);
    const AnyCache c(a + 6);
    const Plan plan(a[10]);
    const float eps = real(a[11]);
    const Workspace w(a[13]);
    const mla_stream_t st = stream_of(a[14]);
    return without_lock([&] {
        if (c.scales)
            return mla_norm_rope_append_fp4(n.x, n.pitch, n.q_lora, n.w_q, n.w_kv, eps, n.starts, n.lens,
                                            n.B, n.tokens, n.t.ptr, n.t.most, c.codes, c.scales,
                                            c.exps, c.keys, c.blocks, &plan.p, n.c_q, w.ptr, w.bytes,
                                            st);
        return c.codes ? mla_norm_rope_append_scaled_fp8(n.x, n.pitch, n.q_lora, n.w_q, n.w_kv, eps,
                                                         n.starts, n.lens, n.B, n.tokens, n.t.ptr,
                                                         n.t.most, c.codes, c.exps, c.blocks, &plan.p,
                                                         n.c_q, w.ptr, w.bytes, st)
                       : mla_norm_rope_append_scaled(n.x, n.pitch, n.q_lora, n.w_q, n.w_kv, eps,
                                                     n.starts, n.lens, n.B, n.tokens, n.t.ptr, n.t.most,
                                                     c.rows, c.blocks, &plan.p, n.c_q, w.ptr, w.bytes,
                                                     st);
    });
}

// cache exps scales keys block_table first row_starts out workspace stream
mla_status_t read(PyObject *const *a) {
    const AnyCache c(a);
    const Table t(a[4]);
    const auto *first = a[5] == Py_None ? nullptr : address<int32_t>(a[5], I32, {t.rows});
    const auto *starts = address<int32_t>(a[6], I32, {t.rows + 1});
    const int64_t n = tensor(a[7], 2).size(0);
    auto *out = address<mla_bf16_t>(a[7], BF16, {n, D_QK});
    const Workspace w(a[8]);
    const int B = integer(t.rows), rows = integer(n);
    const mla_stream_t st = stream_of(a[9]);
    return without_lock([&] {
        if (c.scales)
            return mla_read_kv_fp4(c.codes, c.scales, c.exps, c.keys, c.blocks, t.ptr, t.most, first,
                                   starts, B, rows, out, w.ptr, w.bytes, st);
        return c.codes ? mla_read_kv_fp8(c.codes, c.exps, c.blocks, t.ptr, t.most, first, starts, B, rows,
                                         out, w.ptr, w.bytes, st)
                       : mla_read_kv(c.rows, c.blocks, t.ptr, t.most, first, starts, B, rows, out, w.ptr,
                                     w.bytes, st);
    });
}

// [tokens, heads, width] bf16, each head's values side by side
struct Heads {
    mla_bf16_t *ptr;
    int64_t tokens, heads, width, by_token, by_head;
    explicit Heads(PyObject *o) {
        const at::Tensor &t = tensor(o, 3);
        check_kind(t, BF16);
        if (!t.is_cuda() || (t.size(2) > 1 && t.stride(2) != 1))
            raise(PyExc_ValueError, "expected a CUDA tensor [tokens, heads, width] with its last "
                                    "dimension contiguous");
        check_device(t);
        ptr = static_cast<mla_bf16_t *>(t.data_ptr());
        tokens = t.size(0), heads = t.size(1), width = t.size(2);
        by_token = t.stride(0), by_head = t.stride(1);
    }
    void expect(const Heads &x, int64_t w) const {
        if (tokens != x.tokens || heads != x.heads || width != w)
            raise(PyExc_ValueError, "expected shape " + shape_text({x.tokens, x.heads, w}) + ", got " +
                                        shape_text({tokens, heads, width}));
    }
};

// x pos plan offset out rest stream
mla_status_t rope(PyObject *const *a) {
    const Heads x(a[0]), y(a[4]);
    const auto *pos = address<int32_t>(a[1], I32, {x.tokens});
    const Plan plan(a[2]);
    const int offset = integer(a[3]);
    y.expect(x, plan.p.rot);
    mla_bf16_t *rest = nullptr;
    int64_t rest_token = 0, rest_head = 0;
    if (a[5] != Py_None) {
        const Heads r(a[5]);
        r.expect(x, x.width - plan.p.rot);
        rest = r.ptr, rest_token = r.by_token, rest_head = r.by_head;
    }
    const int tokens = integer(x.tokens), heads = integer(x.heads), width = integer(x.width);
    const mla_stream_t st = stream_of(a[6]);
    return without_lock([&] {
        return mla_rope(x.ptr, x.by_token, x.by_head, tokens, heads, width, offset, &plan.p, pos, y.ptr,
                        y.by_token, y.by_head, rest, rest_token, rest_head, st);
    });
}

// refs block_table seqlens
struct Pages {
    int32_t *refs, *lens;
    Table table;
    int blocks, most, seqs;
    explicit Pages(PyObject *const *a) : table(a[1]) {
        const int64_t n = tensor(a[0], 1).size(0);
        refs = address<int32_t>(a[0], I32, {n});
        lens = address<int32_t>(a[2], I32, {table.rows});
        blocks = integer(n), most = integer(table.most), seqs = integer(table.rows);
    }
};
struct List {
    const int32_t *ptr;
    int n;
    explicit List(PyObject *o) {
        const int64_t m = tensor(o, 1).size(0);
        ptr = address<int32_t>(o, I32, {m});
        n = integer(m);
    }
    List(PyObject *o, int m) : ptr(address<int32_t>(o, I32, {m})), n(m) {}
};

// The mla_page_pool_t of a cache [layers, num_blocks, ...]; the layers may be strided, each contiguous.
mla_page_pool_t pool_of(const at::Tensor &t, int64_t blocks) {
    bool ok = t.dim() >= 3 && t.size(1) == blocks && t.is_cuda();
    int64_t run = 1;  // values of the dimensions behind the present one
    for (int64_t d = t.dim() - 1; ok && d >= 1; --d) {
        ok = t.size(d) == 1 || t.stride(d) == run;
        run *= t.size(d);
    }
    if (!ok)
        raise(PyExc_ValueError,
              "pools are CUDA tensors [layers, num_blocks, ...], each layer contiguous");
    check_device(t);
    const size_t size = t.element_size();
    return {t.data_ptr(), blocks > 0 ? static_cast<size_t>(run / blocks) * size : 0,
            static_cast<size_t>(t.stride(0)) * size, integer(t.size(0))};
}

// pools(list, num_blocks): mla_page_pool_t's as bytes, for the calls below
PyObject *make_pools(PyObject *const *a) {
    const int blocks = integer(a[1]);
    PyObject *s = PySequence_Fast(a[0], "pools: a list of tensors");
    if (!s) throw Raised{};
    mla_page_pool_t p[MLA_MAX_POOLS];
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(s);
    try {
        if (n > MLA_MAX_POOLS)
            raise(PyExc_ValueError, "at most " + std::to_string(MLA_MAX_POOLS) + " pools");
        for (Py_ssize_t k = 0; k < n; ++k)
            p[k] = pool_of(tensor(PySequence_Fast_GET_ITEM(s, k)), blocks);
    } catch (...) {
        Py_DECREF(s);
        throw;
    }
    Py_DECREF(s);
    return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(p), n * sizeof(p[0]));
}
struct Pools {
    mla_page_pool_t p[MLA_MAX_POOLS];
    int n;
    explicit Pools(PyObject *o) {
        if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) > static_cast<Py_ssize_t>(sizeof(p)))
            raise(PyExc_TypeError, "expected what pools() gave");
        std::memcpy(p, PyBytes_AS_STRING(o), PyBytes_GET_SIZE(o));
        n = static_cast<int>(PyBytes_GET_SIZE(o) / sizeof(p[0]));
    }
};

// refs block_table seqlens rows workspace stream
mla_status_t pages_free(PyObject *const *a) {
    const Pages s(a);
    const List rows(a[3]);
    const Workspace w(a[4]);
    const mla_stream_t st = stream_of(a[5]);
    return without_lock([&] {
        return mla_pages_free(s.refs, s.blocks, s.table.ptr, s.most, s.lens, s.seqs, rows.ptr, rows.n,
                              w.ptr, w.bytes, st);
    });
}

// refs block_table seqlens rows new_lens workspace stream
mla_status_t pages_extend(PyObject *const *a) {
    const Pages s(a);
    const List rows(a[3]), lens(a[4], rows.n);
    const Workspace w(a[5]);
    const mla_stream_t st = stream_of(a[6]);
    return without_lock([&] {
        return mla_pages_extend(s.refs, s.blocks, s.table.ptr, s.most, s.lens, s.seqs, rows.ptr,
                                lens.ptr, rows.n, w.ptr, w.bytes, st);
    });
}

// refs block_table seqlens parents children pools workspace stream
mla_status_t pages_fork(PyObject *const *a) {
    const Pages s(a);
    const List parents(a[3]), children(a[4], parents.n);
    const Pools pools(a[5]);
    const Workspace w(a[6]);
    const mla_stream_t st = stream_of(a[7]);
    return without_lock([&] {
        return mla_pages_fork(s.refs, s.blocks, s.table.ptr, s.most, s.lens, s.seqs, parents.ptr,
                              children.ptr, parents.n, pools.p, pools.n, w.ptr, w.bytes, st);
    });
}

// refs block_table seqlens pools refs_out table_out live workspace stream
mla_status_t pages_compact(PyObject *const *a) {
    const Pages s(a);
    const Pools pools(a[3]);
    auto *refs = address<int32_t>(a[4], I32, {s.blocks});
    auto *table = address<int32_t>(a[5], I32, {s.table.rows, s.table.most});
    auto *live = address<int32_t>(a[6], I32, {1});
    const Workspace w(a[7]);
    const mla_stream_t st = stream_of(a[8]);
    return without_lock([&] {
        return mla_pages_compact(s.refs, s.blocks, s.table.ptr, s.most, s.lens, s.seqs, refs, table,
                                 live, pools.p, pools.n, w.ptr, w.bytes, st);
    });
}

// No C++ exception leaves the module.
template <typename F>
PyObject *guarded(const F &f) {
    try {
        return f();
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject *result(PyObject *o) { return o; }
PyObject *result(mla_status_t s) { return PyLong_FromLong(s); }
template <Py_ssize_t N, auto F>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
    here = -1;
    return guarded([&] {
        if (n != N) raise(PyExc_TypeError, "expected " + std::to_string(N) + " arguments");
        return result(F(a));
    });
}

// address(tensor, kind, *shape)
PyObject *checked_address(PyObject *, PyObject *const *a, Py_ssize_t n) {
    here = -1;
    return guarded([&] {
        int64_t shape[8];
        if (n < 2 || n > 10) raise(PyExc_TypeError, "expected a tensor, a kind and a shape");
        const int k = integer(a[1]);
        if (k < BF16 || k > F32) raise(PyExc_ValueError, "no such kind");
        for (Py_ssize_t i = 2; i < n; ++i) shape[i - 2] = integer(a[i]);
        return PyLong_FromVoidPtr(
            address(tensor(a[0]), static_cast<Kind>(k), at::IntArrayRef(shape, n - 2)));
    });
}

template <typename F>
constexpr PyMethodDef method(const char *name, F f) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL,
            nullptr};
}

PyMethodDef methods[] = {method("chunk", entry<15, chunk>),
                         method("window", entry<15, window>),
                         method("shared", entry<14, shared>),
                         method("norm", entry<13, norm>),
                         method("norm_plan", entry<15, norm_plan>),
                         method("read", entry<10, read>),
                         method("rope", entry<7, rope>),
                         method("pages_free", entry<6, pages_free>),
                         method("pages_extend", entry<7, pages_extend>),
                         method("pages_fork", entry<8, pages_fork>),
                         method("pages_compact", entry<9, pages_compact>),
                         method("address", checked_address),
                         method("pools", entry<2, make_pools>),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "The ragged serving calls (see mla.py).", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject *m = PyModule_Create(&module);
    if (m && (PyModule_AddIntConstant(m, "BF16", BF16) < 0 ||
              PyModule_AddIntConstant(m, "I32", I32) < 0)) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
