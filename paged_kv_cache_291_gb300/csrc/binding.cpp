// binding.cpp -- the rotary and linear-attention calls, and those on pools with
// a scale per block, from torch tensors to the C-ABI of include/pkv.h, as a
// CPython module.
//
// These calls are made once per layer and step, and their kernels often take
// less time than it takes Python to read a dozen tensors' attributes.  Each
// function here checks its tensors (type, device, shape, layout), makes the
// library call on torch's current stream and returns its status.  Anything
// that is not a plain valid call (a wrong tensor, an output in host memory)
// gets None and launches nothing: the Python wrapper then says what is wrong,
// or makes the call itself.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "pkv.h"

namespace {

using Args = PyObject* const*;

// One call's tensors: every check clears `ok` when it fails.
struct Call {
    bool ok = true;
    int dev = c10::cuda::current_device();

    const at::Tensor* tensor(PyObject* o, c10::ScalarType type) {
        if (!ok || !THPVariable_Check(o)) return fail();
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type) return fail();
        return &t;
    }
    const at::Tensor* fail() {
        ok = false;
        return nullptr;
    }
    static bool has_shape(const at::Tensor& t, std::initializer_list<int64_t> shape) {
        return t.sizes() == c10::IntArrayRef(shape.begin(), shape.size());
    }
    // A contiguous tensor of the given shape.
    void* plain(PyObject* o, c10::ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor* t = tensor(o, type);
        if (t == nullptr || !has_shape(*t, shape) || !t->is_contiguous()) return const_cast<at::Tensor*>(fail());
        return t->data_ptr();
    }
    // bf16 rows [tokens][heads][d], the tokens any distance apart.
    void* rows(PyObject* o, int64_t tokens, int64_t heads, int64_t d, int64_t* stride) {
        const at::Tensor* t = tensor(o, c10::kBFloat16);
        if (t == nullptr || !has_shape(*t, {tokens, heads, d}) ||
            (tokens > 0 && (t->stride(2) != 1 || (heads > 1 && t->stride(1) != d))))
            return const_cast<at::Tensor*>(fail());
        *stride = tokens > 1 ? t->stride(0) : heads * d;
        return t->data_ptr();
    }
    bool dims(PyObject* o, int64_t n) {
        if (!ok || !THPVariable_Check(o) || THPVariable_Unpack(o).dim() != n) ok = false;
        return ok;
    }
    int64_t size(PyObject* o, int64_t i) const { return ok ? THPVariable_Unpack(o).size(i) : 0; }
    float real(PyObject* o) {
        const double x = PyFloat_AsDouble(o);
        if (x == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return static_cast<float>(x);
    }
    // An int that fits 32 bits.
    int32_t whole(PyObject* o) {
        if (!PyLong_CheckExact(o)) {
            ok = false;
            return 0;
        }
        int overflow = 0;
        const long x = PyLong_AsLongAndOverflow(o, &overflow);
        if (overflow != 0 || x < INT32_MIN || x > INT32_MAX) ok = false;
        return static_cast<int32_t>(x);
    }
    // The stream argument: None is torch's current stream; anything else is the wrapper's.
    void* stream(PyObject* o) {
        if (o != Py_None) {
            ok = false;
            return nullptr;
        }
        return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    }
};

constexpr int64_t kMaxInt = INT32_MAX;

PyObject* none() { Py_RETURN_NONE; }

PyObject* status(pkv_status st) { return PyLong_FromLong(static_cast<long>(st)); }

// positions, inv_freq, sections (None or a sequence of ints), interleaved, adjacent
bool fill_rotary(Call& c, Args a, int64_t tokens, pkv_rotary_t* r) {
    if (!c.ok || !THPVariable_Check(a[0])) return c.ok = false;
    const int64_t nd = THPVariable_Unpack(a[0]).dim();
    if (nd != 1 && nd != 2) return c.ok = false;
    const int64_t axes = nd == 1 ? 1 : c.size(a[0], 0);
    if (!c.dims(a[1], 1) || axes < 1 || axes > 4) return c.ok = false;
    const int64_t pairs = c.size(a[1], 0);
    if (pairs > 64) return c.ok = false;
    r->positions = static_cast<const int32_t*>(nd == 1 ? c.plain(a[0], c10::kInt, {tokens})
                                                       : c.plain(a[0], c10::kInt, {axes, tokens}));
    r->inv_freq = static_cast<const float*>(c.plain(a[1], c10::kFloat, {pairs}));
    r->rot_dim = static_cast<int32_t>(2 * pairs);
    r->num_axes = static_cast<int32_t>(axes);
    for (int i = 0; i < 4; ++i) r->sections[i] = 0;
    if (a[2] == Py_None) {
        if (axes != 1) return c.ok = false;
        r->sections[0] = static_cast<int32_t>(pairs);
    } else {
        if (!PyList_CheckExact(a[2]) && !PyTuple_CheckExact(a[2])) return c.ok = false;
        if (PySequence_Fast_GET_SIZE(a[2]) != axes) return c.ok = false;
        for (int64_t i = 0; i < axes; ++i) {
            const long x = PyLong_AsLong(PySequence_Fast_GET_ITEM(a[2], i));
            if (x < 0 || x > 64) {  // errors included
                PyErr_Clear();
                return c.ok = false;
            }
            r->sections[i] = static_cast<int32_t>(x);
        }
    }
    const int interleaved = PyObject_IsTrue(a[3]), adjacent = PyObject_IsTrue(a[4]);
    if (interleaved < 0 || adjacent < 0) {
        PyErr_Clear();
        return c.ok = false;
    }
    r->flags = (adjacent ? PKV_ROTARY_ADJACENT_PAIRS : 0) | (interleaved ? PKV_ROTARY_INTERLEAVED_AXES : 0);
    return c.ok;
}

// q, k, positions, inv_freq, sections, interleaved, adjacent, q_out, k_out, stream
PyObject* rotary(PyObject*, Args a, Py_ssize_t n) {
    if (n != 10) return none();
    Call c;
    if (!c.dims(a[0], 3) || !c.dims(a[1], 3)) return none();
    const int64_t T = c.size(a[0], 0), hq = c.size(a[0], 1), d = c.size(a[0], 2), hkv = c.size(a[1], 1);
    if (T > kMaxInt || hq > kMaxInt || hkv > kMaxInt || d > kMaxInt) return none();
    int64_t qs = 0, ks = 0;
    pkv_rotary_t r;
    const void* q = c.rows(a[0], T, hq, d, &qs);
    const void* k = c.rows(a[1], T, hkv, d, &ks);
    fill_rotary(c, a + 2, T, &r);
    void* qo = c.plain(a[7], c10::kBFloat16, {T, hq, d});
    void* ko = c.plain(a[8], c10::kBFloat16, {T, hkv, d});
    void* stream = c.stream(a[9]);
    if (!c.ok) return none();
    return status(pkv_rotary(&r, q, qs, static_cast<int32_t>(hq), k, ks, static_cast<int32_t>(hkv),
                             static_cast<int32_t>(d), static_cast<int32_t>(T), qo, ko, stream));
}

// k_pool, v_pool, q, k, v, slot_mapping, positions, inv_freq, sections, interleaved, adjacent, q_out, k_scale,
// v_scale, stream
PyObject* rotary_cache_write(PyObject*, Args a, Py_ssize_t n) {
    if (n != 15) return none();
    Call c;
    if (!c.dims(a[0], 4) || !c.dims(a[2], 3)) return none();
    const at::Tensor& pool = THPVariable_Unpack(a[0]);
    const c10::ScalarType type = pool.scalar_type();
    const bool e4m3 = type == c10::kByte || type == c10::ScalarType::Float8_e4m3fn;
    if (!e4m3 && type != c10::kBFloat16) return none();
    const int64_t nb = c.size(a[0], 0), hkv = c.size(a[0], 1), bs = c.size(a[0], 2), d = c.size(a[0], 3);
    const int64_t T = c.size(a[2], 0), hq = c.size(a[2], 1);
    if (nb > kMaxInt || hkv > kMaxInt || bs != 16 || T > kMaxInt || hq > kMaxInt) return none();
    pkv_cache_t cache;
    cache.k_pool = c.plain(a[0], type, {nb, hkv, bs, d});
    cache.v_pool = c.plain(a[1], type, {nb, hkv, bs, d});
    cache.num_blocks = static_cast<int32_t>(nb);
    cache.num_kv_heads = static_cast<int32_t>(hkv);
    cache.head_dim = static_cast<int32_t>(d);
    cache.block_size = 16;
    cache.kv_dtype = e4m3 ? PKV_KV_E4M3 : PKV_KV_BF16;
    cache.k_scale = cache.v_scale = 1.f;
    cache.block_scales = nullptr;
    if (e4m3) {
        cache.k_scale = c.real(a[12]);
        cache.v_scale = c.real(a[13]);
    }
    int64_t qs = 0, ks = 0, vs = 0;
    pkv_rotary_t r;
    const void* q = c.rows(a[2], T, hq, d, &qs);
    const void* k = c.rows(a[3], T, hkv, d, &ks);
    const void* v = c.rows(a[4], T, hkv, d, &vs);
    const void* slots = c.plain(a[5], c10::kInt, {T});
    fill_rotary(c, a + 6, T, &r);
    void* qo = c.plain(a[11], c10::kBFloat16, {T, hq, d});
    void* stream = c.stream(a[14]);
    if (!c.ok) return none();
    return status(pkv_rotary_cache_write(&cache, &r, q, qs, static_cast<int32_t>(hq), k, ks, v, vs,
                                         static_cast<const int32_t*>(slots), static_cast<int32_t>(T), qo, stream));
}

struct Linear {
    pkv_states_t states;
    const void *q, *k, *v, *slots, *new_slots, *ctx;
    int64_t qs = 0, ks = 0, vs = 0, T, hq, S;
    void *out, *stream;
    float scale;
};

// states, log_decay, q, k, v, state_slots, context_lens, scale, new_slots (or None), out, stream
void fill_linear(Call& c, Args a, Linear* l) {
    if (!c.dims(a[0], 4) || !c.dims(a[2], 3) || !c.dims(a[6], 1)) return;
    const int64_t slots = c.size(a[0], 0), hkv = c.size(a[0], 1), d = c.size(a[2], 2);
    l->T = c.size(a[2], 0);
    l->hq = c.size(a[2], 1);
    l->S = c.size(a[6], 0);
    if (slots > kMaxInt || hkv > kMaxInt || l->T > kMaxInt || l->hq > kMaxInt || l->S > kMaxInt) {
        c.ok = false;
        return;
    }
    l->states.states = static_cast<float*>(c.plain(a[0], c10::kFloat, {slots, hkv, d, d}));
    l->states.log_decay = static_cast<const float*>(c.plain(a[1], c10::kFloat, {hkv}));
    l->states.num_slots = static_cast<int32_t>(slots);
    l->states.num_kv_heads = static_cast<int32_t>(hkv);
    l->states.head_dim = static_cast<int32_t>(d);
    l->q = c.rows(a[2], l->T, l->hq, d, &l->qs);
    l->k = c.rows(a[3], l->T, hkv, d, &l->ks);
    l->v = c.rows(a[4], l->T, hkv, d, &l->vs);
    l->slots = c.plain(a[5], c10::kInt, {l->S});
    l->ctx = c.plain(a[6], c10::kInt, {l->S});
    l->scale = c.real(a[7]);
    l->new_slots = a[8] == Py_None ? nullptr : c.plain(a[8], c10::kInt, {l->S});
    l->out = c.plain(a[9], c10::kFloat, {l->T, l->hq, d});
    l->stream = c.stream(a[10]);
}

PyObject* linear_decode(PyObject*, Args a, Py_ssize_t n) {
    if (n != 11) return none();
    Call c;
    Linear l;
    fill_linear(c, a, &l);
    if (!c.ok || l.T != l.S) return none();
    return status(pkv_linear_decode_attention(&l.states, l.q, l.qs, static_cast<int32_t>(l.hq), l.k, l.ks, l.v, l.vs,
                                              static_cast<const int32_t*>(l.slots),
                                              static_cast<const int32_t*>(l.new_slots),
                                              static_cast<const int32_t*>(l.ctx), static_cast<int32_t>(l.S), l.scale,
                                              static_cast<float*>(l.out), l.stream));
}

// the eleven of the decode call, then query_start_loc, query_start_loc_host (int32 CPU tensor), workspace
PyObject* linear_prefill(PyObject*, Args a, Py_ssize_t n) {
    if (n != 14) return none();
    Call c;
    Linear l;
    fill_linear(c, a, &l);
    if (!c.ok || !THPVariable_Check(a[12]) || !THPVariable_Check(a[13])) return none();
    const void* qsl = c.plain(a[11], c10::kInt, {l.S + 1});
    const at::Tensor& host = THPVariable_Unpack(a[12]);
    const at::Tensor& ws = THPVariable_Unpack(a[13]);
    if (!c.ok || !host.is_cpu() || host.scalar_type() != c10::kInt || host.dim() != 1 || host.size(0) != l.S + 1 ||
        !host.is_contiguous() || !ws.is_cuda() || ws.get_device() != c.dev || !ws.is_contiguous())
        return none();
    return status(pkv_linear_prefill_attention(
        &l.states, l.q, l.qs, static_cast<int32_t>(l.hq), l.k, l.ks, l.v, l.vs, static_cast<int32_t>(l.T),
        static_cast<const int32_t*>(qsl), static_cast<const int32_t*>(host.data_ptr()),
        static_cast<const int32_t*>(l.slots), static_cast<const int32_t*>(l.new_slots),
        static_cast<const int32_t*>(l.ctx), static_cast<int32_t>(l.S), l.scale, static_cast<float*>(l.out),
        ws.data_ptr(), ws.nbytes(), l.stream));
}

// k_pool, v_pool, block_scales: pools with a scale for each (block, kv head).
void fill_scaled(Call& c, Args a, pkv_cache_t* cache) {
    if (!c.dims(a[0], 4)) return;
    const c10::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
    const bool int8 = type == c10::kChar;
    const int64_t nb = c.size(a[0], 0), hkv = c.size(a[0], 1), d = c.size(a[0], 3);
    if ((!int8 && type != c10::kByte && type != c10::ScalarType::Float8_e4m3fn) || nb > kMaxInt || hkv > kMaxInt ||
        d > kMaxInt) {
        c.ok = false;
        return;
    }
    cache->k_pool = c.plain(a[0], type, {nb, hkv, 16, d});
    cache->v_pool = c.plain(a[1], type, {nb, hkv, 16, d});
    cache->block_scales = static_cast<float*>(c.plain(a[2], c10::kFloat, {nb, hkv, 2}));
    cache->num_blocks = static_cast<int32_t>(nb);
    cache->num_kv_heads = static_cast<int32_t>(hkv);
    cache->head_dim = static_cast<int32_t>(d);
    cache->block_size = 16;
    cache->kv_dtype = int8 ? PKV_KV_INT8_BLOCKS : PKV_KV_E4M3_BLOCKS;
    cache->k_scale = cache->v_scale = 1.f;
}

// query_start_loc, context_lens, block_tables
struct Index {
    const int32_t *start, *lens, *tables;
    int32_t seqs, wide;
};

void fill_index(Call& c, PyObject* start, PyObject* lens, PyObject* tables, Index* x) {
    if (!c.dims(lens, 1) || !c.dims(tables, 2)) return;
    const int64_t seqs = c.size(lens, 0), wide = c.size(tables, 1);
    if (seqs >= kMaxInt || wide > kMaxInt) {
        c.ok = false;
        return;
    }
    x->seqs = static_cast<int32_t>(seqs);
    x->wide = static_cast<int32_t>(wide);
    x->start = start == nullptr ? nullptr : static_cast<const int32_t*>(c.plain(start, c10::kInt, {seqs + 1}));
    x->lens = static_cast<const int32_t*>(c.plain(lens, c10::kInt, {seqs}));
    x->tables = static_cast<const int32_t*>(c.plain(tables, c10::kInt, {seqs, wide}));
}

// k_pool, v_pool, block_scales, k_new, v_new, query_start_loc, context_lens, block_tables, stream
PyObject* cache_append(PyObject*, Args a, Py_ssize_t n) {
    if (n != 9) return none();
    Call c;
    pkv_cache_t cache;
    Index x;
    fill_scaled(c, a, &cache);
    fill_index(c, a[5], a[6], a[7], &x);
    if (!c.dims(a[3], 3)) return none();
    const int64_t T = c.size(a[3], 0);
    int64_t ks = 0, vs = 0;
    const void* k = c.rows(a[3], T, cache.num_kv_heads, cache.head_dim, &ks);
    const void* v = c.rows(a[4], T, cache.num_kv_heads, cache.head_dim, &vs);
    void* stream = c.stream(a[8]);
    if (!c.ok || T > kMaxInt) return none();
    return status(pkv_cache_append(&cache, k, ks, v, vs, static_cast<int32_t>(T), x.start, x.lens, x.seqs, x.tables,
                                   x.wide, stream));
}

// k_pool, v_pool, block_scales, query_start_loc, context_lens, block_tables, num_tokens, k_out, v_out, stream
PyObject* cache_read(PyObject*, Args a, Py_ssize_t n) {
    if (n != 10) return none();
    Call c;
    pkv_cache_t cache;
    Index x;
    fill_scaled(c, a, &cache);
    fill_index(c, a[3], a[4], a[5], &x);
    const int32_t T = c.whole(a[6]);
    if (!c.ok) return none();
    void* k = c.plain(a[7], c10::kBFloat16, {T, cache.num_kv_heads, cache.head_dim});
    void* v = c.plain(a[8], c10::kBFloat16, {T, cache.num_kv_heads, cache.head_dim});
    void* stream = c.stream(a[9]);
    if (!c.ok) return none();
    return status(pkv_cache_read(&cache, k, v, T, x.start, x.lens, x.seqs, x.tables, x.wide, stream));
}

// A workspace: any contiguous tensor of the device.
const at::Tensor* workspace(Call& c, PyObject* o) {
    if (!c.ok || !THPVariable_Check(o)) return c.fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != c.dev || !t.is_contiguous()) return c.fail();
    return &t;
}

// k_pool, v_pool, block_scales, q, block_tables, context_lens, max_context_len, scale, out, workspace,
// partition_blocks, stream
PyObject* decode_scaled(PyObject*, Args a, Py_ssize_t n) {
    if (n != 12) return none();
    Call c;
    pkv_cache_t cache;
    Index x;
    fill_scaled(c, a, &cache);
    fill_index(c, nullptr, a[5], a[4], &x);
    if (!c.dims(a[3], 3)) return none();
    const int64_t hq = c.size(a[3], 1);
    const void* q = c.plain(a[3], c10::kBFloat16, {x.seqs, hq, cache.head_dim});
    const int32_t longest = c.whole(a[6]), part = c.whole(a[10]);
    const float scale = c.real(a[7]);
    void* out = c.plain(a[8], c10::kFloat, {x.seqs, hq, cache.head_dim});
    const at::Tensor* ws = workspace(c, a[9]);
    void* stream = c.stream(a[11]);
    if (!c.ok || hq > kMaxInt) return none();
    return status(pkv_decode_attention(&cache, q, static_cast<int32_t>(hq), x.tables, x.wide, x.lens, x.seqs, longest,
                                       scale, static_cast<float*>(out), ws->data_ptr(), ws->nbytes(), part, stream));
}

// k_pool, v_pool, block_scales, q, query_start_loc, query_start_loc_host (int32 CPU tensor), context_lens,
// block_tables, max_context_len, scale, out, workspace, stream
PyObject* prefill_scaled(PyObject*, Args a, Py_ssize_t n) {
    if (n != 13) return none();
    Call c;
    pkv_cache_t cache;
    Index x;
    fill_scaled(c, a, &cache);
    fill_index(c, a[4], a[6], a[7], &x);
    if (!c.dims(a[3], 3) || !THPVariable_Check(a[5])) return none();
    const int64_t T = c.size(a[3], 0), hq = c.size(a[3], 1);
    const void* q = c.plain(a[3], c10::kBFloat16, {T, hq, cache.head_dim});
    const int32_t longest = c.whole(a[8]);
    const float scale = c.real(a[9]);
    void* out = c.plain(a[10], c10::kFloat, {T, hq, cache.head_dim});
    const at::Tensor* ws = workspace(c, a[11]);
    void* stream = c.stream(a[12]);
    const at::Tensor& host = THPVariable_Unpack(a[5]);
    if (!c.ok || T > kMaxInt || hq > kMaxInt || !host.is_cpu() || host.scalar_type() != c10::kInt || host.dim() != 1 ||
        host.size(0) != x.seqs + 1 || !host.is_contiguous())
        return none();
    return status(pkv_chunked_prefill_attention(
        &cache, q, static_cast<int32_t>(hq), static_cast<int32_t>(T), x.start,
        static_cast<const int32_t*>(host.data_ptr()), x.lens, x.seqs, x.tables, x.wide, longest, scale,
        static_cast<float*>(out), ws->data_ptr(), ws->nbytes(), stream));
}

// C++ exceptions end here: torch's accessors may throw on unusual tensors.
template <PyObject* (*F)(PyObject*, Args, Py_ssize_t)>
PyObject* guarded(PyObject* self, Args a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (...) {
        return none();
    }
}

template <PyObject* (*F)(PyObject*, Args, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&guarded<F>)), METH_FASTCALL,
            nullptr};
}

PyMethodDef g_methods[] = {method<rotary>("rotary"), method<rotary_cache_write>("rotary_cache_write"),
                           method<linear_decode>("linear_decode"), method<linear_prefill>("linear_prefill"),
                           method<cache_append>("cache_append"), method<cache_read>("cache_read"),
                           method<decode_scaled>("decode_scaled"), method<prefill_scaled>("prefill_scaled"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
