// binding.cpp -- the torch side of the calls of a serving step with drafted tokens.
//
// These calls take 2 to 20 us on the GPU, and a step makes several in every layer. Checking ten tensors from
// Python and marshalling twenty arguments takes as long again, so that it is done here: a tensor's type, shape,
// strides, device and address are read from the object itself. Every check raises before anything is launched.
// Nothing is computed here; each function ends in one call of the C ABI.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>

#include "mla_latent_kv.h"

namespace {

struct Raised {};  // a Python exception is set

PyObject* g_error = nullptr;  // MlaError

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Raised{};
}

std::string shape_of(c10::IntArrayRef s) {
    std::ostringstream o;
    o << '(';
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << ')';
    return o.str();
}

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}
const at::Tensor* maybe(const char* name, PyObject* o) { return o == Py_None ? nullptr : &tensor(name, o); }

[[noreturn]] void wrong(const char* name, const at::Tensor& t, const std::string& wanted) {
    std::ostringstream o;
    o << name << " must be " << wanted << ", got " << t.scalar_type() << ' ' << shape_of(t.sizes())
      << " (contiguous=" << (t.is_contiguous() ? "True" : "False") << ", device=" << t.device() << ')';
    refuse(PyExc_ValueError, o.str());
}
// A contiguous tensor of the type and shape, or number of dimensions.
void is_shape(const char* name, const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape) {
    if (t.scalar_type() != type || !t.sizes().equals(c10::IntArrayRef(shape.begin(), shape.size())) || !t.is_contiguous())
        wrong(name, t, std::string("a contiguous ") + c10::toString(type) + " tensor of shape " +
                           shape_of(c10::IntArrayRef(shape.begin(), shape.size())));
}
void has_dims(const char* name, const at::Tensor& t, at::ScalarType type, int64_t dims) {
    if (t.scalar_type() != type || t.dim() != dims || !t.is_contiguous())
        wrong(name, t, std::string("a contiguous ") + c10::toString(type) + " tensor with " + std::to_string(dims) + " dimensions");
}
// bf16 rows of the shape with unit inner stride; their own strides are free.
void is_rows(const char* name, const at::Tensor& t, std::initializer_list<int64_t> shape) {
    if (t.scalar_type() != at::kBFloat16 || !t.sizes().equals(c10::IntArrayRef(shape.begin(), shape.size())) ||
        t.strides().back() != 1)
        wrong(name, t, "BFloat16 of shape " + shape_of(c10::IntArrayRef(shape.begin(), shape.size())) + " with unit inner stride");
}
const double* frequencies(const at::Tensor& t) {
    if (t.scalar_type() != at::kDouble || t.dim() != 1 || t.size(0) != MLA_ROPE_DIM / 2 || !t.is_contiguous() || !t.is_cpu())
        wrong("inv_freq", t, "a contiguous float64 CPU tensor of 32 elements");
    return static_cast<const double*>(t.data_ptr());
}
int32_t* status_word(const at::Tensor* t) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kInt || t->numel() < 1) wrong("dev_status", *t, "an int32 tensor of at least one element");
    return static_cast<int32_t*>(t->data_ptr());
}

// The launches go to the current device, which must be that of every tensor; the stream is the one given as an
// integer, else the current one.
mla_stream_t stream_for(PyObject* stream, const at::Tensor& first, std::initializer_list<const at::Tensor*> others) {
    if (!first.is_cuda() || first.get_device() != c10::cuda::current_device())
        refuse(PyExc_ValueError, "tensors must be on the current CUDA device, got " + first.device().str());
    for (const at::Tensor* t : others)
        if (t && t->device() != first.device())
            refuse(PyExc_ValueError, "tensors must be on one CUDA device, got " + first.device().str() + " and " + t->device().str());
    if (stream == Py_None) return reinterpret_cast<mla_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
    void* s = PyLong_AsVoidPtr(stream);
    if (PyErr_Occurred()) throw Raised{};
    return static_cast<mla_stream_t>(s);
}

void check(mla_status st) {
    if (st == MLA_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, mla_last_error_detail());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
int number(PyObject* o) {
    const int64_t v = integer(o);
    if (v != (int)v) refuse(PyExc_OverflowError, "a number is out of the range of a C int");
    return (int)v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}
int truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v;
}

int64_t page_bytes(int kv) {
    const int64_t row = mla_kv_row_bytes((mla_kv_dtype)kv);
    if (row < 0) {
        PyObject* e = PyObject_CallFunction(g_error, "is", (int)MLA_ERR_INVALID_ARG, "unknown kv_dtype");
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        throw Raised{};
    }
    return row * MLA_PAGE_SIZE;
}
int as_int(int64_t v) {
    if (v > INT32_MAX) refuse(PyExc_ValueError, "a tensor has " + std::to_string(v) + " rows, too many");
    return (int)v;
}
// Blocks of the cache, checked against its size when given.
int64_t cache_blocks(const at::Tensor& t, int kv, PyObject* num_blocks) {
    const int64_t have = (int64_t)t.nbytes() / page_bytes(kv), n = num_blocks == Py_None ? have : integer(num_blocks);
    if (!t.is_contiguous() || n > have)
        refuse(PyExc_ValueError, "kv_cache must be contiguous and hold num_blocks=" + std::to_string(n) + " pages (it holds " +
                                     std::to_string(have) + ")");
    return n;
}
// (layers, blocks) of a cache [num_blocks, page] or [layers, num_blocks, page].
std::pair<int, int64_t> layer_blocks(const at::Tensor& t, int kv) {
    const int64_t page = page_bytes(kv);
    if ((t.dim() != 2 && t.dim() != 3) || !t.is_contiguous() || t.size(-1) * (int64_t)t.element_size() != page)
        wrong("kv_cache", t, "contiguous [num_blocks, page] or [layers, num_blocks, page] with pages of " + std::to_string(page) +
                                 " bytes");
    return {t.dim() == 2 ? 1 : as_int(t.size(0)), t.size(-2)};
}

at::Tensor make(c10::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::empty(shape, like.options().dtype(type).requires_grad(false));
}

template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
void wants(Py_ssize_t n, Py_ssize_t got) {
    if (n != got) refuse(PyExc_TypeError, "wrong number of arguments");
}
PyObject* keep(PyObject* o) {
    Py_INCREF(o);
    return o;
}

// rope(x, positions, inv_freq, adjacent, mscale, out | None, stream | None) -> out
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded([&]() -> PyObject* {
        wants(7, na);
        const at::Tensor &x = tensor("x", a[0]), &pos = tensor("positions", a[1]), &freq = tensor("inv_freq", a[2]);
        if (x.dim() != 3) wrong("x", x, "[T, N, 64]");
        const int64_t T = x.size(0), N = x.size(1);
        is_rows("x", x, {T, N, MLA_ROPE_DIM});
        is_shape("positions", pos, at::kInt, {T});
        const double* w = frequencies(freq);
        at::Tensor made;
        const at::Tensor* out = maybe("out", a[5]);
        if (!out) {
            made = make(x.sizes(), at::kBFloat16, x);
            out = &made;
        }
        is_rows("out", *out, {T, N, MLA_ROPE_DIM});
        const mla_stream_t s = stream_for(a[6], x, {&pos, out});
        check(mla_rope(x.data_ptr(), x.stride(0), x.stride(1), (const int32_t*)pos.data_ptr(), w, real(a[4]), truth(a[3]),
                       out->data_ptr(), out->stride(0), out->stride(1), as_int(T), as_int(N), s));
        return made.defined() ? THPVariable_Wrap(made) : keep(a[5]);
    });
}

// rope_cache_write(kv_c, k_pe, positions, inv_freq, slot_mapping, kv_cache, kv_dtype, adjacent, mscale, kv_scale,
//                  q_pe | None, q_out | None, dev_status | None, stream | None, num_blocks | None) -> kv_cache
PyObject* rope_cache_write(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded([&]() -> PyObject* {
        wants(15, na);
        const at::Tensor &kv_c = tensor("kv_c", a[0]), &k_pe = tensor("k_pe", a[1]), &pos = tensor("positions", a[2]),
                         &freq = tensor("inv_freq", a[3]), &slots = tensor("slot_mapping", a[4]), &cache = tensor("kv_cache", a[5]);
        const at::Tensor *q = maybe("q_pe", a[10]), *out = maybe("q_out", a[11]), *st = maybe("dev_status", a[12]);
        const int kv = number(a[6]);
        has_dims("slot_mapping", slots, at::kLong, 1);
        const int64_t T = slots.size(0);
        is_rows("kv_c", kv_c, {T, MLA_KV_LORA_RANK});
        is_rows("k_pe", k_pe, {T, MLA_ROPE_DIM});
        is_shape("positions", pos, at::kInt, {T});
        const double* w = frequencies(freq);
        if (!q != !out) refuse(PyExc_ValueError, "q_pe and q_out go together");
        int64_t H = 1;
        if (q) {
            if (q->dim() != 3) wrong("q_pe", *q, "[T, H, 64]");
            H = q->size(1);
            is_rows("q_pe", *q, {T, H, MLA_ROPE_DIM});
            is_rows("q_out", *out, {T, H, MLA_ROPE_DIM});
        }
        const int64_t nb = cache_blocks(cache, kv, a[14]);
        int32_t* status = status_word(st);
        const mla_stream_t s = stream_for(a[13], cache, {&kv_c, &k_pe, &pos, &slots, q, out, st});
        check(mla_rope_cache_write(kv_c.data_ptr(), kv_c.stride(0), k_pe.data_ptr(), k_pe.stride(0), q ? q->data_ptr() : nullptr,
                                   q ? q->stride(0) : 0, q ? q->stride(1) : 0, q ? out->data_ptr() : nullptr,
                                   q ? out->stride(0) : 0, q ? out->stride(1) : 0, (const int32_t*)pos.data_ptr(), w, real(a[8]),
                                   truth(a[7]), (const int64_t*)slots.data_ptr(), as_int(T), as_int(H), cache.data_ptr(),
                                   (mla_kv_dtype)kv, nb, real(a[9]), status, s));
        return keep(a[5]);
    });
}

// decode_tree(q, kv_cache, block_table, seq_lens, tree_mask, max_seq_len, scale, kv_dtype, workspace | None,
//             o_latent | None, o_dtype | None, lse | None, dev_status | None, stream | None, num_blocks | None) -> (o_latent, lse)
PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded([&]() -> PyObject* {
        wants(15, na);
        const at::Tensor &q = tensor("q", a[0]), &cache = tensor("kv_cache", a[1]), &table = tensor("block_table", a[2]),
                         &lens = tensor("seq_lens", a[3]), &mask = tensor("tree_mask", a[4]);
        const at::Tensor *ws = maybe("workspace", a[8]), *o = maybe("o_latent", a[9]), *lse = maybe("lse", a[11]),
                         *st = maybe("dev_status", a[12]);
        const int max_len = number(a[5]), kv = number(a[7]);
        has_dims("q", q, at::kBFloat16, 4);
        const int64_t B = q.size(0), Sq = q.size(1), H = q.size(2);
        is_shape("q", q, at::kBFloat16, {B, Sq, H, MLA_HEAD_DIM});
        has_dims("block_table", table, at::kInt, 2);
        is_shape("block_table", table, at::kInt, {B, table.size(1)});
        is_shape("seq_lens", lens, at::kInt, {B});
        is_shape("tree_mask", mask, at::kLong, {B, Sq});
        const int64_t nb = cache_blocks(cache, kv, a[14]);
        const int o_dtype = a[10] != Py_None ? number(a[10]) : o && o->scalar_type() == at::kBFloat16 ? MLA_DT_BF16 : MLA_DT_F32;
        const at::ScalarType o_type = o_dtype == MLA_DT_F32 ? at::kFloat : at::kBFloat16;
        at::Tensor made_o, made_lse, made_ws;
        if (!o) made_o = make({B, Sq, H, MLA_KV_LORA_RANK}, o_type, q);
        if (!lse) made_lse = make({B, Sq, H}, at::kFloat, q);
        if (o && (o->scalar_type() != o_type || o->numel() < B * Sq * H * MLA_KV_LORA_RANK || !o->is_contiguous()))
            wrong("o_latent", *o, std::string("a contiguous ") + c10::toString(o_type) + " tensor that holds the result");
        if (lse && (lse->scalar_type() != at::kFloat || lse->numel() < B * Sq * H || !lse->is_contiguous()))
            wrong("lse", *lse, "a contiguous Float tensor that holds the result");
        if (ws && !ws->is_contiguous()) wrong("workspace", *ws, "contiguous");
        const at::Tensor *ot = o ? o : &made_o, *lt = lse ? lse : &made_lse;
        int32_t* status = status_word(st);
        const mla_stream_t s = stream_for(a[13], q, {&cache, &table, &lens, &mask, ot, lt, ws, st});
        if (!ws) {
            const size_t need = mla_decode_tree_workspace_bytes((mla_kv_dtype)kv, as_int(B), as_int(Sq), as_int(H), max_len);
            if (need) {
                made_ws = make({(int64_t)need}, at::kByte, q);
                ws = &made_ws;
            }
        }
        check(mla_decode_tree(q.data_ptr(), cache.data_ptr(), (mla_kv_dtype)kv, nb, (const int32_t*)table.data_ptr(),
                              as_int(table.size(1)), (const int32_t*)lens.data_ptr(), (const uint64_t*)mask.data_ptr(), max_len,
                              as_int(B), as_int(Sq), as_int(H), real(a[6]), ws ? ws->data_ptr() : nullptr, ws ? ws->nbytes() : 0,
                              ot->data_ptr(), (mla_dtype)o_dtype, (float*)lt->data_ptr(), status, s));
        PyObject* ro = o ? keep(a[9]) : THPVariable_Wrap(made_o);
        PyObject* rl = lse ? keep(a[11]) : THPVariable_Wrap(made_lse);
        return Py_BuildValue("(NN)", ro, rl);
    });
}

// accept_tokens(kv_cache, block_table, seq_lens, path, counts, kv_dtype, new_lens | None, dev_status | None,
//               stream | None) -> new_lens
PyObject* accept_tokens(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded([&]() -> PyObject* {
        wants(9, na);
        const at::Tensor &cache = tensor("kv_cache", a[0]), &table = tensor("block_table", a[1]), &lens = tensor("seq_lens", a[2]),
                         &path = tensor("path", a[3]), &counts = tensor("counts", a[4]);
        const at::Tensor *out = maybe("new_lens", a[6]), *st = maybe("dev_status", a[7]);
        const int kv = number(a[5]);
        has_dims("block_table", table, at::kInt, 2);
        const int64_t B = table.size(0);
        is_shape("seq_lens", lens, at::kInt, {B});
        has_dims("path", path, at::kInt, 2);
        is_shape("path", path, at::kInt, {B, path.size(1)});
        is_shape("counts", counts, at::kInt, {B});
        const auto [layers, nb] = layer_blocks(cache, kv);
        at::Tensor made;
        if (!out) {
            made = make({B}, at::kInt, lens);
            out = &made;
        }
        is_shape("new_lens", *out, at::kInt, {B});
        int32_t* status = status_word(st);
        const mla_stream_t s = stream_for(a[8], cache, {&table, &lens, &path, &counts, out, st});
        check(mla_accept_tokens(cache.data_ptr(), (mla_kv_dtype)kv, layers, nb, (const int32_t*)table.data_ptr(),
                                as_int(table.size(1)), (const int32_t*)lens.data_ptr(), (const int32_t*)path.data_ptr(),
                                (const int32_t*)counts.data_ptr(), as_int(B), as_int(path.size(1)), (int32_t*)out->data_ptr(), status, s));
        return made.defined() ? THPVariable_Wrap(made) : keep(a[6]);
    });
}

// fork_pages(kv_cache, block_table, page_counts, seq_lens, refs, parents, room, kv_dtype, out | None, workspace | None,
//            dev_status | None, stream | None) -> (table, page_counts, seq_lens, refs)
PyObject* fork_pages(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded([&]() -> PyObject* {
        wants(12, na);
        const at::Tensor &cache = tensor("kv_cache", a[0]), &table = tensor("block_table", a[1]),
                         &counts = tensor("page_counts", a[2]), &lens = tensor("seq_lens", a[3]), &refs = tensor("refs", a[4]),
                         &parents = tensor("parents", a[5]), &room = tensor("room", a[6]);
        const at::Tensor *ws = maybe("workspace", a[9]), *st = maybe("dev_status", a[10]);
        const int kv = number(a[7]);
        has_dims("block_table", table, at::kInt, 2);
        const int64_t B = table.size(0), width = table.size(1);
        is_shape("page_counts", counts, at::kInt, {B});
        is_shape("seq_lens", lens, at::kInt, {B});
        const auto [layers, nb] = layer_blocks(cache, kv);
        is_shape("refs", refs, at::kInt, {nb});
        has_dims("parents", parents, at::kInt, 1);
        const int64_t B2 = parents.size(0);
        is_shape("room", room, at::kInt, {B2});
        at::Tensor made[4], made_ws;
        const at::Tensor* out[4];
        if (a[8] == Py_None) {
            made[0] = make({B2, width}, at::kInt, refs);
            for (int i = 1; i < 4; ++i) made[i] = make({i < 3 ? B2 : nb}, at::kInt, refs);
            for (int i = 0; i < 4; ++i) out[i] = &made[i];
        } else {
            if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 4)
                refuse(PyExc_TypeError, "out must be a tuple (table, page_counts, seq_lens, refs)");
            for (int i = 0; i < 4; ++i) out[i] = &tensor("out", PyTuple_GET_ITEM(a[8], i));
        }
        is_shape("out[0]", *out[0], at::kInt, {B2, width});
        is_shape("out[1]", *out[1], at::kInt, {B2});
        is_shape("out[2]", *out[2], at::kInt, {B2});
        is_shape("out[3]", *out[3], at::kInt, {nb});
        if (ws && !ws->is_contiguous()) wrong("workspace", *ws, "contiguous");
        int32_t* status = status_word(st);
        const mla_stream_t s = stream_for(a[11], refs, {&cache, &table, &counts, &lens, &parents, &room, out[0], out[1], out[2],
                                                        out[3], ws, st});
        if (!ws) {
            made_ws = make({(int64_t)mla_fork_pages_workspace_bytes(as_int(B), as_int(B2), nb)}, at::kByte, refs);
            ws = &made_ws;
        }
        auto p = [](const at::Tensor& t) { return (int32_t*)t.data_ptr(); };
        check(mla_fork_pages(cache.data_ptr(), (mla_kv_dtype)kv, layers, nb, p(table), as_int(width), p(counts), p(lens), p(refs), as_int(B),
                             p(parents), p(room), as_int(B2), p(*out[0]), p(*out[1]), p(*out[2]), p(*out[3]), ws->data_ptr(),
                             ws->nbytes(), status, s));
        if (a[8] != Py_None) return keep(a[8]);
        return Py_BuildValue("(NNNN)", THPVariable_Wrap(made[0]), THPVariable_Wrap(made[1]), THPVariable_Wrap(made[2]),
                             THPVariable_Wrap(made[3]));
    });
}

// set_error(MlaError): the exception of a call that the library refuses
PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XDECREF(g_error);
    g_error = type;
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(rope), FAST(rope_cache_write), FAST(decode_tree), FAST(accept_tokens), FAST(fork_pages),
                           {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_mla_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mla_torch(void) { return PyModule_Create(&g_module); }
