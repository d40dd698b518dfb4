// bind_latent.cpp -- the latent calls from Python: checks of the tensors, their
// outputs and scratch, and the call, as one extension function each.
//
// A decode step's call is a few microseconds of GPU time; attribute look-ups,
// three allocations and 24 converted arguments in Python took 16 to 22 us of
// host time on a Grace core (here 7 to 8).  The functions come as addresses of the loaded
// library (bind), so there is one copy of it in the process.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>
#include <optional>
#include <string>

#include "idx.h"

namespace {

constexpr int64_t kLatent = 512, kRope = 64, kNope = 128, kV = 128;

decltype(&idx_latent_store) f_store;
decltype(&idx_latent_gather) f_gather;
decltype(&idx_latent_attention) f_attention;
decltype(&idx_paged_latent_attention) f_paged;
decltype(&idx_latent_prefill) f_prefill;
decltype(&idx_latent_attention_workspace_size) f_attention_size;
decltype(&idx_latent_prefill_workspace_size) f_prefill_size;
decltype(&idx_latent_attention_launches) f_attention_launches;
PyObject *g_check;  // check(status, name) raises

struct Refusal {
    std::string text;
};

[[noreturn]] void refuse(std::string text)
{
    throw Refusal{std::move(text)};
}

const at::Tensor &tensor_of(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int int_of(PyObject *o, const char *name)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    if (v < INT_MIN || v > INT_MAX)
        refuse(std::string(name) + " is out of range");
    return (int)v;
}

float float_of(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return (float)v;
}

bool truth_of(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw python_error();
    return v != 0;
}

// Every tensor of a call lives on one device, and it is the current one: the
// stream, the scratch's size and the launch are the current device's.
void on_one_device(std::initializer_list<const at::Tensor *> tensors)
{
    const at::Tensor &first = **tensors.begin();
    for (const at::Tensor *t : tensors) {
        if (!t->defined())
            continue;
        if (!t->is_cuda())
            refuse("indexer tensors must live on a CUDA device");
        if (t->device() != first.device())
            refuse("tensors of one call are on " + first.device().str() + " and " +
                   t->device().str());
    }
    const int current = c10::cuda::current_device();
    if (first.device().index() != current)
        refuse("tensors on " + first.device().str() + ", but the current device is cuda:" +
               std::to_string(current));
}

template <typename T>
T *address(const at::Tensor &t)
{
    return static_cast<T *>(t.data_ptr());
}

// bf16, `dims` dimensions, the last one of `dim` contiguous elements.
const at::Tensor &need_heads(PyObject *o, int64_t dims, int64_t dim, const char *name)
{
    const at::Tensor &t = tensor_of(o, name);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != dims || t.size(-1) != dim ||
        t.stride(-1) != 1)
        refuse(std::string(name) + " must be bfloat16 [..., " + std::to_string(dim) + "] of " +
               std::to_string(dims) + " dimensions with unit last stride");
    return t;
}

const at::Tensor &need(PyObject *o, at::ScalarType type, const char *name)
{
    const at::Tensor &t = tensor_of(o, name);
    if (t.scalar_type() != type)
        refuse(std::string(name) + " must be " + c10::toString(type) + ", got " +
               c10::toString(t.scalar_type()));
    if (!t.is_contiguous())
        refuse(std::string(name) + " must be contiguous");
    return t;
}

void need_count(const at::Tensor &t, int64_t n, const char *name)
{
    if (t.numel() != n)
        refuse(std::string(name) + " must hold " + std::to_string(n) + " entries");
}

const at::Tensor &need_pages(PyObject *o)
{
    const at::Tensor &t = tensor_of(o, "kv_pages");
    if (t.scalar_type() != at::kByte || t.dim() != 2 || t.stride(1) != 1)
        refuse("kv_pages must be uint8 [num_pages, page_stride] with unit byte stride");
    return t;
}

// The stride of dimension d in elements; over one element any stride will do,
// and a tensor may have one without meaning there.
int64_t ld(const at::Tensor &t, int64_t d, int64_t natural)
{
    return t.size(d) > 1 ? t.stride(d) : natural;
}

int64_t page_stride(const at::Tensor &pages)
{
    return ld(pages, 0, (pages.size(1) + 15) / 16 * 16);
}

// What a launch counts in 32 bits.
int count(int64_t n, const char *name)
{
    if (n > INT_MAX)
        refuse(std::string(name) + " is out of range");
    return (int)n;
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device device)
{
    return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

// The outputs of an attention call, made here unless given (lse False: none),
// and its scratch (True: made here; or None, or a tensor).
struct Outputs {
    at::Tensor out, lse, ws;
    int64_t ld_row, ld_head, ld_lse = 0;
    size_t ws_bytes = 0;

    Outputs(PyObject *out_o, PyObject *lse_o, PyObject *ws_o, const at::Tensor &q, int64_t dim)
    {
        const int64_t R = q.size(0), H = q.size(1);
        if (out_o != Py_None) {
            out = need_heads(out_o, 3, dim, "out");
            if (out.size(0) != R || out.size(1) != H)
                refuse("out must be [" + std::to_string(R) + ", " + std::to_string(H) + ", " +
                       std::to_string(dim) + "]");
        }
        if (lse_o != Py_None && lse_o != Py_False) {
            lse = tensor_of(lse_o, "lse");
            if (lse.scalar_type() != at::kFloat || lse.dim() != 2 || lse.size(0) != R ||
                lse.size(1) != H || ld(lse, 1, 1) != 1)
                refuse("lse must be float32 [" + std::to_string(R) + ", " + std::to_string(H) +
                       "] with unit column stride");
        }
        if (ws_o != Py_True && ws_o != Py_None) {
            ws = tensor_of(ws_o, "workspace");
            if (!ws.is_contiguous())  // its bytes are counted, and have to be there
                refuse("workspace must be contiguous");
            ws_bytes = ws.numel() * ws.element_size();
        }
    }
    // The ones that were not given, once the device is known to be good.
    void make(PyObject *lse_o, PyObject *ws_o, const at::Tensor &q, int64_t dim, size_t size)
    {
        const int64_t R = q.size(0), H = q.size(1);
        if (!out.defined())
            out = empty({R, H, dim}, at::kBFloat16, q.device());
        if (lse_o == Py_None)
            lse = empty({R, H}, at::kFloat, q.device());
        if (ws_o == Py_True && size > 0) {
            ws = empty({(int64_t)size}, at::kByte, q.device());
            ws_bytes = size;
        }
        ld_row = ld(out, 0, H * dim);
        ld_head = ld(out, 1, dim);
        if (lse.defined())
            ld_lse = ld(lse, 0, H);
    }
    uint16_t *out_at() const { return address<uint16_t>(out); }
    float *lse_at() const { return lse.defined() ? address<float>(lse) : nullptr; }
    void *ws_at() const { return ws.defined() ? address<void>(ws) : nullptr; }
};

PyObject *wrap(const at::Tensor &t)
{
    if (t.defined())
        return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

PyObject *wrap(const void *p)
{
    if (p)
        return PyLong_FromVoidPtr(const_cast<void *>(p));
    Py_RETURN_NONE;
}

PyObject *keep(PyObject *o)
{
    Py_INCREF(o);
    return o;
}

// The launch on the current stream; raises by the status.
template <typename F, typename... A>
void launch(F f, const char *name, A... args)
{
    void *stream = c10::cuda::getCurrentCUDAStream().stream();
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = (int)f(args..., static_cast<idx_stream_t>(stream));
    Py_END_ALLOW_THREADS
    if (status != 0) {
        PyObject *r = PyObject_CallFunction(g_check, "is", status, name);
        Py_XDECREF(r);
        throw python_error();
    }
}

// Arguments as the library's function takes them, for a call that is made
// again and again.
PyObject *item(const void *p) { return wrap(p); }
PyObject *item(int v) { return PyLong_FromLong(v); }
PyObject *item(int64_t v) { return PyLong_FromLongLong(v); }
PyObject *item(size_t v) { return PyLong_FromSize_t(v); }
PyObject *item(float v) { return PyFloat_FromDouble(v); }
PyObject *item(idx_latent_format v) { return PyLong_FromLong((long)v); }

template <typename... A>
PyObject *arguments(A... args)
{
    PyObject *t = PyTuple_New(sizeof...(A));
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(t, i++, item(args)), ...);
    return t;
}

// Launches (returns `result`), or with prepare returns (arguments, tensors to
// keep, launches of the call, device).
template <typename F, typename R, typename K, typename... A>
PyObject *call(bool prepare, F f, const char *name, int launches, R result, K kept, A... args)
{
    if (prepare)
        return Py_BuildValue("(NNii)", arguments(args...), kept(), launches,
                             (int)c10::cuda::current_device());
    launch(f, name, args...);
    return result();
}

PyObject *store(PyObject *, PyObject *const *a, Py_ssize_t)
{
    const at::Tensor &kv = need_heads(a[1], 2, kLatent + kRope, "kv");
    const int64_t T = kv.size(0);
    const at::Tensor &pages = need_pages(a[6]), &slots = need(a[8], at::kLong, "slot_mapping");
    need_count(slots, T, "slot_mapping");
    if ((a[2] == Py_None) != (a[3] == Py_None))
        refuse("positions and cos_sin come together");
    at::Tensor p, c, w;
    int rows = 0;
    int64_t ld_cs = 0;
    if (a[3] != Py_None) {
        p = need(a[2], at::kInt, "positions");
        c = tensor_of(a[3], "cos_sin");
        need_count(p, T, "positions");
        if (c.scalar_type() != at::kFloat || c.dim() != 2 || c.stride(1) != 1 || c.size(1) < kRope)
            refuse("cos_sin must be float32 [positions, " + std::to_string(kRope) + "]");
        rows = count(c.size(0), "cos_sin");
        ld_cs = ld(c, 0, kRope);
    }
    if (a[4] != Py_None) {
        w = need(a[4], at::kFloat, "norm_weight");
        need_count(w, kLatent, "norm_weight");
    }
    on_one_device({&kv, &pages, &slots, &p, &c, &w});
    const int32_t *positions = c.defined() ? address<int32_t>(p) : nullptr;
    const float *cos_sin = c.defined() ? address<float>(c) : nullptr;
    const float *weight = w.defined() ? address<float>(w) : nullptr;
    return call(
        a[0] == Py_True, f_store, "idx_latent_store", T > 0, [] { Py_RETURN_NONE; },
        [&] {
            return Py_BuildValue("(OOOOOO)", a[1], a[2], a[3], a[4], a[6], a[8]);
        },
        (const uint16_t *)address<uint16_t>(kv), ld(kv, 0, kLatent + kRope), positions, cos_sin,
        ld_cs, rows, weight,
        float_of(a[5]), count(T, "kv"), (int)kLatent, (int)kRope,
        (idx_latent_format)int_of(a[9], "fmt"), address<uint8_t>(pages), page_stride(pages),
        count(pages.size(0), "kv_pages"), int_of(a[7], "page_size"),
        (const int64_t *)address<int64_t>(slots));
}

PyObject *gather(PyObject *, PyObject *const *a, Py_ssize_t)
{
    const at::Tensor &pages = need_pages(a[1]);
    const at::Tensor &out = need_heads(a[6], 2, kLatent + kRope, "out");
    const at::Tensor &table = need(a[4], at::kInt, "block_table"), &cu = need(a[5], at::kInt, "cu_lens");
    const int64_t B = cu.numel() - 1;
    if (table.dim() != 2 || table.size(0) < B || B < 0)
        refuse("block_table must be [B, blocks] and cu_lens [B + 1]");
    at::Tensor s;
    if (a[7] != Py_None) {
        s = need(a[7], at::kInt, "seq_starts");
        need_count(s, B, "seq_starts");
    }
    on_one_device({&pages, &out, &table, &cu, &s});
    const int32_t *starts = s.defined() ? address<int32_t>(s) : nullptr;
    return call(
        a[0] == Py_True, f_gather, "idx_latent_gather", B > 0 && out.size(0) > 0,
        [&] { return keep(a[6]); },
        [&] {
            return Py_BuildValue("(OOOOO)", a[1], a[4], a[5], a[7], a[6]);
        },
        (const uint8_t *)address<uint8_t>(pages), page_stride(pages), count(pages.size(0), "kv_pages"),
        int_of(a[2], "page_size"), (idx_latent_format)int_of(a[3], "fmt"), (int)kLatent, (int)kRope,
        (const int32_t *)address<int32_t>(table), table.size(1),
        count(table.size(1), "block_table"), (const int32_t *)address<int32_t>(cu), starts,
        count(B, "cu_lens"), count(out.size(0), "out"), address<uint16_t>(out),
        ld(out, 0, kLatent + kRope));
}

PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t)
{
    const at::Tensor &q = need_heads(a[1], 3, kLatent + kRope, "q");
    const at::Tensor &pages = need_pages(a[2]);
    const at::Tensor &slots = need(a[5], at::kInt, "slots"), &indptr = need(a[6], at::kInt, "indptr");
    const int R = count(q.size(0), "q"), H = count(q.size(1), "q");
    need_count(indptr, (int64_t)R + 1, "indptr");
    Outputs o(a[8], a[9], a[10], q, kLatent);
    on_one_device({&q, &pages, &slots, &indptr, &o.out, &o.lse, &o.ws});
    const size_t size = f_attention_size(R, H, slots.numel());
    o.make(a[9], a[10], q, kLatent, size);
    return call(
        a[0] == Py_True, f_attention, "idx_latent_attention",
        f_attention_launches(R, 1, H, slots.numel()),
        [&] { return Py_BuildValue("(NN)", wrap(o.out), wrap(o.lse)); },
        [&] {
            return Py_BuildValue("(OOOONNN)", a[1], a[2], a[5], a[6], wrap(o.out), wrap(o.lse),
                                 wrap(o.ws));
        },
        (const uint16_t *)address<uint16_t>(q), ld(q, 0, H * (kLatent + kRope)),
        ld(q, 1, kLatent + kRope), (const uint8_t *)address<uint8_t>(pages), page_stride(pages),
        count(pages.size(0), "kv_pages"),
        int_of(a[3], "page_size"), (idx_latent_format)int_of(a[4], "fmt"),
        (const int32_t *)address<int32_t>(slots), (const int32_t *)address<int32_t>(indptr),
        slots.numel(), R, H, (int)kLatent, (int)kRope, float_of(a[7]), o.out_at(), o.ld_row,
        o.ld_head, o.lse_at(), o.ld_lse, o.ws_at(), o.ws_bytes);
}

PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t)
{
    const at::Tensor &q = need_heads(a[1], 3, kLatent + kRope, "q");
    const at::Tensor &pages = need_pages(a[2]);
    const at::Tensor &table = need(a[5], at::kInt, "block_table");
    const at::Tensor &lens = need(a[6], at::kInt, "context_lens");
    const int R = count(q.size(0), "q"), H = count(q.size(1), "q"), next = int_of(a[7], "next_n");
    if (next <= 0 || R % next)
        refuse("q must hold B * next_n rows");
    const int B = R / next, per_row = truth_of(a[10]);
    need_count(lens, per_row ? R : B, "context_lens");
    if (table.dim() != 2 || table.size(0) < B)
        refuse("block_table must be [" + std::to_string(B) + ", blocks]");
    const int longest = int_of(a[9], "max_model_len");
    Outputs o(a[11], a[12], a[13], q, kLatent);
    on_one_device({&q, &pages, &table, &lens, &o.out, &o.lse, &o.ws});
    const size_t size = f_attention_size(R, H, longest);
    o.make(a[12], a[13], q, kLatent, size);
    return call(
        a[0] == Py_True, f_paged, "idx_paged_latent_attention",
        f_attention_launches(R, next, H, longest),
        [&] { return Py_BuildValue("(NN)", wrap(o.out), wrap(o.lse)); },
        [&] {
            return Py_BuildValue("(OOOONNN)", a[1], a[2], a[5], a[6], wrap(o.out), wrap(o.lse),
                                 wrap(o.ws));
        },
        (const uint16_t *)address<uint16_t>(q), ld(q, 0, H * (kLatent + kRope)),
        ld(q, 1, kLatent + kRope), (const uint8_t *)address<uint8_t>(pages), page_stride(pages),
        count(pages.size(0), "kv_pages"),
        int_of(a[3], "page_size"), (idx_latent_format)int_of(a[4], "fmt"),
        (const int32_t *)address<int32_t>(table), table.size(1),
        (const int32_t *)address<int32_t>(lens), per_row, B, next, longest, H, (int)kLatent,
        (int)kRope, float_of(a[8]), o.out_at(), o.ld_row, o.ld_head, o.lse_at(), o.ld_lse,
        o.ws_at(), o.ws_bytes);
}

PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t)
{
    const at::Tensor &q = need_heads(a[1], 3, kNope + kRope, "q");
    const at::Tensor &k = need_heads(a[2], 3, kNope, "k");
    const at::Tensor &rope = need_heads(a[3], 2, kRope, "k_rope");
    const at::Tensor &v = need_heads(a[4], 3, kV, "v");
    const at::Tensor &cu_q = need(a[5], at::kInt, "cu_q"), &cu_k = need(a[6], at::kInt, "cu_k");
    const int Tq = count(q.size(0), "q"), H = count(q.size(1), "q"), Tk = count(k.size(0), "k");
    const int causal = truth_of(a[8]);
    if (k.size(1) != H || v.size(1) != H || v.size(0) != Tk || rope.size(0) != Tk)
        refuse("k, k_rope and v must hold the same tokens, and the heads of q");
    const int64_t B = cu_q.numel() - 1;
    if (cu_k.numel() != B + 1 || B < 0)
        refuse("cu_q and cu_k must both hold B + 1 entries");
    Outputs o(a[9], a[10], a[11], q, kV);
    on_one_device({&q, &k, &rope, &v, &cu_q, &cu_k, &o.out, &o.lse, &o.ws});
    const size_t size = f_prefill_size(Tq, Tk, H);
    o.make(a[10], a[11], q, kV, size);
    return call(
        a[0] == Py_True, f_prefill, "idx_latent_prefill", Tq == 0 || B == 0 ? 0 : size ? 2 : 1,
        [&] { return Py_BuildValue("(NN)", wrap(o.out), wrap(o.lse)); },
        [&] {
            return Py_BuildValue("(OOOOOONNN)", a[1], a[2], a[3], a[4], a[5], a[6], wrap(o.out),
                                 wrap(o.lse), wrap(o.ws));
        },
        (const uint16_t *)address<uint16_t>(q), ld(q, 0, H * (kNope + kRope)), ld(q, 1, kNope + kRope),
        (const uint16_t *)address<uint16_t>(k), ld(k, 0, H * kNope), ld(k, 1, kNope),
        (const uint16_t *)address<uint16_t>(rope), ld(rope, 0, kRope),
        (const uint16_t *)address<uint16_t>(v), ld(v, 0, H * kV), ld(v, 1, kV),
        (const int32_t *)address<int32_t>(cu_q), (const int32_t *)address<int32_t>(cu_k),
        count(B, "cu_q"), Tq, Tk, H, (int)kNope, (int)kRope, (int)kV, float_of(a[7]),
        causal, o.out_at(), o.ld_row, o.ld_head, o.lse_at(), o.ld_lse, o.ws_at(),
        o.ws_bytes);
}

// Errors as Python's: refusals are ValueErrors.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t), int N>
PyObject *entry(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(self, a, n);
    } catch (const Refusal &r) {
        PyErr_SetString(PyExc_ValueError, r.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// bind(check, addresses of the library's functions)
PyObject *bind(PyObject *, PyObject *args)
{
    unsigned long long p[8];
    PyObject *check;
    if (!PyArg_ParseTuple(args, "OKKKKKKKK", &check, p, p + 1, p + 2, p + 3, p + 4, p + 5, p + 6,
                          p + 7))
        return nullptr;
    f_store = reinterpret_cast<decltype(f_store)>(p[0]);
    f_gather = reinterpret_cast<decltype(f_gather)>(p[1]);
    f_attention = reinterpret_cast<decltype(f_attention)>(p[2]);
    f_paged = reinterpret_cast<decltype(f_paged)>(p[3]);
    f_prefill = reinterpret_cast<decltype(f_prefill)>(p[4]);
    f_attention_size = reinterpret_cast<decltype(f_attention_size)>(p[5]);
    f_prefill_size = reinterpret_cast<decltype(f_prefill_size)>(p[6]);
    f_attention_launches = reinterpret_cast<decltype(f_attention_launches)>(p[7]);
    Py_INCREF(check);
    Py_XSETREF(g_check, check);
    Py_RETURN_NONE;
}

#define IDX_ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(entry<f, n>), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    IDX_ENTRY(store, 10),
    IDX_ENTRY(gather, 8),
    IDX_ENTRY(attention, 11),
    IDX_ENTRY(paged_attention, 14),
    IDX_ENTRY(prefill, 12),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_latent_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__latent_calls()
{
    return PyModule_Create(&module);
}
