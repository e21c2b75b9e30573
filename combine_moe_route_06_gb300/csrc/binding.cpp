// binding.cpp -- Python entry points of the training, expert and norm calls.
//
// They check torch tensors and call the C ABI on the current stream, like the
// ctypes functions of the package, but read a tensor's type, sizes and address
// through its C++ object: a call with one launch takes 2 to 3 us of host time
// instead of 7 to 10, which small batches would wait for.  Each function
// returns the library's status code; arguments that do not fit raise TypeError
// or ValueError, and nothing is enqueued then.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "../../include/moe_route.h"

namespace {

// Thrown with the Python error set.
struct Refused {};

[[noreturn]] void refuse(PyObject *type, const std::string &text)
{
    PyErr_SetString(type, text.c_str());
    throw Refused{};
}

enum Types { kF32 = 1, kBf16 = 2, kI32 = 4, kU8 = 8, kRow = 16 };   // kRow: bf16 or its bits

bool fits(at::ScalarType t, int types)
{
    switch (t) {
    case at::kFloat: return types & kF32;
    case at::kBFloat16: return types & (kBf16 | kRow);
    case at::kInt: return types & kI32;
    case at::kByte: return types & kU8;
    case at::kShort:
    case at::kUInt16: return types & kRow;
    default: return false;
    }
}

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); i++) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name, int types)
{
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + ": expected a torch.Tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + ": must be a CUDA tensor");
    if (!fits(t.scalar_type(), types))
        refuse(PyExc_TypeError, std::string(name) + ": dtype " + toString(t.scalar_type()) + " is not taken");
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + ": must be contiguous");
    return t;
}

const at::Tensor &shaped(PyObject *o, const char *name, int types, at::IntArrayRef shape)
{
    const at::Tensor &t = tensor(o, name, types);
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, std::string(name) + ": expected shape " + shape_text(shape) +
                                     ", got " + shape_text(t.sizes()));
    return t;
}

const at::Tensor &ranked(PyObject *o, const char *name, int types, int64_t dims)
{
    const at::Tensor &t = tensor(o, name, types);
    if (t.dim() != dims)
        refuse(PyExc_ValueError, std::string(name) + ": expected " + std::to_string(dims) +
                                     " dims, got shape " + shape_text(t.sizes()));
    return t;
}

template <typename T>
T *data(const at::Tensor &t)
{
    return (T *)t.const_data_ptr();
}
template <typename T>
T *at_shape(PyObject *o, const char *name, int types, at::IntArrayRef shape)
{
    return data<T>(shaped(o, name, types, shape));
}
template <typename T>
T *optional(PyObject *o, const char *name, int types, at::IntArrayRef shape)
{
    return o == Py_None ? nullptr : at_shape<T>(o, name, types, shape);
}
uint32_t *status_word(PyObject *o)
{
    return o == Py_None ? nullptr : data<uint32_t>(tensor(o, "dev_status", kI32));
}

int size32(int64_t n, const char *name)
{
    if (n > 0x7fffffff) refuse(PyExc_ValueError, std::string(name) + ": too large");
    return (int)n;
}

int int32(PyObject *o, const char *name)
{
    int past = 0;
    const long n = PyLong_AsLongAndOverflow(o, &past);
    if (n == -1 && PyErr_Occurred()) throw Refused{};
    if (past || n != (int)n) refuse(PyExc_ValueError, std::string(name) + ": does not fit 32 bits");
    return (int)n;
}

bool truth(PyObject *o)
{
    const int is = PyObject_IsTrue(o);
    if (is < 0) throw Refused{};
    return is;
}

cudaStream_t stream_of(PyObject *o)
{
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject *handle = PyObject_GetAttrString(o, "cuda_stream");
    if (!handle) throw Refused{};
    void *p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!p && PyErr_Occurred()) throw Refused{};
    return (cudaStream_t)p;
}

int logits_type(const at::Tensor &t) { return t.scalar_type() == at::kFloat ? MOE_TYPE_F32 : MOE_TYPE_BF16; }

using Args = PyObject *const *;

// Calls the library with the interpreter given up, as ctypes does: a launch waits when the
// device's queue is full, perhaps behind a host function that needs the interpreter.  The
// arguments are all evaluated before; the caller's references keep the tensors.
template <typename... P, typename... A>
moe_status_t enqueue(moe_status_t (*call)(P...), A... args)
{
    PyThreadState *state = PyEval_SaveThread();
    const moe_status_t status = call(args...);
    PyEval_RestoreThread(state);
    return status;
}

moe_status_t balance_loss(Args a)
{
    enum { logits, ids, counts, prob, lse, n_valid, losses, ws, mask, status, stream };
    const at::Tensor &l = ranked(a[logits], "logits", kF32 | kBf16, 3);
    const at::Tensor &i = ranked(a[ids], "topk_ids", kI32, 3);
    const int64_t S = l.size(0), T = l.size(1), E = l.size(2), k = i.size(2);
    shaped(a[ids], "topk_ids", kI32, {S, T, k});
    const at::Tensor &w = tensor(a[ws], "ws", kU8);
    return enqueue(
        moe_balance_loss, data<void>(l), logits_type(l), size32(S, "S"), size32(T, "T"), size32(E, "E"),
        size32(k, "k"), data<int32_t>(i), optional<uint8_t>(a[mask], "token_mask", kU8, {S, T}),
        at_shape<int32_t>(a[counts], "counts", kI32, {S, E}),
        at_shape<float>(a[prob], "prob_mean", kF32, {S, E}), at_shape<float>(a[lse], "lse", kF32, {S, T}),
        at_shape<int32_t>(a[n_valid], "n_valid", kI32, {S}), at_shape<float>(a[losses], "losses", kF32, {2}),
        data<void>(w), (size_t)w.numel(), status_word(a[status]), stream_of(a[stream]));
}

moe_status_t route_backward(Args a)
{
    enum { logits, ids, tw, dw, lse, counts, n_valid, d_losses, d_logits, mask, status, stream };
    if (a[ids] == Py_None) {
        if (a[tw] != Py_None) refuse(PyExc_ValueError, "topk_ids: needed with topk_w");
        if (a[d_losses] != Py_None)
            refuse(PyExc_ValueError, "topk_ids: needed with d_losses (k enters the balance loss)");
    }
    const at::Tensor &d = ranked(a[d_logits], "d_logits", kF32 | kBf16, 3);
    const int64_t S = d.size(0), T = d.size(1), E = d.size(2);
    const int64_t k = a[ids] == Py_None ? 1 : ranked(a[ids], "topk_ids", kI32, 3).size(2);
    const bool loss = a[d_losses] != Py_None;
    if (loss && a[logits] == Py_None) refuse(PyExc_ValueError, "logits: needed with d_losses");
    const int like = d.scalar_type() == at::kFloat ? kF32 : kBf16;
    return enqueue(
        moe_route_backward,
        loss ? at_shape<void>(a[logits], "logits", like, {S, T, E}) : nullptr, logits_type(d),
        size32(S, "S"), size32(T, "T"), size32(E, "E"), size32(k, "k"),
        optional<int32_t>(a[ids], "topk_ids", kI32, {S, T, k}),
        optional<float>(a[tw], "topk_w", kF32, {S, T, k}), optional<float>(a[dw], "d_topk_w", kF32, {S, T, k}),
        loss ? optional<float>(a[lse], "lse", kF32, {S, T}) : nullptr,
        loss ? optional<int32_t>(a[counts], "counts", kI32, {S, E}) : nullptr,
        loss ? optional<int32_t>(a[n_valid], "n_valid", kI32, {S}) : nullptr,
        optional<float>(a[d_losses], "d_losses", kF32, {2}),
        optional<uint8_t>(a[mask], "token_mask", kU8, {S, T}), data<void>(d), status_word(a[status]),
        stream_of(a[stream]));
}

moe_status_t combine_backward(Args a)
{
    enum { d_out, y, pair_row, w, d_y, dw, recv_pair, status, stream };
    const at::Tensor &g = ranked(a[d_out], "d_out", kRow, 3);
    const at::Tensor &r = ranked(a[y], "y", kRow, 2);
    const int64_t S = g.size(0), T = g.size(1), H = g.size(2), rows = r.size(0);
    const int64_t k = ranked(a[pair_row], "pair_row", kI32, 3).size(2);
    shaped(a[y], "y", kRow, {rows, H});
    return enqueue(
        moe_combine_backward, data<uint16_t>(g), data<uint16_t>(r), size32(rows, "y_rows"),
        at_shape<int32_t>(a[pair_row], "pair_row", kI32, {S, T, k}),
        at_shape<float>(a[w], "topk_w", kF32, {S, T, k}),
        optional<int32_t>(a[recv_pair], "recv_pair", kI32, {rows}), size32(S, "S"), size32(T, "T"),
        size32(k, "k"), size32(H, "H"), at_shape<uint16_t>(a[d_y], "d_y", kRow, {rows, H}),
        at_shape<float>(a[dw], "d_topk_w", kF32, {S, T, k}), status_word(a[status]),
        stream_of(a[stream]));
}

moe_status_t w4_pack(Args a)
{
    enum { codes, scales, w4, gated, stream };
    const at::Tensor &c = ranked(a[codes], "codes", kU8, 3);
    const int64_t E = c.size(0), rows = c.size(1), K = 2 * c.size(2);
    const bool two = truth(a[gated]);
    if (two && rows % 2)
        refuse(PyExc_ValueError, "codes: gated weights have an even number of rows, got " +
                                     std::to_string(rows));
    const at::Tensor &p = tensor(a[w4], "w4", kU8);
    return enqueue(moe_w4_pack, data<uint8_t>(c),
                   at_shape<uint8_t>(a[scales], "scales", kU8, {E, rows, K / 16}), size32(E, "E"),
                   size32(two ? rows / 2 : rows, "N"), size32(K, "K"), two, data<uint8_t>(p),
                   (size_t)p.numel(), stream_of(a[stream]));
}

moe_status_t expert_product_w4(Args a)
{
    enum { x, w4, factor, y, ws, offsets, counts, block_rows, gated, status, stream };
    const at::Tensor &r = ranked(a[x], "a", kRow, 2);
    const at::Tensor &out = ranked(a[y], "y", kRow, 2);
    const int64_t rows = r.size(0), K = r.size(1), N = out.size(1);
    const at::Tensor &f = ranked(a[factor], "w_factor", kF32, 1);
    const int64_t E = f.size(0);
    const at::Tensor &p = tensor(a[w4], "w4", kU8);
    const at::Tensor &w = tensor(a[ws], "ws", kU8);
    const int block = int32(a[block_rows], "block_rows");
    const int two = truth(a[gated]);
    // sizes that the library refuses have no packed size; it says why
    const size_t need = moe_w4_bytes(size32(E, "E"), size32(N, "N"), size32(K, "K"), two);
    if ((size_t)p.numel() < need)
        refuse(PyExc_ValueError, "w4: " + std::to_string(p.numel()) + " bytes are not the packed weights of E=" +
                                     std::to_string(E) + ", N=" + std::to_string(N) + ", K=" +
                                     std::to_string(K) + ", gated=" + std::to_string(two));
    return enqueue(
        moe_expert_product_w4, data<uint16_t>(r), size32(rows, "a_rows"),
        optional<int32_t>(a[offsets], "expert_offsets", kI32, {E + 1}),
        optional<int32_t>(a[counts], "masked_counts", kI32, {E}), block, data<uint8_t>(p),
        data<float>(f), (int)E, (int)N, (int)K, two, at_shape<uint16_t>(a[y], "y", kRow, {rows, N}),
        data<void>(w), (size_t)w.numel(), status_word(a[status]), stream_of(a[stream]));
}

// The calls below also see to it that all tensors are on the current device.
void here(const at::Tensor &t, const char *name, const at::Tensor &first)
{
    if (t.device() != first.device())
        refuse(PyExc_ValueError, std::string(name) + ": is on another device than the other tensors");
}
template <typename T>
T *here_shaped(PyObject *o, const char *name, int types, at::IntArrayRef shape, const at::Tensor &first)
{
    if (o == Py_None) return nullptr;
    const at::Tensor &t = shaped(o, name, types, shape);
    here(t, name, first);
    return data<T>(t);
}
void current(const at::Tensor &first, const char *name)
{
    if (first.device().index() != c10::cuda::current_device())
        refuse(PyExc_ValueError, std::string(name) + ": is not on the current device");
}

struct ProductShape {
    int rows, E, N, K;
    const int32_t *offsets, *counts;
    int block_rows;
    void *ws;
    size_t ws_bytes;
};

// What both products have: the sizes by the rows' and the weights' shapes, the experts'
// rows and the workspace.
ProductShape product_shape(const at::Tensor &w, int64_t rows, PyObject *offsets, PyObject *counts,
                           PyObject *block_rows, PyObject *ws)
{
    current(w, "w");
    const at::Tensor &s = tensor(ws, "ws", kU8);
    here(s, "ws", w);
    const int64_t E = w.size(0);
    return {size32(rows, "a_rows"), size32(E, "E"), size32(w.size(1), "N"), size32(w.size(2), "K"),
            here_shaped<int32_t>(offsets, "expert_offsets", kI32, {E + 1}, w),
            here_shaped<int32_t>(counts, "masked_counts", kI32, {E}, w), int32(block_rows, "block_rows"),
            data<void>(s), (size_t)s.numel()};
}

moe_status_t expert_product(Args a)
{
    enum { x, w, y, ws, offsets, counts, block_rows, gated, pre, status, stream };
    const at::Tensor &t = ranked(a[w], "w", kRow, 3);
    const int64_t rows = ranked(a[x], "a", kRow, 2).size(0);
    const bool two = truth(a[gated]);
    if (two && t.size(1) % 2)
        refuse(PyExc_ValueError, "w: gated weights have an even number of rows, got " +
                                     std::to_string(t.size(1)));
    const ProductShape p = product_shape(t, rows, a[offsets], a[counts], a[block_rows], a[ws]);
    const int N = two ? p.N / 2 : p.N;
    uint16_t *const out = here_shaped<uint16_t>(a[y], "y", kRow, {rows, N}, t);
    if (a[y] == Py_None) refuse(PyExc_TypeError, "y: expected a torch.Tensor");
    return enqueue(moe_expert_product, here_shaped<uint16_t>(a[x], "a", kRow, {rows, p.K}, t), p.rows,
                   p.offsets, p.counts, p.block_rows, data<uint16_t>(t), p.E, N, p.K, (int)two, out,
                   here_shaped<uint16_t>(a[pre], "pre", kRow, {rows, 2 * (int64_t)N}, t), p.ws, p.ws_bytes,
                   status_word(a[status]), stream_of(a[stream]));
}

moe_status_t expert_product_backward(Args a)
{
    enum { d_y, x, w, ws, d_a, d_w, offsets, counts, block_rows, pre, status, stream };
    const at::Tensor &t = ranked(a[w], "w", kRow, 3);
    const int64_t rows = ranked(a[d_y], "d_y", kRow, 2).size(0);
    const ProductShape p = product_shape(t, rows, a[offsets], a[counts], a[block_rows], a[ws]);
    const bool gate = a[pre] != Py_None;
    if (a[d_w] != Py_None && a[x] == Py_None) refuse(PyExc_ValueError, "a: needed with d_w");
    if (gate && a[d_a] == Py_None) refuse(PyExc_ValueError, "d_a: needed with pre");
    if (a[d_a] == Py_None && a[d_w] == Py_None)
        refuse(PyExc_ValueError, "d_a, d_w: neither is wanted");
    void *const weights = here_shaped<void>(a[d_w], "d_w", kF32 | kBf16, t.sizes(), t);
    const int type = weights && THPVariable_Unpack(a[d_w]).scalar_type() == at::kFloat ? MOE_TYPE_F32 : MOE_TYPE_BF16;
    return enqueue(moe_expert_product_backward, here_shaped<uint16_t>(a[d_y], "d_y", kRow, {rows, p.N}, t),
                   here_shaped<uint16_t>(a[x], "a", kRow, {rows, p.K}, t), p.rows, p.offsets, p.counts,
                   p.block_rows, data<uint16_t>(t),
                   here_shaped<uint16_t>(a[pre], "pre", kRow, {rows, 2 * (int64_t)p.K}, t), p.E, p.N, p.K,
                   here_shaped<uint16_t>(a[d_a], "d_a", kRow, {rows, (gate ? 2 : 1) * (int64_t)p.K}, t),
                   weights, type, p.ws, p.ws_bytes, status_word(a[status]), stream_of(a[stream]));
}

int norm_type(const at::Tensor &t) { return t.scalar_type() == at::kFloat ? MOE_TYPE_F32 : MOE_TYPE_BF16; }

float positive(PyObject *o, const char *name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    if (!(v > 0)) refuse(PyExc_ValueError, std::string(name) + ": must be positive");
    return (float)v;
}

// Rows [..., H] of a norm: any leading sizes, the same for all of its tensors.
int64_t row_count(const at::Tensor &t, const char *name)
{
    if (t.dim() < 1 || t.size(-1) == 0)
        refuse(PyExc_ValueError, std::string(name) + ": expected rows, got shape " + shape_text(t.sizes()));
    return t.numel() / t.size(-1);
}

moe_status_t rms_norm(Args a)
{
    enum { x, weight, y, record, residual, residual_out, eps, stream };
    const at::Tensor &t = tensor(a[x], "x", kRow);
    const int64_t rows = row_count(t, "x"), H = t.size(-1);
    current(t, "x");
    const at::Tensor &w = shaped(a[weight], "weight", kF32 | kBf16, {H});
    here(w, "weight", t);
    const bool add = a[residual] != Py_None;
    const int kind = add && tensor(a[residual], "residual", kF32 | kBf16).scalar_type() == at::kFloat ? kF32 : kBf16;
    if (!add && a[residual_out] != Py_None) refuse(PyExc_ValueError, "residual_out: without a residual");
    if (a[y] == Py_None && a[record] == Py_None) refuse(PyExc_ValueError, "y, record: neither is wanted");
    uint8_t *bytes = nullptr;
    if (a[record] != Py_None) {
        const at::Tensor &r = tensor(a[record], "record", kU8);
        here(r, "record", t);
        if (r.dim() < 1 || r.size(-1) != H + H / 32 || r.numel() != rows * (H + H / 32))
            refuse(PyExc_ValueError, "record: expected " + std::to_string(rows) + " rows of " +
                                         std::to_string(H + H / 32) + " bytes, got shape " +
                                         shape_text(r.sizes()));
        bytes = data<uint8_t>(r);
    }
    return enqueue(moe_rms_norm, data<uint16_t>(t), here_shaped<void>(a[residual], "residual", kind, t.sizes(), t),
                   kind == kF32 ? MOE_TYPE_F32 : MOE_TYPE_BF16, data<void>(w), norm_type(w), rows,
                   size32(H, "H"), positive(a[eps], "eps"),
                   here_shaped<void>(a[residual_out], "residual_out", kind, t.sizes(), t),
                   here_shaped<uint16_t>(a[y], "y", kRow, t.sizes(), t), bytes, stream_of(a[stream]));
}

moe_status_t rms_norm_backward(Args a)
{
    enum { d_y, h, weight, d_h, ws, d_weight, d_residual, d_x, eps, stream };
    const at::Tensor &t = tensor(a[d_y], "d_y", kRow);
    const int64_t rows = row_count(t, "d_y"), H = t.size(-1);
    current(t, "d_y");
    const at::Tensor &w = shaped(a[weight], "weight", kF32 | kBf16, {H});
    here(w, "weight", t);
    const at::Tensor &r = shaped(a[h], "h", kF32 | kBf16, t.sizes());
    here(r, "h", t);
    const int kind = r.scalar_type() == at::kFloat ? kF32 : kBf16;
    if (a[d_h] == Py_None) refuse(PyExc_TypeError, "d_h: expected a torch.Tensor");
    void *scratch = nullptr;
    size_t bytes = 0;
    if (a[d_weight] != Py_None) {
        const at::Tensor &s = tensor(a[ws], "ws", kU8);
        here(s, "ws", t);
        scratch = data<void>(s);
        bytes = (size_t)s.numel();
    }
    return enqueue(moe_rms_norm_backward, data<uint16_t>(t), data<void>(r), norm_type(r), data<void>(w),
                   norm_type(w), here_shaped<void>(a[d_residual], "d_residual", kind, t.sizes(), t), rows,
                   size32(H, "H"), positive(a[eps], "eps"),
                   here_shaped<void>(a[d_h], "d_h", kind, t.sizes(), t),
                   here_shaped<uint16_t>(a[d_x], "d_x", kRow, t.sizes(), t),
                   here_shaped<float>(a[d_weight], "d_weight", kF32, {H}, t), scratch, bytes,
                   stream_of(a[stream]));
}

template <moe_status_t (*CALL)(Args), int COUNT>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != COUNT) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", COUNT, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(CALL(args));
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <moe_status_t (*CALL)(Args), int COUNT>
PyMethodDef method(const char *name)
{
    return {name, (PyCFunction)(void (*)(void))entry<CALL, COUNT>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<balance_loss, 11>("balance_loss"),
    method<route_backward, 12>("route_backward"),
    method<combine_backward, 9>("combine_backward"),
    method<w4_pack, 5>("w4_pack"),
    method<expert_product_w4, 11>("expert_product_w4"),
    method<expert_product, 11>("expert_product"),
    method<expert_product_backward, 12>("expert_product_backward"),
    method<rms_norm, 8>("rms_norm"),
    method<rms_norm_backward, 10>("rms_norm_backward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_ops", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_ops() { return PyModule_Create(&module); }
