// twell_call.cpp -- the calls a decode step makes many of, from Python without ctypes: a module (_twell_call) that checks
// the tensors of one call, takes their pointers and the stream, and calls the C ABI of twell.h. The kernels of
// such a step take a few microseconds, and so does a ctypes call with its checks in Python; here the checks cost
// nanoseconds. Nothing is computed here.
//
// Each function takes its arguments by position (None where there is none) and returns the twell_status; a tensor of
// another shape, type, layout or device raises ValueError, a type the library has no code for TypeError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAException.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <map>
#include <mutex>
#include <tuple>

#include "twell.h"

namespace {

using Shape = std::initializer_list<int64_t>;

constexpr int32_t kLoraMaxTokens = 1 << 20, kLoraMaxRank = 128;  // of one twell_lora_add

std::string text(const at::Tensor& t)
{
    std::ostringstream s;
    s << t.scalar_type() << ' ' << t.sizes() << " with strides " << t.strides() << " on " << t.device();
    return s.str();
}

// The tensor in `o`, null for None where `optional`.
const at::Tensor* tensor(PyObject* o, const char* what, bool optional = false)
{
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) C10_THROW_ERROR(TypeError, std::string(what) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

int device_of(const at::Tensor& t, const char* what)
{
    if (!t.is_cuda()) C10_THROW_ERROR(ValueError, std::string(what) + " is on " + t.device().str());
    return t.get_device();
}

// A contiguous tensor of that shape and type on that device: its address, null for a null tensor.
void* need(const at::Tensor* t, const char* what, c10::ScalarType type, Shape shape, int dev)
{
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != type || t->sizes() != at::IntArrayRef(shape) || !t->is_contiguous() || !t->is_cuda() ||
        t->get_device() != dev) {
        std::ostringstream s;
        s << what << " must be a contiguous " << type << " tensor of shape " << at::IntArrayRef(shape) << " on cuda:" << dev
          << ", not " << text(*t);
        C10_THROW_ERROR(ValueError, s.str());
    }
    return t->data_ptr();
}

twell_dtype code(const at::Tensor& t)
{
    if (t.scalar_type() == at::kBFloat16) return TWELL_BF16;
    if (t.scalar_type() == at::kFloat) return TWELL_F32;
    std::ostringstream s;
    s << "unsupported element type " << t.scalar_type();
    C10_THROW_ERROR(TypeError, s.str());
}

// A torch stream's raw handle as an int, or None for the current stream.
c10::cuda::CUDAStream stream_of(PyObject* o, int dev)
{
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev);
    const auto raw = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(o));
    if (PyErr_Occurred()) throw python_error();
    return c10::cuda::getStreamFromExternal(raw, dev);
}

int32_t integer(PyObject* o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    if (v < INT32_MIN || v > INT32_MAX) C10_THROW_ERROR(ValueError, "an argument does not fit 32 bits");
    return static_cast<int32_t>(v);
}

float number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return static_cast<float>(v);
}

// A call's workspace: its memory, held while the call launches, and the lock that its launches are made under where
// other calls use the same one.
struct Workspace {
    at::Tensor t;
    std::mutex* turn;
};

// Bytes that any call of an operator needs. Its buffers have this size from the start (10 MB, 26 MB and 9 MB) and are never
// replaced.
int64_t most_bytes(twell_op op)
{
    if (op == TWELL_OP_LORA_ADD)
        return std::max<int64_t>(static_cast<int64_t>(twell_workspace_bytes(op, kLoraMaxTokens, kLoraMaxRank, 1, 0, 0, 0)), 1);
    if (op == TWELL_OP_PAGED_ATTN) return static_cast<int64_t>(twell_workspace_bytes(op, 1, 256, 1, 0, 0, 0));
    size_t most = 1;
    for (int32_t d = 8; d <= 16384; d += 8) most = std::max(most, twell_workspace_bytes(op, INT32_MAX, d, 1, 0, 0, 0));
    return static_cast<int64_t>(most);
}

at::Tensor bytes_on(int64_t n, int dev, const c10::cuda::CUDAStream& s)
{
    const c10::cuda::CUDAStreamGuard guard(s);
    return at::empty({n}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev));
}

// The workspace of one operator on one device and stream: the kernels of one stream run one after the other, so calls can
// share it, each making its launches (two where a second kernel reads what a first left there) without another thread's
// between them. A call that is being captured into a graph gets one of its own, from the graph's memory: the graph
// may replay on any stream, beside any other call. The map is never destroyed (its tensors would outlive the
// CUDA context).
Workspace workspace(twell_op op, int32_t N, int32_t d, int dev, const c10::cuda::CUDAStream& s)
{
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    C10_CUDA_CHECK(cudaStreamIsCapturing(s.stream(), &capture));
    if (capture != cudaStreamCaptureStatusNone)
        return {bytes_on(std::max<int64_t>(static_cast<int64_t>(twell_workspace_bytes(op, N, d, 1, 0, 0, 0)), 1), dev, s), nullptr};
    struct Shared {
        at::Tensor t;
        std::mutex turn;
    };
    static auto* all = new std::map<std::tuple<int, int, cudaStream_t>, Shared>();
    Shared& w = (*all)[{static_cast<int>(op), dev, s.stream()}];
    if (!w.t.defined()) w.t = bytes_on(most_bytes(op), dev, s);
    return {w.t, &w.turn};
}

// The caller's workspace, or the stream's.
Workspace workspace(PyObject* o, twell_op op, int32_t N, int32_t d, int dev, const c10::cuda::CUDAStream& s)
{
    if (o == Py_None) return workspace(op, N, d, dev, s);
    const at::Tensor* t = tensor(o, "ws");
    need(t, "ws", at::kByte, {t->numel()}, dev);
    return {*t, nullptr};
}

const twell_kv_cache* cache_at(PyObject* o)
{
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw python_error();
    return static_cast<const twell_kv_cache*>(p);
}

// A tensor's size, which the C ABI takes in 32 bits.
int32_t size32(int64_t n, const char* what)
{
    if (n > INT32_MAX) {
        std::ostringstream s;
        s << what << ": " << n << " does not fit 32 bits";
        C10_THROW_ERROR(ValueError, s.str());
    }
    return static_cast<int32_t>(n);
}

// [n, heads, head_dim] bf16 with contiguous heads and any token stride, and its address.
struct Heads {
    const void* at;
    int64_t stride;
};
Heads need_heads(const at::Tensor& t, const char* what, int64_t n, int64_t heads, int64_t hd, int dev)
{
    if (t.scalar_type() != at::kBFloat16 || t.sizes() != at::IntArrayRef({n, heads, hd}) || !t.is_cuda() || t.get_device() != dev ||
        (t.numel() > 0 && ((heads > 1 && t.stride(1) != hd) || t.stride(2) != 1))) {
        std::ostringstream s;
        s << what << " must be bf16 [" << n << ", " << heads << ", " << hd << "] on cuda:" << dev << " with contiguous heads, not "
          << text(t);
        C10_THROW_ERROR(ValueError, s.str());
    }
    return {t.data_ptr(), n > 1 ? t.stride(0) : heads * hd};
}

// The C call on device `dev`, which is made current for it (the entries launch on the current device, and a default
// stream's handle is the same on all), without the interpreter's lock; under a shared workspace's own, which is taken and given back while the
// interpreter's is not held, so that neither waits for the other. `f` throws nothing: no tensor is touched in it.
template <typename F>
PyObject* call(int dev, F f, std::mutex* turn = nullptr)
{
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != dev) guard.set_index(static_cast<c10::DeviceIndex>(dev));
    twell_status st;
    Py_BEGIN_ALLOW_THREADS
    {
        std::unique_lock<std::mutex> lock;
        if (turn != nullptr) lock = std::unique_lock<std::mutex>(*turn);
        st = f();
    }
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

PyObject* count_error(const char* name, Py_ssize_t want, Py_ssize_t got)
{
    return PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, not %zd", name, want, got);
}
#define TWELL_ARGS(NAME, WANT) \
    if (n != WANT) return count_error(NAME, WANT, n)

// x, w, res, eps, h, y, y8, y8_scale, group, rstd, stream
PyObject* add_rmsnorm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TWELL_ARGS("add_rmsnorm_fwd", 11);
    const at::Tensor &x = *tensor(a[0], "x"), *res = tensor(a[2], "res", true), *h = tensor(a[4], "h", true);
    const int dev = device_of(x, "x");
    if (x.dim() != 2) C10_THROW_ERROR(ValueError, "x must have two dimensions");
    const int32_t N = size32(x.size(0), "rows of x"), d = size32(x.size(1), "columns of x");
    const auto t = x.scalar_type();
    const auto rt = res ? res->scalar_type() : t;
    const twell_dtype ct = code(x), cr = res ? code(*res) : ct;
    if (!res && h) C10_THROW_ERROR(ValueError, "h is the sum x + res: without res it is x");
    const int32_t group = integer(a[8]);
    if (group < 0) C10_THROW_ERROR(ValueError, "group must not be negative");
    const void* px = need(&x, "x", t, {N, d}, dev);
    const void* pw = need(tensor(a[1], "w"), "w", t, {d}, dev);
    const void* pr = need(res, "res", rt, {N, d}, dev);
    void* ph = need(h, "h", rt, {N, d}, dev);
    void* py_ = need(tensor(a[5], "y", true), "y", t, {N, d}, dev);
    void* p8 = need(tensor(a[6], "the 8-bit rows", true), "the 8-bit rows", at::kFloat8_e4m3fn, {N, d}, dev);
    void* ps = need(tensor(a[7], "the 8-bit rows' scale", true), "the 8-bit rows' scale", at::kFloat,
                    {N, group ? (static_cast<int64_t>(d) + group - 1) / group : 1}, dev);
    void* pd = need(tensor(a[9], "rstd", true), "rstd", at::kFloat, {N}, dev);
    const float eps = number(a[3]);
    const auto s = stream_of(a[10], dev);
    return call(dev, [&] {
        return twell_add_rmsnorm_fwd(px, pr, pw, N, d, eps, ct, cr, ph, py_, p8, static_cast<float*>(ps), group,
                                     static_cast<float*>(pd), s.stream());
    });
    END_HANDLE_TH_ERRORS
}

// dy, h, w, rstd, dh, dx, dw, ws, stream
PyObject* add_rmsnorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TWELL_ARGS("add_rmsnorm_bwd", 9);
    const at::Tensor &dy = *tensor(a[0], "dy"), &h = *tensor(a[1], "h"), &w = *tensor(a[2], "w");
    const int dev = device_of(h, "h");
    if (h.dim() != 2) C10_THROW_ERROR(ValueError, "h must have two dimensions");
    const int32_t N = size32(h.size(0), "rows of h"), d = size32(h.size(1), "columns of h");
    const twell_dtype ct = code(w), cr = code(h), cg = code(dy);
    const auto g = dy.scalar_type();
    const void* ph = need(&h, "h", h.scalar_type(), {N, d}, dev);
    const void* pdy = need(&dy, "dy", g, {N, d}, dev);
    const void* pw = need(&w, "w", w.scalar_type(), {d}, dev);
    const void* prs = need(tensor(a[3], "rstd"), "rstd", at::kFloat, {N}, dev);
    const void* pdh = need(tensor(a[4], "dh", true), "dh", g, {N, d}, dev);
    void* pdx = need(tensor(a[5], "dx"), "dx", g, {N, d}, dev);
    void* pdw = need(tensor(a[6], "dw"), "dw", at::kFloat, {d}, dev);
    const auto s = stream_of(a[8], dev);
    const Workspace ws = workspace(a[7], TWELL_OP_ADD_RMSNORM_BWD, N, d, dev, s);
    void* pws = ws.t.data_ptr();
    const size_t bytes = static_cast<size_t>(ws.t.numel());
    return call(dev, [&] {
        return twell_add_rmsnorm_bwd(pdy, ph, pw, static_cast<const float*>(prs), pdh, N, d, ct, cr, cg, pdx,
                                     static_cast<float*>(pdw), pws, bytes, s.stream());
    }, ws.turn);
    END_HANDLE_TH_ERRORS
}

// cache, device, k, v, slots, status, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TWELL_ARGS("kv_append", 7);
    const twell_kv_cache* c = cache_at(a[0]);
    const int dev = integer(a[1]);
    const at::Tensor &k = *tensor(a[2], "k"), &v = *tensor(a[3], "v"), &slots = *tensor(a[4], "slots");
    const int32_t m = size32(slots.numel(), "slots");
    const void* psl = need(&slots, "slots", at::kInt, {m}, dev);
    const Heads hk = need_heads(k, "k", m, c->n_kv_heads, c->head_dim, dev);
    const Heads hv = need_heads(v, "v", m, c->n_kv_heads, c->head_dim, dev);
    void* st = need(tensor(a[5], "status"), "status", at::kInt, {1}, dev);
    const auto s = stream_of(a[6], dev);
    return call(dev, [&] {
        return twell_kv_append(c, hk.at, hv.at, hk.stride, hv.stride, static_cast<const int32_t*>(psl), m,
                               static_cast<int32_t*>(st), s.stream());
    });
    END_HANDLE_TH_ERRORS
}

// cache, device, slots, k_out, v_out, status, stream
PyObject* kv_gather(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TWELL_ARGS("kv_gather", 7);
    const twell_kv_cache* c = cache_at(a[0]);
    const int dev = integer(a[1]);
    const at::Tensor& slots = *tensor(a[2], "slots");
    const int32_t m = size32(slots.numel(), "slots"), H = c->n_kv_heads, hd = c->head_dim;
    const void* psl = need(&slots, "slots", at::kInt, {m}, dev);
    void* pk = need(tensor(a[3], "k_out"), "k_out", at::kBFloat16, {m, H, hd}, dev);
    void* pv = need(tensor(a[4], "v_out"), "v_out", at::kBFloat16, {m, H, hd}, dev);
    void* st = need(tensor(a[5], "status"), "status", at::kInt, {1}, dev);
    const auto s = stream_of(a[6], dev);
    return call(dev, [&] {
        return twell_kv_gather(c, static_cast<const int32_t*>(psl), m, pk, pv, static_cast<int32_t*>(st), s.stream());
    });
    END_HANDLE_TH_ERRORS
}

// q, cache, device, page_table, seq_lens, scale, window, out, lse, ws, status, stream
PyObject* paged_attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TWELL_ARGS("paged_attn_decode", 12);
    const twell_kv_cache* c = cache_at(a[1]);
    const int dev = integer(a[2]);
    const at::Tensor &q = *tensor(a[0], "q"), &table = *tensor(a[3], "page_table");
    if (q.dim() != 3) C10_THROW_ERROR(ValueError, "q must be bf16 [B, n_q_heads, head_dim]");
    if (table.dim() != 2) C10_THROW_ERROR(ValueError, "page_table must be int32 [B, max_pages]");
    const int32_t B = size32(q.size(0), "sequences"), H = size32(q.size(1), "query heads"), hd = c->head_dim;
    const int32_t max_pages = size32(table.size(1), "page_table's columns");
    const Heads hq = need_heads(q, "q", B, H, hd, dev);
    const void* pt = need(&table, "page_table", at::kInt, {B, max_pages}, dev);
    const void* pl = need(tensor(a[4], "seq_lens"), "seq_lens", at::kInt, {B}, dev);
    void* po = need(tensor(a[7], "out"), "out", at::kBFloat16, {B, H, hd}, dev);
    void* ps = need(tensor(a[8], "lse", true), "lse", at::kFloat, {B, H}, dev);
    void* st = need(tensor(a[10], "status"), "status", at::kInt, {1}, dev);
    const float scale = number(a[5]);
    const int32_t window = integer(a[6]);
    const auto s = stream_of(a[11], dev);
    const Workspace ws = workspace(a[9], TWELL_OP_PAGED_ATTN, B, hd, dev, s);
    void* pws = ws.t.data_ptr();
    const size_t bytes = static_cast<size_t>(ws.t.numel());
    return call(dev, [&] {
        return twell_paged_attn_decode(hq.at, hq.stride, c, static_cast<const int32_t*>(pt), static_cast<const int32_t*>(pl),
                                       B, H, max_pages, scale, window, po, static_cast<float*>(ps), pws, bytes,
                                       static_cast<int32_t*>(st), s.stream());
    }, ws.turn);
    END_HANDLE_TH_ERRORS
}

// x, words, scales, n, k, group, y, stream
PyObject* w4_matvec(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TWELL_ARGS("w4_matvec", 8);
    const at::Tensor &x = *tensor(a[0], "x"), &words = *tensor(a[1], "words"), &scales = *tensor(a[2], "scales");
    const int dev = device_of(words, "words");
    const int32_t rows = integer(a[3]), cols = integer(a[4]);
    const int32_t group = integer(a[5]);
    if (x.dim() != 2) C10_THROW_ERROR(ValueError, "x must have two dimensions");
    if (rows <= 0 || cols <= 0 || group <= 0 || group > 128 || 128 % group != 0) C10_THROW_ERROR(ValueError, "the weights' sizes");
    const int32_t N = size32(x.size(0), "rows of x");
    const int64_t nt = (static_cast<int64_t>(rows) + 15) / 16, kt = (static_cast<int64_t>(cols) + 127) / 128;
    const void* px = need(&x, "x", at::kBFloat16, {N, cols}, dev);
    const void* pw = need(&words, "words", at::kInt, {nt, kt, 8, 4, 2, 4}, dev);
    const void* ps = need(&scales, "scales", at::kBFloat16, {nt, kt, 8, 2, 128 / group}, dev);
    void* po = need(tensor(a[6], "y"), "y", at::kBFloat16, {N, rows}, dev);
    const auto s = stream_of(a[7], dev);
    return call(dev, [&] {
        return twell_w4_matvec(px, pw, ps, N, rows, cols, group, po, s.stream());
    });
    END_HANDLE_TH_ERRORS
}

// A side of a rotation: [n, heads, head_dim] or [sequences, n, heads, head_dim], head_dim contiguous, in and out.
twell_rope_heads rope_side(const at::Tensor& in, const at::Tensor& out, const char* what, const at::Tensor& like, int64_t hd, int dev)
{
    const int64_t dims = like.dim();
    bool ok = true;
    for (const at::Tensor* t : {&in, &out}) {
        ok = ok && t->dim() == dims && t->scalar_type() == like.scalar_type() && t->is_cuda() && t->get_device() == dev;
        if (!ok) break;
        for (int64_t i = 0; i < dims - 2; ++i) ok = ok && t->size(i) == like.size(i);
        ok = ok && t->size(dims - 2) == in.size(dims - 2) && t->size(dims - 1) == hd && (t->numel() == 0 || t->stride(dims - 1) == 1 || hd == 1);
    }
    if (!ok) {
        std::ostringstream s;
        s << what << " and where it goes must be of q's type, device, sequences and tokens, with contiguous heads of " << hd
          << ", not " << text(in) << " and " << text(out);
        C10_THROW_ERROR(ValueError, s.str());
    }
    auto batch = [&](const at::Tensor& t) { return dims == 4 ? t.stride(0) : int64_t{0}; };
    return {in.data_ptr(), out.data_ptr(), size32(in.size(dims - 2), "heads"), batch(in), in.stride(dims - 3), in.stride(dims - 2),
            batch(out), out.stride(dims - 3), out.stride(dims - 2)};
}

// q, k, positions, turns, factor, neighbours, head_dim, q_out, k_out, backward, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TWELL_ARGS("rope", 11);
    const at::Tensor &q = *tensor(a[0], "q"), *k = tensor(a[1], "k", true), &pos = *tensor(a[2], "positions");
    const at::Tensor &turns = *tensor(a[3], "turns"), &q_out = *tensor(a[7], "q_out"), *k_out = tensor(a[8], "k_out", true);
    const int dev = device_of(q, "q");
    if (q.dim() != 3 && q.dim() != 4) C10_THROW_ERROR(ValueError, "q must be [tokens, heads, head_dim] or [sequences, tokens, heads, head_dim]");
    if ((k == nullptr) != (k_out == nullptr)) C10_THROW_ERROR(ValueError, "k and k_out go together");
    const twell_dtype ct = code(q);
    const bool many = q.dim() == 4;
    const int32_t B = many ? size32(q.size(0), "sequences") : 1, S = size32(q.size(many ? 1 : 0), "tokens");
    const int32_t hd = integer(a[6]), neighbours = integer(a[5]), rot = size32(2 * turns.numel(), "the rotation's pairs");
    const twell_rope_heads hq = rope_side(q, q_out, "q", q, hd, dev);
    const twell_rope_heads hk = k ? rope_side(*k, *k_out, "k", q, hd, dev) : twell_rope_heads{};
    const bool own = many && pos.dim() == 2;  // positions of each sequence's own
    const void* pp = own ? need(&pos, "positions", at::kInt, {B, S}, dev) : need(&pos, "positions", at::kInt, {S}, dev);
    const void* pt = need(&turns, "turns", at::kLong, {turns.numel()}, dev);
    const float factor = number(a[4]);
    const bool backward = integer(a[9]) != 0;
    const auto s = stream_of(a[10], dev);
    return call(dev, [&] {
        return (backward ? twell_rope_bwd : twell_rope_fwd)(&hq, k ? &hk : nullptr, static_cast<const int32_t*>(pp), own ? S : 0,
                                                            static_cast<const uint64_t*>(pt), factor, B, S, hd, rot, neighbours, ct,
                                                            s.stream());
    });
    END_HANDLE_TH_ERRORS
}

// ring, state, page_size, page_table, seq_lens, new_lens, labels, slots, positions, owner, starts, seq_lens_out, state_out,
// status, stream
PyObject* kv_plan(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TWELL_ARGS("kv_plan", 15);
    const at::Tensor &ring = *tensor(a[0], "ring"), &table = *tensor(a[3], "page_table"), &slots = *tensor(a[7], "slots");
    const int dev = device_of(ring, "ring");
    if (table.dim() != 2) C10_THROW_ERROR(ValueError, "page_table must be int32 [B, max_pages]");
    const int32_t B = size32(table.size(0), "requests"), max_pages = size32(table.size(1), "page_table's columns");
    const int32_t M = size32(slots.numel(), "slots");
    auto ints = [&](int i, const char* what, Shape shape, bool optional = false) {
        return static_cast<int32_t*>(need(tensor(a[i], what, optional), what, at::kInt, shape, dev));
    };
    const twell_page_pool pool = {size32(ring.numel(), "pages"), integer(a[2]), ints(0, "ring", {ring.numel()}), ints(1, "state", {4})};
    int32_t* pt = ints(3, "page_table", {B, max_pages});
    const int32_t *pl = ints(4, "seq_lens", {B}), *pn = ints(5, "new_lens", {B}), *pb = ints(6, "labels", {B}, true);
    int32_t *ps = ints(7, "slots", {M}), *pp = ints(8, "positions", {M}), *po = ints(9, "owner", {M});
    int32_t* pst = ints(10, "starts", {static_cast<int64_t>(B) + 1});
    int32_t *lo = ints(11, "seq_lens_out", {B}), *so = ints(12, "state_out", {4}), *st = ints(13, "status", {1});
    const auto s = stream_of(a[14], dev);
    return call(dev, [&] {
        return twell_kv_plan(&pool, pt, max_pages, pl, pn, pb, B, M, ps, pp, po, pst, lo, so, st, s.stream());
    });
    END_HANDLE_TH_ERRORS
}

// [n, columns] bf16 with contiguous columns and any row stride, and its address.
Heads need_rows(const at::Tensor& t, const char* what, int64_t n, int64_t columns, int dev)
{
    if (t.scalar_type() != at::kBFloat16 || t.sizes() != at::IntArrayRef({n, columns}) || !t.is_cuda() || t.get_device() != dev ||
        (t.numel() > 0 && columns > 1 && t.stride(1) != 1)) {
        std::ostringstream s;
        s << what << " must be bf16 [" << n << ", " << columns << "] on cuda:" << dev << " with contiguous rows, not " << text(t);
        C10_THROW_ERROR(ValueError, s.str());
    }
    return {t.data_ptr(), n > 1 ? t.stride(0) : columns};
}

// y, x, a, b, scale, ranks, ids, out, ws, status, stream
PyObject* lora_add(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TWELL_ARGS("lora_add", 11);
    const at::Tensor &y = *tensor(a[0], "y"), &x = *tensor(a[1], "x"), &A = *tensor(a[2], "a"), &B = *tensor(a[3], "b");
    const int dev = device_of(A, "a");
    if (A.dim() != 3 || B.dim() != 3 || x.dim() != 2) C10_THROW_ERROR(ValueError, "a and b must have three dimensions, x two");
    const int32_t L = size32(A.size(0), "adapters"), R = size32(A.size(1), "rank"), k = size32(A.size(2), "columns of a");
    const int32_t rows = size32(B.size(1), "rows of b"), N = size32(x.size(0), "tokens");
    twell_adapters ad = {L, R, k, rows, need(&A, "a", at::kBFloat16, {L, R, k}, dev), need(&B, "b", at::kBFloat16, {L, rows, R}, dev),
                         static_cast<const float*>(need(tensor(a[4], "scale"), "scale", at::kFloat, {L}, dev)),
                         static_cast<const int32_t*>(need(tensor(a[5], "ranks", true), "ranks", at::kInt, {L}, dev))};
    const Heads hx = need_rows(x, "x", N, k, dev), hy = need_rows(y, "y", N, rows, dev), ho = need_rows(*tensor(a[7], "out"), "out", N, rows, dev);
    const void* pi = need(tensor(a[6], "ids"), "ids", at::kInt, {N}, dev);
    void* st = need(tensor(a[9], "status"), "status", at::kInt, {1}, dev);
    if (N > kLoraMaxTokens || R > kLoraMaxRank) return PyLong_FromLong(TWELL_ERR_UNSUPPORTED);
    const auto s = stream_of(a[10], dev);
    const Workspace ws = workspace(a[8], TWELL_OP_LORA_ADD, N, R, dev, s);
    void* pws = ws.t.data_ptr();
    const size_t bytes = static_cast<size_t>(ws.t.numel());
    return call(dev, [&] {
        return twell_lora_add(hy.at, hy.stride, hx.at, hx.stride, &ad, static_cast<const int32_t*>(pi), N, const_cast<void*>(ho.at),
                              ho.stride, pws, bytes, static_cast<int32_t*>(st), s.stream());
    }, ws.turn);
    END_HANDLE_TH_ERRORS
}

#define TWELL_METHOD(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TWELL_METHOD(add_rmsnorm_fwd), TWELL_METHOD(add_rmsnorm_bwd), TWELL_METHOD(kv_append),
                         TWELL_METHOD(kv_gather), TWELL_METHOD(paged_attn_decode), TWELL_METHOD(w4_matvec),
                         TWELL_METHOD(rope),            TWELL_METHOD(kv_plan),         TWELL_METHOD(lora_add),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_twell_call", "Calls of libtwell_gb300.so on tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__twell_call() { return PyModule_Create(&module); }
