// Native half of the Python binding of the serving operators and the backward
// passes: the checks on
// torch tensors, the allocation of outputs and workspace, and the call of the
// C ABI, in one step per operator. A serving step makes four short calls per
// layer or step; from Python objects through ctypes each costs 10-14 us of host
// time before its kernel is launched (measured on GB300's Arm cores: decode
// 10.8 us, page maps 13.8 us), more than the kernels of a small step take, and
// here 2-4 us. libfa.so itself stays free of torch types.
//
// Allocations and launches may wait for the GPU, and the GPU for a Python function of
// its stream: they run without the interpreter's lock.
//
// Every function takes its arguments by position (the Python wrappers name and
// document them). A C call's negative status is raised as FaError; setup() hands
// in that class, and PageMaps, the class of maps()'s result.
#include <Python.h>

#include <cmath>
#include <cstdint>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

namespace fa {
int host_probe(int* device, int* sm_count);  // fa_host.h, without its CUDA headers
}

namespace {

using at::Tensor;

PyObject* g_error = nullptr;
PyTypeObject* g_page_maps = nullptr;

PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 2 || !PyType_Check(a[1]) || !PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(a[1]), &PyTuple_Type)) {
        PyErr_SetString(PyExc_TypeError, "setup(FaError, PageMaps)");
        return nullptr;
    }
    g_error = Py_NewRef(a[0]);
    g_page_maps = reinterpret_cast<PyTypeObject*>(Py_NewRef(a[1]));
    Py_RETURN_NONE;
}

PyObject* failed(long long status, const char* what) {
    PyObject* e = PyObject_CallFunction(g_error, "Ls", status, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

// A tensor argument, or the type error.
const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// The same, undefined for None.
const Tensor& tensor_or_none(PyObject* o, const char* name) {
    static const Tensor none;
    return o == Py_None ? none : tensor(o, name);
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

void on(const Tensor& t, c10::Device device) {
    TORCH_CHECK_VALUE(!t.defined() || t.device() == device, "all tensors must be on the same CUDA device");
}

void cuda(const Tensor& t) { TORCH_CHECK_VALUE(t.is_cuda(), "all tensors must be CUDA tensors"); }

void int32(const Tensor& t, const char* name) {
    TORCH_CHECK_TYPE(t.scalar_type() == at::kInt, name, " must be int32");
}

bool is(const Tensor& t, at::IntArrayRef shape) { return t.sizes() == shape; }

// d's values side by side; the last dimension of a table's rows
bool dense_last(const Tensor& t) { return t.size(-1) <= 1 || t.stride(-1) == 1; }

double number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}

int64_t integer(PyObject* o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
}

bool truth(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x != 0;
}

int to_int(int64_t x) {  // (a size past int is refused by the C call's own limits)
    return x > 0x7fffffffLL || x < 0 ? -1 : static_cast<int>(x);
}

// The interpreter's lock, let go.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

Tensor make(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
    return at::detail::empty_cuda(shape, type, like.device(), c10::nullopt);  // (no dispatcher on the way)
}

// A tensor that the call was given and wrote to: what autograd saved of it before is
// no longer that (a backward pass that needs it raises instead of using it).
void wrote(const Tensor& t) {
    if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void arguments(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "wrong number of arguments"); }

// The C description of caches indexed [block, token, head, d].
fa_paged_cache paged_cache(const Tensor& k, const Tensor& v, const Tensor& k_scale, const Tensor& v_scale,
                           c10::Device device) {
    const at::ScalarType t = k.scalar_type();
    TORCH_CHECK_TYPE(v.scalar_type() == t && (t == at::kBFloat16 || t == at::kFloat8_e4m3fn),
                     "k_cache and v_cache must both be bf16 or both float8_e4m3fn");
    TORCH_CHECK_VALUE(k.dim() == 4 && v.sizes() == k.sizes(),
                      "k_cache and v_cache must both be [num_blocks, page_size, heads, d]");
    TORCH_CHECK_VALUE(k.stride(3) == 1 && v.stride(3) == 1, "the d values of a cache row must be contiguous");
    on(k, device);
    on(v, device);
    for (const Tensor* s : {&k_scale, &v_scale}) {
        if (!s->defined()) continue;
        TORCH_CHECK_VALUE(s->scalar_type() == at::kFloat && is(*s, {k.size(2)}) && s->is_contiguous(),
                          "k_scale and v_scale must be contiguous fp32 tensors of one value per key head");
        on(*s, device);
    }
    fa_paged_cache c{};
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.k_scale = static_cast<const float*>(ptr(k_scale));
    c.v_scale = static_cast<const float*>(ptr(v_scale));
    c.k_block = k.stride(0), c.k_token = k.stride(1), c.k_head = k.stride(2);
    c.v_block = v.stride(0), c.v_token = v.stride(1), c.v_head = v.stride(2);
    c.type = t == at::kFloat8_e4m3fn ? FA_CACHE_E4M3 : FA_CACHE_BF16;
    c.num_blocks = to_int(k.size(0)), c.page_size = to_int(k.size(1));
    c.heads = to_int(k.size(2)), c.d = to_int(k.size(3));
    return c;
}

// Frequencies: their number times two.
int frequencies(const Tensor& f, c10::Device device) {
    if (!f.defined()) return 0;
    TORCH_CHECK_VALUE(f.scalar_type() == at::kDouble && f.dim() == 1 && f.is_contiguous(),
                      "inv_freq must be a contiguous fp64 tensor [rotary_dim / 2]");
    on(f, device);
    return to_int(2 * f.numel());
}

PyObject* pair(Tensor a, Tensor b) {
    PyObject* t = PyTuple_New(2);
    if (!t) throw python_error();
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(a)));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(b)));
    return t;
}

// q, k_cache, v_cache, block_table, seq_lens, scale, k_scale, v_scale, out, lse,
// return_lse, workspace, and for groups that share a prefix prefix_lens
PyObject* decode_any(PyObject* const* a, PyObject* prefix_lens) {
    static const Tensor none;
    const Tensor& prefix = prefix_lens ? tensor(prefix_lens, "prefix_lens") : none;
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache");
    const Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
    const Tensor &ks = tensor_or_none(a[6], "k_scale"), &vs = tensor_or_none(a[7], "v_scale");
    Tensor out = tensor_or_none(a[8], "out"), lse = tensor_or_none(a[9], "lse");
    const bool return_lse = truth(a[10]);
    Tensor ws = tensor_or_none(a[11], "workspace");
    TORCH_CHECK_TYPE(q.scalar_type() == at::kBFloat16, "q must be bf16");
    int32(table, "block_table");
    int32(lens, "seq_lens");
    if (prefix_lens) int32(prefix, "prefix_lens");
    TORCH_CHECK_VALUE(q.dim() == 3 && table.dim() == 2 && table.size(0) == q.size(0) && is(lens, {q.size(0)}),
                      "q must be [B, Hq, d], block_table [B, width] and seq_lens [B]");
    TORCH_CHECK_VALUE(q.is_contiguous() && lens.is_contiguous() && dense_last(table),
                      "q, seq_lens and the rows of block_table must be contiguous");
    const int64_t B = q.size(0), Hq = q.size(1), d = q.size(2), width = table.size(1);
    const float scale = static_cast<float>(a[5] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : number(a[5]));
    TORCH_CHECK_VALUE(k.dim() == 4 && k.size(3) == d, "q and the caches must have the same d");
    TORCH_CHECK_VALUE(!out.defined() || (out.scalar_type() == at::kBFloat16 && out.sizes() == q.sizes() &&
                                         out.is_contiguous()), "out must be a contiguous bf16 tensor of q's shape");
    TORCH_CHECK_VALUE(!lse.defined() || (lse.scalar_type() == at::kFloat && is(lse, {B, Hq}) && lse.is_contiguous()),
                      "lse must be a contiguous fp32 tensor [B, Hq]");
    TORCH_CHECK_VALUE(!ws.defined() || (ws.scalar_type() == at::kByte && ws.is_contiguous()),
                      "workspace must be a contiguous uint8 tensor");
    const int64_t groups = prefix_lens && prefix.dim() == 1 ? prefix.numel() : 0;
    TORCH_CHECK_VALUE(!prefix_lens || (groups > 0 && B % groups == 0 && prefix.is_contiguous()),
                      "prefix_lens must be [groups], contiguous, and B a multiple of groups");
    const c10::Device device = q.device();
    const fa_paged_cache cache = paged_cache(k, v, ks, vs, device);
    cuda(q);
    for (const Tensor* t : {&table, &lens, &prefix, static_cast<const Tensor*>(&out), static_cast<const Tensor*>(&lse),
                            static_cast<const Tensor*>(&ws)})
        on(*t, device);
    const long long rc = [&]() -> long long {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard(device);
        if (!out.defined()) out = make(q.sizes(), at::kBFloat16, q);
        if (!lse.defined() && return_lse) lse = make({B, Hq}, at::kFloat, q);
        if (!ws.defined()) {
            int dev = 0, sms = 0;
            const int probed = fa::host_probe(&dev, &sms);
            if (probed != FA_OK) return probed;
            const long long room =
                prefix_lens ? fa_decode_shared_workspace(to_int(B), to_int(Hq), cache.heads, cache.d, cache.type,
                                                         cache.page_size, to_int(width), to_int(groups), sms)
                            : fa_decode_paged_workspace(to_int(B), to_int(Hq), cache.heads, cache.d, cache.type,
                                                        cache.page_size, to_int(width), sms);
            if (room < 0) return room;
            if (room > 0) ws = make({room}, at::kByte, q);
        }
        void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        const size_t room = ws.defined() ? static_cast<size_t>(ws.numel()) : 0;
        const int *tables = static_cast<const int*>(table.data_ptr()), *keys = static_cast<const int*>(lens.data_ptr());
        float* l = static_cast<float*>(ptr(lse));
        if (prefix_lens)
            return fa_decode_shared(q.data_ptr(), &cache, tables, keys, static_cast<const int*>(prefix.data_ptr()),
                                    out.data_ptr(), l, to_int(B), to_int(Hq), to_int(groups), to_int(width),
                                    table.stride(0), scale, ptr(ws), room, stream);
        return fa_decode_paged(q.data_ptr(), &cache, tables, keys, out.data_ptr(), l, to_int(B), to_int(Hq),
                               to_int(width), table.stride(0), scale, ptr(ws), room, stream);
    }();
    if (rc != FA_OK) return failed(rc, prefix_lens ? "fa_decode_shared" : "fa_decode_paged");
    wrote(out);
    wrote(lse);
    wrote(ws);
    return return_lse ? pair(std::move(out), std::move(lse)) : THPVariable_Wrap(std::move(out));
}

PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 12);
    return decode_any(a, nullptr);
    END_HANDLE_TH_ERRORS
}

PyObject* decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 13);
    return decode_any(a, a[12]);
    END_HANDLE_TH_ERRORS
}

PyObject* three(Tensor a, Tensor b, Tensor c) {
    PyObject* t = PyTuple_New(3);
    if (!t) throw python_error();
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(a)));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(b)));
    PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(std::move(c)));
    return t;
}

// A contiguous bf16 tensor of this shape, or none.
void bf16_of(const Tensor& t, at::IntArrayRef shape, const char* name) {
    TORCH_CHECK_TYPE(!t.defined() || t.scalar_type() == at::kBFloat16, name, " must be bf16");
    TORCH_CHECK_VALUE(!t.defined() || (t.sizes() == shape && t.is_contiguous()), name,
                      " must be contiguous and of the shape ", shape);
}

void fp32_of(const Tensor& t, at::IntArrayRef shape, const char* name) {
    TORCH_CHECK_TYPE(!t.defined() || t.scalar_type() == at::kFloat, name, " must be fp32");
    TORCH_CHECK_VALUE(!t.defined() || (t.sizes() == shape && t.is_contiguous()), name,
                      " must be contiguous and of the shape ", shape);
}

// Both backward passes: dout, q, k, v, out, lse, dlse, then (packed) the offsets and the longest counts, then causal,
// scale, dq, dk, dv, workspace
PyObject* backward_any(PyObject* const* a, bool packed) {
    const Tensor &dout = tensor(a[0], "dout"), &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
    const Tensor &o = tensor(a[4], "out"), &lse = tensor(a[5], "lse"), &dlse = tensor_or_none(a[6], "dlse");
    static const Tensor none;
    const Tensor& cu_q = packed ? tensor(a[7], "cu_seqlens_q") : none;
    const Tensor& cu_k = packed ? tensor(a[8], "cu_seqlens_k") : none;
    const int64_t max_q = packed ? integer(a[9]) : 0, max_k = packed ? integer(a[10]) : 0;
    PyObject* const* b = a + (packed ? 11 : 7);
    const bool causal = truth(b[0]);
    Tensor dq = tensor_or_none(b[2], "dq"), dk = tensor_or_none(b[3], "dk"), dv = tensor_or_none(b[4], "dv");
    Tensor ws = tensor_or_none(b[5], "workspace");
    TORCH_CHECK_VALUE(packed ? q.dim() == 3 && k.dim() == 3 && q.size(1) == k.size(1) && q.size(2) == k.size(2)
                             : q.dim() == 4 && k.sizes() == q.sizes(),
                      packed ? "q must be [total_q, H, d] and k, v [total_k, H, d]" : "q, k, v must all be [B, H, N, d]");
    const at::DimVector qs(q.sizes()), ks(k.sizes());
    bf16_of(q, qs, "q");
    bf16_of(k, ks, "k");
    bf16_of(v, ks, "v");
    bf16_of(o, qs, "out");
    bf16_of(dout, qs, "dout");
    bf16_of(dq, qs, "dq");
    bf16_of(dk, ks, "dk");
    bf16_of(dv, ks, "dv");
    const int64_t d = q.size(-1), H = q.size(1);
    const at::DimVector stats = packed ? at::DimVector{H, q.size(0)} : at::DimVector{q.size(0), H, q.size(2)};
    fp32_of(lse, stats, "lse");
    fp32_of(dlse, stats, "dlse");
    if (packed) {
        int32(cu_q, "cu_seqlens_q");
        int32(cu_k, "cu_seqlens_k");
        TORCH_CHECK_VALUE(cu_q.dim() == 1 && cu_k.sizes() == cu_q.sizes() && cu_q.numel() >= 2 &&
                              cu_q.is_contiguous() && cu_k.is_contiguous(),
                          "cu_seqlens_q and cu_seqlens_k must both hold B + 1 offsets");
    }
    TORCH_CHECK_VALUE(!ws.defined() || (ws.scalar_type() == at::kByte && ws.is_contiguous()),
                      "workspace must be a contiguous uint8 tensor");
    const float scale = static_cast<float>(b[1] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : number(b[1]));
    const c10::Device device = q.device();
    cuda(q);
    for (const Tensor* t : {&dout, &k, &v, &o, &lse, &dlse, &cu_q, &cu_k, static_cast<const Tensor*>(&dq),
                            static_cast<const Tensor*>(&dk), static_cast<const Tensor*>(&dv),
                            static_cast<const Tensor*>(&ws)})
        on(*t, device);
    const int64_t rows = packed ? q.size(0) : q.size(0) * q.size(2);
    const long long rc = [&]() -> long long {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard(device);
        if (!dq.defined()) dq = make(qs, at::kBFloat16, q);
        if (!dk.defined()) dk = make(ks, at::kBFloat16, q);
        if (!dv.defined()) dv = make(ks, at::kBFloat16, q);
        if (!ws.defined()) {
            const long long room = fa_bwd_workspace(rows, to_int(H));
            if (room < 0) return room;
            if (room > 0) ws = make({room}, at::kByte, q);
        }
        const size_t room = ws.defined() ? static_cast<size_t>(ws.numel()) : 0;
        void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        const auto stat = [](const Tensor& t) { return static_cast<const float*>(ptr(t)); };
        if (!packed)
            return fa_bwd(ptr(dout), ptr(q), ptr(k), ptr(v), ptr(o), stat(lse), stat(dlse), ptr(dq), ptr(dk), ptr(dv),
                          to_int(q.size(0)), to_int(H), to_int(q.size(2)), to_int(d), scale, causal, ptr(ws), room,
                          stream);
        return fa_bwd_varlen(ptr(dout), ptr(q), ptr(k), ptr(v), ptr(o), stat(lse), stat(dlse), ptr(dq), ptr(dk),
                             ptr(dv), static_cast<const int*>(cu_q.data_ptr()), static_cast<const int*>(cu_k.data_ptr()),
                             to_int(cu_q.numel() - 1), to_int(H), to_int(q.size(0)), to_int(k.size(0)), to_int(max_q),
                             to_int(max_k), to_int(d), scale, causal, ptr(ws), room, stream);
    }();
    if (rc != FA_OK) return failed(rc, packed ? "fa_bwd_varlen" : "fa_bwd");
    for (const Tensor* t : {&dq, &dk, &dv, &ws}) wrote(*t);
    return three(std::move(dq), std::move(dk), std::move(dv));
}

PyObject* backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 13);
    return backward_any(a, false);
    END_HANDLE_TH_ERRORS
}

PyObject* backward_varlen(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 17);
    return backward_any(a, true);
    END_HANDLE_TH_ERRORS
}

// x, positions, inv_freq, interleaved, inverse, factor, out
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 7);
    const Tensor &x = tensor(a[0], "x"), &pos = tensor(a[1], "positions"), &freq = tensor_or_none(a[2], "inv_freq");
    Tensor out = tensor_or_none(a[6], "out");
    TORCH_CHECK_TYPE(x.scalar_type() == at::kBFloat16, "x must be bf16");
    int32(pos, "positions");
    TORCH_CHECK_VALUE(x.dim() == 3 || x.dim() == 4, "x must be [B, H, N, d] or [T, H, d]");
    const bool four = x.dim() == 4;
    const int64_t B = four ? x.size(0) : 1, H = x.size(1), N = four ? x.size(2) : x.size(0), d = x.size(-1);
    const bool each = four && pos.dim() == 2;
    TORCH_CHECK_VALUE(each ? is(pos, {B, N}) : is(pos, {N}),
                      "positions must be [N] or [B, N] (x [B, H, N, d]), or [T] (x [T, H, d])");
    TORCH_CHECK_VALUE(x.stride(-1) == 1 && dense_last(pos), "d of x and the rows of positions must be contiguous");
    TORCH_CHECK_VALUE(!out.defined() || (out.scalar_type() == at::kBFloat16 && out.sizes() == x.sizes() &&
                                         out.stride(-1) == 1),
                      "out must be a bf16 tensor of x's shape with d contiguous");
    const double factor = number(a[5]);
    const bool interleaved = truth(a[3]), inverse = truth(a[4]);
    const c10::Device device = x.device();
    const int r = frequencies(freq, device);
    cuda(x);
    on(pos, device);
    on(out, device);
    const int rc = [&] {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard(device);
        if (!out.defined()) out = make(x.sizes(), at::kBFloat16, x);
        const long long xs[3] = {four ? x.stride(0) : 0, x.stride(1), four ? x.stride(2) : x.stride(0)};
        const long long ys[3] = {four ? out.stride(0) : 0, out.stride(1), four ? out.stride(2) : out.stride(0)};
        return fa_rotary(x.data_ptr(), out.data_ptr(), static_cast<const int*>(pos.data_ptr()),
                         static_cast<const double*>(ptr(freq)), to_int(B), to_int(H), to_int(N), to_int(d), xs, ys,
                         each ? pos.stride(0) : 0, r, interleaved, inverse, static_cast<float>(factor),
                         c10::cuda::getCurrentCUDAStream(device.index()).stream());
    }();
    if (rc != FA_OK) return failed(rc, "fa_rotary");
    wrote(out);
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// q, k, v, positions, slots, inv_freq, k_cache, v_cache, interleaved, factor,
// k_scale, v_scale, q_out, k_out
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 14);
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const Tensor &pos = tensor(a[3], "positions"), &slots = tensor(a[4], "slots");
    const Tensor &freq = tensor_or_none(a[5], "inv_freq"), &kc = tensor(a[6], "k_cache"), &vc = tensor(a[7], "v_cache");
    const Tensor &ks = tensor_or_none(a[10], "k_scale"), &vs = tensor_or_none(a[11], "v_scale");
    Tensor q_out = tensor_or_none(a[12], "q_out");
    const Tensor& k_out = tensor_or_none(a[13], "k_out");
    TORCH_CHECK_TYPE(q.scalar_type() == at::kBFloat16 && k.scalar_type() == at::kBFloat16 &&
                         v.scalar_type() == at::kBFloat16, "q, k, v must be bf16");
    int32(pos, "positions");
    int32(slots, "slots");
    TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() == 3 && v.sizes() == k.sizes() && k.size(0) == q.size(0) &&
                          k.size(2) == q.size(2), "q must be [T, Hq, d] and k, v [T, heads, d]");
    const int64_t T = q.size(0), Hq = q.size(1), heads = k.size(1), d = q.size(2);
    TORCH_CHECK_VALUE(kc.dim() == 4 && kc.size(2) == heads && kc.size(3) == d,
                      "q, k, v and the caches do not fit together");
    TORCH_CHECK_VALUE(is(pos, {T}) && is(slots, {T}) && pos.is_contiguous() && slots.is_contiguous(),
                      "positions and slots must be contiguous [T]");
    TORCH_CHECK_VALUE(!q_out.defined() || (q_out.scalar_type() == at::kBFloat16 && q_out.sizes() == q.sizes()),
                      "q_out must be bf16 and of q's shape");
    TORCH_CHECK_VALUE(!k_out.defined() || (k_out.scalar_type() == at::kBFloat16 && k_out.sizes() == k.sizes()),
                      "k_out must be bf16 and of k's shape");
    for (const Tensor* t : {&q, &k, &v, static_cast<const Tensor*>(&q_out), &k_out})
        TORCH_CHECK_VALUE(!t->defined() || (t->stride(2) == 1 && (t->size(1) <= 1 || t->stride(1) == d)),
                          "the heads of a token of q, k, v, q_out and k_out must be contiguous");
    const double factor = number(a[9]);
    const bool interleaved = truth(a[8]);
    const c10::Device device = q.device();
    const fa_paged_cache cache = paged_cache(kc, vc, ks, vs, device);
    const int r = frequencies(freq, device);
    cuda(q);
    for (const Tensor* t : {&k, &v, &pos, &slots, static_cast<const Tensor*>(&q_out), &k_out}) on(*t, device);
    const int rc = [&] {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard(device);
        if (!q_out.defined()) q_out = make(q.sizes(), at::kBFloat16, q);
        return fa_cache_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), q.stride(0), k.stride(0), v.stride(0),
                               static_cast<const int*>(pos.data_ptr()), static_cast<const int*>(slots.data_ptr()),
                               static_cast<const double*>(ptr(freq)), &cache, q_out.data_ptr(), ptr(k_out),
                               q_out.stride(0), k_out.defined() ? k_out.stride(0) : 0, to_int(T), to_int(Hq), r,
                               interleaved, static_cast<float>(factor),
                               c10::cuda::getCurrentCUDAStream(device.index()).stream());
    }();
    if (rc != FA_OK) return failed(rc, "fa_cache_append");
    wrote(q_out);
    wrote(k_out);
    wrote(kc);
    wrote(vc);
    return THPVariable_Wrap(std::move(q_out));
    END_HANDLE_TH_ERRORS
}

// context_lens, new_lens, block_table, unused_blocks, page_size, num_tokens, out
// (None or a PageMaps). Returns a PageMaps.
PyObject* maps(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 7);
    const Tensor &ctx = tensor(a[0], "context_lens"), &fresh = tensor(a[1], "new_lens");
    const Tensor &table = tensor(a[2], "block_table"), &unused = tensor(a[3], "unused_blocks");
    const int64_t page = integer(a[4]), T = integer(a[5]);
    int32(ctx, "context_lens");
    int32(fresh, "new_lens");
    int32(table, "block_table");
    int32(unused, "unused_blocks");
    TORCH_CHECK_VALUE(table.dim() == 2 && unused.dim() == 1,
                      "block_table must be [B, width] and unused_blocks one list");
    const int64_t B = table.size(0), width = table.size(1);
    TORCH_CHECK_VALUE(is(ctx, {B}) && is(fresh, {B}), "context_lens and new_lens must be [B]");
    TORCH_CHECK_VALUE(dense_last(table) && ctx.is_contiguous() && fresh.is_contiguous() && unused.is_contiguous(),
                      "the rows of block_table, the lengths and unused_blocks must be contiguous");
    TORCH_CHECK_VALUE(T >= 0, "num_tokens must be >= 0");
    const c10::Device device = table.device();
    const int64_t sizes[5] = {T, T, B + 1, B, 4};
    Tensor out[5];
    if (a[6] != Py_None) {
        TORCH_CHECK_TYPE(PyTuple_Check(a[6]) && PyTuple_GET_SIZE(a[6]) == 5, "out must be a PageMaps");
        for (int i = 0; i < 5; ++i) {
            out[i] = tensor(PyTuple_GET_ITEM(a[6], i), "out");
            TORCH_CHECK_VALUE(out[i].scalar_type() == at::kInt && is(out[i], {sizes[i]}) && out[i].is_contiguous(),
                              "out must be int32 tensors [T], [T], [B + 1], [B] and [4]");
        }
    }
    cuda(table);
    for (const Tensor* t : {&ctx, &fresh, &unused}) on(*t, device);
    for (const Tensor& t : out) on(t, device);
    const bool given = a[6] != Py_None;
    const int rc = [&] {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard(device);
        if (!given) {
            // five parts of one allocation (each at a 16-byte boundary): allocations take most of a short call
            int64_t at = 0;
            for (int64_t n : sizes) at += (n + 3) / 4 * 4;
            const Tensor whole = make({at}, at::kInt, table);
            at = 0;
            for (int i = 0; i < 5; ++i) {
                out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(whole.storage()),
                                                                  whole.key_set(), whole.dtype());
                out[i].unsafeGetTensorImpl()->set_storage_offset(at);
                out[i].unsafeGetTensorImpl()->set_sizes_contiguous({sizes[i]});
                at += (sizes[i] + 3) / 4 * 4;
            }
        }
        int* p[5];
        for (int i = 0; i < 5; ++i) p[i] = static_cast<int*>(out[i].data_ptr());
        return fa_page_maps(static_cast<const int*>(ctx.data_ptr()), static_cast<const int*>(fresh.data_ptr()),
                            static_cast<int*>(table.data_ptr()), static_cast<const int*>(unused.data_ptr()), p[0], p[1],
                            p[2], p[3], p[4], to_int(B), to_int(width), table.stride(0), to_int(unused.numel()),
                            to_int(page), to_int(T), c10::cuda::getCurrentCUDAStream(device.index()).stream());
    }();
    if (rc != FA_OK) return failed(rc, "fa_page_maps");
    wrote(table);
    if (given) {
        for (const Tensor& t : out) wrote(t);
        return Py_NewRef(a[6]);
    }
    PyObject* t = g_page_maps->tp_alloc(g_page_maps, 5);  // a named tuple: filled as one
    if (!t) throw python_error();
    for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(std::move(out[i])));
    return t;
    END_HANDLE_TH_ERRORS
}

#define FA_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef kMethods[] = {{"setup", FA_FAST(setup), METH_FASTCALL, nullptr},
                          {"decode", FA_FAST(decode), METH_FASTCALL, nullptr},
                          {"decode_shared", FA_FAST(decode_shared), METH_FASTCALL, nullptr},
                          {"backward", FA_FAST(backward), METH_FASTCALL, nullptr},
                          {"backward_varlen", FA_FAST(backward_varlen), METH_FASTCALL, nullptr},
                          {"rotary", FA_FAST(rotary), METH_FASTCALL, nullptr},
                          {"append", FA_FAST(append), METH_FASTCALL, nullptr},
                          {"maps", FA_FAST(maps), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fa_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_bind() { return PyModule_Create(&kModule); }
