// The packed-step calls (include/mla_step.h) on torch tensors: argument checks,
// output allocation, the tensors' device and its current stream, then the C call.
// A step's small calls take a few microseconds on the GPU, so their host side is
// compiled: 5 to 7 us a call, 4 of them the launch, against 10 to 19 us of the same
// checks through ctypes.
#include <Python.h>

#include <string>

#include <ATen/ATen.h>
#include <ATen/cuda/CUDAContextLight.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mla_step.h"

namespace {

PyObject *g_error = nullptr;   // MLAError(status, what)
PyObject *g_dims = nullptr;    // the ctypes struct of mla_dims

struct Refused {
    mla_status status;
    std::string what;
};

void require(bool ok, const char *call, const char *what) {
    if (!ok) throw Refused{MLA_ERR_INVALID_ARG, std::string(call) + ": " + what};
}

void check(mla_status st, const char *call) {
    if (st != MLA_OK) throw Refused{st, call};
}

// Runs `f` with Refused turned into MLAError and torch's errors into theirs.
template <typename F>
PyObject *guarded(F f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refused &r) {
        PyObject *e = PyObject_CallFunction(g_error, "is", static_cast<int>(r.status), r.what.c_str());
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

bool none(PyObject *o) { return o == Py_None; }

const at::Tensor &tensor(PyObject *o, const char *call, const char *name) {
    if (!THPVariable_Check(o)) throw Refused{MLA_ERR_INVALID_ARG, std::string(call) + ": " + name + " is a tensor"};
    return THPVariable_Unpack(o);
}

// A contiguous tensor of one type on the call's device; none allowed if `opt`.
at::Tensor flat(PyObject *o, const char *call, const char *name, at::ScalarType type, int index, bool opt = false) {
    if (opt && none(o)) return at::Tensor();
    const at::Tensor &t = tensor(o, call, name);
    if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != type || !t.is_contiguous())
        throw Refused{MLA_ERR_INVALID_ARG, std::string(call) + ": " + name + " is a contiguous " + at::toString(type) +
                                               " tensor on cuda:" + std::to_string(index)};
    return t;
}

int device_of(PyObject *o, const char *call, const char *name) {
    const at::Tensor &t = tensor(o, call, name);
    if (!t.is_cuda()) throw Refused{MLA_ERR_INVALID_ARG, std::string(call) + ": " + name + " is on a CUDA device"};
    return t.get_device();
}

int64_t integer(PyObject *o, const char *call, const char *name, int64_t lo, int64_t hi) {
    int over = 0;
    PyObject *whole = PyNumber_Index(o);   // Python's and numpy's integers
    const int64_t v = whole ? PyLong_AsLongLongAndOverflow(whole, &over) : (over = 1, 0);
    Py_XDECREF(whole);
    PyErr_Clear();
    if (over || v < lo || v > hi)
        throw Refused{MLA_ERR_INVALID_ARG, std::string(call) + ": " + name + " is a whole number in range"};
    return v;
}

double real(PyObject *o, const char *call, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{MLA_ERR_INVALID_ARG, std::string(call) + ": " + name + " is a number"};
    }
    return v;
}

int32_t layout_of(PyObject *o, const char *call) {
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "interleaved") == 0) return MLA_ROPE_INTERLEAVED;
        if (PyUnicode_CompareWithASCIIString(o, "half") == 0) return MLA_ROPE_HALF;
    }
    throw Refused{MLA_ERR_INVALID_ARG, std::string(call) + ": layout is \"interleaved\" or \"half\""};
}

mla_dims dims_of(PyObject *o, const char *call) {
    mla_dims d;
    Py_buffer view;
    if (PyObject_IsInstance(o, g_dims) != 1 || PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) {
        PyErr_Clear();
        throw Refused{MLA_ERR_INVALID_ARG, std::string(call) + ": dims are make_dims'"};
    }
    const bool fits = view.len == static_cast<Py_ssize_t>(sizeof(d));
    if (fits) std::memcpy(&d, view.buf, sizeof(d));
    PyBuffer_Release(&view);
    require(fits, call, "dims are make_dims'");
    return d;
}

void *ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
template <typename T>
T *ptr(const at::Tensor &t) {
    return static_cast<T *>(ptr(t));
}

PyObject *wrap(const at::Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

// What a call writes is written behind autograd's back: a tensor that it tracks is refused, as torch
// refuses a leaf in place, and the version of one that was written moves on, as after an operation of torch in
// place, so that a backward pass which has saved it says so. (Tensors of inference mode have no version.)
void may_write(const at::Tensor &t, const char *call, const char *name) {
    if (t.defined() && t.requires_grad() && c10::GradMode::is_enabled())
        throw Refused{MLA_ERR_INVALID_ARG, std::string(call) + ": " + name +
                                               " requires grad, and autograd would not see that it is written"};
}
void wrote(const at::Tensor &t) {
    if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// The tensors' device made current where it is not, and its current stream.
struct Place {
    c10::cuda::OptionalCUDAGuard guard;
    at::AutoDispatchBelowADInplaceOrView below;   // outputs take no part in autograd
    void *stream;
    explicit Place(int index) {
        if (c10::cuda::current_device() != index) guard.set_index(index);
        stream = c10::cuda::getCurrentCUDAStream(index).stream();
    }
};

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, int index) {
    return at::empty(sizes, at::TensorOptions(at::Device(at::kCUDA, index)).dtype(type));
}

// A contiguous tensor of `type` inside the allocation of a byte tensor, `first` elements in.
at::Tensor piece(const at::Tensor &bytes, at::ScalarType type, int64_t first, at::IntArrayRef sizes) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(bytes.storage()), bytes.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(first);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    return t;
}

struct Pools {
    mla_pool ckv, kr;
    int32_t pages;
};

Pools pools(PyObject *ckv, PyObject *kr, const mla_dims &d, at::ScalarType type, int index, const char *call) {
    const at::Tensor &c = tensor(ckv, call, "the c_KV pool"), &k = tensor(kr, call, "the k_R pool");
    require(c.is_cuda() && k.is_cuda() && c.get_device() == index && k.get_device() == index &&
                c.scalar_type() == type && k.scalar_type() == at::kBFloat16 && c.dim() == 3 && k.dim() == 3 &&
                c.size(0) == k.size(0) && c.size(0) <= INT32_MAX && c.size(1) == 64 && k.size(1) == 64 &&
                c.size(2) == d.d_latent && k.size(2) == d.d_rope && c.stride(2) == 1 && k.stride(2) == 1,
            call, "pools [pages, 64, d_c] (bf16, or uint8 codes) and [pages, 64, d_R] bf16 on one device");
    return {{c.data_ptr(), c.stride(0), c.stride(1)},
            {k.data_ptr(), k.stride(0), k.stride(1)},
            static_cast<int32_t>(c.size(0))};
}

// plan(cached_lens, new_lens, free_pages, free_head, block_table, num_tokens, parents, max_nodes, out)
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t) {
    return guarded([&]() -> PyObject * {
        const char *call = "step_plan";
        const int index = device_of(a[4], call, "block_table");
        const Place here(index);
        const at::Tensor cached = flat(a[0], call, "cached_lens", at::kInt, index),
                         fresh = flat(a[1], call, "new_lens", at::kInt, index),
                         pages = flat(a[2], call, "free_pages", at::kInt, index),
                         head = flat(a[3], call, "free_head", at::kInt, index),
                         table = flat(a[4], call, "block_table", at::kInt, index),
                         parents = flat(a[6], call, "parents", at::kInt, index, true);
        const int64_t T = integer(a[5], call, "num_tokens", 0, INT32_MAX);
        const bool tree = parents.defined();
        const int64_t nodes = integer(a[7], call, "max_nodes", tree ? 1 : 0, tree ? MLA_TREE_MAX_NODES : INT32_MAX);
        require(table.dim() == 2, call, "block_table [B, max_pages]");
        const int64_t B = table.size(0), words = tree ? (nodes + 31) / 32 : 0;
        require(B < INT32_MAX && table.size(1) <= INT32_MAX && pages.numel() <= INT32_MAX, call, "sizes");
        require(cached.sizes() == at::IntArrayRef({B}) && fresh.sizes() == at::IntArrayRef({B}) && head.numel() == 1 &&
                    (!tree || parents.numel() == T),
                call, "cached_lens and new_lens [B], one free_head, parents [num_tokens]");
        at::Tensor o[7];   // seq_lens, cu_tokens, seq_ids, positions, slots, free_head, masks
        const int64_t sizes[7] = {B, B + 1, T, T, T, 1, T * words};
        if (none(a[8])) {
            // one allocation: slots (int64) first, then the int32 ones
            const at::Tensor all = empty({8 * T + 4 * (2 * B + 2 + 2 * T + T * words)}, at::kByte, index);
            o[4] = piece(all, at::kLong, 0, {T});
            int64_t first = 2 * T;
            for (int i : {0, 1, 2, 3, 5}) {
                o[i] = piece(all, at::kInt, first, {sizes[i]});
                first += sizes[i];
            }
            if (tree) o[6] = piece(all, at::kInt, first, {T, words});
        } else {
            require(PyTuple_Check(a[8]) && PyTuple_GET_SIZE(a[8]) == 7, call, "out is a StepPlan");
            for (int i = 0; i < 7; ++i) {
                o[i] = flat(PyTuple_GET_ITEM(a[8], i), call, "out", i == 4 ? at::kLong : at::kInt, index, i == 6 && !tree);
                require((i == 6 && !tree) || (o[i].numel() == sizes[i] && (i != 6 || o[i].size(0) == T)), call,
                        "out of other sizes");
            }
        }
        check(mla_step_plan(ptr<int32_t>(cached), ptr<int32_t>(fresh), static_cast<int32_t>(B), ptr<int32_t>(pages),
                            static_cast<int32_t>(pages.numel()), ptr<int32_t>(head), ptr<int32_t>(table),
                            static_cast<int32_t>(table.size(1)), ptr<int32_t>(parents), static_cast<int32_t>(nodes),
                            static_cast<int32_t>(T), ptr<int32_t>(o[0]), ptr<int32_t>(o[1]), ptr<int32_t>(o[2]),
                            ptr<int32_t>(o[3]), ptr<int64_t>(o[4]), tree ? ptr<uint32_t>(o[6]) : nullptr,
                            ptr<int32_t>(o[5]), here.stream),
              "mla_step_plan");
        wrote(table);
        if (!none(a[8])) {
            for (const at::Tensor &t : o) wrote(t);
            return Py_NewRef(a[8]);
        }
        PyObject *r = PyTuple_New(7);
        if (!r) return nullptr;
        for (int i = 0; i < 7; ++i) PyTuple_SET_ITEM(r, i, wrap(o[i]));
        return r;
    });
}

// rotary(x, positions, inv_freq, mscale, layout, offset, inverse, out, k, k_out)
PyObject *rotary(PyObject *, PyObject *const *a, Py_ssize_t) {
    return guarded([&]() -> PyObject * {
        const char *call = "rotary";
        const int index = device_of(a[0], call, "x");
        const Place here(index);
        const at::Tensor &x = tensor(a[0], call, "x");
        const at::ScalarType type = x.scalar_type();
        const int32_t dtype = type == at::kBFloat16 ? MLA_BF16 : type == at::kHalf ? MLA_FP16 : MLA_FP32;
        require(dtype != MLA_FP32 || type == at::kFloat, call, "x is bf16, fp16 or fp32");
        const at::Tensor pos = flat(a[1], call, "positions", at::kInt, index),
                         freq = flat(a[2], call, "inv_freq", at::kDouble, index);
        const int32_t order = layout_of(a[4], call);
        require(x.dim() == 3 && pos.sizes() == at::IntArrayRef({x.size(0)}) && freq.dim() == 1 &&
                    x.size(0) <= INT32_MAX && x.size(2) <= 65536 && freq.numel() <= 65536,
                call, "x [T, heads, width], positions [T], inv_freq [rot / 2]");
        at::Tensor outs[2];
        mla_rotary_tensor arg[2];
        const int n = none(a[8]) ? 1 : 2;
        for (int i = 0; i < n; ++i) {
            const at::Tensor &t = tensor(a[i ? 8 : 0], call, "k");
            PyObject *o = a[i ? 9 : 7];
            outs[i] = none(o) ? at::zeros(t.sizes(), t.options()) : tensor(o, call, "out");
            const at::Tensor &y = outs[i];
            require(t.is_cuda() && y.is_cuda() && t.get_device() == index && y.get_device() == index &&
                        t.scalar_type() == type && y.scalar_type() == type && t.dim() == 3 && t.size(0) == x.size(0) &&
                        t.size(2) == x.size(2) && t.size(1) <= INT32_MAX && t.sizes() == y.sizes() &&
                        ((t.stride(2) == 1 && y.stride(2) == 1) || t.size(2) == 1),
                    call, "[T, heads, width] tensors of one type, tokens and width, out of the same shape");
            may_write(y, call, "out");
            arg[i] = {t.data_ptr(), y.data_ptr(), t.stride(0), t.stride(1), y.stride(0), y.stride(1),
                      static_cast<int32_t>(t.size(1))};
        }
        const int64_t offset = integer(a[5], call, "offset", 0, 65536);
        const int inverse = PyObject_IsTrue(a[6]);
        if (inverse < 0) throw python_error();
        check(mla_rotary(&arg[0], n == 2 ? &arg[1] : nullptr, dtype, static_cast<int32_t>(x.size(0)),
                         static_cast<int32_t>(x.size(2)), static_cast<int32_t>(offset),
                         static_cast<int32_t>(2 * freq.numel()), ptr<int32_t>(pos), ptr<double>(freq),
                         static_cast<float>(real(a[3], call, "mscale")), order, inverse, here.stream),
              "mla_rotary");
        for (int i = 0; i < n; ++i) wrote(outs[i]);
        PyObject *first = none(a[7]) ? wrap(outs[0]) : Py_NewRef(a[7]);
        if (n == 1 || !first) return first;
        return Py_BuildValue("(NN)", first, none(a[9]) ? wrap(outs[1]) : Py_NewRef(a[9]));
    });
}

// append(ckv_new, kr_new, slots, ckv_pool, scales, kr_pool, dims, positions, inv_freq, mscale, layout)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t) {
    return guarded([&]() -> PyObject * {
        const bool fp8 = !none(a[4]);
        const char *call = fp8 ? "append_kv_slots_fp8" : "append_kv_slots";
        const int index = device_of(a[0], call, "ckv_new");
        const Place here(index);
        const at::Tensor &c = tensor(a[0], call, "ckv_new"), &k = tensor(a[1], call, "kr_new");
        const at::Tensor slots = flat(a[2], call, "slots", at::kLong, index),
                         pos = flat(a[7], call, "positions", at::kInt, index, true),
                         freq = flat(a[8], call, "inv_freq", at::kDouble, index, true);
        const mla_dims d = dims_of(a[6], call);
        const int64_t T = slots.numel();
        require(c.scalar_type() == at::kBFloat16 && k.scalar_type() == at::kBFloat16 && k.is_cuda() &&
                    k.get_device() == index && c.dim() == 2 && k.dim() == 2 && c.size(0) == T && k.size(0) == T &&
                    c.size(1) == d.d_latent && k.size(1) == d.d_rope && c.stride(1) == 1 && k.stride(1) == 1 &&
                    T <= INT32_MAX,
                call, "ckv_new [T, d_c] and kr_new [T, d_R] bf16 rows, slots [T]");
        require(!pos.defined() || (pos.numel() == T && freq.defined() && 2 * freq.numel() == d.d_rope), call,
                "positions [T] and inv_freq [d_R / 2]");
        const int32_t order = layout_of(a[10], call);
        const float mscale = static_cast<float>(real(a[9], call, "mscale"));
        const Pools p = pools(a[3], a[5], d, fp8 ? at::kByte : at::kBFloat16, index, call);
        const at::Tensor scales = flat(a[4], call, "scales", at::kFloat, index, true);
        const at::Tensor *const cache[] = {&THPVariable_Unpack(a[3]), &THPVariable_Unpack(a[5]), &scales};
        for (const at::Tensor *t : cache) may_write(*t, call, "the cache");
        if (fp8) {
            require(scales.sizes() == at::IntArrayRef({p.pages, 64}), call, "scales [pages, 64]");
            check(mla_append_kv_slots_fp8(&d, c.data_ptr(), c.stride(0), k.data_ptr(), k.stride(0), ptr<int64_t>(slots),
                                          ptr<int32_t>(pos), ptr<double>(freq), mscale, order, static_cast<int32_t>(T),
                                          &p.ckv, ptr<float>(scales), &p.kr, p.pages, here.stream),
                  "mla_append_kv_slots_fp8");
        } else {
            check(mla_append_kv_slots(&d, c.data_ptr(), c.stride(0), k.data_ptr(), k.stride(0), ptr<int64_t>(slots),
                                      ptr<int32_t>(pos), ptr<double>(freq), mscale, order, static_cast<int32_t>(T),
                                      &p.ckv, &p.kr, p.pages, here.stream),
                  "mla_append_kv_slots");
        }
        for (const at::Tensor *t : cache) wrote(*t);
        Py_RETURN_NONE;
    });
}

// tree(q, ckv_pool, scales, kr_pool, block_table, seq_lens, cu_tokens, dims, max_nodes, masks,
//      num_parts, workspace, o_lat, lse_out)
PyObject *tree(PyObject *, PyObject *const *a, Py_ssize_t) {
    return guarded([&]() -> PyObject * {
        const bool fp8 = !none(a[2]);
        const char *call = fp8 ? "decode_tree_fp8" : "decode_tree";
        const int index = device_of(a[0], call, "q");
        const Place here(index);
        const mla_dims d = dims_of(a[7], call);
        const at::Tensor q = flat(a[0], call, "q", at::kBFloat16, index),
                         scales = flat(a[2], call, "scales", at::kFloat, index, true),
                         table = flat(a[4], call, "block_table", at::kInt, index),
                         lens = flat(a[5], call, "seq_lens", at::kInt, index),
                         cu = flat(a[6], call, "cu_tokens", at::kInt, index),
                         masks = flat(a[9], call, "masks", at::kInt, index, true);
        at::Tensor ws = flat(a[11], call, "workspace", at::kByte, index, true),
                   o = flat(a[12], call, "o_lat", at::kBFloat16, index, true),
                   lse = flat(a[13], call, "lse_out", at::kFloat, index, true);
        const int64_t nodes = integer(a[8], call, "max_nodes", 1, MLA_TREE_MAX_NODES);
        require(q.dim() == 3 && table.dim() == 2, call, "q [T, H, d_c + d_R], block_table [B, max_pages]");
        const int64_t T = q.size(0), H = q.size(1), B = table.size(0);
        require(T <= INT32_MAX && B < INT32_MAX && table.size(1) <= INT32_MAX && H == d.num_heads &&
                    q.size(2) == d.d_latent + d.d_rope && lens.sizes() == at::IntArrayRef({B}) &&
                    cu.sizes() == at::IntArrayRef({B + 1}) &&
                    (!masks.defined() || masks.sizes() == at::IntArrayRef({T, (nodes + 31) / 32})),
                call, "q [T, H, d_c + d_R], seq_lens [B], cu_tokens [B + 1], masks [T, ceil(max_nodes / 32)]");
        const Pools p = pools(a[1], a[3], d, fp8 ? at::kByte : at::kBFloat16, index, call);
        require(!fp8 || scales.sizes() == at::IntArrayRef({p.pages, 64}), call, "scales [pages, 64]");
        int32_t parts;
        if (none(a[10])) {
            parts = mla_tree_num_parts(&d, at::cuda::getDeviceProperties(index)->multiProcessorCount);
            if (parts == 0) throw Refused{MLA_ERR_UNSUPPORTED, call};
        } else {
            parts = static_cast<int32_t>(integer(a[10], call, "num_parts", 1, 1 << 20));
        }
        if (!ws.defined()) {
            const size_t bytes = mla_tree_workspace_bytes(&d, parts);
            if (bytes == 0) throw Refused{MLA_ERR_UNSUPPORTED, call};
            ws = empty({static_cast<int64_t>(bytes)}, at::kByte, index);
        }
        const bool new_o = !o.defined(), new_lse = !lse.defined();
        if (new_o) o = empty({T, H, d.d_latent}, at::kBFloat16, index);
        if (new_lse) lse = empty({T, H}, at::kFloat, index);
        require(o.sizes() == at::IntArrayRef({T, H, d.d_latent}) && lse.sizes() == at::IntArrayRef({T, H}), call,
                "o_lat [T, H, d_c], lse_out [T, H]");
        may_write(o, call, "o_lat");
        may_write(lse, call, "lse_out");
        const int32_t t32 = static_cast<int32_t>(T), b32 = static_cast<int32_t>(B), n32 = static_cast<int32_t>(nodes),
                      w32 = static_cast<int32_t>(table.size(1));
        check(fp8 ? mla_decode_tree_fp8(&d, q.data_ptr(), t32, &p.ckv, ptr<float>(scales), &p.kr, p.pages,
                                        ptr<int32_t>(table), w32, ptr<int32_t>(lens), ptr<int32_t>(cu), b32,
                                        ptr<uint32_t>(masks), n32, parts, ws.data_ptr(), ws.numel(), o.data_ptr(),
                                        ptr<float>(lse), here.stream)
                  : mla_decode_tree(&d, q.data_ptr(), t32, &p.ckv, &p.kr, p.pages, ptr<int32_t>(table), w32,
                                    ptr<int32_t>(lens), ptr<int32_t>(cu), b32, ptr<uint32_t>(masks), n32, parts,
                                    ws.data_ptr(), ws.numel(), o.data_ptr(), ptr<float>(lse), here.stream),
              fp8 ? "mla_decode_tree_fp8" : "mla_decode_tree");
        wrote(o);
        wrote(lse);
        return Py_BuildValue("(NN)", new_o ? wrap(o) : Py_NewRef(a[12]), new_lse ? wrap(lse) : Py_NewRef(a[13]));
    });
}

// types(MLAError, MLADims): what the calls raise, and what dims are
PyObject *types(PyObject *, PyObject *const *a, Py_ssize_t) {
    Py_XSETREF(g_error, Py_NewRef(a[0]));
    Py_XSETREF(g_dims, Py_NewRef(a[1]));
    Py_RETURN_NONE;
}

using Fast = PyObject *(*)(PyObject *, PyObject *const *, Py_ssize_t);

// The number of arguments is fixed: the callers are api.py's functions.
template <Fast F, int N>
PyObject *exactly(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments are wanted, not %zd", N, n);
        return nullptr;
    }
    return F(self, a, n);
}

template <Fast F, int N>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(static_cast<Fast>(exactly<F, N>))),
            METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<plan, 9>("plan"),     method<rotary, 10>("rotary"), method<append, 11>("append"),
                           method<tree, 14>("tree"),    method<types, 2>("types"),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_step", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step() { return PyModule_Create(&g_module); }
