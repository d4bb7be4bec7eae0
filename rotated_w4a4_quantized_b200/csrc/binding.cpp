// binding.cpp -- the decoding calls' common case in native code (extension
// module _decoding of the package).
//
// A decoding step makes these calls once a layer, and their kernels take a few
// microseconds; the checks, allocations and argument conversions of a ctypes
// call take more than that.  Each function here makes a call of the C ABI with
// results and workspace of its own on the current stream of the operands'
// device.  It returns the result, a status of the C ABI as an int where that
// is not CONVROT_OK, or None where an argument is not plainly right (another
// type, device, layout or shape): the package's Python code then says what is
// wrong, or handles what is unusual.
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/convrot_kv4.h"
#include "../../include/convrot_w4g.h"

namespace {

using at::Tensor;

// `o` as a dense tensor of `dtype` on CUDA device `index` (any device: -1,
// which is then set), or nullptr.
const Tensor *dense(PyObject *o, at::ScalarType dtype, int64_t dim, int &index) {
    if (!THPVariable_Check(o)) return nullptr;
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != dtype || t.dim() != dim || !t.is_contiguous()) return nullptr;
    if (index < 0) index = t.get_device();
    return t.get_device() == index ? &t : nullptr;
}

// bf16 [T][heads][D], dense within a token; `ld` gets the values between tokens.
const Tensor *tokens(PyObject *o, int64_t heads, int64_t D, int index, int64_t &ld) {
    if (!THPVariable_Check(o)) return nullptr;
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.size(2) != D || (heads >= 0 && t.size(1) != heads) ||
        t.get_device() != index || t.size(0) == 0 || t.size(1) == 0)
        return nullptr;
    const int64_t row = t.size(1) * D;
    if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != D) || (t.size(0) > 1 && t.stride(0) < row)) return nullptr;
    ld = t.size(0) > 1 ? t.stride(0) : row;
    return &t;
}

bool whole(PyObject *o, int64_t &v) {
    if (!PyLong_CheckExact(o)) return false;
    int overflow = 0;
    v = PyLong_AsLongLongAndOverflow(o, &overflow);
    return !overflow && v >= 0 && v < (int64_t(1) << 31);
}

bool current(int index) { return c10::cuda::current_device() == index; }

convrot_stream_t stream_of(int index) {
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
}

Tensor empty(at::IntArrayRef size, at::ScalarType dtype, int index) {
    return at::detail::empty_cuda(size, dtype, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index)), std::nullopt);
}

// `count` values at `at` bytes of a buffer, as a tensor of its own (a dispatched
// view costs as much as an allocation).
Tensor part(const Tensor &buffer, int64_t at, at::ScalarType dtype, int64_t count) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buffer.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                        c10::scalarTypeToTypeMeta(dtype));
    t.unsafeGetTensorImpl()->set_storage_offset(at / static_cast<int64_t>(c10::elementSize(dtype)));
    t.unsafeGetTensorImpl()->set_sizes_contiguous({count});
    return t;
}

PyObject *status(convrot_status st) { return PyLong_FromLong(st); }

// A function's body.  Where memory runs out the Python code makes the call
// again, and its error.
template <class F>
PyObject *guarded(F body) {
    try {
        return body();
    } catch (const c10::OutOfMemoryError &) {
        Py_RETURN_NONE;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

struct CacheArg {
    convrot_kv4_cache c;
    int index;
};

// (k_codes, k_scales, v_codes, v_scales) and the rotation group.
bool cache_of(PyObject *o, PyObject *group, CacheArg &a) {
    int64_t g;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4 || !whole(group, g)) return false;
    a.index = -1;
    const Tensor *kc = dense(PyTuple_GET_ITEM(o, 0), at::kByte, 4, a.index);
    const Tensor *ks = kc ? dense(PyTuple_GET_ITEM(o, 1), at::kBFloat16, 3, a.index) : nullptr;
    const Tensor *vc = ks ? dense(PyTuple_GET_ITEM(o, 2), at::kByte, 4, a.index) : nullptr;
    const Tensor *vs = vc ? dense(PyTuple_GET_ITEM(o, 3), at::kBFloat16, 3, a.index) : nullptr;
    if (!vs || vc->sizes() != kc->sizes() || ks->sizes() != kc->sizes().slice(0, 3) || vs->sizes() != ks->sizes()) return false;
    for (int64_t i = 1; i < 4; ++i)
        if (kc->size(i) > 65536) return false;
    a.c = convrot_kv4_cache{static_cast<uint8_t *>(kc->data_ptr()), ks->data_ptr(), static_cast<uint8_t *>(vc->data_ptr()),
                            vs->data_ptr(), kc->size(0), static_cast<int>(kc->size(1)), static_cast<int>(kc->size(2)),
                            static_cast<int>(2 * kc->size(3)), static_cast<int>(g)};
    return current(a.index);
}

// x, qw, sg, bias, group, scale_group -> y
PyObject *w4g_linear(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        int index = -1;
        int64_t group, sgroup;
        if (n != 6 || !whole(args[4], group) || !whole(args[5], sgroup) || sgroup == 0) Py_RETURN_NONE;
        const Tensor *x = dense(args[0], at::kBFloat16, 2, index);
        const Tensor *qw = x ? dense(args[1], at::kByte, 2, index) : nullptr;
        const Tensor *sg = qw ? dense(args[2], at::kBFloat16, 2, index) : nullptr;
        if (!sg) Py_RETURN_NONE;
        const int64_t M = x->size(0), K = x->size(1), N = qw->size(0);
        const Tensor *bias = nullptr;
        if (args[3] != Py_None && (!(bias = dense(args[3], at::kBFloat16, 1, index)) || bias->size(0) != N)) Py_RETURN_NONE;
        if (2 * qw->size(1) != K || sg->size(0) != N || sg->size(1) != K / sgroup || !current(index)) Py_RETURN_NONE;
        const size_t need = convrot_w4g_workspace_size(M, K);
        Tensor workspace;
        if (need) workspace = empty({static_cast<int64_t>(need)}, at::kByte, index);
        Tensor y = empty({M, N}, at::kBFloat16, index);
        const convrot_status st = convrot_w4g_linear(
            x->data_ptr(), static_cast<const uint8_t *>(qw->data_ptr()), sg->data_ptr(), bias ? bias->data_ptr() : nullptr, M, N,
            K, static_cast<int>(group), static_cast<int>(sgroup), need ? workspace.data_ptr() : nullptr, need, y.data_ptr(),
            stream_of(index));
        return st == CONVROT_OK ? THPVariable_Wrap(y) : status(st);
    });
}

// cached, new_tokens, block_table, free_pages, free_count, page, max_tokens ->
// (seq_lens, cu_q, slots, positions, result, its first value)
PyObject *kv4_plan(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        int index = -1;
        int64_t page, most;
        if (n != 7 || !whole(args[5], page) || !whole(args[6], most)) Py_RETURN_NONE;
        const Tensor *cached = dense(args[0], at::kInt, 1, index);
        const Tensor *fresh = cached ? dense(args[1], at::kInt, 1, index) : nullptr;
        const Tensor *table = fresh ? dense(args[2], at::kInt, 2, index) : nullptr;
        const Tensor *pages = table ? dense(args[3], at::kInt, 1, index) : nullptr;
        const Tensor *count = pages ? dense(args[4], at::kInt, 1, index) : nullptr;
        if (!count) Py_RETURN_NONE;
        const int64_t B = cached->size(0);
        if (reinterpret_cast<uintptr_t>(cached->data_ptr()) % 16) Py_RETURN_NONE;   // taken as a copy
        if (fresh->size(0) != B || table->size(0) != B || count->size(0) != 1 || !current(index)) Py_RETURN_NONE;
        // the results in one buffer, each on 256 bytes
        auto room = [](int64_t bytes) { return (bytes + 255) & ~int64_t(255); };
        const int64_t at_cu = room(4 * B), at_slots = at_cu + room(4 * (B + 1)), at_positions = at_slots + room(8 * most),
                      at_result = at_positions + room(4 * most);
        const Tensor buffer = empty({at_result + 16}, at::kByte, index);
        const Tensor lens = part(buffer, 0, at::kInt, B), cu_q = part(buffer, at_cu, at::kInt, B + 1),
                     slots = part(buffer, at_slots, at::kLong, most), positions = part(buffer, at_positions, at::kInt, most),
                     result = part(buffer, at_result, at::kInt, 4);
        auto p = [](const Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); };
        const convrot_status st = convrot_kv4_plan(p(*cached), p(*fresh), B, static_cast<int>(page), p(*table), table->size(1),
                                                   p(*pages), pages->size(0), p(*count), most, p(lens), p(cu_q),
                                                   static_cast<int64_t *>(slots.data_ptr()), p(positions), p(result), stream_of(index));
        if (st != CONVROT_OK) return status(st);
        const Tensor left = part(buffer, at_result, at::kInt, 1);
        return Py_BuildValue("(NNNNNN)", THPVariable_Wrap(lens), THPVariable_Wrap(cu_q), THPVariable_Wrap(slots),
                             THPVariable_Wrap(positions), THPVariable_Wrap(result), THPVariable_Wrap(left));
    });
}

// k, v, cache, slots, group -> 0
PyObject *kv4_append(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        CacheArg a;
        int64_t ldk, ldv;
        if (n != 5 || !cache_of(args[2], args[4], a)) Py_RETURN_NONE;
        const Tensor *k = tokens(args[0], a.c.kv_heads, a.c.head_dim, a.index, ldk);
        const Tensor *v = k ? tokens(args[1], a.c.kv_heads, a.c.head_dim, a.index, ldv) : nullptr;
        const Tensor *slots = v ? dense(args[3], at::kLong, 1, a.index) : nullptr;
        if (!slots || v->size(0) != k->size(0) || slots->size(0) != k->size(0)) Py_RETURN_NONE;
        return status(convrot_kv4_append(&a.c, k->data_ptr(), ldk, v->data_ptr(), ldv,
                                         static_cast<const int64_t *>(slots->data_ptr()), k->size(0), stream_of(a.index)));
    });
}

// cache, slots, group -> (k, v)
PyObject *kv4_read(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        CacheArg a;
        if (n != 3 || !cache_of(args[0], args[2], a)) Py_RETURN_NONE;
        const Tensor *slots = dense(args[1], at::kLong, 1, a.index);
        if (!slots) Py_RETURN_NONE;
        const int64_t T = slots->size(0);
        Tensor k = empty({T, a.c.kv_heads, a.c.head_dim}, at::kBFloat16, a.index), v = empty(k.sizes(), at::kBFloat16, a.index);
        const convrot_status st = convrot_kv4_read(&a.c, static_cast<const int64_t *>(slots->data_ptr()), T, k.data_ptr(),
                                                   v.data_ptr(), stream_of(a.index));
        return st == CONVROT_OK ? Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v)) : status(st);
    });
}

// q, cache, block_table, seq_lens, cu_q, scale, group -> out
PyObject *kv4_attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        CacheArg a;
        int64_t ldq;
        if (n != 7 || !cache_of(args[1], args[6], a) || !PyFloat_CheckExact(args[5])) Py_RETURN_NONE;
        const Tensor *q = tokens(args[0], -1, a.c.head_dim, a.index, ldq);
        const Tensor *table = q ? dense(args[2], at::kInt, 2, a.index) : nullptr;
        const Tensor *lens = table ? dense(args[3], at::kInt, 1, a.index) : nullptr;
        const Tensor *cu_q = lens ? dense(args[4], at::kInt, 1, a.index) : nullptr;
        if (!cu_q) Py_RETURN_NONE;
        const int64_t T = q->size(0), B = lens->size(0), heads = q->size(1);
        if (table->size(0) != B || cu_q->size(0) != B + 1 || heads > 65536) Py_RETURN_NONE;
        const size_t need = convrot_kv4_attention_workspace_size(T, B, static_cast<int>(heads), a.c.kv_heads, a.c.head_dim,
                                                                 table->size(1) * a.c.page);
        Tensor workspace = empty({static_cast<int64_t>(need ? need : 1)}, at::kByte, a.index);
        Tensor out = empty({T, heads, a.c.head_dim}, at::kBFloat16, a.index);
        auto p = [](const Tensor *t) { return static_cast<const int32_t *>(t->data_ptr()); };
        const convrot_status st = convrot_kv4_attention(
            &a.c, q->data_ptr(), ldq, T, static_cast<int>(heads), p(table), table->size(1), p(lens), p(cu_q), B,
            static_cast<float>(PyFloat_AS_DOUBLE(args[5])), workspace.data_ptr(), need, out.data_ptr(), stream_of(a.index));
        return st == CONVROT_OK ? THPVariable_Wrap(out) : status(st);
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"w4g_linear", fast<w4g_linear>(), METH_FASTCALL, nullptr},
    {"kv4_plan", fast<kv4_plan>(), METH_FASTCALL, nullptr},
    {"kv4_append", fast<kv4_append>(), METH_FASTCALL, nullptr},
    {"kv4_read", fast<kv4_read>(), METH_FASTCALL, nullptr},
    {"kv4_attention", fast<kv4_attention>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decoding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decoding() { return PyModule_Create(&module); }
