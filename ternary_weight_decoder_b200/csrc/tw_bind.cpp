// tw_bind.cpp — argument marshalling of the calls that stand between kernels
// of a few microseconds (the paged cache, its attention, the residual norms):
// checks tensors, makes outputs, and calls the C entry points of
// libternary_decoder.so on the tensors' device and its current stream.  The
// entry points are handed in by init(): nothing is linked or loaded twice.
#include <Python.h>

#include <string>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ternary_decoder.h"

namespace {

struct Entries {
    decltype(&tw_kv_assign) kv_assign;
    decltype(&tw_rope_append) rope_append;
    decltype(&tw_paged_attention) paged_attention;
    decltype(&tw_paged_attention_workspace_bytes) paged_attention_workspace_bytes;
    decltype(&tw_residual_norm) residual_norm;
    decltype(&tw_last_error) last_error;
} entry;
PyObject *status_error = nullptr;   // TernaryError(status, message)

// A refused argument; `raised`: the Python error is set already.
struct Refused {
    PyObject *type = nullptr;
    std::string what;
};

[[noreturn]] void type_error(const std::string &s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string &s) { throw Refused{PyExc_ValueError, s}; }

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int64_t device_of(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        value_error(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o).get_device();
}

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i)
        t += (i ? ", " : "") + (s[i] < 0 ? std::string("any") : std::to_string(s[i]));
    return t + "]";
}

// Type, device and shape (-1: any size) of a tensor.
const at::Tensor &checked(PyObject *o, at::ScalarType type, at::IntArrayRef shape, const char *name, int64_t index)
{
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be a tensor of " + c10::toString(type));
    if (!t.is_cuda() || t.get_device() != index)
        value_error(std::string(name) + " must be on cuda:" + std::to_string(index) + ", is on " + t.device().str());
    bool same = (size_t)t.dim() == shape.size();
    for (size_t i = 0; same && i < shape.size(); ++i)
        same = shape[i] < 0 || t.size(i) == shape[i];
    if (!same)
        value_error(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    return t;
}

const at::Tensor &dense(PyObject *o, at::ScalarType type, at::IntArrayRef shape, const char *name, int64_t index)
{
    const at::Tensor &t = checked(o, type, shape, name, index);
    if (!t.is_contiguous())
        value_error(std::string(name) + " must be contiguous");
    return t;
}

// The same where None stands for no tensor: its address, or null.
template <class T>
T *dense_or_null(PyObject *o, at::ScalarType type, at::IntArrayRef shape, const char *name, int64_t index)
{
    return o == Py_None ? nullptr : static_cast<T *>(dense(o, type, shape, name, index).data_ptr());
}

// An fp32 matrix with contiguous rows, and its row stride.
struct Rows {
    float *p = nullptr;
    int64_t ld = 0;
};

Rows rows(PyObject *o, int64_t n, int64_t width, const char *name, int64_t index)
{
    const at::Tensor &t = checked(o, at::kFloat, {n, width}, name, index);
    if (width > 1 && t.stride(1) != 1)
        value_error(std::string(name) + " must have contiguous rows");
    // one row has no stride of its own
    return Rows{t.data_ptr<float>(), n > 1 ? t.stride(0) : (width + 3) / 4 * 4};
}

void matrix(const at::Tensor &t, const char *name)
{
    if (t.dim() != 2)
        value_error(std::string(name) + " must have two dimensions, has " + std::to_string(t.dim()));
}

struct Table {
    int32_t *p;
    int64_t pages, stride;
};

Table table(PyObject *o, int64_t requests, int64_t index)
{
    const at::Tensor &t = checked(o, at::kInt, {requests, -1}, "block_table", index);
    const int64_t pages = t.size(1);
    if (pages > 1 && t.stride(1) != 1)
        value_error("block_table must have contiguous rows");
    return Table{t.data_ptr<int32_t>(), pages, requests > 1 ? t.stride(0) : pages};
}

int64_t integer(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be an integer");
    }
    return v;
}

float real(PyObject *o, const char *name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be a number");
    }
    return (float)v;
}

bool truth(PyObject *o)
{
    const int is = PyObject_IsTrue(o);
    if (is < 0)
        throw Refused{};   // (the object's own error)
    return is;
}

// Outputs are made below the dispatcher, and parts of one buffer below the
// tracking of views (the parts do not overlap and each is an output of its
// own): kv_assign took 8.9 us with both, 7.2 without.
at::Tensor make(at::IntArrayRef size, at::ScalarType type, const at::Tensor &beside)
{
    return at::Tensor(at::detail::empty_cuda(size, type, beside.device(), std::nullopt));
}

// Device `index`, made current for the call, and its current stream.
struct Place {
    c10::cuda::OptionalCUDAGuard guard;
    tw_stream_t stream;
    explicit Place(int64_t index)
    {
        if (c10::cuda::current_device() != index)
            guard.set_index((c10::DeviceIndex)index);
        stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    }
};

void raise_on(int status)
{
    if (status == TW_OK)
        return;
    PyObject *e = PyObject_CallFunction(status_error, "is", status, entry.last_error());
    if (e) {
        PyErr_SetObject(status_error, e);
        Py_DECREF(e);
    }
    throw Refused{};
}

PyObject *wrap_or_none(const at::Tensor &t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

// The given tensor, or a new one.
at::Tensor given_or(PyObject *o, const at::Tensor &made) { return o == Py_None ? made : THPVariable_Unpack(o); }

template <class F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F body)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused &r) {
        if (r.type)
            PyErr_SetString(r.type, r.what.c_str());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// kv_assign(lengths, delta, block_table, free_pages, free_count, page_size, rows, lengths_out, free_count_out)
PyObject *kv_assign(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    return guarded(n_args, 9, [&]() -> PyObject * {
        const int64_t index = device_of(a[0], "lengths");
        const at::Tensor &lengths = dense(a[0], at::kInt, {-1}, "lengths", index);
        const int64_t n = lengths.size(0), page_size = integer(a[5], "page_size"), count = integer(a[6], "rows");
        const at::Tensor &delta = dense(a[1], at::kInt, {n}, "delta", index);
        const Table t = table(a[2], n, index);
        const at::Tensor &free_pages = dense(a[3], at::kInt, {-1}, "free_pages", index);
        const at::Tensor &free_count = dense(a[4], at::kInt, {1}, "free_count", index);
        if (count < 0 || count > INT32_MAX)
            value_error("rows must be in 0 .. 2^31 - 1");
        int32_t *lengths_out = dense_or_null<int32_t>(a[7], at::kInt, {n}, "lengths_out", index);
        int32_t *count_out = dense_or_null<int32_t>(a[8], at::kInt, {1}, "free_count_out", index);
        Place place(index);
        // slots, positions and requests of the rows, row starts, lengths, free count
        at::Tensor made = make({3 * count + 2 * n + 2}, at::kInt, lengths);
        int32_t *p = made.data_ptr<int32_t>(), *starts = p + 3 * count, *own = starts + n + 1;
        raise_on(entry.kv_assign(lengths.data_ptr<int32_t>(), delta.data_ptr<int32_t>(), n, page_size, t.p, t.pages,
                                 t.stride, free_pages.data_ptr<int32_t>(), free_pages.size(0),
                                 free_count.data_ptr<int32_t>(), lengths_out ? lengths_out : own,
                                 count_out ? count_out : own + n, p, p + count, p + 2 * count, count, starts,
                                 place.stream));
        at::AutoDispatchBelowADInplaceOrView no_views;
        auto part = [&](int64_t at, int64_t size) { return made.as_strided({size}, {1}, at); };
        const int64_t s = 3 * count;
        return Py_BuildValue("(NNNNNN)", THPVariable_Wrap(lengths_out ? given_or(a[7], made) : part(s + n + 1, n)),
                             THPVariable_Wrap(count_out ? given_or(a[8], made) : part(s + 2 * n + 1, 1)),
                             THPVariable_Wrap(part(0, count)), THPVariable_Wrap(part(count, count)),
                             THPVariable_Wrap(part(2 * count, count)), THPVariable_Wrap(part(s, n + 1)));
    });
}

// The cache handle: address of its struct, and its device.
const tw_kv_cache *cache_of(PyObject *address, PyObject *device, int64_t index)
{
    if (integer(device, "cache device") != index)
        value_error("the cache must be on cuda:" + std::to_string(index));
    return static_cast<const tw_kv_cache *>(PyLong_AsVoidPtr(address));
}

int64_t heads_of(int64_t width, const tw_kv_cache *cache)
{
    if (width % cache->head_dim)
        value_error("q has " + std::to_string(width) + " columns, not whole heads of " +
                    std::to_string(cache->head_dim));
    return width / cache->head_dim;
}

// rope_append(q, k, v, positions, slots, cache, device, inv_freq, interleaved, q_out)
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    return guarded(n_args, 10, [&]() -> PyObject * {
        const int64_t index = device_of(a[0], "q");
        const at::Tensor &q = THPVariable_Unpack(a[0]);
        matrix(q, "q");
        const tw_kv_cache *cache = cache_of(a[5], a[6], index);
        const int64_t n = q.size(0), width = q.size(1), heads = heads_of(width, cache);
        const int64_t wide = cache->kv_heads * cache->head_dim;
        const Rows qr = rows(a[0], n, width, "q", index), kr = rows(a[1], n, wide, "k", index);
        const Rows vr = rows(a[2], n, wide, "v", index);
        const at::Tensor &positions = dense(a[3], at::kInt, {n}, "positions", index);
        const at::Tensor &slots = dense(a[4], at::kInt, {n}, "slots", index);
        const double *freq = dense_or_null<double>(a[7], at::kDouble, {-1}, "inv_freq", index);
        const int64_t rotary = a[7] == Py_None ? 0 : 2 * THPVariable_Unpack(a[7]).size(0);
        const bool interleaved = truth(a[8]);
        Rows to;
        if (a[9] != Py_None)
            to = rows(a[9], n, width, "q_out", index);
        Place place(index);
        at::Tensor made;
        if (!to.p && a[9] == Py_None) {
            made = make({n, width}, at::kFloat, q);
            to = Rows{made.data_ptr<float>(), width};
        }
        raise_on(entry.rope_append(qr.p, qr.ld, kr.p, kr.ld, vr.p, vr.ld, n, heads, rotary, freq,
                                   interleaved, positions.data_ptr<int32_t>(), slots.data_ptr<int32_t>(),
                                   cache, to.p, to.ld, place.stream));
        return THPVariable_Wrap(given_or(a[9], made));
    });
}

// paged_attention(q, cache, device, block_table, lengths, first, scale, out, lse, ws, return_lse)
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    return guarded(n_args, 11, [&]() -> PyObject * {
        const int64_t index = device_of(a[0], "q");
        const at::Tensor &q = THPVariable_Unpack(a[0]);
        matrix(q, "q");
        const tw_kv_cache *cache = cache_of(a[1], a[2], index);
        const int64_t n = q.size(0), width = q.size(1), heads = heads_of(width, cache);
        const Rows qr = rows(a[0], n, width, "q", index);
        const Table t = table(a[3], n, index);
        const at::Tensor &lengths = dense(a[4], at::kInt, {n}, "lengths", index);
        const int32_t *first = dense_or_null<int32_t>(a[5], at::kInt, {n}, "first", index);
        const float scale = real(a[6], "scale");
        Rows to;
        if (a[7] != Py_None)
            to = rows(a[7], n, width, "out", index);
        float *lse = dense_or_null<float>(a[8], at::kFloat, {n, heads}, "lse", index);
        const bool want_lse = truth(a[10]);
        if (a[9] != Py_None)
            dense(a[9], at::kByte, {-1}, "ws", index);
        Place place(index);
        at::Tensor out, sums, ws;
        if (a[7] == Py_None) {
            out = make({n, width}, at::kFloat, q);
            to = Rows{out.data_ptr<float>(), width};
        }
        if (want_lse && a[8] == Py_None) {
            sums = make({n, heads}, at::kFloat, q);
            lse = sums.data_ptr<float>();
        }
        if (a[9] == Py_None)
            ws = at::zeros({(int64_t)entry.paged_attention_workspace_bytes(n, heads, cache->kv_heads, cache->head_dim)},
                           q.options().dtype(at::kByte));
        const at::Tensor &scratch = a[9] == Py_None ? ws : THPVariable_Unpack(a[9]);
        raise_on(entry.paged_attention(qr.p, qr.ld, n, heads, cache, t.p, t.pages, t.stride,
                                       lengths.data_ptr<int32_t>(), first, scale, to.p, to.ld, lse,
                                       scratch.data_ptr(), (size_t)scratch.numel(), place.stream));
        if (!want_lse)
            return THPVariable_Wrap(given_or(a[7], out));
        return Py_BuildValue("(NN)", THPVariable_Wrap(given_or(a[7], out)), THPVariable_Wrap(given_or(a[8], sums)));
    });
}

// residual_norm(x, y, post, post_weight, post_bias, gate, alpha, pre, pre_weight, pre_bias, eps, h, n, quantize)
PyObject *residual_norm(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    return guarded(n_args, 14, [&]() -> PyObject * {
        const int64_t index = device_of(a[0], "x");
        const at::Tensor &x = THPVariable_Unpack(a[0]);
        matrix(x, "x");
        const int64_t M = x.size(0), K = x.size(1);
        const bool quantize = truth(a[13]);
        tw_residual_norm_args g{};
        g.M = M, g.K = K;
        auto take = [&](PyObject *o, const char *name, auto &p, int64_t &ld) {
            if (o == Py_None)
                return;
            const Rows r = rows(o, M, K, name, index);
            p = r.p, ld = r.ld;
        };
        take(a[0], "x", g.x, g.ldx);
        take(a[1], "y", g.y, g.ldy);
        g.post = (int32_t)integer(a[2], "post"), g.pre = (int32_t)integer(a[7], "pre");
        g.post_weight = dense_or_null<float>(a[3], at::kFloat, {K}, "post_weight", index);
        g.post_bias = dense_or_null<float>(a[4], at::kFloat, {K}, "post_bias", index);
        if (a[5] != Py_None && tensor(a[5], "gate").dim() == 1)
            g.gate = dense_or_null<float>(a[5], at::kFloat, {K}, "gate", index);
        else
            take(a[5], "gate", g.gate, g.ldgate);
        g.alpha = real(a[6], "alpha");
        g.pre_weight = dense_or_null<float>(a[8], at::kFloat, {K}, "pre_weight", index);
        g.pre_bias = dense_or_null<float>(a[9], at::kFloat, {K}, "pre_bias", index);
        g.eps = real(a[10], "eps");
        take(a[11], "h", g.h, g.ldh);
        take(a[12], "n", g.n, g.ldn);
        if (quantize && a[12] != Py_None)
            value_error("quantize gives codes: n cannot be passed in");
        Place place(index);
        at::Tensor h, n, xq, amax, qsum;
        if (a[11] == Py_None && a[1] != Py_None) {   // (neither: h is x as it stands)
            h = make({M, K}, at::kFloat, x);
            g.h = h.data_ptr<float>(), g.ldh = K;
        }
        if (quantize) {
            xq = make({M, K}, at::kChar, x), amax = make({M}, at::kFloat, x), qsum = make({M}, at::kInt, x);
            g.xq = xq.data_ptr<int8_t>(), g.amax = amax.data_ptr<float>(), g.qsum = qsum.data_ptr<int32_t>();
        } else if (a[12] == Py_None && g.pre != TW_NORM_NONE) {
            n = make({M, K}, at::kFloat, x);
            g.n = n.data_ptr<float>(), g.ldn = K;
        } else if (a[12] == Py_None && a[11] == Py_None && a[1] == Py_None) {
            value_error("nothing to compute: no y, no norm and no codes");
        }
        raise_on(entry.residual_norm(&g, place.stream));
        auto given = [](PyObject *o, const at::Tensor &made) {
            return o == Py_None ? wrap_or_none(made) : Py_NewRef(o);
        };
        return Py_BuildValue("(NNNNN)", a[11] == Py_None && !h.defined() ? Py_NewRef(a[0]) : given(a[11], h),
                             given(a[12], n), wrap_or_none(xq), wrap_or_none(amax), wrap_or_none(qsum));
    });
}

// init(error class, addresses of the entry points in the order of Entries)
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    return guarded(n_args, 7, [&]() -> PyObject * {
        void *p[6];
        for (int i = 0; i < 6; ++i) {
            p[i] = PyLong_AsVoidPtr(a[i + 1]);
            if (!p[i])
                value_error("an entry point is missing");
        }
        Py_XSETREF(status_error, Py_NewRef(a[0]));
        entry.kv_assign = reinterpret_cast<decltype(entry.kv_assign)>(p[0]);
        entry.rope_append = reinterpret_cast<decltype(entry.rope_append)>(p[1]);
        entry.paged_attention = reinterpret_cast<decltype(entry.paged_attention)>(p[2]);
        entry.paged_attention_workspace_bytes =
            reinterpret_cast<decltype(entry.paged_attention_workspace_bytes)>(p[3]);
        entry.residual_norm = reinterpret_cast<decltype(entry.residual_norm)>(p[4]);
        entry.last_error = reinterpret_cast<decltype(entry.last_error)>(p[5]);
        Py_RETURN_NONE;
    });
}

#define TW_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TW_METHOD(init),          TW_METHOD(kv_assign), TW_METHOD(rope_append), TW_METHOD(paged_attention),
                         TW_METHOD(residual_norm), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Argument marshalling of libternary_decoder.so.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
