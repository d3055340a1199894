// The speculative-decoding calls of binding.py on torch tensors: checks of
// types, shapes and devices, allocation of results, and the call into
// libgpt2.so on the current stream.  Argument marshalling only, compiled
// because it is most of a small call's time: for the attention of one
// sequence's tree the checks and allocations took 8 us in Python and take 1 us
// here, next to 8 us on the GPU.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <sstream>

#include "../../include/gpt2.h"

namespace {

PyObject *g_error = nullptr;   // binding.GPT2Error

// The library's functions, from the copy that the binding has loaded.
struct {
    decltype(&gpt2_op_kv_store) kv_store;
    decltype(&gpt2_op_kv_load) kv_load;
    decltype(&gpt2_op_kv_commit) kv_commit;
    decltype(&gpt2_op_tree_attention_workspace) tree_attention_workspace;
    decltype(&gpt2_op_tree_attention) tree_attention;
    decltype(&gpt2_op_verify_tree_workspace) verify_tree_workspace;
    decltype(&gpt2_op_verify_tree) verify_tree;
} g_lib;

struct Bad {                   // a ValueError
    std::string what;
};

std::string describe(const at::Tensor &t)
{
    std::ostringstream s;
    s << t.scalar_type() << " " << t.sizes() << " on " << t.device();
    return s.str();
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) throw Bad{std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}

// A contiguous tensor of this type and shape on the current device.
void *whole(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, int dev)
{
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous() || !t.is_cuda() || t.get_device() != dev) {
        std::ostringstream s;
        s << name << " must be a contiguous " << type << " tensor of shape " << shape
          << " on the current device cuda:" << dev << ", not " << describe(t);
        throw Bad{s.str()};
    }
    return t.data_ptr();
}

template <typename T>
T *whole(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int dev)
{
    return static_cast<T *>(whole(tensor(o, name), name, type, shape, dev));
}

int row_type(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return GPT2_F32;
    case at::kHalf: return GPT2_F16;
    case at::kBFloat16: return GPT2_BF16;
    default: return -1;
    }
}

int64_t one_dim(const at::Tensor &t) { return t.dim() == 1 ? t.size(0) : -1; }

struct Cache {
    gpt2_kv kv{};
    int layers = 1;
    at::TensorOptions options;

    // [slots][heads][positions][head_dim], or with layers before
    Cache(PyObject *ko, PyObject *vo, PyObject *kso, PyObject *vso, int dev, bool many = false)
    {
        const at::Tensor &k = tensor(ko, "k_cache");
        const int64_t nd = k.dim();
        if (nd != 4 && !(many && nd == 5)) {
            std::ostringstream s;
            s << "a cache is [slots][heads][positions][head_dim], not " << k.sizes();
            throw Bad{s.str()};
        }
        kv.dtype = row_type(k.scalar_type());
        if (k.scalar_type() == at::kChar) kv.dtype = GPT2_INT8;
        if (k.scalar_type() == at::kFloat8_e4m3fn) kv.dtype = GPT2_E4M3;
        if (kv.dtype < 0) throw Bad{"unsupported cache type: " + describe(k)};
        kv.k = whole(k, "k_cache", k.scalar_type(), k.sizes(), dev);
        kv.v = whole<void>(vo, "v_cache", k.scalar_type(), k.sizes(), dev);
        if (kv.dtype >= GPT2_INT8) {
            if (kso == Py_None || vso == Py_None) throw Bad{"an 8-bit cache needs k_scale and v_scale"};
            kv.k_scale = whole<float>(kso, "k_scale", at::kFloat, k.sizes().slice(0, nd - 1), dev);
            kv.v_scale = whole<float>(vso, "v_scale", at::kFloat, k.sizes().slice(0, nd - 1), dev);
        } else if (kso != Py_None || vso != Py_None) {
            throw Bad{"only an 8-bit cache has scales"};
        }
        for (int64_t i = 0; i < nd; ++i)
            if (k.size(i) >= (int64_t(1) << 31)) throw Bad{"a cache dimension is too large"};
        layers = nd == 5 ? int(k.size(0)) : 1;
        kv.n_slots = int(k.size(nd - 4));
        kv.n_head = int(k.size(nd - 3));
        kv.n_positions = int(k.size(nd - 2));
        kv.head_dim = int(k.size(nd - 1));
        options = k.options();
    }
};

// The row stride of a [rows][H][D] tensor whose rows are contiguous.
int64_t row_stride(const at::Tensor &t, const char *name, int64_t H, int64_t D, int dev)
{
    if (t.dim() != 3 || t.size(1) != H || t.size(2) != D) {
        std::ostringstream s;
        s << name << " must be [rows][" << H << "][" << D << "], not " << t.sizes();
        throw Bad{s.str()};
    }
    if (row_type(t.scalar_type()) < 0 || !t.is_cuda() || t.get_device() != dev)
        throw Bad{std::string(name) + " must be float32, float16 or bfloat16 on the current device, not " + describe(t)};
    if (t.stride(2) != 1 || (H > 1 && t.stride(1) != D))
        throw Bad{std::string("the heads of a row of ") + name + " must be contiguous"};
    if (t.size(0) >= (int64_t(1) << 31)) throw Bad{std::string("too many rows of ") + name};
    return t.size(0) > 1 ? t.stride(0) : H * D;
}

// A tensor of this shape in `whole`'s memory, from element `from` on: results of
// one call are made in one allocation (1.3 us each on the Arm host, as long as
// the marshalling itself).
at::Tensor part(const at::Tensor &whole, int64_t from, at::IntArrayRef shape)
{
    auto t = c10::make_intrusive<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), whole.dtype());
    t->set_sizes_contiguous(shape);
    t->set_storage_offset(from);
    return at::Tensor(std::move(t));
}

// Memory of a call in flight, returned to torch's allocator when the call has
// been queued: what takes it next on this stream runs after it.
c10::DataPtr scratch(size_t bytes) { return c10::cuda::CUDACachingAllocator::get()->allocate(bytes); }

int32_t to_int(PyObject *o, const char *name)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Bad{std::string(name) + " must be an integer"};
    }
    if (v < INT32_MIN || v > INT32_MAX) throw Bad{std::string(name) + " is too large"};
    return int32_t(v);
}

float to_float(PyObject *o, const char *name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Bad{std::string(name) + " must be a number"};
    }
    return float(v);
}

struct Failed {                // a GPT2Error
    int status;
    const char *what;
};

void check(int status, const char *what)
{
    if (status != GPT2_OK) throw Failed{status, what};
}

struct Call {
    int dev = c10::cuda::current_device();
    void *stream = c10::cuda::getCurrentCUDAStream(dev).stream();
};

// Runs f with the number of arguments checked and every C++ exception turned
// into a Python one.
template <typename F>
PyObject *guarded(const char *name, Py_ssize_t want, Py_ssize_t got, F f)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, want);
        return nullptr;
    }
    try {
        return f();
    } catch (const Bad &e) {
        PyErr_SetString(PyExc_ValueError, e.what.c_str());
    } catch (const Failed &e) {
        PyObject *x = PyObject_CallFunction(g_error, "is", e.status, e.what);
        if (x) {
            PyErr_SetObject(g_error, x);
            Py_DECREF(x);
        }
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// The caller's workspace, or one of `need` bytes.
struct Workspace {
    void *p = nullptr;
    size_t bytes = 0;
    c10::DataPtr own;
    Workspace(PyObject *o, size_t need, int dev)
    {
        if (o != Py_None) {
            const at::Tensor &t = tensor(o, "workspace");
            if (!t.is_contiguous() || !t.is_cuda() || t.get_device() != dev)
                throw Bad{"workspace must be contiguous and on the current device"};
            p = t.data_ptr();
            bytes = t.nbytes();
        } else if (need) {
            own = scratch(need);
            p = own.get();
            bytes = need;
        }
    }
};

// k, v, k_cache, v_cache, slot, pos, k_scale, v_scale
PyObject *kv_store(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("kv_store", 8, n, [&]() -> PyObject * {
        const Call c;
        const Cache cache(a[2], a[3], a[6], a[7], c.dev);
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        const int64_t H = cache.kv.n_head, D = cache.kv.head_dim, stride = row_stride(k, "k", H, D, c.dev);
        if (v.scalar_type() != k.scalar_type() || v.sizes() != k.sizes() || row_stride(v, "v", H, D, c.dev) != stride)
            throw Bad{"k and v must have the same type, shape and row stride"};
        const int64_t rows = k.size(0);
        const int32_t *slot = whole<int32_t>(a[4], "slot", at::kInt, {rows}, c.dev);
        const int32_t *pos = whole<int32_t>(a[5], "pos", at::kInt, {rows}, c.dev);
        if (rows > 0)
            check(g_lib.kv_store(&cache.kv, k.data_ptr(), v.data_ptr(), row_type(k.scalar_type()), stride, slot, pos,
                                   int32_t(rows), c.stream),
                  "gpt2_op_kv_store");
        Py_RETURN_NONE;
    });
}

// k_cache, v_cache, slot, pos, k_scale, v_scale, dtype (a torch dtype or None), k, v
PyObject *kv_load(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("kv_load", 9, n, [&]() -> PyObject * {
        const Call c;
        const Cache cache(a[0], a[1], a[4], a[5], c.dev);
        const int64_t H = cache.kv.n_head, D = cache.kv.head_dim;
        const int64_t rows = one_dim(tensor(a[2], "slot"));
        const int32_t *slot = whole<int32_t>(a[2], "slot", at::kInt, {rows}, c.dev);
        const int32_t *pos = whole<int32_t>(a[3], "pos", at::kInt, {rows}, c.dev);
        if (rows >= (int64_t(1) << 31)) throw Bad{"too many rows"};
        if (a[6] != Py_None && !THPDtype_Check(a[6])) throw Bad{"dtype must be a torch dtype"};
        if ((a[7] == Py_None) != (a[8] == Py_None)) throw Bad{"give both k and v, or neither"};
        at::Tensor k, v;
        int64_t stride = H * D;
        if (a[7] == Py_None) {
            const at::ScalarType t =
                a[6] == Py_None ? at::kFloat : reinterpret_cast<THPDtype *>(a[6])->scalar_type;
            if (row_type(t) < 0) throw Bad{"rows are float32, float16 or bfloat16"};
            const at::Tensor both = at::empty({2, rows, H, D}, cache.options.dtype(t));
            k = part(both, 0, {rows, H, D});
            v = part(both, rows * H * D, {rows, H, D});
        } else {
            k = tensor(a[7], "k");
            v = tensor(a[8], "v");
            stride = row_stride(k, "k", H, D, c.dev);
            if (a[6] != Py_None && reinterpret_cast<THPDtype *>(a[6])->scalar_type != k.scalar_type())
                throw Bad{"k is not of the given dtype"};
            if (k.size(0) != rows || v.scalar_type() != k.scalar_type() || v.sizes() != k.sizes() ||
                row_stride(v, "v", H, D, c.dev) != stride)
                throw Bad{"k and v must be [rows][heads][head_dim] of the same type and row stride"};
        }
        if (rows > 0)
            check(g_lib.kv_load(&cache.kv, slot, pos, int32_t(rows), k.data_ptr(), v.data_ptr(),
                                  row_type(k.scalar_type()), stride, c.stream),
                  "gpt2_op_kv_load");
        return Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v));
    });
}

// k_cache, v_cache, slot, cached, path, n_path, k_scale, v_scale
PyObject *kv_commit(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("kv_commit", 8, n, [&]() -> PyObject * {
        const Call c;
        const Cache cache(a[0], a[1], a[6], a[7], c.dev, true);
        const at::Tensor &p = tensor(a[4], "path");
        if (p.dim() != 2 || p.size(1) < 1 || p.size(1) > GPT2_MAX_NODES)
            throw Bad{"path must be [sequences][nodes], at most 64 nodes"};
        const int64_t B = p.size(0);
        const int32_t *path = whole<int32_t>(a[4], "path", at::kInt, p.sizes(), c.dev);
        const int32_t *slot = whole<int32_t>(a[2], "slot", at::kInt, {B}, c.dev);
        const int32_t *cached = whole<int32_t>(a[3], "cached", at::kInt, {B}, c.dev);
        const int32_t *n_path = whole<int32_t>(a[5], "n_path", at::kInt, {B}, c.dev);
        if (B >= (int64_t(1) << 31)) throw Bad{"too many sequences"};
        if (B > 0)
            check(g_lib.kv_commit(&cache.kv, cache.layers, slot, cached, path, n_path, int32_t(B), int32_t(p.size(1)),
                                    c.stream),
                  "gpt2_op_kv_commit");
        Py_RETURN_NONE;
    });
}

// q, k_cache, v_cache, slot, cached, first, mask, max_nodes, k_scale, v_scale, scale, out, workspace (the
// last three may be None)
PyObject *tree_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("tree_attention", 13, n, [&]() -> PyObject * {
        const Call c;
        const Cache cache(a[1], a[2], a[8], a[9], c.dev);
        const at::Tensor &q = tensor(a[0], "q");
        const int64_t D = cache.kv.head_dim;
        if (q.dim() != 3) throw Bad{"q must be [rows][heads][head_dim]"};
        const int64_t rows = q.size(0), H = q.size(1), stride = row_stride(q, "q", H, D, c.dev);
        const int64_t B = one_dim(tensor(a[3], "slot"));
        const int32_t *slot = whole<int32_t>(a[3], "slot", at::kInt, {B}, c.dev);
        const int32_t *cached = whole<int32_t>(a[4], "cached", at::kInt, {B}, c.dev);
        const int32_t *first = whole<int32_t>(a[5], "first", at::kInt, {B + 1}, c.dev);
        const uint64_t *mask = whole<uint64_t>(a[6], "mask", at::kLong, {rows}, c.dev);
        const int32_t nodes = to_int(a[7], "max_nodes");
        const float scale = a[10] == Py_None ? float(1.0 / std::sqrt(double(D))) : to_float(a[10], "scale");
        if (H >= (1 << 30) || B >= (int64_t(1) << 31)) throw Bad{"too many heads or sequences"};
        at::Tensor out;
        int64_t out_stride = H * D;
        if (a[11] == Py_None) {
            out = at::empty({rows, H, D}, q.options());
        } else {
            out = tensor(a[11], "out");
            if (out.scalar_type() != q.scalar_type() || out.sizes() != q.sizes())
                throw Bad{"out must have q's type and shape"};
            out_stride = row_stride(out, "out", H, D, c.dev);
        }
        if (rows > 0 && B > 0) {
            const int type = row_type(q.scalar_type());
            const size_t need = g_lib.tree_attention_workspace(&cache.kv, type, int32_t(H), nodes);
            const Workspace ws(a[12], need, c.dev);
            check(g_lib.tree_attention(&cache.kv, q.data_ptr(), type, stride, int32_t(H), slot, cached, first, mask,
                                       int32_t(B), int32_t(rows), nodes, scale, out.data_ptr(), out_stride,
                                       ws.p, ws.bytes, c.stream),
                  "gpt2_op_tree_attention");
        }
        if (a[11] != Py_None) return Py_NewRef(a[11]);
        return THPVariable_Wrap(out);
    });
}

// logits, tokens, parents, first, max_nodes, temperature, draft_probs, u_accept, u_draw, path, n_path, next_token,
// workspace (the last seven may be None)
PyObject *verify_tree(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("verify_tree", 13, n, [&]() -> PyObject * {
        const Call c;
        const at::Tensor &logits = tensor(a[0], "logits");
        if (logits.dim() != 2) throw Bad{"logits must be [rows][vocab]"};
        const int64_t rows = logits.size(0), V = logits.size(1), B = one_dim(tensor(a[3], "first")) - 1;
        const int32_t T = to_int(a[4], "max_nodes");
        const float temperature = to_float(a[5], "temperature");
        if (T < 1 || T > GPT2_MAX_NODES) throw Bad{"max_nodes must be 1 to 64"};
        if (V < 1 || V >= (int64_t(1) << 31) || rows >= (int64_t(1) << 31) || B < 0 || B >= (int64_t(1) << 31))
            throw Bad{"logits or first have a wrong shape"};
        const float *lg = static_cast<float *>(whole(logits, "logits", at::kFloat, logits.sizes(), c.dev));
        const int32_t *tokens = whole<int32_t>(a[1], "tokens", at::kInt, {rows}, c.dev);
        const int32_t *parents = whole<int32_t>(a[2], "parents", at::kInt, {rows}, c.dev);
        const int32_t *first = whole<int32_t>(a[3], "first", at::kInt, {B + 1}, c.dev);
        const float *draft = nullptr, *ua = nullptr, *ud = nullptr;
        if (a[6] != Py_None) draft = whole<float>(a[6], "draft_probs", at::kFloat, {rows, V}, c.dev);
        if (temperature != 0.f) {
            if (a[7] == Py_None || a[8] == Py_None) throw Bad{"temperature > 0 needs u_accept and u_draw"};
            ua = whole<float>(a[7], "u_accept", at::kFloat, {rows}, c.dev);
            ud = whole<float>(a[8], "u_draw", at::kFloat, {B, V}, c.dev);
        }
        const at::TensorOptions ints = logits.options().dtype(at::kInt);
        at::Tensor made;                           // the results that are not given, one after another
        if (a[9] == Py_None || a[10] == Py_None || a[11] == Py_None) made = at::empty({B * (T + 2)}, ints);
        auto result = [&](PyObject *o, const char *name, int64_t from, at::IntArrayRef shape) {
            if (o == Py_None) return part(made, from, shape);
            whole(tensor(o, name), name, at::kInt, shape, c.dev);
            return tensor(o, name);
        };
        at::Tensor path = result(a[9], "path", 0, {B, T}), n_path = result(a[10], "n_path", B * T, {B}),
                   next = result(a[11], "next_token", B * (T + 1), {B});
        const Workspace ws(a[12], g_lib.verify_tree_workspace(int32_t(rows), int32_t(V)), c.dev);
        if (B > 0 && rows == 0) {
            path.fill_(-1);
            n_path.zero_();
            next.fill_(-1);
        } else if (B > 0) {
            check(g_lib.verify_tree(lg, int32_t(V), tokens, parents, first, int32_t(B), int32_t(rows), T, temperature,
                                      draft, ua, ud, path.data_ptr<int32_t>(), n_path.data_ptr<int32_t>(),
                                      next.data_ptr<int32_t>(), ws.p, ws.bytes, c.stream),
                  "gpt2_op_verify_tree");
        }
        return Py_BuildValue("(NNN)", THPVariable_Wrap(path), THPVariable_Wrap(n_path), THPVariable_Wrap(next));
    });
}

// GPT2Error, then the addresses of the library's functions in g_lib's order.
PyObject *bind(PyObject *, PyObject *args)
{
    PyObject *cls;
    unsigned long long f[7];
    if (!PyArg_ParseTuple(args, "OKKKKKKK", &cls, f, f + 1, f + 2, f + 3, f + 4, f + 5, f + 6)) return nullptr;
    g_lib.kv_store = reinterpret_cast<decltype(g_lib.kv_store)>(f[0]);
    g_lib.kv_load = reinterpret_cast<decltype(g_lib.kv_load)>(f[1]);
    g_lib.kv_commit = reinterpret_cast<decltype(g_lib.kv_commit)>(f[2]);
    g_lib.tree_attention_workspace = reinterpret_cast<decltype(g_lib.tree_attention_workspace)>(f[3]);
    g_lib.tree_attention = reinterpret_cast<decltype(g_lib.tree_attention)>(f[4]);
    g_lib.verify_tree_workspace = reinterpret_cast<decltype(g_lib.verify_tree_workspace)>(f[5]);
    g_lib.verify_tree = reinterpret_cast<decltype(g_lib.verify_tree)>(f[6]);
    Py_XSETREF(g_error, Py_NewRef(cls));
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(kv_store),       FAST(kv_load),     FAST(kv_commit),
                           FAST(tree_attention), FAST(verify_tree), {"bind", bind, METH_VARARGS, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops() { return PyModule_Create(&g_module); }
