// kvd_binding.cpp -- the Python side of the entry points whose calls are short:
// the checks of kvd.py's other functions (dtype, device, contiguity, shapes) on
// torch tensors and the C call, compiled, so that a call costs the host little
// more than its launches (the same checks in Python: 10 us a call and more).
//
// Every function takes positional arguments in the order of its wrapper in
// kvd.py, raises ValueError for what the wrapper documents, and returns the C
// status.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>
#include <string>

#include "kvd.h"

namespace {

struct Refused {
    PyObject *type;
    std::string what;
};
[[noreturn]] void refuse(const std::string &what) { throw Refused{PyExc_ValueError, what}; }

// The arguments of one call, taken in order.
class Args {
  public:
    Args(const char *fn, PyObject *const *a, Py_ssize_t n, Py_ssize_t want) : a_(a)
    {
        if (n != want)
            throw Refused{PyExc_TypeError, std::string(fn) + " takes " + std::to_string(want) + " arguments, got " +
                                               std::to_string(n)};
    }

    // A CUDA tensor on the current device; `dtype` of kAny is not checked.
    static constexpr c10::ScalarType kAny = c10::ScalarType::Undefined;
    const at::Tensor *tensor(const char *name, c10::ScalarType dtype, bool contiguous = true, bool optional = false)
    {
        PyObject *o = a_[i_++];
        if (optional && o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
        if (contiguous && !t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
        if (dtype != kAny && t.scalar_type() != dtype)
            refuse(std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
        if (t.get_device() != device())
            refuse(std::string(name) + " must be on the current CUDA device (cuda:" + std::to_string(dev_) + "), got cuda:" +
                   std::to_string(t.get_device()));
        return &t;
    }
    const at::Tensor *optional(const char *name, c10::ScalarType dtype) { return tensor(name, dtype, true, true); }

    // A whole number of 32 bits.
    int integer(const char *name, long long lo = -(1ll << 31), long long hi = (1ll << 31) - 1)
    {
        PyObject *o = PyNumber_Index(a_[i_++]);
        if (o == nullptr) throw Refused{nullptr, ""};
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(o, &over);
        Py_DECREF(o);
        if (over != 0 || v < lo || v > hi)
            refuse(std::string(name) + " must be between " + std::to_string(lo) + " and " + std::to_string(hi));
        return (int)v;
    }
    bool truth()
    {
        const int v = PyObject_IsTrue(a_[i_++]);
        if (v < 0) throw Refused{nullptr, ""};
        return v != 0;
    }
    float number()
    {
        const double v = PyFloat_AsDouble(a_[i_++]);
        if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
        return (float)v;
    }
    // A stream's handle, or the current stream for None.
    void *stream()
    {
        PyObject *o = a_[i_++];
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device()).stream();
        void *s = PyLong_AsVoidPtr(o);
        if (s == nullptr && PyErr_Occurred()) throw Refused{nullptr, ""};
        return s;
    }

  private:
    int device()
    {
        if (dev_ < 0) dev_ = c10::cuda::current_device();
        return dev_;
    }
    PyObject *const *a_;
    Py_ssize_t i_ = 0;
    int dev_ = -1;
};

kvd_dtype dtype_code(const at::Tensor &t)
{
    switch (t.scalar_type()) {
    case c10::ScalarType::Float: return KVD_F32;
    case c10::ScalarType::BFloat16: return KVD_BF16;
    case c10::ScalarType::Half: return KVD_F16;
    default: refuse(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
    }
}

bool is(const at::Tensor &t, std::initializer_list<int64_t> shape)
{
    return t.sizes() == at::IntArrayRef(shape.begin(), shape.size());
}

void need(bool ok, const char *what)
{
    if (!ok) refuse(what);
}

int dim32(int64_t n)
{
    if (n > 0x7fffffff) refuse("a tensor has a dimension of 2^31 or more");
    return (int)n;
}

void *ptr(const at::Tensor *t) { return t == nullptr ? nullptr : t->data_ptr(); }
size_t bytes(const at::Tensor *t) { return t == nullptr ? 0 : (size_t)t->numel() * t->element_size(); }

constexpr auto kInt = c10::ScalarType::Int;
constexpr auto kFloat = c10::ScalarType::Float;
constexpr auto kDouble = c10::ScalarType::Double;
constexpr auto kByte = c10::ScalarType::Byte;

// A page pool and the sequences' table.
struct Pool {
    int num_pages, H_kv, page_size, D, max_pages;
};
Pool pool_of(const at::Tensor &k, const at::Tensor &v, const at::Tensor &table, int64_t B)
{
    need(table.dim() == 2 && table.size(0) == B, "block_table must be [B, max_pages]");
    need(k.dim() == 4 && v.sizes() == k.sizes(), "k_pages and v_pages must be the same [num_pages, H_kv, page_size, D]");
    return Pool{dim32(k.size(0)), dim32(k.size(1)), dim32(k.size(2)), dim32(k.size(3)), dim32(table.size(1))};
}

// [B, H, N, D] rows: each row contiguous, the rows at any strides.
void need_rows(const char *name, const at::Tensor &t)
{
    if (t.dim() != 4 || (t.size(3) != 1 && t.stride(3) != 1)) refuse(std::string(name) + " must be [B, H, N, D] with contiguous rows");
}

// q, q_out, k, v, k_new, v_new, (block_table), past_len, max_past_len, inv_freq,
// interleaved, pos_base, positions, err_word, stream
int rope(Args &a, bool paged)
{
    const at::Tensor &q = *a.tensor("q", Args::kAny, false);
    const auto dt = q.scalar_type();
    const at::Tensor &q_out = *a.tensor("q_out", dt), &kc = *a.tensor(paged ? "k_pages" : "k_cache", dt),
                     &vc = *a.tensor(paged ? "v_pages" : "v_cache", dt), &kn = *a.tensor("k_new", dt, false),
                     &vn = *a.tensor("v_new", dt, false);
    const at::Tensor *table = paged ? a.tensor("block_table", kInt) : nullptr;
    const at::Tensor &past = *a.tensor("past_len", kInt);
    const int max_past = a.integer("max_past_len");
    const at::Tensor &freq = *a.tensor("inv_freq", kDouble);
    const bool interleaved = a.truth();
    const int pos_base = a.integer("pos_base");
    const at::Tensor *positions = a.optional("positions", kInt), *err = a.optional("err_word", kInt);
    void *stream = a.stream();
    need_rows("q", q);
    need_rows("k_new", kn);
    need_rows("v_new", vn);
    const int64_t B = q.size(0), H_q = q.size(1), N = q.size(2), D = q.size(3), H_kv = kn.size(1);
    need(is(kn, {B, H_kv, N, D}) && vn.sizes() == kn.sizes() && q_out.sizes() == q.sizes(),
         "shape mismatch between q, q_out and the new K/V");
    need(kc.dim() == 4 && vc.sizes() == kc.sizes() && kc.size(1) == H_kv && kc.size(3) == D && (paged || kc.size(0) == B),
         "shape mismatch between the caches and the new K/V");
    need(past.numel() == B, "past_len must hold B entries");
    need(positions == nullptr || is(*positions, {B, N}), "positions must be [B, N]");
    const kvd_dtype code = dtype_code(q);
    int64_t strides[9];
    const bool dense = q.is_contiguous() && kn.is_contiguous() && vn.is_contiguous();
    if (!dense) {
        need(q.is_contiguous() || q_out.data_ptr() != q.data_ptr(), "q_out may be q only when q is contiguous");
        int64_t *s = strides;
        for (const at::Tensor *t : {&q, &kn, &vn})
            for (int d = 0; d < 3; ++d) *s++ = t->size(d) > 1 ? t->stride(d) : 0;  // (one row: any stride)
    }
    const int64_t *st = dense ? nullptr : strides;
    const int rot = dim32(2 * freq.numel());
    if (paged) {
        const Pool p = pool_of(kc, vc, *table, B);
        return kvd_paged_rope_append(q.data_ptr(), q_out.data_ptr(), kc.data_ptr(), vc.data_ptr(), kn.data_ptr(),
                                     vn.data_ptr(), st, (const int32_t *)table->data_ptr(), (const int32_t *)past.data_ptr(),
                                     (const int32_t *)ptr(positions), pos_base, (const double *)freq.data_ptr(), rot,
                                     interleaved, dim32(B), dim32(H_q), dim32(H_kv), dim32(D), dim32(N), p.page_size,
                                     p.max_pages, p.num_pages, max_past, code, (uint32_t *)ptr(err), stream);
    }
    return kvd_rope_append(q.data_ptr(), q_out.data_ptr(), kc.data_ptr(), vc.data_ptr(), kn.data_ptr(), vn.data_ptr(), st,
                           (const int32_t *)past.data_ptr(), (const int32_t *)ptr(positions), pos_base,
                           (const double *)freq.data_ptr(), rot, interleaved, dim32(B), dim32(H_q), dim32(H_kv),
                           dim32(kc.size(2)), dim32(D), dim32(N), max_past, code, (uint32_t *)ptr(err), stream);
}

// q, k, v, out, (block_table), past_len, max_past_len, softcap, slopes, window,
// doc_start, prefix_len, scale, workspace, err_word, stream
int scored(Args &a, bool paged)
{
    const at::Tensor &q = *a.tensor("q", Args::kAny);
    const auto dt = q.scalar_type();
    const at::Tensor &k = *a.tensor(paged ? "k_pages" : "k_cache", dt), &v = *a.tensor(paged ? "v_pages" : "v_cache", dt),
                     &out = *a.tensor("out", dt);
    const at::Tensor *table = paged ? a.tensor("block_table", kInt) : nullptr;
    const at::Tensor &past = *a.tensor("past_len", kInt);
    const int max_past = a.integer("max_past_len");
    kvd_score s = {};
    s.softcap = a.number();
    const at::Tensor *slopes = a.optional("slopes", kFloat);
    s.window = a.integer("window", 0);
    const at::Tensor *docs = a.optional("doc_start", kInt), *prefix = a.optional("prefix_len", kInt);
    const float scale = a.number();
    const at::Tensor *ws = a.optional("workspace", kByte), *err = a.optional("err_word", kInt);
    void *stream = a.stream();
    need(q.dim() == 4, "q must be [B, H_q, N, D]");
    const int64_t B = q.size(0), H_q = q.size(1), N = q.size(2), D = q.size(3);
    need(out.sizes() == q.sizes() && k.dim() == 4 && v.sizes() == k.sizes() && k.size(3) == D && (paged || k.size(0) == B),
         paged ? "shape mismatch between q, out and the pages" : "shape mismatch between q, out and the caches");
    need(past.numel() == B, "past_len must hold B entries");
    need(slopes == nullptr || is(*slopes, {H_q}), "slopes must be [H_q]");
    need(docs == nullptr || is(*docs, {B, N}), "doc_start must be [B, N]");
    need(prefix == nullptr || is(*prefix, {B}), "prefix_len must be [B]");
    s.slopes = (const float *)ptr(slopes);
    s.doc_start = (const int32_t *)ptr(docs);
    s.prefix_len = (const int32_t *)ptr(prefix);
    const kvd_dtype code = dtype_code(q);
    if (paged) {
        const Pool p = pool_of(k, v, *table, B);
        return kvd_paged_decode_attention_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                                 (const int32_t *)table->data_ptr(), (const int32_t *)past.data_ptr(), &s,
                                                 dim32(B), dim32(H_q), p.H_kv, dim32(D), dim32(N), p.page_size, p.max_pages,
                                                 p.num_pages, max_past, scale, code, ptr(ws), bytes(ws), (uint32_t *)ptr(err),
                                                 stream);
    }
    return kvd_decode_attention_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                       (const int32_t *)past.data_ptr(), &s, dim32(B), dim32(H_q), dim32(k.size(1)),
                                       dim32(k.size(2)), dim32(D), dim32(N), max_past, scale, code, ptr(ws), bytes(ws),
                                       (uint32_t *)ptr(err), stream);
}

// q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, out, past_len, max_past_len, scale, workspace, err_word, stream
// (paged: q, k_pages, v_pages, prefix_table, prefix_len, out, block_table, past_len, ...)
int shared_prefix(Args &a, bool paged)
{
    const at::Tensor &q = *a.tensor("q", Args::kAny);
    const auto dt = q.scalar_type();
    const at::Tensor &kp = *a.tensor(paged ? "k_pages" : "k_prefix", dt), &vp = *a.tensor(paged ? "v_pages" : "v_prefix", dt);
    const at::Tensor *ptable = paged ? a.tensor("prefix_table", kInt) : nullptr;
    const int S = a.integer("prefix_len");
    const at::Tensor *kc = paged ? nullptr : a.tensor("k_cache", dt), *vc = paged ? nullptr : a.tensor("v_cache", dt);
    const at::Tensor &out = *a.tensor("out", dt);
    const at::Tensor *table = paged ? a.tensor("block_table", kInt) : nullptr;
    const at::Tensor &past = *a.tensor("past_len", kInt);
    const int max_past = a.integer("max_past_len");
    const float scale = a.number();
    const at::Tensor *ws = a.optional("workspace", kByte), *err = a.optional("err_word", kInt);
    void *stream = a.stream();
    need(q.dim() == 4, "q must be [B, H_q, N, D]");
    const int64_t B = q.size(0), H_q = q.size(1), N = q.size(2), D = q.size(3);
    need(past.numel() == B, "past_len must hold B entries");
    const kvd_dtype code = dtype_code(q);
    if (paged) {
        const Pool p = pool_of(kp, vp, *table, B);
        need(out.sizes() == q.sizes() && p.D == D, "shape mismatch between q, out and the pages");
        need(ptable->numel() * p.page_size >= S, "prefix_table must name every page of the prefix");
        return kvd_paged_shared_prefix_attention(q.data_ptr(), kp.data_ptr(), vp.data_ptr(), out.data_ptr(),
                                                 (const int32_t *)ptable->data_ptr(), (const int32_t *)table->data_ptr(),
                                                 (const int32_t *)past.data_ptr(), dim32(B), dim32(H_q), p.H_kv, dim32(D),
                                                 dim32(N), p.page_size, p.max_pages, p.num_pages, S, max_past, scale, code,
                                                 ptr(ws), bytes(ws), (uint32_t *)ptr(err), stream);
    }
    need(out.sizes() == q.sizes() && kc->dim() == 4 && vc->sizes() == kc->sizes() && kc->size(0) == B && kc->size(3) == D,
         "shape mismatch between q, out and the caches");
    need(kp.dim() == 3 && vp.sizes() == kp.sizes() && kp.size(0) == kc->size(1) && kp.size(2) == D,
         "k_prefix and v_prefix must be the same [H_kv, S_max, D]");
    return kvd_shared_prefix_attention(q.data_ptr(), kp.data_ptr(), vp.data_ptr(), kc->data_ptr(), vc->data_ptr(),
                                       out.data_ptr(), (const int32_t *)past.data_ptr(), dim32(B), dim32(H_q),
                                       dim32(kc->size(1)), dim32(kp.size(1)), dim32(kc->size(2)), dim32(D), dim32(N), S,
                                       max_past, scale, code, ptr(ws), bytes(ws), (uint32_t *)ptr(err), stream);
}

// No C++ exception leaves a call.
template <int (*F)(Args &, bool), bool kPaged, int kArgs> PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        Args a("this function", args, n, kArgs);
        return PyLong_FromLong(F(a, kPaged));
    } catch (const Refused &r) {
        if (r.type != nullptr) PyErr_SetString(r.type, r.what.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <int (*F)(Args &, bool), bool kPaged, int kArgs> PyMethodDef method(const char *name)
{
    return {name, (PyCFunction)(void (*)(void))(&call<F, kPaged, kArgs>), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<rope, false, 14>("rope_append"),
    method<rope, true, 15>("paged_rope_append"),
    method<scored, false, 15>("decode_attention_scored"),
    method<scored, true, 16>("paged_decode_attention_scored"),
    method<shared_prefix, false, 13>("shared_prefix_attention"),
    method<shared_prefix, true, 13>("paged_shared_prefix_attention"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvd", "Compiled calls of the decode library.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__kvd() { return PyModule_Create(&module); }
