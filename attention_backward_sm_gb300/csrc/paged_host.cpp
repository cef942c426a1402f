// Host side of the paged-cache operators and of the rotation by positions for
// Python: checks tensors, allocates outputs and workspace and calls the C entry
// points.
//
// One call here costs a few microseconds less than the same steps in Python
// and ctypes (decode: 25 -> 6.5 us of host time on a Grace core, with kernels
// of 5.4 us for a single short request), which is what bounds small batches.
// The arguments are positional; paged.py and rope.py have the documented
// signatures.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/TensorImpl.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "../../include/fabwd.h"

namespace {

using at::Tensor;

// Raised as ValueError: what only the binding can see (types, shapes,
// strides, devices).
struct Refusal {
  std::string message;
};
[[noreturn]] void refuse(const std::string& message) { throw Refusal{message}; }

// A refusal of the C layer, raised as the package's FabwdError.
struct CError {
  int code;
};

void check(int rc) {
  if (rc != FA_OK) throw CError{rc};
}

PyObject* raise(const CError& e) {
  PyObject* mod = PyImport_ImportModule("attention_backward_sm_gb300");
  PyObject* cls = mod ? PyObject_GetAttrString(mod, "FabwdError") : nullptr;
  PyObject* err = cls ? PyObject_CallFunction(cls, "is", e.code, fa_last_error()) : nullptr;
  if (err) PyErr_SetObject(cls, err);
  Py_XDECREF(err);
  Py_XDECREF(cls);
  Py_XDECREF(mod);
  return nullptr;
}

std::string dims(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + ")";
}

std::string kind(const Tensor& t) { return std::string(c10::toString(t.scalar_type())) + " " + dims(t.sizes()); }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

std::optional<Tensor> tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return std::nullopt;
  return tensor(o, name);
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

int integer32(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v != static_cast<int>(v)) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}

int size32(int64_t v, const char* name) {
  if (v > 0x7fffffff) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}

// A contiguous vector of a type, of n entries (n < 0: any number).
void vector(const Tensor& t, const char* name, at::ScalarType type, int64_t n = -1) {
  if (t.scalar_type() != type || t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " vector" +
           (n >= 0 ? " of " + std::to_string(n) : "") + ", got " + kind(t));
}

void vector(const std::optional<Tensor>& t, const char* name, at::ScalarType type, int64_t n) {
  if (t) vector(*t, name, type, n);
}

// Elements from one row of a [n, heads, dim] bf16 tensor to the next.
int64_t row_stride(const Tensor& t, const char* name, int64_t n, int64_t heads, int64_t dim,
                   const char* dim_is = ", the last being the cache's head_dim") {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != dim)
    refuse(std::string(name) + " must be bfloat16 (" + std::to_string(n) + ", " + std::to_string(heads) + ", " +
           std::to_string(dim) + ")" + dim_is + ", got " + kind(t));
  if (t.numel() && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != dim)))
    refuse(std::string(name) + " must have its heads packed in each row, got strides " + dims(t.strides()));
  return n > 1 ? t.stride(0) : heads * dim;
}

struct Cache {
  Tensor k, v;
  std::optional<Tensor> k_scale, v_scale;
  int type, pages, page_size, heads_kv, dim;

  Cache(PyObject* pk, PyObject* pv, PyObject* pks, PyObject* pvs)
      : k(tensor(pk, "k_cache")), v(tensor(pv, "v_cache")), k_scale(tensor_or_none(pks, "k_scale")),
        v_scale(tensor_or_none(pvs, "v_scale")) {
    if (k.dim() != 4 || k.sizes() != v.sizes())
      refuse("k_cache and v_cache must have one shape [num_pages, page_size, Hkv, d], got " + dims(k.sizes()) +
             " and " + dims(v.sizes()));
    const auto st = k.scalar_type();
    if ((st != at::kBFloat16 && st != at::kFloat8_e4m3fn) || v.scalar_type() != st)
      refuse("k_cache and v_cache must both be bfloat16 or both float8_e4m3fn, got " + kind(k) + " and " + kind(v));
    bool alike = true;   // where there is more than one of something
    for (int i = 0; i < 4; ++i) alike = alike && (k.size(i) <= 1 || k.stride(i) == v.stride(i));
    if (k.numel() && (k.stride(3) != 1 || v.stride(3) != 1 || !alike))
      refuse("k_cache and v_cache must have the same strides, the last 1, got " + dims(k.strides()) + " and " +
             dims(v.strides()));
    type = st == at::kBFloat16 ? FA_KV_BF16 : FA_KV_E4M3;
    pages = size32(k.size(0), "num_pages");
    page_size = size32(k.size(1), "page_size");
    heads_kv = size32(k.size(2), "Hkv");
    dim = size32(k.size(3), "head_dim");
    vector(k_scale, "k_scale", at::kFloat, heads_kv);
    vector(v_scale, "v_scale", at::kFloat, heads_kv);
  }
  const float* ks() const { return k_scale ? static_cast<const float*>(k_scale->const_data_ptr()) : nullptr; }
  const float* vs() const { return v_scale ? static_cast<const float*>(v_scale->const_data_ptr()) : nullptr; }
};

struct Table {
  Tensor t;
  int batch, width;
  int64_t stride;
  explicit Table(PyObject* o) : t(tensor(o, "block_table")) {
    if (t.scalar_type() != at::kInt || t.dim() != 2)
      refuse("block_table must be int32 [batch, max_pages], got " + kind(t));
    batch = size32(t.size(0), "batch");
    width = size32(t.size(1), "max_pages");
    if (batch > 0 && width > 1 && t.stride(1) != 1)
      refuse("block_table must have contiguous rows, got strides " + dims(t.strides()));
    stride = batch > 1 ? t.stride(0) : width;
  }
};

// All tensors on one CUDA device; then that device, and the caller's stream
// if there is one, are current for the rest of the call.
class Place {
 public:
  explicit Place(const Tensor& t) : device_(t.device()) {
    if (!device_.is_cuda()) refuse("the tensors must be on a CUDA device, got " + device_.str());
    used_[count_++] = &t;
  }
  Place& with(const Tensor& t, const char* name) {
    if (t.device() != device_)
      refuse(std::string(name) + " is on " + t.device().str() + ", the others on " + device_.str());
    used_[count_++] = &t;
    return *this;
  }
  Place& with(const std::optional<Tensor>& t, const char* name) { return t ? with(*t, name) : *this; }
  Place& enter(PyObject* stream) {
    if (stream == Py_None) {
      device_guard_.reset_device(device_);
      return *this;
    }
    const int64_t id = attr(stream, "stream_id"), index = attr(stream, "device_index"),
                  type = attr(stream, "device_type");
    if (index != device_.index())
      refuse("the stream is on device " + std::to_string(index) + ", the tensors on " + device_.str());
    const auto s = c10::cuda::CUDAStream::unpack3(id, static_cast<c10::DeviceIndex>(index),
                                                  static_cast<c10::DeviceType>(type));
    // The tensors belong to other streams perhaps: their memory is not to be
    // handed out again before this stream is done with it.
    for (int i = 0; i < count_; ++i)
      c10::cuda::CUDACachingAllocator::recordStream(used_[i]->storage().data_ptr(), s);
    stream_guard_.emplace(s);
    return *this;
  }
  fa_stream_t stream() const {
    return reinterpret_cast<fa_stream_t>(c10::cuda::getCurrentCUDAStream(device_.index()).stream());
  }
  // Device memory of the current stream.
  c10::Storage bytes(int64_t n) const {
    auto* const a = c10::cuda::CUDACachingAllocator::get();
    return c10::Storage(c10::Storage::use_byte_size_t(), n, a->allocate(n), a, /*resizable=*/false);
  }

 private:
  static int64_t attr(PyObject* o, const char* name) {
    PyObject* v = PyObject_GetAttrString(o, name);
    if (!v) throw python_error();
    const long long n = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (n == -1 && PyErr_Occurred()) throw python_error();
    return n;
  }
  c10::Device device_;
  const Tensor* used_[16];   // every tensor of the call
  int count_ = 0;
  c10::cuda::OptionalCUDAGuard device_guard_;
  std::optional<c10::cuda::CUDAStreamGuard> stream_guard_;
};

// Contiguous tensors cut one after the other out of one allocation of bytes
// (an allocation is the dearest step of a small call).
class Cutter {
 public:
  static int64_t size(int64_t n, int64_t element) { return (n * element + 255) / 256 * 256; }
  explicit Cutter(c10::Storage base) : base_(std::move(base)) {}
  Tensor next(at::IntArrayRef shape, at::ScalarType type) {
    const int64_t element = static_cast<int64_t>(c10::elementSize(type));
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base_),
                                                        c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                        c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    t.unsafeGetTensorImpl()->set_storage_offset(at_ / element);
    at_ += size(t.numel(), element);
    return t;
  }

 private:
  c10::Storage base_;
  int64_t at_ = 0;
};

template <class T>
T* ptr(const Tensor& t) {
  return t.numel() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

// The launch itself without the interpreter's lock.
template <class F>
int unlocked(F f) {
  struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
  } released;
  return f();
}

// An undefined tensor becomes None.
PyObject* pack(std::initializer_list<Tensor> ts) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
  return false;
}

#define FAB_BEGIN HANDLE_TH_ERRORS try {
#define FAB_END           \
  }                                                                                                  \
  catch (const CError& e) { return raise(e); } \
  catch (const Refusal& e) { PyErr_SetString(PyExc_ValueError, e.message.c_str()); return nullptr; } \
  END_HANDLE_TH_ERRORS

// block_table, seq_lens, new_lens, free_pages, page_size, num_tokens,
// free_start, out (None or 5 tensors), stream
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FAB_BEGIN
  if (!arity(n, 9)) return nullptr;
  const Table table(a[0]);
  const Tensor &seq = tensor(a[1], "seq_lens"), &fresh = tensor(a[2], "new_lens"), &list = tensor(a[3], "free_pages");
  vector(seq, "seq_lens", at::kInt, table.batch);
  vector(fresh, "new_lens", at::kInt, table.batch);
  vector(list, "free_pages", at::kInt);
  const int page_size = integer32(a[4], "page_size");
  const int64_t tokens = integer32(a[5], "num_tokens");
  if (tokens < 0) refuse("num_tokens must be >= 0");
  const auto start = tensor_or_none(a[6], "free_start");
  vector(start, "free_start", at::kInt, 1);
  Place place(table.t);
  place.with(seq, "seq_lens").with(fresh, "new_lens").with(list, "free_pages").with(start, "free_start");
  Tensor slots, positions, cu, after, next;
  if (a[7] != Py_None) {
    if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 5) refuse("out must be a tuple of 5 tensors");
    slots = tensor(PyTuple_GET_ITEM(a[7], 0), "slots");
    positions = tensor(PyTuple_GET_ITEM(a[7], 1), "positions");
    cu = tensor(PyTuple_GET_ITEM(a[7], 2), "cu_new");
    after = tensor(PyTuple_GET_ITEM(a[7], 3), "seq_lens_out");
    next = tensor(PyTuple_GET_ITEM(a[7], 4), "free_next");
    vector(slots, "slots", at::kLong, tokens);
    vector(positions, "positions", at::kInt, tokens);
    vector(cu, "cu_new", at::kInt, table.batch + 1);
    vector(after, "seq_lens_out", at::kInt, table.batch);
    vector(next, "free_next", at::kInt, 1);
    place.with(slots, "slots").with(positions, "positions").with(cu, "cu_new").with(after, "seq_lens_out");
    place.with(next, "free_next").enter(a[8]);
  } else {
    place.enter(a[8]);
    Cutter out(place.bytes(Cutter::size(tokens, 8) + Cutter::size(tokens, 4) + Cutter::size(table.batch + 1, 4) +
                           Cutter::size(table.batch, 4) + Cutter::size(1, 4)));
    slots = out.next({tokens}, at::kLong);
    positions = out.next({tokens}, at::kInt);
    cu = out.next({table.batch + 1}, at::kInt);
    after = out.next({table.batch}, at::kInt);
    next = out.next({1}, at::kInt);
  }
  const int num_free = size32(list.numel(), "free_pages");
  check(unlocked([&] {
    return fa_kv_plan(ptr<int32_t>(table.t), table.stride, table.width, ptr<int32_t>(seq), ptr<int32_t>(fresh),
                      ptr<int32_t>(list), num_free, start ? ptr<int32_t>(*start) : nullptr, page_size, table.batch,
                      static_cast<int>(tokens), ptr<int64_t>(slots), ptr<int32_t>(positions), ptr<int32_t>(cu),
                      ptr<int32_t>(after), ptr<int32_t>(next), place.stream());
  }));
  return pack({slots, positions, cu, after, next});
  FAB_END
}

// k, v, slots, k_cache, v_cache, k_scale, v_scale, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FAB_BEGIN
  if (!arity(n, 8)) return nullptr;
  const Cache c(a[3], a[4], a[5], a[6]);
  const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots");
  vector(slots, "slots", at::kLong);
  const int tokens = size32(slots.numel(), "num_tokens");
  const int64_t ks = row_stride(k, "k", tokens, c.heads_kv, c.dim), vs = row_stride(v, "v", tokens, c.heads_kv, c.dim);
  Place place(c.k);
  place.with(c.v, "v_cache").with(k, "k").with(v, "v").with(slots, "slots").with(c.k_scale, "k_scale");
  place.with(c.v_scale, "v_scale").enter(a[7]);
  check(unlocked([&] {
    return fa_kv_append(ptr<fa_bf16>(k), ptr<fa_bf16>(v), ks, vs, ptr<int64_t>(slots), tokens, ptr<void>(c.k),
                        ptr<void>(c.v), c.type, c.ks(), c.vs(), c.k.stride(0), c.k.stride(1), c.k.stride(2), c.pages,
                        c.page_size, c.heads_kv, c.dim, place.stream());
  }));
  Py_RETURN_NONE;
  FAB_END
}

// q, k_cache, v_cache, block_table, seq_lens, scale, window, k_scale, v_scale,
// out (None or (o, lse or None)), workspace, stream
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FAB_BEGIN
  if (!arity(n, 12)) return nullptr;
  const Cache c(a[1], a[2], a[7], a[8]);
  const Table table(a[3]);
  const Tensor &q = tensor(a[0], "q"), &seq = tensor(a[4], "seq_lens");
  if (q.dim() != 3) refuse("q must be [batch, H, d], got " + kind(q));
  const int64_t batch = table.batch, heads = q.size(1), dim = c.dim;
  const int64_t q_stride = row_stride(q, "q", batch, heads, dim);
  vector(seq, "seq_lens", at::kInt, batch);
  const double scale = PyFloat_AsDouble(a[5]);
  if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  const int window = integer32(a[6], "window"), h32 = size32(heads, "H");
  auto work = tensor_or_none(a[10], "workspace");
  if (work && !work->is_contiguous()) refuse("workspace must be contiguous");
  Place place(q);
  place.with(c.k, "k_cache").with(c.v, "v_cache").with(table.t, "block_table").with(seq, "seq_lens");
  place.with(c.k_scale, "k_scale").with(c.v_scale, "v_scale").with(work, "workspace");
  // 0 for shapes that fa_decode refuses, below, with its code.
  const size_t need = fa_decode_workspace_size(table.batch, h32, c.heads_kv, c.dim);
  Tensor o;
  std::optional<Tensor> lse;
  if (a[9] != Py_None) {
    if (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 2) refuse("out must be a tuple (o, lse)");
    o = tensor(PyTuple_GET_ITEM(a[9], 0), "o");
    lse = tensor_or_none(PyTuple_GET_ITEM(a[9], 1), "lse");
    row_stride(o, "o", batch, heads, dim);
    if (!o.is_contiguous()) refuse("o must be contiguous");
    if (lse && (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != batch ||
                lse->size(1) != heads || !lse->is_contiguous()))
      refuse("lse must be contiguous float32 [batch, H], got " + kind(*lse));
    place.with(o, "o").with(lse, "lse").enter(a[11]);
  } else {
    place.enter(a[11]);
    Cutter out(place.bytes(Cutter::size(batch * heads * dim, 2) + Cutter::size(batch * heads, 4)));
    o = out.next({batch, heads, dim}, at::kBFloat16);
    lse = out.next({batch, heads}, at::kFloat);
  }
  // A workspace of this call alone goes back to the allocator with the return,
  // for later work on the same stream.
  c10::DataPtr own_work;
  if (!work && need > 0) own_work = c10::cuda::CUDACachingAllocator::get()->allocate(need);
  void* const work_ptr = work ? ptr<void>(*work) : own_work.get();
  const size_t work_bytes = work ? work->nbytes() : need;
  check(unlocked([&] {
    return fa_decode(ptr<fa_bf16>(q), q_stride, ptr<void>(c.k), ptr<void>(c.v), c.type, c.ks(), c.vs(),
                     c.k.stride(0), c.k.stride(1), c.k.stride(2), c.pages, c.page_size, ptr<int32_t>(table.t),
                     table.stride, table.width, ptr<int32_t>(seq), table.batch, h32, c.heads_kv, c.dim, window,
                     static_cast<float>(scale), ptr<fa_bf16>(o), lse ? ptr<float>(*lse) : nullptr,
                     work_ptr, work_bytes, place.stream());
  }));
  if (!lse) {
    PyObject* w = THPVariable_Wrap(o);
    return w ? Py_BuildValue("(NO)", w, Py_None) : nullptr;
  }
  return pack({o, *lse});
  FAB_END
}

// q, k_cache, v_cache, block_table, seq_lens, cu_new, scale, window, k_scale,
// v_scale, out (None or (o, lse or None)), workspace, stream
PyObject* extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FAB_BEGIN
  if (!arity(n, 13)) return nullptr;
  const Cache c(a[1], a[2], a[8], a[9]);
  const Table table(a[3]);
  const Tensor &q = tensor(a[0], "q"), &seq = tensor(a[4], "seq_lens"), &cu = tensor(a[5], "cu_new");
  if (q.dim() != 3) refuse("q must be [num_tokens, H, d], got " + kind(q));
  const int64_t tokens = q.size(0), heads = q.size(1), dim = c.dim;
  const int64_t q_stride = row_stride(q, "q", tokens, heads, dim);
  vector(seq, "seq_lens", at::kInt, table.batch);
  vector(cu, "cu_new", at::kInt, table.batch + int64_t{1});
  const double scale = PyFloat_AsDouble(a[6]);
  if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  const int window = integer32(a[7], "window"), h32 = size32(heads, "H"), t32 = size32(tokens, "num_tokens");
  auto work = tensor_or_none(a[11], "workspace");
  if (work && !work->is_contiguous()) refuse("workspace must be contiguous");
  Place place(q);
  place.with(c.k, "k_cache").with(c.v, "v_cache").with(table.t, "block_table").with(seq, "seq_lens").with(cu, "cu_new");
  place.with(c.k_scale, "k_scale").with(c.v_scale, "v_scale").with(work, "workspace");
  // 0 for a head_dim that fa_extend refuses, below, with its code.
  const size_t need = fa_extend_workspace_size(c.dim);
  Tensor o;
  std::optional<Tensor> lse;
  if (a[10] != Py_None) {
    if (!PyTuple_Check(a[10]) || PyTuple_GET_SIZE(a[10]) != 2) refuse("out must be a tuple (o, lse)");
    o = tensor(PyTuple_GET_ITEM(a[10], 0), "o");
    lse = tensor_or_none(PyTuple_GET_ITEM(a[10], 1), "lse");
    row_stride(o, "o", tokens, heads, dim);
    if (!o.is_contiguous()) refuse("o must be contiguous");
    if (lse && (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != tokens ||
                lse->size(1) != heads || !lse->is_contiguous()))
      refuse("lse must be contiguous float32 [num_tokens, H], got " + kind(*lse));
    place.with(o, "o").with(lse, "lse").enter(a[12]);
  } else {
    place.enter(a[12]);
    Cutter out(place.bytes(Cutter::size(tokens * heads * dim, 2) + Cutter::size(tokens * heads, 4)));
    o = out.next({tokens, heads, dim}, at::kBFloat16);
    lse = out.next({tokens, heads}, at::kFloat);
  }
  c10::DataPtr own_work;
  if (!work && need > 0) own_work = c10::cuda::CUDACachingAllocator::get()->allocate(need);
  void* const work_ptr = work ? ptr<void>(*work) : own_work.get();
  const size_t work_bytes = work ? work->nbytes() : need;
  check(unlocked([&] {
    return fa_extend(ptr<fa_bf16>(q), q_stride, ptr<void>(c.k), ptr<void>(c.v), c.type, c.ks(), c.vs(), c.k.stride(0),
                     c.k.stride(1), c.k.stride(2), c.pages, c.page_size, ptr<int32_t>(table.t), table.stride,
                     table.width, ptr<int32_t>(seq), ptr<int32_t>(cu), table.batch, t32, h32, c.heads_kv, c.dim, window,
                     static_cast<float>(scale), ptr<fa_bf16>(o), lse ? ptr<float>(*lse) : nullptr, work_ptr, work_bytes,
                     place.stream());
  }));
  return pack({o, lse ? *lse : Tensor()});
  FAB_END
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// Rows [n, heads, dim] of bf16 values that may be absent (heads 0).
struct Rows {
  std::optional<Tensor> t;
  int heads = 0;
  int64_t stride = 0;
  Rows() = default;
  // n, dim, heads < 0: whatever the tensor has
  Rows(PyObject* o, const char* name, int64_t& n, int64_t& dim, int64_t want_heads = -1) : t(tensor_or_none(o, name)) {
    if (!t) return;
    if (t->dim() != 3) refuse(std::string(name) + " must be [num_tokens, heads, d], got " + kind(*t));
    if (n < 0) n = t->size(0);
    if (dim < 0) dim = t->size(2);
    stride = row_stride(*t, name, n, want_heads < 0 ? t->size(1) : want_heads, dim, "");
    heads = size32(t->size(1), "heads");
  }
  fa_bf16* p() const { return t ? ptr<fa_bf16>(*t) : nullptr; }
};

// What the three rotation calls share.
struct Turns {
  Tensor positions, freqs;
  std::optional<Tensor> q_weight, k_weight;
  int rotary, layout, weight_type = FA_WEIGHT_BF16;
  float mscale, eps;
  // positions, freqs, layout, mscale, q_weight, k_weight, eps
  Turns(PyObject* const* a, int64_t tokens, int64_t dim)
      : positions(tensor(a[0], "positions")), freqs(tensor(a[1], "freqs")), q_weight(tensor_or_none(a[4], "q_weight")),
        k_weight(tensor_or_none(a[5], "k_weight")), layout(integer32(a[2], "layout")),
        mscale(static_cast<float>(real(a[3]))), eps(static_cast<float>(real(a[6]))) {
    vector(positions, "positions", at::kInt, tokens);
    vector(freqs, "freqs", at::kLong);
    rotary = size32(2 * freqs.numel(), "rotary_dim");
    for (const auto* w : {&q_weight, &k_weight}) {
      const char* const name = w == &q_weight ? "q_weight" : "k_weight";
      if (!*w) continue;
      const auto st = (*w)->scalar_type();
      if (st != at::kBFloat16 && st != at::kFloat) refuse(std::string(name) + " must be bfloat16 or float32, got " + kind(**w));
      vector(**w, name, st, dim);
      weight_type = st == at::kFloat ? FA_WEIGHT_F32 : FA_WEIGHT_BF16;
    }
    if (q_weight && k_weight && q_weight->scalar_type() != k_weight->scalar_type())
      refuse("q_weight and k_weight must have one type, got " + kind(*q_weight) + " and " + kind(*k_weight));
  }
  void place(Place& pl) const {
    pl.with(positions, "positions").with(freqs, "freqs").with(q_weight, "q_weight").with(k_weight, "k_weight");
  }
  const uint64_t* f() const { return reinterpret_cast<const uint64_t*>(ptr<int64_t>(freqs)); }
  static void* w(const std::optional<Tensor>& t) { return t ? t->data_ptr() : nullptr; }
};

const Tensor& first_of(const Rows& a, const Rows& b, const char* what) {
  if (!a.t && !b.t) refuse(std::string("one at least of ") + what + " must be given");
  return a.t ? *a.t : *b.t;
}

// q, k, [positions, freqs, layout, mscale, q_weight, k_weight, eps], out, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FAB_BEGIN
  if (!arity(n, 11)) return nullptr;
  int64_t tokens = -1, dim = -1;
  const Rows q(a[0], "q", tokens, dim), k(a[1], "k", tokens, dim);
  const Tensor& lead = first_of(q, k, "q and k");
  const Turns r(a + 2, tokens, dim);
  Place place(lead);
  place.with(k.t, "k");
  r.place(place);
  Rows qo, ko;
  if (a[9] != Py_None) {
    if (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 2) refuse("out must be a tuple (q_out, k_out)");
    qo = Rows(PyTuple_GET_ITEM(a[9], 0), "q_out", tokens, dim, q.heads);
    ko = Rows(PyTuple_GET_ITEM(a[9], 1), "k_out", tokens, dim, k.heads);
    if (!qo.t != !q.t || !ko.t != !k.t) refuse("out must have a tensor for q and for k where they are given");
    place.with(qo.t, "q_out").with(ko.t, "k_out").enter(a[10]);
  } else {
    place.enter(a[10]);
    Cutter out(place.bytes(Cutter::size(tokens * q.heads * dim, 2) + Cutter::size(tokens * k.heads * dim, 2)));
    if (q.t) qo.t = out.next({tokens, q.heads, dim}, at::kBFloat16);
    if (k.t) ko.t = out.next({tokens, k.heads, dim}, at::kBFloat16);
    qo.stride = q.heads * dim;
    ko.stride = k.heads * dim;
  }
  const int t32 = size32(tokens, "num_tokens"), d32 = size32(dim, "head_dim");
  check(unlocked([&] {
    return fa_qk_rope(q.p(), k.p(), q.stride, k.stride, ptr<int32_t>(r.positions), r.f(), r.rotary, r.layout, r.mscale,
                      r.w(r.q_weight), r.w(r.k_weight), r.weight_type, r.eps, t32, q.heads, k.heads, d32, qo.p(),
                      ko.p(), qo.stride, ko.stride, place.stream());
  }));
  return pack({qo.t ? *qo.t : Tensor(), ko.t ? *ko.t : Tensor()});
  FAB_END
}

// dq_out, dk_out, [as above], q, k, out (None or 4 tensors), workspace, stream
PyObject* rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FAB_BEGIN
  if (!arity(n, 14)) return nullptr;
  int64_t tokens = -1, dim = -1;
  const Rows gq(a[0], "dq_out", tokens, dim), gk(a[1], "dk_out", tokens, dim);
  const Tensor& lead = first_of(gq, gk, "dq_out and dk_out");
  const Turns r(a + 2, tokens, dim);
  const Rows q(a[9], "q", tokens, dim, gq.heads), k(a[10], "k", tokens, dim, gk.heads);
  if ((r.q_weight && gq.t && !q.t) || (r.k_weight && gk.t && !k.t))
    refuse("the gradient of a norm needs its input (q for q_weight, k for k_weight)");
  auto work = tensor_or_none(a[12], "workspace");
  if (work && !work->is_contiguous()) refuse("workspace must be contiguous");
  Place place(lead);
  place.with(gk.t, "dk_out").with(q.t, "q").with(k.t, "k").with(work, "workspace");
  r.place(place);
  Rows dq, dk;
  Tensor dqw, dkw;
  if (a[11] != Py_None) {
    if (!PyTuple_Check(a[11]) || PyTuple_GET_SIZE(a[11]) != 4) refuse("out must be a tuple (dq, dk, dq_weight, dk_weight)");
    dq = Rows(PyTuple_GET_ITEM(a[11], 0), "dq", tokens, dim, gq.heads);
    dk = Rows(PyTuple_GET_ITEM(a[11], 1), "dk", tokens, dim, gk.heads);
    const auto wq = tensor_or_none(PyTuple_GET_ITEM(a[11], 2), "dq_weight"),
               wk = tensor_or_none(PyTuple_GET_ITEM(a[11], 3), "dk_weight");
    if (!dq.t != !gq.t || !dk.t != !gk.t || !wq != !r.q_weight || !wk != !r.k_weight)
      refuse("out must have a tensor for each of dq, dk and the weights' gradients that the call computes, else None");
    vector(wq, "dq_weight", at::kFloat, dim);
    vector(wk, "dk_weight", at::kFloat, dim);
    if (wq) dqw = *wq;
    if (wk) dkw = *wk;
    place.with(dq.t, "dq").with(dk.t, "dk").with(wq, "dq_weight").with(wk, "dk_weight").enter(a[13]);
  } else {
    place.enter(a[13]);
    Cutter out(place.bytes(Cutter::size(tokens * gq.heads * dim, 2) + Cutter::size(tokens * gk.heads * dim, 2) +
                           2 * Cutter::size(dim, 4)));
    if (gq.t) dq.t = out.next({tokens, gq.heads, dim}, at::kBFloat16);
    if (gk.t) dk.t = out.next({tokens, gk.heads, dim}, at::kBFloat16);
    if (r.q_weight) dqw = out.next({dim}, at::kFloat);
    if (r.k_weight) dkw = out.next({dim}, at::kFloat);
    dq.stride = gq.heads * dim;
    dk.stride = gk.heads * dim;
  }
  const int t32 = size32(tokens, "num_tokens"), d32 = size32(dim, "head_dim");
  // 0 for a head_dim that fa_qk_rope_bwd refuses, below, with its code.
  const size_t need = r.q_weight || r.k_weight ? fa_qk_rope_bwd_workspace_size(d32) : 0;
  c10::DataPtr own_work;
  if (!work && need > 0) own_work = c10::cuda::CUDACachingAllocator::get()->allocate(need);
  void* const work_ptr = work ? ptr<void>(*work) : own_work.get();
  const size_t work_bytes = work ? work->nbytes() : need;
  check(unlocked([&] {
    return fa_qk_rope_bwd(gq.p(), gk.p(), gq.stride, gk.stride, q.p(), k.p(), q.stride, k.stride,
                          ptr<int32_t>(r.positions), r.f(), r.rotary, r.layout, r.mscale, r.w(r.q_weight),
                          r.w(r.k_weight), r.weight_type, r.eps, t32, gq.heads, gk.heads, d32, dq.p(), dk.p(),
                          dq.stride, dk.stride, dqw.defined() ? ptr<float>(dqw) : nullptr,
                          dkw.defined() ? ptr<float>(dkw) : nullptr, work_ptr, work_bytes, place.stream());
  }));
  return pack({dq.t ? *dq.t : Tensor(), dk.t ? *dk.t : Tensor(), dqw, dkw});
  FAB_END
}

// q, k, v, [as above], k_cache, v_cache, slots, k_scale, v_scale, out (None or
// q_out), stream
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FAB_BEGIN
  if (!arity(n, 17)) return nullptr;
  const Cache c(a[10], a[11], a[13], a[14]);
  const Tensor& slots = tensor(a[12], "slots");
  vector(slots, "slots", at::kLong);
  int64_t tokens = slots.numel(), dim = c.dim;
  const Rows q(a[0], "q", tokens, dim), k(a[1], "k", tokens, dim, c.heads_kv), v(a[2], "v", tokens, dim, c.heads_kv);
  if (!q.t || !k.t || !v.t) refuse("q, k and v must be tensors");
  const Turns r(a + 3, tokens, dim);
  Place place(c.k);
  place.with(c.v, "v_cache").with(*q.t, "q").with(*k.t, "k").with(*v.t, "v").with(slots, "slots");
  place.with(c.k_scale, "k_scale").with(c.v_scale, "v_scale");
  r.place(place);
  Rows qo;
  if (a[15] != Py_None) {
    qo = Rows(a[15], "out", tokens, dim, q.heads);
    place.with(qo.t, "out").enter(a[16]);
  } else {
    place.enter(a[16]);
    Cutter out(place.bytes(Cutter::size(tokens * q.heads * dim, 2)));
    qo.t = out.next({tokens, q.heads, dim}, at::kBFloat16);
    qo.stride = q.heads * dim;
  }
  const int t32 = size32(tokens, "num_tokens");
  check(unlocked([&] {
    return fa_qk_rope_append(q.p(), k.p(), v.p(), q.stride, k.stride, v.stride, ptr<int32_t>(r.positions), r.f(),
                             r.rotary, r.layout, r.mscale, r.w(r.q_weight), r.w(r.k_weight), r.weight_type, r.eps, t32,
                             q.heads, qo.p(), qo.stride, ptr<int64_t>(slots), ptr<void>(c.k), ptr<void>(c.v), c.type,
                             c.ks(), c.vs(), c.k.stride(0), c.k.stride(1), c.k.stride(2), c.pages, c.page_size,
                             c.heads_kv, c.dim, place.stream());
  }));
  return THPVariable_Wrap(*qo.t);
  FAB_END
}

PyMethodDef methods[] = {
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(plan)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL, nullptr},
    {"extend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(extend)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"rope_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_bwd)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_append)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_host(void) { return PyModule_Create(&module); }
