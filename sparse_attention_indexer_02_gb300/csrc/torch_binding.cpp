// Python entry of the serving operators for torch tensors (module _qsa_torch):
// checks of the tensors, descriptors, output allocation and the C-ABI call.
//
// A decode step makes these calls once a layer with a few rows each, where the
// kernels take a few microseconds: reading shapes, strides and addresses
// through Python attributes and ctypes took 12 to 35 us a call, several times
// the work itself.  Here a tensor's fields are read in place.
//
// Every function returns normally or with a Python exception set; no C++
// exception leaves it.  ValueError: the tensors do not fit the call.  The
// status of the C-ABI call is returned, the caller raises on it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cuda_runtime.h>

#include <cmath>
#include <exception>
#include <map>
#include <stdexcept>
#include <string>
#include <utility>

#include "../../include/qsa.h"

namespace {

struct Refused : std::exception {
  std::string what_;
  explicit Refused(std::string w) : what_(std::move(w)) {}
  const char* what() const noexcept override { return what_.c_str(); }
};

void need(bool ok, const char* what) {
  if (!ok) throw Refused(what);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

bool given(PyObject* o) { return o != Py_None; }

long long integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be an integer that fits 64 bits");
  }
  return v;
}

int32_t integer32(PyObject* o, const char* name) {
  const long long v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be true or false");
  }
  return v == 1;
}

int32_t size32(int64_t v, const char* name) {
  if (v > INT32_MAX) throw Refused(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}

// Element stride of dimension d; of a dimension with one entry, whose stride
// may be anything, what a contiguous tensor has.
int64_t step_of(const at::Tensor& t, int64_t d) {
  if (t.size(d) > 1) return t.stride(d);
  int64_t s = 1;
  for (int64_t i = d + 1; i < t.dim(); ++i) s *= t.size(i) > 0 ? t.size(i) : 1;
  return s;
}

// A contiguous vector of n entries (n < 0: any).
void vec(const at::Tensor& t, const char* name, at::ScalarType ty, int64_t n) {
  if (t.scalar_type() != ty || t.dim() != 1 || !t.is_contiguous() || (n >= 0 && t.size(0) != n))
    throw Refused(std::string(name) + " must be a contiguous " + c10::toString(ty) + " vector" +
                  (n >= 0 ? " of " + std::to_string(n) + " entries" : ""));
}

void table(const at::Tensor& t) {
  need(t.scalar_type() == at::kInt && t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1),
       "block_table must be an int32 [num_requests, max_pages] tensor with contiguous rows");
}

// All tensors of a call lie on one CUDA device, the current one: the library
// launches there, whatever device the stream and the addresses are of.
struct Place {
  c10::Device dev;
  explicit Place(const at::Tensor& t) : dev(t.device()) {
    need(dev.is_cuda(), "the tensors must be on a CUDA device");
    int current = -1;
    if (cudaGetDevice(&current) != cudaSuccess) {
      cudaGetLastError();
      current = -1;
    }
    need((int)dev.index() == current, "the tensors must be on the current CUDA device");
  }
  void also(const at::Tensor& t) const { need(t.device() == dev, "the tensors are on different devices"); }
  cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
};

int32_t half_dtype(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return QSA_HALF_BF16;
  if (t.scalar_type() == at::kHalf) return QSA_HALF_F16;
  throw Refused("the caches must be bf16 or fp16");
}

qsa_kv_desc kv_desc(const at::Tensor& k, const at::Tensor& v) {
  qsa_kv_desc d = {};
  d.dtype = half_dtype(k);
  need(v.scalar_type() == k.scalar_type(), "the caches must both be bf16 or both fp16");
  need(k.dim() == 4 && v.sizes() == k.sizes(),
       "the caches must be [num_pages, page_tokens, num_kv_heads, head_dim], values like keys");
  need(step_of(k, 3) == 1 && step_of(v, 3) == 1, "the caches' last dimension must be contiguous");
  d.num_pages = size32(k.size(0), "num_pages");
  d.page_tokens = size32(k.size(1), "page_tokens");
  d.num_kv_heads = size32(k.size(2), "num_kv_heads");
  d.head_dim = size32(k.size(3), "head_dim");
  d.k_page_stride = 2 * step_of(k, 0);
  d.k_token_stride = 2 * step_of(k, 1);
  d.k_head_stride = 2 * step_of(k, 2);
  d.v_page_stride = 2 * step_of(v, 0);
  d.v_token_stride = 2 * step_of(v, 1);
  d.v_head_stride = 2 * step_of(v, 2);
  return d;
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

void arity(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw Refused("wrong number of arguments");
}

template <typename F>
PyObject* guarded(F&& f) noexcept {
  try {
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// A contiguous tensor of `sizes` at byte `at` of a buffer tensor's storage.
at::Tensor slice_of(const at::Tensor& buf, at::ScalarType ty, int64_t at, at::IntArrayRef sizes) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(),
                                                          c10::scalarTypeToTypeMeta(ty));
  t.unsafeGetTensorImpl()->set_storage_offset(at / (int64_t)c10::elementSize(ty));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
  return t;
}

// (context_lens, new_lens, free_pages, block_table, page_tokens, max_tokens,
//  ratio, partial_cols, out: PageMaps or None, PageMaps) -> (status, PageMaps)
PyObject* build_page_maps(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 10);
    need(PyType_Check(a[9]) && PyType_IsSubtype((PyTypeObject*)a[9], &PyTuple_Type), "the result's type must be a tuple");
    const at::Tensor &ctx = tensor(a[0], "context_lens"), &nw = tensor(a[1], "new_lens"),
                     &fp = tensor(a[2], "free_pages"), &bt = tensor(a[3], "block_table");
    vec(ctx, "context_lens", at::kInt, -1);
    const int64_t B = ctx.size(0);
    vec(nw, "new_lens", at::kInt, B);
    vec(fp, "free_pages", at::kInt, -1);
    table(bt);
    need(bt.size(0) == B, "block_table must have a row a request");
    qsa_page_maps_desc d = {};
    d.num_requests = size32(B, "num_requests");
    d.page_tokens = integer32(a[4], "page_tokens");
    d.max_pages = size32(bt.size(1), "max_pages");
    d.ratio = integer32(a[6], "ratio");
    d.partial_cols = truth(a[7], "partial_cols") ? 1 : 0;
    d.table_stride = step_of(bt, 0);
    d.num_free = fp.size(0);
    d.max_tokens = integer(a[5], "max_tokens");
    const int64_t T = d.max_tokens;
    need(T >= 0 && T <= INT32_MAX, "max_tokens out of range");
    static const char* const names[8] = {"query_start", "seq_lens", "slots", "positions", "token_request",
                                         "visible_cols", "column_slots", "pages_used"};
    const int64_t sizes[8] = {B + 1, B, T, T, T, T, T, 1};
    static const at::ScalarType types[8] = {at::kInt, at::kInt, at::kLong, at::kInt, at::kInt, at::kInt, at::kLong,
                                            at::kInt};
    at::Tensor o[8];
    const Place place(ctx);
    place.also(nw), place.also(fp), place.also(bt);
    if (given(a[8])) {
      need(PyTuple_Check(a[8]) && PyTuple_GET_SIZE(a[8]) == 8, "out must be a PageMaps");
      for (int i = 0; i < 8; ++i) {
        o[i] = tensor(PyTuple_GET_ITEM(a[8], i), names[i]);
        vec(o[i], names[i], types[i], sizes[i]);
        place.also(o[i]);
      }
    } else {
      // one allocation for all: the 8-byte outputs first, then the 4-byte ones, each on 16 bytes
      int64_t at[8], bytes = 0;
      for (int pass = 0; pass < 2; ++pass)
        for (int i = 0; i < 8; ++i)
          if ((types[i] == at::kInt) == (pass == 1)) {
            at[i] = bytes;
            bytes += (sizes[i] * (pass ? 4 : 8) + 15) & ~int64_t(15);
          }
      const at::Tensor buf = at::empty({bytes}, ctx.options().dtype(at::kByte));
      for (int i = 0; i < 8; ++i) o[i] = slice_of(buf, types[i], at[i], at::IntArrayRef(&sizes[i], 1));
    }
    const qsa_status st = qsa_build_page_maps(
        &d, ctx.data_ptr<int32_t>(), nw.data_ptr<int32_t>(), fp.data_ptr<int32_t>(), bt.data_ptr<int32_t>(),
        o[0].data_ptr<int32_t>(), o[1].data_ptr<int32_t>(), o[2].data_ptr<int64_t>(), o[3].data_ptr<int32_t>(),
        o[4].data_ptr<int32_t>(), o[5].data_ptr<int32_t>(), o[6].data_ptr<int64_t>(), o[7].data_ptr<int32_t>(),
        place.stream());
    PyObject* maps = a[8];
    if (given(maps)) {
      Py_INCREF(maps);
    } else {
      // the named tuple from a plain one, as its own _make does
      PyObject* plain = PyTuple_New(8);
      if (!plain) return nullptr;
      for (int i = 0; i < 8; ++i) PyTuple_SET_ITEM(plain, i, wrap(o[i]));
      PyObject* args = PyTuple_Pack(1, plain);
      Py_DECREF(plain);
      if (!args) return nullptr;
      maps = PyTuple_Type.tp_new((PyTypeObject*)a[9], args, nullptr);
      Py_DECREF(args);
      if (!maps) return nullptr;
    }
    PyObject* r = PyTuple_New(2);
    if (!r) {
      Py_DECREF(maps);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(st));
    PyTuple_SET_ITEM(r, 1, maps);
    return r;
  });
}

// (k, v, slots, k_cache, v_cache) -> status
PyObject* store_paged_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 5);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots"),
                     &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache");
    const qsa_kv_desc d = kv_desc(kc, vc);
    vec(slots, "slots", at::kLong, -1);
    const int64_t T = slots.size(0);
    for (const at::Tensor* t : {&k, &v})
      need(t->scalar_type() == kc.scalar_type() && t->dim() == 3 && t->size(0) == T && t->size(1) == kc.size(2) &&
               t->size(2) == kc.size(3) && step_of(*t, 2) == 1,
           "k and v must be [T, num_kv_heads, head_dim] in the cache's type, last dimension contiguous");
    const Place place(kc);
    place.also(vc), place.also(k), place.also(v), place.also(slots);
    return PyLong_FromLong(qsa_store_paged_kv(&d, k.data_ptr(), 2 * step_of(k, 0), 2 * step_of(k, 1), v.data_ptr(),
                                              2 * step_of(v, 0), 2 * step_of(v, 1), slots.data_ptr<int64_t>(), T,
                                              kc.data_ptr(), vc.data_ptr(), place.stream()));
  });
}

// (keys, slots, kv_cache, page_cols, kv_dtype, scale_offset) -> status
PyObject* store_index_keys(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 6);
    const at::Tensor &keys = tensor(a[0], "keys"), &slots = tensor(a[1], "slots"), &cache = tensor(a[2], "kv_cache");
    vec(slots, "slots", at::kLong, -1);
    const int64_t T = slots.size(0);
    need(keys.scalar_type() == at::kBFloat16 && keys.dim() == 2 && keys.size(0) == T && step_of(keys, 1) == 1,
         "keys must be bf16 [T, head_dim] with contiguous rows");
    qsa_index_cache_desc d = {};
    d.page_cols = integer32(a[3], "page_cols");
    d.kv_dtype = integer32(a[4], "kv_dtype");
    const int64_t off = integer(a[5], "scale_offset");
    const bool fp8 = d.kv_dtype == QSA_KV_FP8_E4M3;
    const int64_t e = (int64_t)cache.element_size();
    need(cache.dim() >= 2, "kv_cache must be [num_pages, ...]");
    need(!fp8 || off >= 0, "fp8 keys need the scale offset inside a block");
    need(fp8 ? e == 1 : cache.scalar_type() == at::kBFloat16,
         "the index cache must be a bf16 tensor, or one of bytes for fp8 keys");
    int64_t inner = 1;  // the elements of a page, and whether they follow one another
    bool dense = true;
    for (int64_t i = cache.dim() - 1; i > 0; --i) {
      dense = dense && (cache.size(i) == 1 || cache.stride(i) == inner);
      inner *= cache.size(i);
    }
    const int64_t keys_end = (int64_t)d.page_cols * keys.size(1) * (fp8 ? 1 : 2);
    need(dense && inner * e >= (fp8 ? off + 4 * (int64_t)d.page_cols : keys_end) && inner * e >= keys_end,
         "a page of kv_cache must be contiguous and hold page_cols keys (and their scales)");
    need(!fp8 || off >= keys_end, "the scales must lie behind the keys of a block");
    d.num_pages = size32(cache.size(0), "num_pages");
    d.head_dim = size32(keys.size(1), "head_dim");
    d.key_page_stride = step_of(cache, 0) * e;
    d.scale_page_stride = fp8 ? d.key_page_stride : 0;
    const Place place(cache);
    place.also(keys), place.also(slots);
    uint8_t* base = static_cast<uint8_t*>(cache.data_ptr());
    return PyLong_FromLong(qsa_store_index_keys(&d, keys.data_ptr(), 2 * step_of(keys, 0), slots.data_ptr<int64_t>(), T,
                                                base, fp8 ? reinterpret_cast<float*>(base + off) : nullptr,
                                                place.stream()));
  });
}

// One a device and stream, guarded by the GIL; never destroyed: the CUDA
// context may be gone before static destructors run.  At most kMaxKept, as many
// as torch's pool has streams of a priority (5 or 43 MB each): then the one
// unused longest goes.  Its memory returns to its own stream, so a call that
// still runs there is not disturbed.
struct Kept {
  at::Tensor ws;
  uint64_t used = 0;
};
constexpr size_t kMaxKept = 32;
std::map<std::pair<int, cudaStream_t>, Kept>& kept_workspaces() {
  static auto* kept = new std::map<std::pair<int, cudaStream_t>, Kept>;
  return *kept;
}

// () -> None: forgets the kept workspaces.
PyObject* drop_workspaces(PyObject*, PyObject* const*, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 0);
    kept_workspaces().clear();
    Py_INCREF(Py_None);
    return Py_None;
  });
}

// The workspace kept for a stream; under graph capture a new one, which the
// graph owns (replays must not meet eager calls in it).  Only its counters
// need zeroing, in stream order.
at::Tensor attention_workspace(size_t bytes, const at::Tensor& like, cudaStream_t stream) {
  auto fresh = [&] {
    at::Tensor w = at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
    w.narrow(0, 0, QSA_ATTN_COUNTER_BYTES).zero_();
    return w;
  };
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess) {
    cudaGetLastError();
    throw std::runtime_error("the stream's capture status cannot be read");
  }
  if (cs != cudaStreamCaptureStatusNone) return fresh();
  auto& kept = kept_workspaces();
  static uint64_t calls = 0;
  const std::pair<int, cudaStream_t> key((int)like.device().index(), stream);
  auto at = kept.find(key);
  if (at == kept.end() || at->second.ws.numel() < (int64_t)bytes) {
    Kept made;
    made.ws = fresh();
    if (at == kept.end() && kept.size() >= kMaxKept) {
      auto oldest = kept.begin();
      for (auto i = kept.begin(); i != kept.end(); ++i)
        if (i->second.used < oldest->second.used) oldest = i;
      kept.erase(oldest);
    }
    at = kept.insert_or_assign(key, std::move(made)).first;
  }
  at->second.used = ++calls;
  return at->second.ws;
}

// (q, k_cache, v_cache, block_table, query_start, seq_lens, scale or None, max_new, selected or None, ratio,
//  local_tokens, form, out or None, lse or None, return_lse, workspace or None, window, sink_tokens)
//  -> (status, out, lse or None)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 18);
    const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"),
                     &bt = tensor(a[3], "block_table"), &qs = tensor(a[4], "query_start"),
                     &sl = tensor(a[5], "seq_lens");
    qsa_attn_desc d = {};
    d.kv = kv_desc(kc, vc);
    need(q.dim() == 3 && q.scalar_type() == kc.scalar_type() && step_of(q, 2) == 1,
         "q must be [T, num_q_heads, head_dim] in the caches' type, last dimension contiguous");
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    need(D == kc.size(3), "q and the caches differ in head_dim");
    table(bt);
    const int64_t B = bt.size(0);
    vec(qs, "query_start", at::kInt, B + 1);
    vec(sl, "seq_lens", at::kInt, B);
    const Place place(q);
    place.also(kc), place.also(vc), place.also(bt), place.also(qs), place.also(sl);
    const int32_t* sel = nullptr;
    if (given(a[8])) {
      const at::Tensor& s = tensor(a[8], "selected");
      need(s.scalar_type() == at::kInt && s.dim() == 2 && s.is_contiguous() && s.size(0) == T && s.size(1) > 0,
           "selected must be a contiguous int32 [T, k] tensor, k > 0");
      place.also(s);
      d.num_selected = size32(s.size(1), "k");
      sel = s.data_ptr<int32_t>();
    }
    d.num_requests = size32(B, "num_requests");
    d.num_q_heads = size32(H, "num_q_heads");
    d.max_pages = size32(bt.size(1), "max_pages");
    d.max_new = integer32(a[7], "max_new");
    d.ratio = integer32(a[9], "ratio");
    d.local_tokens = integer32(a[10], "local_tokens");
    d.form = integer32(a[11], "form");
    const int32_t window = integer32(a[16], "window"), sinks = integer32(a[17], "sink_tokens");
    d.num_tokens = T;
    d.table_stride = step_of(bt, 0);
    d.q_token_stride = 2 * step_of(q, 0);
    d.q_head_stride = 2 * step_of(q, 1);
    if (given(a[6])) {
      const double s = PyFloat_AsDouble(a[6]);
      if (s == -1.0 && PyErr_Occurred()) return nullptr;
      d.scale = (float)s;
    } else {
      d.scale = (float)(1.0 / std::sqrt((double)(D > 0 ? D : 1)));
    }
    at::Tensor out, lse, ws;
    if (given(a[12])) {
      out = tensor(a[12], "out");
      need(out.sizes() == q.sizes() && out.scalar_type() == q.scalar_type() && step_of(out, 2) == 1,
           "out must have q's shape and type, last dimension contiguous");
      place.also(out);
    } else {
      out = at::empty({T, H, D}, q.options());
    }
    if (given(a[13])) {
      lse = tensor(a[13], "lse");
      need(lse.scalar_type() == at::kFloat && lse.dim() == 2 && lse.is_contiguous() && lse.size(0) == T &&
               lse.size(1) == H,
           "lse must be a contiguous fp32 [T, num_q_heads] tensor");
      place.also(lse);
    } else if (truth(a[14], "return_lse")) {
      lse = at::empty({T, H}, q.options().dtype(at::kFloat));
    }
    d.out_token_stride = 2 * step_of(out, 0);
    d.out_head_stride = 2 * step_of(out, 1);
    size_t bytes = 0;
    qsa_status st = qsa_paged_attention_workspace(&d, &bytes);
    if (st == QSA_OK) {
      const cudaStream_t stream = place.stream();
      if (given(a[15])) {
        ws = tensor(a[15], "workspace");
        need(ws.is_contiguous(), "workspace must be contiguous");
        place.also(ws);
      } else if (B > 0 && T > 0) {
        ws = attention_workspace(bytes, q, stream);
      }
      float* const z = lse.defined() ? lse.data_ptr<float>() : nullptr;
      void* const w = ws.defined() ? ws.data_ptr() : nullptr;
      const size_t have = ws.defined() ? ws.nbytes() : 0;
      if (window != 0 || sinks != 0) {
        need(sel == nullptr, "a window takes no selected columns");
        st = qsa_paged_attention_window(&d, window, sinks, q.data_ptr(), kc.data_ptr(), vc.data_ptr(),
                                        bt.data_ptr<int32_t>(), qs.data_ptr<int32_t>(), sl.data_ptr<int32_t>(),
                                        out.data_ptr(), z, w, have, stream);
      } else {
        st = qsa_paged_attention(&d, q.data_ptr(), kc.data_ptr(), vc.data_ptr(), bt.data_ptr<int32_t>(),
                                 qs.data_ptr<int32_t>(), sl.data_ptr<int32_t>(), sel, out.data_ptr(), z, w, have,
                                 stream);
      }
    }
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(st));
    PyTuple_SET_ITEM(r, 1, wrap(out));
    if (lse.defined()) {
      PyTuple_SET_ITEM(r, 2, wrap(lse));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(r, 2, Py_None);
    }
    return r;
  });
}

// What of a call is fp32 where Python gives a number.
float real32(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be a number");
  }
  return (float)v;
}

// A weight or bias vector of head_dim entries: null when not given.  `f32`: -1
// while none of the call's vectors has been seen.
const void* head_vector(PyObject* o, const char* name, const at::Tensor& rows, const Place& place, int& f32) {
  if (!given(o)) return nullptr;
  const at::Tensor& t = tensor(o, name);
  const int is32 = t.scalar_type() == at::kFloat ? 1 : 0;
  if (!(is32 || t.scalar_type() == rows.scalar_type()) || t.dim() != 1 || t.size(0) != rows.size(2) ||
      !t.is_contiguous())
    throw Refused(std::string(name) + " must be a contiguous [head_dim] vector in the rows' type or fp32");
  need(f32 < 0 || f32 == is32, "weights and biases must all be of one type");
  f32 = is32;
  place.also(t);
  return t.data_ptr();
}

void head_rows(const at::Tensor& t, const at::Tensor& q, const char* name) {
  if (t.dim() != 3 || t.scalar_type() != q.scalar_type() || t.size(0) != q.size(0) || t.size(2) != q.size(2) ||
      step_of(t, 2) != 1)
    throw Refused(std::string(name) + " must be [T, heads, head_dim] in q's type, last dimension contiguous");
}

// An output like `like`: the given tensor, or a new one.
at::Tensor output_rows(PyObject* o, const char* name, const at::Tensor& like, const Place& place) {
  if (!given(o)) return at::empty(like.sizes(), like.options());
  const at::Tensor& t = tensor(o, name);
  head_rows(t, like, name);
  if (t.size(1) != like.size(1)) throw Refused(std::string(name) + " must have as many heads as its input");
  place.also(t);
  return t;
}

void strides_of(qsa_head_rows& r, const at::Tensor& x) {
  r.x = x.data_ptr();
  r.x_row_stride = 2 * step_of(x, 0);
  r.x_head_stride = 2 * step_of(x, 1);
  r.num_heads = size32(x.size(1), "heads");
}

// (q, k or None, positions, freqs, layout, offset, magnitude, norm, q_weight, k_weight, q_bias, k_bias, eps,
//  q_out or None, k_out or None, v or None, slots, k_cache, v_cache) -> (status, q_out, k_out or None)
// With v: keys and values go to the caches.
PyObject* rotate_heads(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 19);
    const at::Tensor &q = tensor(a[0], "q"), &pos = tensor(a[2], "positions"), &freqs = tensor(a[3], "freqs");
    need(q.scalar_type() == at::kBFloat16 || q.scalar_type() == at::kHalf, "q must be bf16 or fp16");
    head_rows(q, q, "q");
    const int64_t T = q.size(0);
    vec(pos, "positions", at::kInt, T);
    vec(freqs, "freqs", at::kLong, -1);
    const Place place(q);
    place.also(pos), place.also(freqs);
    qsa_rotary_desc d = {};
    d.dtype = q.scalar_type() == at::kHalf ? QSA_HALF_F16 : QSA_HALF_BF16;
    d.head_dim = size32(q.size(2), "head_dim");
    need(freqs.size(0) < (1 << 20), "freqs is too long");
    d.rot_dim = (int32_t)(2 * freqs.size(0));
    d.layout = integer32(a[4], "layout");
    d.rot_offset = integer32(a[5], "offset");
    d.magnitude = real32(a[6], "magnitude");
    d.norm = integer32(a[7], "norm");
    d.eps = real32(a[12], "eps");
    d.num_tokens = T;
    qsa_head_rows rq = {}, rk = {};
    int f32 = -1;
    strides_of(rq, q);
    rq.weight = head_vector(a[8], "q_weight", q, place, f32);
    rq.bias = head_vector(a[10], "q_bias", q, place, f32);
    const bool has_k = given(a[1]), stored = given(a[15]);
    const at::Tensor* k = nullptr;
    if (has_k) {
      k = &tensor(a[1], "k");
      head_rows(*k, q, "k");
      place.also(*k);
      strides_of(rk, *k);
      rk.weight = head_vector(a[9], "k_weight", q, place, f32);
      rk.bias = head_vector(a[11], "k_bias", q, place, f32);
    } else {
      need(!given(a[9]) && !given(a[11]) && !given(a[14]), "k_weight, k_bias and k_out need k");
    }
    d.weight_f32 = f32 == 1 ? 1 : 0;
    at::Tensor q_out = output_rows(a[13], "q_out", q, place), k_out;
    rq.out = q_out.data_ptr();
    rq.out_row_stride = 2 * step_of(q_out, 0);
    rq.out_head_stride = 2 * step_of(q_out, 1);
    qsa_status st;
    if (stored) {
      need(has_k && !given(a[14]), "the store takes k, and its output is the cache");
      const at::Tensor &v = tensor(a[15], "v"), &slots = tensor(a[16], "slots"), &kc = tensor(a[17], "k_cache"),
                       &vc = tensor(a[18], "v_cache");
      head_rows(v, q, "v");
      need(v.size(1) == k->size(1), "v must have as many heads as k");
      const qsa_kv_desc kv = kv_desc(kc, vc);
      vec(slots, "slots", at::kLong, T);
      place.also(v), place.also(slots), place.also(kc), place.also(vc);
      st = qsa_rotate_store_kv(&d, &rq, &rk, pos.data_ptr<int32_t>(),
                               reinterpret_cast<const uint64_t*>(freqs.data_ptr<int64_t>()), &kv, v.data_ptr(),
                               2 * step_of(v, 0), 2 * step_of(v, 1), slots.data_ptr<int64_t>(), kc.data_ptr(),
                               vc.data_ptr(), place.stream());
    } else {
      if (has_k) {
        k_out = output_rows(a[14], "k_out", *k, place);
        rk.out = k_out.data_ptr();
        rk.out_row_stride = 2 * step_of(k_out, 0);
        rk.out_head_stride = 2 * step_of(k_out, 1);
      }
      st = qsa_rotate_heads(&d, &rq, has_k ? &rk : nullptr, pos.data_ptr<int32_t>(),
                            reinterpret_cast<const uint64_t*>(freqs.data_ptr<int64_t>()), place.stream());
    }
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(st));
    PyTuple_SET_ITEM(r, 1, wrap(q_out));
    if (k_out.defined()) {
      PyTuple_SET_ITEM(r, 2, wrap(k_out));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(r, 2, Py_None);
    }
    return r;
  });
}

int32_t probs_dtype(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return QSA_PROBS_F32;
  if (t.scalar_type() == at::kBFloat16) return QSA_PROBS_BF16;
  if (t.scalar_type() == at::kHalf) return QSA_PROBS_F16;
  throw Refused("probabilities must be fp32, bf16 or fp16");
}

// (draft_tokens, target_probs, uniforms, draft_probs or None, num_drafts or None, context_lens or None,
//  tokens or None, num_accepted or None, next_lens or None) -> (status, tokens, num_accepted, next_lens or None)
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 9);
    const at::Tensor &tok = tensor(a[0], "draft_tokens"), &p = tensor(a[1], "target_probs"),
                     &u = tensor(a[2], "uniforms");
    need(tok.dim() == 2 && tok.scalar_type() == at::kInt && tok.is_contiguous(),
         "draft_tokens must be a contiguous int32 [B, K] tensor");
    const int64_t B = tok.size(0), K = tok.size(1);
    need(p.dim() == 3 && p.size(0) == B && p.size(1) == K + 1 && step_of(p, 2) == 1,
         "target_probs must be [B, K + 1, V], last dimension contiguous");
    need(u.dim() == 2 && u.scalar_type() == at::kFloat && u.is_contiguous() && u.size(0) == B && u.size(1) == K + 1,
         "uniforms must be a contiguous fp32 [B, K + 1] tensor");
    const Place place(p);
    place.also(tok), place.also(u);
    qsa_verify_desc d = {};
    d.num_requests = size32(B, "B");
    d.max_drafts = size32(K, "K");
    d.vocab = size32(p.size(2), "V");
    d.dtype = probs_dtype(p);
    d.target_request_stride = step_of(p, 0);
    d.target_row_stride = step_of(p, 1);
    const void* q = nullptr;
    if (given(a[3])) {
      const at::Tensor& t = tensor(a[3], "draft_probs");
      need(t.dim() == 3 && t.scalar_type() == p.scalar_type() && t.size(0) == B && t.size(1) == K &&
               t.size(2) == p.size(2) && step_of(t, 2) == 1,
           "draft_probs must be [B, K, V] in target_probs' type, last dimension contiguous");
      place.also(t);
      d.draft_request_stride = step_of(t, 0);
      d.draft_row_stride = step_of(t, 1);
      q = t.data_ptr();
    }
    auto ints = [&](PyObject* o, const char* name) -> int32_t* {
      if (!given(o)) return nullptr;
      const at::Tensor& t = tensor(o, name);
      vec(t, name, at::kInt, B);
      place.also(t);
      return t.data_ptr<int32_t>();
    };
    const int32_t *num = ints(a[4], "num_drafts"), *ctx = ints(a[5], "context_lens");
    need(given(a[5]) || !given(a[8]), "next_lens needs context_lens");
    at::Tensor out[3], fresh;
    const int64_t row = (B * 4 + 15) & ~int64_t(15);  // bytes of a [B] output; new ones share an allocation
    if (!given(a[6]) || !given(a[7]) || (given(a[5]) && !given(a[8])))
      fresh = at::empty({2 * row + B * (K + 1) * 4}, tok.options().dtype(at::kByte));
    if (given(a[6])) {
      out[0] = tensor(a[6], "tokens");
      need(out[0].dim() == 2 && out[0].scalar_type() == at::kInt && out[0].is_contiguous() && out[0].size(0) == B &&
               out[0].size(1) == K + 1,
           "tokens must be a contiguous int32 [B, K + 1] tensor");
      place.also(out[0]);
    } else {
      out[0] = slice_of(fresh, at::kInt, 2 * row, {B, K + 1});
    }
    for (int i = 1; i < 3; ++i) {
      if (i == 2 && !given(a[5])) break;
      if (given(a[6 + i])) {
        ints(a[6 + i], i == 1 ? "num_accepted" : "next_lens");
        out[i] = tensor(a[6 + i], "");
      } else {
        out[i] = slice_of(fresh, at::kInt, (i - 1) * row, {B});
      }
    }
    const qsa_status st =
        qsa_verify_drafts(&d, tok.data_ptr<int32_t>(), num, p.data_ptr(), q, u.data_ptr<float>(), ctx,
                          out[0].data_ptr<int32_t>(), out[1].data_ptr<int32_t>(),
                          out[2].defined() ? out[2].data_ptr<int32_t>() : nullptr, place.stream());
    PyObject* r = PyTuple_New(4);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(st));
    for (int i = 0; i < 3; ++i) {
      if (out[i].defined()) {
        PyTuple_SET_ITEM(r, i + 1, wrap(out[i]));
      } else {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(r, i + 1, Py_None);
      }
    }
    return r;
  });
}

template <typename F>
constexpr PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"build_page_maps", fast(build_page_maps), METH_FASTCALL, nullptr},
    {"store_paged_kv", fast(store_paged_kv), METH_FASTCALL, nullptr},
    {"store_index_keys", fast(store_index_keys), METH_FASTCALL, nullptr},
    {"paged_attention", fast(paged_attention), METH_FASTCALL, nullptr},
    {"rotate_heads", fast(rotate_heads), METH_FASTCALL, nullptr},
    {"verify_drafts", fast(verify_drafts), METH_FASTCALL, nullptr},
    {"drop_workspaces", fast(drop_workspaces), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qsa_torch", "torch-tensor entries of the serving operators", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qsa_torch(void) { return PyModule_Create(&module); }
