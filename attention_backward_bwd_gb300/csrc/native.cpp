// Argument marshalling of cache8.py and pages.py: the checks of tensors, the outputs that a call
// allocates itself (on the current stream) and the call of the C ABI (include/attn_cache8.h).
// In C++, since a call on a few tokens runs for a few microseconds on the GPU: a decode of one
// short sequence took 22 us of a host's time marshalled in Python, and takes 5 here.  No computation
// is done here.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/CUDAContext.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/attn_cache8.h"

namespace {

// Entry points of libattn_gb300.so, handed over by bind().
struct Api {
  decltype(&attn_cache_append8) append8;
  decltype(&attn_cache_load8) load8;
  decltype(&attn_decode8) decode8;
  decltype(&attn_decode_workspace_size) decode_size;
  decltype(&attn_cache_fork) fork;
  decltype(&attn_cache_fork_workspace_size) fork_size;
  decltype(&attn_cache_copy) copy;
  decltype(&attn_last_error) last_error;
} api;
PyObject* g_error = nullptr;  // AttnError

struct Refused {
  int code;
  std::string text;
};
struct Raised {};  // a Python exception is set

template <typename... A>
[[noreturn]] void refuse(int code, const A&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw Refused{code, s.str()};
}

std::string shape(const at::Tensor& t) {
  std::ostringstream s;
  s << t.sizes();
  return s.str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(-9, name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* name) {
  PyObject* n = PyNumber_Index(o);
  if (n == nullptr) throw Raised();
  int over = 0;
  const int64_t v = PyLong_AsLongLongAndOverflow(n, &over);
  Py_DECREF(n);
  if (over == 0 && v == -1 && PyErr_Occurred()) throw Raised();
  if (over != 0 || v < INT32_MIN || v > INT32_MAX) refuse(-9, name, " does not fit 32 bits");
  return v;
}
int int32(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(-9, name, " (", v, ") does not fit 32 bits");
  return static_cast<int>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}

// What the tensors of a call share.
struct Place {
  int index;             // of the device
  at::ScalarType dtype;  // of q, k and v
  int code;
};
int code_of(at::ScalarType t) { return t == at::kHalf ? ATTN_FP16 : (t == at::kBFloat16 ? ATTN_BF16 : -1); }

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(-9, name, " must be a CUDA tensor, got ", t.device().str());
  return t.get_device();
}
Place first(const at::Tensor& t, const char* name) {
  const int code = code_of(t.scalar_type());
  if (code < 0) refuse(-1, name, " must be float16 or bfloat16, got ", t.scalar_type());
  return {device_of(t, name), t.scalar_type(), code};
}

void on(const at::Tensor& t, const char* name, int index) {
  if (!t.is_cuda() || t.get_device() != index)
    refuse(-9, name, " must be a CUDA tensor on cuda:", index, ", got ", t.device().str());
}

// A tensor of head rows: device, type, rank, unit stride over the head dimension.
attn_tensor rows(const at::Tensor& t, const char* name, int index, at::ScalarType dtype, int dims) {
  on(t, name, index);
  if (t.scalar_type() != dtype) refuse(-1, name, " has dtype ", t.scalar_type(), ", ", dtype, " was expected");
  if (t.dim() != dims) refuse(-2, name, " must have ", dims, " dimensions, got ", shape(t));
  if (t.stride(dims - 1) != 1 && t.numel() > 0) refuse(-3, name, " must have unit stride over the head dimension");
  return attn_tensor{t.data_ptr(), dims == 4 ? t.stride(0) : 0, t.stride(dims - 3), t.stride(dims - 2)};
}

// Pointer of a contiguous int32 tensor of n entries (None: none).
int* ints(PyObject* o, const char* name, int index, int64_t n) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(-9, name, " must be a contiguous int32 tensor [", n, "] on cuda:", index, ", got ", t.scalar_type(), " ", shape(t),
           " on ", t.device().str());
  return t.data_ptr<int>();
}
int* some_ints(PyObject* o, const char* name, int index, int64_t n) {
  if (o == Py_None) refuse(-9, name, " must be given");
  return ints(o, name, index, n);
}

int64_t batch_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 1) refuse(-9, name, " must be a 1-D int32 tensor, got ", shape(t));
  return t.size(0);
}

struct Cache8 {
  attn_paged_kv8 c;
  int64_t heads, dim, slots;
};

void factors(attn_paged_kv8* c, PyObject* k, PyObject* v, const at::Tensor& codes, int index, int kind) {
  const at::Tensor& ks = tensor(k, "k_scale");
  const at::Tensor& vs = tensor(v, "v_scale");
  const int64_t pages = codes.size(0), size = codes.size(1), heads = codes.size(2);
  const char* name = "k_scale";
  for (const at::Tensor* t : {&ks, &vs}) {
    if (!t->is_cuda() || t->get_device() != index || t->scalar_type() != at::kFloat || t->dim() != 3 || t->size(0) != pages ||
        t->size(2) != heads || t->size(1) < 1 || size % t->size(1) != 0)
      refuse(-9, name, " must be a float32 tensor [", pages, ", blocks of a page of ", size, ", ", heads, "] on cuda:", index,
             ", got ", t->scalar_type(), " ", shape(*t), " on ", t->device().str());
    name = "v_scale";
  }
  if (ks.size(1) != vs.size(1)) refuse(-2, "v_scale has shape ", shape(vs), ", k_scale ", shape(ks));
  c->k_scale = ks.data_ptr<float>();
  c->v_scale = vs.data_ptr<float>();
  c->k_scale_page = ks.stride(0);
  c->k_scale_block = ks.stride(1);
  c->k_scale_head = ks.stride(2);
  c->v_scale_page = vs.stride(0);
  c->v_scale_block = vs.stride(1);
  c->v_scale_head = vs.stride(2);
  c->block = int32(size / ks.size(1), "the block");
  c->kind = kind;
}

int kind_of(at::ScalarType t) { return t == at::kFloat8_e4m3fn ? ATTN_E4M3 : (t == at::kChar ? ATTN_INT8 : -1); }

// Keys and values of a paged cache.
void pages_of(attn_paged_kv* kv, const at::Tensor& kc, const at::Tensor& vc, int index) {
  kv->k = rows(kc, "k_cache", index, kc.scalar_type(), 4);
  kv->v = rows(vc, "v_cache", index, kc.scalar_type(), 4);
  if (vc.sizes() != kc.sizes()) refuse(-2, "v_cache has shape ", shape(vc), ", k_cache ", shape(kc));
  kv->num_pages = int32(kc.size(0), "the pages' number");
  kv->page_size = int32(kc.size(1), "the page's size");
}

Cache8 cache8(PyObject* const* a, PyObject* table_, int index, int64_t batch) {  // k_cache, v_cache, k_scale, v_scale
  const at::Tensor& kc = tensor(a[0], "k_cache");
  const at::Tensor& vc = tensor(a[1], "v_cache");
  const int kind = kind_of(kc.scalar_type());
  if (kind < 0) refuse(-1, "k_cache must be float8_e4m3fn or int8, got ", kc.scalar_type());
  Cache8 r = {};
  pages_of(&r.c.kv, kc, vc, index);
  const at::Tensor& table = tensor(table_, "block_table");
  if (!table.is_cuda() || table.get_device() != index || table.scalar_type() != at::kInt || table.dim() != 2 ||
      table.size(0) != batch || (table.size(1) > 1 && table.stride(1) != 1))
    refuse(-9, "block_table must be an int32 tensor [", batch, ", pages] on cuda:", index, " with contiguous rows, got ",
           table.scalar_type(), " ", shape(table), " on ", table.device().str());
  r.c.kv.block_table = table.data_ptr<int>();
  r.c.kv.table_stride = table.stride(0);
  r.c.kv.max_pages = int32(table.size(1), "the pages of a sequence");
  factors(&r.c, a[2], a[3], kc, index, kind);
  r.heads = kc.size(2);
  r.dim = kc.size(3);
  r.slots = table.size(1) * kc.size(1);
  return r;
}

// Rotary positions of [tokens]; false: none.
bool rotary(attn_rotary* r, PyObject* positions, PyObject* inv, PyObject* sections, PyObject* interleaved, int index, int64_t tokens) {
  if ((positions == Py_None) != (inv == Py_None)) refuse(-9, "positions and inv_freq go together");
  if (positions == Py_None) return false;
  const at::Tensor& f = tensor(inv, "inv_freq");
  if (!f.is_cuda() || f.get_device() != index || f.scalar_type() != at::kFloat || f.dim() != 1 || !f.is_contiguous())
    refuse(-9, "inv_freq must be a contiguous 1-D float32 tensor on cuda:", index);
  *r = attn_rotary{};
  r->n_freq = int32(f.size(0), "inv_freq's number");
  r->n_axes = 1;
  r->sections[0] = r->n_freq;
  if (sections != Py_None) {
    PyObject* seq = PySequence_Fast(sections, "sections must be a sequence");
    if (seq == nullptr) throw Raised();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    try {
      if (n < 1 || n > 4) refuse(-2, "sections must name 1 to 4 axes, got ", n);
      for (Py_ssize_t i = 0; i < n; ++i) r->sections[i] = static_cast<int>(integer(PySequence_Fast_GET_ITEM(seq, i), "a section"));
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
    Py_DECREF(seq);
    r->n_axes = static_cast<int>(n);
  }
  const at::Tensor& pos = tensor(positions, "positions");
  const bool fits = (pos.dim() == 2 && pos.size(0) == r->n_axes && pos.size(1) == tokens) ||
                    (r->n_axes == 1 && pos.dim() == 1 && pos.size(0) == tokens);
  if (!fits) refuse(-2, "positions must be [", r->n_axes, ", ", tokens, "], got ", shape(pos));
  if (!pos.is_cuda() || pos.get_device() != index || pos.scalar_type() != at::kInt || !pos.is_contiguous())
    refuse(-9, "positions must be a contiguous int32 tensor on cuda:", index, ", got ", pos.scalar_type(), " on ", pos.device().str());
  r->positions = pos.data_ptr<int>();
  r->axis_stride = tokens;
  r->inv_freq = f.data_ptr<float>();
  const int truth = PyObject_IsTrue(interleaved);
  if (truth < 0) throw Raised();
  r->interleaved = truth;
  return true;
}

// A new contiguous tensor beside `like` (without the dispatcher: a microsecond less each).
at::Tensor fresh(at::IntArrayRef size, at::ScalarType dtype, const at::Tensor& like) {
  return at::detail::empty_cuda(size, dtype, like.device(), std::nullopt);
}

// An output of x's shape: allocated, or checked against it.
at::Tensor output(PyObject* o, const char* name, const at::Tensor& x, int index, int dims, attn_tensor* arg) {
  at::Tensor out = o == Py_None ? fresh(x.sizes(), x.scalar_type(), x) : tensor(o, name);
  *arg = rows(out, name, index, x.scalar_type(), dims);
  if (out.sizes() != x.sizes()) refuse(-2, name, " has shape ", shape(out), ", its input ", shape(x));
  if (out.data_ptr() == x.data_ptr() && out.strides() != x.strides() && out.numel() > 0)
    refuse(-9, name, " starts where its input does but has other strides");
  return out;
}

// (pointer, bytes) of the caller's workspace, or of a new one that `held` keeps until the call is queued.
void* workspace(PyObject* o, size_t need, const at::Tensor& like, int index, size_t* bytes, at::Tensor* held) {
  *bytes = 0;
  if (o == Py_None) {
    if (need == 0) return nullptr;
    *held = fresh({static_cast<int64_t>(need)}, at::kByte, like);
  } else {
    const at::Tensor& t = tensor(o, "workspace");
    if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != at::kByte || !t.is_contiguous())
      refuse(-9, "workspace must be a contiguous uint8 tensor on cuda:", index);
    *held = t;
  }
  *bytes = static_cast<size_t>(held->numel());
  return held->data_ptr();
}

// Runs f(stream) with device `index` current; stream: None or a handle.
template <typename F>
void call(int index, PyObject* stream, F f) {
  attn_stream_t s;
  if (stream == Py_None) {
    s = reinterpret_cast<attn_stream_t>(at::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
  } else {
    const unsigned long long h = PyLong_AsUnsignedLongLong(stream);
    if (PyErr_Occurred()) throw Raised();
    s = reinterpret_cast<attn_stream_t>(static_cast<uintptr_t>(h));
  }
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != index) guard.set_index(static_cast<c10::DeviceIndex>(index));
  int rc;
  std::string text;
  Py_BEGIN_ALLOW_THREADS
  rc = f(s);
  if (rc != 0) text = api.last_error();
  Py_END_ALLOW_THREADS
  if (rc != 0) throw Refused{rc, text};
}

PyObject* raised(int code, const std::string& text) {
  PyObject* e = PyObject_CallFunction(g_error, "is", code, text.c_str());
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// Runs f() and turns what it throws into a Python exception.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", wanted, given);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    return raised(r.code, r.text);
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* none() { Py_RETURN_NONE; }
PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (r == nullptr) throw Raised();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (o == nullptr) {
      Py_DECREF(r);
      throw Raised();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// k, v, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, cu_seqlens, q, positions, inv_freq,
// sections, interleaved, out_q, stream
PyObject* append8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const at::Tensor& k = tensor(a[0], "k");
    const at::Tensor& v = tensor(a[1], "v");
    const Place where = first(k, "k");
    const attn_tensor ka = rows(k, "k", where.index, where.dtype, 3), va = rows(v, "v", where.index, where.dtype, 3);
    const int64_t tokens = k.size(0), hk = k.size(1), d = k.size(2);
    if (v.sizes() != k.sizes()) refuse(-2, "v has shape ", shape(v), ", k ", shape(k));
    const int64_t batch = batch_of(a[7], "seqlens");
    int32(tokens, "the tokens' number");
    const int* lens = some_ints(a[7], "seqlens", where.index, batch);
    const Cache8 c = cache8(a + 2, a[6], where.index, batch);
    if (c.heads != hk || c.dim != d) refuse(-2, "k ", shape(k), " does not fit a cache of ", c.heads, " heads of ", c.dim);
    const int* cu = ints(a[8], "cu_seqlens", where.index, batch + 1);
    if (cu == nullptr && tokens != batch)
      refuse(-9, "without cu_seqlens there is one token a sequence: ", tokens, " tokens, ", batch, " sequences");
    attn_rotary rot;
    const bool turn = rotary(&rot, a[10], a[11], a[12], a[13], where.index, tokens);
    attn_tensor qa = {}, oa = {};
    at::Tensor out;
    int64_t hq = hk;
    if (a[9] != Py_None) {
      if (!turn) refuse(-9, "q is only taken to be rotated: give positions and inv_freq, or no q");
      const at::Tensor& q = tensor(a[9], "q");
      qa = rows(q, "q", where.index, where.dtype, 3);
      hq = q.size(1);
      if (q.size(0) != tokens || q.size(2) != d) refuse(-2, "q ", shape(q), " and k ", shape(k), " disagree on tokens or D");
      out = output(a[14], "out_q", q, where.index, 3, &oa);
    } else if (a[14] != Py_None) {
      refuse(-9, "out_q without q");
    }
    if (tokens > 0)
      call(where.index, a[15], [&](attn_stream_t s) {
        return api.append8(out.defined() ? &qa : nullptr, out.defined() ? &oa : nullptr, &ka, &va, where.code, static_cast<int>(tokens),
                           static_cast<int>(batch), static_cast<int>(hq), static_cast<int>(hk), static_cast<int>(d), &c.c, lens, cu,
                           turn ? &rot : nullptr, s);
      });
    return out.defined() ? wrap(out) : none();
  });
}

// k_cache, v_cache, k_scale, v_scale, block_table, starts, cu_seqlens, tokens, out_k, out_v, dtype like (code), stream
PyObject* load8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor& kc = tensor(a[0], "k_cache");
    const int index = device_of(kc, "k_cache");
    const int64_t code = integer(a[10], "dtype");
    const at::ScalarType dtype = code == ATTN_BF16 ? at::kBFloat16 : at::kHalf;
    const int64_t batch = batch_of(a[5], "starts"), tokens = integer(a[7], "tokens");
    if (tokens < 0) refuse(-2, "tokens must be >= 0, got ", tokens);
    const int* starts = some_ints(a[5], "starts", index, batch);
    const int* cu = some_ints(a[6], "cu_seqlens", index, batch + 1);
    const Cache8 c = cache8(a, a[4], index, batch);
    at::Tensor out[2];
    attn_tensor arg[2];
    const char* names[2] = {"out_k", "out_v"};
    for (int i = 0; i < 2; ++i) {
      if (a[8 + i] == Py_None) {
        out[i] = fresh({tokens, c.heads, c.dim}, dtype, kc);
      } else {
        out[i] = tensor(a[8 + i], names[i]);
        if (out[i].sizes() != at::IntArrayRef({tokens, c.heads, c.dim}))
          refuse(-2, names[i], " has shape ", shape(out[i]), ", [", tokens, ", ", c.heads, ", ", c.dim, "] was expected");
      }
      arg[i] = rows(out[i], names[i], index, dtype, 3);
    }
    if (tokens > 0 && batch > 0)
      call(index, a[11], [&](attn_stream_t s) {
        return api.load8(&arg[0], &arg[1], static_cast<int>(code), static_cast<int>(tokens), static_cast<int>(batch),
                         static_cast<int>(c.heads), static_cast<int>(c.dim), &c.c, starts, cu, s);
      });
    return tuple({out[0], out[1]});
  });
}

// q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, max_seqlen, scale, window, softcap, out, lse,
// workspace, stream
PyObject* decode8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const Place where = first(q, "q");
    const attn_tensor qp = rows(q, "q", where.index, where.dtype, 3);
    const int64_t batch = q.size(0), hq = q.size(1), d = q.size(2);
    const Cache8 c = cache8(a + 1, a[5], where.index, batch);
    if (c.dim != d || c.heads == 0 || hq % c.heads != 0)
      refuse(-2, "q ", shape(q), " does not fit a cache of ", c.heads, " heads of ", c.dim);
    const int* lens = some_ints(a[6], "seqlens", where.index, batch);
    const int most = a[7] == Py_None ? int32(c.slots, "max_seqlen") : static_cast<int>(integer(a[7], "max_seqlen"));
    const float scale = a[8] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(d))) : static_cast<float>(number(a[8]));
    attn_opts opts = {};
    opts.window_left = opts.window_right = -1;
    if (a[9] != Py_None)
      for (int i = 0; i < 2; ++i) {
        PyObject* w = PySequence_GetItem(a[9], i);
        if (w == nullptr) throw Raised();
        int side;
        try {
          side = static_cast<int>(integer(w, "a side of the window"));
        } catch (...) {
          Py_DECREF(w);
          throw;
        }
        Py_DECREF(w);
        (i == 0 ? opts.window_left : opts.window_right) = side;
      }
    opts.softcap = a[10] == Py_None ? 0.f : static_cast<float>(number(a[10]));
    attn_tensor qa, oa;
    at::Tensor out = output(a[11], "out", q, where.index, 3, &oa);
    qa = attn_tensor{qp.ptr, qp.stride_s, 0, qp.stride_h};  // [B, H, D]
    oa = attn_tensor{oa.ptr, oa.stride_s, 0, oa.stride_h};
    at::Tensor lse;
    if (a[12] == Py_None) {
      lse = fresh({batch, hq}, at::kFloat, q);
    } else {
      lse = tensor(a[12], "lse");
      if (!lse.is_cuda() || lse.get_device() != where.index || lse.scalar_type() != at::kFloat || lse.dim() != 2 ||
          lse.size(0) != batch || lse.size(1) != hq || !lse.is_contiguous())
        refuse(-2, "lse must be a contiguous float32 tensor [", batch, ", ", hq, "] on cuda:", where.index);
    }
    if (batch > 0) {
      size_t bytes;
      at::Tensor held;
      const size_t need = api.decode_size(static_cast<int>(batch), static_cast<int>(hq), static_cast<int>(c.heads), static_cast<int>(d), most, 0);
      void* ws = workspace(a[13], need, q, where.index, &bytes, &held);
      call(where.index, a[14], [&](attn_stream_t s) {
        return api.decode8(&qa, &oa, lse.data_ptr<float>(), where.code, static_cast<int>(batch), static_cast<int>(hq),
                           static_cast<int>(c.heads), static_cast<int>(d), scale, &c.c, lens, most, &opts, ws, bytes, s);
      });
    }
    return tuple({out, lse});
  });
}

const at::Tensor& table_of(PyObject* o, const char* name, int index) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != at::kInt || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
    refuse(-9, name, " must be an int32 tensor [rows, pages] on cuda:", index, " with contiguous rows, got ", t.scalar_type(), " ",
           shape(t), " on ", t.device().str());
  return t;
}

// block_table, seqlens, refs, page_size, parents, room, share, table_out, seqlens_out, refs_out, copies, counts,
// workspace, stream
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const int index = device_of(tensor(a[0], "block_table"), "block_table");
    const at::Tensor& table = table_of(a[0], "block_table", index);
    const int64_t rows = table.size(0), width = table.size(1), pages = batch_of(a[2], "refs");
    PyObject* to[3] = {a[7] == Py_None ? a[0] : a[7], a[8] == Py_None ? a[1] : a[8], a[9] == Py_None ? a[2] : a[9]};
    const at::Tensor& out = table_of(to[0], "table_out", index);
    if (out.sizes() != table.sizes()) refuse(-9, "table_out has shape ", shape(out), ", block_table ", shape(table));
    const int *lens = some_ints(a[1], "seqlens", index, rows), *refs = some_ints(a[2], "refs", index, pages);
    int *lens_out = some_ints(to[1], "seqlens_out", index, rows), *refs_out = some_ints(to[2], "refs_out", index, pages);
    const int size = static_cast<int>(integer(a[3], "page_size"));
    const int* parents = ints(a[4], "parents", index, rows);
    const int* room = nullptr;
    int room_all = 0;
    if (THPVariable_Check(a[5])) room = ints(a[5], "room", index, rows);
    else room_all = static_cast<int>(integer(a[5], "room"));
    const int share = PyObject_IsTrue(a[6]);
    if (share < 0) throw Raised();
    int32(rows, "the rows' number");
    int32(width, "the pages of a sequence");
    int32(pages, "the pages' number");
    if (rows * width > INT32_MAX) refuse(-2, "the table must have less than 2^31 entries");
    const int64_t most = share ? rows : rows * width;
    at::Tensor copies, counts;
    if (a[10] == Py_None) {
      copies = fresh({most, 2}, at::kInt, table);
    } else {
      copies = tensor(a[10], "copies");
      if (!copies.is_cuda() || copies.get_device() != index || copies.scalar_type() != at::kInt || copies.dim() != 2 ||
          copies.size(1) != 2 || copies.size(0) < most || !copies.is_contiguous())
        refuse(-9, "copies must be a contiguous int32 tensor [>= ", most, ", 2] on cuda:", index, ", got ", copies.scalar_type(), " ",
               shape(copies), " on ", copies.device().str());
    }
    if (a[11] == Py_None) {
      counts = fresh({2}, at::kInt, table);
    } else {
      ints(a[11], "counts", index, 2);
      counts = tensor(a[11], "counts");
    }
    size_t bytes;
    at::Tensor held;
    const size_t need = api.fork_size(static_cast<int>(rows), static_cast<int>(width), static_cast<int>(pages));
    void* ws = workspace(a[12], need, table, index, &bytes, &held);
    call(index, a[13], [&](attn_stream_t s) {
      return api.fork(table.data_ptr<int>(), table.stride(0), out.data_ptr<int>(), out.stride(0), lens, lens_out, refs, refs_out,
                      static_cast<int>(pages), static_cast<int>(rows), static_cast<int>(width), size, parents, room, room_all, share,
                      copies.data_ptr<int>(), counts.data_ptr<int>(), ws, bytes, s);
    });
    return tuple({out, tensor(to[1], "seqlens_out"), tensor(to[2], "refs_out"), copies, counts});
  });
}

// k_cache, v_cache, pairs, counts, k_scale, v_scale, stream
PyObject* copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const at::Tensor& kc = tensor(a[0], "k_cache");
    const int index = device_of(kc, "k_cache"), kind = kind_of(kc.scalar_type());
    const bool eight = kind >= 0;
    if (!eight && code_of(kc.scalar_type()) < 0)
      refuse(-1, "k_cache must be float16, bfloat16, float8_e4m3fn or int8, got ", kc.scalar_type());
    attn_paged_kv8 c = {};
    pages_of(&c.kv, kc, tensor(a[1], "v_cache"), index);
    if (eight != (a[4] != Py_None) || eight != (a[5] != Py_None)) refuse(-9, "k_scale and v_scale belong to a cache in 8 bits");
    const at::Tensor& pairs = tensor(a[2], "pairs");
    if (!pairs.is_cuda() || pairs.get_device() != index || pairs.scalar_type() != at::kInt || pairs.dim() != 2 || pairs.size(1) != 2 ||
        !pairs.is_contiguous())
      refuse(-9, "pairs must be a contiguous int32 tensor [N, 2] on cuda:", index, ", got ", pairs.scalar_type(), " ", shape(pairs),
             " on ", pairs.device().str());
    const int* count = nullptr;
    if (a[3] != Py_None) {
      const at::Tensor& t = tensor(a[3], "counts");
      if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != at::kInt || t.numel() < 1)
        refuse(-9, "counts must be an int32 tensor on cuda:", index, ", got ", t.scalar_type(), " on ", t.device().str());
      count = t.data_ptr<int>();
    }
    if (eight) factors(&c, a[4], a[5], kc, index, kind);
    const int number = int32(pairs.size(0), "the pairs' number");
    const int heads = int32(kc.size(2), "the heads' number"), dim = int32(kc.size(3), "the head dimension");
    call(index, a[6], [&](attn_stream_t s) {
      return api.copy(&c, eight ? 1 : 2, heads, dim, pairs.data_ptr<int>(), count, number, s);
    });
    return none();
  });
}

// AttnError, and the addresses of the entry points in the order of Api.
PyObject* bind(PyObject*, PyObject* args) {
  PyObject* error;
  unsigned long long p[8];
  if (!PyArg_ParseTuple(args, "OKKKKKKKK", &error, &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6], &p[7])) return nullptr;
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  auto to = [](auto& f, unsigned long long at) { f = reinterpret_cast<std::decay_t<decltype(f)>>(static_cast<uintptr_t>(at)); };
  to(api.append8, p[0]);
  to(api.load8, p[1]);
  to(api.decode8, p[2]);
  to(api.decode_size, p[3]);
  to(api.fork, p[4]);
  to(api.fork_size, p[5]);
  to(api.copy, p[6]);
  to(api.last_error, p[7]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<append8>("append8"), method<load8>("load8"), method<decode8>("decode8"), method<fork>("fork"),
                         method<copy>("copy"), {"bind", bind, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
