// Compiled half of the Python binding, for the calls of the decode step around
// the products (paged cache, attention, norm). A decode step issues one of them
// every few microseconds, and on the host cores of a GB300 machine the same
// marshalling through ctypes takes 15 to 35 us a call (torch's current stream
// 3 us, each new tensor 1.5 us, the argument conversions 2 us) against 2 to 4 us
// of launch. Here tensors are read through torch's C++ types; nothing is computed.
//
// A function checks its tensors (ValueError), allocates the outputs that were not
// given, and calls the C entry point of the same name, whose status other than
// QG_OK is raised as QGError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <map>
#include <string>
#include <tuple>

#include "qgemv.h"

namespace {

PyObject* g_raise = nullptr;  // Python callable (status, name) that raises QGError

struct Refused {  // becomes a ValueError
  std::string why;
};
struct Raised {};  // a Python exception is set

[[noreturn]] void refuse(const std::string& why) { throw Refused{why}; }

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor* tensor_or_null(PyObject* o, const char* name) { return o == Py_None ? nullptr : tensor(o, name); }

long long whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  (void)name;
  return v;
}
int whole32(PyObject* o, const char* name) {
  const long long v = whole(o, name);
  if (v > 0x7FFFFFFFLL || v < -0x80000000LL) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}
int size32(int64_t v, const char* name) {
  if (v > 0x7FFFFFFFLL) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

// A call: its device (the first tensor's), stream and checks.
struct Call {
  c10::Device dev;
  c10::cuda::OptionalCUDAGuard guard;
  c10::cuda::OptionalCUDAStreamGuard on;  // a given stream is the current one while outputs are allocated
  void* stream;
  const char* where;

  Call(const char* name, const at::Tensor& first, PyObject* stream_obj)
      : dev(first.device()), stream(nullptr), where(name) {
    if (!first.is_cuda()) refuse(std::string(name) + ": tensors must be CUDA tensors");
    if (c10::cuda::current_device() != dev.index()) guard.set_device(dev);
    if (stream_obj == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    } else {
      PyObject* h = PyObject_GetAttrString(stream_obj, "cuda_stream");
      if (!h) throw Raised{};
      stream = reinterpret_cast<void*>(PyLong_AsUnsignedLongLong(h));
      Py_DECREF(h);
      if (PyErr_Occurred()) throw Raised{};
      on.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), dev.index()));
    }
  }
  void on_device(const at::Tensor& t, const char* name) const {
    if (t.device() != dev) refuse(std::string(name) + " must be a CUDA tensor on the other tensors' device");
  }
  void dense(const at::Tensor& t, const char* name) const {
    on_device(t, name);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  }
  // dense, of one type and shape (-1: any extent)
  void need(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape, const char* name) const {
    dense(t, name);
    if (t.scalar_type() != type) refuse(std::string(name) + " must be " + c10::toString(type));
    bool ok = t.dim() == static_cast<int64_t>(shape.size());
    int i = 0;
    for (int64_t n : shape) {
      ok = ok && (n < 0 || t.size(i) == n);
      ++i;
    }
    if (!ok) refuse(std::string(name) + " has another shape than the other arguments ask for");
  }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
  }
  // the given output, checked, or none yet (Outputs makes those that are missing)
  at::Tensor output(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, const char* name) const {
    if (o == Py_None) return at::Tensor();
    const at::Tensor& t = *tensor(o, name);
    need(t, type, shape, name);
    return t;
  }
  void done(qg_status s) const {
    if (s == QG_OK) return;
    PyObject* r = PyObject_CallFunction(g_raise, "is", static_cast<int>(s), where);
    Py_XDECREF(r);
    throw Raised{};
  }
};

// The outputs that a call makes. Small ones share one allocation (0.8 us each on
// the host cores, of a call that takes 4); large ones get their own, so that
// one does not keep another's memory.
class Outputs {
 public:
  explicit Outputs(const Call& c) : c_(c) {}
  void add(at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape) {
    if (t.defined()) return;
    Want& w = wants_[n_++];
    w.to = &t;
    w.type = type;
    w.dims = 0;
    w.bytes = c10::elementSize(type);
    for (int64_t d : shape) w.shape[w.dims++] = d, w.bytes *= d;
  }
  void make() {
    size_t total = 0;
    for (int i = 0; i < n_; ++i) total += (wants_[i].bytes + 255) / 256 * 256;
    if (n_ < 2 || total > (1u << 20)) {
      for (int i = 0; i < n_; ++i) *wants_[i].to = c_.make(at::IntArrayRef(wants_[i].shape, wants_[i].dims), wants_[i].type);
      return;
    }
    const at::Tensor base = c_.make({static_cast<int64_t>(total)}, at::kByte);
    size_t at = 0;
    for (int i = 0; i < n_; ++i) {
      const Want& w = wants_[i];
      auto impl = c10::make_intrusive<at::TensorImpl>(c10::Storage(base.storage()), base.key_set(),
                                                      c10::scalarTypeToTypeMeta(w.type));
      impl->set_storage_offset(static_cast<int64_t>(at / c10::elementSize(w.type)));
      impl->set_sizes_contiguous(at::IntArrayRef(w.shape, w.dims));
      *w.to = at::Tensor(std::move(impl));
      at += (w.bytes + 255) / 256 * 256;
    }
  }

 private:
  struct Want {
    at::Tensor* to;
    at::ScalarType type;
    int64_t shape[4];
    int dims;
    size_t bytes;
  };
  const Call& c_;
  Want wants_[5];
  int n_ = 0;
};

// A workspace whose counters every call leaves at zero, kept per (use, device,
// stream): calls on one stream are ordered, so they may share it. A stream that
// is being captured has one per capture instead, zeroed within the graph and of
// the graph's own memory: a graph may be replayed on any stream, next to eager
// calls on the captured one, and outlives what is kept for those. (It is held
// until the stream's next call that is not of that capture, so that one zero fill
// serves all of the graph's calls.) Only its first `zeros` bytes are zeroed, all of them by default.
at::Tensor zeroed_workspace(c10::Device dev, cudaStream_t st, const char* use, size_t bytes, size_t zeros = ~size_t{0}) {
  using Key = std::tuple<std::string, int, void*>;
  static auto* kept = new std::map<Key, at::Tensor>;  // both outlive the interpreter's end
  static auto* captured = new std::map<Key, std::pair<unsigned long long, at::Tensor>>;
  const Key key(use, static_cast<int>(dev.index()), st);
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (cudaStreamGetCaptureInfo(st, &capturing, &id) != cudaSuccess) {
    cudaGetLastError();
    capturing = cudaStreamCaptureStatusNone;
  }
  auto make = [&]() {
    c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(st, dev.index()));
    if (zeros >= bytes) return at::zeros({static_cast<int64_t>(bytes)}, at::TensorOptions().dtype(at::kByte).device(dev));
    const at::Tensor ws = at::detail::empty_cuda({static_cast<int64_t>(bytes)}, at::kByte, dev, std::nullopt);
    ws.narrow(0, 0, static_cast<int64_t>(zeros)).zero_();
    return ws;
  };
  if (capturing != cudaStreamCaptureStatusNone) {
    auto it = captured->find(key);
    if (it != captured->end() && it->second.first == id && it->second.second.nbytes() >= bytes) return it->second.second;
    const at::Tensor ws = make();
    (*captured)[key] = {id, ws};
    return ws;
  }
  if (!captured->empty()) captured->erase(key);
  auto it = kept->find(key);
  if (it != kept->end() && it->second.nbytes() >= bytes) return it->second;
  return (*kept)[key] = make();
}

at::Tensor workspace(const Call& c, PyObject* given, const char* use, size_t bytes, size_t zeros = ~size_t{0}) {
  if (given == Py_None)
    return bytes ? zeroed_workspace(c.dev, static_cast<cudaStream_t>(c.stream), use, bytes, zeros) : at::Tensor();
  const at::Tensor& t = *tensor(given, "workspace");
  c.dense(t, "workspace");
  return t;
}

int dtype_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return QG_DT_BF16;
  if (t.scalar_type() == at::kFloat) return QG_DT_F32;
  refuse(std::string(name) + " must be bfloat16 or float32");
}

template <typename T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <typename T>
T* ptr(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

struct Cache {
  int num_blocks, Hkv, block_size, D, format;
};
Cache cache_of(const Call& c, const at::Tensor& k, const at::Tensor& v, const at::Tensor& scales) {
  const auto type = k.scalar_type();
  if ((type != at::kChar && type != at::kFloat8_e4m3fn) || v.scalar_type() != type)
    refuse("k_cache and v_cache must both be int8 or both float8_e4m3fn");
  if (k.dim() != 4 || v.sizes() != k.sizes())
    refuse("k_cache and v_cache must have one shape [num_blocks][Hkv][block_size][D]");
  c.dense(k, "k_cache");
  c.dense(v, "v_cache");
  c.need(scales, at::kFloat, {k.size(0), k.size(1), 2}, "scales");
  return {size32(k.size(0), "num_blocks"), size32(k.size(1), "Hkv"), size32(k.size(2), "block_size"),
          size32(k.size(3), "D"), type == at::kChar ? QG_KV_I8 : QG_KV_E4M3};
}

// elements between the tokens of a [T][heads][D] tensor whose tokens are dense
int64_t token_stride(const Call& c, const at::Tensor& t, const char* name) {
  c.on_device(t, name);
  if (t.dim() != 3 || (t.size(2) > 1 && t.stride(2) != 1) || (t.size(1) > 1 && t.stride(1) != t.size(2)))
    refuse(std::string(name) + " must be [T][heads][D] with dense tokens");
  return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
template <typename... Ts>
PyObject* tuple(const Ts&... ts) {
  PyObject* out = PyTuple_New(sizeof...(ts));
  if (!out) throw Raised{};
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(out, i++, ts.defined() ? wrap(ts) : Py_NewRef(Py_None)), ...);
  return out;
}

PyObject* block_plan(PyObject* const* a) {
  const at::Tensor &old_lens = *tensor(a[0], "old_lens"), &new_lens = *tensor(a[1], "new_lens"),
                   &table = *tensor(a[2], "block_table"), &free_list = *tensor(a[3], "free_list"),
                   &count = *tensor(a[4], "free_count");
  const Call c("kv8_block_plan", old_lens, a[13]);
  const int64_t R = old_lens.numel();
  c.need(old_lens, at::kInt, {R}, "old_lens");
  c.need(new_lens, at::kInt, {R}, "new_lens");
  c.need(table, at::kInt, {R, -1}, "block_table");
  c.need(free_list, at::kInt, {-1}, "free_list");
  c.need(count, at::kInt, {1}, "free_count");
  const int bs = whole32(a[5], "block_size"), max_tokens = whole32(a[6], "max_tokens");
  if (max_tokens < 0) refuse("max_tokens is negative");
  at::Tensor count_out = c.output(a[7], at::kInt, {1}, "free_count_out"),
             cu = c.output(a[8], at::kInt, {R + 1}, "cu_new"),
             slots = c.output(a[9], at::kInt, {max_tokens}, "slot_map"),
             pos = c.output(a[10], at::kInt, {max_tokens}, "positions"), info = c.output(a[11], at::kInt, {4}, "info");
  Outputs outs(c);
  outs.add(count_out, at::kInt, {1});
  outs.add(cu, at::kInt, {R + 1});
  outs.add(slots, at::kInt, {max_tokens});
  outs.add(pos, at::kInt, {max_tokens});
  outs.add(info, at::kInt, {4});
  outs.make();
  const at::Tensor ws = workspace(c, a[12], "plan", qg_kv8_plan_workspace_size());
  c.done(kv8_block_plan(ptr<int32_t>(old_lens), ptr<int32_t>(new_lens), size32(R, "R"), bs, ptr<int32_t>(table),
                        size32(table.size(1), "max_blocks"), ptr<int32_t>(free_list),
                        size32(free_list.numel(), "num_blocks"), ptr<int32_t>(count), ptr<int32_t>(count_out),
                        ptr<int32_t>(cu), ptr<int32_t>(slots), ptr<int32_t>(pos), max_tokens, ptr<int32_t>(info),
                        ptr<void>(ws), ws.nbytes(), c.stream));
  return tuple(count_out, cu, slots, pos, info);
}

PyObject* append(PyObject* const* a) {
  const at::Tensor &k = *tensor(a[0], "k"), &v = *tensor(a[1], "v"), &slots = *tensor(a[2], "slot_map"),
                   &kc = *tensor(a[3], "k_cache"), &vc = *tensor(a[4], "v_cache"), &sc = *tensor(a[5], "scales");
  const Call c("kv8_append", kc, a[6]);
  const Cache s = cache_of(c, kc, vc, sc);
  const int64_t ks = token_stride(c, k, "k"), vs = token_stride(c, v, "v");
  const int64_t T = k.size(0);
  if (k.size(1) != s.Hkv || k.size(2) != s.D || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
    refuse("k and v must have one type and shape [T][Hkv][D]");
  c.need(slots, at::kInt, {T}, "slot_map");
  c.done(kv8_append(ptr<void>(k), ptr<void>(v), dtype_of(k, "k"), ks, vs, ptr<int32_t>(slots), size32(T, "T"), s.Hkv,
                    s.D, s.block_size, s.num_blocks, s.format, ptr<void>(kc), ptr<void>(vc), ptr<float>(sc),
                    c.stream));
  Py_RETURN_NONE;
}

PyObject* read(PyObject* const* a) {
  const at::Tensor &ids = *tensor(a[0], "block_ids"), &kc = *tensor(a[1], "k_cache"), &vc = *tensor(a[2], "v_cache"),
                   &sc = *tensor(a[3], "scales");
  const Call c("kv8_read", kc, a[4]);
  const Cache s = cache_of(c, kc, vc, sc);
  const int64_t B = ids.numel();
  c.need(ids, at::kInt, {B}, "block_ids");
  at::Tensor k, v, so;
  Outputs outs(c);
  outs.add(k, at::kBFloat16, {B, s.Hkv, s.block_size, s.D});
  outs.add(v, at::kBFloat16, {B, s.Hkv, s.block_size, s.D});
  outs.add(so, at::kFloat, {B, s.Hkv, 2});
  outs.make();
  c.done(kv8_read(ptr<int32_t>(ids), size32(B, "B"), s.Hkv, s.D, s.block_size, s.num_blocks, s.format, ptr<void>(kc),
                  ptr<void>(vc), ptr<float>(sc), ptr<uint16_t>(k), ptr<uint16_t>(v), ptr<float>(so), c.stream));
  return tuple(k, v, so);
}

PyObject* attention(PyObject* const* a) {
  const at::Tensor &q = *tensor(a[0], "q"), &kc = *tensor(a[1], "k_cache"), &vc = *tensor(a[2], "v_cache"),
                   &sc = *tensor(a[3], "scales"), &table = *tensor(a[4], "block_table"),
                   &ctx = *tensor(a[5], "ctx_lens"), &cu = *tensor(a[6], "cu_q");
  const at::Tensor* tree = tensor_or_null(a[7], "tree_mask");
  const Call c("attn_kv8_paged", q, a[11]);
  const Cache s = cache_of(c, kc, vc, sc);
  const int64_t stride = token_stride(c, q, "q");
  const int64_t T = q.size(0), Hq = q.size(1), R = ctx.numel();
  if (q.scalar_type() != at::kBFloat16 || q.size(2) != s.D) refuse("q must be bfloat16 [T][Hq][D] with the cache's D");
  c.need(ctx, at::kInt, {R}, "ctx_lens");
  c.need(cu, at::kInt, {R + 1}, "cu_q");
  c.need(table, at::kInt, {R, -1}, "block_table");
  if (tree) c.need(*tree, at::kInt, {T}, "tree_mask");
  const float scale = a[8] == Py_None ? 1.f / std::sqrt(static_cast<float>(s.D)) : real(a[8]);
  at::Tensor out = c.output(a[9], at::kBFloat16, {T, Hq, s.D}, "out");
  if (!out.defined()) out = c.make({T, Hq, s.D}, at::kBFloat16);
  const int hq = size32(Hq, "Hq");
  const at::Tensor ws = workspace(c, a[10], "attn", qg_attn_kv8_workspace_size(hq, s.Hkv, s.D));
  c.done(attn_kv8_paged(ptr<uint16_t>(q), stride, ptr<void>(kc), ptr<void>(vc), ptr<float>(sc), ptr<int32_t>(table),
                        ptr<int32_t>(ctx), ptr<int32_t>(cu), ptr<uint32_t>(tree), size32(R, "R"), size32(T, "T"), hq,
                        s.Hkv, s.D, s.block_size, s.num_blocks, size32(table.size(1), "max_blocks"), s.format, scale,
                        ptr<uint16_t>(out), ws.defined() ? ptr<void>(ws) : nullptr, ws.defined() ? ws.nbytes() : 0,
                        c.stream));
  return wrap(out);
}

PyObject* attention_shared(PyObject* const* a) {
  const at::Tensor &q = *tensor(a[0], "q"), &kc = *tensor(a[1], "k_cache"), &vc = *tensor(a[2], "v_cache"),
                   &sc = *tensor(a[3], "scales"), &ptable = *tensor(a[4], "prefix_table"),
                   &plens = *tensor(a[5], "prefix_lens"), &cu_req = *tensor(a[6], "cu_req"),
                   &table = *tensor(a[7], "block_table"), &ctx = *tensor(a[8], "ctx_lens"),
                   &cu = *tensor(a[9], "cu_q");
  const at::Tensor* tree = tensor_or_null(a[10], "tree_mask");
  const Call c("attn_kv8_shared", q, a[14]);
  const Cache s = cache_of(c, kc, vc, sc);
  const int64_t stride = token_stride(c, q, "q");
  const int64_t T = q.size(0), Hq = q.size(1), R = ctx.numel(), G = plens.numel();
  if (q.scalar_type() != at::kBFloat16 || q.size(2) != s.D) refuse("q must be bfloat16 [T][Hq][D] with the cache's D");
  c.need(plens, at::kInt, {G}, "prefix_lens");
  c.need(cu_req, at::kInt, {G + 1}, "cu_req");
  c.need(ptable, at::kInt, {G, -1}, "prefix_table");
  c.need(ctx, at::kInt, {R}, "ctx_lens");
  c.need(cu, at::kInt, {R + 1}, "cu_q");
  c.need(table, at::kInt, {R, -1}, "block_table");
  if (tree) c.need(*tree, at::kInt, {T}, "tree_mask");
  const float scale = a[11] == Py_None ? 1.f / std::sqrt(static_cast<float>(s.D)) : real(a[11]);
  at::Tensor out = c.output(a[12], at::kBFloat16, {T, Hq, s.D}, "out");
  if (!out.defined()) out = c.make({T, Hq, s.D}, at::kBFloat16);
  const int hq = size32(Hq, "Hq"), t = size32(T, "T");
  const at::Tensor ws = workspace(c, a[13], "attn_shared", qg_attn_kv8_shared_workspace_size(t, hq, s.Hkv, s.D), 4096);
  c.done(attn_kv8_shared(ptr<uint16_t>(q), stride, ptr<void>(kc), ptr<void>(vc), ptr<float>(sc), ptr<int32_t>(ptable),
                         ptr<int32_t>(plens), ptr<int32_t>(cu_req), ptr<int32_t>(table), ptr<int32_t>(ctx),
                         ptr<int32_t>(cu), ptr<uint32_t>(tree), size32(G, "groups"), size32(R, "R"), t, hq, s.Hkv, s.D,
                         s.block_size, s.num_blocks, size32(ptable.size(1), "max_prefix_blocks"),
                         size32(table.size(1), "max_blocks"), s.format, scale, ptr<uint16_t>(out),
                         ws.defined() ? ptr<void>(ws) : nullptr, ws.defined() ? ws.nbytes() : 0, c.stream));
  return wrap(out);
}

struct Norm {
  int M, K, xd, rd, wd;
  at::Tensor res_out;
};
Norm norm_args(const Call& c, const at::Tensor& x, const at::Tensor& w, const at::Tensor* res, PyObject* res_out) {
  c.dense(x, "x");
  if (x.dim() != 2) refuse("x must be [M][K]");
  Norm n = {};
  n.M = size32(x.size(0), "M"), n.K = size32(x.size(1), "K");
  n.xd = dtype_of(x, "x");
  c.need(w, w.scalar_type(), {n.K}, "weight");
  n.wd = dtype_of(w, "weight");
  n.rd = QG_DT_F32;
  if (res) {
    c.need(*res, res->scalar_type(), {n.M, n.K}, "residual");
    n.rd = dtype_of(*res, "residual");
    n.res_out = c.output(res_out, res->scalar_type(), {n.M, n.K}, "residual_out");
  } else if (res_out != Py_None) {
    n.res_out = *tensor(res_out, "residual_out");
    c.need(n.res_out, n.res_out.scalar_type(), {n.M, n.K}, "residual_out");
    n.rd = dtype_of(n.res_out, "residual_out");
  }
  return n;
}

PyObject* norm_bf16(PyObject* const* a) {
  const at::Tensor &x = *tensor(a[0], "x"), &w = *tensor(a[1], "weight");
  const at::Tensor* res = tensor_or_null(a[2], "residual");
  const Call c("rmsnorm_residual", x, a[6]);
  Norm n = norm_args(c, x, w, res, a[4]);
  at::Tensor out = c.output(a[5], at::kBFloat16, {n.M, n.K}, "out");
  Outputs outs(c);
  outs.add(out, at::kBFloat16, {n.M, n.K});
  if (res) outs.add(n.res_out, res->scalar_type(), {n.M, n.K});
  outs.make();
  c.done(rmsnorm_residual(ptr<void>(x), n.xd, ptr<void>(res), n.rd, ptr<void>(w), n.wd, real(a[3]), n.M, n.K,
                          n.res_out.defined() ? ptr<void>(n.res_out) : nullptr, ptr<uint16_t>(out), c.stream));
  return tuple(out, n.res_out);
}

PyObject* norm_i8(PyObject* const* a) {
  const at::Tensor &x = *tensor(a[0], "x"), &w = *tensor(a[1], "weight");
  const at::Tensor *res = tensor_or_null(a[2], "residual"), *sb = tensor_or_null(a[3], "sign_bits");
  const Call c("rmsnorm_residual_i8", x, a[8]);
  Norm n = norm_args(c, x, w, res, a[5]);
  if (sb) c.need(*sb, at::kInt, {n.K / 32}, "sign_bits");
  at::Tensor q = c.output(a[6], at::kChar, {n.M, n.K}, "q"), scale = c.output(a[7], at::kFloat, {n.M}, "scale");
  Outputs outs(c);
  outs.add(q, at::kChar, {n.M, n.K});
  outs.add(scale, at::kFloat, {n.M});
  if (res) outs.add(n.res_out, res->scalar_type(), {n.M, n.K});
  outs.make();
  c.done(rmsnorm_residual_i8(ptr<void>(x), n.xd, ptr<void>(res), n.rd, ptr<void>(w), n.wd, real(a[4]),
                             ptr<uint32_t>(sb), n.M, n.K, n.res_out.defined() ? ptr<void>(n.res_out) : nullptr,
                             ptr<int8_t>(q), ptr<float>(scale), c.stream));
  return tuple(q, scale, n.res_out);
}

PyObject* qk_rope(PyObject* const* a) {
  const at::Tensor &q = *tensor(a[0], "q"), &k = *tensor(a[1], "k"), &pos = *tensor(a[2], "positions"),
                   &freq = *tensor(a[3], "inv_freq");
  const at::Tensor *qw = tensor_or_null(a[4], "q_weight"), *kw = tensor_or_null(a[5], "k_weight");
  const Call c("qk_norm_rope", q, a[11]);
  const int64_t qs = token_stride(c, q, "q"), ks = token_stride(c, k, "k");
  const int64_t T = q.size(0), Hq = q.size(1), Hkv = k.size(1), D = q.size(2);
  if (k.size(0) != T || k.size(2) != D || k.scalar_type() != q.scalar_type())
    refuse("q and k must have one type, T and D");
  const int xd = dtype_of(q, "q");
  const int64_t axes = pos.dim() == 2 ? pos.size(0) : 1;
  if (pos.dim() == 2)
    c.need(pos, at::kInt, {axes, T}, "positions");
  else
    c.need(pos, at::kInt, {T}, "positions");
  c.need(freq, at::kDouble, {-1}, "inv_freq");
  int wd = QG_DT_F32;
  if (qw) c.need(*qw, qw->scalar_type(), {D}, "q_weight"), wd = dtype_of(*qw, "q_weight");
  if (kw) c.need(*kw, kw->scalar_type(), {D}, "k_weight"), wd = dtype_of(*kw, "k_weight");
  if (qw && kw && qw->scalar_type() != kw->scalar_type()) refuse("q_weight and k_weight must have one type");
  const int inter = PyObject_IsTrue(a[7]);
  if (inter < 0) throw Raised{};
  const uint8_t* pair_axis = nullptr;
  if (a[8] != Py_None) {
    if (!PyBytes_Check(a[8]) || PyBytes_GET_SIZE(a[8]) != freq.numel())
      refuse("pair_axis must have one entry for each of inv_freq");
    pair_axis = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(a[8]));
  } else if (axes > 1) {
    refuse("positions on several axes need pair_axis");
  }
  at::Tensor qo = c.output(a[9], at::kBFloat16, {T, Hq, D}, "q_out"), ko;
  if (a[10] != Py_None) {
    ko = *tensor(a[10], "k_out");
    dtype_of(ko, "k_out");
    c.need(ko, ko.scalar_type(), {T, Hkv, D}, "k_out");
  }
  Outputs outs(c);
  outs.add(qo, at::kBFloat16, {T, Hq, D});
  outs.add(ko, k.scalar_type(), {T, Hkv, D});
  outs.make();
  c.done(qk_norm_rope(ptr<void>(q), qs, ptr<void>(k), ks, xd, ptr<int32_t>(pos), size32(axes, "axes"),
                      ptr<double>(freq), size32(2 * freq.numel(), "rotary_dim"), pair_axis, inter, ptr<void>(qw),
                      ptr<void>(kw), wd, real(a[6]), size32(T, "T"), size32(Hq, "Hq"), size32(Hkv, "Hkv"),
                      size32(D, "D"), ptr<uint16_t>(qo), ptr<void>(ko), dtype_of(ko, "k_out"), c.stream));
  return tuple(qo, ko);
}

PyObject* sample(PyObject* const* a) {
  const at::Tensor &x = *tensor(a[0], "logits"), &u = *tensor(a[1], "u");
  const at::Tensor *temp = tensor_or_null(a[2], "temperature"), *k = tensor_or_null(a[3], "top_k"),
                   *p = tensor_or_null(a[4], "top_p"), *mp = tensor_or_null(a[5], "min_p");
  const Call c("sample_logits", x, a[8]);
  if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1)) refuse("logits must be [M][V] with dense rows");
  const int64_t M = x.size(0), V = x.size(1), stride = M > 1 ? x.stride(0) : V;
  const int dt = dtype_of(x, "logits");
  c.need(u, at::kFloat, {M}, "u");
  if (temp) c.need(*temp, at::kFloat, {M}, "temperature");
  if (k) c.need(*k, k->scalar_type() == at::kLong ? at::kLong : at::kInt, {M}, "top_k");
  if (p) c.need(*p, at::kFloat, {M}, "top_p");
  if (mp) c.need(*mp, at::kFloat, {M}, "min_p");
  at::Tensor tokens = c.output(a[6], at::kInt, {M}, "tokens"), probs = c.output(a[7], at::kFloat, {M}, "probs");
  Outputs outs(c);
  outs.add(tokens, at::kInt, {M});
  outs.add(probs, at::kFloat, {M});
  outs.make();
  c.done(sample_logits(ptr<void>(x), dt, stride, size32(M, "M"), size32(V, "V"), ptr<float>(u), ptr<float>(temp),
                       ptr<void>(k), k ? static_cast<int>(k->element_size()) : 0, ptr<float>(p), ptr<float>(mp), ptr<int32_t>(tokens), ptr<float>(probs),
                       c.stream));
  return tuple(tokens, probs);
}

// (use, bytes, device index, stream handle): the workspace, for the calls that are marshalled in Python
PyObject* make_workspace(PyObject* const* a) {
  const char* use = PyUnicode_AsUTF8(a[0]);
  if (!use) throw Raised{};
  const int bytes = whole32(a[1], "bytes"), index = whole32(a[2], "device");
  const auto st = reinterpret_cast<cudaStream_t>(PyLong_AsUnsignedLongLong(a[3]));
  if (PyErr_Occurred()) throw Raised{};
  if (bytes < 0) refuse("bytes is negative");
  const c10::Device dev(c10::kCUDA, static_cast<c10::DeviceIndex>(index));
  const c10::cuda::CUDAGuard guard(dev);
  return wrap(zeroed_workspace(dev, st, use, static_cast<size_t>(bytes)));
}

// no C++ exception passes into Python
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.why.c_str());
  } catch (const std::exception& e) {  // torch's own, an allocation that failed among them
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* set_raise(PyObject*, PyObject* f) {
  Py_XSETREF(g_raise, Py_NewRef(f));
  Py_RETURN_NONE;
}

#define QG_FAST(f, n) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL
PyMethodDef kMethods[] = {
    {"block_plan", QG_FAST(block_plan, 14), nullptr}, {"append", QG_FAST(append, 7), nullptr},
    {"read", QG_FAST(read, 5), nullptr},              {"attention", QG_FAST(attention, 12), nullptr},
    {"attention_shared", QG_FAST(attention_shared, 15), nullptr},
    {"norm_bf16", QG_FAST(norm_bf16, 7), nullptr},    {"norm_i8", QG_FAST(norm_i8, 9), nullptr},
    {"qk_rope", QG_FAST(qk_rope, 12), nullptr},
    {"sample", QG_FAST(sample, 9), nullptr},
    {"workspace", QG_FAST(make_workspace, 4), nullptr},
    {"set_raise", set_raise, METH_O, nullptr},        {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_qgbind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qgbind() { return PyModule_Create(&kModule); }
