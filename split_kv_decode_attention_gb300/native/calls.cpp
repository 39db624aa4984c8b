// calls.cpp -- the Python entries of the operators around the cache as a
// CPython extension over the C ABI: it checks the tensors, fills the parameter
// structs, allocates what the caller left out and makes one C call.
//
// A decode step makes these calls once per layer, and their kernels take 2 to
// 10 us.  Host time of a call on a Grace core, marshalled through ctypes and
// here, launches included: append 25 and 4 us, digest 17 and 3, attention 42 to
// 49 and 7 to 10, sparse attention 53 and 16.
//
// Every function takes its arguments by position; binding.py holds the
// keyword signatures and the documentation.

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <optional>
#include <string>

#include "decode_attn.h"

namespace {

constexpr int64_t kD = DECODE_ATTN_HEAD_DIM;

struct Refusal {
  std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw Refusal{what}; }

struct CallError {
  int code;
  const char* where;
};

void check(int code, const char* where) {
  if (code != DA_OK) throw CallError{code, where};
}

PyObject* g_error = nullptr;  // DecodeAttnError

std::string dims(std::initializer_list<int64_t> v) {
  std::string s = "[";
  for (int64_t x : v) s += (s.size() > 1 ? ", " : "") + std::to_string(x);
  return s + "]";
}

// ---- arguments
const at::Tensor& undefined() {
  static const at::Tensor t;
  return t;
}

// A tensor, or (None) an undefined one.
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (o == Py_None) return undefined();
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (!t.defined()) refuse(std::string(name) + " is needed");
  return t;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int32_t>(v);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

void type_of(const at::Tensor& t, at::ScalarType want, const char* name) {
  if (t.scalar_type() != want)
    refuse(std::string(name) + " is " + c10::toString(t.scalar_type()) + "; expected " + c10::toString(want));
}

void byte_type(const at::Tensor& t, const char* name) {
  if (t.scalar_type() != at::kByte && t.scalar_type() != at::kFloat8_e4m3fn)
    refuse(std::string(name) + " is " + c10::toString(t.scalar_type()) + "; expected uint8 or float8_e4m3fn");
}

bool same_steps(const at::Tensor& x, const at::Tensor& y) {
  for (int64_t d = 0; d < x.dim(); ++d)
    if (x.size(d) > 1 && x.stride(d) != y.stride(d)) return false;
  return true;
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

size_t bytes_of(const at::Tensor& t) {
  return t.defined() ? static_cast<size_t>(t.numel()) * t.element_size() : 0;
}

// Every given tensor lies on the current CUDA device: the one whose stream the
// call takes and whose planner it asks.
void on_current_device(std::initializer_list<const at::Tensor*> ts) {
  int cur = -1;
  for (const at::Tensor* t : ts) {
    if (!t->defined()) continue;
    const at::Device d = t->device();
    if (cur < 0 && d.is_cuda()) cur = c10::cuda::current_device();
    if (!d.is_cuda() || d.index() != cur)
      refuse("a tensor is on " + d.str() + ", not on the current CUDA device");
  }
}

// The stream of a call.  Where it is not the current one, it is made current
// until the call returns: what the call allocates then comes from that stream's
// memory (a block that the current stream has freed may still be in use there),
// and the allocator is told that the results are read on the caller's.
class Stream {
 public:
  explicit Stream(PyObject* o) {
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream();
    raw = current.stream();
    if (o == Py_None) return;
    void* p = nullptr;
    if (PyLong_Check(o)) {
      p = PyLong_AsVoidPtr(o);
    } else {
      PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
      if (h == nullptr) throw python_error();
      p = PyLong_AsVoidPtr(h);
      Py_DECREF(h);
    }
    if (PyErr_Occurred()) throw python_error();
    if (p == raw) return;
    raw = p;
    caller_ = current;
    guard_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), current.device_index()));
  }

  // (a tensor that the call allocated and hands out)
  void returns(const at::Tensor& t) const {
    if (caller_ && t.numel() > 0) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *caller_);
  }

  void* raw;

 private:
  std::optional<c10::cuda::CUDAStream> caller_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

int32_t* status_of(const at::Tensor& t) {
  if (!t.defined()) return nullptr;
  type_of(t, at::kInt, "status");
  if (t.numel() < 1) refuse("status is empty");
  return static_cast<int32_t*>(t.data_ptr());
}

// ---- shapes
// The stride of a dimension; one of at most one entry is never stepped along
// and may hold anything: a multiple of every alignment stands for it.
int64_t step(const at::Tensor& t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 4 * kD; }

void int_vector(const at::Tensor& t, int64_t n, const char* name) {
  type_of(t, at::kInt, name);
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    refuse(std::string(name) + " must be dense " + dims({n}));
}

// [batch, tokens, heads, 128] bf16 with a dense last dimension
void heads_tensor(const at::Tensor& t, int64_t B, int64_t T, const char* name) {
  type_of(t, at::kBFloat16, name);
  if (t.dim() != 4 || t.size(0) != B || t.size(1) != T || t.size(3) != kD || t.stride(3) != 1)
    refuse(std::string(name) + " must be " + dims({B, T}) + " + [heads, 128], its last dimension dense");
}

void dense(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape, const char* name) {
  type_of(t, type, name);
  if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size()) || !t.is_contiguous())
    refuse(std::string(name) + " must be dense " + dims(shape));
}

struct Cache {
  decode_attn_cache c;
  int64_t groups, tokens, heads;
};

Cache cache_args(const at::Tensor& k, const at::Tensor& v, const at::Tensor& k_sf, const at::Tensor& v_sf,
                 bool need_v) {
  Cache r;
  std::memset(&r.c, 0, sizeof(r.c));
  int64_t width = kD;
  if (k_sf.defined() || v_sf.defined()) {
    r.c.type = DA_CACHE_FP4_E2M1;
    width = kD / 2;
    if (!k_sf.defined() || (need_v && !v_sf.defined()))
      refuse("a 4-bit cache needs the block scales of K and of V");
    type_of(k, at::kByte, "k_cache");
  } else if (k.element_size() == 1) {
    r.c.type = DA_CACHE_FP8_E4M3;
    byte_type(k, "k_cache");
  } else {
    r.c.type = DA_CACHE_BF16;
    type_of(k, at::kBFloat16, "k_cache");
  }
  if (k.dim() != 4 || k.size(3) != width || k.stride(3) != 1)
    refuse("k_cache must be [groups, tokens, heads, " + std::to_string(width) + "], its last dimension dense");
  if (v.defined() && (v.sizes() != k.sizes() || !same_steps(v, k) || v.scalar_type() != k.scalar_type()))
    refuse("k_cache and v_cache differ in shape, strides or type");
  r.groups = k.size(0);
  r.tokens = k.size(1);
  r.heads = k.size(2);
  r.c.k = ptr(k);
  r.c.v = ptr(v);
  if (r.c.type == DA_CACHE_FP4_E2M1) {
    for (const at::Tensor* t : {&k_sf, &v_sf}) {
      if (!t->defined()) continue;
      byte_type(*t, "k_sf or v_sf");
      if (t->dim() != 4 || t->size(0) != r.groups || t->size(1) != r.heads || t->size(2) != r.tokens ||
          t->size(3) != 8 || (t->size(2) > 1 && t->stride(2) != 8) || t->stride(3) != 1)
        refuse("k_sf and v_sf must be " + dims({r.groups, r.heads, r.tokens, 8}) + " with dense tokens");
    }
    if (v_sf.defined() && !same_steps(v_sf, k_sf)) refuse("k_sf and v_sf differ in strides");
    r.c.k_block_scale = ptr(k_sf);
    r.c.v_block_scale = ptr(v_sf);
    r.c.bs_stride_page = step(k_sf, 0);
    r.c.bs_stride_head = step(k_sf, 1);
  }
  return r;
}

decode_attn_params cache_params(int64_t B, int64_t T, int64_t Hq, const Cache& c, const at::Tensor& k,
                                const at::Tensor& bt, int32_t max_seq_len, bool causal, float scale,
                                double k_scale, double v_scale) {
  decode_attn_params p;
  std::memset(&p, 0, sizeof(p));
  for (int64_t x : {B, T, Hq, c.heads, c.groups, c.tokens})
    if (x > INT32_MAX) refuse("a size does not fit 32 bits");
  p.batch = static_cast<int32_t>(B);
  p.q_len = static_cast<int32_t>(T);
  p.num_q_heads = static_cast<int32_t>(Hq);
  p.num_kv_heads = static_cast<int32_t>(c.heads);
  p.head_dim = kD;
  p.max_seq_len = max_seq_len;
  p.causal = causal ? 1 : 0;
  p.scale = scale;
  p.kv_stride_page = step(k, 0);
  p.kv_stride_token = step(k, 1);
  p.kv_stride_head = step(k, 2);
  p.k_scale = static_cast<float>(k_scale);
  p.v_scale = static_cast<float>(v_scale);
  if (bt.defined()) {
    type_of(bt, at::kInt, "block_table");
    if (bt.dim() != 2 || bt.size(0) != B || (bt.size(1) > 1 && bt.stride(1) != 1))
      refuse("block_table must be [batch, pages], its last dimension dense");
    p.page_size = static_cast<int32_t>(c.tokens);
    p.num_pages = static_cast<int32_t>(c.groups);
    p.max_pages_per_seq = static_cast<int32_t>(bt.size(1));
    p.block_table_stride = bt.size(0) > 1 ? bt.stride(0) : bt.size(1);
  } else if (c.groups != B || c.tokens < max_seq_len) {
    refuse("a contiguous cache holds max_seq_len tokens of every request");
  }
  return p;
}

void q_strides(decode_attn_params& p, const at::Tensor& q, const at::Tensor& out) {
  p.q_stride_batch = step(q, 0);
  p.q_stride_token = step(q, 1);
  p.q_stride_head = step(q, 2);
  p.o_stride_batch = step(out, 0);
  p.o_stride_token = step(out, 1);
  p.o_stride_head = step(out, 2);
}

float scale_or_default(PyObject* o) {
  return o == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(kD))) : static_cast<float>(number(o));
}

// (a CUDA tensor by then: on_current_device has looked)
at::Tensor empty_like_device(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

at::Tensor new_result(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like, const Stream& stream) {
  at::Tensor t = empty_like_device(shape, type, like);
  stream.returns(t);
  return t;
}

at::Tensor out_or_new(const at::Tensor& out, const at::Tensor& q, const Stream& stream) {
  if (!out.defined()) return new_result(q.sizes(), at::kBFloat16, q, stream);
  heads_tensor(out, q.size(0), q.size(1), "out");
  if (out.size(2) != q.size(2)) refuse("out and q differ in heads");
  return out;
}

at::Tensor lse_or_new(const at::Tensor& lse, const at::Tensor& q, const Stream& stream) {
  if (!lse.defined()) return new_result({q.size(0), q.size(1), q.size(2)}, at::kFloat, q, stream);
  dense(lse, at::kFloat, {q.size(0), q.size(1), q.size(2)}, "lse");
  return lse;
}

at::Tensor workspace_or_new(const at::Tensor& given, size_t need, const at::Tensor& like) {
  if (need == 0 || (given.defined() && given.is_contiguous() && bytes_of(given) >= need)) return given;
  return empty_like_device({static_cast<int64_t>((need + 15) / 16 * 16)}, at::kByte, like);
}

PyObject* give(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* give(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (r == nullptr) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (o == nullptr) {
      Py_DECREF(r);
      throw python_error();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("called with " + std::to_string(n) + " arguments, " + std::to_string(want) + " are needed");
}

// ---- the entries
PyObject* rope_table(PyObject* const* a, Py_ssize_t n) {
  count(n, 6);  // inv_freq, max_pos, amplitude, first, out, stream
  const at::Tensor& f = needed(a[0], "inv_freq");
  type_of(f, at::kDouble, "inv_freq");
  if (f.dim() != 1 || !f.is_contiguous()) refuse("inv_freq must be a dense vector");
  const int64_t rows = integer(a[1]), nf = f.size(0);
  const double amplitude = number(a[2]);
  const int64_t first = integer(a[3]);
  at::Tensor out = tensor(a[4], "out");
  if (rows < 0) refuse("max_pos is negative");
  on_current_device({&f, &out});
  const Stream stream(a[5]);
  if (out.defined()) {
    dense(out, at::kFloat, {rows, 2 * nf}, "out");
  } else {
    out = new_result({rows, 2 * nf}, at::kFloat, f, stream);
  }
  check(decode_attn_rope_table(static_cast<const double*>(ptr(f)), static_cast<int32_t>(std::min<int64_t>(nf, 1 << 20)),
                               first, rows, amplitude, static_cast<float*>(ptr(out)), stream.raw),
        "decode_attn_rope_table");
  return give(out);
}

PyObject* rope_append(PyObject* const* a, Py_ssize_t n) {
  count(n, 19);
  // q, k, v, table, k_cache, v_cache, block_table, seq_lens, max_seq_len,
  // interleaved, positions, new_lens, k_scale, v_scale, k_sf, v_sf, q_out, status, stream
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const at::Tensor& table = tensor(a[3], "table");
  const at::Tensor &kc = needed(a[4], "k_cache"), &vc = needed(a[5], "v_cache");
  const at::Tensor &bt = tensor(a[6], "block_table"), &lens = needed(a[7], "seq_lens");
  const int32_t max_seq_len = integer32(a[8], "max_seq_len");
  const at::Tensor &pos = tensor(a[10], "positions"), &new_lens = tensor(a[11], "new_lens");
  const at::Tensor &k_sf = tensor(a[14], "k_sf"), &v_sf = tensor(a[15], "v_sf");
  at::Tensor q_out = tensor(a[16], "q_out");
  const at::Tensor& status = tensor(a[17], "status");
  const at::Tensor& lead = q.defined() ? q : k;
  if (!lead.defined() || k.defined() != v.defined()) refuse("q, or k and v, or all three are needed");
  if (lead.dim() != 4) refuse("q, k and v must be [batch, tokens, heads, 128]");
  const int64_t B = lead.size(0), T = lead.size(1);
  const Cache c = cache_args(kc, vc, k_sf, v_sf, true);
  int_vector(lens, B, "seq_lens");
  decode_attn_rope r;
  std::memset(&r, 0, sizeof(r));
  if (table.defined()) {
    type_of(table, at::kFloat, "table");
    if (table.dim() != 2 || !table.is_contiguous() || table.size(0) > INT32_MAX || table.size(1) > 2 * kD)
      refuse("table must be dense [positions, rotary_dim]");
    r.table_positions = static_cast<int32_t>(table.size(0));
    r.rotary_dim = static_cast<int32_t>(table.size(1));
  }
  r.interleaved = truth(a[9]) ? 1 : 0;
  if (k.defined()) {
    heads_tensor(k, B, T, "k");
    heads_tensor(v, B, T, "v");
    if (k.size(2) != c.heads || v.size(2) != c.heads) refuse("k and v must have the cache's heads");
    r.k_stride_batch = step(k, 0);
    r.k_stride_token = step(k, 1);
    r.k_stride_head = step(k, 2);
    r.v_stride_batch = step(v, 0);
    r.v_stride_token = step(v, 1);
    r.v_stride_head = step(v, 2);
  }
  decode_attn_params p = cache_params(B, T, c.heads, c, kc, bt, max_seq_len, false, 1.f, number(a[12]), number(a[13]));
  if (q.defined()) {
    heads_tensor(q, B, T, "q");
    if (c.heads == 0 || q.size(2) % c.heads != 0) refuse("the query heads are no multiple of the cache's heads");
    if (q_out.defined()) {
      heads_tensor(q_out, B, T, "q_out");
      if (q_out.size(2) != q.size(2)) refuse("q_out and q differ in heads");
    }
    p.num_q_heads = static_cast<int32_t>(q.size(2));
  } else if (q_out.defined()) {
    refuse("q_out without q");
  }
  if (pos.defined()) dense(pos, at::kInt, {B, T}, "positions");
  if (new_lens.defined()) int_vector(new_lens, B, "new_lens");
  on_current_device({&q, &k, &v, &table, &kc, &vc, &bt, &lens, &pos, &new_lens, &k_sf, &v_sf, &q_out, &status});
  const Stream stream(a[18]);
  if (q.defined()) {
    if (!q_out.defined()) q_out = new_result(q.sizes(), at::kBFloat16, q, stream);
    q_strides(p, q, q_out);
  }
  check(decode_attn_rope_append(&p, &c.c, &r, ptr(q), ptr(k), ptr(v), static_cast<const float*>(ptr(table)),
                                static_cast<const int32_t*>(ptr(pos)), static_cast<const int32_t*>(ptr(new_lens)),
                                static_cast<const int32_t*>(ptr(bt)), static_cast<const int32_t*>(ptr(lens)),
                                ptr(q_out), status_of(status), stream.raw),
        "decode_attn_rope_append");
  if (!q.defined()) Py_RETURN_NONE;
  return give(q_out);
}

void digest_tensors(const at::Tensor& digest, const at::Tensor& scale, int64_t pages, int64_t heads) {
  dense(digest, at::kChar, {pages, heads, 2, kD}, "digest");
  dense(scale, at::kFloat, {pages, heads}, "digest_scale");
}

PyObject* block_digest(PyObject* const* a, Py_ssize_t n) {
  count(n, 10);
  // k_cache, block_table, seq_lens, digest, digest_scale, max_seq_len, max_new, k_sf, status, stream
  const at::Tensor& kc = needed(a[0], "k_cache");
  const at::Tensor &bt = needed(a[1], "block_table"), &lens = needed(a[2], "seq_lens");
  at::Tensor digest = tensor(a[3], "digest"), scale = tensor(a[4], "digest_scale");
  const at::Tensor &k_sf = tensor(a[7], "k_sf"), &status = tensor(a[8], "status");
  const Cache c = cache_args(kc, undefined(), k_sf, undefined(), false);
  if (bt.dim() != 2) refuse("block_table must be [batch, pages]");
  const int64_t B = bt.size(0);
  int_vector(lens, B, "seq_lens");
  decode_attn_params p =
      cache_params(B, 1, c.heads, c, kc, bt, integer32(a[5], "max_seq_len"), false, 1.f, 1.0, 1.0);
  on_current_device({&kc, &bt, &lens, &digest, &scale, &k_sf, &status});
  const Stream stream(a[9]);
  if (!digest.defined()) {
    digest = at::zeros({c.groups, c.heads, 2, kD}, kc.options().dtype(at::kChar));
    stream.returns(digest);
  }
  if (!scale.defined()) {
    scale = at::zeros({c.groups, c.heads}, kc.options().dtype(at::kFloat));
    stream.returns(scale);
  }
  digest_tensors(digest, scale, c.groups, c.heads);
  check(decode_attn_block_digest(&p, &c.c, static_cast<const int32_t*>(ptr(bt)), static_cast<const int32_t*>(ptr(lens)),
                                 integer32(a[6], "max_new"), static_cast<int8_t*>(ptr(digest)),
                                 static_cast<float*>(ptr(scale)), status_of(status), stream.raw),
        "decode_attn_block_digest");
  return give({digest, scale});
}

PyObject* decode_cached(PyObject* const* a, Py_ssize_t n) {
  count(n, 19);
  // q, k_cache, v_cache, k_sf, v_sf, block_table, seq_lens, max_seq_len, causal, scale,
  // num_splits, out, lse, workspace, status, stream, two_pass, k_scale, v_scale
  const at::Tensor& q = needed(a[0], "q");
  const at::Tensor &kc = needed(a[1], "k_cache"), &vc = needed(a[2], "v_cache");
  const at::Tensor &k_sf = tensor(a[3], "k_sf"), &v_sf = tensor(a[4], "v_sf");
  const at::Tensor &bt = tensor(a[5], "block_table"), &lens = needed(a[6], "seq_lens");
  const at::Tensor &given = tensor(a[13], "workspace"), &status = tensor(a[14], "status");
  const at::Tensor &out0 = tensor(a[11], "out"), &lse0 = tensor(a[12], "lse");
  if (q.dim() != 4) refuse("q must be [batch, tokens, heads, 128]");
  const int64_t B = q.size(0), T = q.size(1);
  heads_tensor(q, B, T, "q");
  int_vector(lens, B, "seq_lens");
  const Cache c = cache_args(kc, vc, k_sf, v_sf, true);
  decode_attn_params p = cache_params(B, T, q.size(2), c, kc, bt, integer32(a[7], "max_seq_len"), truth(a[8]),
                                      scale_or_default(a[9]), number(a[17]), number(a[18]));
  p.flags = truth(a[16]) ? DA_FLAG_TWO_PASS : 0;
  on_current_device({&q, &kc, &vc, &k_sf, &v_sf, &bt, &lens, &given, &status, &out0, &lse0});
  const Stream stream(a[15]);
  const at::Tensor out = out_or_new(out0, q, stream), lse = lse_or_new(lse0, q, stream);
  q_strides(p, q, out);
  const int32_t splits = std::max<int32_t>(0, integer32(a[10], "num_splits"));
  size_t need = 0;
  check(decode_attn_cached_workspace_bytes(&p, &c.c, splits, &need), "decode_attn_cached_workspace_bytes");
  const at::Tensor ws = workspace_or_new(given, need, q);
  check(decode_attn_cached(&p, &c.c, ptr(q), static_cast<const int32_t*>(ptr(bt)),
                           static_cast<const int32_t*>(ptr(lens)), ptr(out), static_cast<float*>(ptr(lse)), splits,
                           ptr(ws), bytes_of(ws), status_of(status), stream.raw),
        "decode_attn_cached");
  return give({out, lse});
}

PyObject* sparse(PyObject* const* a, Py_ssize_t n) {
  count(n, 23);
  // q, k_cache, v_cache, block_table, seq_lens, digest, digest_scale, max_seq_len, top_k,
  // sink, local, causal, scale, k_scale, v_scale, k_sf, v_sf, out, lse, blocks, workspace, status, stream
  const at::Tensor& q = needed(a[0], "q");
  const at::Tensor &kc = needed(a[1], "k_cache"), &vc = needed(a[2], "v_cache");
  const at::Tensor &bt = needed(a[3], "block_table"), &lens = needed(a[4], "seq_lens");
  const at::Tensor &digest = needed(a[5], "digest"), &dscale = needed(a[6], "digest_scale");
  const at::Tensor &k_sf = tensor(a[15], "k_sf"), &v_sf = tensor(a[16], "v_sf");
  const at::Tensor &out0 = tensor(a[17], "out"), &lse0 = tensor(a[18], "lse");
  at::Tensor blocks = tensor(a[19], "blocks");
  const at::Tensor &given = tensor(a[20], "workspace"), &status = tensor(a[21], "status");
  if (q.dim() != 4) refuse("q must be [batch, tokens, heads, 128]");
  const int64_t B = q.size(0), T = q.size(1);
  heads_tensor(q, B, T, "q");
  int_vector(lens, B, "seq_lens");
  const Cache c = cache_args(kc, vc, k_sf, v_sf, true);
  digest_tensors(digest, dscale, c.groups, c.heads);
  decode_attn_params p = cache_params(B, T, q.size(2), c, kc, bt, integer32(a[7], "max_seq_len"), truth(a[11]),
                                      scale_or_default(a[12]), number(a[13]), number(a[14]));
  decode_attn_select s;
  std::memset(&s, 0, sizeof(s));
  s.top_k = integer32(a[8], "top_k");
  s.sink = integer32(a[9], "sink");
  s.local = integer32(a[10], "local");
  if (s.top_k < 1) refuse("top_k must be at least 1");
  on_current_device({&q, &kc, &vc, &k_sf, &v_sf, &bt, &lens, &digest, &dscale, &given, &status, &out0, &lse0, &blocks});
  const Stream stream(a[22]);
  const at::Tensor out = out_or_new(out0, q, stream), lse = lse_or_new(lse0, q, stream);
  q_strides(p, q, out);
  if (blocks.defined()) dense(blocks, at::kInt, {B, T, c.heads, s.top_k}, "blocks");
  else blocks = new_result({B, T, c.heads, s.top_k}, at::kInt, q, stream);
  size_t need = 0;
  check(decode_attn_sparse_workspace_bytes(&p, &c.c, &s, &need), "decode_attn_sparse_workspace_bytes");
  const at::Tensor ws = workspace_or_new(given, need, q);
  check(decode_attn_sparse(&p, &c.c, &s, ptr(q), static_cast<const int8_t*>(ptr(digest)),
                           static_cast<const float*>(ptr(dscale)), static_cast<const int32_t*>(ptr(bt)),
                           static_cast<const int32_t*>(ptr(lens)), ptr(out), static_cast<float*>(ptr(lse)),
                           static_cast<int32_t*>(ptr(blocks)), ptr(ws), bytes_of(ws), status_of(status),
                           stream.raw),
        "decode_attn_sparse");
  return give({out, lse, blocks});
}

PyObject* block_select(PyObject* const* a, Py_ssize_t n) {
  count(n, 15);
  // q, digest, digest_scale, block_table, seq_lens, page_size, max_seq_len, top_k, sink,
  // local, causal, blocks, workspace, status, stream
  const at::Tensor &q = needed(a[0], "q"), &digest = needed(a[1], "digest"), &dscale = needed(a[2], "digest_scale");
  const at::Tensor &bt = needed(a[3], "block_table"), &lens = needed(a[4], "seq_lens");
  at::Tensor blocks = tensor(a[11], "blocks");
  const at::Tensor &given = tensor(a[12], "workspace"), &status = tensor(a[13], "status");
  if (q.dim() != 4 || digest.dim() != 4) refuse("q must be [batch, tokens, heads, 128], digest [pages, heads, 2, 128]");
  const int64_t B = q.size(0), T = q.size(1);
  heads_tensor(q, B, T, "q");
  int_vector(lens, B, "seq_lens");
  Cache c;
  std::memset(&c.c, 0, sizeof(c.c));
  c.groups = digest.size(0);
  c.heads = digest.size(1);
  c.tokens = integer32(a[5], "page_size");
  digest_tensors(digest, dscale, c.groups, c.heads);
  decode_attn_params p = cache_params(B, T, q.size(2), c, digest, bt, integer32(a[6], "max_seq_len"), truth(a[10]), 1.f,
                                      1.0, 1.0);
  q_strides(p, q, q);
  decode_attn_select s;
  std::memset(&s, 0, sizeof(s));
  s.top_k = integer32(a[7], "top_k");
  s.sink = integer32(a[8], "sink");
  s.local = integer32(a[9], "local");
  if (s.top_k < 1) refuse("top_k must be at least 1");
  on_current_device({&q, &digest, &dscale, &bt, &lens, &blocks, &given, &status});
  const Stream stream(a[14]);
  if (blocks.defined()) dense(blocks, at::kInt, {B, T, c.heads, s.top_k}, "blocks");
  else blocks = new_result({B, T, c.heads, s.top_k}, at::kInt, q, stream);
  const at::Tensor pages = new_result({B, T, c.heads, s.top_k}, at::kInt, q, stream);
  const at::Tensor tokens = new_result({B, T, c.heads}, at::kInt, q, stream);
  size_t need = 0;
  check(decode_attn_block_select_workspace_bytes(&p, &s, &need), "decode_attn_block_select_workspace_bytes");
  const at::Tensor ws = workspace_or_new(given, need, q);
  check(decode_attn_block_select(&p, &s, ptr(q), static_cast<const int8_t*>(ptr(digest)),
                                 static_cast<const float*>(ptr(dscale)), static_cast<const int32_t*>(ptr(bt)),
                                 static_cast<const int32_t*>(ptr(lens)), static_cast<int32_t*>(ptr(blocks)),
                                 static_cast<int32_t*>(ptr(pages)), static_cast<int32_t*>(ptr(tokens)), ptr(ws),
                                 bytes_of(ws), status_of(status), stream.raw),
        "decode_attn_block_select");
  return give({blocks, pages, tokens});
}

int64_t mask_words(int64_t T) { return (T + 31) / 32; }

PyObject* tree_mask(PyObject* const* a, Py_ssize_t n) {
  count(n, 8);  // parents, seq_lens, max_seq_len, new_lens, mask, positions, status, stream
  const at::Tensor &parents = needed(a[0], "parents"), &lens = needed(a[1], "seq_lens");
  const at::Tensor& new_lens = tensor(a[3], "new_lens");
  at::Tensor mask = tensor(a[4], "mask"), pos = tensor(a[5], "positions");
  const at::Tensor& status = tensor(a[6], "status");
  type_of(parents, at::kInt, "parents");
  if (parents.dim() != 2 || !parents.is_contiguous()) refuse("parents must be dense [batch, tokens]");
  const int64_t B = parents.size(0), T = parents.size(1);
  if (B > 65535 || T < 1 || T > DECODE_ATTN_MAX_TREE)
    refuse("parents must be of 1 to " + std::to_string(DECODE_ATTN_MAX_TREE) + " tokens and at most 65535 requests");
  int_vector(lens, B, "seq_lens");
  if (new_lens.defined()) int_vector(new_lens, B, "new_lens");
  on_current_device({&parents, &lens, &new_lens, &mask, &pos, &status});
  const Stream stream(a[7]);
  if (mask.defined()) dense(mask, at::kInt, {B, T, mask_words(T)}, "mask");
  else mask = new_result({B, T, mask_words(T)}, at::kInt, parents, stream);
  if (pos.defined()) dense(pos, at::kInt, {B, T}, "positions");
  else pos = new_result({B, T}, at::kInt, parents, stream);
  check(decode_attn_tree_mask(static_cast<int32_t>(B), static_cast<int32_t>(T), integer32(a[2], "max_seq_len"),
                              static_cast<const int32_t*>(ptr(parents)), static_cast<const int32_t*>(ptr(new_lens)),
                              static_cast<const int32_t*>(ptr(lens)), static_cast<uint32_t*>(ptr(mask)),
                              static_cast<int32_t*>(ptr(pos)), status_of(status), stream.raw),
        "decode_attn_tree_mask");
  return give({mask, pos});
}

// Attention whose rows see what a tree's mask (or, without one, cross
// attention) says.
PyObject* rows_attention(PyObject* const* a, const at::Tensor& mask, bool tree) {
  // q, k_cache, v_cache, block_table, seq_lens, [mask], own_lens, max_seq_len, scale, num_splits,
  // k_scale, v_scale, k_sf, v_sf, out, lse, workspace, status, stream
  const at::Tensor& q = needed(a[0], "q");
  const at::Tensor &kc = needed(a[1], "k_cache"), &vc = needed(a[2], "v_cache");
  const at::Tensor &bt = tensor(a[3], "block_table"), &lens = needed(a[4], "seq_lens");
  a += tree ? 1 : 0;
  const at::Tensor& own = tensor(a[5], tree ? "new_lens" : "q_lens");
  const at::Tensor &k_sf = tensor(a[11], "k_sf"), &v_sf = tensor(a[12], "v_sf");
  const at::Tensor &out0 = tensor(a[13], "out"), &lse0 = tensor(a[14], "lse");
  const at::Tensor &given = tensor(a[15], "workspace"), &status = tensor(a[16], "status");
  if (q.dim() != 4) refuse("q must be [batch, tokens, heads, 128]");
  const int64_t B = q.size(0), T = q.size(1);
  heads_tensor(q, B, T, "q");
  int_vector(lens, B, "seq_lens");
  if (own.defined()) int_vector(own, B, tree ? "new_lens" : "q_lens");
  int64_t mask_step = 0;
  if (tree) {
    type_of(mask, at::kInt, "mask");
    const int64_t W = mask_words(T);
    if (mask.dim() != 3 || (mask.size(0) != B && mask.size(0) != 1) || mask.size(1) != T || mask.size(2) != W ||
        (W > 1 && mask.stride(2) != 1) || (T > 1 && mask.stride(1) != W) || (mask.size(0) > 1 && mask.stride(0) < 0))
      refuse("mask must be " + dims({B, T, W}) + " (or one request's, for all), its rows dense");
    mask_step = mask.size(0) > 1 ? mask.stride(0) : 0;
  }
  const Cache c = cache_args(kc, vc, k_sf, v_sf, true);
  decode_attn_params p = cache_params(B, T, q.size(2), c, kc, bt, integer32(a[6], "max_seq_len"), false,
                                      scale_or_default(a[7]), number(a[9]), number(a[10]));
  on_current_device({&q, &kc, &vc, &k_sf, &v_sf, &bt, &lens, &own, &mask, &given, &status, &out0, &lse0});
  const Stream stream(a[17]);
  const at::Tensor out = out_or_new(out0, q, stream), lse = lse_or_new(lse0, q, stream);
  q_strides(p, q, out);
  const int32_t splits = std::max<int32_t>(0, integer32(a[8], "num_splits"));
  const char* where = tree ? "decode_attn_tree" : "decode_attn_cross";
  const int32_t *own_p = static_cast<const int32_t*>(ptr(own)), *bt_p = static_cast<const int32_t*>(ptr(bt)),
                *lens_p = static_cast<const int32_t*>(ptr(lens));
  auto run = [&](const at::Tensor& ws) {
    return tree ? decode_attn_tree(&p, &c.c, ptr(q), static_cast<const uint32_t*>(ptr(mask)), mask_step, own_p, bt_p,
                                   lens_p, ptr(out), static_cast<float*>(ptr(lse)), splits, ptr(ws), bytes_of(ws),
                                   status_of(status), stream.raw)
                : decode_attn_cross(&p, &c.c, ptr(q), own_p, bt_p, lens_p, ptr(out), static_cast<float*>(ptr(lse)),
                                    splits, ptr(ws), bytes_of(ws), status_of(status), stream.raw);
  };
  // (a call that the workspace given, or none, suffices for runs in it: nothing is
  // launched where it does not)
  int rc = run(given.defined() && given.is_contiguous() ? given : undefined());
  if (rc == DA_ERR_WORKSPACE) {
    size_t need = 0;
    check(tree ? decode_attn_tree_workspace_bytes(&p, &c.c, splits, &need)
               : decode_attn_cross_workspace_bytes(&p, &c.c, splits, &need),
          where);
    rc = run(workspace_or_new(undefined(), need, q));
  }
  check(rc, where);
  return give({out, lse});
}

PyObject* tree(PyObject* const* a, Py_ssize_t n) {
  count(n, 19);
  return rows_attention(a, needed(a[5], "mask"), true);
}

PyObject* cross(PyObject* const* a, Py_ssize_t n) {
  count(n, 18);
  return rows_attention(a, undefined(), false);
}

PyObject* cache_keep(PyObject* const* a, Py_ssize_t n) {
  count(n, 14);
  // k_cache, v_cache, block_table, seq_lens, keep, counts, new_tokens, max_seq_len, new_lens,
  // k_sf, v_sf, out_lens, status, stream
  const at::Tensor &kc = needed(a[0], "k_cache"), &vc = needed(a[1], "v_cache");
  const at::Tensor &bt = tensor(a[2], "block_table"), &lens = needed(a[3], "seq_lens");
  const at::Tensor &keep = needed(a[4], "keep"), &counts = needed(a[5], "counts");
  const at::Tensor& new_lens = tensor(a[8], "new_lens");
  const at::Tensor &k_sf = tensor(a[9], "k_sf"), &v_sf = tensor(a[10], "v_sf");
  at::Tensor out_lens = tensor(a[11], "out_lens");
  const at::Tensor& status = tensor(a[12], "status");
  type_of(keep, at::kInt, "keep");
  if (keep.dim() != 2 || !keep.is_contiguous()) refuse("keep must be dense [batch, tokens]");
  const int64_t B = keep.size(0), M = keep.size(1);
  const int32_t T = integer32(a[6], "new_tokens");
  if (T < 1 || T > DECODE_ATTN_MAX_TREE || M > T)
    refuse("new_tokens must be 1 to " + std::to_string(DECODE_ATTN_MAX_TREE) + ", and keep no wider");
  int_vector(lens, B, "seq_lens");
  int_vector(counts, B, "counts");
  if (new_lens.defined()) int_vector(new_lens, B, "new_lens");
  if (out_lens.defined()) int_vector(out_lens, B, "out_lens");
  const Cache c = cache_args(kc, vc, k_sf, v_sf, true);
  const decode_attn_params p =
      cache_params(B, T, c.heads, c, kc, bt, integer32(a[7], "max_seq_len"), false, 1.f, 1.0, 1.0);
  on_current_device({&kc, &vc, &bt, &lens, &keep, &counts, &new_lens, &k_sf, &v_sf, &out_lens, &status});
  const Stream stream(a[13]);
  if (!out_lens.defined()) out_lens = new_result({B}, at::kInt, lens, stream);
  check(decode_attn_cache_keep(&p, &c.c, static_cast<const int32_t*>(ptr(keep)), static_cast<int32_t>(M),
                               static_cast<const int32_t*>(ptr(counts)), static_cast<const int32_t*>(ptr(new_lens)),
                               static_cast<const int32_t*>(ptr(bt)), static_cast<const int32_t*>(ptr(lens)),
                               static_cast<int32_t*>(ptr(out_lens)), status_of(status), stream.raw),
        "decode_attn_cache_keep");
  return give(out_lens);
}

PyObject* cache_read(PyObject* const* a, Py_ssize_t n) {
  count(n, 15);
  // k_cache, v_cache, block_table, seq_lens, max_seq_len, starts, offsets, k_scale, v_scale,
  // k_sf, v_sf, k_out, v_out, status, stream
  const at::Tensor &kc = needed(a[0], "k_cache"), &vc = needed(a[1], "v_cache");
  const at::Tensor &bt = tensor(a[2], "block_table"), &lens = needed(a[3], "seq_lens");
  const int32_t max_seq_len = integer32(a[4], "max_seq_len");
  const at::Tensor &starts = tensor(a[5], "starts"), &offsets = tensor(a[6], "offsets");
  const at::Tensor &k_sf = tensor(a[9], "k_sf"), &v_sf = tensor(a[10], "v_sf");
  at::Tensor k = tensor(a[11], "k_out"), v = tensor(a[12], "v_out");
  const at::Tensor& status = tensor(a[13], "status");
  if (lens.dim() != 1) refuse("seq_lens must be [batch]");
  const int64_t B = lens.size(0);
  int_vector(lens, B, "seq_lens");
  if (starts.defined()) int_vector(starts, B, "starts");
  if (offsets.defined()) int_vector(offsets, B, "offsets");
  const Cache c = cache_args(kc, vc, k_sf, v_sf, true);
  const decode_attn_params p =
      cache_params(B, 1, c.heads, c, kc, bt, max_seq_len, false, 1.f, number(a[7]), number(a[8]));
  if (k.defined() != v.defined()) refuse("k_out and v_out are given together");
  if (!k.defined() && offsets.defined()) refuse("offsets need k_out and v_out");
  on_current_device({&kc, &vc, &bt, &lens, &starts, &offsets, &k_sf, &v_sf, &k, &v, &status});
  const Stream stream(a[14]);
  if (!k.defined()) {
    if (max_seq_len < 0) refuse("max_seq_len is negative");
    for (at::Tensor* t : {&k, &v}) {
      *t = at::zeros({B, max_seq_len, c.heads, kD}, kc.options().dtype(at::kBFloat16));
      stream.returns(*t);
    }
  }
  decode_attn_read r;
  std::memset(&r, 0, sizeof(r));
  const int64_t first = offsets.defined() ? 0 : 1;  // the dimension of tokens
  for (const at::Tensor* t : {&k, &v}) {
    type_of(*t, at::kBFloat16, "k_out or v_out");
    if (t->dim() != 3 + first || (first == 1 && t->size(0) != B) || t->size(first + 1) != c.heads ||
        t->size(first + 2) != kD || t->stride(first + 2) != 1)
      refuse("k_out and v_out must be " +
             (first == 1 ? "[" + std::to_string(B) + ", tokens, " : std::string("[rows, ")) + std::to_string(c.heads) +
             ", 128], their last dimension dense");
  }
  if (k.sizes() != v.sizes() || !same_steps(k, v)) refuse("k_out and v_out differ in shape or strides");
  if (k.size(first) > INT32_MAX) refuse("k_out has too many rows");
  r.max_tokens = offsets.defined() ? max_seq_len : static_cast<int32_t>(k.size(1));
  r.rows = first == 0 ? k.size(0) : 0;
  r.stride_batch = first == 1 ? step(k, 0) : 4 * kD;
  r.stride_token = step(k, first);
  r.stride_head = step(k, first + 1);
  check(decode_attn_cache_read(&p, &c.c, &r, static_cast<const int32_t*>(ptr(starts)),
                               static_cast<const int32_t*>(ptr(offsets)), static_cast<const int32_t*>(ptr(bt)),
                               static_cast<const int32_t*>(ptr(lens)), ptr(k), ptr(v), status_of(status), stream.raw),
        "decode_attn_cache_read");
  return give({k, v});
}

PyObject* set_error(PyObject* const* a, Py_ssize_t n) {
  count(n, 1);
  Py_INCREF(a[0]);
  Py_XDECREF(g_error);
  g_error = a[0];
  Py_RETURN_NONE;
}

// Runs an entry and turns what it throws into Python exceptions: a refusal
// into ValueError, a code of the C ABI into DecodeAttnError, torch's own
// errors (out of memory) as torch raises them.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Refusal& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const CallError& e) {
    PyObject* x = g_error != nullptr ? PyObject_CallFunction(g_error, "is", e.code, e.where) : nullptr;
    if (x != nullptr) {
      PyErr_SetObject(g_error, x);
      Py_DECREF(x);
    } else if (!PyErr_Occurred()) {
      PyErr_Format(PyExc_RuntimeError, "%s failed (code %d)", e.where, e.code);
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

// (FASTCALL functions are registered through PyCFunction's type)
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>));
}

PyMethodDef g_methods[] = {
    {"rope_table", fast<rope_table>(), METH_FASTCALL, nullptr},
    {"rope_append", fast<rope_append>(), METH_FASTCALL, nullptr},
    {"block_digest", fast<block_digest>(), METH_FASTCALL, nullptr},
    {"decode_cached", fast<decode_cached>(), METH_FASTCALL, nullptr},
    {"block_select", fast<block_select>(), METH_FASTCALL, nullptr},
    {"sparse", fast<sparse>(), METH_FASTCALL, nullptr},
    {"tree_mask", fast<tree_mask>(), METH_FASTCALL, nullptr},
    {"tree", fast<tree>(), METH_FASTCALL, nullptr},
    {"cross", fast<cross>(), METH_FASTCALL, nullptr},
    {"cache_keep", fast<cache_keep>(), METH_FASTCALL, nullptr},
    {"cache_read", fast<cache_read>(), METH_FASTCALL, nullptr},
    {"set_error", fast<set_error>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&g_module); }
