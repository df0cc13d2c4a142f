// fa_binding.cpp - the Python binding of the calls that are short on the GPU (norm
// and rotation, append, pages, shared-prefix decode): checks of arguments,
// outputs and workspaces, and the call of the C ABI in include/fa_b200.h.
//
// These calls run for 3 to 30 us, and their checks and marshalling in Python
// took 11 to 37 us of the host; here a tensor's type, device, shape and strides
// are fields.  A call, one after another: qk_norm_rope of 335 tokens 16.1 -> 7.2
// us, its gradient of 999 tokens 26.8 -> 12.0, append_paged of 16 tokens 17.6 ->
// 6.5, decode_shared of 3 sequences 25.4 -> 13.4.
//
// The module calls whichever build of libfa_b200 the Python side has loaded: bind()
// hands over the addresses of its entry points.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <optional>
#include <string>
#include <vector>

#include "../../include/fa_b200.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;

struct {
  decltype(&fa_qk_norm_rope) qk_norm_rope;
  decltype(&fa_qk_norm_rope_bwd) qk_norm_rope_bwd;
  decltype(&fa_qk_norm_rope_bwd_workspace_size) qk_norm_rope_bwd_workspace_size;
  decltype(&fa_append_paged) append_paged;
  decltype(&fa_pages_workspace_size) pages_workspace_size;
  decltype(&fa_pages_copy) pages_copy;
  decltype(&fa_pages_reserve) pages_reserve;
  decltype(&fa_pages_fork) pages_fork;
  decltype(&fa_pages_free) pages_free;
  decltype(&fa_pages_compact) pages_compact;
  decltype(&fa_decode_shared_workspace_size) decode_shared_workspace_size;
  decltype(&fa_decode_shared) decode_shared;
} api;
PyObject* failure = nullptr;  // the class FAError

void bind(const py::dict& at, const py::object& error) {
  auto set = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(at[name].cast<uintptr_t>());
  };
  set(api.qk_norm_rope, "fa_qk_norm_rope");
  set(api.qk_norm_rope_bwd, "fa_qk_norm_rope_bwd");
  set(api.qk_norm_rope_bwd_workspace_size, "fa_qk_norm_rope_bwd_workspace_size");
  set(api.append_paged, "fa_append_paged");
  set(api.pages_workspace_size, "fa_pages_workspace_size");
  set(api.pages_copy, "fa_pages_copy");
  set(api.pages_reserve, "fa_pages_reserve");
  set(api.pages_fork, "fa_pages_fork");
  set(api.pages_free, "fa_pages_free");
  set(api.pages_compact, "fa_pages_compact");
  set(api.decode_shared_workspace_size, "fa_decode_shared_workspace_size");
  set(api.decode_shared, "fa_decode_shared");
  failure = py::object(error).release().ptr();
}

std::string word(const std::string& v) { return v; }
std::string word(const char* v) { return v; }
std::string word(int v) { return std::to_string(v); }
std::string word(int64_t v) { return std::to_string(v); }
template <typename... A>
std::string text(const A&... a) {
  return (word(a) + ...);
}

std::string list(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + ")";
}

[[noreturn]] void refuse(const std::string& why) { throw py::value_error(why); }

// Calls into the library without the interpreter's lock; raises FAError.
template <typename F, typename... A>
void call(const char* name, F f, A... a) {
  fa_status st;
  {
    py::gil_scoped_release unlocked;
    st = f(a...);
  }
  if (st != FA_OK) {
    const py::object e =
        py::reinterpret_borrow<py::object>(failure)(name, static_cast<int>(st));
    PyErr_SetObject(failure, e.ptr());
    throw py::error_already_set();
  }
}

// The current device, which has to hold t.
int home(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(text(name, " must be a CUDA tensor"));
  const int dev = t.get_device();
  if (dev != c10::cuda::current_device())
    refuse(text(name, " is on cuda:", dev, ", not on the current device"));
  return dev;
}

// Type, dimensions and device; strides are the caller's business.
void on(const Tensor& t, const char* name, at::ScalarType type, int ndim, int dev) {
  if (t.scalar_type() != type)
    throw py::type_error(text(name, " must be ", toString(type), ", got ", toString(t.scalar_type())));
  if (t.dim() != ndim) refuse(text(name, " must have ", ndim, " dims, got ", list(t.sizes())));
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(text(name, " must be on cuda:", dev, ", got ", t.device().str()));
}

// A contiguous vector of n values.
template <typename V>
V* vec(const Tensor& t, const char* name, at::ScalarType type, int64_t n, int dev) {
  on(t, name, type, 1, dev);
  if (t.numel() != n || !t.is_contiguous())
    refuse(text(name, " must be contiguous with ", n, " entries, got ", list(t.sizes())));
  return static_cast<V*>(t.data_ptr());
}
int* ints(const Tensor& t, const char* name, int64_t n, int dev) {
  return vec<int>(t, name, at::kInt, n, dev);
}
int* ints(const Maybe& t, const char* name, int64_t n, int dev) {
  return t ? ints(*t, name, n, dev) : nullptr;
}

int small(int64_t v, const char* name) {
  if (v < 0 || v > 0x7fffffff) refuse(text(name, " is out of range: ", v));
  return static_cast<int>(v);
}

// The stream of a call: the given one (a torch.cuda.Stream) or the current one.
// While it lives, allocations belong to that stream.
struct OnStream {
  c10::cuda::OptionalCUDAStreamGuard guard;
  cudaStream_t raw;
  OnStream(const py::object& stream, int dev) {
    if (stream.is_none()) {
      raw = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
      return;
    }
    if (stream.attr("device_index").cast<int>() != dev)
      refuse("stream belongs to another device than the tensors");
    const c10::cuda::CUDAStream s = c10::cuda::CUDAStream::unpack3(
        stream.attr("stream_id").cast<int64_t>(), static_cast<c10::DeviceIndex>(dev),
        static_cast<c10::DeviceType>(stream.attr("device_type").cast<int64_t>()));
    guard.reset_stream(s);
    raw = s.stream();
  }
  operator fa_stream_t() const { return raw; }
};

Tensor bytes(size_t n, const Tensor& like) {
  return at::empty({static_cast<int64_t>(n)}, like.options().dtype(at::kByte));
}
size_t size_of(const Tensor& t) { return static_cast<size_t>(t.nbytes()); }
// The caller's workspace: as many bytes on the call's device as it says.
const Tensor& scratch(const Tensor& t, int dev) {
  if (!t.is_contiguous()) refuse("workspace must be contiguous");
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(text("workspace must be on cuda:", dev, ", got ", t.device().str()));
  return t;
}

// ---------------------------------------------------------------- rows
// Element strides (batch, head, token) of [B, H, N, d] or [T, H, d] rows.
void row_strides(const Tensor& t, const char* name, bool written, long long* out) {
  const auto size = t.sizes();
  const auto stride = t.strides();
  const bool packed = t.dim() == 3;
  const int64_t n[3] = {packed ? 1 : size[0], size[1], packed ? size[0] : size[2]};
  const int64_t s[3] = {packed ? 0 : stride[0], stride[1], packed ? stride[0] : stride[2]};
  bool bad = stride.back() != 1, overlap = false;
  for (int i = 0; i < 3; ++i) {
    out[i] = n[i] > 1 ? s[i] : 0;
    bad = bad || (out[i] & 7) != 0;
    overlap = overlap || (n[i] > 1 && out[i] == 0);
  }
  if (bad)
    refuse(text(name, ": rows must be contiguous and their strides multiples of 8 elements, got "
                "strides ", list(stride)));
  if (written && overlap && t.numel() > 0) refuse(text(name, ": rows that are written must not overlap"));
}

// The given or a new contiguous output in the shape of `like`, and its strides.
Tensor output(const Maybe& given, const Tensor& like, const char* name, int dev, long long* strides) {
  if (given) {
    on(*given, name, at::kBFloat16, static_cast<int>(like.dim()), dev);
    if (given->sizes() != like.sizes())
      refuse(text(name, " must have the shape ", list(like.sizes()), ", got ", list(given->sizes())));
    row_strides(*given, name, true, strides);
    return *given;
  }
  Tensor o = at::empty(like.sizes(), like.options());
  row_strides(o, name, false, strides);
  return o;
}

struct Heads {
  int B, H, Hkv, N, d;
  bool packed;
  Heads(const Tensor& q, const Tensor& k, int dev) {
    packed = q.dim() == 3;
    on(q, "q", at::kBFloat16, packed ? 3 : 4, dev);
    on(k, "k", at::kBFloat16, packed ? 3 : 4, dev);
    const int n = packed ? 0 : 2;
    if (q.size(n) != k.size(n) || q.size(-1) != k.size(-1) || (!packed && q.size(0) != k.size(0)))
      refuse(text("q and k must be [B, H, N, d] and [B, Hkv, N, d], or [T, H, d] and [T, Hkv, d]; got ",
                  list(q.sizes()), " and ", list(k.sizes())));
    B = packed ? 1 : small(q.size(0), "B");
    H = small(q.size(1), "H");
    Hkv = small(k.size(1), "Hkv");
    N = small(q.size(n), "N");
    d = small(q.size(-1), "d");
  }
};

// Both weights and their common type (0: bf16, 1: float32).
struct Weights {
  const void *q = nullptr, *k = nullptr;
  int type = FA_WEIGHT_BF16;
  Weights(const Maybe& wq, const Maybe& wk, int d, int dev) {
    if (!wq && !wk) return;
    const at::ScalarType t = (wq ? *wq : *wk).scalar_type();
    if (t != at::kBFloat16 && t != at::kFloat)
      throw py::type_error(text("weights must be bfloat16 or float32, got ", toString(t)));
    if (wq) q = vec<void>(*wq, "q_weight", t, d, dev);
    if (wk) k = vec<void>(*wk, "k_weight", t, d, dev);
    type = t == at::kFloat ? FA_WEIGHT_F32 : FA_WEIGHT_BF16;
  }
};

struct Rotation {
  const int* pos = nullptr;
  long long pos_b = 0;
  const float* inv = nullptr;
  int R = 0;
  Rotation(const Maybe& positions, const Maybe& inv_freq, const Heads& s, int dev) {
    if (!inv_freq || inv_freq->numel() == 0) return;
    inv = vec<float>(*inv_freq, "inv_freq", at::kFloat, inv_freq->numel(), dev);
    R = small(2 * inv_freq->numel(), "rotary_dim");
    if (!positions) throw py::type_error("positions must be a tensor");
    if (!s.packed && positions->dim() == 2) {
      on(*positions, "positions", at::kInt, 2, dev);
      if (positions->size(0) != s.B || positions->size(1) != s.N ||
          (s.N > 1 && positions->stride(1) != 1))
        refuse(text("positions must be [", s.B, ", ", s.N, "] with contiguous rows"));
      pos = static_cast<const int*>(positions->data_ptr());
      pos_b = s.B > 1 ? positions->stride(0) : 0;
    } else {
      pos = ints(*positions, "positions", s.N, dev);
    }
  }
};

py::tuple qk_norm_rope(const Tensor& q, const Tensor& k, const Maybe& positions,
                       const Maybe& inv_freq, const Maybe& q_weight, const Maybe& k_weight,
                       double eps, bool interleaved, const Maybe& q_out, const Maybe& k_out,
                       const py::object& stream) {
  const int dev = home(q, "q");
  const Heads s(q, k, dev);
  const Weights w(q_weight, k_weight, s.d, dev);
  const Rotation rot(positions, inv_freq, s, dev);
  const OnStream on_stream(stream, dev);
  long long strides[12];
  row_strides(q, "q", false, strides);
  row_strides(k, "k", false, strides + 3);
  const Tensor qo = output(q_out, q, "q_out", dev, strides + 6);
  const Tensor ko = output(k_out, k, "k_out", dev, strides + 9);
  call("fa_qk_norm_rope", api.qk_norm_rope, q.data_ptr(), k.data_ptr(), w.q, w.k, w.type, rot.pos,
       rot.pos_b, rot.inv, qo.data_ptr(), ko.data_ptr(), strides, s.B, s.H, s.Hkv, s.N, s.d, rot.R,
       interleaved ? 1 : 0, static_cast<float>(eps), static_cast<fa_stream_t>(on_stream));
  return py::make_tuple(qo, ko);
}

py::tuple qk_norm_rope_bwd(const Tensor& q, const Tensor& k, const Tensor& dq_out,
                           const Tensor& dk_out, const Maybe& positions, const Maybe& inv_freq,
                           const Maybe& q_weight, const Maybe& k_weight, double eps,
                           bool interleaved, const Maybe& dq, const Maybe& dk,
                           const Maybe& workspace, const py::object& stream) {
  const int dev = home(q, "q");
  const Heads s(q, k, dev);
  on(dq_out, "dq_out", at::kBFloat16, static_cast<int>(q.dim()), dev);
  on(dk_out, "dk_out", at::kBFloat16, static_cast<int>(q.dim()), dev);
  if (dq_out.sizes() != q.sizes() || dk_out.sizes() != k.sizes())
    refuse("dq_out and dk_out must match q's and k's shapes");
  const Weights w(q_weight, k_weight, s.d, dev);
  const Rotation rot(positions, inv_freq, s, dev);
  const OnStream on_stream(stream, dev);
  long long strides[18];
  row_strides(q, "q", false, strides);
  row_strides(k, "k", false, strides + 3);
  row_strides(dq_out, "dq_out", false, strides + 6);
  row_strides(dk_out, "dk_out", false, strides + 9);
  const Tensor gq = output(dq, q, "dq", dev, strides + 12);
  const Tensor gk = output(dk, k, "dk", dev, strides + 15);
  Maybe dwq, dwk, ws;
  if (workspace) ws = scratch(*workspace, dev);
  const auto f32 = q.options().dtype(at::kFloat);
  if (q_weight) dwq = at::empty({s.d}, f32);
  if (k_weight) dwk = at::empty({s.d}, f32);
  if (!ws && (dwq || dwk)) ws = bytes(api.qk_norm_rope_bwd_workspace_size(s.d), q);
  call("fa_qk_norm_rope_bwd", api.qk_norm_rope_bwd, q.data_ptr(), k.data_ptr(), dq_out.data_ptr(),
       dk_out.data_ptr(), w.q, w.k, w.type, rot.pos, rot.pos_b, rot.inv, gq.data_ptr(), gk.data_ptr(),
       dwq ? static_cast<float*>(dwq->data_ptr()) : nullptr,
       dwk ? static_cast<float*>(dwk->data_ptr()) : nullptr, strides, s.B, s.H, s.Hkv, s.N, s.d, rot.R,
       interleaved ? 1 : 0, static_cast<float>(eps), ws ? ws->data_ptr() : nullptr,
       ws ? size_of(*ws) : size_t{0}, static_cast<fa_stream_t>(on_stream));
  return py::make_tuple(gq, gk, dwq, dwk);
}

// ---------------------------------------------------------------- tables and pools
// A table whose rows are contiguous.
struct Table {
  int* at;
  int rows, cols;
  long long stride;
  Table(const Tensor& t, const char* name, int dev) {
    on(t, name, at::kInt, 2, dev);
    rows = small(t.size(0), name);
    cols = small(t.size(1), name);
    if (cols > 1 && t.stride(1) != 1) refuse(text(name, ": rows must be contiguous"));
    stride = rows > 1 ? t.stride(0) : cols;
    if (stride < cols) refuse(text(name, ": rows must not overlap"));
    this->at = static_cast<int*>(t.data_ptr());
  }
};

struct KvPages {
  int P, Hkv, page, d;
  KvPages(const Tensor& k, const Tensor& v, int dev) {
    on(k, "kpages", at::kBFloat16, 4, dev);
    on(v, "vpages", at::kBFloat16, 4, dev);
    if (k.sizes() != v.sizes() || !k.is_contiguous() || !v.is_contiguous())
      refuse("kpages and vpages must be contiguous [num_pages, Hkv, page_size, d]");
    P = small(k.size(0), "num_pages");
    Hkv = small(k.size(1), "Hkv");
    page = small(k.size(2), "page_size");
    d = small(k.size(3), "d");
  }
};

Tensor append_paged(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& kpages,
                    const Tensor& vpages, const Tensor& block_table, const Tensor& positions,
                    const Maybe& inv_freq, const Maybe& q_weight, const Maybe& k_weight,
                    const Maybe& batch_idx, const Maybe& cache_positions, double eps,
                    bool interleaved, const Maybe& q_out, const py::object& stream) {
  const int dev = home(q, "q");
  on(q, "q", at::kBFloat16, 3, dev);
  on(k, "k", at::kBFloat16, 3, dev);
  on(v, "v", at::kBFloat16, 3, dev);
  const KvPages pages(kpages, vpages, dev);
  const Table table(block_table, "block_table", dev);
  const int T = small(q.size(0), "T"), H = small(q.size(1), "H"), d = small(q.size(2), "d");
  if (pages.d != d || k.size(0) != T || k.size(1) != pages.Hkv || k.size(2) != d ||
      v.sizes() != k.sizes())
    refuse("k and v must be [T, Hkv, d] with the pages' Hkv and d");
  const Weights w(q_weight, k_weight, d, dev);
  const int* pos = ints(positions, "positions", T, dev);
  const float* inv = nullptr;
  int R = 0;
  if (inv_freq && inv_freq->numel() > 0) {
    inv = vec<float>(*inv_freq, "inv_freq", at::kFloat, inv_freq->numel(), dev);
    R = small(2 * inv_freq->numel(), "rotary_dim");
  }
  const int* places = ints(cache_positions, "cache_positions", T, dev);
  const int* seq = ints(batch_idx, "batch_idx", T, dev);
  if (!batch_idx && T > table.rows)
    refuse("without batch_idx there is at most one token per block-table row");
  const OnStream on_stream(stream, dev);
  long long strides[12];
  row_strides(q, "q", false, strides);
  row_strides(k, "k", false, strides + 3);
  row_strides(v, "v", false, strides + 6);
  const Tensor qo = output(q_out, q, "q_out", dev, strides + 9);
  call("fa_append_paged", api.append_paged, q.data_ptr(), k.data_ptr(), v.data_ptr(), w.q, w.k, w.type,
       pos, places, seq, inv, qo.data_ptr(), kpages.data_ptr(), vpages.data_ptr(), table.at, strides, T,
       H, pages.Hkv, d, R, interleaved ? 1 : 0, static_cast<float>(eps), table.rows, pages.page,
       table.cols, table.stride, pages.P, static_cast<fa_stream_t>(on_stream));
  return qo;
}

struct Pools {
  std::vector<void*> at;
  std::vector<size_t> bytes;
  int n, pages = 0;
  Pools(const std::vector<Tensor>& pools, int dev) : n(static_cast<int>(pools.size())) {
    at.reserve(pools.size());
    bytes.reserve(pools.size());
    for (const Tensor& t : pools) {
      if (!t.is_cuda() || t.get_device() != dev)
        refuse(text("pools must be on cuda:", dev, ", got ", t.device().str()));
      if (t.dim() < 2 || !t.is_contiguous() || t.size(0) != pools[0].size(0))
        refuse("pools must be contiguous with the same number of pages");
      at.push_back(t.data_ptr());
      bytes.push_back(t.nbytes() / std::max<int64_t>(t.size(0), 1));
    }
    if (n > 0) pages = small(pools[0].size(0), "num_pages");
  }
  void match(int64_t P) const {
    if (n > 0 && pages != P) refuse(text("refs has ", P, " entries for pools of ", pages, " pages"));
  }
};

void pages_copy(const std::vector<Tensor>& pools, const Tensor& src, const Tensor& dst,
                const py::object& stream) {
  const int dev = home(src, "src");
  const int n = small(src.numel(), "src");
  const int *s = ints(src, "src", n, dev), *d = ints(dst, "dst", n, dev);
  const Pools all(pools, dev);
  const OnStream on_stream(stream, dev);
  call("fa_pages_copy", api.pages_copy, all.at.data(), all.bytes.data(), all.n, all.pages, s, d, n,
       static_cast<fa_stream_t>(on_stream));
}

Tensor pages_reserve(const Tensor& block_table, const Tensor& refs, const Tensor& seq_ids,
                     const Tensor& new_lens, int page_size, const Maybe& granted,
                     const Maybe& workspace, const py::object& stream) {
  const int dev = home(block_table, "block_table");
  const Table table(block_table, "block_table", dev);
  const int P = small(refs.numel(), "refs"), n = small(seq_ids.numel(), "seq_ids");
  int* r = ints(refs, "refs", P, dev);
  const int *ids = ints(seq_ids, "seq_ids", n, dev), *lens = ints(new_lens, "new_lens", n, dev);
  const OnStream on_stream(stream, dev);
  const Tensor out = granted ? *granted : at::empty({n}, seq_ids.options());
  int* g = ints(out, "granted", n, dev);
  const Tensor ws = workspace ? scratch(*workspace, dev) : bytes(api.pages_workspace_size(P, n), refs);
  call("fa_pages_reserve", api.pages_reserve, table.at, table.stride, r, ids, lens, g, table.rows,
       table.cols, P, page_size, n, ws.data_ptr(), size_of(ws), static_cast<fa_stream_t>(on_stream));
  return out;
}

Tensor pages_fork(const std::vector<Tensor>& pools, const Tensor& block_table, const Tensor& seqlens,
                  const Tensor& refs, const Tensor& src, const Tensor& dst, int page_size,
                  const Maybe& made, const Maybe& workspace, const py::object& stream) {
  const int dev = home(block_table, "block_table");
  const Table table(block_table, "block_table", dev);
  const int P = small(refs.numel(), "refs"), n = small(src.numel(), "src");
  const Pools all(pools, dev);
  all.match(P);
  int *r = ints(refs, "refs", P, dev), *lens = ints(seqlens, "seqlens", table.rows, dev);
  const int *a = ints(src, "src", n, dev), *b = ints(dst, "dst", n, dev);
  const OnStream on_stream(stream, dev);
  const Tensor out = made ? *made : at::empty({n}, src.options());
  int* m = ints(out, "made", n, dev);
  const Tensor ws = workspace ? scratch(*workspace, dev) : bytes(api.pages_workspace_size(P, n), refs);
  call("fa_pages_fork", api.pages_fork, all.at.data(), all.bytes.data(), all.n, table.at, table.stride,
       lens, r, a, b, m, table.rows, table.cols, P, page_size, n, ws.data_ptr(), size_of(ws),
       static_cast<fa_stream_t>(on_stream));
  return out;
}

void pages_free(const Tensor& block_table, const Tensor& seqlens, const Tensor& refs,
                const Tensor& seq_ids, const py::object& stream) {
  const int dev = home(block_table, "block_table");
  const Table table(block_table, "block_table", dev);
  const int P = small(refs.numel(), "refs"), n = small(seq_ids.numel(), "seq_ids");
  int *lens = ints(seqlens, "seqlens", table.rows, dev), *r = ints(refs, "refs", P, dev);
  const int* ids = ints(seq_ids, "seq_ids", n, dev);
  const OnStream on_stream(stream, dev);
  call("fa_pages_free", api.pages_free, table.at, table.stride, lens, r, ids, table.rows, table.cols, P,
       n, static_cast<fa_stream_t>(on_stream));
}

Tensor pages_compact(const std::vector<Tensor>& pools, const Tensor& block_table, const Tensor& refs,
                     const Maybe& used, const Maybe& workspace, const py::object& stream) {
  const int dev = home(block_table, "block_table");
  const Table table(block_table, "block_table", dev);
  const int P = small(refs.numel(), "refs");
  const Pools all(pools, dev);
  all.match(P);
  int* r = ints(refs, "refs", P, dev);
  const OnStream on_stream(stream, dev);
  const Tensor out = used ? *used : at::empty({1}, refs.options());
  int* u = ints(out, "used", 1, dev);
  const Tensor ws = workspace ? scratch(*workspace, dev) : bytes(api.pages_workspace_size(P, 0), refs);
  call("fa_pages_compact", api.pages_compact, all.at.data(), all.bytes.data(), all.n, table.at,
       table.stride, r, u, table.rows, table.cols, P, ws.data_ptr(), size_of(ws),
       static_cast<fa_stream_t>(on_stream));
  return out;
}

py::tuple decode_shared(const Tensor& q, const Tensor& kpages, const Tensor& vpages,
                        const Tensor& prefix_table, const Tensor& prefix_lens,
                        const Tensor& block_table, const Tensor& seqlens, const Maybe& cu_batch,
                        const std::optional<double>& scale, const Maybe& out, const Maybe& lse,
                        bool want_lse, const Maybe& workspace, const py::object& stream) {
  const int dev = home(q, "q");
  on(q, "q", at::kBFloat16, 3, dev);
  if (!q.is_contiguous()) refuse("q must be contiguous");
  const int B = small(q.size(0), "B"), H = small(q.size(1), "H"), d = small(q.size(2), "d");
  const KvPages pages(kpages, vpages, dev);
  const Table table(block_table, "block_table", dev), prefix(prefix_table, "prefix_table", dev);
  if (pages.d != d || pages.Hkv < 1 || H % pages.Hkv != 0)
    refuse("page pools must be [num_pages, Hkv, page_size, d] with Hkv dividing H");
  if (table.rows != B) refuse("block_table must have B rows");
  const int* lens = ints(seqlens, "seqlens", B, dev);
  const int* pre_lens = ints(prefix_lens, "prefix_lens", prefix.rows, dev);
  if (!cu_batch && prefix.rows > 1) refuse("several prefixes need cu_batch");
  const int* cu = ints(cu_batch, "cu_batch", static_cast<int64_t>(prefix.rows) + 1, dev);
  const OnStream on_stream(stream, dev);
  Tensor o;
  if (out) {
    o = *out;
    on(o, "out", at::kBFloat16, 3, dev);
    if (o.sizes() != q.sizes() || !o.is_contiguous()) refuse("out must be contiguous and match q");
  } else {
    o = at::empty(q.sizes(), q.options());
  }
  Maybe l = lse;
  if (l) {
    on(*l, "lse", at::kFloat, 2, dev);
    if (l->size(0) != B || l->size(1) != H || !l->is_contiguous())
      refuse("lse must be contiguous [B, H]");
  } else if (want_lse) {
    l = at::empty({B, H}, q.options().dtype(at::kFloat));
  }
  const Tensor ws = workspace ? scratch(*workspace, dev)
                              : bytes(api.decode_shared_workspace_size(B, H, pages.Hkv, prefix.rows, pages.page,
                                                                       prefix.cols, table.cols, d), q);
  call("fa_decode_shared", api.decode_shared, q.data_ptr(), kpages.data_ptr(), vpages.data_ptr(),
       prefix.at, prefix.stride, pre_lens, cu, table.at, table.stride, lens, o.data_ptr(),
       l ? static_cast<float*>(l->data_ptr()) : nullptr, B, H, pages.Hkv, prefix.rows, pages.page,
       prefix.cols, table.cols, pages.P, d,
       static_cast<float>(scale ? *scale : 1.0 / std::sqrt(static_cast<double>(d))), ws.data_ptr(),
       size_of(ws), static_cast<fa_stream_t>(on_stream));
  return py::make_tuple(o, l);
}

}  // namespace

PYBIND11_MODULE(_fa_native, m) {
  m.def("bind", &bind);
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("qk_norm_rope_bwd", &qk_norm_rope_bwd);
  m.def("append_paged", &append_paged);
  m.def("pages_copy", &pages_copy);
  m.def("pages_reserve", &pages_reserve);
  m.def("pages_fork", &pages_fork);
  m.def("pages_free", &pages_free);
  m.def("pages_compact", &pages_compact);
  m.def("decode_shared", &decode_shared);
  m.def("check_workspace", [](const Tensor& t, int dev) { scratch(t, dev); });
  m.def("row_strides", [](const Tensor& t, const char* name, bool written) {
    long long s[3];
    row_strides(t, name, written, s);
    return py::make_tuple(s[0], s[1], s[2]);
  });
}
