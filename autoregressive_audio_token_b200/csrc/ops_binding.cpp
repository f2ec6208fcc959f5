// ops_binding.cpp -- Python binding of include/m3_ops.h (module _ops): shapes,
// types, devices and layouts are checked here, numbers and alignment in the
// library, whose calls it makes.
//
// Native, unlike the ctypes bindings of the other headers: these calls take a
// few microseconds on the GPU and up to 24 arguments, and checking and
// converting those from Python takes longer (12 to 15 us a call, against 3
// to 4 us here).
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>

#include "m3_ops.h"

namespace py = pybind11;
using at::Tensor;
typedef std::optional<Tensor> Maybe;

namespace {

[[noreturn]] void raise(int code, const std::string& what) {
  // M3Error of the package's m3 module, as every binding raises it
  py::object cls = py::module_::import("autoregressive_audio_token_b200.m3").attr("M3Error");
  py::object e = cls(code, what);
  PyErr_SetObject(cls.ptr(), e.ptr());
  throw py::error_already_set();
}

void check(int rc) {
  if (rc != M3_OK) raise(rc, m3_last_error());
}

void want(bool ok, const char* what) {
  if (!ok) raise(M3_EINVAL, what);
}

std::string shape_text(std::initializer_list<int64_t> shape) {
  std::string s = "[";
  for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
  return s + "]";
}

// The address of a contiguous tensor of this type, shape and device.
template <typename T>
T* arr(const char* name, const Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape,
       const at::Device& dev) {
  if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous() ||
      t.device() != dev)
    raise(M3_EINVAL, std::string(name) + ": a contiguous " + at::toString(type) +
                         " tensor of shape " + shape_text(shape) + " on " + dev.str() + " is wanted");
  return static_cast<T*>(t.data_ptr());
}
template <typename T>
T* arr(const char* name, const Maybe& t, at::ScalarType type, std::initializer_list<int64_t> shape,
       const at::Device& dev) {
  return t ? arr<T>(name, *t, type, shape, dev) : nullptr;
}

int count(int64_t n) {
  want(n >= 0 && n <= INT32_MAX, "a size past 2^31 - 1");
  return (int)n;
}

// The device's stream (the given one, or the current one), with the device
// made current while the call runs.
struct On {
  c10::DeviceIndex before, now;
  void* stream;
  On(const at::Device& dev, const py::object& given) {
    want(dev.is_cuda(), "the tensors have to be on a GPU");
    now = dev.index();
    if (given.is_none()) {
      stream = c10::cuda::getCurrentCUDAStream(now).stream();
    } else {
      want(given.attr("device").attr("index").cast<int>() == now,
           "the stream belongs to another device");
      stream = reinterpret_cast<void*>(given.attr("cuda_stream").cast<uintptr_t>());
    }
    before = c10::cuda::current_device();
    if (before != now) c10::cuda::set_device(now);
  }
  ~On() {
    if (before != now) c10::cuda::set_device(before);
  }
};

int kv_type(const Tensor& t) {
  want(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf,
       "the type has to be bfloat16 or float16");
  return t.scalar_type() == at::kHalf ? M3_KV_F16 : M3_KV_BF16;
}

struct Heads {
  void* p;
  int64_t row, head;
};
// A [n, heads, d] tensor with D contiguous.
Heads heads(const char* name, const Tensor& t, int64_t n, int64_t h, int64_t d, const Tensor& like) {
  if (t.scalar_type() != like.scalar_type() || t.device() != like.device() || t.dim() != 3 ||
      t.size(0) != n || t.size(1) != h || t.size(2) != d || (t.stride(2) != 1 && d > 1))
    raise(M3_EINVAL, std::string(name) + ": a " + at::toString(like.scalar_type()) +
                         " tensor of shape " + shape_text({n, h, d}) + " on " +
                         like.device().str() + ", its last dimension contiguous, is wanted");
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}

int32_t* table_of(const Tensor& t, int64_t n, const at::Device& dev) {
  want(t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) == n && t.device() == dev &&
           (t.stride(1) == 1 || t.size(1) <= 1),
       "table: an int32 tensor [requests, max_pages] with contiguous rows is wanted");
  return static_cast<int32_t*>(t.data_ptr());
}

void* pool_of(const Tensor& t, const Tensor& like) {
  want(t.scalar_type() == like.scalar_type() && t.dim() == 5 && t.size(1) == 2 &&
           t.is_contiguous() && t.device() == like.device(),
       "pool: a contiguous tensor [pages, 2, kv heads, page, D] of the type is wanted");
  return t.data_ptr();
}

void three_dims(const Tensor& t, const char* what) { want(t.dim() == 3, what); }

void kv_map(const Tensor& fresh, const Maybe& cached, const Tensor& free_pages, const Tensor& table,
            int64_t page, int64_t n_pages, const Tensor& cu, const Tensor& positions,
            const Tensor& slots, const Tensor& seqs, const Tensor& lens, const Tensor& taken,
            int64_t start, const Maybe& free_at, const py::object& stream) {
  const at::Device dev = fresh.device();
  const int64_t n = fresh.numel(), nt = slots.numel(), nf = free_pages.numel();
  int32_t* tab = table_of(table, n, dev);
  const auto* f = arr<int32_t>("fresh", fresh, at::kInt, {n}, dev);
  const auto* c = arr<int32_t>("cached", cached, at::kInt, {n}, dev);
  const auto* fp = arr<int32_t>("free_pages", free_pages, at::kInt, {nf}, dev);
  const auto* fa = arr<int32_t>("free_at", free_at, at::kInt, {1}, dev);
  auto* cu_p = arr<int32_t>("cu", cu, at::kInt, {n + 1}, dev);
  auto* pos = arr<int32_t>("positions", positions, at::kInt, {nt}, dev);
  auto* sl = arr<int64_t>("slots", slots, at::kLong, {nt}, dev);
  auto* sq = arr<int32_t>("seqs", seqs, at::kInt, {nt}, dev);
  auto* le = arr<int32_t>("lens", lens, at::kInt, {n}, dev);
  auto* ta = arr<int32_t>("taken", taken, at::kInt, {1}, dev);
  On on(dev, stream);
  check(m3_kv_map(count(n), f, c, fp, count(nf), fa, tab, count(table.size(1)), table.stride(0),
                  count(page), count(n_pages), count(start), count(nt), cu_p, pos, sl, sq, le, ta,
                  on.stream));
}

void kv_store(const Tensor& k, const Tensor& v, const Tensor& slots, const Tensor& pool,
              const py::object& stream) {
  const int dt = kv_type(k);
  const int64_t n = slots.numel();
  void* p = pool_of(pool, k);
  const int64_t hk = pool.size(2), page = pool.size(3), d = pool.size(4);
  const Heads kh = heads("k", k, n, hk, d, k), vh = heads("v", v, n, hk, d, k);
  const auto* sl = arr<int64_t>("slots", slots, at::kLong, {n}, k.device());
  On on(k.device(), stream);
  check(m3_kv_store(dt, count(n), count(hk), count(d), kh.p, kh.row, kh.head, vh.p, vh.row, vh.head,
                    sl, p, count(pool.size(0)), count(page), on.stream));
}

void attn_prompt(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu_q,
                 const Tensor& out, const Maybe& lse, const Maybe& cu_k,
                 const std::optional<double>& scale, const py::object& stream) {
  const int dt = kv_type(q);
  three_dims(q, "q: a tensor [tokens, heads, D] is wanted");
  three_dims(k, "k: a tensor [tokens, kv heads, D] is wanted");
  const int64_t nq = q.size(0), nk = k.size(0), hq = q.size(1), hk = k.size(1), d = q.size(2);
  const Heads qh = heads("q", q, nq, hq, d, q), kh = heads("k", k, nk, hk, d, q);
  const Heads vh = heads("v", v, nk, hk, d, q), oh = heads("out", out, nq, hq, d, q);
  const at::Device dev = q.device();
  const int64_t ns = cu_q.numel() - 1;
  want(ns >= 0, "cu_q is empty");
  const auto* cq = arr<int32_t>("cu_q", cu_q, at::kInt, {ns + 1}, dev);
  const auto* ck = arr<int32_t>("cu_k", cu_k, at::kInt, {ns + 1}, dev);
  auto* l = arr<float>("lse", lse, at::kFloat, {nq, hq}, dev);
  On on(dev, stream);
  check(m3_attn_prompt(dt, count(ns), count(nq), count(nk), count(hq), count(hk), count(d), qh.p,
                       qh.row, qh.head, kh.p, kh.row, kh.head, vh.p, vh.row, vh.head, cq, ck,
                       (float)(scale ? *scale : 1.0 / std::sqrt((double)d)), oh.p, oh.row, oh.head,
                       l, on.stream));
}

int64_t attn_prefix_workspace(int64_t n_rows, int64_t hq, int64_t hk, int64_t d,
                              int64_t prefix_pages, int64_t page, int64_t max_pages) {
  auto i = [](int64_t v) { return v < INT32_MIN || v > INT32_MAX ? -1 : (int)v; };
  return m3_attn_prefix_workspace(i(n_rows), i(hq), i(hk), i(d), i(prefix_pages), i(page),
                                  i(max_pages));
}

void attn_prefix(const Tensor& q, const Tensor& pool, const Tensor& prefix_pages,
                 int64_t prefix_len, const Tensor& table, const Tensor& lens, const Tensor& out,
                 const Maybe& lse, const std::optional<double>& scale, const Maybe& workspace,
                 const py::object& stream) {
  const int dt = kv_type(q);
  three_dims(q, "q: a tensor [rows, heads, D] is wanted");
  const int64_t n = q.size(0), hq = q.size(1), d = q.size(2);
  void* p = pool_of(pool, q);
  const int64_t hk = pool.size(2), page = pool.size(3);
  want(pool.size(4) == d, "q and the pool differ in D");
  const Heads qh = heads("q", q, n, hq, d, q), oh = heads("out", out, n, hq, d, q);
  const at::Device dev = q.device();
  const int64_t npp = prefix_pages.numel();
  const auto* pp = arr<int32_t>("prefix_pages", prefix_pages, at::kInt, {npp}, dev);
  const int32_t* tab = table_of(table, n, dev);
  const int64_t mp = table.size(1);
  const auto* le = arr<int32_t>("lens", lens, at::kInt, {n}, dev);
  auto* l = arr<float>("lse", lse, at::kFloat, {n, hq}, dev);
  On on(dev, stream);
  Tensor ws;
  if (workspace) {
    ws = *workspace;
    want(ws.device() == dev && ws.is_contiguous(),
         "workspace: a contiguous tensor on the same GPU is wanted");
  } else {
    // From the stream's own memory: a block of the current stream's may still be
    // in use there, and nothing makes the given stream wait for that.
    c10::cuda::OptionalCUDAStreamGuard on_stream;
    if (!stream.is_none())
      on_stream.reset_stream(
          c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(on.stream), on.now));
    ws = at::empty({attn_prefix_workspace(n, hq, hk, d, npp, page, mp)},
                   at::TensorOptions().dtype(at::kByte).device(dev));
  }
  check(m3_attn_prefix(dt, count(n), count(hq), count(hk), count(d), qh.p, qh.row, qh.head, p,
                       count(pool.size(0)), count(page), pp, count(npp), count(prefix_len), tab,
                       count(mp), table.stride(0), le,
                       (float)(scale ? *scale : 1.0 / std::sqrt((double)d)), oh.p, oh.row, oh.head,
                       l, ws.data_ptr(), (int64_t)ws.nbytes(), on.stream));
}

void logit_rules(const Tensor& logits, const Tensor& out, const Maybe& history,
                 const Maybe& hist_len, const Maybe& repetition, const Maybe& frequency,
                 const Maybe& presence, const Maybe& bias_ids, const Maybe& bias, const Maybe& mask,
                 const Maybe& mask_row, const py::object& stream) {
  const at::ScalarType t = logits.scalar_type();
  want((t == at::kFloat || t == at::kBFloat16 || t == at::kHalf) && logits.dim() == 2,
       "logits: a float32, bfloat16 or float16 tensor [rows, vocab] is wanted");
  const at::Device dev = logits.device();
  const int64_t r = logits.size(0), n = logits.size(1);
  want(out.scalar_type() == t && out.sizes() == logits.sizes() && out.device() == dev,
       "out has to be like logits");
  want(n <= 1 || (logits.stride(1) == 1 && out.stride(1) == 1),
       "logits and out: rows have to be contiguous");
  const int32_t* h = nullptr;
  int64_t nh = 0, ldh = 0;
  if (history) {
    want(history->scalar_type() == at::kInt && history->dim() == 2 && history->size(0) == r &&
             history->device() == dev && (history->stride(1) == 1 || history->size(1) <= 1),
         "history: an int32 tensor [rows, n] with contiguous rows is wanted");
    h = static_cast<int32_t*>(history->data_ptr());
    nh = history->size(1);
    ldh = history->stride(0);
  }
  want(bias_ids.has_value() == bias.has_value(), "bias_ids and bias come together");
  want(!bias || bias->dim() == 2, "bias: a tensor [rows, n] is wanted");
  want(!mask || mask->dim() == 2, "mask: a tensor [masks, words] is wanted");
  const int64_t nb = bias ? bias->size(-1) : 0;
  const int64_t nm = mask ? mask->size(0) : 0;
  const auto* hl = arr<int32_t>("hist_len", hist_len, at::kInt, {r}, dev);
  const auto* rep = arr<float>("repetition", repetition, at::kFloat, {r}, dev);
  const auto* fr = arr<float>("frequency", frequency, at::kFloat, {r}, dev);
  const auto* pr = arr<float>("presence", presence, at::kFloat, {r}, dev);
  const auto* bi = arr<int32_t>("bias_ids", bias_ids, at::kInt, {r, nb}, dev);
  const auto* bv = arr<float>("bias", bias, at::kFloat, {r, nb}, dev);
  const auto* m = arr<int32_t>("mask", mask, at::kInt, {nm, (n + 31) / 32}, dev);
  const auto* mr = arr<int32_t>("mask_row", mask_row, at::kInt, {r}, dev);
  On on(dev, stream);
  check(m3_logit_rules(t == at::kFloat ? M3_LOGITS_F32
                                       : t == at::kBFloat16 ? M3_LOGITS_BF16 : M3_LOGITS_F16,
                       count(r), count(n), logits.data_ptr(), logits.stride(0), out.data_ptr(),
                       out.stride(0), h, count(nh), ldh, hl, rep, fr, pr, bi, bv, count(nb),
                       reinterpret_cast<const uint32_t*>(m), count(nm), mr, on.stream));
}

void sync_status(const py::object& stream) {
  const c10::DeviceIndex dev =
      stream.is_none() ? c10::cuda::current_device()
                       : (c10::DeviceIndex)stream.attr("device").attr("index").cast<int>();
  On on(at::Device(at::kCUDA, dev), stream);
  int rc;
  {
    py::gil_scoped_release free_gil;
    rc = m3_ops_sync_status(on.stream);
  }
  check(rc);
}

}  // namespace

PYBIND11_MODULE(_ops, m) {
  const auto none = py::none();
  m.def("m3_kv_map", &kv_map, py::arg("fresh"), py::arg("cached"), py::arg("free_pages"),
        py::arg("table"), py::arg("page"), py::arg("n_pages"), py::arg("cu"), py::arg("positions"),
        py::arg("slots"), py::arg("seqs"), py::arg("lens"), py::arg("taken"), py::arg("start") = 0,
        py::arg("free_at") = none, py::arg("stream") = none,
        "Page tables and slot maps from the requests' lengths (see m3_ops.h).  table int32\n"
        "[requests, max_pages], rows may be strided; in and out.");
  m.def("m3_kv_store", &kv_store, py::arg("k"), py::arg("v"), py::arg("slots"), py::arg("pool"),
        py::arg("stream") = none,
        "k, v [tokens, kv heads, D] into the slots of pool [pages, 2, kv heads, page, D] (see\n"
        "m3_ops.h).");
  m.def("m3_attn_prompt", &attn_prompt, py::arg("q"), py::arg("k"), py::arg("v"), py::arg("cu_q"),
        py::arg("out"), py::arg("lse") = none, py::arg("cu_k") = none, py::arg("scale") = none,
        py::arg("stream") = none,
        "Causal attention over packed sequences (see m3_ops.h): q, out [n_q, heads, D], k, v\n"
        "[n_k, kv heads, D], lse float32 [n_q, heads]; scale: by default D^-0.5.");
  m.def("m3_attn_prefix_workspace", &attn_prefix_workspace, py::arg("n_rows"), py::arg("heads"),
        py::arg("kv_heads"), py::arg("d"), py::arg("prefix_pages"), py::arg("page"),
        py::arg("max_pages"), "Bytes of workspace of such an m3_attn_prefix call (see m3_ops.h).");
  m.def("m3_attn_prefix", &attn_prefix, py::arg("q"), py::arg("pool"), py::arg("prefix_pages"),
        py::arg("prefix_len"), py::arg("table"), py::arg("lens"), py::arg("out"),
        py::arg("lse") = none, py::arg("scale") = none, py::arg("workspace") = none,
        py::arg("stream") = none,
        "One-token attention of rows that share a prefix (see m3_ops.h): q, out [rows, heads, D],\n"
        "pool [pages, 2, kv heads, page, D], table int32 [rows, max_pages]; workspace: a tensor of\n"
        "m3_attn_prefix_workspace bytes, by default a new one.");
  m.def("m3_logit_rules", &logit_rules, py::arg("logits"), py::arg("out"),
        py::arg("history") = none, py::arg("hist_len") = none, py::arg("repetition") = none,
        py::arg("frequency") = none, py::arg("presence") = none, py::arg("bias_ids") = none,
        py::arg("bias") = none, py::arg("mask") = none, py::arg("mask_row") = none,
        py::arg("stream") = none,
        "Penalties, biases and grammar masks (see m3_ops.h) on logits [rows, vocab] (rows may be\n"
        "strided); out: another such tensor, or logits itself.  history int32 [rows, n], bias_ids\n"
        "int32 and bias float32 [rows, n], mask int32 [masks, words].");
  m.def("m3_ops_sync_status", &sync_status, py::arg("stream") = none,
        "Wait for the stream and raise what a kernel of these calls recorded (see m3_ops.h).");
}
