// Argument marshalling of the operators on given arrays for Python callers: the
// same calls of the C ABI binding.py makes through ctypes, with the outputs
// allocated and the argument structs filled here.  A call whose work is a few
// microseconds is bound by the host (one quantized row: 7.8 us through ctypes, its
// kernel 4.6).
//
// Each function returns None for anything it does not take as it stands (dtypes,
// devices, shapes, strides that need a copy): the caller then goes through
// binding.py, which copies or says what is wrong.  It computes nothing itself.
// The library's functions arrive as addresses (bind()), the stream as a number.
#include <ATen/ATen.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <unordered_map>

#include "../../include/stce.h"

namespace py = pybind11;
using at::Tensor;
using std::optional;

namespace {

decltype(&stce_fp8_quantize_blocks) f_quantize = nullptr;
decltype(&stce_fp8_block_matmul_workspace_bytes) f_matmul_ws = nullptr;
decltype(&stce_fp8_block_matmul) f_matmul = nullptr;
decltype(&stce_token_workspace_bytes) f_token_ws = nullptr;
decltype(&stce_token_logprobs) f_token = nullptr;
decltype(&stce_token_logprobs_backward) f_token_grad = nullptr;

void bind(const std::unordered_map<std::string, uintptr_t>& a) {
  f_quantize = (decltype(f_quantize))a.at("stce_fp8_quantize_blocks");
  f_matmul_ws = (decltype(f_matmul_ws))a.at("stce_fp8_block_matmul_workspace_bytes");
  f_matmul = (decltype(f_matmul))a.at("stce_fp8_block_matmul");
  f_token_ws = (decltype(f_token_ws))a.at("stce_token_workspace_bytes");
  f_token = (decltype(f_token))a.at("stce_token_logprobs");
  f_token_grad = (decltype(f_token_grad))a.at("stce_token_logprobs_backward");
}

int dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return STCE_DT_BF16;
    case at::kHalf: return STCE_DT_F16;
    case at::kFloat: return STCE_DT_F32;
    default: return 0;
  }
}

// a 2-d matrix on GPU `dev` with unit-stride rows that do not overlap
bool rows_ok(const Tensor& t, int dev) {
  return t.dim() == 2 && t.is_cuda() && t.get_device() == dev && t.size(0) > 0 && t.size(1) > 0 &&
         (t.is_contiguous() ||
          ((t.size(1) == 1 || t.stride(1) == 1) && (t.size(0) == 1 || t.stride(0) >= t.size(1))));
}
int64_t ld_of(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

bool vector_ok(const optional<Tensor>& t, int64_t n, int dev) {
  return !t || (t->dim() == 1 && t->size(0) == n && t->scalar_type() == at::kFloat && t->is_cuda() &&
                t->get_device() == dev && t->is_contiguous());
}

template <class T>
T* ptr(const optional<Tensor>& t) {
  return t ? (T*)t->data_ptr() : nullptr;
}

// (status, codes, scales)
py::object quantize(const Tensor& x, bool tile, bool transpose, int dev, uintptr_t stream) {
  const int dt = dtype_of(x);
  if (!dt || !rows_ok(x, dev)) return py::none();
  const int64_t R = x.size(0), C = x.size(1), Q = transpose ? C : R, L = transpose ? R : C;
  const int64_t kp = (L + 15) / 16 * 16, kb = (L + 127) / 128, sr = tile ? (Q + 127) / 128 : Q;
  Tensor codes = at::empty({Q, kp}, x.options().dtype(at::kFloat8_e4m3fn));
  Tensor scales = at::empty_strided({sr, kb}, {1, sr}, x.options().dtype(at::kFloat));
  const int st = f_quantize(x.data_ptr(), dt, R, C, ld_of(x),
                            (tile ? STCE_QUANT_TILE : 0) | (transpose ? STCE_QUANT_TRANSPOSE : 0),
                            (uint8_t*)codes.data_ptr(), kp, (float*)scales.data_ptr(), (void*)stream);
  return py::make_tuple(st, codes, scales);
}

bool codes_ok(const Tensor& q, const Tensor& s, int dev) {
  return (q.scalar_type() == at::kFloat8_e4m3fn || q.scalar_type() == at::kByte) && rows_ok(q, dev) &&
         q.size(1) % 16 == 0 && ld_of(q) % 16 == 0 && (uintptr_t)q.data_ptr() % 16 == 0 && s.dim() == 2 &&
         s.scalar_type() == at::kFloat && s.is_cuda() && s.get_device() == dev &&
         s.size(1) == (q.size(1) + 127) / 128;
}

// (status, out)
py::object matmul(const Tensor& a, const Tensor& sa, const Tensor& b, const Tensor& sb, at::ScalarType out_dtype,
                  int dev, uintptr_t stream) {
  if (!codes_ok(a, sa, dev) || !codes_ok(b, sb, dev)) return py::none();
  const int64_t M = a.size(0), N = b.size(0), K = a.size(1);
  const bool row = sb.size(0) == N, tile = sb.size(0) == (N + 127) / 128;
  if (b.size(1) != K || sa.size(0) != M || !(row || tile)) return py::none();
  if (out_dtype != at::kBFloat16 && out_dtype != at::kHalf && out_dtype != at::kFloat) return py::none();
  Tensor out = at::empty({M, N}, a.options().dtype(out_dtype));
  stce_block_matmul p{M, N, K, (const uint8_t*)a.data_ptr(), ld_of(a), (const float*)sa.data_ptr(), sa.stride(0),
                      sa.stride(1), (const uint8_t*)b.data_ptr(), ld_of(b), (const float*)sb.data_ptr(),
                      sb.stride(0), sb.stride(1), row ? 1 : 128, dtype_of(out), out.data_ptr(), N, 0};
  size_t nb = 0;
  int st = f_matmul_ws(&p, &nb);
  if (!st) {
    Tensor ws;
    if (nb) ws = at::empty({(int64_t)nb}, a.options().dtype(at::kByte));
    st = f_matmul(&p, nb ? ws.data_ptr() : nullptr, nb, (void*)stream);
  }
  return py::make_tuple(st, out);
}

bool token_problem(stce_token_problem& p, const Tensor& z, const optional<Tensor>& tokens,
                   const optional<Tensor>& temperature, int64_t top_n, const optional<int64_t>& ignore, int dev) {
  const int dt = dtype_of(z);
  if (!dt || !rows_ok(z, dev)) return false;
  const int64_t T = z.size(0);
  if (!vector_ok(temperature, T, dev) || top_n < 0 || top_n > 128) return false;
  int64_t K = 0;
  if (tokens) {
    const Tensor& t = *tokens;
    if (t.scalar_type() != at::kLong || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous() ||
        (t.dim() != 1 && t.dim() != 2) || t.size(0) != T)
      return false;
    K = t.dim() == 1 ? 1 : t.size(1);
    if (K > 1024) return false;
  }
  p = stce_token_problem{T, z.size(1), dt, ignore ? STCE_PROBLEM_IGNORE_INDEX : 0, z.data_ptr(), ld_of(z),
                         ptr<float>(temperature), ptr<int64_t>(tokens), (int32_t)K, (int32_t)top_n,
                         ignore ? *ignore : 0};
  return true;
}

// (status, {outputs}, device status or None)
py::object token_logprobs(const Tensor& z, const optional<Tensor>& tokens, const optional<Tensor>& temperature,
                          int64_t top_n, const optional<int64_t>& ignore, bool check, int dev, uintptr_t stream) {
  stce_token_problem p;
  if (!token_problem(p, z, tokens, temperature, top_n, ignore, dev)) return py::none();
  const auto f = z.options().dtype(at::kFloat);
  py::dict out;
  stce_token_outputs o{};
  const Tensor stats = at::empty({p.T, 4}, f), lse = at::empty({p.T}, f), entropy = at::empty({p.T}, f);
  o.stats = (float*)stats.data_ptr();
  o.lse = (float*)lse.data_ptr();
  o.entropy = (float*)entropy.data_ptr();
  out["stats"] = stats;
  out["lse"] = lse;
  out["entropy"] = entropy;
  if (tokens) {
    const Tensor t = at::empty(tokens->sizes(), f);
    o.logprob = (float*)t.data_ptr();
    out["logprob"] = t;
  }
  if (top_n) {
    const Tensor v = at::empty({p.T, top_n}, f), i = at::empty({p.T, top_n}, z.options().dtype(at::kLong));
    o.top_logprob = (float*)v.data_ptr();
    o.top_id = (int64_t*)i.data_ptr();
    out["top_logprob"] = v;
    out["top_id"] = i;
  }
  py::object status = py::none();
  int64_t* dst = nullptr;
  if (check) {
    const Tensor s = at::empty({1}, z.options().dtype(at::kLong));
    dst = (int64_t*)s.data_ptr();
    status = py::cast(s);
  }
  size_t nb = 0;
  int st = f_token_ws(&p, &nb);
  if (!st) {
    Tensor ws;
    if (nb) ws = at::empty({(int64_t)nb}, z.options().dtype(at::kByte));
    st = f_token(&p, &o, dst, nb ? ws.data_ptr() : nullptr, nb, (void*)stream);
  }
  return py::make_tuple(st, out, status);
}

// (status, gradient)
py::object token_grad(const Tensor& z, const optional<Tensor>& tokens, const Tensor& stats,
                      const optional<Tensor>& g_logprob, const optional<Tensor>& g_entropy,
                      const optional<Tensor>& g_lse, const optional<Tensor>& temperature,
                      const optional<int64_t>& ignore, int dev, uintptr_t stream) {
  stce_token_problem p;
  if (!token_problem(p, z, tokens, temperature, 0, ignore, dev)) return py::none();
  if (stats.dim() != 2 || stats.size(0) != p.T || stats.size(1) != 4 || stats.scalar_type() != at::kFloat ||
      !stats.is_cuda() || stats.get_device() != dev || !stats.is_contiguous())
    return py::none();
  if (g_logprob && (!tokens || g_logprob->sizes() != tokens->sizes() || g_logprob->scalar_type() != at::kFloat ||
                    !g_logprob->is_cuda() || g_logprob->get_device() != dev || !g_logprob->is_contiguous()))
    return py::none();
  if (!vector_ok(g_entropy, p.T, dev) || !vector_ok(g_lse, p.T, dev)) return py::none();
  Tensor out = at::empty({p.T, p.V}, z.options());
  const int st = f_token_grad(&p, (const float*)stats.data_ptr(), ptr<float>(g_logprob), ptr<float>(g_entropy),
                              ptr<float>(g_lse), out.data_ptr(), p.V, (void*)stream);
  return py::make_tuple(st, out);
}

// (an allocation that fails is left to binding.py too, whose own raises)
template <auto F, class... A>
py::object guarded(A... a) {
  try {
    return F(a...);
  } catch (const c10::Error&) {
    return py::none();
  }
}
template <auto F, class... A>
auto guard(py::object (*)(A...)) {
  return &guarded<F, A...>;
}

}  // namespace

PYBIND11_MODULE(_marshal, m) {
  m.def("bind", &bind);
  m.def("quantize", guard<&quantize>(&quantize));
  m.def("matmul", guard<&matmul>(&matmul));
  m.def("token_logprobs", guard<&token_logprobs>(&token_logprobs));
  m.def("token_grad", guard<&token_grad>(&token_grad));
}
