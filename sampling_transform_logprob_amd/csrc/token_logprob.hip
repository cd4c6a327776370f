// Log probabilities of given tokens with entropy and top alternatives, and
// the gradient of the logits.
//
// With m the row's largest logit, c = log2(e) / T and x_j = (z_j - m) c, the
// row needs S = sum 2^x_j and E = sum 2^x_j x_j:
//   lse = m / T + ln 2 log2 S,   logprob_y = (z_y - m) / T - ln 2 log2 S,
//   entropy = ln 2 (log2 S - E / S).
// (The difference z - m is formed before the scaling: a row of the type's
// lowest finite value, or one far from zero, loses nothing to it.)
#include "ops.hpp"

namespace stce {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float NEG_INF = -__builtin_huge_valf();
constexpr int TW = 256;        // threads of a workgroup
constexpr int LIST_CAP = 1024; // candidates kept in LDS

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ inline float log2_fast(float x) { return __builtin_amdgcn_logf(x); }

template <class Z>
__device__ inline float to_f32(Z v) {
  return (float)v;
}

__device__ inline bool bad_temperature(float t) { return !(__builtin_isfinite(t) && t > 0.0f); }

// log2(e) / T, kept finite for the smallest temperatures (0 times it is 0)
__device__ inline float inv_temperature(float t) { return fminf(LOG2E / t, 3.4028235e38f); }

// LDS of the selection of a row's (or segment's) largest logits.
struct TopScratch {
  uint64_t list[LIST_CAP];
  uint64_t sorted[TOP_MAX];
  uint64_t cut;
  int count;
};

// Keeps the n largest of the list's count entries (count <= LIST_CAP) in
// sorted[] in decreasing order, zeros past them.  Composites are distinct, so
// an entry's place is the number of larger ones.  All threads call it;
// entries are visible to all (a barrier precedes).
__device__ inline void rank_list(TopScratch& s, int n) {
  const int cnt = s.count;
  for (int i = threadIdx.x; i < n; i += TW)
    if (i >= cnt) s.sorted[i] = 0;
  for (int i = threadIdx.x; i < cnt; i += TW) {
    const uint64_t mine = s.list[i];
    int rank = 0;
    for (int j = 0; j < cnt; ++j) rank += s.list[j] > mine ? 1 : 0;
    if (rank < n) s.sorted[rank] = mine;
  }
  __syncthreads();
}

// The n largest logits above -inf of z[j0 .. j1) in order, by a scan that
// keeps a list and the n-th largest so far as the bar for further entries:
// right for every row, whatever its ties.
template <class Z>
__device__ void scan_top(const Z* z, int64_t j0, int64_t j1, int n, TopScratch& s) {
  if (threadIdx.x == 0) {
    s.cut = 0;
    s.count = 0;
  }
  __syncthreads();
  for (int64_t b = j0; b < j1; b += TW) {
    const int64_t j = b + threadIdx.x;
    const uint64_t cut = s.cut;
    if (j < j1) {
      const float x = to_f32(z[j]);
      const uint64_t c = composite(order_key(x), (uint32_t)j);
      if (x > NEG_INF && c > cut) s.list[atomicAdd(&s.count, 1)] = c;
    }
    __syncthreads();
    if (s.count > LIST_CAP - TW) {
      rank_list(s, n);
      for (int i = threadIdx.x; i < n; i += TW) s.list[i] = s.sorted[i];
      if (threadIdx.x == 0) {
        s.cut = s.sorted[n - 1];
        s.count = n;
      }
      __syncthreads();
    }
  }
  rank_list(s, n);
}

// Sum (or maximum) over the workgroup in a fixed order; every thread gets it.
template <bool MAX>
__device__ inline float block_reduce(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float u = __shfl_xor(v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < TW / 64; ++w) v = MAX ? fmaxf(v, red[w]) : v + red[w];
  return v;
}

// The outputs of one row from its statistics and sorted alternatives.
struct RowOut {
  stce_token_outputs o;
  const int64_t* tokens;
  int64_t V, ignore_index;
  int K, top_n, ignore;
  int64_t* status;
};

template <class Z>
__device__ inline void write_row(const RowOut& r, const Z* z, int64_t t, float temp, float m, float S, float E,
                                 const uint64_t* sorted, int tid, int nthreads) {
  const float nan = __builtin_nanf("");
  const bool bad_t = bad_temperature(temp);
  const bool bad = bad_t || S != S || m == __builtin_huge_valf();
  const bool empty = !bad && m == NEG_INF;
  const float l2 = log2_fast(S);
  if (tid == 0) {
    const float H = bad ? nan : empty ? 0.0f : fmaxf(LN2 * (l2 - E / S), 0.0f);
    if (bad_t && r.status)
      atomicMin((unsigned long long*)r.status, (unsigned long long)((t << 8) | STCE_FIELD_TEMPERATURE));
    if (r.o.lse) r.o.lse[t] = bad ? nan : empty ? NEG_INF : m / temp + LN2 * l2;
    if (r.o.entropy) r.o.entropy[t] = H;
    if (r.o.stats) {
      ((TokenStats*)r.o.stats)[t] = bad     ? TokenStats{nan, nan, nan, nan}
                                    : empty ? TokenStats{NEG_INF, NEG_INF, 0.0f, 0.0f}
                                            : TokenStats{m, LN2 * l2, H, 0.0f};
    }
  }
  for (int i = tid; i < r.K; i += nthreads) {
    const int64_t y = r.tokens[t * r.K + i];
    float lp;
    if (r.ignore && y == r.ignore_index) {
      lp = 0.0f;
    } else if (y < 0 || y >= r.V) {
      lp = nan;
      if (r.status) atomicMin((unsigned long long*)r.status, (unsigned long long)((t << 8) | STCE_FIELD_TARGET));
    } else if (bad || empty) {
      lp = bad ? nan : NEG_INF;
    } else {
      lp = fminf((to_f32(z[y]) - m) / temp - LN2 * l2, 0.0f);
    }
    if (r.o.logprob) r.o.logprob[t * r.K + i] = lp;
  }
  for (int i = tid; i < r.top_n; i += nthreads) {
    const uint64_t v = bad ? 0 : sorted[i];
    if (r.o.top_id) r.o.top_id[t * r.top_n + i] = v ? (int64_t)comp_id(v) : -1;
    if (r.o.top_logprob) {
      const float lp = fminf((key_value(comp_key(v)) - m) / temp - LN2 * l2, 0.0f);
      r.o.top_logprob[t * r.top_n + i] = bad ? nan : v ? lp : NEG_INF;
    }
  }
}

// One workgroup per row, three passes over it: maximum, sums, alternatives.
template <class Z>
__global__ __launch_bounds__(TW) void token_row_kernel(const Z* logits, int64_t ld, const float* temperature,
                                                       RowOut r) {
  __shared__ TopScratch top;
  __shared__ float red[TW / 64];
  const int64_t t = blockIdx.x;
  const Z* z = logits + t * ld;
  const float temp = temperature ? temperature[t] : 1.0f;
  const float c = inv_temperature(temp);
  float m = NEG_INF;
  for (int64_t j = threadIdx.x; j < r.V; j += TW) m = fmaxf(m, to_f32(z[j]));
  m = block_reduce<true>(m, red);
  const float ref = m == NEG_INF ? 0.0f : m;
  float S = 0.0f, E = 0.0f;
  for (int64_t j = threadIdx.x; j < r.V; j += TW) {
    const float x = (to_f32(z[j]) - ref) * c;
    const float e = exp2_fast(x);
    S += e;
    E = __builtin_fmaf(e, fmaxf(x, -200.0f), E);
  }
  S = block_reduce<false>(S, red);
  E = block_reduce<false>(E, red);
  if (r.top_n) scan_top(z, 0, r.V, r.top_n, top);
  write_row(r, z, t, temp, m, S, E, top.sorted, threadIdx.x, TW);
}

// Gradient of the logits, one workgroup per row.
template <class Z>
__global__ __launch_bounds__(TW) void token_grad_kernel(const Z* logits, int64_t ld, const float* temperature,
                                                        const TokenStats* stats, const int64_t* tokens, int K,
                                                        int64_t V, const float* g_lp, const float* g_ent,
                                                        const float* g_lse, Z* grad, int64_t ld_grad) {
  __shared__ float red[TW / 64];
  __shared__ int32_t tok[TOKENS_MAX];
  __shared__ float tg[TOKENS_MAX];
  const int64_t t = blockIdx.x;
  const Z* z = logits + t * ld;
  Z* dz = grad + t * ld_grad;
  const float temp = temperature ? temperature[t] : 1.0f;
  const TokenStats st = stats[t];
  if (bad_temperature(temp) || !(st.m > NEG_INF && st.m < __builtin_huge_valf()) || st.log_sum != st.log_sum) {
    for (int64_t j = threadIdx.x; j < V; j += TW) dz[j] = (Z)0.0f;
    return;
  }
  const float c = inv_temperature(temp), l2 = st.log_sum * LOG2E;
  float g = 0.0f;
  for (int i = threadIdx.x; i < K; i += TW) {
    const int64_t y = tokens[t * K + i];
    const bool ok = y >= 0 && y < V && g_lp && to_f32(z[y]) > NEG_INF;
    tok[i] = ok ? (int32_t)y : -1;
    tg[i] = ok ? g_lp[t * K + i] : 0.0f;
    g += tg[i];
  }
  g = block_reduce<false>(g, red);
  const float ge = g_ent ? g_ent[t] : 0.0f, gl = g_lse ? g_lse[t] : 0.0f;
  const float a0 = (gl - g - ge * st.entropy) / temp, a1 = ge * LN2 / temp;
  for (int64_t j = threadIdx.x; j < V; j += TW) {
    const float x = fmaxf((to_f32(z[j]) - st.m) * c - l2, -200.0f);
    float d = exp2_fast(x) * __builtin_fmaf(-a1, x, a0);
    float own = 0.0f;
    for (int i = 0; i < K; ++i) own += tok[i] == (int32_t)j ? tg[i] : 0.0f;
    dz[j] = (Z)(d + own / temp);
  }
}

template <class Z>
RowOut row_out(const stce_token_problem& p, const stce_token_outputs& o, int64_t* status) {
  return RowOut{o, p.tokens, p.V, p.ignore_index, p.K, p.top_n, p.flags & STCE_PROBLEM_IGNORE_INDEX, status};
}

template <class Z>
hipError_t run_forward(const stce_token_problem& p, const stce_token_outputs& o, int64_t* status, void*,
                       hipStream_t s) {
  const RowOut r = row_out<Z>(p, o, status);
  ProfScope ps(KIND_TOKEN_LOGPROBS, s);
  hipLaunchKernelGGL(token_row_kernel<Z>, dim3((unsigned)p.T), dim3(TW), 0, s, (const Z*)p.logits, p.ld,
                     p.temperature, r);
  return hipGetLastError();
}

template <class Z>
hipError_t run_grad(const stce_token_problem& p, const TokenStats* stats, const float* g_lp, const float* g_ent,
                    const float* g_lse, void* grad, int64_t ld_grad, hipStream_t s) {
  ProfScope ps(KIND_TOKEN_GRAD, s);
  hipLaunchKernelGGL(token_grad_kernel<Z>, dim3((unsigned)p.T), dim3(TW), 0, s, (const Z*)p.logits, p.ld,
                     p.temperature, stats, p.tokens, p.K, p.V, g_lp, g_ent, g_lse, (Z*)grad, ld_grad);
  return hipGetLastError();
}

}  // namespace

size_t token_workspace_bytes(const stce_token_problem&) { return 0; }

hipError_t launch_token_logprobs(const stce_token_problem& p, const stce_token_outputs& o, int64_t* status, void* ws,
                                 hipStream_t s) {
  if (status) {
    const hipError_t e = launch_fill_i64(status, STCE_STATUS_NONE, s);
    if (e) return e;
  }
  switch (p.dtype) {
    case STCE_DT_BF16: return run_forward<bf16>(p, o, status, ws, s);
    case STCE_DT_F16: return run_forward<_Float16>(p, o, status, ws, s);
    default: return run_forward<float>(p, o, status, ws, s);
  }
}

hipError_t launch_token_grad(const stce_token_problem& p, const TokenStats* stats, const float* g_lp,
                             const float* g_ent, const float* g_lse, void* grad, int64_t ld_grad, hipStream_t s) {
  switch (p.dtype) {
    case STCE_DT_BF16: return run_grad<bf16>(p, stats, g_lp, g_ent, g_lse, grad, ld_grad, s);
    case STCE_DT_F16: return run_grad<_Float16>(p, stats, g_lp, g_ent, g_lse, grad, ld_grad, s);
    default: return run_grad<float>(p, stats, g_lp, g_ent, g_lse, grad, ld_grad, s);
  }
}

}  // namespace stce
