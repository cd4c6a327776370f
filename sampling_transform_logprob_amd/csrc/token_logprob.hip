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
// an entry's place is the number of larger ones, counted by eight lanes.  All
// threads call it; entries are visible to all (a barrier precedes).
__device__ inline void rank_list(TopScratch& s, int n) {
  constexpr int L = 8;
  const int cnt = s.count, sub = threadIdx.x % L;
  for (int i = threadIdx.x; i < n; i += TW)
    if (i >= cnt) s.sorted[i] = 0;
  // (whole groups of lanes run each pass: the last one's entries past cnt do not count)
  for (int i = threadIdx.x / L; i < (cnt + TW / L - 1) / (TW / L) * (TW / L); i += TW / L) {
    const uint64_t mine = i < cnt ? s.list[i] : 0;
    int rank = 0;
    for (int j = sub; j < cnt; j += 4 * L) {
      uint64_t o[4];  // (four reads in flight)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = s.list[min(j + q * L, LIST_CAP - 1)];
#pragma unroll
      for (int q = 0; q < 4; ++q) rank += (j + q * L < cnt) & (o[q] > mine);
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) rank += __shfl_xor(rank, o);
    if (sub == 0 && i < cnt && rank < n) s.sorted[rank] = mine;
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
    const bool full = s.count > LIST_CAP - TW;
    __syncthreads();  // (every thread has read the count before the next step adds to it)
    if (full) {
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

// Appends a thread's elements that reach `bar` (finite) to the list, as far as it
// goes: one counter access for all of them.
template <int N, class Id>
__device__ inline void push_hits(TopScratch& s, float bar, const float* x, Id id) {
  int hits = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) hits += x[e] >= bar;
  if (!hits) return;
  int at = atomicAdd(&s.count, hits);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (x[e] >= bar) {
      if (at < LIST_CAP) s.list[at] = composite(order_key(x[e]), id(e));
      ++at;
    }
  }
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

// A thread's first given token and its logit, loaded while the row is: at the end
// the two dependent loads would be waited for.
struct Given {
  int64_t y;
  float z;
};
template <class Z>
__device__ inline Given load_given(const RowOut& r, const Z* z, int64_t t, int i) {
  Given g{-1, 0.0f};
  if (i < r.K) {
    g.y = r.tokens[t * r.K + i];
    if (g.y >= 0 && g.y < r.V) g.z = to_f32(z[g.y]);
  }
  return g;
}

template <class Z>
__device__ inline void write_row(const RowOut& r, const Z* z, int64_t t, float temp, float m, float S, float E,
                                 const uint64_t* sorted, Given given, int tid, int nthreads) {
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
    if (i != tid) given = load_given(r, z, t, i);
    const int64_t y = given.y;
    float lp;
    if (r.ignore && y == r.ignore_index) {
      lp = 0.0f;
    } else if (y < 0 || y >= r.V) {
      lp = nan;
      if (r.status) atomicMin((unsigned long long*)r.status, (unsigned long long)((t << 8) | STCE_FIELD_TARGET));
    } else if (bad || empty) {
      lp = bad ? nan : NEG_INF;
    } else {
      lp = fminf((given.z - m) / temp - LN2 * l2, 0.0f);
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

// 16 bytes of a row as fp32 values (rows need no more than their element's
// alignment: the loads are unaligned where the row is).
template <class Z>
struct Granule {
  static constexpr int E = 16 / sizeof(Z);
  struct __attribute__((packed, aligned(sizeof(Z)))) Raw {
    Z v[E];
  };
};

template <class Z>
__device__ inline void load_granule(const Z* z, int64_t j, int64_t V, float* x) {
  constexpr int E = Granule<Z>::E;
  if (j + E <= V) {
    const typename Granule<Z>::Raw r = *(const typename Granule<Z>::Raw*)(z + j);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = to_f32(r.v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = j + e < V ? to_f32(z[j + e]) : NEG_INF;
  }
}

// Order keys of a logit type's values: the low SHIFT bits of the fp32 image
// say nothing (zeros, or ones below zero), so a search skips them.
template <class Z>
struct KeyShift;
template <>
struct KeyShift<bf16> {
  static constexpr int SHIFT = 16;
};
template <>
struct KeyShift<_Float16> {
  static constexpr int SHIFT = 13;
};
template <>
struct KeyShift<float> {
  static constexpr int SHIFT = 0;
};
constexpr uint32_t KEY_LOWEST = 0x00800000u;  // of the lowest finite value; -inf lies one below

// The largest multiple k of 2^SHIFT such that at least n of the wave's 64 NK
// keys reach k (all of them reach 0).
template <int SHIFT, int NK>
__device__ inline uint32_t nth_key(const uint32_t (&key)[NK], int n) {
  uint32_t k = 0;
#pragma unroll
  for (int b = 31; b >= SHIFT; --b) {
    const uint32_t t = k | (1u << b);
    int cnt = 0;
#pragma unroll
    for (int q = 0; q < NK; ++q) cnt += __popcll(__ballot(key[q] >= t));
    k = cnt >= n ? t : k;
  }
  return k;
}

// A lower bound of the n-th largest of at least n values (n <= 256), given as 256
// values or maxima of disjoint groups of them, v[q] of lane l the (64 q + l)-th:
// the n-th largest, or, for few n, the n-th largest of the 64 lanes' maxima (a
// quarter of the counting, which costs about ten cycles an instruction; it lets a
// fifth more values through at n = 20).  Never -inf: what reaches the bound is
// above it.
template <int SHIFT>
__device__ inline float nth_bound(const float (&v)[4], int n) {
  uint32_t k;
  if (n <= 48) {
    const uint32_t key[1] = {order_key(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])))};
    k = nth_key<SHIFT>(key, n);
  } else {
    const uint32_t key[4] = {order_key(v[0]), order_key(v[1]), order_key(v[2]), order_key(v[3])};
    k = nth_key<SHIFT>(key, n);
  }
  // (the value whose key's class k names: its low bits are zeros)
  const uint32_t b = __builtin_bit_cast(uint32_t, key_value(k < KEY_LOWEST ? KEY_LOWEST : k));
  return __builtin_bit_cast(float, b & ~((1u << SHIFT) - 1u));
}

// Maximum and sums of a part of a row relative to that maximum.
struct Partial {
  float m, S, E, pad;
};

// Re-bases (S, E) from maximum m to the maximum of m and mn; returns it.
__device__ inline void rebase(float& m, float& S, float& E, float mn, float c) {
  const float ref = mn == NEG_INF ? 0.0f : mn;
  const float d = fmaxf((m - ref) * c, -200.0f);  // (2^-200 is 0: an empty part has S = 0)
  const float r = exp2_fast(d);
  E = r * __builtin_fmaf(S, d, E);
  S *= r;
  m = mn;
}

struct SegmentPlan {
  int segs;            // workgroups per row
  int tiles;           // tiles of a row
  int tps;             // tiles per segment
  int tpc;             // tiles per cell (see below)
};

// Rows are one workgroup's each where they are short, or from ROWS_A_TILE rows for
// each tile of 8,192 elements on; other rows are cut into segments, which a second
// launch joins.  (20 alternatives, bf16, a workgroup a row against segments: 1 x
// 8,000 6.8 and 9.7 us, 1 x 32,000 9.4 and 9.4, 100 x 32,000 10.1 and 13.6; 8 x
// 64,000 12.8 and 10.8, 100 x 64,000 13.8 and 15.6; 70 x 128,256 20.1 and 17.7, 130 x
// 128,256 20.4 and 21.9; 200 x 151,936 22.7 and 26.2.  Without
// alternatives: 1 x 8,000 4.1 and 5.4, 1 x 32,000 5.9 and 5.4, 100 x 64,000 9.5 and
// 9.4, 130 x 128,256 15.5 and 15.0.)
constexpr int SHORT_TILES = 4, ROWS_A_TILE = 8;
// Rows that fill the chip whatever their length (bf16 rows of 1,000,000, a workgroup a
// row against segments: 300 rows 153 and 124 us, 500 rows 187 and 205).
constexpr int ROWS_FILL = 384;
constexpr int CELLS = 16;      // cells of a thread at most
constexpr int CELL_CAP = 512;  // cells that may hold alternatives

// The alternatives of a segment with so many elements at the bound that the lists
// overflow (a constant row; tokens masked with the lowest finite value): those
// above it, from the threads' own cells (fewer than n groups of threads have
// any), then the bound's own lowest ids, in order from the segment's start until
// there are n.  False: even those above overflow (scan_top then).  (2,048 x
// 128,256 equal bf16 logits: 0.13 ms, as for others; scan_top takes 0.95.)
template <class Z, int EPT>
__device__ bool tied_top(const Z* z, int64_t V, const SegmentPlan& pl, int t0, int t1, const float* cells, int ncell,
                         float bar, int n, TopScratch& s) {
  constexpr int E = Granule<Z>::E, NG = EPT / E, TILE = TW * EPT;
  const int tid = threadIdx.x;
  const float above = __builtin_bit_cast(float, [&] {
    const uint32_t b = __builtin_bit_cast(uint32_t, bar);  // the next float up
    return b == 0x80000000u || b == 0u ? 1u : (b & 0x80000000u) ? b - 1u : b + 1u;
  }());
  if (tid == 0) s.count = 0;
  __syncthreads();
  for (int c = 0; c < ncell; ++c) {
    if (!(cells[c * TW + tid] > bar)) continue;
    for (int q = 0; q < pl.tpc * NG; ++q) {
      const int tile = t0 + c * pl.tpc + q / NG;
      const int64_t j = (int64_t)tile * TILE + (q % NG) * TW * E + tid * E;
      if (tile >= t1 || j >= V) break;
      float x[E];
      load_granule(z, j, V, x);
      push_hits<E>(s, above, x, [&](int e) { return (uint32_t)(j + e); });
    }
  }
  __syncthreads();
  const int greater = s.count;
  __syncthreads();
  if (greater > LIST_CAP - TOP_MAX - TW) return false;
  const int64_t j1 = (int64_t)t1 * TILE < V ? (int64_t)t1 * TILE : V;
  for (int64_t b = (int64_t)t0 * TILE; b < j1; b += TW) {
    const int64_t j = b + tid;
    if (j < j1 && to_f32(z[j]) == bar) s.list[atomicAdd(&s.count, 1)] = composite(order_key(bar), (uint32_t)j);
    __syncthreads();
    const int have = s.count;
    __syncthreads();
    if (have >= n) break;
  }
  rank_list(s, n);
  return true;
}

// One workgroup per segment of a row, one pass over it: a tile is EPT elements
// a thread, 16 bytes at a time, all in flight at once; each thread keeps its
// own running maximum and sums, so the loop has no barrier.  16-bit logits are
// loaded a tile ahead (301 x 32,001 fp16: 13.4 us of GPU time against 14.6; 4,096 x
// 32,000 bf16: 62 against 65); fp32 ones, of twice the registers, are not (256 x
// 50,000: 18.0 us ahead, 16.7 without).
//
// Alternatives cost the loop one LDS write per cell, a cell being a thread's
// elements of tpc consecutive tiles: its maximum.  The n-th largest of the 256
// threads' maxima is a lower bound of the n-th largest element, and little more
// than n elements reach it (20.8 expected of 8,192 random ones for n = 20), so
// after the loop only the cells that reach the bound are read again (a segment of
// one tile has them in registers) and their elements above it ranked.  Rows whose
// ties overflow the lists take tied_top.
//
// Bound by the read: 8,192 x 128,256 bf16 with 20 alternatives in 0.374 ms, 5.6
// TB/s, as without them.  (The whole row in one workgroup's registers, or a list
// kept up through the loop, would cost occupancy or a branch a tile.)  One row of
// 151,936: 10.7 us with the joining launch, 5.7 without alternatives.
template <class Z, int EPT, bool TOP>
__global__ __launch_bounds__(TW) void token_segment_kernel(const Z* logits, int64_t ld, const float* temperature,
                                                           RowOut r, SegmentPlan pl, Partial* part, uint64_t* tops) {
  constexpr int E = Granule<Z>::E, NG = EPT / E, TILE = TW * EPT;
  extern __shared__ float cells[];  // [cells][TW] with TOP
  __shared__ Partial red[TW / 64];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t t = blockIdx.x / pl.segs;
  const int seg = blockIdx.x - (int)t * pl.segs;
  const int t0 = seg * pl.tps, t1 = min(t0 + pl.tps, pl.tiles);
  const Z* z = logits + t * ld;
  const float temp = temperature ? temperature[t] : 1.0f;
  const float c = inv_temperature(temp);
  Given given{-1, 0.0f};
  if (!part) given = load_given(r, z, t, tid);
  float m = NEG_INF, S = 0.0f, Es = 0.0f, cmax = NEG_INF;
  int cell = 0, in_cell = 0;
  typedef typename Granule<Z>::Raw Raw;
  constexpr bool AHEAD = sizeof(Z) == 2;
  Raw raw[NG] = {};  // with AHEAD: the next tile
  const auto fetch = [&](int tile) __attribute__((always_inline)) {
    const int64_t j0 = (int64_t)tile * TILE + tid * E;
    if ((int64_t)(tile + 1) * TILE <= r.V) {
#pragma unroll
      for (int g = 0; g < NG; ++g) raw[g] = *(const Raw*)(z + j0 + g * TW * E);
    } else {
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (j0 + g * TW * E + E <= r.V) raw[g] = *(const Raw*)(z + j0 + g * TW * E);
    }
  };
  float x[EPT];
  if constexpr (AHEAD) fetch(t0);
  for (int tile = t0; tile < t1; ++tile) {
    const int64_t j0 = (int64_t)tile * TILE + tid * E;
    const bool whole = (int64_t)(tile + 1) * TILE <= r.V;
    if constexpr (AHEAD) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[g * E + e] = to_f32(raw[g].v[e]);
      }
      if (!whole) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int64_t j = j0 + g * TW * E;
          if (j + E <= r.V) continue;
#pragma unroll
          for (int e = 0; e < E; ++e) x[g * E + e] = j + e < r.V ? to_f32(z[j + e]) : NEG_INF;
        }
      }
      if (tile + 1 < t1) fetch(tile + 1);
    } else if (whole) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const Raw in = *(const Raw*)(z + j0 + g * TW * E);
#pragma unroll
        for (int e = 0; e < E; ++e) x[g * E + e] = to_f32(in.v[e]);
      }
    } else {
#pragma unroll
      for (int g = 0; g < NG; ++g) load_granule(z, j0 + g * TW * E, r.V, x + g * E);
    }
    float mx = x[0];
#pragma unroll
    for (int e = 1; e < EPT; ++e) mx = fmaxf(mx, x[e]);
    if constexpr (TOP) {
      cmax = fmaxf(cmax, mx);
      if (++in_cell == pl.tpc || tile + 1 == t1) {
        cells[cell * TW + tid] = cmax;
        ++cell;
        in_cell = 0;
        cmax = NEG_INF;
      }
    }
    rebase(m, S, Es, fmaxf(m, mx), c);
    const float ref = m == NEG_INF ? 0.0f : m;
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const float d = (x[e] - ref) * c;
      const float p = exp2_fast(d);
      S += p;
      Es = __builtin_fmaf(p, fmaxf(d, -200.0f), Es);
    }
  }
  const float mine = m;  // (a NaN does not reach it)
  // join the threads: lanes, then waves, each in a fixed order
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float om = __shfl_xor(m, o);
    rebase(m, S, Es, fmaxf(m, om), c);
    S += __shfl_xor(S, o);
    Es += __shfl_xor(Es, o);
  }
  if (lane == 0) red[w] = Partial{m, S, Es, 0.0f};
  __shared__ TopScratch top_s;
  TopScratch& top = top_s;
  __shared__ float tmax[TOP ? TW : 1];
  __shared__ uint16_t list[TOP ? CELL_CAP : 1];
  __shared__ int ncell;
  if constexpr (TOP) {
    tmax[tid] = mine;
    if (tid == 0) {
      ncell = 0;
      top.count = 0;
    }
  }
  __syncthreads();
  float M = red[0].m;
#pragma unroll
  for (int i = 1; i < TW / 64; ++i) M = fmaxf(M, red[i].m);
  S = Es = 0.0f;
#pragma unroll
  for (int i = 0; i < TW / 64; ++i) {
    float pm = red[i].m, pS = red[i].S, pE = red[i].E;
    rebase(pm, pS, pE, M, c);
    S += pS;
    Es += pE;
  }
  if constexpr (TOP) {
    const int n = r.top_n;
    float v[4];
#pragma unroll
    for (int q = 0; q < TW / 64; ++q) v[q] = tmax[q * 64 + lane];
    const float bar = nth_bound<KeyShift<Z>::SHIFT>(v, n);
    const bool one = t1 - t0 == 1;  // the segment's elements are still in registers
    if (one) {
      const int64_t j0 = (int64_t)t0 * TILE + tid * E;
      push_hits<EPT>(top, bar, x, [&](int e) { return (uint32_t)(j0 + e / E * TW * E + e % E); });
    }
    for (int i = 0; i < (one ? 0 : cell); ++i) {
      if (cells[i * TW + tid] >= bar) {
        const int at = atomicAdd(&ncell, 1);
        if (at < CELL_CAP) list[at] = (uint16_t)(i * TW + tid);
      }
    }
    __syncthreads();
    const int nc = ncell;
    if (!one && nc <= CELL_CAP) {
      const int per = pl.tpc * NG;
      for (int i = tid; i < nc * per; i += TW) {
        const int ci = list[i / per], q = i % per;
        const int tile = t0 + ci / TW * pl.tpc + q / NG;
        const int64_t j = (int64_t)tile * TILE + (q % NG) * TW * E + (ci % TW) * E;
        if (tile >= t1 || j >= r.V) continue;
        float x[E];
        load_granule(z, j, r.V, x);
        push_hits<E>(top, bar, x, [&](int e) { return (uint32_t)(j + e); });
      }
      __syncthreads();
    }
    if (nc <= CELL_CAP && top.count <= LIST_CAP) {
      rank_list(top, n);
    } else {
      __syncthreads();
      const int64_t j1 = (int64_t)t1 * TILE;
      if (!tied_top<Z, EPT>(z, r.V, pl, t0, t1, cells, cell, bar, n, top))
        scan_top(z, (int64_t)t0 * TILE, j1 < r.V ? j1 : r.V, n, top);
    }
    if (part)
      for (int i = tid; i < n; i += TW) tops[(size_t)blockIdx.x * n + i] = top.sorted[i];
  }
  if (!part) {
    write_row(r, z, t, temp, M, S, Es, top.sorted, given, tid, TW);
  } else if (tid == 0) {
    part[blockIdx.x] = Partial{M, S, Es, 0.0f};
  }
}

constexpr int JOIN_CAP = 1024;  // alternatives of a row's segments together
constexpr int SEGS_MAX = 128;   // segments of a row

// One workgroup per row: its segments' partial statistics and alternatives
// joined.  The segments' lists are sorted, so the n-th largest of the first
// ceil(n / segs) of each bounds the n-th largest from below; the entries that
// reach it (at most JOIN_CAP: there are no more) are ranked.
template <class Z, bool TOP>
__global__ __launch_bounds__(TW) void token_join_kernel(const Z* logits, int64_t ld, const float* temperature,
                                                        RowOut r, int segs, const Partial* part,
                                                        const uint64_t* tops) {
  __shared__ TopScratch top;
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const int n = r.top_n, total = segs * n;
  float head[4];  // the lists' heads
  uint64_t v[JOIN_CAP / TW];
  if constexpr (TOP) {
    const uint64_t* const row = tops + (size_t)t * total;
    const int heads = (n + segs - 1) / segs * segs;  // < n + segs <= 256
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = q * 64 + lane;
      const uint64_t h = i < heads ? row[(size_t)(i % segs) * n + i / segs] : 0;
      head[q] = h ? key_value(comp_key(h)) : NEG_INF;
    }
#pragma unroll
    for (int q = 0; q < JOIN_CAP / TW; ++q) v[q] = q * TW + tid < total ? row[q * TW + tid] : 0;
    if (tid == 0) top.count = 0;
  }
  const Given given = load_given(r, logits + t * ld, t, tid);
  const float temp = temperature ? temperature[t] : 1.0f;
  const float c = inv_temperature(temp);
  // (every wave joins the statistics by itself, in the same order)
  float m = NEG_INF, S = 0.0f, Es = 0.0f;
#pragma unroll
  for (int q = 0; q < SEGS_MAX / 64; ++q) {
    const int s = q * 64 + lane;
    const Partial p = s < segs ? part[t * segs + s] : Partial{NEG_INF, 0.0f, 0.0f, 0.0f};
    float pm = p.m, pS = p.S, pE = p.E;
    const float mn = fmaxf(m, pm);
    rebase(m, S, Es, mn, c);
    rebase(pm, pS, pE, mn, c);
    S += pS;
    Es += pE;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float om = __shfl_xor(m, o);
    rebase(m, S, Es, fmaxf(m, om), c);
    S += __shfl_xor(S, o);
    Es += __shfl_xor(Es, o);
  }
  if constexpr (TOP) {
    const uint32_t bar = order_key(nth_bound<KeyShift<Z>::SHIFT>(head, n));
    __syncthreads();
    int hits = 0;
#pragma unroll
    for (int q = 0; q < JOIN_CAP / TW; ++q) hits += comp_key(v[q]) >= bar;
    int at = hits ? atomicAdd(&top.count, hits) : 0;
#pragma unroll
    for (int q = 0; q < JOIN_CAP / TW; ++q)
      if (comp_key(v[q]) >= bar) top.list[at++] = v[q];
    __syncthreads();
    rank_list(top, n);
  }
  write_row(r, logits + t * ld, t, temp, m, S, Es, top.sorted, given, tid, TW);
}

// How rows are cut.  Short rows, and rows that fill the chip by themselves, take
// one workgroup each, tiles of 8,192 elements.  Others are cut into segments, about 1,024
// workgroups in all (as many as leave a row's segments' alternatives to one
// joining workgroup), with the smallest tile that makes a segment one tile: all
// its loads are then in flight at once.
struct TokenPlan {
  int ept;  // elements a thread and tile
  SegmentPlan s;
};
TokenPlan plan_tokens(const stce_token_problem& p) {
  TokenPlan t{};
  const int64_t long_tiles = ceil_div(p.V, 8192);
  const bool whole = long_tiles <= SHORT_TILES || p.T >= ROWS_FILL || p.T >= ROWS_A_TILE * long_tiles;
  int64_t most = whole ? 1 : ceil_div(1024, p.T);
  if (most > SEGS_MAX) most = SEGS_MAX;
  if (p.top_n && most > JOIN_CAP / p.top_n) most = JOIN_CAP / p.top_n;
  t.ept = ceil_div(p.V, 2048) <= most ? 8 : ceil_div(p.V, 4096) <= most ? 16 : 32;
  const int64_t tiles = ceil_div(p.V, TW * t.ept);
  if (most > tiles) most = tiles;
  const int64_t tps = ceil_div(tiles, most);
  t.s.segs = (int)ceil_div(tiles, tps);
  t.s.tiles = (int)tiles;
  t.s.tps = (int)tps;
  t.s.tpc = (int)ceil_div(tps, CELLS);
  return t;
}

// Gradient of the logits: dz_j = (p_j (a0 - a1 x_j) + the given tokens' terms) / T
// with x_j = log2 p_j, p_j = 2^x_j, a0 = grad_lse - sum g - grad_entropy H and
// a1 = ln 2 grad_entropy.  One read and one write of the row, 16 bytes a
// thread at a time; a workgroup takes `tiles` tiles of 4 granules a thread.
//
// A given token's element is written once more, after a barrier, by the thread of
// its first occurrence: with the sum of the gradients of all its occurrences, in
// order, added before the one rounding.  So a token given twice gets both, and
// equal calls give equal bits.
//
// Bound by the read and the write: 8,192 x 128,256 bf16 in 0.80 ms, 5.2 TB/s.  (A
// search through the row's tokens at every marked granule took 51 us instead of 18
// for 257 x 32,001 fp32 with 64 tokens a row.)
constexpr int GRAD_NG = 4, GRAD_TILES = 8;  // granules a thread and tile; tiles a workgroup at most

template <class Z, bool FEW>
__global__ __launch_bounds__(TW) void token_grad_kernel(const Z* logits, int64_t ld, const float* temperature,
                                                        const TokenStats* stats, const int64_t* tokens, int K,
                                                        int64_t V, const float* g_lp, const float* g_ent,
                                                        const float* g_lse, Z* grad, int64_t ld_grad, int segs,
                                                        int tiles) {
  constexpr int E = Granule<Z>::E, TILE = TW * E * GRAD_NG;
  constexpr int CAP = FEW ? 8 : TOKENS_MAX;
  typedef typename Granule<Z>::Raw Raw;
  typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
  __shared__ float red[TW / 64];
  __shared__ i32x4 tok4[CAP / 4];
  __shared__ f32x4 tg4[CAP / 4];
  int32_t* const tok = (int32_t*)tok4;
  float* const tg = (float*)tg4;
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x / segs;
  const int64_t j0 = (int64_t)(blockIdx.x - (int)t * segs) * tiles * TILE;
  const int64_t j1 = j0 + (int64_t)tiles * TILE < V ? j0 + (int64_t)tiles * TILE : V;
  const Z* z = logits + t * ld;
  Z* dz = grad + t * ld_grad;
  const float temp = temperature ? temperature[t] : 1.0f;
  const TokenStats st = stats[t];
  const bool none =
      bad_temperature(temp) || !(st.m > NEG_INF && st.m < __builtin_huge_valf()) || st.log_sum != st.log_sum;
  const float c = inv_temperature(temp), l2 = st.log_sum * LOG2E;
  const float rt = fminf(1.0f / temp, 3.4028235e38f);
  float g = 0.0f;
  const int K4 = (K + 3) & ~3;
  if (g_lp) {
    for (int i = tid; i < K4; i += TW) {
      const int64_t y = i < K ? tokens[t * K + i] : -1;
      const bool ok = y >= 0 && y < V && to_f32(z[y]) > NEG_INF;
      const float v = ok ? g_lp[t * K + i] : 0.0f;
      tok[i] = ok ? (int32_t)y : -1;
      tg[i] = v;
      g += v;
    }
    g = block_reduce<false>(g, red);  // (its barriers make the tokens visible)
  }
  const float ge = g_ent ? g_ent[t] : 0.0f, gl = g_lse ? g_lse[t] : 0.0f;
  const float a0 = gl - g - ge * st.entropy, a1 = ge * LN2;
  auto one = [&](Z v) __attribute__((always_inline)) {
    const float x = fmaxf((to_f32(v) - st.m) * c - l2, -200.0f);
    return none ? 0.0f : exp2_fast(x) * __builtin_fmaf(-a1, x, a0) * rt;
  };
  for (int tile = 0; tile < tiles; ++tile) {
    const int64_t b = j0 + (int64_t)tile * TILE + tid * E;
    if (j0 + (int64_t)tile * TILE >= j1) break;
    if (j0 + (int64_t)(tile + 1) * TILE <= V) {
      Raw in[GRAD_NG];
#pragma unroll
      for (int q = 0; q < GRAD_NG; ++q) in[q] = *(const Raw*)(z + b + q * TW * E);
#pragma unroll
      for (int q = 0; q < GRAD_NG; ++q) {
        Raw o;
#pragma unroll
        for (int e = 0; e < E; ++e) o.v[e] = (Z)one(in[q].v[e]);
        *(Raw*)(dz + b + q * TW * E) = o;
      }
    } else {
#pragma unroll
      for (int q = 0; q < GRAD_NG; ++q) {
        const int64_t j = b + q * TW * E;
        if (j + E <= V) {
          const Raw in = *(const Raw*)(z + j);
          Raw o;
#pragma unroll
          for (int e = 0; e < E; ++e) o.v[e] = (Z)one(in.v[e]);
          *(Raw*)(dz + j) = o;
        } else {
          for (int e = 0; e < E; ++e)
            if (j + e < V) dz[j + e] = (Z)one(z[j + e]);
        }
      }
    }
  }
  if (!g_lp || none) return;
  __syncthreads();  // the elements written again below were written above by other threads
  for (int i = tid; i < K; i += TW) {
    const int32_t y = tok[i];
    if (y < j0 || y >= j1) continue;
    bool first = true;
    float v = 0.0f;
    for (int k = 0; k < K4; k += 4) {
      const i32x4 o = tok4[k / 4];
      const f32x4 w = tg4[k / 4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (o[e] == y) {
          v += w[e];
          first = first && k + e >= i;
        }
      }
    }
    if (first) dz[y] = (Z)(one(z[y]) + v * rt);
  }
}

template <class Z>
RowOut row_out(const stce_token_problem& p, const stce_token_outputs& o, int64_t* status) {
  return RowOut{o, p.tokens, p.V, p.ignore_index, p.K, p.top_n, p.flags & STCE_PROBLEM_IGNORE_INDEX, status};
}

template <class Z, int EPT, bool TOP>
void launch_segments(const TokenPlan& pl, const stce_token_problem& p, const RowOut& r, Partial* part, uint64_t* tops,
                     hipStream_t s) {
  const size_t lds = TOP ? sizeof(float) * TW * (size_t)ceil_div(pl.s.tps, pl.s.tpc) : 0;
  hipLaunchKernelGGL((token_segment_kernel<Z, EPT, TOP>), dim3((unsigned)(p.T * pl.s.segs)), dim3(TW), lds, s,
                     (const Z*)p.logits, p.ld, p.temperature, r, pl.s, part, tops);
}

template <class Z, bool TOP>
hipError_t run_forward_as(const stce_token_problem& p, const RowOut& r, void* ws, hipStream_t s) {
  const TokenPlan pl = plan_tokens(p);
  Partial* part = pl.s.segs > 1 ? (Partial*)ws : nullptr;
  uint64_t* tops = part ? (uint64_t*)(part + p.T * pl.s.segs) : nullptr;
  {
    ProfScope ps(KIND_TOKEN_LOGPROBS, s);
    if (pl.ept == 32)
      launch_segments<Z, 32, TOP>(pl, p, r, part, tops, s);
    else if (pl.ept == 16)
      launch_segments<Z, 16, TOP>(pl, p, r, part, tops, s);
    else
      launch_segments<Z, 8, TOP>(pl, p, r, part, tops, s);
  }
  hipError_t e = hipGetLastError();
  if (e || !part) return e;
  ProfScope ps(KIND_TOKEN_MERGE, s);
  hipLaunchKernelGGL((token_join_kernel<Z, TOP>), dim3((unsigned)p.T), dim3(TW), 0, s, (const Z*)p.logits, p.ld,
                     p.temperature, r, pl.s.segs, part, tops);
  return hipGetLastError();
}

template <class Z>
hipError_t run_forward(const stce_token_problem& p, const stce_token_outputs& o, int64_t* status, void* ws,
                       hipStream_t s) {
  const RowOut r = row_out<Z>(p, o, status);
  return r.top_n ? run_forward_as<Z, true>(p, r, ws, s) : run_forward_as<Z, false>(p, r, ws, s);
}

template <class Z>
hipError_t run_grad(const stce_token_problem& p, const TokenStats* stats, const float* g_lp, const float* g_ent,
                    const float* g_lse, void* grad, int64_t ld_grad, hipStream_t s) {
  // as many tiles a workgroup as leave about 2,048 workgroups
  const int64_t all = ceil_div(p.V, (int64_t)TW * Granule<Z>::E * GRAD_NG);
  int64_t tiles = all * p.T / 2048;
  tiles = tiles < 1 ? 1 : tiles > GRAD_TILES ? GRAD_TILES : tiles;
  if (tiles > all) tiles = all;
  const int64_t segs = ceil_div(all, tiles);
  ProfScope ps(KIND_TOKEN_GRAD, s);
  const auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.T * segs)), dim3(TW), 0, s, (const Z*)p.logits, p.ld, p.temperature,
                       stats, p.tokens, p.K, p.V, g_lp, g_ent, g_lse, (Z*)grad, ld_grad, (int)segs, (int)tiles);
  };
  if (p.K <= 8)
    launch(token_grad_kernel<Z, true>);
  else
    launch(token_grad_kernel<Z, false>);
  return hipGetLastError();
}

}  // namespace

size_t token_workspace_bytes(const stce_token_problem& p) {
  const TokenPlan pl = plan_tokens(p);
  if (pl.s.segs == 1) return 0;
  return (size_t)p.T * pl.s.segs * (sizeof(Partial) + sizeof(uint64_t) * (size_t)p.top_n);
}

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
