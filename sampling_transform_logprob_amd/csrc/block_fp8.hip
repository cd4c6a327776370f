// e4m3 quantization with a scale per block of 128, and the product of two
// such matrices.
#include "block_gemm.hpp"
#include "epilogues.hpp"
#include "ops.hpp"

namespace stce {
namespace {

constexpr int QB = 128;  // values per scale along the reduction

// A block's scale a, and what its codes are formed with.  The codes need
// fl32(v / a) exactly only where |v / a| >= 2^-11 (below, every code is a zero),
// and |v| <= 448 a (1 + 2^-22): there the correction step of quot_fast (see
// there) gives the correctly rounded quotient as long as ulp(v / a) ulp(a) and
// the reciprocal stay in range, for a in [2^-92, 2^125]; a smaller a and its
// values are first multiplied by f = 2^100, which is exact.  The largest a is
// below 2^120.
struct BlockScale {
  float a, af, r, f;
  bool finite;
};
// From the block's largest magnitude (infinite when it holds a NaN or an
// infinity).
__device__ inline BlockScale block_scale(float mx) {
  BlockScale b;
  b.finite = mx < __builtin_huge_valf();
  const float q = mx * (1.0f / E4M3_MAX);
  b.a = !b.finite ? __builtin_nanf("") : q == 0.0f ? 1.0f : q;
  b.f = b.a < 0x1p-92f ? 0x1p100f : 1.0f;
  b.af = b.a * b.f;
  b.r = 1.0f / b.af;
  return b;
}
// fl32(v / a) clamped to the e4m3 range, with v's sign (a zero keeps it)
__device__ inline float scaled_value(float v, const BlockScale& b) {
  const float q = quot_fast(__builtin_fabsf(v) * b.f, b.af, b.r);
  return __builtin_copysignf(b.finite ? fminf(q, E4M3_MAX) : 0.0f, b.finite ? v : 1.0f);
}
// |v|, with every non-finite value mapped to +inf so a maximum keeps it
__device__ inline float mag(float v) {
  const float x = __builtin_fabsf(v);
  return x < __builtin_huge_valf() ? x : __builtin_huge_valf();
}

__device__ inline uint32_t encode2(float lo, float hi, uint32_t old, bool upper) {
  return upper ? __builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, (int)old, true)
               : __builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, (int)old, false);
}

// Eight neighbouring elements of a row of x.
template <class X>
struct __attribute__((packed, aligned(sizeof(X)))) Eight {
  X v[8];
};

// A workgroup of 256 threads quantizes 128 x 128 elements of x, held in
// registers between the maximum and the codes: thread t has columns 8 (t % 16)
// .. + 8 of rows 8 (t / 16) .. + 8.  One read of x, one write of codes.
//   scale per row and 128 columns (ROWS):     maximum over 16 lanes
//   scale per column and 128 rows (COLUMNS):  over a thread's rows, 4 lanes, 4 waves
//   scale per tile (TILE):                    over the workgroup
// With TR the codes are written transposed, through LDS: a thread's eight codes
// of a column are neighbours there (rows of 128 + 8 bytes; 128-byte rows go
// out); else 8 bytes a row and thread.  The codes come from the hardware's
// conversion to e4m3 (nearest, ties to even).
//
// Bound by its bytes: 32,000 x 2,048 fp32 tiles 62 us (5.3 TB/s), 16,384 x 5,120
// bf16 along the columns 67 us (3.8 TB/s; 5.3 TB/s at 151,936 x 5,120), one row of
// 5,120 4.6 us.  (Holding the elements unconverted, other workgroup orders and
// nontemporal stores changed nothing or cost 5%.)
enum : int { Q_ROWS = 0, Q_COLUMNS = 1, Q_TILE = 2 };
template <class X, int MODE, bool TR>
__global__ __launch_bounds__(256) void quantize_kernel(const X* x, int64_t ld, int64_t R, int64_t C, uint8_t* codes,
                                                       int64_t ldc, float* scales) {
  constexpr int LDT = QB + 8;
  __shared__ float red[MODE == Q_COLUMNS ? 4 * QB : 4];
  __shared__ __attribute__((aligned(16))) uint8_t tile[TR ? QB * LDT : 16];
  const int tid = threadIdx.x, tc = tid & 15, tr = tid >> 4;
  // (neighbouring workgroups share rows of x)
  const int64_t cbs = (C + QB - 1) / QB;
  const int64_t rb = blockIdx.x / cbs, cb = blockIdx.x - rb * cbs;
  const int64_t c0 = cb * QB + tc * 8, r0 = rb * QB + tr * 8;
  float v[8][8];
  if (c0 + 8 <= C) {
    Eight<X> e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r0 + i < R) e[i] = *(const Eight<X>*)(x + (r0 + i) * ld + c0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = r0 + i < R ? (float)e[i].v[k] : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = r0 + i < R && c0 + k < C ? (float)x[(r0 + i) * ld + c0 + k] : 0.0f;
  }
  auto lanes = [](float m, int from, int to) {
    for (int o = from; o < to; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    return m;
  };
  BlockScale s[MODE == Q_TILE ? 1 : 8];  // of the thread's rows, columns, or the tile
  if constexpr (MODE == Q_ROWS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, mag(v[i][k]));
      s[i] = block_scale(lanes(m, 1, 16));
      if (tc == 0 && r0 + i < R) scales[cb * R + r0 + i] = s[i].a;
    }
  } else if constexpr (MODE == Q_COLUMNS) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, mag(v[i][k]));
      m = lanes(m, 16, 64);
      if ((tid & 63) < 16) red[(tid >> 6) * QB + tc * 8 + k] = m;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float m = red[tc * 8 + k];
#pragma unroll
      for (int w = 1; w < 4; ++w) m = fmaxf(m, red[w * QB + tc * 8 + k]);
      s[k] = block_scale(m);
      if (tr == 0 && c0 + k < C) scales[rb * C + c0 + k] = s[k].a;
    }
  } else {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, mag(v[i][k]));
    m = lanes(m, 1, 64);
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
    s[0] = block_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    // (scales [blocks of the reduction][tiles of the other])
    if (tid == 0) scales[TR ? rb * cbs + cb : cb * ((R + QB - 1) / QB) + rb] = s[0].a;
  }
  auto code = [&](int i, int k) __attribute__((always_inline)) {
    return scaled_value(v[i][k], s[MODE == Q_ROWS ? i : MODE == Q_COLUMNS ? k : 0]);
  };
  if constexpr (TR) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; i += 2) w[i >> 2] = encode2(code(i, k), code(i + 1, k), w[i >> 2], i & 2);
      *(u32x2*)(tile + (tc * 8 + k) * LDT + tr * 8) = u32x2{w[0], w[1]};
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ch = i * 256 + tid, c = ch >> 3, r16 = (ch & 7) * 16;
      const int64_t col = cb * QB + c, row = rb * QB + r16;
      const u32x2 lo = *(const u32x2*)(tile + c * LDT + r16), hi = *(const u32x2*)(tile + c * LDT + r16 + 8);
      if (col < C && row < (R + 15) / 16 * 16) *(u32x4*)(codes + col * ldc + row) = u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int k = 0; k < 8; k += 2) w[k >> 2] = encode2(code(i, k), code(i, k + 1), w[k >> 2], k & 2);
      if (r0 + i < R && c0 < (C + 15) / 16 * 16) *(u32x2*)(codes + (r0 + i) * ldc + c0) = u32x2{w[0], w[1]};
    }
  }
}

template <class X>
hipError_t run_quantize(const X* x, int64_t R, int64_t C, int64_t ld, int flags, uint8_t* codes, int64_t ld_codes,
                        float* scales, hipStream_t s) {
  const bool tr = flags & STCE_QUANT_TRANSPOSE, tile = flags & STCE_QUANT_TILE;
  const dim3 grid((unsigned)(ceil_div(R, QB) * ceil_div(C, QB)));
  ProfScope ps(KIND_QUANTIZE_BLOCKS, s);
  const auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, x, ld, R, C, codes, ld_codes, scales);
  };
  if (tile)
    tr ? launch(quantize_kernel<X, Q_TILE, true>) : launch(quantize_kernel<X, Q_TILE, false>);
  else
    tr ? launch(quantize_kernel<X, Q_COLUMNS, true>) : launch(quantize_kernel<X, Q_ROWS, false>);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
// 16 bytes of neighbouring outputs of one row.
template <class O>
struct __attribute__((packed, aligned(sizeof(O)))) OutPiece {
  static constexpr int E = 16 / sizeof(O);
  O v[E];
};

struct BlockOut {
  void* out;
  int64_t ldo;
  int64_t split;  // elements between the partial results of two segments (0: one segment)
  int add;
};

// One output tile per workgroup; segment g of the reduction (blocks [g per,
// (g + 1) per)) goes to its own partial output.
template <class Main, class O>
__global__ __launch_bounds__(64 * Main::W, Main::W == 4 ? 2 : 1) void block_tile_kernel(BlockOps p, BlockOut o,
                                                                                        TileMap map, int per) {
  constexpr int NI = Main::NI, NJ = Main::NJ;
  const int tiles = map.tiles_m * map.tiles_n;
  const int g = blockIdx.x / tiles;
  int tn, tm;
  map.get(blockIdx.x - g * tiles, tn, tm);
  const int n0 = tn * Main::TN, m0 = tm * Main::TM;
  const int nkb = (p.K + QB - 1) / QB;
  typename Main::Acc acc;
  Main::run(p, acc, n0, m0, g * per, min((g + 1) * per, nkb));
  // A lane holds four neighbouring outputs of NI NJ places; stored as they are,
  // they would reach memory in 32- or 64-byte pieces (0.7 TB/s at 8,192 x
  // 16,384 bf16).  Each wave turns its 16 NJ rows of 16 NI outputs round in LDS
  // of its own instead, 16 JG rows at a time, and stores whole rows, 16 bytes a
  // lane.  The 16-byte chunks of a row are XOR-permuted by the row, so neither
  // side meets a bank twice.
  constexpr int ROW = 16 * NI * sizeof(O), NC = ROW / 16, E = OutPiece<O>::E;  // chunks of a row, outputs of a chunk
  constexpr int MASK = NC < 16 ? NC - 1 : 15;
  constexpr int JG = NJ * 16 * ROW > 16384 ? NJ / 2 : NJ;
  constexpr int REGION = JG * 16 * ROW;
  constexpr int PER = Main::STAGE / REGION;  // waves' regions a stage holds
  static_assert(2 * PER >= Main::W, "the stages hold every wave's region");
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char* const lds = (w < PER ? Main::template stage<0>() : Main::template stage<1>()) + w % PER * REGION;
  O* const out = (O*)o.out + g * o.split;
  const int col = lane & 15, quad = lane >> 4;
  const int nw = n0 + w / Main::WM * 16 * NI, mw = m0 + w % Main::WM * 16 * NJ;
#pragma unroll
  for (int jg = 0; jg < NJ; jg += JG) {
#pragma unroll
    for (int j = 0; j < JG; ++j)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        struct __attribute__((aligned(4 * sizeof(O)))) Four {
          O v[4];
        } f;
#pragma unroll
        for (int r = 0; r < 4; ++r) f.v[r] = (O)acc[i][jg + j][r];
        const int at = i * 16 + quad * 4;  // of the row
        *(Four*)(lds + (j * 16 + col) * ROW + ((at / E) ^ (col & MASK)) * 16 + at % E * sizeof(O)) = f;
      }
    __builtin_amdgcn_s_waitcnt(WAIT_LGKM0);
#pragma unroll
    for (int x = 0; x < JG * 16 * NC / 64; ++x) {
      const int row = x * (64 / NC) + lane / NC, ch = lane % NC;
      const int m = mw + jg * 16 + row, n = nw + ch * E;
      OutPiece<O> v = *(const OutPiece<O>*)__builtin_assume_aligned(
          lds + row * ROW + (ch ^ (row & MASK)) * 16, 16);
      if (m >= p.M || n >= p.N) continue;
      O* const dst = out + (int64_t)m * o.ldo + n;
      if (n + E <= p.N) {
        if (o.add) {
          const OutPiece<O> old = *(const OutPiece<O>*)dst;
#pragma unroll
          for (int e = 0; e < E; ++e) v.v[e] = (O)((float)v.v[e] + (float)old.v[e]);
        }
        *(OutPiece<O>*)dst = v;
      } else {
        for (int e = 0; e < E; ++e)
          if (n + e < p.N) dst[e] = (O)(o.add ? (float)dst[e] + (float)v.v[e] : (float)v.v[e]);
      }
    }
  }
}

// out (+)= the segments' partial results [S][M][N], added in order.
template <class O>
__global__ __launch_bounds__(256) void block_sum_kernel(const float* part, int S, int64_t M, int64_t N, O* out,
                                                        int64_t ldo, int add) {
  const int64_t total = M * N;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    float v = part[e];
    for (int s = 1; s < S; ++s) v += part[s * total + e];
    O* dst = out + e / N * ldo + e % N;
    *dst = (O)(add ? (float)*dst + v : v);
  }
}

template <class O>
__global__ __launch_bounds__(256) void block_zero_kernel(int64_t M, int64_t N, O* out, int64_t ldo) {
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < M * N; e += (int64_t)gridDim.x * 256)
    out[e / N * ldo + e % N] = (O)0.0f;
}

// How a product is cut.
//   M <= 64: 128 rows of b by 64 of a, four waves (64 x 32).  Bound by b's
//     bytes, which three such workgroups a compute unit keep in flight (5.8 TB/s
//     of 151,936 x 5,120 codes for one row of a).
//   128 x 128, four waves (64 x 64): two workgroups share a compute unit and
//     cover each other's barriers.  (Waves of 128 x 32 read and convert more
//     fragments a product: 588 against 538 us for 32,000 x 2,048 x 4,096 to
//     fp32 with row scales.)
//   256 x 256, eight waves (128 x 64): 16-bit outputs with tile scales that make
//     at least as good use of the compute units, in whole waves of tiles, as
//     the 128 x 128 ones, which take 1.18 times as long for the same products
//     (8,192 x 128,256 x 4,096: 3.90 against 4.61 ms; 2,048 x 4,096 x 4,096,
//     an eighth of a wave: 57 against 39 us).
// Segments of the reduction fill the chip when there are few output tiles.
struct BlockPlan {
  int shape;  // 0: 128 x 64, 1: 128 x 128, 2: 256 x 256
  int64_t tiles_n, tiles_m;
  int S, per;  // segments, blocks per segment
};

BlockPlan plan_product(const stce_block_matmul& p) {
  BlockPlan b{};
  const int64_t nkb = ceil_div(p.K, QB);
  const int64_t small = ceil_div(p.N, 128) * ceil_div(p.M, 128), large = ceil_div(p.N, 256) * ceil_div(p.M, 256);
  b.shape = p.M <= 64 ? 0 : 1;
  if (p.M > 64 && p.out_dtype != STCE_DT_F32 && p.b_rows == QB &&
      200 * ceil_div(large, 256) <= 118 * ceil_div(small, 512))
    b.shape = 2;
  b.tiles_n = ceil_div(p.N, b.shape == 2 ? 256 : 128);
  b.tiles_m = ceil_div(p.M, 64 << b.shape);
  const int64_t wgs = b.tiles_n * b.tiles_m;
  int64_t S = 256 / wgs;  // (compute units; at least four blocks a segment)
  if (S > ceil_div(nkb, 4)) S = ceil_div(nkb, 4);
  if (S < 1) S = 1;
  b.per = (int)ceil_div(nkb, S);
  b.S = nkb ? (int)ceil_div(nkb, b.per) : 1;
  return b;
}

template <class Main, class O>
void launch_tiles(const BlockPlan& b, const BlockOps& p, const BlockOut& o, hipStream_t s) {
  const TileMap map{(int)b.tiles_n, (int)b.tiles_m, 8};
  hipLaunchKernelGGL((block_tile_kernel<Main, O>), dim3((unsigned)(b.tiles_n * b.tiles_m * b.S)), dim3(64 * Main::W),
                     0, s, p, o, map, b.per);
}

// A 16-bit output is rounded far above what the fp8 matrix instructions drop
// (they align the eight products of a group of consecutive k to the largest
// and keep 13 binary places below it: 1.5e-5 of a 128-term sum of normal
// values); an fp32 output takes the fp16 ones on converted codes, exact
// products summed to 9e-9, at half the rate.
template <bool ROWB, class O, class F>
void launch_product(const BlockPlan& b, const BlockOps& p, const BlockOut& o, hipStream_t s) {
  constexpr bool EXACT = std::is_same<F, FragF16>::value;
  if constexpr (!ROWB && !EXACT)
    if (b.shape == 2) return launch_tiles<BlockMain<8, 4, 2, 4, ROWB, F>, O>(b, p, o, s);
  if (b.shape == 0)
    launch_tiles<BlockMain<4, 2, 2, 2, ROWB, F>, O>(b, p, o, s);
  else
    launch_tiles<BlockMain<4, 4, 2, 2, ROWB, F>, O>(b, p, o, s);
}

unsigned sweep_blocks(int64_t n) { return (unsigned)(ceil_div(n, 256) < 8192 ? ceil_div(n, 256) : 8192); }

template <class O>
hipError_t run_matmul(const stce_block_matmul& p, void* ws, hipStream_t s) {
  using F = typename std::conditional<sizeof(O) == 4, FragF16, FragFp8>::type;
  ProfScope ps(KIND_BLOCK_MATMUL, s);
  if (p.K == 0) {
    if (!p.accumulate)
      hipLaunchKernelGGL(block_zero_kernel<O>, dim3(sweep_blocks(p.M * p.N)), dim3(256), 0, s, p.M, p.N, (O*)p.out,
                         p.ldo);
    return hipGetLastError();
  }
  const BlockPlan b = plan_product(p);
  const BlockOps ops{p.a,           p.b,           p.a_scale,          p.b_scale,          p.lda,    p.ldb,
                     p.a_block_stride, p.b_block_stride, (int)p.a_row_stride, (int)p.b_row_stride, (int)p.M, (int)p.N,
                     (int)p.K};
  const bool rowb = p.b_rows == 1;
  if (b.S == 1) {
    const BlockOut o{p.out, p.ldo, 0, p.accumulate};
    if (rowb)
      launch_product<true, O, F>(b, ops, o, s);
    else
      launch_product<false, O, F>(b, ops, o, s);
    return hipGetLastError();
  }
  const BlockOut o{ws, p.N, p.M * p.N, 0};
  if (rowb)
    launch_product<true, float, F>(b, ops, o, s);
  else
    launch_product<false, float, F>(b, ops, o, s);
  const hipError_t e = hipGetLastError();
  if (e) return e;
  hipLaunchKernelGGL(block_sum_kernel<O>, dim3(sweep_blocks(p.M * p.N)), dim3(256), 0, s, (const float*)ws, b.S, p.M,
                     p.N, (O*)p.out, p.ldo, p.accumulate);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_blocks(const void* x, int dtype, int64_t R, int64_t C, int64_t ld, int flags,
                                  uint8_t* codes, int64_t ld_codes, float* scales, hipStream_t s) {
  switch (dtype) {
    case STCE_DT_BF16: return run_quantize((const bf16*)x, R, C, ld, flags, codes, ld_codes, scales, s);
    case STCE_DT_F16: return run_quantize((const _Float16*)x, R, C, ld, flags, codes, ld_codes, scales, s);
    default: return run_quantize((const float*)x, R, C, ld, flags, codes, ld_codes, scales, s);
  }
}

size_t block_matmul_workspace_bytes(const stce_block_matmul& p) {
  if (p.K == 0) return 0;
  const BlockPlan b = plan_product(p);
  return b.S > 1 ? sizeof(float) * (size_t)b.S * (size_t)p.M * (size_t)p.N : 0;
}

hipError_t launch_block_matmul(const stce_block_matmul& p, void* ws, hipStream_t s) {
  switch (p.out_dtype) {
    case STCE_DT_BF16: return run_matmul<bf16>(p, ws, s);
    case STCE_DT_F16: return run_matmul<_Float16>(p, ws, s);
    default: return run_matmul<float>(p, ws, s);
  }
}

}  // namespace stce
