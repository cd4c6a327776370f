// e4m3 quantization with a scale per block of 128, and the product of two
// such matrices.
#include "epilogues.hpp"
#include "gemm.hpp"
#include "ops.hpp"

namespace stce {
namespace {

constexpr int QB = 128;  // values per scale along the reduction

// fl32(v / a), clamped to the e4m3 range: the correction step of quot_fast
// where it is exact, the IEEE division elsewhere (the same bits).
__device__ inline float scaled_value(float v, float a, float r, bool a_ok) {
  const float x = __builtin_fabsf(v);
  const float q = (a_ok && x >= 0x1p-90f && x <= 0x1p+90f) ? quot_fast(v, a, r) : v / a;
  return fminf(fmaxf(q, -E4M3_MAX), E4M3_MAX);
}

struct BlockScale {
  float a, r;
  bool ok, finite;
};
// From the block's largest magnitude (NaN or infinite when the block holds a
// NaN or an infinity).
__device__ inline BlockScale block_scale(float mx) {
  BlockScale b;
  b.finite = mx < __builtin_huge_valf();
  const float q = mx / E4M3_MAX;
  b.a = !b.finite ? __builtin_nanf("") : q == 0.0f ? 1.0f : q;
  b.r = 1.0f / b.a;
  b.ok = b.a >= 0x1p-30f && b.a <= 0x1p+30f;
  return b;
}
// |v|, with every non-finite value mapped to +inf so a maximum keeps it
__device__ inline float mag(float v) {
  const float x = __builtin_fabsf(v);
  return x < __builtin_huge_valf() ? x : __builtin_huge_valf();
}

// One workgroup per block (128 columns of one row of Y, or a 128 x 128 tile):
// element (q, l) of Y is x[q * sq + l * sl].
template <class X, bool TILE>
__global__ __launch_bounds__(128) void quantize_simple_kernel(const X* x, int64_t sq, int64_t sl, int64_t Q, int64_t L,
                                                              uint8_t* codes, int64_t ld, float* scales) {
  __shared__ float red[2];
  const int64_t qb = blockIdx.x, lb = blockIdx.y;
  const int64_t q0 = TILE ? qb * QB : qb, q1 = TILE ? (q0 + QB < Q ? q0 + QB : Q) : q0 + 1;
  const int64_t l = lb * QB + threadIdx.x;
  float mx = 0.0f;
  if (l < L)
    for (int64_t q = q0; q < q1; ++q) mx = fmaxf(mx, mag((float)x[q * sq + l * sl]));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
  __syncthreads();
  const BlockScale b = block_scale(fmaxf(red[0], red[1]));
  if (threadIdx.x == 0) scales[lb * (TILE ? ceil_div(Q, QB) : Q) + qb] = b.a;
  if (l < round_up(L, 16))
    for (int64_t q = q0; q < q1; ++q) {
      uint32_t c = 0;
      if (l < L && b.finite) c = e4m3_encode(scaled_value((float)x[q * sq + l * sl], b.a, b.r, b.ok));
      codes[q * ld + l] = (uint8_t)c;
    }
}

template <class X>
hipError_t run_quantize(const X* x, int64_t R, int64_t C, int64_t ld, int flags, uint8_t* codes, int64_t ld_codes,
                        float* scales, hipStream_t s) {
  const bool tr = flags & STCE_QUANT_TRANSPOSE, tile = flags & STCE_QUANT_TILE;
  const int64_t Q = tr ? C : R, L = tr ? R : C, sq = tr ? 1 : ld, sl = tr ? ld : 1;
  const dim3 grid((unsigned)(tile ? ceil_div(Q, QB) : Q), (unsigned)ceil_div(L, QB));
  ProfScope ps(KIND_QUANTIZE_BLOCKS, s);
  if (tile)
    hipLaunchKernelGGL((quantize_simple_kernel<X, true>), grid, dim3(128), 0, s, x, sq, sl, Q, L, codes, ld_codes,
                       scales);
  else
    hipLaunchKernelGGL((quantize_simple_kernel<X, false>), grid, dim3(128), 0, s, x, sq, sl, Q, L, codes, ld_codes,
                       scales);
  return hipGetLastError();
}

template <class O>
__device__ inline O to_out(float v) {
  return (O)v;
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Eight e4m3 codes as fp16 (exact: e4m3's smallest value 2^-9 is normal there).
__device__ inline f16x8 codes_f16(u32x2 c) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, false));
    r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, true));
  }
  return __builtin_bit_cast(f16x8, r);
}

// One wave per 16 x 16 block of the output, operands straight from memory.
// The fp8 matrix instructions align the eight products of each group of
// consecutive k to the largest and drop what lies more than 13 binary places
// below it (measured: 1.5e-5 of a 128-term sum of normal values, relative);
// the fp16 ones sum the same products, exact after the conversion, to 9e-9.
template <class O>
__global__ __launch_bounds__(64) void block_matmul_simple_kernel(stce_block_matmul p) {
  const int lane = threadIdx.x, row = lane & 15, quad = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 16, n0 = (int64_t)blockIdx.x * 16;
  const int64_t m = m0 + row, n = n0 + row;
  const int64_t mr = m < p.M ? m : p.M - 1, nr = n < p.N ? n : p.N - 1;
  const uint8_t* a = p.a + mr * p.lda;
  const uint8_t* b = p.b + nr * p.ldb;
  f32x4 sum{};
  for (int64_t k0 = 0, kb = 0; k0 < p.K; k0 += QB, ++kb) {
    u32x4 va[2] = {}, vb[2] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t k = k0 + quad * 32 + h * 16;
      if (k < p.K) {
        va[h] = *(const u32x4*)(a + k);
        vb[h] = *(const u32x4*)(b + k);
      }
    }
    f32x4 part{};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        part = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(u32x2{vb[h][2 * e], vb[h][2 * e + 1]}),
                                                      codes_f16(u32x2{va[h][2 * e], va[h][2 * e + 1]}), part, 0, 0, 0);
    const float sa = p.a_scale[mr * p.a_row_stride + kb * p.a_block_stride];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      int64_t nn = n0 + quad * 4 + r;
      nn = nn < p.N ? nn : p.N - 1;
      const float sb = p.b_scale[(p.b_rows == QB ? nn / QB : nn) * p.b_row_stride + kb * p.b_block_stride];
      sum[r] = __builtin_fmaf(part[r], sa * sb, sum[r]);
    }
  }
  if (m >= p.M) return;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t nn = n0 + quad * 4 + r;
    if (nn >= p.N) continue;
    O* o = (O*)p.out + m * p.ldo + nn;
    *o = to_out<O>(p.accumulate ? (float)*o + sum[r] : sum[r]);
  }
}

template <class O>
hipError_t run_matmul(const stce_block_matmul& p, hipStream_t s) {
  ProfScope ps(KIND_BLOCK_MATMUL, s);
  hipLaunchKernelGGL(block_matmul_simple_kernel<O>, dim3((unsigned)ceil_div(p.N, 16), (unsigned)ceil_div(p.M, 16)),
                     dim3(64), 0, s, p);
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

size_t block_matmul_workspace_bytes(const stce_block_matmul&) { return 0; }

hipError_t launch_block_matmul(const stce_block_matmul& p, void*, hipStream_t s) {
  switch (p.out_dtype) {
    case STCE_DT_BF16: return run_matmul<bf16>(p, s);
    case STCE_DT_F16: return run_matmul<_Float16>(p, s);
    default: return run_matmul<float>(p, s);
  }
}

}  // namespace stce
