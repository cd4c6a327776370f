// Block-tiled product of e4m3 matrices with a scale for each block of 128 of
// the reduction (gfx950): out[m, n] = sum_b sa[m, b] sb[n, b] P_b[m, n], P_b the
// sum over the 128 k of block b.
//
// A workgroup's waves lie WN (n) x WM (m), each forming 16 NI rows n of b by
// 16 NJ rows m of a as NI x NJ blocks of 16 x 16, with b as the first matrix
// operand: a lane then holds one row m and
// four consecutive n, so a per-tile scale of b is one value per wave, and an
// output store four neighbours.  A k-tile is one scale block, 128 bytes of a
// row; the loads, the LDS layout and its swizzle are those of the fp8 loop in
// gemm.hpp, plus the scales (one dword per row).
//
// A matrix instruction of k-tile t starts from zero; its four results are
// scaled into the running fp32 sums by ordinary fma, one row of blocks behind
// the matrix instructions so that both pipes run at once: 32 cycles of matrix
// pipe against 16 of fma per 16 x 16 x 128.  (Row scales of b take a multiply
// more.)
#pragma once

#include "gemm.hpp"

namespace stce {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Eight e4m3 codes as fp16 (exact: e4m3's smallest value 2^-9 is normal there).
__device__ inline f16x8 codes_f16(uint32_t c0, uint32_t c1) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c0, 1.0f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c0, 1.0f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c1, 1.0f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c1, 1.0f, true));
  return __builtin_bit_cast(f16x8, r);
}

// A fragment of 32 codes a lane as a matrix operand: as it lies (fp8
// instructions) or converted (fp16 instructions, four groups of eight codes).
typedef i32x8 Raw;
struct FragFp8 {
  Raw v;
  __device__ inline FragFp8() {}
  __device__ inline explicit FragFp8(const Raw& r) : v(r) {}
};
struct FragF16 {
  f16x8 v[4];
  __device__ inline FragF16() {}
  __device__ inline explicit FragF16(const Raw& r) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = codes_f16((uint32_t)r[2 * e], (uint32_t)r[2 * e + 1]);
  }
};
__device__ inline Raw raw_frag(u32x4 lo, u32x4 hi) {
  return __builtin_bit_cast(Raw, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ inline f32x4 block_mfma(const FragFp8& a, const FragFp8& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4{}, 0, 0, 0, 0, 0, 0);
}
__device__ inline f32x4 block_mfma(const FragF16& a, const FragF16& b) {
  f32x4 p{};
#pragma unroll
  for (int e = 0; e < 4; ++e) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[e], b.v[e], p, 0, 0, 0);
  return p;
}

// s_waitcnt of the LDS counter alone (vmcnt at its largest)
constexpr int WAIT_LGKM0 = 0xc07f;

// Operands of the product.
struct BlockOps {
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  int64_t lda, ldb;
  int64_t sa_blk, sb_blk;  // stride of a scale's block index
  int sa_row, sb_row;      // stride of its row index, < 2^21
  int M, N, K;
};

// ROWB: one scale per row of b (else per 128).  F: the fragment type, FragFp8 or
// FragF16.
template <int NI_, int NJ_, int WN_, int WM_, bool ROWB_, class F_>
struct BlockMain {
  static constexpr int NI = NI_, NJ = NJ_, WN = WN_, WM = WM_, W = WN * WM;
  static constexpr bool ROWB = ROWB_;
  typedef F_ F;
  static constexpr int TN = 16 * NI * WN, TM = 16 * NJ * WM;  // rows of b, of a per workgroup
  static_assert(TN == 32 * W && TM <= TN, "half the waves load the scales of TN rows of an operand, 64 each");
  static_assert(NI % 4 == 0 && (ROWB || 128 % (16 * NI) == 0), "a wave's rows of b lie in one tile");
  static constexpr int LB = TN / 8 / W, LA = TM / 8 / W;  // 1 KB loads per wave, operand and k-tile
  static constexpr int BYTES_B = TN * 128, BYTES_A = TM * 128;
  static constexpr int STAGE = BYTES_B + BYTES_A + 8 * TN;  // + TN scales each of b and of a
  static constexpr int OFF_A = BYTES_B, OFF_SB = BYTES_B + BYTES_A, OFF_SA = OFF_SB + 4 * TN;
  typedef f32x4 Acc[NI][NJ];

  // each stage an object of its own: the compiler then knows that the loads in
  // flight into one do not touch the others
  template <int I>
  __device__ static char* stage() {
    __shared__ __attribute__((aligned(16))) char s[STAGE];
    return s;
  }

  // k-tiles kt0 .. kt1 (kt0 < kt1) of the output tile at (n0, m0)
  __device__ static inline void run(const BlockOps& p, Acc& acc, int n0, int m0, int kt0, int kt1) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wb = w / WM, wa = w % WM;
    const int rowsB = min(p.N - n0, TN), rowsA = min(p.M - m0, TM);
    const int lda = (int)p.lda, ldb = (int)p.ldb;
    const __amdgpu_buffer_rsrc_t rb =
        __builtin_amdgcn_make_buffer_rsrc((void*)(p.b + (int64_t)n0 * ldb), (short)0, rowsB * ldb, RSRC_WORD3);
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + (int64_t)m0 * lda), (short)0, rowsA * lda, RSRC_WORD3);
    // load i of wave w fills tile rows (w L + i) 8 .. + 8: lane l row + l / 8,
    // physical chunk l % 8 (logical chunk: that xor the row's swizzle)
    const int lrow = lane >> 3, lpc = lane & 7;
    const int ce = lpc ^ lds_swz(lrow), co = lpc ^ lds_swz(lrow + 8);
    const int rB = (w * LB * 8 + lrow) * ldb, rA = (w * LA * 8 + lrow) * lda;
    // scales: the first half of the waves loads 64 rows each of b's, the others of a's
    const bool isb = w < W / 2;
    const int sw0 = w % (W / 2) * 64, srow = sw0 + lane;
    const int nbase = ROWB ? n0 : n0 >> 7;
    const int soff = isb ? ((ROWB ? min(n0 + srow, p.N - 1) : min(n0 + srow, p.N - 1) >> 7) - nbase) * p.sb_row * 4
                         : min(srow, rowsA - 1) * p.sa_row * 4;
    const float* const sbase = isb ? p.sb + (int64_t)nbase * p.sb_row : p.sa + (int64_t)m0 * p.sa_row;
    const int64_t sblk = isb ? p.sb_blk : p.sa_blk;
    const int lds_s = (isb ? OFF_SB : OFF_SA) + sw0 * 4;
    // load x of a k-tile: LB of b, LA of a, the scales
    constexpr int LOADS = LB + LA + 1;
    auto issue = [&](auto sg_c, int kt, int x) __attribute__((always_inline)) {
      char* const st = stage<decltype(sg_c)::value>();
      const int k0 = kt * 128;
      const int kend = min(p.K, kt1 * 128);
      // (the row step is formed anew for every load, or the lane offsets of all
      // of them would stay in registers)
      if (x < LB + LA) {
        const bool ofb = x < LB;
        const int i = ofb ? x : x - LB, L = ofb ? LB : LA;
        const bool odd = (w * L + i) & 1;  // (the swizzle takes row bits 1 .. 3, bit 3 this parity)
        const int ch = odd ? co : ce;
        int step = 8 * (ofb ? ldb : lda);
        asm volatile("" : "+s"(step));
        const int off = k0 + ch * 16 < kend ? (ofb ? rB : rA) + ch * 16 + i * step : 0x7ffffff0;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ofb ? rb : ra, STCE_LDS(st + (ofb ? 0 : OFF_A) + (w * L + i) * 1024), 16,
                                                 off, k0, 0, 0);
      } else {
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(sbase + (int64_t)min(kt, kt1 - 1) * sblk), (short)0, 0x7fffffff, RSRC_WORD3);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, STCE_LDS(st + lds_s), 4, soff, 0, 0, 0);
      }
    };
    auto issue_all = [&](auto sg_c, int kt) __attribute__((always_inline)) {
#pragma unroll
      for (int x = 0; x < LOADS; ++x) issue(sg_c, kt, x);
    };
    const int frow = lane & 15, fq = lane >> 4, sw = lds_swz(frow);
    const int offB = (wb * 16 * NI + frow) * 128, offA = OFF_A + (wa * 16 * NJ + frow) * 128;
    const int c0 = ((2 * fq) ^ sw) * 16, c1 = ((2 * fq + 1) ^ sw) * 16;
    auto frag = [&](const char* base) __attribute__((always_inline)) {
      return raw_frag(*(const u32x4*)(base + c0), *(const u32x4*)(base + c1));
    };
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{};
    // Fragments: a's NJ of a tile, reloaded for the next one behind their last
    // use; b's NI through a ring of four, read AHEAD blocks ahead (with, for
    // row scales, the lane's four scales of b).  The results of the matrix
    // instructions wait in a ring too and are scaled in LAG instructions later,
    // across the tile's end, with that tile's scales (s by stage).
    constexpr int LAG = 3, NM = NI * NJ, AHEAD = NJ == 4 ? 2 : 3;
    Raw fa[NJ], fb[4];
    // Row scales of b wait as long as the results they scale: block i's may be
    // read anew (AHEAD blocks ahead) only when the last result of its previous
    // tile is in, LAG instructions after that; where it comes too early, the two
    // tiles' scales take slots by parity.
    constexpr int SLOTS = (NI - AHEAD) * NJ >= NJ + LAG ? NI : 2 * NI;
    f32x4 sbv[SLOTS];
    f32x4 part[4];
    float s[2][NJ];
#pragma unroll
    for (int x = 0; x < 4; ++x) part[x] = f32x4{};
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[0][j] = s[1][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) sbv[i] = f32x4{};
    auto scale_in = [&](int idx, int sg) __attribute__((always_inline)) {  // idx: instruction of the tile of stage sg
      const int i = idx / NJ, j = idx % NJ;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = ROWB ? part[idx & 3][r] * sbv[(SLOTS > NI ? sg * NI : 0) + i][r] : part[idx & 3][r];
        acc[i][j][r] = __builtin_fmaf(v, s[sg][j], acc[i][j][r]);
      }
      // holds the sums here: left free, the compiler collects all of a tile's
      // products before it adds them, and runs out of registers
      asm volatile("" : "+v"(acc[i][j]));
    };
    auto read_b = [&](const char* st, int sg, int i, bool live) __attribute__((always_inline)) {
      fb[i & 3] = frag(st + offB + i * 16 * 128);
      if constexpr (ROWB) {
        f32x4 v = *(const f32x4*)(st + OFF_SB + (wb * 16 * NI + i * 16 + fq * 4) * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = live ? v[r] : 0.0f;
        sbv[(SLOTS > NI ? sg * NI : 0) + i] = v;
      }
    };
    // scales of a tile: read as they lie once it has landed, multiplied when it starts
    float rsa[NJ], rsb = 1.0f;
    auto read_scales = [&](const char* st) __attribute__((always_inline)) {
      const float* sa = (const float*)(st + OFF_SA) + wa * 16 * NJ + frow;
#pragma unroll
      for (int j = 0; j < NJ; ++j) rsa[j] = sa[j * 16];
      if constexpr (!ROWB) rsb = *((const float*)(st + OFF_SB) + wb * 16 * NI);
    };
    auto set_scales = [&](int sg, bool live) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float v = ROWB ? rsa[j] : rsa[j] * rsb;
        s[sg][j] = live ? v : 0.0f;
      }
    };
    auto tile = [&](auto sg_c, int kt) __attribute__((always_inline)) {
      constexpr int sg = decltype(sg_c)::value;
      const char* const st = stage<sg>();
      const char* const nx = stage<1 - sg>();
      F cb;
#pragma unroll
      for (int idx = 0; idx < NM; ++idx) {
        const int i = idx / NJ, j = idx % NJ;
        if (j == 0) {
          if (i == NI - AHEAD) {
            // every wave has read all of this stage, and the next tile has landed
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(WAIT_VM0_LGKM0);
            __syncthreads();
            __builtin_amdgcn_sched_barrier(0);
          }
          if (i + AHEAD < NI)
            read_b(st, sg, i + AHEAD, kt < kt1);
          else
            read_b(nx, 1 - sg, i + AHEAD - NI, kt + 1 < kt1);
          cb = F(fb[i & 3]);
        }
        // (of the tile before: its instruction NM + idx - LAG)
        if (idx < LAG) scale_in(NM + idx - LAG, 1 - sg);
        part[idx & 3] = block_mfma(cb, F(fa[j]));
        if (idx >= LAG) scale_in(idx - LAG, sg);
        if (idx == 0) set_scales(sg, kt < kt1);
        // behind the barrier: the loads of the tile after the next one into the
        // stage just freed, a few behind every matrix instruction
        constexpr int FIRST = (NI - AHEAD) * NJ, PER = (LOADS + NM - FIRST - 1) / (NM - FIRST);
#pragma unroll
        for (int x = 0; x < PER; ++x)
          if (idx >= FIRST && (idx - FIRST) * PER + x < LOADS) issue(sg_c, kt + 2, (idx - FIRST) * PER + x);
        if (idx == FIRST) read_scales(nx);
        if (i == NI - 1) fa[j] = frag(nx + offA + j * 16 * 128);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // Tiles run in pairs, so that stages and slots are constants; an odd count
    // gets one more tile of zeros (its loads fall past the end, its scales are
    // zero).
    constexpr std::integral_constant<int, 0> S0{};
    constexpr std::integral_constant<int, 1> S1{};
    issue_all(S0, kt0);
    issue_all(S1, kt0 + 1);
    __builtin_amdgcn_s_waitcnt(WAIT_VM0_LGKM0);
    __syncthreads();
    read_scales(stage<0>());
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) read_b(stage<0>(), 0, i, true);
#pragma unroll
    for (int j = 0; j < NJ; ++j) fa[j] = frag(stage<0>() + offA + j * 16 * 128);
    for (int kt = kt0; kt < kt1; kt += 2) {
      tile(S0, kt);
      tile(S1, kt + 1);
    }
#pragma unroll
    for (int idx = NM - LAG; idx < NM; ++idx) scale_in(idx, 1);
    // the stages are free: no load of any wave is on its way, no read left
    __builtin_amdgcn_s_waitcnt(WAIT_VM0_LGKM0);
    __syncthreads();
  }
};

}  // namespace stce
