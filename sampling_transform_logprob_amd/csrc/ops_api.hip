// Host side of the C ABI's operators on given arrays (include/stce.h): token
// log probabilities and their gradient, block-scaled fp8 quantization and
// product.  Argument checks, then the launchers of ops.hpp.
#include "api_internal.hpp"
#include "ops.hpp"

using namespace stce;

namespace {

// workgroups of a launch: 256 threads each, fewer than 2^32 in all
constexpr int64_t MAX_WORKGROUPS = (1 << 24) - 1;

bool is_aligned(const void* ptr, size_t a) { return ((uintptr_t)ptr % a) == 0; }

// bytes of an element of a logits / quantizer / output dtype; 0: none
size_t value_size(int32_t dtype) {
  switch (dtype) {
    case STCE_DT_BF16:
    case STCE_DT_F16: return 2;
    case STCE_DT_F32: return 4;
  }
  return 0;
}

stce_status bad_dtype(const char* what, int32_t dtype) {
  return fail(STCE_E_UNSUPPORTED,
              "unsupported %s dtype %d: expected bf16 (STCE_DT_BF16), fp16 (STCE_DT_F16) or fp32 (STCE_DT_F32)", what,
              (int)dtype);
}

// An array of `rows` rows of `cols` elements with a row stride of `ld`: its
// extent in bytes; rows past 2^31 and extents past 2^62 are refused.
bool extent_ok(int64_t rows, int64_t ld, size_t es) {
  return rows <= 1 || ld <= ((int64_t)1 << 61) / ((rows - 1) * (int64_t)es);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na && nb && x < y + nb && y < x + na;
}

size_t bytes_of(int64_t rows, int64_t cols, int64_t ld, size_t es) {
  return rows > 0 ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * es : 0;
}

stce_status check_ws(const void* ws, size_t have, size_t need) {
  if (need && !ws) return fail(STCE_E_WORKSPACE, "workspace is NULL (needs %zu bytes)", need);
  if (have < need) return fail(STCE_E_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", have, need);
  if (need && !is_aligned(ws, 256)) return fail(STCE_E_ARG, "workspace must be 256-byte aligned");
  return STCE_OK;
}

stce_status check_token_shapes(const stce_token_problem* p) {
  if (!p) return fail(STCE_E_ARG, "problem is NULL");
  if (p->flags & ~STCE_PROBLEM_IGNORE_INDEX)
    return fail(STCE_E_ARG, "problem.flags=%d: only STCE_PROBLEM_IGNORE_INDEX is known here", (int)p->flags);
  const size_t es = value_size(p->dtype);
  if (!es) return bad_dtype("logits", p->dtype);
  // (a workgroup per row where there are many)
  if (p->T < 0 || p->T > MAX_WORKGROUPS) return fail(STCE_E_ARG, "T=%lld out of range [0, 2^24)", (long long)p->T);
  if (p->V < 1 || p->V > INT32_MAX - 512)
    return fail(STCE_E_ARG, "V=%lld out of range [1, 2^31-513]", (long long)p->V);
  if (p->ld < p->V || !extent_ok(p->T, p->ld, es))
    return fail(STCE_E_ARG, "ld=%lld must be at least V=%lld", (long long)p->ld, (long long)p->V);
  if (p->K < 0 || p->K > TOKENS_MAX)
    return fail(STCE_E_ARG, "K=%d given tokens per row out of range [0, %d]", (int)p->K, TOKENS_MAX);
  if (p->top_n < 0 || p->top_n > TOP_MAX)
    return fail(STCE_E_ARG, "top_n=%d alternatives per row out of range [0, %d]", (int)p->top_n, TOP_MAX);
  if ((p->flags & STCE_PROBLEM_IGNORE_INDEX) && p->ignore_index >= 0 && p->ignore_index < p->V)
    return fail(STCE_E_ARG, "ignore_index=%lld is a token id of [0, V)", (long long)p->ignore_index);
  return STCE_OK;
}

stce_status check_token_inputs(const stce_token_problem* p) {
  if (!p->logits || (p->K > 0 && !p->tokens)) return fail(STCE_E_ARG, "logits and (with K > 0) tokens are required");
  if (!is_aligned(p->logits, value_size(p->dtype)) || !is_aligned(p->tokens, 8) || !is_aligned(p->temperature, 4))
    return fail(STCE_E_ARG, "arrays must be aligned to their elements");
  return STCE_OK;
}

stce_status check_matmul_shapes(const stce_block_matmul* p) {
  if (!p) return fail(STCE_E_ARG, "problem is NULL");
  const size_t es = value_size(p->out_dtype);
  if (!es) return bad_dtype("output", p->out_dtype);
  if (p->M < 0 || p->N < 0 || p->K < 0 || p->M > INT32_MAX - 512 || p->N > INT32_MAX - 512 || p->K > (1 << 22))
    return fail(STCE_E_ARG, "M=%lld, N=%lld out of range [0, 2^31-513] or K=%lld out of range [0, 2^22]",
                (long long)p->M, (long long)p->N, (long long)p->K);
  if (p->K % 16 != 0 || p->lda % 16 != 0 || p->ldb % 16 != 0)
    return fail(STCE_E_ARG, "K=%lld, lda=%lld and ldb=%lld must be multiples of 16", (long long)p->K,
                (long long)p->lda, (long long)p->ldb);
  // (a tile's rows are addressed with 32-bit byte offsets)
  if (p->lda < p->K || p->ldb < p->K || p->lda > (1 << 22) || p->ldb > (1 << 22))
    return fail(STCE_E_ARG, "lda=%lld and ldb=%lld must be at least K=%lld and at most 2^22", (long long)p->lda,
                (long long)p->ldb, (long long)p->K);
  if (p->ldo < p->N || !extent_ok(p->M, p->ldo, es))
    return fail(STCE_E_ARG, "ldo=%lld must be at least N=%lld", (long long)p->ldo, (long long)p->N);
  if (p->b_rows != 1 && p->b_rows != 128)
    return fail(STCE_E_ARG, "b_rows=%d: one scale per 1 or 128 rows of b", (int)p->b_rows);
  if (p->a_row_stride < 0 || p->a_block_stride < 0 || p->b_row_stride < 0 || p->b_block_stride < 0)
    return fail(STCE_E_ARG, "scale strides must be >= 0");
  // (the rows of a tile's scales are addressed with 32-bit byte offsets)
  if (p->a_row_stride > (1 << 20) || p->b_row_stride > (1 << 20))
    return fail(STCE_E_UNSUPPORTED, "scale row strides must be at most 2^20 elements");
  // (at least 128 x 128 outputs a workgroup, or all of up to 64 rows)
  if (ceil_div(p->M, 128) * ceil_div(p->N, 128) > MAX_WORKGROUPS)
    return fail(STCE_E_UNSUPPORTED, "M=%lld x N=%lld has too many output tiles", (long long)p->M, (long long)p->N);
  if (p->accumulate && p->out_dtype != STCE_DT_F32)
    return fail(STCE_E_UNSUPPORTED, "accumulate takes an fp32 output");
  return STCE_OK;
}

}  // namespace

extern "C" {

stce_status stce_token_workspace_bytes(const stce_token_problem* p, size_t* bytes) {
  const stce_status s = check_token_shapes(p);
  if (s) return s;
  if (!bytes) return fail(STCE_E_ARG, "bytes is NULL");
  *bytes = p->T ? token_workspace_bytes(*p) : 0;
  return STCE_OK;
}

stce_status stce_token_logprobs(const stce_token_problem* p, const stce_token_outputs* o, int64_t* dev_status,
                                void* ws, size_t ws_bytes, void* stream) {
  stce_status s = check_token_shapes(p);
  if (s) return s;
  if (!o) return fail(STCE_E_ARG, "outputs are NULL");
  if (!is_aligned(dev_status, 8)) return fail(STCE_E_ARG, "dev_status must be 8-byte aligned");
  if (p->T == 0) {
    const hipError_t e =
        dev_status ? launch_fill_i64(dev_status, STCE_STATUS_NONE, (hipStream_t)stream) : hipSuccess;
    return e ? hip_fail(e, "status fill") : STCE_OK;
  }
  if ((s = check_token_inputs(p))) return s;
  if (!is_aligned(o->logprob, 4) || !is_aligned(o->lse, 4) || !is_aligned(o->entropy, 4) ||
      !is_aligned(o->top_logprob, 4) || !is_aligned(o->top_id, 8) || !is_aligned(o->stats, 16))
    return fail(STCE_E_ARG, "outputs must be aligned to their elements (stats to 16 bytes)");
  if ((s = check_ws(ws, ws_bytes, token_workspace_bytes(*p)))) return s;
  const hipError_t e = launch_token_logprobs(*p, *o, dev_status, ws, (hipStream_t)stream);
  return e ? hip_fail(e, "token logprobs") : STCE_OK;
}

stce_status stce_token_logprobs_backward(const stce_token_problem* p, const float* stats, const float* grad_logprob,
                                         const float* grad_entropy, const float* grad_lse, void* grad_logits,
                                         int64_t ld_grad, void* stream) {
  stce_status s = check_token_shapes(p);
  if (s) return s;
  const size_t es = value_size(p->dtype);
  if (ld_grad < p->V || !extent_ok(p->T, ld_grad, es))
    return fail(STCE_E_ARG, "ld_grad=%lld must be at least V=%lld", (long long)ld_grad, (long long)p->V);
  if (p->T == 0) return STCE_OK;
  if ((s = check_token_inputs(p))) return s;
  if (!stats || !grad_logits) return fail(STCE_E_ARG, "stats and grad_logits are required");
  if (!is_aligned(stats, 16) || !is_aligned(grad_logits, es) || !is_aligned(grad_logprob, 4) ||
      !is_aligned(grad_entropy, 4) || !is_aligned(grad_lse, 4))
    return fail(STCE_E_ARG, "arrays must be aligned to their elements (stats to 16 bytes)");
  if (overlap(p->logits, bytes_of(p->T, p->V, p->ld, es), grad_logits, bytes_of(p->T, p->V, ld_grad, es)))
    return fail(STCE_E_ARG, "grad_logits overlaps the logits");
  const hipError_t e = launch_token_grad(*p, (const TokenStats*)stats, grad_logprob, grad_entropy, grad_lse,
                                         grad_logits, ld_grad, (hipStream_t)stream);
  return e ? hip_fail(e, "token logprobs gradient") : STCE_OK;
}

stce_status stce_fp8_quantize_blocks(const void* x, int32_t dtype, int64_t R, int64_t C, int64_t ld, int32_t flags,
                                     uint8_t* codes, int64_t ld_codes, float* scales, void* stream) {
  const size_t es = value_size(dtype);
  if (!es) return bad_dtype("input", dtype);
  if (flags & ~(STCE_QUANT_TILE | STCE_QUANT_TRANSPOSE))
    return fail(STCE_E_ARG, "flags=%d has unknown bits", (int)flags);
  if (R < 0 || C < 0 || R > (1 << 28) || C > (1 << 22) || ((flags & STCE_QUANT_TRANSPOSE) && R > (1 << 22)))
    return fail(STCE_E_ARG, "R=%lld, C=%lld out of range (2^28 rows, 2^22 values per row of the result)",
                (long long)R, (long long)C);
  if (ld < C || !extent_ok(R, ld, es))
    return fail(STCE_E_ARG, "ld=%lld must be at least C=%lld", (long long)ld, (long long)C);
  if (ceil_div(R, 128) * ceil_div(C, 128) > MAX_WORKGROUPS)
    return fail(STCE_E_UNSUPPORTED, "R=%lld x C=%lld has too many blocks for one launch", (long long)R, (long long)C);
  const int64_t L = (flags & STCE_QUANT_TRANSPOSE) ? R : C, Q = (flags & STCE_QUANT_TRANSPOSE) ? C : R;
  if (ld_codes % 16 != 0 || ld_codes < round_up(L, 16) || !extent_ok(Q, ld_codes, 1))
    return fail(STCE_E_ARG, "ld_codes=%lld must be a multiple of 16 and at least %lld", (long long)ld_codes,
                (long long)L);
  if (R == 0 || C == 0) return STCE_OK;
  if (!x || !codes || !scales) return fail(STCE_E_ARG, "x, codes and scales are required");
  if (!is_aligned(x, es) || !is_aligned(codes, 16) || !is_aligned(scales, 4))
    return fail(STCE_E_ARG, "x and scales must be aligned to their elements, codes to 16 bytes");
  const size_t nx = bytes_of(R, C, ld, es);
  if (overlap(x, nx, codes, bytes_of(Q, round_up(L, 16), ld_codes, 1)) ||
      overlap(x, nx, scales,
              4 * (size_t)ceil_div(L, 128) * (size_t)((flags & STCE_QUANT_TILE) ? ceil_div(Q, 128) : Q)))
    return fail(STCE_E_ARG, "codes or scales overlap x");
  const hipError_t e = launch_quantize_blocks(x, dtype, R, C, ld, flags, codes, ld_codes, scales, (hipStream_t)stream);
  return e ? hip_fail(e, "quantize blocks") : STCE_OK;
}

stce_status stce_fp8_block_matmul_workspace_bytes(const stce_block_matmul* p, size_t* bytes) {
  const stce_status s = check_matmul_shapes(p);
  if (s) return s;
  if (!bytes) return fail(STCE_E_ARG, "bytes is NULL");
  *bytes = p->M && p->N ? block_matmul_workspace_bytes(*p) : 0;
  return STCE_OK;
}

stce_status stce_fp8_block_matmul(const stce_block_matmul* p, void* ws, size_t ws_bytes, void* stream) {
  stce_status s = check_matmul_shapes(p);
  if (s) return s;
  if (p->M == 0 || p->N == 0) return STCE_OK;
  const size_t es = value_size(p->out_dtype);
  if (!p->out || (p->K > 0 && (!p->a || !p->b || !p->a_scale || !p->b_scale)))
    return fail(STCE_E_ARG, "a, b, their scales and out are required");
  if (!is_aligned(p->a, 16) || !is_aligned(p->b, 16) || !is_aligned(p->a_scale, 4) || !is_aligned(p->b_scale, 4) ||
      !is_aligned(p->out, es))
    return fail(STCE_E_ARG, "a and b must be 16-byte aligned, scales and out aligned to their elements");
  const size_t nout = bytes_of(p->M, p->N, p->ldo, es);
  if (overlap(p->out, nout, p->a, bytes_of(p->M, p->K, p->lda, 1)) ||
      overlap(p->out, nout, p->b, bytes_of(p->N, p->K, p->ldb, 1)))
    return fail(STCE_E_ARG, "out overlaps a or b");
  if ((s = check_ws(ws, ws_bytes, block_matmul_workspace_bytes(*p)))) return s;
  const hipError_t e = launch_block_matmul(*p, ws, (hipStream_t)stream);
  return e ? hip_fail(e, "block matmul") : STCE_OK;
}

}  // extern "C"
