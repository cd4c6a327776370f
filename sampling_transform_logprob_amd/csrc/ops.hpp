// Launchers of the operators on given arrays: token log probabilities and
// their gradient, block-scaled fp8 quantization and product (host side).
#pragma once

#include "../../include/stce.h"
#include "common.hpp"
#include "kernels.hpp"

namespace stce {

constexpr int TOP_MAX = 128;     // alternatives per row
constexpr int TOKENS_MAX = 1024; // given tokens per row

// A row's statistics as the forward leaves them for the backward.
struct TokenStats {
  float m;        // largest logit (raw)
  float log_sum;  // log sum exp((z - m) / T)
  float entropy;
  float zero;
};

size_t token_workspace_bytes(const stce_token_problem& p);
hipError_t launch_token_logprobs(const stce_token_problem& p, const stce_token_outputs& o, int64_t* status, void* ws,
                                 hipStream_t s);
hipError_t launch_token_grad(const stce_token_problem& p, const TokenStats* stats, const float* g_lp,
                             const float* g_ent, const float* g_lse, void* grad, int64_t ld_grad, hipStream_t s);

hipError_t launch_quantize_blocks(const void* x, int dtype, int64_t R, int64_t C, int64_t ld, int flags,
                                  uint8_t* codes, int64_t ld_codes, float* scales, hipStream_t s);

size_t block_matmul_workspace_bytes(const stce_block_matmul& p);
hipError_t launch_block_matmul(const stce_block_matmul& p, void* ws, hipStream_t s);

}  // namespace stce
