// Token log probabilities: kernels in sv_logprob.hip, C entry points in sv_logprob_abi.hip.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "spec_verify.h"

namespace sv {

constexpr int kLogprobMaxTop = 64;  // alternatives a row

// What a part of a row leaves for the others: sums of 2^(x - shift), x = z log2(e) / T.
struct alignas(16) LogprobPart {
  double shift;
  double sum, sum_x;  // of e and of e (x - shift)
  float top;          // largest logit
  int above;          // logits that come before the token's
};

struct LogprobArgs {
  const char* logits;    // [num_rows, V]
  int num_rows, V;
  const int32_t* rows;   // [R] or null
  const int32_t* tokens; // [R] or null
  int R, n;              // n: alternatives
  float c;               // log2(e) / T
  float* logprob;
  int32_t* rank;
  float* entropy;
  int32_t* top_tokens;   // [R, n]
  float* top_logprobs;
  int parts;             // workgroups a row
  int part_vecs;         // 16-byte vectors a part
  LogprobPart* part;     // [R][parts]
  unsigned long long* part_top;  // [R][parts][n]
};

struct LogprobPlan {
  int parts, part_vecs;
  size_t o_top, bytes;  // workspace: parts at 0; 0 bytes where a row is one part
};

LogprobPlan plan_logprobs(int R, int V, sv_dtype dt, int n);
hipError_t launch_logprobs(const LogprobArgs& a, sv_dtype dt, hipStream_t stream);

}  // namespace sv
