// extern "C" entry points of the token log probabilities: host-side argument checks, workspace size
// and dispatch.  See include/spec_verify.h for the contract.

#include <climits>
#include <cmath>

#include "sv_cache_check.hpp"
#include "sv_logprob.hpp"

using namespace sv;

namespace {

bool shape_ok(int R, int V, int n) { return R >= 1 && V >= 1 && n >= 0 && n <= kLogprobMaxTop; }

bool dtype_ok(sv_dtype dt) { return dt == SV_DTYPE_F32 || dt == SV_DTYPE_BF16; }

}  // namespace

extern "C" {

size_t spec_token_logprobs_workspace_size(int R, int V, sv_dtype dtype, int top_n) {
  if (!dtype_ok(dtype) || !shape_ok(R, V, top_n)) return 0;
  const size_t need = plan_logprobs(R, V, dtype, top_n).bytes;
  return need ? need : 16;
}

int spec_token_logprobs(const void* logits, sv_dtype dtype, int num_rows, int V,
                        const int32_t* rows, const int32_t* tokens, int R, float temperature,
                        int top_n, float* out_logprob, int32_t* out_rank, float* out_entropy,
                        int32_t* out_top_tokens, float* out_top_logprobs, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype)) return SV_ERR_UNSUPPORTED_DTYPE;
  const int es = dtype == SV_DTYPE_BF16 ? 2 : 4;
  if (!logits || num_rows < 1 || !shape_ok(R, V, top_n) || (!rows && R != num_rows))
    return SV_ERR_INVALID_ARG;
  if ((uint64_t)num_rows * V > (uint64_t)1 << 60) return SV_ERR_INVALID_ARG;  // no memory holds them
  const double c = 1.44269504088896340736 / (double)temperature;
  if (!(temperature > 0.0f) || !std::isfinite(temperature) || !(c > 0.0) ||
      !std::isfinite((float)c) || (float)c == 0.0f)
    return SV_ERR_INVALID_ARG;
  if ((tokens == nullptr) != (out_logprob == nullptr) || (out_rank && !tokens) ||
      (top_n > 0) != (out_top_tokens != nullptr) || (top_n > 0) != (out_top_logprobs != nullptr) ||
      (!tokens && !out_entropy && !top_n))
    return SV_ERR_INVALID_ARG;
  if (!aligned_to(logits, es) || !aligned_to(rows, 4) || !aligned_to(tokens, 4) ||
      !aligned_to(out_logprob, 4) || !aligned_to(out_rank, 4) || !aligned_to(out_entropy, 4) ||
      !aligned_to(out_top_tokens, 4) || !aligned_to(out_top_logprobs, 4))
    return SV_ERR_INVALID_ARG;
  const LogprobPlan p = plan_logprobs(R, V, dtype, top_n);
  if (p.bytes && (!workspace || workspace_bytes < p.bytes)) return SV_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned_to(workspace, 16)) return SV_ERR_INVALID_ARG;
  const uint64_t word = sizeof(int32_t), some = word * R;
  const Range ranges[] = {{out_logprob, some}, {out_rank, some}, {out_entropy, some},
                          {out_top_tokens, some * top_n}, {out_top_logprobs, some * top_n},
                          {p.bytes ? workspace : nullptr, p.bytes},
                          {logits, (uint64_t)num_rows * V * es}, {rows, some}, {tokens, some}};
  if (!outputs_apart(ranges, 6)) return SV_ERR_INVALID_ARG;
  LogprobArgs a{};
  a.logits = static_cast<const char*>(logits);
  a.num_rows = num_rows;
  a.V = V;
  a.rows = rows;
  a.tokens = tokens;
  a.R = R;
  a.n = top_n;
  a.c = (float)c;
  a.logprob = out_logprob;
  a.rank = out_rank;
  a.entropy = out_entropy;
  a.top_tokens = out_top_tokens;
  a.top_logprobs = out_top_logprobs;
  a.parts = p.parts;
  a.part_vecs = p.part_vecs;
  char* ws = static_cast<char*>(workspace);
  a.part = reinterpret_cast<LogprobPart*>(ws);
  a.part_top = p.bytes ? reinterpret_cast<unsigned long long*>(ws + p.o_top) : nullptr;
  return status_of(launch_logprobs(a, dtype, stream));
}

}  // extern "C"
