// logprobs.cu -- log probabilities of given tokens, with rank, entropy and
// top alternatives.
//
// Per row, with t_x = (z_x - M) / T, M = max z:
//   S = sum e^t, ln p(x) = t_x - ln S, H = ln S - (1 / S) sum e^t t,
//   rank = 1 + #{z_x > z_tok} + #{z_x = z_tok, x < tok},
//   the top n in the order (z descending, index ascending).
//
// One CTA per row: a pass for M, a pass for S, the entropy sum and the rank,
// and one pass per alternative (the largest pair below the last one in that
// order).
#include "../../include/spec_verify.h"
#include "sv_device.cuh"

#include <climits>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

namespace sv {
namespace lp {

struct Params {
  const char* logits;
  long long ld_bytes;
  int V, R, B, n_top;
  const int32_t* tokens;
  const int32_t* cu;
  const int32_t* out_len;
  float c;       // log2(e) / T
  double inv_T;
  float* logprob;
  int32_t* rank;
  float* entropy;
  int32_t* top_ids;
  float* top_lp;
  uint32_t* status;
};

__device__ __forceinline__ void flag(const Params& P, uint32_t bit) {
  if (P.status) atomicOr(P.status, bit);
}

// Whether row r is asked for: with offsets, only a request's committed rows.
// The search ends for any contents of cu, and what it finds is checked.
__device__ __forceinline__ bool row_wanted(const Params& P, int r) {
  if (!P.cu) return true;
  int lo = 0, hi = P.B;  // the request is in [lo, hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((long long)P.cu[mid] + mid <= r)
      lo = mid;
    else
      hi = mid;
  }
  const long long i = (long long)r - P.cu[lo] - lo;
  const long long K = (long long)P.cu[lo + 1] - P.cu[lo];
  const int n = P.out_len[lo];
  return K >= 0 && n <= K + 1 && i >= 0 && i < n;
}

// The packed layout, checked once a call (by one CTA).
__device__ __forceinline__ void check_offsets(const Params& P, int tid) {
  if (!P.cu) return;
  bool bad = tid == 0 && P.cu[0] != 0;
  for (int b = tid; b < P.B; b += kThreads) {
    const long long K = (long long)P.cu[b + 1] - P.cu[b];
    bad |= K < 0 || P.out_len[b] < 0 || P.out_len[b] > K + 1;
  }
  if (bad) flag(P, SV_DATA_BAD_OFFSETS);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(Params P) {
  __shared__ float s_f[kWarps];
  __shared__ int s_i[kWarps];
  __shared__ double s_d[2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x;
  if (r == 0) check_offsets(P, tid);
  if (!row_wanted(P, r)) return;
  const char* row = P.logits + (long long)r * P.ld_bytes;
  const int V = P.V;
  const int tok = P.tokens ? P.tokens[r] : -1;
  const bool tok_ok = tok >= 0 && tok < V;

  float m = -INFINITY;
  bool bad = false;
  for (int x = tid; x < V; x += kThreads) {
    const float z = Elem<DT>::scalar(row, x);
    bad |= !(z < INFINITY);
    m = fmaxf(m, z);
  }
  bad = __syncthreads_or(bad);
  m = warp_max(m);
  if (lane == 0) s_f[warp] = m;
  __syncthreads();
  m = s_f[0];
  for (int w = 1; w < kWarps; ++w) m = fmaxf(m, s_f[w]);
  if (bad || m == -INFINITY || (P.tokens && !tok_ok)) {
    if (tid == 0) {
      if (bad) flag(P, SV_DATA_BAD_LOGIT);
      if (!bad && m == -INFINITY) flag(P, SV_DATA_EMPTY_ROW);
      if (P.tokens && !tok_ok) flag(P, SV_DATA_BAD_TOKEN);
      if (P.logprob) P.logprob[r] = NAN;
      if (P.rank) P.rank[r] = 0;
    }
    if (bad || m == -INFINITY) {
      if (tid == 0 && P.entropy) P.entropy[r] = NAN;
      for (int j = tid; j < P.n_top; j += kThreads) {
        if (P.top_ids) P.top_ids[(long long)r * P.n_top + j] = -1;
        if (P.top_lp) P.top_lp[(long long)r * P.n_top + j] = NAN;
      }
      return;
    }
  }
  const float zt = tok_ok ? Elem<DT>::scalar(row, tok) : 0.f;
  float S = 0.f, S1 = 0.f;
  int above = 0;
  for (int x = tid; x < V; x += kThreads) {
    const float z = Elem<DT>::scalar(row, x);
    const float t = (z - m) * P.c;
    const float e = ex2(t);
    S += e;
    if (e > 0.f) S1 = fmaf(e, t, S1);
    above += z > zt || (z == zt && x < tok);
  }
  double dS = S, dS1 = S1;
  for (int o = 16; o > 0; o >>= 1) {
    dS += __shfl_xor_sync(kFull, dS, o);
    dS1 += __shfl_xor_sync(kFull, dS1, o);
    above += __shfl_xor_sync(kFull, above, o);
  }
  if (lane == 0) {
    s_d[0][warp] = dS;
    s_d[1][warp] = dS1;
    s_i[warp] = above;
  }
  __syncthreads();
  dS = dS1 = 0.0;
  above = 0;
  for (int w = 0; w < kWarps; ++w) {
    dS += s_d[0][w];
    dS1 += s_d[1][w];
    above += s_i[w];
  }
  const double lnS = log(dS);
  if (tid == 0) {
    if (tok_ok) {
      if (P.logprob) P.logprob[r] = (float)(((double)zt - (double)m) * P.inv_T - lnS);
      if (P.rank) P.rank[r] = 1 + above;
    }
    if (P.entropy) P.entropy[r] = (float)(lnS - dS1 / dS * 0.6931471805599453);
  }
  // Alternatives: each pass finds the largest (value, lowest index) below the last.
  float lv = INFINITY;
  int li = -1;
  for (int j = 0; j < P.n_top; ++j) {
    float bv = -INFINITY;
    int bi = INT_MAX;
    for (int x = tid; x < V; x += kThreads) {
      const float z = Elem<DT>::scalar(row, x);
      if (z < lv || (z == lv && x > li)) argmax_merge(bv, bi, z, x);
    }
    warp_argmax(bv, bi);
    __syncthreads();
    if (lane == 0) {
      s_f[warp] = bv;
      s_i[warp] = bi;
    }
    __syncthreads();
    lv = s_f[0];
    li = s_i[0];
    for (int w = 1; w < kWarps; ++w) argmax_merge(lv, li, s_f[w], s_i[w]);
    if (tid == 0) {
      const bool any = lv > -INFINITY;
      if (P.top_ids) P.top_ids[(long long)r * P.n_top + j] = any ? li : -1;
      if (P.top_lp)
        P.top_lp[(long long)r * P.n_top + j] = any ? (float)(((double)lv - (double)m) * P.inv_T - lnS) : -INFINITY;
    }
  }
}

}  // namespace lp
}  // namespace sv

extern "C" sv_status sv_token_logprobs(const void* logits, sv_dtype dtype, int32_t V, int64_t ld, int32_t R,
                                       const int32_t* tokens, int32_t B, const int32_t* cu_draft,
                                       const int32_t* out_len, float temperature, int32_t n_top,
                                       float* out_logprob, int32_t* out_rank, float* out_entropy,
                                       int32_t* out_top_ids, float* out_top_logprobs, uint32_t* status,
                                       void* cuda_stream) {
  using namespace sv;
  if ((dtype != SV_FP32 && dtype != SV_BF16) || V < 1 || ld < V || R < 0 || B < 0) return SV_ERR_INVALID_ARG;
  const int es = dtype == SV_BF16 ? 2 : 4;
  if (ld > INT64_MAX / 4) return SV_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || std::isinf(temperature)) return SV_ERR_INVALID_ARG;
  if (n_top < 0 || n_top > SV_LOGPROBS_MAX_TOP) return SV_ERR_INVALID_ARG;
  if (!tokens && (out_logprob || out_rank)) return SV_ERR_INVALID_ARG;
  if ((cu_draft == nullptr) != (out_len == nullptr) || (!cu_draft && B != 0)) return SV_ERR_INVALID_ARG;
  const void* words[] = {tokens, cu_draft, out_len, out_logprob, out_rank, out_entropy, out_top_ids, out_top_logprobs, status};
  for (const void* p : words)
    if ((uintptr_t)p % 4) return SV_ERR_INVALID_ARG;
  if (R == 0 || (cu_draft && B == 0)) return SV_OK;
  if (!logits || (uintptr_t)logits % es) return SV_ERR_INVALID_ARG;
  lp::Params P{};
  P.logits = static_cast<const char*>(logits);
  P.ld_bytes = ld * es;
  P.V = V;
  P.R = R;
  P.B = B;
  P.n_top = n_top;
  P.tokens = tokens;
  P.cu = cu_draft;
  P.out_len = out_len;
  P.c = (float)(1.4426950408889634 / (double)temperature);
  P.inv_T = 1.0 / (double)temperature;
  P.logprob = out_logprob;
  P.rank = out_rank;
  P.entropy = out_entropy;
  P.top_ids = out_top_ids;
  P.top_lp = out_top_logprobs;
  P.status = status;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (dtype == SV_BF16)
    lp::logprobs_kernel<1><<<R, kThreads, 0, st>>>(P);
  else
    lp::logprobs_kernel<0><<<R, kThreads, 0, st>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
