// attention.cu -- attention of the verify windows over the paged cache.
//
// Row w of a window whose candidate begins at w0 sees tokens 0 .. ctx - 1 and
// ctx + w0 .. ctx + w. With s_t = scale * q . k_t, running maximum m and sum l
// over the tokens seen so far, a new score s updates
//   m' = max(m, s), l' = l e^(m - m') + e^(s - m'), o' = o e^(m - m') + e^(s - m') v
// and out = o / l, lse = m + ln l.
//
// One warp a (row, query head): the lanes hold the head's elements, one token
// at a time.
#include "sv_cache.cuh"

#include <cmath>
#include <cuda_bf16.h>

namespace sv {
namespace att {

constexpr int kT = 256;

struct Params {
  CacheView C;
  SeqView S;
  WindowView W;
  const char* q;
  char* out;
  long long q_row_b, out_row_b;
  float* lse;
  float scale_log2;  // scale * log2(e)
  int group;         // query heads to a key-value head
  uint32_t* status;
};

template <int DT, int D>
__global__ void __launch_bounds__(kT) window_kernel(Params P) {
  constexpr int EPL = D / 32;
  const int lane = threadIdx.x & 31;
  const int heads = P.C.n_heads * P.group;
  for (int b = blockIdx.y; b < P.S.n; b += gridDim.y) {
    const Window w = find_window(P.W, b);
    const long long ctx = P.S.ctx[b];
    if (w.rows < 0 || !length_ok(P.C, P.S, ctx) || !length_ok(P.C, P.S, ctx + w.rows)) {
      if (blockIdx.x == 0 && threadIdx.x == 0)
        set_status(P.status, w.rows < 0 ? SV_DATA_BAD_OFFSETS
                                        : length_ok(P.C, P.S, ctx) ? SV_DATA_BAD_PAGE : SV_DATA_BAD_SEQ);
      continue;
    }
    const int32_t* row = P.S.table + (long long)b * P.S.stride;
    const long long n = (long long)w.rows * heads;
    for (long long u = blockIdx.x * (kT / 32) + (threadIdx.x >> 5); u < n; u += gridDim.x * (kT / 32)) {
      const int r = (int)(u / heads), h = (int)(u % heads);
      int begin = r;  // the candidate's first row
      if (P.W.cu) {
        int lo = w.c0, hi = w.c1;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if ((long long)P.W.cu[mid] + mid - w.r0 <= r)
            lo = mid;
          else
            hi = mid;
        }
        const long long at = (long long)P.W.cu[lo] + lo - w.r0;
        begin = at < 0 || at > r ? r : (int)at;
      }
      const char* qp = P.q + (w.r0 + r) * P.q_row_b + (long long)h * P.C.head_bytes;
      float q[EPL], o[EPL];
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        q[e] = Elem<DT>::scalar(qp, e * 32 + lane) * P.scale_log2;
        o[e] = 0.f;
      }
      float m = -INFINITY, l = 0.f;
      const long long head_at = (long long)(h / P.group) * P.C.head_b;
      for (long long t = 0; t <= ctx + r; ++t) {
        if (t >= ctx && t < ctx + begin) continue;
        const int page = row[t / P.C.page_size];
        if (page < 0 || page >= P.C.n_pages) {
          if (lane == 0) set_status(P.status, SV_DATA_BAD_PAGE);
          continue;
        }
        const long long at = page * P.C.page_b + (t % P.C.page_size) * P.C.token_b + head_at;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) s = fmaf(q[e], Elem<DT>::scalar(P.C.k + at, e * 32 + lane), s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
        const float m2 = fmaxf(m, s), f = ex2(m - m2), p = ex2(s - m2);
        m = m2;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < EPL; ++e) o[e] = fmaf(p, Elem<DT>::scalar(P.C.v + at, e * 32 + lane), o[e] * f);
      }
      char* op = P.out + (w.r0 + r) * P.out_row_b + (long long)h * P.C.head_bytes;
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        const float x = o[e] * inv;
        if (DT == 1)
          reinterpret_cast<__nv_bfloat16*>(op)[e * 32 + lane] = __float2bfloat16_rn(x);
        else
          reinterpret_cast<float*>(op)[e * 32 + lane] = x;
      }
      if (P.lse && lane == 0)
        P.lse[(long long)(w.r0 + r) * heads + h] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
  }
}

}  // namespace att
}  // namespace sv

extern "C" {

size_t sv_window_attention_workspace_size(const sv_kv_cache* cache, int32_t n_q_heads, int32_t R) {
  if (!cache || n_q_heads < 1 || R < 0) return 0;
  return 16;
}

sv_status sv_window_attention(const void* q, int64_t q_stride, int32_t n_q_heads, int32_t R, const sv_kv_cache* cache,
                              int32_t layer, const sv_sequences* seqs, int32_t n_cand, const int32_t* cu_draft,
                              const int32_t* cu_cand, float scale, void* out, int64_t out_stride, float* out_lse,
                              void* workspace, size_t workspace_bytes, uint32_t* status, void* cuda_stream) {
  using namespace sv;
  att::Params P{};
  if (!cache_view(cache, &P.C) || !seq_view(seqs, &P.S) || !window_view(P.S.n, n_cand, cu_draft, cu_cand, R, &P.W))
    return SV_ERR_INVALID_ARG;
  const int es = elem_size(cache->dtype), D = cache->head_dim;
  if (D != 64 && D != 128) return SV_ERR_INVALID_ARG;
  if (n_q_heads < 1 || n_q_heads % P.C.n_heads || n_q_heads / P.C.n_heads > 64) return SV_ERR_INVALID_ARG;
  if (layer < 0 || layer >= P.C.n_layers || !std::isfinite(scale)) return SV_ERR_INVALID_ARG;
  const int64_t strides[2] = {q_stride, out_stride};
  for (int64_t s : strides)
    if (s < (int64_t)n_q_heads * D || s > INT64_MAX / 4 || s * es % 16) return SV_ERR_INVALID_ARG;
  if ((uintptr_t)out_lse % 4 || (uintptr_t)status % 4) return SV_ERR_INVALID_ARG;
  if (P.S.n == 0 || R == 0) return SV_OK;
  if (!q || !out || (uintptr_t)q % 16 || (uintptr_t)out % 16) return SV_ERR_INVALID_ARG;
  if (!workspace || (uintptr_t)workspace % 16 ||
      workspace_bytes < sv_window_attention_workspace_size(cache, n_q_heads, R))
    return SV_ERR_INVALID_ARG;
  P.C.k += layer * P.C.layer_b;
  P.C.v += layer * P.C.layer_b;
  P.q = static_cast<const char*>(q);
  P.out = static_cast<char*>(out);
  P.q_row_b = q_stride * es;
  P.out_row_b = out_stride * es;
  P.lse = out_lse;
  P.scale_log2 = (float)((double)scale * 1.4426950408889634);
  P.group = n_q_heads / P.C.n_heads;
  P.status = status;
  const int gy = P.S.n > 32768 ? 32768 : P.S.n;
  const long long per = ((long long)R * n_q_heads + gy - 1) / gy;
  const long long want = (per + att::kT / 32 - 1) / (att::kT / 32), most = 152 * 64 / gy + 1;
  const dim3 grid((unsigned)(want < most ? want : most), gy);
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (es == 2 && D == 128)
    att::window_kernel<1, 128><<<grid, att::kT, 0, st>>>(P);
  else if (es == 2)
    att::window_kernel<1, 64><<<grid, att::kT, 0, st>>>(P);
  else if (D == 128)
    att::window_kernel<0, 128><<<grid, att::kT, 0, st>>>(P);
  else
    att::window_kernel<0, 64><<<grid, att::kT, 0, st>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
