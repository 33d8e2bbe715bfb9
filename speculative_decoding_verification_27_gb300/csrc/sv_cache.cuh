// sv_cache.cuh -- what the page operations and the attention over the paged
// cache share: the kernels' view of a cache, of its sequences and of the
// windows, the host checks of all three, and the search for a window.
#pragma once

#include "../../include/spec_verify.h"
#include "sv_device.cuh"

#include <cstdint>
#include <cuda_runtime.h>

namespace sv {

// Bytes throughout, so that the copies do not depend on the element type.
struct CacheView {
  char* k;
  char* v;
  long long layer_b, page_b, token_b, head_b;  // strides
  int n_layers, n_pages, page_size, n_heads, head_bytes;
  int32_t* ref;
  uint32_t* free_bits;
  uint32_t div_mul, div_shift;  // t / page_size = t * div_mul >> div_shift
  float* ks;                    // SV_E4M3: scales, else null; their strides in elements
  float* vs;
  long long s_layer, s_page, s_token, s_head;
};

struct SeqView {
  int32_t* table;
  long long stride;
  int width, n;
  int32_t* ctx;
};

struct WindowView {
  const int32_t* cu;    // [n_cand + 1], or null: one row a sequence
  const int32_t* cand;  // [n + 1], or null: candidate b is request b
  int n_cand, R;        // R: rows that the caller holds
};

inline int elem_size(sv_dtype d) { return d == SV_E4M3 ? 1 : d == SV_BF16 ? 2 : 4; }
// Of the rows that go with a cache: queries, outputs, new keys and values.
inline int row_elem_size(sv_dtype d) { return d == SV_FP32 ? 4 : 2; }

// Host checks; null where a description cannot be used.
inline bool cache_view(const sv_kv_cache* c, CacheView* out) {
  if (!c || (c->dtype != SV_FP32 && c->dtype != SV_BF16 && c->dtype != SV_E4M3)) return false;
  if (c->n_layers < 1 || c->n_pages < 1 || c->page_size < 1 || c->n_kv_heads < 1 || c->head_dim < 1) return false;
  if (c->page_size > (1 << 20) || c->head_dim > (1 << 16) || c->n_kv_heads > (1 << 16)) return false;
  if (!c->k || !c->v || (uintptr_t)c->k % 16 || (uintptr_t)c->v % 16) return false;
  if (!c->page_ref || !c->free_bits || (uintptr_t)c->page_ref % 4 || (uintptr_t)c->free_bits % 4) return false;
  const int es = elem_size(c->dtype);
  const int64_t s[4] = {c->layer_stride, c->page_stride, c->token_stride, c->head_stride};
  for (int64_t x : s)
    if (x < 0 || x > INT64_MAX / 4 || x * es % 16) return false;
  if ((int64_t)c->head_dim * es % 16) return false;
  // The 16-byte vectors of a page (of one layer, K or V) are counted in 31 bits.
  if ((int64_t)c->n_kv_heads * (c->head_dim * es / 16) > (1 << 20)) return false;
  if ((int64_t)c->n_kv_heads * (c->head_dim * es / 16) * c->page_size > (1 << 30)) return false;
  *out = CacheView{static_cast<char*>(c->k), static_cast<char*>(c->v), s[0] * es, s[1] * es, s[2] * es, s[3] * es,
                   c->n_layers, c->n_pages, c->page_size, c->n_kv_heads, c->head_dim * es, c->page_ref, c->free_bits, 0, 0,
                   nullptr, nullptr, 0, 0, 0, 0};
  if (c->dtype == SV_E4M3) {
    const int64_t t[4] = {c->scale_layer_stride, c->scale_page_stride, c->scale_token_stride, c->scale_head_stride};
    for (int64_t x : t)
      if (x < 0 || x > INT64_MAX / 4) return false;
    if (!c->k_scale || !c->v_scale || (uintptr_t)c->k_scale % 4 || (uintptr_t)c->v_scale % 4 || c->head_dim > 256) return false;
    out->ks = c->k_scale;
    out->vs = c->v_scale;
    out->s_layer = t[0], out->s_page = t[1], out->s_token = t[2], out->s_head = t[3];
  }
  // A dimension of one element takes no step: give it the one that lets copies run through.
  if (out->n_heads == 1) out->head_b = out->head_bytes;
  if (out->page_size == 1) out->token_b = out->n_heads * out->head_b;
  // For t < 2^31: with 2^s the next power of two, m = ceil(2^(31 + s) / page_size) errs by less than 2^s, so that t m / 2^(31 + s)
  // is less than 1 / page_size too large.
  int log2 = 0;
  while ((1ll << log2) < c->page_size) ++log2;
  out->div_shift = 31 + log2;
  out->div_mul = (uint32_t)(((1ull << (31 + log2)) + c->page_size - 1) / c->page_size);
  return true;
}

// Whether a call may write the scales: each (layer, page, token, head) has one of its own, as far as strides of zero tell.
inline bool scales_apart(const CacheView& C) {
  return !C.ks || !((C.n_layers > 1 && !C.s_layer) || (C.n_pages > 1 && !C.s_page) || (C.page_size > 1 && !C.s_token) ||
                    (C.n_heads > 1 && !C.s_head));
}

inline bool seq_view(const sv_sequences* s, SeqView* out) {
  if (!s || s->n < 0 || s->table_pages < 1 || s->table_stride < s->table_pages) return false;
  if (s->n > 0 && (!s->table || !s->ctx_len || (uintptr_t)s->table % 4 || (uintptr_t)s->ctx_len % 4)) return false;
  *out = SeqView{s->table, s->table_stride, s->table_pages, s->n, s->ctx_len};
  return true;
}

inline bool window_view(int n, int32_t n_cand, const int32_t* cu, const int32_t* cand, int R, WindowView* out) {
  if (n_cand < 0 || R < 0 || (uintptr_t)cu % 4 || (uintptr_t)cand % 4) return false;
  if (!cand && n_cand != n) return false;
  if (cand && !cu) return false;
  *out = WindowView{cu, cand, n_cand, R};
  return true;
}

__device__ __forceinline__ void set_status(uint32_t* status, uint32_t bit) {
  if (status) atomicOr(status, bit);
}

// Request b's candidates [c0, c1) and window rows [r0, r0 + rows); rows = -1
// where the offsets are out of order or out of range (R < 0: no row limit).
// A request's candidates are looked over by the whole warp (all lanes with
// the same b) or, with kWarp false, by the thread.
struct Window {
  int c0, c1, r0, rows;
};
template <bool kWarp>
__device__ __forceinline__ Window find_window(const WindowView& W, int b) {
  if (!W.cu) return W.R < 0 || b < W.R ? Window{b, b + 1, b, 1} : Window{b, b, 0, -1};
  const int c0 = W.cand ? W.cand[b] : b, c1 = W.cand ? W.cand[b + 1] : b + 1;
  if (c0 < 0 || c1 < c0 || c1 > W.n_cand) return Window{0, 0, 0, -1};
  const int first = W.cu[c0], end = W.cu[c1];
  bool bad = false;
  if (W.cand) {  // (looked at beside the two above: behind their test it is one more round trip to memory)
    if constexpr (kWarp) {
      for (int c = c0 + (int)(threadIdx.x & 31); c < c1; c += 32) bad |= W.cu[c + 1] < W.cu[c];
      bad = __any_sync(kFull, bad);
    } else {
#pragma unroll 4
      for (int c = c0; c < c1; ++c) bad |= W.cu[c + 1] < W.cu[c];
    }
  }
  const long long r0 = (long long)first + c0, r1 = (long long)end + c1;
  if (bad || first < 0 || r1 < r0 + (c1 - c0) || r1 > 0x7fffffffll || (W.R >= 0 && r1 > W.R)) return Window{0, 0, 0, -1};
  return Window{c0, c1, (int)r0, (int)(r1 - r0)};
}

// The first row of the candidate that window row w lies in.
__device__ __forceinline__ int candidate_start(const WindowView& W, const Window& win, int w) {
  if (!W.cand) return 0;
  int a = win.c0, z = win.c1;
  while (z - a > 1) {
    const int mid = (a + z) >> 1;
    if ((long long)W.cu[mid] + mid - win.r0 <= w)
      a = mid;
    else
      z = mid;
  }
  const long long at = (long long)W.cu[a] + a - win.r0;
  return at < 0 || at > w ? w : (int)at;
}

// t / page_size, 0 <= t < 2^31.
__device__ __forceinline__ int page_slot(const CacheView& C, int t) {
  return (int)(((unsigned long long)(uint32_t)t * C.div_mul) >> C.div_shift);
}

// A length that fits its table, and 31 bits with the rest of a tile.
__device__ __forceinline__ bool length_ok(const CacheView& C, const SeqView& S, long long len) {
  return len >= 0 && len <= (long long)S.width * C.page_size && len <= 0x7fff0000ll;
}

}  // namespace sv
