// cache.cu -- the pages of a key-value cache around the verify step: fork,
// free, reserve (with the copy of shared partial pages), append, commit.
//
// Free pages are bits, not a stack: whoever releases a page only sets its
// bit when the count falls to zero, and the allocator takes the lowest set
// bits in the order of the sequences. Both are independent of timing, so the
// page tables are the same from run to run.
//
// The calls on tables are bound by their chains of dependent loads (5 us each
// with a cold cache, reserve 10), the copies by their bytes: 256 forks whose
// partial pages of 64 tokens are copied in 4 layers take 27 us for 130 MB, the
// rows of a layer for 64 prompts of 1000 tokens 82 us for 520 MB (94% of the
// copy rate).
#include "sv_cache.cuh"
#include "sv_launch.cuh"

#include <climits>

namespace sv {
namespace cache {

constexpr int kT = 256;

__device__ __forceinline__ int pages_of(long long tokens, int page_size) {
  return (int)((tokens + page_size - 1) / page_size);
}

// One holder less; a page without holders is free.
__device__ __forceinline__ void release(const CacheView& C, int page, uint32_t* status) {
  if (page < 0 || page >= C.n_pages) {
    set_status(status, SV_DATA_BAD_PAGE);
    return;
  }
  const int old = atomicSub(&C.ref[page], 1);
  if (old == 1)
    atomicOr(&C.free_bits[page >> 5], 1u << (page & 31));
  else if (old < 1) {
    atomicAdd(&C.ref[page], 1);
    set_status(status, SV_DATA_BAD_PAGE);
  }
}

// Releases entries from `first` up to the first -1, by one warp.
__device__ __forceinline__ void release_from(const CacheView& C, const SeqView& S, int b, int first, int lane,
                                             uint32_t* status) {
  int32_t* row = S.table + (long long)b * S.stride;
  for (int i0 = first; i0 < S.width; i0 += 32) {
    const int i = i0 + lane;
    const int page = i < S.width ? row[i] : -1;
    const unsigned end = __ballot_sync(kFull, page < 0);
    const int n = end ? __ffs(end) - 1 : 32;
    if (lane < n) {
      release(C, page, status);
      row[i] = -1;
    }
    if (end) return;
  }
}

// ---------------------------------------------------------------------------
// Fork and free: one warp an entry
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kT) fork_kernel(CacheView C, SeqView S, int N, const int32_t* src, const int32_t* dst,
                                                  uint32_t* status) {
  release_stream();
  wait_for_stream();
  const int i = blockIdx.x * (kT / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= N) return;
  const int s = src[i], d = dst[i];
  // The entries' own lists decide who is served, whatever the order of the warps.
  bool clash = false;
  for (int j = lane; j < N; j += 32) {
    const int x = dst[j];
    clash |= x == s || (x == d && j < i);
  }
  clash = __any_sync(kFull, clash);
  bool ok = !clash && s >= 0 && s < S.n && d >= 0 && d < S.n;
  int len = 0;
  if (ok) {
    len = S.ctx[s];
    ok = length_ok(C, S, len) && S.ctx[d] == 0 && S.table[(long long)d * S.stride] < 0;
  }
  if (!ok) {
    if (lane == 0) set_status(status, SV_DATA_BAD_SEQ);
    return;
  }
  const int n = pages_of(len, C.page_size);
  const int32_t* from = S.table + (long long)s * S.stride;
  int32_t* to = S.table + (long long)d * S.stride;
  bool good = true;
  // A page that the counts call free is not the source's. (Forks beside this one only raise the counts of pages that have a holder.)
  for (int k = lane; k < n; k += 32) good &= from[k] >= 0 && from[k] < C.n_pages && C.ref[from[k]] >= 1;
  if (!__all_sync(kFull, good)) {
    if (lane == 0) set_status(status, SV_DATA_BAD_PAGE);
    return;
  }
  for (int k = lane; k < n; k += 32) {
    const int page = from[k];
    to[k] = page;
    atomicAdd(&C.ref[page], 1);
  }
  if (lane == 0) S.ctx[d] = len;
}

__global__ void __launch_bounds__(kT) free_kernel(CacheView C, SeqView S, int N, const int32_t* which, uint32_t* status) {
  release_stream();
  wait_for_stream();
  const int i = blockIdx.x * (kT / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= N) return;
  const int s = which[i];
  if (s < 0 || s >= S.n) {
    if (lane == 0) set_status(status, SV_DATA_BAD_SEQ);
    return;
  }
  bool twice = false;
  for (int j = lane; j < i; j += 32) twice |= which[j] == s;
  if (__any_sync(kFull, twice)) return;
  release_from(C, S, s, 0, lane, status);
  if (lane == 0) S.ctx[s] = 0;
}

// ---------------------------------------------------------------------------
// Reserve
// ---------------------------------------------------------------------------
struct CopyJob {
  int from, to, tokens, pad;
};
struct ReserveWs {
  int n_jobs, pad[3];
  CopyJob jobs[1];
};

constexpr int kR = 1024;  // threads of the one CTA that hands out pages

__device__ __forceinline__ int block_excl_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // s_warp is free again
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  total = s_warp[31];
  return x - v + (warp ? s_warp[warp - 1] : 0);
}

// Place of the n-th set bit (n counts from 0).
__device__ __forceinline__ int nth_bit(uint32_t x, int n) {
  int at = 0;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const int c = __popc(x & ((1u << w) - 1u));
    if (n >= c) {
      n -= c;
      at += w;
      x >>= w;
    }
  }
  return at;
}

// The last i in [0, n) with first[i] <= k, of an ascending list with first[0] <= k.
__device__ __forceinline__ int last_at_most(const int* first, int n, int k) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= k)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// One CTA: needs, the order among the sharers of a partial page, a scan, and
// the lowest free bits, whose k-th goes to the request whose range of the
// scan holds k (a thread a page). Shared memory: three words a sequence.
// Bound by the chain of its steps (9 us for a few requests, of which the
// launch and the first loads are half).
__global__ void __launch_bounds__(kR) reserve_kernel(CacheView C, SeqView S, WindowView W, int32_t* granted, ReserveWs* ws,
                                                     uint32_t* status) {
  release_stream();
  wait_for_stream();
  extern __shared__ __align__(16) int s_mem[];
  const int n_pad = (S.n + 4) & ~3;
  int* s_part = s_mem;             // the shared partial page, or -1
  int* s_first = s_mem + n_pad;    // needs, then their exclusive scan [n + 1]
  int* s_have = s_first + n_pad;   // pages held * 2 + 1 if the partial page is copied; -1: refused
  __shared__ int s_warp[32], s_word_first[kR];
  __shared__ uint32_t s_bits[kR];
  __shared__ int s_jobs, s_end, s_shared;
  const int tid = threadIdx.x, n_words = (C.n_pages + 31) / 32;
  // Free pages of word w; what a caller left in the bits past the last page does not count.
  const uint32_t tail = C.n_pages & 31 ? (1u << (C.n_pages & 31)) - 1u : ~0u;
  auto free_word = [&](int w) { return w < n_words ? C.free_bits[w] & (w + 1 == n_words ? tail : ~0u) : 0u; };
  const uint32_t bits0 = free_word(tid);  // early: needed last
  if (tid == 0) {
    s_jobs = s_shared = 0;
    s_end = INT_MAX;
  }
  __syncthreads();
  for (int b = tid; b < S.n; b += kR) {
    const int len = S.ctx[b];
    const Window w = find_window<false>(W, b);
    const int32_t* row = S.table + (long long)b * S.stride;
    int have = -1, need = 0, part = -1;
    uint32_t bad = 0;
    if (w.rows < 0)
      bad = SV_DATA_BAD_OFFSETS;
    else if (!length_ok(C, S, len))
      bad = SV_DATA_BAD_SEQ;
    else if (w.rows > 0 && !length_ok(C, S, (long long)len + w.rows))
      bad = SV_DATA_BAD_PAGE;
    else {
      const int want = pages_of((long long)len + w.rows, C.page_size);
      const int full = page_slot(C, len);
      have = pages_of(len, C.page_size);
      const bool partial = w.rows > 0 && have > full;
      part = partial ? row[full] : -1;
      while (have < S.width && row[have] >= 0) ++have;  // reserved before
      need = max(0, want - have);
      if (partial) {
        const int ref = part >= 0 && part < C.n_pages ? C.ref[part] : 0;
        if (ref < 1) {
          bad = SV_DATA_BAD_PAGE;
          have = -1;
          need = 0;
        }
        if (ref <= 1)
          part = -1;
        else
          s_shared = 1;
      }
    }
    if (bad) set_status(status, bad);
    s_first[b] = need;
    s_have[b] = have < 0 ? -1 : have * 2;
    s_part[b] = part;
  }
  for (int b = S.n + tid; b < n_pad; b += kR) s_part[b] = -1;
  __syncthreads();
  // Who copies: a sharer, unless those before it in this call leave it alone with the page.
  if (s_shared) {
    for (int b = tid; b < S.n; b += kR) {
      const int part = s_part[b];
      if (part < 0) continue;
      int before = 0;
      for (int j = 0; j < b; j += 4) {
        const int4 y = *reinterpret_cast<const int4*>(s_part + j);
        before += (y.x == part && j < b) + (y.y == part && j + 1 < b) + (y.z == part && j + 2 < b) + (y.w == part && j + 3 < b);
      }
      const int left = C.ref[part] - before;
      if (left < 1) {  // more sharers than the count says
        set_status(status, SV_DATA_BAD_PAGE);
        s_have[b] = -1;
        s_first[b] = 0;
      } else if (left > 1) {
        s_have[b] += 1;
        s_first[b] += 1;
      }
    }
    __syncthreads();
  }
  int total = 0;
  for (int b0 = 0; b0 < S.n; b0 += kR) {
    const int b = b0 + tid, v = b < S.n ? s_first[b] : 0;
    int sum;
    const int at = total + block_excl_scan(v, s_warp, sum);
    if (b < S.n) s_first[b] = at;
    total += sum;
  }
  if (tid == 0) s_first[S.n] = total;
  // Free pages, as far as they are asked for. With up to 32 kR pages this scan serves the hand-out too.
  int avail = 0, word_first = 0;
  for (int w0 = 0; w0 < n_words && avail < total; w0 += kR) {
    const int w = w0 + tid;
    int sum;
    word_first = block_excl_scan(__popc(w0 == 0 ? bits0 : free_word(w)), s_warp, sum);
    avail += sum;
  }
  __syncthreads();
  if (avail < total) {
    for (int b = tid; b < S.n; b += kR)
      if (s_first[b + 1] > s_first[b] && s_first[b + 1] > avail) atomicMin(&s_end, b);
    __syncthreads();
    if (tid == 0) set_status(status, SV_DATA_NO_PAGES);
    total = s_first[s_end];
  }
  const int end = s_end;
  for (int b = tid; b < S.n; b += kR) {
    const bool late = b >= end && (s_first[b + 1] > s_first[b] || s_part[b] >= 0);
    if (late) s_have[b] = -1;
    if (granted) granted[b] = s_have[b] >= 0 ? find_window<false>(W, b).rows : 0;
  }
  int taken = 0;
  for (int w0 = 0; w0 < n_words && taken < total; w0 += kR) {
    const int w = w0 + tid;
    const uint32_t bits = w0 == 0 ? bits0 : free_word(w);
    const int mine = __popc(bits);
    int sum = avail, first = word_first;
    if (n_words > kR) first = block_excl_scan(mine, s_warp, sum);
    s_word_first[tid] = first;
    s_bits[tid] = bits;
    const int use = min(max(total - taken - first, 0), mine);
    if (use) {
      uint32_t left = bits;
      for (int i = 0; i < use; ++i) left &= left - 1;
      C.free_bits[w] = left;
    }
    __syncthreads();
    for (int k = taken + tid; k < min(taken + sum, total); k += kR) {
      const int word = last_at_most(s_word_first, kR, k - taken);
      const int page = (w0 + word) * 32 + nth_bit(s_bits[word], k - taken - s_word_first[word]);
      const int b = last_at_most(s_first, S.n, k);
      const int i = k - s_first[b], have = s_have[b] >> 1, copy = s_have[b] & 1;
      int32_t* row = S.table + (long long)b * S.stride;
      C.ref[page] = 1;
      if (copy && i == 0) {
        const int len = S.ctx[b], at = page_slot(C, len), old = row[at];
        row[at] = page;
        atomicSub(&C.ref[old], 1);
        ws->jobs[atomicAdd(&s_jobs, 1)] = CopyJob{old, page, len - at * C.page_size, 0};
      } else {
        row[have + i - copy] = page;
      }
    }
    taken += sum;
    __syncthreads();
  }
  if (tid == 0) ws->n_jobs = s_jobs;
}

// The copies that reserve asked for: a CTA a (job, layer, K or V), 16-byte
// vectors of whole tokens, four a thread in flight.
__global__ void __launch_bounds__(kT) copy_kernel(CacheView C, const ReserveWs* ws) {
  release_stream();
  wait_for_stream();
  const int vecs = C.head_bytes / 16, n_vec = C.n_heads * vecs;
  const bool whole = C.head_b == C.head_bytes && C.token_b == (long long)C.n_heads * C.head_b;  // tokens lie one after another
  const long long n = (long long)ws->n_jobs * C.n_layers * 2;
  for (long long u = blockIdx.x; u < n; u += gridDim.x) {
    const int part = (int)(u % (C.n_layers * 2));
    const CopyJob j = ws->jobs[u / (C.n_layers * 2)];
    char* base = (part & 1 ? C.v : C.k) + (part >> 1) * C.layer_b;
    const char* from = base + j.from * C.page_b;
    char* to = base + j.to * C.page_b;
    const int items = j.tokens * n_vec;  // page_size <= 2^20, heads and vectors within 2^31 in all: see the host checks
    for (int x0 = threadIdx.x; x0 < items; x0 += kT * 4) {
      uint4 v[4];
      long long at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int x = x0 + i * kT;
        if (x >= items) break;
        if (whole) {
          at[i] = (long long)x * 16;
        } else {
          const int token = x / n_vec, y = x - token * n_vec, head = y / vecs;
          at[i] = token * C.token_b + head * C.head_b + (y - head * vecs) * 16;
        }
        v[i] = *reinterpret_cast<const uint4*>(from + at[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (x0 + i * kT >= items) break;
        *reinterpret_cast<uint4*>(to + at[i]) = v[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Append: blockIdx.y is the sequence, blockIdx.z the layer, one warp a row
// ---------------------------------------------------------------------------
// A warp looks up the pages of its next 32 rows at once (a lane a row), and
// reads a row before it writes the one ahead of it. kIn vectors of K and of V
// a lane.
constexpr int kIn = 4;
__global__ void __launch_bounds__(kT) append_kernel(CacheView C, SeqView S, WindowView W, int layer, int n_layers,
                                                    const char* k_new, const char* v_new, long long new_layer_b,
                                                    long long new_row_b, uint32_t* status) {
  release_stream();
  wait_for_stream();
  k_new = behind_wait(k_new);
  v_new = behind_wait(v_new);
  const int lane = threadIdx.x & 31, vecs = C.head_bytes / 16, n_vec = C.n_heads * vecs;
  const int warp0 = blockIdx.x * (kT / 32) + (threadIdx.x >> 5), step = gridDim.x * (kT / 32);
  const bool whole = C.head_b == C.head_bytes;  // a token's heads lie together
  for (int b = blockIdx.y; b < S.n; b += gridDim.y) {
    const int len = S.ctx[b];
    const Window w = find_window<true>(W, b);
    if (w.rows < 0 || !length_ok(C, S, len)) {
      if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0)
        set_status(status, w.rows < 0 ? SV_DATA_BAD_OFFSETS : SV_DATA_BAD_SEQ);
      continue;
    }
    const int32_t* row = S.table + (long long)b * S.stride;
    for (int l = blockIdx.z; l < n_layers; l += gridDim.z) {
      const char* k_from = k_new + l * new_layer_b + (long long)w.r0 * new_row_b + lane * 16;
      const char* v_from = v_new + (k_from - k_new);
      uint4 kv[2][kIn];
      auto read = [&](int r, int x0) {
        const long long from = (long long)r * new_row_b + (long long)x0 * 16;
#pragma unroll
        for (int j = 0; j < kIn; ++j) {
          if (x0 + j * 32 + lane >= n_vec) break;
          kv[0][j] = ld_once16(k_from + from + j * 512);
          kv[1][j] = ld_once16(v_from + from + j * 512);
        }
      };
      for (long long r0 = warp0; r0 < w.rows; r0 += 32ll * step) {
        read((int)r0, 0);
        const long long mine = r0 + (long long)lane * step;
        long long to = -1;
        if (mine < w.rows) {
          const long long at = len + mine;
          const int slot = at <= 0x7fffffffll ? page_slot(C, (int)at) : S.width;
          const int page = slot < S.width ? row[slot] : -1;
          // A page that others hold too is not written: reserve refused this window.
          if (page >= 0 && page < C.n_pages && C.ref[page] == 1)
            to = (layer + l) * C.layer_b + page * C.page_b + (at - (long long)slot * C.page_size) * C.token_b;
          else
            set_status(status, SV_DATA_BAD_PAGE);
        }
        const int n = (int)min(32ll, (w.rows - r0 + step - 1) / step);
        for (int i = 0; i < n; ++i) {
          const int r = (int)(r0 + (long long)i * step);
          const long long dst = __shfl_sync(kFull, to, i);
          for (int x0 = 0; x0 < n_vec; x0 += kIn * 32) {
            if (x0) read(r, x0);
            uint4 out[2][kIn];
#pragma unroll
            for (int j = 0; j < kIn; ++j) {
              out[0][j] = kv[0][j];
              out[1][j] = kv[1][j];
            }
            if (x0 + kIn * 32 >= n_vec && i + 1 < n) read((int)(r + (long long)step), 0);
            if (dst < 0) continue;
#pragma unroll
            for (int j = 0; j < kIn; ++j) {
              const int x = x0 + j * 32 + lane;
              if (x >= n_vec) break;
              const long long o = dst + (whole ? (long long)x * 16 : (x / vecs) * C.head_b + (x % vecs) * 16);
              *reinterpret_cast<uint4*>(C.k + o) = out[0][j];
              *reinterpret_cast<uint4*>(C.v + o) = out[1][j];
            }
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Commit
// ---------------------------------------------------------------------------
// What request b keeps: `rows` rows from place `begin` of its window.
struct Kept {
  int begin, rows;
  uint32_t bad;
};
__device__ __forceinline__ Kept kept_rows(const CacheView& C, const SeqView& S, const WindowView& W, const int32_t* best,
                                          const int32_t* out_len, int b) {
  // The loads that need nothing first.
  const long long len = S.ctx[b];
  const int c = best ? best[b] : b;
  const bool c_ok = c >= 0 && c < W.n_cand;
  const int n = c_ok ? out_len[c] : 0;
  const int cu0 = c_ok && W.cu ? W.cu[c] : 0, cu1 = c_ok && W.cu ? W.cu[c + 1] : 0;
  const Window w = find_window<true>(W, b);
  if (w.rows < 0) return Kept{0, 0, SV_DATA_BAD_OFFSETS};
  if (!length_ok(C, S, len)) return Kept{0, 0, SV_DATA_BAD_SEQ};
  if (best && c == -1) return Kept{0, 0, 0};
  if (c < w.c0 || c >= w.c1) return Kept{0, 0, SV_DATA_BAD_OFFSETS};
  long long begin = 0, rows = 1;
  if (W.cu) {
    begin = (long long)cu0 + c - w.r0;
    rows = (long long)cu1 + 1 - cu0;
  }
  if (begin < 0 || rows < 1 || begin + rows > w.rows || n < 0 || n > rows) return Kept{0, 0, SV_DATA_BAD_OFFSETS};
  if (n == 0) return Kept{0, 0, 0};
  // Every page from the history's end to the kept rows' must be there, and be this sequence's alone.
  if (!length_ok(C, S, len + begin + n)) return Kept{0, 0, SV_DATA_BAD_PAGE};
  const int32_t* row = S.table + (long long)b * S.stride;
  for (int p = page_slot(C, (int)len), end = page_slot(C, (int)(len + begin + n - 1)); p <= end; ++p)
    if (row[p] < 0 || row[p] >= C.n_pages || C.ref[row[p]] != 1) return Kept{0, 0, SV_DATA_BAD_PAGE};
  return Kept{(int)begin, n, 0};
}

// The kept candidate's rows to the front of the window. A thread owns 16-byte
// columns and walks each upwards, kMove rows at a time, all read before the
// first is written: a row is read before a lower one's place that it lies in
// is written.
constexpr int kMove = 8;
__global__ void __launch_bounds__(kT) move_kernel(CacheView C, SeqView S, WindowView W, const int32_t* best,
                                                  const int32_t* out_len) {
  release_stream();
  wait_for_stream();
  __shared__ long long s_from[kMove], s_to[kMove];
  const int vecs = C.head_bytes / 16;
  const long long cols = 2ll * C.n_layers * C.n_heads * vecs;
  for (int b = blockIdx.y; b < S.n; b += gridDim.y) {
    const Kept kept = kept_rows(C, S, W, best, out_len, b);
    if (kept.bad || kept.begin == 0 || kept.rows == 0) continue;
    const int32_t* row = S.table + (long long)b * S.stride;
    const int len = S.ctx[b];
    for (int j0 = 0; j0 < kept.rows; j0 += kMove) {
      const int n = min(kMove, kept.rows - j0);
      __syncthreads();
      if ((int)threadIdx.x < 2 * n) {
        const int j = threadIdx.x >> 1, t = len + j0 + j + (threadIdx.x & 1 ? 0 : kept.begin), slot = page_slot(C, t);
        (threadIdx.x & 1 ? s_to : s_from)[j] = row[slot] * C.page_b + (t - slot * C.page_size) * C.token_b;
      }
      __syncthreads();
      for (long long x = blockIdx.x * kT + threadIdx.x; x < cols; x += gridDim.x * kT) {
        const int vec = (int)(x % vecs);
        const long long y = x / vecs;
        const int head = (int)(y % C.n_heads), part = (int)(y / C.n_heads);
        char* base = (part & 1 ? C.v : C.k) + (part >> 1) * C.layer_b + head * C.head_b + vec * 16;
        uint4 v[kMove];
#pragma unroll
        for (int j = 0; j < kMove; ++j)
          if (j < n) v[j] = *reinterpret_cast<const uint4*>(base + s_from[j]);
#pragma unroll
        for (int j = 0; j < kMove; ++j)
          if (j < n) *reinterpret_cast<uint4*>(base + s_to[j]) = v[j];
      }
    }
  }
}

// The new length, and the pages behind it released: one warp a request.
__global__ void __launch_bounds__(kT) trim_kernel(CacheView C, SeqView S, WindowView W, const int32_t* best,
                                                  const int32_t* out_len, uint32_t* status) {
  release_stream();
  wait_for_stream();
  const int b = blockIdx.x * (kT / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= S.n) return;
  const Kept kept = kept_rows(C, S, W, best, out_len, b);
  if (kept.bad) {
    if (lane == 0) set_status(status, kept.bad);
    return;
  }
  const int len = S.ctx[b] + kept.rows;
  __syncwarp();
  release_from(C, S, b, pages_of(len, C.page_size), lane, status);
  if (lane == 0) S.ctx[b] = len;
}

inline bool aligned4(const void* p) { return (uintptr_t)p % 4 == 0; }
inline int warps_grid(long long n) {
  const long long g = (n + kT / 32 - 1) / (kT / 32);
  return (int)(g > (1 << 30) ? (1 << 30) : g);
}
template <typename... K, typename... A>
sv_status launch(void (*kernel)(K...), dim3 grid, cudaStream_t st, A... args) {
  return launch_overlapped(kernel, grid, kT, 0, 1, st, args...) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
inline int y_grid(int n) { return n > 32768 ? 32768 : n; }

}  // namespace cache
}  // namespace sv

extern "C" {

sv_status sv_cache_fork(const sv_kv_cache* cache, const sv_sequences* seqs, int32_t N, const int32_t* src,
                        const int32_t* dst, uint32_t* status, void* cuda_stream) {
  using namespace sv;
  CacheView C;
  SeqView S;
  if (!cache_view(cache, &C) || !seq_view(seqs, &S) || N < 0 || !cache::aligned4(status)) return SV_ERR_INVALID_ARG;
  if (N == 0) return SV_OK;
  if (!src || !dst || !cache::aligned4(src) || !cache::aligned4(dst)) return SV_ERR_INVALID_ARG;
  return cache::launch(cache::fork_kernel, dim3((unsigned)cache::warps_grid(N)), static_cast<cudaStream_t>(cuda_stream), C, S, N, src,
                       dst, status);
}

sv_status sv_cache_free(const sv_kv_cache* cache, const sv_sequences* seqs, int32_t N, const int32_t* which,
                        uint32_t* status, void* cuda_stream) {
  using namespace sv;
  CacheView C;
  SeqView S;
  if (!cache_view(cache, &C) || !seq_view(seqs, &S) || N < 0 || !cache::aligned4(status)) return SV_ERR_INVALID_ARG;
  if (N == 0) return SV_OK;
  if (!which || !cache::aligned4(which)) return SV_ERR_INVALID_ARG;
  return cache::launch(cache::free_kernel, dim3((unsigned)cache::warps_grid(N)), static_cast<cudaStream_t>(cuda_stream), C, S, N, which,
                       status);
}

size_t sv_cache_reserve_workspace_size(int32_t n) {
  if (n < 0 || n > SV_CACHE_MAX_SEQS) return 0;
  return 16 + sizeof(sv::cache::CopyJob) * (size_t)n;
}

sv_status sv_cache_reserve(const sv_kv_cache* cache, const sv_sequences* seqs, int32_t n_cand, const int32_t* cu_draft,
                           const int32_t* cu_cand, int32_t* granted, void* workspace, size_t workspace_bytes,
                           uint32_t* status, void* cuda_stream) {
  using namespace sv;
  CacheView C;
  SeqView S;
  WindowView W;
  if (!cache_view(cache, &C) || !seq_view(seqs, &S) || !window_view(S.n, n_cand, cu_draft, cu_cand, 0, &W) ||
      S.n > SV_CACHE_MAX_SEQS || !cache::aligned4(granted) || !cache::aligned4(status))
    return SV_ERR_INVALID_ARG;
  if (S.n == 0) return SV_OK;
  if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < sv_cache_reserve_workspace_size(S.n))
    return SV_ERR_INVALID_ARG;
  W.R = -1;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int smem = 3 * ((S.n + 4) & ~3) * 4;
  static std::atomic<unsigned long long> allowed{0};
  if (allow_smem(cache::reserve_kernel, 3 * 4 * (SV_CACHE_MAX_SEQS + 4), allowed) != cudaSuccess) return SV_ERR_CUDA;
  cache::ReserveWs* ws = static_cast<cache::ReserveWs*>(workspace);
  if (launch_overlapped(cache::reserve_kernel, dim3(1), cache::kR, smem, 1, st, C, S, W, granted, ws, status) != cudaSuccess)
    return SV_ERR_CUDA;
  const long long most = (long long)S.n * C.n_layers * 2;
  return cache::launch(cache::copy_kernel, dim3((unsigned)(most < 152 * 8 ? most : 152 * 8)), st, C,
                             static_cast<const cache::ReserveWs*>(ws));
}

sv_status sv_cache_append(const sv_kv_cache* cache, int32_t layer, int32_t n_layers, const void* k_new, const void* v_new,
                          int64_t new_layer_stride, int64_t new_row_stride, int32_t R, const sv_sequences* seqs,
                          int32_t n_cand, const int32_t* cu_draft, const int32_t* cu_cand, uint32_t* status,
                          void* cuda_stream) {
  using namespace sv;
  CacheView C;
  SeqView S;
  WindowView W;
  if (!cache_view(cache, &C) || !seq_view(seqs, &S) || !window_view(S.n, n_cand, cu_draft, cu_cand, R, &W) ||
      !cache::aligned4(status))
    return SV_ERR_INVALID_ARG;
  if (layer < 0 || n_layers < 0 || layer > C.n_layers - n_layers) return SV_ERR_INVALID_ARG;
  const int es = elem_size(cache->dtype);
  if (new_layer_stride < 0 || new_row_stride < 0 || new_layer_stride > INT64_MAX / 4 || new_row_stride > INT64_MAX / 4 ||
      new_layer_stride * es % 16 || new_row_stride * es % 16)
    return SV_ERR_INVALID_ARG;
  if (S.n == 0 || R == 0 || n_layers == 0) return SV_OK;
  if (!k_new || !v_new || (uintptr_t)k_new % 16 || (uintptr_t)v_new % 16) return SV_ERR_INVALID_ARG;
  // A warp a row of the mean window, up to eight CTAs an SM.
  const int gy = cache::y_grid(S.n), gz = n_layers < 64 ? n_layers : 64;
  const long long gx = (((long long)R + gy - 1) / gy + cache::kT / 32 - 1) / (cache::kT / 32);
  const long long most = (152 * 8 + (long long)gy * gz - 1) / ((long long)gy * gz);
  return cache::launch(cache::append_kernel, dim3((unsigned)(gx < most ? gx : most), gy, gz), static_cast<cudaStream_t>(cuda_stream),
      C, S, W, layer, n_layers, static_cast<const char*>(k_new), static_cast<const char*>(v_new), new_layer_stride * es,
      new_row_stride * es, status);
}

sv_status sv_cache_commit(const sv_kv_cache* cache, const sv_sequences* seqs, int32_t n_cand, const int32_t* cu_draft,
                          const int32_t* cu_cand, const int32_t* best, const int32_t* out_len, uint32_t* status,
                          void* cuda_stream) {
  using namespace sv;
  CacheView C;
  SeqView S;
  WindowView W;
  if (!cache_view(cache, &C) || !seq_view(seqs, &S) || !window_view(S.n, n_cand, cu_draft, cu_cand, 0, &W) ||
      (best == nullptr) != (cu_cand == nullptr) || !cache::aligned4(best) || !cache::aligned4(out_len) ||
      !cache::aligned4(status))
    return SV_ERR_INVALID_ARG;
  if (S.n == 0) return SV_OK;
  if (!out_len) return SV_ERR_INVALID_ARG;
  W.R = -1;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const dim3 trim((unsigned)cache::warps_grid(S.n));
  if (!cu_cand) {  // without candidates the kept rows are in place
    return cache::launch(cache::trim_kernel, trim, st, C, S, W, best, out_len, status);
  }
  const long long cols = 2ll * C.n_layers * C.n_heads * (C.head_bytes / 16);
  const int gy = cache::y_grid(S.n);
  const long long gx = (cols + cache::kT - 1) / cache::kT, most = (152 * 8 + gy - 1) / gy;
  const sv_status moved = cache::launch(cache::move_kernel, dim3((unsigned)(gx < most ? gx : most), gy), st, C, S, W, best, out_len);
  if (moved != SV_OK) return moved;
  return cache::launch(cache::trim_kernel, trim, st, C, S, W, best, out_len, status);
}

}  // extern "C"
