// cache.cu -- the pages of a key-value cache around the verify step: fork,
// free, reserve (with the copy of shared partial pages), append, commit.
//
// Free pages are bits, not a stack: whoever releases a page only sets its
// bit when the count falls to zero, and the allocator takes the lowest set
// bits in the order of the sequences. Both are independent of timing, so the
// page tables are the same from run to run.
#include "sv_cache.cuh"

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
  for (int k = lane; k < n; k += 32) good &= from[k] >= 0 && from[k] < C.n_pages;
  if (!__all_sync(kFull, good)) {
    if (lane == 0) set_status(status, SV_DATA_BAD_PAGE);
    return;
  }
  for (int k = lane; k < n; k += 32) {
    const int page = from[k];
    to[k] = page;
    if (atomicAdd(&C.ref[page], 1) < 1) set_status(status, SV_DATA_BAD_PAGE);
  }
  if (lane == 0) S.ctx[d] = len;
}

__global__ void __launch_bounds__(kT) free_kernel(CacheView C, SeqView S, int N, const int32_t* which, uint32_t* status) {
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

// One CTA: needs, the order among the sharers of a partial page, a scan, and
// the lowest free bits. Shared memory: three words a sequence.
__global__ void __launch_bounds__(kR) reserve_kernel(CacheView C, SeqView S, WindowView W, int32_t* granted, ReserveWs* ws,
                                                     uint32_t* status) {
  extern __shared__ int s_mem[];
  int* s_first = s_mem;            // needs, then their exclusive scan [n + 1]
  int* s_have = s_mem + S.n + 1;   // pages held * 2 + 1 if the partial page is copied; -1: refused
  int* s_part = s_have + S.n;      // the shared partial page, or -1
  __shared__ int s_warp[32];
  __shared__ int s_jobs, s_end;
  const int tid = threadIdx.x, n_words = (C.n_pages + 31) / 32;
  if (tid == 0) {
    s_jobs = 0;
    s_end = INT_MAX;
  }
  for (int b = tid; b < S.n; b += kR) {
    const Window w = find_window(W, b);
    const long long len = S.ctx[b];
    const int32_t* row = S.table + (long long)b * S.stride;
    int have = -1, need = 0, part = -1;
    uint32_t bad = 0;
    if (w.rows < 0)
      bad = SV_DATA_BAD_OFFSETS;
    else if (!length_ok(C, S, len))
      bad = SV_DATA_BAD_SEQ;
    else if (w.rows > 0 && !length_ok(C, S, len + w.rows))
      bad = SV_DATA_BAD_PAGE;
    else {
      const int want = pages_of(len + w.rows, C.page_size);
      have = pages_of(len, C.page_size);
      while (have < S.width && row[have] >= 0) ++have;  // reserved before
      need = max(0, want - have);
      if (w.rows > 0 && len % C.page_size) {
        part = row[len / C.page_size];
        if (part < 0 || part >= C.n_pages || C.ref[part] < 1) {
          bad = SV_DATA_BAD_PAGE;
          have = -1;
          need = 0;
          part = -1;
        } else if (C.ref[part] == 1)
          part = -1;
      }
    }
    if (bad) set_status(status, bad);
    s_first[b] = need;
    s_have[b] = have;
    s_part[b] = part;
  }
  __syncthreads();
  // Who copies: a sharer, unless those before it in this call leave it alone with the page.
  for (int b = tid; b < S.n; b += kR) {
    const int part = s_part[b];
    if (part < 0) {
      s_have[b] = s_have[b] < 0 ? -1 : s_have[b] * 2;
      continue;
    }
    int before = 0;
    for (int j = 0; j < b; ++j) before += s_part[j] == part;
    const int left = C.ref[part] - before;
    if (left < 1) {  // more sharers than the count says
      set_status(status, SV_DATA_BAD_PAGE);
      s_have[b] = -1;
      s_first[b] = 0;
    } else {
      s_have[b] = s_have[b] * 2 + (left > 1);
      s_first[b] += left > 1;
    }
  }
  __syncthreads();
  int total = 0;
  for (int b0 = 0; b0 < S.n; b0 += kR) {
    const int b = b0 + tid, v = b < S.n ? s_first[b] : 0;
    int sum;
    const int at = total + block_excl_scan(v, s_warp, sum);
    if (b < S.n) s_first[b] = at;
    total += sum;
  }
  if (tid == 0) s_first[S.n] = total;
  __syncthreads();
  // Free pages, as far as they are asked for.
  int avail = 0;
  for (int w0 = 0; w0 < n_words && avail < total; w0 += kR) {
    const int w = w0 + tid;
    int sum;
    block_excl_scan(w < n_words ? __popc(C.free_bits[w]) : 0, s_warp, sum);
    avail += sum;
  }
  if (avail < total) {
    for (int b = tid; b < S.n; b += kR)
      if (s_first[b + 1] > s_first[b] && s_first[b + 1] > avail) atomicMin(&s_end, b);
    __syncthreads();
    if (tid == 0) set_status(status, SV_DATA_NO_PAGES);
    total = s_first[s_end];
  }
  const int end = s_end;
  __syncthreads();
  for (int b = tid; b < S.n; b += kR) {
    const bool late = b >= end && (s_first[b + 1] > s_first[b] || s_part[b] >= 0);
    if (late) s_have[b] = -1;
    if (granted) granted[b] = s_have[b] >= 0 ? find_window(W, b).rows : 0;
  }
  __syncthreads();
  // The k-th lowest free page goes to the request whose range of the scan holds k.
  int taken = 0;
  for (int w0 = 0; w0 < n_words && taken < total; w0 += kR) {
    const int w = w0 + tid;
    uint32_t bits = w < n_words ? C.free_bits[w] : 0u;
    int sum;
    int k = taken + block_excl_scan(__popc(bits), s_warp, sum);
    taken += sum;
    uint32_t left = bits;
    for (; left && k < total; ++k) {
      const int bit = __ffs(left) - 1;
      left &= left - 1;
      const int page = w * 32 + bit;
      int lo = 0, hi = S.n;  // the last request that begins at or before k
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_first[mid] <= k)
          lo = mid;
        else
          hi = mid;
      }
      const int i = k - s_first[lo], have = s_have[lo] >> 1, copy = s_have[lo] & 1;
      int32_t* row = S.table + (long long)lo * S.stride;
      C.ref[page] = 1;
      if (copy && i == 0) {
        const int len = S.ctx[lo], at = len / C.page_size, old = row[at];
        row[at] = page;
        atomicSub(&C.ref[old], 1);
        ws->jobs[atomicAdd(&s_jobs, 1)] = CopyJob{old, page, len % C.page_size, 0};
      } else {
        row[have + i - copy] = page;
      }
    }
    if (left != bits) C.free_bits[w] = left;
  }
  __syncthreads();
  if (tid == 0) ws->n_jobs = s_jobs;
}

// The copies that reserve asked for: one warp a (job, layer, K or V, token).
__global__ void __launch_bounds__(kT) copy_kernel(CacheView C, const ReserveWs* ws) {
  const int lane = threadIdx.x & 31;
  const long long warp = blockIdx.x * (long long)(kT / 32) + (threadIdx.x >> 5);
  const long long step = gridDim.x * (long long)(kT / 32);
  const int vecs = C.head_bytes / 16;
  const long long n = (long long)ws->n_jobs * C.n_layers * 2 * C.page_size;
  for (long long u = warp; u < n; u += step) {
    const int token = (int)(u % C.page_size);
    const long long rest = u / C.page_size;
    const int kv = (int)(rest & 1), layer = (int)((rest >> 1) % C.n_layers);
    const CopyJob j = ws->jobs[(rest >> 1) / C.n_layers];
    if (token >= j.tokens) continue;
    char* base = (kv ? C.v : C.k) + layer * C.layer_b + token * C.token_b;
    const char* from = base + j.from * C.page_b;
    char* to = base + j.to * C.page_b;
    for (int x = lane; x < C.n_heads * vecs; x += 32) {
      const long long at = (x / vecs) * C.head_b + (x % vecs) * 16;
      *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(from + at);
    }
  }
}

// ---------------------------------------------------------------------------
// Append: blockIdx.y is the sequence, blockIdx.z the layer, one warp a row
// ---------------------------------------------------------------------------
// A warp's next row is read before its page is looked up: the row's bytes and
// the two lookups are in flight together. kIn vectors of K and of V a lane.
constexpr int kIn = 4;
__global__ void __launch_bounds__(kT) append_kernel(CacheView C, SeqView S, WindowView W, int layer, int n_layers,
                                                    const char* k_new, const char* v_new, long long new_layer_b,
                                                    long long new_row_b, uint32_t* status) {
  const int lane = threadIdx.x & 31, vecs = C.head_bytes / 16, n_vec = C.n_heads * vecs;
  const bool whole = C.head_b == C.head_bytes;  // a token's heads lie together
  for (int b = blockIdx.y; b < S.n; b += gridDim.y) {
    const Window w = find_window(W, b);
    const int len = S.ctx[b];
    if (w.rows < 0 || !length_ok(C, S, len)) {
      if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0)
        set_status(status, w.rows < 0 ? SV_DATA_BAD_OFFSETS : SV_DATA_BAD_SEQ);
      continue;
    }
    const int32_t* row = S.table + (long long)b * S.stride;
    for (int l = blockIdx.z; l < n_layers; l += gridDim.z) {
      for (int r = blockIdx.x * (kT / 32) + (threadIdx.x >> 5); r < w.rows; r += gridDim.x * (kT / 32)) {
        const long long from = l * new_layer_b + (long long)(w.r0 + r) * new_row_b;
        uint4 kv[2][kIn];
#pragma unroll
        for (int j = 0; j < kIn; ++j) {
          const int x = j * 32 + lane;
          if (x < n_vec) {
            kv[0][j] = ld_stream16(k_new + from + (long long)x * 16);
            kv[1][j] = ld_stream16(v_new + from + (long long)x * 16);
          }
        }
        const long long at = (long long)len + r;
        const int slot = at <= 0x7fffffffll ? page_slot(C, (int)at) : S.width;
        const int page = slot < S.width ? row[slot] : -1;
        // A page that others hold too is not written: reserve refused this window.
        if (page < 0 || page >= C.n_pages || C.ref[page] != 1) {
          if (lane == 0) set_status(status, SV_DATA_BAD_PAGE);
          continue;
        }
        const long long to = (layer + l) * C.layer_b + page * C.page_b + (at - (long long)slot * C.page_size) * C.token_b;
        for (int x0 = 0; x0 < n_vec; x0 += kIn * 32) {
#pragma unroll
          for (int j = 0; j < kIn; ++j) {
            const int x = x0 + j * 32 + lane;
            if (x >= n_vec) break;
            if (x0) {
              kv[0][j] = ld_stream16(k_new + from + (long long)x * 16);
              kv[1][j] = ld_stream16(v_new + from + (long long)x * 16);
            }
            const long long o = to + (whole ? (long long)x * 16 : (x / vecs) * C.head_b + (x % vecs) * 16);
            *reinterpret_cast<uint4*>(C.k + o) = kv[0][j];
            *reinterpret_cast<uint4*>(C.v + o) = kv[1][j];
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
  const Window w = find_window(W, b);
  if (w.rows < 0) return Kept{0, 0, SV_DATA_BAD_OFFSETS};
  const long long len = S.ctx[b];
  if (!length_ok(C, S, len)) return Kept{0, 0, SV_DATA_BAD_SEQ};
  const int c = best ? best[b] : b;
  if (best && c == -1) return Kept{0, 0, 0};
  if (c < w.c0 || c >= w.c1) return Kept{0, 0, SV_DATA_BAD_OFFSETS};
  const int n = out_len[c];
  long long begin = 0, rows = 1;
  if (W.cu) {
    begin = (long long)W.cu[c] + c - w.r0;
    rows = (long long)W.cu[c + 1] + 1 - W.cu[c];
  }
  if (begin < 0 || rows < 1 || begin + rows > w.rows || n < 0 || n > rows) return Kept{0, 0, SV_DATA_BAD_OFFSETS};
  if (n == 0) return Kept{0, 0, 0};
  // Every page from the history's end to the kept rows' must be there, and be this sequence's alone.
  if (!length_ok(C, S, len + begin + n)) return Kept{0, 0, SV_DATA_BAD_PAGE};
  const int32_t* row = S.table + (long long)b * S.stride;
  for (long long p = len / C.page_size; p <= (len + begin + n - 1) / C.page_size; ++p)
    if (row[p] < 0 || row[p] >= C.n_pages || C.ref[row[p]] != 1) return Kept{0, 0, SV_DATA_BAD_PAGE};
  return Kept{(int)begin, n, 0};
}

// The kept candidate's rows to the front of the window. A thread owns one
// 16-byte column and walks it upwards: a row is read before a lower one's
// place that it lies in is written.
__global__ void __launch_bounds__(kT) move_kernel(CacheView C, SeqView S, WindowView W, const int32_t* best,
                                                  const int32_t* out_len) {
  const int vecs = C.head_bytes / 16;
  const long long cols = 2ll * C.n_layers * C.n_heads * vecs;
  for (int b = blockIdx.y; b < S.n; b += gridDim.y) {
    const Kept kept = kept_rows(C, S, W, best, out_len, b);
    if (kept.bad || kept.begin == 0 || kept.rows == 0) continue;
    const int32_t* row = S.table + (long long)b * S.stride;
    const long long len = S.ctx[b];
    for (long long x = blockIdx.x * kT + threadIdx.x; x < cols; x += gridDim.x * kT) {
      const int vec = (int)(x % vecs);
      const long long y = x / vecs;
      const int head = (int)(y % C.n_heads);
      const int layer = (int)(y / C.n_heads) >> 1;
      char* base = ((y / C.n_heads) & 1 ? C.v : C.k) + layer * C.layer_b + head * C.head_b + vec * 16;
      for (int j = 0; j < kept.rows; ++j) {
        const long long a = len + kept.begin + j, d = len + j;
        const char* from = base + row[a / C.page_size] * C.page_b + (a % C.page_size) * C.token_b;
        char* to = base + row[d / C.page_size] * C.page_b + (d % C.page_size) * C.token_b;
        *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
      }
    }
  }
}

// The new length, and the pages behind it released: one warp a request.
__global__ void __launch_bounds__(kT) trim_kernel(CacheView C, SeqView S, WindowView W, const int32_t* best,
                                                  const int32_t* out_len, uint32_t* status) {
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
inline sv_status launched() { return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA; }
inline int warps_grid(long long n) {
  const long long g = (n + kT / 32 - 1) / (kT / 32);
  return (int)(g > (1 << 30) ? (1 << 30) : g);
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
  cache::fork_kernel<<<cache::warps_grid(N), cache::kT, 0, static_cast<cudaStream_t>(cuda_stream)>>>(C, S, N, src, dst,
                                                                                                    status);
  return cache::launched();
}

sv_status sv_cache_free(const sv_kv_cache* cache, const sv_sequences* seqs, int32_t N, const int32_t* which,
                        uint32_t* status, void* cuda_stream) {
  using namespace sv;
  CacheView C;
  SeqView S;
  if (!cache_view(cache, &C) || !seq_view(seqs, &S) || N < 0 || !cache::aligned4(status)) return SV_ERR_INVALID_ARG;
  if (N == 0) return SV_OK;
  if (!which || !cache::aligned4(which)) return SV_ERR_INVALID_ARG;
  cache::free_kernel<<<cache::warps_grid(N), cache::kT, 0, static_cast<cudaStream_t>(cuda_stream)>>>(C, S, N, which,
                                                                                                    status);
  return cache::launched();
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
  const int smem = (3 * S.n + 1) * 4;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(cache::reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return SV_ERR_CUDA;
  cache::ReserveWs* ws = static_cast<cache::ReserveWs*>(workspace);
  cache::reserve_kernel<<<1, cache::kR, smem, st>>>(C, S, W, granted, ws, status);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  const int most = cache::warps_grid((long long)S.n * C.n_layers * 2 * C.page_size);
  cache::copy_kernel<<<most < 152 * 8 ? most : 152 * 8, cache::kT, 0, st>>>(C, ws);
  return cache::launched();
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
  const long long gx = ((R + gy - 1) / gy + cache::kT / 32 - 1) / (cache::kT / 32);
  const long long most = (152 * 8 + (long long)gy * gz - 1) / ((long long)gy * gz);
  cache::append_kernel<<<dim3((unsigned)(gx < most ? gx : most), gy, gz), cache::kT, 0, static_cast<cudaStream_t>(cuda_stream)>>>(
      C, S, W, layer, n_layers, static_cast<const char*>(k_new), static_cast<const char*>(v_new), new_layer_stride * es,
      new_row_stride * es, status);
  return cache::launched();
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
  if (cu_cand) {  // without candidates the kept rows are in place
    const long long cols = 2ll * C.n_layers * C.n_heads * (C.head_bytes / 16);
    const int gy = cache::y_grid(S.n);
    const long long gx = (cols + cache::kT - 1) / cache::kT, most = (152 * 8 + gy - 1) / gy;
    cache::move_kernel<<<dim3((unsigned)(gx < most ? gx : most), gy), cache::kT, 0, st>>>(C, S, W, best, out_len);
    if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  }
  cache::trim_kernel<<<cache::warps_grid(S.n), cache::kT, 0, st>>>(C, S, W, best, out_len, status);
  return cache::launched();
}

}  // extern "C"
