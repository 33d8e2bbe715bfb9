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
  float scale_log2;  // scale * log2(e); for the tensor core kernel its absolute value, and
  uint32_t q_sign;   // the bits that turn q's sign; with a scale of zero q is
  uint32_t q_mask;   // masked to zero and scaled by one
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


// ---------------------------------------------------------------------------
// bf16: tensor cores over a paged pipeline
// ---------------------------------------------------------------------------
constexpr int kTK = 64;    // tokens of a key tile

// How the work is cut. A unit is a (request, key-value head, tile of MT
// stacked rows); stacked row i of a window is window row i / group, query
// head i % group of the head's group. Its key tiles follow one another in a
// list of all units' tiles, of which every CTA takes an equal, contiguous
// share: a long request is spread over many CTAs, short ones share one. A
// unit that a share's end cuts leaves partial results, joined by
// join_kernel.
struct Plan {
  char* part;          // partial results: two slots a CTA
  int* cut;            // [grid][4]: the unit that a CTA's share cuts at its end: b, head, row tile, its last CTA (b = -1: none)
  uint32_t div_mul, div_shift;  // t / page_size
};

struct Unit {
  int b, head, mt;     // request, key-value head, row tile
  int keys, tiles;     // tokens, key tiles
  Window w;
  int n_mt, ctx;
};

__device__ __forceinline__ int div_page(const Plan& L, uint32_t t) {
  return (int)(((unsigned long long)t * L.div_mul) >> L.div_shift);
}

// Request b's window, tokens and key tiles, and its number of row tiles (0 tiles where there is nothing to do).
template <int MT>
__device__ __forceinline__ void load_request(const Params& P, int b, Unit& u, bool tell) {
  u.b = b;
  u.w = find_window(P.W, b);
  u.ctx = P.S.ctx[b];
  const bool len = length_ok(P.C, P.S, u.ctx), fits = len && length_ok(P.C, P.S, (long long)u.ctx + max(u.w.rows, 0));
  if (u.w.rows <= 0 || !fits) {
    if (tell && (u.w.rows < 0 || !fits))
      set_status(P.status, u.w.rows < 0 ? SV_DATA_BAD_OFFSETS : len ? SV_DATA_BAD_PAGE : SV_DATA_BAD_SEQ);
    u.keys = u.tiles = u.n_mt = 0;
    return;
  }
  if (tell && P.W.cand)
    for (int c = u.w.c0; c < u.w.c1; ++c)
      if (P.W.cu[c + 1] < P.W.cu[c]) set_status(P.status, SV_DATA_BAD_OFFSETS);
  u.keys = u.ctx + u.w.rows;
  u.tiles = (u.keys + kTK - 1) / kTK;
  u.n_mt = (int)(((long long)u.w.rows * P.group + MT - 1) / MT);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// What sums about maximum m count for about maximum top >= m. The sums' terms
// are 2^(s scale - fl(m scale)), so the rounded products are what differs.
__device__ __forceinline__ float factor(float m, float top, float scale) {
  return m == -INFINITY ? 0.f : ex2(__fmul_rn(m, scale) - __fmul_rn(top, scale));
}
__device__ __forceinline__ float lse_of(float m, float l, float scale) {
  return l > 0.f ? (__fmul_rn(m, scale) + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Bytes of one partial result: MT rows of D sums, then their maxima and sums.
template <int D, int MT>
constexpr size_t part_bytes() {
  return (size_t)MT * (D + 2) * 4;
}

template <int D, int WM>
struct Shape {
  static constexpr int MT = 16 * WM;            // stacked rows of a unit
  static constexpr int WK = WM < 4 ? 4 / WM : 1;  // warps that split a key tile
  static constexpr int kT = 32 * WM * WK;       // threads
  static constexpr int KW = kTK / WK;           // tokens of a tile for one warp
  static constexpr int KS = KW < 32 ? KW : 32;  // tokens that go through the softmax at once
  static constexpr int kCtas = D == 64 && WM == 4 ? 3 : D == 128 && WM == 8 ? 1 : 2;  // an SM
  static constexpr int kStages = D == 128 ? (WM == 8 ? 5 : 3) : (WM == 4 ? 4 : 6);
  static constexpr int kTile = kTK * D * 2;     // bytes of K (or V) of a tile
  static constexpr size_t smem = (size_t)kStages * 2 * kTile + (kStages + 1) * (kTK * 8 + 16);
  // The warps that split the keys join in the stage that they have just used.
  static_assert(WK == 1 || (WK / 2) * MT * (D + 4) * 4 <= 2 * kTile, "a stage holds the results of half the warps");
};

// The address of 16-byte chunk c of row r of a tile: chunks are permuted within their row so that eight rows of one column lie
// in different banks.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

template <int D, int WM>
__global__ void __launch_bounds__(Shape<D, WM>::kT, Shape<D, WM>::kCtas) window_mma_kernel(Params P, Plan L) {
  using Sh = Shape<D, WM>;
  constexpr int kTW = Sh::kT, KS = Sh::KS;
  constexpr int MT = Sh::MT, WK = Sh::WK, KW = Sh::KW, S = Sh::kStages;
  constexpr int ND = D / 8;    // n-tiles of the output
  constexpr int KD = D / 16;   // k-steps of a score
  constexpr int CPR = D / 8;   // 16-byte chunks of a row
  constexpr int RPP = kTW / CPR;  // rows that the CTA copies at once
  extern __shared__ __align__(1024) char smem[];
  char* s_kv = smem;
  long long* s_off = reinterpret_cast<long long*>(smem + S * 2 * Sh::kTile);  // [S + 1][kTK]
  uint32_t* s_valid = reinterpret_cast<uint32_t*>(s_off + (S + 1) * kTK);                  // [S + 1][4]
  __shared__ long long s_scan[kTW / 32];
  __shared__ int s_start[2];
  __shared__ long long s_first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp % WM, wk = warp / WM;

  // This CTA's share. Thread i sums the tiles of its run of requests; a scan over the threads, and the thread whose run holds
  // the first tile of the share walks it.
  const int per = (P.S.n + kTW - 1) / kTW;
  long long mine = 0;
  for (int b = tid * per; b < min((tid + 1) * per, P.S.n); ++b) {
    Unit u;
    load_request<MT>(P, b, u, blockIdx.x == 0);
    mine += (long long)u.tiles * u.n_mt * P.C.n_heads;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < kTW / 32; ++w) {
    if (w < warp) incl += s_scan[w];
    total += s_scan[w];
  }
  const int grid = (int)min((long long)gridDim.x, total);  // shares of a tile at least
  if (blockIdx.x >= grid) {
    if (tid == 0) L.cut[blockIdx.x * 4] = -1;
    return;
  }
  const long long t0 = total * blockIdx.x / grid, t1 = total * (blockIdx.x + 1) / grid;
  if (t0 >= incl - mine && t0 < incl) {
    long long at = incl - mine;
    Unit u;
    int b = tid * per;
    for (;; ++b) {
      load_request<MT>(P, b, u, false);
      const long long n = (long long)u.tiles * u.n_mt * P.C.n_heads;
      if (t0 < at + n) break;
      at += n;
    }
    s_start[0] = b;
    s_first = t0 - at;  // first tile of the share within its request
  }
  __syncthreads();

  // Two cursors over the share: one loads, one computes.
  struct Cursor {
    Unit u;
    int tile;
  };
  auto begin = [&](Cursor& c) {
    load_request<MT>(P, s_start[0], c.u, false);
    const long long first = s_first;
    const long long unit = first / c.u.tiles;
    c.tile = (int)(first - unit * c.u.tiles);
    c.u.head = (int)(unit / c.u.n_mt);
    c.u.mt = (int)(unit - (long long)c.u.head * c.u.n_mt);
  };
  auto next_unit = [&](Cursor& c) {  // false past the last request
    c.tile = 0;
    if (++c.u.mt < c.u.n_mt) return;
    c.u.mt = 0;
    if (++c.u.head < P.C.n_heads) return;
    c.u.head = 0;
    int b = c.u.b + 1;
    for (; b < P.S.n; ++b) {
      load_request<MT>(P, b, c.u, false);
      if (c.u.tiles) return;
    }
  };
  const int n_tiles = (int)(t1 - t0);
  Cursor ld, cp;
  begin(ld);
  cp = ld;

  // Page lookups run one tile ahead of the copies: threads 0 .. kTK - 1 hold a token each. The byte offset of a token in K and
  // V, or -1 where it has no page or lies behind the sequence.
  auto lookup = [&](const Cursor& c, int& page, int& place) {  // issued early
    const int t = c.tile * kTK + tid;
    page = -2;
    place = 0;
    if (tid < kTK && t < c.u.keys) {
      const int slot = div_page(L, t);
      place = t - slot * P.C.page_size;
      page = P.S.table[(long long)c.u.b * P.S.stride + slot];
    }
  };
  auto store_lookup = [&](int ring, int head, int page, int place) {
    if (tid < kTK) {
      const bool ok = page >= 0 && page < P.C.n_pages;
      if (!ok && page != -2) set_status(P.status, SV_DATA_BAD_PAGE);
      s_off[ring * kTK + tid] = ok ? page * P.C.page_b + place * P.C.token_b + head * P.C.head_b : -1;
      const unsigned m = __ballot_sync(kFull, ok);
      if (lane == 0) s_valid[ring * 4 + warp] = m;
    }
  };
  auto copy_tile = [&](int ring, int stage) {
    const uint32_t base = smem_addr(s_kv) + stage * 2 * Sh::kTile;
    const int c = tid % CPR;
#pragma unroll
    for (int i = 0; i < kTK / RPP; ++i) {
      const int r = tid / CPR + i * RPP;
      const long long off = s_off[ring * kTK + r];
      const bool ok = off >= 0;
      const long long at = (ok ? off : 0) + c * 16;
      cp16(base + swz<D>(r, c), P.C.k + at, ok);
      cp16(base + Sh::kTile + swz<D>(r, c), P.C.v + at, ok);
    }
  };

  // The first S - 1 tiles, and the lookup behind them: all S table loads before the first is used.
  int page, place;
  {
    int pages[S], places[S], heads[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (i < n_tiles) {
        lookup(ld, pages[i], places[i]);
        heads[i] = ld.u.head;
        if (i + 1 < n_tiles && ++ld.tile == ld.u.tiles) next_unit(ld);
      }
    }
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (i < n_tiles) store_lookup(i, heads[i], pages[i], places[i]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    if (i < n_tiles) copy_tile(i, i);
    cp_commit();
  }

  float o[ND][4], m_run[2], l_run[2];
  uint32_t q[KD][4];
  int lo[2], hi[2];  // the window places that the thread's two rows see
  bool begun = false, from_start = false;
  const int row0 = wm * 16 + (lane >> 2);  // and row0 + 8

  for (int i = 0; i < n_tiles; ++i) {
    const bool ahead = i + S < n_tiles;
    if (ahead) lookup(ld, page, place);

    if (!begun) {  // a new unit: its rows
      begun = true;
      from_start = cp.tile == 0;
      const int rows = cp.u.w.rows * P.group;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int x = cp.u.mt * MT + row0 + e * 8;
        const bool ok = x < rows;
        const int w = ok ? x / P.group : 0, h = ok ? x - w * P.group : 0;
        lo[e] = 0;
        hi[e] = ok ? w : -1 - cp.u.ctx;  // rows past the window see nothing
        if (ok && P.W.cand) {  // the first row of the row's candidate
          int a = cp.u.w.c0, z = cp.u.w.c1;
          while (z - a > 1) {
            const int mid = (a + z) >> 1;
            if ((long long)P.W.cu[mid] + mid - cp.u.w.r0 <= w)
              a = mid;
            else
              z = mid;
          }
          const long long at = (long long)P.W.cu[a] + a - cp.u.w.r0;
          lo[e] = at < 0 || at > w ? w : (int)at;
        }
        const uint32_t* src = reinterpret_cast<const uint32_t*>(P.q + (long long)(cp.u.w.r0 + w) * P.q_row_b +
                                                                (long long)(cp.u.head * P.group + h) * (D * 2)) + (lane & 3);
#pragma unroll
        for (int k = 0; k < KD; ++k) {
          q[k][e] = ok ? (__ldg(src + k * 8) & P.q_mask) ^ P.q_sign : 0u;
          q[k][e + 2] = ok ? (__ldg(src + k * 8 + 4) & P.q_mask) ^ P.q_sign : 0u;
        }
        m_run[e] = -INFINITY;
        l_run[e] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    }

    cp_wait<S - 2>();
    __syncthreads();  // tile i has landed, the ring's next lookup is there, stage (i - 1) is free
    if (i + S - 1 < n_tiles) copy_tile((i + S - 1) % (S + 1), (i + S - 1) % S);
    cp_commit();

    const uint32_t kb = smem_addr(s_kv) + (i % S) * 2 * Sh::kTile, vb = kb + Sh::kTile;
    const int ring = i % (S + 1);
    const bool masked = (cp.tile + 1) * kTK > cp.u.ctx || (s_valid[ring * 4] & s_valid[ring * 4 + 1]) != 0xffffffffu;
#pragma unroll
    for (int key0 = wk * KW; key0 < (wk + 1) * KW; key0 += KS) {
      float s[KS / 8][4];
#pragma unroll
      for (int n = 0; n < KS / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
      for (int k = 0; k < KD; ++k) {
#pragma unroll
        for (int n = 0; n < KS / 8; n += 2) {
          uint32_t b[4];  // tokens n*8 .. +7 at d k*16 and +8, then tokens +8 .. +15
          const int r = key0 + n * 8 + (lane & 7) + ((lane >> 4) << 3), c = k * 2 + ((lane >> 3) & 1);
          ldsm4(b, kb + swz<D>(r, c));
          mma_bf16(s[n], q[k], b[0], b[1]);
          mma_bf16(s[n + 1], q[k], b[2], b[3]);
        }
      }
      // Hidden tokens: behind the history all but the row's part of the window, and those without a page.
      if (masked) {
        const uint32_t word = s_valid[ring * 4 + (key0 >> 5)];
#pragma unroll
        for (int n = 0; n < KS / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kk = key0 + n * 8 + (lane & 3) * 2 + (e & 1);
            const int at = cp.tile * kTK + kk - cp.u.ctx;
            const bool see = (at < 0 ? hi[e >> 1] >= -cp.u.ctx : at >= lo[e >> 1] && at <= hi[e >> 1]) && (word >> (kk & 31) & 1u);
            if (!see) s[n][e] = -INFINITY;
          }
      }
      float m_new[2] = {m_run[0], m_run[1]};
#pragma unroll
      for (int n = 0; n < KS / 8; ++n) {
        m_new[0] = fmaxf(m_new[0], fmaxf(s[n][0], s[n][1]));
        m_new[1] = fmaxf(m_new[1], fmaxf(s[n][2], s[n][3]));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_new[e] = fmaxf(m_new[e], __shfl_xor_sync(kFull, m_new[e], 1));
        m_new[e] = fmaxf(m_new[e], __shfl_xor_sync(kFull, m_new[e], 2));
      }
      if (__any_sync(kFull, m_new[0] != m_run[0] || m_new[1] != m_run[1])) {
        const float f0 = factor(m_run[0], m_new[0], P.scale_log2), f1 = factor(m_run[1], m_new[1], P.scale_log2);
#pragma unroll
        for (int n = 0; n < ND; ++n) {
          o[n][0] *= f0;
          o[n][1] *= f0;
          o[n][2] *= f1;
          o[n][3] *= f1;
        }
        l_run[0] *= f0;
        l_run[1] *= f1;
        m_run[0] = m_new[0];
        m_run[1] = m_new[1];
      }
      // A row that has seen nothing yet keeps -inf scores: with an offset of 0 their weights are 0.
      const float off0 = m_run[0] == -INFINITY ? 0.f : __fmul_rn(m_run[0], P.scale_log2);
      const float off1 = m_run[1] == -INFINITY ? 0.f : __fmul_rn(m_run[1], P.scale_log2);
      uint32_t pa[KS / 16][4];
#pragma unroll
      for (int n = 0; n < KS / 8; ++n) {
        const float p0 = ex2(fmaf(s[n][0], P.scale_log2, -off0)), p1 = ex2(fmaf(s[n][1], P.scale_log2, -off0));
        const float p2 = ex2(fmaf(s[n][2], P.scale_log2, -off1)), p3 = ex2(fmaf(s[n][3], P.scale_log2, -off1));
        l_run[0] += p0 + p1;
        l_run[1] += p2 + p3;
        pa[n / 2][(n & 1) * 2] = pack_bf16(p0, p1);
        pa[n / 2][(n & 1) * 2 + 1] = pack_bf16(p2, p3);
      }
#pragma unroll
      for (int k = 0; k < KS / 16; ++k) {
#pragma unroll
        for (int n = 0; n < ND; n += 2) {
          uint32_t b[4];  // tokens k*16 .. +7 and +8 .. +15 at d n*8, then at d n*8 + 8
          const int r = key0 + k * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), c = n + (lane >> 4);
          ldsm4t(b, vb + swz<D>(r, c));
          mma_bf16(o[n], pa[k], b[0], b[1]);
          mma_bf16(o[n + 1], pa[k], b[2], b[3]);
        }
      }
    }

    if (ahead) {
      store_lookup((i + S) % (S + 1), ld.u.head, page, place);
      if (i + S + 1 < n_tiles && ++ld.tile == ld.u.tiles) next_unit(ld);
    }

    // The unit's end, or the share's: join the warps that split the keys, then write.
    const bool unit_end = cp.tile + 1 == cp.u.tiles;
    if (unit_end || i + 1 == n_tiles) {
      begun = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l_run[e] += __shfl_xor_sync(kFull, l_run[e], 1);
        l_run[e] += __shfl_xor_sync(kFull, l_run[e], 2);
      }
      if constexpr (WK > 1) {
        float* s_merge = reinterpret_cast<float*>(s_kv + (i % S) * 2 * Sh::kTile);
        __syncthreads();  // every warp is through with the stage
#pragma unroll
        for (int half = WK / 2; half > 0; half >>= 1) {
          float* buf = s_merge + ((size_t)(wk % half) * MT + wm * 16) * (D + 4);
          if (wk >= half && wk < 2 * half) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float* row = buf + ((lane >> 2) + e * 8) * (D + 4);
#pragma unroll
              for (int n = 0; n < ND; ++n) *reinterpret_cast<float2*>(row + n * 8 + (lane & 3) * 2) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
              if ((lane & 3) == 0) *reinterpret_cast<float2*>(row + D) = make_float2(m_run[e], l_run[e]);
            }
          }
          __syncthreads();
          if (wk < half) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float* row = buf + ((lane >> 2) + e * 8) * (D + 4);
              const float2 ml = *reinterpret_cast<const float2*>(row + D);
              const float m = fmaxf(m_run[e], ml.x);
              const float fa = factor(m_run[e], m, P.scale_log2), fb = factor(ml.x, m, P.scale_log2);
              m_run[e] = m;
              l_run[e] = l_run[e] * fa + ml.y * fb;
#pragma unroll
              for (int n = 0; n < ND; ++n) {
                const float2 x = *reinterpret_cast<const float2*>(row + n * 8 + (lane & 3) * 2);
                o[n][2 * e] = o[n][2 * e] * fa + x.x * fb;
                o[n][2 * e + 1] = o[n][2 * e + 1] * fa + x.y * fb;
              }
            }
          }
          __syncthreads();
        }
      }
      const bool split = !from_start || !unit_end;
      if (tid == 0 && i + 1 == n_tiles) {
        // The unit that this share cuts at its end, if it began here: its last CTA ends the unit.
        int* cut = L.cut + blockIdx.x * 4;
        cut[0] = !unit_end && from_start ? cp.u.b : -1;
        cut[1] = cp.u.head;
        cut[2] = cp.u.mt;
        const long long last = t1 - 1 + (cp.u.tiles - 1 - cp.tile);  // the unit's last tile in the list
        cut[3] = (int)(((last + 1) * grid - 1) / total);  // the largest c with total * c / grid <= last
      }
      if (wk == 0) {
        const int rows = cp.u.w.rows * P.group;
        if (split) {
          float* part = reinterpret_cast<float*>(L.part + (size_t)(blockIdx.x * 2 + (from_start ? 1 : 0)) * part_bytes<D, MT>());
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = row0 + e * 8;
#pragma unroll
            for (int n = 0; n < ND; ++n) *reinterpret_cast<float2*>(part + x * D + n * 8 + (lane & 3) * 2) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
            if ((lane & 3) == 0) {
              part[MT * D + x] = m_run[e];
              part[MT * D + MT + x] = l_run[e];
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = cp.u.mt * MT + row0 + e * 8;
            if (x >= rows) continue;
            const int w = x / P.group, h = cp.u.head * P.group + (x - w * P.group);
            const float inv = l_run[e] > 0.f ? 1.f / l_run[e] : 0.f;
            uint32_t* dst = reinterpret_cast<uint32_t*>(P.out + (long long)(cp.u.w.r0 + w) * P.out_row_b + (long long)h * (D * 2)) + (lane & 3);
#pragma unroll
            for (int n = 0; n < ND; ++n) dst[n * 4] = pack_bf16(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
            if (P.lse && (lane & 3) == 0)
              P.lse[(long long)(cp.u.w.r0 + w) * (P.C.n_heads * P.group) + h] =
                  lse_of(m_run[e], l_run[e], P.scale_log2);
          }
        }
      }
    }
    if (++cp.tile == cp.u.tiles && i + 1 < n_tiles) next_unit(cp);
  }
  cp_wait<0>();
}

// Joins the parts of a unit that several CTAs share, in the order of the
// CTAs. Block c takes the unit that CTA c's share cuts at its end, if it began
// there; blockIdx.y splits its rows. A thread holds 4 elements of a row.
template <int DT, int D, int MT>
__global__ void __launch_bounds__(128) join_kernel(Params P, Plan L, int grid) {
  const int c = blockIdx.x;
  const int* cut = L.cut + c * 4;
  const int b = cut[0];
  if (b < 0) return;
  const int head = cut[1], mt = cut[2], last = min(cut[3], grid - 1);
  const Window w = find_window(P.W, b);
  constexpr int TPR = D / 4;
  const int rows = w.rows * P.group;
  for (int r = blockIdx.y * (128 / TPR) + threadIdx.x / TPR; r < MT; r += gridDim.y * (128 / TPR)) {
    const int x = mt * MT + r;
    if (x >= rows) break;
    const int d = threadIdx.x % TPR * 4;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = c; k <= last; ++k) {
      const float* part = reinterpret_cast<const float*>(L.part + (size_t)(k * 2 + (k == c)) * part_bytes<D, MT>());
      const float pm = part[MT * D + r], pl = part[MT * D + MT + r];
      const float4 y = *reinterpret_cast<const float4*>(part + r * D + d);
      const float top = fmaxf(m, pm);
      const float fa = factor(m, top, P.scale_log2), fb = factor(pm, top, P.scale_log2);
      m = top;
      l = l * fa + pl * fb;
      o.x = o.x * fa + y.x * fb;
      o.y = o.y * fa + y.y * fb;
      o.z = o.z * fa + y.z * fb;
      o.w = o.w * fa + y.w * fb;
    }
    const int ww = x / P.group, h = head * P.group + (x - ww * P.group);
    const float inv = l > 0.f ? 1.f / l : 0.f;
    char* dst = P.out + (long long)(w.r0 + ww) * P.out_row_b + ((long long)h * D + d) * Elem<DT>::kBytes;
    if constexpr (DT == 1)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    else
      *reinterpret_cast<float4*>(dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (P.lse && d == 0)
      P.lse[(long long)(w.r0 + ww) * (P.C.n_heads * P.group) + h] =
          lse_of(m, l, P.scale_log2);
  }
}

constexpr int kGrid = 152 * 3;  // CTAs of the pipeline, at most

template <int D, int WM>
cudaError_t launch_mma(const Params& P, Plan L, cudaStream_t st) {
  using Sh = Shape<D, WM>;
  cudaError_t e = cudaFuncSetAttribute(window_mma_kernel<D, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Sh::smem);
  if (e != cudaSuccess) return e;
  constexpr int grid = 152 * Sh::kCtas;
  window_mma_kernel<D, WM><<<grid, Sh::kT, Sh::smem, st>>>(P, L);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  join_kernel<1, D, Sh::MT><<<dim3(grid, Sh::MT / 16), 128, 0, st>>>(P, L, grid);
  return cudaGetLastError();
}

}  // namespace att
}  // namespace sv

extern "C" {

size_t sv_window_attention_workspace_size(const sv_kv_cache* cache, int32_t n_q_heads, int32_t R) {
  if (!cache || n_q_heads < 1 || R < 0) return 0;
  // The cuts, then two partial results of at most 128 rows a CTA.
  return (size_t)sv::att::kGrid * 16 + (size_t)sv::att::kGrid * 2 * 128 * ((size_t)128 + 2) * 4;
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
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (es == 2) {
    att::Plan L{};
    L.cut = static_cast<int*>(workspace);
    L.part = static_cast<char*>(workspace) + att::kGrid * 16;
    // t / page_size for t < 2^31: with 2^s the next power of two, m = ceil(2^(31 + s) / page_size) errs by less than 2^s.
    int s = 0;
    while ((1ll << s) < P.C.page_size) ++s;
    L.div_shift = 31 + s;
    L.div_mul = (uint32_t)(((1ull << (31 + s)) + P.C.page_size - 1) / P.C.page_size);
    P.q_mask = 0xffffffffu;
    if (P.scale_log2 == 0.f) {
      P.scale_log2 = 1.f;
      P.q_mask = 0u;
    }
    if (P.scale_log2 < 0.f) {
      P.scale_log2 = -P.scale_log2;
      P.q_sign = 0x80008000u;
    }
    // Row tiles as high as the windows' mean number of stacked rows.
    const long long rows = ((long long)R + P.S.n - 1) / P.S.n * P.group;
    cudaError_t e;
    if (D == 128)
      e = rows <= 16 ? att::launch_mma<128, 1>(P, L, st) : rows <= 32 ? att::launch_mma<128, 2>(P, L, st)
          : rows <= 64 ? att::launch_mma<128, 4>(P, L, st) : att::launch_mma<128, 8>(P, L, st);
    else
      e = rows <= 16 ? att::launch_mma<64, 1>(P, L, st) : rows <= 32 ? att::launch_mma<64, 2>(P, L, st)
          : rows <= 64 ? att::launch_mma<64, 4>(P, L, st) : att::launch_mma<64, 8>(P, L, st);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  }
  const int gy = P.S.n > 32768 ? 32768 : P.S.n;
  const long long per = ((long long)R * n_q_heads + gy - 1) / gy;
  const long long want = (per + att::kT / 32 - 1) / (att::kT / 32), most = 152 * 64 / gy + 1;
  const dim3 grid((unsigned)(want < most ? want : most), gy);
  if (D == 128)
    att::window_kernel<0, 128><<<grid, att::kT, 0, st>>>(P);
  else
    att::window_kernel<0, 64><<<grid, att::kT, 0, st>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
