// attention.cu -- attention of the verify windows over the paged cache.
//
// Row w of a window whose candidate begins at w0 sees tokens 0 .. ctx - 1 and
// ctx + w0 .. ctx + w. With s_t = scale * q . k_t, running maximum m and sum l
// over the tokens seen so far, a new score s updates
//   m' = max(m, s), l' = l e^(m - m') + e^(s - m'), o' = o e^(m - m') + e^(s - m') v
// and out = o / l, lse = m + ln l.
//
// The query heads that share a key-value head, over all rows of the window,
// are stacked: a tile of stacked rows reads each key and value once. Four
// kernels, all over equal shares of one list of key tiles (see Plan), chosen
// by the type and by the windows' mean number of stacked rows (64 requests of
// 4096 tokens, 8 key-value heads, one token to 32 of them; the copy rate would
// read heads of 128 in 159 us, of 64 in 79):
//   bf16, up to 16 or 32 rows, and up to 64 with heads of 128
//     window_mma_kernel: 184-190 us for heads of 128 (5.7 - 5.9 TB/s) up to
//     32 rows, 240-244 us for 64; heads of 64: 111-117 us;
//   bf16, more rows
//     window_tc_kernel, tiles of 128 rows: 242 us (heads of 128) and 138 us (of
//     64) for 128 rows, where the other took 476 and 293 us. With 64 rows its
//     tiles are half empty and it takes as long: heads of 64 136 us against
//     158, heads of 128 240 against 240;
//   fp32, row tiles of 4, 8, 16 or 32   window_fma_kernel.
// Sums of a split request are joined by join_kernel.
#include "sv_cache.cuh"
#include "sv_launch.cuh"

#include <cmath>
#include <type_traits>
#include <cuda_bf16.h>

namespace sv {
namespace att {

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

// ---------------------------------------------------------------------------
// The list of key tiles and its shares
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
  int* cut;            // [grid][8]: the unit that a CTA's share cuts at its end: its first stacked row's window row and rows
                       // (0: none), head, row tile, its last CTA
};

struct Unit {
  int b, head, mt;     // request, key-value head, row tile
  int keys, tiles;     // tokens, key tiles
  Window w;
  int n_mt, ctx;
};

// Request b's window, tokens and key tiles, and its number of row tiles (0 tiles where there is nothing to do).
template <int MT, bool kWarp>
__device__ __forceinline__ void load_request(const Params& P, int b, Unit& u, bool tell) {
  u.b = b;
  u.w = find_window<kWarp>(P.W, b);
  u.ctx = P.S.ctx[b];
  const bool len = length_ok(P.C, P.S, u.ctx), fits = len && length_ok(P.C, P.S, (long long)u.ctx + max(u.w.rows, 0));
  if (u.w.rows <= 0 || !fits) {
    if (tell && (u.w.rows < 0 || !fits))
      set_status(P.status, u.w.rows < 0 ? SV_DATA_BAD_OFFSETS : len ? SV_DATA_BAD_PAGE : SV_DATA_BAD_SEQ);
    u.keys = u.tiles = u.n_mt = 0;
    return;
  }
  u.keys = u.ctx + u.w.rows;
  u.tiles = (u.keys + kTK - 1) / kTK;
  u.n_mt = (int)(((long long)u.w.rows * P.group + MT - 1) / MT);
}

// The list's tiles in `grid` shares: the first `more` of them hold size + 1, the others size.
struct Share {
  long long t0, t1;  // this CTA's tiles of the list
  long long size;
  int more;
};
struct Cursor {
  Unit u;
  int tile;
};

// n / d and the rest, in 32 bits where that is enough.
__device__ __forceinline__ long long div_small(long long n, int d, int& rest) {
  if (n >> 32 == 0) {
    const uint32_t q = (uint32_t)n / (uint32_t)d;
    rest = (int)((uint32_t)n - q * (uint32_t)d);
    return q;
  }
  const long long q = n / d;
  rest = (int)(n - q * d);
  return q;
}

// This CTA's share, and a cursor on its first tile; false for a CTA without
// one. Thread i sums the tiles of its run of requests; a scan over the threads
// gives the list's length, and the thread whose run holds the share's first
// tile walks it and tells the others the request.
template <int MT, int kThr>
__device__ __forceinline__ bool take_share(const Params& P, const Plan& L, Share& sh, Cursor& c) {
  wait_for_stream();
  __shared__ long long s_scan[kThr / 32];
  __shared__ Unit s_unit;
  __shared__ long long s_first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (P.S.n + kThr - 1) / kThr;
  long long mine = 0;
  for (int b = tid * per; b < min((tid + 1) * per, P.S.n); ++b) {
    load_request<MT, false>(P, b, c.u, blockIdx.x == 0);
    mine += (long long)c.u.tiles * c.u.n_mt * P.C.n_heads;
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
#pragma unroll
  for (int w = 0; w < kThr / 32; ++w) {
    if (w < warp) incl += s_scan[w];
    total += s_scan[w];
  }
  const int grid = (int)min((long long)gridDim.x, total), id = blockIdx.x;  // shares of a tile at least
  if (id >= grid) {
    if (tid == 0) L.cut[id * 8 + 1] = 0;
    return false;
  }
  sh.size = div_small(total, grid, sh.more);
  sh.t0 = sh.size * id + min(id, sh.more);
  sh.t1 = sh.t0 + sh.size + (id < sh.more);
  if (sh.t0 >= incl - mine && sh.t0 < incl) {
    long long at = incl - mine;
    if (per > 1)
      for (int b = tid * per;; ++b) {
        load_request<MT, false>(P, b, c.u, false);
        const long long n = (long long)c.u.tiles * c.u.n_mt * P.C.n_heads;
        if (sh.t0 < at + n) break;
        at += n;
      }
    s_unit = c.u;
    s_first = sh.t0 - at;  // first tile of the share within its request
  }
  if (tid == 0) L.cut[id * 8 + 1] = 0;  // until the share's end is reached
  __syncthreads();
  c.u = s_unit;
  const long long unit = div_small(s_first, c.u.tiles, c.tile);
  c.u.head = (int)div_small(unit, c.u.n_mt, c.u.mt);
  return true;
}

// On to the next unit's first tile (the share holds one), by a whole warp.
template <int MT>
__device__ __forceinline__ void next_unit(const Params& P, Cursor& c) {
  c.tile = 0;
  if (++c.u.mt < c.u.n_mt) return;
  c.u.mt = 0;
  if (++c.u.head < P.C.n_heads) return;
  c.u.head = 0;
  for (int b = c.u.b + 1; b < P.S.n; ++b) {
    load_request<MT, true>(P, b, c.u, false);
    if (c.u.tiles) return;
  }
}

// By one thread on the share's last tile: the unit that the share cuts at its
// end, if it began here, and the last CTA that has a part of it.
__device__ __forceinline__ void tell_cut(const Plan& L, const Share& sh, const Cursor& c, bool cuts) {
  const long long last = sh.t1 - 1 + (c.u.tiles - 1 - c.tile);  // the unit's last tile in the list
  const long long front = (sh.size + 1) * sh.more;               // tiles of the larger shares
  const long long k = last < front ? last / (sh.size + 1) : sh.more + (last - front) / sh.size;
  int4* cut = reinterpret_cast<int4*>(L.cut + blockIdx.x * 8);
  cut[0] = make_int4(c.u.w.r0, cuts ? c.u.w.rows : 0, c.u.head, c.u.mt);
  cut[1] = make_int4((int)k, 0, 0, 0);
}

// The first row of the candidate that window row w lies in.
__device__ __forceinline__ int candidate_start(const Params& P, const Window& win, int w) {
  if (!P.W.cand) return 0;
  int a = win.c0, z = win.c1;
  while (z - a > 1) {
    const int mid = (a + z) >> 1;
    if ((long long)P.W.cu[mid] + mid - win.r0 <= w)
      a = mid;
    else
      z = mid;
  }
  const long long at = (long long)P.W.cu[a] + a - win.r0;
  return at < 0 || at > w ? w : (int)at;
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

// ---------------------------------------------------------------------------
// bf16, few stacked rows: mma.sync over a paged pipeline
// ---------------------------------------------------------------------------
// Bound by the bytes up to 32 rows. K and V tiles are gathered by 16-byte
// asynchronous copies through a ring of swizzled stages (any page size and
// layout; pages of 1, 16 and 64 tokens take the same time), the page table
// looked up a tile ahead of them. With few rows the warps split a tile's
// tokens (WK), with 64 its rows. Two CTAs an SM with three stages for heads of
// 128 (three CTAs with two stages: 7% slower), four with three for heads of 64
// (two with six: 5% slower).
template <int D, int WM>
struct Shape {
  static constexpr int MT = 16 * WM;            // stacked rows of a unit
  static constexpr int WK = 4 / WM;             // warps that split a key tile
  static constexpr int kT = 32 * WM * WK;       // threads
  static constexpr int KW = kTK / WK;           // tokens of a tile for one warp
  static constexpr int KS = KW < 32 ? KW : 32;  // tokens that go through the softmax at once
  static constexpr int kCtas = D == 64 ? 4 : 2;   // an SM
  static constexpr int kStages = 3;
  static constexpr int kTile = kTK * D * 2;     // bytes of K (or V) of a tile
  static constexpr size_t smem = (size_t)kStages * 2 * kTile + (kStages + 1) * (kTK * 8 + 16);
  static_assert(kCtas * MT <= 256, "the workspace has room for the partial results");
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
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp % WM, wk = warp / WM;

  Share sh;
  Cursor ld;
  if (!take_share<MT, kTW>(P, L, sh, ld)) return;
  const int n_tiles = (int)(sh.t1 - sh.t0);
  Cursor cp = ld;  // two cursors over the share: one loads, one computes

  // Page lookups run one tile ahead of the copies: threads 0 .. kTK - 1 hold a token each. The byte offset of a token in K and
  // V, or -1 where it has no page or lies behind the sequence.
  auto lookup = [&](const Cursor& c, int& page, int& place) {  // issued early
    const int t = c.tile * kTK + tid;
    page = -2;
    place = 0;
    if (tid < kTK && t < c.u.keys) {
      const int slot = page_slot(P.C, t);
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
    for (int i = 0; i < kTK / RPP; i += 4) {
      long long off[4];  // read together: 254 -> 242 us for windows of 64 rows
#pragma unroll
      for (int e = 0; e < 4; ++e) off[e] = s_off[ring * kTK + tid / CPR + (i + e) * RPP];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = tid / CPR + (i + e) * RPP;
        const bool ok = off[e] >= 0;
        const long long at = (ok ? off[e] : 0) + c * 16;
        cp16(base + swz<D>(r, c), P.C.k + at, ok);
        cp16(base + Sh::kTile + swz<D>(r, c), P.C.v + at, ok);
      }
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
        if (i + 1 < n_tiles && ++ld.tile == ld.u.tiles) next_unit<MT>(P, ld);
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

  if (S < n_tiles) lookup(ld, page, place);  // tile S, stored in the first round
  for (int i = 0; i < n_tiles; ++i) {
    if (i + 1 == n_tiles) release_stream();  // the join may take its place
    if (!begun) {  // a new unit: its rows
      begun = true;
      from_start = cp.tile == 0;
      const int rows = cp.u.w.rows * P.group;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int x = cp.u.mt * MT + row0 + e * 8;
        const bool ok = x < rows;
        const int w = ok ? x / P.group : 0, h = ok ? x - w * P.group : 0;
        lo[e] = ok ? candidate_start(P, cp.u.w, w) : 0;
        hi[e] = ok ? w : -1 - cp.u.ctx;  // rows past the window see nothing
        const uint32_t* src = reinterpret_cast<const uint32_t*>(P.q + (long long)(cp.u.w.r0 + w) * P.q_row_b +
                                                                (long long)(cp.u.head * P.group + h) * (D * 2)) + (lane & 3);
#pragma unroll
        for (int k = 0; k < KD; ++k) {
          q[k][e] = ok ? (src[k * 8] & P.q_mask) ^ P.q_sign : 0u;
          q[k][e + 2] = ok ? (src[k * 8 + 4] & P.q_mask) ^ P.q_sign : 0u;
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
    if (i + S < n_tiles) {
      store_lookup((i + S) % (S + 1), ld.u.head, page, place);  // for the next round's copy
      if (i + S + 1 < n_tiles) {
        if (++ld.tile == ld.u.tiles) next_unit<MT>(P, ld);
        lookup(ld, page, place);  // has this pass's arithmetic to arrive
      }
    }

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
      // The product takes the weights in V's type; their sum keeps 32 bits. Against 64 bits the output is 0.0018 off, where
      // rounding the exact one to bf16 gives 0.0017 (weights kept in 32 bits would need a product of two parts, twice the work).
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
        tell_cut(L, sh, cp, !unit_end && from_start);
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
    if (++cp.tile == cp.u.tiles && i + 1 < n_tiles) next_unit<MT>(P, cp);
  }
  cp_wait<0>();
}

// ---------------------------------------------------------------------------
// bf16, row tiles of 128: the fifth-generation tensor cores
// ---------------------------------------------------------------------------
// S = Q K^T and O += P V by tcgen05.mma with S, P and O in tensor memory.
// Three roles, joined by mbarriers only:
//   G groups of 4 warps   softmax and output: group i % G takes tile i, with
//                an O of its own (a tile's softmax is a chain of about 1500
//                cycles: two at a time on an SM). A thread owns a row (a TMEM lane). The reference
//                maximum moves only when a row's maximum outgrows it by 2^8,
//                since moving it means rescaling O in TMEM. At a unit's end
//                the group of its last tile joins the groups' O;
//   4 warps      copies: Q tiles (two buffers), then K and V tiles gathered
//                over the pages into a ring of swizzled stages;
//   the last     issues the products: S of tile i, then P V of tile i - 1
//                (two S tiles).
// Every wait is bounded: where one gives up the CTA sets SV_DEV_COPY_TIMEOUT,
// lets its copies and products end, frees its tensor memory and leaves.
template <int D>
struct TcShape {
  static constexpr int MT = 128;
  static constexpr int G = D == 64 ? 1 : 2;         // softmax groups
  static constexpr int NB = 2;                      // S tiles
  static constexpr int NW = D == 64 ? 2 : 4;        // warps that copy
  static constexpr int kMmaWarp = G * 4 + NW;
  static constexpr int kT = (kMmaWarp + 1) * 32;
  static constexpr int kCtas = D == 64 ? 2 : 1;     // an SM
  static constexpr int kStages = 4;
  static constexpr int kRing = kStages + 2;         // tiles whose page lookups are kept
  static constexpr int kTile = kTK * D * 2;         // bytes of K (or V) of a tile
  static constexpr int kQ = MT * D * 2;             // bytes of a Q tile
  static constexpr size_t smem = 1024 + 2 * kQ + (size_t)kStages * 2 * kTile;
  static constexpr int kCols = 512 / kCtas;         // TMEM columns: G times O (D), then the S tiles (64 each, P in their first half)
  static_assert(G * D + NB * kTK <= kCols && kStages > NB && NB >= G && NB % G == 0 && kStages % NW == 0, "");
};

__device__ __forceinline__ uint64_t umma_desc(uint32_t addr, uint32_t lead_bytes) {
  // 128-byte swizzle, eight rows of 128 bytes an atom of 1024 bytes; atoms follow each other.
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lead_bytes >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
constexpr uint32_t umma_idesc(int n, bool b_mn_major) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (uint32_t)(128 / 16) << 24;
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// One lane of the (whole, converged) warp. The products' warp runs its loop
// as a whole and only issues under this, so that the instructions' operands
// stay uniform: issued from a lane's own branch each took about 90 cycles.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
  return is != 0;
}
// Arrives on the mbarrier when the products issued before have ended.
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Arrives on the mbarrier when this thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
  for (int it = 0; it < kSpinLimit; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  set_status(status, SV_DEV_COPY_TIMEOUT);
  return false;
}

template <int S, int G, int NB>
struct TcBars {
  uint64_t full[S], empty[S];  // a stage's tile has landed; its P V has ended
  uint64_t s_full[NB];         // S has been computed
  uint64_t p_ready[NB];        // S has been read, P written, O rescaled
  uint64_t o_done[G];          // a tile's P V has ended
  uint64_t ml[G];              // a group's maxima and sums of a unit are in shared memory
  uint64_t q_full[2], q_empty[2];
  uint64_t o_free;             // a unit's O have been read
  uint64_t end;                // every product has ended
};

template <int D>
__global__ void __launch_bounds__(TcShape<D>::kT, TcShape<D>::kCtas) window_tc_kernel(Params P, Plan L) {
  using Sh = TcShape<D>;
  constexpr int S = Sh::kStages, R = Sh::kRing, G = Sh::G, NB = Sh::NB;
  extern __shared__ char smem_raw[];
  __shared__ TcBars<S, G, NB> bars;
  __shared__ float2 s_ml[G][128];  // a group's (maximum, sum) of a row, at a unit's end
  __shared__ long long s_off[Sh::NW][kTK];  // a copying warp's tile: the tokens' byte offsets
  __shared__ uint32_t s_valid[R][4];        // a tile's tokens that have a page, and whether it is the unit's last here
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  Share sh;
  Cursor c;
  if (!take_share<128, Sh::kT>(P, L, sh, c)) return;
  const int n_tiles = (int)(sh.t1 - sh.t0);

  char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t q_base = smem_addr(smem), kv_base = q_base + 2 * Sh::kQ;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_addr(&bars.full[i]), 32 + 1);
      mbar_init(smem_addr(&bars.empty[i]), 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(smem_addr(&bars.s_full[i]), 1);
      mbar_init(smem_addr(&bars.p_ready[i]), 128);
    }
    for (int i = 0; i < G; ++i) {
      mbar_init(smem_addr(&bars.o_done[i]), 1);
      mbar_init(smem_addr(&bars.ml[i]), 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.q_full[i]), Sh::NW * 32);
      mbar_init(smem_addr(&bars.q_empty[i]), 1);
    }
    mbar_init(smem_addr(&bars.o_free), 128);
    mbar_init(smem_addr(&bars.end), 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == Sh::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)), "r"(Sh::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // Waits for a phase; false once any wait of the CTA has given up. The first try is all that a phase that has ended costs.
  auto wait = [&](uint64_t& bar, int parity) {
    return mbar_try_wait(smem_addr(&bar), (uint32_t)parity) || wait_long(smem_addr(&bar), (uint32_t)parity, &s_abort, P.status);
  };
  const uint32_t s_col = tmem + G * D;  // the first S
  if (warp >= G * 4 && warp < Sh::kMmaWarp) {
    // ---------------------------------------------------------------- copies
    // Copying warp j takes every NW-th tile whole, with nothing shared between the warps but Q, of which each brings its rows.
    const int j = warp - G * 4;
    constexpr int NW = Sh::NW, CPR = D / 8, RPP = 32 / CPR;  // 16-byte chunks of a row; rows that a warp copies at once
    const int ch = lane % CPR, r0 = lane / CPR;
    const uint32_t to = (uint32_t)((ch >> 3) * (kTK * 128) + r0 * 128), x0 = (uint32_t)(((ch & 7) ^ r0) << 4);
    const char* k_ch = P.C.k + ch * 16;
    const long long v_k = P.C.v - P.C.k;
    // The pages of the warp's next tile, two tokens a lane, looked up while the one before it is copied.
    Cursor ld = c;
    int ld_at = 0, page[2], place[2];
    auto lookup = [&](int i) {
      for (; ld_at < i; ++ld_at)
        if (++ld.tile == ld.u.tiles) next_unit<128>(P, ld);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = ld.tile * kTK + h * 32 + lane;
        page[h] = -2;
        if (k < ld.u.keys) {
          const int slot = page_slot(P.C, k);
          place[h] = k - slot * P.C.page_size;
          page[h] = P.S.table[(long long)ld.u.b * P.S.stride + slot];
        }
      }
    };
    if (j < n_tiles) lookup(j);
    bool alive = true;
    int unit = 0;  // units whose rows are loaded
    // A unit's rows: this warp's 128 / NW of them.
    auto load_q = [&](const Cursor& u) {
      if (unit >= 2) alive = __all_sync(kFull, wait(bars.q_empty[unit & 1], ((unit >> 1) - 1) & 1));
      if (!alive) return;
      const uint32_t qb = q_base + (unit & 1) * Sh::kQ + (uint32_t)((ch >> 3) * (128 * 128));
      const int rows = u.u.w.rows * P.group, first = j * (128 / NW) + r0;
      int row = u.u.mt * 128 + first, w = row / P.group, h = row - w * P.group;
      const char* q = P.q + (long long)u.u.w.r0 * P.q_row_b + (long long)u.u.head * P.group * (D * 2) + ch * 16;
      constexpr int N = 128 / NW / RPP, U = 8;  // rows of a lane, of which U are in flight
#pragma unroll 1
      for (int n = 0; n < N; n += U) {
        uint4 v[U];
#pragma unroll
        for (int e = 0; e < U; ++e) {
          v[e] = row < rows ? *reinterpret_cast<const uint4*>(q + w * P.q_row_b + h * (D * 2)) : make_uint4(0u, 0u, 0u, 0u);
          row += RPP;
          h += RPP;
          while (h >= P.group) {
            h -= P.group;
            ++w;
          }
        }
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const int r = first + (n + e) * RPP;
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(qb + r * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                       "r"((v[e].x & P.q_mask) ^ P.q_sign), "r"((v[e].y & P.q_mask) ^ P.q_sign),
                       "r"((v[e].z & P.q_mask) ^ P.q_sign), "r"((v[e].w & P.q_mask) ^ P.q_sign)
                       : "memory");
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(smem_addr(&bars.q_full[unit & 1]));
      ++unit;
    };
    // The first unit's rows at once, the next one's S tiles into a unit, when the buffer has long been free (or at the unit's
    // end): a new unit then does not wait for its rows.
    load_q(c);
    bool next_loaded = false;
    int into = 0;  // tiles into the unit
    for (int i = 0; i < n_tiles && alive; ++i) {
      const int left = c.u.tiles - c.tile;  // tiles of the unit from here on
      if (!next_loaded && i + left < n_tiles && (into == S || left == 1)) {
        Cursor q = c;
        next_unit<128>(P, q);
        load_q(q);
        next_loaded = true;
        if (!alive) break;
      }
      if (i % NW == j) {
        if (i >= S) alive = __all_sync(kFull, wait(bars.empty[i % S], (i / S - 1) & 1));
        if (!alive) break;
        uint32_t valid[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool ok = page[h] >= 0 && page[h] < P.C.n_pages;
          if (!ok && page[h] != -2) set_status(P.status, SV_DATA_BAD_PAGE);
          s_off[j][h * 32 + lane] = ok ? page[h] * P.C.page_b + place[h] * P.C.token_b + ld.u.head * P.C.head_b : -1;
          valid[h] = __ballot_sync(kFull, ok);
        }
        if (lane == 0) {
          s_valid[i % R][0] = valid[0];
          s_valid[i % R][1] = valid[1];
          s_valid[i % R][2] = ld.tile + 1 == ld.u.tiles || i + 1 == n_tiles;
        }
        if (i + NW < n_tiles) lookup(i + NW);
        __syncwarp();
        const uint32_t base = kv_base + (i % S) * 2 * Sh::kTile + to;
        if ((valid[0] & valid[1]) == 0xffffffffu) {
#pragma unroll 1
          for (int n0 = 0; n0 < kTK / RPP; n0 += 8) {
            long long off[8];  // read together: 271 -> 244 us for heads of 128
#pragma unroll
            for (int e = 0; e < 8; ++e) off[e] = s_off[j][(n0 + e) * RPP + r0];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t dst = base + (n0 + e) * RPP * 128 + (x0 ^ ((e * RPP & 7) << 4));
              cp16(dst, k_ch + off[e], true);
              cp16(dst + Sh::kTile, k_ch + off[e] + v_k, true);
            }
          }
        } else {  // zeros where there is no page, and behind the sequence
#pragma unroll 1
          for (int n = 0; n < kTK / RPP; ++n) {
            const long long off = s_off[j][n * RPP + r0];
            const char* src = k_ch + (off < 0 ? 0 : off);
            const uint32_t dst = base + n * RPP * 128 + (x0 ^ ((n * RPP & 7) << 4));
            cp16(dst, src, off >= 0);
            cp16(dst + Sh::kTile, src + v_k, off >= 0);
          }
        }
        cp_arrive(smem_addr(&bars.full[i % S]));
        if (lane == 0) mbar_arrive(smem_addr(&bars.full[i % S]));  // releases what lane 0 wrote to s_valid
        __syncwarp();
      }
      ++into;
      if (++c.tile == c.u.tiles && i + 1 < n_tiles) {
        next_unit<128>(P, c);
        next_loaded = false;
        into = 0;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == Sh::kMmaWarp) {
    // -------------------------------------------------------------- products
    // What a tile needs to know of its unit is whether it ends it, which the copies left beside its lookups: this warp's steps are
    // the chain that bounds short tiles, and a cursor of its own cost as much as the issue itself.
    bool alive = true, first = true;       // the tile begins its unit
    int unit = 0, pv_unit = 0;             // of the S being issued, of the P V
    uint32_t begun = 0;                    // groups that have an O of that unit
    uint32_t ends = 0;                     // of the tiles between their S and their P V: bit k of the tile k behind
    const uint64_t q_desc = umma_desc(q_base, 16), k_desc = umma_desc(kv_base, 16), v_desc = umma_desc(kv_base + Sh::kTile, kTK * 128);
    auto wait_all = [&](uint64_t& bar, int parity) { return __all_sync(kFull, wait(bar, parity)) != 0; };
    auto issue_pv = [&](int i, bool end) {
      const int g = i % G;
      alive = alive && wait_all(bars.p_ready[i % NB], (i / NB) & 1);
      if (alive && !begun && pv_unit > 0) alive = wait_all(bars.o_free, (pv_unit - 1) & 1);
      if (!alive) return;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t vd = v_desc + (uint64_t)((i % S) * 2 * Sh::kTile / 16);
        const bool add = begun >> g & 1u;
#pragma unroll
        for (int k = 0; k < kTK / 16; ++k)
          umma_ts(tmem + g * D, s_col + i % NB * kTK + k * 8, vd + k * (2048 / 16), umma_idesc(D, true), k > 0 || add);
        umma_commit(smem_addr(&bars.empty[i % S]));
        umma_commit(smem_addr(&bars.o_done[g]));
      }
      begun = end ? 0u : begun | 1u << g;
      pv_unit += end;
    };
    for (int i = 0; i < n_tiles && alive; ++i) {
      if (first) alive = wait_all(bars.q_full[unit & 1], (unit >> 1) & 1);
      alive = alive && wait_all(bars.full[i % S], (i / S) & 1);
      if (!alive) break;
      const bool last = s_valid[i % R][2] != 0;
      fence_proxy_async_smem();  // the copies wrote the tile through the generic proxy, the products read it through the other
      tc_fence_after();
      if (elect_one()) {
        const uint64_t qd = q_desc + (uint64_t)((unit & 1) * Sh::kQ / 16), kd = k_desc + (uint64_t)((i % S) * 2 * Sh::kTile / 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_ss(s_col + i % NB * kTK, qd + ((k >> 2) * (128 * 128) + (k & 3) * 32) / 16, kd + ((k >> 2) * (kTK * 128) + (k & 3) * 32) / 16,
                  umma_idesc(kTK, false), k > 0);
        umma_commit(smem_addr(&bars.s_full[i % NB]));
        if (last) umma_commit(smem_addr(&bars.q_empty[unit & 1]));
      }
      ends = ends << 1 | (uint32_t)last;
      first = last;
      unit += last;
      if (i >= NB - 1) issue_pv(i - (NB - 1), ends >> (NB - 1) & 1u);
    }
    for (int i = max(0, n_tiles - (NB - 1)); i < n_tiles && alive; ++i) issue_pv(i, ends >> (n_tiles - 1 - i) & 1u);
    if (elect_one()) umma_commit(smem_addr(&bars.end));
    __syncwarp();
    for (int it = 0; it < kSpinLimit && !__all_sync(kFull, mbar_try_wait(smem_addr(&bars.end), 0)); ++it) {
    }
  } else {
    // --------------------------------------------------- softmax and output
    const int g = warp >> 2, r = tid & 127;  // the group, the row
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, o_addr = tmem + lanes + g * D;
    int unit_begin = 0, parts[G];            // the unit's first tile; units in which each group had one
#pragma unroll
    for (int k = 0; k < G; ++k) parts[k] = 0;
    bool from_start = c.tile == 0, fresh = true;
    int lo = 0, hi = 0;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < n_tiles; ++i) {
      const int rows = c.u.w.rows * P.group, row = c.u.mt * 128 + r;
      const bool last = c.tile + 1 == c.u.tiles || i + 1 == n_tiles;  // of the unit, here
      if (i + 1 == n_tiles) release_stream();
      if (i % G == g) {
        if (fresh) {
          fresh = false;
          const int w = row < rows ? row / P.group : 0;
          lo = row < rows ? candidate_start(P, c.u.w, w) : 0;
          hi = row < rows ? w : -1 - c.u.ctx;  // rows past the window see nothing
          m = -INFINITY;
          l = 0.f;
        }
        const uint32_t s_addr = s_col + lanes + i % NB * kTK;
        const bool ok = wait(bars.full[i % S], (i / S) & 1) && wait(bars.s_full[i % NB], (i / NB) & 1);
        if (__any_sync(kFull, !ok)) break;
        tc_fence_after();
        // Hidden tokens: behind the history all but the row's part of the window, and those without a page. Bit k of `see` is
        // token k of the tile.
        uint64_t see = (uint64_t)s_valid[i % R][1] << 32 | s_valid[i % R][0];
        const bool masked = (c.tile + 1) * kTK > c.u.ctx || see != ~0ull;
        if (masked) {
          const int at0 = c.tile * kTK - c.u.ctx;  // of the tile's first token in the window
          auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; };
          see &= hi < -c.u.ctx ? 0ull : below(-at0) | (below(hi + 1 - at0) & ~below(max(lo, 0) - at0));
        }
        uint32_t s[2][32];
        tc_ld32(s[0], s_addr);
        tc_ld32(s[1], s_addr + 32);
        tc_wait_ld();
        if (masked) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t bits = (uint32_t)(see >> (h * 32));
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(bits & 1u << j)) s[h][j] = 0xff800000u;
          }
        }
        float most[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) most[j] = fmaxf(__uint_as_float(s[0][j]), __uint_as_float(s[1][j]));
#pragma unroll
        for (int j = 4; j < 32; ++j) most[j & 3] = fmaxf(most[j & 3], fmaxf(__uint_as_float(s[0][j]), __uint_as_float(s[1][j])));
        const float top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
        // The reference moves where the maximum is 2^8 above it: the weights, rounded to bf16 as in the kernel above, then reach
        // 2^8 instead of one (that rounding is relative; 0.0022 off 64 bits in all). Before a row's first token there is nothing
        // to rescale.
        float f = 1.f;
        if (m == -INFINITY) {
          m = top;
        } else if ((top - m) * P.scale_log2 > 8.f) {
          f = factor(m, top, P.scale_log2);
          m = top;
          l *= f;
        }
        // The group's last P V: every phase is waited for in turn, so that its parity tells which one has ended.
        const bool done = i < G || wait(bars.o_done[g], (i / G - 1) & 1);
        if (__any_sync(kFull, !done)) break;
        const float off = m == -INFINITY ? 0.f : __fmul_rn(m, P.scale_log2);
        const f2_t sl = f2_splat(P.scale_log2), neg = f2_splat(-off);
        f2_t sum = 0ull;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const f2_t e = f2_ex2(f2_fma(f2_pack(__uint_as_float(s[h][2 * j]), __uint_as_float(s[h][2 * j + 1])), sl, neg));
            sum = f2_add(sum, e);
            float a, b;
            f2_unpack(e, a, b);
            p[j] = pack_bf16(a, b);
          }
          tc_st16(s_addr + h * 16, p);
        }
        float sa, sb;
        f2_unpack(sum, sa, sb);
        l += sa + sb;
        if (__any_sync(kFull, f != 1.f)) {
          tc_fence_after();
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            uint32_t o[16];
            tc_ld16(o, o_addr + d);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tc_st16(o_addr + d, o);
          }
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(smem_addr(&bars.p_ready[i % NB]));
      }
      if (last) {
        // The groups with a tile of this unit; the last of each hands its maxima and sums to the group of the unit's last tile.
        const int count = i + 1 - unit_begin, fin = i % G;
        const int behind = (i - g + G * 2) % G;  // how far the group's last tile lies behind the unit's
        bool ok = true;
        if (behind < count) {
          ok = wait(bars.o_done[g], ((i - behind) / G) & 1);
          if (ok && g != fin) {
            s_ml[g][r] = make_float2(m, l);
            mbar_arrive(smem_addr(&bars.ml[g]));
          }
        }
        if (__any_sync(kFull, !ok)) break;
        if (g == fin) {
          float mg[G], fg[G];
          float top = m;
#pragma unroll
          for (int k = 0; k < G; ++k) {
            mg[k] = -INFINITY;
            if (k != g && (i - k + G * 2) % G < count) {
              ok = ok && wait(bars.ml[k], parts[k] & 1);
              if (ok) mg[k] = s_ml[k][r].x;
            }
            if (k == g) mg[k] = m;
            top = fmaxf(top, mg[k]);
          }
          if (__any_sync(kFull, !ok)) break;
          tc_fence_after();
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < G; ++k) {
            fg[k] = factor(mg[k], top, P.scale_log2);
            if (mg[k] > -INFINITY) sum += fg[k] * (k == g ? l : s_ml[k][r].y);
          }
          const bool unit_end = c.tile + 1 == c.u.tiles, split = !from_start || !unit_end;
          if (r == 0 && i + 1 == n_tiles) tell_cut(L, sh, c, !unit_end && from_start);
          float* part = reinterpret_cast<float*>(L.part + (size_t)(blockIdx.x * 2 + (from_start ? 1 : 0)) * part_bytes<D, 128>());
          const int w = row / P.group, h = c.u.head * P.group + (row - w * P.group);
          char* dst = P.out + (long long)(c.u.w.r0 + w) * P.out_row_b + (long long)h * (D * 2);
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            float o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = 0.f;
#pragma unroll
            for (int k = 0; k < G; ++k) {
              if ((i - k + G * 2) % G >= count) continue;  // the same for the whole CTA
              uint32_t x[16];
              tc_ld16(x, tmem + lanes + k * D + d);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = fmaf(__uint_as_float(x[j]), fg[k], o[j]);
            }
            if (split) {
              float4* to = reinterpret_cast<float4*>(part + r * D + d);
#pragma unroll
              for (int j = 0; j < 4; ++j) to[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            } else if (row < rows) {
              uint4* to = reinterpret_cast<uint4*>(dst + d * 2);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint32_t v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = pack_bf16(o[8 * j + 2 * e] * inv, o[8 * j + 2 * e + 1] * inv);
                to[j] = make_uint4(v[0], v[1], v[2], v[3]);
              }
            }
          }
          if (split) {
            part[128 * D + r] = top;
            part[128 * D + 128 + r] = sum;
          } else if (row < rows && P.lse) {
            P.lse[(long long)(c.u.w.r0 + w) * (P.C.n_heads * P.group) + h] = lse_of(top, sum, P.scale_log2);
          }
          tc_fence_before();
          mbar_arrive(smem_addr(&bars.o_free));
        }
#pragma unroll
        for (int k = 0; k < G; ++k) parts[k] += k != fin && (i - k + G * 2) % G < count;
        unit_begin = i + 1;
        fresh = from_start = true;
      }
      if (++c.tile == c.u.tiles && i + 1 < n_tiles) next_unit<128>(P, c);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == Sh::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kCols) : "memory");
}

// ---------------------------------------------------------------------------
// fp32: the same shares, on the fp32 pipes
// ---------------------------------------------------------------------------
template <int D, int M>
struct Shape32 {
  static constexpr int MT = M;                        // stacked rows of a unit: 4, 8, 16 or 32
  static constexpr int kT = 128;                      // threads
  static constexpr int RT = M < 8 ? M : 8;            // rows of a thread's tile, of scores and of the output
  static constexpr int KT = 4;                        // keys of its tile of scores
  static constexpr int KG = kTK / KT;                 // groups of threads over the keys
  static constexpr int DP = kT / KG / (M / RT);       // threads that split the sum of a score
  static constexpr int WR = M / RT;                   // warps side by side over the rows of the output
  static constexpr int WK = 4 / WR;                   // and over the tokens
  static constexpr int LK = 128 / D;                  // parts of a warp that split its tokens
  static constexpr int kPitch = D * 4 + DP % 8 * 16;  // bytes of a K row: the threads of a quarter warp read different banks
  static constexpr int SP = kTK + 4;                  // row pitch of the scores, in floats
  static constexpr int kK = kTK * kPitch, kV = kTK * D * 4;
  static constexpr int kCtas = D == 64 ? (M <= 8 ? 4 : 3) : (M <= 8 ? 3 : 2);  // an SM
  static constexpr size_t smem = (size_t)kK + kV + (size_t)M * D * 4 + (size_t)M * SP * 4 + M * (WK + 1) * 8 + 2 * kTK * 8 + 16;
  static_assert((WK - 1) * M * D * 4 <= kV, "the sums of the other warps fit the tile of V");
};

// N values of each of DP / X threads summed over them: every exchange adds one half of them to the same half of another
// thread's, and thread i is left with the part that its bits from X on name.
template <int N, int X, int DP>
__device__ __forceinline__ void sum_halves(float* s, int i) {
  if constexpr (X < DP) {
    const bool up = i & X;
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const float give = up ? s[e] : s[e + N / 2], keep = up ? s[e + N / 2] : s[e];
      s[e] = keep + __shfl_xor_sync(kFull, give, X);
    }
    sum_halves<N / 2, X * 2, DP>(s, i);
  }
}

// Bound by the bytes up to 8 rows and by the fp32 pipes' instructions and the
// latencies around them above. A tile's scores: a thread holds 8 rows x 4 keys
// and every DP-th piece of d, 12 reads of shared memory for 128 multiply-adds;
// sum_halves leaves it DP times fewer scores, whose maxima go over the warp
// and over the warps that share the rows; sums of weights stay with their keys
// until the unit ends. The product with V: 8 rows x 4 elements a thread. K is
// loaded while the weights and the product with V are computed and V behind
// it, so that a CTA needs one tile of each and two or more CTAs fit an SM. 64
// requests of 1000 tokens, 8 heads of 64 (32 requests for 128), 262 MB: 4 rows
// 64 us (64), 8 rows 68 (68), 16 rows 89 (84), 32 rows 132 (125), 128 rows 500
// (465: 37 TFLOP/s).
// Packed pairs of multiply-adds were no faster (their sums take twice the
// registers), nor were four CTAs an SM with heads of 64.
template <int D, int MT>
__global__ void __launch_bounds__(128, Shape32<D, MT>::kCtas) window_fma_kernel(Params P, Plan L) {
  using Sh = Shape32<D, MT>;
  constexpr int SP = Sh::SP, RT = Sh::RT, KT = Sh::KT, KG = Sh::KG, DP = Sh::DP, CPR = D / 4;
  constexpr int NR = RT >= DP ? RT / DP : 1;   // rows and keys of the scores that a thread is left with
  constexpr int NK = RT * KT / DP / NR;
  static_assert(KT == 4 && (NK == 4 || NK == 2), "a thread sums its weights in pairs");
  constexpr int TV = kTK / Sh::WK / Sh::LK;    // tokens of a thread's share of the product with V
  extern __shared__ __align__(1024) char smem[];
  char* s_k = smem;
  char* s_v = smem + Sh::kK;
  float* s_q = reinterpret_cast<float*>(s_v + Sh::kV);            // [MT][D]
  float* s_p = s_q + MT * D;                                      // [MT][SP]
  float* s_m = s_p + MT * SP;                                     // [MT] maxima of a unit's end
  float* s_f = s_m + MT;                                          // [MT] factors of the tile
  float* s_top = s_f + MT;                                        // [WK][MT] the warps' maxima of the tile
  float* s_l = s_top + Sh::WK * MT;                               // [WK][MT] their sums of a unit's end
  long long* s_off = reinterpret_cast<long long*>(s_l + Sh::WK * MT);  // [2][kTK]
  uint32_t* s_valid = reinterpret_cast<uint32_t*>(s_off + 2 * kTK);    // [2][2]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Share sh;
  Cursor ld;
  if (!take_share<MT, 128>(P, L, sh, ld)) return;
  const int n_tiles = (int)(sh.t1 - sh.t0);
  Cursor cp = ld;
  // Scores: rows row0 .. row0 + RT - 1, keys key0 + KG j, every DP-th piece of d.
  const int dp = tid % DP, key0 = tid / DP % KG, row0 = tid / (DP * KG) * RT;
  // Output: rows orow .. orow + RT - 1, four elements from d0 on, tokens t0 .. t0 + TV - 1.
  const int d0 = lane % (32 / Sh::LK) * 4, lk = lane / (32 / Sh::LK);
  const int orow = warp % Sh::WR * RT, wk = warp / Sh::WR, t0 = (wk * Sh::LK + lk) * TV;

  // A token of the loading cursor's tile: its page, looked up a tile ahead of the copy.
  int page = -2, place = 0;
  auto lookup = [&]() {
    const int t = ld.tile * kTK + tid;
    page = -2;
    if (tid < kTK && t < ld.u.keys) {
      const int slot = page_slot(P.C, t);
      place = t - slot * P.C.page_size;
      page = P.S.table[(long long)ld.u.b * P.S.stride + slot];
    }
  };
  // The offsets of tile n, and the next one's lookup.
  auto resolve = [&](int n) {
    if (tid < kTK) {
      const bool ok = page >= 0 && page < P.C.n_pages;
      if (!ok && page != -2) set_status(P.status, SV_DATA_BAD_PAGE);
      s_off[n % 2 * kTK + tid] = ok ? page * P.C.page_b + place * P.C.token_b + ld.u.head * P.C.head_b : -1;
      const unsigned all = __ballot_sync(kFull, ok);
      if (lane == 0) s_valid[n % 2 * 2 + warp] = all;
    }
    if (n + 1 < n_tiles) {
      if (++ld.tile == ld.u.tiles) next_unit<MT>(P, ld);
      lookup();
    }
  };
  auto copy = [&](int n, const char* from, char* to, int pitch) {
    if (n < n_tiles) {
      const uint32_t base = smem_addr(to) + tid % CPR * 16;
      const char* src = from + tid % CPR * 16;
      constexpr int kRows = 128 / CPR, kAhead = 8;  // rows that the CTA copies at once; offsets read together
#pragma unroll
      for (int j = 0; j < kTK / kRows; j += kAhead) {
        long long off[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) off[e] = s_off[n % 2 * kTK + tid / CPR + (j + e) * kRows];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          cp16(base + (tid / CPR + (j + e) * kRows) * pitch, src + (off[e] < 0 ? 0 : off[e]), off[e] >= 0);
      }
    }
    cp_commit();
  };
  lookup();
  resolve(0);
  __syncthreads();
  copy(0, P.C.k, s_k, Sh::kPitch);
  copy(0, P.C.v, s_v, D * 4);

  float4 o[RT];
  float m[NR], l[NR];  // maxima of the rows so far, and sums over the keys key0 + KG j
  int lo[NR], hi[NR];
  // The thread's rows of the scores it is left with: each halving over the DP threads takes a bit of dp, rows first.
  int my_row = row0, my_key = 0;
  {
    int nr = RT, nk = KT;
#pragma unroll
    for (int x = 1; x < DP; x <<= 1) {
      if (nr > 1) {
        nr /= 2;
        if (dp & x) my_row += nr;
      } else {
        nk /= 2;
        if (dp & x) my_key += nk;
      }
    }
  }
  bool begun = false, from_start = false;
  for (int i = 0; i < n_tiles; ++i) {
    if (i + 1 == n_tiles) release_stream();
    const int rows = cp.u.w.rows * P.group;
    if (!begun) {
      begun = true;
      from_start = cp.tile == 0;
      float4 qv[(MT * D / 4 + 127) / 128];
#pragma unroll
      for (int j = 0; j < (MT * D / 4 + 127) / 128; ++j) {
        const int x = tid + j * 128, r = cp.u.mt * MT + x / (D / 4);
        qv[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < MT * D / 4 && r < rows) {
          const int w = r / P.group, h = cp.u.head * P.group + (r - w * P.group);
          qv[j] = reinterpret_cast<const float4*>(P.q + (long long)(cp.u.w.r0 + w) * P.q_row_b + (long long)h * (D * 4))[x % (D / 4)];
        }
      }
#pragma unroll
      for (int j = 0; j < (MT * D / 4 + 127) / 128; ++j)
        if (tid + j * 128 < MT * D / 4) reinterpret_cast<float4*>(s_q)[tid + j * 128] = qv[j];
#pragma unroll
      for (int e = 0; e < NR; ++e) {
        m[e] = -INFINITY;
        l[e] = 0.f;
        const int r = cp.u.mt * MT + my_row + e;
        const int w = r < rows ? r / P.group : 0;
        lo[e] = r < rows ? candidate_start(P, cp.u.w, w) : 0;
        hi[e] = r < rows ? w : -1 - cp.u.ctx;
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (i + 1 < n_tiles) resolve(i + 1);
    cp_wait<1>();
    __syncthreads();  // K has landed

    // Scores.
    float s[RT * KT];
#pragma unroll
    for (int e = 0; e < RT * KT; ++e) s[e] = 0.f;
    {
      const char* kr = s_k + key0 * Sh::kPitch + dp * 16;
      const float4* qr = reinterpret_cast<const float4*>(s_q + row0 * D) + dp;
#pragma unroll 2
      for (int d = 0; d < CPR; d += DP) {
        float4 k4[KT];
#pragma unroll
        for (int j = 0; j < KT; ++j) k4[j] = *reinterpret_cast<const float4*>(kr + j * KG * Sh::kPitch + d * 16);
#pragma unroll
        for (int e = 0; e < RT; ++e) {
          const float4 q4 = qr[e * CPR + d];
#pragma unroll
          for (int j = 0; j < KT; ++j) {
            float& x = s[e * KT + j];
            x = fmaf(q4.x, k4[j].x, fmaf(q4.y, k4[j].y, fmaf(q4.z, k4[j].z, fmaf(q4.w, k4[j].w, x))));
          }
        }
      }
    }
    // The DP threads' sums joined: each exchange leaves a thread half of its scores.
    sum_halves<RT * KT, 1, DP>(s, dp);
#pragma unroll
    for (int e = 0; e < NR * NK; ++e) s[e] *= P.scale_log2;
    if ((cp.tile + 1) * kTK > cp.u.ctx || (s_valid[i % 2 * 2] & s_valid[i % 2 * 2 + 1]) != kFull) {
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        const int key = key0 + (my_key + j) * KG, at = cp.tile * kTK + key - cp.u.ctx;
        const bool page_ok = s_valid[i % 2 * 2 + key / 32] >> key % 32 & 1;
#pragma unroll
        for (int e = 0; e < NR; ++e) {
          const bool see = page_ok && (at < 0 ? hi[e] >= -cp.u.ctx : at >= lo[e] && at <= hi[e]);
          if (!see) s[e * NK + j] = -INFINITY;
        }
      }
    }
    // Softmax: the rows' maxima over the warp, then over the warps that share them; the sums stay apart until the unit's end.
    float top[NR];
#pragma unroll
    for (int e = 0; e < NR; ++e) {
      top[e] = s[e * NK];
#pragma unroll
      for (int j = 1; j < NK; ++j) top[e] = fmaxf(top[e], s[e * NK + j]);
    }
#pragma unroll
    for (int x = RT / NR; x < 32; x <<= 1)
#pragma unroll
      for (int e = 0; e < NR; ++e) top[e] = fmaxf(top[e], __shfl_xor_sync(kFull, top[e], x));
    if (Sh::WK > 1 && lane < RT / NR)
#pragma unroll
      for (int e = 0; e < NR; ++e) s_top[warp % Sh::WK * MT + my_row + e] = top[e];
    __syncthreads();  // K is free
    copy(i + 1, P.C.k, s_k, Sh::kPitch);
#pragma unroll
    for (int e = 0; e < NR; ++e) {
      if constexpr (Sh::WK > 1)
#pragma unroll
        for (int y = 0; y < Sh::WK; ++y) top[e] = fmaxf(top[e], s_top[y * MT + my_row + e]);
      top[e] = fmaxf(top[e], m[e]);
      const float off_m = top[e] == -INFINITY ? 0.f : top[e], f = m[e] == -INFINITY ? 0.f : ex2(m[e] - top[e]);
      m[e] = top[e];
      if (warp % Sh::WK == 0 && lane < RT / NR) s_f[my_row + e] = f;
      float p[NK];
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        p[j] = ex2(s[e * NK + j] - off_m);
        s_p[(my_row + e) * SP + key0 + (my_key + j) * KG] = p[j];
      }
      float sum = p[0] + p[1];
      if constexpr (NK == KT)
        sum += p[2] + p[3];
      else
        sum += __shfl_xor_sync(kFull, sum, RT / NR);
      l[e] = fmaf(l[e], f, sum);
    }
    cp_wait<1>();
    __syncthreads();  // the weights are written and V has landed
    // The product with V.
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float f = s_f[orow + r];
      o[r] = make_float4(o[r].x * f, o[r].y * f, o[r].z * f, o[r].w * f);
    }
#pragma unroll 2
    for (int k = t0; k < t0 + TV; k += 4) {
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float4*>(s_v + (k + j) * (D * 4) + d0 * 4);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float4 p = *reinterpret_cast<const float4*>(s_p + (orow + r) * SP + k);
        o[r].x = fmaf(p.x, v[0].x, fmaf(p.y, v[1].x, fmaf(p.z, v[2].x, fmaf(p.w, v[3].x, o[r].x))));
        o[r].y = fmaf(p.x, v[0].y, fmaf(p.y, v[1].y, fmaf(p.z, v[2].y, fmaf(p.w, v[3].y, o[r].y))));
        o[r].z = fmaf(p.x, v[0].z, fmaf(p.y, v[1].z, fmaf(p.z, v[2].z, fmaf(p.w, v[3].z, o[r].z))));
        o[r].w = fmaf(p.x, v[0].w, fmaf(p.y, v[1].w, fmaf(p.z, v[2].w, fmaf(p.w, v[3].w, o[r].w))));
      }
    }
    __syncthreads();  // V is free

    const bool unit_end = cp.tile + 1 == cp.u.tiles;
    if (unit_end || i + 1 == n_tiles) {
      begun = false;
#pragma unroll
      for (int x = DP; x < 32; x <<= 1)
#pragma unroll
        for (int e = 0; e < NR; ++e) l[e] += __shfl_xor_sync(kFull, l[e], x);
      if (lane < RT / NR)
#pragma unroll
        for (int e = 0; e < NR; ++e) {
          s_l[warp % Sh::WK * MT + my_row + e] = l[e];
          if (warp % Sh::WK == 0) s_m[my_row + e] = m[e];
        }
      if constexpr (Sh::LK > 1) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          o[r].x += __shfl_xor_sync(kFull, o[r].x, 16);
          o[r].y += __shfl_xor_sync(kFull, o[r].y, 16);
          o[r].z += __shfl_xor_sync(kFull, o[r].z, 16);
          o[r].w += __shfl_xor_sync(kFull, o[r].w, 16);
        }
      }
      if constexpr (Sh::WK > 1) {  // the warps' shares of the tokens, joined in the place of V
        float4* buf = reinterpret_cast<float4*>(s_v);
        if (wk > 0 && lk == 0)
#pragma unroll
          for (int r = 0; r < RT; ++r) buf[((wk - 1) * MT + orow + r) * CPR + d0 / 4] = o[r];
      }
      __syncthreads();
      if constexpr (Sh::WK > 1) {
        const float4* buf = reinterpret_cast<const float4*>(s_v);
        if (wk == 0)
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int y = 0; y < Sh::WK - 1; ++y) {
              const float4 z = buf[(y * MT + orow + r) * CPR + d0 / 4];
              o[r] = make_float4(o[r].x + z.x, o[r].y + z.y, o[r].z + z.z, o[r].w + z.w);
            }
        __syncthreads();
      }
      const bool split = !from_start || !unit_end;
      if (tid == 0 && i + 1 == n_tiles) tell_cut(L, sh, cp, !unit_end && from_start);
      if (wk == 0) {
        float* part = reinterpret_cast<float*>(L.part + (size_t)(blockIdx.x * 2 + (from_start ? 1 : 0)) * part_bytes<D, MT>());
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if (r % Sh::LK != lk) continue;  // the parts of a warp write a row each
          float sum = s_l[orow + r];
#pragma unroll
          for (int y = 1; y < Sh::WK; ++y) sum += s_l[y * MT + orow + r];
          if (split) {
            reinterpret_cast<float4*>(part + (orow + r) * D)[d0 / 4] = o[r];
            if (d0 == 0) {
              part[MT * D + orow + r] = s_m[orow + r];
              part[MT * D + MT + orow + r] = sum;
            }
            continue;
          }
          const int x = cp.u.mt * MT + orow + r;
          if (x >= rows) break;
          const int w = x / P.group, h = cp.u.head * P.group + (x - w * P.group);
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          reinterpret_cast<float4*>(P.out + (long long)(cp.u.w.r0 + w) * P.out_row_b + (long long)h * (D * 4))[d0 / 4] =
              make_float4(o[r].x * inv, o[r].y * inv, o[r].z * inv, o[r].w * inv);
          if (P.lse && d0 == 0) P.lse[(long long)(cp.u.w.r0 + w) * (P.C.n_heads * P.group) + h] = lse_of(s_m[orow + r], sum, 1.f);
        }
      }
    }
    copy(i + 1, P.C.v, s_v, D * 4);
    if (++cp.tile == cp.u.tiles && i + 1 < n_tiles) next_unit<MT>(P, cp);
  }
  cp_wait<0>();
}

// Joins the parts of a unit that several CTAs share. Block c takes the unit
// that CTA c's share cuts at its end, if it began there. A group of D / 4
// threads holds a row, 4 elements a thread, with four or eight parts' loads in
// flight. A unit of up to eight parts has a row to each group, and no barrier
// (64 requests of 2000 tokens and one head: 31 us a call; with the parts dealt
// out from five on, 35); one of more parts (a long request on an otherwise idle
// machine) has them dealt to the groups of a block, whose sums are joined in
// order (38 parts of one token's unit: eight in flight 15.1 us a call, four
// 16.4). The block is brought up while the parts are still being computed and
// waits for them.
constexpr int kJoinT = 128;

struct RowSum {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void add_row(RowSum& a, float m, float l, const float4& o, float scale) {
  const float top = fmaxf(a.m, m), fa = factor(a.m, top, scale), fb = factor(m, top, scale);
  a.m = top;
  a.l = fmaf(l, fb, a.l * fa);
  a.o = make_float4(fmaf(o.x, fb, a.o.x * fa), fmaf(o.y, fb, a.o.y * fa), fmaf(o.z, fb, a.o.z * fa), fmaf(o.w, fb, a.o.w * fa));
}

template <int DT, int D, int MT>
__global__ void __launch_bounds__(kJoinT) join_kernel(Params P, Plan L, int grid) {
  const float scale = DT == 1 ? P.scale_log2 : 1.f;  // of the maxima: the fp32 kernel's scores are scaled
  constexpr int TPR = D / 4, kG = kJoinT / TPR;
  __shared__ RowSum s_sum[kG][TPR];
  release_stream();
  wait_for_stream();
  const int c = blockIdx.x;
  const int4 cut = *reinterpret_cast<const int4*>(L.cut + c * 8);
  const int last = min(L.cut[c * 8 + 4], grid - 1);
  if (cut.y <= 0) return;
  const int head = cut.z, mt = cut.w;
  const int rows = min(MT, cut.y * P.group - mt * MT);  // of this row tile
  const int g = threadIdx.x / TPR, lane_d = threadIdx.x % TPR;
  // Row r of N parts k0, k0 + step, ..., their loads in flight together.
  auto add_parts = [&](auto n, RowSum& sum, int r, int k0, int step) {
    constexpr int N = decltype(n)::value;
    float m[N], l[N];
    float4 o[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int k = k0 + j * step;
      m[j] = -INFINITY;
      l[j] = 0.f;
      o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k <= last) {
        const float* part = reinterpret_cast<const float*>(L.part + (size_t)(k * 2 + (k == c)) * part_bytes<D, MT>());
        m[j] = part[MT * D + r];
        l[j] = part[MT * D + MT + r];
        o[j] = *reinterpret_cast<const float4*>(part + r * D + lane_d * 4);
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) add_row(sum, m[j], l[j], o[j], scale);
  };
  auto write = [&](const RowSum& sum, int r) {
    const int x = mt * MT + r, ww = x / P.group, h = head * P.group + (x - ww * P.group);
    const float inv = sum.l > 0.f ? 1.f / sum.l : 0.f;
    const float4 o = make_float4(sum.o.x * inv, sum.o.y * inv, sum.o.z * inv, sum.o.w * inv);
    char* dst = P.out + (long long)(cut.x + ww) * P.out_row_b + ((long long)h * D + lane_d * 4) * Elem<DT>::kBytes;
    if constexpr (DT == 1)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
    else
      *reinterpret_cast<float4*>(dst) = o;
    if (P.lse && lane_d == 0) P.lse[(long long)(cut.x + ww) * (P.C.n_heads * P.group) + h] = lse_of(sum.m, sum.l, scale);
  };
  const RowSum none{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  auto row_a_group = [&](auto n) {
    for (int r = blockIdx.y * kG + g; r < rows; r += gridDim.y * kG) {
      RowSum sum = none;
      add_parts(n, sum, r, c, 1);
      write(sum, r);
    }
  };
  constexpr std::integral_constant<int, 4> four;
  constexpr std::integral_constant<int, 8> eight;
  if (last - c < 4) return row_a_group(four);
  if (last - c < 8) return row_a_group(eight);
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    RowSum sum = none;
    if (last - c < kG * 4)
      add_parts(four, sum, r, c + g, kG);
    else
      for (int k0 = c + g; k0 <= last; k0 += kG * 8) add_parts(eight, sum, r, k0, kG);
    s_sum[g][lane_d] = sum;
    __syncthreads();
    if (g == 0) {
#pragma unroll
      for (int j = 1; j < kG; ++j) {
        const RowSum y = s_sum[j][lane_d];
        add_row(sum, y.m, y.l, y.o, scale);
      }
      write(sum, r);
    }
    __syncthreads();
  }
}

constexpr int kGrid = 152 * 4;  // CTAs of the pipeline, at most

// A kernel over the shares, then the join: it is brought up while the shares are computed, and waits for their end.
template <int DT, int D, typename Sh>
cudaError_t launch_shares(void (*kernel)(Params, Plan), const Params& P, const Plan& L, cudaStream_t st,
                          std::atomic<unsigned long long>& allowed) {
  static_assert(Sh::kCtas * Sh::MT <= 256, "the workspace has room for the partial results");
  const int grid = 152 * Sh::kCtas;
  cudaError_t e = allow_smem(kernel, Sh::smem, allowed);
  if (e == cudaSuccess) e = launch_overlapped(kernel, dim3(grid), Sh::kT, Sh::smem, 1, st, P, L);
  if (e == cudaSuccess)
    e = launch_overlapped(join_kernel<DT, D, Sh::MT>, dim3(grid, Sh::MT <= 16 ? 4 : Sh::MT <= 64 ? 8 : 16), kJoinT, 0, 1, st, P, L, grid);
  return e;
}
template <int D, int WM>
cudaError_t launch_mma(const Params& P, const Plan& L, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed{0};
  return launch_shares<1, D, Shape<D, WM>>(window_mma_kernel<D, WM>, P, L, st, allowed);
}
template <int D>
cudaError_t launch_tc(const Params& P, const Plan& L, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed{0};
  return launch_shares<1, D, TcShape<D>>(window_tc_kernel<D>, P, L, st, allowed);
}
template <int D, int M>
cudaError_t launch_fma(const Params& P, const Plan& L, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed{0};
  return launch_shares<0, D, Shape32<D, M>>(window_fma_kernel<D, M>, P, L, st, allowed);
}
template <int D>
cudaError_t launch_rows32(long long rows, const Params& P, const Plan& L, cudaStream_t st) {
  return rows <= 4    ? launch_fma<D, 4>(P, L, st)
         : rows <= 8  ? launch_fma<D, 8>(P, L, st)
         : rows <= 16 ? launch_fma<D, 16>(P, L, st)
                      : launch_fma<D, 32>(P, L, st);
}

}  // namespace att
}  // namespace sv

extern "C" {

size_t sv_window_attention_workspace_size(const sv_kv_cache* cache, int32_t n_q_heads, int32_t R) {
  if (!cache || (cache->head_dim != 64 && cache->head_dim != 128) || n_q_heads < 1 || R < 0) return 0;
  // The cuts, then two partial results a CTA: of any kernel, 256 rows an SM at most.
  return (size_t)sv::att::kGrid * 32 + 2 * (size_t)152 * 256 * ((size_t)cache->head_dim + 2) * 4;
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
  if (layer < 0 || layer >= P.C.n_layers || !(std::fabs(scale) < 0x1p127f)) return SV_ERR_INVALID_ARG;
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
  att::Plan L{};
  L.cut = static_cast<int*>(workspace);
  L.part = static_cast<char*>(workspace) + att::kGrid * 32;
  // Row tiles as high as the windows' mean number of stacked rows.
  const long long rows = ((long long)R * P.group + P.S.n - 1) / P.S.n;
  cudaError_t e;
  if (es == 2) {
    P.q_mask = 0xffffffffu;
    if (P.scale_log2 == 0.f) {
      P.scale_log2 = 1.f;
      P.q_mask = 0u;
    }
    if (P.scale_log2 < 0.f) {
      P.scale_log2 = -P.scale_log2;
      P.q_sign = 0x80008000u;
    }
    if (D == 128)
      e = rows <= 16   ? att::launch_mma<128, 1>(P, L, st)
          : rows <= 32 ? att::launch_mma<128, 2>(P, L, st)
          : rows <= 64 ? att::launch_mma<128, 4>(P, L, st)
                       : att::launch_tc<128>(P, L, st);
    else
      e = rows <= 16   ? att::launch_mma<64, 1>(P, L, st)
          : rows <= 32 ? att::launch_mma<64, 2>(P, L, st)
                       : att::launch_tc<64>(P, L, st);
  } else if (D == 128) {
    e = att::launch_rows32<128>(rows, P, L, st);
  } else {
    e = att::launch_rows32<64>(rows, P, L, st);
  }
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
