// attention8.cu -- attention of the verify windows over a cache of 8 bits.
//
// A key stands for ks_t times its e4m3 values, a value for vs_t times its own:
//   s_t = scale ks_t (q . k8_t),  out = sum_t softmax_t vs_t v8_t,
// so the scales go to the scores and to the weights, one product each, and the
// tensor cores take the cached bytes as they lie in memory. The other operand
// of each product is split in two terms, x = a + b with a = rn_e4m3(x) and b
// the rest as e5m2, eight bits between them (as many as bf16 has), whose
// products go to the same fp32 sums:
//   q      a row is brought to a largest magnitude of 2^7 .. 2^8 by a power of
//          two, which its scores' factor takes back. A bf16 value is the sum
//          of its terms exactly down to 2^-13 of the row's largest, and below
//          off by at most 2^-21 of that.
//   P      the weights p_t vs_t, relative to M, the largest vs_t up to a power
//          of two, and to a reference of the row that may lag behind its
//          maximum by 2^6; scaled so that they are at most 2^8. Off by 2^-8 of
//          themselves (and 2^-11, as f16), or by 2^-16 relative to the
//          reference. The sums are multiplied by M in the end. (With 2^3 in
//          the place of 2^6 a third of the tiles moved a reference, each for
//          4000 cycles.)
//
// The products are taken transposed: S^T = K Q^T, its rows the 128 tokens of a
// tile, and O^T = V^T P^T, its rows the elements of a head, so that the tensor
// cores' 128 rows are full however few rows a window has. With mma.sync (e4m3
// is taken apart into f16 there, two instructions and the conversions for one
// product) the benchmark batch's windows over 1024 - 4096 tokens took 527 us;
// this way 389, of which the bytes at the copy rate are 212. What bounds it is
// the chain of a tile in a CTA (S^T, its 128 maxima and weights a thread, their
// two terms, O^T), about 3500 cycles, two CTAs an SM, and what a unit takes to
// begin and to end, 7 - 9 us of a CTA: the same keys as 32 windows over 20480
// tokens, 256 over 2560 and 1024 over 640 take 257, 312 and 457 us (135 tiles a
// CTA in 0.8, 6.7 and 27 units).
//
// Windows of more than 64 rows go to window_tc_kernel, which takes a tile as
// f16 under 128 rows at once.
#include "sv_window.cuh"

namespace sv {
namespace att {

// Four f16 values as their two terms. An e5m2 value is the upper byte of an f16.
__device__ __forceinline__ void two_terms(uint32_t h01, uint32_t h23, uint32_t& a, uint32_t& b) {
  uint32_t r01, r23;
  asm("{\n\t.reg .b16 p, q;\n\t.reg .b32 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 p, %3;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, %4;\n\tmov.b32 %0, {p, q};\n\t"
      "cvt.rn.f16x2.e4m3x2 x, p;\n\tcvt.rn.f16x2.e4m3x2 y, q;\n\tsub.rn.f16x2 %1, %3, x;\n\tsub.rn.f16x2 %2, %4, y;\n\t}"
      : "=&r"(a), "=&r"(r01), "=&r"(r23)
      : "r"(h01), "r"(h23));
  b = __byte_perm(r01 + 0x00800080u, r23 + 0x00800080u, 0x7531);
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp16_all(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void umma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// Rows of `row` bytes (32, 64 or 128), swizzled over them, eight rows a group,
// or of 16 bytes one after another. Where the rows are the contraction's index
// the blocks along the other one are `lead` bytes apart.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, int row, uint32_t lead) {
  if (row == 16) lead = 128;  // here the groups of eight
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(row * 8 >> 4) << 32 | 1ull << 46 |
         (row == 128 ? 2ull : row == 64 ? 4ull : row == 32 ? 6ull : 0ull) << 61;
}
// A of e4m3; B of N rows, of e4m3 or e5m2; both by the contraction's index first, or last.
constexpr uint32_t tile_idesc(int n, bool mn_major, bool e5m2) {
  return 1u << 4 | (e5m2 ? 1u << 10 : 0u) | (mn_major ? 3u << 15 : 0u) | (uint32_t)(n / 8) << 17 | (uint32_t)(128 / 16) << 24;
}
// Chunk c (16 bytes) of row r of such a tile.
template <int kRow>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (uint32_t)(r * kRow + ((c ^ (kRow == 128 ? r & 7 : kRow == 64 ? (r >> 1) & 3 : kRow == 32 ? (r >> 2) & 1 : 0)) << 4));
}

// N values of each of 32 lanes joined over them (a maximum or a sum), through 128 N bytes of shared memory of the warp's: lane l
// is left with value l % N. (By shuffles it is six times the code, which is run too rarely to stay near.)
template <int N, bool kMax>
__device__ __forceinline__ float join_lanes(const float (&v)[N], char* buf, int lane) {
  constexpr int C = N / 4;
  const uint32_t to = smem_addr(buf) + lane * (N * 4);
#pragma unroll
  for (int c = 0; c < C; ++c)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + ((c ^ (lane & (C - 1))) << 4)), "f"(v[4 * c]), "f"(v[4 * c + 1]),
                 "f"(v[4 * c + 2]), "f"(v[4 * c + 3]) : "memory");
  __syncwarp();
  const int r = lane & (N - 1);
  float x = kMax ? -INFINITY : 0.f;
#pragma unroll 4
  for (int l = 0; l < 32; ++l) {
    const float y = *reinterpret_cast<const float*>(buf + l * (N * 4) + (((r / 4) ^ (l & (C - 1))) << 4) + (r & 3) * 4);
    x = kMax ? fmaxf(x, y) : x + y;
  }
  __syncwarp();
  return x;
}

constexpr int kTK8 = 128;     // tokens of a key tile: the rows of S^T
constexpr float kHead = 2.f;  // weights are 2^2 at the reference

template <int D, int N>
struct Shape8 {
  static constexpr int MT = N;                            // stacked rows of a unit: 16, 32 or 64
  static constexpr int RG = N < 32 ? N : 32;              // rows of a softmax group
  static constexpr int G = N / RG;                        // softmax groups, of four warps
  static constexpr int kCopy = G * 4;                     // the first of the warps that copy: two for K, one for V
  static constexpr int kMmaWarp = G * 4 + 3;
  static constexpr int kT = (kMmaWarp + 1) * 32;
  static constexpr int kCtas = N == 64 ? 1 : 2;           // an SM
  static constexpr int S = N == 64 ? (D == 64 ? 6 : 3) : (D == 64 ? 4 : 2);  // tiles of K, and of V
  static constexpr int R = S + 2;                         // tiles whose scales and lookups are kept
  static constexpr int kTile = kTK8 * D;                  // bytes of K (or V) of a tile
  static constexpr int kQ = N * D;                        // bytes of a unit's rows, one term
  static constexpr int kP = N * kTK8;                     // bytes of the weights of a tile, one term
  static constexpr int kCols = 4 * N;                     // TMEM columns (a power of two): O^T, two S^T
  static constexpr int kJoin = G == 1 ? 0 : G * 4 * 128 * RG;  // bytes to join lanes in; one group takes the place of its P^T
  static constexpr size_t smem = 1024 + 4 * kQ + 4 * kP + (size_t)S * 2 * kTile + (size_t)R * 2 * kTK8 * 4 + kJoin;
  static_assert(kQ % 1024 == 0 && kP % 1024 == 0 && kTile % 1024 == 0 && kCols * kCtas <= 512, "");
};

template <int S>
struct Bars8 {
  uint64_t k_full[S], k_empty[S];  // a tile of K (and its scales) has landed; its product has ended
  uint64_t v_full[S], v_empty[S];
  uint64_t s_full[2];              // S^T has been computed
  uint64_t p_ready[2];             // S^T has been read, P^T written, O^T rescaled
  uint64_t o_done[2];              // a tile's product with V has ended
  uint64_t q_full[2], q_empty[2];
  uint64_t o_free;                 // a unit's O^T has been read
  uint64_t checked[2];             // a softmax group's threads have looked at their scores
  uint64_t met[2];                 // a softmax group's threads have come to a unit's end, or to a move of the reference
  uint64_t looked[S + 2];          // a tile's byte offsets are written
  uint64_t end;                    // every product has ended
};

__device__ __forceinline__ void tc_ld4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// wait_long with a microsecond or two a try, so that the waiting warps leave the others the SM.
static __device__ __noinline__ bool wait_asleep(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
  for (int it = 0; it < kSpinLimit; ++it) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (done) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  set_status(status, SV_DEV_COPY_TIMEOUT);
  return false;
}
// Roles, joined by mbarriers only:
//   G groups of 4 warps   softmax and output, 32 (or 16) rows each: a thread
//                owns a token of the tile, and then an element of the head;
//   2 warps      copies: the rows of Q in their two terms, tiles of K gathered
//                over the pages into a ring of swizzled ones, and the scales;
//   1 warp       the tiles of V;
//   the last     issues the products, S^T of a tile, then O^T of the one
//                before it. K's place is free a softmax earlier than V's.
// Every wait is bounded, as in window_tc_kernel, a softmax group's for one
// another too: a warp whose wait gave up leaves, and the others' waits give up
// behind it.
//
// Only the warps of K walk over the units: what the others need to know of a
// tile lies in a ring beside its offsets. (With a cursor in every role the
// code was 148 KB, and the parts that run once a unit took 8000 cycles and
// more for the instructions to arrive.)
struct TileInfo {
  int ctx, tile;       // the unit's tokens before the window, and the tile's place among its tiles
  int rows, row0;      // stacked rows from the row tile on, and the first one
  int head, r0, first;
  int flags;           // 1: the unit's last tile here; 2: its last of all; 4: it begins a unit here
};

template <int D, int N>
__global__ void __launch_bounds__(Shape8<D, N>::kT, Shape8<D, N>::kCtas) window_tc8_kernel(Params P, Plan L) {
  using Sh = Shape8<D, N>;
  constexpr int S = Sh::S, R = Sh::R, G = Sh::G, RG = Sh::RG, TK = kTK8;
  extern __shared__ char smem_raw[];
  __shared__ Bars8<S> bars;
  __shared__ __align__(16) float s_sc[4][N];   // rows of a unit: what their scores are scaled by,
  __shared__ int2 s_see[4][N];                 // and the window places that they see (units in flight: fewer than four)
  // A softmax warp's own: of its rows, what is added to the scores, and factors.
  __shared__ __align__(16) float s_off[G * 4][RG];
  __shared__ __align__(16) float s_f[G * 4][RG];
  __shared__ __align__(16) float s_g[G * 4][RG];
  __shared__ char* s_dst[G * 4][RG];           // where a row's output goes,
  __shared__ const float* s_src[G * 4][RG];    // and what base holds of it
  __shared__ float s_red[2][G][4][RG];
  __shared__ float s_top[G][4];
  __shared__ long long s_at[R][TK];            // byte offsets of a tile's tokens, -1 where there is nothing
  __shared__ uint32_t s_valid[R][4];           // the tokens that have a page
  __shared__ TileInfo s_info[R];
  __shared__ int s_over[2][4];                 // a softmax group's tile has a weight that is too large
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  Share sh;
  Cursor c;
  if (!take_share<N, Sh::kT, true, TK>(P, L, sh, c)) return;
  const int n_tiles = (int)(sh.t1 - sh.t0);

  char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t q_base = smem_addr(smem), p_base = q_base + 4 * Sh::kQ, k_base = p_base + 4 * Sh::kP, v_base = k_base + S * Sh::kTile;
  float* s_scale = reinterpret_cast<float*>(smem + 4 * Sh::kQ + 4 * Sh::kP + S * 2 * Sh::kTile);  // [R][2][TK]
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_addr(&bars.k_full[i]), 2 * (32 + 1));
      mbar_init(smem_addr(&bars.k_empty[i]), 1);
      mbar_init(smem_addr(&bars.v_full[i]), 32);
      mbar_init(smem_addr(&bars.v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.checked[i]), 128);
      mbar_init(smem_addr(&bars.met[i]), 128);
      mbar_init(smem_addr(&bars.s_full[i]), 1);
      mbar_init(smem_addr(&bars.p_ready[i]), G * 128);
      mbar_init(smem_addr(&bars.o_done[i]), 1);
      mbar_init(smem_addr(&bars.q_full[i]), 2 * 32);
      mbar_init(smem_addr(&bars.q_empty[i]), 1);
    }
    for (int i = 0; i < R; ++i) mbar_init(smem_addr(&bars.looked[i]), 2);
    mbar_init(smem_addr(&bars.o_free), G * 128);
    mbar_init(smem_addr(&bars.end), 1);
    s_abort = 0;
    for (int i = 0; i < 8; ++i) s_over[i >> 2][i & 3] = 0;
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
  auto wait = [&](uint64_t& bar, int parity) {
    return mbar_try_wait(smem_addr(&bar), (uint32_t)parity) || wait_asleep(smem_addr(&bar), (uint32_t)parity, &s_abort, P.status);
  };
  const uint32_t s_col = tmem + N;  // the first S^T, behind O^T
  // Rows t0 .. t0 + n - 1 of a tile, by a warp: zeros where there is no page, and behind the sequence.
  auto copy_rows = [&](const char* from, uint32_t to, const long long* offsets, int t0, int n, bool whole) {
    constexpr int CPR = D / 16, RPP = 32 / CPR;  // 16-byte chunks of a row, rows that the warp copies at once
    const int first = lane / CPR;
    const char* src = from + lane % CPR * 16;
    offsets += t0 + first;
    uint32_t dst = to + tile_at<D>(first, lane % CPR) + t0 * D;
#pragma unroll 1
    for (int r0 = 0; r0 < n; r0 += 8 * RPP, offsets += 8 * RPP, dst += 8 * RPP * D) {
      long long off[8];  // read together, before the copies order them
#pragma unroll
      for (int e = 0; e < 8; ++e) off[e] = offsets[e * RPP];
      // Eight rows further the swizzle is the same again; within them its bits are the row's own and e's.
      if (whole) {
#pragma unroll
        for (int e = 0; e < 8; ++e) cp16_all((dst ^ tile_at<D>(e * RPP % 8, 0) % D) + e * RPP * D, src + off[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          cp16((dst ^ tile_at<D>(e * RPP % 8, 0) % D) + e * RPP * D, src + (off[e] < 0 ? 0 : off[e]), off[e] >= 0);
      }
    }
  };
  if (warp == Sh::kCopy + 2) {
    // ------------------------------------------------------------- tiles of V
    bool alive = true;
    for (int i = 0; i < n_tiles && alive; ++i) {
      alive = __all_sync(kFull, wait(bars.looked[i % R], (i / R) & 1) && (i < S || wait(bars.v_empty[i % S], (i / S - 1) & 1)));
      if (!alive) break;
      copy_rows(P.C.v, v_base + (i % S) * Sh::kTile, s_at[i % R], 0, TK, (s_valid[i % R][0] & s_valid[i % R][1] & s_valid[i % R][2] & s_valid[i % R][3]) == kFull);
      cp_arrive(smem_addr(&bars.v_full[i % S]));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= Sh::kCopy && warp < Sh::kCopy + 2) {
    // ---------------------------------------------- tiles of K, scales, rows of Q
    const int j = warp - Sh::kCopy;
    bool alive = true;
    int unit = 0;  // units whose rows are loaded
    // A unit's rows, eight elements a lane: the two warps bring half of them each.
    auto load_q = [&](const Cursor& u) {
      if (unit >= 2) alive = __all_sync(kFull, wait(bars.q_empty[unit & 1], ((unit >> 1) - 1) & 1));
      if (!alive) return;
      constexpr int LPR = D / 8, RPP = 32 / LPR, M = N / (2 * RPP);  // lanes of a row, rows of a warp at once, times
      const uint32_t qb = q_base + (unit & 1) * 2 * Sh::kQ;
      const int rows = u.u.w.rows * P.group - u.u.mt * N, d0 = lane % LPR * 8;
      const int r_first = j * (N / 2) + lane / LPR;
      // The 16 bytes of a lane go, eight and eight, to where its terms will lie: all copies are in flight together, and neither loop
      // is unrolled.
#pragma unroll 1
      for (int m = 0; m < M; ++m) {
        const int r = r_first + m * RPP, x = u.u.mt * N + r, w = x / P.group, h = x - w * P.group;
        const char* src = P.q;
        if (r < rows) src += (long long)(u.u.w.r0 + w) * P.q_row_b + ((long long)(u.u.head * P.group + h) * D + d0) * 2;
        const uint32_t to = qb + (d0 & 8) + tile_at<D>(r, d0 / 16);
        cp8(to, src, r < rows);
        cp8(to + Sh::kQ, src + 8, r < rows);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
      for (int m = 0; m < M; ++m) {
        const int r = r_first + m * RPP;
        const uint32_t at = (d0 & 8) + tile_at<D>(r, d0 / 16);
        uint2* pa = reinterpret_cast<uint2*>(smem + (unit & 1) * 2 * Sh::kQ + at);
        uint2* pb = reinterpret_cast<uint2*>(smem + (unit & 1) * 2 * Sh::kQ + Sh::kQ + at);
        uint32_t b[4] = {pa->x, pa->y, pb->x, pb->y}, most = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          b[e] = (b[e] & P.q_mask) ^ P.q_sign;
          most = __vmaxu2(most, b[e] & 0x7fff7fffu);
        }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) most = __vmaxu2(most, __shfl_xor_sync(kFull, most, o));
        const float up = pow2_of_row(__uint_as_float(max(most & 0xffffu, most >> 16) << 16));
        uint32_t f[4], lo[2], hi[2];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = pack_f16(__uint_as_float(b[e] << 16) * up, __uint_as_float(b[e] & 0xffff0000u) * up);
        two_terms(f[0], f[1], lo[0], hi[0]);
        two_terms(f[2], f[3], lo[1], hi[1]);
        *pa = make_uint2(lo[0], lo[1]);
        *pb = make_uint2(hi[0], hi[1]);
        if (d0 == 0) s_sc[unit & 3][r] = row_scale(P.scale_log2, up);
      }
      if (lane < N / 2) {  // what a row sees of its window; past the window nothing
        const int r = j * (N / 2) + lane, x = u.u.mt * N + r;
        s_see[unit & 3][r] = r < rows ? make_int2(first_seen<true>(P, u.u, x / P.group), x / P.group) : make_int2(0x7fffffff, -1);
      }
      fence_proxy_async_smem();
      mbar_arrive(smem_addr(&bars.q_full[unit & 1]));
      ++unit;
    };
    int page[2], place[2];
    bool from_start = true;  // tile i's unit begins here
    for (int i = -1; i < n_tiles && alive; ++i) {
      const int ring = i % R;
      bool whole = true;
      if (i >= 0) {
        if (i >= S) alive = __all_sync(kFull, wait(bars.k_empty[i % S], (i / S - 1) & 1));
        if (!alive) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool ok = page[h] >= 0 && page[h] < P.C.n_pages;
          if (!ok && page[h] != -2) set_status(P.status, SV_DATA_BAD_PAGE);
          const int t = j * 64 + h * 32 + lane;
          s_at[ring][t] = ok ? page[h] * P.C.page_b + place[h] * P.C.token_b + c.u.head * P.C.head_b : -1;
          const long long so = ok ? page[h] * P.C.s_page + place[h] * P.C.s_token + c.u.head * P.C.s_head : 0;
          const uint32_t to = smem_addr(s_scale + ring * 2 * TK + t);
          cp4(to, P.C.ks + so, ok);
          cp4(to + TK * 4, P.C.vs + so, ok);
          const unsigned m = __ballot_sync(kFull, ok);
          whole &= m == kFull;
          if (lane == 0) s_valid[ring][j * 2 + h] = m;
        }
        const bool end = c.tile + 1 == c.u.tiles, last = end || i + 1 == n_tiles;
        if (i == 0 || c.tile == 0) from_start = c.tile == 0;
        if (j == 0 && lane == 0) {
          s_info[ring] = TileInfo{c.u.ctx, c.tile, c.u.w.rows * P.group - c.u.mt * N, c.u.mt * N, c.u.head, c.u.w.r0, c.u.first,
                                  (last ? 1 : 0) | (end ? 2 : 0) | (from_start ? 4 : 0)};
          if (i + 1 == n_tiles) tell_cut(L, sh, c, !end && from_start);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&bars.looked[ring]));
        if (i + 1 < n_tiles && ++c.tile == c.u.tiles) next_unit<N, true, TK>(P, c);
      }
      // The next tile's pages, two tokens a lane, looked up before this one's copies.
      if (i + 1 < n_tiles) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = c.tile * TK + j * 64 + h * 32 + lane;
          page[h] = -2;
          place[h] = 0;
          if (k < c.u.keys) {
            const int slot = page_slot(P.C, k + c.u.first);
            place[h] = k + c.u.first - slot * P.C.page_size;
            page[h] = P.S.table[(long long)c.u.seq * P.S.stride + slot];
          }
        }
      }
      if (i >= 0) {
        copy_rows(P.C.k, k_base + (i % S) * Sh::kTile, s_at[ring], j * 64, 64, whole);
        cp_arrive(smem_addr(&bars.k_full[i % S]));
        if (lane == 0) mbar_arrive(smem_addr(&bars.k_full[i % S]));  // releases what lane 0 wrote
      }
      if (i + 1 < n_tiles && (i < 0 || c.tile == 0)) load_q(c);  // the next tile begins a unit
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == Sh::kMmaWarp) {
    // -------------------------------------------------------------- products
    // S^T of a tile, then O^T of the one before it, whose weights are computed meanwhile. (Whichever is ready first, by polling,
    // took half of the SM's instructions.)
    bool alive = true, first = true, begun = false;  // S^T to come begins its unit; O^T holds a product of its unit
    bool ends[2] = {false, false};                   // the tile ends its unit here
    int unit = 0, pv_unit = 0;
    const uint64_t q_desc = tile_desc(q_base, D, 16), k_desc = tile_desc(k_base, D, 16);
    // With heads of 64 the rows of O^T from 64 on are the others again.
    const uint64_t v_desc = tile_desc(v_base, D, 0), p_desc = tile_desc(p_base, N, 0);
    auto wait_all = [&](uint64_t& bar, int parity) { return __all_sync(kFull, wait(bar, parity & 1)) != 0; };
    for (int i = 0; i <= n_tiles && alive; ++i) {
      if (i < n_tiles) {
        if (first) alive = wait_all(bars.q_full[unit & 1], unit >> 1);
        alive = alive && wait_all(bars.k_full[i % S], i / S);
        if (!alive) break;
        const bool last = s_info[i % R].flags & 1;
        fence_proxy_async_smem();  // the copies wrote the tile through the generic proxy, the products read it through the other
        tc_fence_after();
        if (elect_one()) {
          const uint64_t qd = q_desc + (uint64_t)((unit & 1) * 2 * Sh::kQ / 16), kd = k_desc + (uint64_t)((i % S) * Sh::kTile / 16);
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            umma_fp8(s_col + (i & 1) * N, kd + k * 2, qd + k * 2, tile_idesc(N, false, false), k > 0);
            umma_fp8(s_col + (i & 1) * N, kd + k * 2, qd + Sh::kQ / 16 + k * 2, tile_idesc(N, false, true), true);
          }
          umma_commit(smem_addr(&bars.s_full[i & 1]));
          umma_commit(smem_addr(&bars.k_empty[i % S]));
          if (last) umma_commit(smem_addr(&bars.q_empty[unit & 1]));
        }
        ends[i & 1] = last;
        first = last;
        unit += last;
      }
      if (i > 0) {
        const int v = i - 1;
        alive = wait_all(bars.p_ready[v & 1], v >> 1) && wait_all(bars.v_full[v % S], v / S) &&
                (begun || pv_unit == 0 || wait_all(bars.o_free, pv_unit - 1));
        if (!alive) break;
        fence_proxy_async_smem();
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vd = v_desc + (uint64_t)((v % S) * Sh::kTile / 16), pd = p_desc + (uint64_t)((v & 1) * 2 * Sh::kP / 16);
#pragma unroll
          for (int k = 0; k < TK / 32; ++k) {
            umma_fp8(tmem, vd + k * (32 * D / 16), pd + k * (32 * N / 16), tile_idesc(N, true, false), k > 0 || begun);
            umma_fp8(tmem, vd + k * (32 * D / 16), pd + (Sh::kP + k * 32 * N) / 16, tile_idesc(N, true, true), true);
          }
          umma_commit(smem_addr(&bars.v_empty[v % S]));
          umma_commit(smem_addr(&bars.o_done[v & 1]));
        }
        begun = !ends[v & 1];
        pv_unit += ends[v & 1];
      }
    }
    if (elect_one()) umma_commit(smem_addr(&bars.end));
    __syncwarp();
    for (int it = 0; it < kSpinLimit && !__all_sync(kFull, mbar_try_wait(smem_addr(&bars.end), 0)); ++it) {
    }
  } else {
    // --------------------------------------------------- softmax and output
    const int g = G == 1 ? 0 : warp >> 2, wq = warp & 3, tok = tid & 127, row0 = g * RG;  // the group, the token, the group's first row
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t o_addr = tmem + lanes + row0;
    bool fresh = true;
    int unit = 0, phase = 0, met_phase = 0;
    float top_v = 0.f, ref = -INFINITY;  // M, and the reference of the group's row `lane`
    f2_t l[RG / 2];                      // the rows' sums over the thread's tokens
#pragma unroll
    for (int r = 0; r < RG / 2; ++r) l[r] = 0ull;
    float *my_off = s_off[warp], *my_f = s_f[warp], *my_g = s_g[warp];
    // To join lanes: in the place of P^T, where no product reads and no thread of the group writes it, or beside the other group's.
    char* my_buf = smem + 4 * Sh::kQ + (G == 1 ? 0 : 4 * Sh::kP + S * 2 * Sh::kTile + R * 2 * TK * 4) + warp * (128 * RG);
    static_assert(G > 1 || 4 * 128 * RG <= 4 * Sh::kP, "P^T has room for every warp");
    // A barrier of the group's threads; false, for the whole warp, where it gave up.
    auto meet = [&]() {
      mbar_arrive(smem_addr(&bars.met[g]));
      const bool ok = wait(bars.met[g], met_phase);
      met_phase ^= 1;
      return __all_sync(kFull, ok) != 0;
    };
    if (lane < RG) my_off[lane] = 0.f;
    __syncwarp();
    for (int i = 0; i < n_tiles; ++i) {
      if (i + 1 == n_tiles) release_stream();
      const int b = i & 1, ring = i % R;
      // (The scales and what was written beside a unit's rows are there too: S^T waited for them. Their own barriers may have gone
      // on to a later phase.)
      const bool ok = wait(bars.s_full[b], (i >> 1) & 1) && (i < 2 || wait(bars.o_done[b], ((i >> 1) - 1) & 1));  // and P^T is free
      if (!__all_sync(kFull, ok)) goto out;
      tc_fence_after();
      uint32_t a[RG];
      auto load_scores = [&]() {
#pragma unroll
        for (int r = 0; r < RG; r += 16) tc_ld16(*reinterpret_cast<uint32_t(*)[16]>(a + r), s_col + lanes + b * N + row0 + r);
      };
      load_scores();
      const TileInfo T = s_info[ring];  // (behind the weights its place may be another tile's)
      const float ks = s_scale[ring * 2 * TK + tok], vs = s_scale[ring * 2 * TK + TK + tok];
      const uint32_t* valid = s_valid[ring];
      const bool here = valid[wq] >> lane & 1u;
      const bool masked = (T.tile + 1) * TK > T.ctx || (valid[0] & valid[1] & valid[2] & valid[3]) != kFull;
      uint32_t seen = 0xffffffffu;  // bit r: the group's row r sees the token
      if (masked) {
        const int at = T.tile * TK + tok - T.ctx;  // the token's place in the window, below zero in the history
        seen = 0u;
#pragma unroll 4
        for (int r = 0; r < RG; ++r) {
          const int2 w = s_see[unit & 3][row0 + r];  // first and last place, none past the window
          seen |= (uint32_t)(((at < 0) & (w.x != 0x7fffffff)) | ((at >= w.x) & (at <= w.y))) << r;
        }
        if (!here) seen = 0u;
      }
      float t[RG];
      // At first the reference is found: a unit's first tile moves it to begin with, another one only where it has to.
      for (bool move = fresh, checked = fresh;;) {
        // The rows' scores to base two and what is added to them; -inf where the row does not see the token.
        {
          const float* sc = s_sc[unit & 3] + row0;
          const f2_t k2 = f2_splat(ks);
          tc_wait_ld();
#pragma unroll
          for (int r = 0; r < RG; r += 4) {
            const float4 f = *reinterpret_cast<const float4*>(sc + r), o = *reinterpret_cast<const float4*>(my_off + r);
            f2_unpack(f2_fma(f2_mul(f2_pack(__uint_as_float(a[r]), __uint_as_float(a[r + 1])), k2), f2_pack(f.x, f.y), f2_pack(o.x, o.y)),
                      t[r], t[r + 1]);
            f2_unpack(f2_fma(f2_mul(f2_pack(__uint_as_float(a[r + 2]), __uint_as_float(a[r + 3])), k2), f2_pack(f.z, f.w), f2_pack(o.z, o.w)),
                      t[r + 2], t[r + 3]);
          }
          if (masked) {
#pragma unroll
            for (int r = 0; r < RG; ++r)
              if (!(seen >> r & 1u)) t[r] = -INFINITY;
          }
        }
        if (move) {
          // The reference moves to the rows' maxima so far, M to the largest scale; each warp finds the same.
          move = false;
          if (!fresh) {
            if (!__all_sync(kFull, wait(bars.o_done[b ^ 1], ((i - 1) >> 1) & 1))) goto out;  // O^T is at rest, and both P^T are free
            if (!meet()) goto out;                                                           // once all are through with weights that do not count
          }
          const float mine = join_lanes<RG, true>(t, my_buf, lane);
          if (lane < RG) s_red[0][g][wq][lane] = mine;
          const uint32_t most_v = __reduce_max_sync(kFull, here ? __float_as_uint(vs) : 0u);
          if (lane == 0) s_top[g][wq] = __uint_as_float(most_v);
          if (!meet()) goto out;
          const float top =
              pow2_above(fmaxf(fmaxf(fmaxf(s_top[g][0], s_top[g][1]), fmaxf(s_top[g][2], s_top[g][3])), fmaxf(top_v, 0x1p-120f)));
          const float fv = top_v > 0.f ? top_v * pow2_inverse(top) : 1.f;
          top_v = top;
          if (lane < RG) {
            const float old = ref;
            ref = fmaxf(fmaxf(fmaxf(s_red[0][g][0][lane], s_red[0][g][1][lane]), fmaxf(s_red[0][g][2][lane], s_red[0][g][3][lane])) -
                            my_off[lane],
                        old);
            my_off[lane] = kHead - ref;  // (inf for a row that has seen nothing: whatever it sees next moves the reference)
            my_f[lane] = factor(old, ref, 1.f);
          }
          __syncwarp();
          if (!fresh) {
#pragma unroll
            for (int r = 0; r < RG / 2; ++r) l[r] = f2_mul(l[r], f2_pack(my_f[2 * r], my_f[2 * r + 1]));
            tc_fence_after();
#pragma unroll 1
            for (int r = 0; r < RG; r += 16) {
              uint32_t o[16];
              tc_ld16(o, o_addr + r);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * (my_f[r + e] * fv));
              tc_st16(o_addr + r, o);
            }
            tc_wait_st();
          }
          fresh = false;
          load_scores();
          continue;
        }
        if (!checked) {
          // A weight above 2^8, the largest that its terms hold (with a margin for the logarithm), or a sum that may leave fp32, moves
          // the reference. The group's answer is only waited for behind the weights.
          float most = t[0];
#pragma unroll
          for (int r = 1; r < RG; ++r) most = fmaxf(most, t[r]);
          if (most > fminf(7.99f - __log2f(vs * pow2_inverse(top_v)), 100.f)) s_over[g][i & 3] = 1;
          mbar_arrive(smem_addr(&bars.checked[g]));
        }
        // The weights, in their two terms: 16 rows of one token are 16 bytes. t becomes the weights without V's scale.
        const float vm = vs * pow2_inverse(top_v);
        const uint32_t pb = p_base + b * 2 * Sh::kP;
#pragma unroll
        for (int r = 0; r < RG; ++r) t[r] = ex2(t[r]);
#pragma unroll
        for (int r = 0; r < RG; r += 16) {
          uint32_t x[4], y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float* p = t + r + e * 4;
            two_terms(pack_f16(p[0] * vm, p[1] * vm), pack_f16(p[2] * vm, p[3] * vm), x[e], y[e]);
          }
          const uint32_t to = pb + tile_at<N>(tok, (row0 + r) / 16);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + Sh::kP), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
        }
        if (checked) break;
        checked = true;
        if (!__all_sync(kFull, wait(bars.checked[g], phase))) goto out;
        phase ^= 1;
        move = *(volatile int*)&s_over[g][i & 3] != 0;
        if (!move) break;
        if (lane < RG && ref == -INFINITY) my_off[lane] = 0.f;
        __syncwarp();
        load_scores();
      }
#pragma unroll
      for (int r = 0; r < RG / 2; ++r) l[r] = f2_add(l[r], f2_pack(t[2 * r], t[2 * r + 1]));
      if (tok == 0) s_over[g][(i + 2) & 3] = 0;  // two tiles on: nobody is there yet, and all have read what it said two tiles ago
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(smem_addr(&bars.p_ready[b]));
      if (T.flags & 1) {
        // The rows' sums over the tokens, then the output: a thread an element of the head. Each warp works out the rows' factors.
        float sums[RG];
#pragma unroll
        for (int r = 0; r < RG / 2; ++r) f2_unpack(l[r], sums[2 * r], sums[2 * r + 1]);
        if (!__all_sync(kFull, wait(bars.o_done[b], (i >> 1) & 1))) goto out;
        const float mine = join_lanes<RG, false>(sums, my_buf, lane);
        if (lane < RG) s_red[1][g][wq][lane] = mine;
        if (!meet()) goto out;
        const bool from_start = T.flags & 4, split = (T.flags & 6) != 6;
        const int rows = min(N, T.rows) - row0;                 // of the group
        const bool based = T.first > 0 && from_start && rows > 0;  // goes on from what the first pass found (a group without a row has none)
        const bool wide = split || P.groups;                    // fp32 sums, or the output itself
        if (lane < RG) {
          float* part = reinterpret_cast<float*>(L.part + (size_t)(blockIdx.x * 2 + (from_start ? 1 : 0)) * part_bytes<D, N>());
          const int r = row0 + min(lane, max(rows - 1, 0)), x = T.row0 + r, w = x / P.group, h = T.head * P.group + (x - w * P.group);
          const long long row = (long long)(T.r0 + w) * (P.C.n_heads * P.group) + h;
          const bool mine_to_write = wq == 0 && lane < rows;
          float sum = (s_red[1][g][0][lane] + s_red[1][g][1][lane] + s_red[1][g][2][lane] + s_red[1][g][3][lane]) * 0x1p-2f;
          float own = top_v * 0x1p-2f, of_base = 0.f;
          if (based) {
            const float2 ml = P.base_ml[row];
            const float top = fmaxf(ref, ml.x), fa = factor(ref, top, 1.f);
            of_base = factor(ml.x, top, 1.f);
            sum = sum * fa + ml.y * of_base;
            own *= fa;
            ref = top;
          }
          char* dst;
          if (split) {
            dst = reinterpret_cast<char*>(part + r * D);
            if (mine_to_write) {
              part[N * D + r] = ref;
              part[N * D + N + r] = sum;
            }
          } else if (P.groups) {
            dst = reinterpret_cast<char*>(P.base + row * D);
            if (mine_to_write) P.base_ml[row] = make_float2(ref, sum);
          } else {
            dst = P.out + (long long)(T.r0 + w) * P.out_row_b + (long long)h * (D * 2);
            const float inv = sum > 0.f ? 1.f / sum : 0.f;
            own *= inv;
            of_base *= inv;
            if (P.lse && mine_to_write) P.lse[row] = lse_of(ref, sum, 1.f);
          }
          my_f[lane] = own;
          my_g[lane] = of_base;
          s_dst[warp][lane] = dst;
          s_src[warp][lane] = P.base + row * D;
        }
        __syncwarp();
        tc_fence_after();
        const int d = D == 128 ? tok : tok & (D - 1);  // (with heads of 64 the upper half has the same again)
        // Four rows at a time. A row behind the last is the last one again, and not written.
#pragma unroll 1
        for (int r = 0; r < RG; r += 4) {
          uint32_t o[4];
          tc_ld4(o, o_addr + r);
          char* dst[4];
          float v[4], add[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            dst[x] = s_dst[warp][r + x];
            add[x] = based ? s_src[warp][r + x][d] : 0.f;
          }
          tc_wait_ld();
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = fmaf(add[x], my_g[r + x], __uint_as_float(o[x]) * my_f[r + x]);
          if (tok >= D) continue;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (r + x >= rows) break;
            if (wide)
              reinterpret_cast<float*>(dst[x])[d] = v[x];
            else
              reinterpret_cast<__nv_bfloat16*>(dst[x])[d] = __float2bfloat16_rn(v[x]);
          }
        }
        __syncwarp();
        tc_fence_before();
        mbar_arrive(smem_addr(&bars.o_free));
#pragma unroll
        for (int r = 0; r < RG / 2; ++r) l[r] = 0ull;
        top_v = 0.f;
        ref = -INFINITY;
        if (lane < RG) my_off[lane] = 0.f;
        __syncwarp();
        fresh = true;
        ++unit;
      }
    }
  }
out:
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == Sh::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kCols) : "memory");
}

template <int D, int N>
cudaError_t launch_tc8(const Params& P, const Plan& L, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed{0};
  return launch_shares<2, D, Shape8<D, N>, true>(window_tc8_kernel<D, N>, P, L, st, allowed);
}

template <int D>
cudaError_t launch_tc_f16(const Params& P, const Plan& L, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed{0};
  return launch_shares<2, D, TcShape<D>, true>(window_tc_kernel<D, true, true>, P, L, st, allowed);
}

template <int D>
cudaError_t launch_rows8(long long rows, const Params& P, const Plan& L, cudaStream_t st) {
  return rows <= 16   ? launch_tc8<D, 16>(P, L, st)
         : rows <= 32 ? launch_tc8<D, 32>(P, L, st)
         : rows <= 64 ? launch_tc8<D, 64>(P, L, st)
                      : launch_tc_f16<D>(P, L, st);
}

// Up to 64 rows the products of the cached bytes; above, tiles as f16 under 128 rows, each tile read by half as many units: windows
// of 4 - 192 rows over 17 - 8192 tokens, heads of 64: 350 us, with units of 64 rows 524; 64 rows over 1024 - 4096 tokens, heads of
// 128: the bytes' products 189 us, the other 288.
cudaError_t launch_e4m3(int D, long long rows, const Params& P, const Plan& L, cudaStream_t st) {
  return D == 128 ? launch_rows8<128>(rows, P, L, st) : launch_rows8<64>(rows, P, L, st);
}

}  // namespace att
}  // namespace sv
