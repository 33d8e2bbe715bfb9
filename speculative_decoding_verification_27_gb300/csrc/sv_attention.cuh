// sv_attention.cuh -- what the attention kernels share: their parameters, the
// cut of the work into equal shares and the join of what the cuts leave, and
// the instructions that they are made of.
#pragma once

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
  // With shared prefixes (kShared) there are two passes. In the first, a request is a
  // group of sequences, its window all of their rows and its tokens the
  // prefix; what it finds goes to `base`. In the second, sequence b leaves out
  // its first pre[b] tokens and starts from what base holds of them.
  int n_req;                 // requests of the pass
  const int4* groups;        // first pass: first row, rows, tokens, sequence whose table leads to them; else null
  const int* pre;            // second pass, [n]; else null
  float* base;               // [R n_q_heads][D] sums of a row
  float2* base_ml;           // and their maximum (to base two) and sum
};

// ---------------------------------------------------------------------------
// The list of key tiles and its shares
// ---------------------------------------------------------------------------
constexpr int kTK = 64;    // tokens of a key tile (TK below, where a kernel has tiles of its own)

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
  long long rows;      // mean stacked rows of a request (of the host's)
};

struct Unit {
  int b, head, mt;     // request, key-value head, row tile
  int keys, tiles;     // tokens, key tiles
  Window w;
  int n_mt, ctx;
  int seq, first;      // row of the page table; tokens before the pass's
};

// Request b's window, tokens and key tiles, and its number of row tiles (0 tiles where there is nothing to do).
template <int MT, bool kWarp, int TK, bool kShared>
__device__ __forceinline__ void load_request(const Params& P, int b, Unit& u, bool tell) {
  u.b = u.seq = b;
  u.first = 0;
  if (kShared && P.groups) {  // what the plan has looked over
    const int4 g = P.groups[b];
    u.w = Window{0, 1, g.x, g.y};
    u.seq = g.w;
    u.ctx = u.keys = g.y > 0 ? g.z : 0;
    u.tiles = (u.keys + TK - 1) / TK;
    u.n_mt = (int)(((long long)g.y * P.group + MT - 1) / MT);
    return;
  }
  u.w = find_window<kWarp>(P.W, b);
  u.ctx = P.S.ctx[b];
  const bool len = length_ok(P.C, P.S, u.ctx), fits = len && length_ok(P.C, P.S, (long long)u.ctx + max(u.w.rows, 0));
  if (u.w.rows <= 0 || !fits) {
    if (tell && (u.w.rows < 0 || !fits))
      set_status(P.status, u.w.rows < 0 ? SV_DATA_BAD_OFFSETS : len ? SV_DATA_BAD_PAGE : SV_DATA_BAD_SEQ);
    u.keys = u.tiles = u.n_mt = 0;
    return;
  }
  if (kShared && P.pre) {
    u.first = P.pre[b];
    u.ctx -= u.first;
  }
  u.keys = u.ctx + u.w.rows;
  u.tiles = (u.keys + TK - 1) / TK;
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
template <int MT, int kThr, bool kShared, int TK = kTK>
__device__ __forceinline__ bool take_share(const Params& P, const Plan& L, Share& sh, Cursor& c) {
  wait_for_stream();
  __shared__ long long s_scan[kThr / 32];
  __shared__ Unit s_unit;
  __shared__ long long s_first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (P.n_req + kThr - 1) / kThr;
  long long mine = 0;
  for (int b = tid * per; b < min((tid + 1) * per, P.n_req); ++b) {
    load_request<MT, false, TK, kShared>(P, b, c.u, blockIdx.x == 0);
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
        load_request<MT, false, TK, kShared>(P, b, c.u, false);
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
template <int MT, bool kShared, int TK = kTK>
__device__ __forceinline__ void next_unit(const Params& P, Cursor& c) {
  c.tile = 0;
  if (++c.u.mt < c.u.n_mt) return;
  c.u.mt = 0;
  if (++c.u.head < P.C.n_heads) return;
  c.u.head = 0;
  for (int b = c.u.b + 1; b < P.n_req; ++b) {
    load_request<MT, true, TK, kShared>(P, b, c.u, false);
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

// First place of window row w of the unit that it sees of the window: its candidate's.
template <bool kShared>
__device__ __forceinline__ int first_seen(const Params& P, const Unit& u, int w) {
  return kShared && P.groups ? 0 : candidate_start(P.W, u.w, w);
}
// Where base holds the row of query head h of window row w.
__device__ __forceinline__ long long base_row(const Params& P, const Unit& u, int w, int h) {
  return (long long)(u.w.r0 + w) * (P.C.n_heads * P.group) + h;
}
// A maximum to base two (and what goes by it) as one of scores that are scaled by `scale`: the factor that the rounding takes.
__device__ __forceinline__ float unscaled(float m2, float scale, float& fix) {
  const float m = m2 == -INFINITY ? m2 : m2 / scale;
  fix = m2 == -INFINITY ? 0.f : ex2(m2 - __fmul_rn(m, scale));
  return m;
}

// ---------------------------------------------------------------------------
// Caches of 8 bits
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Four e4m3 values as f16, which holds them exactly.
__device__ __forceinline__ void e4m3_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
// x >= 0 up to a power of two, and the inverse of such a power.
__device__ __forceinline__ float pow2_above(float x) { return __uint_as_float((__float_as_uint(x) + 0x7fffffu) & 0x7f800000u); }
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }
// The power of two that brings a row of that largest magnitude to 2^7 .. 2^8 (at most 2^125, so that its inverse is a normal number).
__device__ __forceinline__ float pow2_of_row(float most) {
  const uint32_t e = __float_as_uint(most) & 0x7f800000u;
  return most > 0.f ? __uint_as_float(min((127u + 7u + 127u << 23) - e, 252u << 23)) : 1.f;
}
// What the scores of a row that was multiplied by `up` are scaled by: positive and finite, as maxima of -inf are multiplied by it.
__device__ __forceinline__ float row_scale(float scale_log2, float up) {
  return fminf(fmaxf(scale_log2 * pow2_inverse(up), 0x1p-126f), 0x1p127f);
}

// Bytes of one partial result: MT rows of D sums, then their maxima and sums.
template <int D, int MT>
constexpr size_t part_bytes() {
  return (size_t)MT * (D + 2) * 4;
}

// ---------------------------------------------------------------------------
// The fifth-generation tensor cores
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t umma_desc(uint32_t addr, uint32_t lead_bytes) {
  // 128-byte swizzle, eight rows of 128 bytes an atom of 1024 bytes; atoms follow each other.
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lead_bytes >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
constexpr uint32_t umma_idesc(int n, bool b_mn_major, bool f16 = false) {
  return 1u << 4 | (f16 ? 0u : 1u << 7 | 1u << 10) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (uint32_t)(128 / 16) << 24;
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

static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
  for (int it = 0; it < kSpinLimit; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  set_status(status, SV_DEV_COPY_TIMEOUT);
  return false;
}

// ---------------------------------------------------------------------------
// The join
// ---------------------------------------------------------------------------
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

// DT: 0 fp32, 1 bf16, 2 bf16 over a cache of 8 bits.
template <int DT, int D, int MT, bool kShared>
__global__ void __launch_bounds__(kJoinT) join_kernel(Params P, Plan L, int grid) {
  const float scale = DT == 1 ? P.scale_log2 : 1.f;  // of the maxima: the other kernels' are scaled
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
    if (kShared && P.groups) {
      const long long at = (long long)(cut.x + ww) * (P.C.n_heads * P.group) + h;
      *reinterpret_cast<float4*>(P.base + at * D + lane_d * 4) = sum.o;
      if (lane_d == 0) P.base_ml[at] = make_float2(sum.m == -INFINITY ? sum.m : __fmul_rn(sum.m, scale), sum.l);
      return;
    }
    const float inv = sum.l > 0.f ? 1.f / sum.l : 0.f;
    const float4 o = make_float4(sum.o.x * inv, sum.o.y * inv, sum.o.z * inv, sum.o.w * inv);
    char* dst = P.out + (long long)(cut.x + ww) * P.out_row_b + ((long long)h * D + lane_d * 4) * (DT == 0 ? 4 : 2);
    if constexpr (DT != 0)
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

// The kernels over a cache of 8 bits, by the mean number of stacked rows of a request.
cudaError_t launch_e4m3(int D, long long rows, const Params& P, const Plan& L, cudaStream_t st);

// A kernel over the shares, then the join: it is brought up while the shares are computed, and waits for their end.
template <int DT, int D, typename Sh, bool kShared>
cudaError_t launch_shares(void (*kernel)(Params, Plan), const Params& P, const Plan& L, cudaStream_t st,
                          std::atomic<unsigned long long>& allowed) {
  static_assert(Sh::kCtas * Sh::MT <= 256, "the workspace has room for the partial results");
  const int grid = 152 * Sh::kCtas;
  cudaError_t e = allow_smem(kernel, Sh::smem, allowed);
  if (e == cudaSuccess) e = launch_overlapped(kernel, dim3(grid), Sh::kT, Sh::smem, 1, st, P, L);
  // Blocks side by side for a unit's rows: some, or, where the units are so few that a share holds an eighth of one at most, up to
  // sixteen. 16 forks of 4096 tokens (64 stacked rows, 38 parts a head), a whole call of sv_prefix_attention: 8 blocks 52 us, 16 43,
  // 32 42, 64 48; 5 groups of 3 in fp32, where a block has less to do: 38, 39, 46, 55.
  const int some = Sh::MT <= 16 ? 4 : Sh::MT <= 64 ? 8 : 16, all = (int)(L.rows < 16 ? L.rows : 16);
  const int rows = (long long)P.n_req * P.C.n_heads * 8 <= grid && all > some ? all : some;
  if (e == cudaSuccess)
    e = launch_overlapped(join_kernel<DT, D, Sh::MT, kShared>, dim3(grid, rows), kJoinT, 0, 1, st, P, L, grid);
  return e;
}

}  // namespace att
}  // namespace sv
