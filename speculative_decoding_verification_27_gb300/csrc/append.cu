// append.cu -- rows on their way into the cache: queries and keys normed and
// rotated, keys and values written to their pages, in 8 bits where the cache
// holds those.
//
// With x a head's row in fp32, y = x g / sqrt(mean x^2 + eps); angle j of the
// row's position turns y's elements (j, j + rot/2), or (2j, 2j + 1), from
// (u, w) to (u cos - w sin, w cos + u sin). In 8 bits a row is
// rn_e4m3(y 448 / a) with the scale a / 448, a = max |y|.
//
// Bound by the bytes: every row is read once and written once. A lane holds
// twice eight elements of a head, those that are turned with one another, and
// 4, 8 or 16 lanes hold a head: sums and maxima go by two to four shuffles.
#include "sv_append.cuh"
#include "sv_launch.cuh"

#include <cuda_bf16.h>

namespace sv {
namespace app {

constexpr int kT = 256;
constexpr int kU = 2;  // groups of heads of a warp
template <bool ROPE>
constexpr int kCtas = ROPE ? 2 : 3;  // an SM

struct Params {
  CacheView C;
  SeqView S;
  WindowView W;
  int layer, n_layers, D, n_q;
  const char* q;
  const char* k;
  const char* v;
  char* out;
  long long q_b, out_b, new_b, new_layer_b;  // row strides in bytes, and the layers' of k and v
  const float* cos_sin;
  long long cs_stride;
  int n_pos, half, pairs;
  float eps, inv_D;
  const char* g_q;
  const char* g_k;
  const int32_t* positions;
  uint32_t* status;
};

// Eight elements of a row as they lie in memory.
template <int DT>
struct Raw {
  uint4 v[DT == 0 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Raw<DT> load(const char* p) {
  Raw<DT> r;
  r.v[0] = *reinterpret_cast<const uint4*>(p);
  if constexpr (DT == 0) r.v[1] = *reinterpret_cast<const uint4*>(p + 16);
  return r;
}
template <int DT>
__device__ __forceinline__ void store(char* p, const Raw<DT>& r) {
  *reinterpret_cast<uint4*>(p) = r.v[0];
  if constexpr (DT == 0) *reinterpret_cast<uint4*>(p + 16) = r.v[1];
}
template <int DT>
__device__ __forceinline__ void unpack(const Raw<DT>& r, float (&f)[8]) {
  if constexpr (DT == 0) {
    const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <int DT>
__device__ __forceinline__ Raw<DT> pack(const float (&f)[8]) {
  Raw<DT> r;
  if constexpr (DT == 0) {
    r.v[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    r.v[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  } else {
    r.v[0] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)hi << 16 | lo;
}

// A warp's ring of rows on their way: kU groups of heads, and the row's angles.
template <int DT, bool ROPE, int L>
struct Ring {
  static constexpr int kPart = 32 * 8 * Elem<DT>::kBytes;       // bytes of eight elements a lane; a group of heads has two such parts
  static constexpr int kSlot = 2 * kU * kPart + (ROPE ? L * 64 : 0);
  static constexpr int kSlots = DT == 0 ? 2 : 3;
  static constexpr int kBytes = kSlots * kSlot;
};
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// DT: the rows' type (0 fp32, 1 bf16). Q8: the cache holds 8 bits. ROPE: there
// are queries, norms and angles. L: lanes of a head.
//
// A warp takes up to kU groups of heads, all queries, all keys or all values,
// of a row, and goes on to the same of other rows, of which two (in fp32 one)
// are on their way while one is worked on. Pages are looked up for 32 rows at once. Norm
// and rotation are out = (x A + y B) / sqrt(mean x^2 + eps) with y the element
// that x is turned with, A = g cos and B = (y's g) (+-sin): worked out once
// for the row's heads. 64 prompts of 1000 rows, 48 heads of 128, in bf16: 262
// us (91% of the copy rate); keys and values alone into 8 bits: 65 us (91%).
// With each head's angles and weights applied one after another instructions
// bound it (496 us), as with eight elements a lane, whose partners lie in
// another lane (367 us); neighbouring parts in one lane make half sectors of
// every access (101 us for the second). kPartly: some elements are not turned,
// and y has no part in them, as it may be an infinity or a NaN (the same rows
// packed side by side, half of a head turned: 282 us, and 315 by pairs, where
// the others take 275 and 285).
template <int DT, bool Q8, bool ROPE, int L, bool kPairs, bool kPartly>
__global__ void __launch_bounds__(kT, kCtas<ROPE>) append_rows_kernel(const __grid_constant__ Params P) {
  release_stream();
  wait_for_stream();
  using Rg = Ring<DT, ROPE, L>;
  constexpr int es = Elem<DT>::kBytes, kH = 32 / L, kPer = kU * kH;  // heads of a group, of a warp
  extern __shared__ __align__(16) char smem[];
  char* ring = smem + (threadIdx.x >> 5) * Rg::kBytes;
  const int lane = threadIdx.x & 31, sub = lane / L, j = lane % L;
  const CacheView& C = P.C;
  const int n_q = ROPE ? P.n_q : 0, n_k = C.n_heads;
  const int q_chunks = (n_q + kPer - 1) / kPer, k_chunks = (n_k + kPer - 1) / kPer, chunks = q_chunks + 2 * k_chunks;
  const int warp = blockIdx.x * (kT / 32) + (threadIdx.x >> 5), row_step = (int)(gridDim.x * (kT / 32)) / chunks;
  const int chunk = warp % chunks, row_first = warp / chunks;
  if (row_first >= row_step) return;
  const bool is_q = chunk < q_chunks, is_v = chunk >= q_chunks + k_chunks;
  const int h0 = (is_q ? chunk : is_v ? chunk - q_chunks - k_chunks : chunk - q_chunks) * kPer + sub, heads = is_q ? n_q : n_k;
  const long long head_b = (long long)P.D * es;
  // The lane's two parts of a head, of eight elements: those that are turned with one another, or any; neighbouring lanes have
  // neighbouring parts, so that what they read and write lies together.
  const int h8 = P.half / 8, n_parts = P.D / 8;
  const bool turn = ROPE && P.half && !is_v, across = ROPE && !kPairs;
  const int before = across ? (j < h8 ? 0 : 2 * h8) : 0, k = across && j >= h8 ? j - h8 : j;
  const int ahead = across && j < h8 ? h8 : (n_parts - before + 1) / 2;  // parts of the half
  const int d0 = k < ahead ? (before + k) * 8 : P.D, d1 = k < ahead ? (before + ahead + k) * 8 : P.D;  // (P.D: none)
  const bool turned0 = turn && d0 < 2 * P.half, turned1 = turn && d1 < 2 * P.half;
  const char* g = is_q ? P.g_q : is_v ? nullptr : P.g_k;
  Raw<DT> g0{}, g1{};
  if (ROPE && g) {
    if (d0 < P.D) g0 = load<DT>(g + d0 * es);
    if (d1 < P.D) g1 = load<DT>(g + d1 * es);
  }
  const uint32_t ring_at = smem_addr(ring) + lane * (8 * es);
  const long long group_b = kH * head_b, to_group = kH * C.head_b, to_lane = h0 * C.head_b;
  const long long scale_group = kH * C.s_head, scale_lane = h0 * C.s_head;
  uint32_t have = 0u;  // bits 2u and 2u + 1: the lane's parts of a head of group u are there
#pragma unroll
  for (int u = 0; u < kU; ++u) have |= (uint32_t)(h0 + u * kH < heads && d0 < P.D) << (2 * u) | (uint32_t)(h0 + u * kH < heads && d1 < P.D) << (2 * u + 1);
  for (int b = blockIdx.y; b < P.S.n; b += gridDim.y) {
    const int len = P.S.ctx[b];
    const Window w = find_window<true>(P.W, b);
    if (w.rows < 0 || !length_ok(C, P.S, len)) {
      if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0)
        set_status(P.status, w.rows < 0 ? SV_DATA_BAD_OFFSETS : SV_DATA_BAD_SEQ);
      continue;
    }
    const int32_t* table = P.S.table + (long long)b * P.S.stride;
    for (int l = blockIdx.z; l < P.n_layers; l += gridDim.z) {
      // The rows' places go on by steps: the addresses of each worked out anew were half of the instructions.
      const long long src_step = (is_q ? P.q_b : P.new_b) * row_step;
      const char* src = (is_q ? P.q : (is_v ? P.v : P.k) + l * P.new_layer_b) + (w.r0 + (long long)row_first) * (is_q ? P.q_b : P.new_b) +
                        h0 * head_b;
      char* out = P.out + (w.r0 + (long long)row_first) * P.out_b + h0 * head_b;
      const bool plain = !P.positions && !P.W.cand;
      auto position = [&](long long r) {
        return plain ? len + r : P.positions ? (long long)P.positions[w.r0 + r] : len + r - candidate_start(P.W, w, (int)r);
      };
      // The next of the warp's rows on its way.
      long long coming = row_first;
      int coming_slot = 0;
      auto fetch = [&]() {
        const uint32_t to = ring_at + coming_slot;
        if (coming < w.rows) {
#pragma unroll
          for (int u = 0; u < kU; ++u) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (!(have >> (2 * u + h) & 1)) continue;
              cp16(to + (2 * u + h) * Rg::kPart, src + u * group_b + (h ? d1 : d0) * es);
              if (DT == 0) cp16(to + (2 * u + h) * Rg::kPart + 16, src + u * group_b + (h ? d1 : d0) * es + 16);
            }
          }
          if (turn) {
            const long long pos = position(coming);
            if (pos >= 0 && pos < P.n_pos)
              for (int c = lane; c < P.half / 2; c += 32)
                cp16(ring_at - lane * (8 * es) + coming_slot + 2 * kU * Rg::kPart + c * 16, P.cos_sin + pos * P.cs_stride + c * 4);
          }
          src += src_step;
          coming += row_step;
          coming_slot = coming_slot + Rg::kSlot == Rg::kBytes ? 0 : coming_slot + Rg::kSlot;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int n = 0; n < Rg::kSlots - 1; ++n) fetch();
      char* place_to = nullptr;  // where row n / 32 * 32 + lane of the warp's goes, null where it goes nowhere
      float* place_scale = nullptr;
      long long r = row_first;
      int n = 0, at_slot = 0;
      for (; r < w.rows; r += row_step, ++n, out += P.out_b * row_step) {
        const char* slot = ring + at_slot;
        at_slot = at_slot + Rg::kSlot == Rg::kBytes ? 0 : at_slot + Rg::kSlot;
        if (!is_q && n % 32 == 0) {
          const long long mine = r + (long long)lane * row_step, at = len + mine;
          place_to = nullptr;
          if (mine < w.rows) {
            const int slot = at <= 0x7fffffffll ? page_slot(C, (int)at) : P.S.width;
            const int page = slot < P.S.width ? table[slot] : -1;
            // A page that others hold too is not written: reserve refused this window.
            if (page >= 0 && page < C.n_pages && C.ref[page] == 1) {
              const long long place = at - (long long)slot * C.page_size;
              place_to = (is_v ? C.v : C.k) + (P.layer + l) * C.layer_b + page * C.page_b + place * C.token_b;
              if (Q8) place_scale = (is_v ? C.vs : C.ks) + (P.layer + l) * C.s_layer + page * C.s_page + place * C.s_token;
            } else {
              set_status(P.status, SV_DATA_BAD_PAGE);
            }
          }
        }
        char* to = nullptr;
        float* scale_to = nullptr;
        if (!is_q) {
          to = reinterpret_cast<char*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(place_to), n % 32));
          if (to) to += to_lane;
          if (Q8) scale_to = reinterpret_cast<float*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(place_scale), n % 32)) + scale_lane;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(Rg::kSlots - 2) : "memory");
        __syncwarp();  // row n has landed, and every lane is through with the slot of the one before
        fetch();
        if constexpr (ROPE) {
          if (P.half) {  // the values' rows too are left out
            const long long pos = position(r);
            if (pos < 0 || pos >= P.n_pos) {
              if (lane == 0) set_status(P.status, SV_DATA_BAD_POSITION);
              continue;
            }
          }
        }
        f2_t A[8], B[8];
        if (ROPE && !is_v) {
          float a[16], y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) a[i] = 1.f;
          if (g) {
            float lo[8], hi[8];
            unpack<DT>(g0, lo);
            unpack<DT>(g1, hi);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              a[i] = lo[i];
              a[8 + i] = hi[i];
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = kPairs ? a[i ^ 1] : a[i ^ 8];
          float c[2][8], s[2][8];
          const float* cs = reinterpret_cast<const float*>(slot + 2 * kU * Rg::kPart);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              c[h][i] = 1.f;
              s[h][i] = 0.f;
            }
            if (!(h ? turned1 : turned0) || (h && !kPairs)) continue;  // across, both parts have the first one's angles
#pragma unroll
            for (int i = 0; i < (kPairs ? 4 : 8); i += 4) {
              const float4 u = *reinterpret_cast<const float4*>(cs + (kPairs ? (h ? d1 : d0) / 2 : d0) + i);
              const float4 v = *reinterpret_cast<const float4*>(cs + P.half + (kPairs ? (h ? d1 : d0) / 2 : d0) + i);
              c[h][i] = u.x, c[h][i + 1] = u.y, c[h][i + 2] = u.z, c[h][i + 3] = u.w;
              s[h][i] = v.x, s[h][i + 1] = v.y, s[h][i + 2] = v.z, s[h][i + 3] = v.w;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int h = i / 8, at = kPairs ? i % 8 / 2 : i % 8;
            const float cv = kPairs ? c[h][at] : c[0][at], sv = kPairs ? s[h][at] : s[0][at];
            const bool on = kPairs ? (h ? turned1 : turned0) : turned0;
            a[i] *= cv;
            y[i] = !on ? 0.f : (kPairs ? i % 2 == 0 : i < 8) ? -y[i] * sv : y[i] * sv;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            A[i] = f2_pack(a[2 * i], a[2 * i + 1]);
            B[i] = f2_pack(y[2 * i], y[2 * i + 1]);
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (h0 - sub + u * kH >= heads) break;  // the same for the warp
          Raw<DT> raw[2]{};
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (have >> (2 * u + h) & 1) raw[h] = load<DT>(slot + (2 * u + h) * Rg::kPart + lane * (8 * es));
          float f[2][8];
          if (Q8 || (ROPE && !is_v)) {
            unpack<DT>(raw[0], f[0]);
            unpack<DT>(raw[1], f[1]);
          }
          if (ROPE && !is_v) {
            f2_t x[8], out2[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = f2_pack(f[i / 4][i % 4 * 2], f[i / 4][i % 4 * 2 + 1]);
            float inv = 1.f;
            if (g) {
              f2_t sq = f2_mul(x[0], x[0]), sq2 = f2_mul(x[4], x[4]);
#pragma unroll
              for (int i = 1; i < 4; ++i) {
                sq = f2_fma(x[i], x[i], sq);
                sq2 = f2_fma(x[4 + i], x[4 + i], sq2);
              }
              float s0, s1;
              f2_unpack(f2_add(sq, sq2), s0, s1);
              s0 += s1;
#pragma unroll
              for (int o = 1; o < L; o <<= 1) s0 += __shfl_xor_sync(kFull, s0, o);
              inv = rsqrtf(fmaf(s0, P.inv_D, P.eps));
            }
            if (turn) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const f2_t y = kPairs ? f2_pack(f[i / 4][i % 4 * 2 + 1], f[i / 4][i % 4 * 2]) : x[i ^ 4];
                f2_t of_y = f2_mul(y, B[i]);
                if (kPartly) of_y = (i < 4 ? turned0 : turned1) ? of_y : 0ull;
                out2[i] = f2_fma(x[i], A[i], of_y);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) out2[i] = f2_mul(x[i], A[i]);
            }
            const f2_t inv2 = f2_splat(inv);
#pragma unroll
            for (int i = 0; i < 8; ++i) f2_unpack(g ? f2_mul(out2[i], inv2) : out2[i], f[i / 4][i % 4 * 2], f[i / 4][i % 4 * 2 + 1]);
          }
          if (is_q) {
            if (have >> (2 * u) & 1) store<DT>(out + u * group_b + d0 * es, pack<DT>(f[0]));
            if (have >> (2 * u + 1) & 1) store<DT>(out + u * group_b + d1 * es, pack<DT>(f[1]));
            continue;
          }
          char* dst = to + u * to_group;
          if constexpr (Q8) {
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i / 8][i % 8]));
#pragma unroll
            for (int o = 1; o < L; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
            const float most = fmaxf(amax, 0x1p-100f), up = __fdiv_rn(448.f, most);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int i = 0; i < 8; ++i) f[h][i] = __fmul_rn(f[h][i], up);
              if ((have >> (2 * u + h) & 1) && to)
                *reinterpret_cast<uint2*>(dst + (h ? d1 : d0)) =
                    make_uint2(pack_e4m3(f[h][0], f[h][1], f[h][2], f[h][3]), pack_e4m3(f[h][4], f[h][5], f[h][6], f[h][7]));
            }
            if ((have >> (2 * u) & 1) && to && j == 0) scale_to[u * scale_group] = __fdiv_rn(most, 448.f);
          } else if (to) {
            if (have >> (2 * u) & 1) store<DT>(dst + d0 * es, is_v ? raw[0] : pack<DT>(f[0]));
            if (have >> (2 * u + 1) & 1) store<DT>(dst + d1 * es, is_v ? raw[1] : pack<DT>(f[1]));
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();  // before another window's rows come to the slots
    }
  }
}

// Some CTAs a sequence, up to eight an SM: a warp a row's chunk of the mean window, or, where that is more CTAs than run at once,
// four rows' (256 windows of 8 rows of 48 heads, turned: 20 us, a row each 24; 200 windows of 6 rows of 8 heads into 8 bits, which run
// at once: a row each 4.0 us, four 4.8; with long windows eight CTAs an SM even out their lengths: 262 us, with four 322).
template <int DT, bool Q8, bool ROPE, int L>
sv_status launch_rows(const Params& P, cudaStream_t st) {
  const int gy = P.S.n > 32768 ? 32768 : P.S.n, gz = P.n_layers < 64 ? P.n_layers : 64;
  const long long per = kU * (32 / L), chunks = ((ROPE ? P.n_q : 0) + per - 1) / per + 2 * ((P.C.n_heads + per - 1) / per);
  const long long items = ((long long)P.W.R + gy - 1) / gy * chunks;
  const long long at_once = 152 * kCtas<ROPE>, each = (items + kT / 32 - 1) / (kT / 32), four = (items + kT / 8 - 1) / (kT / 8);
  const long long gx = each * gy * gz > at_once ? four : each, most = (152 * 8 + (long long)gy * gz - 1) / ((long long)gy * gz);
  const long long least = (chunks + kT / 32 - 1) / (kT / 32);  // a warp for every chunk
  const long long x = gx < most ? gx : most;
  const dim3 grid((unsigned)(x > least ? x : least), gy, gz);
  constexpr size_t bytes = (size_t)(kT / 32) * Ring<DT, ROPE, L>::kBytes;
  auto launch = [&](auto kernel, std::atomic<unsigned long long>& allowed) {
    cudaError_t e = allow_smem(kernel, bytes, allowed);
    if (e == cudaSuccess) e = launch_overlapped(kernel, grid, kT, bytes, 1, st, P);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  };
  static std::atomic<unsigned long long> allowed[4]{};
  if constexpr (ROPE) {
    if (P.half && 2 * P.half < P.D)
      return P.pairs ? launch(append_rows_kernel<DT, Q8, true, L, true, true>, allowed[3])
                     : launch(append_rows_kernel<DT, Q8, true, L, false, true>, allowed[2]);
    if (P.pairs) return launch(append_rows_kernel<DT, Q8, true, L, true, false>, allowed[1]);
  }
  return launch(append_rows_kernel<DT, Q8, ROPE, L, false, false>, allowed[0]);
}
template <int DT, bool Q8, bool ROPE>
sv_status launch_lanes(const Params& P, cudaStream_t st) {
  return P.D <= 64    ? launch_rows<DT, Q8, ROPE, 4>(P, st)
         : P.D <= 128 ? launch_rows<DT, Q8, ROPE, 8>(P, st)
                      : launch_rows<DT, Q8, ROPE, 16>(P, st);
}

}  // namespace app

sv_status append_e4m3(const CacheView& C, const SeqView& S, const WindowView& W, int layer, int n_layers, const char* k_new,
                      const char* v_new, long long new_layer_b, long long new_row_b, uint32_t* status, cudaStream_t st) {
  app::Params P{};
  P.C = C, P.S = S, P.W = W;
  P.layer = layer, P.n_layers = n_layers, P.D = C.head_bytes;
  P.k = k_new, P.v = v_new, P.new_b = new_row_b, P.new_layer_b = new_layer_b;
  P.status = status;
  return app::launch_lanes<1, true, false>(P, st);
}

}  // namespace sv

extern "C" sv_status sv_rope_append(const sv_kv_cache* cache, int32_t layer, const sv_rope* rope, const void* q, int64_t q_stride,
                                    int32_t n_q_heads, void* q_out, int64_t q_out_stride, const void* k_new, const void* v_new,
                                    int64_t new_row_stride, int32_t R, const sv_sequences* seqs, int32_t n_cand,
                                    const int32_t* cu_draft, const int32_t* cu_cand, uint32_t* status, void* cuda_stream) {
  using namespace sv;
  app::Params P{};
  if (!cache_view(cache, &P.C) || !seq_view(seqs, &P.S) || !window_view(P.S.n, n_cand, cu_draft, cu_cand, R, &P.W))
    return SV_ERR_INVALID_ARG;
  if (!rope || layer < 0 || layer >= P.C.n_layers || n_q_heads < 1 || n_q_heads > (1 << 16) || (uintptr_t)status % 4 ||
      !scales_apart(P.C))
    return SV_ERR_INVALID_ARG;
  const int es = row_elem_size(cache->dtype), D = cache->head_dim;
  if (D % 8 || D > 256) return SV_ERR_INVALID_ARG;
  if (rope->rot_dim < 0 || rope->rot_dim % 16 || rope->rot_dim > D || (rope->pairs != 0 && rope->pairs != 1)) return SV_ERR_INVALID_ARG;
  if (rope->rot_dim && (!rope->cos_sin || (uintptr_t)rope->cos_sin % 16 || rope->n_pos < 0 || rope->cos_sin_stride % 4 ||
                        rope->cos_sin_stride < rope->rot_dim || rope->cos_sin_stride > INT64_MAX / 8))
    return SV_ERR_INVALID_ARG;
  if ((uintptr_t)rope->q_norm % 16 || (uintptr_t)rope->k_norm % 16 || (uintptr_t)rope->positions % 4) return SV_ERR_INVALID_ARG;
  if ((rope->q_norm || rope->k_norm) && !(rope->eps > 0.f && rope->eps < 0x1p127f)) return SV_ERR_INVALID_ARG;
  const int64_t strides[2] = {q_stride, q_out_stride};
  for (int64_t s : strides)
    if (s < (int64_t)n_q_heads * D || s > INT64_MAX / 4 || s * es % 16) return SV_ERR_INVALID_ARG;
  if (q == q_out && R > 1 && q_stride != q_out_stride) return SV_ERR_INVALID_ARG;
  if (new_row_stride < 0 || new_row_stride > INT64_MAX / 4 || new_row_stride * es % 16) return SV_ERR_INVALID_ARG;
  if (P.S.n == 0 || R == 0) return SV_OK;
  const void* rows[4] = {q, q_out, k_new, v_new};
  for (const void* p : rows)
    if (!p || (uintptr_t)p % 16) return SV_ERR_INVALID_ARG;
  P.layer = layer, P.n_layers = 1, P.D = D, P.n_q = n_q_heads;
  P.q = static_cast<const char*>(q), P.out = static_cast<char*>(q_out);
  P.k = static_cast<const char*>(k_new), P.v = static_cast<const char*>(v_new);
  P.q_b = q_stride * es, P.out_b = q_out_stride * es, P.new_b = new_row_stride * es;
  P.cos_sin = rope->cos_sin, P.cs_stride = rope->cos_sin_stride, P.n_pos = rope->n_pos, P.half = rope->rot_dim / 2, P.pairs = rope->pairs;
  P.eps = rope->eps;
  P.inv_D = 1.f / (float)D;
  P.g_q = static_cast<const char*>(rope->q_norm), P.g_k = static_cast<const char*>(rope->k_norm);
  P.positions = rope->positions;
  P.status = status;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return cache->dtype == SV_FP32   ? app::launch_lanes<0, false, true>(P, st)
         : cache->dtype == SV_BF16 ? app::launch_lanes<1, false, true>(P, st)
                                   : app::launch_lanes<1, true, true>(P, st);
}
