// logprobs.cu -- log probabilities of given tokens, with rank, entropy and
// top alternatives.
//
// Per row, with t_x = (z_x - M) / T, M = max z:
//   S = sum e^t, ln p(x) = t_x - ln S, H = ln S - (1 / S) sum e^t t,
//   rank = 1 + #{z_x > z_tok} + #{z_x = z_tok, x < tok},
//   the top n in the order (z descending, index ascending).
// One pass: every thread keeps the sums relative to its own running maximum
// m; moving the reference from m to m' with d = (m - m') / T multiplies S by
// e^d and turns S1 = sum e^t t into e^d (S1 + d S). The threads' sums are
// joined in double-float.
//
// The alternatives come from the same pass. A floor that n elements of the
// row are known to reach (each warp publishes the ceil(n / warps)-th largest
// of its lanes' maxima, the floor is the least of those) lets almost every
// batch pass with one comparison; elements at or above it go to a buffer, and
// the row's end sorts what reached the last floor. Rows that overflow the
// buffer (long ties at the top) take n passes for the n alternatives. Of the
// 158 us that 2048 rows of V = 151936 bf16 take with rank and 20 alternatives,
// hits after the first batch are 28; a tighter floor (the n-th largest of all
// threads' maxima, searched by one warp after batches 0, 1, 3, 7, ...) halved
// the hits and cost more than they did, and raising it less often did too.
//
// Bound by the bytes for long rows: 2048 rows of V = 151936 bf16 without
// alternatives take 113 us (81% of the copy rate), with 20 of them 141; the
// benchmark batch's 1150 committed rows with rank and 20 alternatives 93 us
// (52 us of bytes). A row's end is a chain of short steps (about 10 us beside
// three other rows on the SM): it weighs on short rows, 2816 rows of V = 32000
// bf16 taking 49 us without and 75 with alternatives (27 us of bytes). Four
// CTAs an SM with four loads a batch beat 3 and 5 CTAs and 2 to 8 loads.
#include "../../include/spec_verify.h"
#include "sv_device.cuh"
#include "sv_launch.cuh"

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
  float c_hi, c_lo;          // log2(e) / T in two parts
  float inv_T_hi, inv_T_lo;  // 1 / T
  // How far below a maximum terms are zero. Up to `large` a step of the type is less than that, and what lies between two maxima and
  // the first one's cut-off stays finite in the exponent: the cut-off is then found once.
  float far, large;
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

// Whether row r is asked for, b being the request that the offsets put it in.
__device__ __forceinline__ bool row_wanted(const Params& P, int r, int b) {
  const long long i = (long long)r - P.cu[b] - b;
  const long long K = (long long)P.cu[b + 1] - P.cu[b];
  const int n = P.out_len[b];
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

#ifndef SV_LP_LOADS
#define SV_LP_LOADS 4
#endif
#ifndef SV_LP_CTAS
#define SV_LP_CTAS 4
#endif
constexpr int kU = SV_LP_LOADS;  // 16-byte loads of a batch, per thread; the next batch's are in flight meanwhile
constexpr int kVecs = 256 * SV_LP_LOADS;      // vectors that a CTA buffers because one of their elements may be an alternative
constexpr int kCap = 1024;       // elements that reached the last floor
constexpr int kMaxCluster = 8;   // CTAs to a row, at most
constexpr float kFar = 200.f;    // 2^-kFar is zero in fp32: exponents are cut off there

// The 16-byte vector at aligned-down place v of a row that begins `off`
// elements behind it; elements outside the row read as -inf.
template <int DT>
__device__ __forceinline__ uint4 load_vec(const char* row, const char* base, int v, int off, int V) {
  constexpr int EPV = Elem<DT>::kEPV;
  const int x0 = v * EPV - off;
  if (x0 >= 0 && x0 + EPV <= V) return ld_stream16(base + (long long)v * 16);
  float f[EPV];
#pragma unroll
  for (int j = 0; j < EPV; ++j) f[j] = x0 + j >= 0 && x0 + j < V ? Elem<DT>::scalar(row, x0 + j) : -INFINITY;
  uint4 r;
  uint32_t* w = &r.x;
  if constexpr (DT == 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (__float_as_uint(f[2 * j]) >> 16) | (__float_as_uint(f[2 * j + 1]) & 0xffff0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(f[j]);
  }
  return r;
}

// Maxima that keep a NaN, so that a row with one is found out.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_nan_bf2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The maxima of a batch's vectors (a bf16 pair of them, or one), and of the whole batch.
template <int DT>
__device__ __forceinline__ uint32_t vec_max(const uint4& v) {
  if constexpr (DT == 1)
    return max_nan_bf2(max_nan_bf2(v.x, v.y), max_nan_bf2(v.z, v.w));
  else
    return __float_as_uint(max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                                   max_nan(__uint_as_float(v.z), __uint_as_float(v.w))));
}
template <int DT>
__device__ __forceinline__ float max_value(uint32_t m) {
  return DT == 1 ? max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u)) : __uint_as_float(m);
}
template <int DT>
__device__ __forceinline__ float batch_max(const uint32_t (&vm)[kU]) {
  uint32_t m = vm[0];
#pragma unroll
  for (int u = 1; u < kU; ++u)
    m = DT == 1 ? max_nan_bf2(m, vm[u]) : __float_as_uint(max_nan(__uint_as_float(m), __uint_as_float(vm[u])));
  return max_value<DT>(m);
}

__device__ __forceinline__ int order_key(float f) {  // whole numbers in the order of the floats
  const int b = __float_as_int(f);
  return b < 0 ? b ^ 0x7fffffff : b;
}
__device__ __forceinline__ float key_value(int k) { return __int_as_float(k < 0 ? k ^ 0x7fffffff : k); }

// The next value of the type below f; -inf stays. Zeros count as one.
template <int DT>
__device__ __forceinline__ float value_below(float f) {
  if (f == -INFINITY) return f;
  const int k = (f == 0.f ? -1 : order_key(f)) - (DT == 1 ? 0x10000 : 1);  // -1: the key of -0
  if (DT == 1) return __uint_as_float(__float_as_uint(key_value(k)) & 0xffff0000u);
  return key_value(k);
}

constexpr uint32_t kAlone = 0xffffffffu;  // no value of the type, nor a NaN that arithmetic gives

// Where logits are cut off below a maximum m whose next lower value is less
// than kFar away in the exponent: kFar below it, rounded down to the type.
template <int DT>
__device__ __forceinline__ uint32_t cut_off(float m, float far) {
  if constexpr (DT == 1) {
    const int k = order_key(m - far) >> 16;
    const uint32_t b = __float_as_uint(key_value((int)((uint32_t)k << 16 | (k < 0 ? 0xffffu : 0u)))) & 0xffff0000u;
    return b | b >> 16;
  } else {
    return __float_as_uint(m - far);
  }
}

// A maximum that no other value of the type comes near (the type's lowest
// one, or a step of the type is more than any exponent reaches): what equals
// it counts one, all else nothing.
template <int DT>
__device__ __forceinline__ void add_equal(const uint4& v, float m, f2_t& S) {
  float f[Elem<DT>::kEPV], n = 0.f;
  Elem<DT>::unpack(v, f);
#pragma unroll
  for (int j = 0; j < Elem<DT>::kEPV; ++j) n += f[j] == m ? 1.f : 0.f;
  S = f2_add(S, f2_pack(n, 0.f));
}

// Adds one vector's terms 2^((z - m) c) and their first moments, in pairs.
// The reference's negative and the two parts of c come as pairs; `lowest`
// cuts off logits so far below m that their term is zero: their exponent
// could leave fp32, and its product with a term of zero not be a number.
template <int DT>
__device__ __forceinline__ void add_terms(const uint4& v, uint32_t lowest, f2_t neg_m, f2_t c_hi, f2_t c_lo, f2_t& S, f2_t& S1) {
  const uint32_t* w = &v.x;
  if constexpr (DT == 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = max_nan_bf2(w[j], lowest);
      const f2_t d = f2_add(f2_pack(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), neg_m);
      const f2_t t = f2_fma(d, c_lo, f2_mul(d, c_hi));
      const f2_t e = f2_ex2(t);
      S = f2_add(S, e);
      S1 = f2_fma(e, t, S1);
    }
  } else {
    const float lo = __uint_as_float(lowest);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const f2_t d = f2_add(f2_pack(max_nan(__uint_as_float(w[j]), lo), max_nan(__uint_as_float(w[j + 1]), lo)), neg_m);
      const f2_t t = f2_fma(d, c_lo, f2_mul(d, c_hi));
      const f2_t e = f2_ex2(t);
      S = f2_add(S, e);
      S1 = f2_fma(e, t, S1);
    }
  }
}

// The q-th largest of the lanes' values (1 <= q <= 32).
__device__ __forceinline__ float warp_nth_largest(float v, int q) {
  const int lane = threadIdx.x & 31;
  int key = order_key(v + 0.f), top = key;
  for (int i = 0; i < q; ++i) {
    top = __reduce_max_sync(kFull, key);
    const unsigned who = __ballot_sync(kFull, key == top);
    if (lane == __ffs(who) - 1) key = INT_MIN;
  }
  return key_value(top);
}

// Sums of 2^((z - m) c) and their first moments about a maximum m.
struct Sums {
  float m;
  DF S, S1;
};

// The sums of the warp's first `lanes` lanes (a power of two; the others
// hold none: m = -inf, 0, 0), moved to their common maximum. The order of
// the additions is fixed.
__device__ __forceinline__ Sums join_lanes(Sums x, int lanes, float c) {
  float m = x.m;
  for (int o = lanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, o));
  if (x.m == -INFINITY) {
    x.S = x.S1 = DF{0.f, 0.f};
  } else {
    const float d = fmaxf((x.m - m) * c, -kFar), f = ex2(d);
    x.S1 = df_mul_f(df_add(x.S1, df_mul_f(x.S, d)), f);
    x.S = df_mul_f(x.S, f);
  }
  for (int o = lanes / 2; o > 0; o >>= 1) {
    x.S = df_add(x.S, DF{__shfl_xor_sync(kFull, x.S.hi, o), __shfl_xor_sync(kFull, x.S.lo, o)});
    x.S1 = df_add(x.S1, DF{__shfl_xor_sync(kFull, x.S1.hi, o), __shfl_xor_sync(kFull, x.S1.lo, o)});
  }
  // To every lane of the warp.
  return Sums{__shfl_sync(kFull, m, 0), DF{__shfl_sync(kFull, x.S.hi, 0), __shfl_sync(kFull, x.S.lo, 0)},
              DF{__shfl_sync(kFull, x.S1.hi, 0), __shfl_sync(kFull, x.S1.lo, 0)}};
}

// The batch's elements that rank above the token: larger ones, and equal
// ones of a lower index. `at` is the thread's first vector.
template <int DT>
__device__ __forceinline__ int count_above_near(const uint4 (&cur)[kU], int at, int v1, int off, int tok, float zt) {
  constexpr int EPV = Elem<DT>::kEPV;
  int n = 0;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int v = at + u * kThreads, x0 = v * EPV - off;
    float f[EPV];
    Elem<DT>::unpack(cur[u], f);
    if (v < v1) {  // what is read behind the slice is -inf, as the token may be
#pragma unroll
      for (int j = 0; j < EPV; ++j) n += f[j] > zt || (f[j] == zt && x0 + j >= 0 && x0 + j < tok);
    }
  }
  return n;
}
// The same for a batch that lies before the token or behind it as a whole:
// how many are above z, which is the token's logit, or the value below it.
template <int DT>
__device__ __forceinline__ int count_above(const uint4 (&cur)[kU], float z) {
  if constexpr (DT == 1) {
    const uint32_t zz = (__float_as_uint(z) >> 16) * 0x10001u;
    uint32_t n = 0;  // two counts to a word, as bf16 numbers (of 4 * kU at most)
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t* w = &cur[u].x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t g;
        asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(g) : "r"(w[j]), "r"(zz));
        asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(n) : "r"(g));
      }
    }
    return (int)(__uint_as_float(n << 16) + __uint_as_float(n & 0xffff0000u));
  } else {
    int n = 0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t* w = &cur[u].x;
#pragma unroll
      for (int j = 0; j < 4; ++j) n += __uint_as_float(w[j]) > z;
    }
    return n;
  }
}

// An alternative as one number: larger logits first, then lower indices.
typedef unsigned long long u64;
__device__ __forceinline__ u64 make_key(float z, int x) {
  return (u64)((uint32_t)order_key(z + 0.f) ^ 0x80000000u) << 32 | (uint32_t)~x;
}
__device__ __forceinline__ float key_logit(u64 k) { return key_value((int)((uint32_t)(k >> 32) ^ 0x80000000u)); }
__device__ __forceinline__ int key_index(u64 k) { return (int)~(uint32_t)k; }
// None: below every finite logit's key, and different for every j.
__device__ __forceinline__ u64 no_key(int j) { return (u64)j; }
__device__ __forceinline__ bool is_key(u64 k) { return (k >> 32) > 0x007fffffull; }

struct Smem {
  uint4 vec[kVecs];                // buffered vectors, and their places
  int vec_at[kVecs];
  alignas(16) u64 cand[kCap];      // alternatives as keys
  alignas(16) u64 best[kMaxCluster * SV_LOGPROBS_MAX_TOP];  // the CTAs' sorted alternatives, in the leader
  float rec[kMaxCluster][6];       // the CTAs' sums (m, S, S1) and rank counts, in the leader
  u64 mine[SV_LOGPROBS_MAX_TOP];
  alignas(16) float floor_w[kWarps];
  Sums sums[kWarps];
  int cnt[kWarps];
  int n, n2;
};

// n elements of the row reach the least of the warps' floors.
__device__ __forceinline__ float shared_floor(const Smem& sm) {
  float f = sm.floor_w[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) f = fminf(f, sm.floor_w[w]);
  return f;
}

// The first n of c keys in descending order, to out[0 .. n); places that
// stay free get keys that stand for none. Each thread counts the keys above
// its own (they are all different); `from` has room for one more.
__device__ __forceinline__ void sort_top(u64* from, int c, int n, u64* out) {
  for (int j = c + threadIdx.x; j < n; j += kThreads) out[j] = no_key(j);
  if (c & 1) {
    if (threadIdx.x == 0) from[c] = 0;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < c; i += kThreads) {
    const u64 x = from[i];
    int k = 0;
#pragma unroll 8
    for (int j = 0; j < c; j += 2) {
      const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(from + j);
      k += (y.x > x) + (y.y > x);
    }
    if (k < n) out[k] = x;
  }
}

// Largest b in [0, B) with cu[b] + b <= t, by every thread of the CTA (as the verify kernels look a row up). Ends for any
// contents of cu.
__device__ __forceinline__ int find_request(const int32_t* cu, int B, int t) {
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + kThreads - 1) / kThreads;
    const int c = lo + (int)threadIdx.x * step;
    const bool pass = c < lo + n && (long long)cu[c] + c <= t;
    const int cnt = max(__syncthreads_count(pass), 1);
    const int end = lo + n;
    lo += (cnt - 1) * step;
    n = min(step, end - lo);
  }
  return lo;
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Writes a word into the leader's shared memory.
__device__ __forceinline__ void to_leader(void* p, float v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_addr(p)));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void to_leader(u64* p, u64 v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_addr(p)));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// A cluster of `cl` CTAs takes a row, each a contiguous slice of its vectors.
template <int DT>
__global__ void __launch_bounds__(kThreads, SV_LP_CTAS) logprobs_kernel(Params P, int cl) {
  constexpr int EPV = Elem<DT>::kEPV;
  __shared__ Smem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cl > 1 ? (int)cluster_rank() : 0;
  const int r = cl > 1 ? blockIdx.x / cl : blockIdx.x;
  if (blockIdx.x == 0) check_offsets(P, tid);
  if (P.cu && !row_wanted(P, r, find_request(P.cu, P.B, r))) return;  // all CTAs of the row alike
  const int V = P.V, n_top = P.n_top;
  const char* row = P.logits + (long long)r * P.ld_bytes;
  const int off = (int)((uintptr_t)row & 15) / Elem<DT>::kBytes;
  const char* base = row - off * Elem<DT>::kBytes;
  const int n_vec = (off + V + EPV - 1) / EPV;
  const int per = (n_vec + cl - 1) / cl;
  const int v0 = min(rank * per, n_vec), v1 = min(v0 + per, n_vec);

  uint4 nxt[kU];
  auto fetch = [&](int at) {
    // Inside the row every vector of the CTA's batch is whole: no tests.
    if (at > 0 && at + kThreads * kU <= v1 && at + kThreads * kU < n_vec) {
      const char* p = base + (long long)(at + tid) * 16;
#pragma unroll
      for (int u = 0; u < kU; ++u) nxt[u] = ld_stream16(p + u * kThreads * 16);
      return;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int v = at + u * kThreads + tid;
      nxt[u] = v < v1 ? load_vec<DT>(row, base, v, off, V) : (DT == 1 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                                                                    : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u));
    }
  };
  fetch(v0);
  const int tok = P.tokens ? P.tokens[r] : -1;
  const bool tok_ok = tok >= 0 && tok < V;
  const float zt = tok_ok ? Elem<DT>::scalar(row, tok) + 0.f : INFINITY;
  const float zt_below = value_below<DT>(zt);
  const int tok_v = (tok + off) / EPV;  // the token's vector
  if (tid < kWarps) sm.floor_w[tid] = -INFINITY;
  if (tid == 0) sm.n = sm.n2 = 0;
  __syncthreads();

  const int q = (n_top + kWarps - 1) / kWarps;
  const f2_t c_hi = f2_splat(P.c_hi), c_lo = f2_splat(P.c_lo);
  float m = -INFINITY;  // this thread's maximum
  uint32_t lowest = 0;  // its cut-off, or kAlone: nothing below m has a term
  f2_t neg_m = 0ull;
  f2_t S = 0ull, S1 = 0ull;
  int above = 0;
  bool first = true;
  float floor = -INFINITY;
  for (int at = v0; at < v1; at += kThreads * kU) {
    uint4 cur[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) cur[u] = nxt[u];
    fetch(at + kThreads * kU);
    uint32_t vm[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) vm[u] = vec_max<DT>(cur[u]);
    const float bm = batch_max<DT>(vm);
    if (!(bm <= m)) {  // a new maximum (or a NaN): move the sums to it
      if (m > -INFINITY) {
        const float d = fmaxf((m - bm) * P.c_hi, -kFar);
        const f2_t f = f2_splat(ex2(d));
        S1 = f2_mul(f, f2_fma(f2_splat(d), S, S1));
        S = f2_mul(f, S);
      }
      if (!(fmaxf(fabsf(m), fabsf(bm)) < P.large)) {
        const bool alone = (bm - value_below<DT>(bm)) * P.c_hi >= kFar && bm < INFINITY;
        lowest = alone ? kAlone : cut_off<DT>(bm, P.far);
      }
      m = bm;
      neg_m = f2_splat(-m);
    }
    if (n_top) {
      if (first) {  // no floor yet: the whole CTA's first maxima make one
        const float w = warp_nth_largest(m, q);
        if (lane == 0) sm.floor_w[warp] = w;
        __syncthreads();
        floor = shared_floor(sm);
      }
      bool hit = bm >= floor && bm > -INFINITY;
      if (__any_sync(kFull, hit)) {
        floor = shared_floor(sm);
        hit = hit && bm >= floor;
        const unsigned hits = __ballot_sync(kFull, hit);
        // A warp that would keep much (values that rise along the row, a mask's end) raises its own floor first.
        if (__popc(hits) > 16) {
          floor = fmaxf(floor, warp_nth_largest(m, n_top));
          hit = hit && bm >= floor;
        }
        if (hit) {  // (one addition a warp, places by a scan over its lanes: 3% slower)
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (max_value<DT>(vm[u]) >= floor) {
              const int k = atomicAdd(&sm.n, 1);
              if (k < kVecs) {
                sm.vec[k] = cur[u];
                sm.vec_at[k] = at + u * kThreads + tid;
              }
            }
        }
        __syncwarp();
        if (!first) {
          const float w = warp_nth_largest(m, q);
          if (lane == 0) sm.floor_w[warp] = w;
        }
      }
      first = false;
    }
    if (__any_sync(kFull, bm >= zt)) {
      // Nothing is below -inf: there, and around the token itself, element by element.
      const bool near = zt == -INFINITY || (tok_v >= at && tok_v < at + kThreads * kU);
      above += near ? count_above_near<DT>(cur, at + tid, v1, off, tok, zt) : count_above<DT>(cur, at < tok_v ? zt_below : zt);
    }
    if (lowest == kAlone) {
#pragma unroll
      for (int u = 0; u < kU; ++u) add_equal<DT>(cur[u], m, S);
    } else if (bm != -INFINITY) {
#pragma unroll
      for (int u = 0; u < kU; ++u) add_terms<DT>(cur[u], lowest, neg_m, c_hi, c_lo, S, S1);
    }
  }

  // Every warp's sums, moved to its maximum.
  {
    float s0, s1, a0, a1;
    f2_unpack(S, s0, s1);
    f2_unpack(S1, a0, a1);
    Sums x{m, df_add_f(DF{s0, 0.f}, s1), df_add_f(DF{a0, 0.f}, a1)};
    x = join_lanes(x, 32, P.c_hi);
    above = __reduce_add_sync(kFull, above);
    if (lane == 0) {
      sm.sums[warp] = x;
      sm.cnt[warp] = above;
    }
  }
  __syncthreads();

  // The CTA's alternatives, in order.
  if (n_top) {
    u64* out = cl > 1 ? sm.mine : sm.best;
    floor = shared_floor(sm);
    if (floor == -INFINITY) {  // short or masked slices: one warp's n elements may still make a floor
      __syncthreads();
      const float w = warp_nth_largest(m, n_top);
      if (lane == 0) sm.floor_w[warp] = w;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWarps; ++k) floor = fmaxf(floor, sm.floor_w[k]);
    }
    const int c = sm.n;
    if (c <= kVecs) {
      // What reached the last floor, in any order: the sort below does not depend on it.
      for (int i = tid; i < c; i += kThreads) {
        float f[EPV];
        Elem<DT>::unpack(sm.vec[i], f);
        const int x0 = sm.vec_at[i] * EPV - off;
#pragma unroll
        for (int j = 0; j < EPV; ++j)
          if (f[j] >= floor && f[j] > -INFINITY) {
            const int k = atomicAdd(&sm.n2, 1);
            if (k < kCap - 1) sm.cand[k] = make_key(f[j], x0 + j);
          }
      }
      __syncthreads();
    }
    if (c <= kVecs && sm.n2 < kCap) {
      sort_top(sm.cand, sm.n2, n_top, out);
    } else {
      __syncthreads();
      // One pass an alternative: the largest key below the last one.
      u64 last = ~0ull;
      for (int j = 0; j < n_top; ++j) {
        u64 best = 0;
        for (int v = v0 + tid; v < v1; v += kThreads) {
          float f[EPV];
          Elem<DT>::unpack(load_vec<DT>(row, base, v, off, V), f);
#pragma unroll
          for (int e = 0; e < EPV; ++e) {
            const u64 k = make_key(f[e], v * EPV - off + e);
            if (f[e] > -INFINITY && k < last && k > best) best = k;
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const u64 k = __shfl_xor_sync(kFull, best, o);
          best = k > best ? k : best;
        }
        if (lane == 0) sm.cand[j % 2 * kWarps + warp] = best;
        __syncthreads();
        last = sm.cand[j % 2 * kWarps];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const u64 k = sm.cand[j % 2 * kWarps + w];
          last = k > last ? k : last;
        }
        if (tid == 0) out[j] = is_key(last) ? last : no_key(j);
      }
    }
    __syncthreads();
  }

  // The CTA's sums by its first warp; in a cluster the leader's joins the CTAs'.
  Sums row_sums{-INFINITY, DF{0.f, 0.f}, DF{0.f, 0.f}};
  int count = 0;
  if (warp == 0) {
    if (lane < kWarps) {
      row_sums = sm.sums[lane];
      count = sm.cnt[lane];
    }
    row_sums = join_lanes(row_sums, kWarps, P.c_hi);
    count = __reduce_add_sync(kFull, count);
  }
  if (cl > 1) {
    cluster_sync();  // the leader has started
    if (tid == 0) {
      const float word[6] = {row_sums.m, row_sums.S.hi, row_sums.S.lo, row_sums.S1.hi, row_sums.S1.lo, __int_as_float(count)};
#pragma unroll
      for (int k = 0; k < 6; ++k) to_leader(&sm.rec[rank][k], word[k]);
    }
    for (int j = tid; j < n_top; j += kThreads) {
      const u64 k = sm.mine[j];
      to_leader(&sm.best[rank * n_top + j], is_key(k) ? k : no_key(rank * n_top + j));
    }
    cluster_sync();
    if (rank != 0) return;
    if (n_top) {
      sort_top(sm.best, cl * n_top, n_top, sm.cand);
      __syncthreads();
    }
    if (warp == 0) {
      row_sums = Sums{-INFINITY, DF{0.f, 0.f}, DF{0.f, 0.f}};
      count = 0;
      if (lane < cl) {
        const float* w = sm.rec[lane];
        row_sums = Sums{w[0], DF{w[1], w[2]}, DF{w[3], w[4]}};
        count = __float_as_int(w[5]);
      }
      row_sums = join_lanes(row_sums, kMaxCluster, P.c_hi);
      count = __reduce_add_sync(kFull, count);
    }
  }
  if (warp != 0) return;
  const u64* top = cl > 1 ? sm.cand : sm.best;
  const float M = row_sums.m;
  const DF rS = row_sums.S;
  const bool empty = M == -INFINITY, bad = !empty && !(rS.hi < INFINITY), ok = !empty && !bad;
  const float lnS = logf(rS.hi) + rS.lo / rS.hi;
  // (z - M) / T - ln S, the quotient with its rounding error.
  auto logprob = [&](float z) {
    const float d = z - M, p = d * P.inv_T_hi, e = fmaf(d, P.inv_T_hi, -p) + d * P.inv_T_lo;
    return isinf(p) ? p : (p - lnS) + e;
  };
  if (lane < n_top) {  // n_top <= 32
    const u64 x = top[lane];
    const bool any = is_key(x);
    const long long o = (long long)r * n_top + lane;
    if (P.top_ids) P.top_ids[o] = any && ok ? key_index(x) : -1;
    if (P.top_lp) P.top_lp[o] = !ok ? NAN : any ? logprob(key_logit(x)) : -INFINITY;
  }
  if (lane == 0) {
    if (bad) flag(P, SV_DATA_BAD_LOGIT);
    if (empty) flag(P, SV_DATA_EMPTY_ROW);
    if (P.tokens && !tok_ok) flag(P, SV_DATA_BAD_TOKEN);
    if (P.logprob) P.logprob[r] = ok && tok_ok ? logprob(zt) : NAN;
    if (P.rank) P.rank[r] = ok && tok_ok ? 1 + count : 0;
    if (P.entropy) P.entropy[r] = ok ? lnS - (row_sums.S1.hi / rS.hi) * 0.69314718056f : NAN;
  }
}

// CTAs to a row: enough for every processor to have work, but slices of a
// few batches at least.
inline int cluster_size(int R, long long row_bytes) {
  int cl = 1;
  while (cl < kMaxCluster && (long long)R * cl < 2 * 152 && row_bytes / (2 * cl) >= 8192) cl *= 2;
  return cl;
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
  if ((dtype != SV_FP32 && dtype != SV_BF16) || V < 1 || V > (1 << 30) || ld < V || R < 0 || B < 0) return SV_ERR_INVALID_ARG;
  const int es = dtype == SV_BF16 ? 2 : 4;
  if (ld > INT64_MAX / 4) return SV_ERR_INVALID_ARG;
  // Up to 2^96 a cut-off kFar below the maximum is finite: 139 T < 2^104, the step of fp32 at its largest values.
  if (!(temperature >= 0x1p-100f && temperature <= 0x1p96f)) return SV_ERR_INVALID_ARG;
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
  const double c = 1.4426950408889634 / (double)temperature, inv_T = 1.0 / (double)temperature;
  P.c_hi = (float)c;
  P.c_lo = std::isinf(P.c_hi) ? 0.f : (float)(c - (double)P.c_hi);
  P.inv_T_hi = (float)inv_T;
  P.inv_T_lo = std::isinf(P.inv_T_hi) ? 0.f : (float)(inv_T - (double)P.inv_T_hi);
  P.far = lp::kFar / P.c_hi;
  P.large = P.far * (dtype == SV_BF16 ? 0x1p7f : 0x1p23f);
  P.logprob = out_logprob;
  P.rank = out_rank;
  P.entropy = out_entropy;
  P.top_ids = out_top_ids;
  P.top_lp = out_top_logprobs;
  P.status = status;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int cl = lp::cluster_size(R, (long long)V * es);
  if ((long long)R * cl > INT32_MAX) return SV_ERR_INVALID_ARG;
  // An ordinary launch: the rows are streamed by read-only loads (3% faster than others here), which a launch that overlaps the
  // kernel before it may not use.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(R * cl));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cl;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cl > 1 ? 1 : 0;
  const cudaError_t e = own_error(dtype == SV_BF16 ? cudaLaunchKernelEx(&cfg, lp::logprobs_kernel<1>, P, cl)
                                                   : cudaLaunchKernelEx(&cfg, lp::logprobs_kernel<0>, P, cl));
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
