// rlk_logits.cuh -- what the operators over logits (token log probabilities, distillation
// from a teacher's top logits) share: element types, the row statistics and their fixed
// order, the gradient's arithmetic and the host-side argument checks.
//
// Row statistics of the scaled logits x = s z (s = 1 / temperature) over v < V_true:
//   M = max z,  S = sum e^{s (z - M)},  U = sum e^{s (z - M)} (z - M)
//   lse = s M + log S,   entropy = -sum p log p = log S - s U / S    (both terms >= 0)
// The row is cut into leaves of 1024 columns. A warp takes a leaf: lane i holds the columns
// 256 j + 8 i .. + 7 (j = 0..3), subtracts the leaf's own maximum (exact, order-free), and
// sums even and odd columns separately in ascending order; the lanes combine by an
// xor-butterfly. Leaves are combined by one warp: lane i folds leaves i, i + 32, ... in
// ascending order, then the same butterfly. The order depends on column indices alone, so
// lse and entropy of a row never depend on T, on the row's address or alignment, on the
// launch shape or on which CTA took which leaf.
#pragma once

#include <cuda_fp16.h>

#include "rlk.h"
#include "rlk_internal.h"
#include "rlk_ptx.cuh"

namespace rlk {

constexpr int ROW_LEAF = 1024;       // columns per leaf (one warp)
constexpr int LEAF_GROUP = 256;      // columns a warp covers with 8 per lane
constexpr int LEAF_GROUPS = ROW_LEAF / LEAF_GROUP;
constexpr uint32_t kFullWarp = 0xffffffffu;

// ---------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------
struct Bf16 {
  using bits = uint16_t;
  static constexpr bits kNegInf = 0xFF80u;
  static __device__ __forceinline__ float to_f32(bits b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
  static __device__ __forceinline__ bits from_f32(float v) { return static_cast<bits>(pack_bf16x2(v, 0.f) & 0xFFFFu); }
};
struct F16 {
  using bits = uint16_t;
  static constexpr bits kNegInf = 0xFC00u;
  static __device__ __forceinline__ float to_f32(bits b) { return __half2float(__ushort_as_half(b)); }
  static __device__ __forceinline__ bits from_f32(float v) { return __half_as_ushort(__float2half_rn(v)); }
};
struct F32 {
  using bits = uint32_t;
  static constexpr bits kNegInf = 0xFF800000u;
  static __device__ __forceinline__ float to_f32(bits b) { return __uint_as_float(b); }
  static __device__ __forceinline__ bits from_f32(float v) { return __float_as_uint(v); }
};

// One launch's logits: T rows of `ld` elements, the first n (= V_true) of each valid.
struct LogitRows {
  const void* base;
  int64_t ld;
  int32_t T, n;
  float s;       // 1 / temperature
  float c;       // rn(s log2 e): e^{s d} = ex2(d c)
  int32_t* err_flag;
};

// ---------------------------------------------------------------------------
// packs: 8 consecutive elements of a row, loaded as aligned 16-byte vectors
// ---------------------------------------------------------------------------
// Rows may start at any multiple of the element size (an odd row length in 16-bit types).
// A pack that is not 16-byte aligned is cut from two (three for fp32) neighbouring aligned
// vectors with funnel shifts: the second vector is the neighbouring lane's first and comes
// from L1, and no lane ever owns other columns than in the aligned case, so alignment cannot
// change the order of a sum. Only vectors that lie wholly inside the row are loaded; packs at
// its ends fall back to single elements.
template <class E>
struct Pack {
  static constexpr int EB = sizeof(typename E::bits);
  static constexpr int WORDS = 2 * EB;  // 4 (16-bit types) or 8
  uint32_t w[WORDS];
};

// A row (or the rest of one): its first n elements are valid.
template <class E>
struct Row {
  const typename E::bits* p;
  int32_t n;
  uint32_t shift;  // bytes that p lies past a 16-byte boundary; the same for every thread
  __device__ __forceinline__ Row(const typename E::bits* p_, int n_)
      : p(p_), n(n_), shift(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p_) & 15u)) {}
  __device__ __forceinline__ float at(int64_t c) const { return E::to_f32(p[c]); }
};

// True when pack columns [c0, c1) (multiples of 8) load as vectors inside the row.
template <class E>
__device__ __forceinline__ bool packs_inside(const Row<E>& r, int c0, int c1) {
  if (r.shift == 0) return c1 <= r.n;
  return c0 > 0 && c1 + static_cast<int>((16u - r.shift) / Pack<E>::EB) <= r.n;
}

__device__ __forceinline__ void ld_vec(uint32_t* w, const void* p) {
  const uint4 v = *static_cast<const uint4*>(p);
  w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
}

// Pack at column c0 (a multiple of 8); packs_inside must hold for it.
template <class E>
__device__ __forceinline__ Pack<E> load_pack(const Row<E>& r, int c0) {
  constexpr int W = Pack<E>::WORDS;
  Pack<E> k;
  const char* q = reinterpret_cast<const char*>(r.p) - r.shift + static_cast<int64_t>(c0) * Pack<E>::EB;
  if (r.shift == 0) {
#pragma unroll
    for (int i = 0; i < W; i += 4) ld_vec(k.w + i, q + 4 * i);
    return k;
  }
  uint32_t y[W + 4];
#pragma unroll
  for (int i = 0; i < W + 4; i += 4) ld_vec(y + i, q + 4 * i);
  // words shift / 4 .. of y, then the bytes within a word
  const bool two = r.shift & 8u, one = r.shift & 4u;
  uint32_t x[W + 2];
#pragma unroll
  for (int i = 0; i < W + 2; ++i) x[i] = two ? y[i + 2] : y[i];
  if constexpr (Pack<E>::EB == 4) {
#pragma unroll
    for (int i = 0; i < W; ++i) k.w[i] = one ? x[i + 1] : x[i];
  } else {
    uint32_t t[W + 1];
#pragma unroll
    for (int i = 0; i < W + 1; ++i) t[i] = one ? x[i + 1] : x[i];
    const uint32_t bits = (r.shift & 3u) * 8u;
#pragma unroll
    for (int i = 0; i < W; ++i) k.w[i] = __funnelshift_r(t[i], t[i + 1], bits);
  }
  return k;
}

// Pack at column c0 near the row's ends, element by element; -inf beyond the row.
template <class E>
__device__ __forceinline__ Pack<E> load_pack_edge(const Row<E>& r, int c0) {
  Pack<E> k;
#pragma unroll
  for (int i = 0; i < Pack<E>::WORDS; ++i) {
    if constexpr (Pack<E>::EB == 4) {
      k.w[i] = c0 + i < r.n ? r.p[c0 + i] : E::kNegInf;
    } else {
      const uint32_t lo = c0 + 2 * i < r.n ? r.p[c0 + 2 * i] : E::kNegInf;
      const uint32_t hi = c0 + 2 * i + 1 < r.n ? r.p[c0 + 2 * i + 1] : E::kNegInf;
      k.w[i] = lo | hi << 16;
    }
  }
  return k;
}

template <class E>
__device__ __forceinline__ void unpack(const Pack<E>& k, float* v) {
#pragma unroll
  for (int i = 0; i < Pack<E>::WORDS; ++i) {
    if constexpr (Pack<E>::EB == 4) {
      v[i] = E::to_f32(k.w[i]);
    } else {
      v[2 * i] = E::to_f32(static_cast<uint16_t>(k.w[i]));
      v[2 * i + 1] = E::to_f32(static_cast<uint16_t>(k.w[i] >> 16));
    }
  }
}

// ---------------------------------------------------------------------------
// row statistics
// ---------------------------------------------------------------------------
struct Stats {
  float m, s, u;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullWarp, v, d));
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFullWarp, v, d));
  return v;
}

// Packs of a lane: k[j] holds columns 256 j + 8 lane .. + 7 of the leaf; -inf beyond the row.
template <class E>
__device__ __forceinline__ void load_leaf(const Row<E>& r, int leaf, int lane, Pack<E> (&k)[LEAF_GROUPS]) {
  const int c0 = leaf * ROW_LEAF + lane * 8;
  if (packs_inside(r, leaf * ROW_LEAF, (leaf + 1) * ROW_LEAF)) {  // the same for the whole warp
#pragma unroll
    for (int j = 0; j < LEAF_GROUPS; ++j) k[j] = load_pack(r, c0 + j * LEAF_GROUP);
  } else {
#pragma unroll
    for (int j = 0; j < LEAF_GROUPS; ++j) {
      const int c = c0 + j * LEAF_GROUP;
      k[j] = packs_inside(r, c, c + 8) ? load_pack(r, c) : load_pack_edge(r, c);
    }
  }
}

// Statistics of one leaf, the same in every lane. NaN or +inf among the columns makes s NaN;
// a leaf that is -inf throughout gives {-inf, 0, 0}.
__device__ __forceinline__ Stats leaf_stats(const float (&v)[32], float c) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < 32; ++i) m = fmaxf(m, v[i]);
  bool nan = false;  // fmaxf drops NaN: only a leaf of nothing but -inf and NaN needs the test
#pragma unroll
  for (int i = 0; i < 32; ++i) nan |= isnan(v[i]);
  m = warp_max(m);
  nan = __any_sync(kFullWarp, nan);
  if (m == neg_inf()) return Stats{m, nan ? __int_as_float(0x7fc00000) : 0.f, 0.f};
  float s2[2] = {0.f, 0.f}, u2[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    // -inf columns have weight 0: a finite d keeps 0 * d out of NaN (fmaxf(NaN, x) = x, but
    // the NaN reaches s through the weight)
    const float d = __fsub_rn(v[i], m);
    const float w = ex2_approx(__fmul_rn(d, c));
    s2[i & 1] = __fadd_rn(s2[i & 1], w);
    u2[i & 1] = __fmaf_rn(w, fmaxf(d, -3.4028235e38f), u2[i & 1]);
  }
  return Stats{m, warp_sum(__fadd_rn(s2[0], s2[1])), warp_sum(__fadd_rn(u2[0], u2[1]))};
}

// One warp folds the leaves' statistics (shared memory); every lane gets the row's.
__device__ __forceinline__ Stats fold_leaves(const Stats* leaf, int n_leaves, float c, int lane) {
  float M = neg_inf();
  for (int l = lane; l < n_leaves; l += 32) M = fmaxf(M, leaf[l].m);
  M = warp_max(M);
  float S = 0.f, U = 0.f;
  for (int l = lane; l < n_leaves; l += 32) {
    const Stats x = leaf[l];
    if (x.s == 0.f) continue;  // nothing but -inf
    const float d = __fsub_rn(x.m, M);
    const float f = ex2_approx(__fmul_rn(d, c));
    S = __fmaf_rn(x.s, f, S);
    // u relative to M: sum w (z - M) = u + s (m - M); a leaf too far down to count adds nothing
    if (f != 0.f) U = __fmaf_rn(f, __fmaf_rn(x.s, d, x.u), U);
  }
  return Stats{M, warp_sum(S), warp_sum(U)};
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

// lse = s M + log S; -inf for an empty row, NaN for one that holds NaN or +inf.
__device__ __forceinline__ float row_lse(const Stats& r, float s) {
  if (isnan(r.s)) return quiet_nan();
  if (r.s == 0.f) return neg_inf();
  return __fmaf_rn(r.m, s, logf(r.s));
}

__device__ __forceinline__ float row_entropy(const Stats& r, float s) {
  if (isnan(r.s)) return quiet_nan();
  if (r.s == 0.f) return 0.f;
  return __fsub_rn(logf(r.s), __fmul_rn(s, __fdiv_rn(r.u, r.s)));
}

// s z - lse with one rounding: log p of the token. -inf where the row is empty.
__device__ __forceinline__ float token_logp(float z, float s, float lse) {
  return lse == neg_inf() ? neg_inf() : __fmaf_rn(z, s, -lse);
}

// e^{s (z - b)} as the gradient forms it: d = s z - lse (one rounding, small where p counts),
// p = ex2(d log2 e).
__device__ __forceinline__ float prob_of(float d) { return ex2_approx(__fmul_rn(d, kLog2e)); }

// ---------------------------------------------------------------------------
// the teacher's distribution of one row, by one warp
// ---------------------------------------------------------------------------
// q = softmax(s t_k) over the entries with an id (id -1: none); lane i holds entries i + 32 r.
struct Teacher {
  int64_t id[RLK_MAX_TOP_K / 32];   // -1: no entry
  float q[RLK_MAX_TOP_K / 32];
  float logq[RLK_MAX_TOP_K / 32];   // 0 where q is 0
  bool any;                         // some entry has q > 0
  bool bad_id, nonfinite;           // an id outside [-1, n) / a teacher value that is NaN or +inf
};

__device__ __forceinline__ void load_teacher(Teacher& r, const int64_t* ids, const float* t, int K, int n,
                                             float s, float c, int lane) {
  constexpr int R = RLK_MAX_TOP_K / 32;
  float v[R];
  float m = neg_inf();
  bool bad = false, inf = false;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int k = lane + 32 * i;
    r.id[i] = k < K ? ids[k] : -1;
    v[i] = k < K ? t[k] : neg_inf();
    if (r.id[i] < -1 || r.id[i] >= n) {
      bad = true;
      r.id[i] = -1;
    }
    if (r.id[i] < 0) v[i] = neg_inf();
    inf |= !(v[i] < __int_as_float(0x7f800000));  // NaN or +inf
    m = fmaxf(m, v[i]);
  }
  r.bad_id = __any_sync(kFullWarp, bad);
  r.nonfinite = __any_sync(kFullWarp, inf);
  m = warp_max(m);
  r.any = m > neg_inf();
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float d = v[i] > neg_inf() ? __fsub_rn(v[i], m) : neg_inf();
    r.q[i] = ex2_approx(__fmul_rn(d, c));
    r.logq[i] = __fmul_rn(d, s);
    sum = __fadd_rn(sum, r.q[i]);
  }
  sum = warp_sum(sum);
  const float ls = r.any ? logf(sum) : 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const bool some = r.q[i] > 0.f;
    r.q[i] = some ? __fdiv_rn(r.q[i], sum) : 0.f;
    r.logq[i] = some ? __fsub_rn(r.logq[i], ls) : 0.f;
  }
}

// ---------------------------------------------------------------------------
// host-side checks shared by the entry points
// ---------------------------------------------------------------------------
inline int dtype_bytes(int32_t dtype) {
  return dtype == RLK_DTYPE_F32 ? 4 : (dtype == RLK_DTYPE_BF16 || dtype == RLK_DTYPE_F16) ? 2 : 0;
}

// Fills `r`; RLK_OK or the refusal.
inline rlk_status check_logits(const void* logits, int32_t dtype, int64_t T, int64_t ld, int64_t V_true,
                               double temperature, int32_t* err_flag, LogitRows* r) {
  const int eb = dtype_bytes(dtype);
  if (eb == 0 || T < 0 || V_true <= 0 || ld < V_true) return RLK_ERR_INVALID_ARG;
  if (T > 0 && (!logits || reinterpret_cast<uintptr_t>(logits) % eb != 0)) return RLK_ERR_INVALID_ARG;
  if (!(temperature >= RLK_MIN_TEMPERATURE && temperature <= RLK_MAX_TEMPERATURE)) return RLK_ERR_INVALID_ARG;
  if (V_true > RLK_MAX_LOGITS_VOCAB || T > RLK_MAX_LOGITS_ROWS) return RLK_ERR_UNSUPPORTED;
  r->base = logits;
  r->ld = ld;
  r->T = static_cast<int32_t>(T);
  r->n = static_cast<int32_t>(V_true);
  r->s = static_cast<float>(1.0 / temperature);
  r->c = static_cast<float>(1.4426950408889634 / temperature);
  r->err_flag = err_flag;
  return RLK_OK;
}

}  // namespace rlk
