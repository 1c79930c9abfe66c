// rlk_logits.cuh -- what the operators over logits (token log probabilities, distillation
// from a teacher's top logits) share: element types, the row statistics and their fixed
// order, the gradient's arithmetic and the host-side argument checks.
//
// Row statistics of the scaled logits s z (s = 1 / temperature) over v < V_true, with
// x = c (z - M), c = s log2 e, so that 2^x = e^{s (z - M)}:
//   M = max z,  S = sum 2^x,  U = sum 2^x x
//   lse = s M + log S,   entropy = -sum p log p = log S - log 2 U / S    (both terms >= 0)
//   log p = s (z - M) - log S: not s z - lse, whose fp32 lse has lost log S where |s M| is large
// The row is cut into leaves of 1024 columns. A warp takes a leaf: lane i holds the columns
// 256 j + 8 i .. + 7 (j = 0..3), takes x about the leaf's own maximum (exact, order-free), and
// sums even and odd columns separately in ascending order; the lanes combine by an
// xor-butterfly. Leaves are combined by one warp: lane i folds leaves i, i + 32, ... in
// ascending order, then the same butterfly. The order depends on column indices alone, so
// lse and entropy of a row never depend on T, on the row's address or alignment, on the
// launch shape or on which CTA took which leaf.
#pragma once

#include <cuda_bf16.h>
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
  static constexpr float kLseRange = 4096.f;  // see lse_is_coarse
  static constexpr int kKeyShift = 16;  // low bits of the fp32 image that carry nothing
  static __device__ __forceinline__ float to_f32(bits b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
  static __device__ __forceinline__ bits from_f32(float v) { return static_cast<bits>(pack_bf16x2(v, 0.f) & 0xFFFFu); }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ float2 to_f32x2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2(reinterpret_cast<__nv_bfloat162&>(a), reinterpret_cast<__nv_bfloat162&>(b));
    return reinterpret_cast<const uint32_t&>(r);
  }
  // acc + (a >= b), per half; counts up to 256 are exact
  static __device__ __forceinline__ uint32_t count_ge2(uint32_t a, uint32_t b, uint32_t acc) {
    const __nv_bfloat162 r = __hadd2(reinterpret_cast<__nv_bfloat162&>(acc),
                                     __hge2(reinterpret_cast<__nv_bfloat162&>(a), reinterpret_cast<__nv_bfloat162&>(b)));
    return reinterpret_cast<const uint32_t&>(r);
  }
};
struct F16 {
  using bits = uint16_t;
  static constexpr bits kNegInf = 0xFC00u;
  static constexpr float kLseRange = 512.f;  // see lse_is_coarse
  static constexpr int kKeyShift = 13;
  static __device__ __forceinline__ float to_f32(bits b) { return __half2float(__ushort_as_half(b)); }
  static __device__ __forceinline__ bits from_f32(float v) { return __half_as_ushort(__float2half_rn(v)); }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return reinterpret_cast<const uint32_t&>(r);
  }
  static __device__ __forceinline__ float2 to_f32x2(uint32_t w) {
    return __half22float2(reinterpret_cast<const __half2&>(w));
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __half2 r = __hmax2(reinterpret_cast<__half2&>(a), reinterpret_cast<__half2&>(b));
    return reinterpret_cast<const uint32_t&>(r);
  }
  static __device__ __forceinline__ uint32_t count_ge2(uint32_t a, uint32_t b, uint32_t acc) {
    const __half2 r = __hadd2(reinterpret_cast<__half2&>(acc),
                              __hge2(reinterpret_cast<__half2&>(a), reinterpret_cast<__half2&>(b)));
    return reinterpret_cast<const uint32_t&>(r);
  }
};
struct F32 {
  using bits = uint32_t;
  static constexpr bits kNegInf = 0xFF800000u;
  static constexpr float kLseRange = 256.f;  // see lse_is_coarse
  static constexpr int kKeyShift = 0;
  static __device__ __forceinline__ float to_f32(bits b) { return __uint_as_float(b); }
  static __device__ __forceinline__ bits from_f32(float v) { return __float_as_uint(v); }
};

// The next value above b in its type (b not NaN or +inf): z > b exactly when z >= next_above(b).
template <class E>
__device__ __forceinline__ typename E::bits next_above(typename E::bits b) {
  using B = typename E::bits;
  constexpr B sign = static_cast<B>(B(1) << (8 * sizeof(B) - 1));
  if ((b & static_cast<B>(~sign)) == 0) return 1;  // either zero
  return static_cast<B>((b & sign) ? b - 1 : b + 1);
}

// Order-preserving unsigned image of a float (both zeros alike) and back.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.f));
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// Two fp32 values in one 64-bit register: one instruction rounds both (the same rounding as the
// scalar operations).
using F32x2 = unsigned long long;
__device__ __forceinline__ F32x2 pack_f32x2(float lo, float hi) {
  F32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(F32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F32x2 add2(F32x2 a, F32x2 b) {
  F32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F32x2 mul2(F32x2 a, F32x2 b) {
  F32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F32x2 fma2(F32x2 a, F32x2 b, F32x2 c) {
  F32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

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

// A row (or the rest of one): its first n elements are valid. AL: it starts on a 16-byte boundary
// (decided once for a launch; the general form costs 15 more instructions a pack, 1.9 an element,
// which at 16-bit types is a quarter of what the row statistics take).
template <class E_, bool AL_>
struct Row {
  using E = E_;
  static constexpr bool AL = AL_;
  const typename E::bits* p;
  int32_t n;
  uint32_t shift;  // bytes that p lies past a 16-byte boundary; the same for every thread
  int32_t* err;    // for the index checks of debug-checks builds
  int32_t room;    // likewise: bytes before p that may be read (a copy of a part of a row has some)
  __device__ __forceinline__ Row(const typename E::bits* p_, int n_, int32_t* err_, int room_ = 0)
      : p(p_), n(n_), shift(AL ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p_) & 15u)), err(err_),
        room(room_) {}
  __device__ __forceinline__ float at(int64_t c) const { return dbg_ok(c >= 0 && c < n, err) ? E::to_f32(p[c]) : 0.f; }
};

// True when pack columns [c0, c1) (multiples of 8) load as vectors inside the row.
template <class R>
__device__ __forceinline__ bool packs_inside(const R& r, int c0, int c1) {
  if constexpr (R::AL) return c1 <= r.n;
  return (c0 > 0 || r.shift == 0) && c1 + static_cast<int>((16u - r.shift) / sizeof(*r.p)) <= r.n;
}

__device__ __forceinline__ void ld_vec(uint32_t* w, const void* p) {
  const uint4 v = *static_cast<const uint4*>(p);
  w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
}

// Pack at column c0 (a multiple of 8); packs_inside must hold for it.
template <class R, class E = typename R::E>
__device__ __forceinline__ Pack<E> load_pack(const R& r, int c0) {
  constexpr int W = Pack<E>::WORDS, EB = Pack<E>::EB;
  Pack<E> k{};
  // the first byte of the first vector and the last of the last one lie in the row
  if (!dbg_ok(c0 >= 0 && static_cast<int64_t>(c0) * EB + r.room >= r.shift &&
                  static_cast<int64_t>(c0 + 8) * EB + (R::AL ? 0 : 16 - static_cast<int>(r.shift)) <=
                      static_cast<int64_t>(r.n) * EB,
              r.err))
    return k;
  const char* q = reinterpret_cast<const char*>(r.p) + static_cast<int64_t>(c0) * EB;
  if constexpr (R::AL) {
#pragma unroll
    for (int i = 0; i < W; i += 4) ld_vec(k.w + i, q + 4 * i);
  } else {
    q -= r.shift;
    uint32_t y[W + 4];
#pragma unroll
    for (int i = 0; i < W + 4; i += 4) ld_vec(y + i, q + 4 * i);
    // words shift / 4 .. of y, then the bytes within a word
    const bool two = r.shift & 8u, one = r.shift & 4u;
    uint32_t x[W + 2];
#pragma unroll
    for (int i = 0; i < W + 2; ++i) x[i] = two ? y[i + 2] : y[i];
    if constexpr (EB == 4) {
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
  }
  return k;
}

// Pack at column c0 near the row's ends, element by element; -inf beyond the row.
template <class R, class E = typename R::E>
__device__ __noinline__ Pack<E> load_pack_edge(const R r, int c0) {
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

// Elements 2 i and 2 i + 1 of a pack.
template <class E>
__device__ __forceinline__ float2 pair(const Pack<E>& k, int i) {
  if constexpr (Pack<E>::EB == 4) return make_float2(__uint_as_float(k.w[2 * i]), __uint_as_float(k.w[2 * i + 1]));
  else return E::to_f32x2(k.w[i]);
}

// Largest element of a lane's packs (NaN is passed over).
template <class E, int N>
__device__ __forceinline__ float pack_max(const Pack<E> (&k)[N]) {
  if constexpr (Pack<E>::EB == 4) {
    float m = __uint_as_float(k[0].w[0]);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, __uint_as_float(k[j].w[i]));
    return m;
  } else {
    uint32_t x[Pack<E>::WORDS];
#pragma unroll
    for (int i = 0; i < Pack<E>::WORDS; ++i) {
      x[i] = k[0].w[i];
#pragma unroll
      for (int j = 1; j < N; ++j) x[i] = E::max2(x[i], k[j].w[i]);
    }
    const float2 m = E::to_f32x2(E::max2(E::max2(x[0], x[1]), E::max2(x[2], x[3])));
    return fmaxf(m.x, m.y);
  }
}

// ---------------------------------------------------------------------------
// row statistics
// ---------------------------------------------------------------------------
struct alignas(16) Stats {
  float m, s, u, r;
};

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFullWarp, v, d));
  return v;
}

// Packs of a lane: k[j] holds columns 256 j + 8 lane .. + 7 of the leaf; -inf beyond the row.
template <class R>
__device__ __forceinline__ void load_leaf(const R& r, int leaf, int lane, Pack<typename R::E> (&k)[LEAF_GROUPS]) {
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

// Butterfly sums of two values with one exchange a level (the bits of warp_sum): lanes 0-15 work
// on the first, lanes 16-31 on the second; lane 0 gets both.
__device__ __forceinline__ float2 warp_sum_pair(float a, float b, int lane) {
  const bool low = lane < 16;
  float v = __fadd_rn(low ? a : b, __shfl_xor_sync(kFullWarp, low ? b : a, 16));
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFullWarp, v, d));
  return make_float2(v, __shfl_down_sync(kFullWarp, v, 16));
}

// The exponents of a leaf about its maximum m (not -inf), in powers of two: x = c z - b with b = rn(c m),
// so that an element takes one product-and-sum, and r = b - c m, which fold_leaves takes out again. Where |b| is
// so large that its rounding counts in the exponent (`over`), x comes from z - m (r = 0). of() gives
// either in one form, c (z - 0) - b with the same bits or c (z - m) - 0.
struct LeafBase {
  float b, r, nm, nb;
  bool over;
  __device__ __forceinline__ float of(float z, float c) const { return __fmaf_rn(__fadd_rn(z, nm), c, nb); }
};
__device__ __forceinline__ LeafBase leaf_base(float m, float c) {
  const float b = __fmul_rn(m, c);
  const bool over = !(fabsf(b) <= 268435456.f);  // 2^28: up to there |r| <= 16, far inside the range of 2^r
  return LeafBase{b, over ? 0.f : -__fmaf_rn(m, c, -b), over ? -m : 0.f, over ? 0.f : -b, over};
}

// s and, with ENT, u of a leaf about its maximum m (not -inf), and *r. NaN or +inf among the columns makes
// s NaN.
template <bool ENT, class E>
__device__ __forceinline__ float2 leaf_sums(const Pack<E> (&k)[LEAF_GROUPS], float m, float c, float* r, int lane) {
  constexpr float kHuge = 3.4028235e38f;
  const LeafBase at = leaf_base(m, c);
  *r = at.r;
  float sl = 0.f, ul = 0.f;
  const auto sums = [&] {
    const F32x2 nb = pack_f32x2(-at.b, -at.b), cc = pack_f32x2(c, c);
    F32x2 s2 = 0, u2 = 0;  // even and odd columns
#pragma unroll
    for (int j = 0; j < LEAF_GROUPS; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 z = pair(k[j], i);
        const F32x2 xx = fma2(pack_f32x2(z.x, z.y), cc, nb);
        const float2 x = unpack_f32x2(xx);
        const F32x2 w = pack_f32x2(ex2_approx(x.x), ex2_approx(x.y));
        s2 = add2(s2, w);
        if constexpr (ENT) u2 = fma2(w, xx, u2);
      }
    const float2 s = unpack_f32x2(s2), u = unpack_f32x2(u2);
    sl = __fadd_rn(s.x, s.y);
    if constexpr (ENT) ul = __fadd_rn(u.x, u.y);
  };
  // x kept finite where a masked column (weight 0) has -inf (a NaN logit reaches s through its weight), or
  // with `over`. In single values: paired ones spill (4096 rows of 151936 in fp32 with 64 alternatives: 386 -> 418 us).
  const auto careful_sums = [&] {
    float v[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < LEAF_GROUPS; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 z = pair(k[j], i / 2);
        const float x = at.of(i & 1 ? z.y : z.x, c), e = ex2_approx(x);
        w[i & 1] = __fadd_rn(w[i & 1], e);
        if constexpr (ENT) v[i & 1] = __fmaf_rn(e, fmaxf(x, -kHuge), v[i & 1]);
      }
    sl = __fadd_rn(w[0], w[1]);
    ul = __fadd_rn(v[0], v[1]);
  };
  if constexpr (!ENT) {
    if (at.over) careful_sums();
    else sums();
  } else {
    sums();
    if (at.over || __any_sync(kFullWarp, isnan(ul))) careful_sums();
  }
  if constexpr (!ENT) return make_float2(warp_sum(sl), 0.f);
  return warp_sum_pair(sl, ul, lane);
}

template <class E>
__device__ __forceinline__ bool any_nan(const Pack<E> (&k)[LEAF_GROUPS]) {
  bool nan = false;
#pragma unroll
  for (int j = 0; j < LEAF_GROUPS; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 z = pair(k[j], i);
      nan |= isnan(z.x) || isnan(z.y);
    }
  return __any_sync(kFullWarp, nan);
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
    const float e = __fmaf_rn(__fsub_rn(x.m, M), c, x.r);  // the leaf's base against the row's
    const float f = ex2_approx(e);
    S = __fmaf_rn(x.s, f, S);
    // u relative to M: sum w (x + e); a leaf too far down to count adds nothing
    if (f != 0.f) U = __fmaf_rn(f, __fmaf_rn(x.s, e, x.u), U);
  }
  return Stats{M, warp_sum(S), warp_sum(U), 0.f};
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

// What a row's log probabilities are formed from: log p = s (z - m) - l, with m = M and l = log S. An
// empty row has m = -inf (and l = 0), a row that holds NaN or +inf l = NaN.
struct RowLog {
  float m, l;
};

__device__ __forceinline__ RowLog row_log(const Stats& r) {
  if (isnan(r.s)) return RowLog{quiet_nan(), quiet_nan()};
  if (r.s == 0.f) return RowLog{neg_inf(), 0.f};
  return RowLog{r.m, fmaxf(logf(r.s), 0.f)};  // S >= 1, the maximum's own term, but for its rounding
}

// lse = s M + log S; -inf for an empty row alone, NaN for one that holds NaN or +inf. Where s M is beyond
// fp32 it is +inf or, below, the lowest finite value.
__device__ __forceinline__ float row_lse(const RowLog& q, float s) {
  if (q.m == neg_inf()) return neg_inf();
  const float lse = __fmaf_rn(q.m, s, q.l);
  return lse == neg_inf() ? -3.4028235e38f : lse;
}

__device__ __forceinline__ float row_entropy(const Stats& r) {
  if (isnan(r.s)) return quiet_nan();
  if (r.s == 0.f) return 0.f;
  constexpr float kLn2 = 0.69314718f;
  // neither term is below 0 but for the rounding of S and of the leaf's base
  return fmaxf(__fsub_rn(logf(r.s), __fmul_rn(kLn2, __fdiv_rn(r.u, r.s))), 0.f);
}

// log p = s (z - m) - l of a column. -inf where the row is empty. With s < 1, s z - s m may be within fp32
// where z - m is not.
__device__ __forceinline__ float token_logp(float z, float s, const RowLog& q) {
  if (q.m == neg_inf()) return neg_inf();
  const float d = __fsub_rn(z, q.m);
  return d == neg_inf() && s < 1.f ? __fsub_rn(__fmaf_rn(z, s, -__fmul_rn(q.m, s)), q.l) : __fmaf_rn(d, s, -q.l);
}

// log p of a column and of a pair, d = s (z - m) - l, as the gradients form it. AWAY: m may be other than 0
// (z - 0 is z: the bits are the same).
template <bool AWAY>
__device__ __forceinline__ float log_p(float z, float s, const RowLog& q) {
  return __fmaf_rn(AWAY ? __fsub_rn(z, q.m) : z, s, -q.l);
}
template <bool AWAY>
__device__ __forceinline__ F32x2 log_p(float2 z, float s, const RowLog& q) {
  F32x2 x = pack_f32x2(z.x, z.y);
  if constexpr (AWAY) x = add2(x, pack_f32x2(-q.m, -q.m));
  return fma2(x, pack_f32x2(s, s), pack_f32x2(-q.l, -q.l));
}

// e^d as the gradients form it, d = log p.
__device__ __forceinline__ float prob_of(float d) { return ex2_approx(__fmul_rn(d, kLog2e)); }

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
