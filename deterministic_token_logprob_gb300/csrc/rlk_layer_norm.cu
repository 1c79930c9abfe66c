// rlk_layer_norm.cu -- layer norm over rows of hidden values, and its gradient.
//
//   m = mean_c x_c (0 when not centered),  r = (mean_c (x_c - m)^2 + eps)^(-1/2)
//   h_c = (x_c - m) r,  y_c = h_c w_c + b_c
// and, with g_c = dy_c w_c,
//   dx_c = r (g_c - [centered] mean g - h_c mean(g h)),   dw_c = sum_t dy_tc h_tc,   db_c = sum_t dy_tc
//
// Both directions are bound by memory: the forward reads x and writes y, the backward reads x and dy
// and writes dx, once each.
#include <type_traits>

#include "rlk_rows.cuh"

namespace rlk {
namespace {


// Warps that take a row in the backward. A row's two sums and its few scalars cost every warp the same, so a thread has 2 packs,
// whose sums of dw and db it keeps, before another warp has any (in the forward 4: with_fwd_team).
__host__ __device__ constexpr int bwd_warps(int n) { return n <= 512 ? 1 : n <= 1024 ? 2 : n <= 2048 ? 4 : 8; }

// Rows are dealt to strips, whose parts of dw and db are summed apart: row t belongs to strip t mod S. S follows
// from T and the width alone, and so does the order of the sum over rows: two CTAs on each of 152 SMs,
// each of as many teams as the width leaves room for.
constexpr int NORM_CTAS = 304;
__host__ __device__ constexpr int strips_of(int64_t T, int n) {
  return static_cast<int>(T < NORM_CTAS * (8 / bwd_warps(n)) ? T : NORM_CTAS * (8 / bwd_warps(n)));
}

// A row that overflows fp32 in its sums is taken once more as x 2^-80.
constexpr float kShrink = 8.271806125530277e-25f;  // 2^-80
constexpr float kGrow = 1.2089258196146292e24f;    // 2^80

struct Vector {  // weight or bias: fp32 or the rows' type, or absent
  const void* p;
  bool f32;
};

// 8 columns of a vector; AL: it starts on a 32-byte boundary and n is a multiple of 8.
template <class E, bool AL>
__device__ __forceinline__ void vector8(const Vector& w, int c0, int n, float absent, F32x2 (&v)[4], int32_t* err) {
  if (!w.p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = both(absent);
  } else if (sizeof(typename E::bits) == 4 || w.f32) {
    unpack(load_columns<F32, AL>(static_cast<const uint32_t*>(w.p), c0, n, err), v);
  } else {
    unpack(load_columns<E, AL>(static_cast<const typename E::bits*>(w.p), c0, n, err), v);
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
struct RowStats {
  float k;     // what x is multiplied by (1, or 2^-80 for a row whose sums are beyond fp32)
  float m, c;  // mean of k x: m + c (m rounded, c what that lost)
  float r;     // 1 / sqrt(mean (k x - mean)^2 + k^2 eps)
};

__device__ __forceinline__ void shrink(F32x2 (&v)[4], float k) {
  if (k == 1.f) return;  // the same for the whole team
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(k));
}

// 1 / sqrt(v) of a normal v: the approximation and one Newton step
__device__ __forceinline__ float inverse_root(float v) {
  const float y = rsqrtf(v);
  return __fmaf_rn(__fmul_rn(0.5f, y), __fmaf_rn(-__fmul_rn(v, y), y, 1.f), y);
}

// r from the mean square q of k x - m
__device__ __forceinline__ float row_scale(const RowStats& s, float q, float eps) {
  const float var = fmaxf(__fmaf_rn(-s.c, s.c, q), 0.f);
  if (!isfinite(q)) return quiet_nan();  // a NaN or an infinity in the row
  if (s.k == 1.f) return inverse_root(__fadd_rn(var, eps));
  if (var > 1.17549435e-38f) return inverse_root(var);  // eps is 2^-34 of it at most
  return __fmul_rn(inverse_root(__fadd_rn(__fmul_rn(__fmul_rn(var, kGrow), kGrow), eps)), kGrow);
}

struct NormArgs {
  const void* x;
  void* y;
  int64_t T, ld, out_ld;
  int32_t H;
  int32_t ahead; // rows from one to the one that is asked for with it
  float inv;     // 1 / H
  bool centered;
  float eps;
  Vector w, b;
  float *mean, *rstd;
  int32_t* err;
};

__device__ __forceinline__ void put_stats(const NormArgs& a, int64_t t, const RowStats& s) {
  const float back = s.k == 1.f ? 1.f : kGrow;
  if (a.mean) a.mean[t] = isnan(s.r) ? s.r : __fmul_rn(__fadd_rn(s.m, s.c), back);
  if (a.rstd) a.rstd[t] = __fmul_rn(s.r, s.k);
  if (isnan(s.r) && a.err) atomicOr(a.err, RLK_FLAG_NONFINITE);
}

// A row of n results by way of shared memory, for rows of any alignment: packs are put there as they come, then the team's W
// warps write them out in the order of addresses. (Element by element from the packs, every store touches as many sectors as
// the pack's eight together.) `stage`: n elements rounded up to a pack; a team barrier stands before its next use.
template <class O, int W>
__device__ __forceinline__ void write_out(typename O::bits* out, const typename O::bits* stage, int n, int tid, int32_t* err) {
  team_barrier<W>();
  if constexpr (W == 1) __syncwarp();
#pragma unroll 8
  for (int c = tid; c < n; c += 32 * W)
    if (dbg_ok(c >= 0 && c < n, err)) out[c] = stage[c];
}

// y of a pack, v its k x - m
template <class E, bool AL>
__device__ __forceinline__ void norm_pack(const NormArgs& a, int c0, F32x2 (&v)[4], const RowStats& s) {
  F32x2 w[4], b[4];
  vector8<E, AL>(a.w, c0, a.H, 1.f, w, a.err);
  vector8<E, AL>(a.b, c0, a.H, 0.f, b, a.err);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (a.centered) v[i] = add2(v[i], both(-s.c));
    v[i] = fma2(mul2(v[i], both(s.r)), w[i], b[i]);
  }
}

// Rows of up to 16384 columns, K packs a thread, which stay in registers (as k x, then k x - m) between the two sums and the
// result. W warps a row: 8 / W rows a CTA, four CTAs an SM. Bound by memory in fp32 (0.91 of the copy rate at 8192 rows of 4096
// into bf16), by instructions and latency in 16-bit types (0.67).
template <class E, class O, int W, int K, bool AL>
__global__ void __launch_bounds__(ROW_CTA, K <= 4 ? 4 : 2) norm_fwd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];  // stages (write_out), unless AL
  __shared__ __align__(16) float rooms[32];
  const int team = threadIdx.x / (32 * W), tid = threadIdx.x % (32 * W), packs = (a.H + 7) / 8;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (8 / W) + team;
  if (t >= a.T) return;  // the whole team
  const auto* x = static_cast<const typename E::bits*>(a.x) + t * a.ld;
  float* room = rooms + team * 4 * W;
  F32x2 v[K][4];
  const auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (tid + j * 32 * W < packs) f(v[j], 8 * (tid + j * 32 * W));
  };
  RowStats s{1.f, 0.f, 0.f, 0.f};
  float q;
  if (AL && tid == 0 && t + a.ahead < a.T)  // the row of a CTA to come, into L2: more on its way than registers hold
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(x + a.ahead * a.ld), "r"(a.H * static_cast<int>(sizeof(*x))) : "memory");
  for (;;) {
    each([&](F32x2 (&d)[4], int c0) { unpack(load_columns<E, AL>(x, c0, a.H, a.err), d); });
    if (s.k != 1.f) each([&](F32x2 (&d)[4], int) { shrink(d, s.k); });
    F32x2 p = 0, b = 0;
    if (a.centered) {
      each([&](F32x2 (&d)[4], int) { p = add2(p, tree4(d)); });
      s.m = __fmul_rn(team_sum<W>(low_plus_high(p), 0.f, room).x, a.inv);
      p = 0;
      each([&](F32x2 (&d)[4], int c0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = add2(d[i], both(-s.m));
        if (!AL && c0 + 8 > a.H) clear_beyond(d, c0, a.H);
        b = add2(b, tree4(d));
      });
    }
    each([&](F32x2 (&d)[4], int) { p = dot4(d, d, p); });
    const float2 sums = team_sum<W>(low_plus_high(p), low_plus_high(b), room + 2 * W);
    q = __fmul_rn(sums.x, a.inv);
    s.c = __fmul_rn(sums.y, a.inv);
    if (isfinite(q) || s.k != 1.f) break;
    s.k = kShrink;
    team_barrier<W>();  // the sums to come use the room again
  }
  s.r = row_scale(s, q, a.eps);
  if (tid == 0) put_stats(a, t, s);
  auto* y = static_cast<typename O::bits*>(a.y) + t * a.out_ld;
  auto* stage = reinterpret_cast<typename O::bits*>(dyn) + team * 8 * packs;
  each([&](F32x2 (&d)[4], int c0) {
    norm_pack<E, AL>(a, c0, d, s);
    if constexpr (AL) store_columns<O, true>(y, c0, a.H, d, a.err);
    else store_columns<O, true, false>(stage, c0, 8 * packs, d, a.err);
  });
  if constexpr (!AL) write_out<O, W>(y, stage, a.H, tid, a.err);
}

// Longer rows, and many misaligned ones of more than 8192 columns, by 8 warps: they are read three times (from L1 or L2 after the
// first). Misaligned rows keep registers from more than two CTAs an SM otherwise (4096 of 12001 in bf16: 110 us for 141, in fp32 171 for
// 179), which few rows do not need (400 of 16383 in fp32: 29.4 us for 25.6).
template <class E, class O>
__global__ void __launch_bounds__(ROW_CTA) norm_fwd_long_kernel(const NormArgs a) {
  __shared__ __align__(16) float rooms[32];
  constexpr int W = 8;
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  const auto* x = static_cast<const typename E::bits*>(a.x) + t * a.ld;
  float* room = rooms;
  RowStats s{1.f, 0.f, 0.f, 0.f};
  const auto each = [&](auto f) {  // k x - m of every pack
    for (int c = 8 * tid; c < a.H; c += 8 * 32 * W) {
      F32x2 v[4];
      unpack(load_columns<E, false>(x, c, a.H, a.err), v);
      shrink(v, s.k);
      if (a.centered) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = add2(v[i], both(-s.m));
      }
      f(c, v);
    }
  };
  float q;
  for (;;) {
    s.m = 0.f;
    F32x2 p = 0, b = 0;
    if (a.centered) {
      each([&](int, F32x2 (&d)[4]) { p = add2(p, tree4(d)); });
      s.m = __fmul_rn(team_sum<W>(low_plus_high(p), 0.f, room).x, a.inv);
      p = 0;
    }
    each([&](int c0, F32x2 (&d)[4]) {
      if (c0 + 8 > a.H) clear_beyond(d, c0, a.H);
      if (a.centered) b = add2(b, tree4(d));
      p = dot4(d, d, p);
    });
    const float2 sums = team_sum<W>(low_plus_high(p), low_plus_high(b), room + 2 * W);
    q = __fmul_rn(sums.x, a.inv);
    s.c = __fmul_rn(sums.y, a.inv);
    if (isfinite(q) || s.k != 1.f) break;
    s.k = kShrink;
    team_barrier<W>();
  }
  s.r = row_scale(s, q, a.eps);
  if (tid == 0) put_stats(a, t, s);
  auto* y = static_cast<typename O::bits*>(a.y) + t * a.out_ld;
  each([&](int c0, F32x2 (&d)[4]) {
    norm_pack<E, false>(a, c0, d, s);
    store_columns<O, false>(y, c0, a.H, d, a.err);
  });
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct NormGradArgs {
  const void *dy, *x;
  void* dx;
  int64_t T, dy_ld, ld, dx_ld;
  int32_t H;
  float inv;               // 1 / H
  Vector w;
  const float *mean, *rstd;
  float* row;              // [T][2]: mean g, mean(g h)
  float *part_w, *part_b;  // [strips][H]
  float *dw, *db;
  int32_t strips, stages;
  int32_t* err;
};

// h of a pack, into x. A finite row may differ from its mean by more than fp32 holds (its r is 2^-120 at most, H being 2^16): it is halved
// first, which loses nothing there, and r doubled.
__device__ __forceinline__ void norm_h(F32x2 (&x)[4], float m, float r) {
  const bool wide = r < 7.888609052210118e-31f;  // 2^-100
  const float k = wide ? 0.5f : 1.f, km = __fmul_rn(-k, m), rk = wide ? __fadd_rn(r, r) : r;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = mul2(fma2(x[i], both(k), both(km)), both(rk));
}

// the pack's part of sum g (where the mean counts) and sum g h
__device__ __forceinline__ void norm_sums(const F32x2 (&h)[4], const F32x2 (&dy)[4], const F32x2 (&w)[4], bool centered, F32x2& s1,
                                          F32x2& s2) {
  F32x2 g[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = mul2(dy[i], w[i]);
  if (centered) s1 = dot4(dy, w, s1);
  s2 = dot4(g, h, s2);
}

// dx of a pack
__device__ __forceinline__ void norm_dx(const F32x2 (&h)[4], const F32x2 (&dy)[4], const F32x2 (&w)[4], float c1, float c2,
                                        float r, F32x2 (&dx)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) dx[i] = mul2(fma2(h[i], both(-c2), fma2(dy[i], w[i], both(-c1))), both(r));
}

// the pack's part of dw and, where it is wanted, db
__device__ __forceinline__ void norm_vectors(const F32x2 (&h)[4], const F32x2 (&dy)[4], bool bias, F32x2 (&sw)[4], F32x2 (&sb)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sw[i] = fma2(dy[i], h[i], sw[i]);
  if (!bias) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) sb[i] = add2(sb[i], dy[i]);
}

__device__ __forceinline__ void copy_async_16(void* shared, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(shared)), "l"(global) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The packs of one row that a warp's threads own (32 W packs apart for the j-th of each), copied into shared memory and read from it
// by the same warp. Copies go by 16-byte vectors in the order of addresses, into the same order, but that the two halves of
// an fp32 pack change places in every other four packs: its reads, 32 bytes apart, then meet no bank twice. (Halves kept apart in
// two arrays cost the copies: 8192 rows of 4096 in fp32 105 us.)
template <class E, int W, int K>
struct RowRing {
  static constexpr int HALVES = sizeof(typename E::bits) * 8 / 16;
  static constexpr int STEP = 32 * W * HALVES;  // vectors from a thread's pack to its next
  static __device__ __forceinline__ int place(int vec) { return HALVES == 2 ? vec ^ (vec >> 3 & 1) : vec; }
  // row: of the matrix, from the warp's vector `lane` on; room: of the ring, from the place of that vector on; left: vectors from
  // that one to the row's end. (Places differ as vectors do over multiples of 16.)
  static __device__ __forceinline__ void fetch(uint4* room, const uint4* row, int left) {
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int i = 0; i < HALVES; ++i)
        if (const int u = j * STEP + i * 32; u < left) copy_async_16(room + u, row + u);
  }
  static __device__ __forceinline__ void read(const uint4* room, int p, F32x2 (&v)[4]) {
    Pack<E> k;
#pragma unroll
    for (int i = 0; i < HALVES; ++i) ld_vec(k.w + 4 * i, room + place(p * HALVES + i));
    unpack(k, v);
  }
};

// Rows of up to 8192 columns. A team of W warps takes a strip's rows in turn; the next stages - 1 rows are on their way into
// shared memory meanwhile (unless they are misaligned). Each thread keeps the sums of dw and db of its columns. 8192 rows of 4096 in
// bf16 take 37.8 us with the fold (0.78 of the copy rate: 16 warps an SM issue in 47 % of the cycles), in fp32 64 (0.93).
template <class E, class O, int W, int K, bool AL>
__global__ void __launch_bounds__(ROW_CTA, K <= 2 ? 2 : 1) norm_bwd_kernel(const NormGradArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];  // AL: the rows to come; else stages (write_out)
  __shared__ __align__(16) float rooms[32];
  using XRing = RowRing<E, W, K>;
  using DRing = RowRing<O, W, K>;
  constexpr int XH = XRing::HALVES, DH = DRing::HALVES;
  const int team = threadIdx.x / (32 * W), tid = threadIdx.x % (32 * W), warp = tid >> 5, lane = tid & 31, packs = (a.H + 7) / 8;
  const int64_t strip = static_cast<int64_t>(blockIdx.x) * (8 / W) + team;
  if (strip >= a.strips) return;  // the whole team
  const int stage_vecs = packs * (XH + DH);
  uint4* ring = reinterpret_cast<uint4*>(dyn) + static_cast<int64_t>(team) * a.stages * stage_vecs;
  auto* staged = reinterpret_cast<typename E::bits*>(dyn) + team * 8 * packs;
  float* room = rooms + team * 4 * W;
  const auto x_row = [&](int64_t t) { return static_cast<const typename E::bits*>(a.x) + t * a.ld; };
  const auto dy_row = [&](int64_t t) { return static_cast<const typename O::bits*>(a.dy) + t * a.dy_ld; };
  // the copies: of row t_in, this thread's first vector of it, and where that goes in stage 0
  const int xv = warp * 32 * XH + lane, dv = warp * 32 * DH + lane;
  const uint4 *x_in = reinterpret_cast<const uint4*>(x_row(strip)) + xv, *dy_in = reinterpret_cast<const uint4*>(dy_row(strip)) + dv;
  const int64_t x_step = a.strips * a.ld * static_cast<int64_t>(sizeof(typename E::bits)) / 16;
  const int64_t dy_step = a.strips * a.dy_ld * static_cast<int64_t>(sizeof(typename O::bits)) / 16;
  uint4 *x_to = ring + XRing::place(xv), *dy_to = ring + packs * XH + DRing::place(dv);
  int64_t t_in = strip;
  const auto fetch = [&](int stage) {
    if constexpr (AL) {
      if (t_in < a.T) {
        XRing::fetch(x_to + stage * stage_vecs, x_in, packs * XH - xv);
        DRing::fetch(dy_to + stage * stage_vecs, dy_in, packs * DH - dv);
      }
      copies_commit();
      x_in += x_step;
      dy_in += dy_step;
      t_in += a.strips;
    }
  };
  for (int i = 0; i < a.stages - 1; ++i) fetch(i);
  F32x2 w[K][4], sw[K][4], sb[K][4];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int c0 = 8 * (tid + j * 32 * W);
    if (c0 < a.H) vector8<E, AL>(a.w, c0, a.H, 1.f, w[j], a.err);
#pragma unroll
    for (int i = 0; i < 4; ++i) sw[j][i] = sb[j][i] = 0;
  }
  const bool centered = a.mean, bias = a.part_b;
  float m = centered ? a.mean[strip] : 0.f, r = a.rstd[strip];
  int stage = 0, odd = 0;
  for (int64_t t = strip; t < a.T; t += a.strips) {
    if constexpr (AL) __syncwarp();  // the stage that is filled next has been read by the whole warp
    fetch(stage == 0 ? a.stages - 1 : stage - 1);
    const int64_t next = t + a.strips < a.T ? t + a.strips : t;
    const float m1 = centered ? a.mean[next] : 0.f, r1 = a.rstd[next];
    F32x2 h[K][4], dy[K][4], s1 = 0, s2 = 0;
    if constexpr (AL) {
      if (a.stages == 3) copies_wait<2>();
      else copies_wait<3>();
      __syncwarp();
    }
    const uint4* xs = ring + stage * stage_vecs;
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (const int p = tid + j * 32 * W; p < packs) {
        if constexpr (AL) {
          XRing::read(xs, p, h[j]);
          DRing::read(xs + packs * XH, p, dy[j]);
        } else {
          unpack(load_columns<E, false>(x_row(t), 8 * p, a.H, a.err), h[j]);
          unpack(load_columns<O, false>(dy_row(t), 8 * p, a.H, a.err), dy[j]);
        }
      }
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (const int p = tid + j * 32 * W; p < packs) {
        norm_h(h[j], m, r);
        if (!AL && 8 * p + 8 > a.H) clear_beyond(h[j], 8 * p, a.H);
        norm_vectors(h[j], dy[j], bias, sw[j], sb[j]);
        norm_sums(h[j], dy[j], w[j], centered, s1, s2);
      }
    if (a.dx) {
      const float2 s = team_sum<W>(low_plus_high(s1), low_plus_high(s2), room + odd * 2 * W);
      const float c1 = __fmul_rn(s.x, a.inv), c2 = __fmul_rn(s.y, a.inv);
      auto* dx = static_cast<typename E::bits*>(a.dx) + t * a.dx_ld;
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (const int p = tid + j * 32 * W; p < packs) {
          F32x2 v[4];
          norm_dx(h[j], dy[j], w[j], c1, c2, r, v);
          if constexpr (AL) store_columns<E, true>(dx, 8 * p, a.H, v, a.err);
          else store_columns<E, true, false>(staged, 8 * p, 8 * packs, v, a.err);
        }
      if constexpr (!AL) write_out<E, W>(dx, staged, a.H, tid, a.err);  // the next row's sum stands before the next stage's packs
      if constexpr (!AL && W == 1) __syncwarp();
    }
    m = m1;
    r = r1;
    odd ^= 1;
    stage = stage + 1 == a.stages ? 0 : stage + 1;
  }
  griddep_launch_dependents();
  if constexpr (AL) copies_wait<0>();
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int c0 = 8 * (tid + j * 32 * W);
    if (c0 >= a.H) continue;
    if (a.part_w) store_columns<F32, AL>(reinterpret_cast<uint32_t*>(a.part_w) + strip * a.H, c0, a.H, sw[j], a.err);
    if (a.part_b) store_columns<F32, AL>(reinterpret_cast<uint32_t*>(a.part_b) + strip * a.H, c0, a.H, sb[j], a.err);
  }
}

// Longer rows: first what the whole row gives (8 warps), then the columns.
template <class E, class O, bool AL>
__global__ void __launch_bounds__(ROW_CTA) norm_bwd_rows_kernel(const NormGradArgs a) {
  __shared__ __align__(16) float room[16];
  const int64_t t = blockIdx.x;
  const auto* x = static_cast<const typename E::bits*>(a.x) + t * a.ld;
  const auto* dy = static_cast<const typename O::bits*>(a.dy) + t * a.dy_ld;
  const float m = a.mean ? a.mean[t] : 0.f, r = a.rstd[t];
  F32x2 s1 = 0, s2 = 0;
#pragma unroll 2
  for (int c = 8 * threadIdx.x; c < a.H; c += 8 * ROW_CTA) {
    F32x2 h[4], dv[4], w[4];
    unpack(load_columns<E, AL>(x, c, a.H, a.err), h);
    unpack(load_columns<O, AL>(dy, c, a.H, a.err), dv);
    vector8<E, AL>(a.w, c, a.H, 1.f, w, a.err);
    norm_h(h, m, r);
    if (!AL && c + 8 > a.H) clear_beyond(h, c, a.H);
    norm_sums(h, dv, w, a.mean, s1, s2);
  }
  const float2 s = team_sum<8>(low_plus_high(s1), low_plus_high(s2), room);
  if (threadIdx.x == 0) {
    a.row[2 * t] = __fmul_rn(s.x, a.inv);
    a.row[2 * t + 1] = __fmul_rn(s.y, a.inv);
  }
}

template <class E, class O, bool AL>
__global__ void __launch_bounds__(ROW_CTA) norm_bwd_columns_kernel(const NormGradArgs a) {
  const int c0 = 8 * static_cast<int>(blockIdx.x * ROW_CTA + threadIdx.x);
  if (c0 >= a.H) return;
  F32x2 w[4], sw[4] = {}, sb[4] = {};
  vector8<E, AL>(a.w, c0, a.H, 1.f, w, a.err);
#pragma unroll 2
  for (int64_t t = blockIdx.y; t < a.T; t += a.strips) {
    F32x2 h[4], dv[4], v[4];
    unpack(load_columns<E, AL>(static_cast<const typename E::bits*>(a.x) + t * a.ld, c0, a.H, a.err), h);
    unpack(load_columns<O, AL>(static_cast<const typename O::bits*>(a.dy) + t * a.dy_ld, c0, a.H, a.err), dv);
    const float m = a.mean ? a.mean[t] : 0.f, r = a.rstd[t];
    norm_h(h, m, r);
    norm_vectors(h, dv, a.part_b, sw, sb);
    if (!a.dx) continue;
    norm_dx(h, dv, w, a.row[2 * t], a.row[2 * t + 1], r, v);
    store_columns<E, AL>(static_cast<typename E::bits*>(a.dx) + t * a.dx_ld, c0, a.H, v, a.err);
  }
  const int64_t at = static_cast<int64_t>(blockIdx.y) * a.H;
  if (a.part_w) store_columns<F32, AL>(reinterpret_cast<uint32_t*>(a.part_w) + at, c0, a.H, sw, a.err);
  if (a.part_b) store_columns<F32, AL>(reinterpret_cast<uint32_t*>(a.part_b) + at, c0, a.H, sb, a.err);
}

// dw and db from the strips' parts: warp i adds strips i, i + 32, ... in ascending order, then the 32 sums are added as a
// balanced tree.
__global__ void __launch_bounds__(1024) norm_fold_kernel(const NormGradArgs a) {
  __shared__ float sums[32][33];
  const float* part = blockIdx.y ? a.part_b : a.part_w;
  float* out = blockIdx.y ? a.db : a.dw;
  if (!part) return;
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < a.H) {
#pragma unroll 8
    for (int i = warp; i < a.strips; i += 32) s = __fadd_rn(s, part[static_cast<int64_t>(i) * a.H + c]);
  }
  sums[lane][warp] = s;
  __syncthreads();
  const float v = warp_sum(sums[warp][lane]);  // a column a warp
  if (lane == 0 && blockIdx.x * 32 + warp < a.H) out[blockIdx.x * 32 + warp] = v;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline bool vector_ok(const void* p, int32_t dtype, int32_t rows_dtype) {
  return !p || ((dtype == rows_dtype || dtype == RLK_DTYPE_F32) && on_boundary(p, dtype_bytes(dtype)));
}

template <int V>
using Int = std::integral_constant<int, V>;

// Calls f with the warps a row and the packs a thread, for rows of H columns. Forward: up to 4 packs a thread in 16-bit types,
// where instructions count (8192 rows of 4096 in bf16: 29.5 us, with 2 packs 34.4), and 2 in fp32 (to bf16: 32.7 us, with 4 34.9).
template <class F>
inline rlk_status with_fwd_team(int64_t H, bool fp32, F f) {
  if (H <= 256) return f(Int<1>{}, Int<1>{});
  if (H <= 512) return f(Int<1>{}, Int<2>{});
  if (H > 8192) return f(Int<8>{}, Int<8>{});
  if (H > 4096) return f(Int<8>{}, Int<4>{});
  if (fp32) return H <= 1024 ? f(Int<2>{}, Int<2>{}) : H <= 2048 ? f(Int<4>{}, Int<2>{}) : f(Int<8>{}, Int<2>{});
  return H <= 1024 ? f(Int<1>{}, Int<4>{}) : H <= 2048 ? f(Int<2>{}, Int<4>{}) : f(Int<4>{}, Int<4>{});
}
template <class F>
inline rlk_status with_bwd_team(int64_t H, F f) {
  if (H <= 256) return f(Int<1>{}, Int<1>{});
  if (H <= 512) return f(Int<1>{}, Int<2>{});
  if (H <= 1024) return f(Int<2>{}, Int<2>{});
  if (H <= 2048) return f(Int<4>{}, Int<2>{});
  if (H <= 4096) return f(Int<8>{}, Int<2>{});
  return f(Int<8>{}, Int<4>{});
}

constexpr int64_t FWD_KEPT = 16384;  // columns of a row that stays in registers (8 packs a thread)
constexpr int64_t FWD_KEPT_ODD = 8192; // of many misaligned rows
constexpr int64_t FWD_MANY = 1024;     // rows
constexpr int64_t BWD_KEPT = 8192;   // and of one whose sums of dw and db do (4 packs)
constexpr int BWD_SMEM = 110 * 1024;      // of each of the two CTAs of an SM
constexpr int BWD_SMEM_ONE = 220 * 1024;  // of its only one
constexpr int64_t FWD_AHEAD = 16 << 20;   // bytes
constexpr int FWD_SMEM = static_cast<int>(FWD_KEPT * sizeof(float));

// Launches a kernel whose dynamic shared memory may be up to `most` bytes.
template <auto Kernel, class A>
inline rlk_status launch_rows_of(const A& a, int64_t ctas, int64_t smem, int most, cudaStream_t s) {
  static OncePerDevice allowed;
  if (!allowed([&] { return cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) == cudaSuccess; }))
    return RLK_ERR_CUDA;
  Kernel<<<static_cast<unsigned>(ctas), ROW_CTA, static_cast<size_t>(smem), s>>>(a);
  return launched();
}

template <class E, class O, int W, int K>
inline rlk_status launch_norm_fwd(const NormArgs& a, bool aligned, cudaStream_t s) {
  const int64_t ctas = (a.T + 8 / W - 1) / (8 / W);
  if (aligned) return launch_rows_of<norm_fwd_kernel<E, O, W, K, true>>(a, ctas, 0, FWD_SMEM, s);
  const int64_t stages = static_cast<int64_t>(8 / W) * ((a.H + 7) / 8 * 8) * sizeof(typename O::bits);
  return launch_rows_of<norm_fwd_kernel<E, O, W, K, false>>(a, ctas, stages, FWD_SMEM, s);
}

template <class E, class O, int W, int K>
inline rlk_status launch_norm_bwd(NormGradArgs a, bool aligned, cudaStream_t s) {
  constexpr int most = K <= 2 ? BWD_SMEM : BWD_SMEM_ONE;
  const int64_t ctas = (a.strips + 8 / W - 1) / (8 / W), columns = static_cast<int64_t>(8 / W) * ((a.H + 7) / 8 * 8);
  a.stages = 1;
  if (!aligned) return launch_rows_of<norm_bwd_kernel<E, O, W, K, false>>(a, ctas, columns * sizeof(typename E::bits), most, s);
  // 4 stages, or as many as the CTAs of an SM (two of up to 2 packs a thread, by registers) have room for: 3 at least
  const int64_t stage = columns * (sizeof(typename E::bits) + sizeof(typename O::bits));
  a.stages = static_cast<int32_t>(most / stage > 4 ? 4 : most / stage);
  return launch_rows_of<norm_bwd_kernel<E, O, W, K, true>>(a, ctas, a.stages * stage, most, s);
}

}  // namespace
}  // namespace rlk

using namespace rlk;

extern "C" {

rlk_status rlk_layer_norm_fwd(const void* x, int32_t dtype, int64_t T, int64_t H, int64_t ld, const void* weight,
                              const void* bias, int32_t weight_dtype, int32_t centered, double eps, void* y,
                              int32_t out_dtype, int64_t out_ld, float* mean, float* rstd, int32_t* err_flag,
                              void* stream) {
  rlk_status st = check_rows(x, dtype, T, H, ld);
  if (st == RLK_OK) st = check_pair(dtype, out_dtype);
  if (st == RLK_OK) st = check_rows(y, out_dtype, T, H, out_ld);
  if (st != RLK_OK) return st;
  if (!(eps >= RLK_MIN_NORM_EPS && eps <= 1.0) || dtype_bytes(weight_dtype) == 0) return RLK_ERR_INVALID_ARG;
  if (!vector_ok(weight, weight_dtype, dtype) || !vector_ok(bias, weight_dtype, dtype)) return RLK_ERR_INVALID_ARG;
  const RowSpan in{x, T, H, ld, dtype_bytes(dtype)}, out{y, T, H, out_ld, dtype_bytes(out_dtype)};
  if (!same_rows(in, out) && !rows_apart(in, out)) return RLK_ERR_INVALID_ARG;
  if (T == 0) return RLK_OK;
  const bool f32 = weight_dtype == RLK_DTYPE_F32;
  const NormArgs a{x, y, T, ld, out_ld, static_cast<int32_t>(H), static_cast<int32_t>(FWD_AHEAD / (H * in.eb)), 1.f / static_cast<float>(H), centered != 0, static_cast<float>(eps),
                   Vector{weight, f32}, Vector{bias, f32}, mean, rstd, err_flag};
  const bool al = whole_packs(x, T, H, ld, in.eb) && whole_packs(y, T, H, out_ld, out.eb) && on_boundary(weight, 32) &&
                  on_boundary(bias, 32);
  const auto s = static_cast<cudaStream_t>(stream);
  return with_pair(dtype, out_dtype, [&](auto e, auto o) {
    using E = decltype(e);
    using O = decltype(o);
    if (H > (!al && T > FWD_MANY ? FWD_KEPT_ODD : FWD_KEPT)) {
      norm_fwd_long_kernel<E, O><<<static_cast<unsigned>(T), ROW_CTA, 0, s>>>(a);
      return launched();
    }
    return with_fwd_team(H, in.eb == 4, [&](auto w, auto k) {
      constexpr int W = decltype(w)::value, K = decltype(k)::value;
      constexpr bool taken = sizeof(typename E::bits) == 4 ? !(W < 8 && K == 4) : !(K == 2 && W > 1);
      if constexpr (taken) return launch_norm_fwd<E, O, W, K>(a, al, s);
      else return RLK_ERR_UNSUPPORTED;  // with_fwd_team does not choose it for this type
    });
  });
}

size_t rlk_layer_norm_bwd_workspace(int64_t T, int64_t H) {
  if (T <= 0 || H <= 0 || H > RLK_MAX_HIDDEN) return 0;
  return carved(T * 2 * sizeof(float)) + 2 * carved(strips_of(T, static_cast<int>(H)) * H * sizeof(float));
}

rlk_status rlk_layer_norm_bwd(const void* dy, int32_t dy_dtype, int64_t dy_ld, const void* x, int32_t dtype, int64_t ld,
                              int64_t T, int64_t H, const void* weight, int32_t weight_dtype, const float* mean,
                              const float* rstd, void* dx, int64_t dx_ld, float* dw, float* db, int32_t* err_flag,
                              void* workspace, size_t workspace_bytes, void* stream) {
  rlk_status st = check_rows(x, dtype, T, H, ld);
  if (st == RLK_OK) st = check_pair(dtype, dy_dtype);
  if (st == RLK_OK) st = check_rows(dy, dy_dtype, T, H, dy_ld);
  if (st == RLK_OK && dx) st = check_rows(dx, dtype, T, H, dx_ld);
  if (st != RLK_OK) return st;
  if (dtype_bytes(weight_dtype) == 0 || !vector_ok(weight, weight_dtype, dtype)) return RLK_ERR_INVALID_ARG;
  if (!dx && !dw && !db) return RLK_ERR_INVALID_ARG;
  if (T > 0 && !rstd) return RLK_ERR_INVALID_ARG;
  const RowSpan xs{x, T, H, ld, dtype_bytes(dtype)}, ds{dy, T, H, dy_ld, dtype_bytes(dy_dtype)};
  const RowSpan os{dx, T, H, dx_ld, dtype_bytes(dtype)};
  if (dx && !((same_rows(os, xs) || rows_apart(os, xs)) && (same_rows(os, ds) || rows_apart(os, ds))))
    return RLK_ERR_INVALID_ARG;
  const auto s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // sums over no rows
    if (dw && cudaMemsetAsync(dw, 0, H * sizeof(float), s) != cudaSuccess) return RLK_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, H * sizeof(float), s) != cudaSuccess) return RLK_ERR_CUDA;
    return RLK_OK;
  }
  if (!workspace || !on_boundary(workspace, 256) || workspace_bytes < rlk_layer_norm_bwd_workspace(T, H))
    return RLK_ERR_WORKSPACE;
  NormGradArgs a{dy, x, dx, T, dy_ld, ld, dx_ld, static_cast<int32_t>(H), 1.f / static_cast<float>(H), Vector{weight, weight_dtype == RLK_DTYPE_F32},
                 mean, rstd, static_cast<float*>(workspace), nullptr, nullptr, dw, db,
                 strips_of(T, static_cast<int>(H)), 0, err_flag};
  const size_t part = carved(a.strips * H * sizeof(float));
  char* after = static_cast<char*>(workspace) + carved(T * 2 * sizeof(float));
  if (dw) a.part_w = reinterpret_cast<float*>(after);
  if (db) a.part_b = reinterpret_cast<float*>(after + part);
  const bool al = whole_packs(x, T, H, ld, xs.eb) && whole_packs(dy, T, H, dy_ld, ds.eb) &&
                  (!dx || whole_packs(dx, T, H, dx_ld, os.eb)) && on_boundary(weight, 32);
  st = with_pair(dtype, dy_dtype, [&](auto e, auto o) {
    using E = decltype(e);
    using O = decltype(o);
    if (H <= BWD_KEPT)
      return with_bwd_team(H, [&](auto w, auto k) { return launch_norm_bwd<E, O, decltype(w)::value, decltype(k)::value>(a, al, s); });
    const auto go = [&](auto aligned) {
      constexpr bool AL = decltype(aligned)::value;
      if (dx) norm_bwd_rows_kernel<E, O, AL><<<static_cast<unsigned>(T), ROW_CTA, 0, s>>>(a);
      const unsigned blocks = static_cast<unsigned>((H + 8 * ROW_CTA - 1) / (8 * ROW_CTA));
      norm_bwd_columns_kernel<E, O, AL><<<dim3(blocks, a.strips), ROW_CTA, 0, s>>>(a);
      return launched();
    };
    return al ? go(Is<true>{}) : go(Is<false>{});
  });
  if (st != RLK_OK || !(dw || db)) return st;
  return launch_after(norm_fold_kernel, dim3(static_cast<unsigned>((H + 31) / 32), 2), 1024, s, a);
}

}  // extern "C"
