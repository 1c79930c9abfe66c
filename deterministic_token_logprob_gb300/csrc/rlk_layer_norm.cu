// rlk_layer_norm.cu -- layer norm over rows of hidden values, and its gradient.
//
//   m = mean_c x_c (0 when not centered),  r = (mean_c (x_c - m)^2 + eps)^(-1/2)
//   h_c = (x_c - m) r,  y_c = h_c w_c + b_c
// and, with g_c = dy_c w_c,
//   dx_c = r (g_c - [centered] mean g - h_c mean(g h)),   dw_c = sum_t dy_tc h_tc,   db_c = sum_t dy_tc
#include "rlk_rows.cuh"

namespace rlk {
namespace {

constexpr int NORM_THREADS = SLOTS;
// Strips of rows whose parts of dw and db are summed apart: row t belongs to strip t mod 152, so that
// the order of the sum over rows depends on T alone.
constexpr int NORM_STRIPS = 152;

// A row that overflows fp32 in its sums is taken once more as x 2^-80.
constexpr float kShrink = 8.271806125530277e-25f;  // 2^-80
constexpr float kGrow = 1.2089258196146292e24f;    // 2^80

struct Vector {  // weight or bias: fp32 or the rows' type, or absent
  const void* p;
  int32_t dtype;
};

__device__ __forceinline__ float element(const Vector& w, int c) {
  if (w.dtype == RLK_DTYPE_F32) return static_cast<const float*>(w.p)[c];
  const uint16_t b = static_cast<const uint16_t*>(w.p)[c];
  return w.dtype == RLK_DTYPE_BF16 ? Bf16::to_f32(b) : F16::to_f32(b);
}

__device__ __forceinline__ void vector8(const Vector& w, int c0, int n, float absent, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = w.p && c0 + i < n ? element(w, c0 + i) : absent;
}

// Sums of two values over the 256 slots, in the fixed order; every thread gets both. `room`: 16 floats of
// shared memory that no other call is using.
__device__ __forceinline__ float2 slots_sum(float a, float b, float* room) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float2 s = warp_sum_pair(a, b, lane);
  __syncthreads();
  if (lane == 0) room[warp] = s.x, room[8 + warp] = s.y;
  __syncthreads();
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = room[i], y[i] = room[8 + i];
  return make_float2(tree8(x), tree8(y));
}

struct RowStats {
  float k;     // what x is multiplied by (1, or 2^-80 for a row whose sums are beyond fp32)
  float m, c;  // mean of k x: m + c (m rounded, c what that lost)
  float r;     // 1 / sqrt(mean (k x - mean)^2 + k^2 eps)
};

// The statistics of a row; f(j, v) gives the j-th of this thread's packs as 8 values (0 beyond the row),
// n is the row's length.
template <class F>
__device__ __forceinline__ RowStats row_stats(int n, bool centered, float eps, float* room, const F& f) {
  const int packs = (n + 7) / 8;
  const float len = static_cast<float>(n);
  RowStats s{1.f, 0.f, 0.f, 0.f};
  float q;
  for (;;) {
    if (centered) {
      float a = 0.f;
      for (int p = threadIdx.x; p < packs; p += SLOTS) {
        float v[8];
        f(p, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], s.k);
        a = __fadd_rn(a, tree8(v));
      }
      s.m = __fdiv_rn(slots_sum(a, 0.f, room).x, len);
    }
    float a = 0.f, b = 0.f;
    for (int p = threadIdx.x; p < packs; p += SLOTS) {
      float v[8], d[8];
      f(p, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = 8 * p + i < n ? __fsub_rn(__fmul_rn(v[i], s.k), s.m) : 0.f;
        v[i] = __fmul_rn(d[i], d[i]);
      }
      a = __fadd_rn(a, tree8(v));
      b = __fadd_rn(b, tree8(d));
    }
    const float2 t = slots_sum(a, b, room);
    q = __fdiv_rn(t.x, len);
    s.c = centered ? __fdiv_rn(t.y, len) : 0.f;
    if (isfinite(q) || s.k != 1.f) break;
    s.k = kShrink;
  }
  const float var = fmaxf(__fmaf_rn(-s.c, s.c, q), 0.f);
  if (!isfinite(q)) s.r = quiet_nan();  // a NaN or an infinity in the row
  else if (s.k == 1.f) s.r = __frcp_rn(__fsqrt_rn(__fadd_rn(var, eps)));
  else if (var > 1.17549435e-38f) s.r = __frcp_rn(__fsqrt_rn(var));  // eps is 2^-34 of it at most
  else s.r = __fmul_rn(__frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(__fmul_rn(var, kGrow), kGrow), eps))), kGrow);
  return s;
}

struct NormArgs {
  const void* x;
  void* y;
  int64_t T, ld, out_ld;
  int32_t H;
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

template <class E, class O, bool AL>
__global__ void __launch_bounds__(NORM_THREADS) norm_fwd_any_kernel(const NormArgs a) {
  __shared__ float room[16];
  const int64_t t = blockIdx.x;
  const auto* x = static_cast<const typename E::bits*>(a.x) + t * a.ld;
  auto* y = static_cast<typename O::bits*>(a.y) + t * a.out_ld;
  const auto get = [&](int p, float (&v)[8]) { unpack(load_columns<E, AL>(x, 8 * p, a.H, a.err), v); };
  const RowStats s = row_stats(a.H, a.centered, a.eps, room, get);
  if (threadIdx.x == 0) put_stats(a, t, s);
  for (int p = threadIdx.x; p < (a.H + 7) / 8; p += SLOTS) {
    float v[8], w[8], b[8];
    get(p, v);
    vector8(a.w, 8 * p, a.H, 1.f, w);
    vector8(a.b, 8 * p, a.H, 0.f, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = __fsub_rn(__fsub_rn(__fmul_rn(v[i], s.k), s.m), s.c);
      v[i] = __fmaf_rn(__fmul_rn(d, s.r), w[i], b[i]);
    }
    store_columns<O, AL>(y, 8 * p, a.H, v, a.err);
  }
}

struct NormGradArgs {
  const void *dy, *x;
  void* dx;
  int64_t T, dy_ld, ld, dx_ld;
  int32_t H;
  Vector w;
  const float *mean, *rstd;
  float* row;         // [T][2]: mean g, mean(g h)
  float *part_w, *part_b;  // [strips][H]
  float *dw, *db;
  int32_t strips;
  int32_t* err;
};

// h and g of 8 columns
__device__ __forceinline__ void norm_terms(const float (&x)[8], const float (&dy)[8], const float (&w)[8], float m, float r,
                                           float (&h)[8], float (&g)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = __fmul_rn(__fsub_rn(x[i], m), r);
    g[i] = __fmul_rn(dy[i], w[i]);
  }
}

template <class E, class O, bool AL>
__global__ void __launch_bounds__(NORM_THREADS) norm_bwd_rows_kernel(const NormGradArgs a) {
  __shared__ float room[16];
  const int64_t t = blockIdx.x;
  const auto* x = static_cast<const typename E::bits*>(a.x) + t * a.ld;
  const auto* dy = static_cast<const typename O::bits*>(a.dy) + t * a.dy_ld;
  const float m = a.mean ? a.mean[t] : 0.f, r = a.rstd[t];
  float s1 = 0.f, s2 = 0.f;
  for (int p = threadIdx.x; p < (a.H + 7) / 8; p += SLOTS) {
    float xv[8], dv[8], w[8], h[8], g[8];
    unpack(load_columns<E, AL>(x, 8 * p, a.H, a.err), xv);
    unpack(load_columns<O, AL>(dy, 8 * p, a.H, a.err), dv);
    vector8(a.w, 8 * p, a.H, 1.f, w);
    norm_terms(xv, dv, w, m, r, h, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = 8 * p + i < a.H ? __fmul_rn(g[i], h[i]) : 0.f;
    s1 = __fadd_rn(s1, tree8(g));
    s2 = __fadd_rn(s2, tree8(h));
  }
  const float2 s = slots_sum(s1, s2, room);
  if (threadIdx.x == 0) {
    const float len = static_cast<float>(a.H);
    a.row[2 * t] = a.mean ? __fdiv_rn(s.x, len) : 0.f;
    a.row[2 * t + 1] = __fdiv_rn(s.y, len);
  }
}

// dx, and the strip's part of dw and db, of 8 columns a thread.
template <class E, class O, bool AL>
__global__ void __launch_bounds__(NORM_THREADS) norm_bwd_columns_kernel(const NormGradArgs a) {
  const int c0 = 8 * static_cast<int>(blockIdx.x * NORM_THREADS + threadIdx.x);
  if (c0 >= a.H) return;
  float w[8], sw[8] = {}, sb[8] = {};
  vector8(a.w, c0, a.H, 1.f, w);
  for (int64_t t = blockIdx.y; t < a.T; t += a.strips) {
    float xv[8], dv[8], h[8], g[8];
    unpack(load_columns<E, AL>(static_cast<const typename E::bits*>(a.x) + t * a.ld, c0, a.H, a.err), xv);
    unpack(load_columns<O, AL>(static_cast<const typename O::bits*>(a.dy) + t * a.dy_ld, c0, a.H, a.err), dv);
    const float m = a.mean ? a.mean[t] : 0.f, r = a.rstd[t];
    norm_terms(xv, dv, w, m, r, h, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sw[i] = __fmaf_rn(dv[i], h[i], sw[i]);
      sb[i] = __fadd_rn(sb[i], dv[i]);
    }
    if (!a.dx) continue;
    const float c1 = a.row[2 * t], c2 = a.row[2 * t + 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = __fmul_rn(__fmaf_rn(-h[i], c2, __fsub_rn(g[i], c1)), r);
    store_columns<E, AL>(static_cast<typename E::bits*>(a.dx) + t * a.dx_ld, c0, a.H, g, a.err);
  }
  const int64_t at = static_cast<int64_t>(blockIdx.y) * a.H;
  if (a.part_w) store_columns<F32, false>(reinterpret_cast<uint32_t*>(a.part_w) + at, c0, a.H, sw, a.err);
  if (a.part_b) store_columns<F32, false>(reinterpret_cast<uint32_t*>(a.part_b) + at, c0, a.H, sb, a.err);
}

// dw and db from the strips' parts, added in ascending order.
__global__ void __launch_bounds__(NORM_THREADS) norm_fold_kernel(const NormGradArgs a) {
  const int c = blockIdx.x * NORM_THREADS + threadIdx.x;
  if (c >= a.H) return;
  const float* part = blockIdx.y ? a.part_b : a.part_w;
  float* out = blockIdx.y ? a.db : a.dw;
  if (!part) return;
  float s = 0.f;
#pragma unroll 8
  for (int i = 0; i < a.strips; ++i) s = __fadd_rn(s, part[static_cast<int64_t>(i) * a.H + c]);
  out[c] = s;
}

inline int32_t strips_of(int64_t T) { return static_cast<int32_t>(T < NORM_STRIPS ? T : NORM_STRIPS); }

inline bool vector_ok(const void* p, int32_t dtype, int32_t rows_dtype) {
  return !p || ((dtype == rows_dtype || dtype == RLK_DTYPE_F32) && on_boundary(p, dtype_bytes(dtype)));
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
  const NormArgs a{x, y, T, ld, out_ld, static_cast<int32_t>(H), centered != 0, static_cast<float>(eps),
                   Vector{weight, weight_dtype}, Vector{bias, weight_dtype}, mean, rstd, err_flag};
  const bool al = whole_packs(x, T, H, ld, in.eb) && whole_packs(y, T, H, out_ld, out.eb);
  return with_pair(dtype, out_dtype, [&](auto e, auto o) {
    using E = decltype(e);
    using O = decltype(o);
    const auto s = static_cast<cudaStream_t>(stream);
    if (al) norm_fwd_any_kernel<E, O, true><<<static_cast<unsigned>(T), NORM_THREADS, 0, s>>>(a);
    else norm_fwd_any_kernel<E, O, false><<<static_cast<unsigned>(T), NORM_THREADS, 0, s>>>(a);
    return launched();
  });
}

size_t rlk_layer_norm_bwd_workspace(int64_t T, int64_t H) {
  if (T <= 0 || H <= 0) return 0;
  return carved(T * 2 * sizeof(float)) + 2 * carved(strips_of(T) * H * sizeof(float));
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
  NormGradArgs a{dy, x, dx, T, dy_ld, ld, dx_ld, static_cast<int32_t>(H), Vector{weight, weight_dtype}, mean, rstd,
                 static_cast<float*>(workspace), nullptr, nullptr, dw, db, strips_of(T), err_flag};
  const size_t part = carved(a.strips * H * sizeof(float));
  char* after = static_cast<char*>(workspace) + carved(T * 2 * sizeof(float));
  if (dw) a.part_w = reinterpret_cast<float*>(after);
  if (db) a.part_b = reinterpret_cast<float*>(after + part);
  const bool al = whole_packs(x, T, H, ld, xs.eb) && whole_packs(dy, T, H, dy_ld, ds.eb) &&
                  (!dx || whole_packs(dx, T, H, dx_ld, os.eb));
  const unsigned blocks = static_cast<unsigned>((H + 8 * NORM_THREADS - 1) / (8 * NORM_THREADS));
  return with_pair(dtype, dy_dtype, [&](auto e, auto o) {
    using E = decltype(e);
    using O = decltype(o);
    const auto go = [&](auto aligned) {
      constexpr bool AL = decltype(aligned)::value;
      if (dx) norm_bwd_rows_kernel<E, O, AL><<<static_cast<unsigned>(T), NORM_THREADS, 0, s>>>(a);
      norm_bwd_columns_kernel<E, O, AL><<<dim3(blocks, a.strips), NORM_THREADS, 0, s>>>(a);
    };
    if (al) go(Is<true>{});
    else go(Is<false>{});
    if (dw || db)
      norm_fold_kernel<<<dim3(static_cast<unsigned>((H + NORM_THREADS - 1) / NORM_THREADS), 2), NORM_THREADS, 0, s>>>(a);
    return launched();
  });
}

}  // extern "C"
