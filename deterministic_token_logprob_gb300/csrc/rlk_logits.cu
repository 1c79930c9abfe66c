// rlk_logits.cu -- the operators over logits of include/rlk.h: token log probabilities with
// entropy and top alternatives, their gradient, and distillation from a teacher's top logits
// (forward, backward, both in one call).
#include <cuda_runtime.h>

#include <utility>

#include "rlk_logits.cuh"

namespace rlk {
namespace {

constexpr int ROW_THREADS = 256;
constexpr int ROW_WARPS = ROW_THREADS / 32;

// ---------------------------------------------------------------------------
// statistics of one row by one CTA: every warp takes every ROW_WARPS-th leaf
// ---------------------------------------------------------------------------
template <class E>
__device__ __forceinline__ Stats row_stats(const Row<E>& row, float c, Stats* leaves) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_leaves = (row.n + ROW_LEAF - 1) / ROW_LEAF;
  for (int l = warp; l < n_leaves; l += ROW_WARPS) {
    Pack<E> k[LEAF_GROUPS];
    load_leaf(row, l, lane, k);
    float v[32];
#pragma unroll
    for (int j = 0; j < LEAF_GROUPS; ++j) unpack(k[j], v + 8 * j);
    const Stats x = leaf_stats(v, c);
    if (lane == 0) leaves[l] = x;
  }
  __syncthreads();
  return fold_leaves(leaves, n_leaves, c, lane);  // every warp: the same bits
}

struct ScoreArgs {
  LogitRows in;
  const int64_t* y;
  int32_t top_k;
  float* logp;
  int32_t* rank;
  float* lse;
  float* entropy;
  int64_t* top_ids;
  float* top_logp;
};

// a before b in the order of the alternatives
__device__ __forceinline__ bool ahead(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }

template <class E>
__global__ void __launch_bounds__(ROW_THREADS) token_logprobs_kernel(const ScoreArgs a) {
  extern __shared__ Stats leaves[];
  __shared__ float best_v[ROW_WARPS];
  __shared__ int best_i[ROW_WARPS];
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const LogitRows& in = a.in;
  const auto* row = static_cast<const typename E::bits*>(in.base) + static_cast<int64_t>(t) * in.ld;
  const Stats r = row_stats(Row<E>(row, in.n), in.c, leaves);
  const float lse = row_lse(r, in.s);
  const bool bad = isnan(lse);
  const int64_t y = a.y ? a.y[t] : 0;
  const bool y_ok = y >= 0 && y < in.n;
  const float zy = y_ok ? E::to_f32(row[y]) : 0.f;
  int ahead_of_y = 0;
  if (a.rank && y_ok && !bad)
    for (int v = threadIdx.x; v < in.n; v += ROW_THREADS) ahead_of_y += ahead(E::to_f32(row[v]), v, zy, static_cast<int>(y));
  ahead_of_y = __reduce_add_sync(kFullWarp, ahead_of_y);
  if (lane == 0) best_i[warp] = ahead_of_y;
  __syncthreads();
  if (threadIdx.x == 0) {
    int rank = 1;
    for (int w = 0; w < ROW_WARPS; ++w) rank += best_i[w];
    if (a.lse) a.lse[t] = lse;
    if (a.entropy) a.entropy[t] = row_entropy(r, in.s);
    if (a.logp) a.logp[t] = y_ok && !bad ? token_logp(zy, in.s, lse) : quiet_nan();
    if (a.rank) a.rank[t] = y_ok && !bad ? rank : 0;
    if (in.err_flag && bad) atomicOr(in.err_flag, RLK_FLAG_NONFINITE);
    if (in.err_flag && a.y && !y_ok) atomicOr(in.err_flag, RLK_FLAG_BAD_TARGET);
  }
  // k rounds: the best column after the one chosen last
  float pv = __int_as_float(0x7f800000);
  int pi = -1;
  for (int k = 0; k < a.top_k; ++k) {
    float bv = neg_inf();
    int bi = INT32_MAX;
    if (!bad)
      for (int v = threadIdx.x; v < in.n; v += ROW_THREADS) {
        const float z = E::to_f32(row[v]);
        if (ahead(pv, pi, z, v) && ahead(z, v, bv, bi)) bv = z, bi = v;
      }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      const float ov = __shfl_xor_sync(kFullWarp, bv, d);
      const int oi = __shfl_xor_sync(kFullWarp, bi, d);
      if (ahead(ov, oi, bv, bi)) bv = ov, bi = oi;
    }
    __syncthreads();
    if (lane == 0) best_v[warp] = bv, best_i[warp] = bi;
    __syncthreads();
    bv = best_v[0], bi = best_i[0];
    for (int w = 1; w < ROW_WARPS; ++w)
      if (ahead(best_v[w], best_i[w], bv, bi)) bv = best_v[w], bi = best_i[w];
    const bool none = bv == neg_inf();
    if (threadIdx.x == 0) {
      a.top_ids[static_cast<int64_t>(t) * a.top_k + k] = none ? -1 : bi;
      a.top_logp[static_cast<int64_t>(t) * a.top_k + k] = bad ? quiet_nan() : none ? neg_inf() : token_logp(bv, in.s, lse);
    }
    pv = bv, pi = bi;
  }
}

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
struct GradOut {
  void* base;
  int64_t ld;
  int32_t V;
};

struct TokenGradArgs {
  LogitRows in;
  GradOut out;
  const int64_t* y;
  const float* lse;
  const float* entropy;
  const float* g_logp;
  const float* g_entropy;
};

template <class E, class O>
__global__ void __launch_bounds__(ROW_THREADS) token_grad_kernel(const TokenGradArgs a) {
  const int t = blockIdx.x;
  const LogitRows& in = a.in;
  const auto* row = static_cast<const typename E::bits*>(in.base) + static_cast<int64_t>(t) * in.ld;
  auto* out = static_cast<typename O::bits*>(a.out.base) + static_cast<int64_t>(t) * a.out.ld;
  const float lse = a.lse[t], g = a.g_logp[t], ge = a.g_entropy ? a.g_entropy[t] : 0.f;
  const int64_t y = a.y[t];
  const bool y_ok = y >= 0 && y < in.n;
  if (!y_ok && threadIdx.x == 0 && in.err_flag) atomicOr(in.err_flag, RLK_FLAG_BAD_TARGET);
  const bool live = y_ok && !isnan(lse) && lse != neg_inf() && !(g == 0.f && ge == 0.f);
  // dz = p (A + B d) (+ C at y), d = log p
  const float ent = a.g_entropy ? a.entropy[t] : 0.f;
  const float A = __fmul_rn(-in.s, __fmaf_rn(ge, ent, g)), B = __fmul_rn(-in.s, ge), C = __fmul_rn(in.s, g);
  for (int v = threadIdx.x; v < a.out.V; v += ROW_THREADS) {
    float dz = 0.f;
    if (live && v < in.n) {
      const float d = __fmaf_rn(E::to_f32(row[v]), in.s, -lse);
      dz = __fmaf_rn(prob_of(d), __fmaf_rn(B, fmaxf(d, -1e30f), A), v == y ? C : 0.f);
    }
    out[v] = O::from_f32(dz);
  }
}

struct DistillArgs {
  LogitRows in;
  GradOut out;
  const int64_t* ids;
  const float* teacher;
  int32_t K;
  const float* g;
  const float* lse_in;   // backward alone
  float* loss;           // forward
  float* lse;
};

// Loss of one row by one warp (every lane gets it).
template <class E>
__device__ __forceinline__ float row_loss(const Teacher& q, const typename E::bits* row, float lse, float s) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < RLK_MAX_TOP_K / 32; ++i)
    if (q.q[i] > 0.f)
      sum = __fmaf_rn(q.q[i], __fsub_rn(q.logq[i], token_logp(E::to_f32(row[q.id[i]]), s, lse)), sum);
  return warp_sum(sum);
}

template <class E, class O, bool FWD, bool BWD>
__global__ void __launch_bounds__(ROW_THREADS) distill_kernel(const DistillArgs a) {
  extern __shared__ Stats leaves[];
  __shared__ int ids[RLK_MAX_TOP_K];
  __shared__ float qs[RLK_MAX_TOP_K], zs[RLK_MAX_TOP_K];
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const LogitRows& in = a.in;
  const auto* row = static_cast<const typename E::bits*>(in.base) + static_cast<int64_t>(t) * in.ld;
  Teacher q;
  load_teacher(q, a.ids + static_cast<int64_t>(t) * a.K, a.teacher + static_cast<int64_t>(t) * a.K, a.K, in.n, in.s,
               in.c, lane);
  float lse;
  if constexpr (FWD) {
    lse = row_lse(row_stats(Row<E>(row, in.n), in.c, leaves), in.s);
    if (warp == 0) {
      const float l = row_loss<E>(q, row, lse, in.s);
      if (lane == 0) {
        a.loss[t] = isnan(lse) || q.bad_id || q.nonfinite ? quiet_nan() : l;
        if (a.lse) a.lse[t] = lse;
        if (in.err_flag && (isnan(lse) || q.nonfinite)) atomicOr(in.err_flag, RLK_FLAG_NONFINITE);
      }
    }
  } else {
    lse = a.lse_in[t];
    if (threadIdx.x == 0 && in.err_flag && q.nonfinite) atomicOr(in.err_flag, RLK_FLAG_NONFINITE);
  }
  if (threadIdx.x == 0 && in.err_flag && q.bad_id) atomicOr(in.err_flag, RLK_FLAG_BAD_TARGET);
  if constexpr (BWD) {
    auto* out = static_cast<typename O::bits*>(a.out.base) + static_cast<int64_t>(t) * a.out.ld;
    const float g = a.g[t];
    const bool live = !isnan(lse) && lse != neg_inf() && q.any && !q.bad_id && !q.nonfinite && g != 0.f;
    const float A = __fmul_rn(in.s, g);
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < RLK_MAX_TOP_K / 32; ++i) {
        const int k = lane + 32 * i;
        const bool some = live && q.q[i] > 0.f;
        ids[k] = some ? static_cast<int>(q.id[i]) : -1;
        qs[k] = some ? q.q[i] : 0.f;
        zs[k] = some ? E::to_f32(row[q.id[i]]) : 0.f;
      }
    }
    __syncthreads();
    for (int v = threadIdx.x; v < a.out.V; v += ROW_THREADS) {
      float dz = 0.f;
      if (live && v < in.n) dz = __fmul_rn(A, prob_of(__fmaf_rn(E::to_f32(row[v]), in.s, -lse)));
      out[v] = O::from_f32(dz);
    }
    __syncthreads();
    // the teacher's columns: the first entry of an id writes the sum over its entries
    for (int k = threadIdx.x; k < a.K; k += ROW_THREADS) {
      const int id = ids[k];
      bool first = id >= 0;
      float qk = 0.f;
      for (int j = 0; j < a.K; ++j) {
        if (ids[j] != id) continue;
        if (j < k) first = false;
        qk = __fadd_rn(qk, qs[j]);
      }
      if (first) out[id] = O::from_f32(__fmul_rn(A, __fsub_rn(prob_of(__fmaf_rn(zs[k], in.s, -lse)), qk)));
    }
  }
}

size_t leaves_bytes(const LogitRows& in) {
  return static_cast<size_t>((in.n + ROW_LEAF - 1) / ROW_LEAF) * sizeof(Stats);
}

rlk_status launched() { return cudaGetLastError() == cudaSuccess ? RLK_OK : RLK_ERR_CUDA; }

// dlogits: the logits' type, or bf16 for fp32 logits
rlk_status check_out(const LogitRows& in, int32_t dtype, void* dlogits, int32_t out_dtype, int64_t V, int64_t out_ld,
                     GradOut* o) {
  const int eb = dtype_bytes(out_dtype);
  if (eb == 0 || V < in.n || out_ld < V) return RLK_ERR_INVALID_ARG;
  if (out_dtype != dtype && !(dtype == RLK_DTYPE_F32 && out_dtype == RLK_DTYPE_BF16)) return RLK_ERR_UNSUPPORTED;
  if (V > RLK_MAX_LOGITS_VOCAB) return RLK_ERR_UNSUPPORTED;
  if (in.T > 0 && (!dlogits || reinterpret_cast<uintptr_t>(dlogits) % eb != 0)) return RLK_ERR_INVALID_ARG;
  // in place: the very same array; otherwise the two address ranges are apart
  if (in.T > 0 && !(dlogits == in.base && out_dtype == dtype && (out_ld == in.ld || in.T == 1))) {
    const auto span = [&](const void* p, int64_t ld, int64_t n, int bytes) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(p);
      return std::pair<uintptr_t, uintptr_t>(a, a + static_cast<uintptr_t>(((in.T - 1) * ld + n) * bytes));
    };
    const auto z = span(in.base, in.ld, in.n, dtype_bytes(dtype)), d = span(dlogits, out_ld, V, eb);
    if (z.first < d.second && d.first < z.second) return RLK_ERR_INVALID_ARG;
  }
  *o = GradOut{dlogits, out_ld, static_cast<int32_t>(V)};
  return RLK_OK;
}

// Calls f with the element types of (dtype, out_dtype).
template <class F>
void with_types(int32_t dtype, int32_t out_dtype, F f) {
  if (dtype == RLK_DTYPE_BF16) f(Bf16{}, Bf16{});
  else if (dtype == RLK_DTYPE_F16) f(F16{}, F16{});
  else if (out_dtype == RLK_DTYPE_BF16) f(F32{}, Bf16{});
  else f(F32{}, F32{});
}

}  // namespace
}  // namespace rlk

using namespace rlk;

extern "C" {

rlk_status rlk_token_logprobs(const void* logits, int32_t dtype, int64_t T, int64_t ld, int64_t V_true,
                              double temperature, const int64_t* y, int32_t top_k, float* logp, int32_t* rank,
                              float* lse, float* entropy, int64_t* top_ids, float* top_logp, int32_t* err_flag,
                              void* stream) {
  ScoreArgs a{};
  const rlk_status st = check_logits(logits, dtype, T, ld, V_true, temperature, err_flag, &a.in);
  if (st != RLK_OK) return st;
  if (top_k < 0 || (T > 0 && !y && (logp || rank))) return RLK_ERR_INVALID_ARG;
  if (top_k > RLK_MAX_TOP_K) return RLK_ERR_UNSUPPORTED;
  if (T > 0 && top_k > 0 && (!top_ids || !top_logp)) return RLK_ERR_INVALID_ARG;
  if (T == 0) return RLK_OK;
  a.y = y;
  a.top_k = top_k;
  a.logp = logp;
  a.rank = rank;
  a.lse = lse;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  with_types(dtype, dtype, [&](auto e, auto) {
    token_logprobs_kernel<decltype(e)><<<static_cast<unsigned>(T), ROW_THREADS, leaves_bytes(a.in),
                                         static_cast<cudaStream_t>(stream)>>>(a);
  });
  return launched();
}

rlk_status rlk_token_logprobs_bwd(const void* logits, int32_t dtype, int64_t T, int64_t ld, int64_t V_true,
                                  double temperature, const int64_t* y, const float* lse, const float* entropy,
                                  const float* g_logp, const float* g_entropy, void* dlogits, int32_t out_dtype,
                                  int64_t V, int64_t out_ld, int32_t* err_flag, void* stream) {
  TokenGradArgs a{};
  rlk_status st = check_logits(logits, dtype, T, ld, V_true, temperature, err_flag, &a.in);
  if (st == RLK_OK) st = check_out(a.in, dtype, dlogits, out_dtype, V, out_ld, &a.out);
  if (st != RLK_OK) return st;
  if (T > 0 && (!y || !lse || !g_logp || (g_entropy && !entropy))) return RLK_ERR_INVALID_ARG;
  if (T == 0) return RLK_OK;
  a.y = y;
  a.lse = lse;
  a.entropy = entropy;
  a.g_logp = g_logp;
  a.g_entropy = g_entropy;
  with_types(dtype, out_dtype, [&](auto e, auto o) {
    token_grad_kernel<decltype(e), decltype(o)>
        <<<static_cast<unsigned>(T), ROW_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(a);
  });
  return launched();
}

}  // extern "C"

namespace rlk {
namespace {

rlk_status check_distill(const void* logits, int32_t dtype, int64_t T, int64_t ld, int64_t V_true, double temperature,
                         const int64_t* ids, const float* teacher, int32_t K, int32_t* err_flag, DistillArgs* a) {
  const rlk_status st = check_logits(logits, dtype, T, ld, V_true, temperature, err_flag, &a->in);
  if (st != RLK_OK) return st;
  if (K < 1 || (T > 0 && (!ids || !teacher))) return RLK_ERR_INVALID_ARG;
  if (K > RLK_MAX_TOP_K) return RLK_ERR_UNSUPPORTED;
  a->ids = ids;
  a->teacher = teacher;
  a->K = K;
  return RLK_OK;
}

template <bool FWD, bool BWD>
rlk_status launch_distill(const DistillArgs& a, int32_t dtype, int32_t out_dtype, void* stream) {
  with_types(dtype, out_dtype, [&](auto e, auto o) {
    distill_kernel<decltype(e), decltype(o), FWD, BWD>
        <<<static_cast<unsigned>(a.in.T), ROW_THREADS, leaves_bytes(a.in), static_cast<cudaStream_t>(stream)>>>(a);
  });
  return launched();
}

}  // namespace
}  // namespace rlk

extern "C" {

rlk_status rlk_distill_topk_fwd(const void* logits, int32_t dtype, int64_t T, int64_t ld, int64_t V_true,
                                double temperature, const int64_t* ids, const float* teacher, int32_t K, float* loss,
                                float* lse, int32_t* err_flag, void* stream) {
  DistillArgs a{};
  const rlk_status st = check_distill(logits, dtype, T, ld, V_true, temperature, ids, teacher, K, err_flag, &a);
  if (st != RLK_OK) return st;
  if (T > 0 && !loss) return RLK_ERR_INVALID_ARG;
  if (T == 0) return RLK_OK;
  a.loss = loss;
  a.lse = lse;
  return launch_distill<true, false>(a, dtype, dtype, stream);
}

rlk_status rlk_distill_topk_bwd(const void* logits, int32_t dtype, int64_t T, int64_t ld, int64_t V_true,
                                double temperature, const int64_t* ids, const float* teacher, int32_t K,
                                const float* lse, const float* g, void* dlogits, int32_t out_dtype, int64_t V,
                                int64_t out_ld, int32_t* err_flag, void* stream) {
  DistillArgs a{};
  rlk_status st = check_distill(logits, dtype, T, ld, V_true, temperature, ids, teacher, K, err_flag, &a);
  if (st == RLK_OK) st = check_out(a.in, dtype, dlogits, out_dtype, V, out_ld, &a.out);
  if (st != RLK_OK) return st;
  if (T > 0 && (!lse || !g)) return RLK_ERR_INVALID_ARG;
  if (T == 0) return RLK_OK;
  a.lse_in = lse;
  a.g = g;
  return launch_distill<false, true>(a, dtype, out_dtype, stream);
}

rlk_status rlk_distill_topk_fwd_bwd(const void* logits, int32_t dtype, int64_t T, int64_t ld, int64_t V_true,
                                    double temperature, const int64_t* ids, const float* teacher, int32_t K,
                                    const float* g, float* loss, float* lse, void* dlogits, int32_t out_dtype,
                                    int64_t V, int64_t out_ld, int32_t* err_flag, void* stream) {
  DistillArgs a{};
  rlk_status st = check_distill(logits, dtype, T, ld, V_true, temperature, ids, teacher, K, err_flag, &a);
  if (st == RLK_OK) st = check_out(a.in, dtype, dlogits, out_dtype, V, out_ld, &a.out);
  if (st != RLK_OK) return st;
  if (T > 0 && (!g || !loss)) return RLK_ERR_INVALID_ARG;
  if (T == 0) return RLK_OK;
  a.g = g;
  a.loss = loss;
  a.lse = lse;
  return launch_distill<true, true>(a, dtype, out_dtype, stream);
}

}  // extern "C"
