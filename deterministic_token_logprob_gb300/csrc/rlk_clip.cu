// rlk_clip.cu -- the 2-norm over many tensors, and scaling them so that it is at most a bound.
//
//   norm = sqrt(sum over tensors and elements of g^2),   out = g min(1, max_norm / norm)
//
// The tensors are cut into chunks of 16 KB; the chunks, in order, are dealt to 608 shares of equal
// length, and a CTA takes a share. What a share adds up, and in what order, follows from the tensors' sizes
// and types alone, and so does the order of the 608 sums: the norm has the same bits wherever the tensors lie.
#include <algorithm>
#include <new>

#include "rlk_rows.cuh"

namespace rlk {
namespace {

constexpr int CLIP_THREADS = 256;
constexpr int SHARES = 608;          // four CTAs on each of 152 SMs
constexpr int CHUNK_BYTES = 16384;   // 64 bytes a thread: two packs of fp32, four of 16-bit types
constexpr int BATCH = 512;           // tensors of one launch: their table is a kernel parameter (16 KB)
constexpr int FEW = 32;              // a smaller table, for the calls that are bound by the host

struct Piece {
  const void* in;
  void* out;
  int64_t n;
  uint32_t chunk0;      // chunks of the pieces before
  int16_t dtype, out_dtype;
};

template <int N>
struct ClipArgs {
  Piece piece[N];
  int32_t n;
  uint32_t chunks;
  double* sums;         // [launches][SHARES], this launch's first
  int32_t* err;
};

__host__ __device__ constexpr int chunk_elements(int eb) { return CHUNK_BYTES / eb; }

// Sums of squares at three scales (Blue's sums): what would overflow or vanish in fp32 is squared as x 2^-80 or x 2^80.
struct Squares {
  float mid = 0.f, big = 0.f, small = 0.f;
};
constexpr float kTiny = 8.271806125530277e-25f;  // 2^-80
constexpr float kHuge = 1.2089258196146292e24f;  // 2^80

template <class E>
__device__ __forceinline__ float squares(const Pack<E>& k, float f) {
  F32x2 v[4];
  unpack(k, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(f));  // a power of two
  return low_plus_high(dot4(v, v, 0));
}

template <class E>
__device__ __forceinline__ void add_squares(const Pack<E>& k, Squares& s) {
  const float q = squares(k, 1.f);
  if (q >= 8.077935669463161e-28f && q <= 1.2676506002282294e30f) s.mid = __fadd_rn(s.mid, q);  // 2^-90 .. 2^100
  else if (q < 1.f) s.small = __fadd_rn(s.small, squares(k, kHuge));
  else s.big = __fadd_rn(s.big, squares(k, kTiny));  // NaN and infinities too
}

// The sum over the CTA's threads, in one order; valid in every thread.
__device__ __forceinline__ double block_sum(double v, double* room) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v = __dadd_rn(v, __shfl_xor_sync(kFullWarp, v, d));
  if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = v;
  __syncthreads();
  v = room[0];
#pragma unroll
  for (int w = 1; w < CLIP_THREADS / 32; ++w) v = __dadd_rn(v, room[w]);
  return v;
}

template <int N>
__device__ __forceinline__ int piece_of(const ClipArgs<N>& a, uint32_t chunk) {
  int lo = 0, hi = a.n - 1;  // the last piece that starts at or before the chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.piece[mid].chunk0 <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ uint32_t share_start(uint32_t chunks, int share) {
  return static_cast<uint32_t>(static_cast<uint64_t>(chunks) * share / SHARES);
}

template <class E>
__device__ __forceinline__ void add_chunk(const Piece& p, uint32_t chunk, Squares& s, int32_t* err) {
  constexpr int CE = chunk_elements(sizeof(typename E::bits));
  const int64_t at = static_cast<int64_t>(chunk) * CE;
  const int n = static_cast<int>(min(static_cast<int64_t>(CE), p.n - at));
  const auto* row = static_cast<const typename E::bits*>(p.in) + at;
#pragma unroll
  for (int j = 0; j < CE / (8 * CLIP_THREADS); ++j) {
    const int c = 8 * (j * CLIP_THREADS + static_cast<int>(threadIdx.x));
    if (c < n) add_squares<E>(load_columns<E, false>(row, c, n, err), s);
  }
}

template <int N>
__global__ void __launch_bounds__(CLIP_THREADS) sum_squares_kernel(const __grid_constant__ ClipArgs<N> a) {
  __shared__ double room[CLIP_THREADS / 32];
  uint32_t c = share_start(a.chunks, blockIdx.x);
  const uint32_t end = share_start(a.chunks, blockIdx.x + 1);
  Squares s;
  if (c < end) {
    for (int i = piece_of(a, c); c < end; ++i) {
      const Piece& p = a.piece[i];
      const uint32_t stop = i + 1 < a.n ? min(end, a.piece[i + 1].chunk0) : end;
      for (; c < stop; ++c) {
        if (p.dtype == RLK_DTYPE_F32) add_chunk<F32>(p, c - p.chunk0, s, a.err);
        else if (p.dtype == RLK_DTYPE_BF16) add_chunk<Bf16>(p, c - p.chunk0, s, a.err);
        else add_chunk<F16>(p, c - p.chunk0, s, a.err);
      }
    }
  }
  // 2^160 and 2^-160 undo the scales
  double d = __dadd_rn(static_cast<double>(s.mid), __dmul_rn(static_cast<double>(s.small), 6.842277657836021e-49));
  d = __dadd_rn(d, __dmul_rn(static_cast<double>(s.big), 1.461501637330903e48));
  d = block_sum(d, room);
  if (threadIdx.x == 0) a.sums[blockIdx.x] = d;
}

// The norm from the shares' sums, by one CTA; the same bits in each.
__device__ __forceinline__ double norm_of(const double* sums, int n, double* room) {
  double d = 0.;
  for (int i = threadIdx.x; i < n; i += CLIP_THREADS) d = __dadd_rn(d, sums[i]);
  return __dsqrt_rn(block_sum(d, room));
}

__global__ void __launch_bounds__(CLIP_THREADS) norm_kernel(const double* sums, int n, float* norm, int32_t* err) {
  __shared__ double room[CLIP_THREADS / 32];
  const float v = static_cast<float>(norm_of(sums, n, room));
  if (threadIdx.x != 0) return;
  *norm = v;
  if (!isfinite(v) && err) atomicOr(err, RLK_FLAG_NONFINITE);
}

template <class E, class O>
__device__ __forceinline__ void scale_chunk(const Piece& p, uint32_t chunk, float f, int32_t* err) {
  constexpr int CE = chunk_elements(sizeof(typename E::bits));
  const int64_t at = static_cast<int64_t>(chunk) * CE;
  const int n = static_cast<int>(min(static_cast<int64_t>(CE), p.n - at));
  const auto* row = static_cast<const typename E::bits*>(p.in) + at;
  auto* out = static_cast<typename O::bits*>(p.out) + at;
  const bool al = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
  for (int j = 0; j < CE / (8 * CLIP_THREADS); ++j) {
    const int c = 8 * (j * CLIP_THREADS + static_cast<int>(threadIdx.x));
    if (c >= n) break;
    F32x2 v[4];
    unpack(load_columns<E, false>(row, c, n, err), v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f == 1.f ? v[i] : mul2(v[i], both(f));  // a NaN's bits survive a copy
    if (al && c + 8 <= n) store_columns<O, true>(out, c, n, v, err);
    else store_columns<O, false>(out, c, n, v, err);
  }
}

struct ClipNorm {
  const double* sums;
  int32_t n;
  double max_norm;
  float* norm;
};

// A norm beyond fp32, or none, leaves the gradients as they are.
template <int N>
__global__ void __launch_bounds__(CLIP_THREADS) scale_kernel(const __grid_constant__ ClipArgs<N> a, const ClipNorm q) {
  __shared__ double room[CLIP_THREADS / 32];
  const double norm = norm_of(q.sums, q.n, room);
  const float v = static_cast<float>(norm);
  if (blockIdx.x == 0 && threadIdx.x == 0 && q.norm) {
    *q.norm = v;
    if (!isfinite(v) && a.err) atomicOr(a.err, RLK_FLAG_NONFINITE);
  }
  const float f = isfinite(v) && norm > q.max_norm ? static_cast<float>(__ddiv_rn(q.max_norm, norm)) : 1.f;
  uint32_t c = share_start(a.chunks, blockIdx.x);
  const uint32_t end = share_start(a.chunks, blockIdx.x + 1);
  if (c >= end) return;
  for (int i = piece_of(a, c); c < end; ++i) {
    const Piece& p = a.piece[i];
    const uint32_t stop = i + 1 < a.n ? min(end, a.piece[i + 1].chunk0) : end;
    if (f == 1.f && p.in == p.out && p.dtype == p.out_dtype) {
      c = max(c, stop);
      continue;
    }
    for (; c < stop; ++c) {
      if (p.dtype == RLK_DTYPE_BF16) scale_chunk<Bf16, Bf16>(p, c - p.chunk0, f, a.err);
      else if (p.dtype == RLK_DTYPE_F16) scale_chunk<F16, F16>(p, c - p.chunk0, f, a.err);
      else if (p.out_dtype == RLK_DTYPE_F32) scale_chunk<F32, F32>(p, c - p.chunk0, f, a.err);
      else scale_chunk<F32, Bf16>(p, c - p.chunk0, f, a.err);
    }
  }
}

struct Tensors {
  const void* const* in;
  const int64_t* sizes;
  const int32_t* dtypes;
  void* const* out;          // null: none are written
  const int32_t* out_dtypes;
  int32_t n;
};

inline int64_t chunks_of(int64_t n, int32_t dtype) {
  const int64_t each = chunk_elements(dtype_bytes(dtype));
  return (n + each - 1) / each;
}

struct Extent {
  uintptr_t from, to;
};

// Every written tensor is its own gradient, or meets no gradient and no other written one.
inline rlk_status check_written(const Tensors& t) {
  Extent* e = new (std::nothrow) Extent[2 * static_cast<size_t>(t.n)];
  if (!e) return RLK_ERR_CUDA;
  int32_t k = 0;
  for (int32_t i = 0; i < t.n; ++i) {
    if (t.sizes[i] == 0) continue;
    const uintptr_t in = reinterpret_cast<uintptr_t>(t.in[i]), out = reinterpret_cast<uintptr_t>(t.out[i]);
    e[k++] = Extent{in, in + t.sizes[i] * dtype_bytes(t.dtypes[i])};
    if (out != in || t.dtypes[i] != t.out_dtypes[i]) e[k++] = Extent{out, out + t.sizes[i] * dtype_bytes(t.out_dtypes[i])};
  }
  const auto before = [](const Extent& a, const Extent& b) { return a.from < b.from; };
  if (!std::is_sorted(e, e + k, before)) std::sort(e, e + k, before);
  bool apart = true;
  for (int32_t i = 1; i < k; ++i) apart &= e[i - 1].to <= e[i].from;
  delete[] e;
  return apart ? RLK_OK : RLK_ERR_INVALID_ARG;
}

inline rlk_status check_tensors(const Tensors& t) {
  if (t.n < 0 || (t.n > 0 && (!t.in || !t.sizes || !t.dtypes))) return RLK_ERR_INVALID_ARG;
  if (t.n > RLK_MAX_TENSORS) return RLK_ERR_UNSUPPORTED;
  int64_t chunks = 0;
  for (int32_t i = 0; i < t.n; ++i) {
    const int eb = dtype_bytes(t.dtypes[i]);
    if (eb == 0 || t.sizes[i] < 0) return RLK_ERR_INVALID_ARG;
    if (t.sizes[i] > RLK_MAX_TENSOR_ELEMENTS) return RLK_ERR_UNSUPPORTED;
    if (t.sizes[i] > 0 && (!t.in[i] || !on_boundary(t.in[i], eb))) return RLK_ERR_INVALID_ARG;
    chunks += chunks_of(t.sizes[i], t.dtypes[i]);
    if (!t.out) continue;
    const rlk_status st = check_pair(t.dtypes[i], t.out_dtypes[i]);
    if (st != RLK_OK) return st;
    if (t.sizes[i] > 0 && (!t.out[i] || !on_boundary(t.out[i], dtype_bytes(t.out_dtypes[i])))) return RLK_ERR_INVALID_ARG;
  }
  if (chunks > INT32_MAX) return RLK_ERR_UNSUPPORTED;
  return t.out ? check_written(t) : RLK_OK;
}

inline int32_t launches_of(int32_t n) { return n <= FEW ? 1 : (n + BATCH - 1) / BATCH; }

// Calls f with the table of each launch.
template <int N, class F>
inline rlk_status each_batch(const Tensors& t, double* sums, int32_t* err, F f) {
  for (int32_t first = 0, k = 0; first == 0 || first < t.n; first += N, ++k) {
    ClipArgs<N> a;
    a.n = std::min(N, t.n - first);
    a.chunks = 0;
    a.sums = sums + static_cast<int64_t>(k) * SHARES;
    a.err = err;
    for (int32_t j = 0; j < a.n; ++j) {
      const int32_t i = first + j;
      a.piece[j] = Piece{t.in[i], t.out ? t.out[i] : nullptr, t.sizes[i], a.chunks, static_cast<int16_t>(t.dtypes[i]),
                         static_cast<int16_t>(t.out ? t.out_dtypes[i] : t.dtypes[i])};
      a.chunks += static_cast<uint32_t>(chunks_of(t.sizes[i], t.dtypes[i]));
    }
    const rlk_status st = f(a, k);
    if (st != RLK_OK) return st;
  }
  return RLK_OK;
}

template <int N>
inline rlk_status run_clip(const Tensors& t, double max_norm, float* norm, int32_t* err, double* sums, cudaStream_t s) {
  rlk_status st = each_batch<N>(t, sums, err, [&](const ClipArgs<N>& a, int32_t) {
    sum_squares_kernel<N><<<SHARES, CLIP_THREADS, 0, s>>>(a);
    return launched();
  });
  if (st != RLK_OK) return st;
  const int32_t n = launches_of(t.n) * SHARES;
  if (!t.out) {
    norm_kernel<<<1, CLIP_THREADS, 0, s>>>(sums, n, norm, err);
    return launched();
  }
  return each_batch<N>(t, sums, err, [&](const ClipArgs<N>& a, int32_t k) {
    scale_kernel<N><<<SHARES, CLIP_THREADS, 0, s>>>(a, ClipNorm{sums, n, max_norm, k == 0 ? norm : nullptr});
    return launched();
  });
}

inline rlk_status clip(const Tensors& t, double max_norm, float* norm, int32_t* err, void* workspace, size_t bytes,
                       void* stream) {
  const rlk_status st = check_tensors(t);
  if (st != RLK_OK) return st;
  if (!norm || !on_boundary(norm, 4)) return RLK_ERR_INVALID_ARG;
  if (!workspace || !on_boundary(workspace, 256) || bytes < rlk_grad_norm_workspace(t.n)) return RLK_ERR_WORKSPACE;
  double* sums = static_cast<double*>(workspace);
  const auto s = static_cast<cudaStream_t>(stream);
  return t.n <= FEW ? run_clip<FEW>(t, max_norm, norm, err, sums, s) : run_clip<BATCH>(t, max_norm, norm, err, sums, s);
}

}  // namespace
}  // namespace rlk

using namespace rlk;

extern "C" {

size_t rlk_grad_norm_workspace(int32_t n) { return n < 0 ? 0 : static_cast<size_t>(launches_of(n)) * SHARES * sizeof(double); }

rlk_status rlk_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n, float* norm,
                         int32_t* err_flag, void* workspace, size_t workspace_bytes, void* stream) {
  return clip(Tensors{grads, sizes, dtypes, nullptr, nullptr, n}, 0., norm, err_flag, workspace, workspace_bytes, stream);
}

rlk_status rlk_clip_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                              double max_norm, void* const* outs, const int32_t* out_dtypes, float* norm,
                              int32_t* err_flag, void* workspace, size_t workspace_bytes, void* stream) {
  if (!(max_norm > 0.)) return RLK_ERR_INVALID_ARG;
  if (n > 0 && (!outs || !out_dtypes)) return RLK_ERR_INVALID_ARG;
  static void* const none[1] = {nullptr};
  return clip(Tensors{grads, sizes, dtypes, n > 0 ? outs : none, out_dtypes, n}, max_norm, norm, err_flag, workspace,
              workspace_bytes, stream);
}

}  // extern "C"
