// rlk_clip.cu -- the 2-norm over many tensors, and scaling them so that it is at most a bound.
//
//   norm = sqrt(sum over tensors and elements of g^2),   out = g min(1, max_norm / norm)
//
// The tensors are cut into chunks of 16 KB, which are dealt in turn to 912 shares, a CTA each. What a share adds up, and in
// what order, follows from the tensors' sizes and types alone, and so does the order of the 912 sums: the norm has the same
// bits wherever the tensors lie. The sum reads 2.5 GB of fp32 in 338 us (7.4 TB/s). Scaling reads and writes: there CTAs that
// stay and take chunk after chunk are slower (920 us) than a CTA a chunk (683 us, 7.3 TB/s), which then needs the factor ready; for few
// chunks, where the launch between would cost more, every CTA folds the shares itself.
#include <algorithm>
#include <new>

#include "rlk_rows.cuh"

namespace rlk {
namespace {

constexpr int CLIP_THREADS = 256;
constexpr int SHARES = 912;          // six CTAs on each of 152 SMs
constexpr int SCALERS = 608;         // CTAs that scale few chunks
constexpr int CHUNK_BYTES = 16384;   // 64 bytes a thread: two packs of fp32, four of 16-bit types
constexpr int MANY_CHUNKS = 8 * SCALERS;  // beyond, a CTA scales one chunk (80 MB; the launch between costs 2 us)
constexpr int BATCH = 512;           // tensors of one launch: their table is a kernel parameter (16 KB)
constexpr int FEW = 32;              // a smaller table, for the calls that are bound by the host

struct Piece {
  const void* in;
  void* out;
  int64_t n;
  uint32_t chunk0;      // chunks of the pieces before
  int16_t dtype, out_dtype;
};

// Sums of squares at three scales (Blue's sums): what would overflow or vanish in fp32 is squared as x 2^-80 or x 2^80. All in
// fp32, with what the sums' roundings lose (a thread may add many chunks, 18000 of 280 GB): this GPU adds two doubles an SM and cycle,
// and a fold of the shares in doubles by every CTA took 7 us.
struct alignas(16) Share {
  float mid = 0.f, big = 0.f, small = 0.f;
};
template <int N>
struct ClipArgs {
  Piece piece[N];
  int32_t n;
  uint32_t chunks;
  Share* sums;          // [launches][SHARES], this launch's first
  int32_t* err;
};

constexpr float kShrunk = 8.271806125530277e-25f;  // 2^-80
constexpr float kGrown = 1.2089258196146292e24f;   // 2^80

template <class E>
constexpr int CHUNK = CHUNK_BYTES / static_cast<int>(sizeof(typename E::bits));  // elements
template <class E>
constexpr int PACKS = CHUNK<E> / (8 * CLIP_THREADS);                             // of a thread

// hi + lo: a sum and what its roundings have lost (two-sum)
struct Exact {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = __fadd_rn(hi, v), b = __fsub_rn(t, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(v, b)));
    hi = t;
  }
  // An infinity has lost nothing (what add takes for its loss is NaN)
  __device__ __forceinline__ float sum() const { return isfinite(hi) ? __fadd_rn(hi, lo) : hi; }
};

// A thread's sums at the outer scales are seldom touched, and stay out of the way of the others: in shared memory, behind a call
// (216 tensors of 302 MB in bf16 take 49.6 us; written out in line 50.5, in registers, of which 16-bit types spill, 51.8; without
// what the outer scales lose 49.2).
struct Rare {
  Exact big, small;
};
__device__ __forceinline__ Rare& rare_sums() {
  __shared__ __align__(16) float room[CLIP_THREADS][4];
  uint32_t tid;  // read again by each use: kept from the first to the last it takes a register from the loop between
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
  return reinterpret_cast<Rare&>(room[tid]);
}
__device__ __noinline__ void add_rare(bool tiny, float r) { (tiny ? rare_sums().small : rare_sums().big).add(r); }

// The sum of squares of a thread's packs of a chunk, get(j) the j-th of them, at the scale that holds it.
template <class E, int UNROLL, class Get>
__device__ __forceinline__ void add_squares(Exact& mid, const Get& get) {
  const auto at = [&](float f) {
    F32x2 a = 0;
#pragma unroll(UNROLL)
    for (int j = 0; j < PACKS<E>; ++j) {
      F32x2 v[4];
      unpack(get(j), v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(f));  // a power of two
      a = dot4(v, v, a);
    }
    return low_plus_high(a);
  };
  const float q = at(1.f);
  if (q >= 8.077935669463161e-28f && q <= 1.2089258196146292e24f) {  // 2^-90 .. 2^80: 2^39 of them stay in fp32
    mid.add(q);
    return;
  }
  const bool tiny = q < 1.f;  // else too large, NaN or infinite
  const float r = at(tiny ? kGrown : kShrunk);
  if (r != 0.f) add_rare(tiny, r);
}

// The sum over the CTA's threads, in one order; every thread gets it. room: 8 floats each.
__device__ __forceinline__ float block_sum(float v, float* room) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = v;
  __syncthreads();
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = room[i];
  return __fadd_rn(__fadd_rn(__fadd_rn(x[0], x[1]), __fadd_rn(x[2], x[3])), __fadd_rn(__fadd_rn(x[4], x[5]), __fadd_rn(x[6], x[7])));
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

__device__ __forceinline__ bool on_vector_boundary(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Chunks lo, lo + SHARES, ... below hi of a tensor. A misaligned one's packs are cut from their neighbours' vectors, so that every thread owns the
// elements that it owns of an aligned one.
template <class E>
__device__ __noinline__ Exact sum_chunks(const Piece p, uint32_t lo, uint32_t hi, Exact s, int32_t* err) {
  const int tid = static_cast<int>(threadIdx.x);
  const auto* in = static_cast<const typename E::bits*>(p.in) + static_cast<int64_t>(lo) * CHUNK<E>;
  int64_t left = p.n - static_cast<int64_t>(lo) * CHUNK<E>;
  const bool aligned = on_vector_boundary(p.in);
#pragma unroll 1
  for (uint32_t c = lo; c < hi; c += SHARES) {
    if (aligned && left >= CHUNK<E>) {
      Pack<E> k[PACKS<E>];
#pragma unroll
      for (int j = 0; j < PACKS<E>; ++j) k[j] = load_columns<E, true, false>(in + 8 * tid, 8 * j * CLIP_THREADS, CHUNK<E> - 8 * tid, err);
      add_squares<E, PACKS<E>>(s, [&](int j) { return k[j]; });
    } else {
      const int n = static_cast<int>(min(static_cast<int64_t>(CHUNK<E>), left));
      add_squares<E, 1>(s, [&](int j) {
        const int at = 8 * (j * CLIP_THREADS + tid);
        return at < n ? load_columns<E, false>(in, at, n, err) : Pack<E>{};
      });
    }
    in += static_cast<int64_t>(SHARES) * CHUNK<E>;
    left -= static_cast<int64_t>(SHARES) * CHUNK<E>;
  }
  return s;
}

template <int N>
__global__ void __launch_bounds__(CLIP_THREADS, 6) sum_squares_kernel(const __grid_constant__ ClipArgs<N> a) {
  __shared__ float room[CLIP_THREADS / 32];
  Exact s;
  rare_sums() = Rare{};
  for (uint32_t c = blockIdx.x; c < a.chunks;) {
    const int i = piece_of(a, c);
    const Piece& p = a.piece[i];
    const uint32_t end = i + 1 < a.n ? a.piece[i + 1].chunk0 : a.chunks, lo = c - p.chunk0, hi = end - p.chunk0;
    if (p.dtype == RLK_DTYPE_F32) s = sum_chunks<F32>(p, lo, hi, s, a.err);
    else if (p.dtype == RLK_DTYPE_BF16) s = sum_chunks<Bf16>(p, lo, hi, s, a.err);
    else s = sum_chunks<F16>(p, lo, hi, s, a.err);
    c += (end - c + SHARES - 1) / SHARES * SHARES;
  }
  griddep_launch_dependents();
  Share all;
  const Rare rare = rare_sums();
  const bool odd = __syncthreads_or(rare.big.hi != 0.f || rare.small.hi != 0.f);  // NaN counts
  all.mid = block_sum(s.sum(), room);
  if (odd) {
    all.big = block_sum(rare.big.sum(), room);
    all.small = block_sum(rare.small.sum(), room);
  }
  if (threadIdx.x == 0) a.sums[blockIdx.x] = all;
}

// The norm from the shares' sums, by one CTA; the same bits in each, and in every thread.
__device__ __forceinline__ float norm_of(const Share* sums, int n, float* room) {
  Exact mid, big, small;
  for (int i = threadIdx.x; i < n; i += CLIP_THREADS) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(sums + i));
    mid.add(v.x);
    if (v.y != 0.f) big.add(v.y);
    if (v.z != 0.f) small.add(v.z);
  }
  const bool odd = __syncthreads_or(big.hi != 0.f || small.hi != 0.f);
  float m = block_sum(mid.sum(), room), b = 0.f, s = 0.f;
  if (odd) {
    b = block_sum(big.sum(), room);
    s = block_sum(small.sum(), room);
  }
  // each scale against the next larger one in which there is something
  const auto down = [](float v) { return __fmul_rn(__fmul_rn(v, kShrunk), kShrunk); };
  if (b != 0.f) return __fmul_rn(__fsqrt_rn(__fadd_rn(b, down(m))), kGrown);
  if (m != 0.f) return __fsqrt_rn(__fadd_rn(m, down(s)));
  return __fmul_rn(__fsqrt_rn(s), kShrunk);
}

struct ClipNorm {
  const Share* sums;
  int32_t n;
  float max_norm;
  float* norm;
  float* factor;        // null: not wanted, or (in scaling) not known yet
  int32_t* err;
};

// The norm and the factor, by a CTA that writes them or by one that wants the factor alone. A norm beyond fp32, or none, leaves
// the gradients as they are. A factor below fp32's normal values would have lost digits (1e-41 has 13): then it is taken for the gradients
// times 2^-126, and less than 0 to say so.
constexpr float kLeast = 1.1754943508222875e-38f;  // 2^-126
__device__ __forceinline__ float find_norm(const ClipNorm& q, bool write, float* room) {
  const float v = norm_of(q.sums, q.n, room);
  if (write && threadIdx.x == 0) {
    *q.norm = v;
    if (!isfinite(v) && q.err) atomicOr(q.err, RLK_FLAG_NONFINITE);
  }
  if (!(isfinite(v) && v > q.max_norm)) return 1.f;
  const float f = __fdiv_rn(q.max_norm, v);
  return f >= kLeast || q.max_norm == 0.f ? f : -__fdiv_rn(q.max_norm, __fmul_rn(v, kLeast));
}

__global__ void __launch_bounds__(CLIP_THREADS) norm_kernel(const ClipNorm q) {
  __shared__ float room[CLIP_THREADS / 32];
  griddep_wait();
  const float f = find_norm(q, true, room);
  griddep_launch_dependents();
  if (q.factor && threadIdx.x == 0) *q.factor = f;
}

// Chunks c, c - step, ... down to 0 of a tensor, times f; the last ones first, since L2 holds them from the sum. A thread owns packs that
// are aligned in the output; where the gradient lies alike (in place above all) it reads what it writes and no more.
template <class E, class O>
__device__ __noinline__ void scale_chunks(const Piece p, uint32_t c, uint32_t step, float f, int32_t* err) {
  const int tid = static_cast<int>(threadIdx.x);
  const auto* in0 = static_cast<const typename E::bits*>(p.in);
  auto* out0 = static_cast<typename O::bits*>(p.out);
  const int head0 = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(out0) & 15)) & 15) / static_cast<int>(sizeof(*out0));
  const bool plain = f == 1.f;  // not even a NaN's bits change in fp32 (16-bit types have one NaN on the way back)
  const auto put = [&](const Pack<E>& k, typename O::bits* out, int c, int n) {
    F32x2 v[4];
    unpack(k, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = plain ? v[i] : mul2(v[i], both(f));
    store_columns<O, true, false>(out, c, n, v, err);
  };
  const bool alike = on_vector_boundary(in0 + head0);
#pragma unroll 1
  for (;; c -= step) {
    const int64_t at = static_cast<int64_t>(c) * CHUNK<E>;
    const int n = static_cast<int>(min(static_cast<int64_t>(CHUNK<E>), p.n - at)), head = min(head0, n), packs = (n - head) / 8;
    const auto* in = in0 + at + head;
    auto* out = out0 + at + head;
    if (tid < 16) {  // the elements outside the packs
      const int i = tid < 8 ? tid - head : 8 * packs + tid - 8;
      if ((tid < 8 ? i < 0 : i < n - head) && dbg_ok(i >= -head && i < n - head, err)) {
        const float v = E::to_f32(in[i]);
        out[i] = O::from_f32(plain ? v : __fmul_rn(v, f));
      }
    }
    if (alike && packs >= PACKS<E> * CLIP_THREADS - 1) {  // a whole chunk: all packs, or all but one where there is a head
      const bool last = (PACKS<E> - 1) * CLIP_THREADS + tid < packs;
      Pack<E> k[PACKS<E>];
#pragma unroll
      for (int j = 0; j < PACKS<E>; ++j)
        if (j < PACKS<E> - 1 || last) k[j] = load_columns<E, true, false>(in + 8 * tid, 8 * j * CLIP_THREADS, n - head - 8 * tid, err);
#pragma unroll
      for (int j = 0; j < PACKS<E>; ++j)
        if (j < PACKS<E> - 1 || last) put(k[j], out + 8 * tid, 8 * j * CLIP_THREADS, n - head - 8 * tid);
    } else {
#pragma unroll 1
      for (int q = tid; q < packs; q += CLIP_THREADS)
        put(alike ? load_columns<E, true, false>(in, 8 * q, n - head, err) : load_columns<E, false>(in, 8 * q, n - head, err), out, 8 * q,
            n - head);
    }
    if (c < step) return;
  }
}

// The same chunks times 2^-126 and then f, element by element: a norm of more than 2^126 times max_norm is no step's to be fast.
template <class E, class O>
__device__ __noinline__ void scale_chunks_twice(const Piece p, uint32_t c, uint32_t step, float f, int32_t* err) {
  const auto* in = static_cast<const typename E::bits*>(p.in);
  auto* out = static_cast<typename O::bits*>(p.out);
  for (;; c -= step) {
    const int64_t at = static_cast<int64_t>(c) * CHUNK<E>, end = min(p.n, at + CHUNK<E>);
    for (int64_t i = at + threadIdx.x; i < end; i += CLIP_THREADS)
      if (dbg_ok(i >= 0 && i < p.n, err)) out[i] = O::from_f32(__fmul_rn(__fmul_rn(E::to_f32(in[i]), kLeast), f));
    if (c < step) return;
  }
}

template <class E, class O>
__device__ __forceinline__ void scale_piece(const Piece& p, uint32_t c, uint32_t step, float f, int32_t* err) {
  if (!(f > 0.f)) scale_chunks_twice<E, O>(p, c, step, fabsf(f), err);  // -0 is one of those factors, too
  else scale_chunks<E, O>(p, c, step, f, err);
}

template <int N>
__global__ void __launch_bounds__(CLIP_THREADS, 4) scale_kernel(const __grid_constant__ ClipArgs<N> a, const ClipNorm q) {
  __shared__ float room[CLIP_THREADS / 32];
  griddep_wait();
  const float f = q.factor ? *q.factor : find_norm(q, blockIdx.x == 0 && q.norm, room);
  if (blockIdx.x >= a.chunks) return;
  for (uint32_t c = a.chunks - 1 - blockIdx.x;;) {  // the last ones first
    const Piece& p = a.piece[piece_of(a, c)];
    const uint32_t at = c - p.chunk0;
    if (!(f == 1.f && p.in == p.out && p.dtype == p.out_dtype)) {
      if (p.dtype == RLK_DTYPE_BF16) scale_piece<Bf16, Bf16>(p, at, gridDim.x, f, a.err);
      else if (p.dtype == RLK_DTYPE_F16) scale_piece<F16, F16>(p, at, gridDim.x, f, a.err);
      else if (p.out_dtype == RLK_DTYPE_F32) scale_piece<F32, F32>(p, at, gridDim.x, f, a.err);
      else scale_piece<F32, Bf16>(p, at, gridDim.x, f, a.err);
    }
    const uint32_t back = at / gridDim.x * gridDim.x + gridDim.x;  // past the tensor's first chunk of this CTA
    if (c < back) return;
    c -= back;
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
  const int64_t each = CHUNK_BYTES / dtype_bytes(dtype);
  return (n + each - 1) / each;
}

struct Extent {
  uintptr_t from, to;
};

// Every written tensor is its own gradient, or meets no gradient and no other written one; the norm meets none of them.
inline rlk_status check_written(const Tensors& t, const float* norm) {
  Extent* e = new (std::nothrow) Extent[2 * static_cast<size_t>(t.n) + 1];
  if (!e) return RLK_ERR_CUDA;
  int32_t k = 0;
  e[k++] = Extent{reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm) + sizeof(float)};
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

inline rlk_status check_tensors(const Tensors& t, const float* norm) {
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
  if (!norm || !on_boundary(norm, 4)) return RLK_ERR_INVALID_ARG;
  return t.out ? check_written(t, norm) : RLK_OK;
}

inline int32_t launches_of(int32_t n) { return n <= FEW ? 1 : (n + BATCH - 1) / BATCH; }

// Calls f with the table of each launch.
template <int N, class F>
inline rlk_status each_batch(const Tensors& t, Share* sums, int32_t* err, F f) {
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
inline rlk_status run_clip(const Tensors& t, double max_norm, float* norm, int32_t* err, Share* sums, cudaStream_t s) {
  rlk_status st = each_batch<N>(t, sums, err, [&](const ClipArgs<N>& a, int32_t) {
    sum_squares_kernel<N><<<SHARES, CLIP_THREADS, 0, s>>>(a);
    return launched();
  });
  if (st != RLK_OK) return st;
  const int32_t n = launches_of(t.n) * SHARES;
  ClipNorm q{sums, n, static_cast<float>(max_norm), norm, nullptr, err};
  if (!t.out) return launch_after(norm_kernel, dim3(1), CLIP_THREADS, s, q);
  int64_t chunks = 0;
  for (int32_t i = 0; i < t.n; ++i) chunks += chunks_of(t.sizes[i], t.dtypes[i]);
  const bool many = chunks > MANY_CHUNKS || launches_of(t.n) > 1;
  if (many) {
    q.factor = reinterpret_cast<float*>(sums + n);
    st = launch_after(norm_kernel, dim3(1), CLIP_THREADS, s, q);
    if (st != RLK_OK) return st;
  }
  return each_batch<N>(t, sums, err, [&](const ClipArgs<N>& a, int32_t k) {
    const dim3 grid(std::max(many ? a.chunks : std::min<uint32_t>(a.chunks, SCALERS), 1u));
    if (k == 0) return launch_after(scale_kernel<N>, grid, CLIP_THREADS, s, a, q);
    scale_kernel<N><<<grid, CLIP_THREADS, 0, s>>>(a, q);
    return launched();
  });
}

inline rlk_status clip(const Tensors& t, double max_norm, float* norm, int32_t* err, void* workspace, size_t bytes,
                       void* stream) {
  const rlk_status st = check_tensors(t, norm);
  if (st != RLK_OK) return st;
  if (!workspace || !on_boundary(workspace, 256) || bytes < rlk_grad_norm_workspace(t.n)) return RLK_ERR_WORKSPACE;
  auto* sums = static_cast<Share*>(workspace);
  const auto s = static_cast<cudaStream_t>(stream);
  return t.n <= FEW ? run_clip<FEW>(t, max_norm, norm, err, sums, s) : run_clip<BATCH>(t, max_norm, norm, err, sums, s);
}

}  // namespace
}  // namespace rlk

using namespace rlk;

extern "C" {

size_t rlk_grad_norm_workspace(int32_t n) { return n < 0 ? 0 : (static_cast<size_t>(launches_of(n)) * SHARES + 1) * sizeof(Share); }

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
