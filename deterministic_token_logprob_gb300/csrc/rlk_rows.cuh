// rlk_rows.cuh -- what the operators around the head (embedding, layer norm) share: rows of hidden
// values cut into packs of 8 columns, their loads and stores at any alignment, sums over a row in one
// fixed order, and the host-side argument checks.
//
// Order of a row's sums over n columns: pack p (columns 8 p .. 8 p + 7) belongs to slot p mod S, S = 32 W with W warps a row
// (a power of two that follows from n and the kind of sum); a slot adds the even and the odd columns of its packs apart, in
// ascending order of packs (a pack's four pairs as a balanced tree; sums of products one by one, each product
// unrounded), and then the two; 32 slots combine by an xor-butterfly, the groups of 32 by a balanced tree. The
// order depends on column indices alone: not on the row's address, on alignment or on how many rows a CTA takes.
#pragma once

#include <atomic>

#include "rlk_logits.cuh"

namespace rlk {
namespace {

constexpr int ROW_CTA = 256;  // threads of a CTA: 8 / W teams, a row each

template <bool V>
struct Is {
  static constexpr bool value = V;
};

// A pack at a row's end or before its first boundary, element by element; 0 beyond the row.
template <class E>
__device__ __noinline__ Pack<E> load_edge(const typename E::bits* row, int c0, int n) {
  Pack<E> k{};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = c0 + i < n ? row[c0 + i] : 0u;
    if constexpr (Pack<E>::EB == 4) k.w[i] = b;
    else k.w[i / 2] |= b << (i & 1 ? 16 : 0);
  }
  return k;
}

// 8 columns of a row of n, from column c0 (a multiple of 8) on; 0 beyond the row. AL: every pack lies on a boundary of its
// own size (whole_packs). An fp32 pack is then one 32-byte load: two of 16 bytes each, 32 apart from lane to lane, take L1
// twice as long (8192 rows of 4096, fp32 to bf16 forward: L1 73 % busy). Without WIDE 16-byte boundaries do, and loads.
template <class E, bool AL, bool WIDE = true>
__device__ __forceinline__ Pack<E> load_columns(const typename E::bits* row, int c0, int n, int32_t* err) {
  if constexpr (AL && WIDE && sizeof(typename E::bits) == 4) {
    Pack<E> k{};
    if (dbg_ok(c0 >= 0 && c0 + 8 <= n && (reinterpret_cast<uintptr_t>(row + c0) & 31) == 0, err))
      asm("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
          : "=r"(k.w[0]), "=r"(k.w[1]), "=r"(k.w[2]), "=r"(k.w[3]), "=r"(k.w[4]), "=r"(k.w[5]), "=r"(k.w[6]), "=r"(k.w[7])
          : "l"(row + c0)
          : "memory");
    return k;
  }
  const Row<E, AL> r(row, n, err);
  if (AL || packs_inside(r, c0, c0 + 8)) return load_pack(r, c0);
  return load_edge<E>(row, c0, n);
}

// The four pairs of a pack in fp32.
template <class E>
__device__ __forceinline__ void unpack(const Pack<E>& k, F32x2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = pair(k, i);
    v[i] = pack_f32x2(x.x, x.y);
  }
}

// The assembler turns a packed product whose one use is a packed sum into a fused operation, whatever their rounding
// modifiers say (seen on inputs that tell the two apart), and so differently from kernel to kernel. Products that
// are added are therefore written as fused operations throughout; mul2 serves where no add2 follows, or where the product is exact.
__device__ __forceinline__ F32x2 both(float v) { return pack_f32x2(v, v); }

// 0 in the columns at and beyond n of a pack that starts at c0.
__device__ __forceinline__ void clear_beyond(F32x2 (&v)[4], int c0, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack_f32x2(v[i]);
    v[i] = pack_f32x2(c0 + 2 * i < n ? x.x : 0.f, c0 + 2 * i + 1 < n ? x.y : 0.f);
  }
}

template <class O, bool AL, bool WIDE = true>
__device__ __forceinline__ void store_columns(typename O::bits* row, int c0, int n, const F32x2 (&x)[4], int32_t* err) {
  if (!dbg_ok(c0 >= 0 && c0 < n && (!AL || c0 + 8 <= n), err)) return;
  float2 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = unpack_f32x2(x[i]);
  if constexpr (AL) {
    if constexpr (sizeof(typename O::bits) == 4 && !WIDE) {
      float4* q = reinterpret_cast<float4*>(row + c0);
      q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    } else if constexpr (sizeof(typename O::bits) == 4) {
      if (!dbg_ok((reinterpret_cast<uintptr_t>(row + c0) & 31) == 0, err)) return;
      asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y),
                   "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y), "l"(row + c0)
                   : "memory");
    } else {
      *reinterpret_cast<uint4*>(row + c0) = make_uint4(O::pack2(v[0].x, v[0].y), O::pack2(v[1].x, v[1].y), O::pack2(v[2].x, v[2].y), O::pack2(v[3].x, v[3].y));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < n) row[c0 + i] = O::from_f32(i & 1 ? v[i / 2].y : v[i / 2].x);
  }
}

__device__ __forceinline__ F32x2 tree4(const F32x2 (&v)[4]) { return add2(add2(v[0], v[1]), add2(v[2], v[3])); }
// a + sum of x y over a pack's pairs, in ascending order
__device__ __forceinline__ F32x2 dot4(const F32x2 (&x)[4], const F32x2 (&y)[4], F32x2 a) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a = fma2(x[i], y[i], a);
  return a;
}
__device__ __forceinline__ float low_plus_high(F32x2 v) {
  const float2 x = unpack_f32x2(v);
  return __fadd_rn(x.x, x.y);
}

// Sums of two values over the slots of a row that W warps (a team, one of 8 / W of a CTA of 256) hold, in the fixed
// order; every thread of the team gets both. `room`: 2 W floats of shared memory of the team's own (16-byte aligned), which the call
// after this one does not use (one barrier a call then does).
template <int W>
__device__ __forceinline__ void team_barrier();
template <int W>
__device__ __forceinline__ float2 team_sum(float a, float b, float* room) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W;
  const bool low = lane < 16;
  float v = __fadd_rn(low ? a : b, __shfl_xor_sync(kFullWarp, low ? b : a, 16));
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFullWarp, v, d));
  if constexpr (W == 1) return make_float2(__shfl_sync(kFullWarp, v, 0), __shfl_sync(kFullWarp, v, 16));
  if ((lane & 15) == 0) room[(low ? 0 : W) + warp] = v;
  team_barrier<W>();
  float x[2 * W];
  if constexpr (W >= 4) {
#pragma unroll
    for (int i = 0; i < 2 * W; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(room + i);
      x[i] = q.x, x[i + 1] = q.y, x[i + 2] = q.z, x[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) x[i] = room[i];
  }
#pragma unroll
  for (int d = 1; d < W; d *= 2)
#pragma unroll
    for (int i = 0; i < 2 * W; i += 2 * d) x[i] = __fadd_rn(x[i], x[i + d]);
  return make_float2(x[0], x[W]);
}

// Another barrier of a team of W warps.
template <int W>
__device__ __forceinline__ void team_barrier() {
  if constexpr (W == 8) __syncthreads();
  else if constexpr (W > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x / (32 * W))), "n"(32 * W) : "memory");
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline bool on_boundary(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// T rows of n elements of eb bytes, `ld` elements apart: whether every row is a whole number of packs of 8, each on a boundary
// of its own size (16 bytes, 32 for fp32).
inline bool whole_packs(const void* p, int64_t T, int64_t n, int64_t ld, int eb) {
  return on_boundary(p, 8 * eb) && n % 8 == 0 && (T <= 1 || ld % 8 == 0);
}

struct RowSpan {  // T rows of n elements of eb bytes, ld elements apart
  const void* p;
  int64_t T, n, ld;
  int eb;
};

// Whether no row of one meets a row of the other: the arrays are apart, or their rows are the same
// number of bytes apart and lie side by side.
inline bool rows_apart(const RowSpan& a, const RowSpan& b) {
  if (a.T == 0 || b.T == 0) return true;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t da = a.ld * a.eb, db = b.ld * b.eb, na = a.n * a.eb, nb = b.n * b.eb;
  if (pa + (a.T - 1) * da + na <= pb || pb + (b.T - 1) * db + nb <= pa) return true;
  if (da != db || a.T == 1 || b.T == 1) return false;
  const uintptr_t at = (pb % da + da - pa % da) % da;  // where b's rows start, from a's on
  return at >= na && at + nb <= da;
}

inline bool same_rows(const RowSpan& a, const RowSpan& b) {
  return a.p == b.p && a.eb == b.eb && (a.ld == b.ld || (a.T <= 1 && b.T <= 1));
}

// Rows of hidden values: RLK_OK or the refusal.
inline rlk_status check_rows(const void* p, int32_t dtype, int64_t T, int64_t H, int64_t ld) {
  const int eb = dtype_bytes(dtype);
  if (eb == 0 || T < 0 || H <= 0 || ld < H) return RLK_ERR_INVALID_ARG;
  if (H > RLK_MAX_HIDDEN || T > RLK_MAX_TOKENS) return RLK_ERR_UNSUPPORTED;
  if (T > 0 && (!p || !on_boundary(p, eb))) return RLK_ERR_INVALID_ARG;
  return RLK_OK;
}

// A result's type: that of the values it comes from, or bf16 for fp32 ones.
inline rlk_status check_pair(int32_t dtype, int32_t out_dtype) {
  if (dtype_bytes(dtype) == 0 || dtype_bytes(out_dtype) == 0) return RLK_ERR_INVALID_ARG;
  if (dtype != out_dtype && !(dtype == RLK_DTYPE_F32 && out_dtype == RLK_DTYPE_BF16)) return RLK_ERR_UNSUPPORTED;
  return RLK_OK;
}

template <class F>
inline rlk_status with_type(int32_t dtype, F f) {
  if (dtype == RLK_DTYPE_BF16) return f(Bf16{});
  if (dtype == RLK_DTYPE_F16) return f(F16{});
  return f(F32{});
}

template <class F>
inline rlk_status with_pair(int32_t dtype, int32_t out_dtype, F f) {
  if (dtype == RLK_DTYPE_BF16) return f(Bf16{}, Bf16{});
  if (dtype == RLK_DTYPE_F16) return f(F16{}, F16{});
  return out_dtype == RLK_DTYPE_BF16 ? f(F32{}, Bf16{}) : f(F32{}, F32{});
}

// What a kernel has to be allowed, asked for once per device (racing first calls ask for the same).
struct OncePerDevice {
  std::atomic<uint64_t> done{0};
  template <class F>
  bool operator()(F ask) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (!ask()) return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
  }
};

// The same for a whole number above 0 (0: it could not be found out, and is asked for again).
struct KnownPerDevice {
  std::atomic<int> of[64] = {};
  template <class F>
  int operator()(F ask) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 0 || dev >= 64) return ask();
    int v = of[dev].load(std::memory_order_acquire);
    if (v == 0) of[dev].store(v = ask(), std::memory_order_release);
    return v;
  }
};

// CTAs of a cluster: `want`, or half of it and so on while fits(ctas) says that the device has no place for it (a part of a
// GPU may have none for more than the 8 that every device takes).
template <class Fits>
inline int cluster_that_fits(int want, Fits fits) {
  while (want > 8 && !fits(want)) want /= 2;
  return want;
}

// A kernel that may start while the one before it on the stream ends (it waits for it by itself).
template <class... A>
inline rlk_status launch_after(void (*kernel)(A...), dim3 grid, int threads, cudaStream_t s, const A&... a) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a...) == cudaSuccess ? RLK_OK : RLK_ERR_CUDA;
}

inline rlk_status launched() { return cudaGetLastError() == cudaSuccess ? RLK_OK : RLK_ERR_CUDA; }

// Workspaces are carved into arrays that start on 256-byte boundaries.
inline size_t carved(size_t bytes) { return (bytes + 255) & ~size_t{255}; }

}  // namespace
}  // namespace rlk
