// rlk_rows.cuh -- what the operators around the head (embedding, layer norm) share: rows of hidden
// values cut into packs of 8 columns, their loads and stores at any alignment, sums over a row in one
// fixed order, and the host-side argument checks.
//
// Order of a row's sums: pack p (columns 8 p .. 8 p + 7) belongs to slot p mod 256; a slot adds its
// packs in ascending order, each pack's 8 values as a balanced tree; 32 slots combine by an
// xor-butterfly, the eight groups of 32 by a balanced tree. Slots without packs hold 0, so that a row
// of few packs can be taken by fewer warps with the same bits. The order depends on column indices
// alone: not on the row's address, on alignment or on how many rows a CTA takes.
#pragma once

#include "rlk_logits.cuh"

namespace rlk {
namespace {

constexpr int SLOTS = 256;  // of a row's sums; the threads of the widest team that takes one row

template <bool V>
struct Is {
  static constexpr bool value = V;
};

// 8 columns of a row of n, from column c0 (a multiple of 8) on; 0 beyond the row. AL: the row starts on
// a 16-byte boundary and n is a multiple of 8.
template <class E, bool AL>
__device__ __forceinline__ Pack<E> load_columns(const typename E::bits* row, int c0, int n, int32_t* err) {
  const Row<E, AL> r(row, n, err);
  if (AL || packs_inside(r, c0, c0 + 8)) return load_pack(r, c0);
  Pack<E> k{};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = c0 + i < n ? row[c0 + i] : 0u;
    if constexpr (Pack<E>::EB == 4) k.w[i] = b;
    else k.w[i / 2] |= b << (i & 1 ? 16 : 0);
  }
  return k;
}

template <class E>
__device__ __forceinline__ void unpack(const Pack<E>& k, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = pair(k, i);
    v[2 * i] = x.x;
    v[2 * i + 1] = x.y;
  }
}

template <class O, bool AL>
__device__ __forceinline__ void store_columns(typename O::bits* row, int c0, int n, const float (&v)[8], int32_t* err) {
  if (!dbg_ok(c0 >= 0 && c0 < n && (!AL || c0 + 8 <= n), err)) return;
  if constexpr (AL) {
    uint4* q = reinterpret_cast<uint4*>(row + c0);
    if constexpr (sizeof(typename O::bits) == 4) {
      q[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      q[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
      q[0] = make_uint4(O::pack2(v[0], v[1]), O::pack2(v[2], v[3]), O::pack2(v[4], v[5]), O::pack2(v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < n) row[c0 + i] = O::from_f32(v[i]);
  }
}

__device__ __forceinline__ float tree8(const float (&v)[8]) {
  return __fadd_rn(__fadd_rn(__fadd_rn(v[0], v[1]), __fadd_rn(v[2], v[3])),
                   __fadd_rn(__fadd_rn(v[4], v[5]), __fadd_rn(v[6], v[7])));
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline bool on_boundary(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// T rows of n elements, `ld` elements apart: whether every row starts on a 16-byte boundary and is a
// whole number of packs.
inline bool whole_packs(const void* p, int64_t T, int64_t n, int64_t ld, int eb) {
  return on_boundary(p, 16) && n % 8 == 0 && (T <= 1 || ld * eb % 16 == 0);
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

inline rlk_status launched() { return cudaGetLastError() == cudaSuccess ? RLK_OK : RLK_ERR_CUDA; }

// Workspaces are carved into arrays that start on 256-byte boundaries.
inline size_t carved(size_t bytes) { return (bytes + 255) & ~size_t{255}; }

}  // namespace
}  // namespace rlk
