// rlk_logits_grad.cuh -- writing the gradient with respect to a row of logits: which CTA writes which
// columns, in packs that are aligned in the output whatever their alignment in the logits.
#pragma once

#include "rlk_logits_row.cuh"

namespace rlk {
namespace {

constexpr int GRAD_PACKS = 4;                                // packs a thread has in flight in the gradients

struct GradOut {
  void* base;
  int64_t ld;
  int32_t V;
};

// The columns of one row of dlogits that one CTA writes, in packs of 8 that are 16-byte aligned in
// the output: `head` columns lie before the first of them, fewer than 8 after the last. The row is
// divided into `parts` runs of packs; the first part takes the head, the last the tail. The input
// packs of the same columns may lie at any alignment (Row); where dlogits are the logits
// themselves they are aligned as well, so no thread reads a column that another one writes.
template <class E_, class O_, bool AL>
struct GradPart {
  using E = E_;
  using O = O_;
  Row<E, AL> in;              // from column `head` on
  typename O::bits* out;      // the row's first column
  int n, V, head, packs, q0, q1, lo, hi;
  __device__ __forceinline__ GradPart(const typename E::bits* z, int n_, typename O::bits* o, int V_, int part, int parts,
                                      int32_t* err)
      : in(z, n_, err), out(o), n(n_), V(V_) {
    constexpr int OB = sizeof(typename O::bits);
    head = min(V, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(o) & 15u)) & 15u) / OB);
    packs = (V - head) / 8;
    const int per = (packs + parts - 1) / parts;
    q0 = min(packs, part * per);
    q1 = min(packs, q0 + per);
    lo = part == 0 ? 0 : head + 8 * q0;
    hi = part == parts - 1 ? V : head + 8 * q1;
    in = Row<E, AL>(z + head, max(0, n - head), err);
  }
  // Starts the copy of the part's logits into L2 (the whole vectors among them), by one thread.
  __device__ __forceinline__ void prefetch() const {
    const uintptr_t a = (reinterpret_cast<uintptr_t>(in.p + 8 * q0) + 15) & ~uintptr_t{15};
    const uintptr_t b = reinterpret_cast<uintptr_t>(in.p + min(in.n, 8 * q1)) & ~uintptr_t{15};
    if (a < b)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"(static_cast<uint32_t>(b - a)) : "memory");
  }
  __device__ __forceinline__ bool owns(int64_t c) const { return c >= lo && c < hi; }
  __device__ __forceinline__ void put(int c, float v) const {
    if (dbg_ok(c >= 0 && c < V, in.err)) out[c] = O::from_f32(v);
  }
};

template <class O>
__device__ __forceinline__ void store_pack(typename O::bits* p, const float (&v)[8]) {
  uint4* q = reinterpret_cast<uint4*>(p);
  if constexpr (sizeof(typename O::bits) == 4) {
    q[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    q[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    q[0] = make_uint4(O::pack2(v[0], v[1]), O::pack2(v[2], v[3]), O::pack2(v[4], v[5]), O::pack2(v[6], v[7]));
  }
}

// Writes f(z, column) for the part's columns (0 past the row's n columns, and everywhere when !live,
// without reading). Each thread has U packs in flight.
template <int U, class G, class F>
__device__ __forceinline__ void write_part(const G& g, bool live, const F& f) {
  using E = typename G::E;
  using O = typename G::O;
  const int tid = threadIdx.x, threads = blockDim.x;
  const auto put_pack = [&](const Pack<E>& k, int c) {
    float v[8];
    f.pack(k, g.head + c, v);
    if (c + 8 > g.in.n) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i >= g.in.n) v[i] = 0.f;
    }
    if (dbg_ok(g.head + c + 8 <= g.V, g.in.err)) store_pack<O>(g.out + g.head + c, v);
  };
  // the columns outside the packs: before the head and after the last pack
  if (tid < 16) {
    const int c = tid < 8 ? tid : g.head + 8 * g.packs + tid - 8;
    if (g.owns(c) && (tid >= 8 || c < g.head))
      g.put(c, live && c < g.n ? f.one(E::to_f32(g.in.p[c - g.head]), c) : 0.f);
  }
  for (int q = g.q0; q < g.q1; q += U * threads) {
    Pack<E> k[U];
    const bool full = live && q + U * threads <= g.q1 && packs_inside(g.in, q * 8, (q + U * threads) * 8);
    if (full) {
#pragma unroll
      for (int u = 0; u < U; ++u) k[u] = load_pack(g.in, (q + tid + u * threads) * 8);
    } else if (live) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = q + tid + u * threads;
        if (p < g.q1) k[u] = packs_inside(g.in, p * 8, p * 8 + 8) ? load_pack(g.in, p * 8) : load_pack_edge(g.in, p * 8);
      }
    }
    if (full) {
#pragma unroll
      for (int u = 0; u < U; ++u) put_pack(k[u], (q + tid + u * threads) * 8);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = q + tid + u * threads;
        if (p >= g.q1) break;
        if (live) {
          put_pack(k[u], p * 8);
        } else {
          const float v[8] = {};
          store_pack<O>(g.out + g.head + p * 8, v);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// log p from the caller's lse, or from the row again
// ---------------------------------------------------------------------------
// The gradient needs log p = s (z - m) - l of every column. The forward's lse serves as l, with m = 0,
// while its rounding, 2^-24 |lse|, which is a relative error of every p, stays small against what p has
// anyway: against the sum's error (2^-17) for a gradient in fp32, up to |lse| = 256; against an eighth of
// the gradient's own rounding in f16 (2^-12, up to 512) and in bf16 (2^-9, up to 4096). Beyond that --
// a large offset, a low temperature, a row masked wholly by a finite value -- one fp32 does not hold
// log S well enough (at 10^9 not at all), and M and log S come from the row once more.

// Whether the row of this lse (not NaN) is to be read again, for a gradient of type O.
template <class O>
__device__ __forceinline__ bool lse_is_coarse(float lse) {
  return fabsf(lse) > O::kLseRange && lse != neg_inf();
}

// M and log S of a row, by one CTA, with the forward's bits: every leaf as in leaf_pass, its statistics
// (leaf: shared memory for the row's leaves) folded by fold_leaves. Every thread has read the row when it
// returns. A leaf is read twice, pack by pack, and write_row goes element by element: such rows are rare,
// and this small they leave the stream over the others its registers (whole leaves in registers, or packs in
// write_row, cost the gradients of other rows 2 to 13 %). 8192 rows of 151936 in bf16 take 4.0 ms where all
// of them come here (711 us where none does), 2000 of 50264 in fp32 531 us (122).
template <class E>
__device__ __noinline__ RowLog read_row_log(const typename E::bits* z, int n, float c, Stats* leaf, int32_t* err) {
  __shared__ RowLog found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, L = leaves_of(n);
  const Row<E, false> row(z, n, err);
  for (int l = warp; l < L; l += warps) {
    const int c0 = l * ROW_LEAF + lane * 8;
    const auto octet = [&](int j) {  // this lane's j-th pack
      const int x = c0 + j * LEAF_GROUP;
      return packs_inside(row, x, x + 8) ? load_pack(row, x) : load_pack_edge(row, x);
    };
    float m = neg_inf();
#pragma unroll 1
    for (int j = 0; j < LEAF_GROUPS; ++j) {
      const Pack<E> k[1] = {octet(j)};
      m = fmaxf(m, pack_max(k));
    }
    m = warp_max(m);
    const LeafBase at = leaf_base(m, c);
    float even = 0.f, odd = 0.f;
#pragma unroll 1
    for (int j = 0; j < LEAF_GROUPS; ++j) {
      const Pack<E> k = octet(j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = pair(k, i);
        even = __fadd_rn(even, ex2_approx(at.of(x.x, c)));
        odd = __fadd_rn(odd, ex2_approx(at.of(x.y, c)));
      }
    }
    const float s = m == neg_inf() ? 0.f : warp_sum(__fadd_rn(even, odd));
    if (lane == 0) leaf[l] = Stats{m, s, 0.f, at.r};
  }
  __syncthreads();
  if (warp == 0) {
    const RowLog p = row_log(fold_leaves(leaf, L, c, lane));
    if (lane == 0) found = p;
  }
  __syncthreads();
  return found;
}

// Writes f of a whole row, by one CTA (zeros when !live); a thread reads the columns that it writes.
template <class E, class O, class F>
__device__ __forceinline__ void write_row(const typename E::bits* z, int n, typename O::bits* out, int V, bool live, const F& f) {
#pragma unroll 4
  for (int i = threadIdx.x; i < V; i += ROW_THREADS) out[i] = O::from_f32(live && i < n ? f.one(E::to_f32(z[i]), i) : 0.f);
}

// CTAs of a row in a kernel that writes gradients alone: parts of up to four rounds of every thread's
// packs (what a CTA does once -- its row's scalars, the teacher's softmax -- is then small: 8192 rows of
// 151936 in bf16 take 711 us with four rounds, 954 with one), as long as that leaves the GPU full.
inline int grad_parts(const LogitRows& in, const GradOut& o) {
  constexpr int kCols = 8 * GRAD_PACKS * ROW_THREADS;
  constexpr int64_t kEnough = 6 * 152;
  const int64_t rounds = (o.V + kCols - 1) / kCols;
  int64_t each = in.T * rounds / kEnough;
  each = each < 1 ? 1 : each > 4 ? 4 : each;
  return static_cast<int>((rounds + each - 1) / each);
}

// dlogits: the logits' type, or bf16 for fp32 logits
inline rlk_status check_out(const LogitRows& in, int32_t dtype, void* dlogits, int32_t out_dtype, int64_t V,
                            int64_t out_ld, GradOut* o) {
  const int eb = dtype_bytes(out_dtype);
  if (eb == 0 || V < in.n || out_ld < V) return RLK_ERR_INVALID_ARG;
  if (out_dtype != dtype && !(dtype == RLK_DTYPE_F32 && out_dtype == RLK_DTYPE_BF16)) return RLK_ERR_UNSUPPORTED;
  if (V > RLK_MAX_LOGITS_VOCAB) return RLK_ERR_UNSUPPORTED;
  if (in.T > 0 && (!dlogits || reinterpret_cast<uintptr_t>(dlogits) % eb != 0)) return RLK_ERR_INVALID_ARG;
  // in place: the very same array; otherwise no row of one meets a row of the other
  const int64_t zd = in.ld * dtype_bytes(dtype), dd = out_ld * eb;  // bytes from row to row
  if (in.T > 0 && !(dlogits == in.base && out_dtype == dtype && (zd == dd || in.T == 1))) {
    const uintptr_t z = reinterpret_cast<uintptr_t>(in.base), d = reinterpret_cast<uintptr_t>(dlogits);
    const uintptr_t zn = static_cast<uintptr_t>(in.n) * dtype_bytes(dtype), dn = static_cast<uintptr_t>(V) * eb;
    if (z < d + (in.T - 1) * dd + dn && d < z + (in.T - 1) * zd + zn) {
      // the arrays as a whole meet: rows the same distance apart may lie side by side all the same
      if (in.T == 1 || zd != dd) return RLK_ERR_INVALID_ARG;
      const uintptr_t at = ((d % zd) + zd - z % zd) % zd;  // where the gradient's rows start, from the logits' on
      if (at < zn || at + dn > static_cast<uintptr_t>(zd)) return RLK_ERR_INVALID_ARG;
    }
  }
  *o = GradOut{dlogits, out_ld, static_cast<int32_t>(V)};
  return RLK_OK;
}

// Whether the packs of every row's gradient are aligned in the logits as well: both sets of rows
// are, or they lie alike (the same type, and the same distance from a boundary in every row).
inline bool aligned_pair(const LogitRows& in, int32_t dtype, const GradOut& o, int32_t out_dtype) {
  const int eb = dtype_bytes(dtype), ob = dtype_bytes(out_dtype);
  if (aligned_rows(in.base, in.ld, eb) && aligned_rows(o.base, o.ld, ob)) return true;
  return eb == ob && (reinterpret_cast<uintptr_t>(in.base) - reinterpret_cast<uintptr_t>(o.base)) % 16 == 0 &&
         (in.ld - o.ld) * eb % 16 == 0;
}

template <class F>
inline rlk_status with_types(int32_t dtype, int32_t out_dtype, bool aligned, F f) {
  const auto al = [&](auto e, auto o) { return aligned ? f(e, o, Flag<true>{}) : f(e, o, Flag<false>{}); };
  if (dtype == RLK_DTYPE_BF16) return al(Bf16{}, Bf16{});
  if (dtype == RLK_DTYPE_F16) return al(F16{}, F16{});
  return out_dtype == RLK_DTYPE_BF16 ? al(F32{}, Bf16{}) : al(F32{}, F32{});
}

}  // namespace
}  // namespace rlk
