// rlk_logits_row.cuh -- one pass over a row of logits by a cluster of CTAs: the statistics (fixed order,
// rlk_logits.cuh), the target's rank and the maxima that the search for alternatives starts from; and
// the launch shapes of the kernels that make it.
#pragma once

#include "rlk_logits.cuh"

namespace rlk {
namespace {

constexpr int ROW_THREADS = 256;
constexpr int MAX_CLUSTER = 8;                               // CTAs of one row (the portable cluster size)
constexpr int MAX_ROW_THREADS = 1024;
constexpr int MAX_ROW_WARPS = MAX_CLUSTER * MAX_ROW_THREADS / 32;

// ---------------------------------------------------------------------------
// one pass over a row by a cluster of CTAs (one CTA when there are rows enough)
// ---------------------------------------------------------------------------
// Warp g of the row's C x (blockDim / 32) warps takes leaves g, g + (number of warps), ... and
// leaves what it found in the shared memory of the cluster's CTA 0 (distributed shared memory):
// (m, s, u, r) of each leaf, the maxima of its 32 cells (TOP: a cell is the 32 columns that a lane
// holds, so its maximum costs nothing), and how many columns stand ahead of the target.
struct RowSmem {
  Stats* leaf;      // [n_leaves]
  float* cell;      // [cell_room(n)]
  int* count;       // [MAX_ROW_WARPS]
};

__host__ __device__ constexpr int leaves_of(int n) { return (n + ROW_LEAF - 1) / ROW_LEAF; }
__host__ __device__ constexpr int cells_of(int n) { return leaves_of(n) * 32; }
__host__ __device__ constexpr int cell_room(int n) { return (cells_of(n) + 127) / 128 * 128; }

// The target of a row.
struct RankOf {
  bool ok = false;       // it is a column
  bool on = false;       // and its rank is wanted
  int y = 0;
  float z = 0.f;
  uint32_t ge = 0, gt = 0;  // its logit and the next value above it, in both halves of a word for 16-bit types
  template <class R>
  __device__ __forceinline__ void load(const R& row, const int64_t* y_ptr, bool wanted) {
    using E = typename R::E;
    const int64_t v = y_ptr ? *y_ptr : -1;
    ok = v >= 0 && v < row.n;
    on = ok && wanted;
    if (!ok) return;
    y = static_cast<int>(v);
    const typename E::bits b = row.p[v];
    z = E::to_f32(b);
    ge = b;
    gt = next_above<E>(b);
    if constexpr (sizeof(b) == 2) ge *= 0x10001u, gt *= 0x10001u;
  }
};

__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.relaxed.cluster.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}

// a before b in the order of the alternatives
__device__ __forceinline__ bool ahead(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }

// Columns of this lane's packs that stand ahead of the target.
template <class E>
__device__ __forceinline__ int count_ahead(const Pack<E> (&k)[LEAF_GROUPS], const RankOf& q, int leaf, int lane) {
  int n = 0;
  if (leaf == q.y / ROW_LEAF) {
#pragma unroll
    for (int j = 0; j < LEAF_GROUPS; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 z = pair(k[j], i / 2);
        n += ahead(i & 1 ? z.y : z.x, leaf * ROW_LEAF + j * LEAF_GROUP + lane * 8 + i, q.z, q.y);
      }
    return n;
  }
  const uint32_t bar = leaf < q.y / ROW_LEAF ? q.ge : q.gt;  // ties count before the target, not after
  if constexpr (Pack<E>::EB == 4) {
#pragma unroll
    for (int j = 0; j < LEAF_GROUPS; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) n += __uint_as_float(k[j].w[i]) >= __uint_as_float(bar);
  } else {
    uint32_t acc = 0;
#pragma unroll
    for (int j = 0; j < LEAF_GROUPS; ++j)
#pragma unroll
      for (int i = 0; i < Pack<E>::WORDS; ++i) acc = E::count_ge2(k[j].w[i], bar, acc);
    const float2 c = E::to_f32x2(acc);
    n = static_cast<int>(c.x) + static_cast<int>(c.y);
  }
  return n;
}

// What one leaf leaves behind (see RowSmem), at leaf0 / cell0 of the cluster's shared memory, from
// each lane that `puts` (lane 0 alone with ENT: the others lack u). Returns how many of the lane's
// columns stand ahead of the target.
template <bool ENT, bool TOP, class E>
__device__ __forceinline__ int leaf_pass(const Pack<E> (&k)[LEAF_GROUPS], int l, float c, const RankOf& rank,
                                         uint32_t leaf0, uint32_t cell0, bool puts, int lane) {
  float m = pack_max(k), r = 0.f;
  if constexpr (TOP) st_cluster_u32(cell0 + static_cast<uint32_t>(l * 32 + lane) * 4, __float_as_uint(m));
  m = warp_max(m);
  float2 x;
  if (m == neg_inf()) x = make_float2(any_nan(k) ? quiet_nan() : 0.f, 0.f);
  else x = leaf_sums<ENT>(k, m, c, &r, lane);
  if (puts) {
    st_cluster_f32x4(leaf0 + static_cast<uint32_t>(l * 16), m, x.x, x.y, r);
  }
  // a leaf whose best column is below the target has none ahead of it: for a likely token, most
  return rank.on && m >= rank.z ? count_ahead(k, rank, l, lane) : 0;
}

// Starts the copy of a leaf into L2, where the whole leaf lies inside the row: the passes that have no
// registers for a second leaf have the next one on its way all the same (8192 rows of 151936 in bf16
// with 20 alternatives: 464 -> 433 us; two leaves ahead 436).
template <class R>
__device__ __forceinline__ void prefetch_leaf(const R& row, int l) {
  constexpr int EB = sizeof(*row.p);
  if ((l + 1) * ROW_LEAF > row.n) return;
  const char* p = reinterpret_cast<const char*>(row.p) - row.shift + static_cast<int64_t>(l) * ROW_LEAF * EB;
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(ROW_LEAF * EB) : "memory");
}

// `begin` runs in every thread after the first loads have been issued: what it loads arrives with them.
template <bool ENT, bool TOP, class R, class B, class E = typename R::E>
__device__ __forceinline__ void row_pass(const R& row, float c, RankOf& rank, const RowSmem& sm, int C, int r, B begin) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5, g = r * warps + warp, n_leaves = leaves_of(row.n), step = C * warps;
  if (C > 1) cluster_arrive();  // CTA 0 must have started before anyone writes to it
  const uint32_t leaf0 = map_to_cta(smem_u32(sm.leaf), 0);
  const uint32_t cell0 = TOP ? map_to_cta(smem_u32(sm.cell), 0) : 0;
  int count = 0;
  // 64 registers have room for the next leaf's packs in the lean pass over 16-bit types alone (8192
  // rows of 151936 in bf16: 357 -> 351 us); elsewhere the other warps hide the loads
  constexpr bool AHEAD = !ENT && sizeof(typename E::bits) == 2;
  Pack<E> k[AHEAD ? 2 : 1][LEAF_GROUPS];
  if (g < n_leaves) load_leaf(row, g, lane, k[0]);
  begin();
  if (C > 1) cluster_wait();
  if constexpr (AHEAD) {
    for (int l = g; l < n_leaves; l += 2 * step) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = l + u * step;
        if (i >= n_leaves) break;
        if (i + step < n_leaves) load_leaf(row, i + step, lane, k[u ^ 1]);
        leaf_pass<ENT, TOP>(k[u], i, c, rank, leaf0, cell0, lane == 0, lane);
      }
    }
  } else {
    for (int l = g; l < n_leaves;) {
      if (lane == 0) prefetch_leaf(row, l + step);
      count += leaf_pass<ENT, TOP>(k[0], l, c, rank, leaf0, cell0, lane == 0, lane);
      l += step;
      if (l < n_leaves) load_leaf(row, l, lane, k[0]);
    }
  }
  if (rank.on) {
    count = __reduce_add_sync(kFullWarp, count);
    if (lane == 0) st_cluster_u32(map_to_cta(smem_u32(sm.count + g), 0), static_cast<uint32_t>(count));
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
}

// ---------------------------------------------------------------------------
// launch shapes and types (host)
// ---------------------------------------------------------------------------
// The numbers below are of the whole GPU: 152 SMs of 228 KB. On fewer SMs the shapes are other than the best, and
// the results the same.
// CTAs (c, a cluster) and warps (w) of a row in the statistics passes. With 64 registers a thread an
// SM runs 32 warps, so floor(32 / w) CTAs, if their shared memory (smem bytes each) fits; a row takes
// ceil(leaves / (c w)) rounds of leaves, about two more for what surrounds them (the target, the fold,
// the alternatives) and half a one for each doubling of the cluster. The shape with the least waves x
// rounds is taken, among widths that use the 32 warps well: 8 CTAs of 19 for a single row of 149 leaves.
// Where rows fill the GPU many times over the answer is known. Without alternatives it is one CTA of 4
// warps (4096 rows of 32000 in bf16, distillation's forward: 51 us, with 8 warps 61), with them one of 8,
// for they need shared memory and every warp (8192 rows of 151936 in bf16 with 20: 4 warps take 528 us, 8
// 433, 16 501). In between, narrow CTAs save a wave (796 rows of 50257 in f16 with 20: 35 -> 32.5 us).
// Rows of more than 100 leaves have rounds enough and take 8 warps in any case (4096 rows of 151936 in
// fp32: 338 us with 8, 350 with 4; 800 in bf16 with 20 alternatives 59.6 with 10, 62.7 with 5, where rows
// of 100000 take 43.7 and 42.6). Short rows take a warp a leaf; a few of them at least 4 or 8, to find
// the alternatives (64 rows of 1000 with k = 100: 33 -> 17 us; 4096 rows with k = 50 take 37 us with 2
// warps, 56 with 8).
struct RowShape {
  int cluster, threads;
};
constexpr size_t SM_SMEM = 228 << 10;     // shared memory of an SM
constexpr size_t ROW_SMEM_FIXED = 4 << 10;  // what a row kernel takes besides its dynamic part (and 1 KB of the system's)
inline RowShape row_shape(const LogitRows& in, int top_k, size_t smem) {
  const int L = leaves_of(in.n);
  const uint32_t T = static_cast<uint32_t>(in.T);
  const bool few_rows = T <= 4 * 152, top = top_k > 0;
  const int usual = L >= 8 || (few_rows && top_k > 32) ? 8 : few_rows && top && L < 4 ? 4 : L < 2 ? 2 : L;
  const int least_warps = L >= 8 && L <= 100 ? 4 : usual;  // of a CTA that has a row to itself
  RowShape best{1, 32 * (top ? usual : least_warps)};
  if (T >= 16 * 152) return best;
  const uint32_t fit = static_cast<uint32_t>(SM_SMEM / smem);
  uint32_t least = UINT32_MAX;
  for (int c = 1, half = 0; c <= MAX_CLUSTER; c *= 2, ++half) {
    const int each = (L + c - 1) / c;  // leaves of a CTA: more warps would idle
    for (int w : {4, 5, 6, 7, usual, 10, 12, 14, 16, 20, 25, 32, each}) {
      if (w > 32 || w < (c == 1 ? least_warps : usual) || (w > usual && w > each)) continue;
      const uint32_t ctas = 32u / w < fit ? 32u / w : fit, room = 152u * (ctas ? ctas : 1), waves = (T * c + room - 1) / room;
      const uint32_t cost = waves * (2 * ((L + c * w - 1) / (c * w)) + 4 + half);
      if (cost < least) least = cost, best = RowShape{c, 32 * w};
    }
  }
  return best;
}

// Launches `ctas` CTAs in clusters of `cluster`.
template <class K, class A>
inline rlk_status launch_rows(K kernel, const A& args, int64_t ctas, int cluster, size_t smem, void* stream,
                              int threads = ROW_THREADS, bool opt_in = true) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  // beyond what any kernel may have without asking (its static part takes up to 14 KB of 48): rows of
  // more than about 230,000 columns, with alternatives
  if (smem > (32 << 10) && opt_in &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return RLK_ERR_CUDA;
  if (cudaLaunchKernelEx(&cfg, kernel, args) != cudaSuccess) return RLK_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? RLK_OK : RLK_ERR_CUDA;
}

// Whether every row starts on a 16-byte boundary.
inline bool aligned_rows(const void* base, int64_t ld, int bytes) {
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 && ld * bytes % 16 == 0;
}

template <bool B>
struct Flag {
  static constexpr bool value = B;
};

// Calls f with the element type(s) and the alignment as types.
template <class F>
inline rlk_status with_types(int32_t dtype, bool aligned, F f) {
  const auto al = [&](auto e) { return aligned ? f(e, Flag<true>{}) : f(e, Flag<false>{}); };
  return dtype == RLK_DTYPE_BF16 ? al(Bf16{}) : dtype == RLK_DTYPE_F16 ? al(F16{}) : al(F32{});
}

}  // namespace
}  // namespace rlk
