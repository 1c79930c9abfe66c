// rlk_embedding.cu -- rows of a table by token, and the table's gradient by sorted tokens.
//
//   out[t] = s E[id_t],   dE[v] (+)= s sum_{t : id_t = v} dout[t]
//
// The gradient sorts (token, position) stably, so that a token's positions stand side by side in
// ascending order, and adds their rows in runs of 32 positions of that token: a run in ascending order,
// then the runs in ascending order. What a row of dE holds depends on that token's rows alone, not on
// which other tokens the batch or the shard has.
#include <algorithm>

#include "rlk_rows.cuh"

namespace rlk {
namespace {

struct Shard {  // the table's rows are tokens [start, start + rows) of those below V_true
  int64_t start, rows, V_true;
  int32_t* err;
  // This shard's row of a token, -1: none (padding, another shard's), -2: not a token
  __device__ __forceinline__ int32_t row_of(int64_t id) const {
    if (id < -1 || id >= V_true) {
      if (err) atomicOr(err, RLK_FLAG_BAD_TARGET);
      return -2;
    }
    const int64_t r = id - start;
    return id < 0 || r < 0 || r >= rows ? -1 : static_cast<int32_t>(r);
  }
};

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
struct LookupArgs {
  const void* table;
  void* out;
  const int64_t* ids;
  int64_t T, ld, out_ld;
  int32_t H;
  float scale;
  Shard shard;
};

template <class E, class O, bool AL>
__global__ void __launch_bounds__(256) lookup_kernel(const LookupArgs a) {
  const int64_t t = blockIdx.x;
  const int32_t r = a.shard.row_of(a.ids[t]);
  const auto* row = static_cast<const typename E::bits*>(a.table) + static_cast<int64_t>(r < 0 ? 0 : r) * a.ld;
  auto* out = static_cast<typename O::bits*>(a.out) + t * a.out_ld;
  for (int c = 8 * threadIdx.x; c < a.H; c += 8 * 256) {
    F32x2 v[4];
    if (r >= 0) {
      unpack(load_columns<E, AL>(row, c, a.H, a.shard.err), v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(a.scale));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = both(r == -2 ? quiet_nan() : 0.f);
    }
    store_columns<O, AL>(out, c, a.H, v, a.shard.err);
  }
}

// ---------------------------------------------------------------------------
// sorting tokens
// ---------------------------------------------------------------------------
// A radix sort from the low digits up, by one cluster: warp w of the cluster's W owns the w-th run of
// positions, counts its digits, gets from the counts of all warps where each of its digits goes, and goes through
// its run again to put the entries there. Runs and lanes are in ascending order of position, so that the sort is
// stable and its result unique. A token without a row here sorts behind the last row.
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_BINS = 512;  // 9 bits at most at a time: two passes for up to 2^18 rows
constexpr int SORT_CTAS = 16;
constexpr int RUN = 32;         // positions of one token that are added in one go

struct Entry {
  uint32_t row;  // of the table; `rows`: none
  uint32_t t;
};

struct SortArgs {
  const int64_t* ids;
  Entry *a, *b;        // [T] each
  int32_t T, bits, passes;
  Shard shard;
  int32_t* done;       // counters of the runs, to be zeroed
  int32_t n_done;
  float* dW;           // to be zeroed by the other clusters, where n_zero > 0
  int64_t n_zero;
};

struct SortSmem {
  uint32_t count[SORT_WARPS][SORT_BINS];  // digits of each warp; then how many stand before the warp in this CTA
  uint32_t total[SORT_CTAS][SORT_BINS];   // of each CTA of the cluster, which puts its own into all of them
  uint32_t base[SORT_BINS];               // where this CTA's entries of a digit start
  uint32_t warp_sum[SORT_WARPS];
};

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ Entry sort_entry(const SortArgs& a, const Entry* src, int32_t t) {
  if (src) {
    const uint2 v = __ldcg(reinterpret_cast<const uint2*>(src + t));
    return Entry{v.x, v.y};
  }
  const int32_t r = a.shard.row_of(a.ids[t]);
  return Entry{r < 0 ? static_cast<uint32_t>(a.shard.rows) : static_cast<uint32_t>(r), static_cast<uint32_t>(t)};
}

// KEPT: every warp has up to KEPT groups of 32 positions, which stay in registers between the two ways through them;
// 0: any number, read again.
template <int KEPT>
__device__ __forceinline__ void sort_tokens(const SortArgs& a, SortSmem& m) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), ctas = cluster_size();
  const int64_t warps = static_cast<int64_t>(ctas) * SORT_WARPS;
  const int32_t per = static_cast<int32_t>((a.T + 32 * warps - 1) / (32 * warps)) * 32;
  const int64_t lo = (static_cast<int64_t>(rank) * SORT_WARPS + warp) * per;
  const int32_t first = static_cast<int32_t>(min(static_cast<int64_t>(a.T), lo));
  const int32_t last = static_cast<int32_t>(min(static_cast<int64_t>(a.T), lo + per));
  const int each = (a.bits + a.passes - 1) / a.passes;
  const int bins = 1 << each;
  uint32_t* mine = m.count[warp];

  for (int i = rank * SORT_THREADS + threadIdx.x; i < a.n_done; i += ctas * SORT_THREADS) a.done[i] = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    const Entry* src = pass == 0 ? nullptr : pass & 1 ? a.a : a.b;
    Entry* dst = pass & 1 ? a.b : a.a;
    const int shift = pass * each;
    Entry kept[KEPT ? KEPT : 1];
    if constexpr (KEPT > 0) {
#pragma unroll
      for (int g = 0; g < KEPT; ++g)
        if (first + 32 * g + lane < last) kept[g] = sort_entry(a, src, first + 32 * g + lane);
    }
    // f(digit, entry, lanes of the same digit) of each group; a digit beyond the bins: no entry
    const auto groups = [&](auto f) {
      const auto group = [&](const Entry& e, bool on) {
        const uint32_t d = on ? (e.row >> shift) & static_cast<uint32_t>(bins - 1) : 0xFFFFFFFFu;
        f(d, e, __match_any_sync(kFullWarp, d), on);
      };
      if constexpr (KEPT > 0) {
#pragma unroll
        for (int g = 0; g < KEPT; ++g)
          if (first + 32 * g < last) group(kept[g], first + 32 * g + lane < last);
      } else {
        for (int32_t t = first; t < last; t += 32) {
          Entry e{0, 0};
          if (t + lane < last) e = sort_entry(a, src, t + lane);
          group(e, t + lane < last);
        }
      }
    };
    for (int b = lane; b < bins; b += 32) mine[b] = 0;
    __syncwarp();
    groups([&](uint32_t d, const Entry&, uint32_t like, bool on) {
      if (on && lane == __ffs(like) - 1) mine[d] += __popc(like);
      __syncwarp();
    });
    __syncthreads();
    const int b = threadIdx.x;
    if (b < bins) {
      uint32_t c[SORT_WARPS], run = 0;
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) c[w] = m.count[w][b];
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) {
        m.count[w][b] = run;
        run += c[w];
      }
      const uint32_t to = smem_u32(&m.total[rank][b]);
      for (uint32_t c = 0; c < ctas; ++c) st_cluster_u32(map_to_cta(to, c), run);
    }
    cluster_sync();
    // all entries of lower digits, and those of this digit in CTAs before this one
    uint32_t before = 0, all = 0;
    if (b < bins) {
#pragma unroll 8
      for (uint32_t c = 0; c < ctas; ++c) {
        const uint32_t v = m.total[c][b];
        all += v;
        before += c < rank ? v : 0;
      }
    }
    uint32_t sum = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(kFullWarp, sum, d);
      if (lane >= d) sum += v;
    }
    if (lane == 31) m.warp_sum[warp] = sum;
    __syncthreads();
    const uint32_t lower = __reduce_add_sync(kFullWarp, lane < warp ? m.warp_sum[lane] : 0);
    if (b < bins) {
      m.base[b] = lower + sum - all + before;
    }
    __syncthreads();
    groups([&](uint32_t d, const Entry& e, uint32_t like, bool on) {
      const uint32_t at = on ? m.base[d] + mine[d] + __popc(like & ((1u << lane) - 1)) : 0;
      __syncwarp();
      if (on && lane == __ffs(like) - 1) mine[d] += __popc(like);
      __syncwarp();
      if (on && dbg_ok(at < static_cast<uint32_t>(a.T), a.shard.err)) dst[at] = e;
    });
    cluster_sync();  // the entries, and the totals, are through before the next pass (and before the CTA ends)
  }
}

template <int KEPT>
__global__ void __launch_bounds__(SORT_THREADS) sort_tokens_kernel(const SortArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  const uint32_t ctas = cluster_size();
  if (blockIdx.x < ctas) {
    sort_tokens<KEPT>(a, *reinterpret_cast<SortSmem*>(dyn));
    griddep_launch_dependents();
    return;
  }
  // every other cluster: zeros into dW, whole vectors between its first and last boundary
  const int64_t i0 = static_cast<int64_t>(blockIdx.x - ctas) * SORT_THREADS + threadIdx.x;
  const int64_t n = static_cast<int64_t>(gridDim.x - ctas) * SORT_THREADS;
  const int64_t head = min(a.n_zero, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(a.dW) & 15)) & 15) / 4);
  const int64_t vecs = (a.n_zero - head) / 4;
  uint4* v = reinterpret_cast<uint4*>(a.dW + head);
#pragma unroll 4
  for (int64_t i = i0; i < vecs; i += n) v[i] = make_uint4(0, 0, 0, 0);
  if (i0 < head) a.dW[i0] = 0.f;
  if (i0 < a.n_zero - head - 4 * vecs) a.dW[head + 4 * vecs + i0] = 0.f;
  griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// adding rows
// ---------------------------------------------------------------------------
struct GatherArgs {
  const Entry* sorted;  // [T]
  const void* dout;
  float* dW;
  int64_t ld;
  int32_t T, H, rows;
  float scale;
  bool add;
  float* part;          // [2 slots][H rounded up to 8]: sums of the runs of tokens of more than one run
  int32_t* done;        // [slots][slices]: runs of such a token that are through
  int32_t slots;
  int32_t* err;
};

__device__ __forceinline__ Entry entry_at(const GatherArgs& a, int32_t p) {
  return dbg_ok(p >= 0 && p < a.T, a.err) ? a.sorted[p] : Entry{0xFFFFFFFFu, 0};
}
__device__ __forceinline__ uint32_t row_at(const GatherArgs& a, int32_t p) { return entry_at(a, p).row; }

// The first position in [lo, hi] from which on all rows are >= row (hi is such a one), by a whole warp.
__device__ __forceinline__ int32_t first_not_below(const GatherArgs& a, uint32_t row, int32_t lo, int32_t hi, int lane) {
  while (lo < hi) {
    const int32_t step = (hi - lo + 31) / 32;
    const int64_t q = static_cast<int64_t>(lo) + static_cast<int64_t>(lane) * step;
    const bool yes = q >= hi || row_at(a, static_cast<int32_t>(q)) >= row;
    const uint32_t m = __ballot_sync(kFullWarp, yes);
    const int f = m ? __ffs(m) - 1 : 32;
    const int32_t base = lo;
    if (f < 32) hi = static_cast<int32_t>(min(static_cast<int64_t>(hi), static_cast<int64_t>(base) + static_cast<int64_t>(f) * step));
    if (f > 0) lo = static_cast<int32_t>(min(static_cast<int64_t>(hi), static_cast<int64_t>(base) + static_cast<int64_t>(f - 1) * step + 1));
  }
  return hi;
}

constexpr int GATHER_WARPS = 8;

// A CTA takes a position, each of its warps a slice of 256 C columns; it has work where a run starts there. Bound by memory where
// the tokens are many; what it takes is a chain of two loads (entries, then rows) and many warps to hide it, so everything
// that the entries around the position tell is read at once, and the row of dW with the rows that are added to it.
template <class E, bool AL, int C>
__global__ void __launch_bounds__(32 * GATHER_WARPS) gather_kernel(const GatherArgs a) {
  const int lane = threadIdx.x & 31;
  const int slice = static_cast<int>(blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5));
  const int slices = static_cast<int>(gridDim.y * (blockDim.x >> 5));
  const int32_t p = static_cast<int32_t>(blockIdx.x);
  griddep_wait();
  // this position and those after it, and the 32 before it
  const int32_t back = p - 1 - lane, at = p + lane, beyond = p + RUN;
  const Entry e = at < a.T ? entry_at(a, at) : Entry{0xFFFFFFFFu, 0};
  const uint32_t row_back = back >= 0 ? row_at(a, back) : 0xFFFFFFFFu;
  const uint32_t row_beyond = beyond < a.T ? row_at(a, beyond) : 0xFFFFFFFFu;
  const uint32_t row = __shfl_sync(kFullWarp, e.row, 0);
  if (row >= static_cast<uint32_t>(a.rows)) return;
  // does a run start here?
  const uint32_t same = __ballot_sync(kFullWarp, row_back == row);
  int32_t start = p;
  if (same & 1u) {
    if (same != kFullWarp) return;
    start = first_not_below(a, row, 0, p - RUN, lane);
    if ((p - start) % RUN != 0) return;
  }
  const int n = __popc(__ballot_sync(kFullWarp, e.row == row));  // its length
  const bool more = row_beyond == row, alone = start == p && !more;

  const int c0 = 256 * C * slice + 8 * lane;
  const auto on = [&](int j) { return c0 + 256 * j < a.H; };
  auto* out = reinterpret_cast<uint32_t*>(a.dW) + static_cast<int64_t>(row) * a.H;
  Pack<F32> old[C];
  if (a.add && alone) {
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (on(j)) old[j] = load_columns<F32, AL>(out, c0 + 256 * j, a.H, a.err);
  }
  F32x2 s[C][4];
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[j][i] = 0;
  constexpr int U = 8 / C > 4 ? 4 : 8 / C;  // rows in flight
  for (int i = 0; i < n; i += U) {
    Pack<E> k[U][C];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t t = __shfl_sync(kFullWarp, e.t, (i + u) & 31);
      const auto* r = static_cast<const typename E::bits*>(a.dout) + static_cast<int64_t>(t) * a.ld;
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (i + u < n && on(j)) k[u][j] = load_columns<E, AL>(r, c0 + 256 * j, a.H, a.err);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= n) break;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if (!on(j)) continue;
        F32x2 v[4];
        unpack(k[u][j], v);
#pragma unroll
        for (int q = 0; q < 4; ++q) s[j][q] = add2(s[j][q], v[q]);
      }
    }
  }
  if (!alone) {
    // leave the run's sum; the warp that is through last adds them up
    const int width = (a.H + 7) / 8 * 8;
    const int32_t seg = (start + RUN - 1) / RUN;  // a token of several runs starts with a whole one
    const int32_t slot = n == RUN ? (p + RUN - 1) / RUN : a.slots + seg;
    const bool ok = dbg_ok(slot < 2 * a.slots && seg < a.slots, a.err);
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (on(j) && ok)
        store_columns<F32, true>(reinterpret_cast<uint32_t*>(a.part) + static_cast<int64_t>(slot) * width, c0 + 256 * j, width,
                                 s[j], a.err);
    const int32_t end = more ? first_not_below(a, row + 1, p + RUN, a.T, lane) : p + n;
    const int32_t runs = (end - start + RUN - 1) / RUN;
    __threadfence();
    __syncwarp();
    int32_t before = 0;
    if (lane == 0 && ok) before = atomicAdd(&a.done[static_cast<int64_t>(seg) * slices + slice], 1);
    if (__shfl_sync(kFullWarp, before, 0) != runs - 1) return;
    __threadfence();
    if (a.add) {
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (on(j)) old[j] = load_columns<F32, AL>(out, c0 + 256 * j, a.H, a.err);
    }
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j][i] = 0;
#pragma unroll(4 / C)
    for (int32_t i = 0; i < runs; ++i) {
      const int32_t q = start + i * RUN;
      const int32_t from = q + RUN <= end ? (q + RUN - 1) / RUN : a.slots + seg;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if (!on(j)) continue;
        const float4* r = reinterpret_cast<const float4*>(a.part + static_cast<int64_t>(from) * width + c0 + 256 * j);
        const float4 x = __ldcg(r), y = __ldcg(r + 1);
        s[j][0] = add2(s[j][0], pack_f32x2(x.x, x.y));
        s[j][1] = add2(s[j][1], pack_f32x2(x.z, x.w));
        s[j][2] = add2(s[j][2], pack_f32x2(y.x, y.y));
        s[j][3] = add2(s[j][3], pack_f32x2(y.z, y.w));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    if (!on(j)) continue;
    if (a.add) {
      F32x2 v[4];
      unpack(old[j], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j][i] = fma2(s[j][i], both(a.scale), v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j][i] = mul2(s[j][i], both(a.scale));
    }
    store_columns<F32, AL>(out, c0 + 256 * j, a.H, s[j], a.err);
  }
}

// Packs of a slice's columns a lane: with 4, up to 1024 columns a warp.
inline int slice_packs(int64_t H, bool aligned) { return !aligned || H <= 1024 ? 1 : 2; }

struct Room {  // the workspace of a gradient
  size_t a, b, done, part, all;
  int32_t slots;
};

inline Room room_of(int64_t T, int64_t H) {
  Room r{};
  r.slots = static_cast<int32_t>(T / RUN + 1);
  r.a = 0;
  r.b = carved(T * sizeof(Entry));
  r.done = 2 * r.b;
  r.part = r.done + carved(static_cast<size_t>(r.slots) * ((H + 255) / 256 + GATHER_WARPS) * sizeof(int32_t));
  r.all = r.part + carved(2 * static_cast<size_t>(r.slots) * ((H + 7) / 8 * 8) * sizeof(float));
  return r;
}

// A kernel that may start while the one before it on the stream ends (it waits for it by itself).
template <class A>
inline rlk_status launch_after(void (*kernel)(A), const A& a, dim3 grid, int threads, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? RLK_OK : RLK_ERR_CUDA;
}

inline rlk_status check_shard(int64_t rows, int64_t start, int64_t V_true) {
  if (rows <= 0 || start < 0 || V_true <= 0) return RLK_ERR_INVALID_ARG;
  if (rows > RLK_MAX_VOCAB || V_true > RLK_MAX_VOCAB || start > RLK_MAX_VOCAB) return RLK_ERR_UNSUPPORTED;
  return RLK_OK;
}

inline bool scale_ok(double scale) { return scale >= -3.4028234663852886e38 && scale <= 3.4028234663852886e38; }

}  // namespace
}  // namespace rlk

using namespace rlk;

extern "C" {

rlk_status rlk_embedding_fwd(const void* table, int32_t dtype, int64_t V_local, int64_t H, int64_t ld, int64_t vocab_start,
                             int64_t V_true, const int64_t* ids, int64_t T, double scale, void* out, int32_t out_dtype,
                             int64_t out_ld, int32_t* err_flag, void* stream) {
  rlk_status st = check_shard(V_local, vocab_start, V_true);
  if (st == RLK_OK) st = check_rows(table, dtype, V_local, H, ld);
  if (st == RLK_OK) st = check_pair(dtype, out_dtype);
  if (st == RLK_OK) st = check_rows(out, out_dtype, T, H, out_ld);
  if (st != RLK_OK) return st;
  if (!scale_ok(scale) || (T > 0 && !ids)) return RLK_ERR_INVALID_ARG;
  const RowSpan in{table, V_local, H, ld, dtype_bytes(dtype)}, to{out, T, H, out_ld, dtype_bytes(out_dtype)};
  if (!rows_apart(in, to)) return RLK_ERR_INVALID_ARG;
  if (T == 0) return RLK_OK;
  const LookupArgs a{table, out, ids, T, ld, out_ld, static_cast<int32_t>(H), static_cast<float>(scale),
                     Shard{vocab_start, V_local, V_true, err_flag}};
  const bool al = whole_packs(table, V_local, H, ld, in.eb) && whole_packs(out, T, H, out_ld, to.eb);
  return with_pair(dtype, out_dtype, [&](auto e, auto o) {
    const auto s = static_cast<cudaStream_t>(stream);
    if (al) lookup_kernel<decltype(e), decltype(o), true><<<static_cast<unsigned>(T), 256, 0, s>>>(a);
    else lookup_kernel<decltype(e), decltype(o), false><<<static_cast<unsigned>(T), 256, 0, s>>>(a);
    return launched();
  });
}

size_t rlk_embedding_bwd_workspace(int64_t T, int64_t H) {
  return T <= 0 || H <= 0 ? 0 : room_of(T, H).all;
}

rlk_status rlk_embedding_bwd(const void* dout, int32_t dtype, int64_t T, int64_t H, int64_t ld, const int64_t* ids,
                             int64_t V_local, int64_t vocab_start, int64_t V_true, double scale, float* dW,
                             int32_t accumulate, int32_t* err_flag, void* workspace, size_t workspace_bytes,
                             void* stream) {
  rlk_status st = check_shard(V_local, vocab_start, V_true);
  if (st == RLK_OK) st = check_rows(dout, dtype, T, H, ld);
  if (st != RLK_OK) return st;
  if (!scale_ok(scale) || (T > 0 && !ids) || !dW || !on_boundary(dW, 4)) return RLK_ERR_INVALID_ARG;
  const RowSpan in{dout, T, H, ld, dtype_bytes(dtype)}, to{dW, V_local, H, H, 4};
  if (!rows_apart(in, to)) return RLK_ERR_INVALID_ARG;
  const auto s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (!accumulate && cudaMemsetAsync(dW, 0, static_cast<size_t>(V_local) * H * sizeof(float), s) != cudaSuccess)
      return RLK_ERR_CUDA;
    return RLK_OK;
  }
  const Room r = room_of(T, H);
  if (!workspace || !on_boundary(workspace, 256) || workspace_bytes < r.all) return RLK_ERR_WORKSPACE;
  const bool al = whole_packs(dout, T, H, ld, in.eb) && on_boundary(dW, 16);
  const int packs = slice_packs(H, al);
  const int warps = static_cast<int>(std::min<int64_t>(GATHER_WARPS, (H + 256 * packs - 1) / (256 * packs)));
  const int blocks = static_cast<int>((H + 256 * packs * warps - 1) / (256 * packs * warps)), slices = blocks * warps;
  char* ws = static_cast<char*>(workspace);
  SortArgs q{ids, reinterpret_cast<Entry*>(ws + r.a), reinterpret_cast<Entry*>(ws + r.b), static_cast<int32_t>(T), 0, 0,
             Shard{vocab_start, V_local, V_true, err_flag}, reinterpret_cast<int32_t*>(ws + r.done), r.slots * slices,
             dW, accumulate ? 0 : V_local * H};
  while (V_local >> q.bits) ++q.bits;  // rows and the mark behind them: 0 .. V_local
  q.passes = (q.bits + 8) / 9;

  // one cluster sorts, the others (if any) zero dW
  int ctas = 1;
  while (ctas < SORT_CTAS && T > 2 * SORT_THREADS * ctas) ctas *= 2;
  int64_t zero = accumulate ? 0 : (V_local * H + 16 * 4 * SORT_THREADS - 1) / (16 * 4 * SORT_THREADS);
  if (zero > 456) zero = 456;
  zero = (zero + ctas - 1) / ctas * ctas;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas + zero));
  cfg.blockDim = dim3(SORT_THREADS);
  cfg.dynamicSmemBytes = sizeof(SortSmem);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const int64_t groups = (T + 32 * SORT_WARPS * ctas - 1) / (32 * SORT_WARPS * ctas);
  const auto sort = groups <= 1 ? sort_tokens_kernel<1> : groups <= 4 ? sort_tokens_kernel<4> : sort_tokens_kernel<0>;
  if (cudaFuncSetAttribute(sort, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortSmem)) != cudaSuccess ||
      cudaFuncSetAttribute(sort, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return RLK_ERR_CUDA;
  if (cudaLaunchKernelEx(&cfg, sort, q) != cudaSuccess) return RLK_ERR_CUDA;

  const GatherArgs g{q.passes & 1 ? q.a : q.b, dout, dW, ld, q.T, static_cast<int32_t>(H), static_cast<int32_t>(V_local),
                     static_cast<float>(scale), accumulate != 0, reinterpret_cast<float*>(ws + r.part), q.done, r.slots,
                     err_flag};
  return with_type(dtype, [&](auto e) {
    using E = decltype(e);
    const auto kernel = !al ? gather_kernel<E, false, 1>
                        : packs == 1 ? gather_kernel<E, true, 1> : gather_kernel<E, true, 2>;
    return launch_after(kernel, g, dim3(static_cast<unsigned>(T), blocks), 32 * warps, s);
  });
}

}  // extern "C"
