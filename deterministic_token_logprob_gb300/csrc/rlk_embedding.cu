// rlk_embedding.cu -- rows of a table by token, and the table's gradient by sorted tokens.
//
//   out[t] = s E[id_t],   dE[v] (+)= s sum_{t : id_t = v} dout[t]
//
// The gradient sorts (token, position) stably, so that a token's positions stand side by side in
// ascending order, and adds their rows in runs of 32 positions of that token: a run in ascending order,
// then the runs in ascending order. What a row of dE holds depends on that token's rows alone, not on
// which other tokens the batch or the shard has.
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
constexpr int SORT_THREADS = 1024;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_BINS = 512;  // 9 bits at most at a time: two passes for up to 2^18 rows
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
  uint32_t total[SORT_BINS];              // of this CTA, read by the cluster
  uint32_t base[SORT_BINS];               // where this CTA's entries of a digit start
  uint32_t warp_sum[SORT_WARPS];
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.relaxed.cluster.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

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

__device__ void sort_tokens(const SortArgs& a, SortSmem& m) {
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
    // a digit beyond the bins: no entry
    const auto digit_of = [&](int32_t t, Entry* e) {
      if (t >= last) return 0xFFFFFFFFu;
      *e = sort_entry(a, src, t);
      return (e->row >> shift) & static_cast<uint32_t>(bins - 1);
    };
    for (int b = lane; b < bins; b += 32) mine[b] = 0;
    __syncwarp();
    for (int32_t t = first; t < last; t += 32) {
      Entry e;
      const uint32_t d = digit_of(t + lane, &e);
      const uint32_t like = __match_any_sync(kFullWarp, d);
      if (d < static_cast<uint32_t>(bins) && lane == __ffs(like) - 1) mine[d] += __popc(like);
      __syncwarp();
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += SORT_THREADS) {
      uint32_t run = 0;
      for (int w = 0; w < SORT_WARPS; ++w) {
        const uint32_t c = m.count[w][b];
        m.count[w][b] = run;
        run += c;
      }
      m.total[b] = run;
    }
    cluster_sync();
    // all entries of lower digits, and those of this digit in CTAs before this one
    uint32_t before = 0, all = 0;
    const int b = threadIdx.x;
    if (b < bins) {
      const uint32_t at = smem_u32(&m.total[b]);
      for (uint32_t c = 0; c < ctas; ++c) {
        const uint32_t v = ld_cluster_u32(map_to_cta(at, c));
        all += v;
        if (c < rank) before += v;
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
    uint32_t lower = sum - all;
    for (int w = 0; w < warp; ++w) lower += m.warp_sum[w];
    if (b < bins) m.base[b] = lower + before;
    __syncthreads();
    for (int32_t t = first; t < last; t += 32) {
      Entry e;
      const uint32_t d = digit_of(t + lane, &e);
      const uint32_t like = __match_any_sync(kFullWarp, d);
      const bool on = d < static_cast<uint32_t>(bins);
      const uint32_t at = on ? m.base[d] + mine[d] + __popc(like & ((1u << lane) - 1)) : 0;
      __syncwarp();
      if (on && lane == __ffs(like) - 1) mine[d] += __popc(like);
      __syncwarp();
      if (on && dbg_ok(at < static_cast<uint32_t>(a.T), a.shard.err)) dst[at] = e;
    }
    __threadfence();
    cluster_sync();  // the entries, and the totals, are through before the next pass (and before the CTA ends)
  }
}

__global__ void __launch_bounds__(SORT_THREADS) sort_tokens_kernel(const SortArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  const uint32_t ctas = cluster_size();
  if (blockIdx.x < ctas) {
    sort_tokens(a, *reinterpret_cast<SortSmem*>(dyn));
    return;
  }
  // every other cluster: zeros into dW, whole vectors between its first and last boundary
  const int64_t i0 = static_cast<int64_t>(blockIdx.x - ctas) * SORT_THREADS + threadIdx.x;
  const int64_t n = static_cast<int64_t>(gridDim.x - ctas) * SORT_THREADS;
  const int64_t head = min(a.n_zero, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(a.dW) & 15)) & 15) / 4);
  const int64_t vecs = (a.n_zero - head) / 4;
  uint4* v = reinterpret_cast<uint4*>(a.dW + head);
  for (int64_t i = i0; i < vecs; i += n) v[i] = make_uint4(0, 0, 0, 0);
  if (i0 < head) a.dW[i0] = 0.f;
  if (i0 < a.n_zero - head - 4 * vecs) a.dW[head + 4 * vecs + i0] = 0.f;
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
  int32_t* done;        // [slots][column blocks]: runs of such a token that are through
  int32_t slots;
  int32_t* err;
};

__device__ __forceinline__ uint32_t row_at(const GatherArgs& a, int32_t p) {
  return dbg_ok(p >= 0 && p < a.T, a.err) ? a.sorted[p].row : 0xFFFFFFFFu;
}

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

template <class E, bool AL>
__global__ void __launch_bounds__(256) gather_kernel(const GatherArgs a) {
  __shared__ int32_t last;
  const int lane = threadIdx.x & 31;
  const int32_t p = static_cast<int32_t>(blockIdx.x);
  const uint32_t row = row_at(a, p);
  if (row >= static_cast<uint32_t>(a.rows)) return;
  // does a run start at p?
  const int32_t back = p - 1 - lane;
  const uint32_t same = __ballot_sync(kFullWarp, back >= 0 && row_at(a, back < 0 ? 0 : back) == row);
  int32_t start = p;
  if (same & 1u) {
    if (same != kFullWarp) return;
    start = first_not_below(a, row, 0, p - 32, lane);
    if ((p - start) % RUN != 0) return;
  }
  const int32_t next = p + 1 + lane;
  const uint32_t more = __ballot_sync(kFullWarp, next < a.T && row_at(a, next < a.T ? next : p) == row);
  const int n = min(RUN, ~more == 0 ? RUN : __ffs(~more));  // length of the run
  const bool alone = start == p && !(more >> 31 && n == RUN);
  const uint32_t mine = lane < n ? a.sorted[p + lane].t : 0;
  const int width = (a.H + 7) / 8 * 8;
  const int c = 8 * static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x);
  const bool on = c < a.H;
  F32x2 s[4] = {};
  for (int i = 0; i < n; ++i) {
    const uint32_t t = __shfl_sync(kFullWarp, mine, i);
    if (!on) continue;
    F32x2 v[4];
    unpack(load_columns<E, AL>(static_cast<const typename E::bits*>(a.dout) + static_cast<int64_t>(t) * a.ld, c, a.H, a.err), v);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = add2(s[j], v[j]);
  }
  if (!alone) {
    // leave the run's sum; the CTA that is through last adds them up
    const int32_t seg = (start + RUN - 1) / RUN;  // a token of several runs starts with a whole one
    const int32_t slot = n == RUN ? (p + RUN - 1) / RUN : a.slots + seg;
    const bool ok = dbg_ok(slot < 2 * a.slots && seg < a.slots, a.err);
    if (on && ok) {
      store_columns<F32, true>(reinterpret_cast<uint32_t*>(a.part) + static_cast<int64_t>(slot) * width, c, width, s, a.err);
    }
    const int32_t end = more >> 31 && n == RUN ? first_not_below(a, row + 1, p + RUN, a.T, lane) : p + n;
    const int32_t runs = (end - start + RUN - 1) / RUN;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = ok ? atomicAdd(&a.done[seg * gridDim.y + blockIdx.y], 1) == runs - 1 : 0;
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (!on) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = 0;
    for (int i = 0; i < runs; ++i) {
      const int32_t q = start + i * RUN;
      const int32_t from = q + RUN <= end ? (q + RUN - 1) / RUN : a.slots + seg;
      const float4* at = reinterpret_cast<const float4*>(a.part + static_cast<int64_t>(from) * width + c);
      const float4 x = __ldcg(at), y = __ldcg(at + 1);
      const F32x2 v[4] = {pack_f32x2(x.x, x.y), pack_f32x2(x.z, x.w), pack_f32x2(y.x, y.y), pack_f32x2(y.z, y.w)};
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = add2(s[j], v[j]);
    }
  }
  if (!on) return;
  auto* out = reinterpret_cast<uint32_t*>(a.dW) + static_cast<int64_t>(row) * a.H;
  F32x2 old[4] = {};
  if (a.add) unpack(load_columns<F32, AL>(out, c, a.H, a.err), old);
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] = a.add ? fma2(s[j], both(a.scale), old[j]) : mul2(s[j], both(a.scale));
  store_columns<F32, AL>(out, c, a.H, s, a.err);
}

struct Room {  // the workspace of a gradient
  size_t a, b, done, part, all;
  int32_t slots, blocks, threads;
};

inline Room room_of(int64_t T, int64_t H) {
  Room r{};
  r.threads = static_cast<int32_t>(H >= 2048 ? 256 : (H + 255) / 256 * 32);
  r.blocks = static_cast<int32_t>((H + 8 * r.threads - 1) / (8 * r.threads));
  r.slots = static_cast<int32_t>(T / RUN + 1);
  r.a = 0;
  r.b = carved(T * sizeof(Entry));
  r.done = 2 * r.b;
  r.part = r.done + carved(static_cast<size_t>(r.slots) * r.blocks * sizeof(int32_t));
  r.all = r.part + carved(2 * static_cast<size_t>(r.slots) * ((H + 7) / 8 * 8) * sizeof(float));
  return r;
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
  char* ws = static_cast<char*>(workspace);
  SortArgs q{ids, reinterpret_cast<Entry*>(ws + r.a), reinterpret_cast<Entry*>(ws + r.b), static_cast<int32_t>(T), 0, 0,
             Shard{vocab_start, V_local, V_true, err_flag}, reinterpret_cast<int32_t*>(ws + r.done), r.slots * r.blocks,
             dW, accumulate ? 0 : V_local * H};
  while (V_local >> q.bits) ++q.bits;  // rows and the mark behind them: 0 .. V_local
  q.passes = (q.bits + 8) / 9;

  // one cluster sorts, the others (if any) zero dW
  const int ctas = T <= 4096 ? 1 : 8;
  int64_t zero = accumulate ? 0 : (V_local * H + 16 * 4 * SORT_THREADS - 1) / (16 * 4 * SORT_THREADS);
  if (zero > 152) zero = 152;
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
  if (cudaFuncSetAttribute(sort_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortSmem)) != cudaSuccess)
    return RLK_ERR_CUDA;
  if (cudaLaunchKernelEx(&cfg, sort_tokens_kernel, q) != cudaSuccess) return RLK_ERR_CUDA;

  const GatherArgs g{q.passes & 1 ? q.a : q.b, dout, dW, ld, q.T, static_cast<int32_t>(H), static_cast<int32_t>(V_local),
                     static_cast<float>(scale), accumulate != 0, reinterpret_cast<float*>(ws + r.part), q.done, r.slots,
                     err_flag};
  const bool al = whole_packs(dout, T, H, ld, in.eb) && on_boundary(dW, 16);
  return with_type(dtype, [&](auto e) {
    const dim3 grid(static_cast<unsigned>(T), r.blocks);
    if (al) gather_kernel<decltype(e), true><<<grid, r.threads, 0, s>>>(g);
    else gather_kernel<decltype(e), false><<<grid, r.threads, 0, s>>>(g);
    return launched();
  });
}

}  // extern "C"
