// rlk_embedding.cu -- rows of a table by token, and the table's gradient by sorted tokens.
//
//   out[t] = s E[id_t],   dE[v] (+)= s sum_{t : id_t = v} dout[t]
//
// The gradient sorts (token, position) stably, so that a token's positions stand side by side in
// ascending order, and adds their rows in a fixed order: runs of 16 positions of that token, groups of 8
// runs, all groups, each in ascending order. What a row of dE holds depends on that token's rows alone,
// not on which other tokens the batch or the shard has.
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
  int32_t H, packs;   // of a row
  int32_t each;       // rows a CTA
  uint32_t magic;     // ceil(2^20 / packs): q / packs = q magic >> 20 for q < 256, where a CTA has several rows
  float scale;
  Shard shard;
};

// A CTA takes a row, or as many short ones as have 256 packs. Bound by HBM; few registers and full occupancy hide the two loads
// (token, then row) best: 8192 rows of 4096 in bf16 take 17.1 us (7.8 TB/s: a part is still in L2); with four packs a thread on their way, and half the
// warps, 19.3. 16384 rows of 2048 take 16.2 us with two packs a thread of 128, with one of 256 21.6; 32768 of 512 9.5 us, where a
// CTA a row took 10.2; 8192 of 1001, at any alignment, 11.1 us element by element and 18.4 by packs.
template <class E, class O, bool AL, int THREADS>
__global__ void __launch_bounds__(THREADS) lookup_kernel(const LookupArgs a) {
  const int i = a.each == 1 ? 0 : static_cast<int>(threadIdx.x * a.magic >> 20);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * a.each + i;
  if (i >= a.each || t >= a.T) return;
  const int32_t r = a.shard.row_of(a.ids[t]);
  const auto* row = static_cast<const typename E::bits*>(a.table) + static_cast<int64_t>(r < 0 ? 0 : r) * a.ld;
  auto* out = static_cast<typename O::bits*>(a.out) + t * a.out_ld;
  const int first = static_cast<int>(threadIdx.x) - i * a.packs;
  if constexpr (AL) {
    for (int c = 8 * first; c < a.H; c += 8 * THREADS) {  // once for a short row: 8 packs <= 8 THREADS
      F32x2 v[4];
      if (r >= 0) {
        unpack(load_columns<E, true>(row, c, a.H, a.shard.err), v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], both(a.scale));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = both(r == -2 ? quiet_nan() : 0.f);
      }
      store_columns<O, true>(out, c, a.H, v, a.shard.err);
    }
  } else {  // element by element: packs that lie anywhere touch each sector eight times
    const int step = a.each == 1 ? THREADS : a.packs;
    const float none = r == -2 ? quiet_nan() : 0.f;
#pragma unroll 8
    for (int c = first; c < a.H; c += step)
      if (dbg_ok(c >= 0 && c < a.H, a.shard.err)) out[c] = O::from_f32(r >= 0 ? __fmul_rn(E::to_f32(row[c]), a.scale) : none);
  }
}

// ---------------------------------------------------------------------------
// sorting tokens
// ---------------------------------------------------------------------------
// A radix sort from the low digits up, by one cluster: warp w of the cluster's W owns the w-th run of
// positions, counts its digits, gets from the counts of all warps where each of its digits goes, and goes through
// its run again to put the entries there. Runs and lanes are in ascending order of position, so that the sort is
// stable and its result unique, whatever the cluster's size. A token without a row here sorts behind the last row. 16384 tokens take
// 16.5 us (ncu), 1 of them until every CTA of the cluster is known to have started.
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_BINS = 512;  // 9 bits at most at a time: two passes for up to 2^18 - 1 rows (and the mark behind them)
constexpr int SORT_CTAS = 16;
constexpr int RUN = 16;         // positions of one token that are added in one go
constexpr int GROUP = 8;        // runs

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
  uint4* runs;         // [T]: those of tokens of several runs from the front, the others from the back
  int32_t* n_runs;     // how many of each
};

struct alignas(16) SortSmem {
  uint32_t count[SORT_WARPS][SORT_BINS];  // digits of each warp; then how many stand before the warp in this CTA
  uint32_t lanes[SORT_WARPS][SORT_BINS];  // of a group's digits
  uint32_t total[SORT_CTAS][SORT_BINS];   // of each CTA of the cluster, which puts its own into all of them
  uint32_t base[SORT_BINS];               // where this CTA's entries of a digit start
  uint32_t warp_sum[SORT_WARPS];
};

__device__ __forceinline__ void st_cluster_u32x4(uint32_t addr, uint4 v) {
  asm volatile("st.relaxed.cluster.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Entries t, t + 32, ... below last, all of them on their way at once.
template <int N>
__device__ __forceinline__ void read_entries(const SortArgs& a, const Entry* src, int32_t t, int32_t last, Entry (&e)[N]) {
  if (src) {
#pragma unroll
    for (int g = 0; g < N; ++g)
      if (t + 32 * g < last) {
        const uint2 v = __ldcg(reinterpret_cast<const uint2*>(src + t + 32 * g));
        e[g] = Entry{v.x, v.y};
      }
    return;
  }
  int64_t id[N];
#pragma unroll
  for (int g = 0; g < N; ++g) id[g] = t + 32 * g < last ? a.ids[t + 32 * g] : -1;
#pragma unroll
  for (int g = 0; g < N; ++g) {
    const int32_t r = a.shard.row_of(id[g]);
    e[g] = Entry{r < 0 ? static_cast<uint32_t>(a.shard.rows) : static_cast<uint32_t>(r), static_cast<uint32_t>(t + 32 * g)};
  }
}

// A warp's positions go by in groups of 32, KEPT of them read at a time. ALL: those are all that a warp has, and they stay in
// registers between the two ways through them.
template <int KEPT, bool ALL>
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
  uint32_t *mine = m.count[warp], *same = m.lanes[warp];

  if (ctas > 1) cluster_arrive();
  for (int i = rank * SORT_THREADS + threadIdx.x; i < a.n_done; i += ctas * SORT_THREADS) a.done[i] = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    const Entry* src = pass == 0 ? nullptr : pass & 1 ? a.a : a.b;
    Entry* dst = pass & 1 ? a.b : a.a;
    const int shift = pass * each;
    Entry kept[KEPT];
    // f(entry, digit, whether there is an entry) of each group
    const auto groups = [&](bool again, auto f) {
      for (int32_t t0 = first; t0 < last; t0 += 32 * KEPT) {
        if (!ALL || !again) read_entries<KEPT>(a, src, t0 + lane, last, kept);
#pragma unroll
        for (int g = 0; g < KEPT; ++g) {
          if (t0 + 32 * g >= last) break;
          const bool on = t0 + 32 * g + lane < last;
          f(kept[g], on ? (kept[g].row >> shift) & static_cast<uint32_t>(bins - 1) : 0, on);
        }
        if (ALL) break;
      }
    };
    for (int b = lane; b < bins; b += 32) mine[b] = same[b] = 0;
    __syncwarp();
    groups(false, [&](const Entry&, uint32_t d, bool on) {
      if (on) atomicAdd(&mine[d], 1u);
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
      m.total[rank][b] = run;
    }
    __syncthreads();
    if (pass == 0 && ctas > 1) cluster_wait();  // every CTA has started: its shared memory may be written
    if (warp < static_cast<int>(ctas) && warp != static_cast<int>(rank)) {  // a warp for each other CTA
      const uint32_t to = map_to_cta(smem_u32(m.total[rank]), warp);
      for (int i = 4 * lane; i < bins; i += 128) st_cluster_u32x4(to + 4 * i, *reinterpret_cast<const uint4*>(&m.total[rank][i]));
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
    groups(true, [&](const Entry& e, uint32_t d, bool on) {
      if (on) atomicOr(&same[d], 1u << lane);  // the lanes of each digit
      __syncwarp();
      const uint32_t like = on ? same[d] : 0, before = like & ((1u << lane) - 1);
      const uint32_t at = on ? m.base[d] + mine[d] + __popc(before) : 0;
      __syncwarp();
      if (on && before == 0) {
        mine[d] += __popc(like);
        same[d] = 0;
      }
      __syncwarp();
      if (on && dbg_ok(at < static_cast<uint32_t>(a.T), a.shard.err)) dst[at] = e;
    });
    cluster_sync();  // the entries, and the totals, are through before the next pass (and before the CTA ends)
  }
}

// The first position in [lo, hi] from which on all rows are >= row (hi is such a one), by a whole warp.
template <class At>
__device__ __forceinline__ int32_t first_not_below(uint32_t row, int32_t lo, int32_t hi, int lane, const At& row_at) {
  while (lo < hi) {
    const int32_t step = (hi - lo + 31) / 32, base = lo;
    const int64_t q = static_cast<int64_t>(lo) + static_cast<int64_t>(lane) * step;
    const bool yes = q >= hi || row_at(static_cast<int32_t>(q)) >= row;
    const uint32_t m = __ballot_sync(kFullWarp, yes);
    const int f = m ? __ffs(m) - 1 : 32;
    if (f < 32) hi = static_cast<int32_t>(min(static_cast<int64_t>(hi), static_cast<int64_t>(base) + static_cast<int64_t>(f) * step));
    if (f > 0) lo = static_cast<int32_t>(min(static_cast<int64_t>(hi), static_cast<int64_t>(base) + static_cast<int64_t>(f - 1) * step + 1));
  }
  return hi;
}

// A run: its first position and whether it is the token's only one, the token's first position, row, and the run's first t.
__device__ __forceinline__ uint4 pack_run(int32_t p, int32_t start, bool alone, uint32_t row, uint32_t t) {
  return make_uint4(static_cast<uint32_t>(p) | (alone ? 0x80000000u : 0u), static_cast<uint32_t>(start), row, t);
}

// Lists the runs of the sorted positions: a warp goes through as many as it sorted, 4 groups of 32 at a time. The list's order
// is whatever the counters give: which warp adds up which run changes nothing. Tokens of several runs come first, so that the
// chain of sums that they end in does not come last.
__device__ __forceinline__ void list_runs(const SortArgs& a, const Entry* sorted) {
  constexpr int G = 4;
  constexpr uint32_t kNone = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(cluster_size()) * SORT_WARPS;
  const int32_t per = static_cast<int32_t>((a.T + 32 * warps - 1) / (32 * warps)) * 32;
  const int64_t lo = (static_cast<int64_t>(cluster_ctarank()) * SORT_WARPS + (threadIdx.x >> 5)) * per;
  const int32_t first = static_cast<int32_t>(min(static_cast<int64_t>(a.T), lo));
  const int32_t last = static_cast<int32_t>(min(static_cast<int64_t>(a.T), lo + per));
  const auto row_at = [&](int32_t p) { return __ldcg(&sorted[p].row); };
  int32_t start0 = -1;           // where the token of the position before the group starts; -1: not known
  uint32_t row0 = kNone;         // its row
  if (first < last && first > 0) row0 = row_at(first - 1);
  for (int32_t p0 = first; p0 < last; p0 += 32 * G) {
    Entry e[G];
    uint32_t far[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int32_t p = p0 + 32 * g + lane;
      const uint2 v = p < last ? __ldcg(reinterpret_cast<const uint2*>(sorted + p)) : make_uint2(kNone, 0);
      e[g] = Entry{v.x, v.y};
      far[g] = p < last && p + RUN < a.T ? row_at(p + RUN) : kNone;
    }
    int32_t start[G];
    uint32_t here[G], alone[G];
    int several = 0, single = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int32_t q0 = p0 + 32 * g;
      uint32_t before = __shfl_up_sync(kFullWarp, e[g].row, 1);
      if (lane == 0) before = row0;
      const uint32_t heads = __ballot_sync(kFullWarp, e[g].row != before);
      const uint32_t mine = heads & (0xFFFFFFFFu >> (31 - lane));  // heads at or before this lane
      if (!(heads & 1u) && start0 < 0) start0 = first_not_below(row0, 0, q0 - 1, lane, row_at);
      start[g] = mine ? q0 + 31 - __clz(mine) : start0;
      here[g] = __ballot_sync(kFullWarp, e[g].row < static_cast<uint32_t>(a.shard.rows) && (q0 + lane - start[g]) % RUN == 0);
      alone[g] = here[g] & __ballot_sync(kFullWarp, start[g] == q0 + lane && far[g] != e[g].row);
      several += __popc(here[g] & ~alone[g]);
      single += __popc(alone[g]);
      row0 = __shfl_sync(kFullWarp, e[g].row, 31);
      start0 = __shfl_sync(kFullWarp, start[g], 31);
    }
    int32_t at = 0;
    if (lane < 2 && (lane ? single : several)) at = atomicAdd(&a.n_runs[lane], lane ? single : several);
    int32_t front = __shfl_sync(kFullWarp, at, 0), back = a.T - 1 - __shfl_sync(kFullWarp, at, 1);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int32_t p = p0 + 32 * g + lane;
      const uint32_t below = (1u << lane) - 1;
      const bool one = alone[g] >> lane & 1u;
      const int32_t to = one ? back - __popc(alone[g] & below) : front + __popc(here[g] & ~alone[g] & below);
      if ((here[g] >> lane & 1u) && dbg_ok(to >= 0 && to < a.T, a.shard.err)) a.runs[to] = pack_run(p, start[g], one, e[g].row, e[g].t);
      front += __popc(here[g] & ~alone[g]);
      back -= __popc(alone[g]);
    }
  }
}

template <int KEPT, bool ALL>
__global__ void __launch_bounds__(SORT_THREADS) sort_tokens_kernel(const SortArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x < 2) a.n_runs[threadIdx.x] = 0;  // the cluster's barriers stand before its first use
  sort_tokens<KEPT, ALL>(a, *reinterpret_cast<SortSmem*>(dyn));
  list_runs(a, a.passes & 1 ? a.a : a.b);
}

// ---------------------------------------------------------------------------
// adding rows
// ---------------------------------------------------------------------------
struct GatherArgs {
  const Entry* sorted;  // [T]
  const uint4* runs;
  const int32_t* n_runs;
  const int64_t* ids;   // of few tokens, which are not sorted
  Shard shard;
  const void* dout;
  float* dW;
  int64_t ld;
  int32_t T, H, rows;
  float scale;
  bool add;
  float* part;          // [2 slots][H rounded up to 8]: sums of the runs of tokens of more than one run
  int32_t* done;        // [3 slots][slices]: runs of such a group, and groups of such a token, that are through
  int32_t slots, slices;
  int32_t ahead;        // rows of dout that a CTA asks for while the tokens are sorted
  int32_t zero_per;     // rows that a CTA behind those of the runs zeroes, where dW is new (0: it is not)
  int32_t* err;
};

constexpr int GATHER_THREADS = 256;
constexpr int ZERO_ROWS = 2048;  // zero_per at most
// 16-bit rows: up to so many warps of a pack a lane, each has 8 rows in flight, else two packs and 2 rows. Few warps wait for the longest chain
// of rows (2048 rows of 2048 added to dW, tokens as in text: 19.0 us for 22.7; spread evenly 16.9 for 16.2), many for the memory (16384
// rows: 44.6 us for 51.7, evenly 65.4 for 74.5). fp32 rows have a pack a lane and 4 rows (8192 rows of 2048: 31.5 us, two and 2 37.5).
constexpr int64_t FEW_WARPS = 16384;
// While one cluster sorts, the first CTAs of the next kernel ask for dout, if L2 holds that much besides the rows of dW (16384 rows of
// 2048 in bf16, 67 MB: 44.6 us for 46.9; of 512 CTAs instead of 128 8192 rows of 4096 take 48.3 us for 46.1). These figures, and those
// above, are from before the sort's CTAs waited for one another's start: 45.4 us now, and 47.8.
constexpr int AHEAD_CTAS = 128;
constexpr int64_t AHEAD_BYTES = 80 << 20;

// Zeros into the rows r0 .. r0 + n of dW that are not met, by a CTA.
template <bool AL>
__device__ __forceinline__ void zero_rows(const GatherArgs& a, int32_t r0, int32_t n, const uint8_t* met) {
  const int threads = blockDim.x;
  // tx threads a row, of threads / tx (1 at least) rows at a time; threads beyond them have none
  int tx = 1;
  while (2 * tx <= threads && tx * 4 < a.H) tx *= 2;
  const int x = threadIdx.x % tx, ty = threads / tx;
  for (int i = threadIdx.x / tx; i < n && static_cast<int>(threadIdx.x) < tx * ty; i += ty) {
    if (met[i]) continue;
    float* row = a.dW + static_cast<int64_t>(r0 + i) * a.H;
    if constexpr (AL) {
#pragma unroll 4
      for (int c = 4 * x; c < a.H; c += 4 * tx) *reinterpret_cast<float4*>(row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
#pragma unroll 4
      for (int c = x; c < a.H; c += tx) row[c] = 0.f;
    }
  }
}

// The same by the sorted tokens.
template <bool AL>
__device__ __forceinline__ void zero_absent_rows(const GatherArgs& a, int32_t z, uint8_t* met) {
  const int32_t r0 = z * a.zero_per, n = min(a.zero_per, a.rows - r0), lane = threadIdx.x & 31;
  const auto row_at = [&](int32_t q) { return a.sorted[q].row; };
  const int32_t lo = first_not_below(static_cast<uint32_t>(r0), 0, a.T, lane, row_at);
  const int32_t hi = first_not_below(static_cast<uint32_t>(r0 + n), lo, a.T, lane, row_at);
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int32_t from = lo, to = hi;  // the row's first entry is in [from, to]
    while (from < to) {
      const int32_t mid = (from + to) / 2;
      if (row_at(mid) < static_cast<uint32_t>(r0 + i)) from = mid + 1;
      else to = mid;
    }
    met[i] = from < hi && row_at(from) == static_cast<uint32_t>(r0 + i);
  }
  __syncthreads();
  zero_rows<AL>(a, r0, n, met);
}

// s += n rows of dout, row at(i) as the i-th, in C packs of a thread 256 columns apart from column c0 on.
template <class E, bool AL, int C, int U, class At>  // U rows in flight
__device__ __forceinline__ void add_rows(const GatherArgs& a, int n, int c0, F32x2 (&s)[C][4], const At& at) {
  for (int i = 0; i < n; i += U) {
    Pack<E> k[U][C];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const auto* row = static_cast<const typename E::bits*>(a.dout) + static_cast<int64_t>(at(min(i + u, n - 1))) * a.ld;
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (i + u < n && c0 + 256 * j < a.H) k[u][j] = load_columns<E, AL>(row, c0 + 256 * j, a.H, a.err);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= n) break;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        F32x2 v[4];
        unpack(k[u][j], v);
#pragma unroll
        for (int q = 0; q < 4; ++q) s[j][q] = add2(s[j][q], v[q]);
      }
    }
  }
}

// Writes a pack of a row of dW; old: what it held, where the gradient is added.
template <bool AL>
__device__ __forceinline__ void put_row(const GatherArgs& a, uint32_t* out, int c0, F32x2 (&s)[4], const Pack<F32>& old) {
  F32x2 v[4];
  unpack(old, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = a.add ? fma2(s[i], both(a.scale), v[i]) : mul2(s[i], both(a.scale));
  store_columns<F32, AL>(out, c0, a.H, s, a.err);
}

// Leaves a warp's part of a sum in its slot and counts it; whether it was the last of `parts`.
template <int C>
__device__ __forceinline__ bool leave_part(const GatherArgs& a, int32_t slot, int32_t counter, int32_t parts, int slice, int c0,
                                           const F32x2 (&s)[C][4]) {
  const int width = (a.H + 7) / 8 * 8;
  const bool ok = dbg_ok(slot >= 0 && slot < 2 * a.slots && counter >= 0 && counter < 3 * a.slots, a.err);
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (ok && c0 + 256 * j < a.H)
      store_columns<F32, true>(reinterpret_cast<uint32_t*>(a.part) + static_cast<int64_t>(slot) * width, c0 + 256 * j, width, s[j], a.err);
  __threadfence();
  __syncwarp();
  int32_t before = -1;
  if ((threadIdx.x & 31) == 0 && ok) before = atomicAdd(&a.done[static_cast<int64_t>(counter) * a.slices + slice], 1);
  const bool last = __shfl_sync(kFullWarp, before, 0) == parts - 1;
  if (last) __threadfence();
  return last;
}

// The runs of a token of several: a whole run's slot is the multiple of RUN that it holds (over RUN), the last and shorter
// one's follows from the token's first position (such a token starts with a whole run).
struct Token {
  int32_t start, end;
  __device__ __forceinline__ int32_t first() const { return (start + RUN - 1) / RUN; }
  __device__ __forceinline__ int32_t slot(const GatherArgs& a, int32_t run) const {
    const int32_t q = start + run * RUN;
    return q + RUN <= end ? (q + RUN - 1) / RUN : a.slots + first();
  }
};

// s = the sum of runs lo, lo + each, ... of a token below hi, in that order
template <int C>
__device__ __forceinline__ void add_parts(const GatherArgs& a, const Token& k, int32_t lo, int32_t hi, int32_t each, int c0,
                                          F32x2 (&s)[C][4]) {
  constexpr int U = 4;  // of a pack's in flight
  const int width = (a.H + 7) / 8 * 8;
#pragma unroll
  for (int j = 0; j < C; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[j][i] = 0;
    if (c0 + 256 * j >= a.H) continue;
#pragma unroll 1
    for (int32_t r = lo; r < hi; r += U * each) {
      float4 x[U], y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* at = a.part + static_cast<int64_t>(k.slot(a, min(r + u * each, hi - 1))) * width + c0 + 256 * j;
        x[u] = __ldcg(reinterpret_cast<const float4*>(at));
        y[u] = __ldcg(reinterpret_cast<const float4*>(at) + 1);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r + u * each >= hi) break;
        s[j][0] = add2(s[j][0], pack_f32x2(x[u].x, x[u].y));
        s[j][1] = add2(s[j][1], pack_f32x2(x[u].z, x[u].w));
        s[j][2] = add2(s[j][2], pack_f32x2(y[u].x, y[u].y));
        s[j][3] = add2(s[j][3], pack_f32x2(y[u].z, y[u].w));
      }
    }
  }
}

// A CTA takes a run, each of its warps a slice of 256 C columns, U rows in flight. A run is a chain of loads -- where it starts, its rows
// and the row of dW -- which many small CTAs hide: 16384 rows of 2048 in bf16 added to dW, tokens spread evenly, move 321 MB in 65 us with the
// sort (at 24 warps an SM 8 us more, with warps that stay and take run after run 43). Runs and groups are short
// so that a token that comes often is spread over CTAs and its chain of sums is short; the warp that is through last in a
// group of runs adds up the group, and the last of the groups the token (a group's sum takes the place of its first run's).
template <class E, bool AL, int C, int U>
__global__ void __launch_bounds__(GATHER_THREADS, U == 8 ? 3 : 4) gather_kernel(const GatherArgs a) {
  const int lane = threadIdx.x & 31;
  const int slice = static_cast<int>(blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5)), c0 = 256 * C * slice + 8 * lane;
  __shared__ uint8_t met[ZERO_ROWS];
  if (AL && blockIdx.y == 0) {  // dout into L2
    for (int i = threadIdx.x; i < a.ahead; i += blockDim.x)
      if (const int64_t t = static_cast<int64_t>(blockIdx.x) * a.ahead + i; t < a.T)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const typename E::bits*>(a.dout) + t * a.ld),
                     "r"(a.H * static_cast<int>(sizeof(typename E::bits))) : "memory");
  }
  griddep_wait();
  if (static_cast<int>(blockIdx.x) >= a.T) {
    if (blockIdx.y == 0) zero_absent_rows<AL>(a, static_cast<int32_t>(blockIdx.x) - a.T, met);
    return;
  }
  const int several = a.n_runs[0], runs_in_all = several + a.n_runs[1], i = static_cast<int>(blockIdx.x);
  if (i >= runs_in_all) return;
  const uint4 run = a.runs[i < several ? i : a.T - 1 - (i - several)];
  const int32_t p = static_cast<int32_t>(run.x & 0x7FFFFFFFu);
  const bool alone = run.x >> 31;
  const uint32_t row = run.z;
  if (!dbg_ok(p < a.T && row < static_cast<uint32_t>(a.rows) && run.w < static_cast<uint32_t>(a.T), a.err)) return;
  const auto in = [&](uint32_t t) { return static_cast<const typename E::bits*>(a.dout) + static_cast<int64_t>(t) * a.ld; };
  auto* out = reinterpret_cast<uint32_t*>(a.dW) + static_cast<int64_t>(row) * a.H;
  // the run's other entries, its first row and the row of dW, all at once
  const Entry e = lane < RUN && p + lane < a.T ? a.sorted[p + lane] : Entry{0xFFFFFFFFu, 0};
  Pack<E> k0[C];
  Pack<F32> old[C];
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (c0 + 256 * j < a.H) k0[j] = load_columns<E, AL>(in(run.w), c0 + 256 * j, a.H, a.err);
  const auto read_old = [&] {
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (a.add && c0 + 256 * j < a.H) old[j] = load_columns<F32, AL>(out, c0 + 256 * j, a.H, a.err);
  };
  if (alone) read_old();
  const int n = __popc(__ballot_sync(kFullWarp, e.row == row) & 0xFFFFu);
  F32x2 s[C][4];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    unpack(k0[j], s[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[j][i] = add2(s[j][i], 0);  // -0 becomes 0, as in a sum of several
  }
  add_rows<E, AL, C, U>(a, n - 1, c0, s, [&](int r) { return __shfl_sync(kFullWarp, e.t, r + 1); });
  if (!alone) {
    Token k{static_cast<int32_t>(run.y), p + n};
    if (n == RUN && p + RUN < a.T)
      k.end = first_not_below(row + 1, p + RUN, a.T, lane, [&](int32_t q) { return a.sorted[q].row; });
    const int32_t runs = (k.end - k.start + RUN - 1) / RUN, mine = (p - k.start) / RUN, lo = mine / GROUP * GROUP, hi = min(runs, lo + GROUP);
    if (!leave_part<C>(a, k.slot(a, mine), k.slot(a, lo), hi - lo, slice, c0, s)) return;
    add_parts<C>(a, k, lo, hi, 1, c0, s);
    if (runs > GROUP) {
      if (!leave_part<C>(a, k.slot(a, lo), 2 * a.slots + k.first(), (runs + GROUP - 1) / GROUP, slice, c0, s)) return;
      add_parts<C>(a, k, 0, runs, GROUP, c0, s);
    }
    read_old();
  }
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (c0 + 256 * j < a.H) put_row<AL>(a, out, c0 + 256 * j, s[j], old[j]);
}

// ---------------------------------------------------------------------------
// few tokens
// ---------------------------------------------------------------------------
// Up to FEW_TOKENS tokens need no sorting: every CTA reads all ids, and the one of a token's first position has its others
// from that. The CTAs behind those write zeros into the rows that no token points at (where dW is new). One launch: 64
// rows of 256 into 4096 take 3 us on the GPU, with the sort 7.5. Sums in the same order as above, the same bits.
constexpr int FEW_TOKENS = 256;

template <class E, bool AL>
__global__ void __launch_bounds__(GATHER_THREADS) gather_few_kernel(const GatherArgs a, int32_t blocks) {
  __shared__ int32_t row_at_t[FEW_TOKENS];
  __shared__ uint32_t list[FEW_TOKENS];
  __shared__ int32_t found;  // positions of the token, 0: this is not its first
  __shared__ uint8_t met[ZERO_ROWS];
  const int tid = threadIdx.x, threads = blockDim.x;
  for (int t = tid; t < a.T; t += threads) row_at_t[t] = a.shard.row_of(a.ids[t]);
  const int32_t z = static_cast<int32_t>(blockIdx.x) - a.T * blocks;
  if (z >= 0) {
    const int32_t r0 = z * a.zero_per, n = min(a.zero_per, a.rows - r0);
    for (int i = tid; i < n; i += threads) met[i] = 0;
    __syncthreads();
    for (int t = tid; t < a.T; t += threads) {
      const int32_t i = row_at_t[t] - r0;
      if (row_at_t[t] >= 0 && i >= 0 && i < n) met[i] = 1;
    }
    __syncthreads();
    zero_rows<AL>(a, r0, n, met);
    return;
  }
  __syncthreads();
  const int p = static_cast<int>(blockIdx.x) / blocks, block = static_cast<int>(blockIdx.x) % blocks;
  const int32_t row = row_at_t[p];
  if (row < 0) return;
  if (tid < 32) {
    int n = 0;
    bool first = true;
    for (int t = 0; t < a.T; t += 32) {
      const bool like = t + tid < a.T && row_at_t[t + tid] == row;
      const uint32_t m = __ballot_sync(kFullWarp, like);
      if (like) list[n + __popc(m & ((1u << tid) - 1))] = t + tid;
      if (n == 0 && m != 0) first = t + __ffs(m) - 1 == p;
      n += __popc(m);
    }
    if (tid == 0) found = first ? n : 0;
  }
  __syncthreads();
  const int n = found, c0 = 8 * (block * threads + tid);
  if (n == 0 || c0 >= a.H) return;
  auto* out = reinterpret_cast<uint32_t*>(a.dW) + static_cast<int64_t>(row) * a.H;
  Pack<F32> old{};
  if (a.add) old = load_columns<F32, AL>(out, c0, a.H, a.err);
  F32x2 s[1][4] = {};
  const auto add = [](F32x2 (&to)[1][4], const F32x2 (&v)[1][4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) to[0][j] = add2(to[0][j], v[0][j]);
  };
  if (n <= RUN) {
    add_rows<E, AL, 1, 4>(a, n, c0, s, [&](int i) { return list[i]; });
  } else {
    for (int g = 0; g < n; g += RUN * GROUP) {
      const int stop = min(n, g + RUN * GROUP);
      F32x2 sum[1][4] = {};
      for (int i = g; i < stop; i += RUN) {
        F32x2 v[1][4] = {};
        add_rows<E, AL, 1, 4>(a, min(RUN, stop - i), c0, v, [&](int q) { return list[i + q]; });
        add(sum, v);
      }
      add(s, sum);
    }
  }
  put_row<AL>(a, out, c0, s[0], old);
}

struct Room {  // the workspace of a gradient
  size_t a, b, runs, done, part, all;
  int32_t slots;
};

// CTAs of a run, and the warps of each: a slice of 256 `packs` columns a warp.
struct Slices {
  int warps, blocks;
  Slices(int64_t H, int packs)
      : warps(static_cast<int>(std::min<int64_t>(GATHER_THREADS / 32, (H + 256 * packs - 1) / (256 * packs)))),
        blocks(static_cast<int>((H + 256 * packs * warps - 1) / (256 * packs * warps))) {}
  int all() const { return blocks * warps; }
};

inline Room room_of(int64_t T, int64_t H) {
  Room r{};
  if (T <= FEW_TOKENS) return r;
  r.slots = static_cast<int32_t>(T / RUN + 1);
  r.b = carved(T * sizeof(Entry));
  r.runs = 2 * r.b;
  r.done = r.runs + carved((T + 1) * sizeof(uint4));  // the list, and how many it has
  const int slices = std::max(Slices(H, 1).all(), Slices(H, 2).all());
  r.part = r.done + carved(3 * static_cast<size_t>(r.slots) * slices * sizeof(int32_t));
  r.all = r.part + carved(2 * static_cast<size_t>(r.slots) * ((H + 7) / 8 * 8) * sizeof(float));
  return r;
}

// A launch of the sort as a cluster of `ctas`.
struct SortLaunch {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  SortLaunch(int ctas, cudaStream_t s) {
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(SORT_THREADS);
    cfg.dynamicSmemBytes = sizeof(SortSmem);
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  SortLaunch(const SortLaunch&) = delete;  // cfg points into it
};

using SortKernel = void (*)(SortArgs);
constexpr SortKernel kSorts[] = {sort_tokens_kernel<2, true>, sort_tokens_kernel<8, true>, sort_tokens_kernel<8, false>};

// The largest cluster of the sort, 0 for an error: SORT_CTAS where the device can place one.
inline int sort_ctas_at_most() {
  static KnownPerDevice known;
  return known([] {
    for (SortKernel k : kSorts)
      if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortSmem)) != cudaSuccess ||
          cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return 0;
    return cluster_that_fits(SORT_CTAS, [](int ctas) {
      const SortLaunch l(ctas, nullptr);
      for (SortKernel k : kSorts) {
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, k, &l.cfg) != cudaSuccess || n < 1) {
          cudaGetLastError();
          return false;
        }
      }
      return true;
    });
  });
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
  const int32_t packs = static_cast<int32_t>((H + 7) / 8), each = packs > 128 ? 1 : 256 / packs;
  const LookupArgs a{table, out, ids, T, ld, out_ld, static_cast<int32_t>(H), packs, each,
                     static_cast<uint32_t>(((1 << 20) + packs - 1) / packs), static_cast<float>(scale),
                     Shard{vocab_start, V_local, V_true, err_flag}};
  const unsigned ctas = static_cast<unsigned>((T + each - 1) / each);
  const bool al = whole_packs(table, V_local, H, ld, in.eb) && whole_packs(out, T, H, out_ld, to.eb);
  return with_pair(dtype, out_dtype, [&](auto e, auto o) {
    const auto s = static_cast<cudaStream_t>(stream);
    using A = decltype(e);
    using B = decltype(o);
    if (!al) lookup_kernel<A, B, false, 256><<<ctas, 256, 0, s>>>(a);
    else if (packs > 128 && packs <= 256) lookup_kernel<A, B, true, 128><<<ctas, 128, 0, s>>>(a);  // two packs a thread
    else lookup_kernel<A, B, true, 256><<<ctas, 256, 0, s>>>(a);
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
  if (r.all > 0 && (!workspace || !on_boundary(workspace, 256) || workspace_bytes < r.all)) return RLK_ERR_WORKSPACE;
  const bool al = whole_packs(dout, T, H, ld, in.eb) && on_boundary(dW, 32);
  const Shard shard{vocab_start, V_local, V_true, err_flag};
  GatherArgs g{nullptr, nullptr, nullptr, ids, shard, dout, dW, ld, static_cast<int32_t>(T), static_cast<int32_t>(H),
               static_cast<int32_t>(V_local), static_cast<float>(scale), accumulate != 0, nullptr, nullptr, r.slots, 0, 0, 0, err_flag};
  // the CTAs that write zeros: eight an SM at least, of half a megabyte at most (151936 rows of 4096, 8192 tokens: 366 us;
  // eight an SM of 2 MB each 378, four of 4 MB 434; 4096 rows of 256, 64 tokens: 3.3 us, with four times the CTAs 4.6)
  const int64_t share = std::min<int64_t>((V_local + 1215) / 1216, std::max<int64_t>(1, 131072 / H));
  g.zero_per = accumulate ? 0 : static_cast<int32_t>(std::min<int64_t>(ZERO_ROWS, share));
  const int64_t zero = accumulate ? 0 : (V_local + g.zero_per - 1) / g.zero_per;
  if (T <= FEW_TOKENS) {
    const int threads = static_cast<int>(H >= 8 * GATHER_THREADS ? GATHER_THREADS : (H + 255) / 256 * 32);
    const int32_t blocks = static_cast<int32_t>((H + 8 * threads - 1) / (8 * threads));
    const int64_t ctas = T * blocks + zero;
    return with_type(dtype, [&](auto e) {
      const auto kernel = al ? gather_few_kernel<decltype(e), true> : gather_few_kernel<decltype(e), false>;
      kernel<<<static_cast<unsigned>(ctas), threads, 0, s>>>(g, blocks);
      return launched();
    });
  }
  const int packs = in.eb == 4 || H <= 256 || T * ((H + 255) / 256) <= FEW_WARPS ? 1 : 2;  // a lane's in a slice
  const Slices cut(H, packs);
  g.slices = cut.all();
  char* ws = static_cast<char*>(workspace);
  auto* runs = reinterpret_cast<uint4*>(ws + r.runs);
  auto* n_runs = reinterpret_cast<int32_t*>(runs + T);
  SortArgs q{ids, reinterpret_cast<Entry*>(ws + r.a), reinterpret_cast<Entry*>(ws + r.b), static_cast<int32_t>(T), 0, 0, shard,
             reinterpret_cast<int32_t*>(ws + r.done), 3 * r.slots * g.slices, runs, n_runs};
  while (V_local >> q.bits) ++q.bits;  // rows and the mark behind them: 0 .. V_local
  q.passes = (q.bits + 8) / 9;
  const int most = sort_ctas_at_most();
  if (most == 0) return RLK_ERR_CUDA;
  int ctas = 1;  // two positions a thread while there are CTAs
  while (ctas < most && T > 2 * SORT_THREADS * ctas) ctas *= 2;
  const int64_t groups = (T + SORT_THREADS * ctas - 1) / (SORT_THREADS * ctas);
  const SortLaunch sort(ctas, s);
  if (cudaLaunchKernelEx(&sort.cfg, kSorts[groups <= 2 ? 0 : groups <= 8 ? 1 : 2], q) != cudaSuccess) return RLK_ERR_CUDA;
  g.sorted = q.passes & 1 ? q.a : q.b;
  g.runs = runs;
  g.n_runs = n_runs;
  g.part = reinterpret_cast<float*>(ws + r.part);
  g.done = q.done;
  if (al && T * H * in.eb <= AHEAD_BYTES) g.ahead = static_cast<int32_t>((T + AHEAD_CTAS - 1) / AHEAD_CTAS);
  const auto go = [&](auto kernel) { return launch_after(kernel, dim3(static_cast<unsigned>(T + zero), cut.blocks), 32 * cut.warps, s, g); };
  return with_type(dtype, [&](auto e) {
    using E = decltype(e);
    if constexpr (sizeof(typename E::bits) == 4) return go(al ? gather_kernel<E, true, 1, 4> : gather_kernel<E, false, 1, 4>);
    else if (packs == 2) return go(al ? gather_kernel<E, true, 2, 2> : gather_kernel<E, false, 2, 2>);
    else return go(al ? gather_kernel<E, true, 1, 8> : gather_kernel<E, false, 1, 8>);
  });
}

}  // extern "C"
