// rlk_logits.cu -- the operators over logits of include/rlk.h: token log probabilities with
// entropy and top alternatives, their gradient, and distillation from a teacher's top logits
// (forward, backward, both in one call).
#include <cuda_runtime.h>

#include <atomic>
#include <utility>

#include "rlk_logits.cuh"

namespace rlk {
namespace {

constexpr int ROW_THREADS = 256;
constexpr int MAX_CLUSTER = 8;                               // CTAs of one row (the portable cluster size)
constexpr int MAX_ROW_THREADS = 1024;
constexpr int MAX_ROW_WARPS = MAX_CLUSTER * MAX_ROW_THREADS / 32;
// The units in which the pass keeps maxima for the alternatives' search: groups of 256 columns (four
// a leaf), or in short rows octets, the packs themselves.
enum TopCells : int { TOP_NONE = 0, TOP_GROUPS = 1, TOP_OCTETS = 2 };
constexpr int GRAD_PACKS = 4;                                // packs a thread has in flight in the gradients
constexpr int SHORT_ROW = 32768;                             // columns up to which the cells are octets
constexpr int CAND = 8 * RLK_MAX_TOP_K;                      // most candidates: 8 columns of each chosen octet
constexpr int PLACES = 2 * RLK_MAX_TOP_K;                    // most groups at the first attempt
constexpr int OCTETS = 4 * RLK_MAX_TOP_K;                    // most octets at the first attempt

// ---------------------------------------------------------------------------
// one pass over a row by a cluster of CTAs (one CTA when there are rows enough)
// ---------------------------------------------------------------------------
// Warp g of the row's C x (blockDim / 32) warps takes leaves g, g + (number of warps), ... and
// leaves what it found in the shared memory of the cluster's CTA 0 (distributed shared memory):
// (m, s, u) of each leaf, the maxima of its cells (TOP), and how many columns stand ahead of the
// target.
struct RowSmem {
  Stats* leaf;      // [n_leaves]
  float* cell;      // [cell_room(n, TOP)]
  int* count;       // [MAX_ROW_WARPS]
};

__host__ __device__ constexpr int leaves_of(int n) { return (n + ROW_LEAF - 1) / ROW_LEAF; }
__host__ __device__ constexpr int cells_of(int n, int top) {
  return top == TOP_OCTETS ? (n + 7) / 8 : (n + LEAF_GROUP - 1) / LEAF_GROUP;
}
__host__ __device__ constexpr int cell_room(int n, int top) {  // whole leaves, a multiple of 128
  return top == TOP_NONE ? 0 : top == TOP_OCTETS ? leaves_of(n) * 128 : (leaves_of(n) * LEAF_GROUPS + 127) / 128 * 128;
}

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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

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
template <bool ENT, int TOP, class E>
__device__ __forceinline__ int leaf_pass(const Pack<E> (&k)[LEAF_GROUPS], int l, float c, const RankOf& rank,
                                         uint32_t leaf0, uint32_t cell0, bool puts, int lane) {
  float gm[LEAF_GROUPS], m;
#pragma unroll
  for (int j = 0; j < LEAF_GROUPS; ++j) {
    gm[j] = pack_max(k[j]);
    if constexpr (TOP == TOP_OCTETS)
      st_cluster_u32(cell0 + static_cast<uint32_t>((l * LEAF_GROUPS + j) * 32 + lane) * 4, __float_as_uint(gm[j]));
    if constexpr (TOP == TOP_GROUPS) gm[j] = warp_max(gm[j]);
  }
  m = fmaxf(fmaxf(gm[0], gm[1]), fmaxf(gm[2], gm[3]));
  if constexpr (TOP != TOP_GROUPS) m = warp_max(m);
  float2 x;
  if (m == neg_inf()) x = make_float2(any_nan(k) ? quiet_nan() : 0.f, 0.f);
  else x = leaf_sums<ENT>(k, m, c, lane);
  if (puts) {
    st_cluster_f32x4(leaf0 + static_cast<uint32_t>(l * 16), m, x.x, x.y, 0.f);
    if (TOP == TOP_GROUPS) st_cluster_f32x4(cell0 + static_cast<uint32_t>(l * 16), gm[0], gm[1], gm[2], gm[3]);
  }
  // a leaf whose best column is below the target has none ahead of it: for a likely token, most
  return rank.on && m >= rank.z ? count_ahead(k, rank, l, lane) : 0;
}

// Starts the copy of a leaf into L2, where the whole leaf lies inside the row: the passes that have no
// registers for a second leaf have the next one on its way all the same (8192 rows of 151936 in bf16
// with 20 alternatives: 509 -> 485 us; two leaves ahead 488, four 497).
template <class R>
__device__ __forceinline__ void prefetch_leaf(const R& row, int l) {
  constexpr int EB = sizeof(*row.p);
  if ((l + 1) * ROW_LEAF > row.n) return;
  const char* p = reinterpret_cast<const char*>(row.p) - row.shift + static_cast<int64_t>(l) * ROW_LEAF * EB;
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(ROW_LEAF * EB) : "memory");
}

// `begin` runs in every thread after the first loads have been issued: what it loads arrives with them.
template <bool ENT, int TOP, class R, class B, class E = typename R::E>
__device__ __forceinline__ void row_pass(const R& row, float c, RankOf& rank, const RowSmem& sm, int C, int r, B begin) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5, g = r * warps + warp, n_leaves = leaves_of(row.n), step = C * warps;
  if (C > 1) cluster_arrive();  // CTA 0 must have started before anyone writes to it
  const uint32_t leaf0 = map_to_cta(smem_u32(sm.leaf), 0);
  const uint32_t cell0 = TOP ? map_to_cta(smem_u32(sm.cell), 0) : 0;
  int count = 0;
  // 64 registers have room for the next leaf's packs in the lean pass over 16-bit types alone (8192
  // rows of 151936 in bf16: 378 -> 354 us); elsewhere the other warps hide the loads
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
// the best of N values, by one warp
// ---------------------------------------------------------------------------
// The value of the type whose order key >> shift is `bar` (its low bits are 0 in the fp32 image, so
// 1 in the key of a negative value); the lowest finite value for -inf and below.
__device__ __forceinline__ float bar_value(uint32_t bar, int shift) {
  uint32_t key = bar << shift;
  if (!(key & 0x80000000u)) key |= (1u << shift) - 1u;
  return key <= order_key(neg_inf()) ? -3.4028235e38f : key_value(key);
}

// A bar that the k best of v[0 .. N) reach and at most `most` of them, -inf never (all that are not
// -inf reach the lowest finite value, the bar for N <= k). v is padded with -inf to a multiple of 128.
// The first try is the k-th of the 32 lanes' maxima, or for k > 32 steps down from the least of them,
// doubled until k values reach it; where more than `most` do, bisection raises it on the values' order
// keys, which hold nothing in their low `shift` bits, counting the values at or above the middle.
// *ties: how many of those equal to the bar are to be taken, lower places first -- all of them, unless
// ties stand in the way of any such bar.
__device__ __forceinline__ float choose_bar(const float* v, int N, int k, int most, int shift, int* ties, int lane) {
  constexpr float kLowest = -3.4028235e38f;
  *ties = N;
  if (N <= k) return kLowest;
  const int padded = (N + 127) / 128 * 128;
  const auto reach = [&](float bar) {
    int n = 0;
#pragma unroll 4
    for (int i = lane * 4; i < padded; i += 128) {
      const float4 x = *reinterpret_cast<const float4*>(v + i);
      n += (x.x >= bar) + (x.y >= bar) + (x.z >= bar) + (x.w >= bar);
    }
    return __reduce_add_sync(kFullWarp, n);
  };
  float top = neg_inf();
#pragma unroll 4
  for (int i = lane * 4; i < padded; i += 128) {
    const float4 x = *reinterpret_cast<const float4*>(v + i);
    top = fmaxf(fmaxf(top, fmaxf(x.x, x.y)), fmaxf(x.z, x.w));
  }
  int before = 0;  // lanes whose maximum stands ahead of this one's
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float other = __shfl_sync(kFullWarp, top, j);
    before += other > top || (other == top && j < lane);
  }
  const auto ranked = [&](int r) {  // the r-th largest of them (r from 0; -inf where a NaN is among them)
    const uint32_t at = __ballot_sync(kFullWarp, before == r);
    const float x = __shfl_sync(kFullWarp, top, at ? __ffs(at) - 1 : 0);
    return at ? x : neg_inf();
  };
  const float best = ranked(0);
  uint32_t hi = (order_key(best) >> shift) + 1;  // fewer than k reach it
  uint32_t lo = order_key(ranked(min(k, 32) - 1)) >> shift;
  float bar = bar_value(lo, shift);
  int n = reach(bar);
  for (float d = __fsub_rn(best, bar); n < k && bar > kLowest; d = __fadd_rn(d, d)) {
    hi = lo;
    const float next = __fsub_rn(bar, d);
    lo = next < bar ? order_key(next) >> shift : 0u;  // (no step: d is 0 or lost against the bar)
    bar = bar_value(lo, shift);
    n = reach(bar);
  }
  if (n > most) {
    while (n > most && hi > lo + 1) {
      const uint32_t mid = lo + (hi - lo) / 2;
      const int m = reach(bar_value(mid, shift));
      if (m >= k) lo = mid, n = m;
      else hi = mid;
    }
    bar = bar_value(lo, shift);
    if (n > most) *ties = k - reach(bar_value(lo + 1, shift));
  }
  return bar;
}

// The places that choose_bar chose, in ascending order; how many there are (at most `most`).
__device__ __forceinline__ int take_places(const float* v, int N, float bar, int ties, int* place, int most, int lane) {
  int out = 0;
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = 0; i0 < N; i0 += 32) {
    const float x = i0 + lane < N ? v[i0 + lane] : neg_inf();
    const uint32_t eq = __ballot_sync(kFullWarp, x == bar);
    const bool take = x > bar || (x == bar && __popc(eq & below) < ties);
    const uint32_t taken = __ballot_sync(kFullWarp, take);
    const int at = out + __popc(taken & below);
    if (take && at < most) place[at] = i0 + lane;
    out += __popc(taken);
    ties -= min(ties, __popc(eq));
  }
  return min(out, most);
}

struct ScoreArgs {
  LogitRows in;
  int32_t cluster;
  const int64_t* y;
  int32_t top_k;
  float* logp;
  int32_t* rank;
  float* lse;
  float* entropy;
  int64_t* top_ids;
  float* top_logp;
};

// Shared memory of the alternatives' search.
struct TopSmem {
  unsigned long long cand[CAND];   // order key in the high word, ~column in the low one
  int place[PLACES];               // chosen groups
  int octet[OCTETS];               // first columns of the chosen octets
  int n_place, n_octet, n_cand, ties;
  float bar, lse;
};

// Dynamic shared memory of a row. Where the cells are groups, the maxima of the chosen groups' octets
// may take the place of the leaves' statistics and the cells, which have been used by then.
__host__ __device__ constexpr size_t row_smem_bytes(int n, int top) {
  const size_t b = leaves_of(n) * sizeof(Stats) + static_cast<size_t>(cell_room(n, top)) * 4;
  const size_t octets = RLK_MAX_TOP_K * 32 * 4;
  return top == TOP_GROUPS && b < octets ? octets : b;
}

// So many may reach a bar: with room above k, a bar is found in fewer steps.
__device__ __forceinline__ int chosen_most(int k, int room) { return min(room, 2 * k + 16); }

// The top_k alternatives of a row, by one CTA, from its cells' maxima and the bar that choose_bar found
// for them.
//  1. The k cells with the largest maxima (lower cell first among equals) hold the k best columns: a
//     column outside them has k cells' maxima ahead of it. Chosen are they and some more that reach
//     the bar, which k columns reach; of groups, the octets (8 columns) that reach it.
//  2. The octets' columns that reach the bar are the candidates: little more than k, unless good
//     columns crowd into few groups or are tied. If there are more than CAND of them, the same
//     choice among the octets' maxima leaves 128 octets at most, and so no more than CAND.
//  3. Each candidate's place is the number of candidates ahead of it (many are sorted instead).
template <int TOP, class R, class E = typename R::E>
__device__ void find_top(const R& row, const ScoreArgs& a, int64_t t, const RowSmem& sm, TopSmem& ts,
                         bool bad, float lse) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int K = a.top_k, cells = cells_of(row.n, TOP);
  const float bar = ts.bar;
  const auto octet_max = [&](int c) {
    return pack_max(packs_inside(row, c, c + 8) ? load_pack(row, c) : load_pack_edge(row, c));
  };
  const auto collect = [&](float reached) {
    for (int i = threadIdx.x; i < 8 * ts.n_octet; i += blockDim.x) {
      const int c = ts.octet[i / 8] + i % 8;
      const float z = c < row.n ? row.at(c) : neg_inf();
      if (!(z >= reached)) continue;
      const int at = atomicAdd(&ts.n_cand, 1);
      if (at < CAND) ts.cand[at] = static_cast<unsigned long long>(order_key(z)) << 32 | static_cast<uint32_t>(~c);
    }
    __syncthreads();
  };
  // without ties at the bar, and with cells to choose among
  bool many = !bad && (ts.ties < cells || (TOP == TOP_GROUPS && cells <= K));
  if (!many && !bad) {
    int* list = TOP == TOP_GROUPS ? ts.place : ts.octet;
    int* count = TOP == TOP_GROUPS ? &ts.n_place : &ts.n_octet;
    for (int i = threadIdx.x; i < cells; i += blockDim.x)
      if (sm.cell[i] >= bar) {
        const int at = atomicAdd(count, 1);
        if (at < (TOP == TOP_GROUPS ? PLACES : OCTETS)) list[at] = TOP == TOP_GROUPS ? i : i * 8;
      }
    __syncthreads();
    if constexpr (TOP == TOP_GROUPS) {
      const int chosen = min(ts.n_place, PLACES);
#pragma unroll 4
      for (int i = warp; i < chosen; i += warps) {
        const int c = ts.place[i] * LEAF_GROUP + lane * 8;
        if (octet_max(c) >= bar) {
          const int at = atomicAdd(&ts.n_octet, 1);
          if (at < OCTETS) ts.octet[at] = c;
        }
      }
      __syncthreads();
    }
    many = ts.n_octet > OCTETS;
    if (!many) {
      collect(bar);
      many = ts.n_cand > CAND;
    }
  }
  if (many) {  // the same for the whole CTA
    const float* omax = sm.cell;
    int N = cells;
    if constexpr (TOP == TOP_GROUPS) {
      if (warp == 0) {
        int ties;
        const float b = choose_bar(sm.cell, cells, K, RLK_MAX_TOP_K, E::kKeyShift, &ties, lane);
        const int m = take_places(sm.cell, cells, b, ties, ts.place, RLK_MAX_TOP_K, lane);
        if (lane == 0) ts.n_place = m;
      }
      __syncthreads();
      float* o = reinterpret_cast<float*>(sm.leaf);
      const int chosen = ts.n_place;
      omax = o;
      N = chosen * 32;
      for (int i = warp; i < chosen; i += warps) o[i * 32 + lane] = octet_max(ts.place[i] * LEAF_GROUP + lane * 8);
      for (int i = N + threadIdx.x; i < (N + 127) / 128 * 128; i += blockDim.x) o[i] = neg_inf();
      __syncthreads();
    }
    if (warp == 0) {
      int ties;
      const float b = choose_bar(omax, N, K, RLK_MAX_TOP_K, E::kKeyShift, &ties, lane);
      const int m = take_places(omax, N, b, ties, ts.octet, RLK_MAX_TOP_K, lane);
      __syncwarp();
      for (int i = lane; i < m; i += 32) {
        const int o = ts.octet[i];
        ts.octet[i] = TOP == TOP_GROUPS ? ts.place[o / 32] * LEAF_GROUP + o % 32 * 8 : o * 8;
      }
      if (lane == 0) ts.bar = b, ts.n_octet = m, ts.n_cand = 0;
    }
    __syncthreads();
    collect(ts.bar);
  }
  const int n = ts.n_cand;
  int64_t* ids = a.top_ids + t * K;
  float* lps = a.top_logp + t * K;
  const auto put = [&](int place, unsigned long long c) {
    ids[place] = static_cast<int64_t>(~static_cast<uint32_t>(c));
    lps[place] = token_logp(key_value(static_cast<uint32_t>(c >> 32)), a.in.s, lse);
  };
  if ((n + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x) * n <= 1024) {  // a pass over the others for each
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const unsigned long long me = ts.cand[i];
      int place = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) place += ts.cand[j] > me;
      if (place < K) put(place, me);
    }
  } else {  // for a small CTA, or many of them, a bitonic network over the next power of two is less (64 rows of
            // 1000 with k = 100: 115 -> 31 us)
    const int size = n <= 256 ? 256 : n <= 512 ? 512 : 1024;
    static_assert(CAND == 1024, "the network's largest size");
    for (int i = n + threadIdx.x; i < size; i += blockDim.x) ts.cand[i] = 0;
    for (int run = 2; run <= size; run *= 2)
      for (int d = run / 2; d >= 1; d /= 2) {
        __syncthreads();
        for (int i = threadIdx.x; i < size / 2; i += blockDim.x) {
          const int x = 2 * i - (i & (d - 1)), y = x + d;  // i-th pair at distance d
          const unsigned long long p = ts.cand[x], q = ts.cand[y];
          if ((p < q) == ((x & run) == 0)) ts.cand[x] = q, ts.cand[y] = p;
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < min(n, K); i += blockDim.x) put(i, ts.cand[i]);
  }
  for (int i = n + threadIdx.x; i < K; i += blockDim.x) {
    ids[i] = -1;
    lps[i] = bad ? quiet_nan() : neg_inf();
  }
}

// 64 registers a thread, whatever the number of threads: 1024 of them fill an SM.
template <class E, int TOP, bool AL>
__global__ void __launch_bounds__(MAX_ROW_THREADS, 1) token_logprobs_kernel(const ScoreArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ int counts[MAX_ROW_WARPS];
  __shared__ __align__(16) unsigned char top_raw[TOP ? sizeof(TopSmem) : 16];
  TopSmem& ts = *reinterpret_cast<TopSmem*>(top_raw);
  const LogitRows& in = a.in;
  const int C = a.cluster, r = blockIdx.x % C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x / C;
  const Row<E, AL> row(static_cast<const typename E::bits*>(in.base) + t * in.ld, in.n, in.err_flag);
  const RowSmem sm{reinterpret_cast<Stats*>(dyn), reinterpret_cast<float*>(dyn + leaves_of(in.n) * sizeof(Stats)), counts};
  if (TOP && r == 0) {
    if (threadIdx.x == 0) ts.n_cand = ts.n_place = ts.n_octet = 0;
    if (TOP == TOP_GROUPS)
      for (int i = leaves_of(in.n) * LEAF_GROUPS + threadIdx.x; i < cell_room(in.n, TOP); i += blockDim.x) sm.cell[i] = neg_inf();
  }
  RankOf rank;
  row_pass<true, TOP>(row, in.c, rank, sm, C, r, [&] { rank.load(row, a.y ? a.y + t : nullptr, a.rank != nullptr); });
  if (r != 0) return;
  if (warp == (blockDim.x > 32)) {
    const Stats x = fold_leaves(sm.leaf, leaves_of(in.n), in.c, lane);
    const float lse = row_lse(x, in.s);
    const bool bad = isnan(lse);
    int before = 0;
    if (rank.on)
      for (int i = lane; i < C * static_cast<int>(blockDim.x >> 5); i += 32) before += counts[i];
    before = __reduce_add_sync(kFullWarp, before);
    if (lane == 0) {
      if (TOP) ts.lse = lse;
      if (a.lse) a.lse[t] = lse;
      if (a.entropy) a.entropy[t] = row_entropy(x, in.s);
      if (a.logp) a.logp[t] = rank.ok && !bad ? token_logp(rank.z, in.s, lse) : quiet_nan();
      if (a.rank) a.rank[t] = rank.ok && !bad ? 1 + before : 0;
      if (in.err_flag && bad) atomicOr(in.err_flag, RLK_FLAG_NONFINITE);
      if (in.err_flag && a.y && !rank.ok) atomicOr(in.err_flag, RLK_FLAG_BAD_TARGET);
    }
  }
  if constexpr (TOP) {
    if (warp == 0) {
      int ties;
      const float b = choose_bar(sm.cell, cells_of(in.n, TOP), a.top_k, chosen_most(a.top_k, TOP == TOP_GROUPS ? PLACES : OCTETS),
                                 E::kKeyShift, &ties, lane);
      if (lane == 0) ts.bar = b, ts.ties = ties;
    }
    __syncthreads();
    find_top<TOP>(row, a, t, sm, ts, isnan(ts.lse), ts.lse);
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
  int32_t parts;     // CTAs of a row
  const int64_t* y;
  const float* lse;
  const float* entropy;
  const float* g_logp;
  const float* g_entropy;
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
// without reading). Each thread has U packs in flight; `first` runs in every thread between the
// first loads and the first store.
template <int U, class G, class F, class B>
__device__ __forceinline__ void write_part(const G& g, bool live, F f, B first) {
  using E = typename G::E;
  using O = typename G::O;
  const int tid = threadIdx.x, threads = blockDim.x;
  bool begun = false;
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
  for (int q = g.q0; !begun || q < g.q1; q += U * threads) {
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
    if (!begun) {
      begun = true;
      first();
      // the columns outside the packs: before the head and after the last pack
      const int tail0 = g.head + 8 * g.packs;
      if (tid < 16) {
        const int c = tid < 8 ? tid : tail0 + tid - 8;
        if (g.owns(c) && (tid >= 8 || c < g.head))
          g.put(c, live && c < g.n ? f.one(E::to_f32(g.in.p[c - g.head]), c) : 0.f);
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

constexpr float kLowestLogp = -1e4f;  // p = 0 far above it, and B d stays a number

// dz = p (A + B d), and p (A + B d) + C at the target, with d = s z - lse = log p. A masked column
// (d = -inf) has p = 0 and a finite d.
struct TokenDz {
  float s, lse, A, B, C;
  int y;
  __device__ __forceinline__ float one(float z, int c) const {
    const float d = fmaxf(__fmaf_rn(z, s, -lse), kLowestLogp);
    const float p = prob_of(d), t = __fmaf_rn(B, d, A);
    return c == y ? __fmaf_rn(p, t, C) : __fmul_rn(p, t);
  }
  template <class E>
  __device__ __forceinline__ void pack(const Pack<E>& k, int c, float (&v)[8]) const {
    const F32x2 ss = pack_f32x2(s, s), nl = pack_f32x2(-lse, -lse), le = pack_f32x2(kLog2e, kLog2e);
    const F32x2 AA = pack_f32x2(A, A), BB = pack_f32x2(B, B);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 z = pair(k, i);
      const float2 d = unpack_f32x2(fma2(pack_f32x2(z.x, z.y), ss, nl));
      const F32x2 dd = pack_f32x2(fmaxf(d.x, kLowestLogp), fmaxf(d.y, kLowestLogp));
      const float2 x = unpack_f32x2(mul2(dd, le));
      const float2 r = unpack_f32x2(mul2(pack_f32x2(ex2_approx(x.x), ex2_approx(x.y)), fma2(BB, dd, AA)));
      v[2 * i] = r.x;
      v[2 * i + 1] = r.y;
    }
    if (static_cast<unsigned>(y - c) < 8u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 z = pair(k, i);
        if (y == c + 2 * i) v[2 * i] = one(z.x, y);
        if (y == c + 2 * i + 1) v[2 * i + 1] = one(z.y, y);
      }
    }
  }
};

template <class E, class O, bool AL>
__global__ void __launch_bounds__(ROW_THREADS) token_grad_kernel(const TokenGradArgs a) {
  const LogitRows& in = a.in;
  const int64_t t = blockIdx.x / a.parts;
  const GradPart<E, O, AL> part(static_cast<const typename E::bits*>(in.base) + t * in.ld, in.n,
                                static_cast<typename O::bits*>(a.out.base) + t * a.out.ld, a.out.V,
                                static_cast<int>(blockIdx.x % a.parts), a.parts, in.err_flag);
  const float lse = a.lse[t], g = a.g_logp[t], ge = a.g_entropy ? a.g_entropy[t] : 0.f;
  const float ent = a.g_entropy ? a.entropy[t] : 0.f;
  const int64_t y = a.y[t];
  const bool y_ok = y >= 0 && y < in.n;
  if (!y_ok && threadIdx.x == 0 && part.lo == 0 && in.err_flag) atomicOr(in.err_flag, RLK_FLAG_BAD_TARGET);
  const bool live = y_ok && !isnan(lse) && lse != neg_inf() && !(g == 0.f && ge == 0.f);
  const TokenDz dz{in.s, lse, __fmul_rn(-in.s, __fmaf_rn(ge, ent, g)), __fmul_rn(-in.s, ge), __fmul_rn(in.s, g),
                   static_cast<int>(y)};
  write_part<GRAD_PACKS>(part, live, dz, [] {});  // every thread reads and writes columns of its own
}

struct DistillArgs {
  LogitRows in;
  GradOut out;
  int32_t cluster;       // CTAs of a row (a cluster in the forward)
  const int64_t* ids;
  const float* teacher;
  int32_t K;
  const float* g;
  const float* lse_in;   // backward alone
  float* loss;           // forward
  float* lse;
};

// Loss of one row by one warp (every lane gets it); zk: the student's logits of the entries.
__device__ __forceinline__ float row_loss(const TeacherRow& q, const float* zk, float lse, float s, int lane) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < RLK_MAX_TOP_K / 32; ++i) {
    const int k = lane + 32 * i;
    if (q.q[k] > 0.f) sum = __fmaf_rn(q.q[k], __fsub_rn(q.logq[k], token_logp(zk[k], s, lse)), sum);
  }
  return warp_sum(sum);
}

// The student's logits at the entries' columns (0 without an entry), by the warp that made q.
template <class R>
__device__ __forceinline__ void gather_logits(const TeacherRow& q, const R& row, float* zk, int lane) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < RLK_MAX_TOP_K / 32; ++i) {
    const int id = q.id[lane + 32 * i];
    zk[lane + 32 * i] = id >= 0 ? row.at(id) : 0.f;
  }
}

// The loss's outputs of a row, by one warp.
__device__ __forceinline__ void put_loss(const DistillArgs& a, int64_t t, const TeacherRow& q, const float* zk, float lse,
                                         int lane) {
  const float l = row_loss(q, zk, lse, a.in.s, lane);
  if (lane != 0) return;
  a.loss[t] = isnan(lse) || q.bad ? quiet_nan() : l;
  if (a.lse) a.lse[t] = lse;
  const int flags = q.bad | (isnan(lse) ? RLK_FLAG_NONFINITE : 0);
  if (flags && a.in.err_flag) atomicOr(a.in.err_flag, flags);
}

__device__ __forceinline__ bool distill_live(const TeacherRow& q, float lse, float g) {
  return !isnan(lse) && lse != neg_inf() && q.any && !q.bad && g != 0.f;
}

// dz of entry k's column, A (p - sum of q over the entries of that column in ascending order), if k
// is the first of them; false otherwise.
__device__ __forceinline__ bool entry_dz(const TeacherRow& q, int k, int K, float z, float s, float lse, float A, float* dz) {
  const int id = q.id[k];
  float qk = 0.f;
  for (int j = 0; j < K; j += 4) {  // places past K hold no entry
    const int4 o = *reinterpret_cast<const int4*>(q.id + j);
    if (o.x != id && o.y != id && o.z != id && o.w != id) continue;
    for (int e = 0; e < 4; ++e) {
      if (q.id[j + e] != id) continue;
      if (j + e < k) return false;
      qk = __fadd_rn(qk, q.q[j + e]);
    }
  }
  *dz = __fmul_rn(A, __fsub_rn(prob_of(__fmaf_rn(z, s, -lse)), qk));
  return true;
}

// dz = A p, p = e^{s z - lse}.
struct DistillDz {
  float s, lse, A;
  __device__ __forceinline__ float one(float z, int) const { return __fmul_rn(A, prob_of(__fmaf_rn(z, s, -lse))); }
  template <class E>
  __device__ __forceinline__ void pack(const Pack<E>& k, int, float (&v)[8]) const {
    const F32x2 ss = pack_f32x2(s, s), nl = pack_f32x2(-lse, -lse), le = pack_f32x2(kLog2e, kLog2e), AA = pack_f32x2(A, A);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 z = pair(k, i);
      const float2 x = unpack_f32x2(mul2(fma2(pack_f32x2(z.x, z.y), ss, nl), le));
      const float2 r = unpack_f32x2(mul2(AA, pack_f32x2(ex2_approx(x.x), ex2_approx(x.y))));
      v[2 * i] = r.x;
      v[2 * i + 1] = r.y;
    }
  }
};

// Backward alone: a.cluster CTAs of a row, each its own part.
template <class E, class O, bool AL>
__global__ void __launch_bounds__(ROW_THREADS) distill_grad_kernel(const DistillArgs a) {
  __shared__ TeacherRow q;
  __shared__ float zk[RLK_MAX_TOP_K];
  const LogitRows& in = a.in;
  const int64_t t = blockIdx.x / a.cluster;
  const auto* z = static_cast<const typename E::bits*>(in.base) + t * in.ld;
  const GradPart<E, O, AL> part(z, in.n, static_cast<typename O::bits*>(a.out.base) + t * a.out.ld, a.out.V,
                                static_cast<int>(blockIdx.x % a.cluster), a.cluster, in.err_flag);
  const float lse = a.lse_in[t], g = a.g[t];
  if (threadIdx.x < 32) {
    teacher_softmax(q, a.ids + t * a.K, a.teacher + t * a.K, a.K, in.n, in.s, in.c, threadIdx.x);
    __syncwarp();
    // the logits of the teacher's columns, read before anything is written; other parts may already
    // have written theirs
    const bool in_use = g != 0.f;
#pragma unroll
    for (int i = 0; i < RLK_MAX_TOP_K / 32; ++i) {
      const int k = threadIdx.x + 32 * i;
      zk[k] = in_use && part.owns(q.id[k]) ? E::to_f32(z[q.id[k]]) : 0.f;
    }
  }
  __syncthreads();
  if (q.bad && part.lo == 0 && threadIdx.x == 0 && in.err_flag) atomicOr(in.err_flag, q.bad);
  const bool live = distill_live(q, lse, g);
  const float A = __fmul_rn(in.s, g);
  write_part<GRAD_PACKS>(part, live, DistillDz{in.s, lse, A}, [] {});
  __syncthreads();
  if (!live) return;
  for (int k = threadIdx.x; k < a.K; k += ROW_THREADS) {
    float dz;
    if (q.id[k] >= 0 && part.owns(q.id[k]) && entry_dz(q, k, a.K, zk[k], in.s, lse, A, &dz)) part.put(q.id[k], dz);
  }
}

// Forward: a cluster of CTAs a row.
template <class E, bool AL>
__global__ void __launch_bounds__(MAX_ROW_THREADS, 1) distill_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ TeacherRow q;
  __shared__ float zk[RLK_MAX_TOP_K];
  const LogitRows& in = a.in;
  const int C = a.cluster, r = blockIdx.x % C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x / C;
  const Row<E, AL> row(static_cast<const typename E::bits*>(in.base) + t * in.ld, in.n, in.err_flag);
  const bool reads = r == 0 && warp == static_cast<int>(blockDim.x >> 5) - 1;
  if (reads) {
    teacher_softmax(q, a.ids + t * a.K, a.teacher + t * a.K, a.K, in.n, in.s, in.c, lane);
    gather_logits(q, row, zk, lane);
  }
  RowSmem sm{reinterpret_cast<Stats*>(dyn), nullptr, nullptr};
  RankOf none;
  row_pass<false, TOP_NONE>(row, in.c, none, sm, C, r, [] {});
  if (r == 0 && warp == 0) put_loss(a, t, q, zk, row_lse(fold_leaves(sm.leaf, leaves_of(in.n), in.c, lane), in.s), lane);
}

// ---------------------------------------------------------------------------
// forward and backward in one launch
// ---------------------------------------------------------------------------
// The cluster's CTAs keep the row in their shared memory between the sum and the gradient, so it
// is read from memory once. CTA r takes leaves r, r + C, ...; its warp w those with local index w,
// w + W, ..., and copies all of them asynchronously before anything else, one copy group a leaf,
// so that the whole row is in flight at once and each leaf is summed as it arrives. The warp that
// summed a leaf writes its gradient: nothing but the leaves' statistics (to every CTA) and the
// lse crosses warps.
constexpr int STEP_THREADS = 288;
constexpr int STEP_CTAS = 4;              // of one SM
constexpr int STEP_MAX_ROUNDS = 8;        // leaves of one warp
constexpr int SLOT_SLACK = 32;            // a misaligned pack is cut from up to 32 bytes more

template <class E>
__host__ __device__ constexpr int slot_bytes() { return ROW_LEAF * static_cast<int>(sizeof(typename E::bits)) + SLOT_SLACK; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Wait until at most n of this thread's copy groups are pending.
__device__ __forceinline__ void cp_async_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}

// Copies leaf l into a slot, by one warp: vector v holds the 16 bytes of the row that start
// `shift` bytes before column 8 v (4 v) of the leaf. Vectors that do not lie inside the row are
// filled element by element, -inf beyond it.
template <class R, class E = typename R::E>
__device__ __forceinline__ void copy_leaf(const R& row, int l, unsigned char* slot, int lane) {
  constexpr int EB = sizeof(typename E::bits), PER = 16 / EB;
  constexpr int VECS = ROW_LEAF / PER + (R::AL ? 0 : 1);
  const int c0 = l * ROW_LEAF - static_cast<int>(row.shift) / EB;  // column of the slot's first element
  const char* src = reinterpret_cast<const char*>(row.p) + static_cast<int64_t>(c0) * EB;
  const uint32_t dst = smem_u32(slot);
  if (c0 >= 0 && c0 + VECS * PER <= row.n) {
#pragma unroll
    for (int v = lane; v < VECS; v += 32) cp_async16(dst + v * 16, src + v * 16);
    return;
  }
  auto* out = reinterpret_cast<typename E::bits*>(slot);
  for (int v = lane; v < VECS; v += 32) {
    const int c = c0 + v * PER;
    if (c >= 0 && c + PER <= row.n) {
      cp_async16(dst + v * 16, src + v * 16);
    } else {
      for (int i = 0; i < PER; ++i) out[v * PER + i] = c + i >= 0 && c + i < row.n ? row.p[c + i] : E::kNegInf;
    }
  }
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.relaxed.cluster.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t ld_cluster_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.relaxed.cluster.shared::cluster.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}

// Writes the gradient of a leaf (first column c0) from its slot, by one warp; zeros when !live.
template <class O, class V, class F>
__device__ __forceinline__ void leaf_grad(const V& view, typename O::bits* out, int c0, int head, int n, int V_, bool live,
                                          const F& f, int lane) {
  using E = typename V::E;
  const int end = min(V_ - c0, ROW_LEAF);        // columns of the leaf to write
  if (end == ROW_LEAF && head == 0 && c0 + ROW_LEAF <= n && live) {
#pragma unroll
    for (int u = 0; u < LEAF_GROUPS; ++u) {
      const int c = u * LEAF_GROUP + lane * 8;
      float v[8];
      f.pack(load_pack(view, c), c0 + c, v);
      if (dbg_ok(c0 + c + 8 <= V_, view.err)) store_pack<O>(out + c0 + c, v);
    }
    return;
  }
  const int packs = max(0, end - head) / 8;      // 128 of a whole leaf, 127 with a head
  for (int p = lane; p < packs; p += 32) {
    const int c = c0 + head + p * 8;
    float v[8];
    f.pack(load_pack(view, p * 8), c, v);        // the slot is filled in any case
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!live || c + e >= n) v[e] = 0.f;
    if (dbg_ok(c + 8 <= V_, view.err)) store_pack<O>(out + c, v);
  }
  if (lane < 16) {  // before the first pack and after the last
    const int c = lane < 8 ? lane : head + packs * 8 + lane - 8;
    if (c < end && (lane >= 8 || c < head))
      out[c0 + c] = O::from_f32(live && c0 + c < n ? f.one(E::to_f32(view.p[c - head]), 0) : 0.f);
  }
}

// AL: the rows are aligned; GAL: the gradient's packs are (always where dlogits are the logits).
template <class E, class O, bool AL, bool GAL>
__global__ void __launch_bounds__(STEP_THREADS, STEP_CTAS) distill_step_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ TeacherRow q;
  __shared__ float zk[RLK_MAX_TOP_K];
  __shared__ float lse_s;
  constexpr int EB = sizeof(typename E::bits), OB = sizeof(typename O::bits), SLOT = slot_bytes<E>();
  const LogitRows& in = a.in;
  const int C = a.cluster, r = blockIdx.x % C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = (blockDim.x >> 5) - 1;                       // warps that take leaves; one more for the rest
  const int64_t t = blockIdx.x / C;
  const int n_leaves = leaves_of(in.n);
  const int mine = (n_leaves - r + C - 1) / C;               // this CTA's leaves
  const int rounds = warp < min(W, mine) ? (mine - warp + W - 1) / W : 0;
  Stats* leaf = reinterpret_cast<Stats*>(dyn);               // of the whole row
  unsigned char* slots = dyn + n_leaves * sizeof(Stats);
  if (C > 1) cluster_arrive();
  const Row<E, AL> row(static_cast<const typename E::bits*>(in.base) + t * in.ld, in.n, in.err_flag);
  const float g = a.g[t];
  for (int j = 0; j < rounds; ++j) {
    copy_leaf(row, r + (warp + j * W) * C, slots + (warp + j * W) * SLOT, lane);
    cp_async_commit();
  }
  if (warp == W) teacher_softmax(q, a.ids + t * a.K, a.teacher + t * a.K, a.K, in.n, in.s, in.c, lane);
  if (C > 1) cluster_wait();  // every CTA has started: its shared memory may be written
  const uint32_t to = map_to_cta(smem_u32(leaf), lane < C ? lane : 0);
  for (int j = 0; j < rounds; ++j) {
    const int i = warp + j * W;
    cp_async_wait(rounds - 1 - j);
    __syncwarp();
    const Row<E, AL> view(reinterpret_cast<const typename E::bits*>(slots + i * SLOT + row.shift), ROW_LEAF + SLOT_SLACK / EB,
                          in.err_flag);
    Pack<E> k[LEAF_GROUPS];
#pragma unroll
    for (int u = 0; u < LEAF_GROUPS; ++u) k[u] = load_pack(view, u * LEAF_GROUP + lane * 8);
    leaf_pass<false, TOP_NONE>(k, r + i * C, in.c, RankOf{}, to, 0u, lane < C, lane);
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  if (warp == 0) {
    const float lse = row_lse(fold_leaves(leaf, n_leaves, in.c, lane), in.s);
    if (lane == 0) lse_s = lse;
  } else {
    // the student's logits of the entries: CTA 0 takes all of them from the cluster's slots, for the
    // loss, the others their own, for the gradient
    for (int k = threadIdx.x - 32; k < a.K; k += blockDim.x - 32) {
      const int id = q.id[k], l = id / ROW_LEAF;
      float z = 0.f;
      if (id >= 0 && (r == 0 || l % C == r)) {
        const uint32_t at = map_to_cta(smem_u32(slots + (l / C) * SLOT + row.shift + id % ROW_LEAF * EB), l % C);
        if constexpr (EB == 4) z = E::to_f32(ld_cluster_u32(at));
        else z = E::to_f32(ld_cluster_u16(at));
      }
      zk[k] = z;
    }
  }
  __syncthreads();
  if (C > 1) cluster_arrive();  // CTA 0 has read the others' slots
  const float lse = lse_s;
  if (r == 0 && warp == 0) put_loss(a, t, q, zk, lse, lane);
  const bool live = distill_live(q, lse, g);
  const DistillDz f{in.s, lse, __fmul_rn(in.s, g)};
  auto* out = static_cast<typename O::bits*>(a.out.base) + t * a.out.ld;
  const int V = a.out.V;
  const int head = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(out) & 15u)) & 15u) / OB;  // of the row and of every leaf
  for (int j = 0; j < rounds; ++j) {
    const int i = warp + j * W;
    const Row<E, GAL> view(reinterpret_cast<const typename E::bits*>(slots + i * SLOT + row.shift) + head,
                           ROW_LEAF + SLOT_SLACK / EB, in.err_flag);
    leaf_grad<O>(view, out, (r + i * C) * ROW_LEAF, head, in.n, V, live, f, lane);
  }
  // columns past the last leaf
  for (int c = n_leaves * ROW_LEAF + r * blockDim.x + threadIdx.x; c < V; c += C * blockDim.x) out[c] = O::from_f32(0.f);
  __syncthreads();
  if (live) {  // the teacher's columns
    for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
      const int id = q.id[k];
      float dz;
      if (id >= 0 && id / ROW_LEAF % C == r && entry_dz(q, k, a.K, zk[k], in.s, lse, f.A, &dz)) out[id] = O::from_f32(dz);
    }
  }
  if (C > 1) cluster_wait();
}

// CTAs (c, a cluster) and warps (w) of a row in the statistics passes. With 64 registers a thread an
// SM runs 32 warps, so floor(32 / w) CTAs; a row takes ceil(leaves / (c w)) rounds of leaves, about
// two more for what surrounds them (the target, the fold, the alternatives) and half a one for each
// doubling of the cluster. The shape with the least waves x rounds: one CTA of 8 warps where rows
// fill the GPU (4 take 579 us where 8 take 509 and 16 564: 8192 rows of 151936 in bf16 with 20
// alternatives), 8 CTAs of 19 for a single row of 149 leaves. Short rows take a warp a leaf; a few of
// them at least 4 or 8, to find the alternatives (64 rows of 1000 with k = 100: 31 -> 15 us; 4096
// rows with k = 50 take 46 us with 2 warps, 55 with 8).
struct RowShape {
  int cluster, threads;
};
RowShape row_shape(const LogitRows& in, int top_k) {
  const int64_t L = leaves_of(in.n);
  RowShape best{1, ROW_THREADS};
  int64_t least = INT64_MAX;
  const bool few_rows = in.T <= 4 * 152;
  const int fewest = L >= 8 || (few_rows && top_k > 32) ? 8 : few_rows && top_k > 0 && L < 4 ? 4 : L < 2 ? 2 : static_cast<int>(L);
  for (int c = 1, half = 0; c <= MAX_CLUSTER; c *= 2, ++half)
    for (int w = fewest; w <= 32; ++w) {
      if (w > 8 && c * (w - 1) >= L) break;  // more warps than leaves
      const int64_t waves = (in.T * static_cast<int64_t>(c) + 152 * (32 / w) - 1) / (152 * (32 / w));
      const int64_t cost = waves * (2 * ((L + c * w - 1) / (c * w)) + 4 + half);
      if (cost < least) least = cost, best = RowShape{c, 32 * w};
    }
  return best;
}

// Launches `ctas` CTAs in clusters of `cluster`.
template <class K, class A>
rlk_status launch_rows(K kernel, const A& args, int64_t ctas, int cluster, size_t smem, void* stream,
                       int threads = ROW_THREADS) {
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
  if (cudaLaunchKernelEx(&cfg, kernel, args) != cudaSuccess) return RLK_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? RLK_OK : RLK_ERR_CUDA;
}

// CTAs of a row in a kernel that writes gradients alone.
// Parts of up to four rounds of every thread's packs (the work that
// a CTA does once -- its row's scalars, the teacher's softmax -- is then small: 8192 rows of 151936
// in bf16 take 715 us with four rounds, 954 with one), as long as that leaves CTAs enough for the GPU.
int grad_parts(const LogitRows& in, const GradOut& o) {
  constexpr int kCols = 8 * GRAD_PACKS * ROW_THREADS;
  constexpr int64_t kEnough = 6 * 152;
  const int64_t rounds = (o.V + kCols - 1) / kCols;
  int64_t each = in.T * rounds / kEnough;
  each = each < 1 ? 1 : each > 4 ? 4 : each;
  return static_cast<int>((rounds + each - 1) / each);
}

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

// Whether every row starts on a 16-byte boundary.
bool aligned_rows(const void* base, int64_t ld, int bytes) {
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 && ld * bytes % 16 == 0;
}

// Whether the packs of every row's gradient are aligned in the logits as well: both sets of rows
// are, or they lie alike (the same type, and the same distance from a boundary in every row).
bool aligned_pair(const LogitRows& in, int32_t dtype, const GradOut& o, int32_t out_dtype) {
  const int eb = dtype_bytes(dtype), ob = dtype_bytes(out_dtype);
  if (aligned_rows(in.base, in.ld, eb) && aligned_rows(o.base, o.ld, ob)) return true;
  return eb == ob && (reinterpret_cast<uintptr_t>(in.base) - reinterpret_cast<uintptr_t>(o.base)) % 16 == 0 &&
         (in.ld - o.ld) * eb % 16 == 0;
}

template <bool B>
struct Flag {
  static constexpr bool value = B;
};

// Calls f with the element type(s) and the alignment as types.
template <class F>
rlk_status with_types(int32_t dtype, bool aligned, F f) {
  const auto al = [&](auto e) { return aligned ? f(e, Flag<true>{}) : f(e, Flag<false>{}); };
  return dtype == RLK_DTYPE_BF16 ? al(Bf16{}) : dtype == RLK_DTYPE_F16 ? al(F16{}) : al(F32{});
}

template <class F>
rlk_status with_types(int32_t dtype, int32_t out_dtype, bool aligned, F f) {
  const auto al = [&](auto e, auto o) { return aligned ? f(e, o, Flag<true>{}) : f(e, o, Flag<false>{}); };
  if (dtype == RLK_DTYPE_BF16) return al(Bf16{}, Bf16{});
  if (dtype == RLK_DTYPE_F16) return al(F16{}, F16{});
  return out_dtype == RLK_DTYPE_BF16 ? al(F32{}, Bf16{}) : al(F32{}, F32{});
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
  const RowShape shape = row_shape(a.in, top_k);
  a.cluster = shape.cluster;
  return with_types(dtype, aligned_rows(logits, ld, dtype_bytes(dtype)), [&](auto e, auto al) {
    using E = decltype(e);
    constexpr bool AL = decltype(al)::value;
    const int top = top_k == 0 ? TOP_NONE : V_true <= SHORT_ROW ? TOP_OCTETS : TOP_GROUPS;
    const auto kernel = top == TOP_NONE     ? token_logprobs_kernel<E, TOP_NONE, AL>
                        : top == TOP_OCTETS ? token_logprobs_kernel<E, TOP_OCTETS, AL>
                                            : token_logprobs_kernel<E, TOP_GROUPS, AL>;
    return launch_rows(kernel, a, T * a.cluster, a.cluster, row_smem_bytes(a.in.n, top), stream, shape.threads);
  });
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
  a.parts = grad_parts(a.in, a.out);
  if (T * a.parts > INT32_MAX) return RLK_ERR_UNSUPPORTED;
  return with_types(dtype, out_dtype, aligned_pair(a.in, dtype, a.out, out_dtype), [&](auto e, auto o, auto al) {
    return launch_rows(token_grad_kernel<decltype(e), decltype(o), decltype(al)::value>, a, T * a.parts, 1, 0, stream);
  });
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

rlk_status launch_distill_fwd(DistillArgs a, int32_t dtype, void* stream) {
  const RowShape shape = row_shape(a.in, 0);
  a.cluster = shape.cluster;
  return with_types(dtype, aligned_rows(a.in.base, a.in.ld, dtype_bytes(dtype)), [&](auto e, auto al) {
    return launch_rows(distill_kernel<decltype(e), decltype(al)::value>, a, static_cast<int64_t>(a.in.T) * a.cluster,
                       a.cluster, row_smem_bytes(a.in.n, TOP_NONE), stream, shape.threads);
  });
}

rlk_status launch_distill_bwd(DistillArgs a, int32_t dtype, int32_t out_dtype, void* stream) {
  a.cluster = grad_parts(a.in, a.out);
  const int64_t ctas = static_cast<int64_t>(a.in.T) * a.cluster;
  if (ctas > INT32_MAX) return RLK_ERR_UNSUPPORTED;
  return with_types(dtype, out_dtype, aligned_pair(a.in, dtype, a.out, out_dtype), [&](auto e, auto o, auto al) {
    return launch_rows(distill_grad_kernel<decltype(e), decltype(o), decltype(al)::value>, a, ctas, 1, 0, stream);
  });
}

// The one-launch step: the smallest cluster whose CTAs hold their share of the row in a quarter of
// an SM's shared memory, or else in a half or the whole. 0: take two launches -- where the row does
// not fit, or where a cluster of more than two has more than four waves of rows to work through. A
// cluster's CTAs wait for one another's sums, and what is resident does not cover that wait: 1024
// rows of 151936 in bf16 (clusters of 8) take 158 us in one launch and 155 in two, 8192 1205 and
// 1083, but 256 rows 46 and 57; 2048 rows of 50257 (clusters of 2) 112 and 134.
constexpr size_t kStepSmem = 220 << 10;

size_t step_smem(int n_leaves, int cluster, int slot) {
  return n_leaves * sizeof(Stats) + static_cast<size_t>((n_leaves + cluster - 1) / cluster) * slot;
}

int step_cluster(const LogitRows& in, int slot) {
  const int L = leaves_of(in.n);
  for (int ctas = STEP_CTAS; ctas >= 1; ctas /= 2)
    for (int c = 1; c <= MAX_CLUSTER; c *= 2)
      if (step_smem(L, c, slot) <= kStepSmem / ctas && (L + c - 1) / c <= STEP_MAX_ROUNDS * (STEP_THREADS / 32 - 1))
        return c <= 2 || static_cast<int64_t>(in.T) * c <= 4 * 152 * ctas ? c : 0;
  return 0;
}

template <class E, class O, bool AL, bool GAL>
rlk_status launch_step(DistillArgs a, void* stream) {
  const int L = leaves_of(a.in.n);
  const size_t smem = step_smem(L, a.cluster, slot_bytes<E>());
  const auto kernel = distill_step_kernel<E, O, AL, GAL>;
  if (smem > (40 << 10)) {  // the opt-in for more shared memory, once per device
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return RLK_ERR_CUDA;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kStepSmem)) !=
          cudaSuccess)
        return RLK_ERR_CUDA;
      if (dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  const int share = (L + a.cluster - 1) / a.cluster, most = STEP_THREADS / 32 - 1;
  const int threads = 32 * ((share < most ? share : most) + 1);
  return launch_rows(kernel, a, static_cast<int64_t>(a.in.T) * a.cluster, a.cluster, smem, stream, threads);
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
  return launch_distill_fwd(a, dtype, stream);
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
  return launch_distill_bwd(a, dtype, out_dtype, stream);
}

rlk_status rlk_distill_topk_fwd_bwd(const void* logits, int32_t dtype, int64_t T, int64_t ld, int64_t V_true,
                                    double temperature, const int64_t* ids, const float* teacher, int32_t K,
                                    const float* g, float* loss, float* lse, void* dlogits, int32_t out_dtype,
                                    int64_t V, int64_t out_ld, int32_t* err_flag, void* stream) {
  DistillArgs a{};
  rlk_status st = check_distill(logits, dtype, T, ld, V_true, temperature, ids, teacher, K, err_flag, &a);
  if (st == RLK_OK) st = check_out(a.in, dtype, dlogits, out_dtype, V, out_ld, &a.out);
  if (st != RLK_OK) return st;
  if (T > 0 && (!g || !loss || !lse)) return RLK_ERR_INVALID_ARG;
  if (T == 0) return RLK_OK;
  a.g = g;
  a.loss = loss;
  a.lse = lse;
  a.cluster = step_cluster(a.in, dtype_bytes(dtype) == 4 ? slot_bytes<F32>() : slot_bytes<Bf16>());
  if (a.cluster == 0) {  // the two calls
    st = launch_distill_fwd(a, dtype, stream);
    a.lse_in = lse;
    return st != RLK_OK ? st : launch_distill_bwd(a, dtype, out_dtype, stream);
  }
  const bool aligned = aligned_rows(logits, ld, dtype_bytes(dtype));
  return with_types(dtype, out_dtype, aligned_pair(a.in, dtype, a.out, out_dtype), [&](auto e, auto o, auto gal) {
    using E = decltype(e);
    using O = decltype(o);
    constexpr bool GAL = decltype(gal)::value;
    return aligned && GAL ? launch_step<E, O, GAL, GAL>(a, stream) : launch_step<E, O, false, GAL>(a, stream);
  });
}

}  // extern "C"
