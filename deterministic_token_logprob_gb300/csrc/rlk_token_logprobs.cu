// rlk_token_logprobs.cu -- rlk_token_logprobs and rlk_token_logprobs_bwd: log probabilities of given
// tokens from logits, with rank, entropy and top alternatives, and the gradient of logp and entropy.
#include <cuda_runtime.h>

#include "rlk_logits_grad.cuh"

namespace rlk {
namespace {

constexpr int CAND = 8 * RLK_MAX_TOP_K;     // most candidates: 8 columns of each of 128 octets
constexpr int PLACES = 2 * RLK_MAX_TOP_K;   // most cells at the first attempt
constexpr int OCTETS = 4 * RLK_MAX_TOP_K;   // most octets at the first attempt

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

// A bar that the k best of N values reach and at most `most` of them, -inf never (all that are not
// -inf reach the lowest finite value, the bar for N <= k). get(i) gives values i .. i + 3 (i a multiple
// of 4), -inf from N up to the next multiple of 128.
// The first try is the k-th of the 32 lanes' maxima, or for k > 32 steps down from the least of them,
// doubled until k values reach it; where more than `most` do, bisection raises it on the values' order
// keys, which hold nothing in their low `shift` bits, counting the values at or above the middle.
// *ties: how many of those equal to the bar are to be taken, lower places first -- all of them, unless
// ties stand in the way of any such bar.
template <class G>
__device__ __forceinline__ float choose_bar(const G& get, int N, int k, int most, int shift, int* ties, int lane) {
  constexpr float kLowest = -3.4028235e38f;
  *ties = N;
  if (N <= k) return kLowest;
  const int padded = (N + 127) / 128 * 128;
  const auto reach = [&](float bar) {
    int n = 0;
#pragma unroll 4
    for (int i = lane * 4; i < padded; i += 128) {
      const float4 x = get(i);
      n += (x.x >= bar) + (x.y >= bar) + (x.z >= bar) + (x.w >= bar);
    }
    return __reduce_add_sync(kFullWarp, n);
  };
  float top = neg_inf();
  if (N <= 256) {  // few values: every lane its share of them
    for (int i = lane; i < N; i += 32) {
      const float4 x = get(i & ~3);
      top = fmaxf(top, i & 2 ? (i & 1 ? x.w : x.z) : (i & 1 ? x.y : x.x));
    }
  } else {
#pragma unroll 4
    for (int i = lane * 4; i < padded; i += 128) {
      const float4 x = get(i);
      top = fmaxf(fmaxf(top, fmaxf(x.x, x.y)), fmaxf(x.z, x.w));
    }
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
  int place[PLACES];               // chosen cells (groups at the second attempt)
  int octet[OCTETS];               // first columns of the chosen octets
  int n_place, n_octet, n_cand;
  float bar;
  RowLog q;
};

// Dynamic shared memory of a row: leaves and cells, or in their place, once they have been used, the
// maxima of the groups (256 columns) and of the octets of 128 groups.
__host__ __device__ constexpr int groups_of(int n) { return (n + LEAF_GROUP - 1) / LEAF_GROUP; }
__host__ __device__ constexpr int group_room(int n) { return (groups_of(n) + 127) / 128 * 128; }
__host__ __device__ constexpr size_t row_smem_bytes(int n, bool top) {
  const size_t b = leaves_of(n) * sizeof(Stats);
  if (!top) return b;
  const size_t first = b + cell_room(n) * 4;
  const size_t exact = group_room(n) * 4 + (groups_of(n) < RLK_MAX_TOP_K ? (groups_of(n) + 3) / 4 * 4 : RLK_MAX_TOP_K) * 32 * 4;
  return first > exact ? first : exact;
}

// The top_k alternatives of a row, by one CTA, from its cells' maxima and a bar that k of them reach.
//  1. The k best columns reach the bar, so they stand in cells that reach it, and there in octets (8
//     consecutive columns) that do. In a short row the octets' own maxima give a higher bar.
//  2. The octets' columns that reach the bar are the candidates: little more than k.
//  3. If there are too many on the way (good columns crowd into few cells, or ties stand at the bar), the
//     row is gone through once more for its groups of 256 columns: the k groups with the largest maxima
//     (lower group first among equals) hold the k best columns, for a column outside them has k
//     groups' maxima ahead of it; and so do the k best of those groups' octets.
//  4. Each candidate's place is the number of candidates ahead of it (many are sorted instead).
template <class R, class E = typename R::E>
__device__ void find_top(const R& row, const ScoreArgs& a, int64_t t, unsigned char* dyn, const float* cell, TopSmem& ts) {
  const RowLog q = ts.q;
  const bool bad = isnan(q.l);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int K = a.top_k, cells = cells_of(row.n);
  const float bar = ts.bar;
  const auto octet_max = [&](int c) {
    const Pack<E> k[1] = {packs_inside(row, c, c + 8) ? load_pack(row, c) : load_pack_edge(row, c)};
    return pack_max(k);
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
  bool many = false;
  if (!bad) {
    for (int i = threadIdx.x; i < cells; i += blockDim.x)
      if (cell[i] >= bar) {
        const int at = atomicAdd(&ts.n_place, 1);
        if (at < PLACES) ts.place[at] = i;
      }
    __syncthreads();
    many = ts.n_place > PLACES;
  }
  if (!many && !bad) {
    const int octets = LEAF_GROUPS * ts.n_place;
    const auto column_of = [&](int i) {
      const int x = ts.place[i / LEAF_GROUPS];
      return x / 32 * ROW_LEAF + i % LEAF_GROUPS * LEAF_GROUP + x % 32 * 8;
    };
    const auto list = [&](int c) {
      const int at = atomicAdd(&ts.n_octet, 1);
      if (at < OCTETS) ts.octet[at] = c;
    };
    if (cells >= 3 * K) {
      for (int i = threadIdx.x; i < octets; i += blockDim.x) {
        const int c = column_of(i);
        if (octet_max(c) >= bar) list(c);
      }
    } else {  // few cells against k: the bar is low, and the octets raise it
      float* omax = reinterpret_cast<float*>(ts.cand);  // not yet in use
      static_assert(LEAF_GROUPS * PLACES * sizeof(float) <= sizeof(ts.cand), "room for the octets' maxima");
      for (int i = threadIdx.x; i < (octets + 127) / 128 * 128; i += blockDim.x)
        omax[i] = i < octets ? octet_max(column_of(i)) : neg_inf();
      __syncthreads();
      if (warp == 0) {
        int ties;
        const auto get = [&](int i) { return *reinterpret_cast<const float4*>(omax + i); };
        const float b = choose_bar(get, octets, K, min(OCTETS, K + K / 2 + 16), E::kKeyShift, &ties, lane);
        if (lane == 0) ts.bar = b;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < octets; i += blockDim.x)
        if (omax[i] >= ts.bar) list(column_of(i));
    }
    __syncthreads();
    many = ts.n_octet > OCTETS;
    if (!many) {
      collect(ts.bar);
      many = ts.n_cand > CAND;
    }
  }
  if (many) {  // the same for the whole CTA
    __syncthreads();  // cells and leaves have been read, the counts too
    const int groups = groups_of(row.n);
    float* gmax = reinterpret_cast<float*>(dyn);
    float* omax = gmax + group_room(row.n);
    const auto best_of = [&](const float* v, int N, int* place) {
      int ties;
      const auto get = [&](int i) { return *reinterpret_cast<const float4*>(v + i); };
      const float b = choose_bar(get, N, K, RLK_MAX_TOP_K, E::kKeyShift, &ties, lane);
      if (lane == 0) ts.bar = b;
      return take_places(v, N, b, ties, place, RLK_MAX_TOP_K, lane);
    };
    for (int g = warp; g < group_room(row.n); g += warps) {
      const float m = g < groups ? warp_max(octet_max(g * LEAF_GROUP + lane * 8)) : neg_inf();
      if (lane == 0) gmax[g] = m;
    }
    __syncthreads();
    if (warp == 0) {
      const int m = best_of(gmax, groups, ts.place);
      if (lane == 0) ts.n_place = m;
    }
    __syncthreads();
    const int chosen = ts.n_place, N = chosen * 32;
    for (int i = warp; i < chosen; i += warps) omax[i * 32 + lane] = octet_max(ts.place[i] * LEAF_GROUP + lane * 8);
    for (int i = N + threadIdx.x; i < (N + 127) / 128 * 128; i += blockDim.x) omax[i] = neg_inf();
    __syncthreads();
    if (warp == 0) {
      const int m = best_of(omax, N, ts.octet);
      __syncwarp();
      for (int i = lane; i < m; i += 32) ts.octet[i] = ts.place[ts.octet[i] / 32] * LEAF_GROUP + ts.octet[i] % 32 * 8;
      if (lane == 0) ts.n_octet = m, ts.n_cand = 0;
    }
    __syncthreads();
    collect(ts.bar);
  }
  const int n = ts.n_cand;
  int64_t* ids = a.top_ids + t * K;
  float* lps = a.top_logp + t * K;
  const auto put = [&](int place, unsigned long long c) {
    ids[place] = static_cast<int64_t>(~static_cast<uint32_t>(c));
    lps[place] = token_logp(key_value(static_cast<uint32_t>(c >> 32)), a.in.s, q);
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
            // 1000 with k = 100: 39 -> 17 us)
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

// logp, rank, lse and entropy in one pass over the row, the alternatives from what the pass left in
// shared memory and a few hundred columns read again (from L2). The pass reads each logit once. With
// 16-bit types and alternatives the instructions bind, not the memory: about 10 an element, of which a
// third is what each lane does once for the 32 elements that it has of a leaf (8192 rows of 151936 in
// bf16 with 20 alternatives: 429 us for 2.49 GB, 5.8 TB/s; without any 382 us, 6.5 TB/s; 4096 in fp32 with
// 64: 386 us, 6.4 TB/s, with none 338 us, 7.3 TB/s). Few rows are bound by latency: a single one takes
// 8 us on the GPU, on 8 SMs.
// Persistent CTAs, whose finishing warp overlaps the next row's pass, are slower (749 us against 485 at
// that step): finishing a row takes one warp 30 us.
// 64 registers a thread, whatever the number of threads: 1024 of them fill an SM. In 16-bit types that
// spills three to eight of them (20 bytes stored and 12 loaded in the aligned bf16 form with alternatives,
// 32 and 28 in the misaligned one), in fp32 none but one in the misaligned form with alternatives.
template <class E, bool TOP, bool AL>
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
    for (int i = cells_of(in.n) + threadIdx.x; i < cell_room(in.n); i += blockDim.x) sm.cell[i] = neg_inf();
  }
  RankOf rank;
  row_pass<true, TOP>(row, in.c, rank, sm, C, r, [&] { rank.load(row, a.y ? a.y + t : nullptr, a.rank != nullptr); });
  if (r != 0) return;
  if (warp == (blockDim.x > 32)) {
    const Stats x = fold_leaves(sm.leaf, leaves_of(in.n), in.c, lane);
    const RowLog q = row_log(x);
    const bool bad = isnan(q.l);
    int before = 0;
    if (rank.on)
      for (int i = lane; i < C * static_cast<int>(blockDim.x >> 5); i += 32) before += counts[i];
    before = __reduce_add_sync(kFullWarp, before);
    if (lane == 0) {
      if (TOP) ts.q = q;
      if (a.lse) a.lse[t] = row_lse(q, in.s);
      if (a.entropy) a.entropy[t] = row_entropy(x);
      if (a.logp) a.logp[t] = rank.ok && !bad ? token_logp(rank.z, in.s, q) : quiet_nan();
      if (a.rank) a.rank[t] = rank.ok && !bad ? 1 + before : 0;
      if (in.err_flag && bad) atomicOr(in.err_flag, RLK_FLAG_NONFINITE);
      if (in.err_flag && a.y && !rank.ok) atomicOr(in.err_flag, RLK_FLAG_BAD_TARGET);
    }
  }
  if constexpr (TOP) {
    if (warp == 0) {
      // from the leaves' maxima where they are many against k, else from the cells'
      const int L = leaves_of(in.n), K = a.top_k;
      int ties;
      float b;
      if (L >= 2 * K && L >= 32) {
        const auto get = [&](int i) {
          const auto at = [&](int j) { return j < L ? sm.leaf[j].m : neg_inf(); };
          return make_float4(at(i), at(i + 1), at(i + 2), at(i + 3));
        };
        b = choose_bar(get, L, K, K + 16, E::kKeyShift, &ties, lane);
      } else {
        const auto get = [&](int i) { return *reinterpret_cast<const float4*>(sm.cell + i); };
        b = choose_bar(get, cells_of(in.n), K, min(PLACES, 2 * K + 16), E::kKeyShift, &ties, lane);
      }
      if (lane == 0) ts.bar = b;
    }
    __syncthreads();
    find_top(row, a, t, dyn, sm.cell, ts);
  }
}

// ---------------------------------------------------------------------------
// the gradient
// ---------------------------------------------------------------------------
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

constexpr float kLowestLogp = -1e4f;  // p = 0 far above it, and B d stays a number

// dz = p (A + B d), and p (A + B d) + C at the target, with d = s (z - m) - l = log p. A masked column
// (d = -inf) has p = 0 and a finite d.
template <bool AWAY>
struct TokenDz {
  float s;
  RowLog r;
  float A, B, C;
  int y;
  __device__ __forceinline__ float one(float z, int c) const {
    const float d = fmaxf(log_p<AWAY>(z, s, r), kLowestLogp);
    const float p = prob_of(d), t = __fmaf_rn(B, d, A);
    return c == y ? __fmaf_rn(p, t, C) : __fmul_rn(p, t);
  }
  template <class E>
  __device__ __forceinline__ void pack(const Pack<E>& k, int c, float (&v)[8]) const {
    const F32x2 le = pack_f32x2(kLog2e, kLog2e), AA = pack_f32x2(A, A), BB = pack_f32x2(B, B);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 d = unpack_f32x2(log_p<AWAY>(pair(k, i), s, r));
      const F32x2 dd = pack_f32x2(fmaxf(d.x, kLowestLogp), fmaxf(d.y, kLowestLogp));
      const float2 x = unpack_f32x2(mul2(dd, le));
      const float2 dz = unpack_f32x2(mul2(pack_f32x2(ex2_approx(x.x), ex2_approx(x.y)), fma2(BB, dd, AA)));
      v[2 * i] = dz.x;
      v[2 * i + 1] = dz.y;
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

struct TokenRow {  // what a row of the gradient has of its own
  float g, ge, ent;
  int64_t y;
};

template <bool AWAY>
__device__ __forceinline__ TokenDz<AWAY> token_dz(const TokenGradArgs& a, const RowLog& r, const TokenRow& x) {
  const float s = a.in.s;
  return TokenDz<AWAY>{s, r, __fmul_rn(-s, __fmaf_rn(x.ge, x.ent, x.g)), __fmul_rn(-s, x.ge), __fmul_rn(s, x.g),
                       static_cast<int>(x.y)};
}

// Nothing but the row's lse, entropy and two weights crosses columns, so a row is cut at will: parts of
// 8192 to 32768 columns a CTA (grad_parts), in packs whose stores are whole aligned vectors. Bound by
// memory: 8192 rows of 151936 in bf16 take 711 us for 4.97 GB, 7.0 TB/s.
// In fp32 to bf16 four CTAs an SM (64 registers) are best: 2000 rows of 50264 take 88.2 us, with the 76 registers
// that the compiler takes by itself 89.4; in fp32 throughout 129.9 and 120.9.
template <class E, class O, bool AL>
__global__ void __launch_bounds__(ROW_THREADS, AL && sizeof(typename E::bits) > sizeof(typename O::bits) ? 4 : 0)
token_grad_kernel(const TokenGradArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  const LogitRows& in = a.in;
  const int64_t t = blockIdx.x / a.parts;
  const auto* z = static_cast<const typename E::bits*>(in.base) + t * in.ld;
  const GradPart<E, O, AL> part(z, in.n, static_cast<typename O::bits*>(a.out.base) + t * a.out.ld, a.out.V,
                                static_cast<int>(blockIdx.x % a.parts), a.parts, in.err_flag);
  const float lse = a.lse[t];
  const TokenRow x{a.g_logp[t], a.g_entropy ? a.g_entropy[t] : 0.f, a.g_entropy ? a.entropy[t] : 0.f, a.y[t]};
  const bool y_ok = x.y >= 0 && x.y < in.n;
  if (!y_ok && threadIdx.x == 0 && part.lo == 0 && in.err_flag) atomicOr(in.err_flag, RLK_FLAG_BAD_TARGET);
  const bool live = y_ok && !isnan(lse) && !(x.g == 0.f && x.ge == 0.f);
  if (live && lse_is_coarse<O>(lse)) {  // the first of the row's CTAs reads and writes all of it
    if (part.lo != 0) return;
    const RowLog r = read_row_log<E>(z, in.n, in.c, reinterpret_cast<Stats*>(dyn), in.err_flag);
    write_row<E, O>(z, in.n, part.out, a.out.V, r.m != neg_inf(), token_dz<true>(a, r, x));
    return;
  }
  // every thread reads and writes columns of its own
  write_part<GRAD_PACKS>(part, live && lse != neg_inf(), token_dz<false>(a, RowLog{0.f, lse}, x));
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
  const size_t smem = row_smem_bytes(a.in.n, top_k > 0);
  const RowShape shape = row_shape(a.in, top_k, smem + (top_k ? sizeof(TopSmem) : 0) + ROW_SMEM_FIXED);
  a.cluster = shape.cluster;
  return with_types(dtype, aligned_rows(logits, ld, dtype_bytes(dtype)), [&](auto e, auto al) {
    using E = decltype(e);
    constexpr bool AL = decltype(al)::value;
    return top_k ? launch_rows(token_logprobs_kernel<E, true, AL>, a, T * a.cluster, a.cluster, smem, stream, shape.threads)
                 : launch_rows(token_logprobs_kernel<E, false, AL>, a, T * a.cluster, a.cluster, smem, stream, shape.threads);
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
    return launch_rows(token_grad_kernel<decltype(e), decltype(o), decltype(al)::value>, a, T * a.parts, 1,
                       leaves_of(a.in.n) * sizeof(Stats), stream);
  });
}

}  // extern "C"
