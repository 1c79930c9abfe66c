// rlk_distill.cu -- rlk_distill_topk_fwd / _bwd / _fwd_bwd: distillation from a teacher's top logits.
#include <cuda_runtime.h>

#include <atomic>

#include "rlk_logits_grad.cuh"

namespace rlk {
namespace {

// ---------------------------------------------------------------------------
// the teacher's distribution of one row
// ---------------------------------------------------------------------------
struct alignas(16) TeacherRow {    // in shared memory, one entry per k < RLK_MAX_TOP_K
  int32_t id[RLK_MAX_TOP_K];       // -1: no entry
  float q[RLK_MAX_TOP_K];          // 0 without an entry
  float logq[RLK_MAX_TOP_K];       // 0 where q is 0
  int32_t any;                     // some entry has q > 0
  int32_t bad;                     // RLK_FLAG_BAD_TARGET / RLK_FLAG_NONFINITE of the row
};

// q = softmax(s t_k) over the row's K entries, by one warp: lane i takes entries i, i + 32, ...
__device__ __forceinline__ void teacher_softmax(TeacherRow& r, const int64_t* ids, const float* t, int K, int n,
                                                float s, float c, int lane) {
  constexpr int R = RLK_MAX_TOP_K / 32;
  int32_t id[R];
  float v[R];
  float m = neg_inf();
  bool bad = false, inf = false;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int k = lane + 32 * i;
    const int64_t x = k < K ? ids[k] : -1;
    v[i] = k < K ? t[k] : neg_inf();
    bad |= x < -1 || x >= n;
    id[i] = x < 0 || x >= n ? -1 : static_cast<int32_t>(x);
    if (id[i] < 0) v[i] = neg_inf();
    inf |= !(v[i] < __int_as_float(0x7f800000));  // NaN or +inf
    m = fmaxf(m, v[i]);
  }
  bad = __any_sync(kFullWarp, bad);
  inf = __any_sync(kFullWarp, inf);
  m = warp_max(m);
  float w[R], sum = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    v[i] = v[i] > neg_inf() ? __fsub_rn(v[i], m) : neg_inf();
    w[i] = ex2_approx(__fmul_rn(v[i], c));
    sum = __fadd_rn(sum, w[i]);
  }
  sum = warp_sum(sum);
  const float ls = logf(sum);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int k = lane + 32 * i;
    const bool some = w[i] > 0.f;
    r.id[k] = id[i];
    r.q[k] = some ? __fdiv_rn(w[i], sum) : 0.f;
    r.logq[k] = some ? __fmaf_rn(v[i], s, -ls) : 0.f;
  }
  if (lane == 0) {
    r.any = m > neg_inf();
    r.bad = (bad ? RLK_FLAG_BAD_TARGET : 0) | (inf ? RLK_FLAG_NONFINITE : 0);
  }
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
__device__ __forceinline__ float row_loss(const TeacherRow& q, const float* zk, const RowLog& p, float s, int lane) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < RLK_MAX_TOP_K / 32; ++i) {
    const int k = lane + 32 * i;
    if (q.q[k] > 0.f) sum = __fmaf_rn(q.q[k], __fsub_rn(q.logq[k], token_logp(zk[k], s, p)), sum);
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
__device__ __forceinline__ void put_loss(const DistillArgs& a, int64_t t, const TeacherRow& q, const float* zk,
                                         const RowLog& p, int lane) {
  const float l = row_loss(q, zk, p, a.in.s, lane);
  if (lane != 0) return;
  a.loss[t] = isnan(p.l) || q.bad ? quiet_nan() : l;
  if (a.lse) a.lse[t] = row_lse(p, a.in.s);
  const int flags = q.bad | (isnan(p.l) ? RLK_FLAG_NONFINITE : 0);
  if (flags && a.in.err_flag) atomicOr(a.in.err_flag, flags);
}

__device__ __forceinline__ bool distill_live(const TeacherRow& q, float lse, float g) {
  return !isnan(lse) && q.any && !q.bad && g != 0.f;
}

// dz of entry k's column, A (p - sum of q over the entries of that column in ascending order), if k
// is the first of them; false otherwise.
__device__ __forceinline__ bool entry_dz(const TeacherRow& q, int k, int K, float z, float s, const RowLog& p, float A,
                                         float* dz) {
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
  *dz = __fmul_rn(A, __fsub_rn(prob_of(log_p<true>(z, s, p)), qk));
  return true;
}

// dz = A p, log p = s (z - m) - l.
template <bool AWAY>
struct DistillDz {
  float s;
  RowLog p;
  float A;
  __device__ __forceinline__ float one(float z, int) const {
    return __fmul_rn(A, prob_of(log_p<AWAY>(z, s, p)));
  }
  template <class E>
  __device__ __forceinline__ void pack(const Pack<E>& k, int, float (&v)[8]) const {
    const F32x2 le = pack_f32x2(kLog2e, kLog2e), AA = pack_f32x2(A, A);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack_f32x2(mul2(log_p<AWAY>(pair(k, i), s, p), le));
      const float2 r = unpack_f32x2(mul2(AA, pack_f32x2(ex2_approx(x.x), ex2_approx(x.y))));
      v[2 * i] = r.x;
      v[2 * i + 1] = r.y;
    }
  }
};

// The teacher's columns, written over the stream's; k: this thread's entry if it is one to write, else -1.
template <class G>
__device__ __forceinline__ void patch_entry(const TeacherRow& q, int k, int K, float z, float s, const RowLog& p, float A,
                                            const G& out) {
  __syncthreads();
  float dz;
  if (k >= 0 && entry_dz(q, k, K, z, s, p, A, &dz)) out.put(q.id[k], dz);
}

// Backward alone: a.cluster CTAs of a row, each its own part. Columns outside the teacher's entries have
// dz = A p; the entries, few, are written over it, so the stream over the row does not look for them.
// Bound by memory: 1000 rows of 32003, fp32 to bf16, take 38 us (5.0 TB/s: one and a half waves of
// CTAs), 8192 rows of 151936 in bf16 713 us (7.0 TB/s). The teacher's columns are read again at the end,
// from L2 (728 us against 716 where the CTA waited for them at the start).
template <class E, class O, bool AL>
__global__ void __launch_bounds__(ROW_THREADS) distill_grad_kernel(const DistillArgs a) {
  __shared__ TeacherRow q;
  __shared__ float zk[RLK_MAX_TOP_K];
  extern __shared__ __align__(16) unsigned char dyn[];
  const LogitRows& in = a.in;
  const int64_t t = blockIdx.x / a.cluster;
  const auto* z = static_cast<const typename E::bits*>(in.base) + t * in.ld;
  const GradPart<E, O, AL> part(z, in.n, static_cast<typename O::bits*>(a.out.base) + t * a.out.ld, a.out.V,
                                static_cast<int>(blockIdx.x % a.cluster), a.cluster, in.err_flag);
  // The first CTAs, two of an SM, wait for their teachers all at once while the memory has nothing to do
  // (200 rows of 151936 in bf16: 24.1 -> 21.7 us); later ones wait while others work, and prefetching for
  // them only crowds the writes (all CTAs: 8192 rows 716 -> 781 us).
  if (blockIdx.x < 2 * 152 && threadIdx.x == 32) part.prefetch();
  const float lse = a.lse_in[t], g = a.g[t];
  const bool in_place = in.base == a.out.base;
  if (threadIdx.x < 32) {
    teacher_softmax(q, a.ids + t * a.K, a.teacher + t * a.K, a.K, in.n, in.s, in.c, threadIdx.x);
    __syncwarp();
    // in place: the logits of the teacher's columns, read before anything is written; other parts may
    // already have written theirs
    if (in_place && g != 0.f)
      for (int k = threadIdx.x; k < a.K; k += 32)
        if (part.owns(q.id[k])) zk[k] = E::to_f32(z[q.id[k]]);
  }
  __syncthreads();
  if (q.bad && part.lo == 0 && threadIdx.x == 0 && in.err_flag) atomicOr(in.err_flag, q.bad);
  const bool live = distill_live(q, lse, g);
  const float A = __fmul_rn(in.s, g);
  const int k = threadIdx.x;
  static_assert(RLK_MAX_TOP_K <= ROW_THREADS, "a thread an entry");
  if (live && lse_is_coarse<O>(lse)) {  // the first of the row's CTAs reads and writes all of it
    if (part.lo != 0) return;
    const bool entry = k < a.K && q.id[k] >= 0;
    const float zy = entry ? E::to_f32(z[q.id[k]]) : 0.f;
    const RowLog p = read_row_log<E>(z, in.n, in.c, reinterpret_cast<Stats*>(dyn), in.err_flag);
    write_row<E, O>(z, in.n, part.out, a.out.V, p.m != neg_inf(), DistillDz<true>{in.s, p, A});
    patch_entry(q, entry && p.m != neg_inf() ? k : -1, a.K, zy, in.s, p, A, part);
    return;
  }
  const RowLog p{0.f, lse};
  write_part<GRAD_PACKS>(part, live && lse != neg_inf(), DistillDz<false>{in.s, p, A});
  const bool patches = live && lse != neg_inf() && k < a.K && part.owns(q.id[k]);
  const float zy = !patches ? 0.f : in_place ? zk[k] : E::to_f32(z[q.id[k]]);  // from L2 now
  patch_entry(q, patches ? k : -1, a.K, zy, in.s, p, A, part);
}

// Forward: a cluster of CTAs a row. The last warp of CTA 0 gathers the student's logits at the teacher's
// columns while the others go over the row. Bound by memory with many rows: 8192 rows of 151936 in bf16
// take 351 us (7.1 TB/s), 512 29 us (5.4 TB/s: one wave, whose start and end count).
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
  RowSmem sm{reinterpret_cast<Stats*>(dyn), nullptr, nullptr};
  RankOf none;
  const auto read_teacher = [&] {
    if (!reads) return;
    teacher_softmax(q, a.ids + t * a.K, a.teacher + t * a.K, a.K, in.n, in.s, in.c, lane);
    gather_logits(q, row, zk, lane);
  };
  // behind the first leaf's loads (4096 rows of 8000 in bf16: 33.1 -> 28.5 us), but for misaligned rows of
  // 16-bit types, where both together spill (796 rows of 50257: 25.4 -> 27.3; as it is, 16 bytes stored and 56
  // loaded)
  constexpr bool BEHIND = AL || sizeof(typename E::bits) == 4;
  if constexpr (!BEHIND) read_teacher();
  row_pass<false, false>(row, in.c, none, sm, C, r, [&] {
    if constexpr (BEHIND) read_teacher();
  });
  if (r == 0 && warp == 0) put_loss(a, t, q, zk, row_log(fold_leaves(sm.leaf, leaves_of(in.n), in.c, lane)), lane);
}

// ---------------------------------------------------------------------------
// forward and backward in one launch
// ---------------------------------------------------------------------------
// The cluster's CTAs keep the row in their shared memory between the sum and the gradient, so it
// is read from memory once. CTA r takes leaves r, r + C, ...; its warp w those with local index w,
// w + W, ..., and copies all of them asynchronously before anything else, one copy group a leaf,
// so that the whole row is in flight at once and each leaf is summed as it arrives. The warp that
// summed a leaf writes its gradient: nothing but the leaves' statistics (to every CTA) and the
// lse crosses warps. 2048 rows of 50257 in bf16 take 113 us, two launches 123; 16 rows of 4096 in
// fp32 6.5 us with 64 entries, 4.2 with 8, two launches 8.5. 56 registers a thread: the forms for misaligned
// fp32 rows spill (8 to 12 bytes stored, 8 to 36 loaded).
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
  __shared__ RowLog p_s;
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
                          in.err_flag, row.shift);
    Pack<E> k[LEAF_GROUPS];
#pragma unroll
    for (int u = 0; u < LEAF_GROUPS; ++u) k[u] = load_pack(view, u * LEAF_GROUP + lane * 8);
    leaf_pass<false, false>(k, r + i * C, in.c, RankOf{}, to, 0u, lane < C, lane);
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  if (warp == 0) {
    const RowLog p = row_log(fold_leaves(leaf, n_leaves, in.c, lane));
    if (lane == 0) p_s = p;
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
  RowLog p = p_s;
  if (r == 0 && warp == 0) put_loss(a, t, q, zk, p, lane);
  const float lse = row_lse(p, in.s);
  const bool live = p.m != neg_inf() && distill_live(q, lse, g);
  const bool coarse = lse_is_coarse<O>(lse);
  if (!coarse) p = RowLog{0.f, lse};  // as the backward alone
  const float A = __fmul_rn(in.s, g);
  auto* out = static_cast<typename O::bits*>(a.out.base) + t * a.out.ld;
  const int V = a.out.V;
  const int head = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(out) & 15u)) & 15u) / OB;  // of the row and of every leaf
  // Coarse rows are rare, and z - m in the stream over all rows takes 2 % with 16-bit types (2048 of 50257 in bf16:
  // 112 -> 114 us): they get a plain loop. In fp32 the loop costs more, by spills (4096 misaligned rows of 12001: 100 ->
  // 110), and the difference nothing.
  constexpr bool ONE = EB == 4;
  for (int j = 0; j < rounds; ++j) {
    const int i = warp + j * W, c0 = (r + i * C) * ROW_LEAF;
    const auto* first = reinterpret_cast<const typename E::bits*>(slots + i * SLOT + row.shift);
    if (!ONE && coarse) {
      const DistillDz<true> f{in.s, p, A};
#pragma unroll 1
      for (int c = lane; c < min(V - c0, ROW_LEAF); c += 32)
        out[c0 + c] = O::from_f32(live && c0 + c < in.n ? f.one(E::to_f32(first[c]), c0 + c) : 0.f);
    } else {
      const Row<E, GAL> view(first + head, ROW_LEAF + SLOT_SLACK / EB, in.err_flag, row.shift + head * EB);
      leaf_grad<O>(view, out, c0, head, in.n, V, live, DistillDz<ONE>{in.s, p, A}, lane);
    }
  }
  // columns past the last leaf
  for (int c = n_leaves * ROW_LEAF + r * blockDim.x + threadIdx.x; c < V; c += C * blockDim.x) out[c] = O::from_f32(0.f);
  __syncthreads();
  if (live) {  // the teacher's columns
    for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
      const int id = q.id[k];
      float dz;
      if (id >= 0 && id / ROW_LEAF % C == r && entry_dz(q, k, a.K, zk[k], in.s, p, A, &dz)) out[id] = O::from_f32(dz);
    }
  }
  if (C > 1) cluster_wait();
}

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
  const size_t smem = leaves_of(a.in.n) * sizeof(Stats);
  const RowShape shape = row_shape(a.in, 0, smem + ROW_SMEM_FIXED);
  a.cluster = shape.cluster;
  return with_types(dtype, aligned_rows(a.in.base, a.in.ld, dtype_bytes(dtype)), [&](auto e, auto al) {
    return launch_rows(distill_kernel<decltype(e), decltype(al)::value>, a, static_cast<int64_t>(a.in.T) * a.cluster,
                       a.cluster, smem, stream, shape.threads);
  });
}

rlk_status launch_distill_bwd(DistillArgs a, int32_t dtype, int32_t out_dtype, void* stream) {
  a.cluster = grad_parts(a.in, a.out);
  const int64_t ctas = static_cast<int64_t>(a.in.T) * a.cluster;
  if (ctas > INT32_MAX) return RLK_ERR_UNSUPPORTED;
  return with_types(dtype, out_dtype, aligned_pair(a.in, dtype, a.out, out_dtype), [&](auto e, auto o, auto al) {
    return launch_rows(distill_grad_kernel<decltype(e), decltype(o), decltype(al)::value>, a, ctas, 1,
                       leaves_of(a.in.n) * sizeof(Stats), stream);
  });
}

// The one-launch step: the smallest cluster whose CTAs hold their share of the row in a quarter of
// an SM's shared memory, or else in a half or the whole. 0: take two launches -- where the row does
// not fit, or where a cluster of more than two (in fp32, with half as many leaves in the same memory, of
// two) has more than four waves of rows to work through. A cluster's CTAs wait for one another's sums,
// and what is resident does not cover that wait: 8192 rows of 151936 in bf16 (clusters of 8) take 1205
// us in one launch and 1069 in two, 4096 of 16000 in fp32 (of 2) 156 and 137, but 600 of them 25 and
// 30, 500 of 100000 in bf16 (of 4) 50 and 59, 4096 of 50176 (of 2) 184 and 201, 8192 of 16000 (one CTA)
// 119 and 153.
constexpr size_t kStepSmem = 220 << 10;

size_t step_smem(int n_leaves, int cluster, int slot) {
  return n_leaves * sizeof(Stats) + static_cast<size_t>((n_leaves + cluster - 1) / cluster) * slot;
}

int step_cluster(const LogitRows& in, int slot) {
  const int L = leaves_of(in.n);
  for (int ctas = STEP_CTAS; ctas >= 1; ctas /= 2)
    for (int c = 1; c <= MAX_CLUSTER; c *= 2)
      if (step_smem(L, c, slot) <= kStepSmem / ctas && (L + c - 1) / c <= STEP_MAX_ROUNDS * (STEP_THREADS / 32 - 1))
        return c <= (slot == slot_bytes<F32>() ? 1 : 2) || static_cast<int64_t>(in.T) * c <= 4 * 152 * ctas ? c : 0;
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
  return launch_rows(kernel, a, static_cast<int64_t>(a.in.T) * a.cluster, a.cluster, smem, stream, threads, false);
}

}  // namespace
}  // namespace rlk

using namespace rlk;

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
