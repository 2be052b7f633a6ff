// ss_distill.cu -- distillation from a teacher's top log probabilities: loss and
// gradient in one call (ss_distill_topk), and the gradient from saved
// normalisers (ss_distill_topk_grad).
#include "ss_logits.cuh"

namespace ss {
namespace {

// Vectors a thread in a block's part of a row shared by a cluster. 4096 x 128256 bf16 with 8, 16, 32, 64: 620, 458,
// 375, 428 us (below, each part's fixed work shows; above, the rows in flight no longer fit L2).
constexpr int kPartVectors = 32;
constexpr int kFewVectors = 8;  // with few rows (64 x 128256 fp32: parts of 32 vectors 18.3 us, of 16 16.4 us)

struct DistillArgs {
  const void* x;
  const void* ids;
  const void* teacher;
  const float* weight;
  const float* d_loss;       // gradient from saved normalisers only
  const float2* norm_in;     // the same
  const float* tail_in;      // the same
  float* loss;
  float2* norm;
  float* tail;
  void* d;
  int64_t rows, vocab, ld, d_ld;
  float c, eps, scale, t_scale;
  int32_t k, mode, t_dtype;
  bool wide, vec, in_place;
  uint32_t split;    // gradient from saved normalisers: blocks that share a row
  int32_t resident;  // rows in flight at a time
};

__device__ __forceinline__ float load_teacher(const void* p, int64_t i, int dtype) {
  if (dtype == SS_FP32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == SS_BF16 ? widen1<SS_BF16>(h) : widen1<SS_FP16>(h);
}

// ------------------------------------------------------------------ a row's list
//
// One warp of the block has the list, lane i its slots i, i + 32, ...: it loads
// them and their logits, drops repeated ids, sums them up and writes their
// gradients, while the block's other warps go through the row's elements.

constexpr int kListThreads = kRowThreads + 32;  // the row's warps and the list's
constexpr int kSlots = SS_MAX_TOP / 32;

struct RowMass {
  float m, s;
};

template <int DT>
struct RowList {
  int32_t id[kSlots];    // -1: unused
  float lq[kSlots];      // log q
  float q[kSlots];
  float x[kSlots];       // the token's logit
  RowMass in;            // the listed tokens' mass
  float q_sum, q_tail;   // Q and q_t
  bool bad;              // an id past the vocabulary

  // The ids and the teacher's values (the list's warp only): all loads first, then what is made of them.
  __device__ __forceinline__ void start(const DistillArgs& a, int64_t row) {
    const int lane = threadIdx.x & 31;
    const int64_t at = row * a.k + lane;
    int64_t given[kSlots];
    if (a.wide) {
      const int64_t* p = static_cast<const int64_t*>(a.ids) + at;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) given[i] = lane + 32 * i < a.k ? p[32 * i] : -1;
    } else {
      const int32_t* p = static_cast<const int32_t*>(a.ids) + at;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) given[i] = lane + 32 * i < a.k ? p[32 * i] : -1;
    }
    if (a.t_dtype == SS_FP32) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        lq[i] = lane + 32 * i < a.k ? static_cast<const float*>(a.teacher)[at + 32 * i] : -kInf;
    } else {
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        lq[i] = lane + 32 * i < a.k ? load_teacher(a.teacher, at + 32 * i, a.t_dtype) : -kInf;
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      id[i] = given[i] < 0 ? -1 : (given[i] >= a.vocab ? INT32_MAX : static_cast<int32_t>(given[i]));
      lq[i] *= a.t_scale;
    }
  }
  // The ids checked, and their logits on their way. ids_shared: SS_MAX_TOP / 4 int4 of shared memory, this warp's own.
  __device__ __forceinline__ void look_up(const DistillArgs& a, const Elem<DT>* xr, int4* ids_shared) {
    const int lane = threadIdx.x & 31;
    bool past = false;
    Elem<DT> raw[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      past = past || id[i] == INT32_MAX;
      if (id[i] == INT32_MAX) id[i] = -1;
      raw[i] = xr[max(id[i], 0)];
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      if (32 * i < a.k) (&ids_shared[0].x)[lane + 32 * i] = id[i];
    }
    bad = __any_sync(0xFFFFFFFFu, past);
#pragma unroll
    for (int i = 0; i < kSlots; ++i) x[i] = to_float<DT>(raw[i]);
  }

  // Drops the slots whose id an earlier slot has: of its own 32, or of those before them.
  __device__ __forceinline__ void drop_repeated(const DistillArgs& a, const int4* ids_shared) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      if (32 * i < a.k) {
        int again = __match_any_sync(0xFFFFFFFFu, id[i]) & ((1u << lane) - 1u);
        for (int q = 0; q < 8 * i; ++q) {
          const int4 v = ids_shared[q];
          again |= (v.x == id[i]) | (v.y == id[i]) | (v.z == id[i]) | (v.w == id[i]);
        }
        if (again) id[i] = -1;
      }
      if (id[i] < 0) {
        lq[i] = -kInf;
        x[i] = -kInf;
      }
    }
  }

  // max and sum of exp(scale (v - max)) over the list; -inf for masked or unused slots, NaN sum for NaN and +inf.
  __device__ __forceinline__ static RowMass mass(const float (&v)[kSlots], float scale) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < kSlots; ++i) m = fmaxf(m, v[i]);
    m = key_value(__reduce_max_sync(0xFFFFFFFFu, order_key(m == m ? m : -kInf)));
    const float ref = m == -kInf ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) s += expf(scaled_gap(v[i], ref, scale));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    return {m, s};
  }

  __device__ __forceinline__ void mass_in(const DistillArgs& a) { in = mass(x, a.scale); }
  // log q, q, Q and q_t.
  __device__ __forceinline__ void sums(const DistillArgs& a) {
    q_sum = q_tail = 0.0f;
    if (a.mode == SS_TAIL_RENORM) {
      const RowMass t = mass(lq, 1.0f);
      const float shift = t.s == 0.0f ? 0.0f : t.m + logf(t.s);
      q_sum = t.s == t.s ? (t.s == 0.0f ? 0.0f : 1.0f) : t.s;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        lq[i] -= shift;
        q[i] = 32 * i < a.k ? expf(lq[i]) : 0.0f;
      }
    } else {
      // q_t = 1 - Q is small when the list has nearly all the mass: Q is added as a pair
      dd s = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        q[i] = 32 * i < a.k ? expf(lq[i]) : 0.0f;
        const dd t = two_sum(s.hi, q[i]);
        s = {t.hi, t.lo + s.lo};
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const float h = __shfl_xor_sync(0xFFFFFFFFu, s.hi, off), lo = __shfl_xor_sync(0xFFFFFFFFu, s.lo, off);
        const dd t = two_sum(s.hi, h);
        s = {t.hi, t.lo + (s.lo + lo)};
      }
      q_sum = s.hi + s.lo;
      if (a.mode == SS_TAIL_BUCKET) {
        const float rest = (1.0f - s.hi) - s.lo;
        q_tail = rest <= 0.0f ? 0.0f : rest;
      }
    }
  }
};

// ------------------------------------------------------------------ loss and gradient in one call
//
// The gradient needs the row's sums and then the row again. A row is shared by
// the blocks of a cluster: small enough parts that all the rows in flight stay
// in L2, so the second pass reads them from there, and HBM sees each logit read
// once (1.09 times, by the counters) and each gradient written once. With
// z = scale x, p over the whole row, p_t over its unlisted tokens, b = Q + q_t:
//   unlisted  d = w scale (p / p_t) (p_t b - q_t)    listed  d = w scale (p b - q)
// where without a bucket q_t = 0 and the first is p b.
//
// 4096 x 128256 bf16, 64 listed: 376 us, 5.59 TB/s of the bytes that have to move,
// 0.82 of the measured copy. What is left is the time from a part's last sum to its
// first gradient and from its start to the list's marks, a fifth of a block's life,
// which two other blocks on the SM cover in part: more of them (4: 409 us against
// 390 then) put L2 over its size. A row held in shared memory (445 us) or in
// registers (495) between the passes leaves room for fewer blocks. The loss alone
// (1024 x 50257 fp16: 24 us, 0.63) is one pass, four blocks an SM.
//
// Eight warps go through the elements and do as little else as can be; the ninth
// has the row's list, the exchange between the blocks and the row's loss:
//   clear   row -> list    the marks are zero
//   ready   list -> row    the listed tokens are marked
//   added   row -> list    the warps' sums are in `red`
//   scales  list -> row    the gradient's factors are in `unlisted`
//   written row -> list    the gradient is written; the list's own goes on top
// The listed tokens are left out of the sums (a bit per element of the part says
// which they are), so the unlisted mass is a sum of its own terms and not a
// difference: log p_t keeps its digits however little is left.

enum Barrier : int { kReady = 1, kAdded = 2, kScales = 3, kWritten = 4, kClear = 5 };

// Marks the elements of packed vector w whose bits are set in `bits` as masked.
template <int DT>
__device__ __forceinline__ void mask_elements(uint4& w, uint32_t bits) {
  uint32_t* p = &w.x;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if constexpr (DT == SS_FP32) {
      if ((bits >> h) & 1u) p[h] = 0xFF800000u;
    } else {
      constexpr uint32_t kNegInf = DT == SS_BF16 ? 0xFF80u : 0xFC00u;
      if ((bits >> (2 * h)) & 1u) p[h] = (p[h] & 0xFFFF0000u) | kNegInf;
      if ((bits >> (2 * h + 1)) & 1u) p[h] = (p[h] & 0xFFFFu) | (kNegInf << 16);
    }
  }
}

// The gradient's factors for the unlisted tokens: a 2^(arg(x) + lift), arg as ExpRef has it. The lift is added to the
// argument: in r it would be rounded to r's digits.
struct Unlisted {
  float r, a, lift;
  bool far;

  // The gradient of the part's elements, the listed ones' to be written over.
  template <int DT>
  __device__ __forceinline__ void map(const RowPart<DT>& part, float scale2, uint4 (&w)[kBatch], Elem<DT>* d, bool vec,
                                      float edge) const {
    const Pair c = Pair::both(scale2), a2 = Pair::both(a), r2 = Pair::both(-r);
    if (!far && lift == 0.0f) {
      part.map(w, d, vec, edge, [&](Pair x) { return mul2(ex2_pair(fma2(x, c, r2)), a2); });
    } else {
      const Pair from = Pair::both(far ? -r : 0.0f), back = Pair::both(far ? 0.0f : -r), up = Pair::both(lift);
      part.map(w, d, vec, edge,
               [&](Pair x) { return mul2(ex2_pair(add2(fma2(add2(x, from), c, back), up)), a2); });
    }
  }
};

struct DistillShared {
  RowSum red[kRowWarps];
  RowSum parts[kMaxCluster];
  int4 list_ids[SS_MAX_TOP / 4];
  Unlisted unlisted;
  uint32_t edge_listed;
};

// Of the row that comes after, with the loss alone: 0, 16, 32, 64 KB: 24.6, 24.3, 23.6, 22.9 us when it was chosen,
// 23.4, 23.3, 23.5, 24.1 with the loop as it is now. (With a gradient: 385, 398, 404, 434 us; the rows in flight need
// the L2.)
constexpr int kAheadBytes = 65536;

// The ninth warp's part in a row. `marks`: a word of listed bits for each batch of vectors, by thread.
template <int DT, bool GRAD>
__device__ __forceinline__ void list_warp(const DistillArgs& a, const Cluster& cl, const RowPart<DT>& part, int64_t row,
                                          float w, RowList<DT>& l, const Elem<DT>* x, Elem<DT>* d, DistillShared& sh,
                                          uint32_t* marks) {
  const int lane = threadIdx.x & 31;
  const float c = a.c;
  l.look_up(a, x, sh.list_ids);
  barrier_sync<kClear, kListThreads>();
  unsigned mine = 0u;  // slots whose element is this block's
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    int owner, slot;
    if (32 * i < a.k && l.id[i] >= 0 && part.owns(l.id[i], &owner, &slot)) {
      mine |= 1u << i;
      if (slot < 0) atomicOr(&sh.edge_listed, 1u << owner);
      else atomicOr(&marks[(slot / kBatch) * kRowThreads + owner],
                    1u << (slot % kBatch * 8 + (l.id[i] - part.sl.head) % kVecOf<DT>));
    }
  }
  barrier_arrive<kReady, kListThreads>();
  const int64_t after = row + a.resident;
  if (after < a.rows) {  // the list that comes after on this SM
    const int64_t id_bytes = a.k * (a.wide ? 8 : 4), t_bytes = a.k * (a.t_dtype == SS_FP32 ? 4 : 2);
    if (lane * 128 < id_bytes) prefetch_line(static_cast<const char*>(a.ids) + after * id_bytes + lane * 128);
    if (lane * 128 < t_bytes) prefetch_line(static_cast<const char*>(a.teacher) + after * t_bytes + lane * 128);
  }
  l.drop_repeated(a, sh.list_ids);
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (l.id[i] < 0) mine &= ~(1u << i);
  l.sums(a);
  l.mass_in(a);
  cl.started();
  barrier_sync<kAdded, kListThreads>();
  if (!GRAD && lane == 0 && after < a.rows)  // HBM has little else to do while the blocks exchange their sums
    prefetch_row<DT>(static_cast<const Elem<DT>*>(a.x) + after * a.ld, a.vocab, kAheadBytes, cl.rank, cl.size);
  RowSum out = merge_lanes(sh.red[lane % kRowWarps], c, kRowWarps);
  if (cl.size > 1) {
    if (lane < cl.size) cl.at(sh.parts, lane)[cl.rank] = out;
    cl.arrive();
    cl.wait();
    out = merge_lanes(sh.parts[lane % cl.size], c, static_cast<int>(cl.size));
  }
  out.mend(a.eps);
  // the row's mass: the listed tokens' and the unlisted ones', around the larger of their maxima
  RowMass all = {fmaxf(l.in.m, out.m), 0.0f};
  all.s = (l.in.m == all.m ? l.in.s : l.in.s * expf(scaled_gap(l.in.m, all.m, a.scale))) +
          (out.m == all.m ? out.s : out.s * expf(scaled_gap(out.m, all.m, a.scale)));
  const bool empty = all.s == 0.0f;
  // all unlisted tokens masked, by -inf or by values so low that no p_t is left
  const bool no_tail = out.s == 0.0f || scaled_gap(out.m, all.m, c) <= kFloor;
  const float p_t = no_tail ? 0.0f : expf(scaled_gap(out.m, all.m, a.scale)) * (out.s / all.s);
  const float ws = l.bad ? nan_f() : w * a.scale;
  const float b = l.q_sum + l.q_tail;
  if constexpr (GRAD) {
    // unlisted: (p / p_t) (p_t b - q_t) = 2^((x - m_out) c) / s_out (p_t b - q_t)
    const float A = no_tail ? ws * 0.0f * all.s : ws * (p_t * b - l.q_tail) / out.s;
    const ExpRef ref(out.m, c);
    if (lane == 0) sh.unlisted = {ref.r, A * ref.k, 0.0f, ref.far};
    barrier_arrive<kScales, kListThreads>();
  }
  if (cl.rank == 0) {
    const float ln_s = logf(all.s);
    // logs of p_t and p themselves while there is something of them: log s is a few units, and its rounding would be
    // in every digit of a small divergence
    float tail = p_t > 1e-30f ? logf(p_t) : scaled_gap(out.m, all.m, a.scale, logf(out.s) - ln_s);
    if (no_tail) tail = all.s == all.s ? -kInf : nan_f();
    float loss = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      if (l.id[i] >= 0 && l.q[i] != 0.0f) {
        const float half = half_gap(l.x[i], all.m), p = expf(half * (2.0f * a.scale)) / all.s;
        // a small p's log by its logit, times q before the scale, which may take the log alone past fp32's range
        if (empty) loss += kInf;
        else if (p > 1e-30f) loss += l.q[i] * (l.lq[i] - logf(p));
        else loss += fmaf(-l.q[i] * half, 2.0f * a.scale, l.q[i] * (l.lq[i] + ln_s));
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) loss += __shfl_xor_sync(0xFFFFFFFFu, loss, off);
    if (lane == 0) {
      if (l.q_tail > 0.0f && !no_tail) loss += l.q_tail * (logf(l.q_tail) - tail);
      if (l.bad || !(all.s == all.s) || !(l.q_sum == l.q_sum)) loss = nan_f();
      if (a.loss) a.loss[row] = w * loss;
      if (a.norm) a.norm[row] = make_float2(all.m, all.s);
      if (a.tail) a.tail[row] = tail;
    }
  }
  if constexpr (GRAD) {
    const ExpRef top(all.m, c);
    const float over = top.k / all.s;
    barrier_sync<kWritten, kListThreads>();
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if ((mine >> i) & 1u)
        d[l.id[i]] = from_float<DT>(empty ? 0.0f : ws * fmaf(top.exp(l.x[i]) * over, b, -l.q[i]));
  }
}

// A row of weight 0: its zeros, by every block of its cluster.
template <int DT, bool GRAD>
__device__ __forceinline__ void skip_row(const DistillArgs& a, const Cluster& cl, int64_t row, Elem<DT>* d) {
  if (GRAD && threadIdx.x < kRowThreads) zero_part<DT>(d, a.vocab, cl.rank, cl.size);
  if (cl.rank == 0 && threadIdx.x == kRowThreads) {
    if (a.loss) a.loss[row] = 0.0f;
    if (a.norm) a.norm[row] = make_float2(0.0f, 0.0f);
    if (a.tail) a.tail[row] = 0.0f;
  }
  cl.started();
}

// Marks cleared by the row's warps before the list's sets its own.
__device__ __forceinline__ void clear_marks(uint32_t* marks, DistillShared& sh, int vectors) {
  for (int j = 0; j < vectors; j += kBatch) marks[j / kBatch * kRowThreads + threadIdx.x] = 0u;
  if (threadIdx.x == 0) sh.edge_listed = 0u;
  barrier_arrive<kClear, kListThreads>();
}

// Masks a batch's listed elements.
template <int DT>
__device__ __forceinline__ void mask_batch(uint4* v, uint32_t bits) {
  if (bits != 0u) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if ((bits >> (8 * u)) & 0xFFu) mask_elements<DT>(v[u], bits >> (8 * u));
  }
}

// BLOCKS: blocks an SM.
template <int DT, bool GRAD, int BLOCKS>
__global__ void __launch_bounds__(kListThreads, BLOCKS) distill_kernel(const __grid_constant__ DistillArgs a) {
  extern __shared__ uint32_t marks[];
  __shared__ DistillShared sh;
  const Cluster cl = Cluster::start();
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / cl.size;
  const Elem<DT>* x = static_cast<const Elem<DT>*>(a.x) + row * a.ld;
  Elem<DT>* d = static_cast<Elem<DT>*>(a.d) + row * a.d_ld;
  const float c = a.c;
  RowList<DT> l;
  if (tid >= kRowThreads) l.start(a, row);
  const float w = a.weight ? a.weight[row] : 1.0f;
  const RowPart<DT> part(x, a.vocab, cl.rank, cl.size);
  const int vectors = part.vectors();
  const int64_t sb = part.step_bytes();
  const char* src = part.at();
  auto fetch = [&](const char* p, int j, uint4 (&v)[kBatch]) {
    if (j + kBatch <= part.whole) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) v[u] = load_row<GRAD>(p + u * sb);
    } else {
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        v[u] = part.more(j + u) ? load_row<GRAD>(p + u * sb)
                                : make_uint4(kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>);
    }
  };
  uint4 v[kBatch];
  if (tid < kRowThreads) fetch(src, 0, v);  // on its way while the weight is
  if (w == 0.0f) return skip_row<DT, GRAD>(a, cl, row, d);
  if (tid >= kRowThreads) return list_warp<DT, GRAD>(a, cl, part, row, w, l, x, d, sh, marks);
  clear_marks(marks, sh, vectors);
  const float edge = part.edge >= 0 ? to_float<DT>(x[part.edge]) : -kInf;
  barrier_sync<kReady, kListThreads>();
  const bool edge_out = part.edge >= 0 && !((sh.edge_listed >> tid) & 1u);
  RunningMass out(one_element(edge_out ? edge : -kInf), c);
  const uint32_t* listed = marks + tid;
#pragma unroll 1
  for (int j = 0; j < vectors; j += kBatch, listed += kRowThreads) {
    uint4 next[kBatch];
    src += kBatch * sb;
    fetch(src, j + kBatch, next);
    mask_batch<DT>(v, *listed);
    add_mass<DT>(v, c, out);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) v[u] = next[u];
  }
  const RowSum warp_out = merge_lanes(out.done(c), c);
  if ((tid & 31) == 0) sh.red[tid >> 5] = warp_out;
  barrier_arrive<kAdded, kListThreads>();
  cl.started();
  if (cl.size > 1) cl.arrive();
  if constexpr (GRAD) {
    part.load(0, v);
    barrier_sync<kScales, kListThreads>();
    sh.unlisted.map<DT>(part, c, v, d, a.vec, edge);
    barrier_arrive<kWritten, kListThreads>();
  }
  if (cl.size > 1) cl.wait();
}

// ------------------------------------------------------------------ the gradient from saved normalisers
//
// One pass: blocks share a row as above, but nothing is exchanged between them.
// A ninth warp has the list while the first vectors are on their way. Bound by HBM:
// 2048 x 128256 bf16 165 us, 6.4 TB/s, 0.94 of the copy (parts of 16, 32, 64 vectors
// a thread: 172, 166, 170 us: every part looks its list up).
template <int DT>
__global__ void __launch_bounds__(kListThreads, 4) distill_grad_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ int4 list_ids[SS_MAX_TOP / 4];
  __shared__ Unlisted unlisted;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const unsigned rank = blockIdx.x % a.split;
  const int64_t row = blockIdx.x / a.split;
  const Elem<DT>* x = static_cast<const Elem<DT>*>(a.x) + row * a.ld;
  Elem<DT>* d = static_cast<Elem<DT>*>(a.d) + row * a.d_ld;
  RowList<DT> l;
  if (tid >= kRowThreads) l.start(a, row);
  const float wt = a.weight ? a.weight[row] : 1.0f, dl = a.d_loss ? a.d_loss[row] : 1.0f;
  const float2 norm = a.norm_in[row];
  const RowPart<DT> part(x, a.vocab, rank, a.split);
  uint4 first[kBatch];
  if (tid < kRowThreads) part.load(0, first);  // on its way while the row's scalars are
  if (wt == 0.0f || dl == 0.0f || norm.y == 0.0f) {
    if (tid < kRowThreads) zero_part<DT>(d, a.vocab, rank, a.split);
    return;
  }
  if (tid < kRowThreads) {
    const float edge = part.edge >= 0 ? to_float<DT>(x[part.edge]) : 0.0f;
    barrier_sync<kScales, kListThreads>();
    unlisted.map<DT>(part, a.c, first, d, a.vec, edge);
    barrier_arrive<kWritten, kListThreads>();
    return;
  }
  l.look_up(a, x, list_ids);
  l.drop_repeated(a, list_ids);
  l.sums(a);
  const float ws = l.bad ? nan_f() : wt * dl * a.scale;
  const float b = l.q_sum + l.q_tail;
  // p = k 2^arg / s; with the bucket the unlisted take (p / p_t) (p_t b - q_t), p_t inside the exponent where it is
  // so small that the exponentials without it would vanish
  const ExpRef ref(norm.x, a.c);
  const float over = ref.k / norm.y;
  float A = ws * b * over, lift = 0.0f;
  if (a.mode == SS_TAIL_BUCKET) {
    const float tail = a.tail_in[row], p_t = expf(tail);
    if (tail == -kInf) {
      A = ws * 0.0f * norm.y;  // NaN for a row that is
    } else if (tail > -60.0f) {
      A = ws * (p_t * b - l.q_tail) * (over / p_t);
    } else {
      A = ws * (p_t * b - l.q_tail) * over;
      lift = -tail * kLog2e;
    }
  }
  if ((tid & 31) == 0) unlisted = {ref.r, A, lift, ref.far};
  float g[kSlots];
  if (a.in_place) {  // the logits have to be here before the other warps write over them
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      g[i] = ws * fmaf(ref.exp(l.x[i]) * over, b, -l.q[i]);
      asm volatile("" ::"f"(g[i]) : "memory");
    }
  }
  barrier_arrive<kScales, kListThreads>();
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    int owner, slot;
    if (l.id[i] >= 0 && !part.owns(l.id[i], &owner, &slot)) l.id[i] = -1;
    if (!a.in_place) g[i] = ws * fmaf(ref.exp(l.x[i]) * over, b, -l.q[i]);
  }
  barrier_sync<kWritten, kListThreads>();
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (l.id[i] >= 0) d[l.id[i]] = from_float<DT>(g[i]);
}

ss_status distill_impl(const ss_logits* x, const ss_teacher* t, const float* norm_in, const float* tail_in,
                       const float* d_loss, float* loss, float* norm, float* tail, void* d_logits, int64_t d_ld,
                       void* stream) {
  const bool saved = norm_in != nullptr;
  int64_t x_bytes = 0;
  ss_status st = check_logits(x, &x_bytes);
  if (st != SS_OK) return st;
  if (!t->ids || !t->logprob || t->k < 1 || t->k > SS_MAX_TOP) return SS_ERR_INVALID_ARG;
  if (!(t->scale > 0.0f) || !std::isfinite(t->scale)) return SS_ERR_INVALID_ARG;
  if (t->tail != SS_TAIL_DROP && t->tail != SS_TAIL_RENORM && t->tail != SS_TAIL_BUCKET) return SS_ERR_INVALID_ARG;
  if ((t->idtype != SS_I32 && t->idtype != SS_I64) || !is_float_dtype(t->dtype)) return SS_ERR_DTYPE;
  if (x->vocab > SS_MAX_DISTILL_VOCAB || x->rows > INT32_MAX) return SS_ERR_OVERFLOW;
  const int64_t rows = x->rows, ib = t->idtype == SS_I64 ? 8 : 4;
  if (misaligned(t->ids, ib) || misaligned(t->logprob, dtype_bytes(t->dtype)) || misaligned(t->row_weight, 4) ||
      misaligned(loss, 4) || misaligned(norm, 8) || misaligned(tail, 4) || misaligned(norm_in, 8) ||
      misaligned(tail_in, 4) || misaligned(d_loss, 4))
    return SS_ERR_ALIGN;
  Ranges ranges;
  if (d_logits) {
    st = check_grad_out(x, x_bytes, d_logits, d_ld, &ranges);
    if (st != SS_OK) return st;
  } else {
    ranges.add(x->data, x_bytes, false);
  }
  ranges.add(t->ids, rows * t->k * ib, false);
  ranges.add(t->logprob, rows * t->k * dtype_bytes(t->dtype), false);
  ranges.add(t->row_weight, rows * 4, false);
  ranges.add(loss, rows * 4, true);
  ranges.add(norm, rows * 8, true);
  ranges.add(tail, rows * 4, true);
  ranges.add(norm_in, rows * 8, false);
  ranges.add(tail_in, rows * 4, false);
  ranges.add(d_loss, rows * 4, false);
  if (ranges.overlap()) return SS_ERR_OVERLAP;
  const int64_t vec = x->dtype == SS_FP32 ? 4 : 8, nvec = x->vocab / vec;
  const int split = split_for(nvec, 32);
  const Scale2 s2(x->scale);
  DistillArgs a = {x->data, t->ids, t->logprob, t->row_weight, d_loss, reinterpret_cast<const float2*>(norm_in),
                   tail_in, loss, reinterpret_cast<float2*>(norm), tail, d_logits, rows, x->vocab, x->ld, d_ld, s2.c,
                   s2.eps, x->scale, t->scale, t->k, t->tail, t->dtype, t->idtype == SS_I64,
                   d_logits && same_phase(x, d_logits, d_ld), d_logits == x->data, static_cast<uint32_t>(split), 0};
  if (saved) {
    auto* fn = x->dtype == SS_BF16
                   ? distill_grad_kernel<SS_BF16>
                   : (x->dtype == SS_FP16 ? distill_grad_kernel<SS_FP16> : distill_grad_kernel<SS_FP32>);
    if (rows * split > INT32_MAX) return SS_ERR_OVERFLOW;
    return launch(fn, static_cast<unsigned>(rows * split), a, stream, kListThreads);
  }
  const auto pick = [&](auto grad, auto blocks) {
    constexpr bool kGrad = decltype(grad)::value;
    constexpr int kBlocks = decltype(blocks)::value;
    return x->dtype == SS_BF16 ? distill_kernel<SS_BF16, kGrad, kBlocks>
                               : (x->dtype == SS_FP16 ? distill_kernel<SS_FP16, kGrad, kBlocks>
                                                      : distill_kernel<SS_FP32, kGrad, kBlocks>);
  };
  constexpr std::integral_constant<int, 3> three;
  constexpr std::integral_constant<int, 4> four;
  const auto vectors = [&](int n) { return (nvec + n * kRowThreads - 1) / (n * kRowThreads); };
  int cluster = 1;
  while (cluster < kMaxCluster && vectors(cluster) > kPartVectors) cluster *= 2;
  // few rows: smaller parts, as long as all of them run at once
  const int64_t places = 4 * sm_count();
  const bool few = rows * cluster * 2 <= places;
  while (cluster < kMaxCluster && rows * cluster * 2 <= places && vectors(cluster) > kFewVectors) cluster *= 2;
  const int blocks = d_logits && !few ? 3 : 4;
  auto* fn = !d_logits ? pick(std::false_type(), four)
                       : (few ? pick(std::true_type(), four) : pick(std::true_type(), three));
  const size_t smem = static_cast<size_t>((vectors(cluster) + kBatch - 1) / kBatch) * kRowThreads * sizeof(uint32_t);
  if (rows * cluster > INT32_MAX) return SS_ERR_OVERFLOW;
  a.resident = blocks * sm_count() / cluster;
  return launch_rows(fn, rows, cluster, kListThreads, smem, a, stream);
}

}  // namespace
}  // namespace ss

extern "C" {

ss_status ss_distill_topk(const ss_logits* x, const ss_teacher* teacher, float* loss, float* norm,
                          float* tail_logprob, void* d_logits, int64_t d_ld, void* stream) {
  if (!x || !teacher || x->rows < 0) return SS_ERR_INVALID_ARG;
  if (x->rows == 0) return SS_OK;
  if (!loss && !norm && !tail_logprob && !d_logits) return SS_ERR_INVALID_ARG;
  return ss::distill_impl(x, teacher, nullptr, nullptr, nullptr, loss, norm, tail_logprob, d_logits, d_ld, stream);
}

ss_status ss_distill_topk_grad(const ss_logits* x, const ss_teacher* teacher, const float* norm,
                               const float* tail_logprob, const float* d_loss, void* d_logits, int64_t d_ld,
                               void* stream) {
  if (!x || !teacher || x->rows < 0) return SS_ERR_INVALID_ARG;
  if (x->rows == 0) return SS_OK;
  if (!norm || !d_logits) return SS_ERR_INVALID_ARG;
  if (teacher->tail == SS_TAIL_BUCKET && !tail_logprob) return SS_ERR_INVALID_ARG;
  return ss::distill_impl(x, teacher, norm, teacher->tail == SS_TAIL_BUCKET ? tail_logprob : nullptr, d_loss, nullptr,
                          nullptr, nullptr, d_logits, d_ld, stream);
}

}  // extern "C"
