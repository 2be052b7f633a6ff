// ss_distill.cu -- distillation from a teacher's top log probabilities: loss and
// gradient in one call (ss_distill_topk), and the gradient from saved
// normalisers (ss_distill_topk_grad).
#include "ss_logits.cuh"

namespace ss {
namespace {

#ifndef SS_PART_VECTORS
#define SS_PART_VECTORS 16
#endif
constexpr int kPartVectors = SS_PART_VECTORS;

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
  float c, scale, t_scale;
  int32_t k, mode, t_dtype;
  bool wide, vec;
  uint32_t split;   // gradient from saved normalisers: blocks that share a row
  int32_t batches;  // of vectors a thread holds
};

__device__ __forceinline__ float load_teacher(const void* p, int64_t i, int dtype) {
  if (dtype == SS_FP32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == SS_BF16 ? widen1<SS_BF16>(h) : widen1<SS_FP16>(h);
}

// ------------------------------------------------------------------ a row's list
//
// Thread j < k holds slot j. The list's sums come in three steps around barriers
// that the callers place other work between: list_unique (which slots count),
// list_partials (per warp), list_sums (after a barrier).

constexpr int kListWarps = SS_MAX_TOP / 32;

struct ListShared {
  int4 id[SS_MAX_TOP / 4];      // -1: unused
  uint8_t again[SS_MAX_TOP];    // slots whose id occurs earlier in the list
  RowMass in[kListWarps];       // the listed tokens' mass
  RowMass teacher[kListWarps];  // SS_TAIL_RENORM: mass of the teacher's values
  float2 q[kListWarps];         // else: sum of q as a pair
};

struct Slot {
  int32_t id;  // -1: unused
  float lq;    // log q, before SS_TAIL_RENORM's normalisation
  float x;     // the token's logit
};

struct ListSums {
  float shift;   // what log q is short of: log q = lq - shift
  float q_sum;   // Q
  float q_tail;  // q_t
};

// The calling thread's slot as given (x not yet); *past: its id is past the vocabulary.
__device__ __forceinline__ Slot list_fetch(const DistillArgs& a, int64_t row, bool* past) {
  Slot s = {-1, -kInf, -kInf};
  *past = false;
  if (threadIdx.x < a.k) {
    const int64_t at = row * a.k + threadIdx.x;
    const int64_t id = load_id(a.ids, at, a.wide);
    s.lq = load_teacher(a.teacher, at, a.t_dtype) * a.t_scale;
    *past = id >= a.vocab;
    if (id >= 0 && id < a.vocab) s.id = static_cast<int32_t>(id);
  }
  return s;
}

// After the slots' ids are in l.id and a barrier: finds the repeated ones, two threads a slot (a barrier follows,
// then list_drop).
__device__ __forceinline__ void list_unique(const DistillArgs& a, ListShared& l) {
  static_assert(kRowThreads == 2 * SS_MAX_TOP, "two threads a slot");
  const int j = threadIdx.x >> 1;
  if (j < a.k) {  // k threads pairs, so whole pairs
    const int32_t* ids = &l.id[0].x;
    const int32_t mine = ids[j];
    int again = 0;
    for (int q = threadIdx.x & 1; 4 * q < j; q += 2) {
      const int4 v = l.id[q];
      again |= (v.x == mine) | ((v.y == mine) & (4 * q + 1 < j)) | ((v.z == mine) & (4 * q + 2 < j)) |
               ((v.w == mine) & (4 * q + 3 < j));
    }
    const unsigned pair = 3u << (threadIdx.x & 30);
    again |= __shfl_xor_sync(pair, again, 1);
    if ((threadIdx.x & 1) == 0) l.again[j] = static_cast<uint8_t>(again);
  }
}

__device__ __forceinline__ void list_drop(const DistillArgs& a, const ListShared& l, Slot& s) {
  if (threadIdx.x < a.k && (s.id < 0 || l.again[threadIdx.x])) s.id = -1;
  if (s.id < 0) s.lq = -kInf;
}

// The warps' partial sums (a barrier follows).
__device__ __forceinline__ void list_partials(const DistillArgs& a, ListShared& l, const Slot& s) {
  if (threadIdx.x >= SS_MAX_TOP) return;
  const int warp = threadIdx.x >> 5;
  auto one = [](float v, bool used) {  // the mass of one value
    if (!used || v == -kInf) return RowMass::none();
    return v <= 3.402823466e38f ? RowMass{v, 1.0f} : RowMass{-kInf, nan_f()};
  };
  const RowMass in = merge_lanes(one(s.x, s.id >= 0), a.c);
  if ((threadIdx.x & 31) == 0) l.in[warp] = in;
  if (a.mode == SS_TAIL_RENORM) {
    const RowMass t = merge_lanes(one(s.lq, s.id >= 0), kLog2e);
    if ((threadIdx.x & 31) == 0) l.teacher[warp] = t;
  } else {
    // q_t = 1 - Q is small when the list has nearly all the mass: Q is added as a pair
    dd q = {expf(s.lq), 0.0f};
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float h = __shfl_xor_sync(0xFFFFFFFFu, q.hi, off), lo = __shfl_xor_sync(0xFFFFFFFFu, q.lo, off);
      const dd t = two_sum(q.hi, h);
      q = {t.hi, t.lo + (q.lo + lo)};
    }
    if ((threadIdx.x & 31) == 0) l.q[warp] = make_float2(q.hi, q.lo);
  }
}

__device__ __forceinline__ ListSums list_sums(const DistillArgs& a, const ListShared& l) {
  ListSums o = {0.0f, 0.0f, 0.0f};
  if (a.mode == SS_TAIL_RENORM) {
    const RowMass t = merge_lanes(l.teacher[threadIdx.x % kListWarps], kLog2e, kListWarps);
    if (t.s != 0.0f) {
      o.shift = t.m + logf(t.s);
      o.q_sum = t.s == t.s ? 1.0f : t.s;
    }
  } else {
    dd q = {l.q[0].x, l.q[0].y};
#pragma unroll
    for (int i = 1; i < kListWarps; ++i) {
      const dd t = two_sum(q.hi, l.q[i].x);
      q = {t.hi, t.lo + (q.lo + l.q[i].y)};
    }
    o.q_sum = q.hi + q.lo;
    if (a.mode == SS_TAIL_BUCKET) {
      const float rest = (1.0f - q.hi) - q.lo;
      o.q_tail = rest <= 0.0f ? 0.0f : rest;
    }
  }
  return o;
}

// ------------------------------------------------------------------ loss and gradient in one call
//
// The gradient needs the row's sums and then the row again. A row is shared by
// the blocks of a cluster, each holding its part in shared memory: the logits
// are read from HBM once, with asynchronous copies that are all issued at the
// start, and the gradient is computed from shared memory and written once. The
// grid is one wave of clusters that go through the rows; a thread that has read
// a batch for the last time starts the copy of the next row's batch into its
// place, so the next row arrives while this one's gradient is written (or, for
// the loss alone, while the row's other batches are added up). Two to four
// blocks fit an SM, and one's sums and barriers pass under another's traffic.
//
// The listed tokens are left out of the first pass (a bit per element of the
// part says which they are), so the unlisted mass is a sum of its own terms and
// not a difference: log p_t keeps its digits however little is left. Their
// logits come with the list; their gradients are written last, over what the
// second pass put there.

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

template <int DT>
constexpr uint32_t kMaskedWord = DT == SS_FP32 ? 0xFF800000u : (DT == SS_BF16 ? 0xFF80FF80u : 0xFC00FC00u);

// N vectors into the running sum, `ref` being that of acc.m.
template <int DT, int N>
__device__ __forceinline__ void add_mass(const uint4 (&w)[N], float c, RowMass& acc, ExpRef& ref) {
  float m = vec_max<DT>(w[0]);
#pragma unroll
  for (int u = 1; u < N; ++u) m = fmaxf(m, vec_max<DT>(w[u]));
  if (m > acc.m) {
    acc.move(m, c);
    ref = ExpRef(m, c);
  }
  Pair s = Pair::both(0.0f);
#pragma unroll
  for (int u = 0; u < N; ++u) {
    Pair f[kPairsOf<DT>];
    unpack_pairs<DT>(w[u], f);
#pragma unroll
    for (int j = 0; j < kPairsOf<DT>; ++j) s = add2(s, ex2_pair(ref.arg(f[j])));
  }
  acc.s = fmaf(s.sum(), ref.k, acc.s);
}

// Dynamic shared memory: the part's vectors [batches * kBatch][T], then a byte of listed bits for each, by thread.
// SIZE: blocks of the cluster.
template <int DT, bool GRAD, int SIZE>
__global__ void __launch_bounds__(kRowThreads, 3) distill_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int V = kVecOf<DT>;
  extern __shared__ uint4 held[];
  __shared__ RowMass red[kRowWarps];
  __shared__ RowMass parts[2][kMaxCluster];  // by turns: a block may be one row ahead of another's reading
  __shared__ ListShared l;
  __shared__ float part_loss[kListWarps];
  __shared__ uint32_t edge_listed;
  Cluster cl = Cluster::start();
  cl.size = SIZE;
  using Part = RowPart<DT, SIZE>;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t clusters = gridDim.x / cl.size;
  const float c = a.c;
  auto row_x = [&](int64_t row) { return static_cast<const Elem<DT>*>(a.x) + row * a.ld; };
  auto row_d = [&](int64_t row) { return static_cast<Elem<DT>*>(a.d) + row * a.d_ld; };
  auto weight = [&](int64_t row) { return a.weight && row < a.rows ? a.weight[row] : 1.0f; };
  // The first row from `row` on, of this cluster's, that counts (w: its weight); those before it get their zeros.
  auto next_live = [&](int64_t row, float* w) {
    while (row < a.rows && *w == 0.0f) {
      if (GRAD) zero_part<DT>(row_d(row), a.vocab, cl.rank, cl.size);
      if (cl.rank == 0 && tid == 0) {
        if (a.loss) a.loss[row] = 0.0f;
        if (a.norm) a.norm[row] = make_float2(0.0f, 0.0f);
        if (a.tail) a.tail[row] = 0.0f;
      }
      row += clusters;
      *w = weight(row);
    }
    return row;
  };
  auto copy_batch = [&](const Part& part, int q) {
    const char* src = part.at() + q * kBatch * part.step_bytes();
    uint4* h = held + q * kBatch * kRowThreads + tid;
    if ((q + 1) * kBatch <= part.whole) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) copy_async16(h + u * kRowThreads, src + u * part.step_bytes());
    } else {
#pragma unroll 1
      for (int u = 0; u < kBatch && part.more(q * kBatch + u); ++u)
        copy_async16(h + u * kRowThreads, src + u * part.step_bytes());
    }
  };
  // Rows differ by their 16-byte phase alone, so by one vector: the buffer has room for the longer ones.
  const int held_batches = a.batches;
  uint32_t* listed = reinterpret_cast<uint32_t*>(held + static_cast<size_t>(held_batches) * kBatch * kRowThreads);
  const int quarter = (held_batches + 3) / 4;

  int64_t row = blockIdx.x / cl.size;
  float w = weight(row);
  row = next_live(row, &w);
  bool past = false;
  Slot s = {-1, -kInf, -kInf};
  float edge = -kInf;
  Part part(row_x(row < a.rows ? row : 0), a.vocab, cl.rank, cl.size);
  if (row < a.rows) {
    s = list_fetch(a, row, &past);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      for (int q = g * quarter; q < min((g + 1) * quarter, held_batches); ++q) copy_batch(part, q);
      copies_commit();
    }
    if (part.edge >= 0) edge = to_float<DT>(part.x[part.edge]);
  }
  cl.started();
  for (int turn = 0; row < a.rows; turn ^= 1) {
    const Elem<DT>* x = part.x;
    Elem<DT>* d = row_d(row);
    float next_w = weight(row + clusters);
    for (int q = 0; q < held_batches; ++q) listed[q * kRowThreads + tid] = 0u;
    if (tid == 0) edge_listed = 0u;
    if (tid < SS_MAX_TOP) (&l.id[0].x)[tid] = s.id;
    const bool bad = __syncthreads_or(past);
    int owner = 0, slot = 0;
    bool mine = s.id >= 0 && part.owns(s.id, &owner, &slot);
    if (s.id >= 0) s.x = to_float<DT>(x[s.id]);
    if (mine) {
      if (slot < 0) atomicOr(&edge_listed, 1u << owner);
      else atomicOr(&listed[(slot / kBatch) * kRowThreads + owner],
                    1u << (slot % kBatch * 8 + (s.id - part.sl.head) % V));
    }
    list_unique(a, l);
    __syncthreads();
    list_drop(a, l, s);
    mine = mine && s.id >= 0;

    // the next row, its list, and (loss alone) its copies as this row's batches are done with
    int64_t next = row + clusters;
    bool next_past = false;
    Slot next_s = {-1, -kInf, -kInf};
    float next_edge = -kInf;
    Part next_part = part;
    auto look_ahead = [&] {
      next = next_live(next, &next_w);
      if (next < a.rows) {
        next_part = Part(row_x(next), a.vocab, cl.rank, cl.size);
        next_s = list_fetch(a, next, &next_past);
        if (next_part.edge >= 0) next_edge = to_float<DT>(next_part.x[next_part.edge]);
      }
    };
    if (!GRAD) look_ahead();

    RowMass out = RowMass::none();  // unlisted tokens
    if (part.edge >= 0 && !((edge_listed >> tid) & 1u)) {
      if (edge > out.m) out.m = edge;
      out.s = edge == -kInf ? 0.0f : (edge <= 3.402823466e38f ? 1.0f : nan_f());
    }
    ExpRef ref(out.m, c);
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
      // copies still under way: this row's later quarters, and (loss alone) the next row's earlier ones
      if (!GRAD || g == 0) copies_wait<3>();
      else if (g == 1) copies_wait<2>();
      else if (g == 2) copies_wait<1>();
      else copies_wait<0>();
#pragma unroll 1
      for (int q = g * quarter; q < min((g + 1) * quarter, held_batches); ++q) {
        const uint4* h = held + q * kBatch * kRowThreads + tid;
        const uint32_t bits = listed[q * kRowThreads + tid];
        if ((q + 1) * kBatch <= part.whole) {
          uint4 v[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) v[u] = h[u * kRowThreads];
          if (bits != 0u) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) mask_elements<DT>(v[u], (bits >> (8 * u)) & 0xFFu);
          }
          add_mass<DT>(v, c, out, ref);
        } else {
#pragma unroll 1
          for (int u = 0; u < kBatch && part.more(q * kBatch + u); ++u) {
            uint4 v[1] = {h[u * kRowThreads]};
            mask_elements<DT>(v[0], (bits >> (8 * u)) & 0xFFu);
            add_mass<DT>(v, c, out, ref);
          }
        }
        if (!GRAD && next < a.rows) {
          // the sums that the held vectors went into are formed before their place is given away
          asm volatile("" ::"f"(out.s) : "memory");
          copy_batch(next_part, q);
        }
      }
      if (!GRAD) copies_commit();
    }
    list_partials(a, l, s);
    out = block_merge(out, c, red);
    if (cl.size > 1) {
      if (tid < cl.size) cl.at(parts[turn], tid)[cl.rank] = out;
      cl.arrive();
    }
    RowMass all = merge_lanes(l.in[tid % kListWarps], c, kListWarps);
    const ListSums sums = list_sums(a, l);
    const float lq = s.lq - sums.shift, q = expf(lq);
    if (cl.size > 1) {
      cl.wait();
      out = merge_lanes(parts[turn][tid % cl.size], c, static_cast<int>(cl.size));
    }
    {
      const float top = fmaxf(all.m, out.m);
      RowMass o = out;
      if (top > all.m) all.move(top, c);
      if (top > o.m) o.move(top, c);
      all.s += o.s;
    }
    const bool empty = all.s == 0.0f;
    // all unlisted tokens masked, by -inf or by values so low that no p_t is left
    const bool no_tail = out.s == 0.0f || (out.m - all.m) * c <= kFloor;
    if (cl.rank == 0) {
      const float ln_s = logf(all.s);
      const float tail = no_tail ? -kInf : fmaf(out.m - all.m, a.scale, logf(out.s) - ln_s);
      float term = 0.0f;
      if (s.id >= 0 && q != 0.0f) {
        const float lp = empty ? -kInf : fmaf(s.x - all.m, a.scale, -ln_s);
        term = q * (lq - lp);
      }
      if (tid < SS_MAX_TOP) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, off);
        if ((tid & 31) == 0) part_loss[tid >> 5] = term;
      }
      __syncthreads();
      if (tid == 0) {
        float loss = 0.0f;
        for (int i = 0; i < kListWarps; ++i) loss += part_loss[i];
        if (sums.q_tail > 0.0f && !no_tail) loss += sums.q_tail * (logf(sums.q_tail) - tail);
        if (bad || !(all.s == all.s) || !(sums.q_sum == sums.q_sum)) loss = nan_f();
        if (a.loss) a.loss[row] = w * loss;
        if (a.norm) a.norm[row] = make_float2(all.m, all.s);
        if (a.tail) a.tail[row] = tail;
      }
    }
    if constexpr (GRAD) {
      look_ahead();
      const float ws = bad ? nan_f() : w * a.scale;
      const float b = sums.q_sum + sums.q_tail;
      // unlisted: (p / p_t) (p_t b - q_t) = 2^((x - m_out) c) / s_out (p_t b - q_t)
      const float p_t = no_tail ? 0.0f : ex2((out.m - all.m) * c) * (out.s / all.s);
      const float A = no_tail ? ws * 0.0f * all.s : ws * (p_t * b - sums.q_tail) / out.s;
      const ExpRef outer(out.m, c);
      const float B = A * outer.k;
      if (part.edge >= 0) d[part.edge] = from_float<DT>(outer.exp(edge) * B);
      char* dst = part.at(d);
      auto put = [&](const uint4& v, char* o) {
        Pair p[kPairsOf<DT>];
        unpack_pairs<DT>(v, p);
#pragma unroll
        for (int e = 0; e < kPairsOf<DT>; ++e) p[e] = mul2(ex2_pair(outer.arg(p[e])), Pair::both(B));
        store_vector<DT>(o, p, a.vec);
      };
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
#pragma unroll 1
        for (int r = g * quarter; r < min((g + 1) * quarter, held_batches); ++r) {
          const uint4* h = held + r * kBatch * kRowThreads + tid;
          if ((r + 1) * kBatch <= part.whole) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) put(h[u * kRowThreads], dst + u * part.step_bytes());
          } else {
#pragma unroll 1
            for (int u = 0; u < kBatch && part.more(r * kBatch + u); ++u)
              put(h[u * kRowThreads], dst + u * part.step_bytes());
          }
          dst += kBatch * part.step_bytes();
          if (next < a.rows) copy_batch(next_part, r);
        }
        copies_commit();
      }
      __syncthreads();
      if (mine) {
        const ExpRef top(all.m, c);
        d[s.id] = from_float<DT>(empty ? 0.0f : ws * fmaf(top.exp(s.x) * (top.k / all.s), b, -q));
      }
    }
    row = next;
    w = next_w;
    s = next_s;
    past = next_past;
    edge = next_edge;
    part = next_part;
  }
}

// ------------------------------------------------------------------ the gradient from saved normalisers
//
// One pass: blocks share a row as above, but nothing is exchanged between them.
// The list's sums are taken while the first vectors are on their way.
template <int DT>
__global__ void __launch_bounds__(kRowThreads, 4) distill_grad_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ ListShared l;
  pdl_wait();
  pdl_trigger();
  const unsigned rank = blockIdx.x % a.split;
  const int64_t row = blockIdx.x / a.split;
  const Elem<DT>* x = static_cast<const Elem<DT>*>(a.x) + row * a.ld;
  Elem<DT>* d = static_cast<Elem<DT>*>(a.d) + row * a.d_ld;
  const float wt = a.weight ? a.weight[row] : 1.0f, dl = a.d_loss ? a.d_loss[row] : 1.0f;
  const float2 norm = a.norm_in[row];
  bool past;
  Slot s = list_fetch(a, row, &past);
  if (wt == 0.0f || dl == 0.0f || norm.y == 0.0f) {
    zero_part<DT>(d, a.vocab, rank, a.split);
    return;
  }
  const RowPart<DT> part(x, a.vocab, rank, a.split);
  uint4 first[kBatch];
  part.load(0, first);
  const float edge = part.edge >= 0 ? to_float<DT>(x[part.edge]) : 0.0f;
  if (threadIdx.x < SS_MAX_TOP) (&l.id[0].x)[threadIdx.x] = s.id;
  const bool bad = __syncthreads_or(past);
  int owner, slot;
  const bool mine = s.id >= 0 && part.owns(s.id, &owner, &slot);
  if (mine) s.x = to_float<DT>(x[s.id]);
  list_unique(a, l);
  __syncthreads();
  list_drop(a, l, s);
  list_partials(a, l, s);
  __syncthreads();
  const ListSums sums = list_sums(a, l);
  const float ws = bad ? nan_f() : wt * dl * a.scale;
  const float b = sums.q_sum + sums.q_tail;
  // p = k 2^arg / s; with the bucket the unlisted take (p / p_t) (p_t b - q_t), p_t inside the exponent where it is
  // so small that the exponentials without it would vanish
  const ExpRef ref(norm.x, a.c);
  const float over = ref.k / norm.y;
  float A = ws * b * over, r = ref.r;
  if (a.mode == SS_TAIL_BUCKET) {
    const float tail = a.tail_in[row], p_t = expf(tail);
    if (tail == -kInf) {
      A = ws * 0.0f;
    } else if (tail > -60.0f) {
      A = ws * (p_t * b - sums.q_tail) * (over / p_t);
    } else {
      A = ws * (p_t * b - sums.q_tail) * over;
      r = fmaf(tail, kLog2e, r);
    }
  }
  const float rc = ref.c;
  part.map(first, d, a.vec, edge, [&](Pair f) {
    return mul2(ex2_pair(fma2(f, Pair::both(rc), Pair::both(-r))), Pair::both(A));
  });
  __syncthreads();
  if (mine && s.id >= 0)
    d[s.id] = from_float<DT>(ws * fmaf(ref.exp(s.x) * over, b, -expf(s.lq - sums.shift)));
}

template <bool GRAD, int DT>
auto distill_of_size(int cluster) {
  return cluster == 1   ? distill_kernel<DT, GRAD, 1>
         : cluster == 2 ? distill_kernel<DT, GRAD, 2>
         : cluster == 4 ? distill_kernel<DT, GRAD, 4>
                        : distill_kernel<DT, GRAD, 8>;
}
template <bool GRAD>
auto distill_for(int32_t dtype, int cluster) {
  return dtype == SS_BF16   ? distill_of_size<GRAD, SS_BF16>(cluster)
         : dtype == SS_FP16 ? distill_of_size<GRAD, SS_FP16>(cluster)
                            : distill_of_size<GRAD, SS_FP32>(cluster);
}

// Clusters of `cluster` blocks of `fn` that the GPU holds at once with `smem` bytes of dynamic shared memory, which
// are allowed to it here (kept per device, kernel and size, without allocation).
ss_status resident_clusters(const void* fn, size_t smem, int cluster, int* out) {
  struct Entry {
    int dev, cluster;
    const void* fn;
    size_t smem;
    int clusters;
  };
  static std::mutex mu;
  static Entry cache[64] = {};
  static int used = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < std::min(used, 64); ++i) {
    const Entry& c = cache[i];
    if (c.dev == dev && c.fn == fn && c.smem == smem && c.cluster == cluster) {
      *out = c.clusters;
      return SS_OK;
    }
  }
  // the limit only grows: another thread may be about to launch with a larger size
  cudaFuncAttributes now;
  e = cudaFuncGetAttributes(&now, fn);
  if (e != cudaSuccess) return cuda_fail(e);
  if (static_cast<size_t>(now.maxDynamicSharedSizeBytes) < smem) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return cuda_fail(e);
  }
  int n = 0;
  if (cluster == 1) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, kRowThreads, smem);
    n *= sm_count();
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
  }
  if (e != cudaSuccess) return cuda_fail(e);
  n = std::max(n, 1);
  cache[used++ % 64] = {dev, cluster, fn, smem, n};
  *out = n;
  return SS_OK;
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
  const int split = split_for(nvec);
  DistillArgs a = {x->data, t->ids, t->logprob, t->row_weight, d_loss,
                         reinterpret_cast<const float2*>(norm_in), tail_in, loss, reinterpret_cast<float2*>(norm),
                         tail, d_logits, rows, x->vocab, x->ld, d_ld, x->scale * kLog2e, x->scale, t->scale, t->k,
                         t->tail, t->dtype, t->idtype == SS_I64, d_logits && same_phase(x, d_logits, d_ld),
                         static_cast<uint32_t>(split), 0};
  if (saved) {
    auto* fn = x->dtype == SS_BF16
                   ? distill_grad_kernel<SS_BF16>
                   : (x->dtype == SS_FP16 ? distill_grad_kernel<SS_FP16> : distill_grad_kernel<SS_FP32>);
    if (rows * split > INT32_MAX) return SS_ERR_OVERFLOW;
    return launch(fn, static_cast<unsigned>(rows * split), a, stream, kRowThreads);
  }
  // a part of at most kPartVectors vectors a thread, or what 8 blocks leave
  const auto vectors = [&](int n) { return (nvec + n * kRowThreads - 1) / (n * kRowThreads); };
  int cluster = 1;
  while (cluster < kMaxCluster && vectors(cluster) > kPartVectors) cluster *= 2;
  auto* fn = d_logits ? distill_for<true>(x->dtype, cluster) : distill_for<false>(x->dtype, cluster);
  a.batches = static_cast<int>((vectors(cluster) + kBatch - 1) / kBatch);
  const size_t smem = static_cast<size_t>(a.batches) * kRowThreads * (kBatch * sizeof(uint4) + sizeof(uint32_t));
  int clusters = 0;
  st = resident_clusters(reinterpret_cast<const void*>(fn), smem, cluster, &clusters);
  if (st != SS_OK) return st;
  return launch_rows(fn, std::min<int64_t>(rows, clusters), cluster, smem, a, stream);
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
