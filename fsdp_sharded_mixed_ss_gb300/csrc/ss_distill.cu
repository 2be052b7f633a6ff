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
  bool wide, vec, in_place;
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
// One warp of the block has the list, lane i its slots i, i + 32, ...: it loads
// them and their logits, drops repeated ids, sums them up and writes their
// gradients, while the block's other warps go through the row's elements.

constexpr int kListThreads = kRowThreads + 32;  // the row's warps and the list's
constexpr int kSlots = SS_MAX_TOP / 32;

template <int DT>
struct RowList {
  int32_t id[kSlots];    // -1: unused
  float lq[kSlots];      // log q
  float q[kSlots];
  float x[kSlots];       // the token's logit
  RowMass in;            // the listed tokens' mass
  float q_sum, q_tail;   // Q and q_t
  bool bad;              // an id past the vocabulary

  // ids_shared: SS_MAX_TOP / 4 int4 of shared memory, this warp's own.
  __device__ __forceinline__ void load(const DistillArgs& a, int64_t row, const Elem<DT>* xr, int4* ids_shared) {
    const int lane = threadIdx.x & 31;
    bool past = false;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      id[i] = -1;
      lq[i] = x[i] = -kInf;
      const int j = lane + 32 * i;
      if (32 * i < a.k) {
        if (j < a.k) {
          const int64_t wide_id = load_id(a.ids, row * a.k + j, a.wide);
          lq[i] = load_teacher(a.teacher, row * a.k + j, a.t_dtype) * a.t_scale;
          past = past || wide_id >= a.vocab;
          if (wide_id >= 0 && wide_id < a.vocab) id[i] = static_cast<int32_t>(wide_id);
        }
        (&ids_shared[0].x)[j] = id[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (id[i] >= 0) x[i] = to_float<DT>(xr[id[i]]);
    bad = __any_sync(0xFFFFFFFFu, past);
    __syncwarp();
    // an id that an earlier slot has: of its own 32, or of those before them
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

  __device__ __forceinline__ static RowMass mass(const float (&v)[kSlots], float c) {
    RowMass m = one_element<RowMass>(v[0]);
#pragma unroll
    for (int i = 1; i < kSlots; ++i) {
      RowMass o = one_element<RowMass>(v[i]);
      if (o.m > m.m) m.move(o.m, c);
      else if (m.m > o.m) o.move(m.m, c);
      m.s += o.s;
    }
    return merge_lanes(m, c);
  }

  __device__ __forceinline__ void mass_in(const DistillArgs& a) { in = mass(x, a.c); }
  // log q, q, Q and q_t.
  __device__ __forceinline__ void sums(const DistillArgs& a) {
    q_sum = q_tail = 0.0f;
    if (a.mode == SS_TAIL_RENORM) {
      const RowMass t = mass(lq, kLog2e);
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
// the blocks of a cluster, each holding its part in shared memory: the logits
// are read from HBM once, with asynchronous copies, and the gradient is computed
// from shared memory and written once. The grid is one wave of clusters that go
// through the rows; a thread that has read a batch for the last time starts the
// copy of the next row's batch into its place, so the next row arrives while
// this one's gradient is written (or, for the loss alone, while the row's other
// batches are added up). Two to four blocks fit an SM, and one's sums and
// barriers pass under another's traffic.
//
// Eight warps go through the elements and do as little else as can be; the ninth
// has the row's list, the exchange between the blocks and the row's loss, and
// prepares the next row's list meanwhile. Per row:
//   ready   list -> row    the listed tokens are marked
//   added   row -> list    the warps' sums are in `red`
//   scales  list -> row    the gradient's factors are in `factor`
//   written row -> list    the gradient is written; the list's own goes on top
// The listed tokens are left out of the sums (a bit per element of the part says
// which they are), so the unlisted mass is a sum of its own terms and not a
// difference: log p_t keeps its digits however little is left.

enum Barrier : int { kReady = 1, kAdded = 3, kScales = 5, kWritten = 6 };  // kReady, kAdded: two each, by turns

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

using RunningMass = Running<RowMass, 40>;

// A batch of vectors into the running sum.
template <int DT>
__device__ __forceinline__ void add_mass(const uint4 (&w)[kBatch], float c, RunningMass& acc) {
  float m = vec_max<DT>(w[0]);
#pragma unroll
  for (int u = 1; u < kBatch; ++u) m = fmaxf(m, vec_max<DT>(w[u]));
  acc.see(m, c);
  Pair s = Pair::both(0.0f);
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    Pair f[kPairsOf<DT>];
    unpack_pairs<DT>(w[u], f);
#pragma unroll
    for (int j = 0; j < kPairsOf<DT>; ++j) s = add2(s, ex2_pair(acc.ref.arg(f[j])));
  }
  acc.at.s = fmaf(s.sum(), acc.ref.k, acc.at.s);
}

// Dynamic shared memory: the part's vectors [batches * kBatch][T], then a word of listed bits for each batch, by
// thread (twice for the loss alone, where a row's marks are set while the last one's are read).
// SIZE: blocks of the cluster.
template <int DT, bool GRAD, int SIZE>
__global__ void __launch_bounds__(kListThreads, 3) distill_kernel(const __grid_constant__ DistillArgs a) {
  extern __shared__ uint4 held[];
  __shared__ RowMass red[2][kRowWarps];
  __shared__ RowMass parts[2][kMaxCluster];  // by turns: a block may be one row ahead of another's reading
  __shared__ int4 list_ids[SS_MAX_TOP / 4];
  __shared__ float factor[3];
  __shared__ uint32_t edge_listed[2];
  Cluster cl = Cluster::start();
  cl.size = SIZE;
  using Part = RowPart<DT, SIZE>;
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t clusters = gridDim.x / SIZE;
  const float c = a.c;
  const int batches = a.batches;
  uint32_t* marks = reinterpret_cast<uint32_t*>(held + static_cast<size_t>(batches) * kBatch * kRowThreads);
  auto row_x = [&](int64_t row) { return static_cast<const Elem<DT>*>(a.x) + row * a.ld; };
  auto row_d = [&](int64_t row) { return static_cast<Elem<DT>*>(a.d) + row * a.d_ld; };
  auto weight = [&](int64_t row) { return a.weight && row < a.rows ? a.weight[row] : 1.0f; };
  // The first row from `row` on, of this cluster's, that counts (w: its weight); those before it get their zeros.
  auto next_live = [&](int64_t row, float* w) {
    while (row < a.rows && *w == 0.0f) {
      if (GRAD && tid < kRowThreads) zero_part<DT>(row_d(row), a.vocab, cl.rank, SIZE);
      if (cl.rank == 0 && tid == kRowThreads) {
        if (a.loss) a.loss[row] = 0.0f;
        if (a.norm) a.norm[row] = make_float2(0.0f, 0.0f);
        if (a.tail) a.tail[row] = 0.0f;
      }
      row += clusters;
      *w = weight(row);
    }
    return row;
  };
  int64_t row = blockIdx.x / SIZE;
  float w = weight(row);
  row = next_live(row, &w);
  for (int i = tid; i < (GRAD ? 1 : 2) * batches * kRowThreads; i += kListThreads) marks[i] = 0u;
  if (tid < 2) edge_listed[tid] = 0u;
  __syncthreads();
  cl.started();

  if (tid < kRowThreads) {  // ---------------------------------------------------- the row's warps
    // Rows differ by their 16-byte phase alone, so by one vector: the buffer has room for the longer ones.
    const int quarter = (batches + 3) / 4;
    auto copy_batch = [&](const Part& part, int q) {
      const char* src = part.at() + q * kBatch * part.step_bytes();
      uint4* h = held + q * kBatch * kRowThreads + tid;
      if ((q + 1) * kBatch <= part.whole) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) copy_async16(h + u * kRowThreads, src + u * part.step_bytes());
      } else {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (part.more(q * kBatch + u)) copy_async16(h + u * kRowThreads, src + u * part.step_bytes());
      }
    };
    Part part(row_x(row < a.rows ? row : 0), a.vocab, cl.rank, SIZE);
    float edge = -kInf;
    if (row < a.rows) {
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        for (int q = g * quarter; q < min((g + 1) * quarter, batches); ++q) copy_batch(part, q);
        copies_commit();
      }
      if (part.edge >= 0) edge = to_float<DT>(part.x[part.edge]);
    }
    bool waits = false;  // a cluster barrier that this thread has announced itself at and not yet waited for
    for (int turn = 0; row < a.rows; turn ^= 1) {
      int64_t next = row + clusters;
      float next_edge = -kInf;
      Part next_part = part;
      auto look_ahead = [&] {
        float next_w = weight(next);
        next = next_live(next, &next_w);
        if (next < a.rows) {
          next_part = Part(row_x(next), a.vocab, cl.rank, SIZE);
          if (next_part.edge >= 0) next_edge = to_float<DT>(next_part.x[next_part.edge]);
        }
      };
      if (!GRAD) look_ahead();
      const uint32_t* listed = marks + (GRAD ? 0 : turn * batches * kRowThreads) + tid;
      if (turn == 0) barrier_sync<kReady, kListThreads>();
      else barrier_sync<kReady + 1, kListThreads>();
      const bool edge_out = part.edge >= 0 && !((edge_listed[GRAD ? 0 : turn] >> tid) & 1u);
      RunningMass out(one_element<RowMass>(edge_out ? edge : -kInf), c);
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        // copies still under way: this row's later quarters, and (loss alone) the next row's earlier ones
        if (!GRAD || g == 0) copies_wait<3>();
        else if (g == 1) copies_wait<2>();
        else if (g == 2) copies_wait<1>();
        else copies_wait<0>();
#pragma unroll 1
        for (int q = g * quarter; q < min((g + 1) * quarter, batches); ++q) {
          const uint4* h = held + q * kBatch * kRowThreads + tid;
          uint4 v[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) v[u] = h[u * kRowThreads];
          const uint32_t bits = listed[q * kRowThreads];
          if (bits != 0u) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
              if ((bits >> (8 * u)) & 0xFFu) mask_elements<DT>(v[u], bits >> (8 * u));
          }
          if ((q + 1) * kBatch > part.whole) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
              if (!part.more(q * kBatch + u))
                v[u] = make_uint4(kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>);
          }
          add_mass<DT>(v, c, out);
          if (!GRAD && next < a.rows) {
            // the sums that the held vectors went into are formed before their place is given away
            asm volatile("" ::"f"(out.at.s) : "memory");
            copy_batch(next_part, q);
          }
        }
        if (!GRAD) copies_commit();
      }
      const RowMass warp_out = merge_lanes(out.done(c), c);
      if ((tid & 31) == 0) red[turn][tid >> 5] = warp_out;
      if (turn == 0) barrier_arrive<kAdded, kListThreads>();
      else barrier_arrive<kAdded + 1, kListThreads>();
      if (SIZE > 1) {
        if (waits) cl.wait();
        cl.arrive();
        waits = true;
      }
      if constexpr (GRAD) {
        look_ahead();
        Elem<DT>* d = row_d(row);
        barrier_sync<kScales, kListThreads>();
        const float f_c = factor[0], f_r = factor[1], f_a = factor[2];
        if (part.edge >= 0) d[part.edge] = from_float<DT>(ex2(fmaf(edge, f_c, -f_r)) * f_a);
        const Pair pc = Pair::both(f_c), pr = Pair::both(-f_r), pa = Pair::both(f_a);
        char* dst = part.at(d);
        auto put = [&](const uint4& v, char* o) {
          Pair p[kPairsOf<DT>];
          unpack_pairs<DT>(v, p);
#pragma unroll
          for (int e = 0; e < kPairsOf<DT>; ++e) p[e] = mul2(ex2_pair(fma2(p[e], pc, pr)), pa);
          store_vector<DT>(o, p, a.vec);
        };
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
#pragma unroll 1
          for (int q = g * quarter; q < min((g + 1) * quarter, batches); ++q) {
            const uint4* h = held + q * kBatch * kRowThreads + tid;
            if ((q + 1) * kBatch <= part.whole) {
#pragma unroll
              for (int u = 0; u < kBatch; ++u) put(h[u * kRowThreads], dst + u * part.step_bytes());
            } else {
#pragma unroll 1
              for (int u = 0; u < kBatch && part.more(q * kBatch + u); ++u)
                put(h[u * kRowThreads], dst + u * part.step_bytes());
            }
            dst += kBatch * part.step_bytes();
            if (next < a.rows) copy_batch(next_part, q);
          }
          copies_commit();
        }
        barrier_arrive<kWritten, kListThreads>();
      }
      row = next;
      edge = next_edge;
      part = next_part;
    }
    if (SIZE > 1 && waits) cl.wait();
  } else {  // -------------------------------------------------------------------- the list's warp
    const int lane = tid & 31;
    RowList<DT> l;
    int marked[2][kSlots];  // the words of `marks` that were set (-1: none), by turn
#pragma unroll
    for (int i = 0; i < kSlots; ++i) marked[0][i] = marked[1][i] = -1;
    unsigned mine = 0u;  // slots whose element is this block's
    auto fetch = [&](int64_t r) {
      l.load(a, r, row_x(r), list_ids);
      l.sums(a);
      l.mass_in(a);
    };
    // Row r's marks for `turn`, and word that they are ready.
    auto mark = [&](int64_t r, int turn) {
      const Part part(row_x(r), a.vocab, cl.rank, SIZE);
      const int set = GRAD ? 0 : turn;
      uint32_t* listed = marks + set * batches * kRowThreads;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const int old = set ? marked[1][i] : marked[0][i];
        if (old >= 0) listed[old] = 0u;
      }
      if (lane == 0) edge_listed[set] = 0u;
      __syncwarp();
      mine = 0u;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        int owner, slot, word = -1;
        if (l.id[i] >= 0 && part.owns(l.id[i], &owner, &slot)) {
          mine |= 1u << i;
          if (slot < 0) {
            atomicOr(&edge_listed[set], 1u << owner);
          } else {
            word = (slot / kBatch) * kRowThreads + owner;
            atomicOr(&listed[word], 1u << (slot % kBatch * 8 + (l.id[i] - part.sl.head) % kVecOf<DT>));
          }
        }
        if (set) marked[1][i] = word;
        else marked[0][i] = word;
      }
      if (turn == 0) barrier_arrive<kReady, kListThreads>();
      else barrier_arrive<kReady + 1, kListThreads>();
    };
    if (row < a.rows) {
      fetch(row);
      mark(row, 0);
    }
    for (int turn = 0; row < a.rows; turn ^= 1) {
      int64_t next = row + clusters;
      float next_w = weight(next);
      const RowList<DT> now = l;  // this row's; `l` is the next one's from its fetch on
      const unsigned now_mine = mine;  // as `mark` left it
      next = next_live(next, &next_w);
      if (next < a.rows) {
        fetch(next);
        if (!GRAD) mark(next, turn ^ 1);
      }
      if (turn == 0) barrier_sync<kAdded, kListThreads>();
      else barrier_sync<kAdded + 1, kListThreads>();
      RowMass out = merge_lanes(red[turn][lane % kRowWarps], c, kRowWarps);
      if (SIZE > 1) {
        if (lane < SIZE) cl.at(parts[turn], lane)[cl.rank] = out;
        cl.arrive();
        cl.wait();
        out = merge_lanes(parts[turn][lane % SIZE], c, SIZE);
      }
      RowMass all = now.in, o = out;
      if (o.m > all.m) all.move(o.m, c);
      else if (all.m > o.m) o.move(all.m, c);
      all.s += o.s;
      const bool empty = all.s == 0.0f;
      // all unlisted tokens masked, by -inf or by values so low that no p_t is left
      const bool no_tail = out.s == 0.0f || (out.m - all.m) * c <= kFloor;
      const float ws = now.bad ? nan_f() : w * a.scale;
      const float b = now.q_sum + now.q_tail;
      if constexpr (GRAD) {
        // unlisted: (p / p_t) (p_t b - q_t) = 2^((x - m_out) c) / s_out (p_t b - q_t)
        const float p_t = no_tail ? 0.0f : ex2((out.m - all.m) * c) * (out.s / all.s);
        const float A = no_tail ? ws * 0.0f * all.s : ws * (p_t * b - now.q_tail) / out.s;
        const ExpRef ref(out.m, c);
        if (lane == 0) {
          factor[0] = ref.c;
          factor[1] = ref.r;
          factor[2] = A * ref.k;
        }
        barrier_arrive<kScales, kListThreads>();
        if (next < a.rows) mark(next, turn ^ 1);
      }
      if (cl.rank == 0) {
        const float ln_s = logf(all.s);
        const float tail = no_tail ? -kInf : fmaf(out.m - all.m, a.scale, logf(out.s) - ln_s);
        float loss = 0.0f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          if (now.id[i] >= 0 && now.q[i] != 0.0f) {
            const float lp = empty ? -kInf : fmaf(now.x[i] - all.m, a.scale, -ln_s);
            loss += now.q[i] * (now.lq[i] - lp);
          }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) loss += __shfl_xor_sync(0xFFFFFFFFu, loss, off);
        if (lane == 0) {
          if (now.q_tail > 0.0f && !no_tail) loss += now.q_tail * (logf(now.q_tail) - tail);
          if (now.bad || !(all.s == all.s) || !(now.q_sum == now.q_sum)) loss = nan_f();
          if (a.loss) a.loss[row] = w * loss;
          if (a.norm) a.norm[row] = make_float2(all.m, all.s);
          if (a.tail) a.tail[row] = tail;
        }
      }
      if constexpr (GRAD) {
        const ExpRef top(all.m, c);
        const float over = top.k / all.s;
        Elem<DT>* d = row_d(row);
        barrier_sync<kWritten, kListThreads>();
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
          if ((now_mine >> i) & 1u)
            d[now.id[i]] = from_float<DT>(empty ? 0.0f : ws * fmaf(top.exp(now.x[i]) * over, b, -now.q[i]));
      }
      row = next;
      w = next_w;
    }
  }
  // Late: the next kernel's blocks would else take the places that this wave leaves one by one, and its clusters,
  // of which all have to be resident for an even share of the rows, would not all find room.
  pdl_trigger();
}

// ------------------------------------------------------------------ the gradient from saved normalisers
//
// One pass: blocks share a row as above, but nothing is exchanged between them.
// A ninth warp has the list while the first vectors are on their way.
template <int DT>
__global__ void __launch_bounds__(kListThreads, 3) distill_grad_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ int4 list_ids[SS_MAX_TOP / 4];
  __shared__ float factor[3];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const unsigned rank = blockIdx.x % a.split;
  const int64_t row = blockIdx.x / a.split;
  const Elem<DT>* x = static_cast<const Elem<DT>*>(a.x) + row * a.ld;
  Elem<DT>* d = static_cast<Elem<DT>*>(a.d) + row * a.d_ld;
  const float wt = a.weight ? a.weight[row] : 1.0f, dl = a.d_loss ? a.d_loss[row] : 1.0f;
  const float2 norm = a.norm_in[row];
  if (wt == 0.0f || dl == 0.0f || norm.y == 0.0f) {
    if (tid < kRowThreads) zero_part<DT>(d, a.vocab, rank, a.split);
    return;
  }
  const RowPart<DT> part(x, a.vocab, rank, a.split);
  if (tid < kRowThreads) {
    uint4 first[kBatch];
    part.load(0, first);
    const float edge = part.edge >= 0 ? to_float<DT>(x[part.edge]) : 0.0f;
    barrier_sync<kScales, kListThreads>();
    const Pair c = Pair::both(factor[0]), r = Pair::both(-factor[1]), A = Pair::both(factor[2]);
    part.map(first, d, a.vec, edge, [&](Pair f) { return mul2(ex2_pair(fma2(f, c, r)), A); });
    barrier_arrive<kWritten, kListThreads>();
    return;
  }
  RowList<DT> l;
  l.load(a, row, x, list_ids);
  l.sums(a);
  const float ws = l.bad ? nan_f() : wt * dl * a.scale;
  const float b = l.q_sum + l.q_tail;
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
      A = ws * (p_t * b - l.q_tail) * (over / p_t);
    } else {
      A = ws * (p_t * b - l.q_tail) * over;
      r = fmaf(tail, kLog2e, r);
    }
  }
  if ((tid & 31) == 0) {
    factor[0] = ref.c;
    factor[1] = r;
    factor[2] = A;
  }
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
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, kListThreads, smem);
    n *= sm_count();
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(kListThreads);
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
                         t->tail, t->dtype, t->idtype == SS_I64, d_logits && same_phase(x, d_logits, d_ld), d_logits == x->data,
                         static_cast<uint32_t>(split), 0};
  if (saved) {
    auto* fn = x->dtype == SS_BF16
                   ? distill_grad_kernel<SS_BF16>
                   : (x->dtype == SS_FP16 ? distill_grad_kernel<SS_FP16> : distill_grad_kernel<SS_FP32>);
    if (rows * split > INT32_MAX) return SS_ERR_OVERFLOW;
    return launch(fn, static_cast<unsigned>(rows * split), a, stream, kListThreads);
  }
  // a part of at most kPartVectors vectors a thread, or what 8 blocks leave
  const auto vectors = [&](int n) { return (nvec + n * kRowThreads - 1) / (n * kRowThreads); };
  int cluster = 1;
  while (cluster < kMaxCluster && vectors(cluster) > kPartVectors) cluster *= 2;
  auto* fn = d_logits ? distill_for<true>(x->dtype, cluster) : distill_for<false>(x->dtype, cluster);
  a.batches = static_cast<int>((vectors(cluster) + kBatch - 1) / kBatch);
  const size_t smem = static_cast<size_t>(a.batches) * kRowThreads * (kBatch * sizeof(uint4) + (d_logits ? 1 : 2) * sizeof(uint32_t));
  int clusters = 0;
  st = resident_clusters(reinterpret_cast<const void*>(fn), smem, cluster, &clusters);
  if (st != SS_OK) return st;
  return launch_rows(fn, std::min<int64_t>(rows, clusters), cluster, kListThreads, smem, a, stream);
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
