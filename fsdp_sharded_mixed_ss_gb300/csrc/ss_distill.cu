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
};

__device__ __forceinline__ float load_teacher(const void* p, int64_t i, int dtype) {
  if (dtype == SS_FP32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == SS_BF16 ? widen1<SS_BF16>(h) : widen1<SS_FP16>(h);
}

// A row's list in shared memory, filled by list_load: slot j < k is used when
// id[j] >= 0, with log q and q of its token.
struct List {
  int32_t id[SS_MAX_TOP];
  float lq[SS_MAX_TOP];
  float q[SS_MAX_TOP];
  float x[SS_MAX_TOP];  // the tokens' logits
  float q_sum, q_tail;  // Q and q_t
  bool bad;             // an id past the vocabulary
};

// All threads of the block call it. Q is added in double: q_t = 1 - Q keeps the
// digits that a teacher with nearly all its mass on the list leaves.
template <int DT>
__device__ __forceinline__ void list_load(const DistillArgs& a, int64_t row, const Elem<DT>* x, List& l) {
  const int j = threadIdx.x;
  if (j == 0) l.bad = false;
  __syncthreads();
  if (j < a.k) {
    const int64_t id = load_id(a.ids, row * a.k + j, a.wide);
    if (id >= a.vocab) l.bad = true;
    const bool used = id >= 0 && id < a.vocab;
    l.id[j] = used ? static_cast<int32_t>(id) : -1;
    l.lq[j] = used ? load_teacher(a.teacher, row * a.k + j, a.t_dtype) * a.t_scale : -kInf;
    l.x[j] = used ? to_float<DT>(x[id]) : 0.0f;
  }
  __syncthreads();
  bool again = false;
  if (j < a.k && l.id[j] >= 0)
    for (int i = 0; i < j; ++i) again = again || l.id[i] == l.id[j];
  __syncthreads();
  if (again) {
    l.id[j] = -1;
    l.lq[j] = -kInf;
  }
  __syncthreads();
  if (j < 32) {
    float shift = 0.0f;
    if (a.mode == SS_TAIL_RENORM) {
      float m = -kInf, s = 0.0f;
      bool nan = false;
      for (int i = j; i < a.k; i += 32) {
        m = fmaxf(m, l.lq[i]);
        nan = nan || !(l.lq[i] == l.lq[i]);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
      const float ref = m == -kInf ? 0.0f : m;
      for (int i = j; i < a.k; i += 32) s += expf(l.lq[i] - ref);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
      nan = __any_sync(0xFFFFFFFFu, nan);
      shift = nan ? nan_f() : (s == 0.0f ? 0.0f : m + logf(s));
    }
    double sum = 0.0;
    for (int i = j; i < a.k; i += 32) {
      const float lq = l.lq[i] - shift;
      const float q = expf(lq);
      l.lq[i] = lq;
      l.q[i] = q;
      sum += static_cast<double>(q);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    if (j == 0) {
      l.q_sum = static_cast<float>(sum);
      const double rest = 1.0 - sum;
      l.q_tail = a.mode == SS_TAIL_BUCKET && !(rest <= 0.0) ? static_cast<float>(rest) : 0.0f;
    }
  }
  __syncthreads();
}

// Writes f(x) over the row, then each used slot's own gradient g[j] (all threads
// call it; the slots' logits were read before).
template <int DT, class F>
__device__ __forceinline__ void write_row(const Elem<DT>* x, Elem<DT>* d, int64_t n, bool vec, const F& f,
                                          int32_t my_id, float mine) {
  constexpr int V = kVecOf<DT>;
  if (vec) {
    const Slice<DT> sl(x, n);
    for (int64_t i = threadIdx.x; i < sl.head; i += kRowThreads) d[i] = from_float<DT>(f(to_float<DT>(x[i])));
    for (int64_t i = sl.tail() + threadIdx.x; i < sl.n; i += kRowThreads)
      d[i] = from_float<DT>(f(to_float<DT>(x[i])));
    const uint4* v = reinterpret_cast<const uint4*>(x + sl.head);
    uint4* w = reinterpret_cast<uint4*>(d + sl.head);
    for (int64_t i = threadIdx.x; i < sl.nvec; i += kRowThreads) {
      float e[V];
      unpack<DT>(v[i], e);
#pragma unroll
      for (int j = 0; j < V; ++j) e[j] = f(e[j]);
      w[i] = pack<DT>(e);
    }
  } else {
    for (int64_t i = threadIdx.x; i < n; i += kRowThreads) d[i] = from_float<DT>(f(to_float<DT>(x[i])));
  }
  __syncthreads();
  if (my_id >= 0) d[my_id] = from_float<DT>(mine);
}

template <int DT>
__device__ __forceinline__ void zero_row(Elem<DT>* d, int64_t n) {
  const Slice<DT> sl(d, n);
  for (int64_t i = threadIdx.x; i < sl.head; i += kRowThreads) d[i] = from_float<DT>(0.0f);
  for (int64_t i = sl.tail() + threadIdx.x; i < sl.n; i += kRowThreads) d[i] = from_float<DT>(0.0f);
  uint4* w = reinterpret_cast<uint4*>(d + sl.head);
  for (int64_t i = threadIdx.x; i < sl.nvec; i += kRowThreads) w[i] = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------ loss and gradient in one call
//
// The gradient needs the row's sums and then the row again. A row is shared by
// the blocks of a cluster, each holding its part in shared memory: the logits
// are read from HBM once, with asynchronous copies that are all issued at the
// start, and the gradient is computed from shared memory and written once. Two
// to four blocks fit an SM, so one's sums and barriers pass under another's
// copies and stores.
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

template <int DT>
__device__ __forceinline__ void add_mass(const uint4 (&w)[kBatch], float c, RowMass& acc) {
  constexpr int V = kVecOf<DT>;
  float m = vec_max<DT>(w[0]);
#pragma unroll
  for (int u = 1; u < kBatch; ++u) m = fmaxf(m, vec_max<DT>(w[u]));
  if (m > acc.m) acc.move(m, c);
  const float ref = acc.ref();
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    float f[V];
    unpack<DT>(w[u], f);
#pragma unroll
    for (int j = 0; j < V; ++j) s[j & 1] += ex2((f[j] - ref) * c);
  }
  acc.s += s[0] + s[1];
}

// Zeros in this block's part of a gradient row.
template <int DT>
__device__ __forceinline__ void zero_part(Elem<DT>* d, int64_t n, unsigned rank, unsigned size) {
  const Slice<DT> sl(d, n);
  if (rank == 0) {
    for (int64_t i = threadIdx.x; i < sl.head; i += kRowThreads) d[i] = from_float<DT>(0.0f);
    for (int64_t i = sl.tail() + threadIdx.x; i < sl.n; i += kRowThreads) d[i] = from_float<DT>(0.0f);
  }
  uint4* w = reinterpret_cast<uint4*>(d + sl.head);
  for (int64_t i = rank * kRowThreads + threadIdx.x; i < sl.nvec; i += size * kRowThreads)
    __stcs(w + i, make_uint4(0u, 0u, 0u, 0u));
}

// Dynamic shared memory: the part's vectors [batches * kBatch][T], then a byte of listed bits for each, by thread.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) distill_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int V = kVecOf<DT>;
  extern __shared__ uint4 held[];
  __shared__ RowMass red[kRowThreads / 32];
  __shared__ RowMass parts[kMaxCluster];
  __shared__ List l;
  __shared__ float part_loss[kRowThreads / 32];
  __shared__ uint32_t edge_listed;
  const Cluster cl = Cluster::start();
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / cl.size;
  const Elem<DT>* x = static_cast<const Elem<DT>*>(a.x) + row * a.ld;
  Elem<DT>* d = static_cast<Elem<DT>*>(a.d) + row * a.d_ld;
  const float w = a.weight ? a.weight[row] : 1.0f;
  if (w == 0.0f) {  // every block of the cluster
    if (a.d) zero_part<DT>(d, a.vocab, cl.rank, cl.size);
    if (cl.rank == 0 && tid == 0) {
      if (a.loss) a.loss[row] = 0.0f;
      if (a.norm) a.norm[row] = make_float2(0.0f, 0.0f);
      if (a.tail) a.tail[row] = 0.0f;
    }
    cl.started();
    return;
  }
  const RowPart<DT> part(x, a.vocab, cl.rank, cl.size);
  const int nvec = static_cast<int>(part.sl.nvec);
  const int batches = (part.vectors() + kBatch - 1) / kBatch;
  uint32_t* listed = reinterpret_cast<uint32_t*>(held + static_cast<size_t>(batches) * kBatch * kRowThreads);
  // four groups of copies, so that the first quarter is added up while the rest is on its way
  const int quarter = (batches + 3) / 4;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    for (int j = g * quarter * kBatch; j < min((g + 1) * quarter, batches) * kBatch; ++j) {
      const int i = part.first + j * part.step;
      if (i < nvec) copy_async16(held + j * kRowThreads + tid, part.vec(i));
    }
    copies_commit();
  }
  for (int q = 0; q < batches; ++q) listed[q * kRowThreads + tid] = 0u;
  if (tid == 0) edge_listed = 0u;
  const float edge = part.edge >= 0 ? to_float<DT>(x[part.edge]) : -kInf;
  list_load<DT>(a, row, x, l);
  const int32_t my_id = tid < a.k ? l.id[tid] : -1;
  int owner = 0, slot = 0;
  const bool mine = my_id >= 0 && part.owns(my_id, &owner, &slot);
  if (mine) {
    if (slot < 0) atomicOr(&edge_listed, 1u << owner);
    else atomicOr(&listed[(slot / kBatch) * kRowThreads + owner],
                  1u << (slot % kBatch * 8 + (my_id - part.sl.head) % V));
  }
  __syncthreads();
  RowMass out = RowMass::none();  // unlisted tokens
  if (part.edge >= 0 && !((edge_listed >> tid) & 1u)) {
    out.m = edge;
    out.s = ex2((edge - out.ref()) * a.c);
  }
  auto add_group = [&](int g) {
    for (int q = g * quarter; q < min((g + 1) * quarter, batches); ++q) {
      uint4 v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        v[u] = held[(q * kBatch + u) * kRowThreads + tid];
        if (part.first + (q * kBatch + u) * part.step >= nvec)
          v[u] = make_uint4(kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>);
      }
      const uint32_t bits = listed[q * kRowThreads + tid];
      if (bits != 0u) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) mask_elements<DT>(v[u], (bits >> (8 * u)) & 0xFFu);
      }
      add_mass<DT>(v, a.c, out);
    }
  };
  copies_wait<3>();
  add_group(0);
  copies_wait<2>();
  add_group(1);
  copies_wait<1>();
  add_group(2);
  copies_wait<0>();
  add_group(3);
  out = block_merge<kRowThreads>(out, a.c, red);
  RowMass in = RowMass::none();
  if (my_id >= 0) in = {l.x[tid], ex2((l.x[tid] - (l.x[tid] == -kInf ? 0.0f : l.x[tid])) * a.c)};
  cl.started();
  if (cl.size > 1 && tid < cl.size) cl.at(parts, tid)[cl.rank] = out;
  in = block_merge<kRowThreads>(in, a.c, red);
  if (cl.size > 1) {
    cl.sync();
    out = parts[0];
    for (unsigned r = 1; r < cl.size; ++r) out.merge(parts[r], a.c);
  }
  RowMass all = out;
  all.merge(in, a.c);
  const bool empty = all.s == 0.0f;
  // all unlisted tokens masked, by -inf or by values so low that no p_t is left
  const bool no_tail = out.s == 0.0f || (out.m - all.m) * a.c <= kFloor;
  if (cl.rank == 0) {
    const float ln_s = logf(all.s);
    const float tail = no_tail ? -kInf : fmaf(out.m - all.m, a.scale, logf(out.s) - ln_s);
    float term = 0.0f;
    if (my_id >= 0 && l.q[tid] != 0.0f) {
      const float lp = empty ? -kInf : fmaf(l.x[tid] - all.m, a.scale, -ln_s);
      term = l.q[tid] * (l.lq[tid] - lp);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, off);
    if ((tid & 31) == 0) part_loss[tid >> 5] = term;
    __syncthreads();
    if (tid == 0) {
      float loss = 0.0f;
      for (int i = 0; i < kRowThreads / 32; ++i) loss += part_loss[i];
      if (l.q_tail > 0.0f && !no_tail) loss += l.q_tail * (logf(l.q_tail) - tail);
      if (l.bad || !(all.s == all.s) || !(l.q_sum == l.q_sum)) loss = nan_f();
      if (a.loss) a.loss[row] = w * loss;
      if (a.norm) a.norm[row] = make_float2(all.m, all.s);
      if (a.tail) a.tail[row] = tail;
    }
  }
  if (!a.d) return;
  if (empty) {
    zero_part<DT>(d, a.vocab, cl.rank, cl.size);
    return;
  }
  const float ws = l.bad ? nan_f() : w * a.scale;
  const float b = l.q_sum + l.q_tail;
  // unlisted: (p / p_t) (p_t b - q_t) = 2^((x - m_out) c) / s_out (p_t b - q_t)
  const float p_t = no_tail ? 0.0f : ex2((out.m - all.m) * a.c) * (out.s / all.s);
  const float A = no_tail ? ws * 0.0f * all.s : ws * (p_t * b - l.q_tail) / out.s;
  const float ref = out.ref();
  const float c = a.c;
  auto grad = [&](float f) { return ex2((f - ref) * c) * A; };
  if (part.edge >= 0) d[part.edge] = from_float<DT>(grad(edge));
  for (int q = 0; q < batches; ++q) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = q * kBatch + u, i = part.first + j * part.step;
      if (i < nvec) {
        float f[V];
        unpack<DT>(held[j * kRowThreads + tid], f);
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = grad(f[e]);
        Elem<DT>* o = d + part.sl.head + static_cast<int64_t>(i) * V;
        if (a.vec) {
          __stcs(reinterpret_cast<uint4*>(o), pack<DT>(f));
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = from_float<DT>(f[e]);
        }
      }
    }
  }
  __syncthreads();
  if (mine) d[my_id] = from_float<DT>(ws * fmaf(ex2((l.x[tid] - all.ref()) * a.c) / all.s, b, -l.q[tid]));
}

// The gradient from saved normalisers: one pass.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) distill_grad_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ List l;
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const Elem<DT>* x = static_cast<const Elem<DT>*>(a.x) + row * a.ld;
  Elem<DT>* d = static_cast<Elem<DT>*>(a.d) + row * a.d_ld;
  const float wt = a.weight ? a.weight[row] : 1.0f, dl = a.d_loss ? a.d_loss[row] : 1.0f;
  const float2 norm = a.norm_in[row];
  if (wt == 0.0f || dl == 0.0f || norm.y == 0.0f) {
    zero_row<DT>(d, a.vocab);
    return;
  }
  list_load<DT>(a, row, x, l);
  const int j = threadIdx.x;
  const int32_t my_id = j < a.k ? l.id[j] : -1;
  const float ws = l.bad ? nan_f() : wt * dl * a.scale;
  const float b = l.q_sum + l.q_tail;
  const float l2 = log2f(norm.y);
  float A = ws * b, K = l2;
  if (a.mode == SS_TAIL_BUCKET) {
    const float tail = a.tail_in[row];
    if (tail == -kInf) {
      A = ws * 0.0f;
    } else {
      A = ws * (expf(tail) * b - l.q_tail);
      K = fmaf(tail, kLog2e, l2);
    }
  }
  const float g = my_id >= 0 ? ws * fmaf(ex2(fmaf(l.x[j] - norm.x, a.c, -l2)), b, -l.q[j]) : 0.0f;
  write_row<DT>(x, d, a.vocab, a.vec, [&](float f) { return ex2(fmaf(f - norm.x, a.c, -K)) * A; }, my_id, g);
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
  const DistillArgs a = {x->data, t->ids, t->logprob, t->row_weight, d_loss,
                         reinterpret_cast<const float2*>(norm_in), tail_in, loss, reinterpret_cast<float2*>(norm),
                         tail, d_logits, rows, x->vocab, x->ld, d_ld, x->scale * kLog2e, x->scale, t->scale, t->k,
                         t->tail, t->dtype, t->idtype == SS_I64, d_logits && same_phase(x, d_logits, d_ld)};
  if (saved) {
    auto* fn = x->dtype == SS_BF16
                   ? distill_grad_kernel<SS_BF16>
                   : (x->dtype == SS_FP16 ? distill_grad_kernel<SS_FP16> : distill_grad_kernel<SS_FP32>);
    return launch(fn, static_cast<unsigned>(rows), a, stream, kRowThreads);
  }
  auto* fn = x->dtype == SS_BF16 ? distill_kernel<SS_BF16>
                                 : (x->dtype == SS_FP16 ? distill_kernel<SS_FP16> : distill_kernel<SS_FP32>);
  // a part of at most kPartVectors vectors a thread, or what 8 blocks leave
  const int64_t vec = x->dtype == SS_FP32 ? 4 : 8, nvec = x->vocab / vec;
  const auto vectors = [&](int c) { return (nvec + c * kRowThreads - 1) / (c * kRowThreads); };
  int cluster = 1;
  while (cluster < kMaxCluster && vectors(cluster) > kPartVectors) cluster *= 2;
  const int64_t batches = (vectors(cluster) + kBatch - 1) / kBatch;
  const size_t smem = static_cast<size_t>(batches) * kRowThreads * (kBatch * sizeof(uint4) + sizeof(uint32_t));
  if (rows * cluster > INT32_MAX) return SS_ERR_OVERFLOW;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return cuda_fail(e);
  return launch_rows(fn, rows, cluster, smem, a, stream);
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
