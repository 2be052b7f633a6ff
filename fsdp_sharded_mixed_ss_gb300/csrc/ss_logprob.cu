// ss_logprob.cu -- log probabilities of given tokens with entropy and top
// alternatives (ss_token_logprobs), and their gradient (ss_token_logprobs_grad).
#include "ss_logits.cuh"

namespace ss {
namespace {

struct LogprobArgs {
  const void* x;
  const void* tokens;
  float* logprob;
  float* entropy;
  float* lse;
  float2* norm;
  float* top_logprob;
  void* top_id;
  int64_t rows, vocab, ld;
  float c, scale;
  int32_t top_k;
  bool wide;  // int64 ids
};

// ------------------------------------------------------------------ forward
//
// A row belongs to a cluster of 1 to 8 blocks (RowPart says which elements are
// whose). One pass gives the row's maximum, sum and entropy's sum. The alternatives come
// from the same pass: the maximum of every unit (4 vectors of a thread, more in
// rows longer than 16 units a thread) stays in shared memory, and every thread's
// maximum is a key. Some threshold that k of the 256 keys reach is a bound that
// at least k elements of the row reach, and few more: for k of 256 keys drawn at
// random -256 ln(1 - k / 256) elements, 21 for k = 20 and 177 for k = 128. Only
// units whose maximum reaches it are read again (from L2), their elements at or
// above it are the candidates, and each candidate's rank is the number of
// candidates above it. Where the candidates pass the buffer (ties), the exact
// k-th pair is searched for by counting.

constexpr int kUnits = 16;    // maxima kept per thread
constexpr int kCand = 2048;   // candidates of a row, shared out over the cluster's blocks
constexpr int kFlagged = 1024;  // units of a block that are read again
constexpr uint32_t kMaskedKey = 0x007FFFFFu;  // order_key(-inf)

struct TopShared {
  float unit[kUnits][kRowThreads];
  uint64_t cand[kCand];          // block 0's is used
  uint32_t keys[kRowThreads];
  int count[kMaxCluster];        // candidates of every block
  int sums[2][kMaxCluster];      // counts being added up over the cluster
  int warp_sums[kRowThreads / 32];
  uint16_t flagged[kFlagged];
  int n, n_flagged;
};
struct NoTops {};

using RunningSum = Running<RowSum, 8>;

// N vectors into the running sums; returns their maximum.
template <int DT, int N>
__device__ __forceinline__ float add_vectors(const uint4 (&w)[N], float c, RunningSum& acc) {
  constexpr int V = kVecOf<DT>;
  float m = vec_max<DT>(w[0]);
#pragma unroll
  for (int u = 1; u < N; ++u) m = fmaxf(m, vec_max<DT>(w[u]));
  acc.see(m, c);
  const ExpRef& ref = acc.ref;
  Pair s = Pair::both(0.0f), t = s;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    Pair f[kPairsOf<DT>];
    unpack_pairs<DT>(w[u], f);
#pragma unroll
    for (int j = 0; j < kPairsOf<DT>; ++j) {
      const Pair d = ref.arg(f[j]), e = ex2_pair(d);
      s = add2(s, e);
      t = fma2(e, d, t);
    }
  }
  const float ss = s.sum();
  float tt = t.sum();
  if (!(tt == tt)) {  // masked elements (0 * -inf): the same sum with them at kFloor
    tt = 0.0f;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float f[V];
      unpack<DT>(w[u], f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = fmaxf(ref.arg(f[j]), kFloor);
        tt = fmaf(ex2(d), d, tt);
      }
    }
  }
  acc.at.s = fmaf(ss, ref.k, acc.at.s);
  acc.at.t = fmaf(fmaf(ref.shift, ss, tt), ref.k, acc.at.t);
  return m;
}

// Sum of v over all threads of the cluster, the same in each (all call it; `it` counts the calls).
__device__ __forceinline__ int cluster_count(const Cluster& cl, TopShared& ts, int v, int it) {
  v = __reduce_add_sync(0xFFFFFFFFu, v);
  if ((threadIdx.x & 31) == 0) ts.warp_sums[threadIdx.x >> 5] = v;
  __syncthreads();
  int* slots = ts.sums[it & 1];
  if (threadIdx.x < cl.size) {
    int b = 0;
    for (int w = 0; w < kRowThreads / 32; ++w) b += ts.warp_sums[w];
    cl.at(slots, threadIdx.x)[cl.rank] = b;
  }
  cl.sync();
  int all = 0;
  for (unsigned r = 0; r < cl.size; ++r) all += slots[r];
  return all;
}

// The exact k-th largest pair as (key, id): elements above `key`, and those equal to it with ids up to `id`, are
// the k. At least k elements reach the key `lo`; none is above `top`.
template <int DT>
__device__ __noinline__ uint2 search_pair(const Cluster& cl, TopShared& ts, const RowPart<DT>& part, int vectors,
                                          uint32_t lo, uint32_t top, int k) {
  const int vocab = static_cast<int>(part.sl.n);
  int it = 0;
  auto count = [&](auto pred) {
    int c = 0;
    part.each(0, vectors, [&](float f, int id) { c += pred(order_key(f), id) ? 1 : 0; });
    if (part.edge >= 0) c += pred(order_key(to_float<DT>(part.x[part.edge])), part.edge) ? 1 : 0;
    return cluster_count(cl, ts, c, it++);
  };
  uint32_t hi = top;  // count(key > hi) = above < k, count(key >= lo) >= k
  int above = 0;
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const int c = count([&](uint32_t key, int) { return key >= mid; });
    if (c >= k) {
      lo = mid;
    } else {
      hi = mid - 1;
      above = c;
    }
  }
  const int need = k - above;
  int a = 0, b = vocab - 1;  // the smallest id bound that gives `need` elements equal to the key
  while (a < b) {
    const int mid = a + (b - a) / 2;
    const int c = count([&](uint32_t key, int id) { return key == lo && id <= mid; });
    if (c >= need) b = mid;
    else a = mid + 1;
  }
  return make_uint2(lo, static_cast<uint32_t>(a));
}

template <int DT, bool TOPS>
__global__ void __launch_bounds__(kRowThreads, 4) logprob_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ RowSum red[kRowThreads / 32];
  __shared__ RowSum parts[kMaxCluster];
  __shared__ std::conditional_t<TOPS, TopShared, NoTops> tops;
  const Cluster cl = Cluster::start();
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / cl.size;
  const RowPart<DT> part(static_cast<const Elem<DT>*>(a.x) + row * a.ld, a.vocab, cl.rank, cl.size);
  const int vectors = part.vectors();
  const int full = part.whole / kBatch;  // batches that every thread has whole
  const int64_t sb = part.step_bytes();
  const char* src = part.at();
  const int unit_batches = ((vectors + kBatch - 1) / kBatch + kUnits - 1) / kUnits;
  const float edge = part.edge >= 0 ? to_float<DT>(part.x[part.edge]) : -kInf;
  RunningSum run(one_element<RowSum>(edge), a.c);
  float unit = -kInf;
  int in_unit = 0, units = 0;
  auto end_batch = [&](float m) {
    if constexpr (TOPS) {
      unit = fmaxf(unit, m);
      if (++in_unit == unit_batches) {
        tops.unit[units++][tid] = unit;
        in_unit = 0;
        unit = -kInf;
      }
    }
  };
  for (int b = 0; b < full; ++b, src += kBatch * sb) {
    uint4 w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) w[u] = __ldg(reinterpret_cast<const uint4*>(src + u * sb));
    end_batch(add_vectors<DT>(w, a.c, run));
  }
  if (full * kBatch < vectors) {
    uint4 w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      w[u] = part.more(full * kBatch + u)
                 ? __ldg(reinterpret_cast<const uint4*>(src + u * sb))
                 : make_uint4(kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>);
    end_batch(add_vectors<DT>(w, a.c, run));
  }
  if constexpr (TOPS) {
    if (in_unit > 0) tops.unit[units++][tid] = unit;
  }
  const float thread_max = run.top;
  RowSum acc = block_merge(run.done(a.c), a.c, red);
  cl.started();
  if (cl.size > 1) {
    if (tid < cl.size) cl.at(parts, tid)[cl.rank] = acc;
  }
  if constexpr (TOPS) {
    // 256 keys of the whole row: the maxima of groups of `size` neighbouring threads of every block
    uint32_t key = order_key(thread_max);
    for (unsigned off = 1; off < cl.size; off <<= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, off));
    if (tid % cl.size == 0) {
      const unsigned at = cl.rank * (kRowThreads / cl.size) + tid / cl.size;
      for (unsigned r = 0; r < cl.size; ++r) cl.at(tops.keys, r)[at] = key;
    }
    if (tid == 0) tops.n = tops.n_flagged = 0;
  }
  if (TOPS || cl.size > 1) cl.sync();
  if (cl.size > 1) {
    acc = merge_lanes(parts[tid % cl.size], a.c, static_cast<int>(cl.size));
  }
  const bool nan = !(acc.s == acc.s);
  const bool empty = acc.s == 0.0f;
  const float ln_s = logf(acc.s);
  auto logp = [&](float f) {
    if (nan) return nan_f();
    return empty ? -kInf : fmaf(f - acc.m, a.scale, -ln_s);
  };
  if (cl.rank == 0 && tid == 0) {
    if (a.norm) a.norm[row] = make_float2(acc.m, acc.s);
    if (a.lse) a.lse[row] = empty ? -kInf : fmaf(acc.m, a.scale, ln_s);
    if (a.entropy) {
      const float h = empty ? 0.0f : ln_s - acc.t / acc.s * kLn2;
      a.entropy[row] = h < 0.0f ? 0.0f : h;
    }
    if (a.logprob) {
      const int64_t t = load_id(a.tokens, row, a.wide);
      a.logprob[row] = t < 0 ? 0.0f : (t >= a.vocab ? nan_f() : logp(to_float<DT>(part.x[t])));
    }
  }
  if constexpr (TOPS) {
    const int k = a.top_k;
    auto put = [&](int j, int64_t id, float lp) {
      const int64_t o = row * k + j;
      if (a.top_id) store_id(a.top_id, o, id, a.wide);
      if (a.top_logprob) a.top_logprob[o] = lp;
    };
    if (nan) {  // in every block of the cluster: all have merged the same parts
      if (cl.rank == 0 && tid < k) put(tid, -1, nan_f());
      return;
    }
    // the threshold: bit by bit, the largest that k keys reach; a little less is as good
    constexpr int kLowBit = DT == SS_BF16 ? 16 : (DT == SS_FP16 ? 13 : 0);
    const uint32_t my_key = tops.keys[tid];
    const uint32_t top_key = order_key(acc.m);
    uint32_t tau = 0;
    for (int bit = 31; bit >= kLowBit; --bit) {
      const uint32_t t = tau | (1u << bit);
      if (t > top_key) continue;
      const int c = __syncthreads_count(my_key >= t);
      if (c >= k) {
        tau = t;
        if (c <= k + k / 8) break;
      }
    }
    const bool few = tau <= kMaskedKey;  // fewer than k threads hold unmasked tokens: all of those are candidates
    if (few) tau = kMaskedKey + 1;
    const float bound = few ? -kInf : key_value(tau);
    auto wanted = [&](float f) { return few ? f > bound : f >= bound; };
    const int room = kCand / static_cast<int>(cl.size);
    uint64_t* out = cl.at(tops.cand, 0) + cl.rank * room;
    auto add = [&](float f, int id) {
      const int n = atomicAdd(&tops.n, 1);
      if (n < room) out[n] = order_pair(f, id);
    };
    for (int u = 0; u < units; ++u) {
      if (wanted(tops.unit[u][tid])) {
        const int f = atomicAdd(&tops.n_flagged, 1);
        if (f < kFlagged) tops.flagged[f] = static_cast<uint16_t>(u * kRowThreads + tid);
      }
    }
    if (part.edge >= 0 && wanted(edge)) add(edge, part.edge);
    __syncthreads();
    // a warp reads a flagged unit's elements again, one a lane, four units at a time
    constexpr int V = kVecOf<DT>;
    const int flagged = min(tops.n_flagged, kFlagged), lane = tid & 31;
    const int unit_elems = unit_batches * kBatch * V;
#pragma unroll 1
    for (int f0 = (tid >> 5) * 4; f0 < flagged; f0 += kRowWarps * 4) {
#pragma unroll 1
      for (int e = lane; e < unit_elems; e += 32) {
        float val[4];
        int id[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          id[q] = -1;
          if (f0 + q < flagged) {
            const int unit_at = tops.flagged[f0 + q];
            const int64_t vec = static_cast<int64_t>((unit_at / kRowThreads) * unit_batches * kBatch + e / V) * part.step() +
                                part.rank * kRowThreads + unit_at % kRowThreads;
            if (vec < part.sl.nvec) {
              id[q] = part.sl.head + static_cast<int>(vec) * V + e % V;
              val[q] = to_float<DT>(part.x[id[q]]);
            }
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bool hit = id[q] >= 0 && wanted(val[q]);
          const unsigned hits = __ballot_sync(__activemask(), hit);
          if (hit) {
            const int leader = __ffs(hits) - 1;
            int at = 0;
            if (lane == leader) at = atomicAdd(&tops.n, __popc(hits));
            at = __shfl_sync(hits, at, leader) + __popc(hits & ((1u << lane) - 1u));
            if (at < room) out[at] = order_pair(val[q], id[q]);
          }
        }
      }
    }
    if (tid == 0 && tops.n_flagged > kFlagged) tops.n = room + 1;
    __syncthreads();
    if (tid < cl.size) cl.at(tops.count, tid)[cl.rank] = tops.n;
    cl.sync();
    int total = 0;
    bool over = false;
    for (unsigned r = 0; r < cl.size; ++r) {
      total += tops.count[r];
      over = over || tops.count[r] > room;
    }
    if (over) {
      const uint2 kth = search_pair<DT>(cl, tops, part, vectors, tau, order_key(acc.m), k);
      if (tid == 0) tops.n = 0;
      __syncthreads();
      auto kept = [&](float f, int id) {
        const uint32_t key = order_key(f);
        if (key > kth.x || (key == kth.x && id <= static_cast<int>(kth.y))) add(f, id);
      };
      part.each(0, vectors, kept);
      if (part.edge >= 0) kept(edge, part.edge);
      __syncthreads();
      if (tid < cl.size) cl.at(tops.count, tid)[cl.rank] = tops.n;
      cl.sync();
      total = k;
    }
    if (cl.rank != 0) return;
    for (int i = tid; i < total; i += kRowThreads) {
      int r = 0, at = i;
      while (at >= tops.count[r]) at -= tops.count[r++];
      const uint64_t mine = tops.cand[r * room + at];
      int rank = 0;
      for (unsigned q = 0; q < cl.size; ++q)
        for (int j = 0; j < tops.count[q]; ++j) rank += tops.cand[q * room + j] > mine ? 1 : 0;
      if (rank < k)
        put(rank, static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(mine)),
            logp(key_value(static_cast<uint32_t>(mine >> 32))));
    }
    if (few && total < k) {  // the rest are masked tokens, by ascending id
      int have = total;
      for (int64_t base = 0; base < a.vocab && have < k; base += kRowThreads) {
        const int64_t i = base + tid;
        const bool masked = i < a.vocab && to_float<DT>(part.x[i]) == -kInf;
        const unsigned votes = __ballot_sync(0xFFFFFFFFu, masked);
        __syncthreads();  // the last round's sums have been read
        if ((tid & 31) == 0) tops.warp_sums[tid >> 5] = __popc(votes);
        __syncthreads();
        int before = have;
        for (int w = 0; w < kRowThreads / 32; ++w) {
          if (w < tid >> 5) before += tops.warp_sums[w];
          have += tops.warp_sums[w];
        }
        const int j = before + __popc(votes & ((1u << (tid & 31)) - 1u));
        if (masked && j < k) put(j, i, -kInf);
      }
    }
  }
}

// Blocks that share a row: rows alone fill the GPU from about 4 blocks on each SM; fewer rows are split while
// every thread keeps a batch of vectors.
int cluster_for(int64_t rows, int64_t vocab, int vec) {
  const int64_t blocks = 4 * std::max(1, sm_count());
  int c = 1;
  while (c < kMaxCluster && rows * c * 2 <= blocks && vocab >= static_cast<int64_t>(c) * 2 * kRowThreads * kBatch * vec / 2)
    c *= 2;
  return c;
}

struct LogprobGradArgs {
  const void* x;
  const void* tokens;
  const void* top_id;
  const float2* norm;
  const float* entropy;
  const float* d_logprob;
  const float* d_entropy;
  const float* d_lse;
  const float* d_top;
  void* d;
  int64_t rows, vocab, ld, d_ld;
  float c, scale;
  int32_t top_k;
  bool wide, vec;
  uint32_t split;  // blocks that share a row
};

// One pass, each row shared by blocks that exchange nothing. Every element is
// p (A + B log2 p); the listed ids, whose logits are read before anything is
// written (the gradient may replace the logits), get their own terms on top.
template <int DT>
__global__ void __launch_bounds__(kRowThreads, 4) logprob_grad_kernel(const __grid_constant__ LogprobGradArgs a) {
  __shared__ int32_t ids[SS_MAX_TOP + 1];
  __shared__ float up[SS_MAX_TOP + 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const unsigned rank = blockIdx.x % a.split;
  const int64_t row = blockIdx.x / a.split;
  const Elem<DT>* x = static_cast<const Elem<DT>*>(a.x) + row * a.ld;
  Elem<DT>* d = static_cast<Elem<DT>*>(a.d) + row * a.d_ld;
  const int n_ids = a.top_k + 1;
  int64_t id = -1;
  float u = 0.0f;
  if (tid < a.top_k) {
    id = load_id(a.top_id, row * a.top_k + tid, a.wide);
    u = a.d_top[row * a.top_k + tid];
  } else if (tid == a.top_k && a.d_logprob) {
    id = load_id(a.tokens, row, a.wide);
    u = a.d_logprob[row];
  }
  const float2 norm = a.norm[row];
  const float dl = a.d_lse ? a.d_lse[row] : 0.0f;
  const float dh = a.d_entropy ? a.d_entropy[row] : 0.0f;
  const float h = a.d_entropy ? a.entropy[row] : 0.0f;
  const RowPart<DT> part(x, a.vocab, rank, a.split);
  uint4 first[kBatch];
  part.load(0, first);
  const float edge = part.edge >= 0 ? to_float<DT>(x[part.edge]) : 0.0f;
  u = id < 0 ? 0.0f : (id >= a.vocab ? nan_f() : u);
  if (id >= a.vocab) id = -1;
  if (tid < n_ids) {
    ids[tid] = static_cast<int32_t>(id);
    up[tid] = u;
  }
  const bool any = __syncthreads_or(u != 0.0f) || dl != 0.0f || dh != 0.0f;
  if (!any || norm.y == 0.0f) {
    zero_part<DT>(d, a.vocab, rank, a.split);
    return;
  }
  float sum = 0.0f;
  for (int j = 0; j < n_ids; ++j) sum += up[j];
  // p = 2^l with l = arg(x) + lift = log2 p; the gradient is p (A + B l)
  const ExpRef ref(norm.x, a.c);
  const float lift = ref.shift - log2f(norm.y), over = ref.k / norm.y;
  const float B = -a.scale * dh * kLn2 * over;
  const float A = a.scale * (dl - sum - (a.d_entropy ? dh * h : 0.0f)) * over;
  auto grad = [&](Pair f) {
    const Pair l = ref.arg(f);
    const float2 g = add2(l, Pair::both(lift)).split();
    const Pair clear = Pair::of(fmaxf(g.x, kFloor), fmaxf(g.y, kFloor));
    return mul2(ex2_pair(l), fma2(Pair::both(B), clear, Pair::both(A)));
  };
  auto grad_flat = [&](Pair f) { return mul2(ex2_pair(ref.arg(f)), Pair::both(A)); };  // no entropy
  // a listed element's whole gradient, by the thread that holds its slot: several slots may name one id, and all
  // of them write the same
  float whole = 0.0f;
  int owner, slot;
  const bool mine = id >= 0 && part.owns(static_cast<int>(id), &owner, &slot);
  if (mine) {
    float v = 0.0f;
    for (int j = 0; j < n_ids; ++j)
      if (ids[j] == static_cast<int32_t>(id)) v += up[j];
    whole = fmaf(a.scale, v, grad(Pair::both(to_float<DT>(x[id]))).split().x);
  }
  __syncthreads();
  if (dh != 0.0f) part.map(first, d, a.vec, edge, grad);
  else part.map(first, d, a.vec, edge, grad_flat);
  __syncthreads();
  if (mine) d[id] = from_float<DT>(whole);
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

ss_status ss_token_logprobs(const ss_logits* x, const void* tokens, ss_idtype idtype, int32_t top_k,
                            const ss_logprob_out* out, void* stream) {
  if (!x || !out || x->rows < 0) return SS_ERR_INVALID_ARG;
  if (idtype != SS_I32 && idtype != SS_I64) return SS_ERR_DTYPE;
  if (x->rows == 0) return SS_OK;
  int64_t x_bytes = 0;
  const ss_status st = check_logits(x, &x_bytes);
  if (st != SS_OK) return st;
  const bool tops = out->top_logprob || out->top_id;
  if (!out->logprob && !out->entropy && !out->lse && !out->norm && !tops) return SS_ERR_INVALID_ARG;
  if (top_k < 0 || top_k > SS_MAX_TOP || top_k > x->vocab || (top_k > 0) != tops) return SS_ERR_INVALID_ARG;
  if (out->logprob && !tokens) return SS_ERR_INVALID_ARG;
  if (x->rows > INT32_MAX) return SS_ERR_OVERFLOW;
  const int64_t ib = idtype == SS_I64 ? 8 : 4, rows = x->rows;
  if (misaligned(tokens, ib) || misaligned(out->top_id, ib) || misaligned(out->logprob, 4) ||
      misaligned(out->entropy, 4) || misaligned(out->lse, 4) ||
      misaligned(out->norm, 8) || misaligned(out->top_logprob, 4))
    return SS_ERR_ALIGN;
  Ranges ranges;
  ranges.add(x->data, x_bytes, false);
  if (out->logprob) ranges.add(tokens, rows * ib, false);
  ranges.add(out->logprob, rows * 4, true);
  ranges.add(out->entropy, rows * 4, true);
  ranges.add(out->lse, rows * 4, true);
  ranges.add(out->norm, rows * 8, true);
  ranges.add(out->top_logprob, rows * top_k * 4, true);
  ranges.add(out->top_id, rows * top_k * ib, true);
  if (ranges.overlap()) return SS_ERR_OVERLAP;
  const LogprobArgs a = {x->data, tokens, out->logprob, out->entropy, out->lse,
                         reinterpret_cast<float2*>(out->norm), out->top_logprob, out->top_id,
                         rows, x->vocab, x->ld, x->scale * kLog2e, x->scale, top_k, idtype == SS_I64};
  const auto pick = [&](auto tops) {
    constexpr bool kTops = decltype(tops)::value;
    return x->dtype == SS_BF16 ? logprob_kernel<SS_BF16, kTops>
                               : (x->dtype == SS_FP16 ? logprob_kernel<SS_FP16, kTops> : logprob_kernel<SS_FP32, kTops>);
  };
  auto* fn = top_k > 0 ? pick(std::true_type()) : pick(std::false_type());
  const int cluster = cluster_for(rows, x->vocab, x->dtype == SS_FP32 ? 4 : 8);
  if (rows * cluster > INT32_MAX) return SS_ERR_OVERFLOW;
  return launch_rows(fn, rows, cluster, kRowThreads, 0, a, stream);
}

ss_status ss_token_logprobs_grad(const ss_logits* x, const void* tokens, ss_idtype idtype, int32_t top_k,
                                 const void* top_id, const float* norm, const float* entropy,
                                 const ss_logprob_grad* up, void* d_logits, int64_t d_ld, void* stream) {
  if (!x || !up || x->rows < 0) return SS_ERR_INVALID_ARG;
  if (idtype != SS_I32 && idtype != SS_I64) return SS_ERR_DTYPE;
  if (x->rows == 0) return SS_OK;
  int64_t x_bytes = 0;
  ss_status st = check_logits(x, &x_bytes);
  if (st != SS_OK) return st;
  if (!norm || !d_logits) return SS_ERR_INVALID_ARG;
  if (!up->d_logprob && !up->d_entropy && !up->d_lse && !up->d_top_logprob) return SS_ERR_INVALID_ARG;
  if (up->d_logprob && !tokens) return SS_ERR_INVALID_ARG;
  if (up->d_entropy && !entropy) return SS_ERR_INVALID_ARG;
  if (top_k < 0 || top_k > SS_MAX_TOP || (top_k > 0) != (up->d_top_logprob != nullptr)) return SS_ERR_INVALID_ARG;
  if (up->d_top_logprob && !top_id) return SS_ERR_INVALID_ARG;
  if (x->rows > INT32_MAX) return SS_ERR_OVERFLOW;
  const int64_t ib = idtype == SS_I64 ? 8 : 4, rows = x->rows;
  if (misaligned(tokens, ib) || misaligned(top_id, ib) || misaligned(norm, 8) || misaligned(entropy, 4) ||
      misaligned(up->d_logprob, 4) || misaligned(up->d_entropy, 4) || misaligned(up->d_lse, 4) ||
      misaligned(up->d_top_logprob, 4))
    return SS_ERR_ALIGN;
  Ranges ranges;
  st = check_grad_out(x, x_bytes, d_logits, d_ld, &ranges);
  if (st != SS_OK) return st;
  if (up->d_logprob) ranges.add(tokens, rows * ib, false);
  ranges.add(norm, rows * 8, false);
  if (up->d_entropy) ranges.add(entropy, rows * 4, false);
  if (up->d_top_logprob) ranges.add(top_id, rows * top_k * ib, false);
  ranges.add(up->d_logprob, rows * 4, false);
  ranges.add(up->d_entropy, rows * 4, false);
  ranges.add(up->d_lse, rows * 4, false);
  ranges.add(up->d_top_logprob, rows * top_k * 4, false);
  if (ranges.overlap()) return SS_ERR_OVERLAP;
  const int split = split_for(x->vocab / (x->dtype == SS_FP32 ? 4 : 8), 16);
  if (rows * split > INT32_MAX) return SS_ERR_OVERFLOW;
  const LogprobGradArgs a = {x->data, tokens, top_id, reinterpret_cast<const float2*>(norm), entropy, up->d_logprob,
                             up->d_entropy, up->d_lse, up->d_top_logprob, d_logits, rows, x->vocab, x->ld, d_ld,
                             x->scale * kLog2e, x->scale, top_k, idtype == SS_I64, same_phase(x, d_logits, d_ld),
                             static_cast<uint32_t>(split)};
  auto* fn = x->dtype == SS_BF16
                 ? logprob_grad_kernel<SS_BF16>
                 : (x->dtype == SS_FP16 ? logprob_grad_kernel<SS_FP16> : logprob_grad_kernel<SS_FP32>);
  return launch(fn, static_cast<unsigned>(rows * split), a, stream, kRowThreads);
}

}  // extern "C"
