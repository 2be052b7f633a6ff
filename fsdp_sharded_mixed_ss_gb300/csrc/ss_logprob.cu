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
  float c, eps, scale;
  int32_t top_k;
  bool wide;  // int64 ids
};

// ------------------------------------------------------------------ forward
//
// One pass over the row gives m = max x, s = sum 2^d and t = sum 2^d d over
// d = (x - m) c: the normaliser, log p_i = (x_i - m) scale - ln s, and the entropy
// H = ln s - ln 2 t / s. It is bound by HBM: 4096 x 128256 bf16 without
// alternatives 164 us, 6.4 TB/s, 0.94 of the measured copy.
//
// The alternatives come from the same pass: the maximum of every unit (4 vectors of
// a thread, more in rows longer than 4096 units a block) stays in shared memory,
// and threads' maxima are 256 keys. Some threshold that k of the keys reach is a
// bound that at least k elements of the row reach, and few more: for k of 256
// keys drawn at random -256 ln(1 - k / 256) elements, 21 for k = 20 and 177 for
// k = 128. Only units whose maximum reaches it are read again, their elements at
// or above it are the candidates, and a candidate's place is the number of
// candidates above it. Where the candidates pass the buffer (ties), the part's
// elements go through the buffer once more, which is cut to the k best whenever
// it is full.
//
// The selection is a chain of small dependent reads beside a loaded memory system,
// as long as a quarter of a 128256-token row's stream, and what bounds the kernel
// with alternatives (2048 x 128256 bf16, 64 of them: 103 us, 5.1 TB/s, 0.75 of the
// copy; the units read again are a tenth more of DRAM traffic). Blocks of 128
// threads, eight to an SM, hide some of it where there are rows enough (103 us
// against 121, and 1021 x 50257 fp32 42 against 48), and the less shared memory
// they take the more L1 is left to the loads in flight (32 maxima a thread in 32
// bits: 128 and 57 us; in 16 bits 114 and 43; candidates in the units' place, 11 KB
// a block instead of 16: a last 1%). What a row issues counts as well: maxima cut
// instead of rounded and a 32-bit index took 114 to 108 us; a batch instead of a
// vector a thread when units are read again (no division, one place taken for all
// its candidates), the bits that all keys share skipped in the search and eight
// candidates compared a step 108 to 105. A ninth warp that selects while eight
// stream the next row measured 139 us, a threshold counted by all threads instead of
// a search in one warp 131, both against 119 then.
//
// A call on a few rows is bound by latencies: 8 x 128256 takes 9 us, of which the
// stream is a fifth, the cluster's two barriers a third.

template <int T>
constexpr int kUnits = 4096 / T;   // maxima kept per thread
template <int T>
constexpr int kFlagged = 4 * T;    // units that are read again
constexpr int kKeys = 256;         // threads' maxima that the threshold is taken from
constexpr int kManyThreads = 128;  // threads of a block that selects alternatives of one of many rows
// So many rows an SM. 256 and 128 threads, us: 50257 bf16 with 20 alternatives, 608 rows 20.0 21.1, 684 rows 30.1 25.1,
// 836 rows 32.1 25.7, 912 rows 33.3 26.4; 128256 bf16 with 64, 36.7 41.6, 55.0 50.2, 58.0 51.7, 60.4 52.7; 50257 fp32
// with 20, 28.7 31.5, 42.6 34.3, 44.6 36.6, 46.1 38.5. Up to 4 rows an SM, one wave of the larger blocks, those are
// ahead; beyond, where they need a second wave, the smaller ones: the rule is never wrong where it takes them, and
// leaves 609 to 911 rows to the slower form.
constexpr int kManyRows = 6;
constexpr uint32_t kMaskedKey = 0x007FFFFFu;  // order_key(-inf)

// Batches in a unit, and units of each thread (the same for all).
template <int DT, int T>
__device__ __forceinline__ int part_unit_batches(const RowPart<DT, T>& part) {
  return ((part.vectors() + kBatch - 1) / kBatch + kUnits<T> - 1) / kUnits<T>;
}
template <int DT, int T>
__device__ __forceinline__ int part_units(const RowPart<DT, T>& part) {
  const int batches = (part.vectors() + kBatch - 1) / kBatch, each = part_unit_batches(part);
  return each > 0 ? (batches + each - 1) / each : 0;
}

// A unit's maximum as the upper half of its key: 16 bits of shared memory, which is the L1 that the loads in flight
// need. Compared with a threshold cut likewise, no unit is missed.
__device__ __forceinline__ uint16_t upper_key(uint32_t key) { return static_cast<uint16_t>(key >> 16); }

// The pass over a thread's vectors; `unit` (with TOPS) receives its units' maxima, `maxima` those of its even and its
// odd units (the even ones' with the edge element).
template <int DT, bool TOPS, int T>
__device__ __forceinline__ RowSum stream_row(const RowPart<DT, T>& part, float c, float edge, uint16_t (*unit)[T],
                                             float (&maxima)[2]) {
  const int full = part.whole / kBatch;  // batches that every thread has whole
  const int batches = (part.vectors() + kBatch - 1) / kBatch;
  const int unit_batches = part_unit_batches(part);
  // ordinary loads, kept in L1 for the units that are read again: the kernel may start while the one ahead still writes
  // the logits, which loads by way of the read-only path do not allow for (they take as long)
  // a 32-bit index beside the units' work, a pointer that advances without it: 2048 x 128256 with 64 alternatives 105 us
  // against 109, 4096 x 128256 without 166 against 168
  const int step = part.step();
  const uint4* src = reinterpret_cast<const uint4*>(part.x + part.sl.head) + (TOPS ? 0 : part.first);
  int at = TOPS ? part.first : 0;
  RunningSum run(one_element(edge), c);
  float best = -kInf;
  maxima[0] = edge;
  maxima[1] = -kInf;
  int in_unit = 0, units = 0;
  for (int b = 0; b < batches; ++b) {
    uint4 w[kBatch];
    if (b < full) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) w[u] = __ldca(src + at + u * step);
    } else {
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        w[u] = part.more(b * kBatch + u)
                   ? __ldca(src + at + u * step)
                   : make_uint4(kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>);
    }
    if constexpr (TOPS) at += kBatch * step;
    else src += kBatch * step;
    const float m = add_vectors<DT>(w, c, run);
    if constexpr (TOPS) {
      best = fmaxf(best, m);
      if (++in_unit == unit_batches || b + 1 == batches) {
        unit[units][threadIdx.x] = upper_key(order_key(best));
        if (units & 1) maxima[1] = fmaxf(maxima[1], best);
        else maxima[0] = fmaxf(maxima[0], best);
        ++units;
        in_unit = 0;
        best = -kInf;
      }
    }
  }
  return run.done(c);
}

template <int T>
struct TopShared {
  static constexpr int kCand = T == kRowThreads ? 1024 : 512;
  static constexpr bool kCandInUnits = T != kRowThreads;  // no cluster: nobody writes before the units are read
  alignas(16) uint16_t unit[kUnits<T>][T];
  alignas(16) uint64_t own_cand[kCandInUnits ? 2 : kCand];
  uint64_t best[SS_MAX_TOP];
  uint32_t keys[kKeys];
  uint16_t flagged[kFlagged<T>];
  int count[kMaxCluster];  // candidates of every block
  int warp_sums[T / 32];
  uint32_t tau;
  int n, n_flagged;

  // Candidates; block 0's are used, shared out over the cluster's blocks.
  __device__ __forceinline__ uint64_t* cand() {
    if constexpr (kCandInUnits) {
      static_assert(sizeof(unit) >= kCand * sizeof(uint64_t), "they fit");
      return reinterpret_cast<uint64_t*>(unit);
    } else {
      return own_cand;
    }
  }
};
struct NoTops {};

// The largest threshold, to the type's digits, that k of the 256 keys reach; a little less is as good. All lanes of
// one warp call it.
template <int DT>
__device__ __forceinline__ uint32_t find_threshold(const uint32_t* key, uint32_t top_key, int k) {
  constexpr int kLowBit = DT == SS_BF16 ? 16 : (DT == SS_FP16 ? 13 : 0);
  uint32_t keys[kKeys / 32];
#pragma unroll
  for (int i = 0; i < kKeys / 32; ++i) keys[i] = key[(threadIdx.x & 31) + 32 * i];
  uint32_t low = keys[0];
#pragma unroll
  for (int i = 1; i < kKeys / 32; ++i) low = min(low, keys[i]);
  const int differ = 32 - __clz(__reduce_min_sync(0xFFFFFFFFu, low) ^ top_key);  // above, all keys are alike
  uint32_t t = differ < 32 ? top_key >> differ << differ : 0u;
#pragma unroll 1
  for (int bit = differ - 1; bit >= kLowBit; --bit) {
    const uint32_t next = t | (1u << bit);
    if (next > top_key) continue;
    int c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kKeys / 32; ++i) c[i & 1] += keys[i] >= next ? 1 : 0;
    const int all = __reduce_add_sync(0xFFFFFFFFu, c[0] + c[1]);
    if (all >= k) {
      t = next;
      if (all <= k + k / 8) break;
    }
  }
  return t;
}

// What a candidate is: at or above the threshold, or, where fewer than k threads hold unmasked tokens, unmasked.
struct Wanted {
  float bound;
  bool few;

  __device__ __forceinline__ explicit Wanted(uint32_t tau) : few(tau <= kMaskedKey) {
    bound = few ? -kInf : key_value(tau);
  }
  __device__ __forceinline__ bool operator()(float f) const { return few ? f > bound : f >= bound; }
};

// The part's candidates into out[0, room); returns their number, to all threads (above `room`: they did not fit).
// s.n and s.n_flagged are zero before; s is the caller's again when this returns.
template <int DT, int T>
__device__ __forceinline__ int collect(const RowPart<DT, T>& part, const Wanted& wanted, uint32_t tau, TopShared<T>& s,
                                       uint64_t* out, int room) {
  constexpr int V = kVecOf<DT>;
  const int tt = threadIdx.x, lane = tt & 31;
  const int unit_batches = part_unit_batches(part), units = part_units(part);
  unsigned mask = 0u;  // this thread's flagged units
  const uint16_t least = upper_key(tau);
  for (int u = 0; u < units; ++u) mask |= s.unit[u][tt] >= least ? 1u << u : 0u;
  int before = __popc(mask);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, before, off);
    if (lane >= off) before += o;
  }
  int base = 0;
  if (lane == 31 && before > 0) base = atomicAdd(&s.n_flagged, before);
  base = __shfl_sync(0xFFFFFFFFu, base, 31) + before - __popc(mask);
  for (; mask != 0u; mask &= mask - 1u, ++base)
    if (base < kFlagged<T>) s.flagged[base] = static_cast<uint16_t>((__ffs(mask) - 1) * T + tt);
  __syncthreads();  // the units have been read: candidates may take their place
  if (part.rank == 0 && tt < 16) {  // the elements outside the vectors
    const int id = tt < 8 ? (tt < part.sl.head ? tt : -1)
                          : (tt - 8 < part.sl.n - part.sl.tail() ? part.sl.tail() + tt - 8 : -1);
    if (id >= 0) {
      const float f = to_float<DT>(part.x[id]);
      if (wanted(f)) {
        const int at = atomicAdd(&s.n, 1);
        if (at < room) out[at] = order_pair(f, id);
      }
    }
  }
  // one batch of a flagged unit a thread
  const int items = min(s.n_flagged, kFlagged<T>) * unit_batches;
#pragma unroll 1
  for (int i = tt; i < items; i += T) {
    const int q = unit_batches == 1 ? i : i / unit_batches;
    const int f = s.flagged[q];
    const int vec = ((f / T) * unit_batches + i - q * unit_batches) * kBatch * part.step() + part.rank * T + f % T;
    uint4 w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      w[u] = vec + u * part.step() < part.sl.nvec
                 ? __ldca(reinterpret_cast<const uint4*>(part.x + part.sl.head) + vec + u * part.step())
                 : make_uint4(kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>);
    unsigned hits = 0u;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      float e[V];
      unpack<DT>(w[u], e);
#pragma unroll
      for (int j = 0; j < V; ++j) hits |= wanted(e[j]) ? 1u << (u * V + j) : 0u;
    }
    int n = hits != 0u ? atomicAdd(&s.n, __popc(hits)) : 0;
    for (; hits != 0u; hits &= hits - 1u, ++n) {
      const int bit = __ffs(hits) - 1;
      const int id = part.sl.head + (vec + bit / V * part.step()) * V + bit % V;
      if (n < room) out[n] = order_pair(to_float<DT>(part.x[id]), id);
    }
  }
  __syncthreads();
  const int n = s.n_flagged > kFlagged<T> ? room + 1 : s.n;
  __syncthreads();  // every thread has read them
  return n;
}

// The k largest of the part's pairs that reach the threshold, into s.best[0, k) in order: the elements go through a
// buffer of pairs (the units' memory), which is cut to its k best, and the bound raised to the last of them,
// whenever it is full. Returns how many there are (k, or all that reach the threshold). Ascending ids make ties cheap:
// a later one is below the bound. How full the buffer is, each thread counts for itself (`n`, from block-wide counts), so all
// decide alike; s.n only hands out places.
template <int DT, int T>
__device__ __noinline__ int select_through_buffer(const RowPart<DT, T>& part, TopShared<T>& s, uint32_t tau, int k) {
  constexpr int V = kVecOf<DT>;
  constexpr int kUnitPairs = static_cast<int>(sizeof(s.unit) / sizeof(uint64_t));
  static_assert(kUnitPairs >= SS_MAX_TOP + T, "a step fits after a cut");
  const int tt = threadIdx.x;
  uint64_t* buffer = reinterpret_cast<uint64_t*>(s.unit);
  uint64_t bound = static_cast<uint64_t>(tau) << 32;  // pairs above it are wanted
  int n = 0;
  if (tt == 0) s.n = 0;
  __syncthreads();
  auto cut = [&] {  // the buffer to its k best, the bound to the k-th
    const int kept = min(n, k);
    for (int i = tt; i < n; i += T) {
      const uint64_t mine = buffer[i];
      int above = 0;
      for (int j = 0; j < n; ++j) above += buffer[j] > mine ? 1 : 0;
      if (above < k) s.best[above] = mine;
    }
    __syncthreads();
    for (int i = tt; i < kept; i += T) buffer[i] = s.best[i];
    if (tt == 0) s.n = kept;
    if (kept == k) bound = s.best[k - 1];
    n = kept;
    __syncthreads();
  };
  auto step = [&](bool there, float f, int id) {  // one element of every thread
    if (n + T > kUnitPairs) cut();
    const uint64_t pair = order_pair(f, id);
    const bool enters = there && pair > bound;
    if (enters) buffer[atomicAdd(&s.n, 1)] = pair;
    n += __syncthreads_count(enters);
  };
  if (part.rank == 0) {
    const bool there = tt < part.sl.head;
    step(there, there ? to_float<DT>(part.x[tt]) : 0.0f, tt);
  }
  const int vectors = part.vectors();
#pragma unroll 1
  for (int j = 0; j < vectors; ++j) {
    const int vec = part.first + j * part.step();
    const bool there = vec < part.sl.nvec;
    uint4 w = make_uint4(kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>, kMaskedWord<DT>);
    if (there) w = __ldca(reinterpret_cast<const uint4*>(part.x + part.sl.head) + vec);
    float e[V];
    unpack<DT>(w, e);
    unsigned hits = 0u;
#pragma unroll
    for (int q = 0; q < V; ++q)
      if (there && order_pair(e[q], part.sl.head + vec * V + q) > bound) hits |= 1u << q;
    if (!__syncthreads_or(hits != 0u)) continue;
#pragma unroll
    for (int q = 0; q < V; ++q) step((hits >> q) & 1u, e[q], part.sl.head + vec * V + q);
  }
  if (part.rank == 0) {
    const int id = part.sl.tail() + tt;
    const bool there = tt < part.sl.n - part.sl.tail();
    step(there, there ? to_float<DT>(part.x[id]) : 0.0f, id);
  }
  cut();
  return n;
}

// Where a row's alternatives go.
struct TopOut {
  float* logprob;
  void* id;
  int64_t base;
  bool wide;

  __device__ __forceinline__ void put(int j, int64_t i, float lp) const {
    if (id) store_id(id, base + j, i, wide);
    if (logprob) logprob[base + j] = lp;
  }
};

// What a row's sums say.
struct RowValues {
  RowSum all;
  float scale, ln_s;
  bool nan, empty;

  __device__ __forceinline__ RowValues(const RowSum& a, float scale_)
      : all(a), scale(scale_), ln_s(logf(a.s)), nan(!(a.s == a.s)), empty(a.s == 0.0f) {}
  __device__ __forceinline__ float logp(float x) const {
    if (nan) return nan_f();
    return empty ? -kInf : scaled_gap(x, all.m, scale, -ln_s);
  }
  __device__ __forceinline__ void write(const LogprobArgs& a, int64_t row, int64_t token, float token_x) const {
    if (a.norm) a.norm[row] = make_float2(all.m, all.s);
    if (a.lse) a.lse[row] = empty ? -kInf : fmaf(all.m, scale, ln_s);
    if (a.entropy) {
      const float h = empty ? 0.0f : ln_s - all.t / all.s * kLn2;
      a.entropy[row] = h < 0.0f ? 0.0f : h;
    }
    if (a.logprob) a.logprob[row] = token < 0 ? 0.0f : (token >= a.vocab ? nan_f() : logp(token_x));
  }
};

// Masked tokens by ascending id into the places from `have` on.
template <int DT, int T>
__device__ __forceinline__ void put_masked(const Elem<DT>* x, int64_t vocab, int have, int k, const TopOut& out,
                                           int* warp_sums) {
  const int tt = threadIdx.x;
  for (int64_t base = 0; base < vocab && have < k; base += T) {
    const int64_t i = base + tt;
    const bool masked = i < vocab && to_float<DT>(x[i]) == -kInf;
    const unsigned votes = __ballot_sync(0xFFFFFFFFu, masked);
    __syncthreads();  // the last round's sums have been read
    if ((tt & 31) == 0) warp_sums[tt >> 5] = __popc(votes);
    __syncthreads();
    int before = have;
    for (int w = 0; w < (T / 32); ++w) {
      if (w < tt >> 5) before += warp_sums[w];
      have += warp_sums[w];
    }
    const int j = before + __popc(votes & ((1u << (tt & 31)) - 1u));
    if (masked && j < k) out.put(j, i, -kInf);
  }
}

// T: threads of a block; 128 for alternatives of many rows, without clusters.
template <int DT, bool TOPS, int T>
__global__ void __launch_bounds__(T, 1024 / T) logprob_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ RowSum red[T / 32];
  __shared__ RowSum parts[kMaxCluster];
  __shared__ std::conditional_t<TOPS, TopShared<T>, NoTops> tops;
  const Cluster cl = T == kRowThreads ? Cluster::start() : Cluster{1, 0};
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / cl.size;
  const RowPart<DT, T> part(static_cast<const Elem<DT>*>(a.x) + row * a.ld, a.vocab, cl.rank, cl.size);
  const float edge = part.edge >= 0 ? to_float<DT>(part.x[part.edge]) : -kInf;
  // the row's token comes beside the pass, its logit beside the sums
  const bool writes = cl.rank == 0 && tid == T - 1;
  int64_t token = -1;
  if (writes && a.logprob) token = load_id(a.tokens, row, a.wide);
  float maxima[2];
  uint16_t(*unit)[T] = nullptr;
  if constexpr (TOPS) unit = tops.unit;
  const RowSum mine_sum = stream_row<DT, TOPS, T>(part, a.c, edge, unit, maxima);
  const Elem<DT> token_x = token >= 0 && token < a.vocab ? part.x[token] : Elem<DT>(0);
  RowSum acc = block_merge<T / 32>(mine_sum, a.c, red);
  cl.started();
  if (cl.size > 1) {
    if (tid < cl.size) cl.at(parts, tid)[cl.rank] = acc;
  }
  if constexpr (TOPS) {
    if constexpr (T == kRowThreads) {
      // 256 keys of the whole row: the maxima of groups of `size` neighbouring threads of every block
      uint32_t key = order_key(fmaxf(maxima[0], maxima[1]));
      for (unsigned off = 1; off < cl.size; off <<= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, off));
      if (tid % cl.size == 0) {
        const unsigned at = cl.rank * (kKeys / cl.size) + tid / cl.size;
        for (unsigned r = 0; r < cl.size; ++r) cl.at(tops.keys, r)[at] = key;
      }
    } else {
      static_assert(kKeys == 2 * T || T == kRowThreads, "two keys a thread");
      tops.keys[tid] = order_key(maxima[0]);
      tops.keys[T + tid] = order_key(maxima[1]);
    }
    if (tid == 0) tops.n = tops.n_flagged = 0;
  }
  if (TOPS || cl.size > 1) cl.sync();
  if (cl.size > 1) acc = merge_lanes(parts[tid % cl.size], a.c, static_cast<int>(cl.size));
  acc.mend(a.eps);
  const RowValues v(acc, a.scale);
  if constexpr (!TOPS) {
    if (writes) v.write(a, row, token, to_float<DT>(token_x));
  } else {
    const int k = a.top_k;
    const TopOut out = {a.top_logprob, a.top_id, row * k, a.wide};
    if (v.nan) {  // in every block of the cluster: all have merged the same parts
      if (writes) v.write(a, row, token, to_float<DT>(token_x));
      if (cl.rank == 0 && tid < k) out.put(tid, -1, nan_f());
      return;
    }
    if (tid < 32) {
      const uint32_t t = find_threshold<DT>(tops.keys, order_key(acc.m), k);
      if (tid == 0) tops.tau = t;
    }
    __syncthreads();
    const uint32_t tau = tops.tau;
    const Wanted wanted(tau);
    const int room = TopShared<T>::kCand / static_cast<int>(cl.size);
    uint64_t* mine = cl.at(tops.cand(), 0) + cl.rank * room;
    const uint32_t least = wanted.few ? kMaskedKey + 1 : tau;
    int found = collect<DT, T>(part, wanted, least, tops, mine, room);
    if (writes) v.write(a, row, token, to_float<DT>(token_x));
    if (found > room) {  // this block's own k best instead
      found = select_through_buffer<DT, T>(part, tops, least, k);
      if (tid < found) mine[tid] = tops.best[tid];
    }
    if (tid < (-found & 7)) mine[found + tid] = 0;  // below every pair: eight are read at a time
    if (tid < cl.size) cl.at(tops.count, tid)[cl.rank] = found;
    cl.sync();
    if (cl.rank != 0) return;
    int total = 0;
    for (unsigned r = 0; r < cl.size; ++r) total += tops.count[r];
    for (int i = tid; i < total; i += T) {
      int r = 0, at = i;
      while (at >= tops.count[r]) at -= tops.count[r++];
      const uint64_t pair = tops.cand()[r * room + at];
      int place = 0;
      for (unsigned q = 0; q < cl.size; ++q)
        for (int j = 0; j < tops.count[q]; j += 8) {
          const auto* four = reinterpret_cast<const ulonglong2*>(tops.cand() + q * room + j);
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const ulonglong2 two = four[h];
            place += (two.x > pair ? 1 : 0) + (two.y > pair ? 1 : 0);
          }
        }
      if (place < k)
        out.put(place, static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(pair)),
                v.logp(key_value(static_cast<uint32_t>(pair >> 32))));
    }
    if (wanted.few && total < k) put_masked<DT, T>(part.x, a.vocab, total, k, out, tops.warp_sums);
  }
}

// Blocks that share a row: rows alone fill the GPU from about 4 blocks on each SM; fewer rows are split while
// every thread keeps half a batch of vectors. 1, 2, 4, 8 blocks: 8 x 128256 bf16 14.3, 11.4, 9.4, 9.1 us; 4096 rows
// of it (no alternatives) 164, 177, 213 us for 1, 2, 4.
int cluster_for(int64_t rows, int64_t vocab, int vec) {
  const int64_t blocks = 4 * std::max(1, sm_count());
  int c = 1;
  const int64_t least = static_cast<int64_t>(kRowThreads) * kBatch * vec;
  while (c < kMaxCluster && rows * c * 2 <= blocks && vocab >= c * least)
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
// Bound by HBM: 2048 x 128256 bf16 156 us, 6.74 TB/s, as fast as the copy (parts
// of 8, 16, 32, 64 vectors a thread: 165, 156, 160, 165 us); 509 x 50257 fp32 36 us,
// 0.85 of it, a row and a half of such parts an SM slot.
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
  auto from_arg = [&](Pair l) {
    const float2 g = add2(l, Pair::both(lift)).split();
    const Pair clear = Pair::of(fmaxf(g.x, kFloor), fmaxf(g.y, kFloor));
    return mul2(ex2_pair(l), fma2(Pair::both(B), clear, Pair::both(A)));
  };
  auto grad = [&](Pair f) { return from_arg(ref.arg<false>(f)); };
  auto grad_flat = [&](Pair f) { return mul2(ex2_pair(ref.arg<false>(f)), Pair::both(A)); };  // no entropy
  auto grad_far = [&](Pair f) { return from_arg(ref.arg<true>(f)); };
  // a listed element's whole gradient, by the thread that holds its slot: several slots may name one id, and all
  // of them write the same
  float whole = 0.0f;
  int owner, slot;
  const bool mine = id >= 0 && part.owns(static_cast<int>(id), &owner, &slot);
  if (mine) {
    float v = 0.0f;
    for (int j = 0; j < n_ids; ++j)
      if (ids[j] == static_cast<int32_t>(id)) v += up[j];
    whole = fmaf(a.scale, v, from_arg(Pair::both(ref.arg(to_float<DT>(x[id])))).split().x);
  }
  __syncthreads();
  if (ref.far) part.map(first, d, a.vec, edge, grad_far);
  else if (dh != 0.0f) part.map(first, d, a.vec, edge, grad);
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
  const Scale2 s2(x->scale);
  const LogprobArgs a = {x->data, tokens, out->logprob, out->entropy, out->lse,
                         reinterpret_cast<float2*>(out->norm), out->top_logprob, out->top_id,
                         rows, x->vocab, x->ld, s2.c, s2.eps, x->scale, top_k, idtype == SS_I64};
  const auto pick = [&](auto tops, auto threads) {
    constexpr bool kTops = decltype(tops)::value;
    constexpr int T = decltype(threads)::value;
    return x->dtype == SS_BF16 ? logprob_kernel<SS_BF16, kTops, T>
                               : (x->dtype == SS_FP16 ? logprob_kernel<SS_FP16, kTops, T>
                                                      : logprob_kernel<SS_FP32, kTops, T>);
  };
  constexpr std::integral_constant<int, kRowThreads> wide_block;
  constexpr std::integral_constant<int, kManyThreads> small_block;
  const int vec = x->dtype == SS_FP32 ? 4 : 8, cluster = cluster_for(rows, x->vocab, vec);
  if (rows * cluster > INT32_MAX) return SS_ERR_OVERFLOW;
  if (top_k > 0 && rows >= kManyRows * sm_count() && x->vocab / vec >= 8 * kBatch * kManyThreads) {
    return launch_rows(pick(std::true_type(), small_block), rows, 1, kManyThreads, 0, a, stream);
  }
  auto* fn = top_k > 0 ? pick(std::true_type(), wide_block) : pick(std::false_type(), wide_block);
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
                             Scale2(x->scale).c, x->scale, top_k, idtype == SS_I64, same_phase(x, d_logits, d_ld),
                             static_cast<uint32_t>(split)};
  auto* fn = x->dtype == SS_BF16
                 ? logprob_grad_kernel<SS_BF16>
                 : (x->dtype == SS_FP16 ? logprob_grad_kernel<SS_FP16> : logprob_grad_kernel<SS_FP32>);
  return launch(fn, static_cast<unsigned>(rows * split), a, stream, kRowThreads);
}

}  // extern "C"
