// ss_embed.cu -- rows of an embedding table by token, scaled (ss_embedding), and the
// table's gradient as the sums of each token's positions in sorted order
// (ss_embedding_grad).
#include "ss_logits.cuh"

namespace ss {
namespace {

// ------------------------------------------------------------------ eight elements of a row

// Elements e .. e + 7 of a row as fp32: as 16-byte vectors (VEC), or one by one, those from `dim` on left 0.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* row, int e, int dim, float (&f)[8]) {
  const Elem<DT>* p = static_cast<const Elem<DT>*>(row) + e;
  if (VEC && e + 8 <= dim) {
    if constexpr (DT == SS_FP32) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
      widen8<DT>(*reinterpret_cast<const uint4*>(p), f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = e + j < dim ? to_float<DT>(p[j]) : 0.0f;
  }
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(void* row, int e, int dim, const float (&f)[8]) {
  Elem<DT>* p = static_cast<Elem<DT>*>(row) + e;
  if (VEC && e + 8 <= dim) {
    if constexpr (DT == SS_FP32) {
      reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *reinterpret_cast<uint4*>(p) = narrow8<DT>(f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + j < dim) p[j] = from_float<DT>(f[j]);
  }
}

// Eight elements as they lie in memory.
template <int DT>
struct Raw8 {
  uint4 w[DT == SS_FP32 ? 2 : 1];

  template <bool VEC>
  __device__ __forceinline__ void load(const void* row, int e, int dim) {
    const Elem<DT>* p = static_cast<const Elem<DT>*>(row) + e;
    if (VEC && e + 8 <= dim) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(w) / 16); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
      uint32_t* q = &w[0].x;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Elem<DT> v = e + j < dim ? p[j] : Elem<DT>(0);
        if constexpr (DT == SS_FP32) q[j] = __float_as_uint(v);
        else q[j / 2] = j % 2 ? q[j / 2] | static_cast<uint32_t>(v) << 16 : v;
      }
    }
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    if constexpr (DT == SS_FP32) {
      const uint32_t* q = &w[0].x;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(q[j]);
    } else {
      widen8<DT>(w[0], f);
    }
  }
  __device__ __forceinline__ void add_to(float (&sum)[8]) const {
    float f[8];
    unpack(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += f[j];
  }
};

// The same of a type known at run time (a branch that all threads take alike).
template <bool VEC>
__device__ __forceinline__ void load8(int dt, const void* row, int e, int dim, float (&f)[8]) {
  if (dt == SS_BF16) load8<SS_BF16, VEC>(row, e, dim, f);
  else if (dt == SS_FP16) load8<SS_FP16, VEC>(row, e, dim, f);
  else load8<SS_FP32, VEC>(row, e, dim, f);
}
template <bool VEC>
__device__ __forceinline__ void store8(int dt, void* row, int e, int dim, const float (&f)[8]) {
  if (dt == SS_BF16) store8<SS_BF16, VEC>(row, e, dim, f);
  else if (dt == SS_FP16) store8<SS_FP16, VEC>(row, e, dim, f);
  else store8<SS_FP32, VEC>(row, e, dim, f);
}

struct Rows {
  void* data;
  int64_t ld;
  int32_t dtype;

  __device__ __forceinline__ char* row(int64_t r) const {
    return static_cast<char*>(data) + r * ld * (dtype == SS_FP32 ? 4 : 2);
  }
};

constexpr int kRowPiece = 1024;  // elements of a row that a warp takes at a time

// ------------------------------------------------------------------ lookup
//
// A warp takes up to 1024 elements of a position's row.

struct LookupArgs {
  const void* ids;
  Rows table, out;
  int64_t n, vocab;
  int32_t dim, pieces;  // pieces of a row
  float scale;
  bool wide;
};

template <int DT, int OT, bool VEC>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const __grid_constant__ LookupArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32), tasks = a.n * a.pieces;
  int64_t task = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  // the next task's row is on its way while this one's is written, and the id of the one after
  auto id_at = [&](int64_t t) { return t < tasks ? load_id(a.ids, t / a.pieces, a.wide) : -1; };
  auto fetch = [&](int64_t t, int64_t id, Raw8<DT> (&raw)[4]) {
    if (id < 0 || id >= a.vocab) return;
    const char* row = a.table.row(id);
    const int from = static_cast<int>(t % a.pieces) * kRowPiece;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = from + (u * 32 + lane) * 8;
      if (e < a.dim) raw[u].template load<VEC>(row, e, a.dim);
    }
  };
  int64_t id = id_at(task), next_id = id_at(task + warps);
  Raw8<DT> raw[4];
  fetch(task, id, raw);
  for (; task < tasks; task += warps) {
    Raw8<DT> next[4];
    fetch(task + warps, next_id, next);
    const int64_t after = id_at(task + 2 * warps);
    char* out = a.out.row(task / a.pieces);
    const int from = static_cast<int>(task % a.pieces) * kRowPiece;
    const bool there = id >= 0 && id < a.vocab;
    const float none = id < 0 ? 0.0f : nan_f();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = from + (u * 32 + lane) * 8;
      float f[8];
      raw[u].unpack(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = there ? f[j] * a.scale : none;
      if (e < a.dim) store8<OT, VEC>(out, e, a.dim, f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) raw[u] = next[u];
    id = next_id;
    next_id = after;
  }
}

// ------------------------------------------------------------------ positions in order of their tokens
//
// A stable radix sort of (token, position) by one cluster of blocks, so that a
// token's positions stand together and in ascending order: that order is the order
// of the sums. Every warp has a run of consecutive pairs. A pass counts each warp's
// digits, turns the counts into places (by digit, then by warp) and moves the pairs
// there, 32 at a time; the places of equal digits within them come from a match over
// the lanes. Positions without a token (a negative id, or one past the vocabulary)
// go behind the last one.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBlocks = 8;
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;

// What the sums are made of: up to kChunk sorted positions of one token, those of one aligned run of kChunk.
constexpr int kChunk = 32;  // a warp's lanes: a warp that goes through the sorted positions sees a whole run at a time
struct Task {
  int32_t at;        // first sorted position
  uint32_t token;
  int32_t count;     // positions; negative where the token has positions in other runs as well
  int32_t first;     // its first position's row; its token's number among those that occur where count is negative
};

struct SortArgs {
  const void* ids;
  uint64_t* pairs[2];  // token << 32 | position; the sorted ones are in pairs[passes & 1 ? 0 : 1]
  Task* tasks;
  int32_t* first_task;  // of every token that occurs; then their number
  int32_t* n_tasks;
  uint32_t* arrived;    // n_arrived counters, to be cleared
  int64_t n_arrived, vocab;
  int32_t n, passes, bits;  // bits of a digit
  bool wide;
};

__device__ __forceinline__ uint32_t token_of(uint64_t pair) { return static_cast<uint32_t>(pair >> 32); }

struct SortShared {
  uint32_t count[kSortWarps][kDigits];  // of a warp's digits; then the next place of each
  uint32_t total[kDigits];              // of the block's digits
  uint32_t base[kDigits];
  uint32_t warp_sum[kSortWarps];
  uint2 warp_tasks[kSortWarps];  // tasks and tokens that begin in a warp's run
  uint2 block_tasks;
};

__device__ void sort_positions(const SortArgs& a, const Cluster& cl, SortShared& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.n;
  // this warp's run
  const int64_t each = (static_cast<int64_t>(n) + kSortBlocks * kSortWarps * 32 - 1) / (kSortBlocks * kSortWarps * 32) * 32;
  const int64_t first = (static_cast<int64_t>(cl.rank) * kSortWarps + warp) * each;
  const int64_t last = min(first + each, static_cast<int64_t>(n));
  const uint32_t none = static_cast<uint32_t>(a.vocab);
  for (int64_t i = static_cast<int64_t>(cl.rank) * kSortThreads + tid; i < a.n_arrived; i += kSortBlocks * kSortThreads)
    a.arrived[i] = 0u;
  for (int pass = 0; pass < a.passes; ++pass) {
    const uint64_t* from = a.pairs[(pass & 1) ^ 1];
    uint64_t* to = a.pairs[pass & 1];
    const int shift = pass * a.bits;
    const uint32_t mask = (1u << a.bits) - 1u;
    auto pair_at = [&](int64_t i) -> uint64_t {
      if (pass > 0) return __ldcg(reinterpret_cast<const unsigned long long*>(from) + i);
      const int64_t id = load_id(a.ids, i, a.wide);
      const uint32_t key = id < 0 || id >= a.vocab ? none : static_cast<uint32_t>(id);
      return static_cast<uint64_t>(key) << 32 | static_cast<uint32_t>(i);
    };
    auto digit_of = [&](uint64_t pair) { return static_cast<uint32_t>(pair >> (32 + shift)) & mask; };
    for (int d = lane; d < kDigits; d += 32) s.count[warp][d] = 0;
    __syncwarp();
    for (int64_t i = first + lane; i < last; i += 32) atomicAdd(&s.count[warp][digit_of(pair_at(i))], 1u);
    __syncthreads();
    if (tid < kDigits) {
      uint32_t sum = 0;
      for (int w = 0; w < kSortWarps; ++w) sum += s.count[w][tid];
      s.total[tid] = sum;
    }
    cl.sync();
    // places: all smaller digits of all blocks, this digit of the blocks before, of the warps before
    if (tid < kDigits) {
      uint32_t all = 0, before = 0;
      for (unsigned r = 0; r < cl.size; ++r) {
        const uint32_t t = cl.at(s.total, r)[tid];
        before += r < cl.rank ? t : 0u;
        all += t;
      }
      uint32_t upto = all;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
        if (lane >= off) upto += o;
      }
      if (lane == 31) s.warp_sum[warp] = upto;
      s.base[tid] = upto - all + before;
    }
    __syncthreads();
    if (tid < kDigits) {
      uint32_t at = s.base[tid];
      for (int w = 0; w < warp; ++w) at += s.warp_sum[w];
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = s.count[w][tid];
        s.count[w][tid] = at;
        at += c;
      }
    }
    __syncthreads();
    for (int64_t i = first; i < last; i += 32) {
      const bool there = i + lane < last;
      const uint64_t pair = there ? pair_at(i + lane) : 0u;
      const uint32_t digit = there ? digit_of(pair) : kDigits;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, digit);
      if (there) {
        const uint32_t at = s.count[warp][digit] + __popc(same & ((1u << lane) - 1u));
        to[at] = pair;
      }
      __syncwarp();
      if (there && (same >> lane) == 1u) s.count[warp][digit] += __popc(same);  // the last of its digit
      __syncwarp();
    }
    // the pairs, and the reads of this block's totals, are over before the next pass begins in any block
    __threadfence();
    cl.sync();
  }
  // the tasks, in the order of their positions: counted, then written
  const auto* sorted = reinterpret_cast<const unsigned long long*>(a.pairs[a.passes & 1 ? 0 : 1]);
  auto over_runs = [&](const auto& f) {
    uint32_t before = first > 0 && first < last ? token_of(__ldcg(sorted + first - 1)) : ~0u;
    for (int64_t i = first; i < last; i += kChunk) {
      const uint64_t pair = i + lane < last ? __ldcg(sorted + i + lane) : ~0ull;
      const uint32_t token = token_of(pair);
      uint32_t prev = __shfl_up_sync(0xFFFFFFFFu, token, 1);
      if (lane == 0) prev = before;
      before = __shfl_sync(0xFFFFFFFFu, token, 31);
      const bool live = token < none, begins = live && token != prev;
      f(i, pair, live, begins, __ballot_sync(0xFFFFFFFFu, begins), __ballot_sync(0xFFFFFFFFu, begins || (live && lane == 0)));
    }
  };
  uint2 here = make_uint2(0, 0);
  over_runs([&](int64_t, uint64_t, bool, bool, unsigned tokens, unsigned tasks) {
    here.x += __popc(tasks);
    here.y += __popc(tokens);
  });
  if (lane == 0) s.warp_tasks[warp] = here;
  __syncthreads();
  if (warp == 0) {  // sums before each warp, and the block's
    const uint2 own = s.warp_tasks[lane];
    uint2 upto = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, upto.x, off), y = __shfl_up_sync(0xFFFFFFFFu, upto.y, off);
      if (lane >= off) upto = make_uint2(upto.x + x, upto.y + y);
    }
    s.warp_tasks[lane] = make_uint2(upto.x - own.x, upto.y - own.y);
    if (lane == 31) s.block_tasks = upto;
  }
  cl.sync();
  uint2 at = s.warp_tasks[warp], all = make_uint2(0, 0);
  for (unsigned r = 0; r < cl.size; ++r) {
    const uint2 b = *cl.at(&s.block_tasks, r);
    if (r < cl.rank) at = make_uint2(at.x + b.x, at.y + b.y);
    all = make_uint2(all.x + b.x, all.y + b.y);
  }
  over_runs([&](int64_t i, uint64_t pair, bool live, bool begins, unsigned tokens, unsigned tasks) {
    const uint32_t token = token_of(pair);
    const unsigned below = (1u << lane) - 1u, behind = lane == 31 ? 0u : tasks >> (lane + 1) << (lane + 1);
    const int in_run = __popc(__ballot_sync(0xFFFFFFFFu, live));
    if ((tasks >> lane) & 1u) {
      const int end = behind ? __ffs(behind) - 1 : in_run;
      const bool goes_on = end == kChunk && i + kChunk < n && token_of(__ldcg(sorted + i + kChunk)) == token;
      const uint32_t task = at.x + __popc(tasks & below), number = at.y + __popc(tokens & (below | 1u << lane)) - 1u;
      const bool parts = goes_on || !begins;
      a.tasks[task] = {static_cast<int32_t>(i) + lane, token, parts ? lane - end : end - lane,
                       parts ? static_cast<int32_t>(number) : static_cast<int32_t>(static_cast<uint32_t>(pair))};
      if (begins) a.first_task[number] = static_cast<int32_t>(task);
    }
    at.x += __popc(tasks);
    at.y += __popc(tokens);
  });
  if (cl.rank == 0 && tid == 0) {
    *a.n_tasks = static_cast<int32_t>(all.x);
    a.first_task[all.y] = static_cast<int32_t>(all.x);
  }
  cl.sync();  // the other blocks have read this one's totals
}

struct FillArgs {
  Rows base, table;  // base.data null: zeros
  int64_t vocab;
  int32_t dim, pieces;
};

// The table's rows as they are without any token: zeros, or the base's.
template <bool VEC>
__device__ __forceinline__ void fill_rows(const FillArgs& a, int64_t warp, int64_t warps) {
  const int lane = threadIdx.x & 31;
  for (int64_t task = warp; task < a.vocab * a.pieces; task += warps) {
    const int64_t r = task / a.pieces;
    const int from = static_cast<int>(task - r * a.pieces) * kRowPiece;
    char* out = a.table.row(r);
    const char* base = a.base.data ? a.base.row(r) : nullptr;
    float f[4][8] = {};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = from + (u * 32 + lane) * 8;
      if (base && e < a.dim) load8<VEC>(a.base.dtype, base, e, a.dim, f[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = from + (u * 32 + lane) * 8;
      if (e < a.dim) store8<VEC>(a.table.dtype, out, e, a.dim, f[u]);
    }
  }
}

struct SortFillArgs {
  SortArgs sort;
  FillArgs fill;
};

// Cluster 0 sorts; the others fill the table meanwhile.
template <bool VEC>
__global__ void __launch_bounds__(kSortThreads, 1) sort_fill_kernel(const __grid_constant__ SortFillArgs a) {
  extern __shared__ char shared[];
  const Cluster cl = Cluster::start();
  pdl_wait();
  pdl_trigger();
  cl.started();
  if (blockIdx.x < kSortBlocks) {
    if (a.sort.n == 0) return;  // there is no workspace then
    sort_positions(a.sort, cl, *reinterpret_cast<SortShared*>(shared));
  } else {
    const int64_t warp = static_cast<int64_t>(blockIdx.x - kSortBlocks) * kSortWarps + (threadIdx.x >> 5);
    fill_rows<VEC>(a.fill, warp, static_cast<int64_t>(gridDim.x - kSortBlocks) * kSortWarps);
  }
}

// ------------------------------------------------------------------ the sums
//
// A warp takes a task's positions and up to 512 columns. A token with one task is
// finished by it. A token with more leaves each task's sum in the workspace, and
// whichever warp is the last to do so of kGroup neighbouring runs adds these up, and the
// last of those the groups' sums: the order of the sums is that of the positions
// whichever warp adds them.

constexpr int kGroup = 16;
constexpr int kSumThreads = 256;
constexpr int kVecs = 2;                   // groups of eight columns that a lane has
constexpr int kSumPiece = kVecs * 32 * 8;  // columns that a warp takes at a time

struct SumArgs {
  const uint64_t* pairs;
  const Task* tasks;
  const int32_t* first_task;
  const int32_t* n_tasks;
  uint32_t* arrived;  // [2][2 runs][pieces]: of a token's tasks in a group of runs, of its groups
  float* partial;     // [2 runs][pitch]: of the token that a run begins with, of the one that it ends with
  Rows d_out, base, table;
  int64_t pitch;
  int32_t runs, dim, pieces;
  float scale;
};

struct Columns {
  int from, dim, lane;
  __device__ __forceinline__ int at(int u) const { return from + (u * 32 + lane) * 8; }
};

// A token's row from its sum.
template <bool VEC>
__device__ __forceinline__ void finish_row(const SumArgs& a, uint32_t token, const Columns& c, const float (&sum)[kVecs][8]) {
  char* out = a.table.row(token);
  float f[kVecs][8] = {};
  if (a.base.data) {
    const char* base = a.base.row(token);
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
      if (c.at(u) < c.dim) load8<VEC>(a.base.dtype, base, c.at(u), c.dim, f[u]);
  }
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[u][j] = fmaf(sum[u][j], a.scale, f[u][j]);
    if (c.at(u) < c.dim) store8<VEC>(a.table.dtype, out, c.at(u), c.dim, f[u]);
  }
}

// The sums of a token's tasks: one in each of the runs from `first` to `last`.
struct TokenParts {
  int first, last;  // runs
  bool inside;      // it begins inside its first run

  __device__ __forceinline__ int64_t slot(int run) const { return 2 * static_cast<int64_t>(run) + (run == first && inside); }
};

__device__ __forceinline__ void add_partial(const SumArgs& a, int64_t slot, const Columns& c, float (&sum)[kVecs][8]) {
  const float* p = a.partial + slot * a.pitch;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int e = c.at(u);
    if (e < c.dim) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(p + e)), y = __ldcg(reinterpret_cast<const float4*>(p + e + 4));
      const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[u][j] += f[j];
    }
  }
}

__device__ __forceinline__ void put_partial(const SumArgs& a, int64_t slot, const Columns& c, const float (&sum)[kVecs][8]) {
  float* p = a.partial + slot * a.pitch;
#pragma unroll
  for (int u = 0; u < kVecs; ++u)
    if (c.at(u) < c.dim) store8<SS_FP32, true>(p, c.at(u), static_cast<int>(a.pitch), sum[u]);
}

// Whether this warp is the last of `of` that arrive at a counter; what the others wrote before they did is then seen.
__device__ __forceinline__ bool last_to_arrive(uint32_t* counter, int of, int lane) {
  __threadfence();
  __syncwarp();
  uint32_t before = 0;
  if (lane == 0) before = atomicAdd(counter, 1u);
  const bool last = __shfl_sync(0xFFFFFFFFu, before, 0) == static_cast<uint32_t>(of - 1);
  __threadfence();
  return last;
}

// A part's sum on its way to its token's row.
template <bool VEC>
__device__ __forceinline__ void join_parts(const SumArgs& a, const Task& task, int piece, const Columns& c,
                                           float (&sum)[kVecs][8]) {
  const int begin = a.first_task[task.first], parts = a.first_task[task.first + 1] - begin;
  const int start = a.tasks[begin].at;
  TokenParts t;
  t.first = start / kChunk;
  t.last = t.first + parts - 1;
  t.inside = start % kChunk != 0;
  const int run = task.at / kChunk;
  put_partial(a, t.slot(run), c, sum);
  // this group's parts
  const int lo = max(t.first, run / kGroup * kGroup), hi = min(t.last, run / kGroup * kGroup + kGroup - 1);
  uint32_t* arrived = a.arrived + t.slot(lo) * a.pieces + piece;
  if (!last_to_arrive(arrived, hi - lo + 1, c.lane)) return;
#pragma unroll
  for (int u = 0; u < kVecs; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[u][j] = 0.0f;
#pragma unroll 2
  for (int r = lo; r <= hi; ++r) add_partial(a, t.slot(r), c, sum);
  const int groups = t.last / kGroup - t.first / kGroup + 1;
  if (groups > 1) {
    put_partial(a, t.slot(lo), c, sum);
    arrived = a.arrived + (2 * static_cast<int64_t>(a.runs) + t.slot(t.first)) * a.pieces + piece;
    if (!last_to_arrive(arrived, groups, c.lane)) return;
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[u][j] = 0.0f;
#pragma unroll 2
    for (int g = t.first / kGroup; g <= t.last / kGroup; ++g) add_partial(a, t.slot(max(t.first, g * kGroup)), c, sum);
  }
  finish_row<VEC>(a, task.token, c, sum);
}

template <int DT>
constexpr int kInFlight = DT == SS_FP32 ? 1 : 2;  // rows that a warp has in flight

template <int DT, bool VEC, bool TVEC>
__global__ void __launch_bounds__(kSumThreads, 4) sum_kernel(const __grid_constant__ SumArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kSumThreads / 32);
  const int64_t items = static_cast<int64_t>(*a.n_tasks) * a.pieces;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kSumThreads / 32) + (threadIdx.x >> 5); item < items;
       item += warps) {
    const int64_t j = item / a.pieces;
    const int piece = static_cast<int>(item - j * a.pieces);
    const int4 words = *reinterpret_cast<const int4*>(a.tasks + j);
    const Task task = {words.x, static_cast<uint32_t>(words.y), words.z, words.w};
    const int count = abs(task.count);
    const Columns c = {piece * kSumPiece, a.dim, lane};
    // lane i has the row of the task's i-th position
    const int32_t row = task.count == 1 ? task.first
                                        : static_cast<int32_t>(static_cast<uint32_t>(a.pairs[task.at + min(lane, count - 1)]));
    float sum[kVecs][8] = {};
    for (int i = 0; i < count; i += kInFlight<DT>) {
      Raw8<DT> f[kInFlight<DT>][kVecs];
#pragma unroll
      for (int r = 0; r < kInFlight<DT>; ++r) {
        const char* p = a.d_out.row(__shfl_sync(0xFFFFFFFFu, row, min(i + r, count - 1)));
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
          if (i + r < count && c.at(u) < c.dim) f[r][u].template load<VEC>(p, c.at(u), c.dim);
      }
#pragma unroll
      for (int r = 0; r < kInFlight<DT>; ++r)
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
          if (i + r < count && c.at(u) < c.dim) f[r][u].add_to(sum[u]);
    }
    if (task.count > 0) finish_row<TVEC>(a, task.token, c, sum);
    else join_parts<TVEC>(a, task, piece, c, sum);
  }
}

// ------------------------------------------------------------------ host

int64_t pitch_of(int64_t dim) { return (dim + 7) / 8 * 8; }
int pieces_of(int64_t dim, int piece) { return static_cast<int>((dim + piece - 1) / piece); }

// The workspace's parts, each on a 16-byte boundary: where they begin, and its bytes (-1: more than int64 holds).
struct Workspace {
  int64_t runs, n_arrived;
  int64_t pairs[2], tasks, first_task, n_tasks, arrived, partial, bytes;

  Workspace(int64_t n, int64_t dim) {
    runs = (n + kChunk - 1) / kChunk;
    n_arrived = 4 * runs * pieces_of(dim, kSumPiece);
    __int128 at = 0;
    const auto take = [&](__int128 size) {
      const __int128 from = at;
      at += (size + 15) / 16 * 16;
      return static_cast<int64_t>(from);
    };
    pairs[0] = take(static_cast<__int128>(n) * 8);
    pairs[1] = take(static_cast<__int128>(n) * 8);
    tasks = take(static_cast<__int128>(n) * static_cast<int64_t>(sizeof(Task)));
    first_task = take((static_cast<__int128>(n) + 1) * 4);
    n_tasks = take(4);
    arrived = take(static_cast<__int128>(n_arrived) * 4);
    partial = take(static_cast<__int128>(runs) * 2 * pitch_of(dim) * 4);
    bytes = at > INT64_MAX ? -1 : static_cast<int64_t>(at);
  }
};

ss_status check_table(const ss_table* t, int64_t* bytes) {
  if (!t->data || t->vocab < 1 || t->dim < 1 || t->ld < t->dim) return SS_ERR_INVALID_ARG;
  if (t->vocab >= INT32_MAX || t->dim > SS_MAX_DIM) return SS_ERR_OVERFLOW;
  if (!is_float_dtype(t->dtype)) return SS_ERR_DTYPE;
  if (misaligned(t->data, dtype_bytes(t->dtype))) return SS_ERR_ALIGN;
  if (!span_bytes(t->vocab, t->dim, t->ld, dtype_bytes(t->dtype), bytes)) return SS_ERR_OVERFLOW;
  return SS_OK;
}

// The same of the positions' rows (n > 0).
ss_status check_rows(const void* p, int64_t n, int64_t dim, int64_t ld, int32_t dtype, int64_t* bytes) {
  if (!p || ld < dim) return SS_ERR_INVALID_ARG;
  if (!is_float_dtype(dtype)) return SS_ERR_DTYPE;
  if (misaligned(p, dtype_bytes(dtype))) return SS_ERR_ALIGN;
  if (!span_bytes(n, dim, ld, dtype_bytes(dtype), bytes)) return SS_ERR_OVERFLOW;
  return SS_OK;
}

// Whether every row begins on a 16-byte boundary.
bool aligned_rows(const Rows& r) {
  return !misaligned(r.data, 16) && r.ld * dtype_bytes(r.dtype) % 16 == 0;
}

template <int DT, bool VEC>
auto pick_lookup(int32_t out) {
  return out == SS_BF16 ? lookup_kernel<DT, SS_BF16, VEC>
                        : (out == SS_FP16 ? lookup_kernel<DT, SS_FP16, VEC> : lookup_kernel<DT, SS_FP32, VEC>);
}
template <bool VEC>
auto pick_lookup(int32_t table, int32_t out) {
  return table == SS_BF16 ? pick_lookup<SS_BF16, VEC>(out)
                          : (table == SS_FP16 ? pick_lookup<SS_FP16, VEC>(out) : pick_lookup<SS_FP32, VEC>(out));
}

ss_status lookup_impl(const ss_table* t, const void* ids, ss_idtype idtype, int64_t n, float scale, void* out,
                      int32_t out_dtype, int64_t out_ld, void* stream) {
  int64_t t_bytes = 0, o_bytes = 0;
  ss_status st = check_table(t, &t_bytes);
  if (st != SS_OK) return st;
  if (!ids || !std::isfinite(scale)) return SS_ERR_INVALID_ARG;
  if (idtype != SS_I32 && idtype != SS_I64) return SS_ERR_DTYPE;
  st = check_rows(out, n, t->dim, out_ld, out_dtype, &o_bytes);
  if (st != SS_OK) return st;
  const int64_t ib = idtype == SS_I64 ? 8 : 4;
  if (misaligned(ids, ib)) return SS_ERR_ALIGN;
  if (n > INT32_MAX) return SS_ERR_OVERFLOW;
  Ranges ranges;
  ranges.add(t->data, t_bytes, false);
  ranges.add(ids, n * ib, false);
  ranges.add(out, o_bytes, true);
  if (ranges.overlap()) return SS_ERR_OVERLAP;
  const LookupArgs a = {ids, {t->data, t->ld, t->dtype}, {out, out_ld, out_dtype}, n, t->vocab,
                        static_cast<int32_t>(t->dim), pieces_of(t->dim, kRowPiece), scale, idtype == SS_I64};
  auto* fn = aligned_rows(a.table) && aligned_rows(a.out) ? pick_lookup<true>(t->dtype, out_dtype)
                                                          : pick_lookup<false>(t->dtype, out_dtype);
  return launch(fn, grid_for(reinterpret_cast<const void*>(fn), n * a.pieces * 32), a, stream);
}

template <int DT>
auto pick_sum(bool vec, bool tvec) {
  return vec ? (tvec ? sum_kernel<DT, true, true> : sum_kernel<DT, true, false>)
             : (tvec ? sum_kernel<DT, false, true> : sum_kernel<DT, false, false>);
}

// Shared memory past 48 KB has to be asked for, once a device.
template <typename Fn>
ss_status allow_shared(Fn* fn, size_t bytes) {
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  return e == cudaSuccess ? SS_OK : cuda_fail(e);
}

ss_status grad_impl(const void* d_out, int32_t d_dtype, int64_t d_ld, const void* ids, ss_idtype idtype, int64_t n,
                    float scale, const ss_table* base, const ss_table* t, void* workspace, int64_t workspace_bytes,
                    void* stream) {
  int64_t t_bytes = 0, b_bytes = 0, d_bytes = 0;
  ss_status st = check_table(t, &t_bytes);
  if (st != SS_OK) return st;
  if (base) {
    st = check_table(base, &b_bytes);
    if (st != SS_OK) return st;
    if (base->vocab != t->vocab || base->dim != t->dim) return SS_ERR_INVALID_ARG;
  }
  if (!std::isfinite(scale)) return SS_ERR_INVALID_ARG;
  if (idtype != SS_I32 && idtype != SS_I64) return SS_ERR_DTYPE;
  const int64_t ib = idtype == SS_I64 ? 8 : 4;
  const Workspace ws(std::min<int64_t>(n, INT32_MAX), t->dim);
  if (n > 0) {
    if (!ids || !workspace) return SS_ERR_INVALID_ARG;
    st = check_rows(d_out, n, t->dim, d_ld, d_dtype, &d_bytes);
    if (st != SS_OK) return st;
    if (misaligned(ids, ib) || misaligned(workspace, 16)) return SS_ERR_ALIGN;
    if (n > INT32_MAX) return SS_ERR_OVERFLOW;
    if (ws.bytes < 0) return SS_ERR_OVERFLOW;
    if (workspace_bytes < ws.bytes) return SS_ERR_INVALID_ARG;
  }
  const bool in_place = base && base->data == t->data && base->ld == t->ld && base->dtype == t->dtype;
  Ranges ranges;
  ranges.add(t->data, t_bytes, true);
  if (base && !in_place) ranges.add(base->data, b_bytes, false);
  if (n > 0) {
    ranges.add(d_out, d_bytes, false);
    ranges.add(ids, n * ib, false);
    ranges.add(workspace, ws.bytes, true);
  }
  if (ranges.overlap()) return SS_ERR_OVERLAP;
  if (n == 0 && in_place) return SS_OK;
  const int32_t dim = static_cast<int32_t>(t->dim);
  const Rows table = {t->data, t->ld, t->dtype};
  const Rows from = base ? Rows{base->data, base->ld, base->dtype} : Rows{nullptr, 0, SS_FP32};
  const bool tvec = aligned_rows(table) && (!base || aligned_rows(from));
  SortFillArgs sf = {};
  char* w = static_cast<char*>(workspace);
  if (n > 0) {
    int bits = 1;  // of the keys 0 .. vocab
    while ((t->vocab >> bits) != 0) ++bits;
    const int passes = (bits + kDigitBits - 1) / kDigitBits;
    sf.sort = {ids, {reinterpret_cast<uint64_t*>(w + ws.pairs[0]), reinterpret_cast<uint64_t*>(w + ws.pairs[1])},
               reinterpret_cast<Task*>(w + ws.tasks), reinterpret_cast<int32_t*>(w + ws.first_task),
               reinterpret_cast<int32_t*>(w + ws.n_tasks), reinterpret_cast<uint32_t*>(w + ws.arrived), ws.n_arrived,
               t->vocab, static_cast<int32_t>(n), passes, (bits + passes - 1) / passes, idtype == SS_I64};
  }
  sf.fill = {from, table, in_place ? 0 : t->vocab, dim, pieces_of(dim, kRowPiece)};
  auto* sort_fill = tvec ? sort_fill_kernel<true> : sort_fill_kernel<false>;
  st = allow_shared(sort_fill, sizeof(SortShared));
  if (st != SS_OK) return st;
  const int fill_clusters = in_place ? 0 : std::max(1, 2 * sm_count() / kSortBlocks);
  st = launch_rows(sort_fill, 1 + fill_clusters, kSortBlocks, kSortThreads, sizeof(SortShared), sf, stream);
  if (st != SS_OK || n == 0) return st;
  // tasks: one for each token, and one more at most for each run that a token's positions pass into
  const int64_t most = std::min(n, t->vocab + ws.runs);
  const SumArgs a = {sf.sort.pairs[sf.sort.passes & 1 ? 0 : 1], sf.sort.tasks, sf.sort.first_task, sf.sort.n_tasks,
                     sf.sort.arrived, reinterpret_cast<float*>(w + ws.partial), {const_cast<void*>(d_out), d_ld, d_dtype},
                     from, table, pitch_of(dim), static_cast<int32_t>(ws.runs), dim, pieces_of(dim, kSumPiece), scale};
  const bool vec = aligned_rows(a.d_out);
  auto* fn = d_dtype == SS_BF16 ? pick_sum<SS_BF16>(vec, tvec)
                                : (d_dtype == SS_FP16 ? pick_sum<SS_FP16>(vec, tvec) : pick_sum<SS_FP32>(vec, tvec));
  const unsigned grid = grid_for(reinterpret_cast<const void*>(fn), most * a.pieces * 32, kSumThreads);
  return launch(fn, grid, a, stream, kSumThreads);
}

}  // namespace
}  // namespace ss

extern "C" {

ss_status ss_embedding(const ss_table* table, const void* ids, ss_idtype idtype, int64_t n, float scale, void* out,
                       int32_t out_dtype, int64_t out_ld, void* stream) {
  if (!table || n < 0) return SS_ERR_INVALID_ARG;
  if (n == 0) return SS_OK;
  return ss::lookup_impl(table, ids, idtype, n, scale, out, out_dtype, out_ld, stream);
}

int64_t ss_embedding_grad_workspace(int64_t n, int64_t vocab, int64_t dim) {
  if (n < 0 || n > INT32_MAX || vocab < 1 || vocab >= INT32_MAX || dim < 1 || dim > SS_MAX_DIM) return -1;
  return ss::Workspace(n, dim).bytes;
}

ss_status ss_embedding_grad(const void* d_out, int32_t d_dtype, int64_t d_ld, const void* ids, ss_idtype idtype,
                            int64_t n, float scale, const ss_table* base, const ss_table* d_table, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  if (!d_table || n < 0) return SS_ERR_INVALID_ARG;
  return ss::grad_impl(d_out, d_dtype, d_ld, ids, idtype, n, scale, base, d_table, workspace, workspace_bytes, stream);
}

}  // extern "C"
