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
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); task < tasks;
       task += warps) {
    const int64_t pos = task / a.pieces;
    const int from = static_cast<int>(task - pos * a.pieces) * kRowPiece;
    const int64_t id = load_id(a.ids, pos, a.wide);
    char* out = a.out.row(pos);
    const bool there = id >= 0 && id < a.vocab;
    const char* row = a.table.row(there ? id : 0);
    const float none = id < 0 ? 0.0f : nan_f();
    float f[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = from + (u * 32 + lane) * 8;
      if (there && e < a.dim) load8<DT, VEC>(row, e, a.dim, f[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = from + (u * 32 + lane) * 8;
      if (e >= a.dim) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[u][j] = there ? f[u][j] * a.scale : none;
      store8<OT, VEC>(out, e, a.dim, f[u]);
    }
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

struct SortArgs {
  const void* ids;
  uint64_t* pairs[2];  // token << 32 | position; the sorted ones are in pairs[passes & 1 ? 0 : 1]
  int64_t vocab;
  int32_t n, passes, bits;  // bits of a digit
  bool wide;
};

struct SortShared {
  uint32_t count[kSortWarps][kDigits];  // of a warp's digits; then the next place of each
  uint32_t total[kDigits];              // of the block's digits
  uint32_t base[kDigits];
  uint32_t warp_sum[kSortWarps];
};

__device__ void sort_positions(const SortArgs& a, const Cluster& cl, SortShared& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.n;
  // this warp's run
  const int64_t each = (static_cast<int64_t>(n) + kSortBlocks * kSortWarps * 32 - 1) / (kSortBlocks * kSortWarps * 32) * 32;
  const int64_t first = (static_cast<int64_t>(cl.rank) * kSortWarps + warp) * each;
  const int64_t last = min(first + each, static_cast<int64_t>(n));
  const uint32_t none = static_cast<uint32_t>(a.vocab);
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
    sort_positions(a.sort, cl, *reinterpret_cast<SortShared*>(shared));
  } else {
    const int64_t warp = static_cast<int64_t>(blockIdx.x - kSortBlocks) * kSortWarps + (threadIdx.x >> 5);
    fill_rows<VEC>(a.fill, warp, static_cast<int64_t>(gridDim.x - kSortBlocks) * kSortWarps);
  }
}

// ------------------------------------------------------------------ the sums
//
// A block takes kChunk consecutive sorted positions and 1024 columns: a thread adds
// its eight columns of one position after another and writes them out where the
// token changes. A token whose positions reach into other chunks leaves its sum of
// each chunk in the workspace; the join adds them in the chunks' order.

constexpr int kChunk = 32;
constexpr int kSumThreads = 128;
constexpr int kSumColumns = kSumThreads * 8;
constexpr int kInFlight = 8;  // rows that a thread has in flight

struct SumArgs {
  const uint64_t* pairs;
  Rows d_out, base, table;
  float* partial;  // [chunks][2][pitch]: of the token that began before the chunk, of the one that goes on behind it
  int64_t pitch, vocab;
  int32_t n, dim;
  float scale;
};

__device__ __forceinline__ uint32_t token_of(uint64_t pair) { return static_cast<uint32_t>(pair >> 32); }

// A token's row from its sum.
template <bool VEC>
__device__ __forceinline__ void finish_row(const SumArgs& a, uint32_t token, int e, const float (&sum)[8]) {
  float f[8] = {};
  if (a.base.data) load8<VEC>(a.base.dtype, a.base.row(token), e, a.dim, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = fmaf(sum[j], a.scale, f[j]);
  store8<VEC>(a.table.dtype, a.table.row(token), e, a.dim, f);
}

template <int DT, bool VEC, bool TVEC>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const __grid_constant__ SumArgs a) {
  __shared__ uint64_t pairs[kChunk + 2];
  pdl_wait();
  pdl_trigger();
  const int64_t chunk = blockIdx.x, first = chunk * kChunk;
  const int cnt = static_cast<int>(min(static_cast<int64_t>(kChunk), a.n - first));
  const uint32_t none = static_cast<uint32_t>(a.vocab);
  for (int i = threadIdx.x; i < cnt + 2; i += kSumThreads) {
    const int64_t at = first + i - 1;
    pairs[i] = at < 0 || at >= a.n ? ~0ull : a.pairs[at];
  }
  __syncthreads();
  const int e = (blockIdx.y * kSumThreads + threadIdx.x) * 8;
  if (e >= a.dim) return;
  float sum[8] = {};
  bool began = token_of(pairs[0]) != token_of(pairs[1]);  // in this chunk
  for (int i0 = 0; i0 < cnt; i0 += kInFlight) {
    float f[kInFlight][8];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (i0 + u < cnt && token_of(pairs[i0 + u + 1]) < none)
        load8<DT, VEC>(a.d_out.row(static_cast<uint32_t>(pairs[i0 + u + 1])), e, a.dim, f[u]);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int i = i0 + u;
      if (i >= cnt) break;
      const uint32_t token = token_of(pairs[i + 1]);
      if (token >= none) return;  // and all behind it
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[u][j];
      const bool ends = token_of(pairs[i + 2]) != token;
      if (ends && began) {
        finish_row<TVEC>(a, token, e, sum);
      } else if (ends || i + 1 == cnt) {
        float* p = a.partial + (2 * chunk + (began ? 1 : 0)) * a.pitch;
        store8<SS_FP32, true>(p, e, static_cast<int>(a.pitch), sum);
      }
      if (ends) {
        began = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
      }
    }
  }
}

// The tokens that begin in a chunk and go on behind it.
template <bool TVEC>
__global__ void __launch_bounds__(kSumThreads) join_kernel(const __grid_constant__ SumArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t chunk = blockIdx.x, end = (chunk + 1) * kChunk;
  if (end >= a.n) return;
  const uint32_t token = token_of(a.pairs[end - 1]);
  if (token >= static_cast<uint32_t>(a.vocab) || token_of(a.pairs[end]) != token) return;
  if (chunk > 0 && token_of(a.pairs[end - kChunk - 1]) == token) return;  // it began before
  const int e = (blockIdx.y * kSumThreads + threadIdx.x) * 8;
  if (e >= a.dim) return;
  float sum[8];
  load8<SS_FP32, true>(a.partial + (2 * chunk + 1) * a.pitch, e, static_cast<int>(a.pitch), sum);
  for (int64_t c = chunk + 1;; ++c) {
    float f[8];
    load8<SS_FP32, true>(a.partial + 2 * c * a.pitch, e, static_cast<int>(a.pitch), f);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += f[j];
    const int64_t next = (c + 1) * kChunk;
    if (next >= a.n || token_of(a.pairs[next]) != token) break;
  }
  finish_row<TVEC>(a, token, e, sum);
}

// ------------------------------------------------------------------ host

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }
int64_t pitch_of(int64_t dim) { return (dim + 7) / 8 * 8; }

// Bytes of the workspace, or -1 where they do not fit in int64.
int64_t workspace_bytes_of(int64_t n, int64_t dim) {
  const __int128 v = static_cast<__int128>(n) * 16 + static_cast<__int128>(chunks_of(n)) * 2 * pitch_of(dim) * 4 + 16;
  return v > INT64_MAX ? -1 : static_cast<int64_t>(v);
}

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

int pieces_of(int64_t dim) { return static_cast<int>((dim + kRowPiece - 1) / kRowPiece); }

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
                        static_cast<int32_t>(t->dim), pieces_of(t->dim), scale, idtype == SS_I64};
  auto* fn = aligned_rows(a.table) && aligned_rows(a.out) ? pick_lookup<true>(t->dtype, out_dtype)
                                                          : pick_lookup<false>(t->dtype, out_dtype);
  const int64_t blocks = (n * a.pieces + kThreads / 32 - 1) / (kThreads / 32);
  return launch(fn, static_cast<unsigned>(std::min<int64_t>(blocks, INT32_MAX)), a, stream);
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
  if (n > 0) {
    if (!ids || !workspace) return SS_ERR_INVALID_ARG;
    st = check_rows(d_out, n, t->dim, d_ld, d_dtype, &d_bytes);
    if (st != SS_OK) return st;
    if (misaligned(ids, ib) || misaligned(workspace, 16)) return SS_ERR_ALIGN;
    if (n > INT32_MAX) return SS_ERR_OVERFLOW;
    const int64_t need = workspace_bytes_of(n, t->dim);
    if (need < 0) return SS_ERR_OVERFLOW;
    if (workspace_bytes < need) return SS_ERR_INVALID_ARG;
  }
  const bool in_place = base && base->data == t->data && base->ld == t->ld && base->dtype == t->dtype;
  Ranges ranges;
  ranges.add(t->data, t_bytes, true);
  if (base && !in_place) ranges.add(base->data, b_bytes, false);
  if (n > 0) {
    ranges.add(d_out, d_bytes, false);
    ranges.add(ids, n * ib, false);
    ranges.add(workspace, workspace_bytes_of(n, t->dim), true);
  }
  if (ranges.overlap()) return SS_ERR_OVERLAP;
  if (n == 0 && in_place) return SS_OK;
  const int32_t dim = static_cast<int32_t>(t->dim);
  const Rows table = {t->data, t->ld, t->dtype};
  const Rows from = base ? Rows{base->data, base->ld, base->dtype} : Rows{nullptr, 0, SS_FP32};
  const bool tvec = aligned_rows(table) && (!base || aligned_rows(from));
  SortFillArgs sf = {};
  uint64_t* pairs = static_cast<uint64_t*>(workspace);
  if (n > 0) {
    int bits = 1;  // of the keys 0 .. vocab
    while ((t->vocab >> bits) != 0) ++bits;
    const int passes = (bits + kDigitBits - 1) / kDigitBits;
    sf.sort = {ids, {pairs, pairs + n}, t->vocab, static_cast<int32_t>(n), passes, (bits + passes - 1) / passes,
               idtype == SS_I64};
  }
  sf.fill = {from, table, in_place ? 0 : t->vocab, dim, pieces_of(dim)};
  auto* sort_fill = tvec ? sort_fill_kernel<true> : sort_fill_kernel<false>;
  st = allow_shared(sort_fill, sizeof(SortShared));
  if (st != SS_OK) return st;
  const int fill_clusters = in_place ? 0 : std::max(1, 2 * sm_count() / kSortBlocks);
  st = launch_rows(sort_fill, 1 + fill_clusters, kSortBlocks, kSortThreads, sizeof(SortShared), sf, stream);
  if (st != SS_OK || n == 0) return st;
  const SumArgs a = {sf.sort.pairs[sf.sort.passes & 1 ? 0 : 1], {const_cast<void*>(d_out), d_ld, d_dtype}, from, table,
                     reinterpret_cast<float*>(pairs + 2 * n), pitch_of(dim), t->vocab, static_cast<int32_t>(n), dim,
                     scale};
  const bool vec = aligned_rows(a.d_out);
  auto* fn = d_dtype == SS_BF16 ? pick_sum<SS_BF16>(vec, tvec)
                                : (d_dtype == SS_FP16 ? pick_sum<SS_FP16>(vec, tvec) : pick_sum<SS_FP32>(vec, tvec));
  const dim3 grid(static_cast<unsigned>(chunks_of(n)), static_cast<unsigned>((dim + kSumColumns - 1) / kSumColumns));
  st = launch_dependent(fn, grid, dim3(kSumThreads), 0, stream, a);
  if (st != SS_OK) return st;
  return launch_dependent(tvec ? join_kernel<true> : join_kernel<false>, grid, dim3(kSumThreads), 0, stream, a);
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
  return ss::workspace_bytes_of(n, dim);
}

ss_status ss_embedding_grad(const void* d_out, int32_t d_dtype, int64_t d_ld, const void* ids, ss_idtype idtype,
                            int64_t n, float scale, const ss_table* base, const ss_table* d_table, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  if (!d_table || n < 0) return SS_ERR_INVALID_ARG;
  return ss::grad_impl(d_out, d_dtype, d_ld, ids, idtype, n, scale, base, d_table, workspace, workspace_bytes, stream);
}

}  // extern "C"
