// ss_logits.cuh -- pieces shared by the operators on rows of logits: element
// access, the running maximum and sum of a softmax in base 2, and the host-side
// checks of their arguments.
//
// Arithmetic. With c = scale * log2(e) and m the running maximum of x, a row's
// exponentials are 2^((x - m) c), one FMA and one hardware ex2 an element: ExpRef
// holds the FMA's constants and the factor that makes good the rounding of m c,
// by which a thread's sums are multiplied once (where m c is 2^24 or more, the
// difference is formed first). Their relative error is 2^-22 and the argument's
// rounding.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "ss_common.cuh"

namespace ss {

constexpr int kRowThreads = 256;
constexpr int kMaxCluster = 8;  // blocks that share a row (the portable cluster size)

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();
constexpr float kFloor = -1e4f;  // 2^kFloor is 0, and 0 * kFloor is 0 where 0 * -inf would be NaN

__device__ __forceinline__ float nan_f() { return __int_as_float(0x7FFFFFFF); }

template <int DT>
struct ElemOf {
  using T = uint16_t;
  static constexpr int kVec = 8;  // elements in 16 bytes
};
template <>
struct ElemOf<SS_FP32> {
  using T = float;
  static constexpr int kVec = 4;
};
template <int DT>
using Elem = typename ElemOf<DT>::T;
template <int DT>
constexpr int kVecOf = ElemOf<DT>::kVec;

// Packed masked elements (-inf).
template <int DT>
constexpr uint32_t kMaskedWord = DT == SS_FP32 ? 0xFF800000u : (DT == SS_BF16 ? 0xFF80FF80u : 0xFC00FC00u);

template <int DT>
__device__ __forceinline__ float to_float(Elem<DT> e) {
  if constexpr (DT == SS_FP32) return e;
  else return widen1<DT>(e);
}

template <int DT>
__device__ __forceinline__ Elem<DT> from_float(float f) {
  if constexpr (DT == SS_FP32) return f;
  else return narrow1<DT>(f);
}

template <int DT>
__device__ __forceinline__ void unpack(const uint4& w, float (&f)[kVecOf<DT>]) {
  if constexpr (DT == SS_FP32) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  } else {
    widen8<DT>(w, f);
  }
}

// Two floats in a register pair: Blackwell's packed fp32 instructions do both at once, which halves the issue slots
// of everything here but the conversions and ex2.
struct Pair {
  unsigned long long v;

  __device__ __forceinline__ static Pair of(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(lo), "f"(hi));
    return p;
  }
  __device__ __forceinline__ static Pair both(float f) { return of(f, f); }
  __device__ __forceinline__ float2 split() const {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
  }
  __device__ __forceinline__ float sum() const {
    const float2 f = split();
    return f.x + f.y;
  }
};
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return p;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}

template <int DT>
constexpr int kPairsOf = kVecOf<DT> / 2;

template <int DT>
__device__ __forceinline__ void unpack_pairs(const uint4& w, Pair (&p)[kPairsOf<DT>]) {
  float f[kVecOf<DT>];
  unpack<DT>(w, f);
#pragma unroll
  for (int i = 0; i < kPairsOf<DT>; ++i) p[i] = Pair::of(f[2 * i], f[2 * i + 1]);
}

template <int DT>
__device__ __forceinline__ uint4 pack_pairs(const Pair (&p)[kPairsOf<DT>]) {
  float f[kVecOf<DT>];
#pragma unroll
  for (int i = 0; i < kPairsOf<DT>; ++i) {
    const float2 v = p[i].split();
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
  if constexpr (DT == SS_FP32)
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  else return narrow8<DT>(f);
}

// The largest of one vector's elements; NaN elements are passed over (a vector of nothing else gives NaN).
template <int DT>
__device__ __forceinline__ float vec_max(const uint4& w) {
  if constexpr (DT == SS_FP32) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  } else {
    using P = std::conditional_t<DT == SS_BF16, __nv_bfloat162, __half2>;
    P a, b, c, d;
    std::memcpy(&a, &w.x, 4);
    std::memcpy(&b, &w.y, 4);
    std::memcpy(&c, &w.z, 4);
    std::memcpy(&d, &w.w, 4);
    const P m = __hmax2(__hmax2(a, b), __hmax2(c, d));
    uint32_t o;
    std::memcpy(&o, &m, 4);
    const float2 f = widen2<DT>(o);
    return fmaxf(f.x, f.y);
  }
}

// 16 bytes of a row: AGAIN when a later pass reads them again (from L2), else read once.
template <bool AGAIN>
__device__ __forceinline__ uint4 load_row(const void* p) {
  if constexpr (AGAIN) return __ldcg(static_cast<const uint4*>(p));
  else return __ldcs(static_cast<const uint4*>(p));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ Pair ex2_pair(Pair a) {
  const float2 f = a.split();
  return Pair::of(ex2(f.x), ex2(f.y));
}

// A row's slice [0, n) of elements at p: `head` elements up to the first 16-byte
// boundary, `nvec` whole vectors, then the rest.
template <int DT>
struct Slice {
  int n, nvec, head;
  __device__ __forceinline__ Slice(const Elem<DT>* p, int64_t len) : n(static_cast<int>(len)) {
    constexpr int V = kVecOf<DT>;
    const int off = static_cast<int>(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u) /
                    static_cast<int>(sizeof(Elem<DT>));
    head = min((V - off) % V, n);
    nvec = (n - head) / V;
  }
  __device__ __forceinline__ int tail() const { return head + nvec * kVecOf<DT>; }
};

// 2^((x - m) c).
//   |m c| < 2^24: k 2^(x c - r), one FMA an element. r = fl(m c) is off by half a unit in its last place, 1/2 at most,
//   which k = 2^(r - m c) makes good.
//   else (far): 2^((x - r) c) with r = m and k = 1. The rounding of m c would be whole powers of two there and, from
//   2^31 on, more than k can hold; x - m is exact where the exponential is not 0. Such a reference is rare (a mask's
//   finite fill, a temperature near 0).
// Before the first unmasked element (m = -inf) r = 0, and all exponentials are 0.
constexpr float kFarFrom = 16777216.0f;

struct ExpArg {
  float c, r;
  bool far;

  __device__ __forceinline__ float arg(float x) const { return far ? (x - r) * c : fmaf(x, c, -r); }
  __device__ __forceinline__ float exp(float x) const { return ex2(arg(x)); }  // without k
  template <bool FAR>
  __device__ __forceinline__ Pair arg(Pair x) const {
    if constexpr (FAR) return mul2(add2(x, Pair::both(-r)), Pair::both(c));
    else return fma2(x, Pair::both(c), Pair::both(-r));
  }
};
struct ExpRef : ExpArg {
  float k, shift;  // k = 2^shift

  __device__ __forceinline__ ExpRef(float m, float scale2) : ExpArg{scale2, m * scale2, false}, k(1.0f), shift(0.0f) {
    if (fabsf(r) < kFarFrom) {
      shift = fmaf(-m, scale2, r);
      k = ex2(shift);
    } else if (m == -kInf) {
      r = 0.0f;
    } else {
      r = m;
      far = true;
    }
  }
};

// (x - m) / 2, which does not overflow, and (x - m) scale + add from it.
__device__ __forceinline__ float half_gap(float x, float m) { return fmaf(0.5f, x, -0.5f * m); }
__device__ __forceinline__ float scaled_gap(float x, float m, float scale, float add = 0.0f) {
  return fmaf(half_gap(x, m), 2.0f * scale, add);
}

// m = max x (-inf before the first unmasked element), s = sum 2^d and
// t = sum 2^d d over d = (x - m) c.
struct RowSum {
  float m, s, t;

  __device__ __forceinline__ static RowSum none() { return {-kInf, 0.0f, 0.0f}; }
  // Moves the maximum up to `to` (> m).
  __device__ __forceinline__ void move(float to, float c) {
    if (s != 0.0f) {  // NaN sums move too
      const float d = fmaxf(scaled_gap(m, to, c), kFloor), f = ex2(d);
      t = f * fmaf(s, d, t);
      s *= f;
    }
    m = to;
  }
  // Two small systematic errors of s, mended to first order. c is the scale's product with log2(e) rounded to 24 bits,
  // which is a slightly different temperature: eps ln 2 t (eps: its relative error, 2^-25 at most). And ex2.approx
  // falls short by 9e-8 on average, but for the maximum's own 2^0 (sums of 9291 to 128256 terms against float64, over
  // four spreads and three scales: 4e-8 to 1.7e-7; mended, 9e-8 at most on average over rows); a loss of a few
  // hundredths would lose its sixth digit to that. The price: sums whose terms are exactly 2^0, of rows without any
  // spread, come out up to a unit in their last place too large (6e-8 to 1.1e-7).
  __device__ __forceinline__ void mend(float eps) { s += fmaf(eps * kLn2, t, 9e-8f * fmaxf(s - 1.0f, 0.0f)); }
};

// Order of logits as unsigned integers (-0 counts as +0; NaN rows do not come here).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// Larger logit first, equal logits by ascending id; 0 is below every element.
__device__ __forceinline__ uint64_t order_pair(float x, int64_t id) {
  return (static_cast<uint64_t>(order_key(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}

// A thread's running sums around a reference that stays where it is while the elements are at most 2^SLACK times its
// exponential: the reference is the first batch's maximum for nearly all threads, and `top` the maximum.
template <int SLACK>
struct Running {
  float m;      // the reference
  float s, t;   // sums of 2^a and 2^a a, a = reference().arg(x): those around m when m moves and at the end
  float top;    // max x
  float limit;  // elements above it move the reference
  float r;      // a = x c - r; NaN where m is far: a loop that looks at its sums for NaN, as masked elements give it,
                // has this for nothing (a look of its own: 2048 x 128256 with 64 alternatives 108.5 us against 104.5)

  __device__ __forceinline__ Running(RowSum first, float c) : top(first.m) { put(first, c); }
  __device__ __forceinline__ void see(float to, float c) {
    top = fmaxf(top, to);
    if (to > limit) {
      RowSum a = around(c);
      a.move(to, c);
      put(a, c);
    }
  }
  __device__ __forceinline__ ExpArg reference(float c) const { return {c, r == r ? r : m, !(r == r)}; }
  // The sums around the maximum.
  __device__ __forceinline__ RowSum done(float c) const {
    RowSum a = around(c);
    if (top > m) a.move(top, c);
    return a;
  }

 private:
  __device__ __forceinline__ RowSum around(float c) const {
    const ExpRef e(m, c);
    return {m, s * e.k, fmaf(e.shift, s, t) * e.k};
  }
  __device__ __forceinline__ void put(const RowSum& a, float c) {
    const ExpRef e(a.m, c);
    const float back = ex2(-e.shift);
    m = a.m;
    r = e.far ? nan_f() : e.r;
    s = a.s * back;
    t = fmaf(-e.shift, s, a.t * back);
    limit = m == -kInf ? m : m + SLACK / c;  // SLACK / c may be infinite
  }
};

// One element as a sum: 2^0 (0 when masked, NaN for NaN and +inf, with any maximum that is a number).
__device__ __forceinline__ RowSum one_element(float x) {
  RowSum a = RowSum::none();
  if (x == -kInf) return a;
  if (x <= 3.402823466e38f) {
    a.m = x;
    a.s = 1.0f;
  } else {
    a.s = nan_f();
  }
  return a;
}

// Merged over the `width` (a power of two) lanes of each aligned group, the groups being copies of one another;
// the same in every lane. One rescale a lane: first the maximum, then plain sums.
__device__ __forceinline__ RowSum merge_lanes(RowSum a, float c, int width = 32) {
  const float top = key_value(__reduce_max_sync(0xFFFFFFFFu, order_key(a.m)));
  if (top > a.m) a.move(top, c);
  for (int off = width >> 1; off > 0; off >>= 1) {
    a.s += __shfl_xor_sync(0xFFFFFFFFu, a.s, off);
    a.t += __shfl_xor_sync(0xFFFFFFFFu, a.t, off);
  }
  return a;
}

constexpr int kRowWarps = kRowThreads / 32;

// Merged over the block, the same in every thread. `red`: a slot per warp, used by one call only.
template <int WARPS = kRowWarps>
__device__ __forceinline__ RowSum block_merge(RowSum a, float c, RowSum* red) {
  a = merge_lanes(a, c);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  return merge_lanes(red[threadIdx.x % WARPS], c, WARPS);
}

__device__ __forceinline__ int64_t load_id(const void* p, int64_t i, bool wide) {
  return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}
__device__ __forceinline__ void store_id(void* p, int64_t i, int64_t v, bool wide) {
  if (wide) static_cast<int64_t*>(p)[i] = v;
  else static_cast<int32_t*>(p)[i] = static_cast<int32_t>(v);
}

// Hardware barrier ID (1 to 15) of the block, for THREADS threads of which some only announce themselves.
template <int ID, int THREADS>
__device__ __forceinline__ void barrier_sync() {
  asm volatile("barrier.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}
template <int ID, int THREADS>
__device__ __forceinline__ void barrier_arrive() {
  asm volatile("barrier.arrive %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

// ------------------------------------------------------------------ rows shared by a cluster of blocks
//
// With few rows a row is shared by the blocks of a cluster, which exchange their
// parts through distributed shared memory: one launch, no workspace. The arrive
// of start() and the wait of started() make sure that every block runs before
// another one writes into its shared memory; the waits are the hardware's
// cluster barrier, which every block of the cluster reaches.

struct Cluster {
  unsigned size, rank;
  __device__ __forceinline__ static Cluster start() {
    Cluster c;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(c.size));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(c.rank));
    if (c.size > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    return c;
  }
  __device__ __forceinline__ void started() const {
    if (size > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  }
  // Barrier over all threads of the cluster; shared memory written before it, in any block, is seen after it.
  __device__ __forceinline__ void sync() const {
    if (size > 1) {
      arrive();
      wait();
    } else {
      __syncthreads();
    }
  }
  // The two halves of sync() for a cluster of more than one block.
  __device__ __forceinline__ void arrive() const { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
  __device__ __forceinline__ void wait() const { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
  // `p` (in this block's shared memory) at the same place in block r's.
  template <class T>
  __device__ __forceinline__ T* at(T* p, unsigned r) const {
    return size > 1 ? cooperative_groups::this_cluster().map_shared_rank(p, r) : p;
  }
};

// ------------------------------------------------------------------ a block's part of a row
//
// Of a row shared by `size` blocks (a power of two) of T threads, its whole 16-byte vector i
// belongs to thread i mod T of block (i / T) mod size: a warp reads 512
// consecutive bytes, and neighbouring ids are spread over threads and blocks.
// The fewer than 8 elements before the first boundary and after the last vector
// are one each of block 0's first 16 threads.

constexpr int kBatch = 4;  // vectors that a thread has in flight

// One vector's elements to d: as 16 bytes when d lies so, else one by one.
template <int DT>
__device__ __forceinline__ void store_vector(void* d, const Pair (&p)[kPairsOf<DT>], bool aligned) {
  const uint4 v = pack_pairs<DT>(p);
  if (aligned) {
    __stcs(static_cast<uint4*>(d), v);
  } else {
    Elem<DT>* e = static_cast<Elem<DT>*>(d);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == SS_FP32) {
        e[i] = __uint_as_float(w[i]);
      } else {
        e[2 * i] = static_cast<uint16_t>(w[i]);
        e[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
      }
    }
  }
}

// Zeros in block `rank`'s part, of `size`, of a gradient row.
template <int DT>
__device__ __forceinline__ void zero_part(Elem<DT>* d, int64_t n, unsigned rank, unsigned size) {
  const Slice<DT> sl(d, n);
  if (rank == 0) {
    for (int64_t i = threadIdx.x; i < sl.head; i += kRowThreads) d[i] = from_float<DT>(0.0f);
    for (int64_t i = sl.tail() + threadIdx.x; i < sl.n; i += kRowThreads) d[i] = from_float<DT>(0.0f);
  }
  uint4* w = reinterpret_cast<uint4*>(d + sl.head);
  for (int i = rank * kRowThreads + threadIdx.x; i < sl.nvec; i += size * kRowThreads)
    __stcs(w + i, make_uint4(0u, 0u, 0u, 0u));
}

// Asks the L2 for the first `bytes` bytes of block `rank`'s of `size` equal runs of a row (as many of its whole
// vectors as that is).
template <int DT>
__device__ __forceinline__ void prefetch_row(const Elem<DT>* row, int64_t vocab, int bytes, int rank = 0,
                                             int size = 1) {
  const Slice<DT> sl(row, vocab);
  const int64_t vecs = sl.nvec, first = vecs * rank / size, last = vecs * (rank + 1) / size;
  const char* p = reinterpret_cast<const char*>(row + sl.head) + first * 16;
  const int64_t n = min(static_cast<int64_t>(bytes), (last - first) * 16);
  constexpr int64_t kPiece = 16384;
  for (int64_t at = 0; at < n; at += kPiece) prefetch_l2(p + at, static_cast<uint32_t>(min(n - at, kPiece)));
}

// Asks the L2 for the line at p.
__device__ __forceinline__ void prefetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ int log2_of(unsigned power) { return 31 - __clz(static_cast<int>(power)); }

template <int DT, int T = kRowThreads>
struct RowPart {
  static constexpr int V = kVecOf<DT>;
  const Elem<DT>* x;
  Slice<DT> sl;
  int rank, blocks, log2_blocks;
  int first;  // this thread's vectors: first, first + step(), ... < nvec
  int whole;  // vectors that every thread of every block has
  int edge;   // this thread's element outside the vectors, or -1

  __device__ __forceinline__ RowPart(const Elem<DT>* row, int64_t vocab, unsigned rank_, unsigned size_)
      : x(row),
        sl(row, vocab),
        rank(static_cast<int>(rank_)),
        blocks(static_cast<int>(size_)),
        log2_blocks(log2_of(size_)) {
    const int t = threadIdx.x;
    first = rank * T + t;
    whole = sl.nvec / T >> log2_blocks;
    edge = -1;
    if (rank == 0) {
      const int after = t - 8;
      if (t < sl.head) edge = t;
      else if (after >= 0 && after < sl.n - sl.tail()) edge = sl.tail() + after;
    }
  }
  __device__ __forceinline__ int step() const { return blocks * T; }
  __device__ __forceinline__ int64_t step_bytes() const { return static_cast<int64_t>(step()) * 16; }
  // Vectors of the thread that has most.
  __device__ __forceinline__ int vectors() const { return whole + (whole * step() < sl.nvec ? 1 : 0); }
  // Whether this thread has a vector number j.
  __device__ __forceinline__ bool more(int j) const {
    return j < whole || (j == whole && first + whole * step() < sl.nvec);
  }
  // The thread's first vector in x, and in an array that lies as x does or not.
  __device__ __forceinline__ const char* at() const {
    return reinterpret_cast<const char*>(x + sl.head) + static_cast<int64_t>(first) * 16;
  }
  __device__ __forceinline__ char* at(Elem<DT>* d) const {
    return reinterpret_cast<char*>(d + sl.head) + static_cast<int64_t>(first) * 16;
  }
  // Whether element `id` is this block's; then `j` and `thread` say which of its vectors (j = -1: an edge).
  __device__ __forceinline__ bool owns(int id, int* thread, int* j) const {
    const int o = id - sl.head;
    if (o < 0 || o >= sl.nvec * V) {
      *j = -1;
      *thread = o < 0 ? id : id - sl.tail() + 8;
      return rank == 0;
    }
    const int i = o / V, q = i / T;
    *thread = i % T;
    *j = q >> log2_blocks;
    return (q & (blocks - 1)) == rank;
  }
  // The thread's vectors number j0 .. j0 + kBatch - 1 (those past its last one are left as they are).
  __device__ __forceinline__ void load(int j0, uint4 (&w)[kBatch]) const {
    const char* p = at() + j0 * step_bytes();
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (more(j0 + u)) w[u] = __ldcs(reinterpret_cast<const uint4*>(p + u * step_bytes()));
  }
  // d = f(x) over the part, in one pass with the next batch's loads in flight. `w` holds the first batch and
  // `edge_x` the thread's edge element; d may be x. `aligned`: d's vectors lie as x's do.
  template <class F>
  __device__ __forceinline__ void map(uint4 (&w)[kBatch], Elem<DT>* d, bool aligned, float edge_x, const F& f) const {
    if (edge >= 0) d[edge] = from_float<DT>(f(Pair::both(edge_x)).split().x);
    auto put = [&](const uint4& v, char* o) {
      Pair p[kPairsOf<DT>];
      unpack_pairs<DT>(v, p);
#pragma unroll
      for (int q = 0; q < kPairsOf<DT>; ++q) p[q] = f(p[q]);
      store_vector<DT>(o, p, aligned);
    };
    const int64_t sb = step_bytes();
    const char* src = at() + kBatch * sb;
    char* dst = at(d);
    int j = 0;
#pragma unroll 1
    for (; j + 2 * kBatch <= whole; j += kBatch, src += kBatch * sb, dst += kBatch * sb) {
      uint4 next[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) next[u] = __ldcs(reinterpret_cast<const uint4*>(src + u * sb));
#pragma unroll
      for (int u = 0; u < kBatch; ++u) put(w[u], dst + u * sb);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) w[u] = next[u];
    }
#pragma unroll 1
    for (; more(j); j += kBatch, dst += kBatch * sb) {
      uint4 next[kBatch];
      load(j + kBatch, next);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (more(j + u)) put(w[u], dst + u * sb);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) w[u] = next[u];
    }
  }
};

// ------------------------------------------------------------------ host checks

// Byte ranges of one call's arrays; no allocation, so nothing can throw.
struct Ranges {
  Range r[16];
  int n = 0;
  void add(const void* p, int64_t bytes, bool out) {
    if (p && bytes > 0) r[n++] = rng(p, bytes, out);
  }
  bool overlap() const {
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j)
        if ((r[i].out || r[j].out) && r[i].lo < r[j].hi && r[j].lo < r[i].hi) return true;
    return false;
  }
};

inline int64_t dtype_bytes(int32_t dt) { return dt == SS_FP32 ? 4 : 2; }
inline bool is_float_dtype(int32_t dt) { return dt == SS_BF16 || dt == SS_FP16 || dt == SS_FP32; }
inline bool misaligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Bytes from the first to the last element of rows x width elements of row stride ld.
inline bool span_bytes(int64_t rows, int64_t width, int64_t ld, int64_t es, int64_t* out) {
  const __int128 v = (static_cast<__int128>(rows - 1) * ld + width) * es;
  if (v > INT64_MAX) return false;
  *out = static_cast<int64_t>(v);
  return true;
}

// The rules every operator has for its logits (rows > 0 is checked by the caller first).
inline ss_status check_logits(const ss_logits* x, int64_t* bytes) {
  if (!x->data || x->vocab < 1 || x->vocab > INT32_MAX || x->ld < x->vocab) return SS_ERR_INVALID_ARG;
  if (!(x->scale > 0.0f) || !(x->scale <= 1e20f)) return SS_ERR_INVALID_ARG;
  if (!is_float_dtype(x->dtype)) return SS_ERR_DTYPE;
  if (misaligned(x->data, dtype_bytes(x->dtype))) return SS_ERR_ALIGN;
  if (!span_bytes(x->rows, x->vocab, x->ld, dtype_bytes(x->dtype), bytes)) return SS_ERR_OVERFLOW;
  return SS_OK;
}

// The gradient array: x's dtype; either x itself or apart from it (`ranges` gets it as an output, and x
// as an input unless they are the same array).
inline ss_status check_grad_out(const ss_logits* x, int64_t x_bytes, const void* d, int64_t d_ld, Ranges* ranges) {
  if (d_ld < x->vocab) return SS_ERR_INVALID_ARG;
  if (misaligned(d, dtype_bytes(x->dtype))) return SS_ERR_ALIGN;
  int64_t bytes = 0;
  if (!span_bytes(x->rows, x->vocab, d_ld, dtype_bytes(x->dtype), &bytes)) return SS_ERR_OVERFLOW;
  ranges->add(d, bytes, true);
  if (d != x->data || d_ld != x->ld) ranges->add(x->data, x_bytes, false);
  return SS_OK;
}

// Blocks that share a row where nothing is exchanged between them (a power of two): parts of at most `vectors` vectors
// a thread.
inline int split_for(int64_t nvec, int vectors) {
  int64_t split = 1;
  while (split * vectors * kRowThreads < nvec) split *= 2;
  return static_cast<int>(split);
}

// Launches `clusters` clusters of `cluster` blocks (a plain launch for 1).
template <typename Args>
ss_status launch_rows(void (*fn)(Args), int64_t clusters, int cluster, int threads, size_t smem, const Args& args,
                      void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args);
  return e == cudaSuccess ? SS_OK : cuda_fail(e);
}

// scale * log2(e) as c (1 + eps), c in fp32.
struct Scale2 {
  float c, eps;
  explicit Scale2(float scale) {
    const double exact = static_cast<double>(scale) * 1.4426950408889634;
    c = static_cast<float>(exact);
    eps = static_cast<float>((exact - static_cast<double>(c)) / static_cast<double>(c));
  }
};

// True when every row of the gradient starts at its logits row's 16-byte phase, so both take the same vectors.
inline bool same_phase(const ss_logits* x, const void* d, int64_t d_ld) {
  const int64_t es = dtype_bytes(x->dtype);
  return ((reinterpret_cast<uintptr_t>(x->data) ^ reinterpret_cast<uintptr_t>(d)) & 15u) == 0 &&
         (x->rows == 1 || ((x->ld - d_ld) * es) % 16 == 0);
}

}  // namespace ss
