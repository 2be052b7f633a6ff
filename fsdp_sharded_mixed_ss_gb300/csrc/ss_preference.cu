// ss_preference.cu -- the loss of pairs of sequences (chosen, rejected) from their
// tokens' log probabilities, and its gradient (ss_preference_loss).
#include "ss_logits.cuh"

namespace ss {
namespace {

constexpr int kMaxThreads = 512;

struct PreferenceArgs {
  const float* logprob;
  const float* ref;
  const float* weight;
  const float* pair_weight;
  const void* offsets;
  float* loss;
  float2* reward;
  float* d;
  int64_t rows, pairs;
  float beta, margin, smooth;
  int32_t kind;
  bool wide, halves, average;
};

// A sequence's weighted sum, as a pair (thousands of log ratios cancel against those of the other answer), and the
// weights' sum.
struct SeqSum {
  dd s, w;

  // lo is NaN once hi is infinite or NaN, and then not used
  __device__ __forceinline__ static void add(dd& a, dd b) {
    const dd t = two_sum(a.hi, b.hi);
    a = {t.hi, t.lo + (a.lo + b.lo)};
  }
  __device__ __forceinline__ void add(const SeqSum& o) {
    add(s, o.s);
    add(w, o.w);
  }
  __device__ __forceinline__ SeqSum from_lane(int off) const {
    return {{__shfl_xor_sync(0xFFFFFFFFu, s.hi, off), __shfl_xor_sync(0xFFFFFFFFu, s.lo, off)},
            {__shfl_xor_sync(0xFFFFFFFFu, w.hi, off), __shfl_xor_sync(0xFFFFFFFFu, w.lo, off)}};
  }
  __device__ __forceinline__ static double value(dd a) {
    return finite(a.hi) ? static_cast<double>(a.hi) + static_cast<double>(a.lo) : static_cast<double>(a.hi);
  }
};

struct Span {
  int64_t lo, hi;
};

constexpr int kTokens = 4;  // of a thread in flight

// f(i, step) over block `rank`'s of `size` parts of a sequence: the thread's tokens i, i + step, ... below q.hi, kTokens
// of them a call.
template <class F>
__device__ __forceinline__ void over_tokens(const Span& q, unsigned rank, unsigned size, const F& f) {
  const int64_t step = static_cast<int64_t>(size) * blockDim.x;
  for (int64_t i = q.lo + static_cast<int64_t>(rank) * blockDim.x + threadIdx.x; i < q.hi; i += kTokens * step) f(i, step);
}

// A block of `blockDim.x` threads a pair, or the blocks of a cluster: the two sums, the pair's loss, and its derivative
// to every token.
__global__ void __launch_bounds__(kMaxThreads) preference_kernel(const __grid_constant__ PreferenceArgs a) {
  __shared__ SeqSum red[2][kMaxThreads / 32];
  __shared__ SeqSum parts[2][kMaxCluster];
  __shared__ float slope[2];
  const Cluster cl = Cluster::start();
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
  const int64_t pair = blockIdx.x / cl.size;
  const int64_t seq[2] = {a.halves ? pair : 2 * pair, a.halves ? a.pairs + pair : 2 * pair + 1};
  Span at[2];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    at[k] = {load_id(a.offsets, seq[k], a.wide), load_id(a.offsets, seq[k] + 1, a.wide)};
    bad = bad || at[k].lo < 0 || at[k].hi < at[k].lo || at[k].hi > a.rows;
  }
  const float wp = a.pair_weight ? a.pair_weight[pair] : 1.0f;
  cl.started();
  if (bad || wp == 0.0f) {  // the same in all blocks of the cluster
    const float v = bad && wp != 0.0f ? nan_f() : 0.0f;
    if (cl.rank == 0 && tid == 0) {
      if (a.loss) a.loss[pair] = v;
      if (a.reward) a.reward[pair] = make_float2(v, v);
    }
    if (!bad && a.d) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        over_tokens(at[k], cl.rank, cl.size, [&](int64_t i, int64_t step) {
#pragma unroll
          for (int u = 0; u < kTokens; ++u)
            if (i + u * step < at[k].hi) a.d[i + u * step] = 0.0f;
        });
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    SeqSum sum = {{0.0f, 0.0f}, {0.0f, 0.0f}};
    over_tokens(at[k], cl.rank, cl.size, [&](int64_t i, int64_t step) {
      float lp[kTokens], ref[kTokens], w[kTokens];
#pragma unroll
      for (int u = 0; u < kTokens; ++u) {
        const bool there = i + u * step < at[k].hi;
        lp[u] = there ? a.logprob[i + u * step] : 0.0f;
        ref[u] = there && a.ref ? a.ref[i + u * step] : 0.0f;
        w[u] = !there ? 0.0f : (a.weight ? a.weight[i + u * step] : 1.0f);
      }
#pragma unroll
      for (int u = 0; u < kTokens; ++u) {
        if (w[u] == 0.0f) continue;  // whatever the token's log probability
        SeqSum::add(sum.s, {w[u] * (lp[u] - ref[u]), 0.0f});
        SeqSum::add(sum.w, {w[u], 0.0f});
      }
    });
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum.add(sum.from_lane(off));
    if (lane == 0) red[k][tid >> 5] = sum;
  }
  __syncthreads();
  if (tid < 2) {  // one thread a sequence
    SeqSum sum = red[tid][0];
    for (int i = 1; i < warps; ++i) sum.add(red[tid][i]);
    for (unsigned r = 0; r < cl.size; ++r) cl.at(&parts[tid][0], r)[cl.rank] = sum;
  }
  cl.sync();
  if (tid == 0) {
    double score[2], per[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      SeqSum sum = parts[k][0];
      for (unsigned r = 1; r < cl.size; ++r) sum.add(parts[k][r]);
      const double w = SeqSum::value(sum.w);
      per[k] = !a.average ? 1.0 : (w == 0.0 ? 0.0 : 1.0 / w);
      score[k] = SeqSum::value(sum.s) * per[k];
    }
    const float h = static_cast<float>(static_cast<double>(a.beta) * (score[0] - score[1]) - a.margin);
    float loss, d_h;
    if (a.kind == SS_PREF_SIGMOID) {
      const float e = expf(-fabsf(h)), soft = log1pf(e);
      loss = (1.0f - a.smooth) * (fmaxf(-h, 0.0f) + soft);
      if (a.smooth != 0.0f) loss += a.smooth * (fmaxf(h, 0.0f) + soft);
      d_h = a.smooth - (h >= 0.0f ? e / (1.0f + e) : 1.0f / (1.0f + e));  // sigmoid(h) - (1 - smooth)
    } else if (a.kind == SS_PREF_HINGE) {
      loss = fmaxf(1.0f - h, 0.0f);
      d_h = h < 1.0f ? -1.0f : 0.0f;
    } else {
      const float q = (h - 0.5f) / a.beta;
      loss = q * q;
      d_h = 2.0f * q / a.beta;
    }
    if (!(h == h)) loss = d_h = nan_f();
    slope[0] = static_cast<float>(static_cast<double>(wp * d_h) * a.beta * per[0]);
    slope[1] = static_cast<float>(-static_cast<double>(wp * d_h) * a.beta * per[1]);
    if (cl.rank == 0) {
      if (a.loss) a.loss[pair] = wp * loss;
      if (a.reward)
        a.reward[pair] = make_float2(static_cast<float>(a.beta * score[0]), static_cast<float>(a.beta * score[1]));
    }
  }
  if (!a.d) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float g = slope[k];
    over_tokens(at[k], cl.rank, cl.size, [&](int64_t i, int64_t step) {
      float w[kTokens];
#pragma unroll
      for (int u = 0; u < kTokens; ++u) w[u] = a.weight && i + u * step < at[k].hi ? a.weight[i + u * step] : 1.0f;
#pragma unroll
      for (int u = 0; u < kTokens; ++u)
        if (i + u * step < at[k].hi) a.d[i + u * step] = w[u] == 0.0f ? 0.0f : w[u] * g;
    });
  }
}

ss_status preference_impl(const float* logprob, int64_t rows, const ss_preference* p, int64_t pairs, float* loss,
                          float* reward, float* d_logprob, void* stream) {
  if (!p->offsets || (!logprob && rows > 0)) return SS_ERR_INVALID_ARG;
  if (p->kind != SS_PREF_SIGMOID && p->kind != SS_PREF_HINGE && p->kind != SS_PREF_SQUARE) return SS_ERR_INVALID_ARG;
  if (!(p->beta > 0.0f) || !std::isfinite(p->beta) || !std::isfinite(p->margin)) return SS_ERR_INVALID_ARG;
  if (!(p->label_smoothing >= 0.0f) || !(p->label_smoothing <= 1.0f)) return SS_ERR_INVALID_ARG;
  if (p->label_smoothing != 0.0f && p->kind != SS_PREF_SIGMOID) return SS_ERR_INVALID_ARG;
  if (p->idtype != SS_I32 && p->idtype != SS_I64) return SS_ERR_DTYPE;
  if (rows > INT64_MAX / 4 || pairs > INT32_MAX / 8) return SS_ERR_OVERFLOW;
  const int64_t ib = p->idtype == SS_I64 ? 8 : 4;
  if (misaligned(logprob, 4) || misaligned(p->ref_logprob, 4) || misaligned(p->row_weight, 4) ||
      misaligned(p->pair_weight, 4) || misaligned(p->offsets, ib) || misaligned(loss, 4) || misaligned(reward, 8) ||
      misaligned(d_logprob, 4))
    return SS_ERR_ALIGN;
  Ranges ranges;
  ranges.add(logprob, rows * 4, false);
  ranges.add(p->ref_logprob, rows * 4, false);
  ranges.add(p->row_weight, rows * 4, false);
  ranges.add(p->pair_weight, pairs * 4, false);
  ranges.add(p->offsets, (2 * pairs + 1) * ib, false);
  ranges.add(loss, pairs * 4, true);
  ranges.add(reward, pairs * 8, true);
  ranges.add(d_logprob, rows * 4, true);
  if (ranges.overlap()) return SS_ERR_OVERLAP;
  const PreferenceArgs a = {logprob, p->ref_logprob, p->row_weight, p->pair_weight, p->offsets, loss,
                            reinterpret_cast<float2*>(reward), d_logprob, rows, pairs, p->beta, p->margin,
                            p->label_smoothing, p->kind, p->idtype == SS_I64, p->halves != 0, p->average != 0};
  // threads and blocks by the tokens of a pair, on average: eight of each sequence a thread
  const int64_t each = rows / pairs;
  int threads = 64;
  while (threads < kMaxThreads && each > 16 * threads) threads *= 2;
  int cluster = 1;
  while (cluster < kMaxCluster && each > 16 * cluster * threads && pairs * cluster * threads * 2 <= 1024 * sm_count())
    cluster *= 2;
  return launch_rows(preference_kernel, pairs, cluster, threads, 0, a, stream);
}

}  // namespace
}  // namespace ss

extern "C" {

ss_status ss_preference_loss(const float* logprob, int64_t rows, const ss_preference* preference, int64_t pairs,
                             float* loss, float* reward, float* d_logprob, void* stream) {
  if (!preference || rows < 0 || pairs < 0) return SS_ERR_INVALID_ARG;
  if (pairs == 0) return SS_OK;
  if (!loss && !reward && !d_logprob && rows > 0) return SS_ERR_INVALID_ARG;
  return ss::preference_impl(logprob, rows, preference, pairs, loss, reward, d_logprob, stream);
}

}  // extern "C"
