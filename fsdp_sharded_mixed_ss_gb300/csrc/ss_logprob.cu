// ss_logprob.cu -- log probabilities of given tokens with entropy and top
// alternatives (ss_token_logprobs), and their gradient (ss_token_logprobs_grad).
#include "ss_logits.cuh"

namespace ss {
namespace {

constexpr int kRowThreads = 256;

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

// One block per row: one pass for the maximum, the sum and the entropy's sum,
// then one pass per alternative for the largest pair below the last.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) logprob_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int V = kVecOf<DT>;
  __shared__ RowSum red[kRowThreads / 32];
  __shared__ uint64_t best[kRowThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const Elem<DT>* x = static_cast<const Elem<DT>*>(a.x) + row * a.ld;
  const Slice<DT> sl(x, a.vocab);
  RowSum acc = RowSum::none();
  auto add1 = [&](float f) {
    if (f > acc.m) acc.move(f, a.c);
    acc.add(f, a.c, acc.ref());
  };
  for (int64_t i = threadIdx.x; i < sl.head; i += kRowThreads) add1(to_float<DT>(x[i]));
  for (int64_t i = sl.tail() + threadIdx.x; i < sl.n; i += kRowThreads) add1(to_float<DT>(x[i]));
  const uint4* v = reinterpret_cast<const uint4*>(x + sl.head);
  for (int64_t i = threadIdx.x; i < sl.nvec; i += kRowThreads) {
    float f[V];
    unpack<DT>(v[i], f);
    float m = f[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, f[j]);
    if (m > acc.m) acc.move(m, a.c);
    const float ref = acc.ref();
#pragma unroll
    for (int j = 0; j < V; ++j) acc.add(f[j], a.c, ref);
  }
  acc = block_merge<kRowThreads>(acc, a.c, red);
  const bool nan = !(acc.s == acc.s);
  const bool empty = acc.s == 0.0f;
  const float ln_s = logf(acc.s);
  auto logp = [&](float f) {
    if (nan) return nan_f();
    return empty ? -kInf : fmaf(f - acc.m, a.scale, -ln_s);
  };
  if (threadIdx.x == 0) {
    if (a.norm) a.norm[row] = make_float2(acc.m, acc.s);
    if (a.lse) a.lse[row] = empty ? -kInf : fmaf(acc.m, a.scale, ln_s);
    if (a.entropy) {
      const float h = empty ? 0.0f : ln_s - acc.t / acc.s * kLn2;
      a.entropy[row] = h < 0.0f ? 0.0f : h;
    }
    if (a.logprob) {
      const int64_t t = load_id(a.tokens, row, a.wide);
      a.logprob[row] = t < 0 ? 0.0f : (t >= a.vocab ? nan_f() : logp(to_float<DT>(x[t])));
    }
  }
  uint64_t last = ~0ull;
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t m = 0;
    if (!nan) {
      for (int64_t i = threadIdx.x; i < a.vocab; i += kRowThreads) {
        const uint64_t p = order_pair(to_float<DT>(x[i]), i);
        if (p < last && p > m) m = p;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, m, off);
      m = o > m ? o : m;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) best[threadIdx.x >> 5] = m;
    __syncthreads();
    m = best[0];
#pragma unroll
    for (int w = 1; w < kRowThreads / 32; ++w) m = best[w] > m ? best[w] : m;
    last = m;
    if (threadIdx.x == 0) {
      const int64_t o = row * a.top_k + j;
      if (a.top_id) store_id(a.top_id, o, nan ? -1 : static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(m)), a.wide);
      if (a.top_logprob) a.top_logprob[o] = logp(key_value(static_cast<uint32_t>(m >> 32)));
    }
  }
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
};

// One block per row. Every element is p (A + B log2 p); the listed ids, whose
// logits are read before anything is written (the gradient may replace the
// logits), get their own terms on top afterwards.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) logprob_grad_kernel(const __grid_constant__ LogprobGradArgs a) {
  constexpr int V = kVecOf<DT>;
  __shared__ int64_t ids[SS_MAX_TOP + 1];
  __shared__ float up[SS_MAX_TOP + 1];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const Elem<DT>* x = static_cast<const Elem<DT>*>(a.x) + row * a.ld;
  Elem<DT>* d = static_cast<Elem<DT>*>(a.d) + row * a.d_ld;
  const int n_ids = a.top_k + 1;
  for (int j = threadIdx.x; j < n_ids; j += kRowThreads) {
    int64_t id = -1;
    float u = 0.0f;
    if (j < a.top_k) {
      if (a.d_top) {
        id = load_id(a.top_id, row * a.top_k + j, a.wide);
        u = a.d_top[row * a.top_k + j];
      }
    } else if (a.d_logprob) {
      id = load_id(a.tokens, row, a.wide);
      u = a.d_logprob[row];
    }
    ids[j] = id;
    up[j] = id < 0 ? 0.0f : (id >= a.vocab ? nan_f() : u);
  }
  __syncthreads();
  const float dl = a.d_lse ? a.d_lse[row] : 0.0f;
  const float dh = a.d_entropy ? a.d_entropy[row] : 0.0f;
  float sum = 0.0f;
  bool any = dl != 0.0f || dh != 0.0f;
  for (int j = 0; j < n_ids; ++j) {
    sum += up[j];
    any = any || up[j] != 0.0f;
  }
  const float2 norm = a.norm[row];
  const bool dead = !any || norm.y == 0.0f;
  const float l2 = log2f(norm.y);
  const float A = dead ? 0.0f : a.scale * (dl - sum - (a.d_entropy ? dh * a.entropy[row] : 0.0f));
  const float B = dead ? 0.0f : -a.scale * dh * kLn2;
  // the listed elements' whole gradients, by the threads that hold them: several slots may name one id
  float mine = 0.0f;
  int64_t my_id = -1;
  auto grad = [&](float f) {
    const float l = fmaf(f - norm.x, a.c, -l2);
    return ex2(l) * fmaf(B, fmaxf(l, kFloor), A);
  };
  if (threadIdx.x < n_ids && !dead && ids[threadIdx.x] >= 0 && ids[threadIdx.x] < a.vocab) {
    my_id = ids[threadIdx.x];
    float u = 0.0f;
    for (int j = 0; j < n_ids; ++j)
      if (ids[j] == my_id) u += up[j];
    mine = fmaf(a.scale, u, grad(to_float<DT>(x[my_id])));
  }
  __syncthreads();
  if (a.vec) {
    const Slice<DT> sl(x, a.vocab);
    for (int64_t i = threadIdx.x; i < sl.head; i += kRowThreads)
      d[i] = from_float<DT>(dead ? 0.0f : grad(to_float<DT>(x[i])));
    for (int64_t i = sl.tail() + threadIdx.x; i < sl.n; i += kRowThreads)
      d[i] = from_float<DT>(dead ? 0.0f : grad(to_float<DT>(x[i])));
    const uint4* v = reinterpret_cast<const uint4*>(x + sl.head);
    uint4* w = reinterpret_cast<uint4*>(d + sl.head);
    for (int64_t i = threadIdx.x; i < sl.nvec; i += kRowThreads) {
      float f[V];
      if (dead) {
        w[i] = make_uint4(0u, 0u, 0u, 0u);
      } else {
        unpack<DT>(v[i], f);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = grad(f[j]);
        w[i] = pack<DT>(f);
      }
    }
  } else {
    for (int64_t i = threadIdx.x; i < a.vocab; i += kRowThreads)
      d[i] = from_float<DT>(dead ? 0.0f : grad(to_float<DT>(x[i])));
  }
  __syncthreads();
  if (my_id >= 0) d[my_id] = from_float<DT>(mine);
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
  auto* fn = x->dtype == SS_BF16 ? logprob_kernel<SS_BF16>
                                 : (x->dtype == SS_FP16 ? logprob_kernel<SS_FP16> : logprob_kernel<SS_FP32>);
  return launch(fn, static_cast<unsigned>(rows), a, stream, kRowThreads);
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
  const LogprobGradArgs a = {x->data, tokens, top_id, reinterpret_cast<const float2*>(norm), entropy, up->d_logprob, up->d_entropy, up->d_lse,
                             up->d_top_logprob, d_logits, rows, x->vocab, x->ld, d_ld, x->scale * kLog2e, x->scale,
                             top_k, idtype == SS_I64, same_phase(x, d_logits, d_ld)};
  auto* fn = x->dtype == SS_BF16
                 ? logprob_grad_kernel<SS_BF16>
                 : (x->dtype == SS_FP16 ? logprob_grad_kernel<SS_FP16> : logprob_grad_kernel<SS_FP32>);
  return launch(fn, static_cast<unsigned>(rows), a, stream, kRowThreads);
}

}  // extern "C"
