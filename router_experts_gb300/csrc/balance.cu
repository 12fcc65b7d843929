// balance.cu -- expert-load balance loss, per-expert counts and the gradient
// of the gate's logits.
//
//   f_be = E c_be / A_b,  A_b = sum_e c_be;   p_te = d-normalised scores
//   L = coef / B' * sum_b 1/n_b sum_t sum_e f_be p_te
//   dL/dl_te = coef / (B' n_b) * d_te * (f_be - sum_j f_bj p_tj)
//
// Near balance every f is close to one and the bracket cancels.  With
// g = f - 1 = (E c - A) / A, whose numerator is a whole number, and
// sum_j p_tj = 1 - r (r = 1e-20 / sum, zero for softmax),
//   f_e - sum_j f_j p_j = g_e - sum_j g_j p_j + r
// keeps the bracket's relative precision, and sum f p = sum g p + 1 - r.
//
// Two launches: the counts (integer atomics: any order gives the same sums),
// then one warp per token that reads the row once.  Each lane owns the same
// experts for every token, so it keeps their g in registers.
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;

struct BalanceArgs {
  const void* logits;
  const int32_t* ids;
  const uint8_t* mask;
  const int32_t* starts;
  int32_t* counts;
  int32_t* tokens;
  const float* dloss;
  float* loss;
  void* dlogits;
  double* part;  // [grid] sums of the CTAs
  int* ticket;
  int* err;
  float coef;
  int B, T, E, k, scoring;
  int chunk;     // tokens of a CTA
};

// Sequence of token t: the last one that starts at or before it; -1 when t is
// before the first start or past the last end.
MOE_DEV int sequence_of(const int32_t* starts, int B, int t) {
  if (!starts) return 0;
  if (t < __ldg(starts)) return -1;
  int lo = 0, hi = B;  // starts[lo] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(starts + mid) <= t) lo = mid;
    else hi = mid;
  }
  return t < __ldg(starts + lo + 1) ? lo : -1;
}

__global__ void __launch_bounds__(kBalThreads) balance_count_kernel(const BalanceArgs a) {
  __shared__ int hist[512];
  __shared__ int seen;
  const int t0 = blockIdx.x * a.chunk;
  const int t1 = static_cast<int>(min(static_cast<long long>(a.T),
                                      static_cast<long long>(t0) + a.chunk));
  bool bad = false;
  for (int t = t0; t < t1;) {
    // the piece of this CTA's tokens that lies in one sequence
    const int b = sequence_of(a.starts, a.B, t);
    int end = t1;
    if (a.starts) {
      const int nxt = b >= 0 ? __ldg(a.starts + b + 1) : __ldg(a.starts);
      if (nxt > t) end = min(end, nxt);
    }
    if (b >= 0) {
      for (int e = threadIdx.x; e < a.E; e += kBalThreads) hist[e] = 0;
      if (threadIdx.x == 0) seen = 0;
      __syncthreads();
      for (long long i = static_cast<long long>(t) * a.k + threadIdx.x;
           i < static_cast<long long>(end) * a.k; i += kBalThreads) {
        const int tok = static_cast<int>(i / a.k);
        if (a.mask && !a.mask[tok]) continue;
        const int e = __ldg(a.ids + i);
        if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
        else bad = true;
        if (i % a.k == 0) atomicAdd(&seen, 1);
      }
      __syncthreads();
      for (int e = threadIdx.x; e < a.E; e += kBalThreads)
        if (hist[e]) atomicAdd(a.counts + static_cast<size_t>(b) * a.E + e, hist[e]);
      if (threadIdx.x == 0 && seen) atomicAdd(a.tokens + b, seen);
      __syncthreads();
    }
    t = end;
  }
  if (bad) raise_error(a.err, kErrBadExpert);
}

MOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
MOE_DEV float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Score s(l) and its derivative.
template <int SCORING>
MOE_DEV void score_of(float l, float* s, float* d) {
  if constexpr (SCORING == 1) {
    const float q = 1.f / (1.f + expf(-l));
    *s = q;
    *d = q * (1.f / (1.f + expf(l)));  // 1 - q without its cancellation at large l
  } else {
    // sqrt(softplus): softplus = max(l, 0) + log1p(e^-|l|); d = sigmoid / (2 s)
    const float sp = fmaxf(l, 0.f) + log1pf(expf(-fabsf(l)));
    const float r = sqrtf(sp);
    *s = r;
    // below -15, sigmoid = softplus to 32 bits: d = s / 2 (no 0 / 0 at -inf)
    *d = l < -15.f ? 0.5f * r : 0.5f / (r * (1.f + expf(-l)));
  }
}

// Expert of slot i of a lane: vector loads of four experts (VEC) or one.
template <bool VEC>
MOE_DEV int expert_of(int lane, int i) {
  return VEC ? (i >> 2) * 128 + lane * 4 + (i & 3) : i * 32 + lane;
}

template <bool VEC, int SLOTS, bool BF16>
MOE_DEV void load_row(const void* logits, size_t row, int lane, int E, float (&l)[SLOTS]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < SLOTS; i += 4) {
      const int e = expert_of<VEC>(lane, i);
      if (e < E) {
        if constexpr (BF16) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(
              static_cast<const __nv_bfloat16*>(logits) + row + e));
          l[i] = __uint_as_float(v.x << 16);
          l[i + 1] = __uint_as_float(v.x & 0xFFFF0000u);
          l[i + 2] = __uint_as_float(v.y << 16);
          l[i + 3] = __uint_as_float(v.y & 0xFFFF0000u);
        } else {
          const float4 v =
              __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(logits) + row + e));
          l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int e = expert_of<VEC>(lane, i);
      if (e < E)
        l[i] = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(logits)[row + e])
                    : static_cast<const float*>(logits)[row + e];
    }
  }
}

template <bool VEC, int SLOTS, bool BF16>
MOE_DEV void store_row(void* out, size_t row, int lane, int E, const float (&d)[SLOTS]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < SLOTS; i += 4) {
      const int e = expert_of<VEC>(lane, i);
      if (e < E) {
        if constexpr (BF16)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + row + e) =
              make_uint2(pack_bf16x2(d[i], d[i + 1]), pack_bf16x2(d[i + 2], d[i + 3]));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(out) + row + e) =
              make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int e = expert_of<VEC>(lane, i);
      if (e < E) {
        if constexpr (BF16) static_cast<__nv_bfloat16*>(out)[row + e] = __float2bfloat16_rn(d[i]);
        else static_cast<float*>(out)[row + e] = d[i];
      }
    }
  }
}

// One warp per token; a CTA's warps walk its chunk of consecutive tokens.
template <int SCORING, bool VEC, int SLOTS, bool BF16>
__global__ void __launch_bounds__(kBalThreads) balance_token_kernel(const BalanceArgs a) {
  __shared__ double sums[kBalWarps];
  __shared__ int nseq, last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // B': sequences that hold a counted token
  if (threadIdx.x == 0) nseq = 0;
  __syncthreads();
  int mine = 0;
  for (int b = threadIdx.x; b < a.B; b += kBalThreads) mine += __ldcg(a.tokens + b) > 0;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0 && mine) atomicAdd(&nseq, mine);
  __syncthreads();
  const int Bp = nseq;
  const float scale = a.dloss ? a.coef * __ldg(a.dloss) : a.coef;

  const int t0 = blockIdx.x * a.chunk;
  const int t1 = static_cast<int>(min(static_cast<long long>(a.T),
                                      static_cast<long long>(t0) + a.chunk));
  double acc = 0.0;
  int cur = -2, until = 0;  // sequence in the registers below, and where it ends
  float g[SLOTS], share = 0.f;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) g[i] = 0.f;
  for (int t = t0 + warp; t < t1; t += kBalWarps) {
    if (cur == -2 || t >= until) {
      const int b = sequence_of(a.starts, a.B, t);
      until = a.starts ? (b >= 0 ? __ldg(a.starts + b + 1) : t + 1) : a.T;
      if (b != cur) {
        cur = b;
        share = 0.f;
        if (b >= 0) {
          const int n = __ldcg(a.tokens + b);
          share = n > 0 ? static_cast<float>(1.0 / (static_cast<double>(Bp) * n)) : 0.f;
          int c[SLOTS];
          int placed = 0;
#pragma unroll
          for (int i = 0; i < SLOTS; ++i) {
            const int e = expert_of<VEC>(lane, i);
            c[i] = e < a.E ? __ldcg(a.counts + static_cast<size_t>(b) * a.E + e) : 0;
            placed += c[i];
          }
          placed = __reduce_add_sync(0xffffffffu, placed);
          // no assignment placed (all ids bad): f = 0
          const float inv = placed > 0 ? 1.f / static_cast<float>(placed) : 0.f;
#pragma unroll
          for (int i = 0; i < SLOTS; ++i)
            g[i] = placed > 0 ? static_cast<float>(static_cast<long long>(a.E) * c[i] - placed) * inv
                              : -1.f;
        }
      }
    }
    const size_t row = static_cast<size_t>(t) * a.E;
    const bool counted = cur >= 0 && (!a.mask || a.mask[t]);
    float d[SLOTS];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) d[i] = 0.f;
    if (counted) {
      float l[SLOTS];
      load_row<VEC, SLOTS, BF16>(a.logits, row, lane, a.E, l);
      float sum = 0.f, gs = 0.f;
      if constexpr (SCORING == 0) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
          if (expert_of<VEC>(lane, i) < a.E) m = l[i] > m || l[i] != l[i] ? l[i] : m;
        m = warp_max(m);
        const float m0 = m == -INFINITY ? 0.f : m;  // all -inf: every term stays zero
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
          if (expert_of<VEC>(lane, i) < a.E) d[i] = expf(l[i] - m0);
          sum += d[i];
          gs = fmaf(g[i], d[i], gs);
        }
      } else {
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
          float s = 0.f;
          if (expert_of<VEC>(lane, i) < a.E) score_of<SCORING>(l[i], &s, &d[i]);
          sum += s;
          gs = fmaf(g[i], s, gs);
        }
      }
      sum = warp_sum(sum);
      gs = warp_sum(gs);
      float inv, rest;  // 1 / normaliser, 1 - sum p
      if constexpr (SCORING == 0) {
        inv = sum == 0.f ? 0.f : 1.f / sum;
        rest = sum == 0.f ? 1.f : 0.f;
      } else {
        inv = 1.f / (sum + 1e-20f);
        rest = 1e-20f * inv;
      }
      const float mean = gs * inv - rest;  // sum f p - 1
      acc += static_cast<double>(share) * (1.0 + static_cast<double>(mean));
      const float c = share * scale * inv;
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) d[i] = c * d[i] * (g[i] - mean);
    }
    if (a.dlogits) store_row<VEC, SLOTS, BF16>(a.dlogits, row, lane, a.E, d);
  }
  if (!a.loss) return;
  // the CTAs' sums in a fixed order, by the last CTA to finish
  if (lane == 0) sums[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kBalWarps; ++w) s += sums[w];
    __stcg(a.part + blockIdx.x, s);
    last = ticket_add_acq_rel(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    if (last) store_relaxed_gpu(a.ticket, 0);
  }
  __syncthreads();
  if (last) {
    double s = 0.0;
    for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kBalThreads)
      s += __ldcg(a.part + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      s = 0.0;
      for (int w = 0; w < kBalWarps; ++w) s += sums[w];
      *a.loss = static_cast<float>(s * a.coef);
    }
  }
}

template <int SCORING, bool BF16>
void launch_slots(const BalanceArgs& a, bool vec, int grid, cudaStream_t st) {
  if (vec) {
    if (a.E <= 128) balance_token_kernel<SCORING, true, 4, BF16><<<grid, kBalThreads, 0, st>>>(a);
    else if (a.E <= 256) balance_token_kernel<SCORING, true, 8, BF16><<<grid, kBalThreads, 0, st>>>(a);
    else if (a.E <= 384) balance_token_kernel<SCORING, true, 12, BF16><<<grid, kBalThreads, 0, st>>>(a);
    else balance_token_kernel<SCORING, true, 16, BF16><<<grid, kBalThreads, 0, st>>>(a);
  } else {
    if (a.E <= 32) balance_token_kernel<SCORING, false, 1, BF16><<<grid, kBalThreads, 0, st>>>(a);
    else if (a.E <= 64) balance_token_kernel<SCORING, false, 2, BF16><<<grid, kBalThreads, 0, st>>>(a);
    else if (a.E <= 128) balance_token_kernel<SCORING, false, 4, BF16><<<grid, kBalThreads, 0, st>>>(a);
    else if (a.E <= 256) balance_token_kernel<SCORING, false, 8, BF16><<<grid, kBalThreads, 0, st>>>(a);
    else balance_token_kernel<SCORING, false, 16, BF16><<<grid, kBalThreads, 0, st>>>(a);
  }
}

int launch_tokens(BalanceArgs a, bool bf16, bool vec, cudaStream_t st) {
  const int grid = balance_grid(a.T);
  a.chunk = (a.T + grid - 1) / grid;
  if (a.scoring == 0) {
    if (bf16) launch_slots<0, true>(a, vec, grid, st);
    else launch_slots<0, false>(a, vec, grid, st);
  } else if (a.scoring == 1) {
    if (bf16) launch_slots<1, true>(a, vec, grid, st);
    else launch_slots<1, false>(a, vec, grid, st);
  } else {
    if (bf16) launch_slots<2, true>(a, vec, grid, st);
    else launch_slots<2, false>(a, vec, grid, st);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_balance_loss(const void* logits, bool bf16, const int32_t* ids, const uint8_t* mask,
                        const int32_t* starts, int B, int T, int E, int k, int scoring,
                        float coef, float* loss, int32_t* counts, int32_t* tokens, void* dlogits,
                        bool vec, double* part, int* ticket, int* err, cudaStream_t st) {
  if (cudaMemsetAsync(counts, 0, static_cast<size_t>(B) * E * 4, st) != cudaSuccess ||
      cudaMemsetAsync(tokens, 0, static_cast<size_t>(B) * 4, st) != cudaSuccess)
    return -1;
  if (T == 0) return cudaMemsetAsync(loss, 0, 4, st) == cudaSuccess ? 0 : -1;
  BalanceArgs a{};
  a.logits = logits;
  a.ids = ids;
  a.mask = mask;
  a.starts = starts;
  a.counts = counts;
  a.tokens = tokens;
  a.loss = loss;
  a.dlogits = dlogits;
  a.part = part;
  a.ticket = ticket;
  a.err = err;
  a.coef = coef;
  a.B = B;
  a.T = T;
  a.E = E;
  a.k = k;
  a.scoring = scoring;
  const int grid = balance_grid(T);
  a.chunk = (T + grid - 1) / grid;
  balance_count_kernel<<<grid, kBalThreads, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return -1;
  return launch_tokens(a, bf16, vec, st);
}

int launch_balance_loss_backward(const float* dloss, const void* logits, bool bf16,
                                 const int32_t* counts, const int32_t* tokens,
                                 const uint8_t* mask, const int32_t* starts, int B, int T, int E,
                                 int scoring, float coef, void* dlogits, bool vec,
                                 cudaStream_t st) {
  BalanceArgs a{};
  a.logits = logits;
  a.mask = mask;
  a.starts = starts;
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.coef = coef;
  a.B = B;
  a.T = T;
  a.E = E;
  a.scoring = scoring;
  return launch_tokens(a, bf16, vec, st);
}

}  // namespace moe
