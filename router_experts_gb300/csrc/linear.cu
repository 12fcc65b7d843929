// linear.cu -- dense product with bias, activation and residual in its
// epilogue:  out[t, n] = act(sum_k x[t, k] w[n, k] + bias[n]) + residual[t, n].
//
// Tiles put the weights on the MMA's 128 rows (TMEM lanes) and the tokens on
// its columns: a thread of the epilogue owns one output column n and walks
// the tile's tokens, so the 32 lanes of a warp touch 32 neighbouring outputs
// of one token whatever N's alignment, and one token costs a tile of 16
// columns and not of 128.  A gated tile (swiglu) takes the 128 gate rows and
// the matching 128 up rows into two accumulators, which the same thread reads.
//
// One persistent kernel, six warps:
//   warp 0     TMA producer into a ring of 64-wide K steps
//   warp 1     TMEM allocator; one thread issues tcgen05.mma
//   warps 2-5  epilogue (two accumulators: it overlaps the next tile's MMAs)
// Few tokens and few tiles leave SMs idle, so the K range is split; the last
// split of a tile to finish (ticket, no spinning) sums the 32-bit partials in
// split order and runs the epilogue: the same inputs give the same bits.
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kBK = 64;  // K elements of a stage (128 bytes of bf16)

struct LinearArgs {
  const float* bias;
  const void* residual;
  void* out;
  float* partial;
  int* tickets;
  int* err;
  int act, residual_f32, out_f32;
  int T, K, N;
  int tiles_n, tiles_t, splits;
};

template <bool GATED, int BN>
struct LinearCfg {
  static constexpr int A_BYTES = (GATED ? 2 : 1) * 128 * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES_RAW = 200 * 1024 / STAGE_BYTES;
  static constexpr int STAGES = STAGES_RAW > 12 ? 12 : STAGES_RAW;
  static constexpr int ACC_COLS = (GATED ? 2 : 1) * BN;
  static constexpr int TMEM_COLS = 2 * ACC_COLS < 32 ? 32 : 2 * ACC_COLS;  // powers of two
  static constexpr int THREADS = 192;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 512;
  static_assert(TMEM_COLS <= 512 && SMEM_BYTES <= 232448, "budgets");
};

MOE_DEV float silu_f(float v) { return __fdividef(v, 1.f + __expf(-v)); }
MOE_DEV float activate(int act, float v, float u) {
  if (act == 3) return silu_f(v) * u;
  if (act == 1) return silu_f(v);
  if (act == 2) return 0.5f * v * erfcf(v * -0.70710678f);  // no 1 + erf near -1
  return v;
}

// Outputs of one thread: column n, tokens t0 .. t0 + 15 of which `cols` exist.
MOE_DEV void write_cols(const LinearArgs& a, int n, int t0, int cols, const float (&v)[16],
                        const float (&u)[16], float bg, float bu) {
  if (n >= a.N) return;
  float r[16];
  if (a.residual) {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const size_t at = static_cast<size_t>(t0 + c) * a.N + n;
      r[c] = 0.f;
      if (c < cols)
        r[c] = a.residual_f32 ? static_cast<const float*>(a.residual)[at]
                              : __bfloat162float(static_cast<const __nv_bfloat16*>(a.residual)[at]);
    }
  }
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    if (c < cols) {
      float o = activate(a.act, v[c] + bg, u[c] + bu);
      if (a.residual) o += r[c];
      const size_t at = static_cast<size_t>(t0 + c) * a.N + n;
      if (a.out_f32) static_cast<float*>(a.out)[at] = o;
      else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(o);
    }
  }
}

MOE_DEV void load_acc(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  tmem_ld16(taddr, r);
  tmem_ld_wait();
  reg_fence16(r);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

template <bool GATED, int BN>
__global__ void __launch_bounds__(LinearCfg<GATED, BN>::THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tm_w,
                  const __grid_constant__ CUtensorMap tm_x, const LinearArgs a) {
  using C = LinearCfg<GATED, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE_BYTES);
  uint64_t* empty_bar = full_bar + C::STAGES;
  uint64_t* tfull_bar = empty_bar + C::STAGES;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty_bar + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = abort_flag + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = (a.K + kBK - 1) / kBK;
  const int units = a.tiles_n * a.tiles_t * a.splits;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], 4);
    }
    *abort_flag = 0;
    *last_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // unit u: split fastest, then the token tiles of one weight tile
  struct Unit {
    int tile, n0, t0, s, kb0, kb1;
  };
  auto unit_of = [&](int u) {
    Unit x;
    x.s = u % a.splits;
    x.tile = u / a.splits;
    x.n0 = x.tile / a.tiles_t * 128;
    x.t0 = x.tile % a.tiles_t * BN;
    x.kb0 = static_cast<int>(static_cast<long long>(x.s) * KB / a.splits);
    x.kb1 = static_cast<int>(static_cast<long long>(x.s + 1) * KB / a.splits);
    return x;
  };

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_w);
      tma_prefetch_desc(&tm_x);
      uint32_t it = 0;
      bool alive = true;
      for (int uu = blockIdx.x; alive && uu < units; uu += gridDim.x) {
        const Unit u = unit_of(uu);
        for (int kb = u.kb0; kb < u.kb1; ++kb, ++it) {
          const int st = it % C::STAGES;
          if (!mbar_wait(&empty_bar[st], ((it / C::STAGES) & 1u) ^ 1u, abort_flag, a.err)) {
            alive = false;
            break;
          }
          uint8_t* sa = smem + st * C::STAGE_BYTES;
          mbar_arrive_expect_tx(&full_bar[st], C::STAGE_BYTES);
          tma_load_2d(sa, &tm_w, &full_bar[st], kb * kBK, u.n0);
          if constexpr (GATED)
            tma_load_2d(sa + 128 * 128, &tm_w, &full_bar[st], kb * kBK, a.N + u.n0);
          tma_load_2d(sa + C::A_BYTES, &tm_x, &full_bar[st], kb * kBK, u.t0);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t it = 0, acc_it = 0;
      bool alive = true;
      for (int uu = blockIdx.x; alive && uu < units; uu += gridDim.x, ++acc_it) {
        const Unit u = unit_of(uu);
        const int buf = acc_it & 1;
        if (!mbar_wait(&tempty_bar[buf], ((acc_it >> 1) & 1u) ^ 1u, abort_flag, a.err)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * C::ACC_COLS;
        for (int kb = u.kb0; kb < u.kb1; ++kb, ++it) {
          const int st = it % C::STAGES;
          if (!mbar_wait(&full_bar[st], (it / C::STAGES) & 1u, abort_flag, a.err)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + st * C::STAGE_BYTES);
          const uint32_t sb = sa + C::A_BYTES;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint32_t acc = (kb > u.kb0 || kk > 0) ? 1u : 0u;
            const uint64_t bdesc = sw128_desc(sb + kk * 32);
            umma_f16(d, sw128_desc(sa + kk * 32), bdesc, idesc_bf16_f32(128, BN), acc);
            if constexpr (GATED)
              umma_f16(d + BN, sw128_desc(sa + 128 * 128 + kk * 32), bdesc,
                       idesc_bf16_f32(128, BN), acc);
          }
          umma_commit(&empty_bar[st]);
        }
        if (!alive) break;
        umma_commit(&tfull_bar[buf]);
      }
    }
  } else {
    const int ew = warp & 3;  // a warp reads the TMEM lane quarter warp % 4
    const int row = ew * 32 + lane;
    uint32_t acc_it = 0;
    for (int uu = blockIdx.x; uu < units; uu += gridDim.x, ++acc_it) {
      const Unit u = unit_of(uu);
      const int buf = acc_it & 1;
      const bool ok = mbar_wait(&tfull_bar[buf], (acc_it >> 1) & 1u, abort_flag, a.err);
      if (named_bar_any(1, 128, !ok || *abort_flag)) break;
      tc_fence_after();
      const uint32_t tb =
          tmem_base + (static_cast<uint32_t>(ew * 32) << 16) + buf * C::ACC_COLS;
      const int n = u.n0 + row;
      const int cols = min(BN, a.T - u.t0);
      float bg = 0.f, bu = 0.f;
      if (a.bias && n < a.N) {
        bg = __ldg(a.bias + n);
        if constexpr (GATED) bu = __ldg(a.bias + a.N + n);
      }
      if (a.splits == 1) {
#pragma unroll 1
        for (int c0 = 0; c0 < cols; c0 += 16) {
          float v[16], w[16];
          load_acc(tb + c0, v);
          if constexpr (GATED) load_acc(tb + BN + c0, w);
          write_cols(a, n, u.t0 + c0, cols - c0, v, w, bg, bu);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty_bar[buf]);
      } else {
        // partial [tile][split][column][128 rows]: lanes are neighbours
        const size_t slot = static_cast<size_t>(C::ACC_COLS) * 128;
        float* base = a.partial + static_cast<size_t>(u.tile) * a.splits * slot + row;
        float* mine = base + u.s * slot;
#pragma unroll 1
        for (int c0 = 0; c0 < cols; c0 += 16) {
#pragma unroll
          for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            float v[16];
            load_acc(tb + h * BN + c0, v);
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (c0 + c < cols) __stcg(mine + static_cast<size_t>(h * BN + c0 + c) * 128, v[c]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty_bar[buf]);
        named_bar_sync(1, 128);
        if (threadIdx.x == 64) {
          const int last = ticket_add_acq_rel(a.tickets + u.tile, 1) == a.splits - 1;
          if (last) store_relaxed_gpu(a.tickets + u.tile, 0);  // ready for the next launch
          *last_flag = last;
        }
        named_bar_sync(1, 128);
        if (*last_flag) {
#pragma unroll 1
          for (int c0 = 0; c0 < cols; c0 += 16) {
            float v[16], w[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] = w[c] = 0.f;
            for (int s = 0; s < a.splits; ++s) {
              const float* p = base + s * slot;
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (c0 + c < cols) {
                  v[c] += __ldcg(p + static_cast<size_t>(c0 + c) * 128);
                  if constexpr (GATED) w[c] += __ldcg(p + static_cast<size_t>(BN + c0 + c) * 128);
                }
            }
            write_cols(a, n, u.t0 + c0, cols - c0, v, w, bg, bu);
          }
        }
      }
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <bool GATED, int BN>
int launch_tile(const CUtensorMap& tw, const CUtensorMap& tx, const LinearArgs& a, int num_sms,
                cudaStream_t stream) {
  using C = LinearCfg<GATED, BN>;
  static std::atomic<unsigned long long> smem_set{0};
  if (!ensure_smem_limit(reinterpret_cast<const void*>(linear_kernel<GATED, BN>), C::SMEM_BYTES,
                         smem_set))
    return -1;
  const int units = a.tiles_n * a.tiles_t * a.splits;
  const int grid = units < num_sms ? units : num_sms;
  linear_kernel<GATED, BN><<<grid, C::THREADS, C::SMEM_BYTES, stream>>>(tw, tx, a);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

LinearPlan plan_linear(int T, int K, int N, bool gated, int num_sms) {
  LinearPlan p{};
  p.bn = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
  p.tiles_n = (N + 127) / 128;
  p.tiles_t = (T + p.bn - 1) / p.bn;
  const int KB = (K + kBK - 1) / kBK;
  const long long tiles = static_cast<long long>(p.tiles_n) * p.tiles_t;
  p.splits = 1;
  if (tiles > 0 && tiles < num_sms) {
    int s = static_cast<int>(num_sms / tiles);
    if (s > KB / 4) s = KB / 4;  // at least four K steps a unit
    if (s > 1) p.splits = s;
  }
  p.partial_bytes = p.splits > 1 ? align_up(static_cast<size_t>(tiles) * p.splits *
                                                (gated ? 2 : 1) * p.bn * 128 * 4,
                                            256)
                                 : 0;
  return p;
}

int launch_linear(const void* x, const void* w, const float* bias, int act, const void* residual,
                  int residual_f32, int T, int K, int N, void* out, int out_f32,
                  const LinearPlan& plan, float* partial, int* tickets, int* err, int num_sms,
                  cudaStream_t stream, const char** why) {
  const bool gated = act == 3;
  CUtensorMap tw, tx;
  if (!make_map_bf16(&tw, w, static_cast<uint64_t>(N) * (gated ? 2 : 1), K, 128) ||
      !make_map_bf16(&tx, x, T, K, plan.bn)) {
    *why = "cuTensorMapEncodeTiled failed for the dense product";
    return -1;
  }
  LinearArgs a{};
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.partial = partial;
  a.tickets = tickets;
  a.err = err;
  a.act = act;
  a.residual_f32 = residual_f32;
  a.out_f32 = out_f32;
  a.T = T;
  a.K = K;
  a.N = N;
  a.tiles_n = plan.tiles_n;
  a.tiles_t = plan.tiles_t;
  a.splits = plan.splits;
  int rc;
  if (gated) {
    rc = plan.bn == 16   ? launch_tile<true, 16>(tw, tx, a, num_sms, stream)
         : plan.bn == 32 ? launch_tile<true, 32>(tw, tx, a, num_sms, stream)
         : plan.bn == 64 ? launch_tile<true, 64>(tw, tx, a, num_sms, stream)
                         : launch_tile<true, 128>(tw, tx, a, num_sms, stream);
  } else {
    rc = plan.bn == 16   ? launch_tile<false, 16>(tw, tx, a, num_sms, stream)
         : plan.bn == 32 ? launch_tile<false, 32>(tw, tx, a, num_sms, stream)
         : plan.bn == 64 ? launch_tile<false, 64>(tw, tx, a, num_sms, stream)
                         : launch_tile<false, 128>(tw, tx, a, num_sms, stream);
  }
  if (rc != 0) *why = "dense product kernel";
  return rc;
}

}  // namespace moe
