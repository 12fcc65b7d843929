// norm.cu -- residual addition + root-mean-square norm in one pass over the
// row, with bf16 rows and / or e4m3 codes + UE8M0 scales as its output.
//
//   s = x + residual,  y = s * rsqrt(mean(s^2) + eps) * weight
//
// s, its squares' sum and y are 32-bit; what is rounded is only what leaves
// the kernel, each once (s to the residual's type, y to bf16, y / 2^p to
// e4m3).  A row is read once: its s stays in registers between the sum and
// the scaling.  The kernel is bound by HBM (it moves 2-16 bytes per element
// and does about five operations on it).
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

struct NormArgs {
  const void* x;
  const void* res;
  const void* w;
  void* res_out;
  __nv_bfloat16* y;
  uint8_t* codes;
  uint8_t* scales;
  float eps;
  int T, H;
  int w_f32;
  int group;  // threads of one row (a multiple of 32)
};

template <int N>
MOE_DEV void load_f32(const float* p, float (&v)[N]) {
  if constexpr (N == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = *p;
  }
}
template <int N>
MOE_DEV void load_bf16(const __nv_bfloat16* p, float (&v)[N]) {
  if constexpr (N == 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
    v[0] = __bfloat162float(*p);
  }
}
template <int N>
MOE_DEV void store_bf16(__nv_bfloat16* p, const float (&v)[N]) {
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  else
    *p = __float2bfloat16_rn(v[0]);
}
template <int N>
MOE_DEV void store_f32(float* p, const float (&v)[N]) {
  if constexpr (N == 8) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}

// V elements per access; IT accesses of each thread cover a row (V = 8) or
// the row is walked twice (IT = 0, any length).
template <int V, int IT, bool XF32, int RES>  // RES: 0 none, 1 bf16, 2 f32
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a) {
  __shared__ float part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = threadIdx.x / a.group, tg = threadIdx.x % a.group;
  const int t = blockIdx.x * (blockDim.x / a.group) + g;
  const int nv = a.H / V;
  const bool live = t < a.T;
  const size_t row = static_cast<size_t>(live ? t : 0) * a.H;

  auto load_s = [&](int v, float (&s)[V]) {
    const size_t at = row + static_cast<size_t>(v) * V;
    if constexpr (XF32) load_f32<V>(static_cast<const float*>(a.x) + at, s);
    else load_bf16<V>(static_cast<const __nv_bfloat16*>(a.x) + at, s);
    if constexpr (RES != 0) {
      float r[V];
      if constexpr (RES == 2) load_f32<V>(static_cast<const float*>(a.res) + at, r);
      else load_bf16<V>(static_cast<const __nv_bfloat16*>(a.res) + at, r);
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] += r[i];
    }
  };

  constexpr int KEEP = IT > 0 ? IT : 1;
  float s[KEEP][V];
  float sum = 0.f;
  if constexpr (IT > 0) {
#pragma unroll
    for (int k = 0; k < IT; ++k) {
      const int v = tg + k * a.group;
      if (live && v < nv) load_s(v, s[k]);
      else
#pragma unroll
        for (int i = 0; i < V; ++i) s[k][i] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < IT; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) sum = fmaf(s[k][i], s[k][i], sum);
  } else if (live) {
    for (int v = tg; v < nv; v += a.group) {
      load_s(v, s[0]);
#pragma unroll
      for (int i = 0; i < V; ++i) sum = fmaf(s[0][i], s[0][i], sum);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int wpg = a.group >> 5;  // warps of a row
  if (wpg > 1) {
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    const int w0 = warp / wpg * wpg;
    sum = lane < wpg ? part[w0 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  const float rs = rsqrtf(sum / static_cast<float>(a.H) + a.eps);

  auto finish = [&](int v, float (&sv)[V]) {
    const bool in = live && v < nv;
    const size_t at = row + static_cast<size_t>(v) * V;
    float y[V];
    if (in) {
      float w[V];
      if (a.w_f32) load_f32<V>(static_cast<const float*>(a.w) + v * V, w);
      else load_bf16<V>(static_cast<const __nv_bfloat16*>(a.w) + v * V, w);
      if constexpr (RES == 1) store_bf16<V>(static_cast<__nv_bfloat16*>(a.res_out) + at, sv);
      if constexpr (RES == 2) store_f32<V>(static_cast<float*>(a.res_out) + at, sv);
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = sv[i] * rs * w[i];
      if (a.y) store_bf16<V>(a.y + at, y);
    }
    if constexpr (V == 8) {
      if (a.codes) {
        // the 32 values of a scale are four neighbouring lanes' (a row's
        // vectors are a multiple of four, so the four are in or out together)
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) amax = fmaxf(amax, in ? fabsf(y[i]) : 0.f);
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        if (in) {
          float mul;
          const int p = e4m3_scale_exponent(amax, &mul);
          uint32_t c[2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            c[i] = pack_e4m3x4(y[4 * i] * mul, y[4 * i + 1] * mul, y[4 * i + 2] * mul,
                               y[4 * i + 3] * mul);
          *reinterpret_cast<uint2*>(a.codes + at) = make_uint2(c[0], c[1]);
          if ((v & 3) == 0) a.scales[at >> 5] = static_cast<uint8_t>(p + 127);
        }
      }
    }
  };
  if constexpr (IT > 0) {
#pragma unroll
    for (int k = 0; k < IT; ++k) finish(tg + k * a.group, s[k]);
  } else {
    // whole warps walk together: the shuffles of the codes need every lane
    for (int v0 = 0; v0 < nv; v0 += a.group) {
      const int v = v0 + tg;
      if (live && v < nv) load_s(v, s[0]);
      finish(v, s[0]);
    }
  }
}

template <int V, int IT>
void launch_types(const NormArgs& a, int x_f32, int res, int grid, int threads,
                  cudaStream_t stream) {
  if (x_f32) {
    if (res == 0) norm_kernel<V, IT, true, 0><<<grid, threads, 0, stream>>>(a);
    else if (res == 1) norm_kernel<V, IT, true, 1><<<grid, threads, 0, stream>>>(a);
    else norm_kernel<V, IT, true, 2><<<grid, threads, 0, stream>>>(a);
  } else {
    if (res == 0) norm_kernel<V, IT, false, 0><<<grid, threads, 0, stream>>>(a);
    else if (res == 1) norm_kernel<V, IT, false, 1><<<grid, threads, 0, stream>>>(a);
    else norm_kernel<V, IT, false, 2><<<grid, threads, 0, stream>>>(a);
  }
}

}  // namespace

int launch_add_rms_norm(const void* x, int x_f32, const void* res, int res_f32, const void* w,
                        int w_f32, float eps, int T, int H, void* res_out, void* y,
                        uint8_t* codes, uint8_t* scales, bool vec, cudaStream_t stream) {
  NormArgs a{};
  a.x = x;
  a.res = res;
  a.w = w;
  a.res_out = res_out;
  a.y = static_cast<__nv_bfloat16*>(y);
  a.codes = codes;
  a.scales = scales;
  a.eps = eps;
  a.T = T;
  a.H = H;
  a.w_f32 = w_f32;
  const int r = res ? (res_f32 ? 2 : 1) : 0;
  const int V = vec ? 8 : 1;
  const int nv = H / V;
  // threads of a row: at most two 16-byte (eight scalar) accesses a thread
  const int per = vec ? 2 : 8;
  int group = ((nv + per - 1) / per + 31) / 32 * 32;
  if (group > 1024) group = 1024;
  a.group = group;
  const int rows = group >= 256 ? 1 : 256 / group;
  const int grid = (T + rows - 1) / rows;
  const int threads = rows * group;
  if (vec) {
    if (nv <= 2 * group) launch_types<8, 2>(a, x_f32, r, grid, threads, stream);
    else if (nv <= 4 * group) launch_types<8, 4>(a, x_f32, r, grid, threads, stream);
    else launch_types<8, 0>(a, x_f32, r, grid, threads, stream);
  } else {
    if (nv <= 8 * group) launch_types<1, 8>(a, x_f32, r, grid, threads, stream);
    else launch_types<1, 0>(a, x_f32, r, grid, threads, stream);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace moe
