// Residual addition + RMS norm + FP8 rows with a scale per 128 values.
//
// "MiniMax-M3.1-Flash Day-0 対応" (aisoku.org), section "最適化と数値": the norm
// in front of the fused projection; the pages give no formula. Per row of W
// values, in fp32:
//   h = x + r,   y = h / sqrt(mean(h^2) + eps) * w   (y = h without a weight),
//   per 128 values: s = max|y| / 448, code = E4M3_RNE_satfinite(y / s).
// The sum h is what the norm sees, unrounded; the residual stream receives it
// rounded once to its own type.
//
// One CTA per row, the row in registers (8 values per thread and pass), so that
// every value is read once and written once: the mean takes one CTA barrier, a
// scale's maximum four shuffles among the 16 lanes that hold its group. What
// bounds it is bytes for many rows and the chain load - sum - barrier - store for
// few.
#include <cstring>

#include "msa_internal.h"

namespace msa {

constexpr int kScaleGroup = 128;                       // values per scale
constexpr float kE4m3Max = 448.f;

struct NormParams {
  const uint16_t* x;
  const void* residual;
  void* residual_out;
  const float* weight;
  uint16_t* out;
  uint8_t* codes;
  float* scales;
  int64_t x_stride;
  int width;
  float eps;
};

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum over the CTA, the same bits for every thread.
__device__ __forceinline__ float cta_sum(float v, float* warp_sums) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
  __syncthreads();
  v = static_cast<int>(threadIdx.x & 31) < warps ? warp_sums[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// kRes: 0 no residual, 1 bf16, 2 fp32. kVpt: passes of 8 values per thread.
template <int kVpt, int kRes>
__global__ void __launch_bounds__(kVpt <= 2 ? 1024 : 256) add_norm_quant_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sums[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = blockIdx.x;
  const int chunks = p.width / 8;
  float h[kVpt][8];
#pragma unroll
  for (int v = 0; v < kVpt; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    if (c < chunks) {
      const uint4 a = *reinterpret_cast<const uint4*>(p.x + row * p.x_stride + 8 * c);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[v][2 * i] = bf16_bits_to_f32(w[i] & 0xFFFF);
        h[v][2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
      }
      const int64_t at = row * p.width + 8 * c;
      if (kRes == 1) {
        const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.residual) + at);
        const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[v][2 * i] += bf16_bits_to_f32(u[i] & 0xFFFF);
          h[v][2 * i + 1] += bf16_bits_to_f32(u[i] >> 16);
        }
      } else if (kRes == 2) {
        const float4* b = reinterpret_cast<const float4*>(static_cast<const float*>(p.residual) + at);
        const float4 b0 = b[0], b1 = b[1];
        h[v][0] += b0.x; h[v][1] += b0.y; h[v][2] += b0.z; h[v][3] += b0.w;
        h[v][4] += b1.x; h[v][5] += b1.y; h[v][6] += b1.z; h[v][7] += b1.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = 0.f;
    }
  }
  if (kRes != 0 && p.residual_out != nullptr) {
#pragma unroll
    for (int v = 0; v < kVpt; ++v) {
      const int c = v * blockDim.x + threadIdx.x;
      if (c >= chunks) continue;
      const int64_t at = row * p.width + 8 * c;
      if (kRes == 1) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.residual_out) + at) =
            make_uint4(pack_bf16x2(h[v][0], h[v][1]), pack_bf16x2(h[v][2], h[v][3]), pack_bf16x2(h[v][4], h[v][5]),
                       pack_bf16x2(h[v][6], h[v][7]));
      } else {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.residual_out) + at);
        d[0] = make_float4(h[v][0], h[v][1], h[v][2], h[v][3]);
        d[1] = make_float4(h[v][4], h[v][5], h[v][6], h[v][7]);
      }
    }
  }

  if (p.weight != nullptr) {
    auto squares = [&](float f) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int v = 0; v < kVpt; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = h[v][i] * f;
          s[i & 1] = fmaf(t, t, s[i & 1]);
        }
      return s[0] + s[1];
    };
    const float inv_w = 1.f / static_cast<float>(p.width);
    float ms = cta_sum(squares(1.f), sums[0]) * inv_w;
    // Squares that leave fp32's range: the same with values scaled by a power of two, f h / sqrt(mean((f h)^2) + f^2 eps).
    // (A NaN takes this way too, and stays one.)
    float f = 1.f;
    if (!(ms <= 0x1p120f)) f = 0x1p-80f;
    else if (ms + p.eps < 0x1p-100f) f = 0x1p80f;
    if (f != 1.f) ms = cta_sum(squares(f), sums[1]) * inv_w;
    const float rinv = __fdiv_rn(1.f, __fsqrt_rn(ms + p.eps * f * f));
#pragma unroll
    for (int v = 0; v < kVpt; ++v) {
      const int c = v * blockDim.x + threadIdx.x;
      if (c >= chunks) continue;
      const float4* wv = reinterpret_cast<const float4*>(p.weight + 8 * c);
      const float4 w0 = wv[0], w1 = wv[1];
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * f * rinv * w[i];
    }
  }

#pragma unroll
  for (int v = 0; v < kVpt; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    const bool live = c < chunks;
    const int64_t at = row * p.width + 8 * c;
    if (p.out != nullptr && live)
      *reinterpret_cast<uint4*>(p.out + at) =
          make_uint4(pack_bf16x2(h[v][0], h[v][1]), pack_bf16x2(h[v][2], h[v][3]), pack_bf16x2(h[v][4], h[v][5]),
                     pack_bf16x2(h[v][6], h[v][7]));
    if (p.codes != nullptr) {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) a = max_nan(a, fabsf(h[v][i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
      const float s = __fdiv_rn(a, kE4m3Max);
      uint2 code = make_uint2(0u, 0u);
      if (s != 0.f) {
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = f32x2_to_e4m3x2(__fdiv_rn(h[v][2 * i], s), __fdiv_rn(h[v][2 * i + 1], s));
        code = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      }
      if (live) {
        *reinterpret_cast<uint2*>(p.codes + at) = code;
        if ((c & 15) == 0) p.scales[row * ((p.width + kScaleGroup - 1) / kScaleGroup) + c / 16] = s;
      }
    }
  }
}

template <int kVpt>
static cudaError_t launch_vpt(const NormParams& p, int res, int rows, int threads, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(rows)), block(static_cast<unsigned>(threads));
  if (res == 0) return launch_pdl(add_norm_quant_kernel<kVpt, 0>, grid, block, 0, stream, p);
  if (res == 1) return launch_pdl(add_norm_quant_kernel<kVpt, 1>, grid, block, 0, stream, p);
  return launch_pdl(add_norm_quant_kernel<kVpt, 2>, grid, block, 0, stream, p);
}

cudaError_t launch_add_norm_quant(const NormArgs& a, cudaStream_t stream, DispatchRecord* rec) {
  NormParams p;
  memset(&p, 0, sizeof(p));
  p.x = static_cast<const uint16_t*>(a.x);
  p.residual = a.residual;
  p.residual_out = a.residual_out;
  p.weight = a.weight;
  p.out = static_cast<uint16_t*>(a.out);
  p.codes = static_cast<uint8_t*>(a.codes);
  p.scales = a.scales;
  p.x_stride = a.x_stride;
  p.width = a.width;
  p.eps = a.eps;
  const int chunks = a.width / 8;
  const int res = a.residual == nullptr ? 0 : a.residual_f32 ? 2 : 1;
  // Passes per thread: two at most for few rows (all the SM's threads on a row's latency), more for many.
  const bool few = a.rows <= 2 * device_sm_count();
  int vpt = 1;
  while ((chunks + vpt - 1) / vpt > (few ? 1024 : 256) && vpt < 8) vpt *= 2;
  const int threads = ((chunks + vpt - 1) / vpt + 31) / 32 * 32;
  cudaError_t err;
  if (vpt == 1) err = launch_vpt<1>(p, res, a.rows, threads, stream);
  else if (vpt == 2) err = launch_vpt<2>(p, res, a.rows, threads, stream);
  else if (vpt == 4) err = launch_vpt<4>(p, res, a.rows, threads, stream);
  else err = launch_vpt<8>(p, res, a.rows, threads, stream);
  if (err != cudaSuccess) return err;
  rec->set("add_norm_quant%s%s%s%s grid=%d block=%d passes=%d", res == 0 ? "" : res == 1 ? " +bf16" : " +f32",
           a.weight ? " norm" : "", a.out ? " bf16" : "", a.codes ? " fp8" : "", a.rows, threads, vpt);
  return cudaGetLastError();
}

}  // namespace msa
