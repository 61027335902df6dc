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
// A CTA has a row at a time, in registers (8 values per thread and pass), so that
// every value is read once and written once: the mean takes one CTA barrier, a
// scale's maximum four shuffles among the 16 lanes that hold its group. What
// bounds it is bytes for many rows and the chain load - sum - barrier - store for
// few (64 x 4,096: 2.9 us).
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

// Eight values of x, as loaded, plus those of the residual (kRes: 0 none, 1 bf16, 2 fp32).
template <int kRes>
__device__ __forceinline__ void sum8(const uint4& x, const uint4& r0, const uint4& r1, float (&h)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w}, u[4] = {r0.x, r0.y, r0.z, r0.w}, v[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFF);
    h[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
    if (kRes == 1) {
      h[2 * i] += bf16_bits_to_f32(u[i] & 0xFFFF);
      h[2 * i + 1] += bf16_bits_to_f32(u[i] >> 16);
    }
  }
  if (kRes == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] += __uint_as_float(u[i]);
      h[4 + i] += __uint_as_float(v[i]);
    }
  }
}

__device__ __forceinline__ uint4 bf16x8(const float (&h)[8]) {
  return make_uint4(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]), pack_bf16x2(h[4], h[5]), pack_bf16x2(h[6], h[7]));
}

// The residual stream's new values.
template <int kRes>
__device__ __forceinline__ void store_residual(const NormParams& p, int64_t at, const float (&h)[8]) {
  if (kRes == 1) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.residual_out) + at) = bf16x8(h);
  } else if (kRes == 2) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.residual_out) + at);
    d[0] = make_float4(h[0], h[1], h[2], h[3]);
    d[1] = make_float4(h[4], h[5], h[6], h[7]);
  }
}

// The factors (f, 1 / sqrt(mean((f h)^2) + f^2 eps)) of a row; every thread of the CTA calls it. `sums` has room for two
// sums of 32 warps.
template <int kVpt>
__device__ __forceinline__ float2 row_factors(const NormParams& p, const float (&h)[kVpt][8], float (*sums)[32]) {
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
  // Squares that leave fp32's range: the same with values scaled by a power of two. (A NaN takes this way too, and stays
  // one.)
  float f = 1.f;
  if (!(ms <= 0x1p120f)) f = 0x1p-80f;
  else if (ms + p.eps < 0x1p-100f) f = 0x1p80f;
  if (f != 1.f) ms = cta_sum(squares(f), sums[1]) * inv_w;
  return make_float2(f, __fdiv_rn(1.f, __fsqrt_rn(ms + p.eps * f * f)));
}

// Eight results of chunk c; the 16 lanes of a group call it together, `live` ones store.
__device__ __forceinline__ void store_results(const NormParams& p, int64_t row, int c, bool live, float (&y)[8]) {
  const int64_t at = row * p.width + 8 * c;
  if (p.out != nullptr && live) *reinterpret_cast<uint4*>(p.out + at) = bf16x8(y);
  if (p.codes == nullptr) return;
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max_nan(a, fabsf(y[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
  const float s = __fdiv_rn(a, kE4m3Max);
  uint2 code = make_uint2(0u, 0u);
  if (s != 0.f) {
    // The quotients' codes with one division per group: the reciprocal is held in two parts, so that a product is the
    // quotient within 2^-46 in front of its one rounding, which leaves every code the quotient's (with one exception, a
    // divisor a step below a power of two, where the second part is a little nearer zero). Scales far from one are moved by a
    // power of two, so that the second part keeps its bits. 8,191 x 4,096: 41.4 us; a division per value 51.0,
    // the product with a rounded reciprocal, whose codes differ at borders, 40.5.
    const float up = s < 0x1p-64f ? 0x1p100f : s > 0x1p64f ? 0x1p-100f : 1.f;
    const float d = s * up, inv = __fdiv_rn(1.f, d);
    float rest = inv == 0.f ? 0.f : fmaf(-d, inv, 1.f) * inv;
    if ((__float_as_uint(d) & 0x7FFFFFu) == 0x7FFFFFu) rest *= 1.f - 0x1p-22f;
    if (up != 1.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= up;
    }
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float c0, c1;
      asm("{\n .reg .b64 y, v, r, t;\n mov.b64 y, {%2, %3};\n mov.b64 v, {%4, %4};\n mov.b64 r, {%5, %5};\n"
          " mul.rn.f32x2 t, y, r;\n fma.rn.f32x2 t, y, v, t;\n mov.b64 {%0, %1}, t;\n}"
          : "=f"(c0), "=f"(c1) : "f"(y[2 * i]), "f"(y[2 * i + 1]), "f"(inv), "f"(rest));
      q[i] = f32x2_to_e4m3x2(c0, c1);
    }
    code = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
  }
  if (!live) return;
  *reinterpret_cast<uint2*>(p.codes + at) = code;
  if ((c & 15) == 0) p.scales[row * ((p.width + kScaleGroup - 1) / kScaleGroup) + c / 16] = s;
}

__device__ __forceinline__ void weights8(const NormParams& p, int c, float (&w)[8]) {
  const float4* wv = reinterpret_cast<const float4*>(p.weight + 8 * c);
  const float4 w0 = wv[0], w1 = wv[1];
  w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
  w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
}

// Few rows: a CTA each, all of its threads on the row's latency. kVpt: passes of 8 values per thread.
template <int kVpt, int kRes>
__global__ void __launch_bounds__(1024) add_norm_quant_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sums[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = blockIdx.x;
  const int chunks = p.width / 8;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  float h[kVpt][8];
#pragma unroll
  for (int v = 0; v < kVpt; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    uint4 x = none, r0 = none, r1 = none;
    if (c < chunks) {
      const int64_t at = row * p.width + 8 * c;
      x = *reinterpret_cast<const uint4*>(p.x + row * p.x_stride + 8 * c);
      if (kRes == 1) r0 = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.residual) + at);
      if (kRes == 2) {
        const uint4* r = reinterpret_cast<const uint4*>(static_cast<const float*>(p.residual) + at);
        r0 = r[0];
        r1 = r[1];
      }
    }
    sum8<kRes>(x, r0, r1, h[v]);
  }
  if (kRes != 0 && p.residual_out != nullptr) {
#pragma unroll
    for (int v = 0; v < kVpt; ++v) {
      const int c = v * blockDim.x + threadIdx.x;
      if (c < chunks) store_residual<kRes>(p, row * p.width + 8 * c, h[v]);
    }
  }
  if (p.weight != nullptr) {
    const float2 f = row_factors<kVpt>(p, h, sums);
#pragma unroll
    for (int v = 0; v < kVpt; ++v) {
      const int c = v * blockDim.x + threadIdx.x;
      if (c >= chunks) continue;
      float w[8];
      weights8(p, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * f.x * f.y * w[i];
    }
  }
#pragma unroll
  for (int v = 0; v < kVpt; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    store_results(p, row, c, c < chunks, h[v]);
  }
}

// Many rows: CTAs that stay, rows strided over them, the weight in registers, and the next two rows on their way into a
// ring in shared memory of which every thread has its own 16-byte places: it waits for its own copies only. 8,191 rows of
// 4,096 / 8,192 / 16,384 values, bf16 residual, FP8 out: 41.4 / 76.4 / 143.7 us (84 / 91 / 97 % of a copy's rate), a CTA
// per row 45.1 / 98.5 / 204.1.
constexpr int kRingVpt = 2, kRingRows = 3;

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int kRes, int kMost>
__global__ void __launch_bounds__(kMost, 1024 / kMost) add_norm_quant_ring_kernel(const __grid_constant__ NormParams p, int rows) {
  constexpr int kVpt = kRingVpt, kParts = 1 + kRes;     // 16-byte pieces of 8 values: x, residual
  extern __shared__ uint4 ring[];
  __shared__ float sums[2][2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int chunks = p.width / 8;
  auto place = [&](int slot, int part, int v) { return ((slot * kParts + part) * kVpt + v) * blockDim.x + threadIdx.x; };
  auto fetch = [&](int64_t row, int slot) {
    if (row < rows) {
#pragma unroll
      for (int v = 0; v < kVpt; ++v) {
        const int c = v * blockDim.x + threadIdx.x;
        if (c >= chunks) continue;
        const int64_t at = row * p.width + 8 * c;
        copy16(smem_addr(&ring[place(slot, 0, v)]), p.x + row * p.x_stride + 8 * c);
        if (kRes == 1) copy16(smem_addr(&ring[place(slot, 1, v)]), static_cast<const uint16_t*>(p.residual) + at);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kRingRows - 1; ++s) fetch(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
  float w[kVpt][8];
#pragma unroll
  for (int v = 0; v < kVpt; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[v][i] = 0.f;         // behind the row: its lanes take part in the last group's maximum
    if (p.weight != nullptr && c < chunks) weights8(p, c, w[v]);
  }
  int slot = 0, turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    fetch(row + static_cast<int64_t>(kRingRows - 1) * gridDim.x, slot == 0 ? kRingRows - 1 : slot - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kRingRows - 1) : "memory");
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    float h[kVpt][8];
#pragma unroll
    for (int v = 0; v < kVpt; ++v) {
      const int c = v * blockDim.x + threadIdx.x;
      const bool live = c < chunks;
      sum8<kRes>(live ? ring[place(slot, 0, v)] : none, kRes != 0 && live ? ring[place(slot, kRes, v)] : none, none, h[v]);
      if (kRes != 0 && p.residual_out != nullptr && live) store_residual<kRes>(p, row * p.width + 8 * c, h[v]);
    }
    if (p.weight != nullptr) {
      const float2 f = row_factors<kVpt>(p, h, sums[turn]);
#pragma unroll
      for (int v = 0; v < kVpt; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * f.x * f.y * w[v][i];
    }
#pragma unroll
    for (int v = 0; v < kVpt; ++v) {
      const int c = v * blockDim.x + threadIdx.x;
      store_results(p, row, c, c < chunks, h[v]);
    }
    if (++slot == kRingRows) slot = 0;
    turn ^= 1;                                         // the sums of the row before may still be read
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int kRes>
static cudaError_t launch_few(const NormParams& p, int vpt, int rows, int threads, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(rows)), block(static_cast<unsigned>(threads));
  return vpt == 1 ? launch_pdl(add_norm_quant_kernel<1, kRes>, grid, block, 0, stream, p)
                  : launch_pdl(add_norm_quant_kernel<2, kRes>, grid, block, 0, stream, p);
}
template <int kRes, int kMost>
static cudaError_t launch_ring(const NormParams& p, int rows, int threads, int sms, int& grid, cudaStream_t stream) {
  constexpr size_t per_thread = kRingRows * (1 + kRes) * kRingVpt * 16;
  const size_t smem = threads * per_thread;
  const int room = static_cast<int>((220u << 10) / (smem + 2048)), ctas = room < 1024 / threads ? room : 1024 / threads;
  grid = rows < sms * ctas ? rows : sms * ctas;
  // The most that any width takes: the limit is the function's, and another thread's launch may come in between.
  const cudaError_t err = cudaFuncSetAttribute(add_norm_quant_ring_kernel<kRes, kMost>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kMost * per_thread));
  if (err != cudaSuccess) return err;
  return launch_pdl(add_norm_quant_ring_kernel<kRes, kMost>, dim3(static_cast<unsigned>(grid)),
                    dim3(static_cast<unsigned>(threads)), smem, stream, p, rows);
}
template <int kRes>
static cudaError_t launch_many(const NormParams& p, int rows, int threads, int sms, int& grid, cudaStream_t stream) {
  return threads <= 256   ? launch_ring<kRes, 256>(p, rows, threads, sms, grid, stream)
         : threads <= 512 ? launch_ring<kRes, 512>(p, rows, threads, sms, grid, stream)
                          : launch_ring<kRes, 1024>(p, rows, threads, sms, grid, stream);
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
  const int sms = device_sm_count();
  // The ring from 2^23 values in rows of at least 4,096. Ring and CTA per row, us, bf16 residual: 2,432 x 4,096 16.1 and 16.1,
  // 1,216 x 8,192 15.8 and 18.0, 700 x 12,288 14.8 and 19.6; 700 x 8,192 12.2 and 11.9, 30,000 x 1,024 41.8 and 39.5. Below
  // 4,096 the two lie close together, by the number of values: 2^23 of them in rows of 2,048 / 2,560 / 3,584 / 4,080 14.7 and
  // 13.5 / 14.9 and 13.8 / 14.7 and 14.4 / 15.4 and 14.2, 2^25 42.1 and 43.6 / 44.9 and 44.5 / 43.3 and 46.5 / 42.4 and 45.9
  // (without a residual 24.8 and 24.0 / 26.4 and 24.6 / 25.1 and 25.6 / 24.3 and 24.9). An fp32 residual, 32 bytes per
  // thread, is better loaded than copied: 8,191 x 4,096 57.1 us, by a ring 76.0.
  const bool many = res != 2 && a.width >= 4096 && static_cast<int64_t>(a.rows) * a.width >= (1ll << 23);
  const int vpt = many ? kRingVpt : chunks > 1024 ? 2 : 1;
  const int threads = ((chunks + vpt - 1) / vpt + 31) / 32 * 32;
  int grid = a.rows;
  cudaError_t err;
  if (many)
    err = res == 0 ? launch_many<0>(p, a.rows, threads, sms, grid, stream) : launch_many<1>(p, a.rows, threads, sms, grid, stream);
  else
    err = res == 0 ? launch_few<0>(p, vpt, a.rows, threads, stream)
        : res == 1 ? launch_few<1>(p, vpt, a.rows, threads, stream) : launch_few<2>(p, vpt, a.rows, threads, stream);
  if (err != cudaSuccess) return err;
  rec->set("add_norm_quant%s%s%s%s%s grid=%d block=%d passes=%d", res == 0 ? "" : res == 1 ? " +bf16" : " +f32",
           a.weight ? " norm" : "", a.out ? " bf16" : "", a.codes ? " fp8" : "", many ? " ring" : "", grid, threads, vpt);
  return cudaGetLastError();
}

}  // namespace msa
