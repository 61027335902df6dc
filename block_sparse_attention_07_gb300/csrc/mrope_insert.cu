// QK-norm + rotary embedding on several axes + cache insert.
//
// "MiniMax M3 vLLM サポート：…" (agentlenshq.com): image and video input, and in
// section "カーネル融合" the fusion of QK-norm, rotary embedding and the K/V
// insert. Per (token, head) row of 128 values x:
//   y = x / sqrt(mean(x^2) + eps) * w,
//   (y_i, y_{i+64}) <- (y_i cos phi - y_{i+64} sin phi, y_i sin phi + y_{i+64} cos phi),
//   phi_i = positions[axis(i), t] * theta^(-2i/128),
// rounded to bf16; keys and V then go through the cache's quantiser.
//
// A row belongs to 8 lanes; lane l holds dims 8l .. 8l+7 and 64 + 8l .. 64 + 8l+7
// (two 16-byte loads), so both dims of its 8 pairs are in its registers: the
// rotation needs no exchange and the norm three shuffles for four rows of a
// warp. A warp takes groups of four rows of one token; `parts` warps share a
// token's.
//
// What bounds it is the rows' bytes, and what it takes to reach that rate is
// bytes in flight: each warp has its next six groups of queries (1 KB each,
// contiguous) on their way to its own part of shared memory by bulk copies,
// and does the keys and values while the first of them arrive. 8,191 tokens,
// 64 + 4 + 4 heads, FP8 cache: 51.3 us, 5.7 TB/s (85 % of a copy's rate); with
// loads into registers, two groups ahead, 59.2 us. 64 tokens, bf16 cache: 3.9
// us. With fewer heads a warp has fewer groups than its part
// holds, and what comes before the first of them (position, sines, slot, weights)
// shows: 32 + 2 + 2 heads 34.6 us (63 % of a copy's rate), 16 + 1 + 1 29.9 (37 %).
//
// Phases: theta^(-2i/128) / 2 pi is held as a 64-bit fraction of a turn, so that
// position times it, modulo one turn, is one integer product. The fraction comes
// from doubles, 2^-51 relative: a phase is off by at most 2^-22 of a turn at the
// largest 32-bit position.
#include <cmath>
#include <cstring>

#include "rope_rows.cuh"

namespace msa {

constexpr int kMropeWarps = 2, kMropeCtas = 14;   // warps per CTA, CTAs per SM (72 registers); 8,191 tokens 51.4 us, 4 x 7 52.0, 8 x 3 54.3
constexpr int kRingSlots = 6;                     // passes of a warp's queries in flight
constexpr uint32_t kPassBytes = 4 * kDim * 2;

struct MropeParams {
  InsertParams ins;
  const uint16_t* q;           // bf16 [T, H, D]
  const uint16_t* idx_q;       // bf16 [T, I, D] or null
  uint16_t* q_out;
  uint16_t* idx_q_out;
  const int32_t* positions;    // [A] rows, pos_stride apart
  int64_t pos_stride;
  const float* wq;
  const float* wk;
  const float* wiq;
  const float* wik;
  float eps;
  int H, I;
  int parts;                   // warps per token
  alignas(16) uint64_t turn[kDim / 2];     // theta^(-2i/D) / 2 pi, in units of 2^-64 of a turn
  alignas(16) uint8_t axis[kDim / 2];
};

// One half (8 values) of an NVFP4 row: a 16-value group belongs to two lanes.
__device__ __forceinline__ void store_fp4_half(const float* x, uint8_t* codes, uint8_t* scales, float g, int l, int half,
                                               bool live) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  const float sb_in = __fdiv_rn(__fdiv_rn(a, 6.0f), g);
  const uint8_t sb = static_cast<uint8_t>(f32x2_to_e4m3x2(sb_in, 0.f) & 0xFF);
  const float denom = __fmul_rn(e4m3_to_f32(sb), g);
  uint32_t packed = 0;
  if (denom > 0.f) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], denom);
    packed = f32x8_to_e2m1x8(y);
  }
  if (!live) return;
  *reinterpret_cast<uint32_t*>(codes + 32 * half + 4 * l) = packed;
  if ((l & 1) == 0) scales[4 * half + (l >> 1)] = sb;
}

// The row writers take the row as two halves of 8 values per lane; every lane of
// the warp calls them (the group maxima are warp shuffles), `live` lanes store.
__device__ __forceinline__ void store_kv16(const InsertParams& p, bool is_v, int64_t row, const float (&x)[16], int l,
                                           bool live) {
  void* base = is_v ? p.v : p.k;
  const float s = is_v ? p.v_global : p.k_global;
  if (p.kv_nvfp4) {
    uint8_t* codes = static_cast<uint8_t*>(base) + row * (kDim / 2);
    uint8_t* scales = (is_v ? p.v_scale : p.k_scale) + row * (kDim / 16);
    store_fp4_half(x, codes, scales, s, l, 0, live);
    store_fp4_half(x + 8, codes, scales, s, l, 1, live);
  } else if (live && p.kv_fp8) {
    uint8_t* d = static_cast<uint8_t*>(base) + row * kDim + 8 * l;
    *reinterpret_cast<uint2*>(d) = e4m3x8(x, s);
    *reinterpret_cast<uint2*>(d + 64) = e4m3x8(x + 8, s);
  } else if (live) {
    uint16_t* d = static_cast<uint16_t*>(base) + row * kDim + 8 * l;
    *reinterpret_cast<uint4*>(d) = pack8(x);
    *reinterpret_cast<uint4*>(d + 64) = pack8(x + 8);
  }
}

__device__ __forceinline__ void store_idx16(const InsertParams& p, int64_t row, const float (&x)[16], int l, bool live) {
  if (p.idx_fp4) {
    uint8_t* codes = static_cast<uint8_t*>(p.idx_keys) + row * (kDim / 2);
    uint8_t* scales = p.idx_block_scale + row * (kDim / 16);
    store_fp4_half(x, codes, scales, p.idx_global, l, 0, live);
    store_fp4_half(x + 8, codes, scales, p.idx_global, l, 1, live);
    return;
  }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  const float s = __fdiv_rn(a, 448.0f);
  if (!live) return;
  uint8_t* d = static_cast<uint8_t*>(p.idx_keys) + row * kDim + 8 * l;
  *reinterpret_cast<uint2*>(d) = s > 0.f ? e4m3x8(x, s) : make_uint2(0u, 0u);
  *reinterpret_cast<uint2*>(d + 64) = s > 0.f ? e4m3x8(x + 8, s) : make_uint2(0u, 0u);
  if (l == 0) p.idx_scale[row] = s;
}

template <bool kFew>                      // all warps begin at one time
__global__ void __launch_bounds__(32 * kMropeWarps, kMropeCtas) qk_norm_mrope_insert_kernel(const __grid_constant__ MropeParams pp) {
  __shared__ alignas(128) uint8_t ring_rows[kMropeWarps * kRingSlots * kPassBytes];
  __shared__ uint64_t ring_bars[kMropeWarps * kRingSlots];
  griddep_launch_dependents();
  griddep_wait();
  const InsertParams& p = pp.ins;
  const int lane = threadIdx.x & 31, l = lane & 7;
  const int nq = pp.H, nk = p.G, ni = pp.idx_q != nullptr ? pp.I : 0;
  const int rows = nq + 2 * nk + 2 * ni;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * kMropeWarps + (threadIdx.x >> 5);
  const int64_t t = wid / pp.parts;
  const int part = static_cast<int>(wid - t * pp.parts);
  if (t >= p.T) return;

  const int q_passes = nq / 4;
  const uint32_t rows_at = smem_addr(ring_rows) + (threadIdx.x >> 5) * kRingSlots * kPassBytes;
  const uint32_t bars_at = smem_addr(ring_bars) + (threadIdx.x >> 5) * kRingSlots * 8;
  uint64_t policy = 0;
  auto fetch = [&](int pass, int slot) {
    mbar_arrive_expect_tx(bars_at + 8 * slot, kPassBytes);
    bulk_g2s(rows_at + slot * kPassBytes, pp.q + (t * nq + 4 * pass) * kDim, kPassBytes, bars_at + 8 * slot, policy);
  };
  if (lane == 0) {
    for (int i = 0; i < kRingSlots; ++i) mbar_init(bars_at + 8 * i, 1);
    fence_mbar_init();
    policy = l2_evict_first_policy();
    for (int i = 0; i < kRingSlots && part + i * pp.parts < q_passes; ++i) fetch(part + i * pp.parts, i);
  }
  __syncwarp();

  // cos and sin of the lane's 8 pairs (8 l + i): each is computed by one of the
  // four lanes that use it
  float cs[8], sn[8];
  {
    // Axes and frequencies of two pairs. Read as parameters, lanes at 32 places take 32 turns, which shows where all warps
    // begin at one time: so through addresses, as memory (64 tokens, calls in a row: 6.6 -> 3.9 us, 512 9.8 -> 7.9). Where
    // warps follow one another it does not, and spreads them (8,191 tokens: 52.0 as memory, 51.0 as parameters).
    const int i = 8 * l + 2 * (lane >> 3);
    uchar2 ax = make_uchar2(0, 0);
    ulonglong2 two = make_ulonglong2(0, 0);
    if (kFew) {
      const uint64_t* turns = pp.turn;
      const uint8_t* axes = pp.axis;
      asm volatile("" : "+l"(turns), "+l"(axes));
      ax = *reinterpret_cast<const uchar2*>(axes + i);
      two = *reinterpret_cast<const ulonglong2*>(turns + i);
    }
    float c2[2], s2[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t pos = pp.positions[(!kFew ? pp.axis[i + e] : e ? ax.y : ax.x) * pp.pos_stride + t];
      const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(pos) * (!kFew ? pp.turn[i + e] : e ? two.y : two.x));   // modulo one turn
      sincospif(static_cast<float>(turn) * 0x1p-63f, &s2[e], &c2[e]);                        // half turns in [-1, 1]
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = __shfl_sync(0xffffffffu, c2[i & 1], 8 * (i >> 1) + l);
      sn[i] = __shfl_sync(0xffffffffu, s2[i & 1], 8 * (i >> 1) + l);
    }
  }
  const int64_t slot = p.slots[t];
  const int64_t page = slot / kBlock, off = slot % kBlock;
  const bool held = slot >= 0 && slot < p.num_slots;
  if (slot >= p.num_slots && part == 0 && lane == 0) set_flag(p.flags, MSA_FLAG_BAD_SLOT);

  auto weights = [&](const float* wv, float (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(wv + (i < 2 ? 8 * l + 4 * i : 64 + 8 * l + 4 * (i - 2)));
      w[4 * i] = f.x; w[4 * i + 1] = f.y; w[4 * i + 2] = f.z; w[4 * i + 3] = f.w;
    }
  };
  // 1 / sqrt(mean of the row's squares + eps), by its 8 lanes
  auto row_scale = [&](const float (&x)[16]) {
    float s2[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) s2[i & 1] = fmaf(x[i], x[i], s2[i & 1]);
    float ss = s2[0] + s2[1];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    return rsqrtf(fmaf(ss, 1.0f / kDim, pp.eps));
  };

  // While the queries are on their way, the rows behind them: any last queries, keys, values, index rows
  int pass = part;
  if (pass < q_passes) pass += (q_passes - pass + pp.parts - 1) / pp.parts * pp.parts;
  for (; 4 * pass < rows; pass += pp.parts) {
    const int r = 4 * pass + (lane >> 3);
    const bool live = r < rows;
    // kind 0 q, 1 k, 2 v, 3 index q, 4 index k
    int kind = 0, h = live ? r : 0;
    const uint16_t* src = pp.q + (t * nq + h) * kDim;
    const float* wv = pp.wq;
    if (live && r >= nq) {
      h = r - nq;
      if (h < nk) { kind = 1; src = p.k_new + (t * nk + h) * kDim; wv = pp.wk; }
      else if ((h -= nk) < nk) { kind = 2; src = p.v_new + (t * nk + h) * kDim; }
      else if ((h -= nk) < ni) { kind = 3; src = pp.idx_q + (t * ni + h) * kDim; wv = pp.wiq; }
      else { h -= ni; kind = 4; src = static_cast<const uint16_t*>(p.idx_new) + (t * ni + h) * kDim; wv = pp.wik; }
    }
    float x[16];
    unpack8(*reinterpret_cast<const uint4*>(src + 8 * l), x);
    unpack8(*reinterpret_cast<const uint4*>(src + 64 + 8 * l), x + 8);
    const float rinv = row_scale(x);
    if (kind != 2) {
      float w[16];
      weights(wv, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // rounded to bf16 here: what the outputs hold and the caches quantise
        const float a = (x[i] * (w[i] * cs[i]) - x[8 + i] * (w[8 + i] * sn[i])) * rinv;
        const float b = (x[i] * (w[i] * sn[i]) + x[8 + i] * (w[8 + i] * cs[i])) * rinv;
        x[i] = bf16_bits_to_f32(static_cast<uint16_t>(pack_bf16x2(a, 0.f) & 0xFFFF));
        x[8 + i] = bf16_bits_to_f32(static_cast<uint16_t>(pack_bf16x2(b, 0.f) & 0xFFFF));
      }
    }
    if (live && (kind == 0 || kind == 3)) {
      uint16_t* dst = (kind == 0 ? pp.q_out + (t * nq + h) * kDim : pp.idx_q_out + (t * ni + h) * kDim) + 8 * l;
      *reinterpret_cast<uint4*>(dst) = pack8(x);
      *reinterpret_cast<uint4*>(dst + 64) = pack8(x + 8);
    }
    // the cache rows; the writers' shuffles take the whole warp
    const bool kv = kind == 1 || kind == 2;
    if (__any_sync(0xffffffffu, kv && live)) {
      const int64_t row = kv ? (page * nk + h) * kBlock + off : 0;
      store_kv16(p, kind == 2, row, x, l, kv && live && held);
    }
    if (__any_sync(0xffffffffu, kind == 4 && live)) {
      const int64_t row = kind == 4 ? (page * ni + h) * kBlock + off : 0;
      store_idx16(p, row, x, l, kind == 4 && live && held);
    }
  }

  // Most rows are queries, four at a time: with their weights folded into the cosines and sines a pair is four
  // products and two scalings.
  if (part >= q_passes) return;
  float wc[8], ws[8], vs[8], vc[8];
  {
    float w[16];
    weights(pp.wq, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      wc[i] = w[i] * cs[i]; ws[i] = w[i] * sn[i];
      vs[i] = w[8 + i] * sn[i]; vc[i] = w[8 + i] * cs[i];
    }
  }
  uint16_t* dst = pp.q_out + (t * nq + 4 * part + (lane >> 3)) * kDim + 8 * l;
  const int64_t hop = 4ll * pp.parts * kDim;
  auto rotate = [&](const uint4& lo, const uint4& hi) {
    float x[16], y[16];
    unpack8(lo, x);
    unpack8(hi, x + 8);
    const float rinv = row_scale(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = (x[i] * wc[i] - x[8 + i] * vs[i]) * rinv;
      y[8 + i] = (x[i] * ws[i] + x[8 + i] * vc[i]) * rinv;
    }
    *reinterpret_cast<uint4*>(dst) = pack8(y);
    *reinterpret_cast<uint4*>(dst + 64) = pack8(y + 8);
    dst += hop;
  };
  int buf = 0;
  uint32_t phase = 0;
  for (pass = part; pass < q_passes; pass += pp.parts) {
    if (__all_sync(0xffffffffu, mbar_wait(bars_at + 8 * buf, phase)) == 0) {
      // a copy that did not come in time; those behind it are waited for, so that none outlives the CTA
      if (lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
      for (int i = 1; i < kRingSlots && pass + i * pp.parts < q_passes; ++i) {
        if (++buf == kRingSlots) { buf = 0; phase ^= 1u; }
        mbar_wait(bars_at + 8 * buf, phase);
      }
      return;
    }
    const uint32_t at = rows_at + buf * kPassBytes + (lane >> 3) * (kDim * 2) + 16 * l;
    rotate(ld_shared16(at), ld_shared16(at + kDim));
    __syncwarp();                                    // the buffer has been read
    if (lane == 0 && pass + kRingSlots * pp.parts < q_passes) fetch(pass + kRingSlots * pp.parts, buf);
    if (++buf == kRingSlots) { buf = 0; phase ^= 1u; }
  }
}

cudaError_t launch_qk_norm_mrope_insert(const PrologueArgs& a, const msa_rope_axes_t& axes, int64_t pos_stride,
                                        cudaStream_t stream, DispatchRecord* rec) {
  MropeParams pp;
  memset(&pp, 0, sizeof(pp));
  pp.ins = make_insert_params(a.ins);
  pp.q = static_cast<const uint16_t*>(a.q);
  pp.idx_q = static_cast<const uint16_t*>(a.idx_q);
  pp.q_out = static_cast<uint16_t*>(a.q_out);
  pp.idx_q_out = static_cast<uint16_t*>(a.idx_q_out);
  pp.positions = a.positions;
  pp.pos_stride = pos_stride;
  pp.wq = a.wq; pp.wk = a.wk; pp.wiq = a.wiq; pp.wik = a.wik;
  pp.eps = a.eps;
  pp.H = a.H;
  pp.I = a.I;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  // theta^(-2i/128) as a product of two powers, i = 8 hi + lo: 16 powers instead of 64 on every call
  double hi[8], lo[8];
  for (int i = 0; i < 8; ++i) {
    hi[i] = pow(static_cast<double>(a.theta), -16.0 * i / kDim) / kTwoPi;
    lo[i] = pow(static_cast<double>(a.theta), -2.0 * i / kDim);
  }
  for (int i = 0; i < kDim / 2; ++i) {
    pp.turn[i] = static_cast<uint64_t>(hi[i >> 3] * lo[i & 7] * 0x1p64);
    pp.axis[i] = axes.axis[i];
  }
  const int rows = a.H + 2 * a.ins.G + (a.idx_q ? 2 * a.I : 0);
  const int passes = (rows + 3) / 4;
  // Warps per token: one once there are 64 tokens per SM (16,000 tokens 92.9 us, two 95.3), two below (4,096
  // tokens 28.6, one 31.0, three 31.2), more when there are few tokens (16 warps per SM: 1,024 tokens 11.5 us;
  // 32 per SM 14.9, 8 per SM 13.7). All with 64 + 4 + 4 heads: the rule counts tokens, not rows.
  const int64_t sms = device_sm_count();
  int64_t parts = a.ins.T >= 64 * sms ? 1 : (16 * sms + a.ins.T - 1) / a.ins.T;
  if (parts < 2 && a.ins.T < 64 * sms) parts = 2;
  if (parts > passes) parts = passes;
  pp.parts = static_cast<int>(parts);
  const int64_t grid = (a.ins.T * parts + kMropeWarps - 1) / kMropeWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const bool few = a.ins.T * parts <= kMropeWarps * kMropeCtas * sms;
  const cudaError_t err = launch_pdl(few ? qk_norm_mrope_insert_kernel<true> : qk_norm_mrope_insert_kernel<false>,
                                     dim3(static_cast<unsigned>(grid)), dim3(32 * kMropeWarps), 0, stream, pp);
  if (err != cudaSuccess) return err;
  rec->set("qk_norm_mrope_insert %s%s grid=%lld block=%d warps_per_token=%d heads=%d+%d+%d axes=%d",
           a.ins.kv_nvfp4 ? "nvfp4" : a.ins.kv_fp8 ? "fp8" : "bf16",
           a.idx_q ? (a.ins.idx_fp4 ? "+idx_nvfp4" : "+idx_fp8") : "", static_cast<long long>(grid), 32 * kMropeWarps,
           pp.parts, a.H, a.ins.G, a.idx_q ? a.I : 0, axes.num_axes);
  return cudaGetLastError();
}

}  // namespace msa
