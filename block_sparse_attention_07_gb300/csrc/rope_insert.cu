// Rotary forms + head norms + cache insert on packed projection rows.
//
// "MiniMax-M3.1-Flash Day-0 対応" (aisoku.org), section "最適化と数値": projection,
// norm, rotary embedding and K/V insert in a row; "MiniMax M3 vLLM サポート：…"
// (agentlenshq.com), sections "カーネル融合" and on the 1M-token context. The pages
// give no formulas. Per (token, head) row of 128 values x:
//   y = x / sqrt(mean(x^2) + eps) * w, or y = x without norm;
//   for i < R/2, (y_a, y_b) <- gain (y_a cos phi - y_b sin phi, y_a sin phi + y_b cos phi),
//   phi_i = position * freq_i, (a, b) = (i, i + R/2) or (2i, 2i + 1); dims >= R pass;
// rounded to bf16; keys, values and index keys then go through the cache's quantiser.
//
// A row belongs to 8 lanes of two 16-byte chunks each, chosen so that both dims of
// a pair are the lane's: in the half layout with n = R/16, lane l < n holds chunks
// l and n + l, the others chunks n + l and 8 + l, which pass; interleaved, chunks l
// and 8 + l. So the rotation needs no exchange and the norm three shuffles for four
// rows of a warp. The cache writers want 16 dims in a row (an NVFP4 scale's group):
// keys and values change places through 1 KB of shared memory per warp.
//
// Bound by the rows' bytes: as many as possible are kept in flight, the queries of
// a token (contiguous, whatever the token's stride) by bulk copies into a ring per
// warp, with keys and values done while the first of them arrive. 8,191 tokens, 64 +
// 4 + 4 heads, FP8 cache: 52.5 us, 5.6 TB/s (83 % of a copy's rate); 16,000 tokens
// 93.7 us (90 %); 64 tokens, bf16 cache: 4.0 us, of which 0.7 pass until a kernel may
// start and 0.5 each for positions and for rows. With fewer heads what
// comes before a warp's queries (position, sines, slot, keys) shows: 16 + 1 + 1 heads
// 20.3 us for 8,191 tokens (53 % of a copy's rate): a warp has one token, and four passes of queries behind that chain.
//
// Phases: freq / 2 pi modulo one is held as a 64-bit fraction of a turn, so that
// position times it, modulo one turn, is one integer product: 2^-53 relative to
// the frequency, 2^-24 of a turn at the largest 32-bit position and frequency 1.
#include <cmath>
#include <cstring>
#include <type_traits>

#include "rope_rows.cuh"

namespace msa {

constexpr int kRopeWarps = 1, kRopeCtas = 28;     // warps per CTA, CTAs per SM: 8,191 tokens 52.9 us, 2 x 14 54.7, 4 x 7 55.1
constexpr int kRopeSlots = 6;                     // groups of four queries in flight per warp
constexpr uint32_t kRopeGroup = 4 * kDim * 2;     // their bytes

struct RopeParams {
  InsertParams ins;            // caches and slots
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* idx_q;       // null: no index rows
  const uint16_t* idx_k;
  int64_t q_stride, k_stride, v_stride, iq_stride, ik_stride;      // elements between tokens
  uint16_t* q_out;             // [T, H, D]
  uint16_t* idx_q_out;         // [T, I, D]
  const int32_t* positions;
  const float* wq;             // null: no norm
  const float* wk;
  const float* wiq;
  const float* wik;
  float eps, gain;
  float low;                   // mean squares below it are too small beside eps
  int H, I, R;
  int parts;                   // warps per token
  alignas(16) uint64_t turn[kDim / 2];     // freq / 2 pi, in units of 2^-64 of a turn
};

__device__ __forceinline__ void st_shared16(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Eight E4M3 codes of eight values over s.
__device__ __forceinline__ uint2 codes8(const float* x, float s) { return e4m3x8(x, s); }

// Sixteen values -> E2M1 codes and their scale's E4M3 code.
__device__ __forceinline__ uint2 fp4_group(const float (&x)[16], float g, uint8_t& sb) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]));
  sb = static_cast<uint8_t>(f32x2_to_e4m3x2(__fdiv_rn(__fdiv_rn(a, 6.0f), g), 0.f) & 0xFF);
  const float denom = __fmul_rn(e4m3_to_f32(sb), g);
  if (!(denom > 0.f)) return make_uint2(0u, 0u);
  float y[2][8];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i >> 3][i & 7] = __fdiv_rn(x[i], denom);
  return make_uint2(f32x8_to_e2m1x8(y[0]), f32x8_to_e2m1x8(y[1]));
}

// Dims 16 l .. 16 l + 15 of a cache row. The K/V writer has no exchange; the index
// writer's row maximum takes the whole warp.
__device__ __forceinline__ void write_kv(const InsertParams& p, bool is_v, int64_t row, const float (&x)[16], int l) {
  void* base = is_v ? p.v : p.k;
  const float s = is_v ? p.v_global : p.k_global;
  if (p.kv_nvfp4) {
    uint8_t sb;
    const uint2 c = fp4_group(x, s, sb);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + row * (kDim / 2) + 8 * l) = c;
    (is_v ? p.v_scale : p.k_scale)[row * (kDim / 16) + l] = sb;
  } else if (p.kv_fp8) {
    const uint2 a = codes8(x, s), b = codes8(x + 8, s);
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + row * kDim + 16 * l) = make_uint4(a.x, a.y, b.x, b.y);
  } else {
    uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + row * kDim + 16 * l);
    d[0] = pack8(x);
    d[1] = pack8(x + 8);
  }
}
__device__ __forceinline__ void write_idx(const InsertParams& p, int64_t row, const float (&x)[16], int l, bool live) {
  if (p.idx_fp4) {
    uint8_t sb;
    const uint2 c = fp4_group(x, p.idx_global, sb);
    if (!live) return;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.idx_keys) + row * (kDim / 2) + 8 * l) = c;
    p.idx_block_scale[row * (kDim / 16) + l] = sb;
    return;
  }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  const float s = __fdiv_rn(a, 448.0f);
  if (!live) return;
  uint4 c = make_uint4(0u, 0u, 0u, 0u);
  if (s > 0.f) {
    const uint2 lo = codes8(x, s), hi = codes8(x + 8, s);
    c = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.idx_keys) + row * kDim + 16 * l) = c;
  if (l == 0) p.idx_scale[row] = s;
}

template <bool kPairs, bool kNorm, bool kFew>       // interleaved pairs (2i, 2i + 1); norms; all warps begin at one time
__global__ void __launch_bounds__(32 * kRopeWarps, kRopeCtas) qkv_rope_insert_kernel(const __grid_constant__ RopeParams pp) {
  __shared__ alignas(128) uint8_t ring_rows[kRopeWarps * kRopeSlots * kRopeGroup];
  __shared__ alignas(16) uint8_t turn_rows[kRopeWarps * kRopeGroup];
  __shared__ uint64_t ring_bars[kRopeWarps * kRopeSlots];
  griddep_launch_dependents();
  griddep_wait();
  const InsertParams& p = pp.ins;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7;
  const int nq = pp.H, nk = p.G, ni = pp.idx_q != nullptr ? pp.I : 0;
  const int rows = nq + 2 * nk + 2 * ni;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
  const int64_t t = wid / pp.parts;
  const int part = static_cast<int>(wid - t * pp.parts);
  if (t >= p.T) return;

  const int q_passes = pp.parts * 4 >= rows ? 0 : nq / 4;       // a warp with one pass loads its rows itself (64 tokens: 4.7 -> 4.6 us)
  const uint16_t* q_row = pp.q + t * pp.q_stride;
  const uint32_t rows_at = smem_addr(ring_rows) + warp * kRopeSlots * kRopeGroup;
  const uint32_t bars_at = smem_addr(ring_bars) + warp * kRopeSlots * 8;
  uint64_t policy = 0;
  auto fetch = [&](int pass, int slot) {
    mbar_arrive_expect_tx(bars_at + 8 * slot, kRopeGroup);
    bulk_g2s(rows_at + slot * kRopeGroup, q_row + 4 * pass * kDim, kRopeGroup, bars_at + 8 * slot, policy);
  };
  if (lane == 0) {
    for (int i = 0; i < kRopeSlots; ++i) mbar_init(bars_at + 8 * i, 1);
    fence_mbar_init();
    policy = l2_evict_first_policy();
    for (int i = 0; i < kRopeSlots && part + i * pp.parts < q_passes; ++i) fetch(part + i * pp.parts, i);
  }
  __syncwarp();

  const int64_t slot = p.slots[t];
  // the lane's chunks, and which of its pairs turn: all or none of a chunk's
  const int n = pp.R / 16;
  const int ca = kPairs || l < n ? l : n + l, cb = kPairs || l >= n ? 8 + l : n + l;
  const bool turn_a = kPairs ? ca < 2 * n : l < n, turn_b = kPairs ? cb < 2 * n : l < n;
  // pair i of the lane: elements i and 8 + i, or 2i and 2i + 1
  auto ea = [](int i) { return kPairs ? 2 * i : i; };
  auto eb = [](int i) { return kPairs ? 2 * i + 1 : 8 + i; };
  // cos and sin of the lane's 8 pairs: each is computed by one of the four lanes that use it
  float cs[8], sn[8];
  {
    const int64_t pos = pp.positions[t];
    float c2[2], s2[2];
    // pairs i and i + 1 of the lane
    const int i = 2 * (lane >> 3);
    const bool on = kPairs && i >= 4 ? turn_b : turn_a;
    const int at = !kPairs ? 8 * l + i : i < 4 ? 4 * ca + i : 4 * cb + i - 4;
    // Read as parameters, lanes at 32 places take 32 turns, which shows where all warps begin at one time: so through an
    // address, as memory (64 tokens: 4.6 -> 4.0 us, whole heads 5.7 -> 4.3). Where warps follow one another it does not, and
    // spreads them (8,191 tokens: 53.1 as memory, 52.4 as parameters).
    ulonglong2 two = make_ulonglong2(0, 0);
    if (on && kFew) {
      const uint64_t* turns = pp.turn;
      asm volatile("" : "+l"(turns));
      two = *reinterpret_cast<const ulonglong2*>(turns + at);
    } else if (on) {
      two = make_ulonglong2(pp.turn[at], pp.turn[at + 1]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      c2[e] = 1.f;
      s2[e] = 0.f;
      if (on) {
        const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(pos) * (e ? two.y : two.x));   // modulo one turn
        sincospif(static_cast<float>(turn) * 0x1p-63f, &s2[e], &c2[e]);                                 // half turns in [-1, 1]
        c2[e] *= pp.gain;
        s2[e] *= pp.gain;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = __shfl_sync(0xffffffffu, c2[i & 1], 8 * (i >> 1) + l);
      sn[i] = __shfl_sync(0xffffffffu, s2[i & 1], 8 * (i >> 1) + l);
    }
  }
  const int64_t page = slot / kBlock, off = slot % kBlock;
  const bool held = slot >= 0 && slot < p.num_slots;
  if (slot >= p.num_slots && part == 0 && lane == 0) set_flag(p.flags, MSA_FLAG_BAD_SLOT);

  auto weights = [&](const float* wv, float (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(wv + (i < 2 ? 8 * ca + 4 * i : 8 * cb + 4 * (i - 2)));
      w[4 * i] = f.x; w[4 * i + 1] = f.y; w[4 * i + 2] = f.z; w[4 * i + 3] = f.w;
    }
  };
  // 1 / sqrt(mean of the row's squares + eps), by its 8 lanes; the whole warp calls it. Squares that leave fp32's range:
  // the row is scaled by a power of two.
  auto row_scale = [&](float (&x)[16]) {
    auto squares = [&]() {
      float s2[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 16; ++i) s2[i & 1] = fmaf(x[i], x[i], s2[i & 1]);
      float ss = s2[0] + s2[1];
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      return ss * (1.0f / kDim);
    };
    float ms = squares(), eps = pp.eps;
    if (__any_sync(0xffffffffu, !(ms <= 0x1p120f) || ms < pp.low)) {
      const float f = !(ms <= 0x1p120f) ? 0x1p-80f : ms < pp.low ? 0x1p80f : 1.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= f;
      eps = eps * f * f;
      ms = squares();
    }
    return rsqrtf(ms + eps);
  };
  // The row turned: with a norm its weights are folded into cosines and sines (wa cos, wb sin, wa sin, wb cos), so that a
  // pair is four products and two scalings; without one, dims that pass are kept from their neighbours' infinities.
  auto turned = [&](const float (&x)[16], const float (&k)[4][8], float rinv, float (&y)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[ea(i)], b = x[eb(i)];
      if (kNorm) {
        y[ea(i)] = (a * k[0][i] - b * k[1][i]) * rinv;
        y[eb(i)] = (a * k[2][i] + b * k[3][i]) * rinv;
      } else {
        const bool on = kPairs && i >= 4 ? turn_b : turn_a;
        y[ea(i)] = on ? a * cs[i] - b * sn[i] : a;
        y[eb(i)] = on ? a * sn[i] + b * cs[i] : b;
      }
    }
  };
  auto folded = [&](const float* wv, float (&k)[4][8]) {
    if (!kNorm) return;
    float w[16];
    weights(wv, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      k[0][i] = w[ea(i)] * cs[i]; k[1][i] = w[eb(i)] * sn[i];
      k[2][i] = w[ea(i)] * sn[i]; k[3][i] = w[eb(i)] * cs[i];
    }
  };

  // While the queries are on their way, the rows behind them: any last queries, keys, values, index rows
  const uint32_t swap_at = smem_addr(turn_rows) + warp * kRopeGroup + (lane >> 3) * (kDim * 2);
  int pass = part;
  if (pass < q_passes) pass += (q_passes - pass + pp.parts - 1) / pp.parts * pp.parts;
  for (; 4 * pass < rows; pass += pp.parts) {
    const int r = 4 * pass + (lane >> 3);
    const bool live = r < rows;
    // kind 0 q, 1 k, 2 v, 3 index q, 4 index k
    int kind = 0, h = live ? r : 0;
    const uint16_t* src = q_row + h * kDim;
    const float* wv = pp.wq;
    if (live && r >= nq) {
      h = r - nq;
      if (h < nk) { kind = 1; src = pp.k + t * pp.k_stride + h * kDim; wv = pp.wk; }
      else if ((h -= nk) < nk) { kind = 2; src = pp.v + t * pp.v_stride + h * kDim; }
      else if ((h -= nk) < ni) { kind = 3; src = pp.idx_q + t * pp.iq_stride + h * kDim; wv = pp.wiq; }
      else { h -= ni; kind = 4; src = pp.idx_k + t * pp.ik_stride + h * kDim; wv = pp.wik; }
    }
    uint4 lo = *reinterpret_cast<const uint4*>(src + 8 * ca), hi = *reinterpret_cast<const uint4*>(src + 8 * cb);
    {
      float x[16];
      unpack8(lo, x);
      unpack8(hi, x + 8);
      const float rinv = kNorm ? row_scale(x) : 1.f;
      if (kind != 2) {
        float k[4][8], y[16];
        folded(wv, k);
        turned(x, k, rinv, y);
        // rounded to bf16 here: what the outputs hold and the caches quantise
        lo = pack8(y);
        hi = pack8(y + 8);
      }
    }
    if (live && (kind == 0 || kind == 3)) {
      uint16_t* dst = kind == 0 ? pp.q_out + (t * nq + h) * kDim : pp.idx_q_out + (t * ni + h) * kDim;
      *reinterpret_cast<uint4*>(dst + 8 * ca) = lo;
      *reinterpret_cast<uint4*>(dst + 8 * cb) = hi;
    }
    const bool kv = kind == 1 || kind == 2;
    if (!__any_sync(0xffffffffu, live && (kv || kind == 4))) continue;
    st_shared16(swap_at + 16 * ca, lo);
    st_shared16(swap_at + 16 * cb, hi);
    __syncwarp();
    float x[16];
    unpack8(ld_shared16(swap_at + 32 * l), x);
    unpack8(ld_shared16(swap_at + 32 * l + 16), x + 8);
    __syncwarp();
    if (live && kv && held) write_kv(p, kind == 2, (page * nk + h) * kBlock + off, x, l);
    if (__any_sync(0xffffffffu, live && kind == 4))
      write_idx(p, kind == 4 ? (page * ni + h) * kBlock + off : 0, x, l, live && kind == 4 && held);
  }

  // Most rows are queries, four at a time
  if (part >= q_passes) return;
  float k[4][8];
  folded(pp.wq, k);
  uint16_t* dst = pp.q_out + (t * nq + 4 * part + (lane >> 3)) * kDim;
  const int64_t hop = 4ll * pp.parts * kDim;
  int buf = 0;
  uint32_t phase = 0;
  for (pass = part; pass < q_passes; pass += pp.parts) {
    if (__all_sync(0xffffffffu, mbar_wait(bars_at + 8 * buf, phase)) == 0) {
      // a copy that did not come in time; those behind it are waited for, so that none outlives the CTA
      if (lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
      for (int i = 1; i < kRopeSlots && pass + i * pp.parts < q_passes; ++i) {
        if (++buf == kRopeSlots) { buf = 0; phase ^= 1u; }
        mbar_wait(bars_at + 8 * buf, phase);
      }
      return;
    }
    const uint32_t at = rows_at + buf * kRopeGroup + (lane >> 3) * (kDim * 2);
    float x[16], y[16];
    unpack8(ld_shared16(at + 16 * ca), x);
    unpack8(ld_shared16(at + 16 * cb), x + 8);
    turned(x, k, kNorm ? row_scale(x) : 1.f, y);
    *reinterpret_cast<uint4*>(dst + 8 * ca) = pack8(y);
    *reinterpret_cast<uint4*>(dst + 8 * cb) = pack8(y + 8);
    dst += hop;
    __syncwarp();                                    // the buffer has been read
    if (lane == 0 && pass + kRopeSlots * pp.parts < q_passes) fetch(pass + kRopeSlots * pp.parts, buf);
    if (++buf == kRopeSlots) { buf = 0; phase ^= 1u; }
  }
}

cudaError_t launch_qkv_rope_insert(const RopeArgs& a, cudaStream_t stream, DispatchRecord* rec) {
  RopeParams pp;
  memset(&pp, 0, sizeof(pp));
  pp.ins = make_insert_params(a.ins);
  pp.q = static_cast<const uint16_t*>(a.q);
  pp.k = static_cast<const uint16_t*>(a.ins.k_new);
  pp.v = static_cast<const uint16_t*>(a.ins.v_new);
  pp.idx_q = static_cast<const uint16_t*>(a.idx_q);
  pp.idx_k = static_cast<const uint16_t*>(a.ins.idx_new);
  pp.q_stride = a.q_stride; pp.k_stride = a.k_stride; pp.v_stride = a.v_stride;
  pp.iq_stride = a.iq_stride; pp.ik_stride = a.ik_stride;
  pp.q_out = static_cast<uint16_t*>(a.q_out);
  pp.idx_q_out = static_cast<uint16_t*>(a.idx_q_out);
  pp.positions = a.positions;
  pp.wq = a.wq; pp.wk = a.wk; pp.wiq = a.wiq; pp.wik = a.wik;
  pp.eps = a.eps;
  pp.gain = a.rope->gain;
  pp.low = a.eps < 0x1p-100f ? 0x1p-100f : 0.f;
  pp.H = a.H;
  pp.I = a.I;
  pp.R = a.rope->rotary_dim;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  for (int i = 0; i < pp.R / 2; ++i) {
    const double turns = a.rope->freq[i] / kTwoPi;
    const double part = (turns - floor(turns)) * 0x1p64;
    pp.turn[i] = part < 0x1p64 ? static_cast<uint64_t>(part) : 0;
  }
  const int rows = a.H + 2 * a.ins.G + (a.idx_q ? 2 * a.I : 0);
  const int passes = (rows + 3) / 4;
  // Warps per token: about 16 warps per SM for few tokens, two per token for some, one from 32 tokens per SM on. Measured, 64
  // + 4 + 4 heads, FP8 cache, us by warps per token (the rule's in parentheses): 64 tokens on 4 / 8 / 16 / (18) 5.1 / 4.5 / 4.1
  // / (4.5); 512 on 3 / 4 / (5) / 6 / 8 10.3 / 8.8 / (8.3) / 8.0 / 8.3; 1,024 on 2 / (3) / 4 / 6 13.8 / (11.8) / 10.8 / 11.7;
  // 2,048 on 1 / (2) / 3 22.9 / (16.3) / 18.3; 4,500 35.8 / (32.9) / 33.1; 4,864 on (1) / 2 (38.7) / 34.9; 8,191 (52.2) /
  // 51.9. One KV head: 512 on 4 / (5) 4.9 / (5.1); 1,024 on 2 / (3) / 4 6.7 / (6.5) / 6.9; 2,048 on 1 / (2) 10.1 / (8.4);
  // 3,000 10.9 / (11.1); 4,864 on (1) / 2 (15.0) / 15.1; 8,191 (20.3) / 22.3; 16,000 (35.1) / 39.1. So the change from two to
  // one lies between that of few heads (some 18 tokens per SM) and that of many (over 50), and costs the latter 10 % there.
  const int64_t sms = device_sm_count();
  int64_t parts = a.ins.T >= 32 * sms ? 1 : (16 * sms + a.ins.T - 1) / a.ins.T;
  if (parts < 2 && a.ins.T < 32 * sms) parts = 2;
  if (parts > passes) parts = passes;
  pp.parts = static_cast<int>(parts);
  const int64_t grid = (a.ins.T * parts + kRopeWarps - 1) / kRopeWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const bool pairs = a.rope->layout == MSA_ROPE_INTERLEAVED;
  const bool few = a.ins.T * parts <= kRopeWarps * kRopeCtas * sms;
  auto pick = [&](auto all) {
    constexpr bool kFew = decltype(all)::value;
    return pairs ? (a.wq ? qkv_rope_insert_kernel<true, true, kFew> : qkv_rope_insert_kernel<true, false, kFew>)
                 : (a.wq ? qkv_rope_insert_kernel<false, true, kFew> : qkv_rope_insert_kernel<false, false, kFew>);
  };
  const cudaError_t err = launch_pdl(few ? pick(std::true_type()) : pick(std::false_type()),
                                     dim3(static_cast<unsigned>(grid)), dim3(32 * kRopeWarps), 0, stream, pp);
  if (err != cudaSuccess) return err;
  rec->set("qkv_rope_insert %s%s %s%s dims=%d grid=%lld block=%d warps_per_token=%d heads=%d+%d+%d",
           a.ins.kv_nvfp4 ? "nvfp4" : a.ins.kv_fp8 ? "fp8" : "bf16",
           a.idx_q ? (a.ins.idx_fp4 ? "+idx_nvfp4" : "+idx_fp8") : "", pairs ? "interleaved" : "half", a.wq ? " norm" : "",
           pp.R, static_cast<long long>(grid), 32 * kRopeWarps, pp.parts, a.H, a.ins.G, a.idx_q ? a.I : 0);
  return cudaGetLastError();
}

}  // namespace msa
