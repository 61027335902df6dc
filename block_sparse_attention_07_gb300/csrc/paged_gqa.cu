// Dense GQA decode over the paged cache: attention of 1 to 8 new tokens per
// request over all of its cached tokens, split over their length and joined.
//
// "vLLM、AMD Instinct MI355X上で…" (news.ainew.jp): 57 of the 60 decoder layers
// are sparse; the others attend over every token. "MiniMax M3 vLLM サポート：…",
// section "EAGLE3 を用いた投機的デコード": a split-K decode path that serves every
// decode_query_len.
//
// Mathematics. With logits s_t = scale * log2(e) * q . k_t, a range of tokens
// gives (m, l, o) = (max s, sum 2^(s - m), sum 2^(s - m) v); two ranges join as
// m = max(m1, m2), l = sum 2^(mi - m) li, o = sum 2^(mi - m) oi, and the result is
// o / l, lse = ln 2 * (m + log2 l). Probabilities, sums and states are fp32.
//
// Work split. The items are the (request, KV head, block) triples in that
// order, W in all; CTA c takes items [W c / C, W (c + 1) / C). It finds them
// from seq_lens itself, so the host needs no lengths and a captured graph
// serves changing ones. A (request, KV head) row inside one CTA is finished
// there; a row cut by CTA boundaries leaves one partial per CTA, which
// paged_join_kernel joins in CTA order.
#include <cuda.h>

#include <cstring>

#include "msa_internal.h"

namespace msa {

constexpr uint32_t kEvery = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2f = 0.693147180559945309f;
constexpr float kSlack = 8.f;       // log2 units a maximum may exceed the reference by before a rescale
constexpr int kMaxCtas = 320;       // partial slots in the workspace, two per CTA

// A row cut by CTA boundaries: written by the CTA behind the first cut.
struct CutRow {
  int b, g, n, pad;                 // n partials: CTA c - 1's slot 1, then slot 0 of CTAs c, c + 1, ...
};

struct PagedParams {
  const uint16_t* q;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* ks;
  const uint8_t* vs;
  const int32_t* block_table;
  const int32_t* seq_lens;
  uint16_t* out;
  float* lse;
  float* parts;                     // [C][2] partials of part_floats(R)
  CutRow* cuts;                     // [C]
  uint32_t* flags;
  float k_global, v_global, scale_log2;
  int B, Q, H, G, NB, P;
  int group, R;                     // query heads per KV head; rows Q * group
};

// Cached tokens of request b (0 when the length is out of range).
__device__ __forceinline__ int paged_len(const PagedParams& p, int b) {
  const int L = p.seq_lens[b];
  return L < 0 || L > static_cast<int64_t>(p.NB) * kBlock ? 0 : L;
}
__device__ __forceinline__ int paged_blocks(const PagedParams& p, int b) {
  return static_cast<int>((static_cast<int64_t>(paged_len(p, b)) + kBlock - 1) / kBlock);
}

// First CTA whose range [W c / C, W (c + 1) / C) contains item x.
__device__ __forceinline__ int paged_cta_of(int64_t x, int64_t W, int C) {
  return static_cast<int>(((x + 1) * C + W - 1) / W) - 1;
}

// A place in the item order.
struct Walk {
  int b, g, blk, nb, L;
  __device__ __forceinline__ void next(const PagedParams& p) {
    if (++blk < nb) return;
    blk = 0;
    if (++g < p.G) return;
    g = 0;
    skip(p, b + 1);
  }
  __device__ __forceinline__ void skip(const PagedParams& p, int from) {
    for (b = from; b < p.B; ++b) {
      L = paged_len(p, b);
      nb = (L + kBlock - 1) / kBlock;
      if (nb > 0) return;
    }
    nb = 0;
  }
};

struct Range {
  int64_t x0, x1, W;
  int ctas;                         // CTAs that take items: at most W, so that none is empty
  Walk at;                          // place of x0
  int64_t row0;                     // first item of x0's row
};

// The CTA's item range, found by all of its threads (kThreads of them): each
// sums the blocks of a run of requests; the thread whose run holds x0 walks it.
template <int kThreads>
__device__ void find_range(const PagedParams& p, int cta, int ctas, int64_t* warp_sums, Range* shared, Range& r) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = tid * per, b1 = b0 + per < p.B ? b0 + per : p.B;
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += paged_blocks(p, b);
  int64_t in = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(kEvery, in, o);
    if (lane >= o) in += t;
  }
  if (lane == 31) warp_sums[warp] = in;
  __syncthreads();
  int64_t before = in - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t s = warp_sums[w];
    if (w < warp) before += s;
    total += s;
  }
  const int64_t W = total * p.G;
  if (W < ctas) ctas = static_cast<int>(W);
  const int64_t x0 = cta < ctas ? W * cta / ctas : W, x1 = cta < ctas ? W * (cta + 1) / ctas : W;
  if (tid == 0) { shared->x0 = x0; shared->x1 = x1; shared->W = W; shared->ctas = ctas; }
  if (x0 < x1 && x0 >= before * p.G && x0 < (before + mine) * p.G) {
    int64_t base = before * p.G;
    for (int b = b0; b < b1; ++b) {
      const int nb = paged_blocks(p, b);
      const int64_t n = static_cast<int64_t>(nb) * p.G;
      if (x0 < base + n) {
        const int64_t d = x0 - base;
        Walk w;
        w.b = b;
        w.nb = nb;
        w.L = paged_len(p, b);
        w.g = static_cast<int>(d / nb);
        w.blk = static_cast<int>(d - static_cast<int64_t>(w.g) * nb);
        shared->at = w;
        shared->row0 = x0 - w.blk;
        break;
      }
      base += n;
    }
  }
  __syncthreads();
  r = *shared;
}

// Page of a block, or -1 (flagged by the caller that reports).
__device__ __forceinline__ int paged_page(const PagedParams& p, const Walk& w, bool report) {
  const int page = p.block_table[static_cast<int64_t>(w.b) * p.NB + w.blk];
  if (page >= 0 && page < p.P) return page;
  if (report) set_flag(p.flags, MSA_FLAG_BAD_PAGE);
  return -1;
}

// Row r of a (request, KV head): position r / group, head r % group.
__device__ __forceinline__ int64_t paged_head(const PagedParams& p, int b, int g, int r) {
  const int j = r / p.group, h = r - j * p.group;
  return (static_cast<int64_t>(b) * p.Q + j) * p.H + static_cast<int64_t>(g) * p.group + h;
}

// Floats of a partial: o [R][128], m [R], l [R], rounded up so that every partial
// starts on a 16-byte boundary whatever R is.
__host__ __device__ __forceinline__ int part_floats(int R) { return (R * (kDim + 2) + 3) & ~3; }

__device__ __forceinline__ float* paged_part(const PagedParams& p, int cta, int slot) {
  return p.parts + (static_cast<int64_t>(cta) * 2 + slot) * part_floats(p.R);
}

// Outputs of requests without tokens, and the flag of bad lengths.
__device__ void paged_empty_requests(const PagedParams& p, int nthreads) {
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (paged_len(p, b) > 0) continue;
    if (threadIdx.x == 0 && p.seq_lens[b] != 0) set_flag(p.flags, MSA_FLAG_BAD_SEQLEN);
    const int64_t row0 = static_cast<int64_t>(b) * p.Q * p.H;
    uint4* o = reinterpret_cast<uint4*>(p.out + row0 * kDim);
    for (int i = threadIdx.x; i < p.Q * p.H * kDim / 8; i += nthreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse != nullptr)
      for (int i = threadIdx.x; i < p.Q * p.H; i += nthreads) p.lse[row0 + i] = -INFINITY;
  }
}

// The cut this CTA describes for the join: its range starts inside a row whose
// first CTA is the one before it.
__device__ void paged_describe_cut(const PagedParams& p, const Range& r, int cta) {
  CutRow c{0, 0, 0, 0};
  if (r.x0 < r.x1 && r.at.blk > 0 && paged_cta_of(r.row0, r.W, r.ctas) == cta - 1) {
    c.b = r.at.b;
    c.g = r.at.g;
    c.n = paged_cta_of(r.row0 + r.at.nb - 1, r.W, r.ctas) - (cta - 1) + 1;
  }
  p.cuts[cta] = c;
}

// ---------------------------------------------------------------------------
// All formats, any number of rows, on warp-level mma. Eight warps: MT row tiles
// of 16 x 8 / MT token slices. Blocks arrive by cp.async into two stages; FP8
// and NVFP4 values are expanded (exactly) to f16 in shared memory.
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kHalfBox = kBlock * 128;               // 128 rows of 64 16-bit values, swizzled

template <int kKv>
__host__ __device__ constexpr uint32_t raw_bytes() {
  return kKv == MSA_BF16 ? 4 * kHalfBox : kKv == MSA_FP8_E4M3 ? 2 * kBlock * kDim : 2 * (kBlock * kDim / 2 + kBlock * kDim / 16);
}
template <int kKv>
__host__ __device__ constexpr uint32_t simple_smem() {
  return 2 * raw_bytes<kKv>() + 4 * kHalfBox + kWarps * 16 * 2 * 4;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Address of 16-byte chunk c (0..15) of row `row` in a [128][128] 16-bit tile of
// two swizzled 64-column boxes.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int row, int c) {
  return tile + (c >> 3) * kHalfBox + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

template <int kKv>
__device__ __forceinline__ void load_block(const PagedParams& p, uint32_t stage, int page, int g) {
  const int64_t slab = static_cast<int64_t>(page) * p.G + g;
  const int tid = threadIdx.x;
  if (kKv == MSA_BF16) {
    const uint8_t* k = p.k + slab * (kBlock * kDim * 2);
    const uint8_t* v = p.v + slab * (kBlock * kDim * 2);
    for (int i = tid; i < kBlock * 16; i += kThreads) {
      cp_async16(tile_at(stage, i >> 4, i & 15), k + i * 16);
      cp_async16(tile_at(stage + 2 * kHalfBox, i >> 4, i & 15), v + i * 16);
    }
  } else {
    constexpr int row = kKv == MSA_FP8_E4M3 ? kDim : kDim / 2;
    constexpr int n = kBlock * row / 16;
    const uint8_t* k = p.k + slab * (kBlock * row);
    const uint8_t* v = p.v + slab * (kBlock * row);
    for (int i = tid; i < n; i += kThreads) {
      cp_async16(stage + i * 16, k + i * 16);
      cp_async16(stage + kBlock * row + i * 16, v + i * 16);
    }
    if (kKv == MSA_NVFP4) {
      const int64_t at = slab * (kBlock * kDim / 16);
      const uint32_t sc = stage + 2 * kBlock * row;
      if (tid < 64) cp_async16(sc + tid * 16, p.ks + at + tid * 16);
      else if (tid < 128) cp_async16(sc + tid * 16, p.vs + at + (tid - 64) * 16);
    }
  }
}

// Expands a raw stage into the f16 tile; V rows from `live` on become zero.
template <int kKv>
__device__ __forceinline__ void expand_block(uint8_t* sm, uint32_t raw, uint32_t base, uint32_t tile, int live) {
  for (int i = threadIdx.x; i < 2 * kBlock * 16; i += kThreads) {
    const int isv = i >= kBlock * 16, row = (i >> 4) & (kBlock - 1), c = i & 15;
    uint32_t h[4];
    if (kKv == MSA_FP8_E4M3) {
      const uint2 w = *reinterpret_cast<const uint2*>(sm + (raw - base) + isv * kBlock * kDim + row * kDim + 8 * c);
      h[0] = e4m3x2_to_f16x2(static_cast<uint16_t>(w.x & 0xFFFF));
      h[1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w.x >> 16));
      h[2] = e4m3x2_to_f16x2(static_cast<uint16_t>(w.y & 0xFFFF));
      h[3] = e4m3x2_to_f16x2(static_cast<uint16_t>(w.y >> 16));
    } else {
      constexpr int rowb = kDim / 2;
      const uint8_t* st = sm + (raw - base);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(st + isv * kBlock * rowb + row * rowb + 4 * c);
      const uint8_t s = st[2 * kBlock * rowb + isv * (kBlock * kDim / 16) + row * (kDim / 16) + (c >> 1)];
      e2m1x8_to_f16x2x4(w, h);
      const uint32_t s2 = e4m3x2_to_f16x2(static_cast<uint16_t>(s | (s << 8)));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&h[k]), *reinterpret_cast<const __half2*>(&s2));
        h[k] = *reinterpret_cast<const uint32_t*>(&y);
      }
    }
    if (isv && row >= live) h[0] = h[1] = h[2] = h[3] = 0u;
    *reinterpret_cast<uint4*>(sm + (tile_at(tile + isv * 2 * kHalfBox, row, c) - base)) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

template <int kKv, int MT>
__global__ void __launch_bounds__(kThreads, 1) paged_gqa_kernel(const __grid_constant__ PagedParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Range shared_range;
  __shared__ int64_t warp_sums[kWarps];
  constexpr int kSlices = kWarps / MT, kSliceTok = kBlock / kSlices;
  constexpr bool kF16 = kKv != MSA_BF16;
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const uint32_t stage0 = base, extra = base + 2 * raw_bytes<kKv>();
  float* merge = reinterpret_cast<float*>(sm + 2 * raw_bytes<kKv>());      // the f16 tile; row merges between blocks
  float* merge_m = reinterpret_cast<float*>(sm + 2 * raw_bytes<kKv>() + 4 * kHalfBox);
  float* merge_l = merge_m + kWarps * 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mt = warp % MT, sl = warp / MT;
  const int gr = lane >> 2, c = lane & 3;

  griddep_launch_dependents();
  griddep_wait();
  const int cta = blockIdx.x;
  Range rg;
  find_range<kThreads>(p, cta, gridDim.x, warp_sums, &shared_range, rg);
  paged_empty_requests(p, kThreads);
  if (threadIdx.x == 0) paged_describe_cut(p, rg, cta);
  if (rg.x0 >= rg.x1) return;

  uint32_t qf[8][4];
  float o[16][4], m_r[2], l_r[2], mul[2];
  int limit[2];                                   // last token each of the thread's two rows sees

  auto begin = [&](const Walk& w) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 16 * mt + gr + 8 * r;
      const bool live = row < p.R;
      const uint16_t* qh = p.q + (live ? paged_head(p, w.b, w.g, row) : 0) * kDim;
      limit[r] = live ? w.L - p.Q + row / p.group : -1;
      float amax = 0.f;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        qf[s][r] = live ? *reinterpret_cast<const uint32_t*>(qh + 16 * s + 2 * c) : 0u;
        qf[s][2 + r] = live ? *reinterpret_cast<const uint32_t*>(qh + 16 * s + 8 + 2 * c) : 0u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t wq = qf[s][2 * h + r];
          amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_f32(wq & 0xFFFF)), fabsf(bf16_bits_to_f32(wq >> 16))));
        }
      }
      mul[r] = p.scale_log2;
      if (kF16) {
        // f16 operands: the row times an exact power of two that brings it into f16's range
        amax = fmaxf(amax, __shfl_xor_sync(kEvery, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kEvery, amax, 2));
        const int sh = fp16_shift_for(amax);
        const float f = exp2_int(sh);
        mul[r] = p.scale_log2 * p.k_global * exp2_int(-sh);
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t wq = qf[s][2 * h + r];
            qf[s][2 * h + r] = pack_f16x2(bf16_bits_to_f32(wq & 0xFFFF) * f, bf16_bits_to_f32(wq >> 16) * f);
          }
      }
      m_r[r] = -INFINITY;
      l_r[r] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  };

  // One block's tokens of this warp's slice, 16 at a time.
  auto compute = [&](const Walk& w, uint32_t tile) {
    const bool edge = (w.blk + 1) * kBlock - 1 > w.L - p.Q;      // some row's limit lies before the block's end
#pragma unroll 1
    for (int t16 = sl * kSliceTok; t16 < (sl + 1) * kSliceTok; t16 += 16) {
      float sc[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
      for (int sp = 0; sp < 4; ++sp) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          uint32_t b[4];
          ldsm_x4(tile_at(tile, t16 + 8 * nt + (lane & 7), 4 * sp + (lane >> 3)), b[0], b[1], b[2], b[3]);
          if (kF16) {
            mma_f16(sc[nt], qf[2 * sp], b[0], b[1]);
            mma_f16(sc[nt], qf[2 * sp + 1], b[2], b[3]);
          } else {
            mma_bf16(sc[nt], qf[2 * sp], b[0], b[1]);
            mma_bf16(sc[nt], qf[2 * sp + 1], b[2], b[3]);
          }
        }
      }
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (w.blk * kBlock + t16 + 8 * nt + 2 * c + (e & 1) > limit[e >> 1]) sc[nt][e] = -INFINITY;
      }
      float alpha[2];
      bool raise = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(kEvery, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kEvery, mx, 2)) * mul[r];
        alpha[r] = 1.f;
        if (mx > m_r[r] + kSlack) {
          alpha[r] = ex2_approx(m_r[r] - mx);
          m_r[r] = mx;
          raise = true;
        }
      }
      if (__any_sync(kEvery, raise)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          l_r[r] *= alpha[r];
#pragma unroll
          for (int n = 0; n < 16; ++n) { o[n][2 * r] *= alpha[r]; o[n][2 * r + 1] *= alpha[r]; }
        }
      }
      float pr[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float neg = m_r[r] == -INFINITY ? 0.f : -m_r[r];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float pv = ex2_approx(fmaf(sc[nt][2 * r + e], mul[r], neg));
            pr[nt][2 * r + e] = pv;
            l_r[r] += pv;
          }
      }
      uint32_t a[4];
      if (kF16) {
        a[0] = pack_f16x2(pr[0][0], pr[0][1]); a[1] = pack_f16x2(pr[0][2], pr[0][3]);
        a[2] = pack_f16x2(pr[1][0], pr[1][1]); a[3] = pack_f16x2(pr[1][2], pr[1][3]);
      } else {
        a[0] = pack_bf16x2(pr[0][0], pr[0][1]); a[1] = pack_bf16x2(pr[0][2], pr[0][3]);
        a[2] = pack_bf16x2(pr[1][0], pr[1][1]); a[3] = pack_bf16x2(pr[1][2], pr[1][3]);
      }
#pragma unroll
      for (int np = 0; np < 8; ++np) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(tile_at(tile + 2 * kHalfBox, t16 + 8 * ((lane >> 3) & 1) + (lane & 7), 2 * np + (lane >> 4)), b0, b1, b2, b3);
        if (kF16) {
          mma_f16(o[2 * np], a, b0, b1);
          mma_f16(o[2 * np + 1], a, b2, b3);
        } else {
          mma_bf16(o[2 * np], a, b0, b1);
          mma_bf16(o[2 * np + 1], a, b2, b3);
        }
      }
    }
  };

  // Joins the token slices of the row tiles; the row's output, or a partial.
  auto flush = [&](const Walk& w, bool from_start, bool to_end) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float v = l_r[r];
      v += __shfl_xor_sync(kEvery, v, 1);
      v += __shfl_xor_sync(kEvery, v, 2);
      const int at = warp * 16 + gr + 8 * r;
      if (c == 0) { merge_m[at] = m_r[r]; merge_l[at] = v; }
#pragma unroll
      for (int n = 0; n < 16; ++n)
        *reinterpret_cast<float2*>(merge + at * kDim + 8 * n + 2 * c) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
    }
    __syncthreads();
    const bool whole = from_start && to_end;
    float* part = whole ? nullptr : paged_part(p, cta, from_start ? 1 : 0);
    for (int i = threadIdx.x; i < p.R * 32; i += kThreads) {
      const int row = i >> 5, d = (i & 31) * 4, tm = row >> 4, tr = row & 15;
      float M = -INFINITY;
#pragma unroll
      for (int s = 0; s < kSlices; ++s) M = fmaxf(M, merge_m[(s * MT + tm) * 16 + tr]);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (M != -INFINITY) {
#pragma unroll
        for (int s = 0; s < kSlices; ++s) {
          const int at = (s * MT + tm) * 16 + tr;
          const float f = ex2_approx(merge_m[at] - M);
          const float4 x = *reinterpret_cast<const float4*>(merge + at * kDim + d);
          L += f * merge_l[at];
          acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
        }
      }
      if (whole) {
        const float inv = L > 0.f ? p.v_global / L : 0.f;
        const int64_t head = paged_head(p, w.b, w.g, row);
        *reinterpret_cast<uint2*>(p.out + head * kDim + d) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (p.lse != nullptr && d == 0) p.lse[head] = L > 0.f ? (M + log2f(L)) * kLn2f : -INFINITY;
      } else {
        *reinterpret_cast<float4*>(part + row * kDim + d) = acc;
        if (d == 0) { part[p.R * kDim + row] = M; part[p.R * (kDim + 1) + row] = L; }
      }
    }
    __syncthreads();
  };

  Walk cur = rg.at, nxt = rg.at;
  int page = paged_page(p, cur, threadIdx.x == 0);
  if (page >= 0) load_block<kKv>(p, stage0, page, cur.g);
  asm volatile("cp.async.commit_group;" ::: "memory");
  bool from_start = cur.blk == 0;
  begin(cur);
  for (int64_t x = rg.x0; x < rg.x1; ++x) {
    const uint32_t stage = stage0 + static_cast<uint32_t>((x - rg.x0) & 1) * raw_bytes<kKv>();
    int npage = -1;
    nxt.next(p);
    if (x + 1 < rg.x1) {
      npage = paged_page(p, nxt, threadIdx.x == 0);
      if (npage >= 0) load_block<kKv>(p, stage0 + static_cast<uint32_t>((x + 1 - rg.x0) & 1) * raw_bytes<kKv>(), npage, nxt.g);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    if (page >= 0) {
      const int live = cur.L - cur.blk * kBlock;                  // cached tokens of this block
      uint32_t tile = stage;
      if (kF16) {
        expand_block<kKv>(sm, stage, base, extra, live);
        tile = extra;
        __syncthreads();
      } else if (live < kBlock) {
        // V rows never written may hold NaN patterns, and 0 x NaN is NaN
        for (int i = threadIdx.x; i < (kBlock - live) * 16; i += kThreads)
          *reinterpret_cast<uint4*>(sm + (tile_at(stage + 2 * kHalfBox, live + (i >> 4), i & 15) - base)) =
              make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
      }
      compute(cur, tile);
    }
    __syncthreads();                                               // the stage and the tile are free
    const bool row_ends = cur.blk == cur.nb - 1;
    if (row_ends || x + 1 == rg.x1) flush(cur, from_start, row_ends);
    if (x + 1 < rg.x1 && row_ends) {
      from_start = true;
      begin(nxt);
    }
    cur = nxt;
    page = npage;
  }
}

// Joins the partials of a cut row, in CTA order. One CTA per (cut, group of
// rows); with few rows the eight warps share a row's partials.
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const __grid_constant__ PagedParams p, int rows_per_cta) {
  __shared__ float sm_o[kWarps][kDim];
  __shared__ float sm_m[kWarps], sm_l[kWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int chunks = (p.R + rows_per_cta - 1) / rows_per_cta;
  const int cta = 1 + static_cast<int>(blockIdx.x) / chunks, chunk = static_cast<int>(blockIdx.x) % chunks;
  const CutRow cut = p.cuts[cta];
  if (cut.n == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = kWarps / rows_per_cta;                           // warps per row
  const int row = chunk * rows_per_cta + warp / wpr, sub = warp % wpr;
  const bool live = row < p.R;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    for (int i = sub; i < cut.n; i += wpr) {
      const float* part = i == 0 ? paged_part(p, cta - 1, 1) : paged_part(p, cta - 1 + i, 0);
      M = fmaxf(M, part[p.R * kDim + row]);
    }
    if (M != -INFINITY) {
#pragma unroll 4
      for (int i = sub; i < cut.n; i += wpr) {
        const float* part = i == 0 ? paged_part(p, cta - 1, 1) : paged_part(p, cta - 1 + i, 0);
        const float f = ex2_approx(part[p.R * kDim + row] - M);
        const float4 x = *reinterpret_cast<const float4*>(part + row * kDim + 4 * lane);
        L += f * part[p.R * (kDim + 1) + row];
        acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
      }
    }
  }
  if (wpr > 1) {
    *reinterpret_cast<float4*>(&sm_o[warp][4 * lane]) = acc;
    if (lane == 0) { sm_m[warp] = M; sm_l[warp] = L; }
    __syncthreads();
    if (sub != 0) return;
    const float M0 = M, L0 = L;
    for (int k = 1; k < wpr; ++k) M = fmaxf(M, sm_m[warp + k]);
    const float f0 = M0 == -INFINITY ? 0.f : ex2_approx(M0 - M);
    L = f0 * L0;
    acc.x *= f0; acc.y *= f0; acc.z *= f0; acc.w *= f0;
    for (int k = 1; k < wpr; ++k) {
      const float mk = sm_m[warp + k];
      const float f = mk == -INFINITY ? 0.f : ex2_approx(mk - M);
      const float4 x = *reinterpret_cast<const float4*>(&sm_o[warp + k][4 * lane]);
      L += f * sm_l[warp + k];
      acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
    }
  }
  if (!live) return;
  const float inv = L > 0.f ? p.v_global / L : 0.f;
  const int64_t head = paged_head(p, cut.b, cut.g, row);
  *reinterpret_cast<uint2*>(p.out + head * kDim + 4 * lane) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse != nullptr && lane == 0) p.lse[head] = L > 0.f ? (M + log2f(L)) * kLn2f : -INFINITY;
}

size_t paged_gqa_workspace_bytes(int Q, int H, int G) {
  return kMaxCtas * sizeof(CutRow) + kMaxCtas * 2 * static_cast<size_t>(part_floats(Q * (H / G))) * sizeof(float);
}

template <int kKv>
static cudaError_t launch_rows(const PagedParams& p, int mt, int ctas, cudaStream_t stream) {
  constexpr size_t smem = simple_smem<kKv>() + 1024;
  auto kern = mt == 1 ? paged_gqa_kernel<kKv, 1> : mt == 2 ? paged_gqa_kernel<kKv, 2>
            : mt == 4 ? paged_gqa_kernel<kKv, 4> : paged_gqa_kernel<kKv, 8>;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  return launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, stream, p);
}

cudaError_t launch_paged_gqa(const PagedArgs& a, cudaStream_t stream, DispatchRecord* rec) {
  PagedParams p;
  memset(&p, 0, sizeof(p));
  p.q = a.q;
  p.k = static_cast<const uint8_t*>(a.k);
  p.v = static_cast<const uint8_t*>(a.v);
  p.ks = a.k_scale;
  p.vs = a.v_scale;
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.out = a.out;
  p.lse = a.lse;
  p.cuts = static_cast<CutRow*>(a.workspace);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kMaxCtas * sizeof(CutRow));
  p.flags = a.flags;
  p.k_global = a.k_global;
  p.v_global = a.v_global;
  p.scale_log2 = a.softmax_scale * kLog2e;
  p.B = a.B; p.Q = a.Q; p.H = a.H; p.G = a.G; p.NB = a.NB; p.P = a.P;
  p.group = a.H / a.G;
  p.R = a.Q * p.group;
  const int sms = device_sm_count();
  int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  const int64_t most = static_cast<int64_t>(a.B) * a.G * a.NB;
  if (most < ctas) ctas = static_cast<int>(most);
  const int tiles = (p.R + 15) / 16;
  const int mt = tiles <= 1 ? 1 : tiles <= 2 ? 2 : tiles <= 4 ? 4 : 8;
  cudaError_t err = a.kv == MSA_BF16 ? launch_rows<MSA_BF16>(p, mt, ctas, stream)
                  : a.kv == MSA_FP8_E4M3 ? launch_rows<MSA_FP8_E4M3>(p, mt, ctas, stream)
                                         : launch_rows<MSA_NVFP4>(p, mt, ctas, stream);
  if (err != cudaSuccess) return err;
  if (ctas > 1) {
    const int rpc = p.R <= 16 ? 1 : 8;
    const int chunks = (p.R + rpc - 1) / rpc;
    err = launch_pdl(paged_join_kernel, dim3((ctas - 1) * chunks), dim3(kThreads), 0, stream, p, rpc);
    if (err != cudaSuccess) return err;
  }
  rec->set("paged_gqa %s mma rows=%d tiles=%d grid=%d block=%d + join", a.kv == MSA_BF16 ? "bf16"
           : a.kv == MSA_FP8_E4M3 ? "fp8" : "nvfp4", p.R, mt, ctas, kThreads);
  return cudaGetLastError();
}

}  // namespace msa
