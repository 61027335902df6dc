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
// o / l, lse = ln 2 * (m + log2 l). Logits, sums and states are fp32. The weights
// of P V are rounded to the type its tensor-core product takes: bf16 for bf16
// caches (2^-8, V being bf16 and both operands of one type; a second product for
// the rest would double P V's share of the tensor pipe), f16 times 2^kPLift for
// NVFP4 and FP8 (2^-11, plus at most 2^-30 of the row's largest weight).
//
// Work split. The (request, KV head, block) triples in that order are the items;
// a (request, KV head) row is as long as its blocks plus row_cost (what starting
// and finishing a row costs, in blocks), W in all, and CTA c takes the items in
// [W c / C, W (c + 1) / C). It finds them from seq_lens itself, so the host needs
// no lengths and a captured graph serves changing ones. A row inside one CTA is
// finished there; a row cut by CTA boundaries leaves one partial per CTA, which
// paged_join_kernel joins in CTA order. One CTA per SM; the splitting itself
// costs under a microsecond, the join's launch about five (an empty pair of
// dependent launches takes 5.1 us, an empty launch 3.6).
#include <cuda.h>

#include <cstring>

#include "msa_internal.h"

namespace msa {

constexpr uint32_t kEvery = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2f = 0.693147180559945309f;
constexpr float kSlack = 8.f;       // log2 units a maximum may exceed the reference by before a rescale
// Quantised caches hold P as f16, times 2^kPLift: with the slack it fills f16's range up to 2^15, so that weights are
// exact to 2^-11 relative down to 2^-21 of the reference and to 2^-32 of it below. Without the lift those below 2^-25
// of the reference would leave the numerator while the sum (fp32) keeps them.
constexpr float kPLift = 7.f;
constexpr int kMaxCtas = 320;       // partial slots in the workspace, two per CTA

// A row cut by CTA boundaries, written by the CTA behind the first cut: n
// partials, CTA cta - 1's slot 1, then slot 0 of CTAs cta, cta + 1, ... The list
// holds one entry per CTA (its own cut, n = 0 if it describes none), or, where
// there are fewer rows than CTAs, one per row, so that the join is a small grid.
struct CutRow {
  int b, g, n, cta;
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
  int row_cost;
  int by_row;                       // the cuts are listed by row
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
  int end;                          // request behind the range's last: the unused places that follow may be many
  __device__ __forceinline__ void next(const PagedParams& p) {
    if (++blk < nb) return;
    blk = 0;
    if (++g < p.G) return;
    g = 0;
    skip(p, b + 1);
  }
  __device__ __forceinline__ void skip(const PagedParams& p, int from) {
    for (b = from; b < end; ++b) {
      L = paged_len(p, b);
      nb = (L + kBlock - 1) / kBlock;
      if (nb > 0) return;
    }
    nb = 0;
  }
};

struct Range {
  int64_t W;                        // length of all rows, row_cost included
  int64_t row0;                     // where the row of `at` starts in it
  int64_t n0, n1;                   // items before the CTA's first and behind its last
  int ctas;                         // CTAs that share W: at most W
  Walk at;                          // place of the first item
};

// The CTA's items, found by all of its threads (kThreads of them): each sums a
// run of requests; the threads whose runs hold the ends of the CTA's range walk
// them.
template <int kThreads>
__device__ void find_range(const PagedParams& p, int cta, int ctas, int64_t* warp_sums, Range* shared, Range& r) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = tid * per, b1 = b0 + per < p.B ? b0 + per : p.B;
  // blocks, and from bit 48 on the requests that have any
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int nb = paged_blocks(p, b);
    mine += nb + (static_cast<int64_t>(nb > 0) << 48);
  }
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
  auto blocks = [](int64_t v) { return v & ((1ll << 48) - 1); };
  auto length = [&](int64_t v) { return (blocks(v) + (v >> 48) * p.row_cost) * p.G; };
  const int64_t W = length(total);
  if (W < ctas) ctas = static_cast<int>(W);
  const int64_t x0 = cta < ctas ? W * cta / ctas : W, x1 = cta < ctas ? W * (cta + 1) / ctas : W;
  if (tid == 0) {
    shared->W = W;
    shared->ctas = ctas;
    shared->n0 = shared->n1 = blocks(total) * p.G;   // for an end at W
  }
  __syncthreads();
  const int64_t lo = length(before), hi = length(before + mine);
  if (x1 == W && mine > 0 && hi == W) shared->at.end = b1;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int64_t x = which ? x1 : x0;
    if (x < lo || x >= hi) continue;
    int64_t base = lo, done = blocks(before) * p.G;
    for (int b = b0; b < b1; ++b) {
      const int nb = paged_blocks(p, b);
      if (nb == 0) continue;
      const int span = nb + p.row_cost;
      if (x < base + static_cast<int64_t>(span) * p.G) {
        Walk w;
        w.b = b;
        w.nb = nb;
        w.L = paged_len(p, b);
        w.g = static_cast<int>((x - base) / span);
        const int64_t row0 = base + static_cast<int64_t>(w.g) * span;
        const int d = static_cast<int>(x - row0);
        w.blk = d > p.row_cost ? d - p.row_cost : 0;  // a row's cost lies in front of its blocks
        const int64_t n = done + static_cast<int64_t>(w.g) * nb + w.blk;
        if (which) {
          shared->n1 = n;
          shared->at.end = b + 1;
        } else {
          shared->n0 = n;
          shared->at.b = w.b;
          shared->at.g = w.g;
          shared->at.blk = w.blk;
          shared->at.nb = w.nb;
          shared->at.L = w.L;
          shared->row0 = row0;
        }
        break;
      }
      base += static_cast<int64_t>(span) * p.G;
      done += static_cast<int64_t>(nb) * p.G;
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

// Maximum of a state with sum l: -inf for an empty one; a finite one where NaN logits left no other, so that joins
// take the state up and the NaN reaches the output.
__device__ __forceinline__ float partial_max(float m, float l) { return l > 0.f ? m : l == 0.f ? -INFINITY : 0.f; }

// Outputs of requests without tokens, and the flag of bad lengths.
__device__ void paged_empty_requests(const PagedParams& p, int nthreads) {
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (paged_len(p, b) > 0) continue;
    if (threadIdx.x == 0 && p.seq_lens[b] != 0) set_flag(p.flags, MSA_FLAG_BAD_SEQLEN);
    if (p.by_row)
      for (int g = threadIdx.x; g < p.G; g += nthreads) p.cuts[b * p.G + g] = CutRow{b, g, 0, 0};
    const int64_t row0 = static_cast<int64_t>(b) * p.Q * p.H;
    uint4* o = reinterpret_cast<uint4*>(p.out + row0 * kDim);
    for (int i = threadIdx.x; i < p.Q * p.H * kDim / 8; i += nthreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse != nullptr)
      for (int i = threadIdx.x; i < p.Q * p.H; i += nthreads) p.lse[row0 + i] = -INFINITY;
  }
}

// The cuts this CTA describes for the join (one warp): its own, when its range
// starts inside a row whose first CTA is the one before it; listed by row, every
// row that starts in its range.
__device__ void paged_describe_cuts(const PagedParams& p, const Range& r, int cta) {
  const int lane = threadIdx.x & 31;
  int64_t left = r.n1 - r.n0;
  if (!p.by_row) {
    CutRow c{0, 0, 0, cta};
    if (left > 0 && r.at.blk > 0 && paged_cta_of(r.row0 + p.row_cost, r.W, r.ctas) == cta - 1) {
      c.b = r.at.b;
      c.g = r.at.g;
      c.n = paged_cta_of(r.row0 + p.row_cost + r.at.nb - 1, r.W, r.ctas) - (cta - 1) + 1;
    }
    if (lane == 0) p.cuts[cta] = c;
    return;
  }
  if (left <= 0) return;
  Walk w = r.at;
  int64_t row0 = r.row0;
  for (;;) {
    if (w.blk == 0) {
      const int last = paged_cta_of(row0 + p.row_cost + w.nb - 1, r.W, r.ctas);
      if (lane == 0) p.cuts[w.b * p.G + w.g] = CutRow{w.b, w.g, last > cta ? last - cta + 1 : 0, cta + 1};
    }
    left -= w.nb - w.blk;
    if (left <= 0) return;
    row0 += w.nb + p.row_cost;
    w.blk = w.nb - 1;
    w.next(p);
  }
}

// ---------------------------------------------------------------------------
// bf16 K/V, up to 16 query rows and a block table of moderate size, on warp-level
// mma. Eight warps take 16 tokens of every block each, with their own running
// maxima; blocks arrive by cp.async into two stages. Nothing passes between warps
// until the row ends, which is what small calls need: 2 requests of 4,096 tokens
// 11.6 us (over caches that L2 does not hold 13.2; rows as M on tcgen05: 14.6),
// bound by the two launches and the chain of latencies. Large ones are bound by
// the cache's bytes (32x32k: 322 us, 99 % of a copy's rate), where the rows-as-M
// form's third stage gains 2 %.
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kHalfBox = kBlock * 128;               // 128 rows of 64 16-bit values, swizzled

// Bytes of a block's K and V of one head, scales included.
template <int kKv>
__host__ __device__ constexpr uint32_t raw_bytes() {
  return kKv == MSA_BF16 ? 4 * kHalfBox : kKv == MSA_FP8_E4M3 ? 2 * kBlock * kDim : 2 * (kBlock * kDim / 2 + kBlock * kDim / 16);
}
constexpr uint32_t kMmaSmem = 2 * 4 * kHalfBox + kWarps * 16 * kDim * 4 + kWarps * 16 * 2 * 4;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Address of 16-byte chunk c (0..15) of row `row` in a [128][128] 16-bit tile of
// two swizzled 64-column boxes.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int row, int c) {
  return tile + (c >> 3) * kHalfBox + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ void load_block(const PagedParams& p, uint32_t stage, int page, int g) {
  const int64_t slab = static_cast<int64_t>(page) * p.G + g;
  const uint8_t* k = p.k + slab * (kBlock * kDim * 2);
  const uint8_t* v = p.v + slab * (kBlock * kDim * 2);
  for (int i = threadIdx.x; i < kBlock * 16; i += kThreads) {
    cp_async16(tile_at(stage, i >> 4, i & 15), k + i * 16);
    cp_async16(tile_at(stage + 2 * kHalfBox, i >> 4, i & 15), v + i * 16);
  }
}

__global__ void __launch_bounds__(kThreads, 1) paged_gqa_kernel(const __grid_constant__ PagedParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Range shared_range;
  __shared__ int64_t warp_sums[kWarps];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  float* merge = reinterpret_cast<float*>(sm + 2 * 4 * kHalfBox);          // the warps' states at a row's end
  float* merge_m = merge + kWarps * 16 * kDim;
  float* merge_l = merge_m + kWarps * 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gr = lane >> 2, c = lane & 3;

  griddep_launch_dependents();
  griddep_wait();
  const int cta = blockIdx.x;
  Range rg;
  find_range<kThreads>(p, cta, gridDim.x, warp_sums, &shared_range, rg);
  paged_empty_requests(p, kThreads);
  if (warp == kWarps - 1) paged_describe_cuts(p, rg, cta);
  const int64_t items = rg.n1 - rg.n0;
  if (items <= 0) return;

  uint32_t qf[8][4];
  float o[16][4], m_r[2], l_r[2];
  int limit[2];                                   // last token each of the thread's two rows sees

  auto begin = [&](const Walk& w) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = gr + 8 * r;
      const bool live = row < p.R;
      const uint16_t* qh = p.q + (live ? paged_head(p, w.b, w.g, row) : 0) * kDim;
      limit[r] = live ? w.L - p.Q + row / p.group : -1;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        qf[s][r] = live ? *reinterpret_cast<const uint32_t*>(qh + 16 * s + 2 * c) : 0u;
        qf[s][2 + r] = live ? *reinterpret_cast<const uint32_t*>(qh + 16 * s + 8 + 2 * c) : 0u;
      }
      m_r[r] = -INFINITY;
      l_r[r] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  };

  // One block's 16 tokens of this warp.
  auto compute = [&](const Walk& w, uint32_t tile) {
    const bool edge = (w.blk + 1) * kBlock - 1 > w.L - p.Q;      // some row's limit lies before the block's end
    const int t16 = 16 * warp;
    {
      float sc[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
      for (int sp = 0; sp < 4; ++sp) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          uint32_t b[4];
          ldsm_x4(tile_at(tile, t16 + 8 * nt + (lane & 7), 4 * sp + (lane >> 3)), b[0], b[1], b[2], b[3]);
          mma_bf16(sc[nt], qf[2 * sp], b[0], b[1]);
          mma_bf16(sc[nt], qf[2 * sp + 1], b[2], b[3]);
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
        mx = fmaxf(mx, __shfl_xor_sync(kEvery, mx, 2)) * p.scale_log2;
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
            const float pv = ex2_approx(fmaf(sc[nt][2 * r + e], p.scale_log2, neg));
            pr[nt][2 * r + e] = pv;
            l_r[r] += pv;
          }
      }
      uint32_t a[4];
      a[0] = pack_bf16x2(pr[0][0], pr[0][1]); a[1] = pack_bf16x2(pr[0][2], pr[0][3]);
      a[2] = pack_bf16x2(pr[1][0], pr[1][1]); a[3] = pack_bf16x2(pr[1][2], pr[1][3]);
#pragma unroll
      for (int np = 0; np < 8; ++np) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(tile_at(tile + 2 * kHalfBox, t16 + 8 * ((lane >> 3) & 1) + (lane & 7), 2 * np + (lane >> 4)), b0, b1, b2, b3);
        mma_bf16(o[2 * np], a, b0, b1);
        mma_bf16(o[2 * np + 1], a, b2, b3);
      }
    }
  };

  // Joins the warps' states: the row's output, or a partial.
  auto flush = [&](const Walk& w, bool from_start, bool to_end) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float v = l_r[r];
      v += __shfl_xor_sync(kEvery, v, 1);
      v += __shfl_xor_sync(kEvery, v, 2);
      const int at = warp * 16 + gr + 8 * r;
      if (c == 0) { merge_m[at] = partial_max(m_r[r], v); merge_l[at] = v; }
#pragma unroll
      for (int n = 0; n < 16; ++n)
        *reinterpret_cast<float2*>(merge + at * kDim + 8 * n + 2 * c) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
    }
    __syncthreads();
    const bool whole = from_start && to_end;
    float* part = whole ? nullptr : paged_part(p, cta, from_start ? 1 : 0);
    for (int i = threadIdx.x; i < p.R * 32; i += kThreads) {
      const int row = i >> 5, d = (i & 31) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int s = 0; s < kWarps; ++s) M = fmaxf(M, merge_m[16 * s + row]);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (M != -INFINITY) {
#pragma unroll
        for (int s = 0; s < kWarps; ++s) {
          const int at = 16 * s + row;
          const float f = ex2_approx(merge_m[at] - M);
          const float4 x = *reinterpret_cast<const float4*>(merge + at * kDim + d);
          L += f * merge_l[at];
          acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
        }
      }
      if (whole) {
        const float inv = L != 0.f ? 1.f / L : 0.f;
        const int64_t head = paged_head(p, w.b, w.g, row);
        *reinterpret_cast<uint2*>(p.out + head * kDim + d) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (p.lse != nullptr && d == 0) p.lse[head] = L != 0.f ? (M + log2f(L)) * kLn2f : -INFINITY;
      } else {
        *reinterpret_cast<float4*>(part + row * kDim + d) = acc;
        if (d == 0) { part[p.R * kDim + row] = M; part[p.R * (kDim + 1) + row] = L; }
      }
    }
    __syncthreads();
  };

  Walk cur = rg.at, nxt = rg.at;
  int page = paged_page(p, cur, threadIdx.x == 0);
  if (page >= 0) load_block(p, base, page, cur.g);
  asm volatile("cp.async.commit_group;" ::: "memory");
  bool from_start = cur.blk == 0;
  begin(cur);
  for (int64_t x = 0; x < items; ++x) {
    const uint32_t stage = base + static_cast<uint32_t>(x & 1) * 4 * kHalfBox;
    int npage = -1;
    nxt.next(p);
    if (x + 1 < items) {
      npage = paged_page(p, nxt, threadIdx.x == 0);
      if (npage >= 0) load_block(p, base + static_cast<uint32_t>((x + 1) & 1) * 4 * kHalfBox, npage, nxt.g);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    if (page >= 0) {
      const int live = cur.L - cur.blk * kBlock;                  // cached tokens of this block
      if (live < kBlock) {
        // V rows never written may hold NaN patterns, and 0 x NaN is NaN
        for (int i = threadIdx.x; i < (kBlock - live) * 16; i += kThreads)
          *reinterpret_cast<uint4*>(sm + (tile_at(stage + 2 * kHalfBox, live + (i >> 4), i & 15) - base)) =
              make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
      }
      compute(cur, stage);
    }
    __syncthreads();                                               // the stage is free
    const bool row_ends = cur.blk == cur.nb - 1;
    if (row_ends || x + 1 == items) flush(cur, from_start, row_ends);
    if (x + 1 < items && row_ends) {
      from_start = true;
      begin(nxt);
    }
    cur = nxt;
    page = npage;
  }
}

// ---------------------------------------------------------------------------
// FP8 and NVFP4 K/V on the fifth-generation tensor cores. mma.sync needs the
// values as f16 register fragments, and expanding them is what bounds it (32x32k
// FP8 417 us, 16x256k NVFP4 1,730); here both products take the tokens (then the dims) as the 128 rows of A,
//   S^T = K Q^T   (M = 128 tokens, N = NR query rows, K = 128 dims)
//   O^T = V^T P^T (M = 128 dims,   N = NR query rows, K = 128 tokens)
// so that K and V are A operands.
//   FP8: the stage is the operand: nothing is converted. Q and P are split into
//   8-bit parts that are accumulated one after the other: Q = two E4M3 parts
//   after a power-of-two scaling of its row (4 significant bits each, a bf16
//   query's 8; the second times 2^5, so that the split is exact to 2^-22 of the
//   row's largest value), P = three E5M2
//   parts of its f16 value (each the rest rounded to 3 significant bits, the rests
//   scaled by 2^3 and 2^7 into E5M2's range: exact down to 2^-13 of f16's 1, off by
//   at most f16's last step of 2^-24 below).
//   NVFP4: further warps expand each block (e2m1 x e4m3, exact in f16) into tensor
//   memory, V transposed on the way (its rows are tokens, and as A it is needed by
//   dims). Q is scaled into f16's range and P rounded to f16.
// Roles: warp 0 copies, warps 1 and 2 issue the MMAs of S and of P V, warp 3 lists
// the cut rows, then two groups of 4 softmax warps (a thread owns a token of S and
// a dim of O; the group with a row's first block also brings the next row's
// queries into shared memory), then the expanding warps. The softmax warps agree on
// a rescale with one barrier-with-vote per block; a row's reference is raised only
// when a logit exceeds it by 2^8, so that after a row's first block they hardly
// ever have to. P's columns are written token by token (MN-major, unswizzled: a
// thread's rows are 16-byte runs). Every wait on memory is bounded; a warp whose
// wait ran out still votes, so its group leaves together.
// Measured, one position, 4 KV heads of 16 query heads: FP8 32x32k 167 us (96 % of
// a copy's rate: the bytes bound it). NVFP4 16x256k 595 us (61 %): the softmax
// groups' chains of waits and exchanges take 480 us without the expansion, whose
// warps take issue slots from them. Its steps: K in tensor memory instead of shared
// memory 852 -> 740 us; S and P V issued by a warp each 676; two softmax groups 627;
// expanding warps in turns 620; V in tensor memory 595. A second P buffer per group:
// 632. All quantised forms keep a few values on the stack (bytes stored / loaded:
// FP8 136 / 188, NVFP4 4 / 4 with 16 rows and 130 / 168 with 32).
constexpr int kTcS = 2;                 // S buffers in tensor memory
constexpr int kInfos = 16;              // ring of block descriptions, longer than anything in flight

struct BlockInfo {
  int live, lim0;                       // cached tokens of the block; last token of position 0, both from its start
  int b, g, seg;                        // row; the CTA's segment (its run of one row's blocks)
  int idx, left;                        // blocks of the segment before and after this one, held to 2
  int flags;                            // 4: the segment starts its row, 8: it ends it
};

// The copy thread's view of the CTA's blocks, one after the other.
struct BlockFeed {
  static constexpr int kAhead = 4;      // page ids are fetched this many blocks ahead
  int page[kAhead];
  Walk far, cur;
  int items, n, seg, idx;
  bool from_start;
  __device__ __forceinline__ BlockFeed(const PagedParams& p, const Walk& at, int count)
      : far(at), cur(at), items(count), n(0), seg(0), idx(0), from_start(at.blk == 0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      page[i] = i < items ? paged_page(p, far, true) : -1;
      if (i < items) far.next(p);
    }
  }
  // Describes the next block and returns its (page, KV head) slab.
  __device__ __forceinline__ int64_t next(const PagedParams& p, BlockInfo& bi) {
    const int pg = page[0];
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i) page[i] = page[i + 1];
    if (n + kAhead < items) {
      page[kAhead - 1] = paged_page(p, far, true);
      far.next(p);
    }
    const int toks = cur.L - cur.blk * kBlock;
    bi.live = pg < 0 ? 0 : toks < kBlock ? toks : kBlock;
    bi.lim0 = pg < 0 ? -kBlock : toks - p.Q;
    bi.b = cur.b;
    bi.g = cur.g;
    const int row_left = cur.nb - 1 - cur.blk, left_here = row_left < items - 1 - n ? row_left : items - 1 - n;
    bi.seg = seg;
    bi.idx = idx < 2 ? idx : 2;
    bi.left = left_here < 2 ? left_here : 2;
    bi.flags = (from_start ? 4 : 0) | (row_left == left_here ? 8 : 0);
    ++idx;
    if (left_here == 0) {
      ++seg;
      idx = 0;
      from_start = true;                             // only the CTA's first segment may start inside a row
    }
    const int64_t slab = static_cast<int64_t>(pg < 0 ? 0 : pg) * p.G + cur.g;     // a bad page's place is taken by page 0
    ++n;
    cur.next(p);
    return slab;
  }
};

// Issues the copies of a block's K and V (codes and scales) into a stage.
template <int kKv>
__device__ __forceinline__ void copy_block(const PagedParams& p, const CUtensorMap* tk, const CUtensorMap* tv, int64_t slab,
                                           uint32_t dst, uint32_t full, uint64_t policy) {
  const int y = static_cast<int>(slab * kBlock);
  mbar_arrive_expect_tx(full, raw_bytes<kKv>());
  if (kKv == MSA_BF16) {
    tma_load_2d(dst, tk, 0, y, full);
    tma_load_2d(dst + kHalfBox, tk, 64, y, full);
    tma_load_2d(dst + 2 * kHalfBox, tv, 0, y, full);
    tma_load_2d(dst + 3 * kHalfBox, tv, 64, y, full);
  } else if (kKv == MSA_FP8_E4M3) {
    tma_load_2d(dst, tk, 0, y, full);
    tma_load_2d(dst + kBlock * kDim, tv, 0, y, full);
  } else {
    constexpr uint32_t codes = kBlock * kDim / 2, scales = kBlock * kDim / 16;
    tma_load_2d(dst, tk, 0, y, full);
    tma_load_2d(dst + codes, tv, 0, y, full);
    bulk_g2s(dst + 2 * codes, p.ks + slab * scales, scales, full, policy);
    bulk_g2s(dst + 2 * codes + scales, p.vs + slab * scales, scales, full, policy);
  }
}

__device__ __forceinline__ void st_shared16(uint32_t a, const uint32_t* v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// A warp's V scales of a block: two groups of 16 dims x 128 tokens, as f16 pairs of two tokens in rows of 20 words
// [group][(token / 2) % 4][token / 8], so that neither the stores nor the reads meet in a bank.
constexpr uint32_t kVScaleRow = 20, kVScaleBuf = 8 * kVScaleRow * 4;

template <int kKv, int NR>
struct TcCfg {
  static constexpr bool kFp8 = kKv == MSA_FP8_E4M3;
  // Two softmax groups of 4 warps take alternate blocks, each with its own references, sums and O, joined at the
  // segment's end: a block's chain of waits, exchange and stores is longer than its arithmetic.
  static constexpr int kGroups = 2;
  static constexpr int kTurns = NR <= 16 ? 2 : 1;              // groups of 4 warps that expand K, and V, taking turns
  static constexpr int kConv = kFp8 ? 0 : 8 * kTurns;          // expanding warps
  static constexpr int kSoft0 = 4, kConv0 = 4 + 4 * kGroups;
  static constexpr int kWarpsAll = kConv0 + kConv;
  // Registers per thread, moved between the warpgroups from what the launch gives each alike (65,536 over the
  // threads, in eights): the sum over the warpgroups stays the launch's.
  static constexpr int kRegs = 65536 / (32 * kWarpsAll) / 8 * 8;
  static constexpr int kRegsCtl = kFp8 ? 72 : NR <= 16 ? 56 : 64, kRegsConv = kFp8 ? 0 : NR <= 16 ? 56 : 64;
  static constexpr int kRegsFit = (kRegs * (kWarpsAll / 4) - kRegsCtl - (kConv / 4) * kRegsConv) / kGroups / 8 * 8;
  static constexpr int kRegsSoft = kRegsFit > 232 ? 232 : kRegsFit;
  static constexpr int kQParts = kFp8 ? 2 : 1, kPParts = kFp8 ? 3 : 1;
  static constexpr float kPUp1 = 8.f, kPUp2 = 128.f;           // scales of P's second and third part
  static constexpr uint32_t kQPart = NR * (kFp8 ? 128 : 256);  // bytes of one part
  static constexpr uint32_t kPPart = NR * (kFp8 ? 128 : 256);
  // One P buffer (there is one per group); it also stages 16 output rows
  static constexpr uint32_t kPBuf = kPParts * kPPart < 16 * kDim * 4 ? 16 * kDim * 4 : kPParts * kPPart;
  static constexpr uint32_t kStage = raw_bytes<kKv>();
  static constexpr uint32_t kVScales = kFp8 ? 0 : kTurns * 4 * kVScaleBuf;   // V's scales in f16, of a warp each
  static constexpr uint32_t kFixed = kVScales + 2 * kQParts * kQPart + 2 * kPBuf;
  static constexpr uint32_t kSmall = 2048 + NR * 128;
  static constexpr int kFit = static_cast<int>((231424 - 1024 - kFixed - kSmall) / kStage);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  // The parts of Q and P lie side by side as columns of one MMA (few and wide ones; the sums of the parts are
  // taken where S and O are read)
  static constexpr int kSCols = kQParts * NR, kOCols = kPParts * NR;
  static constexpr int kKCols = kFp8 ? 0 : 2 * (kDim / 2);     // NVFP4: K[2] in f16, two dims per column
  static constexpr int kVCols = kFp8 ? 0 : 2 * (kBlock / 2);   // and V[2], two tokens per column
  static constexpr int kSets = 4;                              // states: of each group, for this segment and the one before
  static constexpr int kUsedCols = kTcS * kSCols + kSets * kOCols + kKCols + kVCols;
  static constexpr uint32_t kCols = kUsedCols <= 64 ? 64 : kUsedCols <= 128 ? 128 : kUsedCols <= 256 ? 256 : 512;
  static constexpr float kOff = kPLift;                        // P, sums and O are held times 2^kOff
  // shared memory
  static constexpr uint32_t oStage = 0;
  static constexpr uint32_t oQ = (kStages * kStage + 1023) & ~1023u;
  static constexpr uint32_t oP = oQ + 2 * kQParts * kQPart;
  static constexpr uint32_t oVScales = oP + 2 * kPBuf;
  static constexpr uint32_t oInfo = oVScales + kVScales;
  static constexpr uint32_t oRow = oInfo + kInfos * sizeof(BlockInfo);   // [2 q buffers][NR] multiplier
  static constexpr uint32_t oRef = oRow + 2 * NR * 4;                    // [sets][NR] kOff - reference
  static constexpr uint32_t oAlpha = oRef + kSets * NR * 4;              // [sets][NR]
  static constexpr uint32_t oRed = oAlpha + kSets * NR * 4;              // [sets][4][NR]
  static constexpr uint32_t oPos = oRed + kSets * 4 * NR * 4;            // [NR] position of a row
  static constexpr uint32_t oBars = oPos + NR * 4;
  static constexpr int kBars = 2 * kStages + 2 * kTcS + 4 + 4 + (kFp8 ? 0 : 8) + 5;
  static constexpr uint32_t oSlot = oBars + kBars * 8;
  static constexpr uint32_t kTotal = oSlot + 16;
  static_assert(kStages >= 3, "at least three stages");
  // a wait by parity needs every phase of a stage to be seen by the same warps
  static_assert(kStages % kTurns == 0, "a stage's blocks belong to one turn");
  static_assert(kTotal - oInfo <= kSmall, "small area");
  static_assert(kUsedCols <= 512, "tensor memory");
};

// Shared-memory matrix descriptors: start address and leading and stride byte
// offsets in 16-byte units, descriptor version 1, swizzle. Swizzled 128 B: as the
// tensor maps write. Plain: core matrices of 8 rows of 16 bytes.
constexpr uint32_t kSwz128 = 2, kSwzNone = 0;
// The descriptor's upper half, and its lower half at `saddr`: within one operand
// only the address changes, by plain additions to the lower half.
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t swizzle) {
  return (sbo >> 4) | (1u << 14) | (swizzle << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  // one lane's value for the whole warp, so that it is kept in a uniform register
  return __shfl_sync(kEvery, (saddr >> 4) | ((lbo >> 4) << 16), 0);
}
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) { return static_cast<uint64_t>(hi) << 32 | lo; }

// Instruction descriptor: fp32 accumulator, operand types, majorness (0 K, 1 MN), N / 8, M / 16.
__host__ __device__ constexpr uint32_t mma_idesc(int a_type, int b_type, int N, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_type) << 7) | (static_cast<uint32_t>(b_type) << 10) |
         (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
// kind::f16 operand types: 0 f16, 1 bf16. kind::f8f6f4: 0 E4M3, 1 E5M2.

__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0) : "memory");
}
// A from tensor memory (kind::f16).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0) : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void smem_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld16(uint32_t a, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
                 "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
               : "r"(a));
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const float* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
               ::"r"(a), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]),
                 "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
               : "memory");
}
// 16 lanes x 16 columns: lane i of the warp holds lanes i / 4 (r[2k]) and 8 + i / 4 (r[2k + 1]) of column 4 k + i % 4.
__device__ __forceinline__ void tmem_st_16x16(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
               "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
               ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                 "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                 "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
                 "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

// A wait of a whole warp, with one answer for all of its lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(kEvery, mbar_wait(bar, parity)) != 0;
}

// Barrier of a softmax group (128 threads) that returns whether any thread voted yes.
__device__ __forceinline__ bool group_any(int id, bool vote) {
  uint32_t r;
  asm volatile("{\n .reg .pred q, a;\n setp.ne.u32 q, %2, 0;\n barrier.cta.red.or.pred a, %1, 128, q;\n selp.u32 %0, 1, 0, a;\n}"
               : "=r"(r) : "r"(id), "r"(vote ? 1u : 0u) : "memory");
  return r != 0;
}

constexpr float kQUp = 32.f;        // scale of Q's second part: half a step of a value below 2^8 is 2^3 at most
__device__ __forceinline__ uint2 fp8_parts(const float (&x)[4], float f) {
  const float y0 = x[0] * f, y1 = x[1] * f, y2 = x[2] * f, y3 = x[3] * f;
  const uint32_t a = f32x2_to_e4m3x2(y0, y1), b = f32x2_to_e4m3x2(y2, y3);
  const uint32_t ha = e4m3x2_to_f16x2(static_cast<uint16_t>(a)), hb = e4m3x2_to_f16x2(static_cast<uint16_t>(b));
  const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&ha));
  const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&hb));
  const uint32_t la = f32x2_to_e4m3x2((y0 - fa.x) * kQUp, (y1 - fa.y) * kQUp);
  const uint32_t lb = f32x2_to_e4m3x2((y2 - fb.x) * kQUp, (y3 - fb.y) * kQUp);
  return make_uint2(a | (b << 16), la | (lb << 16));
}

// Reduces N (16 or 32) values per lane over the warp, all of them at once: each
// step halves the values a lane keeps. Lane i ends with value i mod N in v[0].
template <int N, bool kMax>
__device__ __forceinline__ void warp_reduce_rows(float (&v)[N]) {
  auto op = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
  if (N == 16) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = op(v[i], __shfl_xor_sync(kEvery, v[i], 16));
  }
#pragma unroll
  for (int o = N == 16 ? 8 : 16; o > 0; o >>= 1) {
    const bool up = (threadIdx.x & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float a = v[i], b = v[i + o];
      v[i] = op(up ? b : a, __shfl_xor_sync(kEvery, up ? a : b, o));
    }
  }
}

template <int kKv, int NR>
__global__ void __launch_bounds__(32 * TcCfg<kKv, NR>::kWarpsAll, 1)
    paged_gqa_tc_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ PagedParams p) {
  using C = TcCfg<kKv, NR>;
  constexpr bool kFp8 = C::kFp8;
  constexpr int kAllThreads = 32 * C::kWarpsAll;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Range shared_range;
  __shared__ int64_t warp_sums[C::kWarpsAll];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  BlockInfo* infos = reinterpret_cast<BlockInfo*>(sm + C::oInfo);
  float* row_mul = reinterpret_cast<float*>(sm + C::oRow);
  float* row_ref = reinterpret_cast<float*>(sm + C::oRef);
  float* row_alpha = reinterpret_cast<float*>(sm + C::oAlpha);
  float* row_red = reinterpret_cast<float*>(sm + C::oRed);
  int* row_pos = reinterpret_cast<int*>(sm + C::oPos);
  const uint32_t bars = base + C::oBars;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  constexpr int b0 = 2 * C::kStages;
  auto s_full = [&](int i) { return bars + 8u * (b0 + i); };                       // S of a block is there
  auto p_full = [&](int i) { return bars + 8u * (b0 + kTcS + i); };                // P is written
  auto p_free = [&](int i) { return bars + 8u * (b0 + kTcS + 2 + i); };    // P V is done
  auto s_free = [&](int i) { return bars + 8u * (b0 + kTcS + 4 + i); }; // S is in the softmax warps' registers
  constexpr int b1 = b0 + 2 * kTcS + 4;
  auto q_full = [&](int i) { return bars + 8u * (b1 + i); };
  auto q_free = [&](int i) { return bars + 8u * (b1 + 2 + i); };
  auto k_full = [&](int i) { return bars + 8u * (b1 + 4 + i); };                   // NVFP4: f16 tiles
  auto k_free = [&](int i) { return bars + 8u * (b1 + 6 + i); };
  auto v_full = [&](int i) { return bars + 8u * (b1 + 8 + i); };
  auto v_free = [&](int i) { return bars + 8u * (b1 + 10 + i); };
  auto join_full = [&](int i) { return bars + 8u * (C::kBars - 5 + i); };           // a group's state of a segment
  auto join_free = [&](int i) { return bars + 8u * (C::kBars - 3 + i); };
  const uint32_t done_bar = bars + 8u * (C::kBars - 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kFp8 ? 1 : 8);                              // NVFP4: the expanding warps of K and of V
    }
    for (int i = 0; i < kTcS; ++i) {
      mbar_init(s_full(i), 2);                                        // the commit, and the issuing thread's own arrival
      mbar_init(s_free(i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(p_full(i), 4);
      mbar_init(p_free(i), 1);
      mbar_init(q_full(i), 4);
      mbar_init(q_free(i), 1 + 4);                       // S is done with Q, softmax with its multipliers
      if (!kFp8) {
        mbar_init(k_full(i), 4);
        mbar_init(k_free(i), 1);
        mbar_init(v_full(i), 4);
        mbar_init(v_free(i), 1);
      }
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(join_full(i), 4);
      mbar_init(join_free(i), 4);
    }
    mbar_init(done_bar, 2);
    fence_mbar_init();
    prefetch_tensormap(&tk);
    prefetch_tensormap(&tv);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + C::oSlot), "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  for (int r = threadIdx.x; r < NR; r += kAllThreads) row_pos[r] = r < p.R ? r / p.group : 0;
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + C::oSlot);
  const uint32_t tO = tmem + kTcS * C::kSCols, tK = tO + C::kSets * C::kOCols, tV = tK + C::kKCols;
  griddep_wait();

  const int cta = blockIdx.x;
  Range rg;
  find_range<kAllThreads>(p, cta, gridDim.x, warp_sums, &shared_range, rg);
  paged_empty_requests(p, kAllThreads);
  if (warp == 3) paged_describe_cuts(p, rg, cta);
  const int items = static_cast<int>(rg.n1 - rg.n0);
  bool ok = true;

  if (warp < C::kSoft0) {
  regs_dec<C::kRegsCtl>();
  if (items > 0 && warp == 0) {
    // ----------------------------------------------------------- copies --
    if (lane == 0) {
      BlockFeed feed(p, rg.at, items);
      const uint64_t policy = l2_evict_first_policy();
      int s = 0;
      uint32_t ph = 0;
      for (int n = 0; n < items; ++n) {
        if (!mbar_wait(empty(s), ph ^ 1u)) { ok = false; break; }
        const int64_t slab = feed.next(p, infos[n & (kInfos - 1)]);
        copy_block<kKv>(p, &tk, &tv, slab, base + C::oStage + s * C::kStage, full(s), policy);
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
      // no copy may be in flight when the CTA ends, whatever the others did
      for (int k = 0; k < C::kStages; ++k) mbar_wait(full(k), ph ^ (k < s ? 0u : 1u));
      if (!ok) set_flag(p.flags, MSA_FLAG_TIMEOUT);
    }
    __syncwarp();
  } else if (items > 0 && warp <= 2) {
    // ------------------------------------------------------------- MMAs --
    // S and P V are issued by a warp each, so that one's waits do not hold up the other. The whole warp runs the
    // loop and one elected lane issues, with descriptors in uniform registers: 40 cycles per MMA, which is A's
    // 4 KB at 128 bytes a cycle (10 from tensor memory), against 68 from a lane's branch.
    const bool lead = elect_one();
    if (warp == 1) {
      constexpr uint32_t id_s = mma_idesc(0, 0, C::kSCols, 0, 0), hi = desc_hi(1024, kSwz128);
      const uint32_t q0 = desc_lo(base + C::oQ, 16), k0 = desc_lo(base + C::oStage, 16);
      int stage = 0;
      uint32_t ph = 0;
      for (int n = 0; n < items; ++n) {
        ok = kFp8 ? warp_wait(full(stage), ph) : warp_wait(k_full(n & 1), (n >> 1) & 1);
        if (n >= kTcS) ok = ok && warp_wait(s_free(n & 1), ((n >> 1) - 1) & 1);
        if (!ok) break;
        const int seg = infos[n & (kInfos - 1)].seg, left = infos[n & (kInfos - 1)].left;
        if (infos[n & (kInfos - 1)].idx == 0 && !warp_wait(q_full(seg & 1), (seg >> 1) & 1)) { ok = false; break; }
        tmem_fence_after();
        if (lead) {
          const uint32_t q = q0 + (seg & 1) * (C::kQParts * C::kQPart >> 4);
          const uint32_t d = tmem + (n & 1) * C::kSCols;
          if (kFp8) {
            const uint32_t k = k0 + stage * (C::kStage >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_fp8(d, desc_of(k + kk * 2, hi), desc_of(q + kk * 2, hi), id_s, kk > 0);
          } else {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(d, tK + (n & 1) * (kDim / 2) + 8 * kk, desc_of(q + (kk >> 2) * (NR * 128 >> 4) + (kk & 3) * 2, hi), id_s, kk > 0);
            mma_commit(k_free(n & 1));
          }
          mma_commit(s_full(n & 1));
          mbar_arrive(s_full(n & 1));
          if (left == 0) mma_commit(q_free(seg & 1));
        }
        __syncwarp();
        if (++stage == C::kStages) { stage = 0; ph ^= 1u; }
      }
    } else {
      constexpr uint32_t id_o = mma_idesc(0, kFp8 ? 1 : 0, C::kOCols, kFp8 ? 1 : 0, 1);
      constexpr uint32_t hi_v = desc_hi(1024, kSwz128), hi_p = desc_hi(2048, kSwzNone);
      const uint32_t p0 = desc_lo(base + C::oP, 128);
      const uint32_t v0 = desc_lo(base + C::oStage + kBlock * kDim, 16384);             // (FP8)
      int stage = 0;
      for (int n = 0; n < items; ++n) {
        const int pb = n & 1;
        ok = (kFp8 || warp_wait(v_full(pb), (n >> 1) & 1)) && warp_wait(p_full(pb), (n >> 1) & 1);
        if (!ok) break;
        const bool fresh = infos[n & (kInfos - 1)].idx < 2;
        const uint32_t d = tO + ((infos[n & (kInfos - 1)].seg & 1) * 2 + (n & 1)) * C::kOCols;
        tmem_fence_after();
        if (lead) {
          const uint32_t pt = p0 + pb * (C::kPBuf >> 4);
          if (kFp8) {
            const uint32_t v = v0 + stage * (C::kStage >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_fp8(d, desc_of(v + kk * 256, hi_v), desc_of(pt + kk * 32, hi_p), id_o, !(fresh && kk == 0));
            mma_commit(empty(stage));
          } else {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(d, tV + (n & 1) * (kBlock / 2) + 8 * kk, desc_of(pt + kk * 16, hi_p), id_o, !(fresh && kk == 0));
            mma_commit(v_free(n & 1));
          }
          mma_commit(p_free(pb));
        }
        __syncwarp();
        if (++stage == C::kStages) stage = 0;
      }
    }
    if (!ok && lead) set_flag(p.flags, MSA_FLAG_TIMEOUT);
    if (lead) mma_commit(done_bar);                 // every MMA has finished before tensor memory is freed
    __syncwarp();
    mbar_wait(done_bar, 0);
    __syncwarp();
  }
  } else if (warp < C::kConv0) {
    // ---------------------------------------------------------- softmax --
    regs_inc<C::kRegsSoft>();
    const int grp = (warp - C::kSoft0) >> 2, wl = warp & 3, bar_id = 1 + grp;
    const int t = 32 * wl + lane;                   // token of S
    const int o_dim = kFp8 ? t : 32 * wl + 4 * (lane & 7) + (lane >> 3);        // dim of O: V's order of the lanes
    const uint32_t lanes = static_cast<uint32_t>(32 * wl) << 16;
    // The queries of a segment, by the group with the first block of the segment before it: 16 lanes take a row,
    // 8 dims each, all loads before the first use.
    constexpr int kQPasses = NR / 8;
    Walk w = rg.at;
    int w_seg = 0;
    int64_t w_left = items;
    auto put_q = [&](int seg) -> bool {
      for (; w_seg < seg; ++w_seg) {
        w_left -= w.nb - w.blk;
        w.blk = w.nb - 1;
        if (w_left <= 0) return true;               // there is no such segment
        w.next(p);
      }
      const int qb = seg & 1, hl = lane & 15;
      const int row = wl * 2 * kQPasses + (lane >> 4);
      uint4 v[kQPasses];
#pragma unroll
      for (int i = 0; i < kQPasses; ++i) {
        const int r = row + 2 * i, j = row_pos[r];
        const int64_t head = (static_cast<int64_t>(w.b) * p.Q + j) * p.H + w.g * p.group + (r - j * p.group);
        v[i] = r < p.R ? *reinterpret_cast<const uint4*>(p.q + head * kDim + 8 * hl) : make_uint4(0u, 0u, 0u, 0u);
      }
      if (seg >= 2 && !warp_wait(q_free(qb), ((seg >> 1) - 1) & 1)) return false;
      uint8_t* q = sm + C::oQ + qb * (C::kQParts * C::kQPart);
#pragma unroll
      for (int i = 0; i < kQPasses; ++i) {
        const int r = row + 2 * i;
        const float x0[4] = {bf16_bits_to_f32(v[i].x & 0xFFFF), bf16_bits_to_f32(v[i].x >> 16),
                             bf16_bits_to_f32(v[i].y & 0xFFFF), bf16_bits_to_f32(v[i].y >> 16)};
        const float x1[4] = {bf16_bits_to_f32(v[i].z & 0xFFFF), bf16_bits_to_f32(v[i].z >> 16),
                             bf16_bits_to_f32(v[i].w & 0xFFFF), bf16_bits_to_f32(v[i].w >> 16)};
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(x0[e]), fabsf(x1[e])));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kEvery, amax, o));
        // a power of two that brings it to [2^7, 2^8) (E4M3) or [2^14, 2^15) (f16)
        int sh = fp16_shift_for(amax) - (kFp8 ? 7 : 0);
        sh = sh < -126 ? -126 : sh;
        const float f = exp2_int(sh);
        if (kFp8) {
          const uint2 a = fp8_parts(x0, f), b = fp8_parts(x1, f);
          const uint32_t at = r * 128 + ((((hl >> 1) ^ r) & 7) << 4) + (hl & 1) * 8;
          *reinterpret_cast<uint2*>(q + at) = make_uint2(a.x, b.x);
          *reinterpret_cast<uint2*>(q + C::kQPart + at) = make_uint2(a.y, b.y);
        } else {
          *reinterpret_cast<uint4*>(q + (hl >> 3) * (NR * 128) + r * 128 + (((hl ^ r) & 7) << 4)) =
              make_uint4(pack_f16x2(x0[0] * f, x0[1] * f), pack_f16x2(x0[2] * f, x0[3] * f),
                         pack_f16x2(x1[0] * f, x1[1] * f), pack_f16x2(x1[2] * f, x1[3] * f));
        }
        // (an infinite query would be a finite code: its row is NaN)
        if (hl == 0) row_mul[qb * NR + r] = p.scale_log2 * p.k_global * (amax < INFINITY ? exp2_int(-sh) : NAN);
      }
      smem_to_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(qb));
      return true;
    };
    if (items > 0 && grp == 0) ok = put_q(0);
    float l[NR];
    int stage = grp;
    uint32_t joins = 0;                             // parity of the joins so far on either segment parity (bits 0, 1)
    bool first = false;                             // no block of the segment has set the references yet
    uint32_t lent = 0;                              // bits 0, 1: the other group may still read this one's state
    for (int n = grp; n < items; n += 2) {
      // (n & 1, the buffer of S and P, is grp)
      ok = mbar_wait(s_full(grp), (n >> 1) & 1) && ok;
      if (n >= 2) ok = mbar_wait(p_free(grp), ((n >> 1) - 1) & 1) && ok;
      const BlockInfo bi = infos[n & (kInfos - 1)];
      if (bi.idx < 2) {
        first = true;
#pragma unroll
        for (int r = 0; r < NR; ++r) l[r] = 0.f;
        if (lent >> (bi.seg & 1) & 1) ok = mbar_wait(join_free(bi.seg & 1), ((joins >> (bi.seg & 1)) & 1) ^ 1) && ok;
        lent &= ~(1u << (bi.seg & 1));
      }
      const int set = (bi.seg & 1) * 2 + grp;
      const uint32_t tOg = tO + set * C::kOCols + lanes;
      float* ref = row_ref + set * NR;
      float* alphas = row_alpha + set * NR;
      float* red = row_red + set * 4 * NR;
      const float* mul = row_mul + (bi.seg & 1) * NR ;
      float x[NR];
      tmem_fence_after();
#pragma unroll
      for (int i = 0; i < NR / 16; ++i) tmem_ld16(tmem + lanes + grp * C::kSCols + 16 * i, x + 16 * i);
      if (kFp8) {
        float lo[NR];
#pragma unroll
        for (int i = 0; i < NR / 16; ++i) tmem_ld16(tmem + lanes + grp * C::kSCols + NR + 16 * i, lo + 16 * i);
        tmem_wait_ld();
#pragma unroll
        for (int r = 0; r < NR; ++r) x[r] = fmaf(lo[r], 1.f / kQUp, x[r]);
      }
      tmem_wait_ld();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free(grp));
      const bool edge = bi.lim0 < kBlock - 1;
      float top = -INFINITY;
#pragma unroll
      for (int r = 0; r < NR; r += 4) {
        const float4 m4 = *reinterpret_cast<const float4*>(mul + r);
        const float4 f4 = *reinterpret_cast<const float4*>(ref + r);
        const float mm[4] = {m4.x, m4.y, m4.z, m4.w}, ff[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[r + e] = first ? x[r + e] * mm[e] : fmaf(x[r + e], mm[e], ff[e]);
          if (edge && t > bi.lim0 + row_pos[r + e]) x[r + e] = -INFINITY;
          top = fmaxf(top, x[r + e]);
        }
      }
      if (group_any(bar_id, first || !ok || top > C::kOff + kSlack)) {
        // the block's maxima over all tokens; rows that rise by more than the slack get a new reference
        {
          float v[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) v[r] = x[r];
          warp_reduce_rows<NR, true>(v);
          if (lane < NR) red[wl * NR + lane] = v[0];
        }
        if (group_any(bar_id, !ok)) { ok = false; break; }
        if (t < NR) {
          // x = s - reference + kOff, s itself in a first block; ref holds kOff - reference. A row that its
          // first block masks is masked by every later one: its reference stays -inf and its x with it
          const int r = t;
          const float v = fmaxf(fmaxf(red[r], red[NR + r]), fmaxf(red[2 * NR + r], red[3 * NR + r]));
          float alpha = 1.f, delta = 0.f;
          if (first) {
            delta = v == -INFINITY ? -INFINITY : C::kOff - v;
            ref[r] = delta;
          } else if (v > C::kOff + kSlack) {
            delta = C::kOff - v;
            alpha = ex2_approx(delta);
            ref[r] += delta;
          }
          alphas[r] = alpha;
          red[r] = delta;                            // (no other thread reads this row's maxima)
        }
        group_any(bar_id, false);
        tmem_fence_after();
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          x[r] += red[r];
          l[r] *= alphas[r];
        }
        if (!first) {
#pragma unroll
          for (int i = 0; i < C::kPParts * (NR / 16); ++i) {
            const int at = 16 * i;
            float o[16];
            tmem_ld16(tOg + at, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= alphas[16 * (i % (NR / 16)) + e];
            tmem_st16(tOg + at, o);
          }
          tmem_wait_st();
        }
        if (bi.live > 0) first = false;              // (a block whose page is bad sets nothing)
        group_any(bar_id, false);                    // `red` may change again
      }
      // probabilities
      const uint32_t pt = C::oP + grp * C::kPBuf + (t >> 3) * 128 + (t & 7) * 16;
#pragma unroll
      for (int i = 0; i < NR / 16; ++i) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = ex2_approx(x[16 * i + 2 * e]), b = ex2_approx(x[16 * i + 2 * e + 1]);
          l[16 * i + 2 * e] += a;
          l[16 * i + 2 * e + 1] += b;
          h[e] = pack_f16x2(a, b);
        }
        if (kFp8) {
          // An E5M2 byte is the upper byte of an f16. Each part is the rest rounded to 3 significant bits (sign and
          // magnitude, so adding half a step rounds either sign), and what it leaves fits the next one scaled by
          // 2^3 (at most half a step of 2^-2 relative), then by 2^4.
          uint8_t* d = sm + pt + (i) * 2048;
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            uint32_t w[4];
            const __half2 up = __float2half2_rn(part == 0 ? C::kPUp1 : C::kPUp2 / C::kPUp1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t r[2] = {h[2 * e] + 0x00800080u, h[2 * e + 1] + 0x00800080u};
              w[e] = __byte_perm(r[0], r[1], 0x7531);
              if (part < 2) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const uint32_t hi = r[k] & 0xFF00FF00u;
                  const __half2 rest = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&h[2 * e + k]),
                                                       *reinterpret_cast<const __half2*>(&hi)), up);
                  h[2 * e + k] = *reinterpret_cast<const uint32_t*>(&rest);
                }
              }
            }
            *reinterpret_cast<uint4*>(d + part * C::kPPart) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          uint8_t* d = sm + pt + (2 * i) * 2048;
          *reinterpret_cast<uint4*>(d) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(d + 2048) = make_uint4(h[4], h[5], h[6], h[7]);
        }
      }
      if (kFp8 && t >= bi.live) {
        // a V row that was never written may hold NaN patterns, and 0 x NaN is NaN
        uint4* v = reinterpret_cast<uint4*>(sm + C::oStage + stage * C::kStage + kBlock * kDim + t * kDim);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k ^ (t & 7)] = make_uint4(0u, 0u, 0u, 0u);     // (eight rows, eight banks)
      }
      stage += 2;
      if (stage >= C::kStages) stage -= C::kStages;
      smem_to_async();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(grp));

      if (bi.idx == 0) ok = put_q(bi.seg + 1);
      if (bi.left < 2) {
        // the group's last block of the segment
        warp_reduce_rows<NR, false>(l);
        if (lane < NR) red[wl * NR + lane] = l[0];
        ok = mbar_wait(p_free(grp), (n >> 1) & 1) && ok;
        const bool two = bi.idx + bi.left > 0;       // the other group has blocks of it too
        const int sp = bi.seg & 1;
        if (two && bi.left == 0) ok = mbar_wait(join_full(sp), (joins >> sp) & 1) && ok;
        if (two) joins ^= 1u << sp;
        if (group_any(bar_id, !ok)) { ok = false; break; }
        tmem_fence_after();
        if (two && bi.left == 1) {
          // the state stays where it is (O in tensor memory, references and sums in shared memory); the group
          // with the last block reads it
          if (lane == 0) mbar_arrive(join_full(sp));
          lent |= 1u << sp;
          continue;
        }
        // the segment's output: 16 rows at a time through shared memory (P's, which no MMA reads now), so that
        // the stores are whole rows and the code is short
        const bool whole = (bi.flags & 12) == 12;
        float* part = whole ? nullptr : paged_part(p, cta, (bi.flags & 4) ? 1 : 0);
        float* stg = reinterpret_cast<float*>(sm + C::oP + grp * C::kPBuf);
        const int other = set ^ 1;
        const float* red2 = row_red + other * 4 * NR;
        const float* ref2 = row_ref + other * NR;
        float* alphas2 = row_alpha + other * NR;
        const uint32_t tO2 = tO + other * C::kOCols + lanes;
        if (two && t < NR) {
          // the groups' common maximum and sum; alphas: what each group's O is multiplied by
          float l1 = red[t] + red[NR + t] + red[2 * NR + t] + red[3 * NR + t];
          float l2 = red2[t] + red2[NR + t] + red2[2 * NR + t] + red2[3 * NR + t];
          const float m1 = l1 > 0.f ? -ref[t] : -INFINITY, m2 = l2 > 0.f ? -ref2[t] : -INFINITY;
          const float m = fmaxf(m1, m2);
          const float f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m), f2 = m2 == -INFINITY ? 0.f : ex2_approx(m2 - m);
          alphas[t] = f1;
          alphas2[t] = f2;
          red[t] = f1 * l1 + f2 * l2;                // (no other thread reads this row's sums before the barrier)
          red[NR + t] = red[2 * NR + t] = red[3 * NR + t] = 0.f;
          ref[t] = -m;
        }
        if (two) group_any(bar_id, false);
#pragma unroll 1
        for (int i = 0; i < NR / 16 && 16 * i < p.R; ++i) {
          constexpr int kParts = C::kPParts;
          float o[kParts][16], o2[kParts][16];
#pragma unroll
          for (int k = 0; k < kParts; ++k) {
            tmem_ld16(tOg + k * NR + 16 * i, o[k]);
            if (two) tmem_ld16(tO2 + k * NR + 16 * i, o2[k]);
          }
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
#pragma unroll
            for (int k = 1; k < kParts; ++k) {
              const float down = 1.f / (k == 1 ? C::kPUp1 : C::kPUp2);
              o[0][e] = fmaf(o[k][e], down, o[0][e]);
              o2[0][e] = fmaf(o2[k][e], down, o2[0][e]);
            }
          }
          if (two) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 f1 = *reinterpret_cast<const float4*>(alphas + 16 * i + e);
              const float4 f2 = *reinterpret_cast<const float4*>(alphas2 + 16 * i + e);
              o[0][e] = f1.x * o[0][e] + f2.x * o2[0][e];
              o[0][e + 1] = f1.y * o[0][e + 1] + f2.y * o2[0][e + 1];
              o[0][e + 2] = f1.z * o[0][e + 2] + f2.z * o2[0][e + 2];
              o[0][e + 3] = f1.w * o[0][e + 3] + f2.w * o2[0][e + 3];
            }
          }
          if (i > 0) group_any(bar_id, false);
#pragma unroll
          for (int e = 0; e < 16; ++e) stg[e * kDim + o_dim] = o[0][e];
          group_any(bar_id, false);
#pragma unroll 1
          for (int e = wl; e < 16; e += 4) {
            const int r = 16 * i + e;
            if (r >= p.R) break;
            const float L = red[r] + red[NR + r] + red[2 * NR + r] + red[3 * NR + r];
            const float M = partial_max(-ref[r], L);                // L and O are in units of 2^M
            const float4 v = *reinterpret_cast<const float4*>(stg + e * kDim + 4 * lane);
            if (whole) {
              const float inv = L != 0.f ? p.v_global / L : 0.f;
              const int j = row_pos[r];
              const int64_t head = (static_cast<int64_t>(bi.b) * p.Q + j) * p.H + bi.g * p.group + (r - j * p.group);
              *reinterpret_cast<uint2*>(p.out + head * kDim + 4 * lane) =
                  L != 0.f ? make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv)) : make_uint2(0u, 0u);
              if (p.lse != nullptr && lane == 0) p.lse[head] = L != 0.f ? (M + log2f(L)) * kLn2f : -INFINITY;
            } else {
              *reinterpret_cast<float4*>(part + r * kDim + 4 * lane) = L != 0.f ? v : make_float4(0.f, 0.f, 0.f, 0.f);
              if (lane == 0) { part[p.R * kDim + r] = M; part[p.R * (kDim + 1) + r] = L; }
            }
          }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(q_free(bi.seg & 1));
          if (two) mbar_arrive(join_free(bi.seg & 1));
        }
        group_any(bar_id, false);                     // `red` and the references may change again
      }
    }
    if (!ok && lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
  } else if (C::kConv > 0) {
    regs_dec<C::kConv ? C::kRegsConv : C::kRegsCtl>();
    // -------------------------------------------------- NVFP4 expansion --
    // Four warps at a time expand K into tensor memory, four V. Of K a thread takes a token's row. V has to lie
    // with a dim per lane and two tokens per column: a warp takes 32 dims, transposed on the way from shared memory
    // (16-bit transposition: four dims of two tokens per register), in the order of lanes 8 k + j = dim 4 j + k. The
    // codes' 64-byte swizzle keeps the reads of eight rows in eight banks.
    const int cg = (warp - C::kConv0) >> 2, turn = cg % C::kTurns, wq = warp & 3;
    const bool isv = cg >= C::kTurns;
    constexpr uint32_t codes = kBlock * kDim / 2, scales = kBlock * kDim / 16;
    const uint32_t lanes = static_cast<uint32_t>(32 * wq) << 16;
    const int swz = ((lane >> 1) & 3) << 4;
    uint32_t* vs = reinterpret_cast<uint32_t*>(sm + C::oVScales + (turn * 4 + wq) * kVScaleBuf);
    int s = turn;
    uint32_t ph = 0;
    for (int n = turn; n < items; n += C::kTurns) {
      ok = mbar_wait(full(s), ph);
      if (n >= 2) ok = mbar_wait(isv ? v_free(n & 1) : k_free(n & 1), ((n >> 1) - 1) & 1) && ok;
      ok = __all_sync(kEvery, ok);
      if (!ok) break;
      tmem_fence_after();
      const uint8_t* st = sm + C::oStage + s * C::kStage;
      if (isv) {
        // a row that was never written may hold NaN patterns, and 0 x NaN is NaN: its scales count as 0
        const int live = infos[n & (kInfos - 1)].live;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int t = 32 * q + lane;
          uint32_t sc = *reinterpret_cast<const uint16_t*>(st + 2 * codes + scales + t * (kDim / 16) + 2 * wq);
          if (t >= live) sc = 0u;
          const uint32_t pair = e4m3x2_to_f16x2(static_cast<uint16_t>(sc)), other = __shfl_xor_sync(kEvery, pair, 1);
          vs[((lane & 1) * 4 + ((lane >> 1) & 3)) * kVScaleRow + 4 * q + (lane >> 3)] =
              lane & 1 ? __byte_perm(other, pair, 0x7632) : __byte_perm(pair, other, 0x5410);
        }
        __syncwarp();
        const uint32_t src = base + C::oStage + s * C::kStage + codes + lane * (kDim / 2) + ((16 * wq) ^ swz);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[4], a[8], b[8];
          ldsm_x4_t(src + q * 32 * (kDim / 2), w[0], w[1], w[2], w[3]);
          const uint4 f4 = *reinterpret_cast<const uint4*>(vs + ((lane >> 4) * 4 + (lane & 3)) * kVScaleRow + 4 * q);
          const uint32_t f[4] = {f4.x, f4.y, f4.z, f4.w};
          if (q == 3) {
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(s));
          }
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t e[4];
            e2m1x8_to_f16x2x4(w[m], e);              // dims (0, 1), (2, 3) of one token, then of the next
            const uint32_t y[4] = {__byte_perm(e[0], e[2], 0x5410), __byte_perm(e[0], e[2], 0x7632),
                                   __byte_perm(e[1], e[3], 0x5410), __byte_perm(e[1], e[3], 0x7632)};
            uint32_t z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&y[k]), *reinterpret_cast<const __half2*>(&f[m]));
              z[k] = *reinterpret_cast<const uint32_t*>(&v);
            }
            a[2 * m] = z[0]; a[2 * m + 1] = z[1];
            b[2 * m] = z[2]; b[2 * m + 1] = z[3];
          }
          const uint32_t to = tV + lanes + (n & 1) * (kBlock / 2) + 16 * q;
          tmem_st_16x16(to, a);
          tmem_st_16x16(to + (16u << 16), b);
        }
      } else {
        const int row = 32 * wq + lane;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          // 32 values, two scale groups
          const uint4 w = *reinterpret_cast<const uint4*>(st + row * (kDim / 2) + ((16 * c) ^ swz));
          const uint32_t sc = *reinterpret_cast<const uint16_t*>(st + 2 * codes + row * (kDim / 16) + 2 * c);
          if (c == 3) {
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(s));
          }
          const uint32_t words[4] = {w.x, w.y, w.z, w.w};
          const uint32_t pair = e4m3x2_to_f16x2(static_cast<uint16_t>(sc));
          const __half2 s01 = *reinterpret_cast<const __half2*>(&pair);
          const __half2 s2[2] = {__low2half2(s01), __high2half2(s01)};
          uint32_t h[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t e[4];
            e2m1x8_to_f16x2x4(words[k], e);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&e[j]), s2[k >> 1]);
              h[4 * k + j] = *reinterpret_cast<const uint32_t*>(&y);
            }
          }
          tmem_st16(tK + lanes + (n & 1) * (kDim / 2) + 16 * c, reinterpret_cast<const float*>(h));
        }
      }
      tmem_wait_st();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(isv ? v_full(n & 1) : k_full(n & 1));
      s += C::kTurns;
      if (s >= C::kStages) { s -= C::kStages; ph ^= 1u; }
    }
    if (!ok && lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
  }

  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
  }
}

// ---------------------------------------------------------------------------
// Many query rows per KV head (several positions; bf16 above 16, FP8 and NVFP4
// above 32): the rows are the M = 128 of both products,
//   S = Q K^T (N = 128 tokens, K = 128 dims), O += P V (N = 128 dims, K = 128 tokens),
// with Q and P as A operands in tensor memory. A softmax thread owns a row: its
// 128 logits of a block are in its registers and nothing is exchanged. bf16 K and
// V are B operands as the copies leave them; FP8 and NVFP4 blocks are expanded
// (exactly) by eight warps into f16 tiles, with Q scaled into f16's range by a
// power of two per row. Tensor memory: Q of this row and of the next (64 columns
// each, two dims per column), S twice (128; P over its first 64), O (128). Roles:
// copies, S, P V, the cut rows, four softmax warps, the expanding warps.
// Measured, 8 positions of 16 query heads, 4 KV heads: bf16 32x64k 630 us (the
// copy's rate: the bytes bound it; the warp mma form needs 1,712); FP8 32x32k 253
// us, 1,087 TFLOP/s, and NVFP4 16x64k 257 us. What bounds these is neither the
// softmax (two threads per row, on eight warps: 276 and 277 us) nor the expansion
// alone (twice the warps: 252 and 255): a block passes through expansion, S, softmax
// and P V one after the other, two blocks at a time, and three f16 tile pairs do not
// fit shared memory. One position: 32x32k 315 us, 102 % of a copy's rate.
template <int kKv>
struct RwCfg {
  static constexpr bool kQuant = kKv != MSA_BF16;
  static constexpr int kConv0 = 8, kWarpsAll = kQuant ? 16 : 8;
  static constexpr uint32_t kStage = raw_bytes<kKv>();
  static constexpr uint32_t kTiles = kQuant ? 8 * kHalfBox : 0;          // [2] of K, V in f16
  static constexpr int kStages = kKv == MSA_NVFP4 ? 5 : 3;
  static constexpr uint32_t oTiles = (kStages * kStage + 1023) & ~1023u;
  static constexpr uint32_t oInfo = oTiles + kTiles, oBars = oInfo + kInfos * sizeof(BlockInfo);
  static constexpr int kBars = 2 * kStages + 9 + (kQuant ? 6 : 0);
  static constexpr uint32_t oSlot = oBars + kBars * 8, kTotal = oSlot + 16;
  static_assert(kTotal <= 230912, "shared memory");
  static constexpr float kOff = kQuant ? kPLift : 0.f;                   // P, sums and O are held times 2^kOff (bf16 has fp32's range)
  // 512 threads have 128 registers each: 56 + 208 + 2 * 120 of the 4 * 128
  static constexpr int kRegsCtl = 56, kRegsSoft = 208, kRegsConv = 120;
};
constexpr uint32_t kRwQ = 0, kRwS = 128, kRwO = 384, kRwCols = 512;

__device__ __forceinline__ void tmem_ld32(uint32_t a, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
                 "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
                 "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
                 "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
               : "r"(a));
}

template <int kKv>
__global__ void __launch_bounds__(32 * RwCfg<kKv>::kWarpsAll, 1)
    paged_gqa_rows_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                          const __grid_constant__ PagedParams p) {
  using C = RwCfg<kKv>;
  constexpr bool kQuant = C::kQuant;
  constexpr int kAllThreads = 32 * C::kWarpsAll;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Range shared_range;
  __shared__ int64_t warp_sums[C::kWarpsAll];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  BlockInfo* infos = reinterpret_cast<BlockInfo*>(sm + C::oInfo);
  const uint32_t bars = base + C::oBars;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  constexpr int b0 = 2 * C::kStages;
  auto s_full = [&](int i) { return bars + 8u * (b0 + i); };
  auto p_full = [&](int i) { return bars + 8u * (b0 + 2 + i); };
  auto p_free = [&](int i) { return bars + 8u * (b0 + 4 + i); };       // P V is done: the S buffer and V's tile are free
  auto q_full = [&](int i) { return bars + 8u * (b0 + 6 + i); };
  const uint32_t done_bar = bars + 8u * (b0 + 8);
  auto k_full = [&](int i) { return bars + 8u * (b0 + 9 + i); };       // the f16 tiles
  auto k_free = [&](int i) { return bars + 8u * (b0 + 11 + i); };
  auto v_full = [&](int i) { return bars + 8u * (b0 + 13 + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), kQuant ? 8 : 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 2);
      mbar_init(p_full(i), 4);
      mbar_init(p_free(i), 1);
      mbar_init(q_full(i), 4);
      if (kQuant) {
        mbar_init(k_full(i), 4);
        mbar_init(k_free(i), 1);
        mbar_init(v_full(i), 4);
      }
    }
    mbar_init(done_bar, 2);
    fence_mbar_init();
    prefetch_tensormap(&tk);
    prefetch_tensormap(&tv);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + C::oSlot), "r"(kRwCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + C::oSlot);
  griddep_wait();

  const int cta = blockIdx.x;
  Range rg;
  find_range<kAllThreads>(p, cta, gridDim.x, warp_sums, &shared_range, rg);
  paged_empty_requests(p, kAllThreads);
  if (warp == 3) paged_describe_cuts(p, rg, cta);
  const int items = static_cast<int>(rg.n1 - rg.n0);
  bool ok = true;

  if (warp < 4) {
  if (kQuant) regs_dec<C::kRegsCtl>();
  if (items > 0 && warp == 0) {
    // ----------------------------------------------------------- copies --
    if (lane == 0) {
      BlockFeed feed(p, rg.at, items);
      const uint64_t policy = l2_evict_first_policy();
      int s = 0;
      uint32_t ph = 0;
      for (int n = 0; n < items; ++n) {
        if (!mbar_wait(empty(s), ph ^ 1u)) { ok = false; break; }
        const int64_t slab = feed.next(p, infos[n & (kInfos - 1)]);
        copy_block<kKv>(p, &tk, &tv, slab, base + s * C::kStage, full(s), policy);
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
      // no copy may be in flight when the CTA ends, whatever the others did
      for (int k = 0; k < C::kStages; ++k) mbar_wait(full(k), ph ^ (k < s ? 0u : 1u));
      if (!ok) set_flag(p.flags, MSA_FLAG_TIMEOUT);
    }
    __syncwarp();
  } else if (items > 0 && warp <= 2) {
    // ------------------------------------------------------------- MMAs --
    const bool lead = elect_one();
    constexpr uint32_t hi = desc_hi(1024, kSwz128);
    constexpr int type = kQuant ? 0 : 1;             // f16, bf16
    int stage = 0;
    uint32_t ph = 0;
    if (warp == 1) {
      constexpr uint32_t id_s = mma_idesc(type, type, 128, 0, 0);
      const uint32_t k0 = desc_lo(base + (kQuant ? C::oTiles : 0), 16);
      for (int n = 0; n < items; ++n) {
        ok = kQuant ? warp_wait(k_full(n & 1), (n >> 1) & 1) : warp_wait(full(stage), ph);
        if (n >= 2) ok = ok && warp_wait(p_free(n & 1), ((n >> 1) - 1) & 1);
        if (!ok) break;
        const int seg = infos[n & (kInfos - 1)].seg;
        if (infos[n & (kInfos - 1)].idx == 0 && !warp_wait(q_full(seg & 1), (seg >> 1) & 1)) { ok = false; break; }
        tmem_fence_after();
        if (lead) {
          const uint32_t k = k0 + (kQuant ? n & 1 : stage) * (4 * kHalfBox >> 4);
          const uint32_t d = tmem + kRwS + 128 * (n & 1), q = tmem + kRwQ + 64 * (seg & 1);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(d, q + 8 * kk, desc_of(k + (kk >> 2) * (kHalfBox >> 4) + (kk & 3) * 2, hi), id_s, kk > 0);
          if (kQuant) mma_commit(k_free(n & 1));
          mma_commit(s_full(n & 1));
          mbar_arrive(s_full(n & 1));
        }
        __syncwarp();
        if (++stage == C::kStages) { stage = 0; ph ^= 1u; }
      }
    } else {
      constexpr uint32_t id_o = mma_idesc(type, type, 128, 0, 1);
      const uint32_t v0 = desc_lo(base + (kQuant ? C::oTiles : 0) + 2 * kHalfBox, kHalfBox);
      for (int n = 0; n < items; ++n) {
        ok = warp_wait(p_full(n & 1), (n >> 1) & 1);
        if (kQuant) ok = ok && warp_wait(v_full(n & 1), (n >> 1) & 1);
        if (!ok) break;
        const bool fresh = infos[n & (kInfos - 1)].idx == 0;
        tmem_fence_after();
        if (lead) {
          const uint32_t v = v0 + (kQuant ? n & 1 : stage) * (4 * kHalfBox >> 4), pt = tmem + kRwS + 128 * (n & 1);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma_ts(tmem + kRwO, pt + 8 * kk, desc_of(v + kk * 128, hi), id_o, !(fresh && kk == 0));
          if (!kQuant) mma_commit(empty(stage));
          mma_commit(p_free(n & 1));
        }
        __syncwarp();
        if (++stage == C::kStages) stage = 0;
      }
    }
    if (!ok && lead) set_flag(p.flags, MSA_FLAG_TIMEOUT);
    if (lead) mma_commit(done_bar);                 // every MMA has finished before tensor memory is freed
    __syncwarp();
    mbar_wait(done_bar, 0);
    __syncwarp();
  }
  } else if (warp < C::kConv0) {
    // ---------------------------------------------------------- softmax --
    const int r = 32 * (warp & 3) + lane;           // query row, tensor-memory lane; token of V's dead rows
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const bool live_warp = 32 * (warp & 3) < p.R, live_row = r < p.R;
    const int j = live_row ? r / p.group : 0;
    if (kQuant) regs_inc<C::kRegsSoft>();
    Walk w = rg.at;                                 // row of the queries loaded next
    int64_t w_left = items;
    float mul = 0.f, mul_next = 0.f;                // log2 units of a logit, of this row's and the next row's queries
    auto load_q = [&](int buf) {
      if (live_warp) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (live_row ? paged_head(p, w.b, w.g, r) : 0) * kDim);
        uint32_t v[64];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint4 x = live_row ? src[k] : make_uint4(0u, 0u, 0u, 0u);
          v[4 * k] = x.x; v[4 * k + 1] = x.y; v[4 * k + 2] = x.z; v[4 * k + 3] = x.w;
        }
        mul_next = p.scale_log2;
        if (kQuant) {
          // f16 operands: the row times a power of two that brings its largest value to [2^14, 2^15)
          uint32_t big = 0u;                         // bf16 magnitudes order as their bits
#pragma unroll
          for (int k = 0; k < 64; ++k) big = __vmaxu2(big, v[k] & 0x7FFF7FFFu);
          const int sh = fp16_shift_for(fmaxf(bf16_bits_to_f32(big & 0xFFFF), bf16_bits_to_f32(big >> 16)));
          const float f = exp2_int(sh);
          // not below 2^-126 (logits of less than 2^-80 either way): a masked -inf times 0 would be NaN
          mul_next = fmaxf(p.scale_log2 * p.k_global * exp2_int(-sh), 0x1p-126f);
#pragma unroll
          for (int k = 0; k < 64; ++k) v[k] = pack_f16x2(bf16_bits_to_f32(v[k] & 0xFFFF) * f, bf16_bits_to_f32(v[k] >> 16) * f);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t h[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) h[k] = v[32 * half + k];
          tmem_st32(tmem + lanes + kRwQ + 64 * buf + 32 * half, h);
        }
        tmem_wait_st();
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(buf));
      w_left -= w.nb - w.blk;
      w.blk = w.nb - 1;
      if (w_left > 0) w.next(p);
    };
    if (items > 0) load_q(0);
    float ref = -INFINITY, l = 0.f;
    int stage = 0;
    for (int n = 0; n < items; ++n) {
      const int sb = n & 1;
      ok = warp_wait(s_full(sb), (n >> 1) & 1);
      if (!ok) break;
      const BlockInfo bi = infos[n & (kInfos - 1)];
      if (bi.idx == 0) {
        ref = -INFINITY;
        l = 0.f;
        mul = mul_next;
        if (w_left > 0) load_q((bi.seg + 1) & 1);   // S of the row before this one is done with that buffer
      }
      tmem_fence_after();
      if (live_warp) {
        const uint32_t sbuf = tmem + lanes + kRwS + 128 * sb;
        float x[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(sbuf + 32 * q, x + 32 * q);
        tmem_wait_ld();
        if (bi.lim0 < kBlock - 1) {
          const int lim = bi.lim0 + j;
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (k > lim) x[k] = -INFINITY;
        }
        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; ++k) top4[k & 3] = fmaxf(top4[k & 3], x[k]);
        const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * mul;
        const bool raise = top > ref + kSlack;
        const float alpha = raise && ref != -INFINITY ? ex2_approx(ref - top) : 1.f;
        if (__any_sync(kEvery, raise && ref != -INFINITY)) {
          // O *= alpha once the block before has landed
          ok = warp_wait(p_free((n - 1) & 1), ((n - 1) >> 1) & 1);
          if (!ok) break;
          tmem_fence_after();
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            float o[16];
            tmem_ld16(tmem + lanes + kRwO + 16 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] *= alpha;
            tmem_st16(tmem + lanes + kRwO + 16 * q, o);
          }
        }
        if (raise) ref = top;
        l *= alpha;
        const float neg = ref == -INFINITY ? 0.f : C::kOff - ref;
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float a = ex2_approx(fmaf(x[64 * q + 2 * k], mul, neg));
            const float b = ex2_approx(fmaf(x[64 * q + 2 * k + 1], mul, neg));
            l4[k & 3] += a + b;
            pk[k] = kQuant ? pack_f16x2(a, b) : pack_bf16x2(a, b);
          }
          tmem_st32(sbuf + 32 * q, pk);
        }
        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
      }
      if (!kQuant && r >= bi.live) {
        // a V row that was never written may hold NaN patterns, and 0 x NaN is NaN
        uint8_t* v = sm + stage * 4 * kHalfBox + 2 * kHalfBox + r * 128;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          *reinterpret_cast<uint4*>(v + 16 * (k ^ (r & 7))) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(v + kHalfBox + 16 * (k ^ (r & 7))) = make_uint4(0u, 0u, 0u, 0u);
        }
        smem_to_async();
      }
      if (++stage == C::kStages) stage = 0;
      tmem_wait_st();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(sb));
      if (bi.left == 0) {
        // the segment's output, a row per thread
        ok = warp_wait(p_free(sb), (n >> 1) & 1);
        if (!ok) break;
        tmem_fence_after();
        if (live_warp) {
          const bool whole = (bi.flags & 12) == 12;
          const float inv = l != 0.f ? p.v_global / l : 0.f, M = partial_max(ref - C::kOff, l);
          const int64_t head = live_row ? paged_head(p, bi.b, bi.g, r) : 0;
          float* part = whole ? nullptr : paged_part(p, cta, (bi.flags & 4) ? 1 : 0);
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            float o[16];
            tmem_ld16(tmem + lanes + kRwO + 16 * q, o);
            tmem_wait_ld();
            if (!live_row) continue;
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(p.out + head * kDim + 16 * q);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                dst[k] = l != 0.f ? make_uint4(pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
                                              pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                              pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                              pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv))
                                 : make_uint4(0u, 0u, 0u, 0u);
            } else {
              float4* dst = reinterpret_cast<float4*>(part + r * kDim + 16 * q);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                dst[k] = l != 0.f ? make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3])
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            }
          }
          if (live_row && whole && p.lse != nullptr) p.lse[head] = l != 0.f ? (M + log2f(l)) * kLn2f : -INFINITY;
          if (live_row && !whole) { part[p.R * kDim + r] = M; part[p.R * (kDim + 1) + r] = l; }
        }
        tmem_fence_before();
      }
    }
    if (!ok && lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
  } else if (kQuant) {
    // -------------------------------------------------------- expansion --
    // Four warps K, four V; a thread takes a token's row. The copies' swizzle keeps the reads of eight rows in
    // eight banks, the tiles' the stores.
    regs_dec<C::kRegsConv>();
    const bool isv = warp >= C::kConv0 + 4;
    const int row = 32 * (warp & 3) + lane;
    constexpr uint32_t rowb = kKv == MSA_FP8_E4M3 ? kDim : kDim / 2;
    constexpr uint32_t scales = kBlock * kDim / 16;
    const uint8_t* src = sm + (isv ? kBlock * rowb : 0) + row * rowb;
    const uint8_t* ssrc = sm + 2 * kBlock * rowb + (isv ? scales : 0) + row * (kDim / 16);
    const int swz = (kKv == MSA_FP8_E4M3 ? row & 7 : (row >> 1) & 3) << 4;
    int s = 0;
    uint32_t ph = 0;
    for (int n = 0; n < items; ++n) {
      ok = mbar_wait(full(s), ph);
      if (n >= 2) ok = mbar_wait(isv ? p_free(n & 1) : k_free(n & 1), ((n >> 1) - 1) & 1) && ok;
      ok = __all_sync(kEvery, ok);
      if (!ok) break;
      // a row that was never written may hold NaN patterns, and 0 x NaN is NaN
      const bool dead = isv && row >= infos[n & (kInfos - 1)].live;
      const uint32_t tile = base + C::oTiles + (n & 1) * 4 * kHalfBox + (isv ? 2 * kHalfBox : 0);
#pragma unroll
      for (int c = 0; c < static_cast<int>(rowb / 16); ++c) {
        uint4 w = *reinterpret_cast<const uint4*>(src + s * C::kStage + ((16 * c) ^ swz));
        if (dead) w = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
        if (kKv == MSA_FP8_E4M3) {
          uint32_t h[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            h[2 * k] = e4m3x2_to_f16x2(static_cast<uint16_t>(words[k] & 0xFFFF));
            h[2 * k + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(words[k] >> 16));
          }
          st_shared16(tile_at(tile, row, 2 * c), h);
          st_shared16(tile_at(tile, row, 2 * c + 1), h + 4);
        } else {
          uint32_t sc = *reinterpret_cast<const uint16_t*>(ssrc + s * C::kStage + 2 * c);
          if (dead) sc = 0u;
          const uint32_t pair = e4m3x2_to_f16x2(static_cast<uint16_t>(sc));
          const __half2 s01 = *reinterpret_cast<const __half2*>(&pair);
          const __half2 s2[2] = {__low2half2(s01), __high2half2(s01)};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[4];
            e2m1x8_to_f16x2x4(words[k], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&h[e]), s2[k >> 1]);
              h[e] = *reinterpret_cast<const uint32_t*>(&y);
            }
            st_shared16(tile_at(tile, row, 4 * c + k), h);
          }
        }
      }
      smem_to_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(empty(s));
        mbar_arrive(isv ? v_full(n & 1) : k_full(n & 1));
      }
      if (++s == C::kStages) { s = 0; ph ^= 1u; }
    }
    if (!ok && lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
  }

  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kRwCols) : "memory");
  }
}

// Joins the partials of a cut row, in CTA order. One CTA per (cut, group of
// rows); with few rows its warps share a row's partials. Bound by latencies: 6.7 us
// for 128 rows' cuts of 16 queries on cold caches, 10 us for 32 of 128 queries (12 MB).
constexpr int kJoinWarps = 16;
template <int kChunk>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(const __grid_constant__ PagedParams p, int rows_per_cta) {
  __shared__ float sm_o[kJoinWarps][kDim];
  __shared__ float sm_m[kJoinWarps], sm_l[kJoinWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int chunks = (p.R + rows_per_cta - 1) / rows_per_cta;
  const int entry = static_cast<int>(blockIdx.x) / chunks + (p.by_row ? 0 : 1);
  const int chunk = static_cast<int>(blockIdx.x) % chunks;
  const CutRow cut = p.cuts[entry];
  if (cut.n == 0) return;
  const int cta = cut.cta;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = kJoinWarps / rows_per_cta;                       // warps per row
  const int row = chunk * rows_per_cta + warp / wpr, sub = warp % wpr;
  const bool live = row < p.R;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto part_of = [&](int i) { return i == 0 ? paged_part(p, cta - 1, 1) : paged_part(p, cta - 1 + i, 0); };
  // kChunk partials at a time, all loads in flight together: their maxima and sums by lane, and their rows
#pragma unroll 1
  for (int base = sub; live && base < cut.n; base += kChunk * wpr) {
    float4 x[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (base + i * wpr < cut.n) x[i] = *reinterpret_cast<const float4*>(part_of(base + i * wpr) + row * kDim + 4 * lane);
    const int mine = base + (lane & (kChunk - 1)) * wpr;
    const float* part = part_of(mine < cut.n ? mine : 0);
    const float m = mine < cut.n ? part[p.R * kDim + row] : -INFINITY;
    const float l = mine < cut.n ? part[p.R * (kDim + 1) + row] : 0.f;
    float top = fmaxf(M, m);
#pragma unroll
    for (int o = kChunk / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kEvery, top, o));
    if (top == -INFINITY) continue;                  // every partial so far is empty
    const float was = ex2_approx(M - top), f = ex2_approx(m - top);
    float ls = f * l;
#pragma unroll
    for (int o = kChunk / 2; o > 0; o >>= 1) ls += __shfl_xor_sync(kEvery, ls, o);
    M = top;
    L = L * was + ls;
    acc.x *= was; acc.y *= was; acc.z *= was; acc.w *= was;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const float fi = __shfl_sync(kEvery, f, i);
      if (base + i * wpr < cut.n) {
        acc.x += fi * x[i].x; acc.y += fi * x[i].y; acc.z += fi * x[i].z; acc.w += fi * x[i].w;
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
  const float inv = L != 0.f ? p.v_global / L : 0.f;
  const int64_t head = paged_head(p, cut.b, cut.g, row);
  *reinterpret_cast<uint2*>(p.out + head * kDim + 4 * lane) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse != nullptr && lane == 0) p.lse[head] = L != 0.f ? (M + log2f(L)) * kLn2f : -INFINITY;
}

size_t paged_gqa_workspace_bytes(int Q, int H, int G) {
  return kMaxCtas * sizeof(CutRow) + kMaxCtas * 2 * static_cast<size_t>(part_floats(Q * (H / G))) * sizeof(float);
}

static cudaError_t launch_mma(const PagedParams& p, int ctas, cudaStream_t stream) {
  constexpr size_t smem = kMmaSmem + 1024;
  const cudaError_t err =
      cudaFuncSetAttribute(paged_gqa_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  return launch_pdl(paged_gqa_kernel, dim3(ctas), dim3(kThreads), smem, stream, p);
}

// cuTensorMapEncodeTiled from the driver, looked up through the runtime (the
// library does not link libcuda).
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool got = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                         cudaSuccess && q == cudaDriverEntryPointSuccess;
    return got ? reinterpret_cast<EncodeFn>(ptr) : nullptr;
  }();
  return fn;
}

// 2-D map over a cache's rows [P * G * 128][128 dims]: boxes of 128 rows x 128 bytes
// (bf16: half a row) in the 128-byte swizzle, or NVFP4 codes, 128 rows x 64 bytes in
// the 64-byte swizzle.
static cudaError_t cache_map(CUtensorMap* map, const void* base, int64_t rows, msa_dtype_t kv) {
  const bool bf16 = kv == MSA_BF16, fp4 = kv == MSA_NVFP4;
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(fp4 ? kDim / 2 : kDim), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(bf16 ? 2 * kDim : fp4 ? kDim / 2 : kDim)};
  const cuuint32_t box[2] = {bf16 || fp4 ? 64u : 128u, static_cast<cuuint32_t>(kBlock)};
  const cuuint32_t ones[2] = {1, 1};
  const CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                        const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        fp4 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int kKv, int NR>
static cudaError_t launch_tc(const PagedParams& p, int ctas, cudaStream_t stream) {
  using C = TcCfg<kKv, NR>;
  CUtensorMap tk, tv;
  memset(&tk, 0, sizeof(tk));
  memset(&tv, 0, sizeof(tv));
  cudaError_t err;
  const int64_t rows = static_cast<int64_t>(p.P) * p.G * kBlock;
  if ((err = cache_map(&tk, p.k, rows, static_cast<msa_dtype_t>(kKv))) != cudaSuccess) return err;
  if ((err = cache_map(&tv, p.v, rows, static_cast<msa_dtype_t>(kKv))) != cudaSuccess) return err;
  constexpr size_t smem = C::kTotal + 1024;
  err = cudaFuncSetAttribute(paged_gqa_tc_kernel<kKv, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  return launch_pdl(paged_gqa_tc_kernel<kKv, NR>, dim3(ctas), dim3(32 * C::kWarpsAll), smem, stream, tk, tv, p);
}

template <int kKv>
static cudaError_t launch_many(const PagedParams& p, int ctas, cudaStream_t stream) {
  CUtensorMap tk, tv;
  cudaError_t err;
  const int64_t rows = static_cast<int64_t>(p.P) * p.G * kBlock;
  if ((err = cache_map(&tk, p.k, rows, static_cast<msa_dtype_t>(kKv))) != cudaSuccess) return err;
  if ((err = cache_map(&tv, p.v, rows, static_cast<msa_dtype_t>(kKv))) != cudaSuccess) return err;
  constexpr size_t smem = RwCfg<kKv>::kTotal + 1024;
  err = cudaFuncSetAttribute(paged_gqa_rows_kernel<kKv>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  return launch_pdl(paged_gqa_rows_kernel<kKv>, dim3(ctas), dim3(32 * RwCfg<kKv>::kWarpsAll), smem, stream, tk, tv, p);
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
  const int64_t rows = static_cast<int64_t>(a.B) * a.G;
  p.by_row = rows < ctas - 1;
  const int cuts = p.by_row ? static_cast<int>(rows) : ctas - 1;
  // One form per number of query rows R. FP8 and NVFP4: tokens as M for 16 and 32 rows, rows as M above (32x16k, FP8
  // with 16 / 32 rows 91.3 / 98.0 us against 128.7 / 129.2, NVFP4 89.2 / 109.7 against 135.8 / 136.5; 64 rows on the
  // 32-row form would read the cache twice). bf16: up to 16 rows, warp mma for what a small block table can hold,
  // rows as M for a table of at least 64 blocks per CTA (32x32k 321.7 and 315.8; 64 requests of 8k-128k 1,322 and
  // 1,284). The host knows the table's width only, so short requests in a wide table take rows as M too; on cold caches
  // 2x4k 14.6 us instead of 13.2, 4x2k 14.5 and 13.0, 64 requests of up to 2,047 tokens 36.8 and 36.0, 8x8k 32.4 and
  // 31.6, 16x16k 90.0 and 89.7.
  const bool large = most >= 64ll * ctas;
  const int rows_of = a.kv == MSA_BF16 ? (p.R <= 16 && !large ? 16 : 128) : p.R <= 16 ? 16 : p.R <= 32 ? 32 : 128;
  // A row's start and end, in blocks of its form. 64 requests of up to 2,047 tokens, 4 KV heads, at 0 / 2 / 3 / 5 / 8:
  // bf16 with 16 rows 54.7 / 39.2 / 36.6 / 37.3 / 39.9 us, 64 rows 56.0 / 43.6 / 41.8 / 41.7 / 42.8; FP8 16 rows
  // 37.7 / 30.2 / 28.0 / 26.7 / 26.4, 64 rows 60.6 / 45.4 / 40.7 / 39.2 / 40.8; NVFP4 32 rows 58.7 / 43.3 / 38.7 / 37.4 / 37.5.
  p.row_cost = a.kv == MSA_BF16 ? 3 : 5;
  cudaError_t err;
  if (a.kv == MSA_BF16)
    err = rows_of == 16 ? launch_mma(p, ctas, stream) : launch_many<MSA_BF16>(p, ctas, stream);
  else if (a.kv == MSA_FP8_E4M3)
    err = rows_of == 16 ? launch_tc<MSA_FP8_E4M3, 16>(p, ctas, stream)
        : rows_of == 32 ? launch_tc<MSA_FP8_E4M3, 32>(p, ctas, stream) : launch_many<MSA_FP8_E4M3>(p, ctas, stream);
  else
    err = rows_of == 16 ? launch_tc<MSA_NVFP4, 16>(p, ctas, stream)
        : rows_of == 32 ? launch_tc<MSA_NVFP4, 32>(p, ctas, stream) : launch_many<MSA_NVFP4>(p, ctas, stream);
  if (err != cudaSuccess) return err;
  if (ctas > 1) {
    // Query rows per CTA: as few as a grid of two CTAs per SM allows, so that their warps share a row's partials
    // (1x128k, 152 partials of a row: 16.0 us, with 8 warps 16.9, with 4 20.6; 4x2k bf16 11.5 us, one warp per row
    // 13.9; 2x4k with 4 positions 13.9 and 18.4, a grid of one CTA per SM 14.4).
    int rpc = 1;
    while (rpc < kJoinWarps && static_cast<int64_t>(cuts) * ((p.R + rpc - 1) / rpc) > 2 * sms) rpc *= 2;
    const int wpr = kJoinWarps / rpc;
    const bool deep = p.by_row && ctas / rows + 2 > 4 * wpr;       // more partials than the warps take at once by fours
    const int chunks = (p.R + rpc - 1) / rpc;
    err = launch_pdl(deep ? paged_join_kernel<16> : paged_join_kernel<4>, dim3(cuts * chunks), dim3(32 * kJoinWarps), 0, stream, p, rpc);
    if (err != cudaSuccess) return err;
  }
  rec->set("paged_gqa %s %s rows=%d of %d grid=%d + join", a.kv == MSA_BF16 ? "bf16"
           : a.kv == MSA_FP8_E4M3 ? "fp8" : "nvfp4", a.kv == MSA_BF16 && rows_of == 16 ? "mma" : "tcgen05", p.R, rows_of, ctas);
  return cudaGetLastError();
}

}  // namespace msa
