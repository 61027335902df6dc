// Projection of FP8 rows: both operands E4M3 with fp32 scales per block of 128.
//
// "MiniMax-M3.1-Flash Day-0 対応" (aisoku.org), section "最適化と数値": the fused
// projection in front of norm, rotary embedding and insert; the pages give no
// formula. With g the blocks of 128 along K,
//   out[t, n] = sum_g sa[t, g] sw[n / 128, g] sum_{k in g} a[t, k] w[n, k].
// The inner sum is one tcgen05 product of K = 128 into tensor memory, fresh for
// every block; the outer one is kept in fp32 registers, which read the block's
// sums back and add them times their scales. Blocks of K beyond its end and rows
// beyond the operands' arrive as zeros.
#include <cstdlib>
#include <cstring>

#include "tcgen05.cuh"

namespace msa {

constexpr int kTile = 128;                              // weight rows of a tile, and K of a block
constexpr int kChunk = 16;                              // blocks of K whose scales are held in shared memory

struct LinearParams {
  const float* sa;              // [T, KB]
  const float* sw;              // [ceil(N / 128), KB]
  void* out;                    // [T] rows of N, out_stride apart
  uint32_t* flags;
  int64_t out_stride;
  int T, N, KB;
  int split;                    // CTAs (pairs) of a cluster, which share a tile's K
  int f32;
  int tiles_m, tiles_n, group;  // pairs: tiles of 256 tokens and of 256 weight rows, token tiles that are walked together
  int wide, quads;              // rows of the output start on 32-byte boundaries, on those of four values
};

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// 16 bytes of another CTA's shared memory.
__device__ __forceinline__ float4 ld_cluster(uint32_t saddr, int rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// 32 columns of the warp's 32 lanes, a lane each.
__device__ __forceinline__ void tmem_ld32(uint32_t a, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
                 "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
                 "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
                 "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
               : "r"(a));
}
// Waits for the loads so far; the values are tied to it, so that nothing reads them earlier.
__device__ __forceinline__ void tmem_wait_ld32(float* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                 "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
                 "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
               ::"memory");
}
// (d0, d1) += (a0, a1) * s
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float s) {
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 c, {%0, %1};\n"
      " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}"
      : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1), "f"(s));
}

// (d0, d1) += (a0, a1) * (s0, s1)
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float s0, float s1) {
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%0, %1};\n"
      " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}"
      : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1), "f"(s0), "f"(s1));
}

__device__ __forceinline__ void store_out(const LinearParams& p, int64_t t, int n, float v) {
  if (p.f32) static_cast<float*>(p.out)[t * p.out_stride + n] = v;
  else static_cast<__nv_bfloat16*>(p.out)[t * p.out_stride + n] = __float2bfloat16_rn(v);
}

// Four outputs of a row in a row; `quads`: they are aligned to their size.
__device__ __forceinline__ void store4(const LinearParams& p, int64_t t, int n, const float4& v) {
  if (p.quads && n + 4 <= p.N) {
    if (p.f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + t * p.out_stride + n) = v;
    else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + t * p.out_stride + n) =
             make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    return;
  }
  const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (n + u < p.N) store_out(p, t, n + u, e[u]);
}

// ---------------------------------------------------------------------------
// Weights as M. A CTA has 128 weight rows and up to NT tokens as the product's N,
// so that few tokens waste nothing but columns; the CTAs of a cluster share the
// tile's K and add their sums through distributed shared memory, in rank order.
template <int NT>
struct RowsCfg {
  static constexpr int kPer = NT < 32 ? NT : 32;                      // a thread's tokens
  static constexpr int kSumThreads = 128 * (NT / kPer), kThreads = kSumThreads + 64;
  static constexpr int kCtas = NT <= 64 ? 2 : 1;                      // per SM
  static constexpr int kAcc = NT <= 64 ? 4 : 2;                       // blocks' sums in tensor memory
  static constexpr uint32_t kCols = kAcc * NT < 32 ? 32 : kAcc * NT;
  static constexpr int kStages = NT <= 32 ? 5 : NT == 64 ? 4 : 6;
  static constexpr uint32_t kStage = (kTile + NT) * 128;
  static constexpr int kRow = NT + 4;                                 // floats of a scale row: 16-byte steps, spread over banks
  static constexpr uint32_t oTable = kStages * kStage;
  static constexpr uint32_t oBars = oTable + 2 * kChunk * kRow * 4;
  static constexpr int kBars = 2 * kStages + 2 * kAcc;
  static constexpr uint32_t oSlot = oBars + kBars * 8;
  static constexpr uint32_t kTotal = oSlot + 16;
  static_assert(NT * kTile * 4 <= kStages * kStage, "the sums of a tile fit into the stages");
  static_assert(kCols * kCtas <= 512, "tensor memory");
};

template <int NT>
__global__ void __launch_bounds__(RowsCfg<NT>::kThreads, RowsCfg<NT>::kCtas)
    fp8_linear_rows_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap ta,
                           const __grid_constant__ LinearParams p) {
  using C = RowsCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  float* table = reinterpret_cast<float*>(sm + C::oTable);
  float* sums = reinterpret_cast<float*>(sm);                         // [NT][128], over the stages when they are done
  const uint32_t bars = base + C::oBars;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto acc_full = [&](int i) { return bars + 8u * (2 * C::kStages + i); };
  auto acc_free = [&](int i) { return bars + 8u * (2 * C::kStages + C::kAcc + i); };
  constexpr int kCopyWarp = C::kSumThreads / 32, kMmaWarp = kCopyWarp + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < C::kAcc; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_free(i), C::kSumThreads / 32);
    }
    fence_mbar_init();
    prefetch_tensormap(&tw);
    prefetch_tensormap(&ta);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + C::oSlot), "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + C::oSlot);
  // Behind the allocation: a kernel that starts early could otherwise hold the columns that this CTA waits for, while
  // it waits for this CTA's end.
  griddep_launch_dependents();
  griddep_wait();

  const int rank = static_cast<int>(blockIdx.x) % p.split, tile = static_cast<int>(blockIdx.x) / p.split;
  const int tok0 = static_cast<int>(blockIdx.y) * NT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.KB) * rank / p.split);
  const int n = static_cast<int>(static_cast<int64_t>(p.KB) * (rank + 1) / p.split) - kb0;
  bool ok = true;

  if (warp == kCopyWarp) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      for (int i = 0; i < n; ++i) {
        if (!mbar_wait(empty(s), ph ^ 1u)) { ok = false; break; }
        const uint32_t at = base + s * C::kStage;
        mbar_arrive_expect_tx(full(s), C::kStage);
        tma_load_2d(at, &tw, (kb0 + i) * kTile, tile * kTile, full(s));
        tma_load_2d(at + kTile * 128, &ta, (kb0 + i) * kTile, tok0, full(s));
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
      // no copy may be in flight when the CTA ends, whatever the others did
      for (int k = 0; k < C::kStages; ++k) mbar_wait(full(k), ph ^ (k < s ? 0u : 1u));
      if (!ok) set_flag(p.flags, MSA_FLAG_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    constexpr uint32_t id = mma_idesc(0, 0, NT, 0, 0), hi = desc_hi(1024, kSwz128);
    const uint32_t w0 = desc_lo(base, 16), a0 = desc_lo(base + kTile * 128, 16);
    const bool lead = elect_one();
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n; ++i) {
      const int b = i % C::kAcc;
      ok = warp_wait(full(s), ph) && (i < C::kAcc || warp_wait(acc_free(b), (i / C::kAcc - 1) & 1));
      if (!ok) break;
      tmem_fence_after();
      if (lead) {
        const uint32_t w = w0 + s * (C::kStage >> 4), a = a0 + s * (C::kStage >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_fp8(tmem + b * NT, desc_of(w + kk * 2, hi), desc_of(a + kk * 2, hi), id, kk > 0);
        mma_commit(empty(s));
        mma_commit(acc_full(b));
      }
      __syncwarp();
      if (++s == C::kStages) { s = 0; ph ^= 1u; }
    }
    if (!ok && lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
  } else {
    // Thread = weight row and up to 32 tokens: their sums over the blocks, times the two scales of the block.
    constexpr int kFetch = NT * kChunk / C::kSumThreads;
    const float* sw = p.sw + static_cast<int64_t>(tile) * p.KB + kb0;
    float next[kFetch];
    auto fetch = [&](int c) {
#pragma unroll
      for (int j = 0; j < kFetch; ++j) {
        const int e = threadIdx.x + C::kSumThreads * j, t = e / kChunk, i = c * kChunk + e % kChunk;
        next[j] = i < n && tok0 + t < p.T ? p.sa[static_cast<int64_t>(tok0 + t) * p.KB + kb0 + i] * sw[i] : 0.f;
      }
    };
    auto keep = [&](int c) {
#pragma unroll
      for (int j = 0; j < kFetch; ++j) {
        const int e = threadIdx.x + C::kSumThreads * j;
        table[((c & 1) * kChunk + e % kChunk) * C::kRow + e / kChunk] = next[j];
      }
    };
    const int sub = warp & 3, tok = warp / 4 * C::kPer;
    float acc[C::kPer];
#pragma unroll
    for (int t = 0; t < C::kPer; ++t) acc[t] = 0.f;
    fetch(0);
    keep(0);
    named_barrier(1, C::kSumThreads);
    const uint32_t mine = tmem + (static_cast<uint32_t>(sub) << 21) + tok;
    for (int i = 0; i < n; ++i) {
      const int b = i % C::kAcc, c = i / kChunk, j = i % kChunk;
      if (j == 0 && c > 0) {
        keep(c);                            // the other half: every thread is behind the barrier of its last use
        named_barrier(1, C::kSumThreads);
      }
      if (j == 0) fetch(c + 1);
      ok = ok && warp_wait(acc_full(b), (i / C::kAcc) & 1);
      tmem_fence_after();
      const float4* scale = reinterpret_cast<const float4*>(table + ((c & 1) * kChunk + j) * C::kRow + tok);
      float x[32];
      if (C::kPer == 32) {
        tmem_ld32(mine + b * NT, x);
      } else {
        tmem_ld16(mine + b * NT, x);
#pragma unroll
        for (int u = C::kPer; u < 32; ++u) x[u] = 0.f;
      }
      tmem_wait_ld32(x);
      tmem_fence_before();
      if (lane == 0) mbar_arrive(acc_free(b));
#pragma unroll
      for (int u = 0; u < C::kPer; u += 4) {
        const float4 f = scale[u / 4];
        fma2(acc[u], acc[u + 1], x[u], x[u + 1], f.x, f.y);
        fma2(acc[u + 2], acc[u + 3], x[u + 2], x[u + 3], f.z, f.w);
      }
    }
    if (!ok && lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
    const int row = sub * 32 + lane;
    if (p.split == 1) {
#pragma unroll
      for (int t = 0; t < C::kPer; ++t)
        if (tile * kTile + row < p.N && tok0 + tok + t < p.T) store_out(p, tok0 + tok + t, tile * kTile + row, acc[t]);
    } else {
#pragma unroll
      for (int t = 0; t < C::kPer; ++t) sums[(tok + t) * kTile + row] = acc[t];
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
  }
  if (p.split == 1) return;

  cluster_sync_all();
  const int tokens = p.T - tok0 < NT ? p.T - tok0 : NT;
  for (int i = rank * blockDim.x + threadIdx.x; i < tokens * (kTile / 4); i += p.split * blockDim.x) {
    const int t = i >> 5, r = 4 * (i & 31);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < p.split; ++q) {
      const float4 x = ld_cluster(base + (t * kTile + r) * 4, q);
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    store4(p, tok0 + t, tile * kTile + r, v);
  }
  cluster_sync_all();                       // no CTA ends while another reads its sums
}

// ---------------------------------------------------------------------------
// Tokens as M, two CTAs of a cluster on one tile: 256 tokens x 256 weight rows per
// pair, each CTA with its 128 tokens' sums in tensor memory and half of the weight
// rows in shared memory, so that a block of K costs a CTA 32 KB of copies for 512
// cycles of tensor core. The first CTA's warp issues for both. Thread = token: one
// product of scales per block of K serves its 128 outputs. With few tiles, `split`
// pairs of a cluster share a tile's K and add their sums through distributed shared
// memory, in rank order; otherwise a pair walks over the tiles.
struct PairCfg {
  static constexpr int kTok = 128, kOut = 256;                        // a CTA's tokens, a tile's weight rows
  static constexpr int kStages = 6, kAcc = 2;
  static constexpr uint32_t kStage = 2 * 128 * 128;
  static constexpr uint32_t oBars = kStages * kStage;
  static constexpr int kBars = 2 * kStages + 2 * kAcc;
  static constexpr uint32_t oSlot = oBars + kBars * 8;
  static constexpr uint32_t kTotal = oSlot + 16;
  static constexpr int kThreads = 384;                                // 4 control warps, 8 that hold the sums
  static constexpr int kRegsCtl = 64, kRegsSum = 216;
  static_assert(128 * kRegsCtl + 256 * kRegsSum <= 384 * 168, "registers of the launch");
  static constexpr uint32_t kSumRow = kOut * 4 + 16;                  // bytes of a token's sums, spread over banks
  static_assert(kTok * kSumRow <= kStages * kStage, "the sums of a tile fit into the stages");
};

__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr), "r"(rank));
  return at;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Says that tensor memory has been read: what was read is in registers, and nothing was written that the other CTA
// would have to see, so the arrival needs no release (whose fence costs a microsecond).
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t at) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
}
// A tensor copy into this CTA that completes on a barrier of its pair's first CTA.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(tmap), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_fp8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0) : "memory");
}
// Arrives on the barrier at this offset in the CTAs of the mask once the products issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(bar), "h"(mask) : "memory");
}
// Sixteen outputs of a row in a row; `wide`: 32-byte stores are aligned.
__device__ __forceinline__ void store16(const LinearParams& p, int64_t t, int n, const float* v, bool wide) {
  if (wide && n + 16 <= p.N) {
    if (p.f32) {
      float* d = static_cast<float*>(p.out) + t * p.out_stride + n;
#pragma unroll
      for (int i = 0; i < 16; i += 8)
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d + i), "f"(v[i]), "f"(v[i + 1]),
                     "f"(v[i + 2]), "f"(v[i + 3]), "f"(v[i + 4]), "f"(v[i + 5]), "f"(v[i + 6]), "f"(v[i + 7]) : "memory");
    } else {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<__nv_bfloat16*>(p.out) + t * p.out_stride + n),
                   "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (n + i < p.N) store_out(p, t, n + i, v[i]);
}

// Tile number -> its 256 tokens and 256 weight rows: tokens fastest within groups of `group` token tiles, so that the
// rows that pairs read at one time stay in L2.
__device__ __forceinline__ void pair_tile(const LinearParams& p, int i, int& tm, int& tn) {
  const int per = p.group * p.tiles_n;
  const int g = i / per, left = i - g * per;
  const int here = p.tiles_m - g * p.group < p.group ? p.tiles_m - g * p.group : p.group;
  tn = left / here;
  tm = g * p.group + left - tn * here;
}

__global__ void __launch_bounds__(PairCfg::kThreads, 1)
    fp8_linear_pair_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap ta,
                           const __grid_constant__ LinearParams p) {
  using C = PairCfg;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const uint32_t bars = base + C::oBars;
  auto full = [&](int s) { return bars + 8u * s; };                   // (the pair's first CTA)
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto acc_full = [&](int i) { return bars + 8u * (2 * C::kStages + i); };
  auto acc_free = [&](int i) { return bars + 8u * (2 * C::kStages + C::kAcc + i); };   // (the pair's first CTA)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank(), half = crank & 1u, lead_rank = crank & ~1u;
  const int part = static_cast<int>(crank >> 1);                      // pair of the cluster

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < C::kAcc; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_free(i), 16);
    }
    fence_mbar_init();
    prefetch_tensormap(&tw);
    prefetch_tensormap(&ta);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + C::oSlot), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  cluster_sync_all();                       // both CTAs' barriers and columns are there
  tmem_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + C::oSlot);
  griddep_launch_dependents();              // behind the allocation, as above
  griddep_wait();

  const int tiles = p.tiles_m * p.tiles_n;
  const int clusters = static_cast<int>(gridDim.x) / (2 * p.split), first = static_cast<int>(blockIdx.x) / (2 * p.split);
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.KB) * part / p.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.KB) * (part + 1) / p.split);
  bool ok = true;

  if (warp < 4) {
    regs_dec<C::kRegsCtl>();
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t full0 = cluster_addr(full(0), lead_rank);
        int s = 0;
        uint32_t ph = 0;
        for (int i = first; i < tiles && ok; i += clusters) {
          int tm, tn;
          pair_tile(p, i, tm, tn);
          const int tok = tm * 2 * C::kTok + static_cast<int>(half) * C::kTok, row = tn * C::kOut + static_cast<int>(half) * 128;
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(empty(s), ph ^ 1u)) { ok = false; break; }
            const uint32_t at = base + s * C::kStage, bar = full0 + 8u * s;
            if (half == 0) mbar_arrive_expect_tx(full(s), 2 * C::kStage);
            tma_load_2d_pair(at, &ta, kb * 128, tok, bar);
            tma_load_2d_pair(at + 128 * 128, &tw, kb * 128, row, bar);
            if (++s == C::kStages) { s = 0; ph ^= 1u; }
          }
        }
        // every stage has been read, so no copy is in flight, and no arrival from the products either
        for (int k = 0; k < C::kStages; ++k) {
          if (!mbar_wait(empty(s), ph ^ 1u)) ok = false;
          if (++s == C::kStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) set_flag(p.flags, MSA_FLAG_TIMEOUT);
      }
      __syncwarp();
    } else if (warp == 1 && half == 0) {
      constexpr uint32_t id = (mma_idesc(0, 0, C::kOut, 0, 0) & ~(0x1Fu << 24)) | ((256u >> 4) << 24), hi = desc_hi(1024, kSwz128);
      const uint32_t a0 = desc_lo(base, 16), b0 = desc_lo(base + 128 * 128, 16);
      const uint16_t mask = static_cast<uint16_t>(3u << lead_rank);
      const bool lead = elect_one();
      int s = 0, n = 0;
      uint32_t ph = 0;
      for (int i = first; i < tiles && ok; i += clusters) {
        for (int kb = kb0; kb < kb1; ++kb, ++n) {
          const int b = n & 1;
          ok = warp_wait(full(s), ph) && (n < C::kAcc || warp_wait(acc_free(b), ((n >> 1) - 1) & 1));
          if (!ok) break;
          tmem_fence_after();
          if (lead) {
            const uint32_t a = a0 + s * (C::kStage >> 4), w = b0 + s * (C::kStage >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_fp8_pair(tmem + b * C::kOut, desc_of(a + kk * 2, hi), desc_of(w + kk * 2, hi), id, kk > 0);
            mma_commit_pair(empty(s), mask);
            mma_commit_pair(acc_full(b), mask);
          }
          __syncwarp();
          if (++s == C::kStages) { s = 0; ph ^= 1u; }
        }
      }
      if (!ok && lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
    }
  } else {
    regs_inc<C::kRegsSum>();
    const int sub = warp & 3, col = (warp - 4) >> 2;                  // tensor-memory lanes, half of the columns
    const uint32_t mine = tmem + (static_cast<uint32_t>(sub) << 21) + col * 128;
    const uint32_t free0 = cluster_addr(acc_free(0), lead_rank);
    int n = 0;
    for (int i = first; i < tiles; i += clusters) {
      int tm, tn;
      pair_tile(p, i, tm, tn);
      const int64_t t = static_cast<int64_t>(tm) * 2 * C::kTok + half * C::kTok + sub * 32 + lane;
      const int blocks = (p.N + 127) / 128, wb = tn * 2 + col < blocks ? tn * 2 + col : blocks - 1;
      const float* sa = p.sa + (t < p.T ? t : 0) * p.KB;
      const float* sw = p.sw + static_cast<int64_t>(wb) * p.KB;
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.f;
      float s_next = sa[kb0], w_next = sw[kb0];
      // 32 columns at a time, the next ones on their way while the last are added, the next block's first among them
      float x[2][32];
      ok = ok && warp_wait(acc_full(n & 1), (n >> 1) & 1);
      tmem_fence_after();
      tmem_ld32(mine + (n & 1) * C::kOut, x[0]);
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        const int b = n & 1;
        const float f = s_next * w_next;
        const int after = kb + 1 < kb1 ? kb + 1 : kb;
        s_next = sa[after];
        w_next = sw[after];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_wait_ld32(x[c & 1]);
          if (c < 3) {
            tmem_ld32(mine + b * C::kOut + 32 * (c + 1), x[(c + 1) & 1]);
          } else {
            tmem_fence_before();
            if (lane == 0) mbar_arrive_relaxed(free0 + 8u * b);
            if (kb + 1 < kb1) {
              ok = ok && warp_wait(acc_full(b ^ 1), ((n + 1) >> 1) & 1);
              tmem_fence_after();
              tmem_ld32(mine + (b ^ 1) * C::kOut, x[0]);
            }
          }
#pragma unroll
          for (int u = 0; u < 32; u += 2) fma2(acc[32 * c + u], acc[32 * c + u + 1], x[c & 1][u], x[c & 1][u + 1], f);
        }
      }
      const int n0 = tn * C::kOut + col * 128;
      if (p.split == 1) {
        if (t < p.T) {
#pragma unroll
          for (int c = 0; c < 128; c += 16) store16(p, t, n0 + c, acc + c, p.wide);
        }
      } else {
        // The stages are done with: the last block's products are.
        float4* sums = reinterpret_cast<float4*>(sm + (sub * 32 + lane) * C::kSumRow + col * 128 * 4);
#pragma unroll
        for (int c = 0; c < 128; c += 4) sums[c / 4] = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
      }
    }
    if (!ok && lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  cluster_sync_all();                       // the pair is done with both CTAs' columns, barriers and stages
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if (p.split == 1) return;

  if (warp >= 4) {
    int tm, tn;
    pair_tile(p, first, tm, tn);
    const int64_t t0 = static_cast<int64_t>(tm) * 2 * C::kTok + half * C::kTok;
    // a warp takes half a token's row: 4 outputs per lane
    for (int i = part * 8 + warp - 4; i < 2 * C::kTok; i += p.split * 8) {
      const int r = i >> 1, c = (i & 1) * 128 + 4 * lane;
      if (t0 + r >= p.T) break;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int q = 0; q < p.split; ++q) {
        const float4 x = ld_cluster(base + r * C::kSumRow + c * 4, 2 * q + static_cast<int>(half));
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      store4(p, t0 + r, tn * C::kOut + c, v);
    }
  }
  cluster_sync_all();                       // no CTA ends while another reads its sums
}

// 2-D map over E4M3 rows [rows][K]: boxes of `box` rows x 128 bytes in the 128-byte swizzle, zeros outside.
static cudaError_t rows_map(CUtensorMap* map, const void* base, int64_t rows, int K, int box) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  memset(map, 0, sizeof(*map));
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t boxes[2] = {128, static_cast<cuuint32_t>(box)};
  const cuuint32_t ones[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int NT>
static cudaError_t launch_rows(const LinearArgs& a, LinearParams p, cudaStream_t stream, DispatchRecord* rec) {
  using C = RowsCfg<NT>;
  CUtensorMap tw, ta;
  cudaError_t err;
  if ((err = rows_map(&tw, a.w, a.N, a.K, kTile)) != cudaSuccess) return err;
  if ((err = rows_map(&ta, a.a, a.T, a.K, NT)) != cudaSuccess) return err;
  constexpr size_t smem = C::kTotal + 1024;
  err = cudaFuncSetAttribute(fp8_linear_rows_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  const int tiles = (a.N + kTile - 1) / kTile, groups = (a.T + NT - 1) / NT;
  int split = 1;
  while (split < 8 && split * 2 <= p.KB && static_cast<int64_t>(tiles) * groups * split < device_sm_count()) split *= 2;
  if (const char* force = getenv("MSA_LINEAR_SPLIT")) {
    const int s = atoi(force);
    if ((s == 1 || s == 2 || s == 4 || s == 8) && s <= p.KB) split = s;
  }
  p.split = split;
  err = launch_pdl_cluster(fp8_linear_rows_kernel<NT>, dim3(tiles * split, groups), dim3(C::kThreads), smem, stream, split, tw, ta, p);
  if (err != cudaSuccess) return err;
  rec->set("fp8_linear rows tokens=%d grid=%dx%d split=%d", NT, tiles * split, groups, split);
  return cudaGetLastError();
}

static cudaError_t launch_pairs(const LinearArgs& a, LinearParams p, cudaStream_t stream, DispatchRecord* rec) {
  using C = PairCfg;
  CUtensorMap tw, ta;
  cudaError_t err;
  if ((err = rows_map(&tw, a.w, a.N, a.K, 128)) != cudaSuccess) return err;
  if ((err = rows_map(&ta, a.a, a.T, a.K, 128)) != cudaSuccess) return err;
  constexpr size_t smem = C::kTotal + 1024;
  err = cudaFuncSetAttribute(fp8_linear_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  p.tiles_m = (a.T + 2 * C::kTok - 1) / (2 * C::kTok);
  p.tiles_n = (a.N + C::kOut - 1) / C::kOut;
  const int64_t rows = (32ll << 20) / (2 * C::kTok * static_cast<int64_t>(a.K));
  p.group = rows < 1 ? 1 : rows > p.tiles_m ? p.tiles_m : static_cast<int>(rows);
  p.wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && (a.out_stride * (a.out_f32 ? 4 : 2)) % 32 == 0;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (tiles > INT32_MAX / 16) return cudaErrorInvalidValue;
  const int pairs = device_sm_count() / 2;
  int split = 1;
  while (split < 4 && split * 2 <= p.KB && tiles * split * 2 <= pairs) split *= 2;
  if (const char* force = getenv("MSA_LINEAR_SPLIT")) {
    const int s = atoi(force);
    if ((s == 1 || s == 2 || s == 4) && s <= p.KB) split = s;
  }
  p.split = split;
  const int64_t clusters = split > 1 ? tiles : tiles < pairs ? tiles : pairs;
  err = launch_pdl_cluster(fp8_linear_pair_kernel, dim3(static_cast<unsigned>(clusters * 2 * split)), dim3(C::kThreads), smem, stream,
                           2 * split, tw, ta, p);
  if (err != cudaSuccess) return err;
  rec->set("fp8_linear pairs tiles=%dx%d grid=%lld split=%d", p.tiles_m, p.tiles_n, static_cast<long long>(clusters * 2 * split), split);
  return cudaGetLastError();
}

cudaError_t launch_fp8_linear(const LinearArgs& a, cudaStream_t stream, DispatchRecord* rec) {
  LinearParams p;
  memset(&p, 0, sizeof(p));
  p.sa = a.sa;
  p.sw = a.sw;
  p.out = a.out;
  p.flags = a.flags;
  p.out_stride = a.out_stride;
  p.T = a.T; p.N = a.N; p.KB = (a.K + kTile - 1) / kTile;
  p.f32 = a.out_f32;
  p.quads = a.out_stride % 4 == 0;                       // (out itself is 16-byte aligned)
  bool pairs = a.T > 128;
  if (const char* form = getenv("MSA_LINEAR_FORM")) pairs = strcmp(form, "pairs") == 0 ? true : strcmp(form, "rows") == 0 ? false : pairs;
  if (pairs) return launch_pairs(a, p, stream, rec);
  if (a.T <= 16) return launch_rows<16>(a, p, stream, rec);
  if (a.T <= 32) return launch_rows<32>(a, p, stream, rec);
  if (a.T <= 64) return launch_rows<64>(a, p, stream, rec);
  return launch_rows<128>(a, p, stream, rec);
}

}  // namespace msa
