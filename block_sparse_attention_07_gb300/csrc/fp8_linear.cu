// Projection of FP8 rows: both operands E4M3 with fp32 scales per block of 128.
//
// "MiniMax-M3.1-Flash Day-0 対応" (aisoku.org), section "最適化と数値": the fused
// projection in front of norm, rotary embedding and insert; the pages give no
// formula. With g the blocks of 128 along K,
//   out[t, n] = sum_g sa[t, g] sw[n / 128, g] sum_{k in g} a[t, k] w[n, k].
// The inner sum is one tcgen05 product of K = 128 into tensor memory, fresh for
// every block; the outer one is kept in fp32 registers, which read the block's
// sums back and add them times their scales' product, an fp32 value: one fused
// addition per sum (the scales one after the other would be two operations, for
// the sake of products below 2^-126). Blocks of K beyond its end and rows beyond
// the operands' arrive as zeros.
//
// What bounds it: the weights' bytes where there are many and few tokens (64 x
// 100,003 x 4,096 to fp32: 71.7 us, 6.1 TB/s with the outputs); launch, first copies
// and the sums' way between CTAs where there are few (1 x 1,280 x 4,096: 3.8 us);
// in between a block's chain of copy, product and sums (256 x 4,096 x 8,192:
// 13.1 us); from some 400 tokens to 2,048 the last wave of tiles, which costs as much
// as a full one (512 x 10,240 x 4,096, 80 tiles on 76 pairs: 30.7 us); for prompts
// the products with the sums' way back beside them (8,191 x 10,240 x 4,096: 234 us,
// 2.94 PFLOP/s; 260 in a run of a second, where the board's power limit takes the
// clock to 1.75 GHz).
#include <cstdlib>
#include <cstring>

#include "at_once.h"
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
  int quads, boxed;             // rows of the output start on boundaries of four values, of 16 bytes
  int whole;                    // boxed: the columns in front of a row's last, unfinished 16 bytes
};

// Asks for a tile of a tensor map in L2. It reads nothing that a later write could make stale: L2 is where all SMs meet.
__device__ __forceinline__ void prefetch_2d(const void* tmap, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tmap), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The two halves of it: what a thread has read and written in front of the first is done for those behind the second. The
// relaxed one is for a thread whose accesses another thread's release covers.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr), "r"(rank));
  return at;
}
// Copies shared memory to another CTA's, completed on a barrier there.
__device__ __forceinline__ void bulk_to_cluster(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "r"(src), "r"(bytes), "r"(bar) : "memory");
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

__device__ __forceinline__ float4 ld_shared4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
// 16 bytes of another CTA's shared memory.
__device__ __forceinline__ float4 ld_cluster(uint32_t saddr, int rank) {
  const uint32_t at = cluster_addr(saddr, rank);
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
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

// A tile's outputs from the sums of a CTA that has it by itself. Thread `me` of kThreads takes four outputs of a row, eight
// times at one time: with all the sums on their way together 128 x 10,240 x 4,096 takes 13.0 us, one after the other 15.6.
template <int kThreads, typename Place>
__device__ __forceinline__ void store_sums(const LinearParams& p, uint32_t base, Place place, int tokens, int tok0, int row0, int me) {
  constexpr int kAhead = 8;
  const int all = tokens * (kTile / 4);
  for (int i0 = me; i0 < all; i0 += kAhead * kThreads) {
    float4 v[kAhead];
    auto live = [&](int b) { return i0 + b * kThreads < all && row0 + 4 * ((i0 + b * kThreads) & 31) < p.N; };
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      const int i = i0 + b * kThreads;
      v[b] = live(b) ? ld_shared4(base + place(i >> 5, i & 31) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      const int i = i0 + b * kThreads;
      if (live(b)) store4(p, tok0 + (i >> 5), row0 + 4 * (i & 31), v[b]);
    }
  }
}

// A CTA's share of a tile's outputs, from the sums of the `split` <= kMost CTAs of its cluster, added in rank order. Thread `me`
// of kThreads takes four outputs of a row, kPer times, kAhead of them at one time: with two CTAs four are 0.5 us shorter than one
// (256 x 4,096 x 8,192), more CTAs have enough on their way with one (64 x 4,096 x 8,192 on four: 9.6 and 9.7).
// No CTA may end while another reads its sums, so behind its last read a thread arrives at the cluster's last meeting, with
// release, which waits for what the thread has under way: so in front of its stores. With many outputs the releases of all warps
// take long too (256 x 4,096 x 8,192 14.9 us); there the threads arrive at a barrier of the CTA, and one warp, which has
// nothing else under way, behind that with release for all (13.1, as much as without order, which holds on the hardware but is
// not promised; 64 x 10,240 x 4,096 11.8, 11.7, without order 11.4). With few outputs every thread by itself is shorter (16 x
// 1,280 x 4,096 4.1 us, by one warp 4.3, without order 4.05).
template <int kMost, int kAhead, int kTokens, int kThreads, bool kByOne, typename Place>
__device__ __forceinline__ void join_sums(const LinearParams& p, uint32_t base, Place place, int tokens, int tok0, int row0, int rank,
                                          int me) {
  constexpr int kFewest = kMost == 2 ? 2 : kMost / 2 + 1;             // the fewest CTAs that come here
  constexpr int kPer = (kTokens * (kTile / 4) + kFewest * kThreads - 1) / (kFewest * kThreads);
  const int hop = p.split * kThreads, all = tokens * (kTile / 4), i0 = rank * kThreads + me;
  auto live = [&](int j) { return i0 + j * hop < all && row0 + 4 * ((i0 + j * hop) & 31) < p.N; };
  float4 v[kPer];
#pragma unroll
  for (int j0 = 0; j0 < kPer; j0 += kAhead) {
    float4 x[kAhead][kMost];
#pragma unroll
    for (int b = 0; b < kAhead && j0 + b < kPer; ++b)
#pragma unroll
      for (int q = 0; q < kMost; ++q) {
        const int i = i0 + (j0 + b) * hop;
        x[b][q] = q < p.split && live(j0 + b) ? ld_cluster(base + place(i >> 5, i & 31) * 4, q) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
    for (int b = 0; b < kAhead && j0 + b < kPer; ++b) {
      float4& s = v[j0 + b];
      s = x[b][0];
#pragma unroll
      for (int q = 1; q < kMost; ++q) { s.x += x[b][q].x; s.y += x[b][q].y; s.z += x[b][q].z; s.w += x[b][q].w; }
    }
  }
  if (kByOne) {
    __syncwarp();
    asm volatile("bar.arrive 2, %0;" ::"n"(kThreads + 32) : "memory");
    cluster_arrive_relaxed();
  } else {
    cluster_arrive();
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = i0 + j * hop;
    if (live(j)) store4(p, tok0 + (i >> 5), row0 + 4 * (i & 31), v[j]);
  }
}

// ---------------------------------------------------------------------------
// One CTA per tile of 128 weight rows and up to NT tokens; the CTAs of a cluster
// share the tile's K and add their sums through distributed shared memory, in rank
// order. Up to 64 tokens the weights are the product's M, so that few tokens waste
// nothing but columns: a thread has a weight row and up to 32 tokens, whose scales
// it reads from shared memory. With 128 tokens those reads are as many bytes as the
// copies and the products take together, so the tokens are M: a thread has a token,
// 64 weight rows and one scale per block of K (256 x 4,096 x 8,192 then: 17.6 -> 14.4 us;
// 64 tokens as M, half of the product's rows unused: 64 x 100,003 x 4,096 72.4 -> 76.3).
// Up to 64 tokens there are two sizes: two CTAs per SM, or one with as much memory for copies in flight. kDeep: the latter.
template <int NT, bool kDeep>
struct RowsCfg {
  static constexpr bool kTokM = NT == 128;
  static constexpr int kWide = kTokM ? kTile : NT;                    // a block's columns in tensor memory
  static constexpr int kPer = kTokM ? 64 : NT < 32 ? NT : 32;         // a thread's columns
  static constexpr int kSumThreads = 128 * (kWide / kPer), kThreads = kSumThreads + 64;
  static constexpr int kCopyWarp = kSumThreads / 32, kMmaWarp = kCopyWarp + 1;
  static constexpr int kCtas = kDeep ? 1 : 2;                         // per SM
  // Blocks that are read back at one time, as far as registers go (64 x 4,096 x 8,192 by twos: 11.8 -> 11.1 us), and how
  // many times as many are in tensor memory.
  static constexpr int kTake = kTokM || (NT == 64 && !kDeep) ? 1 : 2, kSets = 4 / kTake;
  static constexpr int kLoads = kTokM ? 2 : kTake;                    // the reads for it
  static constexpr uint32_t kCols = kSets * kTake * kWide;
  static constexpr int kStages = NT == 128 ? 6 : kDeep ? (NT == 16 ? 11 : NT == 32 ? 10 : 8) : NT == 64 ? 4 : 5;
  static_assert(kDeep || !kTokM, "128 tokens fill an SM");
  static constexpr uint32_t kStage = (kTile + NT) * 128;              // tokens, then weights
  static constexpr int kRow = NT + 4;                                 // floats of a scale row: 16-byte steps, spread over banks
  static constexpr uint32_t oTable = kStages * kStage;
  static constexpr uint32_t oBars = oTable + 2 * kChunk * kRow * 4;
  static constexpr int kBars = 2 * kStages + 2 * kSets;
  static constexpr uint32_t oSlot = oBars + kBars * 8;
  static constexpr uint32_t kTotal = oSlot + 16;
  static_assert(kChunk % kTake == 0, "blocks that are read together have their scales in one half of the table");
  static_assert(NT * kTile * 4 <= kStages * kStage, "the sums of a tile fit into the stages");
  static_assert(kCols >= 32 && kCols * kCtas <= 512, "tensor memory");
};

template <int NT, bool kDeep>
__global__ void __launch_bounds__(RowsCfg<NT, kDeep>::kThreads, RowsCfg<NT, kDeep>::kCtas)
    fp8_linear_rows_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap ta,
                           const __grid_constant__ LinearParams p) {
  using C = RowsCfg<NT, kDeep>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  float* table = reinterpret_cast<float*>(sm + C::oTable);
  float* sums = reinterpret_cast<float*>(sm);                         // over the stages when they are done
  const uint32_t bars = base + C::oBars;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto acc_full = [&](int i) { return bars + 8u * (2 * C::kStages + i); };
  auto acc_free = [&](int i) { return bars + 8u * (2 * C::kStages + C::kSets + i); };
  // Four weight rows of a token, in 16 bytes. With a token per lane they are spread over the banks.
  auto place = [](int t, int quad) { return t * kTile + 4 * (C::kTokM ? quad ^ (t & 31) : quad); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < C::kSets; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_free(i), C::kSumThreads / 32);
    }
    fence_mbar_init();
    prefetch_tensormap(&tw);
    prefetch_tensormap(&ta);
  }
  if (warp == C::kMmaWarp) {
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
  const int rank = static_cast<int>(blockIdx.x) % p.split, tile = static_cast<int>(blockIdx.x) / p.split;
  const int tok0 = static_cast<int>(blockIdx.y) * NT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.KB) * rank / p.split);
  const int n = static_cast<int>(static_cast<int64_t>(p.KB) * (rank + 1) / p.split) - kb0;
  // While the kernel before ends: the first weights on their way to L2.
  if (threadIdx.x == 0)
    for (int i = 0; i < C::kStages && i < n; ++i) prefetch_2d(&tw, (kb0 + i) * kTile, tile * kTile);
  griddep_wait();

  bool ok = true;

  if (warp == C::kCopyWarp) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      for (int i = 0; i < n; ++i) {
        if (!mbar_wait(empty(s), ph ^ 1u)) { ok = false; break; }
        const uint32_t at = base + s * C::kStage;
        mbar_arrive_expect_tx(full(s), C::kStage);
        tma_load_2d(at + NT * 128, &tw, (kb0 + i) * kTile, tile * kTile, full(s));
        tma_load_2d(at, &ta, (kb0 + i) * kTile, tok0, full(s));
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
      // no copy may be in flight when the CTA ends, whatever the others did
      for (int k = 0; k < C::kStages; ++k) mbar_wait(full(k), ph ^ (k < s ? 0u : 1u));
      if (!ok) set_flag(p.flags, MSA_FLAG_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == C::kMmaWarp) {
    constexpr uint32_t id = mma_idesc(0, 0, C::kWide, 0, 0), hi = desc_hi(1024, kSwz128);
    const uint32_t m0 = desc_lo(base + (C::kTokM ? 0 : NT * 128), 16), n0 = desc_lo(base + (C::kTokM ? NT * 128 : 0), 16);
    if (elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      for (int i = 0; i < n; ++i) {
        const int set = i / C::kTake, b = set % C::kSets, in = i % C::kTake;
        if (in == 0 && set >= C::kSets && !mbar_wait(acc_free(b), (set / C::kSets - 1) & 1)) { ok = false; break; }
        if (!mbar_wait(full(s), ph)) { ok = false; break; }
        tmem_fence_after();
        const uint32_t at = s * (C::kStage >> 4), d = tmem + (b * C::kTake + in) * C::kWide;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_fp8(d, desc_of(m0 + at + kk * 2, hi), desc_of(n0 + at + kk * 2, hi), id, kk > 0);
        mma_commit(empty(s));
        if (in == C::kTake - 1 || i == n - 1) mma_commit(acc_full(b));
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
      if (!ok) set_flag(p.flags, MSA_FLAG_TIMEOUT);
    }
    __syncwarp();
  } else {
    // A block's sums, times its two scales, onto the thread's own.
    const int sub = warp & 3, part = warp >> 2;                       // tensor-memory lanes, part of the columns
    constexpr int kFetch = NT * kChunk / C::kSumThreads;
    const float* sw = p.sw + static_cast<int64_t>(tile) * p.KB + kb0;
    static_assert(C::kSumThreads % kChunk == 0, "a thread fetches scales of one block");
    float next[kFetch], next_w;
    auto fetch = [&](int c) {               // (multiplied when they are kept: a product here would wait for the loads)
      const int i = c * kChunk + threadIdx.x % kChunk;
      next_w = i < n ? sw[i] : 0.f;
#pragma unroll
      for (int j = 0; j < kFetch; ++j) {
        const int t = (threadIdx.x + C::kSumThreads * j) / kChunk;
        next[j] = i < n && tok0 + t < p.T ? p.sa[static_cast<int64_t>(tok0 + t) * p.KB + kb0 + i] : 0.f;
      }
    };
    auto keep = [&](int c) {
#pragma unroll
      for (int j = 0; j < kFetch; ++j) {
        const int e = threadIdx.x + C::kSumThreads * j;
        table[((c & 1) * kChunk + e % kChunk) * C::kRow + e / kChunk] = next[j] * next_w;
      }
    };
    float acc[C::kPer];
#pragma unroll
    for (int t = 0; t < C::kPer; ++t) acc[t] = 0.f;
    fetch(0);
    keep(0);
    named_barrier(1, C::kSumThreads);
    const uint32_t mine = tmem + (static_cast<uint32_t>(sub) << 21) + part * C::kPer;
    for (int i = 0; i < n; i += C::kTake) {
      const int set = i / C::kTake, b = set % C::kSets, c = i / kChunk, j = i % kChunk;
      if (j == 0 && c > 0) {
        keep(c);                            // the other half: every thread is behind the barrier of its last use
        named_barrier(1, C::kSumThreads);
      }
      if (j == 0) fetch(c + 1);
      const float* scale = table + ((c & 1) * kChunk + j) * C::kRow + (C::kTokM ? sub * 32 + lane : part * C::kPer);
      const float f = C::kTokM ? *scale : 0.f;
      if (ok && !mbar_wait(acc_full(b), (set / C::kSets) & 1)) ok = false;
      __syncwarp();
      tmem_fence_after();
      float x[C::kLoads][32];
#pragma unroll
      for (int q = 0; q < C::kLoads; ++q) {
        const uint32_t at = mine + b * C::kTake * C::kWide + q * (C::kTokM ? 32 : C::kWide);
        if (NT == 16) tmem_ld16(at, x[q]);
        else tmem_ld32(at, x[q]);
#pragma unroll
        for (int u = NT == 16 ? 16 : 32; u < 32; ++u) x[q][u] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < C::kLoads; ++q) tmem_wait_ld32(x[q]);
      tmem_fence_before();
      if (lane == 0) mbar_arrive(acc_free(b));
#pragma unroll
      for (int q = 0; q < C::kLoads; ++q) {
        if constexpr (C::kTokM) {
#pragma unroll
          for (int u = 0; u < 32; u += 2) fma2(acc[32 * q + u], acc[32 * q + u + 1], x[q][u], x[q][u + 1], f);
        } else if (i + q < n) {             // (behind an odd number of blocks: an older one's columns, or nothing's)
#pragma unroll
          for (int u = 0; u < C::kPer; u += 4) {
            const float4 v = *reinterpret_cast<const float4*>(scale + q * C::kRow + u);
            fma2(acc[u], acc[u + 1], x[q][u], x[q][u + 1], v.x, v.y);
            fma2(acc[u + 2], acc[u + 3], x[q][u + 2], x[q][u + 3], v.z, v.w);
          }
        }
      }
    }
    if (!ok && lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
    const int row = sub * 32 + lane;
    if constexpr (C::kTokM) {
#pragma unroll
      for (int u = 0; u < C::kPer; u += 4)
        *reinterpret_cast<float4*>(sums + place(row, part * (C::kPer / 4) + u / 4)) = make_float4(acc[u], acc[u + 1], acc[u + 2], acc[u + 3]);
    } else {
      const int tok = part * C::kPer;
      if (p.split == 1) {
        const bool in = tile * kTile + row < p.N;
#pragma unroll
        for (int t = 0; t < C::kPer; ++t)
          if (in && tok0 + tok + t < p.T) store_out(p, tok0 + tok + t, tile * kTile + row, acc[t]);
      } else {
#pragma unroll
        for (int t = 0; t < C::kPer; ++t) sums[(tok + t) * kTile + row] = acc[t];
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  // (Without a barrier of the CTA in front of the cluster's: 64 x 4,096 x 8,192 10.1 -> 9.7 us.)
  if (p.split > 1) cluster_sync_all();      // every CTA's sums are written, and tensor memory has been read
  else __syncthreads();
  if (warp == C::kMmaWarp) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
  }
  if (!C::kTokM && p.split == 1) return;

  const int tokens = p.T - tok0 < NT ? p.T - tok0 : NT;
  // With many outputs without the warp that has just given tensor memory back (128 x 4,096 x 8,192 on two CTAs: 13.5 -> 13.3 us); with
  // few the others would take a turn more (16 x 4,096 x 8,192: 8.2 -> 8.5).
  constexpr bool kByOne = NT >= 64;
  constexpr int kStore = kByOne ? C::kThreads - 32 : C::kThreads;
  static_assert(C::kMmaWarp * 32 == C::kThreads - 32, "the warp that does not store");
  const int row0 = tile * kTile, me = threadIdx.x;
  if (C::kTokM && p.split == 1) {
    if (me < kStore) store_sums<kStore>(p, base, place, tokens, tok0, row0, me);
    return;
  }
  if (me >= kStore) {
    __syncwarp();
    named_barrier(2, kStore + 32);          // the others have read
    cluster_arrive();
  } else if (p.split == 2) {
    join_sums<2, 4, NT, kStore, kByOne>(p, base, place, tokens, tok0, row0, rank, me);
  } else if (p.split <= 4) {
    join_sums<4, 1, NT, kStore, kByOne>(p, base, place, tokens, tok0, row0, rank, me);
  } else {
    join_sums<8, 1, NT, kStore, kByOne>(p, base, place, tokens, tok0, row0, rank, me);
  }
  cluster_wait();
}

// ---------------------------------------------------------------------------
// Tokens as M, two CTAs of a cluster on one tile: 256 tokens x 256 weight rows per
// pair, each CTA with its 128 tokens' sums in tensor memory and half of the weight
// rows in shared memory, so that a block of K costs a CTA 32 KB of copies for 512
// cycles of tensor core. The first CTA's warp issues for both. Thread = token: one
// product of scales per block of K serves its 128 outputs. With few tiles, `split`
// pairs of a cluster share a tile's K, and each finishes every split-th 16 columns
// from the sums that the others copy there; otherwise a pair walks over the tiles.
// A block takes some 810 cycles; without reading its sums back 710, as far as the
// power limit lets the products go (8,191 x 10,240 x 4,096: 233 and 204 us).
struct PairCfg {
  static constexpr int kTok = 128, kOut = 256;                        // a CTA's tokens, a tile's weight rows
  static constexpr int kStages = 5, kAcc = 2;
  static constexpr uint32_t kStage = 2 * 128 * 128;
  static constexpr uint32_t oOut = kStages * kStage, kOutBuf = 32 * 128;   // 128 bytes of 32 rows per warp on their way out
  static constexpr uint32_t oBars = oOut + 8 * kOutBuf;
  static constexpr int kBars = 2 * kStages + 2 * kAcc + 1;
  static constexpr uint32_t oSlot = oBars + kBars * 8;
  static constexpr uint32_t kTotal = oSlot + 16;
  static constexpr int kThreads = 384;                                // 4 control warps, 8 that hold the sums
  static constexpr int kRegsCtl = 40, kRegsSum = 232;
  static_assert(128 * kRegsCtl + 256 * kRegsSum <= 384 * 168, "registers of the launch");
  // With a split, 16 columns are a unit of sums: 4 columns of 128 tokens in a row, four times.
  static constexpr int kUnits = kOut / 16;
  static constexpr uint32_t kUnit = 16 * kTok * 4;
};
constexpr int pair_share(int part, int split) { return (PairCfg::kUnits - part + split - 1) / split; }   // units of a pair
constexpr bool pair_sums_fit(int split) {             // those that leave a CTA, and those that come
  const int most = pair_share(0, split);
  return 2 * (split - 1) * most * PairCfg::kUnit <= PairCfg::oBars;
}
static_assert(pair_sums_fit(2) && pair_sums_fit(3) && pair_sums_fit(4), "the others' sums fit into the stages and the buffers behind them");

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Waits on barriers that other CTAs of the cluster, their copies or their products arrive on: mbar_wait with the cluster as
// scope. kData: shared memory that was written in front of the arrival is read or written again behind the wait, which a fence
// for shared memory alone orders (an acquiring wait, for all memory: 8,191 x 10,240 x 4,096 235 -> 245 us). Without, the wait is
// for execution alone: the order of tensor memory's reads and products is that of tcgen05's fences on both sides.
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
template <bool kData>
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity) {
  bool ok = try_wait_cluster(bar, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    do {
#pragma unroll 1
      for (int k = 0; k < 64 && !ok; ++k) ok = try_wait_cluster(bar, parity);
    } while (!ok && globaltimer_ns() - t0 <= kWaitLimitNs);
  }
  if (kData && ok) asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
  return ok;
}
template <bool kData>
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity) {
  return __all_sync(kEvery, mbar_wait_cluster<kData>(bar, parity)) != 0;
}
// Says that tensor memory has been read: what was read is in registers, and nothing was written that the other CTA
// would have to see, so the arrival needs no release (whose fence costs a microsecond). The order of the reads and the next
// products is that of tcgen05.fence::before_thread_sync in front of it and ::after_thread_sync behind the other CTA's wait.
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
// Shared memory to a tile of a tensor map, rows and columns outside it left out.
__device__ __forceinline__ void tma_store_2d(const void* tmap, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
               ::"l"(tmap), "r"(x), "r"(y), "r"(src) : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until the copies out that this thread has issued have read their shared memory.
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void st_shared16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
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
// Sixteen outputs of a row in a row.
__device__ __forceinline__ void store16(const LinearParams& p, int64_t t, int n, const float* v) {
  if (!p.boxed || n + 16 > p.N) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (n + i < p.N) store_out(p, t, n + i, v[i]);
  } else if (p.f32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + t * p.out_stride + n);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    uint4* d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + t * p.out_stride + n);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      d[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                        pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
  }
}

// The columns from p.whole on, of a row that lies at `row_at` of shared memory in 16-byte places swizzled by `swz`, from
// column x0 on.
__device__ __forceinline__ void store_rest(const LinearParams& p, int64_t t, uint32_t row_at, uint32_t swz, int x0) {
  uint32_t w[4];
  const uint32_t at = row_at + ((static_cast<uint32_t>((p.whole - x0) / (p.f32 ? 4 : 8)) ^ swz) << 4);
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
  const int left = p.N - p.whole;
  if (p.f32) {
    uint32_t* d = static_cast<uint32_t*>(p.out) + t * p.out_stride + p.whole;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < left) d[i] = w[i];
  } else {
    uint16_t* d = static_cast<uint16_t*>(p.out) + t * p.out_stride + p.whole;
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) d[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
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
                           const __grid_constant__ CUtensorMap to, const __grid_constant__ LinearParams p) {
  using C = PairCfg;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const uint32_t bars = base + C::oBars;
  auto full = [&](int s) { return bars + 8u * s; };                   // (the pair's first CTA)
  auto empty = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto acc_full = [&](int i) { return bars + 8u * (2 * C::kStages + i); };
  auto acc_free = [&](int i) { return bars + 8u * (2 * C::kStages + C::kAcc + i); };   // (the pair's first CTA)
  const uint32_t got_bar = bars + 8u * (2 * C::kStages + 2 * C::kAcc);
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
    mbar_init(got_bar, 1);
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
            if (!mbar_wait_cluster<true>(empty(s), ph ^ 1u)) { ok = false; break; }
            const uint32_t at = base + s * C::kStage, bar = full0 + 8u * s;
            if (half == 0) mbar_arrive_expect_tx(full(s), 2 * C::kStage);
            tma_load_2d_pair(at, &ta, kb * 128, tok, bar);
            tma_load_2d_pair(at + 128 * 128, &tw, kb * 128, row, bar);
            if (++s == C::kStages) { s = 0; ph ^= 1u; }
          }
        }
        // every stage has been read, so no copy is in flight, and no arrival from the products either
        for (int k = 0; k < C::kStages; ++k) {
          if (!mbar_wait_cluster<true>(empty(s), ph ^ 1u)) ok = false;
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
          ok = warp_wait_cluster<true>(full(s), ph) && (n < C::kAcc || warp_wait_cluster<false>(acc_free(b), ((n >> 1) - 1) & 1));
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
    const int sub = warp & 3, g = (warp - 4) >> 2;                    // tensor-memory lanes, half of the columns
    const uint32_t mine = tmem + (static_cast<uint32_t>(sub) << 21) + g * 128;
    const uint32_t free0 = cluster_addr(acc_free(0), lead_rank);
    const uint32_t out_at = base + C::oOut + (warp - 4) * C::kOutBuf;
    const int blocks = (p.N + 127) / 128;
    int n = 0, tm, tn;
    const float* sa = nullptr;
    const float* sw = nullptr;
    float s_next = 0.f, w_next = 0.f;
    auto token = [&]() { return static_cast<int64_t>(tm) * 2 * C::kTok + half * C::kTok + sub * 32 + lane; };
    auto enter = [&](int i) {                 // the tile's places; its first scales on their way, in front of the last tile's stores
      pair_tile(p, i, tm, tn);
      const int wb = tn * 2 + g < blocks ? tn * 2 + g : blocks - 1;   // (a half without weight rows: any scale)
      sa = p.sa + (token() < p.T ? token() : 0) * p.KB;
      sw = p.sw + static_cast<int64_t>(wb) * p.KB;
      s_next = sa[kb0];
      w_next = sw[kb0];
    };
    enter(first);
    for (int i = first; i < tiles; i += clusters) {
      const int64_t t = token();
      const int n0 = tn * C::kOut + g * 128;
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.f;
      // 32 columns at a time, the next ones on their way while the last are added, the next block's first among them
      float x[2][32];
      ok = ok && warp_wait_cluster<false>(acc_full(n & 1), (n >> 1) & 1);
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
              ok = ok && warp_wait_cluster<false>(acc_full(b ^ 1), ((n + 1) >> 1) & 1);     // one answer per warp: the next tile's wait votes
              tmem_fence_after();
              tmem_ld32(mine + (b ^ 1) * C::kOut, x[0]);
            }
          }
#pragma unroll
          for (int u = 0; u < 32; u += 2) fma2(acc[32 * c + u], acc[32 * c + u + 1], x[c & 1][u], x[c & 1][u + 1], f);
        }
      }
      if (i + clusters < tiles) enter(i + clusters);
      if (p.split == 1 && p.boxed) {
        // 128 bytes of every row at a time, swizzled as the tensor map has them
        const int row0 = static_cast<int>(t) - lane;
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          const int x0 = n0 + c, chunk = p.f32 ? 0 : (c & 32) / 8;
          if (p.f32 || (c & 32) == 0) {
            tma_store_read();
            __syncwarp();
          }
          if (p.f32) {
#pragma unroll
            for (int u = 0; u < 32; u += 4)
              st_shared16(out_at + lane * 128 + (((u >> 2) ^ (lane & 7)) << 4), __float_as_uint(acc[c + u]),
                          __float_as_uint(acc[c + u + 1]), __float_as_uint(acc[c + u + 2]), __float_as_uint(acc[c + u + 3]));
          } else {
#pragma unroll
            for (int u = 0; u < 32; u += 8)
              st_shared16(out_at + lane * 128 + (((chunk + (u >> 3)) ^ (lane & 7)) << 4), pack_bf16x2(acc[c + u], acc[c + u + 1]),
                          pack_bf16x2(acc[c + u + 2], acc[c + u + 3]), pack_bf16x2(acc[c + u + 4], acc[c + u + 5]),
                          pack_bf16x2(acc[c + u + 6], acc[c + u + 7]));
          }
          if (p.f32 || (c & 32) != 0) {
            smem_to_async();
            __syncwarp();
            const int at = p.f32 ? x0 : x0 - 32, cols = p.f32 ? 32 : 64;
            if (lane == 0 && row0 < p.T && at < p.whole) tma_store_2d(&to, at, row0, out_at);
            // Tensor copies write 16 bytes at least: what is left of the row, by its thread.
            if (p.whole < p.N && p.whole >= at && p.whole < at + cols && t < p.T) store_rest(p, t, out_at + lane * 128, lane & 7, at);
          }
        }
      } else if (p.split == 1) {
        if (t < p.T) {
#pragma unroll
          for (int c = 0; c < 128; c += 16) store16(p, t, n0 + c, acc + c);
        }
      } else {
        // Unit u of 16 columns belongs to pair u mod split, as its number u / split: the others' sums of it go there, by
        // one copy of shared memory per CTA.
        const int most = pair_share(0, p.split), own = pair_share(part, p.split), row = sub * 32 + lane;
        const uint32_t box = most * C::kUnit, got0 = (p.split - 1) * box;
        auto unit = [&](int u) { return g * 8 + u; };
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int q = unit(u) % p.split, k = unit(u) / p.split;
          if (q != part) {
            float4* d = reinterpret_cast<float4*>(sm + (q < part ? q : q - 1) * box + k * C::kUnit) + row;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              d[c * C::kTok] = make_float4(acc[16 * u + 4 * c], acc[16 * u + 4 * c + 1], acc[16 * u + 4 * c + 2], acc[16 * u + 4 * c + 3]);
          }
        }
        if (warp == 4 && lane == 0) mbar_arrive_expect_tx(got_bar, (p.split - 1) * own * C::kUnit);
        smem_to_async();
        tmem_fence_before();
        cluster_sync_all();                 // every CTA's sums are written, and what lies behind them is free
        if (warp == 4 && lane < p.split && lane != part) {
          const int slot = part < lane ? part : part - 1;
          const uint32_t to = 2 * lane + half;
          bulk_to_cluster(cluster_addr(base + got0 + slot * box, to), base + (lane < part ? lane : lane - 1) * box,
                          pair_share(lane, p.split) * C::kUnit, cluster_addr(got_bar, to));
        }
        __syncwarp();
        if (!warp_wait_cluster<true>(got_bar, 0)) {
          ok = false;
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int q = unit(u) % p.split, k = unit(u) / p.split;
            if (q == part) {
              for (int j = 0; j + 1 < p.split; ++j) {
                const float4* got = reinterpret_cast<const float4*>(sm + got0 + j * box + k * C::kUnit) + row;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const float4 v = got[c * C::kTok];
                  acc[16 * u + 4 * c] += v.x; acc[16 * u + 4 * c + 1] += v.y;
                  acc[16 * u + 4 * c + 2] += v.z; acc[16 * u + 4 * c + 3] += v.w;
                }
              }
              if (t < p.T) store16(p, t, n0 + 16 * u, acc + 16 * u);
            }
          }
        }
      }
    }
    if (!ok && lane == 0) set_flag(p.flags, MSA_FLAG_TIMEOUT);
  }
  __syncwarp();
  tmem_fence_before();
  if (warp >= 4) tma_store_read();          // (the thread that issued them)
  if (p.split > 1 && warp < 4) cluster_sync_all();                   // (the other warps have been through it)
  cluster_sync_all();                       // the cluster is done with all columns, barriers, stages and sums
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
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

// 2-D map over the output [T] rows of N (whole 16 bytes), `stride` bytes apart: boxes of 32 rows x 128 bytes in the 128-byte swizzle.
static cudaError_t out_map(CUtensorMap* map, void* base, int64_t T, int64_t N, int64_t stride, bool f32) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t boxes[2] = {f32 ? 32u : 64u, 32};
  const cuuint32_t ones[2] = {1, 1};
  const CUresult r = fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides,
                        boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Clusters of n CTAs of a kernel that the device runs at one time, asked once per device: fewer than its SMs would
// hold, 36 clusters of four and 15 of eight CTAs on 152 SMs. (It counts one CTA per SM for these kernels; where two
// fit, there is room for twice as many.)
template <typename Kernel>
static int clusters_at_once(Kernel kernel, AtOnce& cache, int dev, int n, int threads, size_t smem) {
  return cache.get(dev, n, [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int most = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&most, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return -1;
    }
    return most;
  });
}

// What a form costs, in microseconds: `launch` and, for every wave of clusters, its blocks of K and the sums' way
// between CTAs, some more where CTAs follow one another; never less than the weights' bytes at 7 TB/s. The constants are
// fits to calls whose weights come from memory; what they choose was within 4 % of the fastest of these forms and splits at
// 67 of 68 sizes of 16 to 8,191 tokens, 1,280 to 28,672 weight rows and K of 1,024 to 8,192. Some of them (us):
//   rows of 128 tokens: 256 x 4,096 x 8,192 on 1 / 2 / 4 CTAs 18.4 / 13.1 / 20.1; pairs on 1 / 2 / 3 29.6 / 21.4 / 19.4;
//   256 x 10,240 x 4,096: rows 22.7 / 28.1, pairs 18.1 / 32.0; 512 x 4,096 x 8,192: rows 18.8 / 26.0, pairs 29.4 / 21.9;
//   1,536 x 4,096 x 8,192: rows 55.2 / 73.3, pairs 53.7 / 62.7;
//   64 x 10,240 x 4,096 on 1 / 2 / 3 / 4 CTAs, the better of one and two per SM 11.6 / 12.2 / 11.7 / 17.2;
//   64 x 4,096 x 8,192 on 2 / 3 / 4, one per SM 11.1 / 9.8 / 9.9, two per SM on 6 / 8 11.5 / 11.3;
//   16 x 1,280 x 4,096 on 4 / 6 / 8 4.5 / 4.3 / 4.1; 64 x 28,672 x 4,096 on 1, one and two per SM 27.0 and 22.6.
struct FormCost {
  float launch, block, sums;
};
static float form_us(const FormCost& c, const LinearArgs& a, int64_t clusters, int at_once, int split, float restart) {
  const int64_t waves = (clusters + at_once - 1) / at_once;
  const int KB = (a.K + kTile - 1) / kTile;
  const float sums = split > 1 ? c.sums * static_cast<float>(split) : 0.f;
  const float us = static_cast<float>(waves) * (static_cast<float>((KB + split - 1) / split) * c.block + sums);
  const float bytes = static_cast<float>(a.N) * static_cast<float>(a.K) / 7.0e6f + sums;
  return c.launch + (us > bytes ? us : bytes) + restart * static_cast<float>(waves - 1);
}

template <int NT, bool kDeep>
struct RowsForm {
  using C = RowsCfg<NT, kDeep>;
  static constexpr size_t kSmem = C::kTotal + 1024;
  static constexpr FormCost kCost = NT == 128 ? FormCost{6.5f, 0.19f, 0.18f}
                                  : kDeep ? (NT == 16 ? FormCost{3.9f, 0.2f, 0.08f} : NT == 32 ? FormCost{4.1f, 0.215f, 0.1f} : FormCost{5.2f, 0.2f, 0.2f})
                                          : (NT == 16 ? FormCost{3.8f, 0.4f, 0.12f} : NT == 32 ? FormCost{4.6f, 0.45f, 0.2f} : FormCost{5.7f, 0.45f, 0.19f});
  // The number of CTAs that share a tile's K (0: the device has none to give), and what the call then costs.
  static void plan(const LinearArgs& a, int dev, int forced, int& split, float& us) {
    static AtOnce cache;
    const int64_t tiles = static_cast<int64_t>((a.N + kTile - 1) / kTile) * ((a.T + NT - 1) / NT);
    const int KB = (a.K + kTile - 1) / kTile;
    split = cheapest_split(
        KB < 8 ? KB : 8, forced, true,
        [&](int s) { return C::kCtas * clusters_at_once(fp8_linear_rows_kernel<NT, kDeep>, cache, dev, s, C::kThreads, kSmem); },
        [&](int s, int at_once) { return form_us(kCost, a, tiles, at_once, s, C::kCtas == 1 ? 5.f : 2.5f) - (s > 1 ? 0.9f : 0.f); }, us);
  }
  static cudaError_t launch(const LinearArgs& a, LinearParams p, int split, cudaStream_t stream, DispatchRecord* rec) {
    CUtensorMap tw, ta;
    cudaError_t err = cudaFuncSetAttribute(fp8_linear_rows_kernel<NT, kDeep>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;                  // (in front of the maps: see encode_fn)
    if ((err = rows_map(&tw, a.w, a.N, a.K, kTile)) != cudaSuccess) return err;
    if ((err = rows_map(&ta, a.a, a.T, a.K, NT)) != cudaSuccess) return err;
    const int64_t tiles = (a.N + kTile - 1) / kTile, groups = (a.T + NT - 1) / NT;
    if (groups > 65535) return cudaErrorInvalidValue;
    p.split = split;
    err = launch_pdl_cluster(fp8_linear_rows_kernel<NT, kDeep>, dim3(static_cast<unsigned>(tiles * split), static_cast<unsigned>(groups)),
                             dim3(C::kThreads), kSmem, stream, split, tw, ta, p);
    if (err != cudaSuccess) return err;
    rec->set("fp8_linear rows tokens=%d%s grid=%lldx%lld split=%d", NT, kDeep && NT <= 64 ? " deep" : "", static_cast<long long>(tiles * split),
             static_cast<long long>(groups), split);
    return cudaGetLastError();
  }
};

template <int NT>
static cudaError_t launch_rows(const LinearArgs& a, const LinearParams& p, int dev, int forced, cudaStream_t stream, DispatchRecord* rec) {
  int split[2];
  float us[2] = {0.f, 0.f};
  RowsForm<NT, false>::plan(a, dev, forced, split[0], us[0]);
  RowsForm<NT, true>::plan(a, dev, forced, split[1], us[1]);
  const bool deep = split[0] == 0 || (split[1] != 0 && us[1] < us[0]);       // (neither: the launch says what is wrong)
  return deep ? RowsForm<NT, true>::launch(a, p, split[1] ? split[1] : 1, stream, rec) : RowsForm<NT, false>::launch(a, p, split[0], stream, rec);
}

struct PairForm {
  using C = PairCfg;
  static constexpr size_t kSmem = C::kTotal + 1024;
  static int64_t tiles(const LinearArgs& a) {
    return static_cast<int64_t>((a.T + 2 * C::kTok - 1) / (2 * C::kTok)) * ((a.N + C::kOut - 1) / C::kOut);
  }
  static int at_once(int dev, int split) {
    static AtOnce cache;
    return clusters_at_once(fp8_linear_pair_kernel, cache, dev, 2 * split, C::kThreads, kSmem);
  }
  static void plan(const LinearArgs& a, int dev, int forced, int& split, float& us) {
    const int KB = (a.K + kTile - 1) / kTile;
    split = cheapest_split(
        KB < 4 ? KB : 4, forced, false, [&](int s) { return at_once(dev, s); },
        [&](int s, int room) {
          // a tile's outputs 1.1 us; the sums' way 4 us for two pairs, 6 for more
          const float t = form_us(FormCost{4.9f, 0.3875f, s == 2 ? 2.f : 6.f / static_cast<float>(s)}, a, tiles(a), room, s, s > 1 ? 2.5f : 0.f);
          return t + 1.1f * static_cast<float>((tiles(a) + room - 1) / room);
        }, us);
  }
  static cudaError_t launch(const LinearArgs& a, LinearParams p, int dev, int split, cudaStream_t stream, DispatchRecord* rec) {
    CUtensorMap tw, ta, to;
    cudaError_t err = cudaFuncSetAttribute(fp8_linear_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;                  // (in front of the maps: see encode_fn)
    if ((err = rows_map(&tw, a.w, a.N, a.K, 128)) != cudaSuccess) return err;
    if ((err = rows_map(&ta, a.a, a.T, a.K, 128)) != cudaSuccess) return err;
    const int64_t stride = a.out_stride * (a.out_f32 ? 4 : 2);
    p.whole = a.N / (a.out_f32 ? 4 : 8) * (a.out_f32 ? 4 : 8);
    p.boxed = stride % 16 == 0 && stride < (1ll << 40) && p.whole > 0;
    memset(&to, 0, sizeof(to));
    if (p.boxed && (err = out_map(&to, a.out, a.T, p.whole, stride, a.out_f32)) != cudaSuccess) return err;
    p.tiles_m = (a.T + 2 * C::kTok - 1) / (2 * C::kTok);
    p.tiles_n = (a.N + C::kOut - 1) / C::kOut;
    const int64_t rows = (32ll << 20) / (2 * C::kTok * static_cast<int64_t>(a.K));
    p.group = rows < 1 ? 1 : rows > p.tiles_m ? p.tiles_m : static_cast<int>(rows);
    if (tiles(a) > INT32_MAX / 16) return cudaErrorInvalidValue;
    p.split = split;
    const int room = at_once(dev, 1);
    const int64_t clusters = split > 1 || tiles(a) < room ? tiles(a) : room < 1 ? 1 : room;
    err = launch_pdl_cluster(fp8_linear_pair_kernel, dim3(static_cast<unsigned>(clusters * 2 * split)), dim3(C::kThreads), kSmem,
                             stream, 2 * split, tw, ta, to, p);
    if (err != cudaSuccess) return err;
    rec->set("fp8_linear pairs tiles=%dx%d grid=%lld split=%d", p.tiles_m, p.tiles_n, static_cast<long long>(clusters * 2 * split), split);
    return cudaGetLastError();
  }
};

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
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) dev = -1;
  const char* form = getenv("MSA_LINEAR_FORM");
  const bool pairs_only = form != nullptr && strcmp(form, "pairs") == 0, rows_only = form != nullptr && strcmp(form, "rows") == 0;
  const char* force = getenv("MSA_LINEAR_SPLIT");
  int forced = force != nullptr ? atoi(force) : 0;
  if (forced < 0 || forced > 8) forced = 0;
  // Up to 64 tokens weights as M: the tokens' columns are what fills up. Above, what costs less.
  if (!pairs_only) {
    if (a.T <= 16) return launch_rows<16>(a, p, dev, forced, stream, rec);
    if (a.T <= 32) return launch_rows<32>(a, p, dev, forced, stream, rec);
    if (a.T <= 64) return launch_rows<64>(a, p, dev, forced, stream, rec);
  }
  int rows_split = 0, pair_split = 0;
  float rows_us = 0.f, pair_us = 0.f;
  const bool rows_fit = (a.T + 127) / 128 <= 65535;                 // groups of tokens are a grid's y
  if (!pairs_only && rows_fit) RowsForm<128, true>::plan(a, dev, forced, rows_split, rows_us);
  if (!rows_only || !rows_fit) PairForm::plan(a, dev, forced, pair_split, pair_us);
  if (rows_split != 0 && (pair_split == 0 || rows_us <= pair_us)) return RowsForm<128, true>::launch(a, p, rows_split, stream, rec);
  if (pair_split != 0 || pairs_only || !rows_fit) return PairForm::launch(a, p, dev, pair_split ? pair_split : 1, stream, rec);
  return RowsForm<128, true>::launch(a, p, 1, stream, rec);                   // (neither: the launch says what is wrong)
}

}  // namespace msa
