// Step metadata from request lengths: block tables, slot map, positions.
//
// "MiniMax M3 vLLM サポート：…" (agentlenshq.com), section "KV キャッシュ統合": the
// K/V data stays an ordinary paged cache, so a step needs its requests' block
// tables and the cache slot of every new token. With seq = ctx + new and
// blocks(n) = ceil(n / 128), request b takes blocks(seq) - blocks(ctx) pages
// from the free list, at the exclusive prefix sum of these needs, and its
// tokens sit at the exclusive prefix sum of `new`. Both sums run over at most
// 4,096 requests, which every CTA does for itself in shared memory (one pass, no
// second launch and no flags between CTAs); the CTAs then share the tokens.
#include "msa_internal.h"

namespace msa {

constexpr int kStepThreads = 128;
constexpr int kStepWarps = kStepThreads / 32;
constexpr int kTokPerThread = 4;
constexpr int kStepMaxBatch = 4096;               // the entry point refuses larger ones
constexpr int kTokPerPass = kStepThreads * kTokPerThread;

struct StepScan {
  int64_t tokens, pages;
};

// Exclusive sum over the CTA's threads of (tokens, pages), and the totals.
__device__ __forceinline__ StepScan block_exclusive(StepScan v, StepScan* warp_sums, StepScan& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  StepScan in = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, in.tokens, o), p = __shfl_up_sync(0xffffffffu, in.pages, o);
    if (lane >= o) { in.tokens += t; in.pages += p; }
  }
  if (lane == 31) warp_sums[warp] = in;
  __syncthreads();
  StepScan before{0, 0};
  total = StepScan{0, 0};
#pragma unroll
  for (int w = 0; w < kStepWarps; ++w) {
    const StepScan s = warp_sums[w];
    if (w < warp) { before.tokens += s.tokens; before.pages += s.pages; }
    total.tokens += s.tokens;
    total.pages += s.pages;
  }
  return StepScan{before.tokens + in.tokens - v.tokens, before.pages + in.pages - v.pages};
}

__device__ __forceinline__ int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

struct StepReq {
  int ctx, add, need;   // tokens cached, tokens that take a place in the step, pages needed
  bool len_ok;
};

__device__ __forceinline__ StepReq step_req(const StepArgs& p, int b) {
  StepReq r;
  r.ctx = p.ctx_lens[b];
  const int n = p.new_lens[b];
  const int64_t cap = static_cast<int64_t>(p.NB) * kBlock;
  r.add = n < 0 ? 0 : n;
  r.len_ok = r.ctx >= 0 && n >= 0 && static_cast<int64_t>(r.ctx) + n <= cap;
  r.need = r.len_ok ? static_cast<int>(blocks_of(static_cast<int64_t>(r.ctx) + n) - blocks_of(r.ctx)) : 0;
  return r;
}

// What the CTAs keep of a request, in shared memory.
struct StepSlot {
  int ctx, off;                 // tokens cached; rotary offset
  int last;                     // page of the last cached block, which new tokens may fill
  int pages;                    // new pages before this request; negative (~pages): refused
};

// Latency bound: everything a request needs is loaded at once, before the scan;
// after it come only stores. Shared memory: start[B + 1], the places of the
// tokens (held to T), and a StepSlot per request.
__global__ void __launch_bounds__(kStepThreads) build_step_kernel(const __grid_constant__ StepArgs p) {
  extern __shared__ int32_t sm[];
  __shared__ StepScan warp_sums[kStepWarps];
  __shared__ int taken;
  griddep_launch_dependents();
  griddep_wait();
  StepSlot* slots = reinterpret_cast<StepSlot*>(sm);
  int32_t* start = sm + 4 * p.B;
  const int tid = threadIdx.x;
  const bool lead = blockIdx.x == 0;
  if (tid == 0) taken = 0;
  const int head = *p.free_head;

  // each thread sums a run of consecutive requests
  const int per = (p.B + kStepThreads - 1) / kStepThreads;
  const int b0 = tid * per, b1 = b0 + per < p.B ? b0 + per : p.B;
  StepScan mine{0, 0};
  for (int b = b0; b < b1; ++b) {
    const StepReq r = step_req(p, b);
    mine.tokens += r.add;
    mine.pages += r.need;
    StepSlot s;
    s.ctx = r.ctx;
    s.off = p.pos_offset ? p.pos_offset[b] : 0;
    s.last = r.len_ok && r.ctx % kBlock != 0 ? p.block_table[static_cast<int64_t>(b) * p.NB + r.ctx / kBlock] : -1;
    s.pages = 0;
    slots[b] = s;
  }
  StepScan total;
  StepScan at = block_exclusive(mine, warp_sums, total);
  int got = 0;
  for (int b = b0; b < b1; ++b) {
    const StepReq r = step_req(p, b);
    const int64_t end_tok = at.tokens + r.add, end_page = head + at.pages + r.need;
    const bool placed = r.len_ok && end_tok <= p.T;
    const bool fits = r.need == 0 || (head >= 0 && end_page <= p.F);
    start[b] = static_cast<int32_t>(at.tokens < p.T ? at.tokens : p.T);
    // (a count past the free list belongs to refused requests alone, but for those that need no page)
    const int before = static_cast<int>(at.pages < INT32_MAX ? at.pages : INT32_MAX);
    slots[b].pages = placed && fits ? before : ~before;
    if (placed && fits) got += r.need;
    if (lead) {
      if (!placed) set_flag(p.flags, MSA_FLAG_BAD_SEQLEN);
      else if (!fits) set_flag(p.flags, MSA_FLAG_NO_PAGES);
      const int64_t cap = static_cast<int64_t>(p.NB) * kBlock;
      const int64_t keep = r.ctx < 0 ? 0 : (r.ctx > cap ? cap : r.ctx);
      p.seq_lens[b] = static_cast<int32_t>(placed && fits ? r.ctx + r.add : keep);
      p.token_starts[b] = start[b];
    }
    at.tokens = end_tok;
    at.pages += r.need;
  }
  const int placed_tokens = static_cast<int>(total.tokens < p.T ? total.tokens : p.T);
  if (tid == 0) start[p.B] = placed_tokens;
  if (lead && got) atomicAdd(&taken, got);
  __syncthreads();
  if (lead && tid == 0) {
    p.token_starts[p.B] = placed_tokens;
    *p.free_head_out = head + taken;
  }

  // new table entries, a thread per page: the pages before `limit` may be taken
  const int64_t left = head < 0 ? 0 : p.F - static_cast<int64_t>(head);
  const int limit = static_cast<int>(total.pages < left ? total.pages : left);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kStepThreads + tid; i < limit;
       i += static_cast<int64_t>(gridDim.x) * kStepThreads) {
    // the last request whose first page is at or before i
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1, s = slots[mid].pages;
      if ((s < 0 ? ~s : s) <= i) lo = mid; else hi = mid - 1;
    }
    if (slots[lo].pages < 0) continue;
    const int page = p.free_pages[head + i];
    const bool ok = page >= 0 && page < p.P;
    if (!ok) set_flag(p.flags, MSA_FLAG_BAD_PAGE);
    p.block_table[static_cast<int64_t>(lo) * p.NB + blocks_of(slots[lo].ctx) + (i - slots[lo].pages)] = ok ? page : -1;
  }

  // tokens, four consecutive ones per thread
  const bool wide_pos = (p.pos_stride & 3) == 0 && (reinterpret_cast<uintptr_t>(p.positions) & 15u) == 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kTokPerPass; base < p.T;
       base += static_cast<int64_t>(gridDim.x) * kTokPerPass) {
    const int64_t i0 = base + tid * kTokPerThread;
    if (i0 >= p.T) continue;
    // the last request that starts at or before i0 and has tokens there
    int lo = 0, hi = p.B;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (start[mid + 1] <= i0) lo = mid + 1; else hi = mid;
    }
    int b = lo;
    int64_t slot[kTokPerThread];
    int32_t pos[kTokPerThread];
#pragma unroll
    for (int k = 0; k < kTokPerThread; ++k) {
      const int64_t i = i0 + k;
      slot[k] = -1;
      pos[k] = 0;
      if (i >= placed_tokens) continue;
      while (start[b + 1] <= i) ++b;
      const StepSlot s = slots[b];
      const int64_t tok = static_cast<int64_t>(s.ctx) + (i - start[b]);
      pos[k] = static_cast<int32_t>(static_cast<uint32_t>(tok) + static_cast<uint32_t>(s.off));
      if (s.pages < 0) continue;
      const int64_t blk = tok / kBlock, old = blocks_of(s.ctx);
      const int page = blk < old ? s.last : p.free_pages[head + s.pages + (blk - old)];
      if (page < 0 || page >= p.P) {
        set_flag(p.flags, MSA_FLAG_BAD_PAGE);
        continue;
      }
      slot[k] = static_cast<int64_t>(page) * kBlock + tok % kBlock;
    }
    const bool whole = i0 + kTokPerThread <= p.T;
    if (whole) {
      longlong2* d = reinterpret_cast<longlong2*>(p.slots + i0);
      d[0] = make_longlong2(slot[0], slot[1]);
      d[1] = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kTokPerThread; ++k)
        if (i0 + k < p.T) p.slots[i0 + k] = slot[k];
    }
    for (int a = 0; a < p.A; ++a) {
      int32_t* d = p.positions + a * p.pos_stride + i0;
      if (whole && wide_pos) {
        *reinterpret_cast<int4*>(d) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int k = 0; k < kTokPerThread; ++k)
          if (i0 + k < p.T) d[k] = pos[k];
      }
    }
  }
}

cudaError_t launch_build_step(const StepArgs& a, cudaStream_t stream, DispatchRecord* rec) {
  int64_t grid = (static_cast<int64_t>(a.T) + kTokPerPass - 1) / kTokPerPass;
  // Short CTAs and many of them while the scan is short (prefill chunk of 524K tokens: 6.7 us; 256 threads 7.4,
  // 4 CTAs per SM 10.0); with many requests every CTA scans them all, so fewer.
  const int64_t cap = (a.B <= 512 ? 16ll : 4ll) * device_sm_count();
  if (grid > cap) grid = cap;
  const size_t smem = (5ull * a.B + 1) * sizeof(int32_t);
  if (smem > 40 * 1024) {
    // the limit is one for all host threads, so every call sets it to the largest batch's
    const cudaError_t set = cudaFuncSetAttribute(build_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (5 * kStepMaxBatch + 1) * static_cast<int>(sizeof(int32_t)));
    if (set != cudaSuccess) return set;
  }
  const cudaError_t err = launch_pdl(build_step_kernel, dim3(static_cast<unsigned>(grid)), dim3(kStepThreads), smem,
                                     stream, a);
  if (err != cudaSuccess) return err;
  rec->set("build_step grid=%lld block=%d smem=%zu requests=%d tokens=%d axes=%d", static_cast<long long>(grid),
           kStepThreads, smem, a.B, a.T, a.A);
  return cudaGetLastError();
}

}  // namespace msa
