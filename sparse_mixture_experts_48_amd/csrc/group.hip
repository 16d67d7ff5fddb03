// Grouping of T*K routing choices by expert, for up to 512 experts and
// without copied rows: counts, offsets, the token of every grouped row and the
// grouped row of every choice. Stable: inside an expert's group tokens keep
// their order. Ids outside [0, E) get no row.
//
// The rank of a choice in its expert's group = choices of that expert in
// earlier blocks + in earlier waves of the block + in the wave's earlier
// steps + in lower lanes of the step. A block owns a contiguous chunk of
// slots and each of its waves a contiguous part of it. The lanes of a step
// that hold the same id are found with one ballot per id bit.
// One launch when a single block covers the slots, else two (the blocks'
// histograms, then the ranks). Latency-bound: 12 bytes per choice.
#include "common.h"
#include "fp8.h"

namespace moe {

namespace {

constexpr int kGT = 1024;           // threads per block
constexpr int kGW = kGT / 64;       // waves per block
constexpr int kChunkMin = 4096;     // slots per block at least
constexpr int kMaxBlocks = 256;     // every block sums the histograms of all blocks

int group_chunk(int64_t S) {
  const int64_t per = (S + kMaxBlocks - 1) / kMaxBlocks;
  return static_cast<int>((per < kChunkMin ? kChunkMin : per) + kGT - 1) / kGT * kGT;
}

__global__ __launch_bounds__(kGT) void group_hist_kernel(const int32_t* __restrict__ ids, int S, int E, int chunk,
                                                         int32_t* __restrict__ blk_hist) {
  __shared__ int cnt[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += kGT) cnt[e] = 0;
  __syncthreads();
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int n = static_cast<int>(min(static_cast<int64_t>(chunk), S - s0));
  for (int i = threadIdx.x; i < n; i += kGT) {
    const int id = ids[s0 + i];
    if (id >= 0 && id < E) atomicAdd(&cnt[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kGT) blk_hist[static_cast<size_t>(blockIdx.x) * E + e] = cnt[e];
}

__global__ __launch_bounds__(kGT) void group_rank_kernel(const int32_t* __restrict__ ids, int S, int E, int K,
                                                         int chunk, const int32_t* __restrict__ blk_hist,
                                                         int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                         int32_t* __restrict__ slot_token,
                                                         int32_t* __restrict__ token_slot) {
  __shared__ int wcnt[kGW][kMaxExperts];  // per wave: its choices of each expert, then its next row of each
  __shared__ int base[kMaxExperts];       // the block's first row of each expert, less the expert's offset
  __shared__ int tot[kMaxExperts];        // choices of each expert in the whole batch
  __shared__ int wsum[kGW];
  const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
  const int NB = static_cast<int>(gridDim.x);
  for (int i = threadIdx.x; i < kGW * kMaxExperts; i += kGT) (&wcnt[0][0])[i] = 0;
  __syncthreads();
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int n = static_cast<int>(min(static_cast<int64_t>(chunk), S - s0));
  const int part = chunk / kGW;  // a multiple of 64
  const int w0 = min(n, w * part), w1 = min(n, w0 + part);
  for (int i = w0 + lane; i < w1; i += 64) {
    const int id = ids[s0 + i];
    if (id >= 0 && id < E) atomicAdd(&wcnt[w][id], 1);
  }
  __syncthreads();
  // exclusive sums over the block's waves, and the batch's totals
  for (int e = threadIdx.x; e < E; e += kGT) {
    int run = 0;
    for (int v = 0; v < kGW; ++v) {
      const int c = wcnt[v][e];
      wcnt[v][e] = run;
      run += c;
    }
    int before = 0, all = run;
    if (NB > 1) {
      all = 0;
      for (int b = 0; b < NB; ++b) {
        const int c = blk_hist[static_cast<size_t>(b) * E + e];
        before += b < static_cast<int>(blockIdx.x) ? c : 0;
        all += c;
      }
    }
    base[e] = before;
    tot[e] = all;
  }
  __syncthreads();
  // offsets: prefix sum over the experts (threads 0 .. 511 hold one each)
  {
    const int e = threadIdx.x;
    const int c = e < E ? tot[e] : 0;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 63) wsum[w] = incl;
    __syncthreads();
    int off = incl - c;
    for (int v = 0; v < w; ++v) off += wsum[v];
    if (e < E) {
      base[e] += off;
      if (blockIdx.x == 0) {
        counts[e] = c;
        offsets[e] = off;
        if (e == E - 1) offsets[E] = off + c;
      }
      if (e == E - 1) tot[0] = off + c;  // every expert's own total has been read above
    }
  }
  __syncthreads();
  const int total = tot[0];
  for (int e = threadIdx.x; e < E; e += kGT)
    for (int v = 0; v < kGW; ++v) wcnt[v][e] += base[e];
  __syncthreads();
  int bits = 1;
  while ((1 << bits) < E) ++bits;
  for (int i0 = w0; i0 < w1; i0 += 64) {
    const int i = i0 + lane;
    const int id = i < w1 ? ids[s0 + i] : -1;
    const bool live = i < w1 && id >= 0 && id < E;
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot(live && ((id >> b) & 1));
      same &= (id >> b) & 1 ? m : ~m;
    }
    if (live) {
      const int first = wcnt[w][id];
      const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
      const int64_t s = s0 + i;
      slot_token[first + rank] = static_cast<int32_t>(s / K);
      token_slot[s] = first + rank;
      __builtin_amdgcn_wave_barrier();
      if (rank == 0) wcnt[w][id] = first + __popcll(same);
    } else if (i < w1) {
      token_slot[s0 + i] = -1;
    }
    __builtin_amdgcn_wave_barrier();
  }
  for (int64_t s = total + static_cast<int64_t>(blockIdx.x) * kGT + threadIdx.x; s < S;
       s += static_cast<int64_t>(NB) * kGT)
    slot_token[s] = -1;
}

}  // namespace

int group_blocks(int64_t S) {
  const int c = group_chunk(S);
  return static_cast<int>((S + c - 1) / c);
}

hipError_t launch_group(const int32_t* topk_idx, int S, int E, int K, int32_t* counts, int32_t* offsets,
                        int32_t* slot_token, int32_t* token_slot, int32_t* blk_hist, hipStream_t st) {
  const int chunk = group_chunk(S);
  const int NB = S > 0 ? group_blocks(S) : 1;  // S = 0: one block writes zero counts and offsets
  if (NB > 1) {
    hipLaunchKernelGGL(group_hist_kernel, dim3(NB), dim3(kGT), 0, st, topk_idx, S, E, chunk, blk_hist);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(group_rank_kernel, dim3(NB), dim3(kGT), 0, st, topk_idx, S, E, K, chunk, blk_hist, counts,
                     offsets, slot_token, token_slot);
  return hipGetLastError();
}

}  // namespace moe
