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
// One launch when a single block covers the slots (as many waves as it takes),
// else two (the blocks' histograms, then the ranks).
// Bound: the latency of a few dependent passes (12 bytes per choice). Measured:
// 32 choices over 8 experts 3.0 us, 131072 over 256 experts 10.4 us.
#include <type_traits>

#include "common.h"
#include "fp8.h"
#include "quant_fp8.h"

namespace moe {

namespace {

constexpr int kGT = 1024;        // threads per block at most
constexpr int kGW = kGT / 64;
constexpr int kOneBlock = 2048;  // slots that a single block takes
constexpr int kMaxBlocks = 256;  // every block adds up the histograms of all blocks

// Slots per block. Measured at 4096 slots one block 7.2 us, two launches 6.9; blocks of 1024 against 2048 slots:
// 32768 slots 8.6 against 9.2 us, 131072 slots 10.9 against 10.5.
int group_chunk(int64_t S) {
  if (S <= kOneBlock) return kOneBlock;
  const int64_t least = S <= 65536 ? 1024 : 2048, per = (S + kMaxBlocks - 1) / kMaxBlocks;
  return static_cast<int>((per < least ? least : per) + kGT - 1) / kGT * kGT;
}

// Both kernels take NB blocks; the blocks after them quantise rows of H (void: there are none), which saves the layer a
// launch (decode layer 221 -> 219 us, 64 tokens 277 -> 274).
template <typename H>
__global__ __launch_bounds__(kGT) void group_hist_kernel(const int32_t* __restrict__ ids, int S, int E, int chunk, int NB,
                                                         int32_t* __restrict__ blk_hist, QuantRows quant) {
  if constexpr (!std::is_void_v<H>) {
    if (static_cast<int>(blockIdx.x) >= NB) {
      quant_rows<H>(quant, static_cast<int64_t>(blockIdx.x - NB) * blockDim.x + threadIdx.x);
      return;
    }
  }
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

template <typename H>
__global__ __launch_bounds__(kGT) void group_rank_kernel(const int32_t* __restrict__ ids, int S, int E, int K,
                                                         int chunk, int NB, const int32_t* __restrict__ blk_hist,
                                                         int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                         int32_t* __restrict__ slot_token,
                                                         int32_t* __restrict__ token_slot, QuantRows quant) {
  if constexpr (!std::is_void_v<H>) {
    if (static_cast<int>(blockIdx.x) >= NB) {
      quant_rows<H>(quant, static_cast<int64_t>(blockIdx.x - NB) * blockDim.x + threadIdx.x);
      return;
    }
  }
  __shared__ int wcnt[kGW * kMaxExperts];  // [wave][expert]: its choices, then its next row after base
  __shared__ int base[kMaxExperts];        // the block's first row of each expert
  __shared__ int tot[kMaxExperts + 1];     // choices of each expert in the whole batch; [E]: of all
  const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
  const int NT = static_cast<int>(blockDim.x), NW = NT / 64;
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int n = static_cast<int>(min(static_cast<int64_t>(chunk), S - s0));
  const int part = ((n + NW - 1) / NW + 63) / 64 * 64;
  const int w0 = min(n, w * part), w1 = min(n, w0 + part);
  for (int i = threadIdx.x; i < NW * E; i += NT) wcnt[i] = 0;
  for (int e = threadIdx.x; e < E; e += NT) base[e] = tot[e] = 0;
  __syncthreads();
  int* const mine = wcnt + w * E;
  for (int i = w0 + lane; i < w1; i += 64) {
    const int id = ids[s0 + i];
    if (id >= 0 && id < E) atomicAdd(&mine[id], 1);
  }
  if (NB > 1) {
    // the other blocks' choices of each expert: E threads per part of the blocks, eight loads in flight each
    const int P = NT / E;  // (NT = 1024 >= 2 E here)
    const int e = threadIdx.x % E, q = threadIdx.x / E;
    if (q < P) {
      int before = 0, all = 0;
      for (int b0 = q * 8; b0 < NB; b0 += P * 8) {
        int v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = blk_hist[static_cast<size_t>(min(b0 + u, NB - 1)) * E + e];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          all += b0 + u < NB ? v[u] : 0;
          before += b0 + u < static_cast<int>(blockIdx.x) ? v[u] : 0;
        }
      }
      atomicAdd(&base[e], before);  // (whole numbers: any order gives the same sum)
      atomicAdd(&tot[e], all);
    }
  }
  __syncthreads();
  // exclusive sums over the block's waves
  for (int e = threadIdx.x; e < E; e += NT) {
    int run = 0;
    for (int v = 0; v < NW; ++v) {
      const int c = wcnt[v * E + e];
      wcnt[v * E + e] = run;
      run += c;
    }
    if (NB == 1) tot[e] = run;
  }
  __syncthreads();
  if (w == 0) {  // offsets: lane l adds up experts l P .. l P + P - 1
    const int P = (E + 63) / 64;
    int sum = 0;
    for (int i = 0; i < P; ++i) sum += lane * P + i < E ? tot[lane * P + i] : 0;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o);
      if (lane >= o) incl += v;
    }
    int off = incl - sum;
    for (int i = 0; i < P; ++i) {
      const int e = lane * P + i;
      if (e >= E) break;
      base[e] += off;
      if (blockIdx.x == 0) {
        counts[e] = tot[e];
        offsets[e] = off;
      }
      off += tot[e];
    }
    if (lane == 63) {
      tot[E] = incl;
      if (blockIdx.x == 0) offsets[E] = incl;
    }
  }
  __syncthreads();
  const int total = tot[E];
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
    const int before = live ? mine[id] : 0;
    const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();  // every lane has read its count before one of them moves it on
    if (live && rank == 0) mine[id] = before + __popcll(same);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    const int64_t s = s0 + i;
    if (live) {
      const int row = base[id] + before + rank;
      slot_token[row] = static_cast<int32_t>(static_cast<uint32_t>(s) / static_cast<uint32_t>(K));
      token_slot[s] = row;
    } else if (i < w1) {
      token_slot[s] = -1;
    }
  }
  for (int64_t s = total + static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x; s < S; s += static_cast<int64_t>(NB) * NT)
    slot_token[s] = -1;
}

template <typename H>
hipError_t launch(const int32_t* topk_idx, int S, int E, int K, int32_t* counts, int32_t* offsets, int32_t* slot_token,
                  int32_t* token_slot, int32_t* blk_hist, const QuantRows& quant, hipStream_t st) {
  const int chunk = group_chunk(S);
  const int NB = S > 0 ? group_blocks(S) : 1;  // S = 0: one block writes zero counts and offsets
  const int threads = NB > 1 || S >= kGT ? kGT : S <= 64 ? 64 : (S + 63) / 64 * 64;
  // the rows to quantise run beside the first launch
  const int64_t blocks = quant.rows * ((quant.cols + kFp8Block - 1) / kFp8Block);
  const unsigned more = std::is_void_v<H> ? 0 : static_cast<unsigned>((blocks * 16 + threads - 1) / threads);
  if (NB > 1) {
    hipLaunchKernelGGL(group_hist_kernel<H>, dim3(NB + more), dim3(kGT), 0, st, topk_idx, S, E, chunk, NB, blk_hist, quant);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(group_rank_kernel<void>, dim3(NB), dim3(kGT), 0, st, topk_idx, S, E, K, chunk, NB, blk_hist, counts,
                       offsets, slot_token, token_slot, quant);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(group_rank_kernel<H>, dim3(1 + more), dim3(threads), 0, st, topk_idx, S, E, K, chunk, 1, blk_hist,
                     counts, offsets, slot_token, token_slot, quant);
  return hipGetLastError();
}

}  // namespace

int group_blocks(int64_t S) {
  const int c = group_chunk(S);
  return static_cast<int>((S + c - 1) / c);
}

hipError_t launch_group(const int32_t* topk_idx, int S, int E, int K, int32_t* counts, int32_t* offsets,
                        int32_t* slot_token, int32_t* token_slot, int32_t* blk_hist, const QuantRows* quant,
                        bool quant_bf16, hipStream_t st) {
  auto run = [&](auto* type, const QuantRows& q) {
    return launch<std::remove_pointer_t<decltype(type)>>(topk_idx, S, E, K, counts, offsets, slot_token, token_slot,
                                                         blk_hist, q, st);
  };
  if (quant == nullptr) return run(static_cast<void*>(nullptr), QuantRows{});
  return quant_bf16 ? run(static_cast<bf16_t*>(nullptr), *quant) : run(static_cast<float*>(nullptr), *quant);
}

}  // namespace moe
