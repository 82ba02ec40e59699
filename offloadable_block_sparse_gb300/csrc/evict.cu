// Eviction from a block store by accumulated attention weight (nosa_evict).
//
// One CTA per unit: it accumulates the rows' weights, finds the n-th smallest of those that may go, if n rows have to,
// and writes the unit's table.  Rows are ordered by one 64-bit key (weight, then the block's number downwards), which a
// radix selection takes eight bits at a time through a histogram in shared memory; for n = 1, the step of a full store,
// a minimum does.  Counts are the only atomics, so the outcome does not depend on their order.  20 bytes a row: a call
// is bound by its latency, 2.3 us for 256 units of 128 rows of which one goes, 6.4 for 256 units of 1,025 of which three
// quarters go (four rounds of the selection; counting a warp's equal digits before the histogram took 7.3), 34 for 256 of
// 16,384.
#include <algorithm>
#include <mutex>

#include "host.h"
#include "ptx.cuh"

namespace nosa {

constexpr int kEvictSlots = 16384;

struct EvictArgs {
  const float* acc;
  const int32_t* slot_blk;
  const float* mass;
  const int32_t* lens;
  const int32_t* next_block;
  float* acc_out;
  int32_t* slot_blk_out;
  int32_t* next_slot;
  int32_t* err;
  int slots, budget, sink, window;
  float decay;
};

// Sum (or minimum) of one int per thread over the CTA; `tmp` holds 32 ints, and is free again on return.
template <bool kMin>
__device__ __forceinline__ int cta_reduce(int v, int* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = kMin ? __reduce_min_sync(0xffffffffu, v) : __reduce_add_sync(0xffffffffu, v);
  if (lane == 0) tmp[warp] = v;
  __syncthreads();
  v = lane < nw ? tmp[lane] : (kMin ? 0x7fffffff : 0);
  v = kMin ? __reduce_min_sync(0xffffffffu, v) : __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(1024) evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ float2 rows[];  // [slots]: accumulated weight, block (as bits)
  __shared__ int tmp[32], hist[256];
  __shared__ unsigned long long least;
  __shared__ int digit, below;
  const int u = blockIdx.x, n = a.slots, lane = threadIdx.x & 31;
  const size_t base = (size_t)u * n;
  pdl_wait();
  pdl_launch_dependents();
  const int next = a.next_block ? a.next_block[u] : -1;
  const int len = a.lens ? max(a.lens[u], 0) : 0;
  // blocks from here on are the window's (without lengths there is none)
  const long long last = a.lens ? (((long long)len + kBlock - 1) / kBlock) - a.window : 0x7fffffffll + 1;

  auto may_go = [&](int block) { return block >= a.sink && block < last && block != next; };
  // smaller keys go first: smaller weights, of equal ones higher blocks
  auto key = [&](float w, int block) {
    return (unsigned long long)orderable(w) << 32 | (uint32_t)(0x7fffffff - block);
  };

  int held = 0, free = 0, has = n;  // rows with a block, rows that may go, the row that holds the next block
  unsigned long long mine = ~0ull;  // the thread's smallest key
  for (int s = threadIdx.x; s < n; s += blockDim.x) {
    const int block = a.slot_blk[base + s];
    float w = 0.f;
    if (block >= 0) {
      w = __fmul_rn(a.decay, a.acc[base + s]);
      if (a.mass) w = __fadd_rn(w, a.mass[base + s]);
      if (!(w == w)) w = 0.f;
      w += 0.f;  // (-0 as 0: they are equal)
      ++held;
      if (block == next) has = min(has, s);
      if (may_go(block)) {
        ++free;
        mine = min(mine, key(w, block));
      }
    }
    rows[s] = make_float2(w, __int_as_float(block));
  }
  held = cta_reduce<false>(held, tmp);
  free = cta_reduce<false>(free, tmp);
  has = cta_reduce<true>(has, tmp);
  const bool wants = next >= 0 && has == n;
  int go = min(max(held + wants - a.budget, 0), free);  // rows to empty

  unsigned long long most = 0;  // the largest key that goes
  bool some = go > 0;
  if (go == 1) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine = min(mine, __shfl_xor_sync(0xffffffffu, mine, o));
    if (threadIdx.x == 0) least = ~0ull;
    __syncthreads();
    if (lane == 0) atomicMin(&least, mine);
    __syncthreads();
    most = least;
  } else if (go > 1) {
    // `most` has the digits found so far above `shift`; `go` counts the rows still to find among those that share them
    for (int shift = 56; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += blockDim.x) hist[i] = 0;
      __syncthreads();
      const unsigned long long above = shift == 56 ? 0ull : ~0ull << (shift + 8);
      for (int s = threadIdx.x; s < n; s += blockDim.x) {
        const float2 r = rows[s];
        const int block = __float_as_int(r.y);
        if (block < 0 || !may_go(block)) continue;
        const unsigned long long k = key(r.x, block);
        if ((k & above) == most) atomicAdd(&hist[(int)(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (threadIdx.x < 32) {  // lane i has digits 8 i .. + 7
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i] = hist[8 * lane + i];
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        int before = upto - sum;
        if (before < go && go <= upto) {  // one lane
          int d = 0;
          while (before + c[d] < go) before += c[d++];
          digit = 8 * lane + d;
          below = before;
        }
      }
      __syncthreads();
      most |= (unsigned long long)digit << shift;
      go -= below;
      if (go == hist[digit]) {  // all that share these digits go
        most |= shift ? (1ull << shift) - 1 : 0ull;
        break;
      }
      __syncthreads();
    }
  }

  int empty = n;
  for (int s = threadIdx.x; s < n; s += blockDim.x) {
    const float2 r = rows[s];
    int block = __float_as_int(r.y);
    float w = r.x;
    if (some && block >= 0 && may_go(block) && key(w, block) <= most) {
      block = -1;
      w = 0.f;
    }
    if (block < 0) {
      block = -1;
      empty = min(empty, s);
    }
    a.acc_out[base + s] = w;
    a.slot_blk_out[base + s] = block;
  }
  empty = cta_reduce<true>(empty, tmp);  // also: the writes above come before the one below
  if (threadIdx.x == 0) {
    const int row = wants ? empty : has;
    if (wants && row < n) a.slot_blk_out[base + row] = next;
    if (wants && row == n && a.err) atomicOr(a.err, kErrCapacity);
    if (a.next_slot) a.next_slot[u] = next >= 0 && row < n ? row : -1;
  }
}

// The shared memory a call may take is raised once per device.
static std::mutex g_evict_mutex;
static bool g_evict_ready[64] = {};

static bool evict_ready() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    (void)cudaGetLastError();
    return false;
  }
  std::lock_guard<std::mutex> lock(g_evict_mutex);
  if (!g_evict_ready[dev]) {
    if (cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictSlots * (int)sizeof(float2)) !=
        cudaSuccess) {
      (void)cudaGetLastError();
      return false;
    }
    g_evict_ready[dev] = true;
  }
  return true;
}

}  // namespace nosa

using namespace nosa;

extern "C" nosa_status nosa_evict(const float* acc, const int32_t* slot_blk, const float* mass, int units, int slots,
                                  const int32_t* lens, int budget, int sink_blocks, int window_blocks, float decay,
                                  float* acc_out, int32_t* slot_blk_out, const int32_t* next_block, int32_t* next_slot,
                                  int32_t* err_out, void* stream) {
  if (!acc || !slot_blk || !acc_out || !slot_blk_out || units < 1 || slots < 1 || slots > kEvictSlots || budget < 0 ||
      budget > slots || sink_blocks < 0 || window_blocks < 0 || !(decay >= 0.f) || isinf(decay) || (!lens && window_blocks > 0))
    return NOSA_ERR_INVALID_ARG;
  auto off = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; };
  if (off(acc) || off(slot_blk) || off(mass) || off(lens) || off(acc_out) || off(slot_blk_out) || off(next_block) ||
      off(next_slot) || off(err_out))
    return NOSA_ERR_INVALID_ARG;
  if (!evict_ready()) return NOSA_ERR_CUDA;
  EvictArgs a{acc, slot_blk, mass, lens, next_block, acc_out, slot_blk_out, next_slot, err_out, slots, budget, sink_blocks,
              window_blocks, decay};
  const int threads = slots <= 256 ? 128 : slots <= 2048 ? 512 : 1024;
  const cudaError_t e = launch_ex(evict_kernel, dim3((unsigned)units), dim3(threads), slots * sizeof(float2),
                                  static_cast<cudaStream_t>(stream), true, 0, a);
  if (e == cudaSuccess) return NOSA_OK;
  (void)cudaGetLastError();
  return NOSA_ERR_CUDA;
}
