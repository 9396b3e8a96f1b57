// Eviction by accumulated attention weight.  Of a unit's live rows the sinks
// (position < sinks) and the w newest positions stay, and of the others the
// `budget` rows of largest weight (ties: lowest row first; -0 = +0; NaN last).
//
// One CTA per unit.  The weights become order-preserving 32-bit keys; four
// passes of eight bits find the threshold key, and one pass in row order
// writes the keep bytes, the free rows in ascending order, the kept rows'
// weights and (optionally) the kept rows' indices.
#include <limits.h>

#include "ptx.cuh"
#include "rkv_internal.cuh"

namespace rkv {
namespace {

constexpr int kDrThreads = 512;
constexpr int kDrWarps = kDrThreads / 32;

// Order-preserving key of a weight, at least 1: -0 and +0 alike, NaN below
// every number.  0 is left for rows that are not ranked.
__device__ __forceinline__ uint32_t weight_key(float s) {
  const uint32_t b = __float_as_uint(__fadd_rn(s, 0.f));
  const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return s == s ? k : 1u;   // -inf has key 0x007fffff
}

enum : uint32_t { kDead = 0u, kRanked = 1u, kSafe = 2u };

__global__ void __launch_bounds__(kDrThreads) drop_kernel(const DropParams p) {
  __shared__ uint32_t hist[256];
  __shared__ int red[kDrWarps];
  __shared__ int wa[kDrWarps], wb[kDrWarps];
  __shared__ int sh_digit, sh_want;
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int u = blockIdx.x;
  const int64_t base = p.tok_off[u];
  const int N = static_cast<int>(p.tok_off[u + 1] - base);
  const float* acc = p.acc + base;
  const uint8_t* live = p.live ? p.live + base : nullptr;
  const int32_t* pos = p.pos ? p.pos + base : nullptr;

  auto is_live = [&](int i) { return !live || live[i] != 0; };
  auto place = [&](int i) { return pos ? pos[i] : i; };

  // the newest live position, and how many rows are ranked
  int newest = INT_MIN;
  for (int i = tid; i < N; i += kDrThreads)
    if (is_live(i)) newest = max(newest, place(i));
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) red[wp] = newest;
  __syncthreads();
  newest = red[0];
  for (int k = 1; k < kDrWarps; ++k) newest = max(newest, red[k]);
  const int64_t recent = static_cast<int64_t>(newest) - p.w;   // positions above it stay
  auto kind = [&](int i) -> uint32_t {
    if (!is_live(i)) return kDead;
    const int x = place(i);
    return x < p.sinks || x > recent ? kSafe : kRanked;
  };
  int cnt = 0;
  for (int i = tid; i < N; i += kDrThreads) cnt += kind(i) == kRanked;
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  __syncthreads();
  if (lane == 0) red[wp] = cnt;
  __syncthreads();
  int ranked = 0;
  for (int k = 0; k < kDrWarps; ++k) ranked += red[k];
  int budget = p.budget;
  if (p.budgets) budget = min(max(p.budgets[u], 0), p.budget);

  // threshold: ranked rows with key > thr stay, and the first `ties` with key = thr
  uint32_t thr = 0u;
  int ties = 0;
  if (budget == 0) {
    thr = 0xffffffffu;
  } else if (ranked > budget) {
    int want = budget;
    uint32_t prefix = 0u, mask = 0u;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      for (int k = tid; k < 256; k += kDrThreads) hist[k] = 0u;
      __syncthreads();
      for (int i = tid; i < N; i += kDrThreads) {
        if (kind(i) != kRanked) continue;
        const uint32_t k = weight_key(acc[i]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (wp == 0) {   // lane l: bins 255 - 8 l .. 248 - 8 l, from the top
        int h[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          h[k] = static_cast<int>(hist[255 - 8 * lane - k]);
          sum += h[k];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        int before = incl - sum;
        if (before < want && want <= incl) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (before < want && want <= before + h[k]) {
              sh_digit = 255 - 8 * lane - k;
              sh_want = want - before;
            }
            before += h[k];
          }
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(sh_digit) << shift;
      mask |= 255u << shift;
      want = sh_want;
    }
    thr = prefix;
    ties = want;
  }

  // rows in order, kDrThreads at a time; running counts of ties and kept rows
  int nt = 0, nk = 0;
  int32_t* idx = p.idx ? p.idx + static_cast<int64_t>(u) * p.W : nullptr;
  for (int i0 = 0; i0 < N; i0 += kDrThreads) {
    const int i = i0 + tid;
    const uint32_t kd = i < N ? kind(i) : kDead;
    const float a = i < N ? acc[i] : 0.f;
    const uint32_t key = kd == kRanked ? weight_key(a) : 0u;
    const bool tie = kd == kRanked && key == thr;
    const unsigned tb = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) wa[wp] = __popc(tb);
    __syncthreads();
    int before = nt, all = 0;
    for (int k = 0; k < kDrWarps; ++k) {
      before += k < wp ? wa[k] : 0;
      all += wa[k];
    }
    nt += all;
    const bool kept = kd == kSafe || (kd == kRanked && key > thr) ||
                      (tie && before + __popc(tb & ((1u << lane) - 1u)) < ties);
    const unsigned kb = __ballot_sync(0xffffffffu, kept);
    if (lane == 0) wb[wp] = __popc(kb);
    __syncthreads();
    int kbefore = nk, kall = 0;
    for (int k = 0; k < kDrWarps; ++k) {
      kbefore += k < wp ? wb[k] : 0;
      kall += wb[k];
    }
    nk += kall;
    kbefore += __popc(kb & ((1u << lane) - 1u));
    if (i < N) {
      p.keep[base + i] = kept ? 1 : 0;
      if (!kept) p.free_slots[base + i - kbefore] = i;
      if (p.acc_out) p.acc_out[base + i] = kept ? a : 0.f;
      if (kept && idx && kbefore < p.W) idx[kbefore] = i;
    }
    __syncthreads();   // wa, wb are written again
  }
  for (int i = N - nk + tid; i < N; i += kDrThreads) p.free_slots[base + i] = -1;
  if (idx)
    for (int i = nk + tid; i < p.W; i += kDrThreads) idx[i] = -1;
  if (tid == 0) {
    p.n_free[u] = N - nk;
    if (p.n_kept) p.n_kept[u] = min(nk, p.W);
    // more rows than a row of idx holds: positions that occur twice
    if (idx && nk > p.W) atomicOr(p.status, kStatusBadIndex);
  }
}

}  // namespace

cudaError_t drop_configure() { return cudaSuccess; }

cudaError_t launch_drop(const DropParams& p, int U, int nmax, cudaStream_t st) {
  (void)nmax;
  drop_kernel<<<U, kDrThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace rkv
