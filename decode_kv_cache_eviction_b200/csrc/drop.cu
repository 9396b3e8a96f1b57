// Eviction by accumulated attention weight.  Of a unit's live rows the sinks
// (position < sinks) and the w newest positions stay, and of the others the
// `budget` rows of largest weight (ties: lowest row first; -0 = +0; NaN last).
//
// One cluster of 1 to 8 CTAs per unit, each with the keys of a run of the unit's rows
// in shared memory (order-preserving 32-bit keys of the weights; 0 for dead rows, the
// largest for rows that stay unranked).  Histograms of 512 bins over the range of the
// keys that are left (added over distributed shared memory in a cluster) narrow it down
// to the threshold key, and stop as soon as a bin is taken whole; a unit in one CTA ends
// with the few rows of one bin compared with each other, and a bin of equal weights is
// seen by its range.  Starting from the keys' own range spreads them over the bins, so
// few of the shared-memory additions meet.  Ballots then give every row its place among
// the kept and the free rows of the unit.
//
// Bound: instruction issue and the latency of a few dependent block reductions at small
// units, HBM beyond; hence vectors of four rows, loops that stay rolled and few registers
// (keys in registers and unrolled loops at half the resident warps took a fifth longer).
// 2048 units of 2176 rows, a fifth of the weights rounded to eighths, many of them 0: 24.6 us
// (58 MB; 9 at HBM's rate; issue slots 60% used, 1.7 waves of CTAs); 64 units of 31K rows with
// live mask and positions: 26.7 us (36 MB).
#include <limits.h>

#include "ptx.cuh"
#include "rkv_internal.cuh"

namespace rkv {
namespace {

// Order-preserving key of a weight, at least 1: -0 and +0 alike, NaN below
// every number.  0 marks a row that is not ranked.
__device__ __forceinline__ uint32_t number_key(float s) {
  const uint32_t b = __float_as_uint(__fadd_rn(s, 0.f));
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t weight_key(float s) {
  return s == s ? number_key(s) : 1u;   // -inf has key 0x007fffff
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

constexpr int kBinBits = 9;
constexpr int kBins = 1 << kBinBits;   // four per thread of the first 128

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

constexpr int kList = 128;

template <int T>
struct DropShared {
  uint4 hist[2][kBins / 4];      // two in turn
  uint32_t part[2][T / 32][8];   // the warps' values of an exchange (two in turn)
  uint32_t total[2][8];          // this CTA's
  uint32_t wsum[T / 32];
  uint32_t found[3];             // bin, its rows, rows wanted of it
  uint32_t list[kList];          // keys of a small bin
  uint32_t listed;
};

// Exchanges of up to 8 values over the CTA and the cluster.
template <int T>
struct Exchange {
  DropShared<T>& s;
  int cs, rank, turn;
  // v: the warp's values (the same in all lanes).  Combines value k with op(k, ., .)
  // from 0 over the CTA, then over the cluster; before[k]: over CTAs of lower rank.
  template <int n, class Op>
  __device__ void all(uint32_t (&v)[n], uint32_t (&before)[n], Op op) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    if (lane < n) {
      uint32_t x = v[0];
#pragma unroll
      for (int k = 1; k < n; ++k) x = lane == k ? v[k] : x;
      s.part[turn][wp][lane] = x;
    }
    __syncthreads();
    uint32_t x = 0;   // lane k < n: the CTA's value k
    if (lane < n)
      for (int w = 0; w < T / 32; ++w) x = op(lane, x, s.part[turn][w][lane]);
    uint32_t b = 0;
    if (cs > 1) {
      if (wp == 0 && lane < n) s.total[turn][lane] = x;
      cluster_sync_all();
      x = 0;
      uint32_t y[8];   // all loads before their uses
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < cs && lane < n) y[c] = ld_cluster_u32(mapa(smem_u32(&s.total[turn][lane]), c));
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < cs && lane < n) {
          x = op(lane, x, y[c]);
          if (c < rank) b = op(lane, b, y[c]);
        }
    }
#pragma unroll
    for (int k = 0; k < n; ++k) {
      v[k] = __shfl_sync(0xffffffffu, x, k);
      before[k] = __shfl_sync(0xffffffffu, b, k);
    }
    turn ^= 1;   // the next exchange writes the other half while this one is read
  }
};

template <int T, bool kPos>
__global__ void __launch_bounds__(T, 1024 / T) drop_kernel(const DropParams p, int cs) {
  constexpr int kWarps = T / 32;
  constexpr uint32_t kSafe = 0xffffffffu;   // above every key: +inf has 0xff800000
  extern __shared__ uint4 keys[];           // [nv] vectors of four rows, then the places
  __shared__ DropShared<T> sh;
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int rank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int u = blockIdx.x / cs;
  const int64_t base = p.tok_off[u];
  const int N = static_cast<int>(p.tok_off[u + 1] - base);
  // this CTA's rows lo .. lo + n - 1 of the unit, in vectors that start at rows of
  // the whole arrays that are multiples of four: row 4 v + c - skew of the run is
  // element c of vector v; thread t has the vectors t, t + T, ...
  const int run = (N + cs - 1) / cs;
  const int lo = min(N, rank * run), n = min(N, lo + run) - lo;
  const int skew = static_cast<int>((base + lo) & 3);
  const int nv = (n + skew + 3) >> 2;
  const int nr = (nv + T - 1) / T;        // rounds over the vectors
  uint32_t* cnt = reinterpret_cast<uint32_t*>(keys + nv);   // [nr * kWarps + 1]
  const int64_t at0 = base + lo - skew;   // row of element 0 of vector 0
  Exchange<T> ex = {sh, cs, rank, 0};
  if (tid < kBins / 4) sh.hist[0][tid] = sh.hist[1][tid] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) sh.listed = 0u;
  auto whole = [&](int v) { return p.vec && 4 * v >= skew && 4 * v + 4 <= n + skew; };
  auto inside = [&](int v, int c) { return 4 * v + c >= skew && 4 * v + c < n + skew; };
  // the loads of a vector that is not whole
  auto live4 = [&](int v) -> uint32_t {
    uint32_t x = 0u;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (inside(v, c))
        x |= (p.live ? static_cast<uint32_t>(p.live[at0 + 4 * v + c]) : 1u) << (8 * c);
    return x;
  };
  auto pos4 = [&](int v) -> int4 {
    if (!kPos) {
      const int x = lo - skew + 4 * v;
      return make_int4(x, x + 1, x + 2, x + 3);
    }
    int x[4] = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (inside(v, c)) x[c] = p.pos[at0 + 4 * v + c];
    return make_int4(x[0], x[1], x[2], x[3]);
  };
  auto acc4 = [&](int v) -> float4 {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (inside(v, c)) x[c] = p.acc[at0 + 4 * v + c];
    return make_float4(x[0], x[1], x[2], x[3]);
  };

  // Keys of this thread's rows and what they say: the largest, the smallest, the smallest
  // above that of 0 (less it), their number, that of those not above 0, and the newest live
  // position.
  constexpr uint32_t kZero = 0x80000000u;   // the key of 0
  uint32_t kmax, kmin, kpos, count, low_count;
  int newest;
  auto rank_rows = [&](int recent) {
    kmax = count = low_count = 0u;
    kmin = kpos = 0xffffffffu;
    newest = INT_MIN;
    auto see = [&](uint32_t q) {
      kmax = max(kmax, q);
      kmin = min(kmin, q);
      const uint32_t d = q - (kZero + 1u);   // its top bit: not above
      kpos = min(kpos, d);
      low_count += d >> 31;
    };
    // two vectors' loads in flight, without a branch between them (replayed: 23.8 and 26.3 us one
    // by one, 22.5 and 25.8 two, 22.0 and 25.7 four: 2048 units of 2176 rows, 64 of 31K with
    // positions)
    for (int v0 = tid; v0 < nv; v0 += 2 * T) {
      float4 fa[2];
      uint32_t fl[2];
      int4 fy[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int v = v0 + j * T;
        const bool on = v < nv && whole(v);
        fl[j] = 0x01010101u;
        if (on) fa[j] = *reinterpret_cast<const float4*>(p.acc + at0 + 4 * v);
        if (on && p.live) fl[j] = *reinterpret_cast<const uint32_t*>(p.live + at0 + 4 * v);
        if (on && kPos) fy[j] = *reinterpret_cast<const int4*>(p.pos + at0 + 4 * v);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int v = v0 + j * T;
        if (v >= nv) break;
        const bool full = whole(v);
        const float4 a = full ? fa[j] : acc4(v);
        const uint32_t l = full ? fl[j] : live4(v);
        const int4 y = full && kPos ? fy[j] : pos4(v);
        const float sum = (a.x + a.y) + (a.z + a.w);
        const int high = max(max(y.x, y.y), max(y.z, y.w));
        uint4 k;
        if (l == 0x01010101u && sum == sum && min(min(y.x, y.y), min(y.z, y.w)) >= p.sinks &&
            high <= recent) {
          // four ranked rows, and no NaN among them
          k = make_uint4(number_key(a.x), number_key(a.y), number_key(a.z), number_key(a.w));
          see(k.x);
          see(k.y);
          see(k.z);
          see(k.w);
          count += 4u;
          newest = max(newest, high);
        } else {
          auto one = [&](float w, int x, int c) -> uint32_t {
            if (!((l >> (8 * c)) & 0xffu)) return 0u;
            newest = max(newest, x);
            if (x < p.sinks || x > recent) return kSafe;
            const uint32_t q = weight_key(w);
            see(q);
            ++count;
            return q;
          };
          k = make_uint4(one(a.x, y.x, 0), one(a.y, y.y, 1), one(a.z, y.z, 2), one(a.w, y.w, 3));
        }
        keys[v] = k;
      }
    }
  };
  auto window = [&](int x) { return x < INT_MIN + p.w ? INT_MIN : x - p.w; };   // above: stay
  if (kPos || p.live) {
    // the newest live position comes out of the same pass; threads that have rows of the
    // window then go over theirs again
    rank_rows(INT_MAX);
    uint32_t m[1] = {static_cast<uint32_t>(__reduce_max_sync(0xffffffffu, newest)) ^ 0x80000000u};
    uint32_t b[1];
    ex.all(m, b, [](int, uint32_t a, uint32_t x) { return a > x ? a : x; });
    const int recent = window(static_cast<int>(m[0] ^ 0x80000000u));
    if (newest > recent) rank_rows(recent);
    __syncwarp();
  } else {
    rank_rows(window(N - 1));
  }
  // smallest keys as their complements
  uint32_t m[5] = {__reduce_max_sync(0xffffffffu, kmax), ~__reduce_min_sync(0xffffffffu, kmin),
                   __reduce_add_sync(0xffffffffu, count), ~__reduce_min_sync(0xffffffffu, kpos),
                   __reduce_add_sync(0xffffffffu, low_count)};
  uint32_t bm[5];
  ex.all(m, bm, [](int k, uint32_t a, uint32_t x) {
    return k == 2 || k == 4 ? a + x : a > x ? a : x;
  });
  const uint32_t ranked = m[2];
  int budget = p.budget;
  if (p.budgets) budget = min(max(p.budgets[u], 0), p.budget);

  // rows with key > thr stay, and (some_ties) of those with key = thr the unit's first `ties`
  uint32_t thr = 0u, ties = 0u;
  bool some_ties = false;
  if (budget == 0) {
    thr = kSafe - 1u;
  } else if (ranked > static_cast<uint32_t>(budget)) {
    uint32_t want = budget;
    // the keys that are left: low .. high, high = low + span; `want` counts from high down, so
    // a key above it must never be taken in again.  Rows of weight 0 (new tokens) would stretch
    // the range over all exponents and crowd the others into few bins: the last row to stay lies
    // either above 0 or not.
    uint32_t high = m[0], low = ~m[1];
    const uint32_t positive = ranked - m[4];
    if (positive >= want) {
      low = ~m[3] + kZero + 1u;
    } else {
      want -= positive;
      high = kZero;
    }
    uint32_t span = high - low;
    some_ties = true;
    for (int round = 0; span > 0u; ++round) {
      const int shift = max(0, 32 - __clz(span) - kBinBits);
      uint32_t* hist = reinterpret_cast<uint32_t*>(sh.hist[round & 1]);
#pragma unroll 2
      for (int v = tid; v < nv; v += T) {
        const uint4 k = keys[v];
        if (k.x - low <= span) atomicAdd(&hist[(k.x - low) >> shift], 1u);
        if (k.y - low <= span) atomicAdd(&hist[(k.y - low) >> shift], 1u);
        if (k.z - low <= span) atomicAdd(&hist[(k.z - low) >> shift], 1u);
        if (k.w - low <= span) atomicAdd(&hist[(k.w - low) >> shift], 1u);
      }
      if (cs > 1) cluster_sync_all();
      else __syncthreads();
      // thread t < 128: bins kBins - 1 - 4 t downwards
      uint32_t h[4] = {0u, 0u, 0u, 0u};   // from the top
      if (tid < kBins / 4) {
        const int k = kBins / 4 - 1 - tid;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (cs > 1) {
          uint4 y[8];
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < cs) y[q] = ld_cluster_v4(mapa(smem_u32(&sh.hist[round & 1][k]), q));
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < cs) {
              x.x += y[q].x;
              x.y += y[q].y;
              x.z += y[q].z;
              x.w += y[q].w;
            }
        } else {
          x = sh.hist[round & 1][k];
        }
        h[0] = x.w;
        h[1] = x.z;
        h[2] = x.y;
        h[3] = x.x;
        // the other one has been read by every CTA: clear it for the next round
        sh.hist[(round + 1) & 1][k] = make_uint4(0u, 0u, 0u, 0u);
      }
      const uint32_t mine = h[0] + h[1] + h[2] + h[3];
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) sh.wsum[wp] = incl;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 3; ++w)
        if (w < wp) incl += sh.wsum[w];   // bins lie in the first four warps
      uint32_t above = incl - mine;
      if (wp < 4 && above < want && want <= incl) {   // one thread
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (above < want && want <= above + h[k]) {
            sh.found[0] = kBins - 1 - 4 * tid - k;
            sh.found[1] = h[k];
            sh.found[2] = want - above;
          }
          above += h[k];
        }
      }
      __syncthreads();
      const uint32_t in_bin = sh.found[1];
      low += sh.found[0] << shift;
      want = sh.found[2];
      span = min((1u << shift) - 1u, high - low);
      high = low + span;
      if (want == in_bin) {   // the whole bin stays
        thr = low - 1u;
        some_ties = false;
        break;
      }
      if (span == 0u) break;
      if (cs == 1 && in_bin <= kList) {
        // few rows left, in_bin of them: each one's rank by comparing it with the others
        for (int v = tid; v < nv; v += T) {
          const uint4 k = keys[v];
          auto put = [&](uint32_t x) {
            if (x - low > span) return;
            const uint32_t to = atomicAdd(&sh.listed, 1u);
            if (to < kList) sh.list[to] = x;
          };
          put(k.x);
          put(k.y);
          put(k.z);
          put(k.w);
        }
        __syncthreads();
        if (tid < static_cast<int>(in_bin)) {
          const uint32_t own = sh.list[tid];
          uint32_t above_own = 0, same = 0;
          for (uint32_t k = 0; k < in_bin; ++k) {
            const uint32_t x = sh.list[k];
            above_own += x > own ? 1u : 0u;
            same += x == own ? 1u : 0u;
          }
          if (above_own < want && want <= above_own + same) {   // rows of one key
            sh.found[0] = own;
            sh.found[1] = same;
            sh.found[2] = want - above_own;
          }
        }
        __syncthreads();
        thr = low = sh.found[0];
        want = sh.found[2];
        some_ties = want != sh.found[1];
        if (!some_ties) --thr;
        break;
      }
      if (in_bin * 16u > ranked) {
        // so many rows in one bin are likely equal: the range of their keys, which need not
        // end where the next bins cut from it do
        uint32_t x[2] = {0u, 0u}, b[2];
        for (int v = tid; v < nv; v += T) {
          const uint4 k = keys[v];
          auto see = [&](uint32_t y) {
            if (y - low <= span) {
              x[0] = max(x[0], y);
              x[1] = max(x[1], ~y);
            }
          };
          see(k.x);
          see(k.y);
          see(k.z);
          see(k.w);
        }
        x[0] = __reduce_max_sync(0xffffffffu, x[0]);
        x[1] = __reduce_max_sync(0xffffffffu, x[1]);
        ex.all(x, b, [](int, uint32_t a, uint32_t y) { return a > y ? a : y; });
        low = ~x[1];
        high = x[0];
        span = high - low;
      }
    }
    if (some_ties) {
      thr = low;
      ties = want;
    }
  }

  // Bits of every vector's rows that stay (g), and of those equal to a threshold that not
  // all of them pass (e), with the numbers set in lower lanes' vectors of the round, over
  // its keys: g | e << 4 | lower g << 8 | lower e << 24.  cnt[round kWarps + warp] gets the
  // numbers set in this CTA before that warp and round, g | e << 16.
  __syncthreads();
  for (int r = 0; r < nr; ++r) {
    const int v = r * T + tid;
    uint32_t g = 0u, e = 0u;
    if (v < nv) {
      const uint4 k = keys[v];
      g = (k.x > thr ? 1u : 0u) | (k.y > thr ? 2u : 0u) | (k.z > thr ? 4u : 0u) |
          (k.w > thr ? 8u : 0u);
      if (some_ties)
        e = (k.x == thr ? 1u : 0u) | (k.y == thr ? 2u : 0u) | (k.z == thr ? 4u : 0u) |
            (k.w == thr ? 8u : 0u);
    }
    const uint32_t own = __popc(g) | __popc(e) << 16;
    uint32_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (v < nv) keys[v].x = g | e << 4 | (incl - own) << 8;
    if (lane == 31) cnt[r * kWarps + wp] = incl;
  }
  __syncthreads();
  const int used = nr * kWarps;
  if (wp == 0) {
    uint32_t carry = 0;
    for (int k0 = 0; k0 < used; k0 += 32) {
      const uint32_t x = k0 + lane < used ? cnt[k0 + lane] : 0u;
      uint32_t y = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      if (k0 + lane < used) cnt[k0 + lane] = carry + y - x;
      carry += __shfl_sync(0xffffffffu, y, 31);
    }
    if (lane == 0) cnt[used] = carry;
  }
  __syncthreads();
  // the numbers of both in the unit, and in the CTAs before this one
  uint32_t all[2] = {cnt[used] & 0xffffu, cnt[used] >> 16}, before[2] = {0u, 0u};
  if (cs > 1) {
    if (wp > 0) all[0] = all[1] = 0u;
    ex.all(all, before, [](int, uint32_t x, uint32_t y) { return x + y; });
  }
  const int nk = static_cast<int>(all[0] + min(all[1], ties));   // rows that stay
  int32_t* idx = p.idx ? p.idx + static_cast<int64_t>(u) * p.W : nullptr;
  int32_t* fs = p.free_slots + base;
#pragma unroll 2
  for (int r = 0; r < nr; ++r) {
    const int v = r * T + tid;
    if (v >= nv) continue;
    // a row's place among those that stay: the ones before it in g, and of those in e the
    // unit's first `ties`
    const uint32_t x = keys[v].x, first = cnt[r * kWarps + wp];
    uint32_t k = x & 15u;
    int at = static_cast<int>(before[0] + (first & 0xffffu) + ((x >> 8) & 255u));
    if (some_ties) {
      uint32_t ae = before[1] + (first >> 16) + (x >> 24);
      at += min(ae, ties);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if ((x >> (4 + c)) & 1u) {
          if (ae < ties) k |= 1u << c;
          ++ae;
        }
    }
    const int64_t g = at0 + 4 * v;
    const bool full = whole(v);
    const int row0 = lo - skew + 4 * v;
    // the weights again (a key does not tell -0 from 0)
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.acc_out) a = full ? *reinterpret_cast<const float4*>(p.acc + g) : acc4(v);
    const float4 o = make_float4(k & 1u ? a.x : 0.f, k & 2u ? a.y : 0.f, k & 4u ? a.z : 0.f,
                                 k & 8u ? a.w : 0.f);
    if (full) {
      *reinterpret_cast<uint32_t*>(p.keep + g) = (k * 0x00204081u) & 0x01010101u;   // bits to bytes
      if (p.acc_out) *reinterpret_cast<float4*>(p.acc_out + g) = o;
    } else {
      const float w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (inside(v, c)) {
          p.keep[g + c] = (k >> c) & 1u;
          if (p.acc_out) p.acc_out[g + c] = w[c];
        }
    }
    uint32_t gone = ~k & 15u;
    if (!full)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (!inside(v, c)) gone &= ~(1u << c);
    // a free row's place is its row less the rows before it that stay; outside rows (of the
    // first vector) lie before them
    const int out = !full && skew > 4 * v ? skew - 4 * v : 0;
    int32_t* f = fs + (row0 + out - at);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if ((gone >> c) & 1u) *f++ = row0 + c;
    if (idx) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if ((k >> c) & 1u) {
          if (at < p.W) idx[at] = row0 + c;
          ++at;
        }
    }
  }
  // what is left of the list and of idx
  const int rest = N - nk;
  const int whole0 = p.vec ? rest + static_cast<int>(-(base + rest) & 3) : N;   // aligned
  for (int i = rest + rank * T + tid; i < min(whole0, N); i += cs * T) fs[i] = -1;
  for (int i = whole0 + 4 * (rank * T + tid); i < N; i += 4 * cs * T) {
    if (i + 4 <= N) {
      *reinterpret_cast<int4*>(fs + i) = make_int4(-1, -1, -1, -1);
    } else {
      for (int k = i; k < N; ++k) fs[k] = -1;
    }
  }
  if (idx)
    for (int i = nk + rank * T + tid; i < p.W; i += cs * T) idx[i] = -1;
  if (rank == 0 && tid == 0) {
    p.n_free[u] = N - nk;
    if (p.n_kept) p.n_kept[u] = min(nk, p.W);
    // more rows than a row of idx holds: positions that occur twice
    if (idx && nk > p.W) atomicOr(p.status, kStatusBadIndex);
  }
  if (cs > 1) cluster_sync_all();   // a CTA's shared memory is read until here
}

// Dynamic shared memory of a run of r rows: up to (r + 6) / 4 vectors, and their places.
template <int T>
int drop_smem(int run) {
  const int nv = (run + 6) / 4;
  return nv * 16 + ((nv + T - 1) / T * (T / 32) + 1) * 4;
}

template <int T, bool kPos>
cudaError_t launch_one(const DropParams& p, int U, int run, int cs, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(U) * cs);
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = drop_smem<T>(run);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cs > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, drop_kernel<T, kPos>, p, cs);
  return e != cudaSuccess ? e : cudaGetLastError();
}

constexpr int kMaxRun = 16384;   // rows of a CTA, 64 KB of keys

template <int T, bool kPos>
cudaError_t configure_one() {
  return cudaFuncSetAttribute(drop_kernel<T, kPos>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              drop_smem<T>(kMaxRun));
}

}  // namespace

cudaError_t drop_configure() {
  cudaError_t e = configure_one<128, false>();
  if (e == cudaSuccess) e = configure_one<128, true>();
  if (e == cudaSuccess) e = configure_one<256, false>();
  if (e == cudaSuccess) e = configure_one<256, true>();
  if (e == cudaSuccess) e = configure_one<512, false>();
  if (e == cudaSuccess) e = configure_one<512, true>();
  return e;
}

// As many threads per unit as the GPU holds for all units at once (1024 per SM at 64
// registers), at least 128, with a vector each in one CTA and two in a cluster, and at
// most kMaxRun rows a CTA.  Measured, replayed: 2048 units of 2176 rows 23 / 28 / 39 us with
// 128 / 256 / 512 threads, 148 units 6.5 / 5.3 / 5.1; 64 units of 32768 rows, half of them live,
// with positions, 53 / 34 / 25 us in two CTAs, as few as hold them, 24 in four of 512 threads
// and 40 in eight; 8 such units 22 us in two CTAs of 512 threads, 16 in four, 14.5 in eight.
cudaError_t launch_drop(const DropParams& p, int U, int nmax, int nsm, cudaStream_t st) {
  const int64_t threads = 1024ll * nsm / U, nv = (nmax + 3) / 4;
  int T = 128, cs = 1;
  while (T < 512 && 2 * T <= threads && 2 * T <= nv) T *= 2;
  while (cs < 8 && ((T == 512 && 2 * cs * T <= threads && 4 * cs * T <= nv) || nmax > kMaxRun * cs))
    cs *= 2;
  const int run = (nmax + cs - 1) / cs;
  if (T == 128)
    return p.pos ? launch_one<128, true>(p, U, run, cs, st)
                 : launch_one<128, false>(p, U, run, cs, st);
  if (T == 256)
    return p.pos ? launch_one<256, true>(p, U, run, cs, st)
                 : launch_one<256, false>(p, U, run, cs, st);
  return p.pos ? launch_one<512, true>(p, U, run, cs, st)
               : launch_one<512, false>(p, U, run, cs, st);
}

}  // namespace rkv
