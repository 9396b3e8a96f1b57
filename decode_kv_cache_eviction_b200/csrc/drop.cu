// Eviction by accumulated attention weight.  Of a unit's live rows the sinks
// (position < sinks) and the w newest positions stay, and of the others the
// `budget` rows of largest weight (ties: lowest row first; -0 = +0; NaN last).
//
// One cluster of 1 to 8 CTAs per unit, each with a run of the unit's rows in its
// registers (V vectors of four consecutive rows per thread), so acc, live and pos
// are read once.  Weights become order-preserving 32-bit keys; histograms of 512
// bins over the range of the keys that are left (added over distributed shared
// memory in a cluster) narrow it down to the threshold key, and stop as soon as a
// bin is taken whole.  Starting from the keys' own range spreads them over the
// bins, so few of the shared-memory additions meet, and two or three rounds are
// enough where weights differ.  Ballots then give every row its place among the
// kept and the free rows of the unit.
//
// Bound: instruction issue and the latency of a few dependent block reductions
// at small units, HBM beyond; hence the vectors, and short runs on 128-thread
// CTAs, which keep many units in flight.
#include <limits.h>

#include "ptx.cuh"
#include "rkv_internal.cuh"

namespace rkv {
namespace {

// Order-preserving key of a weight, at least 1: -0 and +0 alike, NaN below
// every number.  0 marks a row that is not ranked.
__device__ __forceinline__ uint32_t weight_key(float s) {
  const uint32_t b = __float_as_uint(__fadd_rn(s, 0.f));
  const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return s == s ? k : 1u;   // -inf has key 0x007fffff
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

template <int T>
struct DropShared {
  uint4 hist[2][kBins / 4];      // two in turn
  uint32_t part[2][T / 32][4];   // the warps' values of an exchange (two in turn)
  uint32_t total[2][4];          // this CTA's
  uint32_t wsum[T / 32];
  uint32_t found[3];             // bin, its rows, rows wanted of it
};

// Exchanges of up to 4 values over the CTA and the cluster.
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

template <int T, int V, bool kPos>
__global__ void __launch_bounds__(T) drop_kernel(const DropParams p, int cs) {
  constexpr int kWarps = T / 32;
  __shared__ DropShared<T> sh;
  __shared__ uint32_t cnt[V * kWarps + 1];
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const unsigned below = (1u << lane) - 1u;
  const int rank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int u = blockIdx.x / cs;
  const int64_t base = p.tok_off[u];
  const int N = static_cast<int>(p.tok_off[u + 1] - base);
  // this CTA's rows lo .. lo + n - 1 of the unit, in vectors that start at rows of
  // the whole arrays that are multiples of four: row 4 (v T + tid) + c - skew of
  // the run is element c of vector v
  const int run = (N + cs - 1) / cs;
  const int lo = min(N, rank * run), n = min(N, lo + run) - lo;
  const int skew = static_cast<int>((base + lo) & 3);
  const int nv = (n + skew + 3) >> 2;
  const int64_t at0 = base + lo - skew;   // row of element 0 of vector 0
  Exchange<T> ex = {sh, cs, rank, 0};
  if (tid < kBins / 4) sh.hist[0][tid] = sh.hist[1][tid] = make_uint4(0u, 0u, 0u, 0u);
  auto first = [&](int v) { return 4 * (v * T + tid) - skew; };
  auto whole = [&](int j) { return p.vec && j >= 0 && j + 4 <= n; };

  uint32_t key[V][4];
  int ps[kPos ? V : 1][4];
  uint32_t lv[V];   // live bytes of a vector's rows (kept packed: nothing waits for the loads yet)
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      key[v][c] = 0u;
      if (kPos) ps[v][c] = 0;
    }
    lv[v] = 0u;
    if (v * T < nv) {
      const int j = first(v);
      const int64_t at = at0 + 4 * (v * T + tid);
      if (whole(j)) {
        const uint4 x = *reinterpret_cast<const uint4*>(p.acc + at);
        key[v][0] = x.x;
        key[v][1] = x.y;
        key[v][2] = x.z;
        key[v][3] = x.w;
        lv[v] = p.live ? *reinterpret_cast<const uint32_t*>(p.live + at) : 0x01010101u;
        if (kPos) {
          const int4 z = *reinterpret_cast<const int4*>(p.pos + at);
          ps[v][0] = z.x;
          ps[v][1] = z.y;
          ps[v][2] = z.z;
          ps[v][3] = z.w;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (j + c >= 0 && j + c < n) {
            key[v][c] = __float_as_uint(p.acc[at + c]);
            lv[v] |= (p.live ? static_cast<uint32_t>(p.live[at + c]) : 1u) << (8 * c);
            if (kPos) ps[v][c] = p.pos[at + c];
          }
      }
    }
  }
  auto place = [&](int v, int c) { return kPos ? ps[v][c] : lo + first(v) + c; };
  // the newest live position
  int newest = N - 1;
  if (kPos || p.live) {
    int x = INT_MIN;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * T < nv) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((lv[v] >> (8 * c)) & 0xffu) x = max(x, place(v, c));
      }
    uint32_t m[1] = {static_cast<uint32_t>(__reduce_max_sync(0xffffffffu, x)) ^ 0x80000000u}, b[1];
    ex.all(m, b, [](int, uint32_t a, uint32_t x) { return a > x ? a : x; });
    newest = static_cast<int>(m[0] ^ 0x80000000u);
  }
  // positions above it stay (a position is at least INT_MIN + 1 here or nothing is live)
  const int recent = newest < INT_MIN + p.w ? INT_MIN : newest - p.w;
  uint32_t kmax = 0u, kinv = 0u, count = 0u;   // kinv: complement of the smallest key
  uint32_t safe[V];                            // bit c: element c stays unranked
#pragma unroll
  for (int v = 0; v < V; ++v) {
    safe[v] = 0u;
    if (v * T < nv) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int x = place(v, c);
        const bool s = x < p.sinks || x > recent;
        const bool on = ((lv[v] >> (8 * c)) & 0xffu) != 0u;
        if (on && s) safe[v] |= 1u << c;
        const uint32_t k = on && !s ? weight_key(__uint_as_float(key[v][c])) : 0u;
        key[v][c] = k;
        kmax = max(kmax, k);
        kinv = max(kinv, k ? ~k : 0u);
        count += k ? 1u : 0u;
      }
    }
  }
  uint32_t m[3] = {__reduce_max_sync(0xffffffffu, kmax), __reduce_max_sync(0xffffffffu, kinv),
                   __reduce_add_sync(0xffffffffu, count)};
  uint32_t bm[3];
  ex.all(m, bm, [](int k, uint32_t a, uint32_t x) { return k == 2 ? a + x : a > x ? a : x; });
  const uint32_t ranked = m[2];
  int budget = p.budget;
  if (p.budgets) budget = min(max(p.budgets[u], 0), p.budget);

  // ranked rows with key > thr stay, and the first `ties` rows with key = thr
  uint32_t thr = 0u, ties = 0u;
  bool some_ties = false;
  if (budget == 0) {
    thr = 0xffffffffu;
  } else if (ranked > static_cast<uint32_t>(budget)) {
    uint32_t want = budget;
    uint32_t low = ~m[1];              // the keys that are left: low .. low + 2^bits - 1
    int bits = 32 - __clz(m[0] - low);
    some_ties = true;
    for (int round = 0; bits > 0; ++round) {
      const int shift = max(0, bits - kBinBits);
      const uint32_t bins = 1u << (bits - shift);
      uint32_t* hist = reinterpret_cast<uint32_t*>(sh.hist[round & 1]);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * T < nv) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t x = (key[v][c] - low) >> shift;
            if (key[v][c] >= low && key[v][c] != 0u && x < bins) atomicAdd(&hist[x], 1u);
          }
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
      const uint32_t bin = sh.found[0], in_bin = sh.found[1];
      want = sh.found[2];
      low += bin << shift;
      bits = shift;
      if (want == in_bin) {   // the whole bin stays
        thr = low - 1u;
        some_ties = false;
        break;
      }
    }
    if (some_ties) {
      thr = low;
      ties = want;
    }
  }

  uint32_t kept[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    kept[v] = safe[v];
#pragma unroll
    for (int c = 0; c < 4; ++c) kept[v] |= (key[v][c] > thr ? 1u : 0u) << c;
  }
  // Of one bit per row: the number set in lower lanes' elements of vector v, and in
  // cnt[v kWarps + warp] (after scan) the number set in warps before.
  auto lower = [&](uint32_t b) {
    int k = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) k += __popc(__ballot_sync(0xffffffffu, (b >> c) & 1u) & below);
    return k;
  };
  auto scan = [&](const uint32_t (&b)[V], uint32_t& total) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * T < nv) {
        const uint32_t k = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(__popc(b[v])));
        if (lane == 0) cnt[v * kWarps + wp] = k;
      }
    __syncthreads();
    const int used = ((nv + T - 1) / T) * kWarps;
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
      if (lane == 0) cnt[V * kWarps] = carry;
    }
    __syncthreads();
    total = cnt[V * kWarps];
  };
  // the CTAs' totals: over the cluster, and of the CTAs before this one
  auto across = [&](uint32_t mine, uint32_t& total, uint32_t& before) {
    total = mine;
    before = 0;
    if (cs > 1) {
      uint32_t a[1] = {wp == 0 ? mine : 0u}, b[1];
      ex.all(a, b, [](int, uint32_t x, uint32_t y) { return x + y; });
      total = a[0];
      before = b[0];
    }
  };
  uint32_t total, all, before;
  if (some_ties) {
    uint32_t tb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      tb[v] = 0u;
#pragma unroll
      for (int c = 0; c < 4; ++c) tb[v] |= (key[v][c] == thr ? 1u : 0u) << c;
    }
    scan(tb, total);
    across(total, all, before);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * T < nv) {
        uint32_t at = before + cnt[v * kWarps + wp] + lower(tb[v]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((tb[v] >> c) & 1u) {
            if (at < ties) kept[v] |= 1u << c;
            ++at;
          }
      }
  }
  scan(kept, total);
  across(total, all, before);
  int32_t* idx = p.idx ? p.idx + static_cast<int64_t>(u) * p.W : nullptr;
  int32_t* fs = p.free_slots + base;
  float4 a[V];   // the weights again (a key does not tell -0 from 0), all loads at once
  if (p.acc_out) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * T < nv && whole(first(v)))
        a[v] = *reinterpret_cast<const float4*>(p.acc + at0 + 4 * (v * T + tid));
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * T < nv) {
      int at = static_cast<int>(before + cnt[v * kWarps + wp]) + lower(kept[v]);
      const int j = first(v);
      const int64_t g = at0 + 4 * (v * T + tid);
      const bool full = whole(j);
      const uint32_t k = kept[v];
      if (full) {
        *reinterpret_cast<uchar4*>(p.keep + g) =
            make_uchar4(k & 1u, (k >> 1) & 1u, (k >> 2) & 1u, (k >> 3) & 1u);
        if (p.acc_out) {
          *reinterpret_cast<float4*>(p.acc_out + g) =
              make_float4(k & 1u ? a[v].x : 0.f, k & 2u ? a[v].y : 0.f, k & 4u ? a[v].z : 0.f,
                          k & 8u ? a[v].w : 0.f);
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (j + c >= 0 && j + c < n) {
          const bool stays = (k >> c) & 1u;
          const int row = lo + j + c;
          if (!full) {
            p.keep[g + c] = stays ? 1 : 0;
            if (p.acc_out) p.acc_out[g + c] = stays ? p.acc[g + c] : 0.f;
          }
          if (!stays) fs[row - at] = row;
          else if (idx && at < p.W) idx[at] = row;
          at += stays ? 1 : 0;
        }
    }
  // what is left of the list and of idx
  const int nk = static_cast<int>(all);
  for (int i = N - nk + rank * T + tid; i < N; i += cs * T) fs[i] = -1;
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

template <int T, int V, bool kPos>
cudaError_t launch_one(const DropParams& p, int U, int cs, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(U) * cs);
  cfg.blockDim = dim3(T);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cs > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, drop_kernel<T, V, kPos>, p, cs);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// A run of r rows takes up to (r + 6) / 4 vectors.  With at most one CTA per SM a run is
// spread over more threads: eight units of 32768 rows take 12.7 us instead of 19.3, but
// 64 units 32.4 instead of 25.8, since their CTAs no longer fit on the SMs at once.
template <bool kPos>
cudaError_t launch_pos(const DropParams& p, int U, int run, int cs, bool few, cudaStream_t st) {
  if (few) {
    if (run + 6 <= 4 * 1 * 512) return launch_one<512, 1, kPos>(p, U, cs, st);
    if (run + 6 <= 4 * 3 * 512) return launch_one<512, 3, kPos>(p, U, cs, st);
  }
  if (run + 6 <= 4 * 2 * 128) return launch_one<128, 2, kPos>(p, U, cs, st);
  if (run + 6 <= 4 * 5 * 128) return launch_one<128, 5, kPos>(p, U, cs, st);
  if (run + 6 <= 4 * 9 * 128) return launch_one<128, 9, kPos>(p, U, cs, st);
  return launch_one<512, 9, kPos>(p, U, cs, st);
}

}  // namespace

// CTAs per unit: as many as fill the GPU twice, with runs of 1024 rows at least,
// and at most 16384 rows a CTA (512 threads, nine vectors each).
cudaError_t launch_drop(const DropParams& p, int U, int nmax, int nsm, cudaStream_t st) {
  int cs = 1;
  while (cs < 8 && ((static_cast<int64_t>(U) * cs < 2 * nsm && nmax > 1024 * cs) ||
                    nmax > 16384 * cs))
    cs *= 2;
  const int run = (nmax + cs - 1) / cs;
  const bool few = static_cast<int64_t>(U) * cs <= nsm;
  return p.pos ? launch_pos<true>(p, U, run, cs, few, st)
               : launch_pos<false>(p, U, run, cs, few, st);
}

}  // namespace rkv
