// Attention of many query rows over a shared prefix: all queries of a prefix's
// units against its K and V at once, on the tensor cores.  (A unit of many query
// rows of its own is a prefix with itself as its only unit.)
//
// A CTA takes 128 or 256 query rows (one or two tiles of 128, gathered from their
// units) and a run of 128-token tiles of the prefix:
//   S = Q K^T        tcgen05.mma, Q and K from shared memory (128-byte swizzle),
//                    S in tensor memory: lane = query row, column = token;
//   p = 2^(S - m)    four threads per query row (two shuffles for its maximum), 16 rows
//                    per warp; p goes back over S as bf16;
//   O += p V         tcgen05.mma with p as the A operand from tensor memory and V
//                    (token rows) as an MN-major B operand: V is never transposed.
// With two query tiles their steps alternate, so the tensor cores work on one while
// the other's p is formed, and each K/V tile in shared memory serves 256 query rows;
// with one, it has two S buffers.  (Two buffers of 64 tokens for each of two tiles
// fit as well, but products of N = 64 take as long as of N = 128: 3400 cycles per
// 128 tokens instead of 2900.)  p is handed over in halves of 64 tokens, so the first
// half's product runs while the second is formed.  The MMAs of one thread run in the
// order of their issue; a later S, written over p, therefore follows the product that
// reads p.
//
// One thread per row, 128 tokens each, needs no shuffles, but with one or two warps per
// scheduler its chain of loads, maximum and 2^x took 2300 of a step's 3500 cycles.
//
// The running maximum m is moved (and O, l rescaled by the same threads) only when
// a row's maximum has grown by more than 2^8: p, l and O stay well inside fp32 and
// bf16's relative precision does not depend on the scale, so the result is the
// same and most steps need no pass over O.
//
// p is rounded to bf16 (2^-8 relative at most, once per weight, of random sign): the
// product needs V's type, and a second part would cost half as many MMAs again.
//
// Bound: at 256 rows and d = 128 a 128-token tile takes 2048 tensor-core cycles and as
// many for its 2^x (16 per cycle and SM); a quarter of those run on the FMA pipe.
// With one tile of rows it is HBM.
//
// Roles: warps 0-7 and 8-15 the rows of the first and second query tile (warp w: rows
// 32 (w % 4) + 16 (w / 4 % 2) of its tile, the tensor-memory lanes that it may read),
// then a TMA producer (one lane) and an MMA issuer.  Every wait is bounded.
//
// A row whose result is not finite is marked and computed again, token by token,
// by the join: a value that is not finite in a row that it does not see (behind its
// window, after the prefix's end) also meets its p = 0 in the product.
#include "attend_common.cuh"

namespace rkv {
namespace {

constexpr int kWTile = kWideTile;
constexpr uint32_t kTileB = kWTile * 256;   // a K, V or Q tile: two halves of 64 columns
constexpr uint32_t kHalfB = kTileB / 2;
constexpr uint64_t kDrainNs = 100000000ull;
constexpr float kSlack = 8.f;   // growth of a maximum (log2) that O is not rescaled for

template <int QT>
struct WideLayout {
  static constexpr int kStages = QT == 2 ? 5 : 6;   // K and V tiles in turn
  static constexpr int kBuf = QT == 2 ? 1 : 2;      // S buffers of a query tile
  static constexpr uint32_t q = 0;
  static constexpr uint32_t ring = QT * kTileB;
  static constexpr uint32_t row = ring + kStages * kTileB;      // [QT * 128] rows of Q
  static constexpr uint32_t bars = row + QT * kWTile * 4;
  static constexpr uint32_t misc = bars + (2 * kStages + 10) * 8;
  static constexpr uint32_t total = misc + 96;
  static constexpr uint32_t alloc = total + 1024;               // base aligned to 1024
};

// 2^x for a pair of x in [-126, 127] on the FMA pipe (2^x has 16 lanes' worth of its
// own per cycle and SM, as many as the tensor cores leave for it).  x = n + f with n
// the nearest whole number, added as 1.5 2^23 + n so that its low bits are n; a
// polynomial of degree 4 for 2^f, |f| <= 1/2, fitted for the smallest largest
// relative error, 2.6e-6 (2^-18.5: far below the rounding to bf16 that follows); n is
// added to the exponent.  x <= -126 (an unseen token) gives 2^-126, which is taken off
// everywhere: the largest finite V times what is left is below 1e-5.  NaN is caught by
// the row's maximum.
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x) {
  float x0, x1;
  unpair(x, x0, x1);
  x = pair(fmaxf(x0, -126.f), fmaxf(x1, -126.f));
  const uint64_t t = add_pair(x, pair(12582912.f, 12582912.f));
  const uint64_t n = add_pair(t, pair(-12582912.f, -12582912.f));
  const uint64_t f = fma_pair(n, pair(-1.f, -1.f), x);
  uint64_t y = pair(0.009570101276040077f, 0.009570101276040077f);
  y = fma_pair(y, f, pair(0.05591785907745361f, 0.05591785907745361f));
  y = fma_pair(y, f, pair(0.240247443318367f, 0.240247443318367f));
  y = fma_pair(y, f, pair(0.6931217908859253f, 0.6931217908859253f));
  y = fma_pair(y, f, pair(0.9999992847442627f, 0.9999992847442627f));
  float t0, t1, y0, y1;
  unpair(t, t0, t1);
  unpair(y, y0, y1);
  return add_pair(pair(__uint_as_float(__float_as_uint(y0) + (__float_as_uint(t0) << 23)),
                       __uint_as_float(__float_as_uint(y1) + (__float_as_uint(t1) << 23))),
                  pair(-0x1p-126f, -0x1p-126f));
}

// Teardown: wait (bounded, regardless of an abort) for a phase that is under way.
__device__ __forceinline__ void wide_drain(uint64_t* bar, uint32_t par) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, par))
    if (globaltimer_ns() - t0 > kDrainNs) return;
}

template <int QT>
__global__ void __launch_bounds__(64 + 256 * QT, 1)
    wide_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const __grid_constant__ AttendParams p) {
  using Lay = WideLayout<QT>;
  constexpr int NS = Lay::kStages, kBuf = Lay::kBuf;
  constexpr int kRowWarps = 8 * QT;
  extern __shared__ uint8_t wide_raw[];
  allow_next_launch();   // the units' own rows, on SMs that have none of this
  uint8_t* sm = wide_raw + ((1024u - (smem_u32(wide_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + Lay::bars);
  uint64_t* empty = full + NS;
  // by tile and buffer (two of them in both forms): S is in tensor memory; the halves
  // of p are; their product with V is done
  uint64_t* s_full = empty + NS;    // [2]
  uint64_t* p_full = s_full + 2;    // [2][2]
  uint64_t* o_done = p_full + 4;    // [2]
  uint64_t* q_full = o_done + 2;    // Q is in shared memory
  uint64_t* mdone = q_full + 1;     // teardown: every MMA has completed
  int* s_row = reinterpret_cast<int*>(sm + Lay::row);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Lay::misc);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + Lay::misc + 4);
  int8_t* lastp = reinterpret_cast<int8_t*>(sm + Lay::misc + 8);      // [NS] parity of the last copy
  int* s_lim = reinterpret_cast<int*>(sm + Lay::misc + 16);           // [warp][2] smallest, largest qp
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int item = blockIdx.x / p.maxch, chunk = blockIdx.x - item * p.maxch;
  const unsigned from = (blockIdx.z * gridDim.y + blockIdx.y) * (QT * kWTile);   // below 2^32
  const int64_t base = __ldg(&p.pre_off[item]);
  const int N = static_cast<int>(__ldg(&p.pre_off[item + 1]) - base);
  const int mo = p.mem ? __ldg(&p.mem_off[item]) : item;
  const int total = p.mem ? (__ldg(&p.mem_off[item + 1]) - mo) * p.R : p.R;
  if (from >= static_cast<unsigned>(total)) return;
  const int row0 = static_cast<int>(from);
  const int nrow = min(QT * kWTile, total - row0);
  // Row warps that have query rows (a tile's first always works); the others only copy Q.
  // 64 units of 16000 rows, 32 query rows: 90 us either way at full clock, but 102 with all
  // eight at work and 96 with two in a long run under the power cap.
  auto row_warps = [&](int t) { return max(1, min(8, (nrow - t * kWTile + 15) / 16)); };

  // position of query row `row` (of all units): the newest query of its unit stands behind
  // the prefix and the unit's own rows
  auto place = [&](int row) {
    if (sees_whole_prefix(p)) return INT_MAX;
    const int u = row / p.R, x = row - u * p.R;
    const int64_t own = p.mem ? __ldg(&p.tok_off[u + 1]) - __ldg(&p.tok_off[u]) : 0;
    const int64_t newest = p.q_pos ? __ldg(&p.q_pos[u]) : N + own - 1;
    return clamp32(newest - (p.nq - 1) + x % p.nq);
  };
  if (tid < QT * kWTile) {
    int row = -1, qp = INT_MIN;
    if (tid < nrow) {
      const int k = (row0 + tid) / p.R;
      row = (p.mem ? __ldg(&p.mem[mo + k]) : item) * p.R + row0 + tid - k * p.R;
      qp = place(row);
    }
    s_row[tid] = row;
    const int lo = __reduce_min_sync(0xffffffffu, row >= 0 ? qp : INT_MAX);
    const int hi = __reduce_max_sync(0xffffffffu, qp);
    if (lane == 0) {
      s_lim[2 * warp] = lo;
      s_lim[2 * warp + 1] = hi;
    }
  } else if (warp == kRowWarps + 1) {
    tmem_alloc<1>(tmem_slot, 512);
    tmem_relinquish<1>();
  } else if (tid == kRowWarps * 32) {
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      lastp[s] = -1;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], row_warps(QT == 2 ? i : 0));
      mbar_init(&p_full[2 * i + 1], row_warps(QT == 2 ? i : 0));
      mbar_init(&o_done[i], 1);
    }
    mbar_init(q_full, kRowWarps);
    mbar_init(mdone, 1);
    *abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;   // S of tile t or buffer t: 128 t; O of tile t: 256 + 128 t
  int qmin = INT_MAX, qmax = INT_MIN;
#pragma unroll
  for (int w = 0; w < 4 * QT; ++w) {
    qmin = min(qmin, s_lim[2 * w]);
    qmax = max(qmax, s_lim[2 * w + 1]);
  }
  const Span sp = visible_span<7>(N, 0, qmin, qmax, p.local, p.sinks);
  const int v0 = chunk * p.gpc, nt = min(sp.nv, v0 + p.gpc) - v0;   // token tiles of this CTA
  if (nt <= 0) {
    if (tid < nrow)
      p.part_ml[static_cast<int64_t>(chunk) * p.rows + s_row[tid]] = make_float2(-INFINITY, 0.f);
    if (warp == kRowWarps + 1) tmem_dealloc<1>(tmem, 512);
    return;
  }
  if (warp < kRowWarps) {
    // query rows into the layout that TMA writes for K (zeros past the last row), all of
    // a thread's loads before its stores (one at a time they took 9 us)
    constexpr int kCopies = kWTile * 16 / 256;
    uint4 v[kCopies];
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      const int i = tid + k * kRowWarps * 32;
      const int src = s_row[i >> 4];
      v[k] = make_uint4(0u, 0u, 0u, 0u);
      if (src >= 0)
        v[k] = __ldg(reinterpret_cast<const uint4*>(p.Q) + static_cast<int64_t>(src) * 16 + (i & 15));
    }
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      const int i = tid + k * kRowWarps * 32;
      const int x = i >> 4, c = i & 15, xt = x & (kWTile - 1);
      *reinterpret_cast<uint4*>(sm + Lay::q + (x / kWTile) * kTileB + (c >> 3) * kHalfB + xt * 128 +
                                (((c & 7) ^ (xt & 7)) << 4)) = v[k];
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
  }

  if (warp == kRowWarps) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      for (int i = 0; i < 2 * nt; ++i) {
        const int s = i % NS;
        const uint32_t ph = (i / NS) & 1;
        // the first tiles only, until Q is there: its loads would wait behind the ring's
        // (10 us instead of 2 at 148 CTAs x 160 KB)
        if (i == 2 && !mbar_wait(q_full, 0, abort, p.status)) break;
        if (!mbar_wait(&empty[s], ph ^ 1, abort, p.status)) break;
        uint8_t* dst = sm + Lay::ring + s * kTileB;
        const int y = static_cast<int>(base + static_cast<int64_t>(sp.group(v0 + i / 2)) * kWTile);
        const CUtensorMap* map = (i & 1) ? &vmap : &kmap;
        mbar_arrive_expect_tx(&full[s], kTileB);
        tma_load_2d(dst, map, &full[s], 0, y, pol);
        tma_load_2d(dst + kHalfB, map, &full[s], 64, y, pol);
        lastp[s] = static_cast<int8_t>(ph);
      }
      // teardown: every copy issued has landed before the CTA exits
      for (int s = 0; s < NS; ++s)
        if (lastp[s] >= 0) wide_drain(&full[s], lastp[s]);
    }
    __syncwarp();
  } else if (warp == kRowWarps + 1) {
    // ------------------------------------------------------------ MMA issuer
    // (the whole warp runs this; one lane issues)
    const uint32_t leader = elect_leader();
    const uint32_t id_s = idesc_bf16_f32(128, 128);
    const uint32_t id_o = idesc_bf16_f32(128, 128) | kIdescTransposeB;
    const uint64_t qd = desc_kmajor_sw128(smem_u32(sm + Lay::q));
    const uint64_t kd = desc_kmajor_sw128(smem_u32(sm + Lay::ring));
    const uint64_t vd = desc_mnmajor_sw128(smem_u32(sm + Lay::ring), kHalfB);
    const uint32_t a_sfull = smem_u32(s_full), a_odone = smem_u32(o_done), a_empty = smem_u32(empty);
    // addresses in a descriptor count 16 bytes; x: S tile or buffer
    auto scores = [&](int t, int x, int ks) {   // S = Q_t K^T, K tile in ring slot ks
      const uint64_t a = qd + t * (kTileB >> 4), b = kd + ks * (kTileB >> 4);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t o = ((k >> 2) * kHalfB + (k & 3) * 32) >> 4;
        mma_bf16_by(leader, tmem + x * 128, a + o, b + o, id_s, k > 0);
      }
      mma_commit_by(leader, a_sfull + 8 * x);
    };
    auto product = [&](int t, int x, int vs, int half, uint32_t more) {   // O_t += p V
      const uint64_t b = vd + vs * (kTileB >> 4) + half * (64 * 128 >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_bf16_ts_by(leader, tmem + 256 + t * 128, tmem + x * 128 + 32 * half + 8 * k,
                       b + k * (2048 >> 4), id_o, k > 0 ? 1u : more);
    };
    auto next = [&](int& s, uint32_t& ph) {   // the ring slot after s, and its phase
      if (++s == NS) {
        s = 0;
        ph ^= 1;
      }
    };
    // K tiles are used kBuf ahead of V tiles: ring index 2 (i + kBuf) and 2 i + 1
    int ks = 0, vs = 1;
    uint32_t kph = 0, vph = 0;
    bool ok = mbar_wait(q_full, 0, abort, p.status);
    for (int i = 0; i < kBuf && i < nt; ++i) {
      ok = ok && mbar_wait(&full[ks], kph, abort, p.status);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      if (ok) {
#pragma unroll
        for (int t = 0; t < QT; ++t) scores(t, QT == 2 ? t : i, ks);
        mma_commit_by(leader, a_empty + 8 * ks);
      }
      next(ks, kph);
      next(ks, kph);
    }
    for (int i = 0; ok && i < nt; ++i) {
      const bool more = i + kBuf < nt;
      ok = mbar_wait(&full[vs], vph, abort, p.status);
      if (more) ok = ok && mbar_wait(&full[ks], kph, abort, p.status);
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        const int x = QT == 2 ? t : (i & 1);
        const uint32_t ph = (i / kBuf) & 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ok = ok && mbar_wait(&p_full[2 * x + half], ph, abort, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          product(t, x, vs, half, half || i > 0);
        }
        if (!ok) break;
        mma_commit_by(leader, a_odone + 8 * x);
        if (t == QT - 1) mma_commit_by(leader, a_empty + 8 * vs);
        if (more) {
          scores(t, x, ks);
          if (t == QT - 1) mma_commit_by(leader, a_empty + 8 * ks);
        }
      }
      next(vs, vph);
      next(vs, vph);
      next(ks, kph);
      next(ks, kph);
    }
    // teardown: all MMAs (and their commits) are complete before TMEM is freed
    mma_commit_by(leader, smem_u32(mdone));
    wide_drain(mdone, 0);
    __syncwarp();
  } else if (const int t = warp >> 3,   // query tile, and the warp's first row (lane) in it
                       l0 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);
             l0 < 16 * row_warps(t)) {
    // ------------------------------------------------------------ rows
    const int q = lane & 3;
    const uint32_t lanes = static_cast<uint32_t>(l0) << 16;
    const uint32_t to = tmem + lanes + 256 + t * 128;
    // this thread's rows, lanes l0 + lane / 4 + 8 h, and columns 8 i + 2 q + {0, 1}
    int row[2], lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      row[h] = s_row[t * kWTile + l0 + (lane >> 2) + 8 * h];
      const int qp = row[h] >= 0 ? place(row[h]) : INT_MIN;
      lo[h] = p.local > 0 ? clamp32(static_cast<int64_t>(qp) - p.local) : INT_MIN;
      hi[h] = min(qp, N - 1);
    }
    const int lo_all = p.local > 0 ? clamp32(static_cast<int64_t>(qmax) - p.local) : INT_MIN;
    const float scale = p.scale_log2;
    const uint64_t scale2 = pair(scale, scale);
    float m[2] = {-INFINITY, -INFINITY};
    uint64_t l2[2] = {0ull, 0ull};   // pairs of partial sums
    bool ok = true, odd = false;
    for (int i = 0; ok && i < nt; ++i) {
      const int t0 = sp.group(v0 + i) * kWTile;
      const int x = QT == 2 ? t : (i & 1);          // S tile or buffer
      const uint32_t ts = tmem + lanes + x * 128;
      ok = mbar_wait(&s_full[x], (i / kBuf) & 1, abort, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      // all tokens of the tile seen by all rows of the CTA, or by each row on its own
      const int t1 = t0 + kWTile - 1;
      const bool masked = !(t1 < N && t1 <= qmin && (t0 > lo_all || t1 < p.sinks));
      // s[4 k + 2 h + e]: column 64 b + 8 k + 2 q + e of row h
      uint32_t s[32];
      auto load = [&](int b) {
        tmem_ld16x256b_x8(ts + 64 * b, s);
        tmem_wait_ld_dep(s);
        if (masked) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int y = t0 + 64 * b + 8 * (c >> 2) + 2 * q + (c & 1), h = (c >> 1) & 1;
            if (!(y <= hi[h] && (y > lo[h] || y < p.sinks))) s[c] = 0xff800000u;   // -inf
          }
        }
      };
      // the maximum over both halves; the first stays in registers, the second is read
      // again (all 128 columns of two rows do not fit into the registers of 18 warps)
      float high[2];
#pragma unroll
      for (int b = 1; b >= 0; --b) {
        load(b);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t* y = &s[2 * h];   // columns 0, 1, 4, 5, ...
          auto at = [&](int n) { return __uint_as_float(y[4 * (n >> 1) + (n & 1)]); };
          float u = max3_nan(at(0), at(1), at(2)), v = max3_nan(at(3), at(4), at(5));
          u = max3_nan(u, at(6), at(7));
          v = max3_nan(v, at(8), at(9));
          u = max3_nan(u, at(10), at(11));
          v = max3_nan(v, at(12), at(13));
          u = max3_nan(u, at(14), at(15));
          high[h] = b == 1 ? max3_nan(u, v, v) : max3_nan(high[h], u, v);
        }
      }
      float top[2];
      bool grew[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float o = __shfl_xor_sync(0xffffffffu, high[h], 1);
        high[h] = max3_nan(high[h], o, o);
        o = __shfl_xor_sync(0xffffffffu, high[h], 2);
        high[h] = max3_nan(high[h], o, o);
        odd = odd || !(high[h] < INFINITY);   // NaN or +inf: the row is done again
        top[h] = fmaxf(m[h], scale * high[h]);
        grew[h] = top[h] > m[h] + kSlack;   // from -inf too
      }
      if (__any_sync(0xffffffffu, grew[0] || grew[1])) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f[h] = grew[h] ? ex2(m[h] - top[h]) : 1.f;   // 0 from -inf: O and l are 0 then
          if (grew[h]) m[h] = top[h];
          float a, b;
          unpair(l2[h], a, b);
          l2[h] = pair(a * f[h], b * f[h]);
        }
        if (i > 0) {
          // the product of step i - 1 (earlier ones are done: S of step i came after)
          const int y = QT == 2 ? t : ((i - 1) & 1);
          ok = mbar_wait(&o_done[y], ((i - 1) / kBuf) & 1, abort, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int b = 0; b < 2; ++b) {
            uint32_t o[32];
            tmem_ld16x256b_x8(to + 64 * b, o);
            tmem_wait_ld_dep(o);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              o[c] = __float_as_uint(__uint_as_float(o[c]) * f[(c >> 1) & 1]);
            tmem_st16x256b_x8(to + 64 * b, o);
          }
        }
      }
      uint64_t ref2[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ref = m[h] == -INFINITY ? 0.f : m[h];
        ref2[h] = pair(-ref, -ref);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (b == 1) load(1);
        uint32_t w[16];   // w[2 k + h]
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const int h = c & 1;
          const uint64_t y =
              fma_pair(pair(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2,
                       ref2[h]);
          float u, v;
          // one pair in four on the FMA pipe (none: 79 us for 64 sequences on 32 prefixes of
          // 16384 tokens, one in four 71, three in eight 71, half 76)
          if (c % 8 == 1 || c % 8 == 4) {
            unpair(exp2_pair(y), u, v);
          } else {
            unpair(y, u, v);
            u = ex2(u);
            v = ex2(v);
          }
          l2[h] = add_pair(l2[h], pair(u, v));
          w[c] = pack_bf16(u, v);
        }
        tmem_st16x128b_x8(ts + 32 * b, w);
        // 64 tokens: their product with V can start
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * x + b]);
      }
    }
    // the rows' parts
    float l[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float a;
      unpair(l2[h], l[h], a);
      l[h] += a;
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (m[h] == -INFINITY) l[h] = 0.f;   // saw nothing (an unseen 2^x may be off by 2^-145)
    }
    if (ok)   // the last step
      ok = mbar_wait(&o_done[QT == 2 ? t : ((nt - 1) & 1)], ((nt - 1) / kBuf) & 1, abort, p.status);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      const int64_t at0 = static_cast<int64_t>(chunk) * p.rows;
      bool fin[2] = {!odd, !odd};
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t o[32];
        tmem_ld16x256b_x8(to + 64 * b, o);
        tmem_wait_ld_dep(o);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {   // four lanes write 32 bytes of a row
          const int h = (c >> 1) & 1;
          fin[h] = fin[h] && (o[c] & 0x7f800000u) != 0x7f800000u &&
                   (o[c + 1] & 0x7f800000u) != 0x7f800000u;
          if (row[h] >= 0)
            *reinterpret_cast<uint2*>(p.part_o + (at0 + row[h]) * 128 + 64 * b + 8 * (c >> 2) + 2 * q) =
                make_uint2(o[c], o[c + 1]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned bad = __ballot_sync(0xffffffffu, !fin[h]);
        const bool fine = ((bad >> (lane & ~3)) & 15u) == 0u &&
                          (__float_as_uint(l[h]) & 0x7f800000u) != 0x7f800000u;
        if (row[h] >= 0 && q == 0) p.part_ml[at0 + row[h]] = make_float2(m[h], fine ? l[h] : kRedo);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kRowWarps + 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, 512);
  }
}

}  // namespace

cudaError_t wide_configure() {
  cudaError_t e = cudaFuncSetAttribute(wide_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       WideLayout<1>::alloc);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(wide_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             WideLayout<2>::alloc);
  return e;
}

cudaError_t launch_attend_wide(const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const AttendParams& p, int P, int max_rows, cudaStream_t st) {
  const unsigned x = static_cast<unsigned>(P) * p.maxch;
  if (max_rows <= kWTile) {
    wide_kernel<1><<<dim3(x, 1), 320, WideLayout<1>::alloc, st>>>(kmap, vmap, p);
  } else {
    // blocks of query rows along y and, beyond the 65535 that a grid holds there, z
    const unsigned blocks = (static_cast<unsigned>(max_rows) + 2 * kWTile - 1) / (2 * kWTile);
    const unsigned z = (blocks + 65534) / 65535, y = (blocks + z - 1) / z;
    wide_kernel<2><<<dim3(x, y, z), 576, WideLayout<2>::alloc, st>>>(kmap, vmap, p);
  }
  return cudaGetLastError();
}

}  // namespace rkv
