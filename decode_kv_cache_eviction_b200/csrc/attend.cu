// Decode attention over a live cache: for every unit, G heads x n_q queries
// against the unit's visible rows (live, not later than the query, inside the
// sliding window or a sink),
//   z = q . k / sqrt(d),  out = sum_i softmax(z)_i v_i,  lse = log sum_i e^z_i,
// and optionally the weight of every row, acc_out_i = acc_i + sum_{g,t} p_i.
//
// One pass over K and V with a running maximum and sum.  A unit's rows are cut
// into chunks, one CTA each, and the chunks' (maximum, sum, weighted V) are
// joined in chunk order, by the unit's last CTA (up to 8 query rows) or by
// finish_kernel, so results do not depend on timing.
//
// Bound: HBM.  A row is 512 bytes, and with R = G n_q query rows costs 512 R
// flops; at R <= 16 that is below what mma.sync sustains at full bandwidth, so
// the products run on m16n8k16 steps with the 16 TOKENS as the M side: the few
// query rows are the N side (8 per step), nothing is padded to 16 or 128 rows,
// and a K or V fragment is read once for all query rows of a CTA, at most 16.  More
// query rows go through the kernel on tcgen05, or where that does not apply (live masks,
// positions) or does not pay (short units) to several CTAs per chunk that share its rows
// in L2: 64 units of 16000 rows 99 / 103 / 147 us at 8 / 16 / 32 query rows (81 at HBM's
// rate; one CTA with all 32 query rows held too many registers, 176).
//
// A warp works alone: it scans its 32-row groups (keep byte, position), appends
// the visible rows to a short list, and copies 16 listed rows of K and V per
// stage into its own shared-memory ring with cp.async.  Rows that no query
// sees are never read, and missing rows of the last stage are zero-filled.
// Only __syncwarp and cp.async.wait_group order the ring.
#include "attend_common.cuh"

namespace rkv {
namespace {

constexpr int kAtTok = 16;                     // rows per stage
constexpr int kList = 64;                      // visible-row list (ring) of a warp
constexpr int kAhead = 4;                      // groups whose masks are loaded ahead
constexpr int kRowBytes = 256;
constexpr int kOStride = 132;                  // floats per output row in shared memory

// kBoth: a unit's keys are its prefix's rows, then its own (each unit reads its prefix).
enum AtMode { kOwn = 0, kBoth = 1 };

constexpr int kStageBytes = 2 * kAtTok * kRowBytes;   // K and V

// Ring depth of a warp, and warps per SM.  Twelve warps with two stages each hide the
// steps' latencies better than eight with three (2048 units x 2176 rows: 448 -> 394 us)
// and keep 96 KB in flight per SM.
constexpr int NS = 2;
constexpr int kWarpsPerSm = 12;

struct AtWarpShared {
  int slot[kList];
  int pos[kList];
  int mslot[NS][kAtTok];   // rows of each stage
  int mpos[NS][kAtTok];
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  const int bytes = on ? 16 : 0;   // 0: the 16 bytes are zero-filled, src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&a)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&a)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// D (16 x 8, fp32) += A (16 x 16, bf16, row-major) . B (16 x 8, bf16), one warp.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A query row's state: maximum, sum and this lane's four dimensions.
struct RowSum {
  float M, L;
  float4 o;
};
__device__ __forceinline__ RowSum no_rows() {
  return {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
}

// Both states as one.
__device__ __forceinline__ RowSum add_rows(const RowSum& a, const RowSum& b) {
  if (a.M == -INFINITY && a.L == 0.f) return b;
  if (b.M == -INFINITY && b.L == 0.f) return a;
  const float M = fmaxf(a.M, b.M);
  const float f = a.M == M ? 1.f : ex2(a.M - M), h = b.M == M ? 1.f : ex2(b.M - M);
  return {M, a.L * f + b.L * h,
          make_float4(a.o.x * f + b.o.x * h, a.o.y * f + b.o.y * h, a.o.z * f + b.o.z * h,
                      a.o.w * f + b.o.w * h)};
}

// Joins the n parts of one query row to `s`, one warp: lane = four dimensions,
// parts in order.  Part c is at index at(c) of o / ml.  The parts' (maximum,
// sum) pairs of 32 parts are loaded at once, one per lane, and eight parts' values
// are in flight.
template <class At>
__device__ __forceinline__ RowSum join_row(RowSum s, int n, At at) {
  const int lane = threadIdx.x & 31;
  float M = s.M, L = s.L;
  float4 o = s.o;
  for (int c0 = 0; c0 < n; c0 += 32) {
    float2 ml = make_float2(-INFINITY, 0.f);
    const float4* src = nullptr;
    if (c0 + lane < n) at(c0 + lane, ml, src);
    const unsigned some = __ballot_sync(0xffffffffu, !(ml.x == -INFINITY && ml.y == 0.f));
    if (some == 0) continue;   // nothing visible in these parts
    float top = ml.x;
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float N = fmaxf(M, top);
    const float f = M == N ? 1.f : ex2(M - N);
    const float h = ml.x == N ? 1.f : ex2(ml.x - N);
    float l = ml.y * h;
#pragma unroll
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    M = N;
    L = L * f + l;
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
    const int e = min(32, n - c0);
    for (int k0 = 0; k0 < e; k0 += 8) {
      float4 x[8];
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = (k0 + k) & 31;
        const uint64_t a = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), c);
        w[k] = __shfl_sync(0xffffffffu, h, c);
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if ((some >> c) & 1u) x[k] = __ldcg(reinterpret_cast<const float4*>(a) + lane);
        else w[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        o.x = fmaf(x[k].x, w[k], o.x);
        o.y = fmaf(x[k].y, w[k], o.y);
        o.z = fmaf(x[k].z, w[k], o.z);
        o.w = fmaf(x[k].w, w[k], o.w);
      }
    }
  }
  return {M, L, o};
}

// A query row against its whole prefix, one warp, row by row: for rows whose
// product met a value that is not finite, which need not be one that they see.
__device__ __noinline__ RowSum prefix_row(const AttendParams& p, int64_t row, int u, int r) {
  const int lane = threadIdx.x & 31;
  const int x = p.unit_prefix ? p.unit_prefix[u] : u;
  const int64_t base = p.pre_off[x];
  const int N = static_cast<int>(p.pre_off[x + 1] - base);
  const int qp = clamp32(newest_query(p, u) - (p.nq - 1) + r % p.nq);
  const int lo = p.local > 0 ? clamp32(static_cast<int64_t>(qp) - p.local) : INT_MIN;
  auto four = [&](const uint32_t* src) {
    const uint2 w = *reinterpret_cast<const uint2*>(src + 2 * lane);
    return make_float4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y));
  };
  const float4 q = four(p.Q + row * 64);
  RowSum s = no_rows();
  for (int i = 0; i < N; ++i) {
    if (!sees(i, qp, lo, p.sinks)) continue;
    const float4 k = four(reinterpret_cast<const uint32_t*>(p.PK + (base + i) * 16));
    const float4 v = four(reinterpret_cast<const uint32_t*>(p.PV + (base + i) * 16));
    const float z = p.scale_log2 * warp_reduce_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w);
    const float M = fmaxf(s.M, z);
    const float f = s.M == M ? 1.f : ex2(s.M - M);
    const float w = ex2(z - (M == -INFINITY ? 0.f : M));
    s.M = M;
    s.L = s.L * f + w;
    s.o.x = s.o.x * f + w * v.x;
    s.o.y = s.o.y * f + w * v.y;
    s.o.z = s.o.z * f + w * v.z;
    s.o.w = s.o.w * f + w * v.w;
  }
  return s;
}

// Joins the parts that the prefix kernel left for a query row of unit u.  That kernel may have
// written them while this one was already running: no read-only loads (__ldg), which the
// compiler may move above the wait.
__device__ __forceinline__ RowSum join_prefix(const AttendParams& p, RowSum s, int64_t row, int u) {
  if (!p.pre_o || (p.unit_prefix && __ldg(&p.unit_prefix[u]) < 0)) return s;
  bool redo = false;
  for (int c = threadIdx.x & 31; c < p.pre_chunks; c += 32)
    redo |= __ldcg(&p.pre_ml[c * p.rows + row]).y == kRedo;
  if (__any_sync(0xffffffffu, redo)) {   // from the rows themselves, then the parts of s
    const RowSum x = prefix_row(p, row, u, static_cast<int>(row - static_cast<int64_t>(u) * p.R));
    return add_rows(x, s);
  }
  return join_row(s, p.pre_chunks, [&](int c, float2& ml, const float4*& src) {
    const int64_t at = c * p.rows + row;
    ml = __ldcg(&p.pre_ml[at]);
    src = reinterpret_cast<const float4*>(p.pre_o + at * 128);
  });
}

// acc_out = acc_in + sum_r 2^(z_r - lse2_r) for rows i0 .. i1 of a unit, from the
// logits that the attention pass left in p.z (one query per head, so a row is
// seen by all heads or by none).  GP: floats per row of p.z; kRowsAhead: rows of a thread
// in flight.
template <int GP, int kRowsAhead>
__device__ __forceinline__ void weights_from_logits(const AttendParams& p, int64_t base, int first,
                                                    int64_t qpos, const float* lse2, int i0,
                                                    int i1) {
  const int qp = clamp32(qpos), lo = p.local > 0 ? clamp32(qpos - p.local) : INT_MIN;
  float ls[GP];
#pragma unroll
  for (int r = 0; r < GP; ++r) ls[r] = r < p.R ? lse2[r] : INFINITY;
  for (int i = i0 + threadIdx.x; i < i1; i += kRowsAhead * blockDim.x) {
    float a[kRowsAhead], z[kRowsAhead][GP];
    bool on[kRowsAhead];
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k) {
      const int r = i + k * blockDim.x;
      const int64_t at = base + r;
      on[k] = r < i1;
      a[k] = on[k] && p.acc_in ? p.acc_in[at] : 0.f;
      int ps = first + r;
      if (on[k] && p.pos) ps = p.pos[at];
      if (on[k] && p.keep) on[k] = p.keep[at] != 0;
      on[k] = on[k] && sees(ps, qp, lo, p.sinks);
    }
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k) {
      const float* src = p.z + (base + i + k * blockDim.x) * GP;
#pragma unroll
      for (int r = 0; r < GP; ++r) z[k][r] = -INFINITY;
      if (!on[k]) continue;
      if constexpr (GP == 1) {
        z[k][0] = __ldcg(src);
      } else if constexpr (GP == 2) {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
        z[k][0] = x.x;
        z[k][1] = x.y;
      } else {
#pragma unroll
        for (int c = 0; c < GP / 4; ++c) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src) + c);
          z[k][4 * c] = x.x;
          z[k][4 * c + 1] = x.y;
          z[k][4 * c + 2] = x.z;
          z[k][4 * c + 3] = x.w;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k) {
      const int r = i + k * blockDim.x;
      if (r >= i1) break;
      float w = 0.f;
      if (on[k]) {
#pragma unroll
        for (int q = 0; q < GP; ++q)
          if (q < p.R) w += ex2(fmaf(z[k][q], p.scale_log2, -ls[q]));
      }
      p.acc_out[base + r] = a[k] + w;
    }
  }
}
template <int kRowsAhead>
__device__ __forceinline__ void weights_any(const AttendParams& p, int64_t base, int first,
                                            int64_t qpos, const float* lse2, int i0, int i1) {
  switch (p.gp) {
    case 1: weights_from_logits<1, kRowsAhead>(p, base, first, qpos, lse2, i0, i1); break;
    case 2: weights_from_logits<2, kRowsAhead>(p, base, first, qpos, lse2, i0, i1); break;
    case 4: weights_from_logits<4, kRowsAhead>(p, base, first, qpos, lse2, i0, i1); break;
    default: weights_from_logits<8, kRowsAhead / 2>(p, base, first, qpos, lse2, i0, i1); break;
  }
}

// NB: query rows / 8 of a CTA (1 or 2).  kOne: one query per head, so a row
// is seen by all query rows of its unit or by none.
template <int NB, int kMode, bool kOne, int W>
__global__ void __launch_bounds__(32 * W, kWarpsPerSm / W)
    attend_kernel(const __grid_constant__ AttendParams p) {
  constexpr int kRows = 8 * NB;   // query rows of a CTA
  extern __shared__ __align__(256) uint8_t at_smem[];
  __shared__ AtWarpShared wsh[W];
  __shared__ int s_qp[kRows];   // positions of the query rows
  __shared__ float s_ml[W][2][kRows];
  __shared__ float s_lse2[kRows];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  AtWarpShared& ws = wsh[wp];

  allow_next_launch();   // the join, or the weights
  // what this CTA works on: rows [row0, row0 + nrow) of queries against groups
  // of the sequence of N rows at `base`
  // (more than 16 query rows: the CTAs of one chunk next to each other, so that all but one
  // find its rows in L2)
  const int blocks = NB == 2 ? (p.R + kRows - 1) / kRows : 1;
  const int work = blockIdx.x / blocks, row0 = (blockIdx.x - work * blocks) * kRows;
  const int item = work / p.maxch, chunk = work - item * p.maxch;
  const int64_t base = __ldg(&p.tok_off[item]);
  const int N = static_cast<int>(__ldg(&p.tok_off[item + 1]) - base);
  int NP = 0;   // rows of the prefix, from row pbase of PK and PV
  int64_t pbase = 0;
  if (kMode == kBoth) {
    const int x = __ldg(&p.unit_prefix[item]);
    if (x >= 0) {
      pbase = __ldg(&p.pre_off[x]);
      NP = static_cast<int>(__ldg(&p.pre_off[x + 1]) - pbase);
    }
  }
  const int nrow = min(kRows, p.R - row0);
  // query row r of this CTA: its row of Q
  auto row_of = [&](int r) { return static_cast<int64_t>(item) * p.R + row0 + r; };
  // query rows as B fragments: row 8 nb + g, dimensions 16 ks + 2q + {0, 1} and + 8
  uint32_t bq[NB][8][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = 8 * nb + g;
    const bool on = r < nrow;
    const uint32_t* src = p.Q + (on ? row_of(r) : 0) * 64;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      bq[nb][ks][0] = on ? __ldg(&src[8 * ks + q]) : 0u;
      bq[nb][ks][1] = on ? __ldg(&src[8 * ks + q + 4]) : 0u;
    }
  }
  const int first = kMode == kBoth ? NP : own_first(p, item);
  const int64_t qmax =
      p.q_pos ? static_cast<int64_t>(__ldg(&p.q_pos[item])) : static_cast<int64_t>(first) + N - 1;
  const int64_t qmin = qmax - (p.nq - 1);
  if (!kOne) {
    if (tid < kRows) s_qp[tid] = tid < nrow ? clamp32(qmin + (row0 + tid) % p.nq) : INT_MIN;
    __syncthreads();
  }
  const int qmax32 = clamp32(qmax), qmin32 = clamp32(qmin);
  const int lo_any = p.local > 0 ? clamp32(qmin - p.local) : INT_MIN;
  const int lo_all = p.local > 0 ? clamp32(qmax - p.local) : INT_MIN;
  Span sp;
  if (p.pos) {   // any row may hold any position
    sp.gs = sp.start = 0;
    sp.nv = (N + 31) >> 5;
  } else {
    sp = visible_span<5>(N, first, qmin, qmax, p.local, p.sinks);
  }
  // virtual groups: the prefix's visible ones, then the own rows'
  Span sq = {0, 0, 0};
  if (kMode == kBoth) sq = visible_span<5>(NP, 0, qmin, qmax, p.local, p.sinks);
  const int nP = sq.nv;
  const int v_end = min(nP + sp.nv, (chunk + 1) * p.gpc);
  const uint8_t* keep = p.keep;
  const int32_t* pos = p.pos;

  int qp[NB][2], qlo[NB][2];    // limits of this lane's rows 8 nb + 2q + e
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      qp[nb][e] = kOne ? qmax32 : s_qp[8 * nb + 2 * q + e];
      qlo[nb][e] = p.local > 0 ? clamp32(static_cast<int64_t>(qp[nb][e]) - p.local) : INT_MIN;
    }

  constexpr int kStage = kStageBytes;
  uint8_t* ring = at_smem + wp * (NS * kStage);
  const uint32_t ring_a = smem_u32(ring);
  // ldmatrix lane addresses within a stage, K rows as A (tokens x d) and V rows
  // transposed (d x tokens): 16-byte piece c of row r lies at r 256 + 16 (c ^ (r & 7)),
  // and piece 2 k + b of a lane's row at its piece b's address ^ 32 k
  const int kt = (lane & 7) + ((lane >> 3) & 1) * 8, kc = lane >> 4;
  const int vt = (lane & 7) + ((lane >> 4) & 1) * 8, vc = (lane >> 3) & 1;
  const uint32_t kofs = kt * kRowBytes + ((kc ^ (kt & 7)) << 4);
  const uint32_t vofs = kAtTok * kRowBytes + vt * kRowBytes + ((vc ^ (vt & 7)) << 4);

  float O[8][NB][4];
  float m[NB][2], l[NB][2];
  // A result that is not finite can come from a value in a row that another
  // query of the unit may not see (0 x inf in the product), or from the split
  // of p into two parts.  The chunk is then done again with such V rows taken
  // out of the product and added one by one to the query rows that see them.
#pragma unroll 1
  for (int careful = 0; careful < 2; ++careful) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int mb = 0; mb < 8; ++mb)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[mb][nb][e] = 0.f;
      m[nb][0] = m[nb][1] = -INFINITY;
      l[nb][0] = l[nb][1] = 0.f;
    }
    int v = chunk * p.gpc + wp;   // next group of this warp
    int head = 0, cnt = 0;        // list: first entry, entries
    // a group's live bytes and positions, loaded kAhead groups ahead
    auto fetch = [&](int vv, int& alive, int& ps) {
      if (kMode == kBoth && vv < nP) {
        ps = 32 * sq.group(vv) + lane;
        alive = vv < v_end && ps < NP ? 1 : 0;
        return;
      }
      const int slot = 32 * sp.group(vv - nP) + lane;
      const bool in = vv < v_end && slot < N;
      alive = in ? 1 : 0;
      ps = first + slot;
      if (keep && in) alive = __ldg(&keep[base + slot]);
      if (pos && in) ps = __ldg(&pos[base + slot]);
    };
    int live[kAhead], at[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(v + k * W, live[k], at[k]);
    // rows of group v (virtual order: sinks' groups, then the window's)
    auto scan = [&]() {
      // a prefix's row i is listed as ~i
      const int slot = kMode == kBoth && v < nP ? ~(32 * sq.group(v) + lane)
                                                : 32 * sp.group(v - nP) + lane;
      const int ps = at[0];
      bool on = live[0] != 0;
#pragma unroll
      for (int k = 0; k < kAhead - 1; ++k) {
        live[k] = live[k + 1];
        at[k] = at[k + 1];
      }
      fetch(v + kAhead * W, live[kAhead - 1], at[kAhead - 1]);
      on = on && sees(ps, qmax32, lo_any, p.sinks);
      const uint32_t mask = __ballot_sync(0xffffffffu, on);
      if (on) {
        const int to = (head + cnt + __popc(mask & ((1u << lane) - 1u))) & (kList - 1);
        ws.slot[to] = slot;
        ws.pos[to] = ps;
      }
      cnt += __popc(mask);
      v += W;
    };
    int issued = 0, done = 0, last = kAtTok;   // stages; rows of the last stage
    uint32_t some = 0;   // bit s: a query row does not see a row of stage s
    int si = 0, sd = 0;  // their slots in the ring
    auto produce = [&]() {
      while (cnt < kAtTok && v < v_end) scan();
      __syncwarp();
      if (cnt > 0) {
        const int n = min(cnt, kAtTok);
        const int s = si;
        // lane: 64 bytes of rows lane / 4 and lane / 4 + 8, a quarter at a time
        const uint32_t dst = ring_a + s * kStage + g * kRowBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = g + 8 * h;
          const bool on = r < n;
          const int slot = on ? ws.slot[(head + r) & (kList - 1)] : 0;
          const bool shared = kMode == kBoth && slot < 0;
          const int64_t row = shared ? pbase + ~slot : base + slot;
          const uint4* ks = (shared ? p.PK : p.K) + row * 16 + q;
          const uint4* vs = (shared ? p.PV : p.V) + row * 16 + q;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t d = dst + 8 * h * kRowBytes + (((4 * c + q) ^ g) << 4);
            cp16(d, ks + 4 * c, on);
            cp16(d + kAtTok * kRowBytes, vs + 4 * c, on);
          }
        }
        bool part = false;
        if (lane < kAtTok) {
          const int ps = ws.pos[(head + lane) & (kList - 1)];
          ws.mslot[s][lane] = ws.slot[(head + lane) & (kList - 1)];
          if (!kOne) {
            ws.mpos[s][lane] = ps;
            part = lane >= n || !sees(ps, qmin32, lo_all, p.sinks);
          }
        }
        if (!kOne) {
          const bool any = __any_sync(0xffffffffu, part);
          some = (some & ~(1u << s)) | ((any ? 1u : 0u) << s);
        }
        head = (head + n) & (kList - 1);
        cnt -= n;
        ++issued;
        last = n;
        if (++si == NS) si = 0;
      }
      cp_commit();
      __syncwarp();
    };
#pragma unroll 1
    for (int s = 0; s < NS - 1; ++s) produce();
#pragma unroll 1
    for (;;) {
      produce();
      cp_wait<NS - 1>();
      __syncwarp();
      if (done == issued) break;
      const int s = sd;
      if (++sd == NS) sd = 0;
      ++done;
      const int n = done == issued ? last : kAtTok;
      const uint32_t st_a = ring_a + s * kStage;
      const bool in0 = g < n, in1 = g + 8 < n;      // this lane's tokens g, g + 8
      // which query rows see them
      const bool masked = kOne ? n < kAtTok : ((some >> s) & 1u) != 0;
      auto seen = [&](int nb, int e, int h) {   // query row 8 nb + 2q + e, token g + 8 h
        const bool in = h ? in1 : in0;
        return kOne ? in : in && sees(ws.mpos[s][g + 8 * h], qp[nb][e], qlo[nb][e], p.sinks);
      };
      // logits of 16 tokens x 8 NB query rows
      float c[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[nb][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        uint32_t a[4];
        ldsm4(a, (st_a + kofs) ^ (ks << 5));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma16816(c[nb], a, bq[nb][ks][0], bq[nb][ks][1]);
      }
      if constexpr (kOne) {
        if (p.z && 2 * q < p.gp) {   // logits for the weights, before masks and scaling
          const int r0 = ws.mslot[s][g], r1 = ws.mslot[s][g + 8];   // own rows only
          const bool w0 = in0 && r0 >= 0, w1 = in1 && r1 >= 0;
          float* z0 = p.z + (base + r0) * p.gp + 2 * q;
          float* z1 = p.z + (base + r1) * p.gp + 2 * q;
          if (p.gp == 1) {
            if (w0) *z0 = c[0][0];
            if (w1) *z1 = c[0][2];
          } else {
            if (w0) __stcg(reinterpret_cast<float2*>(z0), make_float2(c[0][0], c[0][1]));
            if (w1) __stcg(reinterpret_cast<float2*>(z1), make_float2(c[0][2], c[0][3]));
          }
        }
      }
      if (masked) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!seen(nb, e, 0)) c[nb][e] = -INFINITY;
            if (!seen(nb, e, 1)) c[nb][2 + e] = -INFINITY;
          }
      }
      uint32_t bh[NB][2], bl[NB][2];
      float mref[NB][2];
      bool grew = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(c[nb][e], c[nb][2 + e]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x *= p.scale_log2;
          grew |= x > m[nb][e];
          mref[nb][e] = fmaxf(x, m[nb][e]);
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // m = -inf (nothing seen yet): the factor is 0, and so are O and l
            const float f = mref[nb][e] == m[nb][e] ? 1.f : ex2(m[nb][e] - mref[nb][e]);
            m[nb][e] = mref[nb][e];
            l[nb][e] *= f;
#pragma unroll
            for (int mb = 0; mb < 8; ++mb) {
              O[mb][nb][e] *= f;
              O[mb][nb][2 + e] *= f;
            }
          }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = m[nb][e] == -INFINITY ? 0.f : m[nb][e];
          c[nb][e] = ex2(fmaf(c[nb][e], p.scale_log2, -ref));
          c[nb][2 + e] = ex2(fmaf(c[nb][2 + e], p.scale_log2, -ref));
          l[nb][e] += c[nb][e] + c[nb][2 + e];
        }
        // p as the sum of two bf16 (about 16 bits) while the steps are not the bound; with
        // more than 8 query rows as one (2^-8 of each weight at most, of random sign): the
        // second part would be a third of the mma.sync steps, which then are
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = c[nb][2 * h], y = c[nb][2 * h + 1];
          const uint32_t hi = pack_bf16(x, y);
          bh[nb][h] = transpose8x8(hi);
          if (NB == 1) bl[nb][h] = transpose8x8(pack_bf16(x - bf_lo(hi), y - bf_hi(hi)));
        }
      }
      if (careful) {
        // tokens whose V row holds a value that is not finite
        uint32_t bad = 0;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const int r = 2 * i + (lane >> 4);
          const uint4 x = *reinterpret_cast<const uint4*>(
              ring + s * kStage + kAtTok * kRowBytes + r * kRowBytes + (lane & 15) * 16);
          auto two = [](uint32_t w) {
            return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
          };
          const uint32_t b =
              __ballot_sync(0xffffffffu, two(x.x) || two(x.y) || two(x.z) || two(x.w));
          bad |= ((b & 0xffffu) ? 1u : 0u) << (2 * i) | ((b >> 16) ? 1u : 0u) << (2 * i + 1);
        }
#pragma unroll 1
        for (; bad; bad &= bad - 1u) {
          const int t = __ffs(bad) - 1;
          uint8_t* vr = ring + s * kStage + kAtTok * kRowBytes + t * kRowBytes;
          float pv[NB][2];
          bool on[NB][2];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a = __shfl_sync(0xffffffffu, c[nb][e], (t & 7) * 4 + q);
              const float b = __shfl_sync(0xffffffffu, c[nb][2 + e], (t & 7) * 4 + q);
              pv[nb][e] = t < 8 ? a : b;
              on[nb][e] = kOne || sees(ws.mpos[s][t], qp[nb][e], qlo[nb][e], p.sinks);
            }
#pragma unroll
          for (int mb = 0; mb < 8; ++mb)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int ch = (2 * mb + h) ^ (t & 7);
              const float x = __bfloat162float(
                  *reinterpret_cast<const __nv_bfloat16*>(vr + ch * 16 + g * 2));
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (on[nb][e]) O[mb][nb][2 * h + e] += pv[nb][e] * x;
            }
          __syncwarp();
          if (lane < 16) *reinterpret_cast<uint4*>(vr + lane * 16) = make_uint4(0, 0, 0, 0);
          __syncwarp();
        }
      }
      // O^T (128 d x 8 NB) += V^T (128 d x 16) . p^T (16 x 8 NB)
#pragma unroll
      for (int mb = 0; mb < 8; ++mb) {
        uint32_t a[4];
        ldsm4_t(a, (st_a + vofs) ^ (mb << 5));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          mma16816(O[mb][nb], a, bh[nb][0], bh[nb][1]);
          if (NB == 1) mma16816(O[mb][nb], a, bl[nb][0], bl[nb][1]);
        }
      }
      __syncwarp();   // this stage's slot is written next
    }
    cp_wait<0>();
    if (careful) break;
    bool ok = true;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mb = 0; mb < 8; ++mb)
#pragma unroll
        for (int e = 0; e < 4; ++e) ok = ok && finite(O[mb][nb][e]);
    if (!__any_sync(0xffffffffu, !ok)) break;
    __syncwarp();
  }
  // the warps' parts to shared memory (the rings are done with), then joined
  __syncthreads();
  float* sO = reinterpret_cast<float*>(at_smem);   // [warp][8 NB][kOStride]
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[nb][e];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      const int r = 8 * nb + 2 * q + e;
      if (g == 0) {
        s_ml[wp][0][r] = m[nb][e];
        s_ml[wp][1][r] = x;
      }
      float* o = sO + (wp * 8 * NB + r) * kOStride;
#pragma unroll
      for (int mb = 0; mb < 8; ++mb) {
        o[16 * mb + g] = O[mb][nb][e];
        o[16 * mb + g + 8] = O[mb][nb][2 + e];
      }
    }
  }
  __syncthreads();
  // The prefix's parts: this launch may have started while they were computed.  A CTA that
  // leaves its part for a join does not hold its place until then, but one of them waits,
  // so that this launch ends after the one before.
  if (kMode == kOwn && p.pre_o && (!p.part_o || blockIdx.x == 0)) wait_for_previous_launch();
  // one warp per query row, lane = four dimensions
  for (int r = wp; r < nrow; r += W) {
    RowSum x = no_rows();
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float4 o = *reinterpret_cast<const float4*>(sO + (w * 8 * NB + r) * kOStride + 4 * lane);
      x = add_rows(x, {s_ml[w][0][r], s_ml[w][1][r], o});
    }
    const int64_t row = row_of(r);
    if (p.part_o) {
      const int64_t at = (static_cast<int64_t>(item) * p.maxch + chunk) * p.R + row0 + r;
      __stcg(reinterpret_cast<float4*>(p.part_o + at * 128 + 4 * lane), x.o);
      if (lane == 0) __stcg(&p.part_ml[at], make_float2(x.M, x.L));
    } else {
      x = join_prefix(p, x, row, item);
      attend_store(p, row, lane, x.M, x.L, x.o);
      if (lane == 0) s_lse2[r] = x.L == 0.f ? INFINITY : x.M + log2f(x.L);
    }
  }
  if (p.count) {
    // the CTA that finishes a unit's rows last joins its parts
    __threadfence();
    __syncthreads();
    int* cnt = p.count + item;
    if (tid == 0) s_last = atomicAdd(cnt, 1) == p.maxch - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    if (tid == 0) *cnt = 0;   // ready for the next call
    if (kMode == kOwn && p.pre_o) wait_for_previous_launch();
    const int64_t at0 = static_cast<int64_t>(item) * p.maxch * p.R + row0;
    for (int r = wp; r < nrow; r += W) {
      RowSum x = join_row(no_rows(), p.maxch, [&](int c, float2& ml, const float4*& src) {
        const int64_t at = at0 + static_cast<int64_t>(c) * p.R + r;
        ml = __ldcg(&p.part_ml[at]);
        src = reinterpret_cast<const float4*>(p.part_o + at * 128);
      });
      x = join_prefix(p, x, row_of(r), item);
      attend_store(p, row_of(r), lane, x.M, x.L, x.o);
    }
  } else if (kOne && p.z && !p.part_o) {
    __syncthreads();   // all logits of the unit are written
    weights_any<8>(p, base, first, qmax, s_lse2, 0, N);
  }
}

// The weights pass from stored logits: chunks of gpc groups of one unit per CTA.
// Latency-bound (live byte and position, then logits, then the store): 1.3 million rows of
// 4 heads 13 us, 18 with live bytes and positions, 6 at HBM's rate; the attention kernel
// takes 8 us more for leaving the logits.  Tried and slower: vectors of four rows per
// thread (fewer rows in flight), the logits loaded beside the live bytes instead of after
// them (more bytes), a unit's weights by its last CTA instead of a launch (46 us).
__global__ void __launch_bounds__(256) weights_kernel(const __grid_constant__ AttendParams p) {
  const int item = blockIdx.x / p.maxch, chunk = blockIdx.x - item * p.maxch;
  const int64_t base = __ldg(&p.tok_off[item]);
  const int N = static_cast<int>(__ldg(&p.tok_off[item + 1]) - base);
  const int first = own_first(p, item);
  const int64_t qpos = p.q_pos ? static_cast<int64_t>(__ldg(&p.q_pos[item]))
                               : static_cast<int64_t>(first) + N - 1;
  const int64_t i0 = static_cast<int64_t>(chunk) * p.gpc * 32;
  wait_for_previous_launch();
  if (i0 >= N) return;
  weights_any<4>(p, base, first, qpos,
              p.lse2 + static_cast<int64_t>(item) * p.R, static_cast<int>(i0),
              static_cast<int>(min(static_cast<int64_t>(N), i0 + static_cast<int64_t>(p.gpc) * 32)));
}

// Joins the parts of every query row, one warp each: those that the wide kernel left in
// p.pre_o (a prefix's, or own rows that went through it as a prefix of their own), and
// those of the unit's chunks in p.part_o.
__global__ void __launch_bounds__(128) finish_kernel(const __grid_constant__ AttendParams p) {
  allow_next_launch();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  wait_for_previous_launch();
  if (row >= p.rows) return;
  const int u = static_cast<int>(row / p.R), r = static_cast<int>(row - static_cast<int64_t>(u) * p.R);
  RowSum x = no_rows();
  if (p.part_o)
    x = join_row(x, p.maxch, [&](int c, float2& ml, const float4*& src) {
      const int64_t at = (static_cast<int64_t>(u) * p.maxch + c) * p.R + r;
      ml = __ldcg(&p.part_ml[at]);
      src = reinterpret_cast<const float4*>(p.part_o + at * 128);
    });
  x = join_prefix(p, x, row, u);
  attend_store(p, row, threadIdx.x & 31, x.M, x.L, x.o);
}

template <int NB, int kMode, int W>
__host__ __device__ constexpr int at_smem_bytes() {
  const int ring = W * NS * kStageBytes;
  const int fin = W * 8 * NB * kOStride * 4;
  return ring > fin ? ring : fin;
}

template <int NB, int kMode, bool kOne, int W>
cudaError_t configure_one() {
  return cudaFuncSetAttribute(attend_kernel<NB, kMode, kOne, W>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              at_smem_bytes<NB, kMode, W>());
}
template <int kMode, int W>
cudaError_t configure_mode() {
  cudaError_t e = configure_one<1, kMode, false, W>();
  if (e == cudaSuccess) e = configure_one<1, kMode, true, W>();
  if (e == cudaSuccess) e = configure_one<2, kMode, false, W>();
  return e;
}

// early: the launch may start when the one before it on the stream lets it
// (allow_next_launch); it waits for that one's results where it reads them.
cudaError_t launch_early(void (*kernel)(const AttendParams), const AttendParams& p, dim3 grid,
                         int threads, int smem, bool early, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = early ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <int NB, int kMode, bool kOne, int W>
cudaError_t launch_one(const AttendParams& p, dim3 grid, bool early, cudaStream_t st) {
  return launch_early(attend_kernel<NB, kMode, kOne, W>, p, grid, 32 * W, at_smem_bytes<NB, kMode, W>(),
                      early, st);
}
template <int kMode, int W>
cudaError_t launch_mode(const AttendParams& p, int rows, dim3 grid, bool early, cudaStream_t st) {
  if (rows <= 8)
    return p.nq == 1 ? launch_one<1, kMode, true, W>(p, grid, early, st)
                     : launch_one<1, kMode, false, W>(p, grid, early, st);
  return launch_one<2, kMode, false, W>(p, grid, early, st);
}

}  // namespace

cudaError_t attend_configure() {
  cudaError_t e = configure_mode<kOwn, 4>();
  if (e == cudaSuccess) e = configure_mode<kOwn, 2>();
  if (e == cudaSuccess) e = configure_mode<kBoth, 4>();
  if (e == cudaSuccess) e = configure_mode<kBoth, 2>();
  return e;
}

int attend_warps_per_sm() { return kWarpsPerSm; }

cudaError_t launch_attend(const AttendParams& p, int U, int warps, bool both, bool early,
                          cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(U) * p.maxch * ((p.R + 15) / 16));
  if (both)
    return warps == 2 ? launch_mode<kBoth, 2>(p, p.R, grid, early, st)
                      : launch_mode<kBoth, 4>(p, p.R, grid, early, st);
  return warps == 2 ? launch_mode<kOwn, 2>(p, p.R, grid, early, st)
                    : launch_mode<kOwn, 4>(p, p.R, grid, early, st);
}

cudaError_t launch_attend_finish(const AttendParams& p, cudaStream_t st) {
  return launch_early(finish_kernel, p, dim3(static_cast<unsigned>((p.rows + 3) / 4)), 128, 0, true,
                      st);
}

cudaError_t launch_attend_weights(const AttendParams& p, int U, cudaStream_t st) {
  return launch_early(weights_kernel, p, dim3(static_cast<unsigned>(U) * p.maxch), 256, 0, true, st);
}

}  // namespace rkv
