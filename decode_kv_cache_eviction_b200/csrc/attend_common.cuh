// What the attention kernels share: positions, visibility and finished rows.
#pragma once
#include <cuda_bf16.h>
#include <limits.h>

#include "ptx.cuh"
#include "rkv_internal.cuh"

namespace rkv {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ bool finite(float x) {
  return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u;
}
__device__ __forceinline__ int clamp32(int64_t x) {
  return x > INT_MAX ? INT_MAX : x < INT_MIN ? INT_MIN : static_cast<int>(x);
}

// A unit's prefix length (0 without one) and the position of its newest query.
__device__ __forceinline__ int prefix_len(const AttendParams& p, int u) {
  if (!p.unit_prefix) return 0;
  const int x = __ldg(&p.unit_prefix[u]);
  return x < 0 ? 0 : static_cast<int>(__ldg(&p.pre_off[x + 1]) - __ldg(&p.pre_off[x]));
}
// The position of a unit's first own row, as far as what its own rows' queries see depends
// on it (positions that are given, or sinks): else 0, as for a unit without a prefix, and
// two loads that wait for one another are saved.
__device__ __forceinline__ int own_first(const AttendParams& p, int u) {
  return p.pos || p.q_pos || (p.local > 0 && p.sinks > 0) ? prefix_len(p, u) : 0;
}
// Whether every query row sees its whole prefix (or, of one query per head, its unit).
__device__ __forceinline__ bool sees_whole_prefix(const AttendParams& p) {
  return p.nq == 1 && p.local == 0 && !p.q_pos;
}
__device__ __forceinline__ int64_t newest_query(const AttendParams& p, int u) {
  if (p.q_pos) return __ldg(&p.q_pos[u]);
  return prefix_len(p, u) + (__ldg(&p.tok_off[u + 1]) - __ldg(&p.tok_off[u])) - 1;
}
__device__ __forceinline__ bool sees(int pos, int qp, int lo, int sinks) {
  return pos <= qp && (pos > lo || pos < sinks);
}

// The groups of 2^kShift rows that can hold visible rows when row i sits at position
// first + i: the sinks' groups [0, gs), then [start, start + nv - gs).
struct Span {
  int gs, start, nv;
  __device__ __forceinline__ int group(int v) const { return v < gs ? v : start + (v - gs); }
};
template <int kShift>
__device__ __forceinline__ Span visible_span(int n, int first, int64_t qmin, int64_t qmax,
                                             int local, int sinks) {
  Span s = {0, 0, 0};
  const int64_t hi = min(static_cast<int64_t>(n), qmax - first + 1);   // rows past hi are later
  if (hi <= 0) return s;
  const int gh = static_cast<int>((hi + (1 << kShift) - 1) >> kShift);
  if (local > 0) {
    const int64_t ns = min(hi, max(static_cast<int64_t>(sinks) - first, static_cast<int64_t>(0)));
    const int64_t lo = max(static_cast<int64_t>(0), qmin - local + 1 - first);
    s.gs = static_cast<int>((ns + (1 << kShift) - 1) >> kShift);
    s.start = max(s.gs, static_cast<int>(min(lo, hi) >> kShift));
  }
  s.nv = s.gs + max(0, gh - s.start);
  return s;
}

// Writes four dimensions of a finished row: out = o / L (0 for a row that saw
// nothing), and from the row's first lane its log-sum-exp.  log2(L) + M is the
// sum's logarithm to base 2; a row without weight gets +inf in lse2, so that the
// weights pass gives it p = 0.
__device__ __forceinline__ void attend_store(const AttendParams& p, int64_t row, int d4, float M,
                                             float L, float4 o) {
  const bool none = L == 0.f;
  const float f = none ? 0.f : 1.f / L;
  if (none) o = make_float4(0.f, 0.f, 0.f, 0.f);
  p.out[row * 32 + d4] = make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
  if (d4 == 0) {
    const float s = M + log2f(L);
    if (p.lse) p.lse[row] = none ? -INFINITY : s * 0.6931471805599453f;
    if (p.lse2) p.lse2[row] = none ? INFINITY : s;
  }
}

// Marks the (maximum, sum) pair of a part that has to be computed again with the
// values that are not finite kept apart (a sum is never negative).
constexpr float kRedo = -1.f;

}  // namespace rkv
