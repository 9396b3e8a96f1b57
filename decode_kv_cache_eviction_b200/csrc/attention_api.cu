// C ABI of the operators that read and keep a live cache: attention over it
// (with a shared prefix or without), eviction by accumulated weight, and new
// tokens into freed slots with their positions.
#include <algorithm>
#include <cmath>

#include "../../include/rkv.h"
#include "engine.cuh"
#include "ptx.cuh"
#include "rkv_internal.cuh"

using namespace rkv;

namespace {

// The engine's device for the length of a call, whichever is current.
struct DeviceGuard {
  int was = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    int cur = 0;
    ok = cudaGetDevice(&cur) == cudaSuccess;
    if (ok && cur != dev) {
      ok = cudaSetDevice(dev) == cudaSuccess;
      if (ok) was = cur;
    }
  }
  ~DeviceGuard() {
    if (was >= 0) cudaSetDevice(was);
  }
};

struct Lengths {
  int64_t T = 0;
  int nmax = 0;
};

// Host-side checks of a batch whose units may have any length from 0 on.
int check_rows(const rkv_engine* e, const rkv_batch* b, Lengths* L) {
  if (!b || b->num_units < 0) return RKV_ERR_INVALID_ARG;
  if (b->num_units > e->cfg.max_units) return RKV_ERR_CAPACITY;
  if (!b->tok_off_host || !b->tok_off || !aligned(b->tok_off, 8)) return RKV_ERR_INVALID_ARG;
  const int64_t* off = b->tok_off_host;
  if (off[0] != 0) return RKV_ERR_INVALID_ARG;
  int64_t nm = 0;
  for (int u = 0; u < b->num_units; ++u) {
    const int64_t n = off[u + 1] - off[u];
    if (n < 0) return RKV_ERR_INVALID_ARG;
    nm = std::max(nm, n);
  }
  if (nm > e->max_n) return RKV_ERR_UNSUPPORTED;
  L->T = off[b->num_units];
  if (L->T > e->cfg.max_tokens) return RKV_ERR_CAPACITY;
  L->nmax = static_cast<int>(nm);
  return RKV_OK;
}

constexpr int64_t kPartFloats = 130;   // a part: 128 values, maximum and sum

// Query rows whose parts the scratch holds: two waves of CTAs (three per SM) of at most
// 32 rows; for shared calls also every query row's own and prefix part, and a wave of
// CTAs of at most 256 rows of a split prefix.
int64_t part_rows(const rkv_engine* e, bool shared) {
  const int64_t one = static_cast<int64_t>(e->cfg.group) * e->cfg.window;
  const int64_t all = one * e->cfg.max_units;
  const int64_t split = 6ll * e->nsm * std::min<int64_t>(one, 32);
  return split + (shared ? 2 * all + static_cast<int64_t>(e->nsm) * std::min<int64_t>(all, 256) : 0);
}

// Scratch of the attention calls, allocated once: `rows` parts, the rows' log2
// sums and the counters (zero between calls).  Not while a stream is captured.
int attend_scratch(rkv_engine* e, float** buf, int64_t rows, bool logits, cudaStream_t st) {
  if (*buf && (e->rf_z || !logits)) return RKV_OK;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cs) != cudaSuccess) return cuda_fail(cudaErrorUnknown);
  if (cs != cudaStreamCaptureStatusNone) return RKV_ERR_INVALID_ARG;
  if (logits) {
    const int rc = rkv_logit_scratch(e);
    if (rc != RKV_OK) return rc;
  }
  if (*buf) return RKV_OK;
  const size_t sums = static_cast<size_t>(rows) * kPartFloats +
                      static_cast<size_t>(e->cfg.max_units) * e->cfg.group * e->cfg.window;
  const size_t counts = static_cast<size_t>(e->cfg.max_units);   // arrived chunks of split units
  if (rkv_engine_alloc(e, reinterpret_cast<void**>(buf), (sums + counts) * sizeof(float)) !=
      cudaSuccess) {
    cudaGetLastError();
    *buf = nullptr;
    return RKV_ERR_OOM;
  }
  if (cudaMemsetAsync(*buf + sums, 0, counts * sizeof(int), st) != cudaSuccess) {
    cudaFree(*buf);
    *buf = nullptr;
    return cuda_fail(cudaErrorUnknown);
  }
  return RKV_OK;
}

// Chunks per item, for items of groups of rows (nmax the longest, sum over all
// items): the cheapest count by waves of `slots` resident CTAs, a CTA costing its
// groups and about `extra` more, at most `cap` and at least `least_groups` each.
int pick_chunks(int64_t items, int64_t sum, int64_t nmax, int64_t slots, int64_t cap,
                int64_t least_groups, double extra) {
  const int64_t avg = std::max<int64_t>(1, (sum + items - 1) / std::max<int64_t>(items, 1));
  const int64_t most =
      std::min<int64_t>(std::max<int64_t>(1, cap), std::max<int64_t>(1, nmax / least_groups));
  int64_t best = 1;
  double least = 1e300;
  for (int64_t c = 1; c <= std::min<int64_t>(most, 4096); c += c < 16 ? 1 : c / 8) {
    const int64_t gpc = (nmax + c - 1) / c;
    const int64_t ctas = items * ((avg + gpc - 1) / gpc);
    const double cost = static_cast<double>((ctas + slots - 1) / slots) * (gpc + extra) +
                        (c > 1 ? extra : 0.0);
    if (cost < least) {
      least = cost;
      best = c;
    }
  }
  return static_cast<int>(best);
}

// Group counts of up to 32 units, evenly spaced over the batch, and what they say of all.
struct Sample {
  int n = 0;
  float groups[32];
  // chunks of gpc groups that a unit takes on average (a product with the reciprocal: whole
  // divisions took the host longer than the launch)
  double per(int64_t gpc) const {
    const float inv = 1.f / static_cast<float>(gpc), up = static_cast<float>(gpc) - 0.5f;
    int s = 0;
    for (int i = 0; i < n; ++i) s += std::max(1, static_cast<int>((groups[i] + up) * inv));
    return static_cast<double>(s) / std::max(n, 1);
  }
};

// Warps per CTA and chunks per unit of the attention over own rows, by waves of CTAs on
// the `resident` warps that the GPU holds at once.  In us: a CTA costs 5 for its start
// and end, and per 16-row stage of a warp `step` when few run beside it and the stage's
// share of HBM (8 KB at `rate` bytes per us) when many do; joining c parts costs 3 and
// 0.1 c for each row that a warp joins, and the weights 5 in a launch of their own or 0.3
// per 32 rows and warp at the unit's end.  Measured: 128 units of 32768 rows 401 / 324 /
// 402 / 334 us in 1 / 2 / 4 / 6 chunks (modelled 389 / 340 / 395 / 344), 509 windows of
// 1028 rows 50 us with two warps and 59 with four (50 / 62).
double pick_shape(const Sample& sample, int64_t items, int64_t sum, int64_t nmax,
                  int64_t resident, int R, double rate, int64_t cap, bool weights, int* warps,
                  int* chunks) {
  const double step = R <= 8 ? 0.75 : R <= 16 ? 1.0 : 1.3;
  const double avg = std::max(1.0, static_cast<double>(sum) / static_cast<double>(items));
  const double share = resident * 8192.0 / rate;
  auto stage = [&](double part) { return std::max(step, share * part); };
  double least = 1e300;
  for (int w = 4; w >= 2; w -= 2)
    for (int64_t c = 1; c <= std::min<int64_t>(std::max<int64_t>(1, cap),
                                               std::max<int64_t>(1, nmax / w));
         c += c < 4 ? 1 : c / 4) {
      const int64_t gpc = (nmax + c - 1) / c;
      const double per = c == 1 ? 1.0 : sample.per(gpc);
      const double waves = static_cast<double>(items) * per * w / resident;
      const double full = std::floor(waves), rest = waves - full;
      const double mean = 2.0 * avg / per / w + 0.5;
      const double most = 2.0 * static_cast<double>((gpc + w - 1) / w);
      const int turns = R <= 8 ? (R + w - 1) / w : 1;   // rows that a warp joins
      double cost = c > 1 ? 3.0 + 0.1 * c * turns + (weights ? 5.0 : 0.0) : 0.0;
      const double fixed = 5.0 + (weights && c == 1 ? 0.3 * avg / w : 0.0);
      if (full > 0) cost += full * (mean * stage(1.0) + fixed);
      cost += full == 0 || rest > 0.02 ? most * stage(rest) + fixed : (most - mean) * step;
      if (w == 2) cost *= 1.05;   // measured beyond the model
      if (cost < least) {
        least = cost;
        *warps = w;
        *chunks = static_cast<int>(c);
      }
    }
  return least;
}

// The same for the wide kernel over units or prefixes (tiles of 128 tokens, one CTA per
// SM): 7 us per CTA, per tile `step` or its share of HBM, and for the join of c parts
// `last` + `join` c.
double pick_wide(const Sample& sample, int64_t items, int64_t sum, int64_t nmax, int64_t slots,
                 double step, double last, double join, int64_t cap, int* chunks) {
  const double avg = std::max(1.0, static_cast<double>(sum) / static_cast<double>(items));
  const double share = slots * 65536.0 / 6.5e6;
  auto tile = [&](double part) { return std::max(step, share * part); };
  double least = 1e300;
  for (int64_t c = 1; c <= std::min(std::max<int64_t>(1, cap), nmax); c += c < 4 ? 1 : c / 4) {
    const int64_t gpc = (nmax + c - 1) / c;
    const double per = c == 1 ? 1.0 : sample.per(gpc);
    const double waves = static_cast<double>(items) * per / slots;
    const double full = std::floor(waves), rest = waves - full;
    double cost = last + full * (avg / per * tile(1.0) + 7.0);
    if (full == 0 || rest > 0.02) cost += gpc * tile(rest) + 7.0;
    cost *= full == 0 ? 0.87 : 1.05;   // against the other model, as measured
    cost += join * c;
    if (cost < least) {
      least = cost;
      *chunks = static_cast<int>(c);
    }
  }
  return least;
}

int check_prefix(const rkv_engine* e, const rkv_batch* b, const rkv_prefix* x, int64_t* sum,
                 int64_t* longest, int* most) {
  if (x->num_prefixes < 0) return RKV_ERR_INVALID_ARG;
  if (!x->off || !x->off_host || !x->unit_prefix || !x->unit_prefix_host || !x->mem_off ||
      !x->mem_off_host || !x->mem || !x->mem_host)
    return RKV_ERR_INVALID_ARG;
  if (!aligned(x->off, 8) || !aligned(x->unit_prefix, 4) || !aligned(x->mem_off, 4) ||
      !aligned(x->mem, 4))
    return RKV_ERR_INVALID_ARG;
  const int P = x->num_prefixes, U = b->num_units;
  if (x->num_units != U || x->off_host[0] != 0 || x->mem_off_host[0] != 0)
    return RKV_ERR_INVALID_ARG;
  *longest = 0;
  *most = 0;
  for (int k = 0; k < P; ++k) {
    const int64_t n = x->off_host[k + 1] - x->off_host[k];
    const int m0 = x->mem_off_host[k], m1 = x->mem_off_host[k + 1];
    if (n < 0 || m1 < m0) return RKV_ERR_INVALID_ARG;
    if (n >= (static_cast<int64_t>(1) << 30)) return RKV_ERR_UNSUPPORTED;
    *longest = std::max(*longest, n);
    *most = std::max(*most, m1 - m0);
  }
  *sum = x->off_host[P];
  if (*sum >= (static_cast<int64_t>(1) << 31)) return RKV_ERR_UNSUPPORTED;   // tile coordinates
  int with = 0;
  for (int u = 0; u < U; ++u) {
    const int k = x->unit_prefix_host[u];
    if (k < -1 || k >= P) return RKV_ERR_INVALID_ARG;
    with += k >= 0;
  }
  // every unit with a prefix is listed once, under its prefix, in ascending order
  if (x->mem_off_host[P] != with) return RKV_ERR_INVALID_ARG;
  for (int k = 0; k < P; ++k)
    for (int i = x->mem_off_host[k]; i < x->mem_off_host[k + 1]; ++i) {
      const int u = x->mem_host[i];
      if (u < 0 || u >= U || x->unit_prefix_host[u] != k ||
          (i > x->mem_off_host[k] && x->mem_host[i - 1] >= u))
        return RKV_ERR_INVALID_ARG;
    }
  if (*sum > 0 && (!x->K || !x->V || !aligned(x->K, 16) || !aligned(x->V, 16)))
    return RKV_ERR_INVALID_ARG;
  (void)e;
  return RKV_OK;
}

// Groups of `per` rows that a window of `local` tokens and the sinks can touch, at most.
int64_t reach(int local, int sinks, int nq, int64_t per) {
  if (local <= 0) return INT64_MAX;
  return (static_cast<int64_t>(sinks) + per - 1) / per +
         (static_cast<int64_t>(local) + nq) / per + 2;
}

int attend(rkv_engine* e, const rkv_batch* b, const rkv_prefix* x, const rkv_attention* a,
           rkv_stream_t stream) {
  if (!e || !a) return RKV_ERR_INVALID_ARG;
  Lengths L;
  int rc = check_rows(e, b, &L);
  if (rc != RKV_OK) return rc;
  const int U = b->num_units;
  if (a->num_queries < 1 || a->local < 0 || a->sinks < 0) return RKV_ERR_INVALID_ARG;
  if (a->num_queries > e->cfg.window) return RKV_ERR_UNSUPPORTED;
  if (U == 0) return RKV_OK;
  if (!a->Q || !a->out || (L.T > 0 && (!b->K || !b->V))) return RKV_ERR_INVALID_ARG;
  if (a->pos && !a->q_pos) return RKV_ERR_INVALID_ARG;
  if (a->acc_in && !a->acc_out) return RKV_ERR_INVALID_ARG;
  // Q is read until the last row is written: no byte of it may be out's
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(a->Q), o0 = reinterpret_cast<uintptr_t>(a->out);
  const uint64_t span = static_cast<uint64_t>(U) * e->cfg.group * a->num_queries * kHeadDim * 2;
  if (q0 < o0 + span && o0 < q0 + span) return RKV_ERR_INVALID_ARG;
  if (!aligned(b->K, 16) || !aligned(b->V, 16) || !aligned(a->Q, 16) || !aligned(a->out, 16) ||
      !aligned(a->lse, 4) || !aligned(a->pos, 4) || !aligned(a->q_pos, 4) ||
      !aligned(a->acc_in, 4) || !aligned(a->acc_out, 4))
    return RKV_ERR_INVALID_ARG;
  int64_t psum = 0, plong = 0;
  int members = 0;
  if (x) {
    rc = check_prefix(e, b, x, &psum, &plong, &members);
    if (rc != RKV_OK) return rc;
    if (members == 0 || psum == 0) x = nullptr;   // no unit has a prefix, or no rows in it
  }
  DeviceGuard dev(e->device);
  if (!dev.ok) return cuda_fail(cudaErrorUnknown);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t cap = part_rows(e, x != nullptr);
  float** buf = x ? &e->at_shared : &e->at_part;
  const int R = e->cfg.group * a->num_queries;
  // weights from stored logits: a row's logits are then all or none visible
  const bool logits = a->acc_out && a->num_queries == 1 && R <= 8;
  rc = attend_scratch(e, buf, cap, logits, st);
  if (rc != RKV_OK) return rc;
  const int64_t rows = static_cast<int64_t>(U) * R;
  const int rg = (R + 15) / 16;   // CTAs that share a chunk
  AttendParams p = {};
  p.tok_off = b->tok_off;
  p.K = static_cast<const uint4*>(b->K);
  p.V = static_cast<const uint4*>(b->V);
  p.Q = static_cast<const uint32_t*>(a->Q);
  p.keep = a->keep;
  p.pos = a->pos;
  p.q_pos = a->q_pos;
  p.R = R;
  p.nq = a->num_queries;
  p.local = a->local;
  p.sinks = a->sinks;
  p.scale_log2 = kLog2e / sqrtf(static_cast<float>(kHeadDim));
  p.out = static_cast<uint2*>(a->out);
  p.lse = a->lse;
  p.rows = rows;
  float* part_o = *buf;
  float2* part_ml = reinterpret_cast<float2*>(part_o + cap * 128);
  float* lse2 = reinterpret_cast<float*>(part_ml + cap);
  int* count = reinterpret_cast<int*>(
      lse2 + static_cast<int64_t>(e->cfg.max_units) * e->cfg.group * e->cfg.window);
  p.lse2 = a->acc_out ? lse2 : nullptr;
  p.acc_in = a->acc_in;
  p.acc_out = a->acc_out;
  if (logits) {
    p.z = e->rf_z;
    p.gp = refree_padded_group(e->cfg.group);
  }
  if (x) {
    p.unit_prefix = x->unit_prefix;
    p.pre_off = x->off;
    p.mem_off = x->mem_off;
    p.mem = x->mem;
    p.PK = static_cast<const uint4*>(x->K);
    p.PV = static_cast<const uint4*>(x->V);
  }

  // the units' own rows
  int64_t gsum = 0, gmax = 1;
  Sample sample;
  const int step = (U + 31) / 32;
  const int64_t within = a->pos ? INT64_MAX : reach(a->local, a->sinks, p.nq, 32);
  for (int u = 0; u < U; ++u) {
    const int64_t n = b->tok_off_host[u + 1] - b->tok_off_host[u];
    const int64_t g = std::min((n + 31) / 32, within);
    gsum += g;
    gmax = std::max(gmax, g);
    if (u == step * sample.n) sample.groups[sample.n++] = static_cast<float>(g);
  }
  const int64_t resident = static_cast<int64_t>(attend_warps_per_sm()) * e->nsm;
  // bytes per us: HBM's, or L2's where units read the same rows (the CTAs of one chunk
  // with more than 16 query rows do too, which measured 8e6)
  constexpr double kHbm = 6.5e6, kL2 = 13e6;
  int own = 1, warps = 4;
  const double narrow =
      pick_shape(sample, rg * static_cast<int64_t>(U), rg * gsum, gmax, resident, R,
                 rg > 1 ? 8e6 : kHbm, cap / rows - (x ? 1 : 0), logits, &warps, &own);
  // parts of own chunks; with more than 8 query rows and a prefix's parts also of a single
  // one, so that every row has a warp of its own for the join (in the unit's CTA up to four
  // rows wait for one another: 88 units of 800 rows, 32 query rows, 2 prefixes: 49.5 us, 47.7 so)
  const int64_t used = own > 1 || (x && R > 8) ? static_cast<int64_t>(own) * rows : 0;
  // which kernels run, and in how many chunks
  bool both = false, wide_own = false;
  AttendParams pp = {};   // the prefixes' launch
  int prefix_rows = 0;    // query rows of its longest item
  if (x) {
    // Either each unit reads its prefix before its own rows (from L2, where others read it
    // too), or the prefixes go through the wide kernel first, for all their units at once.
    // One launch and two, in us: 8 prefixes of 2048 tokens with 4 units each 12.7 and 13.9; 2
    // of 18500 with one unit of 16 query rows 19.9 and 26.8; 128 of 4096 with one unit 50 and
    // 59; 32 of 4096 with 4 units 37 and 28, with 8 units 64 and 32; 1 of 8000 with 64 units
    // 43 and 20.
    Sample all;
    int64_t dsum = 0, dmax = 1;
    const int64_t pwithin = reach(a->local, a->sinks, p.nq, 32);
    for (int u = 0; u < U; ++u) {
      const int k = x->unit_prefix_host[u];
      const int64_t n = b->tok_off_host[u + 1] - b->tok_off_host[u];
      int64_t g = std::min((n + 31) / 32, within);
      if (k >= 0) g += std::min((x->off_host[k + 1] - x->off_host[k] + 31) / 32, pwithin);
      dsum += g;
      dmax = std::max(dmax, g);
      if (u == step * all.n) all.groups[all.n++] = static_cast<float>(g);
    }
    const double again = static_cast<double>(dsum) / (gsum + (psum + 31) / 32);
    int dwarps = 4, dchunks = 1;
    const double direct =
        pick_shape(all, rg * static_cast<int64_t>(U), rg * dsum, dmax, resident, R,
                   std::min(kL2, kHbm * std::max(1.0, again)), cap / rows, logits, &dwarps,
                   &dchunks);
    const int64_t mrows = static_cast<int64_t>(members) * R, blocks = (mrows + 255) / 256;
    Sample tiles;
    const int P = x->num_prefixes, pstep = (P + 31) / 32;
    int64_t pg = 0, pmax = 1;
    for (int k = 0; k < P; ++k) {
      const int64_t g = (x->off_host[k + 1] - x->off_host[k] + kWideTile - 1) / kWideTile;
      pg += g;
      pmax = std::max(pmax, g);
      if (k == pstep * tiles.n) tiles.groups[tiles.n++] = static_cast<float>(g);
    }
    int wchunks = 1;
    // a tile takes 1.5 us with 256 query rows; a warp joins up to four rows one by one
    const double wide = pick_wide(tiles, P * blocks, pg * blocks, pmax, e->nsm,
                                  mrows > kWideTile ? 1.5 : 0.95, 0.0,
                                  0.09 * ((std::min(R, 16) + 3) / 4), (cap - used) / rows, &wchunks);
    both = direct < 1.15 * (wide + narrow - 5.0);   // as measured; 5: the second starts early
    if (both) {
      own = dchunks;
      warps = dwarps;
      gmax = dmax;
    } else {
      pp = p;
      pp.keep = nullptr;
      pp.pos = nullptr;
      pp.status = e->status;
      pp.maxch = wchunks;
      pp.gpc = static_cast<int>((pmax + pp.maxch - 1) / pp.maxch);
      pp.part_o = part_o + used * 128;
      pp.part_ml = part_ml + used;
      prefix_rows = static_cast<int>(mrows);
      p.pre_chunks = pp.maxch;
      p.pre_o = pp.part_o;
      p.pre_ml = pp.part_ml;
    }
  }
  // many query rows over whole units: each unit may go through the wide kernel as a
  // prefix of its own (64 units of 16000 rows, 32 query rows: 147 us narrow, 91 wide; 512
  // units of 300 rows, 16 query rows: 19 and 41)
  if (!x && R > 8 && !a->keep && !a->pos && L.T > 0) {
    const int64_t blocks = (R + 255) / 256;
    int64_t tsum = 0, tmax = 1;
    Sample tiles;
    const int64_t tiles_within = reach(a->local, a->sinks, p.nq, kWideTile);
    for (int u = 0; u < U; ++u) {
      const int64_t n = b->tok_off_host[u + 1] - b->tok_off_host[u];
      const int64_t t = std::min((n + kWideTile - 1) / kWideTile, tiles_within);
      tsum += t;
      tmax = std::max(tmax, t);
      if (u == step * tiles.n) tiles.groups[tiles.n++] = static_cast<float>(t);
    }
    int c = 1;
    const double cost = pick_wide(tiles, U * blocks, tsum * blocks, tmax, e->nsm, 0.95, 4.0, 0.0,
                                  cap / rows, &c);
    wide_own = cost < narrow && static_cast<int64_t>(c) * rows <= cap;
    if (wide_own) {
      p.PK = p.K;
      p.PV = p.V;
      p.pre_off = p.tok_off;
      p.maxch = c;
      p.gpc = static_cast<int>((tmax + c - 1) / c);
      p.part_o = part_o;
      p.part_ml = part_ml;
      p.status = e->status;
    }
  }
  const bool wide_prefix = x && !both;
  // a unit of one chunk whose logits were left does its weights itself
  const bool weights = a->acc_out && L.T > 0 && (own > 1 || !p.z);

  // every tensor map before the first launch: on an error nothing is enqueued
  CUtensorMap pkmap, pvmap, kmap, vmap;
  if (wide_prefix &&
      (make_map(e, &pkmap, x->K, static_cast<uint64_t>(psum), kWideTile) != RKV_OK ||
       make_map(e, &pvmap, x->V, static_cast<uint64_t>(psum), kWideTile) != RKV_OK))
    return RKV_ERR_CUDA;
  if ((wide_own || (weights && !p.z)) &&
      make_map(e, &kmap, b->K, static_cast<uint64_t>(L.T), kWideTile) != RKV_OK)
    return RKV_ERR_CUDA;
  if (wide_own && make_map(e, &vmap, b->V, static_cast<uint64_t>(L.T), kWideTile) != RKV_OK)
    return RKV_ERR_CUDA;

  cudaError_t err;
  if (wide_prefix) {
    t_begin(e, RKV_KERNEL_SHARED, st);
    err = launch_attend_wide(pkmap, pvmap, pp, x->num_prefixes, prefix_rows, st);
    t_end(e, st);
    if (err != cudaSuccess) return cuda_fail(err);
    ++e->launches;
  }
  if (wide_own) {
    t_begin(e, RKV_KERNEL_ATTEND, st);
    err = launch_attend_wide(kmap, vmap, p, U, R, st);
    p.pre_chunks = p.maxch;
    p.pre_o = part_o;
    p.pre_ml = part_ml;
    p.part_o = nullptr;
    if (err == cudaSuccess) err = launch_attend_finish(p, st);
    t_end(e, st);
    if (err != cudaSuccess) return cuda_fail(err);
    e->launches += 2;
  } else {
    p.maxch = own;
    p.gpc = static_cast<int>((gmax + own - 1) / own);
    if (own > 1 || (p.pre_o && R > 8)) {
      p.part_o = part_o;
      p.part_ml = part_ml;
      // up to 8 query rows are joined by the unit's last CTA, two per warp; 32 took it 16 us
      if (R <= 8) p.count = count;
    }
    t_begin(e, RKV_KERNEL_ATTEND, st);
    err = launch_attend(p, U, warps, both, wide_prefix, st);
    if (err == cudaSuccess && p.part_o && R > 8) {
      err = launch_attend_finish(p, st);
      ++e->launches;
    }
    t_end(e, st);
    if (err != cudaSuccess) return cuda_fail(err);
    ++e->launches;
  }
  if (weights) {
    AttendParams pw = p;
    pw.status = e->status;
    const int64_t tile = p.z ? 32 : kWideTile;   // rows of a group
    const int64_t all = (static_cast<int64_t>(L.nmax) + tile - 1) / tile;
    const int64_t wslots = (p.z ? 5 : tile_weights_ctas_per_sm(R)) * static_cast<int64_t>(e->nsm);
    pw.maxch = pick_chunks(U, L.T / tile + U, all, wslots, (static_cast<int64_t>(1) << 30) / U,
                           p.z ? 8 : 1, p.z ? 16.0 : 6.0);
    pw.gpc = static_cast<int>((all + pw.maxch - 1) / pw.maxch);
    t_begin(e, RKV_KERNEL_WEIGHT, st);
    err = p.z ? launch_attend_weights(pw, U, st) : launch_tile_weights(kmap, pw, U, st);
    t_end(e, st);
    if (err != cudaSuccess) return cuda_fail(err);
    ++e->launches;
  }
  return RKV_OK;
}

}  // namespace

extern "C" {

int rkv_attend(rkv_engine* e, const rkv_batch* b, const rkv_attention* a, rkv_stream_t stream) {
  NvtxRange nvtx_("rkv_attend");
  return attend(e, b, nullptr, a, stream);
}

int rkv_attend_shared(rkv_engine* e, const rkv_batch* b, const rkv_prefix* x,
                      const rkv_attention* a, rkv_stream_t stream) {
  NvtxRange nvtx_("rkv_attend_shared");
  if (!x) return RKV_ERR_INVALID_ARG;
  return attend(e, b, x, a, stream);
}

int rkv_evict_accumulated(rkv_engine* e, const rkv_batch* b, const float* acc,
                          const uint8_t* live, const int32_t* pos, int budget,
                          const int32_t* budgets, int sinks, uint8_t* keep, int32_t* free_slots,
                          int32_t* n_free, float* acc_out, int32_t* idx, int32_t* n_kept,
                          rkv_stream_t stream) {
  NvtxRange nvtx_("rkv_evict_accumulated");
  if (!e) return RKV_ERR_INVALID_ARG;
  Lengths L;
  int rc = check_rows(e, b, &L);
  if (rc != RKV_OK) return rc;
  const int U = b->num_units;
  if (budget < 0 || sinks < 0 || (idx == nullptr) != (n_kept == nullptr))
    return RKV_ERR_INVALID_ARG;
  if (U == 0) return RKV_OK;
  if (!n_free || (L.T > 0 && (!acc || !keep || !free_slots))) return RKV_ERR_INVALID_ARG;
  if (!aligned(acc, 4) || !aligned(pos, 4) || !aligned(budgets, 4) || !aligned(free_slots, 4) ||
      !aligned(n_free, 4) || !aligned(acc_out, 4) || !aligned(idx, 4) || !aligned(n_kept, 4))
    return RKV_ERR_INVALID_ARG;
  const int64_t W = static_cast<int64_t>(budget) + sinks + e->cfg.window;
  if (idx && (W >= (static_cast<int64_t>(1) << 30) || U * W >= (static_cast<int64_t>(1) << 31)))
    return RKV_ERR_UNSUPPORTED;
  DeviceGuard dev(e->device);
  if (!dev.ok) return cuda_fail(cudaErrorUnknown);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  DropParams p = {};
  p.tok_off = b->tok_off;
  p.acc = acc;
  p.live = live;
  p.pos = pos;
  p.budgets = budgets;
  p.budget = budget;
  p.sinks = sinks;
  p.w = e->cfg.window;
  p.W = idx ? static_cast<int>(W) : 0;
  p.keep = keep;
  p.free_slots = free_slots;
  p.n_free = n_free;
  p.acc_out = acc_out;
  p.idx = idx;
  p.n_kept = n_kept;
  p.vec = aligned(acc, 16) && aligned(acc_out, 16) && aligned(pos, 16) && aligned(live, 4) &&
          aligned(keep, 4) && aligned(free_slots, 16);
  p.status = e->status;
  t_begin(e, RKV_KERNEL_DROP, st);
  cudaError_t err = launch_drop(p, U, L.nmax, e->nsm, st);
  t_end(e, st);
  if (err != cudaSuccess) return cuda_fail(err);
  ++e->launches;
  return RKV_OK;
}

int rkv_fill_slots_ex(rkv_engine* e, const rkv_batch* b, void* K, void* V,
                      const int64_t* new_off, const int64_t* new_off_host, const void* K_new,
                      const void* V_new, const int32_t* pos_new, uint8_t* keep,
                      const int32_t* free_slots, const int32_t* n_free, int32_t* pos, float* acc,
                      int32_t* free_out, int32_t* n_free_out, rkv_stream_t stream) {
  NvtxRange nvtx_("rkv_fill_slots_ex");
  if (!e) return RKV_ERR_INVALID_ARG;
  Lengths L;
  int rc = check_rows(e, b, &L);
  if (rc != RKV_OK) return rc;
  const int U = b->num_units;
  if (!new_off || !new_off_host || !aligned(new_off, 8) || new_off_host[0] != 0)
    return RKV_ERR_INVALID_ARG;
  for (int u = 0; u < U; ++u)
    if (new_off_host[u + 1] < new_off_host[u]) return RKV_ERR_INVALID_ARG;
  const int64_t Tn = new_off_host[U];
  if (Tn >= (static_cast<int64_t>(1) << 31)) return RKV_ERR_UNSUPPORTED;
  if (U == 0) return RKV_OK;
  if (!n_free || !n_free_out ||
      (L.T > 0 && (!K || !V || !keep || !free_slots || !free_out)) ||
      (Tn > 0 && (!K_new || !V_new || (pos && !pos_new))))
    return RKV_ERR_INVALID_ARG;
  // the list and its counts move together
  if ((free_slots == free_out) != (n_free == n_free_out) && L.T > 0) return RKV_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(K_new, 16) || !aligned(V_new, 16) ||
      !aligned(pos_new, 4) || !aligned(free_slots, 4) || !aligned(n_free, 4) ||
      !aligned(pos, 4) || !aligned(acc, 4) || !aligned(free_out, 4) || !aligned(n_free_out, 4))
    return RKV_ERR_INVALID_ARG;
  DeviceGuard dev(e->device);
  if (!dev.ok) return cuda_fail(cudaErrorUnknown);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const FillExtra x = {pos_new, pos, acc, free_out, n_free_out};
  t_begin(e, RKV_KERNEL_FILL, st);
  cudaError_t err = launch_fill_slots(b->tok_off, U, new_off, Tn, K_new, V_new, K, V, keep,
                                      free_slots, n_free, x, e->status, e->nsm, st);
  t_end(e, st);
  if (err != cudaSuccess) return cuda_fail(err);
  ++e->launches;
  return RKV_OK;
}

}  // extern "C"
