// The weights of every cached row where the attention pass left no logits behind:
// acc_out_i = acc_in_i + sum_r p_{r,i} over a unit's R query rows, from K and the rows'
// log-sums, p = 2^(z - lse2).
//
// The logits are computed again with the TOKENS as the M side of tcgen05.mma: S^T (128
// tokens x R) = K_tile Q^T, a token per tensor-memory lane, so one thread adds its
// token's R weights without any exchange and writes one coalesced float.  K tiles come by
// TMA; a CTA takes a run of a unit's tiles, with two S^T buffers, so the product of the
// next tile and the loads of the ones after it run beside the sums.  Tiles that no query
// sees are not read.
//
// Bound: HBM, 256 + 8 bytes per row (R = 32: a tile of 128 rows costs 256 cycles of 2^x
// and 1400 of its share of HBM); with few units the latency of a tile's chain (product,
// tensor-memory load, 2^x, sums; hence four partial sums and no branch per row).  256
// units of 2900 rows, R = 32: 33 us beyond the attention's time (30 at HBM's rate); 39 units:
// 5 us, and 29 on m16n8k16 steps, which spread a token's query rows over four lanes.
// 256 query rows over 16 units of 8000 rows: 26 us.
#include "attend_common.cuh"

namespace rkv {
namespace {

constexpr int kTok = kWideTile;
constexpr uint32_t kTileB = kTok * 256;     // a K tile: two halves of 64 columns
constexpr uint64_t kDrainNs = 100000000ull;

// Four stages of K tiles for up to 256 query rows and one CTA per SM; two for up to 64 rows
// and two CTAs; one where a CTA has one tile, and five CTAs (671 units of 17 rows, 12 query
// rows: 20.7 us with two stages, 16.9 with one).  Offsets behind the ring and NQ query rows:
template <int NS>
struct WLayout {
  uint32_t q, qp, lse, bars, misc, alloc;   // Q, positions [NQ], log-sums [NQ], barriers, rest
  __host__ __device__ explicit WLayout(int NQ) {
    q = NS * kTileB;
    qp = q + NQ * 256;
    lse = qp + NQ * 4;
    bars = lse + NQ * 4;
    misc = bars + (2 * NS + 5) * 8;
    alloc = misc + 24 + 1024;   // base aligned to 1024
  }
};
__host__ __device__ __forceinline__ int padded_rows(int R) { return (R + 15) & ~15; }

__device__ __forceinline__ void drain(uint64_t* bar, uint32_t par) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, par))
    if (globaltimer_ns() - t0 > kDrainNs) return;
}

template <int NS>
__global__ void __launch_bounds__(192, NS == 4 ? 1 : NS == 2 ? 2 : 5)
    tile_weights_kernel(const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ AttendParams p) {
  const int R = p.R, NQ = padded_rows(R);   // query rows, and as the N side of the product
  const WLayout<NS> lay(NQ);
  extern __shared__ uint8_t w_raw[];
  uint8_t* sm = w_raw + ((1024u - (smem_u32(w_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + lay.bars);
  uint64_t* empty = full + NS;
  uint64_t* d_full = empty + NS;   // [2] S^T of a tile is in tensor memory
  uint64_t* d_empty = d_full + 2;  // [2] it has been read
  uint64_t* mdone = d_empty + 2;
  int* s_qp = reinterpret_cast<int*>(sm + lay.qp);
  float* s_lse = reinterpret_cast<float*>(sm + lay.lse);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + lay.misc);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + lay.misc + 4);
  int8_t* lastp = reinterpret_cast<int8_t*>(sm + lay.misc + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int item = blockIdx.x / p.maxch, chunk = blockIdx.x - item * p.maxch;
  const int64_t base = __ldg(&p.tok_off[item]);
  const int N = static_cast<int>(__ldg(&p.tok_off[item + 1]) - base);
  const int first = own_first(p, item);
  const int tiles = (N + kTok - 1) / kTok;
  const int t_end = min(tiles, (chunk + 1) * p.gpc), t_begin = chunk * p.gpc;
  if (t_begin >= t_end) {
    wait_for_previous_launch();
    return;
  }
  const int64_t qmax = p.q_pos ? static_cast<int64_t>(__ldg(&p.q_pos[item]))
                               : static_cast<int64_t>(first) + N - 1;
  const int64_t qmin = qmax - (p.nq - 1);
  const int qmax32 = clamp32(qmax), qmin32 = clamp32(qmin);
  const int lo_any = p.local > 0 ? clamp32(qmin - p.local) : INT_MIN;
  const int lo_all = p.local > 0 ? clamp32(qmax - p.local) : INT_MIN;
  // whether a query may see a row of tile t (rows in the order of their positions)
  auto needed = [&](int t) {
    if (p.pos) return true;
    const int a = first + t * kTok, b = a + kTok - 1;
    return a <= qmax32 && (b > lo_any || a < p.sinks);
  };

  if (tid == 0) {
    prefetch_tmap(&kmap);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      lastp[s] = -1;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 4);   // warps
    }
    mbar_init(mdone, 1);
    *abort = 0;
    fence_mbar_init();
  }
  // tensor-memory columns: a power of two, two buffers of NQ
  uint32_t cols = 32;
  while (cols < 2u * NQ) cols *= 2;
  if (warp == 1) {
    tmem_alloc<1>(tmem_slot, cols);
    tmem_relinquish<1>();
  }
  // Q in the layout that TMA writes for K, halves of NQ rows of 128 bytes
  for (int i = tid; i < NQ * 16; i += 192) {
    const int r = i >> 4, c = i & 15;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < R)
      v = __ldg(reinterpret_cast<const uint4*>(p.Q) + (static_cast<int64_t>(item) * R + r) * 16 + c);
    *reinterpret_cast<uint4*>(sm + lay.q + (c >> 3) * NQ * 128 + r * 128 +
                              (((c & 7) ^ (r & 7)) << 4)) = v;
  }
  for (int r = tid; r < NQ; r += 192) s_qp[r] = r < R ? clamp32(qmin + r % p.nq) : INT_MIN;
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol = policy_evict_first();
      int n = 0;
      for (int t = t_begin; t < t_end; ++t) {
        if (!needed(t)) continue;
        const int s = n % NS;
        const uint32_t ph = (n / NS) & 1;
        if (!mbar_wait(&empty[s], ph ^ 1, abort, p.status)) break;
        uint8_t* dst = sm + s * kTileB;
        const int y = static_cast<int>(base + static_cast<int64_t>(t) * kTok);
        mbar_arrive_expect_tx(&full[s], kTileB);
        tma_load_2d(dst, &kmap, &full[s], 0, y, pol);
        tma_load_2d(dst + kTileB / 2, &kmap, &full[s], 64, y, pol);
        lastp[s] = static_cast<int8_t>(ph);
        ++n;
      }
      // teardown: every copy issued has landed before the CTA exits
      for (int s = 0; s < NS; ++s)
        if (lastp[s] >= 0) drain(&full[s], lastp[s]);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t leader = elect_leader();
    const uint32_t idesc = idesc_bf16_f32(kTok, NQ);
    const uint64_t kd = desc_kmajor_sw128(smem_u32(sm));
    const uint64_t qd = desc_kmajor_sw128(smem_u32(sm + lay.q));
    const uint32_t a_full = smem_u32(d_full), a_empty = smem_u32(empty);
    int n = 0;
    bool ok = true;
    for (int t = t_begin; ok && t < t_end; ++t) {
      if (!needed(t)) continue;
      const int s = n % NS, b = n & 1;
      ok = mbar_wait(&full[s], (n / NS) & 1, abort, p.status);
      ok = ok && mbar_wait(&d_empty[b], ((n >> 1) & 1) ^ 1, abort, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t ko = ((k >> 2) * (kTileB / 2) + (k & 3) * 32) >> 4;
        const uint32_t qo = ((k >> 2) * NQ * 128 + (k & 3) * 32) >> 4;
        mma_bf16_by(leader, tmem + b * NQ, kd + s * (kTileB >> 4) + ko, qd + qo, idesc, k > 0);
      }
      mma_commit_by(leader, a_empty + 8 * s);
      mma_commit_by(leader, a_full + 8 * b);
      ++n;
    }
    // teardown: all MMAs (and their commits) are complete before TMEM is freed
    mma_commit_by(leader, smem_u32(mdone));
    drain(mdone, 0);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ a token per thread
    const int w4 = warp & 3;   // the tensor-memory lanes that this warp may read
    const uint32_t lanes = static_cast<uint32_t>(32 * w4) << 16;
    int n = 0;
    bool ok = true;
    // the log-sums: this launch may have started while they were computed
    wait_for_previous_launch();
    for (int r = tid - 64; r < NQ; r += 128)
      s_lse[r] = r < R ? __ldcg(&p.lse2[static_cast<int64_t>(item) * R + r]) : INFINITY;
    __syncwarp();
    named_bar_sync(1, 128);
    for (int t = t_begin; ok && t < t_end; ++t) {
      const int i = t * kTok + 32 * w4 + lane;
      const bool in = i < N;
      const int64_t at = base + i;
      float sum = in && p.acc_in ? p.acc_in[at] : 0.f;
      if (needed(t)) {
        int ps = first + i;
        uint32_t live = 1u;
        if (in && p.keep) live = __ldg(&p.keep[at]);
        if (in && p.pos) ps = __ldg(&p.pos[at]);
        const int b = n & 1;
        ok = mbar_wait(&d_full[b], (n >> 1) & 1, abort, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // seen by every query, by none, or by some
        const bool on = in && live != 0u && sees(ps, qmax32, lo_any, p.sinks);
        const bool masked = __any_sync(0xffffffffu, on && !sees(ps, qmin32, lo_all, p.sinks));
        const uint32_t from = tmem + lanes + b * NQ;
        float w[4] = {0.f, 0.f, 0.f, 0.f};
        // adds 16 query rows' weights; some: not every one sees the token
        auto add = [&](const uint32_t (&z)[16], int c0, bool some) {
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const float4 ls = *reinterpret_cast<const float4*>(s_lse + c0 + c);
            const float l[4] = {ls.x, ls.y, ls.z, ls.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float x = ex2(fmaf(__uint_as_float(z[c + k]), p.scale_log2, -l[k]));
              if (some) {   // not seen, or a padded row (0 x inf is not a weight)
                const int qp = s_qp[c0 + c + k];
                const int lo = p.local > 0 ? clamp32(static_cast<int64_t>(qp) - p.local) : INT_MIN;
                if (!(c0 + c + k < R && sees(ps, qp, lo, p.sinks))) x = 0.f;
              }
              w[k] += x;
            }
          }
        };
        uint32_t z[16];
        // blocks whose 16 rows all see the warp's tokens, then the others
        const int whole = masked ? 0 : R & ~15;
        for (int c0 = 0; c0 < NQ; c0 += 16) {
          tmem_ld16(from + c0, z);
          tmem_wait_ld_dep(z);
          if (c0 < whole) add(z, c0, false);
          else add(z, c0, true);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_empty[b]);
        // what lies in a dead row is dropped with its sum
        if (on) sum += (w[0] + w[1]) + (w[2] + w[3]);
        ++n;
      }
      if (in) p.acc_out[at] = sum;
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, cols);
  }
}

template <int NS>
cudaError_t configure_one(int rows) {
  return cudaFuncSetAttribute(tile_weights_kernel<NS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              WLayout<NS>(rows).alloc);
}
template <int NS>
cudaError_t launch_one(const CUtensorMap& kmap, const AttendParams& p, int U, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(U) * p.maxch);
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = WLayout<NS>(padded_rows(p.R)).alloc;
  cfg.stream = st;
  cudaLaunchAttribute at[1];   // starts while the sums are still being joined
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tile_weights_kernel<NS>, kmap, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t tile_weights_configure() {
  cudaError_t e = configure_one<4>(256);
  if (e == cudaSuccess) e = configure_one<2>(64);
  if (e == cudaSuccess) e = configure_one<1>(64);
  return e;
}

int tile_weights_ctas_per_sm(int R) { return R <= 64 ? 2 : 1; }

cudaError_t launch_tile_weights(const CUtensorMap& kmap, const AttendParams& p, int U,
                                cudaStream_t st) {
  if (p.R > 64) return launch_one<4>(kmap, p, U, st);
  return p.gpc > 1 ? launch_one<2>(kmap, p, U, st) : launch_one<1>(kmap, p, U, st);
}

}  // namespace rkv
