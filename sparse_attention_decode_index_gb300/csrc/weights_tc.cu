// Attention weights of selected entries on the 5th-generation tensor cores, for
// batches that fill the GPU (csa2_attn_weights; bf16, 64 heads of 192):
//     w[b, j] = sum_h exp(scale q_h . k_j - lse_h).
//
// The keys are the rows of the product, S^T = K Q^T (128 keys x 64 heads), so
// that a thread owns a key and its sum over the heads needs no exchange.
// Persistent, one CTA an SM; a CTA takes a run of tiles (a query's slots, 128
// at a time), so that neighbouring tiles share their query:
//   8 producer warps gather K rows into a ring of 3 stages, and each query's
//     64 rows and normalisers into one of two buffers;
//   1 warp issues the 12 steps of a tile into one of two TMEM buffers;
//   4 warps turn the scores into weights.
// Bound by the gather (49 KB a tile): 256 queries of 512 slots 10.9 us, of which the
// distinct bytes need 4.3; plain loads and mma.sync took 16.1.
#include "common.cuh"
#include "draft.h"
#include "tc.cuh"

namespace csa2 {

namespace {

constexpr int kH = 64, kDk = 192;
constexpr int kTile = 128;
constexpr int kStages = 3;
constexpr int kOutWarps = 4, kProducerWarps = 8;
constexpr int kProducers = 32 * kProducerWarps;
constexpr int kThreads = 32 * (kOutWarps + kProducerWarps + 1);
constexpr float kLog2e = 1.4426950408889634f;

struct Shared {
  uint8_t k[kStages][kTile * kDk * 2];         // 3 blocks of 64 dims: 128 rows of 128 bytes
  uint8_t q[2][kH * kDk * 2];                  // 3 blocks of 64 dims: 64 rows of 128 bytes
  float shift[2][kH];                          // -lse in base 2
  uint32_t none[2][kH / 32];                    // heads whose lse is -inf
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full[2], shift_full[2], q_empty[2];
  uint64_t s_full[2], s_free[2];
  uint64_t fin;
  uint32_t tmem;
  volatile int abort;
};
constexpr int kSmem = int(sizeof(Shared)) + 1024;   // + room to align to 1,024

CSA2_DEV void cp16(uint32_t dst, const uint8_t* src, bool on) {   // zeros if not on
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16u : 0u) : "memory");
}

__global__ void __launch_bounds__(kThreads, 1) weights_tc_kernel(const AttnWeightsArgs a, int tiles_per_query, int n_tiles) {
  extern __shared__ uint8_t raw[];
  Shared& c = *reinterpret_cast<Shared*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&c.full[i], kProducers);
      mbar_init(&c.empty[i], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.q_full[b], kProducers);
      mbar_init(&c.shift_full[b], kH);
      mbar_init(&c.q_empty[b], 1 + 32 * kOutWarps);
      mbar_init(&c.s_full[b], 1);
      mbar_init(&c.s_free[b], 32 * kOutWarps);
    }
    mbar_init(&c.fin, 1);
    c.abort = 0;
    mbar_fence_init();
  }
  __syncwarp();
  if (warp == 0) tmem_alloc(&c.tmem, 128);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  pdl_wait();
  // this CTA's tiles
  const int lo = int((long long)n_tiles * blockIdx.x / gridDim.x), hi = int((long long)n_tiles * (blockIdx.x + 1) / gridDim.x);
  auto wanted = [&](int b) -> bool { return a.live == nullptr || a.live[b] != 0; };

  if (warp < kOutWarps) {
    // ---------------------------------------------------------------- weights: thread = key
    const float sl2 = a.scale * kLog2e;
    uint32_t tiles = 0, queries = 0;            // wanted ones so far
    for (int x = lo; x < hi;) {
      const int b = x / tiles_per_query, end = min(hi, (b + 1) * tiles_per_query);
      const bool on = wanted(b);
      const uint32_t qb = queries & 1;
      bool ok = !on || tc_wait_warp(c, &c.shift_full[qb], (queries >> 1) & 1, a.err);
      const uint32_t none0 = ok && on ? c.none[qb][0] : 0, none1 = ok && on ? c.none[qb][1] : 0;
      for (; x < end && ok; ++x) {
        const int j = (x - b * tiles_per_query) * kTile + tid;
        const long long at = (long long)b * a.topk + j;
        if (!on) {
          if (j < a.topk) a.weights[at] = 0.f;
          continue;
        }
        const int e = j < a.topk ? a.idx[at] : -1;
        const uint32_t buf = tiles & 1;
        ok = tc_wait_warp(c, &c.s_full[buf], (tiles >> 1) & 1, a.err);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[64];
        tmem_ld64(s, tmem + (uint32_t(warp * 32) << 16) + buf * 64);
        tc_fence_before();
        mbar_arrive(&c.s_free[buf]);
        ++tiles;
        if ((none0 | none1) != 0) {             // a head that attended nothing adds nothing, whatever its scores are
#pragma unroll
          for (int h = 0; h < kH; ++h)
            if (((h < 32 ? none0 : none1) >> (h & 31)) & 1u) s[h] = 0;
        }
        float2 w0 = make_float2(0.f, 0.f), w1 = w0;
#pragma unroll
        for (int h = 0; h < kH; h += 4) {
          const float4 n = *reinterpret_cast<const float4*>(&c.shift[qb][h]);
          w0 = add2(w0, make_float2(ex2(__fmaf_rn(__uint_as_float(s[h]), sl2, n.x)), ex2(__fmaf_rn(__uint_as_float(s[h + 1]), sl2, n.y))));
          w1 = add2(w1, make_float2(ex2(__fmaf_rn(__uint_as_float(s[h + 2]), sl2, n.z)), ex2(__fmaf_rn(__uint_as_float(s[h + 3]), sl2, n.w))));
        }
        w0 = add2(w0, w1);
        if (j < a.topk) a.weights[at] = e >= 0 && e < a.n_entries ? w0.x + w0.y : 0.f;
      }
      if (!ok) break;
      if (on) {
        mbar_arrive(&c.q_empty[qb]);
        ++queries;
      }
    }
  } else if (warp < kOutWarps + kProducerWarps) {
    // ---------------------------------------------------------------- producers: 16 keys of a tile a warp
    const int w = warp - kOutWarps, ptid = w * 32 + lane;
    uint32_t queries = 0, st = 0, lap = 0;
    bool ok = true;
    for (int x = lo; x < hi && ok;) {
      const int b = x / tiles_per_query, end = min(hi, (b + 1) * tiles_per_query);
      if (!wanted(b)) {
        x = end;
        continue;
      }
      const uint32_t qb = queries & 1;
      const uint8_t* k0 = static_cast<const uint8_t*>(a.k_main) + (long long)(b / a.seq_div) * a.n_entries * (kDk * 2);
      const int* idx = a.idx + (long long)b * a.topk;
      auto entry = [&](int tile) -> int {       // this lane's of a tile
        const int j = (tile - b * tiles_per_query) * kTile + w * 16 + lane;
        int e = lane < 16 && tile < end && j < a.topk ? idx[j] : -1;
        if (e >= a.n_entries) {
          report(a.err, kErrBadIndex, e);
          e = -1;
        }
        return e;
      };
      int e = entry(x);
      ok = queries < 2 || tc_wait_warp(c, &c.q_empty[qb], ((queries >> 1) - 1) & 1, a.err);
      if (!ok) break;
      if (ptid < kH) {
        const float l = a.lse[(long long)b * kH + ptid];
        c.shift[qb][ptid] = l == -INFINITY ? -INFINITY : -l * kLog2e;
        const unsigned none = __ballot_sync(0xffffffffu, l == -INFINITY);
        if (lane == 0) c.none[qb][w] = none;
        mbar_arrive(&c.shift_full[qb]);
      }
      const uint8_t* q0 = static_cast<const uint8_t*>(a.q) + (long long)b * kH * (kDk * 2);
      const uint32_t q_st = smem_u32(c.q[qb]);
#pragma unroll
      for (int p = ptid; p < kH * 24; p += kProducers) {
        const int r = p / 24, part = p - r * 24;
        cp16(q_st + (part >> 3) * (kH * 128) + r * 128 + (((part & 7) ^ (r & 7)) << 4), q0 + r * (kDk * 2) + part * 16, true);
      }
      cp_arrive(&c.q_full[qb]);
      ++queries;
      for (; x < end; ++x) {
        ok = tc_wait_warp(c, &c.empty[st], (lap & 1) ^ 1, a.err);
        if (!ok) break;
        const uint32_t k_st = smem_u32(c.k[st]);
#pragma unroll
        for (int f = 0; f < 4; ++f)             // four rows (24 pieces each) in three copies a lane
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const int p = 32 * i + lane, s = 4 * f + p / 24, part = p % 24, r = w * 16 + s;
            const int es = __shfl_sync(0xffffffffu, e, s);
            cp16(k_st + (part >> 3) * (kTile * 128) + r * 128 + (((part & 7) ^ (r & 7)) << 4),
                 k0 + (long long)max(es, 0) * (kDk * 2) + part * 16, es >= 0);
          }
        cp_arrive(&c.full[st]);
        e = entry(x + 1);
        if (++st == kStages) {
          st = 0;
          ++lap;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---------------------------------------------------------------- MMA issue
    constexpr uint32_t desc = idesc_bf16(kTile, kH, false);
    const uint64_t k0 = smem_desc(smem_u32(c.k[0]), 16, 1024), q0 = smem_desc(smem_u32(c.q[0]), 16, 1024);
    uint32_t tiles = 0, queries = 0, st = 0, lap = 0;
    bool ok = true;
    for (int x = lo; x < hi && ok;) {
      const int b = x / tiles_per_query, end = min(hi, (b + 1) * tiles_per_query);
      if (!wanted(b)) {
        x = end;
        continue;
      }
      const uint32_t qb = queries & 1;
      ok = tc_wait_warp(c, &c.q_full[qb], (queries >> 1) & 1, a.err);
      ++queries;
      for (; x < end && ok; ++x, ++tiles) {
        const uint32_t buf = tiles & 1;
        ok = tc_wait_warp(c, &c.full[st], lap & 1, a.err) &&
             (tiles < 2 || tc_wait_warp(c, &c.s_free[buf], ((tiles >> 1) - 1) & 1, a.err));
        if (!ok) break;
        fence_async_smem();                     // the copies are generic-proxy writes, the tensor core reads by the async proxy
        tc_fence_after();
        const uint64_t kd = k0 + st * (kTile * kDk * 2 >> 4), qd = q0 + qb * (kH * kDk * 2 >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kDk / 16; ++k)
            mma_ss(tmem + buf * 64, kd + ((k >> 2) * (kTile * 128) + (k & 3) * 32) / 16,
                   qd + ((k >> 2) * (kH * 128) + (k & 3) * 32) / 16, desc, k > 0);
          tc_commit(&c.empty[st]);
          tc_commit(&c.s_full[buf]);
          if (x == end - 1) tc_commit(&c.q_empty[qb]);
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          ++lap;
        }
      }
    }
    // every MMA has finished before the memory it uses is given up
    if (elect_one()) tc_commit(&c.fin);
    __syncwarp();
    mbar_wait(&c.fin, 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tmem, 128);
}

}  // namespace

cudaError_t launch_attn_weights_tc(const AttnWeightsArgs& a, int batch, cudaStream_t st) {
  const cudaError_t e = once_per_device(kSetupWeightsTc, [] {
    return cudaFuncSetAttribute(weights_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e != cudaSuccess) return e;
  const int per_query = (a.topk + kTile - 1) / kTile, n = batch * per_query;
  const int grid = n < device_sm_count() ? n : device_sm_count();
  note_launch();
  return launch_pdl(weights_tc_kernel, dim3(unsigned(grid)), dim3(kThreads), kSmem, st, 1, a, per_query, n);
}

}  // namespace csa2
