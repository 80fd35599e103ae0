// Attention of drafted trees for shapes outside the fast path, and the
// attention weights of selected entries (csa2_tree_attn, csa2_attn_weights).
//
// tree_generic_kernel -- any head count, dims and element type.  One CTA per
//   (query, up to 8 heads): a warp takes a key slot at a time, its lanes
//   striding the key's dims, and scores all the CTA's heads with the key in
//   registers, so a K row is read once per 8 heads; after the softmax (fp32,
//   one maximum and sum per head over all slots, which fit shared memory) the
//   V rows are read the same way.  Bound by issue and the row loads' latency.
// weights_mma_kernel -- bf16, 64 heads of 192, few queries: one CTA per (query, 64
//   slots) gathers the K rows with 16-byte cp.async; S = Q K^T on mma.sync, and
//   exp2(s - lse) is summed over the heads in fixed order.  No maximum is
//   needed, the lse is the normaliser.  A latency chain (index, rows, product,
//   sum): 3.5 us a launch for up to 16 queries of 512 slots.
// weights_generic_kernel -- any shape: a warp per slot.
#include "common.cuh"
#include "draft.h"
#include "tc.cuh"
#include "tree.cuh"

namespace csa2 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ generic tree attention

constexpr int kGenThreads = 256;
constexpr int kGenHeads = 8;
constexpr int kMaxSlots = 1024;     // topk + swa

CSA2_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kGenThreads) tree_generic_kernel(const TreeArgs a) {
  extern __shared__ float sh[];
  const int b = blockIdx.y, h0 = blockIdx.x * kGenHeads, nh = min(kGenHeads, a.heads - h0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nslots = a.topk + a.swa;
  float* sq = sh;                                       // [kGenHeads][k_dim]
  float* sp = sq + kGenHeads * a.k_dim;                 // [nslots][kGenHeads] logits -> weights
  int* path = reinterpret_cast<int*>(sp + nslots * kGenHeads);
  float* red = reinterpret_cast<float*>(path + kMaxTreeTokens);   // [8 warps][kGenHeads]
  float* acc_s = red + 8 * kGenHeads;                   // [kGenThreads][kGenHeads]
  pdl_wait();
  for (int i = tid; i < kGenHeads * a.k_dim; i += kGenThreads) {
    const int h = i / a.k_dim, d = i - h * a.k_dim;
    sq[i] = h < nh ? load_elem(a.q, ((long long)b * a.heads + h0 + h) * a.k_dim + d, a.dtype) : 0.f;
  }
  const TreeWindow win = tree_window(a, b, path, blockIdx.x == 0);
  __syncthreads();
  const int seq = b / a.tokens;
  // K / V arrays and row of slot j; false: no key
  auto slot_row = [&](int j, const void*& kb, const void*& vb, long long& row) -> bool {
    if (j < a.topk) {
      if (!win.live) return false;
      const int e = a.idx[(long long)b * a.topk + j];
      if (e < 0 || e >= a.n_entries) {
        if (e >= 0 && lane == 0 && blockIdx.x == 0) report(a.err, kErrBadIndex, e);
        return false;
      }
      kb = a.k_main;
      vb = a.v_main;
      row = (long long)seq * a.n_entries + e;
      return true;
    }
    bool drafted;
    if (!win.row(j - a.topk, row, drafted)) return false;
    kb = drafted ? a.k_draft : a.k_swa;
    vb = drafted ? a.v_draft : a.v_swa;
    return true;
  };
  for (int j = warp; j < nslots; j += kGenThreads / 32) {
    const void *kb, *vb;
    long long row;
    const bool ok = slot_row(j, kb, vb, row);
    float s[kGenHeads];
#pragma unroll
    for (int h = 0; h < kGenHeads; ++h) s[h] = 0.f;
    if (ok)
      for (int d = lane; d < a.k_dim; d += 32) {
        const float k = load_elem(kb, row * a.k_dim + d, a.dtype);
#pragma unroll
        for (int h = 0; h < kGenHeads; ++h) s[h] = __fmaf_rn(sq[h * a.k_dim + d], k, s[h]);
      }
#pragma unroll
    for (int h = 0; h < kGenHeads; ++h) s[h] = warp_sum(s[h]);
    if (lane < kGenHeads) {
      float v = s[0];
#pragma unroll
      for (int h = 1; h < kGenHeads; ++h) v = lane == h ? s[h] : v;
      sp[j * kGenHeads + lane] = ok ? v * a.scale : -INFINITY;
    }
  }
  __syncthreads();
  // softmax statistics: head tid % 8 of every eighth thread group
  const int h = tid % kGenHeads, part = tid / kGenHeads;   // 32 parts
  float m = -INFINITY;
  for (int j = part; j < nslots; j += kGenThreads / kGenHeads) m = fmaxf(m, sp[j * kGenHeads + h]);
  for (int o = kGenHeads; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane < kGenHeads) red[warp * kGenHeads + lane] = m;
  __syncthreads();
  m = red[h];
  for (int w = 1; w < 8; ++w) m = fmaxf(m, red[w * kGenHeads + h]);
  __syncthreads();
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int j = part; j < nslots; j += kGenThreads / kGenHeads) {
    const float p = expf(sp[j * kGenHeads + h] - base);
    sp[j * kGenHeads + h] = p;
    l += p;
  }
  for (int o = kGenHeads; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane < kGenHeads) red[warp * kGenHeads + lane] = l;
  __syncthreads();
  l = 0.f;
  for (int w = 0; w < 8; ++w) l += red[w * kGenHeads + h];
  __syncthreads();
  if (tid < nh && a.lse != nullptr)
    a.lse[(long long)b * a.heads + h0 + tid] = m == -INFINITY ? -INFINITY : m + logf(l);
  if (tid < kGenHeads) red[tid] = l > 0.f ? 1.f / l : 0.f;
  __syncthreads();
  // O: `wide` threads cover the dims, the thread groups share out the slots
  int wide = 32;
  while (wide < a.v_dim && wide < kGenThreads) wide <<= 1;
  const int groups = kGenThreads / wide, grp = tid / wide, col = tid - grp * wide;
  for (int d0 = 0; d0 < a.v_dim; d0 += wide) {
    const int d = d0 + col;
    float acc[kGenHeads];
#pragma unroll
    for (int i = 0; i < kGenHeads; ++i) acc[i] = 0.f;
    for (int j = grp; j < nslots; j += groups) {
      const void *kb, *vb;
      long long row;
      if (!slot_row(j, kb, vb, row)) continue;
      const float v = d < a.v_dim ? load_elem(vb, row * a.v_dim + d, a.dtype) : 0.f;
#pragma unroll
      for (int i = 0; i < kGenHeads; ++i) acc[i] = __fmaf_rn(sp[j * kGenHeads + i], v, acc[i]);
    }
#pragma unroll
    for (int i = 0; i < kGenHeads; ++i) acc_s[tid * kGenHeads + i] = acc[i];
    __syncthreads();
    if (grp == 0 && d < a.v_dim)
      for (int i = 0; i < nh; ++i) {
        float o = 0.f;
        for (int g = 0; g < groups; ++g) o += acc_s[(g * wide + col) * kGenHeads + i];
        store_elem(a.out, ((long long)b * a.heads + h0 + i) * a.v_dim + d, a.dtype, o * red[i]);
      }
    __syncthreads();
  }
}

size_t generic_smem(const TreeArgs& a) {
  return (size_t(kGenHeads) * a.k_dim + size_t(a.topk + a.swa) * kGenHeads + kMaxTreeTokens + 8 * kGenHeads +
          size_t(kGenThreads) * kGenHeads) * sizeof(float);
}
constexpr size_t kGenSmemMax = (size_t(kGenHeads) * 1024 + size_t(kMaxSlots) * kGenHeads + kMaxTreeTokens +
                                8 * kGenHeads + size_t(kGenThreads) * kGenHeads) * sizeof(float);

// ------------------------------------------------------------------ attention weights

constexpr int kH = 64, kDk = 192;
constexpr int kWThreads = 128;
constexpr int kWSlots = 64;                     // slots per CTA
constexpr int kKRow = kDk * 2 + 16;             // padded: ldmatrix rows hit distinct banks

__global__ void __launch_bounds__(kWThreads) weights_mma_kernel(const AttnWeightsArgs a) {
  __shared__ __align__(128) uint8_t rows[kWSlots * kKRow];
  __shared__ float sum_s[4][kWSlots];
  const int b = blockIdx.y, j0 = blockIdx.x * kWSlots, nj = min(kWSlots, a.topk - j0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  pdl_wait();
  float* out = a.weights + (long long)b * a.topk + j0;
  if (a.live != nullptr && a.live[b] == 0) {
    for (int j = tid; j < nj; j += kWThreads) out[j] = 0.f;
    return;
  }
  const int* idx = a.idx + (long long)b * a.topk + j0;
  // The warp copies slots 16 * warp .. + 15: four rows (24 pieces of 16 bytes each) in three copies a lane.
  int e = lane < 16 && warp * 16 + lane < nj ? idx[warp * 16 + lane] : -1;
  if (e >= a.n_entries) {
    report(a.err, kErrBadIndex, e);
    e = -1;
  }
  const uint8_t* k0 = static_cast<const uint8_t*>(a.k_main) + (long long)(b / a.seq_div) * a.n_entries * (kDk * 2);
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int p = 32 * i + lane, s = 4 * q + p / 24, part = p % 24;
      const int es = __shfl_sync(0xffffffffu, e, s);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(rows + (warp * 16 + s) * kKRow + part * 16)),
                   "l"(k0 + (es >= 0 ? (long long)es * (kDk * 2) + part * 16 : 0)), "r"(es >= 0 ? 16u : 0u)
                   : "memory");
    }
  asm volatile("cp.async.commit_group;" ::: "memory");
  uint32_t qa[kDk / 16][4];
  {
    const uint32_t* q0 = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.q) +
                                                           ((long long)b * kH + warp * 16 + g) * (kDk * 2)) + t;
    const uint32_t* q1 = q0 + 8 * (kDk / 2);
#pragma unroll
    for (int ks = 0; ks < kDk / 16; ++ks) {
      qa[ks][0] = q0[ks * 8];
      qa[ks][1] = q1[ks * 8];
      qa[ks][2] = q0[ks * 8 + 4];
      qa[ks][3] = q1[ks * 8 + 4];
    }
  }
  // -lse in base 2; a head that attended nothing adds nothing
  float n0 = a.lse[(long long)b * kH + warp * 16 + g], n1 = a.lse[(long long)b * kH + warp * 16 + g + 8];
  n0 = n0 == -INFINITY ? -INFINITY : -n0 * kLog2e;
  n1 = n1 == -INFINITY ? -INFINITY : -n1 * kLog2e;
  const float sl2 = a.scale * kLog2e;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  const uint8_t* krow = rows + ((lane & 7) + 8 * (lane >> 4)) * kKRow + ((lane >> 3) & 1) * 16;
  float s[kWSlots / 8][4] = {};                 // 8 keys each: independent sums, whose steps overlap
#pragma unroll
  for (int ks = 0; ks < kDk / 16; ++ks)
#pragma unroll
    for (int jp = 0; jp < kWSlots / 16; ++jp) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4(b0, b1, b2, b3, krow + jp * 16 * kKRow + ks * 32);
      mma_bf16(s[2 * jp], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b0, b1);
      mma_bf16(s[2 * jp + 1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b2, b3);
    }
#pragma unroll
  for (int n = 0; n < kWSlots / 8; ++n) {
    float w0 = ex2(__fmaf_rn(s[n][0], sl2, n0)) + ex2(__fmaf_rn(s[n][2], sl2, n1));
    float w1 = ex2(__fmaf_rn(s[n][1], sl2, n0)) + ex2(__fmaf_rn(s[n][3], sl2, n1));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      w0 += __shfl_xor_sync(0xffffffffu, w0, o);
      w1 += __shfl_xor_sync(0xffffffffu, w1, o);
    }
    if (g == 0) *reinterpret_cast<float2*>(&sum_s[warp][8 * n + 2 * t]) = make_float2(w0, w1);
  }
  __syncthreads();
  if (tid < nj) {                               // the warps' sums in their order
    const int id = idx[tid];
    out[tid] = id < 0 || id >= a.n_entries ? 0.f : (sum_s[0][tid] + sum_s[1][tid]) + (sum_s[2][tid] + sum_s[3][tid]);
  }
}

__global__ void __launch_bounds__(256) weights_generic_kernel(const AttnWeightsArgs a) {
  extern __shared__ float sq[];                 // [kGenHeads][k_dim]
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int j = blockIdx.x * 8 + warp;
  pdl_wait();
  const bool live = a.live == nullptr || a.live[b] != 0;
  int e = live && j < a.topk ? a.idx[(long long)b * a.topk + j] : -1;
  if (e >= a.n_entries) {
    if (lane == 0) report(a.err, kErrBadIndex, e);
    e = -1;
  }
  const long long row = ((long long)(b / a.seq_div) * a.n_entries + e) * a.k_dim;
  float w = 0.f;
  for (int h0 = 0; live && h0 < a.heads; h0 += kGenHeads) {
    const int nh = min(kGenHeads, a.heads - h0);
    __syncthreads();
    for (int i = tid; i < nh * a.k_dim; i += 256)
      sq[i] = load_elem(a.q, ((long long)b * a.heads + h0) * a.k_dim + i, a.dtype);
    __syncthreads();
    if (e < 0) continue;
    float s[kGenHeads];
#pragma unroll
    for (int h = 0; h < kGenHeads; ++h) s[h] = 0.f;
    for (int d = lane; d < a.k_dim; d += 32) {
      const float k = load_elem(a.k_main, row + d, a.dtype);
#pragma unroll
      for (int h = 0; h < kGenHeads; ++h)
        if (h < nh) s[h] = __fmaf_rn(sq[h * a.k_dim + d], k, s[h]);
    }
#pragma unroll
    for (int h = 0; h < kGenHeads; ++h) {
      if (h >= nh) break;
      const float d = warp_sum(s[h]);
      const float l = a.lse[(long long)b * a.heads + h0 + h];
      if (l != -INFINITY) w += expf(d * a.scale - l);
    }
  }
  if (lane == 0 && j < a.topk) a.weights[(long long)b * a.topk + j] = w;
}

// A cluster of CTAs per query while all the clusters run at once (up to 7/8 of
// two CTAs an SM: clusters do not fill every SM), pairs of tokens on the tensor
// cores beyond.  Measured, clusters / pairs, 512 + 128 slots: 64 queries of one
// token 15.3 / 15.0 us, 66 of trees of 33 16.4 / 19.9, 76 of trees of 4 25.9 / 19.0,
// 256 of one token 60 / 26, 256 of trees of 16 59 / 21.
bool tree_pairs(const TreeArgs& a, int batch, size_t plan_bytes) {
  if (tree_plan_words(batch / a.tokens, a.tokens, a.topk, a.swa) * 4 > plan_bytes) return false;
  return 8 * batch * attn_cluster(a.topk, a.swa) > 7 * 2 * device_sm_count();
}

}  // namespace

cudaError_t launch_tree_attn(const TreeArgs& a, bool fast, int batch, void* plan, size_t plan_bytes, cudaStream_t st) {
  if (batch == 0) return cudaSuccess;
  if (fast) {
    return tree_pairs(a, batch, plan_bytes) ? launch_tree_attn_tc(a, batch / a.tokens, plan, st)
                                            : launch_tree_attn_cluster(a, batch, st);
  }
  const cudaError_t e = once_per_device(kSetupTreeGeneric, [] {
    return cudaFuncSetAttribute(tree_generic_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kGenSmemMax));
  });
  if (e != cudaSuccess) return e;
  note_launch();
  return launch_pdl(tree_generic_kernel, dim3(unsigned((a.heads + kGenHeads - 1) / kGenHeads), unsigned(batch)),
                    dim3(kGenThreads), generic_smem(a), st, 1, a);
}

cudaError_t launch_attn_weights(const AttnWeightsArgs& a, bool fast, int batch, cudaStream_t st) {
  if (batch == 0) return cudaSuccess;
  // Few queries: a CTA for every 64 slots, while each has an SM of its own; the
  // persistent tensor-core kernel beyond.  Measured, former / latter, 512 slots:
  // 1 query 3.5 / 4.3 us, 16 3.5 / 4.4, 24 5.2 / 4.4, 64 7.8 / 5.6, 256 16.0 / 10.8.
  const long long ctas = (long long)batch * ((a.topk + kWSlots - 1) / kWSlots);
  if (fast && ctas > device_sm_count()) return launch_attn_weights_tc(a, batch, st);
  note_launch();
  if (fast)
    return launch_pdl(weights_mma_kernel, dim3(unsigned((a.topk + kWSlots - 1) / kWSlots), unsigned(batch)), dim3(kWThreads), 0,
                      st, 1, a);
  return launch_pdl(weights_generic_kernel, dim3(unsigned((a.topk + 7) / 8), unsigned(batch)), dim3(256),
                    size_t(kGenHeads) * a.k_dim * sizeof(float), st, 1, a);
}

}  // namespace csa2
