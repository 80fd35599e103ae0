// Attention of drafted trees for shapes outside the fast path, and the
// attention weights of selected entries (csa2_tree_attn, csa2_attn_weights).
//
// tree_generic_kernel -- any head count, dims and element type (bf16 rows of
//   whole 8-byte pieces go to tree_mma.cu).  One CTA per
//   (query, up to 8 heads).  A warp scores 16 key slots at a time: a quarter of
//   it takes four, its 8 lanes stride the dims, so that a row is read once per 8
//   heads and 16 rows are on their way; the 32 sums meet in a transposed
//   reduction that leaves four on every lane.  (All 32 lanes on one four of
//   slots spent as long on the reduction as on 64 dims.)  The softmax (fp32)
//   has all slots of its heads in shared memory.  For P V the slots go round
//   the warps, and in a warp round as many groups of lanes as rows of four dims a lane
//   leave; 8 rows of each are on their way, and the sums are added up in a
//   fixed order.  Bound by the rows' latency for few queries (20 queries, 4 heads
//   of 128, 640 slots, fp32: 18.5 us), by the fp32 products' instructions for many (128
//   queries, 40 heads of 100 / 128, 549 slots: 69 us, 19 TFLOP/s).
// weights_mma_kernel -- bf16, 64 heads of 192, few queries: one CTA per (query, 64
//   slots) gathers the K rows with 16-byte cp.async; S = Q K^T on mma.sync, and
//   exp2(s - lse) is summed over the heads in fixed order.  No maximum is
//   needed, the lse is the normaliser.  A latency chain (index, rows, product,
//   sum): 3.5 us a launch for up to 16 queries of 512 slots.
// weights_generic_kernel -- any shape: 16 slots a warp, as above, 8 heads at a time (128 queries of 256
//   slots, 16 heads of 100, fp32: 9.7 us).
#include "common.cuh"
#include "draft.h"
#include "tc.cuh"
#include "tree.cuh"

namespace csa2 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ generic tree attention

constexpr int kGenHeads = 8;
constexpr int kMaxSlots = 1024;     // topk + swa
constexpr int kPvDims = 128;        // dims of a P V pass: four a lane
constexpr int kPvRows = 8;          // V rows a warp has on their way

// Scores of 16 keys against 8 heads (queries in shared memory, fp32), by a
// warp: a quarter of it takes four keys, `row` (null: 0), its 8 lanes the dims,
// four neighbours at a time where rows are whole 16-byte pieces (kWide, fp32).
// Lane l ends with key l / 2 and heads 4 (l % 2) .. + 3.
template <int kDtype, bool kWide>
CSA2_DEV float4 score_keys(const void* const (&row)[4], const float* sq, int dim) {
  constexpr int kBatch = kWide ? 2 : 4;   // pieces of each row a lane has on their way
  const int part = threadIdx.x & 7;
  float acc[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] = 0.f;
  if constexpr (kWide) {
    for (int d0 = 4 * part; d0 < dim; d0 += 32 * kBatch) {
      float4 k[kBatch][4];
#pragma unroll
      for (int y = 0; y < kBatch; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          k[y][x] = row[x] != nullptr && d0 + 32 * y < dim
                        ? *reinterpret_cast<const float4*>(static_cast<const float*>(row[x]) + d0 + 32 * y)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        if (d0 + 32 * y >= dim) break;
#pragma unroll
        for (int h = 0; h < kGenHeads; ++h) {
          const float4 q = *reinterpret_cast<const float4*>(sq + h * dim + d0 + 32 * y);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float& c = acc[8 * x + h];
            c = __fmaf_rn(q.x, k[y][x].x, c);
            c = __fmaf_rn(q.y, k[y][x].y, c);
            c = __fmaf_rn(q.z, k[y][x].z, c);
            c = __fmaf_rn(q.w, k[y][x].w, c);
          }
        }
      }
    }
  } else {
    for (int d0 = part; d0 < dim; d0 += 8 * kBatch) {
      float k[kBatch][4];
#pragma unroll
      for (int y = 0; y < kBatch; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          k[y][x] = row[x] != nullptr && d0 + 8 * y < dim ? load_elem(row[x], d0 + 8 * y, kDtype) : 0.f;
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        if (d0 + 8 * y >= dim) break;
#pragma unroll
        for (int h = 0; h < kGenHeads; ++h) {
          const float q = sq[h * dim + d0 + 8 * y];
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[8 * x + h] = __fmaf_rn(q, k[y][x], acc[8 * x + h]);
        }
      }
    }
  }
  __syncwarp();
  // each step halves the values a lane holds and doubles the lanes they are summed over
#pragma unroll
  for (int n = 16; n >= 4; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool up = (part & (n >> 2)) != 0;
      const float keep = up ? acc[i + n] : acc[i], give = up ? acc[i] : acc[i + n];
      acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, n >> 2);
    }
  return make_float4(acc[0], acc[1], acc[2], acc[3]);
}

// Four elements from `i` on (kWide: one access; otherwise those below `end`).
template <int kDtype, bool kWide>
CSA2_DEV float4 load_four(const void* base, int i, int end) {
  if (kWide) return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
  float4 r;
  r.x = load_elem(base, i, kDtype);
  r.y = i + 1 < end ? load_elem(base, i + 1, kDtype) : 0.f;
  r.z = i + 2 < end ? load_elem(base, i + 2, kDtype) : 0.f;
  r.w = i + 3 < end ? load_elem(base, i + 3, kDtype) : 0.f;
  return r;
}

template <int kDtype, bool kWide, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) tree_generic_kernel(const TreeArgs a) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) float sh[];
  __shared__ int path[kMaxTreeTokens];
  __shared__ float red[kWarps * kGenHeads], inv_s[kGenHeads];
  const int b = blockIdx.y, h0 = blockIdx.x * kGenHeads, nh = min(kGenHeads, a.heads - h0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nslots = a.topk + a.swa, rounded = (nslots + 15) & ~15;
  const void** krow = reinterpret_cast<const void**>(sh);   // [rounded] rows of the slots (null: no key)
  const void** vrow = krow + rounded;
  float* sp = reinterpret_cast<float*>(vrow + rounded);     // [rounded][kGenHeads] logits -> weights
  float* sq = sp + rounded * kGenHeads;                     // [kGenHeads][k_dim]
  float* part = sq;                                         // later: [kWarps][kGenHeads][kPvDims] sums of P V
  const int esize = kDtype == 1 ? 4 : 2, seq = b / a.tokens;
  pdl_wait();
  for (int i = tid; i < kGenHeads * a.k_dim; i += kThreads) {
    const int h = i / a.k_dim;
    sq[i] = h < nh ? load_elem(a.q, ((long long)b * a.heads + h0) * a.k_dim + i, kDtype) : 0.f;
  }
  const TreeWindow win = tree_window(a, b, path, blockIdx.x == 0);
  for (int j = tid; j < rounded; j += kThreads) {
    const void *kb = nullptr, *vb = nullptr;
    long long row = 0;
    if (j < a.topk) {
      const int e = win.live ? a.idx[(long long)b * a.topk + j] : -1;
      if (e >= a.n_entries && blockIdx.x == 0) report(a.err, kErrBadIndex, e);
      if (e >= 0 && e < a.n_entries) {
        kb = a.k_main;
        vb = a.v_main;
        row = (long long)seq * a.n_entries + e;
      }
    } else if (j < nslots) {
      bool drafted;
      if (win.row(j - a.topk, row, drafted)) {
        kb = drafted ? a.k_draft : a.k_swa;
        vb = drafted ? a.v_draft : a.v_swa;
      }
    }
    krow[j] = kb != nullptr ? static_cast<const uint8_t*>(kb) + row * a.k_dim * esize : nullptr;
    vrow[j] = vb != nullptr ? static_cast<const uint8_t*>(vb) + row * a.v_dim * esize : nullptr;
  }
  __syncthreads();
  for (int j = 16 * warp; j < rounded; j += 16 * kWarps) {
    const int own = j + 4 * (lane >> 3);
    const void* const row[4] = {krow[own], krow[own + 1], krow[own + 2], krow[own + 3]};
    float4 s = score_keys<kDtype, kWide>(row, sq, a.k_dim);
    const bool key = krow[j + (lane >> 1)] != nullptr;
    s.x = key ? s.x * a.scale : -INFINITY;
    s.y = key ? s.y * a.scale : -INFINITY;
    s.z = key ? s.z * a.scale : -INFINITY;
    s.w = key ? s.w * a.scale : -INFINITY;
    *reinterpret_cast<float4*>(sp + j * kGenHeads + 4 * lane) = s;
  }
  __syncthreads();
  // softmax statistics: head tid % 8, every (threads / 8)th slot
  const int h = tid % kGenHeads, first = tid / kGenHeads;
  float m = -INFINITY;
  for (int j = first; j < nslots; j += kThreads / kGenHeads) m = fmaxf(m, sp[j * kGenHeads + h]);
  for (int o = kGenHeads; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane < kGenHeads) red[warp * kGenHeads + lane] = m;
  __syncthreads();
  m = red[h];
  for (int w = 1; w < kWarps; ++w) m = fmaxf(m, red[w * kGenHeads + h]);
  __syncthreads();
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int j = first; j < nslots; j += kThreads / kGenHeads) {
    const float p = expf(sp[j * kGenHeads + h] - base);
    sp[j * kGenHeads + h] = p;
    l += p;
  }
  for (int o = kGenHeads; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane < kGenHeads) red[warp * kGenHeads + lane] = l;
  __syncthreads();
  if (tid < kGenHeads) {
    l = 0.f;
    for (int w = 0; w < kWarps; ++w) l += red[w * kGenHeads + h];
    inv_s[tid] = l > 0.f ? 1.f / l : l;       // no key: 0; NaN stays NaN
    if (tid < nh && a.lse != nullptr)
      a.lse[(long long)b * a.heads + h0 + tid] = l == 0.f ? -INFINITY : base + logf(l);
  }
  __syncthreads();
  for (int d0 = 0; d0 < a.v_dim; d0 += kPvDims) {
    // the lanes of a row, as few as have four dims each; the others take other rows
    int lanes = 32;
    while (lanes > 4 && 2 * lanes >= a.v_dim - d0) lanes >>= 1;
    const int d = d0 + 4 * (lane & (lanes - 1)), step = kWarps * (32 / lanes);
    float4 acc[kGenHeads];
#pragma unroll
    for (int i = 0; i < kGenHeads; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = warp + kWarps * (lane / lanes); j0 < nslots; j0 += kPvRows * step) {
      float4 v[kPvRows];
#pragma unroll
      for (int x = 0; x < kPvRows; ++x) {
        const int j = j0 + x * step;
        const void* row = j < nslots ? vrow[j] : nullptr;
        v[x] = row != nullptr && d < a.v_dim ? load_four<kDtype, kWide>(row, d, a.v_dim) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int x = 0; x < kPvRows; ++x) {
        const int j = j0 + x * step;
        if (j >= nslots) break;
        const float4 plo = *reinterpret_cast<const float4*>(sp + j * kGenHeads);
        const float4 phi = *reinterpret_cast<const float4*>(sp + j * kGenHeads + 4);
        const float ps[kGenHeads] = {plo.x, plo.y, plo.z, plo.w, phi.x, phi.y, phi.z, phi.w};
#pragma unroll
        for (int i = 0; i < kGenHeads; ++i) {
          const float p = ps[i];
          acc[i].x = __fmaf_rn(p, v[x].x, acc[i].x);
          acc[i].y = __fmaf_rn(p, v[x].y, acc[i].y);
          acc[i].z = __fmaf_rn(p, v[x].z, acc[i].z);
          acc[i].w = __fmaf_rn(p, v[x].w, acc[i].w);
        }
      }
    }
    __syncwarp();
    for (int o = lanes; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < kGenHeads; ++i) {
        acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, o);
        acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, o);
        acc[i].z += __shfl_xor_sync(0xffffffffu, acc[i].z, o);
        acc[i].w += __shfl_xor_sync(0xffffffffu, acc[i].w, o);
      }
    if (lane < lanes)
#pragma unroll
      for (int i = 0; i < kGenHeads; ++i)
        *reinterpret_cast<float4*>(part + (warp * kGenHeads + i) * kPvDims + 4 * lane) = acc[i];
    __syncthreads();
    for (int i = tid; i < nh * kPvDims; i += kThreads) {
      const int head = i / kPvDims, x = i % kPvDims;
      if (d0 + x >= a.v_dim) continue;
      float o = 0.f;
      for (int w = 0; w < kWarps; ++w) o += part[(w * kGenHeads + head) * kPvDims + x];
      store_elem(a.out, ((long long)b * a.heads + h0 + head) * a.v_dim + d0 + x, kDtype, o * inv_s[head]);
    }
    __syncthreads();
  }
}

constexpr size_t generic_smem(int slots, int k_dim, int threads) {
  const size_t rounded = size_t(slots + 15) / 16 * 16;
  const size_t q = size_t(kGenHeads) * k_dim, sums = size_t(threads / 32) * kGenHeads * kPvDims;
  return rounded * 16 + (rounded * kGenHeads + (q > sums ? q : sums)) * sizeof(float);
}

// One CTA an SM with 16 warps while there are no more CTAs than SMs, two with
// 8 warps beyond (measured on an earlier form, 20 queries of 4 heads: 28 us with 16
// warps, 40 with 8; 128 queries of 40 heads: 116 and 95).
template <int kDtype, bool kWide, int kThreads>
cudaError_t launch_generic(const TreeArgs& a, int batch, cudaStream_t st) {
  const cudaError_t e = once_per_device(kSetupTreeGeneric + 2 * (kDtype + kWide) + (kThreads == 512), [] {
    return cudaFuncSetAttribute(tree_generic_kernel<kDtype, kWide, kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                int(generic_smem(kMaxSlots, 1024, kThreads)));
  });
  if (e != cudaSuccess) return e;
  note_launch();
  return launch_pdl(tree_generic_kernel<kDtype, kWide, kThreads>,
                    dim3(unsigned((a.heads + kGenHeads - 1) / kGenHeads), unsigned(batch)), dim3(kThreads),
                    generic_smem(a.topk + a.swa, a.k_dim, kThreads), st, 1, a);
}

template <int kDtype, bool kWide>
cudaError_t launch_generic(const TreeArgs& a, int batch, cudaStream_t st) {
  const bool few = (long long)batch * ((a.heads + kGenHeads - 1) / kGenHeads) <= device_sm_count();
  return few ? launch_generic<kDtype, kWide, 512>(a, batch, st) : launch_generic<kDtype, kWide, 256>(a, batch, st);
}

// fp32 rows of whole 16-byte pieces.
template <class... P>
bool wide_rows(int dtype, int dim, P... p) {
  uintptr_t at = 0;
  for (const void* x : {static_cast<const void*>(p)...}) at |= reinterpret_cast<uintptr_t>(x);
  return dtype == 1 && dim % 4 == 0 && at % 16 == 0;
}

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
  const bool off0 = n0 == -INFINITY, off1 = n1 == -INFINITY;
  n0 *= -kLog2e;
  n1 *= -kLog2e;
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
    float w0 = (off0 ? 0.f : ex2(__fmaf_rn(s[n][0], sl2, n0))) + (off1 ? 0.f : ex2(__fmaf_rn(s[n][2], sl2, n1)));
    float w1 = (off0 ? 0.f : ex2(__fmaf_rn(s[n][1], sl2, n0))) + (off1 ? 0.f : ex2(__fmaf_rn(s[n][3], sl2, n1)));
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

constexpr int kWGenThreads = 128, kWGenSlots = kWGenThreads / 2;   // 16 slots a warp

template <int kDtype, bool kWide>
__global__ void __launch_bounds__(kWGenThreads) weights_generic_kernel(const AttnWeightsArgs a) {
  extern __shared__ __align__(16) float sq[];   // [kGenHeads][k_dim]
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int j0 = blockIdx.x * kWGenSlots + 16 * warp, esize = kDtype == 1 ? 4 : 2;
  pdl_wait();
  const bool live = a.live == nullptr || a.live[b] != 0;
  int e = live && lane < 16 && j0 + lane < a.topk ? a.idx[(long long)b * a.topk + j0 + lane] : -1;   // of slot j0 + lane
  if (e >= a.n_entries) {
    report(a.err, kErrBadIndex, e);
    e = -1;
  }
  const void* row[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int y = __shfl_sync(0xffffffffu, e, 4 * (lane >> 3) + x);
    row[x] = y < 0 ? nullptr
                   : static_cast<const uint8_t*>(a.k_main) + ((long long)(b / a.seq_div) * a.n_entries + y) * a.k_dim * esize;
  }
  const bool key = __shfl_sync(0xffffffffu, e, lane >> 1) >= 0;
  float w = 0.f;                                // of slot j0 + lane / 2, every other four heads
  for (int h0 = 0; live && h0 < a.heads; h0 += kGenHeads) {
    const int nh = min(kGenHeads, a.heads - h0), h = 4 * (lane & 1);
    __syncthreads();
    for (int i = tid; i < kGenHeads * a.k_dim; i += kWGenThreads)
      sq[i] = i < nh * a.k_dim ? load_elem(a.q, ((long long)b * a.heads + h0) * a.k_dim + i, kDtype) : 0.f;
    float l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] = h + i < nh ? a.lse[(long long)b * a.heads + h0 + h + i] : -INFINITY;
    __syncthreads();
    const float4 s4 = score_keys<kDtype, kWide>(row, sq, a.k_dim);
    const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (key && l[i] != -INFINITY) w += expf(s[i] * a.scale - l[i]);
  }
  w += __shfl_xor_sync(0xffffffffu, w, 1);
  if ((lane & 1) == 0 && j0 + (lane >> 1) < a.topk) a.weights[(long long)b * a.topk + j0 + (lane >> 1)] = w;
}

// A cluster of CTAs per query where it has more than 384 keys and all the
// clusters run at once (up to 7/8 of two CTAs an SM: clusters do not fill every
// SM); groups of tokens on the tensor cores (a plan and a persistent launch)
// otherwise: their time goes with the keys, the clusters', of 160 slots a CTA,
// does not.  Measured, clusters / groups: 8 queries of 640 slots 12.2 / 14.7 us, 36 12.3 / 15.1,
// 64 15.2 / 15.9, 76 trees of 4 25.9 / 18.6, 256 queries 60 / 21; 32 queries of 549 slots
// 12.5 / 14.6, of 448 13.1 / 13.4, of 384 13.0 / 12.3, of 136 13.6 / 10.6; 1 query of 384
// 12.4 / 12.2.
constexpr int kFewSlots = 384;
bool tree_groups(const TreeArgs& a, int batch, size_t plan_bytes) {
  if (tree_plan_words(batch / a.tokens, a.tokens, a.topk, a.swa) * 4 > plan_bytes) return false;
  return a.topk + a.swa <= kFewSlots || 8LL * batch * attn_cluster(a.topk, a.swa) > 7LL * 2 * device_sm_count();
}

}  // namespace

cudaError_t launch_tree_attn(const TreeArgs& a, bool fast, int batch, void* plan, size_t plan_bytes, cudaStream_t st) {
  if (batch == 0) return cudaSuccess;
  if (fast) {
    return tree_groups(a, batch, plan_bytes) ? launch_tree_attn_tc(a, batch / a.tokens, plan, st)
                                            : launch_tree_attn_cluster(a, batch, st);
  }
  if (tree_rows_fit(a)) return launch_tree_rows(a, batch, st);
  if (wide_rows(a.dtype, a.k_dim, a.k_main, a.k_swa, a.k_draft) && wide_rows(a.dtype, a.v_dim, a.v_main, a.v_swa, a.v_draft))
    return launch_generic<1, true>(a, batch, st);
  return a.dtype == 1 ? launch_generic<1, false>(a, batch, st) : launch_generic<0, false>(a, batch, st);
}

cudaError_t launch_attn_weights(const AttnWeightsArgs& a, bool fast, int batch, cudaStream_t st) {
  if (batch == 0) return cudaSuccess;
  // Few queries: a CTA for every 64 slots, while each has an SM of its own; the
  // persistent tensor-core kernel beyond.  Measured, former / latter, 512 slots:
  // 1 query 3.5 / 4.3 us, 16 3.5 / 4.4, 24 5.2 / 4.4, 64 7.8 / 5.6, 256 16.0 / 10.8.
  const long long ctas = (long long)batch * ((a.topk + kWSlots - 1) / kWSlots);
  if (fast && ctas > device_sm_count()) return launch_attn_weights_tc(a, batch, st);
  if (!fast && weights_rows_fit(a)) return launch_weights_rows(a, batch, st);
  note_launch();
  if (fast)
    return launch_pdl(weights_mma_kernel, dim3(unsigned((a.topk + kWSlots - 1) / kWSlots), unsigned(batch)), dim3(kWThreads), 0,
                      st, 1, a);
  const dim3 grid(unsigned((a.topk + kWGenSlots - 1) / kWGenSlots), static_cast<unsigned>(batch));
  const auto kernel = wide_rows(a.dtype, a.k_dim, a.k_main) ? weights_generic_kernel<1, true>
                      : a.dtype == 1                        ? weights_generic_kernel<1, false>
                                                            : weights_generic_kernel<0, false>;
  return launch_pdl(kernel, grid, dim3(kWGenThreads), size_t(kGenHeads) * a.k_dim * sizeof(float), st, 1, a);
}

}  // namespace csa2
