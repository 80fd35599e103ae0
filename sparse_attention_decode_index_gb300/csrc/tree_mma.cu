// Attention of drafted trees and attention weights for bf16 shapes outside the
// fast path whose rows are whole 8-byte pieces: products on mma.sync, operands
// straight from the gathered rows.
//
// tree_rows_kernel -- one CTA per (query, 16 heads).
//   S = Q K^T   a warp takes 16 slots at a time.  mma's B operand wants two pairs of
//     k of one key per lane; a sum has no order, so lane t of a quad takes
//     elements 16 s + 4 t .. + 3 of its key in one 8-byte load and Q is read
//     in the same order: no staging, no shuffles, 16 loads on their way.
//   softmax     fp32, a warp per head, over all slots in shared memory.
//   O = P V     the slots go round the warps, 16 a step.  B wants the pairs along the
//     slots: a lane loads four dims of its four slots and interleaves them, so
//     that column g of product j is dim 4 g + j.  P is rounded to bf16 as on
//     the fast path (half a step, 2^-8 of a weight; its sum is not rounded).
//     The warps' sums are added up in their order.
//   Bound by latency, two round trips to memory per 16 slots of a warp: 126
//   queries, 40 heads of 100 / 64, 576 slots 23.4 us (fp32 products in
//   tree_generic_kernel: 104), 110 queries, 40 heads of 64 / 16, 640 slots 19.6
//   (84), 58 queries, 16 heads of 100 / 128, 640 slots 15.1 (30.2).
// weights_rows_kernel -- one CTA per (query, 64 slots), the same scores for 16
//   heads at a time; exp(s - lse) is summed over the heads in a fixed order.
#include "common.cuh"
#include "draft.h"
#include "tree.cuh"

namespace csa2 {

namespace {

constexpr int kTileHeads = 16, kTileSlots = 16;
constexpr int kStepBatch = 8;       // k steps of 16 whose loads are on their way together
constexpr int kPassDims = 64;       // dims of a P V pass
constexpr int kMaxSlots = 1024;     // topk + swa

// Bytes of a staged Q row: 32 past a multiple of 128, so that eight rows' 8-byte pieces fall into distinct banks.
constexpr int q_stride(int k_dim) { return (k_dim * 2 + 127) / 128 * 128 + 32; }
// Words of a head's logits: 8 past a multiple of 32, for the same reason.
constexpr int p_stride(int slots) { return (slots + 31) / 32 * 32 + 8; }

// Warps' sums of P V that are kept side by side: with 8 warps the upper four hand
// theirs to the lower four, which leaves room for three CTAs an SM (126 queries of 40
// heads of 100 / 64, 576 slots: 23.4 us, two CTAs 28.4; 320 slots 19.6 and 23.7); the one CTA of 16
// warps has room for all, and the turns cost it 0.4 us.
constexpr int sums_of(int threads) { return threads == 256 ? threads / 64 : threads / 32; }

// 16 heads of Q (rows from `heads` on are zero, and so are dims up to the next multiple of 16).
CSA2_DEV void stage_q(uint8_t* sq, const void* q, int heads, int k_dim, int threads) {
  const int pieces = (k_dim + 15) / 16 * 4, stride = q_stride(k_dim);
  for (int i = threadIdx.x; i < kTileHeads * pieces; i += threads) {
    const int h = i / pieces, d = i % pieces * 4;
    uint2 v = make_uint2(0u, 0u);
    if (h < heads && d < k_dim) v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(q) + h * k_dim + d);
    *reinterpret_cast<uint2*>(sq + h * stride + d * 2) = v;
  }
}

// q . k of 16 heads and 16 keys: row[x] is key 8 x + lane / 4 (null: zeros).
// c[x][0, 1] are head lane / 4 and keys 8 x + 2 (lane % 4) + 0, 1; c[x][2, 3] head lane / 4 + 8.
CSA2_DEV void score_rows(const uint8_t* const (&row)[2], const uint8_t* sq, int k_dim, float (&c)[2][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int steps = (k_dim + 15) / 16, stride = q_stride(k_dim);
  const uint8_t* qa = sq + g * stride + 8 * t;
  const uint8_t* qb = qa + 8 * stride;
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[x][i] = 0.f;
  for (int s0 = 0; s0 < steps; s0 += kStepBatch) {
    uint2 k[kStepBatch][2];
#pragma unroll
    for (int y = 0; y < kStepBatch; ++y) {
      const int d = 16 * (s0 + y) + 4 * t;
#pragma unroll
      for (int x = 0; x < 2; ++x)
        k[y][x] = row[x] != nullptr && d < k_dim ? *reinterpret_cast<const uint2*>(row[x] + 2 * d) : make_uint2(0u, 0u);
    }
#pragma unroll
    for (int y = 0; y < kStepBatch; ++y) {
      if (s0 + y >= steps) break;
      const uint2 a = *reinterpret_cast<const uint2*>(qa + 32 * (s0 + y));
      const uint2 b = *reinterpret_cast<const uint2*>(qb + 32 * (s0 + y));
#pragma unroll
      for (int x = 0; x < 2; ++x) mma_bf16(c[x], a.x, b.x, a.y, b.y, k[y][x].x, k[y][x].y);
    }
  }
}

CSA2_DEV uint32_t bf16_pair(float2 p) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(p.x, p.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 3 : 1) tree_rows_kernel(const TreeArgs a) {
  constexpr int kWarps = kThreads / 32, kSums = sums_of(kThreads), kTurns = kWarps / kSums;
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ int path[kMaxTreeTokens];
  __shared__ float inv_s[kTileHeads];
  const int b = blockIdx.y, h0 = blockIdx.x * kTileHeads, nh = min(kTileHeads, a.heads - h0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int nslots = a.topk + a.swa, rounded = (nslots + kTileSlots - 1) / kTileSlots * kTileSlots;
  const int ld = p_stride(nslots), seq = b / a.tokens;
  const uint8_t** krow = reinterpret_cast<const uint8_t**>(sm);   // [rounded] rows of the slots (null: no key)
  const uint8_t** vrow = krow + rounded;
  float* sp = reinterpret_cast<float*>(vrow + rounded);           // [kTileHeads][ld] logits -> weights
  uint8_t* sq = reinterpret_cast<uint8_t*>(sp + kTileHeads * ld); // [kTileHeads][q_stride]
  float* part = reinterpret_cast<float*>(sq);                     // later: [kSums][kTileHeads][kPassDims]
  pdl_wait();
  stage_q(sq, static_cast<const __nv_bfloat16*>(a.q) + ((long long)b * a.heads + h0) * a.k_dim, nh, a.k_dim, kThreads);
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
    krow[j] = kb != nullptr ? static_cast<const uint8_t*>(kb) + row * a.k_dim * 2 : nullptr;
    vrow[j] = vb != nullptr ? static_cast<const uint8_t*>(vb) + row * a.v_dim * 2 : nullptr;
  }
  __syncthreads();
  for (int j = kTileSlots * warp; j < rounded; j += kTileSlots * kWarps) {
    const uint8_t* const row[2] = {krow[j + g], krow[j + 8 + g]};
    float c[2][4];
    score_rows(row, sq, a.k_dim, c);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int at = j + 8 * x + 2 * t;
      const bool key0 = krow[at] != nullptr, key1 = krow[at + 1] != nullptr;
      float2 s;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        s.x = key0 ? c[x][2 * y] * a.scale : -INFINITY;
        s.y = key1 ? c[x][2 * y + 1] * a.scale : -INFINITY;
        *reinterpret_cast<float2*>(sp + (g + 8 * y) * ld + at) = s;
      }
    }
  }
  __syncthreads();
  for (int h = warp; h < kTileHeads; h += kWarps) {
    float* p = sp + h * ld;
    float m = -INFINITY, l = 0.f;
    for (int j = lane; j < rounded; j += 32) m = fmaxf(m, p[j]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    for (int j = lane; j < rounded; j += 32) {
      const float e = expf(p[j] - base);
      p[j] = e;
      l += e;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      inv_s[h] = l > 0.f ? 1.f / l : l;         // no key: 0; NaN stays NaN
      if (h < nh && a.lse != nullptr) a.lse[(long long)b * a.heads + h0 + h] = l == 0.f ? -INFINITY : base + logf(l);
    }
  }
  __syncthreads();
  for (int d0 = 0; d0 < a.v_dim; d0 += kPassDims) {
    float acc[2][4][4];
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i >> 4][(i >> 2) & 3][i & 3] = 0.f;
    for (int j0 = kTileSlots * warp; j0 < rounded; j0 += 2 * kTileSlots * kWarps) {
      uint2 v[2][2][4];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int j = j0 + y * kTileSlots * kWarps + 2 * t;
        const bool in = j0 + y * kTileSlots * kWarps < rounded;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint8_t* row = in ? vrow[j + (r & 1) + 4 * (r & 2)] : nullptr;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int d = d0 + 32 * x + 4 * g;
            v[y][x][r] = row != nullptr && d < a.v_dim ? *reinterpret_cast<const uint2*>(row + 2 * d) : make_uint2(0u, 0u);
          }
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int j = j0 + y * kTileSlots * kWarps;
        if (j >= rounded) break;
        const float* pa = sp + g * ld + j + 2 * t;
        const float* pb = pa + 8 * ld;
        const uint32_t a0 = bf16_pair(*reinterpret_cast<const float2*>(pa)), a1 = bf16_pair(*reinterpret_cast<const float2*>(pb));
        const uint32_t a2 = bf16_pair(*reinterpret_cast<const float2*>(pa + 8));
        const uint32_t a3 = bf16_pair(*reinterpret_cast<const float2*>(pb + 8));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint2(&w)[4] = v[y][x];
          mma_bf16(acc[x][0], a0, a1, a2, a3, __byte_perm(w[0].x, w[1].x, 0x5410), __byte_perm(w[2].x, w[3].x, 0x5410));
          mma_bf16(acc[x][1], a0, a1, a2, a3, __byte_perm(w[0].x, w[1].x, 0x7632), __byte_perm(w[2].x, w[3].x, 0x7632));
          mma_bf16(acc[x][2], a0, a1, a2, a3, __byte_perm(w[0].y, w[1].y, 0x5410), __byte_perm(w[2].y, w[3].y, 0x5410));
          mma_bf16(acc[x][3], a0, a1, a2, a3, __byte_perm(w[0].y, w[1].y, 0x7632), __byte_perm(w[2].y, w[3].y, 0x7632));
        }
      }
    }
    // Columns 2 t and 2 t + 1 of product j are dims 8 t + j and 8 t + 4 + j
    auto place = [&](int w, int x, int i) -> float4& {
      return *reinterpret_cast<float4*>(part + (w * kTileHeads + g + 8 * (i >> 1)) * kPassDims + 32 * x + 8 * t + 4 * (i & 1));
    };
#pragma unroll
    for (int turn = kTurns - 1; turn >= 0; --turn) {
      if (warp / kSums == turn) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float4 v = make_float4(acc[x][0][i], acc[x][1][i], acc[x][2][i], acc[x][3][i]);
            float4& to = place(warp % kSums, x, i);
            if (turn < kTurns - 1) {
              const float4 u = to;
              v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
            to = v;
          }
      }
      __syncthreads();
    }
    for (int i = tid; i < nh * kPassDims; i += kThreads) {
      const int h = i / kPassDims, x = i % kPassDims;
      if (d0 + x >= a.v_dim) continue;
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kSums; ++w) o += part[(w * kTileHeads + h) * kPassDims + x];
      store_elem(a.out, ((long long)b * a.heads + h0 + h) * a.v_dim + d0 + x, 0, o * inv_s[h]);
    }
    __syncthreads();
  }
}

constexpr size_t rows_smem(int slots, int k_dim, int threads) {
  const size_t rounded = size_t(slots + kTileSlots - 1) / kTileSlots * kTileSlots;
  const size_t q = size_t(kTileHeads) * q_stride(k_dim), sums = size_t(sums_of(threads)) * kTileHeads * kPassDims * sizeof(float);
  return rounded * 16 + size_t(kTileHeads) * p_stride(slots) * sizeof(float) + (q > sums ? q : sums);
}

constexpr int kWThreads = 128, kWSlots = kWThreads / 32 * kTileSlots;

__global__ void __launch_bounds__(kWThreads) weights_rows_kernel(const AttnWeightsArgs a) {
  extern __shared__ __align__(16) uint8_t sq[];            // [kTileHeads][q_stride]
  const int b = blockIdx.y, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int j0 = blockIdx.x * kWSlots + (threadIdx.x >> 5) * kTileSlots;
  pdl_wait();
  const bool live = a.live == nullptr || a.live[b] != 0;
  const uint8_t* row[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int j = j0 + 8 * x + g;
    int e = live && j < a.topk ? a.idx[(long long)b * a.topk + j] : -1;
    if (e >= a.n_entries) {
      if (t == 0) report(a.err, kErrBadIndex, e);
      e = -1;
    }
    row[x] = e < 0 ? nullptr
                   : static_cast<const uint8_t*>(a.k_main) + ((long long)(b / a.seq_div) * a.n_entries + e) * a.k_dim * 2;
  }
  bool key[2][2];                                          // keys 8 x + 2 t and 8 x + 2 t + 1
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < 2; ++i) key[x][i] = __shfl_sync(0xffffffffu, int(row[x] != nullptr), 4 * (2 * t + i)) != 0;
  float w[2][2] = {};
  for (int h0 = 0; live && h0 < a.heads; h0 += kTileHeads) {
    const int nh = min(kTileHeads, a.heads - h0);
    __syncthreads();
    stage_q(sq, static_cast<const __nv_bfloat16*>(a.q) + ((long long)b * a.heads + h0) * a.k_dim, nh, a.k_dim, kWThreads);
    float l[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) l[y] = g + 8 * y < nh ? a.lse[(long long)b * a.heads + h0 + g + 8 * y] : -INFINITY;
    __syncthreads();
    float c[2][4];
    score_rows(row, sq, a.k_dim, c);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (key[x][i & 1] && l[i >> 1] != -INFINITY) w[x][i & 1] += expf(c[x][i] * a.scale - l[i >> 1]);
  }
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) w[x][i] += __shfl_xor_sync(0xffffffffu, w[x][i], o);
      const int j = j0 + 8 * x + 2 * t + i;
      if (g == 0 && j < a.topk) a.weights[(long long)b * a.topk + j] = w[x][i];
    }
}

template <int kThreads>
cudaError_t launch_rows(const TreeArgs& a, int batch, cudaStream_t st) {
  const cudaError_t e = once_per_device(kSetupTreeRows + (kThreads == 512), [] {
    return cudaFuncSetAttribute(tree_rows_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                int(rows_smem(kMaxSlots, 1024, kThreads)));
  });
  if (e != cudaSuccess) return e;
  note_launch();
  return launch_pdl(tree_rows_kernel<kThreads>, dim3(unsigned((a.heads + kTileHeads - 1) / kTileHeads), unsigned(batch)),
                    dim3(kThreads), rows_smem(a.topk + a.swa, a.k_dim, kThreads), st, 1, a);
}

// Rows that are whole 8-byte pieces at 8-byte addresses.
template <class... P>
bool pieces(int dim, P... p) {
  uintptr_t at = 0;
  for (const void* x : {static_cast<const void*>(p)...}) at |= reinterpret_cast<uintptr_t>(x);
  return dim % 4 == 0 && at % 8 == 0;
}

}  // namespace

bool tree_rows_fit(const TreeArgs& a) {
  return a.dtype == 0 && pieces(a.k_dim, a.q, a.k_main, a.k_swa, a.k_draft) && pieces(a.v_dim, a.v_main, a.v_swa, a.v_draft);
}

bool weights_rows_fit(const AttnWeightsArgs& a) { return a.dtype == 0 && pieces(a.k_dim, a.q, a.k_main); }

// 16 warps and one CTA an SM while there are no more CTAs than SMs, 8 warps and up to three beyond (tree.cu has both measured).
cudaError_t launch_tree_rows(const TreeArgs& a, int batch, cudaStream_t st) {
  const bool few = (long long)batch * ((a.heads + kTileHeads - 1) / kTileHeads) <= device_sm_count();
  return few ? launch_rows<512>(a, batch, st) : launch_rows<256>(a, batch, st);
}

cudaError_t launch_weights_rows(const AttnWeightsArgs& a, int batch, cudaStream_t st) {
  note_launch();
  return launch_pdl(weights_rows_kernel, dim3(unsigned((a.topk + kWSlots - 1) / kWSlots), unsigned(batch)), dim3(kWThreads),
                    size_t(kTileHeads) * q_stride(a.k_dim), st, 1, a);
}

}  // namespace csa2
