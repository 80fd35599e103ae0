// Sparse attention over a packed main cache for bf16 shapes outside the fast path whose
// window rows are whole 8-byte pieces: products on mma.sync, operands straight from the
// gathered entries.  One CTA per (query, 16 heads), or a cluster of up to 8 that share its slots and join their sums through
// distributed shared memory.
//   S = Q K^T   a warp takes 16 slots at a time.  mma's B operand wants pairs of k of one key
//     per lane; a sum has no order, so lane t of a quad takes group 4 s + t of its key, 16 codes in one
//     8-byte load and their scale, for four products, and Q is read in the same order.  Code * scale is exact in bf16.
//   softmax     fp32, a warp per head, over all slots in shared memory.
//   O = P V     the slots go round the warps, 16 a step.  B wants the pairs along the slots: a lane takes eight
//     dims of its four slots (a word of codes each) and interleaves them, so that column g of product j is dim 8 g + j.
//     P is rounded to bf16 (half a step, 2^-8 of a weight; its sum is not rounded), which a factor of 2^v_exp for
//     entries does not change.  The warps' sums are added up in their order.
// Bound by latency, two round trips to memory per 16 slots of a warp, and the conversions: 90 queries, 40 heads of 192 / 128,
// 640 slots 32.3 us (fp32 products in kv4_attn.cu: 168), 20 queries of 16 heads 15.1 with distinct inputs in turn, 13.6 in calls from Python
// (without clusters 18.8), 1 query of 4 heads of
// 64 / 64 7.9 (10.6).  An entry is gathered and converted once for 16 heads, three times for 40.  Three CTAs an SM leave 80 registers a
// thread, which spills (51.1).
#include "kv4.cuh"

namespace csa2 {

namespace {

constexpr int kTileHeads = 16, kTileSlots = 16;
constexpr int kSpan = 64;           // dims of a step of scores: a group for each lane of a quad
constexpr int kPassDims = 64;       // dims of a P V pass
constexpr int kPassPitch = kPassDims + 4;
constexpr int kMaxSlots = 1024;     // topk + swa
constexpr int kMaxCluster = 8;

// Bytes of a staged Q row: 8 past a multiple of 128, so that the pieces that half a warp reads, 8 bytes of four rows and four
// groups, fall into distinct banks.
constexpr int q_stride(int k_dim) { return (k_dim + kSpan - 1) / kSpan * kSpan * 2 + 8; }
// Words of a head's logits: 8 past a multiple of 32, for the same reason.
constexpr int p_stride(int slots) { return (slots + 31) / 32 * 32 + 8; }
// Codes of a word times their scale as four bf16 pairs, exactly.
CSA2_DEV void bf16_eight(uint32_t codes, uint8_t scale, uint32_t (&w)[4]) {
  float v[8];
  kv4_eight(codes, __half2half2(kv4_scale(scale)), v);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
}

// A slot's numbers as they lie in memory, kWords * 2 of them: bf16 pairs of a window row, or codes and their scale.
template <int kWords>
struct RawDims {
  uint32_t w[kWords];
  uint32_t scale;
  CSA2_DEV void none() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
    scale = 0u;
  }
  CSA2_DEV void packed(const uint8_t* codes, const uint8_t* scale_at) {
    if constexpr (kWords == 8) {
      const uint2 y = *reinterpret_cast<const uint2*>(codes);
      w[0] = y.x, w[1] = y.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(codes);
    }
    scale = *scale_at;
  }
  CSA2_DEV void window(const __nv_bfloat16* row, int d, int dim) {   // from dim d on, zeros behind the last
#pragma unroll
    for (int i = 0; i < kWords; i += 2) {
      const uint2 y = d + 2 * i < dim ? *reinterpret_cast<const uint2*>(row + d + 2 * i) : make_uint2(0u, 0u);
      w[i] = y.x, w[i + 1] = y.y;
    }
  }
  CSA2_DEV void unpack() {                     // codes become pairs
    uint32_t y[4], z[4];
    bf16_eight(w[0], uint8_t(scale), y);
    if constexpr (kWords == 8) bf16_eight(w[1], uint8_t(scale), z);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = y[i];
      if constexpr (kWords == 8) w[4 + i] = z[i];
    }
  }
};

template <int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 2 : 1) kv4_mma_kernel(const Kv4AttnArgs a, int ncta) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ float inv_s[kTileHeads];
  __shared__ float2 total[kTileHeads];         // of a split: the greatest logit and the sum of this CTA's slots
  const int crank = ncta > 1 ? int(cluster_rank()) : 0, tile = int(blockIdx.x) / ncta;
  const int b = blockIdx.y, h0 = tile * kTileHeads, nh = min(kTileHeads, a.heads - h0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int gk = kv4_groups(a.k_dim), gv = kv4_groups(a.v_dim), groups = gk + gv, bytes = kv4_bytes(a.k_dim, a.v_dim);
  const int nslots = a.topk + a.swa, rounded = (nslots + kTileSlots - 1) / kTileSlots * kTileSlots;
  const int ld = p_stride(nslots), stride = q_stride(a.k_dim), spans = (a.k_dim + kSpan - 1) / kSpan;
  const int lo = rounded / kTileSlots * crank / ncta * kTileSlots, hi = rounded / kTileSlots * (crank + 1) / ncta * kTileSlots;   // this CTA's slots
  int* row = reinterpret_cast<int*>(sm);                          // [rounded] entry or window row, or -1
  float* sp = reinterpret_cast<float*>(row + rounded);            // [kTileHeads][ld] logits -> weights
  uint8_t* sq = reinterpret_cast<uint8_t*>(sp + kTileHeads * ld); // [kTileHeads][q_stride]
  float* part = reinterpret_cast<float*>(sq);                     // later: [kWarps][kTileHeads][kPassPitch]
  float* mine = part + max(kTileHeads * stride / 4, kWarps * kTileHeads * kPassPitch);   // of a split: [kTileHeads][v_dim]
  pdl_wait();   // no early trigger: the next launch may read, before its own wait, what the one before this one writes
  for (int i = tid; i < kTileHeads * spans * kSpan; i += kThreads) {
    const int h = i / (spans * kSpan), d = i - h * (spans * kSpan);
    const bool in = h < nh && d < a.k_dim;
    reinterpret_cast<__nv_bfloat16*>(sq + h * stride)[d] =
        in ? static_cast<const __nv_bfloat16*>(a.q)[((long long)b * a.heads + h0 + h) * a.k_dim + d] : __nv_bfloat16(0.f);
  }
  const int ns = a.swa == 0 ? 0 : clamp_count(a.n_swa[b], a.swa, tile == 0 && crank == 0 && tid == 0 ? a.err : nullptr);
  for (int j = lo + tid; j < hi; j += kThreads) {
    int e = -1;
    if (j < a.topk) {
      e = a.idx[(long long)b * a.topk + j];
      if (e >= a.n_entries) {
        if (tile == 0) report(a.err, kErrBadIndex, e);
        e = -1;
      }
    } else if (j - a.topk < ns) {
      e = j - a.topk;
    }
    row[j] = e < 0 ? -1 : e;
  }
  __syncthreads();
  const uint8_t* cache = a.kv + (long long)(b / a.seq_div) * a.n_entries * bytes;
  const __nv_bfloat16* k_swa = static_cast<const __nv_bfloat16*>(a.k_swa) + (long long)b * a.swa * a.k_dim;
  const __nv_bfloat16* v_swa = static_cast<const __nv_bfloat16*>(a.v_swa) + (long long)b * a.swa * a.v_dim;
  // ---- scores
  for (int j = lo + kTileSlots * warp; j < hi; j += kTileSlots * kWarps) {
    constexpr int kBatch = 2;                  // steps whose loads are on their way together
    int e[2];
    float c[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      e[x] = row[j + 8 * x + g];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[x][i] = 0.f;
    }
    for (int s0 = 0; s0 < spans; s0 += kBatch) {
      RawDims<8> k[kBatch][2];
#pragma unroll
      for (int y = 0; y < kBatch; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int group = 4 * (s0 + y) + t;
          if (e[x] < 0 || group >= gk) {
            k[y][x].none();
          } else if (j + 8 * x + g < a.topk) {
            const uint8_t* entry = cache + (long long)e[x] * bytes;
            k[y][x].packed(entry + 8 * group, entry + 8 * groups + group);
          } else {
            k[y][x].window(k_swa + (long long)e[x] * a.k_dim, 16 * group, a.k_dim);
          }
        }
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        if (s0 + y >= spans) break;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (j + 8 * x + g < a.topk) k[y][x].unpack();
        __syncwarp();
        const uint8_t* qa = sq + g * stride + 2 * kSpan * (s0 + y) + 32 * t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2 lo = *reinterpret_cast<const uint2*>(qa + 8 * i), hi = *reinterpret_cast<const uint2*>(qa + 8 * stride + 8 * i);
#pragma unroll
          for (int x = 0; x < 2; ++x) mma_bf16(c[x], lo.x, hi.x, lo.y, hi.y, k[y][x].w[2 * i], k[y][x].w[2 * i + 1]);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {              // c[x][0, 1]: head g and slots at, at + 1; c[x][2, 3]: head g + 8
      const int at = j + 8 * x + 2 * t;
      const float s0 = at < a.topk ? a.scale * a.k_up : a.scale, s1 = at + 1 < a.topk ? a.scale * a.k_up : a.scale;
      const bool key0 = row[at] >= 0, key1 = row[at + 1] >= 0;
#pragma unroll
      for (int y = 0; y < 2; ++y)
        *reinterpret_cast<float2*>(sp + (g + 8 * y) * ld + at) =
            make_float2(key0 ? c[x][2 * y] * s0 : -INFINITY, key1 ? c[x][2 * y + 1] * s1 : -INFINITY);
    }
  }
  __syncthreads();
  // ---- weights and their sums
  for (int h = warp; h < kTileHeads; h += kWarps) {
    float* p = sp + h * ld;
    float m = -INFINITY, l = 0.f;
    for (int j = lo + lane; j < hi; j += 32) m = fmaxf(m, p[j]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    for (int j = lo + lane; j < hi; j += 32) {
      const float w = expf(p[j] - base);       // (NaN of a NaN or an infinite logit, as the sum then is)
      p[j] = j < a.topk ? w * a.v_up : w;
      l += w;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      inv_s[h] = ncta > 1 ? 1.f : l > 0.f ? 1.f / l : l;   // no key: 0; NaN stays NaN
      total[h] = make_float2(m, l);
      if (ncta == 1 && h < nh && a.lse != nullptr) a.lse[(long long)b * a.heads + h0 + h] = l == 0.f ? -INFINITY : base + logf(l);
    }
  }
  __syncthreads();
  // ---- values
  for (int d0 = 0; d0 < a.v_dim; d0 += kPassDims) {
    constexpr int kBatch = 2;
    float acc[8][4];
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i >> 2][i & 3] = 0.f;
    const int group = (d0 >> 4) + (g >> 1);
    for (int j0 = lo + kTileSlots * warp; j0 < hi; j0 += kBatch * kTileSlots * kWarps) {
      RawDims<4> v[kBatch][4];
#pragma unroll
      for (int y = 0; y < kBatch; ++y)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = j0 + y * kTileSlots * kWarps + 2 * t + (r & 1) + 4 * (r & 2);
          const int e = j < hi && group < gv ? row[j] : -1;
          if (e < 0) {
            v[y][r].none();
          } else if (j < a.topk) {
            const uint8_t* entry = cache + (long long)e * bytes;
            v[y][r].packed(entry + 8 * (gk + group) + 4 * (g & 1), entry + 8 * groups + gk + group);
          } else {
            v[y][r].window(v_swa + (long long)e * a.v_dim, d0 + 8 * g, a.v_dim);
          }
        }
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        const int j = j0 + y * kTileSlots * kWarps;
        if (j >= hi) break;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (j + 2 * t + (r & 1) + 4 * (r & 2) < a.topk) v[y][r].unpack();
        __syncwarp();
        const float* pa = sp + g * ld + j + 2 * t;
        const float* pb = pa + 8 * ld;
        auto pair = [](const float* p) -> uint32_t {
          const float2 w = *reinterpret_cast<const float2*>(p);
          return pack_bf16(w.x, w.y);
        };
        const uint32_t a0 = pair(pa), a1 = pair(pb), a2 = pair(pa + 8), a3 = pair(pb + 8);
        const RawDims<4>(&w)[4] = v[y];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mma_bf16(acc[2 * i], a0, a1, a2, a3, __byte_perm(w[0].w[i], w[1].w[i], 0x5410), __byte_perm(w[2].w[i], w[3].w[i], 0x5410));
          mma_bf16(acc[2 * i + 1], a0, a1, a2, a3, __byte_perm(w[0].w[i], w[1].w[i], 0x7632), __byte_perm(w[2].w[i], w[3].w[i], 0x7632));
        }
      }
    }
    // Columns 2 t and 2 t + 1 of product j are dims 16 t + j and 16 t + 8 + j; acc[j][2, 3] belong to head g + 8.
#pragma unroll
    for (int i = 0; i < 8; ++i) {              // head g + 8 (i >> 2), dims 16 t + 8 ((i >> 1) & 1) + 4 (i & 1) .. + 3
      const int y = 2 * (i >> 2) + ((i >> 1) & 1), q = 4 * (i & 1);
      *reinterpret_cast<float4*>(part + (warp * kTileHeads + g + 8 * (i >> 2)) * kPassPitch + 16 * t + 8 * ((i >> 1) & 1) + q) =
          make_float4(acc[q][y], acc[q + 1][y], acc[q + 2][y], acc[q + 3][y]);
    }
    __syncthreads();
    for (int i = tid; i < nh * kPassDims; i += kThreads) {
      const int h = i / kPassDims, x = i % kPassDims;
      if (d0 + x >= a.v_dim) continue;
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) o += part[(w * kTileHeads + h) * kPassPitch + x];
      if (ncta > 1) mine[h * a.v_dim + d0 + x] = o;
      else store_elem(a.out, ((long long)b * a.heads + h0 + h) * a.v_dim + d0 + x, 0, o * inv_s[h]);
    }
    __syncthreads();
  }
  if (ncta == 1) return;
  // ---- a split's parts, a share of the heads a CTA
  cluster_sync_all();
  const int per = kTileHeads / ncta, pieces = a.v_dim / 4;
  for (int i = tid; i < per * pieces; i += kThreads) {
    const int h = crank * per + i / pieces, d = i % pieces * 4;
    if (h >= nh) break;
    float top = -INFINITY, sum = 0.f;
    float2 y[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < ncta) {
        y[c] = make_float2(dsmem_ld_f32(dsmem_addr(&total[h].x, uint32_t(c))), dsmem_ld_f32(dsmem_addr(&total[h].y, uint32_t(c))));
        top = fmaxf(top, y[c].x);
      }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < ncta) {
        const float w = y[c].x == -INFINITY ? 0.f : expf(y[c].x - top);   // (a NaN sum stays)
        const float4 z = dsmem_ld_v4f(dsmem_addr(mine + h * a.v_dim + d, uint32_t(c)));
        sum += w * y[c].y;
        o = make_float4(__fmaf_rn(w, z.x, o.x), __fmaf_rn(w, z.y, o.y), __fmaf_rn(w, z.z, o.z), __fmaf_rn(w, z.w, o.w));
      }
    const float inv = sum > 0.f ? 1.f / sum : sum;
    const long long at = (long long)b * a.heads + h0 + h;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + at * a.v_dim + d;   // (of any address)
    out[0] = __float2bfloat16_rn(o.x * inv);
    out[1] = __float2bfloat16_rn(o.y * inv);
    out[2] = __float2bfloat16_rn(o.z * inv);
    out[3] = __float2bfloat16_rn(o.w * inv);
    if (d == 0 && a.lse != nullptr) a.lse[at] = sum == 0.f ? -INFINITY : (top == -INFINITY ? 0.f : top) + logf(sum);
  }
  cluster_sync_all();                          // every peer has read this CTA's part
}

constexpr size_t smem_of(int slots, int k_dim, int threads, int split_dims) {
  const size_t rounded = size_t(slots + kTileSlots - 1) / kTileSlots * kTileSlots;
  const size_t q = size_t(kTileHeads) * q_stride(k_dim), sums = size_t(threads / 32) * kTileHeads * kPassPitch * sizeof(float);
  return rounded * sizeof(int) + size_t(kTileHeads) * p_stride(slots) * sizeof(float) + (q > sums ? q : sums) +
         size_t(kTileHeads) * split_dims * sizeof(float);
}

template <int kThreads>
cudaError_t launch(const Kv4AttnArgs& a, int batch, int ncta, cudaStream_t st) {
  const cudaError_t e = once_per_device(kThreads == 512 ? kSetupKv4Mma16 : kSetupKv4Mma8, [] {
    return cudaFuncSetAttribute(kv4_mma_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem_of(kMaxSlots, 1024, kThreads, 1024)));
  });
  if (e != cudaSuccess) return e;
  note_launch();
  return launch_pdl(kv4_mma_kernel<kThreads>, dim3(unsigned((a.heads + kTileHeads - 1) / kTileHeads * ncta), unsigned(batch)), dim3(kThreads),
                    smem_of(a.topk + a.swa, a.k_dim, kThreads, ncta > 1 ? a.v_dim : 0), st, unsigned(ncta), a, ncta);
}

}  // namespace

// Window rows that are whole 8-byte pieces at 8-byte addresses.
bool kv4_mma_fits(const Kv4AttnArgs& a) {
  return a.dtype == 0 && a.k_dim % 4 == 0 && a.v_dim % 4 == 0 &&
         ((reinterpret_cast<uintptr_t>(a.k_swa) | reinterpret_cast<uintptr_t>(a.v_swa)) & 7) == 0;
}

// Clusters of 8 warps a CTA while they all fit the SMs and a CTA has 64 slots; else 16 warps and one CTA an SM while there are no more
// CTAs than SMs, 8 warps and two CTAs beyond.  Measured, 640 slots: 8 queries of 16 heads of 192 / 128 in clusters of 8 11.9 us, of 4 13.4, alone
// 18.9; 96 of 16 heads, 828 slots, 16 warps 26.6, 8 warps 34.5; 90 of 40 heads 39.6 and 32.7.
cudaError_t launch_kv4_attn_mma(const Kv4AttnArgs& a, int batch, cudaStream_t st) {
  const int sms = device_sm_count();
  const long long ctas = (long long)batch * ((a.heads + kTileHeads - 1) / kTileHeads);
  int ncta = 1;
  while (ncta < kMaxCluster && 2 * ncta * ctas <= sms && 2 * ncta * 64 <= a.topk + a.swa) ncta *= 2;
  return ncta > 1 ? launch<256>(a, batch, ncta, st) : ctas <= sms ? launch<512>(a, batch, 1, st) : launch<256>(a, batch, 1, st);
}

}  // namespace csa2
