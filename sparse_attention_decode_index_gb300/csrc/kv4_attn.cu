// Sparse attention over a packed main cache (kv4.cuh): for every query head h
//     o_h = softmax(scale * q_h [K_main[idx]; K_swa]^T) [V_main[idx]; V_swa]
// as in attn.cu, K_main and V_main being code * scale * 2^exp.  The powers of two
// are taken out of the rows: a main key's product is multiplied by 2^k_exp with
// the softmax scale, a main value's weight by 2^v_exp.
//
// Any head count, dims and element type, in fp32 (fp32 queries and windows, and bf16 ones that kv4_mma.cu does not take:
// odd dims or addresses): a CTA takes one head or four of a
// query.  Eight lanes go through a row together, a group of 16 dims each, so that a warp has
// four rows on their way, or eight (fp32, 228 CTAs: 103 -> 72 us; the rows' latency bounds it: two products an
// instruction gave 211 -> 201 us for 60 queries of 64 heads, whose 1.6 GFLOP take 21: entries are fetched and converted once
// for four heads, 16 times for 64); a lane multiplies its numbers with every head of the CTA.  Scores stay in
// shared memory; every warp sums the values of its own rows, and the warps' sums are added in order.
#include "kv4.cuh"
#include "tc.cuh"

namespace csa2 {

namespace {

// 16 numbers of dims d .. d + 15 (of dim), zeros behind: of a window row, or of a group's codes.
CSA2_DEV void window16(const void* rows, long long row, int d, int dim, int dtype, bool wide, float (&x)[16]) {
  if (wide) {                                  // (fp32)
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(rows) + row * dim + d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = p[i];
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = d + i < dim ? load_elem(rows, row * dim + d + i, dtype) : 0.f;
  }
}

CSA2_DEV void packed16(const uint8_t* entry, int group, int groups, float (&x)[16]) {
  const uint2 codes = *reinterpret_cast<const uint2*>(entry + 8 * group);
  const __half2 scale = __half2half2(kv4_scale(entry[8 * groups + group]));
  float v[8];
  kv4_eight(codes.x, scale, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = v[i];
  kv4_eight(codes.y, scale, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[8 + i] = v[i];
}

// kHeads heads of query blockIdx.y, kRows rows at a time for eight lanes.  Shared memory: q [kHeads][16 gk], weights [kHeads][slots], rows [slots], the warps'
// sums [kWarps][kHeads][128].
template <int kHeads, int kThreads, int kRows>
__global__ void __launch_bounds__(kThreads) kv4_attn_generic_kernel(const Kv4AttnArgs a) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) float sh[];
  __shared__ float red[2][kHeads][kWarps];
  const int b = blockIdx.y, h0 = blockIdx.x * kHeads, nh = min(kHeads, a.heads - h0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l8 = lane & 7, r4 = lane >> 3;
  const int gk = kv4_groups(a.k_dim), gv = kv4_groups(a.v_dim), groups = gk + gv, bytes = kv4_bytes(a.k_dim, a.v_dim);
  const int slots = a.topk + a.swa;
  float* sq = sh;                                          // [kHeads][16 * gk]
  float* sw = sq + kHeads * 16 * gk;                       // [kHeads][slots]
  float* part = sw + (kHeads * slots + 3) / 4 * 4;         // [kWarps][kHeads][128]
  int* row = reinterpret_cast<int*>(part + kWarps * kHeads * 128);   // [slots]: entry, window row, or -1
  pdl_wait();   // no early trigger: the next launch may read, before its own wait, what the one before this one writes
  const uint8_t* cache = a.kv + (long long)(b / a.seq_div) * a.n_entries * bytes;
  const int ns = a.swa == 0 ? 0 : clamp_count(a.n_swa[b], a.swa, blockIdx.x == 0 && tid == 0 ? a.err : nullptr);
  for (int i = tid; i < kHeads * 16 * gk; i += kThreads) {
    const int h = i / (16 * gk), d = i - h * 16 * gk;
    sq[i] = h < nh && d < a.k_dim ? load_elem(a.q, ((long long)b * a.heads + h0 + h) * a.k_dim + d, a.dtype) : 0.f;
  }
  for (int j = tid; j < slots; j += kThreads) {
    int e = -1;
    if (j < a.topk) {
      e = a.idx[(long long)b * a.topk + j];
      if (e >= a.n_entries) {
        if (blockIdx.x == 0) report(a.err, kErrBadIndex, e);
        e = -1;
      }
    } else if (j - a.topk < ns) {
      e = j - a.topk;
    }
    row[j] = e < 0 ? -1 : e;
    if (e >= 0) {
      if (j < a.topk) {
        const uint8_t* p = cache + (long long)e * bytes;
        for (int i = 0; i < bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" :: "l"(p + i));
        asm volatile("prefetch.global.L2 [%0];" :: "l"(p + bytes - 1));
      }
    }
  }
  __syncthreads();
  // Numbers of group g (of key and value) of slot j's row e; zeros when there is none.
  const auto numbers = [&](int j, int e, int g, float (&x)[16]) {
    if (e < 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
    } else if (j < a.topk) {
      packed16(cache + (long long)e * bytes, g, groups, x);
    } else if (g < gk) {
      window16(a.k_swa, (long long)b * a.swa + e, 16 * g, a.k_dim, a.dtype, a.wide != 0, x);
    } else {
      window16(a.v_swa, (long long)b * a.swa + e, 16 * (g - gk), a.v_dim, a.dtype, a.wide != 0, x);
    }
  };
  // ---- scores
  float top[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) top[h] = -INFINITY;
  for (int j0 = 4 * kRows * warp; j0 < slots; j0 += 4 * kRows * kWarps) {
    int e[kRows];
    float2 dots[kRows][kHeads];                // sums over even and odd dims
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int j = j0 + 4 * u + r4;
      e[u] = j < slots ? row[j] : -1;
#pragma unroll
      for (int h = 0; h < kHeads; ++h) dots[u][h] = make_float2(0.f, 0.f);
    }
    for (int g = l8; g < gk; g += 8) {
      float x[kRows][16];
#pragma unroll
      for (int u = 0; u < kRows; ++u) numbers(j0 + 4 * u + r4, e[u], g, x[u]);
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        const float4* q = reinterpret_cast<const float4*>(sq + (h * gk + g) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 y = q[i];
#pragma unroll
          for (int u = 0; u < kRows; ++u) {
            dots[u][h] = fma2(make_float2(x[u][4 * i], x[u][4 * i + 1]), make_float2(y.x, y.y), dots[u][h]);
            dots[u][h] = fma2(make_float2(x[u][4 * i + 2], x[u][4 * i + 3]), make_float2(y.z, y.w), dots[u][h]);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int j = j0 + 4 * u + r4;
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        float dot = dots[u][h].x + dots[u][h].y;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float s = e[u] >= 0 ? dot * (j < a.topk ? a.scale * a.k_up : a.scale) : -INFINITY;
        if (l8 == 0 && j < slots) sw[h * slots + j] = s;
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(top[h]) : "f"(s));   // a NaN score makes its head's output NaN
      }
    }
  }
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      const float s = __shfl_xor_sync(0xffffffffu, top[h], o);
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(top[h]) : "f"(s));
    }
    if (lane == 0) red[0][h][warp] = top[h];
  }
  __syncthreads();
  // ---- weights and their sums
  float sum[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    top[h] = red[0][h][0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top[h]) : "f"(red[0][h][w]));
    sum[h] = 0.f;
    const float base = top[h] == -INFINITY ? 0.f : top[h];
    for (int j = tid; j < slots; j += kThreads) {
      const float p = expf(sw[h * slots + j] - base);
      sum[h] += p;
      sw[h * slots + j] = j < a.topk ? p * a.v_up : p;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], o);
    if (lane == 0) red[1][h][warp] = sum[h];
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    sum[h] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum[h] += red[1][h][w];
  }
  // ---- values, 8 groups of 16 dims at a time
  for (int g0 = 0; g0 < gv; g0 += 8) {
    const int g = g0 + l8;
    float2 acc[kHeads][8];
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[h][i] = make_float2(0.f, 0.f);
    for (int j = 4 * kRows * warp + r4; g < gv && j < slots; j += 4 * kRows * kWarps) {
      float x[kRows][16];
#pragma unroll
      for (int u = 0; u < kRows; ++u) numbers(j + 4 * u, j + 4 * u < slots ? row[j + 4 * u] : -1, gk + g, x[u]);
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (j + 4 * u >= slots) continue;
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          const float p = sw[h * slots + j + 4 * u];
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[h][i] = fma2(make_float2(p, p), make_float2(x[u][2 * i], x[u][2 * i + 1]), acc[h][i]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float o = i & 1 ? acc[h][i >> 1].y : acc[h][i >> 1].x;
        o += __shfl_xor_sync(0xffffffffu, o, 8);
        o += __shfl_xor_sync(0xffffffffu, o, 16);
        if (r4 == 0) part[(warp * kHeads + h) * 128 + 16 * l8 + i] = o;
      }
    __syncthreads();
    const int n = min(128, a.v_dim - 16 * g0);
    for (int i = tid; i < nh * n; i += kThreads) {
      const int h = i / n, d = i - h * n;
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) o += part[(w * kHeads + h) * 128 + d];
      float total = sum[0];
#pragma unroll
      for (int x = 1; x < kHeads; ++x) total = x == h ? sum[x] : total;
      store_elem(a.out, ((long long)b * a.heads + h0 + h) * a.v_dim + 16 * g0 + d, a.dtype, total == 0.f ? 0.f : o / total);
    }
    __syncthreads();
  }
  if (a.lse != nullptr && tid < nh) {
    float s = sum[0], t = top[0];
#pragma unroll
    for (int x = 1; x < kHeads; ++x) {
      s = x == tid ? sum[x] : s;
      t = x == tid ? top[x] : t;
    }
    a.lse[(long long)b * a.heads + h0 + tid] = s == 0.f ? -INFINITY : t + logf(s);
  }
}

template <int kHeads, int kThreads, int kRows>
cudaError_t launch_generic(const Kv4AttnArgs& a, int batch, cudaStream_t st) {
  const auto kernel = kv4_attn_generic_kernel<kHeads, kThreads, kRows>;
  const int slots = a.topk + a.swa, sums = kThreads / 32 * kHeads * 128;
  const size_t smem = (size_t(kHeads) * 16 * kv4_groups(a.k_dim) + (kHeads * slots + 3) / 4 * 4 + sums + slots) * 4;
  const cudaError_t e = once_per_device(kHeads == 1 ? kSetupKv4One : kThreads == 512 ? kSetupKv4Four : kSetupKv4Full, [] {
    return cudaFuncSetAttribute(kv4_attn_generic_kernel<kHeads, kThreads, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 << 10);
  });
  if (e != cudaSuccess) return e;
  note_launch();
  return launch_pdl(kernel, dim3(unsigned((a.heads + kHeads - 1) / kHeads), unsigned(batch)), dim3(kThreads), smem, st, 1, a);
}

}  // namespace

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, bool fast, int batch, cudaStream_t st) {
  if (batch == 0) return cudaSuccess;
  if (fast) return launch_kv4_attn_tc(a, batch, st);
  if (kv4_mma_fits(a)) return launch_kv4_attn_mma(a, batch, st);
  // Few heads are spread over CTAs of one each; warps that share a query's rows hide their latency while every CTA has
  // an SM to itself; otherwise more CTAs on an SM do.  Measured (queries of 8 heads, 562 keys, 192 / 128, fp32):
  //   CTAs of        1 head, 16 warps   4 heads, 16 warps   4 heads, 8 warps
  //   8 heads        22.5 us            34.7                38.8
  //   304 heads      32.7               34.7                38.9
  //   608 heads      57.3               34.7                38.9
  //   912 heads      83.9               63.4                55.3
  const int sms = device_sm_count();
  if (batch * (long long)a.heads <= 2LL * sms) return launch_generic<1, 512, 1>(a, batch, st);
  if ((a.heads + 3) / 4 * (long long)batch <= sms) return launch_generic<4, 512, 2>(a, batch, st);
  return launch_generic<4, 256, 2>(a, batch, st);
}

}  // namespace csa2
