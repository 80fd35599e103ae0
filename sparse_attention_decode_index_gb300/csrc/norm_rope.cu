// The norm of every head of several tensors (queries, keys, indexer queries, ...) and the
// rotary positions of rope.cu, in one pass over them:
//     y = x / sqrt(mean(x^2) + eps) * gain               (root mean square)
//     y = (x - mean(x)) / sqrt(var(x) + eps) * gain      (layer norm)
//     (a, b) -> mag (a cos t - b sin t, b cos t + a sin t),  t = pos * freq, for the pairs of the turned dims.
// Everything between the load and the one rounding of the store is fp32; the
// variance is taken about the mean in a second pass over registers.
//
// Memory bound: every element is read once and written once.  The rows of a block
// share their angles, as in rope.cu.  A head belongs to a group of 1 to 32 lanes
// that hold up to 4 vectors of it each (192 bf16 dims: 8 lanes with 3 vectors of
// 16 bytes), chosen so that few lanes are left over; its sums go through log2(lanes)
// shuffles.  In the half layout a turned vector's partner is loaded a second time
// (from L1), so that no lane waits for another's numbers.
#include "common.cuh"
#include "kv4.h"
#include "rope.cuh"

namespace csa2 {

namespace {

constexpr int kThreads = kRopeThreads;
constexpr int kMaxVecs = 4;       // of a lane

CSA2_DEV float sum_lanes(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <bool kBf16, int kBytes>
CSA2_DEV void unpack(const Vec<kBytes>& v, float (&f)[kBytes / (kBf16 ? 2 : 4)]) {
#pragma unroll
  for (int i = 0; i < kBytes / 4; ++i) {
    if constexpr (kBf16) {
      f[2 * i] = __uint_as_float(v.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(v.w[i] & 0xffff0000u);
    } else {
      f[i] = __uint_as_float(v.w[i]);
    }
  }
}

template <int kN>
CSA2_DEV void load_gain(const float* g, float (&f)[kN]) {
  if constexpr (kN == 2) {
    const float2 v = *reinterpret_cast<const float2*>(g);
    f[0] = v.x, f[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < kN / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(g)[i];
      f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
    }
  }
}

// One block's heads [h0, h0 + nh) of rows row0 .. row0 + nr - 1 of one tensor.
struct Part {
  int h0, nh, nr;
  long long row0;
  uint32_t m_head;
  CSA2_DEV Part(const NormRopeArgs::Slot& y, long long row0_, int nr_) : nr(nr_), row0(row0_) {
    h0 = int((long long)y.heads * blockIdx.y / gridDim.y);
    nh = int((long long)y.heads * (blockIdx.y + 1) / gridDim.y) - h0;
    m_head = nh <= 1 ? 0u : 0xffffffffu / uint32_t(nh) + 1u;
  }
  // Head i of the part (i < nr * nh <= 2^16): its row in the block and its number.
  CSA2_DEV void at(int i, int& row, int& head) const {
    row = fast_div(i, m_head);
    head = h0 + i - row * nh;
  }
};

template <bool kBf16, int kBytes, int kNv>
CSA2_DEV void norm_vectors(const NormRopeArgs& a, const NormRopeArgs::Slot& y, const Part& part, const float2* cs) {
  constexpr int kE = kBf16 ? 2 : 4, kV = kBytes / kE;
  const int lanes = y.lanes, l = threadIdx.x & (lanes - 1), n_vecs = y.dim / kV;
  const int half = a.rot / 2, v0 = y.off / kV, rv = a.rot / kV, hv = a.interleaved ? 0 : rv / 2;
  const int total = part.nr * part.nh, step = kThreads / lanes;
  const float inv_dim = 1.f / float(y.dim);
  for (int i0 = 0; i0 < total; i0 += step) {       // (uniform: the shuffles need whole warps)
    const int i = i0 + int(threadIdx.x) / lanes;
    const bool on = i < total;
    int row = 0, head = 0;
    if (on) part.at(i, row, head);
    const uint8_t* x = static_cast<const uint8_t*>(y.x) + ((part.row0 + row) * y.x_stride + (long long)head * y.dim) * kE;
    uint8_t* out = static_cast<uint8_t*>(y.out) + ((part.row0 + row) * y.out_stride + (long long)head * y.dim) * kE;
    const float* gain = y.gain == nullptr ? nullptr : y.gain + (y.gain_each ? (long long)head * y.dim : 0);
    Vec<kBytes> va[kNv], vb[kNv];
#pragma unroll
    for (int m = 0; m < kNv; ++m) {
      const int j = l + m * lanes, p = j - v0;      // p: place in the turned vectors
      if (on && j < n_vecs) {
        va[m].load(x + j * kBytes);
        if (hv > 0 && uint32_t(p) < uint32_t(rv)) vb[m].load(x + (p < hv ? j + hv : j - hv) * kBytes);
      } else {
#pragma unroll
        for (int e = 0; e < kBytes / 4; ++e) va[m].w[e] = 0u;
      }
    }
    float f[kNv][kV];
    float mean = 0.f, sum = 0.f;
#pragma unroll
    for (int m = 0; m < kNv; ++m) unpack<kBf16, kBytes>(va[m], f[m]);
    if (a.center) {
#pragma unroll
      for (int m = 0; m < kNv; ++m)
#pragma unroll
        for (int e = 0; e < kV; ++e) sum += f[m][e];   // (vectors that are not there hold zeros)
      mean = sum_lanes(sum, lanes) * inv_dim;
      sum = 0.f;
#pragma unroll
      for (int m = 0; m < kNv; ++m) {
        const bool there = l + m * lanes < n_vecs;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
          f[m][e] -= mean;
          if (there) sum = __fmaf_rn(f[m][e], f[m][e], sum);
        }
      }
    } else {
#pragma unroll
      for (int m = 0; m < kNv; ++m)
#pragma unroll
        for (int e = 0; e < kV; ++e) sum = __fmaf_rn(f[m][e], f[m][e], sum);
    }
    const float inv = __frsqrt_rn(__fmaf_rn(sum_lanes(sum, lanes), inv_dim, a.eps));
    __syncwarp();                                  // in place: every lane has loaded the head
    if (!on) continue;
#pragma unroll
    for (int m = 0; m < kNv; ++m) {
      const int j = l + m * lanes, p = j - v0;
      if (j >= n_vecs) continue;
      float g[kV], r[kV];
#pragma unroll
      for (int e = 0; e < kV; ++e) g[e] = 1.f;
      if (gain != nullptr) load_gain<kV>(gain + j * kV, g);
#pragma unroll
      for (int e = 0; e < kV; ++e) r[e] = f[m][e] * inv * g[e];
      if (uint32_t(p) < uint32_t(rv)) {
        const float2* c = cs + row * half;
        if (hv > 0) {
          const bool low = p < hv;
          float b[kV];
          unpack<kBf16, kBytes>(vb[m], b);
#pragma unroll
          for (int e = 0; e < kV; ++e) g[e] = 1.f;
          if (gain != nullptr) load_gain<kV>(gain + (low ? j + hv : j - hv) * kV, g);
          c += (low ? p : p - hv) * kV;
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            const float other = (b[e] - mean) * inv * g[e];
            const float2 t = c[e];
            r[e] = r[e] * t.x + (low ? -other : other) * t.y;
          }
        } else {
          c += p * (kV / 2);
#pragma unroll
          for (int e = 0; e < kV / 2; ++e) {
            const float2 t = c[e];
            const float u = r[2 * e], v = r[2 * e + 1];
            r[2 * e] = u * t.x - v * t.y;
            r[2 * e + 1] = v * t.x + u * t.y;
          }
        }
      }
      Vec<kBytes> w;
#pragma unroll
      for (int e = 0; e < kBytes / 4; ++e) {
        if constexpr (kBf16) w.w[e] = pack_bf16(r[2 * e], r[2 * e + 1]);
        else w.w[e] = __float_as_uint(r[e]);
      }
      w.store(out + j * kBytes);
    }
  }
}

template <bool kBf16, int kBytes>
CSA2_DEV void norm_wide(const NormRopeArgs& a, const NormRopeArgs::Slot& y, const Part& part, const float2* cs) {
  switch (y.vecs) {
    case 1: norm_vectors<kBf16, kBytes, 1>(a, y, part, cs); break;
    case 2: norm_vectors<kBf16, kBytes, 2>(a, y, part, cs); break;
    case 3: norm_vectors<kBf16, kBytes, 3>(a, y, part, cs); break;
    default: norm_vectors<kBf16, kBytes, 4>(a, y, part, cs); break;
  }
}

CSA2_DEV float get(const float* p, int i) { return p[i]; }
CSA2_DEV float get(const __nv_bfloat16* p, int i) { return __bfloat162float(p[i]); }
CSA2_DEV void put(float* p, int i, float v) { p[i] = v; }
CSA2_DEV void put(__nv_bfloat16* p, int i, float v) { p[i] = __float2bfloat16_rn(v); }

// Any size and alignment: a warp a head, which it goes through again for every sum and for the outputs (pairs, then
// the dims that are not turned, so that a lane alone reads what it writes in place).
template <typename T>
CSA2_DEV void norm_scalar(const NormRopeArgs& a, const NormRopeArgs::Slot& y, const Part& part, const float2* cs) {
  const int lane = threadIdx.x & 31, half = a.rot / 2, total = part.nr * part.nh;
  for (int i = threadIdx.x >> 5; i < total; i += kThreads / 32) {
    int row, head;
    part.at(i, row, head);
    const T* x = static_cast<const T*>(y.x) + (part.row0 + row) * y.x_stride + (long long)head * y.dim;
    T* out = static_cast<T*>(y.out) + (part.row0 + row) * y.out_stride + (long long)head * y.dim;
    const float* gain = y.gain == nullptr ? nullptr : y.gain + (y.gain_each ? (long long)head * y.dim : 0);
    float mean = 0.f, sum = 0.f;
    if (a.center) {
      for (int d = lane; d < y.dim; d += 32) sum += get(x, d);
      mean = sum_lanes(sum, 32) / float(y.dim);
      sum = 0.f;
    }
    for (int d = lane; d < y.dim; d += 32) {
      const float v = get(x, d) - mean;
      sum = __fmaf_rn(v, v, sum);
    }
    const float inv = __frsqrt_rn(sum_lanes(sum, 32) / float(y.dim) + a.eps);
    auto value = [&](int d) -> float { return (get(x, d) - mean) * inv * (gain != nullptr ? gain[d] : 1.f); };
    __syncwarp();
    for (int d = lane; d < y.dim - half; d += 32) {
      if (d < half) {
        const int u = y.off + (a.interleaved ? 2 * d : d), v = u + (a.interleaved ? 1 : half);
        const float2 t = cs[row * half + d];
        const float fu = value(u), fv = value(v);
        put(out, u, fu * t.x - fv * t.y);
        put(out, v, fv * t.x + fu * t.y);
      } else {
        const int c = d - half, at = c < y.off ? c : c + a.rot;
        put(out, at, value(at));
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 2) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  extern __shared__ __align__(16) float2 cs[];           // [per_block][rot / 2]
  __shared__ long long step[kMaxRopePairs];
  const long long row0 = (long long)blockIdx.x * a.per_block;
  const int nr = int(min((long long)a.per_block, a.rows - row0));
  pdl_wait();   // no early trigger: the attention may read what this kernel writes before its own wait
  if (a.rot > 0) rope_angles(cs, step, row0, nr, a.rot / 2, a.pos, a.freqs, a.mag, false);
  __syncthreads();
  for (int k = 0; k < a.n_slots; ++k) {
    const NormRopeArgs::Slot& y = a.slot[k];
    const Part part(y, row0, nr);
    const bool f32 = y.dtype == 1;
    if (y.bytes == 16) f32 ? norm_wide<false, 16>(a, y, part, cs) : norm_wide<true, 16>(a, y, part, cs);
    else if (y.bytes == 8) f32 ? norm_wide<false, 8>(a, y, part, cs) : norm_wide<true, 8>(a, y, part, cs);
    else f32 ? norm_scalar<float>(a, y, part, cs) : norm_scalar<__nv_bfloat16>(a, y, part, cs);
  }
}

// Vectors of 16 or 8 bytes that fit the tensor's sizes and addresses (0: none do), and the lanes of a head with the
// vectors of each that leave the fewest over (of those, the most lanes).
void choose_vectors(NormRopeArgs::Slot& y, int rot, bool interleaved) {
  const int e = y.dtype == 1 ? 4 : 2;
  y.bytes = 0;
  for (int w = 16; w >= 8; w /= 2) {
    const int v = w / e;
    const uintptr_t at = reinterpret_cast<uintptr_t>(y.x) | reinterpret_cast<uintptr_t>(y.out);
    const uintptr_t gains = y.gain != nullptr ? reinterpret_cast<uintptr_t>(y.gain) % (v >= 4 ? 16 : 8) : 0;
    if (at % w != 0 || gains != 0 || y.x_stride % v != 0 || y.out_stride % v != 0 || y.dim % v != 0) continue;
    if (rot > 0 && (y.off % v != 0 || rot % v != 0 || (!interleaved && rot / 2 % v != 0))) continue;
    const int n = y.dim / v;
    if (n > 32 * kMaxVecs) continue;
    int best = 1 << 30;
    for (int lanes = 32; lanes >= 1; lanes /= 2) {
      const int m = (n + lanes - 1) / lanes;
      if (m > kMaxVecs || m * lanes - n >= best) continue;
      best = m * lanes - n;
      y.lanes = lanes;
      y.vecs = m;
    }
    y.bytes = w;
    return;
  }
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeArgs& a, int rows, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  int heads = 0, vecs = 0;   // heads of the tensor with the most; 16-byte pieces of a row of all tensors
  for (int k = 0; k < a.n_slots; ++k) {
    NormRopeArgs::Slot& y = a.slot[k];
    choose_vectors(y, a.rot, a.interleaved != 0);
    heads = heads > y.heads ? heads : y.heads;
    vecs += (y.heads * y.dim * (y.dtype == 1 ? 4 : 2) + 15) / 16;
  }
  // Rows of a block and blocks of a row as in rope.cu.
  const int want = 4 * device_sm_count();
  int most = 64;
  while (most > 8 && (most * (a.rot / 2) > 8 * kMaxRopePairs || most * vecs > 4096)) --most;
  a.rows = rows;
  a.per_block = rows / want < 1 ? 1 : rows / want > most ? most : rows / want;
  const int blocks = (rows - 1) / a.per_block + 1;
  int split = blocks >= want ? 1 : (want + blocks - 1) / blocks;
  split = split > heads ? heads : split;
  note_launch();
  return launch_pdl(norm_rope_kernel, dim3(unsigned(blocks), unsigned(split)), dim3(kThreads),
                    size_t(a.per_block) * (a.rot / 2) * sizeof(float2), st, 1, a);
}

}  // namespace csa2
