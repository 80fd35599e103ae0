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
// shuffles.  The next head is on its way while one is turned, the first while the angles are made (8 rows 6.1 -> 6.0 us),
// and gains stay in registers while the head does.
//
// Measured: 8 rows 6.0 us; 8,192 rows of 64 + 1 heads of 192 in bf16 72.6 us, 5.6 TB/s (62 % of DRAM's cycles, issue
// slots 64 %: the next load waits for the shuffles' turn), in fp32 129.8, 6.3 TB/s; 4,097 rows of 16 + 1 heads of 128 in fp32, layer
// norm with gains of each head, 22.1 us, 3.2 TB/s, root mean square 20.4 (no unit is busy: issue slots 64 %, DRAM 18 %, warps 35 %;
// sums' shuffles one behind the other).  Four blocks an SM leave too few registers (124 us),
// four vectors a lane for fp32 too few lanes (30 us).
#include "common.cuh"
#include "kv4.h"
#include "rope.cuh"

namespace csa2 {

namespace {

constexpr int kThreads = kRopeThreads;
constexpr int kMaxVecs = 4;       // of a lane
constexpr int kPerSm = 3;         // blocks

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

// Where the partner of a turned vector of the half layout is: nowhere (interleaved pairs, or none at all), in the same lane
// `hv / lanes` vectors further, in lane l ^ hv, or anywhere (it is loaded a second time).
enum Partner { kNoPartner, kSameLane, kOtherLane, kLoaded };

template <bool kBf16, int kBytes, int kNv, int kPartner, class F>
CSA2_DEV void norm_vectors(const NormRopeArgs& a, const NormRopeArgs::Slot& y, const Part& part, const float2* cs, F meanwhile) {
  constexpr int kE = kBf16 ? 2 : 4, kV = kBytes / kE;
  const int lanes = y.lanes, l = threadIdx.x & (lanes - 1), n_vecs = y.dim / kV;
  const int half = a.rot / 2, v0 = y.off / kV, rv = a.rot / kV, hv = rv / 2;
  const int total = part.nr * part.nh, step = kThreads / lanes;
  const float inv_dim = 1.f / float(y.dim);
  const bool each = y.gain_each != 0;
  // gains that all heads share stay in registers: a lane's vectors have the same place in every head
  float g[kNv][kV];
  auto load_gains = [&](const float* gain) {
#pragma unroll
    for (int m = 0; m < kNv; ++m) {
#pragma unroll
      for (int e = 0; e < kV; ++e) g[m][e] = 1.f;
      if (gain != nullptr && l + m * lanes < n_vecs) load_gain<kV>(gain + (l + m * lanes) * kV, g[m]);
    }
  };
  int have = -1;                                   // whose gains these are, where heads have their own
  if (!each) load_gains(y.gain);
  auto address = [&](int i, long long stride) -> long long {   // of head i of the part, in bytes
    int row, head;
    part.at(i, row, head);
    return ((part.row0 + row) * stride + (long long)head * y.dim) * kE;
  };
  Vec<kBytes> next[kNv];                           // the next head, on its way while this one is turned
  auto fetch = [&](int i) {
    const uint8_t* x = static_cast<const uint8_t*>(y.x) + (i < total ? address(i, y.x_stride) : 0);
#pragma unroll
    for (int m = 0; m < kNv; ++m) {
      const int j = l + m * lanes;
      if (i < total && j < n_vecs) {
        next[m].load(x + j * kBytes);
      } else {
#pragma unroll
        for (int e = 0; e < kBytes / 4; ++e) next[m].w[e] = 0u;
      }
    }
  };
  const int first = int(threadIdx.x) / lanes;
  fetch(first);
  meanwhile();                                     // what the first head's way leaves time for
  for (int i0 = 0; i0 < total; i0 += step) {       // (uniform: the shuffles need whole warps)
    const int i = i0 + first;
    const bool on = i < total;
    float f[kNv][kV];
    Vec<kBytes> vb[kPartner == kLoaded ? kNv : 1];
#pragma unroll
    for (int m = 0; m < kNv; ++m) unpack<kBf16, kBytes>(next[m], f[m]);
    if constexpr (kPartner == kLoaded) {
      const uint8_t* x = static_cast<const uint8_t*>(y.x) + (on ? address(i, y.x_stride) : 0);
#pragma unroll
      for (int m = 0; m < kNv; ++m) {
        const int j = l + m * lanes, p = j - v0;
        if (on && j < n_vecs && uint32_t(p) < uint32_t(rv)) vb[m].load(x + (p < hv ? j + hv : j - hv) * kBytes);
      }
    }
    fetch(i + step);
    float mean = 0.f, sum = 0.f;
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
    int row = 0, head = 0;
    if (on) part.at(i, row, head);
    const float* gain = y.gain == nullptr || !each ? y.gain : y.gain + (long long)head * y.dim;
    if (each && head != have) {                    // (a group meets the same heads in turn: one, where step is a multiple of them)
      load_gains(gain);
      have = head;
    }
#pragma unroll
    for (int m = 0; m < kNv; ++m)
#pragma unroll
      for (int e = 0; e < kV; ++e) f[m][e] = f[m][e] * inv * g[m][e];
    uint8_t* out = static_cast<uint8_t*>(y.out) + (on ? address(i, y.out_stride) : 0);
    const float2* c = cs + row * half;
    float r[kNv][kV];
#pragma unroll
    for (int m = 0; m < kNv; ++m) {
      const int j = l + m * lanes, p = j - v0;      // p: place in the turned vectors
      const bool turned = uint32_t(p) < uint32_t(rv);
#pragma unroll
      for (int e = 0; e < kV; ++e) r[m][e] = f[m][e];
      if constexpr (kPartner == kNoPartner) {
        if (turned) {
          const float2* t = c + p * (kV / 2);
#pragma unroll
          for (int e = 0; e < kV / 2; ++e) {
            const float2 z = t[e];
            r[m][2 * e] = f[m][2 * e] * z.x - f[m][2 * e + 1] * z.y;
            r[m][2 * e + 1] = f[m][2 * e + 1] * z.x + f[m][2 * e] * z.y;
          }
        }
      } else {
        const bool low = p < hv;
        float b[kV];
        if constexpr (kPartner == kSameLane) {
          const int to = low ? m + hv / lanes : m - hv / lanes;
#pragma unroll
          for (int k = 0; k < kNv; ++k)
            if (k == to) {
#pragma unroll
              for (int e = 0; e < kV; ++e) b[e] = f[k][e];
            }
        } else if constexpr (kPartner == kOtherLane) {
          // (whole warps: a vector is turned in all lanes or, of a narrow range, in some; the others' numbers are not used)
#pragma unroll
          for (int e = 0; e < kV; ++e) b[e] = __shfl_xor_sync(0xffffffffu, f[m][e], hv);
        } else if (turned) {
          unpack<kBf16, kBytes>(vb[m], b);
          float gb[kV];
#pragma unroll
          for (int e = 0; e < kV; ++e) gb[e] = 1.f;
          if (gain != nullptr) load_gain<kV>(gain + (low ? j + hv : j - hv) * kV, gb);
#pragma unroll
          for (int e = 0; e < kV; ++e) b[e] = (b[e] - mean) * inv * gb[e];
        }
        if (turned) {
          const float2* t = c + (low ? p : p - hv) * kV;
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            const float2 z = t[e];
            r[m][e] = f[m][e] * z.x + (low ? -b[e] : b[e]) * z.y;
          }
        }
      }
    }
    if (!on) continue;
#pragma unroll
    for (int m = 0; m < kNv; ++m) {
      const int j = l + m * lanes;
      if (j >= n_vecs) continue;
      Vec<kBytes> w;
#pragma unroll
      for (int e = 0; e < kBytes / 4; ++e) {
        if constexpr (kBf16) w.w[e] = pack_bf16(r[m][2 * e], r[m][2 * e + 1]);
        else w.w[e] = __float_as_uint(r[m][e]);
      }
      w.store(out + j * kBytes);
    }
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

// The tensors of a launch that are alike: one element type, one vector size (0: number by number), one place of partners.
template <bool kBf16, int kBytes, int kNv, int kPartner>
__global__ void __launch_bounds__(kThreads, kNv == 4 ? 2 : kPerSm) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  extern __shared__ __align__(16) float2 cs[];           // [per_block][rot / 2]
  __shared__ long long step[kMaxRopePairs];
  const long long row0 = (long long)blockIdx.x * a.per_block;
  const int nr = int(min((long long)a.per_block, a.rows - row0));
  pdl_wait();   // no early trigger: the attention may read what this kernel writes before its own wait
  auto angles = [&] {
    if (a.rot > 0) rope_angles(cs, step, row0, nr, a.rot / 2, a.pos, a.freqs, a.mag, false);
    __syncthreads();
  };
  if constexpr (kBytes == 0) angles();
  for (int k = 0; k < a.n_slots; ++k) {
    const NormRopeArgs::Slot& y = a.slot[k];
    const Part part(y, row0, nr);
    if constexpr (kBytes == 0) {
      if (kBf16) norm_scalar<__nv_bfloat16>(a, y, part, cs);
      else norm_scalar<float>(a, y, part, cs);
    } else {
      norm_vectors<kBf16, kBytes, kNv, kPartner>(a, y, part, cs, [&] {
        if (k == 0) angles();
      });
    }
  }
}

using Kernel = void (*)(NormRopeArgs);

template <bool kBf16, int kBytes, int kNv>
Kernel kernel_of(int partner) {
  if constexpr (kNv > 1) {   // (where a lane has one vector, its partner is another lane's)
    if (partner == kSameLane) return norm_rope_kernel<kBf16, kBytes, kNv, kSameLane>;
  }
  return partner == kNoPartner    ? norm_rope_kernel<kBf16, kBytes, kNv, kNoPartner>
         : partner == kOtherLane ? norm_rope_kernel<kBf16, kBytes, kNv, kOtherLane>
                                 : norm_rope_kernel<kBf16, kBytes, kNv, kLoaded>;
}

template <bool kBf16, int kBytes>
Kernel kernel_of(int vecs, int partner) {
  return vecs == 1 ? kernel_of<kBf16, kBytes, 1>(partner) : vecs == 2 ? kernel_of<kBf16, kBytes, 2>(partner)
         : vecs == 3 ? kernel_of<kBf16, kBytes, 3>(partner) : kernel_of<kBf16, kBytes, 4>(partner);
}

Kernel kernel_of(const NormRopeArgs::Slot& y) {
  const bool f32 = y.dtype == 1;
  if (y.bytes == 0) return f32 ? norm_rope_kernel<false, 0, 1, kNoPartner> : norm_rope_kernel<true, 0, 1, kNoPartner>;
  if (y.bytes == 16) return f32 ? kernel_of<false, 16>(y.vecs, y.partner) : kernel_of<true, 16>(y.vecs, y.partner);
  return f32 ? kernel_of<false, 8>(y.vecs, y.partner) : kernel_of<true, 8>(y.vecs, y.partner);
}

// Vectors of 16 or 8 bytes that fit the tensor's sizes and addresses (0: none do), the lanes of a head with the
// vectors of each that leave the fewest over (of those, two vectors a lane where they can be had), and where partners are.
void choose_vectors(NormRopeArgs::Slot& y, int rot, bool interleaved) {
  const int e = y.dtype == 1 ? 4 : 2;
  y.bytes = y.vecs = y.partner = 0;
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
      if (m > kMaxVecs || m * lanes - n > best - (m > 2)) continue;   // (two vectors a lane rather than one: more bytes on their way)
      best = m * lanes - n;
      y.lanes = lanes;
      y.vecs = m;
    }
    y.bytes = w;
    const int rv = rot / v, hv = rv / 2, v0 = y.off / v;
    if (rot == 0 || interleaved) y.partner = kNoPartner;
    else if (hv % y.lanes == 0) y.partner = kSameLane;
    else if (y.lanes % rv == 0 && v0 % rv == 0) y.partner = kOtherLane;
    else y.partner = kLoaded;
    return;
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int rows, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  NormRopeArgs left = a;
  for (int k = 0; k < left.n_slots; ++k) choose_vectors(left.slot[k], a.rot, a.interleaved != 0);
  while (left.n_slots > 0) {   // a launch for the tensors that are alike: queries and keys mostly are
    NormRopeArgs now = left;
    now.n_slots = 0;
    const NormRopeArgs::Slot& y = left.slot[0];
    const Kernel kernel = kernel_of(y);
    int rest = 0, heads = 0;   // heads of the tensor with the most
    for (int k = 0; k < left.n_slots; ++k) {
      const NormRopeArgs::Slot z = left.slot[k];
      if (kernel_of(z) == kernel) {
        now.slot[now.n_slots++] = z;
        heads = heads > z.heads ? heads : z.heads;
      } else {
        left.slot[rest++] = z;
      }
    }
    left.n_slots = rest;
    // Rows of a block and blocks of a row as in rope.cu, but that the blocks fit the SMs' places at once.
    const int want = kPerSm * device_sm_count();
    int most = 64;
    while (most > 8 && most * (a.rot / 2) > 8 * kMaxRopePairs) --most;
    now.rows = rows;
    now.per_block = (rows - 1) / want + 1 > most ? most : (rows - 1) / want + 1;
    const int blocks = (rows - 1) / now.per_block + 1;
    int split = blocks >= want ? 1 : want / blocks;
    split = split > heads ? heads : split < 1 ? 1 : split;
    note_launch();
    const cudaError_t e = launch_pdl(kernel, dim3(unsigned(blocks), unsigned(split)), dim3(kThreads),
                                     size_t(now.per_block) * (a.rot / 2) * sizeof(float2), st, 1, now);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace csa2
