// Rotary positions for several tensors of the same rows in one launch
// (queries, keys and indexer queries of drafted or prompt tokens):
//     (a, b) -> mag * (a cos t - b sin t, b cos t + a sin t),  t = pos * freq.
//
// The angle.  pos * freq in fp32 is off by up to 2^-24 of the angle, 0.06 rad
// at a million positions, and fp64 is slow on this GPU.  A frequency is
// therefore turned into turns per position once (a block, where its threads
// have several angles each): a 64-bit fixed-point fraction F = freq / 2 pi mod
// 1 in units of 2^-64.  pos * F modulo 2^64 is then the exact angle of F in
// turns, whatever whole turns it passes, and its top bits, read as a signed
// number, lie in [-1/2, 1/2) turns.  F is rounded from fp64 to whole units, and
// the reduced angle to fp32, which sincospif takes in half turns: the angle is
// off by at most |t| 2^-52 + |pos| 2 pi 2^-65 + 2 pi 2^-26 for any int32 position
// (the last term, 9.4e-8, for all but those beyond a few hundred million radians).
//
// Memory bound: every element is read once and written once.  A block takes
// up to 8 rows, or 64 small ones, and makes all their cos and sin at once (kept
// in shared memory and used by all the heads of all the tensors), so that the
// chain position -> angle -> sincospif is waited for once a block; with one row
// a block its latency, not the memory, set the time (8,192 rows of 64 + 1 heads
// of 192: 239 us; 8 rows a block 69.6 us, 5.9 TB/s, the floor being 60.3).  Few
// rows are split over the heads instead (8 rows: 5.8 us, a launch and that
// chain).  An item is one vector that is copied, or the vectors that hold the
// two halves of pairs: 16 bytes, or 8 where the sizes allow no more (7,716 rows of 48
// heads of 40, 4 pairs: 17.3 us, element by element 71.3); its head comes from a multiplication by a
// precomputed reciprocal.
#include "common.cuh"
#include "draft.h"
#include "rope.cuh"

namespace csa2 {

namespace {

constexpr int kThreads = kRopeThreads;
constexpr int kMaxPairs = kMaxRopePairs;
constexpr int kMaxRows = 8, kMaxAngles = kMaxRows * kMaxPairs, kMaxVecs = 4096;   // of a block
constexpr int kBatch = 4;   // vectors a thread loads before it stores any

CSA2_DEV float to_f32(float v) { return v; }
CSA2_DEV float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
CSA2_DEV void from_f32(float& d, float v) { d = v; }
CSA2_DEV void from_f32(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

// The heads [h0, h0 + nh) of rows row0 .. row0 + nr - 1 of one tensor; `items`
// of a head are shared out over the block's threads.
struct Heads {
  int items, nh, dim, skip, total;
  uint32_t m_item, m_head;

  CSA2_DEV Heads(const RopeArgs::Slot& y, int nr, int nh_, int items_)
      : items(items_), nh(nh_), dim(y.dim), skip((y.heads - nh_) * y.dim), total(nr * nh_ * items_) {
    m_item = items <= 1 ? 0u : 0xffffffffu / uint32_t(items) + 1u;
    m_head = nh <= 1 ? 0u : 0xffffffffu / uint32_t(nh) + 1u;
  }
  // Item i: its place in its head, its row, and the head's offset (total <= 2^21, items <= 1024).
  CSA2_DEV int at(int i, int& it, int& row) const {
    const int h = fast_div(i, m_item);
    it = i - h * items;
    row = fast_div(h, m_head);
    return h * dim + row * skip;
  }
};

// (a, b) -> (a c - b s, b c + a s), two bf16 pairs: words (a0, a1), (b0, b1).
CSA2_DEV void turn_words(uint32_t& a, uint32_t& b, float4 cs) {
  const float a0 = __uint_as_float(a << 16), a1 = __uint_as_float(a & 0xffff0000u);
  const float b0 = __uint_as_float(b << 16), b1 = __uint_as_float(b & 0xffff0000u);
  a = pack_bf16(a0 * cs.x - b0 * cs.y, a1 * cs.z - b1 * cs.w);
  b = pack_bf16(b0 * cs.x + a0 * cs.y, b1 * cs.z + a1 * cs.w);
}

// The same of two fp32 words.
CSA2_DEV void turn_word(uint32_t& a, uint32_t& b, float c, float s) {
  const float f = __uint_as_float(a), g = __uint_as_float(b);
  a = __float_as_uint(f * c - g * s);
  b = __float_as_uint(g * c + f * s);
}

// The turned vectors of the half layout: vector i and its partner rot / 2 further.
template <bool kBf16, int kBytes>
CSA2_DEV void turn_half(const Heads& n, const uint8_t* x, uint8_t* out, int off, int half, const float2* cs) {
  constexpr int kE = kBf16 ? 2 : 4, kV = kBytes / kE, kB = kBatch / 2;
  for (int i0 = threadIdx.x; i0 < n.total; i0 += kB * kThreads) {
    Vec<kBytes> a[kB], b[kB];
    int at[kB], p[kB];
#pragma unroll
    for (int m = 0; m < kB; ++m) {
      const int i = i0 + m * kThreads;
      int it = 0, row = 0;
      at[m] = i < n.total ? n.at(i, it, row) : 0;
      at[m] = (at[m] + off + it * kV) * kE;
      p[m] = row * half + it * kV;
      if (i < n.total) {
        a[m].load(x + at[m]);
        b[m].load(x + at[m] + half * kE);
      }
    }
#pragma unroll
    for (int m = 0; m < kB; ++m) {
      if (i0 + m * kThreads >= n.total) break;
      const float4* c = reinterpret_cast<const float4*>(cs + p[m]);   // p and half are even here
      if (kBf16) {
#pragma unroll
        for (int e = 0; e < kBytes / 4; ++e) turn_words(a[m].w[e], b[m].w[e], c[e]);
      } else {
#pragma unroll
        for (int e = 0; e < kBytes / 8; ++e) {
          const float4 c2 = c[e];
          turn_word(a[m].w[2 * e], b[m].w[2 * e], c2.x, c2.y);
          turn_word(a[m].w[2 * e + 1], b[m].w[2 * e + 1], c2.z, c2.w);
        }
      }
      a[m].store(out + at[m]);
      b[m].store(out + at[m] + half * kE);
    }
  }
}

// The turned vectors of the interleaved layout: pairs of neighbours.
template <bool kBf16, int kBytes>
CSA2_DEV void turn_inter(const Heads& n, const uint8_t* x, uint8_t* out, int off, int half, const float2* cs) {
  constexpr int kE = kBf16 ? 2 : 4, kV = kBytes / kE;
  for (int i0 = threadIdx.x; i0 < n.total; i0 += kBatch * kThreads) {
    Vec<kBytes> a[kBatch];
    int at[kBatch], p[kBatch];
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      const int i = i0 + m * kThreads;
      int it = 0, row = 0;
      at[m] = i < n.total ? n.at(i, it, row) : 0;
      at[m] = (at[m] + off + it * kV) * kE;
      p[m] = row * half + it * (kV / 2);
      if (i < n.total) a[m].load(x + at[m]);
    }
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      if (i0 + m * kThreads >= n.total) break;
      const float2* c = cs + p[m];
      float2 r[kV / 2];
      if constexpr (kV >= 4) {                         // whole float4s: p is even here
#pragma unroll
        for (int e = 0; e < kV / 4; ++e) {
          const float4 c2 = reinterpret_cast<const float4*>(c)[e];
          r[2 * e] = make_float2(c2.x, c2.y);
          r[2 * e + 1] = make_float2(c2.z, c2.w);
        }
      } else {
        r[0] = c[0];
      }
#pragma unroll
      for (int e = 0; e < kV / 2; ++e) {
        if (kBf16) {
          uint32_t& w = a[m].w[e];
          const float f = __uint_as_float(w << 16), g = __uint_as_float(w & 0xffff0000u);
          w = pack_bf16(f * r[e].x - g * r[e].y, g * r[e].x + f * r[e].y);
        } else {
          turn_word(a[m].w[2 * e], a[m].w[2 * e + 1], r[e].x, r[e].y);
        }
      }
      a[m].store(out + at[m]);
    }
  }
}

// The vectors that are not turned: `before` of them in front of the turned range, the others behind it.
template <int kBytes>
CSA2_DEV void copy_rest(const Heads& n, const uint8_t* x, uint8_t* out, int before, int rot_vecs, int esize) {
  for (int i0 = threadIdx.x; i0 < n.total; i0 += kBatch * kThreads) {
    Vec<kBytes> a[kBatch];
    int at[kBatch];
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      const int i = i0 + m * kThreads;
      int it = 0, row = 0;
      at[m] = i < n.total ? n.at(i, it, row) * esize : 0;
      at[m] += (it < before ? it : it + rot_vecs) * kBytes;
      if (i < n.total) a[m].load(x + at[m]);
    }
#pragma unroll
    for (int m = 0; m < kBatch; ++m)
      if (i0 + m * kThreads < n.total) a[m].store(out + at[m]);
  }
}

// Any size and alignment: an item is a pair, or an element that is copied.
template <typename T>
CSA2_DEV void turn_scalar(const RopeArgs::Slot& y, int nr, int nh, const T* x, T* out, int rot, bool inter,
                          const float2* cs) {
  const int half = rot / 2;
  const Heads n(y, nr, nh, half + (y.x != y.out ? y.dim - rot : 0));
  for (int i = threadIdx.x; i < n.total; i += kThreads) {
    int it, row;
    int at = n.at(i, it, row);
    if (it < half) {
      at += y.off + (inter ? 2 * it : it);
      const int to = at + (inter ? 1 : half);
      const float2 r = cs[row * half + it];
      const float u = to_f32(x[at]), v = to_f32(x[to]);
      from_f32(out[at], u * r.x - v * r.y);
      from_f32(out[to], v * r.x + u * r.y);
    } else {
      const int c = it - half;
      at += c < y.off ? c : c + rot;
      out[at] = x[at];
    }
  }
}

// kBytes: of the vectors of the tensors that are wide.  (One kernel for both sizes was 1 us slower: more
// instructions to fetch.)
template <bool kInter, int kBytes>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) float2 cs[];           // [per_block][rot / 2]
  __shared__ long long step[kMaxPairs];                  // turns per position, in units of 2^-64
  const long long row0 = (long long)blockIdx.x * a.per_block;
  const int nr = int(min((long long)a.per_block, a.rows - row0));
  pdl_wait();   // no early trigger: the attention may read what this kernel writes before its own wait
  const int half = a.rot / 2;
  const float mag = a.inverse ? 1.f / a.mag : a.mag;
  rope_angles(cs, step, row0, nr, half, a.pos, a.freqs, mag, a.inverse != 0);
  // tensor k's heads of this block (nh == 0: none) and their place
  auto part = [&](int k, int& nh, const uint8_t*& x, uint8_t*& out) -> const RopeArgs::Slot& {
    const RopeArgs::Slot& y = a.slot[k];
    const int h0 = int((long long)y.heads * blockIdx.y / gridDim.y);
    nh = int((long long)y.heads * (blockIdx.y + 1) / gridDim.y) - h0;
    const long long base = (row0 * y.heads + h0) * (long long)y.dim * (y.dtype == 1 ? 4 : 2);
    x = static_cast<const uint8_t*>(y.x) + base;
    out = static_cast<uint8_t*>(y.out) + base;
    return y;
  };
  for (int k = 0; k < a.n_slots; ++k) {
    int nh;
    const uint8_t* x;
    uint8_t* out;
    const RopeArgs::Slot& y = part(k, nh, x, out);
    if (!y.wide || y.x == y.out) continue;
    const int esize = y.dtype == 1 ? 4 : 2, copy = kBytes == 16 ? 16 : y.copy, v = copy / esize;
    const Heads n(y, nr, nh, (y.dim - a.rot) / v);
    // 16 bytes where only the halves ask for 8 (2,562 rows of 64 heads of 192, 4 pairs: 34.3 -> 27.7 us; where
    // nothing has 16, 48 heads of 40, the choice costs 16.5 -> 17.3)
    if (copy == 16) copy_rest<16>(n, x, out, y.off / v, a.rot / v, esize);
    else copy_rest<8>(n, x, out, y.off / v, a.rot / v, esize);
  }
  __syncthreads();                                       // the angles
  for (int k = 0; k < a.n_slots; ++k) {
    int nh;
    const uint8_t* x;
    uint8_t* out;
    const RopeArgs::Slot& y = part(k, nh, x, out);
    if (!y.wide) {
      if (y.dtype == 1)
        turn_scalar(y, nr, nh, reinterpret_cast<const float*>(x), reinterpret_cast<float*>(out), a.rot, kInter, cs);
      else
        turn_scalar(y, nr, nh, reinterpret_cast<const __nv_bfloat16*>(x), reinterpret_cast<__nv_bfloat16*>(out), a.rot,
                    kInter, cs);
      continue;
    }
    const Heads n(y, nr, nh, (kInter ? a.rot : half) / (y.dtype == 1 ? kBytes / 4 : kBytes / 2));
    if (kInter)
      y.dtype == 1 ? turn_inter<false, kBytes>(n, x, out, y.off, half, cs) : turn_inter<true, kBytes>(n, x, out, y.off, half, cs);
    else
      y.dtype == 1 ? turn_half<false, kBytes>(n, x, out, y.off, half, cs) : turn_half<true, kBytes>(n, x, out, y.off, half, cs);
  }
}

}  // namespace

cudaError_t launch_rope(RopeArgs& a, int rows, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  int heads = 0;   // of the tensor with the most
  int vecs = 0;    // 16-byte pieces of a row of all tensors
  int bytes = 16;  // of a vector: 8 where a tensor cannot have 16 but 8
  auto whole = [&](const RopeArgs::Slot& y, int w) -> bool {  // vectors of w bytes in front of, in and behind the turned dims
    const uintptr_t at = reinterpret_cast<uintptr_t>(y.x) | reinterpret_cast<uintptr_t>(y.out);
    const int e = w / (y.dtype == 1 ? 4 : 2);
    return at % w == 0 && y.dim % e == 0 && y.off % e == 0 && a.rot % e == 0;
  };
  auto fits = [&](const RopeArgs::Slot& y, int w) -> bool {   // and in either half of them
    return whole(y, w) && (a.interleaved || a.rot / 2 % (w / (y.dtype == 1 ? 4 : 2)) == 0);
  };
  for (int k = 0; k < a.n_slots; ++k) {
    RopeArgs::Slot& y = a.slot[k];
    if (!fits(y, 16) && fits(y, 8)) bytes = 8;
    heads = heads > y.heads ? heads : y.heads;
    vecs += (y.heads * y.dim * (y.dtype == 1 ? 4 : 2) + 15) / 16;
  }
  for (int k = 0; k < a.n_slots; ++k) {
    a.slot[k].wide = fits(a.slot[k], bytes);
    a.slot[k].copy = whole(a.slot[k], 16) ? 16 : 8;   // (of wide ones)
  }
  // Four blocks for every SM: as many rows a block as that leaves, up to 8, of
  // small rows up to 64 (16,384 rows of one head of 192, 32 pairs: 22.0 us with 8, 12.2 with 26);
  // when one row each does not give that many blocks, the heads are split.
  const int want = 4 * device_sm_count();
  a.rows = rows;
  int most = 64;
  while (most > kMaxRows && (most * (a.rot / 2) > kMaxAngles || most * vecs > kMaxVecs)) --most;
  a.per_block = rows / want < 1 ? 1 : rows / want > most ? most : rows / want;
  for (int k = 0; k < a.n_slots; ++k)   // keeps fast_div's products below 2^32
    while (a.per_block > 1 && a.per_block * a.slot[k].heads * a.slot[k].dim > (1 << 21)) --a.per_block;
  const int blocks = (rows - 1) / a.per_block + 1;   // (rows go up to 2^31 - 1)
  int split = blocks >= want ? 1 : (want + blocks - 1) / blocks;
  split = split > heads ? heads : split;
  note_launch();
  const auto kernel = a.interleaved ? (bytes == 16 ? rope_kernel<true, 16> : rope_kernel<true, 8>)
                                    : (bytes == 16 ? rope_kernel<false, 16> : rope_kernel<false, 8>);
  return launch_pdl(kernel, dim3(unsigned(blocks), unsigned(split)),
                    dim3(kThreads), size_t(a.per_block) * (a.rot / 2) * sizeof(float2), st, 1, a);
}

}  // namespace csa2
