// Rotary positions for several tensors of the same rows in one launch
// (queries, keys and indexer queries of drafted or prompt tokens):
//     (a, b) -> mag * (a cos t - b sin t, b cos t + a sin t),  t = pos * freq.
//
// The angle.  pos * freq in fp32 is off by up to 2^-24 of the angle, 0.06 rad
// at a million positions, and fp64 is slow on this GPU.  A frequency is
// therefore turned once per block into turns per position as a 64-bit fixed-
// point fraction F = freq / 2 pi mod 1 in units of 2^-64; pos * F modulo 2^64 is
// then the exact angle of F in turns, whatever whole turns it passes, and its
// top bits, read as a signed number, lie in [-1/2, 1/2) turns.  F is rounded
// from fp64, so the angle is off by at most |t| 2^-52 for any int32 position,
// and sincospif takes the reduced angle in half turns.
//
// Memory bound: every element is read once and written once, and the cos and
// sin of a row are made once per block (shared memory) and used by all its heads.  A block
// takes one row and a chunk of heads; an item is one 16-byte vector that is
// copied, or the vectors that hold the two halves of pairs.
#include "common.cuh"
#include "internal.h"

namespace csa2 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;
constexpr int kBatch = 4;   // items a thread loads before it stores any

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

CSA2_DEV float to_f32(float v) { return v; }
CSA2_DEV float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
CSA2_DEV void from_f32(float& d, float v) { d = v; }
CSA2_DEV void from_f32(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

// The heads [h0, h1) of one row.  Items of a head: first the rotating ones
// (half layout: the vector pair at i and i + rot / 2; interleaved: one vector
// of V / 2 pairs, or for V = 1 the two elements of a pair), then, out of place,
// the copied vectors before and behind the turned range.
template <typename T, int V>
CSA2_DEV void turn_heads(const RopeArgs::Slot& y, long long row, int h0, int h1, int rot, bool inter,
                         const float2* cs) {
  using W = Vec<T, V>;
  const int half = rot / 2;
  const bool copy = y.x != y.out;
  const bool two = !inter || V == 1;                     // an item holds two vectors
  const int n_rot = two ? half / V : rot / V;
  const int before = y.off / V, n_copy = copy ? (y.dim - rot) / V : 0;
  const int per_head = n_rot + n_copy;
  const int total = (h1 - h0) * per_head;
  const T* x = static_cast<const T*>(y.x) + (row * y.heads + h0) * (long long)y.dim;
  T* out = static_cast<T*>(y.out) + (row * y.heads + h0) * (long long)y.dim;
  for (int i0 = threadIdx.x; i0 < total; i0 += kBatch * kThreads) {
    W a[kBatch], b[kBatch];
    int at[kBatch], pair[kBatch];                        // pair < 0: a copied vector
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      const int i = i0 + m * kThreads;
      if (i >= total) continue;
      const int h = i / per_head, it = i - h * per_head;
      if (it < n_rot) {
        const int e = two ? (inter ? 2 * it : it * V) : it * V;   // first element in the turned range
        pair[m] = inter ? e / 2 : e;
        at[m] = h * y.dim + y.off + e;
      } else {
        const int c = it - n_rot;
        pair[m] = -1;
        at[m] = h * y.dim + (c < before ? c * V : (c - before) * V + y.off + rot);
      }
      a[m] = *reinterpret_cast<const W*>(x + at[m]);
      if (two && pair[m] >= 0) b[m] = *reinterpret_cast<const W*>(x + at[m] + (inter ? 1 : half));
    }
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      const int i = i0 + m * kThreads;
      if (i >= total) continue;
      if (pair[m] >= 0) {
        if (two) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 r = cs[pair[m] + e];
            const float u = to_f32(a[m].e[e]), v = to_f32(b[m].e[e]);
            from_f32(a[m].e[e], u * r.x - v * r.y);
            from_f32(b[m].e[e], v * r.x + u * r.y);
          }
          *reinterpret_cast<W*>(out + at[m] + (inter ? 1 : half)) = b[m];
        } else {
#pragma unroll
          for (int e = 0; e + 1 < V; e += 2) {
            const float2 r = cs[pair[m] + e / 2];
            const float u = to_f32(a[m].e[e]), v = to_f32(a[m].e[e + 1]);
            from_f32(a[m].e[e], u * r.x - v * r.y);
            from_f32(a[m].e[e + 1], v * r.x + u * r.y);
          }
        }
      }
      *reinterpret_cast<W*>(out + at[m]) = a[m];
    }
  }
}

__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 cs[kMaxPairs];
  const long long row = blockIdx.x;
  int k = 0;
  while (k + 1 < a.n_slots && int(blockIdx.y) >= a.slot[k + 1].first) ++k;
  const RopeArgs::Slot& y = a.slot[k];
  const int h0 = (int(blockIdx.y) - y.first) * y.per_chunk, h1 = min(y.heads, h0 + y.per_chunk);
  pdl_wait();   // no early trigger: the attention may read what this kernel writes before its own wait
  const long long pos = a.pos[row];
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) {
    double f = a.freqs[i] * 0.15915494309189533577;      // turns per position
    f -= rint(f);                                        // whole turns change nothing
    const long long F = __double2ll_rn(f * 18446744073709551616.0);   // saturates at half a turn, 2^-64 off
    const unsigned long long t = (unsigned long long)pos * (unsigned long long)F;
    // the top 32 bits as a signed fraction of a turn, the next ones added in fp32
    const float turn = float((long long)t) * 5.421010862427522e-20f;   // 2^-64: in [-1/2, 1/2]
    float s, c;
    sincospif(2.f * turn, &s, &c);
    const float m = a.inverse ? 1.f / a.mag : a.mag;
    cs[i] = make_float2(c * m, (a.inverse ? -s : s) * m);
  }
  __syncthreads();
  const bool inter = a.interleaved != 0;
  if (y.dtype == 1) {
    if (y.vec == 4) turn_heads<float, 4>(y, row, h0, h1, a.rot, inter, cs);
    else turn_heads<float, 1>(y, row, h0, h1, a.rot, inter, cs);
  } else {
    if (y.vec == 8) turn_heads<__nv_bfloat16, 8>(y, row, h0, h1, a.rot, inter, cs);
    else turn_heads<__nv_bfloat16, 1>(y, row, h0, h1, a.rot, inter, cs);
  }
}

}  // namespace

cudaError_t launch_rope(RopeArgs& a, int rows, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  // Heads per block: all of a row's when the rows alone fill the SMs (the
  // angles are then made once per row), fewer for few rows.
  const int want = 2 * device_sm_count();
  int split = rows >= want ? 1 : (want + rows - 1) / rows;
  int chunks = 0;
  for (int k = 0; k < a.n_slots; ++k) {
    RopeArgs::Slot& y = a.slot[k];
    const int v = y.dtype == 1 ? 4 : 8;
    const uintptr_t at = reinterpret_cast<uintptr_t>(y.x) | reinterpret_cast<uintptr_t>(y.out);
    y.vec = (at % 16 == 0 && y.dim % v == 0 && y.off % v == 0 && (a.interleaved ? a.rot : a.rot / 2) % v == 0) ? v : 1;
    y.per_chunk = (y.heads + split - 1) / split;
    y.first = chunks;
    chunks += (y.heads + y.per_chunk - 1) / y.per_chunk;
  }
  note_launch();
  return launch_pdl(rope_kernel, dim3(unsigned(rows), unsigned(chunks)), dim3(kThreads), 0, st, 1, a);
}

}  // namespace csa2
