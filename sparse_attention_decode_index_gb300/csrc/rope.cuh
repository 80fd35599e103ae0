// Rotary angles of a block's rows, shared by the kernels that turn (rope.cu and
// norm_rope.cu): how they are reduced stands in rope.cu.
#pragma once
#include "common.cuh"

namespace csa2 {

constexpr int kRopeThreads = 256;     // of a block that makes angles
constexpr int kMaxRopePairs = 512;

// n / d for n * d < 2^32, with m = ceil(2^32 / d) (0 for d = 1).
CSA2_DEV int fast_div(int n, uint32_t m) { return m == 0 ? n : int(__umulhi(uint32_t(n), m)); }

// A vector of 16 or 8 bytes, as words.
template <int kBytes>
struct Vec {
  uint32_t w[kBytes / 4];
  CSA2_DEV void load(const uint8_t* p) {
    if constexpr (kBytes == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
  }
  CSA2_DEV void store(uint8_t* p) const {
    if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
};

// cos and sin (times mag) of rows row0 .. row0 + nr - 1 into cs [nr][half], by all kRopeThreads threads of a block; `step`:
// [kMaxRopePairs] in shared memory.  The caller waits (__syncthreads) before it reads cs.
CSA2_DEV void rope_angles(float2* cs, long long* step, long long row0, int nr, int half, const int* pos, const double* freqs,
                          float mag, bool inverse) {
  auto turns = [&](int p) -> long long {                 // per position, in units of 2^-64
    double f = freqs[p] * 0.15915494309189533577;
    f -= rint(f);                                        // whole turns change nothing
    return __double2ll_rn(f * 18446744073709551616.0);   // saturates at half a turn, 2^-64 off
  };
  // Once a block where a thread has several angles (fp64 is slow); otherwise no
  // barrier holds back the threads that have none (8 rows: 6.5 us, with the barrier 6.9).
  auto angle = [&](int i, int r, long long F) {
    const unsigned long long t = (unsigned long long)(long long)pos[row0 + r] * (unsigned long long)F;
    const float turn = float((long long)t) * 5.421010862427522e-20f;  // * 2^-64: in [-1/2, 1/2]
    float s, c;
    sincospif(2.f * turn, &s, &c);
    cs[i] = make_float2(c * mag, (inverse ? -s : s) * mag);
  };
  if (nr * half > kRopeThreads) {
    for (int p = threadIdx.x; p < half; p += kRopeThreads) step[p] = turns(p);
    __syncthreads();
    for (int i = threadIdx.x; i < nr * half; i += kRopeThreads) angle(i, i / half, step[i % half]);
  } else if (int(threadIdx.x) < nr * half) {
    angle(threadIdx.x, threadIdx.x / half, turns(threadIdx.x % half));
  }
}

}  // namespace csa2
