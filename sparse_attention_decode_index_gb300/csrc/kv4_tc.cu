// Sparse attention over a packed main cache (kv4.cuh) on the 5th-generation tensor
// cores (bf16, 64 heads sharing one KV head, dk 192, dv 128).
//
// A query's keys come in tiles of 64: its selected entries first, then its
// window rows.  Code * scale is exact in fp16, so that an entry's row becomes fp16 and its
// products with the query, which is put into fp16's range by a power of two a head, are
// as exact as bf16's (an element 2^34 below its head's largest is lost); its weights have 11 bits
// there instead of 8.  Window rows stay bf16, with bf16 weights and the query as it is.
//
// A row of the tensor cores' 128 is a head and half of a tile's keys: rows 0..63 take
// each tile's first 32 keys, rows 64..127 the other 32, and have weights of 0 for
// the rest.  The scores are computed for all rows anyway, so that this costs the tensor
// cores nothing and halves the exponentials of a thread; the two halves have their own maxima and sums and
// are added at the end, like the parts of a split.
//
// Roles of a CTA (18 warps):
//   4 softmax warps: a thread owns a row; P goes back to TMEM over its S.  O is rescaled only when a
//     maximum grows by more than 2^8;
//   4 end warps put the next query into TMEM (as bf16 and as fp16) and write the last one's O out;
//   8 producer warps in two groups that take turns at the tiles, 16 rows a warp: packed entries come by
//     cp.async one turn ahead, their indices three, and become a stage's K and V rows (K-major, MN-major,
//     128-byte swizzled): lane l takes row l % 8 and the words l / 8, + 4, ... of 8 codes, which meets no bank
//     twice.  A window tile comes by TMA;
//   1 warp issues S = Q K^T, up to three tiles ahead, and 1 warp O += P V.
// Many queries: persistent, a CTA an SM.  Few: a query's tiles are split over a
// cluster of up to 8 CTAs, whose partial O are merged through distributed shared memory as in attn.cu.
//
// P is rounded to fp16 (entries) or bf16 (window) as the tensor core asks for; the weights' sums stay fp32 and unrounded.
//
// Measured (512 entries and 128 window rows a query, distinct inputs in turn in a CUDA graph): 1 query 10.6 us, 64 12.9, 256 24.3,
// 1,024 in sequences of 32 66.1 (20.5 of which their 139 MB would take, and 14 their products); attn.cu on bf16 rows of the same
// entries 9.1, 13.7, 56.2, 207.  Neither bounds it (DRAM 27 %, tensor cores 33 %, issue slots 45 %): a
// tile's way from S to P, 700 to 1,000 cycles one behind the other, and 2,000 to 4,000 between two queries do.  Two groups of
// softmax warps, which hand a row's exponent on, took 73.8 for 65.8: 24 warps leave 80 registers a thread.
#include <cuda.h>

#include "kv4.cuh"
#include "tc.cuh"

namespace csa2 {

namespace {

constexpr int kH = 64, kDk = 192, kDv = 128;
constexpr int kTile = 64;                      // keys a stage
constexpr int kEntry = kv4_bytes(kDk, kDv);    // 192: codes 0..159, scales 160..179
constexpr int kKBytes = kTile * kDk * 2, kVBytes = kTile * kDv * 2;
constexpr int kStages = 4;                     // an even number: a stage always belongs to the same group of producers
constexpr int kScores = 3;                     // buffers of S and P
constexpr int kSoftmaxWarps = 4, kEndWarps = 4, kProducerWarps = 8;
constexpr int kGroups = 2, kGroupWarps = kProducerWarps / kGroups;   // of producers, which take turns at the tiles
constexpr int kRows = kTile / kGroupWarps;     // entries of a producer warp: 16
constexpr int kThreads = 32 * (kSoftmaxWarps + kEndWarps + kProducerWarps + 2);
constexpr int kPackedRow = kEntry + 16;        // padded: rows of 4 lanes' words meet no bank twice
constexpr int kScales = 160;                   // where an entry's scales begin
constexpr int kIndexAhead = 3, kIndexRing = 4;   // tiles whose indices are on their way, of a group, and room for them
constexpr int kScoresWarp = kSoftmaxWarps + kEndWarps + kProducerWarps, kValuesWarp = kScoresWarp + 1;
constexpr int kMaxCluster = 8;
constexpr int kQRow = kDk * 2 + 16;            // query rows on their way to TMEM
constexpr int kXRow = 68;                      // fp32 columns of a row that the halves exchange, padded
constexpr int kPRow = kDv + 4;                 // partial O of a split
// Weights are held as 2^7 times their relation to their row's exponent: at most 2^15, as that grows by steps of 2^8, which
// fp16 holds, and rounded by at most 2^-11 of themselves or, below 2^-21, by 2^-32 of the greatest.
constexpr float kUp = 7.f;
constexpr uint32_t kTmemCols = 512;            // O (128), three S (64 each), Q as fp16 and as bf16 (96 each)
constexpr uint32_t kOCol = 0, kSCol = 128, kQhCol = 320, kQbCol = 416;

struct Shared {
  uint8_t k[kStages][kKBytes];                 // 3 blocks of 64 dims: 64 rows of 128 bytes
  uint8_t v[kStages][kVBytes];                 // 2 blocks of 64 dims: 64 keys of 128 bytes
  uint8_t packed[kProducerWarps][kRows * kPackedRow];
  int index[kProducerWarps][kIndexRing][kRows];
  union {                                      // the next query until it is in TMEM, then what the halves of an O exchange
    uint8_t q[kH * kQRow];
    float x[128 * kXRow];
  };
  uint64_t mask[kStages];                      // the tile's keys that are there
  float2 stat[128];                            // (exponent, sum) of the rows of an item
  float q_scale[2][128];                       // what a row's fp16 products are multiplied by, of even and odd items
  uint32_t top[128];                           // bits of the largest magnitude of half a head's query
  float2 part[kH];                             // (exponent, sum) of the CTAs of a split, of the heads that this one adds up
  uint64_t full[kStages], empty[kStages];      // a tile has landed; has been used
  uint64_t s_full[kScores], p_full[kScores];   // S has been computed; P has been written
  uint64_t s_free[kScores];                    // O holds the tile whose weights lay there
  uint64_t o_last, o_free;                     // O holds the item's last tile; has been read
  uint64_t q_full[2], q_empty[2];              // of the query as fp16 and as bf16
  uint64_t stat_full, stat_free;
  uint64_t window[kGroups];                    // a window tile that is not full has landed
  uint64_t ends;                               // the end warps have come here
  uint64_t fin;                                // every MMA is done
  uint32_t tmem;
  volatile int abort;
};
constexpr int kSmem = int(sizeof(Shared)) + 1024;   // + room to align to 1,024
static_assert(kSmem <= 227 * 1024, "fits an SM");
static_assert(kH * kPRow * 4 + kMaxCluster * kH * 4 <= kStages * kKBytes, "a split's partial O and weights take the K stages");

// Instruction descriptor of kind::f16: fp16 x fp16 -> fp32.
constexpr uint32_t idesc_f16(int m, int n, bool b_mn) { return idesc_bf16(m, n, b_mn) & ~((1u << 7) | (1u << 10)); }

CSA2_DEV void cp16(uint32_t dst, const uint8_t* src) { asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory"); }
CSA2_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
CSA2_DEV uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A bounded wait of a whole warp, which goes on or gives up together (as tc_wait_warp, counted in cycles: many warps wait here).
CSA2_DEV bool wait_warp(Shared& c, uint64_t* bar, uint32_t parity, const Kv4AttnArgs& a) {
  bool here = mbar_try_wait(bar, parity);
  if (!here) {
    const long long t0 = clock64();
    for (uint32_t i = 1;; ++i) {
      here = mbar_try_wait(bar, parity);
      if (here) break;
      if ((i & 31u) == 0u) {
        if (c.abort) break;
        if (clock64() - t0 > a.wait_cycles) {
          c.abort = 1;
          report(a.err, kErrTimeout, int(threadIdx.x));   // which role gave up first
          break;
        }
      }
    }
  }
  return __all_sync(0xffffffffu, here) != 0;
}

// One arrival for a whole warp's reads and writes so far.
CSA2_DEV void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The tiles of a query that CTA `rank` of `n` takes: [first, last) of its tiles, of which those from `window` on are the
// window's.
struct Range {
  int first, last, window;
  CSA2_DEV Range(const Kv4AttnArgs& a, int rank, int n) {
    window = (a.topk + kTile - 1) / kTile;
    const int all = window + (a.swa + kTile - 1) / kTile;
    first = all * rank / n;
    last = all * (rank + 1) / n;
  }
};

// A box of 64 rows of 64 dims, swizzled, from dim x of row y (TMA).
CSA2_DEV void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// The same into L2.
CSA2_DEV void prefetch_box(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    kv4_tc_kernel(const Kv4AttnArgs a, int n_items, int ncta, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ uint8_t raw[];
  Shared& c = *reinterpret_cast<Shared*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int crank = ncta > 1 ? int(cluster_rank()) : 0;
  const int item0 = int(blockIdx.x) / ncta, step = int(gridDim.x) / ncta;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&c.full[i], kGroupWarps + (i == 0 ? a.never : 0));
      mbar_init(&c.empty[i], 1 + kSoftmaxWarps);   // the values' end; its mask has been read
    }
    for (int b = 0; b < kScores; ++b) {
      mbar_init(&c.s_full[b], 1);
      mbar_init(&c.p_full[b], kSoftmaxWarps);
      mbar_init(&c.s_free[b], 1);
    }
    mbar_init(&c.o_last, 1);
    mbar_init(&c.o_free, kEndWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.q_full[i], kEndWarps);
      mbar_init(&c.q_empty[i], 1);
    }
    mbar_init(&c.stat_full, kSoftmaxWarps);
    mbar_init(&c.stat_free, kEndWarps);
    for (int g = 0; g < kGroups; ++g) mbar_init(&c.window[g], 1);
    mbar_init(&c.ends, kEndWarps);
    mbar_init(&c.fin, 2);
    c.abort = 0;
    mbar_fence_init();
  }
  __syncwarp();
  if (warp == 0) tmem_alloc(&c.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  if (ncta > 1) cluster_arrive();              // (waited for before anything is written to a peer)
  bool joined = ncta == 1;                     // this warp has waited for that
  pdl_wait();
  const Range range(a, crank, ncta);
  const float log2e = 1.4426950408889634f;

  if (warp < kSoftmaxWarps) {
    // ---------------------------------------------------------------- softmax: thread = row
    const int half = tid >> 6;                                // of a tile's keys (uniform in a warp)
    const uint32_t lanes = uint32_t(warp * 32) << 16;
    const uint32_t o_addr = tmem + lanes + kOCol;
    const float window_scale = a.scale * log2e, window_up = 1.f / a.v_up;
    uint32_t items = 0, st = 0, buf = 0, turn = 0;            // buf: of S, turn: its times round
    bool ok = true;
    for (int item = item0; item < n_items && ok; item += step) {
      float ref = -INFINITY, sum = 0.f;        // the exponent that P and O are relative to, and the weights' sum
      bool first = true;
      for (int t = range.first; t < range.last; ++t) {
        ok = wait_warp(c, &c.s_full[buf], turn & 1, a);
        if (!ok) break;
        tc_fence_after();
        const uint32_t mask = reinterpret_cast<const uint32_t*>(&c.mask[st])[half];
        warp_arrive(&c.empty[st]);
        if (++st == kStages) st = 0;
        const bool window = t >= range.window;
        const uint32_t s_addr = tmem + lanes + kSCol + buf * 64;
        uint32_t p[16];                        // weights of this half's keys of the tile
        if (mask != 0) {
          const float sl2 = window ? window_scale : c.q_scale[items & 1][tid];
          uint32_t s[32];
          tmem_ld32(s, s_addr + 32 * half);
          if (mask != ~0u) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((mask >> j) & 1u)) s[j] = 0xff800000u;    // -inf
          }
          float m[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            m[e] = __uint_as_float(s[e]);
#pragma unroll
            for (int j = 4; j + 4 < 32; j += 8) m[e] = max3_nan(m[e], __uint_as_float(s[j + e]), __uint_as_float(s[j + 4 + e]));
            m[e] = max3_nan(m[e], m[e], __uint_as_float(s[28 + e]));
          }
          const float top = max3_nan(max3_nan(m[0], m[1], m[2]), m[3], m[3]) * sl2;
          if (!(top < INFINITY)) sum = NAN;                   // as the definition has it
          const bool grows = top > ref + 8.f;
          if (first) {
            ref = top;
          } else if (__any_sync(0xffffffffu, grows)) {
            // O holds tiles up to the one before: wait for it.
            ok = buf > 0 ? wait_warp(c, &c.s_free[buf - 1], turn & 1, a) : wait_warp(c, &c.s_free[kScores - 1], (turn - 1) & 1, a);
            if (!ok) break;
            tc_fence_after();
            const float f = grows ? ex2(ref - top) : 1.f;
            if (grows) ref = top;
            sum *= f;
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
              uint32_t o[16];
              tmem_ld16(o, o_addr + 16 * q);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st16(o_addr + 16 * q, o);
            }
          }
          const float base = ref == -INFINITY ? 0.f : kUp - ref;
          const float2 scale2 = make_float2(sl2, sl2), base2 = make_float2(base, base);
          float2 total = make_float2(0.f, 0.f), other = make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 x = fma2(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), scale2, base2);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            if (j & 1) other = add2(other, x);
            else total = add2(total, x);
            s[2 * j] = __float_as_uint(x.x);
            s[2 * j + 1] = __float_as_uint(x.y);
          }
          if (window) {
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = pack_bf16(__uint_as_float(s[2 * j]) * window_up, __uint_as_float(s[2 * j + 1]) * window_up);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = pack_f16(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
          }
          total = add2(total, other);
          sum += total.x + total.y;
          first = false;
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) p[j] = 0;
        }
        uint32_t zeros[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) zeros[j] = 0;
        tmem_st16(s_addr + 16 * half, p);
        tmem_st16(s_addr + 16 - 16 * half, zeros);
        tc_wait_st();
        tc_fence_before();
        warp_arrive(&c.p_full[buf]);
        if (++buf == kScores) {
          buf = 0;
          ++turn;
        }
      }
      if (!ok) break;
      ok = items == 0 || wait_warp(c, &c.stat_free, (items - 1) & 1, a);
      if (!ok) break;
      c.stat[tid] = make_float2(ref - kUp, sum);
      warp_arrive(&c.stat_full);
      ++items;
    }
  } else if (warp < kSoftmaxWarps + kEndWarps) {
    // ---------------------------------------------------------------- ends of items: Q in, O out; thread = row
    const int row = tid - 32 * kSoftmaxWarps, w = warp - kSoftmaxWarps, head = row & 63, side = row >> 6;
    const uint32_t lanes = uint32_t(w * 32) << 16;
    uint32_t met = 0;
    auto end_sync = [&]() -> bool {                           // the end warps wait for each other (a bounded wait, as all are)
      warp_arrive(&c.ends);
      return wait_warp(c, &c.ends, met++ & 1, a);
    };
    auto copy_q = [&](int item) {                             // into shared memory
      if (item < n_items) {
        const uint8_t* src = static_cast<const uint8_t*>(a.q) + (long long)item * (kH * kDk * 2);
#pragma unroll 4
        for (int x = 0; x < kH * kDk / 8 / 128; ++x) {
          const int i = row + 128 * x, r = i / (kDk / 8), p = i - r * (kDk / 8);
          cp16(smem_u32(c.q) + r * kQRow + p * 16, src + i * 16);
        }
      }
      cp_commit();
    };
    auto q_here = [&]() -> bool {                             // the copy in shared memory is complete
      asm volatile("cp.async.wait_all;" ::: "memory");
      return end_sync();
    };
    const uint4* src = reinterpret_cast<const uint4*>(c.q + head * kQRow);
    int e = 0;                                                // of this row's power of two
    float scale = 0.f;                                        // what the products of its fp16 form are multiplied by
    auto scale_q = [&]() -> bool {
      // Largest magnitudes of 2^9 .. 2^10 (queries below 2^-91 keep less; their products are 0 all the same).  A row and its
      // other half look at half of the head each.
      uint32_t top = 0;                                       // bits of the largest magnitudes of even and odd dims
#pragma unroll 4
      for (int x = 0; x < kDk / 16; ++x) {
        const uint4 y = src[kDk / 16 * side + x];
        top = __vmaxu2(__vmaxu2(__vmaxu2(top, y.x & 0x7fff7fffu), __vmaxu2(y.y & 0x7fff7fffu, y.z & 0x7fff7fffu)), y.w & 0x7fff7fffu);
      }
      c.top[row] = max(top & 0xffffu, top >> 16);
      if (!end_sync()) return false;
      e = max(int(max(c.top[row], c.top[row ^ 64]) >> 7) - 127 - 9, -100);
      // (above 0 whatever the exponents: -inf of keys that are not there is multiplied by it.  Where the bound counts, products of at
      // most 2^30 with the true factor are 0 beside any logit.)
      scale = fminf(fmaxf(ldexpf(a.scale * log2e * a.k_up, e), 1e-37f), 3e38f);
      return true;
    };
    // Words 16 b .. 16 b + 15 of the row, as they are or as fp16.
    auto words = [&](int b, bool half, uint32_t (&r)[16]) {
      const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint4 y = src[4 * b + x];
        const uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          r[4 * x + i] = half ? pack_f16(__uint_as_float(u[i] << 16) * down, __uint_as_float(u[i] & 0xffff0000u) * down) : u[i];
      }
    };
    // The next query into TMEM, as fp16 (i = 0) or as it is (1), as soon as nobody reads the last one there.
    auto store_q = [&](int i, bool wait, uint32_t phase) -> bool {
      const uint32_t to = tmem + lanes + (i == 0 ? kQhCol : kQbCol);
      uint32_t r[16];
      words(0, i == 0, r);
      if (wait && !wait_warp(c, &c.q_empty[i], phase, a)) return false;
      tc_fence_after();
      tmem_st16(to, r);
#pragma unroll 1
      for (int b = 1; b < 6; ++b) {
        words(b, i == 0, r);
        tmem_st16(to + 16 * b, r);
      }
      tc_wait_st();
      tc_fence_before();
      warp_arrive(&c.q_full[i]);
      return true;
    };
    uint32_t items = 0;
    bool ok = true;
    if (item0 < n_items) {
      copy_q(item0);
      ok = q_here() && scale_q();
      c.q_scale[0][row] = scale;
      ok = ok && store_q(0, false, 0) && store_q(1, false, 0) && end_sync();
      copy_q(item0 + step);                                   // (later ones when the exchange is over)
    }
    for (int item = item0; item < n_items && ok; item += step, ++items) {
      if (item + step < n_items) {
        if (!q_here() || !scale_q()) break;
        // (its scales lie where those of the item before this one lay, whose softmax is over)
        c.q_scale[(items + 1) & 1][row] = scale;
        if (!store_q(0, true, items & 1) || !store_q(1, true, items & 1)) break;
      }
      if (!wait_warp(c, &c.stat_full, items & 1, a)) break;
      const float2 mine = c.stat[row], theirs = c.stat[row ^ 64];
      warp_arrive(&c.stat_free);
      const float top = fmaxf(mine.x, theirs.x);
      const float weight = mine.x == -INFINITY ? 0.f : ex2(mine.x - top);
      const float sum = mine.y * weight + theirs.y * (theirs.x == -INFINITY ? 0.f : ex2(theirs.x - top));
      const bool none = sum == 0.f;                           // no key: O may hold anything
      const float f = ncta > 1 ? weight : weight * (a.v_up / sum);
      if (!wait_warp(c, &c.o_last, items & 1, a)) break;
      tc_fence_after();
      // A thread ends with 64 columns of its head: it gives its part of the others to its partner of the other half.  O is free
      // for the next item as soon as this thread's columns are in registers.
      if (!end_sync()) break;                                 // the next query has been read: x lies where it lay
      uint32_t o[64];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t y[32];
        tmem_ld32(y, tmem + lanes + kOCol + 64 * (1 - side) + 32 * b);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(c.x + row * kXRow + 32 * b + 4 * j) =
              make_float4(__uint_as_float(y[4 * j]) * f, __uint_as_float(y[4 * j + 1]) * f, __uint_as_float(y[4 * j + 2]) * f,
                          __uint_as_float(y[4 * j + 3]) * f);
      }
      tmem_ld64(o, tmem + lanes + kOCol + 64 * side);
      tc_fence_before();
      warp_arrive(&c.o_free);
      if (!end_sync()) break;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float4 z = *reinterpret_cast<const float4*>(c.x + (row ^ 64) * kXRow + 4 * j);
        o[4 * j] = __float_as_uint(__fmaf_rn(__uint_as_float(o[4 * j]), f, z.x));
        o[4 * j + 1] = __float_as_uint(__fmaf_rn(__uint_as_float(o[4 * j + 1]), f, z.y));
        o[4 * j + 2] = __float_as_uint(__fmaf_rn(__uint_as_float(o[4 * j + 2]), f, z.z));
        o[4 * j + 3] = __float_as_uint(__fmaf_rn(__uint_as_float(o[4 * j + 3]), f, z.w));
      }
      if (none) {
#pragma unroll
        for (int j = 0; j < 64; ++j) o[j] = 0u;
      }
      if (ncta > 1) {
        uint4* part = reinterpret_cast<uint4*>(reinterpret_cast<float*>(c.k) + head * kPRow + 64 * side);
#pragma unroll
        for (int j = 0; j < 16; ++j) part[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
      } else {
        if (!end_sync()) break;                               // what was given has been read
        // the warp's 32 rows of 128 bytes as whole pieces of lines, through its part of x
        uint4* turn = reinterpret_cast<uint4*>(c.x + w * 32 * kXRow);
        auto at = [&](int r, int p) -> uint4& { return turn[r * 8 + (p ^ (r & 7))]; };
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = pack_bf16(__uint_as_float(o[8 * p + 2 * i]), __uint_as_float(o[8 * p + 2 * i + 1]));
          at(lane, p) = make_uint4(y[0], y[1], y[2], y[3]);
        }
        __syncwarp();
        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + ((long long)item * kH + (w & 1) * 32) * kDv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = 4 * j + (lane >> 3);
          out[r * (kDv / 8) + 8 * side + (lane & 7)] = at(r, lane & 7);
        }
        if (!end_sync()) break;                               // and x is free again
        copy_q(item + 2 * step);
      }
      if (ncta > 1) {
        cluster_wait();                                       // the peers have begun
        joined = true;
        const int own = head / (kH / ncta);
        if (side == 0) {
          const uint32_t to = dsmem_addr(&c.part[crank * (kH / ncta) + head % (kH / ncta)], uint32_t(own));
          dsmem_st_v2(to, top, sum);
        }
      } else if (a.lse != nullptr && side == 0) {
        a.lse[(long long)item * kH + head] = none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      }
    }
  } else if (warp != kScoresWarp && warp != kValuesWarp) {
    // ---------------------------------------------------------------- producers: 16 rows of every second tile a warp
    // (Eight warps on the same tile spent most of it on the latencies of its steps.)
    const int pw = warp - kSoftmaxWarps - kEndWarps, group = pw / kGroupWarps, w = pw % kGroupWarps;
    const int nt = range.last - range.first, main_end = min(range.window, range.last);   // tiles of an item, end of its entries'
    // The group's tiles are every second one of all items'.  A tile's entries are copied while the group waits for its turn, its
    // indices kIndexAhead turns before that.  (Either as loads into registers was slower: they take their lines in an L1 that has
    // few beside this much shared memory.)
    struct Place {
      int item, t, start;                      // start: the group's first tile of the item
    };
    auto next_item = [&](Place& p) {
      p.item += step;
      p.t = p.start = range.first + ((p.start - range.first + nt) & 1);
    };
    auto next_main = [&](Place& p) {           // the group's next tile of entries
      p.t += kGroups;
      while (p.t >= main_end && p.item < n_items) next_item(p);
    };
    const int my_slot = kRows * w + (lane & 15);              // (+ 64 t: of tile t)
    auto copy_index = [&](int n, Place p) {    // of the n-th tile of entries, lanes 0..15
      const int slot = my_slot + p.t * kTile;
      if (lane < kRows && p.item < n_items && slot < a.topk)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&c.index[pw][n % kIndexRing][lane])),
                     "l"(a.idx + (long long)p.item * a.topk + slot)
                     : "memory");
    };
    // Piece i = 32 x + lane of the warp's 16 rows of 12 pieces is of row r = i / 12: it lies 16 (i - 12 r) bytes into entry r, and goes
    // 16 (i + r) bytes into the padded rows.
    const uint32_t packed = smem_u32(c.packed[pw]) + 16 * lane;
    uint32_t rows_of = 0;                      // r of x = 0..5, 4 bits each
#pragma unroll
    for (int x = 0; x < 6; ++x) rows_of |= uint32_t((32 * x + lane) / 12) << (4 * x);
    uint32_t there = 0;                        // the copied tile's rows that are there
    int last_item = -1;                        // whose sequence's cache this is
    const uint8_t* cache = a.kv + 16 * lane;
    auto fetch = [&](Place p, int e) {
      if (lane >= kRows || p.item >= n_items || my_slot + p.t * kTile >= a.topk) e = -1;
      if (e >= a.n_entries) {
        report(a.err, kErrBadIndex, e);
        e = -1;
      }
      there = __ballot_sync(0xffffffffu, e >= 0);
      if (p.item != last_item && p.item < n_items) {
        last_item = p.item;
        cache = a.kv + (long long)(p.item / a.seq_div) * a.n_entries * kEntry + 16 * lane;
      }
#pragma unroll
      for (int x = 0; x < 6; ++x) {
        const int r = (rows_of >> (4 * x)) & 15, entry = __shfl_sync(0xffffffffu, e, r);
        const uint8_t* src = cache + (long long)(max(entry, 0) - r) * kEntry + 512 * x;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(packed + 16 * r + 512 * x), "l"(src), "r"(entry >= 0 ? 16u : 0u)
                     : "memory");
      }
    };
    // the tile in hand, the entries to copy next, the indices to copy next
    Place here{item0, range.first + group, range.first + group}, next, next_index;
    while (here.t >= range.last && here.item < n_items) next_item(here);
    next = here;
    while (next.t >= main_end && next.item < n_items) next_item(next);
    next_index = next;
    int n_index = 0, n_fetch = 0;              // their places among the group's tiles of entries
    for (int j = 0; j < kIndexAhead; ++j) {
      copy_index(n_index++, next_index);
      next_main(next_index);
    }
    cp_commit();
    auto copy_next = [&]() {                   // (every copy of this warp has landed)
      fetch(next, c.index[pw][n_fetch % kIndexRing][lane & 15]);
      next_main(next);
      ++n_fetch;
      copy_index(n_index++, next_index);
      next_main(next_index);
      cp_commit();
    };
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    copy_next();
    const int r8 = lane & 7, q4 = lane >> 3;
    const uint32_t pick = q4 < 2 ? 0x4420u : 0x4431u;   // bytes 0 and 2, or 1 and 3, of four
    // byte offsets of this lane's pieces 4 (k % 2) + q4 of a stage's row 16 w + r8
    const uint32_t even = (kRows * w + r8) * 128 + ((q4 ^ r8) << 4), odd = (kRows * w + r8) * 128 + (((4 + q4) ^ r8) << 4);
    uint32_t st = uint32_t(group) % kStages, lap = uint32_t(group) / kStages, waits = 0;
    int n_item = -1, ns = 0;
    bool ok = true;
    while (here.item < n_items) {
      const bool window = here.t >= range.window;
      ok = wait_warp(c, &c.empty[st], (lap & 1) ^ 1, a);
      if (!ok) break;
      const uint32_t k_st = smem_u32(c.k[st]), v_st = smem_u32(c.v[st]);
      if (window) {
        // window rows lie one behind the other: the group's first warp has them copied by TMA, the others only count the tile
        if (w == 0 && here.item != n_item) {
          n_item = here.item;
          ns = clamp_count(a.n_swa[n_item], a.swa, lane == 0 ? a.err : nullptr);
        }
        const int row0 = (here.t - range.window) * kTile;
        const int n = min(max(ns - row0, 0), kTile), y = here.item * a.swa + row0;
        if (w > 0) {
          warp_arrive(&c.full[st]);
        } else {
          uint64_t* bar = n == kTile ? &c.full[st] : &c.window[group];
          if (lane == 0) {
            c.mask[st] = n == kTile ? ~0ull : (1ull << n) - 1ull;
            if (n > 0) {
              mbar_arrive_expect_tx(bar, kKBytes + kVBytes);
#pragma unroll
              for (int b = 0; b < kDk / 64; ++b) load_box(k_st + b * (kTile * 128), &k_map, 64 * b, y, bar);
#pragma unroll
              for (int b = 0; b < kDv / 64; ++b) load_box(v_st + b * (kTile * 128), &v_map, 64 * b, y, bar);
            }
            if (here.item + step < n_items) {  // the next item's, which would come from memory (2 us)
              const int far = y + step * a.swa;
#pragma unroll
              for (int b = 0; b < kDk / 64; ++b) prefetch_box(&k_map, 64 * b, far);
#pragma unroll
              for (int b = 0; b < kDv / 64; ++b) prefetch_box(&v_map, 64 * b, far);
            }
          }
          __syncwarp();
          if (n < kTile) {                     // values behind the count are zeroed: they meet weights of 0, and might be NaN
            ok = n == 0 || wait_warp(c, &c.window[group], waits++ & 1, a);
            if (!ok) break;
            for (int i = lane; i < (kTile - n) * 16; i += 32) {
              const int r = n + (i >> 4), p = i & 15;
              *reinterpret_cast<uint4*>(c.v[st] + (p >> 3) * (kTile * 128) + r * 128 + (p & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            warp_arrive(&c.full[st]);
          }
        }
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          // (all loads before the first store, which they would otherwise wait for)
          const uint8_t* src = c.packed[pw] + (8 * hf + r8) * kPackedRow;
          uint32_t word[10], four[5];
          __half2 two[5];                      // the scales of groups 4 k + q4 / 2 and 2 behind it
#pragma unroll
          for (int k = 0; k < 5; ++k) four[k] = reinterpret_cast<const uint32_t*>(src + kScales)[k];
#pragma unroll
          for (int k = 0; k < 10; ++k) word[k] = reinterpret_cast<const uint32_t*>(src)[4 * k + q4];
#pragma unroll
          for (int k = 0; k < 5; ++k) two[k] = kv4_scales(__byte_perm(four[k], 0, pick));
#pragma unroll
          for (int k = 0; k < 10; ++k) {       // words 4 k + q4: 0..23 of the key, 24..39 of the value
            const __half2 scale = k & 1 ? __high2half2(two[k >> 1]) : __low2half2(two[k >> 1]);
            __half2 x[4];
            kv4_pairs(word[k], x);
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] = __hmul2(x[i], scale);
              y[i] = *reinterpret_cast<const uint32_t*>(&x[i]);
            }
            const uint32_t to = (k < 6 ? k_st + (k >> 1) * (kTile * 128) : v_st + ((k - 6) >> 1) * (kTile * 128)) + (k & 1 ? odd : even) + hf * 1024;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
          }
        }
        if (lane == 0) reinterpret_cast<uint16_t*>(&c.mask[st])[w] = uint16_t(there);
        warp_arrive(&c.full[st]);              // (and every lane has read the packed entries)
        copy_next();
      }
      here.t += kGroups;
      while (here.t >= range.last && here.item < n_items) next_item(here);
      st += kGroups;
      if (st >= kStages) {
        st -= kStages;
        ++lap;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---------------------------------------------------------------- MMA issue: scores by one warp, values by another
    // (One warp for both left the tensor cores idle while it looked at its barriers: 1,680 cycles a tile.)
    constexpr uint32_t qk_h = idesc_f16(128, kTile, false), pv_h = idesc_f16(128, kDv, true);
    constexpr uint32_t qk_b = idesc_bf16(128, kTile, false), pv_b = idesc_bf16(128, kDv, true);
    const bool scores = warp == kScoresWarp;
    const uint64_t k0 = smem_desc(smem_u32(c.k[0]), 16, 1024), v0 = smem_desc(smem_u32(c.v[0]), kTile * 128, 1024);
    uint32_t items = 0, st = 0, lap = 0, buf = 0, turn = 0;   // as above
    bool ok = true;
    for (int item = item0; item < n_items && ok; item += step, ++items) {
      bool first = true;
      if (scores) ok = wait_warp(c, &c.q_full[0], items & 1, a);
      else if (items > 0) ok = wait_warp(c, &c.o_free, (items - 1) & 1, a);   // (of every item, with keys or without)
      bool half = true;                        // the query as fp16 is still wanted
      auto half_done = [&]() -> bool {
        half = false;
        if (elect_one()) tc_commit(&c.q_empty[0]);
        __syncwarp();
        return wait_warp(c, &c.q_full[1], items & 1, a);
      };
      for (int t = range.first; t < range.last && ok; ++t) {
        const uint32_t here = st;
        const bool window = t >= range.window;
        if (scores) {
          if (turn > 0) ok = wait_warp(c, &c.s_free[buf], (turn - 1) & 1, a);   // (S lies where the weights of the third tile before lay)
          ok = ok && wait_warp(c, &c.full[st], lap & 1, a);
        } else {
          ok = wait_warp(c, &c.p_full[buf], turn & 1, a);
        }
        if (!ok) break;
        if (++st == kStages) {
          st = 0;
          ++lap;
        }
        // The rows are generic-proxy writes, which the tensor core reads, and TMA overwrites, by the async proxy.  The fence stands
        // here, behind the wait, and not with the producers: theirs would wait for the copies that are on their way (1.5 us a tile).
        fence_async_smem();
        if (scores) {
          if (window && half) ok = half_done();
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = k0 + here * (kKBytes >> 4);
          const uint32_t q = tmem + (window ? kQbCol : kQhCol), desc = window ? qk_b : qk_h;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kDk / 16; ++k)
              mma_ts(tmem + kSCol + buf * 64, q + 8 * k, kd + ((k >> 2) * (kTile * 128) + (k & 3) * 32) / 16, desc, k > 0);
            tc_commit(&c.s_full[buf]);
          }
        } else {
          tc_fence_after();
          const uint64_t v = v0 + here * (kVBytes >> 4);
          const uint32_t desc = window ? pv_b : pv_h;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              mma_ts(tmem + kOCol, tmem + kSCol + buf * 64 + 8 * k, v + k * (2048 >> 4), desc, !(first && k == 0));
            tc_commit(&c.empty[here]);
            tc_commit(&c.s_free[buf]);
          }
          first = false;
        }
        __syncwarp();
        if (++buf == kScores) {
          buf = 0;
          ++turn;
        }
      }
      if (ok && scores && half) ok = half_done();
      if (!ok) break;
      if (elect_one()) tc_commit(scores ? &c.q_empty[1] : &c.o_last);
      __syncwarp();
    }
    // every MMA has finished before the memory it uses is given up
    if (elect_one()) tc_commit(&c.fin);
    __syncwarp();
    mbar_wait(&c.fin, 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (c.abort) {                               // given up: what may still be on its way, a query here, 10 ms for window rows, whoever asked
    asm volatile("cp.async.wait_all;" ::: "memory");
    const long long t0 = clock64();
    while (clock64() - t0 < 20000000) {
    }
  }
  if (warp == 0) tmem_free(tmem, kTmemCols);
  if (ncta == 1) return;

  // ---------------------------------------------------------------- merge of a split, as in attn.cu
  if (!joined) cluster_wait();
  cluster_sync_all();                          // the tables and partials of every CTA are complete and visible
  const int per = kH / ncta, hb = crank * per;
  float* part = reinterpret_cast<float*>(c.k);               // [kH][kPRow]
  float* weight = part + kH * kPRow;                         // [kMaxCluster][kH]
  if (tid < per) {
    const int h = hb + tid;
    float top = -INFINITY, sum = 0.f;
    for (int r = 0; r < ncta; ++r) top = fmaxf(top, c.part[r * per + tid].x);
    for (int r = 0; r < ncta; ++r) {
      const float2 y = c.part[r * per + tid];
      const float f = y.x == -INFINITY && y.y == 0.f ? 0.f : ex2(y.x - top);   // (a NaN sum stays)
      weight[r * kH + h] = f;
      sum += f * y.y;
    }
    for (int r = 0; r < ncta; ++r) weight[r * kH + h] *= sum == 0.f ? 0.f : a.v_up / sum;
    if (a.lse != nullptr) a.lse[(long long)item0 * kH + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  }
  __syncthreads();
  for (int i = tid; i < per * (kDv / 4); i += kThreads) {
    const int h = hb + i / (kDv / 4), d = i % (kDv / 4) * 4;
    float4 y[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < ncta) y[r] = dsmem_ld_v4f(dsmem_addr(part + h * kPRow + d, uint32_t(r)));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < ncta) {
        const float f = weight[r * kH + h];
        o.x = __fmaf_rn(f, y[r].x, o.x);
        o.y = __fmaf_rn(f, y[r].y, o.y);
        o.z = __fmaf_rn(f, y[r].z, o.z);
        o.w = __fmaf_rn(f, y[r].w, o.w);
      }
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + ((long long)item0 * kH + h) * kDv + d) =
        make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
  }
  cluster_sync_all();                          // every peer has read this CTA's partial
}

}  // namespace

// Rows of `dim` bf16 numbers as boxes of 64 by 64 in the 128-byte swizzle.
static bool window_map(CUtensorMap* map, const void* rows, int dim, long long n) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) == cudaSuccess &&
                    found == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<Encode>(fn) : nullptr;
  }();
  if (encode == nullptr) return false;
  const cuuint64_t size[2] = {cuuint64_t(dim), cuuint64_t(n)}, stride[1] = {cuuint64_t(dim) * 2};
  const cuuint32_t box[2] = {64, kTile}, each[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(rows), size, stride, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_kv4_attn_tc(const Kv4AttnArgs& a, int batch, cudaStream_t st) {
  const cudaError_t e = once_per_device(kSetupKv4Tc, [] {
    return cudaFuncSetAttribute(kv4_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count(), tiles = (a.swa + kTile - 1) / kTile + (a.topk + kTile - 1) / kTile;
  int ncta = 1;
  while (ncta < kMaxCluster && 2 * ncta <= tiles && 2 * ncta * batch <= sms) ncta *= 2;
  const int grid = ncta > 1 || batch < sms ? batch * ncta : sms;
  CUtensorMap k_map{}, v_map{};
  if (a.swa > 0 && !(window_map(&k_map, a.k_swa, kDk, (long long)batch * a.swa) && window_map(&v_map, a.v_swa, kDv, (long long)batch * a.swa)))
    return cudaErrorInvalidValue;
  note_launch();
  return launch_pdl(kv4_tc_kernel, dim3(unsigned(grid)), dim3(kThreads), kSmem, st, unsigned(ncta), a, batch, ncta, k_map, v_map);
}

}  // namespace csa2
