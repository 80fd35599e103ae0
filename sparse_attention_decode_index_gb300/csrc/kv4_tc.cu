// Sparse attention over a packed main cache (kv4.cuh) on the 5th-generation tensor
// cores (bf16, 64 heads sharing one KV head, dk 192, dv 128).
//
// A query's keys come in tiles of 64: its window rows first, then its selected
// entries.  Code * scale is exact in fp16, so that an entry's row becomes fp16 and its
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
// Roles of a CTA (17 warps):
//   4 softmax warps: a thread owns a row; P goes back to TMEM over its S.  O is rescaled only when a
//     maximum grows by more than 2^8;
//   4 end warps put the next query into TMEM (as bf16 and as fp16) and write the last one's O out;
//   8 producer warps: each fetches 8 of a tile's packed entries (192 bytes, 12 pieces)
//     several tiles ahead, and turns them into a stage's K and V rows (K-major, MN-major, 128-byte swizzled):
//     lane l takes row l % 8 and the words l / 8, + 4, ... of 8 codes, which meets no bank twice;
//   1 warp issues S = Q K^T and, a tile later, O += P V.
// Many queries: persistent, a CTA an SM.  Few: a query's tiles are split over a
// cluster of up to 8 CTAs, whose partial O are merged through distributed shared memory as in attn.cu.
//
// P is rounded to fp16 (entries) or bf16 (window) as the tensor core asks for; the weights' sums stay fp32 and unrounded.
#include "kv4.cuh"
#include "tc.cuh"

namespace csa2 {

namespace {

constexpr int kH = 64, kDk = 192, kDv = 128;
constexpr int kTile = 64;                      // keys a stage
constexpr int kEntry = kv4_bytes(kDk, kDv);    // 192: codes 0..159, scales 160..179
constexpr int kScales = 160;
constexpr int kKBytes = kTile * kDk * 2, kVBytes = kTile * kDv * 2;
constexpr int kStages = 3;
constexpr int kAhead = 4;                      // tiles of packed entries on their way
constexpr int kSoftmaxWarps = 4, kEndWarps = 4, kProducerWarps = 8;
constexpr int kRows = kTile / kProducerWarps;  // entries of a producer warp: 8
constexpr int kPackedRow = kEntry + 16;        // padded: rows of 4 lanes' words meet no bank twice
constexpr int kThreads = 32 * (kSoftmaxWarps + kEndWarps + kProducerWarps + 1);
constexpr int kMaxCluster = 8;
constexpr int kQRow = kDk * 2 + 16;            // query rows on their way to TMEM
constexpr int kXRow = 36;                      // fp32 columns of a row that the halves exchange, padded
constexpr int kPRow = kDv + 4;                 // partial O of a split
// Weights are held as 2^7 times their relation to their row's exponent: at most 2^15, as that grows by steps of 2^8, which
// fp16 holds, and rounded by 2^-12 of themselves or, below 2^-21, by 2^-32 of the greatest.
constexpr float kUp = 7.f;
constexpr uint32_t kTmemCols = 512;            // a power of two over O (128), two S (64 each), Q as fp16 and as bf16 (96 each)
constexpr uint32_t kOCol = 0, kSCol = 128, kQhCol = 256, kQbCol = 352;

struct Shared {
  uint8_t k[kStages][kKBytes];                 // 3 blocks of 64 dims: 64 rows of 128 bytes
  uint8_t v[kStages][kVBytes];                 // 2 blocks of 64 dims: 64 keys of 128 bytes
  uint8_t packed[kProducerWarps][kAhead][kRows * kPackedRow];
  uint8_t q[kH * kQRow];
  float x[128 * kXRow];
  uint64_t mask[kStages];                      // the tile's keys that are there
  float2 stat[128];                            // (exponent, sum) of the rows of an item
  float q_scale[2][128];                       // what a row's fp16 products are multiplied by, of even and odd items
  float2 part[kMaxCluster][kH];                // (exponent, sum) of the CTAs of a split, of the heads that this one adds up
  uint64_t full[kStages], empty[kStages];      // a tile has landed; has been used
  uint64_t s_full[2], p_full[2];               // S has been computed; P has been written
  uint64_t o_done, o_last, o_free;             // O holds a tile more; the item's last; has been read
  uint64_t q_full, q_empty, stat_full, stat_free;
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

CSA2_DEV void cp16(uint32_t dst, const uint8_t* src, const void* any) {   // src null: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src != nullptr ? src : any), "r"(src != nullptr ? 16u : 0u)
               : "memory");
}
CSA2_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
CSA2_DEV uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The tiles of a query that CTA `rank` of `n` takes.
struct Range {
  int first, last, window;                     // [first, last) of a query's tiles; how many are the window's
  CSA2_DEV Range(const Kv4AttnArgs& a, int rank, int n) {
    window = (a.swa + kTile - 1) / kTile;
    const int all = window + (a.topk + kTile - 1) / kTile;
    first = all * rank / n;
    last = all * (rank + 1) / n;
  }
};

__global__ void __launch_bounds__(kThreads, 1) kv4_tc_kernel(const Kv4AttnArgs a, int n_items, int ncta) {
  extern __shared__ uint8_t raw[];
  Shared& c = *reinterpret_cast<Shared*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int crank = ncta > 1 ? int(cluster_rank()) : 0;
  const int item0 = int(blockIdx.x) / ncta, step = int(gridDim.x) / ncta;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&c.full[i], 33 * kProducerWarps);              // every lane's rows, every warp's mask
      mbar_init(&c.empty[i], 1 + kSoftmaxWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.s_full[b], 1);
      mbar_init(&c.p_full[b], 128);
    }
    mbar_init(&c.o_done, 1);
    mbar_init(&c.o_last, 1);
    mbar_init(&c.o_free, 128);
    mbar_init(&c.q_full, 128);
    mbar_init(&c.q_empty, 1);
    mbar_init(&c.stat_full, 128);
    mbar_init(&c.stat_free, 128);
    mbar_init(&c.ends, kEndWarps);
    mbar_init(&c.fin, 1);
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
    uint32_t tiles = 0, items = 0, st = 0, lap = 0;           // tiles that have keys, so far
    bool ok = true;
    for (int item = item0; item < n_items && ok; item += step) {
      float ref = -INFINITY, sum = 0.f;        // the exponent that P and O are relative to, and the weights' sum
      bool first = true;
      for (int t = range.first; t < range.last; ++t) {
        ok = tc_wait_warp(c, &c.full[st], lap & 1, a.err);
        if (!ok) break;
        const uint64_t all = c.mask[st];
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.empty[st]);
        if (++st == kStages) {
          st = 0;
          ++lap;
        }
        if (all == 0) continue;
        const uint32_t mask = uint32_t(all >> (32 * half));
        const bool window = t < range.window;
        const uint32_t buf = tiles & 1, s_addr = tmem + lanes + kSCol + buf * 64;
        ok = tc_wait_warp(c, &c.s_full[buf], (tiles >> 1) & 1, a.err);
        if (!ok) break;
        tc_fence_after();
        uint32_t p[16];
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
            // O holds tiles up to the one before: wait for it.  (S of this tile comes behind O of the last but one,
            // so that the barrier is in the phase of the last or behind it, and the parity tells which.)
            ok = tc_wait_warp(c, &c.o_done, (tiles - 1) & 1, a.err);
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
            p[j] = window ? pack_bf16(x.x * window_up, x.y * window_up) : pack_f16(x.x, x.y);
          }
          total = add2(total, other);
          sum += total.x + total.y;
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) p[j] = 0;
          // Another half's tile may come first: O is then 0 times anything, and this row's exponent is still open.
        }
        first = false;
        uint32_t zero[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) zero[j] = 0;
        tmem_st16(s_addr + 16 * half, p);
        tmem_st16(s_addr + 16 * (1 - half), zero);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&c.p_full[buf]);
        ++tiles;
      }
      if (!ok) break;
      ok = items == 0 || tc_wait_warp(c, &c.stat_free, (items - 1) & 1, a.err);
      if (!ok) break;
      c.stat[tid] = make_float2(ref - kUp, sum);
      mbar_arrive(&c.stat_full);
      ++items;
    }
  } else if (warp < kSoftmaxWarps + kEndWarps) {
    // ---------------------------------------------------------------- ends of items: Q in, O out; thread = row
    const int row = tid - 32 * kSoftmaxWarps, w = warp - kSoftmaxWarps, head = row & 63, side = row >> 6;
    const uint32_t lanes = uint32_t(w * 32) << 16;
    uint32_t met = 0;
    auto end_sync = [&]() -> bool {                           // the end warps wait for each other (a bounded wait, as all are)
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.ends);
      return tc_wait_warp(c, &c.ends, met++ & 1, a.err);
    };
    auto copy_q = [&](int item) {                             // into shared memory
      if (item < n_items) {
        const uint8_t* src = static_cast<const uint8_t*>(a.q) + (long long)item * (kH * kDk * 2);
#pragma unroll
        for (int x = 0; x < kH * kDk / 8 / 128; ++x) {
          const int i = row + 128 * x, r = i / (kDk / 8), p = i - r * (kDk / 8);
          cp16(smem_u32(c.q) + r * kQRow + p * 16, src + i * 16, nullptr);
        }
      }
      cp_commit();
    };
    auto store_q = [&](uint32_t parity) -> bool {             // into TMEM
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!end_sync()) return false;
      const uint4* src = reinterpret_cast<const uint4*>(c.q + head * kQRow);
      uint32_t top = 0;                                       // bits of the largest magnitude
#pragma unroll 1
      for (int b = 0; b < 6; ++b) {
        uint32_t r[16];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint4 y = src[4 * b + x];
          r[4 * x] = y.x, r[4 * x + 1] = y.y, r[4 * x + 2] = y.z, r[4 * x + 3] = y.w;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) top = max(top, max(r[x] & 0x7fffu, (r[x] >> 16) & 0x7fffu));
        tmem_st16(tmem + lanes + kQbCol + 16 * b, r);
      }
      // largest magnitudes of 2^9 .. 2^10 (queries below 2^-91 keep less; their products are 0 all the same)
      const int e = max(int(top >> 7) - 127 - 9, -100);
      const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll 1
      for (int b = 0; b < 6; ++b) {
        uint32_t r[16];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint4 y = src[4 * b + x];
          const uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            r[4 * x + i] = pack_f16(__uint_as_float(u[i] << 16) * down, __uint_as_float(u[i] & 0xffff0000u) * down);
        }
        tmem_st16(tmem + lanes + kQhCol + 16 * b, r);
      }
      c.q_scale[parity][row] = fminf(ldexpf(a.scale * log2e * a.k_up, e), 3e38f);
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(&c.q_full);
      return end_sync();                                      // the copy in shared memory has been read
    };
    uint32_t items = 0;
    bool ok = true;
    if (item0 < n_items) {
      copy_q(item0);
      ok = store_q(0);
      copy_q(item0 + step);
    }
    for (int item = item0; item < n_items && ok; item += step, ++items) {
      if (item + step < n_items) {
        // (its scales lie where those of the item before this one lay, whose softmax is over)
        if (!tc_wait_warp(c, &c.q_empty, items & 1, a.err)) break;
        tc_fence_after();
        if (!store_q((items + 1) & 1)) break;
        copy_q(item + 2 * step);
      }
      if (!tc_wait_warp(c, &c.stat_full, items & 1, a.err)) break;
      const float2 mine = c.stat[row], theirs = c.stat[row ^ 64];
      mbar_arrive(&c.stat_free);
      const float top = fmaxf(mine.x, theirs.x);
      const float weight = mine.x == -INFINITY ? 0.f : ex2(mine.x - top);
      const float sum = mine.y * weight + theirs.y * (theirs.x == -INFINITY ? 0.f : ex2(theirs.x - top));
      const bool none = sum == 0.f;                           // no key: O may hold anything
      const float f = ncta > 1 ? weight : weight * (a.v_up / sum);
      if (!tc_wait_warp(c, &c.o_last, items & 1, a.err)) break;
      tc_fence_after();
      // a thread ends with 64 columns of its head: it gives its part of the others to its partner of the other half
#pragma unroll 1
      for (int b = 0; b < 2 && ok; ++b) {
        uint32_t o[32];
        tmem_ld32(o, tmem + lanes + kOCol + 64 * (1 - side) + 32 * b);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(c.x + row * kXRow + 4 * j) =
              make_float4(__uint_as_float(o[4 * j]) * f, __uint_as_float(o[4 * j + 1]) * f, __uint_as_float(o[4 * j + 2]) * f,
                          __uint_as_float(o[4 * j + 3]) * f);
        tmem_ld32(o, tmem + lanes + kOCol + 64 * side + 32 * b);
        if (b == 1) {
          tc_fence_before();
          mbar_arrive(&c.o_free);
        }
        ok = end_sync();
        if (!ok) break;
        float y[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 z = *reinterpret_cast<const float4*>(c.x + (row ^ 64) * kXRow + 4 * j);
          y[4 * j] = none ? 0.f : __fmaf_rn(__uint_as_float(o[4 * j]), f, z.x);
          y[4 * j + 1] = none ? 0.f : __fmaf_rn(__uint_as_float(o[4 * j + 1]), f, z.y);
          y[4 * j + 2] = none ? 0.f : __fmaf_rn(__uint_as_float(o[4 * j + 2]), f, z.z);
          y[4 * j + 3] = none ? 0.f : __fmaf_rn(__uint_as_float(o[4 * j + 3]), f, z.w);
        }
        ok = end_sync();                                      // what was given has been read
        if (!ok) break;
        if (ncta > 1) {
          float* part = reinterpret_cast<float*>(c.k) + head * kPRow + 64 * side + 32 * b;
#pragma unroll
          for (int j = 0; j < 8; ++j) reinterpret_cast<float4*>(part)[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
        } else {
          // the warp's 32 rows of 64 bytes as whole pieces of lines, through its part of x
          uint4* turn = reinterpret_cast<uint4*>(c.x + w * 32 * kXRow);
          auto at = [&](int r, int p) -> uint4& { return turn[r * 4 + (p ^ ((r >> 1) & 3))]; };
#pragma unroll
          for (int p = 0; p < 4; ++p)
            at(lane, p) = make_uint4(pack_bf16(y[8 * p], y[8 * p + 1]), pack_bf16(y[8 * p + 2], y[8 * p + 3]),
                                     pack_bf16(y[8 * p + 4], y[8 * p + 5]), pack_bf16(y[8 * p + 6], y[8 * p + 7]));
          __syncwarp();
          uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + ((long long)item * kH + (w & 1) * 32) * kDv);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + (lane >> 2);
            out[r * (kDv / 8) + 8 * side + 4 * b + (lane & 3)] = at(r, lane & 3);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      if (ncta > 1) {
        cluster_wait();                                       // the peers have begun
        joined = true;
        const int own = head / (kH / ncta);
        if (side == 0) {
          const uint32_t to = dsmem_addr(&c.part[crank][head], uint32_t(own));
          dsmem_st_v2(to, top, sum);
        }
      } else if (a.lse != nullptr && side == 0) {
        a.lse[(long long)item * kH + head] = none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      }
    }
  } else if (warp < kSoftmaxWarps + kEndWarps + kProducerWarps) {
    // ---------------------------------------------------------------- producers: 8 rows of every tile a warp
    const int w = warp - kSoftmaxWarps - kEndWarps;
    const int m0 = max(range.first, range.window) - range.window, nm = max(range.last, range.window) - range.window - m0;
    const uint32_t ring = smem_u32(c.packed[w][0]);
    // the index of this lane's row (lanes 0..7) of main tile i of an item
    auto index_of = [&](int item, int i) -> int {
      const int slot = (m0 + i) * kTile + kRows * w + lane;
      if (lane >= kRows || item >= n_items || slot >= a.topk) return -1;
      return a.idx[(long long)item * a.topk + slot];
    };
    int f_item = item0, f_i = 0;               // the main tile whose indices are loaded next
    auto advance = [&]() {
      if (++f_i == nm) {
        f_i = 0;
        f_item += step;
      }
    };
    uint32_t there = 0;                        // 8 bits for each tile on its way
    auto fetch = [&](int slot, int item, int e) {
      if (e >= a.n_entries) {
        report(a.err, kErrBadIndex, e);
        e = -1;
      }
      there = (there & ~(0xffu << (8 * slot))) | (__ballot_sync(0xffffffffu, e >= 0) & 0xffu) << (8 * slot);
      if (item < n_items) {
        const uint8_t* cache = a.kv + (long long)(item / a.seq_div) * a.n_entries * kEntry;
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          const int p = 32 * x + lane, r = p / 12, part = p - 12 * r;
          const int entry = __shfl_sync(0xffffffffu, e, r);
          cp16(ring + slot * (kRows * kPackedRow) + r * kPackedRow + 16 * part,
               entry >= 0 ? cache + (long long)entry * kEntry + 16 * part : nullptr, a.kv);
        }
      }
      cp_commit();                             // (possibly of nothing: the groups count the tiles)
    };
    int e = -1, e_item = n_items;              // the indices of the tile to fetch next
    if (nm > 0) {
      int es[kAhead], its[kAhead];             // (their loads together)
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        its[j] = f_item;
        es[j] = index_of(f_item, f_i);
        advance();
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) fetch(j, its[j], es[j]);
      e_item = f_item;
      e = index_of(f_item, f_i);
      advance();
    }
    uint32_t st = 0, lap = 0;
    int slot = 0;
    const int r8 = lane & 7, q4 = lane >> 3;
    // byte offsets of this lane's pieces 4 (k % 2) + q4 of a stage's row 8 w + r8
    const uint32_t even = (kRows * w + r8) * 128 + ((q4 ^ r8) << 4), odd = (kRows * w + r8) * 128 + (((4 + q4) ^ r8) << 4);
    bool ok = true;
    int n_next = item0 < n_items ? a.n_swa[item0] : 0;
    for (int item = item0; item < n_items && ok; item += step) {
      const int ns = clamp_count(n_next, a.swa, w == 0 && lane == 0 && crank == 0 ? a.err : nullptr);
      if (item + step < n_items) n_next = a.n_swa[item + step];
      for (int t = range.first; t < range.last; ++t) {
        ok = tc_wait_warp(c, &c.empty[st], (lap & 1) ^ 1, a.err);
        if (!ok) break;
        const uint32_t k_st = smem_u32(c.k[st]), v_st = smem_u32(c.v[st]);
        uint8_t* mask = reinterpret_cast<uint8_t*>(&c.mask[st]) + w;
        if (t < range.window) {
          const int row0 = t * kTile + kRows * w;             // of the window
          const long long base = (long long)item * a.swa + row0;
#pragma unroll
          for (int x = 0; x < 10; ++x) {
            const int p = 32 * x + lane, r = p / 40, part = p - 40 * r;
            const bool key = part < 24, has = row0 + r < ns;
            const int y = key ? part : part - 24;
            const uint8_t* src = key ? static_cast<const uint8_t*>(a.k_swa) + (base + r) * (kDk * 2)
                                     : static_cast<const uint8_t*>(a.v_swa) + (base + r) * (kDv * 2);
            cp16((key ? k_st : v_st) + (y >> 3) * (kTile * 128) + (kRows * w + r) * 128 + (((y & 7) ^ r) << 4),
                 has ? src + 16 * y : nullptr, a.kv);
          }
          if (lane == 0) {
            *mask = uint8_t((1u << min(max(ns - row0, 0), kRows)) - 1u);
            mbar_arrive(&c.full[st]);
          }
          cp_arrive(&c.full[st]);
        } else {
          asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
          __syncwarp();
          const uint8_t* src = c.packed[w][slot] + r8 * kPackedRow;
          const uint32_t* codes = reinterpret_cast<const uint32_t*>(src) + q4;
          const uint32_t* scales = reinterpret_cast<const uint32_t*>(src + kScales);
#pragma unroll
          for (int k = 0; k < 10; ++k) {                      // words 4 k + q4: 0..23 of the key, 24..39 of the value
            const uint32_t pair = scales[k >> 1] >> (8 * (q4 >> 1));   // groups 2 k + q4 / 2, k even and odd
            const __half2 scale = __half2half2(kv4_scale(uint8_t(k & 1 ? pair >> 16 : pair)));
            const uint32_t word = codes[4 * k];
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __half2 h = __hmul2(kv4_pair(uint8_t(word >> (8 * i))), scale);
              y[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            const uint32_t to = (k < 6 ? k_st + (k >> 1) * (kTile * 128) : v_st + ((k - 6) >> 1) * (kTile * 128)) + (k & 1 ? odd : even);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
          }
          if (lane == 0) {
            *mask = uint8_t(there >> (8 * slot));
            mbar_arrive(&c.full[st]);
          }
          fence_async_smem();
          mbar_arrive(&c.full[st]);
          __syncwarp();                        // every lane has read the packed entries
          fetch(slot, e_item, e);
          e_item = f_item;
          e = index_of(f_item, f_i);
          advance();
          slot = (slot + 1) % kAhead;
        }
        if (++st == kStages) {
          st = 0;
          ++lap;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---------------------------------------------------------------- MMA issue
    constexpr uint32_t qk_h = idesc_f16(128, kTile, false), pv_h = idesc_f16(128, kDv, true);
    constexpr uint32_t qk_b = idesc_bf16(128, kTile, false), pv_b = idesc_bf16(128, kDv, true);
    const uint64_t k0 = smem_desc(smem_u32(c.k[0]), 16, 1024), v0 = smem_desc(smem_u32(c.v[0]), kTile * 128, 1024);
    uint32_t tiles = 0, items = 0, st = 0, lap = 0;
    bool ok = true;
    for (int item = item0; item < n_items && ok; item += step) {
      bool pending = false, first = true, was_window = false;   // a tile whose O is to be added
      uint32_t was_st = 0;
      auto pv = [&]() -> bool {
        const uint32_t x = tiles - 1, buf = x & 1;
        if (first && items > 0 && !tc_wait_warp(c, &c.o_free, (items - 1) & 1, a.err)) return false;
        if (!tc_wait_warp(c, &c.p_full[buf], (x >> 1) & 1, a.err)) return false;
        tc_fence_after();
        const uint64_t v = v0 + was_st * (kVBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_ts(tmem + kOCol, tmem + kSCol + buf * 64 + 8 * k, v + k * (2048 >> 4), was_window ? pv_b : pv_h, !(first && k == 0));
          tc_commit(&c.empty[was_st]);
          tc_commit(&c.o_done);
        }
        __syncwarp();
        first = false;
        return true;
      };
      ok = tc_wait_warp(c, &c.q_full, items & 1, a.err);
      for (int t = range.first; t < range.last && ok; ++t) {
        ok = tc_wait_warp(c, &c.full[st], lap & 1, a.err);
        if (!ok) break;
        const uint64_t mask = c.mask[st];
        const uint32_t here = st;
        if (++st == kStages) {
          st = 0;
          ++lap;
        }
        if (mask == 0) {                       // no key: nobody looks at it
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.empty[here]);
          if (pending) ok = pv();              // (its stage may be what the next tile waits for)
          pending = false;
          continue;
        }
        fence_async_smem();                    // the window's copies are generic-proxy writes, the tensor core reads by the async proxy
        tc_fence_after();
        const bool window = t < range.window;
        const uint32_t buf = tiles & 1, q = tmem + (window ? kQbCol : kQhCol), desc = window ? qk_b : qk_h;
        const uint64_t kd = k0 + here * (kKBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kDk / 16; ++k)
            mma_ts(tmem + kSCol + buf * 64, q + 8 * k, kd + ((k >> 2) * (kTile * 128) + (k & 3) * 32) / 16, desc, k > 0);
          tc_commit(&c.s_full[buf]);
        }
        __syncwarp();
        if (pending) ok = pv();
        pending = true;
        was_st = here;
        was_window = window;
        ++tiles;
      }
      if (!ok) break;
      if (elect_one()) tc_commit(&c.q_empty);
      __syncwarp();
      if (pending) ok = pv();
      if (!ok) break;
      if (elect_one()) tc_commit(&c.o_last);
      __syncwarp();
      ++items;
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
    for (int r = 0; r < ncta; ++r) top = fmaxf(top, c.part[r][h].x);
    for (int r = 0; r < ncta; ++r) {
      const float2 y = c.part[r][h];
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

cudaError_t launch_kv4_attn_tc(const Kv4AttnArgs& a, int batch, cudaStream_t st) {
  const cudaError_t e = once_per_device(kSetupKv4Tc, [] {
    return cudaFuncSetAttribute(kv4_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count(), tiles = (a.swa + kTile - 1) / kTile + (a.topk + kTile - 1) / kTile;
  int ncta = 1;
  while (ncta < kMaxCluster && 2 * ncta <= tiles && 2 * ncta * batch <= sms) ncta *= 2;
  const int grid = ncta > 1 || batch < sms ? batch * ncta : sms;
  note_launch();
  return launch_pdl(kv4_tc_kernel, dim3(unsigned(grid)), dim3(kThreads), kSmem, st, unsigned(ncta), a, batch, ncta);
}

}  // namespace csa2
