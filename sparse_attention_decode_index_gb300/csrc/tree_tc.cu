// Attention of drafted trees on the 5th-generation tensor cores, for batches
// that fill the GPU (bf16, 64 heads sharing one KV head, dk 192, dv 128).
//
// The drafted tokens of a sequence are neighbours: their Top-K lists overlap
// and their windows are nearly the same.  One CTA therefore attends with up to
// 2 or 4 tokens of a sequence at once, over the union of their keys, and masks
// each key to the tokens that have it: a key that several tokens select is
// gathered once.  The gather sets the time of this attention (the load path of
// an SM takes about 34 bytes a cycle of 16-byte cp.async pieces, 12,000 cycles
// for the 640 keys of one query), and the tensor cores' rows come in 128s,
// which two tokens' 64 heads fill, so that attending two tokens to a key that
// only one of them has costs nothing on the tensor cores.
//
// tree_plan_kernel -- one block per group of tokens: the union of the lists
//   (an entry belongs to the first list that has it; its other lists are found
//   by binary search), the window's committed rows and the drafted rows on the
//   tokens' paths, each with a mask of the group's tokens.  Lists that do not
//   ascend strictly are not merged: their entries are taken one by one.
//
// tree_tc_kernel -- persistent, one CTA an SM, one group at a time:
//   4 producer warps gather tiles of 64 keys into a ring of stages, K rows
//     K-major and V rows MN-major, both 128-byte swizzled;
//   1 MMA thread issues S = Q K^T (128 rows x 64 keys, 12 steps) into TMEM and,
//     a tile later, O += P V (P from TMEM, 4 steps);
//   4 softmax warps per 128 rows: a thread owns a row (a token's head), so the
//     maximum and the sum need no exchange; P goes back to TMEM as bf16, over
//     its S.  O is rescaled only when a row's maximum grows by more than 2^8
//     (P then stays below 256, whose rounding is relative like any other).
//   S is double buffered: the scores of tile i + 1 are computed while tile i is in
//   its softmax.
//
// P is rounded to bf16 (half a step, 2^-9 of a weight on average 2^-10), which
// the tensor core asks for; the sums of the weights stay fp32 and unrounded.
// A V row that holds an infinity or NaN for one token must not reach another
// that masks it (0 * inf): rows of O that are not finite are computed again
// from their own keys.
#include "common.cuh"
#include "internal.h"
#include "tc.cuh"
#include "tree.cuh"

namespace csa2 {

namespace {

constexpr int kH = 64, kDk = 192, kDv = 128;
constexpr int kRow = 28;                       // bits of a row id in a plan entry; the mask above
constexpr uint32_t kRowMask = (1u << kRow) - 1;
constexpr int kHeader = 4;                     // words before a group's entries: counts of main, ring, drafted

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;

CSA2_DEV int plan_stride(const TreeArgs& a, int group) {
  return kHeader + group * a.topk + a.swa + a.tokens;
}

// Position of `keep`ing threads behind `base` in thread order; every thread
// gets the block's total added to base.
CSA2_DEV int block_slot(bool keep, int& base, int* warp_s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned m = __ballot_sync(0xffffffffu, keep);
  __syncthreads();
  if (lane == 0) warp_s[warp] = __popc(m);
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    const int v = warp_s[w];
    before += w < warp ? v : 0;
    total += v;
  }
  const int at = base + before + __popc(m & ((1u << lane) - 1u));
  base += total;
  return at;
}

__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const TreeArgs a, uint32_t* plan, int group) {
  extern __shared__ int sid[];                 // [group][topk]
  __shared__ int path[4][kMaxTreeTokens];
  __shared__ int n_path[4], n_ring[4], n_list[4], live_s[4];
  __shared__ uint32_t drafted[kMaxTreeTokens];
  __shared__ int warp_s[kPlanWarps];
  __shared__ int merge, newest_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_seq = (a.tokens + group - 1) / group;
  const int seq = blockIdx.x / per_seq, t0 = (blockIdx.x - seq * per_seq) * group;
  const int ng = min(group, a.tokens - t0);
  pdl_wait();
  if (tid == 0) merge = 1;
  if (tid < kMaxTreeTokens) drafted[tid] = 0;
  if (warp < ng) {                             // a warp per token: its path and its part of the ring
    const int token = t0 + warp;
    const bool live = tree_live(a, seq, token, lane == 0);
    int depth = token + 1, n = min(depth, a.swa);
    if (live && a.parent != nullptr) {
      n = tree_walk(a, seq, token, path[warp], depth, true);
    } else {
      for (int i = lane; i < n; i += 32) path[warp][i] = token - i;
    }
    TreeWindow w;
    tree_ring(a, seq, depth, w, lane == 0 && warp == 0 && t0 == 0);
    if (lane == 0) {
      n_path[warp] = live ? n : 0;
      n_ring[warp] = live ? w.n_ring : 0;
      live_s[warp] = live;
      if (warp == 0) newest_s = w.newest;
    }
  } else if (warp < 4 && lane == 0) {
    n_path[warp] = n_ring[warp] = live_s[warp] = 0;
  }
  if (tid < 4) n_list[tid] = 0;
  __syncthreads();
  const int total = ng * a.topk;
  for (int i = tid; i < total; i += kPlanThreads) {
    const int g = i / a.topk;
    int e = live_s[g] ? a.idx[((long long)seq * a.tokens + t0) * a.topk + i] : -1;
    if (e >= a.n_entries) {
      report(a.err, kErrBadIndex, e);
      e = -1;
    }
    sid[i] = e < 0 ? -1 : e;
  }
  __syncthreads();
  // strictly ascending entries first, -1 behind them?
  for (int i = tid; i < total; i += kPlanThreads) {
    const int g = i / a.topk, j = i - g * a.topk, e = sid[i];
    const int next = j + 1 < a.topk ? sid[i + 1] : -1;
    if (next >= 0 && e >= next) merge = 0;     // (racing writes of the same value)
    if (next >= 0 && e < 0) merge = 0;
    if (e >= 0 && next < 0) n_list[g] = j + 1;
  }
  __syncthreads();
  uint32_t* out = plan + (long long)blockIdx.x * plan_stride(a, group);
  int n_main = 0;
  for (int i0 = 0; i0 < total; i0 += kPlanThreads) {
    const int i = i0 + tid;
    const int e = i < total ? sid[i] : -1;
    const int g = i < total ? i / a.topk : 0;
    bool keep = e >= 0;
    uint32_t mask = 1u << g;
    if (keep && merge) {
      for (int o = 0; o < ng; ++o) {
        if (o == g) continue;
        const int* list = sid + o * a.topk;
        int lo = 0, hi = n_list[o];            // first element >= e
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (list[mid] < e) lo = mid + 1;
          else hi = mid;
        }
        if (lo < n_list[o] && list[lo] == e) {
          if (o < g) keep = false;
          mask |= 1u << o;
        }
      }
    }
    const int at = block_slot(keep, n_main, warp_s);
    if (keep) out[kHeader + at] = uint32_t(e) | (mask << kRow);
  }
  // committed rows, newest first, to the tokens whose window reaches them
  int ring = 0;
  for (int g = 0; g < ng; ++g) ring = max(ring, n_ring[g]);
  for (int i = tid; i < ring; i += kPlanThreads) {
    uint32_t mask = 0;
    for (int g = 0; g < ng; ++g) mask |= i < n_ring[g] ? 1u << g : 0u;
    int r = newest_s - i;
    if (r < 0) r += a.swa;
    out[kHeader + n_main + i] = uint32_t(r) | (mask << kRow);
  }
  // drafted rows on the paths
  for (int g = 0; g < ng; ++g)
    for (int i = tid; i < n_path[g]; i += kPlanThreads) atomicOr(&drafted[path[g][i]], 1u << g);
  __syncthreads();
  int n_all = n_main + ring;
  const uint32_t mask = tid < a.tokens ? drafted[tid] : 0;
  const int at = block_slot(mask != 0, n_all, warp_s);
  if (mask != 0) out[kHeader + at] = uint32_t(tid) | (mask << kRow);
  if (tid == 0) {
    out[0] = uint32_t(n_main);
    out[1] = uint32_t(ring);
    out[2] = uint32_t(n_all - n_main - ring);
  }
}

// ------------------------------------------------------------------ attention

constexpr int kTile = 64;                      // keys a stage
constexpr int kKBytes = kTile * kDk * 2, kVBytes = kTile * kDv * 2;
constexpr int kQBytes = 128 * kDk * 2;         // two tokens' queries
constexpr int kProducers = 128;

template <int MT>
struct Conf {
  static constexpr int stages = MT == 2 ? 3 : 4;
  static constexpr int softmax_warps = 4 * MT;
  static constexpr int threads = 32 * softmax_warps + kProducers + 32;
  static constexpr int q = 0, k = q + MT * kQBytes, v = k + stages * kKBytes, ctl = v + stages * kVBytes;
  static constexpr uint32_t cols = MT == 2 ? 512 : 256;
  static constexpr uint32_t o_col = 0, s_col = MT * 128;   // O: 128 columns a row tile; S: two buffers of 64 each
};

template <int MT>
struct Ctl {
  uint64_t full[Conf<MT>::stages], empty[Conf<MT>::stages];
  uint64_t s_full[MT][2], p_full[MT][2];
  uint64_t o_done[MT], o_last[MT], o_free[MT];   // O holds a tile more; the item's last; has been read
  uint64_t q_full, q_empty, fin;
  uint64_t mask[Conf<MT>::stages][4];          // the tile's keys of each token
  uint32_t tmem;
  volatile int abort;
};

template <int MT>
constexpr int tc_smem = Conf<MT>::ctl + int(sizeof(Ctl<MT>)) + 1024;   // + room to align to 1,024

// A bounded wait that also ends when another role has given up.
template <typename C>
CSA2_DEV bool tc_wait(C& c, uint64_t* bar, uint32_t parity, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 31u) == 0u) {
      if (c.abort) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        c.abort = 1;
        report(err, kErrTimeout, int(threadIdx.x));   // which role gave up first
        return false;
      }
    }
  }
}

// The same by a whole warp, which goes on or gives up together.
template <typename C>
CSA2_DEV bool tc_wait_warp(C& c, uint64_t* bar, uint32_t parity, int* err) {
  return __all_sync(0xffffffffu, tc_wait(c, bar, parity, err)) != 0;
}

// Row `pos` of a group's keys: K and V addresses (null behind the last) and token mask.
struct Key {
  const uint8_t *k, *v;
  uint32_t mask;
};
CSA2_DEV Key resolve(const TreeArgs& a, int seq, int pos, uint32_t entry, int n_main, int n_ring, int n_all) {
  Key y{nullptr, nullptr, 0};
  if (pos >= n_all) return y;
  const long long id = entry & kRowMask;
  y.mask = entry >> kRow;
  const void *kb, *vb;
  long long row;
  if (pos < n_main) {
    kb = a.k_main;
    vb = a.v_main;
    row = (long long)seq * a.n_entries + id;
  } else if (pos < n_main + n_ring) {
    kb = a.k_swa;
    vb = a.v_swa;
    row = (long long)seq * a.swa + id;
  } else {
    kb = a.k_draft;
    vb = a.v_draft;
    row = (long long)seq * a.tokens + id;
  }
  y.k = static_cast<const uint8_t*>(kb) + row * (kDk * 2);
  y.v = static_cast<const uint8_t*>(vb) + row * (kDv * 2);
  return y;
}

CSA2_DEV void cp16(uint32_t dst, const uint8_t* src, const void* any) {   // src null: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src != nullptr ? static_cast<const void*>(src) : any),
               "r"(src != nullptr ? 16u : 0u)
               : "memory");
}

// `bar` gets one arrival when this thread's copies so far have landed; nobody waits for them here.
CSA2_DEV void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One row of O from its own keys alone, by a warp: lane l ends with columns 4 l .. 4 l + 3, unscaled by 1 / l.
__device__ __noinline__ float4 row_alone(const TreeArgs& a, int seq, int query, int head, int token, const uint32_t* list, int n_main, int n_ring,
                          int n_all, float sl2, float base) {
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((long long)query * kH + head) * kDk;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < n_all; ++p) {
    const Key y = resolve(a, seq, p, list[p], n_main, n_ring, n_all);
    if (!((y.mask >> token) & 1u)) continue;
    const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(y.k);
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < kDk / 32; ++d) s = __fmaf_rn(__bfloat162float(q[d * 32 + lane]), __bfloat162float(k[d * 32 + lane]), s);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float w = ex2(__fmaf_rn(s, sl2, -base));
    const uint2 v = reinterpret_cast<const uint2*>(y.v)[lane];
    o.x = __fmaf_rn(w, __uint_as_float(v.x << 16), o.x);
    o.y = __fmaf_rn(w, __uint_as_float(v.x & 0xffff0000u), o.y);
    o.z = __fmaf_rn(w, __uint_as_float(v.y << 16), o.z);
    o.w = __fmaf_rn(w, __uint_as_float(v.y & 0xffff0000u), o.w);
  }
  return o;
}

template <int MT>
__global__ void __launch_bounds__(Conf<MT>::threads, 1)
    tree_tc_kernel(const TreeArgs a, const uint32_t* plan, int group, int n_groups) {
  using C = Conf<MT>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Ctl<MT>& c = *reinterpret_cast<Ctl<MT>*>(smem + C::ctl);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::stages; ++i) {
      mbar_init(&c.full[i], kProducers + 16);   // every producer's copies, 4 masks of every producer warp
      mbar_init(&c.empty[i], 1);
    }
    for (int m = 0; m < MT; ++m) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&c.s_full[m][b], 1);
        mbar_init(&c.p_full[m][b], 128);
      }
      mbar_init(&c.o_done[m], 1);
      mbar_init(&c.o_last[m], 1);
      mbar_init(&c.o_free[m], 128);
    }
    mbar_init(&c.q_full, kProducers);
    mbar_init(&c.q_empty, 1);
    mbar_init(&c.fin, 1);
    c.abort = 0;
    mbar_fence_init();
  }
  __syncwarp();
  if (warp == 0) tmem_alloc(&c.tmem, C::cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  pdl_wait();
  const int per_seq = (a.tokens + group - 1) / group, stride = plan_stride(a, group);
  const float sl2 = a.scale * 1.4426950408889634f;

  if (warp < C::softmax_warps) {
    // ---------------------------------------------------------------- softmax: thread = row
    const int mt = warp >> 2, row = (warp & 3) * 32 + lane;
    const int token = mt * 2 + (row >> 6), head = row & 63;   // of the group (uniform in a warp)
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lanes + C::o_col + mt * 128;
    uint32_t tiles = 0, items = 0;             // of this CTA so far
    bool ok = true;
    for (int item = blockIdx.x; item < n_groups && ok; item += gridDim.x) {
      const uint32_t* list = plan + (long long)item * stride;
      const int n_main = int(list[0]), n_ring = int(list[1]), n_all = n_main + n_ring + int(list[2]);
      const int seq = item / per_seq, t = (item - seq * per_seq) * group + token;
      const bool mine = token < group && t < a.tokens;
      const int query = seq * a.tokens + t;
      const int nt = (n_all + kTile - 1) / kTile;
      float ref = -INFINITY, sum = 0.f;        // the exponent that P and O are relative to, and the weights' sum
      for (int i = 0; i < nt; ++i, ++tiles) {
        const uint32_t buf = tiles & 1, st = tiles % C::stages;
        if (!tc_wait_warp(c, &c.full[st], (tiles / C::stages) & 1, a.err) ||
            !tc_wait_warp(c, &c.s_full[mt][buf], (tiles >> 1) & 1, a.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t mask = c.mask[st][token];
        const uint32_t s_addr = tmem + lanes + C::s_col + (mt * 2 + buf) * 64;
        uint32_t s[64];
        tmem_ld64(s, s_addr);
        if (mask != ~0ull) {
          const uint32_t lo = uint32_t(mask), hi = uint32_t(mask >> 32);
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (!(((j < 32 ? lo : hi) >> (j & 31)) & 1u)) s[j] = 0xff800000u;   // -inf
        }
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          m0 = fmaxf(m0, __uint_as_float(s[j]));
          m1 = fmaxf(m1, __uint_as_float(s[32 + j]));
        }
        const float top = fmaxf(m0, m1) * sl2;
        const bool grows = top > ref + 8.f;
        if (i == 0) {
          ref = top;
        } else if (__any_sync(0xffffffffu, grows)) {
          // O holds tiles up to i - 1: wait for the last of them.  (S of tile i comes behind O of tile i - 2,
          // so that the barrier is in the phase of tile i - 1 or behind it, and the parity tells which.)
          if (!tc_wait_warp(c, &c.o_done[mt], (tiles - 1) & 1, a.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float f = grows ? ex2(ref - top) : 1.f;
          if (grows) ref = top;
          sum *= f;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t o[32];
            tmem_ld32(o, o_addr + 32 * q);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st32(o_addr + 32 * q, o);
          }
        }
        const float base = ref == -INFINITY ? 0.f : ref;
        uint32_t p[32];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float x = ex2(__fmaf_rn(__uint_as_float(s[2 * j]), sl2, -base));
          const float y = ex2(__fmaf_rn(__uint_as_float(s[2 * j + 1]), sl2, -base));
          s0 += x;
          s1 += y;
          p[j] = pack_bf16(x, y);
        }
        sum += s0 + s1;
        tmem_st32(s_addr, p);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&c.p_full[mt][buf]);
      }
      if (!ok) break;
      // epilogue
      const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);   // NaN stays NaN
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((long long)query * kH + head) * kDv;
      if (nt > 0) {   // (o_done may be two phases further by now: a barrier of its own)
        if (!tc_wait_warp(c, &c.o_last[mt], items & 1, a.err)) break;
        ++items;
        tc_fence_after();
      }
      bool bad = false;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t o[32];
        if (nt > 0) {
          tmem_ld32(o, o_addr + 32 * q);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0;
        }
        if (!mine) continue;
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = __uint_as_float(o[j + 2 * e]) * inv, y = __uint_as_float(o[j + 2 * e + 1]) * inv;
            bad = bad || !(fabsf(x) < INFINITY) || !(fabsf(y) < INFINITY);
            w[e] = pack_bf16(x, y);
          }
          *reinterpret_cast<uint4*>(out + 32 * q + j) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (mine && a.lse != nullptr)
        a.lse[(long long)query * kH + head] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
      tc_fence_before();
      if (nt > 0) mbar_arrive(&c.o_free[mt]);
      // rows that are not finite: from their own keys, so that no other token's values reach them
      unsigned again = __ballot_sync(0xffffffffu, bad);
      while (again != 0) {
        const int l = __ffs(again) - 1;
        again &= again - 1;
        const float base = __shfl_sync(0xffffffffu, ref == -INFINITY ? 0.f : ref, l);
        const float scale = __shfl_sync(0xffffffffu, sum > 0.f ? 1.f / sum : sum, l);
        const int h = __shfl_sync(0xffffffffu, head, l);
        float4 o = row_alone(a, seq, query, h, token, list + kHeader, n_main, n_ring, n_all, sl2, base);
        if (scale == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);   // no key at all
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + ((long long)query * kH + h) * kDv + 4 * lane) =
            make_uint2(pack_bf16(o.x * scale, o.y * scale), pack_bf16(o.z * scale, o.w * scale));
      }
    }
  } else if (warp < C::softmax_warps + kProducers / 32) {
    // ---------------------------------------------------------------- producers
    const int w = warp - C::softmax_warps, ptid = w * 32 + lane;
    // pieces of four keys (K row: 0..23, V row: 24..39 of each) in five copies a lane
    int p_key[5], p_src[5], p_dst[5], p_chunk[5];
    bool p_k[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const int p = 32 * k + lane, part = p % 40;
      p_key[k] = p / 40;
      p_k[k] = part < 24;
      const int q = p_k[k] ? part : part - 24;
      p_src[k] = q * 16;
      p_dst[k] = (q >> 3) * (kTile * 128);     // 64-column block
      p_chunk[k] = q & 7;
    }
    uint32_t tiles = 0, items = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < n_groups && ok; item += gridDim.x) {
      const uint32_t* list = plan + (long long)item * stride;
      const int n_main = int(list[0]), n_ring = int(list[1]), n_all = n_main + n_ring + int(list[2]);
      const int seq = item / per_seq, t0 = (item - seq * per_seq) * group;
      const int nt = (n_all + kTile - 1) / kTile;
      if (nt == 0) continue;
      list += kHeader;
      int pos = w * 16 + (lane & 15);
      uint32_t entry = pos < n_all ? list[pos] : 0;
      for (int i = 0; i < nt; ++i, ++tiles) {
        const Key key = resolve(a, seq, pos, entry, n_main, n_ring, n_all);
        pos += kTile;
        entry = pos < n_all ? list[pos] : 0;   // of the next tile
        const uint32_t st = tiles % C::stages;
        if (!tc_wait_warp(c, &c.empty[st], ((tiles / C::stages) & 1) ^ 1, a.err)) {
          ok = false;
          break;
        }
        // the masks of this warp's 16 keys, token by token
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const unsigned m = __ballot_sync(0xffffffffu, lane < 16 && ((key.mask >> g) & 1u));
          if (lane == g) reinterpret_cast<uint16_t*>(&c.mask[st][g])[w] = uint16_t(m);
        }
        if (lane < 4) mbar_arrive(&c.full[st]);   // the masks; the copies arrive by themselves
        const uint32_t k_st = smem_u32(smem + C::k + st * kKBytes), v_st = smem_u32(smem + C::v + st * kVBytes);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int k = 0; k < 5; ++k) {
            const int from = 4 * q + p_key[k], r = w * 16 + from;
            const uint8_t* kr = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(key.k), from));
            const uint8_t* vr = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(key.v), from));
            const uint8_t* src = p_k[k] ? kr : vr;
            cp16((p_k[k] ? k_st : v_st) + p_dst[k] + r * 128 + ((p_chunk[k] ^ (r & 7)) << 4),
                 src != nullptr ? src + p_src[k] : nullptr, a.k_main);
          }
        }
        cp_arrive(&c.full[st]);
        if (i == 0) {
          // the group's queries, behind its first tile: row r of row tile m is head r % 64 of token 2 m + r / 64
          if (!tc_wait_warp(c, &c.q_empty, (items & 1) ^ 1, a.err)) {
            ok = false;
            break;
          }
          for (int x = ptid; x < MT * 128 * 24; x += kProducers) {
            const int r = x / 24, part = x - r * 24, tok = r >> 6;
            const int t = t0 + tok;
            const uint8_t* src = tok < group && t < a.tokens
                                     ? static_cast<const uint8_t*>(a.q) +
                                           (((long long)seq * a.tokens + t) * kH + (r & 63)) * (kDk * 2) + part * 16
                                     : nullptr;
            const int rr = r & 127;
            cp16(smem_u32(smem + C::q + (r >> 7) * kQBytes) + (part >> 3) * (128 * 128) + rr * 128 +
                     (((part & 7) ^ (rr & 7)) << 4),
                 src, a.k_main);
          }
          cp_arrive(&c.q_full);
        }
      }
      ++items;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (lane == 0) {
    // ---------------------------------------------------------------- MMA issue
    constexpr uint32_t qk_desc = idesc_bf16(128, kTile, false), pv_desc = idesc_bf16(128, kDv, true);
    uint32_t tiles = 0, items = 0;
    bool ok = true;
    // O (+)= P V of tile x, tile i of its item
    auto pv = [&](uint32_t x, bool first, bool last) -> bool {
      const uint32_t st = x % C::stages, buf = x & 1;
      const uint32_t v = smem_u32(smem + C::v + st * kVBytes);
      for (int m = 0; m < MT; ++m) {
        if (first && items > 0 && !tc_wait(c, &c.o_free[m], (items - 1) & 1, a.err)) return false;
        if (!tc_wait(c, &c.p_full[m][buf], (x >> 1) & 1, a.err)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ts(tmem + C::o_col + m * 128, tmem + C::s_col + (m * 2 + buf) * 64 + 8 * k,
                 smem_desc(v + k * 2048, kTile * 128, 1024), pv_desc, !(first && k == 0));
        tc_commit(&c.o_done[m]);
        if (last) tc_commit(&c.o_last[m]);
      }
      tc_commit(&c.empty[st]);
      return true;
    };
    for (int item = blockIdx.x; item < n_groups && ok; item += gridDim.x) {
      const uint32_t* list = plan + (long long)item * stride;
      const int n_all = int(list[0]) + int(list[1]) + int(list[2]);
      const int nt = (n_all + kTile - 1) / kTile;
      if (nt == 0) continue;
      for (int i = 0; i < nt && ok; ++i, ++tiles) {
        const uint32_t st = tiles % C::stages, buf = tiles & 1;
        ok = tc_wait(c, &c.full[st], (tiles / C::stages) & 1, a.err) &&
             (i > 0 || tc_wait(c, &c.q_full, items & 1, a.err));
        if (!ok) break;
        fence_async_smem();                    // the copies are generic-proxy writes, the tensor core reads by the async proxy
        tc_fence_after();
        const uint32_t k_st = smem_u32(smem + C::k + st * kKBytes);
        for (int m = 0; m < MT; ++m) {
          const uint32_t q_st = smem_u32(smem + C::q + m * kQBytes);
#pragma unroll
          for (int k = 0; k < kDk / 16; ++k)
            mma_ss(tmem + C::s_col + (m * 2 + buf) * 64,
                   smem_desc(q_st + (k >> 2) * (128 * 128) + (k & 3) * 32, 16, 1024),
                   smem_desc(k_st + (k >> 2) * (kTile * 128) + (k & 3) * 32, 16, 1024), qk_desc, k > 0);
          tc_commit(&c.s_full[m][buf]);
        }
        if (i == nt - 1) tc_commit(&c.q_empty);
        if (i > 0) ok = pv(tiles - 1, i == 1, false);
      }
      if (!ok) break;
      ok = pv(tiles - 1, nt == 1, true);
      ++items;
    }
    // every MMA has finished before the memory it uses is given up
    tc_commit(&c.fin);
    mbar_wait(&c.fin, 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tmem, C::cols);
}

template <int MT>
cudaError_t launch_tc(const TreeArgs& a, const uint32_t* plan, int group, int n_groups, cudaStream_t st) {
  const cudaError_t e = once_per_device(MT == 2 ? kSetupTreeQuad : kSetupTreePair, [] {
    return cudaFuncSetAttribute(tree_tc_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, tc_smem<MT>);
  });
  if (e != cudaSuccess) return e;
  const int grid = n_groups < device_sm_count() ? n_groups : device_sm_count();
  note_launch();
  return launch_pdl(tree_tc_kernel<MT>, dim3(unsigned(grid)), dim3(Conf<MT>::threads), tc_smem<MT>, st, 1, a, plan, group,
                    n_groups);
}

}  // namespace

// Words of the plan of a launch with `group` tokens a CTA.
size_t tree_plan_words(int seqs, int tokens, int topk, int swa, int group) {
  return size_t(seqs) * ((tokens + group - 1) / group) * (size_t(kHeader) + size_t(group) * topk + swa + tokens);
}

cudaError_t launch_tree_attn_tc(const TreeArgs& a, int seqs, int group, void* plan, cudaStream_t st) {
  const int n_groups = seqs * ((a.tokens + group - 1) / group);
  uint32_t* words = static_cast<uint32_t*>(plan);
  note_launch();
  const cudaError_t e = launch_pdl(tree_plan_kernel, dim3(unsigned(n_groups)), dim3(kPlanThreads),
                                   size_t(group) * a.topk * 4, st, 1, a, words, group);
  if (e != cudaSuccess) return e;
  return group > 2 ? launch_tc<2>(a, words, group, n_groups, st) : launch_tc<1>(a, words, group, n_groups, st);
}

}  // namespace csa2
