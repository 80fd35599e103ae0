// Attention of drafted trees on the 5th-generation tensor cores, for batches
// that fill the GPU and for few keys (bf16, 64 heads sharing one KV head, dk 192,
// dv 128).
//
// The drafted tokens of a sequence are neighbours: their Top-K lists overlap
// and their windows are nearly the same.  One CTA therefore attends with two
// tokens of a sequence at once (one, where a sequence has one or every token has
// an SM), over the union of their keys, and masks each key to the tokens that have it: a key that both
// select is gathered once.  The gather sets the time of this attention, and the tensor cores'
// rows come in 128s, which two tokens' 64 heads fill, so that attending both
// tokens to a key that only one of them has costs nothing there.
//
// tree_plan_kernel -- one block per group of tokens: the union of the lists
//   (an entry belongs to the first list that has it; its other list is looked
//   up by binary search), the window's committed rows and the drafted rows on the
//   tokens' paths, each with a mask of the group's tokens.  Lists that do not
//   ascend strictly are not merged: their entries are taken one by one.
//
// tree_tc_kernel -- persistent, one CTA an SM, one group at a time:
//   7 producer warps gather tiles of 64 keys into a ring of 5 stages, K rows
//     K-major and V rows MN-major, both 128-byte swizzled;
//   1 warp issues S = Q K^T (128 rows x 64 keys, 12 steps) into TMEM and, a
//     tile later, O += P V (4 steps).  Q and P are read from TMEM: with Q in
//     shared memory every step of 64 keys reads its 4 KB again, and the shared
//     memory, not the tensor core, set the rate (58 cycles a step against 32);
//   4 softmax warps: a thread owns a row (a token's head), so the maximum and
//     the sum need no exchange; P goes back to TMEM as bf16, over its S.  O is
//     rescaled only when a row's maximum grows by more than 2^8 (P then stays
//     below 256, whose rounding is relative like any other);
//   4 end warps put the next group's Q into TMEM and write the last one's O
//     out, both through shared memory for whole lines, while the others go on.
//   S and O are double buffered: the scores of tile i + 1 are computed while tile i
//   is in its softmax, and a group starts while the one before it is written out.
//   (Two softmax sets for even and odd tiles were slower: their warps share the
//   schedulers, so that each tile waits longer for its weights.)
//
// Bound by the two loops of a tile, about 1,200 cycles each: the softmax warps'
// (their 64 exponentials a row are 570, the maximum 200, TMEM loads and stores 150) and
// the issue of 16 tensor-core steps (690) with its waits.  32 trees of 32 tokens,
// 640 slots: 52.9 us with the plan, 0.50 PFLOP/s by every token's own keys, the tensor
// cores active in 30 % of the cycles; 16 trees of 16: 21.2 us.  Stamps of the latter, from the
// plan's start in ns: its end 5,500; the attention's wait over 6,100, the first tile's copies
// issued 8,200 (counts, entries and rows are read one behind the other) and landed 8,400; the
// first scores 8,900; 13 tiles of 630 until 17,000; O written 18,300, the end 18,700.  Of the
// former: 9,600 until the wait is over, first scores 13,400, then 735 a tile; a CTA has 41
// tiles on average and 51 at most (whole pairs, 3.4 an SM), so that they end between 40,000 and 52,500.
// Groups of four tokens (two row tiles) took 79 us for the former, two softmax sets
// 70, half of the exponentials by a polynomial 66.
//
// P is rounded to bf16 (half a step, 2^-8 of a weight), which the tensor core
// asks for; the sums of the weights stay fp32 and unrounded.
// A V row that holds an infinity or NaN for one token must not reach another
// that masks it (0 * inf): rows of O that are not finite though their sum is a number are computed again
// from their own keys (32 trees of 16 with infinities in every row: 5.6 ms, a warp's 32
// rows one after the other; NaN scores make no such rows and cost nothing).
#include "common.cuh"
#include "draft.h"
#include "tc.cuh"
#include "tree.cuh"

namespace csa2 {

namespace {

constexpr int kH = 64, kDk = 192, kDv = 128;
constexpr int kTile = 64;                      // keys a stage
constexpr int kRow = 28;                       // bits of a row id in a plan entry (ids < 2^28); the mask above
constexpr uint32_t kRowMask = (1u << kRow) - 1;
// A group's part of the plan, in words: the counts of main, ring and drafted
// rows and a spare one; for every tile of 64 keys and token the keys that the
// token has, 64 bits each; the keys.
constexpr int kHeader = 4;
__host__ __device__ constexpr int plan_keys(int topk, int swa, int tokens, int group) {
  return (group * topk + swa + tokens + kTile - 1) / kTile * kTile;
}
__host__ __device__ constexpr int plan_entries(int keys) { return kHeader + keys / kTile * 4; }

// ------------------------------------------------------------------ plan

// 8 warps for the lists, a warp for each token's path: 6 blocks an SM, so that the groups of a large batch run at once.
constexpr int kListThreads = 256, kListWarps = kListThreads / 32, kPlanThreads = kListThreads + 64;
constexpr int kChunks = 4;                     // list elements a thread takes of each list: topk <= 1,024

CSA2_DEV int plan_stride(const TreeArgs& a, int group) {
  const int keys = plan_keys(a.topk, a.swa, a.tokens, group);
  return plan_entries(keys) + keys;
}

// Elements of `list` [n], ascending with -1 behind them, below e; `hit`: whether e is one.
CSA2_DEV int below(const int* list, int n, int e, bool& hit) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (uint32_t(list[mid]) < uint32_t(e)) lo = mid + 1;   // (-1 is above all)
    else hi = mid;
  }
  hit = lo < n && list[lo] == e;
  return lo;
}

// Bits [from, to) of the 32 bits that begin at `at`.
CSA2_DEV uint32_t range_bits(int at, int from, int to) {
  const int lo = max(from - at, 0), hi = min(to - at, 32);
  if (hi <= lo) return 0;
  return (hi == 32 ? ~0u : (1u << hi) - 1u) & ~((1u << lo) - 1u);
}

// One block a group, bound by the latency of its steps (load, search, count,
// write): loads that do not need each other go out together, and the paths are
// walked beside the search.
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const TreeArgs a, uint32_t* plan, int group) {
  extern __shared__ int sid[];                 // [2][topk], then the ranks [topk + 1]
  int* rank = sid + 2 * a.topk;                // keys of the first list before each that the second has too
  __shared__ int path[2][kMaxTreeTokens], jump[2][kMaxTreeTokens];
  __shared__ int n_ring[2], n_list[2], n_draft;
  __shared__ uint32_t drafted[kMaxTreeTokens];
  __shared__ int warp_s[2][kChunks * kListWarps];
  __shared__ int ordered, newest_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lists = warp < kListWarps;
  const int per_seq = (a.tokens + group - 1) / group;
  const int seq = blockIdx.x / per_seq, t0 = (blockIdx.x - seq * per_seq) * group;
  const int ng = min(group, a.tokens - t0);
  pdl_launch_dependents();   // the attention's CTAs set themselves up meanwhile, and wait for this launch's end
  if (tid == 0) ordered = 1;
  if (tid < kMaxTreeTokens) drafted[tid] = 0;
  if (tid < 2) n_list[tid] = n_ring[tid] = 0;
  __syncthreads();
  pdl_wait();
  if (lists) {
    for (int g = 0; g < 2; ++g) {
      const bool live = g < ng && tree_live(a, seq, t0 + g, false);
      for (int j = tid; j < a.topk; j += kListThreads) {
        int e = g < ng ? a.idx[((long long)seq * a.tokens + t0 + g) * a.topk + j] : -1;   // (does not wait for `live`)
        if (!live) e = -1;
        if (e >= a.n_entries) {
          report(a.err, kErrBadIndex, e);
          e = -1;
        }
        sid[g * a.topk + j] = e < 0 ? -1 : e;
      }
    }
  }
  __syncthreads();
  const int max_keys = plan_keys(a.topk, a.swa, a.tokens, group);
  uint32_t* out = plan + (long long)blockIdx.x * plan_stride(a, group);
  uint32_t* entries = out + plan_entries(max_keys);
  int* ids = path[0];                          // the drafted rows on either path, when both have been walked
  bool hit[kChunks] = {};                      // this thread's elements of the first list: the second has them
  int before[2][kChunks] = {};                 // elements of the warp's before them: shared ones, or any, of either list
  int lower[kChunks] = {};                     // of the second: elements of the first below them, -1 where it has them
  if (lists) {
    // Do both lists ascend strictly, with nothing but -1 behind their entries?
    // The searches take it for granted; without it nothing of theirs is used.
#pragma unroll
    for (int x = 0; x < kChunks; ++x) {
      if (x * kListThreads >= a.topk || ng == 1) break;
      const int j = x * kListThreads + tid;
      if (j >= a.topk) continue;
      for (int g = 0; g < 2; ++g) {
        const int e = sid[g * a.topk + j], next = j + 1 < a.topk ? sid[g * a.topk + j + 1] : -1;
        if (next >= 0 && e >= next) ordered = 0;   // (racing writes of the same value)
        if (next >= 0 && e < 0) ordered = 0;
        if (e >= 0 && next < 0) n_list[g] = j + 1;
      }
      if (sid[j] >= 0) below(sid + a.topk, a.topk, sid[j], hit[x]);
      if (sid[a.topk + j] >= 0) {
        bool both;
        lower[x] = below(sid, a.topk, sid[a.topk + j], both);
        if (both) lower[x] = -1;
      }
    }
  } else if (warp - kListWarps < ng) {
    const int g = warp - kListWarps, token = t0 + g;
    TreeWindow w;
    tree_ring(a, seq, w, lane == 0 && g == 0 && t0 == 0);
    const bool live = tree_live(a, seq, token, lane == 0);
    int depth = token + 1, n = min(depth, a.swa);
    if (a.parent != nullptr) {
      n = tree_walk(a, seq, token, path[g], jump[g], depth, live);
    } else {
      for (int i = lane; i < n; i += 32) path[g][i] = token - i;
    }
    if (!live) n = 0;
    __syncwarp();
    for (int i = lane; i < n; i += 32) atomicOr(&drafted[path[g][i]], 1u << g);
    if (lane == 0) {
      n_ring[g] = live ? min(w.n_ring, max(0, a.swa - depth)) : 0;
      if (g == 0) newest_s = w.newest;
    }
  }
  __syncthreads();
  const bool merge = ng > 1 && ordered != 0;   // (a list alone is taken as it is)
  if (lists) {
#pragma unroll
    for (int x = 0; x < kChunks; ++x) {
      const int j = x * kListThreads + tid;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const bool mark = j < a.topk && (merge ? g == 0 && hit[x] : sid[g * a.topk + j] >= 0);
        const unsigned m = __ballot_sync(0xffffffffu, mark);
        before[g][x] = __popc(m & ((1u << lane) - 1u));
        if (lane == 0) warp_s[g][x * kListWarps + warp] = __popc(m);
      }
    }
  } else if (warp == kListWarps) {
    // the drafted rows in order, each with its mask
    int n = 0;
    for (int t = 0; t < a.tokens; t += 32) {
      const uint32_t mask = t + lane < a.tokens ? drafted[t + lane] : 0;
      const unsigned m = __ballot_sync(0xffffffffu, mask != 0);
      if (mask != 0) ids[n + __popc(m & ((1u << lane) - 1u))] = int(uint32_t(t + lane) | (mask << kRow));
      n += __popc(m);
    }
    if (lane == 0) n_draft = n;
  }
  __syncthreads();
  int total[2], first[2][kChunks];             // marked elements, and those before this thread's
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int v = warp_s[g][lane];             // (kChunks * kListWarps == 32)
    int incl = v;
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    total[g] = __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
    for (int x = 0; x < kChunks; ++x)
      first[g][x] = __shfl_sync(0xffffffffu, incl - v, (x * kListWarps + warp) & 31) + before[g][x];
  }
  // Both tokens' keys first, then either's own: most tiles are then wholly a
  // token's or wholly not, which the softmax takes without looking at keys.
  const int n_both = merge ? total[0] : 0;
  const int n_a = merge ? n_list[0] - n_both : total[0], n_b = merge ? n_list[1] - n_both : total[1];
  const int n_main = n_both + n_a + n_b;
  if (lists) {
#pragma unroll
    for (int x = 0; x < kChunks; ++x) {
      const int j = x * kListThreads + tid;
      if (j >= a.topk) break;
      const int e = sid[j], f = sid[a.topk + j];
      if (merge) {
        rank[j] = first[0][x];
        if (e >= 0) entries[hit[x] ? first[0][x] : n_both + j - first[0][x]] = uint32_t(e) | ((hit[x] ? 3u : 1u) << kRow);
      } else {
        if (e >= 0) entries[first[0][x]] = uint32_t(e) | (1u << kRow);
        if (f >= 0) entries[n_a + first[1][x]] = uint32_t(f) | (2u << kRow);
      }
    }
  }
  // committed rows, newest first, to the tokens whose window reaches them; drafted rows
  const int ring = max(n_ring[0], n_ring[1]), draft0 = n_main + ring;
  for (int i = tid; i < ring; i += kPlanThreads) {
    int r = newest_s - i;
    if (r < 0) r += a.swa;
    entries[n_main + i] = uint32_t(r) | ((i < n_ring[0] ? 1u : 0u) | (i < n_ring[1] ? 2u : 0u)) << kRow;
  }
  for (int i = tid; i < n_draft; i += kPlanThreads) entries[draft0 + i] = uint32_t(ids[i]);
  if (tid == 0) {
    out[0] = uint32_t(n_main);
    out[1] = uint32_t(ring);
    out[2] = uint32_t(n_draft);
  }
  // the tiles' masks: 32 keys w of token g at word (w / 2) * 4 + 2 g + w % 2
  for (int i = tid; i < max_keys / kTile * 4; i += kPlanThreads) {
    const int g = (i >> 1) & 1, at = ((i >> 2) * 2 + (i & 1)) * 32;
    uint32_t m = range_bits(at, 0, n_both) | range_bits(at, n_main, n_main + n_ring[g]) |
                 (g == 0 ? range_bits(at, n_both, n_both + n_a) : range_bits(at, n_both + n_a, n_main));
    for (int x = max(at, draft0); x < min(at + 32, draft0 + n_draft); ++x)
      if ((uint32_t(ids[x - draft0]) >> (kRow + g)) & 1u) m |= 1u << (x - at);
    out[kHeader + i] = m;
  }
  if (!merge) return;
  __syncthreads();                             // the ranks
  if (lists) {
#pragma unroll
    for (int x = 0; x < kChunks; ++x) {        // the second's own: less the shared ones, which are the first's below it
      const int j = x * kListThreads + tid;
      if (j >= a.topk) break;
      if (sid[a.topk + j] >= 0 && lower[x] >= 0) {
        const int shared = lower[x] < n_list[0] ? rank[lower[x]] : n_both;
        entries[n_both + n_a + j - shared] = uint32_t(sid[a.topk + j]) | (2u << kRow);
      }
    }
  }
}

// ------------------------------------------------------------------ attention

constexpr int kKBytes = kTile * kDk * 2, kVBytes = kTile * kDv * 2;
constexpr int kStages = 5;
constexpr int kSoftmaxWarps = 4, kEndWarps = 4, kProducerWarps = 7;
constexpr int kFours = (kTile / 4 + kProducerWarps - 1) / kProducerWarps;   // fours of keys of a producer warp
constexpr int kWarpKeys = 4 * kFours;
static_assert(kWarpKeys <= 32, "a lane for every key");
constexpr int kThreads = 32 * (kSoftmaxWarps + kEndWarps + kProducerWarps + 1);
constexpr uint32_t kTmemCols = 512;            // a power of two over two O (128 each), two S (64 each) and Q (96)
constexpr uint32_t kOCol = 0, kSCol = 256, kQCol = 384;

struct Shared {
  uint8_t k[kStages][kKBytes];                 // 3 blocks of 64 dims: 64 rows of 128 bytes
  uint8_t v[kStages][kVBytes];                 // 2 blocks of 64 dims: 64 keys of 128 bytes
  uint64_t row[kProducerWarps][2][kWarpKeys][2];   // K and V addresses of a producer warp's keys, of even and odd tiles
  uint4 turn[kEndWarps][32 * 4];               // 64 bytes of each of an end warp's rows
  float2 stat[128];                            // (exponent, sum) of the rows of an item
  uint64_t full[kStages], empty[kStages];      // a tile has landed; has been used
  uint64_t s_full[2], p_full[2];               // S has been computed; P has been written
  uint64_t o_done, o_last[2], o_free[2];       // O holds a tile more; the item's last; has been read
  uint64_t q_full, q_empty, stat_full, stat_free;
  uint64_t fin;                                // every MMA is done
  uint32_t tmem;
  volatile int abort;
};
constexpr int kSmem = int(sizeof(Shared)) + 1024;   // + room to align to 1,024

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

CSA2_DEV void cp16(uint32_t dst, uint64_t src, int offset, const void* any) {   // src 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src != 0 ? src + offset : reinterpret_cast<uint64_t>(any)), "r"(src != 0 ? 16u : 0u)
               : "memory");
}

// One row of O from its own keys alone, by a warp: lane l ends with columns 4 l .. 4 l + 3, unscaled by 1 / l.
// 32 keys at a time: a lane scores one of them, then all lanes add up the values of those that the token has, 8
// rows on their way.
__device__ __noinline__ float4 row_alone(const TreeArgs& a, int seq, int query, int head, int token, const uint32_t* list, int n_main, int n_ring,
                          int n_all, float sl2, float base) {
  const int lane = threadIdx.x & 31;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + ((long long)query * kH + head) * kDk);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < n_all; p0 += 32) {
    const int p = p0 + lane;
    const Key y = resolve(a, seq, p, p < n_all ? list[p] : 0, n_main, n_ring, n_all);
    const bool has = ((y.mask >> token) & 1u) != 0;
    float w = 0.f;
    if (has) {
      const uint4* k = reinterpret_cast<const uint4*>(y.k);
      float s = 0.f;
#pragma unroll 4
      for (int d = 0; d < kDk / 8; ++d) {
        const uint4 u = q[d], v = k[d];
        const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = __fmaf_rn(__uint_as_float(us[e] << 16), __uint_as_float(vs[e] << 16), s);
          s = __fmaf_rn(__uint_as_float(us[e] & 0xffff0000u), __uint_as_float(vs[e] & 0xffff0000u), s);
        }
      }
      w = ex2(__fmaf_rn(s, sl2, -base));
    }
    __syncwarp();
    const unsigned keys = __ballot_sync(0xffffffffu, has);
    for (int j0 = 0; j0 < 32; j0 += 8) {
      if (((keys >> j0) & 0xffu) == 0) continue;
      uint2 v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint64_t at = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(y.v), j0 + x);
        v[x] = (keys >> (j0 + x)) & 1u ? reinterpret_cast<const uint2*>(at)[lane] : make_uint2(0u, 0u);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float z = __shfl_sync(0xffffffffu, w, j0 + x);   // 0 where the token has no such key, as v is
        o.x = __fmaf_rn(z, __uint_as_float(v[x].x << 16), o.x);
        o.y = __fmaf_rn(z, __uint_as_float(v[x].x & 0xffff0000u), o.y);
        o.z = __fmaf_rn(z, __uint_as_float(v[x].y << 16), o.z);
        o.w = __fmaf_rn(z, __uint_as_float(v[x].y & 0xffff0000u), o.w);
      }
    }
  }
  return o;
}

// The 32 rows of a warp, 64 bytes each, between rows by lane (a lane's four
// pieces are its row's) and by line (piece j of lane l is row 8 j + l / 4,
// part l % 4), through shared memory without bank conflicts.
CSA2_DEV uint4& turn_at(uint4* t, int row, int part) { return t[row * 4 + (part ^ ((row >> 1) & 3))]; }

CSA2_DEV void rows_to_lines(uint4* t, uint4 (&w)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int p = 0; p < 4; ++p) turn_at(t, lane, p) = w[p];
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = turn_at(t, 8 * j + (lane >> 2), lane & 3);
  __syncwarp();
}

CSA2_DEV void lines_to_rows(uint4* t, uint4* w) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 4; ++j) turn_at(t, 8 * j + (lane >> 2), lane & 3) = w[j];
  __syncwarp();
#pragma unroll
  for (int p = 0; p < 4; ++p) w[p] = turn_at(t, lane, p);
  __syncwarp();
}

__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const TreeArgs a, const uint32_t* plan, int group, int n_groups) {
  extern __shared__ uint8_t raw[];
  Shared& c = *reinterpret_cast<Shared*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&c.full[i], 32 * kProducerWarps);
      mbar_init(&c.empty[i], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.s_full[b], 1);
      mbar_init(&c.p_full[b], 128);
      mbar_init(&c.o_last[b], 1);
      mbar_init(&c.o_free[b], 128);
    }
    mbar_init(&c.o_done, 1);
    mbar_init(&c.q_full, 128);
    mbar_init(&c.q_empty, 1);
    mbar_init(&c.stat_full, 128);
    mbar_init(&c.stat_free, 128);
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
  pdl_wait();
  const int per_seq = (a.tokens + group - 1) / group, stride = plan_stride(a, group);
  const int first_key = plan_entries(plan_keys(a.topk, a.swa, a.tokens, group));
  const float sl2 = a.scale * 1.4426950408889634f;
  auto keys_of = [&](int item) -> int {
    const uint32_t* list = plan + (long long)item * stride;
    return int(list[0]) + int(list[1]) + int(list[2]);
  };

  if (warp < kSoftmaxWarps) {
    // ---------------------------------------------------------------- softmax: thread = row
    const int token = tid >> 6;                               // of the group (uniform in a warp)
    const uint32_t lanes = uint32_t(warp * 32) << 16;
    const float2 scale2 = make_float2(sl2, sl2);
    uint32_t tiles = 0, items = 0;                            // of this CTA so far
    bool ok = true;
    for (int item = blockIdx.x; item < n_groups && ok; item += gridDim.x) {
      const int nt = (keys_of(item) + kTile - 1) / kTile;
      if (nt == 0) continue;
      const uint64_t* masks = reinterpret_cast<const uint64_t*>(plan + (long long)item * stride + kHeader) + token;
      uint64_t mask_next = masks[0];                          // the token's keys of the next tile
      const uint32_t o_addr = tmem + lanes + kOCol + (items & 1) * 128;
      float ref = -INFINITY, sum = 0.f;        // the exponent that P and O are relative to, and the weights' sum
      for (int i = 0; i < nt; ++i, ++tiles) {
        const uint64_t mask = mask_next;
        if (i + 1 < nt) mask_next = masks[2 * (i + 1)];
        const uint32_t buf = tiles & 1, s_addr = tmem + lanes + kSCol + buf * 64;
        ok = tc_wait_warp(c, &c.s_full[buf], (tiles >> 1) & 1, a.err);
        if (!ok) break;
        tc_fence_after();
        uint32_t p[32];
        if (mask != 0) {
          uint32_t s[64];
          tmem_ld64(s, s_addr);
          if (mask != ~0ull) {
            const uint32_t lo = uint32_t(mask), hi = uint32_t(mask >> 32);
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (!(((j < 32 ? lo : hi) >> (j & 31)) & 1u)) s[j] = 0xff800000u;   // -inf
          }
          float m[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            m[e] = __uint_as_float(s[e]);
#pragma unroll
            for (int j = 8; j + 8 < 64; j += 16) m[e] = max3_nan(m[e], __uint_as_float(s[j + e]), __uint_as_float(s[j + 8 + e]));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) m[e] = fmaxf(m[e], __uint_as_float(s[56 + e]));
          const float top = max3_nan(max3_nan(m[0], m[1], m[2]), max3_nan(m[3], m[4], m[5]), fmaxf(m[6], m[7])) * sl2;
          if (!(top < INFINITY)) sum = NAN;                   // as the definition has it
          const bool grows = top > ref + 8.f;
          if (i == 0) {
            ref = top;
          } else if (__any_sync(0xffffffffu, grows)) {
            // O holds tiles up to i - 1: wait for the last of them.  (S of tile i comes behind O of tile i - 2,
            // so that the barrier is in the phase of tile i - 1 or behind it, and the parity tells which.)
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
          const float base = ref == -INFINITY ? 0.f : -ref;
          const float2 base2 = make_float2(base, base);
          float2 total = make_float2(0.f, 0.f), other = make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float2 x = fma2(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), scale2, base2);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            if (j & 1) other = add2(other, x);
            else total = add2(total, x);
            p[j] = pack_bf16(x.x, x.y);
          }
          total = add2(total, other);
          sum += total.x + total.y;
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) p[j] = 0;
        }
        tmem_st32(s_addr, p);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&c.p_full[buf]);
      }
      if (!ok) break;
      ok = items == 0 || tc_wait_warp(c, &c.stat_free, (items - 1) & 1, a.err);
      if (!ok) break;
      c.stat[tid] = make_float2(ref, sum);
      mbar_arrive(&c.stat_full);
      ++items;
    }
  } else if (warp < kSoftmaxWarps + kEndWarps) {
    // ---------------------------------------------------------------- ends of items: Q in, O out; thread = row
    const int row = tid - 32 * kSoftmaxWarps, w = warp - kSoftmaxWarps;
    const int token = row >> 6, head0 = (w & 1) * 32;         // of the group; the warp's rows are heads head0 .. head0 + 31
    const uint32_t lanes = uint32_t(w * 32) << 16;
    uint4* turn = c.turn[w];
    auto query_of = [&](int item) -> int {                    // -1: the group has no such token
      const int seq = item / per_seq, t = (item - seq * per_seq) * group + token;
      return token < group && t < a.tokens ? seq * a.tokens + t : -1;
    };
    // A group's queries, this thread's row.  A third at a time is on its way: all
    // of them at once need more lines than the L1 beside this much shared memory
    // has, and the producers' copies then wait behind them.
    uint4 q[24];
    auto fetch_q = [&](int item) {
      const int query = query_of(item);
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) +
                                                        ((long long)max(query, 0) * kH + head0) * (kDk * 2));
#pragma unroll
      for (int b = 0; b < 3; ++b) {
#pragma unroll
        for (int x = 8 * b; x < 8 * b + 8; ++x)
          q[x] = query >= 0 ? src[(8 * (x & 3) + (lane >> 2)) * (kDk / 8) + (x >> 2) * 4 + (lane & 3)] : make_uint4(0, 0, 0, 0);
        lines_to_rows(turn, q + 8 * b);
        lines_to_rows(turn, q + 8 * b + 4);
      }
    };
    auto store_q = [&]() {
#pragma unroll
      for (int b = 0; b < 6; ++b) {
        uint32_t r[16];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          r[4 * x] = q[4 * b + x].x;
          r[4 * x + 1] = q[4 * b + x].y;
          r[4 * x + 2] = q[4 * b + x].z;
          r[4 * x + 3] = q[4 * b + x].w;
        }
        tmem_st16(tmem + lanes + kQCol + 16 * b, r);
      }
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(&c.q_full);
    };
    auto next_item = [&](int item) -> int {                   // the next with any key, from `item` on
      while (item < n_groups && keys_of(item) == 0) item += gridDim.x;
      return item;
    };
    uint32_t items = 0;
    fetch_q(blockIdx.x);                                      // beside its counts
    const int first = next_item(blockIdx.x);
    if (first < n_groups) {
      if (first != int(blockIdx.x)) fetch_q(first);
      store_q();
    }
    for (int item = blockIdx.x; item < n_groups; item += gridDim.x) {
      const int query = query_of(item);
      uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + ((long long)max(query, 0) * kH + head0) * kDv);
      float* lse = a.lse != nullptr ? a.lse + (long long)max(query, 0) * kH + head0 + lane : nullptr;
      const int n_all = keys_of(item);
      if (n_all == 0) {                                       // no live token
        if (query >= 0) {
          for (int x = lane; x < 32 * kDv / 8; x += 32) out[x] = make_uint4(0, 0, 0, 0);
          if (lse != nullptr) *lse = -INFINITY;
        }
        continue;
      }
      const int next = next_item(item + gridDim.x);
      if (next < n_groups) {
        fetch_q(next);
        if (!tc_wait_warp(c, &c.q_empty, items & 1, a.err)) break;
        tc_fence_after();
        store_q();
      }
      if (!tc_wait_warp(c, &c.stat_full, items & 1, a.err)) break;
      const float ref = c.stat[row].x, sum = c.stat[row].y;
      mbar_arrive(&c.stat_free);
      const uint32_t o_addr = tmem + lanes + kOCol + (items & 1) * 128;
      if (!tc_wait_warp(c, &c.o_last[items & 1], (items >> 1) & 1, a.err)) break;
      tc_fence_after();
      const float inv = sum > 0.f ? 1.f / sum : sum;          // no key: 0; NaN stays NaN
      bool bad = false;
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        uint32_t o[32];
        tmem_ld32(o, o_addr + 32 * b);
        if (query < 0) continue;
        uint4 y[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = __uint_as_float(o[8 * x + 2 * e]) * inv, v = __uint_as_float(o[8 * x + 2 * e + 1]) * inv;
            bad = bad || !(fabsf(u) < INFINITY) || !(fabsf(v) < INFINITY);
            p[e] = pack_bf16(u, v);
          }
          y[x] = make_uint4(p[0], p[1], p[2], p[3]);
        }
        rows_to_lines(turn, y);
#pragma unroll
        for (int j = 0; j < 4; ++j) out[(8 * j + (lane >> 2)) * (kDv / 8) + 4 * b + (lane & 3)] = y[j];
      }
      tc_fence_before();
      mbar_arrive(&c.o_free[items & 1]);
      ++items;
      if (query >= 0 && lse != nullptr) *lse = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
      // rows that are not finite: from their own keys, so that no other token's values reach them (one whose sum is
      // NaN is NaN whatever they hold)
      unsigned again = __ballot_sync(0xffffffffu, bad && inv == inv);
      while (again != 0) {
        const int l = __ffs(again) - 1;
        again &= again - 1;
        const uint32_t* list = plan + (long long)item * stride;
        const float base = __shfl_sync(0xffffffffu, ref == -INFINITY ? 0.f : ref, l);
        const float scale = __shfl_sync(0xffffffffu, inv, l);
        float4 o = row_alone(a, item / per_seq, query, head0 + l, token, list + first_key, int(list[0]), int(list[1]), n_all, sl2, base);
        if (scale == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);   // no key at all
        reinterpret_cast<uint2*>(out)[l * (kDv / 4) + lane] =
            make_uint2(pack_bf16(o.x * scale, o.y * scale), pack_bf16(o.z * scale, o.w * scale));
      }
    }
  } else if (warp < kSoftmaxWarps + kEndWarps + kProducerWarps) {
    // ---------------------------------------------------------------- producers: every seventh four keys of a tile a warp
    const int w = warp - kSoftmaxWarps - kEndWarps;
    // The 16-byte pieces of four keys (K row: 0..23, V row: 24..39 of each) in
    // five copies a lane.  Key x of four f lies at row 4 f + x of the tile,
    // whose low three bits swizzle: those of x, and 4 more for odd f.
    int p_row[5], p_src[5], p_dst[5];
    bool p_k[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const int p = 32 * k + lane, part = p % 40, x = p / 40;
      p_k[k] = part < 24;
      const int y = p_k[k] ? part : part - 24;
      p_row[k] = 2 * x + (p_k[k] ? 0 : 1);
      p_src[k] = y * 16;
      p_dst[k] = (y >> 3) * (kTile * 128) + x * 128 + (((y & 7) ^ x) << 4);
    }
    const int mine = 4 * (w + kProducerWarps * (lane >> 2)) + (lane & 3);   // this lane's key of a tile
    const bool on = lane < kWarpKeys && mine < kTile;
    uint32_t tiles = 0, st = 0, lap = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < n_groups && ok; item += gridDim.x) {
      const uint32_t* list = plan + (long long)item * stride;
      const int n_main = int(list[0]), n_ring = int(list[1]), n_all = n_main + n_ring + int(list[2]);
      const int seq = item / per_seq, nt = (n_all + kTile - 1) / kTile;
      list += first_key;
      uint32_t entry = list[on ? mine : 0];   // (beside the counts: a plan has room for a tile at least)
      int pos = on ? mine : n_all;
      for (int i = 0; i < nt; ++i, ++tiles) {
        const Key key = resolve(a, seq, pos, entry, n_main, n_ring, n_all);
        pos += kTile;
        entry = pos < n_all ? list[pos] : 0;   // of the next tile
        uint64_t(*row)[2] = c.row[w][tiles & 1];
        if (lane < kWarpKeys) {
          row[lane][0] = reinterpret_cast<uint64_t>(key.k);
          row[lane][1] = reinterpret_cast<uint64_t>(key.v);
        }
        ok = tc_wait_warp(c, &c.empty[st], (lap & 1) ^ 1, a.err);
        if (!ok) break;
        __syncwarp();                          // the warp's rows are written
        const uint32_t k_st = smem_u32(c.k[st]), v_st = smem_u32(c.v[st]);
        uint64_t src[kFours][5];
#pragma unroll
        for (int q = 0; q < kFours; ++q)
#pragma unroll
          for (int k = 0; k < 5; ++k) src[q][k] = (&row[4 * q][0])[p_row[k]];
#pragma unroll
        for (int q = 0; q < kFours; ++q) {
          const int f = w + kProducerWarps * q;
          if (f < kTile / 4) {                 // a warp's last may not exist
#pragma unroll
            for (int k = 0; k < 5; ++k)
              cp16(((p_k[k] ? k_st : v_st) + p_dst[k] + f * 512) ^ ((f & 1) * 64), src[q][k], p_src[k], a.k_main);
          }
        }
        cp_arrive(&c.full[st]);
        if (++st == kStages) {
          st = 0;
          ++lap;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---------------------------------------------------------------- MMA issue
    constexpr uint32_t qk_desc = idesc_bf16(128, kTile, false), pv_desc = idesc_bf16(128, kDv, true);
    const uint64_t k0 = smem_desc(smem_u32(c.k[0]), 16, 1024), v0 = smem_desc(smem_u32(c.v[0]), kTile * 128, 1024);
    uint32_t tiles = 0, items = 0;
    uint32_t st = 0, lap = 0, st_pv = 0;       // stage of the next scores, times round the ring, stage of the next O
    bool ok = true, landed = false;
    // O (+)= P V of tile x, of the current item
    auto pv = [&](uint32_t x, bool first, bool last) -> bool {
      const uint32_t buf = x & 1, o = items & 1;
      const uint64_t v = v0 + st_pv * (kVBytes >> 4);
      if (first && items > 1 && !tc_wait_warp(c, &c.o_free[o], ((items >> 1) - 1) & 1, a.err)) return false;
      const bool here = mbar_test(&c.p_full[buf], (x >> 1) & 1);
      landed = mbar_test(&c.full[st], lap & 1);               // of the next scores
      if (!__all_sync(0xffffffffu, here) && !tc_wait_warp(c, &c.p_full[buf], (x >> 1) & 1, a.err)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ts(tmem + kOCol + o * 128, tmem + kSCol + buf * 64 + 8 * k, v + k * (2048 >> 4), pv_desc, !(first && k == 0));
        tc_commit(&c.empty[st_pv]);
        tc_commit(&c.o_done);
        if (last) tc_commit(&c.o_last[o]);
      }
      __syncwarp();
      st_pv = st_pv + 1 == kStages ? 0 : st_pv + 1;
      return true;
    };
    for (int item = blockIdx.x; item < n_groups && ok; item += gridDim.x) {
      const int nt = (keys_of(item) + kTile - 1) / kTile;
      if (nt == 0) continue;
      for (int i = 0; i < nt && ok; ++i, ++tiles) {
        const uint32_t buf = tiles & 1;
        ok = (__all_sync(0xffffffffu, landed) || tc_wait_warp(c, &c.full[st], lap & 1, a.err)) &&
             (i > 0 || tc_wait_warp(c, &c.q_full, items & 1, a.err));
        if (!ok) break;
        landed = false;
        fence_async_smem();                    // the copies are generic-proxy writes, the tensor core reads by the async proxy
        tc_fence_after();
        const uint64_t kd = k0 + st * (kKBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kDk / 16; ++k)
            mma_ts(tmem + kSCol + buf * 64, tmem + kQCol + 8 * k, kd + ((k >> 2) * (kTile * 128) + (k & 3) * 32) / 16, qk_desc,
                   k > 0);
          tc_commit(&c.s_full[buf]);
          if (i == nt - 1) tc_commit(&c.q_empty);
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          ++lap;
        }
        if (i > 0) ok = pv(tiles - 1, i == 1, false);
      }
      if (!ok) break;
      ok = pv(tiles - 1, nt == 1, true);
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
}

}  // namespace

// Tokens of a group: two, but one where every token has an SM of its own, which
// then goes through its own keys alone (96 queries of 640 slots, trees of 16: 19.1 us in
// pairs, 15.8 alone; 152, trees of 8: 19.1 and 16.7).
static int group_of(int seqs, int tokens) { return tokens > 1 && seqs * tokens > device_sm_count() ? 2 : 1; }

static size_t plan_words(int seqs, int tokens, int topk, int swa, int group) {
  const int keys = plan_keys(topk, swa, tokens, group);
  return size_t(seqs) * ((tokens + group - 1) / group) * size_t(plan_entries(keys) + keys);
}

// Words of the plan of a launch on the current device, and the most of one on any (of up to 1,024 SMs).
size_t tree_plan_words(int seqs, int tokens, int topk, int swa) {
  return plan_words(seqs, tokens, topk, swa, group_of(seqs, tokens));
}
size_t tree_plan_most(int seqs, int tokens, int topk, int swa) {
  const size_t pairs = tokens > 1 ? plan_words(seqs, tokens, topk, swa, 2) : 0;
  const size_t alone = tokens == 1 || (long long)seqs * tokens <= 1024 ? plan_words(seqs, tokens, topk, swa, 1) : 0;
  return pairs > alone ? pairs : alone;
}

cudaError_t launch_tree_attn_tc(const TreeArgs& a, int seqs, void* plan, cudaStream_t st) {
  cudaError_t e = once_per_device(kSetupTreePair, [] {
    return cudaFuncSetAttribute(tree_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e != cudaSuccess) return e;
  const int group = group_of(seqs, a.tokens), n_groups = seqs * ((a.tokens + group - 1) / group);
  const uint32_t* words = static_cast<const uint32_t*>(plan);
  note_launch();
  e = launch_pdl(tree_plan_kernel, dim3(unsigned(n_groups)), dim3(kPlanThreads), (size_t(3) * a.topk + 1) * 4, st, 1, a,
                 static_cast<uint32_t*>(plan), group);
  if (e != cudaSuccess) return e;
  const int grid = n_groups < device_sm_count() ? n_groups : device_sm_count();
  note_launch();
  return launch_pdl(tree_tc_kernel, dim3(unsigned(grid)), dim3(kThreads), kSmem, st, 1, a, words, group, n_groups);
}

}  // namespace csa2
