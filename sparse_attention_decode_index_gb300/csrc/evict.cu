// Eviction from full caches (csa2_kv_evict).
//
// evict_select_kernel -- one cluster per sequence: the entries that stay, in
//   ascending order.  The k-th greatest 64-bit mass is found by a radix select:
//   first by octaves of the masses, counted while they are loaded, then 8 bits a
//   pass over the range that is left, cut to the masses' own; ties go to the
//   lowest index; each warp then lists its share in order.  Every CTA keeps
//   its share of the masses in shared memory, read once, so that a pass costs a
//   sweep of shared memory, one push of 256 counts into every CTA of the
//   cluster and one cluster barrier.  Masses are skewed (many entries draw next to
//   none), so a bin has 16 counts in different banks, a lane's by its number.
//   Bound by the sweeps' instructions and the passes' cluster barriers: 64 x 8,192
//   masses 12.9 us, 1 x 262,144 on 16 CTAs 21.1 us (one count a bin and a pass of its
//   own for the range: 15.5 and 27; masses read again a pass: 29 and 100).
// evict_move_kernel -- out of place: every row is gathered by its entry, 16
//   bytes a thread, so it runs at the rate of a copy: 64 x 8,192 entries down to 6,145
//   82 to 92 us, where a plain copy of these bytes takes 83.
// evict_shift_kernel -- in place: rows only ever move down, but a row's new
//   place may still hold a row that another one needs.  A CTA therefore owns a
//   column slice of all of a sequence's rows and moves it in ascending order,
//   so that no CTA waits for another.  Few sequences leave it few CTAs: it is
//   bound by their loads' latency then, a tile read ahead of the one that is written
//   (64 x 8,192: 144 us with the selection, 1 x 262,144: 367 us, 49 CTAs).
// evict_block_keys_kernel -- the result's block keys, where the move has not
//   made them (in place, or blocks that do not divide its tiles).
// evict_counts_kernel -- in place, n_valid changes last: the launches before
//   read from it which sequences are evicted from.
#include <atomic>

#include "common.cuh"
#include "draft.h"

namespace csa2 {

namespace {

typedef unsigned long long u64;

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;
constexpr int kLoads = 8;           // masses a thread has on their way
constexpr int kMaxCluster = 16;
constexpr int kMaxCached = 24576;   // masses a CTA keeps in shared memory (192 KB)
static_assert(kMaxCached / kSelWarps <= 32 * 32, "a warp's ballots fit one register a lane");

CSA2_DEV u64 mass_key(long long m) { return u64(m) ^ 0x8000000000000000ull; }   // signed order

CSA2_DEV void dsmem_st_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// The first pass's bin of a key: 0 for masses below 0, then 4 an octave, and the keys of one.
constexpr u64 kZero = 0x8000000000000000ull;
CSA2_DEV int first_bin(u64 k) {
  if (k < kZero) return 0;
  const u64 x = k - kZero;
  const int e = 63 - __clzll((long long)(x | 3));      // >= 1
  return 1 + (x < 4 ? int(x) : (e - 1) * 4 + (int(x >> (e - 2)) & 3));
}
CSA2_DEV void first_range(int bin, u64& low, u64& high) {
  if (bin == 0) {
    low = 0;
    high = kZero - 1;
  } else if (bin <= 4) {                               // one value a bin
    low = high = kZero + u64(bin - 1);
  } else {                                             // the octave e = (bin - 1) / 4 + 1, less the two bits
    const int width = (bin - 1) / 4 - 1;
    low = kZero + (u64(4 + ((bin - 1) & 3)) << width);
    high = low + ((1ull << width) - 1);
  }
}

struct SelectShared {
  int table[2][kMaxCluster][kBins];   // every CTA's counts, of even and odd passes
  u64 range[kMaxCluster][2];          // every CTA's least and greatest key
  int taken[kMaxCluster][2];          // every CTA's keys above the cut and at it
  int hist[kBins];
  int warp_a[kSelWarps], warp_b[kSelWarps];
  u64 warp_mn[kSelWarps], warp_mx[kSelWarps];
  int bin, above, total;
};

template <bool kCached>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];
  SelectShared& sh = *reinterpret_cast<SelectShared*>(dyn);
  u64* cache = reinterpret_cast<u64*>(dyn + sizeof(SelectShared));
  const int seq = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = int(cluster_rank()), ncta = int(cluster_size());
  reinterpret_cast<int4*>(&sh.table[1][0][0])[tid] = make_int4(0, 0, 0, 0);
  pdl_wait();
  const int n = clamp_count(a.n_valid[seq], a.n_entries, rank == 0 && tid == 0 ? a.err : nullptr);
  int* kept = a.kept + (long long)seq * a.n_entries;
  const long long* mass = a.mass + (long long)seq * a.n_entries;
  const bool evicts = n > a.trigger;
  const int n_out = evicts ? a.keep : n;
  // behind the last entry
  for (int j = n_out + rank * kSelThreads + tid; j < a.n_entries; j += ncta * kSelThreads) kept[j] = -1;
  if (!evicts) {
    for (int j = rank * kSelThreads + tid; j < n; j += ncta * kSelThreads) kept[j] = j;
    if (rank == 0 && tid == 0 && !a.in_place) a.n_valid_out[seq] = n;
    return;
  }
  // entries [lo, hi) compete for `need` places.  Shares of [0, n): a CTA's, and
  // in it a warp's (whole groups of 32, so that ballots keep the order).
  const int lo = a.sink, hi = n - a.recent;
  int need = a.keep - a.sink - a.recent;
  const int per_warp = ((n + ncta * kSelWarps - 1) / (ncta * kSelWarps) + 31) & ~31;
  const int cta0 = min(n, rank * kSelWarps * per_warp);
  const int w0 = min(n, (rank * kSelWarps + warp) * per_warp), w1 = min(n, w0 + per_warp);
  const int c0 = max(w0, lo), c1 = min(w1, hi);
  __syncthreads();                                     // the zeros of the first pass's counts
  // its own warp's keys only: no barrier between filling the cache and reading it
  auto key = [&](int j) -> u64 { return kCached ? cache[j - cta0] : mass_key(mass[j]); };

  // The keys, their range, and the first pass's counts: 16 a bin, so that lanes
  // of a warp that share a bin mostly count in words of their own.  A pass's
  // lie in the table that the pass does not exchange counts in: the last pass's, which has
  // been read, and which a peer writes only when all have finished this pass.
  u64 mn = ~0ull, mx = 0;
  for (int j0 = w0 + lane; j0 < w1; j0 += 32 * kLoads) {
    u64 k[kLoads];
#pragma unroll
    for (int x = 0; x < kLoads; ++x) k[x] = j0 + 32 * x < w1 ? mass_key(mass[j0 + 32 * x]) : 0;
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const int j = j0 + 32 * x;
      if (j >= w1) break;
      if (kCached) cache[j - cta0] = k[x];
      if (j >= c0 && j < c1) {
        mn = min(mn, k[x]);
        mx = max(mx, k[x]);
        atomicAdd(&sh.table[1][0][0] + first_bin(k[x]) * 16 + (lane & 15), 1);
      }
    }
  }
  for (int o = 16; o > 0; o >>= 1) {
    mn = min(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (lane == 0) {
    sh.warp_mn[warp] = mn;
    sh.warp_mx[warp] = mx;
  }
  cluster_arrive();                                    // (every CTA of the cluster runs before any writes into it)
  // Invariant: the keys of [low, high] hold the need-th greatest, and every
  // greater key is taken; high - low < 2^shift.  The first pass bins a key by its octave
  // and the two bits below its leading one, the later ones by 8 bits of its
  // distance to low; more keys compete than there are places.
  int shift = 64;
  u64 low = 0, high = ~0ull;
  bool whole = need == 0;                              // all keys of the range are taken (or none, as no place is left)
  if (whole) cluster_wait();
  for (int pass = 0; shift > 0 && !whole; ++pass) {
    const bool first = pass == 0;
    const int bits = min(8, shift), next = shift - bits;
    int* count = &sh.table[(pass + 1) & 1][0][0];
    if (!first) {
      reinterpret_cast<int4*>(count)[tid] = make_int4(0, 0, 0, 0);
      __syncthreads();
#pragma unroll 2
      for (int j0 = c0 & ~31; j0 < c1; j0 += 32) {
        const int j = j0 + lane;
        if (j < c0 || j >= c1) continue;
        const u64 k = key(j);
        if (k >= low && k <= high) atomicAdd(count + int((k - low) >> next) * 16 + (lane & 15), 1);
      }
    }
    __syncthreads();
    int(*table)[kBins] = sh.table[pass & 1];
    const int4 c4 = reinterpret_cast<const int4*>(count)[tid];      // four threads a bin
    int own4 = c4.x + c4.y + c4.z + c4.w;
    own4 += __shfl_xor_sync(0xffffffffu, own4, 1);
    own4 += __shfl_xor_sync(0xffffffffu, own4, 2);
    if ((tid & 3) == 0) sh.hist[tid >> 2] = own4;
    __syncthreads();
    if (first) {
      cluster_wait();
      if (warp == 0) {
        mn = sh.warp_mn[lane];
        mx = sh.warp_mx[lane];
        for (int o = 16; o > 0; o >>= 1) {
          mn = min(mn, __shfl_xor_sync(0xffffffffu, mn, o));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        if (lane < ncta) {
          dsmem_st_u64(dsmem_addr(&sh.range[rank][0], lane), mn);
          dsmem_st_u64(dsmem_addr(&sh.range[rank][1], lane), mx);
        }
      }
    }
    for (int i = tid; i < ncta * kBins; i += kSelThreads)           // (a warp's words go to one peer, side by side)
      dsmem_st_u32(dsmem_addr(&table[rank][i & (kBins - 1)], i / kBins), uint32_t(sh.hist[i & (kBins - 1)]));
    cluster_sync_all();
    if (tid < kBins) {
      int all = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < ncta) all += table[r][tid];
      sh.hist[tid] = all;
    }
    __syncthreads();
    // the bin of the need-th greatest: lane l of warp 0 owns bins 8 l .. 8 l + 7, counted from the top
    if (warp == 0) {
      int own = 0, v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = sh.hist[kBins - 1 - (lane * 8 + i)];
        own += v[i];
      }
      int incl = own;
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      int above = incl - own;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (above < need && need <= above + v[i]) {
          sh.bin = kBins - 1 - (lane * 8 + i);
          sh.above = above;
          sh.total = v[i];
        }
        above += v[i];
      }
    }
    __syncthreads();
    need -= sh.above;
    whole = need == sh.total;
    if (!first) {
      low += u64(sh.bin) << next;
      high = min(high, low + ((1ull << next) - 1));
      shift = next;
    } else {
      first_range(sh.bin, low, high);
      for (int r = 0; r < ncta; ++r) {                 // no wider than the keys are
        mn = min(r == 0 ? ~0ull : mn, sh.range[r][0]);
        mx = max(r == 0 ? 0ull : mx, sh.range[r][1]);
      }
      low = max(low, mn);
      high = min(high, mx);
      shift = high == low ? 0 : 64 - __clzll((long long)(high - low));
    }
  }
  // A key is taken if it is above the range, or in it while places are left:
  // `need` of them, the lowest indices.
  int gt = 0, eq = 0;
  unsigned gt_mask = 0, eq_mask = 0;                   // lane i: the warp's i-th group of 32 entries (kCached: at most 32 groups)
#pragma unroll 4
  for (int j0 = w0, it = 0; j0 < w1; j0 += 32, ++it) {
    const int j = j0 + lane;
    bool g = false, e = false;
    if (j < w1) {
      if (j < lo || j >= hi) {
        g = true;
      } else {
        const u64 k = key(j);
        g = k > high;
        e = k >= low && !g;
      }
    }
    const unsigned mg = __ballot_sync(0xffffffffu, g), me = __ballot_sync(0xffffffffu, e);
    if (lane == it) {
      gt_mask = mg;
      eq_mask = me;
    }
    if (!kCached) {
      gt += __popc(mg);
      eq += __popc(me);
    }
  }
  if (kCached) {
    gt = __reduce_add_sync(0xffffffffu, __popc(gt_mask));
    eq = __reduce_add_sync(0xffffffffu, __popc(eq_mask));
  }
  if (lane == 0) {
    sh.warp_a[warp] = gt;
    sh.warp_b[warp] = eq;
  }
  __syncthreads();
  // before this warp: the CTA's earlier warps (lanes as warps), then the earlier CTAs
  int ga = sh.warp_a[lane], eb = sh.warp_b[lane];
  int g_cta = ga, e_cta = eb, g_warp = lane < warp ? ga : 0, e_warp = lane < warp ? eb : 0;
  for (int o = 16; o > 0; o >>= 1) {
    g_cta += __shfl_xor_sync(0xffffffffu, g_cta, o);
    e_cta += __shfl_xor_sync(0xffffffffu, e_cta, o);
    g_warp += __shfl_xor_sync(0xffffffffu, g_warp, o);
    e_warp += __shfl_xor_sync(0xffffffffu, e_warp, o);
  }
  if (warp == 0 && lane < ncta) {
    dsmem_st_u32(dsmem_addr(&sh.taken[rank][0], lane), uint32_t(g_cta));
    dsmem_st_u32(dsmem_addr(&sh.taken[rank][1], lane), uint32_t(e_cta));
  }
  cluster_sync_all();                                  // the last access to a peer's memory is before it
  int gt_before = g_warp, eq_before = e_warp;
  for (int r = 0; r < rank; ++r) {
    gt_before += sh.taken[r][0];
    eq_before += sh.taken[r][1];
  }
  const unsigned below = (1u << lane) - 1u;
  if (kCached) {
    // lane i: the entries of group i that are taken, and the place of the first
    const int pe = __popc(eq_mask);
    int upto = pe;
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    const int left = max(0, min(pe, need - (eq_before + upto - pe)));
    for (int k = pe; k > left; --k) eq_mask &= ~(1u << (31 - __clz(eq_mask)));   // (some of a group: once in a cluster)
    const unsigned taken = gt_mask | eq_mask;
    const int pt = __popc(taken);
    int start = pt;
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, start, o);
      if (lane >= o) start += u;
    }
    start += gt_before + min(eq_before, need) - pt;
#pragma unroll 4
    for (int j0 = w0, it = 0; j0 < w1; j0 += 32, ++it) {
      const unsigned t = __shfl_sync(0xffffffffu, taken, it);
      const int at = __shfl_sync(0xffffffffu, start, it) + __popc(t & below);
      if (((t >> lane) & 1u) && at < a.keep) kept[at] = j0 + lane;
    }
  } else {
    for (int j0 = w0; j0 < w1; j0 += 32) {
      const int j = j0 + lane;
      const bool in = j < w1, free = in && j >= lo && j < hi;
      const u64 k = free ? key(j) : 0;
      const bool g = in && (!free || k > high), e = free && k >= low && k <= high;
      const unsigned mg = __ballot_sync(0xffffffffu, g), me = __ballot_sync(0xffffffffu, e);
      const int eq_at = eq_before + __popc(me & below);
      const int at = gt_before + __popc(mg & below) + min(eq_at, need);
      if ((g || (e && eq_at < need)) && at < a.keep) kept[at] = j;
      gt_before += __popc(mg);
      eq_before += __popc(me);
    }
  }
  if (rank == 0 && tid == 0 && !a.in_place) a.n_valid_out[seq] = n_out;
}

// ------------------------------------------------------------------ moving the rows

// block_key_elem for entries whose rows lie elsewhere: entry r in row row_of(r).
template <typename RowOf>
CSA2_DEV float block_key_rows(const void* k_idx, const RowOf& row_of, int dim, int block, int n, int j, int d, int dtype,
                              int round_to_int) {
  const int r0 = j * block, members = min(block, n - r0);
  if (members <= 0) return 0.f;
  float sum = 0.f;
  for (int r = 0; r < members; ++r) sum += load_elem(k_idx, (long long)row_of(r0 + r) * dim + d, dtype);
  const float mean = sum / float(members);
  return round_to_int ? rintf(mean) : mean;
}

// Entries of a sequence before and after; in place n_valid holds the former
// until evict_counts_kernel, the last launch.
CSA2_DEV int evict_counts(const EvictArgs& a, int seq, int& n_out) {
  const int n = clamp_count(a.n_valid[seq], a.n_entries, nullptr);
  n_out = n > a.trigger ? a.keep : n;
  return n;
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;   // a tile holds whole blocks of 8 (or any divisor of 32)

// Rows r0 .. r0 + nr - 1 from rows `from`; `copy` (shared memory, nullable) gets them too.
template <typename U>
CSA2_DEV void gather_rows(void* dst, const void* src, int row_bytes, long long row0, int r0, int nr, const int* from,
                          U* copy = nullptr) {
  const int per = row_bytes / int(sizeof(U)), total = nr * per;
  U* d = static_cast<U*>(dst) + (row0 + r0) * per;
  const U* s = static_cast<const U*>(src) + row0 * per;
  constexpr int kU = 4;
  for (int i0 = threadIdx.x; i0 < total; i0 += kU * kMoveThreads) {
    U v[kU];
#pragma unroll
    for (int m = 0; m < kU; ++m) {
      const int i = i0 + m * kMoveThreads;
      if (i < total) v[m] = s[(long long)from[i / per] * per + i % per];
    }
#pragma unroll
    for (int m = 0; m < kU; ++m) {
      const int i = i0 + m * kMoveThreads;
      if (i >= total) break;
      d[i] = v[m];
      if (copy != nullptr) copy[i] = v[m];
    }
  }
}

template <typename U>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  __shared__ int from[kMoveRows];
  extern __shared__ __align__(16) uint8_t keys[];       // [kMoveRows] indexer keys, where the tile makes block keys
  const int seq = blockIdx.y, r0 = blockIdx.x * kMoveRows, tid = threadIdx.x;
  pdl_wait();
  int n;
  evict_counts(a, seq, n);
  const long long row0 = (long long)seq * a.n_entries;
  const int nr = max(0, min(kMoveRows, n - r0));
  if (tid < kMoveRows && r0 + tid < a.n_entries) {
    const int e = tid < nr ? a.kept[row0 + r0 + tid] : -1;
    from[tid] = e;
    a.mass_out[row0 + r0 + tid] = e >= 0 ? a.mass[row0 + e] : 0;
  }
  __syncthreads();
  const bool blocks = a.kb != nullptr && kMoveRows % a.block == 0;
  gather_rows<U>(a.k_idx_out, a.k_idx, a.x_bytes, row0, r0, nr, from, blocks ? reinterpret_cast<U*>(keys) : nullptr);
  gather_rows<U>(a.k_main_out, a.k_main, a.k_bytes, row0, r0, nr, from);
  gather_rows<U>(a.v_main_out, a.v_main, a.v_bytes, row0, r0, nr, from);
  if (!blocks) return;
  __syncthreads();
  const int j0 = r0 / a.block, nb = min(kMoveRows / a.block, a.nb_cap - j0);
  for (int i = tid; i < nb * a.idx_dim; i += kMoveThreads) {
    const int j = j0 + i / a.idx_dim, d = i % a.idx_dim;
    const float v = block_key_rows(keys, [&](int r) { return r - r0; }, a.idx_dim, a.block, n, j, d, a.dtype, a.round_to_int);
    store_elem(a.kb, ((long long)seq * a.nb_cap + j) * a.idx_dim + d, a.dtype, v);
  }
}

constexpr int kShiftThreads = 512;

// Columns [u0, u0 + w) of the rows of `base` (row length `per` units), moved
// down to the places of `kept`, tile by tile.  A tile's rows are read while the
// one before it is written: they lie at or above its own first place, which
// the earlier tile never writes.  Its writes wait until the whole CTA has read it.
template <typename U>
CSA2_DEV void shift_columns(U* base, int per, int u0, int w, const int* kept, int first, int n) {
  constexpr int kU = 8;
  const int step = kShiftThreads / w;                   // rows per round
  const int r = threadIdx.x / w, u = u0 + threadIdx.x - r * w;
  const bool on = r < step;
  int from[kU];
  auto indices = [&](int t0) {
#pragma unroll
    for (int m = 0; m < kU; ++m) {
      const int j = t0 + m * step + r;
      from[m] = on && j < n ? kept[j] : -1;
    }
  };
  U now[kU], next[kU];
  indices(first);
#pragma unroll
  for (int m = 0; m < kU; ++m)
    if (from[m] >= 0) now[m] = base[(long long)from[m] * per + u];
  indices(first + kU * step);
  for (int t0 = first; t0 < n; t0 += kU * step) {
#pragma unroll
    for (int m = 0; m < kU; ++m)
      if (from[m] >= 0) next[m] = base[(long long)from[m] * per + u];
    indices(t0 + 2 * kU * step);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kU; ++m) {
      const int j = t0 + m * step + r;
      if (on && j < n) base[(long long)j * per + u] = now[m];
      now[m] = next[m];
    }
  }
}

// grid.x: the column slices of k, v and k_idx (`width` units each), then one CTA for the masses.
template <typename U>
__global__ void __launch_bounds__(kShiftThreads) evict_shift_kernel(const EvictArgs a, int width) {
  const int seq = blockIdx.y;
  pdl_wait();
  int n;
  if (evict_counts(a, seq, n) <= a.trigger) return;
  const long long row0 = (long long)seq * a.n_entries;
  const int* kept = a.kept + row0;
  int first = 0, end = n;                               // the first row that moves
  while (first < end) {
    const int mid = (first + end) / 2;
    if (kept[mid] == mid) first = mid + 1;
    else end = mid;
  }
  int s = blockIdx.x;
  const int rows[3] = {a.k_bytes, a.v_bytes, a.x_bytes};
  void* const base[3] = {a.k_main_out, a.v_main_out, a.k_idx_out};
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int per = rows[i] / int(sizeof(U)), slices = (per + width - 1) / width;
    if (s >= 0 && s < slices) {
      const int u0 = s * width;
      shift_columns<U>(static_cast<U*>(base[i]) + row0 * per, per, u0, min(width, per - u0), kept, first, n);
      return;
    }
    s -= slices;
  }
  long long* mass = a.mass_out + row0;
  shift_columns<long long>(mass, 1, 0, 1, kept, first, n);
  for (int j = n + int(threadIdx.x); j < a.n_entries; j += kShiftThreads) mass[j] = 0;
}

__global__ void __launch_bounds__(256) evict_block_keys_kernel(const EvictArgs a) {
  const int seq = blockIdx.y;
  pdl_wait();
  int n;
  if (evict_counts(a, seq, n) <= a.trigger && a.in_place) return;
  const long long row0 = (long long)seq * a.n_entries;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)a.nb_cap * a.idx_dim) return;
  const int j = int(i / a.idx_dim), d = int(i % a.idx_dim);
  const float v = block_key_elem(a.k_idx_out, row0, a.idx_dim, a.block, n, j, d, a.dtype, a.round_to_int);
  store_elem(a.kb, (long long)seq * a.nb_cap * a.idx_dim + i, a.dtype, v);
}

__global__ void __launch_bounds__(256) evict_counts_kernel(const EvictArgs a, int seqs) {
  pdl_wait();
  const int seq = blockIdx.x * 256 + threadIdx.x;
  if (seq >= seqs) return;
  int n;
  evict_counts(a, seq, n);
  a.n_valid_out[seq] = n;
}

}  // namespace

// Masses of one CTA of a cluster of c: whole groups of 32 for every warp.
static int share(const EvictArgs& a, int c) {
  return ((a.n_entries + c * kSelWarps - 1) / (c * kSelWarps) + 31) / 32 * 32 * kSelWarps;
}

static cudaError_t select_setup() {
  return once_per_device(kSetupEvict, [] {
    constexpr int most = int(sizeof(SelectShared)) + kMaxCached * 8;
    const cudaError_t r = cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
}

// Whether clusters of 16 CTAs with full caches can run on the current device (asked once per device).
static cudaError_t wide_clusters(bool& fits) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = select_setup();
  if (e != cudaSuccess) return e;
  const bool slot = dev >= 0 && dev < kDevices;
  int got = slot ? known[dev].load(std::memory_order_relaxed) : 0;
  if (got == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = sizeof(SelectShared) + kMaxCached * 8;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int active = 0;
    e = cudaOccupancyMaxActiveClusters(&active, evict_select_kernel<true>, &cfg);
    if (e != cudaSuccess) return e;
    got = active > 0 ? 1 : 2;
    if (slot) known[dev].store(got, std::memory_order_relaxed);
  }
  fits = got == 1;
  return cudaSuccess;
}

cudaError_t launch_kv_evict(const EvictArgs& a, int seqs, cudaStream_t st) {
  if (seqs == 0) return cudaSuccess;
  // CTAs per sequence: as many as leave every sequence's cluster resident (one
  // CTA an SM) and a CTA a thousand masses, up to 8; more where 8, or those,
  // could not keep their masses in shared memory.  16 is not a portable size.
  int c = 8;
  while (c > 1 && (c * seqs > device_sm_count() || a.n_entries < c * 1024)) c >>= 1;
  while (c < 8 && share(a, c) > kMaxCached) c <<= 1;
  if (share(a, 8) > kMaxCached && share(a, 16) <= kMaxCached) {
    bool fits = false;
    const cudaError_t r = wide_clusters(fits);
    if (r != cudaSuccess) return r;
    if (fits) c = 16;
  }
  const bool cached = share(a, c) <= kMaxCached;
  if (cached) {
    const cudaError_t r = select_setup();
    if (r != cudaSuccess) return r;
  }
  const size_t smem = sizeof(SelectShared) + (cached ? size_t(share(a, c)) * 8 : 0);
  note_launch();
  cudaError_t e = launch_pdl(cached ? evict_select_kernel<true> : evict_select_kernel<false>,
                             dim3(unsigned(c), unsigned(seqs)), dim3(kSelThreads), smem, st, unsigned(c), a);
  if (e != cudaSuccess) return e;
  note_launch();
  if (!a.in_place) {
    const dim3 grid(unsigned((a.n_entries + kMoveRows - 1) / kMoveRows), unsigned(seqs));
    const size_t keys = a.kb != nullptr && kMoveRows % a.block == 0 ? size_t(kMoveRows) * a.x_bytes : 0;
    if (keys > 48 * 1024) {
      e = once_per_device(kSetupEvictMove, [] {
        const cudaError_t r = cudaFuncSetAttribute(evict_move_kernel<uint4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kMoveRows * 4096);
        if (r != cudaSuccess) return r;
        return cudaFuncSetAttribute(evict_move_kernel<uint16_t>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kMoveRows * 4096);
      });
      if (e != cudaSuccess) return e;
    }
    e = launch_pdl(a.wide ? evict_move_kernel<uint4> : evict_move_kernel<uint16_t>, grid, dim3(kMoveThreads), keys, st, 1, a);
  } else {
    const int unit = a.wide ? 16 : 2;
    // slices of 128 bytes, down to 16 while the CTAs do not fill the SMs
    int width = 128 / unit;
    auto slices = [&](int w) {
      int s = 1;
      for (int bytes : {a.k_bytes, a.v_bytes, a.x_bytes}) s += (bytes / unit + w - 1) / w;
      return s;
    };
    while (width * unit > 16 && slices(width) * seqs < 2 * device_sm_count()) width >>= 1;
    const dim3 grid(unsigned(slices(width)), unsigned(seqs));
    e = a.wide ? launch_pdl(evict_shift_kernel<uint4>, grid, dim3(kShiftThreads), 0, st, 1, a, width)
               : launch_pdl(evict_shift_kernel<uint16_t>, grid, dim3(kShiftThreads), 0, st, 1, a, width);
  }
  if (e != cudaSuccess) return e;
  if (a.kb != nullptr && (a.in_place || kMoveRows % a.block != 0)) {
    note_launch();
    const long long elems = (long long)a.nb_cap * a.idx_dim;
    e = launch_pdl(evict_block_keys_kernel, dim3(unsigned((elems + 255) / 256), unsigned(seqs)), dim3(256), 0, st, 1, a);
    if (e != cudaSuccess) return e;
  }
  if (!a.in_place) return cudaSuccess;
  note_launch();
  return launch_pdl(evict_counts_kernel, dim3(unsigned((seqs + 255) / 256)), dim3(256), 0, st, 1, a, seqs);
}

}  // namespace csa2
