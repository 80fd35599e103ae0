// Eviction from full caches (csa2_kv_evict).
//
// evict_select_kernel -- one cluster per sequence: the entries that stay, in
//   ascending order.  The k-th greatest 64-bit mass is found by a radix select
//   over the bits in which the masses differ (11 bits a pass: the histograms
//   of the cluster's CTAs are added up through distributed shared memory),
//   ties go to the lowest index; each warp then lists its share in order.
// evict_move_kernel -- out of place: every row is gathered by its entry, 16
//   bytes a thread, so it runs at the rate of a copy.
// evict_shift_kernel -- in place: rows only ever move down, but a row's new
//   place may still hold a row that another one needs.  A CTA therefore owns a
//   column slice of all of a sequence's rows and moves it in ascending order,
//   so that no CTA waits for another: it reads a tile of rows, meets at a
//   barrier, and writes the tile, whose rows lie at or below the rows that
//   later tiles read.
// evict_block_keys_kernel -- the result's block keys (block_key_elem).
// evict_counts_kernel -- in place, n_valid changes last: the launches before
//   read from it which sequences are evicted from.
#include "common.cuh"
#include "internal.h"

namespace csa2 {

namespace {

typedef unsigned long long u64;

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kMaxCluster = 8;

CSA2_DEV u64 mass_key(long long m) { return u64(m) ^ 0x8000000000000000ull; }   // signed order

CSA2_DEV u64 dsmem_ld_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

CSA2_DEV int dsmem_ld_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[kBins];
  __shared__ int sum[kBins];
  __shared__ u64 mn_s[kSelWarps], mx_s[kSelWarps];
  __shared__ u64 mn_c, mx_c;
  __shared__ int warp_s[kSelWarps];
  __shared__ int pick_bin, pick_above;
  __shared__ int gt_w[kSelWarps], eq_w[kSelWarps];
  __shared__ int gt_c, eq_c;
  const int seq = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = int(cluster_rank()), ncta = int(cluster_size());
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
  // entries [lo, hi) compete for `need` places; this warp's share of [0, n)
  const int lo = a.sink, hi = n - a.recent;
  int need = a.keep - a.sink - a.recent;
  const int per_warp = ((n + ncta * kSelWarps - 1) / (ncta * kSelWarps) + 31) & ~31;
  const int w0 = min(n, (rank * kSelWarps + warp) * per_warp), w1 = min(n, w0 + per_warp);
  const int c0 = max(w0, lo), c1 = min(w1, hi);

  // bits in which the competing masses differ
  u64 mn = ~0ull, mx = 0;
  for (int j = c0 + lane; j < c1; j += 32) {
    const u64 k = mass_key(mass[j]);
    mn = min(mn, k);
    mx = max(mx, k);
  }
  for (int o = 16; o > 0; o >>= 1) {
    mn = min(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (lane == 0) {
    mn_s[warp] = mn;
    mx_s[warp] = mx;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 0; w < kSelWarps; ++w) {
      mn = min(mn, mn_s[w]);
      mx = max(mx, mx_s[w]);
    }
    mn_c = mn;
    mx_c = mx;
  }
  cluster_sync_all();
  mn = ~0ull;
  mx = 0;
  for (int r = 0; r < ncta; ++r) {
    mn = min(mn, dsmem_ld_u64(dsmem_addr(&mn_c, r)));
    mx = max(mx, dsmem_ld_u64(dsmem_addr(&mx_c, r)));
  }
  // (count of competing keys > need >= 0, so mn <= mx here)
  // Invariant: the keys whose bits from `shift` up equal `prefix` hold the
  // need-th greatest, and every key with greater such bits is taken.
  int shift = 64 - __clzll((long long)(mn ^ mx));      // mn ^ mx == 0: clz 64, shift 0
  u64 prefix = shift >= 64 ? 0 : mx >> shift;
  bool whole = need == 0;                              // nothing competes for a place
  while (shift > 0 && !whole) {
    const int bits = min(kBits, shift), next = shift - bits, bins = 1 << bits;
    for (int i = tid; i < bins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int j = c0 + lane; j < c1; j += 32) {
      const u64 k = mass_key(mass[j]);
      if ((shift >= 64 ? 0 : k >> shift) == prefix) atomicAdd(&hist[int((k >> next) & u64(bins - 1))], 1);
    }
    cluster_sync_all();
    for (int i = tid; i < bins; i += kSelThreads) {
      int s = 0;
      for (int r = 0; r < ncta; ++r) s += dsmem_ld_s32(dsmem_addr(&hist[i], r));
      sum[i] = s;
    }
    __syncthreads();
    // the bin of the need-th greatest: thread t owns bins [4t, 4t + 4), counted from the top
    int own = 0;
    for (int i = 0; i < kBins / kSelThreads; ++i) {
      const int bin = bins - 1 - (tid * (kBins / kSelThreads) + i);
      if (bin >= 0) own += sum[bin];
    }
    int incl = own;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_s[warp] = incl;
    __syncthreads();
    int above = incl - own;
    for (int w = 0; w < warp; ++w) above += warp_s[w];
    for (int i = 0; i < kBins / kSelThreads; ++i) {
      const int bin = bins - 1 - (tid * (kBins / kSelThreads) + i);
      if (bin < 0) break;
      if (above < need && need <= above + sum[bin]) {
        pick_bin = bin;
        pick_above = above;
      }
      above += sum[bin];
    }
    __syncthreads();
    const int bin = pick_bin;
    need -= pick_above;
    whole = need == sum[bin];                          // all of the bin's keys are taken
    prefix = (prefix << bits) | u64(bin);
    shift = next;
    cluster_sync_all();                                // the peers have read this CTA's histogram
  }
  // a key is taken if its bits from `shift` up are above the prefix, or equal
  // to it while places are left (ties: `need` of them by index; whole: all)
  auto above_cut = [&](u64 k) { return (shift >= 64 ? 0 : k >> shift) > prefix; };
  auto at_cut = [&](u64 k) { return (shift >= 64 ? 0 : k >> shift) == prefix; };
  int gt = 0, eq = 0;
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int j = j0 + lane;
    bool g = false, e = false;
    if (j < w1) {
      if (j < lo || j >= hi) {
        g = true;
      } else {
        const u64 k = mass_key(mass[j]);
        g = above_cut(k);
        e = at_cut(k);
      }
    }
    gt += __popc(__ballot_sync(0xffffffffu, g));
    eq += __popc(__ballot_sync(0xffffffffu, e));
  }
  if (lane == 0) {
    gt_w[warp] = gt;
    eq_w[warp] = eq;
  }
  __syncthreads();
  if (tid == 0) {
    int g = 0, e = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      g += gt_w[w];
      e += eq_w[w];
    }
    gt_c = g;
    eq_c = e;
  }
  cluster_sync_all();
  int gt_before = 0, eq_before = 0;
  for (int r = 0; r < rank; ++r) {
    gt_before += dsmem_ld_s32(dsmem_addr(&gt_c, r));
    eq_before += dsmem_ld_s32(dsmem_addr(&eq_c, r));
  }
  for (int w = 0; w < warp; ++w) {
    gt_before += gt_w[w];
    eq_before += eq_w[w];
  }
  cluster_arrive();                                    // this CTA has read its peers' counts
  const unsigned below = (1u << lane) - 1u;
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int j = j0 + lane;
    bool g = false, e = false;
    if (j < w1) {
      if (j < lo || j >= hi) {
        g = true;
      } else {
        const u64 k = mass_key(mass[j]);
        g = above_cut(k);
        e = at_cut(k);
      }
    }
    const unsigned mg = __ballot_sync(0xffffffffu, g), me = __ballot_sync(0xffffffffu, e);
    const int eq_at = eq_before + __popc(me & below);
    const int at = gt_before + __popc(mg & below) + min(eq_at, need);
    if ((g || (e && eq_at < need)) && at < a.keep) kept[at] = j;
    gt_before += __popc(mg);
    eq_before += __popc(me);
  }
  if (rank == 0 && tid == 0 && !a.in_place) a.n_valid_out[seq] = n_out;
  cluster_wait();                                      // the peers have read this CTA's counts
}

// ------------------------------------------------------------------ moving the rows

// Entries of a sequence before and after; in place n_valid holds the former
// until evict_counts_kernel, the last launch.
CSA2_DEV int evict_counts(const EvictArgs& a, int seq, int& n_out) {
  const int n = clamp_count(a.n_valid[seq], a.n_entries, nullptr);
  n_out = n > a.trigger ? a.keep : n;
  return n;
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;

template <typename U>
CSA2_DEV void gather_rows(void* dst, const void* src, int row_bytes, long long row0, int r0, int nr, const int* from) {
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
      if (i < total) d[i] = v[m];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  __shared__ int from[kMoveRows];
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
  if (a.wide) {
    gather_rows<uint4>(a.k_main_out, a.k_main, a.k_bytes, row0, r0, nr, from);
    gather_rows<uint4>(a.v_main_out, a.v_main, a.v_bytes, row0, r0, nr, from);
    gather_rows<uint4>(a.k_idx_out, a.k_idx, a.x_bytes, row0, r0, nr, from);
  } else {
    gather_rows<uint16_t>(a.k_main_out, a.k_main, a.k_bytes, row0, r0, nr, from);
    gather_rows<uint16_t>(a.v_main_out, a.v_main, a.v_bytes, row0, r0, nr, from);
    gather_rows<uint16_t>(a.k_idx_out, a.k_idx, a.x_bytes, row0, r0, nr, from);
  }
}

constexpr int kShiftThreads = 512;

// Columns [u0, u0 + w) of the rows of `base` (row length `per` units), moved
// down to the places of `kept`, tile by tile.
template <typename U>
CSA2_DEV void shift_columns(U* base, int per, int u0, int w, const int* kept, int first, int n) {
  constexpr int kU = 8;
  const int step = kShiftThreads / w;                   // rows per round
  const int r = threadIdx.x / w, u = u0 + threadIdx.x - r * w;
  const bool on = r < step;
  for (int t0 = first; t0 < n; t0 += kU * step) {
    U v[kU];
#pragma unroll
    for (int m = 0; m < kU; ++m) {
      const int j = t0 + m * step + r;
      if (on && j < n) v[m] = base[(long long)kept[j] * per + u];
    }
    // The tile has been read.  Its writes need no barrier behind them: the next
    // tile reads rows at or above its own first place, which this one never writes.
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kU; ++m) {
      const int j = t0 + m * step + r;
      if (on && j < n) base[(long long)j * per + u] = v[m];
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

cudaError_t launch_kv_evict(const EvictArgs& a, int seqs, cudaStream_t st) {
  if (seqs == 0) return cudaSuccess;
  // CTAs per sequence: 8, unless the sequences alone fill the SMs or are short
  int c = kMaxCluster;
  while (c > 1 && (c * seqs > 2 * device_sm_count() || a.n_entries < c * 2048)) c >>= 1;
  note_launch();
  cudaError_t e = launch_pdl(evict_select_kernel, dim3(unsigned(c), unsigned(seqs)), dim3(kSelThreads), 0, st,
                             unsigned(c), a);
  if (e != cudaSuccess) return e;
  note_launch();
  if (!a.in_place) {
    e = launch_pdl(evict_move_kernel, dim3(unsigned((a.n_entries + kMoveRows - 1) / kMoveRows), unsigned(seqs)),
                   dim3(kMoveThreads), 0, st, 1, a);
  } else {
    const int unit = a.wide ? 16 : 2;
    // slices of 128 bytes, down to 32 (a sector) while the CTAs do not fill the SMs
    int width = 128 / unit;
    auto slices = [&](int w) {
      int s = 1;
      for (int bytes : {a.k_bytes, a.v_bytes, a.x_bytes}) s += (bytes / unit + w - 1) / w;
      return s;
    };
    while (width * unit > 32 && slices(width) * seqs < 2 * device_sm_count()) width >>= 1;
    const dim3 grid(unsigned(slices(width)), unsigned(seqs));
    e = a.wide ? launch_pdl(evict_shift_kernel<uint4>, grid, dim3(kShiftThreads), 0, st, 1, a, width)
               : launch_pdl(evict_shift_kernel<uint16_t>, grid, dim3(kShiftThreads), 0, st, 1, a, width);
  }
  if (e != cudaSuccess) return e;
  if (a.kb != nullptr) {
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
