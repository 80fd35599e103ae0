// The packed main cache: entries appended to it, and rows of it as numbers.
// The format stands in kv4.cuh.
#include "kv4.cuh"

namespace csa2 {

namespace {

constexpr int kThreads = 256;
constexpr int kTileEntries = 64;   // packed in shared memory before they are written as whole lines (half of it beyond 48 KB)

// ------------------------------------------------------------------ append

// Groups of 16 numbers that a thread has on their way: as they lie in memory (kWide), or one by one.
template <bool kF32>
struct Raw {
  uint4 v[kF32 ? 4 : 2];
  CSA2_DEV void load(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < (kF32 ? 4 : 2); ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  CSA2_DEV void numbers(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < (kF32 ? 4 : 2); ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (kF32) {
          x[4 * i + e] = __uint_as_float(w[e]);
        } else {
          x[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
          x[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
      }
    }
  }
};

// Each CTA packs per_cta of a sequence's new entries: a thread packs a group of 16 dims at a time into shared memory, from
// where the entries, contiguous in the cache, go out in 16-byte pieces.  The first groups are asked for beside the counts,
// whatever these say (the rows up to max_new can be read).  A block's summary key is the CTA's that has its first new
// entry; its members come from the cache in front of the new entries and from the new ones, never from what
// another CTA writes.
//
// Measured: one entry of each of 64 sequences 4.9 us, their rows back 2.1 (latency); 8,191 entries of each of
// 16 sequences 33.7 us with the counts, where their 142 MB would take 21, in fp32 58.0 (34): a CTA loads, packs, waits and stores
// once, and nothing of the next entries is on its way meanwhile (DRAM 41 %, issue slots 64 %, fp32 48 % and 48 %; fewer conversions
// gained nothing).
template <bool kF32>
__global__ void __launch_bounds__(kThreads, kF32 ? 3 : 5) kv4_append_kernel(const Kv4AppendArgs a) {
  extern __shared__ __align__(16) uint8_t tile[];          // [per_cta][entry]
  constexpr int kBatch = 2, kE = kF32 ? 4 : 2;             // groups a thread has on their way; an element's bytes
  const int b = blockIdx.y, tid = threadIdx.x;
  const int gk = kv4_groups(a.k_dim), groups = gk + kv4_groups(a.v_dim), bytes = kv4_bytes(a.k_dim, a.v_dim);
  const uint32_t m_groups = 0xffffffffu / uint32_t(groups) + 1u;   // (two at least)
  const int s0 = blockIdx.x * a.per_cta, n_most = min(a.per_cta, a.max_new - s0);
  const long long src = (long long)b * a.max_new + s0;
  const uint8_t *k_new = static_cast<const uint8_t*>(a.k_new) + src * a.k_dim * kE, *v_new = static_cast<const uint8_t*>(a.v_new) + src * a.v_dim * kE;
  pdl_wait();   // no early trigger: the next launch may read what this one writes before its own wait
  const int had = a.n_valid[b], added = a.n_new[b];
  auto place = [&](int i, int& r, int& g) {
    r = int(__umulhi(uint32_t(i), m_groups));
    g = i - r * groups;
  };
  auto from = [&](int r, int g) -> const uint8_t* {
    return g < gk ? k_new + ((long long)r * a.k_dim + 16 * g) * kE : v_new + ((long long)r * a.v_dim + 16 * (g - gk)) * kE;
  };
  Raw<kF32> raw[kBatch];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      int r, g;
      place(i0 + x * kThreads, r, g);
      if (a.wide && r < n_most) raw[x].load(from(r, g));
    }
  };
  fetch(tid);
  int* err = blockIdx.x == 0 && tid == 0 ? a.err : nullptr;
  const int nv0 = clamp_count(had, a.n_entries, err);
  int m = clamp_count(added, a.max_new, err);
  if (m > a.n_entries - nv0) {
    report(err, kErrBadCount, nv0 + m);
    m = a.n_entries - nv0;
  }
  const int n = min(n_most, m - s0);                       // entries of this CTA (none: <= 0)
  for (int i0 = tid; i0 < n * groups; i0 += kBatch * kThreads) {
    if (i0 != tid) fetch(i0);
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      int r, g;
      place(i0 + x * kThreads, r, g);
      if (r >= n) continue;
      float v[16];
      if (a.wide) {
        raw[x].numbers(v);
      } else {
        const int d = 16 * (g < gk ? g : g - gk), dim = g < gk ? a.k_dim : a.v_dim;
        const uint8_t* p = from(r, g);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = d + e < dim ? load_elem(p, e, kF32 ? 1 : 0) : 0.f;
      }
      uint2 codes;
      const uint8_t s = kv4_quantise<kF32>(v, g < gk ? a.k_down : a.v_down, codes);
      *reinterpret_cast<uint2*>(tile + r * bytes + 8 * g) = codes;
      tile[r * bytes + 8 * groups + g] = s;
    }
  }
  const int pad = bytes - 9 * groups;
  for (int i = tid; i < n * pad; i += kThreads) tile[i / pad * bytes + 9 * groups + i % pad] = 0;
  const int x_bytes = a.idx_dim * kE;
  const long long row0 = (long long)b * a.n_entries, dst = row0 + nv0 + s0;
  const uint8_t* xs = static_cast<const uint8_t*>(a.kidx_new) + src * x_bytes;
  uint8_t* xd = static_cast<uint8_t*>(a.k_idx) + dst * x_bytes;
  if (a.wide_idx) {
    for (int i = tid; i < n * (x_bytes / 16); i += kThreads) reinterpret_cast<uint4*>(xd)[i] = __ldg(reinterpret_cast<const uint4*>(xs) + i);
  } else {
    for (int i = tid; i < n * (x_bytes / 2); i += kThreads) reinterpret_cast<uint16_t*>(xd)[i] = reinterpret_cast<const uint16_t*>(xs)[i];
  }
  __syncthreads();   // the tile is packed; and every thread has read n_valid[b]
  uint4* out = reinterpret_cast<uint4*>(a.kv + dst * bytes);
  for (int i = tid; i < n * (bytes / 16); i += kThreads) out[i] = reinterpret_cast<const uint4*>(tile)[i];
  if (gridDim.x == 1 && tid == 0) a.n_valid[b] = nv0 + m;
  if (a.kb != nullptr && n > 0) {
    // blocks whose first new entry is s0 .. s0 + n - 1 of the new ones
    const int nv1 = nv0 + m, p0 = nv0 + s0;
    const int j0 = s0 == 0 ? nv0 / a.block : (p0 - 1) / a.block + 1, j1 = (p0 + n - 1) / a.block;
    auto member = [&](int pos) -> const uint8_t* {         // its indexer key
      return pos < nv0 ? static_cast<const uint8_t*>(a.k_idx) + (row0 + pos) * x_bytes
                       : static_cast<const uint8_t*>(a.kidx_new) + ((long long)b * a.max_new + pos - nv0) * x_bytes;
    };
    // (sums in entry order, as block_key_elem's)
    if (a.wide_idx) {
      constexpr int kN = 16 / kE;
      const int vecs = a.idx_dim / kN;
      for (int i = tid; i < (j1 - j0 + 1) * vecs; i += kThreads) {
        const int j = j0 + i / vecs, v = i % vecs, first = j * a.block, count = min(a.block, nv1 - first);
        float sum[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) sum[e] = 0.f;
#pragma unroll 8
        for (int r = 0; r < count; ++r) {
          const uint4 y = reinterpret_cast<const uint4*>(member(first + r))[v];
          const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (kF32) {
              sum[e] += __uint_as_float(w[e]);
            } else {
              sum[2 * e] += __uint_as_float(w[e] << 16);
              sum[2 * e + 1] += __uint_as_float(w[e] & 0xffff0000u);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          sum[e] = sum[e] / float(count);
          if (a.round_to_int) sum[e] = rintf(sum[e]);
          store_elem(a.kb, ((long long)b * a.nb_cap + j) * a.idx_dim + v * kN + e, a.dtype, sum[e]);
        }
      }
    } else {
      for (int i = tid; i < (j1 - j0 + 1) * a.idx_dim; i += kThreads) {
        const int j = j0 + i / a.idx_dim, d = i % a.idx_dim, first = j * a.block, count = min(a.block, nv1 - first);
        float sum = 0.f;
        for (int r = 0; r < count; ++r) sum += load_elem(member(first + r), d, a.dtype);
        sum = sum / float(count);
        if (a.round_to_int) sum = rintf(sum);
        store_elem(a.kb, ((long long)b * a.nb_cap + j) * a.idx_dim + d, a.dtype, sum);
      }
    }
  }
}

// The fill counts of sequences that several CTAs have read them for.
__global__ void __launch_bounds__(kThreads) kv4_count_kernel(const Kv4AppendArgs a, int batch) {
  const int b = blockIdx.x * kThreads + threadIdx.x;
  pdl_wait();
  if (b >= batch) return;
  const int nv0 = clamp_count(a.n_valid[b], a.n_entries, nullptr);
  a.n_valid[b] = nv0 + min(clamp_count(a.n_new[b], a.max_new, nullptr), a.n_entries - nv0);
}

// ------------------------------------------------------------------ rows

constexpr int kBatch = 5;          // 16-byte pieces of rows a thread has on their way: 32 rows of 192 / 128 dims at once
constexpr int kMaxRows = 32;       // of a CTA

// The entries of a CTA's rows, null where there is none, into shared memory.
CSA2_DEV void row_entries(const Kv4RowsArgs& a, int row0, int n, int bytes, const uint8_t** src) {
  pdl_wait();
  if (int(threadIdx.x) < n) {
    const int row = row0 + threadIdx.x, e = a.idx[row];
    if (e >= a.n_entries) report(a.err, kErrBadIndex, e);
    src[threadIdx.x] = e < 0 || e >= a.n_entries ? nullptr : a.kv + ((long long)(row / a.rows / a.seq_div) * a.n_entries + e) * bytes;
  }
  __syncthreads();
}

// A thread writes 16 bytes of a row at a time (8 bf16 or 4 fp32 numbers: half or a quarter of a group).
// Measured: 32,768 rows of 192 / 128 dims in bf16 8.0 us, 131,072 20.8 us, 5.3 TB/s (issue slots
// 72 %), in fp32 11.8 and 32.6 us, 5.9 TB/s.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) kv4_rows_kernel(const Kv4RowsArgs a, int n_rows, int per_cta) {
  __shared__ const uint8_t* src[kMaxRows];
  constexpr int kN = kF32 ? 4 : 8;                         // numbers of a piece
  const int gk = kv4_groups(a.k_dim), groups = gk + kv4_groups(a.v_dim);
  const int pk = a.k_dim / kN, pv = a.v_dim / kN, pieces = pk + pv;
  const uint32_t m_pieces = 0xffffffffu / uint32_t(pieces) + 1u;
  const int row0 = blockIdx.x * per_cta, n = min(per_cta, n_rows - row0), total = n * pieces;
  row_entries(a, row0, n, kv4_bytes(a.k_dim, a.v_dim), src);
  for (int i0 = threadIdx.x; i0 < total; i0 += kBatch * kThreads) {
    uint32_t codes[kBatch];
    uint8_t scale[kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int i = i0 + x * kThreads, r = int(__umulhi(uint32_t(i), m_pieces)), p = i - r * pieces;
      codes[x] = 0;
      scale[x] = 0;
      const uint8_t* entry = i < total ? src[r] : nullptr;
      if (entry == nullptr) continue;
      const int c = p < pk ? p * kN : gk * 16 + (p - pk) * kN;   // the piece's first code
      codes[x] = kF32 ? *reinterpret_cast<const uint16_t*>(entry + c / 2) : *reinterpret_cast<const uint32_t*>(entry + c / 2);
      scale[x] = entry[8 * groups + c / 16];
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int i = i0 + x * kThreads, r = int(__umulhi(uint32_t(i), m_pieces)), p = i - r * pieces;
      if (i >= total) break;
      const bool key = p < pk;
      const float up = key ? a.k_up : a.v_up;
      float v[8];
      kv4_eight(codes[x], __half2half2(kv4_scale(scale[x])), v);
      uint4 w;
      if (kF32)
        w = make_uint4(__float_as_uint(v[0] * up), __float_as_uint(v[1] * up), __float_as_uint(v[2] * up), __float_as_uint(v[3] * up));
      else
        w = make_uint4(pack_bf16(v[0] * up, v[1] * up), pack_bf16(v[2] * up, v[3] * up), pack_bf16(v[4] * up, v[5] * up),
                       pack_bf16(v[6] * up, v[7] * up));
      static_cast<uint4*>(key ? a.k_out : a.v_out)[(long long)(row0 + r) * (key ? pk : pv) + (key ? p : p - pk)] = w;
    }
  }
}

// Any dims and alignment: a number at a time.
__global__ void __launch_bounds__(kThreads) kv4_rows_any_kernel(const Kv4RowsArgs a, int n_rows, int per_cta) {
  __shared__ const uint8_t* src[kMaxRows];
  const int gk = kv4_groups(a.k_dim), groups = gk + kv4_groups(a.v_dim), dims = a.k_dim + a.v_dim;
  const int row0 = blockIdx.x * per_cta, n = min(per_cta, n_rows - row0);
  row_entries(a, row0, n, kv4_bytes(a.k_dim, a.v_dim), src);
  for (int i = threadIdx.x; i < n * dims; i += kThreads) {
    const int r = i / dims, d = i - r * dims;
    const bool key = d < a.k_dim;
    float v = 0.f;
    if (src[r] != nullptr) {
      const int c = key ? d : gk * 16 + d - a.k_dim;
      const __half2 pair = __hmul2(kv4_pair(src[r][c / 2]), __half2half2(kv4_scale(src[r][8 * groups + c / 16])));
      v = (c & 1 ? __high2float(pair) : __low2float(pair)) * (key ? a.k_up : a.v_up);
    }
    const long long row = row0 + r;
    if (key) store_elem(a.k_out, row * a.k_dim + d, a.dtype, v);
    else store_elem(a.v_out, row * a.v_dim + d - a.k_dim, a.dtype, v);
  }
}

}  // namespace

cudaError_t launch_kv4_append(Kv4AppendArgs& a, int batch, cudaStream_t st) {
  if (batch == 0 || a.max_new == 0) return cudaSuccess;
  const int bytes = kv4_bytes(a.k_dim, a.v_dim);
  a.per_cta = kTileEntries * bytes <= 48 << 10 ? kTileEntries : kTileEntries / 2;
  const unsigned chunks = unsigned((a.max_new - 1) / a.per_cta + 1);
  note_launch();
  const size_t smem = size_t(a.per_cta) * bytes;
  cudaError_t e = launch_pdl(a.dtype == 1 ? kv4_append_kernel<true> : kv4_append_kernel<false>, dim3(chunks, unsigned(batch)), dim3(kThreads),
                             smem, st, 1, a);
  if (e != cudaSuccess || chunks == 1) return e;
  note_launch();
  return launch_pdl(kv4_count_kernel, dim3(unsigned((batch + kThreads - 1) / kThreads)), dim3(kThreads), 0, st, 1, a, batch);
}

cudaError_t launch_kv4_rows(const Kv4RowsArgs& a, int batch, cudaStream_t st) {
  const int n = batch * a.rows;
  if (n == 0) return cudaSuccess;
  int per_cta = kMaxRows;   // fewer rows a CTA where there are few
  while (per_cta > 1 && n / per_cta < 2 * device_sm_count()) per_cta /= 2;
  const dim3 grid(unsigned((n - 1) / per_cta + 1));
  note_launch();
  if (!a.wide) return launch_pdl(kv4_rows_any_kernel, grid, dim3(kThreads), 0, st, 1, a, n, per_cta);
  return launch_pdl(a.dtype == 1 ? kv4_rows_kernel<true> : kv4_rows_kernel<false>, grid, dim3(kThreads), 0, st, 1, a, n, per_cta);
}

}  // namespace csa2
