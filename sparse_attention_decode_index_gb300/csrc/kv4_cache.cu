// The packed main cache: entries appended to it, and rows of it as numbers.
// The format stands in kv4.cuh.
#include "kv4.cuh"

namespace csa2 {

namespace {

constexpr int kThreads = 256;
constexpr int kTileEntries = 32;   // packed in shared memory before they are written as whole lines

// ------------------------------------------------------------------ append

// 16 numbers from p (n of them, zeros behind), in the element type.
CSA2_DEV void load16(const void* p, int n, int dtype, bool wide, float (&x)[16]) {
  if (wide && dtype == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = static_cast<const float4*>(p)[i];
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  } else if (wide) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = static_cast<const uint4*>(p)[i];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
        x[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i < n ? load_elem(p, i, dtype) : 0.f;
  }
}

// Each CTA owns `per_cta` positions of a sequence's cache, whole blocks of it, of which it writes those that the new
// entries take, so that every block's summary key is one CTA's.  A thread packs a group of 16 dims
// at a time into shared memory, from where a tile of entries, contiguous in the cache, goes out in 16-byte pieces.
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4AppendArgs a) {
  extern __shared__ __align__(16) uint8_t tile[];          // [kTileEntries][entry]
  const int b = blockIdx.y, tid = threadIdx.x;
  pdl_wait();   // no early trigger: the next launch may read what this one writes before its own wait
  int* err = blockIdx.x == 0 && tid == 0 ? a.err : nullptr;
  const int nv0 = clamp_count(a.n_valid[b], a.n_entries, err);
  int m = clamp_count(a.n_new[b], a.max_new, err);
  if (m > a.n_entries - nv0) {
    report(err, kErrBadCount, nv0 + m);
    m = a.n_entries - nv0;
  }
  const int gk = kv4_groups(a.k_dim), groups = gk + kv4_groups(a.v_dim), bytes = kv4_bytes(a.k_dim, a.v_dim);
  const int e_size = a.dtype == 1 ? 4 : 2, x_bytes = a.idx_dim * e_size;
  // positions [lo, hi) of this CTA
  const long long first = (long long)(nv0 / a.block) * a.block + (long long)blockIdx.x * a.per_cta;
  const int lo = int(min(max(first, (long long)nv0), (long long)nv0 + m)), hi = int(min(first + a.per_cta, (long long)nv0 + m));
  const uint8_t *k_new = static_cast<const uint8_t*>(a.k_new), *v_new = static_cast<const uint8_t*>(a.v_new);
  for (int p0 = lo; p0 < hi; p0 += kTileEntries) {
    const int n = min(kTileEntries, hi - p0);
    const long long src = (long long)b * a.max_new + (p0 - nv0);
    const uint32_t m_groups = groups == 1 ? 0u : 0xffffffffu / uint32_t(groups) + 1u;
    for (int i = tid; i < n * groups; i += kThreads) {
      const int r = m_groups == 0 ? i : int(__umulhi(uint32_t(i), m_groups)), g = i - r * groups;
      const bool key = g < gk;
      const int d = 16 * (key ? g : g - gk), dim = key ? a.k_dim : a.v_dim;
      float x[16];
      load16((key ? k_new : v_new) + ((src + r) * dim + d) * e_size, dim - d, a.dtype, a.wide != 0, x);
      uint2 codes;
      const float down = key ? a.k_down : a.v_down;
      const uint8_t s = a.dtype == 1 ? kv4_quantise<true>(x, down, codes) : kv4_quantise<false>(x, down, codes);
      *reinterpret_cast<uint2*>(tile + r * bytes + 8 * g) = codes;
      tile[r * bytes + 8 * groups + g] = s;
    }
    for (int i = tid; i < n * (bytes - 9 * groups); i += kThreads) {
      const int r = i / (bytes - 9 * groups);
      tile[r * bytes + 9 * groups + i - r * (bytes - 9 * groups)] = 0;
    }
    __syncthreads();
    uint4* dst = reinterpret_cast<uint4*>(a.kv + ((long long)b * a.n_entries + p0) * bytes);
    for (int i = tid; i < n * (bytes / 16); i += kThreads) dst[i] = reinterpret_cast<const uint4*>(tile)[i];
    const uint8_t* xs = static_cast<const uint8_t*>(a.kidx_new) + src * x_bytes;
    uint8_t* xd = static_cast<uint8_t*>(a.k_idx) + ((long long)b * a.n_entries + p0) * x_bytes;
    if (a.wide_idx) {
      for (int i = tid; i < n * (x_bytes / 16); i += kThreads) reinterpret_cast<uint4*>(xd)[i] = reinterpret_cast<const uint4*>(xs)[i];
    } else {
      for (int i = tid; i < n * (x_bytes / 2); i += kThreads) reinterpret_cast<uint16_t*>(xd)[i] = reinterpret_cast<const uint16_t*>(xs)[i];
    }
    __syncthreads();   // the tile is free again, and its indexer keys are visible to the CTA
  }
  if (a.kb != nullptr && lo < hi) {
    const int j0 = lo / a.block, n = ((hi - 1) / a.block - j0 + 1) * a.idx_dim;
    for (int i = tid; i < n; i += kThreads) {
      const int j = j0 + i / a.idx_dim, d = i % a.idx_dim;
      const float v = block_key_elem(a.k_idx, (long long)b * a.n_entries, a.idx_dim, a.block, nv0 + m, j, d, a.dtype, a.round_to_int);
      store_elem(a.kb, ((long long)b * a.nb_cap + j) * a.idx_dim + d, a.dtype, v);
    }
  }
  if (gridDim.x == 1) {
    __syncthreads();   // every thread read n_valid[b] before it changes
    if (tid == 0) a.n_valid[b] = nv0 + m;
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

constexpr int kBatch = 4;          // 16-byte pieces a thread has on their way
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
  // whole blocks of at least a tile of entries; the first new one may lie within its block
  a.per_cta = a.block >= kTileEntries ? a.block : (kTileEntries + a.block - 1) / a.block * a.block;
  const long long span = (a.max_new < a.n_entries ? a.max_new : a.n_entries) + (a.block - 1LL);
  const unsigned chunks = unsigned((span + a.per_cta - 1) / a.per_cta);
  note_launch();
  const size_t smem = size_t(kTileEntries) * kv4_bytes(a.k_dim, a.v_dim);
  cudaError_t e = launch_pdl(kv4_append_kernel, dim3(chunks, unsigned(batch)), dim3(kThreads), smem, st, 1, a);
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
