// Commit of an accepted path (csa2_tree_commit): the accepted drafted tokens'
// K and V rows into every layer's window ring, and the accepted queries'
// attention weights into the per-entry mass.
//
// A sequence's first CTAs, a cluster, copy its window rows, shared out by
// layer; all of them read the shared head and fill count, meet at a cluster
// barrier, and the first then advances both.  Its other CTAs add up weights: a
// thread takes one selected slot of an accepted token through 8 layers and adds
// up neighbouring layers that selected the same entry (Reuse layers attend with
// their indexing layer's list) before one atomic.  They need only the path,
// which nobody writes, so no barrier holds them, and a sequence with a long
// path has as many of them at work as it needs (paths differ: the weights in
// the clusters, 8 CTAs of 512 threads a sequence, took 18.2 us for 64 sequences of 16
// tokens and 20 layers where these took 11.5, both with atomics that return nothing).
// That case takes 14.5 us, one sequence of 8 tokens and 4 layers 2.8.  Bound by the
// latency of path, idx and weight behind each other, by the reads of 24 MB of idx and
// weights (with the windows 5.2 us at HBM's rate) and by the atomics' old values, which
// come back for the check of the range: 3.0 and 0.4 us of the two.  (Loads of the masses
// behind or in front of atomics that return nothing cost 2 us more than that.)
// The mass is a 64-bit integer in units of 2^-32: integer sums depend on no
// order, so neither the atomics nor the merging change them, and they stay
// exact where fp32 sums would stop growing; they end at 2^63 - 1.  A weight is split into its whole
// part and the rest, which is exact, and the rest rounded once.
//
// Like the cache-maintenance kernels it lets no later launch start early: the
// attention reads n_swa and the windows before its own wait.
#include "common.cuh"
#include "draft.h"

namespace csa2 {

namespace {

constexpr int kThreads = 128;              // (256: 13.2 us, 64: 15.3, where 128 took 11.5)
static_assert(kThreads >= kMaxTreeTokens, "a thread for every token of a path");
constexpr int kCopies = 4;                // row units a thread has in flight
constexpr int kBatch = 8;                 // layers of an item of the mass, their idx and weights in flight together
constexpr float kMaxWeight = 1048576.f;   // 2^20
constexpr long long kMostMass = 0x7fffffffffffffffll;
constexpr int kMassCtas = 16;             // CTAs of the mass for every SM at most (24 took 11.9 us, 8 to 16 11.5)

// The path's rows [j0, n) into the rings of layers rank, rank + ncta, ...: all
// the units of all these rows are one list, so that a thread waits for its
// loads once or twice, not layer by layer.
template <typename U>
CSA2_DEV void copy_rows(const TreeCommitArgs& a, int rank, int ncta, long long ring0, long long draft0, int j0, int n, int slot,
                        const int* path) {
  const int ku = a.k_bytes / int(sizeof(U)), per_row = ku + a.v_bytes / int(sizeof(U)), per_layer = (n - j0) * per_row;
  const int total = (a.n_layers - rank + ncta - 1) / ncta * per_layer;
  for (int i0 = threadIdx.x; i0 < total; i0 += kCopies * kThreads) {
    U w[kCopies];
    U* to[kCopies];
#pragma unroll
    for (int m = 0; m < kCopies; ++m) {
      const int i = i0 + m * kThreads;
      if (i >= total) break;
      const int l = i / per_layer, x = i - l * per_layer, j = j0 + x / per_row;
      int u = x % per_row;
      const TreeCommitArgs::Slot& y = a.slot[rank + l * ncta];
      const bool k = u < ku;
      if (!k) u -= ku;
      const int per = k ? ku : per_row - ku;
      to[m] = static_cast<U*>(k ? y.k_swa : y.v_swa) + (ring0 + (slot + j) % a.swa) * per + u;
      w[m] = static_cast<const U*>(k ? y.k_draft : y.v_draft)[(draft0 + path[j]) * per + u];
    }
#pragma unroll
    for (int m = 0; m < kCopies; ++m)
      if (i0 + m * kThreads < total) *to[m] = w[m];
  }
}

// mass += sum, up to 2^63 - 1 and no further.  Sums here are not negative, so a
// sum that leaves the range passes 2^63 in exactly one addition, whose own old value shows
// it; that thread puts the maximum in its place, and so does any that passes it
// again behind that.  What is left is min(true sum, 2^63 - 1), whatever the order.
CSA2_DEV void add_mass(unsigned long long* mass, unsigned long long sum) {
  const unsigned long long old = atomicAdd(mass, sum);
  if (static_cast<long long>(old) >= 0 && static_cast<long long>(old + sum) < 0)
    atomicMax(reinterpret_cast<long long*>(mass), kMostMass);
}

// The accepted path of a sequence into `path` (shared memory); its length, a bad id ending it.
CSA2_DEV int load_path(const TreeCommitArgs& a, int seq, int* path, int* end, bool reports) {
  const int tid = threadIdx.x;
  if (tid == 0) *end = a.tokens;
  const int n = clamp_count(a.n_path[seq], a.tokens, reports && tid == 0 ? a.err : nullptr);
  __syncthreads();
  if (tid < n) {
    const int t = a.path[(long long)seq * a.tokens + tid];
    path[tid] = t;
    if (t < 0 || t >= a.tokens) {
      if (reports) report(a.err, kErrBadIndex, t);
      atomicMin(end, tid);
    }
  }
  __syncthreads();
  return min(n, *end);
}

// grid.x: the copying cluster of a sequence, then the CTAs of its mass (whole clusters).
__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const __grid_constant__ TreeCommitArgs a) {
  __shared__ int path[kMaxTreeTokens];
  __shared__ int end_s;
  const int seq = blockIdx.y, tid = threadIdx.x;
  const int ncta = int(cluster_size());
  pdl_wait();
  const long long draft0 = (long long)seq * a.tokens;
  if (int(blockIdx.x) < ncta) {
    const int rank = int(cluster_rank());
    int* err = rank == 0 ? a.err : nullptr;
    int slot = a.head[seq];
    if (slot < 0 || slot >= a.swa) {
      if (tid == 0) report(err, kErrBadCount, slot);
      slot = slot < 0 ? 0 : a.swa - 1;
    }
    const int fill = clamp_count(a.n_swa[seq], a.swa, tid == 0 ? err : nullptr);
    const int n = load_path(a, seq, path, &end_s, rank == 0);
    cluster_arrive();                        // this CTA has read the head and the fill count
    const int j0 = max(0, n - a.swa);        // rows that a longer path would push out again are not written
    const long long ring0 = (long long)seq * a.swa;
    if (a.wide) copy_rows<uint4>(a, rank, ncta, ring0, draft0, j0, n, slot, path);
    else copy_rows<uint16_t>(a, rank, ncta, ring0, draft0, j0, n, slot, path);
    cluster_wait();
    if (rank == 0 && tid == 0) {
      a.head[seq] = (slot + n) % a.swa;
      a.n_swa[seq] = min(fill + n, a.swa);
    }
    return;
  }
  // an item: a selected slot of an accepted token in kBatch layers
  const int n = load_path(a, seq, path, &end_s, false);
  const int chunks = (a.n_layers + kBatch - 1) / kBatch, items = n * chunks * a.topk;
  unsigned long long* mass = a.mass + (long long)seq * a.n_entries;
  for (int i = (int(blockIdx.x) - ncta) * kThreads + tid; i < items; i += (int(gridDim.x) - ncta) * kThreads) {
    const int row = i / a.topk, j = row / chunks, l0 = (row - j * chunks) * kBatch;
    const long long at = (draft0 + path[j]) * a.topk + (i - row * a.topk);
    int e[kBatch];
    float w[kBatch];
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      const bool on = l0 + m < a.n_layers && a.slot[l0 + m].weights != nullptr;
      e[m] = on ? a.slot[l0 + m].idx[at] : -1;
      w[m] = on ? a.slot[l0 + m].weights[at] : 0.f;
    }
    int cur = -1, bad = 0, detail = 0;       // the entry that `sum` is for
    unsigned long long sum = 0;
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      if (e[m] < 0) continue;
      if (e[m] >= a.n_entries || !(w[m] >= 0.f && w[m] <= kMaxWeight)) {
        bad |= e[m] >= a.n_entries ? kErrBadIndex : kErrBadWeight;
        detail = e[m];
        continue;
      }
      if (e[m] != cur) {
        if (sum != 0) add_mass(mass + cur, sum);
        cur = e[m];
        sum = 0;
      }
      const uint32_t whole = __float2uint_rd(w[m]);
      sum += ((unsigned long long)whole << 32) + __float2uint_rn((w[m] - float(whole)) * 4294967296.f);
    }
    if (sum != 0) add_mass(mass + cur, sum);
    if (bad != 0) report(a.err, bad, detail);
  }
}

}  // namespace

cudaError_t launch_tree_commit(const TreeCommitArgs& a, int seqs, cudaStream_t st) {
  if (seqs == 0) return cudaSuccess;
  const int c = a.n_layers < 8 ? a.n_layers : 8;   // a portable cluster
  // CTAs of the mass: a thread an item for paths of all T tokens, in whole
  // clusters; no more than kMassCtas an SM over all sequences (each then takes several
  // items), as most of them find nothing to do, but a cluster at least.
  int more = 0;
  if (a.mass != nullptr) {
    const long long items = (long long)a.tokens * ((a.n_layers + kBatch - 1) / kBatch) * a.topk;
    const long long want = (items + kThreads - 1) / kThreads, most = (long long)kMassCtas * device_sm_count() / seqs;
    more = int(((want < most ? want : most) + c - 1) / c) * c;
    if (more < c) more = c;
  }
  note_launch();
  return launch_pdl(tree_commit_kernel, dim3(unsigned(c + more), unsigned(seqs)), dim3(kThreads), 0, st, unsigned(c), a);
}

}  // namespace csa2
