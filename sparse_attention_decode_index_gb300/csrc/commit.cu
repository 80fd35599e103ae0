// Commit of an accepted path (csa2_tree_commit): the accepted drafted tokens'
// K and V rows into every layer's window ring, and the accepted queries'
// attention weights into the per-entry mass.
//
// One cluster of CTAs per sequence.  All of them read the shared head and fill
// count, meet at a cluster barrier, and the first then advances both.  The
// window rows are shared out by layer, the weights by (token, slot): a thread
// takes one selected slot through all the layers and adds up neighbouring layers that
// selected the same entry (Reuse layers attend with their indexing layer's
// list) before one atomic.  The mass is a 64-bit integer in units of 2^-32:
// integer sums depend on no order, so neither the atomics nor the merging
// change them, and they stay exact where fp32 sums would stop growing.  The
// scaling by 2^32 is exact in fp32 and the conversion rounds once.
// Bound by the latency of the loads behind each other (count, path, rows or
// idx, weights, atomics): one sequence of 8 tokens and 4 layers 6.5 us, 64 sequences
// of 16 tokens and 20 layers 18 to 22 us, where the bytes need 5.2.  Leaving out the atomics
// or the copies changed neither by more than 2 us; adding up neighbours first
// took the latter from 44 us.
//
// Like the cache-maintenance kernels it lets no later launch start early: the
// attention reads n_swa and the windows before its own wait.
#include "common.cuh"
#include "draft.h"

namespace csa2 {

namespace {

constexpr int kThreads = 512;
constexpr int kCopies = 2;                // row units a thread has in flight
constexpr int kBatch = 8;                 // layers whose idx and weights a thread has in flight
constexpr float kMaxWeight = 1048576.f;   // 2^20: w * 2^32 stays below 2^53

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

__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const __grid_constant__ TreeCommitArgs a) {
  __shared__ int path[kMaxTreeTokens];
  __shared__ int end_s;
  const int seq = blockIdx.y, tid = threadIdx.x;
  const int rank = int(cluster_rank()), ncta = int(cluster_size());
  pdl_wait();
  int* err = rank == 0 ? a.err : nullptr;
  if (tid == 0) end_s = a.tokens;
  int n = clamp_count(a.n_path[seq], a.tokens, tid == 0 ? err : nullptr);
  int slot = a.head[seq];
  if (slot < 0 || slot >= a.swa) {
    if (tid == 0) report(err, kErrBadCount, slot);
    slot = slot < 0 ? 0 : a.swa - 1;
  }
  const int fill = clamp_count(a.n_swa[seq], a.swa, tid == 0 ? err : nullptr);
  __syncthreads();
  if (tid < n) {
    const int t = a.path[(long long)seq * a.tokens + tid];
    path[tid] = t;
    if (t < 0 || t >= a.tokens) {
      report(err, kErrBadIndex, t);
      atomicMin(&end_s, tid);
    }
  }
  __syncthreads();
  n = min(n, end_s);                         // a bad id ends the path before it
  cluster_arrive();                          // this CTA has read the head and the fill count
  const int j0 = max(0, n - a.swa);          // rows that a longer path would push out again are not written
  const long long draft0 = (long long)seq * a.tokens, ring0 = (long long)seq * a.swa;
  if (a.wide) copy_rows<uint4>(a, rank, ncta, ring0, draft0, j0, n, slot, path);
  else copy_rows<uint16_t>(a, rank, ncta, ring0, draft0, j0, n, slot, path);
  if (a.mass != nullptr) {
    unsigned long long* mass = a.mass + (long long)seq * a.n_entries;
    for (int i = rank * kThreads + tid; i < n * a.topk; i += ncta * kThreads) {
      const int j = i / a.topk;
      const long long at = (draft0 + path[j]) * a.topk + (i - j * a.topk);
      int cur = -1;                          // the entry that `sum` is for
      unsigned long long sum = 0;
      for (int l0 = 0; l0 < a.n_layers; l0 += kBatch) {
        int e[kBatch];
        float w[kBatch];
#pragma unroll
        for (int m = 0; m < kBatch; ++m) {
          const bool on = l0 + m < a.n_layers && a.slot[l0 + m].weights != nullptr;
          e[m] = on ? a.slot[l0 + m].idx[at] : -1;
          w[m] = on ? a.slot[l0 + m].weights[at] : 0.f;
        }
#pragma unroll
        for (int m = 0; m < kBatch; ++m) {
          if (e[m] < 0) continue;
          if (e[m] >= a.n_entries) {
            report(a.err, kErrBadIndex, e[m]);
            continue;
          }
          if (!(w[m] >= 0.f && w[m] <= kMaxWeight)) {
            report(a.err, kErrBadWeight, e[m]);
            continue;
          }
          if (e[m] != cur) {
            if (sum != 0) atomicAdd(mass + cur, sum);
            cur = e[m];
            sum = 0;
          }
          sum += (unsigned long long)__float2ll_rn(w[m] * 4294967296.f);
        }
      }
      if (sum != 0) atomicAdd(mass + cur, sum);
    }
  }
  cluster_wait();
  if (rank == 0 && tid == 0) {
    a.head[seq] = (slot + n) % a.swa;
    a.n_swa[seq] = min(fill + n, a.swa);
  }
}

}  // namespace

cudaError_t launch_tree_commit(const TreeCommitArgs& a, int seqs, cudaStream_t st) {
  if (seqs == 0) return cudaSuccess;
  const int c = a.n_layers < 8 && a.mass == nullptr ? a.n_layers : 8;   // a portable cluster
  note_launch();
  return launch_pdl(tree_commit_kernel, dim3(unsigned(c), unsigned(seqs)), dim3(kThreads), 0, st, unsigned(c), a);
}

}  // namespace csa2
