// The window of a drafted token: which rows stand for the W tokens that end at
// it along its path (device side, shared by the tree attention kernels).
#pragma once
#include "common.cuh"
#include "draft.h"

namespace csa2 {

// Slots 0 .. n_path - 1 are the token and its ancestors, nearest first; slots
// n_path .. n_path + n_ring - 1 the newest committed rows, newest first.
struct TreeWindow {
  const int* path;        // shared memory: drafted token of slot r (null: a chain, token - r)
  int token, n_path, n_ring, newest, swa;
  long long draft0, ring0;
  bool live;

  // Row of slot r in the draft rows or in the rings; false behind the window.
  CSA2_DEV bool row(int r, long long& at, bool& drafted) const {
    drafted = r < n_path;
    if (drafted) {
      at = draft0 + (path != nullptr ? path[r] : token - r);
      return true;
    }
    const int i = r - n_path;
    if (i >= n_ring) return false;
    int p = newest - i;
    if (p < 0) p += swa;
    at = ring0 + p;
    return true;
  }
};

// Path of query b into `path` [kMaxTreeTokens] by the calling warp (all lanes
// call).  The parents are held four to a lane, so that a step of the walk is
// a shuffle; a parent that is not an earlier token ends the path.  Returns
// the number of slots (at most W) and, in `depth`, the whole path's length.
CSA2_DEV int tree_walk(const TreeArgs& a, int seq, int token, int* path, int& depth, bool reports) {
  const int lane = threadIdx.x & 31;
  int p[kMaxTreeTokens / 32];
#pragma unroll
  for (int j = 0; j < kMaxTreeTokens / 32; ++j) {
    const int t = 32 * j + lane;
    p[j] = t < a.tokens && t <= token ? a.parent[(long long)seq * a.tokens + t] : -1;
  }
  int cur = token, n = 0;
  while (cur >= 0) {
    if (n < a.swa && lane == 0) path[n] = cur;
    ++n;
    const int v = cur < 32 ? p[0] : cur < 64 ? p[1] : cur < 96 ? p[2] : p[3];
    int up = __shfl_sync(0xffffffffu, v, cur & 31);
    if (up >= cur || up < -1) {
      if (lane == 0 && reports) report(a.err, kErrBadIndex, up);
      up = -1;
    }
    cur = up;
  }
  depth = n;
  return min(n, a.swa);
}

// The sequence's committed rows, all of them: a path of `depth` tokens leaves the newest swa - depth.
CSA2_DEV void tree_ring(const TreeArgs& a, int seq, TreeWindow& w, bool reports) {
  const int ns = clamp_count(a.n_swa[seq], a.swa, reports ? a.err : nullptr);
  int head = a.swa_head != nullptr ? a.swa_head[seq] : 0;
  if (ns == a.swa && (head < 0 || head >= a.swa)) {
    if (reports) report(a.err, kErrBadCount, head);
    head = head < 0 ? 0 : a.swa - 1;
  }
  w.swa = a.swa;
  w.newest = ns == a.swa ? (head == 0 ? a.swa - 1 : head - 1) : ns - 1;
  w.n_ring = ns;
  w.ring0 = (long long)seq * a.swa;
  w.draft0 = (long long)seq * a.tokens;
}

CSA2_DEV bool tree_live(const TreeArgs& a, int seq, int token, bool reports) {
  if (a.n_draft == nullptr) return true;
  return token < clamp_count(a.n_draft[seq], a.tokens, reports ? a.err : nullptr);
}

// The window of query b, by the whole block; `path` is shared memory.  The
// counts, the parents and whether the token is live are read together.
CSA2_DEV TreeWindow tree_window(const TreeArgs& a, int b, int* path, bool reports) {
  __shared__ int depth_s;
  TreeWindow w;
  const int seq = b / a.tokens;
  reports = reports && threadIdx.x == 0;
  w.token = b - seq * a.tokens;
  w.live = tree_live(a, seq, w.token, reports);
  tree_ring(a, seq, w, reports);
  int depth = w.token + 1;
  w.path = nullptr;
  if (a.parent != nullptr) {
    if (threadIdx.x < 32) {
      tree_walk(a, seq, w.token, path, depth, reports && w.live);
      if (threadIdx.x == 0) depth_s = depth;
    }
    __syncthreads();
    depth = depth_s;
    w.path = path;
  }
  w.n_path = w.live ? min(depth, a.swa) : 0;
  w.n_ring = w.live ? min(w.n_ring, max(0, a.swa - depth)) : 0;
  return w;
}

}  // namespace csa2
