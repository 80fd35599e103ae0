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
// call); `jump` [kMaxTreeTokens] is scratch.  Lane l finds the ancestors at
// distances l, l + 32, ..., by the bits of the distance: after k rounds `jump`
// leads 2^k tokens up, so that a path of any length takes log2 rounds (a walk
// from parent to parent was 60 ns a token).  A parent that is not an earlier
// token ends the path.  Returns the number of slots (at most W) and, in `depth`,
// the whole path's length.
CSA2_DEV int tree_walk(const TreeArgs& a, int seq, int token, int* path, int* jump, int& depth, bool reports) {
  constexpr int kEach = kMaxTreeTokens / 32;
  const int lane = threadIdx.x & 31;
  int cur[kEach];                              // at distance 32 j + lane; -1: there is none
  unsigned bad = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int t = 32 * j + lane;
    cur[j] = -1;
    if (t > token) continue;                   // (distances are at most `token`, too)
    cur[j] = token;
    int p = a.parent[(long long)seq * a.tokens + t];
    if (p >= t || p < -1) {
      bad |= 1u << j;
      p = -1;
    }
    jump[t] = p;
  }
  __syncwarp();
  for (int k = 0; (1 << k) <= token; ++k) {
    int up[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int t = 32 * j + lane;
      if (t > token) continue;
      if (((t >> k) & 1) != 0 && cur[j] >= 0) cur[j] = jump[cur[j]];
      const int p = jump[t];
      up[j] = p >= 0 ? jump[p] : -1;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (32 * j + lane <= token) jump[32 * j + lane] = up[j];
    __syncwarp();
  }
  depth = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int t = 32 * j + lane;
    if (cur[j] >= 0 && t < a.swa) path[t] = cur[j];
    depth += __popc(__ballot_sync(0xffffffffu, cur[j] >= 0));
  }
  if (__any_sync(0xffffffffu, bad != 0) && __any_sync(0xffffffffu, reports)) {   // only the path's last token may be one that was cut off
    int last = -1;
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (32 * j + lane == depth - 1) last = cur[j];
    if (last >= 0) {
      const int p = a.parent[(long long)seq * a.tokens + last];
      if (p >= last || p < -1) report(a.err, kErrBadIndex, p);
    }
  }
  return min(depth, a.swa);
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
  __shared__ int depth_s, jump_s[kMaxTreeTokens];
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
      tree_walk(a, seq, w.token, path, jump_s, depth, reports && w.live);
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
