// Internal interface of the kernels around drafted tokens and bounded caches
// (rope.cu, the tree form of attn.cu, tree.cu, tree_tc.cu, weights_tc.cu,
// commit.cu, evict.cu), beside internal.h.
#pragma once
#include "../../include/csa2.h"
#include "internal.h"

namespace csa2 {

constexpr int kErrBadWeight = 16;   // error word: an attention weight outside [0, 2^20]

// Keys of once_per_device, behind SetupKey's.
enum DraftSetupKey { kSetupTree = 16, kSetupTreePair, kSetupWeightsTc, kSetupEvict, kSetupEvictMove,
                     kSetupTreeRows,        // and the next: warps
                     kSetupTreeGeneric = kSetupTreeRows + 2 };   // and the next five: element types and widths, warps

// Rotary positions (rope.cu).
constexpr int kMaxRopeSlots = 16;

struct RopeArgs {
  struct Slot {
    const void* x;           // [rows, heads, dim]
    void* out;               // [rows, heads, dim]; == x: in place
    int heads, dim, off, dtype;
    int wide, copy;          // whole vectors at aligned addresses; bytes of those that are copied (set by the launcher)
  } slot[kMaxRopeSlots];
  int n_slots;
  int rows, per_block;       // rows, rows per block (set by the launcher)
  int rot, interleaved, inverse;
  float mag;
  const int* pos;            // [rows]
  const double* freqs;       // [rot / 2] radians per position
};

cudaError_t launch_rope(RopeArgs& a, int rows, cudaStream_t st);

// Attention of drafted trees (tree.cu).
constexpr int kMaxTreeTokens = 128;

struct TreeArgs {
  const void* q;             // [B, H, dk]
  const void* k_main;        // [S, N, dk]
  const void* v_main;        // [S, N, dv]
  const int* idx;            // [B, topk]
  const void* k_swa;         // [S, W, dk]
  const void* v_swa;         // [S, W, dv]
  const int* swa_head;       // [S] (nullable)
  const int* n_swa;          // [S]
  const void* k_draft;       // [S, T, dk]
  const void* v_draft;       // [S, T, dv]
  const int* parent;         // [S, T] (nullable: a chain)
  const int* n_draft;        // [S] (nullable: all T)
  void* out;                 // [B, H, dv] element type
  float* lse;                // [B, H] (nullable)
  int tokens, n_entries, topk, swa, heads, k_dim, v_dim, dtype;
  float scale;
  int* err;
};

struct AttnWeightsArgs {
  const void* q;             // [B, H, dk]
  const void* k_main;        // [B / seq_div, N, dk]
  const int* idx;            // [B, topk]
  const float* lse;          // [B, H]
  const int* live;           // [B] (nullable)
  float* weights;            // [B, topk]
  int seq_div, n_entries, topk, heads, k_dim, dtype;
  float scale;
  int* err;
};

// fast: bf16, 64 heads, dk 192, dv 128
cudaError_t launch_tree_attn(const TreeArgs& a, bool fast, int batch, void* plan, size_t plan_bytes, cudaStream_t st);
cudaError_t launch_tree_attn_cluster(const TreeArgs& a, int batch, cudaStream_t st);   // attn.cu
// Tokens alone or in pairs on the tensor cores (tree_tc.cu); `plan` holds tree_plan_words.
cudaError_t launch_tree_attn_tc(const TreeArgs& a, int seqs, void* plan, cudaStream_t st);
size_t tree_plan_words(int seqs, int tokens, int topk, int swa);
size_t tree_plan_most(int seqs, int tokens, int topk, int swa);
// Bytes of workspace that all calls but csa2_tree_attn, which uses more where it gets it, need (0: a bad shape; api.cu).
size_t layer_workspace_bytes(const csa2_shape* shape);
// bf16 rows of whole 8-byte pieces, any heads and dims (tree_mma.cu).
bool tree_rows_fit(const TreeArgs& a);
bool weights_rows_fit(const AttnWeightsArgs& a);
cudaError_t launch_tree_rows(const TreeArgs& a, int batch, cudaStream_t st);
cudaError_t launch_weights_rows(const AttnWeightsArgs& a, int batch, cudaStream_t st);
cudaError_t launch_attn_weights_tc(const AttnWeightsArgs& a, int batch, cudaStream_t st);   // weights_tc.cu
cudaError_t launch_attn_weights(const AttnWeightsArgs& a, bool fast, int batch, cudaStream_t st);

// Commit of an accepted path (commit.cu).
constexpr int kMaxTreeLayers = 64;

struct TreeCommitArgs {
  struct Slot {
    const void* k_draft;     // [S, T, dk]
    const void* v_draft;     // [S, T, dv]
    void* k_swa;             // [S, W, dk]
    void* v_swa;             // [S, W, dv]
    const int* idx;          // [S * T, topk] (nullable)
    const float* weights;    // [S * T, topk] (nullable)
  } slot[kMaxTreeLayers];
  int n_layers;
  const int* path;           // [S, T]
  const int* n_path;         // [S]
  int* head;                 // [S] (read and updated)
  int* n_swa;                // [S] (read and updated)
  unsigned long long* mass;  // [S, N] (nullable)
  int tokens, n_entries, topk, swa;
  int k_bytes, v_bytes;      // bytes of a K / V row
  int wide;                  // rows are whole 16-byte pieces at 16-byte addresses
  int* err;
};

cudaError_t launch_tree_commit(const TreeCommitArgs& a, int seqs, cudaStream_t st);

// Eviction (evict.cu).
struct EvictArgs {
  const void* k_main;        // [S, N, dk]
  const void* v_main;        // [S, N, dv]
  const void* k_idx;         // [S, N, dI]
  const long long* mass;     // [S, N]
  const int* n_valid;        // [S]
  void* k_main_out;
  void* v_main_out;
  void* k_idx_out;
  long long* mass_out;
  int* n_valid_out;
  int* kept;                 // [S, N]
  void* kb;                  // [S, nb_cap, dI] (nullable)
  int trigger, keep, sink, recent;
  int n_entries, nb_cap, idx_dim, block, round_to_int, dtype;
  int k_bytes, v_bytes, x_bytes;   // bytes of a K / V / indexer-key row
  int wide;                  // rows are whole 16-byte pieces at 16-byte addresses
  int in_place;
  int* err;
};

cudaError_t launch_kv_evict(const EvictArgs& a, int seqs, cudaStream_t st);

}  // namespace csa2
