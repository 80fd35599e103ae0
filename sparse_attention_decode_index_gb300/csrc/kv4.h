// Internal interface of the 4-bit main cache (norm_rope.cu, kv4_cache.cu,
// kv4_attn.cu), beside internal.h and draft.h.
#pragma once
#include "draft.h"

namespace csa2 {

// Keys of once_per_device, behind DraftSetupKey's.
enum Kv4SetupKey { kSetupKv4Tc = 32, kSetupKv4One, kSetupKv4Four, kSetupKv4Full, kSetupKv4Mma8, kSetupKv4Mma16 };

// Norm of heads with rotary positions (norm_rope.cu).
struct NormRopeArgs {
  struct Slot {
    const void* x;           // rows of [heads, dim], x_stride elements apart
    void* out;               // the same, out_stride apart; x with x's stride: in place
    const float* gain;       // [dim], or [heads, dim] (nullable: ones)
    long long x_stride, out_stride;
    int heads, dim, off, dtype, gain_each;
    int bytes, lanes, vecs, partner;   // vectors' bytes (0: element by element), lanes of a head, vectors a lane, where partners are (set by the launcher)
  } slot[kMaxRopeSlots];
  int n_slots;
  int rows, per_block;       // rows, rows per block (set by the launcher)
  int rot, interleaved, center;
  float mag, eps;
  const int* pos;            // [rows]
  const double* freqs;       // [rot / 2] radians per position
};

cudaError_t launch_norm_rope(const NormRopeArgs& a, int rows, cudaStream_t st);

// A packed entry: the codes of the key's groups and of the value's, 8 bytes a
// group, then a scale's byte a group, padded with zeros to 16 bytes.
constexpr int kKv4Group = 16;
constexpr int kv4_groups(int dim) { return (dim + kKv4Group - 1) / kKv4Group; }
constexpr int kv4_bytes(int k_dim, int v_dim) { return (9 * (kv4_groups(k_dim) + kv4_groups(v_dim)) + 15) / 16 * 16; }

struct Kv4AppendArgs {
  const int* n_new;          // [B]
  int max_new;
  const void* k_new;         // [B, max_new, k_dim]
  const void* v_new;         // [B, max_new, v_dim]
  const void* kidx_new;      // [B, max_new, idx_dim]
  uint8_t* kv;               // [B, N, kv4_bytes]
  void* k_idx;               // [B, N, idx_dim]
  void* kb;                  // [B, nb_cap, idx_dim] (nullable)
  int* n_valid;              // [B] (read and updated)
  int n_entries, nb_cap, k_dim, v_dim, idx_dim, block, round_to_int, dtype;
  float k_down, v_down;      // 2^-k_exp, 2^-v_exp
  int per_cta;               // entries a CTA packs (set by the launcher)
  int wide, wide_idx;        // whole 16-byte pieces at aligned addresses: of keys and values, of indexer keys
  int* err;
};

cudaError_t launch_kv4_append(Kv4AppendArgs& a, int batch, cudaStream_t st);

struct Kv4RowsArgs {
  const uint8_t* kv;         // [B / seq_div, N, kv4_bytes]
  const int* idx;            // [B, rows]
  void* k_out;               // [B, rows, k_dim]
  void* v_out;               // [B, rows, v_dim]
  int seq_div, n_entries, rows, k_dim, v_dim, dtype;
  float k_up, v_up;          // 2^k_exp, 2^v_exp
  int wide;                  // rows are whole 16-byte pieces at aligned addresses
  int* err;
};

cudaError_t launch_kv4_rows(const Kv4RowsArgs& a, int batch, cudaStream_t st);

struct Kv4AttnArgs {
  const void* q;             // [B, H, dk]
  const uint8_t* kv;         // [B / seq_div, N, kv4_bytes]
  const int* idx;            // [B, topk]
  const void* k_swa;         // [B, W, dk]
  const void* v_swa;         // [B, W, dv]
  const int* n_swa;          // [B]
  void* out;                 // [B, H, dv] element type
  float* lse;                // [B, H] (nullable)
  int seq_div, n_entries, topk, swa, heads, k_dim, v_dim, dtype;
  float scale;               // softmax scale (natural-log domain)
  float k_up, v_up;          // 2^k_exp, 2^v_exp
  int wide;                  // fp32 window rows of 16 dims at 16-byte addresses (kv4_attn.cu)
  long long wait_cycles;     // limit of a wait (kv4_tc.cu)
  int never;                 // 1: the first stage never fills (csa2_debug_kv4_wait_timeout; kv4_tc.cu)
  int* err;
};

constexpr long long kKv4WaitCycles = 4000000000ll;   // 2 s at the highest clock

// kv4_tc.cu: bf16, 64 heads, dk 192, dv 128, arrays at 16-byte addresses (`fast` of launch_kv4_attn).
cudaError_t launch_kv4_attn_tc(const Kv4AttnArgs& a, int batch, cudaStream_t st);
// kv4_mma.cu: other bf16 shapes.
bool kv4_mma_fits(const Kv4AttnArgs& a);
cudaError_t launch_kv4_attn_mma(const Kv4AttnArgs& a, int batch, cudaStream_t st);
cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, bool fast, int batch, cudaStream_t st);

}  // namespace csa2
