// Host side of the C ABI declared in include/csa2.h: argument validation,
// workspace carving, kernel selection and the layer-group sequencing.
//
// Layer-group sequencing follows the mode table of the DeepSeek V4.1 Flash
// architecture page ("CSA2 with cross-layer reuse"): Full and Reindex layers
// compute fresh Top-K indices over the group's shared indexer keys (Reindex
// with its own indexer query), Reuse layers attend with the latest indices,
// and every layer attends with its own query and SWA KV.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <functional>
#include <mutex>

#include "../../include/csa2.h"
#include "draft.h"
#include "kv4.h"

using namespace csa2;

namespace csa2 {
static std::atomic<unsigned long long> g_launches{0};
void note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

constexpr int kMaxSetupDevices = 64;
static std::atomic<uint64_t> g_setup_done[kMaxSetupDevices];
static std::mutex g_setup_mu;

cudaError_t once_per_device(int key, cudaError_t (*set)()) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxSetupDevices || key < 0 || key >= 64) return set();
  const uint64_t bit = uint64_t(1) << key;
  if (g_setup_done[dev].load(std::memory_order_acquire) & bit) return cudaSuccess;
  std::lock_guard<std::mutex> lock(g_setup_mu);
  if (g_setup_done[dev].load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = set();
  if (e == cudaSuccess) g_setup_done[dev].fetch_or(bit, std::memory_order_release);
  return e;
}
}  // namespace csa2

namespace {

constexpr size_t kAlign = 256;
constexpr size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct WsLayout {
  size_t hdr, pool, n_pool, n_blk, blk_scores, tok_scores, tok_cand, n_cand, tk_ids_a, tk_sc_a, tk_ids_b,
      tk_sc_b, idx, total;
  int64_t nb_cap, tok_ld, tk_chunks, tk_kmax;
};

bool hier_possible(const csa2_shape& s) { return s.pool_blocks > 0; }
bool attn_fast(const csa2_shape& s);

WsLayout layout(const csa2_shape& s) {
  WsLayout L{};
  const int64_t B = s.batch;
  L.nb_cap = ceil_div(s.n_entries, s.block);
  const int64_t P = hier_possible(s) ? s.pool_blocks : 0;
  L.tok_ld = s.n_entries > P * s.block ? s.n_entries : P * s.block;
  const int64_t longest = L.tok_ld > L.nb_cap ? L.tok_ld : L.nb_cap;
  const int64_t maxc = topk_max_chunk();
  L.tk_kmax = s.topk > P ? s.topk : P;
  L.tk_chunks = longest > maxc ? ceil_div(longest, maxc) : 0;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes);
    return at;
  };
  L.hdr = take(256);
  L.pool = take(size_t(B * P) * 4);
  L.n_pool = take(size_t(B) * 4);
  L.n_blk = take(size_t(B) * 4);
  L.blk_scores = take(size_t(B * L.nb_cap) * 4);
  L.tok_scores = take(size_t(B * L.tok_ld) * 4);
  L.tok_cand = take(size_t(B * L.tok_ld) * 4);
  L.n_cand = take(size_t(B) * 4);
  const size_t tk = size_t(B * L.tk_chunks * L.tk_kmax) * 4;
  L.tk_ids_a = take(tk);
  L.tk_sc_a = take(tk);
  L.tk_ids_b = take(tk);
  L.tk_sc_b = take(tk);
  L.idx = take(size_t(B) * s.topk * 4);
  L.total = off;
  return L;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

#define CSA2_TRY(x)                   \
  do {                                \
    const int _st = (x);              \
    if (_st != CSA2_OK) return _st;   \
  } while (0)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// Whether every pointer is a multiple of `bytes` (a power of two; null is).
template <class... P>
bool aligned(size_t bytes, P... p) {
  uintptr_t at = 0;
  for (const void* x : {static_cast<const void*>(p)...}) at |= reinterpret_cast<uintptr_t>(x);
  return (at & (bytes - 1)) == 0;
}

size_t elem_size(int dtype) { return dtype == CSA2_F32 ? 4 : 2; }

int check_shape(const csa2_shape* s) {
  if (s == nullptr) return CSA2_ERR_INVALID_ARG;
  if (s->batch < 1 || s->n_entries < 1 || s->idx_heads < 1 || s->idx_dim < 1 || s->block < 1 ||
      s->pool_blocks < 0 || s->topk < 1 || s->q_heads < 1 || s->k_dim < 1 || s->v_dim < 1 || s->swa < 0)
    return CSA2_ERR_INVALID_ARG;
  if (s->dtype != CSA2_BF16 && s->dtype != CSA2_F32) return CSA2_ERR_INVALID_ARG;
  if (s->relu != 0 && s->relu != 1) return CSA2_ERR_INVALID_ARG;
  if (s->tokens < 0 || (s->tokens > 1 && s->batch % s->tokens != 0)) return CSA2_ERR_INVALID_ARG;
  if (s->n_entries > (1 << 28) || s->batch > (1 << 20)) return CSA2_ERR_UNSUPPORTED;
  if (s->idx_heads > 64 || s->idx_dim > 1024 || s->idx_heads * s->idx_dim > 8192) return CSA2_ERR_UNSUPPORTED;
  if (s->topk > 1024 || s->swa > 1024 || s->topk + s->swa > 1024) return CSA2_ERR_UNSUPPORTED;
  if (s->q_heads > 1024 || s->k_dim > 1024 || s->v_dim > 1024) return CSA2_ERR_UNSUPPORTED;
  if (int64_t(s->pool_blocks) * s->block > (1 << 24)) return CSA2_ERR_UNSUPPORTED;
  if (s->pool_blocks > topk_max_chunk() / 2) return CSA2_ERR_UNSUPPORTED;
  return CSA2_OK;
}

// Queries per cache sequence (csa2_shape.tokens; 0 means 1).
int seqdiv(const csa2_shape& s) { return s.tokens > 1 ? s.tokens : 1; }

bool indexer_fast(const csa2_shape& s) { return s.dtype == CSA2_BF16 && s.idx_heads == 8 && s.idx_dim == 64; }
bool pooled_fast(const csa2_shape& s) { return indexer_fast(s) && s.block == 8; }
bool attn_fast(const csa2_shape& s) {
  return s.dtype == CSA2_BF16 && s.q_heads == 64 && s.k_dim == 192 && s.v_dim == 128 &&
         attn_cluster(s.topk, s.swa) > 0;
}

int check_ws(const csa2_shape& s, void* ws, size_t bytes) {
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return CSA2_ERR_WORKSPACE;
  if (bytes < layout(s).total) return CSA2_ERR_WORKSPACE;
  return CSA2_OK;
}

constexpr int kMaxRotDim = 1024;
constexpr int kMaxGridY = 65535;   // queries or sequences are a grid's y dimension

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// An array of a call; null or empty ones touch nothing.
struct Span {
  const void* at;
  uint64_t bytes;
  bool written;
};

// Whether an array that the call writes shares a byte with any other (sorts `v`).
bool written_overlap(Span* v, int n) {
  n = int(std::remove_if(v, v + n, [](const Span& x) { return x.at == nullptr || x.bytes == 0; }) - v);
  std::sort(v, v + n, [](const Span& x, const Span& y) { return std::less<const void*>()(x.at, y.at); });
  uint64_t end = 0, end_written = 0;       // of the arrays so far, of those that are written
  for (int i = 0; i < n; ++i) {
    const uint64_t at = reinterpret_cast<uintptr_t>(v[i].at);
    if (at < end_written || (v[i].written && at < end)) return true;
    end = std::max(end, at + v[i].bytes);
    if (v[i].written) end_written = std::max(end_written, at + v[i].bytes);
  }
  return false;
}

// Rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const void* at;
  uint64_t width, stride, rows;
};

// Whether two of them share a byte.  Rows of one stride may lie between each other (parts of one projection);
// of different strides, the whole ranges count.
bool overlap(const Rows& a, const Rows& b) {
  if (a.at == nullptr || b.at == nullptr) return false;
  if (!overlap(a.at, (a.rows - 1) * a.stride + a.width, b.at, (b.rows - 1) * b.stride + b.width)) return false;
  if (a.stride != b.stride || a.rows != b.rows || a.rows == 1) return true;
  const uint64_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  const uint64_t d = y >= x ? (y - x) % a.stride : (a.stride - (x - y) % a.stride) % a.stride;   // b behind a row of a
  return d < a.width || d + b.width > a.stride;
}

int check_exps(int32_t k_exp, int32_t v_exp) {
  return k_exp < -64 || k_exp > 64 || v_exp < -64 || v_exp > 64 ? CSA2_ERR_INVALID_ARG : CSA2_OK;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }

// Device error word of a cache-maintenance call: the header of the caller's
// workspace, or, when the caller passes no workspace (ws NULL, ws_bytes 0),
// the header of the library's static scratch array on the current device.
int error_word(const csa2_shape& s, void* ws, size_t ws_bytes, int** err) {
  if (ws == nullptr && ws_bytes == 0) {
    void* p = nullptr;
    CSA2_TRY(static_scratch(&p));
    *err = static_cast<int*>(p);
    return CSA2_OK;
  }
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  *err = static_cast<int*>(ws);
  return CSA2_OK;
}

float softmax_scale(const csa2_shape& s) { return s.scale > 0.f ? s.scale : 1.0f / sqrtf(float(s.k_dim)); }

// ---------------------------------------------------------------- internal ops (no validation)

int do_index_flat(const csa2_shape& s, const void* q_idx, const float* w, const void* keys, int64_t rows_per_seq, int seq_div,
                  const int32_t* n_valid, int div, float* scores, int32_t* cand, int32_t* n_cand, int64_t ld,
                  int* err, cudaStream_t st) {
  IndexerArgs a{};
  a.keys = keys;
  a.rows_per_seq = rows_per_seq;
  a.seq_div = seq_div;
  a.q_idx = q_idx;
  a.w = w;
  a.n_valid = n_valid;
  a.valid_cap = s.n_entries;
  a.div = div;
  a.block = s.block;
  a.scores = scores;
  a.cand = cand;
  a.n_cand = n_cand;
  a.ld = ld;
  a.relu = s.relu;
  a.heads = s.idx_heads;
  a.dim = s.idx_dim;
  a.dtype = s.dtype;
  a.err = err;
  const int max_rows = int(ceil_div(s.n_entries, div));
  return cuda_status(launch_indexer(a, false, indexer_fast(s), s.batch, max_rows, st));
}

int do_index_pooled(const csa2_shape& s, const void* q_idx, const float* w, const void* k_idx,
                    const int32_t* n_valid, const int32_t* pool, const int32_t* n_pool, float* scores,
                    int32_t* cand, int32_t* n_cand, int* err, cudaStream_t st) {
  IndexerArgs a{};
  a.keys = k_idx;
  a.rows_per_seq = s.n_entries;
  a.seq_div = seqdiv(s);
  a.q_idx = q_idx;
  a.w = w;
  a.n_valid = n_valid;
  a.valid_cap = s.n_entries;
  a.div = 1;
  a.pool = pool;
  a.n_pool = n_pool;
  a.pool_cap = s.pool_blocks;
  a.block = s.block;
  a.scores = scores;
  a.cand = cand;
  a.n_cand = n_cand;
  a.ld = int64_t(s.pool_blocks) * s.block;
  a.relu = s.relu;
  a.heads = s.idx_heads;
  a.dim = s.idx_dim;
  a.dtype = s.dtype;
  a.err = err;
  return cuda_status(launch_indexer(a, true, pooled_fast(s), s.batch, s.pool_blocks, st));
}

// Exact Top-k: rows longer than one cluster can hold are first cut into chunks
// of <= topk_max_chunk() positions whose Top-k lists are merged, then one
// cluster launch selects the final Top-k.
int do_topk(const csa2_shape& s, const WsLayout& L, void* ws, const float* scores, int64_t ld,
            const int32_t* cand, const int32_t* n_cand, int64_t n_cap, int k, int32_t* idx_out,
            float* score_out, int32_t* n_out, cudaStream_t st) {
  int* err = at<int>(ws, L.hdr);
  const int64_t maxc = topk_max_chunk();
  const int64_t maxcl = topk_cluster_max();
  TopkArgs a{};
  a.scores = scores;
  a.ld_in = ld;
  a.cand = cand;
  a.n_cand = n_cand;
  a.n_fixed = int(n_cap);
  a.n_cap = int(n_cap);
  a.k = k;
  a.err = err;
  int64_t n = n_cap;
  bool use_a = true;
  while (n > maxcl) {
    const int64_t chunks = ceil_div(n, maxc);
    a.chunk = int(ceil_div(n, chunks));
    a.idx_out = at<int32_t>(ws, use_a ? L.tk_ids_a : L.tk_ids_b);
    a.score_out = at<float>(ws, use_a ? L.tk_sc_a : L.tk_sc_b);
    a.n_out = nullptr;
    CSA2_TRY(cuda_status(launch_topk(a, int(chunks), s.batch, st)));
    // next level reads the concatenated chunk lists
    n = chunks * k;
    a.scores = a.score_out;
    a.cand = a.idx_out;
    a.ld_in = n;
    a.n_cand = nullptr;
    a.n_fixed = int(n);
    a.n_cap = int(n);
    use_a = !use_a;
  }
  a.n_cap = int(n > 0 ? n : 1);
  if (a.n_cand == nullptr) a.n_fixed = int(n);
  a.idx_out = idx_out;
  a.score_out = score_out;
  a.n_out = n_out;
  return cuda_status(launch_topk_cluster(a, s.batch, st));
}

int do_attn(const csa2_shape& s, const void* q, const void* k_main, const void* v_main, const int32_t* idx,
            const void* k_swa, const void* v_swa, const int32_t* n_swa, float* out, float* lse, int* err,
            cudaStream_t st, bool swa_only = false, bool release_at_end = false) {
  AttnArgs a{};
  a.release_at_end = release_at_end ? 1 : 0;
  a.q = q;
  a.k_main = k_main;
  a.v_main = v_main;
  a.seq_div = seqdiv(s);
  a.idx = idx;
  a.k_swa = k_swa;
  a.v_swa = v_swa;
  a.n_swa = n_swa;
  a.out = out;
  a.lse = lse;
  a.n_entries = s.n_entries;
  a.topk = swa_only ? 0 : s.topk;   // a pure SWA layer has no main-KV slots
  a.swa = s.swa;
  a.heads = s.q_heads;
  a.k_dim = s.k_dim;
  a.v_dim = s.v_dim;
  a.dtype = s.dtype;
  a.scale = softmax_scale(s);
  a.err = err;
  return cuda_status(launch_attn(a, attn_fast(s), s.batch, st));
}

SelectArgs select_args(const csa2_shape& s, const void* keys, int64_t rows_per_seq, int seq_div, const void* q_idx,
                       const float* w, const int32_t* n_valid, int div, int k, int32_t* out, int64_t ld_out,
                       int32_t* n_out, int* err) {
  SelectArgs a{};
  a.keys = keys;
  a.rows_per_seq = rows_per_seq;
  a.seq_div = seq_div;
  a.q_idx = q_idx;
  a.w = w;
  a.relu = s.relu;
  a.n_valid = n_valid;
  a.valid_cap = s.n_entries;
  a.div = div;
  a.k = k;
  a.out = out;
  a.ld_out = ld_out;
  a.n_out = n_out;
  a.err = err;
  return a;
}

int do_index_blocks(const csa2_shape& s, const WsLayout& L, void* ws, const void* q_idx, const float* w,
                    const void* kb, const int32_t* n_valid, int32_t* pool_out, int32_t* n_pool_out,
                    cudaStream_t st) {
  int* err = at<int>(ws, L.hdr);
  if (indexer_fast(s) && index_select_supported(false, int(L.nb_cap))) {
    // fused: block scoring and pool selection in one cluster launch
    SelectArgs a = select_args(s, kb, L.nb_cap, 1, q_idx, w, n_valid, s.block, s.pool_blocks, pool_out,
                               s.pool_blocks, n_pool_out, err);
    return cuda_status(launch_index_select(a, false, s.batch, int(L.nb_cap), st));
  }
  float* bs = at<float>(ws, L.blk_scores);
  int32_t* nblk = at<int32_t>(ws, L.n_blk);
  CSA2_TRY(do_index_flat(s, q_idx, w, kb, L.nb_cap, 1, n_valid, s.block, bs, nullptr, nblk, L.nb_cap, err, st));
  return do_topk(s, L, ws, bs, L.nb_cap, nullptr, nblk, L.nb_cap, s.pool_blocks, pool_out, nullptr, n_pool_out,
                 st);
}

int check_sswa(const csa2_shape& s, const void* k_swa, const void* v_swa, const int32_t* n_swa) {
  if (n_swa == nullptr) return CSA2_ERR_INVALID_ARG;
  if (s.swa > 0 && (k_swa == nullptr || v_swa == nullptr)) return CSA2_ERR_INVALID_ARG;
  if (attn_fast(s) && s.swa > 0 && (!aligned16(k_swa) || !aligned16(v_swa))) return CSA2_ERR_INVALID_ARG;
  return CSA2_OK;
}

int check_attn_args(const csa2_shape& s, const void* q, const void* k_main, const void* v_main, float* out) {
  if (q == nullptr || k_main == nullptr || v_main == nullptr || out == nullptr) return CSA2_ERR_INVALID_ARG;
  if (attn_fast(s) && (!aligned16(q) || !aligned16(k_main) || !aligned16(v_main))) return CSA2_ERR_INVALID_ARG;
  return CSA2_OK;
}

// The checks and the arguments of csa2_kv4_attn.
int kv4_attn_args(const csa2_shape* shape, const void* q, const void* kv4, const int32_t* idx, const void* k_swa, const void* v_swa,
                  const int32_t* n_swa, void* out, float* lse, int32_t k_exp, int32_t v_exp, void* ws, size_t ws_bytes, Kv4AttnArgs& a) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  if (s.batch > kMaxGridY) return CSA2_ERR_UNSUPPORTED;
  CSA2_TRY(check_exps(k_exp, v_exp));
  if (q == nullptr || kv4 == nullptr || idx == nullptr || out == nullptr) return CSA2_ERR_INVALID_ARG;
  CSA2_TRY(check_sswa(s, k_swa, v_swa, n_swa));
  const bool fast = attn_fast(s);
  if (!aligned16(kv4) || (fast && !(aligned16(q) && aligned16(k_swa) && aligned16(v_swa) && aligned16(out))))
    return CSA2_ERR_INVALID_ARG;
  if (!aligned(elem_size(s.dtype), q, k_swa, v_swa, out) || !aligned(4, idx, n_swa, lse)) return CSA2_ERR_INVALID_ARG;
  const uint64_t B = s.batch, kb = s.k_dim * elem_size(s.dtype), vb = s.v_dim * elem_size(s.dtype);
  Span spans[] = {{q, B * s.q_heads * kb, false}, {kv4, B / seqdiv(s) * s.n_entries * kv4_bytes(s.k_dim, s.v_dim), false},
                  {idx, B * s.topk * 4, false}, {k_swa, B * s.swa * kb, false}, {v_swa, B * s.swa * vb, false}, {n_swa, B * 4, false},
                  {out, B * s.q_heads * vb, true}, {lse, B * s.q_heads * 4, true}, {ws, ws_bytes, true}};
  if (written_overlap(spans, sizeof(spans) / sizeof(spans[0]))) return CSA2_ERR_INVALID_ARG;
  a.q = q;
  a.kv = static_cast<const uint8_t*>(kv4);
  a.idx = idx;
  a.k_swa = k_swa;
  a.v_swa = v_swa;
  a.n_swa = n_swa;
  a.out = out;
  a.lse = lse;
  a.seq_div = seqdiv(s);
  a.n_entries = s.n_entries;
  a.topk = s.topk;
  a.swa = s.swa;
  a.heads = s.q_heads;
  a.k_dim = s.k_dim;
  a.v_dim = s.v_dim;
  a.dtype = s.dtype;
  a.scale = softmax_scale(s);
  a.k_up = std::ldexp(1.f, k_exp);
  a.v_up = std::ldexp(1.f, v_exp);
  a.wide = s.dtype == CSA2_F32 && s.k_dim % 16 == 0 && s.v_dim % 16 == 0 && aligned16(k_swa) && aligned16(v_swa);
  a.wait_cycles = kKv4WaitCycles;
  a.err = static_cast<int*>(ws);
  return CSA2_OK;
}

}  // namespace

namespace csa2 {
size_t layer_workspace_bytes(const csa2_shape* shape) { return check_shape(shape) == CSA2_OK ? layout(*shape).total : 0; }
}  // namespace csa2

// ====================================================================== C ABI

extern "C" {

size_t csa2_workspace_bytes(const csa2_shape* shape) {
  if (check_shape(shape) != CSA2_OK) return 0;
  const csa2_shape& s = *shape;
  const WsLayout L = layout(s);
  if (!attn_fast(s) || s.swa < 1 || seqdiv(s) > kMaxTreeTokens) return L.total;
  // the key lists of csa2_tree_attn, where the caches are shorter than the lists
  const size_t plan = align_up(tree_plan_most(s.batch / seqdiv(s), seqdiv(s), s.topk, s.swa) * 4);
  return std::max(L.total, L.tok_scores + plan);
}

int csa2_workspace_init(void* ws, size_t ws_bytes, csa2_stream_t stream) {
  if (ws == nullptr || ws_bytes < 256 || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0)
    return CSA2_ERR_WORKSPACE;
  return cuda_status(cudaMemsetAsync(ws, 0, 256, stream));
}

int csa2_block_keys(const csa2_shape* shape, const void* k_idx, const int32_t* n_valid, int32_t round_to_int,
                    void* kb, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  if (k_idx == nullptr || n_valid == nullptr || kb == nullptr) return CSA2_ERR_INVALID_ARG;
  if (round_to_int != 0 && round_to_int != 1) return CSA2_ERR_INVALID_ARG;
  int* err = nullptr;
  CSA2_TRY(error_word(s, ws, ws_bytes, &err));
  const WsLayout L = layout(s);
  BlockKeyArgs a{};
  a.k_idx = k_idx;
  a.seq_div = seqdiv(s);
  a.n_valid = n_valid;
  a.kb = kb;
  a.n_entries = s.n_entries;
  a.nb_cap = int(L.nb_cap);
  a.dim = s.idx_dim;
  a.block = s.block;
  a.round_to_int = round_to_int;
  a.dtype = s.dtype;
  a.err = err;
  return cuda_status(launch_block_keys(a, s.batch, stream));
}

int csa2_kv_append(const csa2_shape* shape, int32_t max_new, const int32_t* n_new, const void* k_new,
                   const void* v_new, const void* kidx_new, void* k_main, void* v_main, void* k_idx, void* kb,
                   int32_t* n_valid, int32_t round_to_int, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  if (seqdiv(s) != 1) return CSA2_ERR_UNSUPPORTED;   // appends are per sequence: pass a one-token shape
  if (max_new < 0 || max_new > s.n_entries) return CSA2_ERR_INVALID_ARG;
  if (n_new == nullptr || n_valid == nullptr || k_main == nullptr || v_main == nullptr || k_idx == nullptr)
    return CSA2_ERR_INVALID_ARG;
  if (max_new > 0 && (k_new == nullptr || v_new == nullptr || kidx_new == nullptr)) return CSA2_ERR_INVALID_ARG;
  if (round_to_int != 0 && round_to_int != 1) return CSA2_ERR_INVALID_ARG;
  int* err = nullptr;
  CSA2_TRY(error_word(s, ws, ws_bytes, &err));
  const WsLayout L = layout(s);
  KvAppendArgs a{};
  a.n_new = n_new;
  a.max_new = max_new;
  a.k_new = k_new;
  a.v_new = v_new;
  a.kidx_new = kidx_new;
  a.k_main = k_main;
  a.v_main = v_main;
  a.k_idx = k_idx;
  a.kb = kb;
  a.n_valid = n_valid;
  a.n_entries = s.n_entries;
  a.nb_cap = int(L.nb_cap);
  a.k_dim = s.k_dim;
  a.v_dim = s.v_dim;
  a.idx_dim = s.idx_dim;
  a.block = s.block;
  a.round_to_int = round_to_int;
  a.dtype = s.dtype;
  a.err = err;
  return cuda_status(launch_kv_append(a, s.batch, stream));
}

int csa2_swa_append(const csa2_shape* shape, const csa2_swa_slot* layers, int32_t n_layers, int32_t* swa_head,
                    int32_t* n_swa, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  if (seqdiv(s) != 1) return CSA2_ERR_UNSUPPORTED;   // rings are per query: pass a one-token shape
  if (s.swa < 1 || layers == nullptr || n_layers < 1 || n_layers > kMaxSwaLayers) return CSA2_ERR_INVALID_ARG;
  if (swa_head == nullptr || n_swa == nullptr) return CSA2_ERR_INVALID_ARG;
  int* err = nullptr;
  CSA2_TRY(error_word(s, ws, ws_bytes, &err));
  SwaAppendArgs a{};
  for (int l = 0; l < n_layers; ++l) {
    const csa2_swa_slot& y = layers[l];
    if (y.k_tok == nullptr || y.v_tok == nullptr || y.k_swa == nullptr || y.v_swa == nullptr)
      return CSA2_ERR_INVALID_ARG;
    a.slot[l] = SwaAppendArgs::Slot{y.k_tok, y.v_tok, y.k_swa, y.v_swa};
  }
  a.n_layers = n_layers;
  a.head = swa_head;
  a.n_swa = n_swa;
  a.swa = s.swa;
  a.k_dim = s.k_dim;
  a.v_dim = s.v_dim;
  a.dtype = s.dtype;
  a.err = err;
  return cuda_status(launch_swa_append(a, s.batch, stream));
}

int csa2_index_blocks(const csa2_shape* shape, const void* q_idx, const float* w, const void* kb,
                      const int32_t* n_valid, int32_t* pool_out, int32_t* n_pool_out, void* ws, size_t ws_bytes,
                      csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  if (s.pool_blocks < 1) return CSA2_ERR_INVALID_ARG;
  if (q_idx == nullptr || w == nullptr || kb == nullptr || n_valid == nullptr || pool_out == nullptr ||
      n_pool_out == nullptr)
    return CSA2_ERR_INVALID_ARG;
  if (indexer_fast(s) && !aligned16(kb)) return CSA2_ERR_INVALID_ARG;
  const WsLayout L = layout(s);
  return do_index_blocks(s, L, ws, q_idx, w, kb, n_valid, pool_out, n_pool_out, stream);
}

int csa2_index_tokens(const csa2_shape* shape, const void* q_idx, const float* w, const void* k_idx,
                      const int32_t* n_valid, const int32_t* pool, const int32_t* n_pool, float* scores_out,
                      int32_t* cand_out, int32_t* n_cand_out, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  if (q_idx == nullptr || w == nullptr || k_idx == nullptr || n_valid == nullptr || scores_out == nullptr)
    return CSA2_ERR_INVALID_ARG;
  if (indexer_fast(s) && !aligned16(k_idx)) return CSA2_ERR_INVALID_ARG;
  const WsLayout L = layout(s);
  int* err = at<int>(ws, L.hdr);
  if (pool == nullptr)
    return do_index_flat(s, q_idx, w, k_idx, s.n_entries, seqdiv(s), n_valid, 1, scores_out, cand_out, n_cand_out,
                         s.n_entries, err, stream);
  if (s.pool_blocks < 1 || n_pool == nullptr || cand_out == nullptr || n_cand_out == nullptr)
    return CSA2_ERR_INVALID_ARG;
  if (s.n_entries % s.block != 0) return CSA2_ERR_INVALID_ARG;
  return do_index_pooled(s, q_idx, w, k_idx, n_valid, pool, n_pool, scores_out, cand_out, n_cand_out, err,
                         stream);
}

int csa2_index_topk(const csa2_shape* shape, const void* q_idx, const float* w, const void* k_idx,
                    const int32_t* n_valid, const int32_t* pool, const int32_t* n_pool, int32_t k, int32_t* idx_out,
                    int32_t* n_out, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  if (q_idx == nullptr || w == nullptr || k_idx == nullptr || n_valid == nullptr || idx_out == nullptr || k < 1)
    return CSA2_ERR_INVALID_ARG;
  if (k > s.topk) return CSA2_ERR_INVALID_ARG;      // the workspace is sized for shape.topk
  if (indexer_fast(s) && !aligned16(k_idx)) return CSA2_ERR_INVALID_ARG;
  const WsLayout L = layout(s);
  int* err = at<int>(ws, L.hdr);
  float* ts = at<float>(ws, L.tok_scores);
  int32_t* tc = at<int32_t>(ws, L.tok_cand);
  int32_t* nc = at<int32_t>(ws, L.n_cand);
  if (pool == nullptr) {
    if (indexer_fast(s) && index_select_supported(false, s.n_entries)) {
      SelectArgs a = select_args(s, k_idx, s.n_entries, seqdiv(s), q_idx, w, n_valid, 1, k, idx_out, k, n_out, err);
      return cuda_status(launch_index_select(a, false, s.batch, s.n_entries, stream));
    }
    CSA2_TRY(do_index_flat(s, q_idx, w, k_idx, s.n_entries, seqdiv(s), n_valid, 1, ts, nullptr, nc, s.n_entries, err, stream));
    return do_topk(s, L, ws, ts, s.n_entries, nullptr, nc, s.n_entries, k, idx_out, nullptr, n_out, stream);
  }
  if (s.pool_blocks < 1 || n_pool == nullptr || s.n_entries % s.block != 0) return CSA2_ERR_INVALID_ARG;
  if (pooled_fast(s) && index_select_supported(true, s.pool_blocks)) {
    SelectArgs a = select_args(s, k_idx, s.n_entries, seqdiv(s), q_idx, w, n_valid, 1, k, idx_out, k, n_out, err);
    a.pool = pool;
    a.n_pool = n_pool;
    a.pool_cap = s.pool_blocks;
    return cuda_status(launch_index_select(a, true, s.batch, s.pool_blocks, stream));
  }
  CSA2_TRY(do_index_pooled(s, q_idx, w, k_idx, n_valid, pool, n_pool, ts, tc, nc, err, stream));
  const int64_t ld = int64_t(s.pool_blocks) * s.block;
  return do_topk(s, L, ws, ts, ld, tc, nc, ld, k, idx_out, nullptr, n_out, stream);
}

int csa2_topk(const csa2_shape* shape, const float* scores, int32_t ld, const int32_t* cand,
              const int32_t* n_cand, int32_t k, int32_t* idx_out, float* score_out, void* ws, size_t ws_bytes,
              csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  if (scores == nullptr || idx_out == nullptr || ld < 1 || k < 1) return CSA2_ERR_INVALID_ARG;
  if (k > topk_max_chunk() || ld > (1 << 28)) return CSA2_ERR_UNSUPPORTED;
  const WsLayout L = layout(s);
  // the chunk buffers are sized for the shape's longest candidate list and max(K, P)
  const int64_t maxc = topk_max_chunk();
  if (ld > maxc) {
    const int64_t chunks = ceil_div(ld, maxc);
    if (k > maxc / 2) return CSA2_ERR_UNSUPPORTED;   // merges must shrink the list
    if (chunks > L.tk_chunks || k > L.tk_kmax) return CSA2_ERR_WORKSPACE;
  }
  return do_topk(s, L, ws, scores, ld, cand, n_cand, ld, k, idx_out, score_out, nullptr, stream);
}

int csa2_sparse_attn(const csa2_shape* shape, const void* q, const void* k_main, const void* v_main,
                     const int32_t* idx, const void* k_swa, const void* v_swa, const int32_t* n_swa, float* out,
                     float* lse, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  if (idx == nullptr) return CSA2_ERR_INVALID_ARG;
  CSA2_TRY(check_attn_args(s, q, k_main, v_main, out));
  CSA2_TRY(check_sswa(s, k_swa, v_swa, n_swa));
  const WsLayout L = layout(s);
  return do_attn(s, q, k_main, v_main, idx, k_swa, v_swa, n_swa, out, lse, at<int>(ws, L.hdr), stream);
}

int csa2_layer_group(const csa2_shape* shape, const csa2_layer* layers, int32_t n_layers, const void* k_main,
                     const void* v_main, const void* k_idx, const void* kb, const int32_t* n_valid,
                     const int32_t* n_swa, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  if (layers == nullptr || n_layers < 1 || k_idx == nullptr || n_valid == nullptr) return CSA2_ERR_INVALID_ARG;
  if (indexer_fast(s) && !aligned16(k_idx)) return CSA2_ERR_INVALID_ARG;
  // validate the whole group before enqueueing anything
  bool have_idx = false;
  for (int l = 0; l < n_layers; ++l) {
    const csa2_layer& y = layers[l];
    if (y.mode != CSA2_FULL && y.mode != CSA2_REINDEX && y.mode != CSA2_REUSE && y.mode != CSA2_SWA)
      return CSA2_ERR_INVALID_ARG;
    if (y.hier != 0 && y.hier != 1) return CSA2_ERR_INVALID_ARG;
    CSA2_TRY(check_attn_args(s, y.q, k_main, v_main, y.out));
    CSA2_TRY(check_sswa(s, y.k_swa, y.v_swa, n_swa));
    if (y.mode == CSA2_SWA) {
      if (s.swa < 1) return CSA2_ERR_INVALID_ARG;
      continue;
    }
    if (y.mode == CSA2_REUSE) {
      if (!have_idx) return CSA2_ERR_INVALID_ARG;
      continue;
    }
    if (y.q_idx == nullptr || y.w_idx == nullptr) return CSA2_ERR_INVALID_ARG;
    if (y.hier) {
      if (kb == nullptr || s.pool_blocks < 1 || s.n_entries % s.block != 0) return CSA2_ERR_INVALID_ARG;
      if (indexer_fast(s) && !aligned16(kb)) return CSA2_ERR_INVALID_ARG;
    }
    have_idx = true;
  }
  const WsLayout L = layout(s);
  int* err = at<int>(ws, L.hdr);
  const int32_t* cur = nullptr;
  for (int l = 0; l < n_layers; ++l) {
    const csa2_layer& y = layers[l];
    // Another attention-only launch next (Reuse or SWA layer): release it at this
    // attention's end, unless the batch is small enough that both launches' CTAs
    // find SMs of their own (then its CTAs fetch their window rows early).
    const bool attn_next = l + 1 < n_layers && (layers[l + 1].mode == CSA2_REUSE || layers[l + 1].mode == CSA2_SWA) &&
                           !(attn_fast(s) && 2 * s.batch * attn_cluster(s.topk, s.swa) <= device_sm_count());
    if (y.mode == CSA2_SWA) {
      CSA2_TRY(do_attn(s, y.q, k_main, v_main, nullptr, y.k_swa, y.v_swa, n_swa, y.out, y.lse, err, stream, true,
                       attn_next));
      continue;
    }
    if (y.mode != CSA2_REUSE) {
      int32_t* dst = y.idx_out != nullptr ? y.idx_out : at<int32_t>(ws, L.idx);
      float* ts = at<float>(ws, L.tok_scores);
      int32_t* tc = at<int32_t>(ws, L.tok_cand);
      int32_t* nc = at<int32_t>(ws, L.n_cand);
      if (y.hier) {
        int32_t* pool = at<int32_t>(ws, L.pool);
        int32_t* npool = at<int32_t>(ws, L.n_pool);
        CSA2_TRY(do_index_blocks(s, L, ws, y.q_idx, y.w_idx, kb, n_valid, pool, npool, stream));
        if (pooled_fast(s) && index_select_supported(true, s.pool_blocks)) {
          // fused: pooled token scoring and Top-K in one cluster launch
          SelectArgs a = select_args(s, k_idx, s.n_entries, seqdiv(s), y.q_idx, y.w_idx, n_valid, 1, s.topk, dst, s.topk,
                                     nullptr, err);
          a.pool = pool;
          a.n_pool = npool;
          a.pool_cap = s.pool_blocks;
          CSA2_TRY(cuda_status(launch_index_select(a, true, s.batch, s.pool_blocks, stream)));
        } else {
          CSA2_TRY(do_index_pooled(s, y.q_idx, y.w_idx, k_idx, n_valid, pool, npool, ts, tc, nc, err, stream));
          const int64_t ld = int64_t(s.pool_blocks) * s.block;
          CSA2_TRY(do_topk(s, L, ws, ts, ld, tc, nc, ld, s.topk, dst, nullptr, nullptr, stream));
        }
      } else if (indexer_fast(s) && index_select_supported(false, s.n_entries)) {
        // fused: flat token scoring and Top-K in one cluster launch
        SelectArgs a = select_args(s, k_idx, s.n_entries, seqdiv(s), y.q_idx, y.w_idx, n_valid, 1, s.topk, dst, s.topk,
                                   nullptr, err);
        CSA2_TRY(cuda_status(launch_index_select(a, false, s.batch, s.n_entries, stream)));
      } else {
        CSA2_TRY(do_index_flat(s, y.q_idx, y.w_idx, k_idx, s.n_entries, seqdiv(s), n_valid, 1, ts, nullptr, nc, s.n_entries,
                               err, stream));
        CSA2_TRY(do_topk(s, L, ws, ts, s.n_entries, nullptr, nc, s.n_entries, s.topk, dst, nullptr, nullptr,
                         stream));
      }
      cur = dst;
    }
    CSA2_TRY(do_attn(s, y.q, k_main, v_main, cur, y.k_swa, y.v_swa, n_swa, y.out, y.lse, err, stream, false,
                     attn_next));
  }
  return CSA2_OK;
}

int csa2_shard_slice(const int32_t* ids, int32_t batch, int32_t ld, int32_t lo, int32_t hi, int32_t delta,
                     int32_t* out, int32_t ld_out, int32_t* n_out, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  if (ids == nullptr || out == nullptr || batch < 1 || ld < 1 || ld_out < 1 || lo > hi) return CSA2_ERR_INVALID_ARG;
  if (ld > (1 << 24) || ld_out > (1 << 24) || batch > (1 << 20)) return CSA2_ERR_UNSUPPORTED;
  if (int64_t(hi) + delta > INT32_MAX || int64_t(lo) + delta < INT32_MIN) return CSA2_ERR_INVALID_ARG;
  if (ws == nullptr || ws_bytes < 256 || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return CSA2_ERR_WORKSPACE;
  ShardSliceArgs a{};
  a.ids = ids;
  a.ld = ld;
  a.lo = lo;
  a.hi = hi;
  a.delta = delta;
  a.out = out;
  a.ld_out = ld_out;
  a.n_out = n_out;
  a.err = static_cast<int*>(ws);
  return cuda_status(launch_shard_slice(a, batch, stream));
}

int csa2_shard_counts(const int32_t* n_valid, int32_t batch, int32_t e0, int32_t n_loc, int32_t div, int32_t* out,
                      csa2_stream_t stream) {
  if (n_valid == nullptr || out == nullptr || batch < 1 || e0 < 0 || n_loc < 0 || div < 1) return CSA2_ERR_INVALID_ARG;
  return cuda_status(launch_shard_counts(n_valid, batch, e0, n_loc, div, out, stream));
}

int csa2_concat_parts(int32_t parts, int32_t batch, int32_t k, const int32_t* ids, const float* scores,
                      int32_t* ids_out, float* scores_out, csa2_stream_t stream) {
  if (parts < 1 || batch < 1 || k < 1 || ids == nullptr || ids_out == nullptr) return CSA2_ERR_INVALID_ARG;
  if (scores != nullptr && scores_out == nullptr) return CSA2_ERR_INVALID_ARG;
  if (int64_t(parts) * k > (1 << 28)) return CSA2_ERR_UNSUPPORTED;
  ConcatArgs a{};
  a.ids = ids;
  a.scores = scores;
  a.ids_out = ids_out;
  a.scores_out = scores_out;
  a.parts = parts;
  a.batch = batch;
  a.k = k;
  return cuda_status(launch_concat_parts(a, stream));
}

int csa2_merge_attn(int32_t parts, int32_t rows, int32_t v_dim, const float* out_parts, const float* lse_parts,
                    float* out, float* lse, csa2_stream_t stream) {
  if (parts < 1 || rows < 1 || v_dim < 1 || out_parts == nullptr || lse_parts == nullptr || out == nullptr)
    return CSA2_ERR_INVALID_ARG;
  if (parts > 1024 || v_dim > 1024 || int64_t(rows) * v_dim * parts > (int64_t(1) << 40)) return CSA2_ERR_UNSUPPORTED;
  MergeAttnArgs a{};
  a.out_parts = out_parts;
  a.lse_parts = lse_parts;
  a.out = out;
  a.lse = lse;
  a.parts = parts;
  a.rows = rows;
  a.v_dim = v_dim;
  return cuda_status(launch_merge_attn(a, stream));
}

// ---------------------------------------------------------------- drafted tokens and bounded caches

int csa2_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, int32_t orig_ctx, double beta_fast,
                    double beta_slow, double* freqs, float* mag) {
  if (freqs == nullptr || rot_dim < 2 || rot_dim > kMaxRotDim || rot_dim % 2 != 0) return CSA2_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base)) return CSA2_ERR_INVALID_ARG;
  if (scaling < CSA2_ROPE_PLAIN || scaling > CSA2_ROPE_YARN) return CSA2_ERR_INVALID_ARG;
  if (scaling != CSA2_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return CSA2_ERR_INVALID_ARG;
  if (scaling == CSA2_ROPE_NTK && rot_dim == 2) return CSA2_ERR_INVALID_ARG;
  if (scaling == CSA2_ROPE_YARN &&
      (orig_ctx < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
    return CSA2_ERR_INVALID_ARG;
  const double b = scaling == CSA2_ROPE_NTK ? base * std::pow(factor, double(rot_dim) / (rot_dim - 2)) : base;
  if (!std::isfinite(b)) return CSA2_ERR_INVALID_ARG;   // (its pairs would not turn at all)
  // the (real-valued) pair that turns `turns` times over orig_ctx positions
  const double two_pi = 6.283185307179586476925286766559;
  auto pair_of = [&](double turns) { return rot_dim * std::log(orig_ctx / (turns * two_pi)) / (2.0 * std::log(base)); };
  double lo = 0.0, hi = 1.0;
  if (scaling == CSA2_ROPE_YARN) {
    lo = std::fmax(0.0, std::floor(pair_of(beta_fast)));
    hi = std::fmin(rot_dim - 1.0, std::ceil(pair_of(beta_slow)));
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rot_dim);
    if (scaling == CSA2_ROPE_LINEAR) f /= factor;
    if (scaling == CSA2_ROPE_YARN) {
      const double keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
      f = f / factor * (1.0 - keep) + f * keep;
    }
    freqs[i] = f;
  }
  if (mag != nullptr) *mag = scaling == CSA2_ROPE_YARN ? float(0.1 * std::log(factor) + 1.0) : 1.f;
  return CSA2_OK;
}

int csa2_rope(const csa2_rope_slot* slots, int32_t n_slots, int32_t rows, int32_t rot_dim, int32_t interleaved,
              const int32_t* pos, const double* freqs, float mag, int32_t inverse, csa2_stream_t stream) {
  if (slots == nullptr || n_slots < 1 || n_slots > kMaxRopeSlots || rows < 1) return CSA2_ERR_INVALID_ARG;
  if (rot_dim < 2 || rot_dim % 2 != 0 || pos == nullptr || freqs == nullptr || !aligned(4, pos) || !aligned8(freqs))
    return CSA2_ERR_INVALID_ARG;
  if (rot_dim > kMaxRotDim) return CSA2_ERR_UNSUPPORTED;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1)) return CSA2_ERR_INVALID_ARG;
  if (!(mag > 0.f) || !std::isfinite(mag) || !std::isfinite(1.f / mag)) return CSA2_ERR_INVALID_ARG;
  RopeArgs a{};
  for (int k = 0; k < n_slots; ++k) {
    const csa2_rope_slot& y = slots[k];
    if (y.x == nullptr || y.out == nullptr || y.heads < 1 || y.dim < 1 || y.rot_off < 0) return CSA2_ERR_INVALID_ARG;
    if (int64_t(y.rot_off) + rot_dim > y.dim) return CSA2_ERR_INVALID_ARG;
    if (y.dtype != CSA2_BF16 && y.dtype != CSA2_F32) return CSA2_ERR_INVALID_ARG;
    if (!aligned(elem_size(y.dtype), y.x, y.out)) return CSA2_ERR_INVALID_ARG;
    if (y.heads > 1024 || y.dim > 1024) return CSA2_ERR_UNSUPPORTED;
    a.slot[k].x = y.x;
    a.slot[k].out = y.out;
    a.slot[k].heads = y.heads;
    a.slot[k].dim = y.dim;
    a.slot[k].off = y.rot_off;
    a.slot[k].dtype = y.dtype;
  }
  // an output may be its own input; it may touch nothing else that the call reads or writes
  auto bytes = [&](int k) { return uint64_t(rows) * slots[k].heads * slots[k].dim * (slots[k].dtype == CSA2_F32 ? 4 : 2); };
  for (int k = 0; k < n_slots; ++k) {
    if (overlap(slots[k].out, bytes(k), pos, uint64_t(rows) * 4) || overlap(slots[k].out, bytes(k), freqs, uint64_t(rot_dim) * 4))
      return CSA2_ERR_INVALID_ARG;
    for (int j = 0; j < n_slots; ++j) {
      if ((j != k || slots[k].out != slots[k].x) && overlap(slots[k].out, bytes(k), slots[j].x, bytes(j)))
        return CSA2_ERR_INVALID_ARG;
      if (j != k && overlap(slots[k].out, bytes(k), slots[j].out, bytes(j))) return CSA2_ERR_INVALID_ARG;
    }
  }
  a.n_slots = n_slots;
  a.rot = rot_dim;
  a.interleaved = interleaved;
  a.inverse = inverse;
  a.mag = mag;
  a.pos = pos;
  a.freqs = freqs;
  return cuda_status(launch_rope(a, rows, stream));
}

int csa2_tree_attn(const csa2_shape* shape, const void* q, const void* k_main, const void* v_main, const int32_t* idx,
                   const void* k_swa, const void* v_swa, const int32_t* swa_head, const int32_t* n_swa,
                   const void* k_draft, const void* v_draft, const int32_t* parent, const int32_t* n_draft, void* out,
                   float* lse, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  if (s.swa < 1) return CSA2_ERR_INVALID_ARG;
  if (seqdiv(s) > kMaxTreeTokens || s.batch > kMaxGridY) return CSA2_ERR_UNSUPPORTED;
  for (const void* p : {q, k_main, v_main, static_cast<const void*>(idx), k_swa, v_swa, static_cast<const void*>(n_swa),
                        k_draft, v_draft, static_cast<const void*>(out)})
    if (p == nullptr) return CSA2_ERR_INVALID_ARG;
  if (attn_fast(s))
    for (const void* p : {q, k_main, v_main, k_swa, v_swa, k_draft, v_draft, static_cast<const void*>(out)})
      if (!aligned16(p)) return CSA2_ERR_INVALID_ARG;
  if (!aligned(elem_size(s.dtype), q, k_main, v_main, k_swa, v_swa, k_draft, v_draft, out) ||
      !aligned(4, idx, swa_head, n_swa, parent, n_draft, lse))
    return CSA2_ERR_INVALID_ARG;
  const uint64_t B = s.batch, S = B / seqdiv(s), esize = s.dtype == CSA2_F32 ? 4 : 2;
  const uint64_t kb = s.k_dim * esize, vb = s.v_dim * esize;
  Span spans[] = {{q, B * s.q_heads * kb, false}, {k_main, S * s.n_entries * kb, false}, {v_main, S * s.n_entries * vb, false},
                  {idx, B * s.topk * 4, false}, {k_swa, S * s.swa * kb, false}, {v_swa, S * s.swa * vb, false},
                  {swa_head, S * 4, false}, {n_swa, S * 4, false}, {k_draft, B * kb, false}, {v_draft, B * vb, false},
                  {parent, B * 4, false}, {n_draft, S * 4, false}, {out, B * s.q_heads * vb, true}, {lse, B * s.q_heads * 4, true},
                  {ws, ws_bytes, true}};
  if (written_overlap(spans, sizeof(spans) / sizeof(spans[0]))) return CSA2_ERR_INVALID_ARG;
  TreeArgs a{};
  a.q = q;
  a.k_main = k_main;
  a.v_main = v_main;
  a.idx = idx;
  a.k_swa = k_swa;
  a.v_swa = v_swa;
  a.swa_head = swa_head;
  a.n_swa = n_swa;
  a.k_draft = k_draft;
  a.v_draft = v_draft;
  a.parent = parent;
  a.n_draft = n_draft;
  a.out = out;
  a.lse = lse;
  a.tokens = seqdiv(s);
  a.n_entries = s.n_entries;
  a.topk = s.topk;
  a.swa = s.swa;
  a.heads = s.q_heads;
  a.k_dim = s.k_dim;
  a.v_dim = s.v_dim;
  a.dtype = s.dtype;
  a.scale = softmax_scale(s);
  a.err = static_cast<int*>(ws);
  // the groups' key lists live in the workspace from the token scores on, which hold nothing between calls
  const WsLayout L = layout(s);
  return cuda_status(launch_tree_attn(a, attn_fast(s), s.batch, at<void>(ws, L.tok_scores), ws_bytes - L.tok_scores, stream));
}

int csa2_attn_weights(const csa2_shape* shape, const void* q, const void* k_main, const int32_t* idx, const float* lse,
                      const int32_t* live, float* weights, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  if (s.batch > kMaxGridY) return CSA2_ERR_UNSUPPORTED;
  if (q == nullptr || k_main == nullptr || idx == nullptr || lse == nullptr || weights == nullptr)
    return CSA2_ERR_INVALID_ARG;
  const bool fast = s.dtype == CSA2_BF16 && s.q_heads == 64 && s.k_dim == 192;
  if (fast && (!aligned16(q) || !aligned16(k_main))) return CSA2_ERR_INVALID_ARG;
  if (!aligned(elem_size(s.dtype), q, k_main) || !aligned(4, idx, lse, live, weights)) return CSA2_ERR_INVALID_ARG;
  const uint64_t B = s.batch, kb = uint64_t(s.k_dim) * (s.dtype == CSA2_F32 ? 4 : 2);
  Span spans[] = {{q, B * s.q_heads * kb, false}, {k_main, B / seqdiv(s) * s.n_entries * kb, false}, {idx, B * s.topk * 4, false},
                  {lse, B * s.q_heads * 4, false}, {live, B * 4, false}, {weights, B * s.topk * 4, true}, {ws, ws_bytes, true}};
  if (written_overlap(spans, sizeof(spans) / sizeof(spans[0]))) return CSA2_ERR_INVALID_ARG;
  AttnWeightsArgs a{};
  a.q = q;
  a.k_main = k_main;
  a.idx = idx;
  a.lse = lse;
  a.live = live;
  a.weights = weights;
  a.seq_div = seqdiv(s);
  a.n_entries = s.n_entries;
  a.topk = s.topk;
  a.heads = s.q_heads;
  a.k_dim = s.k_dim;
  a.dtype = s.dtype;
  a.scale = softmax_scale(s);
  a.err = static_cast<int*>(ws);
  return cuda_status(launch_attn_weights(a, fast, s.batch, stream));
}

int csa2_tree_commit(const csa2_shape* shape, const csa2_tree_slot* layers, int32_t n_layers, const int32_t* path,
                     const int32_t* n_path, int32_t* swa_head, int32_t* n_swa, int64_t* mass, void* ws, size_t ws_bytes,
                     csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  if (s.swa < 1 || layers == nullptr || n_layers < 1 || n_layers > kMaxTreeLayers) return CSA2_ERR_INVALID_ARG;
  if (path == nullptr || n_path == nullptr || swa_head == nullptr || n_swa == nullptr) return CSA2_ERR_INVALID_ARG;
  if (!aligned8(mass) || !aligned(4, path, n_path, swa_head, n_swa)) return CSA2_ERR_INVALID_ARG;
  const int T = seqdiv(s), S = s.batch / T;
  if (T > kMaxTreeTokens || S > kMaxGridY) return CSA2_ERR_UNSUPPORTED;
  int* err = nullptr;
  CSA2_TRY(error_word(s, ws, ws_bytes, &err));
  TreeCommitArgs a{};
  const int esize = s.dtype == CSA2_F32 ? 4 : 2;
  a.k_bytes = s.k_dim * esize;
  a.v_bytes = s.v_dim * esize;
  a.wide = a.k_bytes % 16 == 0 && a.v_bytes % 16 == 0;
  const uint64_t nb = uint64_t(s.batch) * 4, sb = uint64_t(S) * 4;
  Span spans[6 + 6 * kMaxTreeLayers] = {{path, nb, false}, {n_path, sb, false}, {swa_head, sb, true}, {n_swa, sb, true},
                                        {mass, uint64_t(S) * s.n_entries * 8, true}, {ws, ws_bytes, true}};
  int n_spans = 6;
  for (int l = 0; l < n_layers; ++l) {
    const csa2_tree_slot& y = layers[l];
    if (y.k_draft == nullptr || y.v_draft == nullptr || y.k_swa == nullptr || y.v_swa == nullptr)
      return CSA2_ERR_INVALID_ARG;
    if ((y.idx == nullptr) != (y.weights == nullptr)) return CSA2_ERR_INVALID_ARG;
    if (!aligned(elem_size(s.dtype), y.k_draft, y.v_draft, y.k_swa, y.v_swa) || !aligned(4, y.idx, y.weights))
      return CSA2_ERR_INVALID_ARG;
    if (!aligned16(y.k_draft) || !aligned16(y.v_draft) || !aligned16(y.k_swa) || !aligned16(y.v_swa)) a.wide = 0;
    a.slot[l] = TreeCommitArgs::Slot{y.k_draft, y.v_draft, y.k_swa, y.v_swa, y.idx, y.weights};
    for (const Span& x : {Span{y.k_draft, uint64_t(s.batch) * a.k_bytes, false}, Span{y.v_draft, uint64_t(s.batch) * a.v_bytes, false},
                          Span{y.k_swa, uint64_t(S) * s.swa * a.k_bytes, true}, Span{y.v_swa, uint64_t(S) * s.swa * a.v_bytes, true},
                          Span{y.idx, nb * s.topk, false}, Span{y.weights, nb * s.topk, false}})
      spans[n_spans++] = x;
  }
  if (written_overlap(spans, n_spans)) return CSA2_ERR_INVALID_ARG;
  a.n_layers = n_layers;
  a.path = path;
  a.n_path = n_path;
  a.head = swa_head;
  a.n_swa = n_swa;
  a.mass = reinterpret_cast<unsigned long long*>(mass);
  a.tokens = T;
  a.n_entries = s.n_entries;
  a.topk = s.topk;
  a.swa = s.swa;
  a.err = err;
  return cuda_status(launch_tree_commit(a, S, stream));
}

int csa2_kv_evict(const csa2_shape* shape, int32_t trigger, int32_t keep, int32_t sink, int32_t recent,
                  const void* k_main, const void* v_main, const void* k_idx, const int64_t* mass, const int32_t* n_valid,
                  void* k_main_out, void* v_main_out, void* k_idx_out, int64_t* mass_out, int32_t* n_valid_out,
                  int32_t* kept, void* kb_out, int32_t round_to_int, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  if (seqdiv(s) != 1) return CSA2_ERR_UNSUPPORTED;   // caches are per sequence: pass a one-token shape
  if (s.batch > kMaxGridY) return CSA2_ERR_UNSUPPORTED;
  if (keep < 1 || trigger < keep || trigger > s.n_entries || sink < 0 || recent < 0 || sink > keep || recent > keep - sink)
    return CSA2_ERR_INVALID_ARG;
  if (round_to_int != 0 && round_to_int != 1) return CSA2_ERR_INVALID_ARG;
  const uint64_t B = s.batch, N = s.n_entries, nb = uint64_t(ceil_div(s.n_entries, s.block));
  const uint64_t esize = s.dtype == CSA2_F32 ? 4 : 2;
  struct Pair {
    const void* in;
    void* out;
    uint64_t bytes;
  };
  const Pair io[5] = {{k_main, k_main_out, B * N * s.k_dim * esize},
                      {v_main, v_main_out, B * N * s.v_dim * esize},
                      {k_idx, k_idx_out, B * N * s.idx_dim * esize},
                      {mass, mass_out, B * N * 8},
                      {n_valid, n_valid_out, B * 4}};
  const Pair extra[2] = {{nullptr, kept, B * N * 4}, {nullptr, kb_out, B * nb * s.idx_dim * esize}};
  if (kept == nullptr || !aligned8(mass) || !aligned8(mass_out)) return CSA2_ERR_INVALID_ARG;
  if (!aligned(size_t(esize), k_main, v_main, k_idx, k_main_out, v_main_out, k_idx_out, kb_out) ||
      !aligned(4, n_valid, n_valid_out, kept))
    return CSA2_ERR_INVALID_ARG;
  int same = 0;
  for (const Pair& x : io) {
    if (x.in == nullptr || x.out == nullptr) return CSA2_ERR_INVALID_ARG;
    same += x.in == x.out;
  }
  if (same != 0 && same != 5) return CSA2_ERR_INVALID_ARG;   // in place wholly, or not at all
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < 5; ++j) {
      if (!(same && i == j) && overlap(io[i].out, io[i].bytes, io[j].in, io[j].bytes)) return CSA2_ERR_INVALID_ARG;
      if (i != j && overlap(io[i].out, io[i].bytes, io[j].out, io[j].bytes)) return CSA2_ERR_INVALID_ARG;
    }
  for (const Pair& x : extra) {
    if (x.out == nullptr) continue;
    for (const Pair& y : io)
      if (overlap(x.out, x.bytes, y.in, y.bytes) || overlap(x.out, x.bytes, y.out, y.bytes)) return CSA2_ERR_INVALID_ARG;
  }
  if (kb_out != nullptr && overlap(kept, extra[0].bytes, kb_out, extra[1].bytes)) return CSA2_ERR_INVALID_ARG;
  int* err = nullptr;
  CSA2_TRY(error_word(s, ws, ws_bytes, &err));
  if (ws != nullptr) {
    for (const Pair& x : io)
      if (overlap(x.in, x.bytes, ws, ws_bytes) || overlap(x.out, x.bytes, ws, ws_bytes)) return CSA2_ERR_INVALID_ARG;
    for (const Pair& x : extra)
      if (x.out != nullptr && overlap(x.out, x.bytes, ws, ws_bytes)) return CSA2_ERR_INVALID_ARG;
  }
  EvictArgs a{};
  a.k_main = k_main;
  a.v_main = v_main;
  a.k_idx = k_idx;
  a.mass = reinterpret_cast<const long long*>(mass);
  a.n_valid = n_valid;
  a.k_main_out = k_main_out;
  a.v_main_out = v_main_out;
  a.k_idx_out = k_idx_out;
  a.mass_out = reinterpret_cast<long long*>(mass_out);
  a.n_valid_out = n_valid_out;
  a.kept = kept;
  a.kb = kb_out;
  a.trigger = trigger;
  a.keep = keep;
  a.sink = sink;
  a.recent = recent;
  a.n_entries = s.n_entries;
  a.nb_cap = int(nb);
  a.idx_dim = s.idx_dim;
  a.block = s.block;
  a.round_to_int = round_to_int;
  a.dtype = s.dtype;
  a.k_bytes = int(s.k_dim * esize);
  a.v_bytes = int(s.v_dim * esize);
  a.x_bytes = int(s.idx_dim * esize);
  a.wide = a.k_bytes % 16 == 0 && a.v_bytes % 16 == 0 && a.x_bytes % 16 == 0;
  for (int i = 0; i < 3; ++i)
    if (!aligned16(io[i].in) || !aligned16(io[i].out)) a.wide = 0;
  a.in_place = same != 0;
  a.err = err;
  return cuda_status(launch_kv_evict(a, s.batch, stream));
}

// ---------------------------------------------------------------- main caches held in 4 bits

size_t csa2_kv4_bytes(int32_t k_dim, int32_t v_dim) {
  if (k_dim < 1 || k_dim > 1024 || v_dim < 1 || v_dim > 1024) return 0;
  return size_t(kv4_bytes(k_dim, v_dim));
}

int csa2_norm_rope(const csa2_norm_rope_slot* slots, int32_t n_slots, int32_t rows, int32_t rot_dim, int32_t interleaved,
                   int32_t center, const int32_t* pos, const double* freqs, float mag, float eps, csa2_stream_t stream) {
  if (slots == nullptr || n_slots < 1 || n_slots > kMaxRopeSlots || rows < 1) return CSA2_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim % 2 != 0) return CSA2_ERR_INVALID_ARG;
  if (rot_dim > 0 && (pos == nullptr || freqs == nullptr || !aligned(4, pos) || !aligned8(freqs))) return CSA2_ERR_INVALID_ARG;
  if (rot_dim > kMaxRotDim) return CSA2_ERR_UNSUPPORTED;
  if ((interleaved != 0 && interleaved != 1) || (center != 0 && center != 1)) return CSA2_ERR_INVALID_ARG;
  if (!(mag > 0.f) || !std::isfinite(mag) || !(eps >= 0.f) || !std::isfinite(eps)) return CSA2_ERR_INVALID_ARG;
  NormRopeArgs a{};
  Rows x[kMaxRopeSlots], out[kMaxRopeSlots], gain[kMaxRopeSlots];
  for (int k = 0; k < n_slots; ++k) {
    const csa2_norm_rope_slot& y = slots[k];
    if (y.x == nullptr || y.out == nullptr || y.heads < 1 || y.dim < 1 || y.rot_off < 0) return CSA2_ERR_INVALID_ARG;
    if (rot_dim > 0 && int64_t(y.rot_off) + rot_dim > y.dim) return CSA2_ERR_INVALID_ARG;
    if (y.dtype != CSA2_BF16 && y.dtype != CSA2_F32) return CSA2_ERR_INVALID_ARG;
    if (y.gain_each != 0 && y.gain_each != 1) return CSA2_ERR_INVALID_ARG;
    if (!aligned(elem_size(y.dtype), y.x, y.out) || !aligned(4, y.gain)) return CSA2_ERR_INVALID_ARG;
    if (y.heads > 1024 || y.dim > 1024) return CSA2_ERR_UNSUPPORTED;
    const int64_t width = int64_t(y.heads) * y.dim;
    if (y.x_stride < width || y.out_stride < width) return CSA2_ERR_INVALID_ARG;
    if (y.x_stride > (int64_t(1) << 28) || y.out_stride > (int64_t(1) << 28)) return CSA2_ERR_UNSUPPORTED;
    if (y.x == y.out && y.x_stride != y.out_stride && rows > 1) return CSA2_ERR_INVALID_ARG;
    const uint64_t e = elem_size(y.dtype);
    a.slot[k] = NormRopeArgs::Slot{y.x, y.out, y.gain, y.x_stride, y.out_stride, y.heads, y.dim, rot_dim > 0 ? y.rot_off : 0,
                                   y.dtype, y.gain_each, 0, 0, 0, 0};
    x[k] = {y.x, width * e, y.x_stride * e, uint64_t(rows)};
    out[k] = {y.out, width * e, y.out_stride * e, uint64_t(rows)};
    gain[k] = {y.gain, uint64_t(y.gain_each ? width : y.dim) * 4, 0, 1};
  }
  // an output may be its own input; it may touch nothing else that the call reads or writes
  const Rows pos_rows{rot_dim > 0 ? pos : nullptr, uint64_t(rows) * 4, 0, 1}, freq_rows{rot_dim > 0 ? freqs : nullptr, uint64_t(rot_dim) * 4, 0, 1};
  for (int k = 0; k < n_slots; ++k) {
    if (overlap(out[k], pos_rows) || overlap(out[k], freq_rows)) return CSA2_ERR_INVALID_ARG;
    for (int j = 0; j < n_slots; ++j) {
      if ((j != k || out[k].at != x[k].at) && overlap(out[k], x[j])) return CSA2_ERR_INVALID_ARG;
      if ((j != k && overlap(out[k], out[j])) || overlap(out[k], gain[j])) return CSA2_ERR_INVALID_ARG;
    }
  }
  a.n_slots = n_slots;
  a.rot = rot_dim;
  a.interleaved = interleaved;
  a.center = center;
  a.mag = mag;
  a.eps = eps;
  a.pos = pos;
  a.freqs = freqs;
  return cuda_status(launch_norm_rope(a, rows, stream));
}

int csa2_kv4_append(const csa2_shape* shape, int32_t max_new, const int32_t* n_new, const void* k_new, const void* v_new,
                    const void* kidx_new, void* kv4, void* k_idx, void* kb, int32_t* n_valid, int32_t k_exp,
                    int32_t v_exp, int32_t round_to_int, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  if (seqdiv(s) != 1 || s.batch > kMaxGridY) return CSA2_ERR_UNSUPPORTED;   // caches are per sequence: pass a one-token shape
  if (max_new < 1 || (round_to_int != 0 && round_to_int != 1)) return CSA2_ERR_INVALID_ARG;
  CSA2_TRY(check_exps(k_exp, v_exp));
  for (const void* p : {static_cast<const void*>(n_new), k_new, v_new, kidx_new, static_cast<const void*>(kv4),
                        static_cast<const void*>(k_idx), static_cast<const void*>(n_valid)})
    if (p == nullptr) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(kv4) || !aligned(elem_size(s.dtype), k_new, v_new, kidx_new, k_idx, kb) || !aligned(4, n_new, n_valid))
    return CSA2_ERR_INVALID_ARG;
  int* err = nullptr;
  CSA2_TRY(error_word(s, ws, ws_bytes, &err));
  const uint64_t B = s.batch, N = s.n_entries, M = max_new, e = elem_size(s.dtype), x = s.idx_dim * e;
  const int64_t nb = ceil_div(s.n_entries, s.block);
  Span spans[] = {{n_new, B * 4, false}, {k_new, B * M * s.k_dim * e, false}, {v_new, B * M * s.v_dim * e, false},
                  {kidx_new, B * M * x, false}, {kv4, B * N * kv4_bytes(s.k_dim, s.v_dim), true}, {k_idx, B * N * x, true},
                  {kb, B * uint64_t(nb) * x, true}, {n_valid, B * 4, true}, {ws, ws_bytes, true}};
  if (written_overlap(spans, sizeof(spans) / sizeof(spans[0]))) return CSA2_ERR_INVALID_ARG;
  Kv4AppendArgs a{};
  a.n_new = n_new;
  a.max_new = max_new;
  a.k_new = k_new;
  a.v_new = v_new;
  a.kidx_new = kidx_new;
  a.kv = static_cast<uint8_t*>(kv4);
  a.k_idx = k_idx;
  a.kb = kb;
  a.n_valid = n_valid;
  a.n_entries = s.n_entries;
  a.nb_cap = int(nb);
  a.k_dim = s.k_dim;
  a.v_dim = s.v_dim;
  a.idx_dim = s.idx_dim;
  a.block = s.block;
  a.round_to_int = round_to_int;
  a.dtype = s.dtype;
  a.k_down = std::ldexp(1.f, -k_exp);
  a.v_down = std::ldexp(1.f, -v_exp);
  a.wide = s.k_dim % 16 == 0 && s.v_dim % 16 == 0 && aligned16(k_new) && aligned16(v_new);
  a.wide_idx = x % 16 == 0 && aligned16(kidx_new) && aligned16(k_idx);
  a.err = err;
  return cuda_status(launch_kv4_append(a, s.batch, stream));
}

int csa2_kv4_rows(const csa2_shape* shape, const void* kv4, const int32_t* idx, int32_t n_rows, void* k_out, void* v_out,
                  int32_t k_exp, int32_t v_exp, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  if (n_rows < 1) return CSA2_ERR_INVALID_ARG;
  if (int64_t(s.batch) * n_rows > 0x7fffffffLL) return CSA2_ERR_UNSUPPORTED;
  CSA2_TRY(check_exps(k_exp, v_exp));
  if (kv4 == nullptr || idx == nullptr || k_out == nullptr || v_out == nullptr) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(kv4) || !aligned(elem_size(s.dtype), k_out, v_out) || !aligned(4, idx)) return CSA2_ERR_INVALID_ARG;
  int* err = nullptr;
  CSA2_TRY(error_word(s, ws, ws_bytes, &err));
  const uint64_t B = s.batch, R = n_rows, e = elem_size(s.dtype);
  Span spans[] = {{kv4, B / seqdiv(s) * s.n_entries * kv4_bytes(s.k_dim, s.v_dim), false}, {idx, B * R * 4, false},
                  {k_out, B * R * s.k_dim * e, true}, {v_out, B * R * s.v_dim * e, true}, {ws, ws_bytes, true}};
  if (written_overlap(spans, sizeof(spans) / sizeof(spans[0]))) return CSA2_ERR_INVALID_ARG;
  Kv4RowsArgs a{};
  a.kv = static_cast<const uint8_t*>(kv4);
  a.idx = idx;
  a.k_out = k_out;
  a.v_out = v_out;
  a.seq_div = seqdiv(s);
  a.n_entries = s.n_entries;
  a.rows = n_rows;
  a.k_dim = s.k_dim;
  a.v_dim = s.v_dim;
  a.dtype = s.dtype;
  a.k_up = std::ldexp(1.f, k_exp);
  a.v_up = std::ldexp(1.f, v_exp);
  a.wide = s.k_dim * e % 16 == 0 && s.v_dim * e % 16 == 0 && aligned16(k_out) && aligned16(v_out);
  a.err = err;
  return cuda_status(launch_kv4_rows(a, s.batch, stream));
}

int csa2_kv4_attn(const csa2_shape* shape, const void* q, const void* kv4, const int32_t* idx, const void* k_swa,
                  const void* v_swa, const int32_t* n_swa, void* out, float* lse, int32_t k_exp, int32_t v_exp, void* ws,
                  size_t ws_bytes, csa2_stream_t stream) {
  Kv4AttnArgs a{};
  CSA2_TRY(kv4_attn_args(shape, q, kv4, idx, k_swa, v_swa, n_swa, out, lse, k_exp, v_exp, ws, ws_bytes, a));
  return cuda_status(launch_kv4_attn(a, attn_fast(*shape), shape->batch, stream));
}

const char* csa2_status_str(int status) {
  switch (status) {
    case CSA2_OK: return "ok";
    case CSA2_ERR_INVALID_ARG: return "invalid argument (null/misaligned pointer, bad size or mode sequence)";
    case CSA2_ERR_UNSUPPORTED: return "unsupported shape";
    case CSA2_ERR_WORKSPACE: return "workspace too small or misaligned";
    case CSA2_ERR_CUDA: return "CUDA launch or runtime error";
    case CSA2_ERR_DEVICE_CHECK: return "a kernel recorded an out-of-range input";
    case CSA2_ERR_TIMEOUT: return "a bounded device wait gave up";
    default: return "unknown status";
  }
}

int csa2_read_device_error(void* ws, csa2_stream_t stream, int32_t* detail) {
  if (ws == nullptr) return CSA2_ERR_WORKSPACE;
  int host[2] = {0, 0};
  if (cudaMemcpyAsync(host, ws, sizeof(host), cudaMemcpyDeviceToHost, stream) != cudaSuccess)
    return CSA2_ERR_CUDA;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return CSA2_ERR_CUDA;
  if (cudaMemsetAsync(ws, 0, sizeof(host), stream) != cudaSuccess) return CSA2_ERR_CUDA;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return CSA2_ERR_CUDA;
  if (detail != nullptr) *detail = host[0] & 0xff;
  if (host[0] == 0) return CSA2_OK;
  return (host[0] & kErrTimeout) ? CSA2_ERR_TIMEOUT : CSA2_ERR_DEVICE_CHECK;
}

unsigned long long csa2_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int csa2_debug_wait_timeout(const csa2_shape* shape, const void* q_idx, const float* w, const void* k_idx,
                            const int32_t* n_valid, int32_t k, int32_t* idx_out, uint32_t wait_limit_ns, void* ws,
                            size_t ws_bytes, csa2_stream_t stream) {
  CSA2_TRY(check_shape(shape));
  const csa2_shape& s = *shape;
  CSA2_TRY(check_ws(s, ws, ws_bytes));
  if (q_idx == nullptr || w == nullptr || k_idx == nullptr || n_valid == nullptr || idx_out == nullptr || k < 1 ||
      k > s.topk)
    return CSA2_ERR_INVALID_ARG;
  if (wait_limit_ns < 1000u || wait_limit_ns > 100000000u) return CSA2_ERR_INVALID_ARG;
  if (!indexer_fast(s) || !index_select_supported(false, s.n_entries) || !aligned16(k_idx))
    return CSA2_ERR_UNSUPPORTED;
  const WsLayout L = layout(s);
  SelectArgs a = select_args(s, k_idx, s.n_entries, seqdiv(s), q_idx, w, n_valid, 1, k, idx_out, k, nullptr,
                             at<int>(ws, L.hdr));
  a.wait_ns = wait_limit_ns;
  a.skip_first_copy = 1;
  return cuda_status(launch_index_select(a, false, s.batch, s.n_entries, stream));
}

int csa2_debug_kv4_wait_timeout(const csa2_shape* shape, const void* q, const void* kv4, const int32_t* idx, const void* k_swa,
                                const void* v_swa, const int32_t* n_swa, void* out, float* lse, int32_t k_exp, int32_t v_exp,
                                uint32_t wait_limit_cycles, void* ws, size_t ws_bytes, csa2_stream_t stream) {
  Kv4AttnArgs a{};
  CSA2_TRY(kv4_attn_args(shape, q, kv4, idx, k_swa, v_swa, n_swa, out, lse, k_exp, v_exp, ws, ws_bytes, a));
  if (wait_limit_cycles < 10000u || wait_limit_cycles > 200000000u) return CSA2_ERR_INVALID_ARG;
  if (!attn_fast(*shape)) return CSA2_ERR_UNSUPPORTED;
  a.wait_cycles = wait_limit_cycles;
  a.never = 1;
  return cuda_status(launch_kv4_attn(a, true, shape->batch, stream));
}

int csa2_fast_path(const csa2_shape* shape, int32_t* indexer_fast_out, int32_t* attention_fast_out) {
  if (check_shape(shape) != CSA2_OK) return 0;
  const int ix = indexer_fast(*shape) ? 1 : 0;
  const int at_ = attn_fast(*shape) ? 1 : 0;
  if (indexer_fast_out != nullptr) *indexer_fast_out = ix;
  if (attention_fast_out != nullptr) *attention_fast_out = at_;
  return ix && at_;
}

}  // extern "C"
