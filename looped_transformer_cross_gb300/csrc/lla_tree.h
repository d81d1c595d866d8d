// lla_tree.h — parameter block and launchers of the attention over drafted trees
// (lla_tree_attn), shared by lla_tree.cu (entry points, plain and finish kernels) and
// lla_tree_tc.cu (tensor-core kernel).
#pragma once

#include "lla_kernels.h"

namespace lla {

constexpr int kTreeMaxNodes = LLA_TREE_MAX_NODES;
constexpr int kTreeHead = 8;            // a record row: {reference, up to four sums, -, -, -, acc[r_v]}
constexpr int kTreePlainRows = 32;      // nodes of a plain block
constexpr int kTreePlainTile = 32;      // cached tokens it takes at a time

// Shared-memory and TMEM plan of the tensor-core kernel (byte offsets from a 1024-aligned base).
struct TreePlan {
  ChunkPlan kplan, vplan;            // K latents and W (64/32/16 wide); V latents (32 wide)
  int SK, SV, k_stage, v_stage;      // rings of K and V tiles
  int blocks;                        // blocks of 128 V columns
  int v_ring, k_ring, w, q, p, ones, mu, refs, base, chunks, misc, bytes;
};

struct TreeMaps {
  CUtensorMap k[3];                  // K latents, boxes 64 / 32 / 16 wide
  CUtensorMap v;                     // V latents, boxes 32 wide
  CUtensorMap v4;                    // the same as (32, row, chunk, ..), a box all of a tile's or page's chunks
  CUtensorMap w[3];                  // W_up,k of the loop as (r_k, pair, member, head), boxes 64 / 32 / 16 wide
};

struct TreeArgs {
  int B, H, r_k, r_v, rope_style, n_tok, max_nodes;
  int64_t L_max, rope_len, mu_hstride;
  const int32_t* tok_start;          // [B + 1]
  const int32_t* parent;             // [n_tok]
  const int32_t* pos;                // [n_tok]
  const void* q;                     // element (n, h, e) at n * stride + h * 128 + e
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* seq_lens;           // [B]
  const void* cache_k;               // dense [B][H][L_max][r] or pools [num_pages][H][page_size][r]
  const void* cache_v;
  const int32_t* block_table;        // [B][max_pages], or nullptr (dense)
  int page_size, max_pages;
  int piece;                         // tokens of a tile that lie in one page wherever it starts: the largest power
                                     // of two that divides page_size, at most 128
  int64_t num_pages;
  const void* w_up_k;                // loop-t slice [H][128][r_k]
  const void* w_up_v;                // loop-t slice [H][128][r_v]
  const float* mu_k;                 // loop-t slice: element (h, e) at h * mu_hstride + e
  const float* mu_v;
  const float* rope_cos;             // [rope_len][64]
  const float* rope_sin;
  void* out;                         // [n_tok][H][128]
  float* lse;                        // [n_tok][H] or nullptr
  uint32_t* status;
  // Partial results of the cached tokens: a record holds rec_rows rows of {m, l's, acc[r_v]}, acc and
  // l relative to 2^m.  Plain kernel: record (b H + h) * splits + s covers tokens s * chunk ..
  float* records;
  int rec_rows, splits, finish_rows;
  int64_t chunk;                     // cached tokens of a split, a multiple of kTreePlainTile
  float* w_turned;                   // plain kernel: [H][r_k][128]
  float* v_turned;                   // finish kernel: [H][r_v][128]
  // Tensor-core kernel (groups > 0): a unit is (b H + h) * groups + block of `group` nodes, and record
  // unit + CTA belongs to every (unit, CTA) that share a tile
  int v_whole;                       // r_v a multiple of 32: V by maps.v4
  int group, groups, rows, grid;     // nodes of a block, blocks a sequence may have, nodes S has room for, CTAs
  int32_t* tile_start;               // [B + 1]: tiles of one head before sequence b
  int4* cta_start;                   // [grid]: first (sequence, head, tile), number of tiles
  uint8_t* qimg;                     // [units][rows * 512] query operands, rows scaled by powers of two
  float* qback;                      // [units][rows] what undoes that
  uint8_t* khat;                     // [B H][max_nodes][512] rotated keys of the nodes, scaled likewise
  float* kback;                      // [B H][max_nodes]
  uint4* paths;                      // [B][max_nodes] nodes on each node's path, as bits
  uint8_t* bias;                     // [H][4096] mu operands
  float2* head_top;                  // [H] largest row sum of |W_up,k|, largest |mu_k|
  float* unit_top;                   // [B H] the size of its K latents: the quartile of some tokens' largest values
  TreePlan plan;
};

// Nodes of sequence b: its first entry, and how many (0 for entries that do not describe a
// sequence, which `flag` records).
__device__ __forceinline__ int tree_nodes(const TreeArgs& a, int b, int& first, bool flag) {
  const int s0 = __ldg(a.tok_start + b), s1 = __ldg(a.tok_start + b + 1);
  first = s0;
  if (s0 < 0 || s1 < s0 || s1 > a.n_tok || s1 - s0 > a.max_nodes) {
    if (flag) record_status(a.status, LLA_ERR_DEVICE_ARG);
    return 0;
  }
  return s1 - s0;
}

// Cached tokens of sequence b, clamped to what the cache can hold.
__device__ __forceinline__ int tree_cached(const TreeArgs& a, int b, bool flag) {
  const int L = __ldg(a.seq_lens + b);
  if (flag && (L < 0 || L > a.L_max)) record_status(a.status, LLA_ERR_DEVICE_ARG);
  return L < 0 ? 0 : (L > a.L_max ? static_cast<int>(a.L_max) : L);
}

// The most nodes of a unit (TMEM has 192 columns left for the sums of 64 nodes, 16 of them for the weights'), and the nodes that S has room
// for in calls of up to max_nodes a sequence.
inline int tree_group(int r_v) { return r_v <= 176 ? 64 : 32; }
inline int tree_rows(int max_nodes, int r_v) { return max_nodes <= 16 ? 16 : max_nodes <= 32 ? 32 : tree_group(r_v); }
// False where the operands do not fit in shared memory.
bool make_tree_plan(int r_k, int r_v, int rows, TreePlan* p);
cudaError_t launch_tree_tensor(const TreeArgs& a, const TreeMaps& maps, cudaStream_t s);
cudaError_t launch_tree_plain(const TreeArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_tree_finish(const TreeArgs& a, bool bf16, cudaStream_t s);

}  // namespace lla
