// lla_q4.h — the 4-bit latent row shared by the kernels that write it (lla_q4.cu) and
// the ones that attend over it (lla_q4.cu, lla_q4_decode.cu).
//
// A row holds one token of one head, K and V together, so that one bulk copy per page
// brings a whole head-tile:
//   [0, r_k/2)           K codes, 8 columns per 32-bit word
//   [r_k/2, (r_k+r_v)/2) V codes
//   then bf16 scales, one per 32 columns of K, then of V; zero padding to 16 bytes.
// Column c of a word (c < 8) sits at bit 4(c/2) + 16(c mod 2) as code + 8: a word's two
// halves hold its even and its odd columns, so one mask yields a pair of neighbouring
// columns as two half-words.  Value = code * scale, code in [-7, 7].
#pragma once

#include "lla_kernels.h"

namespace lla {

constexpr int kQ4Group = 32;          // columns that share a scale
constexpr int kQ4CombineUnits = 4;    // most sequences of a combine block
constexpr int kQ4PrepSeqs = 4;        // sequences of a block that forms query operands

__host__ __device__ inline int q4_groups(int r) { return (r + kQ4Group - 1) / kQ4Group; }
__host__ __device__ inline int q4_scale_offset(int r_k, int r_v) { return (r_k + r_v) / 2; }
__host__ __device__ inline int q4_row_bytes(int r_k, int r_v) {
  return ((r_k + r_v) / 2 + 2 * (q4_groups(r_k) + q4_groups(r_v)) + 15) / 16 * 16;
}

// Shared-memory plan of the tensor-core decode kernel (byte offsets from a 1024-aligned base).
struct Q4Plan {
  int nh, ngroups;                   // heads of a group (1, 2, 4 or 8), groups of a sequence
  int NS, NR;                        // stages of head-tiles, chunks (half tiles) of rotary rows
  int PG, PB, gstep;                 // positions with G in TMEM, their barriers, columns apart
  int N;                             // rows of a head's query operand = columns of G: r_k + 2 (1 + scale groups of 32), in 16s
  int z, z_chunk;                    // query operands of the group's heads: two chunks of coordinates
  int rows;                          // rotary tiles
  int state, misc, ring, stage;      // softmax state of the epilogue; barriers; head-tiles
  int w_bytes;                       // V weights of a stage
  int bytes;                         // total dynamic smem incl. alignment slack
};
// False where no plan fits (never for ranks up to kMaxRankPerHead).
bool make_q4_plan(int H, int r_k, int r_v, Q4Plan* p);
// Floats of a record of one head: 8 (m, l), 8 references (m, E), 8 / nh sums of r_v (even, so that records
// are 8-byte aligned).
inline int q4_record_floats(int nh, int r_v) { return 32 + 8 / nh * r_v; }

struct Q4DecodeArgs {
  int B, H, r_k, r_v, rope_style;
  int row_bytes;
  int64_t L_max, rope_len, mu_hstride;
  const void* q;                     // [B][H][128] storage dtype
  const uint8_t* rows;               // pool [num_pages][H][page_size][row_bytes]
  const int32_t* block_table;        // [B][max_pages]
  int page_size, max_pages;
  int64_t num_pages;
  const int32_t* seq_lens;           // [B]
  const int32_t* q_pos;              // [B]
  const void* w_up_k;                // loop-t slice [H][128][r_k]
  const void* w_up_v;                // loop-t slice [H][128][r_v]
  const float* mu_k;                 // loop-t slice: element (h, e) at mu_k[h*mu_hstride + e]
  const float* mu_v;
  const float* rope_cos;             // [rope_len][64]
  const float* rope_sin;
  void* out;                         // [B][H][128] storage dtype
  float* lse;                        // [B][H], or nullptr
  uint32_t* status;
  float* records;                    // split records (fp32 kernel: {m (log2 units), l, -, -, acc[r_v]})
  int rec_stride;                    // tensor-core kernel: floats of a record
  int64_t chunk;                     // fp32 kernel: tokens of a split
  int splits;                        // fp32 kernel: splits of a (sequence, head)
  uint8_t* row_tiles;                // tensor-core kernel: f16 rotary rows, 32 KB per 128 positions
  uint8_t* zimg;                     // query operands of every (sequence, head group)
  float2* z_unit;                    // [B][H]: units of the folded query's f16 values, and of its bias's
  int z_blocks, rows_grid;           // blocks that form the operands, and the rotary tiles
  int32_t* ranges;                   // first and last CTA of each (sequence, head group)
  int grid;
  int combine_units;                 // sequences per combine block (1..kQ4CombineUnits)
  Q4Plan plan;
};

// Tokens per split of the fp32 kernel: enough splits for two blocks per SM, whole tiles.
int64_t q4_plain_chunk(int B, int H, int64_t L_max, int sms);
cudaError_t launch_q4_f32(const Q4DecodeArgs& a, cudaStream_t s);
cudaError_t launch_q4_tile(const Q4DecodeArgs& a, cudaStream_t s);

// Opt the kernel in to `most` bytes of dynamic shared memory on the current device: the most that any
// call takes, so that two host threads with calls of different sizes set the same; whatever
// the size, because what needs no opt-in is 48 KB less the kernel's own static part.
// Set at every launch: the attribute belongs to a device's copy of the kernel, and a
// process may use several.
template <typename K>
cudaError_t allow_smem(K* kern, size_t most) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
}

}  // namespace lla
