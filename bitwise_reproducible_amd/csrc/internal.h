// Internal interface between the C-ABI front end (api.cpp) and the kernel
// translation units.  Every launcher enqueues on `stream` and returns the
// hipError_t of the launch; argument checking is done by the front end.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "repro.h"

namespace repro {

struct ReplicaPtrs {
  const float* p[REPRO_MAX_REPLICAS];
};

// Algorithm 1 replay: the N * accum gradient buffers in mesh order.
struct ReplayPtrs {
  const float* p[REPRO_MAX_REPLAY_BUFFERS];
};

// Streaming TreeFold: one device buffer per fold level.
constexpr int kFoldSlots = REPRO_FOLD_SLOTS;
struct FoldSlotPtrs {
  float* p[kFoldSlots];
};

// Host-prepared AdamW scalars (binary32, computed under the contract).
struct AdamwScalars {
  float lr, beta1, beta2, eps, wd;
  float c1, c2, r1, r2;
};

// elementwise.hip
hipError_t launch_tree_reduce(const ReplicaPtrs& reps, int R, int64_t n, float* out, int average, float rR,
                              int variant, hipStream_t stream);
hipError_t launch_adamw(float* state, const float* grad, int64_t n, const AdamwScalars& s, int variant,
                        hipStream_t stream);
// The same update on `count` elements of separate w, m, v, g arrays.
hipError_t launch_adamw_ptrs(float* w, float* m, float* v, const float* grad, int64_t count, const AdamwScalars& s,
                             int variant, hipStream_t stream);
hipError_t launch_fp32_ops(int op, const float* a, const float* b, float* out, int64_t n, hipStream_t stream);

// replay.hip
hipError_t launch_replay(const ReplayPtrs& a, int nbuf, int dp_replicate, int dp_shard, int accum, float r_accum,
                         float r_shard, float r_rep, int64_t n, float* out, hipStream_t stream);
hipError_t launch_fold_push(const FoldSlotPtrs& sl, int t, const float* part, int64_t n, hipStream_t stream);
hipError_t launch_fold_result(const FoldSlotPtrs& sl, int pushed, int average, float r, float* out, int64_t n,
                              hipStream_t stream);

// gemm.hip
hipError_t launch_gemm(int trans_a, int trans_b, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                       const float* B, int64_t ldb, float* C, int64_t ldc, int variant, bool fused,
                       hipStream_t stream);

// optimizer.hip
struct OptHeader {  // first bytes of the grad-norm / optimizer workspace
  float norm;       // the pre-clip global norm
  float sumsq;      // the fold of the squares
  int apply;        // 1: the step applies its update
  float coef;       // clip coefficient (1: no clip)
  float c1, c2, r1, r2;
};
constexpr int64_t kOptHeaderBytes = 256;
struct NormPlan {
  static constexpr int kMaxPasses = 8;
  int passes;
  int64_t len[kMaxPasses];         // input length of each pass
  int64_t out_offset[kMaxPasses];  // workspace offset of its block sums (-1: the header)
  int64_t total_bytes;
};
struct StepRule {
  float beta1, beta2, max_norm, spike_threshold;
  int skip_steps;
};
void plan_grad_norm(int64_t n, NormPlan* plan);
hipError_t launch_grad_norm(const void* g, int dtype, int64_t n, uint8_t* ws, const NormPlan& plan, float* out2,
                            repro_step_state* st, const StepRule& rule, hipStream_t stream);
hipError_t launch_adamw_bf16(uint16_t* w, float* m, float* v, const void* g, int dtype, int64_t n, const uint8_t* ws,
                             float lr, float beta1, float beta2, float eps, float wd, hipStream_t stream);

// rope_table.hip
hipError_t launch_rope_table(const double* inv_freq, int half, int64_t start, int64_t length, float* cos, float* sin,
                             hipStream_t stream);

// heads.hip, heads_grad.hip
struct FastDiv {  // division of numbers below 2^31
  uint32_t divisor, factor;
  int32_t shift;
};
FastDiv divide_by(uint32_t d);
struct HeadSide {  // the queries' or the keys' part
  const void* x;
  const void* dy;
  void* out;
  const void* gain;
  float* dgain;
  float* partial;  // workspace: one row of dim floats per workgroup
  int64_t x_stride[3], dy_stride[3], out_stride[3];  // batch, token, head; elements
  int32_t heads;
  uint32_t items, blocks;  // (token, chunk of heads) pairs; workgroups
  FastDiv by_chunks;       // chunks of a token
};
struct HeadsArgs {
  HeadSide side[2];
  const float* cos;
  const float* sin;
  const void* positions;
  int64_t table_rows, table_stride, pos_stride[2];
  uint32_t tokens, seq;
  FastDiv by_seq;
  int32_t dim, half;                          // half: rotated pairs
  int32_t vector, mode;                       // pairs of a lane; what the sizes leave to handle
  int32_t rot_lanes, lanes, log_group;        // of a head
  int32_t pos64, gain_bf16;
  int32_t stream, stream_loads;               // stores, and loads, past the caches
  float inv_dim, eps;
};
// Fills lanes, items and blocks for `per` heads in a group; false when there
// are too many items.
bool plan_heads(HeadsArgs* a, int dtype, int per);
bool plan_heads_forward(HeadsArgs* a, int dtype);
bool plan_heads_backward(HeadsArgs* a, int dtype);
hipError_t launch_heads(const HeadsArgs& a, int dtype, bool inter, hipStream_t stream);
hipError_t launch_heads_grad(const HeadsArgs& a, int dtype, bool inter, hipStream_t stream);

// residual.hip
struct RowView {  // rows of (batch, token), the last dimension contiguous
  const void* data;
  int64_t stride[2];  // elements
};
struct ResidualArgs {
  RowView x;  // the residual stream; its sum y in the backward pass
  RowView block, gate, dy, dz;
  RowView out[3];  // y, z; dx, dblock, dgate in the backward pass (no data: not wanted)
  const void* gain;
  const void* block_gain;
  const void* channel_gate;
  float* partial[3];  // workspace: `blocks` rows of dim floats each for dgain, dblock_gain, the channel gate's
  float* sums[3];     // where they go (null: none)
  uint32_t rows, blocks;
  FastDiv by_seq;
  int32_t dim, gain_bf16, block_norm, stream;
  float inv_dim, eps, x_scale, block_scale;
};
bool plan_residual(ResidualArgs* a, bool branch);  // fills blocks; false when there are too many rows
hipError_t launch_residual(const ResidualArgs& a, int dtype, hipStream_t stream);
hipError_t launch_residual_grad(const ResidualArgs& a, int dtype, hipStream_t stream);

// loss.hip
struct Operand {  // a matrix of bf16 planes
  const uint16_t* at;
  int64_t plane, pitch;  // elements
  int64_t rows, columns;  // that there are
};
struct LossArgs {
  const void* x;
  const void* w;
  const void* labels;
  int64_t x_stride, w_stride, label_stride, ignore_index;
  int64_t tokens, vocab, k;  // k: the width, padded
  uint32_t padded_tokens;
  int32_t dim, label64;
  float z_weight;
  float* loss;
  float* lse_out;
  const float* lse_in;
  const float* dloss;
  int64_t dloss_stride;
  void* dx;
  void* dw;
  int64_t dx_stride, dw_stride;
  float2* stats;      // of each block of 128 entries, by token
  float* picked;      // the labels' logits
  float4* per_token;  // what the gradient's epilogue needs
};
struct LossLayout {
  bool bf16, direct_x, direct_w;  // rows that the products read where they lie
  bool near_w;                    // rows of a tile within 32 bits' reach
};
int64_t loss_workspace(const LossArgs& a, const LossLayout& l, bool backward);
hipError_t launch_loss(LossArgs a, const LossLayout& l, void* workspace, hipStream_t stream);
hipError_t launch_loss_grad(LossArgs a, const LossLayout& l, void* workspace, hipStream_t stream);

// grad_list.hip
struct ListTile {  // at most 64 KB of one tensor
  const void* src;
  void* dst;
  int32_t n;  // elements
  int32_t bf16;
  int32_t index, count;  // among the tensor's tiles
};
struct ListHeader {  // first bytes of the plan, on the host and on the device
  int64_t magic, bytes;
  int64_t tiles, tensors;
  int64_t first_offset, sums_offset;  // tile ranges of the tensors; tiles' sums, then tensors', then their total
  int32_t chunks;    // 1 KB chunks of a wave in a tile
  int32_t reserved;
  int64_t most;      // tiles of one tensor, at most
};
static_assert(sizeof(ListHeader) == 64 && sizeof(ListTile) == 32, "the plan's layout");
// Fills the header; false when the list is too large.
bool size_list(const int64_t* sizes, const int32_t* dtypes, int64_t count, ListHeader* h);
void fill_list(const ListHeader& h, const void* const* grads, void* const* outs, const int64_t* sizes,
               const int32_t* dtypes, void* host_plan);
hipError_t launch_list_norm(const ListHeader& h, uint8_t* plan, float max_norm, float* out3, hipStream_t stream);
hipError_t launch_list_clip(const ListHeader& h, uint8_t* plan, float max_norm, float* out3, hipStream_t stream);

// fused.hip
hipError_t launch_fp32_fma(int unit, const float* a, const float* b, const float* c, float* out, int64_t n,
                           hipStream_t stream);

// state_hash.hip
struct HashPlan {
  static constexpr int kMaxLevels = 64;
  int levels;                       // number of levels, leaves included
  int64_t count[kMaxLevels];        // nodes per level
  int64_t offset[kMaxLevels];       // byte offset of each level's digests in the workspace
  int64_t total_bytes;              // workspace bytes needed
};
void plan_state_hash(int64_t n_words, HashPlan* plan);
// Level 0 only: `ranges` runs of `count` leaves at first + r * stride; then
// the levels above.
hipError_t launch_hash_leaves(const float* words, int64_t n_words, uint8_t* workspace, const HashPlan& plan,
                              int64_t first, int64_t count, int64_t stride, int ranges, hipStream_t stream);
hipError_t launch_hash_upper(uint8_t* workspace, const HashPlan& plan, uint8_t* digest_out, hipStream_t stream);
// AdamW on [w | m | v] and the whole state hash, the update and the leaf
// level in one kernel (n a multiple of 1024, state and grad 16-byte aligned).
hipError_t launch_adamw_hash_fused(float* state, const float* grad, int64_t n, const AdamwScalars& s, uint8_t* ws,
                                   const HashPlan& plan, uint8_t* digest_out, hipStream_t stream);
hipError_t launch_state_hash(const float* words, int64_t n_words, uint8_t* workspace, const HashPlan& plan,
                             uint8_t* digest_out, hipStream_t stream);

}  // namespace repro
