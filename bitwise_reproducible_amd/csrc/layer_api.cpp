// C-ABI front end of the operators around one attention layer and one
// optimizer step: argument checks and launches.  See include/repro.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "checks.h"
#include "internal.h"
#include "repro.h"
#include "views.h"

namespace {

using repro::aligned;
using repro::distinct;
using repro::extent;
using repro::is_dtype;
using repro::size_of;
using repro::status_of;
using repro::HeadsArgs;
using repro::HeadSide;
using repro::ListHeader;
using repro::View;

int check_view(const repro_head_view& v, const int64_t* sizes, int64_t dim, int32_t dtype, bool output,
               int64_t* strides) {
  strides[0] = v.batch_stride;
  strides[1] = v.seq_stride;
  strides[2] = v.head_stride;
  if (sizes[0] == 0 || sizes[1] == 0 || sizes[2] == 0) return REPRO_OK;
  if (v.data == nullptr || strides[0] < 0 || strides[1] < 0 || strides[2] < 0) return REPRO_EINVAL;
  if (!aligned(v.data, size_of(dtype))) return REPRO_EALIGN;
  if (extent(sizes, strides, 3, dim) < 0) return REPRO_EINVAL;
  if (output && !distinct(sizes, strides, dim)) return REPRO_EINVAL;
  return REPRO_OK;
}

// A side's tensor, whose sizes and strides have been checked.
View view_of(const repro_head_view& v, const int64_t* sizes, int64_t dim, int64_t size) {
  View out(v.data, dim * size);
  const int64_t strides[3] = {v.batch_stride, v.seq_stride, v.head_stride};
  for (int d = 0; d < 3; ++d) out.dimension(sizes[d], sizes[d] > 1 ? strides[d] * size : 0);
  return out;
}

// Memory that a call uses.  An output may be the very view of an input of its
// tag, in place; no other use may share memory with an output.
struct Use {
  View view;
  int tag;
};
enum { kHeads = 0, kGain = 2, kOther = 4 };  // and the side

bool outputs_apart(const repro_qk_args& p, const HeadsArgs& a, bool backward, bool work, int64_t workspace_bytes) {
  Use written[5], read[9];
  int outs = 0, ins = 0;
  const int64_t size = (int64_t)size_of(p.dtype);
  for (int k = 0; k < 2; ++k) {
    const int64_t sizes[3] = {p.batch, p.seq, p.heads[k]};
    written[outs++] = {view_of(p.out[k], sizes, p.dim, size), kHeads + k};
    read[ins++] = {view_of(p.x[k], sizes, p.dim, size), kHeads + k};
    if (backward) read[ins++] = {view_of(p.dy[k], sizes, p.dim, size), kHeads + k};
    if (p.gain[k] == nullptr) continue;
    read[ins++] = {View(p.gain[k], p.dim * (int64_t)size_of(p.gain_dtype)), kGain + k};
    if (backward) written[outs++] = {View(p.dgain[k], p.dim * int64_t(4)), kGain + k};
  }
  if (workspace_bytes > 0) written[outs++] = {View(a.side[0].partial, workspace_bytes), kOther};
  if (work) {
    for (const float* table : {p.cos, p.sin}) {
      View v(table, a.half * int64_t(4));
      v.dimension(p.table_rows, p.table_rows > 1 ? p.table_stride * 4 : 0);
      read[ins++] = {v, kOther};
    }
    if (p.positions != nullptr) {
      View v(p.positions, p.position_bytes);
      v.dimension(p.batch, p.batch > 1 ? p.position_batch_stride * p.position_bytes : 0);
      v.dimension(p.seq, p.seq > 1 ? p.position_seq_stride * p.position_bytes : 0);
      read[ins++] = {v, kOther};
    }
  }
  for (int i = 0; i < outs; ++i) {
    const Use& out = written[i];
    for (int j = 0; j < i; ++j)
      if (repro::share_memory(out.view, written[j].view)) return false;
    for (int j = 0; j < ins; ++j)
      if (repro::share_memory(out.view, read[j].view) &&
          (out.tag == kOther || out.tag != read[j].tag || !repro::same_view(out.view, read[j].view)))
        return false;
  }
  return true;
}

// Bytes of one tensor pair from which the heads' data bypasses the caches, in
// both directions.  The backward pass gains from it there; the forward pass
// alone too, but with a reader of its results it loses up to some 2 us between
// 32 MB and 60-80 MB.
// Measured, us a call cached and past the caches, heads of 128 in bf16: 20 MB
// forward 9.1 and 8.3, backward 12.1 and 13.6; 40 MB 17.3 and 15.4, 29.1 and
// 26.6; 80 MB 35.5 and 30.5, 52.9 and 47.7.  With a kernel after it that reads
// the results: 20 MB 16.9 and 17.0, 19.9 and 22.8; 40 MB 30.5 and 32.2, 41.8
// and 41.6; 80 MB 62.9 and 59.8, 83.8 and 74.8.
constexpr int64_t kStreamBytes = int64_t(32) << 20;

// The part of the checks that sizes alone decide, and the launch plan.
int plan_of(const repro_qk_args* p, bool backward, HeadsArgs* a) {
  if (p == nullptr || p->batch < 0 || p->seq < 0 || p->heads[0] < 0 || p->heads[1] < 0) return REPRO_EINVAL;
  if (p->dim < 2 || p->dim > REPRO_MAX_HEAD_DIM || p->dim % 2 != 0) return REPRO_EINVAL;
  if (p->rotary < 2 || p->rotary > p->dim || p->rotary % 2 != 0) return REPRO_EINVAL;
  if (!is_dtype(p->dtype) || (p->interleaved != 0 && p->interleaved != 1) || p->reserved != 0) return REPRO_EINVAL;
  int64_t tokens;
  if (__builtin_mul_overflow(p->batch, p->seq, &tokens) || tokens > 0x7fffffff || p->seq > 0x7fffffff)
    return REPRO_EINVAL;
  *a = {};
  a->tokens = (uint32_t)tokens;
  a->seq = (uint32_t)p->seq;
  a->dim = p->dim;
  a->half = p->rotary / 2;
  a->inv_dim = 1.0f / (float)p->dim;
  a->eps = p->eps;
  for (int k = 0; k < 2; ++k) {
    a->side[k].heads = p->heads[k];
    a->side[k].gain = p->gain[k];
  }
  if (!(backward ? repro::plan_heads_backward(a, p->dtype) : repro::plan_heads_forward(a, p->dtype)))
    return REPRO_EINVAL;
  const int64_t heads = (int64_t)p->heads[0] + p->heads[1];
  a->stream = tokens * heads * p->dim * (int64_t)size_of(p->dtype) >= kStreamBytes;
  // A load past the caches has to use up every line that it touches: halves of
  // whole lines, each one vector's.
  a->stream_loads = a->stream && p->rotary == p->dim && p->interleaved == 0 &&
                    (int64_t)a->half * (int64_t)size_of(p->dtype) % 128 == 0;
  return REPRO_OK;
}

int64_t partial_bytes(const HeadsArgs& a, int side) {
  return a.side[side].gain == nullptr ? 0 : ((int64_t)a.side[side].blocks * a.dim * 4 + 15) / 16 * 16;
}

int heads_checked(const repro_qk_args* p, bool backward, void* workspace, int64_t ws_bytes, void* stream) {
  HeadsArgs a;
  int st = plan_of(p, backward, &a);
  if (st != REPRO_OK) return st;
  if (!(p->eps >= 0.0f) || isinf(p->eps)) return REPRO_EINVAL;
  const bool any_gain = p->gain[0] != nullptr || p->gain[1] != nullptr;
  if (any_gain && !is_dtype(p->gain_dtype)) return REPRO_EINVAL;
  a.gain_bf16 = p->gain_dtype == REPRO_BF16;
  const bool work = a.tokens > 0 && (p->heads[0] > 0 || p->heads[1] > 0);
  if (work) {
    if (p->cos == nullptr || p->sin == nullptr || p->table_rows < 0 || p->table_stride < a.half) return REPRO_EINVAL;
    if (!aligned(p->cos, 4) || !aligned(p->sin, 4)) return REPRO_EALIGN;
    if (extent(&p->table_rows, &p->table_stride, 1, a.half) < 0) return REPRO_EINVAL;
    if (p->positions == nullptr) {
      if (p->seq > p->table_rows) return REPRO_EINVAL;
    } else {
      if (p->position_bytes != 4 && p->position_bytes != 8) return REPRO_EINVAL;
      if (p->position_batch_stride < 0 || p->position_seq_stride < 0) return REPRO_EINVAL;
      if (!aligned(p->positions, (uintptr_t)p->position_bytes)) return REPRO_EALIGN;
      const int64_t sizes[2] = {p->batch, p->seq};
      const int64_t strides[2] = {p->position_batch_stride, p->position_seq_stride};
      if (extent(sizes, strides, 2, 1) < 0) return REPRO_EINVAL;
    }
  }
  a.cos = p->cos;
  a.sin = p->sin;
  a.table_rows = p->table_rows;
  a.table_stride = p->table_stride;
  a.positions = p->positions;
  a.pos_stride[0] = p->position_batch_stride;
  a.pos_stride[1] = p->position_seq_stride;
  a.pos64 = p->position_bytes == 8;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  for (int k = 0; k < 2; ++k) {
    HeadSide& side = a.side[k];
    const int64_t sizes[3] = {p->batch, p->seq, p->heads[k]};
    if ((st = check_view(p->x[k], sizes, p->dim, p->dtype, false, side.x_stride)) != REPRO_OK) return st;
    if ((st = check_view(p->out[k], sizes, p->dim, p->dtype, true, side.out_stride)) != REPRO_OK) return st;
    side.x = p->x[k].data;
    side.out = p->out[k].data;
    if (side.gain != nullptr && !aligned(side.gain, size_of(p->gain_dtype))) return REPRO_EALIGN;
    if (!backward) continue;
    if ((st = check_view(p->dy[k], sizes, p->dim, p->dtype, false, side.dy_stride)) != REPRO_OK) return st;
    side.dy = p->dy[k].data;
    if (side.gain == nullptr) continue;
    if (p->dgain[k] == nullptr) return REPRO_EINVAL;
    if (!aligned(p->dgain[k], 4)) return REPRO_EALIGN;
    side.dgain = p->dgain[k];
  }
  int64_t need = 0;
  if (backward && any_gain) {
    const int64_t first = partial_bytes(a, 0);
    need = first + partial_bytes(a, 1);
    if (need > 0) {
      if (workspace == nullptr || !aligned(workspace, 16)) return workspace == nullptr ? REPRO_EINVAL : REPRO_EALIGN;
      if (ws_bytes < need) return REPRO_ESPACE;
      a.side[0].partial = reinterpret_cast<float*>(ws);
      a.side[1].partial = reinterpret_cast<float*>(ws + first);
    }
  }
  if (!outputs_apart(*p, a, backward, work, need)) return REPRO_EINVAL;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return status_of(backward ? repro::launch_heads_grad(a, p->dtype, p->interleaved != 0, s)
                            : repro::launch_heads(a, p->dtype, p->interleaved != 0, s));
}

// The header of a plan that repro_grad_list_plan filled.
bool header_of(const void* host_plan, ListHeader* h) {
  ListHeader want = {};
  const int64_t none = 0;
  repro::size_list(&none, nullptr, 0, &want);
  memcpy(h, host_plan, sizeof(*h));
  return h->magic == want.magic;
}

int list_checked(const void* host_plan, void* device_plan, float max_norm, float* out3, bool clip, void* stream) {
  if (host_plan == nullptr || device_plan == nullptr || out3 == nullptr || isnan(max_norm)) return REPRO_EINVAL;
  if (!aligned(device_plan, 256) || !aligned(out3, 4)) return REPRO_EALIGN;
  ListHeader h;
  if (!header_of(host_plan, &h)) return REPRO_EINVAL;
  if (repro::share_memory(View(out3, 12), View(device_plan, h.bytes))) return REPRO_EINVAL;
  uint8_t* plan = static_cast<uint8_t*>(device_plan);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return status_of(clip ? repro::launch_list_clip(h, plan, max_norm, out3, s)
                        : repro::launch_list_norm(h, plan, max_norm, out3, s));
}

bool list_sizes(const int64_t* sizes, const int32_t* dtypes, int64_t count, ListHeader* h) {
  if (count < 0 || count > REPRO_MAX_LIST || (count > 0 && (sizes == nullptr || dtypes == nullptr))) return false;
  for (int64_t t = 0; t < count; ++t)
    if (sizes[t] < 0 || !is_dtype(dtypes[t])) return false;
  return repro::size_list(sizes, dtypes, count, h);
}

}  // namespace

extern "C" {

int repro_rope_table(const double* inv_freq, int32_t half, int64_t start, int64_t length, float* cos, float* sin,
                     void* stream) {
  constexpr int64_t kPositions = int64_t(1) << 31;
  if (half < 1 || half > 4096 || start < 0 || length < 0 || start > kPositions || length > kPositions - start)
    return REPRO_EINVAL;
  if (length > ((int64_t(1) << 34) - 1) / half) return REPRO_EINVAL;
  if (length == 0) return REPRO_OK;
  if (inv_freq == nullptr || cos == nullptr || sin == nullptr) return REPRO_EINVAL;
  if (!aligned(inv_freq, 8) || !aligned(cos, 4) || !aligned(sin, 4)) return REPRO_EALIGN;
  const View in(inv_freq, half * int64_t(8)), c(cos, length * half * 4), s(sin, length * half * 4);
  if (repro::share_memory(c, s) || repro::share_memory(c, in) || repro::share_memory(s, in)) return REPRO_EINVAL;
  return status_of(
      repro::launch_rope_table(inv_freq, half, start, length, cos, sin, static_cast<hipStream_t>(stream)));
}

int repro_qk_norm_rope(const repro_qk_args* args, void* stream) {
  return heads_checked(args, false, nullptr, 0, stream);
}

int64_t repro_qk_workspace_bytes(const repro_qk_args* args) {
  HeadsArgs a;
  const int st = plan_of(args, true, &a);
  return st != REPRO_OK ? st : partial_bytes(a, 0) + partial_bytes(a, 1);
}

int repro_qk_norm_rope_backward(const repro_qk_args* args, void* workspace, int64_t ws_bytes, void* stream) {
  return heads_checked(args, true, workspace, ws_bytes, stream);
}

int64_t repro_grad_list_bytes(const int64_t* sizes, const int32_t* dtypes, int64_t count) {
  ListHeader h;
  return list_sizes(sizes, dtypes, count, &h) ? h.bytes : REPRO_EINVAL;
}

int repro_grad_list_plan(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* dtypes,
                         int64_t count, void* host_plan, int64_t bytes) {
  ListHeader h;
  if (!list_sizes(sizes, dtypes, count, &h) || host_plan == nullptr || (count > 0 && grads == nullptr))
    return REPRO_EINVAL;
  if (!aligned(host_plan, 16)) return REPRO_EALIGN;
  if (bytes < h.bytes) return REPRO_ESPACE;
  for (int64_t t = 0; t < count; ++t) {
    if (sizes[t] == 0) continue;
    if (grads[t] == nullptr) return REPRO_EINVAL;
    if (!aligned(grads[t], size_of(dtypes[t]))) return REPRO_EALIGN;
    if (outs != nullptr && !aligned(outs[t], size_of(dtypes[t]))) return REPRO_EALIGN;
  }
  repro::fill_list(h, grads, outs, sizes, dtypes, host_plan);
  return REPRO_OK;
}

int repro_grad_list_norm(const void* host_plan, void* device_plan, float* out3, void* stream) {
  return list_checked(host_plan, device_plan, 0.0f, out3, false, stream);
}

int repro_clip_grad_list(const void* host_plan, void* device_plan, float max_norm, float* out3, void* stream) {
  return list_checked(host_plan, device_plan, max_norm, out3, true, stream);
}

}  // extern "C"
