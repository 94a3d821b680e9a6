// C-ABI front end of the residual stream's operators: argument checks and
// launches.  See include/repro.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "checks.h"
#include "internal.h"
#include "repro.h"
#include "views.h"

namespace {

using repro::aligned;
using repro::extent;
using repro::is_dtype;
using repro::ResidualArgs;
using repro::RowView;
using repro::size_of;
using repro::status_of;
using repro::View;

// Memory that a call reads or writes, and whether an output may be the very
// view of it.
struct Use {
  View view;
  bool rows;
};

// Bytes of one tensor from which the residual norm's stores bypass the caches.
constexpr int64_t kStreamBytes = int64_t(32) << 20;

struct Residual {
  const repro_residual_args& p;
  ResidualArgs a;
  int64_t size, sizes[2];
  Use read[16], written[8];
  int ins = 0, outs = 0;

  explicit Residual(const repro_residual_args& args) : p(args), a{}, size((int64_t)size_of(args.dtype)), sizes{} {}

  // A row tensor; checked unless there are no rows.
  int take(const repro_row_view& v, bool output, RowView* out) {
    out->data = v.data;
    out->stride[0] = v.batch_stride;
    out->stride[1] = v.seq_stride;
    if (a.rows == 0) return REPRO_OK;
    if (v.data == nullptr || v.batch_stride < 0 || v.seq_stride < 0) return REPRO_EINVAL;
    if (!aligned(v.data, (uintptr_t)size)) return REPRO_EALIGN;
    if (extent(sizes, out->stride, 2, p.dim) < 0) return REPRO_EINVAL;
    if (output && !repro::distinct(sizes, out->stride, p.dim, 2)) return REPRO_EINVAL;
    View view(v.data, p.dim * size);
    for (int d = 0; d < 2; ++d) view.dimension(sizes[d], sizes[d] > 1 ? out->stride[d] * size : 0);
    (output ? written[outs++] : read[ins++]) = {view, true};
    return REPRO_OK;
  }

  // A vector of dim elements for the channels, or null.
  int channels(const void* v, const void** out) {
    *out = v;
    if (v == nullptr) return REPRO_OK;
    if (!is_dtype(p.gain_dtype)) return REPRO_EINVAL;
    if (!aligned(v, size_of(p.gain_dtype))) return REPRO_EALIGN;
    read[ins++] = {View(v, p.dim * (int64_t)size_of(p.gain_dtype)), false};
    return REPRO_OK;
  }

  // The gradient of such a vector.
  int gathered(const void* of, float* v, int n) {
    if (of == nullptr) return REPRO_OK;
    if (v == nullptr) return REPRO_EINVAL;
    if (!aligned(v, 4)) return REPRO_EALIGN;
    a.sums[n] = v;
    written[outs++] = {View(v, p.dim * int64_t(4)), false};
    return REPRO_OK;
  }

  bool apart() const {
    for (int i = 0; i < outs; ++i) {
      for (int j = 0; j < i; ++j)
        if (repro::share_memory(written[i].view, written[j].view)) return false;
      for (int j = 0; j < ins; ++j)
        if (repro::share_memory(written[i].view, read[j].view) &&
            !(written[i].rows && read[j].rows && repro::same_view(written[i].view, read[j].view)))
          return false;
    }
    return true;
  }
};

// The checks that sizes alone decide, and the launch plan.
int plan_of(const repro_residual_args* p, ResidualArgs* a) {
  if (p == nullptr || p->batch < 0 || p->seq < 0 || p->dim < 1 || p->dim > REPRO_MAX_WIDTH) return REPRO_EINVAL;
  if (!is_dtype(p->dtype) || (p->block_norm != 0 && p->block_norm != 1) || p->reserved != 0) return REPRO_EINVAL;
  int64_t rows;
  if (__builtin_mul_overflow(p->batch, p->seq, &rows) || rows > 0x7fffffff || p->seq > 0x7fffffff)
    return REPRO_EINVAL;
  if (p->gate.data != nullptr && p->channel_gate != nullptr) return REPRO_EINVAL;
  if (p->block_gain != nullptr && p->block_norm == 0) return REPRO_EINVAL;
  a->rows = (uint32_t)rows;
  a->by_seq = repro::divide_by(p->seq > 0 ? (uint32_t)p->seq : 1);
  a->dim = p->dim;
  a->gain_bf16 = p->gain_dtype == REPRO_BF16;
  a->block_norm = p->block_norm;
  a->inv_dim = 1.0f / (float)p->dim;
  a->eps = p->eps;
  a->x_scale = p->x_scale;
  a->block_scale = p->block_scale;
  a->stream = rows * p->dim * (int64_t)size_of(p->dtype) >= kStreamBytes;
  return repro::plan_residual(a) ? REPRO_OK : REPRO_EINVAL;
}

bool scalars_fine(const repro_residual_args& p) {
  return p.eps >= 0.0f && !isinf(p.eps) && isfinite(p.x_scale) && isfinite(p.block_scale);
}

int64_t part_bytes(const repro_residual_args& p, const ResidualArgs& a) {
  return ((int64_t)a.blocks * p.dim * 4 + 15) / 16 * 16;
}

}  // namespace

#define CHECK(call)                         \
  do {                                      \
    const int status_ = (call);             \
    if (status_ != REPRO_OK) return status_; \
  } while (0)

extern "C" {

int repro_residual_norm(const repro_residual_args* args, void* stream) {
  if (args == nullptr) return REPRO_EINVAL;
  const repro_residual_args& p = *args;
  Residual c(p);
  CHECK(plan_of(args, &c.a));
  if (!scalars_fine(p)) return REPRO_EINVAL;
  c.sizes[0] = p.batch;
  c.sizes[1] = p.seq;
  CHECK(c.take(p.x, false, &c.a.x));
  CHECK(c.take(p.z, true, &c.a.out[1]));
  if (p.block.data != nullptr) {
    CHECK(c.take(p.block, false, &c.a.block));
    CHECK(c.take(p.y, true, &c.a.out[0]));
    if (p.gate.data != nullptr) CHECK(c.take(p.gate, false, &c.a.gate));
  } else if (c.a.rows > 0 && (p.gate.data != nullptr || p.channel_gate != nullptr || p.block_norm != 0 ||
                              p.y.data != nullptr || p.x_scale != 1.0f || p.block_scale != 1.0f)) {
    return REPRO_EINVAL;
  }
  CHECK(c.channels(p.gain, &c.a.gain));
  CHECK(c.channels(p.block_gain, &c.a.block_gain));
  CHECK(c.channels(p.channel_gate, &c.a.channel_gate));
  if (!c.apart()) return REPRO_EINVAL;
  return status_of(repro::launch_residual(c.a, p.dtype, static_cast<hipStream_t>(stream)));
}

int64_t repro_residual_workspace_bytes(const repro_residual_args* args) {
  ResidualArgs a = {};
  CHECK(plan_of(args, &a));
  return part_bytes(*args, a) *
         ((args->gain != nullptr) + (args->block_gain != nullptr) + (args->channel_gate != nullptr));
}

int repro_residual_norm_backward(const repro_residual_args* args, void* workspace, int64_t ws_bytes, void* stream) {
  if (args == nullptr) return REPRO_EINVAL;
  const repro_residual_args& p = *args;
  Residual c(p);
  CHECK(plan_of(args, &c.a));
  if (!scalars_fine(p)) return REPRO_EINVAL;
  c.sizes[0] = p.batch;
  c.sizes[1] = p.seq;
  CHECK(c.take(p.y, false, &c.a.x));
  CHECK(c.take(p.dz, false, &c.a.dz));
  if (p.dy.data != nullptr) CHECK(c.take(p.dy, false, &c.a.dy));
  CHECK(c.take(p.dx, true, &c.a.out[0]));
  const bool gated = p.gate.data != nullptr || p.channel_gate != nullptr;
  if (gated || p.block_norm != 0) {
    CHECK(c.take(p.block, false, &c.a.block));
    CHECK(c.take(p.dblock, true, &c.a.out[1]));
    if (p.gate.data != nullptr) {
      CHECK(c.take(p.gate, false, &c.a.gate));
      CHECK(c.take(p.dgate, true, &c.a.out[2]));
    }
  } else if (p.dblock.data != nullptr) {
    CHECK(c.take(p.dblock, true, &c.a.out[1]));
  }
  CHECK(c.channels(p.gain, &c.a.gain));
  CHECK(c.channels(p.block_gain, &c.a.block_gain));
  CHECK(c.channels(p.channel_gate, &c.a.channel_gate));
  CHECK(c.gathered(p.gain, p.dgain, 0));
  CHECK(c.gathered(p.block_gain, p.dblock_gain, 1));
  CHECK(c.gathered(p.channel_gate, p.dchannel_gate, 2));
  const int64_t part = part_bytes(p, c.a);
  int64_t need = 0;
  for (int n = 0; n < 3; ++n) {
    if (c.a.sums[n] == nullptr) continue;
    c.a.partial[n] = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + need);
    need += part;
  }
  if (need > 0) {
    if (workspace == nullptr) return REPRO_EINVAL;
    if (!aligned(workspace, 16)) return REPRO_EALIGN;
    if (ws_bytes < need) return REPRO_ESPACE;
    c.written[c.outs++] = {View(workspace, need), false};
  }
  if (!c.apart()) return REPRO_EINVAL;
  return status_of(repro::launch_residual_grad(c.a, p.dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
