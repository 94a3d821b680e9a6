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
// Us, cached and so, rows of 2048 in bfloat16: 64 MB 39.4 and 39.0, with a
// kernel behind it that reads y 39.8 and 45.1; 128 MB 92.8 and 75.2, 101.5 and
// 99.2.  64 MB of gradients with norm and gate in binary32: 87 and 94.
constexpr int64_t kStreamBytes = int64_t(128) << 20;

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
  const bool branch = p->block_norm != 0 || p->gate.data != nullptr || p->channel_gate != nullptr;
  return repro::plan_residual(a, branch) ? REPRO_OK : REPRO_EINVAL;
}

bool scalars_fine(const repro_residual_args& p) {
  return p.eps >= 0.0f && !isinf(p.eps) && isfinite(p.x_scale) && isfinite(p.block_scale);
}

int64_t part_bytes(const repro_residual_args& p, const ResidualArgs& a) {
  return ((int64_t)a.blocks * p.dim * 4 + 15) / 16 * 16;
}

// ------------------------------------------------------- the vocabulary loss

constexpr int64_t kMostTokens = int64_t(1) << 22, kMostVocab = int64_t(1) << 24;
constexpr int32_t kMostWidth = 65536;

// Rows closer together are within 32 bits' reach of a tile's first.
constexpr int64_t kNear = int64_t(1) << 22;

// Rows that the products read where they lie.
bool direct(const void* rows, int64_t stride, const repro_vocab_args& p) {
  return p.dtype == REPRO_BF16 && p.dim % 64 == 0 && aligned(rows, 16) && stride % 8 == 0 && stride < kNear;
}

int sizes_of(const repro_vocab_args* p, repro::LossArgs* a, repro::LossLayout* l) {
  if (p == nullptr || p->tokens < 0 || p->tokens > kMostTokens || p->vocab < 1 || p->vocab > kMostVocab)
    return REPRO_EINVAL;
  if (p->dim < 1 || p->dim > kMostWidth || !is_dtype(p->dtype)) return REPRO_EINVAL;
  *a = {};
  a->tokens = p->tokens;
  a->vocab = p->vocab;
  a->dim = p->dim;
  *l = {p->dtype == REPRO_BF16, direct(p->x, p->x_stride, *p), direct(p->weight, p->weight_stride, *p),
        p->weight_stride < kNear};
  return REPRO_OK;
}

struct Vocab {
  View read[6], written[4];
  int ins = 0, outs = 0;

  // `count` runs of `run` bytes, `apart` bytes apart, each at least `run` for
  // an output.
  int take(const void* at, int64_t count, int64_t run, int64_t apart, uintptr_t align, bool output) {
    if (count == 0) return REPRO_OK;
    if (at == nullptr || apart < (output ? run : 0)) return REPRO_EINVAL;
    if (!aligned(at, align)) return REPRO_EALIGN;
    View v(at, run);
    v.dimension(count, apart);
    (output ? written[outs++] : read[ins++]) = v;
    return REPRO_OK;
  }
  bool apart() const {
    for (int i = 0; i < outs; ++i) {
      for (int j = 0; j < i; ++j)
        if (repro::share_memory(written[i], written[j])) return false;
      for (int j = 0; j < ins; ++j)
        if (repro::share_memory(written[i], read[j])) return false;
    }
    return true;
  }
};

// A stride in elements, as bytes; -1 when the rows leave 2^60.
int64_t bytes_apart(int64_t stride, int64_t count, int64_t size) {
  int64_t reach;
  if (stride < 0 || __builtin_mul_overflow(stride, (count > 1 ? count : 1) * size, &reach) ||
      reach > (int64_t(1) << 60))
    return -1;
  return stride * size;
}

int vocab_checked(const repro_vocab_args* args, bool backward, void* workspace, int64_t ws_bytes, void* stream) {
  repro::LossArgs a;
  repro::LossLayout l;
  const int st = sizes_of(args, &a, &l);
  if (st != REPRO_OK) return st;
  const repro_vocab_args& p = *args;
  if (!isfinite(p.z_weight) || (p.label_bytes != 4 && p.label_bytes != 8)) return REPRO_EINVAL;
  const int64_t size = (int64_t)size_of(p.dtype), run = p.dim * size;
  Vocab v;
  const auto rows = [&](const void* at, int64_t count, int64_t stride, bool output) {
    if (count > 0 && (stride < p.dim || bytes_apart(stride, count, size) < 0)) return REPRO_EINVAL;
    return v.take(at, count, run, stride * size, (uintptr_t)size, output);
  };
  const auto numbers = [&](const void* at, int64_t stride, int64_t bytes, bool output) {
    if (bytes_apart(stride, p.tokens, bytes) < 0) return REPRO_EINVAL;
    return v.take(at, p.tokens, bytes, stride * bytes, (uintptr_t)bytes, output);
  };
  int status = rows(p.x, p.tokens, p.x_stride, false);
  // Without tokens the embedding is not read.
  if (status == REPRO_OK) status = rows(p.weight, p.tokens > 0 ? p.vocab : 0, p.weight_stride, false);
  if (status == REPRO_OK) status = numbers(p.labels, p.label_stride, p.label_bytes, false);
  if (status == REPRO_OK) status = numbers(p.lse, 1, 4, !backward);
  if (!backward) {
    if (status == REPRO_OK) status = numbers(p.loss, 1, 4, true);
  } else {
    if (status == REPRO_OK) status = numbers(p.dloss, p.dloss_stride, 4, false);
    if (status == REPRO_OK) status = rows(p.dx, p.tokens, p.dx_stride, true);
    if (status == REPRO_OK) status = rows(p.dweight, p.vocab, p.dweight_stride, true);
  }
  if (status != REPRO_OK) return status;
  const int64_t need = repro::loss_workspace(a, l, backward);
  if (need > 0) {
    if (workspace == nullptr) return REPRO_EINVAL;
    if (!aligned(workspace, 256)) return REPRO_EALIGN;
    if (ws_bytes < need) return REPRO_ESPACE;
    v.written[v.outs++] = View(workspace, need);
  }
  if (!v.apart()) return REPRO_EINVAL;
  a.x = p.x;
  a.w = p.weight;
  a.labels = p.labels;
  a.x_stride = p.x_stride;
  a.w_stride = p.weight_stride;
  a.label_stride = p.label_stride;
  a.ignore_index = p.ignore_index;
  a.label64 = p.label_bytes == 8;
  a.z_weight = p.z_weight;
  a.loss = p.loss;
  a.lse_out = p.lse;
  a.lse_in = p.lse;
  a.dloss = p.dloss;
  a.dloss_stride = p.dloss_stride;
  a.dx = p.dx;
  a.dw = p.dweight;
  a.dx_stride = p.dx_stride;
  a.dw_stride = p.dweight_stride;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return status_of(backward ? repro::launch_loss_grad(a, l, workspace, s) : repro::launch_loss(a, l, workspace, s));
}

int64_t vocab_workspace(const repro_vocab_args* args, bool backward) {
  repro::LossArgs a;
  repro::LossLayout l;
  const int st = sizes_of(args, &a, &l);
  return st != REPRO_OK ? st : repro::loss_workspace(a, l, backward);
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

int64_t repro_vocab_loss_workspace_bytes(const repro_vocab_args* args) { return vocab_workspace(args, false); }

int repro_vocab_loss(const repro_vocab_args* args, void* workspace, int64_t ws_bytes, void* stream) {
  return vocab_checked(args, false, workspace, ws_bytes, stream);
}

int64_t repro_vocab_loss_backward_workspace_bytes(const repro_vocab_args* args) {
  return vocab_workspace(args, true);
}

int repro_vocab_loss_backward(const repro_vocab_args* args, void* workspace, int64_t ws_bytes, void* stream) {
  return vocab_checked(args, true, workspace, ws_bytes, stream);
}

}  // extern "C"
