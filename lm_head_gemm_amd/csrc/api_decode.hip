// C ABI, second part: argument validation, workspace layout and launches of
// the 8-bit head and of beam search. Nothing here allocates device memory;
// every launch goes on the caller's stream.
#include <algorithm>
#include <cmath>

#include "fs_decode.h"

namespace fs {
namespace {

constexpr int64_t kMaxRows = 0x7FFFFFFF;
constexpr int64_t kMaxTiled = 0x7FFF0000;      // rows and channels of a product: a tile's or part's end fits int32
constexpr int64_t kMaxSelectV = 0x7FFF8000;    // a chunk's end fits int32
constexpr int64_t kMaxRowBytes = 159 * 1024;   // a row held in registers by one workgroup
constexpr int64_t kMaxK = 131056;              // 2^31 / 2^14 - 1, a multiple of 16: no int32 sum overflows
constexpr int64_t kMaxLd = 1 << 24;            // row offsets within a tile of 256 rows fit 32 bits
constexpr int64_t kMaxGroups = 65536;
constexpr size_t kAlign = 256;
constexpr int32_t kSamplePart = 2048;          // smallest part of a row per sampler workgroup

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool dtype_ok(int t) { return t == FS_DTYPE_BF16 || t == FS_DTYPE_F32; }
int64_t dtype_size(int t) { return t == FS_DTYPE_BF16 ? 2 : 4; }
bool aligned(const void* p, uintptr_t n) { return (uintptr_t)p % n == 0; }

fs_status_t run(hipError_t e) { return e == hipSuccess ? FS_OK : fail_hip(e); }

// What fs_quantize_i8 and fs_rms_norm_i8 ask of their rows.
fs_status_t check_rows(const void* X, int64_t ldx, int dtype, int64_t M, int64_t D, const int8_t* codes,
                       int64_t ld_codes, const float* scales) {
  if (!X || !codes || !scales) return FS_ERR_INVALID_ARGUMENT;
  if (M <= 0 || D <= 0 || M > kMaxRows || D > kMaxRowBytes || ldx < D || ld_codes < D) return FS_ERR_INVALID_ARGUMENT;
  if (!dtype_ok(dtype)) return FS_ERR_UNSUPPORTED;
  const int64_t esz = dtype_size(dtype), piece = 16 / esz;   // codes are stored a piece at a time
  if (D * esz > kMaxRowBytes) return FS_ERR_UNSUPPORTED;
  if (!aligned(X, 16) || (D * esz) % 16 || (ldx * esz) % 16) return FS_ERR_UNSUPPORTED;
  if (!aligned(codes, piece) || ld_codes % piece || !aligned(scales, 4)) return FS_ERR_UNSUPPORTED;
  return FS_OK;
}

fs_status_t check_product(const int8_t* Q, int64_t ldq, const float* q_scales, const int8_t* W, int64_t ldw,
                          const float* w_scales, int64_t M, int64_t N, int64_t K) {
  if (!Q || !q_scales || !W || !w_scales) return FS_ERR_INVALID_ARGUMENT;
  if (M <= 0 || N <= 0 || K <= 0 || M > kMaxTiled || N > kMaxTiled || ldq < K || ldw < K) return FS_ERR_INVALID_ARGUMENT;
  if (K > kMaxK || K % 16 || ldq % 16 || ldw % 16 || ldq >= kMaxLd || ldw >= kMaxLd) return FS_ERR_UNSUPPORTED;
  if (!aligned(Q, 16) || !aligned(W, 16) || !aligned(q_scales, 4) || !aligned(w_scales, 4)) return FS_ERR_UNSUPPORTED;
  return FS_OK;
}

ProductI8Args product_args(const int8_t* Q, int64_t ldq, const float* q_scales, const int8_t* W, int64_t ldw,
                           const float* w_scales, int64_t M, int64_t N, int64_t K, void* out, int64_t ldo,
                           bool bf16) {
  ProductI8Args a{};
  a.q = Q;
  a.ldq = ldq;
  a.q_scales = q_scales;
  a.w = W;
  a.ldw = ldw;
  a.w_scales = w_scales;
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.K = (int32_t)K;
  a.out = out;
  a.ldo = ldo;
  a.out_bf16 = bf16;
  return a;
}

// Workspace of fs_sample_i8: fp32 logits [B, V rounded up to 8], then the
// sampler's partial keys.
bool sample_sizes_ok(int64_t B, int64_t D, int64_t V) {
  return B > 0 && D > 0 && V > 0 && B <= kMaxGroups && D <= kMaxK && V <= kMaxTiled;
}
int64_t sample_ld(int64_t V) { return (V + 7) / 8 * 8; }
size_t sample_logits_bytes(int64_t B, int64_t V) { return align_up((size_t)B * sample_ld(V) * sizeof(float)); }
size_t sample_bytes(int64_t B, int64_t V) {
  return sample_logits_bytes(B, V) + align_up((size_t)B * ((V + kSamplePart - 1) / kSamplePart) * sizeof(uint64_t));
}

bool select_sizes_ok(int64_t B, int64_t beams, int64_t V, int64_t n) {
  return B > 0 && B <= kMaxGroups && beams > 0 && beams <= FS_BEAM_MAX && V > 0 && V <= kMaxSelectV && n > 0 &&
         n <= FS_BEAM_MAX;
}

// Workspace of fs_beam_select: keys [rows, chunks, n], sums and maxima [rows, chunks].
struct SelectSpace {
  int32_t chunk;
  int64_t chunks;
  size_t sums, maxima, bytes;   // offsets behind the keys, and the end
};
SelectSpace select_space(int64_t B, int64_t beams, int64_t V, int64_t n, bool bf16) {
  SelectSpace s;
  const int64_t rows = B * beams;
  s.chunk = beam_chunk(rows, V, bf16);
  s.chunks = (V + s.chunk - 1) / s.chunk;
  s.sums = align_up((size_t)(rows * s.chunks * n) * sizeof(uint64_t));
  s.maxima = s.sums + align_up((size_t)(rows * s.chunks) * sizeof(double));
  s.bytes = s.maxima + align_up((size_t)(rows * s.chunks) * sizeof(float));
  return s;
}

// One level of a buffer's addresses: count steps of `stride` bytes.
struct Level {
  int64_t count, stride;
};

// A buffer's addresses, largest stride first, levels of one step left out.
// span[i]: bytes that levels i, i + 1, ... cover. False if it meets itself.
struct Levels {
  Level level[3];
  int n = 0;
  int64_t span[4];
};
bool make_levels(const fs_beam_layout_t& l, int64_t rows, Levels* out) {
  const Level all[3] = {{l.outer, l.outer_stride}, {rows, l.row_stride}, {l.blocks, l.block_stride}};
  for (const Level& x : all)
    if (x.count > 1) out->level[out->n++] = x;
  std::sort(out->level, out->level + out->n, [](const Level& x, const Level& y) { return x.stride > y.stride; });
  out->span[out->n] = l.block_bytes;
  for (int i = out->n - 1; i >= 0; --i) {
    if (out->level[i].stride < out->span[i + 1]) return false;
    out->span[i] = out->span[i + 1] + (out->level[i].count - 1) * out->level[i].stride;
  }
  return true;
}

// Whether two buffers with the same levels, the second `delta` bytes behind
// the first, share a byte. At each level at most two steps come near enough.
bool share(const Levels& l, int64_t delta, int i = 0) {
  if (delta <= -l.span[i] || delta >= l.span[i]) return false;
  if (i == l.n) return true;
  const int64_t s = l.level[i].stride, last = l.level[i].count - 1;
  const int64_t j = delta >= 0 ? delta / s : -((-delta + s - 1) / s);   // floor(delta / s)
  for (int64_t k = j; k <= j + 1; ++k)
    if (k >= -last && k <= last && share(l, delta - k * s, i + 1)) return true;
  return false;
}

struct Buffer {
  int64_t at;
  bool written;
};

// Sizes whose byte offsets stay far below 2^63.
bool layout_ok(const fs_beam_layout_t& l, int64_t rows) {
  constexpr int64_t kMost = (int64_t)1 << 48;
  auto level_ok = [](int64_t count, int64_t stride) {
    return count >= 0 && stride >= 0 && count <= kMost && (count <= 1 || stride <= kMost / (count - 1));
  };
  return level_ok(l.outer, l.outer_stride) && level_ok(rows, l.row_stride) && level_ok(l.blocks, l.block_stride) &&
         l.block_bytes >= 0 && l.block_bytes <= kMost;
}

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" {

fs_status_t fs_quantize_i8(const void* X, int64_t ldx, fs_dtype_t dtype, int64_t M, int64_t D, int8_t* codes,
                           int64_t ld_codes, float* scales, hipStream_t stream) {
  const fs_status_t st = check_rows(X, ldx, dtype, M, D, codes, ld_codes, scales);
  if (st != FS_OK) return st;
  RowsI8Args a{};
  a.x = X;
  a.ldx = ldx;
  a.codes = codes;
  a.ldc = ld_codes;
  a.scales = scales;
  a.M = (int32_t)M;
  a.D = (int32_t)D;
  return run(launch_rows_i8(a, dtype == FS_DTYPE_BF16, false, stream));
}

fs_status_t fs_rms_norm_i8(const void* X, int64_t ldx, const void* residual, int64_t ld_residual, const void* gain,
                           fs_dtype_t gain_dtype, fs_dtype_t dtype, int64_t M, int64_t D, float eps, void* sum_out,
                           int64_t ld_sum, int8_t* codes, int64_t ld_codes, float* scales, hipStream_t stream) {
  const fs_status_t st = check_rows(X, ldx, dtype, M, D, codes, ld_codes, scales);
  if (st != FS_OK) return st;
  if (!gain || !(eps >= 0.f) || !std::isfinite(eps)) return FS_ERR_INVALID_ARGUMENT;
  if ((residual != nullptr) != (sum_out != nullptr)) return FS_ERR_INVALID_ARGUMENT;
  if (residual && (ld_residual < D || ld_sum < D)) return FS_ERR_INVALID_ARGUMENT;
  if (gain_dtype != FS_DTYPE_F32 && gain_dtype != dtype) return FS_ERR_UNSUPPORTED;
  const int64_t esz = dtype_size(dtype);
  if (!aligned(gain, 16)) return FS_ERR_UNSUPPORTED;
  if (residual && (!aligned(residual, 16) || !aligned(sum_out, 16) || (ld_residual * esz) % 16 || (ld_sum * esz) % 16))
    return FS_ERR_UNSUPPORTED;
  RowsI8Args a{};
  a.x = X;
  a.ldx = ldx;
  a.residual = residual;
  a.ldr = ld_residual;
  a.gain = gain;
  a.sum = sum_out;
  a.lds = ld_sum;
  a.codes = codes;
  a.ldc = ld_codes;
  a.scales = scales;
  a.M = (int32_t)M;
  a.D = (int32_t)D;
  a.eps = eps;
  return run(launch_rows_i8(a, dtype == FS_DTYPE_BF16, gain_dtype == FS_DTYPE_BF16, stream));
}

fs_status_t fs_matmul_i8(const int8_t* Q, int64_t ldq, const float* q_scales, const int8_t* W, int64_t ldw,
                         const float* w_scales, int64_t M, int64_t N, int64_t K, void* out, int64_t ldo,
                         fs_dtype_t out_dtype, hipStream_t stream) {
  const fs_status_t st = check_product(Q, ldq, q_scales, W, ldw, w_scales, M, N, K);
  if (st != FS_OK) return st;
  if (!out || ldo < N) return FS_ERR_INVALID_ARGUMENT;
  if (!dtype_ok(out_dtype) || !aligned(out, dtype_size(out_dtype))) return FS_ERR_UNSUPPORTED;
  return run(launch_product_i8(product_args(Q, ldq, q_scales, W, ldw, w_scales, M, N, K, out, ldo,
                                            out_dtype == FS_DTYPE_BF16),
                               stream));
}

size_t fs_sample_i8_workspace_bytes(int64_t B, int64_t D, int64_t V) {
  return sample_sizes_ok(B, D, V) ? sample_bytes(B, V) : 0;
}

fs_status_t fs_sample_i8(const int8_t* Q, int64_t ldq, const float* q_scales, const int8_t* W, int64_t ldw,
                         const float* w_scales, int64_t B, int64_t D, int64_t V, float temperature, uint64_t seed,
                         uint64_t step, void* workspace, size_t workspace_bytes, int32_t* out_tokens,
                         hipStream_t stream) {
  const fs_status_t st = check_product(Q, ldq, q_scales, W, ldw, w_scales, B, V, D);
  if (st != FS_OK) return st;
  if (!workspace || !out_tokens || B > kMaxGroups) return FS_ERR_INVALID_ARGUMENT;
  if (!(temperature >= 0.f) || !std::isfinite(temperature)) return FS_ERR_INVALID_ARGUMENT;
  if (!aligned(workspace, 16)) return FS_ERR_UNSUPPORTED;
  if (workspace_bytes < sample_bytes(B, V)) return FS_ERR_WORKSPACE_TOO_SMALL;
  const int64_t ld = sample_ld(V);
  uint64_t* partial = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + sample_logits_bytes(B, V));
  hipError_t e = launch_product_i8(
      product_args(Q, ldq, q_scales, W, ldw, w_scales, B, V, D, workspace, ld, false), stream);
  if (e != hipSuccess) return fail_hip(e);
  const NoiseKey nk{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)step, (uint32_t)(step >> 32)};
  const bool greedy = temperature == 0.f;
  const float scale = greedy ? 0.f : (float)(1.0 / ((double)temperature * 0.693147180559945309417));
  int32_t n_parts = 0;
  e = launch_sample_logits(workspace, ld, 0, (int32_t)B, (int32_t)V, scale, greedy, nk, partial, &n_parts, stream);
  if (e != hipSuccess) return fail_hip(e);
  return run(launch_stage2(partial, (int32_t)B, n_parts, out_tokens, stream));
}

size_t fs_beam_select_workspace_bytes(int64_t B, int64_t beams, int64_t V, int64_t n, fs_dtype_t logits_dtype) {
  if (!select_sizes_ok(B, beams, V, n) || !dtype_ok(logits_dtype)) return 0;
  return select_space(B, beams, V, n, logits_dtype == FS_DTYPE_BF16).bytes;
}

fs_status_t fs_beam_select(const void* logits, int64_t ld_logits, fs_dtype_t logits_dtype, const float* scores,
                           const uint8_t* finished, int32_t pad_token, int64_t B, int64_t beams, int64_t V, int64_t n,
                           void* workspace, size_t workspace_bytes, float* out_scores, int32_t* out_parents,
                           int32_t* out_tokens, hipStream_t stream) {
  if (!logits || !scores || !workspace || !out_scores || !out_parents || !out_tokens) return FS_ERR_INVALID_ARGUMENT;
  if (!select_sizes_ok(B, beams, V, n) || ld_logits < V || pad_token < 0 || pad_token >= V)
    return FS_ERR_INVALID_ARGUMENT;
  if (!dtype_ok(logits_dtype) || !aligned(logits, dtype_size(logits_dtype))) return FS_ERR_UNSUPPORTED;
  if (!aligned(workspace, 16) || !aligned(scores, 4) || !aligned(out_scores, 4) || !aligned(out_parents, 4) ||
      !aligned(out_tokens, 4))
    return FS_ERR_UNSUPPORTED;
  const SelectSpace s = select_space(B, beams, V, n, logits_dtype == FS_DTYPE_BF16);
  if (workspace_bytes < s.bytes) return FS_ERR_WORKSPACE_TOO_SMALL;
  // a group's scores are read before its outputs are written; another group's may be read later
  const bool in_place = scores == out_scores && n == beams;
  if (!in_place && scores < out_scores + B * n && out_scores < scores + B * beams) return FS_ERR_INVALID_ARGUMENT;
  BeamSelectArgs a{};
  a.logits = logits;
  a.ld = ld_logits;
  a.bf16 = logits_dtype == FS_DTYPE_BF16;
  a.scores = scores;
  a.finished = finished;
  a.pad = pad_token;
  a.B = (int32_t)B;
  a.beams = (int32_t)beams;
  a.V = (int32_t)V;
  a.n = (int32_t)n;
  a.chunk = s.chunk;
  a.n_chunks = (int32_t)s.chunks;
  a.cand = static_cast<uint64_t*>(workspace);
  a.sums = reinterpret_cast<double*>(static_cast<char*>(workspace) + s.sums);
  a.maxima = reinterpret_cast<float*>(static_cast<char*>(workspace) + s.maxima);
  a.out_scores = out_scores;
  a.out_parents = out_parents;
  a.out_tokens = out_tokens;
  return run(launch_beam_select(a, stream));
}

fs_status_t fs_beam_reorder(const void* const* states, void* const* out, int64_t n_states,
                            const fs_beam_layout_t* layout, const fs_beam_layout_t* out_layout,
                            const int32_t* parents, int64_t B, int64_t beams, hipStream_t stream) {
  if (!states || !layout || !parents || (out_layout && !out)) return FS_ERR_INVALID_ARGUMENT;
  if (n_states <= 0 || n_states > FS_BEAM_MAX_STATES || B <= 0 || B > kMaxGroups || beams <= 0 || beams > FS_BEAM_MAX)
    return FS_ERR_INVALID_ARGUMENT;
  const fs_beam_layout_t from = *layout, to = out_layout ? *out_layout : from;
  if (!layout_ok(from, B * beams) || !layout_ok(to, B * beams) || from.outer != to.outer || from.blocks != to.blocks ||
      from.block_bytes != to.block_bytes)
    return FS_ERR_INVALID_ARGUMENT;
  for (int64_t i = 0; i < n_states; ++i)
    if (!states[i] || (out && !out[i])) return FS_ERR_INVALID_ARGUMENT;
  if (!aligned(parents, 4)) return FS_ERR_UNSUPPORTED;
  if (from.outer == 0 || from.blocks == 0 || from.block_bytes == 0) return FS_OK;

  Levels written, read;
  if (!make_levels(to, B * beams, &written) || !make_levels(from, B * beams, &read)) return FS_ERR_INVALID_ARGUMENT;
  const bool alike = from.outer_stride == to.outer_stride && from.row_stride == to.row_stride &&
                     from.block_stride == to.block_stride;
  void* targets[FS_BEAM_MAX_STATES];
  Buffer all[2 * FS_BEAM_MAX_STATES];
  int n_all = 0;
  for (int64_t i = 0; i < n_states; ++i) {
    targets[i] = out ? out[i] : const_cast<void*>(states[i]);
    all[n_all++] = Buffer{(int64_t)(intptr_t)targets[i], true};
    if (out) all[n_all++] = Buffer{(int64_t)(intptr_t)states[i], false};
  }
  // pairs of which one is written; in order of address, so that far ones are not looked at
  std::sort(all, all + n_all, [](const Buffer& x, const Buffer& y) { return x.at < y.at; });
  for (int i = 0; i < n_all; ++i)
    for (int j = i + 1; j < n_all; ++j) {
      const int64_t delta = all[j].at - all[i].at;
      if (delta >= std::max(written.span[0], read.span[0])) break;
      if (!all[i].written && !all[j].written) continue;
      const bool same_levels = alike || (all[i].written && all[j].written);
      const bool meet = same_levels ? share(written, delta) : delta < (all[i].written ? written : read).span[0];
      if (meet) return FS_ERR_INVALID_ARGUMENT;
    }
  BeamReorderArgs a{};
  a.from = from;
  a.to = to;
  a.parents = parents;
  a.n_states = (int32_t)n_states;
  a.B = (int32_t)B;
  a.beams = (int32_t)beams;
  a.in_place = out == nullptr;
  return run(launch_beam_reorder(a, states, targets, stream));
}

}  // extern "C"
