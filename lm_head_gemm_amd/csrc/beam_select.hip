// Beam search's selection (fs_beam_select): the n best continuations of each
// group of beams by score[k] + l[k, v] - log sum_v e^l[k, v].
//
// The logarithm of the sum is common to a row, so the best n of a row are the
// best n logits, exactly as they are given; the fp64 scores only merge rows.
// Two launches:
//  * scan: a workgroup reads one chunk of one row once, keeping its values in
//    registers: the chunk's maximum, its sum of e^(l - maximum), and its n
//    best entries as 64-bit keys (value order, then lowest index);
//  * merge: a workgroup per group of beams joins the chunks' sums to the rows'
//    logarithms in fp64, scores the chunks' entries, and picks the n best.
//
// Both pick n of many the same way: split the values into at least n sets,
// take each set's largest, and let t be the smallest of those. At least n
// values reach t, and usually few more do (about n ln n in random order): these
// go to LDS, where each counts the ones ahead of it. If too many reach t
// (long runs of equal values), the scan finds the n-th key bit by bit and the
// merge takes the best one n times.
#include "fs_decode.h"

namespace fs {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kPiece = 8;                 // consecutive entries per thread and step
constexpr int kStep = kThreads * kPiece;  // entries per workgroup and step
constexpr int kListed = 1024;             // scan: entries that may reach the bound
constexpr int kMergeThreads = 1024;
constexpr int kMergeListed = 2048;
constexpr float kLog2e = 1.44269504088896340736f;

// Rows are read at any alignment of their elements: one 16-byte load (two for
// fp32) per piece all the same. Every row is therefore split among threads
// alike, and equal rows give equal sums to the last bit.
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));

template <bool BF16>
__device__ __forceinline__ void load_piece(const void* row, int v, int V, float (&x)[kPiece]) {
  constexpr float kNone = -__builtin_inff();
  if (v + kPiece <= V) {
    if constexpr (BF16) {
      const u32x4_t p = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4_a2*>(static_cast<const uint16_t*>(row) + v));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(p[i]);
        x[2 * i + 1] = bf16_hi(p[i]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4_t p = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_a2*>(static_cast<const float*>(row) + v + 4 * h));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * h + i] = __uint_as_float(p[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      x[i] = kNone;
      if (v + i < V)
        x[i] = BF16 ? bf16_lo(static_cast<const uint16_t*>(row)[v + i]) : static_cast<const float*>(row)[v + i];
    }
  }
#pragma unroll
  for (int i = 0; i < kPiece; ++i) x[i] = x[i] == x[i] ? x[i] + 0.0f : kNone;   // NaN: no entry; -0 is 0
}

// A value's place in the order of numbers, as an unsigned whole number.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint64_t order_of(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

template <typename T>
__device__ __forceinline__ T block_sum(T x, T* red) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) x += red[w];
  return x;
}

// A beam that is continued: in use and not finished.
__device__ __forceinline__ bool continued(const BeamSelectArgs& a, int row) {
  return a.scores[row] > -__builtin_inff() && !(a.finished && a.finished[row]);
}

template <bool BF16, int IT>
__global__ __launch_bounds__(kThreads) void beam_scan_kernel(BeamSelectArgs a) {
  __shared__ float red_f[kWaves * 64];
  __shared__ double red_d[kWaves];
  __shared__ int red_i[kWaves];
  __shared__ uint64_t list[kListed];
  __shared__ int listed;
  const int row = blockIdx.x / a.n_chunks, chunk = blockIdx.x - row * a.n_chunks;
  if (!continued(a, row)) return;   // the merge does not look at this row either
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int begin = chunk * (IT * kStep);
  const int end = min(a.V, begin + IT * kStep);
  const void* base = static_cast<const char*>(a.logits) + (int64_t)row * a.ld * (BF16 ? 2 : 4);

  float x[IT][kPiece];
#pragma unroll
  for (int it = 0; it < IT; ++it) load_piece<BF16>(base, begin + it * kStep + tid * kPiece, end, x[it]);

  float top = -__builtin_inff();
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < kPiece; ++i) top = fmaxf(top, x[it][i]);

  // sets of threads: lane mod S, S the power of two that reaches n
  int S = 4;
  while (S < a.n) S *= 2;
  float best = top;
  for (int m = 32; m >= S; m >>= 1) best = fmaxf(best, __shfl_xor(best, m));
  if (tid == 0) listed = 0;
  red_f[wave * 64 + lane] = best;
  __syncthreads();
  best = red_f[lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) best = fmaxf(best, red_f[w * 64 + lane]);
  // best: of this lane's set over the workgroup; S <= 64
  float bound = best, m = best;
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) {
    bound = fminf(bound, __shfl_xor(bound, s));
    m = fmaxf(m, __shfl_xor(m, s));
  }

  const int64_t at = (int64_t)row * a.n_chunks + chunk;
  uint64_t* out = a.cand + at * a.n;
  if (m == -__builtin_inff() || m == __builtin_inff()) {   // no entry, or a row without continuation
    if (tid < a.n) out[tid] = 0ull;
    if (tid == 0) {
      a.maxima[at] = m;
      a.sums[at] = 0.0;
    }
    return;
  }

  float s = 0.0f;
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < kPiece; ++i) s += __builtin_amdgcn_exp2f((x[it][i] - m) * kLog2e);
  const double sum = block_sum((double)s, red_d);
  if (tid == 0) {
    a.maxima[at] = m;
    a.sums[at] = sum;
  }

  // entries from the bound on
  const float least = fmaxf(bound, -__FLT_MAX__);   // -inf is no entry
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
      if (x[it][i] >= least) {
        const int k = atomicAdd(&listed, 1);
        if (k < kListed) list[k] = pack_key(x[it][i], (uint32_t)(begin + it * kStep + tid * kPiece + i));
      }
  __syncthreads();
  int c = listed;
  if (c > kListed) {
    // Too many: the n-th largest of the keys (order, entry counted from the
    // chunk's end), one bit at a time from the top. Keys are distinct, so
    // exactly n reach it (all of them if there are fewer).
    auto local = [&](int it, int i) -> uint64_t {
      const uint32_t o = x[it][i] >= -__FLT_MAX__ ? order_of(x[it][i]) : 0u;
      return o ? ((uint64_t)o << 14) | (uint64_t)(IT * kStep - 1 - (it * kStep + tid * kPiece + i)) : 0ull;
    };
    static_assert(IT * kStep <= 1 << 14, "entries of a chunk fit 14 bits");
    uint64_t t = 0ull;
    for (int bit = 45; bit >= 0; --bit) {
      const uint64_t probe = t | (1ull << bit);
      int count = 0;
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) count += local(it, i) >= probe;
      if (block_sum(count, red_i) >= a.n) t = probe;
    }
    if (tid == 0) listed = 0;
    __syncthreads();
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
      for (int i = 0; i < kPiece; ++i)
        if (local(it, i) >= t) {
          const int k = atomicAdd(&listed, 1);
          if (k < kListed) list[k] = pack_key(x[it][i], (uint32_t)(begin + it * kStep + tid * kPiece + i));
        }
    __syncthreads();
    c = min(listed, kListed);
  }
  for (int j = tid; j < c; j += kThreads) {
    const uint64_t key = list[j];
    int rank = 0;
    for (int k = 0; k < c; ++k) rank += list[k] > key;
    if (rank < a.n) out[rank] = key;
  }
  if (tid >= c && tid < a.n) out[tid] = 0ull;
}

// A scored continuation; order: higher score, then lower place k * V + v.
struct Scored {
  double score;
  int64_t place;
};
__device__ __forceinline__ bool ahead(const Scored& x, const Scored& y) {
  return x.score > y.score || (x.score == y.score && x.place < y.place);
}

__global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(BeamSelectArgs a) {
  constexpr int kMW = kMergeThreads / 64;
  __shared__ double row_score[FS_BEAM_MAX], row_max[FS_BEAM_MAX], row_log[FS_BEAM_MAX];
  __shared__ int row_state[FS_BEAM_MAX];   // 0: not in use, 1: continued, 2: finished
  __shared__ uint64_t set_best[FS_BEAM_MAX];
  __shared__ double list_score[kMergeListed];
  __shared__ int64_t list_place[kMergeListed];
  __shared__ int listed;
  const int b = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int K = a.beams, n = a.n, nc = a.n_chunks;
  constexpr double kInf = __builtin_inf();

  // each row's maximum and logarithm of the sum: a wave per row
  for (int k = wave; k < K; k += kMW) {
    const int row = b * K + k;
    const float score = a.scores[row];
    const bool in_use = score > -__builtin_inff();   // false for NaN
    const bool done = a.finished && a.finished[row];
    int state = !in_use ? 0 : done ? 2 : 1;
    double m = -kInf, s = 0.0;
    if (state == 1) {
      const float* maxima = a.maxima + (int64_t)row * nc;
      const double* sums = a.sums + (int64_t)row * nc;
      for (int c = lane; c < nc; c += 64) m = fmax(m, (double)maxima[c]);
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) m = fmax(m, __shfl_xor(m, d));
      if (m > -kInf && m < kInf)
        for (int c = lane; c < nc; c += 64)
          if (sums[c] > 0.0) s += sums[c] * exp((double)maxima[c] - m);
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d);
      if (!(m > -kInf && m < kInf)) state = 0;
    }
    if (lane == 0) {
      row_state[k] = state;
      row_score[k] = (double)score + 0.0;   // -0 is 0
      row_max[k] = m;
      row_log[k] = state == 1 ? log(s) : 0.0;
    }
  }
  if (tid == 0) listed = 0;
  if (tid < FS_BEAM_MAX) set_best[tid] = 0ull;
  __syncthreads();

  // entry j of the group: the chunks' entries row by row, then the finished beams
  const int per_row = nc * n;
  const int64_t scanned = (int64_t)K * per_row, total = scanned + K;
  const uint64_t* cand = a.cand + (int64_t)b * scanned;
  auto scored = [&](int64_t j, uint64_t key, Scored* e) -> bool {
    if (j < scanned) {
      const int k = (int)(j / per_row);
      if (row_state[k] != 1 || key == 0ull) return false;
      const uint32_t o = (uint32_t)(key >> 32);
      const double x = (double)__uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
      e->score = row_score[k] + ((x - row_max[k]) - row_log[k]);
      e->place = (int64_t)k * a.V + key_to_token(key);
      return true;
    }
    const int k = (int)(j - scanned);
    if (row_state[k] != 2) return false;
    e->score = row_score[k];
    e->place = (int64_t)k * a.V + a.pad;
    return true;
  };
  auto entry = [&](int64_t j, Scored* e) -> bool { return scored(j, j < scanned ? cand[j] : 0ull, e); };

  // The bound, from the first `ranks` entries of every chunk (about eight per
  // set at least): sets by a multiplicative hash, so that neither the rank nor
  // the beam of an entry decides its set.
  int log_s = 2;
  while ((1 << log_s) < n) ++log_s;
  const int S = 1 << log_s;
  const int64_t lists = (int64_t)K * nc;
  const int ranks = (int)min((int64_t)n, (8 * S + lists - 1) / lists);
  for (int64_t j = tid; j < lists * ranks; j += kMergeThreads) {
    const int64_t l = j / ranks;
    Scored e;
    if (entry(l * n + (j - l * ranks), &e))
      atomicMax(reinterpret_cast<unsigned long long*>(&set_best[((uint32_t)j * 2654435769u) >> (32 - log_s)]),
                (unsigned long long)order_of(e.score));
  }
  __syncthreads();
  uint64_t bound = ~0ull;
  for (int i = 0; i < S; ++i) bound = min(bound, set_best[i]);   // 0: a set without entry

  for (int64_t j = tid; j < total; j += kMergeThreads) {
    Scored e;
    if (entry(j, &e) && order_of(e.score) >= bound) {
      const int k = atomicAdd(&listed, 1);
      if (k < kMergeListed) {
        list_score[k] = e.score;
        list_place[k] = e.place;
      }
    }
  }
  __syncthreads();
  int c = listed;
  if (c > kMergeListed) {
    // too many equal scores: the best one behind the last taken, n times
    Scored last{kInf, -1};
    c = 0;
    for (int i = 0; i < n; ++i) {
      Scored mine{-kInf, INT64_MAX};
      for (int64_t j = tid; j < total; j += kMergeThreads) {
        Scored e;
        if (entry(j, &e) && (i == 0 || ahead(last, e)) && ahead(e, mine)) mine = e;
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) {
        const Scored other{__shfl_xor(mine.score, d), (int64_t)shfl_xor_u64((uint64_t)mine.place, d)};
        if (ahead(other, mine)) mine = other;
      }
      __syncthreads();   // everyone has read the previous round's result
      if (lane == 0) {
        list_score[kMergeListed - kMW + wave] = mine.score;
        list_place[kMergeListed - kMW + wave] = mine.place;
      }
      __syncthreads();
      last = Scored{-kInf, INT64_MAX};
      for (int w = 0; w < kMW; ++w) {
        const Scored other{list_score[kMergeListed - kMW + w], list_place[kMergeListed - kMW + w]};
        if (ahead(other, last)) last = other;
      }
      if (tid == 0) {
        list_score[i] = last.score;
        list_place[i] = last.place;
      }
      c = i + 1;   // more than n entries exist, so every round finds one
    }
    __syncthreads();
  }
  float* out_scores = a.out_scores + (int64_t)b * n;
  int32_t* out_parents = a.out_parents + (int64_t)b * n;
  int32_t* out_tokens = a.out_tokens + (int64_t)b * n;
  for (int j = tid; j < c; j += kMergeThreads) {
    const Scored e{list_score[j], list_place[j]};
    int rank = 0;
    for (int k = 0; k < c; ++k) rank += ahead(Scored{list_score[k], list_place[k]}, e);
    if (rank < n) {
      const int beam = (int)(e.place / a.V);
      out_scores[rank] = (float)e.score;
      out_parents[rank] = beam;
      out_tokens[rank] = (int32_t)(e.place - (int64_t)beam * a.V);
    }
  }
  if (tid >= c && tid < n) {
    out_scores[tid] = -__builtin_inff();
    out_parents[tid] = -1;
    out_tokens[tid] = -1;
  }
}

template <bool BF16>
hipError_t launch_scan(const BeamSelectArgs& a, hipStream_t stream) {
  const int64_t blocks = (int64_t)a.n_chunks * a.B * a.beams;
  if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks);
  switch (a.chunk / kStep) {
    case 1: return launch(beam_scan_kernel<BF16, 1>, grid, dim3(kThreads), 0, stream, a);
    case 2: return launch(beam_scan_kernel<BF16, 2>, grid, dim3(kThreads), 0, stream, a);
    case 4: return launch(beam_scan_kernel<BF16, 4>, grid, dim3(kThreads), 0, stream, a);
    default: return launch(beam_scan_kernel<BF16, 8>, grid, dim3(kThreads), 0, stream, a);
  }
}

}  // namespace

// Chunks of 2048 entries, doubled up to 16384 while 1024 workgroups are left.
int32_t beam_chunk(int64_t rows, int64_t V) {
  const int64_t steps = (V + kStep - 1) / kStep * rows;
  int it = 1;
  while (it < 8 && steps / (2 * it) >= 1024) it *= 2;
  return it * kStep;
}

hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t stream) {
  const hipError_t e = a.bf16 ? launch_scan<true>(a, stream) : launch_scan<false>(a, stream);
  if (e != hipSuccess) return e;
  return launch(beam_merge_kernel, dim3((unsigned)a.B), dim3(kMergeThreads), 0, stream, a);
}

}  // namespace fs
