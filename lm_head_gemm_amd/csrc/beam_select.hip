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
// Both pick n of many the same way: split the values into sets, take each set's
// largest, and let t be (a little below) the n-th largest of those. At least n
// values reach t, and usually few more do (of s sets, about -s ln(1 - n / s)):
// these go to LDS, where each counts the ones ahead of it. 64 sets up to n = 32,
// 256 above: the least of 64 maxima lets in 300 and more (measured, n = 64, 512
// rows of 152064 bf16: scan 343 us, with 256 sets 43). If too many reach t (long
// runs of equal values), the scan finds the n-th value bit by bit and the merge
// takes the best one n times.
//
// Bound: the scan by its vector instructions (busy 80% of the time on long
// rows: an exponential, which takes four issues, and seven others per entry),
// the merge by latency. Measured, 512 rows of 152064 bf16, groups of 8: scan 34
// us (4.6 TB/s), merge 6; 4 rows of 128256 fp32: 5 and 6 us.
#include "fs_decode.h"

namespace fs {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kPiece = 8;                 // consecutive entries per thread and step
constexpr int kStep = kThreads * kPiece;  // entries per workgroup and step
constexpr int kListed = 512;              // scan: entries that may reach the bound
constexpr int kPieces = 256;              // scan: pieces that hold such entries
constexpr int kMergeThreads = 1024;
constexpr int kMergeListed = 1024;
constexpr int kFewSets = 64, kSets = 256;
constexpr int kFewN = 32;                 // largest n for the fewer sets
constexpr int kFirst = 2;                 // merge: entries per thread fetched ahead
constexpr float kLog2e = 1.44269504088896340736f;

// Rows are read at any alignment of their elements: one 16-byte load (two for
// fp32) per piece all the same. Every row is therefore split among threads
// alike, and equal rows give equal sums to the last bit.
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));

// One piece, as it lies in memory.
template <bool BF16>
struct Piece {
  u32x4_t w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* row, int v) {
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h)
      w[h] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4_a2*>(static_cast<const char*>(row) + (int64_t)v * (BF16 ? 2 : 4) + 16 * h));
  }
  __device__ __forceinline__ void clear() {   // all -inf
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[h][i] = BF16 ? 0xFF80FF80u : 0xFF800000u;
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (BF16) return (i & 1) ? bf16_hi(w[0][i / 2]) : bf16_lo(w[0][i / 2]);
    else return __uint_as_float(w[i / 4][i % 4]);
  }
};

// The number at a place of fp32's order (pack_key's), and an fp64 number's place.
__device__ __forceinline__ float number_at(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ uint64_t order_of(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// Lane l's value from an earlier lane of its row of 16 (row_shr) or from the last
// lane of an earlier row (row_bcast); `none` where there is no such lane.
template <int CTRL>
__device__ __forceinline__ uint32_t from_lane(uint32_t x, uint32_t none) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float from_lane(float x, float none) {
  return __uint_as_float(from_lane<CTRL>(__float_as_uint(x), __float_as_uint(none)));
}
template <int CTRL>
__device__ __forceinline__ double from_lane(double x, double none) {
  const uint64_t b = (uint64_t)__double_as_longlong(x), n = (uint64_t)__double_as_longlong(none);
  const uint32_t lo = from_lane<CTRL>((uint32_t)b, (uint32_t)n), hi = from_lane<CTRL>((uint32_t)(b >> 32), (uint32_t)(n >> 32));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
constexpr int kShr1 = 0x111, kShr2 = 0x112, kShr4 = 0x114, kShr8 = 0x118;
constexpr int kBcast15 = 0x142, kBcast31 = 0x143;

// f over the 64 lanes (in lane 63's order of combining; none: f's neutral value).
template <typename T, typename F>
__device__ __forceinline__ T over_lanes(T x, T none, F&& f) {
  x = f(x, from_lane<kShr1>(x, none));
  x = f(x, from_lane<kShr2>(x, none));
  x = f(x, from_lane<kShr4>(x, none));
  x = f(x, from_lane<kShr8>(x, none));
  x = f(x, from_lane<kBcast15>(x, none));
  x = f(x, from_lane<kBcast31>(x, none));
  return x;   // in lane 63
}
__device__ __forceinline__ float lane63(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), 63));
}

// The n-th largest of the lanes' values of `bits` bits, Q per lane (n <= 64 Q), in every lane.
template <int Q>
__device__ __forceinline__ uint32_t nth_of_lanes(const uint32_t (&x)[Q], int bits, int n) {
  uint32_t t = 0u;
  for (int b = bits - 1; b >= 0; --b) {
    const uint32_t probe = t | (1u << b);
    int k = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) k += __popcll(__ballot(x[q] >= probe));
    if (k >= n) t = probe;
  }
  return t;
}

// Sum over the workgroup, in every thread.
__device__ __forceinline__ int block_sum(int x, int* red) {
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
  __shared__ Piece<BF16> pieces[kPieces];
  __shared__ int piece_at[kPieces];
  __shared__ int listed, n_pieces;
  const int row = blockIdx.x / a.n_chunks, chunk = blockIdx.x - row * a.n_chunks;
  if (!continued(a, row)) return;   // the merge does not look at this row either
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int begin = chunk * (IT * kStep);
  const int whole = a.V & ~(kPiece - 1);   // entries in whole pieces; up to seven are left in the last chunk
  const int mine = tid * kPiece;
  const int steps = min(IT, (a.V - begin + kStep - 1) / kStep);   // fewer in a row's last chunk
  const void* base = static_cast<const char*>(a.logits) + (int64_t)row * a.ld * (BF16 ? 2 : 4);

  Piece<BF16> x[IT];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int v = begin + it * kStep + mine;
    x[it].clear();
    if (v < whole) x[it].load(base, v);
  }
  float rest = -__builtin_inff();   // entry whole + tid
  if (chunk == a.n_chunks - 1 && tid < a.V - whole)
    rest = BF16 ? bf16_lo(static_cast<const uint16_t*>(base)[whole + tid]) : static_cast<const float*>(base)[whole + tid];

  // fmaxf and the comparisons below pass over NaN
  float top[IT], best = fmaxf(rest, -__builtin_inff());
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    top[it] = -__builtin_inff();
    if (it >= steps) continue;
    top[it] = x[it].value(0);
#pragma unroll
    for (int i = 1; i < kPiece; ++i) top[it] = fmaxf(top[it], x[it].value(i));
    best = fmaxf(best, top[it]);
  }

  // The pieces stay as they came: unpacked again by each pass over them, so that
  // a thread's registers hold them once and more workgroups share a CU.
  auto hold = [&]() {
    if constexpr (BF16) {
#pragma unroll
      for (int it = 0; it < IT; ++it) asm volatile("" : "+v"(x[it].w[0]));
    }
  };
  hold();

  // the sets: the threads of one lane number, or each thread by itself
  if (tid == 0) listed = n_pieces = 0;
  red_f[wave * 64 + lane] = best;
  __syncthreads();
  best = red_f[lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) best = fmaxf(best, red_f[w * 64 + lane]);
  const float m = lane63(over_lanes(best, -__builtin_inff(), [](float p, float q) { return fmaxf(p, q); }));
  auto place16 = [](float x) { return (uint32_t)(pack_key(x, 0u) >> 48); };
  uint32_t nth;
  if (a.n <= kFewN) {
    const uint32_t sets[1] = {place16(best)};
    nth = nth_of_lanes(sets, 16, a.n);
  } else {
    uint32_t sets[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sets[w] = place16(fmaxf(red_f[w * 64 + lane], -__builtin_inff()));
    nth = nth_of_lanes(sets, 16, a.n);
  }
  const float bound = number_at(nth << 16);

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

  // Sum of e^(l - m) = 2^((l - m) log2 e). Where m is of ordinary size, as
  // 2^(l L - c) with L = fl(log2 e), c = fl(m L), one multiply-add per entry,
  // and 2^(c - m L) put right once for the chunk.
  constexpr float kLargest = 4096.0f;
  float s = 0.0f, residue = 0.0f;   // residue: m L - c, below 2.5e-4
  if (fabsf(m) <= kLargest) {
    const float c = m * kLog2e;
    residue = fmaf(m, kLog2e, -c);
    s = __builtin_amdgcn_exp2f(fmaf(rest, kLog2e, -c));
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if (it >= steps) break;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) s += __builtin_amdgcn_exp2f(fmaf(x[it].value(i), kLog2e, -c));
    }
  }
  if (s != s || !(fabsf(m) <= kLargest)) {   // NaN among this thread's entries: without them
    residue = 0.0f;
    float from = m;
    asm volatile("" : "+v"(from));   // nothing of the sum above is kept for this one
    s = 0.0f;
    auto term = [&](float v) { s += v == v ? __builtin_amdgcn_exp2f((v - from) * kLog2e) : 0.0f; };
    term(rest);
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) term(x[it].value(i));
  }
  const double t = -kLn2f * (double)residue;
  const double sum = over_lanes((double)s * (1.0 + t * (1.0 + t * (0.5 + t * (1.0 / 6.0)))), 0.0,
                                [](double p, double q) { return p + q; });
  if (lane == 63) red_d[wave] = sum;
  hold();

  // Entries that reach `least` (and, where they equal it, lie before `before`
  // in the chunk): first the pieces that hold any go to LDS, then their entries
  // to the list. -0 is listed as 0. False: too many pieces or entries.
  auto list_entries = [&](float least, int before) -> bool {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int first = it * kStep + mine;
      if (top[it] > least || (top[it] == least && first < before)) {
        const int k = atomicAdd(&n_pieces, 1);
        if (k < kPieces) {
          pieces[k] = x[it];
          piece_at[k] = first;
        }
      }
    }
    auto take = [&](float v, int place) {
      if (v > least || (v == least && place < before)) {
        const int k = atomicAdd(&listed, 1);
        if (k < kListed) list[k] = pack_key(v + 0.0f, (uint32_t)(begin + place));
      }
    };
    take(rest, whole + tid - begin);
    __syncthreads();
    const int n_p = n_pieces;
    if (n_p > kPieces) return false;
    for (int k = tid; k < n_p * kPiece; k += kThreads) {
      const int p = k / kPiece, i = k % kPiece;
      float v;
      if constexpr (BF16) v = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(&pieces[p])[i] << 16);
      else v = reinterpret_cast<const float*>(&pieces[p])[i];
      take(v, piece_at[p] + i);
    }
    __syncthreads();
    return listed <= kListed;
  };
  const bool fits = list_entries(fmaxf(bound, -__FLT_MAX__), IT * kStep);   // -inf is no entry
  if (tid == 0) {
    a.maxima[at] = m;
    a.sums[at] = (red_d[0] + red_d[1]) + (red_d[2] + red_d[3]);
  }
  if (!fits) {
    // Too many. The n-th largest value t, one bit of its place at a time from
    // the top, then the place in the chunk before which enough entries equal t.
    auto count = [&](auto&& f) {   // entries of the chunk for which f(value, place in the chunk)
      int k = f(rest, whole + tid - begin);
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) k += f(x[it].value(i), it * kStep + mine + i);
      hold();
      return block_sum(k, red_i);
    };
    uint32_t o = 0u;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t probe = o | (1u << bit);
      const float t = number_at(probe);   // NaN above infinity: no entry reaches it
      if (count([&](float v, int) { return v >= t; }) >= a.n) o = probe;
    }
    const float t = number_at(o);
    const int above = count([&](float v, int) { return v > t; });
    int before = 0;   // the largest place with fewer than n - above equal entries ahead of it
    for (int step = IT * kStep / 2; step >= 1; step >>= 1)
      if (count([&](float v, int p) { return v == t && p < before + step; }) < a.n - above) before += step;
    if (tid == 0) listed = n_pieces = 0;
    __syncthreads();
    list_entries(t, before + 1);   // exactly n entries, in at most n + 1 pieces
  }
  const int c = listed;
  for (int j = tid; j < c; j += kThreads) {   // a thread counts the ones ahead of its entry
    const uint64_t key = list[j];
    int rank = 0;
#pragma unroll 8
    for (int k = 0; k < c; ++k) rank += list[k] > key;
    if (rank < a.n) out[rank] = key;
  }
  if (tid >= c && tid < a.n) out[tid] = 0ull;
}

// A scored continuation: its score's place in fp64's order (0: none), and its
// place k * V + v; higher score first, then lower place.
struct Scored {
  uint64_t order;
  int64_t place;
};
__device__ __forceinline__ bool ahead(const Scored& x, const Scored& y) {
  return x.order > y.order || (x.order == y.order && x.place < y.place);
}
__device__ __forceinline__ double score_at(uint64_t o) {
  return __longlong_as_double((long long)((o >> 63) ? o & 0x7FFFFFFFFFFFFFFFull : ~o));
}

__global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(BeamSelectArgs a) {
  constexpr int kMW = kMergeThreads / 64;
  __shared__ double row_score[FS_BEAM_MAX], row_max[FS_BEAM_MAX], row_log[FS_BEAM_MAX];
  __shared__ int row_state[FS_BEAM_MAX];   // 0: not in use, 1: continued, 2: finished
  __shared__ uint32_t set_best[kSets];
  __shared__ uint64_t list_order[kMergeListed];
  __shared__ int64_t list_place[kMergeListed];
  __shared__ int listed;
  const int b = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int K = a.beams, n = a.n, nc = a.n_chunks;
  constexpr double kInf = __builtin_inf();

  // entry j of the group: the chunks' entries row by row, then the finished
  // beams. Every thread's first entries are on their way before the rows' sums.
  const int per_row = nc * n, scanned = K * per_row, total = scanned + K;   // at most 64 x 2^17 x 64
  const uint64_t* cand = a.cand + (int64_t)b * scanned;
  uint64_t first[kFirst];
#pragma unroll
  for (int i = 0; i < kFirst; ++i) {
    const int j = tid + i * kMergeThreads;
    first[i] = j < scanned ? cand[j] : 0ull;   // rows that are not in use hold anything, and are not looked at
  }

  // each row's maximum and logarithm of the sum: a wave per row
  for (int k = wave; k < K; k += kMW) {
    const int row = b * K + k;
    const float* maxima = a.maxima + (int64_t)row * nc;
    const double* sums = a.sums + (int64_t)row * nc;
    const float score = a.scores[row];
    const bool done = a.finished && a.finished[row];
    const bool in_use = score > -__builtin_inff();   // false for NaN
    int state = !in_use ? 0 : done ? 2 : 1;
    double m = -kInf, s = 0.0;
    if (state == 1) {
      for (int c = lane; c < nc; c += 64) {   // running maximum and sum
        const double mc = (double)maxima[c], sc = sums[c];
        if (mc > m) {
          s = mc < kInf ? s * exp(m - mc) + sc : 0.0;   // m = -inf: s is 0
          m = mc;
        } else if (mc > -kInf && mc < kInf) {
          s += sc * exp(mc - m);
        }
      }
      const double mine = m;
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) m = fmax(m, __shfl_xor(m, d));
      s = mine > -kInf && m < kInf ? s * exp(mine - m) : 0.0;
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
  if (tid < kSets) set_best[tid] = 0u;   // 0: a set without entry
  __syncthreads();

  auto scored = [&](int j, uint64_t key, Scored* e) -> bool {
    if (j < scanned) {
      const int k = j / per_row;
      if (row_state[k] != 1 || key == 0ull) return false;
      e->order = order_of(row_score[k] + (((double)number_at((uint32_t)(key >> 32)) - row_max[k]) - row_log[k]));
      e->place = (int64_t)k * a.V + key_to_token(key);
      return true;
    }
    const int k = j - scanned;
    if (row_state[k] != 2) return false;
    e->order = order_of(row_score[k]);
    e->place = (int64_t)k * a.V + a.pad;
    return true;
  };
  auto entry = [&](int j, Scored* e) -> bool { return scored(j, j < scanned ? cand[j] : 0ull, e); };
  auto each_entry = [&](auto&& f) {   // f(j, entry) of this thread's entries
    Scored e;
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
      const int j = tid + i * kMergeThreads;
      if (j < total && scored(j, first[i], &e)) f(j, e);
    }
    for (int j = tid + kFirst * kMergeThreads; j < total; j += kMergeThreads)
      if (entry(j, &e)) f(j, e);
  };

  // The bound, from the first `ranks` entries of every chunk (about eight per
  // set at least): sets by a mixing hash, so that neither the rank nor the
  // beam of an entry decides its set.
  const int lists = K * nc, n_sets = n <= kFewN ? kFewSets : kSets;
  const int ranks = min(n, (8 * n_sets + lists - 1) / lists);
  each_entry([&](int j, const Scored& e) {
    if (j >= scanned || j % n < ranks) {
      uint32_t h = (uint32_t)j * 2654435769u;
      h = (h ^ (h >> 15)) * 2246822519u;
      atomicMax(&set_best[(h ^ (h >> 13)) & (n_sets - 1)], (uint32_t)(e.order >> 32));
    }
  });
  __syncthreads();
  if (wave == 0) {   // 24 bits: sign, exponent and twelve bits of the scores
    uint32_t t;
    if (n <= kFewN) {
      const uint32_t sets[1] = {set_best[lane] >> 8};
      t = nth_of_lanes(sets, 24, n);
    } else {
      uint32_t sets[kSets / 64];
#pragma unroll
      for (int q = 0; q < kSets / 64; ++q) sets[q] = set_best[q * 64 + lane] >> 8;
      t = nth_of_lanes(sets, 24, n);
    }
    if (lane == 0) set_best[0] = t << 8;
  }
  __syncthreads();
  const uint64_t bound = (uint64_t)set_best[0] << 32;
  each_entry([&](int, const Scored& e) {
    if (e.order >= bound) {
      const int k = atomicAdd(&listed, 1);
      if (k < kMergeListed) {
        list_order[k] = e.order;
        list_place[k] = e.place;
      }
    }
  });
  __syncthreads();
  int c = listed;
  if (c > kMergeListed) {
    // too many equal scores: the best one behind the last taken, n times
    Scored last{~0ull, -1};
    for (int i = 0; i < n; ++i) {
      Scored best{0ull, INT64_MAX};
      each_entry([&](int, const Scored& e) {
        if (ahead(last, e) && ahead(e, best)) best = e;
      });
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) {
        const Scored other{shfl_xor_u64(best.order, d), (int64_t)shfl_xor_u64((uint64_t)best.place, d)};
        if (ahead(other, best)) best = other;
      }
      __syncthreads();   // everyone has read the previous round's result
      if (lane == 0) {
        list_order[kMergeListed - kMW + wave] = best.order;
        list_place[kMergeListed - kMW + wave] = best.place;
      }
      __syncthreads();
      last = Scored{0ull, INT64_MAX};
      for (int w = 0; w < kMW; ++w) {
        const Scored other{list_order[kMergeListed - kMW + w], list_place[kMergeListed - kMW + w]};
        if (ahead(other, last)) last = other;
      }
      if (tid == 0) {
        list_order[i] = last.order;
        list_place[i] = last.place;
      }
    }
    c = n;   // more than n entries exist, so every round found one
    __syncthreads();
  }
  float* out_scores = a.out_scores + (int64_t)b * n;
  int32_t* out_parents = a.out_parents + (int64_t)b * n;
  int32_t* out_tokens = a.out_tokens + (int64_t)b * n;
  for (int j = tid; j < c; j += kMergeThreads) {   // a thread counts the ones ahead of its entry
    const Scored e{list_order[j], list_place[j]};
    int rank = 0;
#pragma unroll 8
    for (int k = 0; k < c; ++k) rank += ahead(Scored{list_order[k], list_place[k]}, e);
    if (rank < n) {
      const int beam = (int)(e.place / a.V);
      out_scores[rank] = (float)score_at(e.order);
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
    default:
      if constexpr (BF16) return launch(beam_scan_kernel<true, 8>, grid, dim3(kThreads), 0, stream, a);
      else return hipErrorInvalidValue;   // beam_chunk gives no such chunk
  }
}

}  // namespace

// Chunks of 2048 entries, doubled while 1024 workgroups are left, up to 16384
// (fp32: 8192). Longer chunks find fewer candidates in all, until a thread's
// registers leave too few workgroups per CU. Measured, 512 rows of 152064, us:
// bf16 16384 35, 8192 40, 4096 59; fp32 16384 60-64, 8192 56, 4096 61-65.
int32_t beam_chunk(int64_t rows, int64_t V, bool bf16) {
  const int64_t steps = (V + kStep - 1) / kStep * rows;
  int it = 1;
  while (it < (bf16 ? 8 : 4) && steps / (2 * it) >= 1024) it *= 2;
  return it * kStep;
}

hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t stream) {
  const hipError_t e = a.bf16 ? launch_scan<true>(a, stream) : launch_scan<false>(a, stream);
  if (e != hipSuccess) return e;
  return launch(beam_merge_kernel, dim3((unsigned)a.B), dim3(kMergeThreads), 0, stream, a);
}

}  // namespace fs
