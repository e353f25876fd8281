// Rows to 8-bit codes with one scale per row, on their own (fs_quantize_i8) or
// behind the root-mean-square norm with the residual's addition
// (fs_rms_norm_i8).
//
// Per row: h = round(x + residual), u_j = h_j gain_j (u = x without a norm),
// a = max |u_j|, rstd = 1 / sqrt(mean(h^2) + eps):
//     codes[j] = rint(127 u_j / a),   scale = a rstd / 127.
// The norm's factor rstd is common to the row and cancels out of the codes, so
// no code depends on a sum. What is left is to round an exact quotient: the
// product u of two 16-bit values is exact in fp32, the product with an fp32
// gain in fp64. Each code is first taken from fp32 products with 127 / a (off
// by at most three roundings, 127 x 3 x 2^-24 = 2.3e-5 steps); one within 1e-4 of the
// middle between two codes is taken again from the fp64 quotient, whose a is
// exact: with an fp32 gain, the largest fp64 product among those whose fp32
// product comes within 2^-22 of the largest. Rows whose largest value fp32
// products may have lost (outside 2^-100 .. 2^126, zero rows, NaN and infinity)
// are done in fp64 throughout.
//
// Bound: memory (x, residual and gain read, h, codes and scales written once).
// The row stays in registers between the reduction and the codes: G threads
// hold V 16-byte pieces each, so a row is read once whatever its length. Gains
// are fetched beside the row: read between the stores of h and of codes, which
// no load may pass, they cost 10-40% of the time.
// Measured: norm with residual, bf16, 4099 x 8192 46.5 us (5.1 TB/s read and
// written, a large copy's rate), with an fp32 gain 52 us; 64 x 7168 4.8 us, 1 x
// 4096 3.6 us; codes of 128256 x 4096 bf16 254-262 us by box (6.0-6.2 TB/s).
#include "fs_decode.h"

namespace fs {
namespace {

constexpr int kWave = 64;

// A 16-byte piece of a row as fp32 values.
template <bool BF16>
__device__ __forceinline__ float piece_value(const uint4& p, int e) {
  if constexpr (BF16) {
    const uint32_t w = e < 2 ? p.x : e < 4 ? p.y : e < 6 ? p.z : p.w;
    return (e & 1) ? bf16_hi(w) : bf16_lo(w);
  } else {
    return __uint_as_float(e == 0 ? p.x : e == 1 ? p.y : e == 2 ? p.z : p.w);
  }
}

// |u| as an unsigned whole number: its order is that of the magnitudes, with
// infinity and then every NaN above all numbers.
__device__ __forceinline__ uint32_t magnitude(float u) { return __float_as_uint(u) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint64_t magnitude(double u) {
  return (uint64_t)__double_as_longlong(u) & 0x7FFFFFFFFFFFFFFFull;
}

__device__ __forceinline__ uint32_t wave_xor(uint32_t x, int m) { return (uint32_t)__shfl_xor((int)x, m); }
__device__ __forceinline__ uint64_t wave_xor(uint64_t x, int m) { return shfl_xor_u64(x, m); }

// Largest value over the G threads of a row, in all of them.
template <int G, typename T>
__device__ __forceinline__ T row_max(T x, T* red, int tid) {
#pragma unroll
  for (int m = kWave / 2; m >= 1; m >>= 1) {
    const T y = wave_xor(x, m);
    x = y > x ? y : x;
  }
  if constexpr (G > kWave) {
    __syncthreads();   // the previous use of red is over
    if (tid % kWave == 0) red[tid / kWave] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < G / kWave; ++w) x = red[w] > x ? red[w] : x;
  }
  return x;
}

template <int G>
__device__ __forceinline__ double row_sum(double x, double* red, int tid) {
#pragma unroll
  for (int m = kWave / 2; m >= 1; m >>= 1) x += __shfl_xor(x, m);
  if constexpr (G > kWave) {
    if (tid % kWave == 0) red[tid / kWave] = x;
    __syncthreads();
    x = 0.0;
#pragma unroll
    for (int w = 0; w < G / kWave; ++w) x += red[w];
  }
  return x;
}

// GAIN: 0 none (no norm), 1 bf16, 2 fp32. RES: with a residual. G threads per
// row, V pieces per thread.
template <bool BF16, int GAIN, bool RES, int G, int V>
__global__ __launch_bounds__(G < 256 ? 256 : G) void rows_i8_kernel(RowsI8Args a) {
  constexpr int E = BF16 ? 8 : 4;                 // values per 16-byte piece
  constexpr int kRows = G < 256 ? 256 / G : 1;    // rows per workgroup
  __shared__ double red_sum[G / kWave];
  __shared__ uint64_t red_max[G / kWave];
  const int tid = threadIdx.x % G;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
  if (row >= a.M) return;                         // whole waves of a workgroup without barriers
  const int np = a.D / E;                         // pieces per row

  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) + row * a.ldx * (16 / E));
  uint4 h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = tid + v * G;
    h[v] = make_uint4(0u, 0u, 0u, 0u);
    if (p < np) h[v] = load_stream16(x + p);
  }
  // gain of piece p, value e
  auto gain_of = [&](int p, int e) -> float {
    if constexpr (GAIN == 1) return piece_value<true>(static_cast<const uint4*>(a.gain)[p], e);
    if constexpr (GAIN == 2) return static_cast<const float*>(a.gain)[(int64_t)p * E + e];
    return 1.0f;
  };
  // The gains, fetched beside the row, then the fp32 products; where a thread's
  // registers do not hold them too, gains are read at each use.
  constexpr bool kKeep = GAIN != 0 && V <= 4;
  float u[kKeep ? V : 1][E];
  if constexpr (kKeep) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = tid + v * G;
#pragma unroll
      for (int e = 0; e < E; ++e) u[v][e] = 0.0f;
      if (p < np)
#pragma unroll
        for (int e = 0; e < E; ++e) u[v][e] = gain_of(p, e);
    }
  }
  if constexpr (RES) {
    const uint4* r = reinterpret_cast<const uint4*>(static_cast<const char*>(a.residual) + row * a.ldr * (16 / E));
    uint4* s = reinterpret_cast<uint4*>(static_cast<char*>(a.sum) + row * a.lds * (16 / E));
    uint4 rr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = tid + v * G;
      rr[v] = make_uint4(0u, 0u, 0u, 0u);
      if (p < np) rr[v] = load_stream16(r + p);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = tid + v * G;
      float f[E];
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = piece_value<BF16>(h[v], e) + piece_value<BF16>(rr[v], e);
      if constexpr (BF16) {
        h[v] = make_uint4((uint32_t)f32_to_bf16_rne(f[0]) | ((uint32_t)f32_to_bf16_rne(f[1]) << 16),
                          (uint32_t)f32_to_bf16_rne(f[2]) | ((uint32_t)f32_to_bf16_rne(f[3]) << 16),
                          (uint32_t)f32_to_bf16_rne(f[4 % E]) | ((uint32_t)f32_to_bf16_rne(f[5 % E]) << 16),
                          (uint32_t)f32_to_bf16_rne(f[6 % E]) | ((uint32_t)f32_to_bf16_rne(f[7 % E]) << 16));
      } else {
        h[v] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      }
      if (p < np) s[p] = h[v];
    }
  }

  // u exactly; the few values that need it read their gain again
  auto exact = [&](int v, int e, int p) -> double {
    const double f = (double)piece_value<BF16>(h[v], e);
    if constexpr (GAIN == 0) return f;
    else return f * (double)gain_of(p, e);
  };
  if constexpr (kKeep) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < E; ++e) u[v][e] *= piece_value<BF16>(h[v], e);
  }
  auto value = [&](int v, int e, int p) -> float {
    if constexpr (kKeep) return u[v][e];
    else if constexpr (GAIN == 0) return piece_value<BF16>(h[v], e);
    else return piece_value<BF16>(h[v], e) * gain_of(p, e);
  };

  double rstd = 1.0;
  if constexpr (GAIN != 0) {
    double ssq = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const double f = (double)piece_value<BF16>(h[v], e);   // pieces past the row are zero
        ssq = fma(f, f, ssq);
      }
    ssq = row_sum<G>(ssq, red_sum, tid);
    if (tid == 0) rstd = 1.0 / sqrt(ssq / (double)a.D + (double)a.eps);
  }

  int8_t* codes = a.codes + row * a.ldc;
  auto store = [&](int p, const uint32_t (&c)[E]) {   // the lowest byte of each
    uint32_t w[E / 4];
#pragma unroll
    for (int k = 0; k < E / 4; ++k)
      w[k] = __builtin_amdgcn_perm(c[4 * k + 1], c[4 * k], 0x0C0C0400u) |
             __builtin_amdgcn_perm(c[4 * k + 3], c[4 * k + 2], 0x04000C0Cu);
    if constexpr (E == 8) *reinterpret_cast<uint2*>(codes + (int64_t)p * E) = make_uint2(w[0], w[E / 4 - 1]);
    else *reinterpret_cast<uint32_t*>(codes + (int64_t)p * E) = w[0];
  };

  // the row's largest |u| as an fp64 number, of all values or of those whose fp32 product reaches `least`
  auto largest = [&](auto all_c, float least) -> uint64_t {
    uint64_t top = 0u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = tid + v * G;
      if (p < np)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (decltype(all_c)::value || fabsf(value(v, e, p)) >= least) {
            const uint64_t m = magnitude(exact(v, e, p));
            top = m > top ? m : top;
          }
    }
    return row_max<G>(top, red_max, tid);
  };
  if constexpr (GAIN != 2 || kKeep) {
    uint32_t top32 = 0u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = tid + v * G;
      if (GAIN == 0 || kKeep || p < np)   // else: pieces past the row are zero
#pragma unroll
        for (int e = 0; e < E; ++e) top32 = max(top32, magnitude(value(v, e, p)));
    }
    top32 = row_max<G>(top32, reinterpret_cast<uint32_t*>(red_max), tid);
    if (top32 >= 0x0D800000u && top32 < 0x7E800000u) {   // 2^-100 <= a < 2^126 (uniform over the row)
      const float a32 = __uint_as_float(top32);
      double amax = (double)a32;
      // rounded products: the exact largest is among those within 2^-22
      if constexpr (GAIN == 2) amax = __longlong_as_double((long long)largest(std::false_type{}, a32 * (1.0f - 0x1p-22f)));
      const float inv = 127.0f / a32;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int p = tid + v * G;
        if (p < np) {
          // x + 1.5 2^23 is x rounded to a whole number, which is in the lowest bits
          constexpr float kWhole = 12582912.0f;
          uint32_t c[E];
          float far = 0.0f;   // largest distance from a whole number
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float x32 = value(v, e, p), k = fmaf(x32, inv, kWhole);
            far = fmaxf(far, fabsf(fmaf(x32, inv, kWhole - k)));
            c[e] = __float_as_uint(k);
          }
          if (far > 0.4999f) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (fabsf(fmaf(value(v, e, p), inv, kWhole - __uint_as_float(c[e]))) > 0.4999f)
                c[e] = (uint32_t)(int)rint(127.0 * (GAIN == 2 ? exact(v, e, p) : (double)value(v, e, p)) / amax);
          }
          store(p, c);
        }
      }
      if (tid == 0) a.scales[row] = (float)(amax * rstd / 127.0);
      return;
    }
  }

  // rows outside fp32's range above, and long ones with fp32 gains: fp64 throughout
  const uint64_t top = largest(std::true_type{}, 0.0f);
  const double amax = __longlong_as_double((long long)top);
  const bool bad = top >= 0x7FF0000000000000ull;   // a NaN or an infinity
  const bool none = bad || top == 0u;
  const double inv = none ? 0.0 : 127.0 / amax;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = tid + v * G;
    if (p < np) {
      uint32_t c[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const double x64 = exact(v, e, p);
        const double t = x64 * inv;
        double k = rint(t);
        if (fabs(t - k) > 0.4999) k = rint(127.0 * x64 / amax);
        c[e] = none ? 0u : (uint32_t)(int)k;
      }
      store(p, c);
    }
  }
  if (tid == 0) a.scales[row] = bad ? __builtin_nanf("") : (float)(amax * rstd / 127.0);
}

template <bool BF16, int GAIN, bool RES, int G, int V>
hipError_t go(const RowsI8Args& a, hipStream_t stream) {
  constexpr int kRows = G < 256 ? 256 / G : 1;
  const int64_t blocks = ((int64_t)a.M + kRows - 1) / kRows;
  return launch(rows_i8_kernel<BF16, GAIN, RES, G, V>, dim3((unsigned)blocks), dim3(G < 256 ? 256 : G), 0, stream, a);
}

// Threads and pieces per row: a wave for short rows (no barrier), 256 threads up
// to 1024 pieces (16 KiB), 1024 threads above. With no more rows than CUs a
// row has its CU to itself: a thread per piece. Measured (us, bf16, residual):
// 64 x 7168 1024 threads 4.8, 256 6.5; 256 x 8192 5.7, 7.4; 1 x 4096 512 threads
// 3.8, 256 4.4 (300 rows: 5.6 either way). 4096 x 5120 three pieces per thread
// 34.0, four 40.9; 4099 x 8192 256 threads of four 48.2, 512 of two 49.4 (fp32
// gain 54, 61).
template <bool BF16, int GAIN, bool RES>
hipError_t by_length(const RowsI8Args& a, hipStream_t stream) {
  const int64_t np = (int64_t)a.D / (BF16 ? 8 : 4);
  if (np <= 64) return go<BF16, GAIN, RES, 64, 1>(a, stream);
  if (np <= 256) return go<BF16, GAIN, RES, 256, 1>(a, stream);
  if (a.M <= 256 && np > 256 && np <= 512) return go<BF16, GAIN, RES, 512, 1>(a, stream);
  if (a.M <= 256 && np > 512 && np <= 1024) return go<BF16, GAIN, RES, 1024, 1>(a, stream);
  if (np <= 512) return go<BF16, GAIN, RES, 256, 2>(a, stream);
  if (np <= 768) return go<BF16, GAIN, RES, 256, 3>(a, stream);
  if (np <= 1024) return go<BF16, GAIN, RES, 256, 4>(a, stream);
  if (np <= 2048) return go<BF16, GAIN, RES, 1024, 2>(a, stream);
  if (np <= 4096) return go<BF16, GAIN, RES, 1024, 4>(a, stream);
  return go<BF16, GAIN, RES, 1024, 10>(a, stream);   // up to 160 KiB, checked by the caller
}

}  // namespace

hipError_t launch_rows_i8(const RowsI8Args& a, bool bf16, bool gain_bf16, hipStream_t stream) {
  if (bf16) {
    if (!a.gain) return by_length<true, 0, false>(a, stream);
    if (gain_bf16)
      return a.residual ? by_length<true, 1, true>(a, stream) : by_length<true, 1, false>(a, stream);
    return a.residual ? by_length<true, 2, true>(a, stream) : by_length<true, 2, false>(a, stream);
  }
  if (!a.gain) return by_length<false, 0, false>(a, stream);
  return a.residual ? by_length<false, 2, true>(a, stream) : by_length<false, 2, false>(a, stream);
}

}  // namespace fs
