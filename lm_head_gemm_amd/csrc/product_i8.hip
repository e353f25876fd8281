// 8-bit integer product with a scale per token and per channel
// (fs_matmul_i8): out[m, n] = round((float(sum_k Q[m, k] W[n, k]) q_scales[m])
// w_scales[n]).
#include "fs_decode.h"

namespace fs {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// One wave per 16 channels x 16 tokens, operands straight from memory.
// v_mfma_i32_16x16x64_i8 with W as A and Q as B: lane (r, q) = (lane mod 16,
// lane / 16) holds bytes 16 q .. 16 q + 15 of the K step of channel (token) r,
// and receives channels 4 q .. 4 q + 3 of token r.
__global__ __launch_bounds__(kThreads) void product_i8_kernel(ProductI8Args a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = (blockIdx.x * (kThreads / 64) + wave) * 16;
  const int m0 = blockIdx.y * 16;
  if (n0 >= a.N) return;
  const int8_t* w = a.w + (int64_t)min(n0 + r, a.N - 1) * a.ldw;
  const int8_t* x = a.q + (int64_t)min(m0 + r, a.M - 1) * a.ldq;
  i32x4 acc = {0, 0, 0, 0};
  for (int k = 16 * q; k - 16 * q < a.K; k += 64) {
    i32x4 av = {0, 0, 0, 0}, bv = {0, 0, 0, 0};
    if (k < a.K) {
      av = *reinterpret_cast<const i32x4*>(w + k);
      bv = *reinterpret_cast<const i32x4*>(x + k);
    }
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, bv, acc, 0, 0, 0);
  }
  const int m = m0 + r;
  if (m >= a.M) return;
  const float qs = a.q_scales[m];
  for (int e = 0; e < 4; ++e) {
    const int n = n0 + 4 * q + e;
    if (n >= a.N) break;
    const float y = ((float)acc[e] * qs) * a.w_scales[n];
    const int64_t at = (int64_t)m * a.ldo + n;
    if (a.out_bf16) static_cast<uint16_t*>(a.out)[at] = f32_to_bf16_rne(y);
    else static_cast<float*>(a.out)[at] = y;
  }
}

}  // namespace

hipError_t launch_product_i8(const ProductI8Args& a, hipStream_t stream) {
  const int64_t gx = ((int64_t)a.N + 63) / 64, gy = ((int64_t)a.M + 15) / 16;
  if (gy > 65535) return hipErrorInvalidConfiguration;
  return launch(product_i8_kernel, dim3((unsigned)gx, (unsigned)gy), dim3(kThreads), 0, stream, a);
}

}  // namespace fs
