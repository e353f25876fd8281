// 8-bit integer product with a scale per token and per channel
// (fs_matmul_i8): out[m, n] = round((float(sum_k Q[m, k] W[n, k]) q_scales[m])
// w_scales[n]).
//
// v_mfma_i32_16x16x64_i8 with W as the A operand (16 channels) and Q as B (16
// tokens): lane (r, q) = (lane mod 16, lane / 16) holds bytes 16 q .. 16 q + 15
// of a 64-byte K step of channel (token) r, and receives channels 4 q .. 4 q + 3
// of token r. Sums are exact in int32, so no order of them matters.
//
// Both operands go from memory straight to LDS (global_load_lds_dwordx4, no
// registers in between), a stage of BKB bytes of K for all rows of the tile at
// a time, in a ring of NS stages.
//  * A wave load fills 1 KiB of LDS, lane i at byte 16 i: 1024 / BKB rows of
//    BKB contiguous bytes. Which 16-byte piece of its row a lane fetches is
//    chosen so that the operand reads (ds_read_b128: 16 rows, one K step) meet
//    no bank twice: piece p of row r lies at p ^ swizzle(r).
//  * Per stage: each wave waits for its own copies of it (later ones stay in
//    flight), one workgroup barrier, all operand reads of stage s, the copies of
//    stage s + NS - 1 into the buffer that stage s - 1 has left, and the matrix
//    instructions.
//  * K need not be a multiple of BKB: for pieces past K the stage's first one is
//    fetched, and Q's are zeroed in LDS by the wave that fetched them.
//    Whatever W holds there counts nothing, the products being integers.
//  * Rows past N and M are fetched from the last one and not stored.
#include "fs_decode.h"

namespace fs {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int N>
__device__ __forceinline__ void wait_copies_and_sync() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  // own copies but the N youngest are done, and own LDS accesses; then
  // everyone's. No memory access may cross.
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 64 x 16 bytes from base + each lane's offset to LDS bytes lds .. lds + 1023
// (base and lds uniform). Written out because the compiler makes every LDS read
// wait for all copies that it knows of; it does not use m0 itself here. ONCE:
// bytes that no one else reads do not displace others in the caches.
template <bool ONCE>
__device__ __forceinline__ void copy_to_lds(const int8_t* base, uint32_t offset, uint32_t lds) {
  const int at = __builtin_amdgcn_readfirstlane((int)lds);
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(offset), "s"(base), "s"(at)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base), "s"(at)
                 : "memory");
}

typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));

// WR x TC blocks of 16 channels x 16 tokens per wave, NWW x NWT waves, one tile
// per workgroup. ONE (a single token tile, memory-bound): W's copies are marked
// as read once, and tiles start at different stages; else the token tiles of the
// same channels run at one time on one XCD (tile_of) and share them in its L2.
template <int WR, int TC, int NWW, int NWT, int BKB, int NS, bool ONE>
__global__ __launch_bounds__(64 * NWW * NWT) void product_i8_kernel(ProductI8Args a, int n_wt, int n_mt) {
  constexpr int NW = NWW * NWT;
  constexpr int BM = 16 * WR * NWW, BN = 16 * TC * NWT;   // channels, tokens per tile
  constexpr int PPR = BKB / 16;                           // pieces per row and stage
  constexpr int RPL = 64 / PPR;                           // rows per wave load
  constexpr int LPW = (BM + BN) / RPL / NW;               // wave loads per wave and stage
  constexpr int STAGE = (BM + BN) * BKB;                  // bytes
  constexpr int KS = BKB / 64;                            // K steps per stage
  constexpr int WRC = WR % 2 == 0 ? 2 : 1;                // epilogue: blocks of channels at a time
  constexpr int ROW = 16 * WRC + 4;                       // padded row of one token, floats
  static_assert((BM + BN) % (RPL * NW) == 0 && BM % RPL == 0, "even shares of the copies");
  static_assert(NW * 16 * ROW * 4 <= NS * STAGE, "the epilogue's tiles fit the ring");
  __shared__ __align__(1024) unsigned char ring[NS * STAGE];

  int vt, mt;
  if (!tile_of(blockIdx.x, n_wt, n_mt, &vt, &mt)) return;   // whole workgroup
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = vt * BM, m0 = mt * BN;
  const int rows = min(BM, a.N - n0);   // channels of this tile
  const int S = (a.K + BKB - 1) / BKB;
  // Rows of a power-of-two stride read at one offset meet on a few memory
  // channels; a multiplicative hash spreads the first stages over the tiles of
  // every XCD (tile vt runs on XCD vt mod 8). Measured, one token, 8192 x
  // 128256: 155 us, against 230 with first stage vt mod S.
  const int s0 = ONE ? (int)((uint32_t)vt * 2654435769u >> 16) % S : 0;

  auto swizzle = [](int row) { return PPR == 8 ? (row >> 1) & 7 : row & 15; };
  static_assert(PPR == 8 || PPR == 16, "rows of 128 or 256 bytes");
  // Wave load i of this wave: rows (wave LPW + i) RPL .. of the stage
  // (channels, then tokens); offset[i]: of this lane's row and piece at stage 0
  // from the tile's first channel or token.
  auto first_row = [&](int i) { return __builtin_amdgcn_readfirstlane((wave * LPW + i) * RPL); };
  auto piece = [&](int i) { return (lane % PPR) ^ swizzle(first_row(i) + lane / PPR); };
  const int8_t* w_tile = a.w + (int64_t)n0 * a.ldw;
  const int8_t* q_tile = a.q + (int64_t)m0 * a.ldq;
  uint32_t offset[LPW];
#pragma unroll
  for (int i = 0; i < LPW; ++i) {
    const int row = first_row(i) + lane / PPR;
    offset[i] = (uint32_t)(row < BM ? min(row, rows - 1) * (int64_t)a.ldw
                                    : min(row - BM, a.M - 1 - m0) * (int64_t)a.ldq) + 16 * piece(i);
  }
  const uint32_t ring_at = (uint32_t)(uintptr_t)ring;
  auto issue = [&](int s, int buf) {   // s: stage in this tile's order
    const int k0 = (s0 + s >= S ? s0 + s - S : s0 + s) * BKB;
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
      const bool of_w = first_row(i) < BM;
      uint32_t o = offset[i];
      if (k0 + BKB > a.K && k0 + 16 * piece(i) >= a.K) o -= 16 * piece(i);   // past K: the stage's first piece
      const uint32_t to = ring_at + buf * STAGE + (wave * LPW + i) * 1024;
      const int8_t* base = (of_w ? w_tile : q_tile) + k0;
      if (ONE && of_w) copy_to_lds<true>(base, o, to);
      else copy_to_lds<false>(base, o, to);
    }
  };
  // zeroes this wave's pieces of Q past K in the partial stage (its copies have arrived)
  auto zero_tail = [&](int buf) {
#pragma unroll
    for (int i = 0; i < LPW; ++i)
      if (first_row(i) >= BM && (S - 1) * BKB + 16 * piece(i) >= a.K)
        *reinterpret_cast<i32x4*>(ring + buf * STAGE + (wave * LPW + i) * 1024 + lane * 16) = i32x4{0, 0, 0, 0};
  };

  const int ww = wave % NWW, wt = wave / NWW;
  const int a_at = (ww * WR * 16 + r) * BKB, b_at = (BM + wt * TC * 16 + r) * BKB;   // of block 0 in a stage
  int k_at[KS];
#pragma unroll
  for (int t = 0; t < KS; ++t) k_at[t] = 16 * ((4 * t + q) ^ swizzle(r));

  i32x4 av[KS][WR], bv[KS][TC];
  i32x4 acc[WR][TC];
  auto read = [&](int buf) {   // the whole stage's operands, so that one wait serves all K steps
    const unsigned char* st = ring + buf * STAGE;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
#pragma unroll
      for (int j = 0; j < WR; ++j) av[t][j] = *reinterpret_cast<const i32x4*>(st + k_at[t] + a_at + j * 16 * BKB);
#pragma unroll
      for (int c = 0; c < TC; ++c) bv[t][c] = *reinterpret_cast<const i32x4*>(st + k_at[t] + b_at + c * 16 * BKB);
    }
  };
  auto multiply = [&]() {
#pragma unroll
    for (int t = 0; t < KS; ++t)
#pragma unroll
      for (int c = 0; c < TC; ++c)
#pragma unroll
        for (int j = 0; j < WR; ++j)
          acc[j][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[t][j], bv[t][c], acc[j][c], 0, 0, 0);
  };
  const int partial = a.K % BKB == 0 ? -1 : S - 1 - s0;   // the partial stage's turn
  // Stage s, in `buf`, is complete in LDS and everyone's reads of earlier ones
  // are done. LEFT: this wave's copies that may stay in flight.
  auto arrive = [&](int s, int buf, auto left_c) {
    if (s == partial) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      zero_tail(buf);
    }
    wait_copies_and_sync<decltype(left_c)::value>();
  };
#pragma unroll
  for (int j = 0; j < WR; ++j)
#pragma unroll
    for (int c = 0; c < TC; ++c) acc[j][c] = i32x4{0, 0, 0, 0};
  for (int s = 0; s < NS - 1 && s < S; ++s) issue(s, s);
  int buf = 0;
  for (int s = 0; s < S; ++s) {
    if (s + NS - 1 <= S) arrive(s, buf, std::integral_constant<int, (NS - 2) * LPW>{});
    else arrive(s, buf, std::integral_constant<int, 0>{});
    read(buf);
    if (s + NS - 1 < S) issue(s + NS - 1, buf == 0 ? NS - 1 : buf - 1);
    multiply();
    buf = buf == NS - 1 ? 0 : buf + 1;
  }

  // A lane holds four neighbouring channels of one token; through a wave's own
  // part of the ring they become whole runs of 16 WRC channels.
  __syncthreads();   // every wave is done with the ring
  auto write = [&](auto bf16_c) {
    constexpr bool kBF16 = decltype(bf16_c)::value;
    constexpr int PER = kBF16 ? 8 : 4;            // channels per lane and store
    constexpr int LPT = 16 * WRC / PER;           // lanes per token
    float* tile = reinterpret_cast<float*>(ring) + wave * 16 * ROW;
#pragma unroll
    for (int j0 = 0; j0 < WR; j0 += WRC) {
      const int nb = (ww * WR + j0) * 16;         // first channel in the tile
      float ws[WRC][4];
#pragma unroll
      for (int j = 0; j < WRC; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = min(nb + j * 16 + 4 * q + e, rows - 1);
          ws[j][e] = a.w_scales[n0 + n];
        }
#pragma unroll
      for (int c = 0; c < TC; ++c) {
        const int mb = m0 + (wt * TC + c) * 16;
        const float qs = a.q_scales[min(mb + r, a.M - 1)];
#pragma unroll
        for (int j = 0; j < WRC; ++j) {
          f32x4 y;
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = ((float)acc[j0 + j][c][e] * qs) * ws[j][e];
          *reinterpret_cast<f32x4*>(tile + r * ROW + 16 * j + 4 * q) = y;
        }
        __builtin_amdgcn_wave_barrier();   // one wave's LDS operations keep their order
#pragma unroll
        for (int i = 0; i < 16 * LPT / 64 || i == 0; ++i) {
          const int x = i * 64 + lane;
          const int tok = x / LPT, n = nb + x % LPT * PER;
          if (tok < 16 && mb + tok < a.M && n < rows) {
            const float* y = tile + tok * ROW + x % LPT * PER;
            const int64_t at = (int64_t)(mb + tok) * a.ldo + n0 + n;
            if constexpr (kBF16) {
              uint16_t* p = static_cast<uint16_t*>(a.out) + at;
              if (n + PER <= rows) {
                u32x4_t v;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  v[k] = (uint32_t)f32_to_bf16_rne(y[2 * k]) | ((uint32_t)f32_to_bf16_rne(y[2 * k + 1]) << 16);
                __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2*>(p));
              } else {
                for (int k = 0; k < PER && n + k < rows; ++k) p[k] = f32_to_bf16_rne(y[k]);
              }
            } else {
              float* p = static_cast<float*>(a.out) + at;
              if (n + PER <= rows) {
                const u32x4_t v = {__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                                   __float_as_uint(y[3])};
                __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a4*>(p));
              } else {
                for (int k = 0; k < PER && n + k < rows; ++k) p[k] = y[k];
              }
            }
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
  };

  if (a.out_bf16) write(std::true_type{});
  else write(std::false_type{});
}

// Few, small tiles: 16 channels x 16 TC tokens per workgroup, whose 8 waves
// share out the K steps (wave w takes steps w, w + 8, ...), straight from memory
// to registers, and add their whole-number sums in LDS. A tile of the kernel
// above spends about 0.55 us on each 256 bytes of K, whatever is in flight
// (its barrier and its waves' instructions, one wave per SIMD); here a wave has
// four K steps in flight at once and no barrier before the end.
template <int TC>
__global__ __launch_bounds__(512) void product_i8_small_kernel(ProductI8Args a, int n_wt) {
  constexpr int NW = 8, U = 4, ROW = 17;
  __shared__ int32_t sums[NW][16 * TC][ROW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int vt = blockIdx.x % n_wt, mt = blockIdx.x / n_wt;
  const int n0 = vt * 16, m0 = mt * 16 * TC;
  const int8_t* w = a.w + (int64_t)min(n0 + r, a.N - 1) * a.ldw;
  const int8_t* x[TC];
  i32x4 acc[TC];
#pragma unroll
  for (int c = 0; c < TC; ++c) {
    x[c] = a.q + (int64_t)min(m0 + 16 * c + r, a.M - 1) * a.ldq;
    acc[c] = i32x4{0, 0, 0, 0};
  }
  for (int k0 = 64 * wave; k0 < a.K; k0 += 64 * NW * U) {
    i32x4 av[U], bv[U][TC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 64 * NW * u + 16 * q;
      av[u] = i32x4{0, 0, 0, 0};
      if (k < a.K) av[u] = *reinterpret_cast<const i32x4*>(w + k);
#pragma unroll
      for (int c = 0; c < TC; ++c) {
        bv[u][c] = i32x4{0, 0, 0, 0};
        if (k < a.K) bv[u][c] = *reinterpret_cast<const i32x4*>(x[c] + k);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < TC; ++c) acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[u], bv[u][c], acc[c], 0, 0, 0);
  }
#pragma unroll
  for (int c = 0; c < TC; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[wave][16 * c + r][4 * q + e] = acc[c][e];
  __syncthreads();
  for (int i = tid; i < 256 * TC; i += 64 * NW) {
    const int m = m0 + i / 16, n = n0 + i % 16;
    if (m >= a.M || n >= a.N) continue;
    int32_t sum = 0;
#pragma unroll
    for (int v = 0; v < NW; ++v) sum += sums[v][i / 16][i % 16];
    const float y = ((float)sum * a.q_scales[m]) * a.w_scales[n];
    const int64_t at = (int64_t)m * a.ldo + n;
    if (a.out_bf16) static_cast<uint16_t*>(a.out)[at] = f32_to_bf16_rne(y);
    else static_cast<float*>(a.out)[at] = y;
  }
}

template <int TC>
hipError_t go_small(const ProductI8Args& a, hipStream_t stream) {
  const int64_t n_wt = ((int64_t)a.N + 15) / 16, n_mt = ((int64_t)a.M + 16 * TC - 1) / (16 * TC);
  if (!grid_fits(n_wt * n_mt, 512)) return hipErrorInvalidConfiguration;
  return launch(product_i8_small_kernel<TC>, dim3((unsigned)(n_wt * n_mt)), dim3(512), 0, stream, a, (int)n_wt);
}

template <int WR, int TC, int NWW, int NWT, int BKB, int NS, bool ONE>
hipError_t go(const ProductI8Args& a, hipStream_t stream) {
  constexpr int BM = 16 * WR * NWW, BN = 16 * TC * NWT;
  const int64_t n_wt = ((int64_t)a.N + BM - 1) / BM, n_mt = ((int64_t)a.M + BN - 1) / BN;
  const int64_t tiles = n_wt * n_mt;
  const int64_t grid = n_mt == 1 ? tiles : (tiles + kXcds - 1) / kXcds * kXcds;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;   // launch() checks grid x threads
  return launch(product_i8_kernel<WR, TC, NWW, NWT, BKB, NS, ONE>, dim3((unsigned)grid), dim3(64 * NWW * NWT), 0,
                stream, a, (int)n_wt, (int)n_mt);
}

}  // namespace

// The tile by the number of tiles it leaves: a launch wants most of the 256 CUs
// busy; beyond that, larger tiles move fewer bytes per product, but write out
// with nothing beside them on their CU, which short sums feel. Measured (us,
// M x N x K; the tile taken first, channels x tokens):
//   M <= 16: 64 x 16 from N = 16384 on (16 x 16384 x 4096: 12.4, small 15.8;
//     1 x 128256 x 4096: 80), else the small kernel (1 x 5003 x 4096: 7.6, 11.5)
//   M <= 32: 128 x 32 (32 x 128256 x 4096: 83, with 128 x 64 tiles 88)
//   64 x 152064 x 3584: 128 x 64 100, 256 x 64 116, 64 x 64 123
//   128 x 128256 x 4096: 256 x 128 118, 128 x 128 134
//   1024 x 16384 x 4096: 256 x 256 75, 128 x 128 81; 1024 x 129280 x 2048: 340,
//     410; but x 512: 128 x 128 149, 256 x 256 162; 359 x 42863 x 704: 35, 66
//   256 x 128256 x 4096: 256 x 256 180, 128 x 128 203: with an odd number of
//     128-token tiles below seven the larger tile's empty half costs more
//   1024 x 5003 x 2320: 128 x 128 27, 256 x 256 47; 300 x 5003 x 512: 128 x 64
//     7.3, 128 x 128 9.1, 32 x 64 9.7; 128 x 5003 x 4096: 32 x 64 14.8, 128 x 64
//     22.8, small 29.7; 45 x 5003 x 2320: small 8.5, 32 x 64 9.7
// Rings of two to four stages and two workgroups per CU (one for the two
// largest tiles, whose LDS holds no more): deeper rings with one workgroup
// measured 5-15% slower on the memory-bound shapes, stages of half the length
// 5-25% slower.
hipError_t launch_product_i8(const ProductI8Args& a, hipStream_t stream) {
  auto tiles = [&](int64_t bm, int64_t bn) { return ((a.N + bm - 1) / bm) * ((a.M + bn - 1) / bn); };
  if (a.M <= 16) {
    if (tiles(64, 16) >= 256) return go<1, 1, 4, 1, 256, 4, true>(a, stream);
    return go_small<1>(a, stream);
  }
  if (a.M <= 32 && tiles(128, 32) >= 192) return go<2, 2, 4, 1, 128, 4, true>(a, stream);
  if (a.M > 64 && a.K >= 1024) {
    const int64_t halves = ((int64_t)a.M + 127) / 128;
    if (halves == 1 && tiles(256, 128) >= 192) return go<4, 4, 4, 2, 128, 3, true>(a, stream);
    if (halves > 1 && (halves % 2 == 0 || halves >= 7) && tiles(256, 256) >= 192)
      return go<4, 8, 4, 2, 128, 2, false>(a, stream);
  }
  if (a.M > 64 && tiles(128, 128) >= 192) return go<2, 4, 4, 2, 128, 2, false>(a, stream);
  if (tiles(128, 64) >= 192)
    return a.M <= 64 ? go<2, 2, 4, 2, 128, 3, true>(a, stream) : go<2, 2, 4, 2, 128, 3, false>(a, stream);
  if (tiles(32, 64) >= 256) return go<1, 2, 2, 2, 256, 3, false>(a, stream);
  return go_small<4>(a, stream);
}

}  // namespace fs
