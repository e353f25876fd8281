// Reordering of beam search's states (fs_beam_reorder): row i of a group
// becomes its former row parents[i], in every buffer and slab.
//
// Bound: memory (every row that moves is read and written once). A thread owns
// one unit (16 bytes where all addresses allow) of all rows of a group: it reads
// the parents' units into registers, then writes them, so the rows may be
// permuted in place, with one parent taken by several rows, and no thread waits
// for another. In place, a row that is its own parent is neither read nor
// written. One unit per thread and as many workgroups as that takes: threads
// that loop over units in a grid of 8192 or 32768 workgroups measured 6-16%
// slower (8 x 4 rows), and faster only where no row moves.
// Measured, bf16 caches of 32 layers, keys and values, 8 heads x 128, 1000 of
// 1024 positions, every row moved, in place: 8 x 4 rows 1555 us (5.4 TB/s read
// and written), 4 x 8 1598, 2 x 16 1678, 1 x 32 1637; 4 layers of 1 x 4 rows, 33
// positions: the launch (8 us a call).
#include "fs_decode.h"

namespace fs {
namespace {

constexpr int kThreads = 256;

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// The buffers of a call, as a kernel argument: short for the few buffers of most
// calls (a launch copies its arguments twice: 3 KiB cost it about 1 us).
template <int N>
struct Buffers {
  const char* src[N];
  char* dst[N];
};

// Unit U, groups of up to KMAX rows.
template <typename U, int KMAX, int N>
__global__ __launch_bounds__(kThreads) void beam_reorder_kernel(BeamReorderArgs a, Buffers<N> buffers,
                                                                uint32_t units_per_block, uint32_t units,
                                                                int64_t groups) {
  const int K = a.beams, lane = threadIdx.x & 63;
  for (int64_t g = blockIdx.y; g < groups; g += gridDim.y) {
    // g = (state * outer + slab) * B + b
    const int b = (int)(g % a.B);
    const int64_t so = g / a.B;
    const int slab = (int)(so % a.from.outer), state = (int)(so / a.from.outer);
    // lane i holds parent i; bit i of moved: row i is written
    const int mine = lane < K ? a.parents[(int64_t)b * K + lane] : -1;
    const uint64_t moved = __ballot(mine >= 0 && mine < K && !(a.in_place && mine == lane));
    const char* src = buffers.src[state] + slab * a.from.outer_stride + (int64_t)b * K * a.from.row_stride;
    char* dst = buffers.dst[state] + slab * a.to.outer_stride + (int64_t)b * K * a.to.row_stride;
    for (uint32_t u = blockIdx.x * kThreads + threadIdx.x; u < units; u += gridDim.x * kThreads) {
      const uint32_t blk = u / units_per_block, off = u - blk * units_per_block;
      const int64_t s = (int64_t)blk * a.from.block_stride + (int64_t)off * sizeof(U);
      const int64_t d = (int64_t)blk * a.to.block_stride + (int64_t)off * sizeof(U);
      // computed anew for each unit: kept for all rows, the rows' conditions and
      // offsets would leave the scalar registers
      uint64_t rows = moved;
      int64_t from_row = a.from.row_stride, to_row = a.to.row_stride;
      asm volatile("" : "+s"(rows), "+s"(from_row), "+s"(to_row));
      U x[KMAX];
#pragma unroll
      for (int i = 0; i < KMAX; ++i)
        if ((rows >> i) & 1) x[i] = *reinterpret_cast<const U*>(src + __builtin_amdgcn_readlane(mine, i) * from_row + s);
      asm volatile("" : "+s"(rows));
#pragma unroll
      for (int i = 0; i < KMAX; ++i)
        if ((rows >> i) & 1) *reinterpret_cast<U*>(dst + i * to_row + d) = x[i];
    }
  }
}

template <typename U, int KMAX, int N>
hipError_t go(const BeamReorderArgs& a, const void* const* states, void* const* out, hipStream_t stream) {
  const int64_t per_block = a.from.block_bytes / (int64_t)sizeof(U);
  // a row's units are counted in 31 bits (units of 16 bytes: rows up to 32 GiB)
  if (per_block > 0x7FFFFFFF / a.from.blocks || a.from.outer > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const int64_t units = per_block * a.from.blocks;
  const int64_t groups = (int64_t)a.n_states * a.from.outer * a.B;
  int64_t gx = (units + kThreads - 1) / kThreads;
  if (gx > 65536) gx = 65536;
  const int64_t gy = groups < 65535 ? groups : 65535;
  Buffers<N> buffers;
  for (int i = 0; i < a.n_states; ++i) {
    buffers.src[i] = static_cast<const char*>(states[i]);
    buffers.dst[i] = static_cast<char*>(out[i]);
  }
  return launch(beam_reorder_kernel<U, KMAX, N>, dim3((unsigned)gx, (unsigned)gy), dim3(kThreads), 0, stream, a,
                buffers, (uint32_t)per_block, (uint32_t)units, groups);
}

// Units of 16 bytes for groups of up to 32 rows, 8 for more: what a thread
// holds leaves three waves per SIMD. Measured, 16 layers of 64 rows (as above):
// 8-byte units 2270 us (3.7 TB/s); 16-byte units, one wave per SIMD, 2981.
template <int N>
hipError_t by_unit(const BeamReorderArgs& a, uint64_t bits, const void* const* states, void* const* out,
                   hipStream_t stream) {
  if (bits % 16 == 0 && a.beams <= 4) return go<u32x4_t, 4, N>(a, states, out, stream);
  if (bits % 16 == 0 && a.beams <= 8) return go<u32x4_t, 8, N>(a, states, out, stream);
  if (bits % 16 == 0 && a.beams <= 16) return go<u32x4_t, 16, N>(a, states, out, stream);
  if (bits % 16 == 0 && a.beams <= 32) return go<u32x4_t, 32, N>(a, states, out, stream);
  if (bits % 8 == 0 && a.beams > 32) return go<u32x2_t, FS_BEAM_MAX, N>(a, states, out, stream);
  if (bits % 4 == 0)
    return a.beams <= 8 ? go<uint32_t, 8, N>(a, states, out, stream) : go<uint32_t, FS_BEAM_MAX, N>(a, states, out, stream);
  return a.beams <= 8 ? go<uint8_t, 8, N>(a, states, out, stream) : go<uint8_t, FS_BEAM_MAX, N>(a, states, out, stream);
}

}  // namespace

hipError_t launch_beam_reorder(const BeamReorderArgs& a, const void* const* states, void* const* out,
                               hipStream_t stream) {
  uint64_t bits = (uint64_t)(a.from.outer_stride | a.from.row_stride | a.from.block_stride | a.from.block_bytes |
                             a.to.outer_stride | a.to.row_stride | a.to.block_stride);
  for (int i = 0; i < a.n_states; ++i) bits |= (uint64_t)(uintptr_t)states[i] | (uint64_t)(uintptr_t)out[i];
  // units that every address and length is a multiple of
  return a.n_states <= 8 ? by_unit<8>(a, bits, states, out, stream)
                         : by_unit<FS_BEAM_MAX_STATES>(a, bits, states, out, stream);
}

}  // namespace fs
