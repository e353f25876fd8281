// Reordering of beam search's states (fs_beam_reorder): row i of a group
// becomes its former row parents[i], in every buffer and slab.
//
// Bound: memory. A thread owns one unit (16 bytes where all addresses allow)
// of all rows of a group: it reads the parents' units into registers, then
// writes them, so the rows may be permuted in place, with one parent taken by
// several rows, and no thread waits for another. In place, a row that is its
// own parent is neither read nor written.
#include "fs_decode.h"

namespace fs {
namespace {

constexpr int kThreads = 256;

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
  const int K = a.beams;
  for (int64_t g = blockIdx.y; g < groups; g += gridDim.y) {
    // g = (state * outer + slab) * B + b
    const int b = (int)(g % a.B);
    const int64_t so = g / a.B;
    const int slab = (int)(so % a.from.outer), state = (int)(so / a.from.outer);
    const int32_t* parents = a.parents + (int64_t)b * K;
    const char* src = buffers.src[state] + slab * a.from.outer_stride + (int64_t)b * K * a.from.row_stride;
    char* dst = buffers.dst[state] + slab * a.to.outer_stride + (int64_t)b * K * a.to.row_stride;
    for (uint32_t u = blockIdx.x * kThreads + threadIdx.x; u < units; u += gridDim.x * kThreads) {
      const uint32_t blk = u / units_per_block, off = u - blk * units_per_block;
      const char* s = src + (int64_t)blk * a.from.block_stride + (int64_t)off * sizeof(U);
      char* d = dst + (int64_t)blk * a.to.block_stride + (int64_t)off * sizeof(U);
      U x[KMAX];
#pragma unroll
      for (int i = 0; i < KMAX; ++i)
        if (i < K) {
          const int p = parents[i];
          if (p >= 0 && p < K && !(a.in_place && p == i))
            x[i] = *reinterpret_cast<const U*>(s + (int64_t)p * a.from.row_stride);
        }
#pragma unroll
      for (int i = 0; i < KMAX; ++i)
        if (i < K) {
          const int p = parents[i];
          if (p >= 0 && p < K && !(a.in_place && p == i))
            *reinterpret_cast<U*>(d + (int64_t)i * a.to.row_stride) = x[i];
        }
    }
  }
}

template <typename U, int KMAX, int N>
hipError_t go(const BeamReorderArgs& a, const void* const* states, void* const* out, hipStream_t stream) {
  const int64_t per_block = a.from.block_bytes / (int64_t)sizeof(U);
  // a row's units are counted in 31 bits (16-byte units: rows up to 32 GiB)
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

template <typename U, int N>
hipError_t by_beams(const BeamReorderArgs& a, const void* const* states, void* const* out, hipStream_t stream) {
  if (a.beams <= 4) return go<U, 4, N>(a, states, out, stream);
  if (a.beams <= 8) return go<U, 8, N>(a, states, out, stream);
  if (a.beams <= 16) return go<U, 16, N>(a, states, out, stream);
  return go<U, 64, N>(a, states, out, stream);
}

template <typename U>
hipError_t by_states(const BeamReorderArgs& a, const void* const* states, void* const* out, hipStream_t stream) {
  return a.n_states <= 8 ? by_beams<U, 8>(a, states, out, stream)
                         : by_beams<U, FS_BEAM_MAX_STATES>(a, states, out, stream);
}

}  // namespace

hipError_t launch_beam_reorder(const BeamReorderArgs& a, const void* const* states, void* const* out,
                               hipStream_t stream) {
  uint64_t bits = (uint64_t)(a.from.outer_stride | a.from.row_stride | a.from.block_stride | a.from.block_bytes |
                             a.to.outer_stride | a.to.row_stride | a.to.block_stride);
  for (int i = 0; i < a.n_states; ++i) bits |= (uint64_t)(uintptr_t)states[i] | (uint64_t)(uintptr_t)out[i];
  // the widest unit that every address and length is a multiple of
  if (bits % 16 == 0) return by_states<uint4>(a, states, out, stream);
  if (bits % 4 == 0) return by_states<uint32_t>(a, states, out, stream);
  return by_states<uint8_t>(a, states, out, stream);
}

}  // namespace fs
