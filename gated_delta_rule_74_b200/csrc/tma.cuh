// Host-side TMA tensor maps for the kernels' tile loads (not part of the C ABI).
// The driver's encoder is reached through the runtime's entry-point query, so the
// library links no driver library.  Every map covers this GPU's own memory and is
// used by plain tile loads only (no cluster multicast).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

// A 3-D tiled map over a [d2][d1][d0] tensor (d0 contiguous; strides in bytes for
// d1 and d2), with boxes of box0 x 1 x box2 elements.  swizzle128: the 128-byte
// swizzle of the tensor cores' shared-memory operands (box0 * element size must
// then be 128).  Returns false if the driver rejects the map (the caller falls
// back to plain loads).
bool make_tile_map_3d(CUtensorMap* map, bool fp32, const void* base, uint64_t d0, uint64_t d1,
                      uint64_t d2, uint64_t stride1, uint64_t stride2, uint32_t box0,
                      uint32_t box2, bool swizzle128);

// A 4-D bf16 map that brings `box_rows` rows of `box_chunks` 64-column chunks in one box,
// chunk after chunk, each [box_rows][128 B] with the 128-byte swizzle (the K-major operand
// layout).  The tensor: [outer][rows][64 * chunks] with row and outer strides in bytes.
bool make_chunk_map_4d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t chunks,
                       uint64_t outer, uint64_t row_stride, uint64_t outer_stride,
                       uint32_t box_rows, uint32_t box_chunks);

}  // namespace kda
