// The layout of the 4-bit pages (include/gdn.h): offsets inside the block that
// holds one head of one page, 72 d bytes.
#pragma once

#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {
namespace kv4 {

constexpr int kPage = GDN_PAGE_TOKENS;  // tokens of a page
constexpr int kGroup = 16;              // channels that share a scale

__host__ __device__ constexpr int block_bytes(int d) { return 72 * d; }
// Sections of a block: codes of K and V, scales of K and V.
__host__ __device__ constexpr int codes_at(int d, int kind) { return 32 * d * kind; }
__host__ __device__ constexpr int scales_at(int d, int kind) { return 64 * d + 4 * d * kind; }
// Where byte `offset` of a block of codes stands.
__host__ __device__ constexpr int swizzle(int offset) { return offset ^ (((offset >> 7) & 7) << 4); }

}  // namespace kv4
}  // namespace gdn
