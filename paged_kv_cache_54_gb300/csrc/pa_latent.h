// Host-side checks shared by the latent cache's entry points.
#pragma once

#include <limits.h>

#include "pa_host.h"

namespace pa {

constexpr int kLatentDim = 512;  // of a token's latent vector, which is also its value
constexpr int kRopeDim = 64;     // of its rotary key
constexpr int kLatentRow = kLatentDim + kRopeDim;

inline bool valid_latent_desc(const pa_latent_desc *c) {
  return c != nullptr && c->num_blocks > 0 && c->block_size > 0 && c->latent_dim > 0 && c->rope_dim > 0;
}
inline bool supported_latent_desc(const pa_latent_desc *c) {
  return (c->block_size == 8 || c->block_size == 16 || c->block_size == 32) && c->latent_dim == kLatentDim &&
         c->rope_dim == kRopeDim && (c->dtype == PA_F16 || c->dtype == PA_BF16) &&
         static_cast<long long>(c->num_blocks) * c->block_size <= INT_MAX;  // 32-bit rows
}
inline int log2_block(int bs) { return bs == 8 ? 3 : bs == 16 ? 4 : 5; }

// [row groups, 128-byte column, row, 64 elements] view of a latent cache
// (nine 128-byte columns a row, groups of 8 rows).  A box of `columns`
// columns and `groups` groups lands group by group, each group column by
// column, as 8-row x 128-byte atoms with the 128-byte swizzle.
bool encode_latent_view(CUtensorMap *map, const void *cache, const pa_latent_desc *c, int columns, int groups);

}  // namespace pa
