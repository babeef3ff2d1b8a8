// Tile kernel of the attention: when it is taken, and the instances without
// changed scores or masks. See attention_tiles.cuh.
#include "attention_tiles.cuh"

namespace sai {

bool attn_tiles_apply(int group, float scale_log2) { return group <= kTile && scale_log2 > 0.f; }

// Few rows, or short ones, are faster row by row: the row kernel reads every
// row's keys anew, but starts and joins in 5 us, where a unit of tiles takes 9 to
// start and end (and again for each request that meets in it). In us, from
// measurements of 4 to 256 rows of 100 to 16000 keys, 8 / 1, 4 / 4 and 64 / 8
// heads: 5 + 1 for each 9 MB of bf16 keys (5.5 MB of e4m3), against waves of
// 9 + 1.4 a key tile, or 28 and the even share of them when dealt out. A
// quarter is granted to the row kernel for requests that share a tile. 64 rows
// on 1000 keys, 8 / 1 heads: 12 us by rows, 22 by tiles; 64 / 8 heads: 44 and 22.
bool attn_tiles_pay(long long rows, int q_heads, int heads, int dim, bool f8, long long max_keys, int num_sms) {
  const int group = q_heads / heads;
  const Work w = work_of(rows, group, heads, dim, max_keys, num_sms);
  const double units = static_cast<double>(w.row_tiles) * heads, tiles = static_cast<double>((max_keys + kTile - 1) / kTile);
  const double tile_us = w.dealt ? 28 + units * tiles * 1.4 / w.shares : std::ceil(units / w.shares) * (9 + 1.4 * tiles);
  const double mb = static_cast<double>(rows) * heads * ((group + 63) / 64) * max_keys * 2e-6 * dim * (f8 ? 1 : 2);
  return 5 + mb / (f8 ? 5.5 : 9.0) > 1.25 * tile_us;
}

bool attn_tiles_fill(long long rows, int q_heads, int heads, int dim, int num_sms) {
  const Work w = work_of(rows, q_heads / heads, heads, dim, 0, num_sms);
  return static_cast<long long>(w.row_tiles) * heads >= w.shares;
}

size_t attn_tiles_workspace(long long rows, int q_heads, int heads, int dim, long long max_keys, int num_sms) {
  const int group = q_heads / heads;
  const Work w = work_of(rows, group, heads, dim, max_keys, num_sms);
  if (!w.dealt) return 0;
  return border_bytes(w) + static_cast<size_t>(2) * w.shares * w.rows_here * group * (static_cast<size_t>(dim) * 4 + 8);
}

cudaError_t launch_attn_tiles(const AttnLaunch& p, long long max_keys, void* workspace, int num_sms,
                              cudaStream_t stream) {
  if (p.modified) return launch_attn_tiles_mod(p, max_keys, workspace, num_sms, stream);
  return launch_tiles<0>(p, max_keys, workspace, num_sms, stream);
}

}  // namespace sai
