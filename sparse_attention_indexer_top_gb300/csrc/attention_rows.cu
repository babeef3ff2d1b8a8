// Row kernel of the attention: its plan, and the instances without changed scores
// or masks. See attention_rows.cuh.
#include "attention_rows.cuh"

namespace sai {

AttnPlan attn_rows_plan(long long rows, int q_heads, int heads, int dim, bool f8, long long max_keys, int num_sms,
                        bool even_out) {
  const int group = q_heads / heads;
  const long long units = rows * heads * (group <= 64 ? 1 : (group + 63) / 64);
  // Chunks of at least 128 keys until a wave of CTAs (three per SM) is full:
  // one row of 700 keys takes 6.2 us with six chunks, 7.4 with three, 8.8 with
  // eleven. Past that only long rows are cut, in chunks of at least 512 keys, up
  // to eight waves, so that rows of unlike lengths even out and the last CTAs
  // are short: 64 rows of 4096-32768 keys, e4m3, take 379 us with eight waves,
  // 412 with four, 389 with sixteen.
  auto up = [](long long a, long long b) { return (a + b - 1) / b; };
  const long long wave = 3LL * num_sms;
  const long long fill = std::min(even_out ? up(wave, std::max(1LL, units)) : wave / std::max(1LL, units), up(max_keys, 128));
  const long long even = even_out ? std::min(up(8 * wave, std::max(1LL, units)), up(max_keys, 512)) : 1;
  const long long chunks = std::max(1LL, std::min(64LL, std::max(fill, even)));
  // a cluster only within the first wave: beyond it, waiting for as many free
  // places at once costs more than the second kernel (37 windowed rows: 67 us
  // clustered, 59 joined)
  AttnPlan pl{static_cast<int>(chunks), 0, false, chunks > 1 && chunks <= 8 && units * chunks <= wave, 2 * units * chunks <= wave};
  // enough units for every team to have its own: no joining
  const int teams = group <= 16 ? 4 : group <= 32 ? 2 : 1;
  pl.own = chunks == 1 && units >= 4LL * num_sms * teams;
  if (chunks > 1 && !pl.clustered)
    pl.workspace_bytes = static_cast<size_t>(rows) * q_heads * chunks * (static_cast<size_t>(dim) * 4 + 8);
  return pl;
}

cudaError_t launch_attn_rows(const AttnLaunch& p, cudaStream_t stream) {
  return p.modified ? launch_attn_rows_mod(p, stream) : launch_rows<false>(p, stream);
}

}  // namespace sai
