// Plan of a packed batch: sequences of different lengths whose rows lie one behind the
// other.  Host only: the caller copies the filled plan to the device once, and every
// packed call on the batch (attention and its gradients, the preference loss) reads it there.
#include <algorithm>
#include <cstring>
#include <new>
#include <vector>

#include "internal.h"

namespace nf4ls {

int check_pack(const nf4ls_pack* p, const char* who) {
  if (!p) return fail(NF4LS_INVALID_ARG, "%s: null pack", who);
  if (p->n_seqs < 1 || p->total < 0 || p->n_tiles < 0 || p->max_len < 0 || p->n_tiles > p->total ||
      (p->total > 0) != (p->n_tiles > 0) || p->n_blocks < p->n_tiles)
    return fail(NF4LS_INVALID_ARG, "%s: not a pack that nf4ls_pack_layout filled", who);
  if (!p->plan_dev) return fail(NF4LS_INVALID_ARG, "%s: the pack has no plan on the device", who);
  if (!aligned(p->plan_dev, 256)) return fail(NF4LS_ALIGN, "%s: the plan must be 256-byte aligned", who);
  return NF4LS_OK;
}

}  // namespace nf4ls

using namespace nf4ls;

extern "C" int nf4ls_pack_layout(const int32_t* lengths_host, int32_t n_seqs, nf4ls_pack* out) {
  clear_error();
  if (!lengths_host || !out) return fail(NF4LS_INVALID_ARG, "nf4ls_pack_layout: null argument");
  if (n_seqs < 1 || n_seqs > NF4LS_PACK_MAX_SEQS)
    return fail(NF4LS_INVALID_ARG, "nf4ls_pack_layout: %d sequences, 1 to %d are supported", n_seqs, NF4LS_PACK_MAX_SEQS);
  int64_t total = 0, tiles = 0, blocks = 0;
  int32_t longest = 0;
  for (int32_t i = 0; i < n_seqs; ++i) {
    if (lengths_host[i] < 0) return fail(NF4LS_INVALID_ARG, "nf4ls_pack_layout: sequence %d has length %d", i, lengths_host[i]);
    total += lengths_host[i];
    if (total > NF4LS_PACK_MAX_ROWS)
      return fail(NF4LS_INVALID_ARG, "nf4ls_pack_layout: more than %d rows", NF4LS_PACK_MAX_ROWS);
    const int64_t n = (lengths_host[i] + 127) / 128;
    tiles += n;
    blocks += n * (n + 1) / 2;
    longest = std::max(longest, lengths_host[i]);
  }
  std::memset(out, 0, sizeof(*out));
  out->n_seqs = n_seqs;
  out->total = (int32_t)total;
  out->n_tiles = (int32_t)tiles;
  out->max_len = longest;
  out->n_blocks = blocks;
  uint64_t off = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t o = off;
    off = round_up(off + bytes, 256);
    return o;
  };
  out->off_cu = take(4ull * (n_seqs + 1));
  out->off_positions = take(4ull * total);
  out->off_seq = take(4ull * total);
  out->off_query_tiles = take(16ull * tiles);
  out->off_key_tiles = take(16ull * tiles);
  out->plan_bytes = off;
  return NF4LS_OK;
}

extern "C" int nf4ls_pack_fill(const int32_t* lengths_host, const nf4ls_pack* pack, void* plan_host, size_t bytes) {
  clear_error();
  if (!lengths_host || !pack || !plan_host) return fail(NF4LS_INVALID_ARG, "nf4ls_pack_fill: null argument");
  nf4ls_pack want;
  NF4_TRY(nf4ls_pack_layout(lengths_host, pack->n_seqs, &want));
  if (want.total != pack->total || want.n_tiles != pack->n_tiles || want.plan_bytes != pack->plan_bytes)
    return fail(NF4LS_INVALID_ARG, "nf4ls_pack_fill: the lengths are not those of the pack");
  if (bytes < want.plan_bytes)
    return fail(NF4LS_INVALID_ARG, "nf4ls_pack_fill: %zu bytes, the plan needs %llu", bytes,
                (unsigned long long)want.plan_bytes);
  uint8_t* base = static_cast<uint8_t*>(plan_host);
  std::memset(base, 0, want.plan_bytes);
  auto* cu = reinterpret_cast<int32_t*>(base + want.off_cu);
  auto* pos = reinterpret_cast<int32_t*>(base + want.off_positions);
  auto* seq = reinterpret_cast<int32_t*>(base + want.off_seq);
  try {
    std::vector<PackTile> tiles;
    tiles.reserve((size_t)want.n_tiles);
    int32_t row = 0;
    for (int32_t s = 0; s < want.n_seqs; ++s) {
      cu[s] = row;
      const int32_t n = lengths_host[s];
      for (int32_t i = 0; i < n; ++i) {
        pos[row + i] = i;
        seq[row + i] = s;
      }
      for (int32_t t = 0; t * 128 < n; ++t) tiles.push_back(PackTile{row, n, t, (int32_t)tiles.size()});
      row += n;
    }
    cu[want.n_seqs] = row;
    // A query tile reads the key tiles up to its own, a key tile the query tiles from its
    // own on: both lists start with the longest, so that the last wave holds short ones.
    std::stable_sort(tiles.begin(), tiles.end(), [](const PackTile& a, const PackTile& b) { return a.tile > b.tile; });
    if (!tiles.empty()) std::memcpy(base + want.off_query_tiles, tiles.data(), tiles.size() * sizeof(PackTile));
    auto left = [](const PackTile& a) { return (a.len + 127) / 128 - a.tile; };
    std::stable_sort(tiles.begin(), tiles.end(), [&](const PackTile& a, const PackTile& b) { return left(a) > left(b); });
    if (!tiles.empty()) std::memcpy(base + want.off_key_tiles, tiles.data(), tiles.size() * sizeof(PackTile));
  } catch (const std::bad_alloc&) {
    return fail(NF4LS_INVALID_ARG, "nf4ls_pack_fill: out of host memory");
  }
  return NF4LS_OK;
}
