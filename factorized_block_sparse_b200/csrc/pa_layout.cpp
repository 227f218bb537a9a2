// Host side of a packing: lengths -> launch slots of the query and key tiles.
#include <algorithm>
#include <new>

#include "pa_internal.h"

namespace {

using pa::kTile;
using pa::Slot;

// Every tile of `height` rows of every sequence; base counts 128-row tiles.
std::vector<Slot> tiles_of(const std::vector<int32_t>& lengths, int height) {
  std::vector<Slot> out;
  int64_t start = 0, base = 0;
  for (int32_t n : lengths) {
    for (int32_t t = 0; t < (int64_t(n) + height - 1) / height; ++t)
      out.push_back(Slot{static_cast<int32_t>(start), n, t, static_cast<int32_t>(base)});
    start += n;
    base += (int64_t(n) + kTile - 1) / kTile;
  }
  return out;
}

int32_t tiles128(const Slot& s) { return static_cast<int32_t>((int64_t(s.len) + kTile - 1) / kTile); }

}  // namespace

extern "C" int packed_attn_layout(const int32_t* lengths, int n_seqs, pa_layout** out) {
  if (!out || n_seqs < 0 || (n_seqs > 0 && !lengths)) return SA_ERR_INVALID_ARG;
  *out = nullptr;
  int64_t rows = 0;
  for (int i = 0; i < n_seqs; ++i) {
    if (lengths[i] < 0) return SA_ERR_INVALID_ARG;
    rows += lengths[i];
    if (rows > (int64_t(1) << 31) - 1024) return SA_ERR_INVALID_ARG;  // row numbers of a whole last tile stay in 31 bits
  }
  try {
    pa_layout* L = new pa_layout;
    *out = L;
    L->rows = rows;
    if (n_seqs > 0) L->lengths.assign(lengths, lengths + n_seqs);
    L->fwd = tiles_of(L->lengths, kTile);
    L->fwd2 = tiles_of(L->lengths, 2 * kTile);
    L->bwd = L->fwd;
    for (const Slot& s : L->fwd) L->steps += s.tile + 1;
    for (int32_t n : L->lengths) L->longest = std::max<int64_t>(L->longest, n);
    // a query tile meets tile + 1 key tiles, a key tile the query tiles from its own to the last
    auto by_tile = [](const Slot& a, const Slot& b) { return a.tile > b.tile; };
    std::stable_sort(L->fwd.begin(), L->fwd.end(), by_tile);
    std::stable_sort(L->fwd2.begin(), L->fwd2.end(), by_tile);
    std::stable_sort(L->bwd.begin(), L->bwd.end(),
                     [](const Slot& a, const Slot& b) { return tiles128(a) - a.tile > tiles128(b) - b.tile; });
  } catch (...) {  // out of host memory: nothing crosses the C boundary
    delete *out;
    *out = nullptr;
    return SA_ERR_INVALID_ARG;
  }
  return SA_OK;
}

extern "C" int64_t packed_attn_layout_rows(const pa_layout* layout) { return layout ? layout->rows : -1; }
