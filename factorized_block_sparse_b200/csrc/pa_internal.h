// Tile tables of a packing, shared by the host side and the kernels of
// libpacked_attn.so.  Not part of the public interface.
#pragma once

#include <cstdint>
#include <mutex>
#include <vector>

#include "packed_attn.h"

namespace pa {

constexpr int kTile = 128;  // rows of a query tile and of a key tile

// One launch slot: a tile of a sequence.
struct Slot {
  int32_t start;  // first row of the sequence
  int32_t len;    // its length
  int32_t tile;   // tile index inside the sequence (the kernel's own tile height)
  int32_t base;   // index of the sequence's first 128-row tile among all of them
};

struct DeviceTables {
  int device = -1;
  void* blob = nullptr;
  const Slot* fwd = nullptr;   // 128-row query tiles, longest key range first
  const Slot* fwd2 = nullptr;  // 256-row query tiles, longest key range first
  const Slot* bwd = nullptr;   // 128-row key tiles, longest query range first
};

}  // namespace pa

struct pa_layout {
  int64_t rows = 0;
  int64_t steps = 0;  // (query tile, key tile) pairs on or below the diagonal
  int64_t longest = 0;  // rows of the longest sequence
  std::vector<int32_t> lengths;
  std::vector<pa::Slot> fwd, fwd2, bwd;
  mutable std::mutex mu;
  mutable std::vector<pa::DeviceTables> dev;
};
