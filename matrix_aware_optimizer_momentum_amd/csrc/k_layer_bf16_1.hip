// The feed-forward layers' products of bf16 operands, tiles of 64 x 64.
#include "k_layer_tile.hpp"

namespace sm {
namespace layer {

void launch_tile_bf16_1(const TileArgs& a, int grid, hipStream_t s) {
  launch_tile<bf16_t, 1>(a, grid, s);
}

}  // namespace layer
}  // namespace sm
