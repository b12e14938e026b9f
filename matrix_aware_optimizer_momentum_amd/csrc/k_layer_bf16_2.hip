// The feed-forward layers' products of bf16 operands, tiles of 128 x 128.
#include "k_layer_tile.hpp"

namespace sm {
namespace layer {

void launch_tile_bf16_2(const TileArgs& a, int grid, hipStream_t s) {
  launch_tile<bf16_t, 2>(a, grid, s);
}

}  // namespace layer
}  // namespace sm
