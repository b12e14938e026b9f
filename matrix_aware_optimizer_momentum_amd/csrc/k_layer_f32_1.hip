// The feed-forward layers' products of f32 operands, tiles of 64 x 64.
#include "k_layer_tile.hpp"

namespace sm {
namespace layer {

void launch_tile_f32_1(const TileArgs& a, int grid, hipStream_t s) {
  launch_tile<float, 1>(a, grid, s);
}

}  // namespace layer
}  // namespace sm
