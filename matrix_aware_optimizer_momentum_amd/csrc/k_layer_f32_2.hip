// The feed-forward layers' products of f32 operands, tiles of 128 x 128.
#include "k_layer_tile.hpp"

namespace sm {
namespace layer {

void launch_tile_f32_2(const TileArgs& a, int grid, hipStream_t s) {
  launch_tile<float, 2>(a, grid, s);
}

}  // namespace layer
}  // namespace sm
