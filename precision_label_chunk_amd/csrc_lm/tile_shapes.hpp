// Which tile shape a tiled product takes (host side): the time that each is expected to take.
#pragma once
#include "lm_kernels.hpp"
#include "tile_product.hpp"

namespace elmo {

static inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// What a unit of a shape takes, in us: its start and its results (`ends`), and a stage with the device nearly empty
// (`alone`) and full (`full`; in between in proportion to the blocks). Fitted to timings between 1 x 1,000 x 64 and
// 4,096 x 131,072 x 4,096; by them the small shape is up to three times faster than the large one at 512 x 1,000
// x 256 (4.5 against 11.9 us for the logits), and 2.4 times slower at 4,096 x 32,768 x 768.
struct ShapeCost { int size, blocks; double ends, alone, full; };
constexpr int SHAPE_COUNT = 3;
static const ShapeCost SHAPES[SHAPE_COUNT] = {{LargeTiles::M, LargeTiles::BLOCKS, 5.5, 0.5, 0.8},
                                              {MediumTiles::M, MediumTiles::BLOCKS, 3.5, 0.25, 0.54},
                                              {SmallTiles::M, SmallTiles::BLOCKS, 2.5, 0.17, 0.6}};

static inline double stage_time(const ShapeCost& c, int64_t units, int cus) {
  const double most = (double)cus * c.blocks, share = (double)units / most;
  return c.alone + (c.full - c.alone) * (share < 1.0 ? share : 1.0);
}
static inline double units_time(const ShapeCost& c, int64_t units, int64_t stages, double stage, int cus) {
  // (a last round that is not full ends sooner: the clock rises)
  const double blocks = (double)cus * c.blocks, rounds = (double)units / blocks, whole = (double)ceil_div(units, (int64_t)cus * c.blocks);
  return (rounds < 1.0 ? 1.0 : 0.5 * (rounds + whole)) * (c.ends + (double)stages * stage);
}
static inline unsigned blocks_for(int shape, int64_t units, int cus) {
  const int64_t most = (int64_t)cus * SHAPES[shape].blocks;
  return (unsigned)(units < most ? units : most);
}
// f(shape) for the shape of a number
template <class F>
static void with_shape(int shape, F&& f) {
  if (shape == 0) f(LargeTiles{});
  else if (shape == 1) f(MediumTiles{});
  else f(SmallTiles{});
}

}  // namespace elmo
