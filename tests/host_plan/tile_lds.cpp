// Every workgroup of k_block_tiles against the LDS of a CU: all instances, group
// sizes, selection lengths and numbers of blocks.
#include <cstdio>

#include "block_plan.hpp"

using namespace msgla;

int main() {
  long cases = 0, over = 0, ring = 0;
  for (int es = 2; es <= 4; es += 2)
    for (int dkp = 64; dkp <= 128; dkp *= 2)
      for (int dvp = 64; dvp <= 256; dvp *= 2)
        for (int gradient = 0; gradient < 2; ++gradient)
          for (int block = 32; block <= 64; block *= 2)
            for (int many = 0; many < 2; ++many)
              for (int group = 1; group <= 33; ++group)  // 16 and fewer heads share a tile; 17 .. 32 take two, 33 three
                for (int n = 1; n <= BLK_MAX_SEL; ++n)
                  for (int words = 1; words <= BLK_TILES_MAX / 32; ++words) {
                    const TileShape s = tile_shape(es, dkp, dvp, gradient, block, many);
                    const int stage = tile_stage(s, es, dkp, dvp);
                    const int qt = group <= BLK_ROWS ? BLK_ROWS / group : 1;
                    const int gt = group <= BLK_ROWS ? 1 : (group + BLK_ROWS - 1) / BLK_ROWS;
                    const TileLds l = tile_lds(s, stage, words * 32, n, qt, gt);
                    const int limit = tile_lds_limit(s.tiles);
                    ++cases;
                    if (l.bytes + 128 > limit && ++over <= 3)
                      std::printf("over: element %d heads %d/%d gradient %d block %d tiles %d group %d n %d words %d: %d of %d\n", es,
                                  dkp, dvp, gradient, block, s.tiles, group, n, words, l.bytes, limit);
                    // a ring of two stages, where the queries' raw rows of 32-bit entries fit first
                    const int queries = gt > 1 ? s.tiles / gt + 2 : s.tiles * qt;
                    if (l.stages < 2 || queries * n * 4 > l.stages * stage) ++ring;
                  }
  std::printf("%ld cases, %ld over, %ld without a ring\n", cases, over, ring);
  return over || ring ? 1 : 0;
}
