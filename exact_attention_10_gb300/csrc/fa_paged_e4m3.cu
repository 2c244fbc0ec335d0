// fa_paged_e4m3.cu -- the paged attention's variants for caches held in 8 bits.
#include "fa_paged_launch.h"

namespace fa_launch {

fa_status launch_paged_e4m3(const fa::paged::Params &p, int D, bool bf16, int tile_rows, int grid, cudaStream_t s, int dev)
{
    return launch_paged_bits<8>(p, D, bf16, tile_rows, grid, s, dev);
}

}  // namespace fa_launch
