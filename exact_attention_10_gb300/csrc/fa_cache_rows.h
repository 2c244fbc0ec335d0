// fa_cache_rows.h -- what fa_cache_rows.cu gives the other translation units:
// the weights of cached tokens for many query rows, and its status word.
#pragma once

#include <cuda_runtime.h>

#include "fa.h"

namespace fa {
namespace cache {
struct Params;
}
}  // namespace fa

namespace fa_launch {

fa_status launch_weights_rows(const fa::cache::Params &p, int D, bool bf16, int sms, cudaStream_t s, int dev);
unsigned int *status_word_rows();

}  // namespace fa_launch
