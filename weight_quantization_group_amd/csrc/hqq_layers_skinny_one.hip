// hqq_layers_skinny_one.hip -- few rows by one weight (the quantized head).
#include "hqq_layers_skinny.h"

namespace hqq {

hipError_t launch_skinny(int nbits, bool bf16, const SkinnyArgs &s, hipStream_t st)
{
    if (s.out == kOutGated || s.out == kOutGatedGrad)
        return launch_skinny_pair(nbits, bf16, s, st);
    return launch_skinny_nm<1>(nbits, bf16, s, st);
}

}  // namespace hqq
