// hqq_layers_skinny_pair.hip -- few rows by two weights of one shape (gate and up).
#include "hqq_layers_skinny.h"

namespace hqq {

hipError_t launch_skinny_pair(int nbits, bool bf16, const SkinnyArgs &s, hipStream_t st)
{
    return launch_skinny_nm<2>(nbits, bf16, s, st);
}

}  // namespace hqq
