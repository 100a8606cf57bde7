// attn_q8_0.hip - attention over a cache of type Q8_0.
#include "attn_kernel.hpp"

namespace qmv {

int launch_attn_q8_0(int nb, const AttnShape& s, const AttnArgs& a, hipStream_t st) {
  return launch_attn_kind<kKvQ8>(nb, s, a, st);
}

}  // namespace qmv
