// attn_q4_0.hip - attention over a cache of type Q4_0.
#include "attn_kernel.hpp"

namespace qmv {

int launch_attn_q4_0(int nb, const AttnShape& s, const AttnArgs& a, hipStream_t st) {
  return launch_attn_kind<kKvQ4>(nb, s, a, st);
}

}  // namespace qmv
