// attn_f16.hip - attention over a cache of type F16.
#include "attn_kernel.hpp"

namespace qmv {

int launch_attn_f16(int nb, const AttnShape& s, const AttnArgs& a, hipStream_t st) {
  return launch_attn_kind<kKvF16>(nb, s, a, st);
}

}  // namespace qmv
