// The launch that has the shared and the own part of attention behind shared
// tokens at once.
#pragma once

#include "sv_attn.hpp"

namespace sv {

// False where the two are better (or only) launched one after the other.
bool launch_shared_and_own(const AttnArgs& a, const SharedPlan& p, int cache_dtype, hipStream_t stream);

}  // namespace sv
