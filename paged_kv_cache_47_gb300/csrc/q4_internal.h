// Checks shared by the 4-bit cache's translation units.
#pragma once

#include "../../include/pkv_q4.h"

namespace pkv {

pkv_status check_q4cache(const pkv_q4cache_desc *c);
pkv_status check_q4pools(const pkv_q4cache_pools *pools);

}  // namespace pkv
