// What every entry point returns: a status, and the calling thread's last error
// message beside it (ivfpq_last_error).
#pragma once

#include "../../include/ivfpq.h"

#include <string>

namespace ivfpq {

ivfpq_status fail(ivfpq_status s, const std::string &msg);
ivfpq_status ok();

} // namespace ivfpq
