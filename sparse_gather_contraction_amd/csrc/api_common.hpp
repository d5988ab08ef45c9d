// api_common.hpp — what the files of the C ABI share: the last error and the device check.
#pragma once

#include <string>

#include "disco.h"

namespace disco {

// Keeps `msg` for disco_last_error() on this thread and returns `s`.
disco_status api_fail(disco_status s, const std::string &msg);
// DISCO_ERR_OOM with a message that needs no allocation.
disco_status api_fail_oom() noexcept;
// DISCO_OK where `device` is one that the library runs on.
disco_status api_check_device(int device);

}  // namespace disco
