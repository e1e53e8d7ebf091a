// Constants of the microscaled (MX) formats, host and device.
#pragma once

#include <stdint.h>

namespace awq {

constexpr int kMxBlock = 32;
constexpr int kMxFp8 = 0, kMxFp4 = 1;  // element formats (AWQ_MX_FP8, AWQ_MX_FP4)
constexpr uint32_t kMxNan = 255;

}  // namespace awq
