// status.h -- bits of the device status word that fp8_status_query reads.
#pragma once
#include <cstdint>

namespace bsfp8 {

enum : uint32_t { STATUS_TIMEOUT = 1u, STATUS_SCALE = 2u, STATUS_RECORD = 4u };

}  // namespace bsfp8
