// Checks of the device and of pointers that the C entry points share
// (defined in api.cu).
#pragma once
#include "moe_experts.h"

namespace bsmoe {

struct DevInfo {
  int id = -1, sms = 0, major = 0, minor = 0;
};
// The calling thread's device, refused unless it is one the kernels run on.
moe_status current_device(DevInfo* d);
// The pointer must be device (or managed) memory of device `dev`.
moe_status check_ptr(const void* p, int dev);

}  // namespace bsmoe
