// Host functions of moe_api.cu that the operators around the experts (router.cu,
// mx_quant.cu, expert_product.cu) launch with.
#pragma once

namespace crs {

// SMs of the current device (0 when the query fails); cached per device.
int num_sms_of_current_device();
// n more kernels were enqueued (moe_launch_count).
void note_launches(int n);

}  // namespace crs
