// mpgemm_handle.hpp -- what a handle holds, for the parts of the C ABI that launch kernels.
#pragma once

#include "mpgemm.h"

struct mpgemm_handle_s {
    int device;
    int num_cus;
    void *scratch;   // the device's address of the fixed scratch buffer, or nullptr
};

namespace mpg_host {

// The handle was created and has not been destroyed.
bool handle_live(mpgemm_handle_t handle);
// SUCCESS when the current device is the handle's.
mpgemm_status_t handle_on_device(mpgemm_handle_t handle);

}  // namespace mpg_host
