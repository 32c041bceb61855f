// What every C entry point that launches kernels shares: the launch-failure
// injection and this thread's last HIP error.  Host only; the kernels do not
// include it.
#pragma once

#include <hip/hip_runtime.h>

#include "ar.h"

namespace ar {

// Takes one from an armed ar_debug_fail_launch counter; true if the launch
// about to be made is the one that has to fail.
bool take_launch_failure();

// Keeps `err` for ar_last_hip_error() on this thread; AR_ERROR_HIP for an
// error, AR_SUCCESS for hipSuccess.
ar_status_t launch_status(hipError_t err);

// Makes one launch, or reports the injected failure in its place.
template <class F>
hipError_t enqueue(F&& launch_fn) {
  if (take_launch_failure()) return hipErrorLaunchFailure;
  return launch_fn();
}

}  // namespace ar
