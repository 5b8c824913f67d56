// Host helpers shared by the files that implement C entry points: every entry
// point ends in one of these, so that sage_last_error() always holds the
// reason of the thread's last call.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sage.h"

namespace sage {

sage_status refuse(sage_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
sage_status succeeded();
sage_status cuda_refused(cudaError_t e, const char* what);
// SAGE_OK on a GB300, with *sms its multiprocessor count.
sage_status require_device(int* sms);
uint64_t device_wait_ns();

}  // namespace sage
