// What the host files of the C ABI share: the calling thread's error text
// (exl3_last_error) and the CU count that planning uses.
#pragma once

#include "../../include/exl3.h"

namespace exl3 {

// Records the message and returns s.
__attribute__((format(printf, 2, 3))) exl3_status host_fail(exl3_status s, const char *fmt, ...);
void host_clear_error();
// CUs of the current device; 256 (an MI355X) when none is visible.
int host_cus();

}  // namespace exl3
