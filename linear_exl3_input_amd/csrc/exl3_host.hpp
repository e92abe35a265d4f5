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

// Held over a call's launches on its workspace (null: none), so that those of
// other host threads' calls with the same one do not come between them: what a
// launch leaves there is for the call's next.
class WorkspaceTurn {
 public:
  explicit WorkspaceTurn(const void *workspace);
  ~WorkspaceTurn();
  WorkspaceTurn(const WorkspaceTurn &) = delete;
  WorkspaceTurn &operator=(const WorkspaceTurn &) = delete;

 private:
  const int turn_;  // -1: none
};

}  // namespace exl3
