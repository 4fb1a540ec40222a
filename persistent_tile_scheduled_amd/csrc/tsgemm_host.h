// Host helpers shared by the files that define the C ABI (tsgemm.hip,
// tsgemm_ops.hip).
#pragma once

namespace tsg {

// Clears the calling thread's last error; every entry point starts with it.
void reset_error();

// Keeps the message and the code for tsgemm_last_error and
// tsgemm_last_error_code of this thread, and returns the code.
int fail(int code, const char* fmt, ...);

}  // namespace tsg
