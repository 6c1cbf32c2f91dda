// What the attention-layer sources need of the rest of the library, for the tests that build
// them by themselves with a shorter limit of their waits.
#include "ar_internal.h"

int arf::set_last_error(int code, const char*) { return code; }
