// Exposes the joining rule of the kernels' ops.h to the CPU tests.
#include "ops.h"

extern "C" bool merges_at_once(int64_t rows, int32_t sms) { return mla::merges_at_once(rows, sms); }
