/* Host-side entry points to csrc/register_split.cuh for tests/test_linear_resources.py. */
#include "register_split.cuh"

extern "C" int split_suffices(int at_launch) { return tr::registers_suffice(at_launch) ? 1 : 0; }
