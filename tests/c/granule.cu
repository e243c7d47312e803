/* Host-side walk of the 16-byte copies that the quantizer makes of bf16 rows off
 * 16-byte boundaries (csrc/granule.cuh).  Built as a host-only shared library by
 * tests/test_granule.py; no device code runs. */
#include "granule.cuh"

extern "C" {

/* Every tile of 128 columns of a row takes the 17 granules from the boundary at or
 * below its first column on.  Counts what an asynchronous copy may not do -- take its
 * bytes from off a 16-byte boundary, from outside the row, or more than 16 -- and adds
 * to `taken` the row's bytes that copies take. */
long long granule_faults(unsigned long long base, long long rows, long long cols, long long ld, long long *taken) {
    const __nv_bfloat16 *x = reinterpret_cast<const __nv_bfloat16 *>(uintptr_t(base));
    long long faults = 0;
    for (long long r = 0; r < rows; ++r) {
        const __nv_bfloat16 *row = x + r * ld;
        for (long long c0 = 0; c0 < cols; c0 += 128)
            for (int g = 0; g < 17; ++g) {
                const long long col = c0 + g * 8 - int(tr::granule_shift(row + c0) / 2);
                if (col < 0) continue; /* the row begins inside it: taken value by value */
                const tr::GranulePart p = tr::granule_part(row, col, cols);
                const uintptr_t a = reinterpret_cast<uintptr_t>(p.src), lo = reinterpret_cast<uintptr_t>(row);
                if (!p.src && p.bytes == 0) continue; /* no copy */
                if (a % 16 || p.bytes < 0 || p.bytes > 16 || a < lo || a + p.bytes > lo + 2 * cols) ++faults;
                if (g < 16) *taken += p.bytes;
            }
    }
    return faults;
}

}  /* extern "C" */
