// bf16 rows to 4-bit pages (sm_103a device helpers shared by the append
// kernels); the format stands in kv4_kernels.cu.
#pragma once
#include <cstdint>

namespace kvp {
namespace {

__device__ __forceinline__ float bf16_bits_to_float(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// e = smallest integer with m <= 7 * 2^e for m > 0, clamped to [-127, 127]:
// m in [2^E, 2^(E+1)) needs e = E - 2 when m <= 1.75 * 2^E, else E - 1 (both
// sides exact in fp32).
__device__ __forceinline__ int row_exponent(float m) {
    if (!(m > 0.f)) return -127;
    int E;
    const float f = frexpf(m, &E);   // m = f * 2^E, f in [0.5, 1)
    E -= 1;                          // m in [2^E, 2^(E+1))
    const int e = (f * 2.f <= 1.75f) ? E - 2 : E - 1;
    return max(-127, min(127, e));
}

// A warp stores one row of d = 32 * vpl values, lane i holding values vpl * i
// on: the exponent from the row's largest, then the codes.
__device__ __forceinline__ void store_row4(const float (&x)[4], int vpl, uint8_t *codes, int8_t *exp, int lane) {
    uint32_t amax = 0;
    for (int j = 0; j < vpl; ++j) amax = max(amax, __float_as_uint(fabsf(x[j])));
    amax = __reduce_max_sync(0xffffffffu, amax);   // |x| bit patterns order like the values
    const int e = row_exponent(__uint_as_float(amax));
    uint32_t packed = 0;
    for (int j = 0; j < vpl; ++j) {
        const float c = fminf(7.f, fmaxf(-7.f, rintf(ldexpf(x[j], -e))));
        packed |= ((uint32_t)(int)c & 0xFu) << (4 * j);
    }
    if (vpl == 2) {
        codes[lane] = (uint8_t)packed;
    } else {
        reinterpret_cast<uint16_t *>(codes)[lane] = (uint16_t)packed;
    }
    if (lane == 0) *exp = (int8_t)e;
}

}  // namespace
}  // namespace kvp
