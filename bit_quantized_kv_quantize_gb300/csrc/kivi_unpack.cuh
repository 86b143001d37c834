// kivi_unpack.cuh -- 2- and 4-bit code fields to fp16 operands (shared by the
// kernels that read the packed cache).
#pragma once
#include <stdint.h>

namespace {

// Unpack field r of both 16-bit halves of w as fp16 (off + code).  The field
// is moved (by a shift shared between fields, or none) to a mantissa
// position p of an fp16 constant whose exponent makes bit p weigh 1, and
// or-ed into it: the value is 2^(10 - p) + code.
//   keys:   p in {4, 6, 8} (offsets 64, 16, 4); the accumulator carries
//           off * sum(q s), removed with the zero-point MMA's sum(q s) row;
//           against score-sized sums this costs < 1e-4 relative.
//   values: any p <= 8; the offset is subtracted in fp16 before the MMA
//           (exact), because the weighted value sums can be far smaller
//           than off * sum(p s).
struct View {
    int shl, shr;          // shift left / right applied to the word
    uint32_t mask, magic;  // field mask at its target position, fp16 pattern of the offset
    float off;
};
__host__ __device__ constexpr View at_pos(int p, int width, int shl, int shr) {
    // field of `width` bits at mantissa bit p; fp16 2^(10 - p) = exponent field 25 - p
    return View{shl, shr, (((1u << width) - 1u) << p) * 0x10001u, (uint32_t)(25 - p) * 0x04000400u,
                (float)(1 << (10 - p))};
}
template <int BITS, bool KEY>
__host__ __device__ constexpr View view_of(int r) {
    if (BITS == 4) {
        if (KEY)   // field bits [4r, 4r + 4) -> bits 6..9, offset 16
            return r <= 1 ? at_pos(6, 4, 6 - 4 * r, 0) : at_pos(6, 4, 0, 4 * r - 6);
        // values: slots 0, 1 in place (p = 0, 4); slots 2, 3 shifted to p = 4
        return r == 0 ? at_pos(0, 4, 0, 0) : (r == 1 ? at_pos(4, 4, 0, 0) : at_pos(4, 4, 0, 4 * r - 4));
    }
    // 2-bit field bits [2r, 2r + 2)
    if (KEY) {
        switch (r) {
        case 0: return at_pos(4, 2, 4, 0);
        case 1: return at_pos(6, 2, 4, 0);
        case 2: return at_pos(4, 2, 0, 0);
        case 3: return at_pos(6, 2, 0, 0);
        case 4: return at_pos(8, 2, 0, 0);
        case 5: return at_pos(4, 2, 0, 6);
        case 6: return at_pos(6, 2, 0, 6);
        default: return at_pos(8, 2, 0, 6);
        }
    }
    // values: slots 0..4 in place (p = 0, 2, 4, 6, 8); slots 5..7 via one shift
    return r <= 4 ? at_pos(2 * r, 2, 0, 0) : at_pos(2 * r - 6, 2, 0, 6);
}
// (x & mask) | magic as one lop3 with both constants as immediates; the
// plain C++ form compiles to two ALU instructions on this target.
template <uint32_t MASK, uint32_t MAGIC>
__device__ __forceinline__ uint32_t and_or(uint32_t x) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "n"(MASK), "n"(MAGIC));
    return r;
}
template <int BITS, bool KEY, int R>
__device__ __forceinline__ uint32_t unpack_t(uint32_t w) {
    constexpr View v = view_of<BITS, KEY>(R);
    const uint32_t x = v.shl ? (w << v.shl) : (v.shr ? (w >> v.shr) : w);
    return and_or<v.mask, v.magic>(x);
}
// runtime-looking slot index r (a constant once the caller's loops unroll)
template <int BITS, bool KEY>
__device__ __forceinline__ uint32_t unpack(uint32_t w, int r) {
    switch (r) {
    case 0: return unpack_t<BITS, KEY, 0>(w);
    case 1: return unpack_t<BITS, KEY, 1>(w);
    case 2: return unpack_t<BITS, KEY, 2>(w);
    case 3: return unpack_t<BITS, KEY, 3>(w);
    case 4: return unpack_t<BITS, KEY, (BITS == 2 ? 4 : 3)>(w);
    case 5: return unpack_t<BITS, KEY, (BITS == 2 ? 5 : 3)>(w);
    case 6: return unpack_t<BITS, KEY, (BITS == 2 ? 6 : 3)>(w);
    default: return unpack_t<BITS, KEY, (BITS == 2 ? 7 : 3)>(w);
    }
}
template <int BITS, bool KEY>
__host__ __device__ constexpr float slot_offset(int r) { return view_of<BITS, KEY>(r).off; }

}  // namespace
