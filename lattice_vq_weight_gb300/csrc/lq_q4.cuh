// The 4-bit format of the paged cache, shared by the kernels that write, read
// and attend to it (lq_kv_q4.cu, lq_attn_q4.cu).  Internal to the library.
//
// A head's vector is cut into groups of neighbouring dimensions, each with an
// fp16 scale s and an fp16 base b; a code c of 0 .. 15 stands for
//     fp16(fma(16 + c, s, b)).
// 0x4C00 is 16 in fp16 and its last place is 2^-6, so 0x4C00 | c << 6 is 16 + c:
// one logic operation puts two codes into place and one packed fp16 fma makes
// their values, which are then exact operands of the matrix products.  The price
// is a base that reaches past the least value by 16 steps: its rounding, up to
// 2^-11 (|least| + 16 s), shifts the grid.  Near zero that is a hundredth of a step, for
// |least| of a thousand steps half of one, and beyond that codes are cut at the grid's
// ends.  Codes are chosen on the grid as stored.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace lq {
namespace q4 {

constexpr float kMost = 16384.f;               // larger values are cut: base and scale stay in fp16's range

// Codes j and j + 4 (j = 0 .. 3) of a word of eight as fp16 numbers 16 + c.
template <int J>
__device__ __forceinline__ uint32_t pair(uint32_t word) {
  const uint32_t at = J == 0 ? word << 6 : J == 1 ? word << 2 : J == 2 ? word >> 2 : word >> 6;
  return (at & 0x03C003C0u) | 0x4C004C00u;
}

// The same with the two constants in registers: an instruction takes one constant,
// so that the above is two where this is one (311 of 1476 instructions of a tile
// were logic, 128 of them for this).
struct Masks {
  uint32_t field, sixteen;
  __device__ __forceinline__ Masks() {
    asm volatile("mov.u32 %0, 0x03C003C0;\n mov.u32 %1, 0x4C004C00;" : "=r"(field), "=r"(sixteen));
  }
  template <int J>
  __device__ __forceinline__ uint32_t pair(uint32_t word) const {
    const uint32_t at = J == 0 ? word << 6 : J == 1 ? word << 2 : J == 2 ? word >> 2 : word >> 6;
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(at), "r"(field), "r"(sixteen));      // (a & b) | c
    return v;
  }
};

// Both halves of a word as one half-pair: scale (low) and base (high) of a group.
__device__ __forceinline__ uint32_t twice_low(uint32_t x) { return __byte_perm(x, x, 0x1010); }
__device__ __forceinline__ uint32_t twice_high(uint32_t x) { return __byte_perm(x, x, 0x3232); }

__device__ __forceinline__ uint32_t fma_h2(uint32_t a, uint32_t s, uint32_t b) {
  const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&s),
                            *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The eight values of a word, in order, for one group's (scale, base).
__device__ __forceinline__ void values8(uint32_t word, uint32_t scale_base, float (&v)[8]) {
  const uint32_t s = twice_low(scale_base), b = twice_high(scale_base);
  const uint32_t h[4] = {fma_h2(pair<0>(word), s, b), fma_h2(pair<1>(word), s, b), fma_h2(pair<2>(word), s, b),
                         fma_h2(pair<3>(word), s, b)};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    v[j] = f.x;
    v[j + 4] = f.y;
  }
}

// ------------------------------------------------------------------ host
inline bool valid_dims(int head_dim, int group_size) {
  return (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
         (group_size == 32 || group_size == 64 || group_size == 128) && group_size <= head_dim;
}

}  // namespace q4
}  // namespace lq
