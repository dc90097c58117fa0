// 16-byte chunks of K-contiguous rows, read in place at any alignment: shared by
// the products that stream a weight for a few tokens.
#pragma once

#include "ffn.h"

namespace tgemm {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// Rows of K elements from which lanes read 16-byte chunks, zeros past K.
// AL: base and strides on 16-byte boundaries and K a multiple of 8; NT:
// non-temporal.
template <bool AL, bool NT>
struct ChunkRows {
  const char* base;
  int kb;  // bytes of K
#if defined(__HIP_DEVICE_COMPILE__)
  __amdgpu_buffer_rsrc_t rs;
#endif
  __device__ __forceinline__ void init(const char* b, int k_bytes) {
    base = b;
    kb = k_bytes;
#if defined(__HIP_DEVICE_COMPILE__)
    // (2^31 - 1 bytes, which no row of a workgroup passes: the host checks
    // the strides; a chunk past K takes an offset past it and reads as zero)
    if constexpr (AL)
      rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(b), (short)0, 0x7fffffff, 0x00020000);
#endif
  }
  __device__ __forceinline__ i32x4_t load(uint32_t row_off, int k) const {
    i32x4_t v = {0, 0, 0, 0};
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (AL) {
      const uint32_t ko = k < kb ? (uint32_t)k : 0x80000000u;
      v = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                          rs, (int)(row_off + ko), 0, NT ? kNonTemporal : 0));
    } else {
      const char* const s = base + row_off + k;
      if (k + 16 <= kb) {
        const u16x8_any a = *reinterpret_cast<const u16x8_any*>(s);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (int)a.w[i];
      } else if (k < kb) {
        // (loads that do not wait for each other)
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          e[i] = *reinterpret_cast<const uint16_t*>(s + (k + 2 * i < kb ? 2 * i : kb - 2 - k));
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + 2 * i < kb) v[i >> 1] |= (int)(e[i] << (16 * (i & 1)));
      }
    }
#endif
    return v;
  }
};

}  // namespace tgemm
