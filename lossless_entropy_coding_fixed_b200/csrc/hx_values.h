// Device helpers of the 8-bit-row kernels (private to the library): element types, the scale and
// byte of a value, and loads and stores of W consecutive elements.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "hx.h"

namespace hxv {

// ------------------------------------------------------------------------------ element types
template <typename T>
struct Type;
template <>
struct Type<float> {
  static constexpr uint32_t kInf = 0x7f800000u;
  static constexpr bool kWide = true;  // the exponents of 32 bits
  static __device__ float from_bits(uint32_t b) { return __uint_as_float(b); }
  static __device__ float to_f(float v) { return v; }
  static __device__ float from_f(float v) { return v; }
};
template <>
struct Type<__half> {
  static constexpr uint32_t kInf = 0x7c00u;
  static constexpr bool kWide = false;
  static __device__ float from_bits(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }
  static __device__ float to_f(__half v) { return __half2float(v); }
  static __device__ __half from_f(float v) { return __float2half_rn(v); }
};
template <>
struct Type<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7f80u;
  static constexpr bool kWide = true;
  static __device__ float from_bits(uint32_t b) { return __uint_as_float(b << 16); }
  static __device__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
};

// Two 16-bit elements of a word as floats, and back.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// max(m, |w|) of both halves.
template <typename T>
__device__ __forceinline__ uint32_t top2(uint32_t m, uint32_t w);
template <>
__device__ __forceinline__ uint32_t top2<__half>(uint32_t m, uint32_t w) {
  const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&m), __habs2(*reinterpret_cast<const __half2*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t top2<__nv_bfloat16>(uint32_t m, uint32_t w) {
  const __nv_bfloat162 r =
      __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// --------------------------------------------------------------------- W consecutive elements
// Loaded as they are in memory: 8 or 4 elements of 32 bits, 8, 4 or 2 of 16 bits, or 1 of either. The address is a
// multiple of min(16, W * sizeof(T)). kRaw: 32-bit registers held.
template <typename T, int W>
struct Vec {
  static constexpr int kRaw = W * sizeof(T) < 4 ? 1 : W * sizeof(T) / 4;
  uint32_t r[kRaw];

  __device__ __forceinline__ void load(const T* p) {
    constexpr int kBytes = W * sizeof(T);
    if constexpr (kBytes == 32) {
      const uint4 a = *reinterpret_cast<const uint4*>(p), b = *(reinterpret_cast<const uint4*>(p) + 1);
      r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w;
      r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
    } else if constexpr (kBytes == 16) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w;
    } else if constexpr (kBytes == 8) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      r[0] = a.x, r[1] = a.y;
    } else if constexpr (kBytes == 4) {
      r[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      r[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kRaw; ++i) r[i] = 0;
  }
  // Keeps what is computed from the values behind this point: without it the compiler may do that work ahead of a
  // reduction that does not need it, and hold its larger results instead of these registers.
  __device__ __forceinline__ void pin() {
#pragma unroll
    for (int i = 0; i < kRaw; ++i) asm volatile("" : "+r"(r[i]));
  }
  // bits of the largest magnitude so far (as T's bits; NaN and infinities compare above all
  // finite values), per 16-bit half for 16-bit types (the packed maximum keeps a NaN)
  __device__ __forceinline__ uint32_t top(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < kRaw; ++i) {
      if constexpr (sizeof(T) == 4)
        m = max(m, r[i] & 0x7fffffffu);
      else
        m = top2<T>(m, r[i]);
    }
    return m;
  }
  __device__ __forceinline__ void floats(float (&f)[W]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] = __uint_as_float(r[i]);
    } else if constexpr (W == 1) {
      f[0] = unpack2<T>(r[0]).x;
    } else {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const float2 v = unpack2<T>(r[i]);
        f[2 * i] = v.x, f[2 * i + 1] = v.y;
      }
    }
  }
};

// One word's worth of top() (both halves of a 16-bit type) as the bits of one element.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(uint32_t m) {
  if constexpr (sizeof(T) == 4) return m;
  return max(m & 0xffffu, m >> 16);
}

template <typename T, int W>
__device__ __forceinline__ void store(T* p, const float (&f)[W]) {
  if constexpr (W == 1) {
    *p = Type<T>::from_f(f[0]);
  } else if constexpr (sizeof(T) == 4) {
    if constexpr (W == 2) {
      *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
  } else {
    uint32_t r[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) r[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    if constexpr (W == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
    else if constexpr (W == 4)
      *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
    else
      *reinterpret_cast<uint32_t*>(p) = r[0];
  }
}

// W bytes, lowest address in the low byte of b[0]; the address is a multiple of W.
template <int W>
struct Bytes {
  static constexpr int kRaw = W < 4 ? 1 : W / 4;
  uint32_t b[kRaw];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (W == 8) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      b[0] = a.x, b[1] = a.y;
    } else if constexpr (W == 4) {
      b[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (W == 2) {
      b[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      b[0] = *p;
    }
  }
  __device__ __forceinline__ void store(uint8_t* p) const {
    if constexpr (W == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(b[0], b[1]);
    else if constexpr (W == 4)
      *reinterpret_cast<uint32_t*>(p) = b[0];
    else if constexpr (W == 2)
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)b[0];
    else
      *p = (uint8_t)b[0];
  }
};

// ------------------------------------------------------------------------- scales and bytes
// A row's scale from the bits of its largest magnitude, and the factor that a value is multiplied
// by on its way to a byte: inv = 1 / s rounded, and rest = 1 / s - inv (INT8 from 16-bit types). A row with a NaN or an infinity has scale NaN and factor 0 (its bytes
// are cleared by the caller).
struct Scale {
  float s, inv, rest;
  bool fine;
};
template <typename T>
__device__ __forceinline__ Scale scale_of(uint32_t fmt, uint32_t bits) {
  Scale r;
  r.fine = bits < Type<T>::kInf;
  r.rest = 0.0f;
  const float top = Type<T>::from_bits(bits);
  if (fmt == HX_ROWS_E4M3) {
    // The smallest power of two with top / s <= 448 = 1.75 * 2^8: a scale that changes no
    // mantissa, so a byte times its scale is exact in every type and the bytes' distribution
    // over e4m3's fraction bits is the values' own. top = f 2^E: s = 2^(E-8), doubled if f > 1.75.
    const uint32_t b = __float_as_uint(top);
    int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u);
    e = min(max(e, 1), 246);  // 2^-126 .. 2^119: 448 s stays finite
    r.s = __uint_as_float((uint32_t)e << 23);
    r.inv = __uint_as_float((uint32_t)(254 - e) << 23);
  } else {
    // Symmetric INT8; 127 s stays finite at s <= 2^121.
    r.s = fminf(fmaxf(__fdiv_rn(top, 127.0f), 0x1p-126f), 0x1p121f);
    r.inv = __frcp_rn(r.s);
    if (sizeof(T) == 2) r.rest = __fmaf_rn(-r.inv, r.s, 1.0f) * r.inv;
  }
  if (top == 0.0f) r.s = r.inv = 1.0f, r.rest = 0.0f;
  if (!r.fine) r.s = __uint_as_float(0x7fc00000u), r.inv = 0.0f;
  return r;
}

// A scale that INT8 bytes of a 16-bit type divide by.
template <typename T>
__device__ __forceinline__ bool huge(const Scale& sc) {
  return sizeof(T) == 2 && Type<T>::kWide && sc.s > 0x1p64f;
}

// W values to bytes. INT8 is the nearest integer (ties to even) of the 32-bit quotient x / s, found in the low byte of
// that quotient + 1.5 * 2^23.
// From 16-bit types the quotient is x * (inv + rest), rounded once to 32 bits but for the 2^-47 that inv + rest are off.
// That could only matter where x / s lies as close as this to a point where the rounding turns. s is a rounded 127th of a
// value of x's type, so such an x and s have few significands: 2^14 pairs for bf16, 2^20 for f16, at nine exponents, and
// with every one of them the integer is the division's (the tests go through all). Scales above 2^64 divide: there
// `rest` nears the smallest numbers. A bf16 gate and up of 33554 x 1000 values take 45 us so, and 61 by the rule below:
// quotients at a half are frequent with bf16 (a third of the warps hold one).
// From f32, one fused step adds x * inv. x * inv is within 2^-16 of the quotient (|x / s| <= 128; inv and the quotient
// each round once, 2 * 2^-24 * 128), so both round to the same integer unless x * inv lies within 2^-14 of a half: then
// the division itself decides. So it does for a scale at its upper bound, under which a value can reach 128.
template <typename T, int W, bool kHuge = true>
__device__ __forceinline__ Bytes<W> to_bytes(uint32_t fmt, const float (&x)[W], const Scale& sc) {
  Bytes<W> out;
  if (fmt == HX_ROWS_E4M3) {
    if constexpr (W >= 4) {
#pragma unroll
      for (int i = 0; i < W / 4; ++i)
        asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
            " mov.b32 %0, {l, h};\n}"
            : "=r"(out.b[i])
            : "f"(x[4 * i] * sc.inv), "f"(x[4 * i + 1] * sc.inv), "f"(x[4 * i + 2] * sc.inv), "f"(x[4 * i + 3] * sc.inv));
    } else {
      const float hi = W == 2 ? x[W - 1] * sc.inv : 0.0f;
      out.b[0] = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * sc.inv, hi), __NV_SATFINITE, __NV_E4M3);
    }
  } else {
    constexpr float kRound = 12582912.0f;
    uint32_t q[W];
    bool divide;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < W; ++i)
        q[i] = __float_as_uint(__fadd_rn(__fmaf_rn(x[i], sc.inv, __fmul_rn(x[i], sc.rest)), kRound));
      divide = kHuge && huge<T>(sc);
    } else {
      float off = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float r = __fmaf_rn(x[i], sc.inv, kRound);
        q[i] = __float_as_uint(r);
        off = fmaxf(off, fabsf(__fmaf_rn(x[i], sc.inv, -__fsub_rn(r, kRound))));
      }
      divide = off > 0.5f - 0x1p-14f || sc.s >= 0x1p121f;
    }
    if (divide) {
#pragma unroll
      for (int i = 0; i < W; ++i)
        q[i] = __float_as_uint(__fadd_rn(fminf(fmaxf(__fdiv_rn(x[i], sc.s), -127.0f), 127.0f), kRound));
    }
#pragma unroll
    for (int i = 0; i < Bytes<W>::kRaw; ++i) {
      if constexpr (W >= 4)
        out.b[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040), __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
      else if constexpr (W == 2)
        out.b[i] = __byte_perm(q[0], q[1], 0x0040);
      else
        out.b[i] = q[0] & 0xffu;
    }
  }
  if (!sc.fine) {
#pragma unroll
    for (int i = 0; i < Bytes<W>::kRaw; ++i) out.b[i] = 0;
  }
  return out;
}

// A thread's units (lane, lane + n, ...) of a row with a huge scale: written over by to_bytes() with the division, apart
// from the loop over all rows: with the division in that loop a bf16 gate and up of 33554 x 1000 values take 55 us, not 45.
template <typename T, int W>
__device__ __forceinline__ void huge_row(const T* x, uint8_t* bytes, uint32_t units, uint32_t lane, uint32_t n, Scale sc) {
#pragma unroll 1
  for (uint32_t u = lane; u < units; u += n) {
#pragma unroll 1
    for (uint32_t i = u * W; i < u * W + W; ++i) {
      const float f[1] = {Type<T>::to_f(x[i])};
      to_bytes<T, 1>(HX_ROWS_INT8, f, sc).store(bytes + i);
    }
  }
}

// W bytes back to values: byte value times scale, one rounding to 32 bits (none for e4m3).
template <int W>
__device__ __forceinline__ void to_values(uint32_t fmt, const Bytes<W>& in, float s, float (&x)[W]) {
  if (fmt == HX_ROWS_E4M3) {
    if constexpr (W >= 4) {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        uint32_t h0, h1;
        asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
            : "=r"(h0), "=r"(h1)
            : "r"(in.b[i]));
        const float2 v0 = unpack2<__half>(h0), v1 = unpack2<__half>(h1);
        x[4 * i] = v0.x * s, x[4 * i + 1] = v0.y * s, x[4 * i + 2] = v1.x * s, x[4 * i + 3] = v1.y * s;
      }
    } else {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(in.b[0] & 0xffffu), __NV_E4M3);
      const float2 v = __half22float2(__half2(h));
      x[0] = v.x * s;
      if (W == 2) x[W - 1] = v.y * s;
    }
  } else {
    // 2^23 + (byte + 128) from its bits (an integer conversion runs at a quarter of this rate)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t f = __byte_perm(in.b[i / 4] ^ 0x80808080u, 0x4b000000u, 0x7650u | (i & 3));
      x[i] = __fsub_rn(__uint_as_float(f), 8388736.0f) * s;
    }
  }
}

// --------------------------------------------------------------------------------------- host
// Allows `kernel` `bytes` of dynamic shared memory on the current device: asked for once per device.
template <auto kernel>
inline bool allow_shared(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

}  // namespace hxv
