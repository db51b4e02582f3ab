// Weight gradient of a linear layer from the 8-bit rows of its input (sm_100a):
//     dW[o][i] = sum over tokens t of dY[t][o] * s_t * q[t][i].
//
// A product of two matrices whose contraction runs over the tokens, so both operands are stored with
// the contraction outermost (MN-major). Tensor cores: tcgen05.mma, accumulators in TMEM, one CTA
// per tile of BM output by BN input features, steps of 64 tokens.
//   warps 0 ..  read the bytes (8 columns of a token per lane, the next steps' already in flight),
//               turn them into s_t q in dY's type and write them to shared memory in the 128-byte
//               swizzle that the tensor core reads; at the end they read TMEM and store the tile.
//   one warp    brings dY's tile by TMA, in the same swizzle.
//   one warp    issues the products.
// The bytes never exist as a 16-bit matrix in memory. s_t q in bf16 is exact for e4m3 (the scale is a
// power of two). For INT8 it is not, and one rounding to bf16 would put an error of the size of the result's
// own rounding into every product: there the tile is held as two, the rounded values and the rounded
// rest (17 bits together in bf16), at twice the products. In f16 the rest of a value below 2^-3 would be below f16's normal
// range, so it is held 2^11 times as large, with accumulators of its own (together 2^-23 of the value, and 2^-36).
// Sums are the tensor core's 32-bit accumulators. It cuts what lies below their 32 bits each time it adds 16 tokens, so that
// a sum of terms of one sign falls short (e4m3, bf16, tokens of one CTA): 8e-7 of it after 1024 tokens, 1.2e-5 after 8192,
// 2.0e-4 after 2^16, 1.2e-3 after 2^18. cuBLAS's product of two bf16 matrices with a 32-bit result falls short by the same.
//
// Few tiles: the tokens are split over up to 8 CTAs (4 pairs) of one cluster, which leave their 32-bit partial
// tiles in shared memory, and each adds the others' share of its rows in their order: no workspace, no second kernel.
//
// Rows of dY that do not start on 16 bytes (TMA's rule), or of X on 8, are first copied to rows that do.
//
// Measured on B200 (bf16): 8192 x 8192 x 8192 from e4m3 rows 655-680 us in short runs, 790 us over seconds at the power
// limit (1425 MHz, 993 W); cuBLAS on two bf16 matrices 660-675 and 793 (1327 MHz) on the same machine. 4096^3 94 us. INT8, at
// twice the products: 4096^3 182 us; 8192^3 1260-1290 us in short runs, 1504 over seconds (1417 MHz, 995 W). What
// brought it there: CTA pairs (each CTA converts and reads half of the tile's columns), several steps in conversion
// at once, no fence wider than the CTA's own shared memory, whole-line stores.
//
// Every wait is bounded (2 s); when one runs out the CTA raises HX_ERR_TIMEOUT, waits for the copies and products
// in flight, frees its TMEM and returns. Its cluster's part of the result is NaN then: whatever sums it has are
// not whole.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "hx.h"
#include "hx_values.h"

namespace {

using namespace hxv;

constexpr int kStep = 64;             // tokens per pipeline stage
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMaxCluster = 8;
constexpr int kBand = 4;              // tile rows that are walked together

struct Args {
  uint32_t fmt;
  const uint8_t* bytes;
  uint64_t ld_x;  // a multiple of 8, as the address
  const float* scale;
  uint64_t tokens;
  uint32_t n_out, n_in;
  void* dw;
  uint64_t ld_dw;
  uint32_t dw_dtype, accumulate, dw_wide;
  uint32_t splits, steps;
  uint32_t* status;
  uint64_t wait_ns, withhold;  // a wait's limit; a CTA whose converting warps do nothing (tests)
};

// ------------------------------------------------------------------------------------ barriers
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same on the barrier at this address in CTA `rank` of the cluster. What was written before it is in the CTA's own
// shared memory, ordered for the tensor core by fence.proxy.async; a release at cluster scope would only add a memory
// barrier (1500 clocks per arrival, measured).
__device__ __forceinline__ void bar_arrive_at(uint32_t bar, uint32_t rank) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n"
      " mbarrier.arrive.shared::cluster.b64 _, [a];\n}" ::"r"(bar), "r"(rank)
      : "memory");
}
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for the phase of `parity` to complete. False once this wait, or any other of the CTA, ran out. The timer goes on
// while the GPU runs another context, so what passes between two looks at it counts as 1/64 of the limit at most.
__device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, volatile uint32_t* failed, uint64_t limit) {
  uint64_t last = now_ns(), spent = 0;
  for (;;) {
    for (int i = 0; i < 16; ++i)
      if (bar_try(bar, parity)) return true;
    if (*failed) return false;
    const uint64_t t = now_ns();
    spent += min(t - last, limit / 64 + 1), last = t;
    if (spent > limit) {
      *failed = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* failed, uint64_t limit) {
  return bar_try(bar, parity) || bar_wait_long(bar, parity, failed, limit);
}

// --------------------------------------------------------------------------------- tensor core
// Shared memory operand, MN-major with 128-byte swizzle: blocks of 64 values of M or N by 64 tokens, a
// token's 64 values in one 128-byte line; 8 lines per swizzle atom (stride 1024), blocks 8192 apart.
// Its descriptor's low word is the address / 16 beside the block stride, so that a step along the operand is an addition;
// the high word is the same for all.
__device__ __forceinline__ uint32_t operand(uint32_t addr) { return (addr & 0x3ffffu) >> 4 | (8192u >> 4) << 16; }
constexpr uint32_t kOperandHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
template <typename T, int M, int N>
__device__ constexpr uint32_t instruction() {
  constexpr uint32_t type = sizeof(T) && Type<T>::kInf == 0x7f80u ? 1 : 0;  // bf16 or f16
  return 1u << 4 | type << 7 | type << 10 | 1u << 15 | 1u << 16 | (uint32_t)(N / 8) << 17 | (uint32_t)(M / 16) << 24;
}
// kAdd: onto the accumulator. One thread issues every product, so an issue is as few instructions as it can be.
template <bool kPair, bool kAdd>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t instr) {
  if constexpr (kPair)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %4, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(kOperandHigh), "r"(instr), "n"((int)kAdd)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(kOperandHigh), "r"(instr), "n"((int)kAdd)
        : "memory");
}
// The products of one stage of 64 tokens; kFirst: the tile's first.
template <typename S, typename T, int MT, bool kPair, int kParts, int kSums, bool kFirst>
__device__ __forceinline__ void stage_products(uint32_t tmem, uint32_t a, uint32_t b) {
  constexpr uint32_t instr = instruction<T, S::M, S::N>();
#pragma unroll
  for (int kk = 0; kk < kStep / 16; ++kk)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        const uint32_t x = a + ((mt * 16384 + kk * 2048) >> 4), y = b + ((p * S::kB + kk * 2048) >> 4);
        const uint32_t d = tmem + (p % kSums * MT + mt) * S::N;
        if (kFirst && kk == 0 && p < kSums)
          mma<kPair, false>(d, x, y, instr);
        else
          mma<kPair, true>(d, x, y, instr);
      }
}
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r;
}
// Arrives on the barrier (of both CTAs of a pair, the first of which has rank `first`) once the products
// issued so far are done.
template <bool kPair>
__device__ __forceinline__ void commit(uint32_t bar, uint32_t first) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)(3u << first))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
      "%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// A CTA, or a pair of CTAs on two SMs of one cluster, per tile. MT accumulators of 128 rows per CTA; 128
// columns of X in each CTA's shared memory. A pair's products take both CTAs' columns (the second CTA's
// through the pair's own path): 256 columns, each converted and read from shared memory by one CTA only.
// kSums: accumulators per 128 rows, 2 where X's second part has its own.
template <int MT, bool kPair, int kParts, int kSums>
struct Tile {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int M = 128 * kCtas, N = 128 * kCtas;  // of one product
  static constexpr int BM = M * MT, BN = N;               // of the tile
  static constexpr int kA = 128 * MT * kStep * 2, kB = 128 * kStep * 2;
  static constexpr int kStage = kA + kParts * kB;
  static constexpr int kStages = 196608 / kStage < 8 ? 196608 / kStage : 8;
  // Groups of converting warps: group g takes steps g, g + kGroups, ... Not more than stages: a group then
  // comes to a stage's next use only after the use before last has been released, which a wait for one
  // bit of phase relies on.
  static constexpr int kGroups = kStages < 4 ? kStages : 4;
  static constexpr int kGroupWarps = 4;
  static constexpr int kWarps = kGroups * kGroupWarps;
  static constexpr int kTokens = kStep / kGroupWarps;  // a converting warp's tokens of its step
  static constexpr int kThreads = 32 * (kWarps + 2);
  static constexpr int kCols = MT * N * kSums;  // TMEM columns: a power of two of at least 32
  static constexpr int kSmem = kStages * kStage + 1024;
  static_assert(kStages * kStage >= kWarps * 4096, "");  // the epilogue's rows
  static_assert(kStages >= 3 && kGroups <= kStages && kCols <= 512 && (kCols & (kCols - 1)) == 0, "");
};

struct Barriers {
  uint64_t copied[8], converted[8], empty[8], done;
  uint32_t tmem, failed;
  uint32_t issued[2];  // in a pair's first CTA: the steps whose copies each CTA asked for
};

// Whether T's second part of a value is held kRestUp times as large, and summed by itself.
constexpr float kRestUp = 2048.0f;
template <typename T, int kParts>
constexpr bool kRestApart = kParts == 2 && Type<T>::kInf == 0x7c00u;

// ---------------------------------------------------------------------------------- conversion
// 8 bytes of a row with scale s as values of type T, in kParts parts (1: e4m3, 2: INT8). kClamp: they may pass T's range.
template <typename T, int kParts, bool kClamp>
__device__ __forceinline__ void convert(const Bytes<8>& b, float s, uint4 (&out)[kParts]) {
  float f[8];
  to_values<8>(kParts == 1 ? HX_ROWS_E4M3 : HX_ROWS_INT8, b, s, f);
  if constexpr (kClamp) {
    // a row near fp16's largest value can round above it in its byte
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] > 65504.0f ? 65504.0f : f[i] < -65504.0f ? -65504.0f : f[i];
  }
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
      if (p + 1 < kParts) {  // what the rounding left
        const float2 v = unpack2<T>(r[i]);
        f[2 * i] -= v.x, f[2 * i + 1] -= v.y;
        if (kRestApart<T, kParts>) f[2 * i] *= kRestUp, f[2 * i + 1] *= kRestUp;
      }
    }
    out[p] = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

// The same for e4m3 and a scale that T holds (twice in s2; in bf16 every scale of the library's, in f16 those within its range):
// e4m3's values are exact in T, so one packed product there rounds as the 32-bit product would.
template <typename T>
__device__ __forceinline__ uint4 convert_packed(const Bytes<8>& b, uint32_t s2) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h0, h1;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(h0), "=r"(h1)
        : "r"(b.b[i]));
    if constexpr (Type<T>::kInf == 0x7f80u) {
      const float2 v0 = unpack2<__half>(h0), v1 = unpack2<__half>(h1);
      const uint32_t w0 = pack2<__nv_bfloat16>(v0.x, v0.y), w1 = pack2<__nv_bfloat16>(v1.x, v1.y);
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r[2 * i]) : "r"(w0), "r"(s2));
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r[2 * i + 1]) : "r"(w1), "r"(s2));
    } else {  // within +-65504; a NaN stays
      asm("{\n .reg .b32 t;\n mul.rn.f16x2 t, %1, %2;\n min.NaN.f16x2 t, t, %3;\n max.NaN.f16x2 %0, t, %4;\n}"
          : "=r"(r[2 * i])
          : "r"(h0), "r"(s2), "r"(0x7bff7bffu), "r"(0xfbfffbffu));
      asm("{\n .reg .b32 t;\n mul.rn.f16x2 t, %1, %2;\n min.NaN.f16x2 t, t, %3;\n max.NaN.f16x2 %0, t, %4;\n}"
          : "=r"(r[2 * i + 1])
          : "r"(h1), "r"(s2), "r"(0x7bff7bffu), "r"(0xfbfffbffu));
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ void put(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// ------------------------------------------------------------------------------------ the tile
// 32 columns of a lane's sums; kRest: the columns from there to the sums of the second parts, or 0.
template <uint32_t kRest>
__device__ __forceinline__ void load_sums(uint32_t addr, uint32_t (&r)[32]) {
  tmem_load32(addr, r);
  if constexpr (kRest != 0) {
    uint32_t q[32];
    tmem_load32(addr + kRest, q);
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(fmaf(__uint_as_float(q[i]), 1.0f / kRestUp, __uint_as_float(r[i])));
  }
}

// A warp's 32 rows of C = 128 / sizeof(O) columns from TMEM (columns tm ..) to the matrix o (n_rows x n_cols, row
// stride ld) at (row, col). The rows pass through 4 KB of shared memory, so that the stores are whole lines (a lane
// per row straight from TMEM would touch 32 lines with each store).
template <typename O, uint32_t kRest>
__device__ __forceinline__ void store_block(uint32_t stage, uint32_t tm, bool any, O* o, uint64_t ld, bool wide, bool add,
                                            uint32_t row, uint32_t col, uint32_t n_rows, uint32_t n_cols) {
  constexpr uint32_t C = 128 / sizeof(O);
  const uint32_t lane = threadIdx.x & 31;
  if (!add) {
#pragma unroll
    for (uint32_t h = 0; h < C / 32; ++h) {
      uint32_t r[32];
      load_sums<kRest>(tm + h * 32, r);
      constexpr uint32_t kChunks = 32 * sizeof(O) / 16, kPer = 16 / sizeof(O);
#pragma unroll
      for (uint32_t c = 0; c < kChunks; ++c) {
        uint32_t w[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          if constexpr (sizeof(O) == 4)
            w[i] = any ? r[4 * c + i] : 0;
          else
            w[i] = any ? pack2<O>(__uint_as_float(r[(kPer * c + 2 * i) % 32]), __uint_as_float(r[(kPer * c + 2 * i + 1) % 32])) : 0;
        }
        put(stage + lane * 128 + (((h * kChunks + c) ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
    __syncwarp();
    if (wide && col + C <= n_cols) {
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i) {
        const uint32_t y = i * 4 + (lane >> 3), c = lane & 7;
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(stage + y * 128 + ((c ^ (y & 7)) << 4)));
        if (row + y < n_rows) *reinterpret_cast<uint4*>(o + (uint64_t)(row + y) * ld + col + c * (16 / sizeof(O))) = v;
      }
    } else {
      for (uint32_t y = 0; y < 32 && row + y < n_rows; ++y)
#pragma unroll
        for (uint32_t h = 0; h < C / 32; ++h) {
          const uint32_t x = h * 32 + lane, byte = x * sizeof(O);
          const uint32_t at = stage + y * 128 + (((byte >> 4) ^ (y & 7)) << 4) + (byte & 15);
          O* p = o + (uint64_t)(row + y) * ld + col + x;
          if constexpr (sizeof(O) == 4) {
            uint32_t v;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
            if (col + x < n_cols) *reinterpret_cast<uint32_t*>(p) = v;
          } else {
            uint16_t v;
            asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(at));
            if (col + x < n_cols) *reinterpret_cast<uint16_t*>(p) = v;
          }
        }
    }
    __syncwarp();
  } else {
    // onto old values: 32-bit sums through shared memory, 32 columns at a time, so that the total rounds once
    for (uint32_t h = 0; h < C / 32; ++h) {
      uint32_t r[32];
      load_sums<kRest>(tm + h * 32, r);
#pragma unroll
      for (uint32_t c = 0; c < 8; ++c)
        put(stage + lane * 128 + ((c ^ (lane & 7)) << 4),
            any ? make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]) : make_uint4(0, 0, 0, 0));
      __syncwarp();
      const uint32_t x = col + h * 32 + lane;
      for (uint32_t y = 0; y < 32 && row + y < n_rows; ++y) {
        float v;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(stage + y * 128 + (((lane >> 2) ^ (y & 7)) << 4) + (lane & 3) * 4));
        O* p = o + (uint64_t)(row + y) * ld + x;
        if (x < n_cols) *p = Type<O>::from_f(Type<O>::to_f(*p) + v);
      }
      __syncwarp();
    }
  }
}

// Rows y0 .. y1 - 1 of the tile at (m0, n0) from the partial tiles of the cluster's splits.
template <typename O, uint32_t N>
__device__ __forceinline__ void join_rows(const Args& a, uint32_t tiles, uint32_t rank, uint32_t ctas, uint32_t m0,
                                          uint32_t n0, uint32_t y0, uint32_t y1) {
  constexpr uint32_t kChunks = N / 4;
  for (uint32_t i = threadIdx.x; i < (y1 - y0) * kChunks; i += blockDim.x) {
    const uint32_t y = y0 + i / kChunks, c = i % kChunks;
    const uint32_t row = m0 + y, col = n0 + c * 4;
    if (row >= a.n_out || col >= a.n_in) continue;
    const uint32_t at = tiles + y * (N * 4) + (c ^ (y & 7)) * 16;
    float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t s = 0; s < a.splits; ++s) {
      float v[4];
      asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                   : "r"(at_rank(at, s * ctas + rank)));
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] += v[k];
    }
    O* o = static_cast<O*>(a.dw) + (uint64_t)row * a.ld_dw + col;
    if (a.dw_wide && col + 4 <= a.n_in) {
      if (a.accumulate) {
        Vec<O, 4> old;
        old.load(o);
        float g[4];
        old.floats(g);
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] += g[k];
      }
      store<O, 4>(o, f);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + k < a.n_in) o[k] = Type<O>::from_f(a.accumulate ? Type<O>::to_f(o[k]) + f[k] : f[k]);
    }
  }
}

// What follows a wait that ran out stands apart from the kernel's code, whose end then has nothing to skip (in line it cost
// a launch 0.2 us or more).
// To every CTA of the cluster: this one gave up.
__device__ __noinline__ void tell_cluster(uint32_t failed, uint32_t ctas) {
  const uint32_t lane = threadIdx.x & 31;
  if (lane < ctas) asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(at_rank(failed, lane)), "r"(1) : "memory");
}
// A phase that completes by itself, in kWaitNs from t0 at most.
__device__ __forceinline__ void wait_out(uint32_t bar, uint32_t parity, uint64_t t0) {
  while (!bar_try(bar, parity) && now_ns() - t0 < kWaitNs) {
  }
}
// NaN to rows y0 .. y1 - 1 of each of the CTA's accumulators (rows m0 + i * M ..).
template <typename O>
__device__ __forceinline__ void lose_rows(const Args& a, uint32_t m0, uint32_t n0, uint32_t y0, uint32_t y1, uint32_t mt,
                                          uint32_t M, uint32_t N) {
  const O nan = Type<O>::from_f(__uint_as_float(0x7fc00000u));
  for (uint32_t i = threadIdx.x; i < mt * (y1 - y0) * N; i += blockDim.x) {
    const uint32_t y = i / N, row = m0 + y / (y1 - y0) * M + y0 + y % (y1 - y0), col = n0 + i % N;
    if (row < a.n_out && col < a.n_in) static_cast<O*>(a.dw)[(uint64_t)row * a.ld_dw + col] = nan;
  }
}
// All threads of all CTAs of a cluster in which a wait ran out: no CTA ends before its copies and the products issued have,
// and its part of the result is NaN. In a pair's first CTA, whose barriers count both CTAs' copies, a step that only one of
// them asked for gets what its barrier misses.
template <typename S, typename T, int MT, bool kPair>
__device__ __noinline__ void give_up(const Args& a, Barriers& bars, uint32_t steps, uint32_t rank, uint32_t m0, uint32_t n0,
                                     uint32_t y0, uint32_t y1) {
  const uint64_t t0 = now_ns();
  if (threadIdx.x == 0 && rank == 0) {
    const uint32_t one = bars.issued[0], two = bars.issued[kPair], low = min(one, two), high = max(one, two);
    for (uint32_t i = high > S::kStages ? high - S::kStages : 0; i < high; ++i) {
      const uint32_t bar = smem_addr(&bars.copied[i % S::kStages]);
      if (i >= low && one < two)  // announced by nobody
        bar_expect(bar, S::kA);
      else if (i >= low)  // announced for both
        asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"((uint32_t)S::kA) : "memory");
      wait_out(bar, (i / S::kStages) & 1, t0);
    }
  }
  if (threadIdx.x == 32 && steps) wait_out(smem_addr(&bars.done), 0, t0);
  if (a.dw_dtype == HX_F32)
    lose_rows<float>(a, m0, n0, y0, y1, MT, S::M, S::N);
  else
    lose_rows<T>(a, m0, n0, y0, y1, MT, S::M, S::N);
  if (threadIdx.x == 0 && a.status) atomicOr(a.status, (uint32_t)HX_ERR_TIMEOUT);
  __syncwarp();
  cluster_sync();
}

template <typename T, int MT, bool kPair, int kParts>
__global__ void __launch_bounds__(Tile<MT, kPair, kParts, 1 + kRestApart<T, kParts>>::kThreads, 1)
    k_wgrad(const __grid_constant__ CUtensorMap map, const __grid_constant__ Args a) {
  constexpr int kSums = 1 + kRestApart<T, kParts>;
  using S = Tile<MT, kPair, kParts, kSums>;
  constexpr uint32_t kRest = kSums > 1 ? MT * S::N : 0;
  constexpr int kGroups = S::kGroups, kGroupWarps = S::kGroupWarps, kWarps = S::kWarps, kTokens = S::kTokens;
  extern __shared__ uint8_t raw[];
  __shared__ Barriers bars;
  const uint32_t tiles = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t in_cluster = cluster_rank(), split = in_cluster / S::kCtas, rank = in_cluster % S::kCtas;
  const uint32_t first = in_cluster - rank;  // the pair's first CTA
  // Tiles in bands of kBand tile rows, columns slowest within a band: what runs at once shares 4 tiles' worth of
  // dY and about 18 of X, whose bytes are the smaller (a tile's dY takes four times its X from memory).
  const uint32_t tile = blockIdx.x / (S::kCtas * a.splits), rows = (a.n_out + S::BM - 1) / S::BM, cols = (a.n_in + S::BN - 1) / S::BN;
  const uint32_t band = tile / (kBand * cols), in_band = tile - band * kBand * cols;
  const uint32_t high = min((uint32_t)kBand, rows - band * kBand);
  const uint32_t m0 = (band * kBand + in_band % high) * S::BM + rank * 128;  // accumulator i: rows m0 + i * M ..
  const uint32_t n0 = in_band / high * S::BN, x0 = n0 + rank * 128;          // the tile's columns, the CTA's
  const uint32_t per = (a.steps + a.splits - 1) / a.splits;
  const uint32_t k0 = min(split * per, a.steps), k1 = min(k0 + per, a.steps), steps = k1 - k0;
  volatile uint32_t* failed = &bars.failed;
  auto copied = [&](uint32_t s) { return smem_addr(&bars.copied[s]); };
  auto converted = [&](uint32_t s) { return smem_addr(&bars.converted[s]); };
  auto empty = [&](uint32_t s) { return smem_addr(&bars.empty[s]); };
  const uint32_t done = smem_addr(&bars.done);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      bar_init(copied(s), 1);
      bar_init(converted(s), S::kCtas * kGroupWarps);  // (of a pair: the first CTA's, for both)
      bar_init(empty(s), 1);
    }
    bar_init(done, 1);
    bars.failed = 0;
    bars.issued[0] = bars.issued[1] = steps;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarps + 1) {
    if constexpr (kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars.tmem)),
                   "r"((uint32_t)S::kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars.tmem)),
                   "r"((uint32_t)S::kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(&bars.tmem), 0);

  if (warp < kWarps) {
    // ---- converting warps. A step's chain (wait, convert, store, fence, arrive) is longer than its products
    // take, so the groups work on three or four steps at once, and a group's next bytes have the others'
    // steps to arrive. 8 columns per lane: a warp's load is two tokens' 128 columns (lanes 16-31 the odd
    // one). Lanes 8 i .. 8 i + 7 write one whole line, so no two share a bank.
    constexpr int kLoads = kTokens / 2;
    const uint32_t group = warp / kGroupWarps, line0 = warp % kGroupWarps * kTokens;
    const uint32_t ch = lane & 15, odd = lane >> 4;
    Bytes<8> b[kLoads];
    float sc = 0.0f;
    // Loads are never conditional (a load that is chosen between is waited for on the spot): past the last token or
    // column they go to the last one's place, and a token past the last is cleared when it is converted. Columns
    // past the last only reach sums that are not stored.
    const uint8_t* x = a.bytes + min((uint64_t)x0 + ch * 8, a.ld_x - 8);
    auto fetch = [&](uint32_t k) {
      const uint64_t t = (uint64_t)(k0 + k) * kStep + line0;
      sc = a.scale[min(t + (lane & (kTokens - 1)), a.tokens - 1)];
      if (t + kTokens <= a.tokens) {
        const uint8_t* p = x + (t + odd) * a.ld_x;
#pragma unroll
        for (int j = 0; j < kLoads; ++j, p += 2 * a.ld_x) b[j].load(p);
      } else {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) b[j].load(x + min(t + 2 * j + odd, a.tokens - 1) * a.ld_x);
      }
    };
    const uint32_t mine = blockIdx.x == a.withhold ? 0 : steps;
    if (group < mine) fetch(group);
    bool ok = true;
    for (uint32_t k = group; k < mine; k += kGroups) {
      const uint32_t s = k % S::kStages;
      // one answer per warp: what follows is for whole warps
      if (!(ok = __all_sync(0xffffffffu, bar_wait(empty(s), ((k / S::kStages) & 1) ^ 1, failed, a.wait_ns)))) break;
      // line line0 + 2 j + odd, its chunks exchanged by the line's place in its eight
      const uint32_t B = tiles + s * S::kStage + S::kA + (ch >> 3) * 8192 + (line0 + odd) * 128;
      const uint32_t swap = ((ch ^ odd) & 7) << 4;
      const uint64_t t = (uint64_t)(k0 + k) * kStep + line0;
      if (t + kTokens > a.tokens) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
          if (t + 2 * j + odd >= a.tokens) b[j].b[0] = b[j].b[1] = 0;
        if (t + (lane & (kTokens - 1)) >= a.tokens) sc = 0.0f;
      }
      const T narrow = Type<T>::from_f(sc);
      const uint32_t bits = *reinterpret_cast<const uint16_t*>(&narrow), s2 = bits | bits << 16;
      if (kParts == 1 && __all_sync(0xffffffffu, Type<T>::to_f(narrow) == sc)) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
          put(B + j * 256 + (swap ^ ((2 * j & 7) << 4)), convert_packed<T>(b[j], __shfl_sync(0xffffffffu, s2, 2 * j + odd)));
      } else {
        const auto put_all = [&](auto clamp) {
#pragma unroll
          for (int j = 0; j < kLoads; ++j) {
            uint4 v[kParts];
            convert<T, kParts, decltype(clamp)::value>(b[j], __shfl_sync(0xffffffffu, sc, 2 * j + odd), v);
#pragma unroll
            for (int p = 0; p < kParts; ++p) put(B + p * S::kB + j * 256 + (swap ^ ((2 * j & 7) << 4)), v[p]);
          }
        };
        if (Type<T>::kInf == 0x7f80u || (kParts == 2 && __all_sync(0xffffffffu, sc <= 65504.0f / 128)))
          put_all(std::false_type{});
        else
          put_all(std::true_type{});
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair)
          bar_arrive_at(converted(s), first);
        else
          bar_arrive(converted(s));
      }
      if (k + kGroups < mine) fetch(k + kGroups);
    }
    // ---- the tile's rows: lanes 32 (warp % 4) .. + 31 of TMEM
    if (ok && steps) ok = bar_wait(done, 0, failed, a.wait_ns);
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (__all_sync(0xffffffffu, ok)) {
      // a block of columns at a time, the warps of a lane quarter in turn; the stages are free by now
      const uint32_t quarter = (warp & 3) * 32;
      if (MT == 1 && a.splits > 1) {
        // the partial tile: 128 rows of N sums, 16-byte chunks exchanged within eights by the row
        for (uint32_t i = warp >> 2; i < S::N / 32; i += kWarps / 4) {
          uint32_t r[32];
          load_sums<kRest>(tmem + (quarter << 16) + i * 32, r);
          const uint32_t y = quarter + lane;
#pragma unroll
          for (uint32_t c = 0; c < 8; ++c)
            put(tiles + y * (S::N * 4) + (i * 8 + (c ^ (y & 7))) * 16,
                make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]));
        }
      } else {
        const uint32_t stage = tiles + warp * 4096;
        const uint32_t width = a.dw_dtype == HX_F32 ? 32 : 64;
        for (uint32_t i = warp >> 2; i < MT * S::N / width; i += kWarps / 4) {
          const uint32_t mt = i / (S::N / width), c = i % (S::N / width) * width;
          const uint32_t row = m0 + mt * S::M + quarter, col = n0 + c;
          const uint32_t tm = tmem + (quarter << 16) + mt * S::N + c;
          if (row >= a.n_out || col >= a.n_in) continue;
          if (a.dw_dtype == HX_F32)
            store_block<float, kRest>(stage, tm, steps > 0, static_cast<float*>(a.dw), a.ld_dw, a.dw_wide, a.accumulate, row, col,
                               a.n_out, a.n_in);
          else
            store_block<T, kRest>(stage, tm, steps > 0, static_cast<T*>(a.dw), a.ld_dw, a.dw_wide, a.accumulate, row, col, a.n_out,
                           a.n_in);
        }
      }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  } else if (warp == kWarps) {
    if (lane == 0) {
      uint32_t k = 0;
      for (; k < steps; ++k) {
        const uint32_t s = k % S::kStages;
        if (!bar_wait(empty(s), ((k / S::kStages) & 1) ^ 1, failed, a.wait_ns)) break;
        const int32_t t = (int32_t)((k0 + k) * kStep);
        if constexpr (kPair) {
          // both CTAs' copies count on the first one's barrier
          if (rank == 0) bar_expect(copied(s), 2 * S::kA);
          const uint32_t bar = at_rank(copied(s), first);
          for (int i = 0; i < 2 * MT; ++i)
            asm volatile(
                "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                    tiles + s * S::kStage + i * 8192),
                "l"(&map), "r"((int32_t)(m0 + i / 2 * S::M + i % 2 * 64)), "r"(t), "r"(bar)
                : "memory");
        } else {
          bar_expect(copied(s), S::kA);
          for (int i = 0; i < 2 * MT; ++i)
            asm volatile(
                "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                    tiles + s * S::kStage + i * 8192),
                "l"(&map), "r"((int32_t)(m0 + i / 2 * S::M + i % 2 * 64)), "r"(t), "r"(copied(s))
                : "memory");
        }
      }
      if (k < steps)  // gave up
        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(at_rank(smem_addr(&bars.issued[rank]), first)), "r"(k) : "memory");
    }
  } else if (rank == 0) {
    // the whole warp walks the steps, so that what the products take stays in uniform registers; one lane issues
    bool ok = true;
    const uint32_t a0 = operand(tiles), b0 = operand(tiles + S::kA);
    uint32_t s = 0, parity = 0;
    for (uint32_t k = 0; k < steps; ++k) {
      ok = bar_wait(converted(s), parity, failed, a.wait_ns) && bar_wait(copied(s), parity, failed, a.wait_ns);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t at = s * (S::kStage >> 4);
      if (elected()) {
        if (k == 0)
          stage_products<S, T, MT, kPair, kParts, kSums, true>(tmem, a0 + at, b0 + at);
        else
          stage_products<S, T, MT, kPair, kParts, kSums, false>(tmem, a0 + at, b0 + at);
        // only where somebody waits for it: an arrival in the pair's other CTA could else come after that CTA's end
        if (k + S::kStages < steps) commit<kPair>(empty(s), first);
      }
      __syncwarp();
      if (++s == S::kStages) s = 0, parity ^= 1;
    }
    // the products issued so far end before the TMEM is freed, also when a wait ran out. (Without steps nobody waits.)
    if (steps && elected()) commit<kPair>(done, first);
  }
  // a CTA that gave up tells its whole cluster: before the cluster's barrier, so that all know it after
  __syncwarp();
  if (__builtin_expect(*failed, 0)) tell_cluster(smem_addr(&bars.failed), S::kCtas * a.splits);
  __syncwarp();
  cluster_sync();
  const bool joined = MT == 1 && a.splits > 1;
  const uint32_t y0 = joined ? split * 128 / a.splits : 0, y1 = joined ? (split + 1) * 128 / a.splits : 128;
  if (__builtin_expect(*failed, 0)) {
    give_up<S, T, MT, kPair>(a, bars, steps, rank, m0, n0, y0, y1);
  } else if (joined) {
    // this split's share of the rows: the splits' sums in their order, four columns per thread
    if (a.dw_dtype == HX_F32)
      join_rows<float, S::N>(a, tiles, rank, S::kCtas, m0, n0, y0, y1);
    else
      join_rows<T, S::N>(a, tiles, rank, S::kCtas, m0, n0, y0, y1);
    __syncwarp();
    cluster_sync();  // a CTA's sums stay until every other one has read them
  }
  if (warp == kWarps + 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if constexpr (kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)S::kCols));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)S::kCols));
  }
}

// Copies rows to a pitch that TMA and the 8-byte loads take: `chunks` pieces of 16 bytes per row, what is behind the row's
// end zero. E: the element (2 or 1 bytes). A piece inside its row is read in five aligned words, which reach up to three
// bytes into the row before and behind it; where the row does not have those, by its elements.
template <typename E>
__device__ __forceinline__ void align_piece(const E* src, uint64_t ld, uint64_t cols, uint4* dst, uint32_t chunks, uint64_t i) {
  constexpr uint32_t kPer = 16 / sizeof(E);
  const uint64_t row = i >> 32 ? i / chunks : (uint32_t)i / chunks, c = (i - row * chunks) * kPer;
  const E* p = src + row * ld + c;
  uint32_t v[4] = {0, 0, 0, 0};
  if (c && c + kPer + 4 / sizeof(E) - 1 <= cols) {
    const uint32_t shift = (reinterpret_cast<uintptr_t>(p) & 3) * 8;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3);
    uint32_t x[5];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = w[k];
    x[4] = shift ? w[4] : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __funnelshift_r(x[k], x[k + 1], shift);
  } else {
#pragma unroll
    for (uint32_t k = 0; k < kPer; ++k)
      if (c + k < cols) v[k * sizeof(E) / 4] |= (uint32_t)p[k] << (8 * (k * sizeof(E) % 4));
  }
  dst[i] = make_uint4(v[0], v[1], v[2], v[3]);
}
__global__ void __launch_bounds__(256)
    k_wgrad_align(const uint16_t* dy, uint64_t ld_dy, uint64_t n_out, uint4* dy_out, const uint8_t* x, uint64_t n_in,
                  uint4* x_out, uint64_t tokens, uint32_t dy_blocks) {
  const uint32_t cy = (uint32_t)((n_out + 7) / 8), cx = (uint32_t)((n_in + 15) / 16);
  const bool first = blockIdx.x < dy_blocks;
  const uint64_t all = tokens * (first ? cy : cx), step = (uint64_t)(first ? dy_blocks : gridDim.x - dy_blocks) * 256;
  for (uint64_t i = (uint64_t)(first ? blockIdx.x : blockIdx.x - dy_blocks) * 256 + threadIdx.x; i < all; i += step) {
    if (first)
      align_piece<uint16_t>(dy, ld_dy, n_out, dy_out, cy, i);
    else
      align_piece<uint8_t>(x, n_in, n_in, x_out, cx, i);
  }
}

// ------------------------------------------------------------------------------------- launch
int launched() { return cudaGetLastError() == cudaSuccess ? HX_OK : HX_ERR_CUDA; }
bool multiple(const void* p, uint64_t of) { return (reinterpret_cast<uintptr_t>(p) % of) == 0; }

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

template <typename T, int MT, bool kPair, int kParts>
int launch_tile(const CUtensorMap& map, const Args& a, cudaStream_t s) {
  using S = Tile<MT, kPair, kParts, 1 + kRestApart<T, kParts>>;
  const auto kernel = k_wgrad<T, MT, kPair, kParts>;
  if (!allow_shared<k_wgrad<T, MT, kPair, kParts>>(S::kSmem)) return HX_ERR_CUDA;
  const uint64_t ctas = ceil_div(a.n_out, S::BM) * ceil_div(a.n_in, S::BN) * S::kCtas * a.splits;
  if (ctas >= (1ull << 31)) return HX_ERR_ARG;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((uint32_t)ctas);
  c.blockDim = dim3(S::kThreads);
  c.dynamicSmemBytes = S::kSmem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {S::kCtas * a.splits, 1, 1};
  c.attrs = at, c.numAttrs = 1;
  if (cudaLaunchKernelEx(&c, kernel, map, a) != cudaSuccess) {
    cudaGetLastError();
    return HX_ERR_CUDA;
  }
  return HX_OK;
}
template <typename T, int MT, bool kPair>
int launch(const CUtensorMap& map, const Args& a, cudaStream_t s) {
  if (a.fmt == HX_ROWS_E4M3) return launch_tile<T, MT, kPair, 1>(map, a, s);
  if constexpr (MT == 2 && kRestApart<T, 2>)
    return HX_ERR_ARG;  // plan() does not give it: its sums would need 1024 columns of TMEM
  else
    return launch_tile<T, MT, kPair, 2>(map, a, s);
}

// The tile and the number of splits of the tokens, by the estimated time: rounds of CTAs over the SMs, each
// its steps of 64 tokens and a fixed part (start, first loads, last products, stores), in nanoseconds as measured on
// B200 (e4m3, INT8). A 128 x 128 tile's step is bound by shared memory (64 KB in and out, 512 clocks for 256 of
// products), a pair's 256 x 256 as much for twice the products per CTA, a pair's 512 x 256 by the products. So: large
// tiles where they fill the GPU, else small ones with more splits. Measured (us), e4m3, tokens x out x in:
//   4096 x 256 x 256    one tile each: 26.6 / 27.7 / 42.4;  128 x 128 in 8 splits 10.6
//   4096 x 1024 x 1024  27.3 / 28.4 / 44.1;  256 x 256 in 3 splits 18.0, 128 x 128 in 2 18.8
//   8192 x 2048 x 2048  95.8 / 51.2 / 79.9
//   4096 x 4096 x 4096  183 / 114 / 94
// INT8 rows in f16 have two accumulators per 128 rows, and the 512 x 256 tile no room for them: 4096^3 199 us (bf16, with
// that tile, 182), 300 x 8192 x 8192 154 (104).
struct Plan {
  int mt;
  bool pair;
  uint32_t splits;
};
Plan plan(uint32_t fmt, bool rest_apart, uint64_t tokens, uint64_t n_out, uint64_t n_in) {
  struct Kind {
    int mt;
    bool pair;
    uint64_t rows, cols, step[2], fixed, join;
  };
  static constexpr Kind kinds[3] = {{1, false, 128, 128, {325, 490}, 5000, 2200},
                                    {1, true, 256, 256, {320, 555}, 6000, 3600},
                                    {2, true, 512, 256, {555, 1110}, 8000, 0}};
  // SMs that clusters of 1 .. 8 CTAs, one per SM, can have at once (the runtime's count of clusters on a B200)
  static constexpr uint64_t kSms[kMaxCluster + 1] = {0, 148, 148, 135, 132, 130, 132, 105, 120};
  const uint64_t steps = ceil_div(tokens, kStep);
  Plan best{1, false, 1};
  uint64_t least = ~0ull;
  for (const Kind& k : kinds) {
    if (k.mt == 2 && rest_apart) continue;  // twice the accumulators do not fit
    const uint64_t ctas = ceil_div(n_out, k.rows) * ceil_div(n_in, k.cols) * (k.pair ? 2 : 1);
    const uint64_t most = k.mt == 2 ? 1 : kMaxCluster / (k.pair ? 2 : 1);
    for (uint64_t s = 1; s <= most && s <= std::max<uint64_t>(1, steps); ++s) {
      const uint64_t per = ceil_div(steps, s);
      if (s > 1 && ceil_div(steps, per) != s) continue;  // an empty split
      const uint64_t t = ceil_div(ctas * s, kSms[s * (k.pair ? 2 : 1)]) * (per * k.step[fmt == HX_ROWS_INT8] + k.fixed + (s > 1 ? k.join : 0));
      if (t < least) least = t, best = Plan{k.mt, k.pair, (uint32_t)s};
    }
  }
  return best;
}

template <typename T>
int run(const Plan& p, const CUtensorMap& map, const Args& a, cudaStream_t s) {
  if (p.mt == 2) return launch<T, 2, true>(map, a, s);
  return p.pair ? launch<T, 1, true>(map, a, s) : launch<T, 1, false>(map, a, s);
}

bool bad_sizes(uint64_t tokens, uint64_t n_out, uint64_t n_in) {
  return tokens >= (1ull << 31) - 64 || !n_out || !n_in || n_out > (1ull << 23) || n_in > (1ull << 22);
}

// What is copied to aligned rows first, and where: bytes of the workspace for dY, then for X.
struct Copies {
  uint64_t dy, x;
};
Copies copies(const void* dy, uint64_t ld_dy, const void* bytes, uint64_t tokens, uint64_t n_out, uint64_t n_in) {
  Copies c{};
  if (!multiple(dy, 16) || (tokens > 1 && ld_dy % 8)) c.dy = tokens * ((n_out + 7) / 8 * 16);
  if (!multiple(bytes, 8) || n_in % 8) c.x = tokens * ((n_in + 15) / 16 * 16);
  return c;
}

}  // namespace

extern "C" {

uint64_t hx_weight_grad_workspace(const void* d_dy, uint64_t ld_dy, const uint8_t* d_bytes, uint64_t tokens,
                                  uint64_t n_out, uint64_t n_in) {
  if (bad_sizes(tokens, n_out, n_in)) return 0;
  const Copies c = copies(d_dy, ld_dy, d_bytes, tokens, n_out, n_in);
  return c.dy + c.x;
}

int hx_weight_grad_bounded(uint32_t format, uint32_t dtype, const void* d_dy, uint64_t ld_dy, const uint8_t* d_bytes,
                           const float* d_scale, uint64_t tokens, uint64_t n_out, uint64_t n_in, uint32_t dw_dtype,
                           void* d_dw, uint64_t ld_dw, int accumulate, void* d_workspace, uint64_t workspace_bytes,
                           uint32_t* d_status, uint64_t wait_ns, uint64_t withhold, void* stream) {
  if (format > HX_ROWS_INT8 || (dtype != HX_F16 && dtype != HX_BF16) || (dw_dtype != HX_F32 && dw_dtype != dtype))
    return HX_ERR_ARG;
  if (bad_sizes(tokens, n_out, n_in) || (tokens > 1 && ld_dy < n_out) || (n_out > 1 && ld_dw < n_in)) return HX_ERR_ARG;
  if (!d_dw || !multiple(d_dw, dw_dtype == HX_F32 ? 4 : 2) || !multiple(d_status, 4)) return HX_ERR_ARG;
  if (tokens && (!d_dy || !d_bytes || !d_scale || !multiple(d_dy, 2) || !multiple(d_scale, 4))) return HX_ERR_ARG;
  if (tokens > 1 && ld_dy >= (1ull << 39)) return HX_ERR_ARG;  // TMA's largest stride
  if (!tokens && accumulate) return HX_OK;
  const Copies need = copies(d_dy, ld_dy, d_bytes, tokens, n_out, n_in);
  if (need.dy + need.x && (!d_workspace || !multiple(d_workspace, 16) || workspace_bytes < need.dy + need.x))
    return HX_ERR_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Plan p = plan(format, format == HX_ROWS_INT8 && dtype == HX_F16, tokens, n_out, n_in);
  Args a{};
  a.fmt = format, a.bytes = d_bytes, a.ld_x = n_in, a.scale = d_scale;
  a.tokens = tokens, a.n_out = (uint32_t)n_out, a.n_in = (uint32_t)n_in;
  a.dw = d_dw, a.ld_dw = ld_dw, a.dw_dtype = dw_dtype, a.accumulate = accumulate != 0;
  a.dw_wide = multiple(d_dw, 16) && (n_out == 1 || ld_dw * (dw_dtype == HX_F32 ? 4 : 2) % 16 == 0);
  a.splits = p.splits, a.steps = (uint32_t)ceil_div(tokens, kStep), a.status = d_status;
  a.wait_ns = wait_ns, a.withhold = withhold;
  const void* dy = d_dy;
  uint64_t pitch = tokens > 1 ? ld_dy * 2 : (n_out + 7) / 8 * 16;
  if (need.dy + need.x) {
    uint8_t* w = static_cast<uint8_t*>(d_workspace);
    const uint64_t by = ceil_div(need.dy / 16, 256), bx = ceil_div(need.x / 16, 256), most = 148 * 8;
    const uint32_t gy = (uint32_t)std::min(by, most), gx = (uint32_t)std::min(bx, most);
    k_wgrad_align<<<gy + gx, 256, 0, s>>>(static_cast<const uint16_t*>(d_dy), ld_dy, n_out, reinterpret_cast<uint4*>(w),
                                          d_bytes, n_in, reinterpret_cast<uint4*>(w + need.dy), tokens, gy);
    if (const int rc = launched()) return rc;
    if (need.dy) dy = w, pitch = (n_out + 7) / 8 * 16;
    if (need.x) a.bytes = w + need.dy, a.ld_x = (n_in + 15) / 16 * 16;
  }
  CUtensorMap map{};
  if (tokens) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return HX_ERR_CUDA;
    const cuuint64_t dims[2] = {n_out, tokens}, strides[1] = {pitch};
    const cuuint32_t box[2] = {64, kStep}, unit[2] = {1, 1};
    const auto encode = [&] {
      return fn(&map, dtype == HX_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                const_cast<void*>(dy), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult rc = encode();
    // a host thread's first CUDA call: the runtime makes the device's context current, a driver call does not
    int dev = 0;
    if (rc == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) rc = encode();
    if (rc != CUDA_SUCCESS) return HX_ERR_CUDA;
  }
  return dtype == HX_F16 ? run<__half>(p, map, a, s) : run<__nv_bfloat16>(p, map, a, s);
}

int hx_weight_grad(uint32_t format, uint32_t dtype, const void* d_dy, uint64_t ld_dy, const uint8_t* d_bytes,
                   const float* d_scale, uint64_t tokens, uint64_t n_out, uint64_t n_in, uint32_t dw_dtype,
                   void* d_dw, uint64_t ld_dw, int accumulate, void* d_workspace, uint64_t workspace_bytes,
                   uint32_t* d_status, void* stream) {
  return hx_weight_grad_bounded(format, dtype, d_dy, ld_dy, d_bytes, d_scale, tokens, n_out, n_in, dw_dtype, d_dw, ld_dw,
                                accumulate, d_workspace, workspace_bytes, d_status, kWaitNs, ~0ull, stream);
}

}  // extern "C"
