// Per-head RMS norm of queries and keys with the position rotation in the same pass (sm_100a), its
// inputs kept as 8-bit rows, and the backward pass that reads those rows.
//
// Forward, for head h of token t with x = x[t][h], D values:
//     r = (mean(x^2) + eps)^(-1/2),  n = x r w (w: the queries' or the keys' weight),
//     y = n with each of its first `rot` values' pairs (a, b) turned by the token's angle:
//         (a c - b s, b c + a s).
// Backward at the saved x~: g = dy turned back, dw = sum over heads and tokens of g x~ r,
//     d = g w,  dx = r (d - x~ r mean(d x~ r)).
//
// Both read and write each value once and are bound by memory. A group of L lanes holds one head, 16
// values per lane, arranged so that both values of a pair are in the same lane (two vectors of PU
// values each): the rotation needs no exchange, the norm one butterfly over L lanes. A group takes up to 8 heads
// of one token one after another, with the token's cosines and sines and the weight in registers; the next four heads'
// values come ahead through asynchronous copies into the thread's own slots of shared memory.
//
// Measured on B200, 8192 tokens of 32 + 8 heads of 128 in bf16, e4m3 rows: forward 39.6 us, backward 49.3 with the weight
// gradients; the bytes at the measured copy rate take 32.7. Without the copies ahead 45.8 and 57.4, whatever
// arithmetic was left out: too few loads in flight. Of the forward pass's loads a third are for nothing: past an item's last
// head the copies ahead go to that head again (L2 answers them). Backward, registers hold it to two blocks of 256 threads per SM
// (120; three blocks spill and take 102 us). At these limits single values per vector spill up to 116 bytes backward, and INT8 from
// bf16 or f32 up to 24 forward.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "hx.h"
#include "hx_values.h"

namespace {

using namespace hxv;

constexpr int kThreads = 256;
constexpr int kMaxDim = 512;       // 32 lanes of 16 values
constexpr int kMaxBlocks = 1024;   // backward: rows of partial weight gradients in the workspace

struct Args {
  uint32_t fmt, w_f32;
  const void* x;       // forward: x; backward: dy
  uint64_t xt, xh;     // element strides of tokens and heads
  void* y;             // forward: y; backward: dx
  uint64_t yt, yh;
  uint8_t* bytes;      // forward: written or null; backward: read
  float* scale;
  uint64_t tokens;
  uint32_t nq, nk, dim, rot;
  const void *wq, *wk;
  const float *cos, *sin;
  const void* pos;
  uint32_t pos64;
  uint64_t places;
  float eps;
  uint32_t* status;
  uint32_t lanes, per;  // lanes per head, heads per item
  float* part;          // backward: [blocks][dim]
  float *dwq, *dwk;     // backward, with one block each at most: written by it
  uint32_t blocks_q;    // backward: the first blocks take queries, the others keys
};

// The places of a lane's values: unit u is two vectors of PU values at off0 and off1. Pairs half the rotated width
// apart: the two vectors of a turned unit hold them, with the angles PU u ..; vectors behind the rotated ones are
// neighbours. Interleaved pairs lie inside a vector, so its two vectors are half the head apart (the lanes' vectors are
// then neighbours, and a warp's loads and stores whole lines), each with the angles off / 2 ..; vectors of one value: the pair.
template <int PU, bool kInter>
struct Units {
  static constexpr bool kApart = kInter && PU > 1;
  uint32_t units, turned, half, far, rot;
  __device__ Units(const Args& a)
      : units(a.dim / (2 * PU)), turned(a.rot / (2 * PU)), half(a.rot / 2), far(a.dim / 2), rot(a.rot) {}
  __device__ bool has(uint32_t u) const { return u < units; }
  __device__ uint32_t off0(uint32_t u) const { return kApart || (!kInter && u < turned) ? PU * u : 2 * PU * u; }
  __device__ uint32_t off1(uint32_t u) const {
    return kApart ? far + PU * u : !kInter && u < turned ? half + PU * u : 2 * PU * u + PU;
  }
};

// A lane's 16 values as 8 slots of two. Vectors of 2 or more: slots are neighbours, first those of vector 0, then those of vector 1; vectors of 1: slot j is unit j's (a, b).
// The other value of a pair is in the same slot (kSwap) or in the same place of the other vector.
template <int PU, bool kInter>
struct Slots {
  static constexpr int N = 8 / PU, H = PU / 2;
  static constexpr bool kSwap = kInter || PU == 1;
  // the slot that holds the pairs' other values, to be swapped if kSwap
  static constexpr __device__ int other(int k) { return kSwap ? k : k % PU < H ? k + H : k - H; }
};

// (Two scalar operations: the packed ones save nothing forward, 45.1 against 45.9 us, and cost moves to register pairs
// backward, 62.5 against 57.9.)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 swapped(float2 v) { return make_float2(v.y, v.x); }

template <int PU>
__device__ __forceinline__ void to_slots(int j, const float (&f0)[PU], const float (&f1)[PU], float2 (&v)[8]) {
  if constexpr (PU == 1) {
    v[j] = make_float2(f0[0], f1[0]);
  } else {
#pragma unroll
    for (int i = 0; i < PU / 2; ++i) {
      v[j * PU + i] = make_float2(f0[2 * i], f0[2 * i + 1]);
      v[j * PU + PU / 2 + i] = make_float2(f1[2 * i], f1[2 * i + 1]);
    }
  }
}
template <int PU>
__device__ __forceinline__ void from_slots(int j, const float2 (&v)[8], float (&f0)[PU], float (&f1)[PU]) {
  if constexpr (PU == 1) {
    f0[0] = v[j].x, f1[0] = v[j].y;
  } else {
#pragma unroll
    for (int i = 0; i < PU / 2; ++i) {
      f0[2 * i] = v[j * PU + i].x, f0[2 * i + 1] = v[j * PU + i].y;
      f1[2 * i] = v[j * PU + PU / 2 + i].x, f1[2 * i + 1] = v[j * PU + PU / 2 + i].y;
    }
  }
}

// Butterflies over a group's lanes: a sum and a maximum, or two sums, in the same rounds.
__device__ __forceinline__ void group_sum_max(float& v, uint32_t& m, uint32_t lanes) {
  for (uint32_t o = lanes >> 1; o; o >>= 1) {
    v += __shfl_xor_sync(0xffffffffu, v, o);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
}
__device__ __forceinline__ void group_sums(float& v, float& w, uint32_t lanes) {
  for (uint32_t o = lanes >> 1; o; o >>= 1) {
    v += __shfl_xor_sync(0xffffffffu, v, o);
    w += __shfl_xor_sync(0xffffffffu, w, o);
  }
}

template <typename T, int PU, bool kInter>
__device__ __forceinline__ void load_weight(const Args& a, const void* w, uint32_t sub, float2 (&out)[8]) {
  const Units<PU, kInter> un(a);
#pragma unroll
  for (int j = 0; j < 8 / PU; ++j) {
    const uint32_t u = j * a.lanes + sub;
    float f0[PU], f1[PU];
    if (!un.has(u)) {
#pragma unroll
      for (int i = 0; i < PU; ++i) f0[i] = f1[i] = 0.0f;
    } else if (a.w_f32) {
      Vec<float, PU> v;
      v.load(static_cast<const float*>(w) + un.off0(u));
      v.floats(f0);
      v.load(static_cast<const float*>(w) + un.off1(u));
      v.floats(f1);
    } else {
      Vec<T, PU> v;
      v.load(static_cast<const T*>(w) + un.off0(u));
      v.floats(f0);
      v.load(static_cast<const T*>(w) + un.off1(u));
      v.floats(f1);
    }
    to_slots<PU>(j, f0, f1, out);
  }
}

// The token's turn of the lane's slots: v -> v * c + (the pairs' other values) * s; c = 1 and s = 0
// where nothing turns. `sign` 1: forward; -1: back. Returns false, with nothing turned, for a
// position outside the tables.
template <int PU, bool kInter>
__device__ __forceinline__ bool load_turn(const Args& a, uint64_t t, uint32_t sub, float sign, float2 (&c)[8],
                                          float2 (&s)[8]) {
  using S = Slots<PU, kInter>;
  const Units<PU, kInter> un(a);
  const int64_t p = a.pos64 ? static_cast<const int64_t*>(a.pos)[t]
                            : (int64_t) static_cast<const int32_t*>(a.pos)[t];
  const bool ok = p >= 0 && (uint64_t)p < a.places;
#pragma unroll
  for (int j = 0; j < S::N; ++j) {
    const uint32_t u = j * a.lanes + sub;
    float fc[PU], fs[PU];
#pragma unroll
    for (int i = 0; i < PU; ++i) fc[i] = 1.0f, fs[i] = 0.0f;
    if constexpr (Units<PU, kInter>::kApart) {
      // half a vector of pairs in each
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t off = k ? un.off1(u) : un.off0(u);
        if (ok && un.has(u) && off < un.rot) {
          const uint64_t at = (uint64_t)p * un.half + off / 2;
          float g[PU / 2];
          Vec<float, PU / 2> v;
          v.load(a.cos + at);
          v.floats(g);
#pragma unroll
          for (int i = 0; i < PU / 2; ++i) fc[k * (PU / 2) + i] = g[i];
          v.load(a.sin + at);
          v.floats(g);
#pragma unroll
          for (int i = 0; i < PU / 2; ++i) fs[k * (PU / 2) + i] = g[i];
        }
      }
    } else if (ok && u < un.turned) {
      const uint64_t at = (uint64_t)p * un.half + PU * u;
      Vec<float, PU> v;
      v.load(a.cos + at);
      v.floats(fc);
      v.load(a.sin + at);
      v.floats(fs);
    }
    // pair (a, b) -> (a c - b s, b c + a s)
#pragma unroll
    for (int i = 0; i < PU; ++i) {
      if constexpr (S::kSwap) {
        c[j * PU + i] = both(fc[i]);
        s[j * PU + i] = make_float2(-sign * fs[i], sign * fs[i]);
      } else if (i < S::H) {
        c[j * PU + i] = c[j * PU + S::H + i] = make_float2(fc[(2 * i) % PU], fc[(2 * i + 1) % PU]);
        const float2 v = make_float2(sign * fs[(2 * i) % PU], sign * fs[(2 * i + 1) % PU]);
        s[j * PU + i] = make_float2(-v.x, -v.y);
        s[j * PU + S::H + i] = v;
      }
    }
  }
  if (!ok && a.status && sub == 0) atomicOr(a.status, (uint32_t)HX_ERR_ARG);
  return ok;
}

// ------------------------------------------------------------------------------ loads ahead
// A thread's vectors of the next heads, on their way through asynchronous copies into slots of shared memory that only
// this thread reads (so that they need neither registers nor a barrier). B: bytes of one vector, 1 .. 32 (1 and 2 have no
// asynchronous copy: loaded and stored).
constexpr int kAhead = 4;
template <int B>
__device__ __forceinline__ void copy_ahead(uint32_t slot, const void* p) {
  if constexpr (B == 32) {
    copy_ahead<16>(slot, p);
    copy_ahead<16>(slot + 16 * kThreads, static_cast<const uint8_t*>(p) + 16);
  } else if constexpr (B == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot), "l"(p) : "memory");
  } else if constexpr (B >= 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(slot), "l"(p), "n"(B) : "memory");
  } else if constexpr (B == 2) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(slot), "h"(*static_cast<const uint16_t*>(p)) : "memory");
  } else {
    asm volatile("st.shared.b8 [%0], %1;" ::"r"(slot), "r"((uint32_t)*static_cast<const uint8_t*>(p)) : "memory");
  }
}
__device__ __forceinline__ void ahead_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void ahead_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory"); }
template <typename T, int PU>
__device__ __forceinline__ void read_ahead(uint32_t slot, Vec<T, PU>& v) {
  constexpr int B = PU * sizeof(T);
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i)
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v.r[4 * i]), "=r"(v.r[4 * i + 1]), "=r"(v.r[4 * i + 2]), "=r"(v.r[4 * i + 3])
                   : "r"(slot + i * 16 * kThreads)
                   : "memory");
  } else if constexpr (B == 8) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.r[0]), "=r"(v.r[1]) : "r"(slot) : "memory");
  } else if constexpr (B == 4) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v.r[0]) : "r"(slot) : "memory");
  } else {
    uint16_t h;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h) : "r"(slot) : "memory");
    v.r[0] = h;
  }
}

template <int PU>
__device__ __forceinline__ void read_ahead(uint32_t slot, Bytes<PU>& v) {
  if constexpr (PU == 8) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.b[0]), "=r"(v.b[1]) : "r"(slot) : "memory");
  } else if constexpr (PU == 4) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v.b[0]) : "r"(slot) : "memory");
  } else if constexpr (PU == 2) {
    uint16_t h;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h) : "r"(slot) : "memory");
    v.b[0] = h;
  } else {
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v.b[0]) : "r"(slot) : "memory");
  }
}

// Item i as (token, chunk of heads).
__device__ __forceinline__ void split_item(uint64_t i, uint32_t chunks, uint64_t& t, uint32_t& ch) {
  t = i >> 32 ? i / chunks : (uint32_t)i / chunks;
  ch = (uint32_t)(i - t * chunks);
}

// With the weight folded into the turn, y = r (x * (w c) + other(x) * (other(w) s)): the products
// w c and w s are made once per token and group of heads.
template <typename T, int PU, bool kInter, uint32_t kFmt>
__global__ void __launch_bounds__(kThreads, 3) k_qk_forward(const __grid_constant__ Args a) {
  using S = Slots<PU, kInter>;
  const Units<PU, kInter> un(a);
  const uint32_t sub = threadIdx.x % a.lanes, groups = kThreads / a.lanes;
  const uint64_t item = blockIdx.x * (uint64_t)groups + threadIdx.x / a.lanes;
  const uint32_t cq = (a.nq + a.per - 1) / a.per, chunks = cq + (a.nk + a.per - 1) / a.per;
  const bool live = item < a.tokens * chunks;
  uint64_t t = 0;
  uint32_t ch = 0;
  if (live) split_item(item, chunks, t, ch);
  const bool key = ch >= cq;
  const uint32_t h0 = key ? a.nq + (ch - cq) * a.per : ch * a.per;
  const uint32_t h1 = live ? min(h0 + a.per, key ? a.nq + a.nk : a.nq) : h0;

  constexpr int B = PU * sizeof(T), kSlot = 16 * sizeof(T) * kThreads;  // a head's 16 values of every thread
  extern __shared__ __align__(16) uint8_t ahead[];
  const uint32_t slots = (uint32_t)__cvta_generic_to_shared(ahead) + threadIdx.x * (B < 16 ? B : 16);
  const T* x = static_cast<const T*>(a.x) + t * a.xt + h0 * a.xh;
  T* y = static_cast<T*>(a.y) + t * a.yt + h0 * a.yh;
  const uint64_t row = t * (a.nq + a.nk) + h0;
  uint8_t* bytes = a.bytes + row * a.dim;
  float* scale = a.scale + row;
  // past the item's last head the loads go to that head again; a lane without values reads the head's first ones and
  // clears them on use
  const bool idle = un.units < a.lanes * S::N;
  auto fetch = [&](uint32_t h) {
    const uint32_t slot = slots + (h - h0) % kAhead * kSlot;
#pragma unroll
    for (int j = 0; j < S::N; ++j) {
      const uint32_t u = j * a.lanes + sub, v = un.has(u) ? u : 0;
      copy_ahead<B>(slot + (2 * j) * B * kThreads, x + un.off0(v));
      copy_ahead<B>(slot + (2 * j + 1) * B * kThreads, x + un.off1(v));
    }
    ahead_commit();
    if (h + 1 < h1) x += a.xh;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(h0 + i);
  float2 c[8], s[8];
  bool ok;
  {
    float2 w[8];
    load_weight<T, PU, kInter>(a, key ? a.wk : a.wq, sub, w);
    ok = load_turn<PU, kInter>(a, t, sub, 1.0f, c, s);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      c[k] = mul2(c[k], w[k]);
      s[k] = mul2(s[k], S::kSwap ? swapped(w[k]) : w[S::other(k)]);
    }
  }
  const float part = 1.0f / (float)a.dim;
  for (uint32_t k = 0; k < a.per; ++k) {  // the same count in every lane: the butterflies need all
    const uint32_t h = h0 + k;
    float2 v[8], q = both(0.0f);
    uint32_t top = 0;
    ahead_wait();
#pragma unroll
    for (int j = 0; j < S::N; ++j) {
      float f0[PU], f1[PU];
      Vec<T, PU> v0[S::N], v1[S::N];
      const uint32_t slot = slots + k % kAhead * kSlot;
      read_ahead<T, PU>(slot + (2 * j) * B * kThreads, v0[j]);
      read_ahead<T, PU>(slot + (2 * j + 1) * B * kThreads, v1[j]);
      if (idle && !un.has(j * a.lanes + sub)) v0[j].zero(), v1[j].zero();
      v0[j].floats(f0);
      v1[j].floats(f1);
      to_slots<PU>(j, f0, f1, v);
      if (a.bytes) top = v1[j].top(v0[j].top(top));
    }
    fetch(h + kAhead);
#pragma unroll
    for (int i = 0; i < 8; ++i) q = fma2(v[i], v[i], q);
    float sq = q.x + q.y;
    if (a.bytes) top = top_bits<T>(top);
    group_sum_max(sq, top, a.lanes);
    float r = rsqrtf(fmaf(sq, part, a.eps));
    if (!ok) r = __uint_as_float(0x7fc00000u);
    if (a.bytes) {
      const Scale sc = scale_of<T>(kFmt, top);
      if (h < h1) {
        if (sub == 0) *scale = sc.s;
#pragma unroll
        for (int j = 0; j < S::N; ++j) {
          const uint32_t u = j * a.lanes + sub;
          if (!un.has(u)) continue;
          float f0[PU], f1[PU];
          from_slots<PU>(j, v, f0, f1);
          to_bytes<T, PU, false>(kFmt, f0, sc).store(bytes + un.off0(u));
          to_bytes<T, PU, false>(kFmt, f1, sc).store(bytes + un.off1(u));
        }
      }
      if (kFmt == HX_ROWS_INT8 && sizeof(T) == 2 && __any_sync(0xffffffffu, huge<T>(sc))) {
        // the division, from the head itself (its normalised values, which may lie in the same place, come later). Asked
        // of the whole warp: 45 us for 8192 tokens of 40 bf16 heads of 128 values, 47 with a branch of each lane's own.
        split_item(item, chunks, t, ch);
        const T* xh = static_cast<const T*>(a.x) + t * a.xt + h * a.xh;
#pragma unroll 1
        for (uint32_t u = sub; h < h1 && huge<T>(sc) && un.has(u); u += a.lanes) {
#pragma unroll 1
          for (uint32_t i = 0; i < 2 * PU; ++i) {
            const uint32_t at = i < PU ? un.off0(u) + i : un.off1(u) + i - PU;
            const float f[1] = {Type<T>::to_f(xh[at])};
            to_bytes<T, 1>(kFmt, f, sc).store(bytes + at);
          }
        }
      }
    }
    float2 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = mul2(fma2(v[i], c[i], mul2(S::kSwap ? swapped(v[i]) : v[S::other(i)], s[i])), both(r));
    if (h < h1) {
#pragma unroll
      for (int j = 0; j < S::N; ++j) {
        const uint32_t u = j * a.lanes + sub;
        if (!un.has(u)) continue;
        float f0[PU], f1[PU];
        from_slots<PU>(j, o, f0, f1);
        store<T, PU>(y + un.off0(u), f0);
        store<T, PU>(y + un.off1(u), f1);
      }
    }
    y += a.yh;
    bytes += a.dim;
    ++scale;
  }
}

// In terms of the bytes' values q (x~ = s q): n = q s r, dw += g n, dx = r (g w - n mean(g w n)).
template <typename T, int PU, bool kInter, uint32_t kFmt>
__global__ void __launch_bounds__(kThreads, 2) k_qk_backward(const __grid_constant__ Args a) {
  using S = Slots<PU, kInter>;
  __shared__ float sums[kThreads * 16];
  const Units<PU, kInter> un(a);
  const uint32_t sub = threadIdx.x % a.lanes, groups = kThreads / a.lanes;
  const uint32_t group = threadIdx.x / a.lanes;
  const bool key = blockIdx.x >= a.blocks_q;
  const uint32_t first = key ? a.nq : 0, heads = key ? a.nk : a.nq;
  const uint32_t chunks = (heads + a.per - 1) / a.per;
  const uint32_t blocks = key ? gridDim.x - a.blocks_q : a.blocks_q;
  const uint32_t block = key ? blockIdx.x - a.blocks_q : blockIdx.x;
  const uint64_t items = a.tokens * chunks;
  const bool idle = un.units < a.lanes * S::N;
  const float part = 1.0f / (float)a.dim;

  float2 w[8], dw[8];
  load_weight<T, PU, kInter>(a, key ? a.wk : a.wq, sub, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = both(0.0f);

  // Slots of a head's values of dy, its bytes and its scale, of every thread. The loads run kAhead heads before their use,
  // through the items in the same order; past an item's last head they go to that head again, past the last item
  // to that item, and a lane without values reads the head's first ones and clears them on use. (An item that is
  // not live reads token 0's first head, and stores nothing.)
  constexpr int B = PU * sizeof(T), kDy = 16 * sizeof(T) * kThreads, kSlot = kDy + 20 * kThreads;
  extern __shared__ __align__(16) uint8_t ahead[];
  const uint32_t slots = (uint32_t)__cvta_generic_to_shared(ahead);
  const uint32_t slot_x = slots + threadIdx.x * (B < 16 ? B : 16), slot_b = slots + kDy + threadIdx.x * PU;
  const uint32_t slot_s = slots + kDy + 16 * kThreads + threadIdx.x * 4;
  struct Item {
    uint64_t t;
    uint32_t h0, n;
  };
  auto item_at = [&](uint64_t base) {
    const uint64_t item = base + group;
    Item it{0, first, 0};
    if (item < items) {
      uint32_t ch;
      split_item(item, chunks, it.t, ch);
      it.h0 = first + ch * a.per;
      it.n = min(a.per, first + heads - it.h0);
    }
    return it;
  };
  const uint64_t step = (uint64_t)blocks * groups;
  uint64_t at = (uint64_t)block * groups;  // of the loads
  uint32_t at_k = 0, at_n = 0, slot = 0;
  const T* dy = nullptr;
  const uint8_t* bytes = nullptr;
  const float* scales = nullptr;
  auto go_to = [&](uint64_t base) {
    const Item it = item_at(base);
    const uint64_t row = it.t * (a.nq + a.nk) + it.h0;
    dy = static_cast<const T*>(a.x) + it.t * a.xt + it.h0 * a.xh;
    bytes = a.bytes + row * a.dim;
    scales = a.scale + row;
    at_n = it.n;
  };
  auto fetch = [&]() {
    const uint32_t o = slot * kSlot;
    copy_ahead<4>(slot_s + o, scales);
#pragma unroll
    for (int j = 0; j < S::N; ++j) {
      const uint32_t u = j * a.lanes + sub, v = un.has(u) ? u : 0;
      copy_ahead<B>(slot_x + o + (2 * j) * B * kThreads, dy + un.off0(v));
      copy_ahead<B>(slot_x + o + (2 * j + 1) * B * kThreads, dy + un.off1(v));
      copy_ahead<PU>(slot_b + o + (2 * j) * PU * kThreads, bytes + un.off0(v));
      copy_ahead<PU>(slot_b + o + (2 * j + 1) * PU * kThreads, bytes + un.off1(v));
    }
    ahead_commit();
    slot = (slot + 1) % kAhead;
    if (++at_k == a.per) {
      at_k = 0;
      if (at + step < items) at += step;
      go_to(at);
    } else if (at_k < at_n) {
      dy += a.xh, bytes += a.dim, ++scales;
    }
  };
  if ((uint64_t)block * groups < items) {
    go_to(at);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch();
  }

  for (uint64_t base = (uint64_t)block * groups; base < items; base += step) {
    const Item it = item_at(base);
    float2 c[8], s[8];
    T* dx = static_cast<T*>(a.y) + it.t * a.yt + it.h0 * a.yh;
    const bool ok = load_turn<PU, kInter>(a, it.t, sub, -1.0f, c, s);
    for (uint32_t k = 0; k < a.per; ++k) {
      const bool live = k < it.n;
      float2 g[8], q[8];
      ahead_wait();
      const uint32_t o = slot * kSlot;  // the oldest, and the next to be filled
      float scale;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(scale) : "r"(slot_s + o) : "memory");
#pragma unroll
      for (int j = 0; j < S::N; ++j) {
        float f0[PU], f1[PU];
        Vec<T, PU> v0, v1;
        Bytes<PU> b0, b1;
        read_ahead<T, PU>(slot_x + o + (2 * j) * B * kThreads, v0);
        read_ahead<T, PU>(slot_x + o + (2 * j + 1) * B * kThreads, v1);
        read_ahead<PU>(slot_b + o + (2 * j) * PU * kThreads, b0);
        read_ahead<PU>(slot_b + o + (2 * j + 1) * PU * kThreads, b1);
        if (idle && !un.has(j * a.lanes + sub)) {
          v0.zero();
          v1.zero();
#pragma unroll
          for (int i = 0; i < Bytes<PU>::kRaw; ++i) b0.b[i] = b1.b[i] = 0;
        }
        v0.floats(f0);
        v1.floats(f1);
        to_slots<PU>(j, f0, f1, g);
        to_values<PU>(kFmt, b0, 1.0f, f0);
        to_values<PU>(kFmt, b1, 1.0f, f1);
        to_slots<PU>(j, f0, f1, q);
      }
      fetch();
      {
        float2 o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fma2(g[i], c[i], mul2(S::kSwap ? swapped(g[i]) : g[S::other(i)], s[i]));
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = o[i];
      }
      float2 sq2 = both(0.0f), dot2 = both(0.0f), gq[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sq2 = fma2(q[i], q[i], sq2);
        gq[i] = mul2(g[i], q[i]);
        dot2 = fma2(gq[i], w[i], dot2);
      }
      float sq = sq2.x + sq2.y, dot = dot2.x + dot2.y;
      group_sums(sq, dot, a.lanes);
      sq = sq * scale * scale, dot *= scale;  // (the scale's square alone falls out of 32 bits long before the sum does)
      float r = rsqrtf(fmaf(sq, part, a.eps));
      if (!ok) r = __uint_as_float(0x7fc00000u);
      const float sr = scale * r;                // n = q sr
      const float2 m = both(-dot * r * part * sr * r);  // dx = g w r - q (mean(g w n) s r r)
      if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[i] = fma2(gq[i], both(sr), dw[i]);
          g[i] = fma2(mul2(g[i], w[i]), both(r), mul2(q[i], m));
        }
#pragma unroll
        for (int j = 0; j < S::N; ++j) {
          const uint32_t u = j * a.lanes + sub;
          if (!un.has(u)) continue;
          float f0[PU], f1[PU];
          from_slots<PU>(j, g, f0, f1);
          store<T, PU>(dx + un.off0(u), f0);
          store<T, PU>(dx + un.off1(u), f1);
        }
      }
      dx += a.yh;
    }
  }

  // (the kernel that adds the blocks' sums may be set up from here on; it waits for this one's end)
  asm volatile("griddepcontrol.launch_dependents;");
  // the block's sum of its groups' weight gradients, in the groups' order
  float* mine = sums + group * (16 * a.lanes);
#pragma unroll
  for (int j = 0; j < S::N; ++j) {
    const uint32_t u = j * a.lanes + sub;
    if (!un.has(u)) continue;
    float f0[PU], f1[PU];
    from_slots<PU>(j, dw, f0, f1);
#pragma unroll
    for (int i = 0; i < PU; ++i) {
      mine[un.off0(u) + i] = f0[i];
      mine[un.off1(u) + i] = f1[i];
    }
  }
  __syncthreads();
  for (uint32_t d = threadIdx.x; d < a.dim; d += kThreads) {
    float v = 0.0f;
    for (uint32_t g = 0; g < groups; ++g) v += sums[g * (16 * a.lanes) + d];
    if (blocks == 1)
      (key ? a.dwk : a.dwq)[d] = v;
    else
      a.part[(uint64_t)blockIdx.x * a.dim + d] = v;
  }
}

// Sums the blocks' partial weight gradients in a fixed order: 32 interleaved sums per column, then
// those 32. blockIdx.y: 0 queries, 1 keys.
__global__ void __launch_bounds__(1024) k_qk_weights(const float* __restrict__ part, uint32_t dim,
                                                     uint32_t blocks_q, uint32_t blocks,
                                                     float* dwq, float* dwk) {
  __shared__ float rows[32][33];
  const uint32_t x = threadIdx.x & 31, k = threadIdx.x >> 5, d = blockIdx.x * 32 + x;
  const uint32_t lo = blockIdx.y ? blocks_q : 0, hi = blockIdx.y ? blocks : blocks_q;
  float* dw = blockIdx.y ? dwk : dwq;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (hi - lo == 1) return;  // written by its one block
  float v = 0.0f;
  for (uint32_t b = lo + k; b < hi; b += 256) {  // eight loads at once: one round for the 256 rows a class mostly has
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = d < dim && b + 32 * i < hi ? part[(uint64_t)(b + 32 * i) * dim + d] : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += p[i];
  }
  rows[k][x] = v;
  __syncthreads();
  v = rows[x][k];  // column k of the block's 32, slice x
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (x == 0 && blockIdx.x * 32 + k < dim && dw) dw[blockIdx.x * 32 + k] = v;
}

// ------------------------------------------------------------------------------------- launch
int launched() { return cudaGetLastError() == cudaSuccess ? HX_OK : HX_ERR_CUDA; }
bool multiple(const void* p, uint64_t of) { return (reinterpret_cast<uintptr_t>(p) % of) == 0; }

// SMs of the current device, 0 on an error; asked for once per device.
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed))) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Values per vector: the widest with which every vector of every head starts on its own boundary.
int vector_of(const Args& a, uint64_t e, bool inter) {
  for (int pu = 8; pu > 1; pu /= 2) {
    const uint64_t al = std::min<uint64_t>(16, pu * e), fl = std::min<uint64_t>(16, pu * 4);
    const bool strides = (a.xt * e) % al == 0 && (a.xh * e) % al == 0 && (a.yt * e) % al == 0 &&
                         (a.yh * e) % al == 0;
    const uint64_t wl = a.w_f32 ? fl : al;
    if (a.dim % (2 * pu) == 0 && a.rot % (inter ? pu : 2 * pu) == 0 && strides && multiple(a.x, al) &&
        multiple(a.y, al) && multiple(a.bytes, pu) && multiple(a.cos, fl) && multiple(a.sin, fl) &&
        multiple(a.wq, wl) && multiple(a.wk, wl))
      return pu;
  }
  return 1;
}

template <void (*kernel)(const Args)>
int launch_ahead(uint64_t smem, const Args& a, uint32_t grid, cudaStream_t s) {
  if (!allow_shared<kernel>((int)smem)) return HX_ERR_CUDA;
  kernel<<<grid, kThreads, smem, s>>>(a);
  return launched();
}

template <typename T, int PU, bool kInter>
int launch(bool backward, const Args& a, uint32_t grid, cudaStream_t s) {
  constexpr uint64_t fwd = 16 * sizeof(T) * kThreads * kAhead, bwd = fwd + 20 * kThreads * kAhead;
  if (backward && a.fmt == HX_ROWS_E4M3) return launch_ahead<k_qk_backward<T, PU, kInter, HX_ROWS_E4M3>>(bwd, a, grid, s);
  if (backward) return launch_ahead<k_qk_backward<T, PU, kInter, HX_ROWS_INT8>>(bwd, a, grid, s);
  if (a.fmt == HX_ROWS_E4M3) return launch_ahead<k_qk_forward<T, PU, kInter, HX_ROWS_E4M3>>(fwd, a, grid, s);
  return launch_ahead<k_qk_forward<T, PU, kInter, HX_ROWS_INT8>>(fwd, a, grid, s);
}
template <typename T, int PU>
int launch_style(bool backward, bool inter, const Args& a, uint32_t grid, cudaStream_t s) {
  return inter ? launch<T, PU, true>(backward, a, grid, s) : launch<T, PU, false>(backward, a, grid, s);
}
template <typename T>
int launch_width(int pu, bool backward, bool inter, const Args& a, uint32_t grid, cudaStream_t s) {
  switch (pu) {
    case 8: return launch_style<T, 8>(backward, inter, a, grid, s);
    case 4: return launch_style<T, 4>(backward, inter, a, grid, s);
    case 2: return launch_style<T, 2>(backward, inter, a, grid, s);
    default: return launch_style<T, 1>(backward, inter, a, grid, s);
  }
}

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

int check(const Args& a, uint32_t dtype, uint32_t w_dtype, uint32_t pos_bits) {
  if (a.fmt > HX_ROWS_INT8 || dtype > HX_BF16 || (w_dtype != HX_F32 && w_dtype != dtype) ||
      (pos_bits != 32 && pos_bits != 64))
    return HX_ERR_ARG;
  if (a.dim < 2 || a.dim > kMaxDim || a.dim % 2 || a.rot > a.dim || a.rot % 2) return HX_ERR_ARG;
  const uint64_t heads = (uint64_t)a.nq + a.nk;
  if (!heads || heads > (1u << 20) || a.tokens >= (1ull << 31) || !(a.eps >= 0.0f) ||
      a.places >= (1ull << 40))
    return HX_ERR_ARG;
  if (a.tokens && a.tokens * heads > (1ull << 40) / a.dim) return HX_ERR_ARG;
  if (a.tokens && ((a.nq && !a.wq) || (a.nk && !a.wk))) return HX_ERR_ARG;
  if (a.tokens && (!a.x || !a.y || !a.pos || !a.places || (a.rot && (!a.cos || !a.sin)))) return HX_ERR_ARG;
  const uint64_t e = dtype == HX_F32 ? 4 : 2, we = w_dtype == HX_F32 ? 4 : 2;
  if (!multiple(a.x, e) || !multiple(a.y, e) || !multiple(a.wq, we) || !multiple(a.wk, we) ||
      !multiple(a.cos, 4) || !multiple(a.sin, 4) || !multiple(a.scale, 4) ||
      !multiple(a.pos, pos_bits / 8) || !multiple(a.status, 4))
    return HX_ERR_ARG;
  return HX_OK;
}

// The lanes per head: a power of two with 16 values each. Heads per item: 8, so that a token's
// angles and the weight are loaded once for them, halved while the items would not fill the GPU.
void arrange(Args* a, int sms) {
  uint32_t lanes = 1;
  while (lanes * 16 < a->dim) lanes *= 2;
  a->lanes = lanes;
  a->per = 8;
  const uint64_t want = (uint64_t)sms * (1024 / lanes);
  while (a->per > 1 && a->tokens * (ceil_div(a->nq, a->per) + ceil_div(a->nk, a->per)) < want)
    a->per /= 2;
}

int run(bool backward, uint32_t dtype, int pu, uint32_t style, const Args& a, uint64_t grid,
        cudaStream_t s) {
  if (grid >= (1ull << 31)) return HX_ERR_ARG;
  if (dtype == HX_F32) return launch_width<float>(pu, backward, style, a, (uint32_t)grid, s);
  if (dtype == HX_F16) return launch_width<__half>(pu, backward, style, a, (uint32_t)grid, s);
  return launch_width<__nv_bfloat16>(pu, backward, style, a, (uint32_t)grid, s);
}

}  // namespace

extern "C" {

int hx_head_norm_rope_forward(const hx_head_norm_rope* p, const void* d_x, uint64_t x_token,
                              uint64_t x_head, void* d_y, uint64_t y_token, uint64_t y_head,
                              uint8_t* d_bytes, float* d_scale, uint32_t* d_status, void* stream) {
  if (!p || !d_bytes != !d_scale) return HX_ERR_ARG;
  Args a{};
  a.fmt = p->format, a.w_f32 = p->weight_dtype == HX_F32;
  a.x = d_x, a.xt = x_token, a.xh = x_head, a.y = d_y, a.yt = y_token, a.yh = y_head;
  a.bytes = d_bytes, a.scale = d_scale, a.tokens = p->tokens;
  a.nq = p->q_heads, a.nk = p->k_heads, a.dim = p->dim, a.rot = p->rot_dim;
  a.wq = p->d_wq, a.wk = p->d_wk, a.cos = p->d_cos, a.sin = p->d_sin;
  a.pos = p->d_positions, a.pos64 = p->position_bits == 64, a.places = p->places;
  a.eps = p->eps, a.status = d_status;
  if (const int rc = check(a, p->dtype, p->weight_dtype, p->position_bits)) return rc;
  if (!a.tokens) return HX_OK;
  const int sms = sm_count();
  if (!sms) return HX_ERR_CUDA;
  const int pu = vector_of(a, p->dtype == HX_F32 ? 4 : 2, p->interleaved != 0);
  arrange(&a, sms);
  const uint64_t items = a.tokens * (ceil_div(a.nq, a.per) + ceil_div(a.nk, a.per));
  return run(false, p->dtype, pu, p->interleaved != 0, a, ceil_div(items, kThreads / a.lanes),
             static_cast<cudaStream_t>(stream));
}

uint64_t hx_head_norm_rope_workspace(uint32_t dim) { return (uint64_t)kMaxBlocks * dim * 4; }

int hx_head_norm_rope_backward(const hx_head_norm_rope* p, const void* d_dy, uint64_t dy_token,
                               uint64_t dy_head, const uint8_t* d_bytes, const float* d_scale,
                               void* d_dx, uint64_t dx_token, uint64_t dx_head, float* d_dwq,
                               float* d_dwk, void* d_workspace, uint64_t workspace_bytes,
                               uint32_t* d_status, void* stream) {
  if (!p) return HX_ERR_ARG;
  Args a{};
  a.fmt = p->format, a.w_f32 = p->weight_dtype == HX_F32;
  a.x = d_dy, a.xt = dy_token, a.xh = dy_head, a.y = d_dx, a.yt = dx_token, a.yh = dx_head;
  a.bytes = const_cast<uint8_t*>(d_bytes), a.scale = const_cast<float*>(d_scale);
  a.tokens = p->tokens;
  a.nq = p->q_heads, a.nk = p->k_heads, a.dim = p->dim, a.rot = p->rot_dim;
  a.wq = p->d_wq, a.wk = p->d_wk, a.cos = p->d_cos, a.sin = p->d_sin;
  a.pos = p->d_positions, a.pos64 = p->position_bits == 64, a.places = p->places;
  a.eps = p->eps, a.status = d_status;
  if (const int rc = check(a, p->dtype, p->weight_dtype, p->position_bits)) return rc;
  if ((a.nq && !d_dwq) || (a.nk && !d_dwk) || !multiple(d_dwq, 4) || !multiple(d_dwk, 4)) return HX_ERR_ARG;
  if (!d_workspace || !multiple(d_workspace, 4) ||
      workspace_bytes < hx_head_norm_rope_workspace(a.dim))
    return HX_ERR_ARG;
  if (a.tokens && (!d_bytes || !d_scale)) return HX_ERR_ARG;
  const int sms = sm_count();
  if (!sms) return HX_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.part = static_cast<float*>(d_workspace);
  uint64_t blocks = 0;
  if (a.tokens) {
    const int pu = vector_of(a, p->dtype == HX_F32 ? 4 : 2, p->interleaved != 0);
    arrange(&a, sms);
    // two blocks per SM hold all groups that fit at once; queries and keys share them by heads
    const uint64_t groups = kThreads / a.lanes;
    const uint64_t bq = ceil_div(a.tokens * ceil_div(a.nq, a.per), groups);
    const uint64_t bk = ceil_div(a.tokens * ceil_div(a.nk, a.per), groups);
    const uint64_t most = std::min<uint64_t>(kMaxBlocks, 2 * (uint64_t)sms);
    uint64_t q = bq, k = bk;
    if (bq + bk > most) {
      q = bq ? std::max<uint64_t>(1, most * bq / (bq + bk)) : 0;
      if (bk && q == most) --q;
      k = bk ? most - q : 0;
    }
    a.blocks_q = (uint32_t)q;
    a.dwq = d_dwq, a.dwk = d_dwk;
    blocks = q + k;
    if (const int rc = run(true, p->dtype, pu, p->interleaved != 0, a, blocks, s)) return rc;
    // a class with one block has its sums; one without heads has none to write
    if (q <= 1 && k <= 1 && (q || !d_dwq) && (k || !d_dwk)) return HX_OK;
  }
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((a.dim + 31) / 32, 2);
  c.blockDim = dim3(1024);
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at, c.numAttrs = a.tokens ? 1 : 0;
  if (cudaLaunchKernelEx(&c, k_qk_weights, static_cast<const float*>(a.part), a.dim, a.blocks_q, (uint32_t)blocks, d_dwq,
                         d_dwk) != cudaSuccess) {
    cudaGetLastError();
    return HX_ERR_CUDA;
  }
  return HX_OK;
}

}  // extern "C"
