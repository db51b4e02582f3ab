// 8-bit rows (sm_100a): a matrix kept as one byte per value and one 32-bit scale per row, the form
// in which a training step keeps its activations for the backward pass and in which the coder
// codes them. The kernels here make the rows (from a matrix, or inside the gated activation) and
// read them back (as values, or inside the gated activation's backward pass).
//
// All are bound by memory: every input is read once and every output written once. A value's unit is W neighbours of a
// row: 8 (16-bit types) or 4 where every row starts on their boundary, else 4, 2 or 1.
//
//   k_quantize     a row's largest magnitude decides its scale, so the row is held in registers
//                  between the two: R units per thread, 1 to 32 lanes per row, one block per row up
//                  to 512 threads, and a second read (from L2) of rows longer than that.
//   k_gated_save   the same over a row's gate half and up half, with silu(gate) * up on the way.
//   k_gated, k_gated_backward, k_dequantize
//                  the scales are known (or not needed): U units per thread of a group of 1 to 32 lanes, the loads
//                  of all before the first is used.
//
// Measured on B200, 8192 x 8192 values (floor: the bytes at the measured copy rate, 6550 GB/s): f32 to INT8 52 us (51),
// bf16 to INT8 33 (31), e4m3 to bf16 33 (31), gated bf16 saved as e4m3 82 (82), its backward pass with h 101 (102). Rows in units of one value
// (odd widths) take 1.6 to 2.5 times the wide ones' time, in units of two 1.2 to 1.5 times.
#include <algorithm>
#include <cstdint>

#include "hx.h"
#include "hx_values.h"

namespace {

using namespace hxv;

// --------------------------------------------------------------------------------- reductions
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  __shared__ uint32_t part[32];
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  const uint32_t nw = blockDim.x >> 5;
  m = (threadIdx.x & 31) < nw ? part[threadIdx.x & 31] : 0;
  return __reduce_max_sync(0xffffffffu, m);
}

// The largest over the lanes of a row: a block's, or `n` (a power of two up to 32) neighbouring lanes'.
template <bool kBlock>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t n) {
  if (kBlock) return block_max(m);
  if (n == 32) return __reduce_max_sync(0xffffffffu, m);
  for (uint32_t o = n >> 1; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// ----------------------------------------------------------------------------------- quantise
template <typename T, int W, int R, bool kBlock, bool kLong, uint32_t fmt>
__global__ void __launch_bounds__(512)
    k_quantize(const T* __restrict__ x, uint64_t rows, uint32_t cols, uint64_t ld,
               uint8_t* __restrict__ bytes, float* __restrict__ scale, uint32_t lanes) {
  const uint32_t n = kBlock ? blockDim.x : lanes;
  const uint32_t lane = kBlock ? threadIdx.x : threadIdx.x & (n - 1);
  const uint64_t row = kBlock ? blockIdx.x : (blockIdx.x * (uint64_t)blockDim.x + threadIdx.x) >> (31 - __clz(n));
  const uint32_t units = row < rows ? cols / W : 0;  // a warp's last rows may not exist
  const T* xr = x + row * ld;
  uint8_t* br = bytes + row * cols;
  Vec<T, W> v[R];
  uint32_t m = 0;
  for (uint32_t base = 0; base < (kLong ? units : 1u); base += R * n) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t u = base + r * n + lane;
      if (u < units)
        v[r].load(xr + (uint64_t)u * W);
      else
        v[r].zero();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) m = v[r].top(m);
  }
  m = row_max<kBlock>(top_bits<T>(m), n);
  if (!kLong) {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r].pin();
  }
  const Scale sc = scale_of<T>(fmt, m);
  if (lane == 0 && units) scale[row] = sc.s;
  for (uint32_t base = 0; base < (kLong ? units : 1u); base += R * n) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t u = base + r * n + lane;
      if (u >= units) continue;
      if (kLong) v[r].load(xr + (uint64_t)u * W);
      float f[W];
      v[r].floats(f);
      to_bytes<T, W, false>(fmt, f, sc).store(br + (uint64_t)u * W);
    }
  }
  if (fmt == HX_ROWS_INT8 && huge<T>(sc)) huge_row<T, W>(xr, br, units, lane, n, sc);
}

// ----------------------------------------------------------------------------- gated forward
// silu(g) = g p with p = sigmoid(g) = 1 / (1 + e^-g), and 1 - p = sigmoid(-g). Both from e = e^-|g|: 1 / (1 + e) and
// e / (1 + e), so that the quotient is one by 1 to 2 (of e^-g itself it would be by numbers that pass 2^126 from g = -87.3 on,
// where the fast one is 0), and p is exactly 1 for large g, where a product g u of 16-bit values can lie at a half.
// The quotient is the fast one (1 unit of the last place). For f32 e is expf (2 units). For 16-bit types it is the fast 2^x, for bf16
// its square at half the exponent: 4 units and 0.75 |g| more (the exponent's rounding), 2^-16 of the result at most. The fast
// 2^x is 0 below 2^-126, which half the exponent reaches at g = -174; the one that is not costs two operations more (bf16
// 8192 x 8192, sustained: 84.5 us, not 82.9). With f16, whose values end at 65504, nothing is left of p below 2^-126.
struct Sigmoid {
  float p, rest;
};
template <typename T>
__device__ __forceinline__ Sigmoid sigmoid(float g) {
  float e, sum, r;
  if constexpr (sizeof(T) == 4) {
    e = expf(-fabsf(g)), sum = 1.0f + e;
  } else if constexpr (!Type<T>::kWide) {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(g) * -1.44269504f));  // 1 / ln 2
    sum = 1.0f + e;
  } else {
    float half;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(half) : "f"(fabsf(g) * -0.72134752f));  // 1 / (2 ln 2)
    e = half * half, sum = fmaf(half, half, 1.0f);
  }
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sum));
  const float t = e * r;
  return g >= 0.0f ? Sigmoid{r, t} : Sigmoid{t, r};
}

template <typename T, int W>
__device__ __forceinline__ void gate(const float (&g)[W], const float (&u)[W], float (&h)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) h[i] = g[i] * sigmoid<T>(g[i]).p * u[i];
}

// At most 64 registers, for two blocks per SM: the compiler's 100 for bf16 and INT8 made 33554 x 1000 values 53 us, not 45,
// its 70 for f32 and INT8 8192 x 8192 values 209 us, not 151.
template <typename T, int W, int R, bool kBlock, bool kLong, uint32_t fmt>
__global__ void __launch_bounds__(512, 2)
    k_gated_save(const T* __restrict__ x, uint64_t rows, uint32_t cols, uint64_t ld,
                 T* __restrict__ out, uint8_t* __restrict__ bytes, float* __restrict__ scale, uint32_t lanes) {
  const uint32_t n = kBlock ? blockDim.x : lanes;
  const uint32_t lane = kBlock ? threadIdx.x : threadIdx.x & (n - 1);
  const uint64_t row = kBlock ? blockIdx.x : (blockIdx.x * (uint64_t)blockDim.x + threadIdx.x) >> (31 - __clz(n));
  const uint32_t units = row < rows ? cols / W : 0;
  const T *gr = x + row * ld, *ur = gr + cols;
  uint8_t *bg = bytes + 2 * row * cols, *bu = bg + cols;
  T* hr = out + row * cols;
  Vec<T, W> g[R], u[R];
  uint32_t mg = 0, mu = 0;
  for (uint32_t base = 0; base < (kLong ? units : 1u); base += R * n) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t i = base + r * n + lane;
      if (i < units) {
        g[r].load(gr + (uint64_t)i * W);
        u[r].load(ur + (uint64_t)i * W);
      } else {
        g[r].zero();
        u[r].zero();
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) mg = g[r].top(mg), mu = u[r].top(mu);
  }
  mg = row_max<kBlock>(top_bits<T>(mg), n);
  if (kBlock) __syncthreads();
  mu = row_max<kBlock>(top_bits<T>(mu), n);
  if (!kLong) {
#pragma unroll
    for (int r = 0; r < R; ++r) g[r].pin(), u[r].pin();
  }
  const Scale sg = scale_of<T>(fmt, mg), su = scale_of<T>(fmt, mu);
  if (lane == 0 && units) scale[2 * row] = sg.s, scale[2 * row + 1] = su.s;
  for (uint32_t base = 0; base < (kLong ? units : 1u); base += R * n) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t i = base + r * n + lane;
      if (i >= units) continue;
      if (kLong) {
        g[r].load(gr + (uint64_t)i * W);
        u[r].load(ur + (uint64_t)i * W);
      }
      float fg[W], fu[W], h[W];
      g[r].floats(fg);
      u[r].floats(fu);
      gate<T>(fg, fu, h);
      store<T, W>(hr + (uint64_t)i * W, h);
      to_bytes<T, W, false>(fmt, fg, sg).store(bg + (uint64_t)i * W);
      to_bytes<T, W, false>(fmt, fu, su).store(bu + (uint64_t)i * W);
    }
  }
  if (fmt == HX_ROWS_INT8) {
    if (huge<T>(sg)) huge_row<T, W>(gr, bg, units, lane, n, sg);
    if (huge<T>(su)) huge_row<T, W>(ur, bu, units, lane, n, su);
  }
}

// ------------------------------------------------------------------- kernels without rows
constexpr int kFlatThreads = 256;

// A thread's U units of a row: first, first + n, ... `n` lanes (a power of two) share a task of n * U units, `per_row` tasks a row.
struct Task {
  uint64_t row;
  uint32_t first, units;  // of the row; 0 where there is no such row
};
struct Tasks {
  uint64_t rows;
  uint32_t cols, n, shift, per_row;  // n = 1 << shift
};
template <int W, int U>
__device__ __forceinline__ Task task_of(const Tasks& t) {
  const uint64_t id = (blockIdx.x * (uint64_t)kFlatThreads + threadIdx.x) >> t.shift;
  Task k;
  k.row = id >> 32 ? id / t.per_row : (uint32_t)id / t.per_row;
  k.first = (uint32_t)(id - k.row * t.per_row) * (t.n * U) + (threadIdx.x & (t.n - 1));
  k.units = k.row < t.rows ? t.cols / W : 0;
  return k;
}

template <typename T, int W, int U>
__global__ void __launch_bounds__(kFlatThreads)
    k_gated(const T* __restrict__ x, const Tasks t, uint64_t ld, T* __restrict__ out) {
  const Task k = task_of<W, U>(t);
  const T* gr = x + k.row * ld;
  Vec<T, W> g[U], u[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t v = k.first + i * t.n;
    if (v < k.units) {
      g[i].load(gr + (uint64_t)v * W);
      u[i].load(gr + t.cols + (uint64_t)v * W);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t v = k.first + i * t.n;
    if (v >= k.units) return;
    float fg[W], fu[W], h[W];
    g[i].floats(fg);
    u[i].floats(fu);
    gate<T>(fg, fu, h);
    store<T, W>(out + k.row * t.cols + (uint64_t)v * W, h);
  }
}

// With four loads on their way per thread (8192 x 8192 to bf16: 41.0 us with one, 34.9 with two, 33.1 with four; 201 MB
// at the measured copy rate are 30.7).
template <typename T, int W, int U>
__global__ void __launch_bounds__(kFlatThreads)
    k_dequantize(uint32_t fmt, const uint8_t* __restrict__ bytes, const float* __restrict__ scale, const Tasks t,
                 T* __restrict__ out, uint64_t ld) {
  const Task k = task_of<W, U>(t);
  if (k.first >= k.units) return;
  const uint8_t* br = bytes + k.row * t.cols;
  T* o = out + k.row * ld;
  Bytes<W> b[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t v = k.first + i * t.n;
    if (v < k.units) b[i].load(br + (uint64_t)v * W);
  }
  const float s = scale[k.row];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t v = k.first + i * t.n;
    if (v >= k.units) return;
    float f[W];
    to_values<W>(fmt, b[i], s, f);
    if constexpr (sizeof(T) == 2) {
      if (Type<T>::kInf == Type<__half>::kInf) {
        // a value just below 65504 can round up in its byte: stay finite. (min and max would drop a NaN.)
#pragma unroll
        for (int j = 0; j < W; ++j)
          f[j] = f[j] > 65504.0f ? 65504.0f : f[j] < -65504.0f ? -65504.0f : f[j];
      }
    }
    store<T, W>(o + (uint64_t)v * W, f);
  }
}

// h = g p u with p = sigmoid(g): dg = dh u p (1 + g (1 - p)), du = dh g p. 64 registers in units of 8, for four blocks per SM
// (the compiler's 80 made 33554 x 1000 values 44.4 us, not 42.6). Smaller units have none stated (0): with one block per SM
// stated the compiler takes 96, and 33554 x 1001 values 120 us, not 75.
template <typename T, int W, int U>
__global__ void __launch_bounds__(kFlatThreads, W == 8 ? 4 : 0)
    k_gated_backward(uint32_t fmt, const T* __restrict__ dh, uint64_t ld, const uint8_t* __restrict__ bytes,
                     const float* __restrict__ scale, const Tasks t, T* __restrict__ dx, T* __restrict__ h) {
  const Task k = task_of<W, U>(t);
  if (k.first >= k.units) return;
  const T* dr = dh + k.row * ld;
  const uint8_t* br = bytes + 2 * k.row * t.cols;
  Vec<T, W> d[U];
  Bytes<W> bg[U], bu[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t v = k.first + i * t.n;
    if (v < k.units) {
      d[i].load(dr + (uint64_t)v * W);
      bg[i].load(br + (uint64_t)v * W);
      bu[i].load(br + t.cols + (uint64_t)v * W);
    }
  }
  const float sg = scale[2 * k.row], su = scale[2 * k.row + 1];
  T* o = dx + 2 * k.row * t.cols;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t v = k.first + i * t.n;
    if (v >= k.units) return;
    float fd[W], fg[W], fu[W], fh[W];
    d[i].floats(fd);
    to_values<W>(fmt, bg[i], sg, fg);
    to_values<W>(fmt, bu[i], su, fu);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const Sigmoid s = sigmoid<T>(fg[j]);
      const float silu = fg[j] * s.p;
      fh[j] = silu * fu[j];
      // dg into fu, du into fd
      fu[j] *= fd[j] * fmaf(silu, s.rest, s.p);
      fd[j] *= silu;
    }
    store<T, W>(o + (uint64_t)v * W, fu);
    store<T, W>(o + t.cols + (uint64_t)v * W, fd);
    if (h) store<T, W>(h + k.row * t.cols + (uint64_t)v * W, fh);
  }
}

// ------------------------------------------------------------------------------------- launch
int launched() { return cudaGetLastError() == cudaSuccess ? HX_OK : HX_ERR_CUDA; }

bool multiple(const void* p, uint64_t of) { return (reinterpret_cast<uintptr_t>(p) % of) == 0; }

uint64_t size_of(uint32_t dtype) { return dtype == HX_F32 ? 4 : 2; }

// What every call here checks first.
bool bad_shape(uint32_t fmt, uint32_t dtype, uint64_t rows, uint64_t cols) {
  return fmt > HX_ROWS_INT8 || dtype > HX_BF16 || !cols || cols >= (1ull << 30) ||
         rows >= (1ull << 31) || (rows && cols > (1ull << 40) / rows);
}

// The widest unit on whose boundary every row of the operands starts (a unit of a 32-bit type is at most 4 values: 16
// bytes, so that a warp's loads are whole lines).
int unit_of(uint32_t dtype, uint64_t cols, uint64_t ld, const void* a, const void* b, const void* bytes) {
  const uint64_t e = size_of(dtype);
  for (int w = e == 4 ? 4 : 8; w > 1; w /= 2)
    if (cols % w == 0 && ld % w == 0 && multiple(a, w * e) && multiple(b, w * e) && multiple(bytes, w)) return w;
  return 1;
}

uint32_t power_of_two(uint64_t v) {
  uint32_t p = 1;
  while (p < v) p *= 2;
  return p;
}

// The block and grid of a kernel that holds a row: R units per thread, as many lanes per row as that takes.
struct RowLaunch {
  bool block, twice;
  uint32_t threads, lanes;
  uint64_t grid;
};
RowLaunch row_launch(uint64_t rows, uint64_t units, int R) {
  RowLaunch l{};
  l.block = units > 32u * R;
  l.twice = units > 512u * R;
  l.threads = 256;
  if (l.block) {
    const uint64_t per = (units + R - 1) / R;
    l.threads = (uint32_t)std::min<uint64_t>(512, (per + 31) / 32 * 32);
    l.grid = rows;
  } else {
    l.lanes = power_of_two((units + R - 1) / R);
    l.grid = (rows * l.lanes + l.threads - 1) / l.threads;
  }
  return l;
}

template <typename T, int W, int R, uint32_t F>
int quantize_f(const void* x, uint64_t rows, uint64_t cols, uint64_t ld,
               uint8_t* bytes, float* scale, cudaStream_t s) {
  const RowLaunch l = row_launch(rows, cols / W, R);
  if (l.grid >= (1ull << 31)) return HX_ERR_ARG;
  const T* p = static_cast<const T*>(x);
  const uint32_t g = (uint32_t)l.grid, c = (uint32_t)cols;
  if (l.twice)
    k_quantize<T, W, R, true, true, F><<<g, l.threads, 0, s>>>(p, rows, c, ld, bytes, scale, l.lanes);
  else if (l.block)
    k_quantize<T, W, R, true, false, F><<<g, l.threads, 0, s>>>(p, rows, c, ld, bytes, scale, l.lanes);
  else
    k_quantize<T, W, R, false, false, F><<<g, l.threads, 0, s>>>(p, rows, c, ld, bytes, scale, l.lanes);
  return launched();
}

template <typename T, int W, int R, uint32_t F>
int gated_save_f(const void* x, uint64_t rows, uint64_t cols, uint64_t ld, void* out,
                 uint8_t* bytes, float* scale, cudaStream_t s) {
  const RowLaunch l = row_launch(rows, cols / W, R);
  if (l.grid >= (1ull << 31)) return HX_ERR_ARG;
  const T* p = static_cast<const T*>(x);
  T* o = static_cast<T*>(out);
  const uint32_t g = (uint32_t)l.grid, c = (uint32_t)cols;
  if (l.twice)
    k_gated_save<T, W, R, true, true, F><<<g, l.threads, 0, s>>>(p, rows, c, ld, o, bytes, scale, l.lanes);
  else if (l.block)
    k_gated_save<T, W, R, true, false, F><<<g, l.threads, 0, s>>>(p, rows, c, ld, o, bytes, scale, l.lanes);
  else
    k_gated_save<T, W, R, false, false, F><<<g, l.threads, 0, s>>>(p, rows, c, ld, o, bytes, scale, l.lanes);
  return launched();
}

template <typename T, int W, int R, typename... A>
int quantize_w(uint32_t fmt, A... a) {
  return fmt == HX_ROWS_E4M3 ? quantize_f<T, W, R, HX_ROWS_E4M3>(a...) : quantize_f<T, W, R, HX_ROWS_INT8>(a...);
}
template <typename T, int W, int R, typename... A>
int gated_save_w(uint32_t fmt, A... a) {
  return fmt == HX_ROWS_E4M3 ? gated_save_f<T, W, R, HX_ROWS_E4M3>(a...) : gated_save_f<T, W, R, HX_ROWS_INT8>(a...);
}

// The tasks of rows in units of W, U units per thread, and their grid.
Tasks tasks_of(uint64_t rows, uint64_t cols, int W, int U, uint64_t* grid) {
  Tasks t{};
  const uint64_t units = cols / W;
  t.rows = rows, t.cols = (uint32_t)cols;
  t.n = std::min<uint32_t>(32, power_of_two((units + U - 1) / U));
  for (t.shift = 0; (1u << t.shift) < t.n; ++t.shift) {
  }
  t.per_row = (uint32_t)((units + t.n * U - 1) / (t.n * U));
  *grid = (rows * t.per_row * t.n + kFlatThreads - 1) / kFlatThreads;
  return t;
}

// f(T{}) for the element type.
template <typename F>
int by_type(uint32_t dtype, F f) {
  if (dtype == HX_F32) return f(float{});
  if (dtype == HX_F16) return f(__half{});
  return f(__nv_bfloat16{});
}

// f(W, U) as compile-time values for the element type, the unit and the units per thread: 32 bytes' worth (4 of 8 or 4
// values, 8 of fewer) once they still make four blocks per SM, else one, for as many threads as there are units.
template <int N>
struct Count {
  static constexpr int value = N;
};
template <typename T, int W, typename F>
int by_count(uint64_t rows, uint64_t cols, F f) {
  constexpr int kMany = W >= 4 ? 4 : 8;
  uint64_t grid;
  Tasks t = tasks_of(rows, cols, W, kMany, &grid);
  const bool many = grid >= 4 * 148;
  if (!many) t = tasks_of(rows, cols, W, 1, &grid);
  if (grid >= (1ull << 31)) return HX_ERR_ARG;
  return many ? f(Count<W>{}, Count<kMany>{}, t, (uint32_t)grid) : f(Count<W>{}, Count<1>{}, t, (uint32_t)grid);
}
template <typename T, typename F>
int by_unit(int w, uint64_t rows, uint64_t cols, F f) {
  if constexpr (sizeof(T) == 2) {
    if (w == 8) return by_count<T, 8>(rows, cols, f);
  }
  if (w == 4) return by_count<T, 4>(rows, cols, f);
  if (w == 2) return by_count<T, 2>(rows, cols, f);
  return by_count<T, 1>(rows, cols, f);
}

}  // namespace

extern "C" {

int hx_quantize_rows(uint32_t format, uint32_t dtype, const void* d_x, uint64_t rows, uint64_t cols,
                     uint64_t ld, uint8_t* d_bytes, float* d_scale, void* stream) {
  if (bad_shape(format, dtype, rows, cols) || (rows > 1 && ld < cols)) return HX_ERR_ARG;
  if (!rows) return HX_OK;
  if (!d_x || !d_bytes || !d_scale || !multiple(d_x, size_of(dtype)) || !multiple(d_scale, 4))
    return HX_ERR_ARG;
  const int w = unit_of(dtype, cols, rows > 1 ? ld : cols, d_x, nullptr, d_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_type(dtype, [&](auto t) {
    using T = decltype(t);
    if constexpr (sizeof(T) == 2) {
      if (w == 8) return quantize_w<T, 8, 4>(format, d_x, rows, cols, ld, d_bytes, d_scale, s);
    }
    if (w == 4) return quantize_w<T, 4, 8>(format, d_x, rows, cols, ld, d_bytes, d_scale, s);
    if (w == 2) return quantize_w<T, 2, 8>(format, d_x, rows, cols, ld, d_bytes, d_scale, s);
    return quantize_w<T, 1, 16>(format, d_x, rows, cols, ld, d_bytes, d_scale, s);
  });
}

int hx_dequantize_rows(uint32_t format, uint32_t dtype, const uint8_t* d_bytes, const float* d_scale,
                       uint64_t rows, uint64_t cols, void* d_out, uint64_t ld, void* stream) {
  if (bad_shape(format, dtype, rows, cols) || (rows > 1 && ld < cols)) return HX_ERR_ARG;
  if (!rows) return HX_OK;
  if (!d_out || !d_bytes || !d_scale || !multiple(d_out, size_of(dtype)) || !multiple(d_scale, 4))
    return HX_ERR_ARG;
  const int w = unit_of(dtype, cols, rows > 1 ? ld : cols, d_out, nullptr, d_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return by_unit<T>(w, rows, cols, [&](auto W, auto U, const Tasks& k, uint32_t grid) {
      k_dequantize<T, decltype(W)::value, decltype(U)::value>
          <<<grid, kFlatThreads, 0, s>>>(format, d_bytes, d_scale, k, static_cast<T*>(d_out), ld);
      return launched();
    });
  });
}

int hx_gated_forward(uint32_t format, uint32_t dtype, const void* d_x, uint64_t rows, uint64_t cols,
                     uint64_t ld, void* d_out, uint8_t* d_bytes, float* d_scale, void* stream) {
  if (bad_shape(format, dtype, rows, cols) || (rows > 1 && ld < 2 * cols)) return HX_ERR_ARG;
  if (!d_bytes != !d_scale) return HX_ERR_ARG;
  if (!rows) return HX_OK;
  if (!d_x || !d_out || !multiple(d_x, size_of(dtype)) || !multiple(d_out, size_of(dtype)) ||
      !multiple(d_scale, 4))
    return HX_ERR_ARG;
  const int w = unit_of(dtype, cols, rows > 1 ? ld : cols, d_x, d_out, d_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_type(dtype, [&](auto t) {
    using T = decltype(t);
    if (d_bytes) {
      if constexpr (sizeof(T) == 2) {
        if (w == 8) return gated_save_w<T, 8, 4>(format, d_x, rows, cols, ld, d_out, d_bytes, d_scale, s);
      }
      if (w == 4) return gated_save_w<T, 4, 4>(format, d_x, rows, cols, ld, d_out, d_bytes, d_scale, s);
      if (w == 2) return gated_save_w<T, 2, 8>(format, d_x, rows, cols, ld, d_out, d_bytes, d_scale, s);
      return gated_save_w<T, 1, 8>(format, d_x, rows, cols, ld, d_out, d_bytes, d_scale, s);
    }
    return by_unit<T>(w, rows, cols, [&](auto W, auto U, const Tasks& k, uint32_t grid) {
      k_gated<T, decltype(W)::value, decltype(U)::value>
          <<<grid, kFlatThreads, 0, s>>>(static_cast<const T*>(d_x), k, ld, static_cast<T*>(d_out));
      return launched();
    });
  });
}

int hx_gated_backward(uint32_t format, uint32_t dtype, const void* d_dout, uint64_t ld,
                      const uint8_t* d_bytes, const float* d_scale, uint64_t rows, uint64_t cols,
                      void* d_dx, void* d_out, void* stream) {
  if (bad_shape(format, dtype, rows, cols) || (rows > 1 && ld < cols)) return HX_ERR_ARG;
  if (!rows) return HX_OK;
  const uint64_t e = size_of(dtype);
  if (!d_dout || !d_bytes || !d_scale || !d_dx || !multiple(d_dout, e) || !multiple(d_dx, e) ||
      !multiple(d_out, e) || !multiple(d_scale, 4))
    return HX_ERR_ARG;
  int w = unit_of(dtype, cols, rows > 1 ? ld : cols, d_dout, d_dx, d_bytes);
  while (w > 1 && !multiple(d_out, w * e)) w /= 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return by_unit<T>(w, rows, cols, [&](auto W, auto U, const Tasks& k, uint32_t grid) {
      k_gated_backward<T, decltype(W)::value, decltype(U)::value><<<grid, kFlatThreads, 0, s>>>(
          format, static_cast<const T*>(d_dout), ld, d_bytes, d_scale, k, static_cast<T*>(d_dx), static_cast<T*>(d_out));
      return launched();
    });
  });
}

}  // extern "C"
