// 8-bit rows (sm_100a): a matrix kept as one byte per value and one 32-bit scale per row, the form
// in which a training step keeps its activations for the backward pass and in which the coder
// codes them. The kernels here make the rows (from a matrix, or inside the gated activation) and
// read them back (as values, or inside the gated activation's backward pass).
//
// All are bound by memory: every input is read once and every output written once.
//
//   k_quantize     a row's largest magnitude decides its scale, so the row is held in registers
//                  between the two: one warp per row of up to 32 * R units, one block per row up
//                  to 512 * R, and a second read (from L2) of rows longer than that.
//   k_gated_save   the same over a row's gate half and up half, with silu(gate) * up on the way.
//   k_gated, k_gated_backward, k_dequantize
//                  the scales are known (or not needed): one unit per thread, no row structure.
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

// ----------------------------------------------------------------------------------- quantise
template <typename T, int W, int R, bool kBlock, bool kLong>
__global__ void __launch_bounds__(512)
    k_quantize(uint32_t fmt, const T* __restrict__ x, uint64_t rows, uint32_t cols, uint64_t ld,
               uint8_t* __restrict__ bytes, float* __restrict__ scale) {
  const uint32_t lane = kBlock ? threadIdx.x : threadIdx.x & 31;
  const uint32_t n = kBlock ? blockDim.x : 32;
  const uint64_t row =
      kBlock ? blockIdx.x : blockIdx.x * (uint64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= rows) return;  // a whole warp (a whole block has a row)
  const uint32_t units = cols / W;
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
  m = top_bits<T>(m);
  m = kBlock ? block_max(m) : __reduce_max_sync(0xffffffffu, m);
  const Scale sc = scale_of<T>(fmt, m);
  if (lane == 0) scale[row] = sc.s;
  for (uint32_t base = 0; base < (kLong ? units : 1u); base += R * n) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t u = base + r * n + lane;
      if (u >= units) continue;
      if (kLong) v[r].load(xr + (uint64_t)u * W);
      float f[W];
      v[r].floats(f);
      to_bytes<W>(fmt, f, sc).store(br + (uint64_t)u * W);
    }
  }
}

// ----------------------------------------------------------------------------- gated forward
// silu(g) = g / (1 + e^-g). The exponential and the quotient are the fast ones (2 ulp each), far below
// the output's own rounding for 16-bit types and at 32 bits' own noise for 32.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

template <int W>
__device__ __forceinline__ void gate(const float (&g)[W], const float (&u)[W], float (&h)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) h[i] = g[i] * sigmoid(g[i]) * u[i];
}

template <typename T, int W, int R, bool kBlock, bool kLong>
__global__ void __launch_bounds__(512)
    k_gated_save(uint32_t fmt, const T* __restrict__ x, uint64_t rows, uint32_t cols, uint64_t ld,
                 T* __restrict__ out, uint8_t* __restrict__ bytes, float* __restrict__ scale) {
  const uint32_t lane = kBlock ? threadIdx.x : threadIdx.x & 31;
  const uint32_t n = kBlock ? blockDim.x : 32;
  const uint64_t row =
      kBlock ? blockIdx.x : blockIdx.x * (uint64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= rows) return;
  const uint32_t units = cols / W;
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
  mg = top_bits<T>(mg), mu = top_bits<T>(mu);
  if (kBlock) {
    mg = block_max(mg);
    __syncthreads();
    mu = block_max(mu);
  } else {
    mg = __reduce_max_sync(0xffffffffu, mg);
    mu = __reduce_max_sync(0xffffffffu, mu);
  }
  const Scale sg = scale_of<T>(fmt, mg), su = scale_of<T>(fmt, mu);
  if (lane == 0) scale[2 * row] = sg.s, scale[2 * row + 1] = su.s;
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
      gate(fg, fu, h);
      store<T, W>(hr + (uint64_t)i * W, h);
      to_bytes<W>(fmt, fg, sg).store(bg + (uint64_t)i * W);
      to_bytes<W>(fmt, fu, su).store(bu + (uint64_t)i * W);
    }
  }
}

// ------------------------------------------------------------------- kernels without rows
// Unit i of the whole matrix as (row, first column); 32-bit division where the count allows.
struct Place {
  uint64_t row;
  uint32_t col;
};
template <int W>
__device__ __forceinline__ Place place_of(uint64_t i, uint32_t units) {
  Place p;
  if (i >> 32)
    p.row = i / units;
  else
    p.row = (uint32_t)i / units;
  p.col = (uint32_t)(i - p.row * units) * W;
  return p;
}

constexpr int kFlatThreads = 256;

template <typename T, int W>
__global__ void __launch_bounds__(kFlatThreads)
    k_gated(const T* __restrict__ x, uint64_t n, uint32_t cols, uint64_t ld, T* __restrict__ out) {
  const uint64_t i = blockIdx.x * (uint64_t)kFlatThreads + threadIdx.x;
  if (i >= n) return;
  const Place p = place_of<W>(i, cols / W);
  Vec<T, W> g, u;
  const T* gr = x + p.row * ld + p.col;
  g.load(gr);
  u.load(gr + cols);
  float fg[W], fu[W], h[W];
  g.floats(fg);
  u.floats(fu);
  gate(fg, fu, h);
  store<T, W>(out + p.row * cols + p.col, h);
}

// U units per thread, a block's width apart: four loads of 8 bytes on their way per thread keep the memory busy
// (8192 x 8192 to bf16: 41.0 us with one, 34.9 with two, 33.3 with four; 201 MB at the measured copy rate are 30.7).
template <typename T, int W, int U>
__global__ void __launch_bounds__(kFlatThreads)
    k_dequantize(uint32_t fmt, const uint8_t* __restrict__ bytes, const float* __restrict__ scale,
                 uint64_t n, uint32_t cols, T* __restrict__ out, uint64_t ld) {
  const uint64_t i0 = blockIdx.x * (uint64_t)(U * kFlatThreads) + threadIdx.x;
  Bytes<W> b[U];
  float s[U];
  Place p[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint64_t i = i0 + k * kFlatThreads;
    if (i < n) {
      p[k] = place_of<W>(i, cols / W);
      b[k].load(bytes + p[k].row * cols + p[k].col);
      s[k] = scale[p[k].row];
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (i0 + k * kFlatThreads >= n) return;
    float f[W];
    to_values<W>(fmt, b[k], s[k], f);
    if constexpr (sizeof(T) == 2) {
      if (Type<T>::kInf == Type<__half>::kInf) {
        // a value just below 65504 can round up in its byte: stay finite. (min and max would drop a NaN.)
#pragma unroll
        for (int j = 0; j < W; ++j)
          f[j] = f[j] > 65504.0f ? 65504.0f : f[j] < -65504.0f ? -65504.0f : f[j];
      }
    }
    store<T, W>(out + p[k].row * ld + p[k].col, f);
  }
}

// h = g p u with p = sigmoid(g): dg = dh u p (1 + g (1 - p)), du = dh g p.
template <typename T, int W>
__global__ void __launch_bounds__(kFlatThreads)
    k_gated_backward(uint32_t fmt, const T* __restrict__ dh, uint64_t ld,
                     const uint8_t* __restrict__ bytes, const float* __restrict__ scale, uint64_t n,
                     uint32_t cols, T* __restrict__ dx, T* __restrict__ h) {
  const uint64_t i = blockIdx.x * (uint64_t)kFlatThreads + threadIdx.x;
  if (i >= n) return;
  const Place p = place_of<W>(i, cols / W);
  Vec<T, W> d;
  Bytes<W> bg, bu;
  d.load(dh + p.row * ld + p.col);
  bg.load(bytes + 2 * p.row * cols + p.col);
  bu.load(bytes + (2 * p.row + 1) * cols + p.col);
  const float sg = scale[2 * p.row], su = scale[2 * p.row + 1];
  float fd[W], fg[W], fu[W], fh[W];
  d.floats(fd);
  to_values<W>(fmt, bg, sg, fg);
  to_values<W>(fmt, bu, su, fu);
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const float s = sigmoid(fg[j]), silu = fg[j] * s;
    fh[j] = silu * fu[j];
    // dg into fu, du into fd
    fu[j] *= fd[j] * fmaf(silu, 1.0f - s, s);
    fd[j] *= silu;
  }
  T* o = dx + 2 * p.row * cols + p.col;
  store<T, W>(o, fu);
  store<T, W>(o + cols, fd);
  if (h) store<T, W>(h + p.row * cols + p.col, fh);
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

// Units of 8 values where every row starts on their boundary, else of one.
bool wide(uint32_t dtype, uint64_t cols, uint64_t ld, const void* a, const void* b,
          const void* bytes) {
  const uint64_t e = size_of(dtype), step = 16 / e;
  return cols % 8 == 0 && ld % step == 0 && multiple(a, 16) && multiple(b, 16) &&
         multiple(bytes, 8);
}

// The block and grid of a kernel with a row per warp or block, R units of a row per thread.
struct RowLaunch {
  bool block, twice;
  uint32_t threads, grid;
};
RowLaunch row_launch(uint64_t rows, uint64_t units, int R) {
  RowLaunch l{};
  l.block = units > 32u * R;
  l.twice = units > 512u * R;
  l.threads = 256;
  l.grid = (uint32_t)((rows + 7) / 8);
  if (l.block) {
    const uint64_t per = (units + R - 1) / R;
    l.threads = (uint32_t)std::min<uint64_t>(512, (per + 31) / 32 * 32);
    l.grid = (uint32_t)rows;
  }
  return l;
}

template <typename T, int W, int R>
int quantize_w(uint32_t fmt, const void* x, uint64_t rows, uint64_t cols, uint64_t ld,
               uint8_t* bytes, float* scale, cudaStream_t s) {
  const RowLaunch l = row_launch(rows, cols / W, R);
  const T* p = static_cast<const T*>(x);
  if (l.twice)
    k_quantize<T, W, R, true, true><<<l.grid, l.threads, 0, s>>>(fmt, p, rows, (uint32_t)cols, ld, bytes, scale);
  else if (l.block)
    k_quantize<T, W, R, true, false><<<l.grid, l.threads, 0, s>>>(fmt, p, rows, (uint32_t)cols, ld, bytes, scale);
  else
    k_quantize<T, W, R, false, false><<<l.grid, l.threads, 0, s>>>(fmt, p, rows, (uint32_t)cols, ld, bytes, scale);
  return launched();
}

template <typename T, int W, int R>
int gated_save_w(uint32_t fmt, const void* x, uint64_t rows, uint64_t cols, uint64_t ld, void* out,
                 uint8_t* bytes, float* scale, cudaStream_t s) {
  const RowLaunch l = row_launch(rows, cols / W, R);
  const T* p = static_cast<const T*>(x);
  T* o = static_cast<T*>(out);
  if (l.twice)
    k_gated_save<T, W, R, true, true><<<l.grid, l.threads, 0, s>>>(fmt, p, rows, (uint32_t)cols, ld, o, bytes, scale);
  else if (l.block)
    k_gated_save<T, W, R, true, false><<<l.grid, l.threads, 0, s>>>(fmt, p, rows, (uint32_t)cols, ld, o, bytes, scale);
  else
    k_gated_save<T, W, R, false, false><<<l.grid, l.threads, 0, s>>>(fmt, p, rows, (uint32_t)cols, ld, o, bytes, scale);
  return launched();
}

uint64_t flat_grid(uint64_t units) { return (units + kFlatThreads - 1) / kFlatThreads; }

// f(T{}) for the element type.
template <typename F>
int by_type(uint32_t dtype, F f) {
  if (dtype == HX_F32) return f(float{});
  if (dtype == HX_F16) return f(__half{});
  return f(__nv_bfloat16{});
}

}  // namespace

extern "C" {

int hx_quantize_rows(uint32_t format, uint32_t dtype, const void* d_x, uint64_t rows, uint64_t cols,
                     uint64_t ld, uint8_t* d_bytes, float* d_scale, void* stream) {
  if (bad_shape(format, dtype, rows, cols) || (rows > 1 && ld < cols)) return HX_ERR_ARG;
  if (!rows) return HX_OK;
  if (!d_x || !d_bytes || !d_scale || !multiple(d_x, size_of(dtype)) || !multiple(d_scale, 4))
    return HX_ERR_ARG;
  const bool w = wide(dtype, cols, rows > 1 ? ld : cols, d_x, nullptr, d_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return w ? quantize_w<T, 8, 4>(format, d_x, rows, cols, ld, d_bytes, d_scale, s)
             : quantize_w<T, 1, 8>(format, d_x, rows, cols, ld, d_bytes, d_scale, s);
  });
}

int hx_dequantize_rows(uint32_t format, uint32_t dtype, const uint8_t* d_bytes, const float* d_scale,
                       uint64_t rows, uint64_t cols, void* d_out, uint64_t ld, void* stream) {
  if (bad_shape(format, dtype, rows, cols) || (rows > 1 && ld < cols)) return HX_ERR_ARG;
  if (!rows) return HX_OK;
  if (!d_out || !d_bytes || !d_scale || !multiple(d_out, size_of(dtype)) || !multiple(d_scale, 4))
    return HX_ERR_ARG;
  const bool w = wide(dtype, cols, rows > 1 ? ld : cols, d_out, nullptr, d_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_type(dtype, [&](auto t) {
    using T = decltype(t);
    const uint64_t n = rows * (w ? cols / 8 : cols);
    if (flat_grid(n) >= (1ull << 31)) return (int)HX_ERR_ARG;
    T* o = static_cast<T*>(d_out);
    const uint32_t grid = (uint32_t)flat_grid(n), many = (grid + 3) / 4;
    // four units per thread once that still makes four blocks per SM, as many as a small input can have else
    if (w && many >= 4 * 148)
      k_dequantize<T, 8, 4><<<many, kFlatThreads, 0, s>>>(format, d_bytes, d_scale, n, (uint32_t)cols, o, ld);
    else if (w)
      k_dequantize<T, 8, 1><<<grid, kFlatThreads, 0, s>>>(format, d_bytes, d_scale, n, (uint32_t)cols, o, ld);
    else if (many >= 4 * 148)
      k_dequantize<T, 1, 4><<<many, kFlatThreads, 0, s>>>(format, d_bytes, d_scale, n, (uint32_t)cols, o, ld);
    else
      k_dequantize<T, 1, 1><<<grid, kFlatThreads, 0, s>>>(format, d_bytes, d_scale, n, (uint32_t)cols, o, ld);
    return launched();
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
  const bool w = wide(dtype, cols, rows > 1 ? ld : cols, d_x, d_out, d_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_type(dtype, [&](auto t) {
    using T = decltype(t);
    if (d_bytes)
      return w ? gated_save_w<T, 8, 4>(format, d_x, rows, cols, ld, d_out, d_bytes, d_scale, s)
               : gated_save_w<T, 1, 8>(format, d_x, rows, cols, ld, d_out, d_bytes, d_scale, s);
    const uint64_t n = rows * (w ? cols / 8 : cols);
    if (flat_grid(n) >= (1ull << 31)) return (int)HX_ERR_ARG;
    const T* x = static_cast<const T*>(d_x);
    T* o = static_cast<T*>(d_out);
    if (w)
      k_gated<T, 8><<<(uint32_t)flat_grid(n), kFlatThreads, 0, s>>>(x, n, (uint32_t)cols, ld, o);
    else
      k_gated<T, 1><<<(uint32_t)flat_grid(n), kFlatThreads, 0, s>>>(x, n, (uint32_t)cols, ld, o);
    return launched();
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
  const bool w = wide(dtype, cols, rows > 1 ? ld : cols, d_dout, d_dx, d_bytes) && multiple(d_out, 16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_type(dtype, [&](auto t) {
    using T = decltype(t);
    const uint64_t n = rows * (w ? cols / 8 : cols);
    if (flat_grid(n) >= (1ull << 31)) return (int)HX_ERR_ARG;
    const T* d = static_cast<const T*>(d_dout);
    T *dx = static_cast<T*>(d_dx), *h = static_cast<T*>(d_out);
    if (w)
      k_gated_backward<T, 8><<<(uint32_t)flat_grid(n), kFlatThreads, 0, s>>>(format, d, ld, d_bytes, d_scale, n, (uint32_t)cols, dx, h);
    else
      k_gated_backward<T, 1><<<(uint32_t)flat_grid(n), kFlatThreads, 0, s>>>(format, d, ld, d_bytes, d_scale, n, (uint32_t)cols, dx, h);
    return launched();
  });
}

}  // extern "C"
