// Row quantisation to 8-bit integers (see quant.cuh for the rule).
//
//   quantize_rows_kernel    x [n, c] BF16 or FP32 -> q [n, c] int8, scale [n]
//   quantize_hidden_kernel  the SwiGLU outputs of the 8-bit up projection, FP32
//                           with each row's largest magnitude already known
//
// Both are bound by memory: one read of the row, one write of a byte per
// element.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace moe {

constexpr int kQuantThreads = 256;

// Rows of more than 16384 BF16 or 8192 FP32 values: one block per row.  A thread keeps up to kQuantKeep
// 16-element pieces of its row in registers between the maximum and the rounding;
// the rest is read again (from L2).
constexpr int kQuantKeep = 2;

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]);
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[16]) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  const uint4 a = q[0], b = q[1];
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&v)[16]) {
  const float4* q = reinterpret_cast<const float4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = q[i];
    v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
  }
}

__device__ __forceinline__ uint4 quant_pack16(const float (&v)[16], float scale, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f[4] = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    w[i] = quant_pack4(f, scale, inv);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ unsigned block_max_u32(unsigned v, unsigned* s_max) {
  v = warp_max_u32(v);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = v;
  __syncthreads();
  unsigned m = 0;
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) m = max(m, s_max[w]);
  __syncthreads();
  return m;
}

template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const T* __restrict__ x, int64_t n_rows,
                                                                      int n_cols, int8_t* __restrict__ q,
                                                                      float* __restrict__ scale) {
  __shared__ unsigned s_max[kQuantThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int pieces = n_cols / 16;
  for (int64_t row = blockIdx.x; row < n_rows; row += gridDim.x) {
    const T* xr = x + row * n_cols;
    int8_t* qr = q + row * n_cols;
    float v[kQuantKeep][16];
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < kQuantKeep; ++i) {
      const int p = threadIdx.x + i * kQuantThreads;
      if (p < pieces) {
        load16(xr + p * 16, v[i]);
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, abs_bits(v[i][j]));
      }
    }
    for (int p = threadIdx.x + kQuantKeep * kQuantThreads; p < pieces; p += kQuantThreads) {
      float t[16];
      load16(xr + p * 16, t);
#pragma unroll
      for (int j = 0; j < 16; ++j) m = max(m, abs_bits(t[j]));
    }
    const float s = quant_scale(block_max_u32(m, s_max));
    const float inv = 1.0f / s;
#pragma unroll
    for (int i = 0; i < kQuantKeep; ++i) {
      const int p = threadIdx.x + i * kQuantThreads;
      if (p < pieces) *reinterpret_cast<uint4*>(qr + p * 16) = quant_pack16(v[i], s, inv);
    }
    for (int p = threadIdx.x + kQuantKeep * kQuantThreads; p < pieces; p += kQuantThreads) {
      float t[16];
      load16(xr + p * 16, t);
      *reinterpret_cast<uint4*>(qr + p * 16) = quant_pack16(t, s, inv);
    }
    if (threadIdx.x == 0) scale[row] = s;
  }
}

// W warps per row: the row's loads (kQuantVecs vectors of 16 bytes per lane) all
// in flight, the row in registers between the maximum and the rounding, at most
// one barrier of W warps.  W is the fewest that hold the row, more while the SMs
// have fewer than 8 warps each (600 rows of 2048 BF16: 2.8 us; with at most 4 or
// up to 16 warps an SM 3.3 and 3.1).  Copy bandwidth for large calls: 65536 rows of
// 2048 BF16 60.8 us (402 MB, 6.6 TB/s), 9600 of 8192 38.0 us (236 MB, 6.2 TB/s); a
// block per row 165 and 52 us.
constexpr int kQuantVecs = 8;
constexpr int kQuantWarps = 8;

// The row's vectors of lane `lane` of its 32 W, and the largest magnitude's bits
// over the row (turn: which half of s_max).
template <typename T, int W>
__device__ __forceinline__ unsigned load_row(const T* xr, int vecs, int lane, int team, unsigned (&s_max)[2][8],
                                             int turn, uint4 (&v)[kQuantVecs]) {
#pragma unroll
  for (int i = 0; i < kQuantVecs; ++i) {
    const int at = lane + i * 32 * W;
    v[i] = make_uint4(0, 0, 0, 0);
    if (at < vecs) v[i] = __ldg(reinterpret_cast<const uint4*>(xr) + at);
  }
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < kQuantVecs; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 2)  // the magnitudes' bits of two BF16 order as 16-bit integers
        m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
      else
        m = max(m, w[j] & 0x7FFFFFFFu);
    }
  }
  if constexpr (sizeof(T) == 2) m = max(m & 0xFFFF0000u, m << 16);
  m = warp_max_u32(m);
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) s_max[turn][threadIdx.x >> 5] = m;
    named_bar_sync(1 + team, W * 32);
#pragma unroll
    for (int w = 0; w < W; ++w) m = max(m, s_max[turn][team * W + w]);
  }
  return m;
}

// Eight BF16 to eight bytes.
__device__ __forceinline__ uint2 quant_pack8(const uint4& v, float s, float inv) {
  const float lo[4] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
  const float hi[4] = {bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
  return make_uint2(quant_pack4(lo, s, inv), quant_pack4(hi, s, inv));
}

template <typename T, int W>
__global__ void __launch_bounds__(kQuantThreads, 4) quantize_rows_warp_kernel(const T* __restrict__ x, int64_t n_rows,
                                                                              int n_cols, int8_t* __restrict__ q,
                                                                              float* __restrict__ scale) {
  constexpr int kTeams = kQuantThreads / 32 / W;  // rows of a block
  __shared__ unsigned s_max[2][kQuantThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int team = (threadIdx.x >> 5) / W, vecs = n_cols / (16 / static_cast<int>(sizeof(T)));
  const int lane = threadIdx.x - team * W * 32;  // of the row's 32 W
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + team; row < n_rows;
       row += static_cast<int64_t>(gridDim.x) * kTeams, turn ^= 1) {
    uint4 v[kQuantVecs];
    const float s = quant_scale(load_row<T, W>(x + row * n_cols, vecs, lane, team, s_max, turn, v));
    const float inv = 1.0f / s;
    int8_t* qr = q + row * n_cols;
#pragma unroll
    for (int i = 0; i < kQuantVecs; ++i) {
      const int at = lane + i * 32 * W;
      if (at < vecs) {
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<uint2*>(qr + static_cast<int64_t>(at) * 8) = quant_pack8(v[i], s, inv);
        } else {
          const float f[4] = {__uint_as_float(v[i].x), __uint_as_float(v[i].y), __uint_as_float(v[i].z),
                              __uint_as_float(v[i].w)};
          *reinterpret_cast<uint32_t*>(qr + static_cast<int64_t>(at) * 4) = quant_pack4(f, s, inv);
        }
      }
    }
    if (lane == 0) scale[row] = s;
  }
}

// The fewest warps that hold a row of vecs vectors, more while the SMs have few.
static int quant_warps(int64_t n_rows, int vecs) {
  int w = 1;
  while (w < 8 && (vecs > 32 * kQuantVecs * w || n_rows * w < kQuantWarps * num_sms())) w *= 2;
  return w;
}

template <typename T>
static cudaError_t run_quantize_rows(const T* x, int64_t n_rows, int n_cols, int8_t* q, float* scale,
                                     cudaStream_t st) {
  const int vecs = n_cols / (16 / static_cast<int>(sizeof(T)));
  const int w = quant_warps(n_rows, vecs);
  if (vecs <= 32 * kQuantVecs * w) {
    const int teams = kQuantThreads / 32 / w;
    const int64_t blocks = (n_rows + teams - 1) / teams;
    const auto run = [&](auto kernel) {
      return launch_k(kernel, dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)), dim3(kQuantThreads), 0, st,
                      x, n_rows, n_cols, q, scale);
    };
    if (w == 1) return run(quantize_rows_warp_kernel<T, 1>);
    if (w == 2) return run(quantize_rows_warp_kernel<T, 2>);
    if (w == 4) return run(quantize_rows_warp_kernel<T, 4>);
    return run(quantize_rows_warp_kernel<T, 8>);
  }
  const unsigned grid = static_cast<unsigned>(n_rows < 65536 ? n_rows : 65536);
  return launch_k(quantize_rows_kernel<T>, dim3(grid), dim3(kQuantThreads), 0, st, x, n_rows, n_cols, q, scale);
}

cudaError_t launch_quantize_rows(int dtype, const void* x, int64_t n_rows, int n_cols, int8_t* q, float* scale,
                                 cudaStream_t st) {
  if (dtype == kBF16)
    return run_quantize_rows(static_cast<const __nv_bfloat16*>(x), n_rows, n_cols, q, scale, st);
  return run_quantize_rows(static_cast<const float*>(x), n_rows, n_cols, q, scale, st);
}

// Tokens to the rows of their kept pairs: a token is read once and stored up to
// K + 1 times.  W warps per token, as for rows
// (16384 tokens of 2048, top-4: 39 -> 22 us against a block that reads each twice).
template <int W>
__global__ void __launch_bounds__(kQuantThreads, 4) quantize_dispatch_warp_kernel(
    const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ slot_of, int64_t T, int d, int K,
    int64_t max_rows, int8_t* __restrict__ x_q, float* __restrict__ x_scale, unsigned* __restrict__ amax,
    int8_t* __restrict__ xs_q, float* __restrict__ xs_scale, unsigned* __restrict__ amax_s) {
  constexpr int kTeams = kQuantThreads / 32 / W;
  __shared__ unsigned s_max[2][kQuantThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int team = (threadIdx.x >> 5) / W, vecs = d / 8;
  const int lane = threadIdx.x - team * W * 32;
  int turn = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTeams + team; t < T;
       t += static_cast<int64_t>(gridDim.x) * kTeams, turn ^= 1) {
    int mine = -1;  // lane k of every warp: the slot of choice k
    if ((lane & 31) < K) mine = slot_of[t * K + (lane & 31)];
    if (mine >= max_rows) mine = -1;
    uint4 v[kQuantVecs];
    const float s = quant_scale(load_row<__nv_bfloat16, W>(x + t * d, vecs, lane, team, s_max, turn, v));
    const float inv = 1.0f / s;
    uint2 p[kQuantVecs];
#pragma unroll
    for (int i = 0; i < kQuantVecs; ++i) p[i] = quant_pack8(v[i], s, inv);
    for (int k = xs_q ? -1 : 0; k < K; ++k) {
      const int slot = __shfl_sync(0xffffffffu, mine, k < 0 ? 0 : k);
      if (k >= 0 && slot < 0) continue;
      int8_t* out = k < 0 ? xs_q + t * d : x_q + static_cast<int64_t>(slot) * d;
#pragma unroll
      for (int i = 0; i < kQuantVecs; ++i) {
        const int at = lane + i * 32 * W;
        if (at < vecs) *reinterpret_cast<uint2*>(out + static_cast<int64_t>(at) * 8) = p[i];
      }
    }
    if (lane < 32 && mine >= 0) {
      x_scale[mine] = s;
      amax[mine] = 0;
    }
    if (lane == 0 && xs_q) {
      xs_scale[t] = s;
      amax_s[t] = 0;
    }
  }
}

// Rows of more than 16384 values: one block per token, which reads it twice.
__global__ void __launch_bounds__(kQuantThreads) quantize_dispatch_kernel(
    const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ slot_of, int64_t T, int d, int K,
    int64_t max_rows, int8_t* __restrict__ x_q, float* __restrict__ x_scale, unsigned* __restrict__ amax,
    int8_t* __restrict__ xs_q, float* __restrict__ xs_scale, unsigned* __restrict__ amax_s) {
  __shared__ unsigned s_max[kQuantThreads / 32];
  __shared__ int s_slot[kMaxTopK];
  pdl_wait();
  pdl_trigger();
  const int pieces = d / 16;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const __nv_bfloat16* xr = x + t * d;
    if (threadIdx.x < K) {
      const int sl = slot_of[t * K + threadIdx.x];
      s_slot[threadIdx.x] = sl < max_rows ? sl : -1;
    }
    unsigned m = 0;
    for (int p = threadIdx.x; p < pieces; p += kQuantThreads) {
      float v[16];
      load16(xr + p * 16, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) m = max(m, abs_bits(v[j]));
    }
    const float s = quant_scale(block_max_u32(m, s_max));
    const float inv = 1.0f / s;
    for (int p = threadIdx.x; p < pieces; p += kQuantThreads) {
      float v[16];
      load16(xr + p * 16, v);
      const uint4 w = quant_pack16(v, s, inv);
      for (int k = 0; k < K; ++k)
        if (s_slot[k] >= 0) *reinterpret_cast<uint4*>(x_q + static_cast<int64_t>(s_slot[k]) * d + p * 16) = w;
      if (xs_q) *reinterpret_cast<uint4*>(xs_q + t * d + p * 16) = w;
    }
    if (threadIdx.x < K && s_slot[threadIdx.x] >= 0) {
      x_scale[s_slot[threadIdx.x]] = s;
      amax[s_slot[threadIdx.x]] = 0;
    }
    if (threadIdx.x == 0 && xs_q) {
      xs_scale[t] = s;
      amax_s[t] = 0;
    }
    __syncthreads();
  }
}

cudaError_t launch_quantize_dispatch(const Problem& p, const void* x, const int32_t* slot_of, int8_t* x_q,
                                     float* x_scale, unsigned* amax, int8_t* xs_q, float* xs_scale, unsigned* amax_s,
                                     cudaStream_t st) {
  const int vecs = p.d / 8, w = quant_warps(p.T, vecs);
  if (vecs <= 32 * kQuantVecs * w) {
    const int teams = kQuantThreads / 32 / w;
    const int64_t blocks = (p.T + teams - 1) / teams;
    const auto run = [&](auto kernel) {
      return launch_k(kernel, dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)), dim3(kQuantThreads), 0, st,
                      static_cast<const __nv_bfloat16*>(x), slot_of, p.T, p.d, p.K, p.max_rows, x_q, x_scale, amax,
                      xs_q, xs_scale, amax_s);
    };
    if (w == 1) return run(quantize_dispatch_warp_kernel<1>);
    if (w == 2) return run(quantize_dispatch_warp_kernel<2>);
    if (w == 4) return run(quantize_dispatch_warp_kernel<4>);
    return run(quantize_dispatch_warp_kernel<8>);
  }
  const unsigned grid = static_cast<unsigned>(p.T < 65536 ? p.T : 65536);
  return launch_k(quantize_dispatch_kernel, dim3(grid), dim3(kQuantThreads), 0, st,
                  static_cast<const __nv_bfloat16*>(x), slot_of, p.T, p.d, p.K, p.max_rows, x_q, x_scale, amax, xs_q,
                  xs_scale, amax_s);
}

// A kernel, not a memset, so that the product behind it may start early
// (programmatic dependent launch).
__global__ void __launch_bounds__(kQuantThreads) clear_amax_kernel(unsigned* __restrict__ amax, int64_t n) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    amax[i] = 0;
}

cudaError_t launch_clear_amax(unsigned* amax, int64_t n, cudaStream_t st) {
  int64_t grid = (n + kQuantThreads - 1) / kQuantThreads;
  if (grid > 1024) grid = 1024;
  return launch_k(clear_amax_kernel, dim3(static_cast<unsigned>(grid)), dim3(kQuantThreads), 0, st, amax, n);
}

// FP32 rows h [*, n_cols], amax [*] bits of each row's largest magnitude; rows
// [0, min(*n_live, n_rows)) (n_live NULL: n_rows).  A warp takes 512 columns of
// a row at a time: four coalesced 16-byte loads per lane in flight.
// blockIdx.y selects one of two sets of rows (routed, shared).
struct HiddenRows {
  const float* h;
  const unsigned* amax;
  const int32_t* n_live;
  int n_rows, n_cols;
  int8_t* q;
  float* scale;
};

__global__ void __launch_bounds__(kQuantThreads) quantize_hidden_kernel(const HiddenRows a0, const HiddenRows a1) {
  pdl_wait();
  pdl_trigger();
  const HiddenRows a = blockIdx.y ? a1 : a0;
  const int rows = a.n_live ? min(max(*a.n_live, 0), a.n_rows) : a.n_rows;
  const int pieces = (a.n_cols + 511) / 512, lane = threadIdx.x & 31;
  const int64_t total = static_cast<int64_t>(rows) * pieces;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5); i < total; i += warps) {
    const int row = static_cast<int>(i / pieces);
    const int c0 = static_cast<int>(i - static_cast<int64_t>(row) * pieces) * 512 + lane * 4;
    const float* hr = a.h + static_cast<int64_t>(row) * a.n_cols;
    float4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + j * 128 < a.n_cols) v[j] = __ldcs(reinterpret_cast<const float4*>(hr + c0 + j * 128));
    const float s = quant_scale(a.amax[row]);
    const float inv = 1.0f / s;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c0 + j * 128 < a.n_cols) {
        const float f[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        *reinterpret_cast<uint32_t*>(a.q + static_cast<int64_t>(row) * a.n_cols + c0 + j * 128) =
            quant_pack4(f, s, inv);
      }
    }
    if (c0 == 0) a.scale[row] = s;
  }
}

cudaError_t launch_quantize_hidden(const float* h, const unsigned* amax, const int32_t* n_live, int64_t n_rows,
                                   int n_cols, int8_t* q, float* scale, cudaStream_t st, const float* h2,
                                   const unsigned* amax2, int64_t n_rows2, int n_cols2, int8_t* q2, float* scale2) {
  const HiddenRows a{h, amax, n_live, static_cast<int>(n_rows), n_cols, q, scale};
  const HiddenRows b{h2, amax2, nullptr, static_cast<int>(n_rows2), n_cols2, q2, scale2};
  int64_t pieces = n_rows * ((n_cols + 511) / 512);
  if (h2) pieces = std::max(pieces, n_rows2 * ((n_cols2 + 511) / 512));
  int64_t grid = (pieces + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
  const int64_t most = static_cast<int64_t>(num_sms()) * 8;
  if (grid > most) grid = most;
  return launch_k(quantize_hidden_kernel, dim3(static_cast<unsigned>(grid), h2 ? 2 : 1), dim3(kQuantThreads), 0, st, a,
                  b);
}

}  // namespace moe
