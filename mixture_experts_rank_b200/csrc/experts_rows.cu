// The experts' operators outside their matrix products, on the CUDA cores: the row layout, the sum
// over a token's slots, the gates' gradients and the rounding of rows to 8 bits.
#include <algorithm>

#include "experts_internal.cuh"

namespace more {
namespace {

constexpr int kScanThreads = 1024;

// Exclusive sum of (rows, tiles) over a CTA of kScanThreads threads; totals in *rows_sum, *tiles_sum.
__device__ void scan_pairs(int& rows, int& tiles, int* warp_rows, int* warp_tiles, int& rows_sum, int& tiles_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int r = rows, t = tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int r2 = __shfl_up_sync(0xffffffffu, r, d), t2 = __shfl_up_sync(0xffffffffu, t, d);
    if (lane >= d) {
      r += r2;
      t += t2;
    }
  }
  if (lane == 31) {
    warp_rows[warp] = r;
    warp_tiles[warp] = t;
  }
  __syncthreads();
  int rb = 0, tb = 0, ra = 0, ta = 0;
  for (int w = 0; w < kScanThreads / 32; ++w) {
    if (w == warp) {
      rb = ra;
      tb = ta;
    }
    ra += warp_rows[w];
    ta += warp_tiles[w];
  }
  rows = rb + r - rows;
  tiles = tb + t - tiles;
  rows_sum = ra;
  tiles_sum = ta;
}

// One CTA: every thread takes a run of experts, sums their padded rows and tiles, and after a scan
// over the threads writes the experts' first rows and tiles.  Offsets that fall, or lie outside
// [0, S], set MORE_DEVERR_BAD_INPUT and leave no expert with rows.
__global__ void __launch_bounds__(kScanThreads)
    rows_scan_kernel(const int32_t* __restrict__ offsets, int64_t S, int M, Rows out, unsigned int* status) {
  __shared__ int warp_rows[kScanThreads / 32], warp_tiles[kScanThreads / 32];
  __shared__ int bad;
  const int run = (M + kScanThreads - 1) / kScanThreads;
  const int e0 = min(M, (int)threadIdx.x * run), e1 = min(M, e0 + run);
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  int rows = 0, tiles = 0, broken = 0;
  int at = offsets[e0];
  if (at < 0 || at > S) broken = 1;
  for (int e = e0; e < e1; ++e) {
    const int next = offsets[e + 1];
    if (next < at || next > S) broken = 1;
    const int n = max(0, next - at);
    rows += (n + kRowPad - 1) / kRowPad * kRowPad;
    tiles += (n + kTileRows - 1) / kTileRows;
    at = next;
  }
  if (broken) atomicOr(&bad, 1);
  __syncthreads();
  const bool none = bad != 0;
  if (none) rows = tiles = 0;
  int rows_sum, tiles_sum;
  scan_pairs(rows, tiles, warp_rows, warp_tiles, rows_sum, tiles_sum);
  at = offsets[e0];
  for (int e = e0; e < e1; ++e) {
    const int next = offsets[e + 1];
    out.row_start[e] = rows;
    if (!none) {
      const int n = next - at;
      for (int r = 0; r < n; r += kTileRows) {
        const int here = min(n - r, kTileRows);
        out.tiles[tiles++] = make_int4(e, rows + r, here, (here + kRowPad - 1) / kRowPad * kRowPad);
      }
      rows += (n + kRowPad - 1) / kRowPad * kRowPad;
    }
    at = next;
  }
  if (threadIdx.x == 0) {
    out.row_start[M] = rows_sum;
    *out.n_tiles = tiles_sum;
    if (none) atomicOr(status, MORE_DEVERR_BAD_INPUT);
  }
}

// One CTA of 128 threads per tile: the rows' slots, tokens and gates, and each slot's row.
__global__ void __launch_bounds__(kTileRows)
    rows_fill_kernel(const int32_t* __restrict__ offsets, const int32_t* __restrict__ slots,
                     const float* __restrict__ gate, int64_t S, int k, Rows out, unsigned int* status) {
  if ((int)blockIdx.x >= *out.n_tiles) return;
  const int4 t = out.tiles[blockIdx.x];
  const int r = threadIdx.x;
  if (r >= t.w) return;
  const int first = offsets[t.x] + (t.y - out.row_start[t.x]);  // sorted position of the tile's first row
  const int slot = slots[first + min(r, t.z - 1)];
  const bool ok = slot >= 0 && slot < S;
  if (!ok) atomicOr(status, MORE_DEVERR_BAD_INPUT);
  const bool real = ok && r < t.z;
  const int row = t.y + r;
  out.row_slot[row] = real ? slot : -1;
  out.row_token[row] = ok ? slot / k : 0;
  out.row_gate[row] = real ? gate[slot] : 0.f;
  if (real) out.slot_row[slot] = row;
}

__device__ __forceinline__ void add8(float* acc, uint4 v) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 f = __bfloat1622float2(p[q]);
    acc[2 * q] += f.x;
    acc[2 * q + 1] += f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint4 v;
  __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int q = 0; q < 4; ++q) p[q] = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
  return v;
}

// One thread per 8 columns of a token; the k rows' loads are issued together.
__global__ void __launch_bounds__(256)
    combine_kernel(const __nv_bfloat16* __restrict__ y, const int32_t* __restrict__ slot_row, int64_t N, int h, int k,
                   __nv_bfloat16* __restrict__ out) {
  const int groups = h >> 3;
  const int64_t total = N * groups;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t n = i / groups;
    const int c = (int)(i - n * groups);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < k; j0 += 8) {
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = j0 + j < k ? slot_row[n * k + j0 + j] : -1;
        v[j] = row >= 0 ? __ldg(reinterpret_cast<const uint4*>(y + (size_t)row * h) + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) add8(acc, v[j]);
    }
    *(reinterpret_cast<uint4*>(out + (size_t)n * h) + c) = pack8(acc);
  }
}

// One thread per token.
__global__ void __launch_bounds__(256)
    gate_grads_kernel(const float* __restrict__ part, int parts, int64_t R, const int32_t* __restrict__ slot_row,
                      const float* __restrict__ gate, int64_t N, int k, float* __restrict__ gate_bar,
                      float* __restrict__ logits_bar) {
  const int64_t n = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (n >= N) return;
  float gb[MORE_KMAX], dot = 0.f;
  for (int j = 0; j < k; ++j) {
    const int row = slot_row[n * k + j];
    float s = 0.f;
    if (row >= 0)
      for (int p = 0; p < parts; ++p) s += part[p * R + row];
    gb[j] = s;
    dot = fmaf(gate[n * k + j], s, dot);
    gate_bar[n * k + j] = s;
  }
  for (int j = 0; j < k; ++j) logits_bar[n * k + j] = gate[n * k + j] * (gb[j] - dot);
}

__device__ __forceinline__ int8_t round8(float v, float top) {
  // 127 v is exact for a bf16 v, so the division's rounding cannot move a value across a half
  return (int8_t)__float2int_rn(__fdiv_rn(127.f * v, top));
}

__device__ __forceinline__ float block_max(float v, float* warps) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  float m = warps[0];
  for (int w = 1; w < (int)blockDim.x >> 5; ++w) m = fmaxf(m, warps[w]);
  return m;
}

constexpr int kQuantThreads = 128;

// One CTA per row (width a multiple of 16); the second reading of the row comes from L1 or L2.
__global__ void __launch_bounds__(kQuantThreads)
    quantize_bf16_kernel(const __nv_bfloat16* __restrict__ v, int width, int8_t* __restrict__ q,
                         float* __restrict__ scale) {
  __shared__ float warps[kQuantThreads / 32];
  const size_t row = blockIdx.x;
  const uint4* src = reinterpret_cast<const uint4*>(v + row * width);
  float top = 0.f;
  for (int c = threadIdx.x; c < width / 8; c += kQuantThreads) {
    const uint4 w = src[c];
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(p[i]);
      top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
  }
  top = block_max(top, warps);
  const float div = top > 0.f ? top : 1.f;
  uint2* dst = reinterpret_cast<uint2*>(q + row * width);
  for (int c = threadIdx.x; c < width / 8; c += kQuantThreads) {
    const uint4 w = src[c];
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&w);
    union {
      int8_t b[8];
      uint2 u;
    } o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(p[i]);
      o.b[2 * i] = round8(f.x, div);
      o.b[2 * i + 1] = round8(f.y, div);
    }
    dst[c] = o.u;
  }
  if (threadIdx.x == 0) scale[row] = __fdiv_rn(top, 127.f);
}

// One warp per row of the tiles' slots.
__global__ void __launch_bounds__(256)
    quantize_rows_kernel(const float* __restrict__ v, int width, Rows r, int8_t* __restrict__ q,
                         float* __restrict__ scale) {
  const int lane = threadIdx.x & 31;
  if ((int)blockIdx.x >= *r.n_tiles) return;
  const int4 t = r.tiles[blockIdx.x];
  for (int i = threadIdx.x >> 5; i < t.z; i += blockDim.x >> 5) {
    const size_t row = t.y + i;
    const float4* src = reinterpret_cast<const float4*>(v + row * width);
    float top = 0.f;
    for (int c = lane; c < width / 4; c += 32) {
      const float4 f = src[c];
      top = fmaxf(fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y))), fmaxf(fabsf(f.z), fabsf(f.w)));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float div = top > 0.f ? top : 1.f;
    for (int c = lane; c < width / 4; c += 32) {
      const float4 f = src[c];
      char4 o;
      o.x = round8(f.x, div);
      o.y = round8(f.y, div);
      o.z = round8(f.z, div);
      o.w = round8(f.w, div);
      reinterpret_cast<char4*>(q + row * width)[c] = o;
    }
    if (lane == 0) scale[row] = __fdiv_rn(top, 127.f);
  }
}

}  // namespace

cudaError_t launch_rows(const ExpertsArgs& a, const Rows& r) {
  const int64_t S = a.S();
  cudaError_t e = cudaMemsetAsync(r.slot_row, 0xff, sizeof(int32_t) * (size_t)S, a.stream);
  if (e != cudaSuccess) return e;
  rows_scan_kernel<<<1, kScanThreads, 0, a.stream>>>(a.offsets, S, a.M, r, a.status);
  rows_fill_kernel<<<(unsigned)max_tiles(S, a.M), kTileRows, 0, a.stream>>>(a.offsets, a.slots, a.gate, S, a.k, r,
                                                                             a.status);
  return cudaGetLastError();
}

cudaError_t launch_combine(const ExpertsArgs& a, const Rows& r, const __nv_bfloat16* y, void* out) {
  const int64_t work = a.N * (a.h / 8);
  const unsigned grid = (unsigned)std::min<int64_t>((work + 255) / 256, 1 << 20);
  combine_kernel<<<grid, 256, 0, a.stream>>>(y, r.slot_row, a.N, a.h, a.k, static_cast<__nv_bfloat16*>(out));
  return cudaGetLastError();
}

cudaError_t launch_gate_grads(const ExpertsArgs& a, const Rows& r, const float* part, int parts, int64_t R) {
  gate_grads_kernel<<<(unsigned)((a.N + 255) / 256), 256, 0, a.stream>>>(part, parts, R, r.slot_row, a.gate, a.N, a.k,
                                                                          a.gate_bar, a.logits_bar);
  return cudaGetLastError();
}

cudaError_t launch_quantize_bf16(const __nv_bfloat16* v, int64_t rows, int width, int8_t* q, float* scale,
                                 cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  quantize_bf16_kernel<<<(unsigned)rows, kQuantThreads, 0, stream>>>(v, width, q, scale);
  return cudaGetLastError();
}

cudaError_t launch_quantize_rows(const ExpertsArgs& a, const Rows& r, const float* v, int width, int8_t* q,
                                 float* scale) {
  quantize_rows_kernel<<<(unsigned)max_tiles(a.S(), a.M), 256, 0, a.stream>>>(v, width, r, q, scale);
  return cudaGetLastError();
}

}  // namespace more
