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
    rows_scan_kernel(const int32_t* __restrict__ offsets, int64_t S, int M, int tile_rows, Rows out,
                     unsigned int* status) {
  after_previous();
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
    tiles += (n + tile_rows - 1) / tile_rows;
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
      for (int r = 0; r < n; r += tile_rows) {
        const int here = min(n - r, tile_rows);
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

// One CTA per tile, a thread per row: the rows' slots, tokens and gates, and each slot's row.
__global__ void __launch_bounds__(2 * kTileRows)
    rows_fill_kernel(const int32_t* __restrict__ offsets, const int32_t* __restrict__ slots,
                     const float* __restrict__ gate, int64_t S, int k, const float* __restrict__ token_scale,
                     float* __restrict__ row_scale, Rows out, unsigned int* status) {
  after_previous();
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
  const int token = ok ? slot / k : 0;
  out.row_token[row] = real ? token : -1 - token;
  if (token_scale) row_scale[row] = token_scale[token];
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

// A thread takes 8 columns of a token (and those `across` threads further on); `across`, a power of two, threads a
// token; `each` tokens one after the other.  Bound by DRAM: every slot's row is read once.  Four rows' loads are in flight
// a thread, and the rows that come next are looked up meanwhile; looked up when they are needed, they take as long as the
// loads themselves (N = 262144, h = 512, k = 4: 282 us; so: 203 us, the rate of a plain copy).
__device__ __forceinline__ void rows_of(const int32_t* __restrict__ slot_row, int64_t n, int j0, int k, int (&r)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = j0 + j < k ? __ldg(slot_row + n * k + j0 + j) : -1;
}

__global__ void __launch_bounds__(256, 5)
    combine_kernel(const __nv_bfloat16* __restrict__ y, const int32_t* __restrict__ slot_row, int64_t N, int h, int k,
                   int log_across, int each, __nv_bfloat16* __restrict__ out) {
  after_previous();
  const int groups = h >> 3, across = 1 << log_across, tokens = 256 >> log_across;
  int64_t n = (int64_t)blockIdx.x * each * tokens + (threadIdx.x >> log_across);
  const int64_t end = min(N, (int64_t)(blockIdx.x + 1) * each * tokens);
  const int c0 = threadIdx.x & (across - 1);
  if (n >= end || c0 >= groups) return;
  int r[4], next[4];
  rows_of(slot_row, n, 0, k, r);
  for (; n < end; n += tokens) {
    for (int c = c0; c < groups; c += across) {
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int j0 = 0; j0 < k; j0 += 4) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = r[j] >= 0 ? __ldcs(reinterpret_cast<const uint4*>(y + (size_t)r[j] * h) + c) : make_uint4(0, 0, 0, 0);
        const bool more = j0 + 4 < k, same = more || c + across < groups;
        const int64_t at = same ? n : n + tokens;
        if (at < end) rows_of(slot_row, at, more ? j0 + 4 : 0, k, next);
#pragma unroll
        for (int j = 0; j < 4; ++j) add8(acc, v[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = next[j];
      }
      reinterpret_cast<uint4*>(out + (size_t)n * h)[c] = pack8(acc);
    }
  }
}

// One warp per row of the padded layout, eight pieces of 16 bytes in flight a lane; zeros for a row that is no slot.
__global__ void __launch_bounds__(256)
    pick_kernel(const uint4* __restrict__ src, const int32_t* __restrict__ row_token, const int32_t* __restrict__ rows,
                int pieces, uint4* __restrict__ dst) {
  after_previous();
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= *rows) return;
  const int token = row_token[row];
  const uint4* from = src + (size_t)max(token, 0) * pieces;
  uint4* to = dst + (size_t)row * pieces;
  for (int c = lane; c < pieces; c += 256) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 32 * i < pieces) v[i] = token >= 0 ? __ldg(from + c + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 32 * i < pieces) to[c + 32 * i] = v[i];
  }
}

// Sixteen lanes a token, one a slot (k <= 16).  The gate of a slot that no expert lists is in no sum: it may be no number.
__global__ void __launch_bounds__(256)
    gate_grads_kernel(const float* __restrict__ part, int parts, int64_t R, const int32_t* __restrict__ slot_row,
                      const float* __restrict__ gate, int64_t N, int k, float* __restrict__ gate_bar,
                      float* __restrict__ logits_bar) {
  after_previous();
  const int64_t n = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int j = threadIdx.x & 15;
  const bool in = n < N && j < k;
  const int row = in ? slot_row[n * k + j] : -1;
  const float g = in ? gate[n * k + j] : 0.f;
  float s = 0.f;
  if (row >= 0) {
#pragma unroll 8
    for (int p = 0; p < parts; ++p) s += part[p * R + row];
  }
  float dot = row >= 0 ? g * s : 0.f;
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if (in) {
    gate_bar[n * k + j] = s;
    logits_bar[n * k + j] = g * (s - dot);
  }
}

constexpr int kHeld = 8;  // 16-byte pieces of a row that a lane keeps between the two passes

// Largest magnitudes of bf16 pairs as their bits, whose order that of the magnitudes is, a NaN above all.
__device__ __forceinline__ uint32_t top_pairs(uint32_t top, uint32_t w) {
  asm("max.u16x2 %0, %0, %1;" : "+r"(top) : "r"(w));
  return top;
}

__device__ __forceinline__ uint32_t top8(uint4 w, uint32_t top) {
  constexpr uint32_t kMagnitude = 0x7fff7fffu;
  return top_pairs(top_pairs(top_pairs(top_pairs(top, w.x & kMagnitude), w.y & kMagnitude), w.z & kMagnitude),
                   w.w & kMagnitude);
}

__device__ __forceinline__ uint2 round8x8(uint4 w, float div, float inv) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&w);
  const float2 a = __bfloat1622float2(p[0]), b = __bfloat1622float2(p[1]), c = __bfloat1622float2(p[2]),
               d = __bfloat1622float2(p[3]);
  return make_uint2(round8x4(a.x, a.y, b.x, b.y, div, inv), round8x4(c.x, c.y, d.x, d.y, div, inv));
}

// One warp per row (width a multiple of 16): no barrier, and enough rows in flight to cover the latency of one.  The
// first 2048 values stay in registers between finding the largest and rounding; what is beyond is read again.
__global__ void __launch_bounds__(128, 8)
    quantize_bf16_kernel(const __nv_bfloat16* __restrict__ v, int64_t rows, int width, int8_t* __restrict__ q,
                         float* __restrict__ scale) {
  after_previous();
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const uint4* src = reinterpret_cast<const uint4*>(v + row * width);
  const int n = width / 8;
  uint4 held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = lane + i * 32;
    held[i] = c < n ? src[c] : make_uint4(0, 0, 0, 0);
  }
  uint32_t tops = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) tops = top8(held[i], tops);
  for (int c = lane + kHeld * 32; c < n; c += 32) tops = top8(src[c], tops);
  const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, max(tops << 16, tops & 0xffff0000u)));
  const float div = divisor_of(top), inv = __fdiv_rn(127.f, div);
  uint2* dst = reinterpret_cast<uint2*>(q + row * width);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = lane + i * 32;
    if (c < n) dst[c] = round8x8(held[i], div, inv);
  }
  for (int c = lane + kHeld * 32; c < n; c += 32) dst[c] = round8x8(src[c], div, inv);
  if (lane == 0) scale[row] = __fdiv_rn(top, 127.f);
}

constexpr int kRowsPerBlock = 32;

// Four rows a warp, one after the other; the first 1024 values of a row stay in registers.
__global__ void __launch_bounds__(256)
    quantize_rows_kernel(const float* __restrict__ v, int width, Rows r, int8_t* __restrict__ q,
                         float* __restrict__ scale) {
  after_previous();
  const int lane = threadIdx.x & 31;
  if ((int)blockIdx.x >= *r.n_tiles) return;
  const int4 t = r.tiles[blockIdx.x];
  const int n = width / 4;
  for (int i = blockIdx.y * kRowsPerBlock + (threadIdx.x >> 5); i < min(t.z, (int)(blockIdx.y + 1) * kRowsPerBlock);
       i += blockDim.x >> 5) {
    const size_t row = t.y + i;
    const float4* src = reinterpret_cast<const float4*>(v + row * width);
    float4 held[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = lane + 32 * j;
      held[j] = c < n ? src[c] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto top4 = [](float4 f, float top) {
      return top_of(top_of(top_of(top_of(top, f.x), f.y), f.z), f.w);
    };
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = top4(held[j], top);
    for (int c = lane + 256; c < n; c += 32) top = top4(src[c], top);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = top_of(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float div = divisor_of(top), inv = __fdiv_rn(127.f, div);
    auto round4 = [&](float4 f) { return round8x4(f.x, f.y, f.z, f.w, div, inv); };
    uint32_t* dst = reinterpret_cast<uint32_t*>(q + row * width);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = lane + 32 * j;
      if (c < n) dst[c] = round4(held[j]);
    }
    for (int c = lane + 256; c < n; c += 32) dst[c] = round4(src[c]);
    if (lane == 0) scale[row] = __fdiv_rn(top, 127.f);
  }
}

}  // namespace

cudaError_t launch_rows(const ExpertsArgs& a, const Rows& r, int tile_rows, const float* token_scale,
                        float* row_scale) {
  const int64_t S = a.S();
  cudaError_t e = cudaMemsetAsync(r.slot_row, 0xff, sizeof(int32_t) * (size_t)S, a.stream);
  if (e != cudaSuccess) return e;
  e = launch_next(rows_scan_kernel, dim3(1), dim3(kScanThreads), 0, a.stream, 1, a.offsets, S, a.M, tile_rows, r, a.status);
  if (e != cudaSuccess) return e;
  return launch_next(rows_fill_kernel, dim3((unsigned)max_tiles(S, a.M, tile_rows)), dim3(tile_rows), 0, a.stream, 1,
                     a.offsets, a.slots, a.gate, S, a.k, token_scale, row_scale, r, a.status);
}

cudaError_t launch_pick(const ExpertsArgs& a, const Rows& r, const void* src, int pitch, void* dst) {
  return launch_next(pick_kernel, dim3((unsigned)(max_rows(a.S(), a.M) / 8)), dim3(256), 0, a.stream, 1,
                     static_cast<const uint4*>(src), r.row_token, r.row_start + a.M, pitch / 16, static_cast<uint4*>(dst));
}

cudaError_t launch_combine(const ExpertsArgs& a, const Rows& r, const __nv_bfloat16* y, void* out) {
  // threads a token: up to 256, fewer where that leaves more of them without a column (h = 1096: 137 groups of 8
  // columns are 5 rounds of 32 threads, 160 places, but 256 places with 128 or 256 threads)
  const int groups = a.h / 8;
  int log_across = 0, places = 1 << 30;
  for (int l = 8; l >= 5; --l) {
    const int here = (groups + (1 << l) - 1) >> l << l;
    if (here < places) {
      places = here;
      log_across = l;
    }
  }
  const int64_t tokens = 256 >> log_across, blocks = (a.N + tokens - 1) / tokens;
  const int each = blocks >= 8192 ? 4 : 1;  // several tokens a thread where the SMs (5 blocks each) still get many blocks
  return launch_next(combine_kernel, dim3((unsigned)((blocks + each - 1) / each)), dim3(256), 0, a.stream, 1, y, r.slot_row,
                     a.N, a.h, a.k, log_across, each, static_cast<__nv_bfloat16*>(out));
}

cudaError_t launch_gate_grads(const ExpertsArgs& a, const Rows& r, const float* part, int parts, int64_t R) {
  return launch_next(gate_grads_kernel, dim3((unsigned)((a.N + 15) / 16)), dim3(256), 0, a.stream, 1, part, parts, R,
                     r.slot_row, a.gate, a.N, a.k, a.gate_bar, a.logits_bar);
}

cudaError_t launch_quantize_bf16(const __nv_bfloat16* v, int64_t rows, int width, int8_t* q, float* scale,
                                 cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  return launch_next(quantize_bf16_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, 1, v, rows, width, q,
                     scale);
}

cudaError_t launch_quantize_rows(const ExpertsArgs& a, const Rows& r, const float* v, int width, int8_t* q,
                                 float* scale, int tile_rows) {
  const dim3 grid((unsigned)max_tiles(a.S(), a.M, tile_rows), tile_rows / kRowsPerBlock);
  return launch_next(quantize_rows_kernel, grid, dim3(256), 0, a.stream, 1, v, width, r, q, scale);
}

}  // namespace more
