// The whole layer for a few tokens, in one cooperative kernel.
//
// The time of such a call is the latency of its steps and the reading of the selected experts' weights, once each, so
// everything is laid out for those: no tensor cores (a handful of rows an expert), every step spread over all CTAs with
// a barrier over the grid behind it, every warp streaming whole rows of weights.
//   1. z = x R1: a CTA takes 16 columns of a token's z, its warps parts of h.  With 8-bit weights other CTAs round x.
//   2. The logits z R2: a warp takes 8 experts of a token, a lane one row of R2 (or r / 32 of them); the N x M logits of
//      these few tokens go through scratch.
//   3. A CTA takes a token's largest k logits and their softmax (for up to kSolo tokens every CTA does so itself, which
//      saves a barrier).  Then every CTA groups the N k selections by expert, up to 8 a group: its own copy.
//   4. Up: a warp takes row i of A_e and of B_e and the group's tokens; m = silu(a) * b goes to scratch in fp32.
//      Where there are too few rows for the machine's warps, 2 to 8 warps share a row, each a part of h.
//   5. Down: every CTA owns h / CTAs output channels for all experts, so a token's k contributions meet in its
//      shared memory, and out[n] = sum_j gate * y is summed there in the order of j: no second pass over a row buffer,
//      and no atomics on the result.
// z is carried as the bf16 pair of the routing kernels; all else stays in fp32 until the output.  With 8-bit weights
// the products are integer dot products (four an instruction); m is rounded to 8 bits when it is read, with its row's
// largest magnitude found after the barrier.
#include <algorithm>
#include <atomic>

#include "experts_internal.cuh"
#include "sm100_ptx.cuh"
#include "warp_simt.cuh"

namespace more {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 8;  // selections of one expert that share a reading of its weights
constexpr int64_t kFewTokens = 64;
constexpr uint32_t kSmemMost = 200 * 1024;
constexpr int kRowBlocks = 4;  // rows (times 32 / lanes a row) that a warp carries in the second product

struct LayerArgs {
  const __nv_bfloat16 *X, *R1, *R2;
  int8_t* Xq;  // int8: X in 8 bits, and its scales
  float* x_scale;
  const void *W_up, *W_down;
  const float *up_scale, *down_scale;
  float* z;       // [N][r]
  float* logits;  // [N][M]
  int32_t* idx;   // [S]
  float* gate;    // [S]
  float* mid;     // [S][s]
  __nv_bfloat16* out;
  unsigned int* barrier;  // 0 at the start
  unsigned int* status;
  int N, h, r, s, M, k, S;
};

// ---- shared memory: the groups, the selections' output channels ------------------------------------------------
struct Shared {
  int32_t* expert;     // [S] expert of a selection (-1: none)
  int16_t* member;     // [S][kGroup] selections of a group
  int16_t* lead;       // [S] group of a leading selection
  int32_t* group_e;    // [S] expert of a group
  int32_t* group_n;    // [S] its selections
  float* gate;         // [S]
  float* top;          // [S] largest |m| (int8)
  float* y;            // [S][R]
};

__host__ __device__ inline uint32_t round16(uint32_t v) { return (v + 15) & ~15u; }

__host__ __device__ inline uint32_t layer_smem(int S, int R) {
  return round16(4 * S) * 5 + round16(2 * kGroup * S) + round16(2 * S) + round16(4 * S * R) + 16;
}

__device__ __forceinline__ Shared shared_at(uint8_t* p, int S, int R) {
  Shared r;
  r.expert = reinterpret_cast<int32_t*>(p);
  p += round16(4 * S);
  r.group_e = reinterpret_cast<int32_t*>(p);
  p += round16(4 * S);
  r.group_n = reinterpret_cast<int32_t*>(p);
  p += round16(4 * S);
  r.gate = reinterpret_cast<float*>(p);
  p += round16(4 * S);
  r.top = reinterpret_cast<float*>(p);
  p += round16(4 * S);
  r.member = reinterpret_cast<int16_t*>(p);
  p += round16(2 * kGroup * S);
  r.lead = reinterpret_cast<int16_t*>(p);
  p += round16(2 * S);
  r.y = reinterpret_cast<float*>(p);
  return r;
}

// Weights are read once: they pass by L1.
__device__ __forceinline__ uint4 load_weights(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// bf16 pairs as fp32
__device__ __forceinline__ void widen(uint32_t u, float& lo, float& hi) {
  lo = __uint_as_float(u << 16);
  hi = __uint_as_float(u & 0xffff0000u);
}

__device__ __forceinline__ void widen8(uint4 v, float (&x)[8]) {
  widen(v.x, x[0], x[1]);
  widen(v.y, x[2], x[3]);
  widen(v.z, x[4], x[5]);
  widen(v.w, x[6], x[7]);
}

__device__ __forceinline__ void dot8(float& acc, uint4 w, const float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    widen(u[i], lo, hi);
    acc = fmaf(lo, x[2 * i], acc);
    acc = fmaf(hi, x[2 * i + 1], acc);
  }
}

// Sums V values over the warp; lane l ends with value l >> (5 - log2 V).
template <int V, class T>
__device__ __forceinline__ T reduce_scatter(T (&v)[V], int lane) {
  int d = 16;
#pragma unroll
  for (int n = V; n > 1; n >>= 1, d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int q = 0; q < n / 2; ++q) {
      const T send = up ? v[q] : v[q + n / 2];
      v[q] = (up ? v[q + n / 2] : v[q]) + __shfl_xor_sync(0xffffffffu, send, d);
    }
  }
#pragma unroll
  for (; d >= 1; d >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
  return v[0];
}

template <int V>
constexpr int log2_of() {
  return V == 1 ? 0 : 1 + log2_of<(V > 1 ? V / 2 : 1)>();
}

// Barrier number `turn` (from 1) over a cooperative grid; false once the wait has run out.
__device__ bool grid_barrier(unsigned int* counter, unsigned turn, unsigned int* status, int* failed) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(counter, 1u);
    *failed = 0;
    const long long t0 = clock64();
    for (unsigned spin = 0;; ++spin) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
      if (v >= turn * gridDim.x) break;
      if ((spin & 255u) == 255u && clock64() - t0 > 8000000000ll) {  // some 4 s
        atomicOr(status, MORE_DEVERR_WAIT_TIMEOUT);
        *failed = 1;
        break;
      }
    }
    __threadfence();
  }
  __syncthreads();
  return *failed == 0;
}

// Step 1.  `part`: 16 sums a warp.
__device__ void project_tokens(const LayerArgs& a, float (*part)[2 * kGroup]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, blocks = a.r / 16;
  for (int u = blockIdx.x; u < a.N * blocks; u += gridDim.x) {
    const int n = u / blocks, b = (u - n * blocks) * 16;
    float v;
    int i;
    warp_partial_z16_strided(a.X + (size_t)n * a.h, a.R1, a.h, a.r, b, threadIdx.x, kThreads, lane, v, i);
    if ((lane & 1) == 0) part[warp][i - b] = v;
    __syncthreads();
    if (threadIdx.x < 16) {
      float z = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) z += part[w][threadIdx.x];
      a.z[n * a.r + b + threadIdx.x] = split_bf16_pair(z);
    }
    __syncthreads();
  }
}

// x in 8 bits, a token a CTA, from the last CTA down (the first have z to compute).
__device__ void round_tokens(const LayerArgs& a, float* warp_tops) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int n = gridDim.x - 1 - blockIdx.x; n < a.N; n += gridDim.x) {
    const uint4* src = reinterpret_cast<const uint4*>(a.X + (size_t)n * a.h);
    float top = 0.f, x[8];
    for (int c = threadIdx.x; c < a.h / 8; c += kThreads) {
      widen8(src[c], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0) warp_tops[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, warp_tops[w]);
    const float div = top > 0.f ? top : 1.f, inv = __fdiv_rn(127.f, div);
    for (int c = threadIdx.x; c < a.h / 8; c += kThreads) {
      widen8(src[c], x);
      uint32_t o[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i >> 2] |= (uint32_t)(uint8_t)round8(x[i], div, inv) << (8 * (i & 3));
      reinterpret_cast<uint2*>(a.Xq + (size_t)n * a.h)[c] = make_uint2(o[0], o[1]);
    }
    if (threadIdx.x == 0) a.x_scale[n] = __fdiv_rn(top, 127.f);
    __syncthreads();
  }
}

// Step 2.
__device__ void expert_logits(const LayerArgs& a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int octets = a.M / 8, mine = (octets - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  for (int u = warp; u < mine * a.N; u += kWarps) {
    const int j = u / a.N, n = u - j * a.N;
    const int e0 = 8 * ((int)blockIdx.x + (int)gridDim.x * j);
    uint4 w[4];
    float zi[4], acc[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = lane + 32 * i;
      const bool in = row < a.r;
      w[i] = in ? __ldg(reinterpret_cast<const uint4*>(a.R2 + (size_t)row * a.M + e0)) : make_uint4(0, 0, 0, 0);
      zi[i] = in ? a.z[n * a.r + row] : 0.f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[8];
      widen8(w[i], x);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = fmaf(zi[i], x[q], acc[q]);
    }
    const float v = reduce_scatter<8>(acc, lane);
    if ((lane & 3) == 0) a.logits[(size_t)n * a.M + e0 + (lane >> 2)] = v;
  }
}

// Step 3 for token n: its selections and gates at idx and gate (shared or global memory).
template <int KCAP>
__device__ void select_experts(const LayerArgs& a, int n, float (*pv)[KCAP], int (*pe)[KCAP], int32_t* idx,
                               float* gate) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* l = a.logits + (size_t)n * a.M;
  TopList<KCAP> list;
  list.init();
  for (int e = threadIdx.x; e < a.M; e += 4 * kThreads) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = e + i * kThreads < a.M ? l[e + i * kThreads] : -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) list.insert(v[i], e + i * kThreads);
  }
  float v;
  int e;
  warp_merge_topk<KCAP>(list, a.k, lane, v, e);
  if (lane < KCAP) {
    pv[warp][lane] = v;
    pe[warp][lane] = e;
  }
  __syncthreads();
  if (warp == 0) {
    TopList<KCAP> all;
    all.init();
    for (int q = lane; q < kWarps * KCAP; q += 32)
      if (q % KCAP < a.k) all.insert_any(pv[q / KCAP][q % KCAP], pe[q / KCAP][q % KCAP]);
    warp_merge_topk<KCAP>(all, a.k, lane, v, e);
    const float top = __shfl_sync(0xffffffffu, v, 0);
    const float ex = lane < a.k ? expf(v - top) : 0.f;
    float sum = ex;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane < a.k) {
      idx[n * a.k + lane] = e;
      gate[n * a.k + lane] = ex / sum;
    }
  }
  __syncthreads();
}

// Groups the selections by expert, in their order; the number of groups.
__device__ int group_selections(const LayerArgs& a, const Shared& sh, bool solo, int* counts) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < a.S; i += kThreads) {
    const int e = solo ? sh.expert[i] : a.idx[i];
    if (!solo) sh.gate[i] = a.gate[i];
    const bool ok = e >= 0 && e < a.M;
    if (!ok && blockIdx.x == 0) atomicOr(a.status, MORE_DEVERR_BAD_INPUT);
    sh.expert[i] = ok ? e : -1;
  }
  __syncthreads();
  int groups = 0;
  for (int base = 0; base < a.S; base += kThreads) {
    const int i = base + threadIdx.x;
    const int e = i < a.S ? sh.expert[i] : -1;
    int before = 0, lead = i;  // earlier selections of the same expert; the one that leads this one's group
    if (e >= 0) {
      for (int q = 0; q < i; ++q)
        if (sh.expert[q] == e) {
          if (before % kGroup == 0) lead = q;
          ++before;
        }
      if (before % kGroup == 0) lead = i;
    }
    const bool leads = e >= 0 && lead == i;
    const unsigned vote = __ballot_sync(0xffffffffu, leads);
    if (lane == 0) counts[warp] = __popc(vote);
    __syncthreads();
    int at = groups;
    for (int w = 0; w < kWarps; ++w) {
      at += w < warp ? counts[w] : 0;
      groups += counts[w];
    }
    if (leads) {
      const int g = at + __popc(vote & ((1u << lane) - 1));
      sh.lead[i] = (int16_t)g;
      sh.group_e[g] = e;
      sh.group_n[g] = 0;
    }
    __syncthreads();
    if (e >= 0) {
      const int g = sh.lead[lead];
      sh.member[g * kGroup + before % kGroup] = (int16_t)i;
      atomicAdd(&sh.group_n[g], 1);
    }
    __syncthreads();
  }
  return groups;
}

// Partial a and b of up to TB selections for this warp's part of h; lane l gets value l >> (5 - log2(2 TB)) of
// (a_0, b_0, a_1, b_1, ...).
template <int TB>
__device__ __forceinline__ float up_bf16(const LayerArgs& a, const uint8_t* ra, const uint8_t* rb, const int (&tok)[TB],
                                         int part, int parts, int lane) {
  float acc[2 * TB];
#pragma unroll
  for (int i = 0; i < 2 * TB; ++i) acc[i] = 0.f;
  constexpr int kAhead = 4;
  const int step = 256 * parts;
  for (int c = part * 256 + lane * 8; c < a.h; c += kAhead * step) {
    uint4 wa[kAhead], wb[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int col = c + i * step;
      if (col < a.h) {
        wa[i] = load_weights(ra + 2 * (size_t)col);
        wb[i] = load_weights(rb + 2 * (size_t)col);
      } else {
        wa[i] = wb[i] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int col = c + i * step;
      if (col >= a.h) break;
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.X + (size_t)tok[t] * a.h + col));
        float x[8];
        widen8(v, x);
        dot8(acc[2 * t], wa[i], x);
        dot8(acc[2 * t + 1], wb[i], x);
      }
    }
  }
  return reduce_scatter<2 * TB>(acc, lane);
}

__device__ __forceinline__ int dot16(uint4 w, uint4 x, int acc) {
  acc = __dp4a((int)w.x, (int)x.x, acc);
  acc = __dp4a((int)w.y, (int)x.y, acc);
  acc = __dp4a((int)w.z, (int)x.z, acc);
  return __dp4a((int)w.w, (int)x.w, acc);
}

template <int TB>
__device__ __forceinline__ float up_int8(const LayerArgs& a, const uint8_t* ra, const uint8_t* rb, const int (&tok)[TB],
                                         int part, int parts, int lane) {
  int acc[2 * TB];
#pragma unroll
  for (int i = 0; i < 2 * TB; ++i) acc[i] = 0;
  constexpr int kAhead = 4;
  const int step = 512 * parts;
  for (int c = part * 512 + lane * 16; c < a.h; c += kAhead * step) {
    uint4 wa[kAhead], wb[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int col = c + i * step;
      if (col < a.h) {
        wa[i] = load_weights(ra + (size_t)col);
        wb[i] = load_weights(rb + (size_t)col);
      } else {
        wa[i] = wb[i] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int col = c + i * step;
      if (col >= a.h) break;
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const uint4 x = *reinterpret_cast<const uint4*>(a.Xq + (size_t)tok[t] * a.h + col);  // written by this kernel
        acc[2 * t] = dot16(wa[i], x, acc[2 * t]);
        acc[2 * t + 1] = dot16(wb[i], x, acc[2 * t + 1]);
      }
    }
  }
  // whole sums of 8-bit products stay below 2^24 for h <= 1024 only: they are added in 32-bit integers
  return __int_as_float(reduce_scatter<2 * TB>(acc, lane));
}

__device__ __forceinline__ float silu_times(float a, float b) { return a * __fdividef(1.f, 1.f + expf(-a)) * b; }

template <bool I8, int TB>
__device__ __forceinline__ float up_unit(const LayerArgs& a, const Shared& sh, int g, int i, int n, int part, int parts,
                                         int lane) {
  int tok[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) tok[t] = sh.member[g * kGroup + min(t, n - 1)] / a.k;
  const size_t row = ((size_t)sh.group_e[g] * 2 * a.s + i) * a.h, to_b = (size_t)a.s * a.h;
  const uint8_t* w = static_cast<const uint8_t*>(a.W_up);
  if constexpr (I8) return up_int8<TB>(a, w + row, w + row + to_b, tok, part, parts, lane);
  return up_bf16<TB>(a, w + 2 * row, w + 2 * (row + to_b), tok, part, parts, lane);
}

// a and b of selection q of group g for row i: m to scratch.
template <bool I8>
__device__ __forceinline__ void finish_up(const LayerArgs& a, const Shared& sh, int g, int i, int q, float va, float vb) {
  const int slot = sh.member[g * kGroup + q];
  if constexpr (I8) {
    const float* sc = a.up_scale + (size_t)sh.group_e[g] * 2 * a.s + i;
    const float xs = a.x_scale[slot / a.k];
    va = (float)__float_as_int(va) * (xs * sc[0]);
    vb = (float)__float_as_int(vb) * (xs * sc[a.s]);
  }
  a.mid[(size_t)slot * a.s + i] = silu_times(va, vb);
}

template <bool I8, int TB>
__device__ __forceinline__ void up_whole(const LayerArgs& a, const Shared& sh, int g, int i, int n, int lane) {
  const float v = up_unit<I8, TB>(a, sh, g, i, n, 0, 1, lane);
  constexpr int sft = 5 - log2_of<2 * TB>();
  const float o = __shfl_xor_sync(0xffffffffu, v, 1 << sft);
  const int val = lane >> sft, q = val >> 1;
  if ((val & 1) == 0 && (lane & ((1 << sft) - 1)) == 0 && q < n) finish_up<I8>(a, sh, g, i, q, v, o);
}

template <bool I8, int TB>
__device__ __forceinline__ void up_part(const LayerArgs& a, const Shared& sh, int g, int i, int n, int part, int parts,
                                        int lane, float* to) {
  const float v = up_unit<I8, TB>(a, sh, g, i, n, part, parts, lane);
  constexpr int sft = 5 - log2_of<2 * TB>();
  if ((lane & ((1 << sft) - 1)) == 0) to[lane >> sft] = v;
}

#define MORE_BY_COUNT(n, CALL) \
  if (n == 1) {                \
    CALL(1);                   \
  } else if (n == 2) {         \
    CALL(2);                   \
  } else if (n <= 4) {         \
    CALL(4);                   \
  } else {                     \
    CALL(8);                   \
  }

template <bool I8>
__device__ void up_phase(const LayerArgs& a, const Shared& sh, int groups, float (*part)[2 * kGroup]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = groups * a.s;
  const int each = (units + gridDim.x - 1) / gridDim.x;  // rows a CTA
  // warps a row: enough rows for every warp of the machine, or the row in up to 8 parts
  const int parts = each >= 12 ? 1 : each >= 6 ? 2 : each >= 3 ? 4 : 8;
  if (parts == 1) {
    for (int u = blockIdx.x + gridDim.x * warp; u < units; u += gridDim.x * kWarps) {
      const int g = u / a.s, i = u - g * a.s, n = sh.group_n[g];
#define MORE_CALL(TB) up_whole<I8, TB>(a, sh, g, i, n, lane)
      MORE_BY_COUNT(n, MORE_CALL)
#undef MORE_CALL
    }
    return;
  }
  const int per = kWarps / parts;  // rows of a CTA at a time
  for (int j = 0; j < each; j += per) {
    const int mine = j + warp / parts, u = blockIdx.x + gridDim.x * mine;
    if (mine < each && u < units) {
      const int g = u / a.s, i = u - g * a.s, n = sh.group_n[g];
#define MORE_CALL(TB) up_part<I8, TB>(a, sh, g, i, n, warp % parts, parts, lane, part[warp])
      MORE_BY_COUNT(n, MORE_CALL)
#undef MORE_CALL
    }
    __syncthreads();
    if (threadIdx.x < per * kGroup) {
      const int r = threadIdx.x / kGroup, q = threadIdx.x % kGroup, ur = blockIdx.x + gridDim.x * (j + r);
      if (j + r < each && ur < units) {
        const int g = ur / a.s, i = ur - g * a.s;
        if (q < sh.group_n[g]) {
          float va = 0.f, vb = 0.f;
          int ia = 0, ib = 0;
          for (int w = r * parts; w < (r + 1) * parts; ++w) {
            if constexpr (I8) {
              ia += __float_as_int(part[w][2 * q]);
              ib += __float_as_int(part[w][2 * q + 1]);
            } else {
              va += part[w][2 * q];
              vb += part[w][2 * q + 1];
            }
          }
          if constexpr (I8) {
            va = __int_as_float(ia);
            vb = __int_as_float(ib);
          }
          finish_up<I8>(a, sh, g, i, q, va, vb);
        }
      }
    }
    __syncthreads();
  }
}

// Rows r0 + rb * rows + lane / L (rb < kRowBlocks) of expert e for up to TB selections of group g.
template <bool I8, int TB>
__device__ __forceinline__ void down_unit(const LayerArgs& a, const Shared& sh, int g, int n, int o0, int R, int r0,
                                          int L, int lane) {
  const int rows = 32 / L, sub = lane / L, l = lane % L;
  const int e = sh.group_e[g];
  constexpr int kBytes = I8 ? 1 : 2, kVec = 16 / kBytes;
  const uint8_t* w = static_cast<const uint8_t*>(a.W_down) + ((size_t)e * a.h + o0) * a.s * kBytes;
  float acc[TB][kRowBlocks];
  int iacc[TB][kRowBlocks];
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int b = 0; b < kRowBlocks; ++b) {
      acc[t][b] = 0.f;
      iacc[t][b] = 0;
    }
  int slot[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) slot[t] = sh.member[g * kGroup + min(t, n - 1)];
  for (int c = l * kVec; c < a.s; c += L * kVec) {
    uint4 v[kRowBlocks];
#pragma unroll
    for (int b = 0; b < kRowBlocks; ++b) {
      const int r = r0 + b * rows + sub;
      v[b] = r < R ? load_weights(w + ((size_t)r * a.s + c) * kBytes) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const float4* m = reinterpret_cast<const float4*>(a.mid + (size_t)slot[t] * a.s + c);
      if constexpr (I8) {
        const float top = sh.top[slot[t]];
        const float f = top > 0.f ? __fdiv_rn(127.f, top) : 0.f;
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = m[i];
          q[i] = (uint32_t)(__float2int_rn(x.x * f) & 255) | (uint32_t)(__float2int_rn(x.y * f) & 255) << 8 |
                 (uint32_t)(__float2int_rn(x.z * f) & 255) << 16 | (uint32_t)(__float2int_rn(x.w * f) & 255) << 24;
        }
#pragma unroll
        for (int b = 0; b < kRowBlocks; ++b) iacc[t][b] = dot16(v[b], make_uint4(q[0], q[1], q[2], q[3]), iacc[t][b]);
      } else {
        const float4 x0 = m[0], x1 = m[1];
        const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int b = 0; b < kRowBlocks; ++b) dot8(acc[t][b], v[b], x);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    if (t >= n) break;
#pragma unroll
    for (int b = 0; b < kRowBlocks; ++b) {
      const int r = r0 + b * rows + sub;
      float y;
      if constexpr (I8) {
        for (int d = L / 2; d >= 1; d >>= 1) iacc[t][b] += __shfl_xor_sync(0xffffffffu, iacc[t][b], d);
        const float sc = r < R ? a.down_scale[(size_t)e * a.h + o0 + r] : 0.f;
        y = (float)iacc[t][b] * (__fdiv_rn(sh.top[slot[t]], 127.f) * sc);
      } else {
        for (int d = L / 2; d >= 1; d >>= 1) acc[t][b] += __shfl_xor_sync(0xffffffffu, acc[t][b], d);
        y = acc[t][b];
      }
      if (l == 0 && r < R) sh.y[slot[t] * R + r] = y;
    }
  }
}

template <bool I8>
__device__ void down_phase(const LayerArgs& a, const Shared& sh, int groups, int rows_each) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int o0 = blockIdx.x * rows_each, R = min(rows_each, a.h - o0);  // this CTA's output channels
  if (R <= 0) return;
  for (int i = threadIdx.x; i < a.S * R; i += kThreads) sh.y[i] = 0.f;  // selections of no expert stay zero
  if constexpr (I8) {
    for (int i = warp; i < a.S; i += kWarps) {
      float top = 0.f;
      if (sh.expert[i] >= 0)
        for (int c = lane * 4; c < a.s; c += 128) {
          const float4 x = *reinterpret_cast<const float4*>(a.mid + (size_t)i * a.s + c);
          top = fmaxf(fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
        }
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      if (lane == 0) sh.top[i] = top;
    }
  }
  __syncthreads();
  int L = 1;  // lanes a row
  while (L < 32 && L * (I8 ? 16 : 8) < a.s) L <<= 1;
  const int step = kRowBlocks * (32 / L), sets = (R + step - 1) / step;
  for (int u = warp; u < groups * sets; u += kWarps) {
    const int g = u / sets, r0 = (u - g * sets) * step, n = sh.group_n[g];
#define MORE_CALL(TB) down_unit<I8, TB>(a, sh, g, n, o0, R, r0, L, lane)
    MORE_BY_COUNT(n, MORE_CALL)
#undef MORE_CALL
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.N * R; i += kThreads) {
    const int n = i / R, r = i - n * R;
    float sum = 0.f;
    for (int j = 0; j < a.k; ++j) sum = fmaf(sh.gate[n * a.k + j], sh.y[(n * a.k + j) * R + r], sum);
    a.out[(size_t)n * a.h + o0 + r] = __float2bfloat16_rn(sum);
  }
}

constexpr int kSolo = 2;

template <bool I8, int KCAP>
__global__ void __launch_bounds__(kThreads, 1) layer_kernel(const LayerArgs a, int rows_each) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[kWarps][2 * kGroup];
  __shared__ float pv[kWarps][KCAP];
  __shared__ int pe[kWarps][KCAP];
  __shared__ int counts[kWarps];
  __shared__ int failed;
  const Shared sh = shared_at(smem, a.S, rows_each);
  unsigned turn = 0;
  project_tokens(a, part);
  if constexpr (I8) round_tokens(a, &part[0][0]);
  if (!grid_barrier(a.barrier, ++turn, a.status, &failed)) return;
  expert_logits(a);
  if (!grid_barrier(a.barrier, ++turn, a.status, &failed)) return;
  const bool solo = a.N <= kSolo;
  if (solo) {
    for (int n = 0; n < a.N; ++n) select_experts<KCAP>(a, n, pv, pe, sh.expert, sh.gate);
  } else {
    for (int n = blockIdx.x; n < a.N; n += gridDim.x) select_experts<KCAP>(a, n, pv, pe, a.idx, a.gate);
    if (!grid_barrier(a.barrier, ++turn, a.status, &failed)) return;
  }
  const int groups = group_selections(a, sh, solo, counts);
  up_phase<I8>(a, sh, groups, part);
  if (!grid_barrier(a.barrier, ++turn, a.status, &failed)) return;
  down_phase<I8>(a, sh, groups, rows_each);
}

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <bool I8, int KCAP>
cudaError_t launch_layer(const LayerArgs& a, cudaStream_t stream) {
  const int grid = sm_count();
  const int rows_each = (a.h + grid - 1) / grid;
  const uint32_t smem = layer_smem(a.S, rows_each);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> done[64] = {};
  if (dev < 0 || dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(layer_kernel<I8, KCAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // every CTA waits for the others at the barriers
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, layer_kernel<I8, KCAP>, a, rows_each);
}

}  // namespace

// The few-token kernel takes the shape: its shared memory holds the selections' output channels (a CTA's share of h,
// at least 132 CTAs assumed), and a batch of up to kFewTokens tokens.
bool layer_few_fits(int64_t N, int h, int k) {
  return N <= kFewTokens && layer_smem((int)(N * k), (h + 131) / 132) <= kSmemMost - 2048;
}

cudaError_t launch_layer_few(const FewArgs& f) {
  LayerArgs a = {};
  a.X = static_cast<const __nv_bfloat16*>(f.X);
  a.R1 = static_cast<const __nv_bfloat16*>(f.R1);
  a.R2 = static_cast<const __nv_bfloat16*>(f.R2);
  a.z = f.z;
  a.logits = f.logits;
  a.r = f.r;
  a.Xq = f.Xq;
  a.x_scale = f.x_scale;
  a.W_up = f.W_up;
  a.W_down = f.W_down;
  a.up_scale = f.up_scale;
  a.down_scale = f.down_scale;
  a.idx = f.idx;
  a.gate = f.gate;
  a.mid = f.mid;
  a.out = static_cast<__nv_bfloat16*>(f.out);
  a.barrier = f.barrier;
  a.status = f.status;
  a.N = (int)f.N;
  a.h = f.h;
  a.s = f.s;
  a.M = f.M;
  a.k = f.k;
  a.S = (int)(f.N * f.k);
  const cudaError_t e = cudaMemsetAsync(f.barrier, 0, sizeof(unsigned int), f.stream);
  if (e != cudaSuccess) return e;
  if (a.k <= 8) return f.Xq ? launch_layer<true, 8>(a, f.stream) : launch_layer<false, 8>(a, f.stream);
  return f.Xq ? launch_layer<true, 16>(a, f.stream) : launch_layer<false, 16>(a, f.stream);
}

}  // namespace more
