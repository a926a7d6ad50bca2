// The whole layer for a few tokens, in one cooperative kernel.
//
// The time of such a call is the latency of its steps and the reading of the selected experts' weights, once each, so
// every step is spread over all CTAs with a barrier over the grid behind it:
//   1. z = x R1: a CTA takes 16 columns of a token's z, its warps parts of h.  With 8-bit weights other CTAs round x.
//   2. The logits z R2: a warp takes 8 experts of a token, a lane one row of R2 (or r / 32 of them); the N x M logits of
//      these few tokens go through scratch.
//   3. A CTA takes a token's largest k logits and their softmax (for up to kSolo tokens every CTA does so itself, which
//      saves a barrier).  Then every CTA groups the N k selections by expert, up to 8 a group: its own copy.
//   4. Up: a warp takes 8 rows of A_e and the same 8 of B_e for a group's tokens; m = silu(a) * b goes to scratch.
//      Where there are too few rows for the machine's warps, 2 to 16 warps of a CTA share them, each a part of h.
//   5. Down: every CTA owns h / CTAs output channels for all experts, so a token's k contributions meet in its
//      shared memory, and out[n] = sum_j gate * y is summed there in the order of j: no second pass over a row buffer,
//      and no atomics on the result.  Where all N k selections of these channels are more than it holds (N = 64, k = 8:
//      from h = 5477 on), the CTA takes its channels in runs, one after the other.
//
// The products of 4 and 5 are warp MMAs (m16n8k16; k32 for 8 bits) with the weights as the 16 rows of A and a group's
// up to 8 tokens as the columns of B.  The tensor cores are not what a few rows an expert need; their operand layout is:
// one instruction takes 512 bytes of weights, where a thread's own multiply-adds, with their conversions and the
// reductions over lanes, took longer than the reading (N = 64, h = 2048, s = 64: 2.6 TB/s in step 5).  A product's terms may
// come in any order as long as both operands keep to it, so a lane's 16 contiguous bytes of a row serve as its fragments of two
// MMAs without any shuffling.  Weights pass through rings of asynchronous copies, three quarters of each in flight, that run on from one group to the next; copies take 128 or 256 contiguous bytes of a row at a time
// (64 at a time, in the MMA's own order, reached 4.8 TB/s where these reach more).
//
// z is carried as the bf16 pair of the routing kernels, and m as such a pair (about 16 bits), since B is bf16: two MMAs
// where one would round m to 8 bits.  All sums are fp32.  With 8-bit weights sums are whole numbers and m is rounded to
// 8 bits, its row's largest magnitude found after one more barrier.
#include <algorithm>
#include <atomic>

#include "experts_internal.cuh"
#include "sm100_ptx.cuh"
#include "warp_simt.cuh"

namespace more {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 8;  // selections of one expert that share a reading of its weights: the columns of an MMA
constexpr int kRows = 16;  // rows of an MMA
constexpr int64_t kFewTokens = 64;
constexpr int64_t kFewRows = 16;  // tokens up to which the experts alone run here whatever they share
constexpr int64_t kFewSums = 1 << 21;  // N k h up to which more than those do
constexpr int kFewExperts = 16384;  // every CTA reads all the offsets of a dispatch
constexpr int kSolo = 2;         // tokens that every CTA routes for itself
constexpr int kSlots = 4;                   // batches of a warp's ring
constexpr uint32_t kRing = 128 * 1024;      // all warps' rings
constexpr uint32_t kSmemMost = 218 * 1024;  // dynamic: 227 KB less the kernel's static 8.1
constexpr int kCandidates = 512;  // as many as threads: where there is no bound there may be that many logits

struct LayerArgs {
  const __nv_bfloat16 *X, *R1, *R2;
  int8_t* Xq;  // int8: X in 8 bits, and its scales
  float* x_scale;
  const void *W_up, *W_down;
  const float *up_scale, *down_scale;
  const int32_t *offsets, *slots;  // selections that were made and dispatched before the call; null: routed here
  const float* given_gate;
  float* z;       // [N][r]
  float* logits;  // [N][M]
  int32_t* idx;   // [S]
  float* gate;    // [S]
  __nv_bfloat16 *mid_hi, *mid_lo;  // [S][s], m as a bf16 pair
  float* mid;                      // int8: [S][s], and its 8 bits with their scales
  int8_t* mid_q;
  float* mid_scale;
  __nv_bfloat16* out;
  unsigned int* barrier;  // 0 at the start
  unsigned int* status;
  int N, h, r, s, M, k, S;
};

// ---- shared memory ---------------------------------------------------------------------------------------------
struct Shared {
  uint32_t ring;       // shared address of the warps' rings
  uint8_t* work;       // the ring's bytes, for steps that have no copies in flight
  int32_t* expert;     // [S] expert of a selection (-1: none)
  float* gate;         // [S]
  int32_t* group_e;    // [S] expert of a group
  int32_t* group_n;    // [S] its selections
  int16_t* member;     // [S][kGroup] selections of a group
  float* y;            // [S][R], R channels of a CTA at a time
};

__host__ __device__ constexpr uint32_t round16(uint32_t v) { return (v + 15) & ~15u; }

__host__ __device__ constexpr uint32_t layer_smem(int S, int R) {
  return kRing + round16(4 * S) * 4 + round16(2 * kGroup * S) + round16(4 * S * R);
}

__device__ __forceinline__ Shared shared_at(uint8_t* p, int S) {
  Shared r;
  r.ring = sm100::smem_u32(p);
  r.work = p;
  p += kRing;
  r.expert = reinterpret_cast<int32_t*>(p);
  p += round16(4 * S);
  r.gate = reinterpret_cast<float*>(p);
  p += round16(4 * S);
  r.group_e = reinterpret_cast<int32_t*>(p);
  p += round16(4 * S);
  r.group_n = reinterpret_cast<int32_t*>(p);
  p += round16(4 * S);
  r.member = reinterpret_cast<int16_t*>(p);
  p += round16(2 * kGroup * S);
  r.y = reinterpret_cast<float*>(p);
  return r;
}

// ---- small pieces -----------------------------------------------------------------------------------------------
// bf16 pairs as fp32
__device__ __forceinline__ void widen8(uint4 v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// Sums V values over the warp; lane l ends with value l >> (5 - log2 V).
template <int V>
__device__ __forceinline__ float reduce_scatter(float (&v)[V], int lane) {
  int d = 16;
#pragma unroll
  for (int n = V; n > 1; n >>= 1, d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int q = 0; q < n / 2; ++q) {
      const float send = up ? v[q] : v[q + n / 2];
      v[q] = (up ? v[q + n / 2] : v[q]) + __shfl_xor_sync(0xffffffffu, send, d);
    }
  }
#pragma unroll
  for (; d >= 1; d >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
  return v[0];
}

// Floats as keys of the same order.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Barrier number `turn` (from 1) over a cooperative grid; false once the wait has run out.  One release and acquire of
// one thread, which the CTA's own barriers extend to the others.
__device__ bool grid_barrier(unsigned int* counter, unsigned turn, unsigned int* status, int* failed) {
  __syncthreads();
  if (threadIdx.x == 0) {
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
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
  }
  __syncthreads();
  return *failed == 0;
}

// ---- routing ------------------------------------------------------------------------------------------------------
// Step 1.  `part`: 16 sums a warp.
__device__ void project_tokens(const LayerArgs& a, float (*part)[16]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, blocks = a.r / 16;
  for (int u = blockIdx.x; u < a.N * blocks; u += gridDim.x) {
    const int n = u / blocks, b = (u - n * blocks) * 16;
    float v;
    int i;
    warp_partial_z16_strided(a.X + (size_t)n * a.h, a.R1, a.h, a.r, b, threadIdx.x, kThreads, lane, v, i);
    if ((lane & 1) == 0) part[warp][i - b] = v;
    __syncthreads();
    if (threadIdx.x < 16) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += part[w][threadIdx.x];
      a.z[n * a.r + b + threadIdx.x] = split_bf16_pair(sum);
    }
    __syncthreads();
  }
}

// The largest of a CTA's values.
__device__ __forceinline__ float block_max(float v, float* warp_tops) {
  // the float order of magnitudes is their bits' order, a NaN above all
  v = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
  if ((threadIdx.x & 31) == 0) warp_tops[threadIdx.x >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v = top_of(v, warp_tops[w]);
  return v;
}

// x in 8 bits, a token a CTA, from the last CTA down (the first have z to compute).
__device__ void round_tokens(const LayerArgs& a, float* warp_tops) {
  for (int n = gridDim.x - 1 - blockIdx.x; n < a.N; n += gridDim.x) {
    const uint4* src = reinterpret_cast<const uint4*>(a.X + (size_t)n * a.h);
    float top = 0.f, x[8];
    for (int c = threadIdx.x; c < a.h / 8; c += kThreads) {
      widen8(src[c], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = top_of(top, x[i]);
    }
    top = block_max(top, warp_tops);
    const float div = divisor_of(top), inv = __fdiv_rn(127.f, div);
    for (int c = threadIdx.x; c < a.h / 8; c += kThreads) {
      widen8(src[c], x);
      reinterpret_cast<uint2*>(a.Xq + (size_t)n * a.h)[c] =
          make_uint2(round8x4(x[0], x[1], x[2], x[3], div, inv), round8x4(x[4], x[5], x[6], x[7], div, inv));
    }
    if (threadIdx.x == 0) a.x_scale[n] = __fdiv_rn(top, 127.f);
    __syncthreads();
  }
}

// Step 2.  `zs`: N r floats of shared memory.  A warp keeps its octet's weights while it goes through tokens.
__device__ void expert_logits(const LayerArgs& a, float* zs) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < a.N * a.r; i += kThreads) zs[i] = a.z[i];
  __syncthreads();
  const int octets = a.M / 8, mine = (octets - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  // units: an octet's tokens in runs, so that few octets still fill the warps
  const int runs = min(a.N, max(1, kWarps / max(mine, 1))), each = (a.N + runs - 1) / runs;
  for (int u = warp; u < mine * runs; u += kWarps) {
    const int j = u / runs, n0 = (u - j * runs) * each;
    const int e0 = 8 * ((int)blockIdx.x + (int)gridDim.x * j);
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = lane + 32 * i < a.r ? __ldg(reinterpret_cast<const uint4*>(a.R2 + (size_t)(lane + 32 * i) * a.M + e0))
                                 : make_uint4(0, 0, 0, 0);
#pragma unroll 2
    for (int n = n0; n < min(a.N, n0 + each); ++n) {
      float acc[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (32 * i >= a.r) break;
        float x[8];
        widen8(w[i], x);
        const float zi = lane + 32 * i < a.r ? zs[n * a.r + lane + 32 * i] : 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] = fmaf(zi, x[q], acc[q]);
      }
      const float v = reduce_scatter<8>(acc, lane);
      if ((lane & 3) == 0) a.logits[(size_t)n * a.M + e0 + (lane >> 2)] = v;
    }
  }
}

// Step 3 for token n: its selections and gates at idx and gate (shared or global memory).
//   The k-th largest of the 16 warps' largest keys bounds the k-th largest logit from below (fewer warps with logits than k:
//   no bound).  It leaves a handful of candidates, which rank one another in parallel: rounds of a block-wide largest value
//   cost 200 cycles each, 16 of them for k = 8.  More candidates than kCandidates (logits that are all but equal) are
//   thinned by bisection, equal ones by their experts.
struct Select {
  uint32_t key[kCandidates];
  int expert[kCandidates];
  float value[MORE_KMAX];
  uint32_t top[kWarps];
  int count;
};

__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// Logits at or above `bound` (equal ones: of experts below `limit`) as candidates; their number.
__device__ __forceinline__ int collect(const float* l, int M, uint32_t bound, int limit, bool any, Select& s) {
  if (threadIdx.x == 0) s.count = 0;
  __syncthreads();
  if (any) {
#pragma unroll 1
    for (int e = threadIdx.x; e < M; e += kThreads) {
      const float v = l[e];
      const uint32_t key = key_of(v);
      if (v == v && key >= bound && (key > bound || e < limit)) {
        const int at = atomicAdd(&s.count, 1);
        if (at < kCandidates) {
          s.key[at] = key;
          s.expert[at] = e;
        }
      }
    }
  }
  __syncthreads();
  return s.count;
}

// Too many candidates: the k-th largest key by bisection, and of its ties the first experts that make k.
__device__ __noinline__ int collect_exactly(const float* l, int M, int k, uint32_t bound, Select& s) {
  uint32_t lo = bound, hi = 0xffffffffu;
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2 + 1;
    int c = 0;
    for (int e = threadIdx.x; e < M; e += kThreads) {
      const float v = l[e];
      c += v == v && key_of(v) >= mid;
    }
    int total = 0;  // a thread counts as many as it has, up to k
    for (int j = 0; j < k; ++j) total += __syncthreads_count(c > j);
    if (total >= k)
      lo = mid;
    else
      hi = mid - 1;
  }
  int from = 0, to = M;
  while (from < to) {
    const int half = (from + to) / 2;
    int c = 0;
    for (int e = threadIdx.x; e < M; e += kThreads) {
      const float v = l[e];
      const uint32_t key = key_of(v);
      c += v == v && (key > lo || (key == lo && e < half));
    }
    int total = 0;
    for (int j = 0; j < k; ++j) total += __syncthreads_count(c > j);
    if (total >= k)
      to = half;
    else
      from = half + 1;
  }
  return collect(l, M, lo, to, true, s);
}

__device__ void select_experts(const LayerArgs& a, int n, Select& s, int32_t* idx, float* gate) {
  const float* l = a.logits + (size_t)n * a.M;
  const int lane = threadIdx.x & 31;
  uint32_t top = 0;  // below every number's key; a NaN logit is never chosen
#pragma unroll 8
  for (int e = threadIdx.x; e < a.M; e += kThreads) {
    const float v = l[e];
    top = max(top, v == v ? key_of(v) : 0);
  }
  const uint32_t warp_top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) s.top[threadIdx.x >> 5] = warp_top;
  __syncthreads();
  const uint32_t mine = lane < kWarps ? s.top[lane] : 0;
  int rank = 0;
#pragma unroll 4
  for (int w = 0; w < kWarps; ++w) {
    const uint32_t o = s.top[w];
    rank += o > mine || (o == mine && w < lane);
  }
  const unsigned at = __ballot_sync(0xffffffffu, lane < kWarps && rank == a.k - 1);  // k <= 16 warps
  const uint32_t bound = __shfl_sync(0xffffffffu, mine, __ffs(at) - 1);
  int count = collect(l, a.M, bound, 0x7fffffff, top >= bound, s);
  if (count > kCandidates) count = collect_exactly(l, a.M, a.k, bound, s);
  for (int c = threadIdx.x; c < count; c += kThreads) {
    const uint32_t key = s.key[c];
    const int e = s.expert[c];
    int r = 0;
#pragma unroll 4
    for (int o = 0; o < count; ++o) r += s.key[o] > key || (s.key[o] == key && s.expert[o] < e);
    if (r < a.k) {
      s.value[r] = value_of(key);
      idx[n * a.k + r] = e;
    }
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    const bool in = lane < a.k && lane < count;
    const float ex = in ? expf(s.value[lane] - s.value[0]) : 0.f;
    float sum = ex;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffu, sum, d, 16);
    if (lane < a.k) {
      gate[n * a.k + lane] = in ? __fdividef(ex, sum) : 0.f;
      if (!in) idx[n * a.k + lane] = -1;  // fewer than k numbers among the logits
    }
  }
  __syncthreads();
}

// Groups the selections by expert, up to kGroup a group, the same way in every CTA; the number of groups.  A hash table
// in the ring's space holds each expert's selections so far and the lowest of them; experts are numbered in the order
// of those, groups of one expert follow one another.  Up to kGroup selections of an expert take the columns of its one
// group as they come: a selection's sums are the same in every column.
constexpr int kTable = 2048;

__device__ __forceinline__ int place_of(int32_t* keys, int key) {
  int at = (int)(((uint32_t)key * 2654435761u) >> 21);  // 11 bits
  for (int tries = 0; tries < kTable; ++tries) {
    const int old = atomicCAS(&keys[at], -1, key);
    if (old == -1 || old == key) return at;
    at = (at + 1) & (kTable - 1);
  }
  return 0;  // not reached: at most 1024 keys
}

// The selections of a dispatch, into shared memory.  As in the row layout of the grouped products, offsets that fall or lie
// outside [0, S] leave nothing, and a slot outside [0, S) is skipped.
__device__ void read_dispatch(const LayerArgs& a, const Shared& sh) {
  for (int i = threadIdx.x; i < a.S; i += kThreads) {
    sh.expert[i] = -1;
    sh.gate[i] = a.given_gate[i];
  }
  int broken = 0;
#pragma unroll 4
  for (int e = threadIdx.x; e < a.M; e += kThreads) {
    const int b = __ldg(a.offsets + e), c = __ldg(a.offsets + e + 1);
    broken |= b < 0 || c < b || c > a.S;
  }
  const bool none = __syncthreads_or(broken);
  bool bad = none;
  if (!none) {
    for (int e = threadIdx.x; e < a.M; e += kThreads) {
      const int c = __ldg(a.offsets + e + 1);
      for (int i = __ldg(a.offsets + e); i < c; ++i) {
        const int slot = __ldg(a.slots + i);
        if (slot >= 0 && slot < a.S)
          sh.expert[slot] = e;
        else
          bad = true;
      }
    }
  }
  if (bad && blockIdx.x == 0) atomicOr(a.status, MORE_DEVERR_BAD_INPUT);
  __syncthreads();
  for (int i = threadIdx.x; i < a.S; i += kThreads)
    if (sh.expert[i] < 0) sh.gate[i] = 0.f;  // its row is zero, and its gate may be no number
}

// `here`: the selections are in shared memory.
__device__ int group_selections(const LayerArgs& a, const Shared& sh, bool here, int* warp_sums) {
  int32_t* t_expert = reinterpret_cast<int32_t*>(sh.work);
  int32_t* t_count = t_expert + kTable;
  int32_t* t_first = t_count + kTable;
  int32_t* t_base = t_first + kTable;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (a.S <= 32) {  // one warp's lanes find one another
    if (warp == 0) {
      int e = lane < a.S ? (here ? sh.expert[lane] : a.idx[lane]) : -1;
      if (!here && lane < a.S) sh.gate[lane] = a.gate[lane];
      const bool ok = e >= 0 && e < a.M;
      if (!ok && lane < a.S && !a.offsets && blockIdx.x == 0) atomicOr(a.status, MORE_DEVERR_BAD_INPUT);
      if (!ok) e = -1;
      if (lane < a.S) sh.expert[lane] = e;
      const unsigned same = __match_any_sync(0xffffffffu, e);
      const int nth = __popc(same & ((1u << lane) - 1)), count = __popc(same), first = __ffs(same) - 1;
      int sum = ok && nth == 0 ? (count + kGroup - 1) / kGroup : 0;
      const int mine = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      const int g = __shfl_sync(0xffffffffu, sum - mine, first) + nth / kGroup;
      if (ok) {
        sh.member[g * kGroup + nth % kGroup] = (int16_t)lane;
        if (nth % kGroup == 0) {
          sh.group_e[g] = e;
          sh.group_n[g] = min(kGroup, count - nth);
        }
      }
      if (lane == 31) warp_sums[0] = sum;
    }
    __syncthreads();
    return warp_sums[0];
  }
  for (int i = threadIdx.x; i < kTable; i += kThreads) {
    t_expert[i] = -1;
    t_count[i] = 0;
    t_first[i] = 0x7fffffff;
  }
  for (int i = threadIdx.x; i < a.S; i += kThreads) {
    const int e = here ? sh.expert[i] : a.idx[i];
    if (!here) sh.gate[i] = a.gate[i];
    const bool ok = e >= 0 && e < a.M;
    if (!ok && !a.offsets && blockIdx.x == 0) atomicOr(a.status, MORE_DEVERR_BAD_INPUT);
    sh.expert[i] = ok ? e : -1;
  }
  __syncthreads();
  int at[2] = {-1, -1}, nth[2] = {0, 0};  // S <= 2 kThreads
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = threadIdx.x + q * kThreads, e = i < a.S ? sh.expert[i] : -1;
    if (e < 0) continue;
    at[q] = place_of(t_expert, e);
    nth[q] = atomicAdd(&t_count[at[q]], 1);
    atomicMin(&t_first[at[q]], i);
  }
  __syncthreads();
  int groups = 0;
#pragma unroll 1
  for (int q = 0; q < 2 && q * kThreads < a.S; ++q) {
    const int i = threadIdx.x + q * kThreads;
    const bool leads = at[q] >= 0 && t_first[at[q]] == i;
    const int mine = leads ? (t_count[at[q]] + kGroup - 1) / kGroup : 0;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    if (lane == 31) warp_sums[warp] = sum;
    __syncthreads();
    int base = groups;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int o = warp_sums[w];
      base += w < warp ? o : 0;
      groups += o;
    }
    if (leads) t_base[at[q]] = base + sum - mine;
    __syncthreads();
  }
#pragma unroll 1
  for (int q = 0; q < 2; ++q) {
    if (at[q] < 0) continue;
    const int i = threadIdx.x + q * kThreads, count = t_count[at[q]];
    if (count > kGroup) {  // which group a selection is in has to be the same everywhere
      nth[q] = 0;
      for (int o = 0; o < i; ++o) nth[q] += sh.expert[o] == sh.expert[i];
    }
    const int g = t_base[at[q]] + nth[q] / kGroup;
    sh.member[g * kGroup + nth[q] % kGroup] = (int16_t)i;
    if (nth[q] % kGroup == 0) {
      sh.group_e[g] = sh.expert[i];
      sh.group_n[g] = min(kGroup, count - nth[q]);
    }
  }
  __syncthreads();
  return groups;
}

// ---- products -----------------------------------------------------------------------------------------------------
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <bool I8>
struct Sums {
  float v[4];
};
template <>
struct Sums<true> {
  int v[4];
};

__device__ __forceinline__ void mma(Sums<false>& c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c.v[0]), "+f"(c.v[1]), "+f"(c.v[2]), "+f"(c.v[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(Sums<true>& c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+r"(c.v[0]), "+r"(c.v[1]), "+r"(c.v[2]), "+r"(c.v[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 64 bytes of K: rows lane / 4 and lane / 4 + 8 of the weights, column lane / 4 of the other operand, bytes
// 16 (lane % 4) on of each.
template <bool I8>
__device__ __forceinline__ void step_products(Sums<I8>& c, uint4 w0, uint4 w1, uint4 x) {
  mma(c, w0.x, w1.x, w0.y, w1.y, x.x, x.y);
  mma(c, w0.z, w1.z, w0.w, w1.w, x.z, x.w);
}

// A warp's ring of batches: 16 rows x BS steps of 64 bytes, fetched kSlots - 1 batches ahead.  A row's 16-byte pieces lie
// together, those of odd rows with their halves of 64 bytes swapped: eight lanes of two rows then read all 32 banks.
template <int BS>
struct Ring {
  static constexpr int kStreams = 32 / BS;      // warps: 16 with batches of 2 KB, 8 with batches of 4 KB
  static constexpr uint32_t kBatch = 64 * BS;   // bytes of a row
  static constexpr uint32_t kBytes = kSlots * 16 * kBatch;
  static_assert(kStreams * kBytes == kRing && kStreams <= kWarps, "rings");
  static constexpr int kPieces = 4 * BS;       // lanes a row
  static constexpr int kAtOnce = 32 / kPieces;  // rows a copy instruction
  uint32_t base;
  int in = 0, out = 0;
  __device__ __forceinline__ uint32_t fill() {
    const uint32_t at = base + in * 16 * kBatch;
    in = (in + 1) & (kSlots - 1);
    return at;
  }
  // The oldest batch, landed and seen by every lane; the batch before it may be overwritten from here on.
  __device__ __forceinline__ uint32_t drain() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory");
    __syncwarp();
    const uint32_t at = base + out * 16 * kBatch;
    out = (out + 1) & (kSlots - 1);
    return at;
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // Where piece p of row r is.
  static __device__ __forceinline__ uint32_t place(int r, int p) { return r * kBatch + ((p ^ ((r & 1) << 2)) << 4); }
};

__device__ __forceinline__ float silu_times(float a, float b) { return a * __fdividef(1.f, 1.f + expf(-a)) * b; }

// m of rows i of group g's selections 2 (lane % 4) and the next, from a (sums 0 and 1) and b (2 and 3).
template <bool I8>
__device__ __forceinline__ void finish_up(const LayerArgs& a, const Shared& sh, int g, int i, int lane,
                                          const Sums<I8>& c) {
  const int n = sh.group_n[g];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int col = 2 * (lane & 3) + q;
    if (col >= n) continue;
    const int slot = sh.member[g * kGroup + col];
    float va, vb;
    if constexpr (I8) {
      const float* sc = a.up_scale + (size_t)sh.group_e[g] * 2 * a.s + i;
      const float xs = a.x_scale[slot / a.k];
      va = (float)c.v[q] * (xs * sc[0]);
      vb = (float)c.v[q + 2] * (xs * sc[a.s]);
    } else {
      va = c.v[q];
      vb = c.v[q + 2];
    }
    const float m = silu_times(va, vb);
    const size_t at = (size_t)slot * a.s + i;
    if constexpr (I8) {
      a.mid[at] = m;
    } else {
      const __nv_bfloat16 hi = __float2bfloat16_rn(m);
      a.mid_hi[at] = hi;
      const float rest = m - __bfloat162float(hi);
      a.mid_lo[at] = __float2bfloat16_rn(fabsf(rest) < INFINITY ? rest : 0.f);  // an infinite m is all in its first half
    }
  }
}

// Step 4.  Unit u: rows 8 (u % (s / 8)) on of group u / (s / 8).  `parts` warps a unit, each a run of its batches.
constexpr int kUpStreams = Ring<4>::kStreams;

template <bool I8>
__device__ void up_phase(const LayerArgs& a, const Shared& sh, int groups, Sums<I8> (*red)[kUpStreams][32]) {
  constexpr int BS = 4;
  using R = Ring<BS>;
  constexpr int kStreams = R::kStreams;
  constexpr int kBytes = I8 ? 1 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int eights = a.s / 8, units = groups * eights;
  const int pitch = a.h * kBytes, batches = (pitch + (int)R::kBatch - 1) / (int)R::kBatch;
  // The fewest batches a warp, a round's end counted as half a one: rounds of all warps' units, shorter with more parts.
  int parts = 1, best = 0x7fffffff;
  for (int p = 1; p <= kStreams; p *= 2) {
    const int per_round = (int)gridDim.x * (kStreams / p), rounds = (units + per_round - 1) / per_round;
    const int cost = rounds * (2 * ((batches + p - 1) / p) + (p > 1 ? 1 : 0));
    if (cost < best) {
      best = cost;
      parts = p;
    }
  }
  const int each = kStreams / parts, stride = (int)gridDim.x * each, first = (int)blockIdx.x * each;
  const bool streams = warp < kStreams;
  const int part = warp % parts, b0 = batches * part / parts, b1 = streams ? batches * (part + 1) / parts : b0;
  R ring{sh.ring + (uint32_t)warp * R::kBytes};
  // copies: this lane's piece and its rows
  const int pc = lane % R::kPieces, r0 = lane / R::kPieces;
  const uint32_t dst = R::place(r0, pc);  // kAtOnce is even: the lane's rows are all odd or all even
  const size_t to_b = (size_t)(a.s - 8) * pitch;
  int fu = first + warp / parts, fb = b0;
  const uint8_t* from = nullptr;
  auto locate = [&]() {
    if (fu >= units) return;
    const int g = fu / eights;
    from = static_cast<const uint8_t*>(a.W_up) +
           ((size_t)sh.group_e[g] * 2 * a.s + (fu - g * eights) * 8 + r0) * pitch + pc * 16;
  };
  locate();
  auto fetch = [&]() {
    const uint32_t at = ring.fill() + dst;
    if (b0 < b1 && fu < units) {
      const int off = fb * (int)R::kBatch;
      if (off + pc * 16 < pitch) {
#pragma unroll
        for (int i = 0; i < 16 / R::kAtOnce; ++i)
          copy16(at + i * R::kAtOnce * R::kBatch,
                 from + off + (size_t)i * R::kAtOnce * pitch + (i * R::kAtOnce >= 8 ? to_b : 0));
      }
      if (++fb == b1) {
        fb = b0;
        fu += stride;
        locate();
      }
    }
    R::commit();
  };
  if (streams) {
#pragma unroll 1
    for (int i = 0; i < kSlots - 1; ++i) fetch();
  }
  // products: this lane's row and 16 bytes of each step
  const int row = lane >> 2, piece = (lane & 3) * 16;
  const uint8_t* X = I8 ? reinterpret_cast<const uint8_t*>(a.Xq) : reinterpret_cast<const uint8_t*>(a.X);
  auto token_at = [&](int u) {
    const int g = u / eights;
    return X + (size_t)(sh.member[g * kGroup + min(row, sh.group_n[g] - 1)] / a.k) * pitch + piece;
  };
  uint4 x[BS], ahead[BS];
  auto load_x = [&](const uint8_t* p, int b, uint4 (&to)[BS]) {
#pragma unroll
    for (int j = 0; j < BS; ++j) {
      const int off = b * (int)R::kBatch + 64 * j;
      to[j] = off + piece < pitch ? *reinterpret_cast<const uint4*>(p + off) : make_uint4(0, 0, 0, 0);
    }
  };
  int parity = 0;
  const uint8_t* p = nullptr;
  if (first + warp / parts < units && b0 < b1) {
    p = token_at(first + warp / parts);
    load_x(p, b0, ahead);
  }
#pragma unroll 1
  for (int u0 = first; u0 < units; u0 += stride) {
    const int u = u0 + warp / parts;
    Sums<I8> c = {};
    if (streams && u < units) {
#pragma unroll 1
      for (int b = b0; b < b1; ++b) {
#pragma unroll
        for (int j = 0; j < BS; ++j) x[j] = ahead[j];
        if (b + 1 < b1) {
          load_x(p, b + 1, ahead);
        } else if (u + stride < units) {
          p = token_at(u + stride);
          load_x(p, b0, ahead);
        }
        const uint32_t at = ring.drain() + row * R::kBatch;
        fetch();
#pragma unroll
        for (int j = 0; j < BS; ++j) {
          const uint32_t q = (uint32_t)(piece + 64 * j) ^ ((row & 1) << 6);
          const bool in = b * (int)R::kBatch + 64 * j + piece < pitch;
          uint4 w0 = sm100::ld_shared_v4(at + q), w1 = sm100::ld_shared_v4(at + 8 * R::kBatch + q);
          if (!in) w0 = w1 = make_uint4(0, 0, 0, 0);
          step_products<I8>(c, w0, w1, x[j]);
        }
      }
      if (parts == 1) {
        const int g = u / eights;
        finish_up<I8>(a, sh, g, (u - g * eights) * 8 + row, lane, c);
      }
    }
    if (parts > 1) {
      if (streams) red[parity][warp][lane] = c;
      __syncthreads();
      const int ur = u0 + warp;  // warp w sums unit w of the round
      if (warp < each && ur < units) {
        Sums<I8> t = red[parity][warp * parts][lane];
        for (int q = 1; q < parts; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) t.v[v] += red[parity][warp * parts + q][lane].v[v];
        const int g = ur / eights;
        finish_up<I8>(a, sh, g, (ur - g * eights) * 8 + row, lane, t);
      }
      parity ^= 1;
    }
  }
}

// The middle rows in 8 bits: a selection a CTA.
__device__ void round_middles(const LayerArgs& a, const Shared& sh, float* warp_tops) {
  for (int i = blockIdx.x; i < a.S; i += gridDim.x) {
    if (sh.expert[i] < 0) continue;
    const float4* src = reinterpret_cast<const float4*>(a.mid + (size_t)i * a.s);
    float top = 0.f;
    for (int c = threadIdx.x; c < a.s / 4; c += kThreads) {
      const float4 f = src[c];
      top = top_of(top_of(top_of(top_of(top, f.x), f.y), f.z), f.w);
    }
    top = block_max(top, warp_tops);
    const float div = divisor_of(top), inv = __fdiv_rn(127.f, div);
    for (int c = threadIdx.x; c < a.s / 4; c += kThreads) {
      const float4 f = src[c];
      reinterpret_cast<uint32_t*>(a.mid_q + (size_t)i * a.s)[c] = round8x4(f.x, f.y, f.z, f.w, div, inv);
    }
    if (threadIdx.x == 0) a.mid_scale[i] = __fdiv_rn(top, 127.f);
    __syncthreads();
  }
}

// Step 5 for a run of this CTA's channels.  Unit u: rows 16 (u % tiles) on of the run for group u / tiles.  The first
// batches' copies start before the barrier: they need the groups alone.
template <bool I8, int BS>
struct Down {
  using R = Ring<BS>;
  static constexpr int kBytes = I8 ? 1 : 2;
  const LayerArgs& a;
  const Shared& sh;
  int groups, o0, rows, tiles, units, batches, pitch, lane, warp, pc, r0;
  R ring;
  int fu, fb, left = 0;
  const uint8_t* from;

  __device__ __forceinline__ int group_of(int u) const { return tiles == 1 ? u : u / tiles; }
  __device__ Down(const LayerArgs& a_, const Shared& sh_, int groups_) : a(a_), sh(sh_), groups(groups_) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    pitch = a.s * kBytes;
    batches = (pitch + (int)R::kBatch - 1) / (int)R::kBatch;
    pc = lane % R::kPieces;
    r0 = lane / R::kPieces;
    ring.base = sh.ring + (uint32_t)warp * R::kBytes;
  }
  __device__ __forceinline__ void locate() {
    if (fu >= units) return;
    const int g = group_of(fu), r = (fu - g * tiles) * kRows + r0;
    left = rows - r;
    from = static_cast<const uint8_t*>(a.W_down) + ((size_t)sh.group_e[g] * a.h + o0 + r) * pitch + pc * 16;
  }
  __device__ __forceinline__ void fetch() {
    const uint32_t at = ring.fill() + R::place(r0, pc);
    if (fu < units) {
      const int off = fb * (int)R::kBatch;
      if (off + pc * 16 < pitch) {
#pragma unroll
        for (int i = 0; i < 16 / R::kAtOnce; ++i)
          if (i * R::kAtOnce < left)
            copy16(at + i * R::kAtOnce * R::kBatch, from + off + (size_t)i * R::kAtOnce * pitch);
      }
      if (++fb == batches) {
        fb = 0;
        fu += R::kStreams;
        locate();
      }
    }
    R::commit();
  }
  // The channels [from_row, to_row); whatever was copied for the last ones has been used.
  __device__ void start(int from_row, int to_row) {
    o0 = from_row;
    rows = max(0, to_row - from_row);
    tiles = (rows + kRows - 1) / kRows;
    units = warp < R::kStreams ? groups * tiles : 0;
    ring.in = ring.out = 0;
    fu = warp;
    fb = 0;
    locate();
    if (warp < R::kStreams) {
#pragma unroll 1
      for (int i = 0; i < kSlots - 1; ++i) fetch();
    }
    for (int i = threadIdx.x; i < a.S * rows; i += kThreads) sh.y[i] = 0.f;  // selections of no expert stay zero
  }
  __device__ __forceinline__ size_t middle_of(int u) const {
    const int g = group_of(u);
    return (size_t)sh.member[g * kGroup + min(lane >> 2, sh.group_n[g] - 1)] * pitch + (lane & 3) * 16;
  }
  __device__ __forceinline__ void load(size_t at, int b, uint4 (&hi)[BS], uint4 (&lo)[BS]) const {
#pragma unroll
    for (int j = 0; j < BS; ++j) {
      const int off = b * (int)R::kBatch + 64 * j;
      hi[j] = lo[j] = make_uint4(0, 0, 0, 0);
      if (off + (lane & 3) * 16 < pitch) {
        if constexpr (I8) {
          hi[j] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(a.mid_q) + at + off);
        } else {
          hi[j] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(a.mid_hi) + at + off);
          lo[j] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(a.mid_lo) + at + off);
        }
      }
    }
  }
  __device__ void run() {
    const int row = lane >> 2, piece = (lane & 3) * 16;
    uint4 hi[BS], lo[BS], next_hi[BS], next_lo[BS];
    size_t mid = 0;
    if (warp < units) {
      mid = middle_of(warp);
      load(mid, 0, next_hi, next_lo);
    }
#pragma unroll 1
    for (int u = warp; u < units; u += R::kStreams) {
      const int g = group_of(u), r = (u - g * tiles) * kRows + row, n = sh.group_n[g];
      Sums<I8> c = {};
#pragma unroll 1
      for (int b = 0; b < batches; ++b) {
#pragma unroll
        for (int j = 0; j < BS; ++j) {
          hi[j] = next_hi[j];
          lo[j] = next_lo[j];
        }
        if (b + 1 < batches) {
          load(mid, b + 1, next_hi, next_lo);
        } else if (u + R::kStreams < units) {
          mid = middle_of(u + R::kStreams);
          load(mid, 0, next_hi, next_lo);
        }
        const uint32_t at = ring.drain() + row * R::kBatch;
        fetch();
        const bool tail = (b + 1) * (int)R::kBatch > pitch;
#pragma unroll
        for (int j = 0; j < BS; ++j) {
          const uint32_t q = (uint32_t)(piece + 64 * j) ^ ((row & 1) << 6);
          // bytes behind a row's end multiply zeros and have to be numbers; rows behind the last only spoil themselves
          const bool in = !tail || b * (int)R::kBatch + 64 * j + piece < pitch;
          uint4 w0 = sm100::ld_shared_v4(at + q), w1 = sm100::ld_shared_v4(at + 8 * R::kBatch + q);
          if (!in) w0 = w1 = make_uint4(0, 0, 0, 0);
          step_products<I8>(c, w0, w1, hi[j]);
          if constexpr (!I8) step_products<I8>(c, w0, w1, lo[j]);
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = 2 * (lane & 3) + (q & 1), rr = r + (q >> 1) * 8;
        if (col >= n || rr >= rows) continue;
        const int slot = sh.member[g * kGroup + col];
        float y;
        if constexpr (I8)
          y = (float)c.v[q] * (a.mid_scale[slot] * a.down_scale[(size_t)sh.group_e[g] * a.h + o0 + rr]);
        else
          y = c.v[q];
        sh.y[slot * rows + rr] = y;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.N * rows; i += kThreads) {
      const int n = i / rows, r = i - n * rows;
      float sum = 0.f;
      for (int j = 0; j < a.k; ++j) sum = fmaf(sh.gate[n * a.k + j], sh.y[(n * a.k + j) * rows + r], sum);
      a.out[(size_t)n * a.h + o0 + r] = __float2bfloat16_rn(sum);
    }
  }
};

// `rows_each` channels a CTA, `rows_once` of them at a time.
template <bool I8, int BS>
__device__ __forceinline__ void down_phase(const LayerArgs& a, const Shared& sh, int groups, int rows_each,
                                           int rows_once, unsigned turn, int* failed) {
  __syncthreads();  // other warps' rings of the first product lie in this one's
  int row = (int)blockIdx.x * rows_each;
  const int end = min(a.h, row + rows_each);
  Down<I8, BS> down(a, sh, groups);
  down.start(row, min(end, row + rows_once));
  if (!grid_barrier(a.barrier, turn, a.status, failed)) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  for (;;) {
    down.run();
    row += rows_once;
    if (row >= end) break;
    __syncthreads();  // sh.y has been summed
    down.start(row, min(end, row + rows_once));
    __syncthreads();  // and is zero
  }
}

template <bool I8>
__global__ void __launch_bounds__(kThreads, 1) layer_kernel(const __grid_constant__ LayerArgs a, int rows_each,
                                                              int rows_once) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ union {
    float part[kWarps][16];
    Select select;
    Sums<I8> red[2][kUpStreams][32];
    float tops[kWarps];
  } u;
  __shared__ int warp_sums[kWarps];
  __shared__ int failed;
  const Shared sh = shared_at(smem, a.S);
  unsigned turn = 0;
  if constexpr (I8) round_tokens(a, u.tops);
  bool here = true;
  if (a.offsets) {
    read_dispatch(a, sh);
    if (I8 && !grid_barrier(a.barrier, ++turn, a.status, &failed)) return;
  } else {
    project_tokens(a, u.part);
    if (!grid_barrier(a.barrier, ++turn, a.status, &failed)) return;
    expert_logits(a, reinterpret_cast<float*>(sh.work));
    if (!grid_barrier(a.barrier, ++turn, a.status, &failed)) return;
    here = a.N <= kSolo;
    for (int n = here ? 0 : blockIdx.x; n < a.N; n += here ? 1 : gridDim.x)
      select_experts(a, n, u.select, here ? sh.expert : a.idx, here ? sh.gate : a.gate);
    if (!here && !grid_barrier(a.barrier, ++turn, a.status, &failed)) return;
  }
  const int groups = group_selections(a, sh, here, warp_sums);
  up_phase<I8>(a, sh, groups, u.red);
  if constexpr (I8) {
    if (!grid_barrier(a.barrier, ++turn, a.status, &failed)) return;
    round_middles(a, sh, u.tops);
  }
  // rows of up to 128 bytes fill the ring in batches of two steps, longer ones in batches of four
  if (a.s * (I8 ? 1 : 2) <= 128)
    down_phase<I8, 2>(a, sh, groups, rows_each, rows_once, ++turn, &failed);
  else
    down_phase<I8, 4>(a, sh, groups, rows_each, rows_once, ++turn, &failed);
}

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <bool I8>
cudaError_t launch_layer(const LayerArgs& a, cudaStream_t stream) {
  const int grid = sm_count();
  // a CTA's share of the channels, in as few runs as their sums' place allows: never less than 14 channels for 1024 selections
  const int rows_each = (a.h + grid - 1) / grid, most = (int)((kSmemMost - layer_smem(a.S, 0)) / (4 * (uint32_t)a.S));
  const int runs = (rows_each + most - 1) / most, rows_once = (rows_each + runs - 1) / runs;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> done[64] = {};
  if (dev < 0 || dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(layer_kernel<I8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = layer_smem(a.S, rows_once);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // every CTA waits for the others at the barriers
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, layer_kernel<I8>, a, rows_each, rows_once);
}

}  // namespace

// The few-token kernel takes up to kFewTokens tokens.  The layer gains by it up to there: it saves the
// router's launches too (N = 64: h = 2048, s = 64, M = 4096, k = 8: 98 us against 139; 1024, 256, 128, 4: 67 against
// 81; h = 4096, s = 64, M = 512, k = 8: 129 against 155; 7168, 64, 512, 8: 217 against 243, in 8 bits 200 against 247).
// It keeps the sizes where reading more than about a GB of weights at 4 to 5 TB/s costs more than the launches (2048,
// 1024, 64, 4: 186 against 177; 5120, 128, 512, 8: 293 against 249; 7168, 256, 256, 8: 497 against 430): what is rounded
// then depends on neither h nor the experts' sizes.
// The experts alone gain while the selections seldom share an expert, whose weights this kernel then reads at 4 TB/s in
// one launch, and the grouped products at 5.8 after five launches.  us, few against grouped:
//   2048, 64, 4096, 8:   N = 8: 25, 39    N = 64: 87, 94        2048, 1024, 64, 4:  N = 16: 107, 108    N = 32: 137, 122
//   512, 64, 1024, 4:    N = 8: 18, 26    N = 64: 31, 30        1024, 256, 128, 4:  N = 32: 49, 48      N = 64: 59, 51
//   4096, 64, 512, 8:    N = 40: 94, 104  N = 64: 117, 118      4096, 128, 512, 8:  N = 40: 170, 143    N = 64: 216, 174
// Beyond N k h = kFewSums the sums would be taken in runs of channels, and they lose: 5120, 128, 512, 8, N = 64: 280, 211;
// 7168, 256, 256, 4, N = 64: 347, 292 (and with narrow rows gain little: 7168, 64, 512, 8, N = 64: 203, 198).
bool experts_few_fits(int64_t N, int h, int M, int k) {
  return N > 0 && M <= kFewExperts && layer_few_fits(N) && (N <= kFewRows || (N * k <= M && N * k * h <= kFewSums));
}

bool layer_few_fits(int64_t N) { return N <= kFewTokens; }
static_assert(kSmemMost >= layer_smem(kFewTokens * MORE_KMAX, 14), "room for a run of channels");

cudaError_t launch_layer_few(const FewArgs& f) {
  LayerArgs a = {};
  a.X = static_cast<const __nv_bfloat16*>(f.X);
  a.R1 = static_cast<const __nv_bfloat16*>(f.R1);
  a.R2 = static_cast<const __nv_bfloat16*>(f.R2);
  a.Xq = f.Xq;
  a.x_scale = f.x_scale;
  a.W_up = f.W_up;
  a.W_down = f.W_down;
  a.up_scale = f.up_scale;
  a.down_scale = f.down_scale;
  a.offsets = f.offsets;
  a.slots = f.slots;
  a.given_gate = f.given_gate;
  a.z = f.z;
  a.logits = f.logits;
  a.idx = f.idx;
  a.gate = f.gate;
  a.mid_hi = f.mid_pair;
  a.mid_lo = f.mid_pair + f.N * f.k * f.s;
  a.mid = f.mid;
  a.mid_q = f.mid_q;
  a.mid_scale = f.mid_scale;
  a.out = static_cast<__nv_bfloat16*>(f.out);
  a.barrier = f.barrier;
  a.status = f.status;
  a.N = (int)f.N;
  a.h = f.h;
  a.r = f.r;
  a.s = f.s;
  a.M = f.M;
  a.k = f.k;
  a.S = (int)(f.N * f.k);
  const cudaError_t e = cudaMemsetAsync(f.barrier, 0, sizeof(unsigned int), f.stream);
  if (e != cudaSuccess) return e;
  return f.Xq ? launch_layer<true>(a, f.stream) : launch_layer<false>(a, f.stream);
}

}  // namespace more
