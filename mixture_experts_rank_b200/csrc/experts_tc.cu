// The experts' matrix products on the tensor cores, grouped by expert.
//
// With x_t the row of token t, (A; B) = W_up[e] and D = W_down[e]:
//   up        H = silu(x A^T) * (x B^T)                     rows gathered from X by token
//   down      Y = gate * H D^T                              rows of H
//   backward  with a = x A^T, b = x B^T, G = y_bar D (rows of y_bar gathered by token), m = silu(a) * b:
//             the gate's gradient sum(G * m), gate * m, and the gradients of a and b,
//             gate * G * b * silu'(a) and gate * G * silu(a)
//   dx        [da, db] W_up[e]                              rows of [da, db]
//   dw up     [da, db]^T x                                  contracted over the expert's rows
//   dw down   y_bar^T (gate * m)
// and up8 / down8, the first two with 8-bit operands and the scales of rows and columns in the epilogue.
//
// A CTA holds 128 rows of one expert (128 output channels for the weights' gradients) on the TMEM lanes and up
// to 256 columns:
//   warp 0       TMA: stages of 128 bytes of K (64 values of 16 bits, 128 of 8), 128B-swizzled;
//   warps 2, 3, 12, 13  asynchronous copies of the rows that are picked by token;
//   warp 1       tcgen05 MMAs into two accumulators in TMEM, so a tile's epilogue runs under the next one's products;
//   warps 4-11   epilogue, two warps a lane group.
// The grid is persistent; tiles come from the row layout that the same call made on the device.
// H and [da, db] are rounded to bf16: they are MMA operands.  Y and the rows of dx are rounded to bf16 before the
// sum over a token's slots, which halves the traffic that bounds these kernels; the sum itself is in fp32.  With the
// result's own rounding that is 0.0029 in the 2-norm, one rounding fewer 0.0024.  To save one costs (prefill of 16384 tokens,
// h = 2048, s = 64, M = 4096, and of 262144, h = 512: 900 and 922 us): H as a bf16 pair 963 and 1019 us; rows as fp16 with a
// power of two for every 64 columns, 11 bits at the same traffic, 1045 and 1045 us, since the epilogue then binds.
#include <cudaTypedefs.h>

#include <atomic>

#include "experts_internal.cuh"
#include "mbar_wait.cuh"
#include "sm100_ptx.cuh"

namespace more {
namespace experts {

using namespace sm100;

enum Mode { kUp, kDown, kUp8, kDown8, kBack, kDx, kDwUp, kDwDown };

constexpr int kEpiWarps = 8;
constexpr int kGatherWarps = 4;
constexpr uint32_t kABytes = kTileRows * 128;  // 16 KB: 128 rows (or 2 boxes of 64 channels x 64 rows) of a stage
constexpr uint32_t kBox = 64 * 128;            // 8 KB: a box of 64 rows x 128 bytes
constexpr uint32_t kStageOut = 32 * 128;       // a warp's staging: 32 rows x 64 bf16 columns
constexpr int kScales = 128;  // column scales that a warp needs of a tile
constexpr int kMaxStages = 6;
constexpr int kRun = 1024;  // of K, between additions in registers

template <int MODE, int HALF, bool PAIR>
struct Shape {
  static constexpr bool kEight = MODE == kUp8 || MODE == kDown8;
  static constexpr bool kIsUp = MODE == kUp || MODE == kUp8;
  static constexpr bool kIsDown = MODE == kDown || MODE == kDown8;
  static constexpr bool kIsDw = MODE == kDwUp || MODE == kDwDown;
  static constexpr bool kGathers = !PAIR && (kIsUp || kIsDw || MODE == kBack);  // one operand is picked by token
  static constexpr int kThreads = kGathers ? 14 * 32 : 12 * 32;
  static constexpr int kRows = PAIR ? 2 * kTileRows : kTileRows;  // rows (or channels) of a tile
  static constexpr bool kStaged = kIsDown || MODE == kDx || kIsDw;  // epilogue goes through shared memory
  // The tensor cores cut sums off, they do not round them: a sum over K comes out too small by about 1e-9 K of itself, and
  // the gate's gradient, which is fp32 to the end, by three times that.  Tiles of 3 x 64 columns therefore take their
  // products in runs of kRun, added in registers; 3 x 128 columns are more than the registers hold.  Runs of 1024 leave
  // 2.9e-6 in the 2-norm.  Runs of 256 would leave 7e-7, as sums in fp32 do, but their reads of the accumulators bind:
  // backward at h = 512, s = 64 312 to 326 us, at h = 2048, s = 64 286 to 326 us, at h = 4096, s = 1024 963 to 1224 us.
  static constexpr bool kRuns = MODE == kBack && HALF == 64;
  // columns of one accumulator, and its place in TMEM
  static constexpr int kCols = kIsUp ? 2 * HALF : MODE == kBack ? 3 * HALF : 256;
  static constexpr int kAccStride = kCols <= 128 ? 128 : 256;
  static constexpr int kAccs = kCols > 256 ? 1 : 2;
  static constexpr uint32_t kTmemCols = kCols > 256 ? 512 : 2 * kAccStride;
  static constexpr int kBN = kIsUp || MODE == kBack ? HALF : 256;  // output columns of a tile
  static constexpr uint32_t kBBytes = PAIR ? 128 * 128 : kIsUp || MODE == kBack ? 2 * HALF * 128 : 256 * 128;
  static constexpr uint32_t kStage = kABytes + kBBytes;
  static constexpr int kStages = MODE == kDown8 ? (PAIR ? 5 : 3) : kStage > 32 * 1024 ? 4 : 6;
  static constexpr int kKBlock = kEight ? 128 : 64;
  static constexpr int kKStep = kEight ? 32 : 16;
  static constexpr uint32_t kOffOut = kStages * kStage;
  static constexpr uint32_t kOffScale = kOffOut + (kStaged ? kEpiWarps * kStageOut : 0);
  static constexpr uint32_t kOffTop = kOffScale + (kEight ? kEpiWarps * kScales * 4 : 0);
  static constexpr uint32_t kOffBar = kOffTop + (MODE == kUp8 ? 2 * 256 * 4 : 0);
  static constexpr uint32_t kSmem = kOffBar + (2 * kMaxStages + 4 + 1 + 4) * 8 + 16 + 1024;
};

struct Params {
  Rows rows;
  int64_t R;      // rows of the row buffers (a column of `part`)
  int nc;         // tiles along the columns
  int nm;         // tiles along the channels (weights' gradients)
  int items;      // weights' gradients: M * nm * nc
  int k1, k2;     // contracted lengths (k2: the second product of kBack)
  int s, h;
  int cols;       // output columns
  const void* X;        // the rows picked by token, and kBack's second set
  const void* out_bar;
  float* out_scale;  // kUp8 with an expert's whole middle in a tile: the rows' scales
  void* out;      // kUp: H; kUp8: H in fp32, or in 8 bits with out_scale; kDown, kDx: rows of h; kBack: [da, db]
  __nv_bfloat16* out2;  // kBack: gate * m
  float* part;          // kBack: the gate's gradient, a partial sum per HALF / 2 columns
  const float* row_scale;  // 8 bits: the rows' scales
  const float* col_scale;
  unsigned int* status;
};

struct Bars {
  uint64_t *full, *empty, *acc_full, *acc_empty, *drain;
  uint64_t* halves;  // [4] the two epilogue warps of a lane group
  uint32_t* tmem_slot;
  int* abort_flag;
};

__device__ __forceinline__ Bars bars_at(uint8_t* p) {
  uint64_t* b = reinterpret_cast<uint64_t*>(p);
  Bars r;
  r.full = b;
  r.empty = b + kMaxStages;
  r.acc_full = b + 2 * kMaxStages;
  r.acc_empty = r.acc_full + 2;
  r.drain = r.acc_empty + 2;
  r.halves = r.drain + 1;
  r.tmem_slot = reinterpret_cast<uint32_t*>(r.halves + 4);
  r.abort_flag = reinterpret_cast<int*>(r.tmem_slot + 1);
  return r;
}

// One tile: rows [row, row + n) of an expert are slots, [row + n, row + padded) padding.
struct Work {
  int expert, row, n, padded;
  int m0, c0;  // first channel (weights' gradients) and column
};

template <bool DW>
__device__ __forceinline__ int work_items(const Params& p) {
  return DW ? p.items : *p.rows.n_tiles * p.nc;
}

template <bool DW>
__device__ __forceinline__ Work work_at(const Params& p, int w, int bn, int rows) {
  Work k;
  if (DW) {
    const int e = w / (p.nm * p.nc), rest = w - e * (p.nm * p.nc);
    k.expert = e;
    k.row = p.rows.row_start[e];
    k.n = k.padded = p.rows.row_start[e + 1] - k.row;
    k.m0 = rest / p.nc * rows;
    k.c0 = rest % p.nc * bn;
  } else {
    const int t = w / p.nc;
    const int4 v = p.rows.tiles[t];
    k.expert = v.x;
    k.row = v.y;
    k.n = v.z;
    k.padded = v.w;
    k.m0 = 0;
    k.c0 = (w - t * p.nc) * bn;
  }
  return k;
}

// This CTA's tiles in turn.  The next tile's entry is fetched a tile ahead: its latency (two dependent reads with the
// rows' own) is that of a whole tile of a short product.
template <class S, bool PAIR>
struct Cursor {
  int w, items;
  Work cur, nxt;
  static __device__ __forceinline__ int first() { return PAIR ? blockIdx.x >> 1 : blockIdx.x; }
  static __device__ __forceinline__ int stride() { return PAIR ? gridDim.x >> 1 : gridDim.x; }
  __device__ __forceinline__ Cursor(const Params& p) {
    items = work_items<S::kIsDw>(p);
    w = first();
    cur = nxt = Work{};
    if (w < items) cur = work_at<S::kIsDw>(p, w, S::kBN, S::kRows);
    fetch(p);
  }
  __device__ __forceinline__ void fetch(const Params& p) {
    if (w + stride() < items) nxt = work_at<S::kIsDw>(p, w + stride(), S::kBN, S::kRows);
  }
  __device__ __forceinline__ bool done() const { return w >= items; }
  __device__ __forceinline__ bool more() const { return w + stride() < items; }
  __device__ __forceinline__ void next(const Params& p) {
    w += stride();
    cur = nxt;
    fetch(p);
  }
};

// ---- loads -----------------------------------------------------------------------------------------------------
// Warp 0 issues the operands that come as boxes; kGatherWarps warps copy the rows that are picked by token, 16 bytes a
// lane, four rows of 128 bytes an instruction, placed as the 128B swizzle places them.  (Gathered TMA loads move no more
// than 3.4 TB/s over the machine however many warps issue them; these copies are not bound by their issue.)
// Every one of these warps waits for every stage and arrives on it.
struct Ring {
  RingPos pos;
  uint32_t issued = 0;
  template <class S>
  __device__ __forceinline__ void next() {
    pos.next(S::kStages);
    ++issued;
  }
};

// The wait for a free stage polls first: the hardware wakes a suspended thread so late that the loads fall behind (first
// product at h = 2048, s = 64: 448 us with suspended waits, 388 us so; polling in the MMA thread's waits as well: 393 us).
__device__ __forceinline__ bool poll_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned int* status) {
  for (int i = 0; i < 4000; ++i)
    if (mbar_test_wait(bar, parity)) return true;
  return bounded_wait(bar, parity, abort_flag, status);
}

// A warp's wait: its lanes go on together or, once the wait has run out for one of them, give up together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Bars& b, unsigned int* status) {
  return __all_sync(0xffffffffu, bounded_wait(bar, parity, b.abort_flag, status));
}
__device__ __forceinline__ bool warp_poll(uint64_t* bar, uint32_t parity, const Bars& b, unsigned int* status) {
  return __all_sync(0xffffffffu, poll_wait(bar, parity, b.abort_flag, status));
}

template <class S>
__device__ __forceinline__ bool wait_empty(const Ring& r, const Bars& b, int lane, unsigned int* status) {
  int ok = 1;
  if (lane == 0) ok = poll_wait(&b.empty[r.pos.i], r.pos.phase ^ 1u, b.abort_flag, status);
  return __shfl_sync(0xffffffffu, ok, 0);
}

// Box loads still in flight when the CTA gives up must land before its shared memory is another's.
template <class S, bool PAIR>
__device__ __noinline__ void settle(const Ring& r, const Bars& b) {
  if constexpr (PAIR) {  // the loads complete on CTA 0's barriers: a millisecond is hundreds of times what they take
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {
    }
  } else {
    for (int i = 0; i < S::kStages; ++i) {
      const uint32_t fills = (r.issued + S::kStages - 1 - i) / S::kStages;
      if (fills == 0) continue;
      const uint64_t t0 = global_timer_ns();
      while (!mbar_test_wait(&b.full[i], (fills - 1) & 1u) && global_timer_ns() - t0 < 1000000000ull) {
      }
    }
  }
}

// This CTA's part of a pair's stage: its 128 rows (or channels) of A, its half of B's columns.
template <int MODE, int HALF>
__device__ __forceinline__ void pair_stage(const Params& p, uint64_t* bar, uint8_t* st, const Work& k, int x, int rank,
                                           const CUtensorMap* m0, const CUtensorMap* m1, const CUtensorMap* m2,
                                           const CUtensorMap* m3) {
  using S = Shape<MODE, HALF, true>;
  uint8_t* bm = st + kABytes;
  const int row = k.row + rank * kTileRows;
  const int round1 = (p.k1 + 63) / 64 * 64;
  if (rank == 0) mbar_arrive_expect_tx(bar, MODE == kBack && x >= round1 ? 2 * (kABytes + kBox) : 2 * S::kStage);
  if constexpr (S::kIsDw) {
    for (int i = 0; i < 2; ++i) {
      tma_load_2d_pair(st + i * kBox, m0, bar, k.m0 + rank * 128 + 64 * i, k.row + x);
      tma_load_2d_pair(bm + i * kBox, m1, bar, k.c0 + rank * 128 + 64 * i, k.row + x);
    }
  } else if constexpr (MODE == kDx) {
    tma_load_2d_pair(st, m0, bar, x, row);
    for (int i = 0; i < 2; ++i)
      tma_load_3d_pair(bm + i * kBox, m1, bar, k.c0 + rank * 128 + 64 * i, x, k.expert);
  } else if constexpr (S::kIsDown) {
    tma_load_2d_pair(st, m0, bar, x, row);
    tma_load_3d_pair(bm, m1, bar, x, k.c0 + rank * 128, k.expert);
  } else if (MODE != kBack || x < round1) {
    tma_load_2d_pair(st, m0, bar, x, row);
    tma_load_3d_pair(bm, m1, bar, x, k.c0 + rank * p.s, k.expert);  // A_e's rows in CTA 0, B_e's in CTA 1
  } else {
    tma_load_2d_pair(st, m2, bar, x - round1, row);
    tma_load_3d_pair(bm, m3, bar, k.c0 + rank * 64, x - round1, k.expert);
  }
}

template <int MODE, int HALF, bool PAIR>
__device__ void box_loads(const Params& p, const Bars& b, uint8_t* smem, const CUtensorMap* m0, const CUtensorMap* m1,
                          const CUtensorMap* m2, const CUtensorMap* m3, int rank) {
  using S = Shape<MODE, HALF, PAIR>;
  const int lane = threadIdx.x & 31;
  Ring r;
  for (Cursor<S, PAIR> at(p); !at.done(); at.next(p)) {
    const Work k = at.cur;
    const int len = S::kIsDw ? k.padded : p.k1 + (MODE == kBack ? (p.k1 + 63) / 64 * 64 - p.k1 + p.k2 : 0);
    for (int x = 0; x < len; x += S::kKBlock) {
      if (!wait_empty<S>(r, b, lane, p.status)) return settle<S, PAIR>(r, b);
      if (lane == 0) {
        uint64_t* bar = &b.full[r.pos.i];
        uint8_t* st = smem + r.pos.i * S::kStage;
        if constexpr (PAIR) {
          pair_stage<MODE, HALF>(p, bar, st, k, x, rank, m0, m1, m2, m3);
        } else if constexpr (MODE == kDwUp) {
          mbar_arrive_expect_tx(bar, 2 * kBox);
          tma_load_2d(st, m0, bar, k.m0, k.row + x);
          tma_load_2d(st + kBox, m0, bar, k.m0 + 64, k.row + x);
        } else if constexpr (MODE == kDwDown) {
          const int boxes = min(4, (p.cols - k.c0 + 63) / 64);
          mbar_arrive_expect_tx(bar, boxes * kBox);
          for (int i = 0; i < boxes; ++i) tma_load_2d(st + kABytes + i * kBox, m1, bar, k.c0 + 64 * i, k.row + x);
        } else if constexpr (S::kIsUp || MODE == kBack) {
          if (x < p.k1) {
            mbar_arrive_expect_tx(bar, 2 * HALF * 128);
            tma_load_3d(st + kABytes, m1, bar, x, k.c0, k.expert);
            tma_load_3d(st + kABytes + HALF * 128, m1, bar, x, k.c0 + p.s, k.expert);
          } else {
            mbar_arrive_expect_tx(bar, HALF / 64 * kBox);
            for (int i = 0; i < HALF / 64; ++i)
              tma_load_3d(st + kABytes + i * kBox, m3, bar, k.c0 + 64 * i, x - (p.k1 + 63) / 64 * 64, k.expert);
          }
        } else {
          mbar_arrive_expect_tx(bar, S::kStage);
          tma_load_2d(st, m0, bar, x, k.row);
          if constexpr (MODE == kDx) {
            for (int i = 0; i < 4; ++i) tma_load_3d(st + kABytes + i * kBox, m1, bar, k.c0 + 64 * i, x, k.expert);
          } else {
            tma_load_3d(st + kABytes, m1, bar, x, k.c0, k.expert);
          }
        }
      }
      __syncwarp();
      r.next<S>();
    }
  }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

// This lane's arrival on a stage, made once its copies so far have landed.  The copies are generic-proxy writes: the
// MMA thread orders its own reads behind them with a proxy fence after its wait.  (The same fence on this side waits
// for every copy in flight and leaves one stage of them at a time: the 8-bit first product took 331 instead of 203 us.)
__device__ __forceinline__ void arrive_landed(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int MODE, int HALF, bool PAIR>
__device__ void row_copies(const Params& p, const Bars& b, uint8_t* smem, int turn) {
  using S = Shape<MODE, HALF, PAIR>;
  const int lane = threadIdx.x & 31, sub = lane >> 3, piece = lane & 7;
  const size_t pitch = (size_t)p.h * (S::kEight ? 1 : 2);
  const uint32_t st0 = smem_u32(smem);
  Ring c;
  int tok[8] = {};
  for (Cursor<S, PAIR> at(p); !at.done(); at.next(p)) {
    const Work k = at.cur;
    if constexpr (S::kIsDw) {
      // stages of 64 rows; boxes of 64 columns: two of y_bar as A, four of x as B
      constexpr int kBoxes = MODE == kDwUp ? 4 : 2;
      const uint8_t* src = static_cast<const uint8_t*>(MODE == kDwUp ? p.X : p.out_bar);
      const int col = MODE == kDwUp ? k.c0 : k.m0;
      const int32_t* tokens = p.rows.row_token + k.row + sub;
#pragma unroll
      for (int i = 0; i < 4; ++i) tok[i] = 4 * (turn + 4 * i) < k.padded ? tokens[4 * (turn + 4 * i)] : 0;
      for (int r0 = 0; r0 < k.padded; r0 += 64) {
        int next[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = r0 + 64 + 4 * (turn + 4 * i);
          next[i] = q < k.padded ? tokens[q] : 0;
        }
        if (!wait_empty<S>(c, b, lane, p.status)) return wait_copies();
        const uint32_t st = st0 + c.pos.i * S::kStage + (MODE == kDwUp ? kABytes : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 4 * (turn + 4 * i) + sub;
          if (r0 + row >= k.padded) continue;
          const uint32_t dst = st + row * 128 + ((piece ^ (row & 7)) << 4);
          const uint8_t* from = src + (size_t)max(tok[i], 0) * pitch;
          const bool slot = tok[i] >= 0;
#pragma unroll
          for (int x = 0; x < kBoxes; ++x) {
            const int cc = col + 64 * x + piece * 8;
            const bool ok = cc < p.h;
            copy16(dst + x * kBox, from + (ok ? 2 * cc : 0), ok && slot);
          }
        }
        arrive_landed(&b.full[c.pos.i]);
        c.next<S>();
#pragma unroll
        for (int i = 0; i < 4; ++i) tok[i] = next[i];
      }
    } else {
      const uint8_t* row[8];
      const uint8_t* X = static_cast<const uint8_t*>(p.X);
      if (at.w == at.first()) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * (turn + 4 * i) + sub;
          tok[i] = r < k.padded ? any_token(p.rows.row_token[k.row + r]) : 0;
        }
      }
      int ahead[8];  // the next tile's tokens
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * (turn + 4 * i) + sub;
        ahead[i] = at.more() && r < at.nxt.padded ? any_token(p.rows.row_token[at.nxt.row + r]) : 0;
        row[i] = X + tok[i] * pitch + piece * 16;
      }
      const int r0 = 4 * turn + sub;  // a lane's rows are 16 apart: the same place in the swizzle
      const uint32_t dst = r0 * 128 + ((piece ^ (r0 & 7)) << 4);
      const int passes = MODE == kBack ? 2 : 1;
      for (int pass = 0; pass < passes; ++pass) {
        if (pass == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            row[i] = static_cast<const uint8_t*>(p.out_bar) + tok[i] * pitch + piece * 16;
        }
        for (int x = 0; x < (int)pitch; x += 128) {
          if (!wait_empty<S>(c, b, lane, p.status)) return wait_copies();
          const uint32_t st = st0 + c.pos.i * S::kStage;
          const bool ok = x + piece * 16 < (int)pitch;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (4 * (turn + 4 * i) < k.padded)
              copy16(st + dst + i * 2048, row[i] + (ok ? x : 0) - (ok ? 0 : piece * 16), ok);
          arrive_landed(&b.full[c.pos.i]);
          c.next<S>();
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) tok[i] = ahead[i];
    }
  }
  wait_copies();
}

// ---- MMA issuer: one thread --------------------------------------------------------------------------------------
// The products of one stage, `steps` MMAs of K = 16 (or 32 bytes).  A step's operands lie 32 bytes on (K-major) or two
// groups of eight rows on (MN-major), so its descriptors are the stage's plus a constant: one thread issues everything,
// and it should not build each descriptor afresh.
template <bool EIGHT, bool A_MN, bool B_MN, int MAX, bool PAIR>
__device__ __forceinline__ void stage_products(uint32_t acc, uint64_t a, uint64_t b, uint32_t idesc, int steps,
                                               bool first) {
  constexpr uint64_t kA = A_MN ? 2048 >> 4 : 32 >> 4, kB = B_MN ? 2048 >> 4 : 32 >> 4;
#pragma unroll
  for (int i = 0; i < MAX; ++i) {
    if (i > 0 && i >= steps) break;
    const uint32_t add = i > 0 || !first;
    if constexpr (EIGHT && PAIR)
      mma_i8_pair(acc, a + i * kA, b + i * kB, idesc, add);
    else if constexpr (EIGHT)
      mma_i8(acc, a + i * kA, b + i * kB, idesc, add);
    else if constexpr (PAIR)
      mma_bf16_pair(acc, a + i * kA, b + i * kB, idesc, add);
    else
      mma_bf16(acc, a + i * kA, b + i * kB, idesc, add);
  }
}

// The MMAs so far are done: tell this CTA's barrier, or both CTAs' of a pair.
template <bool PAIR>
__device__ __forceinline__ void done_with(uint64_t* bar) {
  if constexpr (PAIR)
    mma_commit_pair(bar, 3);
  else
    mma_commit(bar);
}

template <int MODE, int HALF, bool PAIR>
__device__ void mma_role(const Params& p, const Bars& b, uint8_t* smem, uint32_t tmem) {
  using S = Shape<MODE, HALF, PAIR>;
  constexpr int kMax = S::kKBlock / S::kKStep;
  constexpr bool kAMn = S::kIsDw, kBMn = S::kIsDw || MODE == kDx;
  RingPos s, d;
  const uint32_t st0 = smem_u32(smem);
  const uint64_t a0 = smem_desc(st0, kAMn ? kBox : 16, 1024, kSwizzle128B);
  const uint64_t b0 = smem_desc(st0 + kABytes, kBMn ? kBox : 16, 1024, kSwizzle128B);
  for (Cursor<S, PAIR> at(p); !at.done(); at.next(p)) {
    const Work k = at.cur;
    if (S::kIsDw && k.padded == 0) continue;  // the epilogue writes zeros
    const int len1 = S::kIsDw ? k.padded : p.k1;
    // columns of this tile's product: all, or up to the last of the weights' gradient, whole MMA steps
    const int n = MODE == kDwDown && !PAIR ? min(256, (p.cols - k.c0 + 15) & ~15) : S::kIsUp || MODE == kBack ? 2 * HALF : 256;
    const uint32_t idesc = S::kEight ? idesc_s8_s32(S::kRows, n) : idesc_bf16_f32(S::kRows, n, kAMn, kBMn);
    uint32_t acc = 0;
    for (int x = 0; x < len1; x += S::kKBlock) {
      const bool first = S::kRuns ? x % kRun == 0 : x == 0;
      if (first) {
        if (!bounded_wait(&b.acc_empty[d.i], d.phase ^ 1u, b.abort_flag, p.status)) goto done;
        tc_fence_after();
        acc = tmem + d.i * S::kAccStride;
      }
      if (!bounded_wait(&b.full[s.i], s.phase, b.abort_flag, p.status)) goto done;
      if constexpr (S::kGathers) fence_proxy_async_smem();
      tc_fence_after();
      const uint64_t off = (uint32_t)s.i * (S::kStage >> 4);
      stage_products<S::kEight, kAMn, kBMn, kMax, PAIR>(acc, a0 + off, b0 + off, idesc,
                                                        (len1 - x + S::kKStep - 1) / S::kKStep, first);
      done_with<PAIR>(&b.empty[s.i]);
      s.next(S::kStages);
      if (S::kRuns && ((x + S::kKBlock) % kRun == 0 || x + S::kKBlock >= len1)) {
        done_with<PAIR>(&b.acc_full[d.i]);
        d.next(S::kAccs);
      }
    }
    if constexpr (MODE == kBack) {
      const uint64_t b1 = smem_desc(st0 + kABytes, kBox, 1024, kSwizzle128B);
      for (int x = 0; x < p.k2; x += S::kKBlock) {
        const bool first = S::kRuns ? x % kRun == 0 : x == 0;
        if (S::kRuns && first) {
          if (!bounded_wait(&b.acc_empty[d.i], d.phase ^ 1u, b.abort_flag, p.status)) goto done;
          tc_fence_after();
          acc = tmem + d.i * S::kAccStride;
        }
        if (!bounded_wait(&b.full[s.i], s.phase, b.abort_flag, p.status)) goto done;
        if constexpr (S::kGathers) fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t off = (uint32_t)s.i * (S::kStage >> 4);
        stage_products<false, false, true, kMax, PAIR>(acc + 2 * HALF, a0 + off, b1 + off,
                                                       idesc_bf16_f32(S::kRows, HALF, 0, 1),
                                                       (p.k2 - x + S::kKStep - 1) / S::kKStep, first);
        done_with<PAIR>(&b.empty[s.i]);
        s.next(S::kStages);
        if (S::kRuns && ((x + S::kKBlock) % kRun == 0 || x + S::kKBlock >= p.k2)) {
          done_with<PAIR>(&b.acc_full[d.i]);
          d.next(S::kAccs);
        }
      }
    }
    if constexpr (!S::kRuns) {
      done_with<PAIR>(&b.acc_full[d.i]);
      d.next(S::kAccs);
    }
  }
done:
  if constexpr (PAIR)
    mma_commit_pair(b.drain, 1);
  else
    mma_commit(b.drain);
  bounded_wait(b.drain, 0, b.abort_flag, p.status);
}

// ---- epilogue ------------------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// int32 to fp32, in place.  `small`: every |v| < 2^22, where the value drops into a float's mantissa with full-rate
// instructions; conversions run at an eighth of that rate, and a second product of 64 values a row is one MMA step of
// work for 256 columns of conversions.
template <int N>
__device__ __forceinline__ void from_int(uint32_t* v, bool small) {
  if (small) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __float_as_uint(__uint_as_float(v[i] + 0x4b400000u) - 12582912.f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __float_as_uint((float)(int)v[i]);
  }
}

__device__ __forceinline__ float sigmoid(float a) { return __fdividef(1.f, 1.f + expf(-a)); }

// Scale i of those at shared address a, four to a read; i counts up through a group of them in an unrolled loop.
__device__ __forceinline__ float scale_at(uint32_t a, int i, float4& four) {
  if ((i & 3) == 0) {
    const uint4 v = ld_shared_v4(a + i * 4);
    four = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
  }
  return (i & 3) == 0 ? four.x : (i & 3) == 1 ? four.y : (i & 3) == 2 ? four.z : four.w;
}

// What a thread needs of a tile beside the accumulator: its row's factor and slot, the columns' scales.
template <int MODE, int HALF, bool PAIR>
struct Info {
  static constexpr int kOwn = MODE == kUp8 ? HALF / 2 : 64;  // columns of a part: A's and B's, or the two chunks'
  static constexpr int kScaleRegs = Shape<MODE, HALF, PAIR>::kEight ? 2 * kOwn / 32 : 0;
  float factor = 1.f, factor2 = 1.f;  // multiplied when they are used: here that would wait for them
  int slot = -1;
  float scale[kScaleRegs ? kScaleRegs : 1];
};

template <int MODE, int HALF, bool PAIR>
__device__ __forceinline__ Info<MODE, HALF, PAIR> row_info(const Params& p, const Work& k, int t, int lane, int hh) {
  using S = Shape<MODE, HALF, PAIR>;
  using I = Info<MODE, HALF, PAIR>;
  I r;
  if constexpr (!S::kIsDw) {
    const bool in = t < k.padded;
    const int row = k.row + t;
    if constexpr (S::kIsDown || MODE == kBack) r.factor = in ? p.rows.row_gate[row] : 0.f;
    if constexpr (MODE == kDown8) r.factor2 = t < k.n ? p.row_scale[row] : 0.f;
    if constexpr (MODE == kUp8) r.factor = in ? p.row_scale[row] : 0.f;
    if constexpr (MODE == kBack) r.slot = in ? p.rows.row_slot[row] : -1;
  }
#pragma unroll
  for (int i = 0; i < I::kScaleRegs; ++i) {
    const int part = (32 * i + lane) / I::kOwn, x = (32 * i + lane) % I::kOwn;
    const int col = MODE == kUp8 ? k.c0 + hh * I::kOwn + x : k.c0 + hh * 64 + part * 128 + x;
    r.scale[i] = col < p.cols ? p.col_scale[MODE == kUp8 ? (size_t)(2 * k.expert + part) * p.s + col
                                                         : (size_t)k.expert * p.cols + col]
                              : 0.f;
  }
  return r;
}

// A warp is done with an accumulator: the MMA thread (of CTA 0) waits for all of them.
template <bool PAIR>
__device__ __forceinline__ void release(uint64_t* bar) {
  if constexpr (PAIR)
    mbar_arrive_leader(bar);
  else
    mbar_arrive(bar);
}

// The part of a tile that this CTA of a pair holds.
template <bool DW>
__device__ __forceinline__ Work part_of(Work k, int rank) {
  if (DW) {
    k.m0 += rank * kTileRows;
  } else {
    k.row += rank * kTileRows;
    k.n = max(0, min(kTileRows, k.n - rank * kTileRows));
    k.padded = max(0, min(kTileRows, k.padded - rank * kTileRows));
  }
  return k;
}

template <int MODE, int HALF, bool PAIR>
__device__ void epilogue(const Params& p, const Bars& b, uint8_t* smem, uint32_t tmem, const CUtensorMap* m_out,
                         int rank) {
  using S = Shape<MODE, HALF, PAIR>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sp = warp & 3, hh = (warp - 4) >> 2;
  const int t = sp * 32 + lane;  // this thread's row of the tile
  const uint32_t lanes = (uint32_t)(sp * 32) << 16;
  const uint32_t scales = smem_u32(smem + S::kOffScale) + (warp - 4) * kScales * 4;
  const uint32_t stage = smem_u32(smem + S::kOffOut) + (warp - 4) * kStageOut;
  RingPos d;
  Info<MODE, HALF, PAIR> info;
  const uint32_t tops = smem_u32(smem + S::kOffTop);  // two tiles' [2][128] largest magnitudes
  int parity = 0;
  const bool small = p.k1 <= (1 << 22) / (128 * 128);
  for (Cursor<S, PAIR> at(p); !at.done(); at.next(p)) {
    const Work k = PAIR ? part_of<S::kIsDw>(at.cur, rank) : at.cur;
    const bool empty = S::kIsDw && k.padded == 0;
    const int row = k.row + t;
    if (at.w == at.first()) info = row_info<MODE, HALF, PAIR>(p, k, t, lane, hh);
    const float row_factor = info.factor * info.factor2;
    const int slot = info.slot;
    if constexpr (S::kEight) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < Info<MODE, HALF, PAIR>::kScaleRegs; ++i) st_shared_f32(scales + (32 * i + lane) * 4, info.scale[i]);
      __syncwarp();
    }
    if (at.more()) info = row_info<MODE, HALF, PAIR>(p, PAIR ? part_of<S::kIsDw>(at.nxt, rank) : at.nxt, t, lane, hh);  // used a tile from now
    if (!empty && !S::kRuns) {
      if (!warp_wait(&b.acc_full[d.i], d.phase, b, p.status)) break;
      tc_fence_after();
    }
    const uint32_t acc = tmem + lanes + d.i * S::kAccStride;
    if (!S::kIsDw && !S::kRuns && sp * 32 >= k.padded) {  // none of this warp's rows is in the tile
      __syncwarp();
      if (lane == 0) release<PAIR>(&b.acc_empty[d.i]);
      d.next(S::kAccs);
      continue;
    }

    if (MODE == kUp8 && HALF == 64 && p.out_scale) {
      // the expert's whole middle is in this tile, half of a row in each of two threads: round it to 8 bits here
      uint32_t va[32], vb[32];
      tmem_ld_x32(acc + hh * 32, va);
      tmem_ld_x32(acc + HALF + hh * 32, vb);
      tmem_wait_ld();
      reg_fence<32>(va);
      reg_fence<32>(vb);
      from_int<32>(va, small);
      from_int<32>(vb, small);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) release<PAIR>(&b.acc_empty[d.i]);
      float top = 0.f;
      float4 sa, sb;
      const int width = min(32, p.s - hh * 32);  // of this half: 32, 16 or none
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float a = __uint_as_float(va[i]) * (row_factor * scale_at(scales, i, sa));
        const float u = __uint_as_float(vb[i]) * (row_factor * scale_at(scales + HALF / 2 * 4, i, sb));
        const float m = a * sigmoid(a) * u;
        va[i] = __float_as_uint(m);
        if (i < width) top = top_of(top, m);
      }
      st_shared_f32(tops + (parity * 256 + hh * 128 + t) * 4, top);
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.halves[sp]);  // not a named barrier: the other warp may have given up
      if (!warp_poll(&b.halves[sp], parity, b, p.status)) break;
      top = top_of(top, ld_shared_f32(tops + (parity * 256 + (hh ^ 1) * 128 + t) * 4));
      parity ^= 1;
      if (t < k.n) {
        const float div = divisor_of(top), inv = __fdiv_rn(127.f, div);
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
          if (i >= width) break;
          uint32_t o[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t* m = va + i + 4 * q;
            o[q] = round8x4(__uint_as_float(m[0]), __uint_as_float(m[1]), __uint_as_float(m[2]), __uint_as_float(m[3]), div,
                            inv);
          }
          *reinterpret_cast<uint4*>(static_cast<int8_t*>(p.out) + (size_t)row * p.s + hh * 32 + i) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (hh == 0) p.out_scale[row] = __fdiv_rn(top, 127.f);
      }
    } else if constexpr (S::kIsUp) {
#pragma unroll
      for (int c = 0; c < HALF / 2; c += 32) {
        const int col = hh * (HALF / 2) + c;
        uint32_t va[32], vb[32];
        tmem_ld_x32(acc + col, va);
        tmem_ld_x32(acc + HALF + col, vb);
        tmem_wait_ld();
        reg_fence<32>(va);
        reg_fence<32>(vb);
        if constexpr (S::kEight) {
          from_int<32>(va, small);
          from_int<32>(vb, small);
        }
        if (c + 32 >= HALF / 2) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) release<PAIR>(&b.acc_empty[d.i]);
        }
        const int g0 = k.c0 + col;
#pragma unroll
        for (int q = 0; q < 32; q += 8) {
          if (g0 + q >= p.s || t >= k.n) continue;
          float m[8];
          float4 sa, sb;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float a, u;
            if constexpr (S::kEight) {
              a = __uint_as_float(va[q + i]) * (row_factor * scale_at(scales + (c + q) * 4, i, sa));
              u = __uint_as_float(vb[q + i]) * (row_factor * scale_at(scales + (HALF / 2 + c + q) * 4, i, sb));
            } else {
              a = __uint_as_float(va[q + i]);
              u = __uint_as_float(vb[q + i]);
            }
            m[i] = a * sigmoid(a) * u;
          }
          if constexpr (S::kEight) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + (size_t)row * p.s + g0 + q);
            o[0] = make_float4(m[0], m[1], m[2], m[3]);
            o[1] = make_float4(m[4], m[5], m[6], m[7]);
          } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)row * p.s + g0 + q) =
                make_uint4(pack2(m[0], m[1]), pack2(m[2], m[3]), pack2(m[4], m[5]), pack2(m[6], m[7]));
          }
        }
      }
    } else if constexpr (MODE == kBack) {
      float dot = 0.f;
      float run_a[S::kRuns ? 32 : 1], run_b[S::kRuns ? 32 : 1], run_g[S::kRuns ? 32 : 1];
      if constexpr (S::kRuns) {
#pragma unroll
        for (int i = 0; i < 32; ++i) run_a[i] = run_b[i] = run_g[i] = 0.f;
        const int runs = (p.k1 + kRun - 1) / kRun;
        bool ok = true;
#pragma unroll 1
        for (int r = 0; r < 2 * runs; ++r) {
          if (!warp_wait(&b.acc_full[d.i], d.phase, b, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (sp * 32 < k.padded) {
            const uint32_t from = tmem + lanes + d.i * S::kAccStride + hh * 32;
            uint32_t v[32];
            if (r < runs) {
              tmem_ld_x32(from, v);
              tmem_wait_ld();
              reg_fence<32>(v);
#pragma unroll
              for (int i = 0; i < 32; ++i) run_a[i] += __uint_as_float(v[i]);
              tmem_ld_x32(from + HALF, v);
              tmem_wait_ld();
              reg_fence<32>(v);
#pragma unroll
              for (int i = 0; i < 32; ++i) run_b[i] += __uint_as_float(v[i]);
            } else {
              tmem_ld_x32(from + 2 * HALF, v);
              tmem_wait_ld();
              reg_fence<32>(v);
#pragma unroll
              for (int i = 0; i < 32; ++i) run_g[i] += __uint_as_float(v[i]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) release<PAIR>(&b.acc_empty[d.i]);
          d.next(S::kAccs);
        }
        if (!ok) break;
      }
#pragma unroll 1
      for (int c = 0; c < HALF / 2; c += 32) {
        const int col = hh * (HALF / 2) + c;
        uint32_t va[32], vb[32], vg[32];
        if constexpr (S::kRuns) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            va[i] = __float_as_uint(run_a[i]);
            vb[i] = __float_as_uint(run_b[i]);
            vg[i] = __float_as_uint(run_g[i]);
          }
        } else {
          tmem_ld_x32(acc + col, va);
          tmem_ld_x32(acc + HALF + col, vb);
          tmem_ld_x32(acc + 2 * HALF + col, vg);
          tmem_wait_ld();
          reg_fence<32>(va);
          reg_fence<32>(vb);
          reg_fence<32>(vg);
          if (c + 32 >= HALF / 2) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) release<PAIR>(&b.acc_empty[d.i]);
          }
        }
        const int g0 = k.c0 + col;
        if (t >= k.padded) continue;
        __nv_bfloat16* pre = static_cast<__nv_bfloat16*>(p.out) + (size_t)row * 2 * p.s + g0;
        __nv_bfloat16* mid = p.out2 + (size_t)row * p.s + g0;
#pragma unroll
        for (int q = 0; q < 32; q += 8) {
          if (g0 + q >= p.s) continue;
          float da[8], db[8], gm[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = __uint_as_float(va[q + i]), u = __uint_as_float(vb[q + i]);
            const float g = __uint_as_float(vg[q + i]), sg = sigmoid(a);
            const float m = a * sg * u, gg = row_factor * g;
            dot = fmaf(g, m, dot);
            // a row that is no slot contributes zeros to every gradient, whatever its token's values
            da[i] = slot >= 0 ? gg * u * sg * (1.f + a * (1.f - sg)) : 0.f;
            db[i] = slot >= 0 ? gg * a * sg : 0.f;
            gm[i] = slot >= 0 ? row_factor * m : 0.f;
          }
          *reinterpret_cast<uint4*>(pre + q) =
              make_uint4(pack2(da[0], da[1]), pack2(da[2], da[3]), pack2(da[4], da[5]), pack2(da[6], da[7]));
          *reinterpret_cast<uint4*>(pre + p.s + q) =
              make_uint4(pack2(db[0], db[1]), pack2(db[2], db[3]), pack2(db[4], db[5]), pack2(db[6], db[7]));
          *reinterpret_cast<uint4*>(mid + q) =
              make_uint4(pack2(gm[0], gm[1]), pack2(gm[2], gm[3]), pack2(gm[4], gm[5]), pack2(gm[6], gm[7]));
        }
      }
      if (t < k.padded) p.part[(size_t)(k.c0 / (HALF / 2) + hh) * p.R + row] = dot;
    } else {
      // 64 columns at a time through the warp's own staging, 16-byte pieces placed by row so that neither side
      // meets bank conflicts (the 128B swizzle): rows go out as whole 128-byte lines
      const int width = min(256, p.cols - k.c0);
#pragma unroll 1
      for (int c = hh * 64; c < 256; c += 128) {
        const bool last = c + 128 >= 256;
        if (c < width) {
          uint32_t v[64];
          if (empty) {
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = 0u;
          } else {
            tmem_ld_x32(acc + c, v);
            tmem_ld_x32(acc + c + 32, v + 32);
            tmem_wait_ld();
            reg_fence<64>(v);
            if constexpr (S::kEight) {  // all the scales before the first store to shared memory: the reads overlap
              from_int<64>(v, small);
              uint4 sc[8];
#pragma unroll
              for (int half = 0; half < 64; half += 32) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sc[i] = ld_shared_v4(scales + c / 128 * 256 + half * 4 + i * 16);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const uint32_t four[4] = {sc[i].x, sc[i].y, sc[i].z, sc[i].w};
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    uint32_t& x = v[half + 4 * i + j];
                    x = __float_as_uint(__uint_as_float(x) * (row_factor * __uint_as_float(four[j])));
                  }
                }
              }
            }
          }
          if (last && !empty) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) release<PAIR>(&b.acc_empty[d.i]);
          }
          if constexpr (S::kIsDw) {
            if (lane == 0) bulk_wait_group_read<0>();  // the last store has read the staging
          }
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[q * 8 + i]) * (S::kEight ? 1.f : row_factor);
            st_shared_v4(stage + lane * 128 + ((q ^ (lane & 7)) << 4),
                         make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])));
          }
          if constexpr (S::kIsDw) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && k.m0 + sp * 32 < (MODE == kDwUp ? 2 * p.s : p.h)) {
              tma_store_3d(m_out, smem + S::kOffOut + (warp - 4) * kStageOut, k.c0 + c, k.m0 + sp * 32, k.expert);
              bulk_commit_group();
            }
          } else {
            __syncwarp();
            const int piece = lane & 7, col = k.c0 + c + piece * 8;
            uint4 o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = i * 4 + (lane >> 3);
              o[i] = ld_shared_v4(stage + rr * 128 + ((piece ^ (rr & 7)) << 4));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int tr = sp * 32 + i * 4 + (lane >> 3);
              if (tr < k.n && col < p.cols)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)(k.row + tr) * p.cols + col) =
                    o[i];
            }
            __syncwarp();
          }
        } else if (last && !empty) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) release<PAIR>(&b.acc_empty[d.i]);
        }
      }
    }
    if (!empty && !S::kRuns) d.next(S::kAccs);
  }
  if constexpr (S::kIsDw) {
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }
}

template <int MODE, int HALF, bool PAIR>
__global__ void __launch_bounds__(Shape<MODE, HALF, PAIR>::kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap m0, const __grid_constant__ CUtensorMap m1,
                   const __grid_constant__ CUtensorMap m2, const __grid_constant__ CUtensorMap m3, const Params p) {
  using S = Shape<MODE, HALF, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Bars b = bars_at(smem + S::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&b.full[i], 1 + (S::kGathers ? kGatherWarps * 32 : 0));
      mbar_init(&b.empty[i], 1);
    }
    for (int i = 0; i < S::kAccs; ++i) {
      mbar_init(&b.acc_full[i], 1);
      mbar_init(&b.acc_empty[i], PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(b.drain, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&b.halves[i], 2);
    *b.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(b.tmem_slot, S::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(b.tmem_slot, S::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // the other CTA's barriers are used from here on
  tc_fence_after();
  const uint32_t tmem = *b.tmem_slot;
  after_previous();
  if (warp == 0) {
    box_loads<MODE, HALF, PAIR>(p, b, smem, &m0, &m1, &m2, &m3, rank);
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) mma_role<MODE, HALF, PAIR>(p, b, smem, tmem);
    __syncwarp();
  } else if (warp < 4 || warp >= 12) {
    if constexpr (S::kGathers) row_copies<MODE, HALF, PAIR>(p, b, smem, warp < 4 ? warp - 2 : warp - 10);
    __syncwarp();
  } else {
    epilogue<MODE, HALF, PAIR>(p, b, smem, tmem, &m2, rank);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // neither CTA leaves while the other's MMAs or arrivals may reach it
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, S::kTmemCols);
    else
      tmem_dealloc(tmem, S::kTmemCols);
  }
}

// ---- host side ---------------------------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

// A row-major tensor [depth][rows][width] of `bytes`-byte elements, 128B-swizzled boxes of box_w x box_h (x 1).
bool make_map(CUtensorMap* m, const void* base, int bytes, int64_t width, int64_t rows, int64_t depth, int box_w,
              int box_h) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t rank = depth ? 3 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)depth};
  cuuint64_t strides[2] = {(cuuint64_t)(width * bytes), (cuuint64_t)(width * rows * bytes)};
  cuuint32_t box[3] = {(cuuint32_t)box_w, (cuuint32_t)box_h, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, rank,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int HALF, bool PAIR>
cudaError_t launch(const ExpertsArgs& a, Params p, int64_t items, const CUtensorMap& m0, const CUtensorMap& m1,
                   const CUtensorMap& m2, const CUtensorMap& m3) {
  using S = Shape<MODE, HALF, PAIR>;
  static_assert(S::kSmem <= 227 * 1024, "shared memory");
  int dev = 0, sms = 148;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> done[64] = {};
  if (dev < 0 || dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(grouped_kernel<MODE, HALF, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev].store(1, std::memory_order_release);
  }
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  p.status = a.status;
  constexpr int ctas = PAIR ? 2 : 1;
  const int64_t most = sms / ctas;
  return launch_next(grouped_kernel<MODE, HALF, PAIR>, dim3((unsigned)((items < most ? items : most) * ctas)),
                     dim3(S::kThreads), S::kSmem, a.stream, ctas, m0, m1, m2, m3, p);
}

int tiles_of(int n, int bn) { return (n + bn - 1) / bn; }

#define MORE_TRY(expr)                    \
  do {                                    \
    const cudaError_t err_ = (expr);      \
    if (err_ != cudaSuccess) return err_; \
  } while (0)
#define MORE_MAP(...) \
  if (!make_map(__VA_ARGS__)) return cudaErrorInvalidValue

// H = silu(X A^T) * (X B^T).  pair: X holds the rows already picked, [R][h].
template <int MODE>
cudaError_t run_up(const ExpertsArgs& a, const Rows& rows, const void* X, const float* row_scale, void* H,
                   float* h_scale, bool pair) {
  constexpr int bytes = MODE == kUp8 ? 1 : 2, box = 128 / bytes;
  Params p = {};
  p.rows = rows;
  p.k1 = a.h;
  p.s = a.s;
  p.h = a.h;
  p.cols = a.s;
  p.out = H;
  p.row_scale = row_scale;
  p.out_scale = h_scale;
  p.col_scale = a.up_scale;
  p.X = X;
  CUtensorMap m0, m1;
  // 128 + 128 columns a tile; 64 + 64 where the expert has no more
  const int half = a.s <= 64 ? 64 : 128;
  MORE_MAP(&m1, a.W_up, bytes, a.h, 2 * (int64_t)a.s, a.M, box, half);
  p.nc = tiles_of(a.s, half);
  const int64_t items = max_tiles(a.S(), a.M, pair ? 2 * kTileRows : kTileRows) * p.nc;
  if (pair) {
    MORE_MAP(&m0, X, bytes, a.h, max_rows(a.S(), a.M), 0, box, kTileRows);
    return launch<MODE, 128, true>(a, p, items, m0, m1, m1, m1);
  }
  if (half == 64) return launch<MODE, 64, false>(a, p, items, m1, m1, m1, m1);
  return launch<MODE, 128, false>(a, p, items, m1, m1, m1, m1);
}

template <int MODE>
cudaError_t run_down(const ExpertsArgs& a, const Rows& rows, const void* H, const float* h_scale, void* Y, bool pair) {
  constexpr int bytes = MODE == kDown8 ? 1 : 2, box = 128 / bytes;
  Params p = {};
  p.rows = rows;
  p.k1 = a.s;
  p.s = a.s;
  p.h = a.h;
  p.cols = a.h;
  p.out = Y;
  p.row_scale = h_scale;
  p.col_scale = a.down_scale;
  p.nc = tiles_of(a.h, 256);
  CUtensorMap m0, m1;
  MORE_MAP(&m0, H, bytes, a.s, max_rows(a.S(), a.M), 0, box, kTileRows);
  MORE_MAP(&m1, a.W_down, bytes, a.s, a.h, a.M, box, pair ? 128 : 256);
  const int64_t items = max_tiles(a.S(), a.M, pair ? 2 * kTileRows : kTileRows) * p.nc;
  return pair ? launch<MODE, 64, true>(a, p, items, m0, m1, m0, m0) : launch<MODE, 64, false>(a, p, items, m0, m1, m0, m0);
}

}  // namespace experts

using namespace experts;

namespace {

struct Buffers {
  Rows rows;
  void *H, *Hq, *Xq, *Y;
  void *Xr, *Dr;  // X's (or its 8 bits') and y_bar's rows in the padded layout, for CTA pairs
  float *x_scale, *row_scale, *h_scale, *part;
  __nv_bfloat16 *pre, *mid;
  FewArgs few;  // the buffers of the few-token kernel
  size_t bytes;
};

enum Kind { kForward = 0, kInt8 = 1, kBackward = 2 };

// Tiles of the backward's first kernel: 3 x 128 columns, or 3 x 64 for experts that have no more, and where h is so long
// that the products want runs.  In one run the gate's gradient is off by 1.4e-6 of itself at h = 512 and 6.1e-6, the most, at
// h = 2048; 3 x 64 columns from h = 512 on would halve that and take the backward of 8192 tokens, h = 2048, s = 1024,
// from 1455 to 1780 us.
int back_half(int h, int s) { return s <= 64 || h > 2 * kRun ? 64 : 128; }
int gate_parts(int h, int s) { return 2 * tiles_of(s, back_half(h, s)); }

// CTA pairs with 256-row tiles, the rows picked by token copied together first (the copies by token of a pair would
// need both CTAs' loaders).  A pair reads the weights once for 256 rows, but the picked rows are written and read once
// more, and tiles of 256 waste more of the last one.  us a call with and without pairs, for T rows an expert:
//   forward   h = 2048: s = 256, T = 1024: 188, 153    s = 512, T = 1024: 136, 128    s = 704, T = 512: 185, 172
//             s = 1024, T = 256: 282, 263    T = 512: 462, 443    T = 1024: 408, 399    T = 2048: 380, 382
//             s = 2048, T = 512: 421, 415    T = 1024: 370, 377   h = 1096, s = 712, T = 469: 217, 248
//             h = 1024 = s, T = 512: 244, 238    h = 4096: s = 1024, T = 512: 448, 430    s = 4096, T = 1024: 336, 372
//   8 bits    h = 2048: s = 512, T = 1024: 138, 126    s = 704, T = 512: 158, 153    s = 1024, T = 256: 206, 201
//             T = 512: 331, 335    T = 2048: 295, 313    s = 2048, T = 1024: 286, 305    h = 2880 = s, T = 1024: 293, 339
//             h = 1024 = s, T = 512: 231, 224    h = 4096, s = 1024, T = 2048: 265, 278
//   backward  h = 1024: s = 144, T = 512: 437, 405     s = 512, T = 1024: 381, 409     s = 1024, T = 192: 216, 231
//             s = 1024, T = 128: 206, 200              h = 2048, s = 1024, T = 2048: 1245, 1469
//             h = 4096 (its first kernel takes no pairs): s = 512: 435, 428    s = 1024: 762, 785
// The forward's border is a compromise: between s = 704 and 2048 pairs lose up to 7 % where sizes fill tiles of 128, and win
// 12 % where they do not.
bool takes_pairs(int64_t S, int h, int s, int M, int kind) {
  return S >= 192 * (int64_t)M && s >= (kind == kBackward && h <= 2 * kRun ? 512 : 704);
}

Buffers carve(void* scratch, int64_t N, int h, int s, int M, int k, int kind) {
  Buffers b = {};
  Carver c(scratch);
  const int64_t S = N * k, R = max_rows(S, M);
  const bool pair = takes_pairs(S, h, s, M, kind);
  if (kind != kBackward && experts_few_fits(N, h, M, k)) {
    FewArgs& f = b.few;
    f.barrier = c.take<unsigned int>(1);
    if (kind == kForward) {
      f.mid_pair = c.take<__nv_bfloat16>(2 * S * s);
    } else {
      f.mid = c.take<float>(S * s);
      f.mid_q = c.take<int8_t>(S * s);
      f.mid_scale = c.take<float>(S);
      f.Xq = c.take<int8_t>(N * h);
      f.x_scale = c.take<float>(N);
    }
    b.bytes = c.used;
    return b;
  }
  b.rows = carve_rows(c, S, M);
  if (kind == kForward) {
    if (pair) b.Xr = c.take<__nv_bfloat16>(R * h);
    b.H = c.take<__nv_bfloat16>(R * s);
  } else if (kind == kInt8) {
    b.Xq = c.take<int8_t>(N * h);
    b.x_scale = c.take<float>(N);
    b.row_scale = c.take<float>(R);
    if (pair) b.Xr = c.take<int8_t>(R * h);
    if (s > 64) b.H = c.take<float>(R * s);
    b.Hq = c.take<int8_t>(R * s);
    b.h_scale = c.take<float>(R);
  } else {
    if (pair) {
      b.Xr = c.take<__nv_bfloat16>(R * h);
      b.Dr = c.take<__nv_bfloat16>(R * h);
    }
    b.pre = c.take<__nv_bfloat16>(R * 2 * s);
    b.mid = c.take<__nv_bfloat16>(R * s);
    b.part = c.take<float>(R * gate_parts(h, s));
  }
  b.Y = c.take<__nv_bfloat16>(R * h);
  b.bytes = c.used;
  return b;
}

}  // namespace

size_t experts_scratch(int64_t N, int h, int s, int M, int k, int kind) {
  return carve(nullptr, N, h, s, M, k, kind).bytes;
}

namespace {
cudaError_t launch_few(const ExpertsArgs& a, FewArgs f) {
  f.X = a.X;
  f.W_up = a.W_up;
  f.W_down = a.W_down;
  f.up_scale = a.up_scale;
  f.down_scale = a.down_scale;
  f.offsets = a.offsets;
  f.slots = a.slots;
  f.given_gate = a.gate;
  f.out = a.out;
  f.N = a.N;
  f.h = a.h;
  f.s = a.s;
  f.M = a.M;
  f.k = a.k;
  f.status = a.status;
  f.stream = a.stream;
  return launch_layer_few(f);
}
}  // namespace

cudaError_t launch_experts(const ExpertsArgs& a) {
  const Buffers b = carve(a.scratch, a.N, a.h, a.s, a.M, a.k, kForward);
  if (experts_few_fits(a.N, a.h, a.M, a.k)) return launch_few(a, b.few);
  const bool pair = takes_pairs(a.S(), a.h, a.s, a.M, kForward);
  MORE_TRY(launch_rows(a, b.rows, pair ? 2 * kTileRows : kTileRows));
  if (pair) MORE_TRY(launch_pick(a, b.rows, a.X, 2 * a.h, b.Xr));
  MORE_TRY(run_up<kUp>(a, b.rows, pair ? b.Xr : a.X, nullptr, b.H, nullptr, pair));
  MORE_TRY(run_down<kDown>(a, b.rows, b.H, nullptr, b.Y, pair));
  return launch_combine(a, b.rows, static_cast<const __nv_bfloat16*>(b.Y), a.out);
}

cudaError_t launch_experts_int8(const ExpertsArgs& a) {
  const Buffers b = carve(a.scratch, a.N, a.h, a.s, a.M, a.k, kInt8);
  if (experts_few_fits(a.N, a.h, a.M, a.k)) return launch_few(a, b.few);
  const bool pair = takes_pairs(a.S(), a.h, a.s, a.M, kInt8);
  MORE_TRY(launch_quantize_bf16(static_cast<const __nv_bfloat16*>(a.X), a.N, a.h, static_cast<int8_t*>(b.Xq),
                                b.x_scale, a.stream));
  MORE_TRY(launch_rows(a, b.rows, pair ? 2 * kTileRows : kTileRows, b.x_scale, b.row_scale));
  if (pair) MORE_TRY(launch_pick(a, b.rows, b.Xq, a.h, b.Xr));
  if (a.s <= 64) {  // one tile holds the middle of an expert's rows: rounded to 8 bits in the product's epilogue
    MORE_TRY(run_up<kUp8>(a, b.rows, b.Xq, b.row_scale, b.Hq, b.h_scale, false));
  } else {
    MORE_TRY(run_up<kUp8>(a, b.rows, pair ? b.Xr : b.Xq, b.row_scale, b.H, nullptr, pair));
    MORE_TRY(launch_quantize_rows(a, b.rows, static_cast<const float*>(b.H), a.s, static_cast<int8_t*>(b.Hq),
                                  b.h_scale, pair ? 2 * kTileRows : kTileRows));
  }
  MORE_TRY(run_down<kDown8>(a, b.rows, b.Hq, b.h_scale, b.Y, pair));
  return launch_combine(a, b.rows, static_cast<const __nv_bfloat16*>(b.Y), a.out);
}

cudaError_t launch_experts_backward(const ExpertsArgs& a) {
  const Buffers b = carve(a.scratch, a.N, a.h, a.s, a.M, a.k, kBackward);
  const int64_t S = a.S(), R = max_rows(S, a.M);
  const bool pair = takes_pairs(S, a.h, a.s, a.M, kBackward);
  const int rows = pair ? 2 * kTileRows : kTileRows;
  const int64_t tiles = max_tiles(S, a.M, rows);
  const int half = back_half(a.h, a.s);
  const bool back_pair = pair && half == 128;
  MORE_TRY(launch_rows(a, b.rows, back_pair ? 2 * kTileRows : kTileRows));
  if (pair) {
    MORE_TRY(launch_pick(a, b.rows, a.X, 2 * a.h, b.Xr));
    MORE_TRY(launch_pick(a, b.rows, a.out_bar, 2 * a.h, b.Dr));
  }
  CUtensorMap m0, m1, m2, m3;
  Params p = {};
  p.rows = b.rows;
  p.R = R;
  p.s = a.s;
  p.h = a.h;
  p.X = a.X;
  p.out_bar = a.out_bar;
  {
    Params q = p;
    q.k1 = q.k2 = a.h;
    q.cols = a.s;
    q.out = b.pre;
    q.out2 = b.mid;
    q.part = b.part;
    // 3 x 128 columns leave TMEM one accumulator, 3 x 64 two; the wide tile reads x and y_bar half as often
    q.nc = tiles_of(a.s, half);
    MORE_MAP(&m1, a.W_up, 2, a.h, 2 * (int64_t)a.s, a.M, 64, half);
    MORE_MAP(&m3, a.W_down, 2, a.s, a.h, a.M, 64, 64);
    if (back_pair) {
      MORE_MAP(&m0, b.Xr, 2, a.h, R, 0, 64, kTileRows);
      MORE_MAP(&m2, b.Dr, 2, a.h, R, 0, 64, kTileRows);
      MORE_TRY((launch<kBack, 128, true>(a, q, tiles * q.nc, m0, m1, m2, m3)));
    } else if (half == 64) {
      MORE_TRY((launch<kBack, 64, false>(a, q, max_tiles(S, a.M) * q.nc, m1, m1, m1, m3)));
    } else {
      MORE_TRY((launch<kBack, 128, false>(a, q, max_tiles(S, a.M) * q.nc, m1, m1, m1, m3)));
    }
  }
  if (pair && !back_pair) MORE_TRY(launch_rows(a, b.rows, rows));  // the same rows in tiles of 256
  {
    Params q = p;
    q.k1 = 2 * a.s;
    q.cols = a.h;
    q.out = b.Y;
    q.nc = tiles_of(a.h, 256);
    MORE_MAP(&m0, b.pre, 2, 2 * (int64_t)a.s, R, 0, 64, kTileRows);
    MORE_MAP(&m1, a.W_up, 2, a.h, 2 * (int64_t)a.s, a.M, 64, 64);
    MORE_TRY((pair ? launch<kDx, 64, true>(a, q, tiles * q.nc, m0, m1, m0, m0)
                   : launch<kDx, 64, false>(a, q, tiles * q.nc, m0, m1, m0, m0)));
  }
  {
    Params q = p;
    q.cols = a.h;
    q.nc = tiles_of(a.h, 256);
    q.nm = tiles_of(2 * a.s, rows);
    q.items = a.M * q.nm * q.nc;
    MORE_MAP(&m0, b.pre, 2, 2 * (int64_t)a.s, R, 0, 64, 64);
    MORE_MAP(&m2, a.W_up_bar, 2, a.h, 2 * (int64_t)a.s, a.M, 64, 32);
    if (pair) {
      MORE_MAP(&m1, b.Xr, 2, a.h, R, 0, 64, 64);
      MORE_TRY((launch<kDwUp, 64, true>(a, q, q.items, m0, m1, m2, m0)));
    } else {
      MORE_TRY((launch<kDwUp, 64, false>(a, q, q.items, m0, m0, m2, m0)));
    }
  }
  {
    Params q = p;
    q.cols = a.s;
    q.nc = tiles_of(a.s, 256);
    q.nm = tiles_of(a.h, rows);
    q.items = a.M * q.nm * q.nc;
    MORE_MAP(&m1, b.mid, 2, a.s, R, 0, 64, 64);
    MORE_MAP(&m2, a.W_down_bar, 2, a.s, a.h, a.M, 64, 32);
    if (pair) {
      MORE_MAP(&m0, b.Dr, 2, a.h, R, 0, 64, 64);
      MORE_TRY((launch<kDwDown, 64, true>(a, q, q.items, m0, m1, m2, m0)));
    } else {
      MORE_TRY((launch<kDwDown, 64, false>(a, q, q.items, m1, m1, m2, m1)));
    }
  }
  MORE_TRY(launch_gate_grads(a, b.rows, b.part, gate_parts(a.h, a.s), R));
  return launch_combine(a, b.rows, static_cast<const __nv_bfloat16*>(b.Y), a.out);
}

}  // namespace more
