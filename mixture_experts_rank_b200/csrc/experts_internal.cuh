// Shared declarations of the experts' operators: the padded row layout that every product works on,
// its place in the caller's scratch, and the launchers.
//
// The slots sorted by expert (more_dispatch) are laid out as rows, each expert's rows starting at a
// multiple of 16 (kRowPad: the K step of a 16-bit MMA, so that a product over an expert's rows can
// end on a whole step).  A tile is up to 128 rows of one expert, 256 for CTA pairs.  Padding rows, and those of slots
// out of range, carry slot -1.  A product over an expert's rows takes zeros for them, on both sides: a token's values could
// be no numbers, and zero times those is none (backward of 32768 tokens: 339 us, 334 with a token's values).  The other
// products may take any token's, the expert's last one's, since each row's results are its own.
#pragma once
#include "more_internal.cuh"

namespace more {

constexpr int kRowPad = 16;
constexpr int kTileRows = 128;

// Where a call's rows come from; all pointers are in the caller's scratch.
struct Rows {
  int32_t* row_slot;   // [R] slot of a row, -1 for padding (and for a slot outside [0, S))
  int32_t* row_token;  // [R] token of a row; where row_slot < 0, -1 - t with any token t
  float* row_gate;     // [R] gate of a row's slot (0 where row_slot < 0)
  int32_t* slot_row;   // [S] row of a slot, -1 where no expert lists it
  int4* tiles;         // [T] {expert, first row, rows that are slots (at most the call's tile_rows), those padded}
  int32_t* row_start;  // [M + 1] first row of each expert
  int32_t* n_tiles;    // [1]
};

// One call of the experts' operators after validation.
struct ExpertsArgs {
  const void* X;         // bf16 [N][h]
  const void* W_up;      // bf16 or int8 [M][2 s][h]
  const void* W_down;    // bf16 or int8 [M][h][s]
  const float* up_scale;    // [M][2 s], int8 weights only
  const float* down_scale;  // [M][h], int8 weights only
  const float* gate;        // [N][k]
  const int32_t* offsets;   // [M + 1]
  const int32_t* slots;     // [N k]
  int64_t N;
  int h, s, M, k;
  void* out;  // bf16 [N][h]
  // backward
  const void* out_bar;  // bf16 [N][h]
  void* W_up_bar;       // bf16 [M][2 s][h]
  void* W_down_bar;     // bf16 [M][h][s]
  float* gate_bar;      // [N][k]
  float* logits_bar;    // [N][k]
  void* scratch;
  unsigned int* status;
  cudaStream_t stream;
  int64_t S() const { return N * k; }
};

// Upper bounds over every routing of S slots to M experts.
inline int64_t max_rows(int64_t S, int M) {
  const int64_t used = S < M ? S : M;
  return (S + used * (kRowPad - 1) + kTileRows - 1) / kTileRows * kTileRows;
}
inline int64_t max_tiles(int64_t S, int M, int tile_rows = kTileRows) { return S / tile_rows + (S < M ? S : M); }

// Rows, tiles and work items of every kernel count in 32 bits.
inline bool experts_supported(int64_t N, int h, int s, int M, int k) {
  constexpr int64_t most = 0x7fffffffLL;
  if (k > MORE_KMAX || M > MORE_MMAX || N > most / k || h > 131072 || s > 131072) return false;
  const int64_t S = N * k, wide = (h > 2 * s ? h : 2 * s) / 64 + 1;
  return max_rows(S, M) + kTileRows < most && (max_tiles(S, M) + 1) * wide < most &&
         (int64_t)M * (2 * (int64_t)s / 128 + 1) * (h / 128 + 1) < most;
}

// Hands out aligned pieces of a scratch buffer; with a null base it only counts bytes.
struct Carver {
  uint8_t* base;
  size_t used = 0;
  explicit Carver(void* b) : base(static_cast<uint8_t*>(b)) {}
  template <class T>
  T* take(int64_t n) {
    T* p = reinterpret_cast<T*>(base + used);
    used += ((size_t)n * sizeof(T) + 255) / 256 * 256;
    return base ? p : nullptr;
  }
};

__device__ __forceinline__ int any_token(int row_token) { return row_token < 0 ? -1 - row_token : row_token; }

inline Rows carve_rows(Carver& c, int64_t S, int M) {
  Rows r;
  const int64_t R = max_rows(S, M);
  r.row_slot = c.take<int32_t>(R);
  r.row_token = c.take<int32_t>(R);
  r.row_gate = c.take<float>(R);
  r.slot_row = c.take<int32_t>(S);
  r.tiles = c.take<int4>(max_tiles(S, M));
  r.row_start = c.take<int32_t>((int64_t)M + 1);
  r.n_tiles = c.take<int32_t>(1);
  return r;
}

// The larger of a row's largest magnitude so far and |v|, NaN once one of them is: what is no number of a row stays in
// its scale.  One instruction, as the maximum that skips a NaN.
__device__ __forceinline__ float top_of(float top, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(top), "f"(fabsf(v)));
  return r;
}

// round-half-even(127 v / top) of four values |v| <= top, with `inv` = 127 / top, as the four bytes of a word.  127 v is
// exact for a bf16 v, so the division would round no value across a half; the product with inv is off by less than
// 127 * 3 * 2^-24 < 2.3e-5, and where one of the four comes that close to a half, all are divided.  Adding 1.5 * 2^23
// rounds to a whole number in the mantissa's low bits: the conversion instructions run at an eighth of the rate.  Where top
// is below 127 / FLT_MAX, inv is infinite and the product no number: those are divided too.  From 2^121 on 127 v is beyond
// the largest float, so of large rows the division takes 2^-8 of both sides.  With an infinite top infinities give
// +-127 and the rest 0; with one that is no number all give 0.
// The kernels around it branch once for four values (33.5 million of them in quantize_rows_kernel: 30 us, 36 us with a
// branch a value; in quantize_bf16_kernel: 25 and 33 us).
__device__ __forceinline__ uint32_t round8x4(float v0, float v1, float v2, float v3, float top, float inv) {
  constexpr float kRound = 12582912.f;
  const float v[4] = {v0, v1, v2, v3};
  float t[4];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = v[i] * inv;
    t[i] = y + kRound;
    near |= !(fabsf(y - (t[i] - kRound)) <= 0.5f - 4e-5f);
  }
  if (near) {
    const float part = top > 0x1p100f ? 0x1p-8f : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y = __fdiv_rn(127.f * part * v[i], part * top);
      if (y != y) y = top == top ? copysignf(127.f, v[i]) : 0.f;
      t[i] = y + kRound;
    }
  }
  const uint32_t lo = __byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(t[2]), __float_as_uint(t[3]), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// What a row's values are divided by: its largest magnitude, 1 for a row of zeros.
__device__ __forceinline__ float divisor_of(float top) { return top == 0.f ? 1.f : top; }

// A launch that the stream may prepare while the kernel before it ends: the kernel's first action on global memory is
// after_previous(), which waits for everything before it.  A call of the experts is up to nine short kernels, and this
// takes 1 to 2 us off each of their borders.
template <class... Params, class... Args>
cudaError_t launch_next(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster,
                        Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// Lays the rows out from offsets, slots and gates (experts_rows.cu).
// With token_scale also each row's scale.
cudaError_t launch_rows(const ExpertsArgs& a, const Rows& r, int tile_rows, const float* token_scale = nullptr,
                        float* row_scale = nullptr);
// Rows of `pitch` bytes (a multiple of 16) picked by token into the padded layout.
cudaError_t launch_pick(const ExpertsArgs& a, const Rows& r, const void* src, int pitch, void* dst);
// out[n] = sum over j of y[slot_row[n k + j]], fp32 sums in the order of j, rounded once to bf16.
cudaError_t launch_combine(const ExpertsArgs& a, const Rows& r, const __nv_bfloat16* y, void* out);
// gate_bar[slot] = the sum of `parts` partial sums [parts][R] in order, and the logits' gradient
// of a softmax over the k gates.
cudaError_t launch_gate_grads(const ExpertsArgs& a, const Rows& r, const float* part, int parts, int64_t R);
// Symmetric 8-bit rounding of rows: scale = max |v| / 127 (NaN where a value is), q = round-half-even(127 v / max |v|).
cudaError_t launch_quantize_bf16(const __nv_bfloat16* v, int64_t rows, int width, int8_t* q, float* scale,
                                 cudaStream_t stream);
// The same for the rows that a call uses of an fp32 [R][width] buffer (every tile's slots).
cudaError_t launch_quantize_rows(const ExpertsArgs& a, const Rows& r, const float* v, int width, int8_t* q,
                                 float* scale, int tile_rows);

// The whole layer of a few tokens, or its experts alone (moe_layer.cu).  Xq and the scales: 8-bit weights.
struct FewArgs {
  const void *X, *R1, *R2;
  int8_t* Xq;      // [N][h]
  float* x_scale;  // [N]
  const void *W_up, *W_down;
  const float *up_scale, *down_scale;
  const int32_t *offsets, *slots;  // selections made before (with given_gate); null: routed by the call
  const float* given_gate;
  float *z, *logits;  // [N][r], [N][M]
  int32_t* idx;       // [N k]
  float* gate;        // [N k]
  __nv_bfloat16* mid_pair;  // [2][N k][s]
  float* mid;               // int8: [N k][s]
  int8_t* mid_q;            // int8: [N k][s]
  float* mid_scale;         // int8: [N k]
  unsigned int* barrier;
  void* out;
  int64_t N;
  int h, r, s, M, k;
  unsigned int* status;
  cudaStream_t stream;
};
bool layer_few_fits(int64_t N);
// The same kernel for selections that were dispatched before.
bool experts_few_fits(int64_t N, int h, int M, int k);
cudaError_t launch_layer_few(const FewArgs& f);

size_t experts_scratch(int64_t N, int h, int s, int M, int k, int kind);  // kind: 0 bf16, 1 int8, 2 backward
cudaError_t launch_experts(const ExpertsArgs& a);
cudaError_t launch_experts_int8(const ExpertsArgs& a);
cudaError_t launch_experts_backward(const ExpertsArgs& a);

}  // namespace more
