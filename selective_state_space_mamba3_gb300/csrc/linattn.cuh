// Internal declarations of the linear-attention operators (m3_qk_norm_rope,
// m3_linear_attention_*). Validation and dispatch: m3_linattn.cu. Kernels:
// k_qk_norm_rope.cu, k_linattn_mma.cu (prompts and adjoints, bfloat16),
// k_linattn_split.cu (float32, and any width or alignment), k_linattn_short.cu (the
// same for a few tokens), k_linattn_state.cu (states of segments, sums over shared
// heads), k_linattn_step.cu.
#pragma once

#include <cuda_bf16.h>

#include "m3_internal.cuh"

namespace m3 {

// --- norm and rotation of queries and keys ---------------------------------
struct RopeSide {
  const void *x, *dy;  // input; output gradient (backward)
  void* y;             // output, or input gradient
  const float* w;      // null: ones
  int64_t xs, ys, dys; // row strides in elements
  int heads;
};
struct RopeArgs {
  RopeSide side[2];  // queries, keys
  const float *cos_table, *sin_table;
  const int32_t* positions;
  float* gw[2];      // weight gradients (backward; may be null)
  float* partial;    // backward: per-block weight sums
  int64_t rows;
  int D, A, max_pos, dtype;
  float eps;
};
cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t s);
size_t qk_norm_rope_backward_bytes(const RopeArgs& a);
cudaError_t launch_qk_norm_rope_backward(const RopeArgs& a, cudaStream_t s);

// --- linear attention --------------------------------------------------------
// One recurrence over the tokens of every sequence and head,
//   out_t = intra * sum_u lam^|t-u| (q_t.k_u) v_u + inter * lam^(...) state q_t,
//   state' = lam^n state + kv * sum_u lam^(...) v_u k_u^T,
// u <= t walking up, or u >= t walking down (reverse). The forward pass is one
// of them; the backward pass is three, with the operands' roles exchanged.
// N is the width of q and k here, P that of v and out.
struct LaRole {
  const void *q, *k, *v;
  void* out;
  int64_t qs, ks, vs, os;     // row strides in elements
  int q_rep, k_rep, v_rep;    // heads that share one head of the operand
  int out_rep;                // 1, or: out is float32 [rows, H, P] partials to be summed over so many heads
  int N, P;
  int reverse;
  float intra, inter, kv;
  const float* init;          // entry state per (b, h), element (p, n) at p * sp + n * sn
  float* fin;                 // final state, same layout (null: not wanted)
  int sp, sn;
  int shift;                  // the entry state counts as of this many tokens later (0 or 1)
  int fin_shift;              // decays applied to the final state of a non-empty sequence (0 or 1)
};

constexpr int kLaChunk = 128;  // segments are whole numbers of this many tokens

// One launch of the chunk kernels: a role and what every role of the call shares.
struct LaCall {
  LaRole role;
  int B, H, dtype;
  int64_t L, rows;
  const float* log_decay;
  const int32_t* offsets;
  // long sequences are cut into nseg segments of seg_len tokens: `entry` has,
  // for each (segment, b, h), first the segment's own state sum (summary pass),
  // then its entry state (prefix pass); states as [P][N]
  int nseg;
  int64_t seg_len;
  float* entry;
  uint32_t* status;
  int clear;   // the call's first launch clears the status word
  int beside;  // the launch before it is the same pass of another role: run beside it
};
struct LaArgs {
  LaRole role[3];
  int nrole;
  LaCall call;         // (its role and entry: of the role at hand)
  int64_t entry_role;  // floats per role in `entry`
};

enum LaPass { kLaMain = 0, kLaSummary = 1 };
// sequences of at most kLaShort tokens
constexpr int kLaShort = 16;
cudaError_t launch_la_short(const LaCall& a, LaPass pass, cudaStream_t s);
// float32 activations, and bfloat16 ones that the other kernel does not take
cudaError_t launch_la_split(const LaCall& a, LaPass pass, cudaStream_t s);
// bfloat16 operands that tile copies take (widths and strides multiples of
// eight elements, 16-byte addresses): the tensor-core kernel
bool la_mma_supported(const LaArgs& a);
cudaError_t launch_la_mma(const LaCall& a, LaPass pass, cudaStream_t s);
cudaError_t launch_la_prefix(const LaArgs& a, cudaStream_t s);
// out[row][g][w] = sum over the group's heads of part[row][h][w], in head order
cudaError_t launch_la_group_sum(const LaCall& a, const float* part, void* out, int groups, int rep,
                                int width, cudaStream_t s);

struct LaStepArgs {
  const void *q, *k, *v;
  void* out;
  float* state;
  const float* log_decay;
  const int32_t* slots;
  int64_t qs, ks, vs, os;
  int B, H, rep, P, N, dtype;
  int64_t num_slots;
  float scale;
};
cudaError_t launch_la_step(const LaStepArgs& a, cudaStream_t s);

// --- shared device helpers ---------------------------------------------------
template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return (float)v;
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  return (T)v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Rows [begin, end) of sequence b; offsets outside [0, rows] count as the
// nearest row inside, and a sequence is at most L rows long.
__device__ __forceinline__ void la_rows(const LaCall& a, int b, int64_t* begin, int64_t* len) {
  if (!a.offsets) {
    *begin = (int64_t)b * a.L;
    *len = a.L;
    return;
  }
  const int64_t lo = min(max((int64_t)a.offsets[b], (int64_t)0), a.rows);
  const int64_t hi = min(max((int64_t)a.offsets[b + 1], lo), a.rows);
  *begin = lo;
  *len = min(hi - lo, a.L);
}

// Start and end of a block of a chunk kernel. The call's first kernel clears the
// status word (a wait gives up only after about two seconds); every block lets the
// next launch begin, and one that began beside its predecessor ends after it, so
// that the end of the last role's kernel is the end of all.
__device__ __forceinline__ void la_begin(const LaCall& a) {
  if (a.clear && blockIdx.x == 0 && threadIdx.x == 0) atomicExch(a.status, 0u);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void la_end(const LaCall& a) {
  if (a.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// lam^d for d >= 0 (lam = e^ld; 0 * -inf counts as 0).
__device__ __forceinline__ float la_power(float ld, int64_t d) {
  return d == 0 ? 1.0f : expf(ld * (float)d);
}

// Launches a chunk kernel, beside the launch before it where that is another
// role's pass (programmatic stream serialization).
template <typename... Ps, typename... As>
cudaError_t launch_role(void (*kernel)(Ps...), dim3 grid, int threads, size_t smem, bool beside,
                        cudaStream_t s, const As&... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = beside ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace m3
