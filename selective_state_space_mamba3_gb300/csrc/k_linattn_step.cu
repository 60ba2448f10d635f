// m3_linear_attention_step: S <- lam S + v k^T, out = scale S q, one token of
// every (row, head). Bound by the state, read once and written once (8 N P
// bytes a head).
//
// A state row (one p) of N <= 128 floats is held by LPR lanes, four values
// each, so the loads and stores of a warp are whole 512-byte pieces and a row's
// readout needs log2(LPR) shuffles. A warp takes several rows at once with all
// their loads in flight before the first is used. Rows are independent of one
// another: a block takes `rows_per_block` of a head's P rows. Measured: 88 us for 256
// sequences of 32 heads, P 64, N 128 (6.2 TB/s, 91 % of a copy's rate); one sequence
// 2.5 us, a launch's time.
#include "linattn.cuh"

namespace m3 {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;  // rows in flight per lane group

template <bool VEC>
__device__ __forceinline__ float4 load_row(const float* p, int n, int N) {
  if (VEC) return *(const float4*)(p + n);
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n < N) r.x = p[n];
  if (n + 1 < N) r.y = p[n + 1];
  if (n + 2 < N) r.z = p[n + 2];
  if (n + 3 < N) r.w = p[n + 3];
  return r;
}
template <bool VEC>
__device__ __forceinline__ void store_row(float* p, int n, int N, float4 v) {
  if (VEC) {
    *(float4*)(p + n) = v;
    return;
  }
  if (n < N) p[n] = v.x;
  if (n + 1 < N) p[n + 1] = v.y;
  if (n + 2 < N) p[n + 2] = v.z;
  if (n + 3 < N) p[n + 3] = v.w;
}
template <typename T>
__device__ __forceinline__ float4 load_vec(const T* p, int n, int N) {
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n < N) r.x = to_f32(p[n]);
  if (n + 1 < N) r.y = to_f32(p[n + 1]);
  if (n + 2 < N) r.z = to_f32(p[n + 2]);
  if (n + 3 < N) r.w = to_f32(p[n + 3]);
  return r;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_la_step(LaStepArgs a, int lpr, int rows_per_block) {
  const int bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
  const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
  const int p_lo = blockIdx.y * rows_per_block, p_hi = min(a.P, p_lo + rows_per_block);
  T* out = (T*)a.out + (int64_t)b * a.os + (int64_t)h * a.P;
  if (slot < 0 || slot >= a.num_slots) {
    for (int p = p_lo + threadIdx.x; p < p_hi; p += kThreads) out[p] = from_f32<T>(0.f);
    return;
  }
  const int lane = threadIdx.x % lpr, grp = threadIdx.x / lpr, ngrp = kThreads / lpr;
  const int N = a.N, n = 4 * lane;
  const bool on = n < N;
  const float lam = la_power(a.log_decay[h], 1);
  const float4 q = load_vec((const T*)a.q + (int64_t)b * a.qs + (int64_t)(h / a.rep) * N, n, N);
  const float4 k = load_vec((const T*)a.k + (int64_t)b * a.ks + (int64_t)(h / a.rep) * N, n, N);
  const T* v = (const T*)a.v + (int64_t)b * a.vs + (int64_t)h * a.P;
  float* st = a.state + (slot * a.H + h) * (int64_t)a.P * N;
  // every group of lanes takes part in the shuffles of every round
  for (int base = p_lo; base < p_hi; base += ngrp * kUnroll) {
    float4 s[kUnroll];
    float vv[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int p = base + u * ngrp + grp;
      const bool in = p < p_hi;
      s[u] = in && on ? load_row<VEC>(st + (int64_t)p * N, n, N) : make_float4(0.f, 0.f, 0.f, 0.f);
      vv[u] = in ? to_f32(v[p]) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int p = base + u * ngrp + grp;
      s[u].x = fmaf(lam, s[u].x, vv[u] * k.x);
      s[u].y = fmaf(lam, s[u].y, vv[u] * k.y);
      s[u].z = fmaf(lam, s[u].z, vv[u] * k.z);
      s[u].w = fmaf(lam, s[u].w, vv[u] * k.w);
      if (p < p_hi && on) store_row<VEC>(st + (int64_t)p * N, n, N, s[u]);
      float o = s[u].x * q.x + s[u].y * q.y + s[u].z * q.z + s[u].w * q.w;
      for (int x = lpr / 2; x > 0; x >>= 1) o += __shfl_xor_sync(0xffffffffu, o, x);
      if (p < p_hi && lane == 0) out[p] = from_f32<T>(a.scale * o);
    }
  }
}

}  // namespace

cudaError_t launch_la_step(const LaStepArgs& a, cudaStream_t s) {
  int lpr = 1;
  while (lpr * 4 < a.N) lpr *= 2;
  const int round = kThreads / lpr * kUnroll;  // rows a block takes at once
  const int64_t bh = (int64_t)a.B * a.H;
  // one round a block while that leaves the SMs short of blocks, else a whole head
  const int per = bh >= 152 * 8 ? a.P : (round < a.P ? round : a.P);
  const dim3 grid((unsigned)bh, (unsigned)((a.P + per - 1) / per));
  const bool f32 = a.dtype == M3_DTYPE_FP32, vec = a.N % 4 == 0;
  if (f32) {
    if (vec) k_la_step<float, true><<<grid, kThreads, 0, s>>>(a, lpr, per);
    else k_la_step<float, false><<<grid, kThreads, 0, s>>>(a, lpr, per);
  } else {
    if (vec) k_la_step<__nv_bfloat16, true><<<grid, kThreads, 0, s>>>(a, lpr, per);
    else k_la_step<__nv_bfloat16, false><<<grid, kThreads, 0, s>>>(a, lpr, per);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace m3
