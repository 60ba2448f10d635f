// Linear attention with a decay per head, float32 arithmetic, sequences of at most
// kLaShort tokens: the recurrence token by token.
//
// S <- lam S + kv v k^T, out = inter S q, with the layout of the single-token step: a
// state row (one p) lies in LPR lanes, four values each, and stays in registers for
// the whole sequence; a lane group takes four rows at once, whose four sums are
// halved together (6 shuffles for 32 lanes instead of 20). q, k and v of the sequence
// are in shared memory as float32. Bound by its instructions, some 25 a row, token and
// warp, so it serves few tokens: 13 float32 sequences of 12 tokens, 32 heads of
// 128 x 96, take 36 us and of 16 tokens 46 us, where the chunked kernel takes 61 us for
// 12 as for 40; four sequences of two tokens and one head 3.9 us. Small bfloat16 calls
// come here too, where the tensor-core kernel's one chunk takes 7 us.
#include "linattn.cuh"

namespace m3 {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 4;  // state rows a lane group takes at once

template <typename T>
__global__ void __launch_bounds__(kThreads) k_la_short(const __grid_constant__ LaCall a, int lpr, int rows_per_block) {
  __shared__ __align__(16) float sq[kLaShort][128], sk[kLaShort][128], sv[kLaShort][128];
  la_begin(a);
  const LaRole& r = a.role;
  const int bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
  const int N = r.N, P = r.P;
  int64_t row0, len64;
  la_rows(a, b, &row0, &len64);
  const int len = (int)len64;
  const float ld = a.log_decay[h], lam = la_power(ld, 1);
  const T* gq = (const T*)r.q + row0 * r.qs + (int64_t)(h / r.q_rep) * N;
  const T* gk = (const T*)r.k + row0 * r.ks + (int64_t)(h / r.k_rep) * N;
  const T* gv = (const T*)r.v + row0 * r.vs + (int64_t)(h / r.v_rep) * P;
  for (int i = threadIdx.x; i < len * 128; i += kThreads) {
    const int t = i >> 7, n = i & 127;
    sq[t][n] = n < N ? to_f32(gq[t * r.qs + n]) : 0.f;
    sk[t][n] = n < N ? to_f32(gk[t * r.ks + n]) : 0.f;
  }
  const int p_lo = blockIdx.y * rows_per_block, p_hi = min(P, p_lo + rows_per_block);
  for (int i = threadIdx.x; i < len * 128; i += kThreads) {
    const int t = i >> 7, p = i & 127;
    sv[t][p] = p_lo + p < p_hi ? r.kv * to_f32(gv[t * r.vs + p_lo + p]) : 0.f;
  }
  __syncthreads();
  const int lane = threadIdx.x % lpr, grp = threadIdx.x / lpr, ngrp = kThreads / lpr, n0 = 4 * lane;
  const int64_t sbase = (int64_t)bh * N * P;
  // every lane group takes part in the shuffles of every round
  for (int base = p_lo; base < p_hi; base += ngrp * kRows) {
    float s[kRows][4];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int p = base + u * ngrp + grp;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[u][e] = r.init && p < p_hi && n0 + e < N ? r.init[sbase + (int64_t)p * r.sp + (int64_t)(n0 + e) * r.sn] : 0.f;
    }
    // this lane's row of the four sums, and where its outputs go
    const int own = lpr >= 4 ? (lane & lpr / 2 ? 2 : 0) + (lane & lpr / 4 ? 1 : 0) : 0;
    const int p_own = base + own * ngrp + grp;
    const bool writes = lpr >= 4 ? (lane & (lpr / 4 - 1)) == 0 && p_own < p_hi : lane == 0;
    int64_t at = (row0 + (r.reverse ? len - 1 : 0)) * r.os + (int64_t)h * P;
    const int64_t next = r.reverse ? -r.os : r.os;
    auto write = [&](int p, float o) {
      if (r.out_rep > 1) ((float*)r.out)[at + p] = r.inter * o;
      else ((T*)r.out)[at + p] = from_f32<T>(r.inter * o);
    };
    for (int x = 0; x < len; ++x, at += next) {
      const int t = r.reverse ? len - 1 - x : x;
      const float dec = x == 0 && r.shift ? 1.f : lam;
      const float4 q = *reinterpret_cast<const float4*>(&sq[t][n0]), k = *reinterpret_cast<const float4*>(&sk[t][n0]);
      float o[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const float v = sv[t][min(base - p_lo + u * ngrp + grp, 127)];
        s[u][0] = fmaf(dec, s[u][0], v * k.x);
        s[u][1] = fmaf(dec, s[u][1], v * k.y);
        s[u][2] = fmaf(dec, s[u][2], v * k.z);
        s[u][3] = fmaf(dec, s[u][3], v * k.w);
        o[u] = s[u][0] * q.x + s[u][1] * q.y + s[u][2] * q.z + s[u][3] * q.w;
      }
      if (lpr >= 4) {
        const bool hi = lane & lpr / 2, hi2 = lane & lpr / 4;
        float a0 = hi ? o[2] : o[0], a1 = hi ? o[3] : o[1];
        a0 += __shfl_xor_sync(0xffffffffu, hi ? o[0] : o[2], lpr / 2);
        a1 += __shfl_xor_sync(0xffffffffu, hi ? o[1] : o[3], lpr / 2);
        float sum = hi2 ? a1 : a0;
        sum += __shfl_xor_sync(0xffffffffu, hi2 ? a0 : a1, lpr / 4);
        for (int d = lpr / 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (writes) write(p_own, sum);
      } else {
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          for (int d = lpr / 2; d > 0; d >>= 1) o[u] += __shfl_xor_sync(0xffffffffu, o[u], d);
          const int p = base + u * ngrp + grp;
          if (writes && p < p_hi) write(p, o[u]);
        }
      }
    }
    if (r.fin) {
      const float f = len > 0 && r.fin_shift ? lam : 1.f;
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int p = base + u * ngrp + grp;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (p < p_hi && n0 + e < N) r.fin[sbase + (int64_t)p * r.sp + (int64_t)(n0 + e) * r.sn] = f * s[u][e];
      }
    }
  }
  la_end(a);
}

}  // namespace

cudaError_t launch_la_short(const LaCall& a, LaPass, cudaStream_t s) {
  int lpr = 1;
  while (lpr * 4 < a.role.N) lpr *= 2;
  const int round = kThreads / lpr * kRows;  // rows a block takes at once
  const int64_t bh = (int64_t)a.B * a.H;
  // rows of a block: as many as leave eight blocks for every SM, since each block
  // brings q and k into shared memory
  const int64_t want = (a.role.P * bh + 152 * 8 - 1) / (152 * 8);
  int per = (int)((want + round - 1) / round) * round;
  if (per > a.role.P) per = a.role.P;
  const dim3 grid((unsigned)bh, (unsigned)((a.role.P + per - 1) / per));
  return a.dtype == M3_DTYPE_FP32
             ? launch_role(k_la_short<float>, grid, kThreads, 0, a.beside, s, a, lpr, per)
             : launch_role(k_la_short<__nv_bfloat16>, grid, kThreads, 0, a.beside, s, a, lpr, per);
}

}  // namespace m3
