// m3_qk_norm_rope and its adjoint: RMS norm of every query and key head and the
// rotation by the token's position in one pass.
//
// One value is read once and written once; with about 8 operations a value
// the pass is bound by HBM. A head's D values are held by a group of G lanes,
// eight consecutive values each (G = D / 8 rounded up to a power of two, so a
// bfloat16 head of 128 is 16 lanes of 16 bytes), the sum of squares is log2(G)
// shuffles, and the partner of a rotated value (A values away) comes from
// another lane's registers by one shuffle a value. A lane group takes several
// heads of one row, so the row's cosines and sines are loaded once for them.
// Widths, angle counts or addresses that are not multiples of eight values
// take the same arithmetic with one warp per head and single-value loads, a
// lane holding pairs (a, a + A) itself.
//
// Backward: g = dy rotated back, xh = s x; dx = s (w g - xh mean(w g xh)). The
// weight gradients sum g xh over rows and heads in an order fixed by the
// shape: a lane adds its own heads, a block its lane groups in order, a second
// kernel the blocks in order. Sums are float32; outputs are rounded once.
#include "linattn.cuh"

namespace m3 {
namespace {

constexpr int kThreads = 256;
constexpr int kBwdBlocks = 608;  // four blocks on each of 152 SMs
constexpr int kMaxD = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* v) {
  const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* v) {
  const uint4 r = *(const uint4*)p;
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* v) {
  *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
  *(float4*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float* v) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *(uint4*)p = *(const uint4*)h;
}

// Sum over the aligned group of `g` lanes (a power of two) the lane is in.
__device__ __forceinline__ float group_sum(float v, int g) {
  for (int o = g / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The row of the tables for token `row`, or -1: not rotated.
__device__ __forceinline__ int table_row(const RopeArgs& a, int64_t row) {
  if (a.A == 0) return -1;
  const int64_t p = a.positions ? (int64_t)a.positions[row] : row;
  return p >= 0 && p < a.max_pos ? (int)p : -1;
}

// Adds the weight-gradient sums that every thread holds for its columns of
// both sides (gw[side][i], column col + i) over the block and writes them to
// the block's slot of `partial` [block][2][D].
template <int W>
__device__ __forceinline__ void block_weights(const RopeArgs& a, float gw[2][W], int slot, int slots,
                                              const int* cols) {
  extern __shared__ float sm[];
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (cols[i] >= 0) sm[slot * a.D + cols[i]] = gw[side][i];
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += kThreads) {
      float s = 0.f;
      for (int x = 0; x < slots; ++x) s += sm[x * a.D + d];
      a.partial[((int64_t)blockIdx.x * 2 + side) * a.D + d] = s;
    }
  }
}

// Eight consecutive values a lane. `per`: heads of one row that a lane group
// takes in turn; an item is (row, run of `per` heads of one side).
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 3 : 4)
    k_rope_vec(RopeArgs a, int lanes, int per, int64_t items) {
  const int lane = threadIdx.x & 31, li = lane % lanes, base = lane - li;
  const int grp = threadIdx.x / lanes, ngrp = kThreads / lanes;
  const int D = a.D, A = a.A, e = 8 * li;
  const bool on = e < D;
  // the lane that holds the other half of this lane's pairs, and the sign of its term
  const int mate = e < A ? base + li + A / 8 : e < 2 * A ? base + li - A / 8 : lane;
  const float sign = (e < A ? -1.f : 1.f) * (BWD ? -1.f : 1.f);
  const int runs0 = (a.side[0].heads + per - 1) / per, runs1 = (a.side[1].heads + per - 1) / per;
  const int runs = runs0 + runs1;
  const float inv_d = 1.0f / (float)D;
  float gw[2][8] = {};
  // whole warps leave the loop together: the shuffles below name all 32 lanes
  const int64_t stride = (int64_t)gridDim.x * ngrp;
  for (int64_t it0 = (int64_t)blockIdx.x * ngrp + (grp - base / lanes); it0 < items; it0 += stride) {
    const int64_t it = it0 + base / lanes;
    const bool live = it < items;
    const int64_t row = live ? it / runs : 0;
    const int run = live ? (int)(it - row * runs) : 0;
    const int sd = run >= runs0;
    const RopeSide& s = a.side[sd];
    const int h0 = (sd ? run - runs0 : run) * per, h1 = live ? min(s.heads, h0 + per) : h0;
    float c[8], sn[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { c[i] = 1.f; sn[i] = 0.f; w[i] = 1.f; }
    const int tr = live ? table_row(a, row) : -1;
    if (tr >= 0 && e < 2 * A) {
      const int64_t at = (int64_t)tr * A + (e < A ? e : e - A);
      load8(a.cos_table + at, c);
      load8(a.sin_table + at, sn);
    }
    if (on && s.w) load8(s.w + e, w);
    const T* x = (const T*)s.x + row * s.xs + e;
    const T* dy = (const T*)s.dy + row * s.dys + e;
    T* y = (T*)s.y + row * s.ys + e;
    for (int hh = 0; hh < per; ++hh) {
      const int h = h0 + hh;
      const bool in = on && h < h1;
      float v[8] = {}, g[8] = {};
      if (in) {
        load8(x + h * D, v);
        if (BWD) load8(dy + h * D, g);
      }
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
      ss = group_sum(ss, lanes);
      const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
      if (!BWD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * w[i];
      }
      if (A > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& t = BWD ? g[i] : v[i];
          const float o = __shfl_sync(0xffffffffu, t, mate);
          t = fmaf(t, c[i], sign * o * sn[i]);
        }
      }
      if (BWD) {
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] *= inv;
          if (sd) gw[1][i] = fmaf(g[i], v[i], gw[1][i]);
          else gw[0][i] = fmaf(g[i], v[i], gw[0][i]);
          g[i] *= w[i];
          dot = fmaf(g[i], v[i], dot);
        }
        dot = group_sum(dot, lanes) * inv_d;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = inv * fmaf(-v[i], dot, g[i]);
      }
      if (in) store8(y + h * D, v);
    }
  }
  if constexpr (BWD) {
    if (a.partial) {
      int cols[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) cols[i] = on ? e + i : -1;
      block_weights<8>(a, gw, grp, ngrp, cols);
    }
  }
}

// Any width and alignment: one warp per head; a lane holds pairs (a, a + A),
// a = lane + 32 i, and unrotated values 2A + lane + 32 i.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) k_rope_any(RopeArgs a, int64_t items) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kPairs = kMaxD / 64, kRest = kMaxD / 32;
  const int D = a.D, A = a.A;
  const int heads = a.side[0].heads + a.side[1].heads;
  const float inv_d = 1.0f / (float)D;
  constexpr int W = 2 * kPairs + kRest;
  int cols[W];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int p = lane + 32 * i;
    cols[2 * i] = p < A ? p : -1;
    cols[2 * i + 1] = p < A ? p + A : -1;
  }
#pragma unroll
  for (int i = 0; i < kRest; ++i) {
    const int d = 2 * A + lane + 32 * i;
    cols[2 * kPairs + i] = d < D ? d : -1;
  }
  float gw[2][W] = {};
  for (int64_t it = (int64_t)blockIdx.x * 8 + warp; it < items; it += (int64_t)gridDim.x * 8) {
    const int64_t row = it / heads;
    const int hh = (int)(it - row * heads);
    const int sd = hh >= a.side[0].heads;
    const RopeSide& s = a.side[sd];
    const int h = sd ? hh - a.side[0].heads : hh;
    const T* x = (const T*)s.x + row * s.xs + (int64_t)h * D;
    const T* dy = (const T*)s.dy + row * s.dys + (int64_t)h * D;
    T* y = (T*)s.y + row * s.ys + (int64_t)h * D;
    const int tr = table_row(a, row);
    float v[W], g[W];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v[i] = cols[i] >= 0 ? to_f32(x[cols[i]]) : 0.f;
      g[i] = BWD && cols[i] >= 0 ? to_f32(dy[cols[i]]) : 0.f;
      ss = fmaf(v[i], v[i], ss);
    }
    ss = group_sum(ss, 32);
    const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
    if (!BWD) {
#pragma unroll
      for (int i = 0; i < W; ++i)
        v[i] = v[i] * inv * (s.w && cols[i] >= 0 ? s.w[cols[i]] : 1.f);
    }
    if (tr >= 0) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        if (cols[2 * i] < 0) continue;
        const int64_t at = (int64_t)tr * A + cols[2 * i];
        const float c = a.cos_table[at], sn = a.sin_table[at] * (BWD ? -1.f : 1.f);
        float& lo = BWD ? g[2 * i] : v[2 * i];
        float& hi = BWD ? g[2 * i + 1] : v[2 * i + 1];
        const float l = lo, u = hi;
        lo = fmaf(l, c, -(u * sn));
        hi = fmaf(u, c, l * sn);
      }
    }
    if (BWD) {
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v[i] *= inv;
        if (sd) gw[1][i] = fmaf(g[i], v[i], gw[1][i]);
        else gw[0][i] = fmaf(g[i], v[i], gw[0][i]);
        g[i] *= s.w && cols[i] >= 0 ? s.w[cols[i]] : 1.f;
        dot = fmaf(g[i], v[i], dot);
      }
      dot = group_sum(dot, 32) * inv_d;
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = inv * fmaf(-v[i], dot, g[i]);
    }
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (cols[i] >= 0) y[cols[i]] = from_f32<T>(v[i]);
  }
  if constexpr (BWD) {
    if (a.partial) block_weights<W>(a, gw, warp, 8, cols);
  }
}

// Weight gradients from the blocks' sums: 32 columns a block, each of its
// eight warps a run of the blocks in order, then the warps in order.
__global__ void __launch_bounds__(256) k_rope_weights(RopeArgs a, int blocks) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int side = blockIdx.y, d = blockIdx.x * 32 + lane;
  if (!a.gw[side]) return;
  const int per = (blocks + 7) / 8;
  float s = 0.f;
  if (d < a.D)
    for (int x = warp * per; x < min(blocks, (warp + 1) * per); ++x)
      s += a.partial[((int64_t)x * 2 + side) * a.D + d];
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && d < a.D) {
    s = 0.f;
    for (int x = 0; x < 8; ++x) s += part[x][lane];
    a.gw[side][d] = s;
  }
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool vec_ok(const RopeArgs& a, bool bwd) {
  if (a.D % 8 || a.A % 8) return false;
  if (a.A && (!aligned_to(a.cos_table, 16) || !aligned_to(a.sin_table, 16))) return false;
  for (const RopeSide& s : a.side) {
    if (!s.heads) continue;
    if (s.xs % 8 || s.ys % 8 || !aligned_to(s.x, 16) || !aligned_to(s.y, 16)) return false;
    if (s.w && !aligned_to(s.w, 16)) return false;
    if (bwd && (s.dys % 8 || !aligned_to(s.dy, 16))) return false;
  }
  return true;
}

template <typename T, bool BWD>
cudaError_t go(const RopeArgs& a, cudaStream_t s) {
  const int heads = a.side[0].heads + a.side[1].heads;
  unsigned grid;
  if (vec_ok(a, BWD)) {
    int lanes = 1;
    while (lanes * 8 < a.D) lanes *= 2;
    const int ngrp = kThreads / lanes;
    // heads a lane group: as many as leave every SM several blocks
    int per = 8;
    auto count = [&](int p) {
      return a.rows * ((a.side[0].heads + p - 1) / p + (a.side[1].heads + p - 1) / p);
    };
    while (per > 1 && count(per) < (int64_t)152 * 8 * ngrp) per /= 2;
    const int64_t items = count(per), blocks = (items + ngrp - 1) / ngrp;
    const int64_t most = BWD ? kBwdBlocks : 152 * 4 * 8;
    grid = (unsigned)(blocks < most ? blocks : most);
    const size_t smem = BWD && a.partial ? (size_t)ngrp * a.D * sizeof(float) : 0;
    k_rope_vec<T, BWD><<<grid, kThreads, smem, s>>>(a, lanes, per, items);
  } else {
    const int64_t items = a.rows * heads, blocks = (items + 7) / 8;
    const int64_t most = BWD ? kBwdBlocks : 152 * 8 * 8;
    grid = (unsigned)(blocks < most ? blocks : most);
    const size_t smem = BWD && a.partial ? (size_t)8 * a.D * sizeof(float) : 0;
    k_rope_any<T, BWD><<<grid, kThreads, smem, s>>>(a, items);
  }
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !BWD || !a.partial) return e;
  k_rope_weights<<<dim3((unsigned)((a.D + 31) / 32), 2), 256, 0, s>>>(a, (int)grid);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t s) {
  return a.dtype == M3_DTYPE_FP32 ? go<float, false>(a, s) : go<__nv_bfloat16, false>(a, s);
}
size_t qk_norm_rope_backward_bytes(const RopeArgs& a) {
  return (size_t)kBwdBlocks * 2 * a.D * sizeof(float);
}
cudaError_t launch_qk_norm_rope_backward(const RopeArgs& a, cudaStream_t s) {
  return a.dtype == M3_DTYPE_FP32 ? go<float, true>(a, s) : go<__nv_bfloat16, true>(a, s);
}

}  // namespace m3
