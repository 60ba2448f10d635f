// m3_qk_norm_rope and its adjoint: RMS norm of every query and key head and the
// rotation by the token's position in one pass.
//
// One value is read once and written once; with about 8 operations a value
// the pass is bound by HBM. A head's D values are held by a group of G lanes,
// eight consecutive values each (G = D / 8 rounded up to a power of two, so a
// bfloat16 head of 128 is 16 lanes of 16 bytes), the sum of squares is log2(G)
// shuffles, and the partner of a rotated value (A values away) comes from
// another lane's registers by one shuffle a word. A lane group takes up to 16
// heads of one row, four at a time with their loads in flight together, so the
// row's cosines and sines are loaded once for them. Measured: 97 us for 16,384 rows
// of 64 bfloat16 heads of 128 (5.6 TB/s, 83 % of a copy's rate; one head in flight
// took 139 us); the adjoint of 8,192 rows of 36 float32 heads 90 us (5.1 TB/s).
// At four blocks an SM the forward kernel has 64 registers a thread, of which bfloat16
// spills 8 bytes and float32 80 (no float32 prompt has been timed).
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
constexpr int kBwdBlocks = 304;  // two blocks on each of 152 SMs
constexpr int kMaxD = 256;

// Eight values as they lie in memory, and as float32.
template <typename T>
struct Raw {
  uint32_t w[2 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw<T> load8(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    *reinterpret_cast<uint4*>(r.w + 4 * i) = *(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
__device__ __forceinline__ void values(const Raw<float>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void values(const Raw<__nv_bfloat16>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ Raw<T> from_lane(const Raw<T>& r, int lane) {
  Raw<T> o;
#pragma unroll
  for (int i = 0; i < 2 * (int)sizeof(T); ++i) o.w[i] = __shfl_sync(0xffffffffu, r.w[i], lane);
  return o;
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

__device__ __forceinline__ float2 pair(const float* v, int i) { return make_float2(v[i], v[i + 1]); }
__device__ __forceinline__ void set(float* v, int i, float2 p) {
  v[i] = p.x;
  v[i + 1] = p.y;
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

// Blocks of a launch: the first `q_blocks` take queries, the rest keys.
struct Split {
  int q_blocks, blocks;
};
__device__ __forceinline__ int side_of(const Split& p) { return (int)blockIdx.x >= p.q_blocks; }
__device__ __forceinline__ int index_in(const Split& p) { return side_of(p) ? blockIdx.x - p.q_blocks : blockIdx.x; }
__device__ __forceinline__ int blocks_of(const Split& p) { return side_of(p) ? p.blocks - p.q_blocks : p.q_blocks; }

// Adds the weight-gradient sums that every thread holds for its columns
// (cols[i], -1: none) over the block's `slots` in order and writes them to the
// block's row of `partial` [block][D].
template <int W>
__device__ __forceinline__ void block_weights(const RopeArgs& a, const float* gw, int slot, int slots,
                                              const int* cols) {
  extern __shared__ float sm[];
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (cols[i] >= 0) sm[slot * a.D + cols[i]] = gw[i];
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    float s = 0.f;
    for (int x = 0; x < slots; ++x) s += sm[x * a.D + d];
    a.partial[(int64_t)blockIdx.x * a.D + d] = s;
  }
}

// Eight consecutive values a lane. `per`: heads of one row that a lane group
// takes, kAhead at a time with their loads in flight together; an item is (row,
// run of `per` heads). With inv the inverse RMS the forward pass is
// y_i = inv (x_i wc_i + xm_i ws_i), xm the value A away (from lane `mate`), wc = w
// cos and ws = +-w_m sin the same for every head of the row.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 2 : 4)
    k_rope_vec(const __grid_constant__ RopeArgs a, Split split, int lanes, int per) {
  constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;
  const int lane = threadIdx.x & 31, li = lane % lanes, base = lane - li;
  const int grp = threadIdx.x / lanes, ngrp = kThreads / lanes;
  const int D = a.D, A = a.A, e = 8 * li;
  const bool on = e < D;
  // the lane that holds the other half of this lane's pairs, and the sign of its term
  const int em = e < A ? e + A : e < 2 * A ? e - A : e;  // that half's values
  const int mate = base + em / 8;
  const float sign = (e < A ? -1.f : 1.f) * (BWD ? -1.f : 1.f);
  const int sd = side_of(split);
  const RopeSide& s = a.side[sd];
  const int runs = (s.heads + per - 1) / per;
  const int64_t items = a.rows * runs;
  const float inv_d = 1.0f / (float)D;
  float gw[8] = {};
  // whole warps leave the loop together: the shuffles below name all 32 lanes
  const int64_t stride = (int64_t)blocks_of(split) * ngrp;
  for (int64_t it0 = (int64_t)index_in(split) * ngrp + (grp - base / lanes); it0 < items; it0 += stride) {
    const int64_t it = it0 + base / lanes;
    const bool live = it < items;
    const int64_t row = live ? it / runs : 0;
    const int run = live ? (int)(it - row * runs) : 0;
    const int h0 = run * per, h1 = live && on ? min(s.heads, h0 + per) : h0;
    const T* x = (const T*)s.x + row * s.xs + e;
    const T* dy = (const T*)s.dy + row * s.dys + e;
    T* y = (T*)s.y + row * s.ys + e;
    Raw<T> rx[kAhead], rg[BWD ? kAhead : 1];
    auto load = [&](int hb) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int h = h0 + hb + u;
        rx[u] = Raw<T>{};
        if (BWD) rg[BWD ? u : 0] = Raw<T>{};
        if (h < h1 && hb + u < per) {
          rx[u] = load8(x + h * D);
          if (BWD) rg[BWD ? u : 0] = load8(dy + h * D);
        }
      }
    };
    load(0);  // before the position, which the tables wait for
    float c[8], sn[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { c[i] = 1.f; sn[i] = 0.f; w[i] = 1.f; }
    const int tr = live ? table_row(a, row) : -1;
    if (tr >= 0 && e < 2 * A) {
      const int64_t at = (int64_t)tr * A + (e < A ? e : e - A);
      values(load8(a.cos_table + at), c);
      values(load8(a.sin_table + at), sn);
    }
    if (on && s.w) values(load8(s.w + e), w);
    float wm[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wm[i] = 1.f;
    if (!BWD && on && s.w) values(load8(s.w + em), wm);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!BWD) c[i] *= w[i];
      sn[i] *= BWD ? sign : sign * wm[i];
    }
    for (int hb = 0; hb < per; hb += kAhead) {
      if (hb > 0) load(hb);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int h = h0 + hb + u;
        const bool in = h < h1 && hb + u < per;
        float v[8], m[8];
        values(rx[u], v);
        float2 s2 = __fmul2_rn(pair(v, 0), pair(v, 0));
#pragma unroll
        for (int i = 2; i < 8; i += 2) s2 = __ffma2_rn(pair(v, i), pair(v, i), s2);
        const float ss = group_sum(s2.x + s2.y, lanes);
        const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
        if (!BWD) {
          const float2 i2 = make_float2(inv, inv);
          if (A > 0) {
            values(from_lane(rx[u], mate), m);
#pragma unroll
            for (int i = 0; i < 8; i += 2)
              set(v, i, __fmul2_rn(i2, __ffma2_rn(pair(m, i), pair(sn, i), __fmul2_rn(pair(v, i), pair(c, i)))));
          } else {
#pragma unroll
            for (int i = 0; i < 8; i += 2) set(v, i, __fmul2_rn(i2, __fmul2_rn(pair(v, i), pair(c, i))));
          }
        } else {
          float g[8];
          values(rg[BWD ? u : 0], g);
          if (A > 0) {
            values(from_lane(rg[BWD ? u : 0], mate), m);
#pragma unroll
            for (int i = 0; i < 8; i += 2)
              set(g, i, __ffma2_rn(pair(m, i), pair(sn, i), __fmul2_rn(pair(g, i), pair(c, i))));
          }
          const float2 i2 = make_float2(inv, inv);
          float2 d2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 xh = __fmul2_rn(pair(v, i), i2), gi = pair(g, i);
            set(v, i, xh);
            set(gw, i, __ffma2_rn(gi, xh, pair(gw, i)));
            const float2 wg = __fmul2_rn(gi, pair(w, i));
            set(g, i, wg);
            d2 = __ffma2_rn(wg, xh, d2);
          }
          const float dot = -group_sum(d2.x + d2.y, lanes) * inv_d;
          const float2 dd = make_float2(dot, dot);
#pragma unroll
          for (int i = 0; i < 8; i += 2) set(v, i, __fmul2_rn(i2, __ffma2_rn(pair(v, i), dd, pair(g, i))));
        }
        if (in) store8(y + h * D, v);
      }
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
__global__ void __launch_bounds__(kThreads) k_rope_any(const __grid_constant__ RopeArgs a, Split split) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kPairs = kMaxD / 64, kRest = kMaxD / 32;
  const int D = a.D, A = a.A;
  const int sd = side_of(split);
  const RopeSide& s = a.side[sd];
  const int64_t items = a.rows * s.heads;
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
  float gw[W] = {};
  for (int64_t it = (int64_t)index_in(split) * 8 + warp; it < items; it += (int64_t)blocks_of(split) * 8) {
    const int64_t row = it / s.heads;
    const int h = (int)(it - row * s.heads);
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
        gw[i] = fmaf(g[i], v[i], gw[i]);
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

// Weight gradients from the blocks' sums: 32 columns a block, each of its 32
// warps a run of the side's blocks in order, then the warps in order.
__global__ void __launch_bounds__(1024) k_rope_weights(const __grid_constant__ RopeArgs a, Split split) {
  __shared__ float part[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int side = blockIdx.y, d = blockIdx.x * 32 + lane;
  if (!a.gw[side]) return;
  const int first = side ? split.q_blocks : 0, end = side ? split.blocks : split.q_blocks;
  const int per = (end - first + 31) / 32;
  float s = 0.f;
  if (d < a.D)
    for (int x = first + warp * per; x < min(end, first + (warp + 1) * per); ++x)
      s += a.partial[(int64_t)x * a.D + d];
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && d < a.D) {
    s = 0.f;
    for (int x = 0; x < 32; ++x) s += part[x][lane];
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

// At most `most` blocks (one more where a side has few) of `step` items, in the
// two sides' proportion.
Split divide(int64_t q_items, int64_t k_items, int step, int64_t most) {
  int64_t q = (q_items + step - 1) / step, k = (k_items + step - 1) / step;
  if (q + k > most) {
    const int64_t all = q + k;
    if (q > 0) q = q * most / all > 0 ? q * most / all : 1;
    if (k > 0) k = most - q > 0 ? most - q : 1;
  }
  return {(int)q, (int)(q + k)};
}

template <typename T, bool BWD>
cudaError_t go(const RopeArgs& a, cudaStream_t s) {
  Split split;
  if (vec_ok(a, BWD)) {
    int lanes = 1;
    while (lanes * 8 < a.D) lanes *= 2;
    const int ngrp = kThreads / lanes;
    // heads a lane group: as many as leave every SM several blocks
    int per = BWD ? 8 : 16;
    auto runs = [&](int side) { return a.rows * ((a.side[side].heads + per - 1) / per); };
    while (per > 1 && runs(0) + runs(1) < (int64_t)152 * 8 * ngrp) per /= 2;
    split = divide(runs(0), runs(1), ngrp, BWD ? kBwdBlocks : 152 * 4 * 8);
    const size_t smem = BWD && a.partial ? (size_t)ngrp * a.D * sizeof(float) : 0;
    k_rope_vec<T, BWD><<<(unsigned)split.blocks, kThreads, smem, s>>>(a, split, lanes, per);
  } else {
    split = divide(a.rows * a.side[0].heads, a.rows * a.side[1].heads, 8, BWD ? kBwdBlocks : 152 * 8 * 8);
    const size_t smem = BWD && a.partial ? (size_t)8 * a.D * sizeof(float) : 0;
    k_rope_any<T, BWD><<<(unsigned)split.blocks, kThreads, smem, s>>>(a, split);
  }
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !BWD || !a.partial) return e;
  k_rope_weights<<<dim3((unsigned)((a.D + 31) / 32), 2), 1024, 0, s>>>(a, split);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t s) {
  return a.dtype == M3_DTYPE_FP32 ? go<float, false>(a, s) : go<__nv_bfloat16, false>(a, s);
}
size_t qk_norm_rope_backward_bytes(const RopeArgs& a) {
  return (size_t)(kBwdBlocks + 1) * a.D * sizeof(float);
}
cudaError_t launch_qk_norm_rope_backward(const RopeArgs& a, cudaStream_t s) {
  return a.dtype == M3_DTYPE_FP32 ? go<float, true>(a, s) : go<__nv_bfloat16, true>(a, s);
}

}  // namespace m3
