// Linear attention with a decay per head in float32 on the tensor cores: every
// float32 operand is cut into three bfloat16 parts (8 + 8 + 8 significant bits,
// so x = x0 + x1 + x2 exactly) and a product takes the six part products down to
// 2^-16 (x0 y0, x0 y1, x1 y0, x1 y1, x0 y2, x2 y0; the dropped ones are below
// 2^-21 of it), accumulated in float32 in tensor memory. It takes any width up
// to 128, any stride and any alignment, and bfloat16 operands that tile copies
// do not take (those are one part each).
//
// The chunked form is that of the bfloat16 kernel, with chunks of 112 tokens:
// three parts of K [112][128], V and V^ [112][64] and S [128][64] are 216 KB of
// shared memory, and 112 is the largest multiple of 16 that fits. The parts of
// Q are the tensor-memory operand of A = Q K^T and Oi = Q S (rows 112..127 of
// the 128-row tile stay zero), and the parts of P take their columns after
// both, so tensor memory is full: Q / P 192, A 128, O, Oi and K^T V^ 64 each.
// One block of 512 threads an SM; the next chunk's rows are loaded into
// registers while this one's products run, and cut and stored to shared memory
// as soon as the product that read the tile is done.
//
// Bound by the tensor cores: six passes cost 6,900 cycles a chunk at N = 128,
// P = 64, against 7,300 for its bytes at the HBM rate.
#include "linattn_mma.cuh"

namespace m3 {
namespace {

constexpr int kC = 112;
constexpr int kThreads = 512;
constexpr long long kBudget = 4000000000LL;  // clock cycles, about 2 s
constexpr uint32_t kBlk = kC * 128;          // bytes of a 64-column block of a tile part
constexpr int kParts = 3;
constexpr uint32_t kColQ = 0, kColA = 192, kColO = 320, kColI = 384, kColS = 448, kCols = 512;

__host__ __device__ constexpr uint32_t state_bytes(int nb) { return nb * 8192; }
__host__ __device__ constexpr uint32_t tile_bytes(int nb) {
  return kParts * (nb * kBlk + 2 * kBlk + state_bytes(nb));
}
struct Small {
  float pw[kC + 20];  // lam^d, d <= 128
  float col[16];      // column factors of a 16-token block
  uint64_t bar[3];
  uint32_t tmem;
};
static_assert(sizeof(Small) <= 1024, "");
constexpr uint32_t kSmem = tile_bytes(2) + 1024;
static_assert(kSmem <= 227 * 1024, "");

__device__ __forceinline__ float top(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}
// Two truncated values as a pair of bfloat16 (a in the low half).
__device__ __forceinline__ uint32_t pair_top(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
// The three parts of (a, b) as pairs of bfloat16.
__device__ __forceinline__ void cut2(float a, float b, uint32_t* p) {
  p[0] = pair_top(a, b);
  a -= top(a);
  b -= top(b);
  p[1] = pair_top(a, b);
  a -= top(a);
  b -= top(b);
  p[2] = pair_top(a, b);
}
__device__ __forceinline__ void sts2(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
// Byte offset of the four elements at column c (c % 4 == 0) of row r of a part
// with 64-column blocks of kBlk bytes.
__device__ __forceinline__ uint32_t quad_at(int r, int c) {
  return (c >> 6) * kBlk + chunk_at(r, (c & 63) >> 3) + ((c & 4) << 1);
}
__device__ __forceinline__ uint32_t kmajor(uint32_t addr) { return (uint32_t)tc::sdesc(addr, 16, 1024); }
__device__ __forceinline__ uint32_t mnmajor(uint32_t addr) { return (uint32_t)tc::sdesc(addr, kBlk, 1024); }
__host__ __device__ constexpr uint32_t kstep(int ks) { return ((ks >> 2) * kBlk + (ks & 3) * 32) >> 4; }
__host__ __device__ constexpr uint32_t mnstep(int ks) { return ks * 2048 >> 4; }
// Four values of a row of `width`, zeros past it.
template <typename T>
__device__ __forceinline__ float4 load4(const T* p, int c, int width, bool vec);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p, int c, int width, bool vec) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec) {
    if (c < width) v = *(const float4*)(p + c);
    return v;
  }
  if (c < width) v.x = p[c];
  if (c + 1 < width) v.y = p[c + 1];
  if (c + 2 < width) v.z = p[c + 2];
  if (c + 3 < width) v.w = p[c + 3];
  return v;
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p, int c, int width, bool vec) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec) {
    if (c < width) {
      const uint2 w = *(const uint2*)(p + c);
      v = make_float4(lo_f(w.x), hi_f(w.x), lo_f(w.y), hi_f(w.y));
    }
    return v;
  }
  if (c < width) v.x = to_f32(p[c]);
  if (c + 1 < width) v.y = to_f32(p[c + 1]);
  if (c + 2 < width) v.z = to_f32(p[c + 2]);
  if (c + 3 < width) v.w = to_f32(p[c + 3]);
  return v;
}
template <typename T>
__device__ __forceinline__ bool vec_rows(const void* p, int width, int64_t stride) {
  return width % 4 == 0 && stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(T) - 1)) == 0;
}

// One block's walk (see k_linattn_mma.cu). NB: 64-column blocks of N.
template <typename T, int NB, bool SUMMARY>
__device__ __forceinline__ void walk(const LaArgs& a, int ri, int pt, int bh, int seg, char* raw) {
  constexpr int IP = sizeof(T) == 4 ? 3 : 1;  // parts of an input
  constexpr int NK = 64 * NB;
  constexpr int SC = NB == 2 ? 16 : 8;                     // state columns a thread
  constexpr int KQ = (kC * NK / 4 + kThreads - 1) / kThreads;  // quads of K a thread
  constexpr int VQ = (kC * 16 + kThreads - 1) / kThreads;      // quads of V a thread
  const LaRole& r = a.role[ri];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, grp = warp >> 2;
  const int b = bh / a.H, h = bh - b * a.H;
  const int N = r.N, P = r.P, p_lo = 64 * pt;
  int64_t row0, len;
  la_rows(a, b, &row0, &len);
  const int64_t s0 = seg * a.seg_len, s1 = min(len, s0 + a.seg_len);
  const int64_t last_seg = len > 0 ? (len - 1) / a.seg_len : 0;
  if (seg > last_seg) return;
  if (SUMMARY && seg == (r.reverse ? 0 : last_seg)) return;  // the prefix pass never reads it
  const bool first = seg == (r.reverse ? last_seg : 0), last = seg == (r.reverse ? 0 : last_seg);
  const int nchunk = s1 > s0 ? (int)((s1 - s0 + kC - 1) / kC) : 0;
  const T* gq = (const T*)r.q + (int64_t)(h / r.q_rep) * N;
  const T* gk = (const T*)r.k + (int64_t)(h / r.k_rep) * N;
  const T* gv = (const T*)r.v + (int64_t)(h / r.v_rep) * P;
  const bool qvec = vec_rows<T>(gq, N, r.qs), kvec = vec_rows<T>(gk, N, r.ks),
             vvec = vec_rows<T>(gv, P, r.vs);

  const uint32_t base = tc::smem_u32(raw);
  constexpr uint32_t kPartK = NB * kBlk, kPartV = kBlk, kPartS = state_bytes(NB);
  const uint32_t sK = base, sV = sK + kParts * kPartK, sX = sV + kParts * kPartV,
                 sS = sX + kParts * kPartV;
  Small& sm = *reinterpret_cast<Small*>(raw + tile_bytes(2));
  uint64_t *barA = &sm.bar[0], *barB = &sm.bar[1], *barC = &sm.bar[2];
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) tc::bar_init(&sm.bar[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;");
  }
  const float ld = a.log_decay[h];
  if (tid < kC + 20) sm.pw[tid] = la_power(ld, tid);
  if (tid < 16) sm.col[tid] = la_power(ld, r.reverse ? tid : 15 - tid);
  if (warp == 0) tc::tmem_alloc(&sm.tmem, kCols);
  __syncthreads();
  const uint32_t tm = sm.tmem, tw = tm + ((uint32_t)(32 * quad) << 16);

  auto chunk_row = [&](int ci) { return s0 + (int64_t)(r.reverse ? nchunk - 1 - ci : ci) * kC; };
  auto chunk_len = [&](int ci) { return (int)min((int64_t)kC, s1 - chunk_row(ci)); };
  // this thread's rows of the next chunk
  float4 rk[KQ], rv[VQ], rq[NB * 4];
  auto load_k = [&](int ci) {
    const T* g = gk + (row0 + chunk_row(ci)) * r.ks;
    const int n = chunk_len(ci);
#pragma unroll
    for (int x = 0; x < KQ; ++x) {
      const int e = tid + x * kThreads, t = e / (NK / 4), c = e % (NK / 4) * 4;
      rk[x] = t < n ? load4<T>(g + t * r.ks, c, N, kvec) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  auto load_v = [&](int ci) {
    const T* g = gv + (row0 + chunk_row(ci)) * r.vs;
    const int n = chunk_len(ci);
#pragma unroll
    for (int x = 0; x < VQ; ++x) {
      const int e = tid + x * kThreads, t = e / 16, c = p_lo + e % 16 * 4;
      rv[x] = t < n ? load4<T>(g + t * r.vs, c, P, vvec) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  // queries: tensor-memory row 32 quad + lane, columns NB * 16 grp ..
  auto load_q = [&](int ci) {
    const int t = 32 * quad + lane;
    const T* g = gq + (row0 + chunk_row(ci) + t) * r.qs;
    const bool in = t < chunk_len(ci);
#pragma unroll
    for (int x = 0; x < NB * 4; ++x)
      rq[x] = in ? load4<T>(g, NB * 16 * grp + 4 * x, N, qvec) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  auto put_k = [&]() {
#pragma unroll
    for (int x = 0; x < KQ; ++x) {
      const int e = tid + x * kThreads, t = e / (NK / 4), c = e % (NK / 4) * 4;
      if (t >= kC) continue;
      uint32_t lo[3], hi[3];
      cut2(rk[x].x, rk[x].y, lo);
      cut2(rk[x].z, rk[x].w, hi);
#pragma unroll
      for (int p = 0; p < IP; ++p) sts2(sK + p * kPartK + quad_at(t, c), lo[p], hi[p]);
    }
  };
  auto put_v = [&](int n) {  // V and V^
#pragma unroll
    for (int x = 0; x < VQ; ++x) {
      const int e = tid + x * kThreads, t = e / 16, c = e % 16 * 4;
      if (t >= kC) continue;
      uint32_t lo[3], hi[3];
      if (!SUMMARY) {
        cut2(rv[x].x, rv[x].y, lo);
        cut2(rv[x].z, rv[x].w, hi);
#pragma unroll
        for (int p = 0; p < IP; ++p) sts2(sV + p * kPartV + quad_at(t, c), lo[p], hi[p]);
      }
      const float w = t < n ? r.kv * sm.pw[r.reverse ? t : n - 1 - t] : 0.f;
      cut2(w * rv[x].x, w * rv[x].y, lo);
      cut2(w * rv[x].z, w * rv[x].w, hi);
#pragma unroll
      for (int p = 0; p < 3; ++p) sts2(sX + p * kPartV + quad_at(t, c), lo[p], hi[p]);
    }
  };
  auto put_q = [&]() {
#pragma unroll
    for (int y = 0; y < NB; ++y) {
      uint32_t pc[8][3];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        cut2(rq[4 * y + x].x, rq[4 * y + x].y, pc[2 * x]);
        cut2(rq[4 * y + x].z, rq[4 * y + x].w, pc[2 * x + 1]);
      }
#pragma unroll
      for (int p = 0; p < IP; ++p) {
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = pc[e][p];
        st8(tw + kColQ + 64 * p + NB * 8 * grp + 8 * y, v);
      }
    }
    tc::tmem_wait_st();
  };

  const int srow = NB == 2 ? 32 * quad + lane : 16 * quad + (lane & 15);
  const int scol = NB == 2 ? 16 * grp : 16 * grp + 8 * (lane >> 4);
  float st[SC];
  float* entry = a.entry ? a.entry + ri * a.entry_role +
                               ((int64_t)seg * a.B * a.H + bh) * ((int64_t)N * P)
                         : nullptr;
  const int64_t sbase = (int64_t)bh * N * P;
#pragma unroll
  for (int j = 0; j < SC; ++j) {
    const int p = p_lo + scol + j;
    st[j] = 0.f;
    if (!SUMMARY && srow < N && p < P) {
      if (a.nseg > 1) st[j] = entry[(int64_t)p * N + srow];
      else if (r.init) st[j] = r.init[sbase + (int64_t)p * r.sp + (int64_t)srow * r.sn];
    }
  }
  auto put_state = [&]() {
    uint32_t pc[SC / 2][3];
#pragma unroll
    for (int j = 0; j < SC / 2; ++j) cut2(st[2 * j], st[2 * j + 1], pc[j]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int c = 0; c < SC / 8; ++c)
        sts(sS + p * kPartS + chunk_at(srow, scol / 8 + c),
            make_uint4(pc[4 * c][p], pc[4 * c + 1][p], pc[4 * c + 2][p], pc[4 * c + 3][p]));
  };
  bool ok = true;
  int pend[3] = {-1, -1, -1};  // thread 0: phases it still has to see end
  if (nchunk > 0) {
    load_k(0);
    load_v(0);
    if (!SUMMARY) load_q(0);
    put_k();
    put_v(chunk_len(0));
    if (!SUMMARY) put_q();
  }
  if (!SUMMARY) put_state();
  // pairs of parts of a product with `xa` and `xb` parts, the largest last
  auto products = [&](int xa, int xb, auto&& one) {
    bool acc = false;
    for (int s = 2; s >= 0; --s)
      for (int i = 0; i <= s; ++i) {
        if (i >= xa || s - i >= xb) continue;
        one(i, s - i, acc);
        acc = true;
      }
  };

  for (int ci = 0; ci < nchunk && ok; ++ci) {
    const uint32_t ph = ci & 1;
    const int64_t t0 = chunk_row(ci);
    const int n = chunk_len(ci);
    const int shift = ci == 0 && first ? r.shift : 0;
    const int ksn = (n + 15) / 16;
    const bool more = ci + 1 < nchunk;
    tc::fence_before();
    tc::fence_async_smem();
    ok = __syncthreads_and(ok);  // operands of this chunk and the state are in place
    if (!ok) break;
    if (tid == 0) {
      tc::fence_after();
      if (!SUMMARY) {
        const int ksq = (N + 15) / 16;
        products(IP, IP, [&](int i, int j, bool acc) {
          for (int ks = 0; ks < ksq; ++ks)
            mma_ts(tm + kColA, tm + kColQ + 64 * i, 8 * ks, kmajor(sK + j * kPartK), kstep(ks),
                   idesc_bf16(128, kC, 0, 0), acc || ks > 0);
        });
        products(IP, 3, [&](int i, int j, bool acc) {
          for (int ks = 0; ks < ksq; ++ks)
            mma_ts(tm + kColI, tm + kColQ + 64 * i, 8 * ks, mnmajor(sS + j * kPartS), mnstep(ks),
                   idesc_bf16(128, 64, 0, 1), acc || ks > 0);
        });
        tc::commit(barA);
        pend[0] = ph;
      }
      products(IP, 3, [&](int i, int j, bool acc) {
        for (int ks = 0; ks < ksn; ++ks)
          mma_ss(tm + kColS, mnmajor(sK + i * kPartK), mnstep(ks), mnmajor(sX + j * kPartV), mnstep(ks),
                 idesc_bf16(NK, 64, 1, 1), acc || ks > 0);
      });
      tc::commit(barB);
      pend[1] = ph;
    }
    __syncwarp();
    if (more) {
      load_k(ci + 1);
      load_v(ci + 1);
      if (!SUMMARY) load_q(ci + 1);
    }
    if (!SUMMARY) {
      ok = wait_phase(barA, ph, kBudget) && ok;
      tc::fence_after();
      // P: row i of this thread, 16-column blocks grp and grp + 4, into Q's columns
      const int i = 32 * quad + lane;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int jb = grp + 4 * x, j0 = 16 * jb;
        if (jb >= kC / 16) continue;
        uint32_t pc[3][8] = {};
        if (!(r.reverse ? j0 + 15 < 32 * quad : j0 > 32 * quad + 31)) {
          float s[16];
          ld16(tw + kColA + j0, s);
          tc::tmem_wait_ld();
          if (r.reverse ? j0 >= 32 * quad + 31 : j0 + 15 <= 32 * quad) {
            const float f = r.intra * sm.pw[r.reverse ? j0 - i : i - j0 - 15];
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] *= f * sm.col[e];
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int d = r.reverse ? j0 + e - i : i - j0 - e;
              s[e] = d >= 0 ? s[e] * (r.intra * sm.pw[d < 0 ? 0 : d]) : 0.f;
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t t3[3];
            cut2(s[2 * e], s[2 * e + 1], t3);
            pc[0][e] = t3[0];
            pc[1][e] = t3[1];
            pc[2][e] = t3[2];
          }
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) st8(tw + kColQ + 64 * p + 8 * jb, pc[p]);
      }
      tc::tmem_wait_st();
      tc::fence_before();
      ok = __syncthreads_and(ok);
      if (!ok) break;
      if (tid == 0) {
        pend[0] = -1;
        tc::fence_after();
        products(3, IP, [&](int x, int y, bool acc) {
          for (int ks = 0; ks < ksn; ++ks)
            mma_ts(tm + kColO, tm + kColQ + 64 * x, 8 * ks, mnmajor(sV + y * kPartV), mnstep(ks),
                   idesc_bf16(128, 64, 0, 1), acc || ks > 0);
        });
        tc::commit(barC);
        pend[2] = ph;
      }
      __syncwarp();
    }
    ok = wait_phase(barB, ph, kBudget) && ok;
    tc::fence_after();
    {
      const float dec = sm.pw[n - shift];
      float kv[SC];
      if constexpr (NB == 2) ld16(tw + kColS + scol, kv);
      else ld_m64_8(tw + kColS + 16 * grp, kv);
      tc::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < SC; ++j) st[j] = fmaf(dec, st[j], kv[j]);
      if (!SUMMARY) put_state();
    }
    if (more) put_k();
    if (SUMMARY) {
      if (more) put_v(chunk_len(ci + 1));
      continue;
    }
    ok = wait_phase(barC, ph, kBudget) && ok;
    tc::fence_after();
    if (more) {
      put_v(chunk_len(ci + 1));
      put_q();
    }
    {
      const int i = 32 * quad + lane, at = min(max(r.reverse ? n - 1 - i : i, 0), kC - 1);
      const float f = r.inter * sm.pw[at + 1 - shift];
      const int c0 = 16 * grp;
      float o[16], in[16];
      ld16(tw + kColO + c0, o);
      ld16(tw + kColI + c0, in);
      tc::tmem_wait_ld();
      if (i < n) {
        const int64_t at_out = (row0 + t0 + i) * r.os + (int64_t)h * P + p_lo + c0;
        float* of = (float*)r.out + at_out;
        T* ot = (T*)r.out + at_out;
        const bool f32 = r.out_rep > 1 || sizeof(T) == 4;
        const bool vec = f32 && P % 4 == 0 && r.os % 4 == 0 && (reinterpret_cast<uintptr_t>(r.out) & 15) == 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = fmaf(f, in[e], o[e]);
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          if (vec) {
            if (p_lo + c0 + e < P) *(float4*)(of + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            continue;
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            if (p_lo + c0 + e + y >= P) continue;
            if (f32) of[e + y] = o[e + y];
            else ot[e + y] = from_f32<T>(o[e + y]);
          }
        }
      }
    }
  }

  if (tid == 0 && !ok) {
    atomicExch(a.status, kStatusTimeout);
    for (int i = 0; i < 3; ++i)
      if (pend[i] >= 0 && !wait_phase(&sm.bar[i], pend[i], kBudget)) atomicExch(a.status, kStatusUndrained);
  }
  if (ok && (SUMMARY || (r.fin && last))) {
    const float f = !SUMMARY && len > 0 && r.fin_shift ? sm.pw[1] : 1.f;
#pragma unroll
    for (int j = 0; j < SC; ++j) {
      const int p = p_lo + scol + j;
      if (srow < N && p < P) {
        if (SUMMARY) entry[(int64_t)p * N + srow] = st[j];
        else r.fin[sbase + (int64_t)p * r.sp + (int64_t)srow * r.sn] = f * st[j];
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tm, kCols);
}

template <typename T, bool SUMMARY>
__global__ void __launch_bounds__(kThreads, 1)
    k_la_split(const __grid_constant__ LaArgs a, int items) {
  extern __shared__ __align__(1024) char raw[];
  la_clear_status<SUMMARY>(a);
  int item = blockIdx.x % items, ri = 0;
  const int unit = blockIdx.x / items;
  while (item >= (a.role[ri].P + 63) / 64) item -= (a.role[ri++].P + 63) / 64;
  const int bh = unit % (a.B * a.H), seg = unit / (a.B * a.H);
  if (a.role[ri].N > 64) walk<T, 2, SUMMARY>(a, ri, item, bh, seg, raw);
  else walk<T, 1, SUMMARY>(a, ri, item, bh, seg, raw);
}

}  // namespace

cudaError_t launch_la_split(const LaArgs& a, LaPass pass, cudaStream_t s) {
  int items = 0;
  for (int i = 0; i < a.nrole; ++i) items += (a.role[i].P + 63) / 64;
  const unsigned grid = (unsigned)((int64_t)a.B * a.H * a.nseg * items);
  auto go = [&](auto kernel) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, kSmem, s>>>(a, items);
    count_launches(1);
    return cudaGetLastError();
  };
  if (a.dtype == M3_DTYPE_FP32)
    return pass == kLaSummary ? go(k_la_split<float, true>) : go(k_la_split<float, false>);
  return pass == kLaSummary ? go(k_la_split<__nv_bfloat16, true>) : go(k_la_split<__nv_bfloat16, false>);
}

}  // namespace m3
