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
// One block an SM. While the products of a chunk run, the next chunk's rows are
// fetched into L2; K's are cut and stored as soon as K^T V^ has read the tile, those
// of Q and V as soon as P V has.
//
// At N = 128, P = 64 a chunk's 180 products (48 Q K^T, 48 Q S, 42 K^T V^, 42 P V) keep
// the tensor cores active for some 7,000 of its 17,500 cycles (4 x 2048 tokens, one
// block an SM: 40 % of the active cycles by the counter); the rest is the cutting, for
// which the tiles that the products read have to be free, and loads that go through
// what 217 KB of shared memory leave of the L1. Measured on 2 x 16,384 tokens, 32
// heads, 4 groups: 0.81 ms, where float32 arithmetic on the CUDA cores took 4.6 ms and
// the bytes would take 0.10. At N > 64 nothing spills: with no L1 to hold them, spilled
// registers cost as much as the loads they hide. At N <= 64 a thread spills 20 bytes,
// and with bfloat16 operands at N > 64 12.
#include "linattn_mma.cuh"

namespace m3 {
namespace {

constexpr int kC = 112;
constexpr int kWarps = 16;  // compute warps; one more issues
constexpr int kThreads = 32 * (kWarps + 1);
constexpr long long kBudget = 4000000000LL;  // clock cycles, about 2 s
constexpr uint32_t kBlk = kC * 128;          // bytes of a 64-column block of a tile part
constexpr int kParts = 3;
constexpr uint32_t kColQ = 0, kColA = 192, kColO = 320, kColI = 384, kColS = 448, kCols = 512;

__host__ __device__ constexpr uint32_t state_bytes(int nb) { return nb * 8192; }
__host__ __device__ constexpr uint32_t tile_bytes(int nb) {
  return kParts * (nb * kBlk + 2 * kBlk + state_bytes(nb));
}
enum Bar {
  kBarQ,  // Q, K and S are in place, O and Oi read
  kBarX,  // V and V^ are in place
  kBarA,  // A and Oi are done
  kBarB,  // K^T V^ is done
  kBarP,  // P is written
  kBarC,  // O is done
  kBars
};
struct Small {
  alignas(16) float col[16];  // column factors of a 16-token block
  float pw[kC + 20];          // lam^d, d <= 128
  uint64_t bar[kBars];
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

// One block's walk (see k_linattn_mma.cu: warps 0..15 compute, one lane of warp 16
// issues the products, and they meet at mbarriers with bounded waits). NB:
// 64-column blocks of N.
template <typename T, int NB, bool SUMMARY>
__device__ __forceinline__ void walk(const LaCall& a, int pt, int bh, int seg, char* raw) {
  constexpr int IP = sizeof(T) == 4 ? 3 : 1;  // parts of an input
  constexpr int NK = 64 * NB;
  constexpr int SC = NB == 2 ? 16 : 8;                             // state columns a thread
  constexpr int KQ = (kC * NK / 4 + 32 * kWarps - 1) / (32 * kWarps);  // quads of K a thread
  constexpr int VQ = (kC * 16 + 32 * kWarps - 1) / (32 * kWarps);      // quads of V a thread
  const LaRole& r = a.role;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, grp = (warp >> 2) & 3;
  const int b = bh / a.H, h = bh - b * a.H;
  const int N = r.N, P = r.P, p_lo = 64 * pt;
  const bool rev = r.reverse;
  int64_t seq0, len;
  la_rows(a, b, &seq0, &len);
  const int last_seg = len > 0 ? (int)((len - 1) / a.seg_len) : 0;
  if (seg > last_seg) return;
  const int row0 = (int)(seq0 + seg * a.seg_len);  // the segment's rows
  const int ntok = (int)min(len - seg * a.seg_len, a.seg_len);
  if (SUMMARY && seg == (rev ? 0 : last_seg)) return;  // the prefix pass never reads it
  const bool first = seg == (rev ? last_seg : 0), last = seg == (rev ? 0 : last_seg);
  const int nchunk = (ntok + kC - 1) / kC;

  const uint32_t base = tc::smem_u32(raw);
  constexpr uint32_t kPartK = NB * kBlk, kPartV = kBlk, kPartS = state_bytes(NB);
  const uint32_t sK = base, sV = sK + kParts * kPartK, sX = sV + kParts * kPartV,
                 sS = sX + kParts * kPartV;
  Small& sm = *reinterpret_cast<Small*>(raw + tile_bytes(2));
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) tc::bar_init(&sm.bar[i], i == kBarQ || i == kBarX || i == kBarP ? kWarps : 1);
    asm volatile("fence.mbarrier_init.release.cluster;");
  }
  const float ld = a.log_decay[h];
  if (tid < kC + 20) sm.pw[tid] = la_power(ld, tid);
  if (tid < 16) sm.col[tid] = la_power(ld, rev ? tid : 15 - tid);
  if (warp == 0) tc::tmem_alloc(&sm.tmem, kCols);
  __syncthreads();
  const uint32_t tm = sm.tmem, tw = tm + ((uint32_t)(32 * quad) << 16);
  bool ok = true;
  auto wait = [&](int bar, uint32_t phase) {
    if (ok && !wait_phase(&sm.bar[bar], phase, kBudget)) ok = false;
    return ok;
  };
  auto chunk_row = [&](int ci) { return row0 + (rev ? nchunk - 1 - ci : ci) * kC; };
  auto chunk_len = [&](int ci) { return min(kC, row0 + ntok - chunk_row(ci)); };

  if (warp == kWarps) {
    const bool lead = tc::elect_one();
    uint32_t open = 0, odd = 0;  // barriers with products in flight, and their phase
    auto commit = [&](int bar, int ci) {
      if (lead) tc::commit(&sm.bar[bar]);
      open |= 1u << bar;
      odd = (odd & ~(1u << bar)) | (uint32_t)(ci & 1) << bar;
    };
    // pairs of parts of a product with `xa` and `xb` parts, the largest last
    auto products = [&](int xa, int xb, auto&& one) {
      bool acc = false;
#pragma unroll 1
      for (int s = 2; s >= 0; --s)
#pragma unroll 1
        for (int i = 0; i <= s; ++i) {
          if (i >= xa || s - i >= xb) continue;
          one(i, s - i, acc);
          acc = true;
        }
    };
    const int ksq = (N + 15) / 16;
    const uint32_t dK = kmajor(sK), dKt = mnmajor(sK), dV = mnmajor(sV), dX = mnmajor(sX), dS = mnmajor(sS);
    for (int ci = 0; ci < nchunk; ++ci) {
      const uint32_t ph = ci & 1;
      const int ksn = (chunk_len(ci) + 15) / 16;
      if (!SUMMARY) {
        if (!wait(kBarQ, ph)) break;
        tc::fence_after();
        products(IP, IP, [&](int i, int j, bool acc) {
#pragma unroll
          for (int ks = 0; ks < NK / 16; ++ks)
            if (ks < ksq && lead)
              mma_ts(tm + kColA, tm + kColQ + 64 * i, 8 * ks, dK + j * (kPartK >> 4), kstep(ks),
                     idesc_bf16(128, kC, 0, 0), acc || ks > 0);
        });
        products(IP, 3, [&](int i, int j, bool acc) {
#pragma unroll
          for (int ks = 0; ks < NK / 16; ++ks)
            if (ks < ksq && lead)
              mma_ts(tm + kColI, tm + kColQ + 64 * i, 8 * ks, dS + j * (kPartS >> 4), mnstep(ks),
                     idesc_bf16(128, 64, 0, 1), acc || ks > 0);
        });
        commit(kBarA, ci);
      }
      if (!wait(kBarX, ph)) break;
      tc::fence_after();
      products(IP, 3, [&](int i, int j, bool acc) {
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          if (ks < ksn && lead)
            mma_ss(tm + kColS, dKt + i * (kPartK >> 4), mnstep(ks), dX + j * (kPartV >> 4), mnstep(ks),
                   idesc_bf16(NK, 64, 1, 1), acc || ks > 0);
      });
      commit(kBarB, ci);
      if (!SUMMARY) {
        if (!wait(kBarP, ph)) break;
        tc::fence_after();
        products(3, IP, [&](int i, int j, bool acc) {
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks)
            if (ks < ksn && lead)
              mma_ts(tm + kColO, tm + kColQ + 64 * i, 8 * ks, dV + j * (kPartV >> 4), mnstep(ks),
                     idesc_bf16(128, 64, 0, 1), acc || ks > 0);
        });
        commit(kBarC, ci);
      }
    }
    if (!ok) {  // bounded waits for what may still be in flight
      if (lead) atomicExch(a.status, kStatusTimeout);
      for (int i = 0; i < kBars; ++i)
        if ((open >> i & 1) && !wait_phase(&sm.bar[i], odd >> i & 1, kBudget) && lead)
          atomicExch(a.status, kStatusUndrained);
    }
    __syncwarp();
  } else {
    auto arrive = [&](int bar) {
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sm.bar[bar]);
    };
    const T* gq = (const T*)r.q + (int64_t)(h / r.q_rep) * N;
    const T* gk = (const T*)r.k + (int64_t)(h / r.k_rep) * N;
    const T* gv = (const T*)r.v + (int64_t)(h / r.v_rep) * P;
    const bool qvec = vec_rows<T>(gq, N, r.qs), kvec = vec_rows<T>(gk, N, r.ks), vvec = vec_rows<T>(gv, P, r.vs);
    float4 rk[KQ], rv[VQ], rq[4];  // this thread's values of the next chunk
    auto load_k = [&](int ci, int from, int to) {  // quads [from, to)
      const T* g = gk + (int64_t)chunk_row(ci) * r.ks;
      const int n = chunk_len(ci);
#pragma unroll
      for (int x = 0; x < KQ; ++x) {
        if (x < from || x >= to) continue;
        const int t = tid / (NK / 4) + x * (32 * kWarps / (NK / 4)), c = tid % (NK / 4) * 4;
        rk[x] = t < n ? load4<T>(g + t * r.ks, c, N, kvec) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    auto load_v = [&](int ci) {
      const T* g = gv + (int64_t)chunk_row(ci) * r.vs;
      const int n = chunk_len(ci);
#pragma unroll
      for (int x = 0; x < VQ; ++x) {
        const int t = tid / 16 + x * 2 * kWarps, c = p_lo + tid % 16 * 4;
        rv[x] = t < n ? load4<T>(g + t * r.vs, c, P, vvec) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    // Queries: this warp's 32 rows, 16 columns (half y of its NB) at a time, four
    // lanes a row; turn_q() leaves each lane with the columns of one row.
    auto load_q = [&](int ci, int y) {
      const int n = chunk_len(ci);
      const T* g = gq + (int64_t)chunk_row(ci) * r.qs;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int t = 32 * quad + lane / 4 + 8 * x;
        rq[x] = t < n ? load4<T>(g + t * r.qs, NB * 16 * grp + 16 * y + lane % 4 * 4, N, qvec)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    // Register x of lane (l / 4, c) holds quad c of row 8 x + l / 4. The register's
    // index and the lane's low bits change places, a bit a step, and quad x of row i
    // comes to lie in register x.
    auto turn_q = [&]() {
#pragma unroll
      for (int bit = 1; bit < 4; bit *= 2) {
        const bool up = lane & bit;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (x & bit) continue;
          const float4 keep = up ? rq[x | bit] : rq[x];
          float4 give = up ? rq[x] : rq[x | bit];
          give.x = __shfl_xor_sync(0xffffffffu, give.x, bit);
          give.y = __shfl_xor_sync(0xffffffffu, give.y, bit);
          give.z = __shfl_xor_sync(0xffffffffu, give.z, bit);
          give.w = __shfl_xor_sync(0xffffffffu, give.w, bit);
          rq[x] = up ? give : keep;
          rq[x | bit] = up ? keep : give;
        }
      }
    };
    // Rows of a later chunk into L2, one a thread. With 217 KB of shared memory the
    // L1 has room for some 28 KB of loads in flight, so their latency has to be L2's.
    auto prefetch = [&](const T* g, int64_t stride, int width, int ci, int t) {
      if (ci >= nchunk || t < 0 || t >= chunk_len(ci)) return;
      const char* p = (const char*)(g + (int64_t)(chunk_row(ci) + t) * stride);
      const uint32_t skip = (uint32_t)(16 - ((uintptr_t)p & 15)) & 15, bytes = width * (uint32_t)sizeof(T);
      if (bytes > skip + 15) tc::prefetch_l2(p + skip, (bytes - skip) & ~15u);
    };
    // A thread's quads of a tile lie a multiple of eight rows apart, so their places
    // differ by constants.
    auto put2 = [](char* at, uint32_t lo, uint32_t hi) { *reinterpret_cast<uint2*>(at) = make_uint2(lo, hi); };
    constexpr int kRowsK = 32 * kWarps / (NK / 4), kRowsV = 32 * kWarps / 16;
    static_assert(kRowsK % 8 == 0 && kRowsV % 8 == 0, "");
    char* const at_k = raw + quad_at(tid / (NK / 4), tid % (NK / 4) * 4);
    char* const at_v = raw + kParts * kPartK + quad_at(tid / 16, tid % 16 * 4);
    auto put_k = [&]() {
#pragma unroll
      for (int x = 0; x < KQ; ++x) {
        if (tid / (NK / 4) + x * kRowsK >= kC) continue;
        uint32_t lo[3], hi[3];
        cut2(rk[x].x, rk[x].y, lo);
        cut2(rk[x].z, rk[x].w, hi);
#pragma unroll
        for (int p = 0; p < IP; ++p) put2(at_k + p * kPartK + x * kRowsK * 128, lo[p], hi[p]);
      }
    };
    auto put_v = [&](int n) {  // V and V^
#pragma unroll
      for (int x = 0; x < VQ; ++x) {
        const int t = tid / 16 + x * kRowsV;
        if (t >= kC) continue;
        uint32_t lo[3], hi[3];
        if (!SUMMARY) {
          cut2(rv[x].x, rv[x].y, lo);
          cut2(rv[x].z, rv[x].w, hi);
#pragma unroll
          for (int p = 0; p < IP; ++p) put2(at_v + p * kPartV + x * kRowsV * 128, lo[p], hi[p]);
        }
        const float w = t < n ? r.kv * sm.pw[rev ? t : n - 1 - t] : 0.f;
        cut2(w * rv[x].x, w * rv[x].y, lo);
        cut2(w * rv[x].z, w * rv[x].w, hi);
#pragma unroll
        for (int p = 0; p < 3; ++p) put2(at_v + (kParts + p) * kPartV + x * kRowsV * 128, lo[p], hi[p]);
      }
    };
    auto put_q = [&](int y) {
      turn_q();
      uint32_t pc[3][8];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t lo[3], hi[3];
        cut2(rq[x].x, rq[x].y, lo);
        cut2(rq[x].z, rq[x].w, hi);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          pc[p][2 * x] = lo[p];
          pc[p][2 * x + 1] = hi[p];
        }
      }
#pragma unroll
      for (int p = 0; p < IP; ++p) st8(tw + kColQ + 64 * p + NB * 8 * grp + 8 * y, pc[p]);
    };
    const int srow = NB == 2 ? 32 * quad + lane : 16 * quad + (lane & 15);
    const int scol = NB == 2 ? 16 * grp : 16 * grp + 8 * (lane >> 4);
    float st[SC];
    float* entry = a.entry ? a.entry + ((int64_t)seg * a.B * a.H + bh) * ((int64_t)N * P) : nullptr;
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
#pragma unroll
      for (int c = 0; c < SC / 8; ++c) {
        uint32_t pc[4][3];
#pragma unroll
        for (int j = 0; j < 4; ++j) cut2(st[8 * c + 2 * j], st[8 * c + 2 * j + 1], pc[j]);
#pragma unroll
        for (int p = 0; p < 3; ++p)
          sts(sS + p * kPartS + chunk_at(srow, scol / 8 + c), make_uint4(pc[0][p], pc[1][p], pc[2][p], pc[3][p]));
      }
    };
    // this thread's row of A, P and O: the token that its tensor-memory row holds
    const int i = 32 * quad + lane % 4 * 8 + lane / 4;
    // row factors of this warp's blocks of 16 columns before the diagonal
    float fac[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int d = rev ? 16 * (grp + 4 * x) - i : i - 16 * (grp + 4 * x) - 15;
      fac[x] = d < 0 ? 0.f : r.intra * sm.pw[d];
    }
    if (nchunk > 0) {
      load_k(0, 0, KQ);
      load_v(0);
      put_k();
      if (!SUMMARY) {
        put_state();
#pragma unroll
        for (int y = 0; y < NB; ++y) {
          load_q(0, y);
          put_q(y);
        }
        tc::tmem_wait_st();
        tc::fence_before();
        tc::fence_async_smem();
        arrive(kBarQ);
      }
      put_v(chunk_len(0));
      tc::fence_async_smem();
      arrive(kBarX);
    }
    for (int ci = 0; ci < nchunk; ++ci) {
      const uint32_t ph = ci & 1;
      const int n = chunk_len(ci);
      const int shift = ci == 0 && first ? r.shift : 0;
      const bool more = ci + 1 < nchunk;
      prefetch(gk, r.ks, N, ci + 1, tid);
      prefetch(gv + p_lo, r.vs, min(64, P - p_lo), ci + 1, tid - kC);
      if (!SUMMARY) prefetch(gq, r.qs, N, ci + 1, tid - 2 * kC);
      if (!SUMMARY) {
        if (!wait(kBarA, ph)) break;
        tc::fence_after();
        // P: 16-column blocks grp and grp + 4, into Q's columns
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int jb = grp + 4 * x, j0 = 16 * jb;
          if (jb >= kC / 16) continue;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t pc[3][4] = {};
            if (rev ? j0 + 15 >= 32 * quad : j0 <= 32 * quad + 31) {
              float s[8];
              ld8(tw + kColA + j0 + 8 * y, s);
              tc::tmem_wait_ld();
              if (rev ? j0 >= 32 * quad + 31 : j0 + 15 <= 32 * quad) {
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                  const float4 w = *reinterpret_cast<const float4*>(&sm.col[8 * y + e]);
                  s[e] *= fac[x] * w.x;
                  s[e + 1] *= fac[x] * w.y;
                  s[e + 2] *= fac[x] * w.z;
                  s[e + 3] *= fac[x] * w.w;
                }
              } else {
                int d0 = rev ? j0 + 8 * y - i : i - j0 - 8 * y;
                const int step = rev ? 1 : -1;
                asm volatile("" : "+r"(d0));  // not worth registers between chunks
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int d = d0 + step * e;
                  const float w = r.intra * sm.pw[max(d, 0)];
                  s[e] = d >= 0 ? s[e] * w : 0.f;
                }
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t t3[3];
                cut2(s[2 * e], s[2 * e + 1], t3);
                pc[0][e] = t3[0];
                pc[1][e] = t3[1];
                pc[2][e] = t3[2];
              }
            }
#pragma unroll
            for (int p = 0; p < 3; ++p) st4(tw + kColQ + 64 * p + 8 * jb + 4 * y, pc[p]);
          }
        }
        tc::tmem_wait_st();
        tc::fence_before();
        arrive(kBarP);
      }
      constexpr int kEarly = KQ / 2;  // keys loaded while K^T V^ runs: as many as registers are left
      if (more) load_k(ci + 1, 0, kEarly);
      if (!wait(kBarB, ph)) break;
      tc::fence_after();
      {
        const float dec = sm.pw[n - shift];
        float kv[SC];
        if constexpr (NB == 2) ld16(tw + kColS + scol, kv);
        else ld_m64_8(tw + kColS + 16 * grp, kv);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < SC; ++j) st[j] = fmaf(dec, st[j], kv[j]);
        if (!SUMMARY && more) put_state();
      }
      tc::fence_before();
      if (more) {
        load_k(ci + 1, kEarly, KQ);
        put_k();
      }
      if (SUMMARY) {
        if (more) {
          load_v(ci + 1);
          put_v(chunk_len(ci + 1));
          tc::fence_async_smem();
          arrive(kBarX);
        }
        continue;
      }
      if (more) load_q(ci + 1, 0);
      if (!wait(kBarC, ph)) break;
      tc::fence_after();
      {
        const int at = min(max(rev ? n - 1 - i : i, 0), kC - 1);
        const float f = r.inter * sm.pw[at + 1 - shift];
        const bool f32 = r.out_rep > 1 || sizeof(T) == 4;
        const bool vec = f32 && P % 4 == 0 && r.os % 4 == 0 && (reinterpret_cast<uintptr_t>(r.out) & 15) == 0;
        const int64_t base_out = (int64_t)chunk_row(ci) * r.os + (int64_t)h * P + p_lo;
        // rows of lanes l < 16 and l + 16
        constexpr int kHalf = 4;
        const int i_lo = i - (lane & 16 ? kHalf : 0);
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // eight columns at a time: the queries are in registers too
          const int c0 = 16 * grp + 8 * x;
          float o[8], in[8];
          ld8(tw + kColO + c0, o);
          ld8(tw + kColI + c0, in);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = fmaf(f, in[e], o[e]);
          if (vec) {
            // lanes l and l ^ 16 exchange halves: each writes four columns of both
            // rows, so that a row's 32 bytes leave in one store
            const bool up = lane & 16;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float give = __shfl_xor_sync(0xffffffffu, up ? o[e] : o[4 + e], 16);
              const float keep = up ? o[4 + e] : o[e];
              o[e] = up ? give : keep;
              o[4 + e] = up ? keep : give;
            }
            // o[0..3]: the lower lane's row, o[4..7]: the upper lane's
            float* of = (float*)r.out + base_out + c0 + (up ? 4 : 0);
            const int lo = i_lo, hi = i_lo + kHalf;
            if (p_lo + c0 + (up ? 4 : 0) < P) {
              if (lo < n) *(float4*)(of + lo * r.os) = make_float4(o[0], o[1], o[2], o[3]);
              if (hi < n) *(float4*)(of + hi * r.os) = make_float4(o[4], o[5], o[6], o[7]);
            }
          } else if (i < n) {
            float* of = (float*)r.out + base_out + i * r.os + c0;
            T* ot = (T*)r.out + base_out + i * r.os + c0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (p_lo + c0 + e >= P) continue;
              if (f32) of[e] = o[e];
              else ot[e] = from_f32<T>(o[e]);
            }
          }
        }
      }
      if (more) {
#pragma unroll
        for (int y = 0; y < NB; ++y) {
          put_q(y);
          if (y + 1 < NB) load_q(ci + 1, y + 1);
        }
        tc::tmem_wait_st();
        tc::fence_before();
        tc::fence_async_smem();
        arrive(kBarQ);
        // A and Oi, some 4,000 cycles, hide these loads
        load_v(ci + 1);
        put_v(chunk_len(ci + 1));
        tc::fence_async_smem();
        arrive(kBarX);
      }
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
    if (!ok && lane == 0) atomicExch(a.status, kStatusTimeout);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tm, kCols);
}

template <typename T, int NB, bool SUMMARY>
__global__ void __launch_bounds__(kThreads, 1) k_la_split(const __grid_constant__ LaCall a) {
  extern __shared__ __align__(1024) char raw[];
  la_begin(a);
  const int tiles = (a.role.P + 63) / 64, item = blockIdx.x % tiles, unit = blockIdx.x / tiles;
  walk<T, NB, SUMMARY>(a, item, unit % (a.B * a.H), unit / (a.B * a.H), raw);
  la_end(a);
}

template <typename T>
cudaError_t go(const LaCall& a, bool sum, cudaStream_t s) {
  const unsigned grid = (unsigned)((int64_t)a.B * a.H * a.nseg * ((a.role.P + 63) / 64));
  if (a.role.N > 64)
    return sum ? launch_role(k_la_split<T, 2, true>, grid, kThreads, kSmem, a.beside, s, a)
               : launch_role(k_la_split<T, 2, false>, grid, kThreads, kSmem, a.beside, s, a);
  return sum ? launch_role(k_la_split<T, 1, true>, grid, kThreads, kSmem, a.beside, s, a)
             : launch_role(k_la_split<T, 1, false>, grid, kThreads, kSmem, a.beside, s, a);
}

}  // namespace

cudaError_t launch_la_split(const LaCall& a, LaPass pass, cudaStream_t s) {
  return a.dtype == M3_DTYPE_FP32 ? go<float>(a, pass == kLaSummary, s)
                                  : go<__nv_bfloat16>(a, pass == kLaSummary, s);
}

}  // namespace m3
