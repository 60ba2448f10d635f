// Linear attention with a decay per head on the tensor cores: bfloat16
// operands, float32 accumulation and states (tcgen05, kind::f16).
//
// A block of 256 threads walks one (role, segment, sequence, head, 64 columns
// of P) 128 tokens at a time. With w_ij = lam^|i-j| on the causal side of the
// chunk's n tokens, i' and j' counted in walking order, and S [N][64] the state:
//   A    = Q K^T                      [128 x 128]        tensor cores
//   Oi   = Q S                        [128 x 64]         tensor cores
//   P    = intra (A o w)              to bfloat16, kept in tensor memory
//   O    = P V                        [128 x 64]         tensor cores (P from tensor memory)
//   out  = O + inter lam^(i'+1) Oi
//   S'   = lam^n S + K^T V^           V^_j = kv lam^(n-1-j') V_j
// Rounding: P and the S that multiplies Q go to bfloat16, like the output
// itself (a relative 2^-9 rms each). V^ is carried as two bfloat16 parts, so
// the state, whose error would otherwise stay for the length of the decay, is
// exact to 2^-18 a term; S itself is float32 in the threads' registers.
//
// Layout: q, k, v tiles arrive by TMA as 64-column blocks of 128-byte rows with
// the 128-byte swizzle. Q and K are K-major operands of A; the same K tile is
// the transposed (MN-major) operand of K^T V^, and V and S are MN-major
// operands, so nothing is transposed by the threads. The low part of V^ takes
// the Q tile once A and Oi are done, and the output is staged in the high part's
// tile for a TMA store. That is 112 KB at N = 128: two blocks an SM, whose
// phases (copies, products, masks) overlap each other.
//
// The pass is bound by HBM: 2 (2 N + 2 P) bytes a token and head against 900
// tensor cycles a chunk at N = 128, P = 64.
//
// A chunk of n < 128 tokens (a sequence's end) zeroes its K and V rows up to a
// multiple of 16, which is as far as its products reach: rows of the next
// sequence, whatever they hold, take no part.
// Waits are bounded: a wait that gives up is written to the status word.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include "linattn_mma.cuh"

namespace m3 {
namespace {

constexpr int kC = kLaChunk;
constexpr int kThreads = 256;
constexpr long long kBudget = 4000000000LL;  // clock cycles, about 2 s
constexpr uint32_t kBlock = kC * 128;        // bytes of a 64-column block of a tile
// tensor memory columns: A (then P in 0..31 + 32.., O in 64..127), Oi, K^T V^
constexpr uint32_t kColO = 64, kColI = 128, kColS = 192, kCols = 256;

// bytes of the regions: Q, K (NB blocks each), V, X, S; then the small arrays
__host__ __device__ constexpr uint32_t tiles_bytes(int nb) { return 2 * nb * kBlock + 2 * kBlock + nb * 8192; }
struct Small {
  float pw[kC + 4];  // lam^d
  float col[32];     // column factors of a 32-token block
  uint64_t bar[5];
  uint32_t tmem;
};
static_assert(sizeof(Small) <= 1024, "");
// N <= 64 asks for the same memory as N = 128: two blocks an SM in either case,
// since each holds half of the tensor memory
constexpr uint32_t kSmem = tiles_bytes(2) + 1024;

struct Maps {
  CUtensorMap q[3], k[3], v[3], out[3];
};

// K-major 128-byte-swizzled operand: 8-row groups 1024 B apart; 16 columns on = 32 B,
// 64 columns on = one block.
__device__ __forceinline__ uint64_t kmajor(uint32_t addr, int ks) {
  return tc::sdesc(addr + (ks >> 2) * kBlock + (ks & 3) * 32, 16, 1024) | (2ull << 61);
}
// MN-major: 64-column blocks `block` bytes apart, 8-row (K) groups 1024 B apart;
// 16 rows on = 2048 B.
__device__ __forceinline__ uint64_t mnmajor(uint32_t addr, uint32_t block, int ks) {
  return tc::sdesc(addr + ks * 2048, block, 1024) | (2ull << 61);
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* m, int c, int head, int row,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c), "r"(head), "r"(row), "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* m, int c, int head, int row) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(c), "r"(head), "r"(row)
               : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* m, uint32_t src, int c, int head, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(m)),
      "r"(c), "r"(head), "r"(row), "r"(src)
      : "memory");
}
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
// One block's walk. NB: 64-column blocks of N (1: N <= 64, 2: N <= 128).
template <int NB, bool SUMMARY>
__device__ __forceinline__ void walk(const LaArgs& a, const Maps& maps, int ri, int pt, int bh,
                                     int seg, char* raw) {
  constexpr int NK = 64 * NB;
  constexpr int SC = NB == 2 ? 32 : 16;  // state columns a thread
  const LaRole& r = a.role[ri];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, half = warp >> 2;
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
  const int hq = h / r.q_rep, hk = h / r.k_rep, hv = h / r.v_rep;

  const uint32_t base = tc::smem_u32(raw);
  const uint32_t sQ = base, sK = sQ + NB * kBlock, sV = sK + NB * kBlock, sX = sV + kBlock,
                 sS = sX + kBlock;
  Small& sm = *reinterpret_cast<Small*>(raw + tiles_bytes(2));
  uint64_t *barQK = &sm.bar[0], *barV = &sm.bar[1], *barA = &sm.bar[2], *barB = &sm.bar[3],
           *barC = &sm.bar[4];
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) tc::bar_init(&sm.bar[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;");
  }
  const float ld = a.log_decay[h];
  if (tid <= kC) sm.pw[tid] = la_power(ld, tid);
  // lam^(31 - j) (walking up: to the block's end) or lam^j (down: to its start)
  if (tid < 32) sm.col[tid] = la_power(ld, r.reverse ? tid : 31 - tid);
  if (warp == 0) tc::tmem_alloc(&sm.tmem, kCols);
  __syncthreads();
  const uint32_t tm = sm.tmem, tw = tm + ((uint32_t)(32 * quad) << 16);

  auto chunk_row = [&](int ci) { return s0 + (int64_t)(r.reverse ? nchunk - 1 - ci : ci) * kC; };
  auto load_qk = [&](int ci) {
    const int row = (int)(row0 + chunk_row(ci));
    tc::bar_expect_tx(barQK, (SUMMARY ? 1 : 2) * NB * kBlock);
#pragma unroll
    for (int x = 0; x < NB; ++x) {
      if (!SUMMARY) tma_load(sQ + x * kBlock, &maps.q[ri], 64 * x, hq, row, barQK);
      tma_load(sK + x * kBlock, &maps.k[ri], 64 * x, hk, row, barQK);
    }
  };
  auto load_v = [&](int ci) {
    tc::bar_expect_tx(barV, kBlock);
    tma_load(sV, &maps.v[ri], p_lo, hv, (int)(row0 + chunk_row(ci)), barV);
  };
  // phases of the barriers that thread 0 still has to see end, if it leaves early
  int pend[5] = {-1, -1, -1, -1, -1};
  bool ok = true;
  if (tid == 0 && nchunk > 0) {
    load_qk(0);
    load_v(0);
    pend[0] = pend[1] = 0;
  }

  // this thread's part of the state: row n = srow, columns p_lo + scol ..
  const int srow = NB == 2 ? 32 * quad + lane : 16 * quad + (lane & 15);
  const int scol = NB == 2 ? 32 * half : 32 * half + 16 * (lane >> 4);
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
#pragma unroll
    for (int c = 0; c < SC / 8; ++c)
      sts(sS + chunk_at(srow, scol / 8 + c),
          make_uint4(pack(st[8 * c], st[8 * c + 1]), pack(st[8 * c + 2], st[8 * c + 3]),
                     pack(st[8 * c + 4], st[8 * c + 5]), pack(st[8 * c + 6], st[8 * c + 7])));
  };
  if (!SUMMARY) {
    put_state();
    tc::fence_async_smem();
    ok = __syncthreads_and(ok);
  }

  for (int ci = 0; ci < nchunk && ok; ++ci) {
    const uint32_t ph = ci & 1;
    const int64_t t0 = chunk_row(ci);
    const int n = (int)min((int64_t)kC, s1 - t0);
    const int shift = ci == 0 && first ? r.shift : 0;
    const int ksn = (n + 15) / 16;
    if (n < kC) {  // zero rows n .. 16 ksn of K and V
      ok = tc::bar_wait(barQK, ph, kBudget) && tc::bar_wait(barV, ph, kBudget) && ok;
      const int rows = 16 * ksn - n;
      for (int i = tid; i < rows * 8 * (NB + 1); i += kThreads) {
        const int rr = n + i % rows, c = i / rows;  // chunk c % 8 of block c / 8
        sts((c < 8 * NB ? sK + (c >> 3) * kBlock : sV) + chunk_at(rr, c & 7), make_uint4(0, 0, 0, 0));
      }
      tc::fence_async_smem();
      ok = __syncthreads_and(ok);
      if (!ok) break;
    }
    if (!SUMMARY) {
      if (tid == 0) {
        ok = tc::bar_wait(barQK, ph, kBudget) && ok;
        if (ok) {
          pend[0] = -1;
          tc::fence_after();
          const int ksq = (N + 15) / 16;
          for (int ks = 0; ks < ksq; ++ks)
            mma_ss(tm, kmajor(sQ, ks), kmajor(sK, ks), idesc_bf16(128, 128, 0, 0), ks > 0);
          for (int ks = 0; ks < ksq; ++ks)
            mma_ss(tm + kColI, kmajor(sQ, ks), mnmajor(sS, 0, ks), idesc_bf16(128, 64, 0, 1), ks > 0);
          tc::commit(barA);
          pend[2] = ph;
          if (ci + 1 < nchunk) {
            const int row = (int)(row0 + chunk_row(ci + 1));
#pragma unroll
            for (int x = 0; x < NB; ++x) {
              tma_prefetch(&maps.q[ri], 64 * x, hq, row);
              tma_prefetch(&maps.k[ri], 64 * x, hk, row);
            }
            tma_prefetch(&maps.v[ri], p_lo, hv, row);
          }
        }
        tma_store_wait_read();  // the last chunk's output has left X
      }
      ok = __syncthreads_and(ok);
      if (!ok) break;
    }
    // V^: the high part to X, the low part to the Q tile once A and Oi are done
    ok = tc::bar_wait(barV, ph, kBudget) && ok;
    {
      const int j = tid >> 1, c0 = 4 * (tid & 1);
      const float w = j < n ? r.kv * sm.pw[r.reverse ? j : n - 1 - j] : 0.f;
      uint4 low[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 v = lds(sV + chunk_at(j, c0 + c));
        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = w * lo_f(in[e]), y = w * hi_f(in[e]);
          hi[e] = pack(x, y);
          lo[e] = pack(x - lo_f(hi[e]), y - hi_f(hi[e]));
        }
        sts(sX + chunk_at(j, c0 + c), make_uint4(hi[0], hi[1], hi[2], hi[3]));
        low[c] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      if (!SUMMARY) {
        ok = tc::bar_wait(barA, ph, kBudget) && ok;
        tc::fence_after();
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) sts(sQ + chunk_at(j, c0 + c), low[c]);
    }
    if (!SUMMARY) {
      // P: row i of this thread, columns 64 half .. in two blocks of 32
      const int i = 32 * quad + lane;
      uint32_t pk[32];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int jb = 2 * half + x;
        if (r.reverse ? jb < quad : jb > quad) {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[16 * x + e] = 0;
          continue;
        }
        float s[32];
        ld16(tw + 32 * jb, s);
        ld16(tw + 32 * jb + 16, s + 16);
        tc::tmem_wait_ld();
        if (jb == quad) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int d = r.reverse ? e - lane : lane - e;
            s[e] = d >= 0 ? s[e] * (r.intra * sm.pw[d < 0 ? 0 : d]) : 0.f;
          }
        } else {
          const float f = r.intra * sm.pw[r.reverse ? 32 * jb - i : i - 32 * jb - 31];
#pragma unroll
          for (int e = 0; e < 32; ++e) s[e] *= f * sm.col[e];
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) pk[16 * x + e] = pack(s[2 * e], s[2 * e + 1]);
      }
      tc::fence_before();
      pair_sync(1 + quad);  // both warps of these lanes have read A
      tc::fence_after();
      asm volatile(
          "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
          "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(tw + 32 * half),
          "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]),
          "r"(pk[7]), "r"(pk[8]), "r"(pk[9]), "r"(pk[10]), "r"(pk[11]), "r"(pk[12]), "r"(pk[13]),
          "r"(pk[14]), "r"(pk[15]), "r"(pk[16]), "r"(pk[17]), "r"(pk[18]), "r"(pk[19]), "r"(pk[20]),
          "r"(pk[21]), "r"(pk[22]), "r"(pk[23]), "r"(pk[24]), "r"(pk[25]), "r"(pk[26]), "r"(pk[27]),
          "r"(pk[28]), "r"(pk[29]), "r"(pk[30]), "r"(pk[31])
          : "memory");
      tc::tmem_wait_st();
    }
    tc::fence_before();
    tc::fence_async_smem();
    ok = __syncthreads_and(ok);
    if (!ok) break;
    if (tid == 0) {
      pend[1] = pend[2] = -1;
      if (SUMMARY) {
        ok = tc::bar_wait(barQK, ph, kBudget);
        pend[0] = -1;
      }
      tc::fence_after();
      if (ok) {
        for (int part = 0; part < 2; ++part)
          for (int ks = 0; ks < ksn; ++ks)
            mma_ss(tm + kColS, mnmajor(sK, kBlock, ks), mnmajor(part ? sQ : sX, 0, ks),
                   idesc_bf16(NK, 64, 1, 1), part + ks > 0);
        tc::commit(barB);
        pend[3] = ph;
        if (!SUMMARY) {
          for (int ks = 0; ks < ksn; ++ks)
            mma_ts(tm + kColO, tm + 8 * ks, mnmajor(sV, 0, ks), idesc_bf16(128, 64, 0, 1), ks > 0);
          tc::commit(barC);
          pend[4] = ph;
        }
      }
    }
    ok = tc::bar_wait(barB, ph, kBudget) && ok;
    tc::fence_after();
    if (tid == 0 && ok) {
      pend[3] = -1;
      if (ci + 1 < nchunk) {
        load_qk(ci + 1);
        pend[0] = ph ^ 1;
        if (SUMMARY) {
          load_v(ci + 1);
          pend[1] = ph ^ 1;
        }
      }
    }
    __syncwarp();
    {
      const float dec = sm.pw[n - shift];
      float kv[SC];
      if constexpr (NB == 2) {
        ld16(tw + kColS + scol, kv);
        ld16(tw + kColS + scol + 16, kv + 16);
      } else {
        tc::tmem_ld_m64_16(tw + kColS + 32 * half, kv);
      }
      tc::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < SC; ++j) st[j] = fmaf(dec, st[j], kv[j]);
      if (!SUMMARY) put_state();
    }
    if (!SUMMARY) {
      ok = tc::bar_wait(barC, ph, kBudget) && ok;
      tc::fence_after();
      if (tid == 0 && ok) {
        pend[4] = -1;
        if (ci + 1 < nchunk) {
          load_v(ci + 1);
          pend[1] = ph ^ 1;
        }
      }
      __syncwarp();
      const int i = 32 * quad + lane, at = max(r.reverse ? n - 1 - i : i, 0);
      const float f = r.inter * sm.pw[at + 1 - shift];
      const int c0 = 32 * half;
      float o[32];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float in[16];
        ld16(tw + kColO + c0 + 16 * x, o + 16 * x);
        ld16(tw + kColI + c0 + 16 * x, in);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[16 * x + e] = fmaf(f, in[e], o[16 * x + e]);
      }
      const int64_t row = row0 + t0 + i;
      const int64_t at_out = row * r.os + (int64_t)h * P + p_lo + c0;
      if (r.out_rep > 1) {  // float32 partials of a shared head
        if (i < n) {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (p_lo + c0 + 4 * x < P)
              *(float4*)((float*)r.out + at_out + 4 * x) =
                  make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint4 v = make_uint4(pack(o[8 * x], o[8 * x + 1]), pack(o[8 * x + 2], o[8 * x + 3]),
                                     pack(o[8 * x + 4], o[8 * x + 5]), pack(o[8 * x + 6], o[8 * x + 7]));
          if (n == kC) sts(sX + chunk_at(i, c0 / 8 + x), v);
          else if (i < n && p_lo + c0 + 8 * x < P) *(uint4*)((__nv_bfloat16*)r.out + at_out + 8 * x) = v;
        }
      }
    }
    tc::fence_before();
    tc::fence_async_smem();
    ok = __syncthreads_and(ok);
    tc::fence_after();
    if (!SUMMARY && tid == 0 && ok && n == kC && r.out_rep == 1)
      tma_store(&maps.out[ri], sX, p_lo, h, (int)(row0 + t0));
  }

  if (tid == 0) {
    if (!ok) {
      atomicExch(a.status, kStatusTimeout);
      bool drained = true;
      for (int i = 0; i < 5; ++i)
        if (pend[i] >= 0) drained = tc::bar_wait(&sm.bar[i], pend[i], kBudget) && drained;
      if (!drained) atomicExch(a.status, kStatusUndrained);
    }
    tma_store_wait_read();
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

// Blocks: for each (segment, b, h), the column tiles of every role.
template <bool SUMMARY>
__global__ void __launch_bounds__(kThreads, 2)
    k_la_mma(const __grid_constant__ LaArgs a, const __grid_constant__ Maps maps, int items) {
  extern __shared__ __align__(1024) char raw[];
  la_clear_status<SUMMARY>(a);
  int item = blockIdx.x % items, ri = 0;
  const int unit = blockIdx.x / items;
  while (item >= (a.role[ri].P + 63) / 64) item -= (a.role[ri++].P + 63) / 64;
  const int bh = unit % (a.B * a.H), seg = unit / (a.B * a.H);
  if (a.role[ri].N > 64) walk<2, SUMMARY>(a, maps, ri, item, bh, seg, raw);
  else walk<1, SUMMARY>(a, maps, ri, item, bh, seg, raw);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// [rows][heads][width] bfloat16, rows `stride` elements apart: boxes of 64
// columns of one head of 128 rows; columns past the width read as zeros.
bool make_map(CUtensorMap* m, const void* p, int width, int64_t heads, int64_t rows, int64_t stride) {
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, kC}, one[3] = {1, 1, 1};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, one,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tile_ok(const void* p, int width, int64_t stride) {
  return width % 8 == 0 && stride % 8 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

}  // namespace

bool la_mma_supported(const LaArgs& a) {
  if (a.dtype != M3_DTYPE_BF16 || a.rows == 0 || !encoder()) return false;
  for (int i = 0; i < a.nrole; ++i) {
    const LaRole& r = a.role[i];
    if (!tile_ok(r.q, r.N, r.qs) || !tile_ok(r.k, r.N, r.ks) || !tile_ok(r.v, r.P, r.vs) ||
        !tile_ok(r.out, r.P, r.os))
      return false;
  }
  return true;
}

cudaError_t launch_la_mma(const LaArgs& a, LaPass pass, cudaStream_t s) {
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  int items = 0;
  for (int i = 0; i < a.nrole; ++i) {
    const LaRole& r = a.role[i];
    items += (r.P + 63) / 64;
    if (!make_map(&maps.q[i], r.q, r.N, a.H / r.q_rep, a.rows, r.qs) ||
        !make_map(&maps.k[i], r.k, r.N, a.H / r.k_rep, a.rows, r.ks) ||
        !make_map(&maps.v[i], r.v, r.P, a.H / r.v_rep, a.rows, r.vs) ||
        (r.out_rep == 1 && !make_map(&maps.out[i], r.out, r.P, a.H, a.rows, r.os)))
      return cudaErrorInvalidValue;
  }
  const unsigned grid = (unsigned)((int64_t)a.B * a.H * a.nseg * items);
  auto go = [&](auto kernel) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, kSmem, s>>>(a, maps, items);
    count_launches(1);
    return cudaGetLastError();
  };
  return pass == kLaSummary ? go(k_la_mma<true>) : go(k_la_mma<false>);
}

}  // namespace m3
