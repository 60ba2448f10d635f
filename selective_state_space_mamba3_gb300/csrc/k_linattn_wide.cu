// Linear attention with a decay per head on the tensor cores, bfloat16, for more
// than 64 output columns: all of them (up to 128) in one block.
//
// The chunked form, the rounding, the tile layouts and the warps' parts are those
// of k_linattn_mma.cu. Next to two of its blocks, A, P and the copies of Q and K
// are done once instead of twice, and a product has 128 columns instead of 64 in
// the same 64 cycles (measured: what a step of 128 x 64 x 16 takes is the time of
// one of 128 x 128 x 16). One block has the SM: 224 KB of shared memory (Q, V, S
// and both parts of V^ once, K twice) and all of the tensor memory (A twice, O,
// K^T V^). A of the next chunk is computed while this one's P V runs, so what
// ties two chunks together is the state alone.
//
// The third part of V^ (where the state is returned) takes the Q tile after A and
// Oi, as both low parts do in the other kernel.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include <type_traits>

#include "linattn_mma.cuh"

namespace m3 {
namespace {

constexpr int kC = kLaChunk;
constexpr long long kBudget = 4000000000LL;  // clock cycles, about 2 s
constexpr uint32_t kBlock = kC * 128;        // bytes of a 64-column block of a tile
// tensor memory columns: A of even and odd chunks (then P: tokens 32 g .. in 32 g ..
// 32 g + 15, so that a warp writes only over what it has read itself), Oi and O,
// K^T V^
constexpr uint32_t kColO = 256, kColS = 384, kCols = 512;
constexpr int kWarps = 16;  // compute warps; one more issues
constexpr int kThreads = 32 * (kWarps + 1);

// tiles: Q (two blocks), K (twice two), V, V^ high, V^ low, S; then the small arrays
constexpr uint32_t kTiles = 14 * kBlock;
constexpr int kQ = 0, kK = 2 * kBlock, kV = 6 * kBlock, kX = 8 * kBlock, kLow = 10 * kBlock, kS = 12 * kBlock;
enum Bar {
  kBarQ,   // Q has arrived
  kBarK0,  // K of an even chunk has, of an odd one
  kBarK1,
  kBarV,   // V has
  kBarA,   // A is done
  kBarA2,  // Oi is (committed where something waits for it)
  kBarW,   // V^ is written
  kBarB,   // K^T V^ is done, and Oi before it
  kBarP,   // P is written
  kBarC,   // O is done
  kBarE,   // O is read, S written
  kBarF,   // the output is staged
  kBarX,   // the staged output has left V^'s low tile
  kBars
};
struct Small {
  alignas(16) float col[kC];  // column factors of a chunk (mild decays) or of a 16-token block
  float pw[kC / 2 + 4];       // lam^d, d <= 64
  uint64_t bar[kBars];
  uint32_t tmem;
};
static_assert(sizeof(Small) <= 1024, "");
constexpr uint32_t kSmem = kTiles + 1024;
static_assert(kSmem <= 227 * 1024, "");

struct Maps {
  CUtensorMap q[3], k[3], v[3], out[3];
};

// K-major 128-byte-swizzled operand: 8-row groups 1024 B apart; 16 columns on = 32 B,
// 64 columns on = one block. MN-major: 64-column blocks one block apart, 8-row (K)
// groups 1024 B apart; 16 rows on = 2048 B. The steps are in descriptor units of 16 B.
// Low words of the descriptors; the high word (8-row groups, swizzle) is one for all.
__device__ __forceinline__ uint32_t kmajor(uint32_t addr) { return (uint32_t)tc::sdesc(addr, 16, 1024); }
__device__ __forceinline__ uint32_t mnmajor(uint32_t addr, uint32_t block) { return (uint32_t)tc::sdesc(addr, block, 1024); }
__host__ __device__ constexpr uint32_t kstep(int ks) { return ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4; }
__host__ __device__ constexpr uint32_t mnstep(int ks) { return ks * 2048 >> 4; }
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
// One block's walk. NB: 64-column blocks of N.
template <int NB, bool SUMMARY, bool MILD>
__device__ __forceinline__ void walk(const LaArgs& a, const Maps& maps, int ri, int bh, int seg, char* raw) {
  constexpr int NK = 64 * NB;
  constexpr int SC = NB == 2 ? 32 : 16;  // state columns a thread
  constexpr uint32_t kBlockS = NK * 128;  // bytes of a 64-column block of S
  const LaRole& r = a.role[ri];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = bh / a.H, h = bh - b * a.H;
  const int N = r.N, P = r.P;
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
  Small& sm = *reinterpret_cast<Small*>(raw + kTiles);
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i)
      tc::bar_init(&sm.bar[i], i == kBarW || i == kBarP || i == kBarE || i == kBarF ? kWarps : 1);
    asm volatile("fence.mbarrier_init.release.cluster;");
  }
  const float ld = a.log_decay[h];
  if (tid <= kC / 2) sm.pw[tid] = la_power(ld, tid);
  if (tid < kC) {
    if (MILD) sm.col[tid] = expf(ld * (float)(rev ? tid - kC / 2 : kC / 2 - tid));
    else if (tid < 16) sm.col[tid] = la_power(ld, rev ? tid : 15 - tid);
  }
  auto power = [&](int d) { return d <= kC / 2 ? sm.pw[d] : sm.pw[kC / 2] * sm.pw[d - kC / 2]; };
  if (warp == 0) tc::tmem_alloc(&sm.tmem, kCols);

  // this thread's part of the state: row n = srow, columns scol ..
  const int quad = warp & 3, grp = (warp >> 2) & 3;
  const int srow = NB == 2 ? 32 * quad + lane : 16 * quad + (lane & 15);
  const int scol = NB == 2 ? 32 * grp : 32 * grp + 16 * (lane >> 4);
  float st[SC];
  float* entry = a.entry ? a.entry + ri * a.entry_role +
                               ((int64_t)seg * a.B * a.H + bh) * ((int64_t)N * P)
                         : nullptr;
  const int64_t sbase = (int64_t)bh * N * P;
  // chunk c of a row is at the first one's address with c's bits flipped in
  const uint32_t at_state = base + (scol >> 6) * kBlockS + chunk_at(srow, (scol & 63) / 8);
  // the state that multiplies Q; `f`: MILD, what is common to the chunk's rows
  auto put_state = [&](float f) {
#pragma unroll
    for (int c = 0; c < SC / 8; ++c) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = MILD ? f * st[8 * c + j] : st[8 * c + j];
      sts<kS>(at_state ^ (c << 4), make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7])));
    }
  };
  const float ratio = MILD ? r.inter / r.intra : 1.f;
  if (warp < kWarps) {
#pragma unroll
    for (int j = 0; j < SC; ++j) {
      const int p = scol + j;
      st[j] = 0.f;
      if (!SUMMARY && srow < N && p < P) {
        if (a.nseg > 1) st[j] = entry[(int64_t)p * N + srow];
        else if (r.init) st[j] = r.init[sbase + (int64_t)p * r.sp + (int64_t)srow * r.sn];
      }
    }
    if (!SUMMARY)
      put_state(ratio * (!MILD ? 1.f
                         : !rev ? la_power(ld, kC / 2 + 1)
                                : expf(ld * (float)(min(kC, ntok - (nchunk - 1) * kC) - (first ? r.shift : 0) - kC / 2))));
  }
  tc::fence_async_smem();
  __syncthreads();
  const uint32_t tm = sm.tmem, tw = tm + ((uint32_t)(32 * quad) << 16);
  bool ok = true;
  auto wait = [&](int bar, uint32_t phase) {
    if (ok && !wait_phase(&sm.bar[bar], phase & 1, kBudget)) ok = false;
    return ok;
  };
  auto chunk_row = [&](int ci) { return row0 + (rev ? nchunk - 1 - ci : ci) * kC; };
  auto chunk_len = [&](int ci) { return min(kC, row0 + ntok - chunk_row(ci)); };

  if (warp == kWarps && nchunk > 0) {
    // The whole warp walks this code, so that addresses and descriptors stay in
    // uniform registers; one elected lane issues.
    const bool lead = tc::elect_one();
    const int hq = h / r.q_rep, hk = h / r.k_rep, hv = h / r.v_rep;
    uint32_t open = 0, odd = 0;  // barriers with a copy or product in flight, and its phase, one bit each
    auto mark = [&](int bar, int phase) {
      open |= 1u << bar;
      odd = (odd & ~(1u << bar)) | (uint32_t)(phase & 1) << bar;
    };
    auto done = [&](int bar, int phase) {
      if (!wait(bar, phase)) return false;
      open &= ~(1u << bar);
      return true;
    };
    auto load = [&](const CUtensorMap* m, int dst, int blocks, int head, int ci, int bar, int phase) {
      if (lead) {
        tc::bar_expect_tx(&sm.bar[bar], blocks * kBlock);
        for (int x = 0; x < blocks; ++x)
          tma_load(base + dst + x * kBlock, m, 64 * x, head, chunk_row(ci), &sm.bar[bar]);
      }
      mark(bar, phase);
    };
    auto load_q = [&](int ci) { load(&maps.q[ri], kQ, NB, hq, ci, kBarQ, ci); };
    auto load_k = [&](int ci) { load(&maps.k[ri], kK + (ci & 1) * 2 * (int)kBlock, NB, hk, ci, kBarK0 + (ci & 1), ci >> 1); };
    auto load_v = [&](int ci) { load(&maps.v[ri], kV, 2, hv, ci, kBarV, ci); };
    auto commit = [&](int bar, int ci) {
      if (lead) tc::commit(&sm.bar[bar]);
      mark(bar, ci);
    };
    auto store = [&](int ci) {
      if (r.out_rep > 1 || chunk_len(ci) < kC) return;
      for (int x = 0; x < 2; ++x)
        if (64 * x < P) tma_store(&maps.out[ri], base + kLow + x * kBlock, 64 * x, h, chunk_row(ci));
    };
    if (!SUMMARY) load_q(0);
    load_k(0);
    load_v(0);
    if (nchunk > 1) load_k(1);
    const int ksq = (N + 15) / 16, parts = r.fin ? 3 : 2;
    const uint32_t dQ = kmajor(base + kQ), dV = mnmajor(base + kV, kBlock), dS = mnmajor(base + kS, kBlockS);
    // A of chunk ci, once its rows are there
    auto scores = [&](int ci) {
      if (!done(kBarQ, ci) || !done(kBarK0 + (ci & 1), ci >> 1)) return false;
      tc::fence_after();
      const uint32_t dK = kmajor(base + kK + (ci & 1) * 2 * kBlock);
#pragma unroll
      for (int ks = 0; ks < NK / 16; ++ks)
        if (ks < ksq && lead)
          mma_ss(tm + (ci & 1) * 128, dQ, kstep(ks), dK, kstep(ks), idesc_bf16(128, 128, 0, 0), ks > 0);
      commit(kBarA, ci);
      return true;
    };
    if (!SUMMARY) scores(0);
    for (int ci = 0; ci < nchunk && ok; ++ci) {
      const int ksn = (chunk_len(ci) + 15) / 16;
      const bool more = ci + 1 < nchunk;
      if (more && lead) {  // the next chunk's values wait for this one's P V: at least into L2
        tma_prefetch(&maps.v[ri], 0, hv, chunk_row(ci + 1));
        tma_prefetch(&maps.v[ri], 64, hv, chunk_row(ci + 1));
        if (!SUMMARY)
          for (int x = 0; x < NB; ++x) tma_prefetch(&maps.q[ri], 64 * x, hq, chunk_row(ci + 1));
      }
      if (!SUMMARY) {
        if (ci > 0) {  // the state is in place, the last output read
          if (!wait(kBarE, ci - 1)) break;
          tc::fence_after();
        }
#pragma unroll
        for (int ks = 0; ks < NK / 16; ++ks)
          if (ks < ksq && lead)
            mma_ss(tm + kColO, dQ, kstep(ks), dS, mnstep(ks), idesc_bf16(128, 128, 0, 1), ks > 0);
        commit(kBarA2, ci);
        if (ci > 0) {
          if (!wait(kBarF, ci - 1)) break;
          if (lead) {
            store(ci - 1);
            tma_store_wait_read();
            tc::bar_arrive(&sm.bar[kBarX]);
          }
        }
      }
      if (!wait(kBarW, ci)) break;
      open &= ~(1u << kBarV);  // the compute warps have waited for it
      if (SUMMARY && !done(kBarK0 + (ci & 1), ci >> 1)) break;
      tc::fence_after();
      const uint32_t dKt = mnmajor(base + kK + (ci & 1) * 2 * kBlock, kBlock);
      for (int part = 0; part < parts; ++part) {
        const uint32_t dX = mnmajor(base + (part == 0 ? kX : part == 1 ? kLow : kQ), kBlock);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          if (ks < ksn && lead)
            mma_ss(tm + kColS, dKt, mnstep(ks), dX, mnstep(ks), idesc_bf16(NK, 128, 1, 1), part + ks > 0);
      }
      commit(kBarB, ci);
      if (SUMMARY) {
        if (more) load_v(ci + 1);
      } else {
        if (!wait(kBarP, ci)) break;
        tc::fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          if (ks < ksn && lead)
            mma_ts(tm + kColO, tm + (ci & 1) * 128, 32 * (ks >> 1) + 8 * (ks & 1), dV, mnstep(ks),
                   idesc_bf16(128, 128, 0, 1), true);
        commit(kBarC, ci);
      }
      if (!done(kBarB, ci)) break;
      if (!SUMMARY && more) load_q(ci + 1);
      if (ci + 2 < nchunk) load_k(ci + 2);
      if (!SUMMARY) {
        if (!done(kBarC, ci)) break;
        if (more) {
          load_v(ci + 1);
          if (!scores(ci + 1)) break;
        }
      }
    }
    if (!SUMMARY && ok && wait(kBarF, nchunk - 1) && lead) store(nchunk - 1);
    if (lead) tma_store_wait_read();
    if (!ok) {  // bounded waits for what is still in flight
      if (lead) atomicExch(a.status, kStatusTimeout);
      for (int i = 0; i < kBars; ++i)
        if ((open >> i & 1) && !wait_phase(&sm.bar[i], odd >> i & 1, kBudget) && lead)
          atomicExch(a.status, kStatusUndrained);
    }
    __syncwarp();
  } else if (warp < kWarps) {
    auto arrive = [&](int bar) {
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sm.bar[bar]);
    };
    const int i = 32 * quad + lane;  // this thread's row of A, P and O
    const uint32_t at_v = base + chunk_at(tid >> 2, 2 * (tid & 3));
    const uint32_t at_o = base + (grp >> 1) * kBlock + chunk_at(i, 4 * (grp & 1));
    // row and column factors: see k_linattn_mma.cu
    const float intra = r.intra;
    const float rowf = MILD ? intra * expf(ld * (float)(rev ? kC / 2 - i : i - kC / 2)) : 1.f;
    float fac[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int c = 32 * grp + 16 * x, d = rev ? c - i : i - c - 15;
      fac[x] = MILD || d < 0 ? 0.f : intra * power(d);
    }
    for (int ci = 0; ci < nchunk; ++ci) {
      const int n = chunk_len(ci);
      const int shift = ci == 0 && first ? r.shift : 0;
      if (!wait(kBarV, ci)) break;
      if (n < kC) {  // zero rows n .. of K and V up to a multiple of 16
        if (!wait(kBarK0 + (ci & 1), ci >> 1)) break;
        const int rows = (n + 15) / 16 * 16 - n;
        const uint32_t sK = base + kK + (ci & 1) * 2 * kBlock;
        for (int x = tid; x < rows * 8 * (NB + 2); x += 32 * kWarps) {
          const int rr = n + x % rows, c = x / rows;  // chunk c % 8 of block c / 8
          sts((c < 8 * NB ? sK + (c >> 3) * kBlock : base + kV + ((c >> 3) - NB) * kBlock) + chunk_at(rr, c & 7),
              make_uint4(0, 0, 0, 0));
        }
      }
      {  // V^
        const int j = tid >> 2;
        const float w = j < n ? r.kv * power(rev ? j : n - 1 - j) : 0.f;
        if (!SUMMARY && ci > 0 && !wait(kBarX, ci - 1)) break;  // the last output has left the low tile
        if (!SUMMARY && r.fin && !wait(kBarA2, ci)) break;      // A and Oi have read Q
        const bool in = j < n;  // (this thread's own zeros may be another's to write)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t at = (at_v ^ ((c & 1) << 4)) + (c >> 1) * kBlock;
          const uint4 v = in ? lds<kV>(at) : make_uint4(0, 0, 0, 0);
          const uint32_t x4[4] = {v.x, v.y, v.z, v.w};
          uint32_t hi[4], lo[4], rest[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = __fmul2_rn(make_float2(w, w), make_float2(lo_f(x4[e]), hi_f(x4[e])));
            hi[e] = pack(x.x, x.y);
            const float2 d = __fadd2_rn(x, make_float2(-lo_f(hi[e]), -hi_f(hi[e])));
            lo[e] = pack(d.x, d.y);
            if (r.fin) rest[e] = pack(d.x - lo_f(lo[e]), d.y - hi_f(lo[e]));
          }
          sts<kX>(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          sts<kLow>(at, make_uint4(lo[0], lo[1], lo[2], lo[3]));
          if (r.fin) sts<kQ>(at, make_uint4(rest[0], rest[1], rest[2], rest[3]));
        }
        tc::fence_async_smem();
        arrive(kBarW);
      }
      if (!SUMMARY) {
        if (!wait(kBarA, ci)) break;
        tc::fence_after();
        // P: columns 32 grp .. in blocks of 16, over the columns of A already read
        const uint32_t ta = tw + (ci & 1) * 128 + 32 * grp;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int c = 32 * grp + 16 * x;
          uint32_t pk[8] = {};
          if (rev ? c + 15 >= 32 * quad : c <= 32 * quad + 31) {
            float s[16];
            ld16(ta + 16 * x, s);
            tc::tmem_wait_ld();
            const bool full = rev ? c >= 32 * quad + 32 : c < 32 * quad;
            if (MILD || full) {
              const float2 f2 = make_float2(fac[x], fac[x]);
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 w = *reinterpret_cast<const float4*>(&sm.col[(MILD ? c : 0) + e]);
                float2 u = __fmul2_rn(make_float2(s[e], s[e + 1]), make_float2(w.x, w.y));
                float2 v = __fmul2_rn(make_float2(s[e + 2], s[e + 3]), make_float2(w.z, w.w));
                if (!MILD) {
                  u = __fmul2_rn(u, f2);
                  v = __fmul2_rn(v, f2);
                }
                s[e] = u.x;
                s[e + 1] = u.y;
                s[e + 2] = v.x;
                s[e + 3] = v.y;
              }
            }
            if (!full) {
              int d0 = rev ? c - i : i - c;
              const int step = rev ? 1 : -1;
              asm volatile("" : "+r"(d0));  // sixteen addresses and tests are not worth registers between chunks
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int d = d0 + step * e;
                if (!MILD) s[e] *= intra * power(max(d, 0));
                s[e] = d >= 0 ? s[e] : 0.f;
              }
            }
            if (n < kC) {  // A may have read other rows' keys past n
#pragma unroll
              for (int e = 0; e < 16; ++e) s[e] = c + e < n ? s[e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) pk[e] = pack(s[2 * e], s[2 * e + 1]);
          }
          st8(ta + 8 * x, pk);
        }
        if (!MILD) {  // Oi scaled in place, for O to be added
          if (!wait(kBarA2, ci)) break;
          tc::fence_after();
          const int at = max(rev ? n - 1 - i : i, 0);
          const float f = r.inter * power(at + 1 - shift);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float o[16];
            ld16(tw + kColO + 32 * grp + 16 * x, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= f;
            tc::tmem_st16_async(tw + kColO + 32 * grp + 16 * x, o);
          }
        }
        tc::tmem_wait_st();
        tc::fence_before();
        arrive(kBarP);
      }
      if (!wait(kBarB, ci)) break;
      tc::fence_after();
      {
        const float dec = power(n - shift);
#pragma unroll
        for (int x = 0; x < SC / 16; ++x) {
          float kv[16];
          if constexpr (NB == 2) ld16(tw + kColS + scol + 16 * x, kv);
          else tc::tmem_ld_m64_16(tw + kColS + 32 * grp, kv);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) st[16 * x + j] = fmaf(dec, st[16 * x + j], kv[j]);
        }
        if (!SUMMARY) put_state(ratio * power(rev ? kC / 2 : kC / 2 + 1));
      }
      tc::fence_before();
      tc::fence_async_smem();
      if (SUMMARY) continue;
      if (!wait(kBarC, ci)) break;
      tc::fence_after();
      {
        float o[32];
        ld16(tw + kColO + 32 * grp, o);
        ld16(tw + kColO + 32 * grp + 16, o + 16);
        tc::tmem_wait_ld();
        tc::fence_before();
        arrive(kBarE);
        if (MILD) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= rowf;
        }
        const int64_t at_out = (int64_t)(chunk_row(ci) + i) * r.os + (int64_t)h * P + 32 * grp;
        if (r.out_rep > 1) {  // float32 partials of a shared head
          if (i < n) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              if (32 * grp + 4 * x < P)
                *(float4*)((float*)r.out + at_out + 4 * x) =
                    make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint4 v = make_uint4(pack(o[8 * x], o[8 * x + 1]), pack(o[8 * x + 2], o[8 * x + 3]),
                                       pack(o[8 * x + 4], o[8 * x + 5]), pack(o[8 * x + 6], o[8 * x + 7]));
            if (n == kC) sts<kLow>(at_o ^ (x << 4), v);
            else if (i < n && 32 * grp + 8 * x < P)
              *(uint4*)((__nv_bfloat16*)r.out + at_out + 8 * x) = v;
          }
        }
        tc::fence_async_smem();
        arrive(kBarF);
      }
    }
    if (ok && (SUMMARY || (r.fin && last))) {
      const float f = !SUMMARY && len > 0 && r.fin_shift ? power(1) : 1.f;
#pragma unroll
      for (int j = 0; j < SC; ++j) {
        const int p = scol + j;
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

// Blocks: for each role, for each (segment, b, h).
template <bool SUMMARY>
__global__ void __launch_bounds__(kThreads, 1)
    k_la_wide(const __grid_constant__ LaArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) char raw[];
  la_clear_status(a);
  const int units = a.B * a.H * a.nseg;
  const int ri = blockIdx.x / units, unit = blockIdx.x - ri * units;
  const int bh = unit % (a.B * a.H), seg = unit / (a.B * a.H);
  const LaRole& r = a.role[ri];
  const float ld = a.log_decay[bh % a.H], ratio = r.inter / r.intra;
  const bool mild = fabsf(ld) <= 1.f && fabsf(ratio) < 1e6f && fabsf(ratio) > 1e-6f;  // else: strong, or scale 0
  auto go = [&](auto nb) {
    if (mild && !SUMMARY) walk<nb.value, SUMMARY, true>(a, maps, ri, bh, seg, raw);
    else walk<nb.value, SUMMARY, false>(a, maps, ri, bh, seg, raw);
  };
  if (r.N > 64) go(std::integral_constant<int, 2>());
  else go(std::integral_constant<int, 1>());
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

}  // namespace

cudaError_t launch_la_wide(const LaArgs& a, LaPass pass, cudaStream_t s) {
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  for (int i = 0; i < a.nrole; ++i) {
    const LaRole& r = a.role[i];
    if (!make_map(&maps.q[i], r.q, r.N, a.H / r.q_rep, a.rows, r.qs) ||
        !make_map(&maps.k[i], r.k, r.N, a.H / r.k_rep, a.rows, r.ks) ||
        !make_map(&maps.v[i], r.v, r.P, a.H / r.v_rep, a.rows, r.vs) ||
        (r.out_rep == 1 && !make_map(&maps.out[i], r.out, r.P, a.H, a.rows, r.os)))
      return cudaErrorInvalidValue;
  }
  const unsigned grid = (unsigned)((int64_t)a.B * a.H * a.nseg * a.nrole);
  auto go = [&](auto kernel) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, kSmem, s>>>(a, maps);
    count_launches(1);
    return cudaGetLastError();
  };
  return pass == kLaSummary ? go(k_la_wide<true>) : go(k_la_wide<false>);
}

}  // namespace m3
