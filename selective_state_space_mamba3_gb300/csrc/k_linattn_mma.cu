// Linear attention with a decay per head on the tensor cores: bfloat16
// operands, float32 accumulation and states (tcgen05, kind::f16).
//
// A block walks one (role, segment, sequence, head, 64 columns of P) 128 tokens at
// a time. With w_ij = lam^|i-j| on the causal side of the chunk's n tokens, i' and
// j' counted in walking order, and S [N][64] the state:
//   A    = Q K^T                      [128 x 128]        tensor cores
//   Oi   = Q S                        [128 x 64]         tensor cores
//   P    = intra (A o w)              to bfloat16, kept in tensor memory
//   out  = inter lam^(i'+1) Oi + P V  [128 x 64]         tensor cores (P from tensor memory)
//   S'   = lam^n S + K^T V^           V^_j = kv lam^(n-1-j') V_j
// Rounding: P and the S that multiplies Q go to bfloat16, like the output
// itself (a relative 1.6e-3 rms each). V^ is carried as two bfloat16 parts, so
// the state, whose error would otherwise stay for the length of the decay, is
// exact to 2^-16 a term, and as three (2^-24) where the state is returned; S
// itself is float32 in the threads' registers.
//
// Layout: q, k, v tiles arrive by TMA as 64-column blocks of 128-byte rows with
// the 128-byte swizzle. Q and K are K-major operands of A; the same K tile is
// the transposed (MN-major) operand of K^T V^, and V and S are MN-major
// operands, so nothing is transposed by the threads. The low parts of V^ take
// the Q tile once A and Oi are done, and the output is staged in the high part's
// tile for a TMA store. That is 112 KB at N = 128: two blocks an SM, whose
// phases (copies, products, masks) overlap each other. Sixteen warps compute and a
// seventeenth issues copies and products: issued by a compute warp (some 40 of them,
// 50 to 65 cycles each) the others waited for it.
//
// The floor is HBM's: 2 (2 N + 2 P) bytes a token and head, 4,200 cycles a chunk and
// SM at N = 128, P = 64; the products take about 2,600 (a step of 128 x 64 x 16 as
// long as one of 128 x 128 x 16), the threads' instructions about 2,000. Measured on
// prompts of 8 x 2048 tokens, 32 heads, P 64, N 128: 76 us, 5.3 TB/s, 78 % of a copy's
// rate; adjoints of the same 267 us. With few blocks a chunk's own chain binds, some
// 7,000 cycles alone on an SM. Two blocks of 17 warps leave a thread 56 registers: at
// N > 64 it spills 20 bytes, else none.
//
// A chunk of n < 128 tokens (a sequence's end) zeroes its K and V rows up to a
// multiple of 16, which is as far as its products reach: rows of the next
// sequence, whatever they hold, take no part.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include "linattn_mma.cuh"

namespace m3 {
namespace {

constexpr int kC = kLaChunk;
constexpr long long kBudget = 4000000000LL;  // clock cycles, about 2 s
constexpr uint32_t kBlock = kC * 128;        // bytes of a 64-column block of a tile
// tensor memory columns: A in 0..127 (then P: tokens 32 g .. in 32 g .. 32 g + 15, so
// that a warp writes only over what it has read itself), Oi and O, K^T V^
constexpr uint32_t kColO = 128, kColS = 192, kCols = 256;
constexpr int kWarps = 16;  // compute warps; one more issues
constexpr int kThreads = 32 * (kWarps + 1);

// tiles: Q and K (two blocks each), V, X, S; then the small arrays. N <= 64 asks
// for the same memory as N = 128: two blocks an SM in either case, since each
// holds half of the tensor memory
constexpr uint32_t kTiles = 7 * kBlock;
constexpr int kQ = 0, kK = 2 * kBlock, kV = 4 * kBlock, kX = 5 * kBlock, kS = 6 * kBlock;
enum Bar {
  kBarQK,  // Q and K have arrived
  kBarV,   // V has
  kBarA,   // A and Oi are done
  kBarW,   // V^ is written
  kBarB,   // K^T V^ is done
  kBarP,   // P is written and Oi scaled
  kBarC,   // O is done
  kBarE,  // O is read, S written
  kBarF,  // the output is staged
  kBarX,   // the staged output has left X
  kBarZ,   // the rows past the sequence's end are zeroed
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

struct Maps {
  CUtensorMap q, k, v, out;
};

// K-major 128-byte-swizzled operand: 8-row groups 1024 B apart; 16 columns on = 32 B,
// 64 columns on = one block. MN-major: 64-column blocks one block apart, 8-row (K)
// groups 1024 B apart; 16 rows on = 2048 B. The steps are in descriptor units of 16 B.
// Low words of the descriptors; the high word (8-row groups, swizzle) is one for all.
__device__ __forceinline__ uint32_t kmajor(uint32_t addr) { return (uint32_t)tc::sdesc(addr, 16, 1024); }
__device__ __forceinline__ uint32_t mnmajor(uint32_t addr) { return (uint32_t)tc::sdesc(addr, kBlock, 1024); }
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
// One block's walk. NB: 64-column blocks of N (1: N <= 64, 2: N <= 128).
// Warps 0..15 are the compute warps, one lane of warp 16 issues copies and products.
// They meet at mbarriers only (one phase a chunk each, arrivals one a warp), and
// every wait is bounded, so a thread whose wait gives up leaves the loop and the
// others follow as theirs do.
template <int NB, bool SUMMARY, bool MILD>
__device__ __forceinline__ void walk(const LaCall& a, const Maps& maps, int pt, int bh, int seg,
                                     char* raw) {
  constexpr int NK = 64 * NB;
  constexpr int SC = NB == 2 ? 16 : 8;  // state columns a thread
  const LaRole& r = a.role;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = bh / a.H, h = bh - b * a.H;
  const int N = r.N, P = r.P, p_lo = 64 * pt;
  const bool rev = r.reverse;
  int64_t seq0, len;
  la_rows(a, b, &seq0, &len);
  const int last_seg = len > 0 ? (int)((len - 1) / a.seg_len) : 0;
  if (seg > last_seg) return;
  const int row0 = (int)(seq0 + seg * a.seg_len);                        // the segment's rows
  const int ntok = (int)min(len - seg * a.seg_len, a.seg_len);
  if (SUMMARY && seg == (rev ? 0 : last_seg)) return;  // the prefix pass never reads it
  const bool first = seg == (rev ? last_seg : 0), last = seg == (rev ? 0 : last_seg);
  const int nchunk = (ntok + kC - 1) / kC;
  // this block's state is returned, or goes into one that is: three parts of V^
  const bool fin = r.fin && (SUMMARY || last);

  const uint32_t base = tc::smem_u32(raw);
  const uint32_t sQ = base + kQ, sK = base + kK, sV = base + kV, sX = base + kX, sS = base + kS;
  Small& sm = *reinterpret_cast<Small*>(raw + kTiles);
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i)
      tc::bar_init(&sm.bar[i], i == kBarW || i == kBarP || i == kBarE || i == kBarF || i == kBarZ ? kWarps : 1);
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

  // this thread's part of the state: row n = srow, columns p_lo + scol ..
  const int quad = warp & 3, grp = (warp >> 2) & 3;
  const int srow = NB == 2 ? 32 * quad + lane : 16 * quad + (lane & 15);
  const int scol = NB == 2 ? 16 * grp : 16 * grp + 8 * (lane >> 4);
  float st[SC];
  float* entry = a.entry ? a.entry + ((int64_t)seg * a.B * a.H + bh) * ((int64_t)N * P) : nullptr;
  const int64_t sbase = (int64_t)bh * N * P;
  // chunk c of a row is at the first one's address with c's bits flipped in
  const uint32_t at_state = base + chunk_at(srow, scol / 8);
  auto put_state = [&]() {  // the state that multiplies Q
#pragma unroll
    for (int c = 0; c < SC / 8; ++c)
      sts<kS>(at_state ^ (c << 4),
              make_uint4(pack(st[8 * c], st[8 * c + 1]), pack(st[8 * c + 2], st[8 * c + 3]),
                         pack(st[8 * c + 4], st[8 * c + 5]), pack(st[8 * c + 6], st[8 * c + 7])));
  };
  if (warp < kWarps) {
#pragma unroll
    for (int j = 0; j < SC; ++j) {
      const int p = p_lo + scol + j;
      st[j] = 0.f;
      if (!SUMMARY && srow < N && p < P) {
        if (a.nseg > 1) st[j] = entry[(int64_t)p * N + srow];
        else if (r.init) st[j] = r.init[sbase + (int64_t)p * r.sp + (int64_t)srow * r.sn];
      }
    }
    if (!SUMMARY) put_state();
  }
  tc::fence_async_smem();
  __syncthreads();
  const uint32_t tm = sm.tmem, tw = tm + ((uint32_t)(32 * quad) << 16);
  bool ok = true;
  auto wait = [&](int bar, uint32_t phase) {
    if (ok && !wait_phase(&sm.bar[bar], phase, kBudget)) ok = false;
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
    auto mark = [&](int bar, int ci) {
      open |= 1u << bar;
      odd = (odd & ~(1u << bar)) | (uint32_t)(ci & 1) << bar;
    };
    auto load_qk = [&](int ci) {
      const int row = chunk_row(ci);
      if (lead) {
        tc::bar_expect_tx(&sm.bar[kBarQK], (SUMMARY ? 1 : 2) * NB * kBlock);
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          if (!SUMMARY) tma_load(sQ + x * kBlock, &maps.q, 64 * x, hq, row, &sm.bar[kBarQK]);
          tma_load(sK + x * kBlock, &maps.k, 64 * x, hk, row, &sm.bar[kBarQK]);
        }
      }
      mark(kBarQK, ci);
    };
    auto load_v = [&](int ci) {
      if (lead) {
        tc::bar_expect_tx(&sm.bar[kBarV], kBlock);
        tma_load(sV, &maps.v, p_lo, hv, chunk_row(ci), &sm.bar[kBarV]);
      }
      mark(kBarV, ci);
    };
    auto prefetch = [&](int ci) {
      const int row = chunk_row(ci);
      if (!lead) return;
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        if (!SUMMARY) tma_prefetch(&maps.q, 64 * x, hq, row);
        tma_prefetch(&maps.k, 64 * x, hk, row);
      }
      tma_prefetch(&maps.v, p_lo, hv, row);
    };
    auto commit = [&](int bar, int ci) {
      if (lead) tc::commit(&sm.bar[bar]);
      mark(bar, ci);
    };
    auto store = [&](int ci) {
      if (lead && r.out_rep == 1 && chunk_len(ci) == kC)
        tma_store(&maps.out, sX, p_lo, h, chunk_row(ci));
    };
    load_qk(0);
    load_v(0);
    const int ksq = (N + 15) / 16, parts = fin ? 3 : 2;
    const uint32_t dQ = kmajor(sQ), dK = kmajor(sK), dKt = mnmajor(sK), dV = mnmajor(sV), dS = mnmajor(sS);
    for (int ci = 0; ci < nchunk; ++ci) {
      const uint32_t ph = ci & 1;
      const int n = chunk_len(ci), ksn = (n + 15) / 16;
      const bool more = ci + 1 < nchunk;
      if (more) prefetch(ci + 1);
      if (!wait(kBarQK, ph)) break;
      open &= ~(1u << kBarQK);
      if (n < kC && !wait(kBarZ, 0)) break;  // the last rows are zeroed
      if (!SUMMARY) {
        tc::fence_after();
#pragma unroll
        for (int ks = 0; ks < NK / 16; ++ks)
          if (ks < ksq && lead) mma_ss(tm, dQ, kstep(ks), dK, kstep(ks), idesc_bf16(128, 128, 0, 0), ks > 0);
        if (ci > 0) {  // the state is in place, the last output read
          if (!wait(kBarE, ph ^ 1)) break;
          tc::fence_after();
        }
#pragma unroll
        for (int ks = 0; ks < NK / 16; ++ks)
          if (ks < ksq && lead)
            mma_ss(tm + kColO, dQ, kstep(ks), dS, mnstep(ks), idesc_bf16(128, 64, 0, 1), ks > 0);
        commit(kBarA, ci);
        if (ci > 0) {
          if (!wait(kBarF, ph ^ 1)) break;
          store(ci - 1);
          if (lead) {
            tma_store_wait_read();
            tc::bar_arrive(&sm.bar[kBarX]);
          }
        }
      }
      if (!wait(kBarW, ph)) break;
      open &= ~(1u << kBarV);
      if (!SUMMARY) open &= ~(1u << kBarA);  // the compute warps have waited for both
      tc::fence_after();
      for (int part = 0; part < parts; ++part) {
        const uint32_t dX = mnmajor(part == 0 ? sX : sQ + (part - 1) * kBlock);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          if (ks < ksn && lead)
            mma_ss(tm + kColS, dKt, mnstep(ks), dX, mnstep(ks), idesc_bf16(NK, 64, 1, 1), part + ks > 0);
      }
      commit(kBarB, ci);
      if (SUMMARY && more) load_v(ci + 1);
      if (!wait(kBarB, ph)) break;
      open &= ~(1u << kBarB);
      if (more) load_qk(ci + 1);
      if (!SUMMARY) {
        if (!wait(kBarP, ph)) break;
        tc::fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          if (ks < ksn && lead)
            mma_ts(tm + kColO, tm, 32 * (ks >> 1) + 8 * (ks & 1), dV, mnstep(ks),
                   idesc_bf16(128, 64, 0, 1), true);
        commit(kBarC, ci);
        if (!wait(kBarC, ph)) break;
        open &= ~(1u << kBarC);
        if (more) load_v(ci + 1);
      }
    }
    if (!SUMMARY && ok && wait(kBarF, (nchunk - 1) & 1)) store(nchunk - 1);
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
    const uint32_t at_v = base + chunk_at(tid >> 2, 2 * (tid & 3)), at_o = base + chunk_at(i, 2 * grp);
    // A decay of at most e^0.5 a token splits into a factor of the row and one of the
    // column over the whole chunk, lam^(i-j) = lam^(i-64) lam^(64-j), each within e^32
    // and multiplied with each other before the score, so that no term is larger than
    // its result or lost below it. (With the row's factor left to the output, and the
    // readout's in S, calls take 1 to 3 % less time, but scores times values above
    // 10^24 overflow and results below 10^-24 lose their bits.) Stronger decays take
    // a row factor for every block of 16 columns, and lam^d from the table on the
    // diagonal: the layer's prompts 84 us instead of 76, its adjoints 304 instead of 267.
    const float intra = r.intra;
    float fac[2];
    if (MILD) {
      fac[0] = fac[1] = intra * expf(ld * (float)(rev ? kC / 2 - i : i - kC / 2));
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int c = 32 * grp + 16 * x, d = rev ? c - i : i - c - 15;
        fac[x] = d < 0 ? 0.f : intra * power(d);
      }
    }
    for (int ci = 0; ci < nchunk; ++ci) {
      const uint32_t ph = ci & 1;
      const int n = chunk_len(ci);
      const int shift = ci == 0 && first ? r.shift : 0;
      if (n < kC) {  // zero rows n .. of K and V up to a multiple of 16
        if (!wait(kBarQK, ph) || !wait(kBarV, ph)) break;
        const int rows = (n + 15) / 16 * 16 - n;
        for (int x = tid; x < rows * 8 * (NB + 1); x += 32 * kWarps) {
          const int rr = n + x % rows, c = x / rows;  // chunk c % 8 of block c / 8
          sts((c < 8 * NB ? sK + (c >> 3) * kBlock : sV) + chunk_at(rr, c & 7), make_uint4(0, 0, 0, 0));
        }
        tc::fence_async_smem();
        arrive(kBarZ);
        if (!wait(kBarZ, 0)) break;
      }
      uint32_t oi[16];
      // V^: the high part to X, the rest to the Q tile once A and Oi are done
      if (!wait(kBarV, ph)) break;
      {
        const int j = tid >> 2;
        const float w = j < n ? r.kv * power(rev ? j : n - 1 - j) : 0.f;
        uint4 low[2];
        if (!SUMMARY && ci > 0 && !wait(kBarX, ph ^ 1)) break;  // the last output has left X
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 v = lds<kV>(at_v ^ (c << 4));
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = __fmul2_rn(make_float2(w, w), make_float2(lo_f(in[e]), hi_f(in[e])));
            hi[e] = pack(x.x, x.y);
            const float2 d = __fadd2_rn(x, make_float2(-lo_f(hi[e]), -hi_f(hi[e])));
            lo[e] = pack(d.x, d.y);
          }
          sts<kX>(at_v ^ (c << 4), make_uint4(hi[0], hi[1], hi[2], hi[3]));
          low[c] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (!SUMMARY) {
          if (!wait(kBarA, ph)) break;
          tc::fence_after();
          ld16(tw + kColO + 16 * grp, oi);  // while V^ is stored
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) sts<kQ>(at_v ^ (c << 4), low[c]);
        if (fin) {  // a third part
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 v = lds<kV>(at_v ^ (c << 4)), l = low[c];
            const uint32_t in[4] = {v.x, v.y, v.z, v.w}, lo[4] = {l.x, l.y, l.z, l.w};
            uint32_t rest[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = w * lo_f(in[e]), y = w * hi_f(in[e]);
              const uint32_t hi = pack(x, y);
              rest[e] = pack(x - lo_f(hi) - lo_f(lo[e]), y - hi_f(hi) - hi_f(lo[e]));
            }
            sts<kQ + (int)kBlock>(at_v ^ (c << 4), make_uint4(rest[0], rest[1], rest[2], rest[3]));
          }
        }
        tc::fence_async_smem();
        arrive(kBarW);
      }
      if (!SUMMARY) {
        {  // Oi scaled in place, for O to be added
          const float f = r.inter * power(max(rev ? n - 1 - i : i, 0) + 1 - shift);
          float o[16];
          wait_ld16(oi);
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            set(o, e, __fmul2_rn(make_float2(f, f), make_float2(__uint_as_float(oi[e]), __uint_as_float(oi[e + 1]))));
          tc::tmem_st16_async(tw + kColO + 16 * grp, o);
        }
        // P: columns 32 grp .. in blocks of 16, over the columns of A already read
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int c = 32 * grp + 16 * x;
          uint32_t pk[8] = {};
          if (rev ? c + 15 >= 32 * quad : c <= 32 * quad + 31) {
            float s[16];
            ld16(tw + c, s);
            tc::tmem_wait_ld();
            const bool full = rev ? c >= 32 * quad + 32 : c < 32 * quad;
            if (MILD || full) {
              const float2 f2 = make_float2(fac[x], fac[x]);
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 w = *reinterpret_cast<const float4*>(&sm.col[(MILD ? c : 0) + e]);
                set(s, e, __fmul2_rn(pair(s, e), __fmul2_rn(make_float2(w.x, w.y), f2)));
                set(s, e + 2, __fmul2_rn(pair(s, e + 2), __fmul2_rn(make_float2(w.z, w.w), f2)));
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
#pragma unroll
            for (int e = 0; e < 8; ++e) pk[e] = pack(s[2 * e], s[2 * e + 1]);
          }
          st8(tw + 32 * grp + 8 * x, pk);
        }
        tc::tmem_wait_st();
        tc::fence_before();
        arrive(kBarP);
      }
      if (!wait(kBarB, ph)) break;
      tc::fence_after();
      {
        const float dec = power(n - shift);
        float kv[SC];
        if constexpr (NB == 2) {
          ld16(tw + kColS + scol, kv);
        } else {
          ld_m64_8(tw + kColS + 16 * grp, kv);
        }
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < SC; j += 2)
          set(st, j, __ffma2_rn(make_float2(dec, dec), pair(st, j), pair(kv, j)));
        if (!SUMMARY) put_state();
      }
      tc::fence_before();
      tc::fence_async_smem();
      if (SUMMARY) continue;
      if (!wait(kBarC, ph)) break;
      tc::fence_after();
      {
        const int c0 = 16 * grp;
        float o[16];
        ld16(tw + kColO + c0, o);
        tc::tmem_wait_ld();
        tc::fence_before();
        arrive(kBarE);
        const int64_t at_out = (chunk_row(ci) + i) * r.os + (int64_t)h * P + p_lo + c0;
        if (r.out_rep > 1) {  // float32 partials of a shared head
          if (i < n) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (p_lo + c0 + 4 * x < P)
                *(float4*)((float*)r.out + at_out + 4 * x) =
                    make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint4 v = make_uint4(pack(o[8 * x], o[8 * x + 1]), pack(o[8 * x + 2], o[8 * x + 3]),
                                       pack(o[8 * x + 4], o[8 * x + 5]), pack(o[8 * x + 6], o[8 * x + 7]));
            if (n == kC) sts<kX>(at_o ^ (x << 4), v);
            else if (i < n && p_lo + c0 + 8 * x < P)
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

// Blocks: for each (segment, b, h), its column tiles. A launch takes one role, so
// that its settings are constants' operands instead of loads; the next role's
// blocks may take the places that this one's leave (launch_role).
template <int NB, bool SUMMARY>
__global__ void __launch_bounds__(kThreads, 2)
    k_la_mma(const __grid_constant__ LaCall a, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) char raw[];
  la_begin(a);
  const int tiles = (a.role.P + 63) / 64, item = blockIdx.x % tiles, unit = blockIdx.x / tiles;
  const int bh = unit % (a.B * a.H), seg = unit / (a.B * a.H);
  // (the scale is in the row factors, within e^32)
  const float scale = fabsf(a.role.intra);
  const bool mild = fabsf(a.log_decay[bh % a.H]) <= 0.5f && scale < 1e6f && scale > 1e-6f;  // else: strong, or scale 0
  if (mild && !SUMMARY) walk<NB, SUMMARY, true>(a, maps, item, bh, seg, raw);
  else walk<NB, SUMMARY, false>(a, maps, item, bh, seg, raw);
  la_end(a);
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
  if (a.call.dtype != M3_DTYPE_BF16 || a.call.rows == 0 || !encoder()) return false;
  for (int i = 0; i < a.nrole; ++i) {
    const LaRole& r = a.role[i];
    if (!tile_ok(r.q, r.N, r.qs) || !tile_ok(r.k, r.N, r.ks) || !tile_ok(r.v, r.P, r.vs) ||
        !tile_ok(r.out, r.P, r.os))
      return false;
  }
  return true;
}

cudaError_t launch_la_mma(const LaCall& a, LaPass pass, cudaStream_t s) {
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  const LaRole& r = a.role;
  if (!make_map(&maps.q, r.q, r.N, a.H / r.q_rep, a.rows, r.qs) ||
      !make_map(&maps.k, r.k, r.N, a.H / r.k_rep, a.rows, r.ks) ||
      !make_map(&maps.v, r.v, r.P, a.H / r.v_rep, a.rows, r.vs) ||
      (r.out_rep == 1 && !make_map(&maps.out, r.out, r.P, a.H, a.rows, r.os)))
    return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)((int64_t)a.B * a.H * a.nseg * ((r.P + 63) / 64));
  const bool sum = pass == kLaSummary;
  if (r.N > 64)
    return sum ? launch_role(k_la_mma<2, true>, grid, kThreads, kSmem, a.beside, s, a, maps)
               : launch_role(k_la_mma<2, false>, grid, kThreads, kSmem, a.beside, s, a, maps);
  return sum ? launch_role(k_la_mma<1, true>, grid, kThreads, kSmem, a.beside, s, a, maps)
             : launch_role(k_la_mma<1, false>, grid, kThreads, kSmem, a.beside, s, a, maps);
}

}  // namespace m3
