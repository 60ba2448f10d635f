// Linear attention with a decay per head, float32 arithmetic on the CUDA
// cores: the kernel of every shape, alignment and type that the tensor-core
// kernel does not take.
//
// A block of 256 threads walks the tokens of one (role, segment, sequence,
// head) 32 at a time, with q, k, v and the state S [N][P] of the head in shared
// memory as float32:
//   A_ij = lam^|i-j| intra (q_i.k_j)  on the causal side,
//   out_i = sum_j A_ij v_j + inter lam^(i'+1) S^T q_i,
//   S <- lam^n S + kv sum_j lam^(n-1-j') k_j v_j^T,
// where i' counts tokens in walking order. A thread holds small register tiles
// (up to 4 x 4 of the outputs, 16 x 4 of the state), so that a shared-memory
// word feeds 4 to 16 multiply-adds. The kernel is bound by those multiply-adds:
// N P (2 + 32 (1/N + 1/P)) a token.
#include "linattn.cuh"

namespace m3 {
namespace {

constexpr int kT = 32;  // tokens per chunk
constexpr int kThreads = 256;

struct SeqSmem {
  int ldn, ldp, q, k, v, s, a, pw, total;
};
__host__ __device__ inline SeqSmem seq_smem(int N, int P) {
  SeqSmem m;
  m.ldn = (N + 3) / 4 * 4 + 4;
  m.ldp = (P + 3) / 4 * 4 + 4;
  int o = 0;
  m.q = o; o += kT * m.ldn;
  m.k = o; o += kT * m.ldn;
  m.v = o; o += kT * m.ldp;
  m.s = o; o += (N + 3) / 4 * 4 * m.ldp;
  m.a = o; o += kT * (kT + 4);
  m.pw = o; o += kT + 4;
  m.total = o;
  return m;
}

// Rows t < kT of one head of an operand as float32; zeros past n tokens and w values.
template <typename T>
__device__ __forceinline__ void load_tile(float* dst, int ld, const T* src, int64_t stride, int n,
                                          int w) {
  const int wp = (w + 3) / 4 * 4;
  for (int i = threadIdx.x; i < kT * wp; i += kThreads) {
    const int t = i / wp, c = i - t * wp;
    dst[t * ld + c] = (t < n && c < w) ? to_f32(src[(int64_t)t * stride + c]) : 0.f;
  }
}

__device__ __forceinline__ void fma4x(float4& acc, float a, float4 b) {
  acc.x = fmaf(a, b.x, acc.x);
  acc.y = fmaf(a, b.y, acc.y);
  acc.z = fmaf(a, b.z, acc.z);
  acc.w = fmaf(a, b.w, acc.w);
}

// LP: lanes that share a row of P values, four each (32: P > 64, 16: P <= 64).
template <typename T, bool SUMMARY, int LP>
__global__ void __launch_bounds__(kThreads) k_la_seq(LaArgs a) {
  extern __shared__ __align__(16) float sm[];
  const int bh = blockIdx.x % (a.B * a.H);
  const int seg = blockIdx.x / (a.B * a.H) % a.nseg;
  const int ri = blockIdx.x / (a.B * a.H) / a.nseg;
  const LaRole& r = a.role[ri];
  const int b = bh / a.H, h = bh - b * a.H, tid = threadIdx.x;
  const int N = r.N, P = r.P, Np = (N + 3) / 4 * 4;
  const SeqSmem m = seq_smem(N, P);
  float *sq = sm + m.q, *sk = sm + m.k, *sv = sm + m.v, *ss = sm + m.s, *sa = sm + m.a;
  float* pw = sm + m.pw;
  int64_t row0, len;
  la_rows(a, b, &row0, &len);
  const int64_t s0 = seg * a.seg_len, s1 = min(len, s0 + a.seg_len);
  const int64_t last_seg = len > 0 ? (len - 1) / a.seg_len : 0;
  if (seg > last_seg) return;
  // the segment whose state the prefix pass never reads
  if (SUMMARY && seg == (r.reverse ? 0 : last_seg)) return;
  const bool first = seg == (r.reverse ? last_seg : 0), last = seg == (r.reverse ? 0 : last_seg);
  const float ld = a.log_decay[h];
  if (tid <= kT) pw[tid] = la_power(ld, tid);

  float* entry = a.entry ? a.entry + ri * a.entry_role +
                               ((int64_t)seg * a.B * a.H + bh) * ((int64_t)N * P)
                         : nullptr;
  const int64_t sbase = (int64_t)bh * N * P;
  for (int i = tid; i < Np * m.ldp; i += kThreads) ss[i] = 0.f;
  __syncthreads();
  if (!SUMMARY && (a.nseg > 1 || r.init)) {
    for (int i = tid; i < N * P; i += kThreads) {
      const int p = i / N, n = i - p * N;
      ss[n * m.ldp + p] = a.nseg > 1 ? entry[i] : r.init[sbase + (int64_t)p * r.sp + n * r.sn];
    }
  }
  const int shift0 = first ? r.shift : 0;
  const int nchunk = s1 > s0 ? (int)((s1 - s0 + kT - 1) / kT) : 0;
  const T* gq = (const T*)r.q + (int64_t)(h / r.q_rep) * N;
  const T* gk = (const T*)r.k + (int64_t)(h / r.k_rep) * N;
  const T* gv = (const T*)r.v + (int64_t)(h / r.v_rep) * P;
  for (int ci = 0; ci < nchunk; ++ci) {
    const int c = r.reverse ? nchunk - 1 - ci : ci;
    const int64_t t0 = s0 + (int64_t)c * kT;
    const int n = (int)min((int64_t)kT, s1 - t0);
    const int shift = ci == 0 ? shift0 : 0;
    const int64_t row = row0 + t0;
    __syncthreads();
    if (!SUMMARY) load_tile(sq, m.ldn, gq + row * r.qs, r.qs, n, N);
    load_tile(sk, m.ldn, gk + row * r.ks, r.ks, n, N);
    load_tile(sv, m.ldp, gv + row * r.vs, r.vs, n, P);
    __syncthreads();
    if (!SUMMARY) {
      {  // A: two rows and two columns a thread
        const int i0 = tid / 16 * 2, j0 = tid % 16 * 2;
        float acc[2][2] = {};
        for (int x = 0; x < Np; x += 4) {
          float4 qv[2], kv[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qv[e] = *(const float4*)(sq + (i0 + e) * m.ldn + x);
            kv[e] = *(const float4*)(sk + (j0 + e) * m.ldn + x);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acc[i][j] += qv[i].x * kv[j].x + qv[i].y * kv[j].y + qv[i].z * kv[j].z +
                           qv[i].w * kv[j].w;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int d = r.reverse ? j0 + j - i0 - i : i0 + i - j0 - j;
            sa[(i0 + i) * (kT + 4) + j0 + j] =
                (d >= 0 && j0 + j < n) ? acc[i][j] * pw[d] * r.intra : 0.f;
          }
      }
      __syncthreads();
      constexpr int RO = LP == 32 ? 4 : 2;  // output rows a thread
      const int i0 = tid / LP * RO, p0 = tid % LP * 4;
      if (p0 < P) {
        float4 acc[RO];
#pragma unroll
        for (int e = 0; e < RO; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x = 0; x < Np; x += 4) {
          float4 sv4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) sv4[e] = *(const float4*)(ss + (x + e) * m.ldp + p0);
#pragma unroll
          for (int e = 0; e < RO; ++e) {
            const float4 qv = *(const float4*)(sq + (i0 + e) * m.ldn + x);
            fma4x(acc[e], qv.x, sv4[0]);
            fma4x(acc[e], qv.y, sv4[1]);
            fma4x(acc[e], qv.z, sv4[2]);
            fma4x(acc[e], qv.w, sv4[3]);
          }
        }
#pragma unroll
        for (int e = 0; e < RO; ++e) {
          const int i = i0 + e, w = min(max(r.reverse ? n - 1 - i : i, 0), kT - 1);
          const float f = r.inter * pw[w + 1 - shift];
          acc[e].x *= f; acc[e].y *= f; acc[e].z *= f; acc[e].w *= f;
        }
        for (int x = 0; x < kT; x += 4) {
          float4 vv[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) vv[e] = *(const float4*)(sv + (x + e) * m.ldp + p0);
#pragma unroll
          for (int e = 0; e < RO; ++e) {
            const float4 av = *(const float4*)(sa + (i0 + e) * (kT + 4) + x);
            fma4x(acc[e], av.x, vv[0]);
            fma4x(acc[e], av.y, vv[1]);
            fma4x(acc[e], av.z, vv[2]);
            fma4x(acc[e], av.w, vv[3]);
          }
        }
#pragma unroll
        for (int e = 0; e < RO; ++e) {
          const int i = i0 + e;
          if (i >= n) continue;
          const float v4[4] = {acc[e].x, acc[e].y, acc[e].z, acc[e].w};
          const int64_t o = (row + i) * r.os + (int64_t)h * P + p0;
          for (int x = 0; x < 4 && p0 + x < P; ++x) {
            if (r.out_rep > 1) ((float*)r.out)[o + x] = v4[x];
            else ((T*)r.out)[o + x] = from_f32<T>(v4[x]);
          }
        }
      }
      __syncthreads();
    }
    {  // state: rows x of N, four values of P a thread
      constexpr int kGroups = kThreads / LP;
      constexpr int RS = 128 / kGroups;  // rows a thread, at most
      const int rows = (Np + kGroups - 1) / kGroups;
      const int x0 = tid / LP * rows, p0 = tid % LP * 4;
      if (p0 < P && x0 < N) {
        const float dec = pw[n - shift];
        float4 acc[RS];
#pragma unroll
        for (int e = 0; e < RS; ++e) {
          if (e < rows && x0 + e < N) {
            acc[e] = *(const float4*)(ss + (x0 + e) * m.ldp + p0);
            acc[e].x *= dec; acc[e].y *= dec; acc[e].z *= dec; acc[e].w *= dec;
          }
        }
        for (int j = 0; j < n; ++j) {
          const float w = r.kv * pw[r.reverse ? j : n - 1 - j];
          float4 vv = *(const float4*)(sv + j * m.ldp + p0);
          vv.x *= w; vv.y *= w; vv.z *= w; vv.w *= w;
#pragma unroll
          for (int e = 0; e < RS; ++e)
            if (e < rows && x0 + e < N) fma4x(acc[e], sk[j * m.ldn + x0 + e], vv);
        }
#pragma unroll
        for (int e = 0; e < RS; ++e)
          if (e < rows && x0 + e < N) *(float4*)(ss + (x0 + e) * m.ldp + p0) = acc[e];
      }
    }
  }
  __syncthreads();
  if (SUMMARY) {
    for (int i = tid; i < N * P; i += kThreads) {
      const int p = i / N, n = i - p * N;
      entry[i] = ss[n * m.ldp + p];
    }
  } else if (r.fin && last) {
    const float f = len > 0 && r.fin_shift ? pw[1] : 1.f;
    for (int i = tid; i < N * P; i += kThreads) {
      const int p = i / N, n = i - p * N;
      r.fin[sbase + (int64_t)p * r.sp + n * r.sn] = f * ss[n * m.ldp + p];
    }
  }
}

// Entry states of the segments from their own sums, in walking order: one
// thread per state element.
__global__ void __launch_bounds__(256) k_la_prefix(LaArgs a) {
  const int bh = blockIdx.x % (a.B * a.H), ri = blockIdx.x / (a.B * a.H);
  const LaRole& r = a.role[ri];
  const int i = blockIdx.y * 256 + threadIdx.x;
  if (i >= r.N * r.P) return;
  int64_t row0, len;
  la_rows(a, bh / a.H, &row0, &len);
  const float ld = a.log_decay[bh % a.H];
  const int last = len > 0 ? (int)((len - 1) / a.seg_len) : 0;
  const int p = i / r.N, n = i - p * r.N;
  float st = r.init ? r.init[(int64_t)bh * r.N * r.P + (int64_t)p * r.sp + n * r.sn] : 0.f;
  const int64_t step = (int64_t)a.B * a.H * r.N * r.P;
  float* e = a.entry + ri * a.entry_role + (int64_t)bh * r.N * r.P + i;
  for (int x = 0; x <= last; ++x) {
    const int seg = r.reverse ? last - x : x;
    float* at = e + seg * step;
    const float own = x < last ? *at : 0.f;
    *at = st;
    const int64_t n_tok = min(a.seg_len, len - seg * a.seg_len) - (x == 0 ? r.shift : 0);
    if (x < last) st = la_power(ld, n_tok) * st + own;
  }
}

// One row a block. With offsets, rows of no sequence keep what they hold.
template <typename T>
__global__ void __launch_bounds__(128)
    k_la_group_sum(LaArgs a, const float* part, T* out, int groups, int rep, int width) {
  const int64_t row = blockIdx.x;
  if (a.offsets) {
    int lo = 0, hi = a.B;  // the last sequence that begins at or before the row
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.offsets[mid] <= row) lo = mid;
      else hi = mid;
    }
    int64_t begin, len;
    la_rows(a, lo, &begin, &len);
    if (row < begin || row >= begin + len) return;
  }
  const int n = groups * width;
  for (int i = threadIdx.x; i < n; i += 128) {
    const int g = i / width;
    const float* src = part + (row * groups + g) * rep * (int64_t)width + (i - g * width);
    float s = 0.f;
    for (int x = 0; x < rep; ++x) s += src[(int64_t)x * width];
    out[row * n + i] = from_f32<T>(s);
  }
}

template <typename T, bool SUMMARY, int LP>
cudaError_t go(const LaArgs& a, cudaStream_t s) {
  size_t bytes = 0;
  for (int i = 0; i < a.nrole; ++i) {
    const size_t x = seq_smem(a.role[i].N, a.role[i].P).total * sizeof(float);
    bytes = x > bytes ? x : bytes;
  }
  cudaError_t e = cudaFuncSetAttribute(k_la_seq<T, SUMMARY, LP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  k_la_seq<T, SUMMARY, LP><<<(unsigned)((int64_t)a.B * a.H * a.nseg * a.nrole), kThreads, bytes,
                             s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}
template <typename T, bool SUMMARY>
cudaError_t by_width(const LaArgs& a, cudaStream_t s) {
  int P = 0;
  for (int i = 0; i < a.nrole; ++i) P = a.role[i].P > P ? a.role[i].P : P;
  return P > 64 ? go<T, SUMMARY, 32>(a, s) : go<T, SUMMARY, 16>(a, s);
}

}  // namespace

cudaError_t launch_la_seq(const LaArgs& a, LaPass pass, cudaStream_t s) {
  const bool f32 = a.dtype == M3_DTYPE_FP32;
  if (pass == kLaSummary)
    return f32 ? by_width<float, true>(a, s) : by_width<__nv_bfloat16, true>(a, s);
  return f32 ? by_width<float, false>(a, s) : by_width<__nv_bfloat16, false>(a, s);
}

cudaError_t launch_la_prefix(const LaArgs& a, cudaStream_t s) {
  int np = 0;
  for (int i = 0; i < a.nrole; ++i) {
    const int x = a.role[i].N * a.role[i].P;
    np = x > np ? x : np;
  }
  k_la_prefix<<<dim3((unsigned)(a.B * a.H * a.nrole), (unsigned)((np + 255) / 256)), 256, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_la_group_sum(const LaArgs& a, const float* part, void* out, int groups, int rep,
                                int width, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  if (a.dtype == M3_DTYPE_FP32)
    k_la_group_sum<<<(unsigned)a.rows, 128, 0, s>>>(a, part, (float*)out, groups, rep, width);
  else
    k_la_group_sum<<<(unsigned)a.rows, 128, 0, s>>>(a, part, (__nv_bfloat16*)out, groups, rep, width);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace m3
