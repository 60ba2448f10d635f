// Linear attention, the passes around the chunk kernels: entry states of the
// segments of long sequences, and sums of gradients over the heads of a group.
#include "linattn.cuh"

namespace m3 {
namespace {

// Entry states of the segments from their own sums, in walking order: one
// thread per state element, the sums of eight segments in flight at a time.
__global__ void __launch_bounds__(256) k_la_prefix(const __grid_constant__ LaArgs args) {
  constexpr int kAhead = 8;
  const LaCall& a = args.call;
  const int bh = blockIdx.x % (a.B * a.H), ri = blockIdx.x / (a.B * a.H);
  const LaRole& r = args.role[ri];
  const int np = r.N * r.P, i = blockIdx.y * 256 + threadIdx.x;
  if (i >= np) return;
  int64_t row0, len;
  la_rows(a, bh / a.H, &row0, &len);
  const float ld = a.log_decay[bh % a.H];
  const int last = len > 0 ? (int)((len - 1) / a.seg_len) : 0;
  const int p = i / r.N, n = i - p * r.N;
  float st = r.init ? r.init[(int64_t)bh * np + (int64_t)p * r.sp + (int64_t)n * r.sn] : 0.f;
  const int64_t step = (int64_t)a.B * a.H * np;
  float* e = a.entry + ri * args.entry_role + (int64_t)bh * np + i;
  // every segment but the sequence's last rows' one has seg_len tokens
  const float whole = la_power(ld, a.seg_len), tail = la_power(ld, len - last * a.seg_len);
  for (int x0 = 0; x0 <= last; x0 += kAhead) {
    float own[kAhead];
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int x = x0 + y;
      own[y] = x < last ? e[(r.reverse ? last - x : x) * step] : 0.f;
    }
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int x = x0 + y, seg = r.reverse ? last - x : x;
      if (x > last) break;
      e[seg * step] = st;
      float dec = seg == last ? tail : whole;
      if (x == 0 && r.shift) dec = la_power(ld, (seg == last ? len - last * a.seg_len : a.seg_len) - 1);
      st = fmaf(dec, st, own[y]);
    }
  }
}

// One row a block. With offsets, rows of no sequence keep what they hold.
template <typename T>
__global__ void __launch_bounds__(128)
    k_la_group_sum(const __grid_constant__ LaCall a, const float* part, T* out, int groups, int rep, int width) {
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

}  // namespace

cudaError_t launch_la_prefix(const LaArgs& a, cudaStream_t s) {
  int np = 0;
  for (int i = 0; i < a.nrole; ++i) {
    const int x = a.role[i].N * a.role[i].P;
    np = x > np ? x : np;
  }
  k_la_prefix<<<dim3((unsigned)(a.call.B * a.call.H * a.nrole), (unsigned)((np + 255) / 256)), 256, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_la_group_sum(const LaCall& a, const float* part, void* out, int groups, int rep,
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
