// Page summaries, page scores and the selection of the pages that a sparse
// decode step attends to.
//
// Summary of page p with n valid keys, m = page_size / 2 (fp32, rounded to bf16):
//   c_p = (1/n) sum_t R(m - t) k_{p page_size + t}
// i.e. the page's mean key, every key taken from its own position to the page's
// middle one first.  It is a key at position p page_size + m like any other in
// the cache, so it holds for every group size G and is never rewritten when G
// changes.
//
// Score of page p for KV head g, c = p page_size + m, as a remote pair:
//   s = max over the head's queries of <R(p_q(i) - i) q_h, R(f(c) - c) c_p>
// Kept pages: the first sink_pages, those that touch the band j >= L - w0 (base
// RoPE scores) and the last one, and the top_k best scores of the others, ties
// to the lowest page.  Listed in ascending order, the rest of the row is -1.
#include <algorithm>

#include "jl_paged.cuh"

namespace jl {

namespace {

constexpr int kSumThreads = 256;
constexpr int kScoreThreads = 256;
constexpr int kScorePages = 16;  // pages per CTA of the score kernel
constexpr int kSelThreads = 512;

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(u[i]);
    x[2 * i + 1] = bf16hi_to_f32(u[i]);
  }
}

// One warp per (page, KV head).  A key row takes D/16 lanes of two 16-byte loads,
// a warp reads 512 / D rows at a time, and each group of lanes sums its rows by
// Horner's rule in R(-step): sum_i R(-step i) k_{step i + grp}, so that two fixed
// rotations per lane, formed once per warp, serve every page.
template <int D>
__global__ void __launch_bounds__(kSumThreads) page_summary_kernel(const __grid_constant__ PageSummaryArgs a) {
  constexpr int H2 = D / 2;
  constexpr int kLanes = D / 16;
  constexpr int kStep = 32 / kLanes;  // rows per pass
  const int lane = threadIdx.x & 31;
  const int sub = lane % kLanes, grp = lane / kLanes;
  const int P = a.pages.page_size;
  float sc[8], ss[8], mc[8], ms[8];  // R(-step), R(m - grp)
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    sincos_turns(-kStep, a.u_hi[8 * sub + e], a.u_lo[8 * sub + e], &ss[e], &sc[e]);
    sincos_turns(P / 2 - grp, a.u_hi[8 * sub + e], a.u_lo[8 * sub + e], &ms[e], &mc[e]);
  }
  const int64_t tasks = (int64_t)a.B * a.pages_per_seq * a.Hkv;
  const int64_t nwarps = (int64_t)gridDim.x * (kSumThreads / 32);
  for (int64_t task = ((int64_t)blockIdx.x * kSumThreads + threadIdx.x) >> 5; task < tasks; task += nwarps) {
    const int g = (int)(task % a.Hkv);
    const int64_t bp = task / a.Hkv;
    const int b = (int)(bp / a.pages_per_seq);
    const int i = (int)(bp - (int64_t)b * a.pages_per_seq);
    const int L = a.seq_lens[b], start = a.starts[b];
    const bool ok = paged_length_ok(L, a.max_pages, P) && start >= 0;
    // more new pages than the call was sized for: refuse the sequence
    const bool over = ok && start < L && (L - 1) / P - start / P >= a.pages_per_seq;
    if (!ok || over) {
      if (lane == 0 && a.dev_error) atomicExch(a.dev_error, kDevBadLength);
      continue;
    }
    const int lp = start / P + i;
    if (start >= L || lp > (L - 1) / P) continue;
    const int phys = a.block_table[(int64_t)b * a.max_pages + lp];
    if (phys < 0 || phys >= a.pages.num_pages) {
      if (lane == 0 && a.dev_error) atomicExch(a.dev_error, kDevBadLength);
      continue;
    }
    const int n = min(P, L - lp * P);
    const __nv_bfloat16* base = a.pages.k + phys * a.pages.page_stride + g * a.pages.head_stride;
    float x[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
    for (int r0 = (n - 1) / kStep * kStep; r0 >= 0; r0 -= kStep) {
      const int t = r0 + grp;
      uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
      if (t < n) {
        lo = *reinterpret_cast<const uint4*>(base + t * a.pages.row_stride + 8 * sub);
        hi = *reinterpret_cast<const uint4*>(base + t * a.pages.row_stride + H2 + 8 * sub);
      }
      float kx[8], ky[8];
      unpack8(lo, kx);
      unpack8(hi, ky);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xr = kx[e] + (x[e] * sc[e] - y[e] * ss[e]);
        y[e] = ky[e] + (y[e] * sc[e] + x[e] * ss[e]);
        x[e] = xr;
      }
    }
    const float inv = 1.f / (float)n;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xr = x[e] * mc[e] - y[e] * ms[e];
      y[e] = y[e] * mc[e] + x[e] * ms[e];
      x[e] = xr;
#pragma unroll
      for (int m = kLanes; m < 32; m <<= 1) {
        x[e] += __shfl_xor_sync(0xffffffffu, x[e], m);
        y[e] += __shfl_xor_sync(0xffffffffu, y[e], m);
      }
      x[e] *= inv;
      y[e] *= inv;
    }
    if (grp == 0) {
      __nv_bfloat16* dst = a.summaries + ((int64_t)phys * a.Hkv + g) * D + 8 * sub;
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                  pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      *reinterpret_cast<uint4*>(dst + H2) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                       pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    }
  }
}

// First page of the band and of the pages behind the sequence, and the open ones
// between the sink and the band (those that are scored).
struct PageSpan {
  int pages;       // of the sequence
  int sink, band;  // scored pages are [sink, band)
};
__device__ __forceinline__ PageSpan page_span(const PageSelectArgs& a, int b) {
  const int L = a.seq_lens[b];
  if (!paged_length_ok(L, a.max_pages, a.page_size) || L == 0) return {0, 0, 0};
  const int last = (L - 1) / a.page_size;
  const int band = min(last, max(0, L - a.w0) / a.page_size);
  return {last + 1, min(a.sink_pages, band), band};
}

// Scores in 64 bits: products of two bf16 values are exact, the angles are good
// to 1e-10, and the sum is rounded to fp32 once, so that which page lies above a
// border does not depend on the order of a sum.  One warp per KV head and page,
// the factors of a CTA's pages in shared memory.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const __grid_constant__ PageSelectArgs a) {
  constexpr int H2 = D / 2;
  constexpr int kOwn = H2 / 32;
  __shared__ double2 cs[kScorePages + 1][H2];  // row kScorePages: the queries' own factors
  const int b = blockIdx.y;
  const PageSpan sp = page_span(a, b);
  const int p0 = sp.sink + blockIdx.x * kScorePages;
  if (p0 >= sp.band) return;
  const int np = min(kScorePages, sp.band - p0);
  const int L = a.seq_lens[b];
  const int64_t G = group_size(L, a.w_pretrained);
  const int64_t dq = query_remote(L - 1, G, query_shift(a.w0, G, a.qshift)) - (L - 1);
  for (int idx = threadIdx.x; idx < (kScorePages + 1) * H2; idx += kScoreThreads) {
    const int row = idx / H2, t = idx % H2;
    const int64_t c = (int64_t)(p0 + row) * a.page_size + a.page_size / 2;
    const int64_t n = row == kScorePages ? dq : key_remote(c, G) - c;
    double s, co;
    sincos_int_angle(n, a.u_hi[t], a.u_lo[t], &s, &co);
    cs[row][t] = make_double2(co, s);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp % a.Hkv; g < a.Hkv; g += kScoreThreads / 32) {
    const int share = max(1, kScoreThreads / 32 / a.Hkv);  // warps per KV head
    const int first = a.Hkv >= kScoreThreads / 32 ? 0 : warp / a.Hkv;
    if (first >= share) break;
    double qx[8][kOwn], qy[8][kOwn];
#pragma unroll
    for (int h = 0; h < 8; ++h)
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        const int t = lane + 32 * e;
        double x = 0.0, y = 0.0;
        if (h < a.r) {
          const __nv_bfloat16* q = a.q + ((int64_t)b * a.Hq + g * a.r + h) * D;
          x = (double)__bfloat162float(q[t]);
          y = (double)__bfloat162float(q[t + H2]);
        }
        const double2 f = cs[kScorePages][t];
        qx[h][e] = x * f.x - y * f.y;
        qy[h][e] = y * f.x + x * f.y;
      }
    for (int i = first; i < np; i += share) {
      const int phys = a.block_table[(int64_t)b * a.max_pages + p0 + i];
      float best = -INFINITY;
      if (phys >= 0 && phys < a.num_pages) {
        const __nv_bfloat16* k = a.summaries + ((int64_t)phys * a.Hkv + g) * D;
        double kx[kOwn], ky[kOwn];
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
          const int t = lane + 32 * e;
          const double x = (double)__bfloat162float(k[t]), y = (double)__bfloat162float(k[t + H2]);
          const double2 f = cs[i][t];
          kx[e] = x * f.x - y * f.y;
          ky[e] = y * f.x + x * f.y;
        }
        double bd = -INFINITY;
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          if (h >= a.r) break;
          double s = 0.0;
#pragma unroll
          for (int e = 0; e < kOwn; ++e) s += qx[h][e] * kx[e] + qy[h][e] * ky[e];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          bd = s != s || s > bd ? s : bd;  // a NaN stays
          if (s != s) break;
        }
        best = (float)bd;
      } else if (lane == 0 && a.dev_error) {
        atomicExch(a.dev_error, kDevBadLength);
      }
      if (lane == 0) a.scores[((int64_t)b * a.Hkv + g) * a.max_pages + p0 + i] = best;
    }
  }
}

// Order-preserving key of a score: larger score, larger key; -0 = +0; NaN above all.
__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0xffffffffu;
  const uint32_t u = __float_as_uint(s + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (KV head, sequence): radix selection of the top_k-th largest score
// key (four passes of 8 bits over the scores), then one pass in page order that
// writes the kept pages.
__global__ void __launch_bounds__(kSelThreads) page_select_kernel(const __grid_constant__ PageSelectArgs a) {
  __shared__ int hist[256];
  __shared__ int bucket, above;
  __shared__ int wk[kSelThreads / 32], wt[kSelThreads / 32];
  const int g = blockIdx.x, b = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = (int64_t)b * a.Hkv + g;
  const PageSpan sp = page_span(a, b);
  const float* sc = a.scores + row * a.max_pages;
  int* list = a.page_list + row * a.list_stride;
  const int cand = sp.band - sp.sink;
  if (tid == 0 && a.dev_error && !paged_length_ok(a.seq_lens[b], a.max_pages, a.page_size))
    atomicExch(a.dev_error, kDevBadLength);

  uint32_t thr = 0;  // pages with a larger key are kept, and the first `ties` with this key
  int ties = 0;
  if (cand > a.top_k && a.top_k > 0) {
    int need = a.top_k;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int p = sp.sink + tid; p < sp.band; p += kSelThreads) {
        const uint32_t key = score_key(sc[p]);
        if (shift == 24 || (key >> (shift + 8)) == (thr >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255u], 1);
      }
      __syncthreads();
      if (warp == 0) {  // the bucket, from the top, that holds the need-th key
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = hist[255 - (8 * lane + i)];
          sum += c[i];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        int run = incl - sum;
        if (run < need && need <= incl) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (run < need && need <= run + c[i]) {
              bucket = 255 - (8 * lane + i);
              above = run;
            }
            run += c[i];
          }
        }
      }
      __syncthreads();
      thr |= (uint32_t)bucket << shift;
      need -= above;
      __syncthreads();
    }
    ties = need;
  }
  const bool all = cand <= a.top_k;

  int written = 0, seen = 0;  // kept pages so far, pages with the border key so far
  for (int base = 0; base < sp.pages; base += kSelThreads) {
    const int p = base + tid;
    bool keep = false, tie = false;
    if (p < sp.pages) {
      if (p < sp.sink || p >= sp.band || all) {
        keep = true;
      } else if (a.top_k > 0) {
        const uint32_t key = score_key(sc[p]);
        keep = key > thr;
        tie = key == thr;
      }
    }
    const unsigned tb = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) wt[warp] = __popc(tb);
    __syncthreads();
    int trank = seen + __popc(tb & ((1u << lane) - 1u)), tall = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) trank += wt[w];
      tall += wt[w];
    }
    seen += tall;
    keep = keep || (tie && trank < ties);
    const unsigned kb = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) wk[warp] = __popc(kb);
    __syncthreads();
    int at = written + __popc(kb & ((1u << lane) - 1u)), kall = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) at += wk[w];
      kall += wk[w];
    }
    if (keep && at < a.list_stride) list[at] = p;
    written += kall;
  }
  for (int64_t i = written + tid; i < a.list_stride; i += kSelThreads) list[i] = -1;
  if (tid == 0) a.page_counts[row] = written;
}

template <int D>
cudaError_t launch_summary_d(const PageSummaryArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 148, per_sm = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, page_summary_kernel<D>, kSumThreads, 0)) !=
      cudaSuccess)
    return e;
  const int64_t tasks = (int64_t)a.B * a.pages_per_seq * a.Hkv;
  const int64_t blocks = std::min<int64_t>((tasks + kSumThreads / 32 - 1) / (kSumThreads / 32), (int64_t)sms * per_sm);
  page_summary_kernel<D><<<(unsigned)blocks, kSumThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_page_summaries(const PageSummaryArgs& a, int D, cudaStream_t stream) {
  return D == 128 ? launch_summary_d<128>(a, stream) : launch_summary_d<64>(a, stream);
}

cudaError_t launch_page_select(const PageSelectArgs& a, int D, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.max_pages + kScorePages - 1) / kScorePages), a.B);
  if (a.top_k > 0) {
    if (D == 128)
      page_score_kernel<128><<<grid, kScoreThreads, 0, stream>>>(a);
    else
      page_score_kernel<64><<<grid, kScoreThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  page_select_kernel<<<dim3(a.Hkv, a.B), kSelThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace jl
