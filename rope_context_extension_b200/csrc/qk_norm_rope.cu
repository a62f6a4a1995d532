// Norms of queries and keys for each head with the position rotation in the
// same pass, and optionally the append of k and v to a paged cache.
//
//   y = R(pos) (x * rsqrt(mean(x^2) + eps) * w)
//
// per head row x of D values: a root-mean-square norm with one weight vector for
// the query heads and one for the key heads (either may be absent), then the
// rotation of the half-split pairs (t, t + D/2) by pos * theta_t.  Squares, sums
// and the rotation are fp32 on the bf16 inputs; the result is rounded to bf16
// once.  Values go through unrotated.
//
// Memory bound: every row is read once and written once.  A lane holds 8 values
// of a row's first half and the 8 that pair with them in the second (two 16-byte
// loads), so a row takes D/16 lanes, the sum of squares takes log2(D/16)
// shuffles, and no value crosses lanes for the rotation.  A warp handles 512 / D
// rows at a time and a slice of one token's heads per task; the token's D/2
// factors are formed once per task, two per lane (one for D = 64), and shared
// through shared memory.
#include <algorithm>

#include "jl_paged.cuh"

namespace jl {

namespace {

constexpr int kNrThreads = 256;
constexpr int kBlocksPerSm = 3;  // resident at 80 registers a thread

__device__ __forceinline__ void bf16x8_to_f32(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(u[i]);
    x[2 * i + 1] = bf16hi_to_f32(u[i]);
  }
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

template <int D>
__global__ void __launch_bounds__(kNrThreads, kBlocksPerSm) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int H2 = D / 2;
  constexpr int kLanes = D / 16;       // lanes per head row
  constexpr int kRows = 32 / kLanes;   // head rows per pass of a warp
  constexpr int kOwn = H2 / 32;        // angles a lane forms
  __shared__ __align__(16) float2 cs_all[kNrThreads / 32][H2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2* cs = cs_all[warp];
  const int sub = lane % kLanes, grp = lane / kLanes;
  double uh[kOwn], ul[kOwn];
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    uh[e] = a.u_hi[lane + 32 * e];
    ul[e] = a.u_lo[lane + 32 * e];
  }
  const int heads = a.Hq + a.Hkv + (a.v != nullptr ? a.Hkv : 0);
  const int64_t tasks = (int64_t)a.T * a.tasks_per_token;
  const int64_t nwarps = (int64_t)gridDim.x * (kNrThreads / 32);
  for (int64_t task = (int64_t)blockIdx.x * (kNrThreads / 32) + warp; task < tasks; task += nwarps) {
    const int64_t tok = task / a.tasks_per_token;
    const int slice = (int)(task - tok * a.tasks_per_token);
    const int pos = a.positions[tok];
    if (pos == -1) continue;  // a padded token
    bool bad = pos < 0;
    int64_t kv_base = 0;  // offset of the token's row in the pages, head 0
    if (a.v != nullptr) {
      const int sq = a.seq_ids[tok];
      bad = bad || sq < 0 || sq >= a.B || (int64_t)pos >= a.max_pages * a.pages.page_size;
      if (!bad) {
        const int page = a.block_table[(int64_t)sq * a.max_pages + pos / a.pages.page_size];
        bad = page < 0 || page >= a.pages.num_pages;
        kv_base = page * a.pages.page_stride + (int64_t)(pos % a.pages.page_size) * a.pages.row_stride;
      }
    }
    if (bad) {
      if (lane == 0 && a.dev_error) atomicExch(a.dev_error, kDevBadLength);
      continue;
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
      float s, c;
      sincos_turns(pos, uh[e], ul[e], &s, &c);
      cs[lane + 32 * e] = make_float2(c, s);
    }
    __syncwarp();
    float2 f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = cs[8 * sub + e];

    const int h0 = (int)(slice * a.heads_per_task);
    const int h1 = min(heads, (int)(h0 + a.heads_per_task));
    for (int hb = h0; hb < h1; hb += kRows) {
      const int h = hb + grp;
      const bool live = h < h1;
      const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
      const int hk = h - a.Hq - (is_v ? a.Hkv : 0);
      const __nv_bfloat16* src = is_q   ? a.q + tok * a.q_stride + (int64_t)h * D
                                 : is_v ? a.v + tok * a.v_stride + (int64_t)hk * D
                                        : a.k + tok * a.k_stride + (int64_t)hk * D;
      uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
      if (live) {
        lo = *reinterpret_cast<const uint4*>(src + 8 * sub);
        hi = *reinterpret_cast<const uint4*>(src + H2 + 8 * sub);
      }
      float x[8], y[8];
      bf16x8_to_f32(lo, x);
      bf16x8_to_f32(hi, y);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e] + y[e] * y[e];
#pragma unroll
      for (int m = 1; m < kLanes; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      if (!live) continue;
      if (!is_v) {
        const __nv_bfloat16* w = is_q ? a.qw : a.kw;
        if (w != nullptr) {
          const float inv = rsqrtf(ss * (1.f / D) + a.eps);
          float wx[8], wy[8];
          bf16x8_to_f32(*reinterpret_cast<const uint4*>(w + 8 * sub), wx);
          bf16x8_to_f32(*reinterpret_cast<const uint4*>(w + H2 + 8 * sub), wy);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = x[e] * inv * wx[e];
            y[e] = y[e] * inv * wy[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xr = x[e] * f[e].x - y[e] * f[e].y;
          y[e] = y[e] * f[e].x + x[e] * f[e].y;
          x[e] = xr;
        }
        lo = f32_to_bf16x8(x);
        hi = f32_to_bf16x8(y);
      }
      if (is_q || (!is_v && a.k_out != nullptr)) {
        __nv_bfloat16* dst = is_q ? a.q_out + (tok * a.Hq + h) * D : a.k_out + (tok * a.Hkv + hk) * D;
        *reinterpret_cast<uint4*>(dst + 8 * sub) = lo;
        *reinterpret_cast<uint4*>(dst + H2 + 8 * sub) = hi;
      }
      if (!is_q && a.v != nullptr) {
        __nv_bfloat16* dst = (is_v ? a.pages.v : a.pages.k) + kv_base + hk * a.pages.head_stride;
        *reinterpret_cast<uint4*>(dst + 8 * sub) = lo;
        *reinterpret_cast<uint4*>(dst + H2 + 8 * sub) = hi;
      }
    }
  }
}

template <int D>
cudaError_t launch_d(NormRopeArgs& a, cudaStream_t stream) {
  constexpr int kRows = 512 / D;
  const int sms = current_device_sms();
  if (sms == 0) return cudaErrorNoDevice;
  const int heads = a.Hq + a.Hkv + (a.v != nullptr ? a.Hkv : 0);
  const int passes = (heads + kRows - 1) / kRows;
  // One pass of a warp per task while the tokens do not fill the GPU's warps (a
  // decode step's latency); whole tokens per task (the factors formed once) when
  // they do.
  const int64_t warps = (int64_t)sms * kBlocksPerSm * (kNrThreads / 32);
  int64_t per_task = ((int64_t)a.T * passes + warps - 1) / warps;
  if (per_task > passes) per_task = passes;
  a.heads_per_task = per_task * kRows;
  a.tasks_per_token = (int)((passes + per_task - 1) / per_task);
  const int64_t tasks = (int64_t)a.T * a.tasks_per_token;
  const int64_t blocks = std::min<int64_t>((tasks + kNrThreads / 32 - 1) / (kNrThreads / 32), (int64_t)sms * kBlocksPerSm);
  norm_rope_kernel<D><<<(unsigned)blocks, kNrThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeArgs& a, int D, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace jl
