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
// rows at a time, the next ones already on their way, across tasks too, and a slice of
// one token's heads per task; the token's D/2 factors are formed once per task, two per lane,
// and shared through shared memory (64-bit fixed-point angles and the MUFU's sine:
// 2^-21, against the result's 2^-8).
//
// Measured (B200, 32 query and 8 KV heads, D 128): a prompt of 131072 tokens appended
// to its pages 518 us = 6.2 TB/s, 0.95 of a copy; 8192 tokens without an append 32.5
// us = 5.2 TB/s, 0.79 (the launch, the first loads and the uneven end are about 5 us);
// 8 tokens 3.2 us, all latency.
#include <algorithm>

#include "jl_mma.cuh"
#include "jl_paged.cuh"

namespace jl {

namespace {

constexpr int kNrThreads = 256;
constexpr int kBlocksPerSm = 3;  // resident at 80 registers a thread (a grid of four: 131072 tokens 796 us)

// A packed fp32 pair rounded to bf16x2.
__device__ __forceinline__ uint32_t f2_to_bf16x2(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return pack_bf16x2(a, b);
}

template <int D>
__global__ void __launch_bounds__(kNrThreads, kBlocksPerSm) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int H2 = D / 2;
  constexpr int kLanes = D / 16;       // lanes per head row
  constexpr int kRows = 32 / kLanes;   // head rows per pass of a warp
  __shared__ __align__(16) float4 cs_all[kNrThreads / 32][H2 / 2];  // a token's factors (c, c, s, s)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float4* cs = cs_all[warp];
  const int sub = lane % kLanes, grp = lane / kLanes;
  // the pairs ft, ft + 1 whose factors this lane forms, where lanes of a row read them side by side
  const int fl = lane % (H2 / 2), ft = 8 * (fl % kLanes) + 2 * (fl / kLanes);
  uint64_t turn0, turn1;
  {
    const uint64_t* tp = a.turn;  // a generic read: an indexed parameter read serialises
    asm volatile("" : "+l"(tp));
    turn0 = tp[ft];
    turn1 = tp[ft + 1];
  }
  const int heads = a.Hq + a.Hkv + (a.v != nullptr ? a.Hkv : 0);
  const int64_t tasks = (int64_t)a.T * a.tasks_per_token;
  const int64_t nwarps = (int64_t)gridDim.x * (kNrThreads / 32);
  int64_t task = (int64_t)blockIdx.x * (kNrThreads / 32) + warp;
  // The next task: its token, heads, position and row in the pages (head 0), looked up
  // while the task before is worked on; next_h0 = next_h1: none.
  int next_tok = 0, next_h0 = 0, next_h1 = 0, next_pos = -1;
  int64_t next_base = 0;
  auto describe = [&](int64_t t) {
    next_h0 = next_h1 = 0;
    next_pos = -1;
    if (t >= tasks) return;
    next_tok = (int)(a.tasks_per_token == 1 ? t : t / a.tasks_per_token);
    next_h0 = (int)(t - (int64_t)next_tok * a.tasks_per_token) * a.heads_per_task;
    next_h1 = min(heads, next_h0 + a.heads_per_task);
    next_pos = a.positions[next_tok];
    if (next_pos == -1) return;  // a padded token
    bool bad = next_pos < 0;
    if (a.v != nullptr) {
      const int sq = a.seq_ids[next_tok];
      bad = bad || sq < 0 || sq >= a.B || (int64_t)next_pos >= a.max_pages * a.pages.page_size;
      if (!bad) {
        const int lp = next_pos / a.pages.page_size;
        const int page = a.block_table[(int64_t)sq * a.max_pages + lp];
        bad = page < 0 || page >= a.pages.num_pages;
        next_base = page * a.pages.page_stride + (int64_t)(next_pos - lp * a.pages.page_size) * a.pages.row_stride;
      }
    }
    if (bad) {
      if (lane == 0 && a.dev_error) atomicExch(a.dev_error, kDevBadLength);
      next_pos = -1;
    }
  };
  // a pass's rows: loaded one pass ahead, a task's first while the last of the task before is worked on
  uint4 lo, hi, next_lo, next_hi;
  auto load = [&](int64_t tok, int h, int h1) {
    next_lo = next_hi = make_uint4(0, 0, 0, 0);
    if (h < h1) {
      const __nv_bfloat16* src = h < a.Hq ? a.q + tok * a.q_stride + (int64_t)h * D
                                 : h < a.Hq + a.Hkv
                                     ? a.k + tok * a.k_stride + (int64_t)(h - a.Hq) * D
                                     : a.v + tok * a.v_stride + (int64_t)(h - a.Hq - a.Hkv) * D;
      next_lo = *reinterpret_cast<const uint4*>(src + 8 * sub);
      next_hi = *reinterpret_cast<const uint4*>(src + H2 + 8 * sub);
    }
  };
  describe(task);
  load(next_tok, next_h0 + grp, next_h1);
  for (; task < tasks; task += nwarps) {
    const int64_t tok = next_tok, kv_base = next_base;
    const int h0 = next_h0, h1 = next_h1, pos = next_pos;
    describe(task + nwarps);
    if (pos < 0) {
      load(next_tok, next_h0 + grp, next_h1);
      continue;
    }
    {
      float4 f;
      sincos_phase(pos, turn0, &f.z, &f.x);
      sincos_phase(pos, turn1, &f.w, &f.y);
      __syncwarp();
      cs[fl] = f;
      __syncwarp();
    }
    for (int hb = h0; hb < h1; hb += kRows) {
      const int h = hb + grp;
      lo = next_lo;
      hi = next_hi;
      if (hb + kRows < h1)
        load(tok, h + kRows, h1);
      else
        load(next_tok, next_h0 + grp, next_h1);
      const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
      const int hk = h - a.Hq - (is_v ? a.Hkv : 0);
      uint64_t x[4], y[4];  // packed fp32 pairs: half the instructions, which bound short rows
      uint64_t sq = 0ull;
      {
        const uint32_t xw[4] = {lo.x, lo.y, lo.z, lo.w}, yw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = bf16x2_to_f2(xw[e]);
          y[e] = bf16x2_to_f2(yw[e]);
          sq = f2_fma(x[e], x[e], f2_fma(y[e], y[e], sq));
        }
      }
      float ss, ss1;
      f2_unpack(sq, ss, ss1);
      ss += ss1;
#pragma unroll
      for (int m = 1; m < kLanes; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      if (h >= h1) continue;
      if (!is_v) {
        const __nv_bfloat16* w = is_q ? a.qw : a.kw;
        if (w != nullptr) {
          const float inv = rsqrtf(ss * (1.f / D) + a.eps);
          const uint64_t inv2 = f2_pack(inv, inv);
          const uint4 wl = *reinterpret_cast<const uint4*>(w + 8 * sub);
          const uint4 wh = *reinterpret_cast<const uint4*>(w + H2 + 8 * sub);
          const uint32_t wx[4] = {wl.x, wl.y, wl.z, wl.w}, wy[4] = {wh.x, wh.y, wh.z, wh.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = f2_mul(f2_mul(x[e], inv2), bf16x2_to_f2(wx[e]));
            y[e] = f2_mul(f2_mul(y[e], inv2), bf16x2_to_f2(wy[e]));
          }
        }
        uint32_t xo[4], yo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 f = cs[e * kLanes + sub];
          const uint64_t c = f2_pack(f.x, f.y), sn = f2_pack(f.z, f.w);
          xo[e] = f2_to_bf16x2(f2_sub(f2_mul(x[e], c), f2_mul(y[e], sn)));
          yo[e] = f2_to_bf16x2(f2_fma(x[e], sn, f2_mul(y[e], c)));
        }
        lo = make_uint4(xo[0], xo[1], xo[2], xo[3]);
        hi = make_uint4(yo[0], yo[1], yo[2], yo[3]);
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
  // Passes per task: what keeps the resident warps' last round full, counting half a
  // pass for a task's own start (4096 tokens 18.6 us, with two passes 19.5, four 19.5 and
  // 8192 tokens 34.7 instead of 32.5).
  const int64_t warps = (int64_t)sms * kBlocksPerSm * (kNrThreads / 32);
  int64_t best = INT64_MAX;
  for (int per = 1; per <= passes; ++per) {
    const int each = (passes + per - 1) / per;
    const int64_t cost = (((int64_t)a.T * each + warps - 1) / warps) * (2 * per + 1);
    if (cost < best) {
      best = cost;
      a.heads_per_task = per * kRows;
      a.tasks_per_token = each;
    }
  }
  const int64_t tasks = (int64_t)a.T * a.tasks_per_token;
  const int64_t blocks =
      std::min<int64_t>((tasks + kNrThreads / 32 - 1) / (kNrThreads / 32), (int64_t)sms * kBlocksPerSm);
  norm_rope_kernel<D><<<(unsigned)blocks, kNrThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeArgs& a, int D, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace jl
