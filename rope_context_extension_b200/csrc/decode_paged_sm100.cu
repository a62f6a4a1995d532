// Paged Dynamic Bifocal RoPE decode for sm_100a: one new query token per
// sequence against the pages that its row of a block table names, or against a
// selected list of them per KV head.
//
// For sequence b of length L (query at position i = L - 1, G = group size of L):
//   s_j = scale <q, k_j>                                  for i - j < w0 (base RoPE)
//   s_j = scale <R(p_q(i) - i) q, R(f(j) - j) k_j>        otherwise
//   o = softmax(s) V, lse = ln sum_j exp(s_j); an empty sequence or list gives
//   o = 0, lse = -inf.
// Keys sit in the pages rotated at their absolute positions and are only read
// (Jet-Long review, "Method"; gist.science summary, "§2 On-the-Fly Correctie
// Rotatie").
//
// Bound by HBM: every key and value is read once, 4 D bytes per key and KV head,
// against 4 D r flop.
//
// Work split.  A unit is 16 consecutive keys of one (sequence, KV head) item; a
// page holds a whole number of them.  All units of the call, in item order, form
// one line that is cut evenly over the CTAs (one per SM) and again over each
// CTA's warps, from the lengths on the device: a batch of any mix of lengths
// keeps every warp equally busy, whatever the host knew.  A warp walks its units
// through a ring of its own (TMA boxes of 16 rows, one mbarrier per slot, no
// barrier shared between warps).  Where a cut falls inside an item, partials
// (maximum, sum, unnormalised output) join twice: the warps' in shared memory at
// the CTA's end, the CTAs' in scratch by whichever CTA takes the item's last
// ticket (no spinning), each time in unit order, so results do not depend on
// timing.
//
// Scores use mma.sync m16n8k16 with the query heads on the M axis.  A remote
// unit starting at position j0 has dk(j) = dk(j0) - e(j) with e(j) in [0, 15]:
// the query takes R(dq - dk(j0)) (its D/2 factors formed by the warp's lanes for
// each unit) and the keys R(-e) from a 16-row table, in registers.  Corrected
// operands enter the products as bf16 hi + lo pairs (about 16 significant bits;
// one bf16 would put 2^-9 |q| |k| on a score), the query's lo part in the M rows
// 8-15 that at most 8 heads leave free.  Probabilities are carried as hi + lo
// pairs too, so that the output's error is its own rounding; for up to four
// heads the lo parts use the columns 4-7 of the P V product that would be idle.
#include "jl_mma.cuh"
#include "jl_paged.cuh"

namespace jl {

namespace {

constexpr int kWarps = 12;
constexpr int kThreads = 32 * kWarps;
constexpr int kMinUnits = 2 * kWarps;  // units per CTA below which fewer CTAs share a call's work

template <int D>
struct PgCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kHalf = 16 * D * 2;         // bytes of a unit's keys (or values)
  static constexpr int kSlot = 2 * kHalf;
  static constexpr int kSlots = D == 128 ? 2 : 4;  // ring depth of a warp
  static constexpr int kERow = (D / 2 + 8) * 8;    // bytes per row of the key factors (padded)
  static constexpr int kRing = kWarps * kSlots * kSlot;
  static constexpr int kEOff = kRing;
  static constexpr int kUOff = kEOff + 16 * kERow;           // [D/2] (u_hi, u_lo)
  static constexpr int kCsOff = kUOff + (D / 2) * 16;        // [warps][D/2] query factors
  static constexpr int kScanOff = kCsOff + kWarps * (D / 2) * 8;  // [threads + 1] running unit counts
  static constexpr int kBarOff = kScanOff + (kThreads + 1) * 8 + 8;
  static constexpr int kMiscOff = kBarOff + kWarps * kSlots * 8;
  static constexpr int kSmem = kMiscOff + 256 + 1024;
};

// Units of item it = b * Hkv + g.
__device__ __forceinline__ int item_units(const PagedDecodeArgs& a, int64_t it) {
  const int b = (int)(it / a.Hkv);
  const int L = a.seq_lens[b];
  if (!paged_length_ok(L, a.max_pages, a.page_size)) return 0;
  if (a.page_list == nullptr) return (L + 15) >> 4;
  const int n = a.page_counts[it];
  if (L == 0 || n < 0 || (int64_t)n > a.list_stride) return 0;
  return n * (a.page_size >> 4);
}

// Scratch partial: [r] maxima (log2 units), [r] sums, [r][D] outputs.
struct Partial {
  float* m;
  float* l;
  float* o;
};
__device__ __forceinline__ Partial partial_at(float* base, int64_t idx, int r, int D) {
  float* p = base + idx * decode_partial_floats(r, D);
  return {p, p + r, p + 2 * r};
}

// kPack: at most four query heads per KV head, duplicated in M rows 4-7 so that
// those rows' lanes carry the probabilities' lo parts.
template <int D, bool kPack>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedDecodeArgs a) {
  using C = PgCfg<D>;
  constexpr int H2 = D / 2;
  constexpr int KS = D / 16;   // k-steps of the score product
  constexpr int KS2 = D / 32;  // k-steps holding the first half of each pair
  constexpr int S = C::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = a.r;
  const int64_t items = (int64_t)a.B * a.Hkv;

  int64_t* scan = reinterpret_cast<int64_t*>(smem + C::kScanOff);
  volatile int* misc = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  volatile int* abort_flag = misc;               // [0]
  volatile int* ticket = misc + 1;               // [1], [2]
  volatile int* ent_item = misc + 4;             // [2 x warps] items of the partials, -1: none
  double2* utab = reinterpret_cast<double2*>(smem + C::kUOff);

  // ---- how much there is to do, and where this CTA's and this warp's share is
  const int64_t per_thread = (items + kThreads - 1) / kThreads;
  int64_t mine = 0;
  for (int64_t i = tid * per_thread; i < min(items, (tid + 1) * per_thread); ++i) mine += item_units(a, i);
  {
    int64_t v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    scan[tid + 1] = v;
    if (tid == 0) {
      scan[0] = 0;
      *abort_flag = 0;
    }
    if (tid < kWarps * S) mbar_init(smem_addr(smem + C::kBarOff) + 8 * tid, 1);
    if (tid == 0) fence_mbar_init();
    if (tid < 2 * kWarps) ent_item[tid] = -1;
    if (tid < H2) utab[tid] = make_double2(a.u_hi[tid], a.u_lo[tid]);
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += scan[32 * w + 32];
    __syncthreads();
    scan[tid + 1] = v + before;
    __syncthreads();
  }
  const int64_t U = scan[kThreads];

  // Sequences and lists with nothing in them, bad lengths and counts: spread over every CTA.
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    if (item_units(a, it) != 0) continue;
    const int b = (int)(it / a.Hkv);
    for (int i = tid; i < r * D; i += kThreads)
      a.o[((int64_t)b * a.Hq + (it - (int64_t)b * a.Hkv) * r) * D + i] = __float2bfloat16_rn(0.f);
    if (a.lse != nullptr && tid < r) a.lse[(int64_t)b * a.Hq + (it - (int64_t)b * a.Hkv) * r + tid] = -INFINITY;
    if (tid == 0 && a.dev_error) {
      bool bad = !paged_length_ok(a.seq_lens[b], a.max_pages, a.page_size);
      if (a.page_list != nullptr) bad = bad || a.page_counts[it] < 0 || a.page_counts[it] > a.list_stride;
      if (bad) atomicExch(a.dev_error, kDevBadLength);
    }
  }

  const int64_t want = (U + kMinUnits - 1) / kMinUnits;
  const int64_t N = want < gridDim.x ? want : gridDim.x;  // CTAs that share the line
  if (blockIdx.x >= N) return;
  const int64_t c0 = (int64_t)blockIdx.x * U / N, c1 = ((int64_t)blockIdx.x + 1) * U / N;
  const int64_t wb = c0 + warp * (c1 - c0) / kWarps, we = c0 + (warp + 1) * (c1 - c0) / kWarps;
  const int cnt = (int)(we - wb);

  // Key factors E[e][t] = R(-e) for e < 16, as (c_t, c_t+1, s_t, s_t+1) for even t.
  for (int idx = tid; idx < 16 * H2; idx += kThreads) {
    const int e = idx / H2, t = idx % H2;
    float sn, cs;
    sincos_turns(-e, utab[t].x, utab[t].y, &sn, &cs);
    float* dst = reinterpret_cast<float*>(smem + C::kEOff) + e * (C::kERow / 4);
    dst[(t >> 1) * 4 + (t & 1)] = cs;
    dst[(t >> 1) * 4 + 2 + (t & 1)] = sn;
  }

  // ---- the walk over units: lane l holds the description of unit 32 * batch + l
  int64_t cur_it = 0, cur_s = 0;  // an item at or before the batch's first unit, and its first unit
  if (cnt > 0) {
    // the thread segment of items that holds unit wb, found by all lanes together
    int seg = 0;
    for (int t0 = 0; t0 < kThreads; t0 += 32) {
      const unsigned below = __ballot_sync(0xffffffffu, scan[t0 + lane] <= wb);
      if (below == 0u) break;
      seg = t0 + 31 - __clz(below);
      if (below != 0xffffffffu) break;
    }
    cur_it = seg * per_thread;
    cur_s = scan[seg];
  }
  int m_item = 0, m_phys = -1, m_row = 0, m_j0 = 0, m_c = 0;
  auto load_batch = [&](int k0) {
    const int64_t x = wb + k0 + lane;
    const bool valid = k0 + lane < cnt;
    int64_t my_it = -1, my_s = 0;
    bool open = valid;
    while (__any_sync(0xffffffffu, open)) {
      const int64_t i = cur_it + lane;
      int n = i < items ? item_units(a, i) : 0;
      int64_t p = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, p, o);
        if (lane >= o) p += t;
      }
      const int64_t rel = x - cur_s;
      int j = 0;  // the first of the 32 items whose running count passes rel
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const int64_t t = __shfl_sync(0xffffffffu, p, j + o - 1);
        if (t <= rel) j += o;
      }
      const int64_t pj = __shfl_sync(0xffffffffu, p, j & 31);
      const int nj = __shfl_sync(0xffffffffu, n, j & 31);
      if (open && pj > rel) {
        open = false;
        my_it = cur_it + j;
        my_s = cur_s + pj - nj;
      }
      const int64_t tot = __shfl_sync(0xffffffffu, p, 31);
      if (__any_sync(0xffffffffu, open)) {
        cur_it += 32;
        cur_s += tot;
        if (cur_it >= items) break;  // cannot happen while lengths stay as they were scanned
      }
    }
    m_phys = -1;
    m_j0 = -1;
    m_row = 0;
    m_c = 0;
    m_item = (int)my_it;
    if (valid && my_it >= 0) {
      const int b = (int)(my_it / a.Hkv);
      const int c = (int)(x - my_s);
      const int64_t key = (int64_t)c * 16;
      const int64_t e = key / a.page_size;
      m_row = (int)(key - e * a.page_size);
      m_c = c;
      int64_t lp = e;
      if (a.page_list != nullptr) lp = a.page_list[my_it * a.list_stride + e];
      if (lp >= 0 && lp < a.max_pages) {
        const int64_t j0 = lp * a.page_size + m_row;
        if (j0 < a.seq_lens[b]) {
          const int phys = a.block_table[(int64_t)b * a.max_pages + lp];
          if (phys >= 0 && phys < a.num_pages) {
            m_phys = phys;
            m_j0 = (int)j0;
          } else if (a.dev_error) {
            atomicExch(a.dev_error, kDevBadLength);
          }
        }
      } else if (a.dev_error) {
        atomicExch(a.dev_error, kDevBadLength);
      }
    }
  };
  const uint32_t bar0 = smem_addr(smem + C::kBarOff) + 8 * (warp * S);
  const uint32_t ring = sbase + warp * (S * C::kSlot);
  int sl_item[S], sl_j0[S], sl_c[S];
#pragma unroll
  for (int s = 0; s < S; ++s) sl_item[s] = sl_j0[s] = -1, sl_c[s] = 0;
  auto issue = [&](int k, int s) {  // unit k into slot s
    if ((k & 31) == 0) load_batch(k);
    const int item = __shfl_sync(0xffffffffu, m_item, k & 31);
    const int phys = __shfl_sync(0xffffffffu, m_phys, k & 31);
    const int row = __shfl_sync(0xffffffffu, m_row, k & 31);
    sl_item[s] = item;
    sl_j0[s] = __shfl_sync(0xffffffffu, m_j0, k & 31);
    sl_c[s] = __shfl_sync(0xffffffffu, m_c, k & 31);
    if (lane == 0) {
      if (phys >= 0) {
        const int g = item % a.Hkv;
        mbar_arrive_expect_tx(bar0 + 8 * s, (uint32_t)C::kSlot);
        const uint32_t st = ring + s * C::kSlot;
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) {
          tma_load_4d(st + c * 2048, &tm_k, bar0 + 8 * s, c * 64, g, row, phys);
          tma_load_4d(st + C::kHalf + c * 2048, &tm_v, bar0 + 8 * s, c * 64, g, row, phys);
        }
      } else {
        mbar_arrive(bar0 + 8 * s);  // nothing to fetch; the phase completes all the same
      }
    }
  };
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < cnt) issue(s, s);
  __syncthreads();  // key factors are ready

  // ---- per-item state
  const int c4 = lane & 3;       // column group of the mma fragments
  const int hrow = lane >> 2;    // M row of this lane
  const int hq = kPack ? (hrow & 3) : hrow;  // query head of that row
  uint32_t qf[KS][2];            // base query fragments: dims 16 ks + 2 c4 (+ 8) of head hq
  float oacc[D / 16][4];
  float m_used = -INFINITY, l_part = 0.f;
  int item = -1, seg_c = 0, seg_k = 0;  // current item, its unit index at the segment's first unit k
  int L = 0, local_from = 0, G = 1;
  bool all_local = true;
  int64_t dq = 0;
  uint32_t g_magic = 0;
  const float sl2 = a.scale_log2;
#pragma unroll
  for (int n = 0; n < D / 16; ++n) oacc[n][0] = oacc[n][1] = oacc[n][2] = oacc[n][3] = 0.f;

  // Writes the warp's accumulated segment as a partial (m, l, o): heads at rows of `p`.
  auto store_partial = [&](const Partial& p) {
    float l = l_part;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (c4 == 0 && hrow < r) {
      p.m[hrow] = m_used;
      p.l[hrow] = l;
    }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v = oacc[mt][k];
        if (kPack) v += __shfl_down_sync(0xffffffffu, v, 2);  // + the lo parts' product, four columns on
        const int h = 2 * c4 + (k & 1);
        const int d = 16 * mt + hrow + ((k & 2) ? 8 : 0);
        if (h < r) p.o[h * D + d] = v;
      }
  };
  // The whole item was this warp's: normalise and write the results.
  auto store_final = [&](int it) {
    float l = l_part;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int b = it / a.Hkv, g = it - b * a.Hkv;
    const int64_t row = (int64_t)b * a.Hq + g * r;
    if (c4 == 0 && hrow < r && a.lse != nullptr)
      a.lse[row + hrow] = l == 0.f ? -INFINITY : (m_used + __log2f(l)) * 0.69314718055994531f;
    const float i0 = __shfl_sync(0xffffffffu, inv, 8 * c4), i1 = __shfl_sync(0xffffffffu, inv, 8 * c4 + 4);
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v = oacc[mt][k];
        if (kPack) v += __shfl_down_sync(0xffffffffu, v, 2);
        const int h = 2 * c4 + (k & 1);
        const int d = 16 * mt + hrow + ((k & 2) ? 8 : 0);
        if (h < r) a.o[(row + h) * D + d] = __float2bfloat16_rn(v * ((k & 1) ? i1 : i0));
      }
  };

  bool ok = true;
  int k_fail = 0;
  int tail_item = -1, head_item = -1;
  for (int k0 = 0; k0 < cnt && ok; k0 += S) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int k = k0 + s;
      if (k >= cnt || !ok) break;
      if (sl_item[s] != item) {
        if (item >= 0) {  // the previous item ends here, inside the warp's range
          if (wb + seg_k - seg_c >= wb) {
            store_final(item);
          } else {
            store_partial(partial_at(a.warp_parts, (int64_t)blockIdx.x * kWarps + warp, r, D));
            head_item = item;
          }
        }
        item = sl_item[s];
        seg_c = sl_c[s];
        seg_k = k;
        m_used = -INFINITY;
        l_part = 0.f;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) oacc[n][0] = oacc[n][1] = oacc[n][2] = oacc[n][3] = 0.f;
        const int b = item / a.Hkv, g = item - b * a.Hkv;
        L = a.seq_lens[b];
        G = (int)group_size(L, a.w_pretrained);
        all_local = jl::all_local(L, a.w0, G);
        dq = query_remote(L - 1, G, query_shift(a.w0, G, a.qshift)) - (L - 1);
        g_magic = G < 16 ? (uint32_t)((((uint64_t)1 << 32) + (uint64_t)G - 1) / (uint64_t)G) : 0u;
        local_from = all_local ? 0 : L - a.w0;  // keys j >= local_from are scored with base RoPE
        const __nv_bfloat16* qp = a.q + ((int64_t)b * a.Hq + g * r + hq) * D + 2 * c4;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[ks][0] = hq < r ? *reinterpret_cast<const uint32_t*>(qp + 16 * ks) : 0u;
          qf[ks][1] = hq < r ? *reinterpret_cast<const uint32_t*>(qp + 16 * ks + 8) : 0u;
        }
      }
      const int j0 = sl_j0[s];
      const bool t_local = all_local || j0 >= local_from;
      const bool t_remote = !all_local && (j0 + 15 < local_from);
      float* csb = reinterpret_cast<float*>(smem + C::kCsOff) + warp * D;
      int rm = 0;
      if (j0 >= 0 && !t_local) {
        const int qd = j0 / G;
        rm = j0 - qd * G;
        const int64_t turn = dq - ((int64_t)qd - j0);
#pragma unroll
        for (int e = 0; e < H2 / 32; ++e) {
          const int t = lane + 32 * e;
          float sn, cs;
          sincos_turns(turn, utab[t].x, utab[t].y, &sn, &cs);
          csb[(t >> 1) * 4 + (t & 1)] = cs;
          csb[(t >> 1) * 4 + 2 + (t & 1)] = sn;
        }
        __syncwarp();
      }

      ok = mbar_wait(bar0 + 8 * s, (uint32_t)(k0 / S) & 1u, abort_flag, a.dev_error);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        k_fail = k;
        break;
      }

      if (j0 >= 0) {
        const uint32_t kst = ring + s * C::kSlot;
        const uint32_t vst = kst + C::kHalf;
        float sloc[2][4], sah[2][4], sal[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sloc[nt][e] = sah[nt][e] = sal[nt][e] = 0.f;

        // factor rows of this lane's two keys (one per 8-key n-tile):
        // e(u) = u - (floor((j0 + u) / G) - floor(j0 / G))
        const float4* Er[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int u = 8 * nt + (lane >> 2);
          const int q = G >= 16 ? (rm + u >= G ? 1 : 0) : (int)__umulhi((unsigned)(rm + u), g_magic);
          Er[nt] = reinterpret_cast<const float4*>(smem + C::kEOff + (u - (G == 1 ? u : q)) * C::kERow);
        }
        const float4* Qf = reinterpret_cast<const float4*>(csb);

#pragma unroll
        for (int kp = 0; kp < KS2; ++kp) {
          uint32_t klo[4], khi[4];
          {
            const int mi = lane >> 3;
            const int kr = (mi >> 1) * 8 + (lane & 7);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int ks = kp + hf * KS2;
              const int u = 2 * (ks & 3) + (mi & 1);
              const uint32_t addr = kst + (ks >> 2) * 2048 + kr * 128 + ((u ^ (kr & 7)) << 4);
              if (hf == 0)
                ldsm_x4(addr, klo[0], klo[1], klo[2], klo[3]);
              else
                ldsm_x4(addr, khi[0], khi[1], khi[2], khi[3]);
            }
          }
          if (!t_remote) {  // local or straddling: base query, keys as stored
            const uint32_t alo[4] = {qf[kp][0], 0u, qf[kp][1], 0u};
            const uint32_t ahi[4] = {qf[kp + KS2][0], 0u, qf[kp + KS2][1], 0u};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              mma_bf16(sloc[nt], alo, klo[2 * nt], klo[2 * nt + 1]);
              mma_bf16(sloc[nt], ahi, khi[2 * nt], khi[2 * nt + 1]);
            }
          }
          if (!t_local) {  // remote or straddling: corrected query and keys
            uint32_t kah[4], kal[4], kbh[4], kbl[4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const float4 f01 = Er[nt][(16 * kp + 2 * c4) >> 1];
              const float4 f23 = Er[nt][(16 * kp + 8 + 2 * c4) >> 1];
              rot_split_bf16(klo[2 * nt], khi[2 * nt], f01, kah[2 * nt], kal[2 * nt], kbh[2 * nt], kbl[2 * nt]);
              rot_split_bf16(klo[2 * nt + 1], khi[2 * nt + 1], f23, kah[2 * nt + 1], kal[2 * nt + 1],
                             kbh[2 * nt + 1], kbl[2 * nt + 1]);
            }
            uint32_t alo[4], ahi[4];
            rot_split_bf16(qf[kp][0], qf[kp + KS2][0], Qf[(16 * kp + 2 * c4) >> 1], alo[0], alo[1], ahi[0], ahi[1]);
            rot_split_bf16(qf[kp][1], qf[kp + KS2][1], Qf[(16 * kp + 8 + 2 * c4) >> 1], alo[2], alo[3], ahi[2],
                           ahi[3]);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              mma_bf16(sah[nt], alo, kah[2 * nt], kah[2 * nt + 1]);
              mma_bf16(sal[nt], alo, kal[2 * nt], kal[2 * nt + 1]);
              mma_bf16(sah[nt], ahi, kbh[2 * nt], kbh[2 * nt + 1]);
              mma_bf16(sal[nt], ahi, kbl[2 * nt], kbl[2 * nt + 1]);
            }
          }
        }

        // scores in log2 units, the band's choice and the mask behind the sequence
        float x[2][2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = j0 + 8 * nt + 2 * c4 + e;
            const bool loc = all_local || j >= local_from;
            const float rem = (sah[nt][e] + sah[nt][e + 2]) + (sal[nt][e] + sal[nt][e + 2]);
            float v = (loc ? sloc[nt][e] : rem) * sl2;
            if (j >= L) v = -INFINITY;
            x[nt][e] = v;
          }
        float mt = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
        float alpha = 1.f;
        bool resc = false;
        if (mt > m_used + 8.f) {  // a running maximum up to 2^8 behind keeps every p below 2^8
          alpha = (m_used == -INFINITY) ? 0.f : ex2_approx(m_used - mt);
          resc = m_used != -INFINITY;
          l_part *= alpha;
          m_used = mt;
        }
        if (__any_sync(0xffffffffu, resc)) {
          // this lane's O^T columns are heads 2 c4 and 2 c4 + 1
          const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * c4);
          const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * c4 + 4);
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            oacc[n][0] *= a0;
            oacc[n][1] *= a1;
            oacc[n][2] *= a0;
            oacc[n][3] *= a1;
          }
        }
        const float msub = (m_used == -INFINITY) ? 0.f : m_used;
        uint32_t ph[2], pl[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float p0 = ex2_approx(x[nt][0] - msub), p1 = ex2_approx(x[nt][1] - msub);
          l_part += p0 + p1;
          split_f2_bf16(f2_pack(p0, p1), ph[nt], pl[nt]);
        }
        const uint32_t pb0 = kPack && hrow >= 4 ? pl[0] : ph[0];
        const uint32_t pb1 = kPack && hrow >= 4 ? pl[1] : ph[1];
        const bool tail = j0 + 16 > L;  // rows behind the sequence hold anything, NaN included
        uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;
        if (tail) {
          const int u = L - j0 - 2 * c4;  // of the keys 2 c4 + {0, 1} and 8 + 2 c4 + {0, 1}
          vm0 = (u > 0 ? 0xffffu : 0u) | (u > 1 ? 0xffff0000u : 0u);
          vm1 = (u > 8 ? 0xffffu : 0u) | (u > 9 ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int mt2 = 0; mt2 < D / 16; ++mt2) {
          const int mi = lane >> 3;
          const int kr = (mi >> 1) * 8 + (lane & 7);
          const int u = 2 * (mt2 & 3) + (mi & 1);
          const uint32_t addr = vst + (mt2 >> 2) * 2048 + kr * 128 + ((u ^ (kr & 7)) << 4);
          uint32_t va[4];
          ldsm_x4_t(addr, va[0], va[1], va[2], va[3]);
          if (tail) {
            va[0] &= vm0;
            va[1] &= vm0;
            va[2] &= vm1;
            va[3] &= vm1;
          }
          mma_bf16(oacc[mt2], va, pb0, pb1);
          if (!kPack) mma_bf16(oacc[mt2], va, pl[0], pl[1]);
        }
      }
      __syncwarp();  // every lane has read the slot (and the query factors)
      if (k + S < cnt) issue(k + S, s);
    }
  }
  if (!ok) {
    // Gave up at unit k_fail: let the copies in flight land (again with a limit)
    // before the ring is reused or the CTA ends.
    const uint64_t t0 = global_timer_ns();
    for (int k = k_fail; k < min(cnt, k_fail + S); ++k)
      while (!mbar_try_wait(bar0 + 8 * (k % S), (uint32_t)(k / S) & 1u))
        if (global_timer_ns() - t0 > 100000000ull) break;
  }

  // ---- the segment in hand: an item that ended with the range, or runs on
  Partial tails;
  __syncthreads();  // every warp is done with its ring; it holds the partials from here
  {
    tails = partial_at(reinterpret_cast<float*>(smem), warp, r, D);
    if (item >= 0) {
      const bool began = wb + seg_k - seg_c >= wb;
      const bool ends = wb + seg_k - seg_c + item_units(a, item) <= we;
      if (began && ends) {
        store_final(item);
      } else {
        store_partial(tails);
        tail_item = item;
      }
    }
    if (lane == 0) {
      ent_item[2 * warp] = head_item;
      ent_item[2 * warp + 1] = tail_item;
    }
  }
  __syncthreads();

  // ---- join the warps' partials item by item; entries 2 w (head) and 2 w + 1 (tail) are in unit order
  auto entry = [&](int e) -> Partial {
    return (e & 1) ? partial_at(reinterpret_cast<float*>(smem), e >> 1, r, D)
                   : partial_at(a.warp_parts, (int64_t)blockIdx.x * kWarps + (e >> 1), r, D);
  };
  int shared_item[2] = {-1, -1};  // items shared with the CTAs before and behind
  for (int e0 = 0; e0 < 2 * kWarps;) {
    const int it = ent_item[e0];
    if (it < 0) {
      ++e0;
      continue;
    }
    int e1 = e0 + 1;
    while (e1 < 2 * kWarps && (ent_item[e1] < 0 || ent_item[e1] == it)) ++e1;
    // the item's place on the line
    int64_t s = 0;
    {
      const int64_t seg = it / per_thread;
      s = scan[seg];
      for (int64_t i = seg * per_thread; i < it; ++i) s += item_units(a, i);
    }
    const int64_t n = item_units(a, it);
    const bool whole = s >= c0 && s + n <= c1;
    const int slot = s < c0 ? 0 : 1;
    if (!whole) shared_item[slot] = it;
    const Partial out = partial_at(a.cta_parts, (int64_t)blockIdx.x * 2 + slot, r, D);
    const int b = it / a.Hkv, g = it - b * a.Hkv;
    const int64_t row = (int64_t)b * a.Hq + g * r;
    for (int idx = tid; idx < r * D; idx += kThreads) {
      const int h = idx / D;
      float M = -INFINITY;
      for (int e = e0; e < e1; ++e)
        if (ent_item[e] >= 0) M = fmaxf(M, entry(e).m[h]);
      float o = 0.f, l = 0.f;
      for (int e = e0; e < e1; ++e) {
        if (ent_item[e] < 0) continue;
        const Partial p = entry(e);
        // an empty part's sum is 0; a NaN that left the maximum at -inf goes through
        const float wt = p.m[h] == -INFINITY ? p.l[h] : ex2_approx(p.m[h] - M);
        o += wt * p.o[idx];
        l += wt * p.l[h];
      }
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        a.o[row * D + idx] = __float2bfloat16_rn(o * inv);
        if (idx == h * D && a.lse != nullptr)
          a.lse[row + h] = l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.69314718055994531f;
      } else {
        out.o[idx] = o;
        if (idx == h * D) {
          out.m[h] = M;
          out.l[h] = l;
        }
      }
    }
    e0 = e1;
  }

  // ---- join the CTAs' partials: the item's last ticket does it
  auto cta_of = [&](int64_t unit) -> int64_t { return ((unit + 1) * N - 1) / U; };
#pragma unroll 1
  for (int slot = 0; slot < 2; ++slot) {
    const int it = shared_item[slot];
    if (it < 0) continue;  // the same for every thread of the CTA
    int64_t s = 0;
    {
      const int64_t seg = it / per_thread;
      s = scan[seg];
      for (int64_t i = seg * per_thread; i < it; ++i) s += item_units(a, i);
    }
    const int64_t first = cta_of(s), last = cta_of(s + item_units(a, it) - 1);
    __threadfence();
    __syncthreads();
    if (tid == 0) *ticket = atomicInc(&a.counters[first], (unsigned)(last - first)) == (unsigned)(last - first);
    __syncthreads();
    if (*ticket == 0) continue;
    __threadfence();
    const int b = it / a.Hkv, g = it - b * a.Hkv;
    const int64_t row = (int64_t)b * a.Hq + g * r;
    for (int idx = tid; idx < r * D; idx += kThreads) {
      const int h = idx / D;
      // the item begins inside the first CTA's range (slot 1) and before the others' (slot 0)
      auto part = [&](int64_t c) { return partial_at(a.cta_parts, c * 2 + (c == first ? 1 : 0), r, D); };
      float M = -INFINITY;
      for (int64_t c = first; c <= last; ++c) M = fmaxf(M, __ldcg(part(c).m + h));
      float o = 0.f, l = 0.f;
      for (int64_t c = first; c <= last; ++c) {
        const Partial p = part(c);
        const float mc = __ldcg(p.m + h);
        const float lc = __ldcg(p.l + h);
        const float wt = mc == -INFINITY ? lc : ex2_approx(mc - M);
        o += wt * __ldcg(p.o + idx);
        l += wt * lc;
      }
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      a.o[row * D + idx] = __float2bfloat16_rn(o * inv);
      if (idx == h * D && a.lse != nullptr)
        a.lse[row + h] = l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.69314718055994531f;
    }
  }
}

template <int D, bool kPack>
cudaError_t launch_dp(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const PagedDecodeArgs& a, int ctas,
                      cudaStream_t stream) {
  auto k = paged_decode_kernel<D, kPack>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, PgCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  k<<<ctas, kThreads, PgCfg<D>::kSmem, stream>>>(tm_k, tm_v, a);
  return cudaGetLastError();
}

}  // namespace

int decode_paged_max_ctas() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}
int decode_paged_warps() { return kWarps; }

cudaError_t launch_decode_paged(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const PagedDecodeArgs& a, int D,
                                cudaStream_t stream) {
  const int ctas = decode_paged_max_ctas();  // one per SM
  if (D == 128)
    return a.r <= 4 ? launch_dp<128, true>(tm_k, tm_v, a, ctas, stream)
                    : launch_dp<128, false>(tm_k, tm_v, a, ctas, stream);
  return a.r <= 4 ? launch_dp<64, true>(tm_k, tm_v, a, ctas, stream)
                  : launch_dp<64, false>(tm_k, tm_v, a, ctas, stream);
}

}  // namespace jl
