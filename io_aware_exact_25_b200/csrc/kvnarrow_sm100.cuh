// kvnarrow_sm100.cuh -- attention of few rows over the quantised cache.
//
// An item has at most M = 16 MT rows (query tokens x heads of one key head's
// group), so every key and value byte is used for few products and the cache's
// bytes are what the kernel waits for: the aim is to keep them streaming.
//
// Each warp is its own pipeline.  A unit of 128 keys is four slices of 32, one
// per warp: lane 0 of the warp brings the slice's K and V codes (TMA, swizzled
// by the row width so that every read below is free of bank conflicts) and
// scales (bulk copies) into the warp's ring of kStages slices; the warp alone
// consumes and refills it, so the warps of a CTA never wait for one another
// until an item ends, when their (m, l, O) are merged through shared memory.
//
// The products run on mma.sync m16n8k16 in f16, which a 16-row tile fits
// (tcgen05's smallest tile has 64 rows, and at 16 rows the tensor pipe is a
// fifth busy).  Codes become f16 in registers without rounding: an int8 code c
// is the byte c + 128 placed under the exponent of 1024, minus 1152; an e4m3
// code's bits shifted under an f16 sign are its value times 2^-8, subnormals
// included.  No code, not even a NaN pattern in a slot never written, turns
// into an infinity or a NaN.  The K fragment of a lane is 16 consecutive bytes
// of a key row, so the reduction runs over d in a permuted order; Q's
// fragments are loaded in the same order.  V's fragments come from
// ldmatrix.trans on byte pairs; its two columns per pair go to two n-tiles.
//
// Scales: q is held in f16 as q * 2^-e with e from the row's largest |q| (an
// exact shift of the exponent; entries 2^-14 below the largest lose bits that
// stay below 2^-25 of it).  K's scale multiplies the fp32 score.  V's scale
// multiplies p before it is rounded to f16, as a ratio to a running power of
// two above every V scale seen, so that p * ratio <= 2^15 with 11 significant
// bits down to 2^-14; the row sum takes the unrounded fp32 p.
#pragma once

#include "kvcache_sm100.cuh"

namespace fa {

// Two-dimensional tiled load (x innermost).
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, int x, int y, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
      "l"(m), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ float ld_shared_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// mbar_wait by a whole warp, with one answer for all lanes: the warp-wide instructions that follow need every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, const Abort& ab) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The four codes of a word as two f16 pairs: (byte 0, byte 2) and (byte 1, byte 3).  int8: the codes; fp8: the codes' values
// times 2^-8 (kKvCodeScale takes the factor back).
template <int FMT>
__device__ __forceinline__ void kv_unpack(uint32_t w, uint32_t& even, uint32_t& odd) {
  if constexpr (FMT == kKvInt8) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t e = __byte_perm(u, 0x64646464u, 0x4240), o = __byte_perm(u, 0x64646464u, 0x4341);
    const uint32_t bias = 0x64806480u;  // 1152 = 1024 + 128
    const __half2 he = __hsub2(*reinterpret_cast<const __half2*>(&e), *reinterpret_cast<const __half2*>(&bias));
    const __half2 ho = __hsub2(*reinterpret_cast<const __half2*>(&o), *reinterpret_cast<const __half2*>(&bias));
    even = *reinterpret_cast<const uint32_t*>(&he);
    odd = *reinterpret_cast<const uint32_t*>(&ho);
  } else {
    even = ((w << 8) & 0x80008000u) | ((w << 7) & 0x3f803f80u);
    odd = (w & 0x80008000u) | ((w >> 1) & 0x3f803f80u);
  }
}

template <int FMT>
__host__ __device__ constexpr float kv_code_scale() { return FMT == kKvInt8 ? 1.f : 256.f; }

// Which power of two scales a row of q into f16: the factor 2^-e and its inverse, from the row's largest |q|.
__device__ __forceinline__ void kv_q_shift(float amax, float& down, float& up) {
  const uint32_t e = min(max(__float_as_uint(amax) >> 23, 1u), 253u);
  down = __uint_as_float((254u - e) << 23);
  up = __uint_as_float(e << 23);
}

template <int D, int MT, int STAGES, int CTAS>
struct KvNarrowLayout {
  static constexpr int kM = 16 * MT;
  static constexpr int kStages = STAGES, kCtasPerSm = CTAS;
  static constexpr uint32_t kCodes = 32u * D;                     // one slice of K (or V) codes
  static constexpr uint32_t kStageBytes = 2 * kCodes + 256u;      // then 32 K scales, 32 V scales
  static constexpr uint32_t kRingCodes = kStages * 2 * kCodes;    // codes first: they keep 1024-byte alignment
  static constexpr uint32_t kRing = kRingCodes + kStages * 256u;  // one warp's ring
  static constexpr uint32_t kRingPad = (kRing + 1023u) & ~1023u;
  static constexpr uint32_t kRowPad = D + 4;                      // floats of a merged row (bank spread)
  static_assert(kM * kRowPad * 4 <= kRingPad, "a warp's result fits in its ring");
  static constexpr uint32_t kOffMl = 4 * kRingPad;                // [4][kM] m, [4][kM] l, [4] V scale
  static constexpr uint32_t kOffBar = kOffMl + (8 * kM + 4) * 4;
  static constexpr uint32_t kOffScan = kOffBar + 4 * kStages * 8 + 16;
  static constexpr uint32_t kSmem = kOffScan + (uint32_t)sizeof(KvScan);
  static_assert(kOffBar % 8 == 0, "barrier alignment");
  static_assert(kCtasPerSm * (kSmem + 1024) <= 233472, "shared memory budget");
};

// P values carry a factor 2^7 against the running maximum m, which is raised only when a score exceeds it by 8.
constexpr float kKvPShift = 7.f;

template <int D, int FMT, int MT, class L>
__global__ void __launch_bounds__(128, L::kCtasPerSm)
    kv_narrow_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const KvArgs a) {
  constexpr int M = L::kM, S = L::kStages;
  constexpr int NH = D / 64;   // 64-byte halves of a key row
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, c4 = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar) + warp * S;
  int* abort_flag = reinterpret_cast<int*>(smem + L::kOffBar + 4 * S * 8);
  uint8_t* ring = smem + warp * L::kRingPad;
  const uint32_t sring = smem_u32(ring);
  const uint32_t sscale = sring + L::kRingCodes;
  float* s_m = reinterpret_cast<float*>(smem + L::kOffMl);
  float* s_l = s_m + 4 * M;
  float* s_v = s_l + 4 * M;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4 * S; ++i) mbar_init(reinterpret_cast<uint64_t*>(smem + L::kOffBar) + i, 1);
    const bool misaligned = (smem_u32(smem) & 1023u) != 0u;
    *abort_flag = misaligned ? 1 : 0;
    if (misaligned && a.err) atomicCAS(a.err, kDevOk, kDevMisaligned);
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  pdl_trigger();
  int b;
  long long rem;
  const KvLine line =
      kv_place<128>(a, blockIdx.x, gridDim.x, reinterpret_cast<KvScan*>(smem + L::kOffScan), &b, &rem);
  __syncthreads();
  if (a.phase == kKvWhole && threadIdx.x == 0) a.cuts[blockIdx.x].n = 0;  // until this CTA leaves an item unfinished
  if (b < 0 || *abort_flag) {
    if (a.phase == kKvSuffix) pdl_wait();
    return;
  }
  const Abort ab{abort_flag, a.err};
  const uint64_t pol = policy_evict_first();
  const long long u0 = line.cut(blockIdx.x), u1 = line.cut(blockIdx.x + 1);
  KvSeq s = kv_seq(a, b, false);
  KvPlace at = kv_within(a, s, b, rem);
  const int begin = kv_begin(a);
  uint32_t issued = 0, used = 0;  // slices this warp has asked for and consumed, over all items
  bool ok = true;

  for (long long u = u0; u < u1 && ok;) {
    const int n_item = kv_item_units(a, s, at.rt);
    const int n = (int)min((long long)(n_item - at.unit), u1 - u);
    const int item_end = kv_item_end(a, s, at.rt);
    // this warp's slices: 32 keys at first + 128 j, j < steps
    const int first = begin + at.unit * kKvUnit + warp * 32;
    int steps = n;
    if (first + (n - 1) * kKvUnit >= item_end) --steps;  // the last unit may end before this warp's slice
    steps = max(steps, 0);

    // ---- the slices' pages, 32 at a time: lane j holds those of step 32 i + j
    const int* trow = a.table + (a.phase == kKvPrefix ? 0ll : at.b * a.table_stride);
    const bool two = a.page_shift == 4;  // a slice covers two 16-slot pages
    int pg0 = 0, pg1 = 0;
    auto fetch_pages = [&](int j0) {
      const int key = first + (j0 + lane) * kKvUnit;
      pg0 = pg1 = 0;
      if (j0 + lane < steps) {
        pg0 = __ldg(trow + (key >> a.page_shift));
        if (two && key + 16 < item_end) pg1 = __ldg(trow + (key >> 4) + 1);
        if (pg0 < 0 || pg0 >= a.num_pages || pg1 < 0 || pg1 >= a.num_pages) {
          if (a.err) atomicCAS(a.err, kDevOk, kDevBadPage);
          if (pg0 < 0 || pg0 >= a.num_pages) pg0 = 0;
          if (pg1 < 0 || pg1 >= a.num_pages) pg1 = 0;
        }
      }
    };
    int asked = 0;
    auto issue = [&]() {
      const int j = asked++;
      if ((j & 31) == 0) fetch_pages(j);
      const int p0 = __shfl_sync(0xffffffffu, pg0, j & 31), p1 = __shfl_sync(0xffffffffu, pg1, j & 31);
      if (lane == 0) {
        const int key = first + j * kKvUnit;
        const int st = issued % S;
        uint64_t* bar = bars + st;
        const long long r0 = (((long long)p0 * a.Hkv + at.h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
        uint8_t* dk = ring + st * 2 * L::kCodes;
        uint8_t* dsc = ring + L::kRingCodes + st * 256;
        (void)FA_IN(kSiteKvRow, r0, two ? 16 : 32, ((long long)a.num_pages * a.Hkv) << a.page_shift, a.err);
        if (!two) {
          mbar_arrive_expect_tx(bar, 2 * L::kCodes + 256u);
          tma_load_2d(dk, &tm_k, 0, (int)r0, bar, pol);
          tma_load_2d(dk + L::kCodes, &tm_v, 0, (int)r0, bar, pol);
          bulk_load(dsc, a.ks + r0, 128, bar);
          bulk_load(dsc + 128, a.vs + r0, 128, bar);
        } else {
          // the second page only if the sequence reaches into it: its table entry may not exist
          const bool more = key + 16 < item_end;
          mbar_arrive_expect_tx(bar, more ? 2 * L::kCodes + 256u : L::kCodes + 128u);
          tma_load_2d(dk, &tm_k, 0, (int)r0, bar, pol);
          tma_load_2d(dk + L::kCodes, &tm_v, 0, (int)r0, bar, pol);
          bulk_load(dsc, a.ks + r0, 64, bar);
          bulk_load(dsc + 128, a.vs + r0, 64, bar);
          if (more) {
            const long long r1 = ((long long)p1 * a.Hkv + at.h) << 4;
            (void)FA_IN(kSiteKvRow, r1, 16, ((long long)a.num_pages * a.Hkv) << a.page_shift, a.err);
            tma_load_2d(dk + L::kCodes / 2, &tm_k, 0, (int)r1, bar, pol);
            tma_load_2d(dk + L::kCodes + L::kCodes / 2, &tm_v, 0, (int)r1, bar, pol);
            bulk_load(dsc + 64, a.ks + r1, 64, bar);
            bulk_load(dsc + 192, a.vs + r1, 64, bar);
          }
        }
      }
      ++issued;
    };
    for (int j = 0; j < S && j < steps; ++j) issue();

    // ---- Q fragments, in the order the K bytes come: word w of a lane's 16
    // bytes in half hh covers d = 64 hh + 16 c4 + 4 w + {0, 2} and {1, 3}
    uint32_t qa[MT][NH * 4][4];
    float qs[MT][2];   // score factor of rows g8, g8 + 8 of each 16-row tile
    int end[MT][2];    // keys those rows see
    int end_min = item_end;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint2 raw[2][NH * 4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const KvRow x = kv_row_of(a, s, at.h, at.rt, mt * 16 + half * 8 + g8);
        end[mt][half] = x.end;
        if (x.token >= 0) end_min = min(end_min, x.end);
        const long long qo = x.token * a.q_sn + x.head * a.q_sh;
        const bool in = x.token >= 0 && FA_IN(kSiteKvQ, qo, D, extent4(1, a.Hq, a.total, D, 0, a.q_sh, a.q_sn), a.err);
        uint32_t m2 = 0u;
#pragma unroll
        for (int w = 0; w < NH * 4; ++w) {
          raw[half][w] = make_uint2(0u, 0u);
          if (in)
            raw[half][w] = __ldg(reinterpret_cast<const uint2*>(a.q + qo + 64 * (w >> 2) + 16 * c4 + 4 * (w & 3)));
          m2 = __vmaxu2(m2, __vmaxu2(raw[half][w].x & 0x7fff7fffu, raw[half][w].y & 0x7fff7fffu));
        }
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
        float down, up;
        kv_q_shift(__uint_as_float(max(m2 & 0xffffu, m2 >> 16) << 16), down, up);
        qs[mt][half] = up * a.scale_log2 * kv_code_scale<FMT>();
#pragma unroll
        for (int w = 0; w < NH * 4; ++w) {
          qa[mt][w][half] = pack_f16x2(bf16_lo(raw[half][w].x) * down, bf16_lo(raw[half][w].y) * down);
          qa[mt][w][2 + half] = pack_f16x2(bf16_hi(raw[half][w].x) * down, bf16_hi(raw[half][w].y) * down);
        }
      }
    }
    // the smallest reach of any row: slices below it need no mask
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) end_min = min(end_min, __shfl_xor_sync(0xffffffffu, end_min, d));

    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];
    float vscale = 1.1754943508222875e-38f;  // running power of two above every V scale, at least 2^-126
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int t = 0; t < D / 8; ++t) o[mt][t][0] = o[mt][t][1] = o[mt][t][2] = o[mt][t][3] = 0.f;
    }

    // Key order inside an n-tile of 8: column j of the product is key kperm(j).
    // At d = 128 the lanes that read together (columns 2 i, 2 i + 1) take rows
    // that differ by 4, whose swizzles use different halves of the 128-byte
    // line; at d = 64 two consecutive rows share a line and differ already.
    auto kperm = [](int j) { return D == 128 ? (j >> 1) | ((j & 1) << 2) : j; };
    auto chunk_at = [](int row, int ch) {  // byte offset of 16-byte chunk ch of a row under the row width's swizzle
      return D == 128 ? row * 128 + ((ch ^ (row & 7)) << 4) : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
    };

    for (int j = 0; j < steps; ++j) {
      const int st = used % S;
      if (!mbar_wait_warp(bars + st, (used / S) & 1u, ab)) {
        ok = false;
        break;
      }
      const uint32_t sk = sring + st * 2 * L::kCodes, sv = sk + L::kCodes;
      const uint32_t ssk = sscale + st * 256, ssv = ssk + 128;
      const int key0 = first + j * kKvUnit;
      const bool masked = key0 + 32 > end_min;  // uniform over the warp

      // ---- S = Q K^T over 4 n-tiles of 8 keys
      float acc[MT][4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.f;
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
          const uint4 w4 = ld_shared_u4(sk + chunk_at(nt * 8 + kperm(g8), hh * 4 + c4));
          const uint32_t ws[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t b0, b1;
            kv_unpack<FMT>(ws[w], b0, b1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma_16816(acc[mt][nt], qa[mt][hh * 4 + w], b0, b1);
          }
        }
      }

      // ---- V scales: the slice's largest decides whether the running power of two must grow
      float vmine = ld_shared_f(ssv + 4 * lane);
      uint32_t vb = __float_as_uint(vmine) & 0x7fffffffu;
      if (key0 + lane >= item_end || vb >= 0x7f800000u) vb = 0u;  // past the keys, or NaN (which its products carry)
      const uint32_t vmax = __reduce_max_sync(0xffffffffu, vb);
      bool grow = vmax > __float_as_uint(vscale);
      float vgrown = vscale;
      if (grow) vgrown = __uint_as_float(min((vmax & 0x7f800000u) + 0x00800000u, 0x7e800000u));
      const float vinv = __uint_as_float((254u << 23) - __float_as_uint(vgrown));

      // ---- scores times K scales, masks, running maxima
      float kscale[4][2], vratio[4][2];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int kk = nt * 8 + kperm(2 * c4 + e);
          kscale[nt][e] = ld_shared_f(ssk + 4 * kk);
          vratio[nt][e] = ld_shared_f(ssv + 4 * kk) * vinv;
        }
      bool raise = grow;
      float mnew[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float mx = -INFINITY;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& x = acc[mt][nt][half * 2 + e];
              x *= kscale[nt][e];
              if (masked && key0 + nt * 8 + kperm(2 * c4 + e) >= end[mt][half]) x = -INFINITY;
              mx = fmaxf(mx, x);
            }
          mnew[mt][half] = mx * qs[mt][half];
          raise |= mnew[mt][half] > m[mt][half] + 8.f;
        }
      if (__any_sync(0xffffffffu, raise)) {
        const float vs = vscale * vinv;  // both powers of two
        vscale = vgrown;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float alpha[2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float x = fmaxf(m[mt][half], mnew[mt][half]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            alpha[half] = x == -INFINITY ? 1.f : ex2(m[mt][half] - x);
            m[mt][half] = x;
            l[mt][half] *= alpha[half];
            alpha[half] *= vs;
          }
#pragma unroll
          for (int t = 0; t < D / 8; ++t) {
            o[mt][t][0] *= alpha[0], o[mt][t][1] *= alpha[0];
            o[mt][t][2] *= alpha[1], o[mt][t][3] *= alpha[1];
          }
        }
      }

      // ---- P = 2^(x - m + 7); the row sum takes P, the product takes f16(P * V scale ratio)
      uint32_t pa[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float sub = (m[mt][half] == -INFINITY ? 0.f : m[mt][half]) - kKvPShift;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            float pv[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p = ex2(fmaf(acc[mt][nt][half * 2 + e], qs[mt][half], -sub));
              l[mt][half] += p;
              pv[e] = p * vratio[nt][e];
              // a hidden key's scale may be anything, a NaN too
              if (masked && key0 + nt * 8 + kperm(2 * c4 + e) >= end[mt][half]) pv[e] = 0.f;
            }
            pa[mt][nt >> 1][(nt & 1) * 2 + half] = pack_f16x2(pv[0], pv[1]);
          }
        }

      // ---- O += P V: one ldmatrix covers the slice's 32 keys x 16 columns
#pragma unroll
      for (int ch = 0; ch < D / 16; ++ch) {
        uint32_t r[4];
        ldmatrix_x4_trans(r, sv + chunk_at((lane >> 3) * 8 + kperm(lane & 7), ch));
        uint32_t be[4], bo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) kv_unpack<FMT>(r[i], be[i], bo[i]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma_16816(o[mt][2 * ch], pa[mt][0], be[0], be[1]);
          mma_16816(o[mt][2 * ch + 1], pa[mt][0], bo[0], bo[1]);
          mma_16816(o[mt][2 * ch], pa[mt][1], be[2], be[3]);
          mma_16816(o[mt][2 * ch + 1], pa[mt][1], bo[2], bo[3]);
        }
      }
      ++used;
      __syncwarp();  // every lane has read the slice
      if (asked < steps) issue();
    }
    if (!ok) break;

    // ---- the warps' results meet: each leaves (m, l, O) in its own ring, whose slices are all consumed
    float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float lr = l[mt][half];
        lr += __shfl_xor_sync(0xffffffffu, lr, 1);
        lr += __shfl_xor_sync(0xffffffffu, lr, 2);
        const int r = mt * 16 + half * 8 + g8;
        if (c4 == 0) {
          s_m[warp * M + r] = m[mt][half];
          s_l[warp * M + r] = lr;
        }
        // columns 16 ch + 4 c4 + {0, 1, 2, 3}: both n-tiles' columns interleave
#pragma unroll
        for (int ch = 0; ch < D / 16; ++ch)
          *reinterpret_cast<float4*>(mine + r * L::kRowPad + 16 * ch + 4 * c4) =
              make_float4(o[mt][2 * ch][half * 2], o[mt][2 * ch + 1][half * 2], o[mt][2 * ch][half * 2 + 1],
                          o[mt][2 * ch + 1][half * 2 + 1]);
      }
    if (lane == 0) s_v[warp] = vscale * kv_code_scale<FMT>();
    __syncthreads();
    // each row by 128 / 16 = 8 threads, D / 8 columns each
    const bool whole = at.unit == 0 && n == n_item;
    const int slot = u == u0 ? 0 : 1;
    if (at.unit == 0 && threadIdx.x == 0) kv_record(a, line, at, blockIdx.x, u, n_item, whole, u == u0);
#pragma unroll 1
    for (int mt = 0; mt < MT; ++mt) {
      const int r = mt * 16 + (threadIdx.x >> 3), col0 = (threadIdx.x & 7) * (D / 8);
      const KvRow x = kv_row_of(a, s, at.h, at.rt, r);
      if (x.token >= 0) {
        float mx = -INFINITY, f[4], sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) mx = fmaxf(mx, s_m[w * M + r]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          f[w] = s_m[w * M + r] == -INFINITY ? 0.f : ex2(s_m[w * M + r] - mx);
          sum += f[w] * s_l[w * M + r];
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float lse2 = sum == 0.f ? -INFINITY : mx - kKvPShift + log2f(sum);
#pragma unroll
        for (int w = 0; w < 4; ++w) f[w] *= inv * s_v[w];
        float v[D / 8];
#pragma unroll
        for (int e = 0; e < D / 8; e += 4) {
          float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(smem + w * L::kRingPad) + r * L::kRowPad + col0 + e);
            t.x += f[w] * y.x, t.y += f[w] * y.y, t.z += f[w] * y.z, t.w += f[w] * y.w;
          }
          v[e] = t.x, v[e + 1] = t.y, v[e + 2] = t.z, v[e + 3] = t.w;
        }
        kv_put_row<D, D / 8>(a, x, whole, (2ll * blockIdx.x + slot) * M + r, 2ll * gridDim.x * M, col0, v, lse2);
      }
    }
    fence_proxy_async_smem();  // the rings are written by TMA again
    __syncthreads();
    u += n;
    if (u < u1 && !kv_next(a, s, at)) break;
  }
  if (!ok) {
    // leave no copy in flight
    for (uint32_t i = used; i < issued; ++i) mbar_wait_drain(bars + i % S, (i / S) & 1u);
  }
  // the suffix may run beside the prefix; its completion, which the merge waits for, has to mean both
  if (a.phase == kKvSuffix) pdl_wait();
}

}  // namespace fa
