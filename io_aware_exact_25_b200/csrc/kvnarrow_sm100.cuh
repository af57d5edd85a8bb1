// kvnarrow_sm100.cuh -- attention of few rows over the quantised cache.
//
// An item has at most M = 16 rows (query tokens x heads of one key head's
// group), so every key and value byte is used for few products and the cache's
// bytes are what the kernel waits for: the aim is to keep them streaming.
//
// Each warp is its own pipeline.  A unit of 128 keys is four slices of 32, one
// per warp: lane 0 of the warp brings the slice's K and V codes (TMA, swizzled
// by the row width so that every read below is free of bank conflicts) and
// scales (bulk copies) into the warp's ring of kStages slices; the warp alone
// consumes and refills it, running ahead into the CTA's next item, so the warps
// of a CTA never wait for one another until an item ends, when their (m, l, O)
// are merged through shared memory while the next item's bytes arrive.
//
// The products run on mma.sync m16n8k16 in f16, which a 16-row tile fits
// (tcgen05's smallest tile has 64 rows, and at 16 rows the tensor pipe is a
// quarter busy).  Codes become f16 in registers without rounding: an int8 code c
// is the byte c + 128 placed under the exponent of 1024, minus 1152; an e4m3
// code's bits shifted under an f16 sign are its value times 2^-8, subnormals
// included.  No code, not even a NaN pattern in a slot never written, turns
// into an infinity or a NaN.  The K fragment of a lane is 16 consecutive bytes
// of a key row, so the reduction runs over d in a permuted order; Q's
// fragments are loaded in the same order.  V's fragments come from
// ldmatrix.trans on byte pairs; its two columns per pair go to two n-tiles.
//
// Scales: q goes into f16 as it is if the row's largest entry is in [2^-1,
// 2^15), and shifted by a power of two that its scores take back otherwise
// (entries below 2^-14 lose bits that stay below 2^-24 of the largest).  K's
// scale multiplies the fp32 score, in the fma that also subtracts the reference M
// of the row.  V's scale multiplies p = 2^(x - M + 7) before it is rounded to f16:
// M is the running maximum of x plus the exponent of a power of two above every V
// scale that the row has seen (kv_v_top), so p vs <= 2^15 with 11 significant bits
// down to 2^-14.  Keys that the row does not see have no part in M, however large
// their scales.  The row sum takes the unrounded fp32 p, on the same scale as O.
//
// What bounds it: 64 sequences of 512 to 8192 keys, 8 key heads, d = 128, int8:
// 122 us, 4.5 TB/s.  With the products and the softmax left out the call takes 103
// us of 128 (fp8: 110 of 150), so the rest of the way to the bytes' own time is
// arithmetic: the SM issues half of the time and its eight warps wait mostly for
// their own dependent instructions.
#pragma once

#include <type_traits>

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
  asm(
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

// Which power of two scales a row of q into f16: the factor 2^-e and its inverse, from the row's largest |q|.  A row with an
// infinity or a NaN becomes NaN: its scores are infinities or NaN, and so is their softmax.
__device__ __forceinline__ void kv_q_shift(float amax, float& down, float& up) {
  if (__float_as_uint(amax) >= 0x7f800000u) {
    down = __uint_as_float(0x7fc00000u);
    up = 1.f;
    return;
  }
  const uint32_t e = min(max(__float_as_uint(amax) >> 23, 1u), 253u);
  down = __uint_as_float((254u - e) << 23);
  up = __uint_as_float(e << 23);
}

template <int D, int STAGES, int CTAS>
struct KvNarrowLayout {
  static constexpr int kM = 16;
  static constexpr int kStages = STAGES, kCtasPerSm = CTAS;
  static constexpr uint32_t kCodes = 32u * D;                     // one slice of K (or V) codes
  static constexpr uint32_t kStageBytes = 2 * kCodes + 256u;      // then 32 K scales, 32 V scales
  static constexpr uint32_t kRingCodes = kStages * 2 * kCodes;    // codes first: they keep 1024-byte alignment
  static constexpr uint32_t kRing = kRingCodes + kStages * 256u;  // one warp's ring
  static constexpr uint32_t kRingPad = (kRing + 1023u) & ~1023u;
  static constexpr uint32_t kRowPad = D + 4;                      // floats of a merged row (bank spread)
  static constexpr uint32_t kOffMerge = 4 * kRingPad;             // [4 warps][16 rows] O; apart from the rings, which are
                                                                  // already filling for the next item
  static constexpr uint32_t kOffMl = kOffMerge + 4 * 16 * kRowPad * 4;  // [4][kM] M, l and O's factor
  static constexpr uint32_t kOffBar = kOffMl + 12 * kM * 4;
  static constexpr uint32_t kOffScan = kOffBar + 4 * kStages * 8 + 16;
  static constexpr uint32_t kSmem = kOffScan + (uint32_t)sizeof(KvScan);
  static_assert(kOffBar % 8 == 0, "barrier alignment");
  static_assert(kCtasPerSm * (kSmem + 1024) <= 233472, "shared memory budget");
};

// P values carry a factor 2^7 against the running maximum, which is raised only when a score exceeds it by 8.
constexpr float kKvPShift = 7.f;

// A row's range of V scales: ve is the biased exponent of a power of two above every finite one that it has seen, 2^(ve -
// 127).  p carries 2^-(ve - 127) as far as that lies within 2^+-32, which leaves fp32 room for p and its sums; what is
// beyond (`rest`, 1 for scales of ordinary size) multiplies the scale itself.
constexpr int kKvVeMin = 1;

__device__ __forceinline__ int kv_v_shift(int ve) { return min(max(127 - ve, -32), 32); }
__device__ __forceinline__ bool kv_v_beyond(int ve) { return (uint32_t)(ve - 95) > 64u; }
__device__ __forceinline__ float kv_v_rest(int ve) { return __uint_as_float((uint32_t)(254 - ve - kv_v_shift(ve)) << 23); }
__device__ __forceinline__ float kv_v_unrest(int ve) { return __uint_as_float((uint32_t)(ve + kv_v_shift(ve)) << 23); }

// The largest x of a row of its kind: 15 + the shift of p.
__device__ __forceinline__ float kv_v_top(int ve) { return 8.f + kKvPShift + (float)kv_v_shift(ve); }

// Exponent of a power of two above the finite scale of magnitude bits v.
__device__ __forceinline__ int kv_v_exponent(uint32_t v) { return (int)(v >> 23) + 1; }

// A read that stays where it is written (ahead of the copies that are asked for next).
__device__ __forceinline__ uint2 ldg_u2_here(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <int D, int FMT, class L>
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
  float* s_v = s_l + 4 * M;  // what a row's O in a warp is to be multiplied by

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
  KvSeq s{0, 0, 0};
  const KvLine line = kv_place<true, 128>(a, blockIdx.x, gridDim.x, reinterpret_cast<KvScan*>(smem + L::kOffScan), &b,
                                          &s, &rem);
  __syncthreads();
  kv_clear_cuts<true>(a);
  if (b < 0 || *abort_flag) {
    if (a.phase == kKvSuffix) pdl_wait();
    return;
  }
  const Abort ab{abort_flag, a.err};
  const uint64_t pol = policy_evict_first();
  const int total = (int)(line.cut(blockIdx.x + 1) - line.cut(blockIdx.x));  // this CTA's units
  KvPlace at = kv_within<true>(a, s, b, rem);
  const int begin = kv_begin(a);
  const bool two = a.page_shift == 4;  // a slice covers two 16-slot pages
  bool ok = true;

  // ---- the slices this warp asks for, item after item: 32 keys at i_first + 128 j, j < i_steps
  uint32_t issued = 0, used = 0;  // slices asked for and consumed, over all items
  KvSeq is = s;
  KvPlace ia = at;
  int i_left = total, i_j = 0, i_steps = 0, i_first = 0, i_end = 0;
  const int* i_trow = a.table;
  int pg0 = 0, pg1 = 0;  // pages of the item's slices, 32 at a time: lane j holds those of step 32 i + j
  auto slices = [&](int n, int first, int item_end) {  // n units hold n slices of a warp, or one less at the keys' end
    return n == 0 ? 0 : max(first + (n - 1) * kKvUnit >= item_end ? n - 1 : n, 0);
  };
  auto enter = [&]() {
    const KvPart p = kv_part(a, kv_item_units<true>(a, is, 0), ia.from, i_left);
    i_left -= p.take;
    i_end = kv_item_end<true>(a, is, 0);
    i_first = begin + p.start * kKvUnit + warp * 32;
    i_steps = slices(p.n, i_first, i_end);
    i_trow = a.table + (a.phase == kKvPrefix ? 0ll : ia.b * a.table_stride);
    i_j = 0;
  };
  auto issue = [&]() {
    while (i_j == i_steps) {
      if (i_left == 0 || !kv_next<true>(a, is, ia)) return;
      enter();
    }
    const int j = i_j++;
    if ((j & 31) == 0) {
      const int key = i_first + (j + lane) * kKvUnit;
      pg0 = pg1 = 0;
      if (j + lane < i_steps) {
        pg0 = __ldg(i_trow + (key >> a.page_shift));
        if (two && key + 16 < i_end) pg1 = __ldg(i_trow + (key >> 4) + 1);
        if ((uint32_t)pg0 >= (uint32_t)a.num_pages || (uint32_t)pg1 >= (uint32_t)a.num_pages) {
          if (a.err) atomicCAS(a.err, kDevOk, kDevBadPage);
          if ((uint32_t)pg0 >= (uint32_t)a.num_pages) pg0 = 0;
          if ((uint32_t)pg1 >= (uint32_t)a.num_pages) pg1 = 0;
        }
      }
    }
    const int p0 = __shfl_sync(0xffffffffu, pg0, j & 31), p1 = __shfl_sync(0xffffffffu, pg1, j & 31);
    if (lane == 0) {
      const int key = i_first + j * kKvUnit;
      const int st = issued % S;
      uint64_t* bar = bars + st;
      const long long r0 = (((long long)p0 * a.Hkv + ia.h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
      uint8_t* dk = ring + st * 2 * L::kCodes;
      uint8_t* dsc = ring + L::kRingCodes + st * 256;
      // (a row that fails its check: the map answers the codes' load, the scales are not asked for)
      const long long lim = ((long long)a.num_pages * a.Hkv) << a.page_shift;
      (void)lim;
      const bool in0 = FA_IN(kSiteKvRow, r0, two ? 16 : 32, lim, a.err);
      if (!two) {
        mbar_arrive_expect_tx(bar, 2 * L::kCodes + (in0 ? 256u : 0u));
        tma_load_2d(dk, &tm_k, 0, (int)r0, bar, pol);
        tma_load_2d(dk + L::kCodes, &tm_v, 0, (int)r0, bar, pol);
        if (in0) {
          bulk_load(dsc, a.ks + r0, 128, bar);
          bulk_load(dsc + 128, a.vs + r0, 128, bar);
        }
      } else {
        // the second page only if the sequence reaches into it: its table entry may not exist
        const bool more = key + 16 < i_end;
        const long long r1 = ((long long)p1 * a.Hkv + ia.h) << 4;
        const bool in1 = more && FA_IN(kSiteKvRow, r1, 16, lim, a.err);
        mbar_arrive_expect_tx(bar, (more ? 2 * L::kCodes : L::kCodes) + (in0 ? 128u : 0u) + (in1 ? 128u : 0u));
        tma_load_2d(dk, &tm_k, 0, (int)r0, bar, pol);
        tma_load_2d(dk + L::kCodes, &tm_v, 0, (int)r0, bar, pol);
        if (in0) {
          bulk_load(dsc, a.ks + r0, 64, bar);
          bulk_load(dsc + 128, a.vs + r0, 64, bar);
        }
        if (more) {
          tma_load_2d(dk + L::kCodes / 2, &tm_k, 0, (int)r1, bar, pol);
          tma_load_2d(dk + L::kCodes + L::kCodes / 2, &tm_v, 0, (int)r1, bar, pol);
        }
        if (in1) {
          bulk_load(dsc + 64, a.ks + r1, 64, bar);
          bulk_load(dsc + 192, a.vs + r1, 64, bar);
        }
      }
    }
    ++issued;
  };

  for (int left = total; left > 0 && ok;) {
    const int n_item = kv_item_units<true>(a, s, 0);
    const KvPart part = kv_part(a, n_item, at.from, left);
    if (part.n == 0) break;  // the stretch ends before the item's first unit
    const int item_end = kv_item_end<true>(a, s, 0);
    const int first = begin + part.start * kKvUnit + warp * 32;
    const int steps = slices(part.n, first, item_end);

    // ---- Q fragments, in the order the K bytes come: word w of a lane's 16
    // bytes in half hh covers d = 64 hh + 16 c4 + 4 w + {0, 2} and {1, 3}
    uint32_t qa[NH * 4][4];
    float up[2];   // takes back the shift of rows g8, g8 + 8
    bool shifted = false;
    int end[2];    // keys those rows see
    int end_min = item_end;
    uint2 raw[2][NH * 4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const KvRow x = kv_row_of(a, s, at.h, 0, half * 8 + g8);
      end[half] = x.end;
      if (x.token >= 0) end_min = min(end_min, x.end);
      const long long qo = x.token * a.q_sn + x.head * a.q_sh;
      const bool in = x.token >= 0 && FA_IN(kSiteKvQ, qo, D, extent4(1, a.Hq, a.total, D, 0, a.q_sh, a.q_sn), a.err);
#pragma unroll
      for (int w = 0; w < NH * 4; ++w) {
        raw[half][w] = make_uint2(0u, 0u);
        if (in) raw[half][w] = ldg_u2_here(a.q + qo + 64 * (w >> 2) + 16 * c4 + 4 * (w & 3));
      }
    }
    if (left == total) {
      // the first slices, while the first rows of Q are on their way
      enter();
      for (int j = 0; j < S; ++j) issue();
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t m2 = 0u;
#pragma unroll
      for (int w = 0; w < NH * 4; ++w)
        m2 = __vmaxu2(m2, __vmaxu2(raw[half][w].x & 0x7fff7fffu, raw[half][w].y & 0x7fff7fffu));
      m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
      m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
      const float amax = __uint_as_float(max(m2 & 0xffffu, m2 >> 16) << 16);
      float down = 1.f;
      up[half] = 1.f;
      if (!(amax == 0.f || (amax >= 0.5f && amax < 32768.f))) kv_q_shift(amax, down, up[half]);
      shifted |= up[half] != 1.f;
#pragma unroll
      for (int w = 0; w < NH * 4; ++w) {
        qa[w][half] = pack_f16x2(bf16_lo(raw[half][w].x) * down, bf16_lo(raw[half][w].y) * down);
        qa[w][2 + half] = pack_f16x2(bf16_hi(raw[half][w].x) * down, bf16_hi(raw[half][w].y) * down);
      }
    }
    // the smallest reach of any row: slices below it need no mask
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) end_min = min(end_min, __shfl_xor_sync(0xffffffffu, end_min, d));

    shifted = __any_sync(0xffffffffu, shifted);

    float o[D / 8][4];
    float m[2], l[2];  // m, the reference M, means nothing while the row has seen no key (`seen`, bit half)
    uint32_t seen = 0u;
    int ve[2];         // the row's range of V scales
    float top[2];      // kv_v_top of it
    uint32_t vlim = 0u;  // scales from here on (magnitude bits) are above the range of some row of the warp
    bool beyond = false;  // some row's range is outside 2^+-32
    m[0] = m[1] = 0.f;
    ve[0] = ve[1] = kKvVeMin;
    top[0] = top[1] = kv_v_top(kKvVeMin);
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int t = 0; t < D / 8; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

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
      // the four n-tiles side by side: four chains of dependent MMAs, not one after the other
      float acc[4][4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
      for (int hh = 0; hh < NH; ++hh) {
        uint4 w4[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) w4[nt] = ld_shared_u4(sk + chunk_at(nt * 8 + kperm(g8), hh * 4 + c4));
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            uint32_t b0, b1;
            kv_unpack<FMT>(w == 0 ? w4[nt].x : w == 1 ? w4[nt].y : w == 2 ? w4[nt].z : w4[nt].w, b0, b1);
            mma_16816(acc[nt], qa[hh * 4 + w], b0, b1);
          }
      }

      // ---- V scales: the slice's largest decides whether some row's range may have to grow
      uint32_t vb = __float_as_uint(ld_shared_f(ssv + 4 * lane)) & 0x7fffffffu;
      if (key0 + lane >= item_end || vb >= 0x7f800000u) vb = 0u;  // past the keys, or not finite (its products carry that)
      const uint32_t vmax = __reduce_max_sync(0xffffffffu, vb);
      bool raise = vmax >= vlim;

      // ---- x = score * K scale - (M - 7) against the references so far, masks
      const float sl2 = a.scale_log2 * kv_code_scale<FMT>();
      float kscale[4][2], vs[4][2];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int kk = nt * 8 + kperm(2 * c4 + e);
          kscale[nt][e] = ld_shared_f(ssk + 4 * kk) * sl2;
          vs[nt][e] = ld_shared_f(ssv + 4 * kk);
        }
      if (shifted) {
        // (K's scale takes the shift first: a large query's keys may be as small as it is large)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            acc[nt][e] *= kscale[nt][e] * up[0];
            acc[nt][2 + e] *= kscale[nt][e] * up[1];
            kscale[nt][e] = 1.f;
          }
      }
      float mx[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          mx[half] = -INFINITY;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& x = acc[nt][half * 2 + e];
              x = fmaf(x, kscale[nt][e], kKvPShift - m[half]);
              if (masked && key0 + nt * 8 + kperm(2 * c4 + e) >= end[half]) x = -INFINITY;
              mx[half] = fmaxf(mx[half], x);
            }
          const bool first_seen = !((seen >> half) & 1u) && mx[half] != -INFINITY;
          raise |= first_seen || mx[half] > top[half];
        }
      if (__any_sync(0xffffffffu, raise)) {
        // the first visible scores of a row set its maximum, later ones raise it by what they exceed it; a larger range
        // of V scales raises the reference alone
        float alpha[2];  // of O; l's lacks the change of `rest`
        beyond = false;
        if (masked) {  // a row sees the slice's first keys: vb becomes the largest of a lane's key and those before it
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) vb = max(vb, __shfl_up_sync(0xffffffffu, vb, d));
        }
        uint32_t ve_min = 255u;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x = mx[half];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          const uint32_t bit = 1u << half;
          const bool fresh = !(seen & bit) && x != -INFINITY;
          const int nvis = masked ? min(end[half] - key0, 32) : 32;  // keys of the slice that the row sees
          const uint32_t vseen = masked ? __shfl_sync(0xffffffffu, vb, max(nvis - 1, 0)) : vmax;
          const int grown = nvis > 0 ? max(ve[half], kv_v_exponent(vseen)) : ve[half];
          const float top_old = top[half];
          top[half] = kv_v_top(grown);
          const float delta = fresh || x > top_old ? x - (top[half] - 8.f) : top_old - top[half];
          alpha[half] = fresh ? 1.f : ex2(-delta);
          if (fresh) seen |= bit;
          m[half] += delta;
          l[half] *= alpha[half];
          alpha[half] *= kv_v_rest(grown) * kv_v_unrest(ve[half]);
          ve[half] = grown;
          if (seen & bit) {
            beyond |= kv_v_beyond(grown);
            ve_min = min(ve_min, (uint32_t)grown);
          }
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) acc[nt][half * 2 + e] -= delta;
        }
        beyond = __any_sync(0xffffffffu, beyond);
        vlim = __reduce_min_sync(0xffffffffu, ve_min) << 23;
#pragma unroll
        for (int t = 0; t < D / 8; ++t) {
          o[t][0] *= alpha[0], o[t][1] *= alpha[0];
          o[t][2] *= alpha[1], o[t][3] *= alpha[1];
        }
      }

      // ---- P = 2^x; the row sum takes P, the product takes f16(P * V scale)
      uint32_t pa[2][4];
      auto probabilities = [&](auto with_rest) {
        constexpr bool kRest = decltype(with_rest)::value;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float rest = 1.f;
          if constexpr (kRest) rest = kv_v_rest(ve[half]);
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            float pv[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p = ex2(acc[nt][half * 2 + e]);
              l[half] += p;
              pv[e] = p * (kRest ? vs[nt][e] * rest : vs[nt][e]);
              // a hidden key's scale may be anything, a NaN too
              if (masked && key0 + nt * 8 + kperm(2 * c4 + e) >= end[half]) pv[e] = 0.f;
            }
            pa[nt >> 1][(nt & 1) * 2 + half] = pack_f16x2(pv[0], pv[1]);
          }
        }
      };
      if (beyond) probabilities(std::true_type{});
      else probabilities(std::false_type{});

      // ---- O += P V: one ldmatrix covers the slice's 32 keys x 16 columns
#pragma unroll
      for (int cp = 0; cp < D / 16; cp += 2) {
        uint32_t be[2][4], bo[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t r[4];
          ldmatrix_x4_trans(r, sv + chunk_at((lane >> 3) * 8 + kperm(lane & 7), cp + i));
#pragma unroll
          for (int k = 0; k < 4; ++k) kv_unpack<FMT>(r[k], be[i][k], bo[i][k]);
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mma_16816(o[2 * (cp + i)], pa[kk], be[i][2 * kk], be[i][2 * kk + 1]);
              mma_16816(o[2 * (cp + i) + 1], pa[kk], bo[i][2 * kk], bo[i][2 * kk + 1]);
            }
      }
      ++used;
      __syncwarp();  // every lane has read the slice
      issue();
    }
    if (!ok) break;

    // ---- the warps' results meet, 16 rows at a time
    const bool whole = part.n == n_item;
    const long long piece = (2ll * blockIdx.x + (left == total ? 0 : 1)) * M;
    if (part.start == 0 && threadIdx.x == 0)
      kv_record(a, line, s, at, blockIdx.x, line.cut(blockIdx.x) + (total - left) - at.from, n_item, whole, left == total);
    float* mine = reinterpret_cast<float*>(smem + L::kOffMerge) + warp * 16 * L::kRowPad;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float lr = l[half];
      lr += __shfl_xor_sync(0xffffffffu, lr, 1);
      lr += __shfl_xor_sync(0xffffffffu, lr, 2);
      const int r = half * 8 + g8;
      if (c4 == 0) {
        s_m[warp * M + r] = (seen >> half) & 1u ? m[half] : -INFINITY;
        s_l[warp * M + r] = lr;
        s_v[warp * M + r] = kv_v_unrest(ve[half]) * kv_code_scale<FMT>();
      }
      // columns 16 ch + 4 c4 + {0, 1, 2, 3}: both n-tiles' columns interleave
#pragma unroll
      for (int ch = 0; ch < D / 16; ++ch)
        *reinterpret_cast<float4*>(mine + r * L::kRowPad + 16 * ch + 4 * c4) =
            make_float4(o[2 * ch][half * 2], o[2 * ch + 1][half * 2], o[2 * ch][half * 2 + 1],
                        o[2 * ch + 1][half * 2 + 1]);
    }
    __syncthreads();
    // each row by 128 / 16 = 8 threads, D / 8 columns each
    const int rr = threadIdx.x >> 3, r = rr, col0 = (threadIdx.x & 7) * (D / 8);
    const KvRow x = kv_row_of(a, s, at.h, 0, r);
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
      for (int w = 0; w < 4; ++w) f[w] *= inv * s_v[w * M + r];
      float v[D / 8];
#pragma unroll
      for (int e = 0; e < D / 8; e += 4) {
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + L::kOffMerge) +
                                                            (w * 16 + rr) * L::kRowPad + col0 + e);
          t.x += f[w] * y.x, t.y += f[w] * y.y, t.z += f[w] * y.z, t.w += f[w] * y.w;
        }
        v[e] = t.x, v[e + 1] = t.y, v[e + 2] = t.z, v[e + 3] = t.w;
      }
      kv_put_row<D, D / 8>(a, x, whole, piece + r, 2ll * gridDim.x * M, col0, v, lse2);
    }
    __syncthreads();  // the buffer is free again
    left -= part.take;
    if (left > 0 && !kv_next<true>(a, s, at)) break;
  }
  if (!ok) {
    // leave no copy in flight
    for (uint32_t i = used; i < issued; ++i) mbar_wait_drain(bars + i % S, (i / S) & 1u);
  }
  // the suffix may run beside the prefix; its completion, which the merge waits for, has to mean both
  if (a.phase == kKvSuffix) pdl_wait();
}

}  // namespace fa
