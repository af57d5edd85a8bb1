// kvwide_sm100.cuh -- attention of many rows over the quantised cache: a
// prompt's chunk, or a whole batch's queries over its shared prefix.
//
// An item tile is 256 rows (query tokens x heads of one key head's group) as
// two 128-row tiles, the shape of the dense forward (fwd_sm100.cuh): tcgen05
// MMAs S_t = Q_t K^T and O_t += P_t V accumulate in tensor memory and the two
// tiles take turns on the tensor core.  What differs is where K and V come
// from.  Warp roles:
//   warps 0-3   softmax of tile 0 (a thread per row; they also load Q)
//   warps 4-7   softmax of tile 1
//   then CW     converter: codes to f16 operand tiles
//   then one    MMA issue (one thread)
//   then one    producer: codes from the cache's pages to shared memory by bulk
//               copies, a page (or 128 rows) at a time
//   then one    scales, from the pages to what the softmax reads
//               and one that completes the warpgroup
// CW is 4, or 8 where items have at most 128 rows.  Then both row tiles are the
// same rows and share the keys: tile 0 takes the even key tiles, tile 1 the odd
// ones, each with its own maximum, sum and O, and tile 0 adds the two up at the
// end (tile 1's O is in the same tensor-memory lanes).  The two together go through
// the keys in 1.5 us a tile instead of 2.5, hence the 8.
// The converter threads take 16 codes at a time, unpack them exactly as the
// narrow kernel does and write the f16 tile in the 128-byte swizzled layout the
// MMA reads: 256 rows share one conversion.  (They first loaded the codes
// themselves, a tile ahead in registers; every load of a page number, a scale
// or a tile then stood in the way of the next conversion, about 5000 clocks a
// tile.)  Inside each group of four the columns stand in the order 0, 2, 1, 3, in
// which the codes unpack; Q is stored the same way and O's columns are put back
// at the end.
//
// Scales: K's multiply the fp32 scores, in the fma that also subtracts the
// reference M of the row; the softmax scale is folded into them.  V's multiply
// p = 2^(x - M + 7) before its one rounding to f16, where M is the running maximum of
// x plus the exponent of a power of two above every V scale that the row has seen,
// as in the narrow kernel: keys that a row does not see have no part in its result.
// (Multiplied into V's codes during the conversion, as f16 ratios to one power of
// two, they cost two more roundings, and a hidden key's large scale the bits of the
// rows beside it.  The chunk below took 245 us a call then and 224 now, 269 and
// 235 with fp8 codes.)  A scale that is not finite makes its products NaN or
// infinite, of the rows that see its key; only where a tile has one are p vs set to 0
// for the other rows, in a second form of the loop that is kept off the usual path:
// taken by every masked tile, the two forms in turn cost the chunk 14 us.  q goes into f16 as
// it is if the row's largest entry is in [2^-1, 2^15), and shifted by a power of two
// that its scores take back otherwise.
//
// The scores of a row stay in its thread's registers: x = s ks - (M - 7) at
// once, against the reference so far, and only where some x exceeds its row's top
// is M raised and x shifted, so the usual tile costs one fma, half a max3, one
// exponential, half an add, half a product and half a conversion per score.
//
// What bounds it: without masks, one item a CTA, d = 128, 128 keys take 2.5 us at
// 256 rows (int8; 2.6 with fp8) and 1.5 us at up to 128 rows.  Of the 2.5 the MMAs
// are 1.04 us (2048 clocks) and the exponentials as much (32768, 16 a clock): S of
// the next key tile waits for P V of this one, and P for the softmax, so that the two
// hardly overlap within a row tile.  Launch, Q, the first S, the epilogue and the
// merge add about 25 us to a call.  Four prompts' chunks of 256 to 2048 tokens over
// up to 8192 keys, 16 heads, d = 128, int8: 209 us, 620 TFLOP/s of the useful
// products, tensor pipe 33 %; 32768 shared keys of 64 sequences, 8 key heads of 4
// query heads, fp8: 62 us.
#pragma once

#include "kvnarrow_sm100.cuh"

namespace fa {

template <int D, int CW>
struct KvWideLayout {
  static constexpr int kM = 256;
  static constexpr int kSoftmaxWarps = 8, kConvertWarps = CW;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + kConvertWarps + 4);
  static constexpr int kConvert = 32 * kConvertWarps;
  // launched at 128 registers a thread with 4 converter warps (512 x 128 = 256 x 192 + 128 x 72 + 128 x 56), at 96
  // with 8 (640 x 96 = 256 x 176 + 256 x 40 + 128 x 48)
  static constexpr uint32_t kRegsLaunch = CW == 4 ? 128 : 96;
  static constexpr uint32_t kRegsSoftmax = CW == 4 ? 192 : 176, kRegsConvert = CW == 4 ? 72 : 40;
  static constexpr uint32_t kRegsCtl = CW == 4 ? 56 : 48;
  static_assert(CW == 4 || CW == 8, "whole warpgroups");
  static_assert(256 * kRegsSoftmax + 32 * CW * kRegsConvert + 128 * kRegsCtl <= kRegsLaunch * kThreads, "register split");
  static constexpr uint32_t kHalf = 128u * 128u;    // 128 rows x 64 f16 columns
  static constexpr uint32_t kTile = 128u * D * 2u;  // 128 x D f16
  static constexpr bool kSplit = CW == 8;  // at most 128 rows: the two tiles share the keys, and one Q tile is enough
  // K/V operand ring.  Four tiles: K(j + 1) then takes the place of K(j - 1), which the step before freed; with three
  // it took V(j - 1)'s, freed at the end of step j, and its conversion stood in the way (1200 clocks a tile when tried).
  static constexpr int kStages = D == 128 ? 4 : 6;
  // ring of codes: K(j), V(j), K(j + 1), ...; at d = 128 kSplit has the place of the second Q tile for a third
  static constexpr int kRaw = D == 128 ? (kSplit ? 3 : 2) : 4;
  static constexpr uint32_t kRawCodes = 128u * D;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffKV = (kSplit ? 1 : 2) * kTile;
  static constexpr uint32_t kOffRaw = kOffKV + kStages * kTile;
  static constexpr uint32_t kOffScale = kOffRaw + kRaw * kRawCodes;  // [2] 128 K scales times the softmax scale, 128 V scales
  static constexpr uint32_t kOffVMax = kOffScale + 2 * 1024;  // [2][32] largest finite |V scale| of the first 4 (i + 1) keys;
                                                              // the sign says that the tile has one that is not finite
  static constexpr uint32_t kOffBar = kOffVMax + 2 * 128;
  static constexpr int kNumBars = 2 + 2 * kStages + 2 * kRaw + 2 + 4 + 2 + 2 + 2 + 1 + 1;
  static constexpr uint32_t kOffScan = kOffBar + kNumBars * 8 + 16;
  static constexpr uint32_t kSmem = kOffScan + (uint32_t)sizeof(KvScan);
  static constexpr uint32_t kColO = 256;  // tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (D each)
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kOffScan % 8 == 0, "scan scratch alignment");
};

// Instruction descriptor of kind::f16 with f16 inputs and fp32 accumulation (format codes 0; the other fields as
// idesc_bf16).
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Load 16 columns and wait for them.
__device__ __forceinline__ void tmem_ld16_sync(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  tmem_ld_wait();
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// The MMA warp's instructions, reached by all its lanes together and issued by the one that elect.sync names.  Where
// the compiler sees a warp-uniform path and operands they go straight from uniform registers; issued from under
// `lane == 0` the same MMAs took 116-216 clocks each whatever their size, against 64 of tensor-core time.
__device__ __forceinline__ void mma_ss_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_ts_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// Two columns of a thread's lane.
__device__ __forceinline__ void tmem_st2(uint32_t taddr, uint32_t a, uint32_t b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ void tmem_ld2_sync(uint32_t taddr, uint32_t& a, uint32_t& b) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(taddr));
  tmem_ld_wait();
  asm volatile("" : "+r"(a), "+r"(b) : : "memory");
}

__device__ __forceinline__ uint32_t ld_shared_u(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void st_shared_u(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Magnitude bits of a scale, 0 if it is not finite.
__device__ __forceinline__ uint32_t kv_finite_bits(uint32_t v) {
  v &= 0x7fffffffu;
  return v < 0x7f800000u ? v : 0u;
}

template <int D, int FMT, int CW>
__global__ void __launch_bounds__(KvWideLayout<D, CW>::kThreads, 1) kv_wide_kernel(const KvArgs a) {
  using L = KvWideLayout<D, CW>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // (through a shuffle: the roles' branches are then uniform to the compiler)
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* bar_q = bars;                              // [2] Q_t written (128 arrivals)
  uint64_t* bar_kv_full = bars + 2;                    // [S] operand tile written
  uint64_t* bar_kv_empty = bar_kv_full + L::kStages;   // [S] operand tile consumed
  uint64_t* bar_raw_full = bar_kv_empty + L::kStages;  // [R] codes landed
  uint64_t* bar_raw_empty = bar_raw_full + L::kRaw;    // [R] codes converted
  uint64_t* bar_s = bar_raw_empty + L::kRaw;           // [2] S_t ready
  uint64_t* bar_p = bar_s + 2;                         // [2][2] half h of P_t written (128)
  uint64_t* bar_pv = bar_p + 4;                        // [2] O_t += P_t V done
  uint64_t* bar_sc_full = bar_pv + 2;                  // [2] scales of a key tile written (32)
  uint64_t* bar_sc_empty = bar_sc_full + 2;            // [2] scales consumed (8 warps)
  uint64_t* bar_half = bar_sc_empty + 2;               //     kSplit: tile 1's half of the keys is done (4 warps)
  uint64_t* bar_drain = bar_half + 1;                  //     every MMA retired
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sscale = sbase + L::kOffScale, svmax = sbase + L::kOffVMax;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar_q[t], 128);
      mbar_init(&bar_s[t], 1);
      mbar_init(&bar_p[2 * t], 128);
      mbar_init(&bar_p[2 * t + 1], 128);
      mbar_init(&bar_pv[t], 1);
      mbar_init(&bar_sc_full[t], 32);
      mbar_init(&bar_sc_empty[t], L::kSoftmaxWarps);
    }
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&bar_kv_full[i], L::kConvert);
      mbar_init(&bar_kv_empty[i], 1);
    }
    for (int i = 0; i < L::kRaw; ++i) {
      mbar_init(&bar_raw_full[i], 1);
      mbar_init(&bar_raw_empty[i], L::kConvertWarps);
    }
    mbar_init(bar_half, 4);
    mbar_init(bar_drain, 1);
    const bool misaligned = (sbase & 1023u) != 0u;
    *abort_flag = misaligned ? 1 : 0;
    if (misaligned && a.err) atomicCAS(a.err, kDevOk, kDevMisaligned);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_trigger();
  int b;
  long long rem;
  KvSeq s{0, 0, 0};
  const KvLine line = kv_place<false, L::kThreads>(a, blockIdx.x, gridDim.x,
                                                   reinterpret_cast<KvScan*>(smem + L::kOffScan), &b, &s, &rem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const Abort ab{abort_flag, a.err};
  const bool run = b >= 0 && *abort_flag == 0;
  kv_clear_cuts<false>(a);
  const int total = b >= 0 ? (int)(line.cut(blockIdx.x + 1) - line.cut(blockIdx.x)) : 0;  // this CTA's units
  KvLine* s_line = reinterpret_cast<KvLine*>(smem + L::kOffScan);  // kept for kv_record only (the scan is over)
  if (threadIdx.x == 0) *s_line = line;
  const int begin = kv_begin(a);
  KvPlace at{0, 0, 0, 0};
  if (run) at = kv_within<false>(a, s, b, rem);
  // Every role walks the same items: n units of the item at `at`, from key `first` on; act1 if the second row tile
  // has rows.
  auto act1_of = [&]() { return (uint32_t)at.rt * 256u + 128u < (uint32_t)s.lq * (uint32_t)a.g; };

  if (warp >= L::kSoftmaxWarps + L::kConvertWarps) {
    regs_dec<L::kRegsCtl>();
    if (run && warp == L::kSoftmaxWarps + L::kConvertWarps) {
      // ------------------------------------------------------ MMA issue
      // Order for key tile j: O0 += P0 V(j-1), S0(j), O1 += P1 V(j-1), S1(j), as in the dense forward: S_t(j)
      // overwrites the columns of P_t(j-1) behind the product that reads them, and a completed S_t(j) implies that
      // O_t holds every earlier product.
      constexpr uint32_t kIdS = idesc_f16(128, 128, false);
      constexpr uint32_t kIdO = idesc_f16(128, D, true);
      uint32_t pos = 0;           // operand ring position: K(j) then V(j), over all items
      uint32_t nq0 = 0, nq1 = 0;  // items of each row tile so far
      uint32_t np0 = 0, np1 = 0;  // P tiles of each row tile so far
      bool ok = true, issued = false;
      auto full = [&](uint32_t p) { return mbar_wait_warp(&bar_kv_full[p % L::kStages], (p / L::kStages) & 1u, ab); };
      // Descriptors of slice 0; a slice further on is a constant added to the address field (addresses stay below
      // 2^18, so nothing carries out of it).
      const uint64_t dq0 = desc_kmajor(sbase + L::kOffQ, 0, L::kHalf);
      const uint64_t dk0 = desc_kmajor(sbase + L::kOffKV, 0, L::kHalf);
      const uint64_t dv0 = desc_mnmajor(sbase + L::kOffKV, 0, L::kHalf);
      auto stage_step = [](uint32_t p) { return (uint64_t)((p % L::kStages) * (L::kTile >> 4)); };
      auto issue_s = [&](int t, int tq, uint32_t p) {  // S_t = Q_tq K^T
        uint64_t dq = dq0 + (uint64_t)(tq * (L::kTile >> 4)), dk = dk0 + stage_step(p);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          mma_ss_elect(tmem + 128u * t, dq, dk, kIdS, kk > 0 ? 1u : 0u);
          const uint64_t step = kk == 3 ? (uint64_t)((L::kHalf - 96u) >> 4) : 2ull;  // the next 16 columns
          dq += step;
          dk += step;
        }
        mma_commit_elect(&bar_s[t]);
        issued = true;
      };
      auto issue_pv = [&](int t, bool first, uint32_t p) -> bool {
        uint64_t dv = dv0 + stage_step(p);
        const uint32_t ph = (t ? np1++ : np0++) & 1u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!mbar_wait_warp(&bar_p[2 * t + h], ph, ab)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            mma_ts_elect(tmem + L::kColO + D * t, tmem + 128u * t + 32u * h + 8u * kk, dv, kIdO,
                   (!first || h > 0 || kk > 0) ? 1u : 0u);
            dv += 2048u >> 4;  // 16 keys further down
          }
        }
        mma_commit_elect(&bar_pv[t]);
        return true;
      };
      for (int left = total; left > 0 && ok;) {
        const KvPart part = kv_part(a, kv_item_units<false>(a, s, at.rt), at.from, left);
        const int n = part.n;
        if (n == 0) break;  // the stretch ends before the item's first unit
        const int nt = act1_of() ? 2 : 1;
#pragma unroll 1
        for (int t = 0; t < nt && ok; ++t) ok = mbar_wait_warp(&bar_q[t], (t ? nq1++ : nq0++) & 1u, ab);
        if constexpr (L::kSplit) {
          // step j: O_t += P_t V(j - 2), S_t(j), t = j mod 2
#pragma unroll 1
          for (int j = 0; j < n + 2 && ok; ++j) {
            const uint32_t pk = pos + 2u * j, pv = pk - 3u;
            if (j >= 2 && j - 2 < n) {
              if (!(ok = full(pv)) || !(ok = issue_pv(j & 1, j < 4, pv))) break;
              mma_commit_elect(&bar_kv_empty[pv % L::kStages]);
            }
            if (j < n) {
              if (!(ok = full(pk))) break;
              tc_fence_after();
              issue_s(j & 1, 0, pk);
              mma_commit_elect(&bar_kv_empty[pk % L::kStages]);
            }
          }
        } else {
#pragma unroll 1
          for (int j = 0; j <= n && ok; ++j) {
            // tiles in hand: K(j) at pos + 2 j, V(j - 1) at pos + 2 j - 1
            const uint32_t pk = pos + 2u * j, pv = pk - 1u;
            if (j > 0 && !(ok = full(pv))) break;
            if (j < n && !(ok = full(pk))) break;
            tc_fence_after();
#pragma unroll 1
            for (int t = 0; t < nt && ok; ++t) {
              if (j > 0) ok = issue_pv(t, j == 1, pv);
              if (ok && j < n) issue_s(t, t, pk);
            }
            if (!ok) break;
            if (j > 0) mma_commit_elect(&bar_kv_empty[pv % L::kStages]);
            if (j < n) mma_commit_elect(&bar_kv_empty[pk % L::kStages]);
          }
        }
        pos += 2u * n;
        left -= part.take;
        if (left > 0 && !kv_next<false>(a, s, at)) break;
      }
      if (issued) {
        mma_commit_elect(bar_drain);
        mbar_wait_drain(bar_drain, 0);
      }
    }
    if (run && warp == L::kSoftmaxWarps + L::kConvertWarps + 1) {
      // ------------------------------------------------------- producer
      // Lane l brings rows [l g, (l + 1) g) of a tile, g = min(page size, 128): they are contiguous in their page.
      // Rows past the item's keys are not asked for unless they share a page with a key; what the slot held before
      // stands in for them (any code is finite, and such keys have scale 0).
      const int g = min(1 << a.page_shift, 128);
      uint32_t pos = 0;
      bool ok = true;
      for (int left = total; left > 0 && ok;) {
        const KvPart part = kv_part(a, kv_item_units<false>(a, s, at.rt), at.from, left);
        const int n = part.n;
        if (n == 0) break;  // the stretch ends before the item's first unit
        const int item_end = kv_item_end<false>(a, s, at.rt);
        const int first = begin + part.start * kKvUnit;
        const int* trow = a.table + (a.phase == kKvPrefix ? 0ll : at.b * a.table_stride);
        auto fetch = [&](int j) -> int {  // this lane's cache row in tile j, or -1
          const int key = first + j * kKvUnit + g * lane;
          return j < n && g * lane < 128 && key < item_end ? __ldg(trow + (key >> a.page_shift)) : -1;
        };
        auto row_of = [&](int j, int page) -> long long {
          const int key = first + j * kKvUnit + g * lane;
          return (((long long)page * a.Hkv + at.h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
        };
        int page_next = fetch(0);
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          int page = page_next;
          page_next = fetch(j + 1);
          const bool mine = g * lane < 128 && first + j * kKvUnit + g * lane < item_end;
          if (mine && (uint32_t)page >= (uint32_t)a.num_pages) {
            if (a.err) atomicCAS(a.err, kDevOk, kDevBadPage);
            page = 0;
          }
          const long long row = row_of(j, page);
          const bool in = mine && FA_IN(kSiteKvRow, row, g, ((long long)a.num_pages * a.Hkv) << a.page_shift, a.err);
          const uint32_t rows = (uint32_t)g * (uint32_t)__popc(__ballot_sync(0xffffffffu, in));
#pragma unroll 1
          for (int which = 0; which < 2; ++which) {
            const uint32_t sl = pos % L::kRaw;
            if (!(ok = mbar_wait_warp(&bar_raw_empty[sl], ((pos / L::kRaw) & 1u) ^ 1u, ab))) break;
            if (lane == 0) mbar_arrive_expect_tx(&bar_raw_full[sl], rows * (uint32_t)D);
            __syncwarp();
            uint8_t* dst = smem + L::kOffRaw + sl * L::kRawCodes;
            if (in) bulk_load(dst + g * lane * D, (which ? a.v : a.k) + row * D, (uint32_t)(g * D), &bar_raw_full[sl]);
            ++pos;
          }
        }
        left -= part.take;
        if (left > 0 && !kv_next<false>(a, s, at)) break;
      }
      // every copy asked for lands before the CTA may exit
      for (uint32_t p = pos > L::kRaw ? pos - L::kRaw : 0u; p < pos; ++p)
        mbar_wait_drain(&bar_raw_full[p % L::kRaw], (p / L::kRaw) & 1u);
    }
    if (run && warp == L::kSoftmaxWarps + L::kConvertWarps + 2) {
      // --------------------------------------------------------- scales
      // Lane l brings keys 4 l to 4 l + 3 of a tile, which share a page; the page number comes a tile ahead, and the two
      // stages keep the scales ahead of the softmax.  Keys past the item's, or of a page outside the cache, have scale 0.
      uint32_t nsc = 0;
      bool ok = true;
      for (int left = total; left > 0 && ok;) {
        const KvPart part = kv_part(a, kv_item_units<false>(a, s, at.rt), at.from, left);
        const int n = part.n;
        if (n == 0) break;  // the stretch ends before the item's first unit
        const int item_end = kv_item_end<false>(a, s, at.rt);
        const int key_l = begin + part.start * kKvUnit + 4 * lane;  // this lane's first key of the first tile
        const int* trow = a.table + (a.phase == kKvPrefix ? 0ll : at.b * a.table_stride);
        auto page_of = [&](int j) -> int {
          const int key = key_l + j * kKvUnit;
          return j < n && key < item_end ? __ldg(trow + (key >> a.page_shift)) : -1;
        };
        int page = page_of(0);
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++nsc) {
          float4 k4 = make_float4(0.f, 0.f, 0.f, 0.f), v4 = k4;
          const long long row = (((long long)page * a.Hkv + at.h) << a.page_shift) +
                                ((key_l + j * kKvUnit) & ((1 << a.page_shift) - 1));
          if ((uint32_t)page < (uint32_t)a.num_pages &&
              FA_IN(kSiteKvRow, row, 4, ((long long)a.num_pages * a.Hkv) << a.page_shift, a.err)) {
            k4 = __ldg(reinterpret_cast<const float4*>(a.ks + row));
            v4 = __ldg(reinterpret_cast<const float4*>(a.vs + row));
          }
          page = page_of(j + 1);
          const uint32_t st = nsc & 1u;
          if (!(ok = mbar_wait_warp(&bar_sc_empty[st], ((nsc >> 1) & 1u) ^ 1u, ab))) break;
          const int keys = item_end - (key_l + j * kKvUnit);  // of the four
          const float f = a.scale_log2 * kv_code_scale<FMT>();
          const float ks[4] = {k4.x * f, k4.y * f, k4.z * f, k4.w * f}, vs[4] = {v4.x, v4.y, v4.z, v4.w};
          uint32_t kb[4], vb[4], vmax = 0u;
          bool odd = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            kb[i] = i < keys ? __float_as_uint(ks[i]) : 0u;
            vb[i] = i < keys ? __float_as_uint(vs[i]) : 0u;
            vmax = max(vmax, kv_finite_bits(vb[i]));
            odd |= (vb[i] & 0x7fffffffu) >= 0x7f800000u;
          }
          odd = __any_sync(0xffffffffu, odd);
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) vmax = max(vmax, __shfl_up_sync(0xffffffffu, vmax, d));
          st_shared_v4(sscale + st * 1024 + 16 * lane, kb[0], kb[1], kb[2], kb[3]);
          st_shared_v4(sscale + st * 1024 + 512 + 16 * lane, vb[0], vb[1], vb[2], vb[3]);
          st_shared_u(svmax + st * 128 + 4 * lane, odd ? vmax | 0x80000000u : vmax);
          mbar_arrive(&bar_sc_full[st]);
        }
        left -= part.take;
        if (left > 0 && !kv_next<false>(a, s, at)) break;
      }
    }
  } else if (warp >= L::kSoftmaxWarps) {
    regs_dec<L::kRegsConvert>();
    if (run) {
      // ------------------------------------------------------ converter
      constexpr int CH = D / 16;           // 16-code chunks of a row
      constexpr int RP = L::kConvert / CH; // rows the threads cover in one pass
      constexpr int NP = 128 / RP;         // passes of a tile
      const int tid = threadIdx.x - 32 * L::kSoftmaxWarps;
      const int ch = tid % CH, r_in = tid / CH;
      // the chunk's place in its row of the operand tile: 16 f16 columns are two 16-byte chunks of the 64-column half
      // ch / 4.  At d = 128 eight lanes store one row, and those of the upper half write the second one first, so that
      // the eight cover all banks; at d = 64 they store two rows, whose swizzles differ already.
      const int c0 = 2 * (ch & 3), swap = D == 128 ? (ch >> 2) & 1 : 0;
      static_assert(RP % 8 == 0, "a thread's rows share their swizzle");
      const uint32_t row_off = (uint32_t)(ch >> 2) * L::kHalf + r_in * 128;
      const uint32_t off0 = row_off + (((c0 + swap) ^ (r_in & 7)) << 4), off1 = row_off + (((c0 + 1 - swap) ^ (r_in & 7)) << 4);
      uint32_t pos = 0;
      bool ok = true;
      for (int left = total; left > 0 && ok;) {
        const KvPart part = kv_part(a, kv_item_units<false>(a, s, at.rt), at.from, left);
        if (part.n == 0) break;  // the stretch ends before the item's first unit
        // tiles K, V, K, V, ...
#pragma unroll 1
        for (int j = 0; j < 2 * part.n; ++j, ++pos) {
          const uint32_t st = pos % L::kStages, sl = pos % L::kRaw;
          const uint32_t src = sbase + L::kOffRaw + sl * L::kRawCodes + ch * 16;
          if (!(ok = mbar_wait_warp(&bar_raw_full[sl], (pos / L::kRaw) & 1u, ab))) break;
          uint4 raw[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) raw[i] = ld_shared_u4(src + (i * RP + r_in) * D);
          if (!(ok = mbar_wait_warp(&bar_kv_empty[st], ((pos / L::kStages) & 1u) ^ 1u, ab))) break;
          const uint32_t tile = sbase + L::kOffKV + st * L::kTile;
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            uint32_t w[8];
            kv_unpack<FMT>(raw[i].x, w[0], w[1]);
            kv_unpack<FMT>(raw[i].y, w[2], w[3]);
            kv_unpack<FMT>(raw[i].z, w[4], w[5]);
            kv_unpack<FMT>(raw[i].w, w[6], w[7]);
            const uint32_t at0 = tile + off0 + i * (RP * 128), at1 = tile + off1 + i * (RP * 128);
            if (swap) {
              st_shared_v4(at0, w[4], w[5], w[6], w[7]);
              st_shared_v4(at1, w[0], w[1], w[2], w[3]);
            } else {
              st_shared_v4(at0, w[0], w[1], w[2], w[3]);
              st_shared_v4(at1, w[4], w[5], w[6], w[7]);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&bar_kv_full[st]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_raw_empty[sl]);
        }
        left -= part.take;
        if (left > 0 && !kv_next<false>(a, s, at)) break;
      }
    }
  } else {
    regs_inc<L::kRegsSoftmax>();
    if (run) {
      // -------------------------------------------------------- softmax
      const int t = warp >> 2, quad = warp & 3;
      const int r = quad * 32 + lane;  // row of the tile == TMEM lane
      const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
      const uint32_t tS = tmem + lane_off + 128u * t;
      const uint32_t tO = tmem + lane_off + L::kColO + D * t;
      uint32_t ns = 0, nsc = 0;  // score tiles and scale stages so far
      uint32_t nhalf = 0;        // kSplit: items with a second half so far
      bool ok = true;
      for (int left = total; left > 0 && ok;) {
        const int n_item = kv_item_units<false>(a, s, at.rt);
        const KvPart part = kv_part(a, n_item, at.from, left);
        const int n = part.n;
        if (n == 0) break;
        const int first = begin + part.start * kKvUnit;
        if (!L::kSplit && t == 1 && !act1_of()) {
          // no rows here: only release the scales
          for (int j = 0; j < n && ok; ++j, ++nsc) {
            ok = mbar_wait_warp(&bar_sc_full[nsc & 1u], (nsc >> 1) & 1u, ab);
            if (ok && lane == 0) mbar_arrive(&bar_sc_empty[nsc & 1u]);
          }
        } else {
          KvRow x = kv_row_of(a, s, at.h, at.rt, L::kSplit ? r : t * 128 + r);
          if (x.token < 0) x.end = 0x7fffffff;  // a row that is not there needs no mask: nothing of it is stored
          float up = 1.f;
          {
            // this thread's row of Q as f16, columns in the order the codes unpack
            const long long qo = x.token * a.q_sn + x.head * a.q_sh;
            const bool in =
                x.token >= 0 && FA_IN(kSiteKvQ, qo, D, extent4(1, a.Hq, a.total, D, 0, a.q_sh, a.q_sn), a.err);
            const uint4* src = reinterpret_cast<const uint4*>(a.q + (in ? qo : 0));
            uint4 w[D / 8];
            uint32_t m2 = 0u;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) w[c] = in ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu),
                                         __vmaxu2(w[c].z & 0x7fff7fffu, w[c].w & 0x7fff7fffu)));
            const float amax = __uint_as_float(max(m2 & 0xffffu, m2 >> 16) << 16);
            float down = 1.f;
            if (!(amax == 0.f || (amax >= 0.5f && amax < 32768.f))) kv_q_shift(amax, down, up);
            if (!L::kSplit || t == 0) {
              const uint32_t row = sbase + L::kOffQ + t * L::kTile + r * 128;
#pragma unroll
              for (int c = 0; c < D / 8; ++c)
                st_shared_v4(row + (c >> 3) * L::kHalf + (((c & 7) ^ (r & 7)) << 4),
                             pack_f16x2(bf16_lo(w[c].x) * down, bf16_lo(w[c].y) * down),
                             pack_f16x2(bf16_hi(w[c].x) * down, bf16_hi(w[c].y) * down),
                             pack_f16x2(bf16_lo(w[c].z) * down, bf16_lo(w[c].w) * down),
                             pack_f16x2(bf16_hi(w[c].z) * down, bf16_hi(w[c].w) * down));
              fence_proxy_async_smem();
              mbar_arrive(&bar_q[t]);
            }
          }
          const bool shifted = __any_sync(0xffffffffu, up != 1.f);
          float m = 0.f, l = 0.f;  // m, the reference M, means nothing while l = 0
          int ve = kKvVeMin;       // the row's range of V scales
          float top = kv_v_top(kKvVeMin);
          bool beyond = false;     // some row's of the warp is outside 2^+-32
#pragma unroll 1
          for (int j = 0; j < n; ++j) {
            const uint32_t st = nsc & 1u;
            if (!(ok = mbar_wait_warp(&bar_sc_full[st], (nsc >> 1) & 1u, ab))) break;
            if (L::kSplit && (j & 1) != t) {  // the other tile's keys
              if (lane == 0) mbar_arrive(&bar_sc_empty[st]);
              ++nsc;
              continue;
            }
            if (!(ok = mbar_wait_warp(&bar_s[t], ns & 1u, ab))) break;
            tc_fence_after();
            const uint32_t sK = sscale + st * 1024, sV = sK + 512;
            const int lim = x.end - (first + j * kKvUnit);  // of the tile's keys, those below it are visible
            const bool masked = __any_sync(0xffffffffu, lim < 128);
            uint32_t vmax = ld_shared_u(svmax + st * 128 + 124);  // the largest V scale that the row sees in this tile
            const bool odd = (int)vmax < 0;
            vmax &= 0x7fffffffu;
            uint32_t w[4][32];
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) tmem_ld32(tS + 32u * c4, w[c4]);
            tmem_ld_wait();
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) reg_fence(w[c4]);
            const uint64_t sub2 = f2_pack(kKvPShift - m, kKvPShift - m);
            auto scores = [&](auto with_shift) {
#pragma unroll
              for (int c = 0; c < 128; c += 4) {
                float4 k4 = ld_shared_f4(sK + 4 * c);
                // (K's scale takes the shift: a large query's keys may be as small as it is large)
                if constexpr (decltype(with_shift)::value) k4.x *= up, k4.y *= up, k4.z *= up, k4.w *= up;
                uint32_t* p = &w[c >> 5][c & 31];
                float y[4];
                f2_unpack(f2_fma(f2_pack(__uint_as_float(p[0]), __uint_as_float(p[1])), f2_pack(k4.x, k4.y), sub2), y[0],
                          y[1]);
                f2_unpack(f2_fma(f2_pack(__uint_as_float(p[2]), __uint_as_float(p[3])), f2_pack(k4.z, k4.w), sub2), y[2],
                          y[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = __float_as_uint(y[e]);
              }
            };
            if (__builtin_expect(!shifted, 1)) scores(std::false_type{});
            else scores(std::true_type{});
            if (masked) {
#pragma unroll
              for (int c = 0; c < 128; ++c)
                if (c >= lim) w[c >> 5][c & 31] = 0xff800000u;
              if (lim < 128) {
                const int quads = max(lim, 0) >> 2;
                vmax = quads > 0 ? ld_shared_u(svmax + st * 128 + 4 * (quads - 1)) & 0x7fffffffu : 0u;
                for (int c = 4 * quads; c < lim; ++c) vmax = max(vmax, kv_finite_bits(ld_shared_u(sV + 4 * c)));
              }
              __syncwarp();
            }
            float mx4[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) mx4[g] = __uint_as_float(w[g][0]);
#pragma unroll
            for (int c = 1; c < 31; c += 2)
#pragma unroll
              for (int g = 0; g < 4; ++g) mx4[g] = max3(mx4[g], __uint_as_float(w[g][c]), __uint_as_float(w[g][c + 1]));
#pragma unroll
            for (int g = 0; g < 4; ++g) mx4[g] = fmaxf(mx4[g], __uint_as_float(w[g][31]));
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            // the first visible scores of a row set its maximum, later ones raise it by what they exceed it; a larger
            // range of V scales raises the reference alone
            const bool fresh = l == 0.f && mx != -INFINITY;
            const bool raise = fresh || mx > top || kv_v_exponent(vmax) > ve;
            if (__any_sync(0xffffffffu, raise)) {
              const int grown = max(ve, kv_v_exponent(vmax));
              const float top_new = kv_v_top(grown);
              const float delta = fresh || mx > top ? mx - (top_new - 8.f) : top - top_new;
              const float alpha = fresh ? 1.f : ex2(-delta);
              m += delta;
              l *= alpha;
#pragma unroll
              for (int c = 0; c < 128; ++c) w[c >> 5][c & 31] = __float_as_uint(__uint_as_float(w[c >> 5][c & 31]) - delta);
              if (j > (L::kSplit ? 1 : 0)) {
                // O_t holds the sum over the earlier tiles (their products completed before S_t(j)), and none is
                // added before P is published
                const float f = alpha * (kv_v_rest(grown) * kv_v_unrest(ve));
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  uint32_t o[16];
                  tmem_ld16_sync(tO + c, o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                  tmem_st16(tO + c, o);
                }
                tmem_st_wait();
              }
              ve = grown;
              top = top_new;
              beyond = __any_sync(0xffffffffu, (l != 0.f || fresh) && kv_v_beyond(ve));
            }
            uint64_t sum2[2] = {0ull, 0ull};
            // P times V's scales in f16 pairs, 64 keys at a time: the product starts on the first half
            auto probabilities = [&](auto with_care) {
              constexpr bool kCare = decltype(with_care)::value;
              const float rest = kCare ? kv_v_rest(ve) : 1.f;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                  uint32_t pk[16];
#pragma unroll
                  for (int c = 0; c < 16; c += 2) {
                    const int c0 = 64 * h + 32 * g + 2 * c;
                    const float4 v4 = ld_shared_f4(sV + 4 * c0);
                    const uint32_t* y = &w[2 * h + g][2 * c];
                    const uint64_t p01 = f2_pack(ex2(__uint_as_float(y[0])), ex2(__uint_as_float(y[1])));
                    const uint64_t p23 = f2_pack(ex2(__uint_as_float(y[2])), ex2(__uint_as_float(y[3])));
                    sum2[0] = f2_add(sum2[0], p01);
                    sum2[1] = f2_add(sum2[1], p23);
                    float q[4];
                    if constexpr (kCare) {
                      const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
                      f2_unpack(p01, q[0], q[1]);
                      f2_unpack(p23, q[2], q[3]);
#pragma unroll
                      for (int e = 0; e < 4; ++e) q[e] = c0 + e < lim ? q[e] * (vs[e] * rest) : 0.f;
                    } else {
                      f2_unpack(f2_mul(p01, f2_pack(v4.x, v4.y)), q[0], q[1]);
                      f2_unpack(f2_mul(p23, f2_pack(v4.z, v4.w)), q[2], q[3]);
                    }
                    pk[c] = pack_f16x2(q[0], q[1]);
                    pk[c + 1] = pack_f16x2(q[2], q[3]);
                  }
                  tmem_st16(tS + 32u * h + 16u * g, pk);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bar_p[2 * t + h]);
              }
            };
            // (a hidden key's p is 0, but its scale may be a NaN or infinite)
            if (__builtin_expect(!(odd || beyond), 1)) probabilities(std::false_type{});
            else probabilities(std::true_type{});
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_sc_empty[st]);
            {
              float s0, s1, s2, s3;
              f2_unpack(sum2[0], s0, s1);
              f2_unpack(sum2[1], s2, s3);
              l += (s0 + s1) + (s2 + s3);
            }
            ++ns;
            ++nsc;
          }
          const bool mine = !L::kSplit || t == 0 || n > 1;  // (a single key tile is all tile 0's)
          if (ok && mine) ok = mbar_wait_warp(&bar_pv[t], (ns - 1) & 1u, ab);
          if (ok && mine) {
            tc_fence_after();
            const bool whole = n == n_item;
            if (part.start == 0 && threadIdx.x == 0)
              kv_record(a, *s_line, s, at, blockIdx.x, s_line->cut(blockIdx.x) + (total - left) - at.from, n_item, whole,
                        left == total);
            const long long piece = (2ll * blockIdx.x + (left == total ? 0 : 1)) * 256 + (L::kSplit ? 0 : t * 128) + r;
            float f = l == 0.f ? 0.f : kv_v_unrest(ve) * kv_code_scale<FMT>() / l;
            float lse2 = l == 0.f ? -INFINITY : m - kKvPShift + log2f(l);
            float f1 = 0.f;
            if (L::kSplit && n > 1) {
              // tile 1 leaves its factor and logsumexp in the lanes of its scores, which nothing overwrites before tile
              // 0 has loaded the next Q
              if (t == 1) {
                tmem_st2(tS, __float_as_uint(f), __float_as_uint(lse2));
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_half);
              } else if ((ok = mbar_wait_warp(bar_half, nhalf & 1u, ab))) {
                tc_fence_after();
                uint32_t w0, w1;
                tmem_ld2_sync(tS + 128u, w0, w1);
                const float l1 = __uint_as_float(w1), mx = fmaxf(lse2, l1);
                const float a0 = kv_weight(lse2, mx), a1 = kv_weight(l1, mx), sum = a0 + a1;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                f *= a0 * inv;
                f1 = __uint_as_float(w0) * (a1 * inv);
                lse2 = sum == 0.f ? -INFINITY : mx + log2f(sum);
              }
              ++nhalf;
            }
#pragma unroll 1
            for (int c = 0; c < D && ok && (!L::kSplit || t == 0); c += 16) {
              uint32_t o[16];
              tmem_ld16_sync(tO + c, o);
              float v[16];
#pragma unroll
              for (int k = 0; k < 16; ++k)  // columns 1 and 2 of each four change places
                v[(k & ~3) | ((k & 1) << 1) | ((k >> 1) & 1)] = __uint_as_float(o[k]) * f;
              if (L::kSplit && n > 1) {
                tmem_ld16_sync(tO + D + c, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  float& y = v[(k & ~3) | ((k & 1) << 1) | ((k >> 1) & 1)];
                  y = fmaf(__uint_as_float(o[k]), f1, y);
                }
              }
              if (x.token >= 0) kv_put_row<D, 16>(a, x, whole, piece, 2ll * gridDim.x * 256, c, v, lse2);
            }
            tc_fence_before();
          }
        }
        left -= part.take;
        if (left > 0 && !kv_next<false>(a, s, at)) break;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // the suffix may run beside the prefix; its completion, which the merge waits for, has to mean both
  if (a.phase == kKvSuffix) pdl_wait();
}

}  // namespace fa
