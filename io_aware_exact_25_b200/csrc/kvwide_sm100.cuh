// kvwide_sm100.cuh -- attention of many rows over the quantised cache: a
// prompt's chunk, or a whole batch's queries over its shared prefix.
//
// An item tile is 256 rows (query tokens x heads of one key head's group) as
// two 128-row tiles, the shape of the dense forward (fwd_sm100.cuh): tcgen05
// MMAs S_t = Q_t K^T and O_t += P_t V accumulate in tensor memory, one softmax
// thread per row, the two tiles taking turns on the tensor core.  What differs
// is where K and V come from.  Warp roles:
//   warps 0-3   softmax of tile 0 (they also load their rows of Q)
//   warps 4-7   softmax of tile 1
//   warps 8-11  converter: codes from the cache's pages to f16 operand tiles
//   warp  12    MMA issue (one thread); warps 13-15 complete its warpgroup
// The converter threads load 16 codes at a time straight from the pages (one
// tile ahead in registers, so the loads overlap the conversion), unpack them
// exactly as the narrow kernel does and write the f16 tile in the 128-byte
// swizzled layout the MMA reads: 256 rows share one conversion, under half an
// instruction per code and row tile.  Inside each group of four the columns
// stand in the order 0, 2, 1, 3, in which the codes unpack; Q is stored the
// same way and O's columns are put back on the way out.
//
// Scales as in the narrow kernel: K's multiply the fp32 scores and V's, as
// ratios to a running power of two, the probabilities.  The converter keeps
// that power and publishes both scale vectors per tile of 128 keys.
//
// The exponentials (one per score on the MUFU unit, 16 a clock) and the MMAs
// (two of 128 x 128 x d per tile) take the same time at d = 128, 1024 clocks
// a 128-row tile, so neither is far from its limit when the other is.
#pragma once

#include "kvnarrow_sm100.cuh"

namespace fa {

template <int D>
struct KvWideLayout {
  static constexpr int kM = 256;
  static constexpr int kThreads = 512;
  // launched at 128 registers a thread: 2 x 128 x 184 + 128 x 104 + 128 x 40 = 512 x 128
  static constexpr uint32_t kRegsSoftmax = 184, kRegsConvert = 104, kRegsCtl = 40;
  static_assert(2 * kRegsSoftmax + kRegsConvert + kRegsCtl <= 4 * 128, "register split");
  static constexpr uint32_t kHalf = 128u * 128u;    // 128 rows x 64 f16 columns
  static constexpr uint32_t kTile = 128u * D * 2u;  // 128 x D f16
  static constexpr int kStages = D == 128 ? 5 : 8;  // K/V operand ring
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffKV = 2 * kTile;
  static constexpr uint32_t kOffScale = kOffKV + kStages * kTile;  // 2 stages of 128 K scales, 128 V ratios
  static constexpr uint32_t kOffMisc = kOffScale + 2 * 1024;       // [2] {V power, V NaN flag}, [2][4] warp maxima
  static constexpr uint32_t kOffBar = kOffMisc + 2 * 8 + 8 * 4;
  static constexpr int kNumBars = 2 + 2 * kStages + 2 + 2 + 2 + 2 + 2 + 2 + 1 + 1;
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

__device__ __forceinline__ void st_shared_f(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

template <int D, int FMT>
__global__ void __launch_bounds__(512, 1) kv_wide_kernel(const KvArgs a) {
  using L = KvWideLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* bar_q = bars;                              // [2] Q_t written (128 arrivals)
  uint64_t* bar_kv_full = bars + 2;                    // [S] operand tile written (128)
  uint64_t* bar_kv_empty = bar_kv_full + L::kStages;   // [S] operand tile consumed
  uint64_t* bar_s = bar_kv_empty + L::kStages;         // [2] S_t ready
  uint64_t* bar_p = bar_s + 2;                         // [2] P_t written (128)
  uint64_t* bar_pv = bar_p + 2;                        // [2] O_t += P_t V done
  uint64_t* bar_p_half = bar_pv + 2;                   // [2] first half of P_t written (128)
  uint64_t* bar_sc_full = bar_p_half + 2;              // [2] scales of a key tile written (128)
  uint64_t* bar_sc_empty = bar_sc_full + 2;            // [2] scales consumed (8 warps)
  uint64_t* bar_drain = bar_sc_empty + 2;              //     every MMA retired
  uint64_t* bar_vmax = bar_drain + 1;                  //     the converter warps' V maxima written (4 warps)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_vmax + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sscale = sbase + L::kOffScale, smisc = sbase + L::kOffMisc;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar_q[t], 128);
      mbar_init(&bar_s[t], 1);
      mbar_init(&bar_p[t], 128);
      mbar_init(&bar_pv[t], 1);
      mbar_init(&bar_p_half[t], 128);
      mbar_init(&bar_sc_full[t], 128);
      mbar_init(&bar_sc_empty[t], 8);
    }
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&bar_kv_full[i], 128);
      mbar_init(&bar_kv_empty[i], 1);
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_vmax, 4);
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
  const KvLine line =
      kv_place<512>(a, blockIdx.x, gridDim.x, reinterpret_cast<KvScan*>(smem + L::kOffScan), &b, &rem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Abort ab{abort_flag, a.err};
  const bool run = b >= 0 && *abort_flag == 0;
  if (a.phase == kKvWhole && threadIdx.x == 0) a.cuts[blockIdx.x].n = 0;  // until this CTA leaves an item unfinished
  const long long u0 = b >= 0 ? line.cut(blockIdx.x) : 0, u1 = b >= 0 ? line.cut(blockIdx.x + 1) : 0;
  const int begin = kv_begin(a);
  KvSeq s{0, 0, 0};
  KvPlace at{0, 0, 0, 0};
  if (run) {
    s = kv_seq(a, b, false);
    at = kv_within(a, s, b, rem);
  }
  // Every role walks the same items: n units of the item at `at`, from key `first` on; act1 if the second row tile
  // has rows.
  auto act1_of = [&]() { return (uint32_t)at.rt * 256u + 128u < (uint32_t)s.lq * (uint32_t)a.g; };

  if (warp >= 12) {
    regs_dec<L::kRegsCtl>();
    if (run && warp == 12 && lane == 0) {
      // ------------------------------------------------------ MMA issue
      // Order for key tile j: O0 += P0 V(j-1), S0(j), O1 += P1 V(j-1), S1(j), as in the dense forward: S_t(j)
      // overwrites the columns of P_t(j-1) behind the product that reads them, and a completed S_t(j) implies that
      // O_t holds every earlier product.
      constexpr uint32_t kIdS = idesc_f16(128, 128, false);
      constexpr uint32_t kIdO = idesc_f16(128, D, true);
      uint32_t pos = 0;             // operand ring position: K(j) then V(j), over all items
      uint32_t nq[2] = {0, 0};      // items of each row tile so far
      uint32_t np[2] = {0, 0};      // P tiles of each row tile so far
      bool ok = true, issued = false;
      auto full = [&](uint32_t p) { return mbar_wait(&bar_kv_full[p % L::kStages], (p / L::kStages) & 1u, ab); };
      auto tile_of = [&](uint32_t p) { return sbase + L::kOffKV + (p % L::kStages) * L::kTile; };
      auto issue_s = [&](int t, uint32_t sK) {
        const uint32_t sQ = sbase + L::kOffQ + t * L::kTile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + 128u * t, desc_kmajor(sQ, kk, L::kHalf), desc_kmajor(sK, kk, L::kHalf), kIdS, kk > 0 ? 1u : 0u);
        mma_commit(&bar_s[t]);
        issued = true;
      };
      auto issue_pv = [&](int t, bool first, uint32_t sV) -> bool {
        const uint32_t ph = np[t]++ & 1u;
        if (!mbar_wait(&bar_p_half[t], ph, ab)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts(tmem + L::kColO + D * t, tmem + 128u * t + 8u * kk, desc_mnmajor(sV, kk, L::kHalf), kIdO,
                 (!first || kk > 0) ? 1u : 0u);
        if (!mbar_wait(&bar_p[t], ph, ab)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 4; kk < 8; ++kk)
          mma_ts(tmem + L::kColO + D * t, tmem + 128u * t + 8u * kk, desc_mnmajor(sV, kk, L::kHalf), kIdO, 1u);
        mma_commit(&bar_pv[t]);
        return true;
      };
      for (long long u = u0; u < u1 && ok;) {
        const int n = (int)min((long long)(kv_item_units(a, s, at.rt) - at.unit), u1 - u);
        const int nt = act1_of() ? 2 : 1;
        for (int t = 0; t < nt && ok; ++t) ok = mbar_wait(&bar_q[t], nq[t]++ & 1u, ab);
        for (int j = 0; j <= n && ok; ++j) {
          // tiles in hand: K(j) at pos + 2 j, V(j - 1) at pos + 2 j - 1
          const uint32_t pk = pos + 2u * j, pv = pk - 1u;
          if (j > 0 && !(ok = full(pv))) break;
          if (j < n && !(ok = full(pk))) break;
          tc_fence_after();
          for (int t = 0; t < nt && ok; ++t) {
            if (j > 0) ok = issue_pv(t, j == 1, tile_of(pv));
            if (ok && j < n) issue_s(t, tile_of(pk));
          }
          if (!ok) break;
          if (j > 0) mma_commit(&bar_kv_empty[pv % L::kStages]);
          if (j < n) mma_commit(&bar_kv_empty[pk % L::kStages]);
        }
        pos += 2u * n;
        u += n;
        if (u < u1 && !kv_next(a, s, at)) break;
      }
      if (issued) {
        mma_commit(bar_drain);
        mbar_wait_drain(bar_drain, 0);
      }
    }
  } else if (warp >= 8) {
    regs_dec<L::kRegsConvert>();
    if (run) {
      // ------------------------------------------------------ converter
      constexpr int CH = D / 16;        // 16-code chunks of a row
      constexpr int RP = 128 / CH;      // rows the 128 threads cover in one pass
      constexpr int NP = 128 / RP;      // passes of a tile
      const int tid = threadIdx.x - 256;
      const int cw = warp - 8;
      const int ch = tid % CH, r_in = tid / CH;
      // the chunk's place in row r of the operand tile: 16 f16 columns are two 16-byte chunks of the 64-column half
      // ch / 4; lanes of the upper half write the second one first, so that eight lanes cover all banks
      const uint32_t half_off = (uint32_t)(ch >> 2) * L::kHalf;
      const int c0 = 2 * (ch & 3);
      const int swap = D == 128 ? (ch >> 2) & 1 : r_in & 1;
      uint32_t pos = 0, nsc = 0;
      bool ok = true;
      for (long long u = u0; u < u1 && ok;) {
        const int n = (int)min((long long)(kv_item_units(a, s, at.rt) - at.unit), u1 - u);
        const int item_end = kv_item_end(a, s, at.rt);
        const int first = begin + at.unit * kKvUnit;
        const int* trow = a.table + (a.phase == kKvPrefix ? 0ll : at.b * a.table_stride);
        float vpower = 1.1754943508222875e-38f;
        // lane l < 8 of each warp: cache row of the first of keys 16 l .. 16 l + 15 of a tile; -1 past the keys
        auto fetch_rows = [&](int j) -> int {
          const int key = first + j * kKvUnit + 16 * (lane & 7);
          if (j >= n || key >= item_end) return -1;
          int page = __ldg(trow + (key >> a.page_shift));
          if (page < 0 || page >= a.num_pages) {
            if (a.err) atomicCAS(a.err, kDevOk, kDevBadPage);
            page = 0;
          }
          const long long row = (((long long)page * a.Hkv + at.h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
          return FA_IN(kSiteKvRow, row, 16, ((long long)a.num_pages * a.Hkv) << a.page_shift, a.err) ? (int)row : -1;
        };
        auto load_tile = [&](const uint8_t* codes, int rows, uint4 (&raw)[NP]) {
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const int r = i * RP + r_in;  // row of the tile; its group of 16 is the same for the whole warp
            const int base = __shfl_sync(0xffffffffu, rows, r >> 4);
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (base >= 0) raw[i] = __ldg(reinterpret_cast<const uint4*>(codes + ((long long)base + (r & 15)) * D) + ch);
          }
        };
        auto store_tile = [&](const uint4 (&raw)[NP]) -> bool {
          const uint32_t st = pos % L::kStages;
          if (!mbar_wait_warp(&bar_kv_empty[st], ((pos / L::kStages) & 1u) ^ 1u, ab)) return false;
          const uint32_t tile = sbase + L::kOffKV + st * L::kTile + half_off;
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const int r = i * RP + r_in;
            uint32_t e[4], o[4];
            kv_unpack<FMT>(raw[i].x, e[0], o[0]);
            kv_unpack<FMT>(raw[i].y, e[1], o[1]);
            kv_unpack<FMT>(raw[i].z, e[2], o[2]);
            kv_unpack<FMT>(raw[i].w, e[3], o[3]);
            const uint32_t row = tile + r * 128;
            const uint32_t a0 = row + (((c0 + swap) ^ (r & 7)) << 4), a1 = row + (((c0 + 1 - swap) ^ (r & 7)) << 4);
            if (swap) {
              st_shared_v4(a0, e[2], o[2], e[3], o[3]);
              st_shared_v4(a1, e[0], o[0], e[1], o[1]);
            } else {
              st_shared_v4(a0, e[0], o[0], e[1], o[1]);
              st_shared_v4(a1, e[2], o[2], e[3], o[3]);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&bar_kv_full[st]);
          ++pos;
          return true;
        };
        auto load_scale = [&](const float* sc, int rows) -> float {
          const int base = __shfl_sync(0xffffffffu, rows, tid >> 4);
          return base >= 0 ? __ldg(sc + base + (tid & 15)) : 0.f;
        };
        uint4 rk[NP], rv[NP];
        int rows = fetch_rows(0);
        load_tile(a.k, rows, rk);
        load_tile(a.v, rows, rv);
        float ks = load_scale(a.ks, rows), vs = load_scale(a.vs, rows);
        for (int j = 0; j < n; ++j) {
          const int next = fetch_rows(j + 1);
          // scales of this tile
          const bool in = first + j * kKvUnit + tid < item_end;
          uint32_t vb = __float_as_uint(vs) & 0x7fffffffu;
          const bool vnan = in && vb > 0x7f800000u;
          if (!in || vb >= 0x7f800000u) vb = 0u;
          const uint32_t wmax = __reduce_max_sync(0xffffffffu, vb);
          const bool wnan = __any_sync(0xffffffffu, vnan);
          // the four warps' maxima meet (a bounded wait, so that an aborting CTA cannot strand a warp at a barrier)
          const uint32_t red = smisc + 16 + (nsc & 1u) * 16;
          if (lane == 0) {
            st_shared_f(red + 4 * cw, __uint_as_float(wmax | (wnan ? 0x80000000u : 0u)));
            mbar_arrive(bar_vmax);
          }
          if (!(ok = mbar_wait_warp(bar_vmax, nsc & 1u, ab))) break;
          const float4 m4 = ld_shared_f4(red);
          const uint32_t mb[4] = {__float_as_uint(m4.x), __float_as_uint(m4.y), __float_as_uint(m4.z), __float_as_uint(m4.w)};
          uint32_t vmax = 0u, anynan = 0u;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            vmax = max(vmax, mb[i] & 0x7fffffffu);
            anynan |= mb[i] & 0x80000000u;
          }
          if (vmax > __float_as_uint(vpower))
            vpower = __uint_as_float(min((vmax & 0x7f800000u) + 0x00800000u, 0x7e800000u));
          const float vinv = __uint_as_float((254u << 23) - __float_as_uint(vpower));
          const uint32_t st = nsc & 1u;
          if (!(ok = mbar_wait_warp(&bar_sc_empty[st], ((nsc >> 1) & 1u) ^ 1u, ab))) break;
          st_shared_f(sscale + st * 1024 + 4 * tid, in ? ks : 0.f);
          st_shared_f(sscale + st * 1024 + 512 + 4 * tid, in ? vs * vinv : 0.f);
          if (tid == 0) {
            st_shared_f(smisc + st * 8, vpower);
            st_shared_f(smisc + st * 8 + 4, anynan ? 1.f : 0.f);
          }
          mbar_arrive(&bar_sc_full[st]);
          ++nsc;
          // the next tile's loads go out behind each conversion
          if (!(ok = store_tile(rk))) break;
          load_tile(a.k, next, rk);
          ks = load_scale(a.ks, next);
          vs = load_scale(a.vs, next);
          if (!(ok = store_tile(rv))) break;
          load_tile(a.v, next, rv);
        }
        u += n;
        if (u < u1 && !kv_next(a, s, at)) break;
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
      bool ok = true;
      for (long long u = u0; u < u1 && ok;) {
        const int n_item = kv_item_units(a, s, at.rt);
        const int n = (int)min((long long)(n_item - at.unit), u1 - u);
        const int first = begin + at.unit * kKvUnit;
        if (t == 1 && !act1_of()) {
          // no rows here: only release the scales
          for (int j = 0; j < n && ok; ++j, ++nsc) {
            ok = mbar_wait_warp(&bar_sc_full[nsc & 1u], (nsc >> 1) & 1u, ab);
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&bar_sc_empty[nsc & 1u]);
          }
        } else {
          const KvRow x = kv_row_of(a, s, at.h, at.rt, t * 128 + r);
          float qs = 0.f;
          {
            // this thread's row of Q as f16 times 2^-e, columns in the order the codes unpack
            const long long qo = x.token * a.q_sn + x.head * a.q_sh;
            const bool in =
                x.token >= 0 && FA_IN(kSiteKvQ, qo, D, extent4(1, a.Hq, a.total, D, 0, a.q_sh, a.q_sn), a.err);
            const uint4* src = reinterpret_cast<const uint4*>(a.q + (in ? qo : 0));
            uint4 w[D / 8];
            uint32_t m2 = 0u;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              w[c] = in ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu),
                                         __vmaxu2(w[c].z & 0x7fff7fffu, w[c].w & 0x7fff7fffu)));
            float down, up;
            kv_q_shift(__uint_as_float(max(m2 & 0xffffu, m2 >> 16) << 16), down, up);
            qs = up * a.scale_log2 * kv_code_scale<FMT>();
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
          float m = -INFINITY, l = 0.f, vpower = 0.f;
          for (int j = 0; j < n; ++j) {
            const uint32_t st = nsc & 1u;
            if (!(ok = mbar_wait_warp(&bar_sc_full[st], (nsc >> 1) & 1u, ab))) break;
            if (!(ok = mbar_wait_warp(&bar_s[t], ns & 1u, ab))) break;
            tc_fence_after();
            const uint32_t sK = sscale + st * 1024, sV = sK + 512;
            const float vp = ld_shared_f(smisc + st * 8);
            const bool vnan = ld_shared_f(smisc + st * 8 + 4) != 0.f;
            uint32_t w[4][32];
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) tmem_ld32(tS + 32u * c4, w[c4]);
            tmem_ld_wait();
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) reg_fence(w[c4]);
            // scores times K scales
            auto scale_k = [&]() {
#pragma unroll
              for (int c = 0; c < 128; c += 4) {
                const float4 k4 = ld_shared_f4(sK + 4 * c);
                uint32_t* p = &w[c >> 5][c & 31];
                float y[4];
                f2_unpack(f2_mul(f2_pack(__uint_as_float(p[0]), __uint_as_float(p[1])), f2_pack(k4.x, k4.y)), y[0], y[1]);
                f2_unpack(f2_mul(f2_pack(__uint_as_float(p[2]), __uint_as_float(p[3])), f2_pack(k4.z, k4.w)), y[2], y[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = __float_as_uint(y[e]);
              }
            };
            scale_k();
            const int lim = x.end - (first + j * kKvUnit);  // keys below it are visible
            const bool masked = __any_sync(0xffffffffu, lim < 128);
            if (masked) {
#pragma unroll
              for (int c = 0; c < 128; ++c)
                if (c >= lim) w[c >> 5][c & 31] = 0xff800000u;
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
            const float m_new = fmaxf(m, fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * qs);
            if (__any_sync(0xffffffffu, m_new > m + 8.f) || vp != vpower) {
              const float alpha = m_new == -INFINITY ? 1.f : ex2(m - m_new);
              l *= alpha;
              m = m_new;
              if (j > 0) {
                // O_t holds the sum over the earlier tiles (their products completed before S_t(j)); the score
                // registers are released for the rescale and read again after it
                const float f = alpha * vpower * __uint_as_float((254u << 23) - __float_as_uint(vp));
#pragma unroll
                for (int c4 = 0; c4 < D / 32; ++c4) {
                  uint32_t o[32];
                  tmem_ld32_sync(tO + 32u * c4, o);
#pragma unroll
                  for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                  tmem_st32(tO + 32u * c4, o);
                }
                tmem_st_wait();
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4) tmem_ld32(tS + 32u * c4, w[c4]);
                tmem_ld_wait();
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4) reg_fence(w[c4]);
                scale_k();
                if (masked) {
#pragma unroll
                  for (int c = 0; c < 128; ++c)
                    if (c >= lim) w[c >> 5][c & 31] = 0xff800000u;
                }
              }
              vpower = vp;
            }
            const float sub = (m == -INFINITY ? 0.f : m) - kKvPShift;
            const uint64_t mul2 = f2_pack(qs, qs), sub2 = f2_pack(-sub, -sub);
            uint64_t sum2[2] = {0ull, 0ull};
            // P in f16 pairs, 64 keys at a time; the product starts on the first half
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pk[32];
#pragma unroll
              for (int c = 0; c < 64; c += 4) {
                const float4 v4 = ld_shared_f4(sV + 4 * (64 * h + c));
                const uint32_t* p = &w[(64 * h + c) >> 5][c & 31];
                float x0, x1, p0, p1, p2, p3;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(p[0]), __uint_as_float(p[1])), mul2, sub2), x0, x1);
                p0 = ex2(x0), p1 = ex2(x1);
                f2_unpack(f2_fma(f2_pack(__uint_as_float(p[2]), __uint_as_float(p[3])), mul2, sub2), x0, x1);
                p2 = ex2(x0), p3 = ex2(x1);
                const uint64_t q0 = f2_pack(p0, p1), q1 = f2_pack(p2, p3);
                sum2[0] = f2_add(sum2[0], q0);
                sum2[1] = f2_add(sum2[1], q1);
                f2_unpack(f2_mul(q0, f2_pack(v4.x, v4.y)), p0, p1);
                f2_unpack(f2_mul(q1, f2_pack(v4.z, v4.w)), p2, p3);
                pk[c / 2] = pack_f16x2(p0, p1);
                pk[c / 2 + 1] = pack_f16x2(p2, p3);
              }
              if (masked && vnan) {
                // a NaN V scale times the zero probability of a hidden key
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  if (64 * h + 2 * c >= lim) pk[c] = 0u;
                  else if (64 * h + 2 * c + 1 >= lim) pk[c] &= 0xffffu;
                }
              }
              tmem_st32(tS + 32u * h, pk);
              tmem_st_wait();
              tc_fence_before();
              mbar_arrive(h == 0 ? &bar_p_half[t] : &bar_p[t]);
            }
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
          if (ok) ok = mbar_wait_warp(&bar_pv[t], (ns - 1) & 1u, ab);
          if (ok) {
            tc_fence_after();
            const bool whole = at.unit == 0 && n == n_item;
            if (at.unit == 0 && threadIdx.x == 0) kv_record(a, line, at, blockIdx.x, u, n_item, whole, u == u0);
            const long long piece = (2ll * blockIdx.x + (u == u0 ? 0 : 1)) * 256 + t * 128 + r;
            const float f = l == 0.f ? 0.f : vpower * kv_code_scale<FMT>() / l;
            const float lse2 = l == 0.f ? -INFINITY : m - kKvPShift + log2f(l);
#pragma unroll
            for (int c4 = 0; c4 < D / 32; ++c4) {
              uint32_t o[32];
              tmem_ld32_sync(tO + 32u * c4, o);
              float v[32];
#pragma unroll
              for (int k = 0; k < 32; ++k)  // columns 1 and 2 of each four change places
                v[(k & ~3) | ((k & 1) << 1) | ((k >> 1) & 1)] = __uint_as_float(o[k]) * f;
              if (x.token >= 0) kv_put_row<D, 32>(a, x, whole, piece, 2ll * gridDim.x * 256, 32 * c4, v, lse2);
            }
            tc_fence_before();
          }
        }
        u += n;
        if (u < u1 && !kv_next(a, s, at)) break;
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
