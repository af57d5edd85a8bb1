// kvcache_sm100.cuh -- the quantised, paged key/value cache: writing it,
// reading it back, and how attention over it is cut into work.
//
// Cache: pages [num_pages, Hkv, page_size, d] of 8-bit codes for K and for V
// and one fp32 scale per (page, head, slot).  A row x of d values is stored as
//   int8: scale = amax / 127, code = rint(127 x / amax)
//   fp8:  scale = amax / 448, code = e4m3(448 x / amax)
// (round half to even), amax = max |x|, and stands for code * scale.  The
// position p of sequence b sits in page block_table[b][p / page_size], slot
// p % page_size.
#pragma once

#include "debug_check.cuh"
#include "sm100.cuh"

namespace fa {

enum : int { kKvInt8 = 0, kKvFp8 = 1 };
constexpr int kDevBadPage = 5;  // a page number outside the cache, or a position past the block table

struct KvArgs {
  // the cache
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int num_pages, page_shift, Hkv;
  // the sequences
  const int* table;  // [B][max_pages], rows table_stride apart
  long long table_stride;
  int max_pages;
  const int* cu;    // token offsets [B + 1] of q (attention) or of the rows (append, read); may be null
  const int* lens;  // keys per sequence (attention) or first position (append, read; may be null)
  int B, total;     // sequences; rows of the token-major tensors
  int* err;
  // append, read: token-major K and V rows
  __nv_bfloat16* xk;
  __nv_bfloat16* xv;
  long long xk_sn, xk_sh, xv_sn, xv_sh;
  // attention
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  long long q_sn, q_sh, o_sn, o_sh;
  float* lse;  // [Hq, total] natural log; may be null
  int Hq, g;   // query heads; query heads per key head
  int max_q;   // largest number of query rows of a sequence
  int causal;
  float scale_log2;  // scale * log2(e)
  int M, G;          // rows of an item tile; CTAs of the launch
  int item_cost;     // what starting and ending an item takes, in units of work
  int prefix_len;    // keys [0, prefix_len) are the batch's shared prefix (0: none)
  int phase;         // kKvWhole: all keys; kKvPrefix: the shared ones; kKvSuffix: the rest
  // pieces of items that several CTAs share: slot 2 c + s of CTA c
  float* part_o;    // [2 G][M][D], normalised
  float* part_lse;  // [2 G][M], base 2
  // whole results of a phase, merged afterwards (phases other than kKvWhole)
  float* row_o;      // [total * Hq][D], normalised
  float* row_lse;    // [total * Hq], base 2
  struct KvCut* cuts;  // where the pieces are
  int by_item;
  int num_cuts;        // entries that cuts has room for
};

// An item's pieces: `first`, then every second one from `next` on, n in all; n = 1 is a finished item.  The entries go
// by item, or (by_item = 0, kKvWhole only) by CTA, CTA c's being the item that c starts and does not finish (n = 0:
// none).  In the phases other than kKvWhole a finished item's rows are in row_o and row_lse.
struct KvCut {
  int n, first, next, h, rt;
  int row0, lq;  // the sequence's rows
  int pad;
};

enum : int { kKvWhole = 0, kKvPrefix = 1, kKvSuffix = 2 };

// The sequence that owns token t: the last b with cu[b] <= t, by a 32-ary search of one warp (every lane
// gets the result; every probe lies in [0, B], whatever cu holds).
__device__ __forceinline__ int kv_find_seq(const int* cu, int B, int t, int lane) {
  int lo = 0, n = B;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const bool le = at < n && __ldg(cu + lo + at) <= t;
    const int hits = __popc(__ballot_sync(0xffffffffu, le));
    const int skip = hits > 0 ? (hits - 1) * step : 0;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo;
}

// The same for a token of each lane (all lanes call it): 32 samples of cu go round by shuffles, what is left is searched
// in memory.
__device__ __forceinline__ int kv_find_seq_lanes(const int* cu, int B, int t, int lane) {
  const int step = (B + 31) >> 5;  // >= 1; sample i is cu[i * step]
  const int mine = lane * step < B ? __ldg(cu + lane * step) : 0x7fffffff;
  int i = 0;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const int v = __shfl_sync(0xffffffffu, mine, (i + s) & 31);
    if (i + s < 32 && v <= t) i += s;
  }
  int lo = i * step, hi = min(lo + step, B);
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Row of the cache's [page, head, slot] grid that holds position pos of sequence b and head 0, or -1 (and a
// device error) where the block table has no such page.  Head h is h << page_shift rows further on.
__device__ __forceinline__ int kv_row(const KvArgs& a, int b, long long pos, bool report) {
  const long long pi = pos >> a.page_shift;
  int page = -1;
  if (pos >= 0 && pi < a.max_pages) page = __ldg(a.table + b * a.table_stride + pi);
  if (page < 0 || page >= a.num_pages) {
    if (report && a.err) atomicCAS(a.err, kDevOk, kDevBadPage);
    return -1;
  }
  return ((page * a.Hkv) << a.page_shift) + (int)(pos & ((1 << a.page_shift) - 1));  // rows are fewer than 2^31
}

// x / y for x >= 0, y > 0; almost always of 32-bit numbers, whose division is several times shorter.
__device__ __forceinline__ long long kv_div(long long x, long long y) {
  if (((x | y) >> 32) == 0) return (long long)((uint32_t)x / (uint32_t)y);
  return x / y;
}

// Programmatic dependent launch: allow the next kernel of the stream to be scheduled, and wait for the previous one's
// completion (both do nothing in launches without the attribute).
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// --------------------------------------------------------------- rounding

// y rounded to 20 significant bits.  The exact quotient top * x / amax of bf16
// numbers is either on a border between two codes (a dyadic number of few
// bits) or further than 2^-16 of its value away from one: with 8-bit integers
// X, A and a border of M / 2^n, M < 2^8, |top X 2^i - M A| is a whole number of
// units of which M A is at most 2^16.  y carries a relative error below 2^-21 (a
// reciprocal good to an ulp, two rounded products), so this rounding puts every
// border case exactly on its border and moves nothing across one: the code that
// follows is the exact quotient's, half to even, without a division.  The
// rounding is Veltkamp's splitting, p = (2^4 + 1) y, p - (p - y), on both halves
// of a packed pair (integer operations on the bits are fewer, but go to the
// pipe that bounds the kernel); in this order a zero keeps its sign.
__device__ __forceinline__ uint64_t kv_snap2(uint64_t y) {
  const uint64_t p = f2_mul(y, f2_pack(17.f, 17.f));
  const uint64_t minus = f2_pack(-1.f, -1.f);
  return f2_fma(f2_fma(y, minus, p), minus, p);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The codes of two packed pairs of quotients.
template <int FMT>
__device__ __forceinline__ uint32_t kv_encode4(uint64_t y01, uint64_t y23) {
  float a, b, c, d;
  if constexpr (FMT == kKvInt8) {
    // adding 1.5 * 2^23 rounds half to even and leaves the two's complement
    // of the whole number in the low byte
    const uint64_t magic = f2_pack(12582912.f, 12582912.f);
    f2_unpack(f2_add(kv_snap2(y01), magic), a, b);
    f2_unpack(f2_add(kv_snap2(y23), magic), c, d);
    return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                       __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
  } else {
    f2_unpack(kv_snap2(y01), a, b);
    f2_unpack(kv_snap2(y23), c, d);
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
}

// The codes of a word times scale2 = (scale, scale), as four bf16.
template <int FMT>
__device__ __forceinline__ uint2 kv_decode4(uint32_t w, uint64_t scale2) {
  uint64_t x01, x23;
  if constexpr (FMT == kKvInt8) {
    const uint32_t u = w ^ 0x80808080u;  // code + 128 in each byte
    // 2^23 + byte as a float, minus 2^23 + 128
    const uint64_t bias = f2_pack(-8388736.f, -8388736.f);
    x01 = f2_add(f2_pack(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)),
                         __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441))), bias);
    x23 = f2_add(f2_pack(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)),
                         __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443))), bias);
  } else {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(w & 0xffffu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
    const float2 p = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 q = __half22float2(*reinterpret_cast<__half2*>(&hi));
    x01 = f2_pack(p.x, p.y);
    x23 = f2_pack(q.x, q.y);
  }
  // (not f2_mul, which flushes the scales of the smallest rows)
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x01) : "l"(x01), "l"(scale2));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x23) : "l"(x23), "l"(scale2));
  float a, b, c, d;
  f2_unpack(x01, a, b);
  f2_unpack(x23, c, d);
  return make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

// ----------------------------------------------------------- append, read

// Append and read share their decomposition.  A cache row of d codes is the
// work of d / 8 lanes, 16 bytes of bf16 against 8 bytes of codes each, so one
// warp moves 32 / (d / 8) rows at a time and kKvUnroll times that in all, every
// load ahead of every store.  A warp's rows are heads of one token's keys or of
// its values.  Reading back is bound by memory, appending by instruction issue
// (61298 tokens, 16 heads, d = 128, fp8, 761 MB each way: append 158 us, the issue
// slots 83 % taken; read 117 us, the rate of a copy).
constexpr int kKvUnroll = 4;

template <int D>
__host__ __device__ constexpr int kv_rows_per_warp() { return 32 / (D / 8) * kKvUnroll; }

// A warp's token, tensor and heads, and where its sequence keeps them.
struct KvMove {
  int t, h0;       // token; this lane's first head; t < 0: nothing to do
  bool value;      // V instead of K
};

template <int D>
__device__ __forceinline__ KvMove kv_move(const KvArgs& a, int lane) {
  const uint32_t per = (uint32_t)(a.Hkv + kv_rows_per_warp<D>() - 1) / (uint32_t)kv_rows_per_warp<D>();
  const uint32_t w = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const uint32_t tv = w / per;  // 2 token + (0: keys, 1: values)
  KvMove m;
  m.t = (int)(tv >> 1);
  m.value = (tv & 1u) != 0u;
  m.h0 = (int)(w - tv * per) * kv_rows_per_warp<D>() + lane / (D / 8);
  if (m.t >= a.total) m.t = -1;
  return m;
}

// The cache row of head 0 of token t, or -1: a row of no sequence, or (and a device error) one without a page.
__device__ __forceinline__ int kv_place_token(const KvArgs& a, int t, int lane, bool* in_sequence) {
  int b = t, first = t, end = t + 1;
  if (a.cu) {
    b = kv_find_seq(a.cu, a.B, t, lane);
    first = __ldg(a.cu + b);
    end = __ldg(a.cu + b + 1);
  }
  *in_sequence = t >= first && t < end;
  if (!*in_sequence) return -1;
  return kv_row(a, b, (long long)(a.lens ? __ldg(a.lens + b) : 0) + (t - first), lane == 0);
}

template <int D, int FMT>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  constexpr float kTop = FMT == kKvInt8 ? 127.f : 448.f;
  constexpr uint32_t kTinyBits = (127u - 100u) << 7;  // 2^-100 as a bf16
  constexpr uint32_t kHugeBits = (127u + 126u) << 7;  // 2^126: above it the reciprocal is subnormal, with fewer bits
  static_assert(kKvUnroll % 2 == 0, "rows go through the shuffles in pairs");
  const int lane = threadIdx.x & 31;
  const int col = (lane % LPR) * 8;
  const KvMove mv = kv_move<D>(a, lane);
  if (mv.t < 0) return;
  const long long sh = mv.value ? a.xv_sh : a.xk_sh;
  const __nv_bfloat16* src = (mv.value ? a.xv + mv.t * a.xv_sn : a.xk + mv.t * a.xk_sn) + mv.h0 * sh + col;
  uint4 x[kKvUnroll];
#pragma unroll
  for (int u = 0; u < kKvUnroll; ++u) {
    x[u] = make_uint4(0u, 0u, 0u, 0u);
    if (mv.h0 + u * RPW < a.Hkv) x[u] = __ldg(reinterpret_cast<const uint4*>(src + u * RPW * sh));
  }
  bool in_sequence;
  const int row = kv_place_token(a, mv.t, lane, &in_sequence);
  if (row < 0) return;
  // the largest |x| of each row as bf16 bits -- as integers infinities and NaN sort above all numbers --, two rows to
  // a word on their way through the shuffles
  uint32_t mb[kKvUnroll];
#pragma unroll
  for (int u = 0; u < kKvUnroll; ++u) {
    const uint32_t m2 = __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu),
                                 __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu));
    mb[u] = max(m2 & 0xffffu, m2 >> 16);
  }
  bool scaled = false;  // some row's largest is below 2^-100, or 2^126 and more
#pragma unroll
  for (int u = 0; u < kKvUnroll; u += 2) {
    uint32_t m2 = mb[u] | (mb[u + 1] << 16);
#pragma unroll
    for (int s = 1; s < LPR; s <<= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, s));
    mb[u] = m2 & 0xffffu;
    mb[u + 1] = m2 >> 16;
    scaled |= mb[u] - kTinyBits >= kHugeBits - kTinyBits || mb[u + 1] - kTinyBits >= kHugeBits - kTinyBits;
  }
  scaled = __any_sync(0xffffffffu, scaled);
  const int at0 = row + (mv.h0 << a.page_shift), step = RPW << a.page_shift;
  uint8_t* dst = (mv.value ? a.v : a.k) + (long long)at0 * D + col;
  float* dst_scale = (mv.value ? a.vs : a.ks) + at0;
#pragma unroll
  for (int u = 0; u < kKvUnroll; ++u) {
    const float amax = __uint_as_float(mb[u] << 16);
    // top / amax to an ulp or two (the codes ask for no more), and amax / top by one step of Newton's division on
    // the rounded reciprocal of top: the residual fma is exact, so the quotient is correctly rounded.  A row with an
    // infinity or a NaN gets a NaN scale; its codes mean nothing.
    float inv = kTop * rcp_approx(amax);
    const float s0 = amax * (1.f / kTop);
    float scale = fmaf(fmaf(-kTop, s0, amax), 1.f / kTop, s0);
    if (mb[u] >= 0x7f80u) scale = __uint_as_float(0x7fc00000u);
    const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
    uint64_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = f2_pack(bf16_lo(xs[i]), bf16_hi(xs[i]));
    if (scaled) {
      // rows below 2^-100 go up by 2^100 and rows of 2^126 and more down by it, so that nothing leaves fp32's normal
      // range (of a large row entries do that are far too small for a code); a row of zeros keeps scale 0
      const bool t = mb[u] < kTinyBits, h = mb[u] >= kHugeBits;
      const float lift = t ? 1.2676506002282294e30f : h ? 7.888609052210118e-31f : 1.f;
      if (t || h) inv = mb[u] != 0u ? __fdiv_rn(kTop, amax * lift) : 0.f;
      if (t) scale = __fdiv_rn(amax, kTop);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = f2_pack(bf16_lo(xs[i]) * lift, bf16_hi(xs[i]) * lift);
    }
    const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = f2_mul(y[i], inv2);
    const uint32_t c0 = kv_encode4<FMT>(y[0], y[1]), c1 = kv_encode4<FMT>(y[2], y[3]);
    if (mv.h0 + u * RPW < a.Hkv &&
        FA_IN(kSiteKvRow, (long long)at0 + u * step, 1, ((long long)a.num_pages * a.Hkv) << a.page_shift, a.err)) {
      *reinterpret_cast<uint2*>(dst + (long long)u * step * D) = make_uint2(c0, c1);
      if (lane % LPR == 0) dst_scale[u * step] = scale;
    }
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const int col = (lane % LPR) * 8;
  const KvMove mv = kv_move<D>(a, lane);
  if (mv.t < 0) return;
  bool in_sequence;
  const int row = kv_place_token(a, mv.t, lane, &in_sequence);
  if (!in_sequence) return;  // a row of no sequence: left as it was
  const int at0 = row + (mv.h0 << a.page_shift), step = RPW << a.page_shift;
  const uint8_t* src = (mv.value ? a.v : a.k) + (long long)at0 * D + col;
  const float* src_scale = (mv.value ? a.vs : a.ks) + at0;
  uint2 c[kKvUnroll];
  float sc[kKvUnroll];
#pragma unroll
  for (int u = 0; u < kKvUnroll; ++u) {
    c[u] = make_uint2(0u, 0u);
    sc[u] = 0.f;
    if (row >= 0 && mv.h0 + u * RPW < a.Hkv &&
        FA_IN(kSiteKvRow, (long long)at0 + u * step, 1, ((long long)a.num_pages * a.Hkv) << a.page_shift, a.err)) {
      c[u] = __ldg(reinterpret_cast<const uint2*>(src + (long long)u * step * D));
      sc[u] = __ldg(src_scale + u * step);
    }
  }
  const long long sh = mv.value ? a.xv_sh : a.xk_sh;
  __nv_bfloat16* dst = (mv.value ? a.xv + mv.t * a.xv_sn : a.xk + mv.t * a.xk_sn) + mv.h0 * sh + col;
#pragma unroll
  for (int u = 0; u < kKvUnroll; ++u) {
    if (mv.h0 + u * RPW >= a.Hkv) continue;
    const uint64_t s2 = f2_pack(sc[u], sc[u]);
    const uint2 x = kv_decode4<FMT>(c[u].x, s2), y = kv_decode4<FMT>(c[u].y, s2);
    st_global_v4(dst + u * RPW * sh, x.x, x.y, y.x, y.y);
  }
}

// ------------------------------------------------------- work of attention
//
// An item is the rows of one sequence and key head -- its query tokens times
// the g query heads of the group, in tiles of M rows -- against the keys they
// see; its work is counted in units of kKvUnit keys.  The units of all items,
// sequence by sequence, head by head, tile by tile, form one line that the G
// CTAs of the grid cut into equal stretches, whatever the lengths: the cut is
// computed on the device from the lengths, so a captured launch follows them.
// Each item counts item_cost units more than its keys, ahead of them, for what
// starting and ending it takes: without them the CTAs with many short items are
// the last (64 sequences of 512 to 8192 keys, 8 key heads: 127 us with them, 145
// without; with drafts of 1 to 5 tokens over 4 key heads 148 and 176).
// An item inside one stretch is finished by its CTA; an item that is cut
// leaves a normalised piece and its logsumexp per CTA, merged afterwards.  A
// CTA has at most two such pieces, of its first and of its last item.
constexpr int kKvUnit = 128;

struct KvSeq {
  int row0, lq, lk;  // first query row, query rows, keys
};

__device__ __forceinline__ KvSeq kv_seq(const KvArgs& a, int b, bool report) {
  KvSeq s;
  if (a.phase == kKvPrefix) {  // the whole batch as one sequence over the shared keys
    s.row0 = 0;
    s.lq = a.total;
    s.lk = a.prefix_len;
    return s;
  }
  if (a.cu) {
    const SeqSpan sp = varlen_span(a.cu, nullptr, b, a.total, a.max_q, a.err, report);
    s.row0 = sp.row0;
    s.lq = sp.len;
  } else {
    s.row0 = b * a.max_q;
    s.lq = a.max_q;
  }
  const int L = __ldg(a.lens + b);
  const long long cap = min((long long)a.max_pages << a.page_shift, 0x7fffffffll - kKvUnit);
  s.lk = (int)min((long long)max(L, 0), cap);
  if (report && (L < 0 || L > cap) && a.err) atomicCAS(a.err, kDevOk, kDevBadSeqlens);
  return s;
}

// keys that query i (within its sequence) sees: [0, kv_end)
__device__ __forceinline__ int kv_end(const KvArgs& a, const KvSeq& s, int i) {
  if (a.phase == kKvPrefix) return s.lk;
  return a.causal ? min(max(s.lk - s.lq + i + 1, 0), s.lk) : s.lk;
}

__device__ __forceinline__ int kv_begin(const KvArgs& a) { return a.phase == kKvSuffix ? a.prefix_len : 0; }

// In the functions below ONE says that every sequence's rows fit in one tile (the narrow kernel): most of the
// arithmetic, divisions above all, then falls away, and with it a good part of a short call's time.

// one past the last key that some row of tile rt sees
template <bool ONE>
__device__ __forceinline__ int kv_item_end(const KvArgs& a, const KvSeq& s, int rt) {
  if (ONE) return kv_end(a, s, s.lq - 1);
  // rows of a call are fewer than 2^31, so row numbers stay 32-bit
  const uint32_t last = min((uint32_t)(rt + 1) * (uint32_t)a.M, (uint32_t)s.lq * (uint32_t)a.g) - 1u;
  return kv_end(a, s, (int)(last / (uint32_t)a.g));
}

template <bool ONE>
__device__ __forceinline__ int kv_tiles(const KvArgs& a, const KvSeq& s) {
  if (ONE) return s.lq > 0 ? 1 : 0;
  return (int)(((uint32_t)s.lq * (uint32_t)a.g + (uint32_t)a.M - 1u) / (uint32_t)a.M);
}

template <bool ONE>
__device__ __forceinline__ int kv_item_units(const KvArgs& a, const KvSeq& s, int rt) {
  const int keys = kv_item_end<ONE>(a, s, rt) - kv_begin(a);
  return max(1, (keys + kKvUnit - 1) / kKvUnit);  // an item without keys still writes its rows
}

// length on the line of one key head of the sequence
template <bool ONE>
__device__ __forceinline__ long long kv_head_len(const KvArgs& a, const KvSeq& s) {
  if (s.lq == 0) return 0;
  if (ONE) return kv_item_units<true>(a, s, 0) + a.item_cost;
  const int nt = kv_tiles<false>(a, s);
  if (nt == 1 || !a.causal || a.phase == kKvPrefix)
    return (long long)nt * (kv_item_units<false>(a, s, nt - 1) + a.item_cost);
  long long n = 0;
#pragma unroll 1
  for (int rt = 0; rt < nt; ++rt) n += kv_item_units<false>(a, s, rt) + a.item_cost;
  return n;
}

// What a CTA with `left` of its stretch to go does of an item of n_item units from place `from` of the item on: units
// [start, start + n), which take `take` of the line.  n = 0: its stretch ends before the item's first unit.
struct KvPart {
  int start, n, take;
};

__device__ __forceinline__ KvPart kv_part(const KvArgs& a, int n_item, int from, int left) {
  const int take = min(n_item + a.item_cost - from, left);
  const int start = max(from - a.item_cost, 0);
  return KvPart{start, max(from + take - a.item_cost, 0) - start, take};
}

__device__ __forceinline__ int kv_num_seqs(const KvArgs& a) { return a.phase == kKvPrefix ? 1 : a.B; }

// The line of W units in G stretches -- one per CTA of the grid, or one per unit where there are fewer units than
// CTAs, so that none is empty: the first r stretches have q + 1 units, the others q.
struct KvLine {
  long long q;
  int r, G;
  __device__ __forceinline__ long long cut(int c) const { return q * c + min(c, r); }  // first unit of stretch c
  __device__ __forceinline__ int cta_of(long long u) const {                           // stretch that holds unit u
    const long long wide = (q + 1) * r;
    return u < wide ? (int)kv_div(u, q + 1) : r + (int)kv_div(u - wide, q);
  }
};

// A place on the line: place `from` of the item that is row tile rt of head h of sequence b.
struct KvPlace {
  int b, h, rt, from;
};

// Scratch of kv_place.
struct KvScan {
  long long warp_sum[32];
  long long rem;
  int b;
  KvSeq s;
};

// Inclusive sum over the block (NT threads) and its total.
template <int NT>
__device__ __forceinline__ long long kv_block_inclusive(long long x, KvScan* sc, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  __syncthreads();
  if (lane == 31) sc->warp_sum[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    const long long v = sc->warp_sum[i];
    if (i < warp) before += v;
    all += v;
  }
  *total = all;
  return before + x;
}

// The line of work, and the sequence *s = number *b that holds the first unit of CTA c (and the units before it
// within the sequence), by the whole block; *b < 0 if CTA c has no stretch.
template <bool ONE, int NT>
__device__ __forceinline__ KvLine kv_place(const KvArgs& a, int c, int G, KvScan* sc, int* b, KvSeq* s,
                                           long long* rem) {
  const int n = kv_num_seqs(a);
  KvSeq mine{0, 0, 0};
  auto units_of = [&](int i, bool report) -> long long {
    if (i >= n) return 0;
    mine = kv_seq(a, i, report);
    return kv_head_len<ONE>(a, mine) * a.Hkv;
  };
  KvLine line{0, 0, 0};
  *b = -1;
  *rem = 0;
  long long W = 0, u0 = 0, run = 0, x = 0, incl = 0, tot = 0;
  // first the sum of all sequences' units, then the one that holds this CTA's first (one body for both, so that the
  // kernel's cold start fetches its instructions once; up to NT sequences stay in registers)
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int base = 0; base < n; base += NT) {
      if (pass == 0 || n > NT) {
        x = units_of(base + (int)threadIdx.x, pass == 0 && c == 0);
        incl = kv_block_inclusive<NT>(x, sc, &tot);
      }
      if (pass == 0) {
        W += tot;
        continue;
      }
      const long long lo = run + incl - x;
      if (u0 >= lo && u0 < lo + x) {
        sc->b = base + threadIdx.x;
        sc->rem = u0 - lo;
        sc->s = mine;
      }
      run += tot;
      if (u0 < run) break;
    }
    if (pass == 0) {
      line.G = (int)min((long long)G, W);
      if (W == 0) return line;
      line.q = kv_div(W, line.G);
      line.r = (int)(W - line.q * line.G);
      if (c >= line.G) return line;
      u0 = line.cut(c);
    }
  }
  __syncthreads();
  *b = sc->b;
  *rem = sc->rem;
  *s = sc->s;
  return line;
}

// The place `rem` units into sequence b.
template <bool ONE>
__device__ __forceinline__ KvPlace kv_within(const KvArgs& a, const KvSeq& s, int b, long long rem) {
  KvPlace p;
  p.b = b;
  const long long per = kv_head_len<ONE>(a, s);
  p.h = (int)kv_div(rem, per);
  rem -= p.h * per;
  p.rt = 0;
  p.from = (int)rem;
  if (ONE) return p;
  const int nt = kv_tiles<false>(a, s);
  if (nt > 1 && (!a.causal || a.phase == kKvPrefix)) {
    const int n = kv_item_units<false>(a, s, 0) + a.item_cost;
    p.rt = (int)kv_div(rem, n);
    rem -= (long long)p.rt * n;
  } else {
    for (; p.rt + 1 < nt; ++p.rt) {
      const int n = kv_item_units<false>(a, s, p.rt) + a.item_cost;
      if (rem < n) break;
      rem -= n;
    }
  }
  p.from = (int)rem;
  return p;
}

// The item after p; false at the end of the line.  Updates s when the sequence changes.
template <bool ONE>
__device__ __forceinline__ bool kv_next(const KvArgs& a, KvSeq& s, KvPlace& p) {
  p.from = 0;
  if (!ONE && ++p.rt < kv_tiles<false>(a, s)) return true;
  p.rt = 0;
  if (++p.h < a.Hkv) return true;
  p.h = 0;
  const int n = kv_num_seqs(a);
  while (++p.b < n) {
    s = kv_seq(a, p.b, false);
    if (s.lq > 0) return true;
  }
  return false;
}

// Entry of an item.
__device__ __forceinline__ long long kv_item_index(const KvArgs& a, int b, int h, int rt) {
  const uint32_t rows = (uint32_t)(a.phase == kKvPrefix ? a.total : a.max_q) * (uint32_t)a.g;
  const uint32_t tiles = (rows + (uint32_t)a.M - 1u) / (uint32_t)a.M;  // of the longest sequence
  return ((long long)b * a.Hkv + h) * tiles + rt;
}

// Record where the pieces of the item that starts at w0 of the line are; called by one thread of CTA c, which does its
// first unit (as the first item of its stretch, or a later one).
__device__ __forceinline__ void kv_record(const KvArgs& a, const KvLine& line, const KvSeq& s, const KvPlace& p, int c,
                                          long long w0, int n_item, bool whole, bool first_item) {
  if (whole && !a.by_item) return;
  KvCut k;
  k.n = whole ? 1 : line.cta_of(w0 + a.item_cost + n_item - 1) - c + 1;
  k.first = 2 * c + (first_item ? 0 : 1);
  k.next = 2 * c + 2;
  k.h = p.h, k.rt = p.rt;
  k.row0 = s.row0, k.lq = s.lq;
  k.pad = 0;
  const long long at = a.by_item ? kv_item_index(a, p.b, p.h, p.rt) : c;
  if (FA_IN(kSiteKvCut, at, 1, a.num_cuts, a.err)) a.cuts[at] = k;
}

// Entries that no item will write, before anything else: a CTA's own, or those of tiles that a sequence shorter than
// the longest does not have.
template <bool ONE>
__device__ __forceinline__ void kv_clear_cuts(const KvArgs& a) {
  if (a.phase != kKvWhole) return;  // there every entry that is read has its item
  if (!a.by_item) {
    if (threadIdx.x == 0 && FA_IN(kSiteKvCut, (long long)blockIdx.x, 1, a.num_cuts, a.err)) a.cuts[blockIdx.x].n = 0;
    return;
  }
  if (blockIdx.x != 0) return;
  const int tiles = (int)kv_item_index(a, 0, 1, 0);  // of the longest sequence
#pragma unroll 1
  for (int i = threadIdx.x; i < a.B * a.Hkv; i += blockDim.x) {
    const int b = i / a.Hkv;
    for (int rt = kv_tiles<ONE>(a, kv_seq(a, b, false)); rt < tiles; ++rt) {
      const long long at = kv_item_index(a, b, i - b * a.Hkv, rt);
      if (FA_IN(kSiteKvCut, at, 1, a.num_cuts, a.err)) a.cuts[at].n = 0;
    }
  }
}

// Where a row of an item lives: token, query head, and how many keys it sees.
struct KvRow {
  int token, head, end;
};

__device__ __forceinline__ KvRow kv_token_of(const KvArgs& a, const KvSeq& s, int h, int rt, int r) {
  const uint32_t rr = (uint32_t)rt * (uint32_t)a.M + (uint32_t)r;
  if (rr >= (uint32_t)s.lq * (uint32_t)a.g) return KvRow{-1, 0, 0};
  const int i = (int)(rr / (uint32_t)a.g);
  return KvRow{s.row0 + i, h * a.g + (int)(rr - (uint32_t)i * (uint32_t)a.g), 0};
}

// A row with its reach; every lane of the warp calls it.
__device__ __forceinline__ KvRow kv_row_of(const KvArgs& a, const KvSeq& s, int h, int rt, int r) {
  KvRow x = kv_token_of(a, s, h, rt, r);
  const int i = x.token - s.row0;
  if (a.phase != kKvPrefix) {
    if (x.token >= 0) x.end = kv_end(a, s, i);
    return x;
  }
  // the token's own sequence bounds what it sees of the prefix
  int b, first, lq;
  if (a.cu) {
    b = kv_find_seq_lanes(a.cu, a.B, max(x.token, 0), threadIdx.x & 31);
    const SeqSpan sp = varlen_span(a.cu, nullptr, b, a.total, a.max_q, nullptr, false);
    first = sp.row0;
    lq = sp.len;
  } else {
    b = max(x.token, 0) / a.max_q;
    first = b * a.max_q;
    lq = a.max_q;
  }
  const int at = x.token - first;
  if (x.token < 0 || at < 0 || at >= lq) return KvRow{-1, 0, 0};  // a row of no sequence
  const long long cap = min((long long)a.max_pages << a.page_shift, 0x7fffffffll - kKvUnit);
  const int L = (int)min((long long)max(__ldg(a.lens + b), 0), cap);
  x.end = min(s.lk, a.causal ? max(L - lq + at + 1, 0) : L);
  return x;
}

// Columns [col0, col0 + NC) of a row's normalised result, to where the phase wants it: the output (a finished row
// of a kKvWhole launch), the phase's result rows (a finished row otherwise), or a piece.
template <int D, int NC>
__device__ __forceinline__ void kv_put_row(const KvArgs& a, const KvRow& x, bool whole, long long piece,
                                           long long pieces, int col0, const float (&v)[NC], float lse2) {
  static_assert(NC % 8 == 0, "16-byte stores");
  if (whole && a.phase == kKvWhole) {
    const long long at = x.token * a.o_sn + x.head * a.o_sh;
    if (FA_IN(kSiteKvO, at, D, extent4(1, a.Hq, a.total, D, 0, a.o_sh, a.o_sn), a.err)) {
#pragma unroll
      for (int e = 0; e < NC; e += 8)
        st_global_v4(a.o + at + col0 + e, pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]),
                     pack_bf16x2(v[e + 4], v[e + 5]), pack_bf16x2(v[e + 6], v[e + 7]));
    }
    const long long la = (long long)x.head * a.total + x.token;
    if (col0 == 0 && a.lse && FA_IN(kSiteKvLse, la, 1, (long long)a.Hq * a.total, a.err))
      a.lse[la] = lse2 * 0.69314718055994531f;
    return;
  }
  const long long row = whole ? (long long)x.token * a.Hq + x.head : piece;
  const long long lim = whole ? (long long)a.total * a.Hq : pieces;
  (void)lim;
  if (!FA_IN(whole ? kSiteKvRes : kSiteKvPart, row, 1, lim, a.err)) return;
  float* dst = (whole ? a.row_o : a.part_o) + row * D + col0;
#pragma unroll
  for (int e = 0; e < NC; e += 4) *reinterpret_cast<float4*>(dst + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  if (col0 == 0) (whole ? a.row_lse : a.part_lse)[row] = lse2;
}

// ------------------------------------------------------------------ merge

constexpr int kKvMergeThreads = 256;

template <int D>
__device__ __forceinline__ void kv_axpy(float (&acc)[D / 32], float w, const float* src) {
  if constexpr (D == 128) {
    const float4 v = *reinterpret_cast<const float4*>(src);
    acc[0] += w * v.x, acc[1] += w * v.y, acc[2] += w * v.z, acc[3] += w * v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(src);
    acc[0] += w * v.x, acc[1] += w * v.y;
  }
}

template <int D>
__device__ __forceinline__ void kv_store_row(const KvArgs& a, const KvRow& x, int lane, const float (&v)[D / 32],
                                             float lse2) {
  const long long at = x.token * a.o_sn + x.head * a.o_sh;
  if (FA_IN(kSiteKvO, at, D, extent4(1, a.Hq, a.total, D, 0, a.o_sh, a.o_sn), a.err)) {
    __nv_bfloat16* dst = a.o + at + lane * (D / 32);
    if constexpr (D == 128)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    else
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(v[0], v[1]);
  }
  if (lane == 0 && a.lse &&
      FA_IN(kSiteKvLse, (long long)x.head * a.total + x.token, 1, (long long)a.Hq * a.total, a.err))
    a.lse[(long long)x.head * a.total + x.token] = lse2 * 0.69314718055994531f;
}

// weight of a piece against the largest logsumexp mx of its row (pieces of no keys weigh nothing; NaN stays)
__device__ __forceinline__ float kv_weight(float lse2, float mx) {
  return lse2 == -INFINITY ? 0.f : exp2f(lse2 - mx);
}

// The rows of one row of an item in its pieces (or its finished row): row `first`, then n - 1 rows from `next`,
// `stride` apart.
struct KvPieces {
  const float* o;
  const float* lse;
  int n;
  long long first, next, stride;
  __device__ __forceinline__ long long at(int k) const { return k == 0 ? first : next + (k - 1) * stride; }
};

__device__ __forceinline__ KvPieces kv_pieces(const KvArgs& a, const KvCut& k, int r) {
  return KvPieces{a.part_o, a.part_lse, k.n, (long long)k.first * a.M + r, (long long)k.next * a.M + r, 2ll * a.M};
}

// An entry that can be followed.  Every entry is written by the launch before, unless a wait of it ran out: then the
// workspace's old contents must not lead anywhere.
__device__ __forceinline__ bool kv_cut_ok(const KvArgs& a, const KvCut& k) {
  if (k.n < 1 || k.n > a.G || k.first < 0 || k.first >= 2 * a.G) return false;
  return k.n == 1 || (k.next >= 0 && (long long)k.next + 2ll * (k.n - 2) < 2ll * a.G);
}

// The pieces that an entry names lie within the launch's (the bounds-checking build's check of kv_merge_row's reads).
__device__ __forceinline__ bool kv_pieces_in(const KvArgs& a, const KvPieces& p) {
  return FA_IN(kSiteKvPart, p.at(0), 1, 2ll * a.G * a.M, a.err) && FA_IN(kSiteKvPart, p.at(p.n - 1), 1, 2ll * a.G * a.M, a.err);
}

template <int D>
struct KvMergeSmem {
  float sum[kKvMergeThreads / 32], o[kKvMergeThreads / 32][D];
};

// Merge of the pieces in up to two lists into row x by `group` warps: one, or all of the block (which then all call it
// for the same row):
//   lse = log2 sum_s 2^lse_s,  O = sum_s 2^(lse_s - lse) O_s
template <int D>
__device__ void kv_merge_row(const KvArgs& a, const KvRow& x, const KvPieces& p0, const KvPieces& p1, int group,
                             KvMergeSmem<D>& sm) {
  constexpr int NW = kKvMergeThreads / 32, PER = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int me = group == 1 ? 0 : warp;
  const int n = p0.n + p1.n;
  auto lse_of = [&](int k) { return k < p0.n ? p0.lse[p0.at(k)] : p1.lse[p1.at(k - p0.n)]; };
  // up to 32 logsumexps in the lanes at once, and the warp's first pieces of O on their way with them
  const float held = lane < n ? lse_of(lane) : -INFINITY;
  auto src_of = [&](int k) {
    return (k < p0.n ? p0.o + p0.at(k) * D : p1.o + p1.at(k - p0.n) * D) + lane * PER;
  };
  constexpr int kEarly = 4;
  float early[kEarly][PER];
#pragma unroll
  for (int i = 0; i < kEarly; ++i) {
#pragma unroll
    for (int e = 0; e < PER; ++e) early[i][e] = 0.f;
    if (me + i * group < n) kv_axpy<D>(early[i], 1.f, src_of(me + i * group));
  }
  float mx = held;
  for (int k = 32 + lane; k < n; k += 32) mx = fmaxf(mx, lse_of(k));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  float acc[PER] = {}, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kEarly; ++i) {
    const int k = me + i * group;
    if (k >= n) break;
    const float wt = kv_weight(k < 32 ? __shfl_sync(0xffffffffu, held, k) : lse_of(k), mx);
    sum += wt;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] += wt * early[i][e];
  }
#pragma unroll 4
  for (int k = me + kEarly * group; k < n; k += group) {
    const float wt = kv_weight(k < 32 ? __shfl_sync(0xffffffffu, held, k) : lse_of(k), mx);
    sum += wt;
    kv_axpy<D>(acc, wt, src_of(k));
  }
  if (group > 1) {
#pragma unroll
    for (int e = 0; e < PER; ++e) sm.o[warp][lane * PER + e] = acc[e];
    if (lane == 0) sm.sum[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        sum += sm.sum[i];
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] += sm.o[i][lane * PER + e];
      }
    }
  }
  if (me == 0) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= inv;
    kv_store_row<D>(a, x, lane, acc, sum == 0.f ? -INFINITY : mx + log2f(sum));
  }
  if (group > 1) __syncthreads();
}

// Items that the stretches cut.  The blocks (i, .) merge the item of entry i,
// if it is in pieces: a warp a row, or with more than eight pieces
// the block a row with the pieces spread over its warps (one key head's 64K
// keys leave over a hundred pieces, a chain that one warp would walk alone).
template <int D>
__global__ void __launch_bounds__(kKvMergeThreads) kv_merge_cut_kernel(const KvArgs a) {
  constexpr int NW = kKvMergeThreads / 32;
  __shared__ KvMergeSmem<D> sm;
  const int warp = threadIdx.x >> 5;
  pdl_wait();
  if (!FA_IN(kSiteKvCut, (long long)blockIdx.x, 1, a.num_cuts, a.err)) return;
  const KvCut k = a.cuts[blockIdx.x];
  if (k.n < 2 || !kv_cut_ok(a, k)) return;
  const KvSeq s{k.row0, k.lq, 0};
  const int group = k.n > NW ? NW : 1;
  const int rows = group == 1 ? NW : 1;  // rows a block merges at a time
  for (int r0 = blockIdx.y * rows; r0 < a.M; r0 += gridDim.y * rows) {
    const int r = r0 + (group == 1 ? warp : 0);
    const KvRow x = kv_token_of(a, s, k.h, k.rt, r);
    if (r >= a.M || x.token < 0) continue;
    KvPieces p = kv_pieces(a, k, r), none = p;
    none.n = 0;
    if (!kv_pieces_in(a, p)) continue;
    kv_merge_row<D>(a, x, p, none, group, sm);
  }
}

// Shared prefix: every row's result over the prefix (pf: phase kKvPrefix) and over its own keys (sf: kKvSuffix),
// each finished or in pieces; `group` warps a row.
template <int D>
__global__ void __launch_bounds__(kKvMergeThreads) kv_merge_prefix_kernel(const KvArgs pf, const KvArgs sf, int group) {
  constexpr int NW = kKvMergeThreads / 32;
  __shared__ KvMergeSmem<D> sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = NW / group;  // rows a block merges at a time
  const uint32_t rows = (uint32_t)sf.total * (uint32_t)sf.Hq;
  const uint32_t row = blockIdx.x * (uint32_t)per + (group == 1 ? warp : 0);
  if (row >= rows) return;  // (one warp, or the whole block)
  const int t = (int)(row / (uint32_t)sf.Hq), head = (int)(row - (uint32_t)t * (uint32_t)sf.Hq);
  const int h = head / sf.g;
  const int b = sf.cu ? kv_find_seq(sf.cu, sf.B, t, lane) : t / sf.max_q;
  const KvSeq ss = kv_seq(sf, b, false);
  const int i = t - ss.row0;
  const uint32_t rp = (uint32_t)t * (uint32_t)pf.g + (uint32_t)(head - h * pf.g);
  const uint32_t rs = (uint32_t)max(i, 0) * (uint32_t)sf.g + (uint32_t)(head - h * sf.g);
  const uint32_t tp = rp / (uint32_t)pf.M, ts = rs / (uint32_t)sf.M;
  pdl_wait();
  if (i < 0 || i >= ss.lq) return;  // a row of no sequence
  const long long ip = kv_item_index(pf, 0, h, (int)tp), is = kv_item_index(sf, b, h, (int)ts);
  if (!FA_IN(kSiteKvCut, ip, 1, pf.num_cuts, pf.err) || !FA_IN(kSiteKvCut, is, 1, sf.num_cuts, sf.err)) return;
  const KvCut kp = pf.cuts[ip], ks = sf.cuts[is];
  if (!kv_cut_ok(pf, kp) || !kv_cut_ok(sf, ks)) return;
  KvPieces p0 = kv_pieces(pf, kp, (int)(rp - tp * (uint32_t)pf.M));
  KvPieces p1 = kv_pieces(sf, ks, (int)(rs - ts * (uint32_t)sf.M));
  if (!kv_pieces_in(pf, p0) || !kv_pieces_in(sf, p1)) return;
  if (!FA_IN(kSiteKvRes, (long long)row, 1, (long long)sf.total * sf.Hq, sf.err)) return;
  if (kp.n == 1) p0.o = pf.row_o, p0.lse = pf.row_lse, p0.first = row;
  if (ks.n == 1) p1.o = sf.row_o, p1.lse = sf.row_lse, p1.first = row;
  kv_merge_row<D>(sf, KvRow{t, head, 0}, p0, p1, group, sm);
}

}  // namespace fa
