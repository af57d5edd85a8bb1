// fa_kvcache.cu -- host side of the quantised key/value cache and of the
// attention over it (fa_kv_append, fa_kv_read, fa_fwd_kvcache): argument
// checks, the choice of kernel, tensor maps and launches on the caller's
// stream.  Allocates nothing; what it keeps is, per kernel and
// device, that its shared-memory limit has been raised.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstring>

#include "../../include/fa.h"
#include "host.h"
#include "kvcache_sm100.cuh"
#include "kvnarrow_sm100.cuh"
#include "kvwide_sm100.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool tok_strides_ok(const fa_strides& s) {
  return s.h >= 0 && s.n >= 0 && (s.h * 2) % 16 == 0 && (s.n * 2) % 16 == 0;
}

size_t round_up(size_t x, size_t m) { return (x + m - 1) / m * m; }

int page_shift(int page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
  }
}

// The cache's own checks (sizes first, so that a bad size is refused before a pointer is looked at).
int check_cache(const fa_kv_cache* c) {
  if (!c) return FA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_kv_heads < 1) return FA_ERR_INVALID_ARG;
  if (page_shift(c->page_size) < 0) return FA_ERR_INVALID_ARG;
  if (c->format != FA_KV_INT8 && c->format != FA_KV_FP8) return FA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  // rows are addressed by a 32-bit tile coordinate
  if (c->num_kv_heads > (1 << 16) || (long long)c->num_pages * c->num_kv_heads * c->page_size > 0x7fffffffll)
    return FA_ERR_TOO_LARGE;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return FA_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return FA_ERR_ALIGNMENT;
  return FA_OK;
}

// Block table and batch: FA_OK, a negative status, or 1 for nothing to do.
int check_batch(const int32_t* table, int max_pages, int64_t table_stride, int B, int total) {
  if (B < 0 || total < 0 || max_pages < 0) return FA_ERR_INVALID_ARG;
  if (B == 0 || total == 0) return 1;
  if (B > (1 << 24) || total > (1 << 30)) return FA_ERR_TOO_LARGE;
  if (max_pages < 1 || !table || (B > 1 && table_stride < max_pages)) return FA_ERR_INVALID_ARG;
  if (!aligned(table, 4)) return FA_ERR_ALIGNMENT;
  return FA_OK;
}

void fill_cache(fa::KvArgs* a, const fa_kv_cache* c) {
  std::memset(a, 0, sizeof(*a));
  a->k = static_cast<uint8_t*>(c->k);
  a->v = static_cast<uint8_t*>(c->v);
  a->ks = c->k_scale;
  a->vs = c->v_scale;
  a->num_pages = c->num_pages;
  a->page_shift = page_shift(c->page_size);
  a->Hkv = c->num_kv_heads;
}

// fa_kv_append and fa_kv_read: everything but the kernel.
int rows_setup(const fa_kv_cache* c, const void* k, const void* v, const fa_strides* strides, const int32_t* table,
               int max_pages, int64_t table_stride, const int32_t* starts, const int32_t* cu_seqlens, int B, int total,
               fa::KvArgs* a) {
  int rc = check_cache(c);
  if (rc != FA_OK) return rc;
  if ((rc = check_batch(table, max_pages, table_stride, B, total)) != FA_OK) return rc;
  if (!cu_seqlens && total != B) return FA_ERR_INVALID_ARG;
  if (!k || !v || !strides) return FA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(starts, 4) || !aligned(cu_seqlens, 4)) return FA_ERR_ALIGNMENT;
  if (!tok_strides_ok(strides[0]) || !tok_strides_ok(strides[1])) return FA_ERR_ALIGNMENT;
  fill_cache(a, c);
  a->table = table;
  a->max_pages = max_pages;
  a->table_stride = table_stride;
  a->lens = starts;
  a->cu = cu_seqlens;
  a->B = B;
  a->total = total;
  a->xk = static_cast<__nv_bfloat16*>(const_cast<void*>(k));
  a->xv = static_cast<__nv_bfloat16*>(const_cast<void*>(v));
  a->xk_sn = strides[0].n;
  a->xk_sh = strides[0].h;
  a->xv_sn = strides[1].n;
  a->xv_sh = strides[1].h;
  a->err = fa_host::device_error_ptr();
  return a->err ? FA_OK : fa_host::cuda_fail(cudaErrorInvalidSymbol);
}

template <int D>
int launch_rows(const fa::KvArgs& a, int format, bool append, cudaStream_t st) {
  const int rows = fa::kv_rows_per_warp<D>();
  const long long warps = 2ll * ((a.Hkv + rows - 1) / rows) * a.total;
  if (warps > 0x7fffffffll) return FA_ERR_TOO_LARGE;  // more rows than a cache can have
  const unsigned grid = (unsigned)((warps + 7) / 8);
  if (append) {
    if (format == FA_KV_INT8) fa::kv_append_kernel<D, fa::kKvInt8><<<grid, 256, 0, st>>>(a);
    else fa::kv_append_kernel<D, fa::kKvFp8><<<grid, 256, 0, st>>>(a);
  } else {
    if (format == FA_KV_INT8) fa::kv_read_kernel<D, fa::kKvInt8><<<grid, 256, 0, st>>>(a);
    else fa::kv_read_kernel<D, fa::kKvFp8><<<grid, 256, 0, st>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : fa_host::cuda_fail(e);
}

// Tensor map of the cache's codes as [rows, d] bytes, read in box_rows-row boxes swizzled by the row's width.
int make_code_map(CUtensorMap* m, const void* base, const fa_kv_cache* c, int box_rows) {
  fa_host::EncodeTiledFn enc = fa_host::encode_fn();
  if (!enc) return fa_host::cuda_fail(cudaErrorNotSupported);
  cuuint64_t dims[2] = {(cuuint64_t)c->d, (cuuint64_t)c->num_pages * c->num_kv_heads * c->page_size};
  cuuint64_t strides[1] = {(cuuint64_t)c->d};
  cuuint32_t box[2] = {(cuuint32_t)c->d, (cuuint32_t)box_rows};
  cuuint32_t estride[2] = {1u, 1u};
  const CUresult r =
      enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estride,
          CU_TENSOR_MAP_INTERLEAVE_NONE, c->d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : fa_host::cuda_fail(cudaErrorInvalidValue);
}

// ------------------------------------------------------------- attention

constexpr int kSms = 148;

// Ring depth and CTAs per SM of the narrow kernel: at d = 128 two CTAs of two slices a warp are what shared memory has
// room for beside the merge buffer.
template <int D>
using Narrow = fa::KvNarrowLayout<D, D == 128 ? 2 : 3, D == 128 ? 2 : 3>;

// The kernel for items of `rows` rows: rows per item tile and stretches the work is cut into.
struct Choice {
  int M, G;
  int item_cost;  // starting and ending an item, in units of 128 keys
  bool one_tile;  // wide kernel: at most 128 rows an item
};

Choice choose(long long rows, int d) {
  // Up to 16 rows one mma.sync tile holds an item and the cache's bytes are what is waited for (64 sequences of 512 to
  // 8192 keys, 4 rows an item, int8: 126 us here, 227 in the wide kernel, 279 there as two tiles of rows; fp8 150 and
  // 241).  Above, the wide kernel: a 32-row narrow one spilled, and was slower when it was tried.  With at most 128 rows
  // its two softmax tiles share an item's keys: 64 sequences of drafts of 1 to 5 tokens, 6 heads a group: 149 us, 176 as
  // two tiles of rows of which one is empty.  The rows are those of the longest sequence: a batch of 63 single tokens
  // and one chunk of 512 takes 414 us in one call, 141 and 78 as two.
  if (rows <= 16) return {16, kSms * (d == 128 ? Narrow<128>::kCtasPerSm : Narrow<64>::kCtasPerSm), 2, true};
  return {256, kSms, 3, rows <= 128};
}

// Byte offsets in the workspace: the pieces of one launch and the entries that say where they are.
struct Pieces {
  size_t o, lse, cuts, end;
  int num_cuts;
};

Pieces place_pieces(size_t at, const Choice& c, int d, size_t entries) {
  Pieces p;
  const size_t rows = 2ull * c.G * c.M;
  p.o = at;
  p.lse = p.o + rows * d * 4;
  p.cuts = round_up(p.lse + rows * 4, 256);
  p.end = round_up(p.cuts + entries * sizeof(fa::KvCut), 256);
  p.num_cuts = (int)(entries < 0x7fffffff ? entries : 0x7fffffff);  // for the bounds-checking build
  return p;
}

size_t tiles_of(long long rows, const Choice& c) { return (size_t)((rows + c.M - 1) / c.M); }

// Workspace: the pieces of one launch, or, with a shared prefix, the pieces and result rows of both phases.
struct Layout {
  Choice whole, prefix, suffix;
  Pieces pw, pp, ps;
  long long items;
  bool by_item;
  size_t prefix_o, prefix_lse, suffix_o, suffix_lse, bytes;
};

Layout layout_of(int B, int Hq, int Hkv, int d, int total_q, int max_q, int prefix_len) {
  Layout l;
  std::memset(&l, 0, sizeof(l));
  const int g = Hq / Hkv;
  if (prefix_len == 0) {
    l.whole = choose((long long)max_q * g, d);
    // entries by item while there are fewer items than CTAs, so that the merge has few blocks
    l.items = (long long)B * Hkv * tiles_of((long long)max_q * g, l.whole);
    l.by_item = l.items <= l.whole.G;
    l.pw = place_pieces(0, l.whole, d, l.by_item ? l.items : l.whole.G);
    l.bytes = l.pw.end;
    return l;
  }
  l.prefix = choose((long long)total_q * g, d);
  l.suffix = choose((long long)max_q * g, d);
  l.pp = place_pieces(0, l.prefix, d, Hkv * tiles_of((long long)total_q * g, l.prefix));
  l.ps = place_pieces(l.pp.end, l.suffix, d, (size_t)B * Hkv * tiles_of((long long)max_q * g, l.suffix));
  const size_t rows = (size_t)total_q * Hq;
  l.prefix_o = l.ps.end;
  l.suffix_o = l.prefix_o + rows * d * 4;
  l.prefix_lse = l.suffix_o + rows * d * 4;
  l.suffix_lse = l.prefix_lse + rows * 4;
  l.bytes = l.suffix_lse + rows * 4;
  return l;
}

// Launch on st; `beside` lets the kernel be scheduled while its predecessor still runs (it then waits for the
// predecessor's completion itself, where it needs it).
template <class... P, class... A>
int launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool beside, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = beside ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : fa_host::cuda_fail(e);
}

// Allow a kernel its dynamic shared memory, once per device (the attribute stays with the device's context).
template <auto kKernel>
int allow_smem(size_t smem) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fa_host::cuda_fail(e);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return FA_OK;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return fa_host::cuda_fail(e);
  done.fetch_or(bit, std::memory_order_relaxed);
  return FA_OK;
}

template <int D, int FMT>
int launch_narrow(const fa_kv_cache* c, const fa::KvArgs& a, const Choice& ch, cudaStream_t st) {
  using L = Narrow<D>;
  constexpr auto kern = fa::kv_narrow_kernel<D, FMT, L>;
  CUtensorMap mk, mv;
  const int box = c->page_size < 32 ? c->page_size : 32;
  int rc;
  if ((rc = make_code_map(&mk, c->k, c, box)) != FA_OK) return rc;
  if ((rc = make_code_map(&mv, c->v, c, box)) != FA_OK) return rc;
  if ((rc = allow_smem<kern>(L::kSmem)) != FA_OK) return rc;
  return launch(kern, dim3(ch.G), 128, L::kSmem, st, a.phase == fa::kKvSuffix, mk, mv, a);
}

template <int D, int FMT, int CW>
int launch_wide(const fa::KvArgs& a, const Choice& ch, cudaStream_t st) {
  using L = fa::KvWideLayout<D, CW>;
  constexpr auto kern = fa::kv_wide_kernel<D, FMT, CW>;
  const int rc = allow_smem<kern>(L::kSmem);
  if (rc != FA_OK) return rc;
  return launch(kern, dim3(ch.G), L::kThreads, L::kSmem, st, a.phase == fa::kKvSuffix, a);
}

template <int D, int FMT>
int launch_phase_as(const fa_kv_cache* c, const fa::KvArgs& a, const Choice& ch, cudaStream_t st) {
  if (ch.M == 16) return launch_narrow<D, FMT>(c, a, ch, st);
  return ch.one_tile ? launch_wide<D, FMT, 8>(a, ch, st) : launch_wide<D, FMT, 4>(a, ch, st);
}

int launch_phase(const fa_kv_cache* c, const fa::KvArgs& a, const Choice& ch, cudaStream_t st) {
  if (c->d == 128)
    return c->format == FA_KV_INT8 ? launch_phase_as<128, fa::kKvInt8>(c, a, ch, st)
                                   : launch_phase_as<128, fa::kKvFp8>(c, a, ch, st);
  return c->format == FA_KV_INT8 ? launch_phase_as<64, fa::kKvInt8>(c, a, ch, st)
                                 : launch_phase_as<64, fa::kKvFp8>(c, a, ch, st);
}

int launch_merge_cut(const fa::KvArgs& a, int d, const Layout& l, cudaStream_t st) {
  // few items: a block for each row of one, which may be in many pieces; many: a block per eight rows
  const int M = l.whole.M;
  const dim3 grid((unsigned)(l.by_item ? l.items : l.whole.G), (unsigned)(l.items <= 64 && M < 64 ? M : M / 8));
  return d == 64 ? launch(fa::kv_merge_cut_kernel<64>, grid, fa::kKvMergeThreads, 0, st, true, a)
                 : launch(fa::kv_merge_cut_kernel<128>, grid, fa::kKvMergeThreads, 0, st, true, a);
}

int launch_merge_prefix(const fa::KvArgs& pf, const fa::KvArgs& sf, int d, const Choice& cp, cudaStream_t st) {
  // a prefix of few items is in many pieces a row: then a block merges one row
  const size_t items = pf.Hkv * tiles_of((long long)pf.total * pf.g, cp);
  const int group = (size_t)cp.G > 8 * items ? fa::kKvMergeThreads / 32 : 1;
  const size_t per = fa::kKvMergeThreads / 32 / group, rows = (size_t)sf.total * sf.Hq;
  const dim3 grid((unsigned)((rows + per - 1) / per));
  return d == 64 ? launch(fa::kv_merge_prefix_kernel<64>, grid, fa::kKvMergeThreads, 0, st, true, pf, sf, group)
                 : launch(fa::kv_merge_prefix_kernel<128>, grid, fa::kKvMergeThreads, 0, st, true, pf, sf, group);
}

// Checks of sizes that fa_fwd_kvcache and its workspace size share: FA_OK, a negative status, or 1 for nothing to do.
int check_attend(int B, int Hq, int Hkv, int d, int total_q, int max_q, int prefix_len) {
  if (B < 0 || Hq < 0 || total_q < 0 || max_q < 0 || prefix_len < 0) return FA_ERR_INVALID_ARG;
  if (Hkv < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (B == 0 || Hq == 0 || total_q == 0 || max_q == 0) return 1;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (Hq > (1 << 16) || B > (1 << 24) || total_q > (1 << 24) || max_q > (1 << 24)) return FA_ERR_TOO_LARGE;
  if ((long long)total_q * Hq > 0x7fff0000ll) return FA_ERR_TOO_LARGE;  // row numbers are 32-bit
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_kv_append(const fa_kv_cache* cache, const void* k, const void* v, const fa_strides* strides,
                 const int32_t* block_table, int max_pages, int64_t table_stride, const int32_t* starts,
                 const int32_t* cu_seqlens, int B, int total_tokens, void* stream) {
  fa::KvArgs a;
  const int rc = rows_setup(cache, k, v, strides, block_table, max_pages, table_stride, starts, cu_seqlens, B,
                            total_tokens, &a);
  if (rc != FA_OK) return rc == 1 ? FA_OK : rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cache->d == 64 ? launch_rows<64>(a, cache->format, true, st) : launch_rows<128>(a, cache->format, true, st);
}

int fa_kv_read(const fa_kv_cache* cache, void* k, void* v, const fa_strides* strides, const int32_t* block_table,
               int max_pages, int64_t table_stride, const int32_t* starts, const int32_t* cu_seqlens, int B,
               int total_tokens, void* stream) {
  fa::KvArgs a;
  const int rc = rows_setup(cache, k, v, strides, block_table, max_pages, table_stride, starts, cu_seqlens, B,
                            total_tokens, &a);
  if (rc != FA_OK) return rc == 1 ? FA_OK : rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cache->d == 64 ? launch_rows<64>(a, cache->format, false, st) : launch_rows<128>(a, cache->format, false, st);
}

size_t fa_fwd_kvcache_workspace_size(int B, int Hq, int Hkv, int d, int total_q, int max_q, int prefix_len) {
  if (check_attend(B, Hq, Hkv, d, total_q, max_q, prefix_len) != FA_OK) return 0;
  return layout_of(B, Hq, Hkv, d, total_q, max_q < total_q ? max_q : total_q, B > 1 ? prefix_len : 0).bytes;
}

int fa_fwd_kvcache(const void* q, void* o, float* lse, const fa_strides* strides, const fa_kv_cache* cache,
                   const int32_t* block_table, int max_pages, int64_t table_stride, const int32_t* seqlens,
                   const int32_t* cu_seqlens_q, int B, int Hq, int total_q, int max_q, float scale, int causal,
                   int prefix_len, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_cache(cache);
  if (rc != FA_OK) return rc;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  const int Hkv = cache->num_kv_heads, d = cache->d;
  rc = check_attend(B, Hq, Hkv, d, total_q, max_q, prefix_len);
  // without offsets max_q has to give total_q, also where it is 0
  if (rc >= 0 && !cu_seqlens_q && B > 0 && Hq > 0 && total_q > 0 && (long long)B * max_q != total_q)
    return FA_ERR_INVALID_ARG;
  if (rc != FA_OK) return rc == 1 ? FA_OK : rc;
  if ((rc = check_batch(block_table, max_pages, table_stride, B, total_q)) != FA_OK) return rc;
  if (prefix_len % cache->page_size != 0 || (long long)prefix_len > (long long)max_pages * cache->page_size)
    return FA_ERR_INVALID_ARG;
  if (!q || !o || !strides || !seqlens) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(seqlens, 4) || !aligned(cu_seqlens_q, 4))
    return FA_ERR_ALIGNMENT;
  if (!tok_strides_ok(strides[0]) || !tok_strides_ok(strides[1])) return FA_ERR_ALIGNMENT;
  if (B == 1) prefix_len = 0;  // nothing is shared
  if (max_q > total_q) max_q = total_q;
  const Layout l = layout_of(B, Hq, Hkv, d, total_q, max_q, prefix_len);
  if (!workspace || workspace_bytes < l.bytes) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return FA_ERR_ALIGNMENT;
  char* ws = static_cast<char*>(workspace);

  fa::KvArgs a;
  fill_cache(&a, cache);
  a.table = block_table;
  a.max_pages = max_pages;
  a.table_stride = table_stride;
  a.lens = seqlens;
  a.cu = cu_seqlens_q;
  a.B = B;
  a.total = total_q;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.q_sn = strides[0].n;
  a.q_sh = strides[0].h;
  a.o_sn = strides[1].n;
  a.o_sh = strides[1].h;
  a.lse = lse;
  a.Hq = Hq;
  a.g = Hq / Hkv;
  a.max_q = max_q;
  a.causal = causal;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.prefix_len = prefix_len;
  a.err = fa_host::device_error_ptr();
  if (!a.err) return fa_host::cuda_fail(cudaErrorInvalidSymbol);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (prefix_len == 0) {
    a.phase = fa::kKvWhole;
    a.by_item = l.by_item;
    a.M = l.whole.M;
    a.G = l.whole.G;
    a.item_cost = l.whole.item_cost;
    a.part_o = reinterpret_cast<float*>(ws + l.pw.o);
    a.part_lse = reinterpret_cast<float*>(ws + l.pw.lse);
    a.cuts = reinterpret_cast<fa::KvCut*>(ws + l.pw.cuts);
    a.num_cuts = l.pw.num_cuts;
    if ((rc = launch_phase(cache, a, l.whole, st)) != FA_OK) return rc;
    return launch_merge_cut(a, d, l, st);
  }
  fa::KvArgs pf = a, sf = a;
  pf.phase = fa::kKvPrefix;
  pf.by_item = 1;
  pf.M = l.prefix.M;
  pf.G = l.prefix.G;
  pf.item_cost = l.prefix.item_cost;
  pf.part_o = reinterpret_cast<float*>(ws + l.pp.o);
  pf.part_lse = reinterpret_cast<float*>(ws + l.pp.lse);
  pf.cuts = reinterpret_cast<fa::KvCut*>(ws + l.pp.cuts);
  pf.num_cuts = l.pp.num_cuts;
  pf.row_o = reinterpret_cast<float*>(ws + l.prefix_o);
  pf.row_lse = reinterpret_cast<float*>(ws + l.prefix_lse);
  sf.phase = fa::kKvSuffix;
  sf.by_item = 1;
  sf.M = l.suffix.M;
  sf.G = l.suffix.G;
  sf.item_cost = l.suffix.item_cost;
  sf.part_o = reinterpret_cast<float*>(ws + l.ps.o);
  sf.part_lse = reinterpret_cast<float*>(ws + l.ps.lse);
  sf.cuts = reinterpret_cast<fa::KvCut*>(ws + l.ps.cuts);
  sf.num_cuts = l.ps.num_cuts;
  sf.row_o = reinterpret_cast<float*>(ws + l.suffix_o);
  sf.row_lse = reinterpret_cast<float*>(ws + l.suffix_lse);
  if ((rc = launch_phase(cache, pf, l.prefix, st)) != FA_OK) return rc;
  if ((rc = launch_phase(cache, sf, l.suffix, st)) != FA_OK) return rc;
  return launch_merge_prefix(pf, sf, d, l.prefix, st);
}

}  // extern "C"
