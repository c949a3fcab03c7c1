// hylra_paged.cu - C ABI entry points of the paged-cache calls (see include/hylra.h).
//
// Host side only: argument validation, TMA descriptor encoding and launches.
// The kernels live in hylra_paged.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "hylra.h"
#include "hylra_host.h"
#include "hylra_paged.cuh"

using namespace hylra;
using namespace hylra::paged;

namespace {

constexpr size_t kSmemMax = 232448;  // 227 KB of dynamic shared memory per CTA
constexpr size_t kSmemSM = 233472;   // 228 KB of shared memory per SM, 1 KB of it per CTA reserved
// the largest table: 16384 pages of 16 tokens over eight CTAs, 8 heads
static_assert(sizeof(SelectSmem) + 8 * 2048 * 8 + 16384 * 4 <= kSmemMax &&
                  sizeof(SelectSmem) + sizeof(RankSmem) + 16384 * 4 <= kSmemMax,
              "select kernel shared memory");
constexpr int kCtasPerSM = 3;        // of the decode kernel, at most

// The status word, the tables' ticket and the partial results.  The dense calls may use
// the same memory in turn: they need the tickets that follow their status word to be
// zero, 4 bytes for each 4160 or more of their partials, so in a workspace of `bytes`
// these end before byte 256 + bytes / 1024, and the partials here begin after it.
struct PagedLayout {
  size_t ticket, partial_bytes, total;
  int G;  // CTAs of the decode kernel, at most
  size_t partials(size_t bytes) const { return (256 + bytes / 1024 + 255) / 256 * 256; }
};

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int current_device(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
    return HYLRA_ERR_CUDA;
  return HYLRA_OK;
}

// Partial slots are sized for the larger head dimension: one workspace serves
// every shape.
PagedLayout make_layout(int sms) {
  PagedLayout L{};
  L.G = std::min(kCtasPerSM * sms, MAX_GRID);
  L.ticket = 128;
  L.partial_bytes = (size_t)2 * L.G * DecodeShape<128>::SLOT * sizeof(float);
  // partials(bytes) + partial_bytes <= bytes from here on: 512 + bytes / 1024 + them
  L.total = (L.partial_bytes + 512 + (L.partial_bytes + 512) / 1023 + 511) / 256 * 256;
  return L;
}

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

int check_paged(const hylra_paged_t* s) {
  if (!s) return HYLRA_ERR_INVALID;
  if (s->batch < 1 || s->num_q_heads < 1 || s->num_kv_heads < 1 || s->num_pages < 1 ||
      s->max_pages < 1)
    return HYLRA_ERR_INVALID;
  if (s->dtype != HYLRA_BF16 && s->dtype != HYLRA_FP16)
    return s->dtype == HYLRA_FP32 ? HYLRA_ERR_UNSUPPORTED : HYLRA_ERR_INVALID;
  if (s->num_q_heads % s->num_kv_heads != 0) return HYLRA_ERR_INVALID;
  if (!(s->softmax_scale >= 0.f) || !std::isfinite(s->softmax_scale)) return HYLRA_ERR_INVALID;
  if (s->head_dim != 64 && s->head_dim != 128) return HYLRA_ERR_UNSUPPORTED;
  if (s->page_size != 16 && s->page_size != 32 && s->page_size != 64 && s->page_size != 128)
    return HYLRA_ERR_UNSUPPORTED;
  if (s->num_q_heads / s->num_kv_heads > HYLRA_MAX_GROUP || s->batch > HYLRA_MAX_BATCH)
    return HYLRA_ERR_UNSUPPORTED;
  if ((long long)s->num_pages * s->page_size > INT_MAX) return HYLRA_ERR_UNSUPPORTED;
  if ((long long)s->max_pages * s->page_size > HYLRA_MAX_SEQLEN) return HYLRA_ERR_UNSUPPORTED;
  const long long units = ((long long)s->max_pages * s->page_size + 63) / 64;
  if (s->num_kv_heads > INT_MAX / HYLRA_MAX_GROUP / HYLRA_MAX_BATCH ||
      (long long)s->batch * s->num_kv_heads * units > INT_MAX / 4)
    return HYLRA_ERR_UNSUPPORTED;
  return HYLRA_OK;
}

// Strides of the pool: rows of d elements at (page, head, row) must not overlap.
int check_pool(const hylra_paged_t* s) {
  struct Dim {
    int64_t stride, extent;
  } dim[3] = {{s->token_stride, s->page_size},
              {s->head_stride, s->num_kv_heads},
              {s->page_stride, s->num_pages}};
  for (const Dim& x : dim) {
    if (x.extent == 1) continue;  // never used
    if (x.stride < 0 || x.stride % 8 != 0) return HYLRA_ERR_INVALID;
    if (x.stride >= (int64_t(1) << 39)) return HYLRA_ERR_UNSUPPORTED;
  }
  std::sort(dim, dim + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t span = s->head_dim;  // elements covered by the dimensions so far
  for (const Dim& x : dim) {
    if (x.extent == 1) continue;
    if (x.stride < span) return HYLRA_ERR_INVALID;
    if (x.extent - 1 > ((int64_t(1) << 46) - span) / x.stride) return HYLRA_ERR_UNSUPPORTED;
    span += x.stride * (x.extent - 1);
  }
  return HYLRA_OK;
}

int check_workspace(const void* ws, size_t bytes, const PagedLayout& L) {
  if (!ws || !aligned(ws, 256)) return HYLRA_ERR_INVALID;
  return bytes < L.total ? HYLRA_ERR_WORKSPACE : HYLRA_OK;
}

bool bad_ptr(const void* p, size_t a) { return !p || !aligned(p, a); }

// One pool as {64 elements, rows, d / 64, heads, pages}: a box is 64 columns of a
// piece of a page of one head, 128-byte swizzle.
int pool_map(CUtensorMap* tm, const void* base, const hylra_paged_t* s) {
  auto fn = tensor_map_encoder();
  if (!fn) return HYLRA_ERR_CUDA;
  // the stride of a dimension of extent 1 is never used, but must be valid
  auto bytes = [&](int64_t stride, int64_t extent) {
    return (cuuint64_t)(extent == 1 ? s->head_dim : stride) * 2;
  };
  const cuuint64_t dims[5] = {64, (cuuint64_t)s->page_size, (cuuint64_t)(s->head_dim / 64),
                              (cuuint64_t)s->num_kv_heads, (cuuint64_t)s->num_pages};
  const cuuint64_t strides[4] = {bytes(s->token_stride, s->page_size), 128,
                                 bytes(s->head_stride, s->num_kv_heads),
                                 bytes(s->page_stride, s->num_pages)};
  const int utok = s->head_dim == 128 ? DecodeShape<128>::UTOK : DecodeShape<64>::UTOK;
  const cuuint32_t box[5] = {64, (cuuint32_t)std::min(s->page_size, utok), 1, 1, 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(
      tm, s->dtype == HYLRA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
      5, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? HYLRA_OK : HYLRA_ERR_CUDA;
}

// Once per device (`done` holds a bit of each): opt a kernel in to `smem` bytes
// of dynamic shared memory, and have its SMs split their L1 in favour of shared
// memory.  An SM changes that split only when it is idle: a small kernel that
// runs under another split beside the decode kernel's start keeps its SM from
// taking a third decode CTA (16 sequences of up to 128K: 627 against 787 us).
template <typename Kernel>
int prepare(Kernel kernel, std::atomic<uint64_t>& done, int dev, size_t smem = 0) {
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return HYLRA_OK;
  if ((smem > 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)smem) != cudaSuccess) ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared) != cudaSuccess)
    return HYLRA_ERR_CUDA;
  done.fetch_or(bit, std::memory_order_release);
  return HYLRA_OK;
}

// Launch as a programmatic dependent of the preceding kernel, in clusters of
// `cluster` CTAs along x.
template <typename Kernel, typename... Args>
int launch(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster,
           const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? HYLRA_OK : HYLRA_ERR_CUDA;
}

template <int HD, typename T, bool LIST>
int launch_decode(const CUtensorMap& tmK, const CUtensorMap& tmV, DecodeParams& p, int sms,
                  int dev, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int SPLIT = Elem<T>::SPLIT;
  auto kernel = paged_decode_kernel<HD, T, LIST>;
  if (int rc = prepare(kernel, done, dev, kSmemMax)) return rc;
  // three CTAs to an SM with two stages each; where a large batch's lengths do not
  // fit beside them, two with three, or (from about 1000 sequences) with two
  auto fits = [&](int ctas, int nst) {
    return ctas * (decode_smem<HD, SPLIT>(nst, p.B) + 1024) <= kSmemSM;
  };
  const int ctas = fits(kCtasPerSM, 2) ? kCtasPerSM : 2;
  p.nst = ctas == 2 && fits(2, 3) ? 3 : 2;
  const size_t smem = decode_smem<HD, SPLIT>(p.nst, p.B);
  static_assert(2 * (decode_smem<HD, SPLIT>(2, MAX_B) + 1024) <= kSmemSM, "two CTAs to an SM");
  const int G = std::min(ctas * sms, MAX_GRID);
  if (int rc = launch(kernel, dim3(G), NTHR, smem, stream, 1, tmK, tmV, p)) return rc;
  // fewer heads than CTAs: a CTA per head and 32 float4 columns; else a CTA per
  // decode CTA (at most one head that it holds in part ends after it)
  static std::atomic<uint64_t> join_done{0};
  auto join = paged_join_kernel<HD, T, LIST>;
  if (int rc = prepare(join, join_done, dev, kSmemMax - JOIN_STATIC)) return rc;
  const long long nbh = (long long)p.B * p.Hkv;
  const int by_head = nbh <= G ? 1 : 0;
  const int parts = std::min((p.r * HD + 127) / 128, std::max(1, G / (int)std::max(1LL, nbh)));
  const dim3 grid(by_head ? (int)nbh : G, by_head ? parts : 1);
  // its CTAs ask for as much shared memory as the decode kernel's, so that those
  // of the next call find its SMs in pieces that fit (see paged_join_kernel)
  return launch(join, grid, NT_JOIN, smem - JOIN_STATIC, stream, 1, p, G, by_head);
}

int decode(const hylra_paged_t* s, const void* q, const void* K, const void* V,
           const int32_t* table, const int32_t* seqlens, const int32_t* list, int k, bool use_list,
           float* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = check_paged(s);
  if (rc || (rc = check_pool(s))) return rc;
  if (bad_ptr(q, 16) || bad_ptr(K, 16) || bad_ptr(V, 16) || bad_ptr(out, 16) ||
      bad_ptr(table, 4) || bad_ptr(seqlens, 4) || !aligned(lse, 4))
    return HYLRA_ERR_INVALID;
  if (use_list && (bad_ptr(list, 4) || k < 1)) return HYLRA_ERR_INVALID;
  if (use_list && k > HYLRA_MAX_TOPK) return HYLRA_ERR_UNSUPPORTED;
  // the scale times log2(e) must be an fp32 number
  if (s->softmax_scale > 0x1p126f) return HYLRA_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if ((rc = current_device(&dev, &sms))) return rc;
  const PagedLayout L = make_layout(sms);
  if ((rc = check_workspace(ws, ws_bytes, L))) return rc;
  uint8_t* w = static_cast<uint8_t*>(ws);
  DecodeParams p{};
  p.q = q;
  p.table = table;
  p.seqlens = seqlens;
  p.list = list;
  p.out = out;
  p.lse = lse;
  p.status = reinterpret_cast<uint32_t*>(w);
  p.partials = reinterpret_cast<float*>(w + L.partials(ws_bytes));
  p.B = s->batch;
  p.Hq = s->num_q_heads;
  p.Hkv = s->num_kv_heads;
  p.r = s->num_q_heads / s->num_kv_heads;
  p.k = k;
  p.ps_log2 = log2_of(s->page_size);
  p.num_pages = s->num_pages;
  p.max_pages = s->max_pages;
  const double scale =
      s->softmax_scale > 0.f ? (double)s->softmax_scale : 1.0 / std::sqrt((double)s->head_dim);
  p.scale_log2 = (float)(1.4426950408889634 * scale);
  p.wait_limit = host_wait_limit();
  CUtensorMap tmK, tmV;
  if ((rc = pool_map(&tmK, K, s)) || (rc = pool_map(&tmV, V, s))) return rc;
  const bool bf = s->dtype == HYLRA_BF16;
#define HYLRA_DECODE(HD, LIST)                                                              \
  (bf ? launch_decode<HD, __nv_bfloat16, LIST>(tmK, tmV, p, sms, dev, stream)              \
      : launch_decode<HD, __half, LIST>(tmK, tmV, p, sms, dev, stream))
  if (s->head_dim == 128) return use_list ? HYLRA_DECODE(128, true) : HYLRA_DECODE(128, false);
  return use_list ? HYLRA_DECODE(64, true) : HYLRA_DECODE(64, false);
#undef HYLRA_DECODE
}

template <int HD, typename T, int R>
int launch_select_r(const SelectParams& p, int cs, size_t smem, int nbh, int dev, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto kernel = paged_select_kernel<HD, T, R>;
  if (int rc = prepare(kernel, done, dev, kSmemMax)) return rc;
  return launch(kernel, dim3(cs, nbh), NT_SEL, smem, stream, cs, p);
}

template <int HD, typename T>
int launch_select(const SelectParams& p, int cs, size_t smem, int nbh, int dev,
                  cudaStream_t stream) {
  return p.r <= 4 ? launch_select_r<HD, T, 4>(p, cs, smem, nbh, dev, stream)
                  : launch_select_r<HD, T, 8>(p, cs, smem, nbh, dev, stream);
}

template <int HD, typename T>
int launch_append(const AppendParams& p, unsigned ctas, int dev, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto kernel = paged_append_kernel<HD, T>;
  if (int rc = prepare(kernel, done, dev)) return rc;
  return launch(kernel, dim3(ctas), NT_APP, 0, stream, 1, p);
}

}  // namespace

extern "C" {

int hylra_paged_workspace_bytes(const hylra_paged_t* shape, size_t* bytes) {
  int rc = check_paged(shape);
  if (rc) return rc;
  if (!bytes) return HYLRA_ERR_INVALID;
  int dev = 0, sms = 0;
  if ((rc = current_device(&dev, &sms))) return rc;
  *bytes = make_layout(sms).total;
  return HYLRA_OK;
}

int hylra_paged_tables(const hylra_paged_t* shape, const int32_t* cached_lens,
                       const int32_t* new_lens, const int32_t* free_pages,
                       int32_t free_capacity, const int32_t* free_count, int32_t* block_table,
                       int32_t* seqlens_out, int32_t* cu_new, int32_t* slot_map,
                       int32_t slot_capacity, int32_t* free_count_out, void* workspace,
                       size_t workspace_bytes, hylra_stream_t stream) {
  int rc = check_paged(shape);
  if (rc) return rc;
  if (free_capacity < 0 || slot_capacity < 0) return HYLRA_ERR_INVALID;
  if (bad_ptr(cached_lens, 4) || bad_ptr(new_lens, 4) || bad_ptr(free_count, 4) ||
      bad_ptr(block_table, 4) || bad_ptr(seqlens_out, 4) || bad_ptr(cu_new, 4) ||
      bad_ptr(free_count_out, 4) || (free_capacity > 0 && bad_ptr(free_pages, 4)) ||
      (slot_capacity > 0 && bad_ptr(slot_map, 4)))
    return HYLRA_ERR_INVALID;
  int dev = 0, sms = 0;
  if ((rc = current_device(&dev, &sms))) return rc;
  const PagedLayout L = make_layout(sms);
  if ((rc = check_workspace(workspace, workspace_bytes, L))) return rc;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  TablesParams p{};
  p.cached = cached_lens;
  p.added = new_lens;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.table = block_table;
  p.seqlens = seqlens_out;
  p.cu = cu_new;
  p.slots = slot_map;
  p.free_left = free_count_out;
  p.status = reinterpret_cast<uint32_t*>(w);
  p.ticket = reinterpret_cast<uint32_t*>(w + L.ticket);
  p.B = shape->batch;
  p.ps_log2 = log2_of(shape->page_size);
  p.num_pages = shape->num_pages;
  p.max_pages = shape->max_pages;
  p.free_cap = free_capacity;
  p.slot_cap = slot_capacity;
  const long long per_cta = 4 * NT_TAB;
  const int ctas = (int)std::min<long long>(
      sms, std::max<long long>(1, (slot_capacity + per_cta - 1) / per_cta));
  static std::atomic<uint64_t> done{0};
  if ((rc = prepare(paged_tables_kernel, done, dev))) return rc;
  return launch(paged_tables_kernel, dim3(ctas), NT_TAB, 0, (cudaStream_t)stream, 1, p);
}

int hylra_paged_append(const hylra_paged_t* shape, const void* K_new, const void* V_new,
                       int64_t new_stride, const int32_t* slot_map, int32_t num_tokens,
                       void* K_pages, void* V_pages, void* key_means, void* workspace,
                       size_t workspace_bytes, hylra_stream_t stream) {
  int rc = check_paged(shape);
  if (rc || (rc = check_pool(shape))) return rc;
  if (num_tokens < 0) return HYLRA_ERR_INVALID;
  const int64_t width = (int64_t)shape->num_kv_heads * shape->head_dim;
  if (num_tokens > 0 &&
      (bad_ptr(K_new, 16) || bad_ptr(V_new, 16) || bad_ptr(slot_map, 4) || new_stride < width ||
       new_stride % 8 != 0))
    return HYLRA_ERR_INVALID;
  if (new_stride >= (int64_t(1) << 31)) return HYLRA_ERR_UNSUPPORTED;
  if (bad_ptr(K_pages, 16) || bad_ptr(V_pages, 16) || !aligned(key_means, 16))
    return HYLRA_ERR_INVALID;
  int dev = 0, sms = 0;
  if ((rc = current_device(&dev, &sms))) return rc;
  const PagedLayout L = make_layout(sms);
  if ((rc = check_workspace(workspace, workspace_bytes, L))) return rc;
  if (num_tokens == 0) return HYLRA_OK;
  AppendParams p{};
  p.K_new = static_cast<const uint16_t*>(K_new);
  p.V_new = static_cast<const uint16_t*>(V_new);
  p.slots = slot_map;
  p.K = static_cast<uint16_t*>(K_pages);
  p.V = static_cast<uint16_t*>(V_pages);
  p.means = static_cast<uint16_t*>(key_means);
  p.status = static_cast<uint32_t*>(workspace);
  p.new_stride = new_stride;
  p.page_stride = shape->page_stride;
  p.head_stride = shape->head_stride;
  p.token_stride = shape->token_stride;
  p.tokens = num_tokens;
  p.Hkv = shape->num_kv_heads;
  p.ps_log2 = log2_of(shape->page_size);
  p.num_slots = shape->num_pages * shape->page_size;
  // few tokens: a CTA each, so that they spread over the SMs
  p.blocks = (int)((2 * width / 8 + COLS_APP - 1) / COLS_APP);
  p.tile = std::min(std::min(TILE_APP, shape->page_size), std::max(1, num_tokens / (4 * sms)));
  const long long ctas = (long long)p.blocks * (((long long)num_tokens + p.tile - 1) / p.tile);
  if (ctas > INT_MAX) return HYLRA_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  if (shape->head_dim == 128)
    return shape->dtype == HYLRA_BF16 ? launch_append<128, __nv_bfloat16>(p, (unsigned)ctas, dev, st)
                                      : launch_append<128, __half>(p, (unsigned)ctas, dev, st);
  return shape->dtype == HYLRA_BF16 ? launch_append<64, __nv_bfloat16>(p, (unsigned)ctas, dev, st)
                                    : launch_append<64, __half>(p, (unsigned)ctas, dev, st);
}

int hylra_paged_decode(const hylra_paged_t* shape, const void* q, const void* K_pages,
                       const void* V_pages, const int32_t* block_table, const int32_t* seqlens,
                       float* out, float* lse, void* workspace, size_t workspace_bytes,
                       hylra_stream_t stream) {
  return decode(shape, q, K_pages, V_pages, block_table, seqlens, nullptr, 0, false, out, lse,
                workspace, workspace_bytes, (cudaStream_t)stream);
}

int hylra_paged_select(const hylra_paged_t* shape, const void* q, const void* key_means,
                       const int32_t* block_table, const int32_t* seqlens, int32_t topk,
                       int32_t sink, int32_t recent, int32_t* page_idx, void* workspace,
                       size_t workspace_bytes, hylra_stream_t stream) {
  int rc = check_paged(shape);
  if (rc) return rc;
  if (topk < 1 || sink < 0 || recent < 1) return HYLRA_ERR_INVALID;
  if (topk > HYLRA_MAX_TOPK) return HYLRA_ERR_UNSUPPORTED;
  const long long nbh = (long long)shape->batch * shape->num_kv_heads;
  if (nbh > 65535) return HYLRA_ERR_UNSUPPORTED;
  if (bad_ptr(q, 16) || bad_ptr(key_means, 16) || bad_ptr(block_table, 4) ||
      bad_ptr(seqlens, 4) || bad_ptr(page_idx, 4))
    return HYLRA_ERR_INVALID;
  int dev = 0, sms = 0;
  if ((rc = current_device(&dev, &sms))) return rc;
  const PagedLayout L = make_layout(sms);
  if ((rc = check_workspace(workspace, workspace_bytes, L))) return rc;
  SelectParams p{};
  p.q = q;
  p.means = key_means;
  p.table = block_table;
  p.seqlens = seqlens;
  p.idx = page_idx;
  p.status = static_cast<uint32_t*>(workspace);
  p.B = shape->batch;
  p.Hq = shape->num_q_heads;
  p.Hkv = shape->num_kv_heads;
  p.r = shape->num_q_heads / shape->num_kv_heads;
  p.k = topk;
  p.sink = std::min(sink, shape->max_pages);
  p.recent = std::min(recent, shape->max_pages);
  p.ps_log2 = log2_of(shape->page_size);
  p.num_pages = shape->num_pages;
  p.max_pages = shape->max_pages;
  p.scale = shape->softmax_scale > 0.f ? (double)shape->softmax_scale
                                       : 1.0 / std::sqrt((double)shape->head_dim);
  // CTAs per (sequence, KV head): as many as run at once, two to an SM, and more
  // where a CTA would hold the weights of over 1024 pages (eight hold 2048 at most)
  int cs = 1;
  while (cs < MAX_CS && (nbh * cs * 2 <= 2LL * sms || (p.max_pages + cs - 1) / cs > 1024)) cs *= 2;
  p.ppc = (p.max_pages + cs - 1) / cs;
  const size_t smem = select_smem(p.r, p.ppc, p.max_pages);
  cudaStream_t st = (cudaStream_t)stream;
  if (shape->head_dim == 128)
    return shape->dtype == HYLRA_BF16
               ? launch_select<128, __nv_bfloat16>(p, cs, smem, (int)nbh, dev, st)
               : launch_select<128, __half>(p, cs, smem, (int)nbh, dev, st);
  return shape->dtype == HYLRA_BF16
             ? launch_select<64, __nv_bfloat16>(p, cs, smem, (int)nbh, dev, st)
             : launch_select<64, __half>(p, cs, smem, (int)nbh, dev, st);
}

int hylra_paged_decode_topk(const hylra_paged_t* shape, const void* q, const void* K_pages,
                            const void* V_pages, const int32_t* block_table,
                            const int32_t* seqlens, const int32_t* page_idx, int32_t topk,
                            float* out, float* lse, void* workspace, size_t workspace_bytes,
                            hylra_stream_t stream) {
  return decode(shape, q, K_pages, V_pages, block_table, seqlens, page_idx, topk, true, out, lse,
                workspace, workspace_bytes, (cudaStream_t)stream);
}

}  // extern "C"
