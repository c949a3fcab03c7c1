// hylra_paged.cuh - kernels over a paged K/V cache for sm_100a.
//
//   * paged_tables_kernel: pages, slots and lengths of a step's new tokens.
//   * paged_append_kernel: K/V rows into their slots, mean keys of full pages.
//   * paged_select_kernel: per (sequence, KV head) the pages whose mean keys
//     promise most attention mass; one thread-block cluster each.
//   * paged_decode_kernel: attention of one query token over all pages of its
//     sequence or over a list of them; persistent CTAs over a static split of
//     all (sequence, KV head, run of tokens) units.
//   * paged_join_kernel: joins the partial results of heads that several CTAs hold.
//
// Every kernel is launched as a programmatic dependent and waits for the
// preceding kernel before its first access to global memory (but for the join's,
// see there).  Only the decode kernel and the join let their dependents start early.
// The join's CTAs have the decode kernel's shared memory footprint: a decode kernel
// that started beside smaller ones found its SMs' shared memory in pieces, and where
// two of its CTAs lay around a small one, the third had no room until one of them
// ended (16 sequences of up to 128K: 960 us, not 620).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <type_traits>

#include "hylra.h"
#include "hylra_device.cuh"

namespace hylra {
namespace paged {

constexpr int GRP = HYLRA_MAX_GROUP;  // q-heads per KV head, the padded MMA N
constexpr int MAX_PAGE = 128;         // tokens per page
constexpr int MAX_GRID = 512;         // CTAs of the decode kernel
constexpr int MAX_B = HYLRA_MAX_BATCH;

// -------------------------------------------------------- device primitives

// 5-D tiled TMA load (box given by the tensor map) into shared memory, completion
// counted in bytes on an mbarrier.  x must be a multiple of 16 bytes / element size.
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* tm, int x, int y, int z,
                                            int u, int v, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v),
      "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// D(16x8, f32) += A(16x16, fp16, row) * B(16x8, fp16, col)
__device__ __forceinline__ void mma_f16_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Stores to the shared memory of another CTA of the cluster (address from mapa).
__device__ __forceinline__ void st_dsmem_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}
__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// ------------------------------------------------------------ element types

template <typename T>
struct Elem;

// P is multiplied with V on the 16-bit matrix units.  Rounding P to one 16-bit
// value would cost 2^-9 (bf16) of every weight in a result that is kept in
// fp32, so P goes in as a sum of 16-bit terms: three bf16 terms hold all 24
// bits of an fp32 value, two fp16 terms 22 bits.  fp16 has few exponents: P is
// scaled by 2^12 there.  P <= 1, logits being subtracted from their maximum before
// they are scaled, so the first term stays below 65504; two terms are off by 2^-22
// of a weight at most, or by 2^-37 of the largest possible one where the second is
// subnormal.  The scale cancels in O / Z.
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int SPLIT = 3;
  static constexpr float SHIFT = 0.f, SCALE = 1.f;
  static __device__ __forceinline__ uint16_t bits(float x) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  }
  static __device__ __forceinline__ float value(uint16_t b) {
    return __uint_as_float((uint32_t)b << 16);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0,
                                             uint32_t b1) {
    mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
  }
};

template <>
struct Elem<__half> {
  static constexpr int SPLIT = 2;
  static constexpr float SHIFT = 12.f, SCALE = 4096.f;
  static __device__ __forceinline__ uint16_t bits(float x) {
    return __half_as_ushort(__float2half_rn(x));
  }
  static __device__ __forceinline__ float value(uint16_t b) {
    return __half2float(__ushort_as_half(b));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
  static __device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0,
                                             uint32_t b1) {
    mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
  }
};

// ----------------------------------------------------------------- decode

// Four warps, one on each sub-partition of an SM: with a fifth (a producer), three
// CTAs of 128 registers a thread fit only while no two of them put their odd warp
// on the same sub-partition, and beside a CTA of the join kernel some SMs took two
// (16 sequences of up to 128K: 787 us).
constexpr int NWC = 4;
constexpr int NTHR = NWC * 32;
constexpr int MAX_PIECES = 8;            // pieces per unit: 128 tokens of 16-token pages
constexpr int MAX_STAGES = 3;
constexpr int STAGE_BYTES = 32768;       // K and V of one unit

struct DecodeParams {
  const void* q;
  const int32_t* table;
  const int32_t* seqlens;
  const int32_t* list;  // page list (LIST kernels)
  float* out;
  float* lse;           // may be null
  uint32_t* status;
  float* partials;      // [2 * gridDim.x][SLOT]: of a head that began before the CTA, of one
                        // that ends after it
  int B, Hq, Hkv, r, k;
  int ps_log2;          // page size
  int num_pages, max_pages;
  int nst;              // ring stages
  float scale_log2;     // softmax scale * log2(e)
  long long wait_limit;
};

// A unit is UTOK tokens of one (sequence, KV head), read as pieces of
// min(page size, UTOK) rows; warp w computes the logits of tokens 16*TT*w .. and,
// for all of the unit's tokens, the dims 16*DT*w .. of O.  Each warp requests its
// share of a unit's boxes as soon as the stage is free.
template <int HD>
struct DecodeShape {
  static constexpr int UTOK = STAGE_BYTES / (4 * HD);  // 64 (d = 128) or 128 (d = 64)
  static constexpr int UTOK_LOG2 = HD == 128 ? 6 : 7;
  static constexpr int TT = UTOK / (16 * NWC);
  static constexpr int DT = HD / (16 * NWC);
  static constexpr int HALVES = HD / 64;        // 64-column boxes of a row
  static constexpr int HALF_BYTES = UTOK * 128; // one half of all rows: [token][128 bytes]
  static constexpr int SLOT = GRP * HD + 2 * GRP;  // partial: O, m (a raw logit), Z
};

template <int HD, int SPLIT>
struct DecodeSmem {
  using S = DecodeShape<HD>;
  alignas(16) uint16_t P[SPLIT][S::UTOK][GRP];  // the tokens' weights, split into terms
  float mx[GRP][NWC];                 // each warp's largest logit
  float zs[NWC][GRP];
  int nv[MAX_STAGES][MAX_PIECES];     // valid rows of each piece of the unit
  alignas(8) uint64_t fullK[MAX_STAGES];
  alignas(8) uint64_t fullV[MAX_STAGES];
  alignas(8) uint64_t empty[MAX_STAGES];
  int abort;
  int issued[MAX_STAGES];             // requests into each stage so far
  alignas(16) uint8_t qslot[MAX_STAGES][GRP * HD * 2];  // the first nst are used
};

// Dynamic shared memory: nst stages (1024-byte aligned), DecodeSmem without the
// query slots past nst, then the sequences' units (B + 1) and lengths (B).
template <int HD, int SPLIT>
__host__ __device__ constexpr size_t decode_fixed(int nst) {
  return sizeof(DecodeSmem<HD, SPLIT>) - (size_t)(MAX_STAGES - nst) * GRP * HD * 2;
}
template <int HD, int SPLIT>
__host__ __device__ constexpr size_t decode_smem(int nst, int B) {
  return 1024 + (size_t)nst * STAGE_BYTES + decode_fixed<HD, SPLIT>(nst) + (2 * (size_t)B + 1) * 4;
}

struct Unit {
  int b, h, j, U;  // part j of the U units of (b, h)
};

// Units are ordered (sequence, KV head, part); up[b]: the units of one head of
// sequences 0 .. b-1, so that sequence b's begin at up[b] * Hkv.
__device__ __forceinline__ Unit locate(const int* up, int B, int Hkv, int u) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (up[mid] * Hkv <= u) lo = mid; else hi = mid - 1;
  }
  Unit x;
  x.b = lo;
  x.U = up[lo + 1] - up[lo];
  const int off = u - up[lo] * Hkv;
  // off / U by an fp32 quotient, which is off by one at most
  x.h = (int)(__fdividef((float)off, (float)x.U));
  x.j = off - x.h * x.U;
  if (x.j < 0) {
    --x.h;
    x.j += x.U;
  } else if (x.j >= x.U) {
    ++x.h;
    x.j -= x.U;
  }
  return x;
}

__device__ __forceinline__ void advance(const int* up, int B, int Hkv, Unit& x) {
  if (++x.j < x.U) return;
  x.j = 0;
  if (++x.h < Hkv) return;
  x.h = 0;
  do { ++x.b; } while (x.b < B && up[x.b + 1] == up[x.b]);
  if (x.b < B) x.U = up[x.b + 1] - up[x.b];
}

// CTA that holds unit u when CTA c holds [floor(c*T/G), floor((c+1)*T/G)), G <= T.
__device__ __forceinline__ int unit_owner(long long u, long long T, int G) {
  return (int)(((u + 1) * G - 1) / T);
}

// Length of sequence b; a length that no table row can hold counts as 0.
__device__ __forceinline__ int checked_len(const int32_t* seqlens, int b, int cap,
                                           uint32_t* status, bool report) {
  const int n = __ldcg(seqlens + b);
  if (n >= 0 && n <= cap) return n;
  if (report) atomicOr(status, HYLRA_STATUS_BAD_SEQLEN);
  return 0;
}

// up[b + 1]: units of a head of sequence b, by all threads; then their running sum,
// by warp 0.
template <bool LIST, int UTOK>
__device__ __forceinline__ void count_units(const DecodeParams& p, int* up, int* lens,
                                            bool report) {
  const int psl = p.ps_log2;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int n = checked_len(p.seqlens, b, p.max_pages << psl, p.status, report);
    const int nb = (n + (1 << psl) - 1) >> psl;
    const int tokens = LIST ? min(p.k, nb) << psl : n;
    if (lens) lens[b] = n;
    up[b + 1] = (tokens + UTOK - 1) / UTOK;
  }
}
__device__ __forceinline__ void sum_units(const DecodeParams& p, int* up) {
  const int lane = threadIdx.x;
  int carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    int v = b0 + lane < p.B ? up[b0 + lane + 1] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += o;
    }
    v += carry;
    if (b0 + lane < p.B) up[b0 + lane + 1] = v;
    carry = __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) up[0] = 0;
}

// S^T = K Q^T and O^T = V^T P^T on the 16-bit matrix units (M: tokens or dims, N: the
// r <= 8 heads), softmax online in base 2.  One query row per head makes this a
// matrix-vector product: 4 r operations a byte, against 250 that the tensor cores
// could do in the time of a byte from memory; a tcgen05 tile (M of 64 or more, N the
// heads) would be as empty and need its accumulators moved to registers for the
// softmax, so the warps' own matrix instructions are used (16 % of their rate).
// Bound by memory: each key and value is read once.  16 sequences of up to 128K, 8 KV
// heads, d 128: 618 us back to back, 6.8 TB/s; one of 32K: 29 us, of which about 3 are
// the way to the first data and 5 the last CTAs and the join; in between 6.1 TB/s.
// Three CTAs of four warps and two 32 KB stages to an SM: one CTA of nine warps with
// three 64 KB stages waited for its own arithmetic (697 us; a unit's chain of steps
// takes 1 us whatever its size), two CTAs with three stages each take 650 us.  A
// common maximum first, one barrier more than weights relative to each warp's own,
// costs nothing and saves a rescaling path.  One warp in turn requesting a whole unit
// held up the others: 142 instead of 135 us over 4 sequences of 64K..128K in pages of 16
// (d 64), 29.3 instead of 28.9 us over one of 32K.
template <int HD, typename T, bool LIST>
__global__ void __launch_bounds__(NTHR, 4)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ DecodeParams p) {
  using S = DecodeShape<HD>;
  using E = Elem<T>;
  using Smem = DecodeSmem<HD, E::SPLIT>;
  constexpr int UTOK = S::UTOK, TT = S::TT, DT = S::DT, HALF = STAGE_BYTES / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int nst = p.nst;
  Smem& sm = *reinterpret_cast<Smem*>(ring + nst * STAGE_BYTES);
  int* up = reinterpret_cast<int*>(ring + nst * STAGE_BYTES + decode_fixed<HD, E::SPLIT>(nst));
  int* lens = up + p.B + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == NTHR - 1) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&sm.fullK[s], 1);
      mbar_init(&sm.fullV[s], 1);
      mbar_init(&sm.empty[s], NWC);
    }
    sm.abort = 0;
    for (int s = 0; s < MAX_STAGES; ++s) sm.issued[s] = 0;
    fence_mbar_init();
  }
  if (tid == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (tid < MAX_STAGES * MAX_PIECES) (&sm.nv[0][0])[tid] = 0;
  const int psl = p.ps_log2, ps = 1 << psl;
  griddep_wait();
  griddep_launch_dependents();

  count_units<LIST, UTOK>(p, up, lens, blockIdx.x == 0);
  __syncthreads();
  if (warp == 0) sum_units(p, up);
  __syncthreads();
  const int total = up[p.B] * p.Hkv;
  const int G = total > 0 ? min((int)gridDim.x, total) : 1;
  const bool works = (int)blockIdx.x < G && total > 0;
  const int lo = works ? (int)((long long)blockIdx.x * total / G) : 0;
  const int hi = works ? (int)((long long)(blockIdx.x + 1) * total / G) : 0;
  const int n = hi - lo;
  volatile int* abort_flag = &sm.abort;
  const int brl = min(psl, S::UTOK_LOG2);  // rows of a piece
  const int ppl = S::UTOK_LOG2 - brl;      // pieces of a unit
  const uint32_t piece_bytes = (uint32_t)(HD * 2) << brl;

  const int cw = warp;
  // sequences without units: zeros and -inf
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (up[b + 1] != up[b]) continue;
    for (int i = tid; i < p.Hq * HD; i += NTHR) p.out[(size_t)b * p.Hq * HD + i] = 0.f;
    if (p.lse)
      for (int i = tid; i < p.Hq; i += NTHR) p.lse[(size_t)b * p.Hq + i] = -INFINITY;
  }
  if (n == 0) return;

  // Requests.  Every warp looks up the pages of 32 / (pieces of a unit) units at once,
  // lane l those of piece l % ppu, and requests every fourth of a unit's boxes.
  const uint64_t pol = l2_evict_first_policy();
  const int ppu = 1 << ppl, UB = 32 >> ppl;
  int f_page = 0, f_row = 0, f_rows = 0, f_b = 0, f_h = 0, f_start = 0;
  auto fetch = [&](int base) {
    f_rows = f_start = 0;
    const int ui = base + (lane >> ppl);
    if (ui >= n) return;
    const Unit x = locate(up, p.B, p.Hkv, lo + ui);
    f_b = x.b;
    f_h = x.h;
    f_start = ui == 0 || x.j == 0;
    const int len = lens[x.b], nb = (len + ps - 1) >> psl;
    const int first = ((x.j << ppl) + (lane & (ppu - 1))) << brl;  // token (or list) place
    const int e = first >> psl;
    if (e >= (LIST ? min(p.k, nb) : nb)) return;
    int j = e;
    if (LIST) {
      j = __ldcg(p.list + ((size_t)x.b * p.Hkv + x.h) * p.k + e);
      if (j < 0 || j >= nb) {
        if (j != -1) atomicOr(p.status, HYLRA_STATUS_BAD_INDEX);
        return;
      }
    }
    const int pg = __ldcg(p.table + (size_t)x.b * p.max_pages + j);
    if (pg < 0 || pg >= p.num_pages) {
      atomicOr(p.status, HYLRA_STATUS_BAD_INDEX);
      return;
    }
    f_page = pg;
    f_row = first & (ps - 1);
    f_rows = max(0, min(1 << brl, len - (j << psl) - f_row));
  };
  auto issue = [&](int i, int s) {  // this warp's share of unit i into stage s
    const int k = i & (UB - 1), at = k << ppl;
    if (k == 0) fetch(i);
    // box: 64 columns of a piece of K or V; lanes 0..7 take every fourth
    const int box = (lane & 7) * NWC + cw, piece = (box >> 1) / S::HALVES;
    const int half = (box >> 1) % S::HALVES;
    const bool mine = lane < 8 && piece < ppu, keys = (box & 1) == 0;
    const int pg = __shfl_sync(0xffffffffu, f_page, at + (mine ? piece : 0));
    const int rw = __shfl_sync(0xffffffffu, f_rows, at + (mine ? piece : 0));
    const int r0 = __shfl_sync(0xffffffffu, f_row, at + (mine ? piece : 0));
    const int h = __shfl_sync(0xffffffffu, f_h, at);
    if (mine && rw > 0) {
      uint8_t* dst = ring + s * STAGE_BYTES + (keys ? 0 : HALF) + half * S::HALF_BYTES +
                     (piece << (brl + 7));
      tma_load_5d(dst, keys ? &tmK : &tmV, 0, r0, half, h, pg, keys ? &sm.fullK[s] : &sm.fullV[s],
                  pol);
    }
    if (cw != 0) return;
    // warp 0 says what is to come; the bytes of a copy that is done before count too
    const int rows = __shfl_sync(0xffffffffu, f_rows, at + (lane & (ppu - 1)));
    const int b = __shfl_sync(0xffffffffu, f_b, at);
    const int start = __shfl_sync(0xffffffffu, f_start, at);
    const uint32_t np = __popc(__ballot_sync(0xffffffffu, lane < ppu && rows > 0));
    if (lane < MAX_PIECES) sm.nv[s][lane] = lane < ppu ? rows : 0;
    __syncwarp();
    if (lane == 0) {
      const uint32_t qbytes = start ? (uint32_t)(p.r * HD * 2) : 0u;
      const uint32_t bytes = np * piece_bytes, bytesK = bytes + qbytes;
      ++sm.issued[s];
      if (bytesK) mbar_arrive_expect_tx(&sm.fullK[s], bytesK); else mbar_arrive(&sm.fullK[s]);
      if (bytes) mbar_arrive_expect_tx(&sm.fullV[s], bytes); else mbar_arrive(&sm.fullV[s]);
      if (start)
        bulk_load(sm.qslot[s],
                  static_cast<const uint8_t*>(p.q) +
                      ((size_t)b * p.Hq + (size_t)h * p.r) * HD * 2,
                  qbytes, &sm.fullK[s]);
    }
    __syncwarp();
  };
  for (int i = 0; i < nst && i < n; ++i) issue(i, i);

  const int g4 = lane >> 2, c4 = lane & 3, mi = lane >> 3, xr = lane & 7;
  const int h0 = 2 * c4, h1 = 2 * c4 + 1;  // this lane's heads in the C fragments
  const int tw = cw * 16 * TT;  // first token of this warp
  // This lane's ldmatrix rows in K and V.  A 128-byte row holds its 16-byte chunk
  // ch at place ch ^ (row & 7); row & 7 is xr for every row that the lane reads,
  // and K's chunks 2 kt + (mi >> 1) are this base's with bits 5 and 6 flipped.
  const uint32_t kofs = (uint32_t)(tw + xr + (mi & 1) * 8) * 128u + (uint32_t)(((mi >> 1) ^ xr) << 4);
  uint32_t vofs[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) {
    const int ch = 2 * (cw * DT + t) + (mi & 1);
    vofs[t] = (uint32_t)HALF + (uint32_t)(xr + (mi >> 1) * 8) * 128u +
              (uint32_t)(ch >> 3) * S::HALF_BYTES + (uint32_t)(((ch & 7) ^ xr) << 4);
  }
  const float sl = p.scale_log2;
  const uint32_t pofs = smem_u32(&sm.P[0][0][0]) + (uint32_t)(mi * 8 + xr) * 16u;
  uint32_t* const pst = reinterpret_cast<uint32_t*>(&sm.P[0][tw + g4][h0]);

  uint32_t qf[HD / 16][2];
  float o[DT][4];
  float m_run[2], z_run[2];
  Unit x = locate(up, p.B, p.Hkv, lo);
  bool has_start = false;  // this CTA holds the segment's first unit
  int stop = 0;            // a wait has failed
  int s = 0;
  uint32_t ph = 0;

  for (int i = 0; i < n; ++i) {
    const bool seg_start = i == 0 || x.j == 0;
    const bool seg_end = i == n - 1 || x.j == x.U - 1;
    uint8_t* stage = ring + s * STAGE_BYTES;
    mbar_wait_bounded(&sm.fullK[s], ph, abort_flag, p.wait_limit);
    int nvw[TT];  // valid tokens of each 16
    bool ragged = false;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int tok = tw + 16 * t;
      nvw[t] = min(16, max(0, sm.nv[s][tok >> brl] - (tok & ((1 << brl) - 1))));
      ragged |= nvw[t] < 16;
    }
    if (seg_start) {
      has_start = x.j == 0;
      const uint32_t* qs = reinterpret_cast<const uint32_t*>(sm.qslot[s]);
#pragma unroll
      for (int kt = 0; kt < HD / 16; ++kt) {
        qf[kt][0] = g4 < p.r ? qs[(g4 * HD + kt * 16 + 2 * c4) >> 1] : 0u;
        qf[kt][1] = g4 < p.r ? qs[(g4 * HD + kt * 16 + 8 + 2 * c4) >> 1] : 0u;
      }
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
      m_run[0] = m_run[1] = -INFINITY;
      z_run[0] = z_run[1] = 0.f;
    }
    // S^T = K Q^T for this warp's tokens (raw logits; e & 2: token g4 + 8 of 16)
    float a[TT][4];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      float a0[4] = {0.f, 0.f, 0.f, 0.f}, a1[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t kb = smem_u32(stage) + kofs + (uint32_t)t * 2048u;
#pragma unroll
      for (int kt = 0; kt < HD / 16; ++kt) {
        uint32_t f[4];
        ldsm_x4((kb ^ (uint32_t)((kt & 3) << 5)) + (uint32_t)(kt >> 2) * S::HALF_BYTES, f[0], f[1],
                f[2], f[3]);
        E::mma((kt & 1) ? a1 : a0, f, qf[kt][0], qf[kt][1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) a[t][e] = a0[e] + a1[e];
    }
    if (ragged) {
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g4 + ((e & 2) ? 8 : 0) >= nvw[t]) a[t][e] = -INFINITY;
    }
    // the unit's largest logit per head, over all warps
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e & 1] = fmaxf(mx[e & 1], a[t][e]);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
      mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
    }
    if (g4 == 0) {
      sm.mx[h0][cw] = mx[0];
      sm.mx[h1][cw] = mx[1];
    }
    __syncthreads();  // mx is complete; every warp is done with the last unit's P
    float m_new[2], sub[2], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 u = *reinterpret_cast<const float4*>(sm.mx[e ? h1 : h0]);
      m_new[e] = fmaxf(m_run[e], fmaxf(fmaxf(u.x, u.y), fmaxf(u.z, u.w)));
      sub[e] = m_new[e] == -INFINITY ? 0.f : m_new[e];  // nothing attended to yet: weights 0
    }
    // weights relative to the running maximum, split into 16-bit terms: both heads
    // of a token in one word.  Maxima are raw logits: a product with the scale minus
    // a rounded one may be above 0, by 2^-24 of a logit, which at 2^27 is 8 binades
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        float w0 = ex2_approx((a[t][e] - sub[0]) * sl) * E::SCALE;
        float w1 = ex2_approx((a[t][e + 1] - sub[1]) * sl) * E::SCALE;
        sum[0] += w0;
        sum[1] += w1;
#pragma unroll
        for (int u = 0; u < E::SPLIT; ++u) {
          const uint32_t both = E::pack(w0, w1);
          pst[(u * UTOK + 16 * t + 4 * e) * (GRP / 2)] = both;
          const float2 v = E::unpack(both);
          w0 -= v.x;
          w1 -= v.y;
        }
      }
    if (m_new[0] != m_run[0] || m_new[1] != m_run[1]) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float al = ex2_approx((m_run[e] - sub[e]) * sl);
        z_run[e] *= al;
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          o[t][e] *= al;
          o[t][e + 2] *= al;
        }
        m_run[e] = m_new[e];
      }
    }
    z_run[0] += sum[0];
    z_run[1] += sum[1];
    mbar_wait_bounded(&sm.fullV[s], ph, abort_flag, p.wait_limit);
    if (ragged) {
      // rows past the end, or of pages that were not loaded, may hold anything
      // (NaN included): zero weights need zero values
      constexpr int CH = HD / 8;  // 16-byte chunks per row
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        uint8_t* rows = stage + HALF + (tw + 16 * t) * 128;
        for (int idx = lane; idx < 16 * CH; idx += 32) {
          const int row = idx / CH, ch = idx % CH;
          if (row >= nvw[t])
            *reinterpret_cast<uint4*>(rows + (ch >> 3) * S::HALF_BYTES + row * 128 +
                                      (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
    }
    // P and the zeroed rows of all warps.  After a failed wait nothing more is
    // requested, and all warps agree on it here: a unit is requested by the four of them
    // or by none, or the bytes of the last requests would not add up and could not be
    // waited for.
    stop |= __syncthreads_or(*abort_flag);
    // O^T += V^T P^T; the matrix unit's sums cover this unit, the running ones are fp32
    float acc[E::SPLIT][DT][4];
#pragma unroll
    for (int u = 0; u < E::SPLIT; ++u)
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[u][t][e] = 0.f;
    const uint32_t vb = smem_u32(stage);
#pragma unroll
    for (int c2 = 0; c2 < UTOK / 32; ++c2) {
      uint32_t pf[E::SPLIT][4];  // 32 tokens' B fragments of each term
#pragma unroll
      for (int u = 0; u < E::SPLIT; ++u)
        ldsm_x4_trans(pofs + (uint32_t)(u * UTOK + c2 * 32) * 16u, pf[u][0], pf[u][1], pf[u][2],
                      pf[u][3]);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          uint32_t vf[4];
          ldsm_x4_trans(vb + vofs[t] + (uint32_t)(c2 * 32 + c * 16) * 128u, vf[0], vf[1], vf[2],
                        vf[3]);
#pragma unroll
          for (int u = 0; u < E::SPLIT; ++u) E::mma(acc[u][t], vf, pf[u][2 * c], pf[u][2 * c + 1]);
        }
    }
    // the stage is free once all warps are here
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[s]);
    if (i + nst < n && !stop) {
      // Should this wait be the one that fails, the unit is requested all the same:
      // the other warps do so too.  The stage's last copies have all arrived, so the
      // phases hold; its rows may be overwritten under a slower warp, whose outputs
      // the call's status (HYLRA_STATUS_TIMEOUT) makes void.
      mbar_wait_bounded(&sm.empty[s], ph, abort_flag, p.wait_limit);
      __syncwarp();
      issue(i + nst, s);
    }
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = 0.f;
#pragma unroll
        for (int u = E::SPLIT - 1; u >= 0; --u) v += acc[u][t][e];
        o[t][e] += v;
      }
    if (++s == nst) {
      s = 0;
      ph ^= 1u;
    }

    if (seg_end) {
      // the lanes of a head hold parts of its Z; the warps' parts meet in zs
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        z_run[0] += __shfl_xor_sync(0xffffffffu, z_run[0], off);
        z_run[1] += __shfl_xor_sync(0xffffffffu, z_run[1], off);
      }
      if (g4 == 0) {
        sm.zs[cw][h0] = z_run[0];
        sm.zs[cw][h1] = z_run[1];
      }
      __syncthreads();
      const bool whole = has_start && x.j == x.U - 1;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int head = e ? h1 : h0;
        float z = 0.f;
#pragma unroll
        for (int t = 0; t < NWC; ++t) z += sm.zs[t][head];
        if (head >= p.r) continue;
        const bool stats = cw == 0 && g4 == 0;
        const size_t row = (size_t)x.b * p.Hq + (size_t)x.h * p.r + head;
        float* dst = p.out + row * HD;
        float f = z == 0.f ? 0.f : 1.f / z;
        if (whole) {
          if (p.lse && stats)
            p.lse[row] = z == 0.f ? -INFINITY
                                  : fmaf(m_run[e], sl, log2f(z) - E::SHIFT) * 0.69314718f;
        } else {
          float* slot = p.partials + (size_t)(2 * (int)blockIdx.x + (has_start ? 1 : 0)) * S::SLOT;
          if (stats) {
            slot[GRP * HD + head] = m_run[e];
            slot[GRP * HD + GRP + head] = z;
          }
          dst = slot + head * HD;
          f = 1.f;
        }
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          const int d0 = (cw * DT + t) * 16 + g4;
          dst[d0] = o[t][e] * f;
          dst[d0 + 8] = o[t][e + 2] * f;
        }
      }
    }
    advance(up, p.B, p.Hkv, x);
  }
  __syncthreads();
  if (*abort_flag && tid == 0) {
    // never exit with a copy into this CTA's shared memory in flight
    for (int t = 0; t < nst; ++t) {
      if (sm.issued[t] == 0) continue;
      const uint32_t lp = (uint32_t)(sm.issued[t] - 1) & 1u;  // the stage's last phase
      mbar_drain(&sm.fullK[t], lp);
      mbar_drain(&sm.fullV[t], lp);
    }
    atomicOr(p.status, HYLRA_STATUS_TIMEOUT);
  }
}

// Joins by log-sum-exp the heads whose units several CTAs hold.  Grid (heads or
// decode CTAs, column parts): with by_head, x is a (sequence, KV head); else it
// is a decode CTA, for the head that begins in it and ends in a later one (at
// most one).  A warp takes every eighth contributor, a lane one float4 column;
// the loads of 64 contributors go out together, so that a join is one trip to L2
// and costs its latency.  It replaced a join by the last CTA to finish a head (a ticket
// each): one SM then fetched all partials, 7-8 us behind the last unit of one
// 32K sequence, against about 2.5 us here.
constexpr int NT_JOIN = 256;
constexpr size_t JOIN_STATIC = NT_JOIN * 24;  // bytes of static shared memory

template <int HD, typename T, bool LIST>
__global__ void __launch_bounds__(NT_JOIN)
    paged_join_kernel(const __grid_constant__ DecodeParams p, int grid_decode, int by_head) {
  using S = DecodeShape<HD>;
  constexpr int NG = NT_JOIN / 32, CB = 8;
  extern __shared__ int up[];  // [B + 1]
  __shared__ float4 wacc[NG][32];
  __shared__ float wm[NG][32], wz[NG][32];
  static_assert(sizeof(wacc) + sizeof(wm) + sizeof(wz) == JOIN_STATIC, "join footprint");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = p.r;
  griddep_launch_dependents();
  // Lengths are older than the decode kernel, which has waited for everything
  // before it: they are read ahead of the wait.
  count_units<LIST, S::UTOK>(p, up, nullptr, false);
  __syncthreads();
  if (warp == 0) sum_units(p, up);
  __syncthreads();
  const int total = up[p.B] * p.Hkv, G = min(grid_decode, max(total, 1));
  int bh = 0, first = 0, nc = 0;
  if (by_head) {
    bh = (int)blockIdx.x;
    const int b = bh / p.Hkv, U = up[b + 1] - up[b];
    if (U > 0) {
      const int start = up[b] * p.Hkv + (bh - b * p.Hkv) * U;
      first = unit_owner(start, total, G);
      nc = unit_owner((long long)start + U - 1, total, G) - first + 1;
    }
  } else if ((int)blockIdx.x < G && total > 0) {
    first = (int)blockIdx.x;
    const int lo = (int)((long long)first * total / G);
    const int end = (int)((long long)(first + 1) * total / G) - 1;
    const Unit x = locate(up, p.B, p.Hkv, end);
    bh = x.b * p.Hkv + x.h;
    if (end - x.j >= lo) nc = unit_owner((long long)end - x.j + x.U - 1, total, G) - first + 1;
  }
  griddep_wait();
  if (nc < 2) return;
  const float sl = p.scale_log2;
  const int ncol = r * (HD / 4);
  for (int col0 = (int)blockIdx.y * 32; col0 < ncol; col0 += (int)gridDim.y * 32) {
    const int col = min(col0 + lane, ncol - 1), g = col / (HD / 4);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, z = 0.f;
    for (int c0 = warp; c0 < nc; c0 += NG * CB) {
      float4 o[CB];
      float mc[CB], zc[CB];
#pragma unroll
      for (int u = 0; u < CB; ++u) {
        // past the end the last one again: loads under the same condition in all lanes
        const int c = min(c0 + u * NG, nc - 1);
        // contributor 0 holds the head's first unit and left slot 2c + 1, the others slot 2c
        const float* slot = p.partials + (size_t)(2 * (first + c) + (c == 0 ? 1 : 0)) * S::SLOT;
        mc[u] = __ldcg(slot + GRP * HD + g);
        zc[u] = __ldcg(slot + GRP * HD + GRP + g);
        o[u] = __ldcg(reinterpret_cast<const float4*>(slot) + col);
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < CB; ++u) mn = fmaxf(mn, mc[u]);
      const float ms = mn == -INFINITY ? 0.f : mn;
      const float al = ex2_approx((m - ms) * sl);
      acc.x *= al;
      acc.y *= al;
      acc.z *= al;
      acc.w *= al;
      z *= al;
#pragma unroll
      for (int u = 0; u < CB; ++u) {
        if (c0 + u * NG >= nc) break;
        const float f = ex2_approx((mc[u] - ms) * sl);
        z = fmaf(f, zc[u], z);
        acc.x = fmaf(f, o[u].x, acc.x);
        acc.y = fmaf(f, o[u].y, acc.y);
        acc.z = fmaf(f, o[u].z, acc.z);
        acc.w = fmaf(f, o[u].w, acc.w);
      }
      m = mn;
    }
    wacc[warp][lane] = acc;
    wm[warp][lane] = m;
    wz[warp][lane] = z;
    __syncthreads();
    if (warp == 0 && col0 + lane < ncol) {
      float mn = m;
#pragma unroll
      for (int w = 1; w < NG; ++w) mn = fmaxf(mn, wm[w][lane]);
      const float ms = mn == -INFINITY ? 0.f : mn;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float zz = 0.f;
#pragma unroll
      for (int w = 0; w < NG; ++w) {
        const float f = ex2_approx((wm[w][lane] - ms) * sl);
        const float4 x = wacc[w][lane];
        zz = fmaf(f, wz[w][lane], zz);
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
      }
      const size_t row = (size_t)bh * r + g;  // b * Hq + h * r + g
      const float rz = zz == 0.f ? 0.f : 1.f / zz;
      *reinterpret_cast<float4*>(p.out + row * HD + 4 * (col % (HD / 4))) =
          make_float4(v.x * rz, v.y * rz, v.z * rz, v.w * rz);
      if (p.lse && col % (HD / 4) == 0)
        p.lse[row] = zz == 0.f ? -INFINITY
                               : fmaf(mn, sl, log2f(zz) - Elem<T>::SHIFT) * 0.69314718f;
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------- select

constexpr int NT_SEL = 256;
constexpr int NW_SEL = NT_SEL / 32;
constexpr int MAX_CS = 8;  // CTAs per cluster (portable limit)

struct SelectParams {
  const void* q;
  const void* means;
  const int32_t* table;
  const int32_t* seqlens;
  int32_t* idx;
  uint32_t* status;
  int B, Hq, Hkv, r, k, sink, recent;
  int ps_log2, num_pages, max_pages;
  int ppc;       // pages of a CTA, at most
  double scale;  // softmax scale
};

struct SelectSmem {
  double wm[NW_SEL][GRP], wz[NW_SEL][GRP];
  double cm[MAX_CS][GRP], cz[MAX_CS][GRP];  // each CTA's maxima and sums, sent by the peers
  double m[GRP], f[GRP];
  uint32_t top[MAX_CS][NW_SEL];  // in the first CTA: the largest keys of the cluster's warps
  int wsum[NW_SEL];
  int count, last;
  alignas(16) double q[GRP][4][34];  // a head's four quarters of the dims, 4 banks apart
};

constexpr int SEL_CAP = 2048;   // entries that one sort takes
constexpr int SEL_BINS = 4096;  // of the histogram before it

// What ranking needs in the place of the weights.
struct RankSmem {
  uint64_t list[SEL_CAP], sorted[SEL_CAP];
  int bins[SEL_BINS];
};

// Dynamic shared memory: SelectSmem, the weights e[r][ppc] (later RankSmem), and a
// key per page of the table, read four at a time.
inline __host__ __device__ size_t select_weights(int r, int ppc) {
  const size_t e = ((size_t)r * ppc * 8 + 15) / 16 * 16;
  return e > sizeof(RankSmem) ? e : sizeof(RankSmem);
}
inline __host__ __device__ size_t select_smem(int r, int ppc, int max_pages) {
  return sizeof(SelectSmem) + select_weights(r, ppc) + ((size_t)max_pages * 4 + 15) / 16 * 16;
}

// An fp32 value times 2^-896 as a double, by its bits: the fp32 exponent stands in
// the double's field as it is, and the query is multiplied by 2^896 instead.
// Two integer instructions, beside the products (the conversion instruction took
// as long as they do).  Zeros stay zeros; infinity and NaN must be sorted out by
// the caller.  x: a 16-bit value's fp32 pattern (its last three bits are 0).
__device__ __forceinline__ double widen(uint32_t x) {
  return __hiloint2double((int)((uint32_t)((int)x >> 3) & 0x8fffffffu), 0);
}
constexpr double WIDEN_UNIT = 0x1p896;

// 16-bit elements as fp32 bit patterns
template <typename T>
__device__ __forceinline__ void unpack2(uint32_t u, uint32_t& lo, uint32_t& hi) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    lo = u << 16;
    hi = u & 0xffff0000u;
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    lo = __float_as_uint(f.x);
    hi = __float_as_uint(f.y);
  }
}

// The largest magnitude bits of two packed 16-bit values each (for infinity and NaN).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu);
}
template <typename T>
__device__ __forceinline__ bool any_nonfinite(uint32_t m) {
  constexpr uint32_t INF = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
  return (m & 0xffffu) >= INF || (m >> 16) >= INF;
}

// Compare-exchange over a warp's 32 * N values, value lane * N + i in register i:
// neighbours at distance j < N are in one lane, the others a shuffle apart.
template <int N>
__device__ __forceinline__ void sort_pass(uint64_t (&v)[N], int lane, int j, int k) {
  if (j < N) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int jj = 1; jj < N; jj <<= 1)
        if (jj == j && !(i & jj)) {
          const uint64_t a = v[i], b = v[i | jj];
          const bool swap = ((lane * N + i) & k) == 0 ? a < b : a > b;
          v[i] = swap ? b : a;
          v[i | jj] = swap ? a : b;
        }
  } else {
    const int lj = j / N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t o = __shfl_xor_sync(0xffffffffu, v[i], lj);
      const bool larger = (((lane * N + i) & k) == 0) == ((lane & lj) == 0);
      v[i] = larger == (v[i] > o) ? v[i] : o;
    }
  }
}

// Puts list[0 .. 256 N) (distinct entries, zeros at the end) in descending order
// into sorted, of which the first `want` places matter.  Each warp sorts 32 N of
// them in registers; an entry's place is how many entries of the warps' lists exceed
// it: binary searches in lock step, a select per step and no branch.
template <int N>
__device__ void block_sort(uint64_t* list, uint64_t* sorted, int want) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  constexpr int LEN = 32 * N;
  uint64_t v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = list[wid * LEN + lane * N + i];
#pragma unroll 1
  for (int k = 2; k <= LEN; k <<= 1)
#pragma unroll 1
    for (int j = k >> 1; j > 0; j >>= 1) sort_pass<N>(v, lane, j, k);
#pragma unroll
  for (int i = 0; i < N; ++i) list[wid * LEN + lane * N + i] = v[i];
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < N; ++i) {
    uint64_t x = v[0];
#pragma unroll
    for (int t = 1; t < N; ++t) x = t == i ? v[t] : x;
    if (x == 0ull || lane * N + i >= want) continue;
    int pos[NW_SEL], at = 0;
#pragma unroll
    for (int t = 0; t < NW_SEL; ++t) pos[t] = 0;
    for (int step = LEN / 2; step > 0; step >>= 1)
#pragma unroll
      for (int t = 0; t < NW_SEL; ++t)
        pos[t] += list[t * LEN + pos[t] + step - 1] > x ? step : 0;
#pragma unroll
    for (int t = 0; t < NW_SEL; ++t) at += pos[t] + (list[t * LEN + pos[t]] > x ? 1 : 0);
    if (at < want) sorted[at] = x;
  }
  __syncthreads();
}

// list[0 .. count) sorted, its first `want` entries into sorted.
__device__ __forceinline__ void sort_entries(RankSmem& rk, int count, int want) {
  const int n = count <= 256 ? 256 : count <= 512 ? 512 : count <= 1024 ? 1024 : 2048;
  for (int i = count + threadIdx.x; i < n; i += NT_SEL) rk.list[i] = 0ull;
  __syncthreads();
  switch (n) {
    case 256: block_sort<1>(rk.list, rk.sorted, want); break;
    case 512: block_sort<2>(rk.list, rk.sorted, want); break;
    case 1024: block_sort<4>(rk.list, rk.sorted, want); break;
    default: block_sort<8>(rk.list, rk.sorted, want); break;
  }
}

// An entry compares by score (a non-negative fp32 value's bits), then lower page.
__device__ __forceinline__ uint64_t rank_entry(uint32_t key, int page) {
  return (uint64_t)key << 32 | (uint32_t)~(uint32_t)page;
}

// The kr best of keys[0 .. nc), in order, into rk.sorted.  More keys than one sort
// takes cheaply go through a histogram of their distance from the largest, 2^15
// units in the last place (0.4 %) a bin over 16 binades: the bins down to the
// kr-th key hold kr keys and a few more.  Where those are still too many (equal
// scores) or the wanted keys lie deeper, batches of keys are sorted in with the
// best so far.
__device__ void rank_keys(const uint32_t* keys, int nc, int kr, int cs, SelectSmem& sm,
                          RankSmem& rk) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (nc <= 512) {
    for (int i = tid; i < nc; i += NT_SEL) rk.list[i] = rank_entry(keys[i], i);
    sort_entries(rk, nc, kr);
    return;
  }
  uint32_t top = 0u;
  for (int i = lane; i < cs * NW_SEL; i += 32) top = max(top, sm.top[0][i]);
  top = __reduce_max_sync(0xffffffffu, top);
  for (int i = tid; i < SEL_BINS; i += NT_SEL) rk.bins[i] = 0;
  if (tid == 0) {
    sm.last = -1;
    sm.count = 0;
  }
  __syncthreads();
  // the bins of four keys; SEL_BINS past the last key
  auto bins4 = [&](int i, uint32_t (&key)[4], uint32_t (&bin)[4]) {
    const uint4 k = *reinterpret_cast<const uint4*>(keys + min(i, (nc - 1) & ~3));
    key[0] = k.x, key[1] = k.y, key[2] = k.z, key[3] = k.w;
#pragma unroll
    for (int j = 0; j < 4; ++j) bin[j] = i + j < nc ? (top - key[j]) >> 15 : SEL_BINS;
  };
  uint32_t key[4], bin[4];
  for (int i = 4 * tid; i < nc; i += 4 * NT_SEL) {
    bins4(i, key, bin);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (bin[j] < SEL_BINS) atomicAdd(&rk.bins[bin[j]], 1);
  }
  __syncthreads();
  {
    constexpr int PER = SEL_BINS / NT_SEL;
    int cnt[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      cnt[i] = rk.bins[tid * PER + i];
      sum += cnt[i];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) sm.wsum[wid] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW_SEL; ++w) incl += w < wid ? sm.wsum[w] : 0;
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      // the bin of the kr-th key: one thread finds it
      if (run < kr && kr <= run + cnt[i] && run + cnt[i] <= SEL_CAP) sm.last = tid * PER + i;
      run += cnt[i];
    }
  }
  __syncthreads();
  const int last = sm.last;
  if (last >= 0) {
    for (int i0 = 0; i0 < nc; i0 += 4 * NT_SEL) {
      const int i = i0 + 4 * tid;
      bins4(i, key, bin);
      uint32_t in[4];
      int n = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        in[j] = __ballot_sync(0xffffffffu, bin[j] <= (uint32_t)last);
        n += __popc(in[j]);
      }
      if (n == 0) continue;
      int at = lane == 0 ? atomicAdd(&sm.count, n) : 0;
      at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (bin[j] <= (uint32_t)last)
          rk.list[at + __popc(in[j] & ((1u << lane) - 1u))] = rank_entry(key[j], i + j);
        at += __popc(in[j]);
      }
    }
    __syncthreads();
    sort_entries(rk, sm.count, kr);
    return;
  }
  int have = 0;  // the best so far, in rk.sorted
  for (int i0 = 0; i0 < nc; i0 += SEL_CAP / 2) {
    const int n = min(SEL_CAP / 2, nc - i0);
    for (int i = tid; i < have; i += NT_SEL) rk.list[i] = rk.sorted[i];
    for (int i = tid; i < n; i += NT_SEL) rk.list[have + i] = rank_entry(keys[i0 + i], i0 + i);
    __syncthreads();
    const int all = have + n;
    have = min(kr, all);
    sort_entries(rk, all, have);
  }
}

// Grid (cs, B * Hkv), a cluster per (sequence, KV head).  The scores decide
// between pages that are often nearly equal, and one order must come out whatever
// the split: products of 16-bit values and their sums, the exponentials and the
// sums over pages run in 64 bits, and a score is rounded once, to fp32.
// The CTAs of a cluster share the pages; once their maxima and sums have been
// exchanged, they send the scores to the first, which ranks them.
// Bound by its instructions and its chain of steps (page id, mean, products, two
// exchanges, ranking), not by memory (0.9 TB/s, the 64-bit units an eighth busy): 8 KV
// heads, d 128: 256 pages of one sequence 6.8 us, 9362 of three (16 tokens each)
// 22.2 us, 8423 of 16 20.4 us.  Every CTA sorting its own pages and ranking them in
// the others' lists took 8.2, 25.7 and 22.4 us.  At 9362 pages, of that form: CTAs
// of half as many threads in clusters of 16, 38 us; the query in registers with the
// sums as butterflies, 32 us; three CTAs to an SM, 30 us; one, 36 us; and of this
// one: an eighth of the dims and four pages a lane (half the reads of the query, more
// exchanges), 24 us.
// R: r rounded up to 4 or 8; the form for 8 spills at d 128 (68 bytes of stores, 108 of
// loads) and takes 10.1, 35.7 and 34.2 us where that for 4 takes 6.9, 22.4 and 20.5.
template <int HD, typename T, int R>
__global__ void __launch_bounds__(NT_SEL, 2)
    paged_select_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem_sel[];
  SelectSmem& sm = *reinterpret_cast<SelectSmem*>(smem_sel);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int cs = (int)gridDim.x, rank = (int)blockIdx.x;
  double* e = reinterpret_cast<double*>(smem_sel + sizeof(SelectSmem));  // [r][ppc]
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem_sel + sizeof(SelectSmem) +
                                               select_weights(p.r, p.ppc));  // the first CTA's
  const int bh = (int)blockIdx.y, b = bh / p.Hkv, h = bh - b * p.Hkv;
  cluster_arrive_relaxed();
  griddep_wait();
  const int psl = p.ps_log2;
  // the query row by row, while the length is on its way
  constexpr int DL = HD / 4, NV = DL / 8;
  for (int i = tid; i < R * HD / 2; i += NT_SEL) {
    const int g = i / (HD / 2), d = 2 * (i - g * (HD / 2));
    uint32_t u = 0u, lo, hi;
    if (g < p.r)
      u = __ldcg(reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.q) +
                                                   ((size_t)b * p.Hq + (size_t)h * p.r + g) * HD + d));
    unpack2<T>(u, lo, hi);
    double* to = &sm.q[g][(d >> 3) & 3][(d >> 5) * 8 + (d & 7)];
    to[0] = (double)__uint_as_float(lo) * WIDEN_UNIT;
    to[1] = (double)__uint_as_float(hi) * WIDEN_UNIT;
  }
  const int n = checked_len(p.seqlens, b, p.max_pages << psl, p.status,
                            h == 0 && rank == 0 && tid == 0);
  const int nb = (n + (1 << psl) - 1) >> psl;
  const int c0 = min(p.sink, nb);              // pages [c0, c1) are ranked
  const int c1 = max(c0, nb - p.recent);
  const int nc = c1 - c0, forced = nb - nc;
  const int kp = min(p.k, nb);
  const int kr = max(0, kp - forced);
  int32_t* dst = p.idx + (size_t)bh * p.k;
  if (rank == 0) {
    for (int i = tid; i < p.k; i += NT_SEL) {
      if (i < min(forced, kp)) dst[i] = i < c0 ? i : c1 + (i - c0);
      else if (i >= kp) dst[i] = -1;
    }
  }
  if (kr == 0) {  // the same in every CTA of the cluster
    cluster_wait_acquire();
    return;
  }
  const int per = (nc + cs - 1) / cs;
  const int s0 = min(nc, rank * per), s1 = min(nc, s0 + per), np = s1 - s0;

  // Logits: a warp takes 16 pages at a time, a lane a quarter of the dims (8 of every
  // 32, so that four lanes read 64 bytes together) of pages row and row + 8.  Page
  // ids run two steps ahead, the means one.
  const int row = lane >> 2, c = lane & 3;
  constexpr int STEP = NW_SEL * 16;
  auto page_at = [&](int at) {
    return at < np ? __ldcg(p.table + (size_t)b * p.max_pages + c0 + s0 + at) : -1;
  };
  // an entry outside the pool stands for no mean: zeros, so that what any page's
  // mean holds stays out of the test for infinity and NaN below
  auto load_mean = [&](int at, int pg, uint4 (&u)[NV]) {
    const bool ok = pg >= 0 && pg < p.num_pages;
    if (!ok && at < np) atomicOr(p.status, HYLRA_STATUS_BAD_INDEX);
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const T*>(p.means) + ((size_t)(ok ? pg : 0) * p.Hkv + h) * HD + c * 8);
#pragma unroll
    for (int t = 0; t < NV; ++t) u[t] = ok ? __ldcg(src + 4 * t) : make_uint4(0u, 0u, 0u, 0u);
    return ok;
  };
  uint4 u[2][NV];
  bool ok[2], okn[2] = {false, false};
  int pgn[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int at = wid * 16 + row + 8 * t;
    ok[t] = load_mean(at, page_at(at), u[t]);
    pgn[t] = page_at(at + STEP);
  }
  __syncthreads();  // the query
  // after the sum over the quarters this lane holds page row + 8 * (c & 1) and
  // heads hb .. hb + R/2 - 1
  const int hb = (c >> 1) * (R / 2);
  double mx[R / 2];
#pragma unroll
  for (int j = 0; j < R / 2; ++j) mx[j] = -INFINITY;
  for (int g0 = wid * 16; g0 < np; g0 += STEP) {
    uint4 un[2][NV];
    if (g0 + STEP < np) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int at = g0 + STEP + row + 8 * t;
        okn[t] = load_mean(at, pgn[t], un[t]);
        pgn[t] = page_at(at + STEP);
      }
    }
    double acc[2][R];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int g = 0; g < R; ++g) acc[t][g] = 0.0;
    uint32_t mag[2] = {0u, 0u};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        double x[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t w = s == 0 ? u[t][v].x : s == 1 ? u[t][v].y : s == 2 ? u[t][v].z : u[t][v].w;
          uint32_t lo, hi;
          unpack2<T>(w, lo, hi);
          x[t][0] = widen(lo);
          x[t][1] = widen(hi);
          mag[t] = max_abs2(mag[t], w);
        }
#pragma unroll
        for (int g = 0; g < R; ++g) {
          const double2 y = *reinterpret_cast<const double2*>(&sm.q[g][c][8 * v + 2 * s]);
#pragma unroll
          for (int t = 0; t < 2; ++t) acc[t][g] = fma(x[t][1], y.y, fma(x[t][0], y.x, acc[t][g]));
        }
      }
    bool bad[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      bad[t] = any_nonfinite<T>(mag[t]);
      bad[t] |= __shfl_xor_sync(0xffffffffu, (int)bad[t], 1) != 0;
      bad[t] |= __shfl_xor_sync(0xffffffffu, (int)bad[t], 2) != 0;
    }
    // sum over the quarters, each exchange halving what a lane holds
    double one[R], half[R / 2];
#pragma unroll
    for (int g = 0; g < R; ++g) {
      const double keep = (c & 1) ? acc[1][g] : acc[0][g], give = (c & 1) ? acc[0][g] : acc[1][g];
      one[g] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
    }
#pragma unroll
    for (int j = 0; j < R / 2; ++j) {
      const double keep = (c & 2) ? one[R / 2 + j] : one[j], give = (c & 2) ? one[j] : one[R / 2 + j];
      half[j] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
    }
    const int at = g0 + row + 8 * (c & 1);
    const bool has = (c & 1) ? ok[1] : ok[0], nan = (c & 1) ? bad[1] : bad[0];
#pragma unroll
    for (int j = 0; j < R / 2; ++j) {
      const double l = nan ? (double)NAN : has ? half[j] * p.scale : -INFINITY;
      if (at < np && hb + j < p.r) {
        e[(size_t)(hb + j) * p.ppc + at] = l;
        mx[j] = fmax(mx[j], l);
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      ok[t] = okn[t];
#pragma unroll
      for (int v = 0; v < NV; ++v) u[t][v] = un[t][v];
    }
  }
#pragma unroll
  for (int j = 0; j < R / 2; ++j) {
    mx[j] = fmax(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 1));
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) mx[j] = fmax(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], off));
    if (row == 0 && (c & 1) == 0) sm.wm[wid][hb + j] = mx[j];
  }
  __syncthreads();
  if (tid < p.r) {
    double m = sm.wm[0][tid];
    for (int w = 1; w < NW_SEL; ++w) m = fmax(m, sm.wm[w][tid]);
    sm.m[tid] = m;
  }
  __syncthreads();
  // e = exp(logit - this CTA's maximum), and its sum: a head per warp, or
  // several warps a head
  const int wph = NW_SEL / p.r, g = wid % p.r, part = wid / p.r;
  if (part < wph) {
    const double m = sm.m[g] == -INFINITY ? 0.0 : sm.m[g];
    double z = 0.0;
    for (int i = part * 32 + lane; i < np; i += wph * 32) {
      const double v = exp(e[(size_t)g * p.ppc + i] - m);
      e[(size_t)g * p.ppc + i] = v;
      z += v;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    if (lane == 0) sm.wz[part][g] = z;
  }
  __syncthreads();
  cluster_wait_acquire();  // every CTA of the cluster runs: its shared memory may be written
  if (tid < cs * GRP) {
    const int peer = tid / GRP, hg = tid % GRP;
    if (hg < p.r) {
      double z = 0.0;
      for (int w = 0; w < wph; ++w) z += sm.wz[w][hg];
      st_dsmem_f64(mapa_shared(smem_u32(&sm.cm[rank][hg]), peer), sm.m[hg]);
      st_dsmem_f64(mapa_shared(smem_u32(&sm.cz[rank][hg]), peer), z);
    }
  }
  cluster_sync_all();
  if (wid < p.r) {  // warp g: what this CTA's weights of head g are divided by
    const double m = lane < cs ? sm.cm[lane][wid] : -INFINITY;
    double M = m;
#pragma unroll
    for (int off = MAX_CS / 2; off > 0; off >>= 1)
      M = fmax(M, __shfl_xor_sync(0xffffffffu, M, off));
    const double f = m == -INFINITY ? 0.0 : exp(m - M);
    double Z = lane < cs ? f * sm.cz[lane][wid] : 0.0;
#pragma unroll
    for (int off = MAX_CS / 2; off > 0; off >>= 1) Z += __shfl_xor_sync(0xffffffffu, Z, off);
    if (lane == rank) sm.f[wid] = m == -INFINITY ? 0.0 : f / Z;
  }
  __syncthreads();
  const uint32_t kbase = mapa_shared(smem_u32(keys), 0);
  bool odd = false;
  uint32_t top = 0u;
  for (int i = tid; i < np; i += NT_SEL) {
    double sc = 0.0;
    for (int t = 0; t < p.r; ++t) sc += e[(size_t)t * p.ppc + i] * sm.f[t];
    float key = (float)sc;
    if (!(key >= 0.f && key < INFINITY)) {
      key = 0.f;
      odd = true;
    }
    top = max(top, __float_as_uint(key));
    st_dsmem_u32(kbase + (uint32_t)(s0 + i) * 4u, __float_as_uint(key));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) st_dsmem_u32(mapa_shared(smem_u32(&sm.top[rank][wid]), 0), top);
  if (odd) atomicOr(p.status, HYLRA_STATUS_NONFINITE);
  cluster_sync_all();
  if (rank != 0) return;
  RankSmem& rk = *reinterpret_cast<RankSmem*>(e);
  rank_keys(keys, nc, kr, cs, sm, rk);
  for (int i = tid; i < kr; i += NT_SEL)
    dst[forced + i] = c0 + (int32_t)~(uint32_t)(rk.sorted[i] & 0xffffffffull);
}

// ----------------------------------------------------------------- append

constexpr int NT_APP = 256;
constexpr int COLS_APP = 128;  // 16-byte columns of a CTA
constexpr int TILE_APP = 64;  // tokens per CTA, at most
constexpr int BACK_APP = 8 * NT_APP;  // slots of a step of the search behind left-out tokens

struct AppendParams {
  const uint16_t* K_new;
  const uint16_t* V_new;
  const int32_t* slots;
  uint16_t* K;
  uint16_t* V;
  uint16_t* means;  // may be null
  uint32_t* status;
  long long new_stride, page_stride, head_stride, token_stride;
  int tokens, tile, Hkv, ps_log2, num_slots;
  int blocks;  // column blocks of a token's K and V rows
};

// A run is a row of tokens in consecutive slots of one page.  A CTA owns the runs
// that begin in its tile of tokens, for a block of 128 of the 16-byte columns of a
// token's K and V: it copies their rows, each thread one column, and when a run fills
// its page, the threads have summed the page's keys on the way.  Rows of the page
// before the run come from the pool, or from the input where tokens that were left out
// part the page's tokens of this call, whose rows in the pool other threads may be
// writing: the slots are searched back from the run, past any left out, to the first
// of another page (only where the token before the run may be the page's; 1.3 us, and
// 0.4 us per 1024 left-out tokens, read 16 bytes at a time).
// Bound by memory: two rows read and two written a token.  63 132 tokens of 8 heads,
// d 128: 103 us, of which the means take 2; a plain copy of as many bytes takes 83.  Reading a filled page's rows once more for its mean
// took 127-135 us, two rows in flight per thread do as well as four (eight: 118), and
// 64 columns a CTA lose a fifth with 16-token pages.
template <int HD, typename T>
__global__ void __launch_bounds__(NT_APP)
    paged_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float part[NT_APP][9];  // 9: a warp's columns fall into different banks
  __shared__ int slots[TILE_APP + 2 * MAX_PAGE];  // of the tokens a page before the tile and on
  __shared__ int from[MAX_PAGE];  // token of this call that brings a row of a filled page, or -1
  const int tid = threadIdx.x, lane = tid & 31;
  const int blk = (int)(blockIdx.x % (unsigned)p.blocks);
  const long long first = (long long)(blockIdx.x / (unsigned)p.blocks) * p.tile;
  const int width = p.Hkv * (HD / 8);  // columns of K, and of V
  const int cols = min(COLS_APP, 2 * width - blk * COLS_APP);
  const int nrow = NT_APP / cols, rl = tid / cols;  // rows at a time
  const int ckv = blk * COLS_APP + tid - rl * cols;   // column of the token's K, then V
  const bool keys = ckv < width, active = rl < nrow;
  const int cv = keys ? ckv : ckv - width, h = cv / (HD / 8), v = cv % (HD / 8);
  const int psl = p.ps_log2, ps = 1 << psl;
  const uint16_t* src = (keys ? p.K_new : p.V_new) + (size_t)cv * 8;
  uint16_t* pool = (keys ? p.K : p.V) + (size_t)h * p.head_stride + v * 8;
  griddep_wait();
  const int tb = (int)first;
  for (int i = tid; i < p.tile + 2 * ps; i += NT_APP) {
    const long long t = (long long)tb - ps + i;
    int s = t >= 0 && t < p.tokens ? __ldcg(p.slots + t) : -1;
    if (s < 0 || s >= p.num_slots) {
      if (s != -1 && blk == 0 && i >= ps && i < ps + p.tile)
        atomicOr(p.status, HYLRA_STATUS_BAD_INDEX);
      s = -1;
    }
    slots[i] = s;
  }
  __syncthreads();
  const int* tile = slots + ps;  // tile[i]: token tb + i, i from -ps to tile + ps - 1
  auto row_at = [&](int s) {
    return reinterpret_cast<uint4*>(pool + (size_t)(s >> psl) * p.page_stride +
                                    (size_t)(s & (ps - 1)) * p.token_stride);
  };
  auto begins = [&](int l) {  // a run begins at token l of the tile
    return l < p.tile && tile[l] >= 0 &&
           ((tile[l] & (ps - 1)) == 0 || tile[l - 1] < 0 || tile[l - 1] != tile[l] - 1);
  };
  uint64_t starts = (uint64_t)__ballot_sync(0xffffffffu, begins(lane)) |
                    (uint64_t)__ballot_sync(0xffffffffu, begins(lane + 32)) << 32;
  while (starts) {
    const int l = __ffsll((long long)starts) - 1;
    starts &= starts - 1;
    const int s0 = tile[l], off = s0 & (ps - 1), t = tb + l;
    // length of the run: up to the page's end or the first slot out of line
    int len = 0;
    for (bool whole = true; whole && len < ps - off;) {
      const int i = len + lane;
      const uint32_t out =
          ~__ballot_sync(0xffffffffu, off + i < ps && tile[l + min(i, ps - 1)] == s0 + i);
      whole = out == 0u;
      len += whole ? 32 : __ffs(out) - 1;
    }
    const bool fills = p.means != nullptr && off + len == ps;
    // the mean as a sum of shares: 1 / ps is a power of two, so that the roundings are
    // those of the sum, but it cannot pass fp32 as a sum of bf16 keys can
    float sum[8];
    const float inv = 1.f / (float)ps;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = 0.f;
    auto add = [&](const uint4& u) {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sum[2 * k] = fmaf(Elem<T>::value((uint16_t)(w[k] & 0xffffu)), inv, sum[2 * k]);
        sum[2 * k + 1] = fmaf(Elem<T>::value((uint16_t)(w[k] >> 16)), inv, sum[2 * k + 1]);
      }
    };
    constexpr int U = 2;  // rows in flight per thread
    for (int i0 = active ? rl : len; i0 < len; i0 += nrow * U) {
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * nrow < len)
          x[u] = __ldg(reinterpret_cast<const uint4*>(src + (size_t)(t + i0 + u * nrow) * p.new_stride));
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * nrow < len) {
          *row_at(s0 + i0 + u * nrow) = x[u];
          if (fills) add(x[u]);
        }
    }
    if (!fills) continue;
    // rows before the run: from the pool, or from this call, of which the token
    // before the run is then another or was left out
    const int p0 = s0 - off;  // the page's first slot
    const bool mixed =
        off > 0 && t > 0 && (tile[l - 1] < 0 || (tile[l - 1] >= p0 && tile[l - 1] < s0));
    if (mixed) {
      for (int i = tid; i < off; i += NT_APP) from[i] = -1;
      __syncthreads();
      // a token u that may bring a row; says whether the search ends there
      auto look = [&](int u, int slot) {
        const bool here = (uint32_t)slot - (uint32_t)p0 < (uint32_t)off;
        if (here) from[slot - p0] = u;
        return u <= 0 || slot == p0 || ((uint32_t)slot < (uint32_t)p.num_slots && !here);
      };
      // first the tokens whose slots are here, then BACK_APP at a time, as 16-byte groups
      // of four (some looked at once more); the one that holds token 0 may begin before it
      static_assert(TILE_APP + MAX_PAGE <= NT_APP, "a thread per slot before the run");
      const int n = l + ps;
      bool end = tid < n && look(t - 1 - tid, tile[l - 1 - (tid < n ? tid : 0)]);
      const int skew = (int)((reinterpret_cast<uintptr_t>(p.slots) >> 2) & 3);
      const int top = ((t - 1 - n + skew) & ~3) - skew;  // the group of the last slot not seen
      for (int u = top - 4 * tid; !__syncthreads_or(end); u -= BACK_APP) {
        int4 g[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int at = u - v * (BACK_APP / 2);
          g[v] = make_int4(-1, -1, -1, -1);
          if (at >= 0) g[v] = __ldcg(reinterpret_cast<const int4*>(p.slots + at));
          else if (at > -4) {
            g[v].w = __ldcg(p.slots + at + 3);
            if (at > -3) g[v].z = __ldcg(p.slots + at + 2);
            if (at > -2) g[v].y = __ldcg(p.slots + at + 1);
          }
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int at = u - v * (BACK_APP / 2);
          end |= look(at, g[v].x);
          end |= look(at + 1, g[v].y);
          end |= look(at + 2, g[v].z);
          end |= look(at + 3, g[v].w);
        }
      }
    }
    for (int i0 = active && keys ? rl : off; i0 < off; i0 += nrow * U) {
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * nrow;
        if (i >= off) continue;
        const int tok = mixed ? from[i] : -1;
        x[u] = __ldcg(tok >= 0 ? reinterpret_cast<const uint4*>(src + (size_t)tok * p.new_stride)
                               : row_at(s0 - off + i));
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * nrow < off) add(x[u]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) part[tid][k] = sum[k];
    __syncthreads();
    if (rl == 0 && keys) {
      for (int q = 1; q < nrow; ++q)
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += part[tid + q * cols][k];
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = (uint32_t)Elem<T>::bits(sum[2 * k]) |
               (uint32_t)Elem<T>::bits(sum[2 * k + 1]) << 16;
      *reinterpret_cast<uint4*>(p.means + (size_t)(s0 >> psl) * p.Hkv * HD + (size_t)cv * 8) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------- tables

constexpr int NT_TAB = 256;

struct TablesParams {
  const int32_t* cached;
  const int32_t* added;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* table;
  int32_t* seqlens;
  int32_t* cu;
  int32_t* slots;
  int32_t* free_left;
  uint32_t* status;
  uint32_t* ticket;
  int B, ps_log2, num_pages, max_pages, free_cap, slot_cap;
};

struct TablesSmem {
  int cu[MAX_B + 1];     // tokens before request b (saturating)
  int first[MAX_B + 1];  // pages taken before request b
  int held[MAX_B];       // cached tokens; -1: refused
  long long wt[NT_TAB / 32];
  int wp[NT_TAB / 32];
  int free_n, left, last;
};

// Inclusive sums of (tokens, pages) over the block's threads.
__device__ __forceinline__ void scan2(long long& t, int& a, TablesSmem& sm) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long vt = __shfl_up_sync(0xffffffffu, t, off);
    const int va = __shfl_up_sync(0xffffffffu, a, off);
    if (lane >= off) {
      t += vt;
      a += va;
    }
  }
  if (lane == 31) {
    sm.wt[wid] = t;
    sm.wp[wid] = a;
  }
  __syncthreads();
  for (int w = 0; w < wid; ++w) {
    t += sm.wt[w];
    a += sm.wp[w];
  }
}

// Every CTA derives the running sums for itself (a few thousand bytes), then
// writes its share of slots and table entries; the last CTA to have read the
// inputs writes the small outputs, which may be the inputs themselves.
// Bound by latency: two scans, a search per token and the way of two dependent loads.
// 16 requests of a token each 4.6 us, 1024 such 6.5 us, 288 613 new tokens of 64
// requests 8.6 us; a kernel for the sums before one for the slots would add a launch,
// and the smallest one here (an append of 16 tokens) takes 1.9 us.
__global__ void __launch_bounds__(NT_TAB)
    paged_tables_kernel(const __grid_constant__ TablesParams p) {
  __shared__ TablesSmem sm;
  constexpr int PER = MAX_B / NT_TAB;  // requests per thread
  const int tid = threadIdx.x, psl = p.ps_log2, ps = 1 << psl;
  const bool report = blockIdx.x == 0;
  griddep_wait();
  if (tid == 0) {
    int f = __ldcg(p.free_count);
    if (f < 0 || f > p.free_cap) {
      if (report) atomicOr(p.status, HYLRA_STATUS_BAD_INDEX);
      f = 0;
    }
    sm.free_n = f;
  }
  int held[PER], add[PER], need[PER];
  bool bad[PER];
  long long tsum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    held[i] = add[i] = need[i] = 0;
    bad[i] = false;
    if (b < p.B) {
      held[i] = __ldcg(p.cached + b);
      add[i] = __ldcg(p.added + b);
      const int cap = p.max_pages << psl;
      bad[i] = held[i] < 0 || add[i] < 0 || held[i] > cap || add[i] > cap - held[i];
      if (add[i] < 0) add[i] = 0;
    }
    tsum += add[i];
  }
  long long tend = tsum;
  int dummy = 0;
  scan2(tend, dummy, sm);
  long long trun = tend - tsum;
  int psum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    if (b < p.B) sm.cu[b] = (int)min(trun, (long long)INT32_MAX);
    trun += add[i];
    if (b == p.B - 1) sm.cu[p.B] = (int)min(trun, (long long)INT32_MAX);
    if (b < p.B && trun > p.slot_cap && add[i] > 0) bad[i] = true;
    if (b < p.B && !bad[i])
      need[i] = ((held[i] + add[i] + ps - 1) >> psl) - ((held[i] + ps - 1) >> psl);
    psum += need[i];
  }
  __syncthreads();
  long long tdummy = 0;
  int pend = psum;
  scan2(tdummy, pend, sm);
  int prun = pend - psum;
  const int avail = sm.free_n;
  if (tid == 0) sm.left = avail;
  __syncthreads();
  uint32_t bits = 0;
  int taken = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    if (b < p.B) {
      sm.first[b] = prun;
      prun += need[i];
      const bool full = need[i] > 0 && prun > avail;
      if (bad[i]) bits |= HYLRA_STATUS_BAD_SEQLEN;
      if (full) bits |= HYLRA_STATUS_NO_PAGES;
      else taken += need[i];
      sm.held[b] = bad[i] || full ? -1 : held[i];
      if (b == p.B - 1) sm.first[p.B] = prun;
    }
  }
  if (taken) atomicSub(&sm.left, taken);
  if (bits && report) atomicOr(p.status, bits);
  __syncthreads();
  const int left = sm.left, used = avail - left, cu_end = sm.cu[p.B];

  // The last request whose start is <= i[v], for four places at once: the same
  // number of steps for all, so that the searches overlap.
  int top = 1;
  while (2 * top < p.B) top *= 2;
  auto owners = [&](const int* start, const int (&i)[4], int (&b)[4]) {
#pragma unroll
    for (int v = 0; v < 4; ++v) b[v] = 0;
    for (int step = top; step > 0; step >>= 1)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int at = b[v] + step;
        if (at < p.B && start[at] <= i[v]) b[v] = at;
      }
  };
  bool odd = false;
  const int stride = 4 * (int)gridDim.x * NT_TAB;
  // a thread's four places are NT_TAB apart: a warp's stores stay together
  for (int base = (int)blockIdx.x * 4 * NT_TAB + tid; base < used; base += stride) {
    int a[4], b[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) a[v] = min(base + v * NT_TAB, used - 1);
    owners(sm.first, a, b);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (base + v * NT_TAB >= used) break;
      int pg = __ldcg(p.free_pages + (avail - 1 - a[v]));
      if (pg < 0 || pg >= p.num_pages) {
        pg = -1;
        odd = true;
      }
      p.table[(size_t)b[v] * p.max_pages + ((sm.held[b[v]] + ps - 1) >> psl) +
              (a[v] - sm.first[b[v]])] = pg;
    }
  }
  for (long long base = (long long)blockIdx.x * 4 * NT_TAB + tid; base < p.slot_cap;
       base += stride) {
    int t[4], b[4], pg[4], pos[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) t[v] = (int)min(base + v * NT_TAB, (long long)p.slot_cap - 1);
    owners(sm.cu, t, b);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int held = sm.held[b[v]];
      pg[v] = pos[v] = -1;
      if (t[v] < cu_end && held >= 0) {
        pos[v] = held + (t[v] - sm.cu[b[v]]);
        const int j = pos[v] >> psl, have = (held + ps - 1) >> psl;
        pg[v] = __ldcg(j < have ? p.table + (size_t)b[v] * p.max_pages + j
                                : p.free_pages + (avail - 1 - (sm.first[b[v]] + j - have)));
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const bool ok = pg[v] >= 0 && pg[v] < p.num_pages;
      odd |= pos[v] >= 0 && !ok;
      if (base + v * NT_TAB < p.slot_cap)
        p.slots[t[v]] = ok ? (pg[v] << psl) + (pos[v] & (ps - 1)) : -1;
    }
  }
  if (odd) atomicOr(p.status, HYLRA_STATUS_BAD_INDEX);
  if (gridDim.x > 1) {
    __syncthreads();
    if (tid == 0) {
      const bool last = atomic_add_acq_rel_gpu(p.ticket, 1u) == gridDim.x - 1;
      if (last) *p.ticket = 0u;
      sm.last = last;
    }
    __syncthreads();
    if (!sm.last) return;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    if (b < p.B) {
      p.cu[b] = sm.cu[b];
      p.seqlens[b] = sm.held[b] >= 0 ? held[i] + add[i] : held[i];
    }
  }
  if (tid == 0) {
    p.cu[p.B] = cu_end;
    *p.free_left = left;
  }
}

}  // namespace paged
}  // namespace hylra
