// The paged KV cache: slots of new tokens, rotate+quantise into pages, and
// reading rows back.
//
// Layout of one tensor (K or V): codes [n_pages][n_kv_heads][page][16 * BITS
// bytes], scales [n_pages][n_kv_heads][page][128 / G], so one head's tokens of
// a page are contiguous.  A slot is page * page_size + offset (page_size a
// power of two); slots outside [0, n_pages * page_size) mark tokens that have
// no place and are skipped.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "hadq_common.cuh"

namespace hadq {

constexpr int kPagedDim = 128;

// n / d for n < 2^32 by a multiplication (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994, figure 4.1).
struct FastDiv {
  uint32_t d, m, s1, s2;
  FastDiv() = default;
  explicit FastDiv(uint32_t v) : d(v) {
    uint32_t l = 0;
    while ((uint64_t(1) << l) < v) ++l;
    m = uint32_t((uint64_t(1) << 32) * ((uint64_t(1) << l) - v) / v + 1);
    s1 = l < 1 ? l : 1;
    s2 = l < 1 ? 0 : l - 1;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    const uint32_t t = __umulhi(m, n);
    return (t + ((n - t) >> s1)) >> s2;
  }
};

// ------------------------------------------------------------------- slots
//
// Request b has c = cached[b] tokens in ceil(c / page) pages and gets n =
// fresh[b] more.  With need[b] = ceil((c + n) / page) - ceil(c / page) and
// first[b] = sum of need before b, its new pages are free[first[b] ..], its
// tokens start at row cu[b] = sum of fresh before b, and token i of it goes to
// position c + i.  All of that is two prefix sums over the requests, so the
// result does not depend on the order in which CTAs run.
//
// Reads and writes a few bytes per token: bound by latency.  Every CTA forms
// both prefix sums itself (one packed 64-bit scan over the requests, from L2)
// instead of waiting for another launch, then takes its share of the rows and
// of the new pages, finding each one's request by binary search in shared
// memory.  3.7 us for 16 requests, 13.5 us for 2048 requests with 537,498 new
// tokens.
constexpr int kSlotsThreads = 512;
constexpr int kSlotsMaxBatch = 16384;  // two prefix arrays in shared memory

struct SlotsArgs {
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* free_pages;
  int32_t* table;   // [batch][max_pages]
  int32_t* total;   // [batch]
  int32_t* cu;      // [batch + 1]
  int32_t* slots;   // [capacity]
  int32_t* counts;  // [2]
  int64_t capacity;
  int batch, n_free, max_pages, page_log2;
};

struct SlotsReq {
  int64_t c, n;
  int old_pages, need;
  bool fits;  // the table has room for all of its pages
};
__device__ __forceinline__ SlotsReq slots_req(const SlotsArgs& a, int b) {
  SlotsReq r;
  r.c = max(a.cached[b], 0);
  r.n = max(a.fresh[b], 0);
  const int64_t up = (int64_t(1) << a.page_log2) - 1;
  const int64_t p0 = (r.c + up) >> a.page_log2, p1 = (r.c + r.n + up) >> a.page_log2;
  r.fits = p1 <= a.max_pages && r.c + r.n <= 0x7fffffff;
  r.old_pages = int(p0);
  r.need = r.fits ? int(p1 - p0) : 0;
  return r;
}

// The free list still has the request's pages.
__device__ __forceinline__ bool slots_ok(const SlotsArgs& a, const SlotsReq& r, uint32_t first) {
  return r.fits && (r.need == 0 || int64_t(first) + r.need <= a.n_free);
}

// Index of the last entry of the non-decreasing v[0 .. n] (v[0] = 0 <= x)
// that is <= x, at most n - 1.
__device__ __forceinline__ int slots_find(const uint32_t* v, int n, uint32_t x) {
  int lo = 0, hi = n;  // v[lo] <= x; v[hi] > x or hi == n
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) paged_slots_kernel(const SlotsArgs a) {
  extern __shared__ uint32_t slots_smem[];
  uint32_t* cu = slots_smem;                // [batch + 1]
  uint32_t* first = slots_smem + a.batch + 1;  // [batch + 1]
  __shared__ unsigned long long part[THREADS / 32];
  __shared__ int taken, refused;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (tid == 0) taken = refused = 0;

  unsigned long long run = 0;  // totals of the requests before this chunk: rows in the high, pages in the low word
  for (int base = 0; base < a.batch; base += THREADS) {
    const int b = base + tid;
    unsigned long long own = 0;
    if (b < a.batch) {
      const SlotsReq r = slots_req(a, b);
      own = (static_cast<unsigned long long>(r.n) << 32) | unsigned(r.need);
    }
    unsigned long long inc = own;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, m);
      if (lane >= m) inc += o;
    }
    __syncthreads();  // part[] of the previous chunk has been read
    if (lane == 31) part[w] = inc;
    __syncthreads();
    unsigned long long before = run;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < w) before += part[i];
      run += part[i];
    }
    if (b < a.batch) {
      const unsigned long long e = before + inc - own;
      cu[b] = uint32_t(e >> 32);
      first[b] = uint32_t(e);
    }
  }
  if (tid == 0) {
    cu[a.batch] = uint32_t(run >> 32);
    first[a.batch] = uint32_t(run);
  }
  __syncthreads();
  const uint32_t rows = cu[a.batch], pages = first[a.batch];
  const int64_t gtid = int64_t(blockIdx.x) * THREADS + tid, gthreads = int64_t(gridDim.x) * THREADS;
  const int mask = (1 << a.page_log2) - 1;

  for (int64_t t = gtid; t < a.capacity; t += gthreads) {
    int slot = -1;
    if (t < rows) {
      const int b = slots_find(cu, a.batch, uint32_t(t));
      const SlotsReq r = slots_req(a, b);
      if (slots_ok(a, r, first[b])) {
        const int64_t pos = r.c + (t - cu[b]);
        const int p = int(pos >> a.page_log2);
        const int page = p < r.old_pages ? a.table[int64_t(b) * a.max_pages + p] : a.free_pages[first[b] + (p - r.old_pages)];
        if (page >= 0 && page <= (0x7fffffff >> a.page_log2)) slot = (page << a.page_log2) | int(pos & mask);
      }
    }
    a.slots[t] = slot;
  }
  for (int64_t i = gtid; i < pages && i < a.n_free; i += gthreads) {
    const int b = slots_find(first, a.batch, uint32_t(i));
    const SlotsReq r = slots_req(a, b);
    if (slots_ok(a, r, first[b]))
      a.table[int64_t(b) * a.max_pages + r.old_pages + (i - first[b])] = a.free_pages[i];
  }
  for (int64_t b = gtid; b < a.batch; b += gthreads) {
    const SlotsReq r = slots_req(a, int(b));
    a.total[b] = slots_ok(a, r, first[b]) ? int(r.c + r.n) : 0;
    a.cu[b] = int(cu[b]);
  }
  if (blockIdx.x == 0) {
    if (tid == 0) a.cu[a.batch] = int(rows);
    int k = 0, bad = 0;
    for (int b = tid; b < a.batch; b += THREADS) {
      const SlotsReq r = slots_req(a, b);
      if (slots_ok(a, r, first[b])) k += r.need; else ++bad;
    }
    if (k) atomicAdd(&taken, k);
    if (bad) atomicAdd(&refused, bad);
    __syncthreads();
    if (tid == 0) {
      a.counts[0] = taken;
      a.counts[1] = refused;
    }
  }
}

// -------------------------------------------------- 16-point tensor-core stage
//
// Both kernels below take 16 rows of 128 values per warp pass and do four of
// the seven butterfly stages as one exact m16n8k16 product with H_16: A holds
// bf16 inputs (append) or integer codes in f16 (gather), B is +-1, the sums
// are float32.  Which four index bits the product covers is free, as long as
// the lanes of a quad (j = lane & 3) and the two register halves hold them.

__device__ __forceinline__ void mma_h16_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_h16_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// B operand of column tile c (0, 1): contraction index (quad lane jk, half hk,
// element rk) against column n = g -> (quad lane g >> 1, half c, element
// g & 1); entry (-1)^(jk.jn + hk.hn + rk.rn).  `one`: the bit pattern of 1.0.
__device__ __forceinline__ void h16_operand(int g, int j, int c, uint32_t one, uint32_t (&b)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v = 0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int odd = (__popc(j & (g >> 1)) + (h & c) + (r & (g & 1))) & 1;
      v |= (one | (odd ? 0x8000u : 0u)) << (16 * r);
    }
    b[h] = v;
  }
}

// ------------------------------------------------------------------ append
//
// y = (x * s) H_128 of every K and V row of the new tokens, absmax scale and
// codes per group, stored at the token's slot.  Reads 256 bytes and writes
// 16 * BITS + 512 / G per row: bound by HBM (a row is 2.6 bytes per element
// for INT4, 3.1 for INT8, against about 6 instructions per 32 elements).
// 131072 tokens x 8 heads INT4: 133 us (0.79 of the copy rate); 4099 x 32 INT8, groups of
// 64: 17.7 us.
// Lane (g, j) holds elements 32 j .. 32 j + 31 of rows g and g + 8: its codes
// leave as one (INT4) or two 16-byte stores with nothing exchanged, and a
// scale group is 4, 2 or 1 lanes.  Index bits: quad lane = 5-6, register half
// = bit 1, element = bit 0 (the product); bits 2-4 in registers.
struct AppendArgs {
  const uint16_t* x[2];   // K and V rows, bf16 [tokens][heads][128] at a row stride
  int64_t stride[2];      // elements between tokens
  uint8_t* codes[2];
  float* scales[2];
  const int32_t* slots;   // [tokens]
  const int8_t* signs;    // [128] or NULL
  uint32_t rows;          // tokens * heads, below 2^31
  uint32_t nslots;        // n_pages * page_size
  int page_log2;
  FastDiv heads;
  float scale_mul;        // 1 / (sqrt(128) * qmax)
};

constexpr int kAppendThreads = 128;

template <int BITS, int NG, bool SIGNS>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendArgs a) {
  constexpr float QMAX = BITS == 8 ? 127.0f : 7.0f;
  constexpr int RB = 16 * BITS;  // code bytes per row
  const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
  uint32_t bm[2][2];
#pragma unroll
  for (int c = 0; c < 2; ++c) h16_operand(g, j, c, 0x3F80u, bm[c]);
  uint32_t sm[16];  // sign masks of the lane's 16 element pairs
  if constexpr (SIGNS) {
#pragma unroll
    for (int i = 0; i < 16; ++i) sm[i] = pair_sign_mask(a.signs[32 * j + 2 * i], a.signs[32 * j + 2 * i + 1]);
  }
  const uint32_t tiles = (a.rows + 15) / 16, nwarps = gridDim.x * (kAppendThreads / 32);
  const uint32_t t_first = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  // A tile's slots are read one tile, its rows fetched one tile ahead.  K
  // tiles first, then as many V tiles.
  auto find = [&](uint32_t t, int64_t (&dst)[2], const uint4* (&src)[2]) {
    const bool kv = t >= tiles;
    const uint32_t r0 = (t - (kv ? tiles : 0)) * 16;
    const uint16_t* x = (kv ? a.x[1] : a.x[0]) + 32 * j;
    const int64_t stride = kv ? a.stride[1] : a.stride[0];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t r = r0 + g + 8 * u;
      dst[u] = -1;  // row index in the pool, -1 = skip
      src[u] = nullptr;
      if (t < 2 * tiles && r < a.rows) {
        const uint32_t tok = a.heads.div(r), head = r - tok * a.heads.d;
        const uint32_t slot = uint32_t(__ldg(a.slots + tok));
        src[u] = reinterpret_cast<const uint4*>(x + int64_t(tok) * stride + int64_t(head) * kPagedDim);
        if (slot < a.nslots) {
          const uint32_t page = slot >> a.page_log2;
          dst[u] = ((int64_t(page) * a.heads.d + head) << a.page_log2) + (slot - (page << a.page_log2));
        }
      }
    }
  };
  uint4 in[2][4];
  auto fetch = [&](const uint4* const (&src)[2]) {  // (rows without a slot too: the slot may still be on its way)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) in[u][i] = src[u] ? __ldg(src[u] + i) : make_uint4(0u, 0u, 0u, 0u);
  };
  int64_t dst[2], dnext[2];
  const uint4* snext[2];
  find(t_first, dst, snext);
  fetch(snext);
  find(t_first + nwarps, dnext, snext);
  for (uint32_t t = t_first; t < 2 * tiles; t += nwarps) {
    const bool kv = t >= tiles;
    uint8_t* codes = kv ? a.codes[1] : a.codes[0];
    float* scales = kv ? a.scales[1] : a.scales[0];
    float v[2][32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        w[u][0] = in[u][i].x;
        w[u][1] = in[u][i].y;
        w[u][2] = in[u][i].z;
        w[u][3] = in[u][i].w;
        if constexpr (SIGNS) {
#pragma unroll
          for (int k = 0; k < 4; ++k) w[u][k] ^= sm[4 * i + k];
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // words 2h, 2h + 1: elements 8 i + 4 h + {0, 1}, {2, 3}
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_h16_bf16(d, w[0][2 * h], w[1][2 * h], w[0][2 * h + 1], w[1][2 * h + 1], bm[c][0], bm[c][1]);
          v[0][8 * i + 4 * h + 2 * c] = d[0];
          v[0][8 * i + 4 * h + 2 * c + 1] = d[1];
          v[1][8 * i + 4 * h + 2 * c] = d[2];
          v[1][8 * i + 4 * h + 2 * c + 1] = d[3];
        }
    }
    fetch(snext);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      reg_stage<32, 4>(v[u]);
      reg_stage<32, 8>(v[u]);
      float m = reg_stage_absmax<32, 16>(v[u]);
      if constexpr (NG <= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      if constexpr (NG == 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      if (dst[u] < 0) continue;
      if ((j & (4 / NG - 1)) == 0) scales[dst[u] * NG + j / (4 / NG)] = m * a.scale_mul;
      const QInv q = make_qinv(m, QMAX);
      if (q.tiny) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[u][i] *= kUp64;  // exact
      }
      uint32_t c[32];
#pragma unroll
      for (int i = 0; i < 32; i += 2) magic_code2(v[u][i], v[u][i + 1], q.inv, c[i], c[i + 1]);
      if constexpr (BITS == 8) {
        uint4* d = reinterpret_cast<uint4*>(codes + dst[u] * RB + 32 * j);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          d[k] = make_uint4(pack_i8x4(c[16 * k], c[16 * k + 1], c[16 * k + 2], c[16 * k + 3]),
                            pack_i8x4(c[16 * k + 4], c[16 * k + 5], c[16 * k + 6], c[16 * k + 7]),
                            pack_i8x4(c[16 * k + 8], c[16 * k + 9], c[16 * k + 10], c[16 * k + 11]),
                            pack_i8x4(c[16 * k + 12], c[16 * k + 13], c[16 * k + 14], c[16 * k + 15]));
      } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t (&ck)[8] = *reinterpret_cast<const uint32_t(*)[8]>(c + 8 * k);
          w[k] = pack_i4x8(ck);
        }
        *reinterpret_cast<uint4*>(codes + dst[u] * RB + 16 * j) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    dst[0] = dnext[0];
    dst[1] = dnext[1];
    find(t + 2 * nwarps, dnext, snext);
  }
}

// ------------------------------------------------------------------ gather
//
// x = ((q * scale) H_128) * s of the rows at the given slots.  The mirror of
// append: reads 16 * BITS + 512 / G bytes and writes 256 (bf16) or 512
// (float32) per row: bound by HBM.  131072 tokens x 8 heads INT4: 70 us (0.76
// of the copy rate; 112 without rows and codes fetched ahead).  Lane (g, j) holds elements 32 P + 8 j + e
// (P = 0..3, e = 0..7) of rows g and g + 8: each 16-byte bf16 store of a quad
// is 64 contiguous bytes, and a scale group is one, two or all P, so that the
// scales go between the stages over e and j (exact, on integers) and the two
// over P.  Index bits: quad lane = 3-4, element = bit 2, register half =
// bit 0 (the product, whose A operand pairs nibbles e and e + 4 as one mask
// finds them); bits 1, 5, 6 in registers.
struct GatherArgs {
  const uint8_t* codes;
  const float* scales;
  const int32_t* slots;
  const int8_t* signs;
  void* out;              // [tokens][heads][128]
  uint32_t rows;          // tokens * heads, below 2^31
  uint32_t nslots;
  int page_log2;
  FastDiv heads;
};

// bf16x2 of (lo, hi), round to nearest even.
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// f16 pairs (low half: element e, high half: e + 4) of eight codes.
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// (x & mask) ^ magic as one three-input operation.  An instruction takes one
// constant, so the magic comes in a register the compiler cannot fold away;
// with both as constants the codes' unpacking costs a third more.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_xor(uint32_t x, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(x), "n"(MASK), "r"(magic));
  return r;
}
// The f16 magics of the codes: biased INT4, biased INT4 times 16, biased INT8.
struct F16Magic {
  uint32_t m4, m4x16, m8;
  __device__ __forceinline__ F16Magic() {
    asm volatile("mov.u32 %0, 0x64086408;" : "=r"(m4));
    asm volatile("mov.u32 %0, 0x64806480;" : "=r"(m4x16));
    m8 = m4x16;
  }
};
// INT4: nibble n with its sign bit flipped is code + 8; in the mantissa of
// 1024.0 it reads 1032 + code.
__device__ __forceinline__ void i4x8_to_f16_pairs(uint32_t w, const F16Magic& f, uint32_t (&p)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = f16x2_sub(and_xor<0x000F000Fu>(w >> (4 * e), f.m4), f.m4);
}
// INT8: byte with its sign bit flipped is code + 128: 1152 + code.
__device__ __forceinline__ void i8x8_to_f16_pairs(uint32_t lo, uint32_t hi, const F16Magic& f, uint32_t (&p)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t t = __byte_perm(lo, hi, uint32_t(e | (e << 4) | ((4 + e) << 8) | ((4 + e) << 12)));
    p[e] = f16x2_sub(and_xor<0x00FF00FFu>(t, f.m8), f.m8);
  }
}

constexpr int kGatherThreads = 128;

template <int BITS, int NG, bool F32>
__global__ void __launch_bounds__(kGatherThreads) paged_gather_kernel(const GatherArgs a) {
  constexpr int RB = 16 * BITS;
  constexpr float kInvSqrt = 0.08838834764831845f;  // 1 / sqrt(128)
  const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
  uint32_t bm[2][2];
#pragma unroll
  for (int c = 0; c < 2; ++c) h16_operand(g, j, c, 0x3C00u, bm[c]);
  const F16Magic magic;
  uint32_t flip = 0;  // bit 8 P + e: the lane's output 32 P + 8 j + e is negated
  if (a.signs) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (a.signs[32 * (i >> 3) + 8 * j + (i & 7)] < 0) flip |= 1u << i;
  }
  const uint32_t tiles = (a.rows + 15) / 16, nwarps = gridDim.x * (kGatherThreads / 32);
  const uint32_t t_first = blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5);
  // A tile's rows are found one tile, its codes fetched one tile ahead.
  auto find = [&](uint32_t t, int64_t (&src)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t r = t * 16 + g + 8 * u;
      src[u] = -1;
      if (t < tiles && r < a.rows) {
        const uint32_t tok = a.heads.div(r), head = r - tok * a.heads.d;
        const uint32_t slot = uint32_t(__ldg(a.slots + tok));
        if (slot < a.nslots) {
          const uint32_t page = slot >> a.page_log2;
          src[u] = ((int64_t(page) * a.heads.d + head) << a.page_log2) + (slot - (page << a.page_log2));
        }
      }
    }
  };
  float nsc[2][NG];
  uint2 nw[2][4];
  auto fetch = [&](const int64_t (&src)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* p = a.codes + src[u] * RB;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        nw[u][i] = make_uint2(0u, 0u);
        if (src[u] >= 0) {
          if constexpr (BITS == 8)
            nw[u][i] = __ldg(reinterpret_cast<const uint2*>(p + 32 * i + 8 * j));
          else
            nw[u][i].x = __ldg(reinterpret_cast<const uint32_t*>(p + 16 * i + 4 * j));
        }
      }
#pragma unroll
      for (int q = 0; q < NG; ++q) nsc[u][q] = src[u] >= 0 ? __ldg(a.scales + src[u] * NG + q) : 0.f;
    }
  };
  int64_t src[2], next[2];
  find(t_first, src);
  fetch(src);
  find(t_first + nwarps, next);
  for (uint32_t t = t_first; t < tiles; t += nwarps) {
    const uint32_t r0 = t * 16;
    bool have[2];
    float sc[2][NG];
    uint2 w[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      have[u] = src[u] >= 0;
      src[u] = next[u];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[u][i] = nw[u][i];
#pragma unroll
      for (int q = 0; q < NG; ++q) sc[u][q] = nsc[u][q] * kInvSqrt;
    }
    fetch(src);
    find(t + 2 * nwarps, next);
    float v[2][32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t p[2][4];  // pairs (e, e + 4), e = 0..3
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (BITS == 8) i8x8_to_f16_pairs(w[u][i].x, w[u][i].y, magic, p[u]);
        else i4x8_to_f16_pairs(w[u][i].x, magic, p[u]);
      }
#pragma unroll
      for (int o = 0; o < 2; ++o)  // bit 1 of the element
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // bit 0 of the output
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_h16_f16(d, p[0][2 * o], p[1][2 * o], p[0][2 * o + 1], p[1][2 * o + 1], bm[c][0], bm[c][1]);
          v[0][8 * i + 2 * o + c] = d[0];
          v[0][8 * i + 2 * o + c + 4] = d[1];
          v[1][8 * i + 2 * o + c] = d[2];
          v[1][8 * i + 2 * o + c + 4] = d[3];
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!have[u]) continue;
      reg_stage<32, 2>(v[u]);
      if constexpr (NG > 1) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) mul2(v[u][i], v[u][i + 1], sc[u][(i >> 3) * NG / 4]);
      }
      reg_stage<32, 8>(v[u]);
      reg_stage<32, 16>(v[u]);
      if constexpr (NG == 1) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) mul2(v[u][i], v[u][i + 1], sc[u][0]);
      }
      if (flip) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[u][i] = __uint_as_float(__float_as_uint(v[u][i]) ^ (((flip >> i) & 1u) << 31));
      }
      const int64_t r = r0 + g + 8 * u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* x = v[u] + 8 * i;
        if constexpr (F32) {
          float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.out) + r * kPagedDim + 32 * i + 8 * j);
          d[0] = make_float4(x[0], x[1], x[2], x[3]);
          d[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + r * kPagedDim + 32 * i + 8 * j) =
              make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]), bf16x2_rn(x[4], x[5]), bf16x2_rn(x[6], x[7]));
        }
      }
    }
  }
}

}  // namespace hadq
