// Attention of new tokens over the paged, rotated, quantised KV cache: what
// both kernels share (arguments, requests, the cut of the work), and the
// kernel for requests with few query rows.
//
//   q_rot = (q * s) H,  score = scale * q_rot . (kcode * kscale)  (= scale * q . k),
//   p = softmax over the visible keys,  out = ((sum p vcode vscale) H) * s.
//
// Query token i of a request with `len` cached tokens (its n new ones among
// them) sits at position len - n + i and sees the keys at positions up to its
// own (causal), of these only the first `sinks` and the last `window` when a
// window is set; without causal it sees all `len` keys.
//
// A request's query rows against one KV head are its tokens times the g query
// heads that share the head (row = token * g + head).  A unit is a group of
// such rows; all units' key tiles, in the order (request, KV head, row group),
// form one line that is cut into equal pieces, one per CTA.  So the load is
// even whatever the lengths, a long request is split over many CTAs and a
// short one is not, and at most the first and the last unit of a CTA are
// shared: their partial (m, l, O) go to the workspace, and the CTA that
// arrives last at a unit joins them, in CTA order (the result does not depend
// on which CTA that is).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "hadq_attn.cuh"
#include "hadq_common.cuh"
#include "hadq_paged.cuh"

namespace hadq {

struct PagedAttnArgs {
  const uint16_t* q;       // [rows][nqh][128] bf16 at a row stride
  int64_t q_stride;
  int64_t q_rows;
  const int8_t* signs;     // [128] or NULL
  const uint8_t* k_codes;  // [n_pages][nkv][page][16 * BITS]
  const uint8_t* v_codes;
  const float* k_scales;   // [n_pages][nkv][page][NG]
  const float* v_scales;
  const int32_t* table;    // [batch][max_pages]
  const int32_t* lens;     // [batch]
  const int32_t* cu;       // [batch + 1]
  uint16_t* out;           // [rows][nqh][128] bf16
  float* part_o;
  float* part_ml;
  unsigned* counters;      // zero before and after every call
  int batch, nqh, nkv, g, page_log2, max_pages, n_pages;
  int causal, window, sinks;
  int row_lo, row_hi;      // this launch serves requests with row_lo < n * g <= row_hi
  int min_tiles;           // fewest key tiles a CTA takes
  FastDiv by_g;            // division by g
  float qmul;              // softmax scale * log2(e) / sqrt(128)
  float inv_sqrt_dim;      // 1 / sqrt(128)
};

struct PagedReq {
  int row0, n, len;  // first query row, query tokens, cached tokens
  int rows;          // query rows per KV head that this launch serves (0: another launch's)
};
__device__ __forceinline__ PagedReq paged_req(const PagedAttnArgs& a, int b) {
  PagedReq r;
  r.row0 = a.cu[b];
  const int64_t n = int64_t(a.cu[b + 1]) - r.row0;
  // rows outside q are never touched, whatever cu holds
  r.n = r.row0 < 0 || n <= 0 || r.row0 + n > a.q_rows ? 0 : int(n);
  const int64_t room = int64_t(a.max_pages) << a.page_log2;
  r.len = int(min(int64_t(max(a.lens[b], 0)), room));
  const int rows = r.n * a.g;
  r.rows = rows > a.row_lo && rows <= a.row_hi ? rows : 0;
  return r;
}

// The key tiles (TILE tokens) that a group of query tokens first .. last sees:
// [0, head) and [from, head-less end), listed one after the other.
struct PagedTiles {
  int head, from, count;  // tile index i < head: tile i; else tile i - head + from
  int kv_end;             // keys at or past this are seen by none of the group
};
template <int TILE>
__device__ __forceinline__ PagedTiles paged_tiles(const PagedAttnArgs& a, const PagedReq& r, int first, int last) {
  PagedTiles t;
  const int off = r.len - r.n;
  t.kv_end = a.causal ? min(r.len, max(0, off + last + 1)) : r.len;
  const int beg = a.window > 0 ? max(0, off + first - a.window + 1) : 0;
  t.head = (min(min(a.sinks, beg), t.kv_end) + TILE - 1) / TILE;
  t.from = max(beg / TILE, t.head);
  t.count = max(1, t.head + max(0, (t.kv_end + TILE - 1) / TILE - t.from));
  return t;
}

// Inclusive scan over the block; `part` has one entry per warp and may be
// reused after the next barrier.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int nwarps, int64_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += o;
  }
  __syncthreads();
  if (lane == 31) part[w] = v;
  __syncthreads();
  int64_t sum = 0, before = 0;
  for (int i = 0; i < nwarps; ++i) {
    if (i < w) before += part[i];
    sum += part[i];
  }
  *total = sum;
  return v + before;
}

// Where a CTA's piece of the line begins, and how the line is cut.
struct PagedPiece {
  int64_t quota;       // tiles per CTA
  int64_t at, end;     // this CTA's tiles [at, end)
  int b;               // request of the first one
  int64_t in_request;  // its index within the request
};
struct PagedPlanSmem {
  int64_t part[32];
  int64_t at;
  int b;
};
// tiles_of(b): the request's tiles over all heads and row groups.
template <typename F>
__device__ __forceinline__ PagedPiece paged_plan(const PagedAttnArgs& a, PagedPlanSmem& sm, F tiles_of) {
  const int nt = blockDim.x, nwarps = nt >> 5;
  PagedPiece p;
  int64_t total = 0, own = 0, inc = 0;
  for (int base = 0; base < a.batch; base += nt) {
    const int b = base + int(threadIdx.x);
    own = b < a.batch ? tiles_of(b) : 0;
    int64_t sum;
    inc = block_scan(own, sm.part, nwarps, &sum);
    total += sum;
  }
  p.quota = max(int64_t(a.min_tiles), (total + gridDim.x - 1) / int64_t(gridDim.x));
  p.at = int64_t(blockIdx.x) * p.quota;
  p.end = min(total, p.at + p.quota);
  p.b = 0;
  p.in_request = 0;
  if (p.at >= p.end) return p;  // uniform over the block
  int64_t before = 0;
  for (int base = 0; base < a.batch; base += nt) {
    const int b = base + int(threadIdx.x);
    int64_t sum = total;
    if (a.batch > nt) {  // one chunk: the scan above is still in registers
      own = b < a.batch ? tiles_of(b) : 0;
      inc = block_scan(own, sm.part, nwarps, &sum);
    }
    const int64_t lo = before + inc - own;
    if (own > 0 && p.at >= lo && p.at < lo + own) {
      sm.b = b;
      sm.at = p.at - lo;
    }
    before += sum;
    if (before > p.at) break;
  }
  __syncthreads();
  p.b = sm.b;
  p.in_request = sm.at;
  return p;
}

// ------------------------------------------------------- few query rows
//
// One pass over a unit's keys for 8 * RG query rows (RG = 1 or 2).  A warp
// takes 32 keys at a time through its own cp.async ring:
//  * scores by m16n8k32 s8 products: A = the query cut into two signed 8-bit
//    digits of a 16-bit fixed-point number (row r: high digits, row r + 8: low
//    digits), B = the key codes.  The integer sums are exact, and a lane's
//    accumulators hold both digits of one row against its own keys;
//  * the weights as a transposed product O^T += V^T P^T, m16n8k16 f16: A =
//    value codes, exact in f16, B = the weights times the keys' value scales
//    (one such operand per scale group, and the 16 value columns of an MMA lie
//    in one group), which the lane already holds where this operand wants
//    them.  No shuffle but the two of the row maximum.
// A weight enters as f16 times its value scale over 2^e, e the exponent of the
// largest value scale among the 32 keys, and the running reference counts e
// in: m = max(score + e) - 8 when it was last raised, so an f16 weight is below
// 2^16 whatever the scales are; l and O are float32.
//
// Bound by HBM for long INT8 caches.  INT4 uses up no rate (issue 55 %, ALU 46 %,
// DRAM 36 %): about 690 warp instructions per 32 keys, most of them for the
// value codes, form one chain (scores, maximum, exponents, value product), and
// the three CTAs that an SM's registers hold wait on it.  64 ragged requests of
// 17 to 8191 keys, 32 query and 8 KV heads: INT8 117 us (0.84 of the copy rate),
// INT4 94 us (0.54); one request over 131072 INT4 keys 46-48 us.
constexpr int kPdThreads = 128;
constexpr int kPdWarps = 4;
constexpr int kPdStep = 32;                     // keys per warp and step
constexpr int kPdTile = kPdWarps * kPdStep;     // keys per CTA and step
constexpr int kPdPitch = kPagedDim + 4;

__host__ __device__ constexpr int pd_stages(int bits) { return bits == 8 ? 2 : 3; }
// A stage: 32 K rows, 32 V rows, then [32][NG] K scales and as many V scales.
// INT4 rows are 64 bytes, V rows at a pitch of 80; of INT8 rows, 128 bytes,
// the 16-byte piece p of row r lies at p ^ (r & 7).  Either way the fragment
// reads meet no bank twice, and without the contiguous kernel's padding of
// INT8 rows a third CTA fits on an SM.
template <int NG, int BITS>
struct PdStage {
  static constexpr int KROW = 16 * BITS, KP = KROW, VROW = BITS == 8 ? KROW : KROW + 16;
  static constexpr int V = kPdStep * KP;
  static constexpr int S = V + kPdStep * VROW;
  static constexpr int BYTES = S + 2 * kPdStep * 4 * NG;
};

// Weights are held in f16 for the value product, so the reference stays
// kPagedRoom below the largest score + e it has met: a weight down to 2^-22 of
// the largest keeps 11 bits (the bf16 output has 8), and one below that an
// error of 2^-33 of the largest.  It takes that many where one key that adds
// nothing (a sink whose value is near zero) holds nearly all weight, and the
// output is the rest of a long cache: 2047 keys at 2^-24 each came out several
// percent off with the reference at the largest score.
constexpr float kPagedRoom = 8.f;
constexpr float kPdSlack = 5.5f;  // log2 units a score may pass the reference's before that is raised

// The exponent e of a tile's value scales (biased by 127) goes into the
// reference, and l counts a weight as 2^(score + e - m) 2^-e.  For that product
// to hold on to a key whose e is far from the other tiles', e stays at or above
// 2^-80 (l then ends below 2^(80 + 14 + 30)) and, within a unit, no more than
// kPagedExpSpan below the largest so far: a tile of zero value rows still
// counts in l after one of large ones.  Two references may lie 200 apart all
// the same, so sums go from one to the other by the root of the factor, twice.
constexpr int kPagedExpLow = 127 - 80;
constexpr int kPagedExpHigh = 127 + 126;  // (2^-e is a normal number)
constexpr int kPagedExpSpan = 40;

template <int RG, int NG, int BITS>
struct __align__(16) PdSmem {
  union {
    uint8_t stage[kPdWarps][pd_stages(BITS)][PdStage<NG, BITS>::BYTES];
    float comb[kPdWarps][8 * RG][kPdPitch];
  } u;
  int8_t qd[2][8 * RG][kPagedDim];  // query digits: high, low
  float qscale[8 * RG];
  float m[kPdWarps][8 * RG], l[kPdWarps][8 * RG];
  PagedPlanSmem plan;
  int last;
};

template <int V>
struct ConstInt {
  static constexpr int value = V;
};

// 16 bytes at constant offsets from a shared and a global address.
template <int SOFF, int GOFF>
__device__ __forceinline__ void cp_async16_at(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(smem), "l"(gmem), "n"(SOFF), "n"(GOFF) : "memory");
}
// N rows TPP apart, at pitches SP and GP, from shared offset SOFF on.
template <int N, int TPP, int SP, int GP, int SOFF, int P = 0>
__device__ __forceinline__ void cp_rows(uint32_t smem, const void* gmem) {
  if constexpr (P < N) {
    cp_async16_at<SOFF + TPP * P * SP, TPP * P * GP>(smem, gmem);
    cp_rows<N, TPP, SP, GP, SOFF, P + 1>(smem, gmem);
  }
}

// The first of a chain of s8 products: D = A B.
__device__ __forceinline__ void mma_s8_first(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(0));
}

// 4 nibbles of two tokens (a: low half, b: high half of x) -> f16 pairs.
__device__ __forceinline__ void i4x4_to_f16_tokens(uint32_t x, const F16Magic& f, uint32_t (&r)[4]) {
  // 1024 + (code + 8), or 1024 + 16 (code + 8) for the odd nibbles, whose
  // sixteenth is 72 + code
  const uint32_t y = x >> 8;
  r[0] = f16x2_sub(and_xor<0x000F000Fu>(x, f.m4), f.m4);
  r[2] = f16x2_sub(and_xor<0x000F000Fu>(y, f.m4), f.m4);
  const uint32_t t1 = and_xor<0x00F000F0u>(x, f.m4x16), t3 = and_xor<0x00F000F0u>(y, f.m4x16);
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[1]) : "r"(t1), "r"(0x2C002C00u), "r"(0xD480D480u));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[3]) : "r"(t3), "r"(0x2C002C00u), "r"(0xD480D480u));
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// A value scale as the kernels use it: one that is negative or not finite
// counts as zero, so that a key nobody sees cannot reach a sum.
__device__ __forceinline__ float clean_scale(float s) { return s >= 0.f && s < INFINITY ? s : 0.f; }

// H_128 over idx = 4 * lane + r (bits 0-1 in registers, 2-6 on the lanes).
__device__ __forceinline__ void warp_h128(float (&y)[4], int lane) {
  bfly(y[0], y[1]);
  bfly(y[2], y[3]);
  bfly(y[0], y[2]);
  bfly(y[1], y[3]);
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float s = (lane & m) ? -1.f : 1.f;
    lane_stage<4>(y, m, s);
  }
}

// NG floats at an address aligned to them.
template <int NG>
__device__ __forceinline__ void pd_load(const float* p, float (&v)[NG]) {
  if constexpr (NG == 4) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else if constexpr (NG == 2) {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x; v[1] = x.y;
  } else {
    v[0] = *p;
  }
}
template <int NG>
__device__ __forceinline__ void pd_store(float* p, const float (&v)[NG]) {
  if constexpr (NG == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else if constexpr (NG == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  else *p = v[0];
}

// The scales of two consecutive keys (an even one first).
template <int NG>
__device__ __forceinline__ void pd_two_scales(const float* p, float (&s)[2][NG]) {
  if constexpr (NG == 1) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    s[0][0] = v.x;
    s[1][0] = v.y;
  } else if constexpr (NG == 2) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    s[0][0] = v.x; s[0][1] = v.y; s[1][0] = v.z; s[1][1] = v.w;
  } else {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const float4 v = *reinterpret_cast<const float4*>(p + 4 * y);
      s[y][0] = v.x; s[y][1] = v.y; s[y][2] = v.z; s[y][3] = v.w;
    }
  }
}

// The order in which a row's 128 values are kept: a lane's 16 value columns
// are D = 16 / NG consecutive ones of every scale group, column (128 / NG) q +
// D g + e at idx = 8 (D q + e) + g, a permutation of index bits, under which
// H_128 is unchanged.
template <int NG>
__device__ __forceinline__ int pd_column(int idx) {
  constexpr int D = 16 / NG;
  const int qe = idx >> 3, g = idx & 7;
  return (128 / NG) * (qe / D) + D * g + qe % D;
}

// One finished output row: rotate back, normalise, sign, store.  The lane's
// y[r] is index 4 * lane + r.
template <int NG>
__device__ __forceinline__ void pd_finish(const PagedAttnArgs& a, float4 acc, float L, uint16_t* row, int lane) {
  float y[4] = {acc.x, acc.y, acc.z, acc.w};
  warp_h128(y, lane);
  const float inv = L > 0.f ? a.inv_sqrt_dim / L : 0.f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int dim = pd_column<NG>(4 * lane + r);
    float v = y[r] * inv;
    if (a.signs && a.signs[dim] < 0) v = -v;
    row[dim] = uint16_t(bf16x2_rn(v, 0.f));  // (keeps NaN)
  }
}

template <int RG, int NG, int BITS>
__global__ void __launch_bounds__(kPdThreads, RG == 1 ? 3 : 2) paged_decode_kernel(const PagedAttnArgs a) {
  using ST = PdStage<NG, BITS>;
  constexpr int KROW = ST::KROW, KP = ST::KP, VROW = ST::VROW;
  constexpr int STAGES = pd_stages(BITS);
  constexpr int ROWS = 8 * RG;
  extern __shared__ __align__(16) uint8_t pd_smem_raw[];
  PdSmem<RG, NG, BITS>& sm = *reinterpret_cast<PdSmem<RG, NG, BITS>*>(pd_smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
  const F16Magic magic;

  auto group_tiles = [&](const PagedReq& r, int rg) {
    const int f = rg * ROWS, l = min(r.rows, f + ROWS) - 1;
    return paged_tiles<kPdTile>(a, r, f / a.g, l / a.g);
  };
  auto head_tiles = [&](const PagedReq& r) {
    int64_t s = 0;
    for (int rg = 0; rg * ROWS < r.rows; ++rg) s += group_tiles(r, rg).count;
    return s;
  };
  PagedPiece pc = paged_plan(a, sm.plan, [&](int b) { return head_tiles(paged_req(a, b)) * a.nkv; });
  if (pc.at >= pc.end) return;

  // first unit
  int b = pc.b;
  PagedReq rq = paged_req(a, b);
  int h, rg = 0;
  int64_t u;  // tile within the unit
  {
    const int64_t per = head_tiles(rq);
    h = int(pc.in_request / per);
    u = pc.in_request - h * per;
    for (;;) {
      const int c = group_tiles(rq, rg).count;
      if (u < c) break;
      u -= c;
      ++rg;
    }
  }

  const int cta = blockIdx.x;
  int64_t at = pc.at;
  while (at < pc.end) {
    const PagedTiles tl = group_tiles(rq, rg);
    const int i0 = int(u), i1 = int(min(int64_t(tl.count), u + (pc.end - at)));
    const int64_t ustart = at - u;
    const int nw = i1 - i0;
    const int row_base = rg * ROWS;
    const int nrows = min(ROWS, rq.rows - row_base);
    const int off = rq.len - rq.n;

    // ---- queries: rotate, cut into digits ----
    for (int r = w; r < ROWS; r += kPdWarps) {
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < nrows) {
        const int tok = (row_base + r) / a.g, hh = (row_base + r) - tok * a.g;
        const uint2 raw = *reinterpret_cast<const uint2*>(a.q + int64_t(rq.row0 + tok) * a.q_stride +
                                                          int64_t(h * a.g + hh) * kPagedDim + 4 * lane);
        x[0] = bf16lo(raw.x);
        x[1] = bf16hi(raw.x);
        x[2] = bf16lo(raw.y);
        x[3] = bf16hi(raw.y);
        if (a.signs) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (a.signs[4 * lane + i] < 0) x[i] = -x[i];
        }
      }
      warp_h128(x, lane);
      uint32_t top = 0;  // largest magnitude, as bits: NaN above infinity above the rest
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] *= a.qmul;
        top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
      }
      // Infinity in place of NaN: the scale multiplies the -inf of unseen keys.
      const float amax = __uint_as_float(min(__reduce_max_sync(0xffffffffu, top), 0x7f800000u));
      // 32000 steps to the largest entry: an error of 2^-16 of it per entry.
      // Below 2^-100 a query counts as zero; one that is not finite gets digits
      // of zero and an infinite scale, whose product with any key is NaN.
      const bool zero = !(amax >= 7.888609e-31f);
      const float up = zero || amax == INFINITY ? 0.f : 32000.f / amax;
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int qf = up > 0.f ? __float2int_rn(x[i] * up) : 0;
        const int e1 = (qf + 128) >> 8;
        hi |= uint32_t(e1 & 0xff) << (8 * i);
        lo |= uint32_t((qf - 256 * e1) & 0xff) << (8 * i);
      }
      *reinterpret_cast<uint32_t*>(&sm.qd[0][r][4 * lane]) = hi;
      *reinterpret_cast<uint32_t*>(&sm.qd[1][r][4 * lane]) = lo;
      // (positive even then: it multiplies the -inf of unseen keys)
      if (lane == 0) sm.qscale[r] = zero ? 1.f : amax * (BITS == 4 ? 1.f / (16.f * 32000.f) : 1.f / 32000.f);
    }
    __syncthreads();

    uint32_t qa[RG][4][4];
    float qs[RG];
    int lim[RG], low[RG];  // row g sees keys below lim, of these those from low on or below sinks
#pragma unroll
    for (int k = 0; k < RG; ++k) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int d0 = NG == 1 ? 32 * j + 8 * s : 32 * s + 8 * j;  // this lane's 8 dims of k-step s
        const uint2 r0 = *reinterpret_cast<const uint2*>(&sm.qd[0][8 * k + g][d0]);
        const uint2 r1 = *reinterpret_cast<const uint2*>(&sm.qd[1][8 * k + g][d0]);
        qa[k][s][0] = __byte_perm(r0.x, r0.y, 0x6420);
        qa[k][s][1] = __byte_perm(r1.x, r1.y, 0x6420);
        qa[k][s][2] = __byte_perm(r0.x, r0.y, 0x7531);
        qa[k][s][3] = __byte_perm(r1.x, r1.y, 0x7531);
      }
      qs[k] = sm.qscale[8 * k + g];
      const int tok = min(row_base + 8 * k + g, rq.rows - 1) / a.g;
      lim[k] = a.causal ? min(rq.len, off + tok + 1) : rq.len;
      low[k] = a.window > 0 ? off + tok - a.window + 1 : 0;
    }
    // keys that every row of the unit sees need no mask: those below all_lim
    // and, with a window, from all_low on
    const int f_tok = row_base / a.g, l_tok = (row_base + nrows - 1) / a.g;
    const int all_lim = a.causal ? off + f_tok + 1 : rq.len;
    const int all_low = a.window > 0 ? off + l_tok - a.window + 1 : 0;

    // ---- this warp's ring ----
    auto key0 = [&](int k) {  // first of this warp's 32 keys in step k
      const int i = i0 + k;
      return (i < tl.head ? i : i - tl.head + tl.from) * kPdTile + kPdStep * w;
    };
    const int32_t* tab = a.table + int64_t(b) * a.max_pages;
    // Pages of step k's two runs of 16 keys, -1: none of them is cached.
    auto pages_of = [&](int k, int (&pg)[2]) {
      pg[0] = pg[1] = -1;
      if (k >= nw) return;
      const int t = key0(k);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (t + 16 * x < tl.kv_end) pg[x] = __ldg(tab + ((t + 16 * x) >> a.page_log2));
    };
    // Copies: a lane takes piece lane % CPR of rows lane / CPR + TPP p, p =
    // 0 .. NP - 1 for each run of 16 keys.
    constexpr int CPR = KROW / 16, TPP = 32 / CPR, NP = 16 / TPP;
    const int ctok = lane / CPR, cpart = lane % CPR;
    const uint32_t s_ring = static_cast<uint32_t>(__cvta_generic_to_shared(&sm.u.stage[w][0][0]));
    // (INT8: rows ctok + 4 p; the swizzle of odd p is that of even p with bit 2 flipped)
    const uint32_t cdst = (BITS == 8 ? cpart ^ ctok : cpart) * 16;
    const uint32_t d_k = ctok * KP + cdst, d_v = ST::V + ctok * VROW + cdst;
    const uint8_t* gk0 = a.k_codes + ctok * KROW + cpart * 16;
    const uint8_t* gv0 = a.v_codes + ctok * KROW + cpart * 16;
    // Scales: 4 NG pieces of 16 bytes for each run and tensor; lanes below
    // 4 NG take the K scales, the next 4 NG the V scales.
    const float* gs0 = (lane < 4 * NG ? a.k_scales : a.v_scales) + 4 * (lane % (4 * NG));
    const uint32_t d_s = ST::S + (lane < 4 * NG ? 0 : kPdStep * 4 * NG) + 16 * (lane % (4 * NG));
    uint32_t okbits = 0;  // bits 2 (step % STAGES), + 1: the step's runs are in the ring
    int slot_in = 0;      // ring slot of the next step to load
    auto issue = [&](int k, const int (&pg)[2]) {
      const uint32_t st = s_ring + uint32_t(slot_in) * ST::BYTES;
      okbits &= ~(3u << (2 * slot_in));
      const int off = key0(k) & ((1 << a.page_log2) - 1);
      auto run = [&](auto X) {
        constexpr int x = decltype(X)::value;
        if (unsigned(pg[x]) < unsigned(a.n_pages)) {
          okbits |= 1u << (2 * slot_in + x);
          // (the rows of one tensor on one GPU are fewer than 2^32)
          const uint32_t row = ((uint32_t(pg[x]) * uint32_t(a.nkv) + uint32_t(h)) << a.page_log2) +
                               ((off + 16 * x) & ((1 << a.page_log2) - 1));
          const uint64_t at = uint64_t(row) * KROW;
          if constexpr (BITS == 8) {
            cp_rows<2, 8, KP, KROW, 16 * x * KP>(st + d_k, gk0 + at);
            cp_rows<2, 8, KP, KROW, 16 * x * KP + 4 * KP>(st + (d_k ^ 64u), gk0 + at + 4 * KROW);
            cp_rows<2, 8, VROW, KROW, 16 * x * VROW>(st + d_v, gv0 + at);
            cp_rows<2, 8, VROW, KROW, 16 * x * VROW + 4 * VROW>(st + (d_v ^ 64u), gv0 + at + 4 * KROW);
          } else {
            cp_rows<NP, TPP, KP, KROW, 16 * x * KP>(st + d_k, gk0 + at);
            cp_rows<NP, TPP, VROW, KROW, 16 * x * VROW>(st + d_v, gv0 + at);
          }
          if (lane < 8 * NG) cp_async16_at<16 * x * 4 * NG, 0>(st + d_s, gs0 + uint64_t(row) * NG);
        }
      };
      run(ConstInt<0>{});
      run(ConstInt<1>{});
      cp_async_commit();
      slot_in = slot_in + 1 == STAGES ? 0 : slot_in + 1;
    };

    float o[RG][8][4];
    float m_run[RG], l_run[RG];
    int ve_low = kPagedExpLow;  // of the next step
#pragma unroll
    for (int k = 0; k < RG; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[k][i][0] = o[k][i][1] = o[k][i][2] = o[k][i][3] = 0.f;
      m_run[k] = -INFINITY;
      l_run[k] = 0.f;
    }
    {
      int pg[STAGES - 1][2];
#pragma unroll
      for (int k = 0; k < STAGES - 1; ++k) pages_of(k, pg[k]);
#pragma unroll
      for (int k = 0; k < STAGES - 1; ++k) {
        if (k < nw) {
          issue(k, pg[k]);
        } else {
          cp_async_commit();
          slot_in = slot_in + 1 == STAGES ? 0 : slot_in + 1;
        }
      }
    }
    int pg_next[2];
    pages_of(STAGES - 1, pg_next);
    int slot_out = 0;

    for (int k = 0; k < nw; ++k) {
      if (k + STAGES - 1 < nw) {
        issue(k + STAGES - 1, pg_next);
        pages_of(k + STAGES, pg_next);
      } else {
        cp_async_commit();
      }
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      const uint32_t ok = (okbits >> (2 * slot_out)) & 3u;
      uint8_t* st = sm.u.stage[w][slot_out];
      slot_out = slot_out + 1 == STAGES ? 0 : slot_out + 1;
      if (ok) {
        const float* ksc = reinterpret_cast<const float*>(st + ST::S);  // [32][NG]
        float* vsc = reinterpret_cast<float*>(st + ST::S) + kPdStep * NG;
        const int t0 = key0(k);

        // Value scales over 2^e, in place, a key per lane; a key that is not
        // there has none.
        int ve;
        {
          const bool there = t0 + lane < tl.kv_end && ((ok >> (lane >> 4)) & 1u);
          float v[NG], top = 0.f;
          pd_load<NG>(vsc + lane * NG, v);
#pragma unroll
          for (int q = 0; q < NG; ++q) {
            v[q] = there ? clean_scale(v[q]) : 0.f;
            top = fmaxf(top, v[q]);
          }
          ve = min(max(int(__reduce_max_sync(0xffffffffu, __float_as_uint(top)) >> 23), ve_low), kPagedExpHigh);
          ve_low = max(ve_low, ve - kPagedExpSpan);
          const float down = __uint_as_float(uint32_t(254 - ve) << 23);
#pragma unroll
          for (int q = 0; q < NG; ++q) v[q] *= down;
          pd_store<NG>(vsc + lane * NG, v);
          __syncwarp();
        }
        const float vdown = __uint_as_float(uint32_t(254 - ve) << 23);  // 2^-e
        const float vexp = float(ve - 127);                             // e

        // ---- scores of 8 RG rows x 32 keys, over the rows' query scales; this
        // lane's keys are 8 x + 2 j, + 1 ----
        float s[RG][4][2];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint8_t* kr = st + (8 * x + g) * KP;
          int c[RG][NG][4];
          if constexpr (BITS == 4) {
            uint32_t kw[4];
            if constexpr (NG == 1) {
              const uint4 v = *reinterpret_cast<const uint4*>(kr + 16 * j);
              kw[0] = v.x; kw[1] = v.y; kw[2] = v.z; kw[3] = v.w;
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) kw[q] = *reinterpret_cast<const uint32_t*>(kr + 16 * q + 4 * j);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t e, od;
              int4x8_to_s8x16(kw[q], e, od);
#pragma unroll
              for (int r = 0; r < RG; ++r) {
                if (q % (4 / NG) == 0) mma_s8_first(c[r][q * NG / 4], qa[r][q], e, od);
                else mma_s8_16832(c[r][q * NG / 4], qa[r][q], e, od);
              }
            }
          } else {
            uint2 kw[4];
            if constexpr (NG == 1) {
              const uint4 v0 = *reinterpret_cast<const uint4*>(kr + (((2 * j) ^ g) << 4));
              const uint4 v1 = *reinterpret_cast<const uint4*>(kr + (((2 * j + 1) ^ g) << 4));
              kw[0] = make_uint2(v0.x, v0.y); kw[1] = make_uint2(v0.z, v0.w);
              kw[2] = make_uint2(v1.x, v1.y); kw[3] = make_uint2(v1.z, v1.w);
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) kw[q] = *reinterpret_cast<const uint2*>(kr + (((2 * q + (j >> 1)) ^ g) << 4) + 8 * (j & 1));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t e = __byte_perm(kw[q].x, kw[q].y, 0x6420), od = __byte_perm(kw[q].x, kw[q].y, 0x7531);
#pragma unroll
              for (int r = 0; r < RG; ++r) {
                if (q % (4 / NG) == 0) mma_s8_first(c[r][q * NG / 4], qa[r][q], e, od);
                else mma_s8_16832(c[r][q * NG / 4], qa[r][q], e, od);
              }
            }
          }
          float ksl[2][NG];
          pd_two_scales<NG>(ksc + (8 * x + 2 * j) * NG, ksl);
#pragma unroll
          for (int r = 0; r < RG; ++r)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float v = 0.f;
#pragma unroll
              for (int q = 0; q < NG; ++q) {
                const float p = float(c[r][q][y] * 256 + c[r][q][2 + y]);
                v = q == 0 ? p * ksl[y][q] : fmaf(p, ksl[y][q], v);
              }
              s[r][x][y] = v;
            }
        }

        const bool masked = ok != 3u || t0 + kPdStep > all_lim || (a.window > 0 && t0 < all_low);
        float p[RG][4][2];
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          if (masked) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int t = t0 + 8 * x + 2 * j + y;
                if (t >= lim[r] || !((ok >> (x >> 1)) & 1u) || (a.window > 0 && t < low[r] && t >= a.sinks)) s[r][x][y] = -INFINITY;
              }
          }
          float top = max3(s[r][0][0], s[r][0][1], s[r][1][0]);
          top = max3(top, s[r][1][1], s[r][2][0]);
          top = max3(top, s[r][2][1], s[r][3][0]);
          top = fmaxf(top, s[r][3][1]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          top = fmaf(top, qs[r], vexp - kPagedRoom);
          // the reference rises only when the step's maximum asks for more than
          // kPdSlack, so weights stay below 2^13.5
          const bool need = top > m_run[r] + kPdSlack;
          if (__any_sync(0xffffffffu, need)) {
            const float root = need ? exp2f(0.5f * (m_run[r] - top)) : 1.f, alpha = root * root;
            if (need) m_run[r] = top;
            l_run[r] = l_run[r] * root * root;
            // accumulators of this lane belong to rows 2j, 2j + 1
            const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * j), a1 = __shfl_sync(0xffffffffu, alpha, 8 * j + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[r][i][0] *= a0;
              o[r][i][1] *= a1;
              o[r][i][2] *= a0;
              o[r][i][3] *= a1;
            }
          }
          const float sub = m_run[r] == -INFINITY ? 0.f : vexp - m_run[r];
          float sum = 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
#pragma unroll
            for (int y = 0; y < 2; ++y) p[r][x][y] = exp2_ftz(fmaf(s[r][x][y], qs[r], sub));
            sum += p[r][x][0] + p[r][x][1];
          }
          l_run[r] = fmaf(sum, vdown, l_run[r]);
        }

        // ---- O^T += V^T P^T, 16 keys at a time ----
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t pb[RG][NG][2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            float v[2][NG];
            pd_two_scales<NG>(vsc + (16 * x + 8 * z + 2 * j) * NG, v);
#pragma unroll
            for (int q = 0; q < NG; ++q)
#pragma unroll
              for (int r = 0; r < RG; ++r) pb[r][q][z] = cvt_f16x2(p[r][2 * x + z][0] * v[0][q], p[r][2 * x + z][1] * v[1][q]);
          }
          const uint8_t* vt = st + ST::V + 16 * x * VROW;
          // value columns 2 i, 2 i + 1 of the lane's 16: of keys (2j, 2j + 1)
          // in x0, x1, of keys (2j + 8, 2j + 9) in y0, y1
          auto pv = [&](int i, uint32_t x0, uint32_t x1, uint32_t y0, uint32_t y1) {
#pragma unroll
            for (int r = 0; r < RG; ++r) mma_h16_f16(o[r][i], x0, x1, y0, y1, pb[r][i * NG / 8][0], pb[r][i * NG / 8][1]);
          };
          const uint8_t* row[4] = {vt + (2 * j) * VROW, vt + (2 * j + 1) * VROW, vt + (2 * j + 8) * VROW, vt + (2 * j + 9) * VROW};
          if constexpr (BITS == 4) {
            // four columns (16 bits) of each of the four keys
            auto four = [&](int q, uint32_t xa, uint32_t ya) {
              uint32_t u[4], v[4];
              i4x4_to_f16_tokens(xa, magic, u);
              i4x4_to_f16_tokens(ya, magic, v);
              pv(2 * q, u[0], u[1], v[0], v[1]);
              pv(2 * q + 1, u[2], u[3], v[2], v[3]);
            };
            if constexpr (NG == 1) {
              uint2 v[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) v[z] = *reinterpret_cast<const uint2*>(row[z] + 8 * g);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t sel = (q & 1) ? 0x7632u : 0x5410u;
                four(q, __byte_perm(q < 2 ? v[0].x : v[0].y, q < 2 ? v[1].x : v[1].y, sel),
                     __byte_perm(q < 2 ? v[2].x : v[2].y, q < 2 ? v[3].x : v[3].y, sel));
              }
            } else if constexpr (NG == 2) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t v[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) v[z] = *reinterpret_cast<const uint32_t*>(row[z] + 32 * q + 4 * g);
                four(2 * q, __byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410));
                four(2 * q + 1, __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
              }
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t v[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) v[z] = *reinterpret_cast<const uint16_t*>(row[z] + 16 * q + 2 * g);
                four(q, v[0] | (v[1] << 16), v[2] | (v[3] << 16));
              }
            }
          } else {
            auto two = [&](uint32_t p0, uint32_t p1, uint32_t sel) {
              return f16x2_sub(and_xor<0x00FF00FFu>(__byte_perm(p0, p1, sel), magic.m8), magic.m8);
            };
            // four columns (32 bits) of each of the four keys
            auto four = [&](int q, uint32_t wa, uint32_t wb, uint32_t wc, uint32_t wd) {
              pv(2 * q, two(wa, wb, 0x0400), two(wa, wb, 0x0501), two(wc, wd, 0x0400), two(wc, wd, 0x0501));
              pv(2 * q + 1, two(wa, wb, 0x0602), two(wa, wb, 0x0703), two(wc, wd, 0x0602), two(wc, wd, 0x0703));
            };
            if constexpr (NG == 1) {
              uint4 v[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) v[z] = *reinterpret_cast<const uint4*>(row[z] + ((g ^ (2 * j + (z & 1))) << 4));
              four(0, v[0].x, v[1].x, v[2].x, v[3].x);
              four(1, v[0].y, v[1].y, v[2].y, v[3].y);
              four(2, v[0].z, v[1].z, v[2].z, v[3].z);
              four(3, v[0].w, v[1].w, v[2].w, v[3].w);
            } else if constexpr (NG == 2) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint2 v[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  v[z] = *reinterpret_cast<const uint2*>(row[z] + (((4 * q + (g >> 1)) ^ (2 * j + (z & 1))) << 4) + 8 * (g & 1));
                four(2 * q, v[0].x, v[1].x, v[2].x, v[3].x);
                four(2 * q + 1, v[0].y, v[1].y, v[2].y, v[3].y);
              }
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t v[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  v[z] = *reinterpret_cast<const uint32_t*>(row[z] + (((2 * q + (g >> 2)) ^ (2 * j + (z & 1))) << 4) + 4 * (g & 3));
                four(q, v[0], v[1], v[2], v[3]);
              }
            }
          }
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with its ring: the merge area reuses it

    // ---- join the four warps ----
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 1);
      l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 2);
      if (j == 0) {
        sm.m[w][8 * r + g] = m_run[r];
        sm.l[w][8 * r + g] = l_run[r];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // columns 2 i, 2 i + 1 of the lane's 16, of rows 2j, 2j + 1
        sm.u.comb[w][8 * r + 2 * j][16 * i + g] = o[r][i][0];
        sm.u.comb[w][8 * r + 2 * j + 1][16 * i + g] = o[r][i][1];
        sm.u.comb[w][8 * r + 2 * j][16 * i + 8 + g] = o[r][i][2];
        sm.u.comb[w][8 * r + 2 * j + 1][16 * i + 8 + g] = o[r][i][3];
      }
    }
    __syncthreads();
    const bool whole = i0 == 0 && i1 == tl.count;
    const int64_t slot = (2 * int64_t(cta) + (u == 0 ? 1 : 0)) * ROWS;
    auto out_row = [&](int r) {
      const int tok = (row_base + r) / a.g, hh = (row_base + r) - tok * a.g;
      return a.out + (int64_t(rq.row0 + tok) * a.nqh + h * a.g + hh) * kPagedDim;
    };
    for (int r = w; r < nrows; r += kPdWarps) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int x = 0; x < kPdWarps; ++x) M = fmaxf(M, sm.m[x][r]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kPdWarps; ++x) {
        const float root = sm.m[x][r] == -INFINITY ? 0.f : exp2f(0.5f * (sm.m[x][r] - M)), f = root * root;
        L = fmaf(root, root * sm.l[x][r], L);
        const float4 v = *reinterpret_cast<const float4*>(&sm.u.comb[x][r][4 * lane]);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (whole) {
        pd_finish<NG>(a, acc, L, out_row(r), lane);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (slot + r) * kPagedDim + 4 * lane) = acc;
        if (lane == 0) *reinterpret_cast<float2*>(a.part_ml + (slot + r) * 2) = make_float2(M, L);
      }
    }
    if (!whole) {
      const int c0 = int(ustart / pc.quota), c1 = int((ustart + tl.count - 1) / pc.quota);
      __threadfence();
      __syncthreads();
      if (tid == 0) sm.last = atomicAdd(a.counters + c0, 1u) == unsigned(c1 - c0);
      __syncthreads();
      if (sm.last) {
        __threadfence();
        // CTA c0 began the unit (its second slot); the others carry it on (their first)
        for (int r = w; r < nrows; r += kPdWarps) {
          auto at_of = [&](int x) { return (2 * int64_t(x) + (x == c0 ? 1 : 0)) * ROWS + r; };
          float M = -INFINITY;
          for (int x = c0 + lane; x <= c1; x += 32) M = fmaxf(M, __ldcg(a.part_ml + at_of(x) * 2));
#pragma unroll
          for (int m = 16; m; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
          float L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int base = c0; base <= c1; base += 32) {
            float f = 0.f;
            if (base + lane <= c1) {
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + at_of(base + lane) * 2));
              const float root = ml.x == -INFINITY ? 0.f : exp2f(0.5f * (ml.x - M));
              f = root * root;
              L = fmaf(root, root * ml.y, L);
            }
            const int n = min(32, c1 - base + 1);
            for (int x = 0; x < n; x += 8) {
              float4 v[8];
#pragma unroll
              for (int y = 0; y < 8; ++y)
                if (x + y < n) v[y] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at_of(base + x + y) * kPagedDim) + lane);
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                const float fy = __shfl_sync(0xffffffffu, f, x + y);
                if (x + y < n) {
                  acc.x = fmaf(fy, v[y].x, acc.x);
                  acc.y = fmaf(fy, v[y].y, acc.y);
                  acc.z = fmaf(fy, v[y].z, acc.z);
                  acc.w = fmaf(fy, v[y].w, acc.w);
                }
              }
            }
          }
#pragma unroll
          for (int m = 16; m; m >>= 1) L += __shfl_xor_sync(0xffffffffu, L, m);
          pd_finish<NG>(a, acc, L, out_row(r), lane);
        }
        if (tid == 0) a.counters[c0] = 0u;  // ready for the next call
      }
    }
    __syncthreads();  // the merge area becomes the next unit's ring

    // ---- next unit ----
    at += i1 - i0;
    u = 0;
    if (at < pc.end) {
      ++rg;
      if (rg * ROWS >= rq.rows) {
        rg = 0;
        if (++h == a.nkv) {
          h = 0;
          do {
            rq = paged_req(a, ++b);
          } while (rq.rows == 0);
        }
      }
    }
  }
}

}  // namespace hadq
