// Attention over the paged cache for many query rows (prompt chunks, cross
// attention): both products on the fifth-generation tensor cores.
//
// A unit is up to 256 query rows (two M = 128 tiles, groups 0 and 1) of one
// request and KV head; its keys come in tiles of 64.  Per tile and group
//     S = Q K^T    (A = Q, B = K from shared memory, S in TMEM),
//     O += P V     (A = P in TMEM, beside S; B = V),
// eight and four tcgen05.mma of K = 16 each, all operands f16:
//  * keys and values are codes times their scale over 2^e, e the exponent of
//    the tile's largest scale, so both fill the f16 range from the top
//    whatever the scales are.  The scale and the product are rounded to
//    f16: 11 bits, where the output has 8;
//  * each rotated query is scaled by the exponent of a bound of its entries
//    and rounded to f16;
//  * the exponents come back as one multiplier per tile in the exponent's fma
//    (scores) and as a summand of the softmax reference (values): with
//    m = max(score + e) - 8 when it was last raised, a weight is 2^(score + e - m),
//    rounded to f16 for the product (kPagedRoom), and l counts 2^-e of it in
//    float32.  The reference rises only when a row's weights sum past f16's
//    largest number, so that O, in TMEM, is rarely rescaled and no maximum is
//    taken otherwise (802 -> 780 us against maxima of every tile).  m, l and O
//    are float32.
//
// Roles (one CTA per SM, five warpgroups, registers dealt by setmaxnreg):
//  * warps 0-3 and 4-7: softmax of group 0 and 1, a row per thread, the 64
//    scores in registers.  S has two buffers per group, and P takes the upper
//    half of its own, so that S of the next tile is there when a row is done.
//    They also rotate the next unit's queries into shared memory (on the
//    tensor cores by mma.sync, 845 -> 802 us against H_128 in registers)
//    before they finish a unit (rotate back, normalise, store);
//  * warps 18 and 19 plan tiles ahead: the rows' places in the pool, their
//    scales and the largest one's exponent;
//  * warps 8-11 (keys) and 12-15 (values): half a cached row per thread: load
//    codes one tile ahead into registers, convert, scale and store them in the
//    swizzled layout both products read (K: K-major, V: MN-major; the same
//    bytes, and the same code);
//  * warps 16 and 17 issue the MMAs of group 0 and 1.  Group 0's softmax runs
//    under group 1's MMAs and the other way round.
// The roles' loops are kept short (run-time loops instead of straight code):
// with four instruction streams on an SM, fetching them cost more than the
// work did (with everything unrolled, 3700 cycles a tile).
// The columns of Q, K, V are stored in the order in which one mask finds
// them (pt_column): scores do not change, and H_128 of O is the same up to
// that order, a permutation of index bits.
//
// Bound: 4 * 64 * 256 * 128 flops per tile take 1024 cycles at the dense f16
// rate, the 2 * 128 * 64 exponentials as long at 16 a cycle, and the operands'
// 128 KB of shared-memory traffic as long at 128 bytes a cycle.  Measured are
// 2100 cycles a tile: 760-780 us for 4 requests of 1500-2048 queries x 32 heads
// over 2000-8192 INT4 keys x 8 heads, 0.53 of cuBLAS's bf16 rate.  What fills
// the rest is the chain of one row's softmax (read S, 64 exponentials, sum,
// convert, write P) against which two groups hide too little, and the switch
// between units (17,000 cycles: 7000 for queries, 6000 for a join, 5000 to
// finish).  The next unit's queries are therefore brought to L2 a unit ahead
// and loaded 64 bytes of a row at a time, and rows leave in 32-byte stores (16
// requests of 512 tokens: 156 -> 140 us, cross attention 165 -> 154 us; now 132
// and 159-164 us).
//
// Every mbarrier wait gives up after about a second: the kernel then records a
// fault (hadq_device_status reads it); every role runs on to its end without
// waiting, without MMAs and without global writes, so that the CTA's named
// barriers stay matched, and frees the TMEM.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "hadq_paged_attn.cuh"
#include "hadq_tc.cuh"

namespace hadq {

constexpr int kPtThreads = 640;
constexpr int kPtRows = 256;  // query rows per unit
constexpr int kPtTile = 64;   // keys per tile
constexpr int kPtStages = 4;  // tiles of K, and of V, in shared memory
constexpr int kPtHalf = 128 * 128;            // bytes of 64 columns of a group's queries
constexpr int kPtMat = 2 * kPtHalf;           // a group's queries in f16
constexpr int kPtKvHalf = 64 * 128, kPtKv = 2 * kPtKvHalf;  // the same of a tile of K or V
constexpr int kPtPlans = 4;   // tiles whose rows and scales are worked out ahead
constexpr int kPtInfos = 16;  // tiles whose info the softmax may still need: 2 ahead of it in S, 4 in K, 4 planned
constexpr int kPtMaxCtas = 160;
constexpr float kPtWeights = 65504.f;  // a row's weights of a tile: f16's largest number
constexpr float kPtSlack = 7.f;        // log2 units its reference may trail then: weights stay below 2^15
constexpr int kPtCounterBase = 1024;          // first of this kernel's arrival counters

// Instruction descriptors: D float32, A and B f16, M = 128.
constexpr uint32_t kPtIdescQK = (1u << 4) | ((64u >> 3) << 17) | ((128u >> 4) << 24);                  // N = 64 keys
constexpr uint32_t kPtIdescPV = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);  // N = 128 columns, B MN-major

// A CTA's units and tiles in order.  Every warp walks its own copy, in shared
// memory: in registers it would be spilled in the loops that matter.
struct PtIter {
  int64_t at, end;     // next tile on the line, end of the CTA's piece
  int64_t ustart;      // first tile of the unit on the line
  PagedReq rq;
  PagedTiles tl;
  int b, h, qt, first, ntok, i0, i1;  // tiles i0 .. i1 - 1 of the unit are this CTA's
  __device__ __forceinline__ void fill(const PagedAttnArgs& a, int per) {
    first = qt * per;
    ntok = min(rq.n - first, per);
    tl = paged_tiles<kPtTile>(a, rq, first, first + ntok - 1);
  }
  __device__ __forceinline__ void cut(int64_t u) {
    i0 = int(u);
    i1 = int(min(int64_t(tl.count), u + (end - at)));
    ustart = at - u;
  }
  __device__ __forceinline__ int key0(int i) const { return (i < tl.head ? i : i - tl.head + tl.from) * kPtTile; }
  __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == tl.count; }
  // The next unit; false at the end of the piece.
  __device__ __forceinline__ bool next(const PagedAttnArgs& a, int per) {
    at += i1 - i0;
    if (at >= end) return false;
    if ((qt + 1) * per < rq.n) {
      ++qt;
    } else {
      qt = 0;
      if (++h == a.nkv) {
        h = 0;
        do {
          rq = paged_req(a, ++b);
        } while (rq.rows == 0);
      }
    }
    fill(a, per);
    cut(0);
    return true;
  }
  // next() by one lane for the whole warp.
  __device__ __forceinline__ bool warp_next(const PagedAttnArgs& a, int per) {
    int ok = 0;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ok = next(a, per);
    __syncwarp();
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
  }
};

struct PtTail {
  uint64_t q_full[2], s_full[2][2], p_full[2][2];  // by group, S buffer
  uint64_t pv_done[2], o_full[2], o_empty[2];
  uint64_t k_full[kPtStages], k_empty[kPtStages], v_full[kPtStages], v_empty[kPtStages];
  uint64_t plan_full[kPtPlans], plan_empty[kPtPlans];
  uint32_t info[kPtInfos];   // of the last tiles: exponents of the largest K scale (bits 0-7) and V scale
                             // (8-15), whether every key is cached (16), lower limit of the next V one (24-31)
  uint32_t ok[kPtInfos][2];  // the tile's keys that are cached
  uint32_t row[kPtPlans][kPtTile];       // rows of the tile's keys in the pool, ~0: not cached
  uint32_t scale[kPtPlans][2][4][kPtTile];  // K and V scales over 2^e as f16 pairs, by group
  int eq[2][128];            // exponents of the groups' rows
  alignas(16) uint32_t flip[64];  // the signs of the 128 columns as masks of bf16 pairs
  int last[2];
  uint32_t tmem_base;
  uint32_t abort;
  PagedPlanSmem plan;
  PtIter it[20], next[8];  // by warp; the softmax warps also look one unit ahead
};
__host__ __device__ constexpr size_t pt_smem_bytes() { return 1024 + 2 * size_t(kPtMat) + 2 * size_t(kPtStages) * kPtKv + sizeof(PtTail); }

// Wait for the phase of `parity`; false after about a second, or as soon as
// another role has given up.  The clock (the SM's own, which is read at once)
// and the abort word are looked at once in 64 tries.
constexpr long long kPtWaitCycles = 2000000000ll;
__device__ __forceinline__ bool pt_wait(uint64_t* b, uint32_t parity, const volatile uint32_t* abort) {
  long long t0 = 0;
  for (uint32_t spin = 1;; ++spin) {
    if (mbar_test(b, parity)) return true;
    if ((spin & 63) == 0) {
      if (abort && *abort) return false;
      const long long now = clock64();
      if (t0 == 0) t0 = now;
      if (now - t0 > kPtWaitCycles) return false;
    }
  }
}

// The upper word of every operand's descriptor: stride 1024 bytes between
// groups of eight rows, version, 128-byte swizzle; the lower words (address,
// leading stride) are all a step has to change.
constexpr uint32_t kPtDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t pt_desc_lo(const void* p, uint32_t lbo) { return ((smem_addr(p) & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); }

// D[tmem] (+)= A B over K = 16, A from shared memory or (ts) from TMEM; the
// lane with `on` issues.  Each issue is predicated by itself: inside a branch
// of one lane the operands would be moved to uniform registers one by one,
// which a busy scheduler makes slower than the product (110 cycles against 64).
__device__ __forceinline__ void pt_mma_ss(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t accumulate, uint32_t on) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %6, 0;\n"
      " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(kPtDescHi), "r"(on)
      : "memory");
}
__device__ __forceinline__ void pt_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t idesc, uint32_t accumulate, uint32_t on) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %6, 0;\n mov.b64 db, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(idesc), "r"(accumulate), "r"(kPtDescHi), "r"(on)
      : "memory");
}
__device__ __forceinline__ void pt_commit(uint64_t* bar, uint32_t on) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(
          smem_addr(bar)),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ void pt_arrive(uint64_t* bar, uint32_t on) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n}" ::"r"(smem_addr(bar)), "r"(on)
      : "memory");
}
#define HADQ_R32 \
  "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, " \
  "%24, %25, %26, %27, %28, %29, %30, %31"
#define HADQ_R64 \
  "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, " \
  "%24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, " \
  "%46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63"
// 32 lanes x 32 or 64 columns of TMEM; the wait is part of the statement.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {" HADQ_R64 "}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
        "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]),
        "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]),
        "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {" HADQ_R32 "};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
               "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
               "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
               "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// Registers of a thread: 640 threads launch with 96 each, 480 for the five
// warps of a scheduler; two softmax warps, a key, a value and the MMA warp
// get 2 * 152 + 2 * 64 + 48.
constexpr int kPtRegsSoftmax = 152, kPtRegsCodes = 64, kPtRegsMma = 48;
static_assert(2 * kPtRegsSoftmax + 2 * kPtRegsCodes + kPtRegsMma <= 5 * 96, "the launch's registers");

// The column (of a group of eight) that a position of the converted operands
// holds, and the other way round.
template <int BITS>
__host__ __device__ constexpr int pt_column(int p) { return BITS == 4 ? ((p & 1) << 2) | (p >> 1) : (p & 4) | ((p & 1) << 1) | ((p >> 1) & 1); }
template <int BITS>
__host__ __device__ constexpr int pt_position(int d) { return BITS == 4 ? ((d & 3) << 1) | (d >> 2) : (d & 4) | ((d & 1) << 1) | ((d >> 1) & 1); }

template <uint32_t V>
struct PtInt {
  static constexpr uint32_t value = V;
};

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void fma2(float& a, float& b, float m, float c) {
  uint64_t X, M, C, R;
  asm("mov.b64 %0, {%1, %2};" : "=l"(X) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %1};" : "=l"(M) : "f"(m));
  asm("mov.b64 %0, {%1, %1};" : "=l"(C) : "f"(c));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(R) : "l"(X), "l"(M), "l"(C));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(R));
}
__device__ __forceinline__ void sum2(float& a, float& b, float x, float y) {
  uint64_t A, X, R;
  asm("mov.b64 %0, {%1, %2};" : "=l"(A) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(X) : "f"(x), "f"(y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(R) : "l"(A), "l"(X));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(R));
}
// 32 bytes in one store, or (at addresses that are multiples of 16 only) in
// two.  A warp's stores touch a line per lane, so half as many cost half.
__device__ __forceinline__ void pt_store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// 2^e for any integer e (0 and the largest power of two outside the range).
__device__ __forceinline__ float pow2_clamped(int e) {
  return __uint_as_float(uint32_t(min(max(e, -126), 127) + 127) << 23);
}

template <int NG, int BITS>
__global__ void __launch_bounds__(kPtThreads, 1) paged_chunk_kernel(const PagedAttnArgs a, unsigned* fault) {
  extern __shared__ uint8_t pt_smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pt_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = base;                // [group][half][128 rows][128 bytes]
  uint8_t* ks = base + 2 * kPtMat;   // [stage][half][64 keys][128 bytes]
  uint8_t* vs = ks + kPtStages * kPtKv;
  PtTail* tl = reinterpret_cast<PtTail*>(vs + kPtStages * kPtKv);
  const volatile uint32_t* abort = &tl->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = kPtRows / a.g;  // query tokens per unit

  // ---- this CTA's piece ----
  auto head_tiles = [&](const PagedReq& r) {
    int64_t s = 0;
    for (int f = 0; f < r.n && r.rows > 0; f += per) s += paged_tiles<kPtTile>(a, r, f, min(r.n, f + per) - 1).count;
    return s;
  };
  const PagedPiece pc = paged_plan(a, tl->plan, [&](int b) { return head_tiles(paged_req(a, b)) * a.nkv; });
  if (pc.at >= pc.end) return;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tl->q_full[i], 4);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&tl->s_full[i][h], 2);
        mbar_init(&tl->p_full[i][h], 4);
      }
      mbar_init(&tl->pv_done[i], 1);
      mbar_init(&tl->o_full[i], 1);
      mbar_init(&tl->o_empty[i], 4);
    }
    for (int i = 0; i < kPtStages; ++i) {
      mbar_init(&tl->k_full[i], 4);
      mbar_init(&tl->k_empty[i], 2);
      mbar_init(&tl->v_full[i], 4);
      mbar_init(&tl->v_empty[i], 2);
    }
    for (int i = 0; i < kPtPlans; ++i) {
      mbar_init(&tl->plan_full[i], 1);
      mbar_init(&tl->plan_empty[i], 8);
    }
    tl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 64) tl->flip[tid] = a.signs ? pair_sign_mask(a.signs[2 * tid], a.signs[2 * tid + 1]) : 0u;
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tl->tmem_base)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // All 512 columns are this CTA's, so they start at column 0, at constant
  // addresses: S of group 0 and 1 (two buffers of 64 columns each), then O.
  constexpr uint32_t tmem = 0;

  if (lane == 0) {
    PtIter f;
    f.at = pc.at;
    f.end = pc.end;
    f.b = pc.b;
    f.rq = paged_req(a, pc.b);
    const int64_t ph = head_tiles(f.rq);
    f.h = int(pc.in_request / ph);
    int64_t u = pc.in_request - f.h * ph;
    f.qt = 0;
    for (;;) {
      f.fill(a, per);
      if (u < f.tl.count) break;
      u -= f.tl.count;
      ++f.qt;
    }
    f.cut(u);
    tl->it[warp] = f;
    if (warp < 8) tl->next[warp] = f;
  }
  __syncwarp();

  if (warp < 8) {
    // =============================================== softmax, queries, output
    regs_inc<kPtRegsSoftmax>();
    const int m = warp >> 2, r = tid & 127;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t tO = tmem + lanes + uint32_t(256 + 128 * m);
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!pt_wait(bar, parity, abort)) {
        if (!dead) tc_give_up(&tl->abort, fault);
        dead = true;
      }
    };
    int eq = 0;  // this row's query is scaled by 2^eq
    uint32_t n = 0, ns = 0, nu = 0;  // tiles of the CTA, tiles and units of this group
    bool active = false;             // the group has rows in unit `it`
    float M = -INFINITY, l = 0.f;
    PtIter &it = tl->it[warp], &nx = tl->next[warp];

    // A warp rotates its 32 rows 16 at a time: four of the seven stages as an
    // exact bf16 product with H_16 (lane (g, j) holds columns 32 i + 8 j .. + 7,
    // i = 0 .. 3, of rows g and g + 8, so that a load covers 64 bytes of a row),
    // three in registers.  Each row
    // is scaled by the exponent of a bound of its entries, 128 times its
    // largest input.
    auto load_queries = [&](const PtIter& u) {
      const int g = lane >> 2, j = lane & 3;
      uint32_t bm[2][2];
#pragma unroll
      for (int c = 0; c < 2; ++c) h16_operand(g, j, c, 0x3F80u, bm[c]);
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        const int r0 = 32 * (warp & 3) + 16 * pass + g;  // rows r0, r0 + 8 of the group
        uint4 in[2][4];
        float up[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = 128 * m + r0 + 8 * x;
          const int tok = a.by_g.div(row), hh = row - tok * a.g;
          const bool live = row < u.ntok * a.g;
          const uint4* p = reinterpret_cast<const uint4*>(
              a.q + (live ? int64_t(u.rq.row0 + u.first + tok) * a.q_stride + int64_t(u.h * a.g + hh) * kPagedDim + 8 * j : 0));
#pragma unroll
          for (int i = 0; i < 4; ++i) in[x][i] = live ? __ldg(p + 4 * i) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t top = 0;  // largest magnitudes of the even and the odd columns, as bf16 bits
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            top = __vmaxu2(top, in[x][i].x & 0x7FFF7FFFu);
            top = __vmaxu2(top, in[x][i].y & 0x7FFF7FFFu);
            top = __vmaxu2(top, in[x][i].z & 0x7FFF7FFFu);
            top = __vmaxu2(top, in[x][i].w & 0x7FFF7FFFu);
          }
          uint32_t mx = max(top & 0xFFFFu, top >> 16);
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // the bound to [2^14, 2^15); a row whose entries are all below 2^-100
          // counts as zero, one that is not finite as NaN (an infinity alone
          // could give every key the score -infinity, which reads as unseen)
          const float bound = __uint_as_float(mx << 16) * 128.f * a.qmul;
          const int be = min(int(__float_as_uint(bound) >> 23), 253);
          const int e = be < 27 ? 0 : 141 - be;
          up[x] = mx >= 0x7F80u ? NAN : be < 27 ? 0.f : a.qmul * pow2_clamped(e);
          if (j == 0) tl->eq[m][r0 + 8 * x] = e;
        }
        float v[2][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[2][4];
          const uint4 flip = *reinterpret_cast<const uint4*>(&tl->flip[16 * i + 4 * j]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
              w[x][k] = (k == 0 ? in[x][i].x ^ flip.x : k == 1 ? in[x][i].y ^ flip.y : k == 2 ? in[x][i].z ^ flip.z : in[x][i].w ^ flip.w);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_h16_bf16(d, w[0][2 * h], w[1][2 * h], w[0][2 * h + 1], w[1][2 * h + 1], bm[c][0], bm[c][1]);
              v[0][8 * i + 4 * h + 2 * c] = d[0];
              v[0][8 * i + 4 * h + 2 * c + 1] = d[1];
              v[1][8 * i + 4 * h + 2 * c] = d[2];
              v[1][8 * i + 4 * h + 2 * c + 1] = d[3];
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          reg_stage<32, 4>(v[x]);
          reg_stage<32, 8>(v[x]);
          reg_stage<32, 16>(v[x]);
#pragma unroll
          for (int i = 0; i < 32; i += 2) mul2(v[x][i], v[x][i + 1], up[x]);
          const int r = r0 + 8 * x;
          uint8_t* dst = qs + m * kPtMat + r * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = cvt_f16x2(v[x][8 * i + pt_column<BITS>(2 * k)], v[x][8 * i + pt_column<BITS>(2 * k + 1)]);
            *reinterpret_cast<uint4*>(dst + (i >> 1) * kPtHalf + (((4 * (i & 1) + j) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      fence_async_shared();
      named_bar_sync(1 + m, 128);  // the group's rows are written
      if (lane == 0) mbar_arrive(&tl->q_full[m]);
      eq = tl->eq[m][r];
    };

    // The unit's partial O to the workspace; the last CTA to come sums them up
    // and leaves the total in TMEM.  Returns whether this one does.
    auto join = [&]() {
      const int row = 128 * m + r;
      const int c0 = int(it.ustart / pc.quota), c1 = int((it.ustart + it.tl.count - 1) / pc.quota);
      auto slot = [&](int x) { return 2 * int64_t(x) + (x == c0 ? 1 : 0); };
      float4* po = reinterpret_cast<float4*>(a.part_o);
      float2* pm = reinterpret_cast<float2*>(a.part_ml);
      const int64_t mine = slot(int(blockIdx.x));
      if (!dead) pm[mine * kPtRows + row] = make_float2(M, l);
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        float o[32];
        tmem_ld32(tO + 32 * q, o);
        if (!dead) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            po[(mine * 32 + 8 * q + c) * kPtRows + row] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
      }
      __threadfence();
      named_bar_sync(1 + m, 128);
      if (r == 0) tl->last[m] = !dead && atomicAdd(a.counters + kPtCounterBase + 2 * c0 + m, 1u) == unsigned(c1 - c0);
      named_bar_sync(1 + m, 128);
      if (!tl->last[m]) return false;
      __threadfence();
      M = -INFINITY;
      for (int x = c0; x <= c1; ++x) M = fmaxf(M, __ldcg(&pm[slot(x) * kPtRows + row]).x);
      l = 0.f;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        float o[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0.f;
#pragma unroll 1
        for (int x = c0; x <= c1; ++x) {
          const float2 ml = __ldcg(&pm[slot(x) * kPtRows + row]);
          const float root = ml.x == -INFINITY ? 0.f : exp2f(0.5f * (ml.x - M)), w = root * root;
          if (q == 0) l = fmaf(root, root * ml.y, l);
          const float4* px = po + (slot(x) * 32 + 8 * q) * kPtRows + row;
          float4 v[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = __ldcg(px + c * kPtRows);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            o[4 * c] = fmaf(w, v[c].x, o[4 * c]);
            o[4 * c + 1] = fmaf(w, v[c].y, o[4 * c + 1]);
            o[4 * c + 2] = fmaf(w, v[c].z, o[4 * c + 2]);
            o[4 * c + 3] = fmaf(w, v[c].w, o[4 * c + 3]);
          }
        }
        uint32_t y[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(o[k]);
        tmem_st32(tO + 32 * q, y);
      }
      tmem_wait_st();
      if (r == 0) a.counters[kPtCounterBase + 2 * c0 + m] = 0u;  // ready for the next call
      return true;
    };

    // Rotate back (64 columns at a time), normalise, sign, store.
    auto finish = [&]() {
      const int row = 128 * m + r;
      const bool store = row < it.ntok * a.g && !dead;
      const float inv = l > 0.f ? a.inv_sqrt_dim * 0.0078125f / l : 0.f;  // values entered times 2^7
      const int tok = a.by_g.div(row), hh = row - tok * a.g;
      const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
      uint4* dst = reinterpret_cast<uint4*>(a.out + (int64_t(it.rq.row0 + it.first + tok) * a.nqh + it.h * a.g + hh) * kPagedDim);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float y[64];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float w[32];
          tmem_ld32(tO + 32 * q, *reinterpret_cast<float(*)[32]>(y + 32 * q));
          tmem_ld32(tO + 64 + 32 * q, w);
          const float sg = h ? -1.f : 1.f;
#pragma unroll
          for (int k = 0; k < 32; ++k) y[32 * q + k] = fmaf(w[k], sg, y[32 * q + k]);
        }
        reg_fwht<64, 6>(y);
        if (store) {
#pragma unroll
          for (int k = 0; k < 64; k += 2) mul2(y[k], y[k + 1], inv);
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 16 columns, 32 bytes
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float* z = y + 16 * c + 8 * (k >> 2);
              w[k] = cvt_bf16x2(z[pt_position<BITS>(2 * (k & 3))], z[pt_position<BITS>(2 * (k & 3) + 1)]) ^ tl->flip[32 * h + 8 * c + k];
            }
            pt_store32(dst + 8 * h + 2 * c, w, wide);
          }
        }
      }
    };

    for (bool more = true;;) {
      // ---- the next unit's queries, then the output of the unit just done ----
      const bool next_active = more && 128 * m < nx.ntok * a.g;
      if (next_active) load_queries(nx);
      if (active) {
        wait(&tl->o_full[m], nu & 1);
        ++nu;
        tc_fence_after();
        if (it.whole() || join()) finish();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tl->o_empty[m]);
      }
      if (!more) break;
      __syncwarp();
      if (lane == 0) it = nx;
      more = nx.warp_next(a, per);  // (looked up while this unit runs)
      if (more && 128 * m + r < nx.ntok * a.g) {  // its queries to L2: a row per thread
        const int row = 128 * m + r, tok = a.by_g.div(row);
        const uint16_t* p = a.q + int64_t(nx.rq.row0 + nx.first + tok) * a.q_stride + int64_t(nx.h * a.g + row - tok * a.g) * kPagedDim;
        asm volatile("prefetch.global.L2 [%0];\n prefetch.global.L2 [%0 + 128];" ::"l"(p));
      }
      active = next_active;
      M = -INFINITY;
      l = 0.f;
      bool fresh = true;  // some row of the warp has no reference
      if (active) {
        const int off = it.rq.len - it.rq.n;
        const int row = min(128 * m + r, it.ntok * a.g - 1), tok = it.first + int(a.by_g.div(row));
        const int lim = a.causal ? min(it.rq.len, off + tok + 1) : it.rq.len;
        const int low = a.window > 0 ? off + tok - a.window + 1 : 0;
        // keys that every row of the group sees: below all_lim, from all_low on
        const int f_tok = it.first + int(a.by_g.div(128 * m)), l_tok = it.first + int(a.by_g.div(min(128 * m + 127, it.ntok * a.g - 1)));
        const int all_lim = a.causal ? off + f_tok + 1 : it.rq.len;
        const int all_low = a.window > 0 ? off + l_tok - a.window + 1 : 0;
        const int i0 = it.i0, i1 = it.i1, head = it.tl.head, from = it.tl.from - head;
#pragma unroll 1
        for (int i = i0; i < i1; ++i, ++ns, ++n) {
          const int t0 = (i < head ? i : i + from) * kPtTile;
          const uint32_t h = ns & 1;  // S buffer
          const uint32_t tS = tmem + lanes + uint32_t(128 * m) + 64 * h;
          bool masked = t0 + kPtTile > all_lim || (a.window > 0 && t0 < all_low);
          wait(&tl->s_full[m][h], (ns >> 1) & 1);
          tc_fence_after();
          const uint32_t info = tl->info[n % kPtInfos];
          masked |= (info & 0x10000u) == 0;
          if (masked) {  // put -inf where a row sees nothing
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const int tc = t0 + 16 * c;
              auto below = [](int x) { return x <= 0 ? 0u : x >= 16 ? 0xffffu : (1u << x) - 1u; };
              uint32_t see = (tl->ok[n % kPtInfos][c >> 1] >> (16 * (c & 1))) & below(lim - tc);
              if (a.window > 0) see &= ~below(low - tc) | below(a.sinks - tc);
              uint32_t y[16];
              tmem_ld16(tS + 16 * c, y);
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = (see >> k) & 1u ? y[k] : 0xff800000u;
              tmem_st16(tS + 16 * c, y);
            }
            tmem_wait_st();
          }
          uint32_t s[64];
          tmem_ld64(tS, s);
          const float f = pow2_clamped(int(info & 255u) - 134 - eq), vexp = float(int((info >> 8) & 255u) - 127);
          // The weights come first, on the reference as it stands, and no
          // maximum is taken: a row whose weights sum to no more than
          // kPtWeights has none above it.  Where a row's do not, or it has no
          // reference yet, the warp takes the maxima, raises references,
          // rescales O and does the weights again.
          uint32_t p[32];
          float sum = 0.f;
          for (bool fix = fresh;;) {
            float x[64];
#pragma unroll
            for (int k = 0; k < 64; ++k) x[k] = __uint_as_float(s[k]);
            if (fix) {
              float top = x[0];
#pragma unroll
              for (int k = 1; k < 63; k += 2) top = max3(top, x[k], x[k + 1]);
              top = fmaf(fmaxf(top, x[63]), f, vexp - kPagedRoom);
              // (a row that brought the warp here gets its own maximum, so that
              // the tiles after do not: 64 weights of 2^8 stay below kPtWeights)
              const bool need = top > M + kPtSlack || sum > kPtWeights;
              const float root = need ? exp2f(0.5f * (M - top)) : 1.f, alpha = root * root;
              if (need) M = top;
              l = l * root * root;
              // (but for rows that see nothing further on, and those of NaN)
              fresh = __any_sync(0xffffffffu, M == -INFINITY && lim > t0 + kPtTile && top == top);
              if (i > i0 && __any_sync(0xffffffffu, need)) {
                wait(&tl->pv_done[m], (ns - 1) & 1);  // the tile before; S came after the one before that
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                  uint32_t o[16];
                  tmem_ld16(tO + 16 * c, o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                  tmem_st16(tO + 16 * c, o);
                }
              }
            }
            const float sub = M == -INFINITY ? 0.f : vexp - M;
            float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
            for (int k = 0; k < 64; k += 2) fma2(x[k], x[k + 1], f, sub);
#pragma unroll
            for (int k = 0; k < 64; ++k) x[k] = exp2_ftz(x[k]);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if (k & 1) sum2(l2, l3, x[2 * k], x[2 * k + 1]); else sum2(l0, l1, x[2 * k], x[2 * k + 1]);
              p[k] = cvt_f16x2(x[2 * k], x[2 * k + 1]);
            }
            sum = (l0 + l1) + (l2 + l3);
            if (fix) break;
            fix = __any_sync(0xffffffffu, sum > kPtWeights);
            if (!fix) break;
            tmem_ld64(tS, s);
          }
          tmem_st32(tS + 32, p);
          l = fmaf(sum, pow2_clamped(127 - int((info >> 8) & 255u)), l);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tl->p_full[m][h]);
        }
      } else {
        n += it.i1 - it.i0;
      }
    }
  } else if (warp < 16) {
    // ======================================================= keys and values
    regs_dec<kPtRegsCodes>();
    const int role = (warp - 8) >> 2;  // 0: keys, 1: values
    const int t = tid & 127, key = t >> 1, part = t & 1;  // two threads per row, 64 columns each
    constexpr int RB = 16 * BITS, NV = RB / 32;           // 16-byte pieces per half row
    constexpr int NS = NG == 4 ? 2 : 1;                   // scales per half row
    const uint8_t* codes = (role ? a.v_codes : a.k_codes) + part * (RB / 2);
    uint64_t* full = role ? tl->v_full : tl->k_full;
    uint64_t* empty = role ? tl->v_empty : tl->k_empty;
    uint8_t* mat = (role ? vs : ks) + part * kPtKvHalf + key * 128;
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!pt_wait(bar, parity, abort)) {
        if (!dead) tc_give_up(&tl->abort, fault);
        dead = true;
      }
    };
    const F16Magic magic;
    uint4 cur[NV];
    // The codes of tile n's row, once it is planned.  The second threads of
    // the rows take their eight-column pieces four further on (mod 8) than the
    // first: the four rows x two halves that a 128-bit store pass covers then
    // lie in different banks.
    auto load = [&](uint32_t n) {
      wait(&tl->plan_full[n % kPtPlans], (n / kPtPlans) & 1);
      const uint32_t row = tl->row[n % kPtPlans][key];
      const uint4* src = reinterpret_cast<const uint4*>(codes + int64_t(row) * RB);
#pragma unroll
      for (int x = 0; x < NV; ++x) cur[x] = row != ~0u && !dead ? __ldg(src + (x ^ (part * (NV / 2)))) : make_uint4(0u, 0u, 0u, 0u);
    };
    load(0);
    const uint32_t sw = uint32_t((key & 7) ^ (part << 2)) << 4;
    const uint32_t total = uint32_t(pc.end - pc.at);
#pragma unroll 1
    for (uint32_t n = 0; n < total; ++n) {
      const int st = n & (kPtStages - 1);
      uint32_t sc[NS];
#pragma unroll
      for (int q = 0; q < NS; ++q) {  // (in the order of the pieces)
        const int grp = NG == 1 ? 0 : NG == 2 ? part : 2 * part + (q ^ part);
        sc[q] = tl->scale[n % kPtPlans][role][grp][key];
      }
      wait(&empty[st], ((n / kPtStages) & 1) ^ 1u);
      uint8_t* dst = mat + st * kPtKv;
#pragma unroll 1
      for (int c4 = 0; c4 < 2; ++c4) {  // 32 columns: the front pieces of cur, which then moves up
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t p[4];
          if constexpr (BITS == 4) {
            i4x4_to_f16_tokens(x == 0 ? cur[0].x : x == 1 ? cur[0].y : x == 2 ? cur[0].z : cur[0].w, magic, p);
          } else {
            const uint4 v = cur[x >> 1];
            const uint32_t w0 = (x & 1) ? v.z : v.x, w1 = (x & 1) ? v.w : v.y;
            // bytes with the sign bit flipped are code + 128: 1152 + code
            p[0] = f16x2_sub(and_xor<0x00FF00FFu>(w0, magic.m8), magic.m8);
            p[1] = f16x2_sub(and_xor<0x00FF00FFu>(w0 >> 8, magic.m8), magic.m8);
            p[2] = f16x2_sub(and_xor<0x00FF00FFu>(w1, magic.m8), magic.m8);
            p[3] = f16x2_sub(and_xor<0x00FF00FFu>(w1 >> 8, magic.m8), magic.m8);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) p[y] = f16x2_mul(p[y], sc[0]);
          *reinterpret_cast<uint4*>(dst + (sw ^ uint32_t((4 * c4 + x) << 4))) = make_uint4(p[0], p[1], p[2], p[3]);
        }
#pragma unroll
        for (int x = 0; x < NV / 2; ++x) cur[x] = cur[x + NV / 2];
        sc[0] = sc[NS - 1];
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[st]);
        mbar_arrive(&tl->plan_empty[n % kPtPlans]);
      }
      if (n + 1 < total) load(n + 1);
    }
  } else {
    regs_dec<kPtRegsMma>();
    if (warp >= 18) {
      // ============================================================= plan
      // Two warps, every other tile each: where the tile's rows are, their
      // scales, the largest one's exponent.  Two keys per lane.
      bool dead = false;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!pt_wait(bar, parity, abort)) {
          if (!dead) tc_give_up(&tl->abort, fault);
          dead = true;
        }
      };
      PtIter& it = tl->it[warp];
      int i = it.i0;
      const uint32_t total = uint32_t(pc.end - pc.at);
#pragma unroll 1
      for (uint32_t n = 0; n < total; ++n) {
        if (int(n & 1) == warp - 18) {
          const uint32_t sl = n % kPtPlans;
          const int t0 = it.key0(i) + lane;
          uint32_t row[2];
          float sc[2][2][NG], top[2] = {0.f, 0.f};
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int pos = t0 + 32 * x;
            int page = -1;
            if (pos < it.tl.kv_end) page = __ldg(a.table + int64_t(it.b) * a.max_pages + (pos >> a.page_log2));
            // (the rows of one tensor on one GPU are fewer than 2^32)
            row[x] = unsigned(page) < unsigned(a.n_pages)
                         ? uint32_t(((int64_t(page) * a.nkv + it.h) << a.page_log2) + (pos & ((1 << a.page_log2) - 1)))
                         : ~0u;
          }
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int q = 0; q < NG; ++q) {
              const float k = row[x] != ~0u ? __ldg(a.k_scales + int64_t(row[x]) * NG + q) : 0.f;
              // signed; what one past 2^96 or not finite gives is open, but it
              // must not set the tile's exponent, which all queries share
              sc[0][x][q] = fabsf(k) <= 7.9228163e28f ? k : 0.f;
              sc[1][x][q] = row[x] != ~0u ? clean_scale(__ldg(a.v_scales + int64_t(row[x]) * NG + q)) : 0.f;
              top[0] = fmaxf(top[0], fabsf(sc[0][x][q]));
              top[1] = fmaxf(top[1], sc[1][x][q]);
            }
          int e[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) e[y] = min(max(int(__reduce_max_sync(0xffffffffu, __float_as_uint(top[y])) >> 23), 27), kPagedExpHigh);
          int low = kPagedExpLow;
          if (n > 0) {
            // The tile before, of the other warp: for its limit, and (at a
            // unit's first tile too) so that neither warp gets two of its tiles
            // ahead of the other's next, where this barrier's phase would have
            // passed before it is looked at.
            wait(&tl->plan_full[(n - 1) % kPtPlans], ((n - 1) / kPtPlans) & 1);
            if (i > it.i0) low = int(tl->info[(n - 1) % kPtInfos] >> 24);
          }
          e[1] = max(e[1], low);
          low = max(low, e[1] - kPagedExpSpan);
          const uint32_t ok0 = __ballot_sync(0xffffffffu, row[0] != ~0u), ok1 = __ballot_sync(0xffffffffu, row[1] != ~0u);
          wait(&tl->plan_empty[sl], ((n / kPtPlans) & 1) ^ 1u);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            tl->row[sl][lane + 32 * x] = row[x];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float up = pow2_clamped(134 - e[y]);  // the largest scale to [2^7, 2^8)
#pragma unroll
              for (int q = 0; q < NG; ++q) tl->scale[sl][y][q][lane + 32 * x] = cvt_f16x2(sc[y][x][q] * up, sc[y][x][q] * up);
            }
          }
          if (lane == 0) {
            tl->ok[n % kPtInfos][0] = ok0;
            tl->ok[n % kPtInfos][1] = ok1;
            tl->info[n % kPtInfos] = uint32_t(e[0]) | (uint32_t(e[1]) << 8) | ((ok0 & ok1) == ~0u ? 1u << 16 : 0u) | (uint32_t(low) << 24);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&tl->plan_full[sl]);
        }
        if (++i == it.i1) {
          (void)it.warp_next(a, per);
          i = it.i0;
        }
      }
    } else {
    // ================================================================== MMAs
    // One warp per group: the control code between the issues takes as long as
    // the products (one warp for both was busy five cycles of six).
    // The whole warp walks the schedule, one lane issues.  Descriptors and
    // TMEM addresses are sums of warp-uniform bases and constants (group and
    // stage unrolled), so that an issue costs no moves to uniform registers.
    uint32_t on = elect_one();  // this lane issues, until a wait has run out
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!pt_wait(bar, parity, abort)) {
        if (on) tc_give_up(&tl->abort, fault);
        on = 0;
      }
    };
    const uint32_t qd = pt_desc_lo(qs, 16), kd = pt_desc_lo(ks, 16), vd = pt_desc_lo(vs, kPtKvHalf);
    PtIter& it = tl->it[warp];
    const int m = __shfl_sync(0xffffffffu, warp, 0) - 16;  // (uniform to the compiler)
    const uint32_t qm = qd + uint32_t(m) * (kPtMat >> 4), sm = uint32_t(128 * m), om = uint32_t(256 + 128 * m);
    uint32_t n = 0, ns = 0, pu = 0;  // tiles of the CTA and of the group; parity of the group's units
    auto stage = [](uint32_t t) { return t & (kPtStages - 1); };
    auto phase = [](uint32_t t) { return (t / kPtStages) & 1; };
    do {
      const bool active = __shfl_sync(0xffffffffu, int(it.ntok * a.g > 128 * m), 0);
      const int tiles = __shfl_sync(0xffffffffu, it.i1 - it.i0, 0);
      if (!active) {  // the stages pass unused
#pragma unroll 1
        for (int i = 0; i < tiles; ++i, ++n) {
          wait(&tl->k_full[stage(n)], phase(n));
          pt_arrive(&tl->k_empty[stage(n)], on);
          wait(&tl->v_full[stage(n)], phase(n));
          pt_arrive(&tl->v_empty[stage(n)], on);
        }
        continue;
      }
      // Step j: O += P V of tile j, then S of tile j + 2 in P's place.
#pragma unroll 1
      for (int j = -2; j < tiles; ++j) {
        const uint32_t h = (ns + uint32_t(j)) & 1;  // S buffer of both tiles
        const uint32_t vt = n + uint32_t(j), kt = vt + 2;
        if (j >= 0) {
          wait(&tl->v_full[stage(vt)], phase(vt));
          if (j == 0) wait(&tl->o_empty[m], pu ^ 1u);
          wait(&tl->p_full[m][h], ((ns + uint32_t(j)) >> 1) & 1);
          tc_fence_after();
          const uint32_t av = sm + 64 * h + 32, bv = vd + stage(vt) * (kPtKv >> 4);
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k) pt_mma_ts(om, av + 8 * k, bv + k * (2048 >> 4), kPtIdescPV, k > 0 ? 1u : uint32_t(j > 0), on);
          pt_commit(&tl->pv_done[m], on);
          pt_commit(&tl->v_empty[stage(vt)], on);
        }
        if (j + 2 < tiles) {
          if (j == -2) wait(&tl->q_full[m], pu);
          wait(&tl->k_full[stage(kt)], phase(kt));
          tc_fence_after();
          const uint32_t bk = kd + stage(kt) * (kPtKv >> 4);
#pragma unroll
          for (uint32_t k = 0; k < 8; ++k)
            pt_mma_ss(sm + 64 * h, qm + (((k >> 2) * kPtHalf + (k & 3) * 32) >> 4), bk + (((k >> 2) * kPtKvHalf + (k & 3) * 32) >> 4), kPtIdescQK, k > 0, on);
          // The softmax reads what the key warps wrote beside the keys
          // (exponents, cached bits) once S is there: this warp has seen their
          // arrival and passes it on.  (They cannot wait for k_full
          // themselves: it may be a phase further on by then.)
          pt_arrive(&tl->s_full[m][h], on);
          pt_commit(&tl->s_full[m][h], on);
          pt_commit(&tl->k_empty[stage(kt)], on);
        }
      }
      pt_commit(&tl->o_full[m], on);
      n += uint32_t(tiles);
      ns += uint32_t(tiles);
      pu ^= 1;
    } while (it.warp_next(a, per));
    // every MMA is complete before TMEM is freed (passes at once normally)
    if (on) (void)pt_wait(&tl->v_empty[stage(n - 1)], phase(n - 1), nullptr);
    __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace hadq
