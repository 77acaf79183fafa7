// Attention over the paged cache for many query rows (prompt chunks, cross
// attention): both products on the fifth-generation tensor cores.
//
// A unit is up to 256 query rows (two M = 128 tiles, groups 0 and 1) of one
// request and KV head; its keys come in tiles of 128.  Per tile and group
//     S = Q K^T    (A = Q, B = K from shared memory, S in TMEM),
//     O += P V     (A = P in TMEM, where it overwrites S; B = V),
// eight tcgen05.mma of K = 16 each, all operands f16:
//  * keys and values are codes times their scale over 2^e, e the exponent of
//    the tile's largest scale, so both fill the f16 range from the top
//    whatever the scales are.  A key is rounded once (scale in two f16 terms,
//    fma), a value twice (scale and product): 11 bits, where the output has 8;
//  * the rotated query is scaled by the exponent of its group's largest entry;
//  * the exponents come back as one multiplier per tile in the exponent's fma
//    (scores) and as a summand of the softmax reference (values): with
//    m >= max(score + e), a weight is 2^(score + e - m) <= 2^8, and l counts
//    2^-e of it.  The reference rises only by more than 2^8, so that O, in
//    TMEM, is rarely rescaled.  m, l and O are float32.
//
// Roles (one CTA per SM, 512 threads, registers dealt by setmaxnreg):
//  * warps 0-3 and 4-7: softmax of group 0 and 1, a row per thread.  They also
//    rotate the next unit's queries into shared memory (H_128 in registers)
//    before they finish a unit (rotate back, normalise, store);
//  * warps 8-11: a key per thread: load codes one tile ahead into registers,
//    convert, scale and store them in the swizzled layout both products read
//    (K: K-major, V: MN-major; the same bytes);
//  * warp 12: one thread issues the MMAs.  Group 0's softmax runs under group
//    1's MMAs and the other way round.
// The columns of Q, K, V are stored in the order in which one mask finds
// them, dim 8 c + (0, 4, 1, 5, 2, 6, 3, 7): scores do not change, and H_128 of
// O is the same up to that order.
//
// Bound: 4 * 128 * 256 * 128 flops per tile pair take 2048 cycles at the dense
// f16 rate; the 2 * 128 * 128 exponentials take as long at 16 a cycle, and
// the operands' 256 KB of shared-memory traffic as long at 128 bytes a cycle.
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

constexpr int kPtThreads = 512;
constexpr int kPtRows = 256;  // query rows per unit
constexpr int kPtTile = 128;  // keys per tile
constexpr int kPtHalf = 128 * 128;            // bytes of 64 columns x 128 rows
constexpr int kPtMat = 2 * kPtHalf;           // one f16 128 x 128 operand
constexpr int kPtMaxCtas = 160;
constexpr int kPtCounterBase = 1024;          // first of this kernel's arrival counters

// Instruction descriptors: D float32, A and B f16, M = N = 128.
constexpr uint32_t kPtIdescQK = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kPtIdescPV = kPtIdescQK | (1u << 16);  // B MN-major

struct PtTail {
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  int kexp[4], vexp[4];     // exponents of the last four tiles' scales
  uint32_t ok[4][4];        // keys of the tile that are cached (bit per key)
  uint32_t red[2][4];       // group maxima of |q|
  uint32_t dred[2][2][4];   // tile maxima of the scales: [parity][K, V][warp]
  uint32_t sgn[4];          // sign bits of the 128 columns
  int last[2];
  uint32_t tmem_base;
  uint32_t abort;
  PagedPlanSmem plan;
};
static_assert(offsetof(PtTail, ok) % 16 == 0, "the cached bits are read as 16-byte vectors");
__host__ __device__ constexpr size_t pt_smem_bytes() { return 1024 + size_t(6) * kPtMat + sizeof(PtTail); }

// D[tmem] (+)= A[tmem] B over K = 16.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
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

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

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
// 2^e for any integer e (0 and the largest power of two outside the range).
__device__ __forceinline__ float pow2_clamped(int e) {
  return __uint_as_float(uint32_t(min(max(e, -126), 127) + 127) << 23);
}

// A CTA's units and tiles in order; every role walks its own copy.
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
};

template <int NG, int BITS>
__global__ void __launch_bounds__(kPtThreads, 1) paged_chunk_kernel(const PagedAttnArgs a, unsigned* fault) {
  extern __shared__ uint8_t pt_smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pt_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = base;                // [group][half][128 rows][128 bytes]
  uint8_t* ks = base + 2 * kPtMat;   // [stage][half][128 keys][128 bytes]
  uint8_t* vs = base + 4 * kPtMat;
  PtTail* tl = reinterpret_cast<PtTail*>(base + 6 * kPtMat);
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
      mbar_init(&tl->s_full[i], 2);
      mbar_init(&tl->p_full[i], 4);
      mbar_init(&tl->o_full[i], 1);
      mbar_init(&tl->o_empty[i], 4);
      mbar_init(&tl->k_full[i], 4);
      mbar_init(&tl->k_empty[i], 1);
      mbar_init(&tl->v_full[i], 4);
      mbar_init(&tl->v_empty[i], 1);
    }
    tl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp < 4) {
    const uint32_t bits = __ballot_sync(0xffffffffu, a.signs && a.signs[tid] < 0);
    if (lane == 0) tl->sgn[warp] = bits;
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tl->tmem_base)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tl->tmem_base;  // S0, S1, O0, O1: 128 columns each

  PtIter it;
  it.at = pc.at;
  it.end = pc.end;
  it.b = pc.b;
  it.rq = paged_req(a, pc.b);
  {
    const int64_t ph = head_tiles(it.rq);
    it.h = int(pc.in_request / ph);
    int64_t u = pc.in_request - it.h * ph;
    it.qt = 0;
    for (;;) {
      it.fill(a, per);
      if (u < it.tl.count) break;
      u -= it.tl.count;
      ++it.qt;
    }
    it.cut(u);
  }

  if (warp < 8) {
    // =============================================== softmax, queries, output
    regs_inc<176>();
    const int m = warp >> 2, r = tid & 127;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes + uint32_t(128 * m), tO = tmem + lanes + uint32_t(256 + 128 * m);
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!mbar_wait(bar, parity, abort)) {
        if (!dead) tc_give_up(&tl->abort, fault);
        dead = true;
      }
      dead = __any_sync(0xffffffffu, dead);
    };
    int eq = 0;  // the group's queries are scaled by 2^eq

    auto load_queries = [&](const PtIter& u) {
      float x[128];
      const int row = 128 * m + r;
      if (row < u.ntok * a.g) {
        const int tok = row / a.g, hh = row - tok * a.g;
        const uint4* p = reinterpret_cast<const uint4*>(a.q + int64_t(u.rq.row0 + u.first + tok) * a.q_stride + int64_t(u.h * a.g + hh) * kPagedDim);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint4 w = __ldg(p + c);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[8 * c + 2 * k] = bf16lo(ww[k]);
            x[8 * c + 2 * k + 1] = bf16hi(ww[k]);
          }
        }
        if (a.signs) {
#pragma unroll
          for (int i = 0; i < 128; ++i) x[i] = __uint_as_float(__float_as_uint(x[i]) ^ (((tl->sgn[i >> 5] >> (i & 31)) & 1u) << 31));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 128; ++i) x[i] = 0.f;
      }
      reg_fwht<128, 7>(x);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 128; ++i) top = fmaxf(top, fabsf(x[i]));
      const uint32_t wt = __reduce_max_sync(0xffffffffu, __float_as_uint(top * a.qmul));
      if (lane == 0) tl->red[m][warp & 3] = wt;
      named_bar_sync(1 + m, 128);
      const uint32_t gt = max(max(tl->red[m][0], tl->red[m][1]), max(tl->red[m][2], tl->red[m][3]));
      // largest entry to [2^13, 2^14); a group whose entries are all below
      // 2^-100 counts as zero
      const int ge = min(int(gt >> 23), 253);
      const bool zero = ge < 27;
      eq = zero ? 0 : 140 - ge;
      const float up = zero ? 0.f : a.qmul * pow2_clamped(eq);
      uint8_t* dst = qs + m * kPtMat + r * 128;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float* y = x + 8 * c;
        const uint4 w = make_uint4(cvt_f16x2(y[0] * up, y[4] * up), cvt_f16x2(y[1] * up, y[5] * up), cvt_f16x2(y[2] * up, y[6] * up),
                                   cvt_f16x2(y[3] * up, y[7] * up));
        *reinterpret_cast<uint4*>(dst + (c >> 3) * kPtHalf + (((c & 7) ^ (r & 7)) << 4)) = w;
      }
      fence_async_shared();
      named_bar_sync(1 + m, 128);  // tl->red has been read; the group's rows are written
      if (lane == 0) mbar_arrive(&tl->q_full[m]);
    };

    if (128 * m < it.ntok * a.g) load_queries(it);
    uint32_t n = 0, ns = 0, nu = 0;  // tiles of the CTA, tiles and units of this group
    for (bool more = true; more;) {
      const bool active = 128 * m < it.ntok * a.g;
      float M = -INFINITY, l = 0.f;
      if (active) {
        const int off = it.rq.len - it.rq.n;
        const int row = min(128 * m + r, it.ntok * a.g - 1), tok = it.first + row / a.g;
        const int lim = a.causal ? min(it.rq.len, off + tok + 1) : it.rq.len;
        const int low = a.window > 0 ? off + tok - a.window + 1 : 0;
        // keys that every row of the group sees: below all_lim, from all_low on
        const int f_tok = it.first + 128 * m / a.g, l_tok = it.first + min(128 * m + 127, it.ntok * a.g - 1) / a.g;
        const int all_lim = a.causal ? off + f_tok + 1 : it.rq.len;
        const int all_low = a.window > 0 ? off + l_tok - a.window + 1 : 0;
        for (int i = it.i0; i < it.i1; ++i, ++n, ++ns) {
          wait(&tl->s_full[m], ns & 1);
          tc_fence_after();
          const int ve = tl->vexp[n & 3];
          const float f = pow2_clamped(tl->kexp[n & 3] - 134 - eq), vexp = float(ve - 127);
          const uint4 ok = *reinterpret_cast<const uint4*>(tl->ok[n & 3]);
          float s[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<float(*)[32]>(s + 32 * c));
          const int t0 = it.key0(i);
          const bool full = (ok.x & ok.y & ok.z & ok.w) == 0xffffffffu;
          if (!full || t0 + kPtTile > all_lim || (a.window > 0 && t0 < all_low)) {
            const uint32_t okw[4] = {ok.x, ok.y, ok.z, ok.w};
            auto below = [](int x) { return x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u; };
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int tc = t0 + 32 * c;
              uint32_t see = okw[c] & below(lim - tc);
              if (a.window > 0) see &= ~below(low - tc) | below(a.sinks - tc);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!((see >> k) & 1u)) s[32 * c + k] = -INFINITY;
            }
          }
          float top0 = s[0], top1 = s[1], top2 = s[2], top3 = s[3];
#pragma unroll
          for (int k = 4; k < 124; k += 8) {
            top0 = max3(top0, s[k], s[k + 1]);
            top1 = max3(top1, s[k + 2], s[k + 3]);
            top2 = max3(top2, s[k + 4], s[k + 5]);
            top3 = max3(top3, s[k + 6], s[k + 7]);
          }
          top0 = max3(top0, s[124], s[125]);
          top1 = max3(top1, s[126], s[127]);
          const float top = fmaf(fmaxf(fmaxf(top0, top1), fmaxf(top2, top3)), f, vexp);
          const bool need = top > M + kAttnSlack;
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? exp2f(M - top) : 1.f;
            if (need) M = top;
            l *= alpha;
            if (i > it.i0) {  // the previous tiles' products are complete: S came after them
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t o[16];
                asm volatile(
                    "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
                    "tcgen05.wait::ld.sync.aligned;"
                    : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]), "=r"(o[8]),
                      "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
                    : "r"(tO + 16 * c)
                    : "memory");
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tmem_st16(tO + 16 * c, o);
              }
            }
          }
          const float sub = M == -INFINITY ? 0.f : vexp - M;
          float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float x = s[32 * c + 2 * k], y = s[32 * c + 2 * k + 1];
              fma2(x, y, f, sub);
              x = exp2_ftz(x);
              y = exp2_ftz(y);
              if (k & 1) sum2(l2, l3, x, y); else sum2(l0, l1, x, y);
              p[k] = cvt_f16x2(x, y);
            }
            tmem_st16(tS + 16 * c, p);
          }
          l = fmaf((l0 + l1) + (l2 + l3), pow2_clamped(127 - ve), l);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tl->p_full[m]);
        }
      } else {
        n += it.i1 - it.i0;
      }

      // ---- next unit's queries, then this unit's output ----
      PtIter nx = it;
      more = nx.next(a, per);
      if (more && 128 * m < nx.ntok * a.g) load_queries(nx);
      if (active) {
        wait(&tl->o_full[m], nu & 1);
        ++nu;
        tc_fence_after();
        float o[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tO + 32 * c, *reinterpret_cast<float(*)[32]>(o + 32 * c));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tl->o_empty[m]);
        const int row = 128 * m + r;
        bool store = row < it.ntok * a.g && !dead;
        if (!it.whole()) {
          const int c0 = int(it.ustart / pc.quota), c1 = int((it.ustart + it.tl.count - 1) / pc.quota);
          auto slot = [&](int x) { return 2 * int64_t(x) + (x == c0 ? 1 : 0); };
          float4* po = reinterpret_cast<float4*>(a.part_o);
          float2* pm = reinterpret_cast<float2*>(a.part_ml);
          const int64_t mine = slot(int(blockIdx.x));
          if (!dead) {
            pm[mine * kPtRows + row] = make_float2(M, l);
#pragma unroll
            for (int c = 0; c < 32; ++c) po[(mine * 32 + c) * kPtRows + row] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
          __threadfence();
          named_bar_sync(1 + m, 128);
          if (r == 0) tl->last[m] = !dead && atomicAdd(a.counters + kPtCounterBase + 2 * c0 + m, 1u) == unsigned(c1 - c0);
          named_bar_sync(1 + m, 128);
          store = store && tl->last[m];
          if (tl->last[m]) {
            __threadfence();
            M = -INFINITY;
            for (int x = c0; x <= c1; ++x) M = fmaxf(M, __ldcg(&pm[slot(x) * kPtRows + row]).x);
            l = 0.f;
#pragma unroll
            for (int k = 0; k < 128; ++k) o[k] = 0.f;
            for (int x = c0; x <= c1; ++x) {
              const float2 ml = __ldcg(&pm[slot(x) * kPtRows + row]);
              const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
              l = fmaf(w, ml.y, l);
              const float4* px = po + slot(x) * 32 * kPtRows + row;
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const float4 v = __ldcg(px + c * kPtRows);
                o[4 * c] = fmaf(w, v.x, o[4 * c]);
                o[4 * c + 1] = fmaf(w, v.y, o[4 * c + 1]);
                o[4 * c + 2] = fmaf(w, v.z, o[4 * c + 2]);
                o[4 * c + 3] = fmaf(w, v.w, o[4 * c + 3]);
              }
            }
            if (r == 0) a.counters[kPtCounterBase + 2 * c0 + m] = 0u;  // ready for the next call
          }
        }
        if (store) {
          reg_fwht<128, 7>(o);
          const float inv = l > 0.f ? a.inv_sqrt_dim * 0.0078125f / l : 0.f;  // values entered times 2^7
          const int tok = row / a.g, hh = row - tok * a.g;
          uint4* dst = reinterpret_cast<uint4*>(a.out + (int64_t(it.rq.row0 + it.first + tok) * a.nqh + it.h * a.g + hh) * kPagedDim);
#pragma unroll
          for (int k = 0; k < 128; ++k) o[k] *= inv;
          if (a.signs) {
#pragma unroll
            for (int k = 0; k < 128; ++k) {
              const int dim = (k & ~7) | ((k & 1) << 2) | ((k & 6) >> 1);
              o[k] = __uint_as_float(__float_as_uint(o[k]) ^ (((tl->sgn[dim >> 5] >> (dim & 31)) & 1u) << 31));
            }
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float* y = o + 8 * c;  // dims 0, 4, 1, 5, 2, 6, 3, 7
            dst[c] = make_uint4(cvt_bf16x2(y[0], y[2]), cvt_bf16x2(y[4], y[6]), cvt_bf16x2(y[1], y[3]), cvt_bf16x2(y[5], y[7]));
          }
        }
      }
      it = nx;
    }
  } else if (warp < 12) {
    // ======================================================= keys and values
    regs_dec<96>();
    const int t = tid & 127, w = warp & 3;
    constexpr int RB = 16 * BITS, NV = RB / 16;  // 16-byte pieces per row
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!mbar_wait(bar, parity, abort)) {
        if (!dead) tc_give_up(&tl->abort, fault);
        dead = true;
      }
      dead = __any_sync(0xffffffffu, dead);
    };
    // The iterator runs ahead of the tile in work: page ids by two tiles,
    // codes by one.
    int i = it.i0;
    bool more = true;
    int64_t src = -1;  // row in the pool of this thread's key of the tile to load next, -1: none
    auto find = [&]() {
      src = -1;
      if (!more) return;
      const int pos = it.key0(i) + t;
      if (pos < it.tl.kv_end) {
        const int p = __ldg(a.table + int64_t(it.b) * a.max_pages + (pos >> a.page_log2));
        if (unsigned(p) < unsigned(a.n_pages))
          src = ((int64_t(p) * a.nkv + it.h) << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
      }
      if (++i == it.i1) {
        more = it.next(a, per);
        i = it.i0;
      }
    };
    uint4 kr[NV], vr[NV];
    float kscl[NG], vscl[NG];
    bool have = false;  // the loaded key is cached
    int64_t vsrc = -1;
    auto load_k = [&]() {
      have = src >= 0;
      vsrc = src;
#pragma unroll
      for (int x = 0; x < NV; ++x) kr[x] = have ? __ldg(reinterpret_cast<const uint4*>(a.k_codes + src * RB) + x) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        kscl[q] = have ? __ldg(a.k_scales + src * NG + q) : 0.f;
        vscl[q] = have ? __ldg(a.v_scales + src * NG + q) : 0.f;
      }
    };
    auto load_v = [&]() {
#pragma unroll
      for (int x = 0; x < NV; ++x) vr[x] = vsrc >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.v_codes + vsrc * RB) + x) : make_uint4(0u, 0u, 0u, 0u);
    };
    // codes -> f16 pairs (e, e + 4) of 8 columns
    auto pairs = [&](const uint4 (&raw)[NV], int c, uint32_t (&p)[4]) {
      if constexpr (BITS == 4) {
        const uint4 x = raw[c >> 2];
        const uint32_t word = (c & 3) == 0 ? x.x : (c & 3) == 1 ? x.y : (c & 3) == 2 ? x.z : x.w;
        i4x4_to_f16_tokens(word, p);
      } else {
        const uint4 x = raw[c >> 1];
        i8x8_to_f16_pairs((c & 1) ? x.z : x.x, (c & 1) ? x.w : x.y, p);
      }
    };
    find();
    load_k();
    load_v();
    find();
    const uint32_t total = uint32_t(pc.end - pc.at);
    for (uint32_t n = 0; n < total; ++n) {
      const int s = n & 1;
      const uint32_t ph = (n >> 1) & 1;
      // exponents of the tile's largest scales
      float kt = 0.f, vt = 0.f;
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        kscl[q] = clean_scale(kscl[q]);
        vscl[q] = clean_scale(vscl[q]);
        kt = fmaxf(kt, kscl[q]);
        vt = fmaxf(vt, vscl[q]);
      }
      const uint32_t kw = __reduce_max_sync(0xffffffffu, __float_as_uint(kt)), vw = __reduce_max_sync(0xffffffffu, __float_as_uint(vt));
      const uint32_t okw = __ballot_sync(0xffffffffu, have);
      if (lane == 0) {
        tl->dred[s][0][w] = kw;
        tl->dred[s][1][w] = vw;
      }
      wait(&tl->k_empty[s], ph ^ 1u);
      if (lane == 0) tl->ok[n & 3][w] = okw;
      named_bar_sync(3, 128);
      const uint32_t (&dk)[4] = tl->dred[s][0], (&dv)[4] = tl->dred[s][1];
      const int ke = min(max(int(max(max(dk[0], dk[1]), max(dk[2], dk[3])) >> 23), 27), 227);
      const int ve = min(max(int(max(max(dv[0], dv[1]), max(dv[2], dv[3])) >> 23), 27), 227);
      if (t == 0) {
        tl->kexp[n & 3] = ke;
        tl->vexp[n & 3] = ve;
      }
      const float kup = pow2_clamped(134 - ke), vup = pow2_clamped(134 - ve);  // largest scale to [2^7, 2^8)
      uint32_t khi[NG], klo[NG], vhi[NG];
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        const float x = kscl[q] * kup;
        khi[q] = cvt_f16x2(x, x);
        float hi;
        asm("{.reg .f16 l, h;\n mov.b32 {l, h}, %1;\n cvt.f32.f16 %0, l;}" : "=f"(hi) : "r"(khi[q]));
        klo[q] = cvt_f16x2(x - hi, x - hi);
        const float y = vscl[q] * vup;
        vhi[q] = cvt_f16x2(y, y);
      }
      uint8_t* kd = ks + s * kPtMat + t * 128;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        uint32_t p[4];
        pairs(kr, c, p);
        const int q = c * NG / 16;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t y = f16x2_mul(p[x], klo[q]);
          asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[x]) : "r"(p[x]), "r"(khi[q]), "r"(y));
        }
        *reinterpret_cast<uint4*>(kd + (c >> 3) * kPtHalf + (((c & 7) ^ (t & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tl->k_full[s]);
      load_k();  // the next tile's (vr still holds this one's values)
      find();
      wait(&tl->v_empty[s], ph ^ 1u);
      uint8_t* vd = vs + s * kPtMat + t * 128;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        uint32_t p[4];
        pairs(vr, c, p);
        const int q = c * NG / 16;
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x] = f16x2_mul(p[x], vhi[q]);
        *reinterpret_cast<uint4*>(vd + (c >> 3) * kPtHalf + (((c & 7) ^ (t & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tl->v_full[s]);
      load_v();
    }
  } else {
    regs_dec<64>();
    if (warp == 12) {
      // ================================================================ MMAs
      // The whole warp walks the schedule, so that descriptors and loop
      // bounds are warp-uniform; one lane issues.
      bool dead = false;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!mbar_wait(bar, parity, abort)) {
          if (!dead && lane == 0) tc_give_up(&tl->abort, fault);
          dead = true;
        }
        dead = __any_sync(0xffffffffu, dead);
      };
      const uint64_t qd = smem_desc(smem_addr(qs), 16, 1024, 2), kd = smem_desc(smem_addr(ks), 16, 1024, 2);
      const uint64_t vd = smem_desc(smem_addr(vs), kPtHalf, 1024, 2);
      auto mma_s = [&](int m, uint32_t stage) {  // S_m = Q_m K^T
        tc_fence_after();
        if (!dead && elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t o = ((k >> 2) * kPtHalf + (k & 3) * 32) >> 4;
            tc_mma(tmem + uint32_t(128 * m), qd + uint32_t(m * (kPtMat >> 4) + o), kd + (stage * (kPtMat >> 4) + o), kPtIdescQK, k > 0);
          }
          // The softmax reads what the key warps wrote beside the keys
          // (exponents, cached bits) once S is there: this warp has seen their
          // arrival and passes it on.  (They cannot wait for k_full
          // themselves: it may be a phase further on by then.)
          mbar_arrive(&tl->s_full[m]);
          tc_commit(&tl->s_full[m]);
        }
        __syncwarp();
      };
      auto mma_o = [&](int m, uint32_t stage, bool add) {  // O_m (+)= P_m V
        tc_fence_after();
        if (!dead && elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_ts(tmem + uint32_t(256 + 128 * m), tmem + uint32_t(128 * m + 8 * k), vd + (stage * (kPtMat >> 4) + k * (2048 >> 4)), kPtIdescPV,
                      k > 0 ? 1u : uint32_t(add));
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* bar) {
        if (!dead && elect_one()) tc_commit(bar);
        __syncwarp();
      };
      uint32_t n = 0, nu[2] = {0, 0}, np[2] = {0, 0};
      do {
        const int two = __shfl_sync(0xffffffffu, int(it.ntok * a.g > 128), 0), tiles = __shfl_sync(0xffffffffu, it.i1 - it.i0, 0);
        wait(&tl->q_full[0], nu[0] & 1);
        wait(&tl->k_full[n & 1], (n >> 1) & 1);
        mma_s(0, n & 1);
        if (two) {
          wait(&tl->q_full[1], nu[1] & 1);
          mma_s(1, n & 1);
        }
        commit(&tl->k_empty[n & 1]);
        for (int i = 0; i < tiles; ++i, ++n) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (m == 1 && !two) break;
            wait(&tl->p_full[m], np[m] & 1);
            ++np[m];
            if (m == 0) wait(&tl->v_full[n & 1], (n >> 1) & 1);
            if (i == 0) wait(&tl->o_empty[m], (nu[m] & 1) ^ 1u);
            mma_o(m, n & 1, i > 0);
            if (i + 1 < tiles) {
              if (m == 0) wait(&tl->k_full[(n + 1) & 1], ((n + 1) >> 1) & 1);
              mma_s(m, (n + 1) & 1);
            } else {
              commit(&tl->o_full[m]);
              ++nu[m];
            }
          }
          commit(&tl->v_empty[n & 1]);
          if (i + 1 < tiles) commit(&tl->k_empty[(n + 1) & 1]);
        }
      } while (it.next(a, per));
      // every MMA is complete before TMEM is freed (passes at once normally)
      if (!dead) (void)mbar_wait(&tl->v_empty[(n - 1) & 1], ((n - 1) >> 1) & 1, nullptr);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace hadq
