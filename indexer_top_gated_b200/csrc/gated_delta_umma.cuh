// gated_delta_umma.cuh - the chunked gated delta rule's scan on tcgen05, for batches that fill the
// GPU with whole heads.
//
// One CTA walks one sequence's chunks for one head (formulas, pieces and the preparation:
// gated_delta.cuh).  Products are taken transposed with the 128 value columns as the rows M of
// the UMMA, so a TMEM lane is a value column and a warp's rounding between two products is its
// own: accumulators are read from TMEM, scaled and split in registers, and written back to
// TMEM as the next product's A operand (two bf16 to a column).  Nothing crosses warps, and
// shared memory holds only what TMA brought: K and Q (rows of 64 columns, 128-byte swizzle), T
// and P (columns of 16, 32-byte swizzle, zeros above the diagonal), V; and the output on its way.
//   R  = S K^T       A: S in two pieces,  B: K   (N = 64, K-major)
//   QS = S Q^T       the same pieces,     B: Q
//   U  = X T^T       A: X in three,       B: T
//   U' K             A: U' in three,      B: K   (N = 128, MN-major: K's rows are the K axis)
//   O  = QS b + U P^T  A: U in two,       B: P   (added to QS b in its place)
// The chain R -> X -> U -> U' -> S bounds it: each operand is released in quarters, whose products
// run while the next is rounded.  QS and the output are other warps' work, under the chain.
//
// Measured: 2.9 us a chunk alone and 3.1 us with every SM busy (4096 tokens x 148 heads: 200 us).
// Of about 5000 cycles a chunk the tensor pipe has 3400: 24 K steps of U at 38 cycles, 16 of R and
// of QS each at 45, 12 of U' K at 67; the rest is rounding (about 700 cycles for X and for U', bound
// by the integer pipe that splits values) and hand-overs (250 cycles each).  The code's size counts:
// unrolled, with S in registers, a chunk took as long alone and 4.7 us with every SM busy, waiting
// for instructions.  So loops are rolled, X and U' share one, and waits are short.
#pragma once

#include "gated_delta.cuh"

namespace dsa {

constexpr int kUmmaChain = 8;                         // warps of the chain,
constexpr int kUmmaOutWarps = 4;                      // of the output,
constexpr int kUmmaIssue = kUmmaChain + kUmmaOutWarps;  // one that issues and one that loads
constexpr int kUmmaThreads = (kUmmaIssue + 2) * 32;
constexpr int kUmmaV = 2 * kDeltaTile;                // four tiles of 32 columns, 64-byte swizzle
constexpr int kUmmaVTile = kDeltaChunk * 64;
constexpr int kUmmaItem = kUmmaV + 4 * kUmmaVTile;    // three pieces of T, P
constexpr int kUmmaMat = 4 * 2048;                    // four columns of blocks, 64 rows of 32 bytes
constexpr int kUmmaScal = kUmmaItem + 4 * kUmmaMat;
constexpr int kUmmaStage = kUmmaScal + 1024;
static_assert(kUmmaStage % 1024 == 0, "");
constexpr int kUmmaBytes = kUmmaItem + kDeltaItemBytes;  // what a chunk's loads bring
constexpr int kUmmaOut = 2 * kUmmaStage;              // 64 tokens x 32 columns an output warp
constexpr int kUmmaBars = kUmmaOut + kUmmaOutWarps * kUmmaVTile;
constexpr int kUmmaSmem = kUmmaBars + 256;
// TMEM columns: S; its pieces, then U' K; R, then U, then U's second piece; QS, then O; X's
// pieces, then U''s; U's first piece
constexpr uint32_t kTmS = 0, kTmSp = 128, kTmR = 256, kTmQ = 320, kTmX = 384, kTmU = 480;
constexpr uint32_t kTmCols = 512;

struct UmmaSync {
  uint64_t full[2], tail;
  uint64_t r_done, q_done, u_done, s_done, o_done;  // products complete
  uint64_t s_ready[4], x_ready[2][4];               // quarters of S's pieces, and X's or U''s
  uint64_t p_ready;                                 // U's pieces and QS b written
  // O read: one for each stage, since two chunks are under way when the loader asks for the first
  // of them, and a barrier waited for by parity may not be two phases ahead
  uint64_t q_free[2];
  uint64_t drain;                                   // after a wait that ran out
  uint32_t tmem;
  volatile int abort;
};
static_assert(sizeof(UmmaSync) <= 256, "");

// D[tmem] (+)= A[tmem] * B[smem descriptor]; one thread issues.
DSA_DEV void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// B operand whose rows in shared memory are the product's K axis (MN-major, 128-byte swizzle):
// lbo: from 64 columns to the next 64, sbo: from eight rows to the next eight.
DSA_DEV uint64_t umma_smem_desc_mn(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((lbo_bytes >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)((sbo_bytes >> 4) & 0x3FFF) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// This warp's 32 lanes x 8 or 16 columns, a lane a thread
DSA_DEV void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
DSA_DEV void tmem_st16(uint32_t taddr, const float (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]),
      "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
      : "memory");
}
DSA_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 lanes as accumulator tiles of 16 x 8: registers 4 n + 2 e + j hold lane 8 e + (thread / 4),
// column 8 n + 2 (thread % 4) + j.
DSA_DEV void tmem_ld_tile(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}
DSA_DEV void tmem_ld_tiles(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
DSA_DEV void tmem_st_tiles(uint32_t taddr, const float (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
      : "memory");
}
// the same, each pair (j = 0, 1) in one column
DSA_DEV void tmem_st_pair(uint32_t taddr, uint32_t r0, uint32_t r1) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x1.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(r0), "r"(r1)
               : "memory");
}
DSA_DEV void tmem_st_pairs(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
constexpr uint32_t kHalfLanes = 16u << 16;  // the upper 16 of a warp's 32 TMEM lanes

// Eight columns of each of four quarters, or sixteen columns, of the accumulators in this warp's
// lanes, as tiles of either half of the lanes
DSA_DEV void tmem_load_quarters(uint32_t taddr, float (&x)[4][2][4]) {
  uint32_t r[4][2][4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    tmem_ld_tile(taddr + t * 16, r[t][0]);
    tmem_ld_tile(taddr + t * 16 + kHalfLanes, r[t][1]);
  }
  tmem_wait_ld();
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      reg_fence(r[t][h]);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[t][h][i] = __uint_as_float(r[t][h][i]);
    }
}
DSA_DEV void tmem_load16(uint32_t taddr, float (&x)[2][8]) {
  uint32_t r[2][8];
  tmem_ld_tiles(taddr, r[0]);
  tmem_ld_tiles(taddr + kHalfLanes, r[1]);
  tmem_wait_ld();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    reg_fence(r[h]);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[h][i] = __uint_as_float(r[h][i]);
  }
}

DSA_DEV void stmatrix_x4_trans(uint32_t saddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}
// (x, y) = (x, y) * a (+ b), in one packed operation
DSA_DEV void mul_f32x2(float& x, float& y, float2 a) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a.x), "f"(a.y));
}
DSA_DEV void fma_f32x2(float& x, float& y, float2 a, float2 b) {
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "mov.b64 r, {%4, %5};\n\tfma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
}
DSA_DEV void sub_f32x2(float& x, float& y, uint32_t a, uint32_t b) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "sub.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "r"(a), "r"(b));
}
// Two values in two pieces, the first rounded; and in three, the first two cut off: they leave
// eight bits to the third, so that it is exact, without a conversion.
DSA_DEV void umma_split(float x, float y, uint32_t (&p)[2]) {
  p[0] = pack_bf16x2(x, y);
  sub_f32x2(x, y, p[0] << 16, p[0] & 0xffff0000u);
  p[1] = pack_bf16x2(x, y);
}
DSA_DEV void umma_split(float x, float y, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t u = __float_as_uint(x), v = __float_as_uint(y);
    p[i] = __byte_perm(u, v, 0x7632);
    if (i < 2) sub_f32x2(x, y, u & 0xffff0000u, v & 0xffff0000u);
  }
}
DSA_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p;
}

// What a warp wrote to or read from TMEM is done, and the issuing thread may go on.
DSA_DEV void umma_release(uint64_t& bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bar));
}
// A bounded wait like mbar_wait_bounded in fewer instructions (there are eighteen of them; reading
// the clock costs 2 % of the scan): it gives up after as many polls as take 0.1 s or more.
constexpr uint32_t kUmmaPolls = 1u << 22;
DSA_DEV void umma_wait_smem(const DeltaArgs& a, UmmaSync* sy, uint64_t& bar, uint32_t parity) {
  for (uint32_t it = 1; !mbar_try_wait(smem_u32(&bar), parity); ++it) {
    if (it & 63) continue;
    if (sy->abort) break;
    if (it == kUmmaPolls) {
      sy->abort = 1;
      atomicExch(a.status, kDevTimeout);
    }
  }
}
DSA_DEV void umma_wait(const DeltaArgs& a, UmmaSync* sy, uint64_t& bar, uint32_t parity) {
  umma_wait_smem(a, sy, bar, parity);
  tc_fence_after();
}

// The loading warp.
DSA_DEV void umma_load(const DeltaArgs& a, const DeltaMaps& maps, const ScanPlace& at,
                       unsigned char* smem, UmmaSync* sy) {
  const int lane = threadIdx.x & 31;
  int c = 0;
#pragma unroll 1
  for (; c * kDeltaChunk < at.len; ++c) {
    if (c >= 2) {  // chunk c - 2's products are complete and its scalars and V read
      umma_wait_smem(a, sy, sy->q_free[c & 1], (c >> 1 & 1) ^ 1);
      if (__any_sync(~0u, sy->abort)) break;
    }
    const int valid = at.len - c * kDeltaChunk;
    const bool part = valid < kDeltaChunk;
    const uint32_t full = smem_u32(&sy->full[c & 1]);
    const uint32_t bar = part ? smem_u32(&sy->tail) : full;
    unsigned char* to = smem + (c & 1) * kUmmaStage;
    const uint32_t stage = smem_u32(to);
    const int64_t row0 = at.first + (int64_t)c * kDeltaChunk;
    const unsigned char* item = at.items + c * at.item_step;
    if (lane == 0) mbar_arrive_expect_tx(bar, kUmmaBytes);
    __syncwarp();
    if (lane == 0) {
      delta_load_qk(maps, stage, stage + kDeltaTile, bar, at.hk, row0);
    } else if (lane <= 4) {
      const int i = lane - 1;
      tma_load_2d(stage + kUmmaV + i * kUmmaVTile, &maps.v, bar, at.h * kDeltaDim + i * 32,
                  (int)row0);
    } else if (lane == 5) {
      bulk_load(stage + kUmmaScal, item + kDeltaScal, 1024, bar);
    } else if (lane >= 16) {  // a column of blocks from the diagonal on
      const int p = (lane >> 2) & 3, kt = lane & 3;
      bulk_load(stage + kUmmaItem + p * kUmmaMat + kt * (2048 + 512),
                item + p * kDeltaMat + tri_col(kt) + kt * 512, 2048 - kt * 512, bar);
    }
    __syncwarp();
    if (part) {  // the last chunk: the rows behind the sequence's end become zeros first
      umma_wait_smem(a, sy, sy->tail, 0);
      for (int i = 0; i < 4; ++i) {
        delta_zero_rows(to + i * (kDeltaTile / 2), 128, valid, lane, 32);
        delta_zero_rows(to + kUmmaV + i * kUmmaVTile, 64, valid, lane, 32);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the UMMAs read them
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
  }
  scan_drain(at, sy, c);
}

// The issuing thread.
DSA_DEV void umma_issue(const DeltaArgs& a, const ScanPlace& at, unsigned char* smem, UmmaSync* sy) {
  const int n_chunks = (at.len + kDeltaChunk - 1) / kDeltaChunk;
  constexpr uint32_t kN64 = umma_idesc(128, 64, 1);
  constexpr uint32_t kN128Mn = umma_idesc(128, 128, 1) | 1u << 16;  // B is MN-major
#pragma unroll 1
  for (int c = 0; c < n_chunks; ++c) {
    const uint32_t par = c & 1;
    const uint32_t k = smem_u32(smem) + par * kUmmaStage;
    // (descriptors hold addresses in units of 16 bytes)
    const uint64_t dk = umma_smem_desc(k, 1024, 2), dt = umma_smem_desc(k + kUmmaItem, 256, 6);
    const uint64_t dkt = umma_smem_desc_mn(k, kDeltaTile / 2, 1024);
    // quarter h of S's key columns times K or Q
    auto times_s = [&](uint32_t d, int tile, int h) {
      const uint64_t b = dk + (tile + (h >> 1) * (kDeltaTile / 2) + (h & 1) * 64) / 16;
#pragma unroll
      for (int i = 0; i < 4; ++i)  // either piece of two steps
        umma_bf16_ta(d, kTmSp + h * 32 + i * 8, b + (i >> 1) * 2, kN64, h + i != 0);
    };
    umma_wait(a, sy, sy->full[par], c >> 1 & 1);
    if (c) umma_wait(a, sy, sy->o_done, 1 - par);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      umma_wait(a, sy, sy->s_ready[h], par);
      times_s(kTmR, 0, h);
    }
    umma_commit(smem_u32(&sy->r_done));
    if (c) umma_wait(a, sy, sy->q_free[1 - par], (c - 1) >> 1 & 1);
#pragma unroll 1
    for (int h = 0; h < 4; ++h) times_s(kTmQ, kDeltaTile, h);
    umma_commit(smem_u32(&sy->q_done));
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      umma_wait(a, sy, sy->x_ready[0][kt], par);
#pragma unroll
      for (int px = 0; px < 3; ++px)
#pragma unroll
        for (int pt = 0; pt < 3 - px; ++pt)
          umma_bf16_ta(kTmR, kTmX + px * 32 + kt * 8, dt + (pt * kUmmaMat + kt * 2048) / 16, kN64,
                       kt + px + pt != 0);
    }
    umma_commit(smem_u32(&sy->u_done));
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      umma_wait(a, sy, sy->x_ready[1][kt], par);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        umma_bf16_ta(kTmSp, kTmX + p * 32 + kt * 8, dkt + kt * 2048 / 16, kN128Mn, kt + p != 0);
    }
    umma_commit(smem_u32(&sy->s_done));
    umma_wait(a, sy, sy->p_ready, par);
#pragma unroll 1
    for (int kt = 0; kt < 4; ++kt) {
      const uint64_t b = dt + (3 * kUmmaMat + kt * 2048) / 16;
      umma_bf16_ta(kTmQ, kTmU + kt * 8, b, kN64, 1);
      umma_bf16_ta(kTmQ, kTmR + kt * 8, b, kN64, 1);
    }
    umma_commit(smem_u32(&sy->o_done));
  }
  if (sy->abort) {  // a wait ran out: let the products in flight end before TMEM is freed
    umma_commit(smem_u32(&sy->drain));
    mbar_wait_bounded(smem_u32(&sy->drain), 0, nullptr, nullptr);
  }
}

// The chain's rounding warps: warp w has TMEM lanes 32 (w % 4) .. and, of a quarter of the tokens
// or of S's key columns, the first or the second half.
DSA_DEV void umma_round(const DeltaArgs& a, const ScanPlace& at, unsigned char* smem, UmmaSync* sy,
                        int warp) {
  const int lane = threadIdx.x & 31, mi = lane >> 3, mr = lane & 7;
  const int w = warp & 3, part = warp >> 2;
  const uint32_t tm = (uint32_t)(w * 32) << 16;
  const int n_chunks = (at.len + kDeltaChunk - 1) / kDeltaChunk;
  const int64_t soff =
      ((at.slot * a.hv + at.h) * kDeltaDim + w * 32 + lane) * kDeltaDim + part * 16;
  // a quarter of S: kept, and in two pieces
  auto put_s = [&](const float (&s)[16], int h) {
    const uint32_t col = h * 32 + part * 16;
    uint32_t p[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t q[2];
      umma_split(s[2 * j], s[2 * j + 1], q);
      p[0][j] = q[0], p[1][j] = q[1];
    }
    tmem_st8(tm + kTmSp + col, p[0]);
    tmem_st8(tm + kTmSp + col + 8, p[1]);
    tmem_wait_st();
    umma_release(sy->s_ready[h]);
    tmem_st16(tm + kTmS + col, s);  // (complete at the next wait for stores)
  };
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    float s[16];
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.state_in && at.slot >= 0)
        v = *reinterpret_cast<const float4*>(a.state_in + soff + h * 32 + i);
      s[i] = v.x, s[i + 1] = v.y, s[i + 2] = v.z, s[i + 3] = v.w;
    }
    put_s(s, h);
  }

#pragma unroll 1
  for (int c = 0; c < n_chunks; ++c) {
    const uint32_t par = c & 1;
    const unsigned char* stage = smem + par * kUmmaStage;
    const uint32_t v = smem_u32(stage) + kUmmaV + w * kUmmaVTile;
    // this thread's pair of tokens of a quarter
    const float* scal =
        reinterpret_cast<const float*>(stage + kUmmaScal) + part * 8 + (lane & 3) * 2;
    auto put_x = [&](const float (&x)[2][4], int t) {
      const uint32_t to = tm + kTmX + t * 8 + part * 4;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[2][3];
        umma_split(x[h][0], x[h][1], p[0]);
        umma_split(x[h][2], x[h][3], p[1]);
#pragma unroll
        for (int i = 0; i < 3; ++i) tmem_st_pair(to + h * kHalfLanes + i * 32, p[0][i], p[1][i]);
      }
      tmem_wait_st();
    };
    umma_wait(a, sy, sy->full[par], c >> 1 & 1);
    // (read here, not where it is used: after a warp's last release of X or U' nothing keeps the
    // loader from the stage)
    const float decay = reinterpret_cast<const float*>(stage + kUmmaScal)[192];
    // The accumulators are read whole before a quarter is released: its products write over them.
#pragma unroll 1
    for (int p = 0; p < 2; ++p) {  // X = V - R diag(a), then U' = U diag(t)
      float x[4][2][4];
      uint32_t fv[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (p == 0) {
          ldmatrix_x4_trans(v + swz64(t * 16 + part * 8 + mr, mi), fv[t]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) fv[t][e] = 0;
        }
      }
      umma_wait(a, sy, p ? sy->u_done : sy->r_done, par);
      tmem_load_quarters(tm + kTmR + part * 8, x);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float2 m = *reinterpret_cast<const float2*>(scal + p * 64 + t * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          fma_f32x2(x[t][e >> 1][(e & 1) * 2], x[t][e >> 1][(e & 1) * 2 + 1],
                    p ? m : make_float2(-m.x, -m.y),
                    make_float2(bf16_lo(fv[t][e]), bf16_hi(fv[t][e])));
        put_x(x[t], t);
        umma_release(sy->x_ready[p][t]);
      }
    }
    umma_wait(a, sy, sy->s_done, par);
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {  // S = e^(G_C) S + U' K
      uint32_t r[16], y[16];
      float s[16];
      tmem_ld16_async(tm + kTmSp + h * 32 + part * 16, r);
      tmem_ld16_async(tm + kTmS + h * 32 + part * 16, y);
      tmem_wait_ld();
      reg_fence(r);
      reg_fence(y);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        s[i] = __uint_as_float(y[i]), s[i + 1] = __uint_as_float(y[i + 1]);
        fma_f32x2(s[i], s[i + 1], make_float2(decay, decay),
                  make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])));
      }
      if (c + 1 < n_chunks) {
        put_s(s, h);
      } else if (a.state_out && at.slot >= 0) {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(a.state_out + soff + h * 32 + i) =
              make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
      }
    }
  }
}

// The output warps: warp w has TMEM lanes 32 w ..: QS diag(b), U in two pieces, and O.
DSA_DEV void umma_output(const DeltaArgs& a, const DeltaMaps& maps, const ScanPlace& at,
                         unsigned char* smem, UmmaSync* sy, int w) {
  const int lane = threadIdx.x & 31, mi = lane >> 3, mr = lane & 7;
  const uint32_t tm = (uint32_t)(w * 32) << 16;
  const int n_chunks = (at.len + kDeltaChunk - 1) / kDeltaChunk;
  unsigned char* stash = smem + kUmmaOut + w * kUmmaVTile;
  const uint32_t st = smem_u32(stash);
#pragma unroll 1
  for (int c = 0; c < n_chunks; ++c) {
    const uint32_t par = c & 1;
    const float* scal = reinterpret_cast<const float*>(smem + par * kUmmaStage + kUmmaScal) + 128 +
                        (lane & 3) * 2;
    float x[2][8];  // 16 tokens
    umma_wait(a, sy, sy->full[par], c >> 1 & 1);
    umma_wait(a, sy, sy->q_done, par);
#pragma unroll 1
    for (int t = 0; t < 4; ++t) {
      tmem_load16(tm + kTmQ + t * 16, x);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float2 bv = *reinterpret_cast<const float2*>(scal + t * 16 + n * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mul_f32x2(x[i >> 1][n * 4 + (i & 1) * 2], x[i >> 1][n * 4 + (i & 1) * 2 + 1], bv);
      }
      tmem_st_tiles(tm + kTmQ + t * 16, x[0]);
      tmem_st_tiles(tm + kTmQ + t * 16 + kHalfLanes, x[1]);
    }
    // U is there, and the chain has read it: the second piece takes its place
    umma_wait(a, sy, sy->x_ready[1][0], par);
#pragma unroll 1
    for (int t = 0; t < 4; ++t) {
      tmem_load16(tm + kTmR + t * 16, x);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t q[2];
          umma_split(x[h][2 * j], x[h][2 * j + 1], q);
          p[0][j] = q[0], p[1][j] = q[1];
        }
        tmem_st_pairs(tm + kTmU + t * 8 + h * kHalfLanes, p[0]);
        tmem_st_pairs(tm + kTmR + t * 8 + h * kHalfLanes, p[1]);
      }
    }
    tmem_wait_st();
    umma_release(sy->p_ready);
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    umma_wait(a, sy, sy->o_done, par);
#pragma unroll 1
    for (int t = 0; t < 4; ++t) {
      tmem_load16(tm + kTmQ + t * 16, x);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        stmatrix_x4_trans(st + swz64(t * 16 + (mi >> 1) * 8 + mr, h * 2 + (mi & 1)),
                          pack_bf16x2(x[h][0], x[h][1]), pack_bf16x2(x[h][2], x[h][3]),
                          pack_bf16x2(x[h][4], x[h][5]), pack_bf16x2(x[h][6], x[h][7]));
    }
    umma_release(sy->q_free[par]);
    const int row = c * kDeltaChunk, left = at.len - row;
    if (left >= kDeltaChunk) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        asm volatile(
            "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                reinterpret_cast<uint64_t>(&maps.out)),
            "r"(st), "r"(at.h * kDeltaDim + w * 32), "r"((int)at.first + row)
            : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    } else {  // the sequence ends among these tokens
      __syncwarp();
#pragma unroll 1
      for (int i = lane; i < left * 4; i += 32)
        *reinterpret_cast<uint4*>(a.out + ((at.first + row + (i >> 2)) * a.hv + at.h) * kDeltaDim +
                                  w * 32 + (i & 3) * 8) =
            *reinterpret_cast<const uint4*>(stash + swz64(i >> 2, i & 3));
    }
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__global__ void __launch_bounds__(kUmmaThreads, 1) delta_umma_kernel(
    const DeltaArgs a, const __grid_constant__ DeltaMaps maps) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x >> 5;
  const ScanPlace at = scan_place(a, blockIdx.x / a.heads, blockIdx.x % a.heads, 0);
  if (at.len < a.min_len) return;
  UmmaSync* sy = reinterpret_cast<UmmaSync*>(smem + kUmmaBars);
  if (threadIdx.x == 0) {
    for (uint64_t* b : {&sy->full[0], &sy->full[1], &sy->tail, &sy->r_done, &sy->q_done,
                        &sy->u_done, &sy->s_done, &sy->o_done, &sy->drain})
      mbar_init(smem_u32(b), 1);
    for (int h = 0; h < 4; ++h)
      for (uint64_t* b : {&sy->s_ready[h], &sy->x_ready[0][h], &sy->x_ready[1][h]})
        mbar_init(smem_u32(b), kUmmaChain);
    for (uint64_t* b : {&sy->p_ready, &sy->q_free[0], &sy->q_free[1]}) mbar_init(smem_u32(b), kUmmaOutWarps);
    sy->abort = 0;
    fence_mbar_init();
  }
  // zeros above the diagonal of T and P, which no load touches
  for (int i = threadIdx.x; i < 4 * kUmmaMat / 16; i += kUmmaThreads) {
    *reinterpret_cast<uint4*>(smem + kUmmaItem + i * 16) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(smem + kUmmaStage + kUmmaItem + i * 16) = make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (warp == kUmmaIssue) {
    tmem_alloc(smem_u32(&sy->tmem), kTmCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (all of TMEM is this CTA's, so that its columns are 0 .. 511)
  if (warp == kUmmaIssue) {
    if (elect_one()) umma_issue(a, at, smem, sy);
    __syncwarp();
  } else if (warp > kUmmaIssue) {
    umma_load(a, maps, at, smem, sy);
  } else if (warp >= kUmmaChain) {
    umma_output(a, maps, at, smem, sy, warp - kUmmaChain);
  } else {
    umma_round(a, at, smem, sy, warp);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kUmmaIssue) {
    tc_fence_after();
    tmem_dealloc(sy->tmem, kTmCols);
  }
}

}  // namespace dsa
