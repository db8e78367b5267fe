// gated_delta.cuh - the gated delta rule (the hybrid layer's linear branch), recurrent and
// chunked.  Per value head h with key head h / (Hv / Hk), state S [dv, dk] fp32:
//
//   S_t = alpha_t S_{t-1} + u_t k_t^T,  u_t = beta_t (v_t - alpha_t S_{t-1} k_t),  alpha = e^g
//   o_t = scale * S_t q_t
//
// with q and k optionally divided by their norms sqrt(sum x^2 + eps).
//
// Recurrent form (delta_recurrent_kernel): decode and sequences of few tokens.  What it cannot
// do without is the state, 64 KB a head in and out; a warp keeps 16 rows of it in registers, so
// the state crosses HBM once each way however many tokens the sequence has.  Measured: 256
// sequences x 64 heads 326 us, 6.6 TB/s; 64 x 32 heads 46 us, 5.8 TB/s.
//
// Chunked form: with G the running sum of g inside a chunk of 64 tokens,
//   (I + A) U = diag(beta) (V - diag(e^G) K S0^T),  A_ij = beta_i e^(G_i - G_j) k_i.k_j (j < i)
//   O = scale (diag(e^G) Q S0^T + (tril(Q K^T) . e^(G_i - G_j)) U)
//   S = e^(G_C) S0 + U^T diag(e^(G_C - G_j)) K
// delta_prep_kernel computes what does not depend on the state, for every chunk at once:
// T = (I + A)^-1 diag(beta) and P = scale * tril(Q K^T) . e^(G_i - G_j).  delta_scan_kernel (or, for
// batches that fill the GPU with whole heads, gated_delta_umma.cuh's) then
// walks a sequence's chunks with S in registers.  Columns of S^T (the dv axis) never meet, so
// a CTA takes 32 or 16 of the 128, and a pair of warps 16 of them.
//
// Precision: the state, the norms, the decays and every sum are fp32 (the running sum of g
// fp64, since only its differences matter and a strong decay leaves them small beside it).  The
// tensor cores take bf16, so an fp32 operand enters as two or three bf16 pieces (8 mantissa bits
// each): k, q and v are bf16 already and enter whole.  S in K S0^T has two pieces (the third
// moves the state by 1e-7 of itself), T, V - K S0^T and U have three, which leaves the state
// 1e-7 to 1e-6 off, as fp32 products would; with two it is 5e-6 off.  Decays inside a chunk are
// powers of two by ex2.approx (2^-22 off).  The output is rounded to bf16 once, and U and S enter its
// products with two pieces (2^-16); but P is kept as one bf16, which moves an output by up to 2^-8 of
// sum_j |P_ij U_j|: with the output's own rounding 2.3e-3 in all (2-norm), 1.7e-3 without.  A second
// piece of P would be another 5 KB of an item's 21 (written and read once each) and a third product.
#pragma once

#include <cstddef>

#include "common.cuh"
#include "find_last.cuh"

namespace dsa {

constexpr int kDeltaDim = 128;    // dk = dv
constexpr int kDeltaChunk = 64;   // tokens of a chunk

struct DeltaArgs {
  const int32_t* q_offsets;
  int batch;
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements per packed row
  const float *g, *beta;                 // [total_q, Hv]
  const float* state_in;                 // [n_states, Hv, dv, dk] or nullptr: zeros
  float* state_out;                      // the same layout, or nullptr: not kept
  const int32_t* state_index;            // [batch] or nullptr: sequence b uses slot b
  int n_states;
  __nv_bfloat16* out;                    // [total_q, Hv, dv]
  int hk, hv, norm;
  float scale, eps;
  int min_len, max_len;  // a kernel takes the sequences of min_len .. max_len tokens
  // chunked form
  unsigned char* ws;     // kDeltaItemBytes per (chunk slot, head of the pass)
  int head0, heads;      // heads of the pass
  int per_cta;           // value heads of a preparation CTA (of one key head)
  int* status;           // device status word
};

// The rows of q, k and v as TMA sees them: boxes of 64 rows, 64 columns of q and k (128-byte
// swizzle) and kScanNV = 32 of v and out (64-byte swizzle).
struct DeltaMaps {
  CUtensorMap q, k, v, out;
};

// The state slot of sequence b, or -1: none (starts from zero, is not kept).
DSA_DEV int64_t delta_slot(const DeltaArgs& a, int b) {
  const int s = a.state_index ? __ldg(a.state_index + b) : b;
  return s >= 0 && s < a.n_states ? s : -1;
}

DSA_DEV float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
DSA_DEV float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// ------------------------------------------------------------------ recurrent form
//
// A warp holds 16 rows of S, a lane 4 of the 128 key columns of each (one 16-byte load per
// row).  S k and S q of the 16 rows are 32 sums over the warp, folded together by a butterfly
// that halves the values it carries at each step: 31 shuffles in place of 32 * 5.  S_t q is
// formed from S_{t-1} q and the scalar k.q, so both sums come from one pass.
constexpr int kRecRows = 16;
constexpr int kRecWarps = 4;
constexpr int kRecParts = kDeltaDim / (kRecRows * kRecWarps);  // CTAs per (sequence, head)

__global__ void __launch_bounds__(kRecWarps * 32) delta_recurrent_kernel(const DeltaArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % kRecParts;
  const int h = (blockIdx.x / kRecParts) % a.hv;
  const int b = blockIdx.x / (kRecParts * a.hv);
  const int64_t row0 = __ldg(a.q_offsets + b);
  const int n = (int)(__ldg(a.q_offsets + b + 1) - row0);
  if (n < a.min_len || n > a.max_len) return;
  const int64_t slot = delta_slot(a, b);
  const int dv0 = (part * kRecWarps + warp) * kRecRows;
  const int64_t soff = ((slot * a.hv + h) * kDeltaDim + dv0) * kDeltaDim + lane * 4;

  // a token's inputs, asked for one token ahead
  const int hk = h / (a.hv / a.hk);
  struct Token {
    uint2 k, q;
    __nv_bfloat16 v;
    float g, beta;
  };
  auto fetch = [&](int t) {
    const int64_t row = row0 + t;
    Token x;
    x.k = __ldg(reinterpret_cast<const uint2*>(a.k + row * a.k_stride + hk * kDeltaDim) + lane);
    x.q = __ldg(reinterpret_cast<const uint2*>(a.q + row * a.q_stride + hk * kDeltaDim) + lane);
    x.v = a.v[row * a.v_stride + (int64_t)h * kDeltaDim + dv0 + (lane & 15)];
    x.g = __ldg(a.g + row * a.hv + h);
    x.beta = __ldg(a.beta + row * a.hv + h);
    return x;
  };
  Token next = {};
  if (n > 0) next = fetch(0);

  float4 s[kRecRows];
  if (a.state_in && slot >= 0) {
#pragma unroll
    for (int r = 0; r < kRecRows; ++r)
      s[r] = __ldcs(reinterpret_cast<const float4*>(a.state_in + soff + r * kDeltaDim));
  } else {
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) s[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  for (int t = 0; t < n; ++t) {
    const int64_t row = row0 + t;
    const Token x = next;
    if (t + 1 < n) next = fetch(t + 1);
    const float vv = __bfloat162float(x.v), alpha = expf(x.g), beta = x.beta;
    float k[4] = {bf16_lo(x.k.x), bf16_hi(x.k.x), bf16_lo(x.k.y), bf16_hi(x.k.y)};
    float q[4] = {bf16_lo(x.q.x), bf16_hi(x.q.x), bf16_lo(x.q.y), bf16_hi(x.q.y)};
    float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kk = fmaf(k[i], k[i], kk);
      qq = fmaf(q[i], q[i], qq);
      kq = fmaf(k[i], q[i], kq);
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) {
      kq += __shfl_xor_sync(~0u, kq, m);
      if (a.norm) {
        kk += __shfl_xor_sync(~0u, kk, m);
        qq += __shfl_xor_sync(~0u, qq, m);
      }
    }
    float kn = 1.f, qn = a.scale;
    if (a.norm) {
      kn = 1.f / sqrtf(kk + a.eps);
      qn = a.scale / sqrtf(qq + a.eps);
    }
    // w[r] = S_r . k, w[16 + r] = S_r . q, this lane's share of the sums
    float w[32];
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) {
      w[r] = fmaf(s[r].x, k[0], fmaf(s[r].y, k[1], fmaf(s[r].z, k[2], s[r].w * k[3])));
      w[16 + r] = fmaf(s[r].x, q[0], fmaf(s[r].y, q[1], fmaf(s[r].z, q[2], s[r].w * q[3])));
    }
    // after the step with mask m a lane carries the values whose index agrees with it in bit m
#pragma unroll
    for (int m = 16; m; m >>= 1) {
      const bool up = (lane & m) != 0;
#pragma unroll
      for (int i = 0; i < m; ++i) {
        const float send = up ? w[i] : w[i + m];
        const float keep = up ? w[i + m] : w[i];
        w[i] = keep + __shfl_xor_sync(~0u, send, m);
      }
    }
    // lane r < 16: S_r . k; lane 16 + r: S_r . q
    const float sq = __shfl_down_sync(~0u, w[0], 16);
    const float u = beta * (vv - alpha * kn * w[0]);  // of row r, in lanes r < 16
    const float o = qn * (alpha * sq + u * kn * kq);
    if (lane < 16) a.out[(row * a.hv + h) * kDeltaDim + dv0 + lane] = __float2bfloat16_rn(o);
    const float un = u * kn;
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) {
      const float ur = __shfl_sync(~0u, un, r);
      s[r].x = fmaf(ur, k[0], alpha * s[r].x);
      s[r].y = fmaf(ur, k[1], alpha * s[r].y);
      s[r].z = fmaf(ur, k[2], alpha * s[r].z);
      s[r].w = fmaf(ur, k[3], alpha * s[r].w);
    }
  }
  if (a.state_out && slot >= 0) {
#pragma unroll
    for (int r = 0; r < kRecRows; ++r)
      __stcs(reinterpret_cast<float4*>(a.state_out + soff + r * kDeltaDim), s[r]);
  }
}

// ------------------------------------------------------------------ chunked form: layout
//
// Chunk c of sequence b has the workspace slot q_offsets[b] / 64 + b + c: slots of different
// sequences never meet (a sequence of n tokens at offset o has at most (o + n) / 64 - o / 64 + 1
// chunks), and no prefix sum of chunk counts is needed.
DSA_DEV int64_t delta_first_slot(const DeltaArgs& a, int b) {
  return (int64_t)__ldg(a.q_offsets + b) / kDeltaChunk + b;
}

// One item of the workspace: three pieces of T, P (bf16), each the ten 16 x 16 blocks on and below
// the diagonal in column order, 512 bytes a block: 16 rows of two 16-byte units, which trade
// places in rows 4 .. 7 and 12 .. 15 (ldmatrix then meets no bank conflict, and a column of blocks
// is a K-major UMMA operand with 32-byte swizzle); then the scalars of the tokens.
constexpr int kDeltaMat = 10 * 512;
constexpr int kDeltaScal = 4 * kDeltaMat;        // a[64], t[64], b[64], e^(G_C)
constexpr int kDeltaItemBytes = kDeltaScal + 1024;
constexpr int kDeltaTile = kDeltaChunk * kDeltaDim * 2;  // K or Q of a chunk: two halves of the
                                                         // columns, rows of 128 bytes each
// From block (m, 0) of the triangular matrices to block (m, kt), and the 16-byte unit of row r,
// columns 8 unit ..
DSA_DEV constexpr int tri_col(int kt) { return kt * (7 - kt) / 2 * 512; }
DSA_DEV int tri_unit(int r, int unit) {
  return tri_col(unit >> 1) + r * 32 + (((unit & 1) ^ ((r >> 2) & 1)) << 4);
}

// 16-byte unit (columns 8 unit ..) of a row of a K or Q tile
DSA_DEV uint32_t swz(int row, int unit) {
  return (unit >> 3) * (kDeltaTile / 2) + row * 128 + (((unit & 7) ^ (row & 7)) << 4);
}

// K and Q of the chunk at row0, head hk, onto `bar` (kDeltaTile bytes each); one thread.
DSA_DEV void delta_load_qk(const DeltaMaps& maps, uint32_t k, uint32_t q, uint32_t bar, int hk,
                           int64_t row0) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    tma_load_2d(k + i * (kDeltaTile / 2), &maps.k, bar, hk * kDeltaDim + i * 64, (int)row0);
    tma_load_2d(q + i * (kDeltaTile / 2), &maps.q, bar, hk * kDeltaDim + i * 64, (int)row0);
  }
}

// Zeros in rows valid .. 63 of a tile with `row_bytes` per row (TMA brought the next
// sequence's); thread t of n.
DSA_DEV void delta_zero_rows(unsigned char* tile, int row_bytes, int valid, int t, int n) {
  for (int at = valid * row_bytes + t * 16; at < kDeltaChunk * row_bytes; at += n * 16)
    *reinterpret_cast<uint4*>(tile + at) = make_uint4(0, 0, 0, 0);
}

// Two fp32 values as N packed pairs of bf16 whose sum they are, largest first.
template <int N>
DSA_DEV void split_pair(float x, float y, uint32_t (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = pack_bf16x2(x, y);
    if (i + 1 < N) {
      x -= bf16_lo(p[i]);
      y -= bf16_hi(p[i]);
    }
  }
}

// N pieces of the left operand made of two accumulator tiles (16 rows x 16 columns)
template <int N>
DSA_DEV void split_frag(const float (&x)[4], const float (&y)[4], uint32_t (&f)[N][4]) {
  uint32_t p[N];
  split_pair<N>(x[0], x[1], p);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i][0] = p[i];
  split_pair<N>(x[2], x[3], p);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i][1] = p[i];
  split_pair<N>(y[0], y[1], p);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i][2] = p[i];
  split_pair<N>(y[2], y[3], p);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i][3] = p[i];
}

// ------------------------------------------------------------------ chunked form: T and P
//
// One CTA per chunk and one value head, or all value heads of one key head (K K^T and Q K^T are
// theirs in common).  Its four warps form K K^T and Q K^T on and below the
// diagonal (they share K's operands and the decays); then I + A is inverted in place, in
// fp32: its 16 x 16 diagonal blocks by forward substitution, and the blocks below by
//   [T1 0; -T2 A21 T1, T2], twice, 16 -> 32 -> 64.
// Written as loops rather than one unrolled substitution over 64 rows: that was bound by
// instruction fetch.  Measured: 8192 tokens x 32 heads about 80 us (from 158); no pipe is above
// 57 %, waits and barriers of short dependent phases bound it.
constexpr int kPrepThreads = 128;
constexpr int kPrepLd = 68;  // floats per row of A: 16-byte rows, eight rows on distinct banks

struct PrepSmem {
  union {
    struct {
      unsigned char k[kDeltaTile], q[kDeltaTile];
    };
    float A[kDeltaChunk * kPrepLd];  // once the products are in registers
  };
  alignas(16) float2 G[kDeltaChunk];  // running sum of g log2(e), high and low part
  alignas(16) float ink[kDeltaChunk], inq[kDeltaChunk], beta[kDeltaChunk];
  uint64_t bar;
  int abort;
};
static_assert(offsetof(PrepSmem, G) % 16 == 0 && offsetof(PrepSmem, inq) % 16 == 0 &&
                  offsetof(PrepSmem, beta) % 16 == 0,
              "read 16 bytes at a time");

// Pieces of the right operand X^T (k = column of X, n = row of X) of eight rows, 16 columns.
DSA_DEV void prep_right(const float* X, uint32_t (&f)[3][2]) {
  const int lane = threadIdx.x & 31;
  const float* at = X + (lane >> 2) * kPrepLd + (lane & 3) * 2;
  uint32_t p[3];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 x = *reinterpret_cast<const float2*>(at + i * 8);
    split_pair<3>(x.x, x.y, p);
#pragma unroll
    for (int m = 0; m < 3; ++m) f[m][i] = p[m];
  }
}

// y[i] += the products of x with N right operands, in three pieces each; the accumulators take
// turns
template <int N>
DSA_DEV void prep_mma(float (&y)[N][4], const uint32_t (&x)[3][4], const uint32_t (&f)[N][3][2]) {
#pragma unroll
  for (int px = 0; px < 3; ++px)
#pragma unroll
    for (int py = 0; py < 3 - px; ++py)
#pragma unroll
      for (int i = 0; i < N; ++i) mma_bf16_16816(y[i], x[px], f[i][py][0], f[i][py][1]);
}

// Pieces of T1^T: 16 columns of T1 from column 0, its 16 rows from row 0
DSA_DEV void prep_left(const float* T1, uint32_t (&fx)[3][4]) {
  const int lane = threadIdx.x & 31;
  uint32_t p[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // (m, k), (m + 8, k), (m, k + 8), (m + 8, k + 8)
    const float* at = T1 + ((lane & 3) * 2 + (i >> 1) * 8) * kPrepLd + (lane >> 2) + (i & 1) * 8;
    split_pair<3>(at[0], at[kPrepLd], p);
#pragma unroll
    for (int m = 0; m < 3; ++m) fx[m][i] = p[m];
  }
}

// T21 = -t^T: t [16 columns][8 rows]
DSA_DEV void prep_store(float* T21, const float (&t)[4]) {
  const int lane = threadIdx.x & 31;
  float* at = T21 + (lane & 3) * 2 * kPrepLd + (lane >> 2);
  at[0] = -t[0];
  at[kPrepLd] = -t[1];
  at[8] = -t[2];
  at[kPrepLd + 8] = -t[3];
}

template <bool kGroup>
__global__ void __launch_bounds__(kPrepThreads, 4) delta_prep_kernel(
    const DeltaArgs a, const __grid_constant__ DeltaMaps maps) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  PrepSmem& sm = *reinterpret_cast<PrepSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = kGroup ? a.heads / a.per_cta : a.heads;
  const int64_t slot = blockIdx.x / groups;
  const int hl0 = (int)(blockIdx.x % groups) * (kGroup ? a.per_cta : 1);  // first of its value heads
  // the sequence whose slots hold this one
  const int lo =
      find_last<kPrepThreads>(a.batch, [&](int b) { return delta_first_slot(a, b) <= slot; });
  const int64_t first = __ldg(a.q_offsets + lo), end = __ldg(a.q_offsets + lo + 1);
  const int64_t row0 = first + (slot - delta_first_slot(a, lo)) * kDeltaChunk;
  if (end - first < a.min_len || row0 >= end) return;
  const int valid = (int)(end - row0 < kDeltaChunk ? end - row0 : kDeltaChunk);
  const int hk = (a.head0 + hl0) / (a.hv / a.hk);

  const uint32_t sk = smem_u32(sm.k), sq = smem_u32(sm.q);
  const uint32_t bar = smem_u32(&sm.bar);
  if (tid == 0) {
    mbar_init(bar, 1);
    sm.abort = 0;
    fence_mbar_init();
    mbar_arrive_expect_tx(bar, 2 * kDeltaTile);
    delta_load_qk(maps, sk, sq, bar, hk, row0);
  }
  auto gates = [&](int h) {
    if (warp == 0) {
      // running sum of g log2(e), two tokens a lane, in fp64 and then as a pair of fp32.  -inf
      // (alpha = 0) becomes a finite decay that is 0 all the same, so that differences of sums
      // behind it stay numbers.
      double x[2];
  #pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = lane * 2 + i;
        const float g = t < valid ? __ldg(a.g + (row0 + t) * a.hv + h) : 0.f;
        x[i] = (g < -1e5f ? -1e5 : (double)g) * 1.4426950408889634;
      }
      double sum = x[0] + x[1];
      const double own = sum;
  #pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const double up = __shfl_up_sync(~0u, sum, m);
        if (lane >= m) sum += up;
      }
      const double first_of_two = sum - own + x[0];
      float f = (float)first_of_two;
      sm.G[lane * 2] = make_float2(f, (float)(first_of_two - f));
      f = (float)sum;
      sm.G[lane * 2 + 1] = make_float2(f, (float)(sum - f));
    } else if (warp == 1) {
  #pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = lane + i * 32;
        sm.beta[t] = t < valid ? __ldg(a.beta + (row0 + t) * a.hv + h) : 0.f;
      }
    }
  };
  gates(a.head0 + hl0);
  __syncthreads();  // the barrier is there to wait for
  if (!mbar_wait_bounded(bar, 0, a.status, &sm.abort))
    mbar_wait_bounded(bar, 0, nullptr, nullptr);  // not to leave with copies in flight
  if (valid < kDeltaChunk) {
    for (int i = 0; i < 4; ++i)
      delta_zero_rows(sm.k + i * (kDeltaTile / 2), 128, valid, tid, kPrepThreads);
    __syncthreads();
  }
  {
    const int r = tid & 63;
    const unsigned char* tile = tid < 64 ? sm.k : sm.q;
    float ss[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.norm) {
#pragma unroll 4
      for (int c = 0; c < 16; ++c) {
        const uint4 x = *reinterpret_cast<const uint4*>(tile + swz(r, c));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ss[i] = fmaf(bf16_lo(w[i]), bf16_lo(w[i]), ss[i]);
          ss[i] = fmaf(bf16_hi(w[i]), bf16_hi(w[i]), ss[i]);
        }
      }
    }
    (tid < 64 ? sm.ink : sm.inq)[r] = 
        a.norm ? 1.f / sqrtf((ss[0] + ss[1]) + (ss[2] + ss[3]) + a.eps) : 1.f;
  }

  // K K^T and Q K^T on and below the diagonal: twenty tiles of 16 rows and 8 columns, five to a
  // warp: (row tile, column tile) from (3, 0), from (3, 5) and (0, 0), from (2, 0), from (2, 5)
  // and (1, 0).  The roles turn with the CTA, so that none is always on the same scheduler.
  const int mi = lane >> 3, mr = lane & 7;
  const int role = (warp + (int)(blockIdx.x & 3)) & 3;
  const int mt_a = 3 - (role >> 1), mt_b = role >> 1;                // row tiles
  const int n_a = role & 1 ? (role == 1 ? 3 : 1) : 5;                // column tiles of mt_a
  const int nt0 = role & 1 ? 5 : 0;                                  // the first of them
  float kk[5][4], qk[5][4];
#pragma unroll
  for (int j = 0; j < 5; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) kk[j][i] = qk[j][i] = 0.f;
#pragma unroll 1
  for (int k2 = 0; k2 < 4; ++k2) {  // 32 columns of K and Q
    uint32_t fb[5][4];
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      const int nt = j < n_a ? nt0 + j : j - n_a;
      ldmatrix_x4(sk + swz(nt * 8 + mr, k2 * 4 + mi), fb[j]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t fk[4], fq[4];
      const int unit = k2 * 4 + e * 2 + (mi >> 1), r = (mi & 1) * 8 + mr;
      ldmatrix_x4(sk + swz(mt_a * 16 + r, unit), fk);
      ldmatrix_x4(sq + swz(mt_a * 16 + r, unit), fq);
#pragma unroll
      for (int j = 0; j < 5; ++j)
        if (j < n_a) {
          mma_bf16_16816(kk[j], fk, fb[j][2 * e], fb[j][2 * e + 1]);
          mma_bf16_16816(qk[j], fq, fb[j][2 * e], fb[j][2 * e + 1]);
        }
      if (role & 1) {
        ldmatrix_x4(sk + swz(mt_b * 16 + r, unit), fk);
        ldmatrix_x4(sq + swz(mt_b * 16 + r, unit), fq);
#pragma unroll
        for (int j = 0; j < 5; ++j)
          if (j >= n_a) {
            mma_bf16_16816(kk[j], fk, fb[j][2 * e], fb[j][2 * e + 1]);
            mma_bf16_16816(qk[j], fq, fb[j][2 * e], fb[j][2 * e + 1]);
          }
      }
    }
  }
  const int per = kGroup ? a.per_cta : 1;
#pragma unroll 1
  for (int hl = hl0; hl < hl0 + per; ++hl) {
    __syncthreads();  // gates and norms are there; K's and Q's tiles, or the last head's A, are free

    unsigned char* dst = a.ws + (slot * a.heads + hl) * kDeltaItemBytes;
    if (tid < 64) {
      float* scal = reinterpret_cast<float*>(dst + kDeltaScal);
      const float2 g = sm.G[tid], ge = sm.G[63];
      const float eg = exp2f(g.x + g.y);
      scal[tid] = eg * sm.ink[tid];
      scal[64 + tid] = exp2f((ge.x - g.x) + (ge.y - g.y)) * sm.ink[tid];
      scal[128 + tid] = a.scale * eg * sm.inq[tid];
      if (tid == 0) scal[192] = exp2f(ge.x + ge.y);
    }
    // this lane's two rows of either row tile
    float2 gi[2][2];
    float fa[2][2], fp[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = (m ? mt_b : mt_a) * 16 + (lane >> 2) + half * 8;
        gi[m][half] = sm.G[i];
        fa[m][half] = sm.beta[i] * sm.ink[i];
        fp[m][half] = a.scale * sm.inq[i];
      }
#pragma unroll
    for (int t = 0; t < 5; ++t) {
      const bool second = t >= n_a;
      const int mt = second ? mt_b : mt_a, nt = second ? t - n_a : nt0 + t;
      const int j = nt * 8 + (lane & 3) * 2;
      const float4 gj = *reinterpret_cast<const float4*>(sm.G + j);
      const float2 ik = *reinterpret_cast<const float2*>(sm.ink + j);
      const bool diagonal = (nt >> 1) == mt;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = mt * 16 + (lane >> 2) + half * 8;
        const float2 g = second ? gi[1][half] : gi[0][half];
        const float ra = second ? fa[1][half] : fa[0][half], rp = second ? fp[1][half] : fp[0][half];
        // e^(G_i - G_j): the high parts cancel exactly where it matters
        float x0 = (g.x - gj.x) + (g.y - gj.y), x1 = (g.x - gj.z) + (g.y - gj.w);
        if (diagonal) {  // e^-inf = 0 right of the diagonal
          if (j > i) x0 = -INFINITY;
          if (j >= i) x1 = -INFINITY;
        }
        const float d0 = ex2_approx(x0) * ik.x, d1 = ex2_approx(x1) * ik.y;
        float2 x = make_float2(ra * d0 * kk[t][half * 2], ra * d1 * kk[t][half * 2 + 1]);
        if (diagonal) {
          if (j >= i) x.x = 0.f;
          if (j + 1 >= i) x.y = 0.f;
        }
        *reinterpret_cast<float2*>(sm.A + i * kPrepLd + j) = x;
        float2 y = make_float2(rp * d0 * qk[t][half * 2], rp * d1 * qk[t][half * 2 + 1]);
        if (diagonal) {  // (not 0 times a product that may not be a number)
          if (j > i) y.x = 0.f;
          if (j >= i) y.y = 0.f;
        }
        *reinterpret_cast<uint32_t*>(dst + 3 * kDeltaMat + tri_unit(i, nt) + (lane & 3) * 4) =
            pack_bf16x2(y.x, y.y);
      }
    }
    if (tid < 64) {  // above the diagonal inside the 32 x 32 blocks
      const int i = (tid >> 5) * 32 + (tid & 31) / 2, j = (tid >> 5) * 32 + 16 + (tid & 1) * 8;
      *reinterpret_cast<float4*>(sm.A + i * kPrepLd + j) = make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4*>(sm.A + i * kPrepLd + j + 4) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    {
      // column c of the block's inverse: x_i = [i == c] - sum_{m < i} A_im x_m
      const int c = lane & 15;
      float* A = sm.A + warp * 16 * (kPrepLd + 1);
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int m = 0; m < i; m += 4) {
          const float4 v = *reinterpret_cast<const float4*>(A + i * kPrepLd + m);
          s0 = fmaf(v.x, x[m], s0);
          s1 = fmaf(v.y, x[m + 1], s1);
          s0 = fmaf(v.z, x[m + 2], s0);
          s1 = fmaf(v.w, x[m + 3], s1);
        }
        x[i] = (i == c ? 1.f : 0.f) - (s0 + s1);
      }
      __syncwarp();
      if (lane < 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) A[i * kPrepLd + c] = x[i];
      }
    }
    __syncthreads();
    // The steps 16 -> 32 -> 64 on the tensor cores, transposed: Y = T1^T A21^T, then
    // T21^T = -Y T2^T, Y going from accumulator to left operand in registers.  fp32 operands in
    // three bf16 pieces, products below 2^-24 left out.  (As fp32 products out of shared memory
    // these steps were half of the kernel's shared-memory traffic, which bounded it.)
    const int part = warp & 1, half = warp >> 1;
    {  // pair `part` of 16 x 16 blocks; rows 8 half .. of the block below
      float* T1 = sm.A + part * 32 * (kPrepLd + 1);
      float* A21 = T1 + 16 * kPrepLd;
      float y[2][4] = {}, t[1][4] = {};
      uint32_t fx[3][4], fb[2][3][2], f2[1][3][2];
      prep_left(T1, fx);
      prep_right(A21, fb[0]);
      prep_right(A21 + 8 * kPrepLd, fb[1]);
      prep_right(A21 + 16 + half * 8 * kPrepLd, f2[0]);
      prep_mma(y, fx, fb);
      split_frag<3>(y[0], y[1], fx);
      prep_mma(t, fx, f2);
      __syncthreads();
      prep_store(A21 + half * 8 * kPrepLd, t[0]);
    }
    __syncthreads();
    {  // columns 16 part .. of the 32 x 32 block below, rows 16 half ..
      float* A21 = sm.A + 32 * kPrepLd;
      float y[4][4] = {}, t[2][4] = {};
      uint32_t fx[3][4];
      // T1 and T2 are lower triangular: rows 16 part .. of T1, and the first 16 (half + 1) of Y
#pragma unroll 1
      for (int kt = part; kt < 2; ++kt) {
        uint32_t fb[4][3][2];
        prep_left(sm.A + kt * 16 * kPrepLd + part * 16, fx);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) prep_right(A21 + nt * 8 * kPrepLd + kt * 16, fb[nt]);
        prep_mma(y, fx, fb);
      }
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        if (kt > half) continue;
        uint32_t fb[2][3][2];
        split_frag<3>(y[2 * kt], y[2 * kt + 1], fx);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          prep_right(A21 + 32 + (half * 16 + e * 8) * kPrepLd + kt * 16, fb[e]);
        prep_mma(t, fx, fb);
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 2; ++e) prep_store(A21 + (half * 16 + e * 8) * kPrepLd + part * 16, t[e]);
    }
    __syncthreads();
    // T diag(beta) in three pieces, eight columns at a time
#pragma unroll 1
    for (int at = tid; at < kDeltaMat / 16; at += kPrepThreads) {
      const int block = at >> 5, kt = block >= 9 ? 3 : block >= 7 ? 2 : block >= 4 ? 1 : 0;
      const int i = (at - tri_col(kt) / 16) >> 1;
      const int c = kt * 16 + ((at & 1) ^ ((i >> 2) & 1)) * 8;
      uint32_t p[4][3];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 t = *reinterpret_cast<const float4*>(sm.A + i * kPrepLd + c + e * 4);
        const float4 w = *reinterpret_cast<const float4*>(sm.beta + c + e * 4);
        split_pair<3>(t.x * w.x, t.y * w.y, p[2 * e]);
        split_pair<3>(t.z * w.z, t.w * w.w, p[2 * e + 1]);
      }
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint4*>(dst + k * kDeltaMat + at * 16) =
            make_uint4(p[0][k], p[1][k], p[2][k], p[3][k]);
    }
    if (kGroup && hl + 1 < hl0 + per) {
      __syncthreads();
      gates(a.head0 + hl + 1);
    }
  }
}

// ------------------------------------------------------------------ chunked form: the scan
//
// A CTA walks one sequence's chunks for one head and 32 (or 16) of its 128 value columns.  Products
// are taken transposed, with 16 value columns as the rows of the tensor-core tile:
//   R^T = S K^T, QS^T = S Q^T, U^T = X^T T^T, S += U'^T K, O^T = QS^T + U^T P^T
// so that an accumulator tile is, register for register, the next product's left operand, and
// the right operands (K, Q, T, P) come from shared memory by ldmatrix.  Four warps share 16
// value columns.  Two carry the chain R -> X -> U -> S: each owns 64 of the key columns of S (32
// registers) and two of the four 16-token tiles, {0, 3} or {1, 2} (equal work in the triangular
// products), and three exchanges through shared memory a chunk bring the halves of R together
// and hand X and U around.  The other two, off the chain, compute O.  A ninth warp loads, by TMA
// into two stages.
// What bounds it: the chain's latency (220 tensor instructions a warp and chunk, which depend on
// one another in four stages); the tensor pipe, which the output warps fill in the gaps, is the
// next limit (304 a scheduler and chunk).  So accumulators alternate, eight or six between two
// uses of one, and operands are fetched one step ahead.  Measured: a chunk takes 1.65 us with one
// set of warps a CTA (8 heads), 2.1 us with two (32 heads: tensor pipe 63 %, shared-memory pipe
// 72 %); 32768 tokens x 32 heads 1.36 ms with the preparation.
constexpr int kScanNV = 32;  // value columns of a V tile
// one chunk's operands: K, Q, V, the workspace item
constexpr int kScanV = 2 * kDeltaTile;
constexpr int kScanItem = kScanV + kDeltaChunk * kScanNV * 2;
constexpr int kScanBytes = kScanItem + kDeltaItemBytes;
constexpr int kScanStage = (kScanBytes + 1023) / 1024 * 1024;
// exchange areas of 16 value columns, 512 bytes (a fragment of a warp) each unit: S [2 chunks][8
// key tiles][2 pieces], R [2 warps][4], X [4 token tiles][3 pieces], U and U' [4 token tiles][2 + 3]
constexpr int kExS = 0, kExR = kExS + 2 * 16 * 512, kExX = kExR + 8 * 512, kExU = kExX + 12 * 512;
constexpr int kScanExch = kExU + 20 * 512;
// PAIRS sets of four warps (16 value columns each) in a CTA: 2, or 1 where there are too few
// (sequence, head)s to fill the GPU with 2
template <int PAIRS>
struct ScanGeo {
  static constexpr int kParts = kDeltaDim / (16 * PAIRS);  // CTAs of a (sequence, head)
  static constexpr int kWorkers = PAIRS * 4;               // warps
  static constexpr int kThreads = kWorkers * 32 + 32;
  static constexpr int kBars = 2 * kScanStage + PAIRS * kScanExch;
  static constexpr int kSmem = kBars + 64;
};

// Barriers of the two stages: full (the loader's bytes), empty (the worker warps); of the last
// chunk's rows; and the flag that a wait has given up.
struct ScanSync {
  uint64_t full[2], empty[2], tail;
  int abort;
};

// 16-byte unit u (value columns 8u .. 8u+7) of token r in the V tile, rows of 64 bytes
DSA_DEV uint32_t swz64(int r, int u) { return r * 64 + ((u ^ ((r >> 1) & 3)) << 4); }

DSA_DEV void named_barrier_arrive(int id, int count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

DSA_DEV void st_frag(unsigned char* p, const uint32_t (&f)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(f[0], f[1], f[2], f[3]);
}
DSA_DEV void ld_frag(const unsigned char* p, uint32_t (&f)[4]) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
}

// The five (token tile, key token tile) blocks of a triangular product that warp w of a pair
// computes, its tiles being 0 and 3 or 1 and 2.  Both warps run the same code (twice the code
// was bound by instruction fetch): blocks 0 .. 3 are (second, 0), (first, 0), (second, 1),
// (second, 2), and block 4 is (3, 3) of the one or (1, 1) of the other.
DSA_DEV int tri_tile(int w, int i) { return i ? 3 - w : w; }
DSA_DEV constexpr int tri_own(int b) { return b == 1 ? 0 : 1; }
DSA_DEV constexpr int tri_kt(int b) { return b < 2 ? 0 : b - 1; }

struct ScanPlace {
  int64_t first, slot;
  int len, h, hk, dvc;  // dvc: the CTA's first value column
  const unsigned char* items;
  int64_t item_step;
};

// What a loader ends with: the copies of the last two of the `loaded` chunks are complete (or given
// up), so that shared memory is not freed under them after a wait that ran out elsewhere.  (Out of
// line: in line it moved the scan's code: 4096 tokens x 8 heads 129.2 us, so 126.4.)
template <typename Sync>
__device__ __noinline__ void scan_drain(const ScanPlace& at, Sync* sy, int loaded) {
  for (int c = loaded > 2 ? loaded - 2 : 0; c < loaded; ++c) {
    const bool part = at.len - c * kDeltaChunk < kDeltaChunk;
    mbar_wait_bounded(smem_u32(part ? &sy->tail : &sy->full[c & 1]), part ? 0 : c >> 1 & 1, nullptr,
                      nullptr);
  }
}

// The loader, one warp: chunk by chunk into the two stages as they come free.
DSA_DEV void scan_loader(const DeltaArgs& a, const DeltaMaps& maps, const ScanPlace& at,
                         unsigned char* smem, ScanSync* sy) {
  const int lane = threadIdx.x & 31;
  const int n_chunks = (at.len + kDeltaChunk - 1) / kDeltaChunk;
  int c = 0;
  for (; c < n_chunks; ++c) {
    const int valid = at.len - c * kDeltaChunk;
    if (c >= 2) {
      const bool ok =
          mbar_wait_bounded(smem_u32(&sy->empty[c & 1]), ((c >> 1) + 1) & 1, a.status, &sy->abort);
      if (__any_sync(~0u, !ok)) break;
    }
    const bool part = valid < kDeltaChunk;
    const uint32_t full = smem_u32(&sy->full[c & 1]);
    const uint32_t bar = part ? smem_u32(&sy->tail) : full;
    unsigned char* to = smem + (c & 1) * kScanStage;
    const uint32_t stage = smem_u32(to);
    const int64_t row0 = at.first + (int64_t)c * kDeltaChunk;
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, kScanBytes);
      delta_load_qk(maps, stage, stage + kDeltaTile, bar, at.hk, row0);
      tma_load_2d(stage + kScanV, &maps.v, bar, at.h * kDeltaDim + at.dvc, (int)row0);
      bulk_load(stage + kScanItem, at.items + c * at.item_step, kDeltaItemBytes, bar);
    }
    __syncwarp();
    if (part) {  // the last chunk: the rows behind the sequence's end become zeros first
      mbar_wait_bounded(bar, 0, a.status, &sy->abort);
      for (int i = 0; i < 4; ++i)
        delta_zero_rows(to + i * (kDeltaTile / 2), 128, valid, lane, 32);
      delta_zero_rows(to + kScanV, kScanNV * 2, valid, lane, 32);
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
  }
  scan_drain(at, sy, c);
}

// The chain: warp w of the pair whose exchange area is ex.
DSA_DEV void scan_chain(const DeltaArgs& a, const ScanPlace& at, unsigned char* smem,
                        ScanSync* sy, unsigned char* ex, int pair, int w) {
  const int lane = threadIdx.x & 31, mi = lane >> 3, mr = lane & 7;
  const int dv0 = at.dvc + pair * 16;
  const int bar = 1 + 3 * pair;
  const int tile[2] = {tri_tile(w, 0), tri_tile(w, 1)};
  const int their[2] = {tri_tile(1 - w, 0), tri_tile(1 - w, 1)};
  ex += lane * 16;

  // S^T of this warp: rows dv0 + lane/4 (+8), columns 64 w + 8 n + 2 (lane % 4) (+1)
  float s[8][4];
  const int64_t soff =
      ((at.slot * a.hv + at.h) * kDeltaDim + dv0 + (lane >> 2)) * kDeltaDim + w * 64 + (lane & 3) * 2;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    float2 x = make_float2(0.f, 0.f), y = x;
    if (a.state_in && at.slot >= 0) {
      x = *reinterpret_cast<const float2*>(a.state_in + soff + n * 8);
      y = *reinterpret_cast<const float2*>(a.state_in + soff + 8 * kDeltaDim + n * 8);
    }
    s[n][0] = x.x, s[n][1] = x.y, s[n][2] = y.x, s[n][3] = y.y;
  }

  const uint32_t stage0 = smem_u32(smem);
  // byte offsets of this lane's ldmatrix rows: K's token tiles (own first) in this warp's half of
  // the columns, T's blocks (0, 0) of the own tiles
  const int rb = (mi >> 1) * 8 + mr;
  uint32_t k_row[4], t_row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    k_row[i] = w * (kDeltaTile / 2) + (tile[i] * 16 + rb) * 128;
    k_row[2 + i] = w * (kDeltaTile / 2) + (their[i] * 16 + rb) * 128;
    t_row[i] = tri_unit(tile[i] * 16 + rb, mi & 1);
  }
  const int n_chunks = (at.len + kDeltaChunk - 1) / kDeltaChunk;
#pragma unroll 1
  for (int c = 0; c < n_chunks; ++c) {
    mbar_wait_bounded(smem_u32(&sy->full[c & 1]), c >> 1 & 1, a.status, &sy->abort);
    const uint32_t sk = stage0 + (c & 1) * kScanStage;
    const uint32_t st = sk + kScanItem, sv = sk + kScanV;
    const float* scal = reinterpret_cast<const float*>(smem + (c & 1) * kScanStage + kScanItem +
                                                       kDeltaScal);

    // R^T = S K^T over this warp's key columns: r[0..3] the own token tiles, r[4..7] the other's
    float r[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) r[n][i] = 0.f;
    uint32_t fb[2][4][4];
    auto load_k = [&](int kt, uint32_t (&f)[4][4]) {
      const uint32_t unit = ((kt * 2 + (mi & 1)) ^ mr) << 4;
#pragma unroll
      for (int np = 0; np < 4; ++np) ldmatrix_x4(sk + k_row[np] + unit, f[np]);
    };
    load_k(0, fb[0]);
    uint32_t fs[4][2][4];
    // (the output warps may still read the last chunk's S, in the other of two areas; they are
    // done with the one before that once bar + 1 is passed)
    unsigned char* ex_s = ex + kExS + (c & 1) * 16 * 512;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      split_frag<2>(s[2 * kt], s[2 * kt + 1], fs[kt]);
      st_frag(ex_s + ((w * 4 + kt) * 2) * 512, fs[kt][0]);
      st_frag(ex_s + ((w * 4 + kt) * 2 + 1) * 512, fs[kt][1]);
    }
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      if (kt < 3) load_k(kt + 1, fb[(kt + 1) & 1]);
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          const uint32_t(&f)[4] = fb[kt & 1][np];
          mma_bf16_16816(r[2 * np], fs[kt][p], f[0], f[1]);
          mma_bf16_16816(r[2 * np + 1], fs[kt][p], f[2], f[3]);
        }
    }
    // the other warp's tokens to it, its share of the own tokens from it
#pragma unroll
    for (int n = 0; n < 4; ++n)
      *reinterpret_cast<float4*>(ex + kExR + (w * 4 + n) * 512) =
          make_float4(r[4 + n][0], r[4 + n][1], r[4 + n][2], r[4 + n][3]);
    uint32_t fv[2][4];
    float2 av[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ldmatrix_x4_trans(sv + swz64(tile[i] * 16 + rb, pair * 2 + (mi & 1)), fv[i]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        av[i][e] = *reinterpret_cast<const float2*>(scal + tile[i] * 16 + e * 8 + (lane & 3) * 2);
    }
    // The pair's four warps: the halves of R may be read, and S by the output warps: not before,
    // so that their products take the tensor pipe while these exchange and round.  And the output
    // warps are done with the last chunk's U.
    named_barrier(bar + 1, 128);
    // X^T = V^T - R^T diag(a) of the own tokens, in three pieces, and to the other warp
    uint32_t fx[2][3][4], ft[3][3][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 o =
            *reinterpret_cast<const float4*>(ex + kExR + ((1 - w) * 4 + i * 2 + e) * 512);
        const float(&own)[4] = r[2 * i + e];
        x[e][0] = bf16_lo(fv[i][2 * e]) - av[i][e].x * (own[0] + o.x);
        x[e][1] = bf16_hi(fv[i][2 * e]) - av[i][e].y * (own[1] + o.y);
        x[e][2] = bf16_lo(fv[i][2 * e + 1]) - av[i][e].x * (own[2] + o.z);
        x[e][3] = bf16_hi(fv[i][2 * e + 1]) - av[i][e].y * (own[3] + o.w);
      }
      split_frag<3>(x[0], x[1], fx[i]);
#pragma unroll
      for (int p = 0; p < 3; ++p) st_frag(ex + kExX + (tile[i] * 3 + p) * 512, fx[i][p]);
    }
    auto load_t = [&](int own, int kt, uint32_t (&f)[3][4]) {
#pragma unroll
      for (int p = 0; p < 3; ++p) ldmatrix_x4(st + p * kDeltaMat + t_row[own] + tri_col(kt), f[p]);
    };
    load_t(0, tile[0], ft[0]);
    load_t(1, tile[0], ft[1]);
    load_t(1, tile[1], ft[2]);

    // U^T = X^T T^T of the own tokens; products of pieces below 2^-24 of the whole are left out.
    // First the blocks over the own tokens' X, under the exchange: (first tile, first), (second,
    // first), (second, second).
    float u[4][2][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) u[n][e][i] = 0.f;
#pragma unroll
    for (int px = 0; px < 3; ++px)
#pragma unroll
      for (int pt = 0; pt < 3 - px; ++pt)
#pragma unroll
        for (int b = 0; b < 3; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mma_bf16_16816(u[b][e], fx[b >> 1][px], ft[b][pt][2 * e], ft[b][pt][2 * e + 1]);
    // Then those over the other's: tiles 1 and 2 in tile 3, or tile 0 in tiles 1 and 2
    load_t(w ? 0 : 1, their[0], ft[0]);
    load_t(1, w ? their[0] : their[1], ft[1]);
    named_barrier(bar, 64);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      ld_frag(ex + kExX + (their[0] * 3 + p) * 512, fx[0][p]);
      ld_frag(ex + kExX + ((w ? their[0] : their[1]) * 3 + p) * 512, fx[1][p]);
    }
#pragma unroll
    for (int px = 0; px < 3; ++px)
#pragma unroll
      for (int pt = 0; pt < 3 - px; ++pt)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mma_bf16_16816(u[b ? 1 : 3][e], fx[b][px], ft[b][pt][2 * e], ft[b][pt][2 * e + 1]);
    // U to the output warps; U' = U diag(t) in three pieces for S, and to the other warp
    uint32_t fu[2][3][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[2][4], y[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 tv =
            *reinterpret_cast<const float2*>(scal + 64 + tile[i] * 16 + e * 8 + (lane & 3) * 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[e][j] = i ? u[1][e][j] + u[2][e][j] : u[0][e][j];
          if ((i == 0) == (w == 1)) x[e][j] += u[3][e][j];
        }
        y[e][0] = x[e][0] * tv.x;
        y[e][1] = x[e][1] * tv.y;
        y[e][2] = x[e][2] * tv.x;
        y[e][3] = x[e][3] * tv.y;
      }
      split_frag<3>(y[0], y[1], fu[i]);
      unsigned char* to = ex + kExU + tile[i] * 5 * 512;
#pragma unroll
      for (int p = 0; p < 3; ++p) st_frag(to + (2 + p) * 512, fu[i][p]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<float4*>(to + e * 512) = make_float4(x[e][0], x[e][1], x[e][2], x[e][3]);
    }
    named_barrier_arrive(bar + 2, 128);  // the output warps may read U
    // S = e^(G_C) S + U'^T K over this warp's key columns
    // over the own tokens under the exchange of U', then the other's
    auto load_kt = [&](int t, uint32_t (&f)[4][4]) {
#pragma unroll
      for (int np = 0; np < 4; ++np)
        ldmatrix_x4_trans(
            sk + swz(t * 16 + (mi & 1) * 8 + mr, w * 8 + np * 2 + (mi >> 1)), f[np]);
    };
    load_kt(tile[0], fb[0]);
    const float decay = scal[192];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] *= decay;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (g < 3) load_kt(g == 0 ? tile[1] : their[g - 1], fb[(g + 1) & 1]);
      if (g == 2) {
        named_barrier(bar, 64);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int p = 0; p < 3; ++p)
            ld_frag(ex + kExU + (their[i] * 5 + 2 + p) * 512, fu[i][p]);
      }
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          const uint32_t(&f)[4] = fb[g & 1][np];
          mma_bf16_16816(s[2 * np], fu[g & 1][p], f[0], f[1]);
          mma_bf16_16816(s[2 * np + 1], fu[g & 1][p], f[2], f[3]);
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sy->empty[c & 1]));
  }
  if (a.state_out && at.slot >= 0) {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      *reinterpret_cast<float2*>(a.state_out + soff + n * 8) = make_float2(s[n][0], s[n][1]);
      *reinterpret_cast<float2*>(a.state_out + soff + 8 * kDeltaDim + n * 8) =
          make_float2(s[n][2], s[n][3]);
    }
  }
}

// The output warps: O^T = QS^T diag(b) + U^T P^T of the own tokens.
DSA_DEV void scan_output(const DeltaArgs& a, const ScanPlace& at, unsigned char* smem,
                         ScanSync* sy, unsigned char* ex, int pair, int w) {
  const int lane = threadIdx.x & 31, mi = lane >> 3, mr = lane & 7;
  const int dv0 = at.dvc + pair * 16;
  const int bar = 1 + 3 * pair;
  const int tile[2] = {tri_tile(w, 0), tri_tile(w, 1)};
  const int kt4 = w ? 1 : 3;
  ex += lane * 16;
  const uint32_t stage0 = smem_u32(smem);
  const int rb = (mi >> 1) * 8 + mr;
  const int n_chunks = (at.len + kDeltaChunk - 1) / kDeltaChunk;

#pragma unroll 1
  for (int c = 0; c < n_chunks; ++c) {
    mbar_wait_bounded(smem_u32(&sy->full[c & 1]), c >> 1 & 1, a.status, &sy->abort);
    const uint32_t sq = stage0 + (c & 1) * kScanStage + kDeltaTile;
    const uint32_t sp = sq - kDeltaTile + kScanItem + 3 * kDeltaMat;
    const float* scal = reinterpret_cast<const float*>(smem + (c & 1) * kScanStage + kScanItem +
                                                       kDeltaScal);
    float o[3][2][4];  // first tile, second tile, block 4
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][e][j] = 0.f;
    uint32_t fq[2][2][4], fs[2][2][4];
    auto load_q = [&](int kt, uint32_t (&f)[2][4]) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        ldmatrix_x4(sq + swz(tile[i] * 16 + rb, kt * 2 + (mi & 1)), f[i]);
    };
    auto load_s = [&](int kt, uint32_t (&f)[2][4]) {
#pragma unroll
      for (int p = 0; p < 2; ++p) ld_frag(ex + kExS + (c & 1) * 16 * 512 + (kt * 2 + p) * 512, f[p]);
    };
    load_q(0, fq[0]);
    named_barrier(bar + 1, 128);
    load_s(0, fs[0]);
#pragma unroll
    for (int kt = 0; kt < 8; ++kt) {
      if (kt < 7) {
        load_q(kt + 1, fq[(kt + 1) & 1]);
        load_s(kt + 1, fs[(kt + 1) & 1]);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t(&f)[4] = fq[kt & 1][i];
          mma_bf16_16816(o[i][0], fs[kt & 1][p], f[0], f[1]);
          mma_bf16_16816(o[i][1], fs[kt & 1][p], f[2], f[3]);
        }
    }
    uint32_t fp[5][4];
#pragma unroll
    for (int b = 0; b < 5; ++b) {
      const int row = (b < 4 ? tile[tri_own(b)] : kt4) * 16 + rb;
      ldmatrix_x4(sp + tri_unit(row, (b < 4 ? tri_kt(b) : kt4) * 2 + (mi & 1)), fp[b]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 bv =
            *reinterpret_cast<const float2*>(scal + 128 + tile[i] * 16 + e * 8 + (lane & 3) * 2);
        o[i][e][0] *= bv.x;
        o[i][e][1] *= bv.y;
        o[i][e][2] *= bv.x;
        o[i][e][3] *= bv.y;
      }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sy->empty[c & 1]));  // all of the chunk's has been read
    named_barrier(bar + 2, 128);
    uint32_t fu[4][2][4];  // U in two pieces
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      float x[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 v =
            *reinterpret_cast<const float4*>(ex + kExU + ((kt < 3 ? kt : kt4) * 5 + e) * 512);
        x[e][0] = v.x, x[e][1] = v.y, x[e][2] = v.z, x[e][3] = v.w;
      }
      split_frag<2>(x[0], x[1], fu[kt]);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int b = 0; b < 5; ++b) {
        float(&acc)[2][4] = o[b < 4 ? tri_own(b) : 2];
        const uint32_t(&x)[4] = fu[b < 4 ? tri_kt(b) : 3][p];
        mma_bf16_16816(acc[0], x, fp[b][0], fp[b][1]);
        mma_bf16_16816(acc[1], x, fp[b][2], fp[b][3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[j] = (i == 0) == (w == 1) ? o[i][e][j] + o[2][e][j] : o[i][e][j];
        const uint32_t y0 = movmatrix_trans(pack_bf16x2(x[0], x[1]));
        const uint32_t y1 = movmatrix_trans(pack_bf16x2(x[2], x[3]));
        const int t = c * kDeltaChunk + tile[i] * 16 + e * 8 + (lane >> 2);
        if (t < at.len) {
          uint32_t* to = reinterpret_cast<uint32_t*>(
              a.out + ((at.first + t) * a.hv + at.h) * kDeltaDim + dv0 + (lane & 3) * 2);
          to[0] = y0;
          to[4] = y1;
        }
      }
  }
}

// Sequence b, head hl of the pass, value columns from dvc on.
DSA_DEV ScanPlace scan_place(const DeltaArgs& a, int b, int hl, int dvc) {
  ScanPlace at;
  at.h = a.head0 + hl;
  at.hk = at.h / (a.hv / a.hk);
  at.first = __ldg(a.q_offsets + b);
  at.len = (int)(__ldg(a.q_offsets + b + 1) - at.first);
  at.slot = delta_slot(a, b);
  at.dvc = dvc;
  at.items = a.ws + (delta_first_slot(a, b) * a.heads + hl) * (int64_t)kDeltaItemBytes;
  at.item_step = (int64_t)a.heads * kDeltaItemBytes;
  return at;
}

template <int PAIRS>
__global__ void __launch_bounds__(ScanGeo<PAIRS>::kThreads, 1) delta_scan_kernel(
    const DeltaArgs a, const __grid_constant__ DeltaMaps maps) {
  using Geo = ScanGeo<PAIRS>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x >> 5;
  const int part = blockIdx.x % Geo::kParts;
  const int hl = (blockIdx.x / Geo::kParts) % a.heads;
  const int b = blockIdx.x / (Geo::kParts * a.heads);
  const ScanPlace at = scan_place(a, b, hl, part * PAIRS / 2 * kScanNV);
  if (at.len < a.min_len) return;
  ScanSync* sy = reinterpret_cast<ScanSync*>(smem + Geo::kBars);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sy->full[i]), 1);
      mbar_init(smem_u32(&sy->empty[i]), Geo::kWorkers);
    }
    mbar_init(smem_u32(&sy->tail), 1);
    sy->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // chain warps, then output warps (spread over the schedulers), then the loader.  `pair`: which
  // half of the V tile
  const int set = (warp >> 1) % PAIRS, pair = PAIRS == 1 ? part & 1 : set;
  unsigned char* ex = smem + 2 * kScanStage + set * kScanExch;
  if (warp == Geo::kWorkers) scan_loader(a, maps, at, smem, sy);
  else if (warp < 2 * PAIRS) scan_chain(a, at, smem, sy, ex, pair, warp & 1);
  else scan_output(a, at, smem, sy, ex, pair, warp & 1);
}

}  // namespace dsa
