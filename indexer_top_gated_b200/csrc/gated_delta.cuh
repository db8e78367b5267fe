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
// the state crosses HBM once each way however many tokens the sequence has.
//
// Chunked form: with G the running sum of g inside a chunk of 64 tokens,
//   (I + A) U = diag(beta) (V - diag(e^G) K S0^T),  A_ij = beta_i e^(G_i - G_j) k_i.k_j (j < i)
//   O = scale (diag(e^G) Q S0^T + (tril(Q K^T) . e^(G_i - G_j)) U)
//   S = e^(G_C) S0 + U^T diag(e^(G_C - G_j)) K
// delta_prep_kernel computes what does not depend on the state, for every chunk at once:
// T = (I + A)^-1 diag(beta) and P = scale * tril(Q K^T) . e^(G_i - G_j).  delta_scan_kernel then
// walks a sequence's chunks with S in registers.  Columns of S^T (the dv axis) never meet, so
// a CTA takes 32 or 64 of the 128, and a pair of warps 16 of them.
//
// Precision: the state, the norms, the decays and every sum are fp32 (the running sum of g
// fp64, since only its differences matter and a strong decay leaves them small beside it).  The
// tensor cores take bf16, so an fp32 operand enters as two or three bf16 pieces (8 mantissa bits
// each): k, q and v are bf16 already and enter whole.  S in K S0^T has two pieces (the third
// moves the state by 1e-7 of itself), T, V - K S0^T and U have three, which leaves the state
// 1e-7 to 1e-6 off, as fp32 products would; with two it is 5e-6 off.  The output is rounded to
// bf16: P enters rounded once and U with two pieces, an error no larger than that rounding's.
#pragma once

#include <type_traits>

#include "common.cuh"

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

  float4 s[kRecRows];
  if (a.state_in && slot >= 0) {
#pragma unroll
    for (int r = 0; r < kRecRows; ++r)
      s[r] = __ldcs(reinterpret_cast<const float4*>(a.state_in + soff + r * kDeltaDim));
  } else {
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) s[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  const int hk = h / (a.hv / a.hk);
  for (int t = 0; t < n; ++t) {
    const int64_t row = row0 + t;
    const uint2 kr = __ldg(reinterpret_cast<const uint2*>(a.k + row * a.k_stride + hk * kDeltaDim) + lane);
    const uint2 qr = __ldg(reinterpret_cast<const uint2*>(a.q + row * a.q_stride + hk * kDeltaDim) + lane);
    const float vv = __bfloat162float(a.v[row * a.v_stride + (int64_t)h * kDeltaDim + dv0 + (lane & 15)]);
    const float alpha = expf(__ldg(a.g + row * a.hv + h));
    const float beta = __ldg(a.beta + row * a.hv + h);
    float k[4] = {bf16_lo(kr.x), bf16_hi(kr.x), bf16_lo(kr.y), bf16_hi(kr.y)};
    float q[4] = {bf16_lo(qr.x), bf16_hi(qr.x), bf16_lo(qr.y), bf16_hi(qr.y)};
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

// One item of the workspace, in the order in which the scan keeps it in shared memory: three
// pieces of T, P (bf16 [64][64] each, rows of 128 bytes whose 16-byte units are permuted by
// unit ^ (row & 7), which makes ldmatrix free of bank conflicts; the 16 x 16 blocks above the
// diagonal are neither written nor read), then the scalars of the tokens.
constexpr int kDeltaMat = kDeltaChunk * kDeltaChunk * 2;
constexpr int kDeltaScal = 4 * kDeltaMat;        // a[64], t[64], b[64], e^(G_C)
constexpr int kDeltaItemBytes = kDeltaScal + 1024;
constexpr int kDeltaTile = kDeltaChunk * kDeltaDim * 2;  // K or Q of a chunk: rows of 256 bytes

DSA_DEV uint32_t swz256(int row, int unit) { return row * 256 + ((unit ^ (row & 7)) << 4); }
DSA_DEV uint32_t swz128(int row, int unit) { return row * 128 + ((unit ^ (row & 7)) << 4); }

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

// ------------------------------------------------------------------ chunked form: T and P
//
// One CTA per (chunk, value head): K K^T by its four warps, then two warps invert I + A (a
// column of the inverse per thread, forward substitution in fp32 with the column in registers
// and the rows of A broadcast from shared memory) while the other two form P.
constexpr int kPrepThreads = 128;
constexpr int kPrepALd = 68;  // floats per row of A: 16-byte rows, and pairs of rows on other banks

struct PrepSmem {
  unsigned char k[kDeltaTile];
  unsigned char q[kDeltaTile];
  float A[kDeltaChunk * kPrepALd];
  double G[kDeltaChunk];
  float ink[kDeltaChunk], inq[kDeltaChunk], beta[kDeltaChunk];
};

__global__ void __launch_bounds__(kPrepThreads) delta_prep_kernel(const DeltaArgs a) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  PrepSmem& sm = *reinterpret_cast<PrepSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t item = blockIdx.x;
  const int64_t slot = item / a.heads;
  const int h = a.head0 + (int)(item % a.heads);
  // the sequence whose slots hold this one
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (delta_first_slot(a, mid) <= slot) lo = mid;
    else hi = mid - 1;
  }
  const int64_t first = __ldg(a.q_offsets + lo), end = __ldg(a.q_offsets + lo + 1);
  const int64_t row0 = first + (slot - delta_first_slot(a, lo)) * kDeltaChunk;
  const int64_t len = end - first;
  if (len < a.min_len || row0 >= end) return;
  const int valid = (int)(end - row0 < kDeltaChunk ? end - row0 : kDeltaChunk);
  const int hk = h / (a.hv / a.hk);

  const uint32_t sk = smem_u32(sm.k), sq = smem_u32(sm.q);
#pragma unroll
  for (int i = 0; i < kDeltaTile / 16 / kPrepThreads; ++i) {
    const int at = tid + i * kPrepThreads, r = at >> 4, c = at & 15;
    const bool in = r < valid;
    const int64_t row = row0 + (in ? r : 0);
    cp_async_16(sk + swz256(r, c), a.k + row * a.k_stride + hk * kDeltaDim + c * 8, in ? 16 : 0);
    cp_async_16(sq + swz256(r, c), a.q + row * a.q_stride + hk * kDeltaDim + c * 8, in ? 16 : 0);
  }
  cp_async_commit();
  if (warp == 0) {
    // running sum of g, two tokens a lane.  -inf (alpha = 0) becomes a finite decay that is 0
    // all the same, so that differences of sums behind it stay numbers.
    double x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = lane * 2 + i;
      const float g = t < valid ? __ldg(a.g + (row0 + t) * a.hv + h) : 0.f;
      x[i] = g < -1e5f ? -1e5 : (double)g;
    }
    double sum = x[0] + x[1];
    const double own = sum;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const double up = __shfl_up_sync(~0u, sum, m);
      if (lane >= m) sum += up;
    }
    sm.G[lane * 2] = sum - own + x[0];
    sm.G[lane * 2 + 1] = sum;
  } else if (warp == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = lane + i * 32;
      sm.beta[t] = t < valid ? __ldg(a.beta + (row0 + t) * a.hv + h) : 0.f;
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  {
    const int r = tid & 63;
    const unsigned char* tile = tid < 64 ? sm.k : sm.q;
    float ss = 0.f;
    if (a.norm) {
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint4 x = *reinterpret_cast<const uint4*>(tile + swz256(r, c));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ss = fmaf(bf16_lo(w[i]), bf16_lo(w[i]), ss);
          ss = fmaf(bf16_hi(w[i]), bf16_hi(w[i]), ss);
        }
      }
    }
    (tid < 64 ? sm.ink : sm.inq)[r] = a.norm ? 1.f / sqrtf(ss + a.eps) : 1.f;
  }
  __syncthreads();

  unsigned char* dst = a.ws + item * kDeltaItemBytes;
  if (tid < 64) {
    float* scal = reinterpret_cast<float*>(dst + kDeltaScal);
    const float eg = expf((float)sm.G[tid]);
    scal[tid] = eg * sm.ink[tid];
    scal[64 + tid] = expf((float)(sm.G[63] - sm.G[tid])) * sm.ink[tid];
    scal[128 + tid] = a.scale * eg * sm.inq[tid];
    if (tid == 0) scal[192] = expf((float)sm.G[63]);
  }

  // rows of 16 tokens (tile mt) of X K^T, columns up to the diagonal tile
  const int mi = lane >> 3, mr = lane & 7;
  auto rows_x_k = [&](uint32_t xs, int mt, float (&acc)[8][4]) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
#pragma unroll
    for (int kt = 0; kt < 8; ++kt) {
      uint32_t fa[4];
      ldmatrix_x4(xs + swz256(mt * 16 + (mi & 1) * 8 + mr, kt * 2 + (mi >> 1)), fa);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        if (np > mt) break;
        uint32_t fb[4];
        ldmatrix_x4(sk + swz256(np * 16 + (mi >> 1) * 8 + mr, kt * 2 + (mi & 1)), fb);
        mma_bf16_16816(acc[np * 2], fa, fb[0], fb[1]);
        mma_bf16_16816(acc[np * 2 + 1], fa, fb[2], fb[3]);
      }
    }
  };
  // the roles turn with the item: the inversion's long warp is not always on the same scheduler
  const int role = (warp + (int)(item & 3)) & 3;
  {
    float acc[8][4];
    const int mt = role;
    rows_x_k(sk, mt, acc);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt >= 2 * (mt + 1)) break;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = mt * 16 + (lane >> 2) + half * 8, j = nt * 8 + (lane & 3) * 2;
        float2 x;
        x.x = j < i ? sm.beta[i] * sm.ink[i] * sm.ink[j] * expf((float)(sm.G[i] - sm.G[j])) *
                          acc[nt][half * 2]
                    : 0.f;
        x.y = j + 1 < i ? sm.beta[i] * sm.ink[i] * sm.ink[j + 1] *
                              expf((float)(sm.G[i] - sm.G[j + 1])) * acc[nt][half * 2 + 1]
                        : 0.f;
        *reinterpret_cast<float2*>(sm.A + i * kPrepALd + j) = x;
      }
    }
  }
  __syncthreads();
  if (role >= 2) {
    // column j of T: x_i = [i == j] - sum_{m < i} A_im x_m
    const int j = (role - 2) * 32 + lane;
    const int base = (role - 2) * 32;
    float x[kDeltaChunk];
    auto solve = [&](auto from) {
      constexpr int F = decltype(from)::value;
#pragma unroll
      for (int i = F; i < kDeltaChunk; ++i) x[i] = 0.f;
#pragma unroll
      for (int i = F; i < kDeltaChunk; ++i) {
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int m = F; m < i; m += 4) {
          const float4 row = *reinterpret_cast<const float4*>(sm.A + i * kPrepALd + m);
          s0 = fmaf(row.x, x[m], s0);
          s1 = fmaf(row.y, x[m + 1], s1);
          s2 = fmaf(row.z, x[m + 2], s2);
          s3 = fmaf(row.w, x[m + 3], s3);
        }
        x[i] = (i == j ? 1.f : 0.f) - ((s0 + s1) + (s2 + s3));
      }
      const float bj = sm.beta[j];
#pragma unroll
      for (int i = F; i < kDeltaChunk; ++i) {
        if ((i >> 4) < (j >> 4)) continue;
        float y = x[i] * bj;
        unsigned char* at = dst + swz128(i, j >> 3) + (j & 7) * 2;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const __nv_bfloat16 piece = __float2bfloat16_rn(y);
          *reinterpret_cast<__nv_bfloat16*>(at + p * kDeltaMat) = piece;
          y -= __bfloat162float(piece);
        }
      }
    };
    if (base == 0) solve(std::integral_constant<int, 0>{});
    else solve(std::integral_constant<int, 32>{});
  } else {
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
      const int mt = w == 0 ? role : 3 - role;
      float acc[8][4];
      rows_x_k(sq, mt, acc);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        if (nt >= 2 * (mt + 1)) break;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int i = mt * 16 + (lane >> 2) + half * 8, j = nt * 8 + (lane & 3) * 2;
          const float f = a.scale * sm.inq[i];
          const float x = j <= i ? f * sm.ink[j] * expf((float)(sm.G[i] - sm.G[j])) *
                                       acc[nt][half * 2]
                                 : 0.f;
          const float y = j + 1 <= i ? f * sm.ink[j + 1] * expf((float)(sm.G[i] - sm.G[j + 1])) *
                                           acc[nt][half * 2 + 1]
                                     : 0.f;
          *reinterpret_cast<uint32_t*>(dst + 3 * kDeltaMat + swz128(i, nt) + (lane & 3) * 4) =
              pack_bf16x2(x, y);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ chunked form: the scan
//
// A CTA walks one sequence's chunks for one head and NV of its 128 value columns.  Products are
// taken transposed, with 16 value columns as the rows of the tensor-core tile:
//   R^T = S K^T, QS^T = S Q^T, U^T = X^T T^T, S += U'^T K, O^T = QS^T + U^T P^T
// so that an accumulator tile is, register for register, the next product's left operand, and
// the right operands (K, Q, T, P) come from shared memory by ldmatrix.  Two warps share 16 value
// columns.  Each owns 64 of the key columns of S (32 registers) and two of the four 16-token
// tiles, {0, 3} or {1, 2} (equal work in the triangular products); three exchanges through
// shared memory a chunk bring the halves of R and QS together and hand X and U around.
template <int NV>
struct ScanGeo {
  static constexpr int kPairs = NV / 16;
  static constexpr int kThreads = kPairs * 64;
  static constexpr int kVBytes = kDeltaChunk * NV * 2;
  // one chunk's operands: K, Q, the workspace item, V
  static constexpr int kItemOff = 2 * kDeltaTile;
  static constexpr int kVOff = kItemOff + kDeltaItemBytes;
  static constexpr int kStage = kVOff + kVBytes;
  // exchange area of a pair: halves of R and QS (8 KB), later U and U' (10 KB); X (6 KB)
  static constexpr int kExch = 10240 + 6144;
  static constexpr int kSmem = 2 * kStage + kPairs * kExch;
};

// 16-byte unit of value columns 8u .. 8u+7 of token r in the V tile
template <int NV>
DSA_DEV uint32_t swzv(int r, int u) {
  if (NV == 16) return r * 32 + ((u ^ ((r >> 2) & 1)) << 4);
  if (NV == 32) return r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
  return r * 128 + ((u ^ (r & 7)) << 4);
}

template <int NV>
DSA_DEV void scan_load(const DeltaArgs& a, uint32_t stage, int64_t row0, int valid, int h, int hk,
                       int dv0, const unsigned char* item) {
  using Geo = ScanGeo<NV>;
  const int tid = threadIdx.x;
#pragma unroll
  for (int i = 0; i < kDeltaTile / 16 / Geo::kThreads; ++i) {
    const int at = tid + i * Geo::kThreads, r = at >> 4, c = at & 15;
    const bool in = r < valid;
    const int64_t row = row0 + (in ? r : 0);
    cp_async_16(stage + swz256(r, c), a.k + row * a.k_stride + hk * kDeltaDim + c * 8, in ? 16 : 0);
    cp_async_16(stage + kDeltaTile + swz256(r, c), a.q + row * a.q_stride + hk * kDeltaDim + c * 8,
                in ? 16 : 0);
  }
  // T and P: the units of the 16 x 16 blocks up to the diagonal
#pragma unroll
  for (int i = 0; i < 4 * kDeltaMat / 16 / Geo::kThreads; ++i) {
    const int at = tid + i * Geo::kThreads, r = (at >> 3) & 63, c = (at & 7) ^ (r & 7);
    if (c < 2 * ((r >> 4) + 1))
      cp_async_16(stage + Geo::kItemOff + at * 16, item + at * 16, 16);
  }
  if (tid < 52) cp_async_16(stage + Geo::kItemOff + kDeltaScal + tid * 16, item + kDeltaScal + tid * 16, 16);
#pragma unroll
  for (int i = 0; i < Geo::kVBytes / 16 / Geo::kThreads; ++i) {
    const int at = tid + i * Geo::kThreads, r = at / (NV / 8), c = at % (NV / 8);
    const bool in = r < valid;
    const int64_t row = row0 + (in ? r : 0);
    cp_async_16(stage + Geo::kVOff + swzv<NV>(r, c),
                a.v + row * a.v_stride + (int64_t)h * kDeltaDim + dv0 + c * 8, in ? 16 : 0);
  }
}

DSA_DEV void st_frag(unsigned char* p, const uint32_t (&f)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(f[0], f[1], f[2], f[3]);
}
DSA_DEV void ld_frag(const unsigned char* p, uint32_t (&f)[4]) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
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

template <int NV>
__global__ void __launch_bounds__(ScanGeo<NV>::kThreads) delta_scan_kernel(const DeltaArgs a) {
  using Geo = ScanGeo<NV>;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pair = warp >> 1, w = warp & 1;
  constexpr int kParts = kDeltaDim / NV;
  const int part = blockIdx.x % kParts;
  const int hl = (blockIdx.x / kParts) % a.heads;
  const int b = blockIdx.x / (kParts * a.heads);
  const int h = a.head0 + hl, hk = h / (a.hv / a.hk);
  const int64_t first = __ldg(a.q_offsets + b);
  const int len = (int)(__ldg(a.q_offsets + b + 1) - first);
  if (len < a.min_len) return;
  const int64_t slot = delta_slot(a, b);
  const int dvc = part * NV;          // the CTA's first value column
  const int dv0 = dvc + pair * 16;    // the pair's
  const int n_chunks = (len + kDeltaChunk - 1) / kDeltaChunk;
  const unsigned char* items =
      a.ws + (delta_first_slot(a, b) * a.heads + hl) * (int64_t)kDeltaItemBytes;
  const int64_t item_step = (int64_t)a.heads * kDeltaItemBytes;

  unsigned char* ex1 = smem + 2 * Geo::kStage + pair * Geo::kExch;  // R and QS halves, then U
  unsigned char* ex2 = ex1 + 10240;                                 // X
  const uint32_t stage0 = smem_u32(smem);
  const int mi = lane >> 3, mr = lane & 7;

  // S^T of this warp: rows dv0 + lane/4 (+8), columns 64 w + 8 n + 2 (lane % 4) (+1)
  float s[8][4];
  const int64_t soff = ((slot * a.hv + h) * kDeltaDim + dv0 + (lane >> 2)) * kDeltaDim + w * 64 +
                       (lane & 3) * 2;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    float2 x = make_float2(0.f, 0.f), y = x;
    if (a.state_in && slot >= 0) {
      x = *reinterpret_cast<const float2*>(a.state_in + soff + n * 8);
      y = *reinterpret_cast<const float2*>(a.state_in + soff + 8 * kDeltaDim + n * 8);
    }
    s[n][0] = x.x, s[n][1] = x.y, s[n][2] = y.x, s[n][3] = y.y;
  }

  scan_load<NV>(a, stage0, first, len < kDeltaChunk ? len : kDeltaChunk, h, hk, dvc, items);
  cp_async_commit();

#pragma unroll 1
  for (int c = 0; c < n_chunks; ++c) {
    const int64_t row0 = first + (int64_t)c * kDeltaChunk;
    const int valid = len - c * kDeltaChunk < kDeltaChunk ? len - c * kDeltaChunk : kDeltaChunk;
    cp_async_wait<0>();
    __syncthreads();  // chunk c is in place, and every warp is done with chunk c - 1
    if (c + 1 < n_chunks) {
      const int next = len - (c + 1) * kDeltaChunk;
      scan_load<NV>(a, stage0 + ((c + 1) & 1) * Geo::kStage, row0 + kDeltaChunk,
                    next < kDeltaChunk ? next : kDeltaChunk, h, hk, dvc,
                    items + (c + 1) * item_step);
      cp_async_commit();
    }
    const uint32_t sk = stage0 + (c & 1) * Geo::kStage, sq = sk + kDeltaTile;
    const uint32_t st = sk + Geo::kItemOff, sp = st + 3 * kDeltaMat, sv = sk + Geo::kVOff;
    const float* scal = reinterpret_cast<const float*>(smem + (c & 1) * Geo::kStage + Geo::kItemOff +
                                                       kDeltaScal);

    // R^T = S K^T and QS^T = S Q^T over this warp's key columns, all tokens
    float r[8][4], qs[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) r[n][i] = qs[n][i] = 0.f;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      uint32_t fa[2][4];
      split_frag<2>(s[2 * kt], s[2 * kt + 1], fa);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        const uint32_t at = swz256(np * 16 + (mi >> 1) * 8 + mr, w * 8 + kt * 2 + (mi & 1));
        uint32_t fb[4], fq[4];
        ldmatrix_x4(sk + at, fb);
        ldmatrix_x4(sq + at, fq);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          mma_bf16_16816(r[2 * np], fa[p], fb[0], fb[1]);
          mma_bf16_16816(r[2 * np + 1], fa[p], fb[2], fb[3]);
          mma_bf16_16816(qs[2 * np], fa[p], fq[0], fq[1]);
          mma_bf16_16816(qs[2 * np + 1], fa[p], fq[2], fq[3]);
        }
      }
    }
    // own token tiles: w = 0 has 0 and 3, w = 1 has 1 and 2
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int theirs = w ? (i ? 3 : 0) : (i ? 2 : 1);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        unsigned char* at = ex1 + w * 4096 + (i * 2 + e) * 1024 + lane * 16;
        float4 x, y;
        if (w) {
          const int n = 2 * (i ? 3 : 0) + e;
          x = make_float4(r[n][0], r[n][1], r[n][2], r[n][3]);
          y = make_float4(qs[n][0], qs[n][1], qs[n][2], qs[n][3]);
        } else {
          const int n = 2 * (i ? 2 : 1) + e;
          x = make_float4(r[n][0], r[n][1], r[n][2], r[n][3]);
          y = make_float4(qs[n][0], qs[n][1], qs[n][2], qs[n][3]);
        }
        *reinterpret_cast<float4*>(at) = x;
        *reinterpret_cast<float4*>(at + 512) = y;
      }
      (void)theirs;
    }
    named_barrier(1 + pair, 64);
    float ro[4][4], qo[4][4];  // own tiles' R and QS: [2 * tile + 8-token half]
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const unsigned char* at = ex1 + (1 - w) * 4096 + (i * 2 + e) * 1024 + lane * 16;
        const float4 x = *reinterpret_cast<const float4*>(at);
        const float4 y = *reinterpret_cast<const float4*>(at + 512);
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ro[2 * i + e][j] = (w ? r[2 * (i ? 2 : 1) + e][j] : r[2 * (i ? 3 : 0) + e][j]) + xs[j];
          qo[2 * i + e][j] = (w ? qs[2 * (i ? 2 : 1) + e][j] : qs[2 * (i ? 3 : 0) + e][j]) + ys[j];
        }
      }

    // X^T = V^T - R^T diag(a) of the own tokens, handed to both warps in three pieces
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tile = w ? (i ? 2 : 1) : (i ? 3 : 0);
      uint32_t fv[4];
      ldmatrix_x4_trans(sv + swzv<NV>(tile * 16 + (mi >> 1) * 8 + mr, pair * 2 + (mi & 1)), fv);
      float x[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 av = *reinterpret_cast<const float2*>(scal + tile * 16 + e * 8 + (lane & 3) * 2);
        x[e][0] = bf16_lo(fv[2 * e]) - av.x * ro[2 * i + e][0];
        x[e][1] = bf16_hi(fv[2 * e]) - av.y * ro[2 * i + e][1];
        x[e][2] = bf16_lo(fv[2 * e + 1]) - av.x * ro[2 * i + e][2];
        x[e][3] = bf16_hi(fv[2 * e + 1]) - av.y * ro[2 * i + e][3];
      }
      uint32_t f[3][4];
      split_frag<3>(x[0], x[1], f);
#pragma unroll
      for (int p = 0; p < 3; ++p) st_frag(ex2 + (tile * 3 + p) * 512 + lane * 16, f[p]);
    }
    named_barrier(1 + pair, 64);

    // U^T = X^T T^T of the own tokens
    float u[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) u[n][i] = 0.f;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      uint32_t f[3][4];
      bool have = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tile = w ? (i ? 2 : 1) : (i ? 3 : 0);
        if (kt > tile) continue;
        if (!have) {
#pragma unroll
          for (int p = 0; p < 3; ++p) ld_frag(ex2 + (kt * 3 + p) * 512 + lane * 16, f[p]);
          have = true;
        }
#pragma unroll
        for (int pt = 0; pt < 3; ++pt) {
          uint32_t ft[4];
          ldmatrix_x4(st + pt * kDeltaMat + swz128(tile * 16 + (mi >> 1) * 8 + mr, kt * 2 + (mi & 1)),
                      ft);
#pragma unroll
          for (int px = 0; px < 3; ++px) {
            if (px + pt > 2) continue;  // below 2^-24 of the product
            mma_bf16_16816(u[2 * i], f[px], ft[0], ft[1]);
            mma_bf16_16816(u[2 * i + 1], f[px], ft[2], ft[3]);
          }
        }
      }
    }
    // U in two pieces for O, U' = U diag(t) in three for S
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tile = w ? (i ? 2 : 1) : (i ? 3 : 0);
      uint32_t f2[2][4], f3[3][4];
      split_frag<2>(u[2 * i], u[2 * i + 1], f2);
      float y[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 tv =
            *reinterpret_cast<const float2*>(scal + 64 + tile * 16 + e * 8 + (lane & 3) * 2);
        y[e][0] = u[2 * i + e][0] * tv.x;
        y[e][1] = u[2 * i + e][1] * tv.y;
        y[e][2] = u[2 * i + e][2] * tv.x;
        y[e][3] = u[2 * i + e][3] * tv.y;
      }
      split_frag<3>(y[0], y[1], f3);
      unsigned char* at = ex1 + tile * 5 * 512 + lane * 16;
#pragma unroll
      for (int p = 0; p < 2; ++p) st_frag(at + p * 512, f2[p]);
#pragma unroll
      for (int p = 0; p < 3; ++p) st_frag(at + (2 + p) * 512, f3[p]);
    }
    named_barrier(1 + pair, 64);

    // S = e^(G_C) S + U'^T K over this warp's key columns
    const float decay = scal[192];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] *= decay;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      uint32_t f[3][4];
#pragma unroll
      for (int p = 0; p < 3; ++p) ld_frag(ex1 + (kt * 5 + 2 + p) * 512 + lane * 16, f[p]);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t fb[4];
        ldmatrix_x4_trans(
            sk + swz256(kt * 16 + (mi & 1) * 8 + mr, w * 8 + np * 2 + (mi >> 1)), fb);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          mma_bf16_16816(s[2 * np], f[p], fb[0], fb[1]);
          mma_bf16_16816(s[2 * np + 1], f[p], fb[2], fb[3]);
        }
      }
    }

    // O^T = QS^T diag(b) + U^T P^T of the own tokens
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tile = w ? (i ? 2 : 1) : (i ? 3 : 0);
      float o[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 bv =
            *reinterpret_cast<const float2*>(scal + 128 + tile * 16 + e * 8 + (lane & 3) * 2);
        o[e][0] = qo[2 * i + e][0] * bv.x;
        o[e][1] = qo[2 * i + e][1] * bv.y;
        o[e][2] = qo[2 * i + e][2] * bv.x;
        o[e][3] = qo[2 * i + e][3] * bv.y;
      }
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        if (kt > tile) continue;
        uint32_t f[2][4], fp[4];
        ldmatrix_x4(sp + swz128(tile * 16 + (mi >> 1) * 8 + mr, kt * 2 + (mi & 1)), fp);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          ld_frag(ex1 + (kt * 5 + p) * 512 + lane * 16, f[p]);
          mma_bf16_16816(o[0], f[p], fp[0], fp[1]);
          mma_bf16_16816(o[1], f[p], fp[2], fp[3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t y0 = movmatrix_trans(pack_bf16x2(o[e][0], o[e][1]));
        const uint32_t y1 = movmatrix_trans(pack_bf16x2(o[e][2], o[e][3]));
        const int t = tile * 16 + e * 8 + (lane >> 2);
        if (t < valid) {
          uint32_t* at = reinterpret_cast<uint32_t*>(
              a.out + ((row0 + t) * a.hv + h) * kDeltaDim + dv0 + (lane & 3) * 2);
          at[0] = y0;
          at[4] = y1;
        }
      }
    }
  }

  if (a.state_out && slot >= 0) {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      *reinterpret_cast<float2*>(a.state_out + soff + n * 8) = make_float2(s[n][0], s[n][1]);
      *reinterpret_cast<float2*>(a.state_out + soff + 8 * kDeltaDim + n * 8) =
          make_float2(s[n][2], s[n][3]);
    }
  }
}

}  // namespace dsa
