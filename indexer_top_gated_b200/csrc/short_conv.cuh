// short_conv.cuh - the short causal convolution in front of the gated delta rule: each channel
// is filtered over its own last W rows,
//   y[t,c] = act(bias[c] + sum_{j < W} w[c,j] x[t - W + 1 + j, c]),
// the rows before a sequence's first coming from its state (W - 1 rows, newest last).
// Bound: HBM, closely followed by the special-function pipe (74 %: an exponential and a reciprocal
// for each activation).  A thread walks a run of rows of 8 channels (48, in small batches 8, 1 for single
// tokens) with the window in registers, so a row is read once (and W - 1 rows again where a run
// begins).  Measured: 32768 rows x 8192 channels 172 us, 6.2 TB/s.
#pragma once

#include "common.cuh"
#include "find_last.cuh"

namespace dsa {

constexpr int kConvThreads = 128;
constexpr int kConvMaxWidth = 4;

struct ConvArgs {
  const int32_t* q_offsets;
  int batch;
  const __nv_bfloat16* x;
  int64_t x_stride, out_stride;
  const __nv_bfloat16 *weight, *bias;  // [channels, W], [channels] or nullptr
  const __nv_bfloat16* state_in;       // [n_states, W - 1, channels] or nullptr: zeros
  __nv_bfloat16* state_out;            // the same, or nullptr: not kept
  const int32_t* state_index;
  int n_states, channels, silu;
  __nv_bfloat16* out;
};

// Two fp32 values, for the packed multiply-add of sm_100.
DSA_DEV uint64_t f32x2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
DSA_DEV uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
DSA_DEV float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
DSA_DEV void conv_unpack(uint4 x, uint64_t (&f)[4]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

// Grid: x = channel groups, y = runs.  Run k of sequence b is run q_offsets[b] / RUN + b + k
// (runs start at the sequence's first row, so only a sequence's first run reads its state, and
// the threads that read it are those that write the new one: in place is safe).  RUN == 1, for
// single tokens: run b is sequence b, all of it.
// Four CTAs an SM, said to the compiler: left to itself it spilled with three taps for the sake of
// a sixth CTA (14000 rows x 5128 channels 55.4 us, so 51.5; the other widths as fast or 1 % faster).
template <int W, int RUN>
__global__ void __launch_bounds__(kConvThreads, 4) short_conv_kernel(const ConvArgs a) {
  const int c0 = (blockIdx.x * kConvThreads + threadIdx.x) * 8;
  const int64_t run = (int64_t)blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  int b = 0;
  if (RUN == 1) {
    if (run >= a.batch) return;
    b = (int)run;
  } else {
    b = find_last<kConvThreads>(
        a.batch, [&](int i) { return __ldg(a.q_offsets + i) / RUN + (int64_t)i <= run; });
  }
  if (c0 >= a.channels) return;
  const int64_t first = __ldg(a.q_offsets + b);
  const int64_t n = __ldg(a.q_offsets + b + 1) - first;
  const int64_t k = RUN == 1 ? 0 : run - (first / RUN + b);
  constexpr int H = W - 1;
  if (k > 0 && k * RUN >= n) return;
  const __nv_bfloat16* x = a.x + first * a.x_stride + c0;

  uint4 hist[H];  // the H rows before the run, oldest first
  if (k == 0) {
    const int s = a.state_index ? __ldg(a.state_index + b) : b;
    const bool kept = s >= 0 && s < a.n_states;
    const int64_t at = (int64_t)(kept ? s : 0) * H * a.channels + c0;
#pragma unroll
    for (int j = 0; j < H; ++j)
      hist[j] = kept && a.state_in
                    ? *reinterpret_cast<const uint4*>(a.state_in + at + (int64_t)j * a.channels)
                    : make_uint4(0, 0, 0, 0);
    if (kept && a.state_out) {
      // the last H rows of (state, x); with n < H rows some are the old state's
#pragma unroll
      for (int j = 0; j < H; ++j) {
        uint4 v;
        if (n - H + j >= 0) {
          v = __ldg(reinterpret_cast<const uint4*>(x + (n - H + j) * a.x_stride));
        } else {
          v = hist[H - 1];
#pragma unroll
          for (int i = 0; i + 1 < H; ++i)
            if (n + j == i) v = hist[i];
        }
        *reinterpret_cast<uint4*>(a.state_out + at + (int64_t)j * a.channels) = v;
      }
    }
    if (n == 0) return;
  } else {
#pragma unroll
    for (int j = 0; j < H; ++j)
      hist[j] = __ldg(reinterpret_cast<const uint4*>(x + (k * RUN - H + j) * a.x_stride));
  }

  uint64_t w[W][4], bias[4];
  {
    float flat[W * 8];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const uint4 raw = __ldg(reinterpret_cast<const uint4*>(a.weight + (int64_t)c0 * W) + j);
      const uint32_t p[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        flat[j * 8 + 2 * i] = __uint_as_float(p[i] << 16);
        flat[j * 8 + 2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = f32x2(flat[2 * i * W + j], flat[(2 * i + 1) * W + j]);
    conv_unpack(a.bias ? __ldg(reinterpret_cast<const uint4*>(a.bias + c0)) : make_uint4(0, 0, 0, 0),
                bias);
  }
  uint64_t win[H][4];
#pragma unroll
  for (int j = 0; j < H; ++j) conv_unpack(hist[j], win[j]);

  const int64_t t0 = k * RUN;
  const int rows = (int)(RUN == 1 || n - t0 < RUN ? n - t0 : RUN);
  __nv_bfloat16* out = a.out + (first + t0) * a.out_stride + c0;
  x += t0 * a.x_stride;
  // A ring of rows in shared memory keeps kGroup of them in flight without holding registers.  A
  // thread reads back only what it copied itself: no barrier.  A group of rows turns ring and
  // window a whole number of times, so both are indexed by constants (a group of one row turns the
  // window itself).
  constexpr int kGroup = RUN == 1 ? 1 : H == 3 ? 6 : 8;
  __shared__ uint4 ring[kGroup][kConvThreads];
  const uint4* mine = &ring[0][threadIdx.x];
  const uint32_t slot = smem_u32(mine);
  const int64_t x_step = a.x_stride, out_step = a.out_stride;
#pragma unroll
  for (int e = 0; e < kGroup; ++e) {
    if (e < rows) cp_async_16(slot + e * sizeof(ring[0]), x, 16);
    cp_async_commit();
    x += x_step;
  }
#pragma unroll 1
  for (int left = rows; left > 0; left -= kGroup) {
#pragma unroll
    for (int e = 0; e < kGroup; ++e) {
      cp_async_wait<kGroup - 1>();
      uint64_t now[4];
      conv_unpack(mine[e * kConvThreads], now);
      if (e + kGroup < left) cp_async_16(slot + e * sizeof(ring[0]), x, 16);
      cp_async_commit();
      x += x_step;
      uint32_t packed[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint64_t acc = bias[i];
#pragma unroll
        for (int j = 0; j < H; ++j) acc = fma_f32x2(w[j][i], win[(e + j) % H][i], acc);
        acc = fma_f32x2(w[H][i], now[i], acc);
        float y0, y1;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(y0), "=f"(y1) : "l"(acc));
        if (a.silu) {
          // y / (1 + e^-y).  Where 1 + e^-y passes 2^126 (y below -87) its reciprocal is 0.  (One
          // reciprocal for both by their product needs bounded exponents, which is wrong for large
          // -y, and took two instructions more: 199 against 181 us)
          constexpr float kLog2e = 1.44269504f;
          y0 *= rcp_approx(1.f + ex2_approx(-kLog2e * y0));
          y1 *= rcp_approx(1.f + ex2_approx(-kLog2e * y1));
        }
        packed[i] = pack_bf16x2(y0, y1);
        win[e % H][i] = now[i];  // in the oldest row's place
      }
      if (e < left)
        __stcs(reinterpret_cast<uint4*>(out),
               make_uint4(packed[0], packed[1], packed[2], packed[3]));
      out += out_step;
    }
    if (kGroup == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t newest = win[0][i];
#pragma unroll
        for (int j = 0; j + 1 < H; ++j) win[j][i] = win[j + 1][i];
        win[H - 1][i] = newest;
      }
    }
  }
}

}  // namespace dsa
