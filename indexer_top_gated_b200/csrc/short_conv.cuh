// short_conv.cuh - the short causal convolution in front of the gated delta rule: each channel
// is filtered over its own last W rows,
//   y[t,c] = act(bias[c] + sum_{j < W} w[c,j] x[t - W + 1 + j, c]),
// the rows before a sequence's first coming from its state (W - 1 rows, newest last).
// Bound: HBM.  A thread walks kConvRun rows of 8 channels with the window in registers, so a row
// is read once (and W - 1 rows again where a run begins).
#pragma once

#include "common.cuh"

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
DSA_DEV void conv_unpack(uint4 x, uint64_t (&f)[4]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

// Grid: x = channel groups, y = runs.  Run k of sequence b is run q_offsets[b] / RUN + b + k
// (runs start at the sequence's first row, so only a sequence's first run reads its state, and
// the threads that read it are those that write the new one: in place is safe).
template <int W, int RUN>
__global__ void __launch_bounds__(kConvThreads) short_conv_kernel(const ConvArgs a) {
  const int c0 = (blockIdx.x * kConvThreads + threadIdx.x) * 8;
  const int64_t run = (int64_t)blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  int b = 0;
  for (int i = 1; i < a.batch; i += kConvThreads) {
    const int at = i + threadIdx.x;
    b += __syncthreads_count(at < a.batch && __ldg(a.q_offsets + at) / RUN + at <= run);
  }
  if (c0 >= a.channels) return;
  const int64_t first = __ldg(a.q_offsets + b);
  const int64_t n = __ldg(a.q_offsets + b + 1) - first;
  const int64_t k = run - (first / RUN + b);
  if (k > 0 && k * RUN >= n) return;
  constexpr int H = W - 1;
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
  const int rows = (int)(n - t0 < RUN ? n - t0 : RUN);
  __nv_bfloat16* out = a.out + (first + t0) * a.out_stride + c0;
  x += t0 * a.x_stride;
  // kAhead rows in flight per thread; a group of them shifts the window by renaming only
  constexpr int kAhead = W == 3 ? 4 : 6;
  static_assert(kAhead % H == 0, "a group of rows turns the window a whole number of times");
  for (int t = 0; t < rows; t += kAhead) {
    uint4 raw[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (t + e < rows) raw[e] = __ldcs(reinterpret_cast<const uint4*>(x + (t + e) * a.x_stride));
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (t + e >= rows) break;
      uint64_t now[4];
      conv_unpack(raw[e], now);
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
          y0 = __fdividef(y0, 1.f + __expf(-y0));
          y1 = __fdividef(y1, 1.f + __expf(-y1));
        }
        packed[i] = pack_bf16x2(y0, y1);
        win[e % H][i] = now[i];  // in the oldest row's place
      }
      __stcs(reinterpret_cast<uint4*>(out + (t + e) * a.out_stride),
             make_uint4(packed[0], packed[1], packed[2], packed[3]));
    }
  }
}

}  // namespace dsa
