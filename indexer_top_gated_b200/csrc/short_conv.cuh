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

DSA_DEV void conv_unpack(uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Grid: x = channel groups, y = runs.  Run k of sequence b is run q_offsets[b] / RUN + b + k
// (runs start at the sequence's first row, so only a sequence's first run reads its state, and
// the threads that read it are those that write the new one: in place is safe).
template <int W, int RUN>
__global__ void __launch_bounds__(kConvThreads) short_conv_kernel(const ConvArgs a) {
  const int c0 = (blockIdx.x * kConvThreads + threadIdx.x) * 8;
  if (c0 >= a.channels) return;
  const int64_t run = (int64_t)blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)__ldg(a.q_offsets + mid) / RUN + mid <= run) lo = mid;
    else hi = mid - 1;
  }
  const int64_t first = __ldg(a.q_offsets + lo);
  const int64_t n = __ldg(a.q_offsets + lo + 1) - first;
  const int64_t k = run - (first / RUN + lo);
  if (k > 0 && k * RUN >= n) return;
  constexpr int H = W - 1;
  const __nv_bfloat16* x = a.x + first * a.x_stride + c0;

  uint4 hist[H];  // the H rows before the run, oldest first
  if (k == 0) {
    const int s = a.state_index ? __ldg(a.state_index + lo) : lo;
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

  float w[W][8], bias[8];
  {
    uint4 raw[W];
#pragma unroll
    for (int j = 0; j < W; ++j)
      raw[j] = __ldg(reinterpret_cast<const uint4*>(a.weight + (int64_t)c0 * W) + j);
    float flat[W * 8];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float f[8];
      conv_unpack(raw[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) flat[j * 8 + i] = f[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = flat[i * W + j];
    if (a.bias) {
      conv_unpack(__ldg(reinterpret_cast<const uint4*>(a.bias + c0)), bias);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) bias[i] = 0.f;
    }
  }
  float win[W][8];  // win[W - 1]: the current row
#pragma unroll
  for (int j = 0; j < H; ++j) conv_unpack(hist[j], win[j]);

  const int64_t t0 = k * RUN;
  const int rows = (int)(n - t0 < RUN ? n - t0 : RUN);
  __nv_bfloat16* out = a.out + (first + t0) * a.out_stride + c0;
  x += t0 * a.x_stride;
  constexpr int kAhead = RUN < 4 ? RUN : 4;  // rows in flight per thread
  for (int t = 0; t < rows; t += kAhead) {
    uint4 raw[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (t + e < rows) raw[e] = __ldg(reinterpret_cast<const uint4*>(x + (t + e) * a.x_stride));
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (t + e >= rows) break;
      conv_unpack(raw[e], win[H]);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = bias[i];
#pragma unroll
        for (int j = 0; j < W; ++j) y[i] = fmaf(w[j][i], win[j][i], y[i]);
        if (a.silu) y[i] = __fdividef(y[i], 1.f + __expf(-y[i]));
      }
      *reinterpret_cast<uint4*>(out + (t + e) * a.out_stride) =
          make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                     pack_bf16x2(y[6], y[7]));
#pragma unroll
      for (int j = 0; j < H; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) win[j][i] = win[j + 1][i];
    }
  }
}

}  // namespace dsa
