// rope.cuh - rotary positions of a batch's new rows, and their append to the caches.
//
// A pair (x, y) of a head at position p turns by the angle p f_i:
//   x' = m (x cos - y sin),  y' = m (x sin + y cos)
// Bound: HBM.  Each input is read once and each output written once, 16 bytes at a time; the
// angles of a row are formed once, in fp64 (p f_i passes 2^24 long before positions end), and
// shared by all its heads through shared memory, so the arithmetic stays far below the copies.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace dsa {

constexpr int kRopeThreads = 256;
constexpr int kRopePairs = 64;     // pairs of an attention head of 128, at most
constexpr int kRopeIdxPairs = 32;  // pairs of an indexer head of 64, at most

struct RopeTensor {
  const __nv_bfloat16* src;  // nullptr: absent
  void* dst;
  int64_t src_stride;        // elements per packed row
  int heads;
};

struct RopeArgs {
  const int32_t *q_offsets, *kv_offsets;
  const int32_t* positions;  // [total_q] or nullptr: the row's position in its sequence
  CachePages pg;
  int batch;
  int64_t total_q, cache_rows;
  RopeTensor q, k, v, q_idx, k_idx;
  int32_t* err_count;
  int interleaved, idx_fp8;
  int rot, off, idx_rot, idx_off;
  float mscale, idx_scale_q, idx_scale_k;
  double freq[kRopePairs], idx_freq[kRopeIdxPairs];
};

// Two 16-byte units (8 elements each) of a head of D elements, and how they turn.  Item t of a
// head: the rotated units first (a pair's two halves, or two adjacent units of pairs), then the
// units outside them.
struct RopeItem {
  int u0, u1;  // units
  int pair0;   // first pair of unit u0, -1: not rotated
};
template <int D>
DSA_DEV RopeItem rope_item(int t, int rot, int off, bool interleaved) {
  RopeItem it;
  const int turned = rot >> 4, o = off >> 3;
  if (t < turned) {
    if (interleaved) {
      it.u0 = o + 2 * t;
      it.u1 = it.u0 + 1;
    } else {
      it.u0 = o + t;
      it.u1 = it.u0 + turned;
    }
    it.pair0 = t * 8;
  } else {
    int j = (t - turned) * 2;
    it.u0 = j < o ? j : j + 2 * turned;
    ++j;
    it.u1 = j < o ? j : j + 2 * turned;
    it.pair0 = -1;
  }
  return it;
}

DSA_DEV void rope_unpack(uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Turns the item's elements: a = unit u0, b = unit u1, cs = cos and sin of the row's pairs.
DSA_DEV void rope_turn(float (&a)[8], float (&b)[8], const float2* cs, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c = cs[i], d = cs[4 + i];
      const float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = x * c.x - y * c.y;
      a[2 * i + 1] = x * c.y + y * c.x;
      const float z = b[2 * i], w = b[2 * i + 1];
      b[2 * i] = z * d.x - w * d.y;
      b[2 * i + 1] = z * d.y + w * d.x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 c = cs[i];
      const float x = a[i], y = b[i];
      a[i] = x * c.x - y * c.y;
      b[i] = x * c.y + y * c.x;
    }
  }
}

DSA_DEV void rope_store_bf16(__nv_bfloat16* dst, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                 pack_bf16x2(f[6], f[7]));
}

// e4m3 of value / scale, to nearest even, saturating at the largest finite value
DSA_DEV void rope_store_fp8(unsigned char* dst, const float (&f)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[i] |= (uint32_t)__nv_cvt_float_to_fp8(f[4 * i + j] / scale, __NV_SATFINITE, __NV_E4M3)
              << (8 * j);
  }
  *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

// All items of one tensor over the CTA's rows.  dst row of row i: rows[i] (-1: not written).
template <int D, bool kRotate, bool kIdx>
DSA_DEV void rope_tensor(const RopeArgs& a, const RopeTensor& x, int64_t r0, int n,
                         const int64_t* rows, const float2* cs, int cs_ld, float scale) {
  if (!x.src) return;
  const int per_row = x.heads * (D / 16);
  const int rot = !kRotate ? 0 : kIdx ? a.idx_rot : a.rot;
  const int off = kIdx ? a.idx_off : a.off;
  const bool inter = a.interleaved != 0;
#pragma unroll 2
  for (int at = threadIdx.x; at < n * per_row; at += kRopeThreads) {
    const int i = at / per_row, rem = at - i * per_row;
    const int h = rem / (D / 16);
    const RopeItem it = rope_item<D>(rem % (D / 16), rot, off, inter);
    const int64_t row = rows[i];
    if (row < 0) continue;
    const __nv_bfloat16* src = x.src + (r0 + i) * x.src_stride + h * D;
    const uint4 u = *reinterpret_cast<const uint4*>(src + it.u0 * 8);
    const uint4 w = *reinterpret_cast<const uint4*>(src + it.u1 * 8);
    const int64_t to = (row * x.heads + h) * D;
    if (it.pair0 < 0 && !(kIdx && a.idx_fp8)) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(x.dst) + to;
      *reinterpret_cast<uint4*>(dst + it.u0 * 8) = u;
      *reinterpret_cast<uint4*>(dst + it.u1 * 8) = w;
      continue;
    }
    float f[8], g[8];
    rope_unpack(u, f);
    rope_unpack(w, g);
    if (it.pair0 >= 0) rope_turn(f, g, cs + i * cs_ld + it.pair0, inter);
    if (kIdx && a.idx_fp8) {
      unsigned char* dst = static_cast<unsigned char*>(x.dst) + to;
      rope_store_fp8(dst + it.u0 * 8, f, scale);
      rope_store_fp8(dst + it.u1 * 8, g, scale);
    } else {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(x.dst) + to;
      rope_store_bf16(dst + it.u0 * 8, f);
      rope_store_bf16(dst + it.u1 * 8, g);
    }
  }
}

// ROWS consecutive packed rows per CTA.
template <int ROWS>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 cs[ROWS][kRopePairs], ics[ROWS][kRopeIdxPairs];
  __shared__ int64_t q_rows[ROWS], c_rows[ROWS];
  __shared__ int pos[ROWS];
  const int tid = threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.x * ROWS;
  const int n = (int)(a.total_q - r0 < ROWS ? a.total_q - r0 : ROWS);
  const int b0 = seq_of_row_cta<kRopeThreads>(a.q_offsets, a.batch, r0);
  if (tid < n) {
    const int64_t r = r0 + tid;
    int64_t q_row = -1, c_row = -1;
    int p = 0;
    if (r < __ldg(a.q_offsets + a.batch)) {  // rows behind the last sequence stay as they are
      int b = b0;
      int64_t end = __ldg(a.q_offsets + b + 1);
      while (end <= r) end = __ldg(a.q_offsets + ++b + 1);
      const int64_t kv0 = __ldg(a.kv_offsets + b), len = __ldg(a.kv_offsets + b + 1) - kv0;
      const int64_t at = len - (end - r);
      q_row = r;
      p = a.positions ? __ldg(a.positions + r) : (int)at;
      if (at >= 0) {
        if (!a.pg.table) {
          c_row = kv0 + at < a.cache_rows ? kv0 + at : -1;
        } else if ((at >> a.pg.shift) < a.pg.max_pages) {
          const int page = __ldg(a.pg.table + (int64_t)b * a.pg.max_pages + (at >> a.pg.shift));
          if (page >= 0 && page < a.pg.n_pages)
            c_row = ((int64_t)page << a.pg.shift) + (at & ((int64_t(1) << a.pg.shift) - 1));
        }
      }
      if (c_row < 0 && a.err_count) atomicAdd(a.err_count, 1);
    }
    q_rows[tid] = q_row;
    c_rows[tid] = c_row;
    pos[tid] = p;
  }
  __syncthreads();
  const int n_att = a.rot >> 1, n_idx = a.idx_rot >> 1, per = n_att + n_idx;
  for (int at = tid; at < n * per; at += kRopeThreads) {
    const int i = at / per, j = at - i * per;
    const double f = j < n_att ? a.freq[j] : a.idx_freq[j - n_att];
    double x = (double)pos[i] * f;
    x -= rint(x * 0.15915494309189533577) * 6.283185307179586477;
    float s, c;
    sincosf((float)x, &s, &c);
    const float2 v = make_float2(c * a.mscale, s * a.mscale);
    if (j < n_att) cs[i][j] = v;
    else ics[i][j - n_att] = v;
  }
  __syncthreads();
  rope_tensor<128, true, false>(a, a.q, r0, n, q_rows, &cs[0][0], kRopePairs, 1.f);
  rope_tensor<128, true, false>(a, a.k, r0, n, c_rows, &cs[0][0], kRopePairs, 1.f);
  rope_tensor<128, false, false>(a, a.v, r0, n, c_rows, &cs[0][0], kRopePairs, 1.f);
  rope_tensor<64, true, true>(a, a.q_idx, r0, n, q_rows, &ics[0][0], kRopeIdxPairs, a.idx_scale_q);
  rope_tensor<64, true, true>(a, a.k_idx, r0, n, c_rows, &ics[0][0], kRopeIdxPairs, a.idx_scale_k);
}

}  // namespace dsa
