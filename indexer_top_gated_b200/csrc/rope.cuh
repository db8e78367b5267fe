// rope.cuh - rotary positions of a batch's new rows, and their append to the caches.
//
// A pair (x, y) of a head at position p turns by the angle p f_i:
//   x' = m (x cos - y sin),  y' = m (x sin + y cos)
// Bound: HBM.  Each input is read once and each output written once, 16 bytes at a time; the
// angles of a row are formed once, in fp64 (p f_i passes 2^24 long before positions end), and
// shared by all its heads through shared memory, so the arithmetic stays far below the copies.
// Measured: 32768 rows of 32 query and 4 key heads and 4 indexer heads 127 us, 5.8 TB/s; 64 rows
// 4.4 us.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "find_last.cuh"

namespace dsa {

constexpr int kRopeThreads = 256;
constexpr int kRopePairs = 64;     // pairs of an attention head of 128, at most
constexpr int kRopeIdxPairs = 32;  // pairs of an indexer head of 64, at most

struct RopeTensor {
  const __nv_bfloat16* src;
  void* dst;
  int64_t src_stride;        // elements per packed row
  int heads;                 // 0: absent
};

struct RopeArgs {
  const int32_t *q_offsets, *kv_offsets;
  const int32_t* positions;  // [total_q] or nullptr: the row's position in its sequence
  CachePages pg;
  int batch;
  int64_t total_q, cache_rows;
  RopeTensor t[5];           // q, k, v, q_idx, k_idx
  int32_t* err_count;
  int interleaved, idx_fp8;
  int rot, off, idx_rot, idx_off;
  float mscale, idx_scale_q, idx_scale_k;
  double turns[kRopePairs], idx_turns[kRopeIdxPairs];  // f_i / 2 pi
};

// Two 16-byte units (8 elements each) of a head of D elements, and the pairs they hold.  Item t
// of a head: the rotated units first, then those outside them.  Both layouts take units half of
// the part apart (the two halves of eight pairs, or four pairs each), so that neighbouring
// threads touch neighbouring units: whole sectors.
struct RopeItem {
  int u0, u1;        // units
  int pair0, pair1;  // pairs of c[0 .. 3] and c[4 .. 7]; pair0 -1: not rotated
};
template <int D>
DSA_DEV RopeItem rope_item(int t, int rot, int off, bool interleaved) {
  RopeItem it;
  const int turned = rot >> 4, o = off >> 3;
  if (t < turned) {
    it.u0 = o + t;
    it.u1 = it.u0 + turned;
    it.pair0 = interleaved ? t * 4 : t * 8;
    it.pair1 = interleaved ? (t + turned) * 4 : t * 8 + 4;
  } else {
    const int j = t - turned, k = j + D / 16 - turned;
    it.u0 = j < o ? j : j + 2 * turned;
    it.u1 = k < o ? k : k + 2 * turned;
    it.pair0 = it.pair1 = -1;
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

// Turns the item's elements: a = unit u0, b = unit u1, cs = cos and sin of its eight pairs.
DSA_DEV void rope_turn(float (&a)[8], float (&b)[8], const float2 (&cs)[8], bool interleaved) {
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
      const float x = a[i], y = b[i];
      a[i] = x * cs[i].x - y * cs[i].y;
      b[i] = x * cs[i].y + y * cs[i].x;
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

DSA_DEV void rope_pairs(float2 (&c)[8], const float2* row, const RopeItem& it) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    c[j] = it.pair0 < 0 ? make_float2(1.f, 0.f) : row[it.pair0 + j];
    c[4 + j] = it.pair0 < 0 ? make_float2(1.f, 0.f) : row[it.pair1 + j];
  }
}

// One item of a head in registers: turned if it is a rotated one, then stored at element `to` of
// the output.
DSA_DEV void rope_finish(const RopeTensor& x, int64_t to, const RopeItem& it, uint4 u, uint4 w,
                         bool turn, const float2 (&cs)[8], bool inter, bool fp8, float scale) {
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(x.dst) + to;
  if (!turn && !fp8) {
    *reinterpret_cast<uint4*>(dst + it.u0 * 8) = u;
    *reinterpret_cast<uint4*>(dst + it.u1 * 8) = w;
    return;
  }
  float f[8], g[8];
  rope_unpack(u, f);
  rope_unpack(w, g);
  if (turn) rope_turn(f, g, cs, inter);
  if (fp8) {
    unsigned char* d8 = static_cast<unsigned char*>(x.dst) + to;
    rope_store_fp8(d8 + it.u0 * 8, f, scale);
    rope_store_fp8(d8 + it.u1 * 8, g, scale);
  } else {
    rope_store_bf16(dst + it.u0 * 8, f);
    rope_store_bf16(dst + it.u1 * 8, g);
  }
}

// ROWS consecutive packed rows per CTA, 256 / ROWS threads a row.  A thread keeps one item of a
// head and steps over the heads of q, k and v (one list), then those of q_idx and k_idx.  Its
// copies go through its own slots of a ring in shared memory, kRopeAhead items in flight, and the
// first are under way before the row's sequence and angles are known: the kernel is bound by how
// much it keeps in flight, and registers would hold less.
constexpr int kRopeAhead = 4;

template <int ROWS>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ uint4 ring[kRopeAhead + 1][2][kRopeThreads];
  __shared__ float2 cs[ROWS][kRopePairs], ics[ROWS][kRopeIdxPairs];
  __shared__ int64_t q_rows[ROWS], c_rows[ROWS];
  __shared__ int pos[ROWS];
  const int tid = threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.x * ROWS;
  const int n = (int)(a.total_q - r0 < ROWS ? a.total_q - r0 : ROWS);
  constexpr int kThreads = kRopeThreads / ROWS, kHeads = kThreads / 8, kIdxHeads = kThreads / 4;
  const int my = tid / kThreads, t = tid % kThreads;
  const int64_t row = r0 + my;
  const bool inter = a.interleaved != 0;
  const int nq = a.t[0].heads, nk = nq + a.t[1].heads, heads = my < n ? nk + a.t[2].heads : 0;
  const int ni = a.t[3].heads, idx_heads = my < n ? ni + a.t[4].heads : 0;
  const RopeItem it = rope_item<128>(t % 8, a.rot, a.off, inter);
  const RopeItem iit = rope_item<64>(t % 4, a.idx_rot, a.idx_off, inter);

  // head vh of the list q, k, v (an absent tensor has no heads)
  auto source = [&](int vh) {
    const RopeTensor& x = a.t[vh < nq ? 0 : vh < nk ? 1 : 2];
    return x.src + row * x.src_stride + (vh - (vh < nq ? 0 : vh < nk ? nq : nk)) * 128;
  };
  auto idx_source = [&](int vh) {
    const RopeTensor& x = a.t[vh < ni ? 3 : 4];
    return x.src + row * x.src_stride + (vh < ni ? vh : vh - ni) * 64;
  };
  const uint32_t slot = smem_u32(&ring[0][0][tid]);
  constexpr uint32_t kHalf = sizeof(ring[0][0]), kSlot = sizeof(ring[0]);
  auto fetch = [&](uint32_t to, const __nv_bfloat16* src, const RopeItem& i) {
    cp_async_16(to, src + i.u0 * 8, 16);
    cp_async_16(to + kHalf, src + i.u1 * 8, 16);
  };
  if (t / 4 < idx_heads) fetch(slot + kRopeAhead * kSlot, idx_source(t / 4), iit);
#pragma unroll
  for (int e = 0; e < kRopeAhead; ++e) {
    const int vh = t / 8 + e * kHeads;
    if (vh < heads) fetch(slot + e * kSlot, source(vh), it);
    cp_async_commit();
  }

  const int b0 = find_last<kRopeThreads>(
      a.batch, [&](int b) { return (int64_t)__ldg(a.q_offsets + b) <= r0; });
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
    const double x = (double)pos[i] * (j < n_att ? a.turns[j] : a.idx_turns[j - n_att]);
    float s, c;
    sincospif(2.f * (float)(x - rint(x)), &s, &c);
    const float2 v = make_float2(c * a.mscale, s * a.mscale);
    if (j < n_att) cs[i][j] = v;
    else ics[i][j - n_att] = v;
  }
  __syncthreads();
  if (my >= n) return;
  const int64_t q_row = q_rows[my], c_row = c_rows[my];
  float2 c[8];
  rope_pairs(c, cs[my], it);
  const uint4* mine = &ring[0][0][tid];
#pragma unroll 1
  for (int vh = t / 8; vh < heads; vh += kRopeAhead * kHeads) {
#pragma unroll
    for (int e = 0; e < kRopeAhead; ++e) {
      cp_async_wait<kRopeAhead - 1>();
      const uint4 u = mine[e * 2 * kRopeThreads], w = mine[(e * 2 + 1) * kRopeThreads];
      const int now = vh + e * kHeads, next = now + kRopeAhead * kHeads;
      if (next < heads) fetch(slot + e * kSlot, source(next), it);
      cp_async_commit();
      if (now >= heads) continue;
      const RopeTensor& x = a.t[now < nq ? 0 : now < nk ? 1 : 2];
      const int h = now - (now < nq ? 0 : now < nk ? nq : nk);
      const int64_t to = now < nq ? q_row : c_row;
      if (to >= 0)
        rope_finish(x, (to * x.heads + h) * 128, it, u, w, now < nk && it.pair0 >= 0, c, inter,
                    false, 1.f);
    }
  }
  // the indexer's heads, 4 + 4 at most: one item a thread, or none
  static_assert(kIdxHeads >= 8, "");
  const int vh = t / 4;
  if (vh >= idx_heads) return;
  rope_pairs(c, ics[my], iit);
  cp_async_wait<0>();
  const bool first = vh < ni;
  const RopeTensor& x = a.t[first ? 3 : 4];
  const int64_t to = first ? q_row : c_row;
  if (to >= 0)
    rope_finish(x, (to * x.heads + (first ? vh : vh - ni)) * 64, iit,
                mine[kRopeAhead * 2 * kRopeThreads], mine[(kRopeAhead * 2 + 1) * kRopeThreads],
                iit.pair0 >= 0, c, inter, a.idx_fp8, first ? a.idx_scale_q : a.idx_scale_k);
}

}  // namespace dsa
