// kvcache.cuh -- query/key norms with the rotary positions, and the append
// of new keys and values to the paged cache.
//
// A head row x of D elements becomes y = x (mean x^2 + eps)^-1/2 gamma (or
// y = x without a norm), then each rotated pair (a, b) at frequency w and
// position t becomes (a cos tw - b sin tw, b cos tw + a sin tw): all in fp32,
// rounded once when stored.  The angle t w is formed and reduced to a
// fraction of a turn in fp64: in fp32 a position of 10^6 would be off by up
// to 0.06 rad.
//
// What bounds it: one read and one write of every row (plus launch latency
// for a window's few rows).  A block takes ROWS rows, computes
// their rotations once in shared memory for all heads, and streams the heads
// with D / 8 lanes each, two 8-byte (four-element) pieces per lane placed so
// that both elements of a pair sit in the same lane.  A warp stays with one
// row: dealing head rows out across rows cost more in index arithmetic than
// the arithmetic itself.  8192 rows of 16 + 4 heads of 128: 18.1 us, 4.6 TB/s
// (70 % of a copy; the instructions, about 100 per 16 elements of a lane, are
// the rest), with the append's values 22.2 us (25.3 us to an e4m3 cache: the
// divisions by the scale and the conversions); four rows 2.6 to 3.0 and 3.3 us.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

constexpr int kKvRows = 4;  // rows of a block, a warp each, once there are enough of them
// one row's heads are shared by eight warps
constexpr int kv_threads(int rows) { return rows == 1 ? 256 : 32 * rows; }
constexpr int kKvMaxDim = 128;

// A sequence's rows in the call and its cache length, checked: the offsets
// and lengths are device data, and no index formed from them may leave the
// caller's buffers.
struct SeqView {
  int row0, rows, kv;
  bool ok;
};

MOE_HOST_DEV_INLINE SeqView seq_check(int row0, int end, int kv, int n_rows, int max_pages, int page) {
  SeqView s;
  s.row0 = row0;
  s.kv = kv;
  s.ok = row0 >= 0 && end >= row0 && end <= n_rows && kv >= end - row0 &&
         (long long)kv <= (long long)max_pages * page;
  s.rows = s.ok ? end - row0 : 0;
  if (!s.ok) s.kv = 0;
  return s;
}
MOE_DEV SeqView seq_view(const int *row_off, const int *kv_len, int b, int n_rows, int max_pages,
                         int page) {
  return seq_check(__ldg(row_off + b), __ldg(row_off + b + 1), __ldg(kv_len + b), n_rows, max_pages, page);
}

struct KvRowsParams {
  const uint16_t *q, *k, *v;          // bf16 rows; v null without a cache
  long long q_stride, k_stride, v_stride;  // elements between rows
  uint16_t *q_out, *k_out;            // bf16; k_out null with a cache
  long long q_out_stride, k_out_stride;
  const int *pos;                     // [n_rows], without a cache
  const float *q_gamma, *k_gamma;     // [D] or null
  float eps;
  int norm;
  const double *inv_freq;             // [rot / 2] or null
  int rot;
  int n_rows, n_q, n_kv;
  // cache
  uint8_t *k_cache, *v_cache;         // [n_pages][n_kv][page][D]
  const float *k_scale, *v_scale;     // e4m3: [n_kv] or null
  const int *page_table, *row_off, *kv_len;
  int n_pages, n_seqs, max_pages, page;
  int *status;
};

// two bf16 values as a pair of fp32
MOE_DEV uint64_t bf16x2_to_f2(uint32_t u) {
  return f2_pack(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
MOE_DEV uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
MOE_DEV uint32_t f2_to_bf16x2(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16(lo, hi);
}
// Four e4m3 values of v / scale, round to nearest even; finite values past the type's
// largest (and infinities) become +-448, NaN stays NaN.
MOE_DEV uint32_t f2_to_e4m3x4(uint64_t v0, uint64_t v1, float scale) {
  float2 a, b;
  f2_unpack(v0, a.x, a.y);
  f2_unpack(v1, b.x, b.y);
  a.x /= scale, a.y /= scale, b.x /= scale, b.y /= scale;
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// CACHE 0: q and k rows to q_out and k_out; 1: q rows to q_out (when given),
// k and v rows to a bf16 cache; 2: the same with an e4m3 cache.
template <int D, int CACHE, int ROWS, bool INTER>
__global__ void __launch_bounds__(kv_threads(ROWS)) kv_rows_kernel(KvRowsParams p) {
  constexpr int kKvThreads = kv_threads(ROWS);
  constexpr int LPH = D / 8;    // lanes of a head row
  constexpr int HPW = 32 / LPH; // head rows of a warp's step
  constexpr int NW = kKvThreads / 32;
  __shared__ __align__(16) float2 s_cs[ROWS][kKvMaxDim / 2];
  __shared__ int s_seq[ROWS];   // sequences that end at or before the row
  __shared__ int s_pos[ROWS];
  __shared__ long long s_at[ROWS];  // cache row of KV head 0, or -1
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * ROWS;
  const int nr = min(ROWS, p.n_rows - r0);
  if (CACHE && tid < ROWS) s_seq[tid] = 0;
  pdl_wait();

  // A row's heads are shared by NW / ROWS warps, HPW at a time; a
  // warp stays with its row, whose rotation it holds in registers.
  const int heads = p.n_q + p.n_kv * (CACHE ? 2 : 1);
  const int h_first = (CACHE && p.q == nullptr) ? p.n_q : 0;  // first head of the call
  const int parts = NW / ROWS;
  const int r = wid / parts, part = wid % parts, sub = lane % LPH;
  const long long row = r0 + r;
  const bool mine = r < nr;
  // the lane's two pieces of a head row: four first and four second elements
  // of rotated pairs, or eight neighbours
  int e0, e1;
  const int half = p.rot / 2;
  const bool turns = p.inv_freq != nullptr && 4 * sub < half;
  if (turns && !INTER) {
    e0 = 4 * sub;
    e1 = e0 + half;
  } else {
    e0 = 8 * sub;
    e1 = e0 + 4;
  }
  const int step = parts * HPW;
  int h = h_first + part * HPW + lane / LPH;
  const uint16_t *q_row = p.q + row * p.q_stride, *k_row = p.k + row * p.k_stride - (long long)p.n_q * D;
  const uint16_t *v_row = CACHE ? p.v + row * p.v_stride - (long long)(p.n_q + p.n_kv) * D : nullptr;
  auto load = [&](int h, uint2 &a, uint2 &b) {
    const uint16_t *src = h < p.n_q ? q_row : CACHE && h >= p.n_q + p.n_kv ? v_row : k_row;
    src += (long long)h * D;
    a = *reinterpret_cast<const uint2 *>(src + e0);
    b = *reinterpret_cast<const uint2 *>(src + e1);
  };
  // the first heads are on their way while the positions are looked up
  constexpr int PRE = 2;
  uint2 xa[PRE], xb[PRE];
#pragma unroll
  for (int i = 0; i < PRE; ++i)
    if (mine && h + i * step < heads) load(h + i * step, xa[i], xb[i]);

  if (CACHE) {
    // each row's sequence: the number of sequences that end at or before it
    int cnt[ROWS] = {};
    __syncthreads();
    for (int b = tid; b < p.n_seqs; b += kKvThreads) {
      const int end = __ldg(p.row_off + b + 1);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) cnt[r] += end <= r0 + r;
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int c = __reduce_add_sync(0xffffffffu, cnt[r]);
      if ((tid & 31) == 0 && c) atomicAdd(&s_seq[r], c);
    }
    __syncthreads();
    if (tid < nr) {
      const int row = r0 + tid, b = s_seq[tid];
      int pos = -1;
      long long at = -1;
      if (b < p.n_seqs) {
        const SeqView s = seq_view(p.row_off, p.kv_len, b, p.n_rows, p.max_pages, p.page);
        if (!s.ok || row >= s.row0 + s.rows || (row < s.row0 && b > 0)) {
          atomicOr(p.status, kErrBadBatch);
        } else if (row >= s.row0) {  // (rows in front of the first sequence are nobody's)
          pos = s.kv - s.rows + (row - s.row0);
          const int pg = __ldg(p.page_table + (long long)b * p.max_pages + pos / p.page);
          if ((unsigned)pg < (unsigned)p.n_pages)
            at = (long long)pg * p.n_kv * p.page + pos % p.page;
          else
            atomicOr(p.status, kErrBadPage);
        }
      }
      s_pos[tid] = pos;
      s_at[tid] = at;
    }
  } else {
    if (tid < nr) s_pos[tid] = p.pos ? __ldg(p.pos + r0 + tid) : 0;
  }
  __syncthreads();
  if (p.inv_freq) {
    for (int i = tid; i < nr * half; i += kKvThreads) {
      const int r = i / half, j = i - r * half;
      // the angle as a fraction of a turn, in [-1/2, 1/2]
      const double t = (double)s_pos[r] * __ldg(p.inv_freq + j) * 0.15915494309189533577;
      float s, c;
      sincospif(2.f * (float)(t - rint(t)), &s, &c);
      s_cs[r][j] = make_float2(c, s);
    }
    __syncthreads();
  }

  if (!mine) return;
  const int pos = s_pos[r];
  if (CACHE && pos < 0) return;  // a row of no sequence: left as it was
  const long long at = CACHE ? s_at[r] : 0;
  // The lane's four pairs' (cos, sin), laid out for the packed products: half
  // pairs (a0 a1) and (b0 b1) turn by (c0 c1) and (s0 s1), neighbours (a0 b0)
  // by (c0 c0) and (-s0 s0).
  uint64_t co[INTER ? 4 : 2], si[INTER ? 4 : 2];
  if (turns) {
    const float4 *cs = reinterpret_cast<const float4 *>(&s_cs[r][4 * sub]);
    const float4 c01 = cs[0], c23 = cs[1];
    if (INTER) {
      co[0] = f2_pack(c01.x, c01.x), co[1] = f2_pack(c01.z, c01.z);
      co[2] = f2_pack(c23.x, c23.x), co[3] = f2_pack(c23.z, c23.z);
      si[0] = f2_pack(-c01.y, c01.y), si[1] = f2_pack(-c01.w, c01.w);
      si[2] = f2_pack(-c23.y, c23.y), si[3] = f2_pack(-c23.w, c23.w);
    } else {
      co[0] = f2_pack(c01.x, c01.z), co[1] = f2_pack(c23.x, c23.z);
      si[0] = f2_pack(c01.y, c01.w), si[1] = f2_pack(c23.y, c23.w);
    }
  }
  uint16_t *qo_row = p.q_out + row * p.q_out_stride;
  uint16_t *ko_row = CACHE ? nullptr : p.k_out + row * p.k_out_stride - (long long)p.n_q * D;
  const uint32_t lanes = ((1u << LPH) - 1u) << (lane / LPH * LPH);  // the lanes of one head row
  auto finish = [&](int h, uint2 a, uint2 b) {
    const bool is_q = h < p.n_q, is_v = CACHE && h >= p.n_q + p.n_kv;
    uint64_t x[4] = {bf16x2_to_f2(a.x), bf16x2_to_f2(a.y), bf16x2_to_f2(b.x), bf16x2_to_f2(b.y)};
    if (!is_v) {
      if (p.norm) {
        const uint64_t sq = f2_fma(x[0], x[0], f2_fma(x[1], x[1], f2_fma(x[2], x[2], f2_mul(x[3], x[3]))));
        float ss, s1;
        f2_unpack(sq, ss, s1);
        ss += s1;
#pragma unroll
        for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(lanes, ss, o);
        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
        const uint64_t inv2 = f2_pack(inv, inv);
        const float *g = is_q ? p.q_gamma : p.k_gamma;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2_mul(x[i], inv2);
        if (g) {
          const ulonglong2 ga = __ldg(reinterpret_cast<const ulonglong2 *>(g + e0));
          const ulonglong2 gb = __ldg(reinterpret_cast<const ulonglong2 *>(g + e1));
          x[0] = f2_mul(x[0], ga.x), x[1] = f2_mul(x[1], ga.y);
          x[2] = f2_mul(x[2], gb.x), x[3] = f2_mul(x[3], gb.y);
        }
      }
      if (turns) {
        if (INTER) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float u, w;
            f2_unpack(x[i], u, w);
            x[i] = f2_fma(x[i], co[i], f2_mul(f2_pack(w, u), si[i]));
          }
        } else {
          const uint64_t minus = f2_pack(-1.f, -1.f);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint64_t u = x[i], w = x[2 + i];
            x[i] = f2_fma(u, co[i], f2_mul(f2_mul(w, minus), si[i]));
            x[2 + i] = f2_fma(w, co[i], f2_mul(u, si[i]));
          }
        }
      }
    }
    if (is_q || !CACHE) {
      uint16_t *dst = (is_q ? qo_row : ko_row) + (long long)h * D;
      *reinterpret_cast<uint2 *>(dst + e0) = make_uint2(f2_to_bf16x2(x[0]), f2_to_bf16x2(x[1]));
      *reinterpret_cast<uint2 *>(dst + e1) = make_uint2(f2_to_bf16x2(x[2]), f2_to_bf16x2(x[3]));
      return;
    }
    if (!CACHE || at < 0) return;
    const int kh = is_v ? h - p.n_q - p.n_kv : h - p.n_q;
    const long long to = (at + (long long)kh * p.page) * D;
    if (CACHE == 2) {
      const float *scale = is_v ? p.v_scale : p.k_scale;
      const float by = scale ? __ldg(scale + kh) : 1.f;
      uint8_t *dst = (is_v ? p.v_cache : p.k_cache) + to;
      *reinterpret_cast<uint32_t *>(dst + e0) = f2_to_e4m3x4(x[0], x[1], by);
      *reinterpret_cast<uint32_t *>(dst + e1) = f2_to_e4m3x4(x[2], x[3], by);
    } else {
      uint16_t *dst = reinterpret_cast<uint16_t *>(is_v ? p.v_cache : p.k_cache) + to;
      *reinterpret_cast<uint2 *>(dst + e0) = make_uint2(f2_to_bf16x2(x[0]), f2_to_bf16x2(x[1]));
      *reinterpret_cast<uint2 *>(dst + e1) = make_uint2(f2_to_bf16x2(x[2]), f2_to_bf16x2(x[3]));
    }
  };
  // the next heads' loads go out before the present ones are finished, PRE
  // heads a round (while the kernel took 19.0 us for 8192 rows of 16 + 4 heads
  // of 128, reloading each head's registers as it is finished took 22.3 us)
  for (; h < heads; h += PRE * step) {
    uint2 ya[PRE], yb[PRE];
#pragma unroll
    for (int i = 0; i < PRE; ++i) {
      ya[i] = xa[i];
      yb[i] = xb[i];
      const int next = h + (PRE + i) * step;
      if (next < heads) load(next, xa[i], xb[i]);
    }
#pragma unroll
    for (int i = 0; i < PRE; ++i)
      if (h + i * step < heads) finish(h + i * step, ya[i], yb[i]);
  }
}

}  // namespace moe
