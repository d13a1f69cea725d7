// attn.cuh -- attention of decode windows over the paged cache.
//
// Row i of a query head: o_i = sum_j p_ij v_j / sum_j p_ij with
// p_ij = exp(scale q_i.k_j - m_i) over the keys it sees (j <= i, and with a
// window W: i - j < W or j < S sinks), in one pass over the keys with the
// running maximum m and sum; m and the sums are fp32, base 2.
//
// The rows of one KV head's query heads are one block of up to 16 MT rows, so
// every key and value is read once per block.  The work of a call is the list
// of all (sequence, KV head, row block, 64-key tile) units in that order, cut
// into equal runs, one run per thread block (two resident per SM): ragged
// batches and single long sequences load the GPU alike.  A block that covers
// a (sequence, head, row block) only in part leaves its (m, sum, o) in the
// workspace, and the last of its blocks to arrive joins the parts in their
// order, so results do not depend on timing.
//
// Each block: one warp feeds a ring of key/value tiles by TMA (128-byte
// swizzle, one box per page), four warps compute on mma.sync fragments.  A
// window has at most a few dozen rows per KV head, too few for a 128-row
// tcgen05 tile, and the kernel is bound by reading the cache: 64 sequences of
// one token over 32768 keys, 16 heads over 2 of 128, 305 to 319 us from box to
// box, 6.7 to 7.0 TB/s (over e4m3, half the bytes, 248 us: 4.3 TB/s, a warp's
// chain of a tile and the conversions).  With less to read, other costs show:
// one such sequence with 4 KV heads 21 us (10 of reading, the rest start,
// hand-over and joining), 64 ragged windows of up to 5 rows over up to 4096
// keys 52 us (34 of reading; two row tiles, and a warp's chain of a tile is
// longer than its loading), 16 windows of 16 rows over 8000 keys 93 us (40 of
// reading; four row tiles, whose registers spill).
#pragma once

#include <cuda.h>

#include <type_traits>

#include "common.cuh"
#include "kvcache.cuh"

namespace moe {

constexpr int kAtTile = 64;      // keys of a tile
constexpr int kAtWarps = 4;      // computing warps
constexpr int kAtThreads = (kAtWarps + 1) * 32;
constexpr int kAtStages = 3;
constexpr int kAtMaxRows = 64;   // rows of a block (MT = 4)
constexpr float kAtSlack = 8.f;  // log2 of the growth that o is not rescaled for
// log2 of the largest term over an e4m3 cache, whose terms are fp16: with the
// slack they reach 2^15, and what fp16 cannot hold starts 2^-32 below the
// largest (2^-25 without: the 2^20 keys of a long flat tail lose up to 3 % of
// the sum that way).  o and its sum carry the same factor.
constexpr float kAtLift = 7.f;

template <int D, bool FP8>
struct AttnCfg {
  static constexpr int ROWB = D * (FP8 ? 1 : 2);          // bytes of a key
  static constexpr int NB = ROWB > 128 ? ROWB / 128 : 1;  // 128-byte column boxes
  static constexpr int LINE = ROWB / NB;                  // bytes of a box row (64 or 128)
  static constexpr int TILE = kAtTile * ROWB;             // one key or value tile
  static constexpr int JOIN = 2 * 16 * D * 4;             // two warps' fp32 rows
  static constexpr int SMEM = kAtStages * 2 * TILE + JOIN + 1024;  // and the AttnShared block
};
struct AttnShared {
  unsigned long long full[kAtStages], empty[kAtStages];
  long long scan[kAtWarps + 1];
  float ml[kAtWarps][2][8][2];  // (m, sum) of the rows handed over in a join
  int start[3];
  int dead, last;
};
static_assert(sizeof(AttnShared) <= 1024, "fits the block before the ring");

struct AttnParams {
  const uint16_t *q;
  uint16_t *out;
  long long q_stride, out_stride;
  const int *page_table, *row_off, *kv_len;
  const float *k_scale, *v_scale;
  float scale_log2;  // softmax scale times log2(e)
  int window, n_sink;
  int n_rows, n_q, n_kv, group;
  int n_pages, n_seqs, max_pages, page, page_shift;
  int min_units;     // smallest run of a block
  float *ws;         // [grid][2][16 MT][D + 2]
  unsigned int *arrived;  // [grid], zero between calls
  int *status;
};

// The tiles one sequence's rows see: [0, lead) and [first, first + n - lead).
struct SeqTiles {
  int lead, first, n;
};
MOE_HOST_DEV_INLINE SeqTiles seq_tiles(const SeqView &s, int window, int n_sink, int tile = kAtTile) {
  SeqTiles t{0, 0, 0};
  if (s.rows == 0) return t;
  const int end = (s.kv - 1) / tile + 1;
  if (window > 0) {
    const long long lo = (long long)s.kv - s.rows - window + 1;  // first key the first row's window holds
    if (lo > 0) {
      t.first = (int)(lo / tile);
      const long long sk = n_sink < lo ? n_sink : lo;
      const int lead = (int)((sk + tile - 1) / tile);
      t.lead = lead < t.first ? lead : t.first;
    }
  }
  t.n = t.lead + end - t.first;
  return t;
}
// Whether some row of the sequence sees one of the n keys from `key` on (the
// rows together see [0, min(n_sink, lo)) and [lo, kv), lo the first row's
// window).
MOE_HOST_DEV_INLINE bool keys_seen(const SeqView &s, int window, int n_sink, int key, int n) {
  if (key >= s.kv) return false;
  const long long lo = window > 0 ? (long long)s.kv - s.rows - window + 1 : 0;
  return (long long)key + n > lo || key < n_sink;
}
MOE_HOST_DEV_INLINE int tile_at(const SeqTiles &t, int k) { return k < t.lead ? k : k - t.lead + t.first; }
// The same list with the leading tiles at its end: a row's first maximum then
// comes from a full tile of its window, not from a few sinks.
MOE_HOST_DEV_INLINE int tile_at_lead_last(const SeqTiles &t, int k) {
  const int rest = t.n - t.lead;
  return k < rest ? t.first + k : k - rest;
}
// Units of a block's run: equal runs over the grid, none shorter than min_units.
MOE_HOST_DEV_INLINE long long run_length(long long total, long long grid, long long min_units) {
  const unsigned long long x = total + grid - 1;
  const long long run = x <= 0xffffffffull ? (unsigned)x / (unsigned)grid : x / grid;
  return run > min_units ? run : min_units;
}

MOE_DEV void ldsm_x4(uint32_t a, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(a));
}
MOE_DEV void ldsm_x4_t(uint32_t a, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(a));
}
template <bool F16>
MOE_DEV void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
MOE_DEV uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// two e4m3 values (the low 16 bits of v) as two fp16 values, exactly
MOE_DEV uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(v));
  return r;
}
MOE_DEV float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Bounded wait of one thread that also ends when the block gave up (`dead`).
// Each try may suspend the thread for up to 50 us (a poll without that hint
// returns at once and asks again, and a few such pollers hold up every other
// barrier operation of the SM), so the limit is about a second.
MOE_DEV bool mbar_wait_live(uint32_t bar, uint32_t parity, const int *dead) {
  for (uint32_t i = 0; i < 20000; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(50000)
        : "memory");
    if (ok) return true;
    if (dead && *reinterpret_cast<const volatile int *>(dead)) return false;
  }
  return false;
}
// The same for a warp off the tiles' chain: one lane polls.  (32 lanes polling
// one barrier are served one after another and hold up the SM's other
// barriers, which matters where a warp waits most of its time.)
// The shuffle hands the result on but orders no memory: the other lanes touch
// what the barrier guards only behind the __syncwarp.
MOE_DEV bool mbar_wait_warp(uint32_t bar, uint32_t parity, const int *dead) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait_live(bar, parity, dead);
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}
MOE_DEV void bar_sync_n(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
MOE_DEV void tma_box_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
      "%3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}

// Position in the list of units: sequence, (head, row block) within it, tile.
struct AttnCursor {
  int b, seg, k;   // sequence; head * row blocks + row block; tile of the list
  int nblk;        // row blocks of the sequence
  SeqView s;
  SeqTiles t;
};

template <int RB>
MOE_DEV void cursor_load(AttnCursor &c, const AttnParams &p) {
  for (; c.b < p.n_seqs; ++c.b) {
    c.s = seq_view(p.row_off, p.kv_len, c.b, p.n_rows, p.max_pages, p.page);
    c.t = seq_tiles(c.s, p.window, p.n_sink);
    c.nblk = (c.s.rows * p.group + RB - 1) / RB;
    if (c.t.n > 0) return;
  }
}
template <int RB>
MOE_DEV void cursor_next_seg(AttnCursor &c, const AttnParams &p) {
  c.k = 0;
  if (++c.seg == p.n_kv * c.nblk) {
    c.seg = 0;
    ++c.b;
    cursor_load<RB>(c, p);
  }
}

template <int D, bool FP8, int MT>
__global__ void __launch_bounds__(kAtThreads, 2)
    attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const AttnParams p) {
  using C = AttnCfg<D, FP8>;
  constexpr int RB = 16 * MT;
  constexpr int KG = kAtWarps / MT;      // key groups: warps that share a tile's keys
  constexpr int KEYS = kAtTile / KG;     // keys of a warp
  constexpr int NT = KEYS / 8;           // 8-key score tiles
  constexpr int ND = D / 8;              // 8-column output tiles
  constexpr int S = kAtStages;
  // no static shared memory: two blocks fill the SM, and the ring's tiles
  // need the 1024-byte alignment of the array itself
  extern __shared__ __align__(1024) unsigned char at_smem[];
  AttnShared &sh = *reinterpret_cast<AttnShared *>(at_smem);
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const uint32_t stage0 = smem_addr(at_smem) + 1024;
  const uint32_t join = stage0 + S * 2 * C::TILE;
  if (tid == kAtWarps * 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_addr(&sh.full[i]), 1);
      mbar_init(smem_addr(&sh.empty[i]), kAtWarps);
    }
    sh.dead = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();

  // ---- the list of units: its length, and where this block's run begins
  auto units_of = [&](const SeqView &s, const SeqTiles &t) {
    return (((long long)s.rows * p.group + RB - 1) / RB) * p.n_kv * t.n;
  };
  auto view = [&](int b) {
    const SeqView s = seq_view(p.row_off, p.kv_len, b, p.n_rows, p.max_pages, p.page);
    if (!s.ok && blockIdx.x == 0) atomicOr(p.status, kErrBadBatch);
    return s;
  };
  AttnCursor c;
  long long total, run, u0, u1;
  bool own = false;  // each block belongs to one segment: its blocks are
  int own_first = 0, own_last = 0;
  auto cut = [&] {
    run = run_length(total, gridDim.x, p.min_units);
    u0 = run * blockIdx.x;
    u1 = min(u0 + run, total);
  };
  auto place = [&](unsigned long long x, int nt, int &seg, int &k) {  // unit x of a sequence
    const long long q = x <= 0xffffffffull ? (unsigned)x / (unsigned)nt : x / nt;
    seg = (int)q;
    k = (int)(x - q * nt);
  };
  if (p.n_seqs <= 32) {
    // Few sequences: every warp finds the place for itself, a lane per
    // sequence, and what few long segments need is looked for below.  Without
    // all that, by the plain cut of the other branch: one token over 32768 keys
    // 24.2 us against 21.5, 8 sequences over up to 8192 23.4 against 20.2, 32
    // over up to 4096 33.3 against 32.0 (32 over 32768 keys 160 against 162).
    // More sequences than lanes gain less and less, and take the plain cut.
    SeqView s{0, 0, 0, true};
    SeqTiles t{0, 0, 0};
    if (lane < p.n_seqs) {
      s = view(lane);
      t = seq_tiles(s, p.window, p.n_sink);
    }
    const long long units = units_of(s, t);
    total = units;
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    // A part of R rows costs the block that joins it about 0.05 + R / 230 of a
    // tile's time, so the longest segment's n tiles are cut into runs of at
    // least sqrt(n (0.05 + R / 256)): both halves of the chain then take about
    // the same (one window of 8 rows over 32768 keys, 64 rows of a KV head:
    // 72 us, against 99.5 us with 128 parts a head).
    const int n_max = __reduce_max_sync(0xffffffffu, t.n);
    const int r_max = __reduce_max_sync(0xffffffffu, min(s.rows * p.group, RB));
    run = run_length(total, gridDim.x,
                     max(p.min_units, __float2int_ru(sqrtf(n_max * (0.05f + r_max * (1.f / 256.f))))));
    // Where a slightly longer run lets every segment have blocks of its own,
    // no block has two parts to hand over.
    const int segs = t.n ? (int)(units / t.n) : 0;
    int need = 0;
    if (total <= 0x7fffffff) {
      const int most = (int)run + ((int)run + 3) / 4;
      for (int r = (int)run; r <= most && !own; ++r) {
        need = __reduce_add_sync(0xffffffffu, segs * ((t.n + r - 1) / r));
        if (need <= (int)gridDim.x) own = true, run = r;
      }
    }
    const long long mine = own ? segs * ((t.n + (int)run - 1) / (int)run) : units;  // blocks, or units
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    u0 = own ? blockIdx.x : run * blockIdx.x;
    if (u0 >= (own ? need : total)) return;  // block-uniform: no work for this block
    const int f = __ffs(__ballot_sync(0xffffffffu, u0 < inc)) - 1;
    const long long x = u0 - __shfl_sync(0xffffffffu, inc - mine, f);  // within sequence f
    c.b = f;
    c.s.row0 = __shfl_sync(0xffffffffu, s.row0, f);
    c.s.rows = __shfl_sync(0xffffffffu, s.rows, f);
    c.s.kv = __shfl_sync(0xffffffffu, s.kv, f);
    c.s.ok = true;
    c.t.lead = __shfl_sync(0xffffffffu, t.lead, f);
    c.t.first = __shfl_sync(0xffffffffu, t.first, f);
    c.t.n = __shfl_sync(0xffffffffu, t.n, f);
    c.nblk = (c.s.rows * p.group + RB - 1) / RB;
    if (own) {
      const int parts = (c.t.n + (int)run - 1) / (int)run;
      int part;
      place(x, parts, c.seg, part);
      own_first = blockIdx.x - part;
      own_last = own_first + parts - 1;
      c.k = part * (int)run;
      u0 = 0;
      u1 = min((int)run, c.t.n - c.k);
    } else {
      place(x, c.t.n, c.seg, c.k);
      u1 = min(u0 + run, total);
    }
  } else {
    // every thread holds a slice of the sequences; the thread whose slice
    // holds the place tells the others
    const int per = (p.n_seqs + kAtThreads - 1) / kAtThreads;
    const int b_lo = min(tid * per, p.n_seqs), b_hi = min(b_lo + per, p.n_seqs);
    auto seq_units = [&](int b, int &nt) {
      const SeqView s = view(b);
      const SeqTiles t = seq_tiles(s, p.window, p.n_sink);
      nt = t.n;
      return units_of(s, t);
    };
    int nt_lo = 0;  // tiles and units of the thread's first sequence
    long long units_lo = 0;
    if (b_lo < b_hi) units_lo = seq_units(b_lo, nt_lo);
    long long mine = units_lo;
    for (int b = b_lo + 1; b < b_hi; ++b) {
      int nt;
      mine += seq_units(b, nt);
    }
    // inclusive scan over the block: within the warps, then over their totals
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) sh.scan[wid] = inc;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kAtWarps + 1; ++w) {
      if (w < wid) before += sh.scan[w];
      total += sh.scan[w];
    }
    inc += before;
    cut();
    if (u0 >= u1) return;  // block-uniform: no work for this block
    if (u0 >= inc - mine && u0 < inc) {
      long long at = inc - mine, n = units_lo;
      int b = b_lo, nt = nt_lo;
      while (u0 >= at + n) {
        at += n;
        n = seq_units(++b, nt);
      }
      sh.start[0] = b;
      place(u0 - at, nt, sh.start[1], sh.start[2]);
    }
    __syncthreads();
    c.b = sh.start[0];
    cursor_load<RB>(c, p);
    c.seg = sh.start[1];
    c.k = sh.start[2];
  }
  auto dead = [&]() { return *reinterpret_cast<volatile int *>(&sh.dead) != 0; };
  auto give_up = [&]() {
    *reinterpret_cast<volatile int *>(&sh.dead) = 1;
    atomicOr(p.status, kErrTimeout);
  };

  if (wid == kAtWarps) {
    // ---------------------------------------------------------- producer
    const int pr = min(p.page, kAtTile);       // rows of a box
    const int ppt = kAtTile / pr;              // boxes along a tile's keys
    const int boxes = ppt * C::NB * 2;         // at most 4 * 2 * 2
    const uint64_t policy = l2_evict_first();
    const int my_page = lane / (C::NB * 2);    // the box of this lane: page of the tile,
    const int my_col = lane / 2 % C::NB;       // column box, keys or values
    const bool my_v = lane & 1;
    int held_b = -1, held_at = 0, held = 0;    // 32 entries of the page table, one per lane
    int st = 0;
    uint32_t phase = 1;   // a new barrier passes the wait for its preceding phase
    long long u = u0;
    for (; u < u1 && !dead(); ++u) {
      const int tile = tile_at(c.t, c.k);
      const int key0 = tile * kAtTile;
      const int blk_h = c.seg / c.nblk;
      const int pg0 = key0 >> p.page_shift;
      const int n_pg = (c.s.kv + p.page - 1) >> p.page_shift;  // pages that hold keys
      if (held_b != c.b || pg0 < held_at || pg0 + ppt > held_at + 32) {
        held_b = c.b;
        held_at = pg0;
        const int i = pg0 + lane;
        held = i < n_pg ? __ldg(p.page_table + (long long)c.b * p.max_pages + i) : 0;
      }
      const uint32_t bar = smem_addr(&sh.full[st]);
      if (!mbar_wait_warp(smem_addr(&sh.empty[st]), phase, &sh.dead)) {
        if (lane == 0) give_up();
        break;
      }
      // a box is loaded when its page holds a key that some row sees; the
      // entries of other pages (given back, or never there) are not looked at
      int page = __shfl_sync(0xffffffffu, held, min(pg0 - held_at + my_page, 31));
      const int first_key = key0 + my_page * pr;
      const bool need = lane < boxes && keys_seen(c.s, p.window, p.n_sink, first_key, pr);
      if (need && (unsigned)page >= (unsigned)p.n_pages) {
        atomicOr(p.status, kErrBadPage);
        page = 0;  // an in-bounds page; the call's result is reported as bad
      }
      const int n_box = __popc(__ballot_sync(0xffffffffu, need));
      if (lane == 0) mbar_expect_tx(bar, (uint32_t)n_box * pr * C::LINE);
      __syncwarp();
      if (need) {
        const uint32_t dst = stage0 + (uint32_t)(st * 2 + my_v) * C::TILE +
                             (uint32_t)my_col * (kAtTile * C::LINE) + (uint32_t)my_page * pr * C::LINE;
        const int y = (page * p.n_kv + blk_h) * p.page + (key0 & (p.page - 1));
        tma_box_2d(dst, my_v ? &vmap : &kmap, my_col * (FP8 ? 128 : 64), y, bar, policy);
      }
      if (++c.k == c.t.n) cursor_next_seg<RB>(c, p);
      if (++st == S) st = 0, phase ^= 1;
    }
    // no tile may land after the block has gone: each stage's last use
    const long long issued = u - u0;
    for (int i = 0; i < S && i < issued; ++i) {
      const uint32_t uses = (uint32_t)((issued - 1 - i) / S);
      (void)mbar_wait_bounded(smem_addr(&sh.full[i]), uses & 1);
    }
    return;
  }

  // ------------------------------------------------------------ computing
  const int mt = wid % MT, kg = wid / MT;
  const int g = lane >> 2, cq = lane & 3;
  // where this lane reads in a tile.  Keys: row 8 n + lane % 8, 16-byte column
  // 4 i + lane / 8 of a line; values: row 16 ks + lane % 16, column 2 i + lane /
  // 16; the swizzle turns a column's number by the row's (mod 8, or mod 4 of
  // row / 2 in 64-byte lines).
  constexpr int KOFF = C::LINE / 64, VOFF = C::LINE / 32;
  uint32_t koff[KOFF], voff[VOFF];
#pragma unroll
  for (int i = 0; i < KOFF; ++i) {
    const int key = kg * KEYS + (lane & 7), x = C::LINE == 128 ? key & 7 : (key >> 1) & 3;
    koff[i] = key * C::LINE + (((4 * i + (lane >> 3)) ^ x) << 4);
  }
#pragma unroll
  for (int i = 0; i < VOFF; ++i) {
    const int key = kg * KEYS + (lane & 15), x = C::LINE == 128 ? key & 7 : (key >> 1) & 3;
    voff[i] = key * C::LINE + (((2 * i + (lane >> 4)) ^ x) << 4);
  }
  int st = 0;            // the ring's stage and the parity of its present use
  uint32_t phase = 0;
  long long u = u0;
  bool live = true;  // false once a wait of this warp gave up: it goes on through the shared barriers
  while (u < u1) {
    // this block's share of one (sequence, head, row block)
    const int kv_h = c.seg / c.nblk, blk = c.seg % c.nblk;
    const int k_beg = c.k;
    const int k_end = (int)min((long long)c.t.n, k_beg + (u1 - u));
    const int r_all = c.s.rows * p.group;
    const int pos0 = c.s.kv - c.s.rows;
    // the thread's two rows of the block, and their places
    int row_t[2];
    bool row_ok[2];
    const uint16_t *row_q[2];
    long long row_o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = blk * RB + mt * 16 + g + 8 * i;
      row_ok[i] = r < r_all;
      row_t[i] = row_ok[i] ? r / p.group : 0;
      const int head = kv_h * p.group + (row_ok[i] ? r % p.group : 0);
      row_q[i] = p.q + (long long)(c.s.row0 + row_t[i]) * p.q_stride + (long long)head * D;
      row_o[i] = (long long)(c.s.row0 + row_t[i]) * p.out_stride + (long long)head * D;
    }
    // Q fragments.  An e4m3 cache computes in fp16: its values are exact
    // there, and each query row is divided by a power of two near its
    // largest element: exact for what bf16 holds above 2^-14 of that, and
    // rounded by at most 2^-25 of it below.
    uint32_t qf[D / 16][4];
    float row_scale[2] = {p.scale_log2, p.scale_log2};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int m = 0; m < D / 16; ++m) {
        if (FP8) {
          uint2 v = make_uint2(0, 0);
          if (row_ok[i]) v = *reinterpret_cast<const uint2 *>(row_q[i] + 16 * m + 4 * cq);
          qf[m][i] = v.x;
          qf[m][2 + i] = v.y;
        } else {
          uint32_t a = 0, b = 0;
          if (row_ok[i]) {
            a = *reinterpret_cast<const uint32_t *>(row_q[i] + 16 * m + 2 * cq);
            b = *reinterpret_cast<const uint32_t *>(row_q[i] + 16 * m + 8 + 2 * cq);
          }
          qf[m][i] = a;
          qf[m][2 + i] = b;
        }
      }
    }
    if (FP8) {
      const float ks = p.k_scale ? __ldg(p.k_scale + kv_h) : 1.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
        for (int m = 0; m < D / 16; ++m) {
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const uint32_t v = qf[m][j + i];
            top = max(top, max((v << 16) & 0x7FFFFFFFu, v & 0x7FFF0000u));
          }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e of the largest element (at least 2^-63: a row of zeros keeps a
        // scale above zero), kept where 2^-e is a normal number
        const uint32_t e = min(max(top >> 23, 64u), 253u);
        const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23);
        row_scale[i] *= ks * up;
#pragma unroll
        for (int m = 0; m < D / 16; ++m) {
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const uint32_t v = qf[m][j + i];
            qf[m][j + i] =
                pack_f16(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xFFFF0000u) * down);
          }
        }
      }
    }
    float o[ND][4];
#pragma unroll
    for (int n = 0; n < ND; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};

    for (int k = k_beg; k < k_end; ++k) {
      // All lanes wait here, and in the rows' wait of the chunk kernel: with one
      // that polls for the others, every tile waits for the shuffle too (one
      // token over 32768 keys 21.7 against 21.2 us, 64 tokens 320 against 312,
      // 8192 rows over 16384 keys 775 against 725 us).
      live = live && mbar_wait_live(smem_addr(&sh.full[st]), phase, &sh.dead);
      live = __all_sync(0xffffffffu, live);
      if (live) {
        const int tile = tile_at(c.t, k);
        const int key0 = tile * kAtTile + kg * KEYS;  // first key of this warp
        const uint32_t kt = stage0 + (uint32_t)(st * 2) * C::TILE, vt = kt + C::TILE;
        // ---- scores
        float sc[NT][4];
        uint32_t kb[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
        // (the keys' tiles inside, so that NT products are in flight)
#pragma unroll
        for (int ch = 0; ch < C::ROWB / 16; ch += 4) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            // four 8-key x 16-byte matrices of consecutive 16-byte columns
            const uint32_t addr = kt + koff[ch % (4 * KOFF) / 4] + ch / (4 * KOFF) * (kAtTile * C::LINE) +
                                  n * 8 * C::LINE;
            uint32_t (&b)[4] = kb[n];
            ldsm_x4(addr, b[0], b[1], b[2], b[3]);
          }
#pragma unroll
          for (int m = 0; m < (FP8 ? 4 : 2); ++m) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (FP8)  // each matrix: 16 columns, this lane's four neighbours = one step
                mma_16816<true>(sc[n], qf[ch + m], e4m3x2_to_f16x2(kb[n][m]), e4m3x2_to_f16x2(kb[n][m] >> 16));
              else
                mma_16816<false>(sc[n], qf[ch / 2 + m], kb[n][2 * m], kb[n][2 * m + 1]);
            }
          }
        }
        // ---- masks: only tiles that some row sees in part
        const int tile0 = tile * kAtTile, last = tile0 + kAtTile - 1;
        const int pos1 = c.s.kv - 1;
        const bool whole = last <= pos0 && (p.window <= 0 || pos1 - tile0 < p.window || last < p.n_sink);
        if (!whole) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = key0 + n * 8 + 2 * cq + (e & 1), i = pos0 + row_t[e >> 1];
              const bool seen = j <= i && (p.window <= 0 || i - j < p.window || j < p.n_sink);
              if (!seen) sc[n][e] = -INFINITY;
            }
        }
        // ---- running maximum and sum.  The terms are scaled by a reference
        // that follows the maximum only when it fell kAtSlack behind (p then
        // holds values up to 2^kAtSlack, over e4m3 2^(kAtSlack + kAtLift)):
        // o is rarely rescaled
        float corr[2] = {1.f, 1.f}, neg[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = -INFINITY;
#pragma unroll
          for (int n = 0; n < NT; ++n) mx = fmaxf(mx, fmaxf(sc[n][2 * i], sc[n][2 * i + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * row_scale[i];
          if (m_run[i] == -INFINITY) {
            m_run[i] = mx;
          } else if (mx > m_run[i] + kAtSlack) {
            corr[i] = ex2(m_run[i] - mx);
            m_run[i] = mx;
          }
          // nothing seen yet: every p below is 2^-inf = 0
          neg[i] = m_run[i] == -INFINITY ? 0.f : (FP8 ? kAtLift : 0.f) - m_run[i];
        }
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[n][e] = ex2(__fmaf_rn(sc[n][e], row_scale[e >> 1], neg[e >> 1]));
            sum[e >> 1] += sc[n][e];
          }
        l_run[0] = l_run[0] * corr[0] + sum[0];
        l_run[1] = l_run[1] * corr[1] + sum[1];
        if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
          for (int n = 0; n < ND; ++n) {
            o[n][0] *= corr[0];
            o[n][1] *= corr[0];
            o[n][2] *= corr[1];
            o[n][3] *= corr[1];
          }
        }
        // ---- o += p v.  p is rounded to the tensor cores' 16 bits (at most
        // half a step of each term); values no row of the call sees may hold
        // anything, infinities and NaN included, and are read as zeros.
        auto values = [&](auto edge_tile) {
          constexpr bool EDGE = decltype(edge_tile)::value;
          const int seen_end = c.s.kv;                           // keys from here on do not exist
          const int hid0 = p.window > 0 ? p.n_sink : 0x7fffffff; // [hid0, hid1) lies before every window
          const long long hid1 = (long long)pos0 - p.window + 1;
#pragma unroll
          for (int ks = 0; ks < KEYS / 16; ++ks) {
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float lo = sc[2 * ks + (i >> 1)][(i & 1) * 2], hi = sc[2 * ks + (i >> 1)][(i & 1) * 2 + 1];
              a[i] = FP8 ? pack_f16(lo, hi) : pack_bf16(lo, hi);
            }
            // the keys of this lane's fragment registers: j, j+1 and j+8, j+9
            uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
            if (EDGE) {
              keep0 = keep1 = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int j = key0 + ks * 16 + 2 * cq + (e & 1) + 8 * (e >> 1);
                const bool keep = j < seen_end && !(j >= hid0 && j < hid1);
                const uint32_t bits = keep ? ((e & 1) ? 0xffff0000u : 0x0000ffffu) : 0u;
                if (e < 2) keep0 |= bits;
                else keep1 |= bits;
              }
            }
            auto k0 = [&](uint32_t v) { return EDGE ? v & keep0 : v; };
            auto k1 = [&](uint32_t v) { return EDGE ? v & keep1 : v; };
#pragma unroll
            for (int ch = 0; ch < C::ROWB / 16; ch += 2) {
              const uint32_t addr = vt + voff[ch % (2 * VOFF) / 2] + ch / (2 * VOFF) * (kAtTile * C::LINE) +
                                    ks * 16 * C::LINE;
              uint32_t b0, b1, b2, b3;
              ldsm_x4_t(addr, b0, b1, b2, b3);
              if (FP8) {
                // bytes of a register: key j: columns 2g, 2g+1; key j+1: the same
                const uint32_t x0 = __byte_perm(b0, 0, 0x3120), x1 = __byte_perm(b1, 0, 0x3120);
                const uint32_t x2 = __byte_perm(b2, 0, 0x3120), x3 = __byte_perm(b3, 0, 0x3120);
                mma_16816<true>(o[2 * ch], a, k0(e4m3x2_to_f16x2(x0)), k1(e4m3x2_to_f16x2(x1)));
                mma_16816<true>(o[2 * ch + 1], a, k0(e4m3x2_to_f16x2(x0 >> 16)), k1(e4m3x2_to_f16x2(x1 >> 16)));
                mma_16816<true>(o[2 * ch + 2], a, k0(e4m3x2_to_f16x2(x2)), k1(e4m3x2_to_f16x2(x3)));
                mma_16816<true>(o[2 * ch + 3], a, k0(e4m3x2_to_f16x2(x2 >> 16)), k1(e4m3x2_to_f16x2(x3 >> 16)));
              } else {
                mma_16816<false>(o[ch], a, k0(b0), k1(b1));
                mma_16816<false>(o[ch + 1], a, k0(b2), k1(b3));
              }
            }
          }
        };
        if (whole) values(std::false_type{});
        else values(std::true_type{});
      } else if (lane == 0 && !dead()) {
        give_up();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.empty[st]));
      if (++st == S) st = 0, phase ^= 1;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // the four lanes of a row hold parts of its sum
      l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 1);
      l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 2);
    }
    // ---- join the key groups of the block: halves of them, until one is left
#pragma unroll
    for (int h = KG / 2; h >= 1; h >>= 1) {
      // warps with kg in [h, 2h) hand theirs to kg - h; two warps' rows fit
      const uint32_t slot = join + (uint32_t)(((kg % h) * MT + mt) * 16 * D * 4);
      const int peer = (kg % h) * MT + mt;
      if (kg >= h && kg < 2 * h) {
#pragma unroll
        for (int n = 0; n < ND; ++n)
          asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(slot + (uint32_t)(n * 32 + lane) * 16),
                       "f"(o[n][0]), "f"(o[n][1]), "f"(o[n][2]), "f"(o[n][3])
                       : "memory");
        if (cq == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            sh.ml[peer][i][g][0] = m_run[i];
            sh.ml[peer][i][g][1] = l_run[i];
          }
        }
      }
      bar_sync_n(1, kAtWarps * 32);
      if (kg < h) {
        float wa[2], wb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mb = sh.ml[peer][i][g][0], lb = sh.ml[peer][i][g][1];
          const float mx = fmaxf(m_run[i], mb), mu = mx == -INFINITY ? 0.f : mx;
          wa[i] = ex2(m_run[i] - mu);
          wb[i] = ex2(mb - mu);
          l_run[i] = l_run[i] * wa[i] + lb * wb[i];
          m_run[i] = mx;
        }
#pragma unroll
        for (int n = 0; n < ND; ++n) {
          float v[4];
          asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                       : "r"(slot + (uint32_t)(n * 32 + lane) * 16));
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] = o[n][e] * wa[e >> 1] + v[e] * wb[e >> 1];
        }
      }
      bar_sync_n(1, kAtWarps * 32);
    }
    // ---- write the rows, or this block's part of them.  Column of o[n][e]:
    // e4m3 tiles come in pairs of even and odd columns of 16.
    auto col_of = [&](int n, int e) {
      return FP8 ? (n >> 1) * 16 + 4 * cq + 2 * (e & 1) + (n & 1) : n * 8 + 2 * cq + (e & 1);
    };
    const float vs = FP8 && p.v_scale ? __ldg(p.v_scale + kv_h) : 1.f;
    const bool all = k_beg == 0 && k_end == c.t.n;
    if (all) {
      if (kg == 0 && !dead()) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!row_ok[i]) continue;
          const float inv = vs / l_run[i];
          uint16_t *dst = p.out + row_o[i];
          if (FP8) {
#pragma unroll
            for (int n = 0; n < ND; n += 2) {
              const uint2 v = make_uint2(pack_bf16(o[n][2 * i] * inv, o[n + 1][2 * i] * inv),
                                         pack_bf16(o[n][2 * i + 1] * inv, o[n + 1][2 * i + 1] * inv));
              *reinterpret_cast<uint2 *>(dst + col_of(n, 0)) = v;
            }
          } else {
#pragma unroll
            for (int n = 0; n < ND; ++n)
              *reinterpret_cast<uint32_t *>(dst + col_of(n, 0)) =
                  pack_bf16(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
          }
        }
      }
    } else {
      // the segment's first block wrote slot 1 (its run ends inside it), the
      // others slot 0 (their run begins inside it)
      const long long seg_u0 = u - k_beg, seg_u1 = seg_u0 + c.t.n;
      const int first = own ? own_first : (int)(seg_u0 / run);
      const int lastb = own ? own_last : (int)((seg_u1 - 1) / run);
      auto slot_of = [&](int blk_id) {
        return p.ws + ((long long)blk_id * 2 + (blk_id == first ? 1 : 0)) * (RB * (D + 2));
      };
      if (kg == 0) {
        float *w = slot_of(blockIdx.x);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = mt * 16 + g + 8 * i;
          if (!row_ok[i]) continue;
          float *row = w + r * D;
          if (FP8) {
#pragma unroll
            for (int n = 0; n < ND; n += 2)
              *reinterpret_cast<float4 *>(row + col_of(n, 0)) =
                  make_float4(o[n][2 * i], o[n + 1][2 * i], o[n][2 * i + 1], o[n + 1][2 * i + 1]);
          } else {
#pragma unroll
            for (int n = 0; n < ND; ++n)
              *reinterpret_cast<float2 *>(row + col_of(n, 0)) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
          }
          if (cq == 0) {
            w[RB * D + r] = m_run[i];
            w[RB * D + RB + r] = l_run[i];
          }
        }
      }
      bar_sync_n(1, kAtWarps * 32);
      if (tid == 0) {
        const unsigned int parts = lastb - first + 1;
        __threadfence();  // the block's part before its arrival, and every part before the join
        sh.last = atomicAdd(p.arrived + first, 1u) == parts - 1;
        if (sh.last) {
          p.arrived[first] = 0;
          __threadfence();
        }
      }
      bar_sync_n(1, kAtWarps * 32);
      if (sh.last) {
        const int rows_here = min(RB, r_all - blk * RB), parts = lastb - first + 1;
        auto store = [&](int r, int d4, const float (&acc)[4], float inv) {
          const int rr = blk * RB + r, t = rr / p.group, head = kv_h * p.group + rr % p.group;
          uint16_t *dst = p.out + (long long)(c.s.row0 + t) * p.out_stride + (long long)head * D + d4;
          *reinterpret_cast<uint2 *>(dst) =
              make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
        };
        // few parts: U of them for I groups of four columns in flight
        auto join_few = [&](auto u_, auto i_) {
          constexpr int U = decltype(u_)::value, I = decltype(i_)::value, STEP = kAtWarps * 32;
          for (int it0 = tid; it0 < rows_here * (D / 4); it0 += STEP * I) {
            float f[I][U], li[I][U];
            float4 v[I][U];
#pragma unroll
            for (int i = 0; i < I; ++i) {
              const int it = min(it0 + i * STEP, rows_here * (D / 4) - 1), r = it / (D / 4), d4 = it % (D / 4) * 4;
#pragma unroll
              for (int k = 0; k < U; ++k) {
                const float *w = slot_of(first + min(k, parts - 1));
                f[i][k] = __ldcg(w + RB * D + r);
                li[i][k] = __ldcg(w + RB * D + RB + r);
                v[i][k] = ldcg_f4(w + r * D + d4);
              }
            }
#pragma unroll
            for (int i = 0; i < I; ++i) {
              const int it = it0 + i * STEP;
              if (it >= rows_here * (D / 4)) break;
              float mx = f[i][0];
#pragma unroll
              for (int k = 1; k < U; ++k) mx = fmaxf(mx, f[i][k]);
              const float mu = mx == -INFINITY ? 0.f : mx;
              float acc[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
#pragma unroll
              for (int k = 0; k < U; ++k) {
                const float e = k < parts ? ex2(f[i][k] - mu) : 0.f;
                l += e * li[i][k];
                acc[0] += e * v[i][k].x;
                acc[1] += e * v[i][k].y;
                acc[2] += e * v[i][k].z;
                acc[3] += e * v[i][k].w;
              }
              store(it / (D / 4), it % (D / 4) * 4, acc, vs / l);
            }
          }
        };
        // (with one row tile there are few groups, and registers to lose: one
        // token over 32768 keys 21.1 us without the first two, 22.1 us with them)
        if (MT > 1 && parts == 2) {
          join_few(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
        } else if (MT > 1 && parts <= 4) {
          join_few(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
        } else if (parts <= 8) {
          join_few(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
        } else {
          // Each part's weight first, a warp per row (as many rows at once as
          // the join buffer holds weights for), then the weighted sums.
          float *wgt = reinterpret_cast<float *>(at_smem + 1024 + S * 2 * C::TILE);
          float *inv = &sh.ml[0][0][0][0];  // of up to 64 rows
          const int at_once = min(rows_here, (int)(C::JOIN / sizeof(float)) / parts);
          for (int r0 = 0; r0 < rows_here; r0 += at_once) {
            const int nr = min(at_once, rows_here - r0);
            for (int r = wid; r < nr; r += kAtWarps) {
              float mx = -INFINITY, l = 0.f;
#pragma unroll 4
              for (int i = lane; i < parts; i += 32) {
                const float m = __ldcg(slot_of(first + i) + RB * D + r0 + r);
                wgt[r * parts + i] = m;
                mx = fmaxf(mx, m);
              }
#pragma unroll
              for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
              const float mu = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
              for (int i = lane; i < parts; i += 32) {
                const float e = ex2(wgt[r * parts + i] - mu);
                wgt[r * parts + i] = e;
                l += e * __ldcg(slot_of(first + i) + RB * D + RB + r0 + r);
              }
              l = warp_sum(l);
              if (lane == 0) inv[r] = vs / l;
            }
            bar_sync_n(1, kAtWarps * 32);
            for (int it = tid; it < nr * (D / 4); it += kAtWarps * 32) {
              const int r = it / (D / 4), d4 = it % (D / 4) * 4;
              const long long at = (long long)(r0 + r) * D + d4;
              float acc[4] = {0.f, 0.f, 0.f, 0.f};
              constexpr int W = 16;
              for (int i0 = 0; i0 < parts; i0 += W) {
                float4 v[W];
#pragma unroll
                for (int k = 0; k < W; ++k) v[k] = ldcg_f4(slot_of(first + min(i0 + k, parts - 1)) + at);
#pragma unroll
                for (int k = 0; k < W; ++k) {
                  const float e = i0 + k < parts ? wgt[r * parts + i0 + k] : 0.f;
                  acc[0] += e * v[k].x;
                  acc[1] += e * v[k].y;
                  acc[2] += e * v[k].z;
                  acc[3] += e * v[k].w;
                }
              }
              store(r0 + r, d4, acc, inv[r]);
            }
            bar_sync_n(1, kAtWarps * 32);  // the weights have been read
          }
        }
      }
      bar_sync_n(1, kAtWarps * 32);  // sh.last is read before the next segment writes it
    }
    u += k_end - k_beg;
    c.k = k_end;
    if (c.k == c.t.n) cursor_next_seg<RB>(c, p);
  }
}

}  // namespace moe
