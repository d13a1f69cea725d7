// attn_prefill.cuh -- attention of prompt chunks over the paged cache on the
// tensor cores (tcgen05).
//
// The mathematics is attn.cuh's.  A chunk has enough rows per KV head to fill
// 128-row tiles, so here the two products are the work: 4 D flops a visible
// (row, key) pair against one exponential.
//
// A block takes 256 rows: two 128-row tiles, each the rows of `pack` query
// heads of one KV head (the largest power of two dividing the group) at 128 /
// pack consecutive tokens, so few tokens of a tile lie above the diagonal.
// Warps:
//   8      TMA: the query tiles and the first keys, then pairs of a value tile
//          and the next key tile (128 keys each) through a ring (one box per
//          page and 64 columns);
//   9, 10  issue the MMAs of tile 0 and 1: S = Q K^T into tensor memory, O +=
//          P V with P read from tensor memory and V as it lies in the cache
//          ([key][column]: an MN-major operand).  Issuing is paced by the
//          tensor cores (64 cycles an MMA), so each tile has an issuer: one's
//          waits and commits are covered by the other's products.  They take
//          turns, a step's P V and next S at a time; served together the two
//          tiles fall into step and wait for the tensor cores and for the
//          exponentials at the same times (6,200 against 3,800 cycles for 128
//          keys of both);
//   0-3, 4-7  one thread per row of tile 0 and 1: reads its row of S, masks,
//          keeps the running maximum and sum, and writes P (bf16) over S, in
//          two halves so that the first half's product starts early.
// While the tensor cores work for one tile, the other's rows go through the
// exponentials.  O stays in tensor memory; it is rescaled only when a row's
// maximum grew by more than 2^8 over the reference its terms were scaled by
// (P then holds values up to 2^8, rounded to bf16 like any other; sums are
// fp32).
//
// What bounds it: the chain of one tile's step, about 3,800 cycles for 128
// keys -- S read 390, maximum 330, exponentials 1,530 (a warp per scheduler
// reaches two thirds of the special function unit's rate), hand-over 230, P V
// and S 990, commit 360 -- of which the tensor cores work 2,048 for the two
// tiles.  8192 rows of 16 heads over 16384 keys: 782 us, 1.05 PFLOP/s, the
// blocks of the last incomplete wave splitting their keys (812 us without); 680
// to 793 us from box to box.  Over e4m3 875 us: four more warps convert every
// tile, and the rows' threads spill (72 bytes at the launch's 128 registers).
// Measured at earlier stages and not kept: two warps per row (927 against 900
// us), scores double-buffered in steps of 64 keys (876 against 845 us: an MMA
// of 64 columns takes as long as one of 128), exponentials on the FMA units by
// a polynomial (a quarter of them: 872 against 853 us, half: 913).
//
// Tensor memory: S0, S1 (128 columns each, P over the first 64), O0, O1.
#pragma once

#include "attn.cuh"
#include "prefill.cuh"

namespace moe {

constexpr int kApTile = 128;   // keys of a tile
constexpr int kApRows = 256;   // rows of a block
constexpr float kApSlack = 8.f;  // log2 of the growth that O is not rescaled for

template <int D, bool FP8>
struct AttnPfCfg {
  static constexpr int HALVES = D / 64;                // 128-byte column boxes
  static constexpr int BOX = kApTile * 128;            // 128 rows x 64 columns
  static constexpr int TILE = HALVES * BOX;            // a query, key or value tile (bf16)
  static constexpr int PAIRS = D == 128 ? 2 : 4;       // ring of (value tile, next key tile)
  static constexpr int RAW = kApTile * D;              // an e4m3 tile as it lies in the cache
  // rows, producer, two issuers, a spare; e4m3: four converting warps
  static constexpr int THREADS = FP8 ? 512 : 384;
  // registers of the rows' threads and of the others: together those of the launch
  static constexpr int ROW_REGS = FP8 ? 208 : 216, OTHER_REGS = FP8 ? 48 : 72;
  static_assert(256 * ROW_REGS + (THREADS - 256) * OTHER_REGS == THREADS * (65536 / THREADS / 8 * 8), "");
  // queries, the ring, and the first keys' tile or (e4m3, whose first keys lie
  // in the last pair's place) two raw tiles
  static constexpr int SMEM = 1024 + 2 * TILE + 2 * PAIRS * TILE + (FP8 ? 2 * RAW : TILE);
};

struct AttnPfParams {
  uint16_t *out;
  long long out_stride;
  const int *page_table, *row_off, *kv_len;
  const float *k_scale, *v_scale;  // e4m3: [n_kv] or null
  float scale_log2;
  int window, n_sink;
  int n_rows, n_q, n_kv, group, pack, pack_shift;
  int n_pages, n_seqs, max_pages, page, page_shift;
  int n_sm;                // blocks that run at once (and parts that the workspace holds)
  float *ws;               // [n_sm]: a part's rows, see the end of the kernel
  unsigned int *arrived;   // [n_sm], zero between calls
  int *status;
};

// Parts that a block's n key tiles are cut into when it is one of the last
// few: at least four tiles each, and no more than pay for their joining (a tile
// takes about 2 us, a part about 1 us of the join).
MOE_HOST_DEV_INLINE int key_parts(int n, int most) {
  int k = 1;
  while (k < most && n >= 4 * (k + 1) && (k + 1) * (k + 1) <= 2 * n) ++k;
  return k;
}

struct AttnPfShared {
  unsigned long long q_full, kv_full[4], kv_empty[4], s_full[2], p_full[2][2], o_full[2], turn[2], edge, drain[2];
  unsigned long long k0_full, raw_full[2], raw_empty[2];  // e4m3
  long long scan[16];
  uint32_t tmem;
  int item[2];  // sequence, row block
  int dead, last;
};
static_assert(sizeof(AttnPfShared) <= 1024, "fits the block before the tiles");

// Descriptor of an MN-major tile with 128-byte swizzle: lines of 64 columns,
// one line per key; 8-key groups are 1024 B apart (stride offset), 64-column
// halves BOX bytes (leading offset).
MOE_DEV uint64_t umma_desc_mn_sw128(uint32_t saddr, uint32_t half_bytes) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(half_bytes >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D += A B with A (bf16 pairs) in tensor memory
MOE_DEV void umma_f16_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t db, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(db), "r"(idesc), "r"(accumulate));
}
MOE_DEV void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
MOE_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(
          r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
MOE_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
MOE_DEV void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// P of 32 columns of a row: p = 2^(s scale + neg), as bf16 pairs in w, their
// sum added to both halves of `sum`.
MOE_DEV void row_exp2(const uint32_t (&r)[32], uint64_t scale, uint64_t neg, uint32_t (&w)[16], uint64_t &sum) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint64_t x = f2_fma(f2_pack(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), scale, neg);
    float p0, p1;
    f2_unpack(x, p0, p1);
    p0 = ex2(p0);
    p1 = ex2(p1);
    sum = f2_add(sum, f2_pack(p0, p1));
    w[e] = pack_bf16(p0, p1);
  }
}

// Bytes still to come on a barrier, without an arrival.
MOE_DEV void mbar_expect_only(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

template <int D, bool FP8>
__global__ void __launch_bounds__(AttnPfCfg<D, FP8>::THREADS, 1)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const AttnPfParams p) {
  using C = AttnPfCfg<D, FP8>;
  constexpr int kApThreads = C::THREADS;
  extern __shared__ __align__(1024) unsigned char ap_smem[];
  AttnPfShared &sh = *reinterpret_cast<AttnPfShared *>(ap_smem);
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const uint32_t q0 = smem_addr(ap_smem) + 1024, slot0 = q0 + 2 * C::TILE, raw0 = slot0 + 2 * C::PAIRS * C::TILE;
  const uint32_t kfirst = FP8 ? slot0 + (2 * C::PAIRS - 1) * C::TILE : raw0;
  pdl_wait();

  // ---- this block's item: head group fastest (blocks that share keys run
  // together), then row blocks from the sequence's last (the longest) back.
  // What is left after whole waves of one block an SM has its keys split over
  // the SMs: the last `rem` items come in up to n_sm / rem parts.
  const int n_hg = p.n_q >> p.pack_shift;
  const int tokens = kApRows >> p.pack_shift;  // of a block
  const int per = (p.n_seqs + kApThreads - 1) / kApThreads;
  const int b_lo = min(tid * per, p.n_seqs), b_hi = min(b_lo + per, p.n_seqs);
  auto view = [&](int b) { return seq_view(p.row_off, p.kv_len, b, p.n_rows, p.max_pages, p.page); };
  auto blocks_of = [&](const SeqView &s) { return (s.rows + tokens - 1) / tokens; };
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const SeqView s = view(b);
    if (!s.ok && blockIdx.x == 0) atomicOr(p.status, kErrBadBatch);
    mine += blocks_of(s);
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh.scan[wid] = inc;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kApThreads / 32; ++w) {
    if (w < wid) before += sh.scan[w];
    total += sh.scan[w];
  }
  const long long all = total * n_hg, whole = all / p.n_sm * p.n_sm;
  const int rem = (int)(all - whole);
  int tail = -1, part = 0, most = 1;  // index among the last items
  long long at = blockIdx.x;
  if (at >= whole) {
    most = rem ? p.n_sm / rem : 0;
    // Offsets that descend (reported) can make more items than the grid was
    // sized for: then none is split, or some parts would have no block and
    // their arrivals stay counted.
    if (all > (long long)gridDim.x - p.n_sm) most = 1;
    const int x = (int)(at - whole);
    if (x >= rem * most) return;  // block-uniform: the grid is sized for the most blocks there can be
    part = x / rem;
    tail = x - part * rem;
    at = whole + tail;
  }
  const int hg = (int)(at % n_hg), item = (int)(at / n_hg);
  inc += before;
  if (item >= inc - mine && item < inc) {
    long long from = inc - mine;
    for (int b = b_lo; b < b_hi; ++b) {
      const int n = blocks_of(view(b));
      if (item < from + n) {
        sh.item[0] = b;
        sh.item[1] = n - 1 - (int)(item - from);
        break;
      }
      from += n;
    }
  }
  if (tid == 0) {
    mbar_init(smem_addr(&sh.q_full), 1);
    for (int i = 0; i < C::PAIRS; ++i) {
      mbar_init(smem_addr(&sh.kv_full[i]), FP8 ? 8 : 1);  // e4m3: four warps, values and keys
      mbar_init(smem_addr(&sh.kv_empty[i]), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_addr(&sh.s_full[t]), 1);
      mbar_init(smem_addr(&sh.p_full[t][0]), 4);
      mbar_init(smem_addr(&sh.p_full[t][1]), 4);
      mbar_init(smem_addr(&sh.o_full[t]), 1);
      mbar_init(smem_addr(&sh.turn[t]), 1);
      mbar_init(smem_addr(&sh.drain[t]), 1);
    }
    mbar_init(smem_addr(&sh.edge), 1);
    mbar_init(smem_addr(&sh.k0_full), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.raw_full[i]), 1);
      mbar_init(smem_addr(&sh.raw_empty[i]), 4);
    }
    sh.dead = 0;
    fence_mbar_init();
  }
  if (wid == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int b = sh.item[0];
  const SeqView s = view(b);
  const int t_lo = sh.item[1] * tokens, t_hi = min(t_lo + tokens, s.rows);
  const int pos0 = s.kv - s.rows;
  const int kv_h = (hg << p.pack_shift) / p.group;
  // the block's rows as a sequence of their own: its keys end with its last row
  SeqView sv = s;
  sv.rows = t_hi - t_lo;
  sv.kv = pos0 + t_hi;
  const SeqTiles tl = seq_tiles(sv, p.window, p.n_sink, kApTile);
  // this part's tiles
  const int parts = key_parts(tl.n, most);
  if (part >= parts) {  // block-uniform
    if (wid == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    return;
  }
  const int j_lo = (int)((long long)tl.n * part / parts), n_tiles = (int)((long long)tl.n * (part + 1) / parts) - j_lo;
  auto key_of = [&](int j) { return tile_at_lead_last(tl, j_lo + j) * kApTile; };
  auto give_up = [&]() {
    *reinterpret_cast<volatile int *>(&sh.dead) = 1;
    atomicOr(p.status, kErrTimeout);
  };

  auto few_registers = [] { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS)); };
  // keys that some row of the sequence sees: [0, sink_end) and [seen_lo, kv).
  // Values outside may hold anything: such rows of a value tile become zeros
  // before the tensor cores read them.
  const long long seen_lo = p.window > 0 ? (long long)pos0 - p.window + 1 : 0;
  const int sink_end = seen_lo > 0 ? (int)min((long long)p.n_sink, seen_lo) : 0;
  auto seen_by_some = [&](int k) { return k < s.kv && (k < sink_end || k >= seen_lo); };
  // whether a tile from key0 on holds such rows (key0 + kApTile may be 2^31)
  auto edge_tile = [&](int key0) {
    return key0 > s.kv - kApTile || (key0 < seen_lo && key0 > sink_end - kApTile);
  };
  if (wid == 8) {
    // ---------------------------------------------------------- producer
    few_registers();
    const int pr = min(p.page, kApTile);
    const int ppt = kApTile / pr;  // boxes along a tile's keys, at most 8
    constexpr int COLS = FP8 ? 1 : C::HALVES;  // column boxes of a page
    const int my_page = lane / COLS, my_half = lane % COLS;
    // 32 entries of the page table, one per lane, and the 32 behind them
    // already on their way: a look-up is never waited for between tiles
    const int n_pg = (s.kv + p.page - 1) >> p.page_shift;  // pages that hold keys
    const int *table = p.page_table + (long long)b * p.max_pages;
    auto entries = [&](int at) { return at + lane < n_pg ? __ldg(table + at + lane) : 0; };
    int held_at = -64, held = 0, ahead = 0;
    // this lane's box of tile j: whether its page holds a key that is seen,
    // and its row in the cache
    auto box_of = [&](int j, bool &need, int &y) {
      const int key0 = key_of(j), pg0 = key0 >> p.page_shift;
      if (pg0 < held_at || pg0 + ppt > held_at + 32) {
        held = pg0 == held_at + 32 ? ahead : entries(pg0);
        held_at = pg0;
        ahead = entries(pg0 + 32);
      }
      const int first_key = key0 + my_page * pr;
      int page = __shfl_sync(0xffffffffu, held, min(pg0 - held_at + my_page, 31));
      need = lane < ppt * COLS && keys_seen(s, p.window, p.n_sink, first_key, pr);
      if (need && (unsigned)page >= (unsigned)p.n_pages) {
        atomicOr(p.status, kErrBadPage);
        page = 0;  // an in-bounds page; the call's result is reported as bad
      }
      y = (page * p.n_kv + kv_h) * p.page + (first_key & (p.page - 1));
    };
    constexpr int LINE = FP8 ? D : 128;  // bytes of a box row
    const uint32_t box_at = my_half * C::BOX + my_page * pr * LINE;
    auto bytes_of = [&](bool need) { return (uint32_t)__popc(__ballot_sync(0xffffffffu, need)) * pr * LINE; };
    auto load_queries = [&](uint32_t bar) {
      for (int t = 0; t < 2; ++t)
        for (int h = 0; h < C::HALVES; ++h)
          tma_load_3d(q0 + t * C::TILE + h * C::BOX, &qmap, h * 64, hg << p.pack_shift,
                      s.row0 + t_lo + t * (tokens / 2), bar);
    };
    const uint32_t q_bar = smem_addr(&sh.q_full);
    bool ok = true;
    if constexpr (FP8) {
      // the raw tiles in the order they are used: K0, V0, K1, V1, ...
      if (lane == 0) {
        mbar_expect_tx(q_bar, 2 * C::TILE);
        load_queries(q_bar);
      }
      bool need = false;
      int y = 0, issued = 0;
      for (int i = 0; i < 2 * n_tiles; ++i) {
        if (!(i & 1)) box_of(i >> 1, need, y);
        const int st = i & 1, use = i >> 1;
        const uint32_t bytes = bytes_of(need), bar = smem_addr(&sh.raw_full[st]);
        if (use > 0) ok = mbar_wait_warp(smem_addr(&sh.raw_empty[st]), (use - 1) & 1, &sh.dead);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(bar, bytes);
        __syncwarp();
        if (need) tma_load_2d(raw0 + st * C::RAW + box_at, i & 1 ? &vmap : &kmap, 0, y, bar);
        ++issued;
      }
      if (!ok && lane == 0) give_up();
      // no tile may land after the block has gone
      (void)mbar_wait_bounded(q_bar, 0);
      for (int i = max(0, issued - 2); i < issued; ++i)
        (void)mbar_wait_bounded(smem_addr(&sh.raw_full[i & 1]), (i >> 1) & 1);
    } else {
    bool need, need_k;
    int y, y_k;
    box_of(0, need, y);
    const uint32_t bytes0 = bytes_of(need);
    if (lane == 0) {  // the queries and the first keys
      mbar_expect_tx(q_bar, 2 * C::TILE + bytes0);
      load_queries(q_bar);
    }
    __syncwarp();
    if (need) tma_load_2d(kfirst + box_at, &kmap, my_half * 64, y, q_bar);
    int issued = 0, edge_issued = 0, edge_uses = 0;
    for (int j = 0; j < n_tiles; ++j) {
      const int key0 = key_of(j);
      need_k = false;
      if (j + 1 < n_tiles) box_of(j + 1, need_k, y_k);
      const int st = j % C::PAIRS, use = j / C::PAIRS;
      const bool edge = edge_tile(key0);
      const uint32_t bytes_v = bytes_of(need), bytes_k = bytes_of(need_k);
      if (use > 0) ok = mbar_wait_warp(smem_addr(&sh.kv_empty[st]), (use - 1) & 1, &sh.dead);
      if (!ok) break;
      const uint32_t full = smem_addr(&sh.kv_full[st]), bar = edge ? smem_addr(&sh.edge) : full;
      const uint32_t dst = slot0 + st * 2 * C::TILE;
      if (lane == 0) {
        if (edge) {
          mbar_expect_tx(bar, bytes_v);
          mbar_expect_only(full, bytes_k);  // the arrival follows when the values are in order
        } else {
          mbar_expect_tx(full, bytes_v + bytes_k);
        }
      }
      __syncwarp();
      if (need) tma_load_2d(dst + box_at, &vmap, my_half * 64, y, bar);
      if (need_k) tma_load_2d(dst + C::TILE + box_at, &kmap, my_half * 64, y_k, full);
      ++issued;
      edge_issued += edge;
      if (edge) {
        ok = mbar_wait_warp(bar, edge_uses & 1, &sh.dead);
        if (!ok) break;  // not in order: nobody is told to read this tile
        ++edge_uses;
        for (int r = lane; r < kApTile; r += 32) {
          if (seen_by_some(key0 + r)) continue;
#pragma unroll
          for (int i = 0; i < 8 * C::HALVES; ++i)  // a key's line in each half: 8 16-byte pieces
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst + (i >> 3) * C::BOX + r * 128 +
                                                                       ((i + r) & 7) * 16),
                         "r"(0)
                         : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
      }
      need = need_k;
      y = y_k;
    }
    if (!ok && lane == 0) give_up();
    // no tile may land after the block has gone
    (void)mbar_wait_bounded(q_bar, 0);
    if (edge_uses < edge_issued) {
      // given up on an edge tile: its pair's barrier still waits for this
      // warp's arrival, which the values' landing stands in for
      if (mbar_wait_bounded(smem_addr(&sh.edge), edge_uses & 1)) {
        if (lane == 0) mbar_arrive(smem_addr(&sh.kv_full[(issued - 1) % C::PAIRS]));
        __syncwarp();
      } else {
        --issued;
      }
    }
    for (int j = max(0, issued - C::PAIRS); j < issued; ++j)
      (void)mbar_wait_bounded(smem_addr(&sh.kv_full[j % C::PAIRS]), (j / C::PAIRS) & 1);
    }
  } else if (wid == 9 || wid == 10) {
    // ------------------------------------- MMA issuers, one per row tile
    few_registers();
    if (lane == 0) {
      const int t = wid - 9;
      constexpr uint32_t IDESC_S = umma_idesc_bf16(128, kApTile);
      constexpr uint32_t IDESC_O = umma_idesc_bf16(128, D) | (1u << 16);  // B is MN-major
      const uint32_t s_at = tmem + t * 128, o_at = tmem + 256 + t * D;
      const uint64_t qd = umma_desc_sw128(q0 + t * C::TILE);
      auto scores = [&](uint32_t ka) {  // S = Q K^T
        const uint64_t kd = umma_desc_sw128(ka);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          constexpr int half = C::BOX >> 4;
          umma_f16(s_at, qd + (kk >> 2) * half + (kk & 3) * 2, kd + (kk >> 2) * half + (kk & 3) * 2, IDESC_S,
                   kk != 0);
        }
        umma_commit(smem_addr(&sh.s_full[t]));
      };
      bool ok = mbar_wait_live(smem_addr(&sh.q_full), 0, &sh.dead);
      if (FP8) ok = ok && mbar_wait_live(smem_addr(&sh.k0_full), 0, &sh.dead);
      if (ok) {
        tc_fence_after();
        scores(kfirst);
        if (FP8) umma_commit(smem_addr(&sh.kv_empty[C::PAIRS - 1]));  // the first keys' place
        if (t == 1) mbar_arrive(smem_addr(&sh.turn[0]));
      }
      for (int j = 0; j < n_tiles && ok; ++j) {
        const int st = j % C::PAIRS;
        const uint32_t va = slot0 + st * 2 * C::TILE;
        ok = mbar_wait_live(smem_addr(&sh.kv_full[st]), (j / C::PAIRS) & 1, &sh.dead) &&
             mbar_wait_live(smem_addr(&sh.turn[t]), j & 1, &sh.dead);
        const uint64_t vd = umma_desc_mn_sw128(va, C::BOX);
        for (int h = 0; h < 2 && ok; ++h) {
          ok = mbar_wait_live(smem_addr(&sh.p_full[t][h]), j & 1, &sh.dead);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // O += P V, 64 keys
            umma_f16_ta(o_at, s_at + h * 32 + kk * 8, vd + (h * 4 + kk) * (2048 >> 4), IDESC_O, (j | h | kk) != 0);
        }
        if (!ok) break;
        // in order behind the product that reads P, whose columns it overwrites
        if (j + 1 < n_tiles) scores(va + C::TILE);
        else umma_commit(smem_addr(&sh.o_full[t]));
        mbar_arrive(smem_addr(&sh.turn[t ^ 1]));
        umma_commit(smem_addr(&sh.kv_empty[st]));
      }
      if (!ok) {
        give_up();
        // every issued MMA is complete before tensor memory is released
        umma_commit(smem_addr(&sh.drain[t]));
        (void)mbar_wait_bounded(smem_addr(&sh.drain[t]), 0);
      }
    }
  } else if (wid == 11) {
    few_registers();
  } else if (FP8 && wid >= 12) {
    // ------------------- converting warps: e4m3 tiles to bf16, which holds
    // every e4m3 value; the scales go to the scores and the output
    few_registers();
    const int c16 = tid % (D / 16);  // this lane's 16 columns
    bool ok = true;
    for (int i = 0; i <= 2 * n_tiles && ok; ++i) {
      // tile i: key tile i / 2, or value tile i / 2; key tile n does not exist
      const int j = i >> 1, st = i & 1;
      const bool is_v = i & 1, there = i < 2 * n_tiles;
      const int pair = i == 0 ? C::PAIRS - 1 : (is_v ? j : j - 1) % C::PAIRS;
      const uint32_t dst = slot0 + (2 * pair + (is_v ? 0 : 1)) * C::TILE;
      if (is_v) {  // the pair's place is free (the last pair's held the first keys)
        const int free = j / C::PAIRS - (pair == C::PAIRS - 1 ? 0 : 1);
        if (free >= 0) ok = mbar_wait_warp(smem_addr(&sh.kv_empty[pair]), free & 1, &sh.dead);
      }
      if (there && ok) {
        ok = mbar_wait_warp(smem_addr(&sh.raw_full[st]), j & 1, &sh.dead);
        if (ok) {
          const int key0 = key_of(j);
          const bool edge = is_v && edge_tile(key0);
#pragma unroll 2
          for (int r = (tid & 127) / (D / 16); r < kApTile; r += 128 / (D / 16)) {
            uint4 v = lds_u4(raw0 + st * C::RAW + r * D + c16 * 16);
            if (edge && !seen_by_some(key0 + r)) v = make_uint4(0, 0, 0, 0);
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
            uint32_t out[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t h = e4m3x2_to_f16x2(in[e >> 1] >> (16 * (e & 1)));
              out[e] = pack_bf16(half_lo(h), half_hi(h));
            }
            // 16 columns: two 16-byte pieces of the row's line, swizzled by the row
            const uint32_t line = dst + (c16 >> 2) * C::BOX + r * 128;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                               line + (((2 * (c16 & 3) + e) ^ (r & 7)) << 4)),
                           "r"(out[4 * e]), "r"(out[4 * e + 1]), "r"(out[4 * e + 2]), "r"(out[4 * e + 3])
                           : "memory");
          }
        }
      }
      if (!ok) break;
      fence_proxy_async_smem();  // the tensor cores read the tile through the async proxy
      __syncwarp();
      if (lane == 0) {
        if (there) mbar_arrive(smem_addr(&sh.raw_empty[st]));
        mbar_arrive(i == 0 ? smem_addr(&sh.k0_full) : smem_addr(&sh.kv_full[pair]));
      }
    }
    if (!ok && lane == 0) give_up();
  } else {
    // -------------------------------------------------- one thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::ROW_REGS));
    const float scale_log2 = p.scale_log2 * (FP8 && p.k_scale ? __ldg(p.k_scale + kv_h) : 1.f);
    const int t = wid >> 2, row = (wid & 3) * 32 + lane;
    const int tok = t_lo + t * (tokens / 2) + (row >> p.pack_shift);
    const int head = (hg << p.pack_shift) + (row & (p.pack - 1));
    const bool mine_ok = tok < t_hi;
    const int pos = pos0 + min(tok, t_hi - 1);
    const uint32_t lanes = (uint32_t)((wid & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + 256 + t * D;
    float m_ref = -INFINITY, l_run = 0.f;  // m_ref in units of the scores times scale_log2
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      const int key0 = key_of(j);
      // visible columns: c <= hi by position; with a window c >= lo or c < sk
      const int hi = pos - key0;
      const int lo = p.window > 0 ? (int)max(0LL, (long long)hi - p.window + 1) : 0;
      const int sk = max(0, p.n_sink - key0);
      const bool masked = __any_sync(0xffffffffu, !(hi >= kApTile - 1 && (lo <= 0 || sk >= kApTile)));
      ok = mbar_wait_live(smem_addr(&sh.s_full[t]), j & 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t r[4][32];
      tmem_ld32_issue(s_at, r[0]);
      tmem_ld32_issue(s_at + 32, r[1]);
      tmem_ld32_wait(r[0]);
      tmem_ld32_wait(r[1]);
      tmem_ld32_issue(s_at + 64, r[2]);
      tmem_ld32_issue(s_at + 96, r[3]);
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };  // bits [0, n)
      auto look = [&](int c) {  // masks 32 columns and takes their maximum
        if (masked) {
          // a bit per visible column of these 32
          const uint32_t vis = below(hi + 1 - c * 32) & (~below(lo - c * 32) | below(sk - c * 32));
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(vis >> e & 1u)) r[c][e] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            m4[k] = fmaxf(m4[k], fmaxf(__uint_as_float(r[c][e + 2 * k]), __uint_as_float(r[c][e + 2 * k + 1])));
      };
      look(0);
      look(1);
      tmem_ld32_wait(r[2]);
      tmem_ld32_wait(r[3]);
      look(2);
      look(3);
      const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale_log2;
      // the reference follows the maximum when it fell 2^kApSlack behind (the
      // commit that brought S also says that O holds every earlier product)
      const bool first = m_ref == -INFINITY;
      const bool grow = mx > m_ref + kApSlack;
      float corr = 1.f;
      if (first) {
        m_ref = mx;
      } else if (grow) {
        corr = ex2(m_ref - mx);
        m_ref = mx;
      }
      if (__any_sync(0xffffffffu, corr != 1.f)) {
        l_run *= corr;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32_issue(o_at + c * 32, o);
          tmem_ld32_wait(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
          tmem_st32(o_at + c * 32, o);
        }
      }
      const float neg = m_ref == -INFINITY ? 0.f : -m_ref;  // nothing seen yet: 2^-inf = 0
      const uint64_t scale2 = f2_pack(scale_log2, scale_log2), neg2 = f2_pack(neg, neg);
      uint64_t sum = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
        row_exp2(r[c], scale2, neg2, w, sum);
        tmem_st16(s_at + c * 16, w);
        if (c & 1) {  // half of the keys: their product can start
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[t][c >> 1]));
        }
      }
      float sum0, sum1;
      f2_unpack(sum, sum0, sum1);
      l_run += sum0 + sum1;
    }
    if (ok) ok = mbar_wait_warp(smem_addr(&sh.o_full[t]), 0, &sh.dead);
    const float vs = FP8 && p.v_scale ? __ldg(p.v_scale + kv_h) : 1.f;
    uint16_t *dst = p.out + (long long)(s.row0 + tok) * p.out_stride + (long long)head * D;
    auto store = [&](int c, const float (&v)[32]) {  // 32 columns of the row
#pragma unroll
      for (int e = 0; e < 32; e += 8)
        *reinterpret_cast<uint4 *>(dst + c * 32 + e) = make_uint4(
            pack_bf16(v[e], v[e + 1]), pack_bf16(v[e + 2], v[e + 3]), pack_bf16(v[e + 4], v[e + 5]),
            pack_bf16(v[e + 6], v[e + 7]));
    };
    if (!ok && lane == 0) give_up();
    if (parts == 1) {
      if (ok) {
        tc_fence_after();
        const float inv = vs / l_run;
        // Each warp turns its 32 rows in the place of its queries (every
        // product that reads them is through), so that whole rows leave at a
        // time: a thread's own row in 16-byte pieces would touch 32 lines a
        // store.  A row's pieces are swizzled by the row.
        constexpr int PIECES = D / 8;
        const uint32_t mine = q0 + t * C::TILE + (wid & 3) * 32 * D * 2;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          tmem_ld32(o_at + c * 32, v);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(mine + lane * D * 2 +
                                                                       (((c * 4 + e) ^ (lane & 7)) << 4)),
                         "r"(pack_bf16(v[8 * e] * inv, v[8 * e + 1] * inv)),
                         "r"(pack_bf16(v[8 * e + 2] * inv, v[8 * e + 3] * inv)),
                         "r"(pack_bf16(v[8 * e + 4] * inv, v[8 * e + 5] * inv)),
                         "r"(pack_bf16(v[8 * e + 6] * inv, v[8 * e + 7] * inv))
                         : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const int at = i * 32 + lane, r = at / PIECES, piece = at % PIECES;
          const int rr = (wid & 3) * 32 + r, tk = t_lo + t * (tokens / 2) + (rr >> p.pack_shift);
          const uint4 v = lds_u4(mine + r * D * 2 + ((piece ^ (r & 7)) << 4));
          if (tk < t_hi)
            *reinterpret_cast<uint4 *>(p.out + (long long)(s.row0 + tk) * p.out_stride +
                                       (long long)((hg << p.pack_shift) + (rr & (p.pack - 1))) * D + piece * 8) = v;
        }
      }
    } else {
      // A part's rows: o as [D / 4][256 rows] groups of four columns, then the
      // references and the sums.  The last part to arrive adds them up, in
      // their order.
      constexpr int PART = kApRows * (D + 2);
      const int rr = t * 128 + row;
      float *const parts_at = p.ws + (long long)tail * most * PART;
      if (ok) {
        tc_fence_after();
        float *w = parts_at + (long long)part * PART;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          tmem_ld32(o_at + c * 32, v);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4 *>(w + ((c * 8 + e) * kApRows + rr) * 4) =
                make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
        w[kApRows * D + rr] = m_ref;
        w[kApRows * (D + 1) + rr] = l_run;
      }
      bar_sync_n(1, 256);
      if (tid == 0) {
        __threadfence();  // the block's part before its arrival, and every part before the join
        sh.last = atomicAdd(p.arrived + tail, 1u) == (unsigned)parts - 1;
        if (sh.last) p.arrived[tail] = 0;
        __threadfence();
      }
      bar_sync_n(1, 256);
      if (sh.last && mine_ok) {
        float mx = -INFINITY;
        for (int i = 0; i < parts; ++i) mx = fmaxf(mx, __ldcg(parts_at + (long long)i * PART + kApRows * D + rr));
        const float mu = mx == -INFINITY ? 0.f : mx;
        float acc[D / 32][32], l = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[c][e] = 0.f;
        for (int i = 0; i < parts; ++i) {
          const float *w = parts_at + (long long)i * PART;
          const float f = ex2(__ldcg(w + kApRows * D + rr) - mu);
          l += f * __ldcg(w + kApRows * (D + 1) + rr);
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 v = ldcg_f4(w + ((c * 8 + e) * kApRows + rr) * 4);
              acc[c][4 * e] += f * v.x;
              acc[c][4 * e + 1] += f * v.y;
              acc[c][4 * e + 2] += f * v.z;
              acc[c][4 * e + 3] += f * v.w;
            }
        }
        const float inv = vs / l;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[c][e] *= inv;
          store(c, acc[c]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (wid == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

}  // namespace moe
