// Attention of a ragged batch of query tokens over the paged cache:
// causal (pa_prefill: prompts, prompt chunks, drafted tokens) and unmasked
// (pa_cross_attention: a decoder's tokens over an encoder's states).
//
// "KV cache fragmentation" field guide, section "Definition" (the kernel
// walks the page table); the attention formula is Vaswani et al. 2017,
// eq. 1.  Token i of sequence b's nq query tokens sees its first
// lim_i = n - nq + i + 1 (causal) or n (unmasked) cached tokens:
//     out_i = sum_{t < lim_i} softmax(scale <q_i, K_t>)_t V_t,  0 if lim_i = 0.
//
// Rows.  The G query heads of a KV head share its K and V, so the rows of
// one product are (token, head of the group): row r of a tile is its token
// r / G, head r % G, with floor(128 / G) whole tokens in an M = 128 tile.
// An item is two such tiles of one sequence and KV head over the 128-token
// chunks its last row sees: with G = 4 the causal limit moves over only 64
// tokens within an item, so at most one of its chunks is partly masked per
// tile.
//
// Work split.  Items are laid end to end (sequence, KV head, token), each
// kPaItemCost + chunks units long, and CTA c of P takes units
// [U c / P, U (c+1) / P): every CTA gets the same number of chunks whatever
// the lengths.  A sequence's units are a closed form (a floor sum), so a
// CTA finds its first item with one scan over the batch and no plan kernel.
// An item cut by a range boundary leaves a partial (o unnormalised, m, l)
// per piece, which prefill_merge_kernel folds; whole items are written
// directly.  The split depends only on the lengths.
#pragma once

#include "pa_device.cuh"
#include "umma.cuh"

namespace pa {

struct PrefillParams {
  const uint8_t* q;          // [num_tokens][num_q_heads][D] bf16
  __nv_bfloat16* out;        // [num_tokens][num_q_heads][D]
  const int32_t* q_start;    // [num_seqs + 1]; NULL: one token each
  const int32_t* seq_lens;   // [num_seqs]
  const int32_t* block_tables;
  const float* k_scale;      // [num_blocks][num_kv_heads] (FP8)
  const float* v_scale;
  float* ws_o;               // [2 P][D / 4][256] float4
  float2* ws_ml;             // [2 P][256]
  int4* ws_job;              // [P] {last CTA, first token, KV head, tokens}
  int32_t num_seqs, num_tokens, num_q_heads, num_kv_heads, group;
  int32_t tok_per_tile, tok_per_item;  // floor(128 / group), twice that
  int32_t block_size, log2_bs, max_blocks, num_blocks;
  int32_t groups_total;      // 8-row groups of the pool (one past the last: reads zeros)
  int32_t num_ctas;
  int32_t causal;
  int32_t allow_dual;        // the ring is deep enough for both tiles' own chunks
  uint32_t div_group;        // ceil(2^32 / group) for pa_div; 0 when group is 1
  uint32_t q_and, q_xor;     // applied to the query words: negation, or zero
  float sl;                  // |scale| * log2(e), > 0
};

constexpr int kPaRows = 128;           // rows per tile (the MMA's M)
constexpr int kPaTiles = 2;
constexpr int kPaItemRows = kPaRows * kPaTiles;
constexpr int kPaChunk = 128;          // tokens per chunk
// Warps: 0 copies K and V, 1 issues the MMAs, 2 walks the items and loads
// their queries, 3 is idle (the register split takes whole warpgroups); 4-7
// and 8-11 are the softmax of tile 0 and 1.
constexpr int kPaWarps = 12;
constexpr int kPaThreads = 32 * kPaWarps;
constexpr int kPaSoftWarp = 4;
// Registers per thread: all warps start with 168 (65536 / 384 in steps of
// 8); warps 0-3 give up 80 of them to the softmax, whose 128 scores a row
// stay in registers.  128 * 88 + 256 * 208 = 384 * 168.
constexpr int kPaRegs = 168, kPaRegsFew = 88, kPaRegsSoft = 208;
static_assert(128 * kPaRegsFew + 256 * kPaRegsSoft <= kPaThreads * kPaRegs, "register split");
constexpr int kPaItemCost = 1;         // units charged per item besides its chunks
constexpr int kPaTileCols = 256;       // tensor memory per tile: S / P (128), O (D)
constexpr int kPaSCol = 0;
constexpr int kPaOCol = 128;
constexpr int kPaTmemCols = 512;
constexpr int kPaMaxStages = 12;
constexpr int kPaItems = 4;            // item records in flight

constexpr int kPaBarBytes = 1024;

template <int D>
struct PaSmem {
  static constexpr int kKV = kPaChunk * D * 2;  // K (or V) of a chunk
  static constexpr int kStages = D == 64 ? 12 : 5;  // one ring: K_j, V_j, K_j+1, ...
  static constexpr int kQ = kPaRows * D * 2;    // one query tile
  static constexpr int kOffRing = kPaTiles * kQ;
  static constexpr int kOffMl = kOffRing + kStages * kKV;  // tile 1's (m, l), folded by tile 0
  static constexpr int kOffBar = kOffMl + kPaRows * 8;
  static constexpr int kBytes = kOffBar + kPaBarBytes;
  static constexpr int kGroup = D * 16;         // 8 tokens: D / 64 slabs of 8 x 128 bytes
  static_assert(kStages <= kPaMaxStages && kBytes <= 227 * 1024, "shared memory");
};

// One item as the walk hands it to the other warps.
struct alignas(16) PaItem {
  int32_t b, h, n;       // sequence, KV head, cached tokens of the sequence
  int32_t row, nt;       // first token of the batch, tokens
  int32_t seen;          // cached tokens in front of the first token (causal)
  int32_t lim;           // tokens its last row sees
  int32_t j0, j1;        // this CTA's chunks
  int32_t end[2];        // the end of each tile's chunks
  int32_t flags;
  int32_t job;           // the CTA that holds its last chunk
  int32_t pad[3];
};
static_assert(sizeof(PaItem) == 64, "item record");
constexpr int32_t kPaWhole = 1, kPaDual = 2, kPaHead = 4, kPaEnd = 8;

struct PaBars {
  PaItem item[kPaItems];
  uint64_t item_full[kPaItems], item_empty[kPaItems];
  uint64_t full[kPaMaxStages], empty[kPaMaxStages];
  uint64_t q_full[kPaTiles];  // the item's query tile stored
  uint64_t q_raw;             // a query tile before its sign or zero is applied
  uint64_t q_free[kPaTiles];  // the item's last score product of the tile done
  uint64_t s_full[kPaTiles];  // S of the tile's chunk written (and its last product done)
  uint64_t p_full[kPaTiles];  // P of the tile's chunk written
  uint64_t o_last[kPaTiles];  // the tile's last product of the item done
  uint64_t ml_full, o_free;   // dual items: tile 1's (m, l) written; its O read
  uint64_t mma_done;
  int64_t scan[kPaWarps];
  int64_t first_u;            // the CTA's first sequence: units before it
  int32_t first_b;
  int32_t bad;
  uint32_t tmem;
};
static_assert(sizeof(PaBars) <= kPaBarBytes, "barrier block");

// x / group for a row x of an item (below 2^16, where the rounded-up
// reciprocal is exact).
__device__ __forceinline__ uint32_t pa_div(const PrefillParams& p, uint32_t x) {
  return p.div_group == 0u ? x : __umulhi(x, p.div_group);
}

// ------------------------------------------------------------- the plan ---
// sum_{i < n} floor((a i + b) / m), all arguments non-negative.
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t s = 0;
  while (n > 0) {
    if (a >= m) {
      s += static_cast<int64_t>(n) * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      s += static_cast<int64_t>(n) * (b / m);
      b %= m;
    }
    const uint64_t y = static_cast<uint64_t>(a) * n + b;
    if (y < m) break;
    n = static_cast<uint32_t>(y / m);
    b = static_cast<uint32_t>(y % m);
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return s;
}

// One sequence's queries and cached tokens.
struct PaSeq {
  int32_t q0, nq, n, off;  // off: cached tokens before the first query's own
  int32_t items;           // per KV head
};

// Reads sequence b; `bad` when its offsets are out of order or range.
// Lengths outside the table, and more causal queries than tokens, are
// flagged; the latter see nothing (zeros).
__device__ __forceinline__ PaSeq pa_seq(const PrefillParams& p, int32_t b, bool& bad,
                                        bool flag) {
  PaSeq s;
  const int32_t a = p.q_start ? p.q_start[b] : b, e = p.q_start ? p.q_start[b + 1] : b + 1;
  int32_t n = p.seq_lens[b];
  bad = a < 0 || e < a || e > p.num_tokens;
  s.q0 = a;
  s.nq = bad ? 0 : e - a;
  const int32_t cap = p.max_blocks * p.block_size;
  uint32_t err = bad ? PA_DEVERR_BAD_QUERY : 0u;
  if (n < 0 || n > cap) {
    err |= PA_DEVERR_BAD_SEQ_LEN;
    n = n < 0 ? 0 : cap;
  }
  if (p.causal && s.nq > n) {
    err |= PA_DEVERR_BAD_SEQ_LEN;
    n = 0;
  }
  if (flag && err) flag_error(err);
  s.n = n;
  s.off = n - s.nq;
  s.items = (s.nq + p.tok_per_item - 1) / p.tok_per_item;
  return s;
}

// Tokens that the last row of tokens [.., tok_end) of the sequence sees.
__device__ __forceinline__ int32_t pa_limit(const PrefillParams& p, const PaSeq& s,
                                            int32_t tok_end) {
  if (!p.causal) return s.n;
  return s.n == 0 ? 0 : s.off + min(tok_end, s.nq);
}

__device__ __forceinline__ int32_t pa_chunks(int32_t limit) {
  return (limit + kPaChunk - 1) / kPaChunk;
}

// Units of the first k items of one KV head of the sequence.
__device__ __forceinline__ int64_t pa_units(const PrefillParams& p, const PaSeq& s, int32_t k) {
  int64_t u = static_cast<int64_t>(k) * kPaItemCost;
  if (s.n == 0 || k == 0) return u;
  if (!p.causal) return u + static_cast<int64_t>(k) * pa_chunks(s.n);
  int32_t full = k;
  if (k == s.items) {  // the last item may be short
    u += pa_chunks(s.n);
    --full;
  }
  return u + floor_sum(static_cast<uint32_t>(full), kPaChunk,
                       static_cast<uint32_t>(p.tok_per_item),
                       static_cast<uint32_t>(s.off) + p.tok_per_item + (kPaChunk - 1));
}

// The walk over a CTA's items, the same in every thread.
struct PaWalk {
  int64_t lo, hi, u;  // the CTA's units; the current item's first unit
  int32_t b, h, i;    // sequence, KV head, item of the head
  PaSeq s;
  // of the current item
  int32_t tok, nt, lim, chunks;    // first token, tokens, cached tokens seen, chunks
  int32_t j0, j1;                  // this CTA's chunks
  bool mine;                       // this CTA has something to do in it

  __device__ __forceinline__ void item(const PrefillParams& p) {
    tok = i * p.tok_per_item;
    nt = min(p.tok_per_item, s.nq - tok);
    lim = pa_limit(p, s, tok + nt);
    chunks = pa_chunks(lim);
    const int64_t len = chunks + kPaItemCost;
    const int64_t a = lo > u ? lo - u : 0, e = hi - u < len ? hi - u : len;
    j0 = a > kPaItemCost ? static_cast<int32_t>(a - kPaItemCost) : 0;
    j1 = e > kPaItemCost ? static_cast<int32_t>(e - kPaItemCost) : 0;
    mine = chunks == 0 ? a == 0 : j1 > j0;
  }
  __device__ __forceinline__ bool done() const { return u >= hi; }
  __device__ __forceinline__ void next(const PrefillParams& p) {
    u += chunks + kPaItemCost;
    if (u >= hi) return;
    if (++i == s.items) {
      i = 0;
      if (++h == p.num_kv_heads) {
        h = 0;
        bool bad;
        do {
          if (++b >= p.num_seqs) {
            u = hi;
            return;
          }
          s = pa_seq(p, b, bad, false);
        } while (s.items == 0);
      }
    }
    item(p);
  }
  // An item of one tile and several chunks gives both tiles its rows: tile
  // t takes every other chunk from j0 + t, and tile 0 folds the two at the
  // end.
  __device__ __forceinline__ bool dual(const PrefillParams& p) const {
    return p.allow_dual && nt <= p.tok_per_tile && j1 - j0 >= 2;
  }
  // the end of tile t's chunks: past its last row's limit there are none
  __device__ __forceinline__ int32_t tile_end(const PrefillParams& p, int t) const {
    if (nt <= p.tok_per_tile) return t == 0 || dual(p) ? j1 : j0;
    if (t == 1) return j1;
    return max(j0, min(j1, pa_chunks(pa_limit(p, s, tok + p.tok_per_tile))));
  }
};

// Every thread: the batch's units, this CTA's range and its first item.
// Returns false when the CTA has nothing to do.
__device__ __forceinline__ bool pa_plan(const PrefillParams& p, PaBars* bars, PaWalk& w,
                                        int64_t& units, int32_t& parts) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int32_t b0 = static_cast<int32_t>(static_cast<int64_t>(p.num_seqs) * t / kPaThreads);
  const int32_t b1 = static_cast<int32_t>(static_cast<int64_t>(p.num_seqs) * (t + 1) / kPaThreads);
  int64_t sum = 0;
  bool any_bad = false;
  if (t == 0) {
    bars->bad = 0;
    bars->first_b = -1;
  }
  __syncthreads();
  for (int32_t b = b0; b < b1; ++b) {
    bool bad;
    const PaSeq s = pa_seq(p, b, bad, blockIdx.x == 0);
    any_bad |= bad;
    sum += pa_units(p, s, s.items) * p.num_kv_heads;
  }
  if (any_bad) bars->bad = 1;
  int64_t incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == 31) bars->scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kPaWarps; ++i) {
    const int64_t x = bars->scan[i];
    before += i < warp ? x : 0;
    total += x;
  }
  units = total;
  // no more ranges than two units each: a one-chunk item stays whole
  const int64_t most = total / (kPaItemCost + 1);
  parts = static_cast<int32_t>(most < p.num_ctas ? (most < 1 ? 1 : most) : p.num_ctas);
  const int32_t c = blockIdx.x;
  w.lo = c < parts ? total * c / parts : total;
  w.hi = c < parts ? total * (c + 1) / parts : total;
  const bool go = !bars->bad && w.lo < w.hi;
  int64_t at = before + incl - sum;
  if (go && at <= w.lo && w.lo < at + sum) {
    for (int32_t b = b0; b < b1; ++b) {
      bool bad;
      const PaSeq s = pa_seq(p, b, bad, false);
      const int64_t x = pa_units(p, s, s.items) * p.num_kv_heads;
      if (w.lo < at + x) {
        bars->first_b = b;
        bars->first_u = at;
        break;
      }
      at += x;
    }
  }
  __syncthreads();
  if (!go) return false;
  w.b = bars->first_b;
  if (w.b < 0) return false;
  bool bad;
  w.s = pa_seq(p, w.b, bad, false);
  const int64_t per_head = pa_units(p, w.s, w.s.items);
  const int64_t x = w.lo - bars->first_u;
  w.h = static_cast<int32_t>(x / per_head);
  const int64_t y = x - w.h * per_head;
  // the last item that starts at or before y, 32 candidates a round
  int32_t a = 0, e = w.s.items;
  while (e - a > 1) {
    const int32_t step = (e - a + 31) / 32;
    const int64_t k = a + static_cast<int64_t>(lane) * step;
    const bool le = k < e && pa_units(p, w.s, static_cast<int32_t>(k)) <= y;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    a += (31 - __clz(m)) * step;  // lane 0 always holds
    e = min(e, a + step);
  }
  w.i = a;
  w.u = bars->first_u + w.h * per_head + pa_units(p, w.s, a);
  w.item(p);
  return true;
}

// Byte offset of 16-byte chunk c (along the row's D * 2 bytes) of row r in
// a query tile stored as 128-byte slabs (128-byte swizzle).
__device__ __forceinline__ uint32_t pa_q_chunk(int r, int c) {
  return (c >> 3) * (kPaRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// 4D tiled TMA load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int32_t x0,
                                            int32_t x1, int32_t x2, int32_t x3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x0), "r"(x1), "r"(x2), "r"(x3), "r"(bar)
      : "memory");
}

// Producer lane i's block of chunk ch: the table entry of tokens
// [ch * 128 + i * box, + box), or -1 past the sequence.
__device__ __forceinline__ int32_t pa_block_id(const PrefillParams& p, int32_t b, int32_t n,
                                               int32_t ch) {
  const int lane = threadIdx.x & 31;
  const int box = p.block_size < kPaChunk ? p.block_size : kPaChunk;
  const int32_t tok = ch * kPaChunk + lane * box;
  if (lane >= kPaChunk / box || tok >= n) return -1;
  return p.block_tables[static_cast<int64_t>(b) * p.max_blocks + (tok >> p.log2_bs)];
}

// The first 8-row group of that block in the pool; past the sequence, or
// with an id outside the pool (flagged), one past the pool: the TMA fills
// such boxes with zeros.
__device__ __forceinline__ int32_t pa_block_group(const PrefillParams& p, int32_t h, int32_t n,
                                                  int32_t ch, int32_t blk) {
  const int lane = threadIdx.x & 31;
  const int box = p.block_size < kPaChunk ? p.block_size : kPaChunk;
  const int32_t tok = ch * kPaChunk + lane * box;
  if (lane >= kPaChunk / box || tok >= n) return p.groups_total;
  if (blk < 0 || blk >= p.num_blocks) {
    flag_error(PA_DEVERR_BAD_BLOCK_ID);
    return p.groups_total;
  }
  return (blk * p.num_kv_heads + h) * (p.block_size >> 3) +
         ((tok & (p.block_size - 1)) >> 3);
}

// A consumer's place in the item records.
struct PaItems {
  uint32_t k = 0;
  // the next record; NULL after a failed wait
  __device__ __forceinline__ const PaItem* get(PaBars* bars) {
    const bool ok = mbar_wait(smem_addr(&bars->item_full[k % kPaItems]), (k / kPaItems) & 1);
    return __all_sync(0xffffffffu, ok) ? &bars->item[k % kPaItems] : nullptr;
  }
  // the warp has read it
  __device__ __forceinline__ void put(PaBars* bars) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&bars->item_empty[k % kPaItems]));
    ++k;
  }
};

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// ------------------------------------------------------------------ roles ---
// Warp 0: every chunk's K and V into the ring, one 4D box per block by lane
// i: 8-token groups of D / 64 slabs of 8 x 128 bytes, so that a single copy
// carries the block's whole width and successive groups stay one stride
// apart for the matrix descriptors.
template <int D>
__device__ __forceinline__ void pa_copies(const PrefillParams& p, PaBars* bars,
                                          const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                          uint32_t ring) {
  using L = PaSmem<D>;
  const int lane = threadIdx.x & 31;
  const int box = p.block_size < kPaChunk ? p.block_size : kPaChunk;
  PaItems items;
  uint32_t slot = 0;
  bool ok = true;
  while (ok) {
    const PaItem* it = items.get(bars);
    if (it == nullptr || (it->flags & kPaEnd)) break;
    const int32_t b = it->b, h = it->h, n = it->n, j0 = it->j0, j1 = it->j1;
    items.put(bars);
    if (j1 <= j0) continue;
    int32_t e = pa_block_id(p, b, n, j0);
    for (int32_t j = j0; j < j1 && ok; ++j) {
      const int32_t en = j + 1 < j1 ? pa_block_id(p, b, n, j + 1) : -1;  // a chunk ahead
      const int32_t grp = pa_block_group(p, h, n, j, e);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t st = slot % L::kStages, use = slot / L::kStages;
        if (use > 0) ok = mbar_wait(smem_addr(&bars->empty[st]), (use - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t bar = smem_addr(&bars->full[st]);
        if (lane == 0) mbar_arrive_expect_tx(bar, L::kKV);
        __syncwarp();
        if (lane < kPaChunk / box)
          tma_load_4d(ring + st * L::kKV + lane * box * D * 2, kv == 0 ? tm_k : tm_v, 0, 0, 0, grp,
                      bar);
        ++slot;
      }
      e = en;
    }
  }
  // No copy may still target shared memory when the CTA exits: on the
  // normal path the MMAs have consumed every one already.
  if (lane == 0)
    for (uint32_t k = slot < L::kStages ? 0 : slot - L::kStages; k < slot; ++k)
      mbar_wait(smem_addr(&bars->full[k % L::kStages]), (k / L::kStages) & 1, 1u << 16);
}

// Warp 2: walks the CTA's items, hands each to the other warps, and loads
// its query rows into each tile as soon as the item before has done its last
// score product of that tile: the next item's scores start behind its last
// P.V product.  One 4D box per 64-column slab: 64 columns x G heads x the
// tile's tokens.  Tokens past the item are the next sequence's (or zeros
// past the batch): rows that are never stored.
template <int D>
__device__ __forceinline__ void pa_items(const PrefillParams& p, PaBars* bars, PaWalk& w,
                                         const CUtensorMap* tm_q, uint32_t sq, int64_t units,
                                         int32_t parts) {
  using L = PaSmem<D>;
  const int lane = threadIdx.x & 31;
  const uint32_t bytes = static_cast<uint32_t>(p.tok_per_tile * p.group) * D * 2;
  const bool plain = p.q_xor == 0u && p.q_and == 0xffffffffu;
  uint32_t k = 0;           // records written
  uint32_t loaded = 0, phase = 0;  // bit t: tile t has been loaded; parity of its next q_free
  uint32_t raw = 0;         // tiles that took the way over q_raw
  bool ok = true;
  auto publish = [&](const PaItem& it) {
    if (k >= kPaItems) ok = mbar_wait(smem_addr(&bars->item_empty[k % kPaItems]), (k / kPaItems - 1) & 1);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return;
    if (lane == 0) {
      bars->item[k % kPaItems] = it;
      mbar_arrive(smem_addr(&bars->item_full[k % kPaItems]));
    }
    ++k;
  };
  auto record = [&]() {
    PaItem it;
    it.b = w.b;
    it.h = w.h;
    it.n = w.s.n;
    it.row = w.s.q0 + w.tok;
    it.nt = w.nt;
    it.seen = w.s.off + w.tok;
    it.lim = w.lim;
    it.j0 = w.j0;
    it.j1 = w.j1;
    it.end[0] = w.tile_end(p, 0);
    it.end[1] = w.tile_end(p, 1);
    const bool whole = w.j0 == 0 && w.j1 == w.chunks;
    it.flags = (whole ? kPaWhole : 0) | (w.dual(p) ? kPaDual : 0) | (w.j0 == 0 ? kPaHead : 0);
    // the CTA that holds the item's last unit
    const int64_t x = w.u + kPaItemCost + w.chunks;
    it.job = whole ? -1 : static_cast<int32_t>((x * parts - 1) / units);
    return it;
  };
  while (!w.done() && !w.mine) w.next(p);
  PaItem it = {};
  bool have = !w.done();
  if (have)
    it = record();
  else
    it.flags = kPaEnd;
  publish(it);
  while (have && ok) {
    // the record behind this item first: the copies run ahead into it
    const PaItem cur = it;
    do w.next(p);
    while (!w.done() && !w.mine);
    have = !w.done();
    if (have)
      it = record();
    else
      it.flags = kPaEnd;
    publish(it);
    if (!ok || cur.j1 <= cur.j0) continue;
#pragma unroll 1
    for (int t = 0; t < kPaTiles; ++t) {
      if ((t == 0 ? cur.end[0] : cur.end[1]) <= cur.j0) continue;
      if (loaded >> t & 1u) {
        ok = mbar_wait(smem_addr(&bars->q_free[t]), phase >> t & 1u);
        phase ^= 1u << t;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      loaded |= 1u << t;
      const uint32_t dst = sq + t * L::kQ;
      const uint32_t bar = smem_addr(plain ? &bars->q_full[t] : &bars->q_raw);
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int sl = 0; sl < D / 64; ++sl)
          tma_load_4d(dst + sl * (kPaRows * 128), tm_q, 0, cur.h * p.group,
                      cur.row + (cur.flags & kPaDual ? 0 : t * p.tok_per_tile), sl, bar);
      }
      __syncwarp();
      if (plain) continue;
      // a negative or zero scale: the words are changed in place
      ok = mbar_wait(bar, raw++ & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      for (uint32_t i = lane * 16; i < L::kQ; i += 512) {
        uint32_t v[4];
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(dst + i)
                     : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + i),
                     "r"((v[0] & p.q_and) ^ p.q_xor), "r"((v[1] & p.q_and) ^ p.q_xor),
                     "r"((v[2] & p.q_and) ^ p.q_xor), "r"((v[3] & p.q_and) ^ p.q_xor)
                     : "memory");
      }
      fence_proxy_async_smem();  // the MMA (async proxy) reads them
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bars->q_full[t]));
    }
  }
  // no copy in flight at the end: on the normal path the MMAs have read all.
  // A tile's last load has the parity that its next q_free wait would have.
  if (lane == 0 && plain)
    for (int t = 0; t < kPaTiles; ++t)
      if (loaded >> t & 1u)
        mbar_wait(smem_addr(&bars->q_full[t]), phase >> t & 1u, 1u << 16);
}

// Warp 1, lane 0 issuing: per chunk j and tile t, once the softmax has
// written P_j over S_j:
//     O_t += P_j . V_j    (P in tensor memory, V MN-major; N = D)
//     S_t  = Q_t . K_j'^T (the tile's next chunk; both K-major; N = 128)
// in that order: one thread's MMAs run in issue order, so the new scores
// land in P_j's columns only after the product has read them, and their
// completion also means the product is done.  The tiles alternate, so one's
// softmax runs beside the other's MMAs.  The tensor pipe holds some 300
// cycles of issued MMAs: what this warp waits for between two tiles' groups
// stays below that (one wait, for P; the next chunk's copies are looked at
// beforehand, between the tiles).
template <int D>
__device__ __forceinline__ void pa_mma(const PrefillParams& p, PaBars* bars, uint32_t tmem,
                                       uint32_t sq, uint32_t ring) {
  using L = PaSmem<D>;
  constexpr uint32_t kIdQK = idesc_bf16(kPaRows, kPaChunk, false, false);
  constexpr uint32_t kIdPV = idesc_bf16(kPaRows, D, false, true);
  const bool leader = (threadIdx.x & 31) == 0;
  PaItems items;
  uint32_t slot0 = 0;                        // ring slot of the item's first K
  uint32_t qph = 0, pph = 0;  // bit t: parity of tile t's next queries, next P
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(smem_addr(bar), parity));
  };
  auto queries = [&](int t) {
    const bool got = wait(&bars->q_full[t], qph >> t & 1u);
    qph ^= 1u << t;
    return got;
  };
  auto weights = [&](int t) {
    const bool got = wait(&bars->p_full[t], pph >> t & 1u);
    pph ^= 1u << t;
    return got;
  };
  auto landed = [&](uint32_t slot) {
    return wait(&bars->full[slot % L::kStages], (slot / L::kStages) & 1);
  };
  auto there = [&](uint32_t slot) {
    return mbar_test(smem_addr(&bars->full[slot % L::kStages]), (slot / L::kStages) & 1);
  };
  auto scores = [&](int t, uint32_t slot, bool last) {
    if (leader) {
      const uint32_t qb = sq + t * L::kQ, kb = ring + (slot % L::kStages) * L::kKV;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        umma_bf16(tmem + t * kPaTileCols + kPaSCol,
                  smem_desc_sw128(qb + (k >> 2) * (kPaRows * 128) + (k & 3) * 32, 16, 1024),
                  smem_desc_sw128(kb + (k >> 2) * 1024 + (k & 3) * 32, 16, L::kGroup), kIdQK,
                  k > 0);
      umma_commit(smem_addr(&bars->s_full[t]));
      if (last) umma_commit(smem_addr(&bars->q_free[t]));
    }
    __syncwarp();
  };
  auto product = [&](int t, uint32_t slot, bool first) {
    if (leader) {
      const uint32_t tt = tmem + t * kPaTileCols, vb = ring + (slot % L::kStages) * L::kKV;
#pragma unroll
      for (int k = 0; k < kPaChunk / 16; ++k)
        umma_bf16_ta(tt + kPaOCol, tt + kPaSCol + k * 8,
                     smem_desc_sw128(vb + k * 2 * L::kGroup, 1024, L::kGroup), kIdPV,
                     !first || k > 0);
    }
    __syncwarp();
  };
  auto release = [&](uint32_t slot) {
    if (leader) umma_commit(smem_addr(&bars->empty[slot % L::kStages]));
    __syncwarp();
  };
  auto last_of = [&](int t) {
    if (leader) umma_commit(smem_addr(&bars->o_last[t]));
    __syncwarp();
  };
  while (ok) {
    const PaItem* it = items.get(bars);
    if (it == nullptr || (it->flags & kPaEnd)) break;
    const int32_t j0 = it->j0, j1 = it->j1, end0 = it->end[0], end1 = it->end[1];
    const bool dual = it->flags & kPaDual;
    items.put(bars);
    if (j1 <= j0) continue;
    // chunk j: K in slot at(j), V behind it
    auto at = [&](int32_t j) { return slot0 + 2u * static_cast<uint32_t>(j - j0); };
    if (dual) {
      // tile t has chunks j0 + t, j0 + t + 2, ...
      for (int t = 0; t < 2 && ok; ++t) {
        ok = landed(at(j0 + t)) && queries(t);
        if (!ok) break;
        tc_fence_after_sync();
        scores(t, at(j0 + t), j0 + t + 2 >= j1);
        release(at(j0 + t));
      }
      for (int32_t j = j0; j < j1 && ok; ++j) {
        const int t = (j - j0) & 1;
        ok = landed(at(j) + 1) && weights(t);
        if (!ok) break;
        tc_fence_after_sync();
        product(t, at(j) + 1, j - t == j0);
        if (j + 2 < j1) {
          ok = landed(at(j + 2));
          if (!ok) break;
          tc_fence_after_sync();
          scores(t, at(j + 2), j + 4 >= j1);
          release(at(j + 2));
        } else {
          last_of(t);
        }
        release(at(j) + 1);
      }
    } else {
      ok = landed(at(j0));
      for (int t = 0; t < 2 && ok; ++t) {
        if ((t == 0 ? end0 : end1) <= j0) continue;
        ok = queries(t);
        if (!ok) break;
        tc_fence_after_sync();
        scores(t, at(j0), j0 + 1 >= (t == 0 ? end0 : end1));
      }
      if (ok) release(at(j0));
      bool ready = false;  // V_j and K_j+1 have been seen to have landed
      for (int32_t j = j0; j < j1 && ok; ++j) {
        const uint32_t vs = at(j) + 1, ks = at(j + 1);
        if (!ready) ok = landed(vs) && (j + 1 >= j1 || landed(ks));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int32_t end = t == 0 ? end0 : end1;
          if (ok && j < end) {
            ok = weights(t);
            if (ok) {
              tc_fence_after_sync();
              product(t, vs, j == j0);
              if (j + 1 < end)
                scores(t, ks, j + 2 >= end);
              else
                last_of(t);
            }
          }
          if (t == 0 && ok && j + 1 < j1)
            ready = __all_sync(0xffffffffu, there(ks + 1) && (j + 2 >= j1 || there(at(j + 2))));
        }
        if (!ok) break;
        release(vs);
        if (j + 1 < j1) release(ks);
      }
    }
    slot0 += 2u * static_cast<uint32_t>(j1 - j0);
  }
  // every MMA issued has completed before the tensor memory is released
  if (leader) {
    umma_commit(smem_addr(&bars->mma_done));
    mbar_wait(smem_addr(&bars->mma_done), 0, 1u << 16);
  }
  __syncwarp();
}

// -------------------------------------------------------------- softmax ---
// 32 of a thread's raw scores (columns c0 ...); columns from `valid` on
// become -inf.
__device__ __forceinline__ void pa_mask(uint32_t (&u)[32], int32_t c0, int32_t valid) {
#pragma unroll
  for (int i = 0; i < 32; ++i) u[i] = c0 + i < valid ? u[i] : 0xff800000u;
}

// The largest of a thread's 128 scores: three-input maxima in four chains.
__device__ __forceinline__ float pa_row_max(const uint32_t (&u)[4][32]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 32; i += 8)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        m[k] = fmax3(m[k], __uint_as_float(u[c][i + 2 * k]), __uint_as_float(u[c][i + 2 * k + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// 32 columns of an output row as bf16: two stores of a whole 32-byte sector
// each (a row is its own thread's, so narrower stores would send every
// sector twice), or 16-byte stores where out is only 16-byte aligned.
__device__ __forceinline__ void pa_store_out(__nv_bfloat16* dst, const float (&o)[32],
                                             bool wide) {
  uint32_t x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
  if (wide) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 16 * i),
                   "r"(x[8 * i]), "r"(x[8 * i + 1]), "r"(x[8 * i + 2]), "r"(x[8 * i + 3]),
                   "r"(x[8 * i + 4]), "r"(x[8 * i + 5]), "r"(x[8 * i + 6]), "r"(x[8 * i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint4*>(dst)[i] =
          make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
}

// Warps 4-11: four per tile, one row per thread (the warp's quarter of the
// tensor-memory lanes).  A chunk's weights are taken against the running
// maximum m of the chunks before it, without looking for their own maximum:
// a row's weights sum to at most 128 unless a score exceeds m, so while no
// row of the warp sums to more than 2^8, every weight is below 2^8, far from
// overflow.  Otherwise m moves to the true maximum, O and l are scaled, and
// the weights are taken again from the scores still
// in registers.  The first chunk's m is its own maximum.  The weights are
// rounded to bf16 (the A operand of the P.V product; half a step is 2^-8 of
// each) and written over S; l sums them unrounded in fp32.
template <int D>
__device__ __forceinline__ void pa_softmax(const PrefillParams& p, PaBars* bars, int tile,
                                           uint32_t tmem, uint32_t ring, float2* s_ml) {
  using L = PaSmem<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;       // tensor-memory lanes 32 * quarter ...
  const int r = 32 * quarter + lane;  // row within the tile
  const uint32_t tq = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
  const uint32_t tb = tq + tile * kPaTileCols;
  const float sl = p.sl;
  const int32_t rt = static_cast<int32_t>(pa_div(p, static_cast<uint32_t>(r)));  // token of row r
  const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
  PaItems items;
  uint32_t sn = 0, on = 0, cc = 0, dn = 0;  // S tiles, items, chunks of the CTA, dual items
  bool ok = true;
  while (ok) {
    const PaItem* it = items.get(bars);
    if (it == nullptr || (it->flags & kPaEnd)) break;
    const bool dual = it->flags & kPaDual;
    const int32_t j0 = it->j0, begin = j0 + (dual ? tile : 0), step = dual ? 2 : 1;
    const int32_t end = it->end[tile], n = it->n;
    const int32_t tk = rt + (dual ? 0 : tile * p.tok_per_tile);  // the row's token of the item
    const bool has = rt < p.tok_per_tile && tk < it->nt;
    const bool warp_has = __any_sync(0xffffffffu, has);
    // tokens this row sees
    const int32_t lim = !p.causal || !has ? it->lim : it->seen + tk + 1;
    float m = -INFINITY;
    float2 la = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int32_t j = begin; j < end; j += step) {
      ok = mbar_wait(smem_addr(&bars->s_full[tile]), sn++ & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      if (warp_has) {
        uint32_t u[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tb + kPaSCol + 32 * c, u[c]);
        tmem_wait_ld();
        const int32_t valid = lim - j * kPaChunk;
        if (__any_sync(0xffffffffu, valid < kPaChunk)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (__any_sync(0xffffffffu, valid < 32 * c + 32)) pa_mask(u[c], 32 * c, valid);
        }
        bool again = j == begin;  // m is this chunk's maximum: no second pass
        if (again) m = pa_row_max(u) * sl;
        float2 sa, sb;
#pragma unroll 1
        while (true) {
          const float neg = m == -INFINITY ? 0.f : -m;  // a row that sees nothing yet
          const float2 s2 = make_float2(sl, sl), n2 = make_float2(neg, neg);
          sa = sb = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = fma2(
                  make_float2(__uint_as_float(u[c][2 * i]), __uint_as_float(u[c][2 * i + 1])), s2,
                  n2);
              const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              pk[i] = pack_bf16x2(e.x, e.y);
              if (i & 1)
                sb = add2(sb, e);
              else
                sa = add2(sa, e);
            }
            tmem_st16(tb + kPaSCol + 16 * c, pk);
          }
          const float sum = (sa.x + sa.y) + (sb.x + sb.y);
          if (again || !__any_sync(0xffffffffu, sum > 256.f || (m == -INFINITY && sum > 0.f)))
            break;
          // The running max moves: O and l scale by alpha.  O holds the
          // products through the chunk before, all complete (these scores
          // were issued after them), and this chunk's product waits for
          // this warp's P.
          again = true;
          const float mn = fmaxf(m, pa_row_max(u) * sl);
          const float alpha = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
          m = mn;
          la = mul2(la, make_float2(alpha, alpha));
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(tb + kPaOCol + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(tb + kPaOCol + 16 * c, o);
          }
        }
        la = add2(la, add2(sa, sb));
      }
      // The last chunk's tokens past the sequence hold whatever their block
      // held before: their weights are 0, and so must their V be (0 * NaN).
      // The tile clears those rows before its product; when both tiles use
      // the chunk both do, with the same zeros.
      const int32_t past = n - j * kPaChunk;  // valid tokens of the chunk
      if (past < kPaChunk) {
        const uint32_t slot = 2 * (cc + static_cast<uint32_t>(j - j0)) + 1;
        ok = mbar_wait(smem_addr(&bars->full[slot % L::kStages]), (slot / L::kStages) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        constexpr int kCpr = D * 2 / 16;
        const int32_t stop = min(kPaChunk, ((past + p.block_size - 1) >> p.log2_bs) << p.log2_bs);
        const uint32_t vb = ring + (slot % L::kStages) * L::kKV;
        for (int32_t idx = past * kCpr + r; idx < stop * kCpr; idx += kPaRows) {
          const int32_t k = idx / kCpr, c = idx % kCpr;  // the swizzle keeps a row in its row
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                           vb + (k >> 3) * L::kGroup + (c >> 3) * 1024 + (k & 7) * 128 +
                           (c & 7) * 16),
                       "r"(0)
                       : "memory");
        }
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bars->p_full[tile]));
    }
    if (end > begin && ok) {
      ok = mbar_wait(smem_addr(&bars->o_last[tile]), on++ & 1);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (!ok) break;
    tc_fence_after_sync();
    cc += static_cast<uint32_t>(it->j1 - j0);
    float l = la.x + la.y;
    float w0 = 1.f, w1 = 0.f;  // weights of the tiles' O
    if (dual) {
      if (tile == 1) {
        s_ml[r] = make_float2(m, l);
        __syncwarp();
        tc_fence_before_sync();
        if (lane == 0) mbar_arrive(smem_addr(&bars->ml_full));
        ok = mbar_wait(smem_addr(&bars->o_free), dn++ & 1);
        ok = __all_sync(0xffffffffu, ok);
        items.put(bars);
        continue;
      }
      ok = mbar_wait(smem_addr(&bars->ml_full), dn++ & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after_sync();
      const float2 x = s_ml[r];
      const float mn = fmaxf(m, x.x);
      w0 = m == -INFINITY ? 0.f : fast_exp2(m - mn);
      w1 = x.x == -INFINITY ? 0.f : fast_exp2(x.x - mn);
      m = mn;
      l = w0 * l + w1 * x.y;
    }
    if (warp_has) {
      const bool whole = it->flags & kPaWhole;
      const int32_t row = dual ? r : tile * kPaRows + r;  // row within the item
      // a piece: the head of an item in slot 1 of this CTA, a later piece in
      // slot 0 (it is then the CTA's first item)
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (it->flags & kPaHead ? 1 : 0);
      float4* po = reinterpret_cast<float4*>(p.ws_o) + slot * (D / 4) * kPaItemRows + row;
      __nv_bfloat16* po16 =
          p.out + (static_cast<int64_t>(it->row + tk) * p.num_q_heads +
                   it->h * p.group + (r - rt * p.group)) * D;
      if (!whole && has) p.ws_ml[slot * kPaItemRows + row] = make_float2(m, l);
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        w0 *= inv;
        w1 *= inv;
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        float x[32];
        if (end > begin) {
          tmem_ld32(tb + kPaOCol + 32 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = l == 0.f ? 0.f : __uint_as_float(o[i]) * w0;
          if (dual) {
            tmem_ld32(tb + kPaTileCols + kPaOCol + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              x[i] = l == 0.f ? 0.f : fmaf(__uint_as_float(o[i]), w1, x[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.f;
        }
        if (!has) continue;
        if (whole) {
          pa_store_out(po16 + 32 * c, x, wide);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            po[(8 * c + i) * kPaItemRows] =
                make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
      }
      if (!whole && (it->flags & kPaHead) && threadIdx.x == 32 * kPaSoftWarp)
        p.ws_job[blockIdx.x] = make_int4(it->job, it->row, it->h, it->nt);
    }
    tc_fence_before_sync();
    if (dual) {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bars->o_free));
    }
    items.put(bars);
  }
}

template <int D>
__global__ void __launch_bounds__(kPaThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_q, const PrefillParams p) {
  using L = PaSmem<D>;
  extern __shared__ __align__(1024) uint8_t pa_smem[];
  const uint32_t base = smem_addr(pa_smem);
  if (base & 1023u) {  // the same for every CTA of the launch
    if (threadIdx.x == 0) {
      flag_error(PA_DEVERR_LAUNCH);
      p.ws_job[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  PaBars* bars = reinterpret_cast<PaBars*>(pa_smem + L::kOffBar);
  const uint32_t sq = base, ring = base + L::kOffRing;
  const int warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(smem_addr(&bars->full[i]), 1);
      mbar_init(smem_addr(&bars->empty[i]), 1);
    }
    for (int t = 0; t < kPaTiles; ++t) {
      mbar_init(smem_addr(&bars->q_full[t]), 1);
      mbar_init(smem_addr(&bars->q_free[t]), 1);
      mbar_init(smem_addr(&bars->s_full[t]), 1);
      mbar_init(smem_addr(&bars->p_full[t]), 4);
      mbar_init(smem_addr(&bars->o_last[t]), 1);
    }
    for (int i = 0; i < kPaItems; ++i) {
      mbar_init(smem_addr(&bars->item_full[i]), 1);
      mbar_init(smem_addr(&bars->item_empty[i]), 2 + kPaTiles * 4);
    }
    mbar_init(smem_addr(&bars->mma_done), 1);
    mbar_init(smem_addr(&bars->q_raw), 1);
    mbar_init(smem_addr(&bars->ml_full), 4);
    mbar_init(smem_addr(&bars->o_free), 4);
    mbar_fence_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_q);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&bars->tmem), kPaTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem;
  pdl_wait();  // launched as a programmatic dependent: inputs ready below
  pdl_trigger();

  PaWalk w;
  int64_t units;
  int32_t parts;
  const bool work = pa_plan(p, bars, w, units, parts);
  if (threadIdx.x == 32 * kPaSoftWarp) p.ws_job[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (!work) {
    // nothing in this CTA's range
  } else if (warp < kPaSoftWarp) {
    regs_dec<kPaRegsFew>();
    if (warp == 0)
      pa_copies<D>(p, bars, &tm_k, &tm_v, ring);
    else if (warp == 1)
      pa_mma<D>(p, bars, tmem, sq, ring);
    else if (warp == 2)
      pa_items<D>(p, bars, w, &tm_q, sq, units, parts);
  } else {
    regs_inc<kPaRegsSoft>();
    pa_softmax<D>(p, bars, (warp - kPaSoftWarp) >> 2, tmem, ring,
                  reinterpret_cast<float2*>(pa_smem + L::kOffMl));
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kPaTmemCols);
  }
}

// Folds the pieces of each item that a range boundary cut: M = max m_i,
// out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i (0 without any key).
// Block (c, part): 32 rows of the item whose head piece CTA c holds; lane =
// row, so every load of the piece's [D / 4][256] float4 is coalesced; warp w
// takes 8 columns a step.
template <int D>
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillParams p) {
  pdl_wait();
  pdl_trigger();
  const int32_t c = blockIdx.x;
  const int4 job = p.ws_job[c];
  const int row = blockIdx.y * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
  const int32_t r = row & (kPaRows - 1), rt = static_cast<int32_t>(pa_div(p, r));
  const int32_t tk = rt + (row >= kPaRows ? p.tok_per_tile : 0);
  if (rt >= p.tok_per_tile || tk >= job.w || job.x >= p.num_ctas) return;
  auto slot = [&](int32_t i) -> int64_t { return 2 * static_cast<int64_t>(i) + (i == c ? 1 : 0); };
  float M = -INFINITY;
  for (int32_t i = c; i <= job.x; ++i) M = fmaxf(M, p.ws_ml[slot(i) * kPaItemRows + row].x);
  const int64_t orow = static_cast<int64_t>(job.y + tk) * p.num_q_heads + job.z * p.group +
                       (r - rt * p.group);
#pragma unroll
  for (int cc = 0; cc < D / 64; ++cc) {
    const int col = warp + 8 * cc;  // 8 columns each
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    float l = 0.f;
    for (int32_t i = c; i <= job.x; ++i) {
      const int64_t s = slot(i);
      const float2 ml = p.ws_ml[s * kPaItemRows + row];
      const float4* po = reinterpret_cast<const float4*>(p.ws_o) +
                         (s * (D / 4) + 2 * col) * kPaItemRows + row;
      const float4 x = po[0], y = po[kPaItemRows];
      if (ml.x == -INFINITY) continue;  // a piece the row sees nothing of
      const float wgt = fast_exp2(ml.x - M);
      l = fmaf(wgt, ml.y, l);
      a.x = fmaf(wgt, x.x, a.x);
      a.y = fmaf(wgt, x.y, a.y);
      a.z = fmaf(wgt, x.z, a.z);
      a.w = fmaf(wgt, x.w, a.w);
      b.x = fmaf(wgt, y.x, b.x);
      b.y = fmaf(wgt, y.y, b.y);
      b.z = fmaf(wgt, y.z, b.z);
      b.w = fmaf(wgt, y.w, b.w);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint4 o;
    o.x = pack_bf16x2(a.x * inv, a.y * inv);
    o.y = pack_bf16x2(a.z * inv, a.w * inv);
    o.z = pack_bf16x2(b.x * inv, b.y * inv);
    o.w = pack_bf16x2(b.z * inv, b.w * inv);
    reinterpret_cast<uint4*>(p.out + orow * D)[col] = o;
  }
}

}  // namespace pa
