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
//
// FP8 caches: four more warps widen the E4M3 codes to bf16 (exact) between
// the copies and the MMAs; the per-(block, head) scales never touch the
// codes: K's multiply the scores, V's the softmax weights, both in fp32 and
// both inside the exponent's one multiply-add per score,
//     v 2^(s k sl - m) = 2^(s (k sl) + (log2 v - m)).
//
// What bounds it, measured (32 query and 8 KV heads, head_dim 128, bf16,
// captured graph).  One prompt of 8192 tokens: 377 us, 1.46 PFLOP/s, DRAM 6 %:
// per chunk and tile the chain scores -> registers -> exponentials -> weights
// back -> two products, of which two tiles hide half.  8 prompts of 64 to 2048
// tokens: 49 us, of which chunks 23, item ends (the last product, rows out, the
// next item's first scores) 9, set-up, plan and merge 12.  48 sequences of 4
// to 8 drafted tokens over 0.5 to 4 thousand: 62.5 us for 329 MB, DRAM 67 %.
// FP8, 64 / 8 heads, 2 x 1021 tokens over 8 to 9 thousand: 590 us, 1.03
// PFLOP/s, of which the widening costs some 12 %.
// Rows per tile: M = 128 is what one CTA's product takes at full rate, and two
// tiles with scores and output fill the 512 tensor-memory columns at D = 128.
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
  uint32_t div_group;        // ceil(2^32 / group) for pa_div; 0 when group is 1
  uint32_t q_and, q_xor;     // applied to the query words: negation, or zero
  float sl;                  // |scale| * log2(e), > 0
};

constexpr int kPaRows = 128;           // rows per tile (the MMA's M)
constexpr int kPaTiles = 2;
constexpr int kPaItemRows = kPaRows * kPaTiles;
constexpr int kPaChunk = 128;          // tokens per chunk
// Warps: 0 copies K and V, 1 walks the items and loads their queries, 2 and
// 3 issue the MMAs of tile 0 and 1; 4-7 and 8-11 are the softmax of tile 0
// and 1; 12-15 (FP8 only) widen the codes.
constexpr int kPaWarps = 12;
constexpr int kPaThreads = 32 * kPaWarps;
constexpr int kPaSoftWarp = 4;
constexpr int kPaConvWarp = kPaWarps;
// Registers per thread.  The launch gives every thread the same (65536 over
// the threads, in steps of 8); the other warpgroups then give up some to the
// softmax, whose 128 scores a row stay in registers.
template <bool FP8>
struct PaRegs {
  static constexpr int kThreads = kPaThreads + (FP8 ? 128 : 0);
  static constexpr int kLaunch = FP8 ? 128 : 168;
  static constexpr int kFew = FP8 ? 56 : 88;
  static constexpr int kSoft = FP8 ? 192 : 208;
  static constexpr int kConv = 72;
  static_assert(128 * kFew + 256 * kSoft + (FP8 ? 128 * kConv : 0) <= kThreads * kLaunch,
                "register split");
};
constexpr int kPaItemCost = 2;         // units charged per item besides its chunks
constexpr int kPaTileCols = 256;       // tensor memory per tile: S / P (128), O (D)
constexpr int kPaSCol = 0;
constexpr int kPaOCol = 128;
constexpr int kPaTmemCols = 512;
constexpr int kPaMaxStages = 12;
constexpr int kPaItems = 4;            // item records in flight

constexpr int kPaBarBytes = 1024;
constexpr int kPaMaxCodeStages = 8;
// per chunk and 8 tokens: k sl, log2 v, 1 / v
constexpr int kPaScaleFloats = 48;


template <int D, bool FP8>
struct PaSmem {
  static constexpr int kKV = kPaChunk * D * 2;  // K (or V) of a chunk, bf16
  static constexpr int kCodes = kPaChunk * D;   // the same as E4M3
  // one ring: K_j, V_j, K_j+1, ...; FP8 has a second one of codes before it
  static constexpr int kStages = FP8 ? (D == 64 ? 8 : 4) : (D == 64 ? 12 : 5);
  static constexpr int kCodeStages = FP8 ? (D == 64 ? 6 : 2) : 0;
  static constexpr int kQ = kPaRows * D * 2;    // one query tile
  static constexpr int kOffRing = kPaTiles * kQ;
  static constexpr int kOffCodes = kOffRing + kStages * kKV;
  static constexpr int kOffMl = kOffCodes + kCodeStages * kCodes;  // tile 1's (m, l), folded by tile 0
  static constexpr int kScales = D == 64 ? 8 : 4;  // chunks whose FP8 scales are kept
  static constexpr int kOffScale = kOffMl + kPaRows * 8;
  static constexpr int kOffBar = kOffScale + (FP8 ? kScales * kPaScaleFloats * 4 : 0);
  static constexpr int kBytes = kOffBar + kPaBarBytes;
  static constexpr int kGroup = D * 16;         // 8 tokens: D / 64 slabs of 8 x 128 bytes
  static_assert(kStages <= kPaMaxStages && kBytes <= 227 * 1024, "shared memory");
  // The copies run ahead of the products by both rings and the one slot that
  // the widening warps hold in registers: when they write a chunk's scales,
  // the products of the chunk that had the place before are done.
  static_assert(!FP8 || kStages + kCodeStages + 1 <= 2 * kScales - 1, "scale ring");
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
  uint64_t code_full[kPaMaxCodeStages], code_empty[kPaMaxCodeStages];  // FP8
  uint64_t scale_full[kPaMaxCodeStages];
  uint64_t q_full[kPaTiles];  // the item's query tile stored
  uint64_t q_raw;             // a query tile before its sign or zero is applied
  uint64_t q_free[kPaTiles];  // the item's last score product of the tile done
  uint64_t s_full[kPaTiles];  // S of the tile's chunk written (and its last product done)
  uint64_t p_full[kPaTiles];  // P of the tile's chunk written, and the tile's turn
  uint64_t o_last[kPaTiles];  // the tile's last product of the item done
  uint64_t ml_full, o_free;   // dual items: tile 1's (m, l) written; its O read
  uint64_t turn;              // tile 0's first MMAs of an item issued: tile 1's first turn
  uint64_t mma_done[kPaTiles];
  int32_t bad;
  uint32_t tmem;
};
static_assert(sizeof(PaBars) <= kPaBarBytes, "barrier block");

// Bounded wait, as mbar_wait, but a short loop that leaves the flagging of a
// timeout to its role's end: this kernel has some thirty waits, and its
// roles share the SM's instruction cache.
__device__ __forceinline__ bool pa_wait(uint32_t bar, uint32_t parity,
                                        uint32_t limit = (1u << 22)) {
#pragma unroll 1
  for (uint32_t i = 0; i < limit; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

// x / group for a row x of an item (below 2^16, where the rounded-up
// reciprocal is exact).
__device__ __forceinline__ uint32_t pa_div(const PrefillParams& p, uint32_t x) {
  return p.div_group == 0u ? x : __umulhi(x, p.div_group);
}

// ------------------------------------------------------------- the plan ---
// sum_{i < n} floor((a i + b) / 128), with a < 2^16, a n + b and the sum below
// 2^32.
__device__ __forceinline__ uint32_t floor_sum(uint32_t n, uint32_t a, uint32_t b) {
  uint32_t m = 128;
  auto pairs = [](uint32_t x) {  // x (x - 1) / 2
    return x & 1 ? (x - 1) / 2 * x : x / 2 * (x - 1);
  };
  if ((a & (a - 1)) == 0) {
    // a = 2^k.  From 128 on: a multiple of the divisor.  Below, with q = 128
    // / a and x = i + b / a, the terms are floor(x / q): a sum of steps.
    const int k = 31 - __clz(a);
    if (k >= 7)
      return (pairs(n) << (k - 7)) + n * (b >> 7);
    auto steps = [&](uint32_t x) {  // sum_{y < x} floor(y / q)
      const uint32_t w = x >> (7 - k), r = x - (w << (7 - k));
      return (pairs(w) << (7 - k)) + w * r;
    };
    return steps((b >> k) + n) - steps(b >> k);
  }
  uint32_t s = 0;
#pragma unroll 1
  while (n > 0) {  // the Euclidean recursion on (m, a)
    if (a >= m) {
      s += pairs(n) * (a / m);
      a %= m;
    }
    if (b >= m) {
      s += n * (b / m);
      b %= m;
    }
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
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
__device__ __forceinline__ uint32_t pa_units(const PrefillParams& p, const PaSeq& s, int32_t k) {
  uint32_t u = k * kPaItemCost;
  if (s.n == 0 || k == 0) return u;
  if (!p.causal) return u + k * pa_chunks(s.n);
  int32_t full = k;
  if (k == s.items) {  // the last item may be short
    u += pa_chunks(s.n);
    --full;
  }
  return u + floor_sum(static_cast<uint32_t>(full), static_cast<uint32_t>(p.tok_per_item),
                       static_cast<uint32_t>(s.off) + p.tok_per_item + (kPaChunk - 1));
}

// The walk over a CTA's items.
struct PaWalk {
  uint32_t lo, hi, u;  // the CTA's units; the current item's first unit
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
    const uint32_t len = chunks + kPaItemCost;
    const uint32_t a = lo > u ? lo - u : 0, e = min(hi - u, len);
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
    return nt <= p.tok_per_tile && j1 - j0 >= 2;
  }
  // the end of tile t's chunks: past its last row's limit there are none
  __device__ __forceinline__ int32_t tile_end(const PrefillParams& p, int t) const {
    if (nt <= p.tok_per_tile) return t == 0 || dual(p) ? j1 : j0;
    if (t == 1) return j1;
    return max(j0, min(j1, pa_chunks(pa_limit(p, s, tok + p.tok_per_tile))));
  }
};

// The plan.  The launch makes sure that the whole batch's units stay below
// 2^32.  A batch of at most 32 sequences is planned by one warp, a sequence
// per lane; larger ones have a first part in which every thread adds up the
// units of its sequences, thread t taking [B t / 384, B (t + 1) / 384).
__device__ __forceinline__ int32_t pa_first_seq(const PrefillParams& p, int t) {
  return static_cast<int32_t>(static_cast<int64_t>(p.num_seqs) * t / kPaThreads);
}

__device__ __forceinline__ uint32_t pa_thread_units(const PrefillParams& p, PaBars* bars) {
  const int t = threadIdx.x;
  uint32_t sum = 0;
#pragma unroll 1
  for (int32_t b = pa_first_seq(p, t), e = pa_first_seq(p, t + 1); b < e; ++b) {
    bool bad;
    const PaSeq s = pa_seq(p, b, bad, blockIdx.x == 0);
    if (bad) bars->bad = 1;
    sum += pa_units(p, s, s.items) * p.num_kv_heads;
  }
  return sum;
}

__device__ __forceinline__ uint32_t pa_warp_sum(uint32_t x) {  // inclusive, over lanes
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
    if ((threadIdx.x & 31) >= d) x += y;
  }
  return x;
}

// floor(units c / parts): the first unit of CTA c.
__device__ __forceinline__ uint32_t pa_share(uint32_t units, uint32_t parts, uint32_t c) {
  const uint32_t q = units / parts, rest = units - q * parts;
  return q * c + rest * c / parts;
}

// One warp: this CTA's range and its first item.  `sums`: the threads' units
// of a batch of more than 32 sequences.  Returns false when the CTA has
// nothing to do.
__device__ __forceinline__ bool pa_plan(const PrefillParams& p, PaBars* bars,
                                        const uint32_t* sums, PaWalk& w, uint32_t& units,
                                        uint32_t& parts) {
  const int lane = threadIdx.x & 31;
  constexpr int kPer = kPaThreads / 32;
  const bool small = p.num_seqs <= 32;
  PaSeq s = {0, 0, 0, 0, 0};
  uint32_t head = 0, mine = 0;  // units of a KV head of the lane's sequence, of all its sequences
  if (small) {
    bool bad = false;
    if (lane < p.num_seqs) s = pa_seq(p, lane, bad, blockIdx.x == 0);
    if (__any_sync(0xffffffffu, bad)) return false;
    head = pa_units(p, s, s.items);
    mine = head * p.num_kv_heads;
  } else {
    if (bars->bad) return false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += sums[lane * kPer + i];  // threads [12 lane, + 12)
  }
  const uint32_t incl = pa_warp_sum(mine);
  units = __shfl_sync(0xffffffffu, incl, 31);
  // no more ranges than two units each: a one-chunk item stays whole
  parts = max(1u, min(units / (kPaItemCost + 1), static_cast<uint32_t>(p.num_ctas)));
  const uint32_t c = blockIdx.x;
  if (c >= parts) return false;
  const uint32_t q = units / parts, rest = units - q * parts;  // as pa_share
  w.lo = q * c + rest * c / parts;
  w.hi = q * (c + 1) + rest * (c + 1) / parts;
  if (w.lo >= w.hi) return false;
  // the sequence that holds unit lo
  const int li = __ffs(__ballot_sync(0xffffffffu, w.lo < incl)) - 1;
  uint32_t at = __shfl_sync(0xffffffffu, incl - mine, li);
  if (small) {
    w.b = li;
    w.s.q0 = __shfl_sync(0xffffffffu, s.q0, li);
    w.s.nq = __shfl_sync(0xffffffffu, s.nq, li);
    w.s.n = __shfl_sync(0xffffffffu, s.n, li);
    w.s.off = __shfl_sync(0xffffffffu, s.off, li);
    w.s.items = __shfl_sync(0xffffffffu, s.items, li);
    head = __shfl_sync(0xffffffffu, head, li);
  } else {
    int t = li * kPer;
#pragma unroll 1
    for (; t < kPaThreads - 1 && w.lo >= at + sums[t]; ++t) at += sums[t];
    w.b = pa_first_seq(p, t);
#pragma unroll 1
    while (true) {
      if (w.b >= p.num_seqs) return false;  // lengths changed under the call
      bool bad;
      w.s = pa_seq(p, w.b, bad, false);
      head = pa_units(p, w.s, w.s.items);
      if (w.lo - at < head * p.num_kv_heads) break;
      at += head * p.num_kv_heads;
      ++w.b;
    }
  }
  // the KV head, then its last item that starts at or before the rest y, 32
  // candidates a round
  uint32_t y = w.lo - at, start = 0;
  w.h = y / head;
  y -= w.h * head;
  at += w.h * head;
  int32_t a = 0, e = w.s.items;
#pragma unroll 1
  while (e - a > 1) {
    const int32_t step = (e - a + 31) / 32, k = min(a + lane * step, e);
    const uint32_t before = pa_units(p, w.s, k);
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, k < e && before <= y));
    start = __shfl_sync(0xffffffffu, before, last);  // lane 0 always qualifies
    a += last * step;
    e = min(e, a + step);
  }
  w.i = a;
  w.u = at + start;
  w.item(p);
  return true;
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
  // the record `ahead` of this one; NULL after a failed wait
  __device__ __forceinline__ const PaItem* get(PaBars* bars, uint32_t ahead = 0) {
    const uint32_t i = k + ahead;
    const bool ok = pa_wait(smem_addr(&bars->item_full[i % kPaItems]), (i / kPaItems) & 1);
    return __all_sync(0xffffffffu, ok) ? &bars->item[i % kPaItems] : nullptr;
  }
  // the warp has read it
  __device__ __forceinline__ void put(PaBars* bars) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&bars->item_empty[k % kPaItems]));
    ++k;
  }
};

// A position in the ring: its stage and the parity of its current use.
template <int kStages>
struct PaRing {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void advance() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

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
// apart for the matrix descriptors.  FP8: plain rows of codes, and each
// chunk's scales, one per 8 tokens.
template <int D, bool FP8>
__device__ __forceinline__ void pa_copies(const PrefillParams& p, PaBars* bars,
                                          const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                          uint32_t ring, float* scales) {
  using L = PaSmem<D, FP8>;
  constexpr uint32_t kS = FP8 ? L::kCodeStages : L::kStages;
  constexpr uint32_t kBytes = FP8 ? L::kCodes : L::kKV;
  uint64_t* full = FP8 ? bars->code_full : bars->full;
  uint64_t* empty = FP8 ? bars->code_empty : bars->empty;
  const int lane = threadIdx.x & 31;
  const int box = p.block_size < kPaChunk ? p.block_size : kPaChunk;
  PaItems items;
  uint32_t slot = 0;
  bool ok = true;
  while (ok) {
    const PaItem* it = items.get(bars);
    if (it == nullptr) {
      ok = false;
      break;
    }
    if (it->flags & kPaEnd) break;
    const int32_t b = it->b, h = it->h, n = it->n, j0 = it->j0, j1 = it->j1;
    items.put(bars);
    if (j1 <= j0) continue;
    // table entries one chunk ahead; FP8: two, and the scales one
    auto id_of = [&](int32_t j) { return j < j1 ? pa_block_id(p, b, n, j) : -1; };
    float2 f = make_float2(1.f, 1.f);
    auto scales_of = [&](int32_t e) {
      float2 x = make_float2(1.f, 1.f);
      if (e >= 0 && e < p.num_blocks) {
        const int64_t i = static_cast<int64_t>(e) * p.num_kv_heads + h;
        x = make_float2(p.k_scale[i], fmaxf(p.v_scale[i], 0x1p-120f));  // 1 / v stays finite
      }
      return x;
    };
    int32_t e = id_of(j0), e1 = FP8 ? id_of(j0 + 1) : 0;
    if (FP8) f = scales_of(e);
    for (int32_t j = j0; j < j1 && ok; ++j) {
      const int32_t en = id_of(j + (FP8 ? 2 : 1));
      const float2 fn = FP8 ? scales_of(e1) : f;
      const int32_t grp = pa_block_group(p, h, n, j, e);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t st = slot % kS, use = slot / kS;
        if (use > 0) ok = pa_wait(smem_addr(&empty[st]), (use - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (FP8 && kv == 0) {
          // group i of 8 tokens lies in block 8 i / box of the chunk
          const uint32_t c = (slot >> 1) % L::kScales;
          const int src = (lane & 15) * 8 / box;
          const float x = __shfl_sync(0xffffffffu, f.x, src), y = __shfl_sync(0xffffffffu, f.y, src);
          float* to = scales + c * kPaScaleFloats;
          to[lane] = lane < 16 ? x * p.sl : log2f(y);
          if (lane < 16) to[32 + lane] = 1.f / y;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&bars->scale_full[c]));
        }
        const uint32_t bar = smem_addr(&full[st]);
        if (lane == 0) mbar_arrive_expect_tx(bar, kBytes);
        __syncwarp();
        if (lane < kPaChunk / box) {
          const uint32_t dst = ring + st * kBytes + lane * box * (FP8 ? D : D * 2);
          if (FP8)
            tma_load_2d(dst, kv == 0 ? tm_k : tm_v, 0, grp * 8, bar);
          else
            tma_load_4d(dst, kv == 0 ? tm_k : tm_v, 0, 0, 0, grp, bar);
        }
        ++slot;
      }
      e = FP8 ? e1 : en;
      e1 = en;
      f = fn;
    }
  }
  if (!ok) flag_error(PA_DEVERR_TIMEOUT);
  // No copy may still target shared memory when the CTA exits: on the
  // normal path the MMAs have consumed every one already.
  if (lane == 0)
    for (uint32_t k = slot < kS ? 0 : slot - kS; k < slot; ++k)
      pa_wait(smem_addr(&full[k % kS]), (k / kS) & 1, 1u << 16);
}

// Four E4M3 codes -> two pairs of bf16, exact: a code's exponent and
// mantissa bits are those of a bf16 value 2^120 smaller (also where they are
// subnormal), which one multiplication puts right.  Integer instructions: the
// conversion instructions share the unit of the softmax's exponentials.  The
// two NaN codes, which no writer of the library stores, come out as +-480.
__device__ __forceinline__ void e4m3x4_to_bf16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);  // codes << 8
  const uint32_t x = ((a >> 4) & 0x07f007f0u) | (a & 0x80008000u);
  const uint32_t y = ((b >> 4) & 0x07f007f0u) | (b & 0x80008000u);
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(0x7b807b80u));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(0x7b807b80u));
}

// Warps 12-15 (FP8): codes to bf16, 16 a step: a 16-byte read, and two
// 16-byte writes into the layout the copies make of a bf16 cache.  A row's
// two slabs share their banks, so threads of the second slab write their two
// chunks in the other order.  Bound by issue slots and shared memory that the
// softmax and the products use too: a chunk of 2 x 1021 tokens over 8 to 9
// thousand that took 616 us took 541 without these warps' work and 553 with
// V's alone.
template <int D>
__device__ __forceinline__ void pa_widen(PaBars* bars, uint32_t codes, uint32_t ring) {
  using L = PaSmem<D, true>;
  const int t = threadIdx.x - 32 * kPaConvWarp, lane = threadIdx.x & 31;
  constexpr int kPer = D / 16;  // 16-byte pieces per row of codes
  PaItems items;
  uint32_t slot = 0;
  bool ok = true;
  while (ok) {
    const PaItem* it = items.get(bars);
    if (it == nullptr) {
      ok = false;
      break;
    }
    if (it->flags & kPaEnd) break;
    const uint32_t end = slot + 2u * static_cast<uint32_t>(max(it->j1 - it->j0, 0));
    items.put(bars);
    for (; slot < end && ok; ++slot) {
      const uint32_t cs = slot % L::kCodeStages, cu = slot / L::kCodeStages;
      const uint32_t st = slot % L::kStages, use = slot / L::kStages;
      ok = pa_wait(smem_addr(&bars->code_full[cs]), cu & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t src = codes + cs * L::kCodes, dst = ring + st * L::kKV;
      // All of the thread's codes into registers, and the copies may refill
      // the stage while they are widened.  The loads are volatile and fenced
      // against the copies' writes: with plain ones and no fence, rows of V
      // behind an item's start, where this warp waits long for the ring, held
      // the next chunk's codes (in half of the calls made back to back).
      uint32_t w[kPer][4];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        asm volatile("ld.volatile.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                     : "r"(src + (t + 128 * i) * 16)
                     : "memory");
      fence_proxy_async_smem();  // reads before the copies' writes
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bars->code_empty[cs]));
      if (use > 0) ok = pa_wait(smem_addr(&bars->empty[st]), (use - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int idx = t + 128 * i, k = idx / kPer, c = idx % kPer;
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) e4m3x4_to_bf16x2x2(w[i][q], o[2 * q], o[2 * q + 1]);
        const int slab = c >> 2, odd = slab & 1;
        const uint32_t row = dst + (k >> 3) * L::kGroup + slab * 1024 + (k & 7) * 128;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int half = x ^ odd, ch = 2 * (c & 3) + half;
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(row + ((ch ^ (k & 7)) << 4)),
                       "r"(half ? o[4] : o[0]), "r"(half ? o[5] : o[1]), "r"(half ? o[6] : o[2]),
                       "r"(half ? o[7] : o[3])
                       : "memory");
        }
      }
      fence_proxy_async_smem();  // the MMA (async proxy) reads them
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bars->full[st]));
    }
  }
  if (!ok) flag_error(PA_DEVERR_TIMEOUT);
}

// Warp 1: walks the CTA's items, hands each to the other warps, and loads
// its query rows into each tile as soon as the item before has done its last
// score product of that tile: the next item's scores start behind its last
// P.V product.  One 4D box per 64-column slab: 64 columns x G heads x the
// tile's tokens.  Tokens past the item are the next sequence's (or zeros
// past the batch): rows that are never stored.
template <int D, bool FP8>
__device__ __forceinline__ void pa_items(const PrefillParams& p, PaBars* bars,
                                         const CUtensorMap* tm_q, uint32_t sq,
                                         const uint32_t* sums) {
  using L = PaSmem<D, FP8>;
  PaWalk w;
  uint32_t units, parts;
  const bool work = pa_plan(p, bars, sums, w, units, parts);
  const int lane = threadIdx.x & 31;
  const uint32_t bytes = static_cast<uint32_t>(p.tok_per_tile * p.group) * D * 2;
  const bool plain = p.q_xor == 0u && p.q_and == 0xffffffffu;
  uint32_t k = 0;           // records written
  uint32_t loaded = 0, phase = 0;  // bit t: tile t has been loaded; parity of its next q_free
  uint32_t raw = 0;         // tiles that took the way over q_raw
  bool ok = true;
  auto publish = [&](const PaItem& it) {
    if (k >= kPaItems) ok = pa_wait(smem_addr(&bars->item_empty[k % kPaItems]), (k / kPaItems - 1) & 1);
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
    // the CTA that holds the item's last unit: from a lower bound upwards
    it.job = -1;
    if (!whole) {
      const uint32_t x = w.u + kPaItemCost + w.chunks;
      uint32_t c = (x - 1) / (units / parts + 1);
#pragma unroll 1
      while (c < parts - 1 && pa_share(units, parts, c + 1) < x) ++c;
      it.job = static_cast<int32_t>(c);
    }
    return it;
  };
  PaItem it = {};
  bool first = true;
  while (ok && !(it.flags & kPaEnd)) {
    // the record behind an item goes out before its queries: the copies run
    // ahead into it
    const PaItem cur = it;
    while (work && !w.done()) {
      if (!first) w.next(p);
      first = false;
      if (w.done() || w.mine) break;
    }
    if (!work || w.done())
      it.flags = kPaEnd;
    else
      it = record();
    publish(it);
    if (!ok || cur.j1 <= cur.j0) continue;  // no chunks (or nothing before): no queries
#pragma unroll 1
    for (int t = 0; t < kPaTiles; ++t) {
      if ((t == 0 ? cur.end[0] : cur.end[1]) <= cur.j0) continue;
      if (loaded >> t & 1u) {
        ok = pa_wait(smem_addr(&bars->q_free[t]), phase >> t & 1u);
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
      ok = pa_wait(bar, raw++ & 1);
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
  if (!ok) flag_error(PA_DEVERR_TIMEOUT);
  // no copy in flight at the end: on the normal path the MMAs have read all.
  // A tile's last load has the parity that its next q_free wait would have.
  if (lane == 0 && plain)
    for (int t = 0; t < kPaTiles; ++t)
      if (loaded >> t & 1u)
        pa_wait(smem_addr(&bars->q_full[t]), phase >> t & 1u, 1u << 16);
}

// Warps 2 and 3, one thread each: tile t's products.  Per chunk j of the
// tile, once the softmax has written P_j over S_j:
//     O += P_j . V_j     (P in tensor memory, V MN-major; N = D)
//     S  = Q . K_j'^T    (the tile's next chunk; both K-major; N = 128)
// in that order: one thread's MMAs run in issue order, so the new scores
// land in P_j's columns only after the product has read them, and their
// completion also means the product is done.
//
// The tensor pipe takes an MMA of this shape every 64 cycles but queues only
// one or two, and every wait on a barrier costs its thread 100 to 200: with
// one thread for both tiles the pipe ran dry for some 700 cycles between
// two tiles' 1024 (measured with time stamps).  So each tile has its own
// thread, which goes through its waits while the other issues.  While both
// tiles have chunks left the threads take turns, 16 MMAs each: interleaved,
// both tiles' MMAs would end together, and both softmaxes and then both
// products would run at the same time for good; one after the other they
// stay half a period apart.
// A turn is an arrival on the barrier that the softmax's P completes: a wait
// of its own behind that one, though long since complete, cost each chunk
// some 300 of its 3250 cycles.
//
// A stage is free once both threads have passed it; for chunks of the other
// tile (dual items, causal tiles that end earlier) this one only arrives,
// in ring order.
template <int D, bool FP8>
__device__ __forceinline__ void pa_mma(const PrefillParams& p, PaBars* bars, int t, uint32_t tmem,
                                       uint32_t sq, uint32_t ring) {
  using L = PaSmem<D, FP8>;
  constexpr uint32_t kIdQK = idesc_bf16(kPaRows, kPaChunk, false, false);
  constexpr uint32_t kIdPV = idesc_bf16(kPaRows, D, false, true);
  const bool leader = (threadIdx.x & 31) == 0;
  const uint32_t tt = tmem + t * kPaTileCols;
  // the descriptors' address field counts 16 bytes: later operands are sums
  const uint64_t qd = smem_desc_sw128(sq + t * L::kQ, 16, 1024);
  PaItems items;
  PaRing<L::kStages> r;
  uint32_t qph = 0, pph = 0, tph = 0;  // parity of the next queries, P, first turn
  bool ok = true;
  auto full = [&]() { return pa_wait(smem_addr(&bars->full[r.stage]), r.phase); };
  // the stage of a chunk that is not this tile's
  auto pass = [&]() {
    ok = ok && full();
    if (ok) mbar_arrive(smem_addr(&bars->empty[r.stage]));
    r.advance();
  };
  while (ok) {
    const PaItem* it = items.get(bars);
    if (it == nullptr) {
      ok = false;
      break;
    }
    if (it->flags & kPaEnd) break;
    if (leader && it->j1 > it->j0) {
      const int32_t j0 = it->j0, j1 = it->j1, end0 = it->end[0], end1 = it->end[1];
      const int32_t end = t == 0 ? end0 : end1;
      const bool dual = (it->flags & kPaDual) != 0;
      const int32_t step = dual ? 2 : 1;
      // turns of the item: chunks that both tiles have, if tile 0 has two
      const int32_t both = dual || end0 - j0 < 2 ? 0 : min(end0, end1) - j0;
      int32_t j = j0;
      if (dual && t == 1) {
        pass();
        pass();
        ++j;
      }
      auto scores = [&]() {  // of the chunk whose K is the next stage
        const uint64_t kd = smem_desc_sw128(ring + r.stage * L::kKV, 16, L::kGroup);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_bf16(tt + kPaSCol, qd + (((k >> 2) * (kPaRows * 128) + (k & 3) * 32) >> 4),
                    kd + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), kIdQK, k > 0);
      };
      if (j < end && ok) {
        ok = full() && pa_wait(smem_addr(&bars->q_full[t]), qph);
        qph ^= 1u;
        if (ok) {
          tc_fence_after_sync();
          scores();
          umma_commit(smem_addr(&bars->s_full[t]));
          umma_commit(smem_addr(&bars->empty[r.stage]));
          if (j + step >= end) umma_commit(smem_addr(&bars->q_free[t]));
          r.advance();
        }
      }
      for (int32_t n = 0; j < end && ok; j += step, ++n) {
        const bool more = j + step < end;
        ok = full();
        const uint32_t vst = r.stage;
        const uint64_t vd = smem_desc_sw128(ring + vst * L::kKV, 1024, L::kGroup);
        r.advance();
        if (more && !dual) ok = ok && full();
        // tile 0's turn n comes behind tile 1's n - 1, tile 1's behind tile 0's n;
        // without one the thread arrives in the other's place
        if (t == 1 && n == 0 && both > 0) {
          ok = ok && pa_wait(smem_addr(&bars->turn), tph);
          tph ^= 1u;
        }
        if (n == 0 || n >= both + (t == 0 ? 1 : 0)) mbar_arrive(smem_addr(&bars->p_full[t]));
        ok = ok && pa_wait(smem_addr(&bars->p_full[t]), pph);
        pph ^= 1u;
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int k = 0; k < kPaChunk / 16; ++k)
          umma_bf16_ta(tt + kPaOCol, tt + kPaSCol + k * 8, vd + ((k * 2 * L::kGroup) >> 4), kIdPV,
                       n > 0 || k > 0);
        if (dual) {
          // V_j goes back before the wait for K_j+2: the other tile's chunk
          // lies between them in the ring
          umma_commit(smem_addr(&bars->empty[vst]));
          if (more) {
            pass();
            pass();
            ok = ok && full();
            if (!ok) break;
            tc_fence_after_sync();
          }
        }
        if (more) scores();
        if (n < both) {
          if (t == 1) {
            if (n + 1 < end0 - j0) mbar_arrive(smem_addr(&bars->p_full[0]));
          } else {
            mbar_arrive(smem_addr(n == 0 ? &bars->turn : &bars->p_full[1]));
          }
        }
        if (more) {
          umma_commit(smem_addr(&bars->s_full[t]));
          if (j + 2 * step >= end) umma_commit(smem_addr(&bars->q_free[t]));
          if (!dual) umma_commit(smem_addr(&bars->empty[vst]));
          umma_commit(smem_addr(&bars->empty[r.stage]));
          r.advance();
        } else {
          umma_commit(smem_addr(&bars->o_last[t]));
          if (!dual) umma_commit(smem_addr(&bars->empty[vst]));
        }
      }
      // chunks behind the tile's last one
      if (dual) j -= 1;
      for (; j < j1 && ok; ++j) {
        pass();
        pass();
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok) break;
    items.put(bars);
  }
  if (!ok) flag_error(PA_DEVERR_TIMEOUT);
  // every MMA this thread issued has completed before the tensor memory is
  // released
  if (leader) {
    umma_commit(smem_addr(&bars->mma_done[t]));
    pa_wait(smem_addr(&bars->mma_done[t]), 0, 1u << 16);
  }
  __syncwarp();
}

// -------------------------------------------------------------- softmax ---
// The largest of 32 scores: three-input maxima in two chains.
__device__ __forceinline__ float pa_max32(const uint32_t (&u)[32]) {
  float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 32; i += 4)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      m[k] = fmax3(m[k], __uint_as_float(u[i + 2 * k]), __uint_as_float(u[i + 2 * k + 1]));
  return fmaxf(m[0], m[1]);
}

// The same with a factor for each 8 of them.
__device__ __forceinline__ float pa_max32(const uint32_t (&u)[32], float4 f) {
  const float g[4] = {f.x, f.y, f.z, f.w};
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float x = -INFINITY;
#pragma unroll
    for (int i = 8 * q; i < 8 * q + 8; i += 2)
      x = fmax3(x, __uint_as_float(u[i]), __uint_as_float(u[i + 1]));
    m = fmaxf(m, x * g[q]);
  }
  return m;
}

// 16 columns of an output row as bf16: a whole 32-byte sector, or two 16-byte
// stores where out is only 16-byte aligned.
__device__ __forceinline__ void pa_store16(__nv_bfloat16* dst, const uint32_t (&x)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(x[0]),
                 "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// Warps 4-11: four per tile, one row per thread (the warp's quarter of the
// tensor-memory lanes).  A chunk's weights are taken against the running
// maximum m, which need not be the true one: m starts as the maximum of the
// first chunk's first 32 scores, and while no row of the warp has weights
// that sum to more than 2^16, every weight is below 2^16, whose sums and
// products are as exact as those below 1 and far from overflow.  Otherwise
// (or when a row sees its first key) m moves to the true maximum, O and l
// are scaled, and the weights are taken again from the scores still in
// registers.  The weights are rounded to bf16 (the A operand of the P.V
// product; half a step is 2^-8 of each) and written over S; l sums them
// unrounded in fp32.
template <int D, bool FP8>
__device__ __forceinline__ void pa_softmax(const PrefillParams& p, PaBars* bars, int tile,
                                           uint32_t tmem, uint32_t ring, float2* s_ml,
                                           const float* scales) {
  using L = PaSmem<D, FP8>;
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
  const PaItem* it = items.get(bars);
  while (true) {
    if (it == nullptr) {
      ok = false;
      break;
    }
    if (it->flags & kPaEnd) break;
    const bool dual = (it->flags & kPaDual) != 0;
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
      const uint32_t chunk = cc + static_cast<uint32_t>(j - j0);
      ok = !FP8 || pa_wait(smem_addr(&bars->scale_full[chunk % L::kScales]), (chunk / L::kScales) & 1);
      ok = ok && pa_wait(smem_addr(&bars->s_full[tile]), sn++ & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      if (warp_has) {
        // Columns that some row of the warp does not see become -inf in place,
        // in a loop of its own: unrolled into the registers below it would be
        // four times the code for the few chunks that need it.
        const int32_t valid = lim - j * kPaChunk;
#pragma unroll 1
        for (int c = 3; c >= 0 && __any_sync(0xffffffffu, valid < 32 * c + 32); --c) {
          uint32_t x[32];
          tmem_ld32(tb + kPaSCol + 32 * c, x);
          tmem_wait_ld();
          const int32_t here = valid - 32 * c;
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = i < here ? x[i] : 0xff800000u;
          tmem_st32(tb + kPaSCol + 32 * c, x);
          tmem_wait_st();
        }
        uint32_t u[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tb + kPaSCol + 32 * c, u[c]);
        tmem_wait_ld();
        // FP8: the chunk's scales, one of each kind per 8 columns
        const float4* sk =
            reinterpret_cast<const float4*>(scales + (chunk % L::kScales) * kPaScaleFloats);
        auto largest = [&](int c) {  // scaled scores of columns 32 c ..
          return FP8 ? pa_max32(u[c], sk[c]) : pa_max32(u[c]) * sl;
        };
        if (j == begin) m = largest(0);
        bool move = false;  // m moves to the maximum of this chunk too
        float2 sa, sb;
#pragma unroll 1
        while (true) {
          if (move) {
            const float mn =
                fmaxf(m, fmaxf(fmaxf(largest(0), largest(1)), fmaxf(largest(2), largest(3))));
            if (j > begin) {
              // O and l scale by alpha.  O holds the products through the
              // chunk before, all complete (these scores were issued after
              // them), and this chunk's product waits for this warp's P.
              const float alpha = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
              la = mul2(la, make_float2(alpha, alpha));
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(tb + kPaOCol + 16 * c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st16(tb + kPaOCol + 16 * c, o);
              }
            }
            m = mn;
          }
          const float neg = m == -INFINITY ? 0.f : -m;  // a row that sees nothing yet
          const float2 s2 = make_float2(sl, sl), n2 = make_float2(neg, neg);
          sa = sb = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
            if (!FP8) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 x = fma2(
                    make_float2(__uint_as_float(u[c][2 * i]), __uint_as_float(u[c][2 * i + 1])),
                    s2, n2);
                const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                pk[i] = pack_bf16x2(e.x, e.y);
                if (i & 1)
                  sb = add2(sb, e);
                else
                  sa = add2(sa, e);
              }
            } else {
              const float4 fk = sk[c], fl = sk[4 + c], fi = sk[8 + c];
              const float gk[4] = {fk.x, fk.y, fk.z, fk.w}, gl[4] = {fl.x, fl.y, fl.z, fl.w},
                          gi[4] = {fi.x, fi.y, fi.z, fi.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float2 a2 = make_float2(gk[q], gk[q]);
                const float2 b2 = make_float2(neg + gl[q], neg + gl[q]);
                float2 part;  // of the weights times v
#pragma unroll
                for (int i = 4 * q; i < 4 * q + 4; ++i) {
                  const float2 x = fma2(
                      make_float2(__uint_as_float(u[c][2 * i]), __uint_as_float(u[c][2 * i + 1])),
                      a2, b2);
                  const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                  pk[i] = pack_bf16x2(e.x, e.y);
                  part = i == 4 * q ? e : add2(part, e);
                }
                if (q & 1)
                  sb = fma2(part, make_float2(gi[q], gi[q]), sb);
                else
                  sa = fma2(part, make_float2(gi[q], gi[q]), sa);
              }
            }
            tmem_st16(tb + kPaSCol + 16 * c, pk);
          }
          const float sum = (sa.x + sa.y) + (sb.x + sb.y);
          // Rows without a token have no say: behind the last token of a
          // group that does not divide 128 the tile holds earlier contents.
          if (move || !__any_sync(0xffffffffu, has && (sum > 65536.f || m == -INFINITY)))
            break;
          move = true;
        }
        la = add2(la, add2(sa, sb));
      }
      // The last chunk's tokens past the sequence hold whatever their block
      // held before: their weights are 0, and so must their V be (0 * NaN).
      // The tile clears those rows before its product; when both tiles use
      // the chunk both do, with the same zeros.
      const int32_t past = n - j * kPaChunk;  // valid tokens of the chunk
      if (past < kPaChunk) {
        const uint32_t slot = 2 * chunk + 1;
        ok = pa_wait(smem_addr(&bars->full[slot % L::kStages]), (slot / L::kStages) & 1);
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
    const PaItem* next = ok ? items.get(bars, 1) : nullptr;  // there already as a rule
    if (end > begin && ok) {
      ok = pa_wait(smem_addr(&bars->o_last[tile]), on++ & 1);
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
        ok = pa_wait(smem_addr(&bars->o_free), dn++ & 1);
        ok = __all_sync(0xffffffffu, ok);
        items.put(bars);
        it = ok ? next : nullptr;
        continue;
      }
      ok = pa_wait(smem_addr(&bars->ml_full), dn++ & 1);
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
      __nv_bfloat16* to =
          p.out + (static_cast<int64_t>(it->row + tk) * p.num_q_heads + it->h * p.group +
                   (r - rt * p.group)) * D;
      if (!whole && has) p.ws_ml[slot * kPaItemRows + row] = make_float2(m, l);
      // The rows of a lane pair are stored by both its lanes, 32 bytes each:
      // half as many lines per instruction as a row per lane.
      const bool odd = lane & 1;
      const uint64_t mine = has ? reinterpret_cast<uint64_t>(to) : 0;
      const uint64_t theirs = __shfl_xor_sync(0xffffffffu, mine, 1);
      __nv_bfloat16* pair[2] = {reinterpret_cast<__nv_bfloat16*>(odd ? theirs : mine),
                                reinterpret_cast<__nv_bfloat16*>(odd ? mine : theirs)};
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        w0 *= inv;
        w1 *= inv;
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        float x[32];
        if (__any_sync(0xffffffffu, l != 0.f)) {
          tmem_ld32(tb + kPaOCol + 32 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]) * w0;
          if (dual) {
            tmem_ld32(tb + kPaTileCols + kPaOCol + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              x[i] = fmaf(__uint_as_float(o[i]), w1, x[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.f;
        }
        if (l == 0.f) {  // a row that saw nothing: zeros, whatever V holds
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.f;
        }
        if (!whole) {
          if (has) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              po[(8 * c + i) * kPaItemRows] =
                  make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        } else {
          // even lanes take the first half of both rows' 32 columns
          uint32_t y[2][8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t lo = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            const uint32_t hi = pack_bf16x2(x[16 + 2 * i], x[16 + 2 * i + 1]);
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
            y[0][i] = odd ? got : lo;
            y[1][i] = odd ? hi : got;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (pair[k] != nullptr) pa_store16(pair[k] + 32 * c + (odd ? 16 : 0), y[k], wide);
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
    it = next;
  }
  if (!ok) flag_error(PA_DEVERR_TIMEOUT);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(PaRegs<FP8>::kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_q, const PrefillParams p) {
  using L = PaSmem<D, FP8>;
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
      mbar_init(smem_addr(&bars->full[i]), FP8 ? 4 : 1);
      mbar_init(smem_addr(&bars->empty[i]), kPaTiles);
    }
    for (int i = 0; i < kPaMaxCodeStages && FP8; ++i) {
      mbar_init(smem_addr(&bars->code_full[i]), 1);
      mbar_init(smem_addr(&bars->code_empty[i]), 4);
      mbar_init(smem_addr(&bars->scale_full[i]), 1);
    }
    for (int t = 0; t < kPaTiles; ++t) {
      mbar_init(smem_addr(&bars->q_full[t]), 1);
      mbar_init(smem_addr(&bars->q_free[t]), 1);
      mbar_init(smem_addr(&bars->s_full[t]), 1);
      mbar_init(smem_addr(&bars->p_full[t]), 5);
      mbar_init(smem_addr(&bars->o_last[t]), 1);
      mbar_init(smem_addr(&bars->mma_done[t]), 1);
    }
    for (int i = 0; i < kPaItems; ++i) {
      mbar_init(smem_addr(&bars->item_full[i]), 1);
      mbar_init(smem_addr(&bars->item_empty[i]), 1 + kPaTiles * 5 + (FP8 ? 4 : 0));
    }
    mbar_init(smem_addr(&bars->q_raw), 1);
    mbar_init(smem_addr(&bars->turn), 1);
    mbar_init(smem_addr(&bars->ml_full), 4);
    mbar_init(smem_addr(&bars->o_free), 4);
    bars->bad = 0;
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

  if (threadIdx.x == 32 * kPaSoftWarp) p.ws_job[blockIdx.x] = make_int4(0, 0, 0, 0);
  // the threads' units, where the ring will be: the copies start behind the
  // first item's record, which warp 1 writes after it has read them
  uint32_t* sums = reinterpret_cast<uint32_t*>(pa_smem + L::kOffRing);
  if (p.num_seqs > 32) {
    if (!FP8 || threadIdx.x < kPaThreads) sums[threadIdx.x] = pa_thread_units(p, bars);
    fence_proxy_async_smem();
    __syncthreads();
  }
  using R = PaRegs<FP8>;
  float* scales = reinterpret_cast<float*>(pa_smem + L::kOffScale);
  if (warp < kPaSoftWarp) {
    regs_dec<R::kFew>();
    if (warp == 0)
      pa_copies<D, FP8>(p, bars, &tm_k, &tm_v, FP8 ? base + L::kOffCodes : ring, scales);
    else if (warp == 1)
      pa_items<D, FP8>(p, bars, &tm_q, sq, sums);
    else
      pa_mma<D, FP8>(p, bars, warp - 2, tmem, sq, ring);
  } else if (!FP8 || warp < kPaConvWarp) {
    regs_inc<R::kSoft>();
    pa_softmax<D, FP8>(p, bars, (warp - kPaSoftWarp) >> 2, tmem, ring,
                       reinterpret_cast<float2*>(pa_smem + L::kOffMl), scales);
  } else {
    if constexpr (FP8) {
      regs_dec<R::kConv>();
      pa_widen<D>(bars, base + L::kOffCodes, ring);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kPaTmemCols);
  }
}

// Folds the pieces of each item that a range boundary cut: M = max m_i,
// out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i (0 without any key), as a
// running sum over the pieces.  Block (c, part): 32 rows of the item whose
// head piece CTA c holds; lane = row, so every load of a piece's [D / 4][256]
// float4 is coalesced; warp w has columns 16 w ..  Bound by latency (few
// pieces, read from L2): the loads of two pieces, the usual number, are all
// in flight together.  4 to 5 us behind the main launch, for up to 151 cut
// items of 64 tokens.
template <int D>
__global__ void __launch_bounds__(2 * D) prefill_merge_kernel(const PrefillParams p) {
  pdl_wait();
  pdl_trigger();
  const int32_t c = blockIdx.x;
  const int4 job = p.ws_job[c];
  const int row = blockIdx.y * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
  const int32_t r = row & (kPaRows - 1), rt = static_cast<int32_t>(pa_div(p, r));
  const int32_t tk = rt + (row >= kPaRows ? p.tok_per_tile : 0);
  if (rt >= p.tok_per_tile || tk >= job.w || job.x >= p.num_ctas) return;
  constexpr int kBatch = 2;
  float M = -INFINITY, l = 0.f;
  float acc[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.f;
  for (int32_t i0 = c; i0 <= job.x; i0 += kBatch) {
    float2 ml[kBatch];
    float4 x[kBatch][4];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + i <= job.x) {
        const int64_t s = 2 * static_cast<int64_t>(i0 + i) + (i0 + i == c ? 1 : 0);
        ml[i] = p.ws_ml[s * kPaItemRows + row];
        const float4* po = reinterpret_cast<const float4*>(p.ws_o) +
                           (s * (D / 4) + 4 * warp) * kPaItemRows + row;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i][k] = po[k * kPaItemRows];
      }
    }
    float mn = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) mn = fmaxf(mn, ml[i].x);
    if (mn == -INFINITY) {  // no piece so far has a key for the row (or all its scores are NaN)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) l += ml[i].y;
      continue;
    }
    const float w0 = fast_exp2(M - mn);
    M = mn;
    l *= w0;
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] *= w0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // a piece that the row sees nothing of weighs 0
      const float wgt = ml[i].x == -INFINITY ? 0.f : fast_exp2(ml[i].x - mn);
      l = fmaf(wgt, ml[i].y, l);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[4 * k] = fmaf(wgt, x[i][k].x, acc[4 * k]);
        acc[4 * k + 1] = fmaf(wgt, x[i][k].y, acc[4 * k + 1]);
        acc[4 * k + 2] = fmaf(wgt, x[i][k].z, acc[4 * k + 2]);
        acc[4 * k + 3] = fmaf(wgt, x[i][k].w, acc[4 * k + 3]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t orow = static_cast<int64_t>(job.y + tk) * p.num_q_heads + job.z * p.group +
                       (r - rt * p.group);
  uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + 16 * warp);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 o;
    o.x = pack_bf16x2(acc[8 * h] * inv, acc[8 * h + 1] * inv);
    o.y = pack_bf16x2(acc[8 * h + 2] * inv, acc[8 * h + 3] * inv);
    o.z = pack_bf16x2(acc[8 * h + 4] * inv, acc[8 * h + 5] * inv);
    o.w = pack_bf16x2(acc[8 * h + 6] * inv, acc[8 * h + 7] * inv);
    dst[h] = o;
  }
}

}  // namespace pa
