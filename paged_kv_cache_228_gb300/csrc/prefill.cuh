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
// one product are (token, head of the group): row r of a sequence is token
// r / G, head r % G.  An item is TT = 256 / G tokens (<= 256 rows, two
// M = 128 tiles) of one sequence and KV head over the 128-token chunks its
// last row sees: with G = 4 the causal limit moves over only 64 tokens
// within an item, so at most one of its chunks is partly masked per tile.
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
  int4* ws_job;              // [P] {last CTA, first token, KV head, rows}
  int32_t num_seqs, num_tokens, num_q_heads, num_kv_heads, group, tok_per_item;
  int32_t block_size, log2_bs, max_blocks, num_blocks;
  int32_t groups_total;      // 8-row groups of the pool (one past the last: reads zeros)
  int32_t num_ctas;
  int32_t causal;
  uint32_t q_and, q_xor;     // applied to the query words: negation, or zero
  float sl;                  // |scale| * log2(e), > 0
};

constexpr int kPaRows = 128;           // rows per tile (the MMA's M)
constexpr int kPaTiles = 2;
constexpr int kPaItemRows = kPaRows * kPaTiles;
constexpr int kPaChunk = 128;          // tokens per chunk
constexpr int kPaSoftWarps = 4 * kPaTiles;
constexpr int kPaThreads = 96 + 32 * kPaSoftWarps;  // K and V producers, MMA, softmax
constexpr int kPaVWarp = 2 + kPaSoftWarps;
constexpr int kPaItemCost = 1;         // units charged per item besides its chunks
constexpr int kPaTileCols = 256;       // tensor memory per tile: S / P (128), O (D)
constexpr int kPaSCol = 0;
constexpr int kPaOCol = 128;
constexpr int kPaTmemCols = 512;

template <int D>
struct PaSmem {
  static constexpr int kKV = kPaChunk * D * 2;  // K (or V) of a chunk
  static constexpr int kKStages = D == 64 ? 5 : 3;
  static constexpr int kVStages = D == 64 ? 4 : 2;
  static constexpr int kQ = kPaRows * D * 2;    // one query tile
  static constexpr int kOffK = kPaTiles * kQ;
  static constexpr int kOffV = kOffK + kKStages * kKV;
  static constexpr int kOffBar = kOffV + kVStages * kKV;
  static constexpr int kBytes = kOffBar + 512;
  static constexpr int kGroup = D * 16;         // 8 tokens: D / 64 slabs of 8 x 128 bytes
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct PaBars {
  uint64_t k_full[5], k_empty[5], v_full[4], v_empty[4];
  uint64_t q_full[kPaTiles];  // the item's query tile stored
  uint64_t s_full[kPaTiles];  // S of the tile's chunk written (and its last product done)
  uint64_t p_full[kPaTiles];  // P of the tile's chunk written
  uint64_t o_last[kPaTiles];  // the tile's last product of the item done
  uint64_t mma_done;
  int64_t scan[kPaThreads / 32];
  int64_t first_u;            // the CTA's first sequence: units before it
  int32_t first_b;
  int32_t bad;
  uint32_t tmem;
};
static_assert(sizeof(PaBars) <= 512, "barrier block");

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
  int32_t tok, rows, lim, chunks;  // first token, rows, tokens seen, chunks
  int32_t j0, j1;                  // this CTA's chunks
  bool mine;                       // this CTA has something to do in it

  __device__ __forceinline__ void item(const PrefillParams& p) {
    tok = i * p.tok_per_item;
    const int32_t nt = min(p.tok_per_item, s.nq - tok);
    rows = nt * p.group;
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
  // chunks [j0, end) of tile t: its last row sees no further
  __device__ __forceinline__ int32_t tile_end(const PrefillParams& p, int t) const {
    if (t * kPaRows >= rows) return j0;
    if (t == 1 || rows <= kPaRows) return j1;
    const int32_t c = pa_chunks(pa_limit(p, s, tok + (kPaRows - 1) / p.group + 1));
    return max(j0, min(j1, c));
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
  for (int i = 0; i < kPaThreads / 32; ++i) {
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
__device__ __forceinline__ int32_t pa_block_id(const PrefillParams& p, const PaWalk& w,
                                               int32_t ch) {
  const int lane = threadIdx.x & 31;
  const int box = p.block_size < kPaChunk ? p.block_size : kPaChunk;
  const int32_t tok = ch * kPaChunk + lane * box;
  if (lane >= kPaChunk / box || tok >= w.s.n) return -1;
  return p.block_tables[static_cast<int64_t>(w.b) * p.max_blocks + (tok >> p.log2_bs)];
}

// Whole warp: chunk ch's K (or V) rows into one ring stage, one 4D box per
// block by lane i: 8-token groups of D / 64 slabs of 8 x 128 bytes, so that
// a single copy carries the block's whole width and successive groups stay
// one stride apart for the matrix descriptors.  Blocks past the sequence,
// or with an id outside the pool, read past the tensor: zeros.
template <int D>
__device__ __forceinline__ void pa_copy_chunk(const PrefillParams& p, const CUtensorMap* map,
                                              const PaWalk& w, int32_t ch, int32_t blk,
                                              uint32_t dst, uint32_t bar) {
  const int lane = threadIdx.x & 31;
  const int box = p.block_size < kPaChunk ? p.block_size : kPaChunk;
  if (lane == 0) mbar_arrive_expect_tx(bar, PaSmem<D>::kKV);
  __syncwarp();
  if (lane < kPaChunk / box) {
    const int32_t tok = ch * kPaChunk + lane * box;
    int32_t grp = p.groups_total;
    if (tok < w.s.n) {
      if (blk >= 0 && blk < p.num_blocks)
        grp = (blk * p.num_kv_heads + w.h) * (p.block_size >> 3) +
              ((tok & (p.block_size - 1)) >> 3);
      else
        flag_error(PA_DEVERR_BAD_BLOCK_ID);
    }
    tma_load_4d(dst + lane * box * D * 2, map, 0, 0, 0, grp, bar);
  }
}

// -------------------------------------------------------------- softmax ---
// The largest of a thread's 128 raw scores; kMask: columns from `valid` on
// become -inf.
template <bool kMask>
__device__ __forceinline__ float pa_row_max(uint32_t (&u)[kPaChunk], int32_t valid) {
  if (kMask) {
#pragma unroll
    for (int i = 0; i < kPaChunk; ++i) u[i] = i < valid ? u[i] : 0xff800000u;
  }
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < kPaChunk; i += 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m[k] = fmax3(m[k], __uint_as_float(u[i + 2 * k]), __uint_as_float(u[i + 2 * k + 1]));
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

template <int D>
__global__ void __launch_bounds__(kPaThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const PrefillParams p) {
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
  const uint32_t sq = base, sk = base + L::kOffK, sv = base + L::kOffV;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kKStages; ++i) {
      mbar_init(smem_addr(&bars->k_full[i]), 1);
      mbar_init(smem_addr(&bars->k_empty[i]), 1);
    }
    for (int i = 0; i < L::kVStages; ++i) {
      mbar_init(smem_addr(&bars->v_full[i]), 1);
      mbar_init(smem_addr(&bars->v_empty[i]), 1);
    }
    for (int t = 0; t < kPaTiles; ++t) {
      mbar_init(smem_addr(&bars->q_full[t]), 4);
      mbar_init(smem_addr(&bars->s_full[t]), 1);
      mbar_init(smem_addr(&bars->p_full[t]), 4);
      mbar_init(smem_addr(&bars->o_last[t]), 1);
    }
    mbar_init(smem_addr(&bars->mma_done), 1);
    mbar_fence_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
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
  bool ok = true;
  if (threadIdx.x == 64) p.ws_job[blockIdx.x] = make_int4(0, 0, 0, 0);

  if (!work) {
    // nothing in this CTA's range
  } else if (warp == 0 || warp == kPaVWarp) {
    // ----------------------------------------- producers: K (0), V (10) ---
    const bool is_k = warp == 0;
    const uint32_t S = is_k ? L::kKStages : L::kVStages;
    const CUtensorMap* map = is_k ? &tm_k : &tm_v;
    const uint32_t ring = is_k ? sk : sv;
    uint64_t* full = is_k ? bars->k_full : bars->v_full;
    uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
    uint32_t c = 0;  // chunks issued
    for (; !w.done() && ok; w.next(p)) {
      if (w.j1 <= w.j0) continue;
      int32_t e = pa_block_id(p, w, w.j0);
      for (int32_t j = w.j0; j < w.j1; ++j) {
        const int32_t en = j + 1 < w.j1 ? pa_block_id(p, w, j + 1) : -1;
        const uint32_t st = c % S;
        if (lane == 0 && c >= S) ok = mbar_wait(smem_addr(&empty[st]), ((c / S) - 1) & 1);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        pa_copy_chunk<D>(p, map, w, j, e, ring + st * L::kKV, smem_addr(&full[st]));
        ++c;
        e = en;
      }
    }
    // No copy may still target shared memory when the CTA exits: on the
    // normal path the MMAs have consumed every one already.
    if (lane == 0)
      for (uint32_t j = c > S ? c - S : 0; j < c; ++j)
        mbar_wait(smem_addr(&full[j % S]), (j / S) & 1, 1u << 16);
  } else if (warp == 1) {
    // ---------------------------------------------------- MMA issuer ---
    if (lane == 0) {
      constexpr uint32_t kIdQK = idesc_bf16(kPaRows, kPaChunk, false, false);
      constexpr uint32_t kIdPV = idesc_bf16(kPaRows, D, false, true);
      // S_t = Q_t . K^T of the chunk whose K sits at kb
      auto qk = [&](int t, uint32_t kb) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_bf16(tmem + t * kPaTileCols + kPaSCol,
                    smem_desc_sw128(sq + t * L::kQ + (k >> 2) * (kPaRows * 128) + (k & 3) * 32, 16,
                                    1024),
                    smem_desc_sw128(kb + (k >> 2) * 1024 + (k & 3) * 32, 16, L::kGroup), kIdQK,
                    k > 0);
        umma_commit(smem_addr(&bars->s_full[t]));
      };
      uint32_t kc = 0, vc = 0;            // K and V chunks consumed
      uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};  // query tiles, P tiles consumed
      for (; !w.done() && ok; w.next(p)) {
        if (w.j1 <= w.j0) continue;
        const int32_t end[2] = {w.tile_end(p, 0), w.tile_end(p, 1)};
        ok = mbar_wait(smem_addr(&bars->k_full[kc % L::kKStages]), (kc / L::kKStages) & 1);
        for (int t = 0; t < kPaTiles && ok; ++t) {
          if (end[t] <= w.j0) continue;
          ok = mbar_wait(smem_addr(&bars->q_full[t]), qn[t]++ & 1);
          if (!ok) break;
          tc_fence_after_sync();
          qk(t, sk + (kc % L::kKStages) * L::kKV);
        }
        umma_commit(smem_addr(&bars->k_empty[kc % L::kKStages]));
        ++kc;
        for (int32_t j = w.j0; j < w.j1 && ok; ++j) {
          const bool more = j + 1 < w.j1;
          const uint32_t vs = vc % L::kVStages, ks = kc % L::kKStages;
          const uint32_t vb = sv + vs * L::kKV, kb = sk + ks * L::kKV;
          ok = mbar_wait(smem_addr(&bars->v_full[vs]), (vc / L::kVStages) & 1);
          if (ok && more) ok = mbar_wait(smem_addr(&bars->k_full[ks]), (kc / L::kKStages) & 1);
          for (int t = 0; t < kPaTiles && ok; ++t) {
            if (j >= end[t]) continue;
            // P_t of chunk j written (over S_t); then its product and the
            // scores of chunk j + 1, in that order
            ok = mbar_wait(smem_addr(&bars->p_full[t]), pn[t]++ & 1);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t tt = tmem + t * kPaTileCols;
#pragma unroll
            for (int k = 0; k < kPaChunk / 16; ++k)
              umma_bf16_ta(tt + kPaOCol, tt + kPaSCol + k * 8,
                           smem_desc_sw128(vb + k * 2 * L::kGroup, 1024, L::kGroup), kIdPV,
                           j > w.j0 || k > 0);
            if (j + 1 < end[t])
              qk(t, kb);
            else
              umma_commit(smem_addr(&bars->o_last[t]));
          }
          if (!ok) break;
          umma_commit(smem_addr(&bars->v_empty[vs]));
          ++vc;
          if (more) {
            umma_commit(smem_addr(&bars->k_empty[ks]));
            ++kc;
          }
        }
      }
      // every MMA this thread issued has completed before the tensor
      // memory is released
      umma_commit(smem_addr(&bars->mma_done));
      mbar_wait(smem_addr(&bars->mma_done), 0, 1u << 16);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------- softmax ---
    const int tile = (warp - 2) >> 2;
    const int quarter = warp & 3;         // tensor-memory lanes 32 * quarter ...
    const int r = 32 * quarter + lane;    // row within the tile
    const int tid = (threadIdx.x - 64) & 127;
    const int row = tile * kPaRows + r;   // row within the item
    const uint32_t tb =
        tmem + (static_cast<uint32_t>(32 * quarter) << 16) + tile * kPaTileCols;
    const uint32_t sqt = sq + tile * L::kQ;
    const float sl = p.sl;
    const uint32_t G = static_cast<uint32_t>(p.group);
    uint32_t sn = 0, on = 0, vc = 0;  // S tiles and items of this tile, V chunks of the CTA
    constexpr int kCpr = D * 2 / 16;  // 16-byte chunks per row
    auto tile_sync = [&]() {
      if (tile == 0)
        named_bar_sync<1>(128);
      else
        named_bar_sync<2>(128);
    };
    // q / out row of item row x
    auto token_row = [&](uint32_t x) -> int64_t {
      const uint32_t tk = x / G;
      return static_cast<int64_t>(w.s.q0 + w.tok + static_cast<int32_t>(tk)) * p.num_q_heads +
             w.h * p.group + (x - tk * G);
    };
    for (; !w.done() && ok; w.next(p)) {
      if (!w.mine) continue;
      const int32_t end = w.tile_end(p, tile);
      const bool whole = w.j0 == 0 && w.j1 == w.chunks;
      float m = -INFINITY, l = 0.f;
      if (end > w.j0) {
        // the tile's rows (zeros past the item), then the MMA may read them
        uint4 v[kCpr];
#pragma unroll
        for (int i = 0; i < kCpr; ++i) {
          const int idx = tid + 128 * i, x = tile * kPaRows + idx / kCpr, c = idx % kCpr;
          v[i] = make_uint4(0u, 0u, 0u, 0u);
          if (x < w.rows)
            v[i] = *reinterpret_cast<const uint4*>(p.q + token_row(x) * (D * 2) + c * 16);
        }
#pragma unroll
        for (int i = 0; i < kCpr; ++i) {
          const int idx = tid + 128 * i;
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                           sqt + pa_q_chunk(idx / kCpr, idx % kCpr)),
                       "r"((v[i].x & p.q_and) ^ p.q_xor), "r"((v[i].y & p.q_and) ^ p.q_xor),
                       "r"((v[i].z & p.q_and) ^ p.q_xor), "r"((v[i].w & p.q_and) ^ p.q_xor)
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&bars->q_full[tile]));

        // tokens this row sees
        const int32_t lim =
            !p.causal || row >= w.rows ? w.lim : w.s.off + w.tok + row / p.group + 1;
        float2 l2 = make_float2(0.f, 0.f);
        for (int32_t j = w.j0; j < end; ++j) {
          ok = mbar_wait(smem_addr(&bars->s_full[tile]), sn++ & 1);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          uint32_t u[kPaChunk];
#pragma unroll
          for (int c = 0; c < kPaChunk / 32; ++c)
            tmem_ld32(tb + kPaSCol + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&u[32 * c]));
          tmem_wait_ld();
          const int32_t valid = lim - j * kPaChunk;
          float mx = __any_sync(0xffffffffu, valid < kPaChunk) ? pa_row_max<true>(u, valid)
                                                                : pa_row_max<false>(u, valid);
          mx *= sl;
          if (j == w.j0) {
            m = mx;
          } else if (__any_sync(0xffffffffu, mx > m + 8.f)) {
            // the running max moves: O and l scale by alpha.  O holds the
            // products through chunk j - 1, all complete (the scores of
            // chunk j were issued after them), and the product of chunk j
            // waits for this warp's P.
            const float mn = fmaxf(m, mx);
            const float alpha = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
            m = mn;
            l2.x *= alpha;
            l2.y *= alpha;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tb + kPaOCol + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tb + kPaOCol + 32 * c, o);
            }
          }
          const float neg = m == -INFINITY ? 0.f : -m;  // a row that sees nothing yet
          const float2 s2 = make_float2(sl, sl), n2 = make_float2(neg, neg);
#pragma unroll
          for (int c = 0; c < kPaChunk / 32; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int k = 32 * c + 2 * i;
              const float2 x =
                  fma2(make_float2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])), s2, n2);
              const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              pk[i] = pack_bf16x2(e.x, e.y);
              l2 = add2(l2, e);
            }
            tmem_st16(tb + kPaSCol + 16 * c, pk);
          }
          // The last chunk's tokens past the sequence hold whatever their
          // block held before: their weights are 0, and so must their V be
          // (0 * NaN).  The first active tile clears those rows before its
          // product, which the MMA issues before the other tile's.
          const int32_t past = w.s.n - j * kPaChunk;  // valid tokens of the chunk
          if (past < kPaChunk && (tile == 0 || w.tile_end(p, 0) <= j)) {
            const uint32_t vi = vc + static_cast<uint32_t>(j - w.j0);
            ok = mbar_wait(smem_addr(&bars->v_full[vi % L::kVStages]), (vi / L::kVStages) & 1);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            const int32_t stop =
                min(kPaChunk, ((past + p.block_size - 1) >> p.log2_bs) << p.log2_bs);
            const uint32_t vb = sv + (vi % L::kVStages) * L::kKV;
            for (int32_t idx = past * kCpr + tid; idx < stop * kCpr; idx += 128) {
              const int32_t tk = idx / kCpr, c = idx % kCpr;  // swizzle keeps a row in its row
              asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                               vb + (tk >> 3) * L::kGroup + (c >> 3) * 1024 + (tk & 7) * 128 +
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
        l = l2.x + l2.y;
        if (ok) {
          ok = mbar_wait(smem_addr(&bars->o_last[tile]), on++ & 1);
          ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok) break;
        tc_fence_after_sync();
      }
      vc += static_cast<uint32_t>(w.j1 - w.j0);
      if (tile * kPaRows >= w.rows) continue;
      if (whole) {
        // out = O / l, staged where the tile's queries were (every score
        // product of the item is done), then whole rows to memory
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (end > w.j0) {
            tmem_ld32(tb + kPaOCol + 32 * c, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = l == 0.f ? 0u
                              : pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv,
                                            __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                             sqt + pa_q_chunk(r, 4 * c + i)),
                         "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                         : "memory");
          }
        }
        tile_sync();
#pragma unroll
        for (int i = 0; i < kCpr; ++i) {
          const int idx = tid + 128 * i, x = tile * kPaRows + idx / kCpr, c = idx % kCpr;
          uint4 o;
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                       : "r"(sqt + pa_q_chunk(idx / kCpr, c))
                       : "memory");
          if (x < w.rows)
            reinterpret_cast<uint4*>(p.out + token_row(x) * D)[c] = o;
        }
        tile_sync();  // read out before the next item's queries land there
      } else {
        // a piece: the head of an item in slot 1 of this CTA, a later piece
        // in slot 0 (it is then the CTA's first item)
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (w.j0 == 0 ? 1 : 0);
        float4* po = reinterpret_cast<float4*>(p.ws_o) + slot * (D / 4) * kPaItemRows + row;
        if (row < w.rows) p.ws_ml[slot * kPaItemRows + row] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (end > w.j0) {
            tmem_ld32(tb + kPaOCol + 32 * c, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          if (row < w.rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              po[(8 * c + i) * kPaItemRows] =
                  make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                              __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          }
        }
        if (threadIdx.x == 64 && w.j0 == 0) {
          // the CTA that holds the item's last unit
          const int64_t x = w.u + kPaItemCost + w.chunks;
          p.ws_job[blockIdx.x] = make_int4(static_cast<int32_t>((x * parts - 1) / units),
                                           w.s.q0 + w.tok, w.h, w.rows);
        }
        tile_sync();  // both kinds of item leave the tile's warps together
      }
      tc_fence_before_sync();
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
  if (row >= job.w || job.x >= p.num_ctas) return;
  auto slot = [&](int32_t i) -> int64_t { return 2 * static_cast<int64_t>(i) + (i == c ? 1 : 0); };
  float M = -INFINITY;
  for (int32_t i = c; i <= job.x; ++i) M = fmaxf(M, p.ws_ml[slot(i) * kPaItemRows + row].x);
  const uint32_t tk = static_cast<uint32_t>(row) / static_cast<uint32_t>(p.group);
  const int64_t orow = static_cast<int64_t>(job.y + static_cast<int32_t>(tk)) * p.num_q_heads +
                       job.z * p.group + (row - tk * p.group);
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
