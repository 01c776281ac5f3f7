// Block tables and slot maps built on the GPU from request lengths.
//
// "Paged Attention and KV Cache Fragmentation", section "How PagedAttention
// maps an OS concept onto GPU memory": blocks are allocated only as a
// sequence grows and freed when it finishes.  The free list is a stack in
// device memory; a step that grows or shrinks every sequence of a batch
// needs no host round trip.  With have_b = ceil(len_b / bs) and need_b the
// blocks the new tokens cross into, the stack positions are an exclusive sum
// over the batch,
//     id of sequence b's j-th new block = free_ids[F - 1 - base_b - j],
//     base_b = sum of need over the sequences before b,
// the order in which the host manager's LIFO list hands blocks out; a trim
// pushes at F + base_b + j.
//
// Latency-bound: each CTA walks the batch 1024 sequences at a time, one per
// thread, keeps their records in shared memory, and then one thread per
// token (or released block) finds its sequence by binary search there, four
// at a time so that their table loads are in flight together.  A decode
// step's few tokens take one CTA; long slot maps take a grid, every CTA
// redoing the scan, unless the call updates its inputs in place: then a
// cluster of 8, whose CTAs all read num_free and a tile's lengths before a
// cluster barrier and rank 0 writes them after it.  Neither kernel lets its
// dependents start early (a decode kernel reads seq_lens before it waits for
// its predecessor), and each thread's writes are performed before it exits.
//
// Measured inside a captured graph: 256 sequences that grow by one token
// 4.3 us, a map of 58 thousand slots 4.6 us (11.3 with one token a thread in a
// cluster), 256 finished sequences 5.8 us, 1500 that give back up to 8 tokens
// 6.5 us (7.0 before a tile's lengths were loaded ahead).  A launch with
// nothing to do is some 2 us of each; the bytes (0.5 MB at most) are nothing.
#pragma once

#include <cooperative_groups.h>

#include "pa_device.cuh"

namespace pa {

constexpr int kSlThreads = 1024;
constexpr int kSlWarps = kSlThreads / 32;
constexpr int kSlCluster = 8;
constexpr int kSlGrid = 0;  // CTAs without a cluster: outputs apart from the inputs
constexpr int kSlBatch = 4;

struct SlotParams {
  const int32_t* lens;
  const int32_t* change;      // append: new tokens; trim: new lengths
  int32_t* tables;            // [num_seqs][max_blocks] (trim: only read)
  int32_t* free_ids;          // [num_blocks] (append: only read)
  const int32_t* num_free;
  int64_t* slots;             // append: [num_tokens]
  int32_t* q_start;           // append: [num_seqs + 1]
  int32_t* seq_lens;
  int32_t* num_free_out;
  int32_t* num_done;          // append
  int32_t num_seqs, num_tokens, max_blocks, block_size, num_blocks;
};

struct SlotScan {
  int64_t warp_a[kSlWarps], warp_b[kSlWarps];
  int32_t first_fail;
  int32_t redo;
};

// Inclusive sums of a and b over the block's threads; the block's totals in
// (ta, tb).  Begins and ends with a barrier between uses of `s`.
__device__ __forceinline__ void slot_scan(SlotScan& s, int64_t& a, int64_t& b, int64_t& ta,
                                          int64_t& tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d);
    if (lane >= d) {
      a += x;
      b += y;
    }
  }
  __syncthreads();
  if (lane == 31) {
    s.warp_a[warp] = a;
    s.warp_b[warp] = b;
  }
  __syncthreads();
  // every warp sums the warps' totals itself: lane i holds warp i's
  int64_t x = s.warp_a[lane], y = s.warp_b[lane];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) {
      x += u;
      y += v;
    }
  }
  ta = __shfl_sync(0xffffffffu, x, 31);
  tb = __shfl_sync(0xffffffffu, y, 31);
  const int64_t pa = __shfl_sync(0xffffffffu, x, warp > 0 ? warp - 1 : 0);
  const int64_t pb = __shfl_sync(0xffffffffu, y, warp > 0 ? warp - 1 : 0);
  if (warp > 0) {
    a += pa;
    b += pb;
  }
}

template <int kC>
__device__ __forceinline__ void slot_barrier() {
  if (kC == kSlCluster)
    cooperative_groups::this_cluster().sync();
  else
    __syncthreads();
}

// Index of the last of `n` ascending starts that is <= x (start[0] <= x).
__device__ __forceinline__ int slot_find(const int32_t* start, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int kC>
__global__ void __launch_bounds__(kSlThreads) append_slots_kernel(const SlotParams p) {
  __shared__ SlotScan scan;
  __shared__ int32_t s_tok[kSlThreads], s_len[kSlThreads], s_base[kSlThreads];
  const int tid = threadIdx.x;
  const int rank = kC == 1 ? 0 : static_cast<int>(blockIdx.x);
  const int64_t threads = static_cast<int64_t>(kC == 1 ? 1 : gridDim.x) * kSlThreads;
  pdl_wait();
  int32_t F = *p.num_free;
  if (F < 0 || F > p.num_blocks) {
    if (rank == 0 && tid == 0) flag_error(PA_DEVERR_BAD_BLOCK_ID);
    F = F < 0 ? 0 : p.num_blocks;
  }
  const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.block_size;
  int64_t taken = 0, tokens = 0;  // blocks and tokens of the sequences before the tile
  int32_t stop = p.num_seqs;      // the first sequence that fails
  bool stopped = false;
  for (int32_t b0 = 0; b0 < p.num_seqs; b0 += kSlThreads) {
    const int32_t b = b0 + tid;
    const bool in = b < p.num_seqs;
    const int32_t count = min(kSlThreads, p.num_seqs - b0);
    int32_t len = in ? p.lens[b] : 0, n = in ? p.change[b] : 0;
    uint32_t err = 0;
    if (len < 0 || n < 0 || static_cast<int64_t>(len) + n > cap) err = PA_DEVERR_BAD_SEQ_LEN;
    const int64_t grow = n > 0 ? n : 0;
    const int64_t have = len > 0 ? (static_cast<int64_t>(len) + p.block_size - 1) / p.block_size : 0;
    const int64_t need =
        err ? 0 : (static_cast<int64_t>(len) + n + p.block_size - 1) / p.block_size - have;
    int64_t a = need, t = grow, ta, tt;
    if (tid == 0) scan.first_fail = kSlThreads;
    slot_scan(scan, a, t, ta, tt);
    const int64_t tok0 = tokens + t - grow;  // the sequence's first token
    if (!err && taken + a > F) err = PA_DEVERR_OUT_OF_BLOCKS;
    if (!err && tokens + t > p.num_tokens) err = PA_DEVERR_BAD_QUERY;
    if (in && err) atomicMin(&scan.first_fail, tid);
    s_tok[tid] = static_cast<int32_t>(min(tok0, static_cast<int64_t>(p.num_tokens)));
    s_len[tid] = len;
    s_base[tid] = static_cast<int32_t>(taken + a - need - have);  // + j: stack depth of block j
    slot_barrier<kC>();  // the tile is read, its records are written
    const int32_t fail = stopped ? 0 : min(scan.first_fail, count);
    if (rank == 0 && in) {
      if (tid == fail && err && !stopped) flag_error(err);
      p.seq_lens[b] = tid < fail ? len + n : len;
      p.q_start[b] = s_tok[tid];
    }
    // one thread per token of the tile
    const int32_t t0 = s_tok[0];
    const int32_t t1 = static_cast<int32_t>(min(tokens + tt, static_cast<int64_t>(p.num_tokens)));
    for (int64_t x0 = t0 + static_cast<int64_t>(rank) * kSlThreads + tid; x0 < t1;
         x0 += kSlBatch * threads) {
      int32_t id[kSlBatch], o[kSlBatch];
      int32_t* fresh[kSlBatch];  // the table entry of a new block
#pragma unroll
      for (int q = 0; q < kSlBatch; ++q) {
        const int64_t x = x0 + q * threads;
        id[q] = -1;
        o[q] = -1;
        fresh[q] = nullptr;
        if (x >= t1) continue;
        const int i = slot_find(s_tok, count, static_cast<int32_t>(x));
        if (i >= fail) continue;
        const int32_t pos = s_len[i] + static_cast<int32_t>(x) - s_tok[i];
        const int32_t j = pos / p.block_size;
        o[q] = pos - j * p.block_size;
        int32_t* entry = p.tables + static_cast<int64_t>(b0 + i) * p.max_blocks + j;
        const bool held = j < (s_len[i] + p.block_size - 1) / p.block_size;
        id[q] = held ? *entry : p.free_ids[F - 1 - (s_base[i] + j)];
        if (!held && o[q] == 0) fresh[q] = entry;  // a new block's first token is a new token
      }
#pragma unroll
      for (int q = 0; q < kSlBatch; ++q) {
        const int64_t x = x0 + q * threads;
        if (x >= t1) continue;
        if (fresh[q] != nullptr) *fresh[q] = id[q];
        const bool good = id[q] >= 0 && id[q] < p.num_blocks;
        if (o[q] >= 0 && !good) flag_error(PA_DEVERR_BAD_BLOCK_ID);
        p.slots[x] = o[q] >= 0 && good ? static_cast<int64_t>(id[q]) * p.block_size + o[q] : -1;
      }
    }
    if (!stopped && fail < count) {
      stopped = true;
      stop = b0 + fail;
      // blocks taken before the failing sequence: its base
      taken = s_base[fail];
      if (s_len[fail] > 0) taken += (static_cast<int64_t>(s_len[fail]) + p.block_size - 1) / p.block_size;
    } else if (!stopped) {
      taken += ta;
    }
    tokens += tt;
    slot_barrier<kC>();  // the records are read before the next tile's
  }
  // rows past the last sequence have no slot
  const int64_t used = min(tokens, static_cast<int64_t>(p.num_tokens));
  for (int64_t x = used + static_cast<int64_t>(rank) * kSlThreads + tid; x < p.num_tokens;
       x += threads)
    p.slots[x] = -1;
  if (rank == 0 && tid == 0) {
    p.q_start[p.num_seqs] = static_cast<int32_t>(used);
    *p.num_free_out = F - static_cast<int32_t>(taken);
    *p.num_done = stop;
  }
  __threadfence();
}

template <int kC>
__global__ void __launch_bounds__(kSlThreads) trim_slots_kernel(const SlotParams p) {
  __shared__ SlotScan scan;
  __shared__ int32_t s_at[kSlThreads], s_from[kSlThreads], s_bad[kSlThreads];
  const int tid = threadIdx.x;
  const int rank = kC == 1 ? 0 : static_cast<int>(blockIdx.x);
  const int64_t threads = static_cast<int64_t>(kC == 1 ? 1 : gridDim.x) * kSlThreads;
  pdl_wait();
  int32_t F = *p.num_free;
  if (F < 0 || F > p.num_blocks) {
    if (rank == 0 && tid == 0) flag_error(PA_DEVERR_BAD_BLOCK_ID);
    F = F < 0 ? 0 : p.num_blocks;
  }
  const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.block_size;
  int64_t pushed = 0;  // blocks of the sequences before the tile
  // a tile's lengths are loaded while the tile before is worked on
  int32_t len_next = tid < p.num_seqs ? p.lens[tid] : 0;
  int32_t to_next = tid < p.num_seqs ? p.change[tid] : 0;
  for (int32_t b0 = 0; b0 < p.num_seqs; b0 += kSlThreads) {
    const int32_t b = b0 + tid;
    const bool in = b < p.num_seqs;
    const int32_t count = min(kSlThreads, p.num_seqs - b0);
    const int32_t len = len_next, to = to_next;
    const bool more = b < p.num_seqs - kSlThreads;
    len_next = more ? p.lens[b + kSlThreads] : 0;
    to_next = more ? p.change[b + kSlThreads] : 0;
    const bool bad_len = len < 0 || len > cap || to < 0 || to > len;
    const int32_t left = bad_len ? 0 : static_cast<int32_t>((static_cast<int64_t>(to) + p.block_size - 1) / p.block_size);
    const int32_t have = bad_len ? 0 : static_cast<int32_t>((static_cast<int64_t>(len) + p.block_size - 1) / p.block_size);
    s_bad[tid] = 0;
    if (tid == 0) scan.redo = 0;
    slot_barrier<kC>();  // flags cleared everywhere before a round may set them
    int64_t room = static_cast<int64_t>(p.num_blocks) - F - pushed;
    bool kept = bad_len;  // the sequence stays as it is
    int64_t all = 0;      // blocks this tile pushes
    // A further round runs only after one that met an invalid id: its
    // sequence then keeps all its blocks and the others move up, so there
    // are at most count + 1 rounds.
    for (int round = 0; round <= count; ++round) {
      kept = bad_len || s_bad[tid] != 0;
      const int32_t cnt = kept ? 0 : have - left;
      int64_t a = cnt, z = 0, ta, tz;
      slot_scan(scan, a, z, ta, tz);
      const bool over = cnt > 0 && a > room;  // more blocks than the pool has
      kept |= over;
      s_at[tid] = static_cast<int32_t>(a - cnt);
      s_from[tid] = left;
      all = ta;
      if (ta > room) {  // the same in every thread: the first ones that fit
        int64_t fits = over ? 0 : cnt, none = 0, unused;
        slot_scan(scan, fits, none, all, unused);
      }
      __syncthreads();
      for (int64_t x0 = static_cast<int64_t>(rank) * kSlThreads + tid; x0 < all;
           x0 += kSlBatch * threads) {
        int32_t id[kSlBatch], at[kSlBatch];
#pragma unroll
        for (int q = 0; q < kSlBatch; ++q) {
          const int32_t x = static_cast<int32_t>(x0 + q * threads);
          id[q] = 0;
          if (x0 + q * threads >= all) continue;
          at[q] = slot_find(s_at, count, x);
          id[q] = p.tables[static_cast<int64_t>(b0 + at[q]) * p.max_blocks + s_from[at[q]] +
                           (x - s_at[at[q]])];
        }
#pragma unroll
        for (int q = 0; q < kSlBatch; ++q) {
          const int64_t x = x0 + q * threads;
          if (x >= all) continue;
          if (id[q] >= 0 && id[q] < p.num_blocks) {
            p.free_ids[F + pushed + x] = id[q];
          } else if (kC == 1) {
            s_bad[at[q]] = 1;
            scan.redo = round + 1;
          } else {
            auto cl = cooperative_groups::this_cluster();
            for (int r = 0; r < kC; ++r) {
              cl.map_shared_rank(s_bad, r)[at[q]] = 1;
              cl.map_shared_rank(&scan, r)->redo = round + 1;
            }
          }
        }
      }
      slot_barrier<kC>();
      if (scan.redo <= round) break;  // the same in every CTA
    }
    if (rank == 0 && in) {
      p.seq_lens[b] = kept ? len : to;
      if (bad_len) flag_error(PA_DEVERR_BAD_SEQ_LEN);
      if (kept && !bad_len) flag_error(PA_DEVERR_BAD_BLOCK_ID);
    }
    pushed += all;
    slot_barrier<kC>();
  }
  if (rank == 0 && tid == 0) *p.num_free_out = F + static_cast<int32_t>(pushed);
  __threadfence();
}

}  // namespace pa
