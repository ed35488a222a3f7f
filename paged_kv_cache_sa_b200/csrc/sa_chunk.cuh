// sa_chunk.cuh -- how the chunk-attention kernels divide a ragged batch of new tokens among
// the CTAs of one persistent grid.
//
// An item is (sequence, head group, block of consecutive new tokens); its work is the list of
// 128-key tiles that any of the block's rows sees: tiles [0, na) of the sink tokens and tiles
// from bs on (one list when there is no window).  The list is walked in steps of one tile, or
// of two when a block is short enough for its rows to fill one matrix tile only (the kernel
// then works on two key tiles at a time).
//
// Long lists are cut: the costs of all items (their steps, and a few more for what a piece
// takes to start and end), laid end to end in (sequence, head, block) order, are dealt to the
// CTAs in equal runs, so a CTA holds at most two cut pieces (the end of one item, the start of
// another), kept in workspace slots 2 c and 2 c + 1 of CTA c and joined by a second kernel.
// When there is at least four times as much to do per CTA as the longest item takes, nothing is
// cut: whole items, the longest blocks of a head first, go to the CTAs in rounds, forwards and
// backwards in turn.  That keeps the CTAs on the same head and so on the same keys in L2; where the
// last round holds few items, the fullest CTA has up to 1.24 times the mean.  (A
// counter to draw from, in place of the rounds, is 1-4% faster on long chunks and up to 2%
// slower on short ones, and would have to be zero before every call.)
// With inner > 1 the head groups of one piece go to `inner` neighbouring CTAs at the same time
// instead of one after the other: they read the same keys and make the same list.
#pragma once

#include "sa_common.cuh"

namespace sa {

constexpr int kKeyTile = 128;  // keys of one tile
constexpr int kWholeFactor = 4;

// One item's piece, as the producer warp hands it to the other warps.
struct ChunkSeg {
  int valid;       // 0: no more work
  int row0, ntok;  // first row of q/out and count of tokens
  int b, h;
  int s0;          // slot of the first token
  int L;           // the sequence's length
  int na, bs;      // tile i of the list is i < na ? i : i - na + bs
  int i0, i1;      // the piece of the list
  int split;       // two key tiles per step
  int part;        // workspace slot of a cut piece, -1 for a whole item
  int nparts;      // of a cut item, at its first piece (0 elsewhere)
  int it0;         // stages the producer has filled before this piece
  int once;        // no other block reads these keys
};
static_assert(sizeof(ChunkSeg) == 64, "segment is 64 bytes");

// What the joining kernel needs of a cut item; at its first piece's slot.
struct ChunkCut {
  int nparts, row0, ntok, h;  // nparts 0: no item starts (and is cut) in this slot
};

struct ChunkShape {
  const int32_t* cu_new;
  const int32_t* seq_lens;
  int n_tokens, B;
  int H;           // head groups per token, one after the other
  int inner;       // head groups side by side: CTAs [inner w, inner w + inner) share run w
  int BT;          // tokens of a full block
  int ST;          // blocks of at most this many tokens walk two tiles a step
  int extra;       // what a piece costs besides its steps, in steps
  int sink, window;
  int64_t cap;     // max_pages * P
  int32_t* status;
};

struct ChunkBlock {
  int t0, nt, na, bs, tiles, split, steps, cost;
};

__device__ __forceinline__ ChunkBlock chunk_block(const ChunkShape& s, int n, int L, int j) {
  ChunkBlock k;
  k.t0 = j * s.BT;
  k.nt = min(s.BT, n - k.t0);
  const int lo = L - n + k.t0, hi = lo + k.nt - 1;  // slots of the first and last row
  k.na = 0;
  k.bs = 0;
  if (s.window > 0) {
    const int first = max(0, lo - s.window + 1);  // lowest key of any row's window
    k.bs = first / kKeyTile;
    k.na = min((min(s.sink, hi + 1) + kKeyTile - 1) / kKeyTile, k.bs);
  }
  k.tiles = k.na + hi / kKeyTile - k.bs + 1;
  k.split = k.nt <= s.ST;
  k.steps = k.split ? (k.tiles + 1) >> 1 : k.tiles;
  k.cost = k.steps + s.extra;  // the extra ones come first
  return k;
}

// Rows, count of new tokens and length of sequence b (n = 0 when it does not fit).
__device__ __forceinline__ bool chunk_seq(const ChunkShape& s, int b, int& c0, int& n, int& L) {
  c0 = s.cu_new[b];
  const int c1 = s.cu_new[b + 1];
  L = s.seq_lens[b];
  const bool ok = c0 >= 0 && c1 >= c0 && c1 <= s.n_tokens && L >= c1 - c0 && L <= s.cap;
  n = ok ? c1 - c0 : 0;
  return ok;
}

__device__ __forceinline__ uint32_t warp_prefix(uint32_t v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// The list is made by every CTA for itself, before its first copy, by code that runs once: it
// is kept short and free of divisions.  Every member function is called by one whole warp.
struct ChunkSched {
  ChunkShape s;
  int runs, c;           // runs that the CTAs could take, and this CTA's
  int lane_h;            // its head group (inner > 1)
  bool whole;
  uint32_t total, left;  // cost of all items (cut list); of this run still to hand out
  uint32_t per, rem;     // total = per * runs + rem
  uint32_t pos;          // cost before the current item
  int b, h, j, off;      // the current item and how much of its cost is gone
  int n, L, c0;          // its sequence
  int items, round;      // whole items: count, and rounds gone
  int gb, gpre;          // whole items: group of 32 sequences, items before it

  __device__ __forceinline__ int blocks(int nn) const {
    return nn <= s.BT ? nn > 0 : (nn + s.BT - 1) / s.BT;
  }

  // sequence of this lane in the group from `base`: its new tokens and length
  __device__ __forceinline__ void lane_seq(int base, int& nn, int& LL, bool check) {
    const int q = base + (threadIdx.x & 31);
    int cc;
    nn = 0;
    LL = 0;
    if (q < s.B && !chunk_seq(s, q, cc, nn, LL) && check) report(s.status, SA_ERR_DEVICE_CHECK);
  }

  // cost of all blocks (one head) of this lane's sequence, and of its longest block
  __device__ __forceinline__ uint32_t seq_cost(int nn, int LL, uint32_t& longest) {
    const int lane = threadIdx.x & 31;
    const int nb = blocks(nn);
    uint32_t sum = 0, most = 0;
    // one block at a time by the lane itself, or (many blocks) 32 at a time by the warp
    for (unsigned todo = __ballot_sync(0xffffffffu, nb > 0); todo;) {
      const unsigned many = __ballot_sync(0xffffffffu, nb > 1) & todo;
      const int src = many ? __ffs(many) - 1 : lane;
      todo = many ? todo & ~(1u << src) : 0;
      const int n1 = __shfl_sync(0xffffffffu, nn, src), L1 = __shfl_sync(0xffffffffu, LL, src);
      const int nb1 = blocks(n1);
      uint64_t t = 0;
      uint32_t mx = 0;
#pragma unroll 1
      for (int q = many ? lane : 0; q < nb1; q += 32) {
        const uint32_t st = chunk_block(s, n1, L1, q).cost;
        t += st;
        mx = max(mx, st);
      }
      if (many) {  // saturated at 2^31, where no list is cut
        const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)min(t >> 24, (uint64_t)255));
        t = __reduce_add_sync(0xffffffffu, (uint32_t)t & 0xFFFFFFu) + ((uint64_t)hi << 24);
        mx = __reduce_max_sync(0xffffffffu, mx);
      }
      if (many ? lane == src : nb == 1) {
        sum = (uint32_t)min(t, (uint64_t)1 << 31);
        most = mx;
      }
    }
    longest = most;
    return sum;
  }

  // where run r starts, floor(r total / runs), for r <= runs
  __device__ __forceinline__ uint32_t start(uint32_t r) const { return r * per + r * rem / runs; }

  __device__ __forceinline__ void init(const ChunkShape& shape, int cta, int n_cta) {
    s = shape;
    c = s.inner == 1 ? cta : cta / s.inner;
    lane_h = s.inner == 1 ? 0 : cta % s.inner;
    runs = s.inner == 1 ? n_cta : n_cta / s.inner;
    const int lane = threadIdx.x & 31;
    uint64_t all = 0, count = 0;
    uint32_t longest = 0, mine = 0;
#pragma unroll 1
    for (int base = 0; base < s.B; base += 32) {
      int nn, LL;
      uint32_t mx;
      lane_seq(base, nn, LL, cta == 0);
      mine = seq_cost(nn, LL, mx);
      all += __reduce_add_sync(0xffffffffu, mine & 0xFFFFu) +
             ((uint64_t)__reduce_add_sync(0xffffffffu, mine >> 16) << 16);
      count += __reduce_add_sync(0xffffffffu, blocks(nn));
      longest = max(longest, __reduce_max_sync(0xffffffffu, mx));
    }
    all *= s.H;
    // (more items than that only if sequences overlap; next_whole() counts in 32 bits)
    if (count * s.H >> 31) {
      all = 0;
      if (cta == 0) report(s.status, SA_ERR_DEVICE_CHECK);
    }
    items = (int)(count * s.H);
    // whole items, too, where a count of steps would not fit 32 bits
    whole = all >= (uint64_t)kWholeFactor * longest * runs || all >> 31;
    left = 0;
    if (all == 0 || c >= runs) {
      whole = false;
      return;
    }
    if (whole) {
      gb = 0;
      gpre = 0;
      round = 0;
      return;
    }
    total = (uint32_t)all;
    if (total < (uint32_t)runs) runs = (int)total;  // a step each
    per = total / (uint32_t)runs;
    rem = total - per * runs;
    if (c >= runs) return;
    const uint32_t x0 = start(c);
    left = start(c + 1) - x0;
    // the sequence and head that x0 lies in
    pos = 0;
#pragma unroll 1
    for (int base = 0;; base += 32) {
      if (s.B > 32) {
        int nn, LL;
        uint32_t mx;
        lane_seq(base, nn, LL, false);
        mine = seq_cost(nn, LL, mx);
      }
      const uint32_t incl = warp_prefix(mine * s.H);
      const unsigned m = __ballot_sync(0xffffffffu, pos + incl > x0);
      if (m) {
        const int src = __ffs(m) - 1;
        b = base + src;
        const uint32_t cost = __shfl_sync(0xffffffffu, mine, src);
        pos += __shfl_sync(0xffffffffu, incl, src) - cost * s.H;
        for (h = 0; x0 - pos >= cost; ++h) pos += cost;
        break;
      }
      pos += __shfl_sync(0xffffffffu, incl, 31);
    }
    // and its block
    chunk_seq(s, b, c0, n, L);
    j = 0;
    const int nb = blocks(n);
    if (nb > 1) {
#pragma unroll 1
      for (;; j += 32) {
        const uint32_t st = j + lane < nb ? chunk_block(s, n, L, j + lane).cost : 0;
        const uint32_t incl = warp_prefix(st);
        const unsigned m = __ballot_sync(0xffffffffu, pos + incl > x0);
        if (m) {
          const int src = __ffs(m) - 1;
          pos += __shfl_sync(0xffffffffu, incl - st, src);
          j += src;
          break;
        }
        pos += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    off = (int)(x0 - pos);
  }

  // whole items: this CTA's next one -> b, h, j; false when there is none.  Rounds of `runs` items
  // go to the CTAs forwards and backwards in turn: blocks get shorter along a round.
  __device__ __forceinline__ bool next_whole() {
    const int64_t at = (int64_t)round * runs + (round & 1 ? runs - 1 - c : c);
    ++round;
    if (at >= items) return false;  // (so are those of all later rounds)
    const int t = (int)at;
#pragma unroll 1
    for (;; gb += 32) {
      int nn, LL;
      lane_seq(gb, nn, LL, false);
      const int mine = blocks(nn) * s.H;
      const int incl = (int)warp_prefix(mine);
      const unsigned m = __ballot_sync(0xffffffffu, gpre + incl > t);
      if (m) {
        const int src = __ffs(m) - 1;
        b = gb + src;
        const int q = t - gpre - __shfl_sync(0xffffffffu, incl - mine, src);
        const int nb = __shfl_sync(0xffffffffu, mine, src) / s.H;
        h = q / nb;
        j = nb - 1 - (q - h * nb);
        break;
      }
      gpre += __shfl_sync(0xffffffffu, incl, 31);
    }
    chunk_seq(s, b, c0, n, L);
    return true;
  }

  // The next piece; false when there is none.
  __device__ __forceinline__ bool next(ChunkSeg& g) {
    if (whole ? !next_whole() : left == 0) return false;
    const ChunkBlock k = chunk_block(s, n, L, j);
    int from = 0, end = k.steps;  // the piece, in steps
    if (!whole) {
      const int stop = (int)min((uint32_t)k.cost, off + left);
      from = max(off - s.extra, 0);
      end = max(stop - s.extra, 0);
      left -= stop - off;
      off = stop;
      if (end == 0) return false;  // the run ends before the item's first step
    }
    g.nparts = 0;
    g.part = -1;
    const int slot = 2 * (c * s.inner + lane_h);
    if (from > 0) {
      g.part = slot;
    } else if (end < k.steps) {
      g.part = slot + 1;
      // the runs from this one on that start before the item's end
      int before = 0;
#pragma unroll 1
      for (int r = threadIdx.x & 31; r < runs; r += 32) before += start(r) < pos + k.cost;
      g.nparts = __reduce_add_sync(0xffffffffu, before) - c;
    }
    g.valid = 1;
    g.row0 = c0 + k.t0;
    g.ntok = k.nt;
    g.b = b;
    g.h = h * s.inner + lane_h;
    g.s0 = L - n + k.t0;
    g.L = L;
    g.na = k.na;
    g.bs = k.bs;
    g.split = k.split;
    g.i0 = k.split ? 2 * from : from;
    g.i1 = k.split ? min(k.tiles, 2 * end) : end;
    g.once = k.nt == n;
    if (!whole && off == k.cost) {
      pos += k.cost;
      off = 0;
      if (++j == blocks(n)) {
        j = 0;
        if (++h == s.H) {
          h = 0;
          n = 0;
          while (left > 0 && n == 0 && ++b < s.B) chunk_seq(s, b, c0, n, L);
          if (n == 0) left = 0;
        }
      }
    }
    return true;
  }
};

inline size_t chunk_up256(size_t x) { return (x + 255) & ~size_t(255); }

// A launch that may begin before the stream's previous kernel has ended (the kernels wait).
inline cudaError_t chunk_launch(const void* fn, dim3 grid, int threads, size_t smem,
                                cudaStream_t stream, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace sa
