// sa_chunk.cuh -- how the chunk-attention kernels divide a ragged batch of new tokens among
// the CTAs of one persistent grid.
//
// An item is (sequence, head group, block of consecutive new tokens); its work is the list of
// 128-key tiles that any of the block's rows sees: tiles [0, na) of the sink tokens and tiles
// from bs on (one list when there is no window).  The list is walked in steps of one tile, or
// of two when a block is short enough for its rows to fill one matrix tile only (the kernel
// then works on two key tiles at a time).
//
// Long lists are cut: the steps of all items, laid end to end in (sequence, head, block)
// order, are dealt to the CTAs in equal runs, so a CTA holds at most two cut pieces (the end
// of one item, the start of another), kept in workspace slots 2 c and 2 c + 1 of CTA c and
// joined by a second kernel.  When there are at least four times as many steps per CTA as the longest
// item has, nothing is cut: CTAs draw whole items from a counter, which keeps the CTAs on the
// same head and so on the same keys in L2, longest blocks of a head first.
// With inner > 1 the head groups of one piece go to `inner` neighbouring CTAs at the same time
// instead of one after the other: they read the same keys.
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
  int pad;
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
  int sink, window;
  int64_t cap;     // max_pages * P
  int32_t* status;
  int32_t* ticket;  // header word, zero between calls
};

struct ChunkBlock {
  int t0, nt, na, bs, tiles, split, steps;
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
    k.na = min((int)(((int64_t)min(s.sink, hi + 1) + kKeyTile - 1) / kKeyTile), k.bs);
  }
  k.tiles = k.na + hi / kKeyTile - k.bs + 1;
  k.split = k.nt <= s.ST;
  k.steps = k.split ? (k.tiles + 1) >> 1 : k.tiles;
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

// Every member function is called by one whole warp.
struct ChunkSched {
  ChunkShape s;
  int nc, c;             // runs, and this CTA's
  int lane_h;            // its head group (inner > 1)
  bool whole;
  int64_t total, left;   // steps of all items; of this CTA still to hand out
  int64_t pos;           // steps before the current item
  int b, h, j, off;      // the current item and how many of its steps are gone
  int n, L, c0;          // its sequence
  int items, ticket;     // whole items: count, and the next one drawn
  int gb, gpre;          // whole items: group of 32 sequences, items before it

  // steps of all blocks (one head) of sequence (nn, LL) of this lane, and the longest
  __device__ __forceinline__ int64_t seq_steps(int nn, int LL, int& longest) {
    const int lane = threadIdx.x & 31;
    const int nb = (nn + s.BT - 1) / s.BT;
    int64_t sum = 0;
    int most = 0;
    if (nb <= 4)
      for (int q = 0; q < nb; ++q) {
        const int st = chunk_block(s, nn, LL, q).steps;
        sum += st;
        most = max(most, st);
      }
    for (unsigned m = __ballot_sync(0xffffffffu, nb > 4); m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const int n1 = __shfl_sync(0xffffffffu, nn, src), L1 = __shfl_sync(0xffffffffu, LL, src);
      const int nb1 = (n1 + s.BT - 1) / s.BT;
      int64_t t = 0;
      int mx = 0;
      for (int q = lane; q < nb1; q += 32) {
        const int st = chunk_block(s, n1, L1, q).steps;
        t += st;
        mx = max(mx, st);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      mx = __reduce_max_sync(0xffffffffu, mx);
      if (lane == src) {
        sum = t;
        most = mx;
      }
    }
    longest = most;
    return sum;
  }

  __device__ __forceinline__ void lane_seq(int base, int& nn, int& LL, bool check) {
    const int q = base + (threadIdx.x & 31);
    int cc;
    nn = 0;
    LL = 0;
    if (q < s.B && !chunk_seq(s, q, cc, nn, LL) && check) report(s.status, SA_ERR_DEVICE_CHECK);
  }

  __device__ void init(const ChunkShape& shape, int cta, int n_cta) {
    s = shape;
    c = cta / s.inner;
    lane_h = cta % s.inner;
    const int runs = n_cta / s.inner;
    const int lane = threadIdx.x & 31;
    total = 0;
    items = 0;
    int longest = 0;
    for (int base = 0; base < s.B; base += 32) {
      int nn, LL, mx;
      lane_seq(base, nn, LL, cta == 0);
      int64_t t = seq_steps(nn, LL, mx);
      int k = (nn + s.BT - 1) / s.BT;
#pragma unroll
      for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      total += t;
      items += __reduce_add_sync(0xffffffffu, k);
      longest = max(longest, __reduce_max_sync(0xffffffffu, mx));
    }
    total *= s.H;
    items *= s.H;
    nc = (int)min((int64_t)runs, total);
    whole = total >= (int64_t)kWholeFactor * longest * runs;
    left = 0;
    if (total == 0) {
      whole = false;
      return;
    }
    if (whole) {
      gb = 0;
      gpre = 0;
      draw();
      return;
    }
    if (c >= nc) return;
    const int64_t x0 = total * c / nc;
    left = total * (c + 1) / nc - x0;
    // the item that step x0 belongs to
    int64_t pre = 0;
    for (int base = 0; base < s.B; base += 32) {
      int nn, LL, mx;
      lane_seq(base, nn, LL, false);
      const int64_t mine = seq_steps(nn, LL, mx) * s.H;
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned m = __ballot_sync(0xffffffffu, pre + incl > x0);
      if (m) {
        const int src = __ffs(m) - 1;
        b = base + src;
        const int64_t cost = __shfl_sync(0xffffffffu, mine, src) / s.H;
        pos = pre + __shfl_sync(0xffffffffu, incl - mine, src);
        h = (int)((x0 - pos) / cost);
        pos += h * cost;
        break;
      }
      pre += __shfl_sync(0xffffffffu, incl, 31);
    }
    chunk_seq(s, b, c0, n, L);
    const int nb = (n + s.BT - 1) / s.BT;
    for (j = 0; j < nb; j += 32) {
      const int q = j + lane;
      const int mine = q < nb ? chunk_block(s, n, L, q).steps : 0;
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned m = __ballot_sync(0xffffffffu, pos + incl > x0);
      if (m) {
        const int src = __ffs(m) - 1;
        pos += __shfl_sync(0xffffffffu, incl - mine, src);
        j += src;
        break;
      }
      pos += __shfl_sync(0xffffffffu, incl, 31);
    }
    off = (int)(x0 - pos);
  }

  __device__ __forceinline__ void draw() {
    if ((threadIdx.x & 31) == 0) ticket = atomicAdd(s.ticket, 1);
  }

  // The next piece; false when there is none.
  __device__ bool next(ChunkSeg& g) {
    const int lane = threadIdx.x & 31;
    g.nparts = 0;
    g.part = -1;
    if (whole) {
      const int drawn = __shfl_sync(0xffffffffu, ticket, 0), t = drawn / s.inner;
      if (t >= items || drawn < 0) return false;
      lane_h = drawn % s.inner;
      draw();
      for (;; gb += 32) {
        int nn, LL;
        lane_seq(gb, nn, LL, false);
        const int mine = (nn + s.BT - 1) / s.BT * s.H;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        const unsigned m = __ballot_sync(0xffffffffu, gpre + incl > t);
        if (m) {
          const int src = __ffs(m) - 1;
          b = gb + src;
          const int q = t - gpre - __shfl_sync(0xffffffffu, incl - mine, src);
          const int nb = __shfl_sync(0xffffffffu, mine, src) / s.H;
          h = q / nb;
          j = nb - 1 - q % nb;
          break;
        }
        gpre += __shfl_sync(0xffffffffu, incl, 31);
      }
      chunk_seq(s, b, c0, n, L);
      const ChunkBlock k = chunk_block(s, n, L, j);
      fill(g, k, 0, k.tiles);
      return true;
    }
    if (left <= 0) return false;
    const ChunkBlock k = chunk_block(s, n, L, j);
    const int take = (int)min(left, (int64_t)(k.steps - off));
    const int end = off + take;
    fill(g, k, k.split ? 2 * off : off, k.split ? min(k.tiles, 2 * end) : end);
    if (off > 0) {
      g.part = 2 * (c * s.inner + lane_h);
    } else if (end < k.steps) {
      g.part = 2 * (c * s.inner + lane_h) + 1;
      // CTAs whose runs start before the item's end: run r starts at floor(r total / nc)
      const int64_t e = pos + k.steps;
      const int last = (int)min((int64_t)nc - 1, (e * nc + total - 1) / total - 1);
      g.nparts = last - c + 1;
    }
    left -= take;
    off = end;
    if (off == k.steps) {
      pos += k.steps;
      off = 0;
      if (++j == (n + s.BT - 1) / s.BT) {
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

  __device__ __forceinline__ void fill(ChunkSeg& g, const ChunkBlock& k, int i0, int i1) {
    g.valid = 1;
    g.row0 = c0 + k.t0;
    g.ntok = k.nt;
    g.b = b;
    g.h = h * s.inner + lane_h;
    g.s0 = L - n + k.t0;
    g.L = L;
    g.na = k.na;
    g.bs = k.bs;
    g.i0 = i0;
    g.i1 = i1;
    g.split = k.split;
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
