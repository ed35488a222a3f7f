// sa_chunk.cu -- exact attention of a ragged chunk of new tokens over the paged cache,
// grouped-query geometry, on the 5th-generation tensor cores.
//
// Method: x_t = scale q . k_t over the tokens t a query sees, one pass over the keys with the
// running maximum m and sum l of the softmax: out = sum 2^(x_t - m) v_t / l  (x in base 2).
//
// Rows.  The G query heads of a KV head see the same keys, so a matrix tile of 128 rows is
// 128 / G tokens times G heads, and K and V are read once for all of them.
// A CTA holds two accumulators (O0, O1) and two score tiles (S0, S1) in tensor memory, all
// 512 columns at Dk = 128:
//   a full block: two row tiles against one key tile per step (every K and V tile staged in
//   shared memory serves 256 rows);
//   a short block (the rows fit one tile: decode rows, drafts, the end of a prompt): one row
//   tile against two key tiles per step, even ones in (S0, O0) and odd ones in (S1, O1), each
//   with its own m and l, joined at the end.  The work per step is the same, so a single
//   token still keeps two chains of products and exponentials in flight; the rows that are
//   padding cost tensor time (1024 cycles per 64 KB key tile), which HBM hides (2800 cycles).
// Per tile: S = Q K^T (128 x 128 x Dk) from shared memory; four softmax warps (thread = row)
// read S, subtract the row's maximum, write P in bf16 over S's columns and O += P V
// (128 x Dv x 128) takes P from tensor memory.  (bf16 because V is and a product's operands have
// one type: half a step, 2^-9 to 2^-8, of each probability; l sums them before that rounding.)
// While one chain's softmax runs, the other chain's two products do.
// The maximum in use is only raised when a row's new maximum exceeds it by more than 2^8
// (P then stays below 2^8, exact in range for bf16 and fp32): O is rescaled a few times per
// row instead of at every tile, by the softmax warps themselves.
// Warps 0-3 and 4-7: softmax of chain 0 and 1; 8: issues the products; 9: work list, queries
// and K; 10: V (one warp for both had the copies of 16-token pages queue behind one another:
// 212 us instead of 184 for the decode rows below).
// Measured on a B200, 32 / 8 heads of 128 channels, in short graphs at up to 1965 MHz: eight decode
// rows at 32768 tokens 165 us (6.5 TB/s, HBM), 8192 rows at 32768 2.95 ms (1.3 PFLOP/s, tensor pipe
// 65% busy: a chain waits for its softmax, some 2000 cycles a tile, and for its own products between
// two tiles; four products of a step take 2048).  At sustained clocks, on changing inputs: 178 us and
// 3.35 ms.  Pieces of few tiles pay about two tiles for starting and ending.
#include "sa_chunk.cuh"
#include "sa_internal.h"
#include "sa_tc.cuh"

namespace sa {

namespace chunk {

constexpr int kThreads = 384;
// registers: 168 a thread at launch (384 x 168 = 64512); 256 x 208 + 128 x 88 = 64512
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kSegs = 2;
// probabilities are handed over in two parts, so that the product over the first keys runs while
// the last ones are computed (2% of a long chunk against 64 + 64)
constexpr int kFirstKeys = 96;
constexpr uint32_t kHalfBytes = kKeyTile * 128;  // 128 rows of 64 channels

struct Misc {
  float2 ml[2][128];  // (m, l) of both chains, short blocks
  ChunkSeg seg[kSegs];
  uint64_t full[10], empty[10];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full, q_empty, s_full[2], p_part[2], p_full[2], o_full[2], meet, drain;
  uint32_t tmem;
  int quit;
};

template <int D>
struct Lay {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTileBytes = kHalves * kHalfBytes;  // a Q, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kRing = 2 * kTileBytes;
  static constexpr uint32_t kMisc = kRing + kStages * kTileBytes;
  static constexpr uint32_t kSmem = kMisc + sizeof(Misc);
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

struct Args {
  ChunkShape shape;
  const int32_t* page_table;
  uint16_t* out;
  float* lse;
  float* part_o;    // [2 n_cta][rows_cap / 8][D / 4][8][4]
  float2* part_ml;  // [2 n_cta][rows_cap]
  ChunkCut* cut;    // [n_cta]
  int rows_cap;
  int Hq, Hkv, G, TB, P, page_shift, max_pages, n_pool;
  float scale_log2;
};

__device__ __forceinline__ int tile_of(const ChunkSeg& g, int i) {
  return i < g.na ? i : i - g.na + g.bs;
}

// Position in the ring, counted from the piece's first stage, of K and V of its i-th tile: K of
// the first tile (two, if a step takes two), then V of a tile and K of the next without one.
__device__ __forceinline__ int k_pos(bool split, int i) {
  return split ? (i == 0 ? 0 : 2 * i - 1) : 2 * i;
}
__device__ __forceinline__ int v_pos(bool split, int nt, int i) {
  return split && i + 1 < nt ? 2 * i + 2 : 2 * i + 1;
}

// ---- the producer warps: one makes the work list and loads queries and K, one loads V ----
template <int D>
struct Loader {
  using Y = Lay<D>;
  const Args& a;
  uint32_t smem;
  Misc& mi;
  const CUtensorMap* map;
  bool values;  // V's
  int lane, ppt, my_page, my_half;

  __device__ __forceinline__ Loader(const Args& args, uint32_t s, Misc& m, const CUtensorMap* mp,
                                    bool v)
      : a(args), smem(s), mi(m), map(mp), values(v) {
    lane = threadIdx.x & 31;
    ppt = kKeyTile >> a.page_shift;  // pages per tile
    my_page = lane & (ppt - 1);
    my_half = lane / ppt;
  }

  // Tiles of one piece; a lane copies one page's rows of one half of the channels.
  __device__ __forceinline__ bool tiles(const ChunkSeg& g) {
    const int nt = g.i1 - g.i0, shift = a.page_shift;
    const int s_hi = g.s0 + g.ntok - 1, last_page = (g.L - 1) >> shift;
    const int32_t* row = a.page_table + (size_t)g.b * a.max_pages;
    // first page that any row's window reaches; pages of the sink below it
    const int win_page =
        a.shape.window > 0 ? max(0, g.s0 - a.shape.window + 1) >> shift : 0;
    const int sink_pages = (a.shape.sink + (1 << shift) - 1) >> shift;
    // keys that no other CTA reads leave L2 first: what every call starts from stays in it
    const uint64_t policy = g.once ? l2_evict_first() : tc::l2_normal();
    // page of this lane in tile i, and whether it is there and seen by some row
    auto wanted = [&](int i, int& lp) {
      lp = tile_of(g, g.i0 + i) * ppt + my_page;
      return my_half < Y::kHalves && lp <= last_page && (lp >= win_page || lp < sink_pages);
    };
    // page-table entries of tiles i, i + 1, i + 2, looked at only when their tile comes
    int p0 = -1, p1 = -1, p2 = -1, lp;
    for (int i = -3; i < nt; ++i) {
      const int p3 = i + 3 < nt && wanted(i + 3, lp) ? row[lp] : -1;
      if (i >= 0) {
        const int x = g.it0 + (values ? v_pos(g.split, nt, i) : k_pos(g.split, i));
        const int st = x % Y::kStages;
        bool copy = wanted(i, lp);
        if (copy && (p0 < 0 || p0 >= a.n_pool)) {
          if ((lp << shift) <= s_hi) report(a.shape.status, SA_ERR_DEVICE_CHECK);
          copy = false;
        }
        if (x >= Y::kStages && !tc::wait_warp(&mi.empty[st], (x / Y::kStages - 1) & 1, &mi.quit,
                                              a.shape.status))
          return false;
        const unsigned m = __ballot_sync(0xffffffffu, copy);
        if (lane == 0) mbar_arrive_expect_tx(&mi.full[st], __popc(m) * a.P * 128);
        __syncwarp();
        if (copy)
          tc::tma_2d(smem + Y::kRing + st * Y::kTileBytes + my_half * kHalfBytes +
                         ((uint32_t)my_page << shift) * 128,
                     map, my_half * 64, (p0 * a.Hkv + g.h) << shift, &mi.full[st], policy);
      }
      p0 = p1;
      p1 = p2;
      p2 = p3;
    }
    return true;
  }

  // given up: copies in flight land (bounded) before shared memory goes away
  __device__ void drain() {
    for (int st = 0; st < Y::kStages; ++st)
      for (int ph = 0; ph < 2; ++ph) mbar_wait(&mi.full[st], ph);
  }
};

// Both warps run the same code: the kernel is larger than its instruction cache, and a copy each
// is 1% slower on long chunks and 3% on short prompts (6 x 2368 rows 278 -> 270 us).
template <int D>
__device__ __forceinline__ void produce(const Args& a, uint32_t smem, Misc& mi,
                                        const CUtensorMap* qmap, const CUtensorMap* map,
                                        bool values) {
  using Y = Lay<D>;
  Loader<D> load(a, smem, mi, map, values);
  const int lane = load.lane;
  ChunkSched sched;
  if (!values) {
    if (lane == 0) a.cut[blockIdx.x].nparts = 0;
    sched.init(a.shape, blockIdx.x, gridDim.x);
  }
  int it = 0;
#pragma unroll 1
  for (int n = 0;; ++n) {
    const int slot = n % kSegs;
    ChunkSeg g;
    if (values) {
      if (!tc::wait_warp(&mi.seg_full[slot], (n / kSegs) & 1, &mi.quit, a.shape.status)) break;
      g = mi.seg[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&mi.seg_empty[slot]);
      if (!g.valid) return;
    } else {
      if (n >= kSegs && !tc::wait_warp(&mi.seg_empty[slot], (n / kSegs - 1) & 1, &mi.quit,
                                       a.shape.status))
        break;
      const bool more = sched.next(g);
      if (!more) g.valid = 0;
      g.it0 = it;
      if (lane == 0) {
        mi.seg[slot] = g;
        mbar_arrive(&mi.seg_full[slot]);
        if (more && g.nparts > 0) a.cut[blockIdx.x] = ChunkCut{g.nparts, g.row0, g.ntok, g.h};
      }
      if (!more) return;
      // queries: the box is G heads of TB tokens; rows behind the block belong to other
      // sequences (or none) and their results are not kept
      if (n > 0 && !tc::wait_warp(&mi.q_empty, (n - 1) & 1, &mi.quit, a.shape.status)) break;
      const int ntile = g.split ? 1 : 2;
      if (lane == 0) mbar_arrive_expect_tx(&mi.q_full, ntile * Y::kHalves * a.TB * a.G * 128);
      __syncwarp();
      if (lane < ntile * Y::kHalves) {
        const int t = lane / Y::kHalves, hf = lane % Y::kHalves;
        tc::tma_3d(smem + Y::kQ + t * Y::kTileBytes + hf * kHalfBytes, qmap, hf * 64, g.h * a.G,
                   g.row0 + t * a.TB, &mi.q_full);
      }
    }
    if (!load.tiles(g)) break;
    it += 2 * (g.i1 - g.i0);
  }
  load.drain();
  if (!values) mbar_wait(&mi.q_full, 0);
}

// ---- one warp issues every product ----------------------------------------------------
template <int D>
__device__ __forceinline__ void multiply(const Args& a, uint32_t smem, Misc& mi, uint32_t tmem) {
  using Y = Lay<D>;
  constexpr uint32_t id_s = tc::idesc(128, kKeyTile, false, false);
  constexpr uint32_t id_o = tc::idesc(128, D, false, true);
  int32_t* status = a.shape.status;
  int it = 0, np[2] = {0, 0};
  auto staged = [&](int x) {
    const bool r =
        tc::wait_warp(&mi.full[x % Y::kStages], (x / Y::kStages) & 1, &mi.quit, status);
    tc::fence_after();
    return r;
  };
  // (the rest runs in one lane)
  auto scores = [&](int qt, int t, int x) {  // S_t = Q_qt K^T of stage x
    const uint32_t q = smem + Y::kQ + qt * Y::kTileBytes;
    const uint32_t k = smem + Y::kRing + (x % Y::kStages) * Y::kTileBytes;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t o = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
      tc::mma_ss(tmem + t * 128, tc::desc(q + o), tc::desc(k + o), id_s, kk != 0);
    }
    tc::commit(&mi.s_full[t]);
  };
  // O_t += P_t V of stage x, as the two parts of P_t come; `then` follows in the same lane
  auto values = [&](int t, int x, bool first, auto then) -> bool {
    const uint32_t v = smem + Y::kRing + (x % Y::kStages) * Y::kTileBytes;
    const uint32_t parity = np[t]++ & 1;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      if (!tc::wait_warp(hf ? &mi.p_full[t] : &mi.p_part[t], parity, &mi.quit, status))
        return false;
      tc::fence_after();
      if (tc::elect()) {
#pragma unroll
        for (int kk = hf ? kFirstKeys / 16 : 0; kk < (hf ? kKeyTile : kFirstKeys) / 16; ++kk)
          tc::mma_ts(tmem + 256 + t * D, tmem + t * 128 + kk * 8,
                     tc::desc(v + kk * 2048, kHalfBytes), id_o, !(first && kk == 0));
        if (hf) then();
      }
      __syncwarp();
    }
    return true;
  };
  for (int n = 0;; ++n) {
    const int slot = n % kSegs;
    if (!tc::wait_warp(&mi.seg_full[slot], (n / kSegs) & 1, &mi.quit, status)) return;
    const int nt = __shfl_sync(0xffffffffu, mi.seg[slot].i1 - mi.seg[slot].i0, 0);
    const bool valid = __shfl_sync(0xffffffffu, mi.seg[slot].valid, 0) != 0;
    const bool split = __shfl_sync(0xffffffffu, mi.seg[slot].split, 0) != 0;
    if (tc::elect()) mbar_arrive(&mi.seg_empty[slot]);
    if (!valid) return;
    if (!tc::wait_warp(&mi.q_full, n & 1, &mi.quit, status)) return;
    if (!split) {
      int k = it++;
      if (!staged(k)) return;
      if (tc::elect()) {
        scores(0, 0, k);
        scores(1, 1, k);
        tc::commit(&mi.empty[k % Y::kStages]);
        if (nt == 1) tc::commit(&mi.q_empty);
      }
      __syncwarp();
      for (int i = 0; i < nt; ++i) {
        const int v = it++;
        const bool more = i + 1 < nt;
        if (more) k = it++;
        if (!staged(v) || (more && !staged(k))) return;
        if (!values(0, v, i == 0, [&] {
              if (more)
                scores(0, 0, k);
              else
                tc::commit(&mi.o_full[0]);
            }))
          return;
        if (!values(1, v, i == 0, [&] {
              tc::commit(&mi.empty[v % Y::kStages]);
              if (more) {
                scores(1, 1, k);
                tc::commit(&mi.empty[k % Y::kStages]);
                if (i + 2 == nt) tc::commit(&mi.q_empty);
              } else {
                tc::commit(&mi.o_full[1]);
              }
            }))
          return;
      }
    } else {
      for (int i = 0; i < min(nt, 2); ++i) {
        const int k = it++;
        if (!staged(k)) return;
        if (tc::elect()) {
          scores(0, i, k);
          tc::commit(&mi.empty[k % Y::kStages]);
          if (i + 1 == nt) tc::commit(&mi.q_empty);
        }
        __syncwarp();
      }
      for (int i = 0; i < nt; ++i) {
        const int t = i & 1, v = it++;
        if (!staged(v)) return;
        if (!values(t, v, i < 2, [&] {
              tc::commit(&mi.empty[v % Y::kStages]);
              if (i + 2 >= nt) tc::commit(&mi.o_full[t]);
            }))
          return;
        if (i + 2 < nt) {
          const int k = it++;
          if (!staged(k)) return;
          if (tc::elect()) {
            scores(0, t, k);
            tc::commit(&mi.empty[k % Y::kStages]);
            if (i + 3 == nt) tc::commit(&mi.q_empty);
          }
          __syncwarp();
        }
      }
    }
  }
}

// bit c: c < n
__device__ __forceinline__ uint32_t below(int n) {
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1;
}

// ---- softmax and epilogue of chain t (four warps, thread = row) --------------------------
template <int D>
__device__ __forceinline__ void soften(const Args& a, uint32_t smem, Misc& mi, uint32_t tmem,
                                       int t) {
  using Y = Lay<D>;
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3;
  const int r = wq * 32 + lane;  // row of the tile = lane of tensor memory
  const uint32_t lanes = (uint32_t)(wq * 32) << 16;
  const uint32_t s_col = tmem + lanes + t * 128;
  const int tok = r / a.G, gh = r - tok * a.G;
  int32_t* status = a.shape.status;
  int ns = 0, no[2] = {0, 0}, nmeet = 0;
  for (int n = 0;; ++n) {
    const int slot = n % kSegs;
    if (!tc::wait_warp(&mi.seg_full[slot], (n / kSegs) & 1, &mi.quit, status)) return;
    const ChunkSeg g = mi.seg[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&mi.seg_empty[slot]);
    if (!g.valid) return;
    const int nt = g.i1 - g.i0;
    const int mine = g.split ? (nt + 1 - t) >> 1 : nt;  // tiles of this chain
    const int tk = g.split ? tok : tok + t * a.TB;      // token of this row in the block
    const bool real = tok < a.TB && tk < g.ntok;
    const bool any = __any_sync(0xffffffffu, real);
    const int s = real ? g.s0 + tk : 0x3FFFFFFF;  // its slot (padding rows: no mask, unused)
    float m = -INFINITY, l = 0.f;
    // slots and pages that the block's rows together may see (window > 0)
    const int win = a.shape.window, sink = a.shape.sink;
    const int win_page = win > 0 ? max(0, g.s0 - win + 1) >> a.page_shift : 0;
    const int sink_pages = (sink + (1 << a.page_shift) - 1) >> a.page_shift;
    const uint64_t sl2 = tc::pair(a.scale_log2, a.scale_log2);
    for (int i = 0; i < mine; ++i) {
      // all that the scores are not needed for comes before they are waited for
      const int ti = g.split ? 2 * i + t : i;
      const int key0 = tile_of(g, g.i0 + ti) * kKeyTile;
      const int hi = s - key0, lo = win > 0 ? hi - win : -1, sk = sink - key0;
      // some key of the tile is hidden from some row of the warp
      const bool masked = __any_sync(
          0xffffffffu, real && (hi < kKeyTile - 1 || (lo >= 0 && sk <= min(lo, kKeyTile - 1))));
      // some row of V was not loaded or lies behind the sequence's end
      const bool ragged =
          (g.split || t == 0) &&
          (key0 + kKeyTile > g.L ||
           (win > 0 && (key0 < sink || (win_page << a.page_shift) > key0)));
      if (!tc::wait_warp(&mi.s_full[t], ns++ & 1, &mi.quit, status)) return;
      tc::fence_after();
      if (ragged) {
        // such rows would meet a probability of zero; they are zeroed because 0 * NaN is not
        // (only now: with this tile's scores there, what the stage held before has been read, so
        // that the parity names this fill)
        const int x = g.it0 + v_pos(g.split, nt, ti);
        if (!tc::wait_warp(&mi.full[x % Y::kStages], (x / Y::kStages) & 1, &mi.quit, status))
          return;
        const int key = key0 + r, page = key >> a.page_shift;
        if (key >= g.L || (page < win_page && page >= sink_pages)) {
          const uint32_t base = smem + Y::kRing + (x % Y::kStages) * Y::kTileBytes + r * 128;
#pragma unroll
          for (int e = 0; e < Y::kHalves * 8; ++e)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             base + (e >> 3) * kHalfBytes + (e & 7) * 16),
                         "r"(0)
                         : "memory");
        }
        tc::fence_async_smem();
      }
      if (any) {
        uint32_t x[128];
        tc::tmem_ld128(s_col, x);
        if (masked) {
#pragma unroll
          for (int c0 = 0; c0 < 128; c0 += 32) {
            const uint32_t see = below(hi + 1 - c0) & (~below(lo + 1 - c0) | below(sk - c0));
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((see >> c) & 1)) x[c0 + c] = 0xFF800000u;  // -inf
          }
        }
        float mxs[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mxs[e] = tc::max3(mxs[e], __uint_as_float(x[c + 2 * e]),
                              __uint_as_float(x[c + 2 * e + 1]));
        float mx = fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3]));
        mx *= a.scale_log2;
        if (i == 0) {
          m = mx;
        } else if (__any_sync(0xffffffffu, real && mx - m > 8.f)) {
          const float up = fmaxf(m, mx);
          const float f = up == -INFINITY ? 1.f : fast_exp2(m - up);
          m = up;
          l *= f;
          const uint32_t o_col = tmem + lanes + 256 + t * D;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tc::tmem_ld32(o_col + c0, o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tc::tmem_st32(o_col + c0, o);
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;
        const uint64_t off2 = tc::pair(off, off);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint64_t y[16];
          uint32_t p[16];
#pragma unroll
          for (int c = 0; c < 16; ++c)
            y[c] = tc::fma2(tc::pair(__uint_as_float(x[c0 + 2 * c]),
                                     __uint_as_float(x[c0 + 2 * c + 1])),
                            sl2, off2);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float p0, p1;
            tc::unpair(y[c], p0, p1);
            p0 = fast_exp2(p0);
            p1 = fast_exp2(p1);
            y[c] = tc::pair(p0, p1);
            p[c] = pack_bf16(p0, p1);
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) sum[c & 1] = tc::add2(sum[c & 1], y[c]);
          tc::tmem_st16(s_col + (c0 >> 1), p);
          if (c0 + 32 == kFirstKeys) {  // the product over the first keys may start
            tc::tmem_wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&mi.p_part[t]);
          }
        }
        float a0, a1, a2, a3;
        tc::unpair(sum[0], a0, a1);
        tc::unpair(sum[1], a2, a3);
        l += (a0 + a1) + (a2 + a3);
        tc::tmem_wait_st();
      } else {
        __syncwarp();  // every lane's row of V is zeroed before this warp hands the tile over
        if (lane == 0) mbar_arrive(&mi.p_part[t]);
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&mi.p_full[t]);
    }
    // ---- results: whole items are normalised and rounded, pieces leave (O, m, l)
    const int64_t orow = (int64_t)(g.row0 + tk) * a.Hq + g.h * a.G + gh;
    const size_t prow = (size_t)max(g.part, 0) * a.rows_cap + (g.split ? 0 : t * 128) + r;
    int c_from = 0, c_to = D;
    float f0 = 1.f, f1 = 0.f;  // weights of the two accumulators
    uint32_t o_col = tmem + lanes + 256 + t * D;
    if (!g.split) {
      if (!tc::wait_warp(&mi.o_full[t], no[t]++ & 1, &mi.quit, status)) return;
      ++no[1 - t];  // the other chain's completes too; its warps wait for it
    } else {
      // both chains hold a state of the same rows: exchange (m, l), then each group of warps
      // writes half of the channels
      mi.ml[t][r] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&mi.meet);
      if (!tc::wait_warp(&mi.meet, nmeet++ & 1, &mi.quit, status)) return;
      if (!tc::wait_warp(&mi.o_full[0], no[0]++ & 1, &mi.quit, status)) return;
      if (nt > 1 && !tc::wait_warp(&mi.o_full[1], no[1]++ & 1, &mi.quit, status)) return;
      const float2 s0 = mi.ml[0][r], s1 = mi.ml[1][r];
      m = fmaxf(s0.x, s1.x);
      f0 = s0.x == -INFINITY ? 0.f : fast_exp2(s0.x - m);
      f1 = s1.x == -INFINITY ? 0.f : fast_exp2(s1.x - m);
      l = s0.y * f0 + s1.y * f1;
      o_col = tmem + lanes + 256;
      c_from = t * (D / 2);
      c_to = c_from + D / 2;
    }
    tc::fence_after();
    if (any) {
      if (g.part < 0) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        f0 *= inv;
        f1 *= inv;
      }
#pragma unroll 1
      for (int c0 = c_from; c0 < c_to; c0 += 32) {
        uint32_t o[32];
        tc::tmem_ld32(o_col + c0, o);
        float v[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(o[c]) * f0;
        if (g.split && nt > 1) {
          tc::tmem_ld32(o_col + D + c0, o);
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] += __uint_as_float(o[c]) * f1;
        }
        if (g.part >= 0) {
          // [8 rows][D / 4][8][4]: a warp's store is four runs of 128 bytes
          float4* dst = reinterpret_cast<float4*>(a.part_o) +
                        ((prow >> 3) * (D / 4) + (c0 >> 2)) * 8 + (r & 7);
          if (real) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              dst[c * 8] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
          }
        } else {
          // four lanes turn their rows' 64 bytes, so that a store covers 64 bytes of a row
          uint32_t w[4][4];  // [16-byte unit][word]
#pragma unroll
          for (int c = 0; c < 16; ++c) w[c >> 2][c & 3] = pack_bf16(v[2 * c], v[2 * c + 1]);
#pragma unroll
          for (int o2 = 1; o2 < 4; o2 <<= 1)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (!(u & o2)) {
                const bool odd = lane & o2;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t got = __shfl_xor_sync(
                      0xffffffffu, odd ? w[u][e] : w[u | o2][e], o2);
                  if (odd)
                    w[u][e] = got;
                  else
                    w[u | o2][e] = got;
                }
              }
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // row k of the four
            const int64_t to = __shfl_sync(0xffffffffu, orow, (lane & ~3) + k);
            if (__shfl_sync(0xffffffffu, real, (lane & ~3) + k))
              *reinterpret_cast<uint4*>(a.out + to * D + c0 + (lane & 3) * 8) =
                  make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
          }
        }
        __syncwarp();
      }
      if (real && (!g.split || t == 0)) {
        if (g.part >= 0)
          a.part_ml[prow] = make_float2(m, l);
        else
          a.lse[orow] = l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
    }
    tc::fence_before();
    if (g.split) {
      // the other chain's accumulator and state may be overwritten once all have read them
      __syncwarp();
      if (lane == 0) mbar_arrive(&mi.meet);
      if (!tc::wait_warp(&mi.meet, nmeet++ & 1, &mi.quit, status)) return;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const Args a) {
  using Y = Lay<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = smem_u32(smem_raw);
  Misc& mi = *reinterpret_cast<Misc*>(smem_raw + Y::kMisc);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 352) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  if (tid == 0) {
    for (int i = 0; i < Y::kStages; ++i) {
      mbar_init(&mi.full[i], 1);
      mbar_init(&mi.empty[i], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&mi.seg_full[i], 1);
      mbar_init(&mi.seg_empty[i], 10);  // V's, the products' and the eight softmax warps
    }
    mbar_init(&mi.q_full, 1);
    mbar_init(&mi.q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&mi.s_full[t], 1);
      mbar_init(&mi.p_part[t], 4);
      mbar_init(&mi.p_full[t], 4);
      mbar_init(&mi.o_full[t], 1);
    }
    mbar_init(&mi.meet, 8);
    mbar_init(&mi.drain, 1);
    mi.quit = 0;
    fence_mbar_init();
    // everything below reads what earlier kernels of the stream wrote
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  if (warp == 8) tc::tmem_alloc_all(&mi.tmem);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = mi.tmem;
  if (warp < 8) {
    tc::regs_up<kSoftmaxRegs>();
    soften<D>(a, smem, mi, tmem, warp >> 2);
  } else {
    tc::regs_down<kOtherRegs>();
    if (warp == 8) {
      multiply<D>(a, smem, mi, tmem);
      __syncwarp();
      if (tc::elect()) {
        tc::commit(&mi.drain);
        mbar_wait(&mi.drain, 0);
      }
    } else if (warp < 11) {
      produce<D>(a, smem, mi, &qmap, warp == 9 ? &kmap : &vmap, warp == 10);
    }
    __syncwarp();
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 8) tc::tmem_free_all(tmem);
  asm volatile("griddepcontrol.launch_dependents;");
}

// Joins the pieces of the cut items: out = sum_p 2^(m_p - M) O_p / L.  A CTA has eight rows of
// one item; its eight warps take every eighth piece, a lane one row and every fourth 16-byte
// group of its channels; the warps' sums meet in shared memory in warp order.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const float4* __restrict__ part_o,
                                                   const float2* __restrict__ part_ml,
                                                   const ChunkCut* __restrict__ cut,
                                                   uint16_t* __restrict__ out,
                                                   float* __restrict__ lse, int rows_cap, int Hq,
                                                   int G, int TB) {
  constexpr int C = D / 16;  // 16-byte groups of a lane
  __shared__ float4 acc_s[8][D / 4][8];
  __shared__ float2 ml_s[8][8];
  if (threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x;
  const ChunkCut k = cut[c];
  if (k.nparts <= 0) return;
  const int r0 = blockIdx.y * 8;
  {  // nothing to do behind the item's last row
    const int tok = (r0 & 127) / G + (r0 >> 7) * TB;
    if (tok >= k.ntok) return;
  }
  const int r8 = lane & 7, sub = lane >> 3;
  auto slot = [&](int p) {
    return ((size_t)(p == 0 ? 2 * c + 1 : 2 * (c + p)) * rows_cap + r0);
  };
  float M = -INFINITY, l = 0.f;
  float4 acc[C];
#pragma unroll
  for (int e = 0; e < C; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = warp + 8 * sub; p < k.nparts; p += 32) M = fmaxf(M, part_ml[slot(p) + r8].x);
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
#pragma unroll 2
  for (int p = warp; p < k.nparts; p += 8) {
    const size_t at = slot(p);
    const float2 ml = part_ml[at + r8];
    const float4* src = part_o + ((at >> 3) * (D / 4) + sub) * 8 + r8;
    const float f = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
    l += f * ml.y;
#pragma unroll
    for (int e = 0; e < C; ++e) {
      const float4 v = src[e * 32];
      acc[e].x += f * v.x;
      acc[e].y += f * v.y;
      acc[e].z += f * v.z;
      acc[e].w += f * v.w;
    }
  }
#pragma unroll
  for (int e = 0; e < C; ++e) acc_s[warp][4 * e + sub][r8] = acc[e];
  if (sub == 0) ml_s[warp][r8] = make_float2(M, l);
  __syncthreads();
  const int row = warp, r = r0 + row;  // a warp writes one row
  const int tok = (r & 127) / G, gh = (r & 127) % G, tk = tok + (r >> 7) * TB;
  if (tok >= TB || tk >= k.ntok) return;
  float W = -INFINITY;
#pragma unroll
  for (int w = 0; w < 8; ++w) W = fmaxf(W, ml_s[w][row].x);
  l = 0.f;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float2 ml = ml_s[w][row];
    if (ml.x == -INFINITY) continue;
    const float f = fast_exp2(ml.x - W);
    l += f * ml.y;
    if (lane < D / 4) {
      const float4 v = acc_s[w][lane][row];
      sum.x += f * v.x;
      sum.y += f * v.y;
      sum.z += f * v.z;
      sum.w += f * v.w;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t orow = (int64_t)(k.row0 + tk) * Hq + k.h * G + gh;
  if (lane < D / 4)
    reinterpret_cast<uint2*>(out + orow * D)[lane] =
        make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
  if (lane == 0)
    lse[orow] = l > 0.f ? (W + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

static int rows_cap(const sa_geom& g, int n_tokens) {
  const int G = g.Hq / g.Hkv, TB = 128 / G;
  return n_tokens > TB ? 256 : ((n_tokens > 0 ? n_tokens : 1) * G + 7) & ~7;
}

template <int D>
static cudaError_t run(const sa_geom& g, const ChunkCall& c, cudaStream_t stream) {
  using Y = Lay<D>;
  Args a;
  a.G = g.Hq / g.Hkv;
  a.TB = 128 / a.G;
  a.shape.cu_new = c.cu_new;
  a.shape.seq_lens = c.seq_lens;
  a.shape.n_tokens = c.n_tokens;
  a.shape.B = g.B;
  a.shape.H = g.Hkv;
  a.shape.inner = 1;
  a.shape.BT = 2 * a.TB;
  a.shape.ST = a.TB;
  a.shape.extra = 2;
  const int longest = 1 << 30;  // no sequence is longer
  a.shape.sink = c.sink < longest ? c.sink : longest;
  a.shape.window = c.window < longest ? c.window : longest;
  a.shape.cap = (int64_t)g.max_pages * g.P;
  a.shape.status = c.status;
  a.page_table = c.page_table;
  a.out = static_cast<uint16_t*>(c.out);
  a.lse = c.lse;
  a.rows_cap = rows_cap(g, c.n_tokens);
  const size_t slots = 2 * (size_t)c.n_sm * a.rows_cap;
  uint8_t* w = c.scratch;
  a.cut = reinterpret_cast<ChunkCut*>(w);
  w += chunk_up256(c.n_sm * sizeof(ChunkCut));
  a.part_ml = reinterpret_cast<float2*>(w);
  w += chunk_up256(slots * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(w);
  a.Hq = g.Hq;
  a.Hkv = g.Hkv;
  a.P = g.P;
  a.page_shift = g.P == 16 ? 4 : g.P == 32 ? 5 : 6;
  a.max_pages = g.max_pages;
  a.n_pool = g.n_pool;
  a.scale_log2 = c.scale * 1.4426950408889634f;
  CUtensorMap qm, km, vm;
  const uint64_t rows = (uint64_t)g.n_pool * g.Hkv * g.P;
  if (!encode_heads_tmap(&qm, c.q, D, g.Hq, c.n_tokens, 64, a.G, a.TB) ||
      !encode_rows_tmap(&km, c.k_cache, D, rows, 64, g.P) ||
      !encode_rows_tmap(&vm, c.v_cache, D, rows, 64, g.P))
    return cudaErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(attend_kernel<D>);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Y::kSmem);
  if (e != cudaSuccess) return e;
  void* args[] = {&qm, &km, &vm, &a};
  if ((e = chunk_launch(fn, dim3(c.n_sm), kThreads, Y::kSmem, stream, args)) != cudaSuccess) return e;
  void* jargs[] = {&a.part_o, &a.part_ml, &a.cut, &a.out,
                   &a.lse,    &a.rows_cap, &a.Hq, &a.G, &a.TB};
  return chunk_launch(reinterpret_cast<const void*>(join_kernel<D>),
                      dim3(c.n_sm, a.rows_cap / 8), 256, 0, stream, jargs);
}

static size_t bytes(const sa_geom& g, int n_tokens, int n_sm) {
  const size_t slots = 2 * (size_t)n_sm * rows_cap(g, n_tokens);
  return chunk_up256(n_sm * sizeof(ChunkCut)) + chunk_up256(slots * sizeof(float2)) + slots * g.Dv * 4;
}

}  // namespace chunk

size_t chunk_workspace_bytes(const sa_geom& g, int n_tokens, int n_sm) {
  return g.v_aliases_k ? chunk_mla_workspace_bytes(n_sm) : chunk::bytes(g, n_tokens, n_sm);
}

cudaError_t launch_chunk(const sa_geom& g, const ChunkCall& c, cudaStream_t stream) {
  switch (g.Dk) {
    case 64: return chunk::run<64>(g, c, stream);
    case 128: return chunk::run<128>(g, c, stream);
    case 576: return launch_chunk_mla(g, c, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sa
