// sa_chunk_mla.cu -- exact attention of a ragged chunk of new tokens over the paged cache,
// latent geometry (128 query heads share one 576-wide key per token, V its first 512
// channels), on the 5th-generation tensor cores.
//
// Method: as sa_chunk.cu.  A tile is one token's 128 heads against 128 keys, worked on by a pair
// of CTAs (cta_group::2): each CTA has 64 of the heads as its rows, so that
//   S = Q K^T     (128 x 128 x 576)  takes 64 columns of its tensor memory,
//   O += P V      (128 x 512 x 128)  takes 256,
// and two score tiles fit beside the accumulator; one CTA alone would need all 512 columns for
// O.  (Alone, with 64 heads a CTA and both products transposed, every product has N = 64 and
// takes as long as one with N = 128: 1.60 ms instead of 0.90 for 256 + 100 rows at 16K / 5K.)
// Of a key tile a CTA loads what its half of the products reads: 64 keys of all 576 channels
// as B of the first (72 KB), 256 channels of all 128 keys as B of the second (64 KB), with
// 72 KB of queries and 16 KB of probabilities.  The next tile's keys come in while this one's
// softmax and second product run, the next values during the next scores, both in parts that
// follow the products through the one buffer.  Copies of both CTAs are counted at the even one,
// which issues the products.
// A thread has one row and 32 of its 128 scores, so a row's maximum crosses four threads.  It
// is only taken when some score exceeds the maximum in use by more than 2^8 (which a vote
// finds); sums stay in the threads until the end.
// Warps 0-3 and 4-7: softmax; 8: issues the products (even CTA); 9: work list, queries and
// keys; 10: values.
// Probabilities are bf16 in the second product, as there.
// Measured on a B200 in short graphs at up to 1965 MHz: 256 + 100 rows at 16384 / 5001 tokens 0.90 ms
// (1.4 PFLOP/s, tensor pipe 78% busy); sixteen decode rows at 16384 80 us (tensor pipe 49%, DRAM
// 52%: about 3000 cycles a tile against 2176 for its products, the first tile's 32 MB for all CTAs
// and the joining).  At sustained clocks, on changing inputs: 1.05 ms and 94 us.
#include "sa_chunk.cuh"
#include "sa_internal.h"
#include "sa_tc.cuh"

namespace sa {

namespace chunk_mla {

constexpr int kD = 576, kDv = 512, kHeads = 128;
constexpr int kHalf = 64;  // heads of a CTA, and keys that it loads for the scores
constexpr int kThreads = 384;
constexpr int kSegs = 2;
// parts of a key tile that are loaded and given back by themselves: three slices of 64 channels
// for the scores, one block of 256 channels of the values
constexpr int kKGroups = 3, kVGroups = 2;
constexpr uint32_t kQSlice = kHalf * 128;     // 64 rows of 64 channels
constexpr uint32_t kVSlice = kKeyTile * 128;  // 128 keys' 64 channels
constexpr uint32_t kKeys = 9 * kQSlice;       // queries first
constexpr uint32_t kValues = 2 * 9 * kQSlice;
constexpr uint32_t kP = kValues + 4 * kVSlice;  // [2 key halves][64 rows][64 keys]
constexpr uint32_t kMisc = kP + 2 * kQSlice;
constexpr uint32_t kO = 128;  // column of O; the two score tiles are columns 0-63 and 64-127

struct Misc {
  float red[4][64];  // of a row's four threads
  ChunkSeg seg[kSegs];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full, k_full[kKGroups], v_full[kVGroups];  // at the even CTA, for both
  uint64_t q_empty, k_empty[kKGroups], v_empty[kVGroups], v_here;
  uint64_t s_full[2], p_full, o_done, drain, meet;
  uint32_t tmem;
  int quit;
  int vote[3];
};
constexpr uint32_t kSmem = kMisc + sizeof(Misc);
static_assert(kSmem <= 232448, "shared memory of a CTA");

struct Args {
  ChunkShape shape;
  const int32_t* page_table;
  const uint8_t* kv;
  uint16_t* out;
  float* lse;
  float* part_o;    // [2 n_cta][512 / 4 channels][64 heads][4]
  float2* part_ml;  // [2 n_cta][64]
  ChunkCut* cut;    // [n_cta]
  int P, page_shift, max_pages, n_pool;
  float scale_log2;
};

__device__ __forceinline__ int tile_of(const ChunkSeg& g, int i) {
  return i < g.na ? i : i - g.na + g.bs;
}

// pages [0, sink_pages) and from win_page on hold what the segment's row may see
struct Pages {
  int sink_pages, win_page;
  __device__ __forceinline__ Pages(const Args& a, const ChunkSeg& g) {
    win_page = a.shape.window > 0 ? max(0, g.s0 - a.shape.window + 1) >> a.page_shift : 0;
    sink_pages = (a.shape.sink + (1 << a.page_shift) - 1) >> a.page_shift;
  }
  __device__ __forceinline__ bool wanted(int lp) const {
    return lp >= win_page || lp < sink_pages;
  }
};

// Copies of one piece's tiles, counted at the even CTA.  V: this CTA's 128 channels of each block
// of all keys, else its 64 keys of all channels; a lane copies one slice of one page.  `it`: tiles
// before the piece.
template <bool V>
__device__ __forceinline__ bool load_tiles(const Args& a, uint32_t smem, Misc& mi,
                                           const ChunkSeg& g, const CUtensorMap* map, int it,
                                           int rank) {
  constexpr int kGroups = V ? kVGroups : kKGroups, kSlices = V ? 2 : 3;
  const int lane = threadIdx.x & 31, shift = a.page_shift;
  const int ppt = kKeyTile >> shift;                // pages of a tile (2, 4 or 8),
  const int mine = V ? ppt : ppt >> 1;              // of this CTA's copies
  const int from = V ? 0 : rank * mine;             // and the first of those
  const int nt = g.i1 - g.i0, last_page = (g.L - 1) >> shift;
  const Pages pages(a, g);
  const int32_t* row = a.page_table + (size_t)g.b * a.max_pages;
  const uint64_t policy = tc::l2_normal();
  uint64_t* full = V ? mi.v_full : mi.k_full;
  uint64_t* empty = V ? mi.v_empty : mi.k_empty;
  const uint32_t full_at = tc::at_first(full);
  const int pg = lane / kSlices, sl = lane % kSlices;
  // lane p < ppt looks up page p of a tile, two tiles ahead; entries are checked when used
  auto wanted = [&](int i, int& lp) {
    lp = tile_of(g, g.i0 + i) * ppt + lane;
    return lane < ppt && lp <= last_page && pages.wanted(lp);
  };
  int p0 = -1, p1 = -1, lp;
  for (int i = -2; i < nt; ++i) {
    int p2 = -1;
    if (i + 2 < nt && wanted(i + 2, lp)) {
      p2 = row[lp];
      if (!V && g.once && p2 >= 0 && p2 < a.n_pool && lane / mine == rank)  // ask it into L2
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                         a.kv + (size_t)p2 * a.P * (kD * 2)),
                     "r"(a.P * (kD * 2))
                     : "memory");
    }
    if (i >= 0) {
      bool copy = wanted(i, lp);
      if (copy && (p0 < 0 || p0 >= a.n_pool)) {
        if ((lp << shift) <= g.s0) report(a.shape.status, SA_ERR_DEVICE_CHECK);
        copy = false;
      }
      const unsigned have = __ballot_sync(0xffffffffu, copy);
      const int ph = __shfl_sync(0xffffffffu, p0, from + (pg < mine ? pg : 0));
      const bool go = pg < mine && ((have >> (from + pg)) & 1);
      // bytes of both CTAs: each half's pages once (V: every page twice)
      const uint32_t bytes = __popc(have) * (V ? 2 : 1) * kSlices * a.P * 128;
      for (int gr = 0; gr < kGroups; ++gr) {
        if (it + i > 0 &&
            !tc::wait_warp(&empty[gr], (it + i - 1) & 1, &mi.quit, a.shape.status))
          return false;
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&full[gr], bytes);
        __syncwarp();
        const int slice = gr * kSlices + sl;
        if (go)
          tc::pair_tma_2d(smem + (V ? kValues + slice * kVSlice : kKeys + slice * kQSlice) +
                              ((uint32_t)pg << shift) * 128,
                          map, V ? gr * 256 + rank * 128 + sl * 64 : slice * 64, ph << shift,
                          full_at + gr * 8, policy);
      }
    }
    p0 = p1;
    p1 = p2;
  }
  return true;
}

__device__ __forceinline__ void produce_k(const Args& a, uint32_t smem, Misc& mi,
                                          const CUtensorMap* qmap, const CUtensorMap* kmap,
                                          int rank) {
  const int lane = threadIdx.x & 31;
  int32_t* status = a.shape.status;
  ChunkSched sched;
  if (lane == 0) a.cut[blockIdx.x].nparts = 0;
  sched.init(a.shape, blockIdx.x, gridDim.x);
  int it = 0;  // tiles loaded
  for (int n = 0;; ++n) {
    const int slot = n % kSegs;
    if (n >= kSegs &&
        !tc::wait_warp(&mi.seg_empty[slot], (n / kSegs - 1) & 1, &mi.quit, status))
      break;
    ChunkSeg g;
    const bool more = sched.next(g);
    if (!more) g.valid = 0;
    g.it0 = it;
    if (lane == 0) {
      mi.seg[slot] = g;
      mbar_arrive(&mi.seg_full[slot]);
      if (more && g.nparts > 0) a.cut[blockIdx.x] = ChunkCut{g.nparts, g.row0, g.ntok, g.h};
    }
    if (!more) return;
    if (n > 0 && !tc::wait_warp(&mi.q_empty, (n - 1) & 1, &mi.quit, status)) break;
    if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&mi.q_full, 2 * 9 * kQSlice);
    __syncwarp();
    if (lane < 9)
      tc::pair_tma_3d(smem + lane * kQSlice, qmap, lane * 64, g.h * kHalf, g.row0,
                      tc::at_first(&mi.q_full));
    if (!load_tiles<false>(a, smem, mi, g, kmap, it, rank)) break;
    it += g.i1 - g.i0;
  }
  // given up: copies in flight land (bounded) before shared memory goes away
  if (rank == 0)
    for (int ph = 0; ph < 2; ++ph) {
      for (int gr = 0; gr < kKGroups; ++gr) mbar_wait(&mi.k_full[gr], ph);
      mbar_wait(&mi.q_full, ph);
    }
}

// Reads the list as the other warps do: the next piece, or false.
__device__ __forceinline__ bool next_piece(Misc& mi, int n, int32_t* status, ChunkSeg& g) {
  const int slot = n % kSegs;
  if (!tc::wait_warp(&mi.seg_full[slot], (n / kSegs) & 1, &mi.quit, status)) return false;
  g = mi.seg[slot];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&mi.seg_empty[slot]);
  return g.valid != 0;
}

__device__ __forceinline__ void produce_v(const Args& a, uint32_t smem, Misc& mi,
                                          const CUtensorMap* kmap, int rank) {
  ChunkSeg g;
  for (int n = 0; next_piece(mi, n, a.shape.status, g); ++n)
    if (!load_tiles<true>(a, smem, mi, g, kmap, g.it0, rank)) break;
  if (rank == 0 && *(volatile int*)&mi.quit)
    for (int ph = 0; ph < 2; ++ph)
      for (int gr = 0; gr < kVGroups; ++gr) mbar_wait(&mi.v_full[gr], ph);
}

// The even CTA: all products.
__device__ __forceinline__ void multiply(const Args& a, uint32_t smem, Misc& mi, uint32_t tmem) {
  constexpr uint32_t id_s = tc::idesc(128, kKeyTile, false, false);
  constexpr uint32_t id_o = tc::idesc(128, 256, false, true);
  int32_t* status = a.shape.status;
  int it = 0;
  auto arrived = [&](uint64_t* bar, uint32_t parity) {
    const bool r = tc::wait_warp(bar, parity & 1, &mi.quit, status);
    tc::fence_after();
    return r;
  };
  auto scores = [&](int x, bool last) -> bool {  // S of tile x
#pragma unroll
    for (int gr = 0; gr < kKGroups; ++gr) {
      if (!arrived(&mi.k_full[gr], x)) return false;
      if (tc::elect()) {
#pragma unroll
        for (int kk = 12 * gr; kk < 12 * gr + 12; ++kk) {
          const uint32_t o = (kk >> 2) * kQSlice + (kk & 3) * 32;
          tc::pair_mma(tmem + (x & 1) * 64, tc::desc(smem + o), tc::desc(smem + kKeys + o), id_s,
                       kk != 0);
        }
        tc::pair_commit(&mi.k_empty[gr]);
        if (gr == kKGroups - 1) {
          tc::pair_commit(&mi.s_full[x & 1]);
          if (last) tc::pair_commit(&mi.q_empty);
        }
      }
      __syncwarp();
    }
    return true;
  };
  for (int n = 0;; ++n) {
    ChunkSeg g;
    if (!next_piece(mi, n, status, g)) return;
    const int nt = __shfl_sync(0xffffffffu, g.i1 - g.i0, 0);
    if (!arrived(&mi.q_full, n) || !scores(it, nt == 1)) return;
    for (int i = 0; i < nt; ++i, ++it) {
      if (i + 1 < nt && !scores(it + 1, i + 2 == nt)) return;
      if (!arrived(&mi.v_full[0], it) || !arrived(&mi.v_full[1], it)) return;
      if (tc::elect()) tc::pair_commit(&mi.v_here);
      __syncwarp();
      if (!arrived(&mi.p_full, it)) return;
      if (tc::elect()) {
#pragma unroll
        for (int cb = 0; cb < 2; ++cb) {
#pragma unroll
          for (int kk = 0; kk < kKeyTile / 16; ++kk)
            tc::pair_mma(tmem + kO + cb * 128,
                         tc::desc(smem + kP + (kk >> 2) * kQSlice + (kk & 3) * 32),
                         tc::desc(smem + kValues + 2 * cb * kVSlice + kk * 2048, kVSlice), id_o,
                         !(i == 0 && kk == 0));
          tc::pair_commit(&mi.v_empty[cb]);
        }
        tc::pair_commit(&mi.o_done);
      }
      __syncwarp();
    }
  }
}

// softmax and epilogue: columns [32 t, 32 t + 32) of a score tile's 64, accumulator block t
__device__ __forceinline__ void soften(const Args& a, uint32_t smem, Misc& mi, uint32_t tmem,
                                       int t, int rank) {
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3;
  const int l128 = wq * 32 + lane;                   // lane of tensor memory
  const int row = l128 & 63, second = l128 >> 6;     // head of the CTA; half of the columns
  const uint32_t lanes = (uint32_t)(wq * 32) << 16;
  const int key_in = second * 64 + t * 32;           // first key of this thread in a tile
  const uint32_t p_row = smem + kP + second * kQSlice + row * 128;
  int32_t* status = a.shape.status;
  int it = 0, nmeet = 0;
  auto meet = [&]() -> bool {  // the eight warps; shared writes become visible
    __syncwarp();
    if (lane == 0) mbar_arrive(&mi.meet);
    return tc::wait_warp(&mi.meet, nmeet++ & 1, &mi.quit, status);
  };
  ChunkSeg g;
  for (int n = 0; next_piece(mi, n, status, g); ++n) {
    const int nt = g.i1 - g.i0, s = g.s0;
    const Pages pages(a, g);
    float l = 0.f, m = -INFINITY;
    for (int i = 0; i < nt; ++i, ++it) {
      // all that the scores are not needed for comes before they are waited for
      const int key0 = tile_of(g, g.i0 + i) * kKeyTile;
      const int hi = s - key0 - key_in;
      const int lo = a.shape.window > 0 ? hi - a.shape.window : -1;
      const int sk = a.shape.sink - key0 - key_in;
      uint32_t see = 0xFFFFFFFFu;
      if (hi < 31 || (lo >= 0 && sk <= min(lo, 31))) {
        auto below = [](int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1; };
        see = below(hi + 1) & (~below(lo + 1) | below(sk));
      }
      const bool stored = key0 + l128 < g.L && pages.wanted((key0 + l128) >> a.page_shift);
      const bool ragged = !__all_sync(0xffffffffu, stored);
      if (!tc::wait_warp(&mi.s_full[it & 1], (it >> 1) & 1, &mi.quit, status)) return;
      tc::fence_after();
      if (ragged) {
        // keys without a loaded row meet a probability of zero; 0 * NaN is not 0.  (The values
        // before these have been multiplied: that was awaited for the last tile's P.)
        if (it > 0 && !tc::wait_warp(&mi.o_done, (it - 1) & 1, &mi.quit, status)) return;
        if (!tc::wait_warp(&mi.v_here, it & 1, &mi.quit, status)) return;
        if (!stored) {
          const uint32_t base = smem + kValues + 2 * t * kVSlice + l128 * 128;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             base + (e >> 3) * kVSlice + (e & 7) * 16),
                         "r"(0)
                         : "memory");
        }
        __syncwarp();
      }
      uint32_t x[32];
      tc::tmem_ld32(tmem + lanes + (it & 1) * 64 + 32 * t, x);
      if (see != 0xFFFFFFFFu) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (!((see >> c) & 1)) x[c] = 0xFF800000u;  // -inf
      }
      __syncwarp();
      float mxs[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 32; c += 4)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          mxs[e] = tc::max3(mxs[e], __uint_as_float(x[c + 2 * e]),
                            __uint_as_float(x[c + 2 * e + 1]));
      const float mx = fmaxf(mxs[0], mxs[1]) * a.scale_log2;
      // the vote goes round while the exponentials are computed: flag it % 3 is raised; flag
      // (it + 1) % 3 was last read before the last vote
      const bool over = __any_sync(0xffffffffu, mx > -INFINITY && !(mx - m <= 8.f));
      if (lane == 0) {
        if (threadIdx.x == 0) *(volatile int*)&mi.vote[(it + 1) % 3] = 0;
        if (over) *(volatile int*)&mi.vote[it % 3] = 1;
        mbar_arrive(&mi.meet);
      }
      float p[32], add;
      uint32_t w[16];
      auto probabilities = [&]() {
        const float off = m == -INFINITY ? 0.f : -m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 32; ++c)
          p[c] = fast_exp2(fmaf(__uint_as_float(x[c]), a.scale_log2, off));
#pragma unroll
        for (int c = 0; c < 16; ++c) w[c] = pack_bf16(p[2 * c], p[2 * c + 1]);
#pragma unroll
        for (int c = 0; c < 32; ++c) sum[c & 3] += p[c];
        add = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      };
      probabilities();
      if (!tc::wait_warp(&mi.meet, nmeet++ & 1, &mi.quit, status)) return;
      // P's place and O are free once the last product with V is done
      if (it > 0 && !tc::wait_warp(&mi.o_done, (it - 1) & 1, &mi.quit, status)) return;
      if (*(volatile int*)&mi.vote[it % 3]) {
        // raise the maximum of every row to what its four threads have seen
        mi.red[t * 2 + second][row] = mx;
        if (!meet()) return;
        const float up = fmaxf(fmaxf(fmaxf(mi.red[0][row], mi.red[1][row]),
                                     fmaxf(mi.red[2][row], mi.red[3][row])),
                               m);
        const float f = up == -INFINITY ? 1.f : fast_exp2(m - up);
        m = up;
        l *= f;
        if (i > 0) {
          tc::fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < 128; c0 += 32) {
            uint32_t o[32];
            const uint32_t col = tmem + lanes + kO + t * 128 + c0;
            tc::tmem_ld32(col, o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tc::tmem_st32(col, o);
          }
          tc::tmem_wait_st();
        }
        probabilities();
        if (!meet()) return;  // red may be written again
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         p_row + (((4 * t + u) ^ (row & 7)) << 4)),
                     "r"(w[4 * u]), "r"(w[4 * u + 1]), "r"(w[4 * u + 2]), "r"(w[4 * u + 3])
                     : "memory");
      tc::fence_async_smem();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::arrive_at_first(&mi.p_full);
      l += add;
    }
    // ---- results
    mi.red[t * 2 + second][row] = l;
    if (!meet()) return;
    l = (mi.red[0][row] + mi.red[1][row]) + (mi.red[2][row] + mi.red[3][row]);
    if (!tc::wait_warp(&mi.o_done, (it - 1) & 1, &mi.quit, status)) return;
    tc::fence_after();
    const int64_t orow = (int64_t)g.row0 * kHeads + rank * kHalf + row;
    const int ch0 = t * 256 + second * 128;  // channels of this thread's columns
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < 128; c0 += 32) {
      uint32_t o[32];
      tc::tmem_ld32(tmem + lanes + kO + t * 128 + c0, o);
      if (g.part >= 0) {
        float4* dst = reinterpret_cast<float4*>(a.part_o) +
                      ((size_t)g.part * (kDv / 4) + ((ch0 + c0) >> 2)) * kHalf + row;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          dst[c * kHalf] =
              make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                          __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
      } else {
        // four lanes turn their rows' 64 bytes, so that a store covers 64 bytes of a row
        uint32_t v[4][4];  // [16-byte unit][word]
#pragma unroll
        for (int c = 0; c < 16; ++c)
          v[c >> 2][c & 3] = pack_bf16(__uint_as_float(o[2 * c]) * inv,
                                       __uint_as_float(o[2 * c + 1]) * inv);
#pragma unroll
        for (int o2 = 1; o2 < 4; o2 <<= 1)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (!(u & o2)) {
              const bool odd = lane & o2;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t got =
                    __shfl_xor_sync(0xffffffffu, odd ? v[u][e] : v[u | o2][e], o2);
                if (odd)
                  v[u][e] = got;
                else
                  v[u | o2][e] = got;
              }
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)  // row k of the four
          *reinterpret_cast<uint4*>(a.out + (orow - (lane & 3) + k) * kDv + ch0 + c0 +
                                    (lane & 3) * 8) =
              make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
      }
      __syncwarp();
    }
    if (t == 0 && second == 0) {
      if (g.part >= 0)
        a.part_ml[(size_t)g.part * kHalf + row] = make_float2(m, l);
      else
        a.lse[orow] = l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    tc::fence_before();
    if (!meet()) return;  // red may be written again
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = smem_u32(smem_raw);
  Misc& mi = *reinterpret_cast<Misc*>(smem_raw + kMisc);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rank = (int)tc::cluster_rank();
  if (tid == 352) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
  }
  if (tid == 0) {
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&mi.seg_full[i], 1);
      mbar_init(&mi.seg_empty[i], 10 - rank);  // softmax, values', even: products' warp
    }
    mbar_init(&mi.q_full, 1);
    mbar_init(&mi.q_empty, 1);
    for (int i = 0; i < kKGroups; ++i) {
      mbar_init(&mi.k_full[i], 1);
      mbar_init(&mi.k_empty[i], 1);
    }
    for (int i = 0; i < kVGroups; ++i) {
      mbar_init(&mi.v_full[i], 1);
      mbar_init(&mi.v_empty[i], 1);
    }
    mbar_init(&mi.v_here, 1);
    mbar_init(&mi.s_full[0], 1);
    mbar_init(&mi.s_full[1], 1);
    mbar_init(&mi.p_full, 16);  // the softmax warps of both CTAs
    mbar_init(&mi.o_done, 1);
    mbar_init(&mi.drain, 1);
    mbar_init(&mi.meet, 8);
    mi.quit = 0;
    for (int i = 0; i < 3; ++i) mi.vote[i] = 0;
    fence_mbar_init();
    // everything below reads what earlier kernels of the stream wrote
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  if (warp == 8) tc::pair_tmem_alloc_all(&mi.tmem);
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();  // both CTAs' barriers are there
  tc::fence_after();
  const uint32_t tmem = mi.tmem;
  if (warp < 8) {
    soften(a, smem, mi, tmem, warp >> 2, rank);
  } else if (warp == 8) {
    if (rank == 0) {
      multiply(a, smem, mi, tmem);
      __syncwarp();
      if (tc::elect()) tc::pair_commit_here(&mi.drain);
      __syncwarp();
      mbar_wait(&mi.drain, 0);
    }
  } else if (warp == 9) {
    produce_k(a, smem, mi, &qmap, &kmap, rank);
  } else if (warp == 10) {
    produce_v(a, smem, mi, &kmap, rank);
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();  // neither CTA reads the other's memory or arrives there any more
  if (warp == 8) tc::pair_tmem_free_all(tmem);
  asm volatile("griddepcontrol.launch_dependents;");
}

// Joins the pieces of the cut items, in piece order.  CTA = (cut item, 64 channels): a thread sums
// 16 channels of one head.
__global__ void __launch_bounds__(256) join_kernel(const float4* __restrict__ part_o,
                                                   const float2* __restrict__ part_ml,
                                                   const ChunkCut* __restrict__ cut,
                                                   uint16_t* __restrict__ out,
                                                   float* __restrict__ lse) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;");
  const int c = blockIdx.x, tid = threadIdx.x;
  const ChunkCut k = cut[c];
  if (k.nparts <= 0) return;
  // heads side by side (512 bytes of a piece a warp)
  const int head = tid & 63, c4 = blockIdx.y * 16 + (tid >> 6) * 4;
  auto slot = [&](int p) { return (size_t)(p == 0 ? 2 * c + 1 : 2 * (c + 2 * p)); };
  float M = -INFINITY, l = 0.f;
#pragma unroll 8
  for (int p = 0; p < k.nparts; ++p) M = fmaxf(M, part_ml[slot(p) * kHalf + head].x);
  float4 acc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int p = 0; p < k.nparts; ++p) {
    const float2 ml = part_ml[slot(p) * kHalf + head];
    const float4* src = part_o + (slot(p) * (kDv / 4) + c4) * kHalf + head;
    const float f = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
    l += f * ml.y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 v = src[e * kHalf];
      acc[e].x += f * v.x;
      acc[e].y += f * v.y;
      acc[e].z += f * v.z;
      acc[e].w += f * v.w;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t row = (int64_t)k.row0 * kHeads + k.h * kHalf + head;
  uint4* dst = reinterpret_cast<uint4*>(out + row * kDv + c4 * 4);
#pragma unroll
  for (int e = 0; e < 4; e += 2)
    dst[e >> 1] = make_uint4(pack_bf16(acc[e].x * inv, acc[e].y * inv),
                             pack_bf16(acc[e].z * inv, acc[e].w * inv),
                             pack_bf16(acc[e + 1].x * inv, acc[e + 1].y * inv),
                             pack_bf16(acc[e + 1].z * inv, acc[e + 1].w * inv));
  if (c4 == 0)
    lse[row] = l > 0.f ? (M + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace chunk_mla

size_t chunk_mla_workspace_bytes(int n_sm) {
  using namespace chunk_mla;
  const size_t slots = 2 * (size_t)n_sm;
  return chunk_up256(n_sm * sizeof(ChunkCut)) + chunk_up256(slots * kHalf * sizeof(float2)) +
         slots * kDv * kHalf * sizeof(float);
}

cudaError_t launch_chunk_mla(const sa_geom& g, const ChunkCall& c, cudaStream_t stream) {
  using namespace chunk_mla;
  Args a;
  a.shape.cu_new = c.cu_new;
  a.shape.seq_lens = c.seq_lens;
  a.shape.n_tokens = c.n_tokens;
  a.shape.B = g.B;
  a.shape.H = 1;
  a.shape.inner = 2;
  a.shape.BT = 1;
  a.shape.ST = 0;
  a.shape.extra = 2;
  const int longest = 1 << 30;  // no sequence is longer
  a.shape.sink = c.sink < longest ? c.sink : longest;
  a.shape.window = c.window < longest ? c.window : longest;
  a.shape.cap = (int64_t)g.max_pages * g.P;
  a.shape.status = c.status;
  a.page_table = c.page_table;
  a.kv = static_cast<const uint8_t*>(c.k_cache);
  a.out = static_cast<uint16_t*>(c.out);
  a.lse = c.lse;
  uint8_t* w = c.scratch;
  a.cut = reinterpret_cast<ChunkCut*>(w);
  w += chunk_up256(c.n_sm * sizeof(ChunkCut));
  a.part_ml = reinterpret_cast<float2*>(w);
  w += chunk_up256(2 * (size_t)c.n_sm * kHalf * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(w);
  a.P = g.P;
  a.page_shift = g.P == 16 ? 4 : g.P == 32 ? 5 : 6;
  a.max_pages = g.max_pages;
  a.n_pool = g.n_pool;
  a.scale_log2 = c.scale * 1.4426950408889634f;
  CUtensorMap qm, km;
  if (!encode_heads_tmap(&qm, c.q, kD, kHeads, c.n_tokens, 64, kHalf, 1) ||
      !encode_rows_tmap(&km, c.k_cache, kD, (uint64_t)g.n_pool * g.P, 64, g.P))
    return cudaErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(attend_kernel);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  void* args[] = {&qm, &km, &a};
  if ((e = chunk_launch(fn, dim3(c.n_sm & ~1), kThreads, kSmem, stream, args)) != cudaSuccess)
    return e;
  void* jargs[] = {&a.part_o, &a.part_ml, &a.cut, &a.out, &a.lse};
  return chunk_launch(reinterpret_cast<const void*>(join_kernel), dim3(c.n_sm & ~1, kDv / 64), 256, 0,
                      stream, jargs);
}

}  // namespace sa
