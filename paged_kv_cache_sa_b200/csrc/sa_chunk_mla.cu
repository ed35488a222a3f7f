// sa_chunk_mla.cu -- exact attention of a ragged chunk of new tokens over the paged cache,
// latent geometry (128 query heads share one 576-wide key per token, V its first 512
// channels), on the 5th-generation tensor cores.
//
// Method: as sa_chunk.cu, with both products transposed.  An accumulator of 128 heads by 512
// channels would fill tensor memory and leave no place for scores; so a CTA takes 64 heads
// of one token (a neighbouring CTA the other 64, reading the same keys at the same time):
//   S^T = K Q^T   (128 keys x 64 heads, K = 576 channels, keys K-major)
//   O^T += V^T P^T (four blocks of 128 channels x 64 heads, K = 128 keys, keys MN-major)
// which is 64 + 256 columns.  Both products read the keys from the same place in shared
// memory: a tile's nine slices of 64 channels are loaded once (144 KB; with the queries'
// 72 KB all that fits), P^T overwrites the ninth slice (the rotated channels, not part of
// V) once the scores are done, and the loads of the next tile follow the products of this
// one slice pair by slice pair.  The next tiles' pages are asked into L2 ahead of that.
// Softmax: a thread has one key and 32 of the heads, so a maximum over keys crosses threads.
// It is only taken when some score exceeds the maximum in use by more than 2^8 (which a vote
// finds); sums stay in the threads until the end.
// Warps 0-3 and 4-7: softmax of heads 0-31 and 32-63; 8: issues the products; 9: work list
// and TMA.
#include "sa_chunk.cuh"
#include "sa_internal.h"
#include "sa_tc.cuh"

namespace sa {

namespace chunk_mla {

constexpr int kD = 576, kDv = 512, kHeads = 128;
constexpr int kHalf = 64;  // heads of a CTA
constexpr int kThreads = 320;
constexpr int kSegs = 2;
constexpr int kGroups = 5;  // slice pairs 0-1, 2-3, 4-5, 6-7 and slice 8
constexpr uint32_t kSlice = kKeyTile * 128;
constexpr uint32_t kQSlice = kHalf * 128;
constexpr uint32_t kKeys = 9 * kQSlice;  // queries first
constexpr uint32_t kMisc = kKeys + 9 * kSlice;
constexpr uint32_t kP = kKeys + 8 * kSlice;
constexpr uint32_t kO = 64;  // column of O^T; S^T is columns 0-63

struct Misc {
  float off[2][32];  // minus the maximum in use of every head (0 while there is none)
  float fac[2][32];  // rescaling factors, then 1 / l
  float red[2][4][32];
  ChunkSeg seg[kSegs];
  uint64_t full[kGroups], empty[kGroups];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full, q_empty, s_full, p_full, o_full, drain, meet[2];
  uint32_t tmem;
  int quit;
  int vote[2][3];
};
constexpr uint32_t kSmem = kMisc + sizeof(Misc);
static_assert(kSmem <= 232448, "shared memory of a CTA");

struct Args {
  ChunkShape shape;
  const int32_t* page_table;
  const uint8_t* kv;
  uint16_t* out;
  float* lse;
  float* part_o;    // [2 n_cta][512 channels][64 heads]
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

__device__ __forceinline__ void produce(const Args& a, uint32_t smem, Misc& mi,
                                        const CUtensorMap* qmap, const CUtensorMap* kmap) {
  const int lane = threadIdx.x & 31;
  int32_t* status = a.shape.status;
  ChunkSched sched;
  if (lane == 0) a.cut[blockIdx.x].nparts = 0;
  sched.init(a.shape, blockIdx.x, gridDim.x);
  const int ppt = kKeyTile >> a.page_shift;
  const int my_page = lane % ppt, my_sub = lane / ppt;
  const uint64_t policy = tc::l2_normal();
  int it = 0;  // tiles loaded
  bool ok = true;
  for (int n = 0; ok; ++n) {
    const int slot = n % kSegs;
    if (n >= kSegs &&
        !tc::wait_warp(&mi.seg_empty[slot], (n / kSegs - 1) & 1, &mi.quit, status)) {
      ok = false;
      break;
    }
    ChunkSeg g;
    const bool more = sched.next(g);
    if (!more) g.valid = 0;
    g.it0 = it;
    if (lane == 0) {
      mi.seg[slot] = g;
      mbar_arrive(&mi.seg_full[slot]);
      if (more && g.nparts > 0) a.cut[blockIdx.x] = ChunkCut{g.nparts, g.row0, g.ntok, g.h};
    }
    if (!more) break;
    if (n > 0 && !tc::wait_warp(&mi.q_empty, (n - 1) & 1, &mi.quit, status)) {
      ok = false;
      break;
    }
    if (lane == 0) mbar_arrive_expect_tx(&mi.q_full, 9 * kQSlice);
    __syncwarp();
    if (lane < 9)
      tc::tma_3d(smem + lane * kQSlice, qmap, lane * 64, g.h * kHalf, g.row0, &mi.q_full);
    const int nt = g.i1 - g.i0;
    const int last_page = (g.L - 1) >> a.page_shift;
    const Pages pages(a, g);
    const int32_t* row = a.page_table + (size_t)g.b * a.max_pages;
    auto lookup = [&](int i) -> int {
      if (i >= nt) return -1;
      const int lp = tile_of(g, g.i0 + i) * ppt + my_page;
      if (my_sub > 1 || lp > last_page || !pages.wanted(lp)) return -1;
      const int ph = row[lp];
      if (ph < 0 || ph >= a.n_pool) {
        if ((lp << a.page_shift) <= g.s0) report(status, SA_ERR_DEVICE_CHECK);
        return -1;
      }
      return ph;
    };
    auto ask = [&](int ph) {  // a page into L2
      if (ph >= 0 && my_sub == 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                         a.kv + (size_t)ph * a.P * (kD * 2)),
                     "r"(a.P * (kD * 2))
                     : "memory");
    };
    int p0 = lookup(0), p1 = lookup(1), p2 = lookup(2);
    ask(p1);
    for (int i = 0; i < nt && ok; ++i, ++it) {
      const int p3 = lookup(i + 3);
      ask(p2);
      const unsigned m = __ballot_sync(0xffffffffu, p0 >= 0 && my_sub == 0);
      for (int gr = 0; gr < kGroups; ++gr) {
        if (it > 0 && !tc::wait_warp(&mi.empty[gr], (it - 1) & 1, &mi.quit, status)) {
          ok = false;
          break;
        }
        const int subs = gr == 4 ? 1 : 2;
        if (lane == 0) mbar_arrive_expect_tx(&mi.full[gr], subs * __popc(m) * a.P * 128);
        __syncwarp();
        if (p0 >= 0 && my_sub < subs)
          tc::tma_2d(smem + kKeys + (2 * gr + my_sub) * kSlice +
                         ((uint32_t)my_page << a.page_shift) * 128,
                     kmap, (2 * gr + my_sub) * 64, p0 << a.page_shift, &mi.full[gr], policy);
      }
      p0 = p1;
      p1 = p2;
      p2 = p3;
    }
  }
  if (!ok) {  // given up: let copies in flight land (bounded) before shared memory goes away
    for (int gr = 0; gr < kGroups; ++gr)
      for (int x = max(0, it - 1); x <= it; ++x) mbar_wait(&mi.full[gr], x & 1);
  }
}

__device__ __forceinline__ void multiply(const Args& a, uint32_t smem, Misc& mi, uint32_t tmem) {
  constexpr uint32_t id_s = tc::idesc(kKeyTile, kHalf, false, false);
  constexpr uint32_t id_o = tc::idesc(128, kHalf, true, true);
  int32_t* status = a.shape.status;
  int it = 0;
  for (int n = 0;; ++n) {
    const int slot = n % kSegs;
    if (!tc::wait_warp(&mi.seg_full[slot], (n / kSegs) & 1, &mi.quit, status)) return;
    const int nt = __shfl_sync(0xffffffffu, mi.seg[slot].i1 - mi.seg[slot].i0, 0);
    const bool valid = __shfl_sync(0xffffffffu, mi.seg[slot].valid, 0) != 0;
    if (tc::elect()) mbar_arrive(&mi.seg_empty[slot]);
    if (!valid) return;
    if (!tc::wait_warp(&mi.q_full, n & 1, &mi.quit, status)) return;
    for (int i = 0; i < nt; ++i, ++it) {
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) {
        if (!tc::wait_warp(&mi.full[gr], it & 1, &mi.quit, status)) return;
        tc::fence_after();
        if (tc::elect()) {
#pragma unroll
          for (int kk = 0; kk < (gr == 4 ? 4 : 8); ++kk) {
            const int sl = 2 * gr + (kk >> 2);
            tc::mma_ss(tmem, tc::desc(smem + kKeys + sl * kSlice + (kk & 3) * 32),
                       tc::desc(smem + sl * kQSlice + (kk & 3) * 32), id_s, gr + kk != 0);
          }
          if (gr == 4) {
            tc::commit(&mi.s_full);
            if (i + 1 == nt) tc::commit(&mi.q_empty);
          }
        }
        __syncwarp();
      }
      if (!tc::wait_warp(&mi.p_full, it & 1, &mi.quit, status)) return;
      tc::fence_after();
      if (tc::elect()) {
#pragma unroll
        for (int cb = 0; cb < 4; ++cb) {
#pragma unroll
          for (int kk = 0; kk < kKeyTile / 16; ++kk)
            tc::mma_ss(tmem + kO + cb * 64,
                       tc::desc(smem + kKeys + 2 * cb * kSlice + kk * 2048, kSlice),
                       tc::desc(smem + kP + kk * 2048), id_o, !(i == 0 && kk == 0));
          tc::commit(&mi.empty[cb]);
        }
        tc::commit(&mi.empty[4]);
        if (i + 1 == nt) tc::commit(&mi.o_full);
      }
      __syncwarp();
    }
  }
}

// v[c] of every lane combined over the warp: lane c gets column c
template <bool MAX>
__device__ __forceinline__ float across(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, o);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  return v[0];
}

// softmax and epilogue of heads [32 t, 32 t + 32) of the CTA's 64
__device__ __forceinline__ void soften(const Args& a, uint32_t smem, Misc& mi, uint32_t tmem,
                                       int t) {
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3;
  const int r = wq * 32 + lane;  // key of the tile; channel of a block of O^T
  const uint32_t lanes = (uint32_t)(wq * 32) << 16;
  int32_t* status = a.shape.status;
  int it = 0, nmeet = 0;
  auto meet = [&]() -> bool {  // the four warps of these heads; shared writes become visible
    __syncwarp();
    if (lane == 0) mbar_arrive(&mi.meet[t]);
    return tc::wait_warp(&mi.meet[t], nmeet++ & 1, &mi.quit, status);
  };
  for (int n = 0;; ++n) {
    const int slot = n % kSegs;
    if (!tc::wait_warp(&mi.seg_full[slot], (n / kSegs) & 1, &mi.quit, status)) return;
    const ChunkSeg g = mi.seg[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&mi.seg_empty[slot]);
    if (!g.valid) return;
    const int nt = g.i1 - g.i0, s = g.s0;
    const Pages pages(a, g);
    float l[32], m = -INFINITY;  // sums of this thread's keys; maximum of head 32 t + lane
#pragma unroll
    for (int c = 0; c < 32; ++c) l[c] = 0.f;
    bool none = true;  // no key seen yet in this piece
    for (int i = 0; i < nt; ++i, ++it) {
      // all that the scores are not needed for comes before they are waited for
      const int key = tile_of(g, g.i0 + i) * kKeyTile + r;
      const bool stored = key < g.L && pages.wanted(key >> a.page_shift);
      const bool seen = key <= s && (a.shape.window == 0 || key > s - a.shape.window ||
                                     key < a.shape.sink);
      const bool ragged = !__all_sync(0xffffffffu, stored);
      if (!tc::wait_warp(&mi.s_full, it & 1, &mi.quit, status)) return;
      tc::fence_after();
      if (ragged) {
        // rows without a loaded token would meet a probability of zero; 0 * NaN is not 0
        if (!stored) {
          const uint32_t base = smem + kKeys + 4 * t * kSlice + r * 128;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             base + (e >> 3) * kSlice + (e & 7) * 16),
                         "r"(0)
                         : "memory");
        }
        __syncwarp();
      }
      // P with the maximum in use, in place of the scores, while the vote on it goes round
      float p[32];
      auto probabilities = [&](bool vote) {
        uint32_t x[32];
        tc::tmem_ld32(tmem + lanes + 32 * t, x);
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 off = *reinterpret_cast<const float4*>(&mi.off[t][c]);
          p[c] = fmaf(__uint_as_float(x[c]), a.scale_log2, off.x);
          p[c + 1] = fmaf(__uint_as_float(x[c + 1]), a.scale_log2, off.y);
          p[c + 2] = fmaf(__uint_as_float(x[c + 2]), a.scale_log2, off.z);
          p[c + 3] = fmaf(__uint_as_float(x[c + 3]), a.scale_log2, off.w);
        }
        if (vote) {
#pragma unroll
          for (int c = 0; c < 32; c += 2) top = fmaxf(top, fmaxf(p[c], p[c + 1]));
          const bool over = __any_sync(0xffffffffu, seen && (none || top > 8.f));
          // round it: raise flag it % 3; flag (it + 1) % 3 was last read before the last vote
          if (lane == 0) {
            if (wq == 0) *(volatile int*)&mi.vote[t][(it + 1) % 3] = 0;
            if (over) *(volatile int*)&mi.vote[t][it % 3] = 1;
            mbar_arrive(&mi.meet[t]);
          }
        }
        const uint32_t prow = smem + kP + r * 128;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = 8 * u + 2 * e;
            p[c] = seen ? fast_exp2(p[c]) : 0.f;
            p[c + 1] = seen ? fast_exp2(p[c + 1]) : 0.f;
            w[e] = pack_bf16(p[c], p[c + 1]);
          }
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           prow + (((4 * t + u) ^ (r & 7)) << 4)),
                       "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
        }
      };
      probabilities(true);
      tc::fence_async_smem();
      if (!tc::wait_warp(&mi.meet[t], nmeet++ & 1, &mi.quit, status)) return;
      if (*(volatile int*)&mi.vote[t][it % 3]) {
        // raise the maximum: columns' maxima over the tile's keys, O^T and the sums rescaled
        {
          uint32_t x[32];
          tc::tmem_ld32(tmem + lanes + 32 * t, x);
          float v[32];
#pragma unroll
          for (int c = 0; c < 32; ++c)
            v[c] = seen ? __uint_as_float(x[c]) * a.scale_log2 : -INFINITY;
          mi.red[t][wq][lane] = across<true>(v);
        }
        if (!meet()) return;
        const float up = fmaxf(fmaxf(fmaxf(mi.red[t][0][lane], mi.red[t][1][lane]),
                                     fmaxf(mi.red[t][2][lane], mi.red[t][3][lane])),
                               m);
        if (wq == 0) {
          mi.fac[t][lane] = m == -INFINITY ? 0.f : fast_exp2(m - up);
          mi.off[t][lane] = up == -INFINITY ? 0.f : -up;
        }
        m = up;
        if (!meet()) return;
        if (!none) {
#pragma unroll
          for (int c = 0; c < 32; ++c) l[c] *= mi.fac[t][c];
#pragma unroll 1
          for (int cb = 0; cb < 4; ++cb) {
            uint32_t o[32];
            const uint32_t col = tmem + lanes + kO + cb * 64 + 32 * t;
            tc::tmem_ld32(col, o);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              o[c] = __float_as_uint(__uint_as_float(o[c]) * mi.fac[t][c]);
            tc::tmem_st32(col, o);
          }
          tc::tmem_wait_st();
        }
        none = false;
        probabilities(false);
        tc::fence_async_smem();
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&mi.p_full);
#pragma unroll
      for (int c = 0; c < 32; ++c) l[c] += p[c];
    }
    // ---- results
    const float part = across<false>(l);
    mi.red[t][wq][lane] = part;
    if (!meet()) return;
    const float sum = (mi.red[t][0][lane] + mi.red[t][1][lane]) +
                      (mi.red[t][2][lane] + mi.red[t][3][lane]);
    const int head = g.h * kHalf + 32 * t + lane;
    if (wq == 0) {
      mi.fac[t][lane] = g.part >= 0 ? 1.f : sum > 0.f ? 1.f / sum : 0.f;
      if (g.part >= 0)
        a.part_ml[(size_t)g.part * kHalf + 32 * t + lane] = make_float2(m, sum);
      else
        a.lse[(size_t)g.row0 * kHeads + head] =
            sum > 0.f ? (m + __log2f(sum)) * 0.69314718055994531f : -INFINITY;
    }
    if (!meet()) return;
    if (!tc::wait_warp(&mi.o_full, n & 1, &mi.quit, status)) return;
    tc::fence_after();
#pragma unroll 1
    for (int cb = 0; cb < 4; ++cb) {
      uint32_t o[32];
      tc::tmem_ld32(tmem + lanes + kO + cb * 64 + 32 * t, o);
      const int ch = cb * 128 + r;
      if (g.part >= 0) {
        float4* dst = reinterpret_cast<float4*>(
            a.part_o + ((size_t)g.part * kDv + ch) * kHalf + 32 * t);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          dst[c] = make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                               __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
      } else {
        uint16_t* dst =
            a.out + ((size_t)g.row0 * kHeads + g.h * kHalf + 32 * t) * kDv + ch;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          dst[(size_t)c * kDv] =
              (uint16_t)pack_bf16(__uint_as_float(o[c]) * mi.fac[t][c], 0.f);
      }
    }
    // the next piece's first raise of the maximum writes fac and off behind two meetings, and
    // its products into O^T wait for this thread's arrival on p_full
    tc::fence_before();
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = smem_u32(smem_raw);
  Misc& mi = *reinterpret_cast<Misc*>(smem_raw + kMisc);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&mi.full[i], 1);
      mbar_init(&mi.empty[i], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&mi.seg_full[i], 1);
      mbar_init(&mi.seg_empty[i], 9);  // the issuing thread and eight softmax warps
    }
    mbar_init(&mi.q_full, 1);
    mbar_init(&mi.q_empty, 1);
    mbar_init(&mi.s_full, 1);
    mbar_init(&mi.p_full, 8);
    mbar_init(&mi.o_full, 1);
    mbar_init(&mi.drain, 1);
    mbar_init(&mi.meet[0], 4);
    mbar_init(&mi.meet[1], 4);
    mi.quit = 0;
    for (int i = 0; i < 6; ++i) (&mi.vote[0][0])[i] = 0;
    for (int i = 0; i < 64; ++i) (&mi.off[0][0])[i] = 0.f;
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
    soften(a, smem, mi, tmem, warp >> 2);
  } else if (warp == 8) {
    multiply(a, smem, mi, tmem);
    __syncwarp();
    if (tc::elect()) {
      tc::commit(&mi.drain);
      mbar_wait(&mi.drain, 0);
    }
    __syncwarp();
  } else {
    produce(a, smem, mi, &qmap, &kmap);
    __syncwarp();
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 8) tc::tmem_free_all(tmem);
  asm volatile("griddepcontrol.launch_dependents;");
}

// Joins the pieces of the cut items, in piece order.  CTA = (cut item, 32 channels): a thread
// sums 4 heads of 2 channels, the result is turned in shared memory and written by heads.
// Also returns the item counter to zero for the next call.
__global__ void __launch_bounds__(256) join_kernel(const float* __restrict__ part_o,
                                                   const float2* __restrict__ part_ml,
                                                   const ChunkCut* __restrict__ cut,
                                                   int32_t* ticket, uint16_t* __restrict__ out,
                                                   float* __restrict__ lse) {
  __shared__ float tile[kHalf][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int c = blockIdx.x, ch0 = blockIdx.y * 32, tid = threadIdx.x;
  if (c == 0 && blockIdx.y == 0 && tid == 0) *ticket = 0;
  const ChunkCut k = cut[c];
  if (k.nparts <= 0) return;
  const int hq = (tid & 15) * 4, row = tid >> 4;  // heads hq.., channels row and row + 16
  auto slot = [&](int p) { return (size_t)(p == 0 ? 2 * c + 1 : 2 * (c + 2 * p)); };
  float M[4], l[4], acc[2][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    M[e] = -INFINITY;
    l[e] = acc[0][e] = acc[1][e] = 0.f;
  }
#pragma unroll 4
  for (int p = 0; p < k.nparts; ++p) {
    const float2* ml = part_ml + slot(p) * kHalf + hq;
#pragma unroll
    for (int e = 0; e < 4; ++e) M[e] = fmaxf(M[e], ml[e].x);
  }
#pragma unroll 4
  for (int p = 0; p < k.nparts; ++p) {
    const float2* ml = part_ml + slot(p) * kHalf + hq;
    const float* src = part_o + (slot(p) * kDv + ch0 + row) * kHalf + hq;
    const float4 v0 = *reinterpret_cast<const float4*>(src);
    const float4 v1 = *reinterpret_cast<const float4*>(src + 16 * kHalf);
    const float a0[4] = {v0.x, v0.y, v0.z, v0.w}, a1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float f = ml[e].x == -INFINITY ? 0.f : fast_exp2(ml[e].x - M[e]);
      l[e] += f * ml[e].y;
      acc[0][e] += f * a0[e];
      acc[1][e] += f * a1[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float inv = l[e] > 0.f ? 1.f / l[e] : 0.f;
    tile[hq + e][row] = acc[0][e] * inv;
    tile[hq + e][row + 16] = acc[1][e] * inv;
    if (blockIdx.y == 0 && row == 0)
      lse[(size_t)k.row0 * kHeads + k.h * kHalf + hq + e] =
          l[e] > 0.f ? (M[e] + __log2f(l[e])) * 0.69314718055994531f : -INFINITY;
  }
  __syncthreads();
  const int head = tid >> 2, c8 = (tid & 3) * 8;
  const float* src = &tile[head][c8];
  *reinterpret_cast<uint4*>(out + ((size_t)k.row0 * kHeads + k.h * kHalf + head) * kDv + ch0 +
                            c8) = make_uint4(pack_bf16(src[0], src[1]), pack_bf16(src[2], src[3]),
                                             pack_bf16(src[4], src[5]),
                                             pack_bf16(src[6], src[7]));
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
  a.shape.ticket = c.ticket;
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
  if ((e = chunk_launch(fn, dim3(c.n_sm), kThreads, kSmem, stream, args)) != cudaSuccess)
    return e;
  void* jargs[] = {&a.part_o, &a.part_ml, &a.cut, &a.shape.ticket, &a.out, &a.lse};
  return chunk_launch(reinterpret_cast<const void*>(join_kernel), dim3(c.n_sm, kDv / 32), 256, 0,
                      stream, jargs);
}

}  // namespace sa
