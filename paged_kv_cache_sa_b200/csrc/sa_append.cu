// sa_append.cu -- new tokens' keys and values into the paged cache, with the position
// rotation and the refresh of the touched pages' summaries.
//
// Method.  New token i of sequence b goes to slot s = L_b - n_b + i; its position is
// p = (logical length or L_b) - n_b + i.  Rotation pairs (x, y) of a key or query row turn by
// a = p * inv_freq[j]: (x cos a - y sin a, y cos a + x sin a).  p reaches millions, where an
// fp32 product is off by up to 2^-24 * a (0.06 rad at a = 10^6): the angle is formed in fp64
// as a number of turns, its whole turns are dropped there, and only the fraction (rounded
// once, 2^-25 turns) goes to sincospif.  The rotation is fp32; the only rounding to bf16 is
// the store.
//
// Three kinds of CTA, two of them in a launch:
//   pages: one CTA per (sequence, page that receives tokens).  The page is the unit that has a
//     single owner, so the summaries (min/max over all valid rows of the page, the old ones
//     read back from the cache, the new ones still in registers) need no atomics and no second
//     launch.  A warp takes a KV head (latent rows: the CTA's row groups share the page).
//   tokens (grouped-query geometry): a run of rows of the call, as many as make about 1024
//     units; rotates their queries and copies their values.  Queries are most of the bytes, so
//     they are spread over the grid whatever the pages are, and their loads are in flight
//     before the sequence and page of the rows are known.
//   queries (latent geometry): 147 KB a token, of which rotation concerns a ninth.  They pass
//     through shared memory in bulk copies of 18 KB, three per CTA on their way in or out, and
//     threads touch the rotated channels only.  (Through registers, as in the other geometry:
//     59 us instead of 50 for 961 tokens, 11.6 instead of 6.5 us for 16.  The other geometry's
//     queries through shared memory: 78 us instead of 73 for 16390 tokens, where every channel
//     turns, and 15 instead of 12 us for 739 of which half of the channels turn.)
// cos/sin are computed once per CTA (queries: once per token) into shared memory and serve every
// head.  A "unit" is two 16-byte chunks of one row that rotate together (j and j + rot/2 in the
// half-split form, neighbours in the interleaved form); a thread keeps its unit's place and
// walks the rows, so that loads and stores stay 16 bytes wide and coalesced and little is spent
// on addresses (a count through all units of a run instead: 76 us for the 16390 tokens).
// Bound by HBM: every row is read once and written once.
// Measured on a B200: 16390 tokens of 32 / 8 heads of 128 channels 69.3 us in a graph on one input,
// 72.6 on changing ones (5.9 and 5.6 TB/s; the copy reaches 6.5), 961 tokens of the latent geometry
// 50 us (5.7 TB/s), eight decode tokens 4.5 us (latency: lengths, page table, keys and sine table
// one behind the other).  Runs of 2048 units are 6% slower and of 512 13%, 128 threads a CTA 5%
// faster here but 25% slower for a decode step.  Latent pieces of 30 KB, four stages or fewer and larger CTAs: 1 to 7% slower.
#include <algorithm>

#include "sa_common.cuh"
#include "sa_fp8.cuh"
#include "sa_internal.h"
#include "sa_tc.cuh"

namespace sa {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kMaxRun = 64;      // tokens of a token CTA, at most
constexpr int kRunUnits = 1024;  // query units that a token CTA is sized for
constexpr int kMaxKnown = 16;    // tokens that a query CTA looks up at a time
constexpr int kHeads = 16;       // latent heads of a piece
constexpr uint32_t kPieceBytes = kHeads * 576 * 2;
constexpr int kStages = 3;       // pieces in a query CTA's shared memory
constexpr int kQueryCtas = 3;    // query CTAs of an SM
constexpr int kLatentGroups = kAppendThreads / 36;  // thread groups that share a latent page's rows
static_assert(kMaxKnown <= kMaxRun, "Tokens");

struct AppendArgs {
  const uint4* q;
  const uint4* k;
  const uint4* v;
  int64_t q_stride, k_stride, v_stride;  // 16-byte chunks from one token to the next
  const int32_t* cu_new;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* logical_lens;
  const float* inv_freq;
  uint4* q_out;
  uint4* k_cache;
  uint4* v_cache;
  void* summ;
  int32_t* status;
  int n_tokens, B, Hq, Hkv, P, max_pages, n_pool;
  int rot_start, rot_dim, interleaved;
  int want;  // 0: no summaries, 1: bf16 rows, 2: fp8 records
  int n_query_ctas, n_page_ctas;  // latent queries' CTAs come first, then the pages'
  int run;                        // tokens of a token CTA
  uint32_t inv_half, inv_hq, inv_hkv;  // see quot(), of rot_dim / 2 and counts of heads
};

// e / d where inv = ceil(2^32 / d) and e * d < 2^32
__device__ __forceinline__ uint32_t quot(uint32_t e, uint32_t d, uint32_t inv) {
  return d == 1 ? e : __umulhi(e, inv);
}

// shared memory -> global, as part of this thread's current group of copies
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// the two chunks of unit u of a row, and the place of its first rotation pair (-1: not rotated)
struct Unit {
  int ca, cb, pair;
};

template <int CPR>
__device__ __forceinline__ Unit unit_of(int u, int rot_start, int rot_dim, bool interleaved) {
  const int n_rot = rot_dim >> 4, c0 = rot_start >> 3;
  Unit x;
  if (u < n_rot) {
    x.ca = interleaved ? c0 + 2 * u : c0 + u;
    x.cb = interleaved ? x.ca + 1 : x.ca + n_rot;
    x.pair = 2 * u;
  } else {  // the rest in two halves, so that neighbouring lanes copy neighbouring chunks
    x.ca = u - n_rot;
    x.cb = x.ca + CPR / 2 - n_rot;
    if (x.ca >= c0) x.ca += 2 * n_rot;
    if (x.cb >= c0) x.cb += 2 * n_rot;
    x.pair = -1;
  }
  return x;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// (x, y) of both halves of two words turned by cs[0], cs[1]
__device__ __forceinline__ void turn2(uint32_t& a, uint32_t& b, float2 t0, float2 t1) {
  const float x0 = bf_lo(a), x1 = bf_hi(a), y0 = bf_lo(b), y1 = bf_hi(b);
  a = pack_bf16(x0 * t0.x - y0 * t0.y, x1 * t1.x - y1 * t1.y);
  b = pack_bf16(y0 * t0.x + x0 * t0.y, y1 * t1.x + x1 * t1.y);
}
__device__ __forceinline__ uint32_t turn_pair(uint32_t w, float2 t) {
  const float x = bf_lo(w), y = bf_hi(w);
  return pack_bf16(x * t.x - y * t.y, y * t.x + x * t.y);
}

// Place of pair j's (cos, sin) among a token's `half`: [two pairs of a unit][unit], so that the
// lanes of a row, one unit each, read 16 bytes side by side (in pair order they would meet in
// two groups of banks, and shared memory bounded the kernel: 88 us instead of 75 for 16K tokens,
// 32 / 8 heads).
__device__ __forceinline__ int pair_at(int j, int half) {
  return ((j & 7) >> 1) * (half >> 2) + (j >> 3) * 2 + (j & 1);
}

// a unit turned; cs: its first (cos, sin) pair, `half` of them per token
__device__ __forceinline__ void rotate_unit(uint4& a, uint4& b, const float2* cs, int half,
                                            bool interleaved) {
  float2 c[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 t = *reinterpret_cast<const float4*>(cs + k * (half >> 2));
    c[2 * k] = make_float2(t.x, t.y);
    c[2 * k + 1] = make_float2(t.z, t.w);
  }
  if (!interleaved) {
    turn2(a.x, b.x, c[0], c[1]);
    turn2(a.y, b.y, c[2], c[3]);
    turn2(a.z, b.z, c[4], c[5]);
    turn2(a.w, b.w, c[6], c[7]);
  } else {
    a.x = turn_pair(a.x, c[0]);
    a.y = turn_pair(a.y, c[1]);
    a.z = turn_pair(a.z, c[2]);
    a.w = turn_pair(a.w, c[3]);
    b.x = turn_pair(b.x, c[4]);
    b.y = turn_pair(b.y, c[5]);
    b.z = turn_pair(b.z, c[6]);
    b.w = turn_pair(b.w, c[7]);
  }
}

// running min and max of a chunk, on the bf16 order keys
struct Range {
  uint4 mn, mx;
  __device__ __forceinline__ void clear() {
    mn = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
    mx = make_uint4(0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u);
  }
  __device__ __forceinline__ void merge(const uint4& lo, const uint4& hi) {
    mn.x = __vmins2(mn.x, lo.x); mn.y = __vmins2(mn.y, lo.y);
    mn.z = __vmins2(mn.z, lo.z); mn.w = __vmins2(mn.w, lo.w);
    mx.x = __vmaxs2(mx.x, hi.x); mx.y = __vmaxs2(mx.y, hi.y);
    mx.z = __vmaxs2(mx.z, hi.z); mx.w = __vmaxs2(mx.w, hi.w);
  }
  __device__ __forceinline__ void add(const uint4& v) {
    const uint4 k = make_uint4(bf2_key(v.x), bf2_key(v.y), bf2_key(v.z), bf2_key(v.w));
    merge(k, k);
  }
  __device__ __forceinline__ void merge_lane(int off) {
    uint4 lo, hi;
    lo.x = __shfl_xor_sync(0xffffffffu, mn.x, off); lo.y = __shfl_xor_sync(0xffffffffu, mn.y, off);
    lo.z = __shfl_xor_sync(0xffffffffu, mn.z, off); lo.w = __shfl_xor_sync(0xffffffffu, mn.w, off);
    hi.x = __shfl_xor_sync(0xffffffffu, mx.x, off); hi.y = __shfl_xor_sync(0xffffffffu, mx.y, off);
    hi.z = __shfl_xor_sync(0xffffffffu, mx.z, off); hi.w = __shfl_xor_sync(0xffffffffu, mx.w, off);
    merge(lo, hi);
  }
  __device__ __forceinline__ uint4 low() const {
    return make_uint4(bf2_key(mn.x), bf2_key(mn.y), bf2_key(mn.z), bf2_key(mn.w));
  }
  __device__ __forceinline__ uint4 high() const {
    return make_uint4(bf2_key(mx.x), bf2_key(mx.y), bf2_key(mx.z), bf2_key(mx.w));
  }
};

// New tokens of sequence b: first row and count, or n = 0 (reported) when they do not fit.
__device__ __forceinline__ void new_tokens(const int32_t* cu, const int32_t* lens, int b,
                                           int n_tokens, int64_t cap, int32_t* status, int& c0,
                                           int& n, int& L) {
  c0 = cu[b];
  const int c1 = cu[b + 1];
  L = lens[b];
  const bool ok = c0 >= 0 && c1 >= c0 && c1 <= n_tokens && L >= c1 - c0 && L <= cap;
  n = ok ? c1 - c0 : 0;
  if (!ok) report(status, SA_ERR_DEVICE_CHECK);
}

// cos and sin of half a turn's multiples: angle pos * f as a number of turns in fp64
__device__ __forceinline__ float2 cos_sin(int pos, float f) {
  const double turns = (double)pos * (double)f * 0.15915494309189535;
  const float frac = (float)(2.0 * (turns - rint(turns)));  // half turns in [-1, 1]
  float sn, co;
  sincospif(frac, &sn, &co);
  return make_float2(co, sn);
}

// CPR = 16-byte chunks per key row (Dk / 8).
template <int CPR>
__device__ __forceinline__ void append_pages(const AppendArgs& a, uint8_t* smem, int cta) {
  constexpr int U = CPR / 2;  // units per row
  __shared__ int scan[kAppendWarps];
  __shared__ int found[2];  // sequence and page of this CTA's item
  float2* cs = reinterpret_cast<float2*>(smem);  // [tokens][rot_dim / 2]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = a.rot_dim >> 1;
  const bool inter = a.interleaved != 0;
  const int64_t cap = (int64_t)a.max_pages * a.P;

  for (int item = cta;; item += a.n_page_ctas) {
    // ---- the item's sequence and page: running count of touched pages over the batch
    if (tid == 0) found[0] = -1;
    int before = 0;
    for (int b0 = 0; b0 < a.B; b0 += kAppendThreads) {
      const int b = b0 + tid;
      int pages = 0, first = 0;
      if (b < a.B) {
        int c0, n, L;
        new_tokens(a.cu_new, a.seq_lens, b, a.n_tokens, cap, a.status, c0, n, L);
        if (n > 0) {
          first = (L - n) / a.P;
          pages = (L - 1) / a.P - first + 1;
        }
      }
      int incl = pages;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
      }
      __syncthreads();  // scan[] of the previous round was read, found[] is cleared
      if (lane == 31) scan[warp] = incl;
      __syncthreads();
      int base = before, all = before;
#pragma unroll
      for (int w = 0; w < kAppendWarps; ++w) {
        if (w < warp) base += scan[w];
        all += scan[w];
      }
      const int lo = base + incl - pages;
      if (item >= lo && item < lo + pages) {
        found[0] = b;
        found[1] = first + (item - lo);
      }
      before = all;
      if (item < before) break;
    }
    __syncthreads();
    const int b = found[0], lp = found[1];
    if (b < 0) return;
    const int c0 = a.cu_new[b], n = a.cu_new[b + 1] - c0, L = a.seq_lens[b];
    const int page0 = lp * a.P, s0 = L - n;
    const int t0 = max(s0, page0), t1 = min(L, page0 + a.P);
    const int cnt = t1 - t0;           // new tokens of the page
    const int row0 = c0 + (t0 - s0);   // their first input row
    const int slot0 = t0 - page0;      // and slot; rows [0, slot0) are old
    const int phys = a.page_table[(size_t)b * a.max_pages + lp];
    if (phys < 0 || phys >= a.n_pool) {
      if (tid == 0) report(a.status, SA_ERR_DEVICE_CHECK);
      __syncthreads();
      continue;
    }
    const int pos0 = (a.logical_lens ? a.logical_lens[b] : L) - n + (t0 - s0);
    const int rows = slot0 + cnt;
    const int from = a.want ? 0 : slot0;
    // keys of a lane's rows r, r + RPW, ...: old ones from the cache, new ones from the call; the
    // first two are on their way while the angles are computed (four: the registers overflow)
    constexpr bool grouped = 32 % U == 0;
    constexpr int RPW = grouped ? 32 / U : 1, N = 2;
    const int u = grouped ? lane % U : tid % U, rg = grouped ? lane / U : tid / U;
    const Unit x = unit_of<CPR>(u, a.rot_start, a.rot_dim, inter);
    uint4 va[N], vb[N];
    auto fetch = [&](int h, int r0) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int r = r0 + k * RPW;
        if (r < rows) {
          const uint4* src = r < slot0
                                 ? a.k_cache + (((size_t)phys * a.Hkv + h) * a.P + r) * CPR
                                 : a.k + (size_t)(row0 + r - slot0) * a.k_stride + h * CPR;
          va[k] = src[x.ca];
          vb[k] = src[x.cb];
        }
      }
    };
    if (grouped && warp < a.Hkv) fetch(warp, from + rg);
    // ---- cos and sin of every (new token, pair)
    for (int e = tid; e < cnt * half; e += kAppendThreads) {
      const int i = quot(e, half, a.inv_half), j = e - i * half;
      cs[i * half + pair_at(j, half)] = cos_sin(pos0 + i, a.inv_freq[j]);
    }
    __syncthreads();

    // ---- keys: rotate and store the new rows, min/max over the page's valid rows
    if constexpr (grouped) {
      for (int h = warp; h < a.Hkv; h += kAppendWarps) {
        uint4* blk = a.k_cache + ((size_t)phys * a.Hkv + h) * a.P * CPR;
        Range ra, rb;
        ra.clear();
        rb.clear();
        for (int r0 = from + rg; r0 < rows; r0 += N * RPW) {
          if (h != warp || r0 != from + rg) fetch(h, r0);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int r = r0 + k * RPW;
            if (r >= rows) break;
            if (r >= slot0) {
              if (x.pair >= 0)
                rotate_unit(va[k], vb[k], cs + (r - slot0) * half + x.pair, half, inter);
              blk[r * CPR + x.ca] = va[k];
              blk[r * CPR + x.cb] = vb[k];
            }
            ra.add(va[k]);
            rb.add(vb[k]);
          }
        }
        if (a.want) {
#pragma unroll
          for (int off = U; off < 32; off <<= 1) {
            ra.merge_lane(off);
            rb.merge_lane(off);
          }
          const size_t rec = (size_t)phys * a.Hkv + h;
          const uint4 la = ra.low(), ha = ra.high(), lb = rb.low(), hb = rb.high();
          if (a.want == 2) {
            constexpr int D = CPR * 8;
            uint32_t am = max_mag2(max_mag2(max_mag2(max_mag2(0u, la.x), la.y), la.z), la.w);
            am = max_mag2(max_mag2(max_mag2(max_mag2(am, ha.x), ha.y), ha.z), ha.w);
            am = max_mag2(max_mag2(max_mag2(max_mag2(am, lb.x), lb.y), lb.z), lb.w);
            am = max_mag2(max_mag2(max_mag2(max_mag2(am, hb.x), hb.y), hb.z), hb.w);
            am = __reduce_max_sync(0xffffffffu, am);
            const int e = fp8_record_exp(am);
            uint8_t* out = static_cast<uint8_t*>(a.summ) + rec * (2 * D + 16);
            if (lane < U) {
              *reinterpret_cast<uint2*>(out + x.ca * 8) =
                  make_uint2(e4m3_pack(la.x, la.y, e, false), e4m3_pack(la.z, la.w, e, false));
              *reinterpret_cast<uint2*>(out + x.cb * 8) =
                  make_uint2(e4m3_pack(lb.x, lb.y, e, false), e4m3_pack(lb.z, lb.w, e, false));
              *reinterpret_cast<uint2*>(out + D + x.ca * 8) =
                  make_uint2(e4m3_pack(ha.x, ha.y, e, true), e4m3_pack(ha.z, ha.w, e, true));
              *reinterpret_cast<uint2*>(out + D + x.cb * 8) =
                  make_uint2(e4m3_pack(hb.x, hb.y, e, true), e4m3_pack(hb.z, hb.w, e, true));
            }
            if (lane == 0)
              *reinterpret_cast<uint4*>(out + 2 * D) = make_uint4((uint32_t)e & 0xFFu, 0u, 0u, 0u);
          } else if (lane < U) {
            uint4* out = static_cast<uint4*>(a.summ) + rec * 2 * CPR;
            out[x.ca] = la;
            out[x.cb] = lb;
            out[CPR + x.ca] = ha;
            out[CPR + x.cb] = hb;
          }
        }
      }
    } else {
      // latent rows (one KV head): the CTA's row groups split the page's rows, their
      // partial ranges meet in shared memory
      constexpr int NG = kLatentGroups;
      Range(*part)[CPR] = reinterpret_cast<Range(*)[CPR]>(smem + a.P * half * sizeof(float2));
      uint4* blk = a.k_cache + (size_t)phys * a.P * CPR;
      Range ra, rb;
      ra.clear();
      rb.clear();
      if (rg < NG) {
#pragma unroll 4
        for (int r = from + rg; r < rows; r += NG) {
          uint4 va, vb;
          if (r < slot0) {
            va = blk[r * CPR + x.ca];
            vb = blk[r * CPR + x.cb];
          } else {
            const int i = r - slot0;
            const uint4* src = a.k + (size_t)(row0 + i) * a.k_stride;
            va = src[x.ca];
            vb = src[x.cb];
            if (x.pair >= 0) rotate_unit(va, vb, cs + i * half + x.pair, half, inter);
            blk[r * CPR + x.ca] = va;
            blk[r * CPR + x.cb] = vb;
          }
          ra.add(va);
          rb.add(vb);
        }
        if (a.want) {
          part[rg][x.ca] = ra;
          part[rg][x.cb] = rb;
        }
      }
      if (a.want) {
        __syncthreads();
        if (tid < CPR) {
          Range r = part[0][tid];
          for (int g = 1; g < NG; ++g) r.merge(part[g][tid].mn, part[g][tid].mx);
          uint4* out = static_cast<uint4*>(a.summ) + (size_t)phys * 2 * CPR;
          out[tid] = r.low();
          out[CPR + tid] = r.high();
        }
      }
    }

    __syncthreads();  // cs[], found[] and part[] are free for the next item
  }
}

// Where tokens of the call belong.
struct Tokens {
  int seq[kMaxRun], slot[kMaxRun], pos[kMaxRun];  // slot: in its page
  int page[kMaxRun];                              // -1: belongs to no sequence or no page

  // tokens [r0, r0 + cnt), by the whole CTA; a barrier follows before they are read
  __device__ __forceinline__ void find(const AppendArgs& a, int r0, int cnt) {
    const int tid = threadIdx.x;
    const int64_t cap = (int64_t)a.max_pages * a.P;
    if (tid < kMaxRun) page[tid] = -1;
    __syncthreads();
    for (int b = tid; b < a.B; b += kAppendThreads) {
      int c0, n, L;
      new_tokens(a.cu_new, a.seq_lens, b, a.n_tokens, cap, a.status, c0, n, L);
      const int i0 = max(c0, r0), i1 = min(c0 + n, r0 + cnt);
      if (i0 < i1) {
        const int p = (a.logical_lens ? a.logical_lens[b] : L) - n - c0;
        for (int i = i0; i < i1; ++i) {
          seq[i - r0] = b;
          slot[i - r0] = L - n + i - c0;
          pos[i - r0] = p + i;
          page[i - r0] = 0;
        }
      }
    }
    __syncthreads();
    if (tid < cnt && page[tid] == 0) {
      const int lp = slot[tid] / a.P;
      const int phys = a.page_table[(size_t)seq[tid] * a.max_pages + lp];
      const bool ok = phys >= 0 && phys < a.n_pool;
      if (!ok) report(a.status, SA_ERR_DEVICE_CHECK);
      page[tid] = ok ? phys : -1;
      slot[tid] -= lp * a.P;
    }
  }
};

// Tokens [r0, r0 + run) of the call: queries rotated, values to their slots.  A row is a head of a
// token; a thread keeps its place in the rows, one unit of four neighbouring ones.
template <int CPR>
__device__ __forceinline__ void append_tokens(const AppendArgs& a, float2* cs, int r0) {
  __shared__ Tokens tok;
  constexpr int U = CPR / 2, N = 4;  // units of a row, rows of a thread
  const int tid = threadIdx.x;
  const int half = a.rot_dim >> 1;
  const bool inter = a.interleaved != 0;
  const int cnt = min(a.run, a.n_tokens - r0);
  const int rows = a.q ? cnt * a.Hq : 0;
  const uint4* src = a.q + (size_t)r0 * a.q_stride;
  const int64_t skip = a.q_stride - (int64_t)a.Hq * CPR;  // between tokens, past their rows
  uint4* dst = a.q_out + (size_t)r0 * a.Hq * CPR;
  const Unit y = unit_of<CPR>(tid % U, a.rot_start, a.rot_dim, inter);
  const int first = tid / U;
  constexpr int step = kAppendThreads / U * N;
  uint4 va[N], vb[N];
  auto fetch = [&](int row0) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int row = row0 + k * (kAppendThreads / U);
      if (row < rows) {
        const uint4* p = src + (row * CPR + quot(row, a.Hq, a.inv_hq) * skip);
        va[k] = p[y.ca];
        vb[k] = p[y.cb];
      }
    }
  };
  fetch(first);  // before it is known where the tokens belong
  tok.find(a, r0, cnt);
  for (int e = tid; e < (a.q ? cnt * half : 0); e += kAppendThreads) {
    const int i = quot(e, half, a.inv_half), j = e - i * half;
    cs[i * half + pair_at(j, half)] = cos_sin(tok.pos[i], a.inv_freq[j]);
  }
  __syncthreads();
  for (int row0 = first; row0 < rows; row0 += step) {
    if (row0 != first) fetch(row0);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int row = row0 + k * (kAppendThreads / U);
      const int i = quot(row, a.Hq, a.inv_hq);
      if (row < rows && tok.page[i] >= 0) {
        if (y.pair >= 0) rotate_unit(va[k], vb[k], cs + i * half + y.pair, half, inter);
        dst[row * CPR + y.ca] = va[k];
        dst[row * CPR + y.cb] = vb[k];
      }
    }
  }
  // values: chunk vc of rows vy, vy + vp, ...
  constexpr int vp = kAppendThreads / CPR;
  const int vy = tid / CPR, vc = tid % CPR;
  const int v_rows = cnt * a.Hkv;
  const uint4* vsrc = a.v + (size_t)r0 * a.v_stride + vc;
#pragma unroll 4
  for (int row = vy; row < v_rows; row += vp) {
    const int i = quot(row, a.Hkv, a.inv_hkv), h = row - i * a.Hkv;
    const int phys = tok.page[i];
    const uint4 w = vsrc[i * a.v_stride + h * CPR];
    if (phys >= 0)
      a.v_cache[(((size_t)phys * a.Hkv + h) * a.P + tok.slot[i]) * CPR + vc] = w;
  }
  __syncthreads();  // the shared arrays are free for the next run
}

// Queries of the latent geometry, a range of pieces (kHeads heads of a token) per CTA: a piece
// comes into shared memory as one bulk copy, its few rotated channels are turned there, and it
// leaves as one; the other eight ninths are never touched by a thread.  Meanwhile the next
// pieces are on their way in and the last one is on its way out.
__device__ __forceinline__ void append_queries(const AppendArgs& a, uint8_t* smem) {
  constexpr int CPR = 72, kParts = 128 / kHeads;
  __shared__ uint64_t full[kStages];
  __shared__ Tokens tok;  // of tokens [known, known + kMaxKnown)
  __shared__ int quit;
  float2* cs = reinterpret_cast<float2*>(smem + kStages * kPieceBytes);
  const int tid = threadIdx.x;
  const int half = a.rot_dim >> 1, n_rot = a.rot_dim >> 4;
  const bool inter = a.interleaved != 0;
  const int64_t pieces = (int64_t)a.n_tokens * kParts;
  const int64_t p0 = pieces * blockIdx.x / a.n_query_ctas;
  const int np = (int)(pieces * (blockIdx.x + 1) / a.n_query_ctas - p0);
  auto load = [&](int n) {  // piece n of this CTA; one thread
    const int64_t p = p0 + n;
    mbar_arrive_expect_tx(&full[n % kStages], kPieceBytes);
    bulk_load(smem + n % kStages * kPieceBytes,
              a.q + (p / kParts) * a.q_stride + (p % kParts) * (kHeads * CPR), kPieceBytes,
              &full[n % kStages]);
  };
  if (tid == 0) {
    quit = 0;
    for (int x = 0; x < kStages; ++x) mbar_init(&full[x], 1);
    fence_mbar_init();
    for (int n = 0; n < min(np, kStages); ++n) load(n);
  }
  int known = -1, turned = -1;  // first of the known tokens, token that cs is of
  const int h = n_rot ? tid / n_rot : kHeads;  // this thread's head and unit
  const Unit y = unit_of<CPR>(n_rot ? tid % n_rot : 0, a.rot_start, a.rot_dim, inter);
  int n = 0;
  for (; n < np; ++n) {
    const int r = (int)((p0 + n) / kParts), part = (int)((p0 + n) % kParts);
    if (known < 0 || r >= known + kMaxKnown) {
      __syncthreads();  // (quit and the barriers are set up; tok was read)
      known = r;
      tok.find(a, known, min(kMaxKnown, a.n_tokens - known));
    }
    if (turned != r) {
      turned = r;
      for (int j = tid; j < half; j += kAppendThreads)
        cs[pair_at(j, half)] = cos_sin(tok.pos[r - known], a.inv_freq[j]);
    }
    __syncthreads();
    uint4* buf = reinterpret_cast<uint4*>(smem + n % kStages * kPieceBytes);
    const bool here = tc::wait(&full[n % kStages], (n / kStages) & 1, &quit, a.status);
    if (here) {
      for (int row = h; row < kHeads; row += kAppendThreads / n_rot) {
        uint4 va = buf[row * CPR + y.ca], vb = buf[row * CPR + y.cb];
        rotate_unit(va, vb, cs + y.pair, half, inter);
        buf[row * CPR + y.ca] = va;
        buf[row * CPR + y.cb] = vb;
      }
      tc::fence_async_smem();
    }
    if (!__syncthreads_and(here)) break;
    if (tid == 0) {
      if (tok.page[r - known] >= 0)
        bulk_store(a.q_out + ((size_t)r * 128 + part * kHeads) * CPR, buf, kPieceBytes);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      if (n > 0 && n - 1 + kStages < np) {  // into the stage of the piece before this one
        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        load(n - 1 + kStages);
      }
    }
  }
  if (tid == 0) {
    // nothing is on its way when the CTA ends (n < np: a wait ran out)
    for (int i = n; i < min(np, n == 0 ? kStages : n - 1 + kStages); ++i)
      mbar_wait(&full[i % kStages], (i / kStages) & 1);
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
}

template <int CPR>
__global__ void __launch_bounds__(kAppendThreads, CPR == 72 ? 3 : 4)
append_kernel(const AppendArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  if (threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;");
  const int cta = blockIdx.x - a.n_query_ctas;
  if (cta >= 0 && cta < a.n_page_ctas) {
    append_pages<CPR>(a, smem, cta);
  } else if constexpr (CPR == 72) {
    append_queries(a, smem);
  } else {
    const int64_t step = (int64_t)(gridDim.x - a.n_query_ctas - a.n_page_ctas) * a.run;
    for (int64_t r0 = (int64_t)(cta - a.n_page_ctas) * a.run; r0 < a.n_tokens; r0 += step)
      append_tokens<CPR>(a, reinterpret_cast<float2*>(smem), (int)r0);
  }
}

}  // namespace

cudaError_t launch_append(const sa_geom& g, const AppendCall& c, cudaStream_t stream) {
  AppendArgs a;
  a.q = static_cast<const uint4*>(c.q);
  a.k = static_cast<const uint4*>(c.k);
  a.v = static_cast<const uint4*>(c.v);
  a.q_stride = c.q_stride / 8;
  a.k_stride = c.k_stride / 8;
  a.v_stride = c.v_stride / 8;
  a.cu_new = c.cu_new;
  a.page_table = c.page_table;
  a.seq_lens = c.seq_lens;
  a.logical_lens = c.logical_lens;
  a.inv_freq = c.inv_freq;
  a.q_out = static_cast<uint4*>(c.q_out);
  a.k_cache = static_cast<uint4*>(c.k_cache);
  a.v_cache = static_cast<uint4*>(c.v_cache);
  a.summ = c.summ8 ? c.summ8 : c.summ;
  a.status = c.status;
  a.n_tokens = c.n_tokens;
  a.B = g.B;
  a.Hq = g.Hq;
  a.Hkv = g.Hkv;
  a.P = g.P;
  a.max_pages = g.max_pages;
  a.n_pool = g.n_pool;
  a.rot_start = c.rot_start;
  a.rot_dim = c.rot_dim;
  a.interleaved = c.interleaved;
  a.want = c.summ8 ? 2 : c.summ ? 1 : 0;
  // pages that n_tokens new tokens of min(B, n_tokens) sequences can touch: a run of n
  // tokens touches at most (n - 1) / P + 2 pages and no more than n
  const int64_t nseq = g.B < c.n_tokens ? g.B : c.n_tokens;
  int64_t items = c.n_tokens / g.P + 2 * nseq;
  if (items > c.n_tokens) items = c.n_tokens;
  if (items > 1 << 20) items = 1 << 20;  // the kernel strides over the rest
  a.n_page_ctas = (int)items;
  auto inv = [](int d) { return d ? (uint32_t)(((1ull << 32) + d - 1) / d) : 0; };
  a.inv_half = inv(c.rot_dim / 2);
  a.inv_hq = inv(g.Hq);
  a.inv_hkv = inv(g.Hkv);
  // cos and sin of the tokens of a page or a run: at most 32 KB
  const size_t table = (size_t)(c.rot_dim / 2) * sizeof(float2);
  size_t smem = g.P * table;
  int64_t runs = 0;
  a.n_query_ctas = 0;
  if (g.Dk != 576) {
    a.run = kRunUnits / (g.Hq * (g.Dk / 16));
    a.run = a.run < 1 ? 1 : a.run > kMaxRun ? kMaxRun : a.run;
    runs = ((int64_t)c.n_tokens + a.run - 1) / a.run;
    if (runs > 1 << 20) runs = 1 << 20;
    if (a.q) smem = std::max(smem, a.run * table);
  } else {
    smem += kLatentGroups * 72 * sizeof(Range);
    if (a.q) {
      a.n_query_ctas = (int)std::min<int64_t>((int64_t)c.n_tokens * (128 / kHeads),
                                              kQueryCtas * c.n_sm);
      smem = std::max(smem, kStages * kPieceBytes + table);
    }
  }
  const void* fn;
  switch (g.Dk) {
    case 64: fn = reinterpret_cast<const void*>(append_kernel<8>); break;
    case 128: fn = reinterpret_cast<const void*>(append_kernel<16>); break;
    case 576: fn = reinterpret_cast<const void*>(append_kernel<72>); break;
    default: return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t cfg = {};
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kStages * kPieceBytes + 32768);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(a.n_query_ctas + items + runs));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // may begin before the previous kernel has ended (it waits)
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&a};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace sa
