// sa_chunk_mla.cu -- exact attention of a ragged chunk of new tokens over the paged cache,
// latent geometry (128 query heads share one 576-wide key, V its first 512 channels).
//
// Method: x_t = scale q . k_t over the tokens t a query sees, one pass over the keys with the
// running maximum m and sum l of the softmax: out = sum 2^(x_t - m) v_t / l.
// One warp per (row, query head), lanes split the channels.
#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {

namespace {

struct ChunkArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* cu_new;
  const int32_t* page_table;
  const int32_t* seq_lens;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int n_tokens, B, Hq, Hkv, P, max_pages, n_pool, sink, window;
  float scale_log2;
};

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

template <int DK, int DV>
__global__ void __launch_bounds__(256) attend_chunk_kernel(const ChunkArgs a) {
  constexpr int NK = DK / 32, NV = DV / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int row = (int)(w / a.Hq), hq = (int)(w % a.Hq), h = hq / (a.Hq / a.Hkv);
  if (row >= a.n_tokens) return;
  int b = -1;
  for (int i = 0; i < a.B; ++i) {
    const int c0 = a.cu_new[i], c1 = a.cu_new[i + 1], L = a.seq_lens[i];
    if (!(c0 >= 0 && c1 >= c0 && c1 <= a.n_tokens && L >= c1 - c0 &&
          L <= (int64_t)a.max_pages * a.P)) {
      if (lane == 0) report(a.status, SA_ERR_DEVICE_CHECK);
    } else if (row >= c0 && row < c1) {
      b = i;
    }
  }
  if (b < 0) return;
  const int slot = a.seq_lens[b] - a.cu_new[b + 1] + row;
  float q[NK], o[NV], m = -INFINITY, l = 0.f;
  for (int j = 0; j < NK; ++j) q[j] = bf(a.q[((size_t)row * a.Hq + hq) * DK + lane + 32 * j]);
  for (int j = 0; j < NV; ++j) o[j] = 0.f;
  for (int t = 0; t <= slot; ++t) {
    if (a.window > 0 && t >= a.sink && t <= slot - a.window) {
      t = slot - a.window;
      continue;
    }
    const int ph = a.page_table[(size_t)b * a.max_pages + t / a.P];
    if (ph < 0 || ph >= a.n_pool) {
      if (lane == 0) report(a.status, SA_ERR_DEVICE_CHECK);
      continue;
    }
    const size_t r = ((size_t)ph * a.Hkv + h) * a.P + t % a.P;
    float x = 0.f;
    for (int j = 0; j < NK; ++j) x += q[j] * bf(a.k[r * DK + lane + 32 * j]);
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    x *= a.scale_log2;
    const float mn = fmaxf(m, x), alpha = fast_exp2(m - mn), p = fast_exp2(x - mn);
    m = mn;
    l = l * alpha + p;
    const uint16_t* vr = DK == DV ? a.v + r * DV : a.k + r * DK;
    for (int j = 0; j < NV; ++j) o[j] = o[j] * alpha + p * bf(vr[lane + 32 * j]);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int j = 0; j < NV; ++j)
    a.out[((size_t)row * a.Hq + hq) * DV + lane + 32 * j] =
        (uint16_t)(pack_bf16(o[j] * inv, 0.f) & 0xFFFFu);
  if (lane == 0)
    a.lse[(size_t)row * a.Hq + hq] = l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_chunk_mla(const sa_geom& g, const ChunkCall& c, cudaStream_t stream) {
  ChunkArgs a;
  a.q = static_cast<const uint16_t*>(c.q);
  a.k = static_cast<const uint16_t*>(c.k_cache);
  a.v = static_cast<const uint16_t*>(c.v_cache);
  a.cu_new = c.cu_new;
  a.page_table = c.page_table;
  a.seq_lens = c.seq_lens;
  a.out = static_cast<uint16_t*>(c.out);
  a.lse = c.lse;
  a.status = c.status;
  a.n_tokens = c.n_tokens;
  a.B = g.B;
  a.Hq = g.Hq;
  a.Hkv = g.Hkv;
  a.P = g.P;
  a.max_pages = g.max_pages;
  a.n_pool = g.n_pool;
  a.sink = c.sink;
  a.window = c.window;
  a.scale_log2 = c.scale * 1.4426950408889634f;
  const int64_t ctas = ((int64_t)c.n_tokens * g.Hq + 7) / 8;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  switch (g.Dk) {
    case 576: attend_chunk_kernel<576, 512><<<(unsigned)ctas, 256, 0, stream>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace sa
