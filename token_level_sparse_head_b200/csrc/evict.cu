// Eviction from the caches by accumulated attention weight (sm_100a).
//
// Every (b, h) keeps min(N_b, keep_b) rows: the sinks, the newest rows, then the largest weights.
//   evict_keys_kernel  turns weights into order-preserving 32-bit keys (the top-k selection's
//       form) and histograms their first digit; the forced rows get keys above every weight's.
//   select_topk_kernel (the decode step's selection) then lists the kept positions, ascending.
//   move_kernel        moves the kept rows down in place.
// In place: row j of the result is row idx[j] >= j of the source, and idx ascends.  A CTA that
// goes through j in order may write rows up to j as soon as it has read their sources: every
// later source lies behind them.  Nothing orders CTAs, so none shares bytes with another: a CTA
// owns a column slice (64 bytes) of one (b, h)'s rows in one array, from the first row to the
// last.  That makes 2 d / 32 + 2 CTAs per (b, h), each with two steps' loads in flight.
#include "sas_device.cuh"
#include "sas_kernels.h"

namespace sas {
namespace {

constexpr int kKeyThreads = 512;
constexpr int kKeysPerCta = 16384;

// NaN counts as the least weight.  A finite or infinite weight's key is at most 0xff800000; the
// newest rows get 0xffc00000 + position (newest largest), the sinks 0xffffffff (ties to the lower).
__device__ __forceinline__ uint32_t evict_key(float w, int pos, int n, int sinks, int recent) {
  uint32_t k = (w != w) ? 0u : float_key(w);
  if (pos >= n - recent) k = 0xffc00000u + (uint32_t)pos;
  if (pos < sinks) k = 0xffffffffu;
  return k;
}

__global__ void __launch_bounds__(kKeyThreads) evict_keys_kernel(const EvictParams p) {
  extern __shared__ uint32_t h_s[];
  for (int i = threadIdx.x; i < kHistBins; i += kKeyThreads) h_s[i] = 0u;
  pdl_wait();
  pdl_trigger();
  const int bh = blockIdx.y;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  int n = p.seqlens[b];
  const int kb = p.keep[b];
  if (n < 0 || n > p.cap) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0) record_error(p.err, kDevBadSeqlen, (uint32_t)b);
    n = 0;
  }
  if (kb > p.keep_max && threadIdx.x == 0 && blockIdx.x == 0 && h == 0) record_error(p.err, kDevKOverMax, (uint32_t)b);
  const SeqSelection sel = seq_selection(min(kb, p.keep_max), n);
  if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0) p.plan[b] = make_int2(n, sel.k_eff);
  if (!sel.ranked) return;  // the selection then reads neither keys nor histogram
  const int i0 = blockIdx.x * kKeysPerCta;
  const int i1 = min(i0 + kKeysPerCta, n);
  if (i0 >= i1) return;
  const int recent = min(max(p.recent, 0), n);
  __syncthreads();
  const float* w = p.weights + (size_t)bh * p.cap;
  uint32_t* keys = p.keys + (size_t)bh * p.cap;
  // cap is a multiple of 4: 16-byte pieces (the last may reach past n, not past cap)
  for (int i = i0 + (int)threadIdx.x * 4; i < i1; i += kKeyThreads * 4) {
    const float4 v = *reinterpret_cast<const float4*>(w + i);
    uint4 k;
    k.x = evict_key(v.x, i, n, p.sinks, recent);
    k.y = evict_key(v.y, i + 1, n, p.sinks, recent);
    k.z = evict_key(v.z, i + 2, n, p.sinks, recent);
    k.w = evict_key(v.w, i + 3, n, p.sinks, recent);
    *reinterpret_cast<uint4*>(keys + i) = k;
    atomicAdd(&h_s[k.x >> kHistShift], 1u);
    if (i + 1 < n) atomicAdd(&h_s[k.y >> kHistShift], 1u);
    if (i + 2 < n) atomicAdd(&h_s[k.z >> kHistShift], 1u);
    if (i + 3 < n) atomicAdd(&h_s[k.w >> kHistShift], 1u);
  }
  __syncthreads();
  uint32_t* hist = p.hist + (size_t)bh * kHistBins;
  for (int i = threadIdx.x; i < kHistBins; i += kKeyThreads)
    if (h_s[i]) atomicAdd(&hist[i], h_s[i]);
}

constexpr int kMoveThreads = 512;

// A load that stays before the barrier that precedes the stores over its source.
__device__ __forceinline__ uint4 ld_ordered128(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ long long cache_row(const EvictParams& p, int b, int h, int pos) {
  if (!p.paged) return ((long long)b * p.Hkv + h) * p.cap + pos;
  const int pg = p.page_table[(size_t)b * p.max_pages + (pos >> 6)];
  if (pg < 0 || pg >= p.num_pages) {
    record_error(p.err, kDevBadPage, (uint32_t)b);
    return -1;
  }
  return ((long long)pg * p.Hkv + h) * 64 + (pos & 63);
}

// Columns [col, col + LPR * 16) of one (b, h)'s rows of `row_bytes` bytes; LPR lanes per row.
template <int LPR>
__device__ __forceinline__ void move_slice(const EvictParams& p, unsigned char* base, int row_bytes, int col, int b, int h,
                                           const int32_t* idx, int kept) {
  constexpr int U = 4;                          // rows per thread and step
  constexpr int RPS = kMoveThreads / LPR;       // rows per instruction of the CTA
  const int part = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  unsigned char* mine = base + col + part * 16;
  uint4 cur[U], nxt[U];
  long long dc[U], dn[U];
  auto load = [&](int step, uint4* v, long long* dst) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = (step * U + u) * RPS + r0;
      dst[u] = -1;
      if (j < kept) {
        const int src = idx[j];
        if (src > j) {                          // src == j: the row stays where it is
          const long long rs = cache_row(p, b, h, src), rd = cache_row(p, b, h, j);
          if (rs >= 0 && rd >= 0) {
            dst[u] = rd;
            v[u] = ld_ordered128(mine + (size_t)rs * row_bytes);
          }
        }
      }
    }
  };
  const int steps = (kept + U * RPS - 1) / (U * RPS);
  if (steps > 0) load(0, cur, dc);
  for (int s = 0; s < steps; ++s) {
    if (s + 1 < steps) load(s + 1, nxt, dn);
    __syncthreads();                            // every source of this step has been read
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dc[u] >= 0) *reinterpret_cast<uint4*>(mine + (size_t)dc[u] * row_bytes) = cur[u];
      cur[u] = nxt[u];
      dc[u] = dn[u];
    }
  }
}

// One fp32 per row, [B][Hkv][cap]; zeros from the kept rows to n if `clear`.
__device__ __forceinline__ void move_scalars(const float* src, float* dst, const int32_t* idx, int kept, int n, bool clear) {
  for (int j0 = 0; j0 < kept; j0 += kMoveThreads * 4) {
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u * kMoveThreads + (int)threadIdx.x;
      v[u] = j < kept ? *reinterpret_cast<const volatile float*>(src + idx[j]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u * kMoveThreads + (int)threadIdx.x;
      if (j < kept) dst[j] = v[u];
    }
    __syncthreads();
  }
  if (clear)
    for (int j = kept + (int)threadIdx.x; j < n; j += kMoveThreads) dst[j] = 0.f;
}

// blockIdx.x: slices of K, then of V, then of Kproj, then log_g, then the weights.
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p) {
  // No early trigger: this kernel writes the lengths, which the next kernel may read before its wait.
  pdl_wait();
  const int bh = blockIdx.y;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  const int2 pl = p.plan[b];
  const int n = pl.x, kept = pl.y;
  const int32_t* idx = p.idx + (size_t)bh * p.keep_max;
  const int kv_slices = p.row_bytes / 64;
  const int proj_slices = p.Kproj == nullptr ? 0 : (p.proj_bytes + 63) / 64;
  int s = blockIdx.x;
  if (s < 2 * kv_slices) {
    if (kept == n) return;  // nothing is evicted, nothing moves
    move_slice<4>(p, s < kv_slices ? p.K : p.V, p.row_bytes, (s % kv_slices) * 64, b, h, idx, kept);
    return;
  }
  s -= 2 * kv_slices;
  if (s < proj_slices) {
    if (kept == n) return;
    if (p.proj_bytes >= 64) move_slice<4>(p, p.Kproj, p.proj_bytes, s * 64, b, h, idx, kept);
    else if (p.proj_bytes == 32) move_slice<2>(p, p.Kproj, p.proj_bytes, 0, b, h, idx, kept);
    else move_slice<1>(p, p.Kproj, p.proj_bytes, 0, b, h, idx, kept);
    return;
  }
  s -= proj_slices;
  if (s == 0) {
    move_scalars(p.weights + (size_t)bh * p.cap, p.weights_out + (size_t)bh * p.cap, idx, kept, n, true);
    if (h == 0 && threadIdx.x == 0) p.seqlens_out[b] = kept;
  } else if (kept < n) {
    move_scalars(p.log_g + (size_t)bh * p.cap, p.log_g + (size_t)bh * p.cap, idx, kept, n, false);
  }
}

}  // namespace

cudaError_t launch_evict_keys(const EvictParams& p, cudaStream_t stream) {
  const int smem = kHistBins * 4;
  const cudaError_t e = prepare_kernel((const void*)evict_keys_kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(evict_keys_kernel, dim3((unsigned)((p.cap + kKeysPerCta - 1) / kKeysPerCta), (unsigned)(p.B * p.Hkv)),
                    dim3(kKeyThreads), (size_t)smem, stream, p);
}

cudaError_t launch_evict_move(const EvictParams& p, cudaStream_t stream) {
  const int units = 2 * (p.row_bytes / 64) + (p.Kproj == nullptr ? 0 : (p.proj_bytes + 63) / 64) + 1 + (p.log_g != nullptr);
  return launch_pdl(move_kernel, dim3((unsigned)units, (unsigned)(p.B * p.Hkv)), dim3(kMoveThreads), 0, stream, p);
}

}  // namespace sas
