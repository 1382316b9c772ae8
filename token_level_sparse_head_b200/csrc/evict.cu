// Eviction from the caches by accumulated attention weight (sm_100a).
//
// Every (b, h) keeps min(N_b, keep_b) rows: the sinks, the newest rows, then the largest weights.
//   evict_keys_kernel  turns weights into order-preserving 32-bit keys (the top-k selection's
//       form) and histograms their first digit; the forced rows get keys above every weight's.
//   select_topk_kernel (the decode step's selection) then lists the kept positions, ascending.
//   move_kernel        moves the kept rows down in place.
// In place: row j of the result is row idx[j] >= j of the source, and idx ascends.  A CTA takes a
// segment of 64 result rows of one (b, h): it reads all of their sources (K, V, projected rows,
// gate terms, weights: 37 KB with d = 128) into registers, sets the segment's flag, waits for the
// flags of the segments that read the rows it is about to write, and writes.  Those are at most
// two, with lower numbers; segments are handed out by a counter, lower ones first, and none waits
// before it has set its flag, so every wait ends.  The reads and writes of all segments are thus
// in flight together; a CTA that went through a column slice of all rows in order, with no flags,
// took 581 us for the 1.2 GB of a batch of 16 (8K to 128K rows, an eighth kept), this form 256 us
// (4.9 TB/s); for one sequence of 32K 28.8 against 13.7 us.
#include "sas_device.cuh"
#include "sas_kernels.h"

namespace sas {
namespace {

constexpr int kKeyThreads = 512;
// Each CTA clears and adds up a histogram of 8192 counts: many keys per CTA where there are CTAs
// enough for every SM, fewer where there are not.  The call with 4096 and with 16384 keys a CTA: 8 heads
// of 32K rows 21.8 and 25.6 us, 32 of 64K 54.3 and 56.1, 128 of 32K 93.6 and 92.6, 128 of 64K 176 and 171.
constexpr int kKeysPerCta = 16384, kKeysPerCtaFew = 4096;

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
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < p.segs; i += kKeyThreads) p.flags[(size_t)bh * p.segs + i] = 0u;
    if (bh == 0 && threadIdx.x == 0) *p.ticket = 0u;
  }
  if (!sel.ranked) return;  // the selection then reads neither keys nor histogram
  const int i0 = blockIdx.x * p.keys_per_cta;
  const int i1 = min(i0 + p.keys_per_cta, n);
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

constexpr int kMoveThreads = 256;
constexpr int kSeg = 64;                        // rows of a segment: one page of the result
constexpr long long kWaitCycles = 4000000000LL;

// A load that stays before the flag that tells others its source may be overwritten.
__device__ __forceinline__ uint4 ld_ordered128(const void* p) {
  uint4 v;
  asm volatile("ld.relaxed.gpu.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float ld_ordered(const float* p) {
  float v;
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
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

// ROW_BYTES of a K or V row; a segment's rows are read whole before its first row is written.
template <int ROW_BYTES>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p) {
  constexpr int PIECES = ROW_BYTES / 16;                     // 16-byte pieces of a row
  constexpr int PER = kSeg * PIECES / kMoveThreads;          // per thread and array
  constexpr int PROJ = kSeg * 128 / 16 / kMoveThreads;       // of the widest projected row
  __shared__ long long src_s[kSeg], dst_s[kSeg];
  __shared__ int idx_s[kSeg + 1], ticket_s, first_s, go_s;
  // No early trigger: all that the next call's first kernel could do before its wait is set up barriers.
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) ticket_s = (int)atomicAdd(p.ticket, 1u);
  __syncthreads();
  const int BH = p.B * p.Hkv;
  const int bh = ticket_s % BH, sg = ticket_s / BH;          // lower segments of a (b, h) have earlier tickets
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  const int2 pl = p.plan[b];
  const int n = pl.x, kept = pl.y;
  const int j0 = sg * kSeg;
  if (sg == 0 && h == 0 && tid == 0) p.seqlens_out[b] = kept;
  if (n == 0 || (j0 >= kept && sg > 0)) return;
  const int rows = min(kSeg, kept - j0);
  const int32_t* idx = p.idx + (size_t)bh * p.keep_max;
  if (tid < kSeg) {
    long long s = -1, d = -1;
    int i = n;
    if (tid < rows) {
      i = idx[j0 + tid];
      if (i < 0 || i >= n) {                                 // a selection that gave up
        record_error(p.err, kDevBadIndex, (uint32_t)b);
        i = j0 + tid;
      }
      if (i > j0 + tid) {                                    // else the row stays where it is
        s = cache_row(p, b, h, i);
        d = cache_row(p, b, h, j0 + tid);
        if (s < 0 || d < 0) s = d = -1;
      }
    }
    idx_s[tid] = i;
    src_s[tid] = s;
    dst_s[tid] = d;
  } else if (tid < kSeg + 32) {
    // the first kept row whose source lies at or behind j0: idx ascends, 32 probes a step
    int lo = 0, cnt = min(j0 + 1, kept);                     // idx[j0] >= j0
    while (cnt > 0) {
      const int step = (cnt + 31) / 32;
      const int at = lo + min(lane * step + step - 1, cnt - 1);
      const unsigned below = __ballot_sync(0xffffffffu, lane * step < cnt && idx[at] < j0);
      const int k = __popc(below);                           // whole steps below j0
      lo += min(k * step, cnt);
      cnt = step == 1 ? 0 : max(0, min(step - 1, cnt - k * step));
    }
    if (lane == 0) first_s = lo;
  } else if (tid == kSeg + 32) {
    idx_s[kSeg] = j0 + kSeg < kept ? idx[j0 + kSeg] : n;     // where the next segment's rows begin
  }
  __syncthreads();

  // ---- read ----
  uint4 kv[2][PER] = {}, pj[PROJ] = {};
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int e = tid + u * kMoveThreads, r = e / PIECES, c = e % PIECES;
      const long long s = src_s[r];
      if (s >= 0) kv[a][u] = ld_ordered128((a ? p.V : p.K) + (size_t)s * ROW_BYTES + c * 16);
    }
  const int pp = p.Kproj == nullptr ? 0 : p.proj_bytes / 16;
#pragma unroll
  for (int u = 0; u < PROJ; ++u) {
    const int e = tid + u * kMoveThreads;
    if (e < kSeg * pp) {
      const long long s = src_s[e / pp];
      if (s >= 0) pj[u] = ld_ordered128(p.Kproj + (size_t)s * p.proj_bytes + (e % pp) * 16);
    }
  }
  float w = 0.f, g = 0.f;
  const size_t row0 = (size_t)bh * p.cap;
  if (tid < rows) {
    w = ld_ordered(p.weights + row0 + idx_s[tid]);
    if (p.log_g != nullptr) g = ld_ordered(p.log_g + row0 + idx_s[tid]);
  }
  // A barrier that takes what was loaded as its input: no load is still on its way behind it.
  uint32_t x = __float_as_uint(w) ^ __float_as_uint(g);
#pragma unroll
  for (int u = 0; u < PER; ++u) x ^= kv[0][u].x ^ kv[0][u].w ^ kv[1][u].x ^ kv[1][u].w;
#pragma unroll
  for (int u = 0; u < PROJ; ++u) x ^= pj[u].x ^ pj[u].w;
  __syncthreads_or((int)x);

  // ---- the rows to be written may be the sources of this segment or of earlier ones ----
  uint32_t* flag = p.flags + (size_t)bh * p.segs;
  if (tid == 0) {
    // release: the reads of all threads before the barrier come before the flag
    st_release(flag + sg, 1u);
    go_s = 1;
    // rows j0 .. j0 + 63 are the sources of at most 64 kept rows, from first_s on
    const long long t0 = clock64();
    for (int i = first_s / kSeg; i <= min(first_s / kSeg + 1, sg - 1); ++i)
      while (ld_acquire(flag + i) == 0u)
        if (clock64() - t0 > kWaitCycles) {
          record_error(p.err, kDevWaitTimeout, (uint32_t)bh);
          go_s = 0;
          break;
        }
  }
  __syncthreads();
  if (!go_s) return;

  // ---- write ----
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int e = tid + u * kMoveThreads, r = e / PIECES, c = e % PIECES;
      const long long d = dst_s[r];
      if (d >= 0) *reinterpret_cast<uint4*>((a ? p.V : p.K) + (size_t)d * ROW_BYTES + c * 16) = kv[a][u];
    }
#pragma unroll
  for (int u = 0; u < PROJ; ++u) {
    const int e = tid + u * kMoveThreads;
    if (e < kSeg * pp) {
      const long long d = dst_s[e / pp];
      if (d >= 0) *reinterpret_cast<uint4*>(p.Kproj + (size_t)d * p.proj_bytes + (e % pp) * 16) = pj[u];
    }
  }
  if (tid < rows) {
    p.weights_out[row0 + j0 + tid] = w;
    if (p.log_g != nullptr) p.log_g[row0 + j0 + tid] = g;
  }
  // Zeros behind the kept weights: this segment takes the positions from its first source to the
  // next segment's, which nobody else reads.
  const int z0 = max(kept, sg == 0 ? 0 : idx_s[0]), z1 = rows == kSeg ? min(idx_s[kSeg], n) : n;
  float* wo = p.weights_out + row0;
  const int a0 = min((z0 + 3) & ~3, z1), a1 = max(z1 & ~3, a0);
  for (int i = z0 + tid; i < a0; i += kMoveThreads) wo[i] = 0.f;
  for (int i = a0 + tid * 4; i < a1; i += kMoveThreads * 4) *reinterpret_cast<float4*>(wo + i) = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = a1 + tid; i < z1; i += kMoveThreads) wo[i] = 0.f;
}

}  // namespace

cudaError_t launch_evict_keys(EvictParams& p, int sms, cudaStream_t stream) {
  const int smem = kHistBins * 4;
  const cudaError_t e = prepare_kernel((const void*)evict_keys_kernel, smem);
  if (e != cudaSuccess) return e;
  const long long ctas = (long long)((p.cap + kKeysPerCta - 1) / kKeysPerCta) * p.B * p.Hkv;
  p.keys_per_cta = ctas < sms ? kKeysPerCtaFew : kKeysPerCta;
  return launch_pdl(evict_keys_kernel, dim3((unsigned)((p.cap + p.keys_per_cta - 1) / p.keys_per_cta), (unsigned)(p.B * p.Hkv)),
                    dim3(kKeyThreads), (size_t)smem, stream, p);
}

cudaError_t launch_evict_move(const EvictParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((size_t)p.segs * p.B * p.Hkv));
  return p.row_bytes == 256 ? launch_pdl(move_kernel<256>, grid, dim3(kMoveThreads), 0, stream, p)
                            : launch_pdl(move_kernel<128>, grid, dim3(kMoveThreads), 0, stream, p);
}

}  // namespace sas
