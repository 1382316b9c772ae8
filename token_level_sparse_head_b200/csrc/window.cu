// Decode of the newest token of every sequence with a sliding window and sinks, fp32 output, and
// the softmax weights of each KV head's group added up per cached row (sm_100a).
//
//   out = sum_j softmax_j(sigma q.K_j) V_j over the visible j;  weights[j] += sum_g softmax_g(j).
//
// Bound by reading the visible K and V rows once (4 d bytes a row and KV head; about G flop a
// byte).  Work: the visible rows of a (b, h, group of up to 16 query heads) are a list of 64-row
// pages (the sinks' pages, then the window's); the pages of all of them, one after another, are
// cut into equal contiguous shares, one per CTA, so a ragged batch loads every SM alike.  A share
// that holds part of a task leaves a partial (m, l, acc); the last CTA of a task joins them in order.
// CTA: one producer warp feeds a ring of pages with tiled bulk copies (128-byte swizzle); two
// groups of four warps take the pages in turn, 16 rows of a page per warp.  The products run on
// the warp-level matrix instruction with the heads as its 8 columns: 16 rows x 8 heads per
// instruction fit a GEMV-shaped problem (the 128-row form would leave most of its rows empty),
// and the scores S^T = K Q^T come out with a lane's columns = the accumulator's columns of
// O^T = V^T P^T, so the softmax state needs no exchange between lanes but the maximum's.  P enters
// the second product as three bf16 terms of 8 bits each, which hold its 24 bits exactly, because
// the output is fp32: one bf16 term would be off by up to 2^-8, two by 2^-16.
// Measured (8 KV heads, d = 128): window 4096 at B = 16 52 us, 5.2 TB/s; whole caches of 4 x 64K rows
// with weights 197 to 200 us, 5.5 TB/s, of which the weights' own pass takes 13; window 1024 at B = 1 9.7
// us, host time; the kernel's chain of page, products and join counts there and not the bytes.
#include "sas_device.cuh"
#include "sas_kernels.h"

namespace sas {
namespace {

constexpr int kConsumers = 8;
constexpr int kGroups = 2;
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kPage = 64;

template <int D, int NT>
struct Geo {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF_BYTES = kPage * 128;
  static constexpr int OP_BYTES = HALVES * HALF_BYTES;    // K (or V) of a page
  static constexpr int STAGE_BYTES = 2 * OP_BYTES;
  static constexpr int STAGES = D == 64 ? 8 : (NT == 1 ? 6 : 4);
  static constexpr int PITCH = D + 4;                     // floats: heads of a warp's merge rows
  static constexpr int MERGE = kConsumers * NT * 8 * PITCH;
  static_assert(MERGE >= kChunkMaxCtas * 16, "the weights of the partials lie in the merge rows");
  static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + MERGE * 4;
};

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory"); }

__device__ __forceinline__ int seq_len(const WindowParams& p, int b) {
  const int n = p.seqlens[b];
  return (n < 0 || n > p.cap) ? 0 : n;
}
// A sequence without cached rows has one page none of whose rows is visible: its zeros are written
// by the same path.
__device__ __forceinline__ VisiblePages seq_pages(const WindowParams& p, int n) {
  VisiblePages v = visible_pages(n - 1, n - 1, p.window, p.sinks);
  v.nv = max(v.nv, 1);
  return v;
}

// Position in the list of pages: (b, h, head group, page) in this order.
struct Cursor {
  int b, h, hg, page;
};

// Joins np partials of CTAs c0, c0 + 1, ...; the first is c0's second one if `second`.  All consumer threads.
template <int D>
__device__ void join_partials(const WindowParams& p, float (*wts)[16], float* inv_s, int np, int c0, bool second, int heads,
                              size_t o0) {
  auto slot = [&](int i) { return i == 0 ? 2 * (size_t)c0 + (second ? 1 : 0) : 2 * (size_t)(c0 + i); };
  // 16 lanes of a half warp share a head
  const int hd = threadIdx.x / 16, sub = threadIdx.x % 16;
  float M = -INFINITY, L = 0.f;
  if (hd < heads)
    for (int i = sub; i < np; i += 16) M = fmaxf(M, __ldcg(&p.ml[slot(i) * 16 + hd]).x);
#pragma unroll
  for (int o = 8; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (hd < heads)
    for (int i = sub; i < np; i += 16) {
      const float2 x = __ldcg(&p.ml[slot(i) * 16 + hd]);
      const float f = x.x == -INFINITY ? 0.f : ex2(x.x - M);
      wts[i][hd] = f;
      L += f * x.y;
    }
#pragma unroll
  for (int o = 8; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (sub == 0 && hd < heads) {
    inv_s[hd] = L > 0.f ? 1.f / L : 0.f;
    const float ls = L > 0.f ? M + log2f(L) : -INFINITY;
    if (p.lse != nullptr) p.lse[o0 + hd] = ls * 0.69314718055994531f;
    if (p.lse2 != nullptr) p.lse2[o0 + hd] = ls;
  }
  consumers_sync();
  for (int e = threadIdx.x; e < heads * (D / 4); e += kConsumers * 32) {
    const int g = e / (D / 4), c4 = (e % (D / 4)) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < np; ++i) {
      const float f = wts[i][g];
      const float4 y = __ldcg(reinterpret_cast<const float4*>(p.part + (slot(i) * 16 + g) * D + c4));
      x.x += f * y.x;
      x.y += f * y.y;
      x.z += f * y.z;
      x.w += f * y.w;
    }
    const float r = inv_s[g];
    *reinterpret_cast<float4*>(p.out + (o0 + g) * D + c4) = make_float4(x.x * r, x.y * r, x.z * r, x.w * r);
  }
  consumers_sync();
}

template <int D, int NT, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, 1) window_kernel(const __grid_constant__ WindowParams p) {
  using Gm = Geo<D, NT>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* merge = reinterpret_cast<float*>(ring + Gm::STAGES * Gm::STAGE_BYTES);
  __shared__ uint64_t full[Gm::STAGES], empty[Gm::STAGES];
  __shared__ float wm[kConsumers][NT * 8], wl[kConsumers][NT * 8];
  __shared__ int red[kThreads / 32];
  __shared__ Cursor start_s;
  __shared__ float inv_s[16];
  __shared__ int last_s;
  __shared__ volatile int abort_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < Gm::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kConsumers / kGroups);
    }
    fence_barrier_init();
    abort_s = 0;
  }
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's share of the pages ----
  const int per_page = p.Hkv * p.hgs;
  int sum = 0;
  for (int b = tid; b < p.B; b += kThreads) {
    const int n = p.seqlens[b];
    if (blockIdx.x == 0 && (n < 0 || n > p.cap)) record_error(p.err, kDevBadSeqlen, (uint32_t)b);
    sum += seq_pages(p, seq_len(p, b)).nv * per_page;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) total += red[w];
  const int share = (total + p.ctas - 1) / p.ctas;
  const int u0 = min((int)blockIdx.x * share, total), u1 = min(u0 + share, total);
  if (warp == 0) {
    int base = 0;
    Cursor c = {-1, 0, 0, 0};
    for (int b0 = 0; b0 < p.B && u0 < total; b0 += 32) {
      const int b = b0 + lane;
      const int nv = b < p.B ? seq_pages(p, seq_len(p, b)).nv : 0;
      int inc = nv * per_page;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const int lo = base + inc - nv * per_page, hi = base + inc;
      const unsigned hit = __ballot_sync(0xffffffffu, u0 >= lo && u0 < hi);
      if (hit) {
        const int l = __ffs(hit) - 1;
        const int off = u0 - __shfl_sync(0xffffffffu, lo, l);
        const int nv_at = __shfl_sync(0xffffffffu, nv, l);
        const int t = off / nv_at;
        c = Cursor{b0 + l, t / p.hgs, t % p.hgs, off % nv_at};
        break;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) start_s = c;
  }
  __syncthreads();
  Cursor cur = start_s;
  const int hgw = p.hgs == 1 ? p.G : ((p.G + p.hgs - 1) / p.hgs + 1) & ~1;  // heads per group

  if (warp == kConsumers) {
    // ------------------------------------------------------------------ producer
    int cnt = 0, sent = 0;
    for (int u = u0; u < u1;) {
      const int n = seq_len(p, cur.b);
      const VisiblePages vis = seq_pages(p, n);
      const int pe = min(vis.nv, cur.page + (u1 - u));
      for (int v0 = cur.page; v0 < pe; v0 += 32) {
        // 32 page-table entries at a time
        int row = p.row_end;
        const int v = v0 + lane;
        if (v < pe) {
          const int lp = vis.page(v);
          if (lp * kPage < n) {
            if (p.paged) {
              const int pg = p.page_table[(size_t)cur.b * p.max_pages + lp];
              if (pg < 0 || pg >= p.num_pages) record_error(p.err, kDevBadPage, (uint32_t)cur.b);
              else row = (pg * p.Hkv + cur.h) * kPage;
            } else {
              row = (cur.b * p.Hkv + cur.h) * p.cap + lp * kPage;
            }
          }
        }
        for (int i = 0; i < min(32, pe - v0); ++i, ++cnt) {
          const int y = __shfl_sync(0xffffffffu, row, i);
          const int st = cnt % Gm::STAGES;
          if (lane == 0 && !abort_s) {
            const bool ok = cnt < Gm::STAGES || mbar_wait_bounded(&empty[st], ((cnt / Gm::STAGES) & 1) ^ 1);
            if (!ok) {
              abort_s = 1;
            } else {
              sent = cnt + 1;
              unsigned char* dst = ring + (size_t)st * Gm::STAGE_BYTES;
              mbar_arrive_expect_tx(&full[st], Gm::STAGE_BYTES);
#pragma unroll
              for (int hf = 0; hf < Gm::HALVES; ++hf) {
                tma_2d(dst + hf * Gm::HALF_BYTES, &p.kmap, hf * 64, y, &full[st]);
                tma_2d(dst + Gm::OP_BYTES + hf * Gm::HALF_BYTES, &p.vmap, hf * 64, y, &full[st]);
              }
            }
          }
          __syncwarp();
        }
      }
      u += pe - cur.page;
      cur.page = 0;
      if (pe == vis.nv && ++cur.hg == p.hgs) {
        cur.hg = 0;
        if (++cur.h == p.Hkv) {
          cur.h = 0;
          ++cur.b;
        }
      }
    }
    // after a wait that ran out: the copies in flight land before the CTA ends
    if (lane == 0 && abort_s)
      for (int i = max(0, sent - Gm::STAGES); i < sent; ++i) mbar_wait_bounded(&full[i % Gm::STAGES], (i / Gm::STAGES) & 1);
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int grp = warp / (kConsumers / kGroups);
  const int krow = (warp % (kConsumers / kGroups)) * 16;   // first row of this warp in a page
  const int h2 = (lane & 3) * 2;                           // the lane's first head of each 8
  const int r4 = lane >> 2;
  int cnt = 0;
  bool alive = true;
  for (int u = u0; u < u1;) {
    const int b = cur.b, h = cur.h, hg = cur.hg;
    const int n = seq_len(p, b);
    const VisiblePages vis = seq_pages(p, n);
    const int pb = cur.page, pe = min(vis.nv, pb + (u1 - u));
    const int heads = min(hgw, p.G - hg * hgw);
    const int hq0 = h * p.G + hg * hgw;
    const int bh = b * p.Hkv + h;

    // Q^T as the B operand: columns = heads, 2 k-values per register
    uint32_t qf[D / 16][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int head = nt * 8 + r4;
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(p.q + ((size_t)b * p.Hq + hq0 + min(head, heads - 1)) * D);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qf[ks][nt][0] = head < heads ? qp[ks * 8 + (lane & 3)] : 0u;
        qf[ks][nt][1] = head < heads ? qp[ks * 8 + 4 + (lane & 3)] : 0u;
      }
    }
    float m[NT][2], l[NT][2], acc[D / 16][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
    }

    for (int v = pb; v < pe; ++v, ++cnt) {
      if ((cnt % kGroups) != grp) continue;
      const int st = cnt % Gm::STAGES;
      if (alive && !__all_sync(0xffffffffu, mbar_wait_bounded(&full[st], (cnt / Gm::STAGES) & 1))) {
        alive = false;
        abort_s = 1;
        if (lane == 0) record_error(p.err, kDevWaitTimeout, (uint32_t)bh);
      }
      if (!alive) continue;
      const uint32_t kb = smem_u32(ring + (size_t)st * Gm::STAGE_BYTES);
      const uint32_t vb = kb + Gm::OP_BYTES;
      const int lp = vis.page(v);
      const int pos0 = lp * kPage + krow;
      // every row of the page visible?
      const bool whole = lp * kPage + kPage <= n && (p.window <= 0 || lp * kPage >= vis.first || lp * kPage + kPage <= p.sinks);

      // S^T = K Q^T for 16 rows
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
      {
        const int row = krow + (lane & 15);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t a[4];
          const int chunk = ((ks & 3) * 2 + (lane >> 4)) ^ (row & 7);
          ldsm4(a, kb + (ks >> 2) * Gm::HALF_BYTES + row * 128 + chunk * 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a, qf[ks][nt][0], qf[ks][nt][1]);
        }
      }
      bool vis0 = true, vis8 = true;
      uint32_t km0 = 0xffffffffu, km8 = 0xffffffffu;
      if (!whole) {
        auto seen = [&](int r) {
          const int j = pos0 + r;
          return j < n && (p.window <= 0 || j >= vis.first || j < p.sinks);
        };
        vis0 = seen(r4);
        vis8 = seen(r4 + 8);
        km0 = (seen(h2) ? 0xffffu : 0u) | (seen(h2 + 1) ? 0xffff0000u : 0u);
        km8 = (seen(h2 + 8) ? 0xffffu : 0u) | (seen(h2 + 9) ? 0xffff0000u : 0u);
      }
      uint32_t pt[3][NT][2];  // the three terms of P^T as the B operand
      bool grow = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = ((i < 2) ? vis0 : vis8) ? s[nt][i] * p.scale_log2 : -INFINITY;
        if (WEIGHTS) {
          const int hd = nt * 8 + h2;
          if (hd < heads) {
            float* zp = p.z + ((size_t)bh * p.zcap + (size_t)v * kPage + krow + r4) * p.gpad + hg * hgw + hd;
            *reinterpret_cast<float2*>(zp) = make_float2(s[nt][0], s[nt][1]);
            *reinterpret_cast<float2*>(zp + 8 * p.gpad) = make_float2(s[nt][2], s[nt][3]);
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = fmaxf(s[nt][c], s[nt][c + 2]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mx[nt][c] = x;
          grow |= x > m[nt][c];
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float mn = fmaxf(m[nt][c], mx[nt][c]);
            const float f = mn == -INFINITY ? 1.f : ex2(m[nt][c] - mn);
            m[nt][c] = mn;
            l[nt][c] *= f;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
              acc[mt][nt][c] *= f;
              acc[mt][nt][c + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float mm = m[nt][i & 1];
          e[i] = mm == -INFINITY ? 0.f : ex2(s[nt][i] - mm);
        }
        l[nt][0] += e[0] + e[2];
        l[nt][1] += e[1] + e[3];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = e[2 * c], y = e[2 * c + 1];
#pragma unroll
          for (int t = 0; t < 3; ++t) {
            const uint32_t w = pack_bf16(x, y);
            x -= bf16lo(w);
            y -= bf16hi(w);
            pt[t][nt][c] = transpose8(w);
          }
        }
      }
      // O^T += V^T P^T
      {
        const int row = krow + ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          uint32_t a[4];
          const int chunk = ((mt & 3) * 2 + ((lane >> 3) & 1)) ^ (row & 7);
          ldsm4t(a, vb + (mt >> 2) * Gm::HALF_BYTES + row * 128 + chunk * 16);
          if (!whole) {  // rows that nobody sees may hold anything: 0 * NaN is not 0
            a[0] &= km0;
            a[1] &= km0;
            a[2] &= km8;
            a[3] &= km8;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // The instruction truncates its sums: over tens of thousands of rows that adds up to a
            // bias, so the 16 rows' product is formed from zero, the small terms first, and added
            // to the running output with rounding (error of 64K rows 5.1e-6 -> 2.5e-7).
            float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 2; t >= 0; --t) mma16816(o, a, pt[t][nt][0], pt[t][nt][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[mt][nt][i] += o[i];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- join the warps ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[nt][c];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (r4 == 0) {
          wm[warp][nt * 8 + h2 + c] = m[nt][c];
          wl[warp][nt * 8 + h2 + c] = x;
        }
      }
    consumers_sync();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int hd = nt * 8 + h2 + c;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, wm[w][hd]);
        const float f = m[nt][c] == -INFINITY ? 0.f : ex2(m[nt][c] - M);
        float* dst = merge + (warp * NT * 8 + hd) * Gm::PITCH + r4;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          dst[mt * 16] = acc[mt][nt][c] * f;
          dst[mt * 16 + 8] = acc[mt][nt][c + 2] * f;
        }
      }
    consumers_sync();
    const bool done = pb == 0 && pe == vis.nv;
    const size_t slot = 2 * (size_t)blockIdx.x + (u == u0 ? 0 : 1);
    for (int e = tid; e < heads * (D / 4); e += kConsumers * 32) {
      const int hd = e / (D / 4), c4 = (e % (D / 4)) * 4;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, wm[w][hd]);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) L += wm[w][hd] == -INFINITY ? 0.f : ex2(wm[w][hd] - M) * wl[w][hd];
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(merge + (w * NT * 8 + hd) * Gm::PITCH + c4);
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      if (done) {
        const float r = L > 0.f ? 1.f / L : 0.f;
        const size_t o = (size_t)b * p.Hq + hq0 + hd;
        *reinterpret_cast<float4*>(p.out + o * D + c4) = make_float4(x.x * r, x.y * r, x.z * r, x.w * r);
        if (c4 == 0) {
          const float ls = M + log2f(L);
          if (p.lse != nullptr) p.lse[o] = L > 0.f ? ls * 0.69314718055994531f : -INFINITY;
          if (WEIGHTS) p.lse2[o] = ls;
        }
      } else {
        *reinterpret_cast<float4*>(p.part + (slot * 16 + hd) * D + c4) = x;
        if (c4 == 0) p.ml[slot * 16 + hd] = make_float2(M, L);
      }
    }
    consumers_sync();
    if (!done) {
      // The last CTA of the task to get here joins its partials, in CTA order: the sum does not
      // depend on which one that is.
      const int t0 = u - pb;                               // the task's first page
      const int c0 = t0 / share, np = (t0 + vis.nv - 1) / share - c0 + 1;
      if (tid == 0) {
        __threadfence();
        const uint32_t k = atomicAdd(p.arrived + c0, 1u);
        if (k == (uint32_t)np - 1) p.arrived[c0] = 0u;
        __threadfence();
        last_s = k == (uint32_t)np - 1;
      }
      consumers_sync();
      if (last_s) join_partials<D>(p, reinterpret_cast<float(*)[16]>(merge), inv_s, np, c0, t0 != c0 * share, heads, (size_t)b * p.Hq + hq0);
    }
    u += pe - pb;
    cur.page = 0;
    if (pe == vis.nv && ++cur.hg == p.hgs) {
      cur.hg = 0;
      if (++cur.h == p.Hkv) {
        cur.h = 0;
        ++cur.b;
      }
    }
  }
}

// weights[b,h,j] += sum_g 2^(z - lse2).  A thread takes kWeightRows visible rows, all of whose loads
// are in flight at once (one row a thread: 17 us for 4 x 64K rows of 8 heads, four: 12.8 us).
constexpr int kWeightThreads = 256, kWeightRows = 4;
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const __grid_constant__ WindowParams p) {
  pdl_wait();
  pdl_trigger();
  const int bh = blockIdx.y;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  const int n = seq_len(p, b);
  if (n == 0) return;
  const VisiblePages vis = seq_pages(p, n);
  const int vr0 = blockIdx.x * kWeightThreads * kWeightRows + threadIdx.x;
  const float* ls = p.lse2 + (size_t)b * p.Hq + h * p.G;
  const float* z = p.z + (size_t)bh * p.zcap * p.gpad;
  float* w = p.weights + (size_t)bh * p.cap;
  int j[kWeightRows];
  float s[kWeightRows];
#pragma unroll
  for (int i = 0; i < kWeightRows; ++i) {
    const int vr = vr0 + i * kWeightThreads;
    j[i] = -1;
    s[i] = 0.f;
    if (vr >= vis.nv * kPage) continue;
    const int at = vis.page(vr / kPage) * kPage + vr % kPage;
    if (at < n && (p.window <= 0 || at >= vis.first || at < p.sinks)) j[i] = at;
  }
  float was[kWeightRows];
#pragma unroll
  for (int i = 0; i < kWeightRows; ++i) was[i] = j[i] >= 0 ? w[j[i]] : 0.f;
  if (p.G % 4 == 0) {
    for (int g = 0; g < p.G; g += 4) {
      const float l0 = ls[g], l1 = ls[g + 1], l2 = ls[g + 2], l3 = ls[g + 3];
#pragma unroll
      for (int i = 0; i < kWeightRows; ++i) {
        if (j[i] < 0) continue;
        const float4 v = __ldcg(reinterpret_cast<const float4*>(z + (size_t)(vr0 + i * kWeightThreads) * p.gpad + g));
        s[i] += ex2(v.x - l0);
        s[i] += ex2(v.y - l1);
        s[i] += ex2(v.z - l2);
        s[i] += ex2(v.w - l3);
      }
    }
  } else {
    for (int g = 0; g < p.G; ++g) {
      const float l0 = ls[g];
#pragma unroll
      for (int i = 0; i < kWeightRows; ++i)
        if (j[i] >= 0) s[i] += ex2(__ldcg(z + (size_t)(vr0 + i * kWeightThreads) * p.gpad + g) - l0);
    }
  }
#pragma unroll
  for (int i = 0; i < kWeightRows; ++i)
    if (j[i] >= 0) w[j[i]] = was[i] + s[i];
}

template <int D, int NT>
cudaError_t launch_t(const WindowParams& p, cudaStream_t stream) {
  using Gm = Geo<D, NT>;
  auto kern = p.weights != nullptr ? window_kernel<D, NT, true> : window_kernel<D, NT, false>;
  cudaError_t e = prepare_kernel((const void*)kern, Gm::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)p.ctas), dim3(kThreads), (size_t)Gm::SMEM, stream, p);
  if (e != cudaSuccess) return e;
  if (p.weights != nullptr)
    return launch_pdl(weights_kernel, dim3((unsigned)((p.zcap + kWeightThreads * kWeightRows - 1) / (kWeightThreads * kWeightRows)), (unsigned)(p.B * p.Hkv)),
                      dim3(kWeightThreads), 0, stream, p);
  return cudaSuccess;
}

}  // namespace

void plan_window(WindowParams& p) {
  p.hgs = (p.G + 15) / 16;
  p.gpad = (p.G + 1) & ~1;
  long long rows = p.cap;
  if (p.window > 0) {
    const long long seen = (long long)p.window + (p.sinks > 0 ? p.sinks : 0) + 3 * kPage;
    if (seen < rows) rows = seen;
  }
  p.zcap = (int)((rows + kPage - 1) / kPage * kPage);
}

size_t window_workspace_bytes(const WindowParams& p, bool weights) {
  size_t o = (size_t)2 * kChunkMaxCtas * 16 * (sizeof(float2) + (size_t)p.d * 4);
  if (weights) {
    o += ((size_t)p.B * p.Hq * 4 + 255) & ~(size_t)255;
    // for any window: the capacity bounds the visible rows
    o += (size_t)p.B * p.Hkv * (((size_t)p.cap + kPage - 1) / kPage * kPage) * p.gpad * 4;
  }
  return o;
}

void bind_window(WindowParams& p, void* scratch, bool weights) {
  unsigned char* w = static_cast<unsigned char*>(scratch);
  p.ml = reinterpret_cast<float2*>(w);
  w += (size_t)2 * kChunkMaxCtas * 16 * sizeof(float2);
  p.part = reinterpret_cast<float*>(w);
  w += (size_t)2 * kChunkMaxCtas * 16 * p.d * 4;
  p.lse2 = nullptr;
  p.z = nullptr;
  if (weights) {
    p.lse2 = reinterpret_cast<float*>(w);
    w += ((size_t)p.B * p.Hq * 4 + 255) & ~(size_t)255;
    p.z = reinterpret_cast<float*>(w);
  }
}

cudaError_t launch_window(const WindowParams& p, cudaStream_t stream) {
  const int hgw = p.hgs == 1 ? p.G : ((p.G + p.hgs - 1) / p.hgs + 1) & ~1;
  if (p.d == 128) return hgw <= 8 ? launch_t<128, 1>(p, stream) : launch_t<128, 2>(p, stream);
  if (p.d == 64) return hgw <= 8 ? launch_t<64, 1>(p, stream) : launch_t<64, 2>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace sas
