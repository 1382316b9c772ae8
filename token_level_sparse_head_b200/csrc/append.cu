// Rows of a chunk of new tokens into the caches: K, V and the projected rows (sm_100a).
//
// Token t of the batch belongs to the sequence b with q_start[b] <= t < q_start[b+1] and sits at
// position N_b - T_b + (t - q_start[b]); every CTA sees for itself whether q_start is in order.  Per
// token and KV head the call copies 2 d bf16 values and computes r dot products of length d in fp32,
// in the summation order of the projection build (8 partial sums over consecutive blocks of d/8
// channels, in channel order, combined as ((p0+p1)+(p2+p3))+((p4+p5)+(p6+p7))), so a row is the same
// bits whichever call wrote it.
//
// Two kernels, by the number of (token, head) pairs:
//   token_kernel  one CTA per pair, 8 threads per output: few tokens, where latency counts;
//   tile_kernel   tiles of 128 tokens x one head, shared by as many CTAs as are resident at once.
//                 M[h] is staged in shared memory once per CTA, transposed to [channel][output];
//                 a tile's keys come by asynchronous copies while the tile before is worked on.
//                 A thread takes 4 outputs of 4 tokens in paired fp32 FMAs (bit-identical to
//                 single ones).
// What bounds the tiles: moving K and V of 8192 tokens and 8 heads (67 MB in and out) takes 9.6 us
// alone, the call with 32 outputs per row 26.5 us: 268 M fp32 FMAs are 7.5 us at full rate, and the
// conversions and loads of their operands as much again.  A form on the matrix instructions would
// have to be the build's and the one-token append's too, for the rows to stay the same bits.
#include <cuda_fp8.h>

#include "sas_device.cuh"
#include "sas_kernels.h"

namespace sas {
namespace {

// Cache row of token t; -1 if the token belongs to nobody or to a sequence that is skipped, -2 - b
// if its page (of sequence b) lies outside the cache.
// ordered: no entry of q_start is smaller than the one before it, so the last start that is not
// above t is t's.  Otherwise the first sequence that may be taken and holds t, in order.
__device__ __forceinline__ long long token_row(const AppendParams& p, bool ordered, int t, int h) {
  int b = 0;
  LargestStart largest;
  if (ordered) {
    int hi = p.B;  // largest b in [0, B) with q_start[b] <= t
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (p.q_start[mid] <= t) b = mid; else hi = mid;
    }
  } else {
    while (b < p.B - 1 && !(p.q_start[b] >= largest.upto(p.q_start, b) && p.q_start[b] <= t && t < p.q_start[b + 1])) ++b;
  }
  const int s0 = p.q_start[b], s1 = p.q_start[b + 1], n = p.seqlens[b];
  if (t < s0 || t >= s1 || chunk_error(s0, s1, ordered ? s0 : largest.upto(p.q_start, b), n, p.n_new, p.cap) != kDevOk) return -1;
  const int pos = n - (s1 - s0) + (t - s0);
  if (!p.paged) return ((long long)b * p.Hkv + h) * p.cap + pos;
  const int pg = p.page_table[(size_t)b * p.max_pages + (pos >> 6)];
  if (pg < 0 || pg >= p.num_pages) return -2 - b;
  return ((long long)pg * p.Hkv + h) * 64 + (pos & 63);
}
__device__ __forceinline__ void record_row(const AppendParams& p, long long row) {
  if (row < -1) record_error(p.err, kDevBadPage, (uint32_t)(-2 - row));
}
// Records why sequences are skipped, those without tokens among them; one CTA of the grid.
template <int THREADS>
__device__ __forceinline__ void record_skipped(const AppendParams& p, bool ordered) {
  LargestStart largest;
  for (int b = threadIdx.x; b < p.B; b += THREADS) {
    const int s0 = p.q_start[b];
    const uint32_t why = chunk_error(s0, p.q_start[b + 1], ordered ? s0 : largest.upto(p.q_start, b), p.seqlens[b], p.n_new, p.cap);
    if (why != kDevOk) record_error(p.err, why, (uint32_t)b);
  }
}

__device__ __forceinline__ unsigned char fp8_of(float a, float s) {
  return (unsigned char)__nv_cvt_float_to_fp8(__fdiv_rn(a, s), __NV_SATFINITE, __NV_E4M3);
}

template <int D, int R, bool FP8>
__global__ void __launch_bounds__(256) token_kernel(const AppendParams p) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  __shared__ long long row_s;
  // looked up as if q_start were in order, while the other threads see whether it is
  if (threadIdx.x == 0) row_s = token_row(p, true, t, h);
  constexpr int BLK = D / 8;
  const int part = threadIdx.x & 7;
  const __nv_bfloat16* kn = p.K_new + (size_t)t * p.kv_stride + (size_t)h * D;
  const __nv_bfloat16* vn = p.V_new + (size_t)t * p.kv_stride + (size_t)h * D;
  // the loads do not need the row: they are in flight while thread 0 looks it up
  uint4 piece = make_uint4(0, 0, 0, 0);
  constexpr int PPR = D / 8;
  if (threadIdx.x < 2 * PPR)
    piece = *reinterpret_cast<const uint4*>((threadIdx.x < PPR ? kn : vn) + (threadIdx.x % PPR) * 8);
  float out[(R + 31) / 32];
  if (p.Kproj != nullptr) {
    float kf[BLK];
#pragma unroll
    for (int e = 0; e < BLK / 2; ++e) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(kn + part * BLK)[e];
      kf[2 * e] = bf16lo(w);
      kf[2 * e + 1] = bf16hi(w);
    }
#pragma unroll
    for (int pass = 0; pass < (R + 31) / 32; ++pass) {
      const int j = threadIdx.x / 8 + pass * 32;
      float a = 0.f;
      if (j < R) {
        const float4* Mj = reinterpret_cast<const float4*>(p.M + ((size_t)h * R + j) * D + part * BLK);
#pragma unroll
        for (int e = 0; e < BLK / 4; ++e) {
          const float4 m = Mj[e];
          a = fmaf(m.x, kf[4 * e + 0], a);
          a = fmaf(m.y, kf[4 * e + 1], a);
          a = fmaf(m.z, kf[4 * e + 2], a);
          a = fmaf(m.w, kf[4 * e + 3], a);
        }
      }
      a += __shfl_xor_sync(0xffffffffu, a, 1);
      a += __shfl_xor_sync(0xffffffffu, a, 2);
      a += __shfl_xor_sync(0xffffffffu, a, 4);
      out[pass] = a;
    }
  }
  const bool ordered = starts_in_order<256>(p.q_start, p.B);
  if (!ordered) {
    if (threadIdx.x == 0) row_s = token_row(p, false, t, h);
    __syncthreads();
  }
  if (blockIdx.x == 0) record_skipped<256>(p, ordered);
  const long long row = row_s;
  if (row < 0) {
    if (threadIdx.x == 0) record_row(p, row);
    return;
  }
  if (threadIdx.x < 2 * PPR)
    *reinterpret_cast<uint4*>((threadIdx.x < PPR ? p.K : p.V) + (size_t)row * D + (threadIdx.x % PPR) * 8) = piece;
  if (p.Kproj != nullptr && part == 0) {
#pragma unroll
    for (int pass = 0; pass < (R + 31) / 32; ++pass) {
      const int j = threadIdx.x / 8 + pass * 32;
      if (j < R) {
        if constexpr (FP8)
          static_cast<unsigned char*>(p.Kproj)[(size_t)row * R + j] = fp8_of(out[pass], p.kproj_scale[h]);
        else
          static_cast<__nv_bfloat16*>(p.Kproj)[(size_t)row * R + j] = __float2bfloat16_rn(out[pass]);
      }
    }
  }
}

constexpr int kTileTokens = 128;
constexpr int kTileThreads = 256;
// Up to so many (token, head) pairs an SM a CTA each; beyond it tiles, whose first round takes the same
// time whatever share of the SMs it fills.  8 heads, d = 128, r = 32: 140 tokens 5.3 us in pairs and 9.0
// in tiles, 256 tokens (13.8 pairs an SM) 8.8 and 9.2, 320 tokens 10.0 and 9.2, 512 14.1 and 9.2; the
// same crossing with r = 64 (256 tokens 13.5 and 13.9, 320 15.6 and 13.7), with d = 64 and r = 16 (4.7
// and 4.7, 5.5 and 4.7) and with one head (2000 tokens 8.4 and 9.2, 2300 9.2 and 9.2).
constexpr long long kPairsPerSm = 14;

template <int D, int R>
struct TileSmem {
  static constexpr int KPITCH = D * 2 + 16;  // bytes: neighbouring rows start 4 banks apart
  float Mt[D][R];                            // M[h] transposed
  unsigned char K[2][kTileTokens][KPITCH];
  long long row[2][kTileTokens];
};

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <int D, int R, bool FP8>
__global__ void __launch_bounds__(kTileThreads, 2) tile_kernel(const AppendParams p) {
  using SM = TileSmem<D, R>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SM& S = *reinterpret_cast<SM*>(smem_raw);
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y;
  const int tiles = (p.n_new + kTileTokens - 1) / kTileTokens;
  constexpr int PPR = D / 8, PER = kTileTokens * PPR / kTileThreads;
  // A tile's keys are asked for, and its cache rows looked up, while the tile before is worked on.
  auto ask_keys = [&](int tile, int buf) {
    const int t0 = tile * kTileTokens, nt = min(kTileTokens, p.n_new - t0);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + i * kTileThreads, t = e / PPR, c = e % PPR;
      if (t < nt) copy_async16(&S.K[buf][t][c * 16], p.K_new + (size_t)(t0 + t) * p.kv_stride + (size_t)h * D + c * 8);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto look_up = [&](int tile, int buf, bool ordered) {
    const int t = tile * kTileTokens + tid;
    if (tid >= kTileTokens) return;
    const long long row = t < p.n_new ? token_row(p, ordered, t, h) : -1;
    record_row(p, row);
    S.row[buf][tid] = row;
  };
  ask_keys(blockIdx.x, 0);
  if (p.Kproj != nullptr) {
    // M[h] is [R][D]: a thread moves 4 channels of one output (outputs vary fastest over the
    // lanes, so that the transposed stores of a warp fall into different banks)
#pragma unroll 4
    for (int e = tid; e < R * D / 4; e += kTileThreads) {
      const int j = e % R, c = (e / R) * 4;
      const float4 m = __ldg(reinterpret_cast<const float4*>(p.M + ((size_t)h * R + j) * D + c));
      S.Mt[c][j] = m.x;
      S.Mt[c + 1][j] = m.y;
      S.Mt[c + 2][j] = m.z;
      S.Mt[c + 3][j] = m.w;
    }
  }
  const bool ordered = starts_in_order<kTileThreads>(p.q_start, p.B);
  look_up(blockIdx.x, 0, ordered);
  if (blockIdx.x == 0 && h == 0) record_skipped<kTileThreads>(p, ordered);
  int buf = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int t0 = tile * kTileTokens, nt = min(kTileTokens, p.n_new - t0);
    uint4 vr[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + i * kTileThreads, t = e / PPR, c = e % PPR;
      if (t < nt) vr[i] = ldg_stream128(p.V_new + (size_t)(t0 + t) * p.kv_stride + (size_t)h * D + c * 8);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (tile + (int)gridDim.x < tiles) {
      ask_keys(tile + gridDim.x, buf ^ 1);
      look_up(tile + gridDim.x, buf ^ 1, ordered);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + i * kTileThreads, t = e / PPR, c = e % PPR;
      const long long to = S.row[buf][t];
      if (to >= 0) {
        *reinterpret_cast<uint4*>(p.K + (size_t)to * D + c * 8) = *reinterpret_cast<const uint4*>(&S.K[buf][t][c * 16]);
        *reinterpret_cast<uint4*>(p.V + (size_t)to * D + c * 8) = vr[i];
      }
    }
    if (p.Kproj != nullptr) {
      // A lane takes tokens lane, lane + 32, + 64, + 96, a warp OUT outputs at a time: one load of M
      // (the same for the warp) feeds 4 tokens, one 16-byte load of a row 8 channels.
      constexpr int BLK = D / 8, OUT = R == 16 ? 2 : 4, P2 = OUT / 2, TK = 4;
#pragma unroll 1
      for (int j0 = warp * OUT; j0 < R; j0 += kTileThreads / 32 * OUT) {
        asm volatile("" ::: "memory");  // the keys are read again for the next outputs, not kept
        float2 tot[TK][P2], hold[TK][P2], hold2[TK][P2];  // the running combination of the 8 partial sums
#pragma unroll
        for (int blk = 0; blk < 8; ++blk) {
          float2 a[TK][P2];
#pragma unroll
          for (int x = 0; x < TK; ++x)
#pragma unroll
            for (int i = 0; i < P2; ++i) a[x][i] = make_float2(0.f, 0.f);
#pragma unroll
          for (int c8 = 0; c8 < BLK / 8; ++c8) {
            const int c0 = blk * BLK + c8 * 8;
            uint32_t k[TK][4];
#pragma unroll
            for (int x = 0; x < TK; ++x)
              *reinterpret_cast<uint4*>(k[x]) = *reinterpret_cast<const uint4*>(&S.K[buf][lane + 32 * x][c0 * 2]);
#pragma unroll
            for (int o = 0; o < 8; ++o) {
              float2 mm[P2];
              if constexpr (OUT == 4) *reinterpret_cast<float4*>(mm) = *reinterpret_cast<const float4*>(&S.Mt[c0 + o][j0]);
              else mm[0] = *reinterpret_cast<const float2*>(&S.Mt[c0 + o][j0]);
#pragma unroll
              for (int x = 0; x < TK; ++x) {
                const float f = o & 1 ? bf16hi(k[x][o / 2]) : bf16lo(k[x][o / 2]);
#pragma unroll
                for (int i = 0; i < P2; ++i) a[x][i] = ffma2(mm[i], make_float2(f, f), a[x][i]);
              }
            }
          }
          // ((p0+p1)+(p2+p3)) + ((p4+p5)+(p6+p7)), as the partial sums arrive
#pragma unroll
          for (int x = 0; x < TK; ++x)
#pragma unroll
            for (int i = 0; i < P2; ++i) {
              const float2 v = a[x][i];
              if (blk % 2 == 0) {
                hold[x][i] = v;
              } else {
                const float2 pr = make_float2(hold[x][i].x + v.x, hold[x][i].y + v.y);
                if (blk % 4 == 1) {
                  hold2[x][i] = pr;
                } else {
                  const float2 q = make_float2(hold2[x][i].x + pr.x, hold2[x][i].y + pr.y);
                  if (blk == 3) tot[x][i] = q;
                  else tot[x][i] = make_float2(tot[x][i].x + q.x, tot[x][i].y + q.y);
                }
              }
            }
        }
#pragma unroll
        for (int x = 0; x < TK; ++x) {
          const long long row = S.row[buf][lane + 32 * x];
          if (row < 0) continue;
          const size_t at = (size_t)row * R + j0;
          if constexpr (FP8) {
            const float s = p.kproj_scale[h];
            unsigned char* dst = static_cast<unsigned char*>(p.Kproj) + at;
            const uint32_t lo = (uint32_t)fp8_of(tot[x][0].x, s) | ((uint32_t)fp8_of(tot[x][0].y, s) << 8);
            if constexpr (OUT == 4)
              *reinterpret_cast<uint32_t*>(dst) =
                  lo | ((uint32_t)fp8_of(tot[x][P2 - 1].x, s) << 16) | ((uint32_t)fp8_of(tot[x][P2 - 1].y, s) << 24);
            else *reinterpret_cast<unsigned short*>(dst) = (unsigned short)lo;
          } else {
            __align__(8) __nv_bfloat162 w[P2];
#pragma unroll
            for (int i = 0; i < P2; ++i) w[i] = __floats2bfloat162_rn(tot[x][i].x, tot[x][i].y);
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.Kproj) + at;
            if constexpr (OUT == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(w);
            else *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(w);
          }
        }
      }
    }
    __syncthreads();  // this buffer's keys and rows have been used before they are asked for again
  }
}

template <int D, int R, bool FP8>
cudaError_t launch_drf(const AppendParams& p, int sms, cudaStream_t stream) {
  const long long pairs = (long long)p.n_new * p.Hkv;
  if (pairs <= kPairsPerSm * sms)
    return launch_pdl(token_kernel<D, R, FP8>, dim3((unsigned)pairs), dim3(256), 0, stream, p);
  auto kern = tile_kernel<D, R, FP8>;
  const int smem = (int)sizeof(TileSmem<D, R>);
  const cudaError_t e = prepare_kernel((const void*)kern, smem);
  if (e != cudaSuccess) return e;
  // As many CTAs as are resident at once share the tiles of all heads.
  const int tiles = (p.n_new + kTileTokens - 1) / kTileTokens;
  const int per_head = (sms * ctas_per_sm((const void*)kern, kTileThreads, smem) + p.Hkv - 1) / p.Hkv;
  return launch_pdl(kern, dim3((unsigned)(tiles < per_head ? tiles : per_head), (unsigned)p.Hkv), dim3(kTileThreads), (size_t)smem,
                    stream, p);
}

template <int D>
cudaError_t launch_d(const AppendParams& p, int sms, cudaStream_t stream) {
  switch (p.r) {
    case 16: return p.fp8 ? launch_drf<D, 16, true>(p, sms, stream) : launch_drf<D, 16, false>(p, sms, stream);
    case 32: return p.fp8 ? launch_drf<D, 32, true>(p, sms, stream) : launch_drf<D, 32, false>(p, sms, stream);
    case 64: return p.fp8 ? launch_drf<D, 64, true>(p, sms, stream) : launch_drf<D, 64, false>(p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_append_chunk(const AppendParams& p, int sms, cudaStream_t stream) {
  if (p.d == 128) return launch_d<128>(p, sms, stream);
  if (p.d == 64) return launch_d<64>(p, sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace sas
