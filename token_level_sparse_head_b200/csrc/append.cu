// Rows of a chunk of new tokens into the caches: K, V and the projected rows (sm_100a).
//
// Token t of the batch belongs to the sequence b with q_start[b] <= t < q_start[b+1] and sits at
// position N_b - T_b + (t - q_start[b]).  Per token and KV head the call copies 2 d bf16 values and
// computes r dot products of length d in fp32, in the summation order of the projection build (8
// partial sums over consecutive blocks of d/8 channels, in channel order, combined as
// ((p0+p1)+(p2+p3))+((p4+p5)+(p6+p7))), so a row is the same bits whichever call wrote it.
//
// Two kernels, by the number of (token, head) pairs:
//   token_kernel  one CTA per pair, 8 threads per output: few tokens, where latency counts;
//   tile_kernel   CTA = 64 tokens x one head.  K rows and M[h] are staged in shared memory, M
//                 transposed to [channel][output] so that a thread takes 8 outputs of 2 tokens
//                 with two 16-byte loads of M per channel, in paired fp32 FMAs (bit-identical to
//                 single ones).
#include <cuda_fp8.h>

#include "sas_device.cuh"
#include "sas_kernels.h"

namespace sas {
namespace {

// Sequence and cache row of token t; row < 0 if the token belongs to nobody or a check failed.
__device__ __forceinline__ long long token_row(const AppendParams& p, int t, int h) {
  int lo = 0, hi = p.B;  // largest b in [0, B) with q_start[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_start[mid] <= t) lo = mid; else hi = mid;
  }
  const int b = lo, s0 = p.q_start[b], s1 = p.q_start[b + 1];
  if (t < s0 || t >= s1) return -1;
  const int n = p.seqlens[b];
  if (n < 0 || n > p.cap) {
    record_error(p.err, kDevBadSeqlen, (uint32_t)b);
    return -1;
  }
  if (s0 < 0 || s1 > p.n_new || s1 - s0 > n) {
    record_error(p.err, kDevBadChunk, (uint32_t)b);
    return -1;
  }
  const int pos = n - (s1 - s0) + (t - s0);
  if (!p.paged) return ((long long)b * p.Hkv + h) * p.cap + pos;
  const int pg = p.page_table[(size_t)b * p.max_pages + (pos >> 6)];
  if (pg < 0 || pg >= p.num_pages) {
    record_error(p.err, kDevBadPage, (uint32_t)b);
    return -1;
  }
  return ((long long)pg * p.Hkv + h) * 64 + (pos & 63);
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
  if (threadIdx.x == 0) row_s = token_row(p, t, h);
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
  __syncthreads();
  const long long row = row_s;
  if (row < 0) return;
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

constexpr int kTileTokens = 64;
constexpr int kTileThreads = 128;

template <int D, int R>
struct TileSmem {
  static constexpr int KPITCH = D * 2 + 16;  // bytes: rows of a pair of tokens start in other banks
  float Mt[D][R];                            // M[h] transposed
  unsigned char K[kTileTokens][KPITCH];
  long long row[kTileTokens];
};

template <int D, int R, bool FP8>
__global__ void __launch_bounds__(kTileThreads) tile_kernel(const AppendParams p) {
  using SM = TileSmem<D, R>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SM& S = *reinterpret_cast<SM*>(smem_raw);
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int h = blockIdx.y;
  const int t0 = blockIdx.x * kTileTokens;
  const int nt = min(kTileTokens, p.n_new - t0);
  if (tid < kTileTokens) S.row[tid] = tid < nt ? token_row(p, t0 + tid, h) : -1;
  if (p.Kproj != nullptr) {
    // M[h] is [R][D]: a thread moves 4 channels of one output (outputs vary fastest over the
    // lanes, so that the transposed stores of a warp fall into different banks)
    for (int e = tid; e < R * D / 4; e += kTileThreads) {
      const int j = e % R, c = (e / R) * 4;
      const float4 m = *reinterpret_cast<const float4*>(p.M + ((size_t)h * R + j) * D + c);
      S.Mt[c][j] = m.x;
      S.Mt[c + 1][j] = m.y;
      S.Mt[c + 2][j] = m.z;
      S.Mt[c + 3][j] = m.w;
    }
  }
  constexpr int PPR = D / 8;
  for (int e = tid; e < nt * PPR; e += kTileThreads) {
    const int t = e / PPR, c = e % PPR;
    *reinterpret_cast<uint4*>(&S.K[t][c * 16]) =
        ldg_stream128(p.K_new + (size_t)(t0 + t) * p.kv_stride + (size_t)h * D + c * 8);
  }
  __syncthreads();
  for (int e = tid; e < nt * PPR; e += kTileThreads) {
    const int t = e / PPR, c = e % PPR;
    const uint4 v = ldg_stream128(p.V_new + (size_t)(t0 + t) * p.kv_stride + (size_t)h * D + c * 8);
    const long long row = S.row[t];
    if (row >= 0) {
      *reinterpret_cast<uint4*>(p.K + (size_t)row * D + c * 8) = *reinterpret_cast<const uint4*>(&S.K[t][c * 16]);
      *reinterpret_cast<uint4*>(p.V + (size_t)row * D + c * 8) = v;
    }
  }
  if (p.Kproj == nullptr) return;

  // Unit u: outputs 8 * (u / 32) .. + 7 of tokens u % 32 and u % 32 + 32.
  constexpr int BLK = D / 8;
  for (int u = tid; u < (kTileTokens / 2) * (R / 8); u += kTileThreads) {
    const int ta = u % 32, tb = ta + 32, j0 = (u / 32) * 8;
    if (ta >= nt) continue;
    float2 tot[2][4];  // p0+p1, then the running combination
    float2 hold[2][4], hold2[2][4];
#pragma unroll
    for (int blk = 0; blk < 8; ++blk) {
      float2 a[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) a[x][i] = make_float2(0.f, 0.f);
#pragma unroll
      for (int c2 = 0; c2 < BLK / 2; ++c2) {
        const int c = blk * BLK + c2 * 2;
        const uint32_t ka = *reinterpret_cast<const uint32_t*>(&S.K[ta][c * 2]);
        const uint32_t kb = *reinterpret_cast<const uint32_t*>(&S.K[tb][c * 2]);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const float4 m0 = *reinterpret_cast<const float4*>(&S.Mt[c + o][j0]);
          const float4 m1 = *reinterpret_cast<const float4*>(&S.Mt[c + o][j0 + 4]);
          const float fa = o ? bf16hi(ka) : bf16lo(ka), fb = o ? bf16hi(kb) : bf16lo(kb);
          const float2 xa = make_float2(fa, fa), xb = make_float2(fb, fb);
          const float2 mm[4] = {make_float2(m0.x, m0.y), make_float2(m0.z, m0.w), make_float2(m1.x, m1.y),
                                make_float2(m1.z, m1.w)};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[0][i] = ffma2(mm[i], xa, a[0][i]);
            a[1][i] = ffma2(mm[i], xb, a[1][i]);
          }
        }
      }
      // ((p0+p1)+(p2+p3)) + ((p4+p5)+(p6+p7)), as the partial sums arrive
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
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
    for (int x = 0; x < 2; ++x) {
      const int t = x ? tb : ta;
      const long long row = t < nt ? S.row[t] : -1;
      if (row < 0) continue;
      if constexpr (FP8) {
        const float s = p.kproj_scale[h];
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w[i] = (uint32_t)fp8_of(tot[x][2 * i].x, s) | ((uint32_t)fp8_of(tot[x][2 * i].y, s) << 8) |
                 ((uint32_t)fp8_of(tot[x][2 * i + 1].x, s) << 16) | ((uint32_t)fp8_of(tot[x][2 * i + 1].y, s) << 24);
        *reinterpret_cast<uint2*>(static_cast<unsigned char*>(p.Kproj) + (size_t)row * R + j0) = make_uint2(w[0], w[1]);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 pr = __floats2bfloat162_rn(tot[x][i].x, tot[x][i].y);
          w[i] = *reinterpret_cast<const uint32_t*>(&pr);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.Kproj) + (size_t)row * R + j0) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

template <int D, int R, bool FP8>
cudaError_t launch_drf(const AppendParams& p, int sms, cudaStream_t stream) {
  const long long pairs = (long long)p.n_new * p.Hkv;
  if (pairs <= 8LL * sms)
    return launch_pdl(token_kernel<D, R, FP8>, dim3((unsigned)pairs), dim3(256), 0, stream, p);
  auto kern = tile_kernel<D, R, FP8>;
  const int smem = (int)sizeof(TileSmem<D, R>);
  const cudaError_t e = prepare_kernel((const void*)kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)((p.n_new + kTileTokens - 1) / kTileTokens), (unsigned)p.Hkv),
                    dim3(kTileThreads), (size_t)smem, stream, p);
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
