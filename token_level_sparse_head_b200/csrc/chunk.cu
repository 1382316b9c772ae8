// Causal attention of a chunk of new tokens over the cache, with a sliding window and sinks (sm_100a).
//
//   out[t] = sum_j softmax_j(sigma q_t . K_j) V_j over the j visible to token t.
//
// Rows: the G query heads of a KV head read the same K and V, so a 128-row tile holds 128 / G
// tokens times G heads.  A task is up to two tiles of one sequence; its keys are a list of 64-row
// pages (the sinks' pages, then those from the window of its first token to its last token).
// Work: units of all tasks and KV heads, one after another, cut into equal contiguous shares, one
// per CTA, so that ragged batches, causal triangles and few long sequences load every SM alike.
//   two tiles  a unit is one block of 128 keys, read once for both tiles;
//   one tile   a unit is two blocks; each warpgroup takes one, with its own statistics and output
//              (drafted tokens and short chunks: the cache is read at twice the rate per step).
// A share that holds part of a task leaves a partial (m, l, O); join_kernel puts those together in order.
//
// The KV heads are gone through in waves whose K and V stay in L2 (struct Wave).
//
// CTA: two softmax warpgroups (a thread is a row), one warp that issues the matrix instructions,
// one warp that loads.  S = Q K^T goes to tensor memory; the softmax threads read their row and
// write P in bf16 back to tensor memory, where P V takes its left operand from, so P never passes
// through shared memory.  Tensor memory (512 columns) holds P and O of both tiles and, with
// d = 128, one S that the tiles use in turn: it is free again as soon as its rows have been read,
// and the next tile's S is made while this one is exponentiated.  O is rescaled only when a row's
// maximum has grown by 2^8 since the last time (P <= 2^8 keeps bf16's relative rounding and fp32's
// range), which after the first blocks is rare.  Sums and maxima are fp32; P is rounded to bf16,
// which the matrix instructions take, and that rounding (2^-8 of a weight) bounds the error.
// K and V blocks of 128 keys pass through one ring of tiled bulk copies (128-byte swizzle).
//
// What bounds it, for two-tile units with d = 128: a unit is 2048 cycles of matrix instructions and
// takes about 2940.  No unit of the SM is full: matrix pipe 69 %, special functions 70 %, shared memory
// about 2040 of the 2940 cycles (1527 wavefronts of operands, 512 of copies); the tiles share one S and
// take turns, and with the softmax left out a unit still took 2800.  Measured: prompt of 8192 (32 heads,
// 8 KV heads) 562 us, 980 TFLOP/s; 512 tokens on 32K rows 262 to 266 us, 1030 TFLOP/s, both at the 1.1-1.3
// GHz that the power limit leaves; 8 x 5 tokens on 4K to 32K rows 112 to 117 us, 5.2 TB/s.  With d = 64
// the loop over blocks (3100 cycles) and the ends of tasks (4000 each) bound it.
// Tried and not kept: a warp for each of the two products (384K cycles against 345K for 512 on
// 32K); polynomial exponentials on the FMA pipe for part of the row (286 us without, 288 to 316 us
// with); P in the place of S (a tile's products then wait for its softmax).
#include "sas_device.cuh"
#include "sas_kernels.h"

namespace sas {
namespace {

constexpr int kPage = 64;
constexpr int kThreads = 384;      // 8 softmax warps, 1 matrix warp, 1 load warp, 2 idle: three warpgroups
constexpr int kPlanThreads = 1024;
// Up to so many task slots every CTA makes the list itself, which saves a kernel (64 tokens of 64
// sequences of 1K rows: 106 us, with the kernel 112; of 250 sequences, 500 slots, 375 and 381).  More
// would gain 1 % (1125 slots: 899 and 910 us) for 40 bytes a slot and CTA of workspace.
constexpr int kOwnPlanSlots = 256;
constexpr int kTile = 128;
constexpr int kRowsCap = 2 * kTile;  // rows of a partial
// K and V bytes of a wave: more do not stay in the 126 MB of L2, fewer bytes are more waves, each of
// which leaves partials.  Under steady load, where HBM traffic costs clock (32 heads, 8 KV heads): 512
// tokens on 32K rows (128 MB) in one wave 298 us, in two 266; 1024 on 64K in waves of 64 MB 951, of
// 86 MB 989; with d = 64 512 on 64K in waves of 32 MB 377, of 64 MB 370, in one 390.  (A call by itself,
// at full clock, is faster in one wave: 512 on 32K 240 and 250 us.)
constexpr long long kLiveBytes = 72LL << 20;
// Units of a CTA and wave that a partial per wave is worth.  At 24 to 47 units two waves lose: 256 tokens
// on 32K rows 168 us, in one wave 156; 384 on 32K 220 and 204; 128 on 64K 199 and 164.  At 48 to 99 they
// gain: 512 on 32K 275 and 298 (one), 256 on 64K 298 and 312, 512 on 64K in three 540, in two 568.
constexpr int kWaveUnits = 48;

// The matrix instruction truncates its sums, always towards zero (about 2^-23 of the running output
// a step: 262144 rows in one go came out 1.0e-3 low on average, as much as a quarter of bf16's step),
// so an output is summed in tensor memory over this many units at most and then added, with rounding,
// to a sum in the CTA's partial.  4096 tokens on 128K rows take 7.3 ms without, 7.6 with 128 or 256.
constexpr int kFoldUnits = 128;
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct Geo {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF_BYTES = kTile * 128;           // 128 rows of 64 columns
  static constexpr int TILE_BYTES = HALVES * HALF_BYTES;   // Q tile, K block or V block
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr int Q_BUFS = D == 128 ? 1 : 2;          // tasks whose Q is held: the next one's comes ahead
  static constexpr int SMEM = 1024 + (2 * Q_BUFS + STAGES) * TILE_BYTES;
  // Tensor memory, 512 columns: P of the tiles (64 each), S, O of the tiles.  At d = 128 the tiles
  // share one S; at d = 64 there is room for two.
  static constexpr int S_BUFS = D == 128 ? 1 : 2;
  static constexpr int COL_P = 0, COL_S = 128, COL_O = 512 - 2 * D;
  static_assert(COL_S + S_BUFS * kTile <= COL_O, "tensor memory");
};

// ----------------------------------------------------------------------------- tensor memory
__device__ __forceinline__ void tmem_ld32(float* r, uint32_t addr) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(u[0]),
      "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]),
      "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(float* r, uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]) : "r"(addr));
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const float* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(r[0]), "f"(r[1]), "f"(r[2]),
               "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// The matrix warp runs as a whole, so that descriptors are computed once per warp, and its `lead`
// lane issues: a branch around the instructions would move each operand over by itself.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// All matrix instructions the lead lane has issued so far arrive on `bar` when they are done.
__device__ __forceinline__ void tc_commit(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(lead)
      : "memory");
}

// Shared-memory operand of 128-byte swizzled rows.  `lead` is the distance between 64-column
// parts of a row-contiguous (MN-major) operand; consecutive groups of 8 rows lie 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// bf16 x bf16 -> fp32, 128 rows, n columns; b_rows: B is stored [k][n].
constexpr uint32_t mma_form(int n, bool b_rows) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_rows ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t form, bool add, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(form), "r"((uint32_t)add), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t form, bool add, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(form), "r"((uint32_t)add), "r"(lead)
      : "memory");
}

// ----------------------------------------------------------------------------- waits
// Waits for a phase; gives up when another warp has or after the library's limit.  Each lane waits
// for itself: a vote after every wait costs as much as the wait.
__device__ __forceinline__ bool wait_live(uint64_t* bar, uint32_t parity, volatile int* stop) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 15u) == 15u && *stop) return false;
  }
  *stop = 1;
  return false;
}
__device__ __forceinline__ void wait_row(uint64_t* bar, uint32_t parity, volatile int* stop) {
  wait_live(bar, parity, stop);
  __syncwarp();
}
// The matrix warp's: the same answer for all lanes.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* stop) {
  return __all_sync(0xffffffffu, wait_live(bar, parity, stop));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The softmax threads hold a row of 128 scores; the launch's 384 x 168 registers are dealt out
// again as 2 x 128 x 208 + 128 x 88.
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 208;"); }
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 88;"); }
// Bits 0 .. x-1 of a 64-row page.
__device__ __forceinline__ uint64_t low_bits(int x) { return x <= 0 ? 0ull : (x >= 64 ? ~0ull : (1ull << x) - 1); }

// ----------------------------------------------------------------------------- plan
template <int THREADS, typename T>
__device__ __forceinline__ T block_scan(T x, T* warp_sum, T& total) {  // inclusive
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  T before = 0;
  total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  __syncthreads();
  return x + before;
}

template <int THREADS>
struct PlanSmem {
  unsigned long long keys;  // rows that the chunks see, one KV head
  long long lsum[THREADS / 32];
  int sum[THREADS / 32], off[THREADS + 1];
};
// Tasks of every sequence, and the units before each: tasks[slots] holds their number and total.
// A whole CTA; its other threads see the tasks after a barrier.
template <int THREADS>
__device__ __forceinline__ void make_plan(const ChunkParams& p, ChunkTask* tasks, PlanSmem<THREADS>& S) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int span = 2 * p.tok_tile;
  int base = 0;
  if (tid == 0) S.keys = 0;
  const bool ordered = starts_in_order<THREADS>(p.q_start, p.B);
  LargestStart largest;
  for (int b0 = 0; b0 < p.B; b0 += THREADS) {
    const int b = b0 + tid;
    int cnt = 0;
    if (b < p.B) {
      const int s0 = p.q_start[b], s1 = p.q_start[b + 1];
      const uint32_t why = chunk_error(s0, s1, ordered ? s0 : largest.upto(p.q_start, b), p.seqlens[b], p.n_new, p.cap);
      if (why != kDevOk) record_error(p.err, why, (uint32_t)b);
      else cnt = (s1 - s0 + span - 1) / span;
    }
    int total;
    const int end = block_scan<THREADS>(cnt, S.sum, total);
    if (tid == 0) S.off[0] = 0;
    S.off[tid + 1] = end;  // sequences that are taken do not overlap, so their tasks fit the slots
    __syncthreads();
    for (int i = warp; i < min(THREADS, p.B - b0); i += THREADS / 32) {
      const int k0 = S.off[i], k1 = S.off[i + 1];
      if (k0 >= k1) continue;
      const int s0 = p.q_start[b0 + i], T = p.q_start[b0 + i + 1] - s0, n = p.seqlens[b0 + i];
      if (lane == 0) atomicAdd(&S.keys, (unsigned long long)visible_pages(n - T, n - 1, p.window, p.sinks).nv * kPage);
      for (int k = k0 + lane; k < k1; k += 32) {
        const int at = (k - k0) * span;
        ChunkTask t;
        t.b = b0 + i;
        t.tok0 = s0 + at;
        t.ntok = min(span, T - at);
        t.pos0 = n - T + at;
        t.unit0 = 0;
        const int nv = visible_pages(t.pos0, t.pos0 + t.ntok - 1, p.window, p.sinks).nv;
        t.blocks = t.ntok > p.tok_tile ? (nv + 1) >> 1 : (nv + 3) >> 2;
        t.seqlen = n;
        tasks[base + k] = t;
      }
    }
    __syncthreads();
    base += total;
  }
  long long units = 0;
  for (int k0 = 0; k0 < base; k0 += THREADS) {
    const int k = k0 + tid;
    const long long x = k < base ? tasks[k].blocks : 0;
    long long total;
    const long long end = block_scan<THREADS>(x, S.lsum, total);
    if (k < base) tasks[k].unit0 = units + end - x;
    units += total;
  }
  if (tid == 0) {
    ChunkTask t = {};
    t.b = base;
    // Waves of at most kLiveBytes of K and V, where the blocks are read more than once and a
    // CTA's share of a wave stays long against the cost of a partial.
    const long long once = (long long)S.keys * p.d * 4 * p.Hkv, block = (long long)kTile * p.d * 4;
    int waves = 1;
    if (units * p.Hkv * block > once + once / 2)
      while (waves < p.waves_max && once > waves * kLiveBytes && units * p.Hkv > (long long)(waves + 1) * p.ctas * kWaveUnits) ++waves;
    t.tok0 = waves;
    t.unit0 = units;
    tasks[p.slots] = t;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ PlanSmem<kPlanThreads> S;
  pdl_wait();
  pdl_trigger();
  make_plan<kPlanThreads>(p, p.tasks, S);
}

// ----------------------------------------------------------------------------- shares
struct Place {
  int task, h, block;
};
// The KV heads are gone through in waves, so that the K and V that several tasks read stay in L2
// meanwhile.  A CTA's share of a wave: units u0 .. u1 - 1 of it, the first of them at `at`.
struct Share {
  long long u0, u1;
  Place at;
};
struct Wave {
  long long total, share;
  int head0;
};
__device__ __forceinline__ Wave wave_of(const ChunkParams& p, int w, int waves, long long units) {
  Wave x;
  x.head0 = w * p.Hkv / waves;
  x.total = units * ((w + 1) * p.Hkv / waves - x.head0);
  x.share = (x.total + p.ctas - 1) / p.ctas;
  return x;
}
// Task, KV head and unit of the task at global unit u; whole warp.
__device__ __forceinline__ Place find_unit(const ChunkTask* list, long long u, int tasks, long long units) {
  const int lane = threadIdx.x & 31;
  Place c;
  c.h = (int)(u / units);
  const long long rem = u - c.h * units;
  int lo = 0, cnt = tasks;
  while (cnt > 1) {
    const int step = (cnt + 31) / 32;
    const bool in = lane * step < cnt && list[lo + lane * step].unit0 <= rem;
    const int k = __popc(__ballot_sync(0xffffffffu, in)) - 1;
    lo += k * step;
    cnt = min(step, cnt - k * step);
  }
  c.task = lo;
  c.block = (int)(rem - list[lo].unit0);
  return c;
}
__device__ __forceinline__ void next_task(Place& c, int tasks) {
  c.block = 0;
  if (++c.task == tasks) {
    c.task = 0;
    ++c.h;
  }
}

// A place in the ring and the parity of its turn; blocks lie in it in the order of use.  Two tiles:
// K0, then K(j+1) V(j) for unit j; one tile: both warpgroups' K0, then for unit j and each
// warpgroup K(j+1) V(j).
struct Ring {
  int st;
  uint32_t ph;
  template <int ST>
  __device__ __forceinline__ Ring take() {
    const Ring x = *this;
    if (++st == ST) {
      st = 0;
      ph ^= 1;
    }
    return x;
  }
};
// Position of V of unit j among the blocks of a segment of n units.
__device__ __forceinline__ int ring_v(bool one, int j, int x, int n) {
  return one ? (j + 1 < n ? 4 * j + 3 + 2 * x : 4 * j + 2 + x) : (j + 1 < n ? 2 * j + 2 : 2 * j + 1);
}

// What a softmax warpgroup knows of a segment.  Made anew where it is needed, from the list that a
// shared variable points to: kept over the loop on the blocks it would push the scores out of registers.
struct GroupSeg {
  ChunkTask t;
  VisiblePages vis;
  bool one;
  int tile, toks, plo, phi, block;
  __device__ __forceinline__ GroupSeg(const ChunkParams& p, const ChunkTask* const volatile& list, const Place& c, int x) {
    t = list[c.task];
    one = t.ntok <= p.tok_tile;
    vis = visible_pages(t.pos0, t.pos0 + t.ntok - 1, p.window, p.sinks);
    tile = one ? 0 : x;
    toks = min(p.tok_tile, t.ntok - tile * p.tok_tile);
    plo = t.pos0 + tile * p.tok_tile;
    phi = plo + toks - 1;
    block = c.block;
  }
  // Blocks a .. b - 1 of the segment lie inside the window of every row, whole: pages from pg0 to
  // pg1 - 1 of the sequence, behind the sinks' pages of the list.
  __device__ __forceinline__ void plain(const ChunkParams& p, int x, int& a, int& b) const {
    const int pg0 = max(vis.w0, p.window > 0 ? (max(0, phi - p.window + 1) + kPage - 1) / kPage : 0);
    const int pg1 = (plo + 1) / kPage;
    const int a0 = pg0 - vis.w0 + vis.ns, a1 = pg1 - vis.w0 + vis.ns;  // in the list
    if (one) {
      a = ((a0 - 2 * x + 3) >> 2) - block;
      b = ((a1 - 2 * x + 2) >> 2) - block;
    } else {
      a = ((a0 + 1) >> 1) - block;
      b = (a1 >> 1) - block;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
  using Gm = Geo<D>;
  constexpr int ST = Gm::STAGES;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* qs = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* ring = qs + 2 * Gm::Q_BUFS * Gm::TILE_BYTES;
  __shared__ uint64_t full[ST], empty[ST], q_full[Gm::Q_BUFS], q_empty[Gm::Q_BUFS];
  __shared__ uint64_t s_full[2], s_read[2], p_ready[2], pv_done[2], half_full, half_free, drain;
  __shared__ uint32_t tmem_s;
  __shared__ volatile int stop_s;
  __shared__ const ChunkTask* volatile list_s;
  __shared__ Share share_s[kChunkMaxWaves];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < Gm::Q_BUFS; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_ready[t], 4);
      mbar_init(&s_read[t], 4);
      mbar_init(&pv_done[t], 1);
    }
    mbar_init(&half_full, 4);
    mbar_init(&half_free, 4);
    mbar_init(&drain, 1);
    fence_barrier_init();
    stop_s = 0;
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_s)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();
  // Few tasks: every CTA makes the list for itself, which costs less than a kernel before this one.
  const ChunkTask* list = p.tasks;
  if (p.own_plan) {
    ChunkTask* own = p.tasks + (size_t)blockIdx.x * (p.slots + 1);
    make_plan<kThreads>(p, own, *reinterpret_cast<PlanSmem<kThreads>*>(ring));
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the copies write there next
    __syncthreads();
    list = own;
  }
  if (tid == 0) list_s = list;
  const int tasks = list[p.slots].b;
  const long long units = list[p.slots].unit0;
  const int waves = list[p.slots].tok0;
  if (warp < waves) {
    const Wave w = wave_of(p, warp, waves, units);
    Share x;
    x.u0 = min(w.share * blockIdx.x, w.total);
    x.u1 = min(x.u0 + w.share, w.total);
    if (x.u0 < x.u1) x.at = find_unit(list, x.u0, tasks, units);
    x.at.h += w.head0;
    if (lane == 0) share_s[warp] = x;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_s;

  if (warp >= 8) regs_down();
  if (warp == 9) {
    // ---------------------------------------------------------------- loads
    int cnt = 0, seg = 0;  // blocks and Q tiles asked for
    bool live = true;
    for (int w = 0; w < waves; ++w) {
      Place c = share_s[w].at;
      const long long u1 = share_s[w].u1;
      for (long long u = share_s[w].u0; u < u1 && live;) {
        const ChunkTask t = list[c.task];
        const int be = (int)min((long long)t.blocks, c.block + (u1 - u)), units_here = be - c.block;
        const bool one = t.ntok <= p.tok_tile;
        const VisiblePages vis = visible_pages(t.pos0, t.pos0 + t.ntok - 1, p.window, p.sinks);
        // rows of 32 pages, page v with lane v % 32, looked up 16 at a time
        int row = 0, have = c.block * (one ? 4 : 2);
        auto push = [&](const CUtensorMap* map, int v) {
          while (v + 2 > have) {
            const int ahead = have + ((lane - have) & 31);
            if (ahead < have + 16) {
              row = p.row_end;
              const int lp = vis.page(ahead);
              if (ahead < vis.nv) {
                if (p.paged) {
                  const int pg = p.page_table[(size_t)t.b * p.max_pages + lp];
                  if (pg < 0 || pg >= p.num_pages) record_error(p.err, kDevBadPage, (uint32_t)t.b);
                  else row = (pg * p.Hkv + c.h) * kPage;
                } else {
                  row = (t.b * p.Hkv + c.h) * p.cap + lp * kPage;
                }
              }
            }
            have += 16;
          }
          const int y0 = __shfl_sync(0xffffffffu, row, v & 31), y1 = __shfl_sync(0xffffffffu, row, (v + 1) & 31);
          if (lane == 0 && live) {
            const int st = cnt % ST;
            live = cnt < ST || wait_live(&empty[st], ((cnt / ST) & 1) ^ 1, &stop_s);
            if (live) {
              unsigned char* dst = ring + (size_t)st * Gm::TILE_BYTES;
              mbar_arrive_expect_tx(&full[st], Gm::TILE_BYTES);
#pragma unroll
              for (int hf = 0; hf < Gm::HALVES; ++hf) {
                tma_2d(dst + hf * Gm::HALF_BYTES, map, hf * 64, y0, &full[st]);
                tma_2d(dst + hf * Gm::HALF_BYTES + kPage * 128, map, hf * 64, y1, &full[st]);
              }
            }
          }
          live = __shfl_sync(0xffffffffu, live, 0);
          if (live) ++cnt;
        };
        auto load_q = [&] {
          const int qb = seg % Gm::Q_BUFS;
          if (lane == 0 && live) {
            live = seg < Gm::Q_BUFS || wait_live(&q_empty[qb], ((seg / Gm::Q_BUFS) & 1) ^ 1, &stop_s);
            if (live) {
              const int box = p.G * p.tok_tile * 128;
              mbar_arrive_expect_tx(&q_full[qb], (one ? 1 : 2) * Gm::HALVES * box);
              for (int i = 0; i < (one ? 1 : 2); ++i)
#pragma unroll
                for (int hf = 0; hf < Gm::HALVES; ++hf)
                  tma_3d(qs + (2 * qb + i) * Gm::TILE_BYTES + hf * Gm::HALF_BYTES, &p.qmap, hf * 64, c.h * p.G,
                         t.tok0 + i * p.tok_tile, &q_full[qb]);
            }
          }
          live = __shfl_sync(0xffffffffu, live, 0);
          if (live) ++seg;
        };
        // the first keys do not wait for the room that Q waits for
        if (one) {
          push(&p.kmap, 4 * c.block);
          push(&p.kmap, 4 * c.block + 2);
          load_q();
          for (int j = c.block; j < be; ++j)
            for (int x = 0; x < 2; ++x) {
              if (j + 1 < be) push(&p.kmap, 4 * j + 4 + 2 * x);
              push(&p.vmap, 4 * j + 2 * x);
            }
        } else {
          push(&p.kmap, 2 * c.block);
          load_q();
          for (int j = c.block; j < be; ++j) {
            if (j + 1 < be) push(&p.kmap, 2 * j + 2);
            push(&p.vmap, 2 * j);
          }
        }
        u += units_here;
        next_task(c, tasks);
      }
    }
    // after a wait that ran out: the copies in flight land before the CTA ends
    if (lane == 0 && !live) {
      for (int i = max(0, seg - Gm::Q_BUFS); i < seg; ++i) mbar_wait_bounded(&q_full[i % Gm::Q_BUFS], (i / Gm::Q_BUFS) & 1);
      for (int i = max(0, cnt - ST); i < cnt; ++i) mbar_wait_bounded(&full[i % ST], (i / ST) & 1);
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------------- matrix instructions
    // The scores' buffer goes back and forth between this warp and the softmax: what does not
    // depend on a wait is done before it.
    const uint32_t lead = elect_lane();
    constexpr uint32_t kFormS = mma_form(kTile, false), kFormO = mma_form(D, true);
    const uint64_t qd = operand(smem_u32(qs), 16), kd = operand(smem_u32(ring), 16), vd = operand(smem_u32(ring), Gm::HALF_BYTES);
    constexpr uint32_t kStep = Gm::TILE_BYTES >> 4;
    int seg = 0;
    Ring r = {0, 0}, k = {0, 0}, v = {0, 0};
    uint32_t ph_p = 0, ph_read = 1;  // parity of the scores' reads: the first use of a buffer waits for none
    bool live = true;
    auto scores = [&](int x, bool one) {  // S = Q K^T for warpgroup x, K in ring place k
      const int buf = Gm::S_BUFS == 1 ? 0 : x;
      const uint64_t a = qd + (2 * (seg % Gm::Q_BUFS) + (one ? 0 : x)) * kStep, b = kd + k.st * kStep;
      live = live && wait_warp(&full[k.st], k.ph, &stop_s);
      live = live && wait_warp(&s_read[buf], ph_read, &stop_s);  // the scores that were there have been read
      if (Gm::S_BUFS == 1 || x == 1) ph_read ^= 1;
      if (!live) return;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        constexpr int kHalf = Gm::HALF_BYTES >> 4;
        const uint32_t o = (i >> 2) * kHalf + (i & 3) * 2;
        mma_ss(tmem + Gm::COL_S + buf * kTile, a + o, b + o, kFormS, i > 0, lead);
      }
      tc_commit(&s_full[x], lead);
      if (one || x == 1) tc_commit(&empty[k.st], lead);
    };
    for (int w = 0; w < waves; ++w) {
      Place c = share_s[w].at;
      const long long u1 = share_s[w].u1;
      for (long long u = share_s[w].u0; u < u1 && live; ++seg) {
        const ChunkTask t = list[c.task];
        const int n = (int)min((long long)t.blocks - c.block, u1 - u);
        const bool one = t.ntok <= p.tok_tile;
        live = wait_warp(&q_full[seg % Gm::Q_BUFS], (seg / Gm::Q_BUFS) & 1, &stop_s);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x == 0 || one) k = r.take<ST>();
          scores(x, one);
        }
        if (n == 1 && live) tc_commit(&q_empty[seg % Gm::Q_BUFS], lead);
        for (int j = 0; j < n && live; ++j) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // the next block's scores go before this block's output: the softmax need not wait for either
            if (j + 1 < n) {
              if (x == 0 || one) k = r.take<ST>();
              scores(x, one);
              if (j + 2 == n && x == 1 && live) tc_commit(&q_empty[seg % Gm::Q_BUFS], lead);
            }
            if (x == 0 || one) v = r.take<ST>();
            const uint64_t b = vd + v.st * kStep;
            live = live && wait_warp(&full[v.st], v.ph, &stop_s);
            live = live && wait_warp(&p_ready[x], ph_p, &stop_s);
            if (!live) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < kTile / 16; ++i)
              mma_ts(tmem + Gm::COL_O + x * D, tmem + Gm::COL_P + x * (kTile / 2) + i * 8, b + i * (2048 >> 4), kFormO,
                     (j & (kFoldUnits - 1)) > 0 || i > 0, lead);
            tc_commit(&pv_done[x], lead);
            if (one || x == 1) tc_commit(&empty[v.st], lead);
          }
          ph_p ^= 1;
        }
        u += n;
        next_task(c, tasks);
      }
    }
    // every product has left shared and tensor memory before they are given back
    tc_commit(&drain, lead);
    mbar_wait_bounded(&drain, 0);
    __syncwarp();
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax and output
    regs_up();
    const int x = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const int s_buf = Gm::S_BUFS == 1 ? 0 : x;
    const uint32_t tS = tmem + Gm::COL_S + s_buf * kTile + lanes, tP = tmem + Gm::COL_P + x * (kTile / 2) + lanes,
                   tO = tmem + Gm::COL_O + x * D + lanes;
    const float scale = p.scale_log2, grow_by = 8.f / scale;
    int base = 0;
    uint32_t ph_s = 0, ph_o = 0, ph_half = 0;
    bool half_used = false;
    // After a wait that ran out the waits below return at once and what is computed does not count.
    for (int w = 0; w < waves; ++w) {
      Place c = share_s[w].at;
      long long left = share_s[w].u1 - share_s[w].u0;
      bool first = true;
      while (left > 0) {
        int n, plain0, plain1;
        bool one, mine, busy;
        {
          const GroupSeg g(p, list_s, c, x);
          n = (int)min((long long)g.t.blocks - c.block, left);
          one = g.one;
          mine = r < g.toks * p.G;
          busy = quad * 32 < g.toks * p.G;
          g.plain(p, x, plain0, plain1);
        }
        float m = -INFINITY, l = 0.f;

        // V rows that no token sees may hold anything, and 0 * NaN is not 0: a thread clears its row.
        auto clear_row = [&](int j) {
          const GroupSeg g(p, list_s, c, x);
          const int v = (one ? (c.block + j) * 4 + 2 * x : (c.block + j) * 2) + (r >> 6);
          const int pj = g.vis.page(v) * kPage + (r & 63);
          const bool clear = v < g.vis.nv && (pj >= g.t.seqlen || (pj < g.vis.first && pj >= p.sinks));
          if (__any_sync(0xffffffffu, clear)) {
            // The parity tells this turn of the place from the next one only if the block one turn
            // earlier has landed: it is this unit's K or lies before it, which the matrix warp, taking
            // all blocks in order, had waited for before these scores.
            const int idx = base + ring_v(one, j, x, n), st = idx % ST;
            wait_row(&full[st], (idx / ST) & 1, &stop_s);
            if (clear) {
              unsigned char* z = ring + (size_t)st * Gm::TILE_BYTES + r * 128;
#pragma unroll
              for (int hf = 0; hf < Gm::HALVES; ++hf)
#pragma unroll
                for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(z + hf * Gm::HALF_BYTES + i * 16) = make_uint4(0, 0, 0, 0);
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            __syncwarp();
          }
        };

        if (!busy) {  // a warp without rows keeps step
          for (int j = 0; j < n; ++j) {
            wait_row(&s_full[x], ph_s, &stop_s);
            ph_s ^= 1;
            if (j < plain0 || j >= plain1) clear_row(j);
            if (lane == 0) mbar_arrive(&s_read[s_buf]);
            if (j > 0) {
              wait_row(&pv_done[x], ph_o, &stop_s);
              ph_o ^= 1;
            }
            if (lane == 0) mbar_arrive(&p_ready[x]);
          }
        } else {
          // The loop is kept to one straight run of instructions with few branches over rare work:
          // with a branch around each part of it for warps without rows it took 386K cycles instead
          // of 344K for 512 tokens on 32K rows.
          for (int j = 0; j < n; ++j) {
            wait_row(&s_full[x], ph_s, &stop_s);
            ph_s ^= 1;
            tc_fence_after();
            if (j < plain0 || j >= plain1) {
              // Scores that a row does not see are overwritten where they lie.
              clear_row(j);
              const GroupSeg g(p, list_s, c, x);
              const int pos = g.plo + r / p.G, wlo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
#pragma unroll 1
              for (int i = 0; i < 2; ++i) {
                const int v = (one ? (c.block + j) * 4 + 2 * x : (c.block + j) * 2) + i, j0 = g.vis.page(v) * kPage;
                uint64_t see = ~0ull;
                if (mine)
                  see = v < g.vis.nv ? low_bits(pos + 1 - j0) & (~low_bits(wlo - j0) | low_bits(p.sinks - j0)) : 0;
                if (__all_sync(0xffffffffu, see == ~0ull)) continue;
#pragma unroll 1
                for (int k = 0; k < kPage; k += 32, see >>= 32) {
                  float y[32];
                  tmem_ld32(y, tS + i * kPage + k);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (!((uint32_t)see & (1u << e))) y[e] = -INFINITY;
                  tmem_st16(tS + i * kPage + k, reinterpret_cast<const uint32_t*>(y));
                  tmem_st16(tS + i * kPage + k + 16, reinterpret_cast<const uint32_t*>(y) + 16);
                }
              }
              tmem_wait_st();
            }
            float s[kTile];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld32(s + 32 * i, tS + 32 * i);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_read[s_buf]);
            float mx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) mx[e] = max3(s[e], s[8 + e], s[16 + e]);
#pragma unroll
            for (int i = 24; i < kTile - 8; i += 16)
#pragma unroll
              for (int e = 0; e < 8; ++e) mx[e] = max3(mx[e], s[i + e], s[i + 8 + e]);
#pragma unroll
            for (int e = 0; e < 8; ++e) mx[e] = fmaxf(mx[e], s[kTile - 8 + e]);
            const float top = fmaxf(max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[4]), max3(mx[5], mx[6], mx[7]));
            const bool grow = __any_sync(0xffffffffu, mine && top > m + grow_by);
            const float mn = grow ? fmaxf(m, top) : m;
            const float f = m == -INFINITY ? 0.f : ex2((m - mn) * scale);  // 1 where m stays
            m = mn;
            // The product of the block before has read P, and O may be scaled.
            if (j > 0) {
              wait_row(&pv_done[x], ph_o, &stop_s);
              ph_o ^= 1;
              tc_fence_after();
              if ((j & (kFoldUnits - 1)) == 0) {
                // O moves to the partial; its maximum there is the one of now
                const int slot = 2 * (w * p.ctas + (int)blockIdx.x) + (first ? 0 : 1), at = x * kTile + r;
                float4* part = reinterpret_cast<float4*>(p.part) + (size_t)slot * (D / 4) * kRowsCap + at;
                float* was = &p.ml[(size_t)slot * kRowsCap + at].x;
                const float m0 = j == kFoldUnits ? -INFINITY : *was;
                const float g = ex2((m0 == -INFINITY ? m0 : m0 - m) * scale);  // a select: the warp stays together
#pragma unroll 1
                for (int i = 0; i < D / 8; ++i) {
                  float o[8];
                  tmem_ld8(o, tO + 8 * i);
                  float4 y[2] = {};
                  if (j > kFoldUnits) {
                    y[0] = part[(size_t)(2 * i) * kRowsCap];
                    y[1] = part[(size_t)(2 * i + 1) * kRowsCap];
                  }
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    part[(size_t)(2 * i + e) * kRowsCap] = make_float4(y[e].x * g + o[4 * e] * f, y[e].y * g + o[4 * e + 1] * f,
                                                                       y[e].z * g + o[4 * e + 2] * f, y[e].w * g + o[4 * e + 3] * f);
                }
                *was = m;
                __syncwarp();
              } else if (grow) {
#pragma unroll 1
                for (int i = 0; i < D / 8; ++i) {  // 8 columns at a time: the scores stay in registers
                  float o[8];
                  tmem_ld8(o, tO + 8 * i);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 8; ++e) o[e] *= f;
                  tmem_st8(tO + 8 * i, o);
                }
              }
            }
            const float off = m == -INFINITY ? 0.f : -m * scale;
            const float2 sc2 = make_float2(scale, scale), off2 = make_float2(off, off);
            float2 sum[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t q[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float2 z = ffma2(make_float2(s[32 * i + 2 * e], s[32 * i + 2 * e + 1]), sc2, off2);
                z.x = ex2(z.x);
                z.y = ex2(z.y);
                sum[e & 3] = __fadd2_rn(sum[e & 3], z);
                q[e] = pack_bf16(z.x, z.y);
              }
              tmem_st16(tP + 16 * i, q);
            }
            sum[0] = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
            l = l * f + (sum[0].x + sum[0].y);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[x]);
          }
        }

        // ---- this segment's rows ----
        wait_row(&pv_done[x], ph_o, &stop_s);
        ph_o ^= 1;
        tc_fence_after();
        const GroupSeg g(p, list_s, c, x);
        const bool done = n == g.t.blocks;
        const int slot = 2 * (w * p.ctas + (int)blockIdx.x) + (first ? 0 : 1), at = x * kTile + r;
        float4* part = reinterpret_cast<float4*>(p.part) + (size_t)slot * (D / 4) * kRowsCap;
        float2* ml = p.ml + (size_t)slot * kRowsCap;
        const float mz = m == -INFINITY ? m : m * scale;
        // what the partial holds already of a long segment's outputs
        const bool folded = n > kFoldUnits;
        const float m0 = folded ? ml[at].x : -INFINITY;
        const float fold = ex2((m0 == -INFINITY ? m0 : m0 - m) * scale);
        auto add_folded = [&](float (&o)[32], int i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 y = part[(size_t)(8 * i + e) * kRowsCap + at];
            o[4 * e] += y.x * fold;
            o[4 * e + 1] += y.y * fold;
            o[4 * e + 2] += y.z * fold;
            o[4 * e + 3] += y.w * fold;
          }
        };
        if (!done || (one && x == 1)) {
          // the other warpgroup has read the half it got before
          if (done && half_used) wait_row(&half_free, ph_half ^ 1, &stop_s);
          if (busy) {
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              float o[32];
              tmem_ld32(o, tO + 32 * i);
              tmem_wait_ld();
              if (mine) {
                if (folded) add_folded(o, i);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  part[(size_t)(8 * i + e) * kRowsCap + at] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
              }
              __syncwarp();
            }
            if (mine) ml[at] = make_float2(mz, l);
          }
          if (done) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&half_full);
            half_used = true;
            ph_half ^= 1;
          }
        } else {
          float f0 = 1.f, f1 = 0.f, M = mz, L = l;
          if (one) {
            wait_row(&half_full, ph_half, &stop_s);
            ph_half ^= 1;
            if (mine) {
              const float2 y = __ldcg(ml + kTile + r);
              M = fmaxf(mz, y.x);
              f0 = mz == -INFINITY ? 0.f : ex2(mz - M);
              f1 = y.x == -INFINITY ? 0.f : ex2(y.x - M);
              L = l * f0 + y.y * f1;
            }
          }
          if (busy) {
            const float inv = L > 0.f ? 1.f / L : 0.f;
            const size_t o_row = (size_t)(g.t.tok0 + g.tile * p.tok_tile + r / p.G) * p.Hq + c.h * p.G + r % p.G;
            uint4* dst = reinterpret_cast<uint4*>(p.out + o_row * D);
            f0 *= inv;
            f1 *= inv;
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              float o[32];
              tmem_ld32(o, tO + 32 * i);
              tmem_wait_ld();
              if (mine) {
                if (folded) add_folded(o, i);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f0;
                if (one) {
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const float4 y = __ldcg(part + (size_t)(8 * i + e) * kRowsCap + kTile + r);
                    o[4 * e] += y.x * f1;
                    o[4 * e + 1] += y.y * f1;
                    o[4 * e + 2] += y.z * f1;
                    o[4 * e + 3] += y.w * f1;
                  }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  dst[4 * i + e] = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                              pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
              }
              __syncwarp();
            }
            if (mine && p.lse != nullptr) p.lse[o_row] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
          }
          if (one) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&half_free);
          }
        }
        base += (one ? 4 : 2) * n;
        left -= n;
        first = false;
        next_task(c, tasks);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  if (tid == 0 && stop_s) record_error(p.err, kDevWaitTimeout, blockIdx.x);
}

// Joins the partials of a task that several CTAs share, in CTA order.  blockIdx.x names the wave and
// the share whose beginning is looked at: the first one inside a task acts for it.  (A join by the
// last CTA of the task, in the kernel above, has too few loads in flight: 512 tokens on 32K rows
// took 499 us with it, 287 us with a kernel of its own.)
constexpr int kJoinThreads = 1024;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ Place at_s;
  pdl_wait();
  pdl_trigger();
  const int tasks = p.tasks[p.slots].b;
  const long long units = p.tasks[p.slots].unit0;
  const int waves = p.tasks[p.slots].tok0, wi = (int)blockIdx.x / (p.ctas - 1), cta = (int)blockIdx.x % (p.ctas - 1);
  if (wi >= waves) return;
  const Wave wave = wave_of(p, wi, waves, units);
  const long long share = wave.share, u = share * (cta + 1);
  if (u >= wave.total) return;
  if (threadIdx.x < 32) {
    const Place c = find_unit(p.tasks, u, tasks, units);
    if (threadIdx.x == 0) at_s = c;
  }
  __syncthreads();
  Place c = at_s;
  c.h += wave.head0;
  if (c.block == 0) return;
  const ChunkTask t = p.tasks[c.task];
  const long long t0 = u - c.block;                      // the task's first unit
  const int c0 = (int)(t0 / share), c1 = (int)((t0 + t.blocks - 1) / share);
  if (c0 != cta) return;
  const bool one = t.ntok <= p.tok_tile;
  const int per = one ? 2 : 1, np = (c1 - c0 + 1) * per;
  const int slot1 = 2 * (wi * p.ctas + c0), slot0 = slot1 + (t0 != c0 * share ? 1 : 0);
  // Place of partial i of a row; a one-tile task has two per CTA, 128 rows apart.
  auto slot = [&](int i) { return i < per ? slot0 : slot1 + 2 * (one ? i >> 1 : i); };
  auto line = [&](int i, int row) { return one ? row + (i & 1) * kTile : row; };
  auto token = [&](int row) { return (size_t)t.tok0 + (row / kTile) * p.tok_tile + row % kTile / p.G; };
  auto valid = [&](int row) { return row % kTile < (min(p.tok_tile, t.ntok - row / kTile * p.tok_tile)) * p.G; };
  if (threadIdx.x < kRowsCap && valid(threadIdx.x)) {
    const int row = threadIdx.x;
    float M = -INFINITY, L = 0.f;
#pragma unroll 4
    for (int i = 0; i < np; ++i) M = fmaxf(M, p.ml[(size_t)slot(i) * kRowsCap + line(i, row)].x);
#pragma unroll 4
    for (int i = 0; i < np; ++i) {
      float2* y = p.ml + (size_t)slot(i) * kRowsCap + line(i, row);
      const float f = y->x == -INFINITY ? 0.f : ex2(y->x - M);
      L += f * y->y;
      y->x = f;                                          // the partial's factor takes the place of its maximum
    }
    const int tok_row = row % kTile % p.G;
    // the sum's place in the first partial holds its inverse
    p.ml[(size_t)slot0 * kRowsCap + row].y = L > 0.f ? 1.f / L : 0.f;
    if (p.lse != nullptr) p.lse[token(row) * p.Hq + c.h * p.G + tok_row] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
  }
  __syncthreads();
  // A warp takes 8 columns of 32 rows at a time.
  const int lane = threadIdx.x & 31, groups = one ? (min(p.tok_tile, t.ntok) * p.G + 31) / 32 : kRowsCap / 32;
  for (int e = threadIdx.x >> 5; e < groups * (D / 8); e += kJoinThreads / 32) {
    const int row = e % groups * 32 + lane, c8 = e / groups;
    if (!valid(row)) continue;
    float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < np; ++i) {
      const int at = line(i, row);
      const float f = p.ml[(size_t)slot(i) * kRowsCap + at].x;
      const float4* part = reinterpret_cast<const float4*>(p.part) + ((size_t)slot(i) * (D / 4) + 2 * c8) * kRowsCap + at;
      const float4 o0 = __ldcg(part), o1 = __ldcg(part + kRowsCap);
      a[0] += f * o0.x;
      a[1] += f * o0.y;
      a[2] += f * o0.z;
      a[3] += f * o0.w;
      a[4] += f * o1.x;
      a[5] += f * o1.y;
      a[6] += f * o1.z;
      a[7] += f * o1.w;
    }
    const float inv = p.ml[(size_t)slot0 * kRowsCap + row].y;
    reinterpret_cast<uint4*>(p.out + (token(row) * p.Hq + c.h * p.G + row % kTile % p.G) * D)[c8] =
        make_uint4(pack_bf16(a[0] * inv, a[1] * inv), pack_bf16(a[2] * inv, a[3] * inv), pack_bf16(a[4] * inv, a[5] * inv),
                   pack_bf16(a[6] * inv, a[7] * inv));
  }
}

template <int D>
cudaError_t launch_d(const ChunkParams& p, cudaStream_t stream) {
  cudaError_t e = prepare_kernel((const void*)chunk_kernel<D>, Geo<D>::SMEM);
  if (e != cudaSuccess) return e;
  if (!p.own_plan) {
    e = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(chunk_kernel<D>, dim3((unsigned)p.ctas), dim3(kThreads), (size_t)Geo<D>::SMEM, stream, p);
  if (e != cudaSuccess || p.ctas == 1) return e;
  return launch_pdl(join_kernel<D>, dim3((unsigned)((p.ctas - 1) * p.waves_max)), dim3(kJoinThreads), 0, stream, p);
}

// Never less for more new tokens, so that a workspace for many serves a call with few.
size_t task_bytes(const ChunkParams& p) {
  const size_t own = (size_t)kChunkMaxCtas * ((p.slots < kOwnPlanSlots ? p.slots : kOwnPlanSlots) + 1), one = (size_t)p.slots + 1;
  return ((own > one ? own : one) * sizeof(ChunkTask) + 255) & ~(size_t)255;
}

}  // namespace

void plan_chunk(ChunkParams& p) {
  p.tok_tile = kTile / p.G;
  p.slots = p.n_new / (2 * p.tok_tile) + p.B;
  p.own_plan = p.slots <= kOwnPlanSlots ? 1 : 0;
  // More than one wave only where some sequence can have several tasks and the cache can exceed a wave.
  const long long bytes = (p.paged ? (long long)p.num_pages * kPage : (long long)p.B * p.cap) * p.Hkv * p.d * 4;
  const long long most = 1 + bytes / kLiveBytes;
  p.waves_max = p.Hkv < kChunkMaxWaves ? p.Hkv : kChunkMaxWaves;
  if (most < p.waves_max) p.waves_max = (int)most;
  if (p.n_new <= 2 * p.tok_tile) p.waves_max = 1;
}

size_t chunk_workspace_bytes(const ChunkParams& p) {
  return task_bytes(p) +
         (size_t)2 * kChunkMaxCtas * p.waves_max * kRowsCap * (sizeof(float2) + (size_t)p.d * 4);
}

void bind_chunk(ChunkParams& p, void* scratch) {
  unsigned char* w = static_cast<unsigned char*>(scratch);
  p.tasks = reinterpret_cast<ChunkTask*>(w);
  w += task_bytes(p);
  p.ml = reinterpret_cast<float2*>(w);
  w += (size_t)2 * kChunkMaxCtas * p.waves_max * kRowsCap * sizeof(float2);
  p.part = reinterpret_cast<float*>(w);
}

cudaError_t launch_chunk(const ChunkParams& p, cudaStream_t stream) {
  if (p.d == 128) return launch_d<128>(p, stream);
  if (p.d == 64) return launch_d<64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace sas
