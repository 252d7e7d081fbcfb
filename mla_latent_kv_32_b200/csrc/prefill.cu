// Attention of a ragged batch of chunks in the expanded form of MLA: for query
// row t of a sequence with k_len keys, and head h,
//   s_i = (q^C[t,h] . k^C[i,h] + q^R[t,h] . k^R[i]) * scale      (192 columns)
//   o   = sum_i softmax(s)_i v[i,h]                              (128 columns)
// over the keys that the row sees: all of them, or (causal) the first
// k_len - q_len + j + 1 for row j of q_len ("DeepSeek-V3 MLA: Multi-Head
// Latent Attention Guide", "Core Architecture & Mathematics": per-head keys
// [k^C ; k^R] with k^R shared by the heads).
//
// Work: an item is up to 256 query rows of one sequence and head, as two
// streams of 128 rows, and a range of 128-key tiles; a persistent CTA per SM
// runs the items of its list. A tile's keys and values are loaded once for
// both streams. Tensor memory holds, for each stream, 128 columns of scores
// and 128 of output; the probabilities (bf16) overwrite the scores' columns
// and feed the output MMA from there.
//   S_i = Q_i K^T   A = 128 query rows (shared memory), B = 128 keys, K = 192
//   O_i += P_i V    A = P_i (tensor memory),  B = V (128 keys x 128), K = 128
// While one stream's softmax runs on the CUDA cores, the tensor core does the
// other stream's two products: 1280 tensor clocks a stream and tile, against
// 1024 clocks of the SM's exponential unit for its 128 x 128 exponentials.
//
// An item of up to 128 rows would leave the second stream idle and a stream waits
// for its scores and outputs half of its time. There the streams take the key tiles
// in turn, each with a running maximum, sum and output of its own, merged at the
// end; the shared memory holds two slots of keys and two of values, and a tile's
// load waits for nothing but the tile before the last.
//
// Warps (384 threads): 0 TMA, 1 MMA issue and tensor memory, 2 zeroes the
// values behind a sequence's last key, 3 watches the others, 4-7 and 8-11 softmax
// and epilogue of stream 0 and 1 (thread = query row = TMEM lane).
// A ring of eight 16 KB stages carries the tiles in the order they are used:
// three 64-column chunks of the keys (k^C twice, k^R), two 64-key halves of
// the values; a barrier each for a tile's keys and its values. The MMAs of one
// thread complete in the order they are issued, so scores(t + 1) of a stream
// may be issued right behind output(t), and scores being complete means that
// the stream's output so far is, too.
//
// Softmax: running maximum and sum in float32 (log2 units), the reference
// maximum raised (and O rescaled) only when a row's maximum grows by more than
// 8, exact up to rounding since the final division uses the same reference.
// The sum takes the unrounded probabilities; P is rounded to bf16, as V is
// stored, since one MMA takes one operand type.
//
// Scores of keys that a row does not see are replaced, whatever they are; the
// rows of V behind a sequence's last key are zeroed in shared memory. So what
// lies behind a sequence's keys never matters. A row that sees no key gets
// o = 0 and lse = -inf.
//
// Every wait is bounded: warp 3 watches the others (the MMA thread counts its steps, each
// role the items that have none for it) until they are done. When nothing has moved on for
// about a second it sets MLA_DEV_TIMEOUT and tells the waiting warps to give up: the CTA
// stops issuing, lets what it issued land and leaves. The length of a call does not
// matter: the warp that zeroes tails may wait for its first tile as long as the CTA
// works. (A clock in each wait is more code at every one of them: 8 short prompts of 16
// heads 12.4-12.8 us instead of 12.3.)
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "internal.h"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kTmaWarp = 0, kMmaWarp = 1, kTailWarp = 2, kWatchWarp = 3;
// The softmax threads hold a row of a tile; the other warpgroup's registers go to
// them: 256 x 208 + 128 x 88 = 384 x 168, what the block is launched with.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kStages = 8;
constexpr uint32_t kChunk = 128 * 128;               // 128 rows x 64 bf16
constexpr int kKeyChunks = 3, kTileChunks = 5;       // per tile: keys, keys + values
constexpr uint32_t kOffQ = 0;                        // [stream][3 chunks]
constexpr uint32_t kOffRing = 2 * kKeyChunks * kChunk;
constexpr uint32_t kOffBar = kOffRing + kStages * kChunk;
enum {
  B_KFULL = 0,                  // [2] keys of a tile landed (tiles alternate)
  B_VFULL = B_KFULL + 2,        // [2] values of a tile landed
  B_KFREE = B_VFULL + 2,        // [2] keys of a tile used by their last MMA
  B_VFREE = B_KFREE + 2,        // [2] values of a tile used by their last MMA
  B_QFULL = B_VFREE + 2,        // [2] the stream's query rows landed
  B_QFREE = B_QFULL + 2,        // last score MMA of the item complete
  B_SFULL,                      // [2] scores of a tile complete
  B_PFULL = B_SFULL + 2,        // [2][2] half of a tile's probabilities written (4 warps)
  B_OFULL = B_PFULL + 4,        // [2] last output MMA of the item complete
  B_SWAP = B_OFULL + 2,         // turns: maxima and sums posted; outputs read (8 warps)
  B_LANDED,                     // values that need zeroing have landed
  B_TAIL,                       // ... and are zeroed
  B_FINAL,
  B_DONE,                       // the other warps have ended (11 arrivals)
  B_COUNT
};
constexpr uint32_t kOffTmemPtr = kOffBar + 8 * B_COUNT;
constexpr uint32_t kOffAbort = kOffTmemPtr + 4;
constexpr uint32_t kOffMoved = kOffAbort + 4;        // items passed without MMAs; MMA steps
constexpr uint32_t kOffSwap = (kOffMoved + 8 + 15) & ~15u;   // [stream][128] (maximum, sum)
constexpr uint32_t kSmemBytes = kOffSwap + 2 * 128 * 8;
static_assert(kSmemBytes <= 232448, "shared memory budget");

constexpr uint32_t kTmemS = 0, kTmemO = 256;         // stream i at + 128 i
constexpr float kRescale = 8.0f;                     // log2 units

struct Args {
  const int32_t *cta_begin;
  const PrefillItem *items;
  const PrefillCombine *combine;
  int num_items, T_q, T_k, n_h, causal, num_partials;
  int sectors;   // rows and heads of o, and the partial results, start on 32-byte boundaries
  float scale_log2;
  float *ws_o, *ws_lse;
  uint16_t *o;
  long long ld_o, hs_o;
  float *lse;
  uint32_t *status;
  uint64_t wait_ns;     // a wait gives up when nothing has moved for so long
  int suppress_tail;    // test hook: the first tail is not handed back
};

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }

constexpr uint32_t kStepsDone = 0xFFFFFFFFu;

struct Ctx {
  uint32_t bar_base;
  volatile int *abort_flag;
  uint32_t moved;       // kOffMoved
  uint32_t *status;
  uint64_t wait_ns;
  __device__ uint32_t bar(int i) const { return bar_base + 8u * i; }
  // One thread of a role: it comes to an item that has no MMA for it.
  __device__ __forceinline__ void pass_item() const {
    asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(moved) : "memory");
  }
  // The MMA thread: its next step, or the last (kStepsDone).
  __device__ __forceinline__ void step(uint32_t n) const {
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(moved + 4), "r"(n) : "memory");
  }
  __device__ __forceinline__ bool steps_done() const {
    uint32_t steps;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(steps) : "r"(moved + 4) : "memory");
    return steps == kStepsDone;
  }
  __device__ __forceinline__ uint32_t progress() const {
    uint32_t items, steps;
    asm volatile("ld.volatile.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(items), "=r"(steps)
                 : "r"(moved)
                 : "memory");
    return items + steps;
  }
};

// (Inlined: a call would have to save the tile's scores around it.)
__device__ __forceinline__ bool wait_slow(const Ctx &c, uint32_t bar, uint32_t parity) {
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63) == 0 && *c.abort_flag) return false;
  }
}

// What has been issued lands, also after the others have given up.
__device__ __forceinline__ void drain(const Ctx &c, uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > c.wait_ns) {
      *c.abort_flag = 1;
      report(c.status, MLA_DEV_TIMEOUT);
      return;
    }
}

// The watching thread: returns when the other warps have ended or, having told them,
// when nothing has moved on for too long. It sleeps until the MMAs are done, since its
// looks cost large calls 5 % otherwise, and is then there when the others end.
__device__ __forceinline__ void watch(const Ctx &c, uint32_t bar) {
  uint64_t t0 = globaltimer_ns();
  uint32_t seen = c.progress();
  while (!mbar_try_wait(bar, 0)) {
    if (!c.steps_done()) __nanosleep(200);
    const uint32_t now = c.progress();
    if (now != seen) {
      seen = now;
      t0 = globaltimer_ns();
    } else if (globaltimer_ns() - t0 > c.wait_ns) {
      *c.abort_flag = 1;
      report(c.status, MLA_DEV_TIMEOUT);
      return;
    }
  }
}

// Whole warp; false when the wait ran out or another warp has given up.
__device__ __forceinline__ bool wait_warp(const Ctx &c, uint32_t bar, uint32_t parity) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = wait_slow(c, bar, parity);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool wait_one(const Ctx &c, uint32_t bar, uint32_t parity) {
  return wait_slow(c, bar, parity);
}

// D[tmem] (+)= A[tmem] * B[smem desc], bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The value of lane 0, known to the compiler to be the same in every lane (it
// may then stay in the uniform registers that the MMAs take their operands from).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Moves registers between the warpgroups (whole warpgroups, once each).
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// 2^x with the hardware approximation (relative error about 2^-22; 2^-inf = 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 consecutive columns
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// ---- pairs of floats: Blackwell's two-wide float32 operations ----
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// max of three, NaN if any is (the exponent unit's NaN must not get lost)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Items whose tiles the streams take in turn: where tile k's keys and values are.
__device__ __forceinline__ uint32_t turn_keys(uint32_t base, uint32_t k) {
  return base + kOffRing + (k & 1) * kKeyChunks * kChunk;
}
__device__ __forceinline__ uint32_t turn_values(uint32_t base, uint32_t k) {
  return base + ((k & 1) ? kOffQ + kKeyChunks * kChunk : kOffRing + 2 * kKeyChunks * kChunk);
}

struct Item {
  int q_row, q_rows, h, k_row, k_len, lim0, tile_begin, slot;
  int count[2];   // key tiles of each stream
  int tiles;      // tiles to load
  bool turns;     // up to 128 rows: both streams take them, tile t is stream t % 2's
  bool ok;
  // tile t of the range ends behind the sequence's last key
  __device__ __forceinline__ bool tail(int t) const {
    return (tile_begin + t + 1) * kPrefillKeys > k_len;
  }
};

template <bool kTurns>
__device__ __forceinline__ Item load_item(const Args &a, const PrefillItem *p) {
  Item it;
  const int4 x = __ldg(reinterpret_cast<const int4 *>(p));
  const int4 y = __ldg(reinterpret_cast<const int4 *>(p) + 1);
  it.q_row = x.x;
  it.q_rows = x.y;
  it.h = x.z;
  it.k_row = x.w;
  it.k_len = y.x;
  it.lim0 = y.y;
  it.tile_begin = y.z;
  const int tile_end = y.w;
  it.slot = __ldg(&p->slot);
  const int all = it.k_len / kPrefillKeys + (it.k_len % kPrefillKeys != 0);
  it.ok = it.q_rows > 0 && it.q_rows <= kPrefillRows && it.q_row >= 0 &&
          it.q_row <= a.T_q - it.q_rows && it.h >= 0 && it.h < a.n_h && it.k_len >= 0 &&
          it.k_row >= 0 && it.k_row <= a.T_k - it.k_len && it.lim0 <= it.k_len &&
          it.tile_begin >= 0 && tile_end <= all &&
          (it.slot < 0 || it.slot <= a.num_partials - it.q_rows);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // the keys of the stream's last row, in tiles
    const int last = min(it.q_rows, 128 * (i + 1)) - 1;
    const int lim = last < 128 * i ? 0 : min(it.k_len, it.lim0 + (a.causal ? last : 0));
    const int end = min(tile_end, (lim + kPrefillKeys - 1) / kPrefillKeys);
    it.count[i] = lim <= 0 ? 0 : max(0, end - it.tile_begin);
  }
  it.tiles = max(it.count[0], it.count[1]);
  it.turns = kTurns && it.q_rows <= kTurnRows && it.tiles >= kTurnTiles;
  if (it.turns) {
    it.count[1] = it.tiles >> 1;
    it.count[0] = it.tiles - it.count[1];
  }
  return it;
}

// (Each lane has a row of its own, so the time goes by sectors: 16 bytes at a time 3
// prompts of 685 tokens, 128 heads, take 108.6 us instead of 104.3, and 7 of up to 1725,
// 4 heads, whose partial results are stored too, 29.7 instead of 24.7. Passing rows
// around four lanes for 64 bytes a row was slower for short prompts.)
// Stores columns [col, col + 32) of a row, scaled: float32 into the partial
// results (slot >= 0), or bf16 into o.
__device__ __forceinline__ void store32(const Args &a, int slot, int row, size_t out_row, int h,
                                        int col, const uint32_t (&r)[32], float inv) {
  if (slot >= 0) {
    float *dst = a.ws_o + (size_t)(slot + row) * 128 + col;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(u2f(r[8 * k + e]) * inv);
      store_sector(dst + 8 * k, w, a.sectors);
    }
  } else {
    uint16_t *dst = a.o + (long long)out_row * a.ld_o + (long long)h * a.hs_o + col;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = cvt_bf16x2(u2f(r[16 * k + 2 * e]) * inv, u2f(r[16 * k + 2 * e + 1]) * inv);
      store_sector(dst + 16 * k, w, a.sectors);
    }
  }
}

// kTurns: the plan has items of up to 128 rows (the other instance is free of
// their branches, 4-5 % on full items).
template <bool kTurns>
__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap tm_qn, const __grid_constant__ CUtensorMap tm_qp,
               const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ CUtensorMap tm_kp, const Args a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  if (base & 1023u) {   // the swizzled tiles need it
    if (threadIdx.x == 0) report(a.status, MLA_DEV_BAD_PLAN);
    return;
  }
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  // the first item is on its way while the barriers are made
  const PrefillItem *items = a.items;
  int i0 = __ldg(a.cta_begin + blockIdx.x), i1 = __ldg(a.cta_begin + blockIdx.x + 1);
  if (i0 < 0 || i1 > a.num_items || i0 > i1) {   // not the plan that was launched
    if (threadIdx.x == 0) report(a.status, MLA_DEV_BAD_PLAN);
    i0 = i1 = 0;
  }
  if (warp == kTailWarp && lane < 2 && i0 < i1) {   // (into L1, where the other warps' loads find it)
    uint32_t unused;
    asm volatile("ld.global.nc.b32 %0, [%1];"
                 : "=r"(unused)
                 : "l"(reinterpret_cast<const char *>(items + i0) + lane * (sizeof(PrefillItem) - 4)));
  }
  Ctx ctx;
  ctx.bar_base = base + kOffBar;
  ctx.abort_flag = reinterpret_cast<volatile int *>(smem + kOffAbort);
  ctx.moved = base + kOffMoved;
  static_assert(kOffMoved % 8 == 0, "two words read at once");
  ctx.status = a.status;
  ctx.wait_ns = a.wait_ns;
  static_assert(B_COUNT <= 32, "a lane per barrier");
  if (warp == kTmaWarp) {
    if (lane == 0) *ctx.abort_flag = 0;
    if (lane < 2) reinterpret_cast<volatile int *>(smem + kOffMoved)[lane] = 0;
    if (lane < B_COUNT)
      mbar_init(ctx.bar(lane),
                lane >= B_PFULL && lane < B_PFULL + 4 ? 4
                : lane == B_SWAP                    ? 8
                : lane == B_DONE                    ? kThreads / 32 - 1
                                                    : 1);
    fence_mbar_init_cluster();
  }
  if (warp == kMmaWarp) tmem_alloc(base + kOffTmemPtr, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*reinterpret_cast<volatile int *>(smem + kOffTmemPtr));

  const uint32_t ring = base + kOffRing;

  if (warp < 4) regs_dec<kOtherRegs>();
  if (warp == kTmaWarp) {
    if (elect_one()) {
      tma_prefetch_desc(&tm_qn);
      tma_prefetch_desc(&tm_qp);
      tma_prefetch_desc(&tm_kn);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_kp);
      uint32_t n = 0;                 // tiles loaded
      uint32_t runs = 0, nq[2] = {0, 0};
      uint32_t keys = 0, values = 0;  // parts issued
      bool ok = true;
      // Tile n takes the stages 5 n .. 5 n + 4 of the ring: three of keys, two of
      // values. The first three held tile n - 2's last keys and its values, the
      // other two the first keys of tile n - 1.
      auto stage = [&](int c) { return ring + ((n * kTileChunks + c) % kStages) * kChunk; };
      auto freed = [&](int bar, uint32_t tile) {
        ok = ok && wait_one(ctx, ctx.bar(bar + (tile & 1)), (tile >> 1) & 1);
        return ok;
      };
      auto load_keys = [&](const Item &x, int row, uint32_t tile, uint32_t d0, uint32_t d1,
                           uint32_t d2) {
        const uint32_t bar = ctx.bar(B_KFULL + (tile & 1));
        mbar_arrive_expect_tx(bar, kKeyChunks * kChunk);
        tma_load_3d(d0, &tm_kn, 0, row, x.h, bar);
        tma_load_3d(d1, &tm_kn, 64, row, x.h, bar);
        tma_load_3d(d2, &tm_kp, 0, row, 0, bar);
        ++keys;
      };
      auto load_values = [&](const Item &x, int row, uint32_t tile, uint32_t d0, uint32_t d1) {
        const uint32_t bar = ctx.bar(B_VFULL + (tile & 1));
        mbar_arrive_expect_tx(bar, 2 * kChunk);
        for (int j = 0; j < 2; ++j) {
          tma_load_3d(j ? d1 : d0, &tm_v, 0, row + 64 * j, x.h, bar);
          tma_load_3d((j ? d1 : d0) + kChunk / 2, &tm_v, 64, row + 64 * j, x.h, bar);
        }
        ++values;
      };
      // the item's queries, when the last item's are used
      auto load_queries = [&](const Item &x) {
        if (runs > 0) ok = ok && wait_one(ctx, ctx.bar(B_QFREE), (runs - 1) & 1);
        for (int q = 0; q < 2 && ok; ++q) {
          if (x.count[q] == 0 || (q == 1 && x.turns)) continue;
          const uint32_t bar = ctx.bar(B_QFULL + q), dst = base + kOffQ + q * kKeyChunks * kChunk;
          mbar_arrive_expect_tx(bar, kKeyChunks * kChunk);
          tma_load_3d(dst, &tm_qn, 0, x.q_row + 128 * q, x.h, bar);
          tma_load_3d(dst + kChunk, &tm_qn, 64, x.q_row + 128 * q, x.h, bar);
          tma_load_3d(dst + 2 * kChunk, &tm_qp, 0, x.q_row + 128 * q, x.h, bar);
          ++nq[q];
        }
        ++runs;
      };
      bool turns = false;             // how the shared memory is laid out
      for (int i = i0; i < i1 && ok; ++i) {
        const Item it = load_item<kTurns>(a, items + i);
        if (!it.ok || it.tiles == 0) {
          if (!it.ok) report(a.status, MLA_DEV_BAD_PLAN);
          ctx.pass_item();
          continue;
        }
        const int row0 = it.k_row + it.tile_begin * kPrefillKeys;
        if (kTurns && it.turns != turns) {
          // the layouts overlap: everything of the last item is used first
          if (n > 0 && !freed(B_VFREE, n - 1)) break;
          turns = it.turns;
        }
        if (kTurns && turns) {
          // Two slots each of keys and values (the second of the values where the
          // second stream's queries would be). A tile's keys come before the last
          // tile's values: their slot is free as soon as the scores are there.
          auto keys_of = [&](int t) {
            const uint32_t k = n + t, d = turn_keys(base, k);
            if (k >= 2 && !freed(B_KFREE, k - 2)) return;
            load_keys(it, row0 + t * kPrefillKeys, k, d, d + kChunk, d + 2 * kChunk);
          };
          keys_of(0);
          load_queries(it);
          for (int t = 0; t < it.tiles && ok; ++t) {
            if (t + 1 < it.tiles) keys_of(t + 1);
            const uint32_t k = n + t, d = turn_values(base, k);
            if (!ok || (k >= 2 && !freed(B_VFREE, k - 2))) break;
            load_values(it, row0 + t * kPrefillKeys, k, d, d + kChunk);
          }
          n += it.tiles;
          continue;
        }
        for (int t = 0; t < it.tiles; ++t, ++n) {
          const int row = row0 + t * kPrefillKeys;
          // (values of n - 2 used: its keys too, the MMAs complete in order)
          if (n >= 2 && !freed(B_VFREE, n - 2)) break;
          load_keys(it, row, n, stage(0), stage(1), stage(2));
          // (the previous item's queries are used when its last keys are)
          if (t == 0) load_queries(it);
          if (!ok || (n >= 1 && !freed(B_KFREE, n - 1))) break;
          load_values(it, row, n, stage(3), stage(4));
        }
      }
      // what was issued lands before the CTA leaves
      for (uint32_t b = 0; b < 2; ++b) {
        if (keys > b) drain(ctx, ctx.bar(B_KFULL + b), ((keys - 1 - b) >> 1) & 1);
        if (values > b) drain(ctx, ctx.bar(B_VFULL + b), ((values - 1 - b) >> 1) & 1);
        if (nq[b] > 0) drain(ctx, ctx.bar(B_QFULL + b), (nq[b] - 1) & 1);
      }
      mbar_arrive(ctx.bar(B_DONE));
    }
  } else if (warp == kMmaWarp) {
    // One thread waits and issues. The softmax warps leave it few issue slots,
    // and the tensor core queues only about six MMAs (64 clocks each), so the
    // thread has little to do per MMA: one wait per tile and operand.
    if (elect_one()) {
      const uint32_t idesc_s = idesc_bf16(128, kPrefillKeys, 0, 0);
      const uint32_t idesc_o = idesc_bf16(128, MLA_D_V, 0, 1);
      const uint64_t q_desc = smem_desc(base + kOffQ, 16, 1024, kSwizzle128B);
      const uint64_t k_desc = smem_desc(ring, 16, 1024, kSwizzle128B);
      const uint64_t v_desc = smem_desc(ring, kChunk / 2, 1024, kSwizzle128B);
      uint32_t n = 0;                 // tiles of the items before this one
      // phases waited for, a bit per stream: queries, probabilities
      uint32_t nq = 0, np = 0, tails = 0, steps = 0;
      bool ok = true;
      for (int i = i0; i < i1 && ok; ++i) {
        const Item it = load_item<kTurns>(a, items + i);
        if (!it.ok || it.tiles == 0) {
          ctx.pass_item();
          continue;
        }
        const int n0 = it.count[0], n1 = it.count[1];   // no turns: n1 is 0 or >= n0
        const bool turns = kTurns && it.turns;
        // Step j of stream q: its output j, then its scores j + 1 (one piece of code
        // for both streams: the first tiles of short items pay for each line).
        // Address fields count 16 bytes.
#pragma unroll 1
        for (int j = -1; j < max(n0, n1) && ok; ++j)
#pragma unroll 1
          for (int q = 0; q < 2 && ok; ++q) {
            const int count = q ? n1 : n0;
            ctx.step(++steps);
            if (j >= 0 && j < count) {
              const int t = turns ? 2 * j + q : j;
              const uint32_t k = n + t;
              if (turns || q == 0 || j >= n0) {   // the first stream to use the tile
                ok = wait_one(ctx, ctx.bar(B_VFULL + (k & 1)), (k >> 1) & 1);
                if (ok && it.tail(t)) {   // the tail warp takes it, then hands it back
                  mbar_arrive(ctx.bar(B_LANDED));
                  ok = wait_one(ctx, ctx.bar(B_TAIL), tails++ & 1);
                }
              }
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                ok = ok && wait_one(ctx, ctx.bar(B_PFULL + 2 * q + half), (np >> q) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t bd =
                    turns ? smem_desc(turn_values(base, k) + half * kChunk, kChunk / 2, 1024,
                                      kSwizzle128B)
                          : v_desc + ((k * kTileChunks + kKeyChunks + half) % kStages) *
                                         (kChunk >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)   // a step of 16 keys: 2048 bytes
                  mma_f16_ts(tmem + kTmemO + 128 * q,
                             tmem + kTmemS + 128 * q + 32 * half + 8 * kk, bd + 128 * kk, idesc_o,
                             j > 0 || half > 0 || kk > 0 ? 1u : 0u);
              }
              if (!ok) break;
              np ^= 1u << q;
              if (turns || q == 1 || j >= n1) mma_commit(ctx.bar(B_VFREE + (k & 1)));
              if (j + 1 == count) mma_commit(ctx.bar(B_OFULL + q));
            }
            if (j + 1 < count) {
              const int t = turns ? 2 * (j + 1) + q : j + 1;
              const uint32_t k = n + t;
              const int rows = turns ? 0 : q;   // whose query rows
              if (j < 0 && rows == q) {
                ok = wait_one(ctx, ctx.bar(B_QFULL + q), (nq >> q) & 1);
                nq ^= 1u << q;
              }
              if (turns || q == 0 || j + 1 >= n0)
                ok = ok && wait_one(ctx, ctx.bar(B_KFULL + (k & 1)), (k >> 1) & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < kKeyChunks; ++c) {
                const uint64_t ad = q_desc + (rows * kKeyChunks + c) * (kChunk >> 4);
                const uint64_t bd =
                    k_desc + (turns ? ((turn_keys(base, k) - ring) >> 4) + c * (kChunk >> 4)
                                    : ((k * kTileChunks + c) % kStages) * (kChunk >> 4));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)   // a step of 16 columns: 32 bytes
                  mma_f16_ss(tmem + kTmemS + 128 * q, ad + 2 * kk, bd + 2 * kk, idesc_s,
                             c > 0 || kk > 0 ? 1u : 0u);
              }
              mma_commit(ctx.bar(B_SFULL + q));
              if (turns || q == 1 || j + 1 >= n1) {   // the last stream to use the tile
                mma_commit(ctx.bar(B_KFREE + (k & 1)));
                if (t + 1 == it.tiles) mma_commit(ctx.bar(B_QFREE));
              }
            }
          }
        n += it.tiles;
      }
      mma_commit(ctx.bar(B_FINAL));
      drain(ctx, ctx.bar(B_FINAL), 0);
      ctx.step(kStepsDone);
      mbar_arrive(ctx.bar(B_DONE));
    }
    __syncwarp();
  } else if (warp == kTailWarp) {
    // Zeroes the values behind a sequence's last key in its last tile, in both
    // 64-column blocks of both halves: a masked probability is 0, and 0 x (inf
    // or NaN) is not. The MMA thread says when they have landed (this warp does
    // not follow the ring, and could not tell its phases apart).
    uint32_t n = 0, tails = 0;
    for (int i = i0; i < i1; ++i) {
      const Item it = load_item<kTurns>(a, items + i);
      if (!it.ok || it.tiles == 0) {
        if (lane == 0) ctx.pass_item();
        continue;
      }
      const int t = it.tiles - 1;
      if (it.tail(t)) {
        if (!wait_warp(ctx, ctx.bar(B_LANDED), tails++ & 1)) break;
        for (int j = 0; j < 2; ++j) {
          const uint32_t k = n + t;
          const uint32_t d =
              it.turns ? turn_values(base, k) + j * kChunk
                       : ring + ((k * kTileChunks + kKeyChunks + j) % kStages) * kChunk;
          const int left = it.k_len - (it.tile_begin + t) * kPrefillKeys - 64 * j;
          for (int e = min(max(left, 0), 64) * 8 + lane; e < 512; e += 32) {
            sts128(d + 16 * e, make_uint4(0, 0, 0, 0));
            sts128(d + kChunk / 2 + 16 * e, make_uint4(0, 0, 0, 0));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && !(a.suppress_tail && tails == 1)) mbar_arrive(ctx.bar(B_TAIL));
      }
      n += it.tiles;
    }
    if (lane == 0) mbar_arrive(ctx.bar(B_DONE));
  } else if (warp == kWatchWarp) {
    if (lane == 0) watch(ctx, ctx.bar(B_DONE));
  } else if (warp >= 4) {
    regs_inc<kSoftmaxRegs>();
    // softmax and epilogue: thread = query row of the stream
    const int q = (warp >> 2) - 1;
    const int lrow = (warp & 3) * 32 + lane;                // of the stream
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + lane_off + kTmemS + 128 * q;
    const uint32_t tm_o = tmem + lane_off + kTmemO + 128 * q;
    const float c = a.scale_log2;
    float2 *const swap = reinterpret_cast<float2 *>(smem + kOffSwap);
    uint32_t ns = 0, no[2] = {0, 0}, nx = 0;
    bool ok = true, unread = false;
    for (int i = i0; i < i1 && ok; ++i) {
      const Item it = load_item<kTurns>(a, items + i);
      if ((!it.ok || it.count[q] == 0) && lane == 0) ctx.pass_item();
      if (!it.ok) continue;
      const int row = lrow + (kTurns && it.turns ? 0 : 128 * q);   // of the item
      const bool has = row < it.q_rows;
      const int lim = has ? min(it.k_len, it.lim0 + (a.causal ? row : 0)) : 0;
      float m_ref = -INFINITY, sum = 0.f;
      auto zero_weights = [&](int col) {
        const uint32_t p[16] = {};
        tmem_st16(tm_s + col, p);
        tmem_st16(tm_s + col + 16, p);
      };
      // One tile; `rem` of its columns are seen by this row.
      auto tile = [&](bool first, int rem) {
        uint32_t r[4][32];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) tmem_ld32(tm_s + 32 * ch, r[ch]);
        tmem_wait_ld();
        bool half_empty = false;   // no row of the warp's sees the second half's keys
        if (__any_sync(0xffffffffu, rem < kPrefillKeys)) {
          half_empty = !__any_sync(0xffffffffu, rem > 64);
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            const int left = min(max(rem - 32 * ch, 0), 32);
            const uint32_t hide = left == 32 ? 0u : 0xFFFFFFFFu << left;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (hide >> e & 1) r[ch][e] = 0xFF800000u;   // -inf
          }
        }
        float mx4[4];   // four chains of three-input maxima
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          mx4[ch] = max3(u2f(r[ch][0]), u2f(r[ch][1]), u2f(r[ch][2]));
#pragma unroll
          for (int e = 3; e < 31; e += 2) mx4[ch] = max3(mx4[ch], u2f(r[ch][e]), u2f(r[ch][e + 1]));
          mx4[ch] = max3(mx4[ch], u2f(r[ch][31]), u2f(r[ch][31]));
        }
        const float m_new = max3(max3(mx4[0], mx4[1], mx4[2]), mx4[3], mx4[3]) * c;
        // also the first maximum, and NaN
        const bool need = !(m_new <= m_ref + kRescale) && m_new != -INFINITY;
        if (__any_sync(0xffffffffu, need)) {
          const float alpha = need ? ex2(m_ref - m_new) : 1.f;
          // a score of +inf makes the row NaN, as a NaN does
          if (need) m_ref = m_new < INFINITY ? m_new : NAN;
          sum *= alpha;
          if (!first) {
#pragma unroll 1
            for (int ch = 0; ch < 8; ++ch) {
              uint32_t o[16];
              tmem_ld16(tm_o + 16 * ch, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(u2f(o[e]) * alpha);
              tmem_st16(tm_o + 16 * ch, o);
            }
          }
        }
        const float mb = m_ref == -INFINITY ? 0.f : m_ref;
        const uint64_t c2 = pair(c, c), mb2 = pair(-mb, -mb);
        uint64_t part[2] = {0, 0};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half == 1 && half_empty) {
            // (a test per 16 keys instead of 64 keeps the exponentials of full tiles
            // apart: 8 % slower there)
            zero_weights(32);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t p[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t *x = r[2 * half + k / 2] + 16 * (k % 2) + 2 * e;
                const uint64_t x2 = fma2(pair(u2f(x[0]), u2f(x[1])), c2, mb2);
                float y0, y1;
                unpair(x2, y0, y1);
                y0 = ex2(y0);
                y1 = ex2(y1);
                part[e % 2] = add2(part[e % 2], pair(y0, y1));
                p[e] = cvt_bf16x2(y0, y1);
              }
              tmem_st8(tm_s + 32 * half + 8 * k, p);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ctx.bar(B_PFULL + 2 * q + half));
        }
        float s0, s1;
        unpair(add2(part[0], part[1]), s0, s1);
        sum += s0 + s1;
      };
      const bool none = !__any_sync(0xffffffffu, has);
      for (int t = 0; t < it.count[q]; ++t) {
        ok = wait_warp(ctx, ctx.bar(B_SFULL + q), ns++ & 1);
        if (!ok) break;
        if (kTurns && unread) {
          // the other stream's warps still read the last item's outputs
          unread = false;
          ok = wait_warp(ctx, ctx.bar(B_SWAP), nx++ & 1);
          if (!ok) break;
        }
        if (none) {   // no row of the warp's is stored: any weights will do
          if (lane < 2) mbar_arrive(ctx.bar(B_PFULL + 2 * q + lane));
          continue;
        }
        tc_fence_after();
        const int rem =
            lim - (it.tile_begin + (kTurns && it.turns ? 2 * t + q : t)) * kPrefillKeys;
        tile(t == 0, rem);
      }
      if (!ok) break;
      const size_t out_row = (size_t)it.q_row + row;
      if (kTurns && it.turns) {
        // Both streams hold a part of the same rows: each stores 64 columns.
        swap[128 * q + lrow] = make_float2(m_ref, sum);
        __syncwarp();
        if (lane == 0) mbar_arrive(ctx.bar(B_SWAP));
        ok = wait_warp(ctx, ctx.bar(B_SWAP), nx++ & 1);
        for (int k = 0; k < 2 && ok; ++k) ok = wait_warp(ctx, ctx.bar(B_OFULL + k), no[k]++ & 1);
        if (!ok) break;
        tc_fence_after();
        const float2 other = swap[128 * (q ^ 1) + lrow];
        const float m = max3(m_ref, other.x, other.x);
        const float w_own = m_ref == -INFINITY ? 0.f : ex2(m_ref - m);
        const float w_other = other.x == -INFINITY ? 0.f : ex2(other.x - m);
        sum = sum * w_own + other.y * w_other;
        m_ref = m;
        const bool empty = sum == 0.f;
        const float inv = empty ? 0.f : 1.f / sum;
        const float w0 = (q == 0 ? w_own : w_other) * inv, w1 = (q == 0 ? w_other : w_own) * inv;
        const uint32_t tm_a = tmem + lane_off + kTmemO + 64 * q;   // stream 0's output
#pragma unroll 1
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t x[32], y[32];
          tmem_ld32(tm_a + 32 * ch, x);
          tmem_ld32(tm_a + 128 + 32 * ch, y);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            x[e] = empty ? 0u : __float_as_uint(u2f(x[e]) * w0 + u2f(y[e]) * w1);
          if (has) store32(a, it.slot, row, out_row, it.h, 64 * q + 32 * ch, x, 1.f);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ctx.bar(B_SWAP));
        unread = true;
      } else {
        const bool any = it.count[q] > 0;
        if (kTurns && it.count[q ^ 1] > 0) ++no[q ^ 1];
        if (any) {
          ok = wait_warp(ctx, ctx.bar(B_OFULL + q), no[q]++ & 1);
          if (!ok) break;
          tc_fence_after();
        }
        // a row that saw nothing: zeros, whatever the accumulator holds
        const bool empty = sum == 0.f;
        const float inv = empty ? 0.f : 1.f / sum;
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t r[32];
          if (any) {
            tmem_ld32(tm_o + 32 * ch, r);
            tmem_wait_ld();
          }
          if (!any || empty) {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0;
          }
          if (has) store32(a, it.slot, row, out_row, it.h, 32 * ch, r, inv);
        }
        tc_fence_before();
      }
      if (has && !(kTurns && it.turns && q == 1)) {
        const float lse = sum == 0.f ? -INFINITY : (m_ref + log2f(sum)) * 0.6931471805599453f;
        if (it.slot >= 0)
          a.ws_lse[it.slot + row] = lse;
        else if (a.lse != nullptr)
          a.lse[out_row * a.n_h + it.h] = lse;
      }
    }
    if (lane == 0) mbar_arrive(ctx.bar(B_DONE));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// One warp merges the parts of one row: o = sum_p w_p o_p / sum_p w_p with
// w_p = exp(lse_p - max). A part that saw no key has lse = -inf and weight 0.
// Bound by latency: the chain is item, then all lse of the row (a lane each) with
// its first eight partial rows, store.
constexpr int kMergeWarps = 4, kMergeAhead = 8;

__global__ void __launch_bounds__(32 * kMergeWarps) prefill_combine_kernel(const Args a) {
  const int4 *p = reinterpret_cast<const int4 *>(a.combine + blockIdx.x);
  const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int4 x = __ldg(p);
  const int parts = __ldg(reinterpret_cast<const int *>(p + 1));
  const int q_row = x.x, q_rows = x.y, h = x.z, first = x.w;
  // Launched while the attention still runs (the plan is older): its results are
  // there from here on, and are not read as constants of this launch.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= q_rows) return;
  if (q_row < 0 || q_row > a.T_q - q_rows || h < 0 || h >= a.n_h || first < 0 || parts < 1 ||
      (long long)first + (long long)parts * q_rows > a.num_partials) {
    if (lane == 0) report(a.status, MLA_DEV_BAD_PLAN);
    return;
  }
  const float *lse = a.ws_lse + first + row;
  const float4 *o = reinterpret_cast<const float4 *>(a.ws_o + (size_t)(first + row) * 128) + lane;
  const size_t step = (size_t)q_rows * 32;   // float4s from part to part
  float m = -INFINITY, total = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, const float4 &v) {
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  };
  for (int k0 = 0; k0 < parts; k0 += 32) {
    const int n = min(32, parts - k0);
    const float l = lane < n ? __ldcg(lse + (size_t)(k0 + lane) * q_rows) : -INFINITY;
    float4 v[kMergeAhead];
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k)
      if (k < n) v[k] = __ldcg(o + (size_t)(k0 + k) * step);
    float top = l;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    top = fmaxf(top, m);
    const float mb = top == -INFINITY ? 0.f : top;
    const float keep = expf(m - mb);   // of the parts so far: 0 before the first
    acc.x *= keep;
    acc.y *= keep;
    acc.z *= keep;
    acc.w *= keep;
    const float w = expf(l - mb);
    float sum = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    total = total * keep + sum;
    m = top;
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k)
      if (k < n) add(__shfl_sync(0xffffffffu, w, k), v[k]);
#pragma unroll 8
    for (int k = kMergeAhead; k < n; ++k)
      add(__shfl_sync(0xffffffffu, w, k), __ldcg(o + (size_t)(k0 + k) * step));
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  uint16_t *dst = a.o + (long long)(q_row + row) * a.ld_o + (long long)h * a.hs_o + 4 * lane;
  *reinterpret_cast<uint2 *>(dst) = make_uint2(cvt_bf16x2(acc.x * inv, acc.y * inv),
                                               cvt_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0 && a.lse != nullptr)
    a.lse[(size_t)(q_row + row) * a.n_h + h] = total == 0.f ? -INFINITY : m + logf(total);
}

}  // namespace

// failure-detection switch (mla_debug_prefill_wait)
static uint64_t g_wait_ns = 1000000000ull;
static int g_suppress_tail = 0;

mla_status_t set_prefill_wait(double seconds, int suppress_arrive) {
  if (!(seconds > 0.0 && seconds <= 10.0))
    return fail(MLA_ERR_INVALID_ARGUMENT, "wait cap %g s outside (0, 10]", seconds);
  g_wait_ns = (uint64_t)(seconds * 1e9);
  g_suppress_tail = suppress_arrive ? 1 : 0;
  return MLA_OK;
}

mla_status_t launch_prefill(const PrefillArgs &p, cudaStream_t stream) {
  const PrefillHeader *ph = p.plan_host;
  CUtensorMap qn, qp, kn, v, kp;
  // no keys at all: the maps of the keys are not read, but have to be valid
  const bool keys = p.T_k > 0;
  const uint64_t tk = keys ? p.T_k : 1;
  mla_status_t st = make_map3(&qn, p.q_nope, MLA_D_NOPE, p.T_q, p.n_h, p.ld_qn, p.hs_qn, 128);
  if (st == MLA_OK) st = make_map3(&qp, p.q_pe, MLA_D_R, p.T_q, p.n_h, p.ld_qp, p.hs_qp, 128);
  if (st == MLA_OK)
    st = make_map3(&kn, keys ? p.k_nope : p.q_nope, MLA_D_NOPE, tk, p.n_h, p.ld_kn, p.hs_kn, 128);
  if (st == MLA_OK)
    st = make_map3(&v, keys ? p.v : p.q_nope, MLA_D_V, tk, p.n_h, p.ld_v, p.hs_v, 64);
  if (st == MLA_OK)
    st = make_map3(&kp, keys ? p.k_pe : p.q_pe, MLA_D_R, tk, 1, p.ld_kp, p.ld_kp, 128);
  if (st != MLA_OK) return st;
  Args a;
  a.cta_begin = reinterpret_cast<const int32_t *>(p.plan_dev + ph->cta_off);
  a.items = reinterpret_cast<const PrefillItem *>(p.plan_dev + ph->items_off);
  a.combine = reinterpret_cast<const PrefillCombine *>(p.plan_dev + ph->combine_off);
  a.num_items = ph->num_items;
  a.T_q = p.T_q;
  a.T_k = p.T_k;
  a.n_h = p.n_h;
  a.causal = ph->causal;
  a.num_partials = ph->num_partials;
  a.scale_log2 = p.scale_log2;
  a.ws_o = p.ws_o;
  a.ws_lse = p.ws_lse;
  a.o = p.o;
  a.ld_o = p.ld_o;
  a.sectors = reinterpret_cast<uintptr_t>(p.o) % 32 == 0 && p.ld_o % 16 == 0 &&
              p.hs_o % 16 == 0 && reinterpret_cast<uintptr_t>(p.ws_o) % 32 == 0;
  a.hs_o = p.hs_o;
  a.lse = p.lse;
  a.status = p.status;
  a.wait_ns = g_wait_ns;
  a.suppress_tail = g_suppress_tail;
  auto kernel = ph->turns ? prefill_kernel<true> : prefill_kernel<false>;
  MLA_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kSmemBytes));
  kernel<<<ph->num_ctas, kThreads, kSmemBytes, stream>>>(qn, qp, kn, v, kp, a);
  MLA_LAUNCH_CHECK("prefill_kernel");
  if (ph->num_combine > 0) {
    // (programmatic launch: the merge's launch latency hides behind the attention,
    // 2 us of 52 with 17 queries over 20028 keys)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ph->num_combine, (ph->max_merge_rows + kMergeWarps - 1) / kMergeWarps);
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    MLA_CUDA_TRY(cudaLaunchKernelEx(&cfg, prefill_combine_kernel, a));
    MLA_LAUNCH_CHECK("prefill_combine_kernel");
  }
  return MLA_OK;
}

}  // namespace mla
