// Matrix product on tcgen05 tensor cores for the layer's linear maps
// (linear.cu): D[M][N] (+)= sum_k A(m, k) B(n, k), bf16 operands, fp32
// accumulators in TMEM, persistent over output tiles.
//
// Tile: 128 rows of A per CTA.  CG = 2 pairs two CTAs on one 256-row tile
// (cta_group::2): each loads its own 128 rows of A and half of B's BN columns,
// so a CTA fetches (128 + BN/2) operand rows for 128 x BN products; CG = 1
// serves the small outputs, which need more and smaller tiles to fill the SMs.
//
// Operand majors: an operand is either K-major (its k runs along memory rows:
// X and W of the forward, dZ of dX = dZ W) or MN-major (its k is the row index:
// W of dX, dZ and X of dW = dZ^T X).  Both are plain 2-D TMA boxes of 128-byte
// swizzled rows: K-major [rows][64 k], MN-major [64 k][64 mn] per 64 columns.
//
// B8: operand B (MN-major) is an 8-bit checkpoint (ckpt8.cu).  TMA brings the
// codes, two teams of warps turn them into bf16 (exact: 8-bit integer times a
// power of two) in the swizzled layout the tensor cores read.
//
// SUM: the tensor cores add into their fp32 accumulator with truncation, an
// error toward zero that grows with the length of the chain (measured a stage of
// 64 tokens: 7e-8 of the norm for sums of random signs, 3.5e-7 for sums of one
// sign).  An fp32 output therefore takes chains of kChain stages only, and a bf16
// weight gradient none above kLongChain; the epilogue warps add each to rounded
// fp32 sums in registers, while the next chain runs in the other accumulator.
//
// Roles (warps): 0 TMA producer, 1 MMA issuer (CTA 0 of a pair), 2 TMEM owner,
// 3 producer of the codes (B8) or the bias gradient's last step, from 4 on the
// epilogue (two accumulators in TMEM alternate, so the epilogue of one tile runs
// under the products of the next), then the converters of B8.
//
// What bounds it: a 256 x 256 pair tile takes 512 clocks of the tensor pipe a
// stage and 32 KB into each CTA's shared memory, 64 bytes a clock, the most an SM
// takes in from L2; measured, 0.40 us a stage.  In long runs the clock falls to
// 1.3-1.6 GHz under the power cap.  92160 x 1024 x 1024 without epilogue work: 144
// us, 1340 TFLOP/s (cuBLAS 138); with bias and residual 161, with bias and gelu
// 156; 92160 x 4096 x 1024 (dX): 508 us, 1520 TFLOP/s.  The sixth stage, in place
// of a second staging buffer per warp, gave 3%; 128-column tiles run at half the
// rate.
#pragma once

#include "ckpt8.cuh"
#include "common.cuh"
#include "internal.h"

namespace prism {
namespace gemm {

constexpr int BK = 64;  // contraction per stage: one 128-byte swizzle row of bf16
constexpr int kStageBuf = 4096;  // an epilogue warp's staging buffer: 32 rows x 128 bytes
// Converters: two teams of four warps, which take the stages in turn (one team of
// eight: 757 us at 92160 x 1024 x 4096, two of four 705, four of two 705).
constexpr int kConvTeams = 2;
constexpr int kConvTeam = 4;
constexpr int kChain = 8;  // stages per accumulator chain of fp32 outputs: 5e-7 of the norm, 4% of the time
// ... of bf16 weight gradients, whose tokens have no bound (the other products' have:
// 1024 stages, 3.5e-4 where a sum keeps its sign, against a rounding of up to 3.9e-3).
// One chain over 860160 tokens was 5e-3 short on such sums; this length costs nothing
// that could be measured.
constexpr int kLongChain = 512;

enum { SUM_NONE = 0, SUM_FP32 = 1, SUM_BF16 = 2 };  // by the output's type

template <int CG_, int BN_, bool A_MN_, bool B_MN_, bool B8_ = false, int SUM_ = SUM_NONE, int EW_ = 8>
struct Cfg {
  static constexpr int CG = CG_, BN = BN_;
  static constexpr bool A_MN = A_MN_, B_MN = B_MN_, B8 = B8_, SUM = SUM_ != SUM_NONE;
  static constexpr bool SUM16 = SUM_ == SUM_BF16;
  static constexpr int CHAIN = SUM16 ? kLongChain : kChain;
  static constexpr int BM = 128 * CG;
  static constexpr int BNC = BN / CG;  // columns of B a CTA loads
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_BYTES = BNC * BK * 2;
  static constexpr int Q_BYTES = B8 ? BNC * BK : 0;  // codes of the stage's B
  // rings of operand stages: A with B; with B8 three of their own, so that the
  // codes arrive and are converted well ahead of the products
  static constexpr int STAGE = B8 ? A_BYTES : A_BYTES + B_BYTES;
  // Epilogue warps: 8, which leave room for a sixth stage; or 16, one 64-column
  // chunk each of 256 columns, which hide one another's latencies and the
  // exponentials' (wide_epilogue in linear.cu says when).
  static constexpr int EW = EW_;
  // 128-column tiles stage a saved pre-activation in a buffer of its own; the others
  // have no room for one and take a second pass over the accumulator
  static constexpr int NBUF = BN == 128 ? 2 : 1;
  static constexpr int EPI = EW * NBUF * kStageBuf;
  static constexpr int NST_FIT = (232448 - 2048 - EPI) / STAGE;
  static constexpr int NST = B8 ? 5 : NST_FIT < 6 ? NST_FIT : 6;
  static constexpr int NB = B8 ? 4 : NST;
  static constexpr int NQ = 5;
  static constexpr int OFF_B = B8 ? NST * STAGE : A_BYTES;
  static constexpr int B_PITCH = B8 ? B_BYTES : STAGE;
  static constexpr int OFF_Q = NST * STAGE + NB * B_BYTES;
  static constexpr int OFF_EPI = B8 ? OFF_Q + NQ * Q_BYTES : NST * STAGE;
  static constexpr int OFF_BAR = OFF_EPI + EPI;
  static constexpr int OFF_SC = OFF_BAR + 1024;        // B8: scale words of the codes' stages, one per token
  static constexpr int SMEM = OFF_SC + (B8 ? NQ * BK * 4 : 0) + 1024;  // slack to align the base to 1024
  static constexpr int THREADS = 128 + 32 * EW + (B8 ? 32 * kConvTeams * kConvTeam : 0);
  static constexpr bool REGS = THREADS == 640;  // registers move between warpgroups
  static_assert(SMEM <= 232448, "shared memory");
  static constexpr int TMEM_COLS = 2 * BN;
  static_assert(EW == 8 || (EW == 16 && BN == 256 && !B8 && !SUM), "epilogue warps");
  static_assert(BN / 64 % (EW / 4) == 0, "each four epilogue warps own whole 64-column chunks");
  static_assert(!B8 || (B_MN && BNC == 128), "the checkpoint operand comes in 128-channel columns");
};

struct Bars {
  uint64_t full[6], empty[6];          // operand stages: filled (CTA 0's), consumed (each CTA's own)
  uint64_t bfull[6], bempty[6];        // B8: B converted (CTA 0's), consumed (each CTA's own)
  uint64_t qfull[6], qempty[6];        // B8: codes arrived, converted (each CTA's own)
  uint64_t acc_full[2], acc_empty[2];  // accumulators: complete (each CTA's own), read (CTA 0's)
  uint64_t res[16];                    // residual tiles of each epilogue warp
  uint64_t drain;                      // single use, after an abort
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 1024, "barrier space");

// How the output tiles are dealt out to `groups` CTA groups.  Without a split
// every tile is one segment over the whole contraction.  With one, whole waves
// of tiles run unsplit, and the last, partial wave of `rem` tiles is divided
// so that every group gets the same share: group g < rem walks tile g's first
// `km` stages (in step with its neighbours, which read the same tokens), and
// the other groups share the rest of those tiles.  Partial sums go to fp32
// slots: tile g's first part to slot g, helper h's part of tile t to slot
// rem + h + t (helper and tile both only grow along the walk, so the sum is
// unique).  Nothing depends on the order in which groups finish.
struct Sched {
  int tiles, tiles_n, kc, groups;
  int full;  // unsplit tiles (dealt round robin)
  int rem;   // tiles of the split remainder
  int km;    // stages of their first parts
};
struct Seg {
  int tile, k0, k1, slot;  // slot < 0: the segment is the whole tile
};
__host__ __device__ inline long long helper_start(const Sched &s, int h) {
  return (long long)s.rem * (s.kc - s.km) * h / (s.groups - s.rem);
}
struct SegIter {
  int next_tile;
  bool split_done;
  long long pos, end;
  int h;
  __device__ __forceinline__ SegIter(const Sched &s, int g) : next_tile(g), split_done(s.rem == 0), pos(0), end(0), h(-1) {
    if (s.rem && g >= s.rem) {
      h = g - s.rem;
      pos = helper_start(s, h);
      end = helper_start(s, h + 1);
    }
  }
  __device__ __forceinline__ bool next(const Sched &s, Seg &o) {
    if (next_tile < s.full) {
      o = Seg{next_tile, 0, s.kc, -1};
      next_tile += s.groups;
      return true;
    }
    if (split_done) return false;
    if (h < 0) {
      const int r = next_tile % s.groups;  // this group's own index, < rem
      o = Seg{s.full + r, 0, s.km, r};
      split_done = true;
      return true;
    }
    if (pos >= end) return false;
    const int tail = s.kc - s.km;
    const int t = (int)(pos / tail);
    const long long stop = min(end, (long long)(t + 1) * tail);
    o = Seg{s.full + t, s.km + (int)(pos - (long long)t * tail), s.km + (int)(stop - (long long)t * tail),
            s.rem + h + t};
    pos = stop;
    return true;
  }
};

struct Args {
  Sched s;
  int rows, cols;  // extent of the output
  // epilogue
  const uint16_t *bias;  // bf16 [cols] or NULL
  int act;
  int has_res;    // add the residual tile (mapR)
  int save_z;     // 0 none, 1 bf16 (mapZ), 2 checkpoint (codes, scales)
  int8_t *codes;
  uint8_t *scales;
  long long ldq;  // checkpoint row length (multiple of 128)
  // checkpoint operand B8
  const uint8_t *b_scales;  // [k][b_ld / 32]
  long long b_ld;
  int k_total;
  int *status;
  int reset;  // the call's first kernel: clear the status word
  // split_kernel stores without tensor maps
  const uint16_t *R;
  long long ldr;
  void *Y;
  long long ldy;
  uint16_t *Z;
  int out_fp32;
  // the bias gradient's last step, by an idle warp: db = sums of `bias_blocks`
  // rows of bias_part (db NULL: not asked of this launch)
  const float *bias_part;
  int bias_blocks, bias_cols;
  void *db;
  int db_fp32;
};
// The status word starts at 0 with the call's first kernel: cleared by its first
// block, seconds before the shortest wait of any block can run out.
__device__ __forceinline__ void reset_status(int *status, int reset) {
  if (reset && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) status[0] = status[1] = 0;
}

// db[c] = sum of part[0 .. blocks)[c], 32 columns a warp, in a fixed order: four
// running sums of every fourth row, the odd rows on the first
__device__ __forceinline__ void finish_bias(const float *part, int blocks, int cols, void *db, int fp32, int first, int step,
                                            int lane) {
  for (int c = first * 32 + lane; c < cols; c += step * 32) {
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    int b = 0;
#pragma unroll 4
    for (; b + 4 <= blocks; b += 4)
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] += part[(long long)(b + k) * cols + c];
    for (; b < blocks; ++b) a[0] += part[(long long)b * cols + c];
    const float s = (a[0] + a[1]) + (a[2] + a[3]);
    if (fp32)
      static_cast<float *>(db)[c] = s;
    else
      static_cast<uint16_t *>(db)[c] = (uint16_t)(pack_bf16(s, s) & 0xffffu);
  }
}

// ---------------------------------------------------------------------------
// cluster helpers
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the same shared-memory location in another CTA of the cluster
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, int cta) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}
__device__ __forceinline__ uint32_t map_to_cta0(const void *p) { return map_to_cta(smem_u32(p), 0); }
__device__ __forceinline__ float4 load_cta(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
// Arrive on CTA 0's barrier.  What it publishes is not read through the generic
// proxy by CTA 0: accumulators have been read (tcgen05.wait::ld), or this CTA's
// own shared memory has been written and fenced for the tensor cores that read it
// here.  So the arrival carries no cluster-scope release, which would wait for
// every outstanding memory operation (measured: 1.5 us a stage in the converters).
template <int CG>
__device__ __forceinline__ void arrive_cta0(uint64_t *bar) {
  if constexpr (CG == 1) {
    mbar_arrive(bar);
  } else {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_to_cta0(bar)) : "memory");
  }
}
// TMA load into this CTA's shared memory, counted on CTA 0's barrier
template <int CG>
__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y) {
  if constexpr (CG == 1) {
    tma_load_2d(dst, map, bar, x, y);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
        "%4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(map_to_cta0(bar)), "r"(x), "r"(y)
        : "memory");
  }
}
__device__ __forceinline__ void store_2d(const CUtensorMap *map, const void *src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 1) {
    mma_ss(d, a, b, idesc, acc);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  }
}
// arrive on `bar` in every CTA of the group once this thread's products are done
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if constexpr (CG == 1) {
    mma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_alloc_g(uint32_t *dst, uint32_t ncols) {
  if constexpr (CG == 1) {
    tmem_alloc(dst, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_g(uint32_t t, uint32_t ncols) {
  if constexpr (CG == 1)
    tmem_dealloc(t, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// four bytes global -> shared without a register in between (zeros unless `in`)
__device__ __forceinline__ void copy4_async(void *dst, const void *src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// arrive on `bar` once this thread's copies so far have landed
__device__ __forceinline__ void copy_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---------------------------------------------------------------------------
// activations of a pair (fp32).  gelu is the tanh form, z / (1 + e^-v) with
// v = 2 sqrt(2/pi) (z + 0.044715 z^3); silu is the same with v = z.
// ---------------------------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + 2^w)
__device__ __forceinline__ float2 logistic2(float2 w) {
  const float2 d = fadd2(make_float2(ex2f(w.x), ex2f(w.y)), make_float2(1.f, 1.f));
  return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
template <int ACT>
__device__ __forceinline__ float2 act_value(float2 z) {
  if constexpr (ACT == PRISM_ACT_RELU)
    return make_float2(z.x > 0.f ? z.x : (z.x != z.x ? z.x : 0.f), z.y > 0.f ? z.y : (z.y != z.y ? z.y : 0.f));
  if constexpr (ACT == PRISM_ACT_SILU) return fmul2(z, logistic2(fmul2(z, make_float2(-kLog2e, -kLog2e))));
  if constexpr (ACT == PRISM_ACT_GELU)
    return fmul2(z, logistic2(fmul2(z, ffma2(fmul2(z, z), -0.044715f * kGelu2 * kLog2e, -kGelu2 * kLog2e))));
  return z;
}

// ---------------------------------------------------------------------------
// epilogues
// ---------------------------------------------------------------------------
template <int ACT>
__device__ __forceinline__ void act32(float2 (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = act_value<ACT>(v[i]);
}
__device__ __forceinline__ float2 bf16_pair(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }
// eight values of v from index i, rounded
__device__ __forceinline__ uint4 pack8(const float2 (&v)[16], int i) {
  return make_uint4(pack_bf16(v[i].x, v[i].y), pack_bf16(v[i + 1].x, v[i + 1].y), pack_bf16(v[i + 2].x, v[i + 2].y),
                    pack_bf16(v[i + 3].x, v[i + 3].y));
}

// The bias of a warp's 64 columns, four to a lane of the first sixteen, loaded while the
// products still run; add_bias hands a group of 32 columns round by shuffles.
__device__ __forceinline__ uint2 load_bias(const uint16_t *bias, int c0, int lane, int cols) {
  const int c = c0 + lane * 4;
  return bias && c < cols ? __ldg(reinterpret_cast<const uint2 *>(bias + c)) : make_uint2(0, 0);
}
__device__ __forceinline__ void add_bias(float2 (&v)[16], const uint2 &b, int group) {
#pragma unroll
  for (int p = 0; p < 16; ++p)
    v[p] = fadd2(v[p], bf16_pair(__shfl_sync(0xffffffffu, p & 1 ? b.y : b.x, group * 8 + (p >> 1))));
}
__device__ __forceinline__ void apply_act(float2 (&v)[16], int act) {
  switch (act) {
    case PRISM_ACT_RELU:
      act32<PRISM_ACT_RELU>(v);
      break;
    case PRISM_ACT_SILU:
      act32<PRISM_ACT_SILU>(v);
      break;
    case PRISM_ACT_GELU:
      act32<PRISM_ACT_GELU>(v);
      break;
    default:
      break;
  }
}
// one warp's 32 x 32 fp32 values (thread = row) through a staging buffer to
// column x, row y of `map`
__device__ __forceinline__ void stage_fp32(const CUtensorMap *map, uint8_t *buf, const uint32_t (&v)[32], int lane, int x,
                                           int y, bool store) {
  uint8_t *row = buf + lane * 128;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4 *>(row + ((i ^ (lane & 7)) << 4)) =
        make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (store) store_2d(map, buf, x, y);
    store_commit();
  }
}

// A tile of D straight from its accumulator: bias, saved pre-activation,
// activation and residual, rounded to bf16; or fp32 partial sums of a split
// tile.  Each warp owns 32 rows of one 64-column chunk, or of two one after the
// other, and a 4 KB staging buffer, 128-byte swizzled as the tensor maps are: it
// receives the chunk's residual by TMA while the products run, then the result,
// then feeds the TMA store.  A saved pre-activation has a second buffer, or goes
// through the first one before, in a pass of its own over the accumulator.
template <class C>
__device__ __forceinline__ void epilogue_tile(const CUtensorMap &mapY, const CUtensorMap &mapR, const CUtensorMap &mapZ,
                                              const Args &args, Bars &bar, uint8_t *staging, uint32_t tmem, int group,
                                              int rank, int warp, int lane) {
  constexpr int CG = C::CG;
  const Sched &s = args.s;
  int *status = args.status;
  const int ew = warp - 4, q4 = warp & 3;
  uint8_t *buf = staging + ew * C::NBUF * kStageBuf;
  uint8_t *row = buf + lane * 128;
  uint8_t *zbuf = buf + (C::NBUF - 1) * kStageBuf;
  const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
  const int sw = lane & 7;
  SegIter it(s, group);
  Seg sg;
  int t = 0;
  uint32_t res_phase = 0;
  bool ok = true;
  for (; ok && it.next(s, sg); ++t) {
    const int ab = t & 1;
    const int m0 = (sg.tile / s.tiles_n) * C::BM + rank * 128 + q4 * 32;
    const bool parts = sg.slot >= 0;
    const bool rows_in = m0 < args.rows;
    bool res_pending = false;
    // the buffer's last store has been read
    const auto free_buffer = [&] {
      if (lane == 0) store_wait_read<0>();
      __syncwarp();
    };
    const auto load_res = [&](int col0) {
      if (!(args.has_res && rows_in && col0 < args.cols)) return;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar.res[ew], kStageBuf);
        tma_load_2d(buf, &mapR, &bar.res[ew], col0, m0);
      }
      res_pending = true;
    };
    const int n0 = (sg.tile % s.tiles_n) * C::BN;
    const int c_first = ew >> 2;
    // this warp's chunks: known here, so that a single one costs no loop (0.15 us a tile)
    constexpr int CHUNKS = C::BN / 16 / C::EW, CHUNK_STEP = C::EW / 4;
    if (!parts && args.has_res) {
      free_buffer();
      if (C::NBUF == 2 || !args.save_z) load_res(n0 + c_first * 64);
    }
    uint2 bias = load_bias(args.bias, n0 + c_first * 64, lane, min(args.cols, n0 + c_first * 64 + 64));
    ok = __all_sync(0xffffffffu, mbar_wait(&bar.acc_full[ab], (t >> 1) & 1, status, 407));
    if (ok) {
      tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < CHUNKS; ++i) {
        const int c = c_first + i * CHUNK_STEP;
        const int col0 = n0 + c * 64;
        const uint32_t acc = tmem + ab * C::BN + c * 64 + lane_off;
        if (parts) {
#pragma unroll 1
          for (int g = 0; g < 2; ++g) {
            uint32_t v[32];
            tmem_ld32(acc + g * 32, v);
            tmem_wait_ld();
            free_buffer();
            stage_fp32(&mapZ, buf, v, lane, c * 64 + g * 32, sg.slot * C::BM + rank * 128 + q4 * 32, true);
          }
          continue;
        }
        // nothing of this chunk exists, nor of those to its right
        if (!rows_in || col0 >= (args.save_z == 2 ? (int)args.ldq : args.cols)) break;
        const bool in = col0 < args.cols;  // not: the padding of a checkpoint's rows
        if (i == 0 && !args.has_res) free_buffer();
        // 32 columns of the pre-activation
        const auto pre = [&](int g, float2 (&v)[16]) {
          uint32_t u[32];
          tmem_ld32(acc + g * 32, u);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
          if (args.bias) add_bias(v, bias, g);
        };
        uint32_t scale2 = 0;
        // 32 columns of Z into its staging buffer
        const auto stage_z = [&](int g, const float2 (&v)[16]) {
          if (args.save_z == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4 *>(zbuf + lane * 128 + (((g * 4 + i) ^ sw) << 4)) = pack8(v, 4 * i);
          } else {
            // 64 bytes a row, 64-byte swizzled
            uint32_t q[8];
            scale2 |= ckpt8_quantise(v, q) << (8 * g);
            uint8_t *qrow = zbuf + lane * 64;
            const int x = (lane >> 1) & 3;
            *reinterpret_cast<uint4 *>(qrow + (((2 * g) ^ x) << 4)) = make_uint4(q[0], q[1], q[2], q[3]);
            *reinterpret_cast<uint4 *>(qrow + (((2 * g + 1) ^ x) << 4)) = make_uint4(q[4], q[5], q[6], q[7]);
          }
        };
        const auto store_z = [&] {  // by lane 0, after the fence
          if (args.save_z == 2 || in) store_2d(&mapZ, zbuf, col0, m0);
        };
        const auto store_scales = [&] {
          if (args.save_z == 2 && m0 + lane < args.rows)
            *reinterpret_cast<uint16_t *>(args.scales + (long long)(m0 + lane) * (args.ldq / 32) + col0 / 32) =
                (uint16_t)scale2;
        };
        if (C::NBUF == 1 && args.save_z) {
#pragma unroll 1
          for (int g = 0; g < 2; ++g) {
            float2 v[16];
            pre(g, v);
            stage_z(g, v);
          }
          store_scales();
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            store_z();
            store_commit();
          }
          free_buffer();
          load_res(col0);
        }
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          float2 v[16];
          pre(g, v);
          if (C::NBUF == 2 && args.save_z) stage_z(g, v);
          if (!in) continue;
          apply_act(v, args.act);
          if (g == 0 && res_pending) {
            ok = __all_sync(0xffffffffu, mbar_wait(&bar.res[ew], res_phase, status, 408));
            res_phase ^= 1;
            res_pending = false;
            if (!ok) break;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 *p = reinterpret_cast<uint4 *>(row + (((g * 4 + i) ^ sw) << 4));
            if (args.has_res) {
              const uint4 r = *p;
              const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) v[4 * i + k] = fadd2(v[4 * i + k], bf16_pair(w[k]));
            }
            *p = pack8(v, 4 * i);
          }
        }
        if (!ok) break;
        if (C::NBUF == 2 && args.save_z) store_scales();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (in) store_2d(&mapY, buf, col0, m0);
          if (C::NBUF == 2 && args.save_z) store_z();
          store_commit();
        }
        if (i + 1 < CHUNKS) {
          const int next = col0 + CHUNK_STEP * 64;
          bias = load_bias(args.bias, next, lane, min(args.cols, next + 64));
          free_buffer();
          if (C::NBUF == 2 || !args.save_z) load_res(next);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cta0<CG>(&bar.acc_empty[ab]);
    }
    if (!ok) {
      bar.abort = 1;
      if (res_pending) mbar_wait(&bar.res[ew], res_phase, status, 409);  // a load that nothing will read
    }
  }
  if (lane == 0) store_wait_read<0>();
}

// SUM: the chains of a segment added up in registers (a thread's row x its
// warp's columns), then written: a whole tile to the output in its type, a
// partial one to its slot in fp32.
template <class C>
__device__ __forceinline__ void epilogue_sum(const CUtensorMap &mapY, const CUtensorMap &mapZ, const Args &args, Bars &bar,
                                             uint8_t *staging, uint32_t tmem, int group, int rank, int warp, int lane) {
  const Sched &s = args.s;
  const int ew = warp - 4, q4 = warp & 3, half = ew >> 2;
  constexpr int COLS = C::BN / (C::EW / 4);  // this warp's columns
  uint8_t *buf = staging + ew * C::NBUF * kStageBuf;
  const uint32_t acc0 = tmem + half * COLS + ((uint32_t)(q4 * 32) << 16);
  SegIter it(s, group);
  Seg sg;
  int t = 0;
  bool ok = true;
  while (ok && it.next(s, sg)) {
    float sum[COLS];
#pragma unroll
    for (int i = 0; i < COLS; ++i) sum[i] = 0.f;
    for (int k0 = sg.k0; k0 < sg.k1; k0 += C::CHAIN, ++t) {
      const int ab = t & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.acc_full[ab], (t >> 1) & 1, args.status, 411));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < COLS / 8; ++g) {
        uint32_t v[8];
        tmem_ld8(acc0 + ab * C::BN + g * 8, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[g * 8 + i] += __uint_as_float(v[i]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cta0<C::CG>(&bar.acc_empty[ab]);
    }
    if (!ok) break;
    const int m0 = (sg.tile / s.tiles_n) * C::BM + rank * 128 + q4 * 32;
    const int n0 = (sg.tile % s.tiles_n) * C::BN + half * COLS;
    if (C::SUM16 && sg.slot < 0) {
      uint8_t *row = buf + lane * 128;
#pragma unroll
      for (int c = 0; c < COLS / 64; ++c) {
        if (lane == 0) store_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float *v = sum + c * 64 + i * 8;
          *reinterpret_cast<uint4 *>(row + ((i ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (m0 < args.rows && n0 + c * 64 < args.cols) store_2d(&mapY, buf, n0 + c * 64, m0);
          store_commit();
        }
      }
      continue;
    }
#pragma unroll
    for (int g = 0; g < COLS / 32; ++g) {
      if (lane == 0) store_wait_read<0>();
      __syncwarp();
      uint32_t v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(sum[g * 32 + i]);
      if (sg.slot >= 0)
        stage_fp32(&mapZ, buf, v, lane, half * COLS + g * 32,
                   sg.slot * C::BM + rank * 128 + q4 * 32, true);
      else
        stage_fp32(&mapY, buf, v, lane, n0 + g * 32, m0,
                   m0 < args.rows && n0 + g * 32 < args.cols);
    }
  }
  if (!ok) bar.abort = 1;
  if (lane == 0) store_wait_read<0>();
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <class C>
__global__ void __cluster_dims__(C::CG, 1, 1) __launch_bounds__(C::THREADS, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                const __grid_constant__ CUtensorMap mapY, const __grid_constant__ CUtensorMap mapR,
                const __grid_constant__ CUtensorMap mapZ, const Args args) {
  constexpr int CG = C::CG, NST = C::NST;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars &bar = *reinterpret_cast<Bars *>(smem + C::OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0u : cta_rank();
  const int group = blockIdx.x / CG;
  const Sched &s = args.s;
  int *status = args.status;
  reset_status(status, args.reset);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
      mbar_init(&bar.bfull[i], kConvTeam * CG);
      mbar_init(&bar.bempty[i], 1);
      mbar_init(&bar.qfull[i], 1 + 32);  // the codes' TMA, and warp 3's scale copies
      mbar_init(&bar.qempty[i], kConvTeam);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.acc_full[i], 1);
      mbar_init(&bar.acc_empty[i], C::EW * CG);
    }
    for (int i = 0; i < C::EW; ++i) mbar_init(&bar.res[i], 1);
    mbar_init(&bar.drain, 1);
    bar.abort = 0;
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc_g<CG>(&bar.tmem_base, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG > 1) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;
  const auto aborted = [&] { return *reinterpret_cast<volatile int *>(&bar.abort) != 0; };
  // 640 threads: the launch gives each of the five warpgroups 96 registers a thread.
  // The epilogue needs more (B8 with SUM: 128 sums), the others less; the totals are
  // the same: 64 + 4 * 104, and with B8 64 + 2 * 144 + 2 * 64 or 64 + 2 * 128 + 2 * 80, 480.
  if constexpr (C::REGS) {
    if (warp < 4) setmaxnreg_dec<64>();
    if (C::B8 && warp >= 4 + C::EW) setmaxnreg_dec<C::SUM ? 64 : 80>();
  }

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      prefetch_tensormap(&mapA);
      prefetch_tensormap(&mapB);
      SegIter it(s, group);
      Seg sg;
      int j = 0;
      bool ok = true;
      while (ok && it.next(s, sg)) {
        const int m0 = (sg.tile / s.tiles_n) * C::BM + (int)rank * 128;
        const int n0 = (sg.tile % s.tiles_n) * C::BN + (int)rank * C::BNC;
        for (int k = sg.k0; k < sg.k1; ++k, ++j) {
          const int st = j % NST;
          if (j >= NST && !(ok = mbar_wait(&bar.empty[st], ((j / NST) - 1) & 1, status, 401))) break;
          if (aborted()) {
            ok = false;
            break;
          }
          uint8_t *a = smem + st * C::STAGE, *b = smem + C::OFF_B + st * C::B_PITCH;
          if (rank == 0) mbar_arrive_expect_tx(&bar.full[st], CG * (C::A_BYTES + (C::B8 ? 0 : C::B_BYTES)));
          if constexpr (C::A_MN) {
            load_2d<CG>(a, &mapA, &bar.full[st], m0, k * BK);
            load_2d<CG>(a + BK * 128, &mapA, &bar.full[st], m0 + 64, k * BK);
          } else {
            load_2d<CG>(a, &mapA, &bar.full[st], k * BK, m0);
          }
          if constexpr (C::B8) {
            // warp 3 brings the codes
          } else if constexpr (C::B_MN) {
#pragma unroll
            for (int c = 0; c < C::BNC; c += 64)
              load_2d<CG>(b + c * BK * 2, &mapB, &bar.full[st], n0 + c, k * BK);
          } else {
            load_2d<CG>(b, &mapB, &bar.full[st], k * BK, n0);
          }
        }
      }
      if (ok) {
        // every stage consumed: no copy is in flight, and the arrivals of the
        // last products on this CTA's barriers have landed
        for (int i = j > NST ? j - NST : 0; i < j; ++i)
          mbar_wait(&bar.empty[i % NST], (i / NST) & 1, status, 402);
      } else {
        // no copy may still be writing when the CTA leaves: CTA 0's barriers
        // count both CTAs' operand loads, and the pair leaves together
        bar.abort = 1;
        if (rank == 0) drain_loads(bar.full, NST, j, status, 403);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_bf16(C::BM, C::BN, C::B_MN ? 1 : 0) | (C::A_MN ? 1u << 15 : 0u);
      SegIter it(s, group);
      Seg sg;
      int j = 0, t = 0;
      bool ok = true;
      while (ok && it.next(s, sg)) {
        for (int k0 = sg.k0; ok && k0 < sg.k1; ++t) {
          const int k1 = C::SUM ? min(k0 + C::CHAIN, sg.k1) : sg.k1;
          const int ab = t & 1;
          if (t >= 2 && !(ok = mbar_wait(&bar.acc_empty[ab], ((t >> 1) - 1) & 1, status, 404))) break;
          tc_fence_after();
          for (int k = k0; k < k1; ++k, ++j) {
            const int st = j % NST;
            if (!(ok = mbar_wait(&bar.full[st], (j / NST) & 1, status, 405))) break;
            tc_fence_after();
            const int sb = j % C::NB;
            if constexpr (C::B8) {
              if (!(ok = mbar_wait(&bar.bfull[sb], (j / C::NB) & 1, status, 412))) break;
              tc_fence_after();
            }
            const uint32_t a = smem_u32(smem + st * C::STAGE), b = smem_u32(smem + C::OFF_B + sb * C::B_PITCH);
            // MN-major: 64-column chunks BK * 128 bytes apart, 8-k groups of 1024 bytes
            const uint64_t da = C::A_MN ? sdesc_sw128(a, BK * 128, 1024) : sdesc_sw128(a, 16, 1024);
            const uint64_t db = C::B_MN ? sdesc_sw128(b, BK * 128, 1024) : sdesc_sw128(b, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma<CG>(tmem + ab * C::BN, da + (C::A_MN ? (uint64_t)kk * 128 : kslice16(kk, 0)),
                      db + (C::B_MN ? (uint64_t)kk * 128 : kslice16(kk, 0)), idesc, (k > k0 || kk > 0) ? 1u : 0u);
            commit<CG>(&bar.empty[st]);
            if constexpr (C::B8) commit<CG>(&bar.bempty[sb]);
          }
          if (ok) commit<CG>(&bar.acc_full[ab]);
          k0 = k1;
        }
      }
      if (!ok) {
        bar.abort = 1;
        if constexpr (CG == 1) {
          mma_drain(&bar.drain, status, 406);
        } else {
          commit<CG>(&bar.drain);
          mbar_wait(&bar.drain, 0, status, 406);
        }
      }
    }
    __syncwarp();
  } else if (C::B8 && warp == 3) {
    // ---------------------------------------------------------------- producer of the codes and scales
    if constexpr (C::B8) {
      if (lane == 0) prefetch_tensormap(&mapB);
      const long long lds = args.b_ld / 32;
      SegIter it(s, group);
      Seg sg;
      int j = 0;
      bool ok = true;
      while (ok && it.next(s, sg)) {
        const int n0 = (sg.tile % s.tiles_n) * C::BN + (int)rank * C::BNC;
        const bool cols_in = n0 < args.b_ld;
        for (int k = sg.k0; k < sg.k1; ++k, ++j) {
          const int sq = j % C::NQ;
          if (j >= C::NQ) ok = mbar_wait(&bar.qempty[sq], ((j / C::NQ) - 1) & 1, status, 413);
          if (!(ok = __all_sync(0xffffffffu, ok && !aborted()))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar.qfull[sq], C::Q_BYTES);
            tma_load_2d(smem + C::OFF_Q + sq * C::Q_BYTES, &mapB, &bar.qfull[sq], n0, k * BK);
          }
          // a token's four scales of these 128 channels are one word
#pragma unroll
          for (int p = 0; p < BK; p += 32) {
            const int tok = k * BK + p + lane;
            const bool in = cols_in && tok < args.k_total;
            copy4_async(smem + C::OFF_SC + (sq * BK + p + lane) * 4,
                        in ? args.b_scales + (long long)tok * lds + (n0 >> 5) : args.b_scales, in);
          }
          copy_async_arrive(&bar.qfull[sq]);
        }
      }
      if (!ok) bar.abort = 1;
      copy_async_wait();
      if (lane == 0) drain_loads(bar.qfull, C::NQ, j, status, 414);
    }
    __syncwarp();
  } else if (warp == 3) {
    if (args.db)
      finish_bias(args.bias_part, args.bias_blocks, args.bias_cols, args.db, args.db_fp32, blockIdx.x, gridDim.x, lane);
  } else if (warp >= 4 && warp < 4 + C::EW) {
    // ---------------------------------------------------------------- epilogue
    if constexpr (C::REGS) setmaxnreg_inc<!C::B8 ? 104 : C::SUM ? 144 : 128>();
    if constexpr (C::SUM)
      epilogue_sum<C>(mapY, mapZ, args, bar, smem + C::OFF_EPI, tmem, group, (int)rank, warp, lane);
    else
      epilogue_tile<C>(mapY, mapR, mapZ, args, bar, smem + C::OFF_EPI, tmem, group, (int)rank, warp, lane);
  } else if (C::B8 && warp >= 4 + C::EW) {
    // ---------------------------------------------------------------- converters of the checkpoint operand
    if constexpr (C::B8) {
      // lane -> 16 channels (lane % 8) of token rows cw * ROWS + pass * 4 + lane / 8
      constexpr int ROWS = BK / kConvTeam, PASS = ROWS / 4;
      const int cw = (warp - 4 - C::EW) % kConvTeam, team = (warp - 4 - C::EW) / kConvTeam;
      const int unit = lane & 7, sub = lane >> 3;
      const int r0 = cw * ROWS + sub;
      SegIter it(s, group);
      Seg sg;
      int j = 0;
      bool ok = true;
      while (ok && it.next(s, sg)) {
        for (int k = sg.k0; k < sg.k1; ++k, ++j) {
          if (j % kConvTeams != team) continue;
          const int sq = j % C::NQ, sb = j % C::NB;
          ok = mbar_wait(&bar.qfull[sq], (j / C::NQ) & 1, status, 410);
          const uint8_t *qs = smem + C::OFF_Q + sq * C::Q_BYTES + r0 * 128 + unit * 16;
          const uint8_t *ss = smem + C::OFF_SC + (sq * BK + r0) * 4 + (unit >> 1);
          uint4 q[PASS];
          uint32_t sc[PASS];
#pragma unroll
          for (int p = 0; p < PASS; ++p) {
            q[p] = *reinterpret_cast<const uint4 *>(qs + p * 512);
            sc[p] = ss[p * 16];
          }
          if (j >= C::NB) ok = mbar_wait(&bar.bempty[sb], ((j / C::NB) - 1) & 1, status, 415) && ok;
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          // the two 64-channel halves store their units in opposite order: no bank is hit twice
          const int first = unit >> 2, c0 = (unit & 3) * 2;
          uint8_t *b = smem + C::OFF_B + sb * C::B_PITCH + first * (BK * 128) + r0 * 128;
#pragma unroll
          for (int p = 0; p < PASS; ++p) {
            uint4 lo, hi;
            ckpt8_restore16(q[p], sc[p], lo, hi);
            const int x = (r0 + 4 * p) & 7;
            *reinterpret_cast<uint4 *>(b + p * 512 + (((c0 + first) ^ x) << 4)) = first ? hi : lo;
            *reinterpret_cast<uint4 *>(b + p * 512 + (((c0 + 1 - first) ^ x) << 4)) = first ? lo : hi;
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            arrive_cta0<CG>(&bar.bfull[sb]);
            mbar_arrive(&bar.qempty[sq]);
          }
        }
      }
      if (!ok) bar.abort = 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG > 1) cluster_sync_all();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_g<CG>(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// few tiles: the contraction split over a cluster
// ---------------------------------------------------------------------------
// When the output has fewer tiles than the GPU has SMs (few tokens, or a small
// weight), a cluster of up to eight CTAs shares one 128 x 64 tile: each walks
// its part of the contraction and leaves its fp32 partial tile in its own shared
// memory.  After a cluster barrier every thread of the cluster sums its pieces of
// four columns, in the order of the CTAs, over distributed shared memory, and
// finishes them.  One launch, no partial sums in HBM, the same bits every time.
//
// SWAP: up to 64 tokens, as the 64-wide operand B, with the weight's channels as
// the 128 rows: a stage then brings 128 rows of the weight instead of 128 rows
// of mostly absent tokens.
struct SplitBars {
  uint64_t full[4], empty[4], acc_full, drain;
  uint32_t tmem_base;
  int abort;
};
struct SplitSmem {
  static constexpr int NST = 4;
  static constexpr int A_BYTES = 128 * BK * 2, B_BYTES = 64 * BK * 2, STAGE = A_BYTES + B_BYTES;
  static constexpr int OFF_BAR = NST * STAGE;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;  // slack to align the base to 1024
  static_assert(128 * 64 * 4 <= NST * STAGE, "the partial tile takes the stages' place");
  static_assert(sizeof(SplitBars) <= 256, "barrier space");
};

template <bool A_MN, bool B_MN, bool SWAP>
__global__ void __launch_bounds__(256, 2)
    split_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB, const Args args,
                 int split) {
  using L = SplitSmem;
  constexpr int NST = L::NST;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  SplitBars &bar = *reinterpret_cast<SplitBars *>(smem + L::OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % split, tile = blockIdx.x / split;
  const int m0 = (tile / args.s.tiles_n) * 128, n0 = (tile % args.s.tiles_n) * 64;
  const int k0 = (int)((long long)args.s.kc * rank / split), k1 = (int)((long long)args.s.kc * (rank + 1) / split);
  int *status = args.status;
  reset_status(status, args.reset);

  const auto load_stage = [&](int j) {
    const int st = j % NST, k = k0 + j;
    uint8_t *a = smem + st * L::STAGE, *b = a + L::A_BYTES;
    mbar_arrive_expect_tx(&bar.full[st], L::STAGE);
    if constexpr (A_MN) {
      tma_load_2d(a, &mapA, &bar.full[st], m0, k * BK);
      tma_load_2d(a + BK * 128, &mapA, &bar.full[st], m0 + 64, k * BK);
    } else {
      tma_load_2d(a, &mapA, &bar.full[st], k * BK, m0);
    }
    if constexpr (B_MN)
      tma_load_2d(b, &mapB, &bar.full[st], n0, k * BK);
    else
      tma_load_2d(b, &mapB, &bar.full[st], k * BK, n0);
  };
  const int first = min(NST, k1 - k0);  // stages that travel while the rest of the block sets up
  if (threadIdx.x == 0) {
    prefetch_tensormap(&mapA);
    prefetch_tensormap(&mapB);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    mbar_init(&bar.acc_full, 1);
    mbar_init(&bar.drain, 1);
    bar.abort = 0;
    fence_barrier_init();
    fence_async_smem();
    for (int j = 0; j < first; ++j) load_stage(j);
  }
  if (warp == 2) tmem_alloc_g<1>(&bar.tmem_base, 64);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;

  if (warp == 0 && lane == 0) {
    bool ok = true;
    int j = first;
    for (; j < k1 - k0; ++j) {
      const int st = j % NST;
      if (!(ok = mbar_wait(&bar.empty[st], ((j / NST) - 1) & 1, status, 421))) break;
      if (*reinterpret_cast<volatile int *>(&bar.abort)) {
        ok = false;
        break;
      }
      load_stage(j);
    }
    if (!ok) bar.abort = 1;
    drain_loads(bar.full, NST, j, status, 422);
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_bf16(128, 64, B_MN ? 1 : 0) | (A_MN ? 1u << 15 : 0u);
    bool ok = true;
    int j = 0;
    for (int k = k0; k < k1; ++k, ++j) {
      const int st = j % NST;
      if (!(ok = mbar_wait(&bar.full[st], (j / NST) & 1, status, 423))) break;
      tc_fence_after();
      const uint32_t a = smem_u32(smem + st * L::STAGE), b = a + L::A_BYTES;
      const uint64_t da = A_MN ? sdesc_sw128(a, BK * 128, 1024) : sdesc_sw128(a, 16, 1024);
      const uint64_t db = B_MN ? sdesc_sw128(b, BK * 128, 1024) : sdesc_sw128(b, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk)
        mma_ss(tmem, da + (A_MN ? (uint64_t)kk * 128 : kslice16(kk, 0)), db + (B_MN ? (uint64_t)kk * 128 : kslice16(kk, 0)),
               idesc, (j > 0 || kk > 0) ? 1u : 0u);
      mma_commit(&bar.empty[st]);
    }
    if (ok) {
      mma_commit(&bar.acc_full);
    } else {
      bar.abort = 1;
      mma_drain(&bar.drain, status, 424);
    }
  } else if (warp == 3) {
    if (args.db)
      finish_bias(args.bias_part, args.bias_blocks, args.bias_cols, args.db, args.db_fp32, blockIdx.x, gridDim.x, lane);
  } else if (warp >= 4) {
    // partial tile -> shared memory as [output row][output column]: plain, row-per-thread 16-byte units swizzled by
    // the row; swapped, a thread holds an output column, and neighbours' words are neighbours
    const int row = (warp & 3) * 32 + lane;
    if (__all_sync(0xffffffffu, mbar_wait(&bar.acc_full, 0, status, 425))) {
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t v[32];
        tmem_ld32(tmem + g * 32 + ((uint32_t)((warp & 3) * 32) << 16), v);
        tmem_wait_ld();
        if constexpr (SWAP) {
#pragma unroll
          for (int i = 0; i < 32; ++i) *reinterpret_cast<uint32_t *>(smem + (g * 32 + i) * 512 + row * 4) = v[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(smem + row * 256 + (((g * 8 + i) ^ (row & 15)) << 4)) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
    } else {
      bar.abort = 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 2) tmem_dealloc_g<1>(tmem, 64);
  if (!__any_sync(0xffffffffu, *reinterpret_cast<volatile int *>(&bar.abort))) {
    constexpr int UNITS = SWAP ? 32 : 16;  // four-column pieces of a row
    const int om = SWAP ? n0 : m0, on = SWAP ? m0 : n0;  // the tile's place in the output
#pragma unroll 1
    for (int x = rank * 256 + threadIdx.x; x < 2048; x += 256 * split) {
      const int r = x / UNITS, unit = x % UNITS;
      const int m = om + r, c = on + unit * 4;
      const uint32_t src = smem_u32(smem) + (SWAP ? r * 512 + unit * 16 : r * 256 + ((unit ^ (r & 15)) << 4));
      float2 lo = make_float2(0.f, 0.f), hi = lo;
#pragma unroll 8
      for (int q = 0; q < split; ++q) {
        const float4 p = load_cta(map_to_cta(src, q));
        lo = fadd2(lo, make_float2(p.x, p.y));
        hi = fadd2(hi, make_float2(p.z, p.w));
      }
      const bool in = m < args.rows && c < args.cols;
      if (args.bias && c < args.cols) {
        const uint2 b = __ldg(reinterpret_cast<const uint2 *>(args.bias + c));
        lo = fadd2(lo, bf16_pair(b.x));
        hi = fadd2(hi, bf16_pair(b.y));
      }
      if (args.save_z == 1 && in)
        *reinterpret_cast<uint2 *>(args.Z + (long long)m * args.cols + c) =
            make_uint2(pack_bf16(lo.x, lo.y), pack_bf16(hi.x, hi.y));
      if (args.save_z == 2) {
        // eight lanes hold a block
        uint32_t top = max(max(__float_as_uint(lo.x) & 0x7fffffffu, __float_as_uint(lo.y) & 0x7fffffffu),
                           max(__float_as_uint(hi.x) & 0x7fffffffu, __float_as_uint(hi.y) & 0x7fffffffu));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const uint32_t sc = ckpt8_scale(top);
        const float inv = ckpt8_inverse(sc);
        float2 a = lo, b = hi;
        if (top > kCkptTop) {
          const bool bad = sc == kCkptBad;
          a = make_float2(bad ? 0.f : ckpt8_clamp(lo.x), bad ? 0.f : ckpt8_clamp(lo.y));
          b = make_float2(bad ? 0.f : ckpt8_clamp(hi.x), bad ? 0.f : ckpt8_clamp(hi.y));
        }
        if (m < args.rows && c < args.ldq) {
          *reinterpret_cast<uint32_t *>(args.codes + (long long)m * args.ldq + c) = ckpt8_code4(a.x, a.y, b.x, b.y, inv);
          if (unit % 8 == 0) args.scales[(long long)m * (args.ldq / 32) + c / 32] = (uint8_t)sc;
        }
      }
      if (!in) continue;
      if (args.out_fp32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(args.Y) + (long long)m * args.ldy + c) =
            make_float4(lo.x, lo.y, hi.x, hi.y);
        continue;
      }
      switch (args.act) {
        case PRISM_ACT_RELU:
          lo = act_value<PRISM_ACT_RELU>(lo), hi = act_value<PRISM_ACT_RELU>(hi);
          break;
        case PRISM_ACT_SILU:
          lo = act_value<PRISM_ACT_SILU>(lo), hi = act_value<PRISM_ACT_SILU>(hi);
          break;
        case PRISM_ACT_GELU:
          lo = act_value<PRISM_ACT_GELU>(lo), hi = act_value<PRISM_ACT_GELU>(hi);
          break;
        default:
          break;
      }
      if (args.R) {
        const uint2 q = *reinterpret_cast<const uint2 *>(args.R + (long long)m * args.ldr + c);
        lo = fadd2(lo, bf16_pair(q.x));
        hi = fadd2(hi, bf16_pair(q.y));
      }
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(args.Y) + (long long)m * args.ldy + c) =
          make_uint2(pack_bf16(lo.x, lo.y), pack_bf16(hi.x, hi.y));
    }
    // Rows of codes are padded to 128 channels, 64-column tiles to 64: where that leaves
    // half a group behind the last tile, it is part of the checkpoint too (codes 0).
    const int past = n0 + 64;
    if (!SWAP && args.save_z == 2 && past == args.s.tiles_n * 64 && past < args.ldq) {
      for (int x = rank * 256 + threadIdx.x; x < 512; x += 256 * split) {
        const int m = m0 + (x >> 2);
        if (m >= args.rows) break;
        *reinterpret_cast<uint4 *>(args.codes + (long long)m * args.ldq + past + (x & 3) * 16) = make_uint4(0, 0, 0, 0);
        if ((x & 3) == 0)
          *reinterpret_cast<uint16_t *>(args.scales + (long long)m * (args.ldq / 32) + past / 32) = 0x0101;
      }
    }
  }
  // Lanes outside the output have left the loop's body early; the aligned barrier wants
  // the whole warp at once.
  __syncwarp();
  cluster_sync_all();  // no CTA leaves while another reads its partial tile
}

}  // namespace gemm
}  // namespace prism
