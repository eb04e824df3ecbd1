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
// codes, four warps turn them into bf16 (exact: 8-bit integer times a power of
// two) in the swizzled layout the tensor cores read.
//
// SUM: the tensor cores add into their fp32 accumulator with truncation, an
// error that grows with the length of the chain (measured: 7e-8 of the sum's
// norm per 64 tokens, 2e-5 over the 20,000-token chains of a 92160-token weight
// gradient).  An fp32 output therefore takes chains of kChain stages only; the
// epilogue warps add each to rounded fp32 sums in registers, while the next
// chain runs in the other accumulator.
//
// Roles (warps): 0 TMA producer, 1 MMA issuer (CTA 0 of a pair), 2 TMEM owner,
// 3 idle, 4-11 epilogue (two accumulators in TMEM alternate, so the epilogue of
// one tile runs under the products of the next), 12-15 the converters of B8.
#pragma once

#include "ckpt8.cuh"
#include "common.cuh"
#include "internal.h"

namespace prism {
namespace gemm {

constexpr int BK = 64;  // contraction per stage: one 128-byte swizzle row of bf16
constexpr int kEpiWarps = 8;
constexpr int kStageBuf = 4096;  // one epilogue staging buffer: 32 rows x 128 bytes
constexpr int kConvWarps = 4;
constexpr int kChain = 8;  // stages per accumulator chain when SUM

template <int CG_, int BN_, bool A_MN_, bool B_MN_, bool B8_ = false, bool SUM_ = false>
struct Cfg {
  static constexpr int CG = CG_, BN = BN_;
  static constexpr bool A_MN = A_MN_, B_MN = B_MN_, B8 = B8_, SUM = SUM_;
  static constexpr int BM = 128 * CG;
  static constexpr int BNC = BN / CG;  // columns of B a CTA loads
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_BYTES = BNC * BK * 2;
  static constexpr int Q_BYTES = B8 ? BNC * BK : 0;  // codes of the stage's B
  static constexpr int STAGE = A_BYTES + B_BYTES + Q_BYTES;
  static constexpr int EPI = kEpiWarps * 2 * kStageBuf;
  static constexpr int NST_FIT = (232448 - 2048 - EPI) / STAGE;
  static constexpr int NST = NST_FIT < 6 ? NST_FIT : 6;
  static constexpr int OFF_EPI = NST * STAGE;
  static constexpr int OFF_BAR = OFF_EPI + EPI;
  static constexpr int SMEM = OFF_BAR + 1024 + 1024;  // barriers; slack to align the base to 1024
  static constexpr int THREADS = B8 ? 512 : 384;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr bool REGS = B8 && SUM && BN == 256;  // registers move between warpgroups
  static_assert(!B8 || (B_MN && BNC == 128), "the checkpoint operand comes in 128-channel columns");
};

struct Bars {
  uint64_t full[6], empty[6];          // operand stages: filled (CTA 0's), consumed (each CTA's own)
  uint64_t qfull[6];                   // B8: codes arrived (each CTA's own)
  uint64_t acc_full[2], acc_empty[2];  // accumulators: complete (each CTA's own), read (CTA 0's)
  uint64_t res[kEpiWarps][2];          // residual tiles of each epilogue warp
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
};

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
// the same shared-memory location in CTA 0 of the cluster
__device__ __forceinline__ uint32_t map_to_cta0(const void *p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
template <int CG>
__device__ __forceinline__ void arrive_cta0(uint64_t *bar) {
  if constexpr (CG == 1) {
    mbar_arrive(bar);
  } else {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_to_cta0(bar)) : "memory");
  }
}
template <int CG>
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, int *status, int where) {
  if constexpr (CG == 1) {
    return mbar_wait(bar, parity, status, where);
  } else {
    long long t0 = 0;
    for (int spin = 0;; ++spin) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity)
          : "memory");
      if (ok) return true;
      if (spin == 0) {
        t0 = clock64();
      } else if (clock64() - t0 > kWaitLimitCycles) {
        record_timeout(status, where);
        return false;
      }
    }
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---------------------------------------------------------------------------
// activations (fp32).  gelu is the tanh form: z * sigmoid(2u),
// u = sqrt(2/pi) (z + 0.044715 z^3).
// ---------------------------------------------------------------------------
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == PRISM_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if constexpr (ACT == PRISM_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
  if constexpr (ACT == PRISM_ACT_GELU) return __fdividef(z, 1.f + __expf(-kGelu2 * fmaf(0.044715f * z * z, z, z)));
  return z;
}

// ---------------------------------------------------------------------------
// epilogues
// ---------------------------------------------------------------------------
template <int ACT>
__device__ __forceinline__ void act32(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = act_value<ACT>(v[i]);
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
// tile.  Each of the eight warps has two 4 KB staging buffers (32 rows x 64
// bf16, 128-byte swizzled as the tensor maps are), one for each of the at most
// two 64-column chunks it owns: a buffer receives its chunk's residual by TMA
// while the products run, then the result, then feeds the TMA store.  When the
// pre-activation is saved in bf16, it takes the second buffer.
template <class C>
__device__ __forceinline__ void epilogue_tile(const CUtensorMap &mapY, const CUtensorMap &mapR, const CUtensorMap &mapZ,
                                              const Args &args, Bars &bar, uint8_t *staging, uint32_t tmem, int group,
                                              int rank, int warp, int lane) {
  constexpr int CG = C::CG;
  const Sched &s = args.s;
  int *status = args.status;
  const int ew = warp - 4, q4 = warp & 3, half = ew >> 2;
  constexpr int NCH = C::BN / 64;             // 64-column chunks of the tile
  constexpr int PER = NCH > 1 ? NCH / 2 : 1;  // chunks of this warp
  const int c_lo = NCH > 1 ? half * PER : 0;
  const int n_ch = NCH > 1 ? PER : (half == 0 ? 1 : 0);
  uint8_t *buf = staging + ew * 2 * kStageBuf;
  const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
  const int sw = lane & 7;
  const bool z16 = args.save_z == 1;
  SegIter it(s, group);
  Seg sg;
  int t = 0;
  uint32_t res_phase = 0;  // bit i: parity of the next wait on residual buffer i
  bool ok = true;
  for (; ok && it.next(s, sg); ++t) {
    const int ab = t & 1;
    const int m0 = (sg.tile / s.tiles_n) * C::BM + rank * 128 + q4 * 32;
    const int n0 = (sg.tile % s.tiles_n) * C::BN + c_lo * 64;
    const bool parts = sg.slot >= 0;
    const bool rows_in = m0 < args.rows;
    uint32_t res_pending = 0;
    // residual of chunk c into buffer b (its last store has been read)
    const auto load_res = [&](int c, int b) {
      if (!(args.has_res && rows_in && n0 + c * 64 < args.cols)) return;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar.res[ew][b], kStageBuf);
        tma_load_2d(buf + b * kStageBuf, &mapR, &bar.res[ew][b], n0 + c * 64, m0);
      }
      res_pending |= 1u << b;
    };
    if (args.has_res) {
      if (lane == 0) store_wait_read<0>();
      __syncwarp();
      for (int c = 0; c < (z16 ? min(n_ch, 1) : n_ch); ++c) load_res(c, c);
    }
    ok = __all_sync(0xffffffffu, mbar_wait(&bar.acc_full[ab], (t >> 1) & 1, status, 407));
    if (ok) {
      tc_fence_after();
      const uint32_t acc = tmem + ab * C::BN + c_lo * 64 + lane_off;
      if (parts) {
        if (lane == 0) store_wait_read<0>();
        __syncwarp();
#pragma unroll 1
        for (int g = 0; g < 2 * n_ch; ++g) {
          uint32_t v[32];
          tmem_ld32(acc + g * 32, v);
          tmem_wait_ld();
          if (lane == 0) store_wait_read<1>();
          __syncwarp();
          stage_fp32(&mapZ, buf + (g & 1) * kStageBuf, v, lane, c_lo * 64 + g * 32,
                     sg.slot * C::BM + rank * 128 + q4 * 32, true);
        }
      }
#pragma unroll 1
      for (int c = 0; c < (parts ? 0 : n_ch); ++c) {
        const int col0 = n0 + c * 64;
        const bool in = rows_in && col0 < args.cols;
        const int yb = z16 ? 0 : c;
        if (z16 && c > 0) {
          if (lane == 0) store_wait_read<0>();
          __syncwarp();
          load_res(c, 0);
        }
        const bool res = (res_pending >> yb) & 1;
        if (!args.has_res) {
          // this buffer's last store was the one before the last (z16: the last)
          if (lane == 0) {
            if (z16 || C::BN < 256)
              store_wait_read<0>();
            else
              store_wait_read<1>();
          }
          __syncwarp();
        }
        uint32_t scale2 = 0;
        uint8_t *row = buf + yb * kStageBuf + lane * 128;
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          const int cg0 = col0 + g * 32;
          uint32_t u[32];
          tmem_ld32(acc + c * 64 + g * 32, u);
          tmem_wait_ld();
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
          if (args.bias) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (cg0 + i * 8 < args.cols) {
                const uint4 b = __ldg(reinterpret_cast<const uint4 *>(args.bias + cg0) + i);
                const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  v[8 * i + 2 * k] += bf16lo(w[k]);
                  v[8 * i + 2 * k + 1] += bf16hi(w[k]);
                }
              }
            }
          }
          if (z16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4 *>(row + kStageBuf + (((g * 4 + i) ^ sw) << 4)) =
                  make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                             pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
          } else if (args.save_z == 2) {
            uint32_t q[8];
            const uint32_t sc = ckpt8_quantise(v, q);
            if (m0 + lane < args.rows && cg0 < args.ldq) {
              uint4 *dst = reinterpret_cast<uint4 *>(args.codes + (long long)(m0 + lane) * args.ldq + cg0);
              dst[0] = make_uint4(q[0], q[1], q[2], q[3]);
              dst[1] = make_uint4(q[4], q[5], q[6], q[7]);
            }
            scale2 |= sc << (8 * g);
          }
          switch (args.act) {
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
          if (res && g == 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&bar.res[ew][yb], (res_phase >> yb) & 1, status, 408));
            res_phase ^= 1u << yb;
            res_pending &= ~(1u << yb);
            if (!ok) break;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 *p = reinterpret_cast<uint4 *>(row + (((g * 4 + i) ^ sw) << 4));
            if (res) {
              const uint4 r = *p;
              const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                v[8 * i + 2 * k] += bf16lo(w[k]);
                v[8 * i + 2 * k + 1] += bf16hi(w[k]);
              }
            }
            *p = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                            pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
          }
        }
        if (!ok) break;
        if (args.save_z == 2 && m0 + lane < args.rows && col0 < args.ldq)
          *reinterpret_cast<uint16_t *>(args.scales + (long long)(m0 + lane) * (args.ldq / 32) + col0 / 32) =
              (uint16_t)scale2;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (in) {
            store_2d(&mapY, buf + yb * kStageBuf, col0, m0);
            if (z16) store_2d(&mapZ, buf + kStageBuf, col0, m0);
          }
          store_commit();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cta0<CG>(&bar.acc_empty[ab]);
    }
    if (!ok) {
      bar.abort = 1;
      for (int b = 0; b < 2; ++b)  // loads that nothing will read
        if ((res_pending >> b) & 1) mbar_wait(&bar.res[ew][b], (res_phase >> b) & 1, status, 409);
    }
  }
  if (lane == 0) store_wait_read<0>();
}

// SUM: the chains of a segment added up in registers (a thread's row x its
// half of the columns), then written in fp32: a whole tile to the output, a
// partial one to its slot.
template <class C>
__device__ __forceinline__ void epilogue_sum(const CUtensorMap &mapY, const CUtensorMap &mapZ, const Args &args, Bars &bar,
                                             uint8_t *staging, uint32_t tmem, int group, int rank, int warp, int lane) {
  const Sched &s = args.s;
  const int ew = warp - 4, q4 = warp & 3, half = ew >> 2;
  constexpr int COLS = C::BN / 2;
  uint8_t *buf = staging + ew * 2 * kStageBuf;
  const uint32_t acc0 = tmem + half * COLS + ((uint32_t)(q4 * 32) << 16);
  SegIter it(s, group);
  Seg sg;
  int t = 0;
  bool ok = true;
  while (ok && it.next(s, sg)) {
    float sum[COLS];
#pragma unroll
    for (int i = 0; i < COLS; ++i) sum[i] = 0.f;
    for (int k0 = sg.k0; k0 < sg.k1; k0 += kChain, ++t) {
      const int ab = t & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.acc_full[ab], (t >> 1) & 1, args.status, 411));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < COLS / 16; ++g) {
        uint32_t v[16];
        tmem_ld16(acc0 + ab * C::BN + g * 16, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[g * 16 + i] += __uint_as_float(v[i]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cta0<C::CG>(&bar.acc_empty[ab]);
    }
    if (!ok) break;
    const int m0 = (sg.tile / s.tiles_n) * C::BM + rank * 128 + q4 * 32;
    const int n0 = (sg.tile % s.tiles_n) * C::BN + half * COLS;
#pragma unroll
    for (int g = 0; g < COLS / 32; ++g) {
      if (lane == 0) store_wait_read<1>();
      __syncwarp();
      uint32_t v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(sum[g * 32 + i]);
      if (sg.slot >= 0)
        stage_fp32(&mapZ, buf + (g & 1) * kStageBuf, v, lane, half * COLS + g * 32,
                   sg.slot * C::BM + rank * 128 + q4 * 32, true);
      else
        stage_fp32(&mapY, buf + (g & 1) * kStageBuf, v, lane, n0 + g * 32, m0,
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

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&bar.full[i], 1 + (C::B8 ? kConvWarps * CG : 0));
      mbar_init(&bar.empty[i], 1);
      mbar_init(&bar.qfull[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.acc_full[i], 1);
      mbar_init(&bar.acc_empty[i], kEpiWarps * CG);
    }
    for (int i = 0; i < kEpiWarps; ++i)
      for (int j = 0; j < 2; ++j) mbar_init(&bar.res[i][j], 1);
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
  // 512 threads and 128 sums in each of the epilogue's: the launch gives each of
  // the four warpgroups 128 registers a thread; 64 + 176 + 176 + 96 is the same total.
  if constexpr (C::REGS) {
    if (warp < 4) setmaxnreg_dec<64>();
    if (warp >= 12) setmaxnreg_dec<96>();
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
          if (j >= NST && !(ok = wait_cluster<CG>(&bar.empty[st], ((j / NST) - 1) & 1, status, 401))) break;
          if (aborted()) {
            ok = false;
            break;
          }
          uint8_t *a = smem + st * C::STAGE, *b = a + C::A_BYTES;
          if (rank == 0) mbar_arrive_expect_tx(&bar.full[st], CG * (C::A_BYTES + (C::B8 ? 0 : C::B_BYTES)));
          if constexpr (C::A_MN) {
            load_2d<CG>(a, &mapA, &bar.full[st], m0, k * BK);
            load_2d<CG>(a + BK * 128, &mapA, &bar.full[st], m0 + 64, k * BK);
          } else {
            load_2d<CG>(a, &mapA, &bar.full[st], k * BK, m0);
          }
          if constexpr (C::B8) {
            mbar_arrive_expect_tx(&bar.qfull[st], C::Q_BYTES);
            tma_load_2d(b + C::B_BYTES, &mapB, &bar.qfull[st], n0, k * BK);
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
          wait_cluster<CG>(&bar.empty[i % NST], (i / NST) & 1, status, 402);
      } else {
        // no copy may still be writing when the CTA leaves: CTA 0's barriers
        // count both CTAs' operand loads, and the pair leaves together
        bar.abort = 1;
        if (rank == 0) drain_loads(bar.full, NST, j, status, 403);
        if constexpr (C::B8) drain_loads(bar.qfull, NST, j, status, 403);
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
          const int k1 = C::SUM ? min(k0 + kChain, sg.k1) : sg.k1;
          const int ab = t & 1;
          if (t >= 2 && !(ok = wait_cluster<CG>(&bar.acc_empty[ab], ((t >> 1) - 1) & 1, status, 404))) break;
          tc_fence_after();
          for (int k = k0; k < k1; ++k, ++j) {
            const int st = j % NST;
            if (!(ok = wait_cluster<CG>(&bar.full[st], (j / NST) & 1, status, 405))) break;
            tc_fence_after();
            const uint32_t a = smem_u32(smem + st * C::STAGE), b = a + C::A_BYTES;
            // MN-major: 64-column chunks BK * 128 bytes apart, 8-k groups of 1024 bytes
            const uint64_t da = C::A_MN ? sdesc_sw128(a, BK * 128, 1024) : sdesc_sw128(a, 16, 1024);
            const uint64_t db = C::B_MN ? sdesc_sw128(b, BK * 128, 1024) : sdesc_sw128(b, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma<CG>(tmem + ab * C::BN, da + (C::A_MN ? (uint64_t)kk * 128 : kslice16(kk, 0)),
                      db + (C::B_MN ? (uint64_t)kk * 128 : kslice16(kk, 0)), idesc, (k > k0 || kk > 0) ? 1u : 0u);
            commit<CG>(&bar.empty[st]);
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
  } else if (warp >= 4 && warp < 4 + kEpiWarps) {
    // ---------------------------------------------------------------- epilogue
    if constexpr (C::REGS) setmaxnreg_inc<176>();
    if constexpr (C::SUM)
      epilogue_sum<C>(mapY, mapZ, args, bar, smem + C::OFF_EPI, tmem, group, (int)rank, warp, lane);
    else
      epilogue_tile<C>(mapY, mapR, mapZ, args, bar, smem + C::OFF_EPI, tmem, group, (int)rank, warp, lane);
  } else if (C::B8 && warp >= 12) {
    // ---------------------------------------------------------------- converters of the checkpoint operand
    if constexpr (C::B8) {
      const int cw = warp - 12;
      // lane -> 16 channels (lane % 8) of token row cw * 16 + pass * 4 + lane / 8
      const int unit = lane & 7, sub = lane >> 3;
      const long long lds = args.b_ld / 32;
      SegIter it(s, group), ahead(s, group);
      Seg sg, ag;
      // scales travel kAhead stages before their codes are due
      constexpr int kAhead = 3;
      uint32_t sc[kAhead][4];
      bool more = ahead.next(s, ag);
      int ak = more ? ag.k0 : 0;
      const auto fetch = [&](uint32_t (&d)[4]) {
        if (!more) return;
        const int blk = (((ag.tile % s.tiles_n) * C::BN + (int)rank * C::BNC) >> 5) + (unit >> 1);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int tok = ak * BK + cw * 16 + p * 4 + sub;
          d[p] = (tok < args.k_total && blk < lds) ? __ldg(args.b_scales + (long long)tok * lds + blk) : 127u;
        }
        if (++ak == ag.k1) {
          more = ahead.next(s, ag);
          ak = more ? ag.k0 : 0;
        }
      };
#pragma unroll
      for (int a = 0; a < kAhead; ++a) fetch(sc[a]);
      int j = 0, slot = 0;
      bool ok = true;
      // one stage: codes -> bf16 in the B buffer
      const auto convert = [&](uint32_t (&scale)[4]) {
        const int st = j % NST;
        // the stage's codes are loaded only once its products are done, so
        // their arrival also says that B's buffer may be written
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.qfull[st], (j / NST) & 1, status, 410));
        if (!ok) return;
        uint8_t *b = smem + st * C::STAGE + C::A_BYTES;
        const uint8_t *qs = b + C::B_BYTES;
        uint4 q[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) q[p] = *reinterpret_cast<const uint4 *>(qs + (cw * 16 + p * 4 + sub) * 128 + unit * 16);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int r = cw * 16 + p * 4 + sub;
          uint4 lo, hi;
          ckpt8_restore16(q[p], scale[p], lo, hi);
          uint8_t *row = b + (unit >> 2) * (BK * 128) + r * 128;
          const int c0 = (unit & 3) * 2;
          // the two 64-channel halves store their units in opposite order: no bank is hit twice
          const int first = unit >> 2;
          *reinterpret_cast<uint4 *>(row + (((c0 + first) ^ (r & 7)) << 4)) = first ? hi : lo;
          *reinterpret_cast<uint4 *>(row + (((c0 + 1 - first) ^ (r & 7)) << 4)) = first ? lo : hi;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive_cta0<CG>(&bar.full[st]);
        fetch(scale);
        ++j;
      };
      while (ok && it.next(s, sg)) {
        for (int k = sg.k0; ok && k < sg.k1; ++k) {
          if (slot == 0)
            convert(sc[0]);
          else if (slot == 1)
            convert(sc[1]);
          else
            convert(sc[2]);
          slot = slot == kAhead - 1 ? 0 : slot + 1;
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

}  // namespace gemm
}  // namespace prism
