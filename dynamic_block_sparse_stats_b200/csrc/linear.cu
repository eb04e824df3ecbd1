// prism_linear_fwd / prism_linear_bwd: a layer's linear map of its video tokens
// with bias, activation and residual in the epilogue, and its gradients, from
// activations held in bf16 or as 8-bit checkpoints.  Kernels: gemm.cuh (the
// matrix products), act_grad.cu (dZ and db).  Host side: checks, tile choice,
// tensor maps.
#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdio>

#include "gemm.cuh"

namespace prism {

int device_sm_count() {
  static std::atomic<int> known[64];  // by device; a device's count never changes
  int dev = 0, c = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && (c = known[dev].load(std::memory_order_relaxed)) > 0) return c;
  if (cudaDeviceGetAttribute(&c, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || c <= 0) return 148;
  if (dev < 64) known[dev].store(c, std::memory_order_relaxed);
  return c;
}

namespace lin {

using gemm::Args;
using gemm::Cfg;
using gemm::Sched;

// ---------------------------------------------------------------------------
// tile choice
// ---------------------------------------------------------------------------
// Three ways to a matrix product, timed on this GPU (us; kc = 64-deep stages):
//   pairs   256 x 256 tiles on CTA pairs, persistent: 0.40 a stage (power and L2
//           bound, 80% of the tensor pipe), 6.0 around them
//   single  128 x 128 tiles, persistent: 0.35 a stage (L2 bound), 4.2 around
//   split   128 x 64 tiles, the contraction over up to 8 CTAs of a cluster: 0.33
//           a stage, 5.0 (8 CTAs) to 8.1 (one) around, one tile per cluster; 0.3
//           more with what is called heavy below
// A wave of tiles takes no less than its epilogues: 1.8 (pairs) and 1.6 (single)
// us, 4.2 and 3.0 with an activation, a residual or a saved Z ("heavy"); the first
// wave's products and the last one's epilogue (0.1, heavy 2.6 and 2.0) have nothing
// beside them.  The least estimate is taken.  Against all three timed at 42 sizes from
// 1 x 1024 -> 4096 to 92160 x 1024 -> 1024, in seven forms each
// (profiles/linear_tile_choice.md): forward and dX within 3% of the best, dW within 15%,
// but for a checkpointed X with few output channels (40000 x 1152 -> 128: 51.3 us for
// 39.3), whose conversion on the way the estimate does not know.
struct Plan {
  int cg, bn;  // tile: 128 * cg rows, bn columns
  int split;   // > 0: split_kernel with clusters of this size
  bool swap;   // with the tokens as its 64-wide operand
  Sched s;
  double us;
};
constexpr int kMaxSplit = 8;
constexpr int kMaxGroups = 160;

static Sched make_sched(int cg, int bn, int rows, int cols, int kc, bool share) {
  Sched s;
  const int bm = 128 * cg;
  s.tiles_n = (cols + bn - 1) / bn;
  s.tiles = ((rows + bm - 1) / bm) * s.tiles_n;
  s.kc = kc;
  s.full = s.tiles;
  s.rem = 0;
  s.km = kc;
  const int most = std::min(device_sm_count() / cg, kMaxGroups);
  s.groups = std::min(most, s.tiles);
  if (share) {
    // at least 8 stages a group: below that the partial sums cost more than the products
    const long long want = std::max<long long>(s.tiles, (long long)s.tiles * kc / 8);
    s.groups = (int)std::min<long long>(most, want);
    const int rem = s.tiles % s.groups;
    const int km = (int)(((long long)kc * rem + s.groups - 1) / s.groups);
    // every helper gets at least one stage of a tail
    if (rem && km < kc && (long long)rem * (kc - km) >= s.groups - rem) {
      s.rem = rem;
      s.km = km;
      s.full = s.tiles - rem;
    } else if (rem) {
      s.groups = std::min(most, s.tiles);
    }
  }
  return s;
}

// share: the tiles of the last wave may be divided (the weight gradient's);
// chain: longest part of the contraction the split kernel may take in one sum
static Plan make_plan(int rows, int cols, int kc, bool share, int chain, bool may_swap, bool heavy) {
  Plan best = {};
  best.us = 1e300;
  const int sms = device_sm_count();
  for (int big = 0; big < 2; ++big) {
    Plan p = {};
    p.cg = big ? 2 : 1;
    p.bn = big ? 256 : 128;
    p.s = make_sched(p.cg, p.bn, rows, cols, kc, share);
    const double waves = p.s.rem ? (double)p.s.full / p.s.groups : (double)((p.s.tiles + p.s.groups - 1) / p.s.groups);
    const double stage = big ? 0.40 : 0.35, products = kc * stage;
    const double epilogue = big ? (heavy ? 4.2 : 1.8) : (heavy ? 3.0 : 1.6);
    p.us = big ? 6.0 : 4.2;
    if (p.s.rem)  // the shared tiles, and the kernel that adds their parts
      p.us += waves * std::max(products, epilogue) + p.s.km * stage + 5.0 + 0.02 * p.s.groups / p.s.rem;
    else
      p.us += products + (waves - 1) * std::max(products, epilogue) + (heavy ? (big ? 2.6 : 2.0) : 0.1);
    if (p.us < best.us) best = p;
  }
  Plan p = {};
  p.cg = 1;
  p.bn = 64;
  p.swap = may_swap && rows <= 64;  // only ever true of a split plan
  p.s = p.swap ? make_sched(1, 64, cols, rows, kc, false) : make_sched(1, 64, rows, cols, kc, false);
  if (p.s.tiles <= sms) {
    p.split = 1;
    while (p.split < kMaxSplit && 2 * p.split * p.s.tiles <= sms && 2 * p.split <= kc) p.split *= 2;
    const int part = (kc + p.split - 1) / p.split;
    p.us = 4.5 + 3.6 / p.split + (heavy ? 0.3 : 0.0) + part * 0.33;
    if (part <= chain && p.us < best.us) best = p;
  }
  return best;
}

// ---------------------------------------------------------------------------
// partial sums of the weight gradient
// ---------------------------------------------------------------------------
// dW of the split tiles = their slots in a fixed order: the first part, then the
// helpers' parts.  Y rows of threads take every Y-th part each and meet in shared
// memory, so that a small output cut into many parts (64 x 64 over 92160 tokens:
// 149) is read by enough threads; a CTA owns 1024 ITER / Y outputs.
// The helpers [first, last) of each split tile come with the launch: finding them
// takes 64-bit divisions, which cost more than the sums.
struct Helpers {
  uint8_t first[kMaxGroups], last[kMaxGroups];
};
template <int Y, int ITER>
__global__ void __launch_bounds__(256)
    sum_parts_kernel(const float *__restrict__ part, const Sched s, const Helpers who, int bm, int bn, int rows, int cols,
                     void *__restrict__ out, int fp32) {
  constexpr int LANES = 256 / Y;
  __shared__ float4 red[Y > 1 ? Y : 1][LANES];
  const int t = blockIdx.y, lane = threadIdx.x % LANES, y = threadIdx.x / LANES;
  const int tile = s.full + t;
  const int row0 = (tile / s.tiles_n) * bm, col0 = (tile % s.tiles_n) * bn;
  const long long slot = (long long)bm * bn;
  const int h0 = who.first[t], h1 = who.last[t];
  const float *first = part + t * slot, *more = part + (s.rem + h0 + t) * slot;
  const int parts = 1 + h1 - h0;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int e = ((blockIdx.x * ITER + i) * LANES + lane) * 4;
    const int row = row0 + e / bn, col = col0 + e % bn;
    const bool in = row < rows && col < cols;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
#pragma unroll 4
      for (int p = y; p < parts; p += Y) {
        const float4 b = __ldcs(reinterpret_cast<const float4 *>((p == 0 ? first : more + (p - 1) * slot) + e));
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
      }
    }
    if constexpr (Y > 1) {
      if (i > 0) __syncthreads();
      red[y][lane] = a;
      __syncthreads();
      if (y == 0) {
#pragma unroll
        for (int k = 1; k < Y; ++k) {
          const float4 b = red[k][lane];
          a.x += b.x;
          a.y += b.y;
          a.z += b.z;
          a.w += b.w;
        }
      }
    }
    if (y > 0 || !in) continue;
    const long long o = (long long)row * cols + col;
    if (fp32)
      *reinterpret_cast<float4 *>(static_cast<float *>(out) + o) = a;
    else
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + o) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
struct Maps {
  CUtensorMap a, b, y, r, z;
};

template <class C>
static cudaError_t launch(const Maps &m, const Args &args, cudaStream_t st) {
  const auto k = gemm::gemm_kernel<C>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  k<<<args.s.groups * C::CG, C::THREADS, C::SMEM, st>>>(m.a, m.b, m.y, m.r, m.z, args);
  count_launches(1);
  return cudaGetLastError();
}

static cudaError_t rows_map(CUtensorMap *m, const void *base, long long cols, long long rows, long long ld, int box_rows) {
  return make_map_2d(m, MAP_BF16, base, cols, rows, ld, 64, box_rows);
}

template <bool A_MN, bool B_MN, bool SWAP = false>
static cudaError_t launch_split(const Plan &p, const Maps &m, const Args &args, cudaStream_t st) {
  const auto k = gemm::split_kernel<A_MN, B_MN, SWAP>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, gemm::SplitSmem::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(p.s.tiles * p.split));
  c.blockDim = dim3(256);
  c.dynamicSmemBytes = gemm::SplitSmem::SMEM;
  c.stream = st;
  c.attrs = attr;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, k, m.a, m.b, args, p.split);
  count_launches(1);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// Whether a pair tile's epilogue gets 16 warps.  Eight are enough once the
// products of a tile (kc stages) take longer than its epilogue; below that the
// epilogue sets the time, and 16 hide one another's latencies, at the price of a
// stage.  Measured with both from 2 to 48 stages, 46080 tokens -> 1024 channels and
// 92160 -> 512 (us, the first, 8 warps and 16, around where they cross):
//   bias                    6: 47.6, 41.1    7: 47.2, 46.0    8: 48.5, 49.2
//   residual                8: 61.2, 56.1    9: 62.7, 63.1   10: 64.1, 66.7
//   bias, gelu             12: 72.8, 66.2   14: 76.7, 74.6   16: 81.8, 83.2
//   bias, Z in bf16        10: 69.8, 68.4   12: 75.5, 75.2   14: 79.8, 82.8
//   the same with gelu     16: 97.4, 92.5   18: 102.8, 100.5 20: 108.0, 108.2
//   bias, Z in 8 bits      12: 78.1, 72.7   14: 83.6, 80.9   16: 87.8, 89.1
//   the same with gelu     18: 107.2, 100.4 20: 110.8, 108.2 22: 116.7, 116.3
// A residual beside a saved Z moves the last by a stage or two.  Far beyond, 8 warps
// win by 1 to 2% (48 stages, gelu and Z: 220, 222).  Two staging buffers a warp and
// five stages, which this replaced, were ahead at 92160 x 512 -> 512 with a residual
// alone (56.3 against 58.4) and by up to 4% with gelu and Z in 8 bits around 20 stages
// (46080 x 1280 -> 1024: 104.2 against 107.4); level or behind, up to 30%, elsewhere.
static bool wide_epilogue(const Args &a) {
  const bool curved = a.act == PRISM_ACT_SILU || a.act == PRISM_ACT_GELU;  // an exponential and a reciprocal a value
  const int enough = a.save_z == 2   ? (curved ? 22 : 15)
                     : a.save_z == 1 ? (curved ? 19 : 13)
                     : curved        ? 15
                     : a.has_res     ? 9
                                     : 7;
  return a.s.kc < enough;
}

template <bool A_MN, bool B_MN>
static cudaError_t launch_plan(const Plan &p, const Maps &m, const Args &args, cudaStream_t st) {
  if (p.split && p.swap) return launch_split<B_MN, A_MN, true>(p, m, args, st);
  if (p.split) return launch_split<A_MN, B_MN>(p, m, args, st);
  if (p.cg == 1) return launch<Cfg<1, 128, A_MN, B_MN>>(m, args, st);
  if (wide_epilogue(args)) return launch<Cfg<2, 256, A_MN, B_MN, false, gemm::SUM_NONE, 16>>(m, args, st);
  return launch<Cfg<2, 256, A_MN, B_MN>>(m, args, st);
}

static cudaError_t forward(const prism_linear_t &l, const uint16_t *X, long long ldx, const uint16_t *W,
                           const uint16_t *bias, const uint16_t *R, long long ldr, uint16_t *Y, long long ldy,
                           uint16_t *Z, const prism_ckpt8_t *Z8, int *status, cudaStream_t st) {
  const int rows = (int)l.n, cols = l.out;
  const Plan p = make_plan(rows, cols, (l.in + gemm::BK - 1) / gemm::BK, false, 1 << 30, true,
                           l.act != PRISM_ACT_NONE || R || Z || Z8);
  Maps m;
  cudaError_t e;
  CUtensorMap &mx = p.swap ? m.b : m.a, &mw = p.swap ? m.a : m.b;
  if ((e = rows_map(&mx, X, l.in, rows, ldx, p.swap ? 64 : 128)) != cudaSuccess) return e;
  if ((e = rows_map(&mw, W, l.in, cols, l.in, p.swap ? 128 : p.bn / p.cg)) != cudaSuccess) return e;
  Args a = {};
  a.s = p.s;
  a.rows = rows;
  a.cols = cols;
  a.bias = bias;
  a.act = l.act;
  a.has_res = R != nullptr;
  a.save_z = Z ? 1 : Z8 ? 2 : 0;
  if (Z8) {
    a.codes = Z8->codes;
    a.scales = Z8->scales;
    a.ldq = Z8->ld;
  }
  a.status = status;
  a.reset = 1;
  if (p.split) {
    a.R = R;
    a.ldr = ldr;
    a.Y = Y;
    a.ldy = ldy;
    a.Z = Z;
  } else {
    if ((e = rows_map(&m.y, Y, cols, rows, ldy, 32)) != cudaSuccess) return e;
    m.r = m.z = m.y;
    if (R && (e = rows_map(&m.r, R, cols, rows, ldr, 32)) != cudaSuccess) return e;
    if (Z && (e = rows_map(&m.z, Z, cols, rows, cols, 32)) != cudaSuccess) return e;
    if (Z8 && (e = make_map_2d(&m.z, MAP_U8_SW64, Z8->codes, Z8->ld, rows, Z8->ld, 64, 32)) != cudaSuccess) return e;
  }
  return launch_plan<false, false>(p, m, a, st);
}

// The bias gradient's last step, for a launch to take along: its CTAs' idle warps
// own 32 columns each, one round if there are as many CTAs.
struct BiasTail {
  const float *part;
  int blocks, cols;
  void *db;  // NULL: nothing (left) to do
  int fp32;
};
static void take_bias(BiasTail &b, Args &a, int ctas) {
  if (!b.db || (b.cols + 31) / 32 > ctas) return;
  a.bias_part = b.part;
  a.bias_blocks = b.blocks;
  a.bias_cols = b.cols;
  a.db = b.db;
  a.db_fp32 = b.fp32;
  b.db = nullptr;
}
static int ctas_of(const Plan &p) { return p.split ? p.s.tiles * p.split : p.s.groups * p.cg; }

// dX [n][in] = dZ [n][out] W [out][in]
static cudaError_t input_grad(const prism_linear_t &l, const uint16_t *dZ, long long ldd, const uint16_t *W,
                              uint16_t *dX, BiasTail &bias, int *status, int reset, cudaStream_t st) {
  const int rows = (int)l.n, cols = l.in;
  const Plan p = make_plan(rows, cols, (l.out + gemm::BK - 1) / gemm::BK, false, 1 << 30, true, false);
  Maps m;
  cudaError_t e;
  CUtensorMap &mz = p.swap ? m.b : m.a, &mw = p.swap ? m.a : m.b;
  if ((e = rows_map(&mz, dZ, l.out, rows, ldd, p.swap ? 64 : 128)) != cudaSuccess) return e;
  if ((e = rows_map(&mw, W, l.in, l.out, l.in, gemm::BK)) != cudaSuccess) return e;
  Args a = {};
  a.s = p.s;
  a.rows = rows;
  a.cols = cols;
  a.status = status;
  a.reset = reset;
  take_bias(bias, a, ctas_of(p));
  if (p.split) {
    a.Y = dX;
    a.ldy = cols;
  } else {
    if ((e = rows_map(&m.y, dX, cols, rows, cols, 32)) != cudaSuccess) return e;
    m.r = m.z = m.y;
  }
  return launch_plan<false, true>(p, m, a, st);
}

static Plan grad_plan(const prism_linear_t &l, bool fp32) {
  return make_plan(l.out, l.in, (int)((l.n + gemm::BK - 1) / gemm::BK), true, fp32 ? gemm::kChain : gemm::kLongChain, false,
                   false);
}
static size_t grad_part_bytes(const Plan &p) {
  return p.s.rem ? sizeof(float) * (size_t)(p.s.groups + p.s.rem) * (128 * p.cg) * p.bn : 0;
}
// A checkpointed X is converted on its way to the tensor cores, once for every
// 256 output channels.  From 2048 of them on, restoring it once is faster, and
// so it is for the small tiles, whose kernels read bf16 only.  Measured at
// 92160 x 1024 in long runs, converted against restored (us): out = 512, 135 and
// 172; 1024, 251 and 268; 2048, 464 and 434.
static bool grad_restores(const prism_linear_t &l, const Plan &p) { return p.split || p.cg == 1 || l.out >= 2048; }

template <int CG, int BN, bool B8>
static cudaError_t launch_sum(int sum, const Maps &m, const Args &a, cudaStream_t st) {
  if (sum == gemm::SUM_FP32) return launch<Cfg<CG, BN, true, true, B8, gemm::SUM_FP32>>(m, a, st);
  if (sum == gemm::SUM_BF16) return launch<Cfg<CG, BN, true, true, B8, gemm::SUM_BF16>>(m, a, st);
  return launch<Cfg<CG, BN, true, true, B8>>(m, a, st);
}

// dW [out][in] = dZ^T X, summed over the tokens
static cudaError_t weight_grad(const prism_linear_t &l, const uint16_t *dZ, long long ldd, const uint16_t *X,
                               long long ldx, const prism_ckpt8_t *X8, uint16_t *restored, void *dW, int fp32,
                               float *part, BiasTail &bias, int *status, int reset, cudaStream_t st) {
  const Plan p = grad_plan(l, fp32);
  cudaError_t e;
  if (X8 && grad_restores(l, p)) {
    if ((e = launch_ckpt8_unpack(*X8, l.n, l.in, restored, l.in, st)) != cudaSuccess) return e;
    X = restored;
    ldx = l.in;
    X8 = nullptr;
  }
  Args a = {};
  a.s = p.s;
  a.rows = l.out;
  a.cols = l.in;
  a.status = status;
  a.reset = reset;
  if (!X8) take_bias(bias, a, ctas_of(p));
  const int bm = 128 * p.cg;
  Maps m;
  if ((e = rows_map(&m.a, dZ, l.out, l.n, ldd, gemm::BK)) != cudaSuccess) return e;
  if (X8)
    e = make_map_2d(&m.b, MAP_U8, X8->codes, l.in, l.n, X8->ld, 128, gemm::BK);
  else
    e = rows_map(&m.b, X, l.in, l.n, ldx, gemm::BK);
  if (e != cudaSuccess) return e;
  if (p.split) {
    a.Y = dW;
    a.ldy = l.in;
    a.out_fp32 = fp32;
    return launch_split<true, true>(p, m, a, st);
  }
  // whole tiles walk kc stages; where there are none, no group walks more than km
  const int sum = fp32                                                     ? gemm::SUM_FP32
                  : (p.s.full ? p.s.kc : p.s.km) > gemm::kLongChain ? gemm::SUM_BF16
                                                                    : gemm::SUM_NONE;
  if (fp32)
    e = make_map_2d(&m.y, MAP_F32, dW, l.in, l.out, l.in, 32, 32);
  else
    e = rows_map(&m.y, dW, l.in, l.out, l.in, 32);
  if (e != cudaSuccess) return e;
  m.r = m.z = m.y;
  if (p.s.rem &&
      (e = make_map_2d(&m.z, MAP_F32, part, p.bn, (long long)(p.s.groups + p.s.rem) * bm, p.bn, 32, 32)) != cudaSuccess)
    return e;
  if (X8) {
    a.b_scales = X8->scales;
    a.b_ld = X8->ld;
    a.k_total = (int)l.n;
    e = launch_sum<2, 256, true>(sum, m, a, st);
  } else if (p.cg == 2) {
    e = launch_sum<2, 256, false>(sum, m, a, st);
  } else {
    e = launch_sum<1, 128, false>(sum, m, a, st);
  }
  if (e != cudaSuccess || !p.s.rem) return e;
  Helpers who = {};
  const long long tail = p.s.kc - p.s.km;
  for (int t = 0, h = 0; t < p.s.rem; ++t) {
    // shares are at least one stage, so that a tail's helpers follow one another
    while (gemm::helper_start(p.s, h + 1) <= t * tail) ++h;
    who.first[t] = (uint8_t)h;
    int last = h + 1;
    while (last < p.s.groups - p.s.rem && gemm::helper_start(p.s, last) < (t + 1) * tail) ++last;
    who.last[t] = (uint8_t)last;
  }
  // rows of threads by the parts of a tile
  const int parts = p.s.groups / p.s.rem + 2, outputs = bm * p.bn;
  if (parts <= 8)
    sum_parts_kernel<1, 4><<<dim3(outputs / 4096, p.s.rem), 256, 0, st>>>(part, p.s, who, bm, p.bn, l.out, l.in, dW, fp32);
  else
    sum_parts_kernel<8, 1><<<dim3(outputs / 128, p.s.rem), 256, 0, st>>>(part, p.s, who, bm, p.bn, l.out, l.in, dW, fp32);
  count_launches(1);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// checks
// ---------------------------------------------------------------------------
static int refuse(int code, const char *fmt, ...) {
  char buf[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return report_error(code, buf);
}

static int check_linear(const prism_linear_t *l) {
  if (!l) return refuse(PRISM_ERR_INVALID_ARG, "linear: the description is NULL");
  if (l->n < 0 || l->n >= (1LL << 30))
    return refuse(PRISM_ERR_INVALID_ARG, "linear: n must be in [0, 2^30) (got %lld)", (long long)l->n);
  if (l->in <= 0 || l->in % 8 || l->in > (1 << 16) || l->out <= 0 || l->out % 8 || l->out > (1 << 16))
    return refuse(PRISM_ERR_INVALID_ARG, "linear: in and out must be positive multiples of 8, at most 65536 (got %d, %d)",
                  l->in, l->out);
  if (l->n * std::max(l->in, l->out) >= (1LL << 40))
    return refuse(PRISM_ERR_UNSUPPORTED, "linear: more than 2^40 values (n = %lld)", (long long)l->n);
  if (l->act < PRISM_ACT_NONE || l->act > PRISM_ACT_GELU)
    return refuse(PRISM_ERR_INVALID_ARG, "linear: act must be 0..3 (got %d)", l->act);
  return PRISM_OK;
}
// a bf16 matrix with rows of `cols` values `ld` apart
static int check_rows(const char *name, const void *p, long long ld, int cols) {
  if (reinterpret_cast<uintptr_t>(p) % 16) return refuse(PRISM_ERR_INVALID_ARG, "linear: %s is not 16-byte aligned", name);
  if (ld < cols || ld % 8 || ld > (1LL << 30))
    return refuse(PRISM_ERR_INVALID_ARG, "linear: the row stride of %s must be a multiple of 8, >= %d and <= 2^30 (got %lld)",
                  name, cols, ld);
  return PRISM_OK;
}
static int check_ckpt(const char *name, const prism_ckpt8_t *c, int cols) {
  if (!c->codes || !c->scales) return refuse(PRISM_ERR_INVALID_ARG, "linear: the arrays of checkpoint %s are NULL", name);
  if (reinterpret_cast<uintptr_t>(c->codes) % 16 || reinterpret_cast<uintptr_t>(c->scales) % 4)
    return refuse(PRISM_ERR_INVALID_ARG, "linear: checkpoint %s: codes must be 16-byte, scales 4-byte aligned", name);
  if (c->ld != ((long long)cols + 127) / 128 * 128)
    return refuse(PRISM_ERR_INVALID_ARG, "linear: checkpoint %s: ld must be %d rounded up to a multiple of 128 (got %lld)",
                  name, cols, (long long)c->ld);
  return PRISM_OK;
}
static int check_workspace(void *ws, size_t bytes, size_t need) {
  if (!ws) return refuse(PRISM_ERR_INVALID_ARG, "linear: workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % 256) return refuse(PRISM_ERR_INVALID_ARG, "linear: workspace not 256-byte aligned");
  if (bytes < need) return refuse(PRISM_ERR_CAPACITY, "linear: workspace too small: %zu bytes, need %zu", bytes, need);
  return PRISM_OK;
}

// The rules on shared memory: no output on anything that the call reads (but Y in
// place of its residual, where each thread reads what it overwrites), no two outputs
// on one another.
template <size_t O, size_t I>
static int check_apart(const Span (&out)[O], const Span (&in)[I], const Span *in_place = nullptr) {
  for (size_t o = 0; o < O; ++o) {
    for (size_t i = 0; i < I; ++i)
      if (!(o == 0 && &in[i] == in_place) && overlap(out[o], in[i]))
        return refuse(PRISM_ERR_INVALID_ARG, "linear: %s overlaps %s", out[o].name, in[i].name);
    for (size_t k = 0; k < o; ++k)
      if (overlap(out[o], out[k]))
        return refuse(PRISM_ERR_INVALID_ARG, "linear: %s overlaps %s", out[o].name, out[k].name);
  }
  return PRISM_OK;
}
static Span rows_span(const char *name, const void *p, long long rows, int cols, long long ld) {
  return Span(name, p, rows, 2 * (uint64_t)cols, 2 * (uint64_t)ld);
}
static Span flat_span(const char *name, const void *p, uint64_t bytes) { return Span(name, p, 1, bytes); }

// workspace of the backward: header, dZ (with an activation), the bias
// gradient's partial sums, the weight gradient's, X where it is restored
struct BwdWs {
  uint16_t *dZ, *X;
  float *bias_part, *part;
  size_t bytes;
};
static BwdWs carve_bwd(const prism_linear_t &l, bool x8, void *ws) {
  BwdWs b = {};
  size_t at = kWsHeader;
  char *w = static_cast<char *>(ws);
  b.dZ = reinterpret_cast<uint16_t *>(w + at);
  if (l.act != PRISM_ACT_NONE) at += align_up(2 * (size_t)l.n * l.out, 256);
  b.bias_part = reinterpret_cast<float *>(w + at);
  at += act_grad_part_bytes(l.n, l.out);
  b.part = reinterpret_cast<float *>(w + at);
  if (l.n > 0) {
    const Plan p = grad_plan(l, false), q = grad_plan(l, true);  // room for either output type
    at += std::max(grad_part_bytes(p), grad_part_bytes(q));
    b.X = reinterpret_cast<uint16_t *>(w + at);
    if (x8 && (grad_restores(l, p) || grad_restores(l, q))) at += align_up(2 * (size_t)l.n * l.in, 256);
  }
  b.bytes = at;
  return b;
}

}  // namespace lin
}  // namespace prism

using namespace prism;
using namespace prism::lin;

extern "C" {

size_t prism_linear_workspace_size(const prism_linear_t *l, int backward) {
  if (check_linear(l) != PRISM_OK) return 0;
  if (backward < 0 || backward > 2) return 0;
  return backward ? carve_bwd(*l, backward == 2, nullptr).bytes : kWsHeader;
}

int prism_linear_fwd(const prism_linear_t *l, const uint16_t *X, int64_t ldx, const uint16_t *W, const uint16_t *bias,
                     const uint16_t *R, int64_t ldr, uint16_t *Y, int64_t ldy, uint16_t *Z, const prism_ckpt8_t *Z8,
                     void *workspace, size_t ws_bytes, prism_stream_t stream) {
  NvtxRange nvtx_("prism_linear_fwd");
  int rc;
  if ((rc = check_linear(l)) != PRISM_OK) return rc;
  if (!W || (l->n > 0 && (!X || !Y))) return refuse(PRISM_ERR_INVALID_ARG, "linear: X, W or Y is NULL");
  if (Z && Z8) return refuse(PRISM_ERR_INVALID_ARG, "linear: Z is saved in bf16 or as a checkpoint, not both");
  if ((rc = check_rows("X", X, ldx, l->in)) != PRISM_OK || (rc = check_rows("W", W, l->in, l->in)) != PRISM_OK ||
      (rc = check_rows("bias", bias, l->out, l->out)) != PRISM_OK ||
      (rc = check_rows("R", R, R ? ldr : l->out, l->out)) != PRISM_OK ||
      (rc = check_rows("Y", Y, ldy, l->out)) != PRISM_OK || (rc = check_rows("Z", Z, l->out, l->out)) != PRISM_OK)
    return rc;
  if (Z8 && l->n > 0 && (rc = check_ckpt("Z8", Z8, l->out)) != PRISM_OK) return rc;
  if ((rc = check_workspace(workspace, ws_bytes, kWsHeader)) != PRISM_OK) return rc;
  {
    const long long n = l->n, ldq = Z8 ? Z8->ld : 0;
    const Span out[] = {rows_span("Y", Y, n, l->out, ldy), rows_span("Z", Z, n, l->out, l->out),
                        flat_span("Z8 (codes)", Z8 ? Z8->codes : nullptr, n * ldq),
                        flat_span("Z8 (scales)", Z8 ? Z8->scales : nullptr, n * ldq / 32),
                        flat_span("the workspace", workspace, kWsHeader)};
    const Span in[] = {rows_span("R", R, n, l->out, ldr), rows_span("X", X, n, l->in, ldx),
                       rows_span("W", W, l->out, l->in, l->in), flat_span("bias", bias, 2 * (uint64_t)l->out)};
    if ((rc = check_apart(out, in, R == Y && (ldr == ldy || n == 1) ? &in[0] : nullptr)) != PRISM_OK) return rc;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (l->n == 0)
    e = cudaMemsetAsync(workspace, 0, kWsHeader, st);
  else
    e = forward(*l, X, ldx, W, bias, R, ldr, Y, ldy, Z, Z8, &static_cast<WsHeader *>(workspace)->status, st);
  if (e != cudaSuccess) return refuse(PRISM_ERR_CUDA, "prism_linear_fwd: %s", cudaGetErrorString(e));
  clear_error();
  return PRISM_OK;
}

int prism_linear_bwd(const prism_linear_t *l, const uint16_t *dY, int64_t lddy, const uint16_t *X, int64_t ldx,
                     const prism_ckpt8_t *X8, const uint16_t *W, const uint16_t *Z, int64_t ldz,
                     const prism_ckpt8_t *Z8, uint16_t *dX, void *dW, void *db, int grad_fp32, void *workspace,
                     size_t ws_bytes, prism_stream_t stream) {
  NvtxRange nvtx_("prism_linear_bwd");
  int rc;
  if ((rc = check_linear(l)) != PRISM_OK) return rc;
  const bool act = l->act != PRISM_ACT_NONE;
  if (grad_fp32 != 0 && grad_fp32 != 1) return refuse(PRISM_ERR_INVALID_ARG, "linear: grad_fp32 must be 0 or 1");
  if (!dX && !dW && !db) return refuse(PRISM_ERR_INVALID_ARG, "linear: no gradient asked for");
  if (l->n > 0) {
    if (!dY) return refuse(PRISM_ERR_INVALID_ARG, "linear: dY is NULL");
    if (dX && !W) return refuse(PRISM_ERR_INVALID_ARG, "linear: dX needs W");
    if (dW && !X == !X8) return refuse(PRISM_ERR_INVALID_ARG, "linear: dW needs X or its checkpoint, not both");
    if (act && !Z == !Z8) return refuse(PRISM_ERR_INVALID_ARG, "linear: the activation needs Z or its checkpoint, not both");
    if ((rc = check_rows("dY", dY, lddy, l->out)) != PRISM_OK) return rc;
    if (X && (rc = check_rows("X", X, ldx, l->in)) != PRISM_OK) return rc;
    if (Z && (rc = check_rows("Z", Z, ldz, l->out)) != PRISM_OK) return rc;
    if (X8 && (rc = check_ckpt("X8", X8, l->in)) != PRISM_OK) return rc;
    if (Z8 && (rc = check_ckpt("Z8", Z8, l->out)) != PRISM_OK) return rc;
  }
  if ((rc = check_rows("W", W, l->in, l->in)) != PRISM_OK || (rc = check_rows("dX", dX, l->in, l->in)) != PRISM_OK ||
      (rc = check_rows("dW", dW, l->in, l->in)) != PRISM_OK || (rc = check_rows("db", db, l->out, l->out)) != PRISM_OK)
    return rc;
  const BwdWs b = carve_bwd(*l, X8 != nullptr, workspace);
  if ((rc = check_workspace(workspace, ws_bytes, b.bytes)) != PRISM_OK) return rc;
  {
    // what is read: X only for dW, W only for dX, Z only with an activation
    const long long n = l->n;
    const uint64_t elem = grad_fp32 ? 4 : 2;
    const prism_ckpt8_t none = {}, &x8 = X8 && dW ? *X8 : none, &z8 = Z8 && act ? *Z8 : none;
    const Span out[] = {rows_span("dX", dX, n, l->in, l->in), flat_span("dW", dW, elem * l->in * l->out),
                        flat_span("db", db, elem * l->out), flat_span("the workspace", workspace, b.bytes)};
    const Span in[] = {rows_span("dY", dY, n, l->out, lddy), rows_span("X", dW ? X : nullptr, n, l->in, ldx),
                       flat_span("X8 (codes)", x8.codes, n * x8.ld), flat_span("X8 (scales)", x8.scales, n * x8.ld / 32),
                       rows_span("W", dX ? W : nullptr, l->out, l->in, l->in),
                       rows_span("Z", act ? Z : nullptr, n, l->out, ldz), flat_span("Z8 (codes)", z8.codes, n * z8.ld),
                       flat_span("Z8 (scales)", z8.scales, n * z8.ld / 32)};
    if ((rc = check_apart(out, in)) != PRISM_OK) return rc;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  const size_t elem = grad_fp32 ? 4 : 2;
  if (l->n == 0) {  // empty sums
    e = cudaMemsetAsync(workspace, 0, kWsHeader, st);
    if (e == cudaSuccess && dW) e = cudaMemsetAsync(dW, 0, elem * l->in * l->out, st);
    if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, elem * l->out, st);
  } else {
    int *status = &static_cast<WsHeader *>(workspace)->status;
    const uint16_t *dZ = act ? b.dZ : dY;
    const long long ldd = act ? l->out : lddy;
    const bool first = act || db;
    BiasTail bias = {b.bias_part, act_grad_blocks(l->n, l->out), l->out, db, grad_fp32};
    if (first) {
      // a small X is restored in the same launch (2011 x 520: 6.1 + 2.6 us become 6.4),
      // a large one by its own kernel, whose CTAs fit the SMs better (92160 x 1024 with
      // dZ of 4096 columns: 335 + 50 us against 401)
      const prism_ckpt8_t *restore = dW && X8 && l->n * l->in <= (1 << 24) && grad_restores(*l, grad_plan(*l, grad_fp32))
                                         ? X8
                                         : nullptr;
      e = launch_act_grad(l->n, l->out, l->act, dY, lddy, Z, ldz, Z8, b.dZ, db ? b.bias_part : nullptr, status, restore,
                          l->in, b.X, st);
      if (restore) {
        X = b.X;
        ldx = l->in;
        X8 = nullptr;
      }
    }
    if (e == cudaSuccess && dX) e = input_grad(*l, dZ, ldd, W, dX, bias, status, !first, st);
    if (e == cudaSuccess && dW)
      e = weight_grad(*l, dZ, ldd, X, ldx, X8, b.X, dW, grad_fp32, b.part, bias, status, !first && !dX, st);
    if (e == cudaSuccess && bias.db) e = launch_bias_grad(l->n, l->out, b.bias_part, db, grad_fp32, st);
  }
  if (e != cudaSuccess) return refuse(PRISM_ERR_CUDA, "prism_linear_bwd: %s", cudaGetErrorString(e));
  clear_error();
  return PRISM_OK;
}

}  // extern "C"
