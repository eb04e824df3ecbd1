// First pass of prism_linear_bwd: dZ = dY * act'(Z), rounded to bf16 for the two
// matrix products that follow, and the bias gradient db = column sums of dZ
// (taken from the fp32 values before that rounding).
//
// HBM-bound: dY and Z (bf16, or an 8-bit checkpoint) are read once, dZ written
// once.  A thread owns eight columns (one 16-byte vector) of every k-th row of
// its block, so its eight fp32 column sums stay in registers; the block's row
// lanes meet in shared memory, the blocks in the next launch, all in a fixed
// order.  Without an activation dZ is dY itself and only the sums are taken.
#include <algorithm>

#include "gemm.cuh"

namespace prism {
namespace actg {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
// Rows in flight per thread, and the CTAs per SM that the registers must leave
// room for.  Measured over 92160 x 4096 (gelu): bf16 Z, four rows 394 us, three
// rows in four CTAs 368 (6.2 TB/s); checkpoint, four rows 353, six rows 326 (5.8
// TB/s), eight 415.  Bound by memory, with the issue slots 60% busy.
template <int ACT, bool Z8>
struct Depth {
  static constexpr bool kZ16 = ACT != PRISM_ACT_NONE && !Z8;
  static constexpr int rows = kZ16 ? 3 : Z8 ? 6 : kUnroll, ctas = kZ16 ? 4 : 1;
};

// act'(z) of a pair in fp32, with p = 1 / (1 + e^-v).
//   silu = z p(z):             slope p + z p (1 - p)
//   gelu (tanh form) = z p(v), v = 2 sqrt(2/pi) (z + 0.044715 z^3): slope
//                              p + z p (1 - p) v'
// Far out p is 0 or 1 to the last bit (e^-v overflows or vanishes) and the second
// term 0, as long as v' stays finite; it is held at 3e38.  A NaN stays one (a
// restored checkpoint block that held a non-finite value).
template <int ACT>
__device__ __forceinline__ float2 act_slope(float2 z) {
  if constexpr (ACT == PRISM_ACT_RELU)
    return make_float2(z.x > 0.f ? 1.f : (z.x != z.x ? z.x : 0.f), z.y > 0.f ? 1.f : (z.y != z.y ? z.y : 0.f));
  const float2 one = make_float2(1.f, 1.f);
  if constexpr (ACT == PRISM_ACT_SILU) {
    const float2 p = gemm::logistic2(fmul2(z, make_float2(-gemm::kLog2e, -gemm::kLog2e)));
    return ffma2(fmul2(z, p), fsub2(one, p), p);
  } else {
    constexpr float k = gemm::kGelu2;
    const float2 z2 = fmul2(z, z);
    const float2 p = gemm::logistic2(fmul2(z, ffma2(z2, -0.044715f * k * gemm::kLog2e, -k * gemm::kLog2e)));
    float2 dv = ffma2(z2, 0.134145f * k, k);
    dv = make_float2(fminf(dv.x, 3e38f), fminf(dv.y, 3e38f));
    return ffma2(fmul2(fmul2(z, p), fsub2(one, p)), dv, p);
  }
}

struct Src {
  const uint4 *dY;
  long long ldy_vec;
  const uint4 *Z;  // bf16, or NULL
  long long ldz_vec;
  const uint2 *codes;  // checkpoint, or NULL
  const uint8_t *scales;
  long long ldq;
  uint4 *dZ;  // [n][cols]
  int *status;
};

// A checkpointed X that the weight gradient wants restored rides along: the grid's
// rows from `row` on restore it (one launch less; `row` is the grid's height if
// there is none).
struct Restore {
  int row;
  const uint2 *codes;
  const uint8_t *scales;
  Walk w;
  int vec;
  uint4 *x;
};

// tx threads (a power of two, 8..32) cover 8 * tx columns of a row
template <int ACT, bool Z8>
__global__ void __launch_bounds__(kThreads, (Depth<ACT, Z8>::ctas))
    act_grad_kernel(const Src s, const Restore re, long long n, int vecs, int tx, long long rows_per, float *__restrict__ part) {
  constexpr int ROWS = Depth<ACT, Z8>::rows;
  __shared__ float red[kThreads][9];
  gemm::reset_status(s.status, 1);
  if ((int)blockIdx.y >= re.row) {
    const long long cta = (long long)(blockIdx.y - re.row) * gridDim.x + blockIdx.x;
    unpack_walk<4>(re.codes, re.scales, re.w, re.vec, re.x, re.vec, (cta * kThreads + threadIdx.x) >> 4);
    return;
  }
  const int cx = threadIdx.x & (tx - 1), ry = threadIdx.x / tx, rows_step = kThreads / tx;
  const int cv = blockIdx.x * tx + cx;
  const long long r0 = (long long)blockIdx.y * rows_per + ry;
  const long long r1 = min((long long)(blockIdx.y + 1) * rows_per, n);
  float2 sum[4] = {};
  if (cv < vecs && r0 < r1) {
    int left = (int)((r1 - r0 + rows_step - 1) / rows_step);  // rows of this thread
    const uint4 *dy = s.dY + r0 * s.ldy_vec + cv;
    const uint4 *zp = (ACT != PRISM_ACT_NONE && !Z8) ? s.Z + r0 * s.ldz_vec + cv : nullptr;
    const uint2 *qp = Z8 ? s.codes + r0 * (s.ldq >> 3) + cv : nullptr;
    const uint8_t *sp = Z8 ? s.scales + r0 * (s.ldq >> 5) + (cv >> 2) : nullptr;
    uint4 *dz = s.dZ + r0 * vecs + cv;
    const long long dy_step = rows_step * s.ldy_vec, z_step = rows_step * s.ldz_vec, q_step = rows_step * (s.ldq >> 3),
                    s_step = rows_step * (s.ldq >> 5), dz_step = (long long)rows_step * vecs;
    for (; left > 0; left -= ROWS) {
      uint4 d[ROWS], z[ROWS];
      uint32_t sc[ROWS];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        if (u < left) {
          d[u] = __ldcs(dy);
          dy += dy_step;
          if constexpr (Z8) {
            const uint2 q = __ldcs(qp);
            z[u].x = q.x;
            z[u].y = q.y;
            sc[u] = __ldg(sp);
            qp += q_step;
            sp += s_step;
          } else if constexpr (ACT != PRISM_ACT_NONE) {
            z[u] = __ldcs(zp);
            zp += z_step;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        if (u >= left) break;
        const uint32_t dw[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
        if constexpr (ACT != PRISM_ACT_NONE) {
          uint4 zz = z[u];
          if constexpr (Z8) {
            const uint32_t s2 = ckpt8_scale2(sc[u]);
            zz = make_uint4(ckpt8_restore2(z[u].x, 0x4140, s2), ckpt8_restore2(z[u].x, 0x4342, s2),
                            ckpt8_restore2(z[u].y, 0x4140, s2), ckpt8_restore2(z[u].y, 0x4342, s2));
          }
          const uint32_t zw[4] = {zz.x, zz.y, zz.z, zz.w};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 g = fmul2(make_float2(bf16lo(dw[k]), bf16hi(dw[k])),
                                   act_slope<ACT>(make_float2(bf16lo(zw[k]), bf16hi(zw[k]))));
            sum[k] = fadd2(sum[k], g);
            o[k] = pack_bf16(g.x, g.y);
          }
          *dz = make_uint4(o[0], o[1], o[2], o[3]);
          dz += dz_step;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) sum[k] = fadd2(sum[k], make_float2(bf16lo(dw[k]), bf16hi(dw[k])));
        }
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    red[threadIdx.x][2 * k] = sum[k].x;
    red[threadIdx.x][2 * k + 1] = sum[k].y;
  }
  __syncthreads();
  // 8 * tx columns, summed over the row lanes
  for (int c = threadIdx.x; c < 8 * tx; c += kThreads) {
    if (blockIdx.x * tx + (c >> 3) < vecs) {
      float a = 0.f;
      for (int y = 0; y < rows_step; ++y) a += red[y * tx + (c >> 3)][c & 7];
      part[(long long)blockIdx.y * vecs * 8 + (long long)blockIdx.x * tx * 8 + c] = a;
    }
  }
}

// db alone; with a matrix product behind it, that launch's idle warps do this
__global__ void __launch_bounds__(32)
    bias_grad_kernel(const float *__restrict__ part, int blocks, int cols, void *__restrict__ db, int fp32) {
  gemm::finish_bias(part, blocks, cols, db, fp32, blockIdx.x, gridDim.x, threadIdx.x);
}

struct Shape {
  int tx, strips, blocks;
  long long rows_per;
};
// row blocks: enough CTAs for every SM's 8, each thread at least one full
// unrolled step of rows
static Shape shape_of(long long n, int cols) {
  Shape s;
  const int vecs = cols / 8;
  s.tx = vecs >= 32 ? 32 : vecs >= 16 ? 16 : 8;
  s.strips = (vecs + s.tx - 1) / s.tx;
  const long long step = (long long)(kThreads / s.tx) * kUnroll;
  const long long most = std::max<long long>(1, (long long)device_sm_count() * 8 / s.strips);
  const long long want = std::max<long long>(1, std::min(most, (n + step - 1) / step));
  s.rows_per = std::max<long long>(1, (n + want - 1) / want);
  s.blocks = (int)std::max<long long>(1, (n + s.rows_per - 1) / s.rows_per);
  return s;
}

struct Launch {
  Src s;
  Restore re;
  dim3 grid;
  long long n;
  int vecs, tx;
  long long rows_per;
  float *part;
  cudaStream_t st;
};
template <int ACT>
static void run(const Launch &l, bool z8) {
  if (z8)
    act_grad_kernel<ACT, true><<<l.grid, kThreads, 0, l.st>>>(l.s, l.re, l.n, l.vecs, l.tx, l.rows_per, l.part);
  else
    act_grad_kernel<ACT, false><<<l.grid, kThreads, 0, l.st>>>(l.s, l.re, l.n, l.vecs, l.tx, l.rows_per, l.part);
}

}  // namespace actg

size_t act_grad_part_bytes(long long n, int cols) {
  return align_up(sizeof(float) * (size_t)actg::shape_of(n, cols).blocks * cols, 256);
}

cudaError_t launch_act_grad(long long n, int cols, int act, const uint16_t *dY, long long ldy, const uint16_t *Z,
                            long long ldz, const prism_ckpt8_t *Z8, uint16_t *dZ, float *part, int *status,
                            const prism_ckpt8_t *X8, int width, uint16_t *X, cudaStream_t st) {
  const actg::Shape sh = actg::shape_of(n, cols);
  actg::Src s;
  s.dY = reinterpret_cast<const uint4 *>(dY);
  s.ldy_vec = ldy / 8;
  s.Z = reinterpret_cast<const uint4 *>(Z);
  s.ldz_vec = ldz / 8;
  s.codes = Z8 ? reinterpret_cast<const uint2 *>(Z8->codes) : nullptr;
  s.scales = Z8 ? Z8->scales : nullptr;
  s.ldq = Z8 ? Z8->ld : 0;
  s.dZ = reinterpret_cast<uint4 *>(dZ);
  s.status = status;
  dim3 grid(sh.strips, sh.blocks);
  actg::Restore re = {};
  re.row = sh.blocks;
  if (X8) {
    // whole grid rows of CTAs, four groups a half-warp or 24 CTAs an SM
    const long long per_cta = actg::kThreads / 16 * 4, groups = n * (X8->ld / 128);
    const long long ctas = std::min((groups + per_cta - 1) / per_cta, (long long)device_sm_count() * 24);
    const long long rows = std::min((ctas + sh.strips - 1) / sh.strips, 65535LL - sh.blocks);
    grid.y += (unsigned)rows;
    re.codes = reinterpret_cast<const uint2 *>(X8->codes);
    re.scales = X8->scales;
    re.w = make_walk(n, X8->ld, rows * sh.strips * (actg::kThreads / 16));
    re.vec = width / 8;
    re.x = reinterpret_cast<uint4 *>(X);
  }
  const actg::Launch l{s, re, grid, n, cols / 8, sh.tx, sh.rows_per, part, st};
  switch (act) {
    case PRISM_ACT_RELU:
      actg::run<PRISM_ACT_RELU>(l, Z8 != nullptr);
      break;
    case PRISM_ACT_SILU:
      actg::run<PRISM_ACT_SILU>(l, Z8 != nullptr);
      break;
    case PRISM_ACT_GELU:
      actg::run<PRISM_ACT_GELU>(l, Z8 != nullptr);
      break;
    default:
      actg::act_grad_kernel<PRISM_ACT_NONE, false>
          <<<grid, actg::kThreads, 0, st>>>(s, l.re, n, l.vecs, l.tx, l.rows_per, l.part);
  }
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  return e;
}

cudaError_t launch_bias_grad(long long n, int cols, const float *part, void *db, int db_fp32, cudaStream_t st) {
  actg::bias_grad_kernel<<<(cols + 31) / 32, 32, 0, st>>>(part, actg::shape_of(n, cols).blocks, cols, db, db_fp32);
  count_launches(1);
  return cudaGetLastError();
}

int act_grad_blocks(long long n, int cols) { return actg::shape_of(n, cols).blocks; }

}  // namespace prism
