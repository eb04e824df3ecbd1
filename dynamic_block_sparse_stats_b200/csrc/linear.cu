// prism_linear_fwd / prism_linear_bwd: a layer's linear map of its video tokens
// with bias, activation and residual in the epilogue, and its gradients, from
// activations held in bf16 or as 8-bit checkpoints.  Kernels: gemm.cuh (the
// matrix products), act_grad.cu (dZ and db).  Host side: checks, tile choice,
// tensor maps.
#include <algorithm>
#include <cstdarg>
#include <cstdio>

#include "gemm.cuh"

namespace prism {

int device_sm_count() {
  int dev = 0, c = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&c, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && c > 0)
    return c;
  return 148;
}

namespace lin {

using gemm::Args;
using gemm::Cfg;
using gemm::Sched;

// ---------------------------------------------------------------------------
// tile choice
// ---------------------------------------------------------------------------
struct Tile {
  int cg, bn;
};
// A stage's time on one CTA group, in SM clocks
static double stage_cost(const Tile &t) { return t.cg == 2 ? (t.bn == 256 ? 512 : 384) : (t.bn == 128 ? 384 : 320); }

static Sched make_sched(const Tile &t, int rows, int cols, int kc, bool split) {
  Sched s;
  const int bm = 128 * t.cg;
  s.tiles_n = (cols + t.bn - 1) / t.bn;
  s.tiles = ((rows + bm - 1) / bm) * s.tiles_n;
  s.kc = kc;
  s.full = s.tiles;
  s.rem = 0;
  s.km = kc;
  const int most = device_sm_count() / t.cg;
  s.groups = std::min(most, s.tiles);
  if (split) {
    // at least 8 stages a group: below that the partial sums cost more than the products
    const long long want = std::max<long long>(s.tiles, (long long)s.tiles * kc / 8);
    s.groups = (int)std::min<long long>(most, want);
    const int rem = s.tiles % s.groups;
    const int km = (int)(((long long)kc * rem + s.groups - 1) / s.groups);
    if (rem && km < kc) {
      s.rem = rem;
      s.km = km;
      s.full = s.tiles - rem;
    } else if (rem) {
      s.groups = std::min(most, s.tiles);
    }
  }
  return s;
}

static double sched_cost(const Tile &t, const Sched &s) {
  const double tail = 2000.0;  // filling the pipeline and the last epilogue
  const double waves = s.rem ? (double)s.full / s.groups + (double)s.rem / s.groups
                             : (double)((s.tiles + s.groups - 1) / s.groups);
  return waves * s.kc * stage_cost(t) + tail * t.bn / 256;
}

static Tile choose(const Tile *c, int n, int rows, int cols, int kc, bool split) {
  Tile best = c[0];
  double cost = 1e300;
  for (int i = 0; i < n; ++i) {
    const double x = sched_cost(c[i], make_sched(c[i], rows, cols, kc, split));
    if (x < cost) {
      cost = x;
      best = c[i];
    }
  }
  return best;
}

static const Tile kTiles[] = {{2, 256}, {2, 128}, {1, 128}, {1, 64}};
static const Tile kGradTiles[] = {{2, 256}, {1, 128}};

// ---------------------------------------------------------------------------
// partial sums of the weight gradient
// ---------------------------------------------------------------------------
// dW of the split tiles = their slots in a fixed order: first part, then the
// helpers'.  One float4 per thread; 4 * 256 outputs per CTA.
__global__ void __launch_bounds__(256)
    sum_parts_kernel(const float *__restrict__ part, const Sched s, int bm, int bn, int rows, int cols,
                     void *__restrict__ out, int fp32) {
  const int t = blockIdx.y;
  const int e = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int r = e / bn, c = e % bn;
  const int tile = s.full + t;
  const int row = (tile / s.tiles_n) * bm + r, col = (tile % s.tiles_n) * bn + c;
  if (r >= bm || row >= rows || col >= cols) return;
  const long long slot = (long long)bm * bn;
  float4 a = *reinterpret_cast<const float4 *>(part + t * slot + e);
  const int tail = s.kc - s.km, helpers = s.groups - s.rem;
  // the helpers whose ranges meet tile t's tail: their starts are rem * tail * h / helpers, rounded down
  int h = max(0, (int)((long long)t * helpers / s.rem) - 1);
  for (; h < helpers; ++h) {
    const long long lo = gemm::helper_start(s, h), hi = gemm::helper_start(s, h + 1);
    if (lo >= (long long)(t + 1) * tail) break;
    if (hi <= (long long)t * tail || lo == hi) continue;
    const float4 b = *reinterpret_cast<const float4 *>(part + (s.rem + h + t) * slot + e);
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
  }
  const long long o = (long long)row * cols + col;
  if (fp32)
    *reinterpret_cast<float4 *>(static_cast<float *>(out) + o) = a;
  else
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + o) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
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

template <bool A_MN, bool B_MN>
static cudaError_t launch_tile(const Tile &t, const Maps &m, const Args &args, cudaStream_t st) {
  if (t.cg == 2) {
    if (t.bn == 256) return launch<Cfg<2, 256, A_MN, B_MN>>(m, args, st);
    return launch<Cfg<2, 128, A_MN, B_MN>>(m, args, st);
  }
  if (t.bn == 128) return launch<Cfg<1, 128, A_MN, B_MN>>(m, args, st);
  return launch<Cfg<1, 64, A_MN, B_MN>>(m, args, st);
}

template <bool B8, bool SUM>
static cudaError_t launch_grad(const Tile &t, const Maps &m, const Args &args, cudaStream_t st) {
  if (t.cg == 2) return launch<Cfg<2, 256, true, true, B8, SUM>>(m, args, st);
  return launch<Cfg<1, 128, true, true, B8, SUM>>(m, args, st);
}

static cudaError_t forward(const prism_linear_t &l, const uint16_t *X, long long ldx, const uint16_t *W,
                           const uint16_t *bias, const uint16_t *R, long long ldr, uint16_t *Y, long long ldy,
                           uint16_t *Z, const prism_ckpt8_t *Z8, int *status, cudaStream_t st) {
  const int rows = (int)l.n, cols = l.out, kc = (l.in + gemm::BK - 1) / gemm::BK;
  const Tile t = choose(kTiles, 4, rows, cols, kc, false);
  Maps m;
  cudaError_t e;
  if ((e = rows_map(&m.a, X, l.in, rows, ldx, 128)) != cudaSuccess) return e;
  if ((e = rows_map(&m.b, W, l.in, cols, l.in, t.bn / t.cg)) != cudaSuccess) return e;
  if ((e = rows_map(&m.y, Y, cols, rows, ldy, 32)) != cudaSuccess) return e;
  m.r = m.z = m.y;
  if (R && (e = rows_map(&m.r, R, cols, rows, ldr, 32)) != cudaSuccess) return e;
  if (Z && (e = rows_map(&m.z, Z, cols, rows, cols, 32)) != cudaSuccess) return e;
  Args a = {};
  a.s = make_sched(t, rows, cols, kc, false);
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
  return launch_tile<false, false>(t, m, a, st);
}

// dX [n][in] = dZ [n][out] W [out][in]
static cudaError_t input_grad(const prism_linear_t &l, const uint16_t *dZ, long long ldd, const uint16_t *W,
                              uint16_t *dX, int *status, cudaStream_t st) {
  const int rows = (int)l.n, cols = l.in, kc = (l.out + gemm::BK - 1) / gemm::BK;
  const Tile t = choose(kTiles, 4, rows, cols, kc, false);
  Maps m;
  cudaError_t e;
  if ((e = rows_map(&m.a, dZ, l.out, rows, ldd, 128)) != cudaSuccess) return e;
  if ((e = rows_map(&m.b, W, l.in, l.out, l.in, gemm::BK)) != cudaSuccess) return e;
  if ((e = rows_map(&m.y, dX, cols, rows, cols, 32)) != cudaSuccess) return e;
  m.r = m.z = m.y;
  Args a = {};
  a.s = make_sched(t, rows, cols, kc, false);
  a.rows = rows;
  a.cols = cols;
  a.status = status;
  return launch_tile<false, true>(t, m, a, st);
}

static Tile grad_tile(const prism_linear_t &l) {
  return choose(kGradTiles, 2, l.out, l.in, (int)((l.n + gemm::BK - 1) / gemm::BK), true);
}
static Sched grad_sched(const prism_linear_t &l, const Tile &t) {
  return make_sched(t, l.out, l.in, (int)((l.n + gemm::BK - 1) / gemm::BK), true);
}
static size_t grad_part_bytes(const prism_linear_t &l) {
  const Tile t = grad_tile(l);
  const Sched s = grad_sched(l, t);
  return s.rem ? sizeof(float) * (size_t)(s.groups + s.rem) * (128 * t.cg) * t.bn : 0;
}

// dW [out][in] = dZ^T X, summed over the tokens
static cudaError_t weight_grad(const prism_linear_t &l, const uint16_t *dZ, long long ldd, const uint16_t *X,
                               long long ldx, const prism_ckpt8_t *X8, void *dW, int fp32, float *part, int *status,
                               cudaStream_t st) {
  const Tile t = grad_tile(l);
  Args a = {};
  a.s = grad_sched(l, t);
  a.rows = l.out;
  a.cols = l.in;
  a.status = status;
  const int bm = 128 * t.cg;
  Maps m;
  cudaError_t e;
  if ((e = rows_map(&m.a, dZ, l.out, l.n, ldd, gemm::BK)) != cudaSuccess) return e;
  if (X8)
    e = make_map_2d(&m.b, MAP_U8, X8->codes, l.in, l.n, X8->ld, 128, gemm::BK);
  else
    e = rows_map(&m.b, X, l.in, l.n, ldx, gemm::BK);
  if (e != cudaSuccess) return e;
  if (fp32)
    e = make_map_2d(&m.y, MAP_F32, dW, l.in, l.out, l.in, 32, 32);
  else
    e = rows_map(&m.y, dW, l.in, l.out, l.in, 32);
  if (e != cudaSuccess) return e;
  m.r = m.z = m.y;
  if (a.s.rem &&
      (e = make_map_2d(&m.z, MAP_F32, part, t.bn, (long long)(a.s.groups + a.s.rem) * bm, t.bn, 32, 32)) != cudaSuccess)
    return e;
  if (X8) {
    a.b_scales = X8->scales;
    a.b_ld = X8->ld;
    a.k_total = (int)l.n;
    e = fp32 ? launch_grad<true, true>(t, m, a, st) : launch_grad<true, false>(t, m, a, st);
  } else {
    e = fp32 ? launch_grad<false, true>(t, m, a, st) : launch_grad<false, false>(t, m, a, st);
  }
  if (e != cudaSuccess || !a.s.rem) return e;
  sum_parts_kernel<<<dim3(bm * t.bn / 1024, a.s.rem), 256, 0, st>>>(part, a.s, bm, t.bn, l.out, l.in, dW, fp32);
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

// workspace of the backward: header, dZ (with an activation), the bias
// gradient's partial sums, the weight gradient's
struct BwdWs {
  uint16_t *dZ;
  float *bias_part, *part;
  size_t bytes;
};
static BwdWs carve_bwd(const prism_linear_t &l, void *ws) {
  BwdWs b;
  size_t at = kWsHeader;
  char *w = static_cast<char *>(ws);
  b.dZ = reinterpret_cast<uint16_t *>(w + at);
  if (l.act != PRISM_ACT_NONE) at += align_up(2 * (size_t)l.n * l.out, 256);
  b.bias_part = reinterpret_cast<float *>(w + at);
  at += act_grad_part_bytes(l.n, l.out);
  b.part = reinterpret_cast<float *>(w + at);
  at += grad_part_bytes(l);
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
  return backward ? carve_bwd(*l, nullptr).bytes : kWsHeader;
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
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(workspace, 0, kWsHeader, st);
  if (e == cudaSuccess && l->n > 0)
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
  const BwdWs b = carve_bwd(*l, workspace);
  if ((rc = check_workspace(workspace, ws_bytes, b.bytes)) != PRISM_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(workspace, 0, kWsHeader, st);
  const size_t elem = grad_fp32 ? 4 : 2;
  if (l->n == 0) {  // empty sums
    if (e == cudaSuccess && dW) e = cudaMemsetAsync(dW, 0, elem * l->in * l->out, st);
    if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, elem * l->out, st);
  } else {
    int *status = &static_cast<WsHeader *>(workspace)->status;
    const uint16_t *dZ = act ? b.dZ : dY;
    const long long ldd = act ? l->out : lddy;
    if (e == cudaSuccess && (act || db))
      e = launch_act_grad(l->n, l->out, l->act, dY, lddy, Z, ldz, Z8, b.dZ, b.bias_part, db, grad_fp32, st);
    if (e == cudaSuccess && dX) e = input_grad(*l, dZ, ldd, W, dX, status, st);
    if (e == cudaSuccess && dW) e = weight_grad(*l, dZ, ldd, X, ldx, X8, dW, grad_fp32, b.part, status, st);
  }
  if (e != cudaSuccess) return refuse(PRISM_ERR_CUDA, "prism_linear_bwd: %s", cudaGetErrorString(e));
  clear_error();
  return PRISM_OK;
}

}  // extern "C"
