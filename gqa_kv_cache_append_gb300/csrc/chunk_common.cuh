// chunk_common.cuh - what the two kernels of packed chunks share: chunk_attn.cu (causal,
// over the whole cache) and chunk_kernel.cuh (over a part of it).  Sizes, the launch's
// arguments, the join of cut units, argument checks, workspace and launch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/gqa.h"
#include "gqa_internal.h"
#include "serve_device.cuh"

namespace gqa {
namespace {

constexpr int kM = 128;           // query rows of a side
constexpr int kN = 128;           // positions of a tile
constexpr int kThreads = 384;     // two softmax warpgroups, one of single warps
// registers a thread: launched with 168 (65,536 over three warpgroups), then
// split unevenly: 2 x 128 x 208 + 128 x 88 = 384 x 168
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
constexpr int kDescInts = 8;      // per CTA, see below
constexpr int kSegs = 4;          // segments announced ahead
// A row's reference maximum is raised when the new one is this much larger, and
// P is taken this much higher (both base 2).
template <typename T16>
struct PRange {
  static constexpr float kRaise = Half16<T16>::kBf16 ? 8.f : 4.f;
  static constexpr float kLift = Half16<T16>::kBf16 ? 0.f : 11.f;
};

static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split");

struct ChunkArgs {
  const int *cu, *lens, *table;
  int b, total, h, g, r, tq;
  long long cap;       // positions a sequence can hold
  int bsz, max_blocks, num_blocks;
  float scale_log2;
  void* out;
  bool out_sectors;    // out is aligned to 32 bytes
  int* desc;           // [grid][kDescInts]
  float* part_ml;      // [2 * grid][srows][2]
  float* part_o;       // [2 * grid][srows][d_v]
  int srows;
  unsigned int* status;
  long long budget;
};

struct ChunkPos {  // a place in the order of all tiles
  int i, j, qt, lt;
};

__device__ __forceinline__ long long div_pos(long long a, long long b) {  // a >= 0, b > 0
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return static_cast<long long>(static_cast<unsigned long long>(a) /
                                static_cast<unsigned long long>(b));
}

// desc of CTA c: a unit cut at its run's end (head) or start (tail / middle)
enum { D_HEAD = 0, D_TOK0 = 1, D_NTOK = 2, D_J = 3, D_END = 4 };

// Joins the pieces of the units that a run's end cut: block (c, k) handles
// side k of the unit whose first piece is CTA c's, 32 rows at a time, two to a
// warp, four pieces of both with their loads side by side.  (A row after the
// other and a piece after the other took 12 us on cold caches for a few rows,
// this 7; blocks of 32 rows each, in eight waves, 21 us for the mixed batch's
// 300 pieces.)
// With per-piece maxima m, sums l and unnormalised outputs O over disjoint
// positions: M = max m, out = sum 2^(m - M) O / sum 2^(m - M) l, in the
// pieces' order.
constexpr int kJoinThreads = 512;

// Rows [row0, row1) of side `side` of the unit whose first piece is CTA c's, by a
// block of WARPS warps.
template <typename T16, int DV, int WARPS>
__device__ __forceinline__ void join_rows(const ChunkArgs& p, int nc, int c, int side, int row0,
                                          int row1) {
  constexpr int CPL = DV / 32;  // columns a lane
  constexpr int NP = 4;         // pieces at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 d4 = __ldg(reinterpret_cast<const int4*>(p.desc + static_cast<size_t>(c) * kDescInts));
  // the CTA that holds the unit's last piece
  int last = -1;
  for (int base = c + 1; base < nc && last < 0; base += 32) {
    const int k = base + lane;
    const bool e = k < nc && __ldg(p.desc + static_cast<size_t>(k) * kDescInts + D_END);
    const unsigned hit = __ballot_sync(0xffffffffu, e);
    if (hit) last = base + __ffs(hit) - 1;
    if (!d4.x) return;
  }
  if (!d4.x || last < 0) return;  // (none cut here)
  const int tok0 = d4.y, ntok = d4.z, j = d4.w;
  for (int base = row0; base < row1; base += 2 * WARPS) {
    int row[2], orow[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int rr = base + 2 * warp + s, tok = rr / p.r;
      const int t = side * p.tq + tok;
      row[s] = side * kM + rr;
      orow[s] = (tok < p.tq && t < ntok) ? t * p.h + (rr - tok * p.r) : -1;
    }
    if (orow[0] < 0 && orow[1] < 0) return;  // (later rows lie behind, too)
    float M[2] = {-INFINITY, -INFINITY}, den[2] = {0.f, 0.f}, num[2][CPL];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int e = 0; e < CPL; ++e) num[s][e] = 0.f;
    for (int x0 = c; x0 <= last; x0 += NP) {
      float2 ml[2][NP];
      float o[2][NP][CPL];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const int x = x0 + k;
          const bool use = x <= last && orow[s] >= 0;
          const size_t at = static_cast<size_t>(2 * x + (x == c ? 1 : 0)) * p.srows + row[s];
          ml[s][k] = use ? __ldg(reinterpret_cast<const float2*>(p.part_ml) + at)
                         : make_float2(-INFINITY, 0.f);
          const float* src = p.part_o + at * DV + lane * CPL;
          if constexpr (CPL == 4) {
            const float4 v = use ? __ldg(reinterpret_cast<const float4*>(src))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            o[s][k][0] = v.x, o[s][k][1] = v.y, o[s][k][2] = v.z, o[s][k][3] = v.w;
          } else {
            const float2 v =
                use ? __ldg(reinterpret_cast<const float2*>(src)) : make_float2(0.f, 0.f);
            o[s][k][0] = v.x, o[s][k][1] = v.y;
          }
        }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float mb = M[s];
#pragma unroll
        for (int k = 0; k < NP; ++k) mb = fmaxf(mb, ml[s][k].x);
        const float ref = mb == -INFINITY ? 0.f : mb;
        const float sc = ex2(M[s] - ref);
        den[s] *= sc;
#pragma unroll
        for (int e = 0; e < CPL; ++e) num[s][e] *= sc;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          // (a piece that the row sees nothing of may not have been written)
          if (ml[s][k].x == -INFINITY) continue;
          const float wgt = ex2(ml[s][k].x - ref);
          den[s] = fmaf(wgt, ml[s][k].y, den[s]);
#pragma unroll
          for (int e = 0; e < CPL; ++e) num[s][e] = fmaf(wgt, o[s][k][e], num[s][e]);
        }
        M[s] = mb;
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (orow[s] < 0) continue;
      const float inv = 1.f / den[s];
      T16* dst = static_cast<T16*>(p.out) +
                 (static_cast<size_t>(tok0) * p.h + j * p.r + orow[s]) * DV + lane * CPL;
      if constexpr (CPL == 4) {
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(Half16<T16>::pack2(num[s][0] * inv, num[s][1] * inv),
                       Half16<T16>::pack2(num[s][2] * inv, num[s][3] * inv));
      } else {
        *reinterpret_cast<uint32_t*>(dst) = Half16<T16>::pack2(num[s][0] * inv, num[s][1] * inv);
      }
    }
  }
}

template <typename T16, int DV>
__global__ void __launch_bounds__(kJoinThreads, 2)
    chunk_join_kernel(const ChunkArgs p, int nc) {
  pdl_wait_then_release();
  join_rows<T16, DV, kJoinThreads / 32>(p, nc, blockIdx.x, blockIdx.y, 0, kM);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct ChunkCall {
  const void *q, *k, *v;
  const int *cu, *lens, *table;
  int b, total, h, g, dk, dv;
  float scale;
  void* out;
  int cap, bsz, max_blocks, num_blocks, dtype;
  void* ws;
  long long ws_bytes;
};

struct ChunkPlan {
  int srows = 0;
  size_t ml_at = 0, o_at = 0, bytes = 0;
};

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

ChunkPlan chunk_plan(int total, int h, int g, int dv, int num_sms) {
  ChunkPlan pl;
  const int r = h / g, tq = kM / r;
  pl.srows = total <= tq ? kM : 2 * kM;
  pl.ml_at = up256(sizeof(int) * kDescInts * num_sms);
  const size_t rows = 2 * static_cast<size_t>(num_sms) * pl.srows;
  pl.o_at = up256(pl.ml_at + rows * 2 * sizeof(float));
  pl.bytes = up256(pl.o_at + rows * dv * sizeof(float));
  return pl;
}

int chunk_shape_check(int total, int h, int g, int dk, int dv) {
  if (total < 0 || h < 1 || g < 1 || dk < 1 || dv < 1 || h % g != 0) return GQA_ERR_SHAPE;
  if (static_cast<long long>(total) * h > 0x7FFFFFFFll) return GQA_ERR_SHAPE;
  if (h / g > kM || (dk != 64 && dk != 128) || (dv != 64 && dv != 128))
    return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}

int chunk_check(const ChunkCall& x) {
  if (!x.k || !x.v || !x.cu || !x.lens || !x.ws) return GQA_ERR_NULL;
  if (x.total != 0 && (!x.q || !x.out)) return GQA_ERR_NULL;
  if (x.dtype != GQA_F32 && x.dtype != GQA_BF16 && x.dtype != GQA_F16) return GQA_ERR_DTYPE;
  if (x.b < 1 || x.cap < 1) return GQA_ERR_SHAPE;
  if (int e = chunk_shape_check(x.total, x.h, x.g, x.dk, x.dv)) return e;
  if (x.table == nullptr && static_cast<long long>(x.b) * x.g * x.cap + 256 > 0x7FFFFFFFll)
    return GQA_ERR_SHAPE;
  if (x.dtype == GQA_F32 || x.b > 65535) return GQA_ERR_UNSUPPORTED;
  auto off = [](const void* p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) != 0; };
  if (off(x.q, 15) || off(x.k, 15) || off(x.v, 15) || off(x.out, 15) || off(x.cu, 3) ||
      off(x.lens, 3) || off(x.ws, 255))
    return GQA_ERR_ALIGN;
  return GQA_OK;
}

void chunk_args(ChunkArgs& p, const ChunkCall& x, const ChunkPlan& pl, unsigned int* status) {
  p.cu = x.cu;
  p.lens = x.lens;
  p.table = x.table;
  p.b = x.b;
  p.total = x.total;
  p.h = x.h;
  p.g = x.g;
  p.r = x.h / x.g;
  p.tq = kM / p.r;
  p.cap = x.table != nullptr ? static_cast<long long>(x.max_blocks) * x.bsz : x.cap;
  p.bsz = x.bsz;
  p.max_blocks = x.max_blocks;
  p.num_blocks = x.num_blocks;
  p.scale_log2 = static_cast<float>(static_cast<double>(x.scale) * 1.4426950408889634);
  p.out = x.out;
  p.out_sectors = (reinterpret_cast<uintptr_t>(x.out) & 31) == 0;
  char* ws = static_cast<char*>(x.ws);
  p.desc = reinterpret_cast<int*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + pl.ml_at);
  p.part_o = reinterpret_cast<float*>(ws + pl.o_at);
  p.srows = pl.srows;
  p.status = status;
  p.budget = kKernelWaitBudget;
}

// Maps of the query rows (boxes of q_tokens tokens' rows of a KV head) and of the
// caches or pools (boxes of up to `box` positions).
template <typename T16, int DK>
bool map_q(CUtensorMap* m, const ChunkCall& x, int q_tokens) {
  const uint64_t d[3] = {DK, static_cast<uint64_t>(x.h), static_cast<uint64_t>(x.total)};
  const uint64_t s[2] = {DK * 2, static_cast<uint64_t>(x.h) * DK * 2};
  const uint32_t b[3] = {64u, static_cast<uint32_t>(x.h / x.g), static_cast<uint32_t>(q_tokens)};
  return encode_bf16_map(m, x.q, 3, d, s, b, Half16<T16>::kBf16);
}

template <typename T16, int DK, int DV>
bool map_kv(CUtensorMap* mk, CUtensorMap* mv, const ChunkCall& x, int box) {
  const bool paged = x.table != nullptr;
  const uint64_t rows = paged ? static_cast<uint64_t>(x.num_blocks) * x.g * x.bsz
                              : static_cast<uint64_t>(x.b) * x.g * x.cap;
  const uint32_t b[2] = {64u, static_cast<uint32_t>(paged ? std::min(x.bsz, box) : box)};
  const uint64_t kd[2] = {DK, rows}, ks[1] = {DK * 2};
  const uint64_t vd[2] = {DV, rows}, vs[1] = {DV * 2};
  return encode_bf16_map(mk, x.k, 2, kd, ks, b, Half16<T16>::kBf16) &&
         encode_bf16_map(mv, x.v, 2, vd, vs, b, Half16<T16>::kBf16);
}

// Shared memory of a kernel, once a device; `configured`: devices done, a variant each.
template <class Kernel>
cudaError_t chunk_configure(Kernel kern, int smem, std::atomic<unsigned long long>& configured) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (configured.load() & (1ull << dev)) return cudaSuccess;
  if (cudaError_t e =
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))
    return e;
  // the split of registers must not ask for more than the launch brings: a
  // warpgroup would wait for them for ever
  cudaFuncAttributes fa;
  if (cudaError_t e = cudaFuncGetAttributes(&fa, kern)) return e;
  if (fa.numRegs * kThreads < 256 * kRegsSoftmax + 128 * kRegsOther)
    return cudaErrorLaunchOutOfResources;
  configured.fetch_or(1ull << dev);
  return cudaSuccess;
}

// One CTA an SM; the next kernel of the stream may start ahead.
struct ChunkLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  ChunkLaunch(int num_sms, int smem, cudaStream_t st) {
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  ChunkLaunch(const ChunkLaunch&) = delete;
};

// the pieces of cut units, behind the kernel that left them
template <typename T16, int DV>
cudaError_t launch_join(cudaLaunchConfig_t& cfg, const ChunkArgs& p, int num_sms) {
  cfg.gridDim = dim3(num_sms, p.srows / kM);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<T16, DV>, p, num_sms);
}

// Launch<type, d_k, d_v, paged>::run(call, ...) of the call's type, head dims and cache
template <template <typename, int, int, bool> class Launch, typename T16, bool PAGED,
          class Call, class... A>
cudaError_t chunk_dispatch_dims(const Call& x, A... a) {
  if (x.dk == 128)
    return x.dv == 128 ? Launch<T16, 128, 128, PAGED>::run(x, a...)
                       : Launch<T16, 128, 64, PAGED>::run(x, a...);
  return x.dv == 128 ? Launch<T16, 64, 128, PAGED>::run(x, a...)
                     : Launch<T16, 64, 64, PAGED>::run(x, a...);
}

template <template <typename, int, int, bool> class Launch, class Call, class... A>
cudaError_t chunk_dispatch(const Call& x, A... a) {
  if (x.table != nullptr)
    return x.dtype == GQA_F16 ? chunk_dispatch_dims<Launch, __half, true>(x, a...)
                              : chunk_dispatch_dims<Launch, __nv_bfloat16, true>(x, a...);
  return x.dtype == GQA_F16 ? chunk_dispatch_dims<Launch, __half, false>(x, a...)
                            : chunk_dispatch_dims<Launch, __nv_bfloat16, false>(x, a...);
}

}  // namespace
}  // namespace gqa
