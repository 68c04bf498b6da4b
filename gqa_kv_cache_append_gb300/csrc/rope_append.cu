// rope_append.cu - what happens to a token's projections before attention:
// per-head RMS norm of q and k, rotary positions, and the write of k and v
// into the cache (16-bit or fp32 rows, or e4m3 rows with a scale each); and
// the read of an e4m3 cache back into 16-bit or fp32 rows.
//
// For a row x of a query or KV head at position P = L_i - n_i + s:
//   norm      x <- x / sqrt(mean(x^2) + eps) * w
//   rotation  each pair (a, c) of the first `rot` elements becomes
//             (a cos t - c sin t, c cos t + a sin t) * rope_scale,
//             t = P * f_m for pair m: elements (m, m + rot/2) or (2m, 2m + 1)
//   store     rounded once to the type of the call, or for an e4m3 cache
//             s = max|x| / 448, x / s rounded to e4m3
// Everything in between is fp32.  Angles: f_m is kept as the 64-bit fraction
// of a turn per position, so P * f_m mod one turn is one wrapping 64-bit
// product and far positions lose nothing; its upper 32 bits are the angle in
// units of 2^-32 turns (half a unit is 7e-10 rad), rounded to fp32 for
// sincospi.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/gqa.h"
#include "gqa_internal.h"
#include "serve_device.cuh"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRot = 256;

struct RopeLaunch {
  const void *q, *k, *v;                 // [total, heads, d], token strides below
  long long q_stride, k_stride, v_stride;  // elements
  const int *cu, *lens;
  const void *q_w, *k_w;                 // norm weights [d_k], or null
  float eps;
  const unsigned long long* phase;       // [rot / 2] turns per position * 2^64, or null
  int rot, pairs;                        // rotated elements; adjacent pairs or halves
  float rope_scale;
  void* q_out;
  void *k_cache, *v_cache;
  float *k_scale, *v_scale;              // e4m3 caches
  const int* table;                      // null: contiguous, block i of `bsz` = cap rows
  int bsz, max_blocks, num_blocks;
  int b, total, h, g, dk, dv;
  long long cap;                         // positions a sequence can hold
  unsigned int* status;
};

// One block: `rpp` rows (query, then K, then V heads) of one token; GS lanes
// hold a row, eight elements each.  Memory-bound: every row is read and
// written once as 16-byte pieces, all loads of a thread go out before the
// position is known, and sine and cosine are computed once per block for all
// its rows.
template <typename T, bool FP8, int IT>
__global__ void __launch_bounds__(kThreads)
    rope_append_kernel(const RopeLaunch a, int parts, int rpp, int gs) {
  __shared__ float s_cos[kMaxRot / 2], s_sin[kMaxRot / 2];
  pdl_wait_then_release();
  if (blockIdx.x == 0 && threadIdx.x < 32)
    report_bad_packed(a.cu, a.lens, a.b, a.total, a.cap, a.status);
  const int t = blockIdx.x / parts, part = blockIdx.x - t * parts;
  const int ngrp = kThreads / gs;
  const int grp = threadIdx.x / gs, e0 = (threadIdx.x % gs) * 8;
  const int hq = a.q != nullptr ? a.h : 0;
  const int rows = hq + 2 * a.g;
  const int r0 = part * rpp, r1 = min(rows, r0 + rpp);

  Piece8<T> x[IT];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int row = r0 + grp + it * ngrp;
    x[it].zero();
    if (row < r1) {
      if (row < hq) {
        if (e0 < a.dk)
          x[it].load(static_cast<const T*>(a.q) + t * a.q_stride + row * a.dk + e0);
      } else if (row < hq + a.g) {
        if (e0 < a.dk)
          x[it].load(static_cast<const T*>(a.k) + t * a.k_stride + (row - hq) * a.dk + e0);
      } else if (e0 < a.dv) {
        x[it].load(static_cast<const T*>(a.v) + t * a.v_stride + (row - hq - a.g) * a.dv + e0);
      }
    }
  }
  Piece8<T> wq, wk;
  if (a.q_w != nullptr && e0 < a.dk) {
    wq.load(static_cast<const T*>(a.q_w) + e0);
    wk.load(static_cast<const T*>(a.k_w) + e0);
  } else {
    wq.zero();
    wk.zero();
  }

  // the token's sequence and position (every warp; uniform across the block)
  const int i = packed_sequence(a.cu, a.b, t);
  if (i >= a.b) return;  // behind the last sequence
  const int t0 = __ldg(a.cu + i), t1 = __ldg(a.cu + i + 1), L = __ldg(a.lens + i);
  if (t < t0 || packed_errors(t0, t1, L, a.total, a.cap)) return;
  const int P = L - (t1 - t0) + (t - t0);
  int blk = i, prow = P;
  if (a.table != nullptr) {
    blk = __ldg(a.table + static_cast<size_t>(i) * a.max_blocks + P / a.bsz);
    prow = P % a.bsz;
    if (blk < 0 || blk >= a.num_blocks) {
      if (threadIdx.x == 0 && part == 0) atomicOr(a.status, GQA_DEV_BAD_BLOCK);
      blk = -1;
    }
  }
  if (a.phase != nullptr) {
    for (int m = threadIdx.x; m < a.rot / 2; m += kThreads) {
      const unsigned long long ph = __ldg(a.phase + m) * static_cast<unsigned long long>(P);
      // the angle over pi, in [-1, 1)
      const float y = static_cast<float>(static_cast<int>(ph >> 32)) * 0x1p-31f;
      float sn, cs;
      sincospif(y, &sn, &cs);
      s_cos[m] = cs * a.rope_scale;
      s_sin[m] = sn * a.rope_scale;
    }
    __syncthreads();
  }
  // this thread's eight elements of the rotation: y = x * c + partner * s
  const bool rotates = a.phase != nullptr && e0 < a.rot;
  const int half = a.rot >> 1;
  float c[8], s[8];
  if (rotates) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = e0 + k;
      const bool second = a.pairs ? (e & 1) : (e >= half);
      const int m = a.pairs ? (e >> 1) : (second ? e - half : e);
      c[k] = s_cos[m];
      s[k] = second ? s_sin[m] : -s_sin[m];
    }
  }
  // the lane that holds the other halves of this lane's pairs
  const int lane_g = threadIdx.x % gs;
  const int mate = (rotates && !a.pairs) ? (e0 < half ? lane_g + (half >> 3) : lane_g - (half >> 3))
                                         : lane_g;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int row = r0 + grp + it * ngrp;
    // (whole groups of lanes take each branch; the shuffles are among the
    // gs lanes of a row, with every lane of the warp taking part)
    const bool live = row < r1;
    const bool is_v = row >= hq + a.g;
    const int d = is_v ? a.dv : a.dk;
    float v[8];
    x[it].get(v);
    if (a.q_w != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[k], v[k], ss);
      for (int o = gs >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!is_v) {
        const float inv = rsqrtf(ss / static_cast<float>(a.dk) + a.eps);
        float w[8];
        if (row < hq)
          wq.get(w);
        else
          wk.get(w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = v[k] * inv * w[k];
      }
    }
    if (a.phase != nullptr) {
      float p[8];
      if (a.pairs) {
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = v[k ^ 1];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = __shfl_sync(0xffffffffu, v[k], mate, gs);
      }
      if (rotates && !is_v) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = fmaf(v[k], c[k], p[k] * s[k]);
      }
    }
    const bool mine = live && e0 < d;
    if (row < hq) {
      if (mine)
        Piece8<T>::store(
            static_cast<T*>(a.q_out) + (static_cast<size_t>(t) * a.h + row) * a.dk + e0, v);
      if (!FP8) continue;
    }
    const int j = is_v ? row - hq - a.g : row - hq;
    const long long dst = (static_cast<long long>(blk) * a.g + j) * a.bsz + prow;
    if constexpr (FP8) {
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(v[k]));
      for (int o = gs >> 1; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (mine && row >= hq && blk >= 0) {
        const float sc = amax / kE4m3Max;
        const float div = sc > 0.f ? sc : 1.f;
        uint2 pk;
        pk.x = e4m3_pack4(v[0] / div, v[1] / div, v[2] / div, v[3] / div);
        pk.y = e4m3_pack4(v[4] / div, v[5] / div, v[6] / div, v[7] / div);
        uint8_t* base = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache);
        *reinterpret_cast<uint2*>(base + dst * d + e0) = pk;
        if (e0 == 0) (is_v ? a.v_scale : a.k_scale)[dst] = sc;
      }
    } else if (mine && blk >= 0) {
      T* base = static_cast<T*>(is_v ? a.v_cache : a.k_cache);
      if (is_v)
        x[it].copy_to(base + dst * d + e0);  // (bit for bit)
      else
        Piece8<T>::store(base + dst * d + e0, v);
    }
  }
}

// ---------------------------------------------------------------------------
// e4m3 cache -> rows of the call's type: positions [64 x, 64 x + 64) of KV
// head y of sequence z, 16 elements a thread and step.  Memory-bound: (d + 4)
// bytes read and d * sizeof(T) written per row.
// ---------------------------------------------------------------------------
constexpr int kReadRows = 64;

template <typename T>
__device__ __forceinline__ void read_rows(const uint8_t* pool, const float* scale, T* cache,
                                          const int* trow, int p0, int rows, int d, int g, int j,
                                          int bsz, int num_blocks, long long dst_row,
                                          unsigned int* status) {
  const int per = d >> 4;  // 16-byte pieces a row
  for (int idx = threadIdx.x; idx < rows * per; idx += kThreads) {
    const int rr = idx / per, c = idx - rr * per;
    const int p = p0 + rr;
    const int blk = __ldg(trow + p / bsz);
    if (blk < 0 || blk >= num_blocks) {
      if (c == 0) atomicOr(status, GQA_DEV_BAD_BLOCK);
      continue;
    }
    const long long src = (static_cast<long long>(blk) * g + j) * bsz + p % bsz;
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(pool + src * d) + c);
    const float sc = __ldg(scale + src);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    T* dst = cache + (dst_row + rr) * d + 16 * c;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = e4m3_unpack2(w[2 * hf + (k >> 1)] >> (16 * (k & 1)));
        x[2 * k] = f.x * sc;
        x[2 * k + 1] = f.y * sc;
      }
      Piece8<T>::store(dst + 8 * hf, x);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv_read_fp8_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool,
                       const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                       const int* __restrict__ table, const int* __restrict__ lens,
                       T* __restrict__ k_cache, T* __restrict__ v_cache, int g, int dk, int dv,
                       int bsz, int max_blocks, int num_blocks, int cap, unsigned int* status) {
  pdl_wait_then_release();
  const int i = blockIdx.z, j = blockIdx.y, p0 = blockIdx.x * kReadRows;
  const int L = __ldg(lens + i);
  if (L < 0 || L > cap || L > static_cast<long long>(max_blocks) * bsz) {
    if (p0 == 0 && j == 0 && threadIdx.x == 0) atomicOr(status, GQA_DEV_BAD_SEQ_LEN);
    return;
  }
  const int rows = min(kReadRows, L - p0);
  if (rows <= 0) return;
  const int* trow = table + static_cast<size_t>(i) * max_blocks;
  const long long dst_row = (static_cast<long long>(i) * g + j) * cap + p0;
  read_rows(k_pool, k_scale, k_cache, trow, p0, rows, dk, g, j, bsz, num_blocks, dst_row, status);
  read_rows(v_pool, v_scale, v_cache, trow, p0, rows, dv, g, j, bsz, num_blocks, dst_row, status);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kern)(Params...), dim3 grid, int threads, cudaStream_t st,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, bool FP8>
cudaError_t launch_rope_t(const RopeLaunch& a, int num_sms, cudaStream_t st) {
  int gs = 8;
  while (gs * 8 < a.dk || gs * 8 < a.dv) gs *= 2;
  const int ngrp = kThreads / gs;
  const int rows = (a.q != nullptr ? a.h : 0) + 2 * a.g;
  // few tokens: one row a thread group, so that the rows of a token spread
  // over several SMs; many: four, which shares the position's sines among
  // more rows and keeps four loads of a thread in flight
  const bool small = static_cast<long long>(a.total) * ((rows + ngrp - 1) / ngrp) <= 2 * num_sms;
  const int it = small ? 1 : 4;
  const int parts = (rows + ngrp * it - 1) / (ngrp * it);
  const int rpp = (rows + parts - 1) / parts;
  const long long blocks = static_cast<long long>(a.total) * parts;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  return small ? launch_pdl(rope_append_kernel<T, FP8, 1>, grid, kThreads, st, a, parts, rpp, gs)
               : launch_pdl(rope_append_kernel<T, FP8, 4>, grid, kThreads, st, a, parts, rpp, gs);
}

template <bool FP8>
cudaError_t launch_rope(const RopeLaunch& a, int dtype, int num_sms, cudaStream_t st) {
  if (dtype == GQA_BF16) return launch_rope_t<__nv_bfloat16, FP8>(a, num_sms, st);
  if (dtype == GQA_F16) return launch_rope_t<__half, FP8>(a, num_sms, st);
  return launch_rope_t<float, FP8>(a, num_sms, st);
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// Host checks of a rotate-and-append call (no CUDA call).
int rope_check(const RopeLaunch& a, int layout, int dtype, bool fp8) {
  if (!a.cu || !a.lens || !a.k_cache || !a.v_cache) return GQA_ERR_NULL;
  if (a.total != 0 && (!a.k || !a.v)) return GQA_ERR_NULL;
  if ((a.q == nullptr) != (a.q_out == nullptr)) return GQA_ERR_NULL;
  if ((a.q_w == nullptr) != (a.k_w == nullptr)) return GQA_ERR_NULL;
  if (fp8 && (!a.k_scale || !a.v_scale)) return GQA_ERR_NULL;
  if (dtype != GQA_F32 && dtype != GQA_BF16 && dtype != GQA_F16) return GQA_ERR_DTYPE;
  if (a.b < 1 || a.total < 0 || a.h < 1 || a.g < 1 || a.h % a.g != 0 || a.dk < 1 || a.dv < 1 ||
      a.cap < 1)
    return GQA_ERR_SHAPE;
  const int elt = dtype == GQA_F32 ? 4 : 2;
  if (a.dk % 8 != 0 || a.dv % 8 != 0 || a.dk > 256 || a.dv > 256) return GQA_ERR_UNSUPPORTED;
  // (an e4m3 row is read back and copied in 16-byte pieces)
  if (fp8 && (a.dk % 16 != 0 || a.dv % 16 != 0)) return GQA_ERR_UNSUPPORTED;
  if (a.phase != nullptr) {
    if (layout != GQA_ROPE_HALF && layout != GQA_ROPE_PAIRS) return GQA_ERR_UNSUPPORTED;
    if (a.rot < 2 || a.rot > a.dk) return GQA_ERR_SHAPE;
    if (a.rot % 16 != 0) return GQA_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(a.phase) & 7u) return GQA_ERR_ALIGN;
  }
  const long long dq = static_cast<long long>(a.h) * a.dk;
  const long long dkk = static_cast<long long>(a.g) * a.dk, dvv = static_cast<long long>(a.g) * a.dv;
  if (dq > 0x7FFFFFFFll || static_cast<long long>(a.total) * (a.h + 2ll * a.g) > 0x7FFFFFFFll)
    return GQA_ERR_SHAPE;
  if ((a.q != nullptr && a.q_stride < dq) || a.k_stride < dkk || a.v_stride < dvv)
    return GQA_ERR_SHAPE;
  if ((a.q != nullptr && (a.q_stride * elt) % 16 != 0) || (a.k_stride * elt) % 16 != 0 ||
      (a.v_stride * elt) % 16 != 0)
    return GQA_ERR_ALIGN;
  if (off16(a.q) || off16(a.k) || off16(a.v) || off16(a.q_out) || off16(a.k_cache) ||
      off16(a.v_cache) || off16(a.q_w) || off16(a.k_w) || off4(a.k_scale) || off4(a.v_scale) ||
      off4(a.cu) || off4(a.lens))
    return GQA_ERR_ALIGN;
  return GQA_OK;
}

int rope_run(RopeLaunch& a, int layout, int dtype, bool fp8, void* stream) {
  if (int e = rope_check(a, layout, dtype, fp8)) return e;
  int num_sms = 0;
  if (int e = device_query(&num_sms, &a.status)) return e;
  if (a.total == 0) return GQA_OK;
  a.pairs = layout == GQA_ROPE_PAIRS;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = fp8 ? launch_rope<true>(a, dtype, num_sms, st)
                            : launch_rope<false>(a, dtype, num_sms, st);
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

int gqa_rope_table(int rot, double theta, int scaling, double factor, double original_len,
                   double low, double high, uint64_t* phase_out, float* rope_scale_out) {
  if (!phase_out || !rope_scale_out) return GQA_ERR_NULL;
  if (rot < 2 || rot % 2 != 0 || !(theta >= 1.0) || !std::isfinite(theta)) return GQA_ERR_SHAPE;
  if (scaling < GQA_ROPE_PLAIN || scaling > GQA_ROPE_YARN) return GQA_ERR_UNSUPPORTED;
  if (scaling != GQA_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor)))
    return GQA_ERR_SHAPE;
  const bool ramped = scaling == GQA_ROPE_WAVELENGTH || scaling == GQA_ROPE_YARN;
  if (ramped && (!(original_len > 0.0) || !(low > 0.0) || !(high > low) ||
                 !std::isfinite(original_len) || !std::isfinite(high)))
    return GQA_ERR_SHAPE;
  if (scaling == GQA_ROPE_YARN && !(theta > 1.0)) return GQA_ERR_SHAPE;
  const double two_pi = 6.283185307179586476925286766559;
  double first = 0.0, last = 0.0;
  if (scaling == GQA_ROPE_YARN) {
    // the pair index that turns x times over the original length
    auto at = [&](double x) {
      return rot * std::log(original_len / (x * two_pi)) / (2.0 * std::log(theta));
    };
    first = std::max(std::floor(at(high)), 0.0);
    last = std::min(std::ceil(at(low)), rot - 1.0);
  }
  for (int m = 0; m < rot / 2; ++m) {
    double f = std::pow(theta, -2.0 * m / rot);
    if (scaling == GQA_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == GQA_ROPE_WAVELENGTH) {
      const double x =
          std::min(std::max((original_len * f / two_pi - low) / (high - low), 0.0), 1.0);
      f = (1.0 - x) * f / factor + x * f;
    } else if (scaling == GQA_ROPE_YARN) {
      const double x = std::min(std::max((m - first) / std::max(last - first, 1e-3), 0.0), 1.0);
      f = f * (1.0 - x) + f / factor * x;
    }
    double turns = f / two_pi;
    turns -= std::floor(turns);
    // 2^64 * turns, below 2^64 (turns < 1 has 53 bits)
    phase_out[m] = static_cast<uint64_t>(std::ldexp(turns, 64));
  }
  *rope_scale_out = scaling == GQA_ROPE_YARN
                        ? static_cast<float>(factor > 1.0 ? 0.1 * std::log(factor) + 1.0 : 1.0)
                        : 1.0f;
  return GQA_OK;
}

int gqa_rope_append(const void* q, const void* k_new, const void* v_new, long long q_stride,
                    long long k_stride, long long v_stride, const int32_t* cu_tokens,
                    const int32_t* seq_lens, const void* q_weight, const void* k_weight, float eps,
                    const uint64_t* phase, int rot, int layout, float rope_scale, void* q_out,
                    void* k_cache, void* v_cache, int b, int total, int h, int g, int d_k,
                    int d_v, int cap, int dtype, void* stream) {
  if (b >= 1 && g >= 1 && cap >= 1 &&
      static_cast<long long>(b) * g * cap + 256 > 0x7FFFFFFFll)
    return GQA_ERR_SHAPE;
  RopeLaunch a = {q, k_new, v_new, q_stride, k_stride, v_stride, cu_tokens, seq_lens, q_weight,
                  k_weight, eps, reinterpret_cast<const unsigned long long*>(phase), rot, 0,
                  rope_scale, q_out, k_cache, v_cache, nullptr, nullptr, nullptr, cap, 0, 0, b,
                  total, h, g, d_k, d_v, cap, nullptr};
  return rope_run(a, layout, dtype, false, stream);
}

int gqa_rope_append_paged(const void* q, const void* k_new, const void* v_new, long long q_stride,
                          long long k_stride, long long v_stride, const int32_t* cu_tokens,
                          const int32_t* seq_lens, const void* q_weight, const void* k_weight,
                          float eps, const uint64_t* phase, int rot, int layout, float rope_scale,
                          void* q_out, void* k_pool, void* v_pool, const int32_t* block_table,
                          int b, int total, int h, int g, int d_k, int d_v, int block_size,
                          int max_blocks, int num_blocks, int dtype, void* stream) {
  if (int e = paged_args_check(block_table, g, block_size, max_blocks, num_blocks)) return e;
  RopeLaunch a = {q, k_new, v_new, q_stride, k_stride, v_stride, cu_tokens, seq_lens, q_weight,
                  k_weight, eps, reinterpret_cast<const unsigned long long*>(phase), rot, 0,
                  rope_scale, q_out, k_pool, v_pool, nullptr, nullptr, block_table, block_size,
                  max_blocks, num_blocks, b, total, h, g, d_k, d_v,
                  static_cast<long long>(max_blocks) * block_size, nullptr};
  return rope_run(a, layout, dtype, false, stream);
}

int gqa_rope_append_fp8_paged(const void* q, const void* k_new, const void* v_new,
                              long long q_stride, long long k_stride, long long v_stride,
                              const int32_t* cu_tokens, const int32_t* seq_lens,
                              const void* q_weight, const void* k_weight, float eps,
                              const uint64_t* phase, int rot, int layout, float rope_scale,
                              void* q_out, void* k_pool, void* v_pool, float* k_scale,
                              float* v_scale, const int32_t* block_table, int b, int total, int h,
                              int g, int d_k, int d_v, int block_size, int max_blocks,
                              int num_blocks, int dtype, void* stream) {
  if (int e = paged_args_check(block_table, g, block_size, max_blocks, num_blocks)) return e;
  RopeLaunch a = {q, k_new, v_new, q_stride, k_stride, v_stride, cu_tokens, seq_lens, q_weight,
                  k_weight, eps, reinterpret_cast<const unsigned long long*>(phase), rot, 0,
                  rope_scale, q_out, k_pool, v_pool, k_scale, v_scale, block_table, block_size,
                  max_blocks, num_blocks, b, total, h, g, d_k, d_v,
                  static_cast<long long>(max_blocks) * block_size, nullptr};
  return rope_run(a, layout, dtype, true, stream);
}

int gqa_kv_read_fp8_paged(const void* k_pool, const void* v_pool, const float* k_scale,
                          const float* v_scale, const int32_t* block_table,
                          const int32_t* seq_lens, void* k_cache, void* v_cache, int b, int g,
                          int d_k, int d_v, int block_size, int max_blocks, int num_blocks,
                          int cap, int dtype, void* stream) {
  if (!k_pool || !v_pool || !k_scale || !v_scale || !seq_lens || !k_cache || !v_cache)
    return GQA_ERR_NULL;
  if (dtype != GQA_F32 && dtype != GQA_BF16 && dtype != GQA_F16) return GQA_ERR_DTYPE;
  if (int e = paged_args_check(block_table, g, block_size, max_blocks, num_blocks)) return e;
  if (b < 1 || d_k < 1 || d_v < 1 || cap < 1) return GQA_ERR_SHAPE;
  if (static_cast<long long>(b) * g * cap + 256 > 0x7FFFFFFFll) return GQA_ERR_SHAPE;
  if (d_k % 16 != 0 || d_v % 16 != 0 || d_k > 256 || d_v > 256 || b > 65535 || g > 65535)
    return GQA_ERR_UNSUPPORTED;
  if (off16(k_pool) || off16(v_pool) || off16(k_cache) || off16(v_cache) || off4(k_scale) ||
      off4(v_scale) || off4(seq_lens))
    return GQA_ERR_ALIGN;
  int num_sms = 0;
  unsigned int* status = nullptr;
  if (int e = device_query(&num_sms, &status)) return e;
  const long long rows = std::min(static_cast<long long>(cap),
                                  static_cast<long long>(max_blocks) * block_size);
  const dim3 grid(static_cast<unsigned>((rows + kReadRows - 1) / kReadRows), g, b);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint8_t *kp = static_cast<const uint8_t*>(k_pool), *vp = static_cast<const uint8_t*>(v_pool);
  cudaError_t e;
  if (dtype == GQA_BF16)
    e = launch_pdl(kv_read_fp8_kernel<__nv_bfloat16>, grid, kThreads, st, kp, vp, k_scale, v_scale,
                   block_table, seq_lens, static_cast<__nv_bfloat16*>(k_cache),
                   static_cast<__nv_bfloat16*>(v_cache), g, d_k, d_v, block_size, max_blocks,
                   num_blocks, cap, status);
  else if (dtype == GQA_F16)
    e = launch_pdl(kv_read_fp8_kernel<__half>, grid, kThreads, st, kp, vp, k_scale, v_scale,
                   block_table, seq_lens, static_cast<__half*>(k_cache),
                   static_cast<__half*>(v_cache), g, d_k, d_v, block_size, max_blocks, num_blocks,
                   cap, status);
  else
    e = launch_pdl(kv_read_fp8_kernel<float>, grid, kThreads, st, kp, vp, k_scale, v_scale,
                   block_table, seq_lens, static_cast<float*>(k_cache),
                   static_cast<float*>(v_cache), g, d_k, d_v, block_size, max_blocks, num_blocks,
                   cap, status);
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // extern "C"
