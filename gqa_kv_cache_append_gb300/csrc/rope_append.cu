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
//             s = max|x| / 448, x * (448 / max|x|) rounded to e4m3
// Everything in between is fp32.  Angles: f_m is kept as the 64-bit fraction
// of a turn per position, so P * f_m mod one turn is one wrapping 64-bit
// product and far positions lose nothing; as a signed number it is the angle
// over pi in units of 2^-63, rounded to fp32 half by half (2^-23 of itself) for
// sincospi.  (The upper half alone leaves small angles off by up to 1.5e-9
// rad; a 64-bit conversion takes 37.65 us where this takes 37.2.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/gqa.h"
#include "gqa_internal.h"
#include "serve_device.cuh"

namespace gqa {
namespace {

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

constexpr int kRopeThreads = 128;
constexpr int kBatch = 4;  // rows a lane loads ahead of their use

// One warp: a run of the rows of one token, query, then K, then V heads.  GS
// lanes hold a row, eight elements each, so 32 / GS rows go side by side.  A
// lane's eight elements are two pieces of four that hold both elements of
// every pair it turns: 4 g .. and rot/2 + 4 g .. of the halves layout (lanes
// past the rotated part, and the pairs layout: 8 g .. 8 g + 7), so rotation
// needs no exchange between lanes, and either way lane g turns pairs 4 g ..
// 4 g + 3, whose sines it computes once for all rows, with the norm's weights
// multiplied in.  Warps do not wait for one another, and the first rows'
// loads go out before the position is known.
//
// Bound by memory (every row read and written once) where rows are only
// turned; with the norm by its loads' latency, a batch of rows being loaded
// only when the one before it is done and registers holding 28 warps an SM,
// and by instructions close behind (63 % of the issue slots).  Measured (graph
// replay): one block per token, sines in shared memory and a shuffle per
// exchanged element 58 us for 2 x 4096 fp16 tokens and 113 us for 24 ragged
// sequences with norm (11,290 tokens, h = 28); a warp per token, the kind of a
// row chosen row by row 47 and 67 us; this form 36.8 and 45.1 us, 5,480 and
// 4,600 GB/s.  fp32, with norm, 8,192 tokens of h = 32, g = 8: 78.8 us, 5,110
// GB/s; into e4m3 rows, 4,305 tokens of h = 64, g = 8: 40.5 us, 4,140 GB/s.
enum { ROW_Q = 0, ROW_K = 1, ROW_V = 2 };

template <typename T, bool FP8, int GS>
__global__ void __launch_bounds__(kRopeThreads, FP8 ? 8 : 7)
    rope_append_kernel(const RopeLaunch a, int parts, int per_part) {
  constexpr int SIDE = 32 / GS;  // rows side by side
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const long long task =
      static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  if (task == 0) report_bad_packed(a.cu, a.lens, a.b, a.total, a.cap, a.status);
  const int t = static_cast<int>(task / parts);
  const int part = static_cast<int>(task - static_cast<long long>(t) * parts);
  if (t >= a.total) return;
  const int grp = lane / GS, g8 = lane % GS;
  // steps of SIDE rows: those of the query heads, then of K, then of V
  const int hq = a.q != nullptr ? a.h : 0;
  const int nq = (hq + SIDE - 1) / SIDE, nk = (a.g + SIDE - 1) / SIDE;
  const int s0 = part * per_part, s1 = min(nq + 2 * nk, s0 + per_part);
  const bool turns = a.phase != nullptr && 8 * g8 < a.rot;
  const bool halves = turns && !a.pairs;
  const int o0 = halves ? 4 * g8 : 8 * g8, o1 = halves ? (a.rot >> 1) + 4 * g8 : 8 * g8 + 4;

  Piece4<T> x[kBatch][2];
  // rows of kind KIND from its step `st` on
  auto load = [&](auto kind, int st) {
    constexpr int KIND = decltype(kind)::value;
    const int heads = KIND == ROW_Q ? hq : a.g, d = KIND == ROW_V ? a.dv : a.dk;
    const T* src = KIND == ROW_Q   ? static_cast<const T*>(a.q) + t * a.q_stride
                   : KIND == ROW_K ? static_cast<const T*>(a.k) + t * a.k_stride
                                   : static_cast<const T*>(a.v) + t * a.v_stride;
    const int row = st * SIDE + grp;
    src += row * d;
    const int p0 = KIND == ROW_V ? 8 * g8 : o0, p1 = KIND == ROW_V ? 8 * g8 + 4 : o1;
    const bool in = 8 * g8 < d;
    if (KIND == ROW_Q && a.q == a.q_out) {
      // memory that the kernel writes: not through the read-only path (which
      // the others keep: without it the 8-bit append of six chunks and their
      // read takes 58.6 us, with it 57.0)
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (in && row + k * SIDE < heads) {
          x[k][0].load_own(src + k * SIDE * d + p0);
          x[k][1].load_own(src + k * SIDE * d + p1);
        } else {
          x[k][0].zero();
          x[k][1].zero();
        }
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (in && row + k * SIDE < heads) {
        x[k][0].load(src + k * SIDE * d + p0);
        x[k][1].load(src + k * SIDE * d + p1);
      } else {
        x[k][0].zero();
        x[k][1].zero();
      }
    }
  };
  using Q = std::integral_constant<int, ROW_Q>;
  using K = std::integral_constant<int, ROW_K>;
  using V = std::integral_constant<int, ROW_V>;
  if (s0 < nq)
    load(Q{}, s0);
  else if (s0 < nq + nk)
    load(K{}, s0 - nq);
  else
    load(V{}, s0 - nq - nk);

  // the token's sequence and position (uniform across the warp)
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
      if (lane == 0 && s1 > nq) atomicOr(a.status, GQA_DEV_BAD_BLOCK);
      blk = -1;
    }
  }
  float cs[4], sn[4];  // of pairs 4 g8 ..
  if (turns) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned long long ph =
          __ldg(a.phase + 4 * g8 + k) * static_cast<unsigned long long>(P);
      // the angle over pi, in [-1, 1)
      const float turn = fmaf(static_cast<float>(static_cast<uint32_t>(ph)), 0x1p-32f,
                              static_cast<float>(static_cast<int>(ph >> 32)));
      sincospif(turn * 0x1p-31f, &sn[k], &cs[k]);
      cs[k] *= a.rope_scale;
      sn[k] *= a.rope_scale;
    }
  }
  const float inv_d = 1.f / static_cast<float>(a.dk);

  auto run = [&](auto kind, int from, int to, bool loaded) {
    constexpr int KIND = decltype(kind)::value;
    const int heads = KIND == ROW_Q ? hq : a.g, d = KIND == ROW_V ? a.dv : a.dk;
    const bool in = 8 * g8 < d;
    const int p0 = KIND == ROW_V ? 8 * g8 : o0, p1 = KIND == ROW_V ? 8 * g8 + 4 : o1;
    const bool norm = KIND != ROW_V && a.q_w != nullptr;
    float w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = 1.f;
    if (norm && in) {
      Piece4<T> r[2];
      const T* src = static_cast<const T*>(KIND == ROW_Q ? a.q_w : a.k_w);
      r[0].load(src + o0);
      r[1].load(src + o1);
      r[0].get(w);
      r[1].get(w + 4);
    }
    // Rotation two elements at a time, y = x * ca + x' * cb: for halves x is
    // two first (second) elements and x' their mates, for pairs x is a pair
    // and x' the pair turned around.  The weights are multiplied in.
    float2 ca[4], cb[4];
    if (KIND != ROW_V && turns) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (halves) {  // elements 2 k, 2 k + 1 of the eight: k < 2 first
          const int m = 2 * (k & 1), o = k < 2 ? 4 : -4;
          const float sg = k < 2 ? -1.f : 1.f;
          ca[k] = make_float2(w[2 * k] * cs[m], w[2 * k + 1] * cs[m + 1]);
          cb[k] = make_float2(sg * w[2 * k + o] * sn[m], sg * w[2 * k + 1 + o] * sn[m + 1]);
        } else {  // pair k
          ca[k] = make_float2(w[2 * k] * cs[k], w[2 * k + 1] * cs[k]);
          cb[k] = make_float2(-w[2 * k + 1] * sn[k], w[2 * k] * sn[k]);
        }
      }
    }
    for (int st = from; st < to; st += kBatch) {
      if (!loaded) load(kind, st);
      loaded = false;
#pragma unroll
      for (int it = 0; it < kBatch; ++it) {
        if (st + it >= to) break;  // (uniform)
        const int row = (st + it) * SIDE + grp;
        const bool mine = in && row < heads;
        alignas(8) float v[8];
        x[it][0].get(v);
        x[it][1].get(v + 4);
        float2* const v2 = reinterpret_cast<float2*>(v);
        float inv = 1.f;
        if (norm) {
          float2 sq = mul2(v2[0], v2[0]);
#pragma unroll
          for (int k = 1; k < 4; ++k) sq = fma2(v2[k], v2[k], sq);
          float ss = sq.x + sq.y;
#pragma unroll
          for (int o = GS / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          inv = rsqrtf(fmaf(ss, inv_d, a.eps));
        }
        if (KIND != ROW_V) {
          const float2 inv2 = make_float2(inv, inv);
          if (norm) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v2[k] = mul2(v2[k], inv2);
          }
          if (halves) {
            float2 y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = fma2(v2[k], ca[k], mul2(v2[k ^ 2], cb[k]));
#pragma unroll
            for (int k = 0; k < 4; ++k) v2[k] = y[k];
          } else if (turns) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v2[k] = fma2(v2[k], ca[k], mul2(make_float2(v2[k].y, v2[k].x), cb[k]));
          } else if (norm) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v2[k] = mul2(v2[k], make_float2(w[2 * k], w[2 * k + 1]));
          }
        }
        if (KIND == ROW_Q) {
          if (mine) {
            T* dst = static_cast<T*>(a.q_out) + (static_cast<size_t>(t) * a.h + row) * d;
            Piece4<T>::store(dst + p0, v);
            Piece4<T>::store(dst + p1, v + 4);
          }
          continue;
        }
        const long long dst = (static_cast<long long>(blk) * a.g + row) * a.bsz + prow;
        if constexpr (FP8) {
          float amax = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(v[k]));
#pragma unroll
          for (int o = GS / 2; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // (rows so small that the factor would overflow: scaled up first)
          const bool tiny = amax < 0x1p-100f;
          const float up = tiny ? 0x1p60f : 1.f;
          const float f = amax > 0.f ? kE4m3Max / (amax * up) : 0.f;
          if (mine && blk >= 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = v[k] * up * f;
            uint8_t* to8 = static_cast<uint8_t*>(KIND == ROW_V ? a.v_cache : a.k_cache) + dst * d;
            *reinterpret_cast<uint32_t*>(to8 + p0) = e4m3_pack4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint32_t*>(to8 + p1) = e4m3_pack4(v[4], v[5], v[6], v[7]);
            if (g8 == 0) (KIND == ROW_V ? a.v_scale : a.k_scale)[dst] = amax / kE4m3Max;
          }
        } else if (mine && blk >= 0) {
          T* to16 = static_cast<T*>(KIND == ROW_V ? a.v_cache : a.k_cache) + dst * d;
          if (KIND == ROW_V) {  // (bit for bit)
            x[it][0].copy_to(to16 + p0);
            x[it][1].copy_to(to16 + p1);
          } else {
            Piece4<T>::store(to16 + p0, v);
            Piece4<T>::store(to16 + p1, v + 4);
          }
        }
      }
    }
  };
  if (s0 < nq) run(Q{}, s0, min(s1, nq), true);
  if (s0 < nq + nk && s1 > nq)
    run(K{}, max(s0 - nq, 0), min(s1 - nq, nk), s0 >= nq);
  if (s1 > nq + nk) run(V{}, max(s0 - nq - nk, 0), s1 - nq - nk, s0 >= nq + nk);
}

// ---------------------------------------------------------------------------
// e4m3 cache -> rows of the call's type: positions [64 x, 64 x + 64) of KV
// head y of sequence z.  A thread takes one 16-byte piece of every
// (256 / pieces)-th row, two rows of K and of V at a time with their loads
// side by side.
// Memory-bound: d + 4 bytes read and d * sizeof(T) written per row.  Six
// sequences of up to 4,849 positions, g = 8, d = 128, to bf16: 15.2 us, 5,040
// GB/s, 65 % of the issue slots for the conversions.  (Room for four rows side
// by side, 64 registers and four blocks an SM: 16.5 us.)
// ---------------------------------------------------------------------------
constexpr int kReadRows = 64;
constexpr int kReadThreads = 256;

struct ReadRows {  // what a thread reads of one tensor
  uint4 raw[2];
  float sc[2];
  unsigned use;    // bit u: row u is there
  int c, row0, step, d;

  __device__ void start(int d_) {
    d = d_;
    const int per = d >> 4;  // pieces of a row
    row0 = threadIdx.x / per;
    c = threadIdx.x - row0 * per;
    step = kReadThreads / per;
    if (row0 >= step) row0 = 1 << 30;  // (256 not a multiple of the pieces)
  }
  __device__ void load(const uint8_t* __restrict__ pool, const float* __restrict__ scale,
                       const int* trow, int base, int p0, int rows, int g, int j, int bshift,
                       int num_blocks, unsigned int* status) {
    use = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int rr = row0 + base + u * step;
      if (row0 >= rows || rr >= rows) continue;
      const int p = p0 + rr;
      const int blk = __ldg(trow + (p >> bshift));
      if (blk < 0 || blk >= num_blocks) {
        atomicOr(status, GQA_DEV_BAD_BLOCK);
        continue;
      }
      const long long src =
          ((static_cast<long long>(blk) * g + j) << bshift) + (p & ((1 << bshift) - 1));
      raw[u] = __ldg(reinterpret_cast<const uint4*>(pool + src * d) + c);
      sc[u] = __ldg(scale + src);
      use |= 1u << u;
    }
  }
  template <typename T>
  __device__ void store(T* __restrict__ dst, int base, bool sectors) const {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!(use & (1u << u))) continue;
      T* to = dst + static_cast<size_t>(row0 + base + u * step) * d + 16 * c;
      const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      uint32_t y[4 * sizeof(T)];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float2 f = e4m3_unpack2(w[k >> 1] >> (16 * (k & 1)));
        f.x *= sc[u];
        f.y *= sc[u];
        if constexpr (sizeof(T) == 2) {
          y[k] = Half16<T>::pack2(f.x, f.y);
        } else {
          y[2 * k] = __float_as_uint(f.x);
          y[2 * k + 1] = __float_as_uint(f.y);
        }
      }
      store_sectors<sizeof(T) / 2>(to, y, sectors);
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kReadThreads, 5)
    kv_read_fp8_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool,
                       const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                       const int* __restrict__ table, const int* __restrict__ lens,
                       T* __restrict__ k_cache, T* __restrict__ v_cache, int g, int dk, int dv,
                       int bshift, int max_blocks, int num_blocks, int cap, unsigned int* status) {
  pdl_wait_then_release();
  const int i = blockIdx.z, j = blockIdx.y, p0 = blockIdx.x * kReadRows;
  const int L = __ldg(lens + i);
  if (L < 0 || L > cap || L > (static_cast<long long>(max_blocks) << bshift)) {
    if (p0 == 0 && j == 0 && threadIdx.x == 0) atomicOr(status, GQA_DEV_BAD_SEQ_LEN);
    return;
  }
  const int rows = min(kReadRows, L - p0);
  if (rows <= 0) return;
  const int* trow = table + static_cast<size_t>(i) * max_blocks;
  const size_t dst0 = (static_cast<size_t>(i) * g + j) * cap + p0;
  const bool sectors = ((reinterpret_cast<uintptr_t>(k_cache) |
                         reinterpret_cast<uintptr_t>(v_cache)) & 31) == 0;
  ReadRows k, v;
  k.start(dk);
  v.start(dv);
  for (int kb = 0, vb = 0; kb < rows || vb < rows; kb += 2 * k.step, vb += 2 * v.step) {
    k.load(k_pool, k_scale, trow, kb, p0, rows, g, j, bshift, num_blocks, status);
    v.load(v_pool, v_scale, trow, vb, p0, rows, g, j, bshift, num_blocks, status);
    k.store(k_cache + dst0 * dk, kb, sectors);
    v.store(v_cache + dst0 * dv, vb, sectors);
  }
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

template <typename T, bool FP8, int GS>
cudaError_t launch_rope_gs(const RopeLaunch& a, int num_sms, cudaStream_t st) {
  constexpr int SIDE = 32 / GS;
  const int nq = ((a.q != nullptr ? a.h : 0) + SIDE - 1) / SIDE, nk = (a.g + SIDE - 1) / SIDE;
  const int steps = nq + 2 * nk;
  // A warp takes a whole token, unless that leaves the SMs short of warps (16
  // each): then the token's rows are dealt out to several.  (More than 16: 4.0
  // -> 4.6 us for 64 tokens.)  With fewer than 32 tokens an SM (28 to 32 warps
  // fit at once) a token of 16 steps or more goes to two, for a shorter tail.
  // One warp against two, 2,500 and 4,800 tokens: h = 64, g = 8, d = 128 (40
  // steps) bf16 30.6 and 47.9 us against 27.4 and 42.0, fp32 52.9 and 88.7
  // against 49.0 and 76.2, bf16 to e4m3 40.2 and 44.6 against 33.3 and 45.8;
  // h = 16, g = 4 (12 steps) bf16 11.4 and 18.8 against 11.0 and 19.0; h = 8,
  // g = 2 (6 steps) bf16 7.9 and 10.7 against 8.7 and 12.5.
  const long long want = 16ll * num_sms;
  long long deal = (want + a.total - 1) / a.total;
  if (a.total < 2 * want && steps >= 16) deal = std::max(deal, 2ll);
  int parts = static_cast<int>(std::min<long long>(deal, steps));
  const int per_part = (steps + parts - 1) / parts;
  parts = (steps + per_part - 1) / per_part;
  constexpr int kWarps = kRopeThreads / 32;
  const long long blocks = (static_cast<long long>(a.total) * parts + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return launch_pdl(rope_append_kernel<T, FP8, GS>, dim3(static_cast<unsigned>(blocks)),
                    kRopeThreads, st, a, parts, per_part);
}

template <typename T, bool FP8>
cudaError_t launch_rope_t(const RopeLaunch& a, int num_sms, cudaStream_t st) {
  const int d = std::max(a.dk, a.dv);
  return d <= 64    ? launch_rope_gs<T, FP8, 8>(a, num_sms, st)
         : d <= 128 ? launch_rope_gs<T, FP8, 16>(a, num_sms, st)
                    : launch_rope_gs<T, FP8, 32>(a, num_sms, st);
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
  const long long dkk = static_cast<long long>(a.g) * a.dk;
  const long long dvv = static_cast<long long>(a.g) * a.dv;
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
  // in place, a token's output must lie where its query lies
  if (a.q != nullptr && a.q == a.q_out && a.q_stride != dq && a.total > 1) return GQA_ERR_SHAPE;
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
    // 2^64 * turns to the nearest whole number, below 2^64 (turns is at most
    // 1 - 2^-53, where the product is whole)
    phase_out[m] = static_cast<uint64_t>(std::nearbyint(std::ldexp(turns, 64)));
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
  const uint8_t* kp = static_cast<const uint8_t*>(k_pool);
  const uint8_t* vp = static_cast<const uint8_t*>(v_pool);
  int bshift = 0;  // (block_size is a power of two)
  while ((1 << bshift) < block_size) ++bshift;
  cudaError_t e;
  if (dtype == GQA_BF16)
    e = launch_pdl(kv_read_fp8_kernel<__nv_bfloat16>, grid, kReadThreads, st, kp, vp, k_scale,
                   v_scale, block_table, seq_lens, static_cast<__nv_bfloat16*>(k_cache),
                   static_cast<__nv_bfloat16*>(v_cache), g, d_k, d_v, bshift, max_blocks,
                   num_blocks, cap, status);
  else if (dtype == GQA_F16)
    e = launch_pdl(kv_read_fp8_kernel<__half>, grid, kReadThreads, st, kp, vp, k_scale, v_scale,
                   block_table, seq_lens, static_cast<__half*>(k_cache),
                   static_cast<__half*>(v_cache), g, d_k, d_v, bshift, max_blocks, num_blocks,
                   cap, status);
  else
    e = launch_pdl(kv_read_fp8_kernel<float>, grid, kReadThreads, st, kp, vp, k_scale, v_scale,
                   block_table, seq_lens, static_cast<float*>(k_cache),
                   static_cast<float*>(v_cache), g, d_k, d_v, bshift, max_blocks, num_blocks,
                   cap, status);
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // extern "C"
