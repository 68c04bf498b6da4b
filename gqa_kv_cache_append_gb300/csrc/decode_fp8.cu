// decode_fp8.cu - decode attention over an 8-bit paged cache (e4m3 values, one
// fp32 scale for each row of a KV head) on the tcgen05 tensor cores.
//
// The cache rows go to the tensor cores as they lie in memory (kind::f8f6f4);
// the 16-bit query rows and the softmax weights are each split into two e4m3
// pieces, x = hi + lo / 16 with hi = e4m3(x), lo = e4m3(16 (x - hi)): hi is
// off by at most 2^-4 |x|, the residual by 2^-4 of itself, 2^-8 |x| together,
// which is bf16's own rounding (a bf16 x in hi's normal range is exact).  The
// two pieces are two columns of the same product, and the products of the
// narrow matrices are far from the bound, so the split costs no time; the
// cache's bytes are the bound.  Per (sequence, KV head) tile of T = 256
// positions, with NR query rows (n new tokens x r heads, token-major):
//
//   S^T [T x 2 NR]   = K8 . (Qhi, Qlo)^T               (tcgen05.mma, 2 x M=128)
//   x[p, a]          = (Shi + Slo / 16) * ks[p] * qs[a] * scale * log2 e
//   y_a              = max_p x[p, a] + log2|vs[p] / vmax|    (vmax = max |vs| of the tile)
//   w[p, a]          = exp2(x - y_a)
//   P[p, a]          = w * vs[p] * 256 / vmax                (256 at the largest)
//   O^T [d_v x 2 NR] = V8^T . (Phi, Plo)^T                   (tcgen05.mma, M=128)
//   m_a              = max(m_old, y_a)                       (of the tiles so far)
//   l_a              = l_a * 2^(m_old - m) + sum_p w * 2^(y_a - m)
//   o_a              = o_a * 2^(m_old - m) + (Ohi + Olo / 16) * 2^(y_a - m) * vmax / 256
//
// qs[a] is a power of two that puts the row's largest value into [128, 256),
// so scaling loses nothing.  The pieces of P have e4m3's short range, not
// bf16's: below 2^-6 their step stays at 2^-13.  So P is taken against its own
// tile's largest product of weight and V scale, and a term loses more than its
// 8 bits only where it is below 2^-14 of the tile's largest (by 2^-22 of that
// at most).  Taken against the running maximum and the largest scale apart,
// one dominant early position with a small V row wiped out all later tiles:
// 24 % of the output at 32,768 positions, 72 % at 131,072.  The logarithm only
// picks y_a, which cancels; it is held at -64 or above, so w stays below 2^64.
//
// Roles (one persistent CTA per SM; 128 threads and 128 for every eight rows):
//   warp 0     TMA: K and V rows of a tile (boxes of a block's rows, 128- or
//              64-byte swizzle) into a three-stage ring, one lane per block;
//              the tile's scales by 16-byte copies
//   warp 1     issues the S products, warp 2 the O products
//   warp 3     splits a segment's query rows into e4m3 pieces in shared
//              memory, up to two segments ahead
//   warps 4-7  softmax, correction, output of eight query rows (8-11, ... the
//              next eight): thread x holds positions x and x + 128 of S,
//              column x of O
// P is written over the stage's K rows, which S no longer needs.
//
// The tiles of all units are laid end to end and dealt out evenly (Walker); a
// unit cut between CTAs leaves partial results, joined by the combine kernel.
//
// Bound by HBM where sequences are many and long: b = 32, L = 8,192, h = 64,
// g = 8, d = 128: 89.5 us, 6,200 GB/s (graph replay; 88.9 with the weights
// against the running maximum).  A few tiles a CTA: start, first tile and join
// (24 ragged sequences of 512 to 32,766, g = 4, two tokens of seven heads: 43
// us, 3,550 GB/s, 42 with the running maximum; 32-row blocks also cost the TMA
// warp sixteen copies a tile at ~100 cycles each).
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/gqa.h"
#include "gqa_internal.h"
#include "serve_device.cuh"

namespace gqa {
namespace {

constexpr int kTile = 256;   // positions per tile
constexpr int kHalf = 128;   // positions per S product
constexpr int kRing = 3;
constexpr float kLo = 16.f;  // the low piece's factor

template <int NR, int DK, int DV>
struct F8Cfg {
  // softmax warpgroups of eight query rows each: a warpgroup's time per tile
  // (one warp to a sub-partition, long dependent chains) is what bounds the
  // loop.  Sixteen rows on one warpgroup: 51 us where two took 43 (24 ragged
  // sequences of 512 to 32,766, g = 4, two tokens of seven heads)
  static constexpr int HP = 8;
  static constexpr int NWG = NR / HP;
  static constexpr int RP = NR < 16 ? 16 : NR;     // rows of a piece (padded)
  static constexpr int N = 2 * RP;                 // MMA columns: hi rows, lo rows
  static constexpr int THREADS = 128 + 128 * NWG;
  static constexpr int K_BYTES = kTile * DK, V_BYTES = kTile * DV;
  // (d_v = 64: the O product's upper half reads past the V rows, within the
  // shared memory that follows)
  static constexpr int STAGE = K_BYTES + V_BYTES;
  static constexpr int Q_BYTES = N * DK;
  static constexpr int OFF_Q = kRing * STAGE;
  static constexpr int OFF_TAIL = OFF_Q + 2 * Q_BYTES;
  static constexpr int OFF_PAD = OFF_TAIL + (DV == 64 ? V_BYTES : 0);
  static constexpr int OFF_SC = OFF_PAD;                        // float [kRing][2][kTile]
  static constexpr int OFF_RED = OFF_SC + kRing * 2 * kTile * 4;  // [NWG][2][HP][4]
  // of a query row and tile: its reference y, the running maximum m, and the
  // factors 2^(m_old - m) of what is held and 2^(y - m) of the tile's
  static constexpr int OFF_REF = OFF_RED + NWG * 2 * HP * 16;   // float [2][NR] each
  static constexpr int OFF_RUN = OFF_REF + 2 * NR * 4;
  static constexpr int OFF_ALPHA = OFF_RUN + 2 * NR * 4;
  static constexpr int OFF_PART = OFF_ALPHA + 2 * NR * 4;
  static constexpr int OFF_QS = OFF_PART + 2 * NR * 4;          // float [2][NR]
  static constexpr int OFF_COL = OFF_QS + 2 * NR * 4;           // int [2][NR]
  static constexpr int OFF_BAR = (OFF_COL + 2 * NR * 4 + 15) / 16 * 16;
  static constexpr int FULL_K = 0, FULL_V = kRing, EMPTY = 2 * kRing, SC_FULL = 3 * kRing,
                       Q_FULL = 4 * kRing,
                       Q_EMPTY = Q_FULL + 2, S_FULL = Q_EMPTY + 2, S_FREE = S_FULL + 2,
                       P_READY = S_FREE + 2, O_FULL = P_READY + 2, O_FREE = O_FULL + 2,
                       DRAIN = O_FREE + 2, NBAR = DRAIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int SMEM = OFF_MISC + 16;
  static constexpr int T_S = 0, T_O = 4 * N;       // TMEM: S [2][2] and O [2] of N columns
  static constexpr int NCOLS = 6 * N <= 256 ? 256 : 512;
  static constexpr uint32_t K_SWZ = DK == 128 ? SWZ_128B : SWZ_64B;
  static constexpr uint32_t V_SWZ = DV == 128 ? SWZ_128B : SWZ_64B;
  static constexpr uint32_t P_SWZ = N == 32 ? SWZ_32B : SWZ_64B;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(6 * N <= NCOLS, "TMEM columns");
};

struct F8Params {
  const __nv_bfloat16* q;
  const float *k_scale, *v_scale;
  const int *lens, *table;
  int b, nq, h, g, r, cap;
  int bsz, max_blocks, num_blocks;
  float scale_log2;
  __nv_bfloat16* out;
  float *part_o, *part_ml;
  unsigned int* status;
  long long budget;
};

// N floats of shared memory (16-byte aligned) that every lane reads alike
template <int N>
__device__ __forceinline__ void load_all(float (&v)[N], const float* src) {
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    const float4 x = *reinterpret_cast<const float4*>(src + k);
    v[k] = x.x, v[k + 1] = x.y, v[k + 2] = x.z, v[k + 3] = x.w;
  }
}

// e4m3 x e4m3 -> fp32 descriptor: D fp32, both formats 0, A / B transposed
// (MN-major) or not
constexpr uint32_t idesc_e4m3(int m, int n, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// four values as e4m3 pieces: hi bytes, and lo bytes of 16 (x - hi)
__device__ __forceinline__ void split4(const float (&x)[4], uint32_t& hi, uint32_t& lo) {
  hi = e4m3_pack4(x[0], x[1], x[2], x[3]);
  const float2 a = e4m3_unpack2(hi), b = e4m3_unpack2(hi >> 16);
  lo = e4m3_pack4((x[0] - a.x) * kLo, (x[1] - a.y) * kLo, (x[2] - b.x) * kLo, (x[3] - b.y) * kLo);
}

template <int NR, int DK, int DV>
__global__ void __launch_bounds__(F8Cfg<NR, DK, DV>::THREADS, 1)
    decode_fp8_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const F8Params p) {
  using C = F8Cfg<NR, DK, DV>;
  constexpr int HP = C::HP, N = C::N, RP = C::RP, NWG = C::NWG;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t s_base = smem_u32(sm);
  if (s_base & 1023u) {  // never seen; the swizzled layouts need it
    if (threadIdx.x == 0) atomicOr(p.status, GQA_DEV_INTERNAL);
    pdl_wait();  // (what follows this grid is ordered behind what it followed)
    return;
  }
  auto BAR = [&](int k) -> uint32_t { return s_base + C::OFF_BAR + 8u * k; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  // (broadcast, so that what depends on it is known to be uniform)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int nr = p.nq * p.r;

  if (threadIdx.x == 0) {
    for (int k = 0; k < C::NBAR; ++k) {
      const bool by_warps = (k >= C::S_FREE && k < C::O_FULL) || (k >= C::O_FREE && k < C::DRAIN);
      const bool q_empty = k >= C::Q_EMPTY && k < C::S_FULL;  // softmax warps, last S product
      const bool scales = k >= C::SC_FULL && k < C::Q_FULL;  // the copying warp's lanes
      mbar_init(BAR(k), k == C::DRAIN ? 2
                        : scales      ? 32
                        : by_warps    ? 4 * NWG
                        : q_empty     ? 4 * NWG + 1
                                      : 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  // query row a = s * r + t: its token s, and the offset of its output row
  int* col_tok = reinterpret_cast<int*>(sm + C::OFF_COL);
  int* col_off = col_tok + NR;
  if (threadIdx.x >= 64 && threadIdx.x < 64 + NR) {
    const int a = threadIdx.x - 64, s = a / p.r;
    col_tok[a] = a < nr ? s : -(1 << 30);  // (a padded row sees nothing)
    col_off[a] = a < nr ? (s * p.h + (a - s * p.r)) * DV : 0;
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::NCOLS);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait_then_release();
  if (warp == 2 && blockIdx.x == 0) report_bad_lengths(p.lens, p.b, p.nq, p.cap, p.status);

  float* qs_sm = reinterpret_cast<float*>(sm + C::OFF_QS);  // the query rows' factors [2][NR]

  Walker w;
  w.init(p.lens, p.b, p.g, p.nq, p.cap, kTile, blockIdx.x, gridDim.x);
  Segment seg;
  auto wait = [&](int k, uint32_t phase) -> bool {
    return mbar_wait(BAR(k), phase & 1u, abort_flag, p.status, p.budget);
  };

  if (warp == 0) {
    // ============================ TMA producer ============================
    const uint64_t pol = policy_evict_first();
    const int oob_row = p.num_blocks * p.g * p.bsz;
    const int box = min(p.bsz, kTile);
    const int sub = kTile / box;  // boxes a tile
    const int sh = __ffs(p.bsz) - 1, mask = p.bsz - 1;  // (a power of two)
    uint32_t n = 0;
    bool ok = true;
    while (ok && w.next(seg)) {
      // the sequence's table entries, 64 at a time ahead of their use: no load
      // stands before a tile's copies
      PageCursor pc;
      pc.start(p.table + static_cast<size_t>(seg.i) * p.max_blocks,
               static_cast<int>((static_cast<unsigned>(seg.L) + mask) >> sh),
               (seg.lt0 * kTile) >> sh);
      for (int lt = seg.lt0; lt < seg.lt1; ++lt, ++n) {
        // the tile's blocks, one a lane; lane mm < sub: the pool row of box mm
        const int ent = pc.get_lanes((lt * kTile) >> sh);
        const int pm = lt * kTile + lane * box;
        int cur = oob_row;
        if (lane < sub && pm < seg.L) {
          if (ent >= 0 && ent < p.num_blocks)
            cur = (ent * p.g + seg.j) * p.bsz + (pm & mask);
          else
            atomicOr(p.status, GQA_DEV_BAD_BLOCK);
        }
        const int st = n % kRing;
        ok = __all_sync(0xffffffffu, wait(C::EMPTY + st, ((n / kRing) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(BAR(C::FULL_K + st), C::K_BYTES);
          mbar_arrive_expect_tx(BAR(C::FULL_V + st), C::V_BYTES);
        }
        __syncwarp();
        const uint32_t dst = s_base + st * C::STAGE;
        if (lane < sub) {
          tma_load_2d(dst + lane * box * DK, &tm_k, BAR(C::FULL_K + st), 0, cur, pol);
          tma_load_2d(dst + C::K_BYTES + lane * box * DV, &tm_v, BAR(C::FULL_V + st), 0, cur, pol);
        }
        // the scales of this lane's eight positions (past L_i, or through a
        // bad entry: none).  Four instructions a tile; as two more bulk copies a
        // block (~100 cycles of the issuing warp each) they took as long, 41 to
        // 42 us with 32-row blocks.
        const int pos = lt * kTile + lane * 8;
        const int blk = __shfl_sync(0xffffffffu, ent, (lane * 8) >> sh);
        if (pos < seg.L && blk >= 0 && blk < p.num_blocks) {
          const size_t at = (static_cast<size_t>(blk) * p.g + seg.j) * p.bsz + (pos & mask);
          const uint32_t sd = s_base + C::OFF_SC + (st * 2 * kTile + lane * 8) * 4;
          async_copy16(sd, p.k_scale + at);
          async_copy16(sd + 16, p.k_scale + at + 4);
          async_copy16(sd + kTile * 4, p.v_scale + at);
          async_copy16(sd + kTile * 4 + 16, p.v_scale + at + 4);
        }
        async_copies_arrive(BAR(C::SC_FULL + st));
      }
    }
    async_copies_wait();
    if (!ok) {  // copies in flight must land before the CTA exits (bounded)
      const long long t0 = clock64();
      for (int s = 0; s < kRing; ++s) {
        if (n <= static_cast<uint32_t>(s)) continue;
        const uint32_t last = (n - 1 - s) / kRing;
        while (!(mbar_try_wait(BAR(C::FULL_K + s), last & 1) &&
                 mbar_try_wait(BAR(C::FULL_V + s), last & 1)) &&
               clock64() - t0 < p.budget) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    // ============================ MMA issuers =============================
    // (the whole warp walks with warp-uniform values and one elected lane
    // issues: from a single lane's branch the operands take a detour into the
    // uniform registers that costs several times what a product runs)
    constexpr uint32_t kIdescS = idesc_e4m3(128, N, 0, 0);
    constexpr uint32_t kIdescO = idesc_e4m3(128, N, 1, 1);
    const bool s_role = warp == 1;
    const uint64_t dq = smem_desc(s_base + C::OFF_Q, 16, 8 * DK, C::K_SWZ);
    const uint64_t dk = smem_desc(s_base, 16, 8 * DK, C::K_SWZ);
    // A = V^T: 128 head-dim columns contiguous; B = P^T: N columns contiguous,
    // over the stage's K rows
    const uint64_t dv = smem_desc(s_base + C::K_BYTES, C::V_BYTES, 8 * DV, C::V_SWZ);
    const uint64_t dp = smem_desc(s_base, kTile * N, 8 * N, C::P_SWZ);
    uint32_t nb = 0, nph = 0;           // tile's buffer, and its phase
    uint32_t st = 0, sph = 0;           // ring slot, and its phase
    uint32_t qb = 0, qph = 0;
    bool ok = true;
    while (ok && w.next(seg)) {
      const int T = __shfl_sync(0xffffffffu, seg.lt1 - seg.lt0, 0);
      if (s_role) ok = __all_sync(0xffffffffu, wait(C::Q_FULL + qb, qph));
      for (int t = 0; t < T && ok; ++t) {
        const uint32_t at = st * (C::STAGE >> 4);
        if (s_role) {
          ok = __all_sync(0xffffffffu,
                          wait(C::FULL_K + st, sph) && wait(C::S_FREE + nb, nph ^ 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t b0 = dq + qb * (C::Q_BYTES >> 4), a0 = dk + at;
          if (elect_one()) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int kk = 0; kk < DK / 32; ++kk)  // 32 head-dim columns a step
                mma_f8(tmem + C::T_S + (nb * 2 + hf) * N, a0 + ((hf * kHalf * DK + kk * 32) >> 4),
                       b0 + ((kk * 32) >> 4), kIdescS, kk > 0 ? 1u : 0u);
            mma_commit(BAR(C::S_FULL + nb));
            if (t == T - 1) mma_commit(BAR(C::Q_EMPTY + qb));
          }
        } else {
          ok = __all_sync(0xffffffffu, wait(C::FULL_V + st, sph) &&
                                           wait(C::O_FREE + nb, nph ^ 1) &&
                                           wait(C::P_READY + nb, nph));
          if (!ok) break;
          tc_fence_after();
          const uint64_t a0 = dv + at, b0 = dp + at;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kTile / 32; ++kk)  // 32 positions a step
              mma_f8(tmem + C::T_O + nb * N, a0 + ((kk * 32 * DV) >> 4), b0 + ((kk * 32 * N) >> 4),
                     kIdescO, kk > 0 ? 1u : 0u);
            mma_commit(BAR(C::O_FULL + nb));
            mma_commit(BAR(C::EMPTY + st));
          }
        }
        __syncwarp();
        if (nb ^= 1; nb == 0) nph ^= 1;
        if (++st == kRing) {
          st = 0;
          sph ^= 1;
        }
      }
      if (qb ^= 1; qb == 0) qph ^= 1;
    }
    // every product has to be finished before tensor memory is released
    if (elect_one()) {
      mma_commit(BAR(C::DRAIN));
      const long long t0 = clock64();
      while (!mbar_try_wait(BAR(C::DRAIN), 0) && clock64() - t0 < p.budget) {
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ============================ query rows ==============================
    constexpr int EPL = DK / 32;  // elements a lane; a warp to a row, eight rows at a time
    uint32_t k = 0;
    bool ok = true;
    while (w.next(seg)) {
      const uint32_t qb = k & 1;
      ok = __all_sync(0xffffffffu, wait(C::Q_EMPTY + qb, (k >> 1) ^ 1));
      if (!ok) break;
      const __nv_bfloat16* q0 =
          p.q + (static_cast<size_t>(seg.i) * p.nq * p.h + seg.j * p.r) * DK + lane * EPL;
      uint8_t* dst = sm + C::OFF_Q + qb * C::Q_BYTES;
      // K-major rows of DK bytes, 16-byte chunks swizzled by the row
      auto put = [&](int rr, uint32_t v) {
        const int byte = lane * EPL, chunk = byte >> 4;
        const int phys = DK == 128 ? (chunk ^ (rr & 7)) : (chunk ^ ((rr >> 1) & 3));
        uint8_t* d = dst + rr * DK + phys * 16 + (byte & 15);
        if constexpr (EPL == 4)
          *reinterpret_cast<uint32_t*>(d) = v;
        else
          *reinterpret_cast<uint16_t*>(d) = static_cast<uint16_t>(v);
      };
      for (int a0 = 0; a0 < RP; a0 += 8) {
        uint32_t raw[8][2];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          raw[t][0] = raw[t][1] = 0u;
          const int a = a0 + t;
          if (a < nr) {
            // (col_off counts rows of DV elements)
            const __nv_bfloat16* src = q0 + static_cast<size_t>(col_off[a] / DV) * DK;
            if constexpr (EPL == 4) {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
              raw[t][0] = v.x;
              raw[t][1] = v.y;
            } else {
              raw[t][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
            }
          }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const int a = a0 + t;
          float x[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[2 * e] = __uint_as_float(raw[t][e] << 16);
            x[2 * e + 1] = __uint_as_float(raw[t][e] & 0xFFFF0000u);
          }
          const float amax =
              warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
          // 2^ke * amax in [128, 256)
          int ke = 0;
          if (amax > 0.f && amax < INFINITY) ke = min(max(7 - ilogbf(amax), -126), 126);
          // (an infinity would saturate to 448: the row is NaN, as its logits
          // are in the formula)
          const float up = amax < INFINITY ? ldexpf(1.f, ke) : NAN;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] *= up;
          uint32_t hi, lo;
          split4(x, hi, lo);
          put(a, hi);
          put(RP + a, lo);
          if (lane == 0 && a < NR)
            qs_sm[qb * NR + a] = ldexpf(1.f, -ke) * p.scale_log2;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::Q_FULL + qb));
      ++k;
    }
    __syncwarp();
  } else {
    // ====================== softmax, correction, output ===================
    const int wg = (warp - 4) >> 2, wq = warp & 3;
    const int qd = warp & 3;               // TMEM lane quarter of this warp
    const int row = qd * 32 + lane;        // position (S), column (O)
    const int h0 = wg * HP;                // first query row of the warpgroup
    const int bar_id = 1 + wg;
    const uint32_t lane_off = static_cast<uint32_t>(qd * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::T_S + h0, tO = tmem + lane_off + C::T_O + h0;
    float* red = reinterpret_cast<float*>(sm + C::OFF_RED) + wg * 2 * HP * 4;
    float* ref_sm = reinterpret_cast<float*>(sm + C::OFF_REF);
    float* run_sm = reinterpret_cast<float*>(sm + C::OFF_RUN);
    float* alpha_sm = reinterpret_cast<float*>(sm + C::OFF_ALPHA);
    float* part_sm = reinterpret_cast<float*>(sm + C::OFF_PART);
    float l[HP], o[HP];
    float vm = 0.f, vm_last = 0.f;  // largest V scale of the tile, and of the one before
    float m_own = -INFINITY;  // running maximum of query row h0 + row (row < HP)
    uint32_t n = 0, k = 0;
    bool ok = true;

    // o = o * alpha + tile mt's product, whose largest V scale is vt
    auto correct = [&](uint32_t mt, float vt) {
      const uint32_t nb = mt & 1;
      ok = ok && __all_sync(0xffffffffu, wait(C::O_FULL + nb, mt >> 1));
      if (!ok) return;
      tc_fence_after();
      float hi[HP], lo[HP];
#pragma unroll
      for (int c = 0; c < HP; c += 8) {
        tmem_ld8(tO + nb * N + c, hi + c);
        tmem_ld8(tO + nb * N + RP + c, lo + c);
      }
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::O_FREE + nb));
      const float vf = vt * (1.f / 256.f);
      float al[HP], pt[HP];
      load_all(al, alpha_sm + nb * NR + h0);
      load_all(pt, part_sm + nb * NR + h0);
#pragma unroll
      for (int e = 0; e < HP; ++e)
        o[e] = fmaf(o[e], al[e], fmaf(lo[e], 1.f / kLo, hi[e]) * (pt[e] * vf));
    };

    // A warp whose wait gave up walks on without waiting, reading or writing
    // outputs: the warpgroup's named barriers need all its warps.
    while (w.next(seg)) {
      const uint32_t qb = k & 1;
      const int first_new = seg.L - p.nq;  // position of new token 0
      ok = __all_sync(0xffffffffu, ok && wait(C::Q_FULL + qb, k >> 1));  // (the rows' factors)
      m_own = -INFINITY;
#pragma unroll
      for (int e = 0; e < HP; ++e) l[e] = o[e] = 0.f;

      for (int lt = seg.lt0; lt < seg.lt1; ++lt, ++n) {
        const uint32_t nb = n & 1;
        const int st = n % kRing;
        const int valid = min(kTile, seg.L - lt * kTile);
        ok = __all_sync(0xffffffffu, ok && wait(C::S_FULL + nb, n >> 1) &&
                                         wait(C::SC_FULL + st, n / kRing));
        tc_fence_after();
        const float* sc = reinterpret_cast<const float*>(sm + C::OFF_SC) + st * 2 * kTile + row;
        float ks[2], vs[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const bool in = row + hf * kHalf < valid;
          ks[hf] = in ? sc[hf * kHalf] : 0.f;
          vs[hf] = in ? sc[kTile + hf * kHalf] : 0.f;
        }
        float x[2][HP], lo[2][HP];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int c = 0; c < HP; c += 8) {
            tmem_ld8(tS + (nb * 2 + hf) * N + c, &x[hf][c]);
            tmem_ld8(tS + (nb * 2 + hf) * N + RP + c, &lo[hf][c]);
          }
        // the tile's largest V scale, every warp for itself (while S is
        // on its way)
        vm_last = vm;
        vm = 0.f;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int p0 = hf * kHalf + 4 * lane;
          const float4 v = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(sm + C::OFF_SC) + (st * 2 + 1) * kTile + p0);
          vm = fmaxf(vm, p0 < valid ? fabsf(v.x) : 0.f);
          vm = fmaxf(vm, p0 + 1 < valid ? fabsf(v.y) : 0.f);
          vm = fmaxf(vm, p0 + 2 < valid ? fabsf(v.z) : 0.f);
          vm = fmaxf(vm, p0 + 3 < valid ? fabsf(v.w) : 0.f);
        }
        vm = warp_max(vm);
        // (scales so small that the factor would overflow: scaled up first)
        const float up = vm < 0x1p-60f ? 0x1p60f : 1.f;
        const float vinv = vm > 0.f ? __fdividef(256.f, vm * up) : 0.f;
        float fv[2], lv[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          fv[hf] = vs[hf] * up * vinv;  // 256 vs / vmax
          lv[hf] = fmaxf(__log2f(fabsf(fv[hf])) - 8.f, -64.f);
        }
        tmem_wait_ld();
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int e = 0; e < HP; ++e) x[hf][e] = fmaf(lo[hf][e], 1.f / kLo, x[hf][e]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::S_FREE + nb));
        const float* qs = qs_sm + qb * NR + h0;
        if ((lt + 1) * kTile <= first_new + 1) {
          // (uniform) every query row sees every position of the tile
#pragma unroll
          for (int e = 0; e < HP; ++e) {
            const float f = qs[e];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              x[hf][e] = h0 + e < nr ? x[hf][e] * (ks[hf] * f) : -INFINITY;
          }
        } else {
#pragma unroll
          for (int e = 0; e < HP; ++e) {
            const int last = first_new + col_tok[h0 + e];  // last position the row sees
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const bool seen = lt * kTile + row + hf * kHalf <= last;
              x[hf][e] = seen ? x[hf][e] * (ks[hf] * qs[e]) : -INFINITY;
            }
          }
        }
        // ---- maxima over the tile's positions ----
        float mine = -INFINITY;
#pragma unroll
        for (int e = 0; e < HP; ++e) {
          const float wm = warp_max(fmaxf(x[0][e] + lv[0], x[1][e] + lv[1]));
          if (lane == e) mine = wm;
        }
        float* rb = red + nb * HP * 4;
        if (lane < HP) rb[lane * 4 + wq] = mine;
        named_bar_sync(bar_id, 128);
        if (row < HP) {
          const float4 v = *reinterpret_cast<const float4*>(rb + 4 * row);
          const float y = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
          const float mn = fmaxf(m_own, y);
          const float run = mn == -INFINITY ? 0.f : mn;  // nothing seen yet
          const int a = nb * NR + h0 + row;
          ref_sm[a] = y == -INFINITY ? 0.f : y;          // nothing of this tile
          run_sm[a] = run;
          alpha_sm[a] = ex2(m_own - run);
          part_sm[a] = ex2(y - run);
          m_own = mn;
        }
        named_bar_sync(bar_id, 128);
        float ref[HP], al[HP], pt[HP];
        load_all(ref, ref_sm + nb * NR + h0);
        load_all(al, alpha_sm + nb * NR + h0);
        load_all(pt, part_sm + nb * NR + h0);
#pragma unroll
        for (int e = 0; e < HP; ++e) {
          const float w0 = ex2(x[0][e] - ref[e]), w1 = ex2(x[1][e] - ref[e]);
          l[e] = fmaf(l[e], al[e], (w0 + w1) * pt[e]);
          x[0][e] = w0 * fv[0];
          x[1][e] = w1 * fv[1];
        }
        // ---- P pieces: a row of N bytes per position, 16-byte chunks ----
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int pr = row + hf * kHalf;
          uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int c = 0; c < HP / 4; ++c) {
            const float v[4] = {x[hf][4 * c], x[hf][4 * c + 1], x[hf][4 * c + 2],
                                x[hf][4 * c + 3]};
            split4(v, hi[c], lo[c]);
          }
          const uint32_t base = s_base + st * C::STAGE + pr * N;
          // (one warpgroup: the chunk's rows 8-15 are padding, zeros)
          auto put = [&](int cg, const uint32_t (&v)[4]) {
            const int phys = N == 32 ? (cg ^ ((pr >> 2) & 1)) : (cg ^ ((pr >> 1) & 3));
            if constexpr (NWG == 1)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + phys * 16),
                           "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                           : "memory");
            else
              asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(base + phys * 16 +
                                                                    (wg & 1) * 8),
                           "r"(v[0]), "r"(v[1])
                           : "memory");
          };
          if constexpr (NWG == 1) {
            put(0, hi);
            put(1, lo);
          } else {
            put(wg >> 1, hi);
            put(RP / 16 + (wg >> 1), lo);
          }
        }
        // ---- V rows past L_i hold anything: zero them ----
        if (wg == 0 && valid < kTile) {
          ok = __all_sync(0xffffffffu, ok && wait(C::FULL_V + st, n / kRing));
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int pr = row + hf * kHalf;
            if (ok && pr >= valid) {
              const uint32_t dst = s_base + st * C::STAGE + C::K_BYTES + pr * DV;
#pragma unroll
              for (int c = 0; c < DV / 16; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + 16 * c),
                             "r"(0u)
                             : "memory");
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::P_READY + nb));
        if (lt > seg.lt0) correct(n - 1, vm_last);
        if (lt == seg.lt1 - 1) correct(n, vm);
      }
      ++k;
      if (lane == 0) mbar_arrive(BAR(C::Q_EMPTY + qb));
      // ---- segment end: the row sums across the warpgroup, then the output
      // or a partial ----
      const uint32_t nb = (n - 1) & 1;
      float* rb = red + nb * HP * 4;
      {
        // each round trades half of the sums still held with a partner lane;
        // lane x ends with the warp's sum of row x / (32 / HP)
        float v[HP];
#pragma unroll
        for (int e = 0; e < HP; ++e) v[e] = l[e];
#pragma unroll
        for (int o2 = 16, nv = HP; o2 >= 32 / HP; o2 >>= 1, nv >>= 1) {
          const bool up = (lane & o2) != 0;
#pragma unroll
          for (int e = 0; e < nv / 2; ++e) {
            const float send = up ? v[e] : v[e + nv / 2];
            const float keep = up ? v[e + nv / 2] : v[e];
            v[e] = keep + __shfl_xor_sync(0xffffffffu, send, o2);
          }
        }
#pragma unroll
        for (int o2 = 16 / HP; o2 > 0; o2 >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o2);
        if (lane % (32 / HP) == 0) rb[(lane / (32 / HP)) * 4 + wq] = v[0];
      }
      named_bar_sync(bar_id, 128);
      const bool whole = seg.lt0 == 0 && seg.lt1 == seg.ti;
      const int u = seg.i * p.g + seg.j;
      const size_t slot = static_cast<size_t>(u) + blockIdx.x;
      __nv_bfloat16* obase =
          p.out + (static_cast<size_t>(seg.i) * p.nq * p.h + seg.j * p.r) * DV + row;
#pragma unroll
      for (int e = 0; e < HP; ++e) {
        const int a = h0 + e;
        if (ok && a < nr) {
          const float4 v = *reinterpret_cast<const float4*>(rb + 4 * e);
          const float sum = (v.x + v.y) + (v.z + v.w);
          if (whole) {
            if (row < DV) obase[col_off[a]] = __float2bfloat16_rn(o[e] * (1.f / sum));
          } else {
            const size_t sl = slot * nr + a;
            if (row < DV) p.part_o[sl * DV + row] = o[e];
            if (row == 0) {
              p.part_ml[2 * sl] = sum > 0.f ? run_sm[nb * NR + a] : -INFINITY;
              p.part_ml[2 * sl + 1] = sum;
            }
          }
        }
      }
      // (the next tile's exchange uses the other half of `red`, and its
      // barriers come before this half is written again)
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::NCOLS);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct F8Call {
  const void *q, *k, *v;
  const float *k_scale, *v_scale;
  const int *table, *lens;
  int b, n, h, g, dk, dv;
  float scale;
  void* out;
  int bsz, max_blocks, num_blocks, dtype;
  void* ws;
  long long ws_bytes;
};

struct F8Plan {
  long long nc = 0;
  size_t ml_at = 0, bytes = 0;
};

F8Plan f8_plan(int b, int n, int h, int g, int dv, long long cap, int num_sms) {
  F8Plan pl;
  const long long units = static_cast<long long>(b) * g;
  pl.nc = num_sms;
  const long long tiles = units * ((cap + kTile - 1) / kTile);
  if (pl.nc > tiles) pl.nc = tiles;
  const size_t rows = static_cast<size_t>(units + pl.nc) * n * (h / g);
  pl.ml_at = (rows * dv * sizeof(float) + 255) & ~size_t(255);
  pl.bytes = (pl.ml_at + rows * 2 * sizeof(float) + 255) & ~size_t(255);
  return pl;
}

int f8_shape_check(int b, int n, int h, int g, int dk, int dv, long long cap) {
  if (b < 1 || n < 1 || h < 1 || g < 1 || dk < 1 || dv < 1 || cap < 1 || h % g != 0 || n > cap)
    return GQA_ERR_SHAPE;
  if (cap > 0x7FFFFF00ll || static_cast<long long>(b) * n * h > 0x7FFFFFFFll)
    return GQA_ERR_SHAPE;
  if (b > 65535 || static_cast<long long>(n) * (h / g) > 32 || (dk != 64 && dk != 128) ||
      (dv != 64 && dv != 128))
    return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}

int f8_check(const F8Call& x) {
  if (!x.q || !x.k || !x.v || !x.k_scale || !x.v_scale || !x.lens || !x.out || !x.ws)
    return GQA_ERR_NULL;
  if (x.dtype != GQA_F32 && x.dtype != GQA_BF16 && x.dtype != GQA_F16) return GQA_ERR_DTYPE;
  if (int e = f8_shape_check(x.b, x.n, x.h, x.g, x.dk, x.dv,
                             static_cast<long long>(x.max_blocks) * x.bsz))
    return e;
  if (x.dtype != GQA_BF16) return GQA_ERR_UNSUPPORTED;
  auto off = [](const void* p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) != 0; };
  if (off(x.q, 15) || off(x.k, 15) || off(x.v, 15) || off(x.out, 15) || off(x.k_scale, 15) ||
      off(x.v_scale, 15) || off(x.lens, 3) || off(x.ws, 255))
    return GQA_ERR_ALIGN;
  return GQA_OK;
}

template <int NR, int DK, int DV>
cudaError_t launch_f8(const F8Call& x, const F8Plan& pl, F8Params& p, cudaStream_t st) {
  using C = F8Cfg<NR, DK, DV>;
  CUtensorMap mk, mv;
  const uint64_t rows = static_cast<uint64_t>(x.num_blocks) * x.g * x.bsz;
  const uint32_t box_rows = x.bsz < kTile ? x.bsz : kTile;
  if (!encode_u8_map(&mk, x.k, DK, rows, box_rows) || !encode_u8_map(&mv, x.v, DV, rows, box_rows))
    return cudaErrorInvalidValue;
  auto kern = decode_fp8_kernel<NR, DK, DV>;
  static std::atomic<unsigned long long> configured{0};  // devices done, this variant
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(configured.load() & (1ull << dev))) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    configured.fetch_or(1ull << dev);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pl.nc));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, mk, mv, p);
}

template <int NR>
cudaError_t launch_f8_dims(const F8Call& x, const F8Plan& pl, F8Params& p, cudaStream_t st) {
  if (x.dk == 128)
    return x.dv == 128 ? launch_f8<NR, 128, 128>(x, pl, p, st)
                       : launch_f8<NR, 128, 64>(x, pl, p, st);
  return x.dv == 128 ? launch_f8<NR, 64, 128>(x, pl, p, st) : launch_f8<NR, 64, 64>(x, pl, p, st);
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

int gqa_decode_attn_fp8_paged(const void* q, const void* k_pool, const void* v_pool,
                              const float* k_scale, const float* v_scale,
                              const int32_t* block_table, const int32_t* seq_lens, int b, int n,
                              int h, int g, int d_k, int d_v, float scale, void* out,
                              int block_size, int max_blocks, int num_blocks, int dtype,
                              void* workspace, long long workspace_bytes, void* stream) {
  if (int e = paged_args_check(block_table, g, block_size, max_blocks, num_blocks)) return e;
  const F8Call x = {q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, b, n, h, g, d_k,
                    d_v, scale, out, block_size, max_blocks, num_blocks, dtype, workspace,
                    workspace_bytes};
  if (int e = f8_check(x)) return e;
  int num_sms = 0;
  F8Params p;
  if (int e = device_query(&num_sms, &p.status)) return e;
  const int cap = max_blocks * block_size;
  const F8Plan pl = f8_plan(b, n, h, g, d_v, cap, num_sms);
  if (workspace_bytes < static_cast<long long>(pl.bytes)) return GQA_ERR_SCRATCH_LIMIT;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.lens = seq_lens;
  p.table = block_table;
  p.b = b;
  p.nq = n;
  p.h = h;
  p.g = g;
  p.r = h / g;
  p.cap = cap;
  p.bsz = block_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.ml_at);
  p.budget = kKernelWaitBudget;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rows = n * (h / g);
  cudaError_t e = rows <= 8    ? launch_f8_dims<8>(x, pl, p, st)
                  : rows <= 16 ? launch_f8_dims<16>(x, pl, p, st)
                               : launch_f8_dims<32>(x, pl, p, st);
  if (e != cudaSuccess) return GQA_ERR_CUDA;
  DecodeLaunch a = {};
  a.seq_lens = seq_lens;
  a.b = b;
  a.h = h;
  a.g = g;
  a.dv = d_v;
  a.nq = n;
  a.cap = cap;
  a.dtype = dtype;
  a.out = out;
  a.part_o = p.part_o;
  a.part_ml = p.part_ml;
  a.nc = static_cast<int>(pl.nc);
  a.stream = st;
  return launch_unit_combine(a, kTile) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

int gqa_decode_attn_fp8_workspace(int b, int n, int h, int g, int d_k, int d_v, long long cap,
                                  int num_sms, long long* bytes) {
  if (!bytes) return GQA_ERR_NULL;
  if (num_sms < 0) return GQA_ERR_SHAPE;
  if (int e = f8_shape_check(b, n, h, g, d_k, d_v, cap)) return e;
  if (num_sms == 0) {
    unsigned int* status = nullptr;
    if (int e = device_query(&num_sms, &status)) return e;
  }
  *bytes = static_cast<long long>(f8_plan(b, n, h, g, d_v, cap, num_sms).bytes);
  return GQA_OK;
}

}  // extern "C"
