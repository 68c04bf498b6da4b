// chunk_kernel.cuh - attention of packed chunks of new tokens (prompts,
// prompt chunks, single tokens, mixed) over a part of a contiguous or paged
// 16-bit cache, on the tcgen05 tensor cores.
//
// A unit is a block of query rows of one (sequence, KV head): the r = h / g
// query heads of a group share K and V, so rows are packed token-major (row
// s * r + a), tq = 128 / r tokens to an M = 128 tile and two tiles ("sides" A
// and B) to a unit.  Per 128 cached positions and side:
//
//   S [128 x 128] = Q_side . K_tile^T             (tcgen05.mma, operands in shared memory)
//   P = exp2(scale*log2e * S - m)                 (CUDA cores; one thread per row)
//   O [128 x d_v] += P . V_tile                   (tcgen05.mma, P in tensor memory)
//
// While one side's softmax runs, the tensor cores work on the other side.
// m is a row's running maximum, raised only when the exponent grows past it by
// more than a few powers of two (the lazy rescaling known from published
// attention kernels); O is rescaled in tensor memory on those occasions alone.
// P is rounded to the cache's type for the product (the row sum adds the fp32
// values): to bf16's range whatever is raised, so P may grow to 2^8.  fp16 ends
// at 2^-14 (2^-25 with subnormals), where the weights of a long cache behind
// one dominant position lie: there P is taken 2^11 higher and m raised past
// 2^4, which uses the range up to 2^15 and keeps weights down to 2^-25 of the
// largest whole (below, they are off by up to 2^-36 of it).  The factor 2^11 is
// in l and O alike and cancels.
//
// Roles (384 threads, one persistent CTA per SM):
//   warps 0-3  softmax of side A, output; thread = query row = TMEM lane
//   warps 4-7  the same for side B
//   warp 8     issues every product: the whole warp walks the loop and one
//              elected lane issues (from one lane's branch eight products took
//              460 cycles to issue, as long as they run)
//   warp 10    TMA: the sides' query rows once per unit, K and V tiles into a
//              ring (64-column boxes, 128-byte swizzle); finds the run's start
//              and works out each unit for the others (SegPlan)
//   warp 11    the run's end (in the same instructions as its start), then the V
//              rows that nobody sees: zeroed in shared memory
//   (warp 9 checks the lengths: registers are dealt out by warpgroups)
// A unit whose rows fit one side runs as twins: both sides hold its rows and take
// its tiles by turns.  Units of twins follow one another without a break (their
// query rows are staged once, in the two buffers by turns), and softmax warps
// without a row only pass the barriers.
//
// What runs once a unit or once a launch is written for few instructions: it is
// fetched anew each time, at a few hundred cycles a line, and stands on the
// critical path between two units.  (The walk of chunk_part.cu with its scans and
// divisions inlined five times cost 15 us a launch; the softmax's own look at a
// new unit 1.5 us from one unit to the next.)  The warps' waits are the whole
// warp's, so a single lane arrives by a predicated instruction, not behind a
// branch: with the branch one lane ran ahead of the others in some builds.
// TMEM columns: S_A 0-127, S_B 128-255 (each holds P, two 16-bit values a
// column, once its S has been read), O_A 256.., O_B 384...
//
// Work split.  A unit has as many tiles as its last token sees.  All units are
// laid end to end, and each CTA takes a run of equal work, so the triangle of
// a causal prompt, ragged batches and a few long sequences all spread evenly;
// a run's ends snap to a unit's edge when it is close.  A unit cut by a run's
// end leaves partial results (row maximum, sum, unnormalised
// output, all fp32) in the workspace, and a second small kernel joins them.
//
// Rows that no token of the sequence sees: masked out of S, their V rows zeroed in
// shared memory.
//
// Used by chunk_part.cu alone, whose PartWalk (the one Walk there is; it stands
// behind the kernel, with its joins) gives the units, where their rows lie and what
// their tokens see.  chunk_attn.cu has a kernel of its own for causal chunks over the
// whole cache, with the same products and the same roles, but units looked at by each
// role for itself: on this kernel, without what is not needed there, a causal prompt of
// 8,192 took 731 us where that took 715, 32 mixed sequences 138.6 (134.8), packed
// short prompts 36.4 (34.6).  What both share is in chunk_common.cuh.  Figures of this
// one: chunk_part.cu.
#pragma once

#include "chunk_common.cuh"
#include "part_device.cuh"

namespace gqa {
namespace {

constexpr int kSegBytes = 112;  // of an announced segment
constexpr int kEdges = 8;         // V tiles to be zeroed in part: more than a ring holds of V
constexpr int kGrain = 64;        // positions of a box where a part of the cache is read, at most
template <int DK, int DV>
struct ChunkCfg {
  static constexpr int Q_BYTES = kM * DK * 2;  // one side
  static constexpr int SLOT = kN * (DK > DV ? DK : DV) * 2;
  // ring slots: K and V tiles by turns
  static constexpr int NS = DK == 128 ? 5 : (DV == 128 ? 6 : 10);
  static constexpr int OFF_RING = 2 * Q_BYTES;
  static constexpr int OFF_BAR = OFF_RING + NS * SLOT;
  static constexpr int FULL = 0, EMPTY = NS, Q_FULL = 2 * NS, Q_EMPTY = Q_FULL + 2,
                       S_FULL = Q_EMPTY + 2, P_READY = S_FULL + 2, O_DONE = P_READY + 2,
                       SEG_FULL = O_DONE + 2, SEG_EMPTY = SEG_FULL + kSegs,
                       V_EDGE = SEG_EMPTY + kSegs,
                       TWIN = V_EDGE + kEdges, RUN_END = TWIN + 2, DRAIN = RUN_END + 1,
                       NBAR = DRAIN + 1;
  static constexpr int OFF_SEG = (OFF_BAR + 8 * NBAR + 15) / 16 * 16;
  static constexpr int OFF_ML = OFF_SEG + kSegs * kSegBytes;  // float2 [2][kM]: twins' maxima, sums
  static constexpr int OFF_MISC = OFF_ML + 2 * kM * 8;  // TMEM address, abort flag; the run's end
  static constexpr int OFF_EDGE = OFF_MISC + 32;        // int4 [kEdges]
  static constexpr int SMEM = OFF_EDGE + 16 * kEdges;
  static_assert(NS / 2 < kEdges, "edges in flight");
  static constexpr int T_S = 0, T_O = 256;  // TMEM columns, 128 to a side
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct ChunkParams : ChunkArgs {
  // the part of the cache: tokens see their last `window` positions and
  // the first `head` ones, which are read from sequence head_seq (-1: each
  // from its own); positions below base_min belong to the head alone
  int window, head, head_seq, base_min;
  unsigned unit_inv;   // 2^32 / (2 tq), rounded up
  // the head may be attended by units of its own, over the rows of all
  // sequences, when those are group_rows or fewer (0: never); every unit leaves
  // partial results then
  int group_rows;
  int* cut;            // [2][2][group_rows * g]: a unit's first CTA (-1: not cut), its last
  float* row_ml;       // [2][group_rows * h][2] partial results of whole units
  float* row_o;        // [2][group_rows * h][d_v]
};

// What the products and the softmax need of a segment, worked out by the TMA warp
// ahead of time: what they would compute between two units stands on their
// critical path, and as code that runs once a unit it is fetched each time (1.5
// us from one unit to the next).
struct SegPlan {
  int T;         // tiles (0: no more)
  int twin, qb;  // a unit of twins; their query rows' buffer
  int step;      // positions from one of a side's tiles to its next
  int j;         // KV head
  int last;      // 1: the results are final
  int part;      // else the first partial row of the CTA's two units
  int by_row;    // 0: by CTA, 1, 2: by row, over the head, over the sequence's own
  int head, lo_min;
  struct Side {
    int nt;      // tiles
    int first;   // position of the first one
    int tokens;  // tokens with rows
    int row0;    // packed row of the first
    // token k sees [0, min(head, hi)) and [max(lo + k, lo_min), hi + k) of
    // the span; every token [0, all_head) and [all_lo, all_hi)
    int lo, hi, all_head, all_lo, all_hi;
  } side[2];
};
static_assert(sizeof(SegPlan) <= kSegBytes, "segment ring");

// desc of CTA c, beside a cut unit's: the rows of the head's own units, the same from
// every CTA
enum { D_ROWS = 5 };

template <typename T16, int DK, int DV, bool PAGED, class Walk>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_q1,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const ChunkParams p) {
  using C = ChunkCfg<DK, DV>;
  using Seg = typename Walk::Seg;
  using Plan = SegPlan;
  constexpr bool kBf16 = Half16<T16>::kBf16;
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

  if (threadIdx.x == 0) {
    for (int k = 0; k < C::NBAR; ++k)
      mbar_init(BAR(k), (k >= C::P_READY && k < C::O_DONE)                ? 4   // a side's warps
                        : (k >= C::SEG_EMPTY && k < C::SEG_EMPTY + kSegs) ? 9  // all its readers
                        : (k == C::TWIN || k == C::TWIN + 1)              ? 8  // both sides' warps
                                                                          : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 10 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_q1);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 8) tmem_alloc(smem_u32(tmem_slot), 512);
  __syncthreads();
  tc_fence_after();
  // (all of tensor memory is allocated, so it starts at address 0)
  constexpr uint32_t tmem = 0;
  if (*tmem_slot != tmem) {  // never seen
    if (threadIdx.x == 0) {
      atomicOr(p.status, GQA_DEV_INTERNAL);
      *abort_flag = 1;
    }
  }
  pdl_wait_then_release();

  auto seg_at = [&](uint32_t k) -> Plan* {
    return reinterpret_cast<Plan*>(sm + C::OFF_SEG + (k % kSegs) * kSegBytes);
  };
  auto wait = [&](int k, uint32_t phase) -> bool {
    return mbar_wait(BAR(k), phase & 1u, abort_flag, p.status, p.budget);
  };

  ChunkPos* const run_end = reinterpret_cast<ChunkPos*>(sm + C::OFF_MISC + 16);
  if (warp >= 8) {
    // (a warpgroup's four warps at the same instruction, as it has to be)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 9) {
      if (blockIdx.x == 0) Walk::report(p);
    } else if (warp >= 10) {
      // the run's start, and in warp 11 its end, in the same instructions
      Walk w(p);
      ChunkPos from;
      const bool any = w.start(blockIdx.x + (warp - 10), gridDim.x, from);
      if (warp == 11) {
        if (lane == 0) {
          *run_end = from;
          mbar_arrive(BAR(C::RUN_END));
        }
        __syncwarp();
        // V tiles some of whose rows nobody sees: rows [x, y) and from z on are
        // zeroed before the products may read them.  (By the TMA warp it cost a
        // microsecond of its copies for each.)
        for (uint32_t e = 0;; ++e) {
          if (!__all_sync(0xffffffffu, wait(C::V_EDGE + e % kEdges, e / kEdges))) break;
          const int4 v = *reinterpret_cast<const int4*>(sm + C::OFF_EDGE + 16 * (e % kEdges));
          if (v.w < 0) break;
          const uint32_t dst = s_base + C::OFF_RING + v.w * C::SLOT;
          for (int idx = lane; idx < kN * 8; idx += 32) {
            const int r8 = idx >> 3;
            if ((r8 < v.x || r8 >= v.y) && r8 < v.z) continue;
#pragma unroll
            for (int c = 0; c < DV / 64; ++c)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                               dst + c * (kN * 128) + idx * 16),
                           "r"(0u)
                           : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
          mbar_arrive_if(BAR(C::FULL + v.w), lane == 0);
        }
        __syncwarp();
      } else {
        // ============================ TMA producer ============================
        Seg seg;
        const uint64_t pol_keep = policy_evict_last(), pol_once = policy_evict_first();
        const int oob_row = PAGED ? p.num_blocks * p.g * p.bsz
                                  : static_cast<int>(static_cast<long long>(p.b) * p.g * p.cap);
        const int box = PAGED ? min(p.bsz, kGrain) : kGrain;
        const int sub = kN / box;  // boxes a tile and 64-column half
        const int sh = PAGED ? __ffs(p.bsz) - 1 : 0, mask = p.bsz - 1;  // (a power of two)
        uint32_t slot_n = 0, qn[2] = {0, 0}, edge_n = 0;
        uint32_t kn = 0;  // segments announced
        uint32_t twins = 0, twin_q = 0;  // tiles of twins so far; the next twins' query rows
        int d_head = 0, d_tok0 = 0, d_ntok = 0, d_j = 0, d_end = 0;  // (desc)
        bool ok = __all_sync(0xffffffffu, wait(C::RUN_END, 0));
        w.begin(any ? from : ChunkPos{p.b, 0, 0, 0}, ok ? *run_end : ChunkPos{p.b, 0, 0, 0});
        while (true) {
          const bool more = ok && w.next(seg);
          if (!more) seg.lt0 = seg.lt1 = 0;
          const int T = seg.lt1 - seg.lt0;
          const bool twin = seg.twin(p.tq);
          // The position of this lane's box of tile lt (-1: none), and the
          // table entry that holds it.  (One load a box, a tile ahead of its use:
          // a tile's boxes may lie in two places.)
          auto box_at = [&](int lt) -> int {
            const int v = lt * kN + lane * box;
            const bool in_head = v < seg.sb;
            const int pos = in_head ? v : v + seg.shift;
            return lane < sub && pos < (in_head ? seg.head : seg.L) ? pos : -1;
          };
          auto source = [&](int lt) -> int {
            return p.head_seq >= 0 && lt * kN + lane * box < seg.sb ? p.head_seq : seg.i;
          };
          auto entry = [&](int lt) -> int {
            if constexpr (PAGED) {
              const int pos = box_at(lt);
              if (pos >= 0)
                return __ldg(p.table + static_cast<size_t>(source(lt)) * p.max_blocks +
                             (pos >> sh));
            }
            return 0;
          };
          int ent = more ? entry(seg.lt0) : 0, row = 0;
          auto hold = [&](int k, uint32_t phase) {
            ok = __all_sync(0xffffffffu, ok && wait(k, phase));
            return ok;
          };
          const int ph = twins & 1;  // the side of the twins' first tile
          const uint32_t unit_q = twin_q;
          // (Most rows of twins are nobody else's.  Those of a prefix that every
          // sequence reads for itself, or of a prompt's last unit, are: kept in L2
          // these took 1 to 2 % longer, 128 x 31 tokens behind 700 39.0 -> 40.5 us.)
          const uint64_t pol = twin ? pol_once : pol_keep;
          // query rows of a side (twins: of both)
          auto load_q = [&](int side) {
            const int qb = twin ? unit_q : side;
            if (!twin && seg.side_tiles(side, p.tq) == 0) return;
            if (!hold(C::Q_EMPTY + qb, (qb ? qn[1] : qn[0]) ^ 1)) return;
            // (a twin's rows from one token: one box of its heads, the rest of the
            // tile holds anything)
            const bool one = twin && seg.ntok == 1;
            if (lane == 0) {
              const uint32_t dst = s_base + qb * C::Q_BYTES;
              mbar_arrive_expect_tx(BAR(C::Q_FULL + qb), (one ? 1 : p.tq) * p.r * DK * 2);
#pragma unroll 1
              for (int c = 0; c < DK / 64; ++c)
                tma_load_3d(dst + c * (kM * 128), one ? &tm_q1 : &tm_q, BAR(C::Q_FULL + qb), 64 * c,
                            seg.j * p.r, seg.t0 + side * p.tq, pol);
            }
            __syncwarp();
            if (qb)
              ++qn[1];
            else
              ++qn[0];
          };
          // (the first unit's rows before anything else; later ones wait for the unit
          // ahead, whose end waits for this announcement)
          const bool q_early = kn == 0 && more;
          if (q_early) load_q(0);
          if (!hold(C::SEG_EMPTY + kn % kSegs, (kn / kSegs) ^ 1)) break;
          Plan& plan = *seg_at(kn);
          if (lane < 2 && more) {  // (a side each)
            typename Plan::Side& v = plan.side[lane];
            const int tok0 = twin ? 0 : lane * p.tq;
            v.nt = twin ? (T + 1 - (lane ^ ph)) >> 1 : seg.side_tiles(lane, p.tq);
            v.first = (seg.lt0 + (twin ? lane ^ ph : 0)) * kN;
            v.tokens = max(min(seg.ntok - tok0, p.tq), 0);
            v.row0 = seg.t0 + tok0;
            seg.sees(p, tok0, v, plan.lo_min);  // (lo_min: the same from both)
          }
          const bool whole = seg.lt0 == 0 && seg.lt1 == seg.ti;
          if (lane == 0) {
            plan.T = T;
            plan.twin = twin;
            plan.qb = unit_q;
            plan.step = twin ? 2 * kN : kN;
            plan.j = seg.j;
            plan.last = whole;
            plan.part = (2 * static_cast<int>(blockIdx.x) + (seg.lt0 == 0 ? 1 : 0)) * p.srows;
            plan.by_row = 0;
            plan.head = seg.head;
            if (more && w.n_head > 0) {  // a whole unit leaves its result by row, for the join
              const int half = seg.of_head ? 0 : 1;
              if (whole) plan.by_row = 1 + half;
              plan.last = 0;
              const size_t units = static_cast<size_t>(p.group_rows) * p.g;
              int* cut = p.cut + (2 * half) * units + static_cast<size_t>(seg.t0) * p.g + seg.j;
              if (seg.lt0 == 0) cut[0] = whole ? -1 : static_cast<int>(blockIdx.x);
              if (seg.lt0 > 0 && seg.lt1 == seg.ti) cut[units] = static_cast<int>(blockIdx.x);
            }
          }
          __syncwarp();
          mbar_arrive_if(BAR(C::SEG_FULL + kn % kSegs), lane == 0);
          if (more && seg.lt0 == 0 && !whole) {
            d_head = 1;
            d_tok0 = seg.t0;
            d_ntok = seg.ntok;
            d_j = seg.j;
          } else if (more && seg.lt0 > 0) {
            d_end = seg.lt1 == seg.ti;
          }
          ++kn;
          if (!more) break;
          if (twin) twins += T;
          twin_q = twin ? twin_q ^ 1 : 0;
          if (!q_early) load_q(0);
          // K and V of the tiles by turns: the order the products need them
          for (int lt = seg.lt0; lt < seg.lt1 && ok; ++lt) {
            // the pool or cache row of this lane's box, for the tile's K and V
            const int pos = box_at(lt);
            row = oob_row;
            if constexpr (PAGED) {
              if (pos >= 0) {
                if (ent >= 0 && ent < p.num_blocks)
                  row = (ent * p.g + seg.j) * p.bsz + (pos & mask);
                else
                  atomicOr(p.status, GQA_DEV_BAD_BLOCK);
              }
              if (lt + 1 < seg.lt1) ent = entry(lt + 1);
            } else if (pos >= 0) {
              row = pos + static_cast<int>(
                              (static_cast<long long>(source(lt)) * p.g + seg.j) * p.cap);
            }
            int slot = slot_n % C::NS;
            if (!hold(C::EMPTY + slot, (slot_n / C::NS) ^ 1)) break;
            uint32_t to = BAR(C::FULL + slot), dst = s_base + C::OFF_RING + slot * C::SLOT;
            if (lane == 0) mbar_arrive_expect_tx(to, DK / 64 * kN * 128);
            __syncwarp();
            if (lane < sub) {
#pragma unroll
              for (int c = 0; c < DK / 64; ++c)
                tma_load_2d(dst + c * (kN * 128) + lane * box * 128, &tm_k, to, 64 * c, row, pol);
            }
            __syncwarp();
            ++slot_n;
            if (lt == seg.lt0 && !twin) load_q(1);
            slot = slot_n % C::NS;
            if (!hold(C::EMPTY + slot, (slot_n / C::NS) ^ 1)) break;
            to = BAR(C::FULL + slot), dst = s_base + C::OFF_RING + slot * C::SLOT;
            const int v0 = lt * kN;
            if (v0 + kN > seg.end || (seg.head < v0 + kN && seg.z > v0 && seg.z > seg.head)) {
              if (lane == 0)
                *reinterpret_cast<int4*>(sm + C::OFF_EDGE + 16 * (edge_n % kEdges)) =
                    make_int4(max(seg.head - v0, 0), seg.z - v0, max(seg.end - v0, 0), slot);
              to = BAR(C::V_EDGE + edge_n % kEdges);
              ++edge_n;
            }
            if (lane == 0) mbar_arrive_expect_tx(to, DV / 64 * kN * 128);
            __syncwarp();
            if (lane < sub) {
#pragma unroll
              for (int c = 0; c < DV / 64; ++c)
                tma_load_2d(dst + c * (kN * 128) + lane * box * 128, &tm_v, to, 64 * c, row, pol);
            }
            __syncwarp();
            ++slot_n;
          }
          if (!ok) break;
        }
        if (lane == 0) {
          int* d = p.desc + static_cast<size_t>(blockIdx.x) * kDescInts;
          d[D_HEAD] = ok ? d_head : 0;
          d[D_TOK0] = d_tok0;
          d[D_NTOK] = d_ntok;
          d[D_J] = d_j;
          d[D_END] = ok ? d_end : 1;
          d[D_ROWS] = w.n_head;
        }
        if (ok && lane == 0) {  // no more edges
          *reinterpret_cast<int4*>(sm + C::OFF_EDGE + 16 * (edge_n % kEdges)) =
              make_int4(0, 0, 0, -1);
          mbar_arrive(BAR(C::V_EDGE + edge_n % kEdges));
        }
        __syncwarp();
        if (!ok) {
          // copies in flight must land before the CTA exits (bounded)
          const long long t0 = clock64();
          for (int s = 0; s < C::NS; ++s) {
            if (slot_n <= static_cast<uint32_t>(s)) continue;
            const uint32_t last = (slot_n - 1 - s) / C::NS;  // fills of slot s, less one
            while (!mbar_try_wait(BAR(C::FULL + s), last & 1) && clock64() - t0 < p.budget) {
            }
          }
          for (int s = 0; s < 2; ++s)
            while (qn[s] > 0 && !mbar_try_wait(BAR(C::Q_FULL + s), (qn[s] - 1) & 1) &&
                   clock64() - t0 < p.budget) {
            }
        }
        __syncwarp();
      }
    } else {
      // ============================ MMA issuer ==============================
      // The sides by turns: P.V of the side's last tile, then S of its next
      // (of the next unit's first at a unit's end).  One warp issues both sides'
      // products, so each side's run back to back; with an issuer per side they
      // interleave and both sides wait longer.  The whole warp walks through
      // this code with warp-uniform values and one elected lane issues: from a
      // single lane's branch the operands take a detour into the uniform
      // registers that costs as long as a product runs.
      constexpr uint32_t kIdescS = idesc_bf16(kM, kN, 0, 0, kBf16);   // both K-major
      constexpr uint32_t kIdescO = idesc_bf16(kM, DV, 0, 1, kBf16);   // V: MN-major
      const uint64_t q0 = smem_desc(s_base, 16, 1024, SWZ_128B);
      const uint64_t k0 = smem_desc(s_base + C::OFF_RING, 16, 1024, SWZ_128B);
      const uint64_t v0 = smem_desc(s_base + C::OFF_RING, kN * 128, 1024, SWZ_128B);
      struct Ring {  // a ring position: slot and phase
        uint32_t slot = 0, phase = 0;
        __device__ Ring next() const {
          Ring r = *this;
          if (++r.slot == C::NS) {
            r.slot = 0;
            r.phase ^= 1;
          }
          return r;
        }
      };
      bool ok = true;
      auto all_wait = [&](int k, uint32_t phase) {
        ok = __all_sync(0xffffffffu, ok && wait(k, phase));
      };
      uint32_t kn = 0;                // segments read
      uint32_t q_ph = 0, p_ph = 0;    // a bit for each query buffer, each side
      // the next segment: its tiles (0: no more), and the sides'
      struct Todo {
        int T, nt0, nt1, qb;
        bool twin;
      };
      auto next_seg = [&]() -> Todo {
        Todo r = {0, 0, 0, 0, false};
        all_wait(C::SEG_FULL + kn % kSegs, kn / kSegs);
        if (!ok) return r;
        const Plan* sp = seg_at(kn);
        r.T = __shfl_sync(0xffffffffu, sp->T, 0);
        r.twin = __shfl_sync(0xffffffffu, sp->twin, 0) != 0;
        r.qb = __shfl_sync(0xffffffffu, sp->qb, 0);
        r.nt0 = __shfl_sync(0xffffffffu, sp->side[0].nt, 0);
        r.nt1 = r.T;  // (the later tokens: they see what the unit sees)
        __syncwarp();
        mbar_arrive_if(BAR(C::SEG_EMPTY + kn % kSegs), elect_one());
        ++kn;
        return r;
      };
      // Two-sided units: in round t side A's P.V of tile t - 1 and its S of tile t,
      // then side B's; at a unit's end the S of the next unit's first tile.
      Ring at;               // V of tile t - 1 (t = 0: K of tile 0)
      int t = 0, s = 0;
      bool primed = false;   // the next unit's first S are out
      bool ahead = false;    // the next unit is known
      // Twins: tiles by turns, without a break between units, S two tiles ahead of P.V.
      bool stream = false, have = false, ended = false;
      Ring ks, vo;           // K of the next S, V of the next P.V
      uint32_t n_s = 0, n_o = 0, flags = 0;  // tiles so far; first, last of a side (two bits each)
      int ts = 0;
      Todo cur = next_seg(), nx = cur;
      // One loop for everything but the steady rounds of two-sided units, with one
      // place for either product: what runs once a unit is fetched each time.
      while (ok) {
        bool do_o = false, do_s = false, o_first = false, o_last = false, s_first = false,
             s_last = false, o_free = false, s_free = false;
        int side_o = 0, side_s = 0, qb = 0;
        Ring ov, sk;
        if (stream) {
          // S of tiles 0 and 1, then P.V of a tile and S of the one after next
          if (!have && !ended) {
            nx = next_seg();
            if (!ok) break;
            have = nx.T > 0 && nx.twin;
            ended = !have;
            if (have) cur = nx;
            ts = 0;
          }
          if (ended && n_o == n_s) {
            stream = false;
            cur = nx;
            at = ks;
            primed = false;
            t = s = 0;
            continue;
          }
          sk = ks;
          ov = vo;
          qb = cur.qb;
          side_s = n_s & 1;
          side_o = n_o & 1;
          do_o = n_s - n_o == 2 || !have;
          do_s = have;
          s_first = ts == 0;
          s_last = ts == cur.T - 1;
          o_first = (flags >> (2 * side_o)) & 1u;  // (of the tile whose S went out before)
          o_last = (flags >> (2 * side_o + 1)) & 1u;
          o_free = s_free = true;
        } else {
          if (cur.T == 0) break;
          if (cur.twin) {
            stream = have = true;
            ended = false;
            ks = at;
            vo = at.next();
            ts = 0;
            continue;
          }
          // rounds in which both sides have a P.V and an S that is not their last
          if (s == 0 && t >= 2 && t < cur.nt0 - 1) {
            // as below, with as little as can be between one side's products
            // and the other's
            do {
              const Ring v = at, k = at.next();
#pragma unroll
              for (int sd = 0; sd < 2; ++sd) {
                ok = __all_sync(0xffffffffu,
                                ok && (sd == 1 || (wait(C::FULL + v.slot, v.phase) &&
                                                   wait(C::FULL + k.slot, k.phase))) &&
                                    wait(C::P_READY + sd, p_ph >> sd));
                p_ph ^= 1u << sd;
                if (!ok) break;
                tc_fence_after();
                const uint64_t vb = v0 + v.slot * (C::SLOT >> 4), kb = k0 + k.slot * (C::SLOT >> 4);
                const uint64_t qa = q0 + ((sd * C::Q_BYTES) >> 4);
                if (elect_one()) {
#pragma unroll
                  for (int e = 0; e < kN / 16; ++e)
                    mma_16_ts(C::T_O + sd * 128, C::T_S + sd * 128 + 8 * e, vb + e * (2048 >> 4),
                              kIdescO, 1u);
                  if (sd == 1) mma_commit(BAR(C::EMPTY + v.slot));
#pragma unroll
                  for (int e = 0; e < DK / 16; ++e) {
                    const uint32_t o = ((e >> 2) * (kM * 128) + (e & 3) * 32) >> 4;
                    mma_bf16(C::T_S + sd * 128, qa + o, kb + o, kIdescS, e > 0 ? 1u : 0u);
                  }
                  mma_commit(BAR(C::S_FULL + sd));
                  if (sd == 1) mma_commit(BAR(C::EMPTY + k.slot));
                }
                __syncwarp();
              }
              at = k.next();
              ++t;
            } while (ok && t < cur.nt0 - 1);
            continue;
          }
          if (s == 0 && (t == cur.T - 1 || (t == cur.T && !ahead))) {
            // (a round early where there is one: its copies are under way by then)
            nx = next_seg();
            if (!ok) break;
            ahead = true;
          }
          if (t == cur.T) primed = nx.T > 0 && !nx.twin;
          const int nt = s ? cur.nt1 : cur.nt0, nxt = s ? nx.nt1 : nx.nt0;
          ov = at;
          sk = t > 0 ? at.next() : at;
          side_o = side_s = qb = s;
          do_o = t > 0 && t <= nt;
          o_first = t == 1;
          o_last = t == nt;
          do_s = t < cur.T ? t < nt : primed && nxt > 0;
          s_first = t == 0 || t == cur.T;
          s_last = t < cur.T ? t == nt - 1 : nxt == 1;
          o_free = s_free = s == 1;
        }
        if (do_o) {
          all_wait(C::FULL + ov.slot, ov.phase);
          all_wait(C::P_READY + side_o, p_ph >> side_o);
          p_ph ^= 1u << side_o;
          if (!ok) break;
          tc_fence_after();
          const uint64_t b0 = v0 + ov.slot * (C::SLOT >> 4);
          const uint32_t d = C::T_O + side_o * 128, a0 = C::T_S + side_o * 128;
          if (elect_one()) {
#pragma unroll
            for (int e = 0; e < kN / 16; ++e)
              mma_16_ts(d, a0 + 8 * e, b0 + e * (2048 >> 4), kIdescO,
                        (o_first && e == 0) ? 0u : 1u);
            if (o_last) mma_commit(BAR(C::O_DONE + side_o));
            if (o_free) mma_commit(BAR(C::EMPTY + ov.slot));
          }
          __syncwarp();
        }
        if (do_s) {
          if (s_first) {
            all_wait(C::Q_FULL + qb, q_ph >> qb);
            q_ph ^= 1u << qb;
          }
          all_wait(C::FULL + sk.slot, sk.phase);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a0 = q0 + ((qb * C::Q_BYTES) >> 4);
          const uint64_t b0 = k0 + sk.slot * (C::SLOT >> 4);
          const uint32_t d = C::T_S + side_s * 128;
          if (elect_one()) {
#pragma unroll
            for (int e = 0; e < DK / 16; ++e) {
              const uint32_t o = ((e >> 2) * (kM * 128) + (e & 3) * 32) >> 4;
              mma_bf16(d, a0 + o, b0 + o, kIdescS, e > 0 ? 1u : 0u);
            }
            mma_commit(BAR(C::S_FULL + side_s));
            if (s_last) mma_commit(BAR(C::Q_EMPTY + qb));
            if (s_free) mma_commit(BAR(C::EMPTY + sk.slot));
          }
          __syncwarp();
        }
        if (stream) {
          if (do_o) {
            vo = vo.next().next();
            ++n_o;
          }
          if (do_s) {
            const uint32_t f = (ts < 2 ? 1u : 0u) | (ts + 2 >= cur.T ? 2u : 0u);
            flags = (flags & ~(3u << (2 * side_s))) | (f << (2 * side_s));
            ks = ks.next().next();
            ++n_s;
            if (++ts == cur.T) have = false;
          }
        } else {
          if (s == 1) {
            at = t < cur.T || primed ? sk.next() : sk;
            if (t == cur.T) {
              cur = nx;
              t = primed ? 1 : 0;
              primed = ahead = false;
            } else {
              ++t;
            }
          }
          s ^= 1;
        }
      }
      // every product has to be finished before tensor memory is released
      if (elect_one()) {
        mma_commit(BAR(C::DRAIN));
        const long long t0 = clock64();
        while (!mbar_try_wait(BAR(C::DRAIN), 0) && clock64() - t0 < p.budget) {
        }
      }
      __syncwarp();
    }
  } else {
    // ======================= softmax, output ==============================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int side = warp >> 2;
    float2* const ml_sm = reinterpret_cast<float2*>(sm + C::OFF_ML);
    const int row = (warp & 3) * 32 + lane;  // query row of the side = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::T_S + side * 128;
    const uint32_t tO = tmem + lane_off + C::T_O + side * 128;
    const int tok = row / p.r, head = row - tok * p.r;
    // a scale of zero or below would turn the maximum around: it is applied
    // to the logits first then
    const bool pre = !(p.scale_log2 > 0.f);
    const float sl = pre ? 1.f : p.scale_log2;
    uint32_t sn = 0, on = 0, tn = 0;
    bool ok = true;
    for (uint32_t kn = 0;; ++kn) {
      ok = ok && __all_sync(0xffffffffu, wait(C::SEG_FULL + kn % kSegs, (kn / kSegs) & 1));
      if (!ok) break;
      const Plan* const sp = seg_at(kn);
      const typename Plan::Side& my = sp->side[side];
      const int nt = my.nt, first = my.first, step = sp->step, see = my.hi + tok;
      const bool live = tok < my.tokens;
      const bool warp_live = (warp & 3) * 32 < my.tokens * p.r;  // (some row is)
      // This row sees [0, vis.head) and [vis.lo, vis.hi) of the unit's
      // span; `side_vis`: what every row of the side sees
      const PartVisible side_vis = {my.all_head, my.all_lo, my.all_hi};
      PartVisible vis = {min(sp->head, see), max(my.lo + tok, sp->lo_min), see};
      if (vis.lo <= vis.head) vis.lo = 0;
      if (sp->T == 0) break;
      // (lanes without a row hold anything: with their maximum at infinity they
      // have no say in when the others' is raised)
      float m = live ? -INFINITY : INFINITY, l = 0.f;
      for (int t = 0; t < (warp_live ? 0 : nt); ++t) {  // nothing here is read
        ok = __all_sync(0xffffffffu, ok && wait(C::S_FULL + side, sn & 1));
        ++sn;
        mbar_arrive_if(BAR(C::P_READY + side), lane == 0);
      }
      for (int t = 0; t < (warp_live ? nt : 0); ++t) {
        ok = __all_sync(0xffffffffu, wait(C::S_FULL + side, sn & 1));
        ++sn;
        if (!ok) break;
        tc_fence_after();
        float x[kN];
#pragma unroll
        for (int c = 0; c < kN / 32; ++c) tmem_ld32(tS + 32 * c, x + 32 * c);
        tmem_wait_ld();
        if (pre) {
#pragma unroll
          for (int e = 0; e < kN; ++e) x[e] *= p.scale_log2;
        }
        const int base = first + t * step;
        if (!side_vis.all(base, kN)) {
#pragma unroll
          for (int c = 0; c < kN / 32; ++c) {
            const int x0 = base + 32 * c;
            if (side_vis.all(x0, 32)) continue;  // (uniform)
            const uint32_t bits = vis.bits(x0);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(bits & (1u << e))) x[32 * c + e] = -INFINITY;
          }
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int e = 4; e < kN; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = e + 4 < kN ? max3(mx[k], x[e + k], x[e + 4 + k]) : fmaxf(mx[k], x[e + k]);
        const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        // S_FULL also covers the products issued before it: O is complete
        // up to the last tile.
        if (__any_sync(0xffffffffu, (mn - m) * sl > PRange<T16>::kRaise)) {
          const float ref = mn == -INFINITY ? 0.f : mn;
          const float alpha = ex2((m - ref) * sl);
          m = mn;
          l *= alpha;
          if (t > 0) {
#pragma unroll
            for (int c = 0; c < DV / 8; ++c) {
              float o[8];
              tmem_ld8(tO + 8 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] *= alpha;
              tmem_st8(tO + 8 * c, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : PRange<T16>::kLift - m * sl;
        const float2 sl2 = make_float2(sl, sl), off2 = make_float2(off, off);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t u[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float2 y = fma2(make_float2(x[64 * c + 2 * e], x[64 * c + 2 * e + 1]), sl2, off2);
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            sum[e & 1] = add2(sum[e & 1], y);
            u[e] = Half16<T16>::pack2(y.x, y.y);
          }
          tmem_st32(tS + 32 * c, u);
        }
        tmem_wait_st();
        tc_fence_before();
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        __syncwarp();
        mbar_arrive_if(BAR(C::P_READY + side), lane == 0);
      }
      if (!ok) break;
      // ---- unit's end: O / l, or a partial (maximum, sum, O) ----
      const bool twin = sp->twin, last = sp->last;
      const int other = twin ? sp->T - nt : 0;  // tiles of the other side
      const int by_row = sp->by_row;
      const size_t at = sp->part + (twin ? 0 : side * kM);
      const size_t out_row = static_cast<size_t>(my.row0 + tok) * p.h + sp->j * p.r + head;
      __syncwarp();
      mbar_arrive_if(BAR(C::SEG_EMPTY + kn % kSegs), lane == 0);
      // (twins: each side joins and writes half of the columns of both)
      if (nt > 0) {
        ok = __all_sync(0xffffffffu, wait(C::O_DONE + side, on & 1));
        ++on;
        if (!ok) break;
        tc_fence_after();
      }
      // (base 2; a sum that is NaN keeps its piece from counting as empty)
      float ms = l > 0.f ? m * sl : l == 0.f ? -INFINITY : l;
      float wo = 1.f, wt = 0.f;                 // factors of this side's O, of its twin's
      if (twin) {
        // (a bounded wait, as every wait here; then the other side's O is
        // complete too)
        ml_sm[side * kM + row] = make_float2(ms, l);
        __syncwarp();
        mbar_arrive_if(BAR(C::TWIN), lane == 0);
        ok = __all_sync(0xffffffffu, wait(C::TWIN, tn & 1));
        if (!ok) break;
        tc_fence_after();
        const float2 t2 = ml_sm[(side ^ 1) * kM + row];
        const float mj = fmaxf(ms, t2.x);
        const float ref = mj == -INFINITY ? 0.f : mj;
        wo = ex2(ms - ref);
        wt = ex2(t2.x - ref);
        l = l * wo + t2.y * wt;
        ms = l >= 0.f ? mj : l;
      }
      const int c0 = twin ? side * (DV / 64) : 0, c1 = twin ? c0 + DV / 64 : DV / 32;
      const float inv = 1.f / l;
      float* pml = p.part_ml + 2 * (at + row);
      float* pdst = p.part_o + (at + row) * DV;
      if (by_row) {
        const size_t x = (by_row - 1) * static_cast<size_t>(p.group_rows) * p.h + out_row;
        pml = p.row_ml + 2 * x;
        pdst = p.row_o + x * DV;
      }
      if (!last && live && (!twin || side == 0)) {
        pml[0] = ms;
        pml[1] = l;
      }
      // A thread writes its own row, in whole 32-byte sectors where the output
      // is aligned to them.  (Rows turned in shared memory or by shuffles
      // between four lanes touch fewer lines a store but cost more
      // instructions: 155 and 149 us for a mixed batch of prompts, chunks and
      // single tokens where this took 142.)
      T16* const dst = static_cast<T16*>(p.out) + out_row * DV;
      const float fo = last ? wo * inv : wo, ft = last ? wt * inv : wt;
      // (nothing where no row is live or the side has no tokens)
      const int c_end = warp_live && (nt > 0 || other > 0) ? c1 : c0;
#pragma unroll 1
      for (int c = c0; c < c_end; ++c) {
        __syncwarp();  // (the loads of tensor memory are the whole warp's)
        float o[32];
        if (nt > 0) {
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= fo;
        if (other > 0) {
          float o2[32];
          tmem_ld32(tO + (side ? -128 : 128) + 32 * c, o2);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = fmaf(o2[e], ft, o[e]);
        }
        if (live) {
          if (last) {
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = Half16<T16>::pack2(o[2 * e], o[2 * e + 1]);
            store_sectors<2>(dst + 32 * c, u, p.out_sectors);
          } else {
            uint32_t u[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e]);
            store_sectors<4>(pdst + 32 * c, u, true);
          }
        }
      }
      __syncwarp();
      tc_fence_before();
      if (twin) {  // both O and ml_sm are free again
        __syncwarp();
        mbar_arrive_if(BAR(C::TWIN + 1), lane == 0);
        ok = __all_sync(0xffffffffu, wait(C::TWIN + 1, tn & 1));
        ++tn;
      }
    }
  }

  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, 512);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct PartCall : ChunkCall {
  // a part of the cache, as in ChunkParams
  int window = 0, head = 0, head_seq = -1, base_min = 0;
  int group_rows = 0;
};

struct PartPlan : ChunkPlan {
  size_t cut_at = 0, row_ml_at = 0, row_o_at = 0;
};

PartPlan part_plan(int total, int h, int g, int dv, int num_sms, int group_rows) {
  PartPlan pl;
  static_cast<ChunkPlan&>(pl) = chunk_plan(total, h, g, dv, num_sms);
  if (group_rows > 0) {
    const size_t t = group_rows;
    pl.cut_at = pl.bytes;
    pl.row_ml_at = up256(pl.cut_at + 4 * t * g * sizeof(int));
    pl.row_o_at = up256(pl.row_ml_at + 4 * t * h * sizeof(float));
    pl.bytes = up256(pl.row_o_at + 2 * t * h * dv * sizeof(float));
  }
  return pl;
}

template <typename T16, int DK, int DV, bool PAGED, class Walk>
cudaError_t launch_chunk(const PartCall& x, const PartPlan& pl, int num_sms, unsigned int* status,
                         cudaStream_t st) {
  using C = ChunkCfg<DK, DV>;
  ChunkParams p;
  chunk_args(p, x, pl, status);
  p.window = x.window;
  p.unit_inv = static_cast<unsigned>(((1ull << 32) + 2 * p.tq - 1) / (2 * p.tq));
  p.head = x.head;
  p.head_seq = x.head_seq;
  p.base_min = x.base_min;
  p.group_rows = x.group_rows;
  char* ws = static_cast<char*>(x.ws);
  p.cut = reinterpret_cast<int*>(ws + pl.cut_at);
  p.row_ml = reinterpret_cast<float*>(ws + pl.row_ml_at);
  p.row_o = reinterpret_cast<float*>(ws + pl.row_o_at);

  CUtensorMap mq, mq1, mk, mv;
  if (!map_q<T16, DK>(&mq, x, p.tq) || !map_q<T16, DK>(&mq1, x, 1) ||
      !map_kv<T16, DK, DV>(&mk, &mv, x, kGrain))
    return cudaErrorInvalidValue;
  auto kern = chunk_attn_kernel<T16, DK, DV, PAGED, Walk>;
  static std::atomic<unsigned long long> configured{0};
  if (cudaError_t e = chunk_configure(kern, C::SMEM, configured)) return e;
  ChunkLaunch l(num_sms, C::SMEM, st);
  if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, mq, mq1, mk, mv, p)) return e;
  return Walk::template join<T16, DV>(l.cfg, p, num_sms);
}

}  // namespace
}  // namespace gqa
