// chunk_attn.cu - causal attention of packed chunks of new tokens (prompts,
// prompt chunks, single tokens, mixed) over a contiguous or paged 16-bit
// cache, on the tcgen05 tensor cores.
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
//              ring (64-column boxes, 128-byte swizzle)
//   warp 11    the run's end (the TMA warp finds its start meanwhile)
//   (warp 9 checks the lengths: registers are dealt out by warpgroups)
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
// Rows >= L_i: masked out of S, their V rows zeroed in shared memory.
//
// Bound by the tensor cores where units are long: a prompt of 8,192 tokens,
// h = 64, g = 8, d = 128, bf16: 649 to 657 us, 1,680 TFLOP/s, in a short graph replay,
// 684 to 709 us over several GPUs, 1,550 to 1,610, among other passes, as the clock
// falls under the power limit.  What the pipe still waits for is a side's own chain of
// S, softmax and hand-over, which is a little longer than the other side's products.  Short units are bound by their
// fixed cost (query rows in, first logits, output): 135 to 145 us for 32 mixed
// sequences of 5,957 tokens, 34.8 us for 48 packed short prompts with 64-wide heads,
// 18.1 us for eight chunks of 4 to 12 tokens.
#include "chunk_common.cuh"

namespace gqa {
namespace {

constexpr int kSegBytes = 48;  // of an announced segment

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
                       TWIN = V_EDGE + 1, RUN_END = TWIN + 2, DRAIN = RUN_END + 1, NBAR = DRAIN + 1;
  static constexpr int OFF_SEG = (OFF_BAR + 8 * NBAR + 15) / 16 * 16;
  static constexpr int OFF_ML = OFF_SEG + kSegs * kSegBytes;  // float2 [2][kM]: twins' maxima, sums
  static constexpr int OFF_MISC = OFF_ML + 2 * kM * 8;  // TMEM address, abort flag; the run's end
  static constexpr int SMEM = OFF_MISC + 32;
  static constexpr int T_S = 0, T_O = 256;  // TMEM columns, 128 to a side
  static_assert(SMEM <= 232448, "shared memory budget");
};

using ChunkParams = ChunkArgs;

struct ChunkSeg {
  int i, j;        // sequence, KV head
  int t0;          // packed row of the unit's first token
  int pos0;        // its position
  int ntok;        // tokens of the unit
  int L;
  int lt0, lt1;    // tiles of the unit taken here
  int ti;          // tiles of the unit
  // A unit whose rows fit side A alone runs as twins: both sides hold the same
  // rows and take the tiles by turns, and their results are joined at the end.
  __device__ bool twin(int tq) const { return ntok <= tq; }
  // tiles that each side works on of [lt0, lt1)
  __device__ int side_tiles(int side, int tq) const {
    if (twin(tq)) return (lt1 - lt0 + 1 - side) >> 1;
    const int nt = min(ntok - side * tq, tq);
    const int ext = pos0 + side * tq + nt;
    return max(0, min(lt1, (ext + kN - 1) / kN) - lt0);
  }
};

static_assert(sizeof(ChunkSeg) <= kSegBytes, "segment ring");

// The run of work of one CTA, cut into segments of units.  The TMA warp walks
// (warp-uniform values) and announces each segment to the others through a
// ring in shared memory.
//
// Work is counted in cached positions: a unit's is the position behind its
// last token (three quarters of it where it runs as twins: two tiles of twins
// were measured at 4,100 cycles, bound by their copies, a two-sided tile at
// 2,610) plus kUnitCost for what a unit costs however short it is (6,590
// cycles: query rows in, first logits, output), so the units of a sequence but
// the last form an arithmetic progression and sums of them a closed form.  All
// units are laid end to end (sequences, KV heads, blocks of query rows) and run
// c begins at c * W / nc, moved to a tile's edge, or to the unit's when that is
// near.  (With half the work for twins and a cost of 192 the prompt takes 675 us
// where this takes 650.  The cost alone, graph replay: 192, 320, 448, 576 give
// 134, 131, 133, 137 us for the mixed batch, and with 64-wide heads 105, 107,
// 110, 114 us for it and 33.0, 33.6, 34.7, 35.4 us for packed short prompts.)
constexpr int kUnitCost = 320;

struct ChunkWalk {
  const int *cu, *lens;
  int b, g, tq, total;
  long long cap;
  ChunkPos at, end;
  int t0, n, L;  // of sequence at.i
  bool more;
  // sequence `lane` of the batch's first 32: its rows and work, and the work
  // up to its end (of one KV head)
  int c_t0, c_n, c_L;
  long long c_f, c_incl;

  __device__ bool seq(int k, int& a0, int& nn, int& Lk) const {
    a0 = nn = Lk = 0;
    if (k >= b) return false;
    a0 = __ldg(cu + k);
    const int a1 = __ldg(cu + k + 1);
    Lk = __ldg(lens + k);
    if (packed_errors(a0, a1, Lk, total, cap)) return false;
    nn = a1 - a0;
    return nn > 0;
  }
  __device__ int units(int nn) const { return (nn + 2 * tq - 1) / (2 * tq); }
  // is the sequence's last unit one of twins?
  __device__ bool last_twin(int nn, int nu) const { return nn - (nu - 1) * 2 * tq <= tq; }
  // work of the first q units, all of them full
  __device__ long long prefix(long long q, int nn, int Lk) const {
    return q * (Lk - nn + kUnitCost) + tq * (q * (q + 1));
  }
  __device__ long long work(int nn, int Lk) const {
    const int nu = units(nn);
    return last_twin(nn, nu) ? prefix(nu - 1, nn, Lk) + ((3ll * Lk) >> 2) + kUnitCost
                             : prefix(nu, nn, Lk);
  }
  __device__ int tiles(int q, int nn, int Lk) const {
    const long long ext = min(static_cast<long long>(Lk),
                              static_cast<long long>(Lk) - nn + (q + 1ll) * 2 * tq);
    return static_cast<int>((ext + kN - 1) >> 7);
  }

  // work f of each lane's sequence, and its sum up to the lane
  __device__ void scan(int base, int& a0, int& nn, int& Lk, long long& f, long long& incl) const {
    f = seq(base + (threadIdx.x & 31), a0, nn, Lk) ? work(nn, Lk) : 0;
    incl = f;
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if ((threadIdx.x & 31) >= o) incl += y;
    }
  }

  // the place of work x (0 <= x < W): every lane gets it; also t0, n, L
  __device__ ChunkPos locate(long long x, int near) {
    long long carry = 0;
    for (int base = 0; base < b; base += 32) {
      int a0 = c_t0, nn = c_n, Lk = c_L;
      long long f = c_f, incl = c_incl;
      if (base > 0) scan(base, a0, nn, Lk, f, incl);
      const long long hi = (carry + incl) * g, lo = hi - f * g;
      const unsigned hit = __ballot_sync(0xffffffffu, f > 0 && lo <= x && x < hi);
      if (hit) {
        const int src = __ffs(hit) - 1;
        t0 = __shfl_sync(0xffffffffu, a0, src);
        n = __shfl_sync(0xffffffffu, nn, src);
        L = __shfl_sync(0xffffffffu, Lk, src);
        const long long off = x - __shfl_sync(0xffffffffu, lo, src);
        const long long fs = __shfl_sync(0xffffffffu, f, src);
        ChunkPos r;
        r.i = base + src;
        r.j = static_cast<int>(div_pos(off, fs));
        const long long rem = off - r.j * fs;
        // the last unit q with prefix(q) <= rem: the root of the quadratic,
        // put right by steps of one
        const int nu = units(n);
        const float c1 = static_cast<float>(L - n) + (kUnitCost + tq);
        const float rf = static_cast<float>(rem);
        int q = static_cast<int>(2.f * rf / (sqrtf(c1 * c1 + 4.f * tq * rf) + c1));
        q = min(max(q, 0), nu - 1);
        while (q > 0 && prefix(q, n, L) > rem) --q;
        while (q + 1 < nu && prefix(q + 1, n, L) <= rem) ++q;
        r.qt = q;
        const int ti = tiles(q, n, L);
        const bool tw = q == nu - 1 && last_twin(n, nu);
        const long long in = rem - prefix(q, n, L);
        const int lt = static_cast<int>((tw ? (in + in / 3) : in) >> 7);
        r.lt = lt <= near ? 0 : lt >= ti - near ? ti : lt;
        return r;
      }
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    return {b, 0, 0, 0};  // not reached for x < W
  }

  // Run c's start: false when the launch has fewer runs than that (c = their
  // number: the end of the last one, behind every sequence).
  __device__ bool start(const ChunkParams& p, int c, int nc, ChunkPos& r) {
    cu = p.cu;
    lens = p.lens;
    b = p.b;
    g = p.g;
    tq = p.tq;
    total = p.total;
    cap = p.cap;
    scan(0, c_t0, c_n, c_L, c_f, c_incl);
    long long W = __shfl_sync(0xffffffffu, c_incl, 31);
    for (int base = 32; base < b; base += 32) {
      int a0, nn, Lk;
      long long f, incl;
      scan(base, a0, nn, Lk, f, incl);
      W += __shfl_sync(0xffffffffu, incl, 31);
    }
    W *= g;
    r = {b, 0, 0, 0};
    // a run is worth at least a tile (two with much work): less costs more to
    // join than it saves
    nc = static_cast<int>(min(static_cast<long long>(nc), W / (2 * kN) + 1));
    if (W == 0 || c > nc) return false;
    if (c == nc) return true;
    const long long run = div_pos(W, nc);
    const int near = static_cast<int>(run / (32 * kN));
    const int left = static_cast<int>(W - run * nc);  // the first `left` runs are one longer
    r = locate(run * c + min(c, left), near);
    if (c == 0) r.lt = 0;
    return true;
  }

  // Begin run c, whose end is e.
  __device__ void begin(const ChunkPos& from, const ChunkPos& e) {
    at = from;
    end = e;
    more = at.i < b;
    // (a place at its unit's last tile's end is the next unit's start)
    if (more && at.lt >= tiles(at.qt, n, L)) advance();
  }

  __device__ void advance() {  // to the next unit's start
    at.lt = 0;
    if (++at.qt < units(n)) return;
    at.qt = 0;
    if (++at.j < g) return;
    at.j = 0;
    do {
      ++at.i;
    } while (at.i < b && !seq(at.i, t0, n, L));
  }

  __device__ bool next(ChunkSeg& s) {
    if (!more || at.i >= b) return false;
    const int ti = tiles(at.qt, n, L);
    const bool last = at.i == end.i && at.j == end.j && at.qt == end.qt;
    const bool past = at.i > end.i || (at.i == end.i && (at.j > end.j ||
                                       (at.j == end.j && at.qt > end.qt)));
    if (past || (last && end.lt <= at.lt)) return false;
    s.i = at.i;
    s.j = at.j;
    s.t0 = t0 + at.qt * 2 * tq;
    s.pos0 = L - n + at.qt * 2 * tq;
    s.ntok = min(n - at.qt * 2 * tq, 2 * tq);
    s.L = L;
    s.ti = ti;
    s.lt0 = at.lt;
    s.lt1 = last ? end.lt : ti;
    if (last)
      more = false;
    else
      advance();
    return true;
  }
};

template <typename T16, int DK, int DV, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const ChunkParams p) {
  using C = ChunkCfg<DK, DV>;
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

  auto seg_at = [&](uint32_t k) -> ChunkSeg* {
    return reinterpret_cast<ChunkSeg*>(sm + C::OFF_SEG + (k % kSegs) * kSegBytes);
  };
  auto wait = [&](int k, uint32_t phase) -> bool {
    return mbar_wait(BAR(k), phase & 1u, abort_flag, p.status, p.budget);
  };

  ChunkPos* const run_end = reinterpret_cast<ChunkPos*>(sm + C::OFF_MISC + 16);
  // (a warpgroup's four warps at the same instruction, as it has to be)
  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  if (warp == 9) {
    if (blockIdx.x == 0) report_bad_packed(p.cu, p.lens, p.b, p.total, p.cap, p.status);
  } else if (warp == 11) {
    // the run's end, beside the TMA warp's look for its start
    ChunkWalk w;
    ChunkPos e;
    w.start(p, blockIdx.x + 1, gridDim.x, e);
    if (lane == 0) {
      *run_end = e;
      mbar_arrive(BAR(C::RUN_END));
    }
    __syncwarp();
  } else if (warp == 10) {
    // ============================ TMA producer ============================
    ChunkWalk w;
    ChunkSeg seg;
    ChunkPos from;
    const bool any = w.start(p, blockIdx.x, gridDim.x, from);
    const uint64_t pol = policy_evict_last();
    const int oob_row = PAGED ? p.num_blocks * p.g * p.bsz : 0;
    const int box = PAGED ? min(p.bsz, kN) : kN;
    const int sub = kN / box;  // boxes a tile and 64-column half
    const int sh = PAGED ? __ffs(p.bsz) - 1 : 0, mask = p.bsz - 1;  // (a power of two)
    uint32_t slot_n = 0, qn[2] = {0, 0}, edge_n = 0;
    uint32_t kn = 0;  // segments announced
    bool ok = __all_sync(0xffffffffu, wait(C::RUN_END, 0));
    w.begin(any ? from : ChunkPos{p.b, 0, 0, 0}, ok ? *run_end : ChunkPos{p.b, 0, 0, 0});
    auto announce = [&](const ChunkSeg& sg) {
      ok = __all_sync(0xffffffffu, wait(C::SEG_EMPTY + kn % kSegs, ((kn / kSegs) & 1) ^ 1));
      if (!ok) return;
      if (lane == 0) {
        *seg_at(kn) = sg;
        mbar_arrive(BAR(C::SEG_FULL + kn % kSegs));
      }
      __syncwarp();
      ++kn;
    };
    while (ok && w.next(seg)) {
      announce(seg);
      // the sequence's table entries, 64 at a time ahead of their use: no load
      // stands before a tile's copies
      PageCursor pc;
      if (PAGED)
        pc.start(p.table + static_cast<size_t>(seg.i) * p.max_blocks,
                 static_cast<int>((static_cast<unsigned>(seg.L) + mask) >> sh),
                 (seg.lt0 * kN) >> sh);
      // lane mm < sub: the pool row of box mm of tile lt
      auto lookup = [&](int lt) -> int {
        const int pm = lt * kN + lane * box;
        const int blk = pc.get_lanes((lt * kN) >> sh);
        if (lane >= sub || pm >= seg.L) return oob_row;
        if (blk < 0 || blk >= p.num_blocks) {
          atomicOr(p.status, GQA_DEV_BAD_BLOCK);
          return oob_row;
        }
        return (blk * p.g + seg.j) * p.bsz + (pm & mask);
      };
      auto load_q = [&](int side) {
        if (!ok || seg.side_tiles(side, p.tq) == 0) return;
        ok = __all_sync(0xffffffffu, wait(C::Q_EMPTY + side, (qn[side] & 1) ^ 1));
        if (!ok) return;
        if (lane == 0) {
          mbar_arrive_expect_tx(BAR(C::Q_FULL + side), p.tq * p.r * DK * 2);
          for (int c = 0; c < DK / 64; ++c)
            tma_load_3d(s_base + side * C::Q_BYTES + c * (kM * 128), &tm_q, BAR(C::Q_FULL + side),
                        64 * c, seg.j * p.r, seg.t0 + (seg.twin(p.tq) ? 0 : side * p.tq), pol);
        }
        __syncwarp();
        ++qn[side];
      };
      auto load_kv = [&](bool is_v, int lt, int prow) {
        if (!ok) return;
        const int slot = slot_n % C::NS;
        ok = __all_sync(0xffffffffu, wait(C::EMPTY + slot, ((slot_n / C::NS) & 1) ^ 1));
        if (!ok) return;
        const int nbox = (is_v ? DV : DK) / 64;
        // a V tile that runs past L_i: its rows there are zeroed first
        const bool edge = is_v && (lt + 1) * kN > seg.L;
        const uint32_t bar = BAR(edge ? C::V_EDGE : C::FULL + slot);
        const uint32_t dst = s_base + C::OFF_RING + slot * C::SLOT;
        if (lane == 0) mbar_arrive_expect_tx(bar, nbox * kN * 128);
        __syncwarp();
        if (PAGED ? lane < sub : lane == 0) {
          const int row = PAGED ? prow
                                : static_cast<int>((static_cast<long long>(seg.i) * p.g + seg.j) *
                                                   p.cap) + lt * kN;
          for (int c = 0; c < nbox; ++c)
            tma_load_2d(dst + c * (kN * 128) + lane * box * 128, is_v ? &tm_v : &tm_k, bar, 64 * c,
                        row, pol);
        }
        __syncwarp();
        if (edge) {
          ok = __all_sync(0xffffffffu, wait(C::V_EDGE, edge_n & 1));
          ++edge_n;
          if (ok) {
            const int first = seg.L - lt * kN;
            for (int idx = first * 8 + lane; idx < kN * 8; idx += 32)
              for (int c = 0; c < nbox; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 dst + c * (kN * 128) + idx * 16),
                             "r"(0u)
                             : "memory");
            fence_proxy_async_smem();
            __syncwarp();
            mbar_arrive_if(BAR(C::FULL + slot), lane == 0);
          }
        }
        ++slot_n;
      };
      int row = PAGED ? lookup(seg.lt0) : 0;
      load_q(0);
      load_kv(false, seg.lt0, row);
      load_q(1);
      for (int lt = seg.lt0; lt < seg.lt1 && ok; ++lt) {
        const int cur = row;
        if (PAGED && lt + 1 < seg.lt1) row = lookup(lt + 1);
        // tile lt's V, then tile lt + 1's K: the order the products need them
        load_kv(true, lt, cur);
        if (lt + 1 < seg.lt1) load_kv(false, lt + 1, row);
      }
    }
    if (ok) {
      seg.lt0 = seg.lt1 = 0;  // no more
      announce(seg);
    }
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
  } else if (warp == 8) {
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
    Ring at;  // next position to be used
    uint32_t kn = 0, qn[2] = {0, 0}, pn[2] = {0, 0};
    bool ok = true;
    auto all_wait = [&](int k, uint32_t phase) {
      ok = __all_sync(0xffffffffu, ok && wait(k, phase));
    };
    // the next segment: its tiles (0: no more), and the sides'
    struct Todo {
      int T, nt[2];
      bool twin;
    };
    auto next_seg = [&]() -> Todo {
      Todo r = {0, {0, 0}, false};
      all_wait(C::SEG_FULL + kn % kSegs, (kn / kSegs) & 1);
      if (!ok) return r;
      const ChunkSeg seg = *seg_at(kn);
      r.nt[0] = __shfl_sync(0xffffffffu, seg.side_tiles(0, p.tq), 0);
      r.nt[1] = __shfl_sync(0xffffffffu, seg.side_tiles(1, p.tq), 0);
      r.T = __shfl_sync(0xffffffffu, seg.lt1 - seg.lt0, 0);
      r.twin = __shfl_sync(0xffffffffu, seg.twin(p.tq) ? 1 : 0, 0) != 0;
      mbar_arrive_if(BAR(C::SEG_EMPTY + kn % kSegs), elect_one());
      ++kn;
      return r;
    };
    // S of side s with the K tile at ring position x
    auto issue_s = [&](int s, Ring x, bool first, bool last) {
      if (first) {
        all_wait(C::Q_FULL + s, qn[s] & 1);
        ++qn[s];
      }
      all_wait(C::FULL + x.slot, x.phase);
      if (!ok) return;
      tc_fence_after();
      const uint64_t a0 = q0 + ((s * C::Q_BYTES) >> 4);
      const uint64_t b0 = k0 + x.slot * (C::SLOT >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
          const uint32_t o = ((k >> 2) * (kM * 128) + (k & 3) * 32) >> 4;
          mma_bf16(C::T_S + s * 128, a0 + o, b0 + o, kIdescS, k > 0 ? 1u : 0u);
        }
        mma_commit(BAR(C::S_FULL + s));
        if (last) mma_commit(BAR(C::Q_EMPTY + s));
      }
      __syncwarp();
    };
    auto issue_o = [&](int s, Ring x, bool first, bool last) {
      const uint64_t b0 = v0 + x.slot * (C::SLOT >> 4);
      all_wait(C::FULL + x.slot, x.phase);
      all_wait(C::P_READY + s, pn[s] & 1);
      ++pn[s];
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kN / 16; ++k)
          mma_16_ts(C::T_O + s * 128, C::T_S + s * 128 + 8 * k, b0 + k * (2048 >> 4), kIdescO,
                    (first && k == 0) ? 0u : 1u);
        if (last) mma_commit(BAR(C::O_DONE + s));
      }
      __syncwarp();
    };
    auto give_back = [&](Ring x) {  // (some side has waited for its copy)
      if (elect_one()) mma_commit(BAR(C::EMPTY + x.slot));
      __syncwarp();
    };
    Todo cur = next_seg();
    bool primed = false;  // the segment's first S are out already
    while (cur.T > 0 && ok) {
      if (cur.twin) {
        // (K, V of tile t at positions 2 t, 2 t + 1; tile t is side t & 1's)
        Ring k = at;
        issue_s(0, k, true, cur.nt[0] == 1);
        give_back(k);
        if (cur.nt[1] > 0) {
          k = at.next().next();
          issue_s(1, k, true, cur.nt[1] == 1);
          give_back(k);
        }
        for (int t = 0; t < cur.T && ok; t += 2) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (t + s >= cur.T) break;
            at = at.next();
            issue_o(s, at, t == 0, t + s + 2 >= cur.T);
            give_back(at);
            at = at.next();
            k = at.next().next();
            if (t + s + 2 < cur.T) {
              issue_s(s, k, false, t + s + 4 >= cur.T);
              give_back(k);
            }
          }
        }
        cur = next_seg();
        continue;
      }
      if (!primed) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (cur.nt[s] > 0) issue_s(s, at, true, cur.nt[s] == 1);
        give_back(at);
        at = at.next();
      }
      Todo nx = {0, {0, 0}, false};
      // rounds in which both sides have a P.V and an S that is not their last
      const int inner = min(cur.nt[0], cur.nt[1]) - 1;
      for (int t = 1; t <= cur.T && ok; ++t) {
        const Ring v = at, k = at.next();
        if (t >= 2 && t < inner) {
          // as below, with as little as can be between one side's products
          // and the other's
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            ok = __all_sync(0xffffffffu,
                            ok && (s == 1 || (wait(C::FULL + v.slot, v.phase) &&
                                              wait(C::FULL + k.slot, k.phase))) &&
                                wait(C::P_READY + s, pn[s] & 1));
            ++pn[s];
            if (!ok) break;
            tc_fence_after();
            const uint64_t vb = v0 + v.slot * (C::SLOT >> 4), kb = k0 + k.slot * (C::SLOT >> 4);
            const uint64_t qa = q0 + ((s * C::Q_BYTES) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int e = 0; e < kN / 16; ++e)
                mma_16_ts(C::T_O + s * 128, C::T_S + s * 128 + 8 * e, vb + e * (2048 >> 4), kIdescO,
                          1u);
              if (s == 1) mma_commit(BAR(C::EMPTY + v.slot));
#pragma unroll
              for (int e = 0; e < DK / 16; ++e) {
                const uint32_t o = ((e >> 2) * (kM * 128) + (e & 3) * 32) >> 4;
                mma_bf16(C::T_S + s * 128, qa + o, kb + o, kIdescS, e > 0 ? 1u : 0u);
              }
              mma_commit(BAR(C::S_FULL + s));
              if (s == 1) mma_commit(BAR(C::EMPTY + k.slot));
            }
            __syncwarp();
          }
          at = k.next();
          continue;
        }
        if (t == cur.T) {
          nx = next_seg();
          primed = nx.T > 0 && !nx.twin;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (t <= cur.nt[s]) issue_o(s, v, t == 1, t == cur.nt[s]);
          if (t < cur.T) {
            if (t < cur.nt[s]) issue_s(s, k, false, t == cur.nt[s] - 1);
          } else if (primed && nx.nt[s] > 0) {
            issue_s(s, k, true, nx.nt[s] == 1);
          }
        }
        give_back(v);
        at = k;
        if (t < cur.T || primed) {
          give_back(k);
          at = k.next();
        }
      }
      cur = nx;
    }
    // every product has to be finished before tensor memory is released
    if (elect_one()) {
      mma_commit(BAR(C::DRAIN));
      const long long t0 = clock64();
      while (!mbar_try_wait(BAR(C::DRAIN), 0) && clock64() - t0 < p.budget) {
      }
    }
    __syncwarp();
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
    int d_head = 0, d_tok0 = 0, d_ntok = 0, d_j = 0, d_end = 0;
    bool ok = true;
    for (uint32_t kn = 0;; ++kn) {
      ok = ok && __all_sync(0xffffffffu, wait(C::SEG_FULL + kn % kSegs, (kn / kSegs) & 1));
      if (!ok) break;
      const ChunkSeg seg = *seg_at(kn);
      __syncwarp();
      mbar_arrive_if(BAR(C::SEG_EMPTY + kn % kSegs), lane == 0);
      if (seg.lt1 == seg.lt0) break;
      const int nt = seg.side_tiles(side, p.tq);
      const bool whole = seg.lt0 == 0 && seg.lt1 == seg.ti;
      const bool twin = seg.twin(p.tq);
      const int tok0 = twin ? 0 : side * p.tq;
      const int my_tok = tok0 + tok;  // token of the unit
      const bool live = tok < p.tq && my_tok < seg.ntok;
      const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (seg.lt0 == 0 ? 1 : 0);
      if (seg.lt0 == 0 && !whole) {
        d_head = 1;
        d_tok0 = seg.t0;
        d_ntok = seg.ntok;
        d_j = seg.j;
      } else if (seg.lt0 > 0) {
        d_end = seg.lt1 == seg.ti;
      }
      // (lanes without a row hold anything: with their maximum at infinity they
      // have no say in when the others' is raised)
      float m = live ? -INFINITY : INFINITY, l = 0.f;
      const int my_pos = seg.pos0 + my_tok;
      const int first_pos = seg.pos0 + tok0;  // the side's first token
      for (int t = 0; t < nt; ++t) {
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
        const int base = (seg.lt0 + (twin ? 2 * t + side : t)) * kN;
        if (base + kN - 1 > first_pos) {
          // positions past this row's token, 32 at a time (those that the
          // side's first token sees need no mask)
          const int lim = my_pos - base;
#pragma unroll
          for (int c = 0; c < kN / 32; ++c) {
            if (base + 32 * c + 31 <= first_pos) continue;  // (uniform)
            const int see = lim + 1 - 32 * c;
            const uint32_t bits = see >= 32 ? ~0u : see <= 0 ? 0u : (1u << see) - 1u;
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
        // up to the last tile
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
        __syncwarp();
        mbar_arrive_if(BAR(C::P_READY + side), lane == 0);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      // ---- unit's end: O / l, or a partial (maximum, sum, O) ----
      // (twins: each side joins and writes half of the columns of both)
      const int other = twin ? seg.side_tiles(side ^ 1, p.tq) : 0;
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
      const size_t at = slot * p.srows + (twin ? 0 : side * kM);
      if (!whole && live && (!twin || side == 0)) {
        p.part_ml[2 * (at + row)] = ms;
        p.part_ml[2 * (at + row) + 1] = l;
      }
      // A thread writes its own row, in whole 32-byte sectors where the output
      // is aligned to them.  (Rows turned in shared memory or by shuffles
      // between four lanes touch fewer lines a store but cost more
      // instructions: 155 and 149 us for a mixed batch of prompts, chunks and
      // single tokens where this took 142.)
      T16* const dst = static_cast<T16*>(p.out) +
                       (static_cast<size_t>(seg.t0 + my_tok) * p.h + seg.j * p.r + head) * DV;
      float* const pdst = p.part_o + (at + row) * DV;
      const float fo = whole ? wo * inv : wo, ft = whole ? wt * inv : wt;
      for (int c = c0; c < c1; ++c) {
        if (nt == 0 && other == 0) break;  // (a side without tokens)
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
        if (!live) continue;
        if (whole) {
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
      tc_fence_before();
      if (twin) {  // both O and ml_sm are free again
        __syncwarp();
        mbar_arrive_if(BAR(C::TWIN + 1), lane == 0);
        ok = __all_sync(0xffffffffu, wait(C::TWIN + 1, tn & 1));
        ++tn;
      }
    }
    if (threadIdx.x == 0) {
      int* d = p.desc + static_cast<size_t>(blockIdx.x) * kDescInts;
      d[D_HEAD] = ok ? d_head : 0;
      d[D_TOK0] = d_tok0;
      d[D_NTOK] = d_ntok;
      d[D_J] = d_j;
      d[D_END] = ok ? d_end : 1;
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
template <typename T16, int DK, int DV, bool PAGED>
struct CausalLaunch {
  static cudaError_t run(const ChunkCall& x, const ChunkPlan& pl, int num_sms,
                         unsigned int* status, cudaStream_t st) {
    using C = ChunkCfg<DK, DV>;
    ChunkParams p;
    chunk_args(p, x, pl, status);
    CUtensorMap mq, mk, mv;
    if (!map_q<T16, DK>(&mq, x, p.tq) || !map_kv<T16, DK, DV>(&mk, &mv, x, kN))
      return cudaErrorInvalidValue;
    auto kern = chunk_attn_kernel<T16, DK, DV, PAGED>;
    static std::atomic<unsigned long long> configured{0};
    if (cudaError_t e = chunk_configure(kern, C::SMEM, configured)) return e;
    ChunkLaunch l(num_sms, C::SMEM, st);
    if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, mq, mk, mv, p)) return e;
    return launch_join<T16, DV>(l.cfg, p, num_sms);
  }
};

int chunk_run(const ChunkCall& x, void* stream) {
  if (int e = chunk_check(x)) return e;
  int num_sms = 0;
  unsigned int* status = nullptr;
  if (int e = device_query(&num_sms, &status)) return e;
  const ChunkPlan pl = chunk_plan(x.total, x.h, x.g, x.dv, num_sms);
  if (x.ws_bytes < static_cast<long long>(pl.bytes)) return GQA_ERR_SCRATCH_LIMIT;
  if (x.total == 0) return GQA_OK;
  const cudaError_t e = chunk_dispatch<CausalLaunch>(x, pl, num_sms, status,
                                                     static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

int gqa_chunk_attn(const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* cu_tokens, const int32_t* seq_lens, int b, int total, int h,
                   int g, int d_k, int d_v, float scale, void* out, int cap, int dtype,
                   void* workspace, long long workspace_bytes, void* stream) {
  const ChunkCall x = {q, k_cache, v_cache, cu_tokens, seq_lens, nullptr, b, total, h, g, d_k,
                       d_v, scale, out, cap, 0, 0, 0, dtype, workspace, workspace_bytes};
  return chunk_run(x, stream);
}

int gqa_chunk_attn_paged(const void* q, const void* k_pool, const void* v_pool,
                         const int32_t* block_table, const int32_t* cu_tokens,
                         const int32_t* seq_lens, int b, int total, int h, int g, int d_k,
                         int d_v, float scale, void* out, int block_size, int max_blocks,
                         int num_blocks, int dtype, void* workspace, long long workspace_bytes,
                         void* stream) {
  if (int e = paged_args_check(block_table, g, block_size, max_blocks, num_blocks)) return e;
  const ChunkCall x = {q, k_pool, v_pool, cu_tokens, seq_lens, block_table, b, total, h, g, d_k,
                       d_v, scale, out, max_blocks * block_size, block_size, max_blocks,
                       num_blocks, dtype, workspace, workspace_bytes};
  return chunk_run(x, stream);
}

int gqa_chunk_attn_workspace(int total, int h, int g, int d_k, int d_v, int num_sms,
                             long long* bytes) {
  if (!bytes) return GQA_ERR_NULL;
  if (num_sms < 0) return GQA_ERR_SHAPE;
  if (int e = chunk_shape_check(total, h, g, d_k, d_v)) return e;
  if (num_sms == 0) {
    unsigned int* status = nullptr;
    if (int e = device_query(&num_sms, &status)) return e;
  }
  *bytes = static_cast<long long>(chunk_plan(total, h, g, d_v, num_sms).bytes);
  return GQA_OK;
}

}  // extern "C"
