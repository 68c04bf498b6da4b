// chunk_part.cu - attention of packed chunks over a part of the cache (a sliding
// window and the first positions) and over a prefix that the batch shares: the
// kernel of chunk_kernel.cuh, and its split of work.
//
// Window.  A token at position P sees p <= P with p > P - window or p < sinks.
// A unit of ntok tokens reads the span (part_device.cuh) of ceil(sinks / 64) *
// 64 + window + ntok - 1 positions at most, not the P + 1 of the causal form (up to
// 63 more where a paged window's first box, 64 positions or a block, begins before
// it; the split of work leaves those out); its first and last tiles are masked row
// by row, the others are seen whole.
//
// Prefix.  Positions below prefix_len are the same rows for every sequence.
// Where sequences bring few tokens, the prefix is attended by units of its own
// over the packed rows of all sequences (2 tq tokens to a unit, so 64 single
// tokens of eight heads read it twice instead of 64 times), each sequence's
// own positions by units as ever, and every row is joined from both: partial
// results of units that no run's end cuts lie by row, the others by CTA.  With
// units that one sequence fills the prefix is the head of the unit's span: the
// tiles read are the same and nothing has to be joined.
//
// Measured (graph replay, bf16, d = 128, over several GPUs; floors at the measured
// copy and GEMM rates).  64 single tokens over windows of 4,096, h = 64, g = 8, 64-row
// blocks: 168 to 170 us, 6,250 GB/s (157): HBM, then 4 us of start and the join.  A
// prompt of 8,192 in a window of 2,048: 350 to 371 us (254): 17 tiles a unit of 32
// tokens where 16 are seen, 4 us from one unit to the next (three tiles' time), the
// clock under load.  32 mixed sequences, 7,506 tokens, window 1,000: 121 to 125 us
// (38): units of six tiles, join.  64 single tokens behind a prefix of 8,192: 57 us
// (22): 512 units of five tiles and the prefix's long ones beside them.  16 chunks of
// 50 to 400 tokens behind 6,000: 211 to 224 us (147).
//
// Boxes of 64 positions (or a block): with 128, a few sinks cost a whole tile and
// a window begins up to 127 positions early; with 16, a tile is 64 copies.
// Contiguous windows begin at any row.
#include "chunk_kernel.cuh"

namespace gqa {
namespace {

// Are the prefix's units to be shared by the sequences?  (b sequences with `rows`
// packed rows in all; tq: tokens of a side.)  Shared, a row's two results are
// written, read back and joined, which grows with the rows; not shared, every
// sequence reads the prefix for its own rows, which grows with the prefix.  With
// fewer than 64 units (a sequence and KV head each) those are cut among the SMs
// anyway, and their tiles cost no time that a few rows' join would not.
// Measured, us shared / not, n tokens a sequence:
//   16 sequences, h = 32, g = 8 (tq = 32): behind 700 n = 1 18.0 / 20.0, 4 21.6 /
//     21.2, 31 37.3 / 27.1; 1,400 n = 8 25.0 / 26.9, 16 31.4 / 29.7; 2,500 n = 16
//     35.2 / 36.5, 31 48.2 / 41.8; 6,000 n = 31 63.2 / 68.9
//   64, h = 64, g = 8 (16): 350 n = 1 37.0 / 40.2, 2 44.1 / 40.4; 1,400 n = 4 62.0 /
//     66.4, 8 79.1 / 69.1; 3,500 n = 8 104 / 124, 15 151 / 141; 8,192 n = 15 228 / 282
//   12, h = 64, g = 8: 350 n = 1 16.1 / 16.1, 2 17.5 / 17.1
//   128, h = 8, g = 2 (32): 350 n = 1 29.1 / 27.9; 700 n = 1 28.4 / 31.9
//   32, h = 8, g = 1 (16), so 32 units: 3,000 n = 1 21.4 / 18.8, 8 23.8 / 24.4; 6,000
//     n = 1 24.8 / 23.4, 15 28.1 / 32.1
//   4, h = 28, g = 4 (18), 16 units: 700 n = 1 14.5 / 13.6, 17 18.8 / 18.2; 1,400 n = 8
//     18.5 / 19.3; 6,000 n = 1 19.3 / 17.9, 17 26.9 / 29.1
//   2, h = 32, g = 8, 16 units: 20,000 n = 1 28.8 / 30.9
__host__ __device__ __forceinline__ bool prefix_grouped(int b, int rows, int tq, int g,
                                                        int prefix_len) {
  const long long room = static_cast<long long>(b) * tq;  // rows that fill a side for each
  if (b < 2 || prefix_len < 1 || rows >= room) return false;
  const float units = static_cast<float>(b) * static_cast<float>(g);
  const float reads = units * static_cast<float>(prefix_len);  // positions, not shared
  if (units < 64.f) return 8ll * rows >= 3 * room ? prefix_len >= 1024 : reads >= 160000.f;
  return 4096ll * rows <= room * prefix_len && reads >= 80000.f;
}

// Rows that may share at most, of up to b sequences and `total` rows (0: none).
int group_rows(int b, int total, int tq, int prefix_len) {
  if (b < 2 || prefix_len < 1) return 0;
  return static_cast<int>(std::min<long long>(total, static_cast<long long>(b) * tq - 1));
}

struct PartSeg {
  int i, j;        // sequence, KV head
  int t0;          // packed row of the unit's first token
  int pos0;        // its position
  int ntok;        // tokens of the unit
  int lt0, lt1;    // tiles of the unit taken here
  int ti;          // tiles of the unit
  int L;           // positions of the body end here
  int head;        // positions of the span's head
  int shift, sb, z, end;  // the span (end: of its last position seen by the sequence)
  bool of_head;    // a unit over the head alone, for rows of all sequences
  __device__ bool twin(int tq) const { return ntok <= tq; }
  __device__ int side_tiles(int side, int tq) const {
    const int nt = min(ntok - side * tq, tq);
    const int ext = of_head ? head : pos0 + side * tq + nt - shift;
    return max(0, min(lt1, (ext + kN - 1) / kN) - lt0);
  }
  // what the tokens from tok0 on see, the side's last one being tq tokens on
  __device__ void sees(const ChunkParams& p, int tok0, SegPlan::Side& v, int& lo_min) const {
    const int last = min(tok0 + p.tq, ntok) - 1;
    v.hi = pos0 + tok0 + 1 - shift;
    v.lo = pos0 + tok0 - p.window + 1 - shift;
    lo_min = p.base_min - shift;
    if (of_head) {  // (no index of it is behind the head)
      v.hi = 0x7FFFFF00;
      v.lo = 0;
      lo_min = 0x7FFFFFFF;
    }
    v.all_hi = v.hi;
    v.all_head = min(head, v.hi);
    v.all_lo = max(v.lo + last - tok0, lo_min);
    if (v.all_lo <= v.all_head) v.all_lo = 0;
  }
};

// The run of work of one CTA, as in chunk_attn.cu.  A sequence's units grow with
// the position of their last token until the window is full and are alike from
// there on, so sums of their work are an arithmetic progression and a multiple.
// Units of the head come before those of the sequences, as sequence -1.
//
// Every instruction of the walk is fetched once a launch before any copy can
// start, so it is written for few of them, not for few steps: one scan for the
// sum and the search, the two warps that look for a run's ends in the same code,
// divisions by multiplication.  (With five scans and 64-bit divisions inlined a
// call took 5 us longer with one sequence, 15 with 64.)
constexpr unsigned kPartUnitCost = 400;
constexpr unsigned kPartNear = 2;  // tiles

struct PartWalk {
  using Seg = PartSeg;

  const ChunkParams& p;
  int n_head;    // packed rows of the head's units (0: it has none)
  int gran, head_pad;
  ChunkPos at, end;
  int t0, n, L;  // of sequence at.i
  bool more;

  __device__ explicit PartWalk(const ChunkParams& params) : p(params) {
    n_head = head_rows(p);
    gran = p.table != nullptr ? min(p.bsz, kGrain) : kGrain;
    head_pad = (p.head + gran - 1) & ~(gran - 1);
  }

  __device__ static unsigned errors(int a0, int a1, int Lk, int total, long long cap,
                                    int base_min) {
    if (const unsigned e = packed_errors(a0, a1, Lk, total, cap)) return e;
    return a1 > a0 && Lk - (a1 - a0) < base_min ? GQA_DEV_BAD_SEQ_LEN : 0u;
  }
  __device__ static void report(const ChunkParams& p) {
    unsigned bad = 0;
    for (int i = threadIdx.x & 31; i < p.b; i += 32)
      bad |= errors(__ldg(p.cu + i), __ldg(p.cu + i + 1), __ldg(p.lens + i), p.total, p.cap,
                    p.base_min);
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (bad && (threadIdx.x & 31) == 0) atomicOr(p.status, bad);
  }
  // Rows that units of the head's own hold (0: it has none): up to the end of the
  // last usable sequence.  (The entries of cu behind an unusable one say nothing,
  // cu[b] among them.)  Decided by the tokens that are there, not by the call's
  // `total` and b, which may leave room for more.  Warp-cooperative.
  __device__ static int head_rows(const ChunkParams& p) {
    if (p.group_rows == 0) return 0;
    int end = 0, count = 0;
    for (int i = threadIdx.x & 31; i < p.b; i += 32) {
      const int a0 = __ldg(p.cu + i), a1 = __ldg(p.cu + i + 1);
      if (a1 > a0 && !errors(a0, a1, __ldg(p.lens + i), p.total, p.cap, p.base_min)) {
        end = max(end, a1);
        ++count;
      }
    }
    end = __reduce_max_sync(0xffffffffu, end);
    count = __reduce_add_sync(0xffffffffu, count);
    return prefix_grouped(count, end, p.tq, p.g, p.head) ? end : 0;
  }
  // Does usable sequence i hold packed row t?
  __device__ static bool holds(const ChunkParams& p, int i, int t) {
    const int a0 = __ldg(p.cu + i), a1 = __ldg(p.cu + i + 1);
    return a0 <= t && t < a1 && !errors(a0, a1, __ldg(p.lens + i), p.total, p.cap, p.base_min);
  }
  // The usable sequence that holds packed row t (p.b: none).  cu need not ascend
  // around an unusable sequence: where the search by it misses, every sequence is
  // looked at.  Warp-cooperative.
  __device__ static int sequence_of(const ChunkParams& p, int t) {
    const int i = packed_sequence(p.cu, p.b, t);
    if (i < p.b && holds(p, i, t)) return i;
    for (int base = 0; base < p.b; base += 32) {
      const int k = base + (threadIdx.x & 31);
      const unsigned hit = __ballot_sync(0xffffffffu, k < p.b && holds(p, k, t));
      if (hit) return base + __ffs(hit) - 1;
    }
    return p.b;
  }
  template <typename T16, int DV>
  static cudaError_t join(cudaLaunchConfig_t& cfg, const ChunkParams& p, int num_sms);

  // sequence k (-1: the head)
  __device__ bool seq(int k, int& a0, int& nn, int& Lk) const {
    a0 = nn = Lk = 0;
    if (k < 0) {
      nn = n_head;
      Lk = p.head;
    } else if (k < p.b) {
      a0 = __ldg(p.cu + k);
      const int a1 = __ldg(p.cu + k + 1);
      Lk = __ldg(p.lens + k);
      if (!errors(a0, a1, Lk, p.total, p.cap, p.base_min)) nn = a1 - a0;
    }
    return nn > 0;
  }
  // x / (2 tq): 2^32 / (2 tq) rounded up is at most one too large
  __device__ unsigned by_unit(unsigned x) const {
    const unsigned q = __umulhi(x, p.unit_inv), d = 2 * p.tq;
    return q * d > x ? q - 1 : q;
  }
  __device__ int units(int nn) const { return by_unit(static_cast<unsigned>(nn) + 2 * p.tq - 1); }

  // A unit q has min(A + (q + 1) * 2 tq, B) positions (as the split counts them:
  // tiles are cut from the exact span).
  struct Shape {
    unsigned A, B;
    int nu, q0;  // units; those before the window is full
    bool tw;     // the last one is a unit of twins
  };
  __device__ Shape shape(int k, int nn, int Lk) const {
    Shape s;
    const unsigned pad = n_head > 0 ? 0 : head_pad;
    s.nu = units(nn);
    s.tw = nn - (s.nu - 1) * 2 * p.tq <= p.tq;
    s.A = Lk - nn - p.base_min + (p.head_seq >= 0 ? pad : 0);
    s.B = p.head_seq >= 0 ? 0xF0000000u : static_cast<unsigned>(p.window) + 2 * p.tq + pad;
    if (k < 0) s.A = s.B = p.head;
    s.q0 = s.B <= s.A ? 0 : min(s.nu, static_cast<int>(by_unit(s.B - s.A)));
    return s;
  }
  using U64 = unsigned long long;
  __device__ U64 prefix(unsigned q, const Shape& s) const {
    const unsigned k = min(q, static_cast<unsigned>(s.q0));
    return static_cast<U64>(k) * (s.A + kPartUnitCost) + static_cast<U64>(k * p.tq) * (k + 1) +
           static_cast<U64>(q - k) * (s.B + kPartUnitCost);
  }
  __device__ unsigned length(unsigned q, const Shape& s) const {
    return static_cast<int>(q) < s.q0 ? s.A + (q + 1) * 2 * p.tq : s.B;
  }

  // the span and the tiles of unit q of sequence k
  __device__ void span(Seg& s, int k, int q, int nn, int Lk) const {
    const int first = q * 2 * p.tq;
    s.of_head = k < 0;
    s.pos0 = Lk - nn + first;
    s.ntok = min(nn - first, 2 * p.tq);
    s.L = Lk;
    s.head = n_head > 0 && k >= 0 ? 0 : p.head;
    const int lo = max(p.base_min, s.pos0 - p.window + 1);
    const int lo_all = max(p.base_min, Lk - nn - p.window + 1);
    const PartSpan t = part_span(lo, lo_all, s.head, gran, p.table != nullptr,
                                 p.head_seq >= 0);
    s.shift = k < 0 ? 0 : t.shift;
    s.sb = k < 0 ? head_pad : t.sb;
    s.z = k < 0 ? 0 : t.z;
    s.end = Lk - s.shift;
    const int hi = k < 0 ? Lk : s.pos0 + s.ntok - t.shift;
    s.ti = (hi + kN - 1) >> 7;
  }

  // The place where run c begins (the end of the last run for c = their number):
  // false when the launch has fewer runs than that.
  __device__ bool start(int c, int nc, ChunkPos& r) {
    const int lane = threadIdx.x & 31;
    const int k0 = n_head > 0 ? -1 : 0;
    U64 W = 0, x = 0;
    unsigned near = 0;
    r = {p.b, 0, 0, 0};
    // the first pass sums the work, the second one finds the place of x
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      U64 before = 0;  // (of one KV head)
#pragma unroll 1
      for (int base = k0; base < p.b; base += 32) {
        int a0, nn, Lk;
        U64 f = 0;
        if (seq(base + lane, a0, nn, Lk)) {
          const Shape s = shape(base + lane, nn, Lk);
          f = prefix(s.nu, s);
          if (s.tw) f -= length(s.nu - 1, s) >> 2;  // (three quarters of it)
        }
        U64 incl = f;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const U64 y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (pass == 1) {
          const U64 hi = (before + incl) * p.g, lo = hi - f * p.g;
          const unsigned hit = __ballot_sync(0xffffffffu, f > 0 && lo <= x && x < hi);
          if (hit) {
            const int src = __ffs(hit) - 1;
            t0 = __shfl_sync(0xffffffffu, a0, src);
            n = __shfl_sync(0xffffffffu, nn, src);
            L = __shfl_sync(0xffffffffu, Lk, src);
            r.i = base + src;
            U64 rem = x - __shfl_sync(0xffffffffu, lo, src);
            const U64 fs = __shfl_sync(0xffffffffu, f, src);
            // (g is small: steps instead of a 64-bit division)
            r.j = 0;
#pragma unroll 1
            for (int step = 1 << (31 - __clz(p.g)); step > 0; step >>= 1)
              if (r.j + step < p.g && (r.j + step) * fs <= rem) r.j += step;
            rem -= r.j * fs;
            // the last unit q with prefix(q) <= rem
            const Shape s = shape(r.i, n, L);
            int q = 0;
#pragma unroll 1
            for (int step = s.nu > 1 ? 1 << (31 - __clz(s.nu - 1)) : 0; step > 0; step >>= 1)
              if (q + step < s.nu && prefix(q + step, s) <= rem) q += step;
            r.qt = q;
            unsigned in = static_cast<unsigned>(rem - prefix(q, s));
            if (q == s.nu - 1 && s.tw) in += in / 3;
            const unsigned lt = in >> 7, ti = (length(q, s) + kN - 1) >> 7;
            r.lt = lt <= near ? 0 : lt + near >= ti ? 0x7FFFFFFF : static_cast<int>(lt);
            if (c == 0) r.lt = 0;
            return true;
          }
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (pass == 0) {
        W = before * p.g;
        // (a run is worth at least a tile, two with much work)
        const U64 most = W / (2 * kN) + 1;
        if (most < static_cast<U64>(nc)) nc = static_cast<int>(most);
        if (W == 0 || c > nc) return false;
        if (c == nc) return true;
        const U64 run = div_pos(W, nc);
        near = min(static_cast<unsigned>(run / (32 * kN)), kPartNear);
        const int left = static_cast<int>(W - run * nc);  // the first `left` runs are one longer
        x = run * c + min(c, left);
      }
    }
    return true;  // not reached for x < W
  }

  __device__ void begin(const ChunkPos& from, const ChunkPos& e) {
    at = from;
    end = e;
    more = at.i < p.b;
  }

  __device__ bool next(Seg& s) {
    while (more) {
      const bool last = at.i == end.i && at.j == end.j && at.qt == end.qt;
      const bool past = at.i > end.i || (at.i == end.i && (at.j > end.j ||
                                         (at.j == end.j && at.qt > end.qt)));
      if (past || (last && end.lt <= at.lt)) break;
      span(s, at.i, at.qt, n, L);
      s.i = max(at.i, 0);
      s.j = at.j;
      s.t0 = t0 + at.qt * 2 * p.tq;
      s.lt0 = at.lt;
      s.lt1 = last ? min(end.lt, s.ti) : s.ti;
      more = !last;
      if (!last) {  // to the next unit's start
        at.lt = 0;
        if (++at.qt >= units(n)) {
          at.qt = 0;
          if (++at.j >= p.g) {
            at.j = 0;
            do {
              ++at.i;
            } while (at.i < p.b && !seq(at.i, t0, n, L));
            more = at.i < p.b;
          }
        }
      }
      if (s.lt0 < s.lt1) return true;
    }
    more = false;
    return false;
  }
};

// Joins, for a row of two query heads of a token's group, the partial results over the
// head and over the sequence's own positions, each whole (by row) or in pieces (by
// CTA), by a warp, four pieces of both heads with their loads side by side.
template <typename T16, int DV>
__device__ __forceinline__ void join_group(const ChunkParams& p, int nc, int t, int j,
                                           int a_first) {
  constexpr int CPL = DV / 32;
  constexpr int NP = 4;
  const int lane = threadIdx.x & 31;
  const int i = PartWalk::sequence_of(p, t);
  if (i >= p.b) return;
  const int a0 = __ldg(p.cu + i);
  // the units that hold the token: over the head, over its own positions
  const int w = 2 * p.tq;
  const int u0[2] = {t / w * w, a0 + (t - a0) / w * w};
  int first[2], cnt[2], row0[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const size_t units = static_cast<size_t>(p.group_rows) * p.g;
    const int* cut = p.cut + (2 * k) * units + static_cast<size_t>(u0[k]) * p.g + j;
    // (held within the launch's CTAs: where a wait gave up they may not have
    // been written)
    first[k] = min(max(__ldg(cut), -1), nc - 1);
    cnt[k] = first[k] < 0 ? 1 : min(max(__ldg(cut + units), first[k]), nc - 1) - first[k] + 1;
    const int tok = t - u0[k], side = tok >= p.tq ? 1 : 0;
    row0[k] = side * kM + (tok - side * p.tq) * p.r;
  }
  const int all = cnt[0] + cnt[1];
  const size_t orow = static_cast<size_t>(t) * p.h + j * p.r;
  float M[2] = {-INFINITY, -INFINITY}, den[2] = {0.f, 0.f}, num[2][CPL];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int e = 0; e < CPL; ++e) num[s][e] = 0.f;
  for (int k0 = 0; k0 < all; k0 += NP) {
    float2 ml[2][NP];
    float o[2][NP][CPL];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int a = a_first + s;
        const bool use = k0 + k < all && a < p.r;
        const bool own = k0 + k >= cnt[0];
        const int x = own ? first[1] + (k0 + k - cnt[0]) : first[0] + k0 + k;  // its CTA
        const bool by_row = own ? first[1] < 0 : first[0] < 0;
        const size_t at =
            by_row ? (own ? static_cast<size_t>(p.group_rows) * p.h : 0) + orow + a
                   : static_cast<size_t>(2 * x + (x == (own ? first[1] : first[0]) ? 1 : 0)) *
                             p.srows +
                         (own ? row0[1] : row0[0]) + a;
        const float* pm = by_row ? p.row_ml : p.part_ml;
        const float* src = (by_row ? p.row_o : p.part_o) + at * DV + lane * CPL;
        ml[s][k] = use ? __ldg(reinterpret_cast<const float2*>(pm) + at)
                       : make_float2(-INFINITY, 0.f);
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
    if (a_first + s >= p.r) continue;
    const float inv = 1.f / den[s];
    T16* dst = static_cast<T16*>(p.out) + (orow + a_first + s) * DV + lane * CPL;
    if constexpr (CPL == 4) {
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(Half16<T16>::pack2(num[s][0] * inv, num[s][1] * inv),
                     Half16<T16>::pack2(num[s][2] * inv, num[s][3] * inv));
    } else {
      *reinterpret_cast<uint32_t*>(dst) = Half16<T16>::pack2(num[s][0] * inv, num[s][1] * inv);
    }
  }
}

// What follows a launch whose head may have had units of its own: the rows of both
// kinds if it had, else the units that a run's end cut, half a side to a block.
constexpr int kGroupThreads = 256;

template <typename T16, int DV>
__global__ void __launch_bounds__(kGroupThreads) group_join_kernel(const ChunkParams p, int nc) {
  pdl_wait_then_release();
  constexpr int kWarps = kGroupThreads / 32;
  // (held within what the workspace has room for)
  const int rows = min(__ldg(p.desc + D_ROWS), p.group_rows);
  if (rows <= 0) {
    const int sides = p.srows / kM, c = blockIdx.x / (2 * sides), k = blockIdx.x % (2 * sides);
    if (c < nc)
      join_rows<T16, DV, kWarps>(p, nc, c, k >> 1, (k & 1) * (kM / 2), ((k & 1) + 1) * (kM / 2));
    return;
  }
  const int pairs = (p.r + 1) >> 1;
  const long long n = static_cast<long long>(rows) * p.g * pairs;
  for (long long id = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); id < n;
       id += static_cast<long long>(gridDim.x) * kWarps) {
    const long long tj = id / pairs;
    const int t = static_cast<int>(tj / p.g);
    join_group<T16, DV>(p, nc, t, static_cast<int>(tj - static_cast<long long>(t) * p.g),
                        2 * static_cast<int>(id - tj * pairs));
  }
}

template <typename T16, int DV>
cudaError_t PartWalk::join(cudaLaunchConfig_t& cfg, const ChunkParams& p, int num_sms) {
  if (p.group_rows == 0) return launch_join<T16, DV>(cfg, p, num_sms);
  // (Rows are taken by turns, so any grid does; units cut need four blocks an SM.
  // 64 tokens behind 8,192, us: four an SM 63.7, eight 57.1, sixteen 57.6.)
  cfg.gridDim = dim3(8 * num_sms);
  cfg.blockDim = dim3(kGroupThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, group_join_kernel<T16, DV>, p, num_sms);
}

template <typename T16, int DK, int DV, bool PAGED>
struct PartLaunch {
  static cudaError_t run(const PartCall& x, const PartPlan& pl, int num_sms, unsigned int* status,
                         cudaStream_t st) {
    return launch_chunk<T16, DK, DV, PAGED, PartWalk>(x, pl, num_sms, status, st);
  }
};

int part_run(const PartCall& x, void* stream) {
  if (int e = chunk_check(x)) return e;
  if (x.cap > 0x7FFFFF00) return GQA_ERR_SHAPE;  // (indices of a span stay within 31 bits)
  int num_sms = 0;
  unsigned int* status = nullptr;
  if (int e = device_query(&num_sms, &status)) return e;
  const PartPlan pl = part_plan(x.total, x.h, x.g, x.dv, num_sms, x.group_rows);
  if (x.ws_bytes < static_cast<long long>(pl.bytes)) return GQA_ERR_SCRATCH_LIMIT;
  if (x.total == 0) return GQA_OK;
  const cudaError_t e =
      chunk_dispatch<PartLaunch>(x, pl, num_sms, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

// (cap: positions that the cache can hold)
int window_run(PartCall& x, int window, int sinks, void* stream) {
  if (window < 1 || sinks < 0) return GQA_ERR_SHAPE;
  x.window = std::min(window, std::max(x.cap, 1));
  x.head = std::min(sinks, std::max(x.cap, 0));
  return part_run(x, stream);
}

int prefix_run(PartCall& x, int prefix_len, void* stream) {
  if (prefix_len < 0 || (x.cap >= 1 && prefix_len > x.cap)) return GQA_ERR_SHAPE;
  x.window = std::max(x.cap, 1);
  x.head = x.base_min = prefix_len;
  x.head_seq = 0;
  if (x.g > 0 && x.h > 0 && x.h / x.g >= 1 && x.h / x.g <= kM)
    x.group_rows = group_rows(x.b, x.total, kM / (x.h / x.g), prefix_len);
  return part_run(x, stream);
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

int gqa_chunk_attn_window(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* cu_tokens, const int32_t* seq_lens, int b, int total,
                          int h, int g, int d_k, int d_v, float scale, int window, int sinks,
                          void* out, int cap, int dtype, void* workspace,
                          long long workspace_bytes, void* stream) {
  PartCall x;
  static_cast<ChunkCall&>(x) = {q, k_cache, v_cache, cu_tokens, seq_lens, nullptr, b, total, h, g,
                                d_k, d_v, scale, out, cap, 0, 0, 0, dtype, workspace,
                                workspace_bytes};
  return window_run(x, window, sinks, stream);
}

int gqa_chunk_attn_window_paged(const void* q, const void* k_pool, const void* v_pool,
                                const int32_t* block_table, const int32_t* cu_tokens,
                                const int32_t* seq_lens, int b, int total, int h, int g, int d_k,
                                int d_v, float scale, int window, int sinks, void* out,
                                int block_size, int max_blocks, int num_blocks, int dtype,
                                void* workspace, long long workspace_bytes, void* stream) {
  if (int e = paged_args_check(block_table, g, block_size, max_blocks, num_blocks)) return e;
  PartCall x;
  static_cast<ChunkCall&>(x) = {q, k_pool, v_pool, cu_tokens, seq_lens, block_table, b, total, h, g,
                                d_k, d_v, scale, out, max_blocks * block_size, block_size,
                                max_blocks, num_blocks, dtype, workspace, workspace_bytes};
  return window_run(x, window, sinks, stream);
}

int gqa_chunk_attn_prefix(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* cu_tokens, const int32_t* seq_lens, int b, int total,
                          int h, int g, int d_k, int d_v, float scale, int prefix_len, void* out,
                          int cap, int dtype, void* workspace, long long workspace_bytes,
                          void* stream) {
  PartCall x;
  static_cast<ChunkCall&>(x) = {q, k_cache, v_cache, cu_tokens, seq_lens, nullptr, b, total, h, g,
                                d_k, d_v, scale, out, cap, 0, 0, 0, dtype, workspace,
                                workspace_bytes};
  return prefix_run(x, prefix_len, stream);
}

int gqa_chunk_attn_prefix_paged(const void* q, const void* k_pool, const void* v_pool,
                                const int32_t* block_table, const int32_t* cu_tokens,
                                const int32_t* seq_lens, int b, int total, int h, int g, int d_k,
                                int d_v, float scale, int prefix_len, void* out, int block_size,
                                int max_blocks, int num_blocks, int dtype, void* workspace,
                                long long workspace_bytes, void* stream) {
  if (int e = paged_args_check(block_table, g, block_size, max_blocks, num_blocks)) return e;
  PartCall x;
  static_cast<ChunkCall&>(x) = {q, k_pool, v_pool, cu_tokens, seq_lens, block_table, b, total, h, g,
                                d_k, d_v, scale, out, max_blocks * block_size, block_size,
                                max_blocks, num_blocks, dtype, workspace, workspace_bytes};
  return prefix_run(x, prefix_len, stream);
}

int gqa_chunk_attn_prefix_workspace(int b, int total, int h, int g, int d_k, int d_v, int num_sms,
                                    long long* bytes) {
  if (!bytes) return GQA_ERR_NULL;
  if (num_sms < 0 || b < 1) return GQA_ERR_SHAPE;
  if (int e = chunk_shape_check(total, h, g, d_k, d_v)) return e;
  if (b > 65535) return GQA_ERR_UNSUPPORTED;
  if (num_sms == 0) {
    unsigned int* status = nullptr;
    if (int e = device_query(&num_sms, &status)) return e;
  }
  const int rows = group_rows(b, total, kM / (h / g), 1);
  *bytes = static_cast<long long>(part_plan(total, h, g, d_v, num_sms, rows).bytes);
  return GQA_OK;
}

}  // extern "C"
