// chunk_part.cu - attention of packed chunks over a part of the cache (a sliding
// window and the first positions) and over a prefix that the batch shares: the
// kernel of chunk_kernel.cuh with another split of work.
//
// Window.  A token at position P sees p <= P with p > P - window or p < sinks.
// A unit of ntok tokens reads the span (part_device.cuh) of ceil(sinks / 64) *
// 64 + window + ntok - 1 positions at most, not the P + 1 of the causal form;
// its first and last tiles are masked row by row, the others are seen whole.
//
// Prefix.  Positions below prefix_len are the same rows for every sequence.
// Where sequences bring few tokens, the prefix is attended by units of its own
// over the packed rows of all sequences (2 tq tokens to a unit, so 64 single
// tokens of eight heads read it twice instead of 64 times), each sequence's
// own positions by units as ever, and every row is joined from both: partial
// results of units that no run's end cuts lie by row, the others by CTA.  With
// units that one sequence fills the prefix is the head of the unit's span: the
// tiles read are the same and nothing has to be joined.
#include "chunk_kernel.cuh"
#include "part_device.cuh"

namespace gqa {
namespace {

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
    if (twin(tq)) return (lt1 - lt0 + 1 - side) >> 1;
    const int nt = min(ntok - side * tq, tq);
    const int ext = of_head ? head : pos0 + side * tq + nt - shift;
    return max(0, min(lt1, (ext + kN - 1) / kN) - lt0);
  }
  // what every token at positions first .. last sees
  __device__ PartVisible visible(const ChunkParams& p, int first, int last) const {
    if (of_head) return {head, 0, 0};
    PartVisible v;
    v.hi = first + 1 - shift;
    v.lo = max(last - p.window + 1, p.base_min) - shift;
    v.head = min(head, v.hi);
    if (v.lo <= v.head) v.lo = 0;
    return v;
  }
};

// The run of work of one CTA, as in chunk_attn.cu.  A sequence's units grow with
// the position of their last token until the window is full and are alike from
// there on, so sums of their work are an arithmetic progression and a multiple.
// Units of the head come before those of the sequences, as sequence -1.
constexpr int kPartUnitCost = 320;

struct PartWalk {
  using Seg = PartSeg;
  using Visible = PartVisible;
  static constexpr bool kPart = true;

  const int *cu, *lens;
  int b, g, tq, total;
  long long cap;
  int window, head, head_seq, base_min, gran;
  bool grouped, paged;
  int heads_n;            // tokens of the head's units
  long long head_f;       // their work, of one KV head
  ChunkPos at, end;
  int t0, n, L;  // of sequence at.i
  bool more;
  int c_t0, c_n, c_L;     // as in chunk_attn.cu
  long long c_f, c_incl;

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
  // tokens that the head's units hold
  __device__ static int head_tokens(const ChunkParams& p) {
    return p.grouped ? min(max(__ldg(p.cu + p.b), 0), p.total) : 0;
  }
  template <typename T16, int DV>
  static cudaError_t join(cudaLaunchConfig_t& cfg, const ChunkParams& p, int num_sms);

  __device__ bool seq(int k, int& a0, int& nn, int& Lk) const {
    a0 = nn = Lk = 0;
    if (k >= b) return false;
    a0 = __ldg(cu + k);
    const int a1 = __ldg(cu + k + 1);
    Lk = __ldg(lens + k);
    if (errors(a0, a1, Lk, total, cap, base_min)) return false;
    nn = a1 - a0;
    return nn > 0;
  }
  __device__ int units(int nn) const { return (nn + 2 * tq - 1) / (2 * tq); }
  __device__ bool last_twin(int nn, int nu) const { return nn - (nu - 1) * 2 * tq <= tq; }

  // A unit q has min(A + (q + 1) * 2 tq, B) positions.
  struct Shape {
    long long A, B;
    int q0;  // units before the window is full
  };
  __device__ Shape shape(bool of_head, int nn, int Lk) const {
    Shape s;
    const int hp = grouped ? 0 : (head + gran - 1) & ~(gran - 1);
    if (of_head) {
      s.A = s.B = head;
    } else {
      s.A = static_cast<long long>(Lk) - nn - base_min + (head_seq >= 0 ? hp : 0);
      s.B = static_cast<long long>(window) + 2 * tq + hp;
      if (head_seq >= 0) s.B = 1ll << 40;
    }
    s.q0 = s.B <= s.A ? 0
                      : static_cast<int>(min(static_cast<long long>(units(nn)),
                                             div_pos(s.B - s.A, 2 * tq)));
    return s;
  }
  __device__ long long prefix(long long q, const Shape& s) const {
    const long long k = min(q, static_cast<long long>(s.q0));
    return k * (s.A + kPartUnitCost) + tq * (k * (k + 1)) + (q - k) * (s.B + kPartUnitCost);
  }
  __device__ long long work(bool of_head, int nn, int Lk) const {
    const int nu = units(nn);
    const Shape s = shape(of_head, nn, Lk);
    if (!last_twin(nn, nu)) return prefix(nu, s);
    const long long before = prefix(nu - 1, s);
    return before + ((3 * (prefix(nu, s) - before - kPartUnitCost)) >> 2) + kPartUnitCost;
  }

  // the span and the tiles of unit q of a sequence (of the head)
  __device__ void span(Seg& s, bool of_head, int q, int nn, int Lk) const {
    s.of_head = of_head;
    s.pos0 = Lk - nn + q * 2 * tq;
    s.ntok = min(nn - q * 2 * tq, 2 * tq);
    s.L = Lk;
    s.head = grouped && !of_head ? 0 : head;
    int hi;
    if (of_head) {
      s.shift = 0;
      s.sb = (head + gran - 1) & ~(gran - 1);
      s.z = s.end = hi = head;
    } else {
      const int lo = max(base_min, s.pos0 - window + 1);
      const int lo_all = max(base_min, Lk - nn - window + 1);
      const PartSpan t = part_span(lo, lo_all, s.head, gran, paged, head_seq >= 0 || grouped);
      s.shift = t.shift;
      s.sb = t.sb;
      s.z = t.z;
      s.end = Lk - t.shift;
      hi = s.pos0 + s.ntok - t.shift;
    }
    s.ti = (hi + kN - 1) / kN;
  }
  __device__ int tiles(bool of_head, int q, int nn, int Lk) const {
    Seg s;
    span(s, of_head, q, nn, Lk);
    return s.ti;
  }

  __device__ void scan(int base, int& a0, int& nn, int& Lk, long long& f, long long& incl) const {
    f = seq(base + (threadIdx.x & 31), a0, nn, Lk) ? work(false, nn, Lk) : 0;
    incl = f;
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if ((threadIdx.x & 31) >= o) incl += y;
    }
  }

  // the place `off` of the work of sequence i (t0, n, L set), fs for a KV head
  __device__ ChunkPos place(int i, long long off, long long fs, int near) const {
    ChunkPos r;
    r.i = i;
    r.j = static_cast<int>(div_pos(off, fs));
    const long long rem = off - r.j * fs;
    const int nu = units(n);
    const Shape s = shape(i < 0, n, L);
    // the last unit q with prefix(q) <= rem: the root of the quadratic, or a
    // division behind it, put right by steps of one
    const long long full = prefix(s.q0, s);
    int q;
    if (rem < full) {
      const float c1 = static_cast<float>(s.A) + (kPartUnitCost + tq);
      const float rf = static_cast<float>(rem);
      q = static_cast<int>(2.f * rf / (sqrtf(c1 * c1 + 4.f * tq * rf) + c1));
    } else {
      q = s.q0 + static_cast<int>(min(div_pos(rem - full, s.B + kPartUnitCost),
                                      static_cast<long long>(nu)));
    }
    q = min(max(q, 0), nu - 1);
    while (q > 0 && prefix(q, s) > rem) --q;
    while (q + 1 < nu && prefix(q + 1, s) <= rem) ++q;
    r.qt = q;
    const int ti = tiles(i < 0, q, n, L);
    const bool tw = q == nu - 1 && last_twin(n, nu);
    const long long in = rem - prefix(q, s);
    const int lt = static_cast<int>((tw ? (in + in / 3) : in) >> 7);
    r.lt = lt <= near ? 0 : lt >= ti - near ? ti : lt;
    return r;
  }

  __device__ ChunkPos locate(long long x, int near) {
    if (x < head_f * g) {
      t0 = 0;
      n = heads_n;
      L = head;
      return place(-1, x, head_f, near);
    }
    long long carry = head_f;
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
        return place(base + src, off, __shfl_sync(0xffffffffu, f, src), near);
      }
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    return {b, 0, 0, 0};  // not reached for x < W
  }

  __device__ bool start(const ChunkParams& p, int c, int nc, ChunkPos& r) {
    cu = p.cu;
    lens = p.lens;
    b = p.b;
    g = p.g;
    tq = p.tq;
    total = p.total;
    cap = p.cap;
    window = p.window;
    head = p.head;
    head_seq = p.head_seq;
    base_min = p.base_min;
    grouped = p.grouped;
    paged = p.table != nullptr;
    gran = paged ? min(p.bsz, kGrain) : kGrain;
    heads_n = head_tokens(p);
    head_f = heads_n > 0 ? work(true, heads_n, head) : 0;
    scan(0, c_t0, c_n, c_L, c_f, c_incl);
    long long W = head_f + __shfl_sync(0xffffffffu, c_incl, 31);
    for (int base = 32; base < b; base += 32) {
      int a0, nn, Lk;
      long long f, incl;
      scan(base, a0, nn, Lk, f, incl);
      W += __shfl_sync(0xffffffffu, incl, 31);
    }
    W *= g;
    r = {b, 0, 0, 0};
    nc = static_cast<int>(min(static_cast<long long>(nc), W / (2 * kN) + 1));
    if (W == 0 || c > nc) return false;
    if (c == nc) return true;
    const long long run = div_pos(W, nc);
    const int near = static_cast<int>(run / (32 * kN));
    const int left = static_cast<int>(W - run * nc);
    r = locate(run * c + min(c, left), near);
    if (c == 0) r.lt = 0;
    return true;
  }

  __device__ void begin(const ChunkPos& from, const ChunkPos& e) {
    at = from;
    end = e;
    more = at.i < b;
    if (more && at.lt >= tiles(at.i < 0, at.qt, n, L)) advance();
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

  __device__ bool next(Seg& s) {
    if (!more || at.i >= b) return false;
    const bool last = at.i == end.i && at.j == end.j && at.qt == end.qt;
    const bool past = at.i > end.i || (at.i == end.i && (at.j > end.j ||
                                       (at.j == end.j && at.qt > end.qt)));
    if (past || (last && end.lt <= at.lt)) return false;
    span(s, at.i < 0, at.qt, n, L);
    s.i = max(at.i, 0);
    s.j = at.j;
    s.t0 = t0 + at.qt * 2 * tq;
    s.lt0 = at.lt;
    s.lt1 = last ? end.lt : s.ti;
    if (last)
      more = false;
    else
      advance();
    return true;
  }
};

// Joins, for every row, the partial results over the head and over the
// sequence's own positions, each whole (by row) or in pieces (by CTA).  A warp
// takes two query heads of a token's group, four pieces of both with their
// loads side by side.
constexpr int kGroupThreads = 256;

template <typename T16, int DV>
__global__ void __launch_bounds__(kGroupThreads) group_join_kernel(const ChunkParams p, int nc) {
  constexpr int CPL = DV / 32;
  constexpr int NP = 4;
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const int pairs = (p.r + 1) >> 1;
  const long long id =
      static_cast<long long>(blockIdx.x) * (kGroupThreads / 32) + (threadIdx.x >> 5);
  const long long tj = id / pairs;
  const int a_first = 2 * static_cast<int>(id - tj * pairs);
  const int t = static_cast<int>(tj / p.g), j = static_cast<int>(tj - static_cast<long long>(t) * p.g);
  const int T = PartWalk::head_tokens(p);
  if (t >= T) return;  // (uniform across the warp, as all below)
  const int i = packed_sequence(p.cu, p.b, t);
  if (i >= p.b) return;
  const int a0 = __ldg(p.cu + i), a1 = __ldg(p.cu + i + 1);
  if (t < a0 || t >= a1 || PartWalk::errors(a0, a1, __ldg(p.lens + i), p.total, p.cap, p.base_min))
    return;
  // the units that hold the token: over the head, over its own positions
  const int w = 2 * p.tq;
  const int u0[2] = {t / w * w, a0 + (t - a0) / w * w};
  int first[2], cnt[2], row0[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const size_t units = static_cast<size_t>(p.total) * p.g;
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
            by_row ? (own ? static_cast<size_t>(p.total) * p.h : 0) + orow + a
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

template <typename T16, int DV>
cudaError_t PartWalk::join(cudaLaunchConfig_t& cfg, const ChunkParams& p, int num_sms) {
  if (!p.grouped) return launch_join<T16, DV>(cfg, p, num_sms);
  const long long warps = static_cast<long long>(p.total) * p.g * ((p.r + 1) / 2);
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kGroupThreads / 32 - 1) / (kGroupThreads / 32)));
  cfg.blockDim = dim3(kGroupThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, group_join_kernel<T16, DV>, p, num_sms);
}

// Are the prefix's units to be shared by the sequences?  (tq: tokens of a side)
bool prefix_grouped(int b, int total, int tq) {
  return b > 1 && total < static_cast<long long>(b) * tq;
}

int part_run(const ChunkCall& x, void* stream) {
  if (int e = chunk_check(x)) return e;
  if (x.cap > 0x7FFFFF00) return GQA_ERR_SHAPE;  // (indices of a span stay within 31 bits)
  int num_sms = 0;
  unsigned int* status = nullptr;
  if (int e = device_query(&num_sms, &status)) return e;
  const ChunkPlan pl = chunk_plan(x.total, x.h, x.g, x.dv, num_sms, x.grouped);
  if (x.ws_bytes < static_cast<long long>(pl.bytes)) return GQA_ERR_SCRATCH_LIMIT;
  if (x.total == 0) return GQA_OK;
  const cudaError_t e =
      launch_chunk_types<PartWalk>(x, pl, num_sms, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

// (cap: positions that the cache can hold)
int window_run(ChunkCall& x, int window, int sinks, void* stream) {
  if (window < 1 || sinks < 0) return GQA_ERR_SHAPE;
  x.window = window;
  x.head = std::min(sinks, std::max(x.cap, 0));
  return part_run(x, stream);
}

int prefix_run(ChunkCall& x, int prefix_len, void* stream) {
  if (prefix_len < 0 || (x.cap >= 1 && prefix_len > x.cap)) return GQA_ERR_SHAPE;
  x.window = 0x7FFFFFFF;
  x.head = x.base_min = prefix_len;
  x.head_seq = 0;
  if (x.g > 0 && x.h > 0 && x.h / x.g >= 1 && x.h / x.g <= kM)
    x.grouped = prefix_len > 0 && prefix_grouped(x.b, x.total, kM / (x.h / x.g));
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
  ChunkCall x = {q, k_cache, v_cache, cu_tokens, seq_lens, nullptr, b, total, h, g, d_k,
                 d_v, scale, out, cap, 0, 0, 0, dtype, workspace, workspace_bytes};
  return window_run(x, window, sinks, stream);
}

int gqa_chunk_attn_window_paged(const void* q, const void* k_pool, const void* v_pool,
                                const int32_t* block_table, const int32_t* cu_tokens,
                                const int32_t* seq_lens, int b, int total, int h, int g, int d_k,
                                int d_v, float scale, int window, int sinks, void* out,
                                int block_size, int max_blocks, int num_blocks, int dtype,
                                void* workspace, long long workspace_bytes, void* stream) {
  if (int e = paged_args_check(block_table, g, block_size, max_blocks, num_blocks)) return e;
  ChunkCall x = {q, k_pool, v_pool, cu_tokens, seq_lens, block_table, b, total, h, g, d_k,
                 d_v, scale, out, max_blocks * block_size, block_size, max_blocks,
                 num_blocks, dtype, workspace, workspace_bytes};
  return window_run(x, window, sinks, stream);
}

int gqa_chunk_attn_prefix(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* cu_tokens, const int32_t* seq_lens, int b, int total,
                          int h, int g, int d_k, int d_v, float scale, int prefix_len, void* out,
                          int cap, int dtype, void* workspace, long long workspace_bytes,
                          void* stream) {
  ChunkCall x = {q, k_cache, v_cache, cu_tokens, seq_lens, nullptr, b, total, h, g, d_k,
                 d_v, scale, out, cap, 0, 0, 0, dtype, workspace, workspace_bytes};
  return prefix_run(x, prefix_len, stream);
}

int gqa_chunk_attn_prefix_paged(const void* q, const void* k_pool, const void* v_pool,
                                const int32_t* block_table, const int32_t* cu_tokens,
                                const int32_t* seq_lens, int b, int total, int h, int g, int d_k,
                                int d_v, float scale, int prefix_len, void* out, int block_size,
                                int max_blocks, int num_blocks, int dtype, void* workspace,
                                long long workspace_bytes, void* stream) {
  if (int e = paged_args_check(block_table, g, block_size, max_blocks, num_blocks)) return e;
  ChunkCall x = {q, k_pool, v_pool, cu_tokens, seq_lens, block_table, b, total, h, g, d_k,
                 d_v, scale, out, max_blocks * block_size, block_size, max_blocks,
                 num_blocks, dtype, workspace, workspace_bytes};
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
  // (of any number of rows up to `total`: the most that are still grouped)
  const int tq = kM / (h / g);
  const long long most = std::min<long long>(total, static_cast<long long>(b) * tq - 1);
  size_t n = chunk_plan(total, h, g, d_v, num_sms).bytes;
  if (prefix_grouped(b, static_cast<int>(most), tq))
    n = std::max(n, chunk_plan(static_cast<int>(most), h, g, d_v, num_sms, true).bytes);
  *bytes = static_cast<long long>(n);
  return GQA_OK;
}

}  // extern "C"
