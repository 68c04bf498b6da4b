// chunk_attn.cu - causal attention of packed chunks of new tokens over the whole
// cache: the kernel of chunk_kernel.cuh with the split of its causal work.
#include "chunk_kernel.cuh"

namespace gqa {
namespace {

struct ChunkSeg {
  int i, j;        // sequence, KV head
  int t0;          // packed row of the unit's first token
  int pos0;        // its position
  int ntok;        // tokens of the unit
  int L, end;      // (the same: no row behind it is used)
  int lt0, lt1;    // tiles of the unit taken here
  int ti;          // tiles of the unit
  static constexpr int head = 0, z = 0;
  // A unit whose rows fit side A alone runs as twins: both sides hold the same
  // rows and take the tiles by turns, and their results are joined at the end.
  __device__ bool twin(int tq) const { return ntok <= tq; }
  // tiles that a side of two works on of [lt0, lt1)
  __device__ int side_tiles(int side, int tq) const {
    const int nt = min(ntok - side * tq, tq);
    const int ext = pos0 + side * tq + nt;
    return max(0, min(lt1, (ext + kN - 1) / kN) - lt0);
  }
  // what the tokens from tok0 on see
  __device__ void sees(const ChunkParams&, int tok0, SegPlan::Side& v, int& lo_min) const {
    v.lo = lo_min = 0;
    v.hi = v.all_hi = pos0 + tok0 + 1;
    v.all_head = v.all_lo = 0;
  }
};

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
  using Seg = ChunkSeg;
  static constexpr bool kPart = false;
  __device__ static void report(const ChunkParams& p) {
    report_bad_packed(p.cu, p.lens, p.b, p.total, p.cap, p.status);
  }
  template <typename T16, int DV>
  static cudaError_t join(cudaLaunchConfig_t& cfg, const ChunkParams& p, int num_sms) {
    return launch_join<T16, DV>(cfg, p, num_sms);
  }

  const ChunkParams& p;
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

  __device__ explicit ChunkWalk(const ChunkParams& params) : p(params) {}

  // Run c's start: false when the launch has fewer runs than that (c = their
  // number: the end of the last one, behind every sequence).
  __device__ bool start(int c, int nc, ChunkPos& r) {
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
    s.L = s.end = L;
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

int chunk_run(const ChunkCall& x, void* stream) {
  if (int e = chunk_check(x)) return e;
  int num_sms = 0;
  unsigned int* status = nullptr;
  if (int e = device_query(&num_sms, &status)) return e;
  const ChunkPlan pl = chunk_plan(x.total, x.h, x.g, x.dv, num_sms);
  if (x.ws_bytes < static_cast<long long>(pl.bytes)) return GQA_ERR_SCRATCH_LIMIT;
  if (x.total == 0) return GQA_OK;
  const cudaError_t e =
      launch_chunk_types<ChunkWalk>(x, pl, num_sms, status, static_cast<cudaStream_t>(stream));
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
