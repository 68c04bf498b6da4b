// serve_device.cuh - device-side helpers of the kernels around the decode
// step (rotation and append, 8-bit cache, chunk attention): packed tokens,
// row pieces, the e4m3 conversions, wide tensor-memory accesses.
#pragma once

#include <cuda_fp8.h>

#include "gqa_device.cuh"

namespace gqa {

// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// 16 bytes global -> shared without passing registers; the arrival of all of
// this thread's earlier ones on an mbarrier (one of its count); their end
__device__ __forceinline__ void async_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void async_copies_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------------------
// packed tokens: sequence i's new tokens are rows cu[i] .. cu[i + 1] - 1
// ---------------------------------------------------------------------------

// Number of the b entries cu[1 .. b] that are at or below t, i.e. the
// sequence holding packed row t (b when t lies behind the last sequence).
// Warp-cooperative, two rounds of loads for b up to 1024.
__device__ __forceinline__ int packed_sequence(const int* cu, int b, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, cnt = b;
  while (cnt > 32) {
    const int step = (cnt + 31) >> 5;
    const int k = (lane + 1) * step - 1;
    const bool le = k < cnt && __ldg(cu + 1 + lo + k) <= t;
    const int m = __popc(__ballot_sync(0xffffffffu, le));
    lo += m * step;
    cnt = min(step, cnt - m * step);
  }
  const bool le = lane < cnt && __ldg(cu + 1 + lo + lane) <= t;
  return lo + __popc(__ballot_sync(0xffffffffu, le));
}

// Are sequence i's packed rows and length usable?  0 <= cu[i] <= cu[i + 1] <=
// total, and either no new token or n <= L <= cap.
__device__ __forceinline__ unsigned packed_errors(int t0, int t1, int L, int total,
                                                  long long cap) {
  if (t0 < 0 || t1 < t0 || t1 > total) return GQA_DEV_BAD_TOKENS;
  if (t1 > t0 && (L < t1 - t0 || L > cap)) return GQA_DEV_BAD_SEQ_LEN;
  return 0u;
}

// Warp-cooperative: flag every unusable sequence.
__device__ __forceinline__ void report_bad_packed(const int* cu, const int* lens, int b, int total,
                                                  long long cap, unsigned int* status) {
  unsigned bad = 0;
  for (int i = threadIdx.x & 31; i < b; i += 32)
    bad |= packed_errors(__ldg(cu + i), __ldg(cu + i + 1), __ldg(lens + i), total, cap);
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (bad && (threadIdx.x & 31) == 0) atomicOr(status, bad);
}

// ---------------------------------------------------------------------------
// four consecutive elements of a row (8 bytes of a 16-bit type, 16 of fp32)
// ---------------------------------------------------------------------------
template <typename T>
struct Piece4 {
  uint2 raw;
  __device__ void load(const T* p) { raw = __ldg(reinterpret_cast<const uint2*>(p)); }
  // (of memory that this kernel writes)
  __device__ void load_own(const T* p) { raw = *reinterpret_cast<const uint2*>(p); }
  __device__ void zero() { raw = make_uint2(0u, 0u); }
  __device__ void get(float* x) const {
    const uint32_t w[2] = {raw.x, raw.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (Half16<T>::kBf16) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
    }
  }
  __device__ static void store(T* p, const float* x) {
    *reinterpret_cast<uint2*>(p) =
        make_uint2(Half16<T>::pack2(x[0], x[1]), Half16<T>::pack2(x[2], x[3]));
  }
  __device__ void copy_to(T* p) const { *reinterpret_cast<uint2*>(p) = raw; }
};

template <>
struct Piece4<float> {
  float4 raw;
  __device__ void load(const float* p) { raw = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ void load_own(const float* p) { raw = *reinterpret_cast<const float4*>(p); }
  __device__ void zero() { raw = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void get(float* x) const { x[0] = raw.x, x[1] = raw.y, x[2] = raw.z, x[3] = raw.w; }
  __device__ static void store(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
  __device__ void copy_to(float* p) const { *reinterpret_cast<float4*>(p) = raw; }
};

// eight fp32 values as consecutive elements of T
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  Piece4<float>::store(p, x);
  Piece4<float>::store(p + 4, x + 4);
}
template <typename T16>
__device__ __forceinline__ void store8(T16* p, const float (&x)[8]) {
  uint4 v;
  v.x = Half16<T16>::pack2(x[0], x[1]);
  v.y = Half16<T16>::pack2(x[2], x[3]);
  v.z = Half16<T16>::pack2(x[4], x[5]);
  v.w = Half16<T16>::pack2(x[6], x[7]);
  *reinterpret_cast<uint4*>(p) = v;
}

// ---------------------------------------------------------------------------
// e4m3
// ---------------------------------------------------------------------------
constexpr float kE4m3Max = 448.f;

// two fp32 values to two e4m3 bytes (x in the low byte), nearest even,
// saturating
__device__ __forceinline__ uint32_t e4m3_pack2(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t e4m3_pack4(float x, float y, float z, float w) {
  return e4m3_pack2(x, y) | (e4m3_pack2(z, w) << 16);
}

// two e4m3 bytes to fp32 (exact)
__device__ __forceinline__ float2 e4m3_unpack2(uint32_t v) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v & 0xFFFFu), __NV_E4M3);
  return __half22float2(__half2(h));
}

// ---------------------------------------------------------------------------
// tensor memory, 32 lanes x 32 consecutive 32-bit columns: thread t of the
// warp holds lane (base lane + t), columns [col, col + 32)
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]),
        "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
      "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]),
        "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r[k]);
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
      "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T: the A operand's 16-bit elements lie two
// to a 32-bit column, lane = row
__device__ __forceinline__ void mma_16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ---------------------------------------------------------------------------
// fp32 arithmetic on pairs, and the largest of three
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// N x 32 bytes to consecutive addresses, as whole sectors (dst aligned to 32
// bytes) or in 16-byte pieces
template <int N>
__device__ __forceinline__ void store_sectors(void* dst, const uint32_t* v, bool sectors) {
  char* d = static_cast<char*>(dst);
  if (sectors) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d + 32 * k),
                   "r"(v[8 * k]), "r"(v[8 * k + 1]), "r"(v[8 * k + 2]), "r"(v[8 * k + 3]),
                   "r"(v[8 * k + 4]), "r"(v[8 * k + 5]), "r"(v[8 * k + 6]), "r"(v[8 * k + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int k = 0; k < 2 * N; ++k)
      *reinterpret_cast<uint4*>(d + 16 * k) =
          make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  }
}

}  // namespace gqa
