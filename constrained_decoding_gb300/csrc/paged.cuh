// Device helpers of the 8-bit paged K/V cache and of rotary positions.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "paged.h"
#include "pcd_kernels.h"
#include "ptx.cuh"

namespace pcd {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// cos and sin of position p at F turns (2^-64) per position: p F wraps at
// whole turns, so the product is exact; its top 32 bits are the angle in
// (-1/2, 1/2] turns to 2^-32, under fp32's own rounding of it.
__device__ __forceinline__ void turn(int64_t p, int64_t F, float* c, float* s) {
  const uint64_t phase = static_cast<uint64_t>(p) * static_cast<uint64_t>(F);
  sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f /* 2^-31: half turns */, s, c);
}

// Attributes of a kernel, set once a device (a static of its launcher): its
// dynamic shared memory, and an SM split all for shared memory.  An SM that
// last ran a kernel without shared memory keeps its split while CTAs are on
// it, and would hold fewer of these than fit.
struct KernelSetup {
  std::atomic<uint64_t> done{0};
  template <class Kern>
  cudaError_t run(Kern kern, int smem) {
    int dev = 0;
    cudaError_t r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    if (smem > 0) r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (r == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return r;
  }
};

// ------------------------------------------------------------------ sequences
constexpr int kMaxLen = 0x7ffffc00;  // tokens of a sequence: positions and their roundings stay in 32 bits
struct SeqItem {
  int seq, local, row0, n, len;  // sequence (-1: none), item within it, its first row, its rows, its cached tokens
};
// The sequence of work item `idx` when sequence s owns the items
// [f(s), f(s + 1)), f(s) = (q_off[s] * mul >> shift) + add * s: a bound on its
// tiles that needs no prefix sum.  A warp narrows 32 ways at a time; lanes
// fetch all that a sequence has at once, so up to 32 sequences cost one trip
// to memory.  (As unsigned, so that a negative offset stands behind every item.)
__device__ __forceinline__ SeqItem find_item(const SeqView& q, int idx, int mul, int shift, int add) {
  const int lane = threadIdx.x & 31;
  auto f = [&](int off, int s) {
    return (static_cast<unsigned>(off) * static_cast<unsigned>(mul) >> shift) + static_cast<unsigned>(add * s);
  };
  int lo = 0, hi = q.n_seq;
  while (true) {
    const int step = (hi - lo + 31) >> 5;
    const int s = lo + lane * step;
    int off = 0, end = 0, len = 0;
    if (s < hi) {
      off = q.q_off[s];
      if (step == 1) {
        end = q.q_off[s + 1];
        len = q.kv_len[s];
      }
    }
    const unsigned b = __ballot_sync(0xffffffffu, s < hi && f(off, s) <= static_cast<unsigned>(idx));
    if (b == 0) return SeqItem{-1, 0, 0, 0, 0};
    const int l = 31 - __clz(b);
    if (step == 1) {
      SeqItem it;
      it.seq = lo + l;
      it.row0 = __shfl_sync(0xffffffffu, off, l);
      it.n = static_cast<int>(static_cast<unsigned>(__shfl_sync(0xffffffffu, end, l)) - static_cast<unsigned>(it.row0));
      it.len = __shfl_sync(0xffffffffu, len, l);
      it.local = static_cast<int>(static_cast<unsigned>(idx) - f(it.row0, it.seq));
      return it;
    }
    lo += l * step;
    hi = min(hi, lo + step);
  }
}
// The sequence of row `tok`; none (seq -1) for rows of no sequence and of those
// whose offsets are bad, which every kernel skips.
__device__ __forceinline__ SeqItem find_row(const SeqView& q, int tok) {
  SeqItem it = find_item(q, tok, 1, 0, 0);
  if (it.seq >= 0 && (it.row0 < 0 || it.n <= it.local || it.n > q.n_tok - it.row0)) it.seq = -1;
  return it;
}
// The offsets of sequence blockIdx.x, checked by one thread of the grid (every
// grid of items has a CTA for each sequence): where offsets decrease, find_item
// may lead no CTA to the sequence that has them.  Constructed before find_item,
// so that the loads go out together.
struct OffsetCheck {
  int lo = 0, hi = 0;
  __device__ __forceinline__ explicit OffsetCheck(const SeqView& q) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && blockIdx.x < static_cast<unsigned>(q.n_seq)) {
      lo = q.q_off[blockIdx.x];
      hi = q.q_off[blockIdx.x + 1];
    }
  }
  __device__ __forceinline__ void report(const SeqView& q, int* err) const {
    if (lo != hi && (lo < 0 || hi < lo || hi > q.n_tok)) record_error(err, DEV_BAD_INDEX);
  }
};

// ---------------------------------------------------------------------- codes
constexpr float kScaleFloor = 8.673617379884035e-19f;  // 2^-60: a block of zeros has this scale

// Scale of a block whose new rows reach |x| = am, beside `old` when older
// tokens stay in it.  e4m3 scales are powers of two, so a grown scale moves
// the older codes by whole exponents (exact while they stay normal).  A NaN
// or infinity makes the scale so, and everything read from the block NaN.
__device__ __forceinline__ float block_scale(float am, float old, bool held, int format) {
  float need;
  if (format == PCD_KV_INT8) {
    need = am * (1.f / 127.f);
  } else {
    need = am * (1.f / 448.f);
    if (isfinite(need)) need = __uint_as_float((__float_as_uint(need) + 0x7fffffu) & 0xff800000u);
  }
  if (need < kScaleFloor) need = kScaleFloor;
  if (held && (old != old || need <= old)) return old;
  return need;
}
__device__ __forceinline__ uint8_t encode(float x, int format) {
  if (x != x) return 0;  // the scale says so: no code is a NaN
  if (format == PCD_KV_INT8) return static_cast<uint8_t>(static_cast<int8_t>(max(-127, min(127, __float2int_rn(x)))));
  return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float decode(uint8_t q, int format) {
  if (format == PCD_KV_INT8) return static_cast<float>(static_cast<int8_t>(q));
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(q, __NV_E4M3)));
}

// Eight values as they are stored, and in fp32.
template <class T>
struct alignas(16) Eight {
  T v[8];
};
template <class T>
__device__ __forceinline__ void load8(const T* p, Eight<T>* e) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(p)[i];
}
// Their codes at a finite scale (so no value is a NaN or beyond the largest
// code).  int8: the product rounded to an integer by adding 1.5 2^23, whose low
// byte then is the code.
__device__ __forceinline__ uint2 encode8(const float* v, float inv, int format) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v[4 * j + i] * inv;
    if (format == PCD_KV_INT8) {
      uint32_t n[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = __float_as_uint(__fadd_rn(x[i], 12582912.f));
      w[j] = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
    } else {
      w[j] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3)) |
             static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3)) << 16;
    }
  }
  return make_uint2(w[0], w[1]);
}
// The larger magnitude; a NaN wins.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// Codes as fp16, exactly.  e4m3 by the conversion instruction (64 lanes a
// clock on an SM, four times what masks and shifts reach); int8 with the sign
// bit flipped as the low mantissa bits of 1024, minus 1152.
__device__ __forceinline__ uint32_t e4m3x2_half(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t int8_half(uint32_t x) {
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Codes 0, 1 and 2, 3 of a word.
template <int FMT>
__device__ __forceinline__ void codes4_half(uint32_t w, uint32_t* h0, uint32_t* h1) {
  if constexpr (FMT == PCD_KV_E4M3) {
    *h0 = e4m3x2_half(w);
    *h1 = e4m3x2_half(w >> 16);
  } else {
    w ^= 0x80808080u;
    *h0 = int8_half(__byte_perm(w, 0x64646464u, 0x4140));
    *h1 = int8_half(__byte_perm(w, 0x64646464u, 0x4342));
  }
}
// Codes 2b, 2b + 1 of two words, paired across the words.
template <int FMT>
__device__ __forceinline__ void codes_cross_half(uint32_t w0, uint32_t w1, int b, uint32_t* h0, uint32_t* h1) {
  codes4_half<FMT>(__byte_perm(w0, w1, b ? 0x7362 : 0x5140), h0, h1);
}

// ----------------------------------------------------------------------- rows
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// bf16 queries enter the fp16 products scaled by a power of two that takes the
// row's largest |q| (bits am) to [2^14, 2^15): exact down to 2^-29 of it.
// Returns the factor to undo it.
template <class T>
__device__ __forceinline__ float row_power(uint32_t am, float* down) {
  int e = static_cast<int>(am >> 23);
  if (std::is_same<T, __half>::value || e == 0 || e == 255) {
    *down = 1.f;
    return 1.f;
  }
  e = max(1, min(253, 127 + 14 + 127 - e));
  *down = __uint_as_float(static_cast<uint32_t>(e) << 23);
  return __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
}

constexpr float kBias = 8.f;  // weights are exp2(x - M + kBias)

// Partial softmax states of a row joined: reference M, sum L, 4 channels of O.
struct RowState {
  float M = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void top(float2 ml) {
    if (ml.y != 0.f) M = fmaxf(M, ml.x);
  }
  __device__ __forceinline__ void add(float2 ml, float4 v) {
    if (ml.y == 0.f) return;
    const float w = ex2_approx(ml.x - M);
    L = fmaf(w, ml.y, L);
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
};
// Writes 4 channels of an output row, and its log-sum-exp.
template <class T>
__device__ __forceinline__ void finish_row(const PagedAttnArgs& a, const RowState& st, int tok, int hq, int d) {
  const float il = st.L == 0.f ? 0.f : 1.f / st.L;
  T* out = static_cast<T*>(a.out) + tok * a.out_tok + hq * a.out_head + d;
  out[0] = from_f<T>(st.o.x * il);
  out[1] = from_f<T>(st.o.y * il);
  out[2] = from_f<T>(st.o.z * il);
  out[3] = from_f<T>(st.o.w * il);
  if (a.lse && d == 0)
    a.lse[static_cast<int64_t>(tok) * a.Hq + hq] =
        st.L == 0.f ? -INFINITY : (st.M - kBias + log2f(st.L)) * 0.6931471805599453f;
}

}  // namespace pcd
