// Rotary positions, the append to an 8-bit paged K/V cache and the attention
// over it for few query rows.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.cuh"
#include "paged.h"
#include "pcd.h"
#include "pcd_kernels.h"
#include "warp_mma.cuh"

namespace pcd {
namespace {

// ======================================================================== rope
// y = R x per pair; the angle is p F mod 1 turn in 64-bit integers, so it is
// as exact at position 2^31 as at 1.  Bound by the bytes of x and y: a thread
// owns the same VEC channels (and their partners, rot / 2 further, in the half
// layout) of every hgs-th head of one token, so an angle's sine and cosine are
// computed once for all of them, and takes two heads' loads at a time (four cost
// registers and 4 us of 25 at 8192 tokens x 32 heads).  That call, fp16 heads of
// 128: 26.5 us, 5.1 TB/s; 64 tokens of 14 heads 2.5 us.
// VEC: the widest access that pointers, strides and the pair layout allow.
template <class T, int N>
struct alignas(sizeof(T) * N) Chunk {
  T v[N];
};
template <class T, int VEC, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(RopeKArgs a, unsigned units, unsigned rot_units, unsigned hgs,
                                                   unsigned total) {
  constexpr int kN = INTER && VEC == 1 ? 2 : VEC;   // channels of a chunk of the rotated part
  constexpr int kL = INTER && VEC == 1 ? 1 : VEC;   // channels of one access
  constexpr int kPairs = INTER ? kN / 2 : kN;
  constexpr int kHeads = 2;
  griddep_launch_dependents();
  griddep_wait();
  const unsigned idx = blockIdx.x * 256u + threadIdx.x;
  if (idx >= total) return;
  const unsigned u = idx % units, th = idx / units;
  const int hg = static_cast<int>(th % hgs), t = static_cast<int>(th / hgs);
  const T* x = static_cast<const T*>(a.x) + t * a.x_tok;
  T* y = static_cast<T*>(a.y) + t * a.y_tok;
  if (u >= rot_units) {  // a chunk that is copied
    const int d = a.rope.rot + static_cast<int>(u - rot_units) * VEC;
    for (int h = hg; h < a.heads; h += static_cast<int>(hgs))
      *reinterpret_cast<Chunk<T, VEC>*>(y + h * a.y_head + d) = *reinterpret_cast<const Chunk<T, VEC>*>(x + h * a.x_head + d);
    return;
  }
  const int pair = static_cast<int>(u) * kPairs;
  const int d = static_cast<int>(u) * kN, half = a.rope.rot / 2;
  const int64_t p = a.pos ? a.pos[t] : static_cast<int64_t>(a.base) + t;
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    turn(p, a.rope.freqs[pair + i], &c[i], &s[i]);
    c[i] *= a.rope.amp;
    s[i] *= a.rope.transpose ? -a.rope.amp : a.rope.amp;
  }
  using C = Chunk<T, kL>;
  for (int h0 = hg; h0 < a.heads; h0 += kHeads * static_cast<int>(hgs)) {
    C v[kHeads][INTER ? kN / kL : 2];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k * static_cast<int>(hgs);
      if (h >= a.heads) break;
      const T* r = x + h * a.x_head + d;
#pragma unroll
      for (int j = 0; j < (INTER ? kN / kL : 2); ++j) v[k][j] = *reinterpret_cast<const C*>(r + (INTER ? j * kL : j * half));
    }
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k * static_cast<int>(hgs);
      if (h >= a.heads) break;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        T& e0 = INTER ? v[k][2 * i / kL].v[2 * i % kL] : v[k][0].v[i];
        T& e1 = INTER ? v[k][(2 * i + 1) / kL].v[(2 * i + 1) % kL] : v[k][1].v[i];
        const float f0 = to_f(e0), f1 = to_f(e1);
        e0 = from_f<T>(f0 * c[i] - f1 * s[i]);
        e1 = from_f<T>(f1 * c[i] + f0 * s[i]);
      }
      T* r = y + h * a.y_head + d;
#pragma unroll
      for (int j = 0; j < (INTER ? kN / kL : 2); ++j) *reinterpret_cast<C*>(r + (INTER ? j * kL : j * half)) = v[k][j];
    }
  }
}

template <class T, int VEC>
int launch_rope_v(const RopeKArgs& a, int sms, cudaStream_t s) {
  const bool inter = a.rope.interleaved != 0;
  const int rot_units = inter ? a.rope.rot / std::max(VEC, 2) : a.rope.rot / 2 / VEC;
  // in place, the channels behind the rotated ones already stand where they belong
  const int units = rot_units + (a.x == a.y ? 0 : (a.dim - a.rope.rot) / VEC);
  if (units == 0) return 0;
  // as few head groups as fill the GPU's threads
  const int64_t per_group = static_cast<int64_t>(a.n_tok) * units;
  const int64_t fill = (static_cast<int64_t>(sms) * 2048 + per_group - 1) / per_group;
  const int64_t hgs = std::min<int64_t>(a.heads, std::max<int64_t>(1, fill));
  const int64_t total = per_group * hgs;
  if (total >= (int64_t{1} << 31)) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>((total + 255) / 256));
  auto kern = inter ? rope_kernel<T, VEC, true> : rope_kernel<T, VEC, false>;
  return launch_k(kern, grid, dim3(256), 0, s, a, static_cast<unsigned>(units), static_cast<unsigned>(rot_units),
                  static_cast<unsigned>(hgs), static_cast<unsigned>(total));
}

template <class T>
int launch_rope_t(const RopeKArgs& a, int sms, cudaStream_t s) {
  // every chunk starts at a multiple of these, in elements
  uint64_t m = static_cast<uint64_t>(a.dim) | static_cast<uint64_t>(a.rope.rot);
  m |= a.rope.interleaved ? 0 : static_cast<uint64_t>(a.rope.rot / 2);
  if (a.n_tok > 1) m |= static_cast<uint64_t>(a.x_tok) | static_cast<uint64_t>(a.y_tok);
  if (a.heads > 1) m |= static_cast<uint64_t>(a.x_head) | static_cast<uint64_t>(a.y_head);
  m |= (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y)) / sizeof(T);
  if (sizeof(T) == 2 && m % 8 == 0) return launch_rope_v<T, 16 / sizeof(T)>(a, sms, s);
  if (m % 4 == 0) return launch_rope_v<T, 4>(a, sms, s);
  if (m % 2 == 0) return launch_rope_v<T, 2>(a, sms, s);
  return launch_rope_v<T, 1>(a, sms, s);
}

}  // namespace

int launch_rope(const RopeKArgs& a, int sms, cudaStream_t s) {
  if (a.n_tok == 0 || a.heads == 0) return 0;
  switch (a.dtype) {
    case PCD_DTYPE_F32: return launch_rope_t<float>(a, sms, s);
    case PCD_DTYPE_BF16: return launch_rope_t<__nv_bfloat16>(a, sms, s);
    default: return launch_rope_t<__half>(a, sms, s);
  }
}

namespace {
// ====================================================================== append
// One CTA owns one (page, KV head) of K or of V that a sequence's new tokens
// touch: nothing else writes it, so the block's scale needs no atomics and
// comes out the same on every run.
//   amax over the new rows -> scale (grown, never shrunk, while older tokens
//   stay in the page) -> older codes rescaled if it grew -> new codes.
// One token each of 64 sequences takes 5 us, that chain; 14.4 k tokens of four fp16
// heads of 128 17 us (2.6 TB/s of rows read and codes written), 13 with the rows in
// L2, bound by what is in flight: 120 registers let two CTAs on an SM, each with
// one head's rows (16 KB) ahead, and the last of its CTAs start in a second wave.
// The block of a CTA: its new rows and where they go.
struct AppendBlock {
  int held, rows, row0, pos0;  // older tokens in the page; new rows, the first one's index and position
  uint8_t* dst;
  float* scale;
};
__device__ __forceinline__ bool append_block(const AppendArgs& a, bool is_v, int h, AppendBlock* b) {
  const int page = 1 << a.c.page_log2;
  // item -> (sequence, page of its new range)
  const OffsetCheck offsets(a.q);
  const SeqItem it = find_item(a.q, static_cast<int>(blockIdx.x), 1, a.c.page_log2, 2);
  offsets.report(a.q, a.err);
  if (it.seq < 0) return false;
  const int n = it.n, len = it.len;
  if (n == 0) return false;
  if (n < 0 || it.row0 < 0 || n > a.q.n_tok - it.row0 || len < n || len > kMaxLen ||
      len > static_cast<int64_t>(a.q.table_width) << a.c.page_log2) {
    if (threadIdx.x == 0) record_error(a.err, DEV_BAD_INDEX);
    return false;
  }
  if (it.local > (n >> a.c.page_log2) + 1) return false;
  const int start = len - n;
  const int pg = (start >> a.c.page_log2) + it.local;
  const int lo = max(pg << a.c.page_log2, start), hi = min((pg + 1) << a.c.page_log2, len);
  if (lo >= hi) return false;
  const int id = a.q.table[static_cast<int64_t>(it.seq) * a.q.table_stride + pg];
  if (id < 0 || id >= a.c.n_pages) {
    if (threadIdx.x == 0) record_error(a.err, DEV_BAD_INDEX);
    return false;
  }
  b->held = lo & (page - 1);
  b->rows = hi - lo;
  b->row0 = it.row0 + (lo - start);
  b->pos0 = lo;
  b->dst = (is_v ? a.c.v : a.c.k) + id * a.c.page_stride + h * a.c.head_stride;
  b->scale = (is_v ? a.c.vs : a.c.ks) + static_cast<int64_t>(id) * a.c.Hkv + h;
  return true;
}

// The block's scale from every thread's largest |x| (bits), written; the older
// codes are brought to it if it grew.  |x| as integers: their order is the
// floats', and a NaN beats everything.
__device__ __forceinline__ float append_scale(const AppendArgs& a, const AppendBlock& b, uint32_t am) {
  __shared__ uint32_t red[32];
  const int tid = threadIdx.x, nw = blockDim.x >> 5;
  am = __reduce_max_sync(0xffffffffu, am);
  if ((tid & 31) == 0) red[tid >> 5] = am;
  const float old = b.held ? *b.scale : 0.f;
  __syncthreads();  // every thread has read the old scale
  for (int w = 0; w < nw; ++w) am = max(am, red[w]);
  const float scale = block_scale(__uint_as_float(am), old, b.held > 0, a.c.format);
  if (tid == 0) *b.scale = scale;
  if (b.held && !(scale == old)) {
    const float ratio = old / scale;
    const int per = a.c.dim / 4;
    for (int e = tid; e < b.held * per; e += blockDim.x) {
      const int r = e / per;
      uint32_t* q = reinterpret_cast<uint32_t*>(b.dst + r * a.c.tok_stride + (e - r * per) * 4);
      uint32_t w = *q, y = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y |= static_cast<uint32_t>(encode(decode(static_cast<uint8_t>(w >> (8 * i)), a.c.format) * ratio, a.c.format)) << (8 * i);
      *q = y;
    }
  }
  return scale;
}

// Any layout: a thread takes two channels at a time, a pair or two neighbours
// that do not turn, and the rotated rows wait in shared memory as fp32 for the
// scale, so each pair's sine and cosine are computed once (14.4 k tokens of four
// fp16 heads of 128, 54 channels turned: 24.6 us; a channel at a time, computed
// for the maximum and again for its code, 113).
constexpr int kAppendThreads = 256;
template <class T>
__global__ void __launch_bounds__(kAppendThreads) kv_append_any_kernel(AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  extern __shared__ __align__(16) float append_rows[];
  const bool is_v = blockIdx.z != 0;
  AppendBlock b;
  if (!append_block(a, is_v, static_cast<int>(blockIdx.y), &b)) return;
  const int D = a.c.dim, ulog = D == 128 ? 6 : 5;  // pairs of a row: 2^ulog
  const T* src = static_cast<const T*>(is_v ? a.v : a.k) + (is_v ? a.v_head : a.k_head) * blockIdx.y;
  const int64_t ts = is_v ? a.v_tok : a.k_tok;
  const int half = a.rope.rot / 2;
  const int u = threadIdx.x & ((1 << ulog) - 1);  // the thread's pair, in every row it takes
  const bool turns = !is_v && u < half;
  const int i = turns && !a.rope.interleaved ? u : 2 * u, j = turns && !a.rope.interleaved ? u + half : 2 * u + 1;
  const int64_t freq = turns ? a.rope.freqs[u] : 0;
  uint32_t am = 0;
  for (int r = static_cast<int>(threadIdx.x) >> ulog; r < b.rows; r += kAppendThreads >> ulog) {
    const T* row = src + (b.row0 + r) * ts;
    float p = to_f(row[i]), q = to_f(row[j]);
    if (turns) {
      float c, s;
      turn(a.pos ? a.pos[b.row0 + r] : b.pos0 + r, freq, &c, &s);
      c *= a.rope.amp;
      s *= a.rope.amp;
      const float p0 = p;
      p = p0 * c - q * s;
      q = q * c + p0 * s;
    }
    append_rows[r * D + i] = p;
    append_rows[r * D + j] = q;
    am = max(am, max(__float_as_uint(p) & 0x7fffffffu, __float_as_uint(q) & 0x7fffffffu));
  }
  const float scale = append_scale(a, b, am);  // its barrier is also the rows'
  const float inv = 1.f / scale;
  for (int e = threadIdx.x; e < b.rows * (D / 4); e += kAppendThreads) {
    const int r = e >> (ulog - 1), d = (e & (D / 4 - 1)) * 4;
    const float4 x = *reinterpret_cast<const float4*>(&append_rows[r * D + d]);
    const float v[4] = {x.x, x.y, x.z, x.w};
    uint32_t y = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) y |= static_cast<uint32_t>(encode(v[k] * inv, a.c.format)) << (8 * k);
    *reinterpret_cast<uint32_t*>(b.dst + (b.held + r) * a.c.tok_stride + d) = y;
  }
}

// Rows of whole 16-byte chunks: a thread holds NU units of a row's 16 channels
// (two 8-channel chunks, the partners of the half layout's pairs) in registers
// between the maximum and the codes, so each row is read once.  A CTA takes HB
// heads of a page, with the same sines and cosines, and loads the next head's
// rows before it works on the present one's: what bounds a block by itself is
// the chain of loads that finds it.
template <class T, int NU, int HB>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const bool is_v = blockIdx.z != 0;
  const int h0 = static_cast<int>(blockIdx.y) * HB;
  AppendBlock b;
  if (!append_block(a, is_v, h0, &b)) return;
  const int ulog = a.c.dim == 128 ? 3 : 2;  // units of a row: dim / 16
  const int nr = is_v ? 0 : a.rope.rot / 8;  // rotated chunks
  const bool inter = a.rope.interleaved != 0;
  const int64_t ts = is_v ? a.v_tok : a.k_tok, hs = is_v ? a.v_head : a.k_head;
  const int u = threadIdx.x & ((1 << ulog) - 1);  // blockDim.x is a multiple of a row's units
  const bool pairs = !inter && u < nr / 2;        // chunks whose channels turn with one another's
  const bool near1 = inter && 2 * u < nr, near2 = inter && 2 * u + 1 < nr;  // ... neighbours in the first, in both
  const int ca = pairs ? u : 2 * u, cb = pairs ? u + nr / 2 : ca + 1;
  const T* src = static_cast<const T*>(is_v ? a.v : a.k) + hs * h0 + static_cast<int64_t>(b.row0) * ts;
  Eight<T> x[NU][2];
  auto fetch = [&](const T* p) {
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int r = (threadIdx.x + k * blockDim.x) >> ulog;
      if (r < b.rows) {
        load8(p + r * ts + ca * 8, &x[k][0]);
        load8(p + r * ts + cb * 8, &x[k][1]);
      }
    }
  };
  fetch(src);
  float cs[NU][8], sn[NU][8];
  if (pairs || near1) {
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int r = (threadIdx.x + k * blockDim.x) >> ulog;
      if (r < b.rows) {
        const int p = a.pos ? a.pos[b.row0 + r] : b.pos0 + r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int pair = pairs ? ca * 8 + i : min(ca * 4 + i, a.rope.rot / 2 - 1);
          turn(p, a.rope.freqs[pair], &cs[k][i], &sn[k][i]);
          cs[k][i] *= a.rope.amp;
          sn[k][i] *= a.rope.amp;
        }
      }
    }
  }
#pragma unroll 1
  for (int h = h0;; ++h) {
    float v[NU][16];
    float am = 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int r = (threadIdx.x + k * blockDim.x) >> ulog;
      if (r < b.rows) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[k][i] = to_f(x[k][i >> 3].v[i & 7]);
        if (pairs) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float p = v[k][i], q = v[k][8 + i];
            v[k][i] = p * cs[k][i] - q * sn[k][i];
            v[k][8 + i] = q * cs[k][i] + p * sn[k][i];
          }
        } else if (near1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i >= 4 && !near2) break;
            const float p = v[k][2 * i], q = v[k][2 * i + 1];
            v[k][2 * i] = p * cs[k][i] - q * sn[k][i];
            v[k][2 * i + 1] = q * cs[k][i] + p * sn[k][i];
          }
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2) am = max_abs(am, v[k][i], v[k][i + 1]);
      }
    }
    const bool more = h + 1 < min(h0 + HB, a.c.Hkv);
    if (HB > 1 && more) {
      src += hs;
      fetch(src);
    }
    const float scale = append_scale(a, b, __float_as_uint(am) & 0x7fffffffu);
    const bool finite = fabsf(scale) < INFINITY;
    const float inv = 1.f / scale;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int r = (threadIdx.x + k * blockDim.x) >> ulog;
      if (r < b.rows) {
        uint8_t* row = b.dst + (b.held + r) * a.c.tok_stride;
        *reinterpret_cast<uint2*>(row + ca * 8) = finite ? encode8(v[k], inv, a.c.format) : make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(row + cb * 8) = finite ? encode8(v[k] + 8, inv, a.c.format) : make_uint2(0u, 0u);
      }
    }
    if (HB == 1 || !more) return;
    b.dst += a.c.head_stride;
    b.scale += 1;
    __syncthreads();  // the blocks' maxima are exchanged in one place
  }
}

template <class T, int HB>
int launch_append_h(const AppendArgs& a, unsigned items, cudaStream_t s) {
  const int units = (a.c.dim / 16) << a.c.page_log2;  // of a full block: 64 .. 1024
  const dim3 grid(items, static_cast<unsigned>((a.c.Hkv + HB - 1) / HB), 2);
  if (units <= 256) return launch_k(kv_append_kernel<T, 1, HB>, grid, dim3(static_cast<unsigned>(units)), 0, s, a);
  if (units == 512) return launch_k(kv_append_kernel<T, 2, HB>, grid, dim3(256), 0, s, a);
  return launch_k(kv_append_kernel<T, 4, HB>, grid, dim3(256), 0, s, a);
}

template <class T>
int launch_append_t(const AppendArgs& a, int sms, cudaStream_t s) {
  const unsigned items = static_cast<unsigned>((static_cast<int64_t>(a.q.n_tok) >> a.c.page_log2) + 2ll * a.q.n_seq);
  // 16-byte chunks: 8 channels (4 of fp32, loaded in twos)
  uint64_t m = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
  m |= static_cast<uint64_t>(a.k_tok | a.k_head | a.v_tok | a.v_head) * sizeof(T);
  const bool chunks = m % 16 == 0 && a.rope.rot % (a.rope.interleaved ? 8 : 16) == 0;
  if (!chunks) {
    const int smem = (a.c.dim << a.c.page_log2) * 4;  // a page's rows: 4 to 64 KB
    static KernelSetup setup;
    const cudaError_t r = setup.run(kv_append_any_kernel<T>, 128 * 128 * 4);
    if (r != cudaSuccess) return r;
    return launch_k(kv_append_any_kernel<T>, dim3(items, static_cast<unsigned>(a.c.Hkv), 2), dim3(kAppendThreads), smem, s, a);
  }
  // several heads a CTA where the pages alone fill the GPU
  const int64_t pages = static_cast<int64_t>(a.q.n_tok) >> a.c.page_log2;
  return 2 * pages >= 2ll * sms ? launch_append_h<T, 4>(a, items, s) : launch_append_h<T, 1>(a, items, s);
}

}  // namespace

int launch_kv_append(const AppendArgs& a, int sms, cudaStream_t s) {
  if (a.q.n_tok == 0 || a.q.n_seq == 0) return 0;
  switch (a.dtype) {
    case PCD_DTYPE_F32: return launch_append_t<float>(a, sms, s);
    case PCD_DTYPE_BF16: return launch_append_t<__nv_bfloat16>(a, sms, s);
    default: return launch_append_t<__half>(a, sms, s);
  }
}

namespace {
// =================================================================== attention
// Few query rows (8 or 16 to a tile: tokens x the G query heads of one KV
// head), warp tensor-core MMA.
//
// Every warp walks its own 16-key blocks of the tile's key range with a
// private cp.async ring, so no barrier stands in the key loop.  Codes become
// fp16 in registers, exactly.  With S = q . k8 and block scales sk, sv,
//   x = S sk c + log2 sv       (c = softmax scale x log2 e)
//   w = exp2(x - M + 8)        M: a running reference no lower than max x - 7
//   O += w v8,  l += w / sv,   out = O / l
// so the value's scale rides in the exponent: w <= 2^15 fits fp16 whatever the
// scales, and no value is rounded before the product.  Weights 2^-33 of the
// largest are the first that fp16 loses; l keeps them in fp32, down to 2^-126,
// which is enough for value scales 2^100 apart.
//
// The channel order inside a dot product is free, so the K fragments are taken
// as each lane's 16 consecutive bytes (Q's fragments are loaded in the same
// order), and a V fragment's column is any channel, so a lane reads 16
// consecutive channels of its four keys and pairs keys by byte permutes: no
// ldmatrix, no transposition in shared memory.
//
// Tiles of 16 rows compute S = Q K^T and O = w V with the rows as the MMA's 16.
// Tiles of 8 compute the transposes, K Q^T and V^T w^T, with keys and channels as
// the 16 and the rows as the 8: half the MMAs; the weights change sides by a
// register transpose (64 x 8 k keys of 7 query heads: 89 us against 99; 300
// contexts of up to 600: 43 against 53).
//
// Bound by the bytes of the pages: 64 contexts of 4 to 12 k keys 89 us, 5.8
// TB/s; three of 131 k int8 keys 73 us, 5.5 TB/s.  Each warp has two blocks in
// flight while it works on the third of its ring, 96 KB an SM of the rings' 144;
// three in flight (a fourth stage) or a fourth CTA took 115 to 120 us for the
// former, one in flight 92.  One context of 901 keys 8 us, a chain of trips.
//
// How the work is cut: small calls give every item (a tile of one KV head) to a
// thread-block cluster of up to 8 CTAs that divide its keys and join through
// distributed shared memory.  Large ones lay the 16-key blocks of all items on
// one line and give each of the resident CTAs the same stretch of it, so
// ragged lengths leave nobody idle; states of items that a stretch's end cuts go
// to scratch, and a second kernel joins them.
constexpr float kSlack = 7.f;
constexpr int kWarps = 4, kStagesR = 3;

template <int D>
struct RowsCfg {
  static constexpr int kStage = 16 * D * 2;                       // 16 keys: K then V
  static constexpr int kRing = kWarps * kStagesR * kStage;
  static constexpr int kRedLd = D + 4;
  static constexpr int kRedMl = kWarps * 16 * kRedLd * 4;         // partial rows after the key loop, then (M, l)
  static constexpr int kRed = kRedMl + (kWarps + 1) * 16 * 8;     // ... of the warps and of the CTA
  static constexpr int kSmem = kRing > kRed ? kRing : kRed;
};

// A sequence as the rows kernel divides it.
struct RowsSeq {
  int row0, n, len, tiles, blocks;  // tiles of rows (0: nothing to do), 16-key blocks of an item
};
template <int ROWS>
__device__ __forceinline__ RowsSeq rows_seq(const PagedAttnArgs& a, int row0, int n, int len) {
  RowsSeq q{row0, n, len, 0, 1};
  if (n == 0) return q;
  if (n < 0 || row0 < 0 || n > a.q.n_tok - row0) {
    record_error(a.err, DEV_BAD_INDEX);
    return q;
  }
  q.tiles = (n * a.G + ROWS - 1) / ROWS;
  if (len < 0 || len > kMaxLen || len > static_cast<int64_t>(a.q.table_width) << a.c.page_log2) {
    record_error(a.err, DEV_BAD_INDEX);
    q.len = 0;
  }
  q.blocks = max(1, (q.len + 15) >> 4);  // an item without keys still writes its rows
  return q;
}
template <int ROWS>
__device__ __forceinline__ RowsSeq rows_seq(const PagedAttnArgs& a, int s) {
  const int row0 = a.q.q_off[s];
  return rows_seq<ROWS>(a, row0, static_cast<int>(static_cast<unsigned>(a.q.q_off[s + 1]) - static_cast<unsigned>(row0)), a.q.kv_len[s]);
}
__device__ __forceinline__ int64_t rows_units(const PagedAttnArgs& a, const RowsSeq& q) {
  return static_cast<int64_t>(q.tiles) * a.c.Hkv * q.blocks;
}

template <int D, int FMT, class T, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, 3) paged_attn_rows_kernel(PagedAttnArgs a) {
  using C = RowsCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const bool stream = a.plan.stream != 0;
  int seq = 0, hk = blockIdx.y, tile = 0;
  RowsSeq sq;
  // a stretch [u, u_end) of the line of blocks; `before`: the blocks of the sequences ahead of `seq`
  int64_t u = 0, u_begin = 0, u_end = 0, before = 0, line = 0, n_cta = 1;
  if (stream) {
    for (int s0 = 0; s0 < a.q.n_seq; s0 += 32) {
      int64_t w = 0;
      if (s0 + lane < a.q.n_seq) w = rows_units(a, rows_seq<ROWS>(a, s0 + lane));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      line += w;
    }
    n_cta = min(static_cast<int64_t>(gridDim.x), line);  // nobody's stretch is empty
    if (blockIdx.x >= n_cta) return;
    u_begin = u = line * blockIdx.x / n_cta;
    u_end = line * (blockIdx.x + 1) / n_cta;
    for (int s0 = 0;; s0 += 32) {
      int64_t w = 0;
      if (s0 + lane < a.q.n_seq) w = rows_units(a, rows_seq<ROWS>(a, s0 + lane));
      int64_t upto = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + upto > u);
      if (past) {
        const int l = __ffs(past) - 1;
        seq = s0 + l;
        before += __shfl_sync(0xffffffffu, upto - w, l);
        break;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    sq = rows_seq<ROWS>(a, seq);
  } else {
    // (what returns here returns in every CTA of a cluster)
    const OffsetCheck offsets(a.q);
    const SeqItem it = find_item(a.q, static_cast<int>(blockIdx.x), a.G, ROWS == 8 ? 3 : 4, 1);
    offsets.report(a.q, a.err);
    if (it.seq < 0) return;
    seq = it.seq;
    tile = it.local;
    sq = rows_seq<ROWS>(a, it.row0, it.n, it.len);
    if (tile >= sq.tiles) return;
  }
  for (;;) {
  int range0 = 0, range1 = 0, slot = -1;  // blocks of the item; where its state goes
  if (stream) {
    while (u >= before + rows_units(a, sq)) {
      before += rows_units(a, sq);
      sq = rows_seq<ROWS>(a, ++seq);
    }
    const int64_t at = u - before;
    const int64_t item = at / sq.blocks;
    hk = static_cast<int>(item / sq.tiles);
    tile = static_cast<int>(item % sq.tiles);
    range0 = static_cast<int>(at - item * sq.blocks);
    range1 = static_cast<int>(min(static_cast<int64_t>(sq.blocks), range0 + (u_end - u)));
    if (range0 > 0 || range1 < sq.blocks) slot = 2 * blockIdx.x + (u == u_begin ? 0 : 1);
  }
  const int n = sq.n, len = sq.len;
  const int R = n * a.G;
  const int r0 = tile * ROWS;
  const int r_end = min(r0 + ROWS, R);
  const bool upper = ROWS == 16 && r_end - r0 > 8;  // rows 8 .. 15 exist
  // keys seen by a row: all, or up to its own position
  const int first = a.causal ? len - n + 1 : len;  // by the sequence's first token
  auto seen = [&](int r) { return a.causal ? first + min(r, R - 1) / a.G : len; };
  const int kmax = max(0, seen(r_end - 1));
  const int kmin = max(0, seen(r0));
  const int bl = (kmax + 15) >> 4;
  if (!stream) {  // even ranges, whole rounds of the warps
    const int per = ((bl + a.plan.n_splits - 1) / a.plan.n_splits + kWarps - 1) / kWarps * kWarps;
    range0 = static_cast<int>(blockIdx.z) * per;
    range1 = range0 + per;
  }
  const int b0 = min(bl, range0), b1 = min(bl, range1);
  const int nb = b1 > b0 + warp ? (b1 - b0 - warp + kWarps - 1) / kWarps : 0;  // blocks of this warp

  // ---- page ids and constants of 32 of this warp's blocks at a time, one to a lane
  const int32_t* tab = a.q.table + static_cast<int64_t>(seq) * a.q.table_stride;
  auto block_at = [&](int i) { return b0 + warp + i * kWarps; };
  auto fetch_ids = [&](int i0) {
    const int i = i0 + lane;
    int id = -1;
    if (i < nb) {
      id = tab[block_at(i) >> (a.c.page_log2 - 4)];
      if (id < 0 || id >= a.c.n_pages) {
        record_error(a.err, DEV_BAD_INDEX);
        id = -1;
      }
    }
    return id;
  };
  int ids = fetch_ids(0), ids_next = fetch_ids(32);
  float sk, lsv, isv;  // K scale, log2 and reciprocal of the V scale; isv 0: a page the table has wrong
  auto scales = [&](int id) {
    float k = 0.f, v = 1.f;
    if (id >= 0) {
      k = a.c.ks[static_cast<int64_t>(id) * a.c.Hkv + hk];
      v = a.c.vs[static_cast<int64_t>(id) * a.c.Hkv + hk];
      if (v < kScaleFloor) v = kScaleFloor;  // a NaN stays
    }
    sk = k;
    lsv = lg2(v);
    isv = id < 0 ? 0.f : 1.f / (v + (v - v));  // not finite: NaN
  };

  // ---- the ring: a lane copies the same 16 bytes of kCh / 2 keys of K and of V in every block
  constexpr int kCh = D / 16;
  uint8_t* ring = smem + warp * (kStagesR * C::kStage);
  const int key0 = lane / kCh, ch = lane % kCh;  // and keys key0 + 32 / kCh, ...
  const int step = static_cast<int>(a.c.tok_stride) * (32 / kCh);
  const uint8_t* ksrc = a.c.k + hk * a.c.head_stride + key0 * a.c.tok_stride + ch * 16;
  const int64_t vdelta = a.c.v - a.c.k;
  // shared places of key0's chunks; later keys keep K's swizzle, and V's but for its upper bit
  const uint32_t kdst = smem_u32(ring) + key0 * D + ((ch ^ ((key0 & 1) << 2)) & (kCh - 1)) * 16;
  const uint32_t vdst = smem_u32(ring) + 16 * D + key0 * D + ((ch ^ (((key0 >> 1) & 3) << 1)) & (kCh - 1)) * 16;
  auto v_place = [](uint32_t p, int e) { return D == 128 && (e & 1) ? p ^ 64u : p; };
  int ids_at = 0;  // `ids` holds blocks ids_at ..
  uint32_t fill = 0;
  auto issue = [&](int i) {
    if (i < nb) {
      if (i - ids_at >= 32) {
        ids = ids_next;
        ids_at = i;
        ids_next = fetch_ids(i + 32);
      }
      const int id = __shfl_sync(0xffffffffu, ids, i - ids_at);
      const int j0 = block_at(i) << 4;
      const int slot = j0 & ((1 << a.c.page_log2) - 1);
      const uint8_t* src = ksrc + max(id, 0) * a.c.page_stride + slot * a.c.tok_stride;
      if (id >= 0 && j0 + 16 <= len) {
#pragma unroll
        for (int e = 0; e < kCh / 2; ++e) {
          cp_async16_to(kdst + fill + e * (32 / kCh) * D, src + e * step, 16);
          cp_async16_to(v_place(vdst, e) + fill + e * (32 / kCh) * D, src + vdelta + e * step, 16);
        }
      } else {  // slots behind the last token, and pages the table has wrong, read as zeros
#pragma unroll
        for (int e = 0; e < kCh / 2; ++e) {
          const int bytes = id >= 0 && j0 + key0 + e * (32 / kCh) < len ? 16 : 0;
          cp_async16_to(kdst + fill + e * (32 / kCh) * D, src + e * step, bytes);
          cp_async16_to(v_place(vdst, e) + fill + e * (32 / kCh) * D, src + vdelta + e * step, bytes);
        }
      }
    }
    cp_async_commit();
    fill = fill + C::kStage == kStagesR * C::kStage ? 0u : fill + C::kStage;
  };
#pragma unroll 1
  for (int i = 0; i < kStagesR - 1; ++i) issue(i);
  scales(ids);
  int sc_at = 0, drain = 0;

  // ---- Q fragments: k-step t takes channels (64 * (t / 4) + 16 c + 4 (t % 4)) + {0, 1 | 2, 3}
  // Row g of the tile, and row g + 8: rows of MMA's A, or (8 rows) the columns of its B, two registers a step
  constexpr int kE = ROWS / 8;
  uint32_t qf[D / 16][2 * kE];
  float qs[2] = {0.f, 0.f};
  float row_m[2] = {-INFINITY, -INFINITY}, row_l[2] = {0.f, 0.f};  // of rows g, g + 8; or 2c, 2c + 1
  int vis[2];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int r = r0 + g + 8 * e;
    vis[e] = seen(r);
    const bool ok = r < R;
    const int tok = sq.row0 + (ok ? r : r0) / a.G, hq = hk * a.G + (ok ? r : r0) % a.G;
    const T* src = static_cast<const T*>(a.x) + tok * a.x_tok + hq * a.x_head;
    const bool wide = (reinterpret_cast<uintptr_t>(src) & 7) == 0;
    alignas(8) T v[D / 16][4];
    uint32_t am = 0;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      const int d = 64 * (t >> 2) + 16 * c + 4 * (t & 3);
      if (!ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[t][i] = from_f<T>(0.f);
      } else if (wide) {
        *reinterpret_cast<uint2*>(v[t]) = *reinterpret_cast<const uint2*>(src + d);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[t][i] = src[d + i];
      }
    }
    if (!std::is_same<T, __half>::value) {
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) am = max(am, __float_as_uint(to_f(v[t][i])) & 0x7fffffffu);
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
    }
    float down;
    qs[e] = row_power<T>(am, &down) * a.scale_log2;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      if (std::is_same<T, __half>::value) {
        qf[t][e] = reinterpret_cast<const uint32_t*>(v[t])[0];
        qf[t][kE + e] = reinterpret_cast<const uint32_t*>(v[t])[1];
      } else {
        qf[t][e] = pack2(to_f(v[t][0]) * down, to_f(v[t][1]) * down);
        qf[t][kE + e] = pack2(to_f(v[t][2]) * down, to_f(v[t][3]) * down);
      }
    }
  }

  if (ROWS == 8) {  // the softmax's lanes have rows 2c and 2c + 1
    const float q = qs[0];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      qs[e] = __shfl_sync(0xffffffffu, q, (2 * c + e) * 4);
      vis[e] = seen(r0 + 2 * c + e);
    }
  }

  constexpr int kO = ROWS == 8 ? D / 16 : D / 8;
  float o[kO][4];
#pragma unroll
  for (int t = 0; t < kO; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[t][i] = 0.f;

#pragma unroll 1
  for (int i = 0; i < nb; ++i) {
    cp_async_wait<kStagesR - 2>();
    __syncwarp();
    if (i - sc_at >= 32) {
      sc_at = i;
      scales(fetch_ids(i));
    }
    issue(i + kStagesR - 1);
    const float bsk = __shfl_sync(0xffffffffu, sk, i - sc_at);
    const float blsv = __shfl_sync(0xffffffffu, lsv, i - sc_at);
    const float bisv = __shfl_sync(0xffffffffu, isv, i - sc_at);
    const uint8_t* st = ring + drain;
    drain = drain + C::kStage == kStagesR * C::kStage ? 0 : drain + C::kStage;
    // ---- S = Q K^T: two tiles of 8 keys (or K Q^T: 16 keys by 8 rows)
    float s[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int hf = 0; hf < D / 64; ++hf) {
      uint4 w[2];
      uint32_t ka[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = 8 * t + g;
        w[t] = *reinterpret_cast<const uint4*>(st + key * D + (((c + 4 * hf) ^ ((key & 1) << 2)) & (kCh - 1)) * 16);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t h0, h1;
          codes4_half<FMT>(q == 0 ? w[t].x : q == 1 ? w[t].y : q == 2 ? w[t].z : w[t].w, &h0, &h1);
          if constexpr (ROWS == 16) mma16816(s[t], qf[4 * hf + q], h0, h1);
          else ka[t][0] = h0, ka[t][1] = h1;
          if (ROWS == 8 && t == 1) {  // two chains of steps, joined below
            const uint32_t kf[4] = {ka[0][0], h0, ka[0][1], h1};
            mma16816(s[q & 1], kf, qf[4 * hf + q][0], qf[4 * hf + q][1]);
          }
        }
    }
    // ---- weights (rows 8 .. 15 only where the tile has them)
    const int j0 = block_at(i) << 4;
    uint32_t pf[4];
    if constexpr (ROWS == 8) {
      // x[e]: keys g and g + 8 of row 2c + e
      float x[2][2], iv[2];
      const bool edge = j0 + 16 > kmin || bisv == 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ak = qs[e] * bsk;
        x[e][0] = fmaf(s[0][e] + s[1][e], ak, blsv);
        x[e][1] = fmaf(s[0][2 + e] + s[1][2 + e], ak, blsv);
        iv[e] = bisv;
        if (edge) {
          const int lim = bisv == 0.f ? 0 : vis[e] - j0 - g;
          x[e][0] = 0 < lim ? x[e][0] : -INFINITY;
          x[e][1] = 8 < lim ? x[e][1] : -INFINITY;
          if (vis[e] <= j0) iv[e] = 0.f;  // a poisoned scale (NaN) counts only for rows that see its keys
        }
      }
      const float m0 = fmaxf(x[0][0], x[0][1]), m1 = fmaxf(x[1][0], x[1][1]);
      if (__any_sync(0xffffffffu, m0 > row_m[0] + kSlack || m1 > row_m[1] + kSlack)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = e ? m1 : m0;
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
          m = fmaxf(m, row_m[e]);
          const float f = row_m[e] == -INFINITY ? 0.f : ex2_approx(row_m[e] - m);
          row_m[e] = m;
          row_l[e] *= f;
#pragma unroll
          for (int t = 0; t < kO; ++t) {
            o[t][e] *= f;
            o[t][2 + e] *= f;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mb = (row_m[e] == -INFINITY ? 0.f : row_m[e]) - kBias;
        x[e][0] = ex2_approx(x[e][0] - mb);
        x[e][1] = ex2_approx(x[e][1] - mb);
        row_l[e] = fmaf(x[e][0] + x[e][1], iv[e], row_l[e]);
      }
      pf[0] = transpose8x8(pack2(x[0][0], x[1][0]));  // rows by keys 0 .. 7
      pf[1] = transpose8x8(pack2(x[0][1], x[1][1]));  // ... 8 .. 15
    } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (e == 1 && !upper) {
        pf[1] = pf[3] = 0u;
        break;
      }
      const float ak = qs[e] * bsk;
      float x[4] = {s[0][2 * e], s[0][2 * e + 1], s[1][2 * e], s[1][2 * e + 1]};
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = fmaf(x[k], ak, blsv);
      float iv = bisv;
      if (j0 + 16 > kmin || bisv == 0.f) {
        const int lim = bisv == 0.f ? 0 : vis[e] - j0 - 2 * c;
        x[0] = 0 < lim ? x[0] : -INFINITY;
        x[1] = 1 < lim ? x[1] : -INFINITY;
        x[2] = 8 < lim ? x[2] : -INFINITY;
        x[3] = 9 < lim ? x[3] : -INFINITY;
        if (vis[e] <= j0) iv = 0.f;  // a poisoned scale (NaN) counts only for rows that see its keys
      }
      float m = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      if (__any_sync(0xffffffffu, m > row_m[e] + kSlack)) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = fmaxf(m, row_m[e]);
        const float f = row_m[e] == -INFINITY ? 0.f : ex2_approx(row_m[e] - m);
        row_m[e] = m;
        row_l[e] *= f;
#pragma unroll
        for (int t = 0; t < kO; ++t) {
          o[t][2 * e] *= f;
          o[t][2 * e + 1] *= f;
        }
      }
      const float mb = (row_m[e] == -INFINITY ? 0.f : row_m[e]) - kBias;
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = ex2_approx(x[k] - mb);
      row_l[e] = fmaf((x[0] + x[1]) + (x[2] + x[3]), iv, row_l[e]);
      pf[e] = pack2(x[0], x[1]);
      pf[2 + e] = pack2(x[2], x[3]);
    }
    }
    // ---- O += w V: column tile t's lane group g is channel g * (D / 8) + t
    const uint8_t* sv = st + 16 * D;
    constexpr int kLd = D / 8;  // channels of a lane: 16 or 8 bytes
    uint32_t vr[4][kLd / 4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int key = 2 * c + (kk & 1) + 8 * (kk >> 1);
      const int byte = g * kLd;
      const uint8_t* p = sv + key * D + (((byte >> 4) ^ (((key >> 1) & 3) << 1)) & (kCh - 1)) * 16 + (byte & 15);
      if constexpr (kLd == 16) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        vr[kk][0] = w.x, vr[kk][1] = w.y, vr[kk][2] = w.z, vr[kk][3] = w.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        vr[kk][0] = w.x, vr[kk][1] = w.y;
      }
    }
#pragma unroll
    for (int t = 0; t < D / 8; t += 2) {
      uint32_t v0[2], v1[2];
      codes_cross_half<FMT>(vr[0][t >> 2], vr[1][t >> 2], (t >> 1) & 1, &v0[0], &v0[1]);
      codes_cross_half<FMT>(vr[2][t >> 2], vr[3][t >> 2], (t >> 1) & 1, &v1[0], &v1[1]);
      if constexpr (ROWS == 16) {
        mma16816(o[t], pf, v0[0], v1[0]);
        mma16816(o[t + 1], pf, v0[1], v1[1]);
      } else {  // channels g * (D / 8) + t and + 1 of all lane groups as the MMA's rows g and g + 8
        const uint32_t vf[4] = {v0[0], v0[1], v1[0], v1[1]};
        mma16816(o[t / 2], vf, pf[0], pf[1]);
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int w = ROWS == 8 ? 4 : 1; w < (ROWS == 8 ? 32 : 4); w <<= 1) row_l[e] += __shfl_xor_sync(0xffffffffu, row_l[e], w);
  // ---- join the warps
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  float2* ml = reinterpret_cast<float2*>(smem + C::kRedMl);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (ROWS == 16 && e == 1 && !upper) break;
    const int r = ROWS == 8 ? 2 * c + e : g + 8 * e;
    if ((ROWS == 8 ? g : c) == 0) ml[warp * 16 + r] = make_float2(row_m[e], row_l[e]);
#pragma unroll
    for (int t = 0; t < D / 8; t += 2) {
      if constexpr (ROWS == 8) {
        *reinterpret_cast<float2*>(&red[(warp * 16 + r) * C::kRedLd + g * (D / 8) + t]) =
            make_float2(o[t / 2][e], o[t / 2][2 + e]);
      } else {  // accumulator column 2c + i is lane group 2c + i's channel
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<float2*>(&red[(warp * 16 + r) * C::kRedLd + (2 * c + i) * (D / 8) + t]) =
              make_float2(o[t][2 * e + i], o[t + 1][2 * e + i]);
      }
    }
  }
  __syncthreads();
  const bool cluster = a.plan.cluster != 0;
  const int work = (r_end - r0) * (D / 4);
  for (int x = threadIdx.x; x < work; x += kWarps * 32) {
    const int r = x / (D / 4), d = (x % (D / 4)) * 4;
    RowState st;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) st.top(ml[w * 16 + r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      st.add(ml[w * 16 + r], *reinterpret_cast<const float4*>(red + (w * 16 + r) * C::kRedLd + d));
    if (cluster) {  // warp 0's rows now hold the CTA's: each thread read what it overwrites
      *reinterpret_cast<float4*>(red + r * C::kRedLd + d) = st.o;
      if (d == 0) ml[kWarps * 16 + r] = make_float2(st.M, st.L);
      continue;
    }
    const int rr = r0 + r, tok = sq.row0 + rr / a.G, hq = hk * a.G + rr % a.G;
    if (slot < 0) {
      finish_row<T>(a, st, tok, hq, d);
    } else {
      const int64_t p = static_cast<int64_t>(slot) * 16 + r;
      *reinterpret_cast<float4*>(a.part_o + p * D + d) = st.o;
      if (d == 0) a.part_ml[p] = make_float2(st.M, st.L);
    }
    // the CTA of an item's first blocks says where the row's parts are
    if (stream && range0 == 0 && d == 0) {
      int parts = 0;
      if (slot >= 0) {
        const int64_t end = u + sq.blocks;  // the line's end of this item: the CTA of its last block
        int last = static_cast<int>(min(n_cta - 1, end * n_cta / line));
        while (line * last / n_cta >= end) --last;
        parts = last - static_cast<int>(blockIdx.x) + 1;
      }
      a.part_at[static_cast<int64_t>(tok) * a.Hq + hq] = make_int2(slot * 16 + r, parts);
    }
  }
  if (stream) {
    u += range1 - range0;
    if (u >= u_end) return;
    __syncthreads();  // the ring reuses what the join read
    continue;
  }
  if (!cluster) return;
  cluster_sync_all();
  const int nz = a.plan.n_splits;
  for (int x = blockIdx.z * kWarps * 32 + threadIdx.x; x < work; x += nz * kWarps * 32) {
    const int r = x / (D / 4), d = (x % (D / 4)) * 4;
    RowState st;
    float2 m[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < nz) st.top(m[q] = dsmem_ld_f2(dsmem_addr(ml + kWarps * 16 + r, q)));
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < nz) st.add(m[q], dsmem_ld_f4(dsmem_addr(red + r * C::kRedLd + d, q)));
    const int rr = r0 + r;
    finish_row<T>(a, st, sq.row0 + rr / a.G, hk * a.G + rr % a.G, d);
  }
  cluster_sync_all();  // no CTA leaves while another reads its shared memory
  return;
  }
}

// Do the parts of row (tok, hq) come from this call?  Rows of no sequence and of
// sequences with bad offsets have none: they stay as they are.
__device__ __forceinline__ bool row_taken(const PagedAttnArgs& a, int tok, int hq) {
  if (a.q.n_seq <= 32) {  // all offsets good, as nearly always: seen in one trip to memory
    const int lane = threadIdx.x & 31;
    int off = 0, end = 0;
    if (lane < a.q.n_seq) {
      off = a.q.q_off[lane];
      end = a.q.q_off[lane + 1];
    }
    if (!__any_sync(0xffffffffu, off != end && (off < 0 || end < off || end > a.q.n_tok)))
      return __any_sync(0xffffffffu, off <= tok && tok < end);
  }
  const SeqItem it = find_row(a.q, tok);
  if (it.seq < 0 || a.plan.stream) return it.seq >= 0;
  // where other offsets decrease, the tile kernel may not have found the row's item
  const int tile = (it.local * a.G + hq % a.G) >> kTileRowsLog, tiles = (it.n * a.G + kTileRows - 1) >> kTileRowsLog;
  const int item = (it.row0 * a.G >> kTileRowsLog) + it.seq + tiles - 1 - tile;
  return find_item(a.q, item, a.G, kTileRowsLog, 1).seq == it.seq;
}

// Joins the parts of a row: out = sum 2^(M_i - M) O_i / sum 2^(M_i - M) l_i.
// With ranges, part i is range i's state of the row; with stretches, the first
// part is where part_at says and the others begin the stretches of the CTAs
// after it.  A warp takes 32 parts at a time, one (M, l) to a lane, then their O
// rows one after the other with the loads in flight together; W warps share a
// row (4 where a row may have more than 32 parts, else 1).
constexpr int kJoinWarps = 4;
template <int D, class T, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_attn_join_kernel(PagedAttnArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kV = D / 32;  // channels of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = static_cast<int>(blockIdx.x) * (kJoinWarps / W) + warp / W;
  if (row >= a.q.n_tok * a.Hq) return;
  const int tok = row / a.Hq, hq = row % a.Hq;
  if (!row_taken(a, tok, hq)) return;
  int2 at = make_int2(0, a.plan.n_splits);
  if (a.plan.stream) {
    at = a.part_at[row];
    // (offsets that decrease may give a row to two sequences: nothing is followed out of range)
    const int cta = at.x >> 5;
    if (at.x < 0 || at.y < 1 || cta >= a.plan.n_splits || at.y > a.plan.n_splits - cta) return;
  }
  const int64_t rows = static_cast<int64_t>(a.q.n_tok) * a.Hq;
  auto part = [&](int i) {
    if (!a.plan.stream) return i * rows + row;
    return static_cast<int64_t>(i == 0 ? at.x : ((at.x >> 5) + i) * 32 + (at.x & 15));
  };
  float M = -INFINITY, L = 0.f, o[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) o[k] = 0.f;
  for (int i0 = (warp % W) * 32; i0 < at.y; i0 += W * 32) {
    const int n = min(32, at.y - i0);
    const float2 ml = lane < n ? a.part_ml[part(i0 + lane)] : make_float2(-INFINITY, 0.f);
    float m = ml.y != 0.f ? ml.x : -INFINITY;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    m = fmaxf(m, M);
    const float f = M == -INFINITY ? 0.f : ex2_approx(M - m);
    M = m;
    L *= f;
#pragma unroll
    for (int k = 0; k < kV; ++k) o[k] *= f;
    const float w = ml.y != 0.f ? ex2_approx(ml.x - m) : 0.f;
    L = fmaf(w, ml.y, L);  // of this lane's parts
    const unsigned some = __ballot_sync(0xffffffffu, ml.y != 0.f);
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const float* src = a.part_o + part(i0 + j) * D + lane * kV;
      float v[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) v[k] = some >> j & 1 ? src[k] : 0.f;  // an empty part has no O
#pragma unroll
      for (int k = 0; k < kV; ++k) o[k] = fmaf(wj, v[k], o[k]);
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
  __shared__ float2 sml[kJoinWarps];
  __shared__ __align__(16) float so[kJoinWarps][D];
  if (lane == 0) sml[warp] = make_float2(M, L);
#pragma unroll
  for (int k = 0; k < kV; ++k) so[warp][lane * kV + k] = o[k];
  if (W > 1) __syncthreads();  // the warps of a CTA have one row: they return together or not at all
  else __syncwarp();
  if (warp % W || lane >= D / 4) return;
  const int d = lane * 4;
  RowState st;
#pragma unroll
  for (int w = 0; w < W; ++w) st.top(sml[warp + w]);
#pragma unroll
  for (int w = 0; w < W; ++w) st.add(sml[warp + w], *reinterpret_cast<const float4*>(&so[warp + w][d]));
  finish_row<T>(a, st, tok, hq, d);
}

template <int D, class T, int W>
int launch_join_w(const PagedAttnArgs& a, cudaStream_t s) {
  auto kern = paged_attn_join_kernel<D, T, W>;
  static KernelSetup setup;
  const cudaError_t r = setup.run(kern, 0);
  if (r != cudaSuccess) return r;
  constexpr int kRows = kJoinWarps / W;
  return launch_k(kern, dim3(static_cast<unsigned>((a.q.n_tok * a.Hq + kRows - 1) / kRows)), dim3(kJoinWarps * 32), 0, s, a);
}
template <int D, class T>
int launch_join(const PagedAttnArgs& a, cudaStream_t s) {
  return a.plan.parts > 32 ? launch_join_w<D, T, 4>(a, s) : launch_join_w<D, T, 1>(a, s);
}

template <int D, int FMT, class T, int ROWS>
int launch_rows(const PagedAttnArgs& a, cudaStream_t s) {
  using C = RowsCfg<D>;
  auto kern = paged_attn_rows_kernel<D, FMT, T, ROWS>;
  static KernelSetup setup;
  const cudaError_t r = setup.run(kern, C::kSmem);
  if (r != cudaSuccess) return r;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = a.plan.stream ? dim3(static_cast<unsigned>(a.plan.n_splits))
                              : dim3(static_cast<unsigned>(((static_cast<int64_t>(a.q.n_tok) * a.G) / ROWS) + a.q.n_seq),
                                     static_cast<unsigned>(a.c.Hkv), static_cast<unsigned>(a.plan.n_splits));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int na = 0;
  if (a.plan.cluster) {
    at[na].id = cudaLaunchAttributeClusterDimension;
    at[na].val.clusterDim.x = 1;
    at[na].val.clusterDim.y = 1;
    at[na].val.clusterDim.z = static_cast<unsigned>(a.plan.n_splits);
    ++na;
  }
  if (pdl_enabled()) {
    at[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = at;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D, int FMT>
int launch_rows_t(const PagedAttnArgs& a, cudaStream_t s) {
  if (a.plan.rows == 8)
    return a.dtype == PCD_DTYPE_BF16 ? launch_rows<D, FMT, __nv_bfloat16, 8>(a, s) : launch_rows<D, FMT, __half, 8>(a, s);
  return a.dtype == PCD_DTYPE_BF16 ? launch_rows<D, FMT, __nv_bfloat16, 16>(a, s) : launch_rows<D, FMT, __half, 16>(a, s);
}

}  // namespace

void plan_paged_attention(int n_tok, int n_seq, int G, int Hkv, int64_t max_kv, int sms, PagedPlan* p) {
  max_kv = std::min<int64_t>(max_kv, int64_t{1} << 31);
  const int64_t per = n_seq > 0 ? (n_tok + n_seq - 1) / n_seq : 0;  // query tokens of a sequence, on average
  const auto tiles_of = [&](int64_t rows) { return std::max<int64_t>(1, n_seq * ((per * G + rows - 1) / rows) * Hkv); };
  // Up to 32 rows a sequence and KV head the rows kernel reads each page at most
  // twice (64 x 8 k keys, 28 rows: 200 us against 239 in tcgen05 tiles; 35 rows:
  // 290 against 240).  Short contexts of few sequences take it further, while
  // clusters of all their tiles are resident together (901 keys, 144 rows: 12
  // us against 14.5, and one launch).
  p->rows = per * G <= 8 ? 8 : per * G > 32 && (tiles_of(16) * 8 > 3 * sms || max_kv > 1024) ? 256 : 16;
  const int64_t tiles = tiles_of(p->rows);
  const int64_t slots = static_cast<int64_t>(sms) * 3;  // resident CTAs of the rows kernel
  p->stream = p->cluster = 0;
  p->alternate = p->rows == 256 && per * G <= 128;
  int64_t want;
  if (p->rows <= 16) {
    // Ranges for about 7/4 CTAs a slot, at most a cluster's 8.  The even
    // stretches where there is much to read in long contexts (four KV heads, 7
    // query heads each: 64 x 8 k keys take 89 us against 101 in ranges, 16 x 8 k
    // 35 against 41, 64 x 1 k .. 2 k 35 against 37, but 300 x 300 .. 600 58
    // against 44), or where 8 ranges leave most SMs idle and each is longer than
    // the stretches' own 17 us of set-up and joining are worth (1 x 8 k keys: 15
    // us in a cluster against 18.5; 1 x 16 k: 24 against 19.5).
    want = std::max<int64_t>(1, slots * 7 / 4 / tiles);
    p->stream = n_seq <= 4096 && ((max_kv >= 2000 && tiles * max_kv >= slots * 1000) || (want > 8 && max_kv > 10240));
    want = p->stream ? slots : std::min<int64_t>(std::min<int64_t>(want, 8), (max_kv + 63) / 64);
    p->cluster = !p->stream && want > 1;
  } else {
    // The number of ranges with the least time by this account, in us: waves of
    // CTAs, each 8 to start and end and 1.9 a key block, then the join's launch and
    // the parts written and read (1 KB each).  Against one wave where that fits and
    // else no ranges: 26 prompts of 4 to 90 tokens behind 7 k keys, 24 heads, 225 us
    // for 241; 22 of 186 tokens, heads of 64, 169 for 176.  More than 32 MiB
    // of parts have to promise a twentieth, and 512 MiB is the most: 8192 tokens of 64
    // heads at the end of 131072 keys, promised 2.4%, took 26.9 ms in two ranges and
    // 545 MB against 26.3 in one; 3630 of 24 heads at 9812, 3%, 389 us and 91 MB against
    // 352; 2048 of 64 at 131072, 13%, 7.07 ms in five against 7.70.  Less is worth small
    // gains: 26 x 41 tokens of 7 heads at 929 keys, 2.7%, 24.8 us in two against 25.9.
    const int64_t blocks = std::max<int64_t>(1, (max_kv + 127) / 128);
    const double range_bytes = static_cast<double>(n_tok) * G * Hkv * (128 * 4 + 8);
    double best = 0.0, one = 0.0;
    want = 1;
    for (int64_t n = 1; n <= std::min(blocks, std::max<int64_t>(8, sms / tiles)); ++n) {
      const double waves = static_cast<double>((tiles * n + sms - 1) / sms);
      const double t = waves * (8.0 + 1.9 * static_cast<double>((blocks + n - 1) / n)) +
                       (n > 1 ? 4.0 + n * static_cast<double>(n_tok) * G * Hkv * 2e-4 : 0.0);
      if (n == 1) best = one = t;
      else if (t < best && (n * range_bytes <= 33554432.0 || (t < 0.95 * one && n * range_bytes <= 536870912.0))) best = t, want = n;
    }
  }
  p->n_splits = static_cast<int>(std::max<int64_t>(want, 1));
  // parts of a row, about: an item may lie on several stretches
  p->parts = p->stream ? static_cast<int>(slots / tiles + 2) : p->n_splits;
}

int launch_paged_attention(const PagedAttnArgs& a, cudaStream_t s) {
  if (a.q.n_tok == 0 || a.q.n_seq == 0) return 0;
  const bool f8 = a.c.format == PCD_KV_E4M3;
  int r;
  if (a.plan.rows == 256)
    r = launch_paged_attention_tiles(a, s);
  else if (a.c.dim == 64)
    r = f8 ? launch_rows_t<64, PCD_KV_E4M3>(a, s) : launch_rows_t<64, PCD_KV_INT8>(a, s);
  else
    r = f8 ? launch_rows_t<128, PCD_KV_E4M3>(a, s) : launch_rows_t<128, PCD_KV_INT8>(a, s);
  if (r != 0 || a.plan.n_splits == 1 || a.plan.cluster) return r;
  const bool bf = a.dtype == PCD_DTYPE_BF16;
  if (a.c.dim == 64) return bf ? launch_join<64, __nv_bfloat16>(a, s) : launch_join<64, __half>(a, s);
  return bf ? launch_join<128, __nv_bfloat16>(a, s) : launch_join<128, __half>(a, s);
}

}  // namespace pcd
