// Attention over the 8-bit paged cache for many query rows, on the
// 5th-generation tensor cores.
//
// A CTA owns 256 query rows of one sequence and KV head (rows are tokens x
// the G query heads, flattened) as two tiles of 128 and walks key blocks of
// 128:
//   codes -> fp16, exactly     four warps, registers to swizzled shared memory
//   S = Q K^T                  tcgen05.mma, 128 x 128, accumulator in TMEM
//   w = exp2(S sk c + log2 sv - M + 8)   one thread a row
//   O += w V8                  tcgen05.mma, w (fp16) from TMEM over S's columns
//   l += w / sv                so out = O / l (see the rows kernel)
// Each K and V block is converted once for both tiles; while one tile's rows
// are in the softmax the tensor cores work for the other.  M moves, and O and l
// are rescaled, only when a block exceeds it by 2^7.
//
// Registers: 512 threads launch with 128 each; the two softmax warpgroups
// hold a row of 128 scores and take 192, paid for by the converters (88) and
// the issuers (40): 40 + 88 + 192 + 192 = 4 x 128.
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "paged.cuh"
#include "paged.h"
#include "pcd.h"
#include "pcd_kernels.h"
#include "ptx.cuh"

namespace pcd {
namespace {

constexpr int kTile = 128;        // rows of a tile (MMA M)
constexpr int kRowsCta = 2 * kTile;
constexpr int kBlock = 128;       // keys of a block (MMA N of S, K of P V)
constexpr int kHalf = kTile * 128;  // bytes of 64 channels x 128 rows, one 128-byte swizzled row each
constexpr float kSlackTc = 7.f;
constexpr uint64_t kWaitNs = 2000000000ull;

template <int D>
struct TileCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kOp = kHalves * kHalf;           // one operand tile: 128 rows x D fp16
  static constexpr int kOffK = 2 * kOp;                 // after the two Q tiles
  static constexpr int kOffV = kOffK + 2 * kOp;
  static constexpr int kOffSc = kOffV + 2 * kOp;        // [4][8] float4: constants of 16 keys
  static constexpr int kOffBar = kOffSc + 4 * 8 * 16;
  static constexpr int kSmem = kOffBar + 256 + 1024;    // + alignment slack
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

// 32 columns of the warp's 32 TMEM lanes, without waiting.
__device__ __forceinline__ void tmem_ld_32cols_async(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// 16 columns, without waiting.
__device__ __forceinline__ void tmem_st_16cols_async(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t swz128(int row, int chunk) {  // 16-byte chunk of a 128-byte swizzled row
  return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
}

template <int D, int FMT, class T>
__global__ void __launch_bounds__(512, 1) paged_attn_tile_kernel(PagedAttnArgs a) {
  using C = TileCfg<D>;
  extern __shared__ uint8_t tile_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tile_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_full = bars;       // [2] converters -> S issuer
  uint64_t* k_free = bars + 2;   // [2] both tiles' S done
  uint64_t* v_full = bars + 4;   // [2] converters -> P V issuer
  uint64_t* v_free = bars + 6;   // [2] both tiles' P V done
  uint64_t* s_full = bars + 8;   // [tile] S ready; the issuer arrives beside its commit, ordering the constants
  uint64_t* p_full = bars + 10;  // [tile] weights in TMEM
  uint64_t* pv_done = bars + 12; // [tile] O current, S columns free
  uint64_t* q_full = bars + 14;  // [tile] Q rows staged
  uint64_t* drain = bars + 16;   // [2] an issuer's MMAs are done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 18);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float4* sc = reinterpret_cast<float4*>(smem + C::kOffSc);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.y, z = blockIdx.z;
  griddep_launch_dependents();
  griddep_wait();
  // the last rows of a causal prompt see the most keys: they start first
  const SeqItem it = find_item(a.q, static_cast<int>(gridDim.x - 1 - blockIdx.x), a.G, 8, 1);
  if (it.seq < 0 || it.n == 0) return;
  if (it.n < 0 || it.row0 < 0 || it.n > a.q.n_tok - it.row0) {
    if (threadIdx.x == 0) record_error(a.err, DEV_BAD_INDEX);
    return;
  }
  const int R = it.n * a.G;
  if (it.local >= (R + kRowsCta - 1) / kRowsCta) return;
  int len = a.q.kv_len[it.seq];
  if (len < 0 || len > kMaxLen || len > static_cast<int64_t>(a.q.table_stride) << a.c.page_log2) {
    if (threadIdx.x == 0) record_error(a.err, DEV_BAD_INDEX);
    len = 0;
  }
  const int r0 = it.local * kRowsCta;
  const int r_end = min(r0 + kRowsCta, R);
  const bool two = r_end - r0 > kTile;
  const int first = a.causal ? len - it.n + 1 : len;
  auto seen = [&](int r) { return max(0, a.causal ? first + r / a.G : len); };
  const int kmax = seen(r_end - 1);
  const int bl = (kmax + kBlock - 1) / kBlock;
  const int per = (bl + a.plan.n_splits - 1) / a.plan.n_splits;  // this item's blocks, in even ranges
  const int b0 = min(bl, z * per);
  const int nb = min(bl, b0 + per) - b0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], 128);
      mbar_init(&k_free[s], 1);
      mbar_init(&v_full[s], 128);
      mbar_init(&v_free[s], 1);
      mbar_init(&s_full[s], 2);
      mbar_init(&p_full[s], 128);
      mbar_init(&pv_done[s], 1);
      mbar_init(&q_full[s], 128);
      mbar_init(&drain[s], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const uint32_t col_o = 2 * kBlock;
  auto fail = [&](int code) {
    record_error(a.err, code);
    *abort_flag = 1;
  };

  if (warp < 4) {
    // ------------------------------------------------------------ MMA issuers
    regs_down<40>();
    if (warp < 2 && lane == 0 && nb > 0) {
      const bool is_s = warp == 0;
      constexpr uint32_t kIdS = idesc_f16_f32(kTile, kBlock);
      constexpr uint32_t kIdO = idesc_f16_f32(kTile, D) | (1u << 16);  // B (V) is MN-major
      bool ok = true;
      for (int i = 0; ok && i < nb; ++i) {
        const int st = i & 1;
        const uint32_t par = static_cast<uint32_t>((i >> 1) & 1);
        ok = mbar_wait(is_s ? &k_full[st] : &v_full[st], par, kWaitNs);
        for (int t = 0; ok && t < (two ? 2 : 1); ++t) {
          if (is_s) {
            if (i == 0) ok = mbar_wait(&q_full[t], 0, kWaitNs);
            else ok = mbar_wait(&pv_done[t], static_cast<uint32_t>((i - 1) & 1), kWaitNs);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t qa = smem_u32(smem + t * C::kOp), ka = smem_u32(smem + C::kOffK + st * C::kOp);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t o = (k >> 2) * kHalf + (k & 3) * 32;
              umma_f16(tbase + t * kBlock, sdesc_kmajor_sw128(qa + o), sdesc_kmajor_sw128(ka + o), kIdS, k > 0 ? 1u : 0u);
            }
            umma_commit(&s_full[t]);
            mbar_arrive(&s_full[t]);
          } else {
            ok = mbar_wait(&p_full[t], static_cast<uint32_t>(i & 1), kWaitNs);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t va = smem_u32(smem + C::kOffV + st * C::kOp);
#pragma unroll
            for (int k = 0; k < kBlock / 16; ++k)
              umma_f16_ts(tbase + col_o + t * D, tbase + t * kBlock + k * 8,
                          sdesc_mnmajor_sw128(va + k * 16 * 128, kHalf, 1024), kIdO, (i > 0 || k > 0) ? 1u : 0u);
            umma_commit(&pv_done[t]);
          }
        }
        if (ok) umma_commit(is_s ? &k_free[st] : &v_free[st]);
        if (*abort_flag) ok = false;
      }
      if (!ok) fail(DEV_WAIT_TIMEOUT_MMA);
      umma_commit(&drain[warp]);  // every MMA of this thread ends before TMEM is released
      if (!mbar_wait(&drain[warp], 0, kDrainWaitNs)) record_error(a.err, DEV_WAIT_TIMEOUT_DRAIN);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ codes -> fp16
    // Thread -> rows (tid / 4 mod 8) + 8 j, chunk (tid mod 4): eight rows of one chunk make a store phase.
    regs_down<88>();
    const int tid = threadIdx.x - 128;
    constexpr int kCh = D / 16;             // 16-code chunks of a row
    constexpr int kPer = kBlock * kCh / 128;  // chunks of a thread: 8 or 4
    const int32_t* tab = a.q.table + static_cast<int64_t>(it.seq) * a.q.table_stride;
    const int last_page = (len - 1) >> a.c.page_log2;
    auto where = [&](int j, int* row, int* ch) {  // chunk j of this thread
      const int x = j * 128 + tid;
      *row = ((x >> 5) / (kCh / 4)) * 8 + ((x >> 2) & 7);
      *ch = ((x >> 5) % (kCh / 4)) * 4 + (x & 3);
    };
    auto load = [&](const uint8_t* base, int b, uint4* v) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        int row, ch;
        where(j, &row, &ch);
        const int key = b * kBlock + row;
        const int pg = key >> a.c.page_log2;
        const int id = key < len ? tab[pg] : -1;  // slots behind the last token read as zeros, whatever they hold
        v[j] = make_uint4(0u, 0u, 0u, 0u);
        if (id >= 0 && id < a.c.n_pages)
          v[j] = *reinterpret_cast<const uint4*>(base + id * a.c.page_stride + hk * a.c.head_stride +
                                                 (key & ((1 << a.c.page_log2) - 1)) * a.c.tok_stride + ch * 16);
      }
    };
    auto store = [&](uint8_t* dst, const uint4* v) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        int row, ch;
        where(j, &row, &ch);
        const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        uint32_t h[8];
#pragma unroll
        for (int x = 0; x < 4; ++x) codes4_half<FMT>(w[x], &h[2 * x], &h[2 * x + 1]);
        uint8_t* p = dst + (ch >> 2) * kHalf;
        const int c8 = (ch & 3) * 2;
        *reinterpret_cast<uint4*>(p + swz128(row, c8)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(p + swz128(row, c8 + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
      }
    };
    // constants of 16 keys: K scale, log2 and reciprocal of the V scale, seen or not
    auto constants = [&](int i) {
      if (tid < kBlock / 16) {
        const int pg = ((b0 + i) * kBlock + tid * 16) >> a.c.page_log2;
        float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
        if (pg <= last_page) {
          const int id = tab[pg];
          if (id >= 0 && id < a.c.n_pages) {
            float v = a.c.vs[static_cast<int64_t>(id) * a.c.Hkv + hk];
            if (v < kScaleFloor) v = kScaleFloor;  // a NaN stays
            c = make_float4(a.c.ks[static_cast<int64_t>(id) * a.c.Hkv + hk], lg2(v), 1.f / v, 1.f);
          } else {
            record_error(a.err, DEV_BAD_INDEX);
          }
        }
        sc[(i & 3) * 8 + tid] = c;
      }
    };
    uint4 kv[kPer], vv[kPer];
    bool ok = true;
    if (nb > 0) load(a.c.k, b0, kv);
    for (int i = 0; i < nb; ++i) {
      const int st = i & 1;
      const uint32_t par = static_cast<uint32_t>(((i - 2) >> 1) & 1);
      load(a.c.v, b0 + i, vv);
      if (i >= 2) ok = mbar_wait(&k_free[st], par, kWaitNs);
      ok = __all_sync(0xffffffffu, ok && !*abort_flag);
      if (!ok) break;
      constants(i);  // slot i mod 4: block i - 4 left the softmax before v_free of block i - 3
      store(smem + C::kOffK + st * C::kOp, kv);
      fence_proxy_async_smem();
      mbar_arrive(&k_full[st]);
      if (i + 1 < nb) load(a.c.k, b0 + i + 1, kv);
      if (i >= 2) ok = mbar_wait(&v_free[st], par, kWaitNs);
      ok = __all_sync(0xffffffffu, ok && !*abort_flag);
      if (!ok) break;
      store(smem + C::kOffV + st * C::kOp, vv);
      fence_proxy_async_smem();
      mbar_arrive(&v_full[st]);
    }
    if (!ok && lane == 0) fail(DEV_WAIT_TIMEOUT_PRODUCER);
  } else {
    // ------------------------------------------------------------ softmax rows
    regs_up<192>();
    const int t = (warp - 8) >> 2;
    const int rt = 32 * (warp & 3) + lane;  // row of the tile = TMEM lane
    const int r = r0 + t * kTile + rt;
    const bool active = t == 0 || two;
    const bool valid = r < r_end;
    const int rr = min(r, r_end - 1);
    const int tok = it.row0 + rr / a.G, hq = hk * a.G + rr % a.G;
    const int vis = seen(rr);
    const uint32_t trow = tbase + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t ts = trow + t * kBlock, to = trow + col_o + t * D;
    float m_ref = -INFINITY, l = 0.f, qs = 0.f;
    bool ok = active;
    if (active && nb > 0) {
      // ---- this row of Q, as fp16 (bf16 rows scaled by a power of two)
      const T* src = static_cast<const T*>(a.x) + tok * a.x_tok + hq * a.x_head;
      const bool wide = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
      auto eight = [&](int c, T* v) {
        if (wide) {
          *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(src + 8 * c);
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x) v[x] = src[8 * c + x];
        }
      };
      uint32_t am = 0;
      if (!std::is_same<T, __half>::value) {
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          alignas(16) T v[8];
          eight(c, v);
#pragma unroll
          for (int x = 0; x < 8; ++x) am = max(am, __float_as_uint(to_f(v[x])) & 0x7fffffffu);
        }
      }
      float down;
      qs = row_power<T>(am, &down) * a.scale_log2;
      uint8_t* q = smem + t * C::kOp;
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        alignas(16) T v[8];
        eight(c, v);
        uint32_t w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          w[x] = valid ? pack2(to_f(v[2 * x]) * down, to_f(v[2 * x + 1]) * down) : 0u;
        *reinterpret_cast<uint4*>(q + (c >> 3) * kHalf + swz128(rt, c & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(&q_full[t]);
      const int wmin = __reduce_min_sync(0xffffffffu, vis);  // keys that every row of the warp sees
      for (int i = 0; i < nb; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], static_cast<uint32_t>(i & 1), kWaitNs) && !*abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        float s[kBlock];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32cols_async(ts + 32 * c, s + 32 * c);
        const float4* cs = sc + (i & 3) * 8;
        tmem_ld_wait();
        const int j0 = (b0 + i) * kBlock;
        bool plain = j0 + kBlock <= wmin;
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 k = cs[g];
          plain = plain && k.w != 0.f;
          float m = s[16 * g];
#pragma unroll
          for (int e = 1; e < 16; ++e) m = fmaxf(m, s[16 * g + e]);
          mx = fmaxf(mx, fmaf(m, qs * k.x, k.y));
        }
        if (!plain) {
          // some key of the block is hidden from some row: x in place of S, -inf where hidden
          mx = -INFINITY;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const float4 k = cs[g];
            const float ak = qs * k.x;
            const int lim = k.w != 0.f ? vis - j0 - 16 * g : 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              s[16 * g + e] = e < lim ? fmaf(s[16 * g + e], ak, k.y) : -INFINITY;
              mx = fmaxf(mx, s[16 * g + e]);
            }
          }
        }
        if (__any_sync(0xffffffffu, mx > m_ref + kSlackTc)) {
          const float m_new = fmaxf(m_ref, mx);
          const float f = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - m_new);
          if (i > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[t], static_cast<uint32_t>((i - 1) & 1), kWaitNs));
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              asm volatile(
                  "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                  "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                  : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]),
                    "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
                  : "r"(to + 16 * c));
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tmem_st_16cols_async(to + 16 * c, o);
            }
            tmem_st_wait();
          }
          l *= f;
          m_ref = m_new;
        }
        const float mb = (m_ref == -INFINITY ? 0.f : m_ref) - kBias;
#pragma unroll
        for (int q2 = 0; q2 < 4; ++q2) {
          uint32_t w[16];
#pragma unroll
          for (int g = 2 * q2; g < 2 * q2 + 2; ++g) {
            const float4 k = cs[g];
            const float ak = plain ? qs * k.x : 1.f, bk = (plain ? k.y : 0.f) - mb;
            float l0 = 0.f, l1 = 0.f;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float p0 = ex2_approx(fmaf(s[16 * g + e], ak, bk));
              const float p1 = ex2_approx(fmaf(s[16 * g + e + 1], ak, bk));
              l0 += p0;
              l1 += p1;
              w[(g & 1) * 8 + e / 2] = pack2(p0, p1);
            }
            // a poisoned scale (NaN) counts only for rows that see its keys
            l = fmaf(l0 + l1, plain || vis > j0 + 16 * g ? k.z : 0.f, l);
          }
          tmem_st_16cols_async(ts + 16 * q2, w);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&p_full[t]);
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[t], static_cast<uint32_t>((nb - 1) & 1), kWaitNs) && !*abort_flag);
      if (!ok && lane == 0) fail(DEV_WAIT_TIMEOUT_EPILOGUE);
      tc_fence_after_sync();
    }
    // ---- out = O / l, or the state of this key range
    const bool have = ok && nb > 0;
    const bool split = a.plan.n_splits > 1;
    const int64_t prow = (static_cast<int64_t>(z) * a.q.n_tok + tok) * a.Hq + hq;
    T* out = static_cast<T*>(a.out) + tok * a.out_tok + hq * a.out_head;
    const float il = l == 0.f ? 0.f : 1.f / l;
    if (active) {
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        if (have) {
          tmem_ld_32cols_async(to + 32 * c, o);
          tmem_ld_wait();
        }
        __syncwarp();
        if (valid && split && have && l != 0.f) {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            *reinterpret_cast<float4*>(a.part_o + prow * D + 32 * c + 4 * x) =
                make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        } else if (valid && !split) {
          const bool some = have && l != 0.f;
          if ((reinterpret_cast<uintptr_t>(out) & 15) == 0) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              alignas(16) T y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = from_f<T>(some ? o[8 * x + e] * il : 0.f);
              *reinterpret_cast<uint4*>(out + 32 * c + 8 * x) = *reinterpret_cast<const uint4*>(y);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) out[32 * c + x] = from_f<T>(some ? o[x] * il : 0.f);
          }
        }
        __syncwarp();
      }
      if (valid) {
        if (split) a.part_ml[prow] = make_float2(m_ref, l);
        else if (a.lse)
          a.lse[static_cast<int64_t>(tok) * a.Hq + hq] =
              l == 0.f ? -INFINITY : (m_ref - kBias + log2f(l)) * 0.6931471805599453f;
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, int FMT, class T>
int launch_tile(const PagedAttnArgs& a, cudaStream_t s) {
  using C = TileCfg<D>;
  auto kern = paged_attn_tile_kernel<D, FMT, T>;
  static KernelSetup setup;
  const cudaError_t r = setup.run(kern, C::kSmem);
  if (r != cudaSuccess) return r;
  const int64_t items = ((static_cast<int64_t>(a.q.n_tok) * a.G) >> 8) + a.q.n_seq;
  return launch_k(kern, dim3(static_cast<unsigned>(items), static_cast<unsigned>(a.c.Hkv), static_cast<unsigned>(a.plan.n_splits)),
                  dim3(512), C::kSmem, s, a);
}
template <int D, int FMT>
int launch_tile_t(const PagedAttnArgs& a, cudaStream_t s) {
  return a.dtype == PCD_DTYPE_BF16 ? launch_tile<D, FMT, __nv_bfloat16>(a, s) : launch_tile<D, FMT, __half>(a, s);
}

}  // namespace

int launch_paged_attention_tiles(const PagedAttnArgs& a, cudaStream_t s) {
  const bool f8 = a.c.format == PCD_KV_E4M3;
  if (a.c.dim == 64) return f8 ? launch_tile_t<64, PCD_KV_E4M3>(a, s) : launch_tile_t<64, PCD_KV_INT8>(a, s);
  return f8 ? launch_tile_t<128, PCD_KV_E4M3>(a, s) : launch_tile_t<128, PCD_KV_INT8>(a, s);
}

}  // namespace pcd
