// Attention over the 8-bit paged cache for many query rows, on the
// 5th-generation tensor cores.
//
// A CTA owns 256 query rows of one sequence and KV head (rows are tokens x
// the G query heads, flattened) as two tiles of 128 and walks key blocks of
// 128:
//   codes to shared memory     bulk copies, one warp
//   codes -> fp16, exactly     four warps, into 128-byte swizzled operand tiles
//   S = Q K^T                  tcgen05.mma, 128 x 128, accumulator in TMEM
//   w = exp2(S sk c + log2 sv - M + 8)   one thread a row
//   O += w V8                  tcgen05.mma, w (fp16) from TMEM over S's columns
//   l += w / sv                so out = O / l (see the rows kernel)
// Each K and V block is converted once for both tiles.  M moves, and O and l
// are rescaled, only when a block exceeds it by 2^7.
//
// TMEM's 512 columns at head dim 128: S (then the weights over its first half)
// and O of both tiles.  The tiles' MMA issuers take turns (P V, then S of the
// tile's next block, whose columns P V has to free): while one tile's rows are in
// the softmax the tensor cores work for the other.  At head dim 64 the weights
// have columns of their own, so S of the next block is made as soon as the
// softmax holds the present scores, and its threads never wait for the MMAs.
//
// An item of one tile only (33 to 128 rows) gives its even and odd key blocks to
// the two pipelines instead, with the second Q tile's place for codes of odd
// blocks, and joins their states at the end.  64 sequences of 56 rows over 8 k
// keys: 241 us against 274 (one pipeline).  Kernels for more rows are compiled
// without it: its registers cost them 2%.
//
// Measured: 2 x 2048 tokens of 28 heads at the end of 8 k keys 372 us, 1130
// TFLOP/s (bf16 387), bound by the chain of a tile's block (softmax 1900 clocks, P V 550, S
// 600, four hand-offs of about 200); 9 prompts of heads of 64, 56 us.  An item's
// start and end take some 15 k clocks: 2.3 to find its work, 4 to the first
// converted K block with Q staged beside it, 2 to the first scores, 5 for the
// output, 2 to the next CTA's entry.
//
// Registers: 512 threads launch with 128 each; the two softmax warpgroups
// hold a row of 128 scores and take 192, paid for by the other two (64 each):
// 64 + 64 + 192 + 192 = 4 x 128.
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
static_assert(kRowsCta == kTileRows, "rows of an item");
constexpr int kBlock = 128;       // keys of a block (MMA N of S, K of P V)
constexpr int kHalf = kTile * 128;  // bytes of 64 channels x 128 rows, one 128-byte swizzled row each
constexpr float kSlackTc = 7.f;

template <int D>
struct TileCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kOp = kHalves * kHalf;           // one operand tile: 128 rows x D fp16
  static constexpr int kOffK = 2 * kOp;                 // after the two Q tiles
  static constexpr int kOffV = kOffK + 2 * kOp;
  static constexpr int kRaw = kBlock * D;               // a block's K or V codes
  static constexpr int kOffRaw = kOffV + 2 * kOp;       // K's, then V's
  static constexpr int kOffSc = kOffRaw + 2 * kRaw;     // [8][8] float4: constants of 16 keys
  static constexpr int kOffWhole = kOffSc + 8 * 8 * 16;  // [8]: is every key of the block there?
  static constexpr int kOffBar = kOffWhole + 32;
  static constexpr int kSmem = kOffBar + 256 + 1024;    // + alignment slack
  static constexpr bool kOwnP = D == 64;                // the weights' columns: their own, or S's
  static constexpr int kColO = 2 * kBlock, kColP = kOwnP ? kColO + 2 * D : 0, kStepP = kOwnP ? kBlock / 2 : kBlock;
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
// Waits for the loads issued so far; 32 of their values pass through, so that
// nothing uses them before.
__device__ __forceinline__ void tmem_ld_wait32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
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
// Bulk copy of `bytes` (a multiple of 16, both addresses 16-byte aligned) to shared memory.
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
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

template <int D, int FMT, class T, bool ALT>
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
  uint64_t* turn = bars + 16;    // [tile] its issuer's turn
  uint64_t* drain = bars + 18;   // [tile] its issuer's MMAs are done
  uint64_t* s_free = bars + 20;  // [tile] scores are in the softmax's registers (weights with columns of their own)
  uint64_t* raw_full = bars + 22;  // [K, V; K, V of odd blocks] codes landed, constants written
  uint64_t* raw_free = bars + 26;  // ... codes converted
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 30);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float4* sc = reinterpret_cast<float4*>(smem + C::kOffSc);
  volatile int* whole_block = reinterpret_cast<volatile int*>(smem + C::kOffWhole);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.y, z = blockIdx.z;
  griddep_launch_dependents();
  griddep_wait();
  const OffsetCheck offsets(a.q);
  const SeqItem it = find_item(a.q, static_cast<int>(blockIdx.x), a.G, kTileRowsLog, 1);
  offsets.report(a.q, a.err);
  if (it.seq < 0 || it.n == 0) return;
  if (it.n < 0 || it.row0 < 0 || it.n > a.q.n_tok - it.row0) {
    if (threadIdx.x == 0) record_error(a.err, DEV_BAD_INDEX);
    return;
  }
  const int R = it.n * a.G;
  const int tiles = (R + kRowsCta - 1) / kRowsCta;
  if (it.local >= tiles) return;
  int len = it.len;
  if (len < 0 || len > kMaxLen || len > static_cast<int64_t>(a.q.table_width) << a.c.page_log2) {
    if (threadIdx.x == 0) record_error(a.err, DEV_BAD_INDEX);
    len = 0;
  }
  const int r0 = (tiles - 1 - it.local) * kRowsCta;  // the last rows of a causal prompt see the most keys: they start first
  const int r_end = min(r0 + kRowsCta, R);
  const bool two = r_end - r0 > kTile;
  const int first = a.causal ? len - it.n + 1 : len;
  auto seen = [&](int r) { return max(0, a.causal ? first + r / a.G : len); };
  const int kmax = seen(r_end - 1);
  const int bl = (kmax + kBlock - 1) / kBlock;
  const int per = (bl + a.plan.n_splits - 1) / a.plan.n_splits;  // this item's blocks, in even ranges
  const int b0 = min(bl, z * per);
  const int nb = min(bl, b0 + per) - b0;
  // One tile of rows: both pipelines take it, the even blocks and the odd ones.
  // Block i is then pipeline i & 1's, stage i & 1 belongs to it alone, and the
  // second Q tile's place holds the codes of odd blocks.
  const bool alt = ALT && !two && nb > 1;
  auto raw_at = [&](int i, int kv) { return smem + (alt && (i & 1) ? C::kOp : C::kOffRaw) + kv * C::kRaw; };
  auto raw_bar = [&](int i, int kv) { return alt && (i & 1) ? kv + 2 : kv; };
  auto raw_par = [&](int i) { return static_cast<uint32_t>((alt ? i >> 1 : i) & 1); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_free[s], two ? 2 : 1);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_free[s], two ? 2 : 1);
      mbar_init(&s_full[s], 2);
      mbar_init(&p_full[s], 4);
      mbar_init(&pv_done[s], 1);
      mbar_init(&q_full[s], 4);
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_full[s + 2], 1);
      mbar_init(&turn[s], 1);
      mbar_init(&s_free[s], 4);
      mbar_init(&drain[s], 1);
      mbar_init(&raw_free[s], 4);
      mbar_init(&raw_free[s + 2], 4);
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
  auto fail = [&](int code) {
    record_error(a.err, code);
    *abort_flag = 1;
  };

  const int last_page = (len - 1) >> a.c.page_log2;
  int raw_issued = 0;  // blocks whose K (and V) copies were issued, by the copying warp

  if (warp < 4) {
    regs_down<64>();
    if ((warp == 0 || (warp == 2 && (two || alt))) && nb > 0) {
      // ------------------------------------------------------------ MMA issuers, one a tile
      // A warp stays together and one lane issues, so that descriptors are
      // computed in uniform registers (a lone lane took 20 more clocks an MMA).
      constexpr uint32_t kIdS = idesc_f16_f32(kTile, kBlock);
      constexpr uint32_t kIdO = idesc_f16_f32(kTile, D) | (1u << 16);  // B (V) is MN-major
      const int t = __shfl_sync(0xffffffffu, warp >> 1, 0);
      const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
      const uint32_t dS = tb + t * kBlock, dO = tb + C::kColO + t * D;
      const uint64_t dq = sdesc_kmajor_sw128(smem_u32(smem + (alt ? 0 : t * C::kOp))), dk = sdesc_kmajor_sw128(smem_u32(smem + C::kOffK));
      const uint64_t dv = sdesc_mnmajor_sw128(smem_u32(smem + C::kOffV), kHalf, 1024);
      auto issue_s = [&](int st) {
        tc_fence_after_sync();
        const uint64_t k0 = dk + st * (C::kOp >> 4);
        if (elect_one_sync()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
            umma_f16(dS, dq + o, k0 + o, kIdS, k > 0 ? 1u : 0u);
          }
          if (two && !C::kOwnP) mbar_arrive(&turn[t ^ 1]);
          umma_commit(&s_full[t]);
          mbar_arrive(&s_full[t]);  // orders the constants, which the commit alone would not
          umma_commit(&k_free[st]);
        }
        __syncwarp();
      };
      // turn[t] completes once before each of the tile's turns; the first tile's first turn is free
      const int step = alt ? 2 : 1, i0 = alt ? t : 0;
      bool ok = mbar_wait(&k_full[i0], 0, a.wait_ns) && mbar_wait(&q_full[alt ? 0 : t], 0, a.wait_ns) &&
                (t == 0 || alt || C::kOwnP || mbar_wait(&turn[1], 0, a.wait_ns));
      ok = __all_sync(0xffffffffu, ok);
      if (ok) issue_s(i0);
      const uint32_t dP = C::kOwnP ? tb + C::kColP + t * C::kStepP : dS;
      for (int i = i0; ok && i < nb; i += step) {
        const int st = i & 1;
        const uint32_t par = static_cast<uint32_t>((alt ? i >> 1 : i) & 1);
        auto next_s = [&](uint64_t* freed) {
          const int in = i + step;
          if (in >= nb) return;
          ok = mbar_wait(&k_full[in & 1], static_cast<uint32_t>((in >> 1) & 1), a.wait_ns) && mbar_wait(freed, par, a.wait_ns);
          ok = __all_sync(0xffffffffu, ok && !*abort_flag);
          if (ok) issue_s(in & 1);
        };
        if (C::kOwnP) next_s(&s_free[t]);
        if (!ok) break;
        ok = mbar_wait(&v_full[st], static_cast<uint32_t>((i >> 1) & 1), a.wait_ns) &&
             (!two || C::kOwnP || mbar_wait(&turn[t], static_cast<uint32_t>((i + t) & 1), a.wait_ns)) &&
             mbar_wait(&p_full[t], par, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        const uint64_t v = dv + st * (C::kOp >> 4);
        const uint32_t acc = i > i0 ? 1u : 0u;
        if (elect_one_sync()) {
#pragma unroll
          for (int k = 0; k < kBlock / 16; ++k)
            umma_f16_ts(dO, dP + k * 8, v + k * (16 * 128 >> 4), kIdO, k > 0 ? 1u : acc);
          umma_commit(&pv_done[t]);
          umma_commit(&v_free[st]);
          if (two && !C::kOwnP && i + 1 == nb) mbar_arrive(&turn[t ^ 1]);
        }
        __syncwarp();
        if (!C::kOwnP) next_s(&pv_done[t]);  // S takes the columns that P V reads its weights from
      }
      if (!ok && lane == 0) fail(DEV_WAIT_TIMEOUT_MMA);
      if (elect_one_sync()) {
        umma_commit(&drain[t]);  // every MMA ends before TMEM is released
        if (!mbar_wait(&drain[t], 0, kDrainWaitNs)) record_error(a.err, DEV_WAIT_TIMEOUT_DRAIN);
      }
    } else if (warp == 1 && nb > 0) {
      // ------------------------------------------------------------ copies of codes, constants of keys
      const int32_t* tab = a.q.table + static_cast<int64_t>(it.seq) * a.q.table_stride;
      const int page = 1 << a.c.page_log2, npg = kBlock >> a.c.page_log2;
      const bool rows_together = a.c.tok_stride == D;
      auto fetch = [&](int b) {  // the page of lane l of block b
        const int pg = (b << 7 >> a.c.page_log2) + lane;
        return lane < npg && pg <= last_page ? tab[pg] : -1;
      };
      // Ids are fetched two blocks ahead and scales one, so that no copy waits for them.
      int id_next = fetch(b0), id_after = fetch(b0 + 1);
      bool there_next;
      float ks_next, vs_next;
      auto fetch_scales = [&](int b, int id) {  // 16 keys of block b to a lane
        const int cid = __shfl_sync(0xffffffffu, id >= 0 && id < a.c.n_pages ? id : -1, (lane * 16 >> a.c.page_log2) & 31);
        there_next = lane < kBlock / 16 && cid >= 0 && b * kBlock + lane * 16 < len;
        const int64_t at = static_cast<int64_t>(there_next ? cid : 0) * a.c.Hkv + hk;
        ks_next = a.c.ks[at];
        vs_next = a.c.vs[at];
      };
      fetch_scales(b0, id_next);
      bool ok = true;
      for (int i = 0; i < nb && ok; ++i) {
        const int id = id_next, j0 = (b0 + i) * kBlock;
        const bool there = there_next;
        const float k_scale = ks_next;
        float v_scale = vs_next;
        id_next = id_after;
        id_after = fetch(b0 + i + 2);
        fetch_scales(b0 + i + 1, id_next);
        const bool good = id >= 0 && id < a.c.n_pages;
        if (lane < npg && j0 + lane * page < len && !good) record_error(a.err, DEV_BAD_INDEX);
        const int rows = good ? min(page, len - j0 - lane * page) : 0;
        const uint32_t total = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(rows) * D);
        const int64_t off = (good ? id : 0) * a.c.page_stride + hk * a.c.head_stride;
#pragma unroll 1
        for (int kv = 0; kv < 2 && ok; ++kv) {
          const int before = i - (alt ? 2 : 1);  // the block whose codes were here
          if (before >= 0) ok = mbar_wait(&raw_free[raw_bar(before, kv)], raw_par(before), a.wait_ns);
          ok = __all_sync(0xffffffffu, ok && !*abort_flag);
          if (!ok) break;
          const uint8_t* base = kv ? a.c.v : a.c.k;
          uint8_t* raw = raw_at(i, kv);
          uint64_t* full = &raw_full[raw_bar(i, kv)];
          if (kv == 0) {
            // K scale, log2 and reciprocal of the V scale, seen or not
            const uint32_t all = __ballot_sync(0xffffffffu, there) & 0xffu;
            // block i - 8 has left the softmax: K of block i - 2 at least was converted, after V of blocks i - 3
            // and i - 4, for which the P V of blocks i - 5 and i - 6 were done
            if (lane < kBlock / 16) {
              float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
              if (there) {
                if (v_scale < kScaleFloor) v_scale = kScaleFloor;  // a NaN stays
                c = make_float4(k_scale, lg2(v_scale), 1.f / v_scale, 1.f);
              }
              sc[(i & 7) * 8 + lane] = c;
              if (lane == 0) whole_block[i & 7] = all == 0xffu && len - j0 >= kBlock;
            }
            __syncwarp();
          }
          if (lane == 0) mbar_arrive_expect_tx(full, total);
          __syncwarp();
          if (rows_together) {
            if (rows > 0) bulk_g2s(raw + lane * page * D, base + off, rows * D, full);
          } else {
            for (int p = 0; p < npg; ++p) {
              const int n = __shfl_sync(0xffffffffu, rows, p);
              const int64_t o = __shfl_sync(0xffffffffu, off, p);
              for (int r = lane; r < n; r += 32)
                bulk_g2s(raw + (p * page + r) * D, base + o + r * a.c.tok_stride, D, full);
            }
          }
          raw_issued = 2 * i + kv + 1;
        }
      }
      if (!ok && lane == 0) fail(DEV_WAIT_TIMEOUT_PRODUCER);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ codes -> fp16
    // Eight lanes read 128 bytes of a row pair and write 8 different 16-byte
    // places of the swizzled rows: at D 128 lanes 0-3 take the first half of one
    // row and lanes 4-7 the second half of the other, whose XOR differs in its last bit.
    regs_down<64>();
    const int tid = threadIdx.x - 128, q8 = lane & 7, ph = lane >> 3;
    constexpr int kPer = kBlock * D / 16 / 128;  // 16-code chunks of a thread: 8 or 4
    constexpr int kStep = kBlock / kPer;         // rows between them
    const int row0 = D == 128 ? (((tid >> 5) * 2 + (ph >> 1)) * 2 + ((q8 >> 2) ^ (ph & 1))) : ((tid >> 3) * 2 + (q8 >> 2));
    const int ch = D == 128 ? q8 : (q8 & 3);
    const int raw0 = row0 * D + ch * 16;
    const uint32_t dst0 = (ch >> 2) * kHalf + swz128(row0, (ch & 3) * 2), dst1 = (ch >> 2) * kHalf + swz128(row0, (ch & 3) * 2 + 1);
    bool ok = true;
    for (int i = 0; i < nb && ok; ++i) {
      const int st = i & 1;
      const int live = min(kBlock, len - (b0 + i) * kBlock);  // rows behind the last token read as zeros
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        ok = mbar_wait(&raw_full[raw_bar(i, kv)], raw_par(i), a.wait_ns);
        if (ok && i >= 2) ok = mbar_wait(kv ? &v_free[st] : &k_free[st], static_cast<uint32_t>(((i - 2) >> 1) & 1), a.wait_ns);
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        const bool whole = whole_block[i & 7] != 0;
        const uint8_t* src = raw_at(i, kv) + raw0;
        uint8_t* dst = smem + (kv ? C::kOffV : C::kOffK) + st * C::kOp;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          uint4 v = *reinterpret_cast<const uint4*>(src + j * kStep * D);
          if (!whole) {
            const int row = row0 + j * kStep;
            if (row >= live || sc[(i & 7) * 8 + (row >> 4)].w == 0.f) v = make_uint4(0u, 0u, 0u, 0u);
          }
          uint32_t h[8];
          codes4_half<FMT>(v.x, &h[0], &h[1]);
          codes4_half<FMT>(v.y, &h[2], &h[3]);
          codes4_half<FMT>(v.z, &h[4], &h[5]);
          codes4_half<FMT>(v.w, &h[6], &h[7]);
          // kStep is a multiple of 8: the swizzle of row0 holds for its other rows
          *reinterpret_cast<uint4*>(dst + dst0 + j * kStep * 128) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + dst1 + j * kStep * 128) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(kv ? &v_full[st] : &k_full[st]);
          mbar_arrive(&raw_free[raw_bar(i, kv)]);
        }
      }
    }
    if (!ok && lane == 0) fail(DEV_WAIT_TIMEOUT_PRODUCER);
  } else {
    // ------------------------------------------------------------ softmax rows
    regs_up<192>();
    const int t = (warp - 8) >> 2;
    const int rt = 32 * (warp & 3) + lane;  // row of the tile = TMEM lane
    const int r = r0 + (alt ? 0 : t * kTile) + rt;
    const bool active = t == 0 || two || alt;
    const bool valid = r < r_end;
    const int rr = min(r, r_end - 1);
    const int tok = it.row0 + rr / a.G, hq = hk * a.G + rr % a.G;
    const int vis = seen(rr);
    const uint32_t trow = tbase + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t ts = trow + t * kBlock, tp = C::kOwnP ? trow + C::kColP + t * C::kStepP : ts, to = trow + C::kColO + t * D;
    float m_ref = -INFINITY, l = 0.f, qs = 0.f;
    bool ok = active;
    if (active && nb > 0) {
      // ---- the warp's 32 rows of Q, as fp16 (bf16 rows scaled by a power of two): D / 8 lanes to a row,
      // every load in flight at once
      constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // rows of one load
      const int64_t mine = tok * a.x_tok + hq * a.x_head;
      const int c = lane % kLanes;
      // (bf16 as whole words from either branch: elements, which their maxima want, would be taken apart where the
      // branches meet, so that each load waited for the one before: 18 k clocks of a tile's start, now 8 k.  fp16
      // words pass through untouched; loaded the other way their key loop came out 3% slower.)
      uint4 v[32 / kAt];
      if constexpr (std::is_same<T, __half>::value) {
        alignas(16) T h[32 / kAt][8];
#pragma unroll
        for (int j = 0; j < 32 / kAt; ++j) {
          const T* src = static_cast<const T*>(a.x) + __shfl_sync(0xffffffffu, mine, j * kAt + lane / kLanes) + 8 * c;
          if (((reinterpret_cast<uintptr_t>(a.x) | static_cast<uint64_t>(a.x_tok | a.x_head) * 2) & 15) == 0) {
            *reinterpret_cast<uint4*>(h[j]) = *reinterpret_cast<const uint4*>(src);
          } else {
#pragma unroll
            for (int x = 0; x < 8; ++x) h[j][x] = src[x];
          }
        }
#pragma unroll
        for (int j = 0; j < 32 / kAt; ++j) v[j] = *reinterpret_cast<const uint4*>(h[j]);
      } else if (((reinterpret_cast<uintptr_t>(a.x) | static_cast<uint64_t>(a.x_tok | a.x_head) * 2) & 15) == 0) {
#pragma unroll
        for (int j = 0; j < 32 / kAt; ++j)
          v[j] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) +
                                                 __shfl_sync(0xffffffffu, mine, j * kAt + lane / kLanes) + 8 * c);
      } else {
#pragma unroll 1
        for (int j = 0; j < 32 / kAt; ++j) {
          const uint16_t* src = static_cast<const uint16_t*>(a.x) + __shfl_sync(0xffffffffu, mine, j * kAt + lane / kLanes) + 8 * c;
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) w[x] = src[2 * x] | static_cast<uint32_t>(src[2 * x + 1]) << 16;
#pragma unroll
          for (int k = 0; k < 32 / kAt; ++k)
            if (k == j) v[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      uint8_t* q = smem + t * C::kOp + (c >> 3) * kHalf;
      qs = 1.f;
      if (!std::is_same<T, __half>::value) {  // all rows' maxima side by side: one chain of shuffles, not one a row
        uint32_t am[32 / kAt];
#pragma unroll
        for (int j = 0; j < 32 / kAt; ++j) {
          const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
          am[j] = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) am[j] = max(am[j], max(w[x] << 16 & 0x7fffffffu, w[x] & 0x7fff0000u));
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
          for (int j = 0; j < 32 / kAt; ++j) am[j] = max(am[j], __shfl_xor_sync(0xffffffffu, am[j], o));
#pragma unroll
        for (int j = 0; j < 32 / kAt; ++j) {
          float down;
          const float u = __shfl_sync(0xffffffffu, row_power<T>(am[j], &down), (lane % kAt) * kLanes);
          if (lane / kAt == j) qs = u;
          uint32_t* w = reinterpret_cast<uint32_t*>(&v[j]);
#pragma unroll
          for (int x = 0; x < 4; ++x)  // bf16 are the upper halves of fp32
            w[x] = pack2(__uint_as_float(w[x] << 16) * down, __uint_as_float(w[x] & 0xffff0000u) * down);
        }
      }
      if (!alt || t == 0) {  // the first pipeline stages a tile that both take
#pragma unroll
        for (int j = 0; j < 32 / kAt; ++j) {
          const int row = 32 * (warp & 3) + j * kAt + lane / kLanes;
          const bool in = r0 + t * kTile + row < r_end;  // rows behind the last are zeros
          *reinterpret_cast<uint4*>(q + swz128(row, c & 7)) = in ? v[j] : make_uint4(0u, 0u, 0u, 0u);
        }
      }
      qs *= a.scale_log2;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[t]);
      const int wmin = __reduce_min_sync(0xffffffffu, vis);  // keys that every row of the warp sees
      int n = 0;  // blocks done
      for (int i = alt ? t : 0; i < nb; i += alt ? 2 : 1, ++n) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], static_cast<uint32_t>(n & 1), a.wait_ns) && !*abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        float s[kBlock];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32cols_async(ts + 32 * c, s + 32 * c);
        const float4* cs = sc + (i & 7) * 8;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait32(s + 32 * c);
        if (C::kOwnP) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[t]);
        }
        const int j0 = (b0 + i) * kBlock;
        const bool plain = whole_block[i & 7] != 0 && j0 + kBlock <= wmin;
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 k = cs[g];
          float m = max3(s[16 * g], s[16 * g + 1], s[16 * g + 2]), m1 = max3(s[16 * g + 3], s[16 * g + 4], s[16 * g + 5]);
#pragma unroll
          for (int e = 6; e < 14; e += 4) {
            m = max3(m, s[16 * g + e], s[16 * g + e + 1]);
            m1 = max3(m1, s[16 * g + e + 2], s[16 * g + e + 3]);
          }
          m = max3(m, s[16 * g + 14], s[16 * g + 15]);
          mx = fmaxf(mx, fmaf(fmaxf(m, m1), qs * k.x, k.y));
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
          if (n > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[t], static_cast<uint32_t>((n - 1) & 1), a.wait_ns));
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tmem_ld_32cols_async(to + 32 * c, o);
              tmem_ld_wait32(o);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] *= f;
              tmem_st_16cols_async(to + 32 * c, reinterpret_cast<const uint32_t*>(o));
              tmem_st_16cols_async(to + 32 * c + 16, reinterpret_cast<const uint32_t*>(o) + 16);
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
            const float2 a2 = make_float2(ak, ak), b2 = make_float2(bk, bk);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float2 p = __ffma2_rn(make_float2(s[16 * g + e], s[16 * g + e + 1]), a2, b2);
              p.x = ex2_approx(p.x);
              p.y = ex2_approx(p.y);
              sum = __fadd2_rn(sum, p);
              w[(g & 1) * 8 + e / 2] = pack2(p.x, p.y);
            }
            // a poisoned scale (NaN) counts only for rows that see its keys
            l = fmaf(sum.x + sum.y, plain || vis > j0 + 16 * g ? k.z : 0.f, l);
          }
          if (C::kOwnP && q2 == 0 && n > 0) {  // the block before has left the weights' columns
            ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[t], static_cast<uint32_t>((n - 1) & 1), a.wait_ns));
            tc_fence_after_sync();
          }
          tmem_st_16cols_async(tp + 16 * q2, w);
        }
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[t], static_cast<uint32_t>((n - 1) & 1), a.wait_ns) && !*abort_flag);
      if (!ok) {
        tmem_st_wait();  // of weights that no MMA will take
        if (lane == 0) fail(DEV_WAIT_TIMEOUT_EPILOGUE);
      }
      tc_fence_after_sync();
    }
    bool have = ok && nb > 0;
    // ---- the odd blocks' state, handed over in their stage of K (channels below D / 2) and V and their codes' place
    float f0 = 1.f, f1 = 0.f;
    auto handed = [&](int d) {  // channel d of this row
      return reinterpret_cast<float*>(smem + (d < D / 2 ? C::kOffK : C::kOffV) + C::kOp) + (d % (D / 2)) * kTile + rt;
    };
    if (alt) {
      float2* hml = reinterpret_cast<float2*>(smem + C::kOp) + rt;
      if (t == 1) {
        if (have) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld_32cols_async(to + 32 * c, o);
            tmem_ld_wait32(o);
#pragma unroll
            for (int x = 0; x < 32; ++x) handed(32 * c)[x * kTile] = o[x];
          }
        }
        *hml = make_float2(m_ref, l);
      }
      named_barrier_sync(1 + (warp & 3), 64);  // the two warps of these rows
      if (t == 0) {
        have = have && !*abort_flag;
        const float2 ml = *hml;
        const float m = fmaxf(m_ref, ml.x);
        f0 = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - m);
        f1 = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
        m_ref = m;
        l = fmaf(l, f0, ml.y * f1);
      }
    }
    // ---- out = O / l, or the state of this key range
    const bool split = a.plan.n_splits > 1;
    const int64_t prow = (static_cast<int64_t>(z) * a.q.n_tok + tok) * a.Hq + hq;
    const float il = l == 0.f ? 0.f : 1.f / l;
    if (active && nb > 0 && !have && !(alt && t == 1)) {
      // a wait ran out: the rows say so, with every range they are joined from
      if (valid) {
        if (split) {
          a.part_ml[prow] = make_float2(0.f, NAN);
        } else {
          T* dst = static_cast<T*>(a.out) + tok * a.out_tok + hq * a.out_head;
#pragma unroll 1
          for (int d = 0; d < D; ++d) dst[d] = from_f<T>(NAN);
          if (a.lse) a.lse[static_cast<int64_t>(tok) * a.Hq + hq] = NAN;
        }
      }
    } else if (active && !(alt && t == 1)) {
      // The warp turns its rows through its part of the Q tile (every S is done), 256 bytes of a row at a
      // time, so that 16 lanes write them side by side.
      uint8_t* turn = smem + t * C::kOp + (warp & 3) * (C::kOp / 4);
      constexpr int kRowB = D == 128 ? 256 : 128;             // bytes of a row in a pass: the tile's share
      constexpr int kChunks = kRowB / 16;
      const int passes = D * (split ? 4 : 2) / kRowB;
      const int64_t mine = split ? prow * D : tok * a.out_tok + hq * a.out_head;
      const uint32_t kept = __ballot_sync(0xffffffffu, valid && (!split || (have && l != 0.f)));
      const bool wide =
          split || ((reinterpret_cast<uintptr_t>(a.out) | static_cast<uint64_t>(a.out_tok | a.out_head) * 2) & 15) == 0;
#pragma unroll 1
      for (int p = 0; p < passes; ++p) {
        // this thread's row: kRowB bytes from column p * (kRowB / element)
#pragma unroll 1
        for (int c = 0; c < (split ? kRowB / 4 : kRowB / 2) / 32; ++c) {
          float o[32];
          const int d = p * (split ? kRowB / 4 : kRowB / 2) + 32 * c;
          if (have) {
            tmem_ld_32cols_async(to + d, o);
            tmem_ld_wait32(o);
            if (alt) {
              const float* other = handed(d);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = fmaf(o[x], f0, other[x * kTile] * f1);
            }
          }
          const bool some = have && l != 0.f;
          if (split) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              *reinterpret_cast<float4*>(turn + lane * kRowB + (((8 * c + x) ^ (lane & 7)) << 4)) =
                  make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              alignas(16) T y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = from_f<T>(some ? o[8 * x + e] * il : 0.f);
              *reinterpret_cast<uint4*>(turn + lane * kRowB + (((4 * c + x) ^ (lane & 7)) << 4)) = *reinterpret_cast<const uint4*>(y);
            }
          }
          __syncwarp();
        }
#pragma unroll 4
        for (int e = lane; e < 32 * kChunks; e += 32) {
          const int row = e / kChunks, ch = e % kChunks;
          const int64_t at = __shfl_sync(0xffffffffu, mine, row);
          if (!(kept >> row & 1)) continue;
          const uint4 y = *reinterpret_cast<const uint4*>(turn + row * kRowB + ((ch ^ (row & 7)) << 4));
          if (split) {
            *reinterpret_cast<uint4*>(a.part_o + at + p * (kRowB / 4) + ch * 4) = y;
          } else {
            T* dst = static_cast<T*>(a.out) + at + p * (kRowB / 2) + ch * 8;
            if (wide) {
              *reinterpret_cast<uint4*>(dst) = y;
            } else {
              alignas(16) T x[8];
              *reinterpret_cast<uint4*>(x) = y;
#pragma unroll
              for (int k = 0; k < 8; ++k) dst[k] = x[k];
            }
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
  if (warp == 1) {  // nothing of this CTA's copies may still be landing when it exits
    for (int x = max(0, raw_issued - (alt ? 4 : 2)); x < raw_issued; ++x)
      mbar_wait(&raw_full[raw_bar(x >> 1, x & 1)], raw_par(x >> 1), kDrainWaitNs);
  }
  if (warp == 0) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, int FMT, class T, bool ALT>
int launch_tile(const PagedAttnArgs& a, cudaStream_t s) {
  using C = TileCfg<D>;
  auto kern = paged_attn_tile_kernel<D, FMT, T, ALT>;
  static KernelSetup setup;
  const cudaError_t r = setup.run(kern, C::kSmem);
  if (r != cudaSuccess) return r;
  const int64_t items = ((static_cast<int64_t>(a.q.n_tok) * a.G) >> 8) + a.q.n_seq;
  return launch_k(kern, dim3(static_cast<unsigned>(items), static_cast<unsigned>(a.c.Hkv), static_cast<unsigned>(a.plan.n_splits)),
                  dim3(512), C::kSmem, s, a);
}
template <int D, int FMT>
int launch_tile_t(const PagedAttnArgs& a, cudaStream_t s) {
  if (a.plan.alternate)
    return a.dtype == PCD_DTYPE_BF16 ? launch_tile<D, FMT, __nv_bfloat16, true>(a, s) : launch_tile<D, FMT, __half, true>(a, s);
  return a.dtype == PCD_DTYPE_BF16 ? launch_tile<D, FMT, __nv_bfloat16, false>(a, s) : launch_tile<D, FMT, __half, false>(a, s);
}

}  // namespace

int launch_paged_attention_tiles(const PagedAttnArgs& a, cudaStream_t s) {
  const bool f8 = a.c.format == PCD_KV_E4M3;
  if (a.c.dim == 64) return f8 ? launch_tile_t<64, PCD_KV_E4M3>(a, s) : launch_tile_t<64, PCD_KV_INT8>(a, s);
  return f8 ? launch_tile_t<128, PCD_KV_E4M3>(a, s) : launch_tile_t<128, PCD_KV_INT8>(a, s);
}

}  // namespace pcd
