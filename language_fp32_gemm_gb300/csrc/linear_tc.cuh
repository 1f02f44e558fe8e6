// The product with its epilogue on the fifth-generation tensor cores:
//   s_rc = sum_k row_rk col_ck,   out = act(s * scales + bias) + residual.
//
// A persistent kernel, one CTA (or pair of CTAs on neighbouring SMs) per SM
// (pair).  Warp 0 loads operand tiles by TMA into a ring of shared-memory stages,
// 128 bytes of the contraction a stage; one thread of warp 1 issues tcgen05.mma
// into one of two tensor-memory buffers; the other warps add finished partial sums
// into fp32 registers and, at the end of a tile, run the epilogue while the next
// tile's loads and MMAs proceed.
//
// Operands are 16-bit or 8-bit and go from the caller's memory straight to
// shared memory: either layout of a 16-bit operand is a tile of 128-byte swizzled
// rows that the matrix descriptor names (contraction contiguous, or rows
// contiguous), so no operand is ever transposed.  fp32 operands arrive as two fp16
// terms each (linear_prep.cu) and three products are summed, small ones first.
//
// The tensor cores' fp32 accumulation truncates, so a partial sum spans at most
// promote_blocks stages (24 or 36 MMA updates for fp32 operands, 32 for fp32 outputs
// of others, 128 for 16-bit outputs) before it is added, with rounding, into registers.
//
// Tiles: 256 x 256 on a pair for large outputs; 128 x {16, 32, 64, 128} on one CTA
// for few columns, with the output transposed (SWAP) when those columns are the
// caller's rows: a few tokens then ride along the weight's rows, each read once.
// The tiles that do not fill a last wave are cut along the contraction; each piece
// leaves its sum in the workspace and the last one to arrive adds them all in
// order, so that no piece waits for another and the result does not depend on
// their order.
//
// Large products are bound by the MMAs and the power they draw (bf16 8192^3: 592 to 631
// us, up to 1.86 PFLOP/s, with tanh GELU, pre-activation and residual 690 to 752; in
// seconds-long loops at the power cap 712 and, with bias too, 744, at the same clock),
// short contractions by the epilogue (bf16 8192 x 8192 x 512 over the same buffers: 67 us,
// with all four 125), few rows by the weight's way in (fp16 16 x 8192 x 8192: 26.6 us,
// 5.1 TB/s).  8 bits 4096 x 8192 x 8192 with scales, bias, SiLU and residual: 198 us, 2.8
// PFLOP/s; fp32 4096^3 with tanh GELU, pre-activation and residual: 346 to 355 us with its
// operands' split, 1.2 PFLOP/s of fp16 terms.
#pragma once

#include <type_traits>

#include "epilogue.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace phobos {

namespace tc {

constexpr int kRows = 128;  // tile rows of one CTA
constexpr int kSmemLimit = 227 * 1024;
constexpr int kBarrierBytes = 512;

template <int BN, int PASSES, bool PAIR>
struct Shape {
  static constexpr int kTerms = PASSES == 3 ? 2 : 1;
  static constexpr int kColRows = PAIR ? BN / 2 : BN;  // rows of the column operand per CTA
  static constexpr int kRowTile = kRows * 128;         // bytes
  static constexpr int kColTile = kColRows * 128;
  static constexpr int kStage = kTerms * (kRowTile + kColTile);
  // 16 accumulator warps hide more of one another's latency (bf16 8192 x 8192 x 512: 66 us,
  // with eight 87), but leave fp32 blocks half the shared memory each (8192 x 8192 x 512
  // with everything: 374 us, with eight 348).
  static constexpr int kEpiWarps = !PAIR ? 4 : PASSES == 3 ? 8 : 16;
  // In a pair the accumulator warps are warpgroups of their own, which take registers
  // from the first: 64 or 128 sums a thread and the epilogue need more than the 96 or
  // 168 that 20 or 12 warps start with (128 * 40 + 512 * 104 <= 640 * 96, 128 * 104 +
  // 256 * 200 = 384 * 168).
  static constexpr int kRegsFirst = PASSES == 3 ? 104 : 40, kRegsEpi = PASSES == 3 ? 200 : 104;
  static constexpr int kFirstEpi = PAIR ? 4 : 2;
  static constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
  static constexpr int kCols = BN * 4 / kEpiWarps;  // columns summed by one thread
  static constexpr int kTmemCols = 2 * BN;
  static constexpr int kSlots = PAIR ? 2 : 4;  // epilogue blocks of a warp
  static constexpr int kEpiBytes = kEpiWarps * kSlots * kEpilogueBox;
  static constexpr int kAux = 1024 + kBarrierBytes + kEpiBytes;
  static constexpr int kStages = (kSmemLimit - kAux) / kStage < 10 ? (kSmemLimit - kAux) / kStage : 10;
  static constexpr int kSmem = kStages * kStage + kAux;
  static_assert(kStages >= 2 && (2 * kStages + 5 + kEpiWarps * kSlots) * 8 + 8 <= kBarrierBytes, "ring and barriers fit");
};

// MMA with 8-bit operands (e4m3), K = 32 an instruction.
template <bool PAIR>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 tensor-memory columns of a warp's lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// An epilogue block: global to shared (completing on an mbarrier of this CTA) and
// back.  Coordinates outside the matrix are read as zeros and not written.
__device__ __forceinline__ void block_store(const void *map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Until at most `pending` (0 .. 3) of this thread's stores still read shared memory.
__device__ __forceinline__ void block_stores_read(int pending) {
  switch (pending) {
    case 3: asm volatile("cp.async.bulk.wait_group.read 3;" ::: "memory"); break;
    case 2: asm volatile("cp.async.bulk.wait_group.read 2;" ::: "memory"); break;
    case 1: asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); break;
    default: asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); break;
  }
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (TYPE == PHOBOS_TYPE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  } else {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
}
template <int TYPE>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  if constexpr (TYPE == PHOBOS_TYPE_BF16)
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}

// Descriptor of a tile whose rows (not the contraction) are contiguous: boxes of
// 64 rows x 64 contraction steps, 128 swizzled bytes a step; eight steps are
// 1024 bytes apart, the next 64 rows 8192 bytes.
__device__ __forceinline__ uint64_t desc_rowmajor_sw128(uint32_t addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;  // leading offset: the next 64 rows
  d |= static_cast<uint64_t>(1024 >> 4) << 32;  // stride offset: the next 8 steps
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

struct Item {
  int tile, k_lo, k_hi, piece;  // piece -1: the whole tile
};

__device__ __forceinline__ Item item_of(const TcLinearArgs &p, int i) {
  if (i < p.full_tiles) return Item{i, 0, p.k_blocks, -1};
  const int r = i - p.full_tiles, j = r / p.pieces, q = r - j * p.pieces;
  return Item{p.full_tiles + j, static_cast<int>(static_cast<int64_t>(p.k_blocks) * q / p.pieces),
              static_cast<int>(static_cast<int64_t>(p.k_blocks) * (q + 1) / p.pieces),
              p.pieces > 1 ? q : -1};
}

// Tiles in groups of `group` tile rows, column by column inside a group, so that
// the tiles in flight share operand panels in L2.
__device__ __forceinline__ void tile_at(const TcLinearArgs &p, int t, int &tr, int &tc) {
  const int per_group = p.group * p.tiles_c;
  const int g = t / per_group, first = g * p.group;
  const int rows = min(p.group, p.tiles_r - first), r = t - g * per_group;
  tr = first + r % rows;
  tc = r / rows;
}

// How a kernel's epilogue reaches memory: by TMA, element by element, or as the
// launch says.  Pair kernels are made for one way: their epilogue has no registers
// to spare for the other (with both, 7 % more time at 4096^3 in fp32).
enum Way { kByTma, kByElement, kAsLaunched };

template <int BN, int PASSES, bool PAIR, bool SWAP, Way WAY>
__global__ void __launch_bounds__(Shape<BN, PASSES, PAIR>::kThreads, 1)
    linear_tc_kernel(const __grid_constant__ TcLinearArgs p) {
  using S = Shape<BN, PASSES, PAIR>;
  constexpr int STAGES = S::kStages;
  constexpr int kTileR = PAIR ? 2 * kRows : kRows;
  constexpr int kCols = S::kCols;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t *aux = smem_raw + (ring - raw) + STAGES * S::kStage;
  uint64_t *bars = reinterpret_cast<uint64_t *>(aux);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * STAGES + 5);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const uint32_t res_bar0 = smem_u32(tmem_slot + 2);  // one per epilogue block
  const uint32_t epi0 = smem_u32(aux + kBarrierBytes);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * STAGES;
  const uint32_t acc_full0 = full0 + 16u * STAGES, acc_empty0 = acc_full0 + 16u, drained = acc_full0 + 32u;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x) / (PAIR ? 2 : 1);
  const int units = static_cast<int>(gridDim.x) / (PAIR ? 2 : 1);
  auto abort_peer = [&]() {
    if (PAIR)
      st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<int *>(abort_flag)), rank ^ 1u), 1u);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full0 + 8u * b, 1);
      mbar_init(acc_empty0 + 8u * b, (PAIR ? 2 : 1) * S::kEpiWarps);
    }
    mbar_init(drained, 1);
    for (int s = 0; s < S::kEpiWarps * S::kSlots; ++s) mbar_init(res_bar0 + 8u * s, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    for (int t = 0; t < S::kTerms; ++t) {
      prefetch_tmap(&p.row[t]);
      prefetch_tmap(&p.col[t]);
    }
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), S::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), S::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncwarp();
  if (PAIR) cluster_sync();  // the peer's barriers exist before anyone signals them
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_begin();  // the operands; what came before is set up while an earlier kernel runs

  if (warp < S::kFirstEpi) {
  if (PAIR) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsFirst));
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const int k_elems = p.type == PHOBOS_TYPE_E4M3 ? 128 : 64;  // contraction steps of a stage
      uint32_t armed = 0, last_parity = 0, s = 0, ph = 0;
      bool ok = true, withhold = p.withhold_first_load != 0;
      for (int i = unit; ok && i < p.items; i += units) {
        const Item it = item_of(p, i);
        int tr, tc;
        tile_at(p, it.tile, tr, tc);
        const int r0 = tr * kTileR + static_cast<int>(rank) * kRows;
        const int c0 = tc * BN + static_cast<int>(rank) * S::kColRows;
        for (int kb = it.k_lo; kb < it.k_hi; ++kb) {
          auto next_stage = [&]() {
            if (++s == STAGES) {
              s = 0;
              ph ^= 1u;
            }
          };
          if (withhold) {  // failure-detection test
            withhold = false;
            next_stage();
            continue;
          }
          if (!bounded_wait(empty0 + 8u * s, ph ^ 1u, abort_flag, p.err, kDevTimeoutProducer)) {
            abort_peer();
            ok = false;
            break;
          }
          const uint32_t full = full0 + 8u * s;
          const uint32_t bar = PAIR ? mapa_shared(full, 0u) : full;
          if (leader) mbar_arrive_expect_tx(full, (PAIR ? 2 : 1) * S::kStage);
          const int k0 = kb * k_elems;
          uint32_t dst = ring + s * S::kStage;
          auto load = [&](uint32_t to, const CUtensorMap *map, int x, int y) {
            if (PAIR) tma_load_2d_pair(to, map, bar, x, y);
            else tma_load_2d(to, map, bar, x, y);
          };
#pragma unroll
          for (int t = 0; t < S::kTerms; ++t, dst += S::kRowTile) {
            if (p.row_kmajor) {
              load(dst, &p.row[t], k0, r0);
            } else {
              load(dst, &p.row[t], r0, k0);
              load(dst + 8192u, &p.row[t], r0 + 64, k0);
            }
          }
#pragma unroll
          for (int t = 0; t < S::kTerms; ++t, dst += S::kColTile) {
            if (S::kColRows < 64 || p.col_kmajor) {
              load(dst, &p.col[t], k0, c0);
            } else {
#pragma unroll
              for (int b = 0; b < S::kColRows / 64; ++b) load(dst + 8192u * b, &p.col[t], c0 + 64 * b, k0);
            }
          }
          armed |= 1u << s;
          last_parity = (last_parity & ~(1u << s)) | (ph << s);
          next_stage();
        }
      }
      // No bulk copy may still be writing shared memory at exit: the leader's full
      // barriers count every armed stage; a peer cannot see its own copies, so
      // after an abort it gives them a bounded time.
      if (leader) {
        for (int s = 0; s < STAGES; ++s)
          if (armed & (1u << s))
            bounded_wait(full0 + 8u * s, (last_parity >> s) & 1u, abort_flag, p.err, kDevTimeoutDrain, false);
      }
      if (PAIR && *abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0 && leader) {
      // One thread issues four (twelve) MMAs per stage of 512 (1536) tensor cycles,
      // so its instructions count: descriptors advance by an addition (their
      // address field never carries out), stages and phases by counters, and the
      // instruction kind is chosen outside the loop.
      const uint32_t idesc = idesc_f16(kTileR, BN, p.type == PHOBOS_TYPE_BF16) |
                             (p.row_kmajor ? 0u : 1u << 15) | (p.col_kmajor ? 0u : 1u << 16);
      const uint64_t row_desc = p.row_kmajor ? desc_kmajor_sw128(ring) : desc_rowmajor_sw128(ring);
      const uint32_t col_ring = ring + S::kTerms * S::kRowTile;
      const uint64_t col_desc = p.col_kmajor ? desc_kmajor_sw128(col_ring) : desc_rowmajor_sw128(col_ring);
      // from one MMA's slice of the contraction to the next, in units of 16 bytes
      const uint32_t row_step = p.row_kmajor ? 2u : 128u, col_step = p.col_kmajor ? 2u : 128u;
      auto issue = [&](auto eight_bit) {
        auto mma = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
          if constexpr (decltype(eight_bit)::value) mma_f8<PAIR>(d, a, b, idesc, acc);
          else if constexpr (PAIR) mma_f16_pair(d, a, b, idesc, acc);
          else mma_f16(d, a, b, idesc, acc);
        };
        uint32_t s = 0, phase = 0;
        int partial = 0;
        for (int i = unit; i < p.items; i += units) {
          const Item it = item_of(p, i);
          for (int kb = it.k_lo; kb < it.k_hi; ++partial) {
            const int b = partial & 1;
            const uint32_t use = static_cast<uint32_t>(partial >> 1);
            // the accumulator warps have read this buffer's previous partial sum
            const bool free_buf =
                PAIR ? bounded_wait_cluster(acc_empty0 + 8u * b, (use & 1u) ^ 1u, abort_flag, p.err, kDevTimeoutMma)
                     : bounded_wait(acc_empty0 + 8u * b, (use & 1u) ^ 1u, abort_flag, p.err, kDevTimeoutMma);
            if (!free_buf) {
              abort_peer();
              return;
            }
            tc_fence_after();
            const uint32_t d = tmem_base + static_cast<uint32_t>(b * BN);
            const int kb_end = min(it.k_hi, kb + p.promote_blocks);
            uint32_t acc = 0;
            for (; kb < kb_end; ++kb) {
              if (!bounded_wait(full0 + 8u * s, phase, abort_flag, p.err, kDevTimeoutMma)) {
                abort_peer();
                return;
              }
              tc_fence_after();
              const uint64_t row0 = row_desc + s * (S::kStage >> 4), row1 = row0 + (S::kRowTile >> 4);
              const uint64_t col0 = col_desc + s * (S::kStage >> 4), col1 = col0 + (S::kColTile >> 4);
#pragma unroll
              for (uint32_t kk = 0; kk < 4; ++kk) {
                const uint32_t ro = kk * row_step, co = kk * col_step;
                if (PASSES == 3) {
                  mma(d, row1 + ro, col0 + co, acc);
                  mma(d, row0 + ro, col1 + co, 1u);
                  mma(d, row0 + ro, col0 + co, 1u);
                } else {
                  mma(d, row0 + ro, col0 + co, acc);
                }
                acc = 1;
              }
              if (PAIR) mma_commit_pair(empty0 + 8u * s, 0x3);
              else mma_commit(empty0 + 8u * s);
              if (++s == STAGES) {
                s = 0;
                phase ^= 1u;
              }
            }
            if (PAIR) mma_commit_pair(acc_full0 + 8u * b, 0x3);
            else mma_commit(acc_full0 + 8u * b);
          }
        }
      };
      if (PASSES == 1 && p.type == PHOBOS_TYPE_E4M3) issue(std::true_type());
      else issue(std::false_type());
      // every MMA is finished before tensor memory is released
      if (PAIR) mma_commit_pair(drained, 0x1);
      else mma_commit(drained);
      bounded_wait(drained, 0, abort_flag, p.err, kDevTimeoutDrain, false);
    }
  }
  } else {
    if (PAIR) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegsEpi));
    // ------------------------------------------------- accumulate, epilogue
    const int q = warp & 3;         // tensor-memory lane quarter of this warp
    const int h = (warp - S::kFirstEpi) >> 2;  // column half or quarter (pairs)
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const int ew = warp - S::kFirstEpi;
    const uint32_t slots = epi0 + static_cast<uint32_t>(ew * S::kSlots * kEpilogueBox);
    const uint32_t res_bars = res_bar0 + 8u * static_cast<uint32_t>(ew * S::kSlots);
    // The block slots take turns: all for the residual and output of successive
    // blocks, or half of them when pre-activations go out too.
    const int out_slots = p.e.preact ? S::kSlots / 2 : S::kSlots;
    uint32_t res_phase = 0, res_pending = 0;  // bit per slot
    int partial = 0;
    bool ok = true;
    for (int i = unit; ok && i < p.items; i += units) {
      const Item it = item_of(p, i);
      int tr, tc;
      tile_at(p, it.tile, tr, tc);
      const int r0 = tr * kTileR + static_cast<int>(rank) * kRows + q * 32;  // this warp's 32 tile rows
      const int c0 = tc * BN + h * kCols;                                    // and kCols tile columns
      // Blocks of the tile: 64 bytes of the output's columns a lane (row), or, transposed,
      // 32 columns (lanes) x 32 or 16 rows.
      const int elem = p.e.type == PHOBOS_TYPE_F32 ? 4 : 2;
      // (64 bytes, or 32 elements where the kernel only copies element by element)
      const int width = min(kCols, SWAP ? kEpilogueBox / (32 * elem) : WAY == kByElement ? 32 : 64 / elem);
      const int limit = SWAP ? p.M : p.N;  // of tile columns
      const bool inside = r0 < (SWAP ? p.N : p.M);
      const int blocks = inside && c0 < limit ? (min(kCols, limit - c0) + width - 1) / width : 0;
      auto load_residual = [&](int block) {  // one lane
        const int s = block % out_slots;
        mbar_arrive_expect_tx(res_bars + 8u * s, SWAP ? 32 * elem * width : kEpilogueBox);
        tma_load_2d(slots + s * kEpilogueBox, &p.residual, res_bars + 8u * s, SWAP ? r0 : c0 + block * width,
                    SWAP ? c0 + block * width : r0);
        res_pending |= 1u << s;
      };
      const bool use_tma = WAY == kAsLaunched ? p.tma != 0 : WAY == kByTma;
      const bool residual_tma = use_tma && p.e.residual;
      // A tile takes the slots in turn from the first: none of the tile's before may still
      // be read then, whatever its number of blocks was.
      auto begin_blocks = [&]() {
        if (lane == 0 && use_tma) {
          block_stores_read(0);
          for (int b = 0; residual_tma && b < blocks && b < out_slots; ++b) load_residual(b);
        }
      };
      if (it.piece < 0) begin_blocks();
      float sum[kCols];  // the first partial sum is taken as it is
      const int n_partials = (it.k_hi - it.k_lo + p.promote_blocks - 1) / p.promote_blocks;
      for (int c = 0; c < n_partials; ++c, ++partial) {
        const int b = partial & 1;
        // (uniform: a wait that runs out ends the walk of the whole warp)
        if (!__all_sync(0xffffffffu, bounded_wait(acc_full0 + 8u * b, static_cast<uint32_t>(partial >> 1) & 1u,
                                                  abort_flag, p.err, kDevTimeoutEpilogue))) {
          ok = false;
          abort_peer();
          break;
        }
        tc_fence_after();
        const uint32_t col = tmem_base + static_cast<uint32_t>(b * BN + h * kCols) + lane_base;
        if constexpr (kCols >= 32) {
#pragma unroll
          for (int j = 0; j < kCols; j += 32) {
            uint32_t r[32];
            tmem_ld32(col + j, r);
            phobos::tmem_ld_wait(r);
#pragma unroll
            for (int u = 0; u < 32; ++u)
              sum[j + u] = c == 0 ? __uint_as_float(r[u]) : __fadd_rn(sum[j + u], __uint_as_float(r[u]));
          }
        } else {
          uint32_t r[16];
          tmem_ld16(col, r);
          tmem_ld_wait(r);
#pragma unroll
          for (int u = 0; u < 16; ++u) sum[u] = c == 0 ? __uint_as_float(r[u]) : __fadd_rn(sum[u], __uint_as_float(r[u]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_cluster(mapa_shared(acc_empty0 + 8u * b, 0u));
          else mbar_arrive(acc_empty0 + 8u * b);
        }
      }
      if (!ok) break;
      if (it.piece >= 0) {
        // Leave the piece's sum in its slot (float4 v of lane l at v * 32 + l) and
        // count in; the last piece of the tile adds all of them in order (its own too:
        // kept in registers beside the others' they spilled, 10 % at 8192^3).  One
        // atomic a warp releases the lanes' stores and acquires the other pieces': the
        // barriers order the lanes' stores before it and their loads after it (a shuffle
        // orders no memory).
        constexpr int kF4 = kCols / 4;
        constexpr int64_t kSlot = static_cast<int64_t>(PAIR ? 2 : 1) * S::kEpiWarps * kF4 * 32;
        const int jt = it.tile - p.full_tiles;
        float4 *const first = reinterpret_cast<float4 *>(p.partials) + static_cast<int64_t>(jt) * p.pieces * kSlot +
                              (static_cast<int>(rank) * S::kEpiWarps + ew) * (kF4 * 32) + lane;
        float4 *const mine = first + it.piece * kSlot;
#pragma unroll
        for (int v = 0; v < kF4; ++v)
          __stcg(mine + v * 32, make_float4(sum[4 * v], sum[4 * v + 1], sum[4 * v + 2], sum[4 * v + 3]));
        __syncwarp();
        unsigned arrived = 0;
        if (lane == 0) {
          unsigned *counter = p.counters + (jt * (PAIR ? 2 : 1) + static_cast<int>(rank)) * S::kEpiWarps + ew;
          arrived = atom_add_acq_rel_gpu(counter, 1u) + 1u;
          if (arrived == static_cast<unsigned>(p.pieces)) *counter = 0u;  // for the next launch
        }
        if (__shfl_sync(0xffffffffu, arrived, 0) != static_cast<unsigned>(p.pieces)) continue;
        __syncwarp();
        begin_blocks();
        constexpr int kBatch = kF4 < 8 ? kF4 : 8;
#pragma unroll
        for (int v0 = 0; v0 < kF4; v0 += kBatch) {
#pragma unroll 1
          for (int piece = 0; piece < p.pieces; ++piece) {
            float4 x[kBatch];
#pragma unroll
            for (int v = 0; v < kBatch; ++v) x[v] = __ldcg(first + piece * kSlot + (v0 + v) * 32);
#pragma unroll
            for (int v = 0; v < kBatch; ++v) {
              float *s = sum + 4 * (v0 + v);
              s[0] = piece ? __fadd_rn(s[0], x[v].x) : x[v].x;
              s[1] = piece ? __fadd_rn(s[1], x[v].y) : x[v].y;
              s[2] = piece ? __fadd_rn(s[2], x[v].z) : x[v].z;
              s[3] = piece ? __fadd_rn(s[3], x[v].w) : x[v].w;
            }
          }
        }
      }
      with_type(p.e.type, [&](auto type_tag) {
        constexpr int TYPE = decltype(type_tag)::value;
        using E = Elem<TYPE>;
        constexpr int kElem = static_cast<int>(sizeof(typename E::T));
        constexpr int kFull = SWAP ? kEpilogueBox / (32 * kElem) : WAY == kByElement ? 32 : 64 / kElem;
        constexpr int kWidth = kFull < kCols ? kFull : kCols;  // == width
        // Lane l holds the factors of tile columns l, 32 + l, ... and of its own tile row.
        constexpr int kColRegs = (kCols + 31) / 32;
        float bias[kColRegs] = {}, factor[kColRegs] = {}, row_factor = 0.f, row_bias = 0.f;
        auto load_bias = [&](int col) { return p.e.bias && col < p.N ? E::load(static_cast<const typename E::T *>(p.e.bias)[col]) : 0.f; };
        // scales, or the bits of exponents
        const float *of_rows = p.e.row_exp ? reinterpret_cast<const float *>(p.e.row_exp) : p.e.row_scale;
        const float *of_cols = p.e.col_exp ? reinterpret_cast<const float *>(p.e.col_exp) : p.e.col_scale;
        const float *of_tile_rows = SWAP ? of_cols : of_rows, *of_tile_cols = SWAP ? of_rows : of_cols;
        const bool scaled = of_rows != nullptr, powers = p.e.row_exp != nullptr;
        if (scaled && r0 + lane < (SWAP ? p.N : p.M)) row_factor = of_tile_rows[r0 + lane];
        if (SWAP) row_bias = load_bias(r0 + lane);
#pragma unroll
        for (int c = 0; c < kColRegs; ++c) {
          const int col = c0 + c * 32 + lane;
          if (!SWAP) bias[c] = load_bias(col);
          if (scaled && col < limit) factor[c] = of_tile_cols[col];
        }
        // Rows of a block are kRowBytes apart; their 16-byte chunks are permuted so that
        // the lanes' own rows fall on different banks (64 bytes: the TMA's pattern).
        constexpr int kRowBytes = kWidth * kElem;
        auto chunk_of = [&](int row, int chunk) { return chunk ^ (kRowBytes == 64 ? (row >> 1) & 3 : row & 7); };
        auto chunk_at = [&](uint32_t slot, int chunk) { return slot + lane * kRowBytes + (chunk_of(lane, chunk) << 4); };
        // Without TMA: a block between global and shared memory, kPerTurn output rows
        // of kBlockCols elements at a time, a lane per element.
        constexpr int kBlockRows = SWAP ? kWidth : 32, kBlockCols = SWAP ? 32 : kWidth;
        constexpr int kPerTurn = 32 / kBlockCols, kTurns = kBlockRows / kPerTurn, kBatch = kTurns < 8 ? kTurns : 8;
        const int el_row = lane / kBlockCols, el_col = lane % kBlockCols;
        auto element_at = [&](uint32_t slot, int r) {
          return SWAP ? slot + (r * 32 + el_col) * kElem
                      : slot + r * kRowBytes + (chunk_of(r, el_col * kElem >> 4) << 4) + (el_col * kElem & 15);
        };
        auto first_row = [&](int block) { return (SWAP ? c0 + block * kWidth : r0) + el_row; };
        auto this_col = [&](int block) { return (SWAP ? r0 : c0 + block * kWidth) + el_col; };
        using Bits = std::conditional_t<kElem == 4, uint32_t, uint16_t>;
        auto copy_out = [&](uint32_t slot, int block, void *base, int64_t ld) {
          const int row = first_row(block), col = this_col(block);
          Bits *to = static_cast<Bits *>(base) + row * ld + col;
          const int rows = col < p.N ? p.M - row : 0;  // rows of this lane's that exist
#pragma unroll kBatch
          for (int i = 0; i < kTurns; ++i, to += kPerTurn * ld) {
            const uint32_t at = element_at(slot, i * kPerTurn + el_row);
            Bits v;
            if constexpr (kElem == 4) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
            else asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
            if (i * kPerTurn < rows) *to = v;
          }
          __syncwarp();
        };
        // fp32 in the background, 16-bit types (which cp.async cannot) through registers
        auto copy_in = [&](uint32_t slot, int block) {
          const int row = first_row(block), col = this_col(block);
          const Bits *from = static_cast<const Bits *>(p.e.residual) + row * p.e.residual_ld + col;
          const int rows = col < p.N ? p.M - row : 0;
          const int64_t step = kPerTurn * p.e.residual_ld;
#pragma unroll 1
          for (int i0 = 0; i0 < kTurns; i0 += kBatch, from += kBatch * step) {
            Bits v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const bool in = (i0 + i) * kPerTurn < rows;
              if constexpr (kElem == 4) {
                if (in)
                  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(element_at(slot, (i0 + i) * kPerTurn + el_row)),
                               "l"(__cvta_generic_to_global(from + i * step))
                               : "memory");
              } else {
                v[i] = in ? from[i * step] : Bits(0);
              }
            }
            if constexpr (kElem == 2) {
#pragma unroll
              for (int i = 0; i < kBatch; ++i)
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(element_at(slot, (i0 + i) * kPerTurn + el_row)), "h"(v[i]) : "memory");
            }
          }
          cp_async_commit();
        };
        // without TMA one slot serves: the residual of the next block follows this block
        // out, ahead of its use, unless pre-activations need the slot first
        const bool copies = !use_tma && p.e.residual, copies_ahead = copies && !p.e.preact;
        if (copies_ahead && blocks > 0) copy_in(slots, 0);
        // this lane's values of a block to a slot
        auto put = [&](uint32_t slot, const float (&v)[kWidth]) {
          if constexpr (SWAP) {
#pragma unroll
            for (int j = 0; j < kWidth; ++j) {
              const uint32_t at = slot + (j * 32 + lane) * kElem;
              if constexpr (kElem == 4) {
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v[j]) : "memory");
              } else {
                const uint32_t x = pack2<TYPE>(v[j], 0.f);
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(x)) : "memory");
              }
            }
          } else if constexpr (kElem == 4) {
#pragma unroll
            for (int j = 0; j < kWidth; j += 4)
              sts128(chunk_at(slot, j / 4), __float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                     __float_as_uint(v[j + 3]));
          } else {
#pragma unroll
            for (int j = 0; j < kWidth; j += 8)
              sts128(chunk_at(slot, j / 8), pack2<TYPE>(v[j], v[j + 1]), pack2<TYPE>(v[j + 2], v[j + 3]),
                     pack2<TYPE>(v[j + 4], v[j + 5]), pack2<TYPE>(v[j + 6], v[j + 7]));
          }
        };
        auto add_residual = [&](uint32_t slot, float (&v)[kWidth]) {
          if constexpr (SWAP) {
#pragma unroll
            for (int j = 0; j < kWidth; ++j) {
              const uint32_t at = slot + (j * 32 + lane) * kElem;
              if constexpr (kElem == 4) {
                float x;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
                v[j] += x;
              } else {
                uint16_t x;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
                v[j] += unpack2<TYPE>(x).x;
              }
            }
          } else {
            constexpr int kPer = 16 / kElem;
#pragma unroll
            for (int j = 0; j < kWidth; j += kPer) {
              const uint4 x = lds128(chunk_at(slot, j / kPer));
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                if constexpr (kElem == 4) {
                  v[j + t] += __uint_as_float(w[t]);
                } else {
                  const float2 f = unpack2<TYPE>(w[t]);
                  v[j + 2 * t] += f.x;
                  v[j + 2 * t + 1] += f.y;
                }
              }
            }
          }
        };
        // a filled slot to global memory
        auto send = [&](uint32_t slot, int block, const CUtensorMap *map, void *base, int64_t ld) {
          if (use_tma) {
            fence_proxy_async_shared();  // every lane's stores before the TMA's reads
            __syncwarp();
            if (lane == 0)
              block_store(map, slot, SWAP ? r0 : c0 + block * kWidth, SWAP ? c0 + block * kWidth : r0);
          } else {
            __syncwarp();
            copy_out(slot, block, base, ld);
          }
        };
#pragma unroll 1
        for (int block = 0; block < blocks; ++block) {
          const int s = use_tma ? block % out_slots : 0;
          const uint32_t out_slot = slots + s * kEpilogueBox;
          const uint32_t z_slot = use_tma ? out_slot + out_slots * kEpilogueBox : slots;
          if (use_tma) {
            if (lane == 0) {
              // the residual of the block that takes over the previous block's slot
              const bool next = residual_tma && block > 0 && block - 1 + out_slots < blocks;
              block_stores_read(next ? 0 : p.e.preact ? 2 * (out_slots - 1) : out_slots - 1);
              if (next) load_residual(block - 1 + out_slots);
            }
            __syncwarp();  // no store reads these slots any more
          }
          float v[kWidth];
          // column j of the block is column (block * kWidth) % 32 + j of the front registers
          const int from = kWidth < 32 ? (block & (32 / kWidth - 1)) * kWidth : 0;
          if (!scaled) {
#pragma unroll
            for (int j = 0; j < kWidth; ++j) v[j] = sum[j];
          } else if (powers) {
#pragma unroll
            for (int j = 0; j < kWidth; ++j)
              v[j] = times_pow2(sum[j], __float_as_int(__shfl_sync(0xffffffffu, factor[0], from + j)) + __float_as_int(row_factor));
          } else {
#pragma unroll
            for (int j = 0; j < kWidth; ++j) v[j] = sum[j] * __shfl_sync(0xffffffffu, factor[0], from + j) * row_factor;
          }
          if (p.e.bias) {
#pragma unroll
            for (int j = 0; j < kWidth; ++j) v[j] += SWAP ? row_bias : __shfl_sync(0xffffffffu, bias[0], from + j);
          }
          // the next block's sums and factors move to the front: registers have constant names
#pragma unroll
          for (int j = 0; j < kCols - kWidth; ++j) sum[j] = sum[j + kWidth];
          if (kWidth >= 32 || ((block + 1) * kWidth) % 32 == 0) {
#pragma unroll
            for (int c = 0; c + 1 < kColRegs; ++c) {
              bias[c] = bias[c + 1];
              factor[c] = factor[c + 1];
            }
          }
          if (p.e.preact) {
            put(z_slot, v);
            send(z_slot, block, &p.preact, p.e.preact, p.e.preact_ld);
          }
          activate_all(p.e.act, v);
          if (p.e.residual) {
            if (use_tma) {
              if (!__all_sync(0xffffffffu, bounded_wait(res_bars + 8u * s, (res_phase >> s) & 1u, abort_flag, p.err,
                                                        kDevTimeoutEpilogue))) {
                ok = false;
                abort_peer();
                return;
              }
              res_phase ^= 1u << s;
              res_pending &= ~(1u << s);
            } else {
              if (!copies_ahead) copy_in(out_slot, block);
              cp_async_wait_all();
              __syncwarp();
            }
            add_residual(out_slot, v);
          }
          put(out_slot, v);
          send(out_slot, block, &p.out, p.e.out, p.e.out_ld);
          if (copies_ahead && block + 1 < blocks) copy_in(slots, block + 1);
        }
      });
    }
    if (lane == 0) {
      // no bulk copy may still use shared memory at exit (residuals: only after an abort)
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      for (int s = 0; s < S::kSlots; ++s)
        if (res_pending >> s & 1u)
          bounded_wait(res_bars + 8u * s, (res_phase >> s) & 1u, abort_flag, p.err, kDevTimeoutDrain, false);
    }
  }

  tc_fence_before();
  __syncwarp();
  if (PAIR) cluster_sync();  // the leader's MMAs read the peer's shared memory until here
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem_base, S::kTmemCols);
    else tmem_dealloc(tmem_base, S::kTmemCols);
  }
}

template <int BN, int PASSES, bool PAIR, bool SWAP, Way WAY>
cudaError_t launch(const TcLinearArgs &a, int units, cudaStream_t stream) {
  using S = Shape<BN, PASSES, PAIR>;
  auto kernel = linear_tc_kernel<BN, PASSES, PAIR, SWAP, WAY>;
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void *>(kernel), S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, PAIR ? 2 : 1, static_cast<unsigned>(units) * (PAIR ? 2u : 1u), S::kThreads, S::kSmem,
                       stream, a);
}

}  // namespace tc

cudaError_t launch_linear_tc_pair(const TcLinearArgs &a, const TcShapeId &id, int units, cudaStream_t stream);
cudaError_t launch_linear_tc_narrow(const TcLinearArgs &a, const TcShapeId &id, int units, cudaStream_t stream);
cudaError_t launch_linear_tc_split(const TcLinearArgs &a, const TcShapeId &id, int units, cudaStream_t stream);

}  // namespace phobos
