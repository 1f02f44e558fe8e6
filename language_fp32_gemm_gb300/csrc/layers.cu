// C ABI of the layer operators: argument checks, choice of kernel, workspaces.
// See include/phobos_layers.h for the contract of every entry point.
#include "../../include/phobos_layers.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <map>
#include <utility>

#include "host_rules.h"
#include "layers_internal.h"
#include "runtime.h"

namespace phobos {
namespace {

bool float_type(int t) {
  return t == PHOBOS_TYPE_F32 || t == PHOBOS_TYPE_F16 || t == PHOBOS_TYPE_BF16;
}
int type_bytes(int t) {
  return t == PHOBOS_TYPE_F32 ? 4 : t == PHOBOS_TYPE_E4M3 ? 1 : 2;
}
int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// A dimension pair and a row-major matrix of it with unit column stride.
bool good_rows(int64_t cols, int64_t ld) { return ld >= std::max<int64_t>(cols, 1); }

// Either stride is one and the other covers the vectors laid along the first;
// a dimension of one (or none) leaves its stride free.
bool good_strides(int64_t rows, int64_t cols, int64_t row, int64_t col) {
  if (rows <= 1 && cols <= 1) return true;
  if (col == 1 || cols <= 1) {
    if (rows <= 1 || row >= std::max<int64_t>(cols, 1)) return true;
  }
  return (row == 1 || rows <= 1) && (cols <= 1 || col >= std::max<int64_t>(rows, 1));
}

// The operand whose vectors are the `rows` rows of a rows x k matrix.
Operand make_operand(const void *ptr, int64_t rows, int64_t k, int64_t row, int64_t col) {
  Operand o;
  o.ptr = ptr;
  // unit stride along k, or k has no second element to step to
  o.kmajor = (col == 1 || k <= 1) && (rows <= 1 || row >= std::max<int64_t>(k, 1)) ? 1 : 0;
  o.ld = o.kmajor ? row : col;
  if (o.kmajor ? rows <= 1 : k <= 1) o.ld = std::max<int64_t>(o.kmajor ? k : rows, 1);
  return o;
}

// Groups of 16 bytes of every row are aligned.
bool rows_aligned(const void *ptr, int64_t ld, int type) {
  return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld * type_bytes(type) % 16 == 0;
}

// Groups of four elements starting at multiples of four are aligned.
bool groups_aligned(const void *ptr, int64_t ld, int type) {
  return (reinterpret_cast<uintptr_t>(ptr) % (4 * type_bytes(type))) == 0 && ld % 4 == 0;
}

bool good_products(int p) { return p >= PHOBOS_PRODUCTS_AUTO && p <= PHOBOS_PRODUCTS_TENSOR; }

int simt_kslices(int64_t M, int64_t N, int64_t K, int sm_count) {
  const int64_t bm = M <= 16 ? 16 : 64;
  const int64_t tiles = ((M + bm - 1) / bm) * ((N + 63) / 64);
  // about two CTAs an SM, or (few rows, bound by the weight's way in) four; two stages each
  const int64_t s = std::min<int64_t>({8, (M <= 16 ? 4 : 2) * sm_count / std::max<int64_t>(tiles, 1), (K + 63) / 64});
  return s < 1 ? 1 : static_cast<int>(s);
}

phobos_status_t run_simt(const LinearArgs &l, const Runtime &rt, cudaStream_t stream) {
  SimtArgs a{};
  a.l = l;
  a.vec_a = groups_aligned(l.a.ptr, l.a.ld, l.type);
  a.vec_b = groups_aligned(l.b.ptr, l.b.ld, l.type);
  if (l.type == PHOBOS_TYPE_F32 && l.M <= 16 && l.K > 0 && l.a.kmajor && a.vec_a && a.vec_b)
    return runtime_launched(launch_linear_gemv(a, rt.sm_count, stream));
  a.kslices = simt_kslices(l.M, l.N, l.K, rt.sm_count);
  return runtime_launched(launch_linear_simt(a, stream));
}

// -------------------------------------------------------------- tensor-core plan

constexpr int kMaxPieces = 16;

struct TcPlan {
  TcShapeId id;
  int tiles_r, tiles_c, full_tiles, pieces, units;
  double cycles;  // estimate
};

// The estimated time (cycles) of one kernel on R tile rows x C tile columns: rounds
// of whole tiles over the units, then the tail's pieces, and the last epilogue,
// which nothing hides.  A stage of the contraction costs the largest of its MMAs
// (4096 16-bit multiply-adds a cycle and SM), its loads (48 bytes a cycle and SM
// from L2) and, where each operand is read once, its share of the memory's latency
// (2.8 us over the ring, measured with 64 CTAs at 16 x 8192 x 8192); the whole
// cannot be faster than the operands' bytes at 3500 a cycle.  A piece of a tile costs
// its sums' way through L2, which its unit's next piece waits for (16 x 8192 x
// 8192: 42, 28, 37, 32, 37, 35, 40 us with 1, 2, 3, 4, 5, 7, 8 pieces).
TcPlan plan_shape(const TcShapeId &id, int64_t R, int64_t C, int k_blocks, int sm_count) {
  TcPlan p{};
  p.id = id;
  const int tile_r = id.pair ? 256 : 128, passes = id.split ? 3 : 1, terms = id.split ? 2 : 1;
  p.tiles_r = static_cast<int>((R + tile_r - 1) / tile_r);
  p.tiles_c = static_cast<int>((C + id.bn - 1) / id.bn);
  p.units = id.pair ? sm_count / 2 : sm_count;
  const int64_t tiles = static_cast<int64_t>(p.tiles_r) * p.tiles_c;
  const double mma = std::max(id.pair ? 512.0 : 2.0 * id.bn, 64.0) * passes;
  const double bytes = terms * 128.0 * (128 + (id.pair ? 128 : id.bn));  // of a stage and CTA
  const double ring = std::min(10.0, 190000.0 / bytes);
  const double stage = std::max({mma, bytes / 48.0, std::min(p.tiles_r, p.tiles_c) == 1 ? 5300.0 / ring : 0.0});
  const int cols = id.pair ? id.bn / 2 : id.bn;
  const double epilogue = 1500.0 + 25.0 * cols, piece = 2500.0 + 25.0 * cols;
  const int64_t rounds = tiles / p.units, tail = tiles % p.units;
  p.full_tiles = static_cast<int>(tiles - tail);
  p.pieces = 1;
  double best = tail ? k_blocks * stage : 0.0;
  for (int s = 2; tail && s <= kMaxPieces && 4 * s <= k_blocks; ++s) {
    const double turns = static_cast<double>((tail * s + p.units - 1) / p.units);
    const double t = turns * (((k_blocks + s - 1) / s) * stage + piece);
    if (t < best) {
      best = t;
      p.pieces = s;
    }
  }
  const double memory = terms * 128.0 * k_blocks * static_cast<double>(R + C) / 3500.0;
  p.cycles = std::max(rounds * std::max(k_blocks * stage, epilogue) + best, memory) + epilogue;
  return p;
}

// The kernel with the least estimated time.  A column operand whose rows lie side
// by side is loaded in boxes of 64 rows, so narrower tiles cannot take it.
TcPlan plan_tc(const LinearArgs &l, int k_blocks, int sm_count) {
  const bool split = l.type == PHOBOS_TYPE_F32;
  TcPlan best = plan_shape({256, true, split, false}, l.M, l.N, k_blocks, sm_count);
  for (int swap = 0; swap < 2; ++swap) {
    const Operand &col = swap ? l.a : l.b;
    for (int bn = split ? 64 : swap ? 16 : 32; bn <= 128; bn *= 2) {
      if (bn < 64 && !col.kmajor) continue;
      const TcPlan p = plan_shape({bn, false, split, swap != 0}, swap ? l.N : l.M, swap ? l.M : l.N, k_blocks, sm_count);
      if (p.cycles < best.cycles) best = p;
    }
  }
  return best;
}

// Where an operand's prepared form goes in the workspace (nothing for one that the
// TMA can read in place).
struct Prepared {
  bool needed = false;
  size_t hi = 0, lo = 0, exp = 0;  // offsets
  int64_t ld = 0;
};

Prepared place_operand(const Operand &o, int64_t rows, int64_t k, int type, size_t &bytes) {
  Prepared p;
  const int elem = type == PHOBOS_TYPE_F32 ? 2 : type_bytes(type);
  if (type != PHOBOS_TYPE_F32 && reinterpret_cast<uintptr_t>(o.ptr) % 16 == 0 && o.ld * elem % 16 == 0) return p;
  p.needed = true;
  const int64_t inner = o.kmajor ? k : rows, outer = o.kmajor ? rows : k;
  p.ld = round_up(inner, 16 / elem);
  auto take = [&](int64_t n) {
    const size_t at = bytes;
    bytes += static_cast<size_t>(round_up(n, 256));
    return at;
  };
  p.hi = take(outer * p.ld * elem);
  if (type == PHOBOS_TYPE_F32) {
    p.lo = take(outer * p.ld * elem);
    p.exp = take(rows * static_cast<int64_t>(sizeof(int)));
  }
  return p;
}

PrepArgs prep_args(const Operand &o, int rows, int k, int type, const Prepared &p, char *ws) {
  PrepArgs a{};
  a.in = o;
  a.rows = rows;
  a.k = k;
  a.type = type;
  a.vec = groups_aligned(o.ptr, o.ld, type);
  a.hi = ws + p.hi;
  a.lo = ws + p.lo;
  a.ld = p.ld;
  a.exp = reinterpret_cast<int *>(ws + p.exp);
  return a;
}

phobos_status_t prepare_operands(const LinearArgs &l, const Prepared &pa, const Prepared &pb, char *ws,
                                 const Runtime &rt, cudaStream_t stream) {
  const PrepArgs a = prep_args(l.a, l.M, l.K, l.type, pa, ws), b = prep_args(l.b, l.N, l.K, l.type, pb, ws);
  if (l.type == PHOBOS_TYPE_F32) {
    if (l.a.kmajor == l.b.kmajor) return runtime_launched(launch_split(a, &b, rt.sm_count, stream));
    const phobos_status_t first = runtime_launched(launch_split(a, nullptr, rt.sm_count, stream));
    return first == PHOBOS_OK ? runtime_launched(launch_split(b, nullptr, rt.sm_count, stream)) : first;
  }
  phobos_status_t st = PHOBOS_OK;
  if (pa.needed) st = runtime_launched(launch_copy(a, rt.sm_count, stream));
  if (st == PHOBOS_OK && pb.needed) st = runtime_launched(launch_copy(b, rt.sm_count, stream));
  return st;
}

// Maps of an operand's terms: boxes of 128 bytes of the contraction x box_rows, or
// of 64 rows x 64 contraction steps.
phobos_status_t map_operand(CUtensorMap (&maps)[2], const Operand &o, const Prepared &p, char *ws, int64_t rows,
                            int64_t k, int type, int box_rows) {
  const int elem = type == PHOBOS_TYPE_F32 ? 2 : type_bytes(type);
  const CUtensorMapDataType t = type == PHOBOS_TYPE_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                : type == PHOBOS_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int terms = type == PHOBOS_TYPE_F32 ? 2 : 1;
  phobos_status_t st = PHOBOS_OK;
  for (int i = 0; i < terms && st == PHOBOS_OK; ++i) {
    const void *base = p.needed ? ws + (i ? p.lo : p.hi) : o.ptr;
    const uint64_t ld = static_cast<uint64_t>(p.needed ? p.ld : o.ld) * elem;
    st = o.kmajor ? runtime_tensor_map(&maps[i], t, base, k, rows, ld, 128 / elem, box_rows, CU_TENSOR_MAP_SWIZZLE_128B)
                  : runtime_tensor_map(&maps[i], t, base, rows, k, ld, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  return st;
}

// Whether the TMA can reach a matrix: 16-byte aligned base and rows (one row has
// no stride).
bool tma_matrix(const void *ptr, int64_t rows, int64_t ld, int type) {
  return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && (rows == 1 || ld * type_bytes(type) % 16 == 0);
}

// Map of an M x N matrix of the epilogue.
phobos_status_t map_output(CUtensorMap *map, const void *ptr, int64_t ld, const LinearArgs &l, const TcShapeId &id) {
  const int elem = type_bytes(l.e.type);
  const CUtensorMapDataType t = l.e.type == PHOBOS_TYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : l.e.type == PHOBOS_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int rows = id.swap ? std::min(id.bn, kEpilogueBox / (32 * elem)) : 32;
  if (l.M == 1) ld = round_up(l.N, 16);
  return runtime_tensor_map(map, t, ptr, l.N, l.M, static_cast<uint64_t>(ld) * elem, id.swap ? 32 : 64 / elem, rows,
                            id.swap ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_64B);
}

phobos_status_t run_tc(const LinearArgs &l, const Runtime &rt, cudaStream_t stream) {
  const int elem = l.type == PHOBOS_TYPE_F32 ? 2 : type_bytes(l.type);
  const int k_blocks = static_cast<int>((static_cast<int64_t>(l.K) * elem + 127) / 128);
  const TcPlan plan = plan_tc(l, k_blocks, rt.sm_count);
  const int64_t tiles = static_cast<int64_t>(plan.tiles_r) * plan.tiles_c;
  const int64_t tail = tiles - plan.full_tiles;
  if (tiles + tail * plan.pieces > 0x7fffffff) return PHOBOS_ERR_UNSUPPORTED;
  size_t bytes = 0;
  const Prepared pa = place_operand(l.a, l.M, l.K, l.type, bytes);
  const Prepared pb = place_operand(l.b, l.N, l.K, l.type, bytes);
  const size_t partials = bytes;
  if (plan.pieces > 1)
    bytes += static_cast<size_t>(tail * plan.pieces * tc_partial_floats(plan.id)) * sizeof(float);
  phobos_status_t st;
  void *ws_ptr = nullptr;
  if (bytes > 0 && (st = runtime_workspace(rt, stream, kProductSpace, bytes, &ws_ptr)) != PHOBOS_OK) return st;
  char *ws = static_cast<char *>(ws_ptr);
  TcLinearArgs t{};
  if (plan.pieces > 1) {
    if (tail * tc_counters(plan.id) > kTileCounters) return PHOBOS_ERR_UNSUPPORTED;
    if ((st = runtime_counters(rt, stream, &t.counters)) != PHOBOS_OK) return st;
    t.partials = reinterpret_cast<float *>(ws + partials);
  }
  if ((st = prepare_operands(l, pa, pb, ws, rt, stream)) != PHOBOS_OK) return st;
  const bool swap = plan.id.swap;
  const int col_box = plan.id.pair ? plan.id.bn / 2 : plan.id.bn;
  if ((st = map_operand(swap ? t.col : t.row, l.a, pa, ws, l.M, l.K, l.type, swap ? col_box : 128)) != PHOBOS_OK ||
      (st = map_operand(swap ? t.row : t.col, l.b, pb, ws, l.N, l.K, l.type, swap ? 128 : col_box)) != PHOBOS_OK)
    return st;
  const Epilogue &e = l.e;
  t.tma = tma_matrix(e.out, l.M, e.out_ld, e.type) &&
          (!e.residual || tma_matrix(e.residual, l.M, e.residual_ld, e.type)) &&
          (!e.preact || tma_matrix(e.preact, l.M, e.preact_ld, e.type));
  if (t.tma) {
    if ((st = map_output(&t.out, e.out, e.out_ld, l, plan.id)) != PHOBOS_OK ||
        (e.residual && (st = map_output(&t.residual, e.residual, e.residual_ld, l, plan.id)) != PHOBOS_OK) ||
        (e.preact && (st = map_output(&t.preact, e.preact, e.preact_ld, l, plan.id)) != PHOBOS_OK))
      return st;
  }
  t.type = l.type == PHOBOS_TYPE_F32 ? PHOBOS_TYPE_F16 : l.type;
  t.row_kmajor = swap ? l.b.kmajor : l.a.kmajor;
  t.col_kmajor = swap ? l.a.kmajor : l.b.kmajor;
  t.tiles_r = plan.tiles_r;
  t.tiles_c = plan.tiles_c;
  t.group = std::min(plan.tiles_r, 16);
  t.k_blocks = k_blocks;
  // Truncating MMA updates per partial sum: 36 of three fp16 products (24 for short
  // contractions); 32 for fp32 outputs; 128 for 16-bit ones, whose own rounding is
  // 2^-11 or 2^-8.  An update loses up to 2^-23 of the sum so far, so that 128 of them and
  // up to 32 roundings stay within 2^-15 of the terms' magnitudes; with 512, a sum of one
  // large and many small terms of its sign did not.  (bf16 8192^3 with everything: 746 us,
  // with 512 updates 742, with 32 787 to 814; 8 bits 4096 x 8192 x 8192: 196, 196, 212.)
  // fp32, norm of the error over the norm of the result at any K, and time at 4096^3: 1
  // block 2.7e-7, 414 us; 2 blocks 4.8e-7, 351; 3 blocks 6.9e-7, 334; 4 blocks 9.3e-7, 327.
  t.promote_blocks = l.type == PHOBOS_TYPE_F32 ? (l.K <= 512 ? 2 : 3) : l.e.type == PHOBOS_TYPE_F32 ? 8 : 32;
  t.full_tiles = plan.full_tiles;
  t.pieces = plan.pieces;
  t.items = plan.full_tiles + static_cast<int>(tail) * plan.pieces;
  t.M = l.M;
  t.N = l.N;
  t.e = l.e;
  if (l.type == PHOBOS_TYPE_F32) {
    t.e.row_exp = reinterpret_cast<int *>(ws + pa.exp);
    t.e.col_exp = reinterpret_cast<int *>(ws + pb.exp);
  }
  t.err = rt.err;
  t.withhold_first_load = runtime_withhold_load();
  return runtime_launched(launch_linear_tc(t, plan.id, std::min(plan.units, t.items), stream));
}

// AUTO, 16-bit and 8-bit operands: the tensor cores (a 64 x 64 x 256 product: 5.3 us,
// on the CUDA cores 9.2), a few tokens and a weight that is not large without tiles
// (the times on both sides of 40 MB, and of rows of 64 KB, are in linear_token.cu).
bool few_tokens(const LinearArgs &l) {
  const int64_t row = static_cast<int64_t>(l.K) * type_bytes(l.type);
  return l.type != PHOBOS_TYPE_F32 && l.M <= 16 && row <= 65536 && row * l.N <= 40000000 && l.a.kmajor && l.b.kmajor &&
         reinterpret_cast<uintptr_t>(l.a.ptr) % 16 == 0 && (l.M == 1 || rows_aligned(l.a.ptr, l.a.ld, l.type)) &&
         reinterpret_cast<uintptr_t>(l.b.ptr) % 16 == 0 && (l.N == 1 || rows_aligned(l.b.ptr, l.b.ld, l.type));
}

// AUTO, fp32 operands: the way with the shorter estimate, in microseconds, fitted to
// (CUDA cores, tensor cores): 512^3 17, 24; 256 x 1024 x 1024 24, 30; 1024^3 72, 43;
// 64 x 4096 x 4096 72, 60; 16 x 8192 x 8192 93 to 105, 175 to 215.
bool prefer_ffma(const LinearArgs &l, const Runtime &rt) {
  if (l.type != PHOBOS_TYPE_F32) return false;
  const double M = l.M, N = l.N, K = l.K, macs = M * N * K;
  const double few_rows = std::max(K * N * 4 / 5.5e6, macs / 11.5e6) + 6.0;
  const double ffma = l.M <= 16 ? few_rows : macs / 15.6e6 + 7.0;
  // the split operands' way through memory, then the product
  const double prepared = 18.0 + (M * K + K * N) * 8 / 4.5e6;
  return ffma < prepared || ffma < prepared + plan_tc(l, (l.K + 63) / 64, rt.sm_count).cycles / 1900.0;
}

phobos_status_t run_linear(const LinearArgs &l, int products, const Runtime &rt, cudaStream_t stream) {
  const bool ffma = l.K == 0 || products == PHOBOS_PRODUCTS_FFMA ||
                    (products == PHOBOS_PRODUCTS_AUTO && prefer_ffma(l, rt));
  if (ffma) return run_simt(l, rt, stream);
  if (products == PHOBOS_PRODUCTS_AUTO && few_tokens(l)) return runtime_launched(launch_linear_token(l, rt.sm_count, stream));
  return run_tc(l, rt, stream);
}

phobos_status_t check_linear(const phobos_linear_args_t &a) {
  if (a.M < 0 || a.N < 0 || a.K < 0 || !good_products(a.products)) return PHOBOS_ERR_INVALID_VALUE;
  if (!(float_type(a.type) || a.type == PHOBOS_TYPE_E4M3) || !float_type(a.out_type) ||
      a.act < PHOBOS_ACT_NONE || a.act > PHOBOS_ACT_SILU)
    return PHOBOS_ERR_INVALID_VALUE;
  if (!good_strides(a.M, a.K, a.x_row, a.x_col) || !good_strides(a.K, a.N, a.w_row, a.w_col))
    return PHOBOS_ERR_INVALID_VALUE;
  const bool q8 = a.type == PHOBOS_TYPE_E4M3;
  if (q8 && a.K > 1 && (a.x_col != 1 || a.w_row != 1)) return PHOBOS_ERR_INVALID_VALUE;
  if (!good_rows(a.N, a.out_row) || (a.residual && !good_rows(a.N, a.residual_row)) ||
      (a.preact && !good_rows(a.N, a.preact_row)))
    return PHOBOS_ERR_INVALID_VALUE;
  if (a.M > kMaxDim || a.N > kMaxDim || a.K > kMaxDim) return PHOBOS_ERR_UNSUPPORTED;
  if (a.M == 0 || a.N == 0) return PHOBOS_OK;
  if (!a.out || (a.K > 0 && (!a.x || !a.w))) return PHOBOS_ERR_INVALID_VALUE;
  if (q8 != (a.x_scale != nullptr) || q8 != (a.w_scale != nullptr)) return PHOBOS_ERR_INVALID_VALUE;
  return PHOBOS_OK;
}

phobos_status_t linear_impl(const phobos_linear_args_t &a, cudaStream_t stream) {
  phobos_status_t st = check_linear(a);
  if (st != PHOBOS_OK || a.M == 0 || a.N == 0) return st;
  LinearArgs l{};
  l.M = static_cast<int>(a.M);
  l.N = static_cast<int>(a.N);
  l.K = static_cast<int>(a.K);
  l.type = a.type;
  l.a = make_operand(a.x, a.M, a.K, a.x_row, a.x_col);
  l.b = make_operand(a.w, a.N, a.K, a.w_col, a.w_row);
  l.e.type = a.out_type;
  l.e.act = a.act;
  l.e.bias = a.bias;
  l.e.residual = a.residual;
  l.e.preact = a.preact;
  l.e.out = a.out;
  l.e.residual_ld = a.residual_row;
  l.e.preact_ld = a.preact_row;
  l.e.out_ld = a.out_row;
  l.e.row_scale = a.x_scale;
  l.e.col_scale = a.w_scale;
  l.e.vec = groups_aligned(a.out, a.out_row, a.out_type) &&
            (!a.bias || groups_aligned(a.bias, 0, a.out_type)) &&
            (!a.residual || groups_aligned(a.residual, a.residual_row, a.out_type)) &&
            (!a.preact || groups_aligned(a.preact, a.preact_row, a.out_type));
  std::lock_guard<std::mutex> lock(runtime_mutex());
  Runtime rt;
  if ((st = runtime_state(&rt)) != PHOBOS_OK) return st;
  if ((st = run_linear(l, a.products, rt, stream)) != PHOBOS_OK) return st;
  return runtime_finish(rt, stream);
}

phobos_status_t check_linear_backward(const phobos_linear_backward_args_t &a) {
  if (a.M < 0 || a.N < 0 || a.K < 0 || (a.accumulate != 0 && a.accumulate != 1) ||
      !good_products(a.products) || a.reserved != 0)
    return PHOBOS_ERR_INVALID_VALUE;
  if (!float_type(a.type) || (a.grad_type != a.type && a.grad_type != PHOBOS_TYPE_F32) ||
      a.act < PHOBOS_ACT_NONE || a.act > PHOBOS_ACT_SILU)
    return PHOBOS_ERR_INVALID_VALUE;
  if (!good_rows(a.N, a.dout_row) || !good_strides(a.M, a.K, a.x_row, a.x_col) ||
      !good_strides(a.K, a.N, a.w_row, a.w_col) || (a.dx && !good_rows(a.K, a.dx_row)) ||
      (a.dw && !good_strides(a.K, a.N, a.dw_row, a.dw_col)))
    return PHOBOS_ERR_INVALID_VALUE;
  if (a.act != PHOBOS_ACT_NONE && !good_rows(a.N, a.preact_row)) return PHOBOS_ERR_INVALID_VALUE;
  if (a.M > kMaxDim || a.N > kMaxDim || a.K > kMaxDim) return PHOBOS_ERR_UNSUPPORTED;
  const bool has_dz = a.M > 0 && a.N > 0;
  if (has_dz && (a.dx || a.dw || a.dbias) && (!a.dout || (a.act != PHOBOS_ACT_NONE && !a.preact)))
    return PHOBOS_ERR_INVALID_VALUE;
  if (has_dz && a.K > 0 && ((a.dx && !a.w) || (a.dw && !a.x))) return PHOBOS_ERR_INVALID_VALUE;
  return PHOBOS_OK;
}

// Rows per strip of a pass over M x N that leaves one row of sums per strip:
// enough strips for about eight CTAs per SM, at least 64 rows each.
void choose_strips(int64_t M, int64_t col_blocks, int sm_count, int &strips, int &rows) {
  int64_t want = std::max<int64_t>(1, 8 * sm_count / std::max<int64_t>(col_blocks, 1));
  int64_t r = std::max<int64_t>(64, round_up((M + want - 1) / want, 8));
  rows = static_cast<int>(r);
  strips = static_cast<int>((M + r - 1) / r);
}

phobos_status_t linear_backward_impl(const phobos_linear_backward_args_t &a, cudaStream_t stream) {
  phobos_status_t st = check_linear_backward(a);
  if (st != PHOBOS_OK) return st;
  const bool want_dx = a.dx && a.M > 0 && a.K > 0, want_dw = a.dw && a.K > 0 && a.N > 0;
  const bool want_db = a.dbias && a.N > 0;
  if (!want_dx && !want_dw && !want_db) return PHOBOS_OK;
  std::lock_guard<std::mutex> lock(runtime_mutex());
  Runtime rt;
  if ((st = runtime_state(&rt)) != PHOBOS_OK) return st;
  const int M = static_cast<int>(a.M), N = static_cast<int>(a.N), K = static_cast<int>(a.K);
  const int elem = type_bytes(a.type);

  // workspace: [dz][strip sums]
  const bool store_dz = a.act != PHOBOS_ACT_NONE && (want_dx || want_dw);
  const int64_t dz_ld = round_up(a.N, 16 / elem);
  int strips = 0, strip_rows = 1;
  const bool vec = rows_aligned(a.dout, a.dout_row, a.type) &&
                   (a.act == PHOBOS_ACT_NONE || rows_aligned(a.preact, a.preact_row, a.type));
  const int block_cols = 32 * (vec ? 16 / elem : 1);
  choose_strips(a.M, (a.N + block_cols - 1) / block_cols, rt.sm_count, strips, strip_rows);
  const size_t dz_bytes = store_dz ? static_cast<size_t>(round_up(a.M * dz_ld * elem, 256)) : 0;
  const size_t sum_bytes = want_db ? static_cast<size_t>(strips) * a.N * sizeof(float) : 0;
  void *ws = nullptr;
  if (dz_bytes + sum_bytes > 0 &&
      (st = runtime_workspace(rt, stream, kGradientSpace, dz_bytes + sum_bytes, &ws)) != PHOBOS_OK)
    return st;
  float *sums = reinterpret_cast<float *>(static_cast<char *>(ws) + dz_bytes);
  if (M > 0 && N > 0 && (store_dz || want_db)) {
    DzArgs d{};
    d.M = M;
    d.N = N;
    d.type = a.type;
    d.act = a.act;
    d.dout = a.dout;
    d.dout_ld = a.dout_row;
    d.z = a.act != PHOBOS_ACT_NONE ? a.preact : nullptr;
    d.z_ld = a.preact_row;
    d.dz = store_dz ? ws : nullptr;
    d.dz_ld = dz_ld;
    d.partial = want_db ? sums : nullptr;
    d.strips = strips;
    d.strip_rows = strip_rows;
    d.vec = vec;
    if ((st = runtime_launched(launch_dz(d, stream))) != PHOBOS_OK) return st;
  }
  if (want_db && (st = runtime_launched(launch_column_sums(sums, strips, N, a.dbias, a.grad_type,
                                                           a.accumulate, stream))) != PHOBOS_OK)
    return st;
  const void *dz = store_dz ? ws : a.dout;
  const int64_t ld = store_dz ? dz_ld : a.dout_row;
  if (want_dx) {  // dx[M][K] = sum over N of dz_in w_kn
    LinearArgs l{};
    l.M = M;
    l.N = K;
    l.K = N;
    l.type = a.type;
    l.a = make_operand(dz, a.M, a.N, ld, 1);
    l.b = make_operand(a.w, a.K, a.N, a.w_row, a.w_col);
    l.e.type = a.type;
    l.e.out = a.dx;
    l.e.out_ld = a.dx_row;
    l.e.vec = groups_aligned(a.dx, a.dx_row, a.type);
    if ((st = run_linear(l, a.products, rt, stream)) != PHOBOS_OK) return st;
  }
  if (want_dw) {  // dw[K][N] = sum over M of x_mk dz_mn, or its transpose where dw is stored so
    LinearArgs l{};
    const Operand x = make_operand(a.x, a.K, a.M, a.x_col, a.x_row);
    const Operand d = make_operand(dz, a.N, a.M, 1, ld);
    const Operand out = make_operand(a.dw, a.K, a.N, a.dw_row, a.dw_col);
    l.M = out.kmajor ? K : N;
    l.N = out.kmajor ? N : K;
    l.K = M;
    l.type = a.type;
    l.a = out.kmajor ? x : d;
    l.b = out.kmajor ? d : x;
    l.e.type = a.grad_type;
    l.e.out = a.dw;
    l.e.out_ld = out.ld;
    l.e.residual = a.accumulate ? a.dw : nullptr;
    l.e.residual_ld = out.ld;
    l.e.vec = groups_aligned(a.dw, out.ld, a.grad_type);
    if ((st = run_linear(l, a.products, rt, stream)) != PHOBOS_OK) return st;
  }
  return runtime_finish(rt, stream);
}

phobos_status_t rmsnorm_impl(const phobos_rmsnorm_args_t &a, cudaStream_t stream) {
  if (a.rows < 0 || a.cols < 0 || a.reserved != 0 || !float_type(a.type) ||
      (a.out_type != a.type && a.out_type != PHOBOS_TYPE_E4M3) || !(a.eps >= 0.0f))
    return PHOBOS_ERR_INVALID_VALUE;
  const bool q8 = a.out_type == PHOBOS_TYPE_E4M3;
  if (!good_rows(a.cols, a.x_row) || !good_rows(a.cols, a.out_row) ||
      (a.residual != nullptr) != (a.sum != nullptr) ||
      (a.residual && (!good_rows(a.cols, a.residual_row) || !good_rows(a.cols, a.sum_row))))
    return PHOBOS_ERR_INVALID_VALUE;
  if (a.rows > kMaxDim || a.cols > kMaxDim) return PHOBOS_ERR_UNSUPPORTED;
  if (a.rows == 0 || a.cols == 0) return PHOBOS_OK;
  if (!a.x || !a.out || q8 != (a.scale != nullptr)) return PHOBOS_ERR_INVALID_VALUE;
  NormArgs n{};
  n.rows = static_cast<int>(a.rows);
  n.cols = static_cast<int>(a.cols);
  n.type = a.type;
  n.q8 = q8;
  n.eps = a.eps;
  n.x = a.x;
  n.x_ld = a.x_row;
  n.residual = a.residual;
  n.residual_ld = a.residual_row;
  n.weight = a.weight;
  n.sum = a.sum;
  n.sum_ld = a.sum_row;
  n.out = a.out;
  n.out_ld = a.out_row;
  n.scale = a.scale;
  n.vec = rows_aligned(a.x, a.x_row, a.type) && (!a.weight || rows_aligned(a.weight, 0, a.type)) &&
          (!a.residual || rows_aligned(a.residual, a.residual_row, a.type));
  // 16 bytes of the inputs are 8 (4, fp32) bytes of an 8-bit output
  const int out_group = q8 ? 16 / type_bytes(a.type) : 16;
  n.vec_out = reinterpret_cast<uintptr_t>(a.out) % out_group == 0 &&
              a.out_row * type_bytes(a.out_type) % out_group == 0 &&
              (!a.sum || rows_aligned(a.sum, a.sum_row, a.type));
  std::lock_guard<std::mutex> lock(runtime_mutex());
  Runtime rt;
  phobos_status_t st = runtime_state(&rt);
  if (st == PHOBOS_OK) st = runtime_launched(launch_rmsnorm(n, rt.sm_count, stream));
  return st == PHOBOS_OK ? runtime_finish(rt, stream) : st;
}

phobos_status_t rmsnorm_backward_impl(const phobos_rmsnorm_backward_args_t &a, cudaStream_t stream) {
  if (a.rows < 0 || a.cols < 0 || !float_type(a.type) || !(a.eps >= 0.0f))
    return PHOBOS_ERR_INVALID_VALUE;
  if (!good_rows(a.cols, a.dy_row) || !good_rows(a.cols, a.h_row) || !good_rows(a.cols, a.dx_row) ||
      (a.dsum && !good_rows(a.cols, a.dsum_row)))
    return PHOBOS_ERR_INVALID_VALUE;
  if (a.rows > kMaxDim || a.cols > kMaxDim) return PHOBOS_ERR_UNSUPPORTED;
  if (a.cols == 0 || (a.rows == 0 && !a.dweight)) return PHOBOS_OK;
  if (a.rows > 0 && (!a.dy || !a.h || !a.dx)) return PHOBOS_ERR_INVALID_VALUE;
  std::lock_guard<std::mutex> lock(runtime_mutex());
  Runtime rt;
  phobos_status_t st = runtime_state(&rt);
  if (st != PHOBOS_OK) return st;
  NormBackwardArgs n{};
  n.rows = static_cast<int>(a.rows);
  n.cols = static_cast<int>(a.cols);
  n.type = a.type;
  n.eps = a.eps;
  n.dy = a.dy;
  n.dy_ld = a.dy_row;
  n.h = a.h;
  n.h_ld = a.h_row;
  n.weight = a.weight;
  n.dsum = a.dsum;
  n.dsum_ld = a.dsum_row;
  n.dx = a.dx;
  n.dx_ld = a.dx_row;
  n.vec_out = rows_aligned(a.dx, a.dx_row, a.type);
  n.vec = rows_aligned(a.dy, a.dy_row, a.type) && rows_aligned(a.h, a.h_row, a.type) && (!a.weight || rows_aligned(a.weight, 0, a.type)) &&
          (!a.dsum || rows_aligned(a.dsum, a.dsum_row, a.type));
  n.strips = static_cast<int>(std::min<int64_t>(a.rows, rmsnorm_backward_ctas(n) * rt.sm_count));
  if (a.dweight && a.rows > 0) {
    void *ws = nullptr;
    st = runtime_workspace(rt, stream, kGradientSpace, static_cast<size_t>(n.strips) * a.cols * sizeof(float), &ws);
    if (st != PHOBOS_OK) return st;
    n.partial = static_cast<float *>(ws);
  }
  if (a.rows > 0 && (st = runtime_launched(launch_rmsnorm_backward(n, stream))) != PHOBOS_OK) return st;
  if (a.dweight && (st = runtime_launched(launch_column_sums(n.partial, n.strips, n.cols, a.dweight,
                                                             a.type, 0, stream))) != PHOBOS_OK)
    return st;
  return runtime_finish(rt, stream);
}

}  // namespace

cudaError_t allow_shared_memory(const void *kernel, int bytes) {
  static std::map<std::pair<int, const void *>, int> allowed;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  int &have = allowed[{device, kernel}];
  if (have >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) have = bytes;
  return e;
}

}  // namespace phobos

namespace {

// No C++ exception leaves a C entry point: the only ones here are failures to
// allocate host memory.
template <typename Args, typename F>
phobos_status_t entry(const Args *args, void *stream, F run) {
  if (!args) return PHOBOS_ERR_INVALID_VALUE;
  try {
    return run(*args, static_cast<cudaStream_t>(stream));
  } catch (...) {
    return PHOBOS_ERR_OUT_OF_MEMORY;
  }
}

}  // namespace

extern "C" {

phobos_status_t phobos_linear(const phobos_linear_args_t *args, void *stream) {
  return entry(args, stream, phobos::linear_impl);
}

phobos_status_t phobos_linear_backward(const phobos_linear_backward_args_t *args, void *stream) {
  return entry(args, stream, phobos::linear_backward_impl);
}

phobos_status_t phobos_rmsnorm(const phobos_rmsnorm_args_t *args, void *stream) {
  return entry(args, stream, phobos::rmsnorm_impl);
}

phobos_status_t phobos_rmsnorm_backward(const phobos_rmsnorm_backward_args_t *args, void *stream) {
  return entry(args, stream, phobos::rmsnorm_backward_impl);
}

}  // extern "C"
