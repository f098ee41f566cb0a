// The experts' products in bf16 on the tensor cores.
//
// A tile is 128 features f (256 of a cluster of two blocks) times up to TC of
// c, in tensor memory with a lane a feature and a column a c: features lie next
// to one another in the result, and an expert's last rows cost only as many
// columns as there are (in 16s).  A warp sends 32 features of 32 rows away as one
// box, turned on the way through shared memory; fp32, narrow tiles and results
// whose rows are not whole 16-byte pieces go from registers, 32 neighbours of a
// row at once.
//
// Blocks stay and take tiles in turn.  One warp says which (into a ring in
// shared memory), one loads (TMA, 64 of k a stage), one thread issues the
// matrix instructions, eight warps store; two accumulators, so that a tile is
// stored while the next is multiplied.
//
// Forward and rows' gradients have tiles of one size, taken in a fixed turn.  A
// tile of the weights' gradient is as long as its expert has rows: there the
// largest experts come first and blocks take the next tile when they are done
// (a fixed turn was 1.5 to 2 times as long with experts of a router without
// balance).  Which block computes a tile changes nothing in it.
// Operands lie along k or along the other index, as they are in memory: both
// are layouts that the instruction takes, nothing is transposed.
//
// Ragged ends: rows of forward and rows' gradients are columns of their own, so
// what is loaded of another expert's rows is not stored, and k is cut off by the
// tensor map, which fills with zeros.  In the weights' gradient k runs over the
// expert's rows: there a warp sets to zero what the last 16 rows hold beyond the
// expert's end, in both operands (NaN times zero is NaN).
//
// What bounds it: the tensor cores, and with them the power limit.  131072 rows,
// 2048 -> 768, 32 even experts, 20 calls: forward 230 us (1796 TFLOP/s; a
// library product of the same size in one matrix 219 to 224), rows' gradients
// 241 (229 to 242), weights' gradients 234 (263 to 310), in fp32 257; in seconds
// of it the clock falls and forward takes 261 (the library 246).  The tensor
// pipe is 76 to 83 % active at 32768 rows, DRAM moves the operands once.  What
// carried it there: arrivals between the two blocks without cluster-wide
// ordering (547 -> 295 us), an issuing loop in 32 bits (-> 247), eight storing
// warps (-> 240), loops of whole warps with one thread elected (-> 228), and
// where k is short the boxes (32768 rows, 8 experts, 256 -> 2432: 69 -> 40).
// Few rows are bound by what comes one after the other: 20 rows of 13 experts
// take 11 us, of which reading their 41 MB needs 6, launch, offsets and first
// loads 4, the sum of two slices of k 2.
//
// Long sums: the tensor cores add with rounding towards zero, so sums of values
// of one sign are too small by a part that grows with k: 2.5e-5 at 4096, 7.9e-4
// at 131072 (a half step of bf16 is 3.9e-3).  Sections of k are therefore added
// up by ordinary fp32 additions, in the storing warps' registers: of 512 for
// gradients in fp32, of 4096 for every other result.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "device.cuh"
#include "experts.cuh"
#include "internal.h"
#include "launch.cuh"
#include "operators.cuh"
#include "tcgen05.cuh"

namespace grs {
namespace {

constexpr int MMA_STORING = 8;       // storing warps, two for each quarter of the lanes
constexpr int MMA_THREADS = 128 + 32 * MMA_STORING;
constexpr int MMA_K = 64;            // of k a stage: a swizzled row of bf16
constexpr int MMA_F = 128;           // features of a block
// Stages that the tensor cores add up: of gradients in fp32, and of all else, whose result is rounded to bf16 in the end.
constexpr int MMA_SECTION = 8, MMA_LONG_SECTION = 64;
constexpr int RING = 4;              // tiles told ahead
constexpr int TURN_ROW = 64;         // bytes of a row on its way out: 32 features, with the 64-byte swizzle
constexpr int MMA_SMEM = 227 * 1024;
enum : int { SITE_MMA_ROW = 2 };

__device__ int mma_flags[FLAG_COUNT];

template <int TC, int kCtas>
struct Shape {
  static constexpr int A = MMA_F * MMA_K * 2, B = TC / kCtas * MMA_K * 2, STAGE = A + B;
  static constexpr bool TURNED = TC >= 128;  // results go out by store_turned (narrow tiles would lose a stage to it)
  static constexpr int OUT = TURNED ? MMA_STORING * 32 * TURN_ROW : 0;
  static constexpr int FIXED = 1024 + (GRS_MOE_MAX_EXPERTS + 2) * 4 + 832 + OUT;  // alignment, tiles before each expert, barriers, results
  static constexpr int PER_SM = kCtas == 1 && TC <= 64 ? 2 : 1;  // blocks
  static constexpr int FIT = ((PER_SM == 2 ? 113 * 1024 : MMA_SMEM) - FIXED) / STAGE;
  static constexpr int STAGES = FIT < 10 ? FIT : 10;
  static constexpr int BYTES = STAGES * STAGE + FIXED;
};

template <typename O>
struct MmaArgs {
  const int32_t* offsets;
  O* o;
  int64_t o_c, o_e, o_s;   // elements from one c, one expert, one slice to the next
  int64_t f, c, k;         // extents; an expert's rows in the place of c or k
  int32_t rows, experts, slices;
  int32_t pieces;          // rows of the result are whole 16-byte pieces
  ExpQuit quit;
};

struct Tile {
  int32_t e, f0, slice, c0, c1, k0, k1;  // e < 0: no more
};

template <Product kP, int TC, int kCtas>
struct Tiles {
  const int32_t* offsets;
  const int32_t* list;  // c tiles before each expert's; kWeights: the experts by size (NULL: as they come)
  int64_t f, c, k, ft, ct, total;
  int32_t rows, slices;
  int at_e = 0;

  template <typename O>
  __device__ __forceinline__ Tiles(const MmaArgs<O>& a, const int32_t* list_)
      : offsets(a.offsets), list(list_), f(a.f), c(a.c), k(a.k), rows(a.rows), slices(a.slices) {
    ft = (f + MMA_F * kCtas - 1) / (MMA_F * kCtas);
    ct = kP == Product::kWeights ? (c + TC - 1) / TC : list[a.experts];
    total = kP == Product::kWeights ? ft * ct * slices * a.experts : ft * ct * slices;
  }

  __device__ __forceinline__ Tile at(int64_t t) {
    Tile x;
    int64_t ci = t / ft, c0, c1;
    x.f0 = static_cast<int32_t>((t - ci * ft) * (MMA_F * kCtas));
    const int64_t si = ci / ct;  // kWeights: the slices of an expert, c of each; otherwise c of all experts, slice by slice
    ci -= si * ct;
    if constexpr (kP == Product::kWeights) {
      const int32_t e = static_cast<int32_t>(si / slices);
      x.slice = static_cast<int32_t>(si - int64_t(e) * slices);
      x.e = list != nullptr ? list[e] : e;
      c0 = ci * TC;
      c1 = c;
    } else {
      x.slice = static_cast<int32_t>(si);
      if (list[at_e] > ci) at_e = 0;
      while (list[at_e + 1] <= ci) ++at_e;
      x.e = at_e;
    }
    const ExpertRows r(offsets, x.e, rows);
    if constexpr (kP == Product::kWeights) {
      x.k0 = r.from;
      x.k1 = r.to;
    } else {
      c0 = r.from + (ci - list[x.e]) * TC;
      c1 = r.to;
      x.k0 = 0;
      x.k1 = static_cast<int32_t>(k);
    }
    if (slices > 1) {
      const int64_t n = slice_length<MMA_SECTION * MMA_K>(x.k1 - x.k0, slices), from = x.k0 + x.slice * n, to = from + n;
      x.k0 = from < x.k1 ? static_cast<int32_t>(from) : x.k1;
      x.k1 = to < x.k1 ? static_cast<int32_t>(to) : x.k1;
    }
    x.c0 = static_cast<int32_t>(c0);
    x.c1 = static_cast<int32_t>(c1 < c0 + TC ? c1 : c0 + TC);
    return x;
  }
};

// The experts from the one with the most rows on, by a block of at least as many threads.
__device__ __forceinline__ void by_size(const int32_t* offsets, int32_t experts, int32_t* order) {
  int32_t* size = order + experts;
  const int e = threadIdx.x;
  if (e < experts) size[e] = __ldg(offsets + e + 1) - __ldg(offsets + e);
  __syncthreads();
  if (e < experts) {
    const int32_t n = size[e];
    int rank = 0;
    for (int i = 0; i < experts; ++i) rank += size[i] > n || (size[i] == n && i < e);
    order[rank] = e;
  }
}

__device__ __forceinline__ void store_piece(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 shared_piece(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// 32 columns, a lane a feature, to rows `ld` elements apart, the first n of
// them; `on`: there is such a feature.
template <typename O>
__device__ __forceinline__ void store_columns(O* o, int64_t ld, const uint32_t (&v)[32], int n, bool on) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (on && j < n) *o = from_float<O>(__uint_as_float(v[j]));
    o += ld;
  }
}

// The same 32 x 32 results in bf16, where rows of the result are whole 16-byte
// pieces: rounded as fragments and transposed on the way to the warp's own
// swizzled box in shared memory, which leaves as one copy.  With `all` false (a
// row behind the first n is another expert's) its rows go as 16-byte pieces,
// `o` this thread's piece of row t / 4, `on`: there are its eight features.
// us with 32768 rows, 8 experts, 256 -> 2432 in bf16 (26 of memory, 22 of matrix
// instructions): a 16-bit store a feature and row 69; pairs by shuffles longer
// still; pieces only 43; boxes 40.  Boxes of 16 rows of all 128 features, filled
// by four warps together, 57; copies of single rows 114.
__device__ __forceinline__ void store_turned(uint32_t from, uint32_t place, const CUtensorMap* map, int32_t f, int32_t c, int32_t e, bool all,
                                             uint16_t* o, int64_t ld, int n, bool on) {
  const int t = threadIdx.x & 31;
  uint32_t v[2][16];
  tmem_load_fragments(from, v[0]);
  tmem_load_fragments(from + (16u << 16), v[1]);
  tmem_wait_load();
  bulk_wait_read();
  __syncwarp();  // the place has been read
  const uint32_t to = place + ((t >> 4) * 8 + (t & 7)) * TURN_ROW + ((t >> 3 ^ t >> 1) & 1) * 16, flip = (t >> 2 & 1) * 32;
#pragma unroll
  for (int l = 0; l < 2; ++l)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t m[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        m[q] = to_bf16_pair(make_float2(__uint_as_float(v[l][8 * k + 2 * q]), __uint_as_float(v[l][8 * k + 2 * q + 1])));
      store_transposed(to + k * 16 * TURN_ROW + (l * 32 ^ flip), m[0], m[1], m[2], m[3]);
    }
  if (all) {
    fence_async_shared();
    __syncwarp();
    if (t == 0) {
      tma_store(map, place, f, c, e);
      bulk_commit();
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = (t >> 2) + 8 * q;
    const uint4 w = shared_piece(place + row * TURN_ROW + ((t ^ t >> 3) & 3) * 16);
    if (on && row < n) *reinterpret_cast<uint4*>(o + 8 * q * ld) = w;
  }
}

// kLong: k may be more than MMA_LONG_SECTION stages.  Short k, which stores bound, does without the registers of its sums
// (32768 rows, 8 experts, 256 -> 2432: 39.0 us, with them 39.4).
template <Product kP, int TC, int kCtas, typename O, bool kLong>
__global__ void __launch_bounds__(MMA_THREADS, (Shape<TC, kCtas>::PER_SM))
    exp_mma_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_o, const __grid_constant__ MmaArgs<O> a) {
  using S = Shape<TC, kCtas>;
  constexpr bool kWeights = kP == Product::kWeights, kASK = kP == Product::kForward, kBSK = !kWeights;  // operands along k
  constexpr bool kShort = kWeights && sizeof(O) == 4;
  constexpr int32_t SECTION = kShort ? MMA_SECTION : kLong ? MMA_LONG_SECTION : INT32_MAX;
  constexpr uint32_t COLUMNS = 2 * TC;  // two accumulators
  constexpr uint32_t TMEM = COLUMNS <= 64 ? 64 : COLUMNS <= 128 ? 128 : COLUMNS <= 256 ? 256 : 512;
  static_assert(COLUMNS <= 512, "tensor memory has 512 columns");
  static_assert(!kWeights || TC / kCtas % 64 == 0, "operands across k come in 64s");
  extern __shared__ uint8_t smem[];
  uint8_t* stages = smem + (1024 - (smem_addr(smem) & 1023)) % 1024;
  uint8_t* out = stages + S::STAGES * S::STAGE;
  int32_t* first = reinterpret_cast<int32_t*>(out + S::OUT);
  uint64_t* full = reinterpret_cast<uint64_t*>(first + ((GRS_MOE_MAX_EXPERTS + 1 + 1) & ~1));
  uint64_t *empty = full + S::STAGES, *tail = empty + S::STAGES, *done = tail + S::STAGES, *taken = done + 2;
  uint64_t *told = taken + 2, *heard = told + RING, *answered = heard + RING, *asked = answered + 2;
  uint4* answers = reinterpret_cast<uint4*>((reinterpret_cast<uintptr_t>(asked + 2) + 15) & ~uintptr_t(15));
  Tile* ring = reinterpret_cast<Tile*>(answers + 2);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(ring + RING);
  volatile int* abort = reinterpret_cast<int*>(tmem_at + 1);

  const int lane = threadIdx.x & 31, w = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const uint32_t rank = kCtas == 1 ? 0 : cluster_rank();
  if (threadIdx.x == 0) {
    prefetch_map(&map_a);
    prefetch_map(&map_b);
    if (a.pieces) prefetch_map(&map_o);
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(full + s, kCtas);
      mbar_init(empty + s, 1);
      mbar_init(tail + s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(done + i, 1);
      mbar_init(taken + i, MMA_STORING * kCtas);
    }
    for (int i = 0; i < RING; ++i) {
      mbar_init(told + i, 1);
      mbar_init(heard + i, MMA_STORING + 1 + (rank == 0) + kWeights);  // storing warps, the loading one, the issuing thread, the clearing warp
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(answered + i, 1);
      mbar_init(asked + i, kCtas);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (w == 1) tmem_alloc<kCtas>(tmem_at, TMEM);
  pdl_wait();
  if constexpr (kWeights) {
    if (a.experts <= MMA_THREADS) by_size(a.offsets, a.experts, first);
  } else {
    pdl_trigger();  // (kWeights has blocks that never begin)
    group_prefix<TC, MMA_THREADS>(a.offsets, a.experts, a.rows, first);
  }
  tmem_before_sync();
  if constexpr (kCtas == 2) cluster_sync();
  else __syncthreads();
  tmem_after_sync();
  const uint32_t tmem = *tmem_at;

  // The next tile of the ring, for a whole warp; false: a wait gave up.
  uint32_t slot = 0, slot_parity = 0;
  auto wait_for = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, mma_flags, abort); };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_for(bar, parity)) != 0; };
  auto next_tile = [&](Tile& x) {
    if (!wait_all(told + slot, slot_parity)) return false;
    const int32_t* r = reinterpret_cast<const int32_t*>(ring + slot);
    const int32_t v = lane < static_cast<int>(sizeof(Tile) / 4) ? r[lane] : 0;
    x.e = __shfl_sync(0xffffffffu, v, 0);
    x.f0 = __shfl_sync(0xffffffffu, v, 1);
    x.slice = __shfl_sync(0xffffffffu, v, 2);
    x.c0 = __shfl_sync(0xffffffffu, v, 3);
    x.c1 = __shfl_sync(0xffffffffu, v, 4);
    x.k0 = __shfl_sync(0xffffffffu, v, 5);
    x.k1 = __shfl_sync(0xffffffffu, v, 6);
    if (elected()) mbar_arrive(heard + slot);
    if (++slot == RING) {
      slot = 0;
      slot_parity ^= 1;
    }
    return true;
  };

  if (w == 0) {
    // ------------------------------------------------------------- loads
    uint32_t s = 0, parity = 1;
    const uint32_t stages_at = smem_addr(stages);
    // Both blocks' loads are counted by the first one's barriers.
    const uint32_t full_at = kCtas == 1 || rank == 0 ? smem_addr(full) : peer_addr(smem_addr(full), 0);
    bool ok = true;
    int32_t left = static_cast<int32_t>(blockIdx.x) == a.quit.quitter ? a.quit.tile : -1;
    while (ok) {
      Tile x;
      ok = next_tile(x);
      if (!ok || x.e < 0) break;
      if (left-- == 0) {  // the self-test: as if a wait had given up
        if (elected()) {
          atomicOr(mma_flags + FLAG_TIMEOUT, 1);
          *abort = 1;
        }
        __syncwarp();
        break;
      }
      const int32_t f0 = x.f0 + static_cast<int32_t>(rank) * MMA_F;
      // Columns of this block: half of the instruction's.
      const int32_t half = (x.c1 - x.c0 + 15) / 16 * 16 / kCtas;
      const int32_t c0 = x.c0 + static_cast<int32_t>(rank) * half;
      for (int32_t k = x.k0; k < x.k1; k += MMA_K) {
        const bool last = kWeights && x.k1 - k < MMA_K && (x.k1 - k) % 16 != 0;
        ok = wait_all(empty + s, parity);
        if (!ok) break;
        const uint32_t to = stages_at + s * S::STAGE, bar = full_at + s * 8;
        const uint32_t on = last ? smem_addr(tail + s) : bar;
        if (elected()) {
          if (last) mbar_arrive_expect_tx(tail + s, S::STAGE);
          else if (kCtas == 1) mbar_arrive_expect_tx(full + s, S::STAGE);
          else remote_arrive_expect_tx(bar, S::STAGE);
          if constexpr (kP == Product::kForward) {
            tma_load<kCtas>(to, &map_a, k, f0, x.e, on);
          } else if constexpr (kP == Product::kRows) {
            tma_load<kCtas>(to, &map_a, f0, k, x.e, on);
            tma_load<kCtas>(to + 8192, &map_a, f0 + 64, k, x.e, on);
          } else {
            tma_load<kCtas>(to, &map_a, f0, k, on);
            tma_load<kCtas>(to + 8192, &map_a, f0 + 64, k, on);
          }
          if constexpr (!kWeights) {
            tma_load<kCtas>(to + S::A, &map_b, k, c0, on);
          } else {
#pragma unroll
            for (int i = 0; i < TC / kCtas / 64; ++i) tma_load<kCtas>(to + S::A + i * 8192, &map_b, c0 + i * 64, k, on);
          }
        }
        __syncwarp();
        if (++s == S::STAGES) {
          s = 0;
          parity ^= 1;
        }
      }
    }
  } else if (w == 1) {
    // ---------------------------------------------------------- products
    if (rank == 0) {
      uint32_t s = 0, parity = 0, acc = 0, acc_parity = 1;
      const uint32_t a_at = operand<kASK>(smem_addr(stages), 8192), b_at = operand<kBSK>(smem_addr(stages) + S::A, 8192);
      bool ok = true;
      while (ok) {
        Tile x;
        ok = next_tile(x);
        if (!ok || x.e < 0) break;
        const uint32_t n = (static_cast<uint32_t>(x.c1 - x.c0) + 15) / 16 * 16;
        const uint32_t desc = product_desc(kASK, kBSK, MMA_F * kCtas, n);
        int32_t rest = x.k1 - x.k0;
        while (rest > 0 && ok) {
          ok = wait_all(taken + acc, acc_parity);
          if (!ok) break;
          tmem_after_sync();
          const uint32_t d = tmem + acc * TC;
          int32_t section = SECTION;
          bool add = false;
          for (; rest > 0 && section > 0; rest -= MMA_K, --section) {
            ok = wait_all(full + s, parity);
            if (!ok) break;
            tmem_after_sync();
            const uint32_t da = a_at + s * (S::STAGE >> 4), db = b_at + s * (S::STAGE >> 4);
            if (elected()) {
              mma<kCtas>(d, da, db, desc, add);
#pragma unroll
              for (int i = 1; i < MMA_K / 16; ++i)
                if (rest > 16 * i) mma<kCtas>(d, da + i * operand_step<kASK>, db + i * operand_step<kBSK>, desc, true);
              mma_commit<kCtas>(empty + s);
            }
            __syncwarp();
            add = true;
            if (++s == S::STAGES) {
              s = 0;
              parity ^= 1;
            }
          }
          if (!ok) break;
          if (elected()) mma_commit<kCtas>(done + acc);
          __syncwarp();
          acc ^= 1;
          if (acc == 0) acc_parity ^= 1;
        }
      }
    }
  } else if (w == 2) {
    // ------------------------------------------------------------- tiles
    if (lane == 0) {
      Tiles<kP, TC, kCtas> tiles(a, kWeights && a.experts > MMA_THREADS ? nullptr : first);
      int64_t t = blockIdx.x / kCtas;
      uint32_t empty_parity = 1, q = 0, q_parity = 0;
      bool ok = true;
      while (ok) {
        // Ask for the tile after this one while this one is told.
        bool more = t >= 0 && t < tiles.total;
        if (kWeights && more) {
          mbar_arrive_expect_tx(answered + q, 16);
          if (rank == 0) {
            ok = wait_for(asked + q, q_parity ^ 1);  // both blocks have read what was there
            if (!ok) break;
            ask_cluster<kCtas>(answers + q, answered + q);
          }
        }
        ok = wait_for(heard + slot, empty_parity);
        if (!ok) break;
        Tile x;
        x.e = -1;
        if (more) x = tiles.at(t);
        ring[slot] = x;
        mbar_arrive(told + slot);
        if (++slot == RING) {
          slot = 0;
          empty_parity ^= 1;
        }
        if (!more) break;
        if constexpr (kWeights) {
          ok = wait_for(answered + q, q_parity);
          if (!ok) break;
          t = cluster_given(answers + q);
          if (t >= 0) t /= kCtas;
          fence_async_shared();
          if (kCtas == 1) mbar_arrive(asked + q);
          else remote_release(rank == 0 ? smem_addr(asked + q) : peer_addr(smem_addr(asked + q), 0));
          q ^= 1;
          if (q == 0) q_parity ^= 1;
        } else {
          t += gridDim.x / kCtas;
        }
      }
    }
  } else if (w == 3 && kWeights) {
    // ------------------------------------------------------- ragged ends
    // What the last 16 rows of an expert hold of others', once it is there: cleared, then counted as loaded.
    const uint32_t full_at = kCtas == 1 || rank == 0 ? smem_addr(full) : peer_addr(smem_addr(full), 0);
    uint32_t s = 0, parities = 0;  // the stage of the tile's first block; a bit for each stage's `tail`
    bool ok = true;
    while (ok) {
      Tile x;
      ok = next_tile(x);
      if (!ok || x.e < 0) break;
      const int32_t n = x.k1 - x.k0, blocks = (n + MMA_K - 1) / MMA_K, valid = n % MMA_K;
      const uint32_t last = (s + blocks + S::STAGES - 1) % S::STAGES;
      s = (s + blocks) % S::STAGES;
      if (valid % 16 == 0) continue;
      ok = wait_all(tail + last, parities >> last & 1);
      if (!ok) break;
      parities ^= 1u << last;
      const int32_t bad = (16 - valid % 16) * 8;  // 16-byte chunks to clear, in each 64 of f or c
      uint8_t* stage = stages + last * S::STAGE;
      for (int32_t i = lane; i < bad * (S::STAGE / 8192); i += 32)
        *reinterpret_cast<uint4*>(stage + i / bad * 8192 + valid * 128 + i % bad * 16) = make_uint4(0, 0, 0, 0);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        if (kCtas == 1) mbar_arrive(full + last);
        else remote_release(full_at + last * 8);
      }
    }
  } else if (w >= 4) {
    // ------------------------------------------------------------ results
    uint32_t taken_so_far = 0;  // accumulators: their turn and their barriers' parity
    bool ok = true;
    const int quarter = w & 3, half = (w - 4) >> 2;  // 32 lanes; every second 32 columns
    const uint32_t from = tmem + (uint32_t(quarter) << 21) + 32 * half;
    const bool turned = S::TURNED && sizeof(O) == 2 && a.pieces != 0;
    const uint32_t place = smem_addr(out) + (w - 4) * 32 * TURN_ROW;
    while (ok) {
      Tile x;
      ok = next_tile(x);
      if (!ok || x.e < 0) break;
      const int32_t blocks = (x.k1 - x.k0 + MMA_K - 1) / MMA_K, width = static_cast<int32_t>(a.f);
      const int32_t f = x.f0 + static_cast<int32_t>(rank) * MMA_F + quarter * 32 + lane;
      const int n = x.c1 - x.c0;
      O* o = a.o + x.e * a.o_e + x.slice * a.o_s + int64_t(x.c0) * a.o_c + f;
      const bool rows_on = GRS_CHECK(kWeights || (x.c0 >= 0 && x.c1 <= a.rows), mma_flags, SITE_MMA_ROW), on = rows_on && f < width;
      const int32_t sections = blocks / SECTION + (blocks % SECTION != 0);
      uint32_t acc;
      auto begin = [&] {
        acc = taken_so_far & 1;
        ok = wait_all(done + acc, taken_so_far >> 1 & 1);
        tmem_after_sync();
        return ok;
      };
      auto end = [&] {
        tmem_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (kCtas == 1) mbar_arrive(taken + acc);
          else remote_arrive(peer_addr(smem_addr(taken + acc), 0));
        }
        ++taken_so_far;
      };
      if (kShort || (kLong && sections > 1)) {
        // The thread's columns are added up in its registers, section by section, eight at a time: with 16 the registers
        // run over, and a kernel with a stack took 0.5 to 1 us more (5000 rows, 32 experts, 1024 -> 1024, 21.9 to 22.9).
        constexpr int PARTS = TC >= 64 ? TC / 64 : 1, EACH = TC < 32 ? TC : 32;
        float sum[PARTS][EACH];
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
#pragma unroll
          for (int j = 0; j < EACH; ++j) sum[p][j] = 0.0f;
        for (int32_t i = 0; i < sections; ++i) {
          if (!begin()) break;
#pragma unroll
          for (int p = 0; p < PARTS * EACH / 8; ++p) {
            const int part = p * 8 / EACH, q = p * 8 % EACH;
            if (64 * part + 32 * half + q >= n) break;
            uint32_t v[8];
            tmem_load8(from + acc * TC + 64 * part + q, v);
            tmem_wait_load();
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[part][q + j] = __fadd_rn(sum[part][q + j], __uint_as_float(v[j]));
          }
          end();
        }
        if (!ok) break;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
          const int j0 = 64 * p + 32 * half;
          if (j0 >= n) break;
          O* q = o + j0 * a.o_c;
#pragma unroll
          for (int j = 0; j < EACH; ++j) {
            if (on && j0 + j < n) *q = from_float<O>(sum[p][j]);
            q += a.o_c;
          }
        }
        __syncwarp();
      } else if (sections == 1) {
        if (!begin()) break;
        for (int j0 = 32 * half; j0 < n; j0 += 64) {
          if constexpr (S::TURNED && sizeof(O) == 2) {
            if (turned) {
              const int piece = (lane & 3) * 8 - lane;  // from this lane's feature to its piece's
              const int32_t f0 = f - lane;
              // Rows behind the result's and features behind its width are cut off by the map.
              store_turned(from + acc * TC + j0 - 32 * half, place, &map_o, f0, x.c0 + j0, kWeights ? x.e : 0,
                           rows_on && f0 < a.f && (kWeights || n - j0 >= 32), o + piece + (j0 + (lane >> 2)) * a.o_c, a.o_c, n - j0,
                           rows_on && f + piece < a.f);
              continue;
            }
          }
          uint32_t v[32];
          tmem_load32(from + acc * TC + j0 - 32 * half, v);
          tmem_wait_load();
          store_columns(o + j0 * a.o_c, a.o_c, v, n - j0, on);
          __syncwarp();
        }
        end();
      } else {  // an expert without rows, a slice without k
        if (kWeights && turned) {
          const int32_t f0 = f - lane;
          bulk_wait_read();
          __syncwarp();
          for (int i = lane; i < 32 * TURN_ROW / 16; i += 32) store_piece(place + i * 16, make_uint4(0, 0, 0, 0));
          fence_async_shared();
          __syncwarp();
          if (lane == 0 && f0 < a.f) {
            for (int j0 = 32 * half; j0 < n; j0 += 64) tma_store(&map_o, place, f0, x.c0 + j0, x.e);
            bulk_commit();
          }
        } else if (on) {
          for (int j = half; j < n; j += 2) o[j * a.o_c] = from_float<O>(0.0f);
        }
        __syncwarp();
      }
    }
    bulk_wait();
  }
  // A wait that gave up leaves copies and products under way: they end by themselves.  The cluster's other block, which
  // misses this one's loads, arrivals or answers, gives up too, at the limit.
  if (*abort) {
    const uint64_t since = global_ns();
    while (global_ns() - since < 200000) {
    }
  }
  __syncwarp();
  tmem_before_sync();
  if constexpr (kCtas == 2) cluster_sync();
  else __syncthreads();
  tmem_after_sync();
  if (w == 1) tmem_free<kCtas>(tmem, TMEM);
}

// ------------------------------------------------------------------- host
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
    return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiled>(p) : nullptr;
  }();
  return f;
}

// A bf16 tensor of `n` dimensions, its boxes `width` wide: 64 or 32, a row of the 128 or 64-byte swizzle.
bool make_map(CUtensorMap* m, const void* p, int n, const int64_t (&dims)[3], const int64_t (&ld)[2], int box_rows, int width = 64) {
  const EncodeTiled f = encode_tiled();
  if (f == nullptr) return false;
  cuuint64_t d[3], stride[2];
  cuuint32_t box[3] = {static_cast<cuuint32_t>(width), static_cast<cuuint32_t>(box_rows), 1}, one[3] = {1, 1, 1};
  for (int i = 0; i < 3; ++i) d[i] = static_cast<cuuint64_t>(dims[i]);
  for (int i = 0; i < 2; ++i) stride[i] = static_cast<cuuint64_t>(ld[i]) * 2;
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(n), const_cast<void*>(p), d, stride, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Product kP, int TC, int kCtas, typename O, bool kLong>
cudaError_t mma_launch_as(const grs_experts* s, const ExpLd& ld, const void* xs, const void* w, const void* dys, const int32_t* offsets,
                          void* o, int64_t o_ld, const ExpSlices& sl, const ExpQuit& quit, void* stream) {
  using S = Shape<TC, kCtas>;
  const int64_t in = s->in_features, out = s->out_features;
  CUtensorMap ma, mb, mo{};
  MmaArgs<O> a{};
  a.offsets = offsets;
  a.slices = sl.n;
  a.o = static_cast<O*>(sl.n > 1 ? static_cast<void*>(sl.parts) : o);
  a.o_c = sl.n > 1 ? sl.ld : o_ld;
  a.o_s = sl.distance;
  a.rows = static_cast<int32_t>(s->rows);
  a.experts = s->experts;
  a.quit = quit;
  bool fine;
  int64_t tiles;  // at most
  if constexpr (kP == Product::kWeights) {
    fine = make_map(&ma, xs, 2, {in, s->rows, 1}, {ld.x, 0}, 64) && make_map(&mb, dys, 2, {out, s->rows, 1}, {ld.y, 0}, 64);
    a.f = in, a.c = out, a.o_e = out * a.o_c;
    tiles = s->experts * ((out + TC - 1) / TC);
  } else {
    constexpr bool fwd = kP == Product::kForward;
    fine = make_map(&ma, w, 3, {in, out, s->experts}, {ld.w, out * ld.w}, fwd ? MMA_F : 64) &&
           make_map(&mb, fwd ? xs : dys, 2, {fwd ? in : out, s->rows, 1}, {fwd ? ld.x : ld.y, 0}, TC / kCtas);
    a.f = fwd ? out : in, a.k = fwd ? in : out;
    tiles = s->rows / TC + (s->rows < s->experts ? s->rows : s->experts);
  }
  if (!fine) return cudaErrorInvalidValue;
  if (S::TURNED && sizeof(O) == 2 && api_aligned(o, 16) && a.o_c % 8 == 0 && a.f % 8 == 0)
    a.pieces = make_map(&mo, o, 3, {a.f, kP == Product::kWeights ? a.c : s->rows, kP == Product::kWeights ? s->experts : 1},
                        {a.o_c, kP == Product::kWeights ? a.o_e : a.o_c}, 32, 32);
  const int64_t step = MMA_F * kCtas;
  tiles *= (a.f + step - 1) / step * sl.n;
  // Weights: a cluster for each tile, of which those that run take over the others' (ask_cluster).
  const int64_t at_once = kP == Product::kWeights ? INT32_MAX / kCtas : S::PER_SM * 152 / kCtas;
  if (kP == Product::kWeights && tiles > at_once) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>((tiles < at_once ? tiles : at_once) * kCtas);
  const cudaError_t e = allow_smem<exp_mma_kernel<kP, TC, kCtas, O, kLong>>(S::BYTES);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(exp_mma_kernel<kP, TC, kCtas, O, kLong>, kCtas, dim3(grid), dim3(MMA_THREADS), S::BYTES, stream, ma, mb, mo, a);
}

template <Product kP, int TC, int kCtas, typename O>
cudaError_t mma_launch(const grs_experts* s, const ExpLd& ld, const void* xs, const void* w, const void* dys, const int32_t* offsets,
                       void* o, int64_t o_ld, const ExpSlices& sl, const ExpQuit& quit, void* stream) {
  constexpr bool kShort = kP == Product::kWeights && sizeof(O) == 4;  // has sections of its own
  // An expert may have all of the rows.
  const int64_t k = kP == Product::kWeights ? s->rows : kP == Product::kForward ? s->in_features : s->out_features;
  if (!kShort && slice_length<MMA_SECTION * MMA_K>(k, sl.n) > MMA_LONG_SECTION * MMA_K)
    return mma_launch_as<kP, TC, kCtas, O, !kShort>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
  return mma_launch_as<kP, TC, kCtas, O, false>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
}

template <Product kP, int TC>
cudaError_t mma_narrow(const grs_experts* s, const ExpLd& ld, const void* xs, const void* w, const void* dys, const int32_t* offsets, void* o,
                       int64_t o_ld, const ExpSlices& sl, const ExpQuit& quit, void* stream) {
  if (sl.n > 1) return mma_launch<kP, TC, 1, float>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
  return mma_launch<kP, TC, 1, uint16_t>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
}

template <Product kP>
cudaError_t mma_rows(int columns, const grs_experts* s, const ExpLd& ld, const void* xs, const void* w, const void* dys, const int32_t* offsets,
                     void* o, int64_t o_ld, const ExpSlices& sl, const ExpQuit& quit, void* stream) {
  switch (columns) {
    case 16: return mma_narrow<kP, 16>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
    case 64: return mma_narrow<kP, 64>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
    case 128: return mma_narrow<kP, 128>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
    default: return mma_launch<kP, 256, 2, uint16_t>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
  }
}

}  // namespace

cudaError_t experts_mma_flags(int** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), mma_flags); }

ExpTiles experts_mma_tiles(Product p, const grs_experts* s) {
  const int64_t in = s->in_features, out = s->out_features, least = s->rows < s->experts ? s->rows : s->experts;
  auto up = [](int64_t n, int64_t to) { return (n + to - 1) / to; };
  ExpTiles t;
  if (p == Product::kWeights) {
    // Few large tiles are shared badly, small ones read more for each product.  us with small and large ones, even experts
    // and (in brackets) a skewed router's: 12 experts, 1024 -> 520 (144 large tiles), 1500 rows 8.3 and 9.6 (9.6, 10.7),
    // 3000 10.3 and 10.5 (12.8, 14.0), 8000 17.7 and 15.2 (17.8, 16.9); 8 experts, 2048 -> 768 (192), 4000 rows 17.4 and
    // 16.0 (17.7, 17.2); 32 experts, 768 -> 512 (192), 4000 rows 10.2 and 11.6 (12.3, 13.9), 12000 15.3 and 14.2 (18.2,
    // 19.2), 16000 18.0 and 16.7 (20.4, 21.7).  Even experts would have large ones from a mean of 250 to 400 rows on, skewed
    // ones later: 448 lies between.  Nor are 256 features taken where a quarter of what they multiply is not there: 32
    // experts, 36000 rows, 384 -> 768 24.7 and 26.8, 128 -> 2048 32.1 and 38.1.
    const int64_t large = s->experts * up(in, 256) * up(out, 256), mean = s->rows / s->experts;
    t.columns = large < 76 || (large < 4 * 76 && mean < 448) || 2 * up(in, 256) * 3 >= up(in, 128) * 4 ? 128 : 256;
    t.n = t.columns == 256 ? large : s->experts * up(in, 128) * up(out, 128);
    t.k = s->rows / s->experts;
  } else {
    // Columns by the rows that an expert has in the mean, those outside all experts' counted too (the host does not know
    // them).  Forward, 2048 -> 768, 32 even experts, us with 16, 64, 128 and 256 (two blocks), in brackets those of a skewed
    // router: 20 rows 12.4, 17.8, 20.1, 21.4; 512 rows 19.9, 19.7, 21.7, 21.8 (20.2, 17.2, 22.6, 21.6); 2048 rows 30.3,
    // 21.9, 24.8, 25.5 (29.6, 22.2, 24.2, 27.5); 2560 rows 35.9, 27.8, 25.5, 26.0 (36.0, 28.7, 24.7, 26.6); 4096 rows 49.1,
    // 28.9, 26.9, 27.4 (49.5, 28.4, 24.9, 28.9); 6000 rows 64.1, 29.9, 31.3, 30.0 (63.9, 35.3, 30.8, 29.0); 12000 rows
    // (120.4, 51.4, 45.0, 37.8); 131072 rows 1228, 421, 329, 237.  So 128 take over from 64 between means of 64 and 80, and
    // 256 from 128 between 128 and 190; the rule takes the lower ends, where forward of exactly 64 rows an expert is 13 %
    // and of 128 2 to 16 % longer than it could be (rows' gradients 5 and 3 %, skewed not at all).  256 features where there
    // are half of them: 32 experts, 36000 rows, 2048 -> 128 40.8, 128 columns 31.1.
    const int64_t f = p == Product::kForward ? out : in, mean = s->rows / s->experts;
    const int64_t large = (s->rows / 256 + least) * up(f, 256);
    t.columns = mean >= 128 && large >= 76 && f > 128 ? 256 : mean >= 64 ? 128 : mean >= 16 ? 64 : 16;
    t.n = t.columns == 256 ? large : (s->rows / t.columns + least) * up(f, 128);
    t.k = p == Product::kForward ? in : out;
  }
  return t;
}

cudaError_t experts_mma(Product p, const grs_experts* s, const ExpLd& ld, const void* xs, const void* w, const void* dys,
                        const int32_t* offsets, void* o, int64_t o_ld, const ExpSlices& sl, const ExpQuit& quit, void* stream) {
  const int columns = experts_mma_tiles(p, s).columns;
  if (p == Product::kForward) return mma_rows<Product::kForward>(columns, s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
  if (p == Product::kRows) return mma_rows<Product::kRows>(columns, s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
  const bool fp32 = s->grad_dtype == GRS_DTYPE_FP32 || sl.n > 1;
  if (columns == 128) {
    if (fp32) return mma_launch<Product::kWeights, 128, 1, float>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
    return mma_launch<Product::kWeights, 128, 1, uint16_t>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
  }
  if (fp32) return mma_launch<Product::kWeights, 256, 2, float>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
  return mma_launch<Product::kWeights, 256, 2, uint16_t>(s, ld, xs, w, dys, offsets, o, o_ld, sl, quit, stream);
}

}  // namespace grs
