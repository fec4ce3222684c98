// Launchers of the many-row kernels of the low-rank adapters (lowrank_tc.cu).
#pragma once

#include <type_traits>

#include "kernels.h"
#include "tc.h"
#include "tc_internal.h"

namespace qg {

constexpr int kChunkRows = 512;            // rows of one adapter that one block sums
constexpr int64_t kSortAdapters = 4096;    // adapters that get a block each in the sort
constexpr int kSlots = 128;                // adapters of one call that the fused product holds copies of

// Adapters of one row tile that it multiplies, at most.  A k-block per adapter
// beats its rows' turn in the fix: 8192 rows of 4096 x 14336 in random order,
// 128 adapters of rank 64: 3.2 ms, with at most 64 per tile 4.8 ms.
constexpr int kExtPerTile = kSlots;
static_assert(kExtPerTile <= 128, "a place in the list is a signed char");

// Rows in adapter order (device tables in the workspace).
struct AdapterRows {
  int32_t* row;       // [M] rows that have an adapter
  int32_t* offset;    // [G + 1]
};
// Adapter g's chunks of kChunkRows rows have the numbers from first_chunk(g)
// on: at least as many numbers as chunks, since ceil(n / c) <= floor((o + n) /
// c) - floor(o / c) + 1.  The partial sums of an adapter of several chunks (n
// > c rows, so that ceil(n / c) <= floor(n / (c / 2))) start at first_part.
__host__ __device__ __forceinline__ int first_chunk(int offset, int g) { return offset / kChunkRows + g; }
__host__ __device__ __forceinline__ int first_part(int offset) { return offset / (kChunkRows / 2); }
inline int64_t lowrank_max_chunks(const LowRankArgs& l) { return l.M / kChunkRows + l.G; }
inline int64_t lowrank_max_parts(const LowRankArgs& l) { return l.M / (kChunkRows / 2) + 1; }
// The sort's bitmap of the rows lives in shared memory.
inline bool lowrank_sort_supported(const LowRankArgs& l) {
  return l.G >= 1 && l.G <= kSortAdapters && l.M <= (1 << 20);
}

// A factor becomes an MMA operand as the sum of two T values, side by side along
// the contraction: hi = T(z) and what it leaves.  In the fused product that
// doubles the factor's columns, which costs nothing up to rank 32 (a k-block is
// 64 columns, the rest of it zeros) and a k-block per adapter, tile and 64
// ranks above.  Above rank 32 a bf16 factor is therefore T(z) alone there, for an
// error of Y and dX of at most sqrt(2) of their own rounding; f16 keeps both
// parts at any rank, since T(z) alone is off by 2^-25 however small z is.
// 8192 x 4096 x 14336, rank 64, one part and two: 0.69 and 0.70 ms with 12
// adapters in runs, 3.06 and 4.42 ms with 128 in random order.
inline bool lowrank_two_parts(const LowRankArgs& l) { return l.dtype == MM_F16 || l.R <= 32; }
// What hi leaves is at most 2^-12 of z: in f16 it is taken times 2^7, against
// adapters times 2^-7, and is then off by 2^-32.
constexpr float kF16LoScale = 128.f;

// Tables of the fused product Y = A B + z b (device, in the workspace).
struct FusedTables {
  int32_t* head;         // [0] slots in use, [1] whether the fix has work
  int32_t* slot_of;      // [G] of the adapters in use
  int32_t* adapter_of;   // [kSlots]
  int32_t* bad;          // [kSlots] the adapter holds a non-finite value
  int32_t* row_entry;    // [M] place in the row tile's list, -1: not in it
  int32_t* ext_count;    // [row tiles]
  int32_t* ext_slot;     // [row tiles][per_tile]
  int32_t* row_c;        // [M] the product adds what Y holds (written where head[1] is set)
  uint8_t* wide;         // [groups of 64 ranks][M] the row's factor has values that T has no finite number for
};
struct FusedLayout {
  int64_t slots, per_tile, f_ld, c_ld;
  int64_t z_ld;          // ranks rounded up to 8 (zeros): z's row, half a row of zt
  int64_t k_rows;        // rows of an adapter's copy: its ranks, or z_ld for each part
  bool two;              // lowrank_two_parts
  size_t z, head, slot_of, adapter_of, bad, row_entry, ext_count, ext_slot, row_c, wide, factors, copy, total;
};
FusedLayout lowrank_fused_layout(const LowRankArgs& l, int64_t N);
FusedTables lowrank_fused_tables(const FusedLayout& w, char* ws);
bool lowrank_fused_supported(const LowRankArgs& l, const GemmArgs& g, LowRankProduct* plan);

// One or two factors, scaled, each as z [M, z_ld] (fp32, zeros past R; for the
// fused product, with its `wide`) and as zt [M, 2, z_ld] (hi and lo, zeros past
// R; for the gradients), NULL where not wanted.  A row of an f16 zt is divided
// by 2^e, e = zt_exp[rank / 64, row], so that its largest value is in [2^14,
// 2^15).  Rows without adapter are not written.  The same launch makes the
// fused product's slots and the sorted rows where asked for.
// `map` receives x's tensor map.
bool lowrank_shrink_tiles_supported(const LowRankArgs& l, const void* x, int64_t x_rs, int64_t x_cs, int64_t C,
                                    int64_t a_cs, int64_t a_rs, OperandPlan* map);
struct LowRankShrink {
  const OperandPlan* map; int64_t C;
  const void* a; int64_t a_gs, a_cs, a_rs;
  float* z;
  uint8_t* wide;
  void* zt;
  int32_t* zt_exp;
};
mm_status launch_lowrank_shrink_tiles(const LowRankArgs& l, const LowRankShrink* p, int problems, int64_t z_ld,
                                      const FusedTables* slots, const AdapterRows* sort, cudaStream_t stream);
// What follows the factors: the fused product Y = product (A B, 16-bit, no
// batch) + z b (NULL: none), whose z and slots were made before, and one
// or two gradients (`rows` sorted before), each out[g, c, r] from x (16-byte
// aligned rows) and zt; part holds lowrank_max_parts * C * R floats.
struct LowRankFused {
  GemmArgs product;
  const LowRankProduct* plan;
  const FusedLayout* layout;
  char* ws;
  const float* z;
  const void* b; int64_t b_gs, b_rs, b_ns;
};
struct LowRankOuter {
  const void* x; int64_t x_rs, C;
  const void* zt; const int32_t* zt_exp;
  void* out; int64_t o_cs, o_rs;
  float* part;
};
mm_status launch_lowrank_finish(const LowRankArgs& l, const LowRankFused* fused, const AdapterRows* rows,
                                const LowRankOuter* outer, int problems, int64_t z_ld, cudaStream_t stream);

}  // namespace qg
