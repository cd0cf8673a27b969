// Interface of the 16-bit products (dense.cu): grouped by expert or dense, with their gradients.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace nvfp4moe {

struct WsHeader;

constexpr int kMaxGroups = 1024;       // experts of one grouped product (one thread each in the table kernel)

// D[i][j] = sum_r A[i][r] B[j][r], per segment (expert) e:
//   kMmForward  i: token rows of the segment, j: output features, r: input features
//               A = x [rows][R], B = w [E][J][R]
//   kMmDgrad    i: token rows, j: input features, r: output features
//               A = dy [rows][R], B = w [E][R][J]
//   kMmWgrad    i: output features, j: input features, r: token rows of the segment
//               A = dy [rows][I], B = x [rows][J], D = dw [E][I][J]
enum : int { kMmForward = 0, kMmDgrad = 1, kMmWgrad = 2 };

// The segments of a ragged call, written by launch_mm_table into the workspace.
struct MmTable {
  int32_t* seg;          // [E][2] first row, number of rows
  int32_t* tiles;        // [E + 1] row tiles before each segment
  CUtensorMap* maps;     // [E][2] wgrad's operands, rows of one segment (nullptr: not wanted)
};

// The operands of a ragged wgrad: A = dy [rows][I], B = x [rows][J].
struct MmWgradOperands {
  const void *a, *b;
  int I, J;
};

// What the table kernel builds the segments' maps from.
struct MmSegMaps {
  CUtensorMap a, b;      // of the operands' first rows
  const void *a_base, *b_base;
  int64_t a_row_bytes, b_row_bytes;
  CUtensorMap* out;      // nullptr: none
};

// How forward and dgrad run: on CTA pairs with tiles of up to tile_rows token rows (a multiple of 32 up
// to 256), or on single CTAs with tiles of tile_rows (16, 32, 64, 128), `split` CTAs or pairs sharing a tile's
// reduction.  J output columns, R the reduction length.
struct MmPlan {
  bool pair;
  int tile_rows;
  int split;
};
MmPlan mm_plan(int64_t rows, int E, int J, int R, bool ragged);
// In how many parts wgrad's pairs share the token rows (of each segment) of a tile.
int mm_wgrad_split(int64_t rows, int E, int I, int J);
// FP32 parts that workspaces hold for a dense row product and for wgrad: enough for every plan of up to `rows` rows,
// so that a workspace for many rows serves fewer (which are the ones that share tiles among more pairs).
size_t mm_row_part_floats(int64_t rows, int J, int R);
size_t mm_wgrad_part_floats(int64_t rows, int E, int I, int J);

struct MmArgs {
  const int32_t* seg;    // as in MmTable; nullptr: one segment, all `rows` rows
  const int32_t* tiles;
  const CUtensorMap* seg_maps;   // as MmTable.maps; nullptr with one segment
  int E;
  int64_t rows;          // token rows of the tensors
  int I;                 // kMmWgrad: rows of one expert's output
  int J;                 // output columns
  int R;                 // reduction length (not kMmWgrad)
  int fp16;              // operands FP16 (else BF16)
  void* out;
  int out_f32;           // out is FP32 (else the operands' type)
  const float* bias;     // [J] or nullptr
  int act;               // NVFP4MOE_ACT_*
  const void* residual;  // [rows][J] or nullptr, the operands' type
  void* z_out;           // [rows][J] or nullptr: the sums with the bias, before the activation
  uint32_t* status;
  uint64_t wait_ns;      // limit of each bounded wait, a millisecond at least
  int skip_loads;        // test hook: the CTA blockIdx.x + 1 that brings in no operands (0: none)
  int reset_status;      // The product is its call's first kernel: its first CTA clears the status word as it
                         // starts.  Another CTA can raise a bit a wait limit after its own start at the earliest
                         // (an exhausted wait is the only cause).
  int late_wait;         // The previous kernel of the stream is not one this product depends on, and has
                         // itself waited for those it does: it may run beside that kernel, and waits
                         // for it only before it ends (so that the kernel after it can wait for both).
                         // For products whose inputs all come by TMA (no bias, no residual): plain
                         // loads would see earlier kernels' writes only after the wait.
  int* work_counter;     // pairs; zero at launch: tiles handed out beyond the first of each CTA pair
                         // (nullptr: fixed turns, for tiles of one cost)
  MmPlan plan;           // forward, dgrad
  int split;             // pairs: parts of a tile's reduction (forward, dgrad: plan.split, dense calls only)
  float* parts;          // with split > 1: [split][rows][J], wgrad [split][E][I][J], the parts' sums; launch_mm_join
                         // then finishes the product
};

// Zeroes the status word and the work counters and, with offsets, checks them and writes the segment table for row
// tiles of tile_rows.  Offsets that decrease or leave 0 .. rows raise kStatusBadInput and leave
// every segment empty, so no later kernel of the call reads or writes through them.  w: also the
// segments' tensor maps for wgrad (rows > 0).
cudaError_t launch_mm_table(const int32_t* offsets, int E, int64_t rows, int tile_rows, const MmTable& t,
                            WsHeader* hdr, const MmWgradOperands* w, cudaStream_t stream);
// The product.  a, b: the operands' base addresses.
cudaError_t launch_mm(int mode, const void* a, const void* b, const MmArgs& m, cudaStream_t stream);
// Adds the parts of a product of split > 1 in their order and finishes it: epilogue, rounding, store.
cudaError_t launch_mm_join(int mode, const MmArgs& m, cudaStream_t stream);

// dz = dy act'(z) (16 bit, written when act is not NONE) and db[n] = sum_m dy act'(z) (FP32, when
// db is not nullptr; partials: act_grad_partials(M, N) * N floats).  Resets the workspace header as
// launch_mm_table does.
int act_grad_partials(int64_t M, int64_t N);
cudaError_t launch_act_grad(const void* dy, const void* z, int64_t M, int N, int act, bool fp16, void* dz, float* db,
                            float* partials, WsHeader* hdr, int32_t* launches, cudaStream_t stream);

// gemm.cu: tensor map of 2- or 4-byte elements [batch][rows][inner], a box of box_bytes (64 or 128, the
// swizzle's width too) x box_rows x 1.
int make_tma_3d(CUtensorMap* map, const void* base, uint32_t elem_bytes, uint64_t inner, uint64_t rows,
                uint64_t batch, uint32_t box_rows, uint32_t box_bytes);
inline int make_tma_16(CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows, uint64_t batch,
                       uint32_t box_rows) {
  return make_tma_3d(map, base, 2, inner, rows, batch, box_rows, 128);
}

}  // namespace nvfp4moe
