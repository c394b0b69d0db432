// The matrix plan: host description and device tables of the matrices of one
// flat buffer, shared by the Muon and Newton-Schulz translation units.
#pragma once

#include <vector>

#include "zds_internal.h"

namespace zds {

// Padding of a matrix's two sizes in the Newton-Schulz workspace, and the
// depth of a product's steps (elements of fp16).
constexpr int kNsDepth = 64;

// One matrix as the device code sees it. m <= n are its sizes with the
// smaller first (tall: rows > cols, so X is the transpose), mp and np the
// padded ones. Workspace offsets are in fp16 elements from the workspace's
// start; a second plane (the low halves) follows each array of an FP32 plan.
struct NsMatrix {
  int64_t offset;   // flat offset
  int32_t rows, cols;
  int32_t m, n, mp, np;
  int32_t tall;
  int32_t pair;           // of a BF16 plan: A and B have a plane of low halves, too
  int32_t part0, nparts;  // this matrix's partial sums of squares in the group's
  int32_t chunk;          // elements of one
  int64_t x[2];     // X of even and odd steps, mp x np
  int64_t lo;       // what X's fp16 values leave of X, mp x np (pair: of even and odd steps)
  int64_t a, b;     // A and B, mp x mp
};

// A block's piece of work: tile (ti, tj) of matrix `mat`, or chunk ti of it.
// Of a product's sum it takes part `part` of `parts` (1: all of it); `slot`
// numbers a launch's cut tiles.
struct NsTile {
  int32_t mat, ti, tj;
  uint8_t part, parts;
  uint16_t slot;
};

// The launch of one product: blocks first..first + count of the plan's tile
// array. `cut` more tiles, listed from `join` on, are summed in `parts` pieces
// (cut * parts blocks from `pieces` on).
struct NsList {
  int32_t tile, first, count, join, cut, parts, pieces;
};

// Matrices that go through one sequence of launches: X X^T, A A and B X; the
// conversion's 64 x 64 tiles over the padded matrices and the norm's chunks.
struct NsGroup {
  int32_t mat0, nmat;           // matrices in the plan's device array
  int32_t pair;                 // of a BF16 plan: some of them are NsMatrix::pair
  int32_t conv0, nconv, chunk0, nchunk;
  NsList gram, poly, full;
};

// A chunk of a matrix for zds_muon_apply: up to kApplyChunk elements from flat
// offset `first`, and the matrix's two scale factors (zds_muon_scale 1 and 2).
constexpr int kApplyChunk = 2048;
struct ApplyChunk {
  int64_t first;
  int32_t len;
  float aspect, rms;
  int32_t pad_;
};

}  // namespace zds

struct zds_matrix_plan {
  int device = 0;
  int32_t num = 0;
  int64_t first = 0, span = 0;  // the matrices lie in [first, span)
  std::vector<zds::NsGroup> groups[2];  // [FP32]
  // workspace of one group (the largest of all): partial sums and scales in
  // front, then the fp16 arrays
  size_t ws_bytes[2] = {0, 0};      // [FP32]
  int32_t max_parts = 0, max_mats = 0;
  int64_t piece_elems[2] = {0, 0};  // fp32 elements of cut tiles' pieces, the most of a launch
  int64_t arrays[2] = {0, 0};       // fp16 elements
  zds::NsMatrix *d_mats[2] = {nullptr, nullptr};  // [FP32]: workspace offsets differ
  zds::NsTile *d_tiles = nullptr;
  zds::ApplyChunk *d_chunks = nullptr;
  int64_t num_chunks = 0;
};

namespace zds {
// Tables of the Newton-Schulz groups into the plan (sizes already checked).
zds_status build_newton_schulz(zds_matrix_plan *p, const int64_t *offset, const int32_t *rows, const int32_t *cols,
                               int32_t num);
}  // namespace zds
