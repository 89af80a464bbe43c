// TMA descriptors of the cache's pools (host side).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kv_internal.h"

namespace moe {
namespace kv {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// One layer's pools as [D / 64][rows][64], rows = n_pages * Hkv * page, with
// boxes of box_rows rows of all D columns: a box arrives as D / 64 blocks of
// box_rows rows of 128 bytes, 128-byte swizzle.
bool pool_maps(const Cache& c, CUtensorMap* k, CUtensorMap* v, int box_rows);

// The same pools as [rows][D] with boxes of box_rows rows of 64 columns.
bool pool_maps_2d(const Cache& c, CUtensorMap* k, CUtensorMap* v, int box_rows);

// A call's queries as [rows][Hq][D] with boxes of 64 columns of the G heads of
// tq rows: 128-byte rows, a token's heads in a row.
bool query_map(const Attn& a, int D, int n_rows, int tq, CUtensorMap* q);

}  // namespace kv
}  // namespace moe
